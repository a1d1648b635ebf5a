"""MoELayer called with a stream that is not the current one: the memory it
allocates belongs to that stream's pool, and the results are the serial ones,
bit for bit, while the batch grows and dropped tensors are allocated over."""
import pytest
import torch

from tests.gpu_util import load_moe

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


@pytest.fixture(scope="module")
def moe():
    return load_moe()


def make(moe, d=256, E=8, k=2, f=192, seed=3):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def randn(*shape, std=1.0, dtype=BF):
        return (torch.randn(*shape, generator=g, device="cuda") * std).to(dtype)
    return moe.MoELayer(randn(E, d, std=d ** -0.5, dtype=torch.float32), randn(E, d, 2 * f, std=d ** -0.5),
                        randn(E, f, d, std=f ** -0.5), k), randn


def pool_of(t):
    """Handle of the stream whose pool t's memory comes from."""
    for seg in torch.cuda.memory_snapshot():
        if seg["address"] <= t.data_ptr() < seg["address"] + seg["total_size"]:
            return seg["stream"]
    raise AssertionError("not the caching allocator's memory")


@pytest.mark.parametrize("raw", [False, True], ids=["stream", "handle"])
def test_memory_belongs_to_the_stream(moe, raw):
    lay, randn = make(moe)
    x, dout = randn(300, 256), randn(300, 256)
    side = torch.cuda.Stream()
    arg = side.cuda_stream if raw else side
    here = torch.cuda.current_stream().cuda_stream
    assert here != side.cuda_stream
    side.wait_stream(torch.cuda.current_stream())
    out = lay.forward(x, stream=arg)
    grads = lay.backward(x, dout, stream=arg)
    for t in (out, lay.workspace(300, arg), lay._bwd_ws[side.cuda_stream], *grads.values()):
        assert pool_of(t) == side.cuda_stream
    assert pool_of(lay.workspace(300)) == here  # the current stream has its own
    side.synchronize()
    assert moe.moe_last_device_error() == moe.MOE_OK


def test_growing_batches_equal_the_serial_ones(moe):
    lay, randn = make(moe)
    batches = [(randn(T, 256), randn(T, 256)) for T in (40, 700, 90, 2500)]
    want = []
    for x, dout in batches:
        out = lay(x)
        want.append((out, lay.backward(x, dout)))
    torch.cuda.synchronize()
    side, results = torch.cuda.Stream(), []
    side.wait_stream(torch.cuda.current_stream())
    for x, dout in batches:
        x, dout = x.clone(), dout.clone()
        side.wait_stream(torch.cuda.current_stream())
        out = lay.forward(x, stream=side)
        results.append((out, lay.backward(x, dout, stream=side)))
        # dropped here while `side` may still read them; the current stream's
        # next tensors must not take their place before it has
        shape = x.shape
        del x, dout
        for _ in range(4):
            torch.full(shape, float("nan"), device="cuda", dtype=BF)
    side.synchronize()
    assert moe.moe_last_device_error() == moe.MOE_OK
    for (out, grads), (wout, wgrads) in zip(results, want):
        assert torch.equal(out, wout)
        for n in wgrads:
            assert torch.equal(grads[n], wgrads[n]), n


def test_a_graph_after_a_longer_batch(moe):
    """The graph's workspaces are replaced for later calls, not taken from it."""
    lay, randn = make(moe)
    x, dout, out = randn(300, 256), randn(300, 256), torch.empty(300, 256, device="cuda", dtype=BF)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        lay(x, out)
        got = lay.backward(x, dout)  # workspaces from before the capture, as a warm-up leaves them
    side.synchronize()
    want = {"out": out.clone(), **{n: t.clone() for n, t in got.items()}}
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        lay(x, out)
        lay.backward(x, dout, got)
    x2, dout2 = randn(2500, 256), randn(2500, 256)
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        lay(x2)
        lay.backward(x2, dout2)
        for n in (1 << 20, 1 << 22, 1 << 24):  # what a freed workspace's block would go to
            torch.full((n,), float("nan"), device="cuda")
    side.synchronize()
    out.zero_()
    for t in got.values():
        t.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert moe.moe_last_device_error() == moe.MOE_OK
    for n, t in {"out": out, **got}.items():
        assert torch.equal(t, want[n]), n
