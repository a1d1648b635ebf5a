"""bf16 layer calls that take the GPU alone end in the order they were queued in: a call on
one stream follows the call before it on another, held up there, and its results are
the serial ones.  Other calls do not wait."""
import pytest
import torch

from tests.gpu_util import load_moe

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


@pytest.fixture(scope="module")
def moe():
    return load_moe()


def make(moe, seed=3, d=256, E=8, k=2, f=192, dt=BF):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def randn(*shape, std=1.0, dtype=dt):
        return (torch.randn(*shape, generator=g, device="cuda") * std).to(dtype)
    return moe.MoELayer(randn(E, d, std=d ** -0.5, dtype=torch.float32), randn(E, d, 2 * f, std=d ** -0.5),
                        randn(E, f, d, std=f ** -0.5), k), randn


def as_kind(stream, kind):
    return {"stream": stream, "external": torch.cuda.ExternalStream(stream.cuda_stream),
            "handle": stream.cuda_stream}[kind]


@pytest.mark.parametrize("kind", ["stream", "external", "handle"])
def test_a_call_follows_one_that_is_held_up(moe, kind):
    lay, randn = make(moe)
    other, _ = make(moe, 4)
    x, dout = randn(300, 256), randn(300, 256)
    want = lay(x), other(x)
    want = *want, lay.backward(x, dout)["x"], other.backward(x, dout)["x"]
    torch.cuda.synchronize()
    A, B = torch.cuda.Stream(), torch.cuda.Stream()
    for s in (A, B):
        s.wait_stream(torch.cuda.current_stream())
    outs = [torch.empty_like(x) for _ in range(2)]
    with torch.cuda.stream(A):
        torch.cuda._sleep(100_000_000)
    lay(x, outs[0], stream=as_kind(A, kind))
    first = A.record_event()
    other(x, outs[1], stream=as_kind(B, kind))
    with torch.cuda.stream(A):
        torch.cuda._sleep(100_000_000)
    ga = lay.backward(x, dout, stream=as_kind(A, kind))
    second = A.record_event()
    gb = other.backward(x, dout, stream=as_kind(B, kind))
    assert not first.query()  # (nothing above waited on the host)
    B.synchronize()
    assert first.query() and second.query()
    torch.cuda.synchronize()
    assert moe.moe_last_device_error() == moe.MOE_OK
    for a, b in zip(want, (*outs, ga["x"], gb["x"])):
        assert torch.equal(a, b)


def test_the_current_stream_and_a_capture(moe):
    lay, randn = make(moe)
    x = randn(300, 256)
    want = lay(x).clone()
    torch.cuda.synchronize()
    A, B = torch.cuda.Stream(), torch.cuda.Stream()
    out, graph = torch.empty_like(x), torch.cuda.CUDAGraph()
    for s in (A, B):
        s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(A):
        lay(x, out)  # allocates the workspace
        torch.cuda._sleep(100_000_000)
        lay(x, out)
    with torch.cuda.stream(B):
        lay(x, torch.empty_like(x))
        ended = B.record_event()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=A):  # waits for no call on B, which the graph knows nothing of
        lay(x, out)
    with torch.cuda.stream(B):
        lay(x, torch.empty_like(x))
    for _ in range(2):
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)
    assert ended.query()


@pytest.mark.parametrize("T,dt", [(300, torch.float32), (100, BF)])
def test_other_calls_do_not_wait(moe, T, dt):
    lay, randn = make(moe, dt=dt)
    x = randn(T, 256)
    want = lay(x).clone()
    A, B = torch.cuda.Stream(), torch.cuda.Stream()
    outs = [torch.empty_like(x) for _ in range(2)]
    for s, o in zip((A, B), outs):  # (workspaces)
        s.wait_stream(torch.cuda.current_stream())
        lay(x, o, stream=s)
    torch.cuda.synchronize()
    with torch.cuda.stream(A):
        torch.cuda._sleep(200_000_000)
    lay(x, outs[0], stream=A)
    held = A.record_event()
    lay(x, outs[1], stream=B)
    B.synchronize()
    assert not held.query()
    torch.cuda.synchronize()
    assert torch.equal(outs[0], want) and torch.equal(outs[1], want)
