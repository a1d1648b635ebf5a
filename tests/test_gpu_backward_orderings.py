"""The two orders in which the experts' gradient launches its products (weight
products beside the row products while the weights fit in L2, one after another
beyond), in each tile mode, alone and in the whole layer; and two gradients in
flight on two streams.  References and tolerances as in tests/test_gpu_backward.py."""
import pytest
import torch

from tests import test_gpu_backward as small
from tests.gpu_util import load_moe
from tests.test_gpu_backward import check_experts, gen, ok, randn

pytestmark = pytest.mark.gpu
F32, BF = torch.float32, torch.bfloat16


@pytest.fixture(scope="module")
def moe():
    return load_moe()


LARGE = {  # rows of each expert, d, f: the weights' 6 E d f bytes past 128 MB
    "pairs": ([600, 513, 700, 540], 2056, 2744),
    "hybrid": ([300, 90, 0, 257, 128, 40], 2048, 2056),
    "singles": ([20, 0, 9, 33] * 8, 1024, 768),
    "split": ([3, 0, 64, 17], 2048, 2816),
}


@pytest.mark.parametrize("mode", LARGE)
def test_experts_with_large_weights(moe, mode):
    counts, d, f = LARGE[mode]
    assert 6 * len(counts) * d * f > 128 << 20
    check_experts(moe, counts, d, f, BF, seed=21)


@pytest.mark.parametrize("T,d,E,k,f,renorm,scale", [
    (1100, 2048, 4, 2, 2816, True, False),    # pairs
    (150, 2048, 4, 2, 2816, False, False),    # both tile shapes
    (80, 1024, 32, 4, 768, True, True),       # single CTAs
    (20, 2048, 4, 2, 2816, True, False)])     # clusters that share a tile
def test_layer_with_large_weights(moe, T, d, E, k, f, renorm, scale):
    assert 6 * E * d * f > 128 << 20
    small.test_layer_backward(moe, T, d, E, k, f, BF, renorm, scale, True)


@pytest.mark.parametrize("T,d,E,k,f,dtype,renorm", [
    (2048, 256, 64, 4, 256, BF, True),        # both tile shapes, products side by side
    (60, 2048, 8, 2, 768, BF, True),          # clusters that share a tile
    (150, 2048, 4, 2, 2816, BF, False),       # large weights
    (1024, 512, 64, 4, 256, F32, False)])     # dWr beside dx
def test_two_streams_at_once(moe, T, d, E, k, f, dtype, renorm):
    g = gen(T + E)
    lay = moe.MoELayer(randn(g, E, d, std=d ** -0.5), randn(g, E, d, 2 * f, std=d ** -0.5, dtype=dtype),
                       randn(g, E, f, d, std=f ** -0.5, dtype=dtype), k, None, renorm)
    batches = [(randn(g, T, d, dtype=dtype), randn(g, T, d, dtype=dtype)) for _ in range(2)]
    want = []
    for x, dout in batches:
        out = lay(x)
        want.append({"out": out, **lay.backward(x, dout)})
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = [{n: torch.full_like(t, float("nan")) for n, t in w.items()} for w in want]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    for _ in range(4):  # interleaved, so the two streams' kernels overlap
        for s, (x, dout), r in zip(streams, batches, got):
            lay.forward(x, r["out"], stream=s)
            lay.backward(x, dout, r, stream=s)
    ok(moe)
    for r, w in zip(got, want):
        for n in w:
            assert torch.equal(r[n], w[n]), n
