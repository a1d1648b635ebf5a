"""Scored routing of long batches (several tokens a warp), and of batches just below
the length from which it is taken: every token's choice equal to that of 64 bits,
weights as in test_gpu_scored_route.py."""
import pytest
import torch

from tests import scored_ref
from tests.gpu_util import load_moe

pytestmark = pytest.mark.gpu
EPS = 2.0 ** -23


@pytest.fixture(scope="module")
def moe():
    return load_moe()


def check(moe, L, bias, k, score, G=1, Gk=1, top2=False, renorm=True, scale=1.0):
    T, E = L.shape
    r = moe.router(score, G, Gk, "top2" if top2 else "max", scale)
    idx = torch.full((T + 3, k), -7, dtype=torch.int32, device="cuda")
    w = torch.full((T + 3, k), -7.0, device="cuda")
    moe.moe_route_scored_from_logits(moe.config(T, 8, E, k, 8, renormalize=renorm), r, L, bias, idx, w)
    torch.cuda.synchronize()
    assert moe.moe_last_device_error() == moe.MOE_OK
    assert (idx[T:] == -7).all() and (w[T:] == -7).all()  # behind the last token
    want = scored_ref.select_many(L, bias, k, score == "sigmoid", G, Gk, top2)
    bad = (idx[:T] != want).any(-1).nonzero().view(-1)
    assert not len(bad), (len(bad), bad[:5].tolist(), idx[bad[0]].tolist(), want[bad[0]].tolist())
    ref = scored_ref.weights(L.double(), want, score == "sigmoid", renorm, scale)
    span = 0.0 if score == "sigmoid" else float(L.max() - L.min())
    assert ((w[:T].double() - ref).abs() <= (24 + -(-E // 32) + 2 * span) * EPS * ref.abs() + 2.0 ** -126).all()


def logits(T, E, seed, spread=1.5):
    return torch.randn(T, E, generator=torch.Generator(device="cuda").manual_seed(seed), device="cuda") * spread


def steps_bias(E, seed):
    g = torch.Generator().manual_seed(seed)
    return (torch.randint(-100, 101, (E,), generator=g).float() * 1e-3).cuda()


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("biased", [False, True])
@pytest.mark.parametrize("E", [32, 36, 60, 64, 68, 128, 132, 200, 256, 260])
@pytest.mark.parametrize("T,k", [(4095, 8), (4096, 8), (4097, 1), (9001, 5)])
def test_without_groups(moe, T, k, E, biased, score):
    check(moe, logits(T, E, T + E), steps_bias(E, E) if biased else None, k, score,
          renorm=E % 8 == 0, scale=2.5)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("biased,top2", [(False, False), (False, True), (True, False), (True, True)])
@pytest.mark.parametrize("T,E,k,G,Gk", [
    (4097, 32, 4, 8, 4), (5000, 64, 8, 8, 3), (4500, 128, 8, 4, 2), (4099, 128, 6, 8, 5),
    (4096, 128, 8, 2, 1), (16385, 256, 8, 8, 4), (16384, 256, 8, 4, 3), (17001, 256, 2, 8, 1),
    (32768, 256, 8, 8, 4), (33001, 256, 8, 4, 3), (32769, 256, 2, 8, 1), (32790, 160, 8, 8, 4),
    (4097, 96, 4, 8, 4), (5003, 160, 6, 8, 3), (16390, 160, 8, 8, 4), (16384, 256, 8, 16, 8),
    (4096, 64, 8, 1, 1)])
def test_with_groups(moe, T, E, k, G, Gk, biased, top2, score):
    check(moe, logits(T, E, T + G), steps_bias(E, E) if biased else None, k, score, G, Gk, top2,
          renorm=k > 4, scale=1.0)


@pytest.mark.parametrize("E,G,Gk", [(64, 1, 1), (128, 1, 1), (256, 1, 1), (128, 8, 4)])
def test_values_too_near_and_ties(moe, E, G, Gk):
    """Tokens that fp32 cannot rank among others: logits steps of 2^-20 apart, of
    few distinct values, and equal ones (a padded batch)."""
    T = 4100
    L = logits(T, E, 3)
    g = torch.Generator(device="cuda").manual_seed(1)
    steps = torch.rand(T // 3 + 1, E, generator=g, device="cuda").argsort(-1).float()
    L[::3] = 1.0 + steps[:len(L[::3])] * 2.0 ** -20
    L[1::3] = (L[1::3] * 2).round() / 2
    L[5::9] = 0.0
    for bias in (torch.zeros(E, device="cuda"), steps_bias(E, 2), None):
        # (equal logits with biases that make equal group sums in real numbers: only
        # with the rounding of the sums do they differ, which need not be torch's)
        top2 = G > 1 and bias is not None and not bias.any()
        check(moe, L, bias, 8, "sigmoid", G, Gk, top2)


@pytest.mark.parametrize("E", [64, 128, 256])
def test_masked_and_nan_logits(moe, E):
    """-inf, the type's lowest value and NaN in some tokens of a warp, against the
    same tokens in a short batch (another kernel)."""
    T = 4099
    L = logits(T, E, 4)
    L[::5, ::2] = float("-inf")
    L[7] = float("-inf")
    L[11] = torch.finfo(torch.float32).min
    L[13, 3] = float("nan")
    L[14] = float("nan")
    for score in ("softmax", "sigmoid"):
        for bias in (None, steps_bias(E, 5)):
            for renorm in (True, False):
                r, out = moe.router(score), []
                for n in (T, 40):
                    idx = torch.empty(n, 8, dtype=torch.int32, device="cuda")
                    w = torch.empty(n, 8, device="cuda")
                    moe.moe_route_scored_from_logits(moe.config(n, 8, E, 8, 8, renormalize=renorm), r,
                                                     L[:n], bias, idx, w)
                    out.append((idx[:40], w[:40]))
                assert torch.equal(out[0][0], out[1][0])
                a, b = out[0][1], out[1][1]
                assert torch.equal(torch.isnan(a), torch.isnan(b))
                assert ((a - b).abs() <= 64 * EPS * b.abs()).logical_or(torch.isnan(a)).all()
                assert not a[7].any()  # no expert at all: weights of zero


def test_captured_long_batch(moe):
    T, E = 6000, 128
    L, bias = logits(T, E, 6), steps_bias(E, 6)
    cfg, r = moe.config(T, 8, E, 8, 8), moe.router("sigmoid")
    idx, w = torch.empty(T, 8, dtype=torch.int32, device="cuda"), torch.empty(T, 8, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        moe.moe_route_scored_from_logits(cfg, r, L, bias, idx, w)
    for seed in (7, 8):
        L.copy_(logits(T, E, seed))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(idx.long(), scored_ref.select_many(L, bias, 8, True, 1, 1, False))


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("kind", ["none", "zero", "steps"])
@pytest.mark.parametrize("T,E,k,G,Gk", [(300, 256, 8, 1, 1), (4200, 256, 8, 8, 4), (5000, 128, 8, 1, 1),
                                        (300, 1000, 32, 1, 1), (300, 1000, 31, 20, 9), (4100, 60, 3, 1, 1),
                                        (300, 33, 32, 1, 1), (300, 40, 5, 2, 1)])
def test_padded_batches(moe, T, E, k, G, Gk, kind, score):
    """Rows of equal logits, as tokens of zeros give: nothing but ties, which go to
    the lowest ids, or the bias alone decides."""
    L = logits(T, E, T + E)
    L[T // 3:T // 2] = 0.0
    L[T // 2:T // 2 + 20] = -0.0
    L[T - 20:] = 1.75
    L[T - 40:T - 20, ::2] = L[T - 40:T - 20, 1:2]
    bias = {"none": None, "zero": torch.zeros(E, device="cuda"), "steps": steps_bias(E, E)}[kind]
    check(moe, L, bias, k, score, G, Gk, kind != "none")
