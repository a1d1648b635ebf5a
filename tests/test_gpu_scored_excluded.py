"""Experts excluded by a bias of -inf: whole groups of them, all but one of a group, more than
the choice leaves over; ids and weights against 64 bits, in both kernels."""
import pytest
import torch

from tests import scored_ref
from tests.gpu_util import load_moe
from tests.test_gpu_scored_route import check, rng, route

pytestmark = pytest.mark.gpu
INF = float("inf")


@pytest.fixture(scope="module")
def moe():
    return load_moe()


def masks(E, G):
    """Excluded experts of each case."""
    n = E // G
    ids = torch.arange(E)
    yield "one group", ids < n
    yield "every other group", ids // n % 2 == 0
    yield "all but one expert of a group", (ids < n) & (ids != n // 2)
    yield "all but two groups", ids // n >= 2
    yield "all but one group", ids // n != G - 1
    yield "all groups but for an expert each", ids % n != 1
    yield "all but two experts of each group", ids % n >= 2


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("top2", [False, True])
@pytest.mark.parametrize("E,k,G,Gk", [(64, 2, 8, 4), (128, 4, 4, 2), (256, 3, 8, 4), (160, 2, 5, 2), (96, 4, 32, 9),
                                      (12, 2, 6, 3)])
def test_short_batches(moe, E, k, G, Gk, top2, score):
    g = rng(E + G)
    L = torch.randn(12, E, generator=g)
    L[3] = 0.25
    L[4, ::2] = -INF
    for name, out in masks(E, G):
        bias = torch.randint(-100, 101, (E,), generator=g).float() * 1e-3
        bias[out] = -INF
        check(moe, L, bias, k, score, G, Gk, top2)
        bias[~out] = 0.0
        check(moe, L, bias, k, score, G, Gk, top2)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("top2", [False, True])
@pytest.mark.parametrize("T,E,k,G,Gk", [(4100, 128, 4, 4, 2), (4100, 64, 2, 8, 4), (33000, 256, 8, 8, 4),
                                        (5000, 256, 8, 8, 4)])
def test_long_batches(moe, T, E, k, G, Gk, top2, score):
    g = rng(T)
    L = torch.randn(T, E, generator=g)
    for name, out in masks(E, G):
        bias = torch.randint(-100, 101, (E,), generator=g).float() * 1e-3
        bias[out] = -INF
        idx, w = route(moe, L.cuda(), bias.cuda(), k, moe.router(score, G, Gk, "top2" if top2 else "max"))
        torch.cuda.synchronize()
        assert moe.moe_last_device_error() == moe.MOE_OK
        assert torch.isfinite(w).all()
        idx = idx.cpu()
        if name in ("one group", "every other group"):  # (enough experts stay)
            want = scored_ref.select_many(L.cuda(), bias.cuda(), k, score == "sigmoid", G, Gk, top2).cpu()
            assert torch.equal(idx.long(), want), name
        for t in range(0, T, T // 12):
            assert idx[t].tolist() == scored_ref.select(L[t].numpy(), bias.numpy(), k, score == "sigmoid", G, Gk,
                                                        top2), (name, t)
