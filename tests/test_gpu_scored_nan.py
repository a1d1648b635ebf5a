"""A NaN logit under softmax scores: every score of its token is a NaN, so its weights
are, renormalised or not, whatever was chosen; the ids are those of the definition
(NaN below every number, equal ones by id), and the other tokens see nothing of it."""
import numpy as np
import pytest
import torch

from tests import scored_ref
from tests.gpu_util import load_moe

pytestmark = pytest.mark.gpu
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module")
def moe():
    return load_moe()


@pytest.mark.parametrize("kind", ["none", "steps"])
@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("G,Gk,top2", [(1, 1, False), (4, 2, False), (4, 2, True)])
@pytest.mark.parametrize("T,E,k", [(40, 64, 8), (4100, 64, 8), (4100, 128, 8), (4100, 256, 5),
                                   (40, 256, 8), (40, 20, 3), (40, 36, 6), (40, 1000, 32)])
def test_a_nan_logit(moe, T, E, k, G, Gk, top2, renorm, kind):
    g = torch.Generator().manual_seed(T + E + k)
    L = torch.randn(T, E, generator=g)
    bias = None if kind == "none" else torch.randint(-100, 101, (E,), generator=g).float() * 1e-3
    plain = L.clone()
    L[3, 3] = NAN                   # one, seldom among the chosen
    L[5, E - 1] = NAN               # the last
    L[6, L[6].argmax()] = NAN       # in the place of the largest
    L[8] = NAN
    L[9] = -INF
    L[9, 2] = NAN                   # beside no other score
    L[11, ::2] = NAN
    L[T - 1, 1] = NAN
    bad = [3, 5, 6, 8, 9, 11, T - 1]
    cfg = moe.config(T, 8, E, k, 8, renormalize=renorm)
    r = moe.router("softmax", G, Gk, "top2" if top2 else "max", 1.5)
    out = []
    for x in (L, plain):
        idx = torch.full((T, k), -7, dtype=torch.int32, device="cuda")
        w = torch.full((T, k), 9.0, device="cuda")
        moe.moe_route_scored_from_logits(cfg, r, x.cuda(), None if bias is None else bias.cuda(), idx, w)
        out.append((idx, w))
    torch.cuda.synchronize()
    assert moe.moe_last_device_error() == moe.MOE_OK
    (idx, w), (idx0, w0) = out
    for t in bad:
        want = scored_ref.select(L[t].numpy(), None if bias is None else bias.numpy(), k, False, G, Gk, top2)
        assert idx[t].tolist() == want, t
    assert torch.isnan(w[bad]).all()
    others = torch.ones(T, dtype=torch.bool)
    others[bad] = False
    assert torch.equal(idx[others], idx0[others]) and torch.equal(w[others], w0[others])
    assert np.isfinite(w0.cpu().numpy()).all()
