"""Arrays of more than 2^31 elements: offsets past 31 bits in every operator.
The far end of each array is checked, where a wrapped offset would show.
Tolerances as in tests/test_gpu_backward.py and tests/test_gpu_clip.py."""
import pytest
import torch

from tests import backward_ref as ref
from tests.gpu_util import load_moe
from tests.test_gpu_backward import U32, UB, ftol, gen, nan, ok, randn

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


@pytest.fixture(scope="module")
def moe():
    return load_moe()


def rnd(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda", dtype=BF)


def test_permutations(moe):
    T, d, E, k = 150_001, 7168, 2, 2
    P = T * k
    assert P * d > 2 ** 31
    g = gen(1)
    idx = torch.randint(0, 2, (T, 1), generator=g, device="cuda")
    pos, _, _ = ref.permute(torch.cat([idx, 1 - idx], 1), E)
    w = torch.rand(T, k, generator=g, device="cuda")
    dout, y, dy, dw = rnd(g, T, d), rnd(g, P, d), nan(P, d, dtype=BF), nan(T, k)
    cfg = moe.config(T, d, E, k, 8, BF)
    moe.moe_combine_backward(cfg, dout, y, pos.int(), w, dy, dw)
    ok(moe)
    rows = pos.view(T, k)
    for part in (slice(0, 300), slice(T - 300, T)):
        want = (w[part, :, None] * dout[part].float()[:, None, :]).to(BF)
        assert torch.equal(dy[rows[part]], want)
        terms = dout[part].double()[:, None, :] * y[rows[part]].double()
        assert ((dw[part].double() - terms.sum(-1)).abs() <= (d / 32 + 16) * U32 * terms.abs().sum(-1)).all()
    dx, dw2 = dout.clone(), nan(T, k)
    cfg = moe.config(T, d, E, k, 8, BF, scale_inputs=True)
    moe.moe_dispatch_backward(cfg, y, pos.int(), w, dout, dx, dw2)
    ok(moe)
    part = slice(T - 300, T)
    r = y[rows[part]].double()
    want, mag = (r * w[part].double()[:, :, None]).sum(1), (r * w[part].double()[:, :, None]).abs().sum(1)
    tol = (k + 1) * U32 * mag
    assert ((dx[part].double() - want).abs() <= tol + UB * (want.abs() + tol)).all()


def test_experts(moe):
    counts, d, f = [399_900, 301, 77], 64, 2688
    P, E = sum(counts), len(counts)
    assert P * 2 * f > 2 ** 31
    g = gen(2)
    offsets = torch.tensor([0, counts[0], counts[0] + counts[1], P], dtype=torch.int32, device="cuda")
    x, dy, h = rnd(g, P, d), rnd(g, P, d), rnd(g, P, f)
    Wgu, Wd = rnd(g, E, d, 2 * f) / 8, rnd(g, E, f, d) / 51
    dx, dWgu, dWd = nan(P, d, dtype=BF), nan(E, d, 2 * f, dtype=BF), nan(E, f, d, dtype=BF)
    cfg = moe.config(P, d, E, 1, f, BF)
    ws = torch.empty(moe.moe_grouped_swiglu_backward_workspace_size(cfg), dtype=torch.uint8, device="cuda")
    moe.moe_grouped_swiglu_backward(cfg, x, offsets, Wgu, Wd, h, dy, dx, dWgu, dWd, ws)
    ok(moe)
    for e in (1, 2):  # the segments at the far end
        a, b = int(offsets[e]), int(offsets[e + 1])
        xe, dye, We, Wde = x[a:b].double(), dy[a:b].double(), Wgu[e].double(), Wd[e].double()
        rdx, rW = ref.grads(lambda p, q: ref.ffn_rows(p, [0, b - a], q[None], Wde[None]), [xe, We], dye)
        gu = (xe @ We).requires_grad_(True)
        yy = (gu[:, :f] * torch.sigmoid(gu[:, :f]) * gu[:, f:]) @ Wde
        dgu = torch.autograd.grad((yy * dye).sum(), gu)[0].abs()
        tol = ftol(rdx, d, d, 2 * f) + UB * (dgu @ We.abs().t() + rdx.abs())
        assert ((dx[a:b].double() - rdx).abs() <= tol).all()
        tol = ftol(rW, d, d, b - a) + UB * (xe.abs().t() @ dgu + rW.abs())
        assert ((dWgu[e].double() - rW).abs() <= tol).all()
        want = h[a:b].double().t() @ dye
        assert ((dWd[e].double() - want).abs() <= ftol(want, b - a) + UB * want.abs()).all()


def test_route(moe):
    T, d, E, k = 1_100_000, 64, 512, 2
    assert T * 4 * E > 2 ** 31
    g = gen(3)
    idx = torch.randint(0, E // 2, (T, 1), generator=g, device="cuda")
    idx = torch.cat([idx, idx + E // 2], 1)
    w = torch.rand(T, 1, generator=g, device="cuda")
    w = torch.cat([w, 1 - w], 1)
    x, Wr, dw = rnd(g, T, d), randn(g, E, d, std=0.125), randn(g, T, k)
    cfg = moe.config(T, d, E, k, 8, BF)
    ws = torch.empty(moe.moe_route_backward_workspace_size(cfg), dtype=torch.uint8, device="cuda")
    dL, dWr, db, dx = nan(T, E), nan(E, d), nan(E), nan(T, d, dtype=BF)
    moe.moe_route_backward(cfg, x, Wr, None, idx.int(), w, dw, None, dL, dWr, db, dx, ws)
    ok(moe)
    S = (w.double() * dw.double()).sum(-1, keepdim=True)
    want = w.double() * (dw.double() - S)
    got = dL.gather(1, idx).double()
    tol = (k + 32) * 2.0 ** -23 * ((w.double() * dw.double()).abs().sum(-1, keepdim=True)
                                   + dw.double().abs().amax(-1, keepdim=True))
    assert ((got - want).abs() <= tol).all()
    part = slice(T - 500, T)
    rdx = dL[part].double() @ Wr.double()
    tol = ftol(rdx, E) + UB * rdx.abs() + 2.0 ** -16 * rdx.abs().max()
    assert ((dx[part].double() - rdx).abs() <= tol).all()
    rW = torch.zeros(E, d, dtype=torch.float64, device="cuda")
    for j in range(k):
        rW.index_add_(0, idx[:, j], got[:, j:j + 1] * x.double())
    assert (dWr.double() - rW).abs().max() <= ftol(rW, T)
    rb = torch.zeros(E, dtype=torch.float64, device="cuda").index_add_(0, idx.reshape(-1), got.reshape(-1))
    assert (db.double() - rb).abs().max() <= ftol(rb, T) + 1e-6 * U32


def test_clip(moe):
    n = 2 ** 31 + 12345
    g = torch.zeros(n, device="cuda", dtype=BF)
    g[:1000], g[-1000:] = 3.0, 4.0
    out = torch.full_like(g, 9.0)
    norm = torch.zeros(1, device="cuda")
    ws = torch.empty(moe.moe_clip_grad_norm_workspace_size(), dtype=torch.uint8, device="cuda")
    moe.moe_clip_grad_norm(moe.grad_list([g], [out]), 1.0, norm, ws)
    ok(moe)
    want = (25_000.0) ** 0.5
    assert abs(float(norm) - want) <= 34 * U32 * want
    for part, v in ((slice(0, 1000), 3.0), (slice(n - 1000, n), 4.0)):
        assert ((out[part].double() - v / want).abs() <= 2 * UB * v / want).all()
    assert int((out[1000:n - 1000] != 0).sum()) == 0
