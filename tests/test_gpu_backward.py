"""Parity of the backward pass: every gradient entry against a plain 64-bit
implementation of the forward step it differentiates (tests/backward_ref.py),
by automatic differentiation and by central differences.

Tolerances, all fixed by the arithmetic (u32 = 2^-24, ub = 2^-8 the unit
roundoffs of fp32 and bf16):
- a product of two fp32 values rounded once (dy_perm): equal, bit for bit;
- a dot product of n terms summed by 32 lanes in vectors of 16 bytes and then
  across lanes: the longest chain of additions is n/32 + 8 + 5, so the error
  is at most (n/32 + 16) u32 sum|terms|; sums over k slots: k u32 sum|terms|;
- matrix products in series: the rounding model 8 u32 (sum of sqrt n) max|ref|
  of tests/gpu_util.py; with bf16 activations also ub |ref| for the output's
  rounding and, where dgu (rounded to bf16) is an operand, ub sum|dgu| |other|.
"""
import numpy as np
import pytest
import torch

from tests import backward_ref as ref
from tests.gpu_util import fp32_tolerance, load_moe

pytestmark = pytest.mark.gpu

U32, UB = 2.0 ** -24, 2.0 ** -8
DTYPES = [torch.bfloat16, torch.float32]


@pytest.fixture(scope="module")
def moe():
    return load_moe()


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def randn(g, *shape, std=1.0, dtype=torch.float32):
    return (torch.randn(*shape, generator=g, device="cuda") * std).to(dtype)


def nan(*shape, dtype=torch.float32):
    return torch.full(shape, float("nan"), device="cuda", dtype=dtype)


def routing(g, T, E, k, skew=0.0):
    """Distinct experts per token; skew > 0 empties the high expert ids."""
    L = randn(g, T, E) - skew * torch.arange(E, device="cuda").float()
    idx = torch.sort(L, dim=-1, descending=True, stable=True).indices[:, :k].contiguous()
    return L, idx


def ok(moe):
    torch.cuda.synchronize()
    assert moe.moe_last_device_error() == moe.MOE_OK


def ftol(t, *lengths):
    return fp32_tolerance(t.detach().cpu().numpy(), *lengths)


# ------------------------------ permutations -------------------------------
SHAPES = [(1, 8, 1, 1), (1, 2880, 128, 4), (3, 72, 5, 5), (37, 1000, 16, 4), (300, 4096, 8, 2),
          (129, 520, 64, 32), (1025, 264, 12, 6), (2000, 2048, 128, 8)]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("T,d,E,k", SHAPES)
def test_combine_backward(moe, T, d, E, k, dtype):
    g = gen(T + d)
    _, idx = routing(g, T, E, k)
    pos, _, _ = ref.permute(idx, E)
    w = torch.rand(T, k, generator=g, device="cuda")
    dout, y = randn(g, T, d, dtype=dtype), randn(g, T * k, d, dtype=dtype)
    dy, dw = nan(T * k, d, dtype=dtype), nan(T, k)
    cfg = moe.config(T, d, E, k, 8, dtype)
    moe.moe_combine_backward(cfg, dout, y, pos.int(), w, dy, dw)
    ok(moe)
    rows = pos.view(T, k)
    want = nan(T * k, d, dtype=dtype)
    want[pos] = (w[:, :, None] * dout.float()[:, None, :]).view(T * k, d).to(dtype)
    assert torch.equal(dy, want)
    terms = dout.double()[:, None, :] * y.double()[rows]
    assert ((dw.double() - terms.sum(-1)).abs() <= (d / 32 + 16) * U32 * terms.abs().sum(-1)).all()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("T,d,E,k", SHAPES)
def test_combine_backward_unweighted(moe, T, d, E, k, dtype):
    g = gen(T + d + 1)
    pos, _, order = ref.permute(routing(g, T, E, k)[1], E)
    dout, dy = randn(g, T, d, dtype=dtype), nan(T * k, d, dtype=dtype)
    cfg = moe.config(T, d, E, k, 8, dtype, scale_inputs=True)
    moe.moe_combine_backward(cfg, dout, None, pos.int(), None, dy, None)
    ok(moe)
    assert torch.equal(dy, dout[order // k])


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("scale", [False, True])
@pytest.mark.parametrize("T,d,E,k", SHAPES)
def test_dispatch_backward(moe, T, d, E, k, dtype, scale):
    g = gen(T + d + 2)
    pos, _, _ = ref.permute(routing(g, T, E, k)[1], E)
    w = torch.rand(T, k, generator=g, device="cuda")
    x, dxp = randn(g, T, d, dtype=dtype), randn(g, T * k, d, dtype=dtype)
    dx, dw = nan(T, d, dtype=dtype), nan(T, k)
    cfg = moe.config(T, d, E, k, 8, dtype, scale_inputs=scale)
    moe.moe_dispatch_backward(cfg, dxp, pos.int(), w if scale else None, x if scale else None, dx,
                              dw if scale else None)
    ok(moe)
    rows = dxp.double()[pos.view(T, k)]
    terms = rows * w.double()[:, :, None] if scale else rows
    want = terms.sum(1)
    tol = (k + 1) * U32 * terms.abs().sum(1)
    if dtype == torch.bfloat16:
        tol = tol + UB * (want.abs() + tol)
    assert ((dx.double() - want).abs() <= tol + 1e-30).all()
    if scale:
        t = x.double()[:, None, :] * rows
        assert ((dw.double() - t.sum(-1)).abs() <= (d / 32 + 16) * U32 * t.abs().sum(-1)).all()


@pytest.mark.parametrize("dtype", DTYPES)
def test_dropped_pairs_have_no_gradient(moe, dtype):
    """A pair without a row (pos -1): its weight gradient is zero and no row
    is written for it; a token with no rows at all has a zero gradient."""
    T, d, E, k = 70, 136, 6, 3
    g = gen(11)
    pos, _, _ = ref.permute(routing(g, T, E, k)[1], E)
    pos = pos.clone()
    gone = [0, 1, 2, 50, 119]  # token 0 whole, then single slots
    lost = pos[gone].tolist()
    pos[gone] = -1
    w = torch.rand(T, k, generator=g, device="cuda")
    dout, y = randn(g, T, d, dtype=dtype), randn(g, T * k, d, dtype=dtype)
    y[lost] = float("nan")  # rows that nobody may read
    dy, dw = torch.full((T * k, d), 7.0, device="cuda", dtype=dtype), nan(T, k)
    cfg = moe.config(T, d, E, k, 8, dtype)
    moe.moe_combine_backward(cfg, dout, y, pos.int(), w, dy, dw)
    ok(moe)
    assert (dy[lost] == 7.0).all() and (dw.view(-1)[gone] == 0).all()
    assert torch.isfinite(dw).all() and torch.isfinite(dy.float()).all()
    for scale in (False, True):
        dx, dw = nan(T, d, dtype=dtype), nan(T, k)
        cfg = moe.config(T, d, E, k, 8, dtype, scale_inputs=scale)
        moe.moe_dispatch_backward(cfg, y, pos.int(), w, dout, dx, dw)
        ok(moe)
        assert (dx[0] == 0).all() and torch.isfinite(dx.float()).all()
        if scale:
            assert (dw.view(-1)[gone] == 0).all() and torch.isfinite(dw).all()


# -------------------------------- experts ----------------------------------
def run_experts(moe, cfg, offsets, x, Wgu, Wd, h, dy):
    P, d = x.shape
    off = torch.tensor(offsets, dtype=torch.int32, device="cuda")
    dx, dWgu, dWd = nan(P, d, dtype=x.dtype), nan(*Wgu.shape, dtype=x.dtype), nan(*Wd.shape, dtype=x.dtype)
    n = moe.moe_grouped_swiglu_backward_workspace_size(cfg)
    ws = torch.full((n,), 255, dtype=torch.uint8, device="cuda")  # NaN scratch
    moe.moe_grouped_swiglu_backward(cfg, x, off, Wgu, Wd, h, dy, dx, dWgu, dWd, ws)
    ok(moe)
    return dx, dWgu, dWd


def experts_case(seed, counts, d, f, dtype):
    g = gen(seed)
    E, P = len(counts), sum(counts)
    offsets = [0] + list(np.cumsum(counts))
    x, dy = randn(g, P, d, dtype=dtype), randn(g, P, d, std=0.05, dtype=dtype)
    Wgu = randn(g, E, d, 2 * f, std=d ** -0.5, dtype=dtype)
    Wd = randn(g, E, f, d, std=f ** -0.5, dtype=dtype)
    h = torch.empty(P, f, device="cuda", dtype=dtype)
    for e in range(E):
        gu = x[offsets[e]:offsets[e + 1]].double() @ Wgu[e].double()
        h[offsets[e]:offsets[e + 1]] = (gu[:, :f] * torch.sigmoid(gu[:, :f]) * gu[:, f:]).to(dtype)
    return [int(o) for o in offsets], x, Wgu, Wd, h, dy


def check_experts(moe, counts, d, f, dtype, seed=5):
    """P = T*k rows in the given segments (T = P, k = 1)."""
    offsets, x, Wgu, Wd, h, dy = experts_case(seed, counts, d, f, dtype)
    E, P = len(counts), sum(counts)
    cfg = moe.config(P, d, E, 1, f, dtype)
    dx, dWgu, dWd = run_experts(moe, cfg, offsets, x, Wgu, Wd, h, dy)
    xd, Wgud, Wdd, hd, dyd = (t.double() for t in (x, Wgu, Wd, h, dy))
    bf = dtype == torch.bfloat16
    rdx, rWgu = ref.grads(lambda a, b: ref.ffn_rows(a, offsets, b, Wdd), [xd, Wgud], dyd)
    for e in range(E):
        a, b = offsets[e], offsets[e + 1]
        want = hd[a:b].t() @ dyd[a:b]
        tol = ftol(want, max(1, b - a)) + (UB * want.abs() if bf else 0)
        assert ((dWd[e].double() - want).abs() <= tol).all(), ("dWd", e)
        if b == a:
            assert (dWgu[e] == 0).all() and (dWd[e] == 0).all()
            continue
        spread_x = spread_w = 0.0
        if bf:  # dgu's rounding: ub |dgu| through both products
            gu = xd[a:b] @ Wgud[e]
            leaf = gu.detach().requires_grad_(True)
            y = (leaf[:, :f] * torch.sigmoid(leaf[:, :f]) * leaf[:, f:]) @ Wdd[e]
            dgu = torch.autograd.grad((y * dyd[a:b]).sum(), leaf)[0].abs()
            spread_x = UB * (dgu @ Wgud[e].abs().t() + rdx[a:b].abs())
            spread_w = UB * (xd[a:b].abs().t() @ dgu + rWgu[e].abs())
        tol = ftol(rdx[a:b], d, d, 2 * f) + spread_x
        assert ((dx[a:b].double() - rdx[a:b]).abs() <= tol).all(), ("dx", e)
        tol = ftol(rWgu[e], d, d, b - a) + spread_w
        assert ((dWgu[e].double() - rWgu[e]).abs() <= tol).all(), ("dWgu", e)


COUNTS = [
    [1],                                  # one row in all
    [0, 1, 0],                            # experts without rows around one row
    [15, 16, 17, 31, 32, 33, 63, 64, 65],  # around the K steps of the weight gradients
    [0, 130, 1, 0, 257, 128, 127, 0],     # around the row tiles
    [700, 3, 0, 600],                     # long and short
]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("d,f", [(64, 64), (8, 8), (72, 40), (200, 136), (264, 328), (128, 512)])
@pytest.mark.parametrize("counts", COUNTS, ids=lambda c: "x".join(map(str, c))[:24])
def test_experts_backward(moe, counts, d, f, dtype):
    check_experts(moe, counts, d, f, dtype)


@pytest.mark.parametrize("counts,d,f", [
    ([1100, 900, 1300], 512, 384), ([513] * 4, 264, 520), ([2500], 320, 256),
    ([200, 90, 300, 10, 128, 256, 64, 77], 768, 320), ([3] * 70, 256, 192), ([1] * 200, 64, 128)])
def test_experts_backward_larger(moe, counts, d, f):
    check_experts(moe, counts, d, f, torch.bfloat16, seed=6)


@pytest.mark.parametrize("counts,d,f", [
    ([5] * 60 + [0, 9, 1, 40], 96, 360),     # short segments, many columns
    ([70, 3, 0, 150, 90, 33, 64, 190], 200, 488),
    ([1030, 970], 1200, 1000),               # the largest tiles, all cut
    ([600, 1], 200, 200), ([130, 470, 600], 200, 200), ([5000], 64, 64), ([4990], 200, 200)])
def test_experts_backward_f32_tiles(moe, counts, d, f):
    check_experts(moe, counts, d, f, torch.float32, seed=7)


@pytest.mark.parametrize("counts,d,f", [
    ([1], 1096, 72), ([3, 0, 130], 2056, 40), ([1, 2], 64, 1032), ([5] * 6, 4104, 136),
    ([257, 0, 1], 1544, 520), ([0, 128, 129], 640, 2056), ([16] * 8, 2048, 768)])
def test_experts_backward_few_tiles(moe, counts, d, f):
    """Row products whose K axis is split among the CTAs of a cluster."""
    check_experts(moe, counts, d, f, torch.bfloat16, seed=8)


@pytest.mark.parametrize("dtype", DTYPES)
def test_experts_backward_keeps_segments_apart(moe, dtype):
    """NaN and infinite rows of one expert reach that expert's gradients only."""
    counts, d, f = [37, 21, 70, 5], 128, 64
    offsets, x, Wgu, Wd, h, dy = experts_case(9, counts, d, f, dtype)
    cfg = moe.config(sum(counts), d, len(counts), 1, f, dtype)
    clean = run_experts(moe, cfg, offsets, x, Wgu, Wd, h, dy)
    bad = slice(offsets[1], offsets[2])
    x, h, dy = x.clone(), h.clone(), dy.clone()
    x[bad], h[bad], dy[bad] = float("nan"), float("inf"), float("nan")
    dx, dWgu, dWd = run_experts(moe, cfg, offsets, x, Wgu, Wd, h, dy)
    keep = [e for e in range(len(counts)) if e != 1]
    rows = torch.ones(sum(counts), dtype=torch.bool, device="cuda")
    rows[bad] = False
    assert torch.equal(dx[rows], clean[0][rows])
    assert torch.equal(dWgu[keep], clean[1][keep]) and torch.equal(dWd[keep], clean[2][keep])
    assert torch.isnan(dWgu[1].float()).any() and torch.isnan(dWd[1].float()).any()


@pytest.mark.parametrize("dtype", DTYPES)
def test_experts_backward_extreme_gates(moe, dtype):
    """Gates far in both tails of the sigmoid: no overflow, no NaN."""
    counts, d, f = [40, 24], 64, 64
    offsets, x, Wgu, Wd, h, dy = experts_case(13, counts, d, f, dtype)
    Wgu = (Wgu.float() * 60).to(dtype)  # gates of about +-60 standard deviations
    cfg = moe.config(sum(counts), d, len(counts), 1, f, dtype)
    for t in run_experts(moe, cfg, offsets, x, Wgu, Wd, h, dy):
        assert torch.isfinite(t.float()).all()


# --------------------------------- router ----------------------------------
ROUTES = [(1, 64, 2, 1), (5, 8, 3, 2), (70, 72, 8, 2), (333, 264, 100, 7), (64, 128, 64, 32),
          (1000, 512, 128, 8), (2049, 320, 16, 4), (1200, 136, 257, 8), (300, 64, 1024, 8)]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("T,d,E,k", ROUTES)
def test_route_backward(moe, T, d, E, k, renorm, dtype):
    g = gen(T + E)
    L, idx = routing(g, T, E, k, skew=0.01)
    x, Wr, dw = randn(g, T, d, dtype=dtype), randn(g, E, d, std=d ** -0.5), randn(g, T, k)
    w = ref.weights(L.double(), idx, renorm).float()
    dx_in = randn(g, T, d, dtype=dtype)
    cfg = moe.config(T, d, E, k, 8, dtype, renormalize=renorm)
    ws = torch.full((moe.moe_route_backward_workspace_size(cfg),), 255, dtype=torch.uint8, device="cuda")
    dL, dWr, db, dx = nan(T, E), nan(E, d), nan(E), nan(T, d, dtype=dtype)
    moe.moe_route_backward(cfg, x, Wr, None if renorm else L, idx.int(), w, dw, None, dL, dWr, db, dx, ws)
    ok(moe)
    rL = ref.grads(lambda l: ref.weights(l, idx, renorm), [L.double()], dw.double())[0]
    # w and dw are fp32; S sums k products; p by expf over E terms: weights of
    # at most 1, so each term is within (ceil(E/32) + k + 16) ulps of sum|w dw| + |dw|
    scale = (w.double() * dw.double()).abs().sum(-1, keepdim=True) + dw.double().abs().max(-1, keepdim=True).values
    tolL = (-(-E // 32) + k + 16) * 2.0 ** -23 * scale
    assert ((dL.double() - rL).abs() <= tolL).all()
    if renorm:
        mask = torch.ones(T, E, dtype=torch.bool, device="cuda").scatter_(1, idx, False)
        assert (dL[mask] == 0).all()
    used = dL.double()  # the sums are checked on the logit gradients the call wrote
    for got, want, n in ((dWr, used.t() @ x.double(), T), (db, used.sum(0), T)):
        assert (got.double() - want).abs().max() <= ftol(want, n) + 1e-6 * U32, n
    want = used @ Wr.double()
    tol = ftol(want, E) + (UB * want.abs() + 2.0 ** -16 * want.abs().max() if dtype == torch.bfloat16 else 0)
    assert ((dx.double() - want).abs() <= tol).all()
    # on top of another gradient of x, in place
    acc = dx_in.clone()
    dWr2, db2 = nan(E, d), nan(E)
    moe.moe_route_backward(cfg, x, Wr, L, idx.int(), w, dw, acc, dL, dWr2, db2, acc, ws)
    ok(moe)
    assert torch.equal(dWr2, dWr) and torch.equal(db2, db)
    total = want + dx_in.double()
    tol = tol + (UB if dtype == torch.bfloat16 else U32) * total.abs()
    assert ((acc.double() - total).abs() <= tol).all()


@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("T,d,E,k", [(1500, 1096, 9, 2), (1400, 1040, 24, 6), (1300, 1032, 40, 8),
                                     (700, 2064, 72, 15), (200, 4808, 500, 2), (4100, 136, 33, 1)])
def test_route_backward_f32_tiles(moe, T, d, E, k, renorm):
    test_route_backward(moe, T, d, E, k, renorm, torch.float32)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("T,d,E,k", [(1, 2048, 128, 8), (16, 1032, 26, 7), (256, 264, 100, 4), (100, 7168, 9, 2),
                                     (128, 72, 512, 8), (31, 8, 17, 1)])
def test_route_backward_short_batches(moe, T, d, E, k, renorm, dtype):
    test_route_backward(moe, T, d, E, k, renorm, dtype)


def test_route_backward_without_bias_output(moe):
    T, d, E, k = 40, 64, 16, 2
    g = gen(3)
    L, idx = routing(g, T, E, k)
    x, Wr, dw = randn(g, T, d), randn(g, E, d), randn(g, T, k)
    w = ref.weights(L, idx, True)
    cfg = moe.config(T, d, E, k, 8, torch.float32)
    ws = torch.empty(moe.moe_route_backward_workspace_size(cfg), dtype=torch.uint8, device="cuda")
    out = [[nan(T, E), nan(E, d), b, nan(T, d)] for b in (nan(E), None)]
    for o in out:
        moe.moe_route_backward(cfg, x, Wr, None, idx.int(), w, dw, None, *o, ws)
    ok(moe)
    for a, b in zip(out[0], out[1]):
        assert b is None or torch.equal(a, b)


@pytest.mark.parametrize("renorm", [True, False])
def test_route_backward_reports_bad_expert_ids(moe, renorm):
    T, d, E, k = 33, 64, 8, 2
    g = gen(4)
    L, idx = routing(g, T, E, k)
    idx = idx.int()
    w, dw = ref.weights(L, idx.long(), renorm), randn(g, T, k)
    idx[3, 1], idx[9, 0] = E, -1
    cfg = moe.config(T, d, E, k, 8, torch.float32, renormalize=renorm)
    ws = torch.empty(moe.moe_route_backward_workspace_size(cfg), dtype=torch.uint8, device="cuda")
    dL, dWr, db, dx = nan(T, E), nan(E, d), nan(E), nan(T, d)
    moe.moe_route_backward(cfg, randn(g, T, d), randn(g, E, d), L, idx, w, dw, None, dL, dWr, db, dx, ws)
    torch.cuda.synchronize()
    assert moe.moe_last_device_error(raise_on_error=False) == moe.MOE_ERR_BAD_ROUTING
    for t in (dL, dWr, db, dx):
        assert torch.isfinite(t).all()
    assert moe.moe_last_device_error() == moe.MOE_OK


def test_route_backward_infinite_logits(moe):
    """-inf logits (experts masked out of the routing) have a zero gradient."""
    T, d, E, k = 20, 64, 12, 2
    g = gen(8)
    L, _ = routing(g, T, E, k)
    L[:, 5:] = float("-inf")
    idx = torch.sort(L, dim=-1, descending=True, stable=True).indices[:, :k].contiguous()
    w = ref.weights(L.double(), idx, False).float()
    cfg = moe.config(T, d, E, k, 8, torch.float32, renormalize=False)
    ws = torch.empty(moe.moe_route_backward_workspace_size(cfg), dtype=torch.uint8, device="cuda")
    dL, dWr, db, dx = nan(T, E), nan(E, d), nan(E), nan(T, d)
    moe.moe_route_backward(cfg, randn(g, T, d), randn(g, E, d), L, idx.int(), w, randn(g, T, k), None,
                           dL, dWr, db, dx, ws)
    ok(moe)
    assert (dL[:, 5:] == 0).all() and (dWr[5:] == 0).all() and torch.isfinite(dx).all()


# ------------------------------- the layer ---------------------------------
LAYERS = [  # T, d, E, k, f, dtype, renorm, scale, bias
    (64, 128, 8, 2, 256, torch.float32, True, False, False),
    (50, 72, 5, 3, 40, torch.float32, False, False, True),
    (33, 64, 6, 6, 64, torch.float32, False, True, False),
    (90, 64, 4, 2, 72, torch.float32, True, True, True),
    (300, 256, 16, 4, 128, torch.bfloat16, True, False, True),     # rows gathered in the forward
    (300, 200, 16, 4, 136, torch.bfloat16, False, False, False),   # permuted copy
    (200, 128, 4, 4, 192, torch.bfloat16, False, False, False),    # k == E
    (200, 128, 4, 4, 192, torch.bfloat16, True, True, False),      # k == E, weights on the inputs
    (300, 192, 8, 2, 128, torch.bfloat16, True, True, False),      # gathered, weights on the inputs
    (1, 64, 4, 2, 64, torch.bfloat16, True, False, False),
    (250, 200, 8, 2, 136, torch.bfloat16, True, True, True),       # weights on the inputs, copied rows
    (1500, 128, 8, 2, 192, torch.bfloat16, True, False, False),    # both tile shapes
    (3000, 128, 4, 2, 192, torch.bfloat16, False, False, True),    # CTA pairs
    (700, 128, 40, 8, 64, torch.bfloat16, True, False, True),      # single CTAs, E > 8
]


@pytest.mark.parametrize("T,d,E,k,f,dtype,renorm,scale,bias", LAYERS)
def test_layer_backward(moe, T, d, E, k, f, dtype, renorm, scale, bias):
    """MoELayer.backward after its forward: against double-precision automatic
    differentiation of the whole layer (norm-wise: the roundings of up to five
    bf16 values in series, 5 ub, or 2^-16 for fp32), and against central
    differences of the 64-bit layer along random directions."""
    g = gen(T + d + E)
    x = randn(g, T, d, dtype=dtype)
    Wr = randn(g, E, d, std=d ** -0.5)
    b = randn(g, E, std=0.5) if bias else None
    Wgu = randn(g, E, d, 2 * f, std=d ** -0.5, dtype=dtype)
    Wd = randn(g, E, f, d, std=f ** -0.5, dtype=dtype)
    dout = randn(g, T, d, dtype=dtype)
    lay = moe.MoELayer(Wr, Wgu, Wd, k, b, renorm, scale)
    lay(x)
    got = lay.backward(x, dout)
    ok(moe)
    at = moe.moe_workspace_layout(lay.config(T)).topk_idx
    idx = lay.workspace(T)[at:at + 4 * T * k].view(torch.int32).view(T, k).long()
    names = ["x", "Wr", "W_gate_up", "W_down"] + (["logit_bias"] if bias else [])
    args = [t.double() for t in (x, Wr, Wgu, Wd)] + ([b.double()] if bias else [])
    fn = lambda x, Wr, Wgu, Wd, bb=None: ref.layer(x, Wr, bb, Wgu, Wd, idx, renorm, scale)  # noqa: E731
    want = ref.grads(fn, args, dout.double())
    tol = 5 * UB if dtype == torch.bfloat16 else 2.0 ** -16
    for i, (n, r) in enumerate(zip(names, want)):
        assert got[n].shape == r.shape and got[n].dtype == (torch.float32 if n in ("Wr", "logit_bias") else dtype)
        err = (got[n].double() - r).norm() / r.norm()
        assert err <= tol, (n, float(err))
        v = torch.randn(r.shape, generator=g, device="cuda", dtype=torch.float64)
        diff = ref.difference(fn, args, i, v, dout.double(), 1e-5)
        # <grad, v> is off by at most tol |grad| |v|, in a random direction tol |grad|;
        # 6 standard deviations; the difference's own error is about 1e-6 of it
        assert abs(float((got[n].double() * v).sum()) - diff) <= 6 * tol * float(r.norm()) + 1e-5 * abs(diff), n


def test_backward_repeats_bit_for_bit_and_keeps_forward(moe):
    T, d, E, k, f = 700, 256, 8, 2, 192
    g = gen(77)
    x, dout = (randn(g, T, d, dtype=torch.bfloat16) for _ in range(2))
    lay = moe.MoELayer(randn(g, E, d, std=d ** -0.5), randn(g, E, d, 2 * f, std=d ** -0.5, dtype=torch.bfloat16),
                       randn(g, E, f, d, std=f ** -0.5, dtype=torch.bfloat16), k)
    lay(x)
    before = lay.workspace(T).clone()
    a = {n: t.clone() for n, t in lay.backward(x, dout).items()}
    b = lay.backward(x, dout)
    ok(moe)
    for n in a:
        assert torch.equal(a[n], b[n]), n
    assert torch.equal(before, lay.workspace(T))


def test_backward_on_another_stream_and_in_a_graph(moe):
    T, d, E, k, f = 260, 128, 8, 2, 128
    g = gen(78)
    x, dout = (randn(g, T, d, dtype=torch.bfloat16) for _ in range(2))
    lay = moe.MoELayer(randn(g, E, d, std=d ** -0.5), randn(g, E, d, 2 * f, std=d ** -0.5, dtype=torch.bfloat16),
                       randn(g, E, f, d, std=f ** -0.5, dtype=torch.bfloat16), k)
    lay(x)
    want = {n: t.clone() for n, t in lay.backward(x, dout).items()}
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    out = torch.empty_like(x)
    with torch.cuda.stream(side):
        lay(x, out)
        got = lay.backward(x, dout)
    side.synchronize()
    for n in want:
        assert torch.equal(got[n], want[n]), n
        got[n].zero_()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        lay(x, out)
        lay.backward(x, dout, grads=got)
    graph.replay()
    ok(moe)
    for n in want:
        assert torch.equal(got[n], want[n]), n


def test_empty_batch_clears_weight_gradients(moe):
    d, E, k, f = 64, 8, 2, 128
    for dtype in DTYPES:
        g = gen(1)
        lay = moe.MoELayer(randn(g, E, d), randn(g, E, d, 2 * f, dtype=dtype), randn(g, E, f, d, dtype=dtype),
                           k, randn(g, E))
        grads = {"x": nan(0, d, dtype=dtype), "Wr": nan(E, d), "logit_bias": nan(E),
                 "W_gate_up": nan(E, d, 2 * f, dtype=dtype), "W_down": nan(E, f, d, dtype=dtype)}
        x = torch.empty(0, d, dtype=dtype, device="cuda")
        lay.backward(x, x, grads=grads)
        ok(moe)
        for n in ("Wr", "logit_bias", "W_gate_up", "W_down"):
            assert (grads[n] == 0).all(), n
