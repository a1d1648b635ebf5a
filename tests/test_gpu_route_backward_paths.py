"""The router's gradient with expert ids outside [0, E) and with -inf logits, on
each way it is formed: few experts in one pass, short batches in one launch, the
fp32 products with dx gathered or multiplied, and the tensor cores.  The reference
is the formula in 64 bits with the bad slots left out; tolerances as in
tests/test_gpu_backward.py."""
import pytest
import torch

from tests import backward_ref as ref
from tests.gpu_util import load_moe
from tests.test_gpu_backward import U32, UB, ftol, gen, nan, ok, randn, routing

pytestmark = pytest.mark.gpu
F32, BF = torch.float32, torch.bfloat16

PATHS = {  # T, d, E, k, dtype, renorm
    "few-f32": (33, 64, 8, 2, F32, True), "few-f32-softmax": (700, 72, 7, 3, F32, False),
    "few-bf16": (700, 72, 8, 4, BF, True), "few-bf16-softmax": (33, 64, 5, 2, BF, False),
    "short-f32": (100, 72, 40, 3, F32, True), "short-f32-softmax": (100, 72, 40, 3, F32, False),
    "short-bf16": (200, 72, 44, 3, BF, True), "short-bf16-softmax": (200, 72, 44, 3, BF, False),
    "gathered-f32": (300, 136, 48, 4, F32, True),
    "products-f32": (300, 136, 12, 4, F32, True), "products-f32-softmax": (1300, 136, 48, 4, F32, False),
    "tensor-bf16": (600, 136, 48, 4, BF, True), "tensor-bf16-softmax": (600, 136, 48, 4, BF, False),
}


@pytest.fixture(scope="module")
def moe():
    return load_moe()


def run(moe, x, Wr, L, idx, w, dw, dx_in, dtype, renorm):
    (T, d), (E, k) = x.shape, (Wr.shape[0], idx.shape[1])
    cfg = moe.config(T, d, E, k, 8, dtype, renormalize=renorm)
    ws = torch.full((moe.moe_route_backward_workspace_size(cfg),), 255, dtype=torch.uint8, device="cuda")
    out = nan(T, E), nan(E, d), nan(E), nan(T, d, dtype=dtype)
    moe.moe_route_backward(cfg, x, Wr, None if renorm else L, idx, w, dw, dx_in, *out, ws)
    torch.cuda.synchronize()
    return out


def check(got, want, x, Wr, w, dw, dx_in, E, k, dtype):
    dL, dWr, db, dx = got
    scale = (w.double() * dw.double()).abs().sum(-1, keepdim=True) + dw.double().abs().max(-1, keepdim=True).values
    tol = (-(-E // 32) + k + 16) * 2.0 ** -23 * scale
    assert ((dL.double() - want).abs() <= tol).all()
    assert (dL[want == 0] == 0).all()
    used = dL.double()  # the sums are checked on the logit gradients the call wrote
    T = x.shape[0]
    for g, r in ((dWr, used.t() @ x.double()), (db, used.sum(0))):
        assert (g.double() - r).abs().max() <= ftol(r, T) + 1e-6 * U32
    r = used @ Wr.double()
    bf = dtype == BF
    tol = ftol(r, E) + (UB * r.abs() + 2.0 ** -16 * r.abs().max() if bf else 0)
    r = r + dx_in.double()
    assert ((dx.double() - r).abs() <= tol + (UB if bf else U32) * r.abs()).all()


@pytest.mark.parametrize("path", PATHS)
def test_bad_expert_ids(moe, path):
    T, d, E, k, dtype, renorm = PATHS[path]
    g = gen(T + E)
    L, idx = routing(g, T, E, k)
    w, dw = ref.weights(L.double(), idx, renorm).float(), randn(g, T, k)
    x, Wr, dx_in = randn(g, T, d, dtype=dtype), randn(g, E, d, std=d ** -0.5), randn(g, T, d, dtype=dtype)
    bad = idx.int()
    bad[3, 1], bad[9, 0], bad[T - 1, k - 1] = E, -1, 2 ** 31 - 1
    bad[17, :] = -2 ** 31  # a token with no slot left
    got = run(moe, x, Wr, L, bad, w, dw, dx_in, dtype, renorm)
    assert moe.moe_last_device_error(raise_on_error=False) == moe.MOE_ERR_BAD_ROUTING
    assert moe.moe_last_device_error() == moe.MOE_OK
    good = (bad >= 0) & (bad < E)
    wd, dd = w.double() * good, dw.double() * good
    S = (wd * dd).sum(-1, keepdim=True)
    at = torch.where(good, idx, 0)
    if renorm:
        want = torch.zeros(T, E, dtype=torch.float64, device="cuda").scatter_add_(1, at, wd * (dd - S))
    else:
        p = torch.softmax(L.double(), -1)
        want = -p * S
        want.scatter_add_(1, at, p.gather(1, at) * dd)
    check(got, want, x, Wr, w, dw, dx_in, E, k, dtype)


@pytest.mark.parametrize("path", PATHS)
def test_infinite_logits(moe, path):
    """Experts masked out per token; some tokens keep fewer than k, one of them a
    single expert, so that masked experts are chosen with a weight of zero."""
    T, d, E, k, dtype, renorm = PATHS[path]
    g = gen(T + E + 1)
    L, _ = routing(g, T, E, k)
    keep = torch.rand(T, E, generator=g, device="cuda") < 0.5
    keep[5], keep[6] = False, False
    keep[5, 2], keep[6, :k - 1] = True, True
    keep[~keep.any(1), 0] = True
    L[~keep] = float("-inf")
    idx = torch.sort(L, dim=-1, descending=True, stable=True).indices[:, :k].contiguous()
    w, dw = ref.weights(L.double(), idx, renorm).float(), randn(g, T, k)
    x, Wr, dx_in = randn(g, T, d, dtype=dtype), randn(g, E, d, std=d ** -0.5), randn(g, T, d, dtype=dtype)
    got = run(moe, x, Wr, L, idx.int(), w, dw, dx_in, dtype, renorm)
    ok(moe)
    assert (got[0][~keep] == 0).all()
    want = ref.grads(lambda l: ref.weights(l, idx, renorm), [L.double()], dw.double())[0]
    check(got, want, x, Wr, w, dw, dx_in, E, k, dtype)
