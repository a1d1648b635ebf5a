"""moe_route_scored_backward and the layer's gradient with tokens whose logits are
-inf, all of them or some: such scores are 0, and so are their gradients, in each
form of the router's gradient (few experts, CUDA cores, tensor cores)."""
import pytest
import torch

from tests.gpu_util import load_moe

pytestmark = pytest.mark.gpu
EPS = 2.0 ** -23
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def moe():
    return load_moe()


def scores(L, sigmoid):
    """In 64 bits; 0 for a row of -inf."""
    if sigmoid:
        return torch.sigmoid(L)
    m = L.max(-1, keepdim=True).values
    e = torch.where(torch.isinf(m), 0.0, torch.exp(L - m))
    return e / e.sum(-1, keepdim=True).clamp(min=1e-300)


def gradient(L, idx, w, d, sigmoid, renorm, scale):
    """The header's formulas, from the weights as given."""
    s = scores(L, sigmoid)
    S = (w * d).sum(-1, keepdim=True)
    out = torch.zeros_like(L)
    if not sigmoid and not renorm:
        return s * (out.scatter(1, idx, scale * d) - S)
    t = w * (d - S / scale) if renorm else w * d
    if sigmoid:
        t = t * (1.0 - s.gather(1, idx))
    return out.scatter(1, idx, t)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [False, True])
@pytest.mark.parametrize("T,d,E,k,dt", [
    (40, 64, 8, 2, BF), (40, 64, 8, 2, F32), (1500, 64, 6, 2, BF), (1500, 64, 6, 2, F32),
    (300, 128, 64, 4, BF), (600, 64, 64, 4, F32), (20, 256, 40, 6, F32), (30, 64, 200, 8, BF)])
def test_rows_without_scores(moe, T, d, E, k, dt, renorm, score):
    sigmoid, scale = score == "sigmoid", 2.5
    g = torch.Generator().manual_seed(T + E)
    L = torch.randn(T, E, generator=g)
    idx = torch.topk(L, k).indices
    some, none = slice(1, None, 7), slice(3, None, 5)
    L[some, ::3] = float("-inf")
    L[none] = float("-inf")
    s = scores(L.double(), sigmoid).gather(1, idx)
    w = scale * (s / s.sum(-1, keepdim=True).clamp(min=1e-300) if renorm else s).float()
    assert (w[none] == 0).all()
    dw = torch.randn(T, k, generator=g)
    x, Wr = torch.randn(T, d, generator=g).to(dt), torch.randn(E, d, generator=g) * d ** -0.5
    cfg, r = moe.config(T, d, E, k, 8, dt, renorm), moe.router(score, weight_scale=scale)
    nan = float("nan")
    dl, dWr = torch.full((T, E), nan, device="cuda"), torch.full((E, d), nan, device="cuda")
    db, dx = torch.full((E,), nan, device="cuda"), torch.full((T, d), nan, dtype=dt, device="cuda")
    ws = torch.full((moe.moe_route_scored_backward_workspace_size(cfg, r),), 255, dtype=torch.uint8,
                    device="cuda")
    moe.moe_route_scored_backward(cfg, r, x.cuda(), Wr.cuda(), L.cuda(), idx.int().cuda(), w.cuda(),
                                  dw.cuda(), None, dl, dWr, db, dx, ws)
    torch.cuda.synchronize()
    assert moe.moe_last_device_error() == moe.MOE_OK
    want = gradient(L.double(), idx, w.double(), dw.double(), sigmoid, renorm, scale)
    got = dl.double().cpu()
    assert not got[none].any()
    # a score to (24 + E / 32 + the logits' span) ulp of itself, the sum S to k more of
    # its magnitudes
    S = (w.abs() * dw.abs()).sum(-1, keepdim=True).double()
    top = torch.zeros(T, E, dtype=torch.float64).scatter(
        1, idx, (w.abs() * dw.abs()).double() if renorm or sigmoid else scale * dw.abs().double())
    mag = (top + w.double().new_zeros(T, E).scatter(1, idx, w.abs().double()) * S / scale) \
        if renorm or sigmoid else scores(L.double(), False) * (top + S)
    span = torch.where(L.isinf(), 0.0, L).max() - torch.where(L.isinf(), 0.0, L).min()
    assert ((got - want).abs() <= (24 + k + E // 32 + float(span)) * EPS * mag).all()
    # and the sums over them (fp32 sums of n products: u sqrt(n), times 8, of the
    # magnitudes; tensor-core terms 2^-17; bf16's own rounding 2^-8)
    X, W = x.double(), Wr.double()
    for a, ref, size in ((dWr, got.t() @ X, got.abs().t() @ X.abs()), (db, got.sum(0), got.abs().sum(0))):
        assert ((a.double().cpu() - ref).abs() <= 8 * 2.0 ** -24 * T ** 0.5 * size + 1e-30).all()
    tol = (8 * 2.0 ** -24 * E ** 0.5 + (2.0 ** -16 if dt == BF else 0)) * (got.abs() @ W.abs())
    tol = tol + (2.0 ** -8 if dt == BF else 2.0 ** -24) * (got @ W).abs()
    assert ((dx.double().cpu() - got @ W).abs() <= tol + 1e-30).all()


@pytest.mark.parametrize("E,dt", [(8, BF), (8, F32), (64, BF)])
def test_layer_whose_logits_are_all_masked(moe, E, dt):
    """The router's gradients of a layer that sees no expert are 0."""
    T, d, k, f = 70, 64, 2, 128
    g = torch.Generator(device="cuda").manual_seed(E)

    def randn(*shape, t=dt):
        return (torch.randn(*shape, generator=g, device="cuda") * 0.1).to(t)
    bias = torch.full((E,), float("-inf"), device="cuda")
    layer = moe.MoELayer(randn(E, d, t=F32), randn(E, d, 2 * f), randn(E, f, d), k, bias,
                         renormalize=False, router=moe.router())
    x = randn(T, d)
    out = layer(x)
    grads = layer.backward(x, randn(T, d))
    torch.cuda.synchronize()
    assert moe.moe_last_device_error() == moe.MOE_OK
    assert not out.any()
    for n, t in grads.items():
        assert not t.any(), n
