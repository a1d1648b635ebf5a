"""moe_route_scored_from_logits and its gradient against plain 64-bit forms
(scored_ref.py), and the balance bias's update.

The chosen ids are compared for equality: the choice is that of 64-bit values.

Weights.  Sigmoid: expf 2 ulp of 2^-23, the sum 1 + e and the quotient half an
ulp each, 3 * 2^-23; the sum of the chosen 5 roundings more, the last quotient
and the scale one each: below 16 * 2^-23 of the weight.  Softmax adds the
rounding of L - m, 2^-24 |L - m| of the exponential, twice (value and sum), and
the sum's ceil(E/32) + 5 terms.  Below 2^-126 a weight is subnormal: 2^-149.

Gradients.  dl = w (d - S/c) (1 - s) with w rounded to fp32, S of k <= 32
products: each factor within (16 + k) * 2^-23 relative of terms |d| + sum w |d| / c;
softmax without renormalisation the same with s (and its |L - m|) for w."""
import numpy as np
import pytest
import torch

from tests import backward_ref, scored_ref
from tests.gpu_util import load_moe

pytestmark = pytest.mark.gpu
EPS = 2.0 ** -23


@pytest.fixture(scope="module")
def moe():
    return load_moe()


def rng(seed):
    return torch.Generator().manual_seed(seed)


def route(moe, L, bias, k, r, renorm=True, stream=None):
    T, E = L.shape
    idx = torch.full((T, k), -7, dtype=torch.int32, device="cuda")
    w = torch.full((T, k), float("nan"), device="cuda")
    moe.moe_route_scored_from_logits(moe.config(T, 8, E, k, 8, renormalize=renorm), r, L, bias, idx,
                                     w, stream=stream)
    return idx, w


def check(moe, L, bias, k, score="sigmoid", G=1, Gk=1, top2=False, renorm=True, scale=1.0):
    r = moe.router(score, G, Gk, "top2" if top2 else "max", scale)
    idx, w = route(moe, L.cuda(), None if bias is None else bias.cuda(), k, r, renorm)
    torch.cuda.synchronize()
    assert moe.moe_last_device_error() == moe.MOE_OK
    idx, w = idx.cpu().numpy(), w.double().cpu().numpy()
    Ln, b = L.numpy(), None if bias is None else bias.numpy()
    for t in range(L.shape[0]):
        want = scored_ref.select(Ln[t], b, k, score == "sigmoid", G, Gk, top2)
        assert idx[t].tolist() == want, (t, idx[t].tolist(), want)
        s = scored_ref.log_scores(Ln[t], score == "sigmoid")[want]
        ref = scale * (scored_ref.shares(s) if renorm else np.exp(s))
        fin = Ln[t][np.isfinite(Ln[t])]
        span = 0.0 if score == "sigmoid" or not fin.size else float(fin.max()) - float(fin.min())
        tol = (24 + -(-L.shape[1] // 32) + 2 * span) * EPS * np.abs(ref) + scale * 2.0 ** -126
        assert (np.abs(w[t] - ref) <= tol).all(), (t, w[t], ref)


SHAPES = [  # E, k, G, Gk
    (1, 1, 1, 1), (2, 1, 1, 1), (8, 2, 1, 1), (33, 5, 1, 1), (64, 8, 8, 4), (160, 6, 8, 3),
    (256, 8, 8, 4), (256, 32, 16, 2), (96, 4, 3, 2), (40, 7, 5, 5), (12, 6, 12, 6), (32, 3, 32, 3),
    (1000, 10, 10, 4), (1020, 9, 17, 5), (1017, 6, 9, 2), (1024, 32, 1, 1), (1024, 8, 32, 5),
    (30, 30, 1, 1)]


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("biased,top2", [(False, False), (True, False), (True, True), (False, True)])
@pytest.mark.parametrize("E,k,G,Gk", SHAPES)
def test_selection_and_weights(moe, E, k, G, Gk, biased, top2, score):
    g = rng(E * 100 + k)
    T = 37
    L = torch.randn(T, E, generator=g) * 2
    bias = torch.randint(-100, 101, (E,), generator=g).float() * 1e-3 if biased else None
    for renorm, scale in ((True, 2.5), (False, 1.0)):
        check(moe, L, bias, k, score, G, Gk, top2, renorm, scale)


@pytest.mark.parametrize("T", [1, 7, 8, 9, 1000])
def test_lengths(moe, T):
    g = rng(T)
    check(moe, torch.randn(T, 64, generator=g), torch.randn(64, generator=g) * 0.01, 4, G=8, Gk=3,
          top2=True)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("G,Gk,top2", [(1, 1, False), (8, 4, True), (8, 4, False)])
def test_values_that_fp32_cannot_rank(moe, score, G, Gk, top2):
    """Logits a few fp32 steps apart, so that scores round to the same fp32
    value and groups to the same sum; distinct in 64 bits."""
    g = rng(5)
    E, T = 256, 24
    steps = torch.stack([torch.randperm(E, generator=g) for _ in range(T)]).float()
    for base in (1.0, -3.0, 9.0):
        L = torch.full((T, E), base) + steps * 2.0 ** -20  # exact: |L| < 16
        check(moe, L, torch.zeros(E), 8, score, G, Gk, top2)
        check(moe, L, torch.randint(0, 2, (E,), generator=g).float() * 0.5, 8, score, G, Gk, top2)


def test_padded_rows_and_exact_ties(moe):
    """Rows of one value: ids by bias alone, equal biases by id; and logits of
    few distinct values."""
    g = rng(6)
    bias = torch.randint(-5, 6, (256,), generator=g).float() * 1e-3
    for bias_ in (bias, torch.zeros(256)):
        check(moe, torch.zeros(5, 256), bias_, 8)
        check(moe, torch.randint(-2, 3, (40, 256), generator=g).float(), bias_, 8)
    # sums of halves and quarters are exact whatever their order
    check(moe, torch.zeros(5, 64), torch.randint(-4, 5, (64,), generator=g).float() * 0.25, 8, G=8,
          Gk=4, top2=True)
    check(moe, torch.zeros(5, 64), None, 8, "softmax", G=8, Gk=4)


def test_infinities_and_saturated_scores(moe):
    g = rng(7)
    L = torch.randn(16, 64, generator=g) * 3
    L[:, ::3] = float("-inf")
    L[3] = float("-inf")
    L[4] = -3.4028234663852886e38  # a mask of the type's lowest value
    L[5, 1:] = -3.4028234663852886e38
    L[6] = -200 + torch.arange(64.0)  # fp32 sigmoids underflow
    L[7] = torch.arange(64.0) * 0.1 + 20  # ... and reach 1
    bias = torch.randn(64, generator=g) * 0.1
    for score in ("softmax", "sigmoid"):
        for b in (None, bias):
            check(moe, L, b, 6, score)
            check(moe, L, b, 6, score, 8, 3, b is not None)
    out = bias.clone()
    out[10:40] = float("-inf")  # excluded experts
    out[50] = float("inf")      # one that is always there
    check(moe, L[:3], out, 6, "sigmoid")
    check(moe, L[:3], out, 6, "sigmoid", 8, 4, True)


def test_nan_ranks_last(moe):
    g = rng(8)
    L = torch.randn(9, 40, generator=g)
    L[:, 5:30] = float("nan")
    r = moe.router("sigmoid")
    idx, w = route(moe, L.cuda(), torch.zeros(40, device="cuda"), 20, r)
    for t in range(9):
        want = scored_ref.select(L[t].numpy(), np.zeros(40), 20, True, 1, 1, False)
        assert idx[t].tolist() == want
    assert torch.isnan(w).any(-1).all()  # 15 numbers and 5 NaN were chosen


@pytest.mark.parametrize("d,E,dtype", [(64, 256, "bf16"), (72, 20, "bf16"), (128, 160, "f32"),
                                       (64, 16, "bf16")])
@pytest.mark.parametrize("T", [5, 1100])
def test_route_from_tokens(moe, T, d, E, dtype):
    """Every way to the logits (partial sums, tiles, few experts): the choice is
    made on the logits that were written."""
    g = rng(d + E)
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    x = torch.randn(T, d, generator=g).to(dt)
    Wr = torch.randn(E, d, generator=g) * d ** -0.5
    lb, bias = torch.randn(E, generator=g) * 0.1, torch.randn(E, generator=g) * 0.05
    cfg = moe.config(T, d, E, 4, 8, dt)
    r = moe.router("sigmoid", 4, 2, "top2", 2.5)
    L = torch.full((T, E), float("nan"), device="cuda")
    idx = torch.empty(T, 4, dtype=torch.int32, device="cuda")
    w = torch.empty(T, 4, device="cuda")
    ws = torch.full((max(256, moe.moe_route_workspace_size(cfg)),), 255, dtype=torch.uint8,
                    device="cuda")
    moe.moe_route_scored(cfg, r, x.cuda(), Wr.cuda(), lb.cuda(), bias.cuda(), L, idx, w, ws)
    idx2, w2 = route(moe, L, bias.cuda(), 4, r)
    torch.cuda.synchronize()
    assert moe.moe_last_device_error() == moe.MOE_OK
    assert torch.equal(idx, idx2) and torch.equal(w, w2)
    want = x.double() @ Wr.double().t() + lb.double()
    mag = x.double().abs() @ Wr.double().abs().t() + lb.double().abs()
    assert ((L.double().cpu() - want).abs() <= 34 * EPS * mag).all()
    for t in range(0, T, max(1, T // 40)):
        assert idx[t].tolist() == scored_ref.select(L[t].cpu().numpy(), bias.numpy(), 4, True, 4, 2,
                                                    True)


def test_without_bias_or_groups_it_is_moe_route(moe):
    g = rng(9)
    L = torch.randn(300, 128, generator=g).cuda()
    cfg = moe.config(300, 8, 128, 8, 8)
    idx = torch.empty(300, 8, dtype=torch.int32, device="cuda")
    w = torch.empty(300, 8, device="cuda")
    moe.moe_route_from_logits(cfg, L, idx, w)
    idx2, w2 = route(moe, L, None, 8, moe.router())
    assert torch.equal(idx, idx2)
    assert ((w - w2).abs() <= 32 * EPS * w).all()


# -------------------------------- gradient ---------------------------------
def grad_case(seed, T, E, k, score, renorm, scale, spread=1.0):
    g = rng(seed)
    L = torch.randn(T, E, generator=g) * spread
    idx = torch.topk(L + 0.3 * torch.randn(T, E, generator=g), k).indices
    w = scored_ref.weights(L.double(), idx, score == "sigmoid", renorm, scale)
    return L, idx, w.float(), torch.randn(T, k, generator=g)


def bound(L, idx, w, d, score, renorm, scale):
    k = idx.shape[1]
    terms = d.abs() + ((w.abs() * d.abs()).sum(-1, keepdim=True) / scale if renorm else 0)
    if score == "softmax" and not renorm:
        s = torch.softmax(L.double(), -1)
        span = (L.max(-1, keepdim=True).values - L.min(-1, keepdim=True).values).double()
        g = (w.abs() * d.abs()).sum(-1, keepdim=True).double().expand_as(L).clone()
        g.scatter_add_(1, idx, scale * d.abs().double())
        return (24 + k + L.shape[1] // 32 + span) * EPS * s * g
    out = torch.zeros(L.shape, dtype=torch.float64)
    return out.scatter_(1, idx, (24 + k) * EPS * (w.abs() * terms).double())


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("T,E,k,scale", [
    (1, 2, 1, 1.0), (5, 7, 3, 2.5), (64, 8, 8, 1.0), (33, 256, 8, 2.5), (9, 130, 6, 16.0),
    (17, 500, 32, 1.0), (3, 1024, 16, 0.5), (6, 1001, 5, 1.0), (8, 33, 4, 1.0), (12, 64, 2, 3.0)])
def test_gradient_to_the_logits(moe, T, E, k, scale, renorm, score):
    L, idx, w, d = grad_case(E + k, T, E, k, score, renorm, scale, 2.0)
    dl = torch.full((T, E), float("nan"), device="cuda")
    moe.moe_route_scored_from_logits_backward(
        moe.config(T, 8, E, k, 8, renormalize=renorm), moe.router(score, weight_scale=scale), L.cuda(),
        idx.int().cuda(), w.cuda(), d.cuda(), dl)
    torch.cuda.synchronize()
    assert moe.moe_last_device_error() == moe.MOE_OK

    def f(x):
        return scored_ref.weights(x, idx, score == "sigmoid", renorm, scale)
    ref, = backward_ref.grads(f, [L.double()], d.double())
    # (2^-50: the reference's own rounding, zeros of the formula among its values)
    tol = bound(L, idx, w, d, score, renorm, scale) + 2.0 ** -50 * scale * float(d.abs().max())
    assert ((dl.double().cpu() - ref).abs() <= tol).all()
    # against differences: two steps of h lose h^2 of the third derivatives
    way = torch.randn(T, E, generator=rng(1)).double()
    diff = backward_ref.difference(f, [L.double()], 0, way, d.double(), 1e-5)
    got = float((dl.double().cpu() * way).sum())
    assert abs(got - diff) <= float((tol * way.abs()).sum()) + 1e-7 * scale * float(d.abs().sum())


def test_gradient_edges(moe):
    """Ids outside [0, E), a row of -inf, and a NaN in one token alone."""
    L, idx, w, d = grad_case(3, 6, 16, 3, "sigmoid", False, 1.0)
    bad = idx.int().clone()
    bad[2, 1], bad[4, 0] = 16, -1
    L[3] = float("-inf")
    d[5, 0] = float("nan")
    for score, renorm in (("sigmoid", False), ("sigmoid", True), ("softmax", False), ("softmax", True)):
        dl = torch.full((6, 16), 9.0, device="cuda")
        moe.moe_route_scored_from_logits_backward(
            moe.config(6, 8, 16, 3, 8, renormalize=renorm), moe.router(score), L.cuda(), bad.cuda(),
            w.cuda(), d.cuda(), dl)
        assert moe.moe_last_device_error(raise_on_error=False) == moe.MOE_ERR_BAD_ROUTING
        assert torch.isfinite(dl[:5]).all()
        assert torch.isnan(dl[5]).any()
        if score == "sigmoid" and not renorm:
            keep = [j for j in range(3) if j != 1]
            want = torch.zeros(16, dtype=torch.float64)
            want[idx[2, keep]] = (w[2] * d[2])[keep].double() * torch.sigmoid(-L[2, idx[2, keep]].double())
            assert ((dl[2].double().cpu() - want).abs() <= 30 * EPS * want.abs()).all()


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("T,d,E,k,dtype", [
    (40, 64, 8, 2, "bf16"), (40, 64, 8, 2, "f32"), (300, 128, 64, 4, "bf16"), (700, 64, 48, 4, "f32"),
    (600, 64, 64, 4, "f32"), (20, 256, 40, 6, "f32"), (30, 64, 200, 8, "bf16")])
def test_gradient_through_the_products(moe, T, d, E, k, dtype, renorm, score):
    """moe_route_scored_backward in each of its forms: dlogits as the entry
    above gives them, and the sums of moe_route_backward over them."""
    scale = 2.5
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    L, idx, w, dw = grad_case(T + E, T, E, k, score, renorm, scale)
    g = rng(T)
    x, Wr = torch.randn(T, d, generator=g).to(dt), torch.randn(E, d, generator=g) * d ** -0.5
    cfg, r = moe.config(T, d, E, k, 8, dt, renorm), moe.router(score, weight_scale=scale)
    want = torch.empty(T, E, device="cuda")
    args = [L.cuda(), idx.int().cuda(), w.cuda(), dw.cuda()]
    moe.moe_route_scored_from_logits_backward(cfg, r, *args, want)
    dl = torch.full((T, E), float("nan"), device="cuda")
    dWr, db = torch.full((E, d), float("nan"), device="cuda"), torch.full((E,), float("nan"), device="cuda")
    dx = torch.full((T, d), float("nan"), dtype=dt, device="cuda")
    ws = torch.full((moe.moe_route_scored_backward_workspace_size(cfg, r),), 255, dtype=torch.uint8,
                    device="cuda")
    moe.moe_route_scored_backward(cfg, r, x.cuda(), Wr.cuda(), *args, None, dl, dWr, db, dx, ws)
    torch.cuda.synchronize()
    assert moe.moe_last_device_error() == moe.MOE_OK
    tol = bound(L, idx, w, dw, score, renorm, scale)
    assert ((dl - want).abs().cpu().double() <= 2 * tol + 2.0 ** -126).all()
    D, X, W = dl.double().cpu(), x.double(), Wr.double()
    # fp32 sums of T (E) products: the probabilistic u sqrt(n), times 8, of the
    # magnitudes; tensor-core terms 2^-17 (dx), bf16's own rounding 2^-8
    for got, ref, mag, n in ((dWr, D.t() @ X, D.abs().t() @ X.abs(), T), (db, D.sum(0), D.abs().sum(0), T)):
        assert ((got.double().cpu() - ref).abs() <= 8 * 2.0 ** -24 * n ** 0.5 * mag + 1e-30).all()
    tol = (8 * 2.0 ** -24 * E ** 0.5 + (2.0 ** -16 if dtype == "bf16" else 0)) * (D.abs() @ W.abs())
    tol = tol + (2.0 ** -8 if dtype == "bf16" else 2.0 ** -24) * (D @ W).abs()
    assert ((dx.double().cpu() - D @ W).abs() <= tol + 1e-30).all()


# ------------------------------- balance bias -------------------------------
@pytest.mark.parametrize("layers,E", [(1, 1), (1, 8), (3, 7), (5, 256), (64, 1000), (2, 1024)])
def test_balance_bias(moe, layers, E):
    g = rng(layers * E)
    counts = torch.randint(0, 50, (layers, E), generator=g, dtype=torch.int32)
    counts[0, :] = 7  # every expert at the mean: no change
    if layers > 1:
        counts[1] = 0
    if layers > 2:
        counts[2] = 2 ** 31 - 1 - torch.randint(0, 2, (E,), generator=g, dtype=torch.int32)
    bias = torch.randn(layers, E, generator=g)
    n = counts.long()
    want = bias + 1e-3 * torch.sign(n.sum(1, keepdim=True) - E * n).float()
    imb = n.max(1).values.double() * E / n.sum(1).clamp(min=1).double()
    b, i = bias.cuda(), torch.full((layers,), float("nan"), device="cuda")
    moe.moe_update_balance_bias(counts.cuda(), 1e-3, b, i)
    assert torch.equal(b.cpu(), want)
    assert ((i.double().cpu() - imb).abs() <= 2 * EPS * imb).all()
    moe.moe_update_balance_bias(counts.cuda(), 1e-3, b)  # without the imbalance
    want = want + 1e-3 * torch.sign(n.sum(1, keepdim=True) - E * n).float()
    assert torch.equal(b.cpu(), want)


# ------------------------------ streams, graphs ------------------------------
def test_captured_and_on_two_streams(moe):
    g = rng(11)
    r, cfg = moe.router("sigmoid", 8, 4, "top2"), moe.config(512, 8, 64, 4, 8)
    Ls = [torch.randn(512, 64, generator=g).cuda() for _ in range(4)]
    bias = (torch.randn(64, generator=g) * 0.01).cuda()
    want = [[t.clone() for t in route(moe, L, bias, 4, r)] for L in Ls]
    torch.cuda.synchronize()
    sides = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = [route(moe, L, bias, 4, r, stream=sides[i % 2]) for i, L in enumerate(Ls)]
    torch.cuda.synchronize()
    for (i, w), (i2, w2) in zip(got, want):
        assert torch.equal(i, i2) and torch.equal(w, w2)
    L, d = Ls[0].clone(), torch.randn(512, 4, generator=g).cuda()
    idx, w = torch.empty(512, 4, dtype=torch.int32, device="cuda"), torch.empty(512, 4, device="cuda")
    dl, counts = torch.empty(512, 64, device="cuda"), torch.ones(64, dtype=torch.int32, device="cuda")
    moved = bias.clone()

    def calls():
        moe.moe_route_scored_from_logits(cfg, r, L, bias, idx, w)
        moe.moe_route_scored_from_logits_backward(cfg, r, L, idx, w, d, dl)
        moe.moe_update_balance_bias(counts, 1e-3, moved)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        calls()
    for n in (1, 2, 3):
        L.copy_(Ls[n])
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(idx, want[n][0]) and torch.equal(w, want[n][1])
        ref = dl.clone()
        moe.moe_route_scored_from_logits_backward(cfg, r, L, idx, w, d, dl)
        assert torch.equal(dl, ref)
    assert torch.equal(moved, bias)  # every load is the mean


def test_logits_past_32_bit_offsets(moe):
    """More than 2^32 logits: sampled tokens' choice and gradient."""
    T, E, k = (1 << 23) + 100, 512, 2
    L = torch.randn(T, E, generator=torch.Generator(device="cuda").manual_seed(1), device="cuda")
    bias = torch.zeros(E, device="cuda")
    cfg, r = moe.config(T, 8, E, k, 8, renormalize=False), moe.router("softmax")
    idx, w = route(moe, L, bias, k, r, renorm=False)
    dl = torch.empty_like(L)
    d = torch.ones_like(w)
    moe.moe_route_scored_from_logits_backward(cfg, r, L, idx, w, d, dl)
    torch.cuda.synchronize()
    for t in (0, 1, T // 2, (1 << 22) - 1, 1 << 22, (1 << 23) - 1, 1 << 23, T - 1):
        row = L[t].cpu()
        want = scored_ref.select(row.numpy(), np.zeros(E), k, False, 1, 1, False)
        assert idx[t].tolist() == want
        one = torch.tensor([want])
        ref, = backward_ref.grads(lambda x: scored_ref.weights(x, one, False, False, 1.0),
                                  [row[None].double()], torch.ones(1, k).double())
        assert ((dl[t].double().cpu() - ref[0]).abs() <= 100 * EPS * ref[0].abs().max()).all()
