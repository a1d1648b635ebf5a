"""The whole layer with a scored router (moe_forward_scored,
moe_backward_scored through MoELayer) and its balance bias.

Tolerances: the layer's for its output, five bf16 roundings in series (fp32:
2^-16) in norm for the gradients; routing is that of the layer's own logits."""
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


def layer_of(moe, T, d, E, k, f, dt, score, renorm, scale_inputs, seed=0):
    g = rng(seed)
    x = torch.randn(T, d, generator=g).to(dt)
    Wr = torch.randn(E, d, generator=g) * d ** -0.5
    Wgu = (torch.randn(E, d, 2 * f, generator=g) * d ** -0.5).to(dt)
    Wd = (torch.randn(E, f, d, generator=g) * f ** -0.5).to(dt)
    lb = torch.randn(E, generator=g) * 0.1
    bias = torch.randint(-50, 51, (E,), generator=g).float() * 1e-3
    G = 4 if E % 4 == 0 and k <= E // 2 else 1
    r = moe.router(score, G, max(1, G // 2), "top2", 2.5)
    layer = moe.MoELayer(Wr.cuda(), Wgu.cuda(), Wd.cuda(), k, lb.cuda(), renorm, scale_inputs, r,
                         bias.cuda())
    return layer, x, (Wr, Wgu, Wd, lb, bias)


def routing(moe, layer, T):
    at = moe.moe_workspace_layout(layer.config(T))
    ws = layer.workspace(T)

    def view(off, n, dt):
        return ws[off:off + 4 * n].view(dt)
    return (view(at.logits, T * layer.E, torch.float32).view(T, -1).cpu(),
            view(at.topk_idx, T * layer.k, torch.int32).view(T, -1).cpu(),
            view(at.counts, layer.E, torch.int32).cpu())


def plain_layer(x, Wr, lb, Wgu, Wd, idx, score, renorm, scale_inputs):
    T, k = idx.shape
    w = scored_ref.weights(x @ Wr.t() + lb, idx, score == "sigmoid", renorm, 2.5)
    pos, offsets, order = backward_ref.permute(idx, Wr.shape[0])
    rows = x[order // k]
    if scale_inputs:
        rows = rows * w.reshape(-1)[order][:, None]
    y = backward_ref.ffn_rows(rows, offsets, Wgu, Wd)[pos].view(T, k, -1)
    return y.sum(1) if scale_inputs else (w[:, :, None] * y).sum(1)


@pytest.mark.parametrize("score,renorm,scale_inputs", [
    ("sigmoid", True, False), ("sigmoid", False, True), ("softmax", False, False),
    ("softmax", True, True)])
@pytest.mark.parametrize("T,d,E,k,f,dtype", [
    (50, 64, 8, 2, 64, "f32"), (200, 64, 64, 4, 64, "bf16"), (1, 128, 16, 3, 72, "bf16"),
    (1030, 128, 16, 2, 64, "bf16"), (40, 64, 4, 4, 64, "bf16"), (300, 72, 24, 3, 40, "f32"),
    (4500, 64, 64, 8, 64, "bf16"), (4500, 64, 32, 8, 64, "f32")])
def test_layer(moe, T, d, E, k, f, dtype, score, renorm, scale_inputs):
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    layer, x, (Wr, Wgu, Wd, lb, bias) = layer_of(moe, T, d, E, k, f, dt, score, renorm, scale_inputs)
    xd = x.cuda()
    out = layer(xd)
    torch.cuda.synchronize()
    assert moe.moe_last_device_error() == moe.MOE_OK
    L, idx, counts = routing(moe, layer, T)
    r = layer.router
    for t in range(0, T, max(1, T // 30)):
        assert idx[t].tolist() == scored_ref.select(L[t].numpy(), bias.numpy(), k, score == "sigmoid",
                                                    r.groups, r.topk_groups, True)
    assert counts.tolist() == torch.bincount(idx.long().reshape(-1), minlength=E).tolist()
    args = [t.double() for t in (x, Wr, lb, Wgu, Wd)]

    def fn(*a):
        return plain_layer(*a, idx.long(), score, renorm, scale_inputs)
    ref = fn(*args)
    tol = 2e-2 * float(ref.abs().max()) + 1e-3 if dtype == "bf16" else \
        (8 * 2.0 ** -24 * (2 * d ** 0.5 + f ** 0.5) + k * 40 * EPS) * float(ref.abs().max())
    assert float((out.double().cpu() - ref).abs().max()) <= tol
    dout = torch.randn(T, d, generator=rng(4)).to(dt)
    grads = layer.backward(xd, dout.cuda())
    torch.cuda.synchronize()
    assert moe.moe_last_device_error() == moe.MOE_OK
    want = backward_ref.grads(fn, args, dout.double())
    lim = 5 * 2.0 ** -8 if dtype == "bf16" else 2.0 ** -16
    for n, ref in zip(("x", "Wr", "logit_bias", "W_gate_up", "W_down"), want):
        got = grads[n].double().cpu()
        assert float((got - ref).norm()) <= lim * float(ref.norm()), n


def test_layer_balance_bias_update(moe):
    layer, x, (*_, bias) = layer_of(moe, 100, 64, 16, 2, 64, torch.bfloat16, "sigmoid", True, False)
    with pytest.raises(RuntimeError):
        layer.update_balance_bias(0.01)
    layer(x.cuda())
    n = routing(moe, layer, 100)[2].long()
    imb = torch.empty(1, device="cuda")
    layer.update_balance_bias(0.01, imb)
    assert torch.equal(layer.balance_bias.cpu(), bias + 0.01 * torch.sign(n.sum() - 16 * n).float())
    want = 16 * int(n.max()) / int(n.sum())
    assert abs(float(imb) - want) <= 2 * EPS * want
    for bad in (torch.empty(2, device="cuda"), torch.empty(1), torch.empty(1, device="cuda").double()):
        with pytest.raises(ValueError):
            layer.update_balance_bias(0.01, bad)
    plain = moe.MoELayer(layer.Wr, layer.W_gate_up, layer.W_down, 2)
    plain(x.cuda())
    with pytest.raises(RuntimeError):
        plain.update_balance_bias(0.01)


def test_backward_refuses_another_router(moe):
    layer, x, _ = layer_of(moe, 20, 64, 16, 2, 64, torch.bfloat16, "sigmoid", True, False)
    x = x.cuda()
    layer(x)
    layer.router = moe.router("softmax", 4, 2, "top2", 2.5)
    with pytest.raises(RuntimeError):
        layer.backward(x, x)


def test_empty_batch(moe):
    layer, x, _ = layer_of(moe, 8, 64, 16, 2, 64, torch.bfloat16, "sigmoid", True, False)
    empty = x[:0].cuda()
    assert layer(empty).shape == (0, 64)
    grads = layer.backward(empty, empty)
    for n in ("Wr", "W_gate_up", "W_down", "logit_bias"):
        assert not grads[n].any()
