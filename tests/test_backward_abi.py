"""Refusals and size queries of the backward pass and of gradient clipping:
each call here returns before it touches a device."""
import ctypes
import math

import pytest
import torch


@pytest.fixture(scope="module")
def moe():
    from token_dispatch_grouped_fp32_gb300 import build
    build.build()
    from token_dispatch_grouped_fp32_gb300 import moe as _moe
    return _moe


A = 256  # an aligned address that is never read
BIG = 1 << 40


def calls(moe, cfg, a=A, ws_bytes=BIG, **swap):
    """Every entry with valid-looking arguments, some replaced by position."""
    def go(fn, *args, n=None):
        args = list(args)
        for i, v in swap.items():
            if i.startswith("_") and int(i[1:]) < len(args):
                args[int(i[1:])] = v
        kw = {} if n is None else {"ws_bytes": n}
        return fn(cfg, *args, stream=0, raise_on_error=False, **kw)
    return {
        "combine": lambda: go(moe.moe_combine_backward, a, a, a, a, a, a),
        "dispatch": lambda: go(moe.moe_dispatch_backward, a, a, a, a, a, a),
        "experts": lambda: go(moe.moe_grouped_swiglu_backward, a, a, a, a, a, a, a, a, a, a, n=ws_bytes),
        "route": lambda: go(moe.moe_route_backward, a, a, a, a, a, a, a, a, a, a, a, a, n=ws_bytes),
    }


@pytest.mark.parametrize("bad,code", [
    (dict(T=-1), -1), (dict(d=12), -1), (dict(f=20), -1), (dict(k=9), -1), (dict(k=0), -1),
    (dict(E=2048), -2), (dict(dtype=7), -2), (dict(T=2 ** 29, k=8), -1)])
def test_bad_configs(moe, bad, code):
    base = dict(T=16, d=64, E=8, k=2, f=64, dtype="bf16")
    base.update(bad)
    cfg = moe.config(**base)
    for name, call in calls(moe, cfg).items():
        assert call() == code, name
    assert moe.moe_backward(cfg, A, A, A, A, A, A, A, A, A, A, A, 2 * A, fwd_ws_bytes=BIG,
                            ws_bytes=BIG, stream=0, raise_on_error=False) == code
    for size in (moe.moe_grouped_swiglu_backward_workspace_size, moe.moe_route_backward_workspace_size,
                 moe.moe_backward_workspace_size):
        assert size(cfg) == 0


def test_null_and_misaligned_arguments(moe):
    """Every argument that must be given, NULL and off by 8 bytes."""
    optional = {  # positions that may be NULL: per entry, without scale_inputs, renormalised
        "combine": set(), "dispatch": {2, 3, 5}, "experts": set(), "route": {2, 6, 9}}
    cfg = moe.config(16, 64, 8, 2, 64)
    n_args = {"combine": 6, "dispatch": 6, "experts": 10, "route": 12}
    for name, n in n_args.items():
        for i in range(n):
            if i in optional[name]:
                continue
            for v in (None, A + 8):
                assert calls(moe, cfg, **{f"_{i}": v})[name]() == moe.MOE_ERR_INVALID_ARG, (name, i, v)
                assert moe.moe_last_error_message()
    # given but misaligned, where NULL is fine
    for i in (6, 9):
        assert calls(moe, cfg, **{f"_{i}": A + 8})["route"]() == moe.MOE_ERR_INVALID_ARG


def test_arguments_that_a_mode_needs(moe):
    scaled = moe.config(16, 64, 8, 2, 64, scale_inputs=True)
    for i in (2, 3, 5):  # weights on the inputs: the dispatch's gradient needs w, x and dw
        assert calls(moe, scaled, **{f"_{i}": None})["dispatch"]() == moe.MOE_ERR_INVALID_ARG
    plain = moe.config(16, 64, 8, 2, 64, renormalize=False)
    assert calls(moe, plain, _2=None)["route"]() == moe.MOE_ERR_INVALID_ARG  # logits


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_workspaces(moe, dtype):
    T, d, E, k, f = 1000, 256, 16, 4, 128
    cfg = moe.config(T, d, E, k, f, dtype)
    P, es = T * k, 2 if dtype == "bf16" else 4
    n = moe.moe_grouped_swiglu_backward_workspace_size(cfg)
    # dgu [P][2f] in the act dtype; bf16: dh [P][f] fp32 besides
    assert n == P * 2 * f * es + (4 * P * f if dtype == "bf16" else 0)
    r = moe.moe_route_backward_workspace_size(cfg)
    assert r >= 4 * E * d
    b = moe.moe_backward_workspace_size(cfg)
    assert b >= n + r + 2 * P * d * es
    for name, need in (("experts", n), ("route", r)):
        assert calls(moe, cfg, ws_bytes=need - 1)[name]() == moe.MOE_ERR_WORKSPACE
    fwd = moe.moe_workspace_size(cfg)
    args = (A, A, A, A, A, A, A, A, A, A, A)
    short = dict(stream=0, raise_on_error=False)
    assert moe.moe_backward(cfg, *args, 2 * A, fwd_ws_bytes=fwd - 1, ws_bytes=b, **short) == \
        moe.MOE_ERR_WORKSPACE
    assert moe.moe_backward(cfg, *args, 2 * A, fwd_ws_bytes=fwd, ws_bytes=b - 1, **short) == \
        moe.MOE_ERR_WORKSPACE
    assert moe.moe_backward(cfg, *args, A, fwd_ws_bytes=fwd, ws_bytes=b, **short) == \
        moe.MOE_ERR_INVALID_ARG  # one buffer for both workspaces
    for i in range(len(args)):
        if i == 8:  # the bias gradient is optional
            continue
        bad = list(args)
        bad[i] = None
        assert moe.moe_backward(cfg, *bad, 2 * A, fwd_ws_bytes=fwd, ws_bytes=b, **short) == \
            moe.MOE_ERR_INVALID_ARG, i
    assert moe.moe_backward_workspace_size(moe.config(0, d, E, k, f, dtype)) == 0


def test_empty_batch_without_weight_gradients(moe):
    cfg = moe.config(0, 64, 8, 2, 64)
    assert moe.moe_combine_backward(cfg, A, A, A, A, A, A, stream=0) == moe.MOE_OK
    assert moe.moe_dispatch_backward(cfg, A, A, A, A, A, A, stream=0) == moe.MOE_OK
    # with them, the buffers to clear have to be there
    assert calls(moe, cfg, _7=None)["experts"]() == moe.MOE_ERR_INVALID_ARG
    assert calls(moe, cfg, _8=None)["route"]() == moe.MOE_ERR_INVALID_ARG


def entry(moe, **kw):
    e = moe.moe_grad_t(grad=A, out=A, numel=10, dtype=moe.MOE_F32, reserved=0)
    for n, v in kw.items():
        setattr(e, n, v)
    return (moe.moe_grad_t * 1)(e)


@pytest.mark.parametrize("kw,code", [
    (dict(numel=-1), -1), (dict(grad=None), -1), (dict(grad=A + 2), -1), (dict(out=A + 2), -1),
    (dict(dtype=1, grad=A + 1), -1), (dict(dtype=5), -2), (dict(numel=1 << 60), -1)])
def test_clip_refuses_bad_tensors(moe, kw, code):
    n = moe.moe_clip_grad_norm_workspace_size()
    assert moe.moe_clip_grad_norm(entry(moe, **kw), 1.0, A, A, ws_bytes=n, n=1, stream=0,
                                  raise_on_error=False) == code
    assert moe.moe_last_error_message()


def test_clip_refuses_bad_arguments(moe):
    ok, n = entry(moe), moe.moe_clip_grad_norm_workspace_size()

    def go(grads=ok, max_norm=1.0, norm=A, ws=A, ws_bytes=n, count=1):
        return moe.moe_clip_grad_norm(grads, max_norm, norm, ws, ws_bytes=ws_bytes, n=count, stream=0,
                                      raise_on_error=False)
    assert go(count=-1) == moe.MOE_ERR_INVALID_ARG
    assert go(grads=None) == moe.MOE_ERR_INVALID_ARG
    for v in (-1.0, math.nan, -math.inf):
        assert go(max_norm=v) == moe.MOE_ERR_INVALID_ARG
    assert go(norm=None) == moe.MOE_ERR_INVALID_ARG and go(norm=A + 2) == moe.MOE_ERR_INVALID_ARG
    assert go(ws=None) == moe.MOE_ERR_INVALID_ARG and go(ws=A + 8) == moe.MOE_ERR_INVALID_ARG
    assert go(ws_bytes=n - 1) == moe.MOE_ERR_WORKSPACE


def test_grad_list(moe):
    g = [torch.zeros(5), torch.zeros(3, dtype=torch.bfloat16)]
    lst = moe.grad_list(g)
    assert lst.count == 2 and lst[0].grad == lst[0].out == g[0].data_ptr()
    assert [e.numel for e in lst] == [5, 3] and [e.dtype for e in lst] == [moe.MOE_F32, moe.MOE_BF16]
    assert moe.grad_list(g, [None, g[1]])[0].out is None
    assert moe.grad_list([]).count == 0
    with pytest.raises(TypeError):
        moe.grad_list([torch.zeros(3, dtype=torch.float64)])
    with pytest.raises(ValueError):
        moe.grad_list(g, [g[0]])
    with pytest.raises(ValueError):
        moe.grad_list(g, [g[0], g[0]])
    with pytest.raises(ValueError):
        moe.grad_list([torch.zeros(4, 4).t()])


def test_struct_layouts_match(moe):
    assert ctypes.sizeof(moe.moe_grad_t) == 32


def test_layer_backward_refuses_what_it_cannot_use(moe):
    """Before any launch: no forward on the stream, other sizes or types, and
    gradient buffers of another shape."""
    d, E, k, f = 64, 8, 2, 128
    bf = torch.bfloat16
    lay = moe.MoELayer(torch.zeros(E, d), torch.zeros(E, d, 2 * f, dtype=bf), torch.zeros(E, f, d, dtype=bf), k)
    x = torch.zeros(16, d, dtype=bf)
    with pytest.raises(RuntimeError, match="latest forward"):
        lay.backward(x, x, stream=0)
    lay._tokens[0] = 16
    with pytest.raises(RuntimeError, match="latest forward"):
        lay.backward(x[:8], x[:8], stream=0)
    for bad in (x.float(), x[:, :32], x[:8]):
        with pytest.raises(ValueError):
            lay.backward(x, bad, stream=0)
    with pytest.raises(ValueError):
        lay.backward(x.float(), x.float(), stream=0)
    good = {"x": torch.empty_like(x), "Wr": torch.empty_like(lay.Wr),
            "W_gate_up": torch.empty_like(lay.W_gate_up), "W_down": torch.empty_like(lay.W_down)}
    for n, t in good.items():
        for bad in (None, t[:1], t.double()):
            with pytest.raises(ValueError, match=n):
                lay.backward(x, x, grads={**good, n: bad}, stream=0)
