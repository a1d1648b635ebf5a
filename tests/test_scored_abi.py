"""Refusals and size queries of scored routing, the balance bias and AdamW:
each call here returns before it touches a device."""
import ctypes
import math
import weakref
from types import SimpleNamespace

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
KW = dict(stream=0, raise_on_error=False)


def calls(moe, cfg, r, a=None, n=BIG):
    """Every entry, with the arguments of `a` (name -> address) replaced."""
    v = dict.fromkeys("x Wr lb bb L idx w dw dx_in dl dWr db dx ws Wgu Wd out fws dout dWgu dWd".split(), A)
    v["ws"] = 2 * A
    v.update(a or {})
    g = v.__getitem__
    return {
        "route": lambda: moe.moe_route_scored(cfg, r, g("x"), g("Wr"), g("lb"), g("bb"), g("L"), g("idx"),
                                              g("w"), g("ws"), n, **KW),
        "from_logits": lambda: moe.moe_route_scored_from_logits(cfg, r, g("L"), g("bb"), g("idx"), g("w"),
                                                                **KW),
        "logits_grad": lambda: moe.moe_route_scored_from_logits_backward(
            cfg, r, g("L"), g("idx"), g("w"), g("dw"), g("dl"), **KW),
        "route_grad": lambda: moe.moe_route_scored_backward(
            cfg, r, g("x"), g("Wr"), g("L"), g("idx"), g("w"), g("dw"), g("dx_in"), g("dl"), g("dWr"),
            g("db"), g("dx"), g("ws"), n, **KW),
        "forward": lambda: moe.moe_forward_scored(cfg, r, g("x"), g("Wr"), g("lb"), g("bb"), g("Wgu"),
                                                  g("Wd"), g("out"), g("ws"), n, **KW),
        "backward": lambda: moe.moe_backward_scored(
            cfg, r, g("x"), g("Wr"), g("Wgu"), g("Wd"), g("fws"), g("dout"), g("dx"), g("dWr"), g("db"),
            g("dWgu"), g("dWd"), g("ws"), n, n, **KW),
    }


BASE = dict(T=16, d=64, E=128, k=4, f=64)


@pytest.mark.parametrize("bad,code", [
    (dict(score=2), -2), (dict(score=-1), -2), (dict(group_score=2), -2), (dict(groups=0), -1),
    (dict(groups=3), -1), (dict(groups=256), -1), (dict(groups=64), -2), (dict(groups=8, topk_groups=0), -1),
    (dict(groups=8, topk_groups=9), -1), (dict(groups=32, topk_groups=0), -1),
    (dict(weight_scale=0.0), -1), (dict(weight_scale=-1.0), -1), (dict(weight_scale=math.inf), -1),
    (dict(weight_scale=math.nan), -1)])
def test_bad_routers(moe, bad, code):
    cfg = moe.config(**BASE)
    r = moe.router(**bad)
    for name, call in calls(moe, cfg, r).items():
        assert call() == code, name
        assert moe.moe_last_error_message()
    assert moe.moe_route_scored_backward_workspace_size(cfg, r) == 0
    assert moe.moe_backward_scored_workspace_size(cfg, r) == 0


def test_too_few_experts_in_the_groups(moe):
    cfg = moe.config(**{**BASE, "k": 17})
    for name, call in calls(moe, cfg, moe.router(groups=8, topk_groups=1)).items():
        assert call() == -1, name


@pytest.mark.parametrize("bad,code", [
    (dict(T=-1), -1), (dict(d=12), -1), (dict(k=129), -1), (dict(E=2048), -2), (dict(dtype=2), -2),
    (dict(dtype=7), -2)])
def test_bad_configs(moe, bad, code):
    cfg = moe.config(**{**BASE, **bad})
    for name, call in calls(moe, cfg, moe.router()).items():
        assert call() == code, name


def test_null_and_misaligned_arguments(moe):
    takes = {"route": "x Wr L idx w ws", "from_logits": "L idx w", "logits_grad": "L idx w dw dl",
             "route_grad": "x Wr L idx w dw dl dWr dx ws", "forward": "x Wr Wgu Wd out ws",
             "backward": "x Wr Wgu Wd fws dout dx dWr dWgu dWd ws"}
    optional = {"route": "lb bb", "from_logits": "bb", "route_grad": "dx_in db", "forward": "lb bb",
                "backward": "db"}
    cfg, r = moe.config(**BASE), moe.router("sigmoid")
    for name, args in takes.items():
        for arg in args.split():
            for value in (None, A + 8):
                assert calls(moe, cfg, r, {arg: value})[name]() == -1, (name, arg, value)
        for arg in optional.get(name, "").split():
            assert calls(moe, cfg, r, {arg: A + 4})[name]() == -1, (name, arg)


def test_null_struct_and_workspace(moe):
    cfg, r = moe.config(**BASE), moe.router()
    lib = ctypes.CDLL(moe.LIB_PATH)
    assert lib.moe_route_scored_from_logits(ctypes.byref(cfg), None, *[ctypes.c_void_p(A)] * 4, None) == -1
    for name in ("route", "route_grad", "forward", "backward"):
        assert calls(moe, cfg, r, n=16)[name]() == -3, name
    assert moe.moe_backward_scored(cfg, r, A, A, A, A, A, A, A, A, A, A, A, A, BIG, BIG, **KW) == -1


def test_sizes(moe):
    """The gradient's workspace goes by which logits have one: sigmoid weights
    that are not renormalised are sparse too."""
    for dtype in ("bf16", "f32"):
        for T, E in ((16, 8), (600, 64), (5000, 128)):
            sizes = {}
            for renorm in (False, True):
                cfg = moe.config(T, 64, E, 4, 64, dtype, renorm)
                plain = moe.moe_route_backward_workspace_size(cfg)
                assert moe.moe_route_scored_backward_workspace_size(cfg, moe.router()) == plain
                assert moe.moe_backward_scored_workspace_size(cfg, moe.router()) == \
                    moe.moe_backward_workspace_size(cfg)
                sizes[renorm] = moe.moe_route_scored_backward_workspace_size(cfg, moe.router("sigmoid"))
            assert sizes[False] == sizes[True] == plain  # the last: renormalised
    empty = moe.config(0, 64, 8, 2, 64)
    assert moe.moe_backward_scored_workspace_size(empty, moe.router()) == 0


def test_empty_batch_launches_nothing(moe):
    cfg, r = moe.config(**{**BASE, "T": 0}), moe.router("sigmoid", 8, 4)
    none = dict.fromkeys("x Wr lb bb L idx w dw dl ws Wgu Wd out".split())
    for name in ("route", "from_logits", "logits_grad", "forward"):
        assert calls(moe, cfg, r, none)[name]() == 0, name
    bad = moe.router("sigmoid", 7)
    assert calls(moe, cfg, bad, none)["forward"]() == -1


@pytest.mark.parametrize("args,code", [
    (dict(layers=-1), -1), (dict(E=0), -1), (dict(E=1025), -2), (dict(layers=2 ** 31), -2),
    (dict(rate=math.nan), -1), (dict(rate=math.inf), -1), (dict(counts=None), -1), (dict(bias=None), -1),
    (dict(counts=A + 1), -1), (dict(bias=A + 2), -1), (dict(imbalance=A + 3), -1), (dict(layers=0), 0)])
def test_balance_bias_refusals(moe, args, code):
    a = {**dict(counts=A, rate=1e-3, bias=A, imbalance=A, layers=1, E=8), **args}
    assert moe.moe_update_balance_bias(a["counts"], a["rate"], a["bias"], a["imbalance"], a["layers"],
                                       a["E"], **KW) == code


def test_balance_bias_shapes(moe):
    n, b = torch.zeros(3, 8, dtype=torch.int32), torch.zeros(3, 8)
    for counts, bias, imb in ((n.long(), b, None), (n, b.double(), None), (n, b[0], None),
                              (n, b, torch.zeros(2)), (n, b, torch.zeros(3).double())):
        with pytest.raises(ValueError):
            moe.moe_update_balance_bias(counts, 1e-3, bias, imb, **KW)


# ----------------------------------- AdamW -----------------------------------
HYPER = dict(lr=1e-3, beta1=0.9, beta2=0.95, eps=1e-8, step=1)


def tensor(moe, **kw):
    t = moe.moe_adamw_tensor_t(A, A, A, A, None, None, None, 100, moe.MOE_BF16, moe.MOE_BF16, moe.MOE_F32,
                               0.1)
    for k, v in kw.items():
        setattr(t, k, v)
    return t


def step(moe, t=None, norm=None, scalars=None, n=1, **hyper):
    arr = (moe.moe_adamw_tensor_t * 1)(t if t is not None else tensor(moe))
    return moe.moe_adamw_step(arr, moe.adamw_hyper(**{**HYPER, **hyper}), norm, scalars, n=n, **KW)


@pytest.mark.parametrize("bad", [
    dict(lr=-1.0), dict(lr=math.nan), dict(lr=math.inf), dict(beta1=1.0), dict(beta1=-0.1),
    dict(beta2=1.0), dict(beta2=math.nan), dict(eps=-1e-8), dict(eps=math.inf), dict(step=0),
    dict(step=-3), dict(n=-1), dict(norm=A + 2), dict(scalars=A + 8), dict(norm=A, max_norm=-1.0),
    dict(norm=A, max_norm=math.nan)])
def test_adamw_bad_arguments(moe, bad):
    assert step(moe, **bad) == -1
    assert moe.moe_last_error_message()


@pytest.mark.parametrize("bad,code", [
    (dict(param=None), -1), (dict(grad=None), -1), (dict(exp_avg=None), -1), (dict(exp_avg_sq=None), -1),
    (dict(param=A + 1), -1), (dict(grad=A + 1), -1), (dict(exp_avg=A + 2), -1),
    (dict(exp_avg_sq=A + 2), -1), (dict(master=A + 2), -1), (dict(numel=-1), -1),
    (dict(weight_decay=math.nan), -1), (dict(param_dtype=0, master=A), -1), (dict(param_dtype=2), -2),
    (dict(grad_dtype=2), -2), (dict(grad_dtype=5), -2), (dict(state_dtype=1), -2),
    (dict(exp_avg_scale=A), -1), (dict(exp_avg_sq_scale=A), -1), (dict(state_dtype=2), -1),
    (dict(state_dtype=2, exp_avg_scale=A), -1),
    (dict(state_dtype=2, exp_avg_scale=A + 2, exp_avg_sq_scale=A), -1), (dict(numel=2 ** 62), -1)])
def test_adamw_bad_tensors(moe, bad, code):
    assert step(moe, tensor(moe, **bad)) == code
    assert moe.moe_last_error_message()


def test_adamw_null_list_and_hyper(moe):
    lib = ctypes.CDLL(moe.LIB_PATH)
    h = moe.adamw_hyper(**HYPER)
    args = [ctypes.c_void_p(None)] * 3
    assert lib.moe_adamw_step(None, ctypes.c_int64(1), ctypes.byref(h), *args) == -1
    assert lib.moe_adamw_step(None, ctypes.c_int64(0), None, *args) == -1
    assert lib.moe_adamw_scalars(ctypes.byref(h), None) == -1


def test_adamw_scalars(moe):
    s = moe.moe_adamw_scalars(moe.adamw_hyper(0.1, 0.9, 0.99, step=3, seed=(5 << 32) + 7))
    assert (s.seed_lo, s.seed_hi) == (7, 5)
    for got, want in ((s.lr, 0.1), (s.step_size, 0.1 / (1 - 0.9 ** 3)),
                      (s.inv_sqrt_bc2, (1 - 0.99 ** 3) ** -0.5)):
        assert abs(got - want) <= 2.0 ** -24 * want
    assert ctypes.sizeof(s) == 32


def test_adamw_list_refuses(moe):
    def t(n=300, p=torch.bfloat16, **kw):
        d = dict(param=torch.zeros(n, dtype=p), grad=torch.zeros(n), exp_avg=torch.zeros(n),
                 exp_avg_sq=torch.zeros(n))
        d.update(kw)
        return d
    assert moe.adamw_list([t(), t(master=torch.zeros(300))]).count == 2
    e4 = torch.zeros(300).to(torch.float8_e4m3fn)
    two = dict(exp_avg=e4, exp_avg_sq=e4.clone(), exp_avg_scale=torch.zeros(2), exp_avg_sq_scale=torch.zeros(2))
    assert moe.adamw_list([t(**two)])[0].state_dtype == moe.MOE_E4M3
    for bad in (dict(p=torch.float16), dict(grad=torch.zeros(300).double()), dict(exp_avg=e4),
                dict(exp_avg=torch.zeros(300, dtype=torch.bfloat16),
                     exp_avg_sq=torch.zeros(300, dtype=torch.bfloat16))):
        with pytest.raises(TypeError):
            moe.adamw_list([t(**bad)])
    for bad in (dict(grad=torch.zeros(299)), dict(exp_avg_sq=torch.zeros(301)),
                dict(p=torch.float32, master=torch.zeros(300)), dict(master=torch.zeros(300).double()),
                dict(exp_avg=e4, exp_avg_sq=e4), dict(exp_avg_scale=torch.zeros(2)),
                dict(**{**two, "exp_avg_scale": torch.zeros(1)}),
                dict(exp_avg=torch.zeros(300, device="meta"))):
        with pytest.raises(ValueError):
            moe.adamw_list([t(**bad)])
    with pytest.raises(ValueError):
        moe.adamw_list([t(param=torch.zeros(600, dtype=torch.bfloat16)[::2])])


def test_adamw_class_refuses(moe):
    p, g = [torch.zeros(300)], [torch.zeros(300)]
    for bad in (dict(params=p, grads=[]), dict(params=[], grads=[]), dict(bits=16),
                dict(weight_decay=[0.1, 0.2]), dict(grads=[torch.zeros(299)])):
        with pytest.raises(ValueError):
            moe.AdamW(**{**dict(params=p, grads=g, lr=1e-3), **bad})


def _plain(**kw):
    z = lambda: torch.zeros(300)
    return {**dict(param=z(), grad=z(), exp_avg=z(), exp_avg_sq=z()), **kw}


def test_adamw_list_refuses_overlapping_tensors(moe):
    a, b = _plain(), _plain()
    moe.adamw_list([a, b])
    moe.adamw_list([a, {**b, "grad": a["grad"]}])  # read only
    buf = torch.zeros(600)
    moe.adamw_list([{**a, "param": buf[:300]}, {**b, "param": buf[300:]}])
    for bad in ([a, a], [a, {**b, "param": a["param"]}], [a, {**b, "exp_avg_sq": a["exp_avg"]}],
                [{**a, "param": buf[:300]}, {**b, "param": buf[299:599]}]):
        with pytest.raises(ValueError):
            moe.adamw_list(bad)
    with pytest.raises(ValueError):
        moe.AdamW([buf, buf], [torch.zeros(600)] * 2, lr=1e-3)
    m = lambda: torch.zeros(300, device="meta")
    with pytest.raises(ValueError):
        moe.adamw_list([a, dict(param=m(), grad=m(), exp_avg=m(), exp_avg_sq=m())])


class _Elsewhere(torch.Tensor):
    device = property(lambda self: torch.device("cuda", 1))


def test_tensors_off_the_current_gpu_are_refused(moe, monkeypatch):
    launched = []
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(moe, "_stream", lambda s: 0)
    monkeypatch.setattr(moe, "_lib", SimpleNamespace(
        moe_adamw_step=lambda *a: launched.append(a) or 0))
    hyper = moe.adamw_hyper(1e-3)
    with pytest.raises(ValueError):  # host memory
        moe.moe_adamw_step(moe.adamw_list([_plain()]), hyper)
    with pytest.raises(ValueError):
        moe.AdamW([torch.zeros(300)], [torch.zeros(300)], lr=1e-3).step()
    there = moe.adamw_list([{n: x.as_subclass(_Elsewhere) for n, x in _plain().items()}])
    with pytest.raises(ValueError):
        moe.moe_adamw_step(there, hyper)
    assert not launched
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 1)
    moe.moe_adamw_step(there, hyper)
    assert len(launched) == 1


@pytest.mark.parametrize("hyper,ok", [(dict(eps=0.0), True), (dict(eps=2.0 ** -126), True),
                                      (dict(eps=2.0 ** -127), False), (dict(eps=1e-60), False),
                                      (dict(lr=1e300), False), (dict(eps=1e300), False)])
def test_adamw_hyperparameters_as_floats(moe, hyper, ok):
    h = moe.adamw_hyper(**{**dict(lr=1e-3), **hyper})
    if ok:
        moe.moe_adamw_scalars(h)
    else:
        with pytest.raises(moe.MoEError):
            moe.moe_adamw_scalars(h)


@pytest.mark.parametrize("scale,ok", [(2.0 ** -100, True), (2.0 ** 100, True), (2.0 ** -101, False),
                                      (1e-40, False), (2.0 ** 101, False)])
def test_weight_scales(moe, scale, ok):
    s = moe.moe_route_scored_from_logits(moe.config(0, 8, 16, 4, 8), moe.router(weight_scale=scale),
                                         None, None, None, None, stream=0, raise_on_error=False)
    assert (s == moe.MOE_OK) is ok


def test_a_captured_balance_update_keeps_its_workspace(moe, monkeypatch):
    class OnDevice(torch.Tensor):
        is_cuda = property(lambda self: True)

    capturing = [False]
    monkeypatch.setattr(moe, "_stream", lambda s: 7 if s is None else int(s))
    monkeypatch.setattr(moe, "_on_current", lambda device: None)
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: capturing[0])
    empty = torch.empty
    monkeypatch.setattr(torch, "empty", lambda *a, **kw: empty(*a, **kw).as_subclass(OnDevice))
    monkeypatch.setattr(moe, "moe_forward_scored", lambda *a, **kw: None)
    monkeypatch.setattr(moe, "moe_update_balance_bias", lambda *a, **kw: None)
    bf = torch.bfloat16
    lay = moe.MoELayer(torch.zeros(8, 64), torch.zeros(8, 64, 256, dtype=bf),
                       torch.zeros(8, 128, 64, dtype=bf), 2, router=moe.router("sigmoid"),
                       balance_bias=torch.zeros(8))
    lay(torch.zeros(16, 64, dtype=bf))
    capturing[0] = True
    lay.update_balance_bias(1e-3)
    capturing[0] = False
    held = weakref.ref(next(iter(lay._ws.values())))
    lay(torch.zeros(4000, 64, dtype=bf))
    assert held() is not None


def test_layer_refuses(moe):
    w = torch.zeros(8, 64), torch.zeros(8, 64, 128), torch.zeros(8, 64, 64)
    with pytest.raises(ValueError):
        moe.MoELayer(*w, 2, balance_bias=torch.zeros(8))
    for b in (torch.zeros(7), torch.zeros(8).double(), torch.zeros(8, device="meta")):
        with pytest.raises(ValueError):
            moe.MoELayer(*w, 2, router=moe.router(), balance_bias=b)
