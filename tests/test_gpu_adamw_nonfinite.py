"""8-bit states after gradients that fp32 cannot square, and after NaN and infinite ones:
only the elements that had them are lost, as with fp32 states; the others of their
block go on as if those were not there, for any number of steps."""
import pytest
import torch

from tests.gpu_util import load_moe
from tests.test_gpu_adamw import BF, E4, F32, copy, entry, reference, step_of, wide

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module")
def moe():
    return load_moe()


def others_are_right(before, after, h, lost, stochastic):
    """Every element but the `lost` ones against the 64-bit step; scales from the
    largest finite magnitude of the block."""
    r, n = reference(before, h), lost.numel()
    store = 0.0 if after["param"].dtype == F32 else 2.0 ** -7 if stochastic else 2.0 ** -8
    stepped = after.get("master") if after.get("master") is not None else after["param"]
    store = 0.0 if after.get("master") is not None else store
    err = (stepped.double() - r["p"]).abs()
    assert (err <= r["p_tol"] + store * (r["p"].abs() + r["p_tol"]) + 2.0 ** -133)[~lost].all()
    for name, x, tol in (("exp_avg", r["m"], r["m_tol"]),
                         ("exp_avg_sq", r["v"].sqrt(), 8 * U * r["v"].sqrt() + 2.0 ** -70)):
        s = after[name + "_scale"].double()
        pad = torch.zeros(s.numel() * 256, dtype=torch.float64, device="cuda")
        # (finite in fp32)
        value = x if name == "exp_avg" else x * x
        pad[:n] = torch.where(value.abs() < 2.0 ** 128, x.abs(), torch.zeros_like(x))
        top = pad.view(-1, 256).amax(1)
        assert (top < 256 * s * (1 + 16 * U)).all() and \
            (top >= 128 * s * (1 - 16 * U)).logical_or(s <= 2.0 ** -126).all(), name
        each = s.repeat_interleave(256)[:n]
        got = after[name].double() * each
        floor = torch.where(x > 0, 2.0 ** -9 * each, 0.0) if name == "exp_avg_sq" else torch.zeros_like(x)
        near = (got - x).abs() <= step_of(x.abs() + tol, each) * (1 + 2.0 ** -16) + tol
        assert (near | (got == floor))[~lost].all(), name
        if name == "exp_avg_sq":
            assert ((got > 0) == (x > 0))[~lost].all()


@pytest.mark.parametrize("kind", [dict(p=BF, g=F32), dict(p=BF, g=BF), dict(p=F32, g=F32),
                                  dict(p=BF, g=F32, master=True)])
@pytest.mark.parametrize("value", [1e20, -3e38, NAN, INF, -INF])
def test_one_element_does_not_cost_its_block(moe, value, kind):
    n = 1500
    e = entry(n, 4, bits=8, **kind)
    good = e["grad"].clone()
    at = [7, 300, 301, 1499]
    lost = torch.zeros(n, dtype=torch.bool, device="cuda")
    lost[at] = True
    whole = entry(n, 4, bits=32, **kind)  # fp32 states: the same elements, stepped beside
    arr, ref = moe.adamw_list([e]), moe.adamw_list([whole])
    for step in range(1, 9):
        for x in (e, whole):
            x["grad"].copy_(good)
            if step == 1:
                x["grad"][at] = value
            elif step > 4:
                x["grad"][~lost] *= 0.0 if step % 2 else 0.5
        before, h = copy(e), dict(lr=1e-2, beta1=0.9, beta2=0.95, eps=1e-8, step=step)
        hyper = moe.adamw_hyper(**h, seed=step, stochastic=True)
        moe.moe_adamw_step(arr, hyper)
        moe.moe_adamw_step(ref, hyper)
        torch.cuda.synchronize()
        assert moe.moe_last_device_error() == moe.MOE_OK
        # (a huge m is the block's largest magnitude: the others' m have its scale)
        others_are_right(before, e, h, lost, True)
        # what is lost is lost as with fp32 states: a NaN, or a parameter that only decays
        p, q = e["param"].float()[lost], whole["param"].float()[lost]
        assert torch.equal(torch.isnan(p), torch.isnan(q))
        if torch.isfinite(torch.tensor(value)):
            assert torch.isinf(whole["exp_avg_sq"][lost]).all()
            # (eight roundings to one of two neighbours)
            assert ((p - q).abs() <= 8 * 2.0 ** -7 * q.abs()).all()


def test_codes_of_what_is_lost(moe):
    """NaN as NaN, an infinite m as the largest value, an infinite v as a negative NaN,
    which the next step reads as infinite."""
    e = entry(512, 5, p=F32, g=F32, bits=8, wd=0.0)
    e["grad"][[3, 300]], e["grad"][[4, 301]] = NAN, torch.tensor([INF, -INF], device="cuda")
    e["grad"][5] = 1e25
    moe.moe_adamw_step(moe.adamw_list([e]), moe.adamw_hyper(1e-2))
    m, r = e["exp_avg"].view(torch.uint8), e["exp_avg_sq"].view(torch.uint8)
    assert m[[3, 300]].tolist() == [0x7f, 0x7f] and m[[4, 301]].tolist() == [0x7e, 0xfe]
    assert r[[3, 300]].tolist() == [0x7f, 0x7f] and r[[4, 301, 5]].tolist() == [0xff] * 3
    before = e["param"].clone()
    e["grad"].zero_()
    moe.moe_adamw_step(moe.adamw_list([e]), moe.adamw_hyper(1e-2, step=2))
    assert e["param"][5] == before[5] and r[5] == 0xff


def test_zeros_of_either_sign_are_zeros(moe):
    """r of -0 (another program's state) is 0."""
    out = []
    for code in (0x00, 0x80):
        e = entry(600, 6, p=F32, g=F32, bits=8)
        e["exp_avg_sq"].view(torch.uint8)[::3] = code
        moe.moe_adamw_step(moe.adamw_list([e]), moe.adamw_hyper(1e-2))
        out.append(e)
    for name in ("param", "exp_avg", "exp_avg_sq"):
        assert torch.equal(*(e[name].view(torch.uint8) for e in out)), name
