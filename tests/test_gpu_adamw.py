"""moe_adamw_step against a 64-bit step from the same inputs.

With u = 2^-24: m is two products and a sum, with b1 and 1 - b1 rounded once, and
the clipped gradient three roundings: within 8 u of b1 |m| + (1 - b1) |g|.  v the
same with the square: 12 u of itself (all terms positive).  The update is
step m / (r i + eps): m's error, and below 16 u of itself (root 1 + 6, quotient 2
ulp, step and i rounded once, their products).  The decay 1 - lr wd is rounded
twice, its product and the last sum once: 4 u of |p|.  Storage in bf16 adds 2^-8
of |p| (nearest) or 2^-7 (one of both neighbours).

8-bit states: a value lies between its neighbours in e4m3 times the block's
scale: 2^-3 of itself, or 2^-9 of the scale, at most."""
import pytest
import torch

from tests.gpu_util import load_moe

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
BF, F32, E4 = torch.bfloat16, torch.float32, torch.float8_e4m3fn
HYPER = dict(lr=1e-2, beta1=0.9, beta2=0.95, eps=1e-8, step=7)


@pytest.fixture(scope="module")
def moe():
    return load_moe()


def entry(n, seed, p=BF, g=BF, bits=32, master=False, wd=0.1, shift=0):
    """One parameter with its states; shift: elements by which every pointer is
    off an allocation's start."""
    gen = torch.Generator(device="cuda").manual_seed(seed)

    def rand(dt):
        return torch.randn(n + shift, generator=gen, device="cuda").to(dt)[shift:]
    e = dict(param=rand(p), grad=rand(g), weight_decay=wd)
    if master:
        e["master"] = rand(F32)
    if bits == 32:
        e["exp_avg"], e["exp_avg_sq"] = rand(F32).mul_(0.1), rand(F32).square_()
    else:
        nb = -(-n // 256)
        for name, low in (("exp_avg", -240), ("exp_avg_sq", 0)):
            codes = torch.empty(n + shift, device="cuda").uniform_(low, 240, generator=gen).to(E4)
            e[name] = codes.view(torch.uint8)[shift:].view(E4)
            e[name + "_scale"] = torch.exp2(torch.randint(-16, -6, (nb,), generator=gen,
                                                          device="cuda").float())
    return e


def copy(e):
    out = {}
    for k, v in e.items():
        if isinstance(v, torch.Tensor):  # the same offset from an allocation's start
            raw = v.view(torch.uint8) if v.dtype == E4 else v
            buf = torch.empty(raw.storage_offset() + raw.numel(), dtype=raw.dtype, device="cuda")
            part = buf[raw.storage_offset():]
            part.copy_(raw.reshape(-1))
            v = part.view(E4) if v.dtype == E4 else part
        out[k] = v
    return out


def wide(e, name):
    x = e[name].double()
    if e[name].dtype == E4:
        x = x * e[name + "_scale"].double().repeat_interleave(256)[:x.numel()]
        return x * x if name == "exp_avg_sq" else x
    return x


def reference(e, h, coef=1.0):
    g = e["grad"].double() * coef
    m, v = wide(e, "exp_avg"), wide(e, "exp_avg_sq")
    mag = h["beta1"] * m.abs() + (1 - h["beta1"]) * g.abs()
    m = h["beta1"] * m + (1 - h["beta1"]) * g
    v = h["beta2"] * v + (1 - h["beta2"]) * g * g
    p = (e["master"] if e.get("master") is not None else e["param"]).double()
    step = h["lr"] / (1 - h["beta1"] ** h["step"])
    denom = v.sqrt() / (1 - h["beta2"] ** h["step"]) ** 0.5 + h["eps"]
    new = p * (1 - h["lr"] * e["weight_decay"]) - step * m / denom
    tol = 4 * U * p.abs() + step * 8 * U * mag / denom + 16 * U * (step * m / denom).abs() + 2.0 ** -149
    return dict(p=new, m=m, v=v, m_tol=8 * U * mag + 2.0 ** -149, p_tol=tol)


def power(e):
    """2^e, exactly (ldexp and exp2 are not, on the GPU)."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def step_of(x, scale):
    """Distance of x's neighbours in e4m3 times scale (both per element)."""
    e = (torch.frexp(x.abs() / scale).exponent - 1).clamp(min=-6)
    return scale * power(e - 3)


def verify(before, after, h, coef=1.0, stochastic=False):
    r = reference(before, h, coef)
    p = after["param"].double()
    if after.get("master") is not None:
        assert ((after["master"].double() - r["p"]).abs() <= r["p_tol"]).all()
        assert torch.equal(after["param"], after["master"].to(BF))
    else:
        store = 0.0 if after["param"].dtype == F32 else 2.0 ** -7 if stochastic else 2.0 ** -8
        assert ((p - r["p"]).abs() <= r["p_tol"] + store * (r["p"].abs() + r["p_tol"]) +
                (2.0 ** -133 if store else 0)).all()
    if after["exp_avg"].dtype == F32:
        assert ((after["exp_avg"].double() - r["m"]).abs() <= r["m_tol"]).all()
        assert ((after["exp_avg_sq"].double() - r["v"]).abs() <= 12 * U * r["v"] + 2.0 ** -140).all()
        return
    n = p.numel()
    for name, x, tol in (("exp_avg", r["m"], r["m_tol"]),
                         ("exp_avg_sq", r["v"].sqrt(), 8 * U * r["v"].sqrt() + 2.0 ** -70)):
        scale = after[name + "_scale"].double()
        pad = torch.zeros(scale.numel() * 256, dtype=torch.float64, device="cuda")
        pad[:n] = x.abs()
        top = pad.view(-1, 256).amax(1)
        # 2^(e-7) with 2^e <= the largest < 2^(e+1), to the rounding of the largest
        assert (torch.frexp(scale).mantissa == 0.5).all()  # powers of two
        assert (top < 256 * scale * (1 + 16 * U)).all() and \
            (top >= 128 * scale * (1 - 16 * U)).logical_or(scale <= 2.0 ** -126).all()
        s = scale.repeat_interleave(256)[:n]
        got = after[name].double() * s
        floor = torch.where(x > 0, 2.0 ** -9 * s, 0.0) if name == "exp_avg_sq" else torch.zeros_like(x)
        near = (got - x).abs() <= step_of(x.abs() + tol, s) * (1 + 2.0 ** -16) + tol
        assert (near | (got == floor)).all()
        if name == "exp_avg_sq":
            assert ((got > 0) == (x > 0)).all()


def run(moe, entries, h=HYPER, norm=None, max_norm=0.0, seed=3, stochastic=False, **kw):
    moe.moe_adamw_step(moe.adamw_list(entries), moe.adamw_hyper(**h, seed=seed, max_norm=max_norm,
                                                                stochastic=stochastic), norm, **kw)
    torch.cuda.synchronize()
    assert moe.moe_last_device_error() == moe.MOE_OK


KINDS = [dict(p=F32, g=F32), dict(p=F32, g=BF), dict(p=BF, g=BF), dict(p=BF, g=F32),
         dict(p=BF, g=BF, master=True), dict(p=BF, g=F32, master=True)]


@pytest.mark.parametrize("stochastic", [False, True])
@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("kind", range(len(KINDS)))
def test_types_and_sizes(moe, kind, bits, stochastic):
    sizes = [1, 7, 8, 9, 255, 256, 257, 1000, 16383, 16384, 16385, 70001]
    es = [entry(n, 10 * n + kind, bits=bits, wd=0.1 * (i % 2), **KINDS[kind]) for i, n in enumerate(sizes)]
    before = [copy(e) for e in es]
    run(moe, es, stochastic=stochastic)
    for b, a in zip(before, es):
        verify(b, a, HYPER, stochastic=stochastic)
        assert torch.equal(b["grad"], a["grad"])


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("shift", [1, 2, 4, 8])
def test_pointers_off_16_bytes(moe, shift, bits):
    """Every tensor off its allocation's start, and the elements before and
    after it left as they were."""
    for kind in KINDS:
        e = entry(5001, shift, bits=bits, shift=shift, **kind)
        whole = torch.full((5001 + 64,), 7.0, dtype=e["param"].dtype, device="cuda")
        whole[shift:shift + 5001] = e["param"]
        e["param"] = whole[shift:shift + 5001]
        before = copy(e)
        run(moe, [e])
        verify(before, e, HYPER)
        assert (whole[:shift] == 7).all() and (whole[shift + 5001:] == 7).all()


@pytest.mark.parametrize("n", [299, 300, 301, 1300])
def test_many_tensors(moe, n):
    es = [entry(1 + (37 * i) % 900, i, bits=8 if i % 3 == 1 else 32, **KINDS[i % 6]) for i in range(n)]
    before = [copy(e) for e in es]
    run(moe, es)
    for b, a in zip(before, es):
        verify(b, a, HYPER)


def test_no_and_empty_tensors(moe):
    run(moe, [])
    es = [entry(0, 1), entry(300, 2), entry(0, 3, bits=8), entry(300, 4, bits=8)]
    before = [copy(e) for e in es]
    run(moe, es)
    for b, a in zip(before[1::2], es[1::2]):
        verify(b, a, HYPER)


@pytest.mark.parametrize("hyper", [dict(step=1), dict(lr=0.0), dict(eps=0.0), dict(beta1=0.0, beta2=0.0),
                                   dict(step=10 ** 9), dict(beta2=0.999, step=2)])
@pytest.mark.parametrize("bits", [32, 8])
def test_hyperparameters(moe, hyper, bits):
    h = {**HYPER, **hyper}
    e = entry(3000, 5, p=F32, g=F32, bits=bits)
    before = copy(e)
    run(moe, [e], h)
    verify(before, e, h)


def test_first_steps_from_zero_states(moe):
    """Zeros in all bytes are valid states; an element without gradients keeps them."""
    for bits in (32, 8):
        e = entry(1000, 6, p=F32, g=F32, bits=bits)
        for name in ("exp_avg", "exp_avg_sq", "exp_avg_scale", "exp_avg_sq_scale"):
            if name in e:
                e[name].view(torch.uint8).zero_()
        e["grad"][::5] = 0
        e["grad"][512:768] = 0
        for step in (1, 2, 3):
            before = copy(e)
            run(moe, [e], {**HYPER, "step": step})
            verify(before, e, {**HYPER, "step": step})
        assert not e["exp_avg"].double()[::5].any() and not e["exp_avg_sq"].double()[::5].any()


@pytest.mark.parametrize("norm,max_norm", [(0.5, 1.0), (4.0, 1.0), (4.0, 0.0), (0.0, 1.0)])
def test_clipping_by_a_given_norm(moe, norm, max_norm):
    for bits in (32, 8):
        e = entry(3000, 7, bits=bits)
        before = copy(e)
        run(moe, [e], norm=torch.full((1,), norm, device="cuda"), max_norm=max_norm)
        verify(before, e, HYPER, min(1.0, max_norm / (norm + 1e-6)))


@pytest.mark.parametrize("value", [float("inf"), float("nan")])
def test_a_step_without_a_finite_norm_is_skipped(moe, value):
    for bits in (32, 8):
        e = entry(3000, 8, bits=bits, master=True)
        before = copy(e)
        norm = torch.full((1,), value, device="cuda")
        moe.moe_adamw_step(moe.adamw_list([e]), moe.adamw_hyper(**HYPER, max_norm=1.0,
                                                                skip_nonfinite=True), norm)
        for k, v in e.items():
            if isinstance(v, torch.Tensor):
                assert torch.equal(v.view(torch.uint8), before[k].view(torch.uint8)), k


@pytest.mark.parametrize("bits", [32, 8])
def test_nonfinite_gradients_stay_with_their_elements(moe, bits):
    """... of the parameters: an 8-bit block's other states lose their scale."""
    e = entry(2048, 9, p=BF, g=F32, bits=bits)
    e["grad"][5], e["grad"][1000] = float("nan"), float("inf")
    before = copy(e)
    run(moe, [e], stochastic=True)
    bad = torch.zeros(2048, dtype=torch.bool, device="cuda")
    bad[5] = bad[1000] = True
    assert torch.isnan(e["param"][bad]).all()
    assert torch.isfinite(e["param"][~bad].float()).all()
    assert torch.isnan(e["exp_avg"].float()[5]) and torch.isnan(e["exp_avg_sq"].float()[5])
    if bits == 32:
        r = reference(before, HYPER)
        assert ((e["exp_avg"].double() - r["m"]).abs() <= r["m_tol"])[~bad].all()


def test_rounding_is_right_on_average(moe):
    """2^20 equal elements: the mean of the rounded values is the value to 5
    standard deviations of that many throws, for parameters and both states."""
    n = 1 << 20
    h = dict(lr=1.0, beta1=0.9, beta2=0.95, eps=1e-8, step=10 ** 9)

    def filled(x, dt):
        return torch.full((n,), x, device="cuda", dtype=dt)
    e = dict(param=filled(1.0, BF), grad=filled(0.3711, F32), exp_avg=filled(0.0, E4),
             exp_avg_sq=filled(0.0, E4), exp_avg_scale=torch.ones(n // 256, device="cuda"),
             exp_avg_sq_scale=torch.ones(n // 256, device="cuda"), weight_decay=0.0)
    e["grad"][::256] = 1.0  # sets the scale
    r = reference(e, h)
    run(moe, [e], h, stochastic=True)
    pick = torch.ones(n, dtype=torch.bool, device="cuda")
    pick[::256] = False
    s = e["exp_avg_scale"].double().repeat_interleave(256), \
        e["exp_avg_sq_scale"].double().repeat_interleave(256)
    for got, want in ((e["param"].double(), r["p"]), (e["exp_avg"].double() * s[0], r["m"]),
                      (e["exp_avg_sq"].double() * s[1], r["v"].sqrt())):
        x = got[pick]
        lo, hi = float(x.min()), float(x.max())
        value = float(want[1])
        assert x.unique().numel() == 2 and lo < value < hi
        share = (value - lo) / (hi - lo)
        sd = (hi - lo) * (share * (1 - share) / x.numel()) ** 0.5
        # (16 bits of chance: 2^-16 of a step)
        assert abs(float(x.mean()) - value) <= 5 * sd + (hi - lo) * 2.0 ** -16


def test_long_run_of_8_bit_states(moe):
    """Gradients of a known size for 400 steps: r settles at it (a state rounded
    to the nearest sticks at twice the size)."""
    gen = torch.Generator(device="cuda").manual_seed(1)
    n = 1 << 16
    size = torch.exp(torch.randn(n, generator=gen, device="cuda"))
    e = entry(n, 2, p=F32, g=F32, bits=8)
    for name in ("exp_avg", "exp_avg_sq", "exp_avg_scale", "exp_avg_sq_scale"):
        e[name].view(torch.uint8).zero_()
    arr, acc, k = moe.adamw_list([e]), 0.0, 0
    for t in range(1, 401):
        e["grad"].copy_(torch.randn(n, generator=gen, device="cuda") * size)
        moe.moe_adamw_step(arr, moe.adamw_hyper(**{**HYPER, "lr": 0.0, "step": t}, seed=t))
        if t > 200 and t % 10 == 0:
            acc, k = acc + wide(e, "exp_avg_sq"), k + 1
    ratio = (acc / k / size.double().square()).mean()
    assert 0.9 <= float(ratio) <= 1.15


def test_repeats_and_seeds(moe):
    es = [entry(5000, 1, bits=8), entry(700, 2, bits=8), entry(3000, 3)]

    def go(seed, order=(0, 1, 2)):
        mine = [copy(e) for e in es]
        run(moe, [mine[i] for i in order], seed=seed, stochastic=True)
        return [torch.cat([m["param"].view(torch.uint8), m["exp_avg"].view(torch.uint8)]) for m in mine]
    a, b, c = go(5), go(5), go(6)
    assert all(torch.equal(x, y) for x, y in zip(a, b))
    assert all(not torch.equal(x, y) for x, y in zip(a, c))
    # the numbers go by the block's place in the list, whatever the launches
    assert not torch.equal(go(5, (1, 0, 2))[0], a[0]) and torch.equal(go(5, (1, 0, 2))[2], a[2])
    assert all(not torch.equal(x, y) for x, y in zip(a, go(5 + (1 << 32))))


M32 = 0xFFFFFFFF
CONST = (0x9E3779B1, 0xD6E8FEB9, 0xA24BAED5, 0xCA5A8263)


def fold(a, c):
    """High and low words of the 32-bit product, xor'ed."""
    a = a & M32
    hi = (a * (c >> 16) + ((a * (c & 0xFFFF)) >> 16)) >> 16
    return (hi ^ (a * (c & 0xFFFF) + (((a * (c >> 16)) & 0xFFFF) << 16))) & M32


def random_bits(block, seed):
    x = fold(block + CONST[0], CONST[1])
    x = fold(x ^ (seed & M32), CONST[2])
    x = fold(x + (seed >> 32) + (block >> 32), CONST[3])
    y = fold(x ^ CONST[0], CONST[3])
    place = torch.arange(256, device="cuda") * CONST[0]
    return fold(fold(x[:, None] + place, CONST[2]) ^ y[:, None], CONST[1]).view(-1)


@pytest.mark.parametrize("seed", [0, 12345, (7 << 32) + 99])
def test_the_random_numbers(moe, seed):
    """Bits 0 to 15 round a bf16 parameter, 8 to 23 m and 16 to 31 r: away from
    zero where the part of a step that is lost, plus the bits' part, reaches one.
    (But for values whose fp32 rounding decides: under 1 in 10,000.)"""
    skip, n = 700, 50_000
    es = [entry(skip, 1), entry(n, 2, p=BF, g=F32, bits=8)]
    before = copy(es[1])
    run(moe, es, seed=seed, stochastic=True)
    r = reference(before, HYPER)
    blocks = torch.arange(-(-n // 256), device="cuda") + -(-skip // 256)
    u = random_bits(blocks, seed)[:n]

    def check(got, x, step, bits):
        low = torch.floor(x.abs() / step)
        up = (x.abs() / step - low + (bits.double() + 0.5) / 65536) >= 1
        want = torch.copysign((low + up) * step, x)
        assert float((got != want).double().mean()) < 1e-4
        assert float(up.double().mean()) > 0.2
    p = r["p"]
    e = (torch.frexp(p.abs()).exponent - 1).clamp(min=-126)
    check(es[1]["param"].double(), p, power(e - 7), u & 0xFFFF)
    for name, x, bits in (("exp_avg", r["m"], (u >> 8) & 0xFFFF), ("exp_avg_sq", r["v"].sqrt(), u >> 16)):
        s = es[1][name + "_scale"].double().repeat_interleave(256)[:n]
        got = es[1][name].double() * s
        if name == "exp_avg_sq":  # (the smallest code instead of zero)
            keep = x > 2.0 ** -9 * s
            check(got[keep], x[keep], step_of(x, s)[keep], bits[keep])
        else:
            check(got, x, step_of(x, s), bits)


def test_the_moments_are_rounded_products_and_sums(moe):
    """Bit for bit, whole blocks and the last one: 8-bit scales hang on the last bit."""
    e = entry(1_000_003, 4, p=F32, g=F32)
    b1, c1, b2, c2 = (torch.tensor(x, dtype=F32, device="cuda") for b in ("beta1", "beta2")
                      for x in (HYPER[b], 1 - HYPER[b]))
    m = e["exp_avg"] * b1 + e["grad"] * c1
    v = e["exp_avg_sq"] * b2 + (e["grad"] * e["grad"]) * c2
    run(moe, [e])
    assert torch.equal(e["exp_avg"], m) and torch.equal(e["exp_avg_sq"], v)


def test_a_random_part_is_centred_in_its_step(moe):
    """The same for m alone, whose fp32 value two rounded products and a sum give:
    only where the lost part and the bits' part sum to one (exactly: 2^-20 of all) may
    either neighbour be taken.  (To 2^-20: a magnitude below 2^-6 of the scale may have
    bits that its sum with the random part, a float below 2^-5, rounds away: 2^-30,
    or 2^-21 of a step of 2^-9; the part itself is off by 2^-27 2^-6, 2^-24 of one.)
    Half a number off would turn 2^-17 of them."""
    n = 1 << 22
    e = entry(n, 5, p=F32, g=F32, bits=8)
    old = e["exp_avg"].float() * e["exp_avg_scale"].repeat_interleave(256)
    b1, c1 = (torch.tensor(x, dtype=F32, device="cuda") for x in (HYPER["beta1"], 1 - HYPER["beta1"]))
    m = old * b1 + e["grad"] * c1
    run(moe, [e], seed=77)
    s = e["exp_avg_scale"].double().repeat_interleave(256)
    step = step_of(m.double(), s)
    bits = (random_bits(torch.arange(n // 256, device="cuda"), 77) >> 8) & 0xFFFF
    low = torch.floor(m.double().abs() / step)
    part = m.double().abs() / step - low + (bits.double() + 0.5) / 65536
    want = torch.copysign((low + (part >= 1)) * step, m.double())
    off = e["exp_avg"].double() * s != want
    assert not (off & ((part - 1).abs() > 2.0 ** -20)).any()
    assert int(off.sum()) <= 16  # (4 expected)


def test_streams_and_graph(moe):
    """Two lists on two streams at once; a captured step that is replayed with
    new scalars, equal to eager steps bit for bit."""
    sides = [torch.cuda.Stream(), torch.cuda.Stream()]
    es = [entry(200_000, i, bits=8 if i else 32) for i in range(2)]
    ref = [copy(e) for e in es]
    for e in ref:
        run(moe, [e], stochastic=True)
    torch.cuda.synchronize()
    for e, s in zip(es, sides):
        moe.moe_adamw_step(moe.adamw_list([e]), moe.adamw_hyper(**HYPER, seed=3, stochastic=True),
                           stream=s)
    torch.cuda.synchronize()
    for a, b in zip(es, ref):
        for k in a:
            if isinstance(a[k], torch.Tensor):
                assert torch.equal(a[k].view(torch.uint8), b[k].view(torch.uint8))

    for bits in (32, 8):
        runs = []
        for captured in (False, True):
            gen = torch.Generator(device="cuda").manual_seed(4)
            p = [torch.randn(n, generator=gen, device="cuda").to(BF) for n in (3000, 77)]
            g = [torch.empty_like(x) for x in p]
            opt = moe.AdamW(p, g, 1e-2, weight_decay=[0.1, 0.0], bits=bits, master=False, max_norm=1.0,
                            seed=9, capturable=captured)
            if captured:
                for x in g:
                    x.zero_()
                torch.cuda.synchronize()
                graph = torch.cuda.CUDAGraph()
                with torch.cuda.graph(graph):
                    opt.step()
            for t in range(5):
                for x in g:
                    x.copy_(torch.randn(x.numel(), generator=gen, device="cuda"))
                opt.lr = 1e-2 / (t + 1)
                if captured:
                    opt.advance()
                    graph.replay()
                else:
                    opt.step()
            torch.cuda.synchronize()
            runs.append([x.clone() for x in p] + [opt.norm.clone()])
        for a, b in zip(*runs):
            assert torch.equal(a, b)


def test_class_against_the_reference(moe):
    """AdamW: norm, clipping and step of a list, twice, against 64 bits; on
    another stream too."""
    gen = torch.Generator(device="cuda").manual_seed(5)
    p = [torch.randn(n, generator=gen, device="cuda").to(t) for n, t in ((5000, BF), (300, F32))]
    p[0] = p[0].view(50, 100)
    g = [torch.randn(x.shape, generator=gen, device="cuda").to(x.dtype) for x in p]
    opt = moe.AdamW(p, g, 1e-2, weight_decay=0.1, max_norm=2.0)
    side = torch.cuda.Stream()
    for t, stream in ((1, None), (2, side), (3, side.cuda_stream)):
        before = [copy(e) for e in opt.tensors]
        torch.cuda.synchronize()
        opt.step(stream)
        torch.cuda.synchronize()
        total = float(sum(x.double().square().sum() for x in g)) ** 0.5
        assert abs(float(opt.norm) - total) <= 40 * U * total
        h = dict(lr=1e-2, beta1=0.9, beta2=0.95, eps=1e-8, step=t)
        for b, a in zip(before, opt.tensors):
            flat = {k: v.reshape(-1) if isinstance(v, torch.Tensor) else v for k, v in a.items()}
            verify(b, flat, h, 2.0 / (float(opt.norm) + 1e-6))


def test_arrays_past_32_bit_offsets(moe):
    """More than 2^32 bytes of parameters and 2^31 elements: blocks at the
    start, around 2^31 and at the end."""
    n = (1 << 31) + 5000
    gen = torch.Generator(device="cuda").manual_seed(6)
    e = dict(param=torch.empty(n, dtype=BF, device="cuda").normal_(generator=gen),
             grad=torch.empty(n, dtype=F32, device="cuda").normal_(generator=gen), weight_decay=0.1,
             exp_avg=torch.zeros(n, dtype=torch.uint8, device="cuda").view(E4),
             exp_avg_sq=torch.zeros(n, dtype=torch.uint8, device="cuda").view(E4),
             exp_avg_scale=torch.zeros(-(-n // 256), device="cuda"),
             exp_avg_sq_scale=torch.zeros(-(-n // 256), device="cuda"))
    where = [slice(a, min(n, a + 2560)) for a in (0, (1 << 30), (1 << 31) - 1280, n - n % 256 - 2304)]

    def parts():
        out = []
        for s in where:
            b = slice(s.start // 256, -(-s.stop // 256))
            out.append({k: (v if not isinstance(v, torch.Tensor) else
                            v[b].clone() if k.endswith("scale") else
                            v.view(torch.uint8)[s].clone().view(E4) if v.dtype == E4 else v[s].clone())
                        for k, v in e.items()})
        return out
    before = parts()
    run(moe, [e], stochastic=True)
    for b, a in zip(before, parts()):
        verify(b, a, HYPER, stochastic=True)


def test_a_training_step(moe):
    """Forward, backward, AdamW with clipping and the balance bias in one go, as
    a training loop calls them, captured in a graph and eager: the same."""
    T, d, E, k, f = 300, 64, 16, 2, 64
    results = []
    for captured in (False, True):
        gen = torch.Generator(device="cuda").manual_seed(8)

        def rand(*shape, std=1.0, dt=BF):
            return (torch.randn(*shape, generator=gen, device="cuda") * std).to(dt)
        layer = moe.MoELayer(rand(E, d, std=d ** -0.5, dt=F32), rand(E, d, 2 * f, std=d ** -0.5),
                             rand(E, f, d, std=f ** -0.5), k, router=moe.router("sigmoid", 4, 2, "top2", 2.5),
                             balance_bias=torch.zeros(E, device="cuda"))
        params = [layer.Wr, layer.W_gate_up, layer.W_down]
        grads = {n: torch.empty_like(p) for n, p in zip(("Wr", "W_gate_up", "W_down"), params)}
        opt = moe.AdamW(params, list(grads.values()), 1e-3, weight_decay=0.1, bits=8, master=False,
                        max_norm=1.0, capturable=captured)
        x, dout = torch.empty(T, d, dtype=BF, device="cuda"), torch.empty(T, d, dtype=BF, device="cuda")
        grads["x"] = torch.empty_like(x)
        out, imb = torch.empty_like(x), torch.empty(1, device="cuda")

        def step():
            layer(x, out=out)
            layer.backward(x, dout, grads=grads)
            opt.step()
            layer.update_balance_bias(1e-3, imb)
        if captured:
            x.zero_(), dout.zero_()
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                step()
        for _ in range(4):
            x.copy_(rand(T, d))
            dout.copy_(rand(T, d, std=0.1))
            if captured:
                opt.advance()
                graph.replay()
            else:
                step()
        torch.cuda.synchronize()
        assert moe.moe_last_device_error() == moe.MOE_OK
        results.append([t.clone() for t in (*params, layer.balance_bias, out, imb, opt.norm)])
    for a, b in zip(*results):
        assert torch.equal(a, b) and torch.isfinite(a.float()).all()
    assert results[0][3].any()
