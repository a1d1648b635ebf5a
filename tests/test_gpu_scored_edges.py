"""Scored routing, its gradient, the balance bias and AdamW beside what they must not
touch, on several streams at once and in replayed graphs: results equal bit for bit
to those of a plain call."""
import pytest
import torch

from tests import scored_ref
from tests.gpu_util import load_moe
from tests.test_gpu_adamw import BF, E4, F32, HYPER, copy, entry, verify

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def moe():
    return load_moe()


def inside(x, margin=64):
    """x within a larger buffer, and that buffer's bytes on both sides."""
    raw = x.contiguous().view(torch.uint8).view(-1)
    buf = torch.full((raw.numel() + 2 * margin,), 0x5A, dtype=torch.uint8, device="cuda")
    mid = buf[margin:margin + raw.numel()]
    mid.copy_(raw)
    return mid.view(x.dtype).view(x.shape), (buf[:margin], buf[margin + raw.numel():])


def untouched(sides):
    return all(bool((s == 0x5A).all()) for pair in sides for s in pair)


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("p,master", [(F32, False), (BF, False), (BF, True)])
@pytest.mark.parametrize("n", [1, 7, 255, 256, 257, 2048, 16_385, 70_001])
def test_adamw_stays_inside_its_tensors(moe, n, p, master, bits):
    e, sides = entry(n, n, p=p, g=p, bits=bits, master=master), []
    for k, v in e.items():
        if isinstance(v, torch.Tensor):
            if v.dtype == E4:
                v, s = inside(v.view(torch.uint8))
                v = v.view(E4)
            else:
                v, s = inside(v)
            e[k] = v
            sides.append(s)
    before = copy(e)
    moe.moe_adamw_step(moe.adamw_list([e]), moe.adamw_hyper(**HYPER, stochastic=not master))
    torch.cuda.synchronize()
    assert untouched(sides)
    assert torch.equal(e["grad"], before["grad"])
    verify(before, e, HYPER, stochastic=not master and p == BF)


@pytest.mark.parametrize("T,E,k", [(1, 8, 8), (3, 37, 5), (33, 256, 8), (4099, 64, 8), (9, 1024, 32)])
@pytest.mark.parametrize("score,renorm", [("softmax", True), ("softmax", False), ("sigmoid", True),
                                          ("sigmoid", False)])
def test_routing_and_gradient_stay_inside_their_tensors(moe, T, E, k, score, renorm):
    g = torch.Generator(device="cuda").manual_seed(T + E)
    cfg, r = moe.config(T, 8, E, k, 8, renormalize=renorm), moe.router(score, weight_scale=2.5)
    L, s0 = inside(torch.randn(T, E, generator=g, device="cuda"))
    bias = torch.randn(E, generator=g, device="cuda") * 0.01
    idx, s1 = inside(torch.zeros(T, k, dtype=torch.int32, device="cuda"))
    w, s2 = inside(torch.zeros(T, k, device="cuda"))
    dl, s3 = inside(torch.zeros(T, E, device="cuda"))
    dw = torch.randn(T, k, generator=g, device="cuda")
    held = L.clone()
    moe.moe_route_scored_from_logits(cfg, r, L, bias, idx, w)
    moe.moe_route_scored_from_logits_backward(cfg, r, L, idx, w, dw, dl)
    torch.cuda.synchronize()
    assert moe.moe_last_device_error() == moe.MOE_OK
    assert untouched([s0, s1, s2, s3]) and torch.equal(L, held)
    want = scored_ref.select_many(L, bias, k, score == "sigmoid", 1, 1, False)
    assert torch.equal(idx.long(), want.long())


def test_balance_bias_stays_inside_its_tensors(moe):
    counts = torch.randint(0, 100, (5, 37), dtype=torch.int32, device="cuda")
    bias, s0 = inside(torch.zeros(5, 37, device="cuda"))
    imbalance, s1 = inside(torch.zeros(5, device="cuda"))
    moe.moe_update_balance_bias(counts, 0.5, bias, imbalance)
    torch.cuda.synchronize()
    n = counts.long()
    assert untouched([s0, s1])
    assert torch.equal(bias, 0.5 * (n.sum(-1, keepdim=True) - 37 * n).sign().float())


def test_calls_on_four_streams_at_once(moe):
    """Nothing is shared between calls: each stream's results are those of a call alone."""
    r = moe.router("sigmoid", 8, 4, "top2")
    sets = []
    for i, T in enumerate((5000, 40_000, 300, 8192)):
        g = torch.Generator(device="cuda").manual_seed(i)
        L = torch.randn(T, 256, generator=g, device="cuda")
        L[: T // 3] = 0.0  # ties too
        bias = torch.randint(-9, 9, (256,), generator=g, device="cuda").float() * 2.0 ** -7
        e = entry(100_000 + i, i, bits=8)
        new = lambda: (torch.zeros(T, 8, dtype=torch.int32, device="cuda"), torch.zeros(T, 8, device="cuda"),
                       torch.zeros(T, 256, device="cuda"))
        sets.append((moe.config(T, 8, 256, 8, 8), L, bias, torch.randn(T, 8, generator=g, device="cuda"),
                     e, copy(e), new(), new()))
    hyper = moe.adamw_hyper(**HYPER, seed=5)

    def go(s, which, stream=None):
        cfg, L, bias, dw, e0, e1, out0, out1 = s
        idx, w, dl = (out0, out1)[which]
        moe.moe_route_scored_from_logits(cfg, r, L, bias, idx, w, stream=stream)
        moe.moe_route_scored_from_logits_backward(cfg, r, L, idx, w, dw, dl, stream=stream)
        moe.moe_adamw_step(moe.adamw_list([(e0, e1)[which]]), hyper, stream=stream)
    for s in sets:
        go(s, 0)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sets]
    for _ in range(2):  # (the second: the routing again, over its own outputs)
        for s, st in zip(sets, streams):
            go(s, 1, st)
    torch.cuda.synchronize()
    for s in sets:
        for a, b in zip(s[6], s[7]):
            assert torch.equal(a, b)
        moe.moe_adamw_step(moe.adamw_list([s[4]]), hyper)  # the second step
        torch.cuda.synchronize()
        assert all(torch.equal(s[4][n].view(torch.uint8), s[5][n].view(torch.uint8))
                   for n in ("param", "exp_avg", "exp_avg_sq", "exp_avg_scale", "exp_avg_sq_scale"))


def test_a_captured_training_step(moe):
    """Routing, its gradient, the bias's update and AdamW in one graph, replayed on
    new logits: as the same calls made one by one."""
    T, E, k = 6000, 64, 4
    cfg, r = moe.config(T, 8, E, k, 8), moe.router("softmax")
    make = lambda seed: torch.randn(T, E, generator=torch.Generator(device="cuda").manual_seed(seed),
                                    device="cuda")
    dw = torch.ones(T, k, device="cuda")

    def state():
        return dict(L=make(0), bias=torch.zeros(E, device="cuda"),
                    idx=torch.zeros(T, k, dtype=torch.int32, device="cuda"), w=torch.zeros(T, k, device="cuda"),
                    dl=torch.zeros(T, E, device="cuda"), counts=torch.zeros(E, dtype=torch.int32, device="cuda"),
                    p=torch.zeros(T, E, device="cuda"))
    a, b = state(), state()
    opts = [moe.AdamW([s["p"]], [s["dl"]], lr=1e-2, bits=8, max_norm=1.0, seed=3, capturable=c)
            for s, c in ((a, False), (b, True))]

    def step(s, opt):
        moe.moe_route_scored_from_logits(cfg, r, s["L"], s["bias"], s["idx"], s["w"])
        moe.moe_route_scored_from_logits_backward(cfg, r, s["L"], s["idx"], s["w"], dw * s["w"], s["dl"])
        s["counts"].zero_().index_add_(0, s["idx"].view(-1), torch.ones(T * k, dtype=torch.int32, device="cuda"))
        moe.moe_update_balance_bias(s["counts"], 2.0 ** -8, s["bias"])
        opt.step()
    graph = torch.cuda.CUDAGraph()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        torch.ones(1, device="cuda").add_(1)
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        step(b, opts[1])
    for seed in range(1, 5):
        a["L"].copy_(make(seed))
        step(a, opts[0])
        b["L"].copy_(make(seed))
        opts[1].advance()
        graph.replay()
        torch.cuda.synchronize()
        for n in a:
            assert torch.equal(a[n], b[n]), (seed, n)
        assert torch.equal(opts[0].norm, opts[1].norm)


@pytest.mark.parametrize("E,G,Gk,score", [(256, 1, 1, "sigmoid"), (256, 8, 4, "sigmoid"), (260, 1, 1, "softmax")])
def test_logits_past_32_bit_offsets(moe, E, G, Gk, score):
    """More than 2^31 logits: the last tokens as in a batch of their own, and their
    gradient."""
    T, k, tail = (1 << 31) // E + 4099, 8, 9000
    g = torch.Generator(device="cuda").manual_seed(E)
    L = torch.zeros(T, E, device="cuda")
    for at in range(0, T, 1 << 21):
        L[at:at + (1 << 21)].normal_(generator=g)
    bias = torch.randn(E, generator=g, device="cuda") * 0.01
    r = moe.router(score, G, Gk, "top2")
    idx, w = torch.zeros(T, k, dtype=torch.int32, device="cuda"), torch.zeros(T, k, device="cuda")
    moe.moe_route_scored_from_logits(moe.config(T, 8, E, k, 8, renormalize=False), r, L, bias, idx, w)
    torch.cuda.synchronize()
    last = L[T - tail:].clone()
    want = scored_ref.select_many(last, bias, k, score == "sigmoid", G, Gk, True)
    assert torch.equal(idx[T - tail:].long(), want.long())
    dw = torch.zeros(T, k, device="cuda")
    dw[T - tail:] = 1.0
    dl = torch.ones(T, E, device="cuda")
    moe.moe_route_scored_from_logits_backward(moe.config(T, 8, E, k, 8, renormalize=False), r, L, idx, w, dw, dl)
    alone = torch.zeros(tail, E, device="cuda")
    moe.moe_route_scored_from_logits_backward(
        moe.config(tail, 8, E, k, 8, renormalize=False), r, last, idx[T - tail:].clone(), w[T - tail:].clone(),
        dw[T - tail:].clone(), alone)
    torch.cuda.synchronize()
    assert moe.moe_last_device_error() == moe.MOE_OK
    assert torch.equal(dl[T - tail:], alone) and not dl[:T - tail].any()
