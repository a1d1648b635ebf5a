"""Scored routing and the optimizer step, as cases that can be timed and checked.

Four operators, in the notation of include/moe.h (T tokens, E experts, k
experts per token, G groups of E/G consecutive experts):

``route``    selection and weights from given logits: softmax or sigmoid
             scores, a balance bias on the choice, groups, renormalised and
             scaled weights
``grad``     the gradient of those weights with respect to the logits
``balance``  the balance bias moved against the experts' loads, layer by layer
``adamw``    one AdamW step over many tensors, states in 32 bits or in 8

``run`` computes an operator's plain form (elementary torch operations) or,
with ``own`` set, calls the framework.  Sizes are those of the workloads in
token_dispatch_grouped_fp32_gb300/synth.py, or generic.
"""
import math
import random

import torch

own = False

BF16, F32 = "bf16", "f32"
BLOCK = 256  # elements under one scale of an 8-bit state


# ------------------------------- the cases ---------------------------------
def listed():
    return [
        # one training batch of the DeepSeek-shaped layer: the best four of eight groups
        dict(name="route_groups_8192", op="route", T=8192, E=256, k=8, score="sigmoid", bias=True,
             G=8, Gk=4, top2=True, renorm=True, scale=2.5),
        # the same router while decoding: latency
        dict(name="route_groups_64", op="route", T=64, E=256, k=8, score="sigmoid", bias=True,
             G=8, Gk=4, top2=True, renorm=True, scale=2.5),
        # softmax scores, groups by their best expert, weights kept: groups that split a warp unevenly
        dict(name="route_softmax_groups_odd", op="route", T=3001, E=160, k=6, score="softmax",
             bias=False, G=8, Gk=3, top2=False, renorm=False, scale=16.0),
        # a long packed batch over the Qwen3 shape's experts, no groups
        dict(name="route_long_131072", op="route", T=131072, E=128, k=8, score="sigmoid", bias=True,
             G=1, Gk=1, top2=False, renorm=True, scale=1.0),
        # the DeepSeek-shaped batch backward: gradient on the chosen logits only
        dict(name="grad_sigmoid_8192", op="grad", T=8192, E=256, k=8, score="sigmoid", renorm=True,
             scale=2.5),
        # the long batch backward, softmax weights kept: every logit has a gradient
        dict(name="grad_softmax_131072", op="grad", T=131072, E=128, k=8, score="softmax",
             renorm=False, scale=1.0),
        # one layer's bias after a step: latency
        dict(name="balance_one_layer", op="balance", layers=1, E=256, rate=1e-3),
        # all layers of a model at once
        dict(name="balance_64_layers", op="balance", layers=64, E=256, rate=1e-3),
        # the Mixtral-shaped layer's parameters with fp32 masters: bytes
        dict(name="adamw_mixtral_layer", op="adamw", layer="mixtral", dtype="mixed", bits=32,
             master=True),
        # the same parameters in their smallest form: 8-bit states, no masters
        dict(name="adamw_mixtral_layer_8bit", op="adamw", layer="mixtral", dtype="mixed", bits=8,
             master=False),
        # hundreds of small tensors of odd sizes: few bytes, many pointers
        dict(name="adamw_many_small", op="adamw", layer="", n=300, small=1, large=20000,
             dtype="mixed", bits=32, master=True),
        # ragged 8-bit blocks, bf16 parameters
        dict(name="adamw_ragged_8bit", op="adamw", layer="", n=40, small=100, large=1_000_000,
             dtype=BF16, bits=8, master=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["route", "route", "grad", "balance", "adamw", "adamw"])
    if op == "balance":
        return dict(op=op, layers=_log(rng, 1, 128), E=_log(rng, 2, 1024), rate=rng.choice([1e-3, 1e-2]))
    if op == "adamw":
        bits = rng.choice([8, 32])
        return dict(op=op, layer="", n=_log(rng, 1, 400), small=1, large=_log(rng, 10, 2_000_000),
                    dtype=rng.choice([BF16, F32, "mixed"]), bits=bits, master=rng.random() < 0.4)
    c = dict(op=op, T=_log(rng, 1, 131072), score=rng.choice(["sigmoid", "softmax"]),
             renorm=rng.random() < 0.6, scale=rng.choice([1.0, 2.5, 16.0]))
    if op == "grad":
        c["E"] = _log(rng, 2, 1024)
        c["k"] = min(c["E"], rng.randint(1, 16))
    else:
        c["bias"] = rng.random() < 0.6
        c["G"] = rng.choice([1, 1, 2, 4, 8, 16, 5])
        per = _log(rng, 2, 1024 // c["G"])
        c["E"] = c["G"] * per
        c["Gk"] = rng.randint(1, c["G"])
        c["k"] = min(c["Gk"] * per, rng.randint(1, 16))
        c["top2"] = rng.random() < 0.5
    # (one expert with a renormalised weight has no gradient at all)
    if op == "grad" and c["k"] == 1:
        c["renorm"] = False
    while c["T"] * c["E"] > 131072 * 128:
        c["T"] //= 2
    return c


# ------------------------------- the inputs --------------------------------
def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _randn(g, *shape, std=1.0, dtype=torch.float32):
    return torch.randn(*shape, generator=g, device="cuda", dtype=dtype).mul_(std)


def _tensors(case):
    """(elements, type, weight decay) of every parameter tensor of a case."""
    if case["layer"]:  # gate/up, down, router weight, router bias of the Mixtral-shaped layer
        return [(8 * 4096 * 28672, BF16, 0.1), (8 * 14336 * 4096, BF16, 0.1),
                (8 * 4096, F32, 0.1), (8, F32, 0.0)]
    r = random.Random(case["n"] * 1000003 + case["large"])
    sizes = [_log(r, case["small"], case["large"]) for _ in range(case["n"])]
    return [(n, F32 if case["dtype"] == F32 or (case["dtype"] == "mixed" and i % 3 == 2) else BF16,
             0.1 if i % 2 == 0 else 0.0) for i, n in enumerate(sizes)]


def _blocks(n):
    return (n + BLOCK - 1) // BLOCK


def _prepare_adamw(case, g, s):
    """Parameters, gradients and states of one type as views of flat buffers, each
    tensor from a multiple of BLOCK elements (as an allocator places them); the
    filling between them is zero and stays so."""
    tensors = _tensors(case)
    s["norm"] = torch.full((), 2.0, device="cuda")
    s["max_norm"], s["seed"] = 1.0, 0x9ABCDEF0 + 7919 * (int(case.get("n", 0)) + 1)
    s["hyper"] = dict(lr=3e-4, beta1=0.9, beta2=0.95, eps=1e-8, step=1000)
    s["groups"], first = [], []
    total = 0
    for n, _, _ in tensors:  # the number of a tensor's first block, counted over the list
        first.append(total)
        total += _blocks(n)
    for name, dtype in ((BF16, torch.bfloat16), (F32, torch.float32)):
        of = [i for i, t in enumerate(tensors) if t[1] == name]
        if not of:
            continue
        nb, start, size = [_blocks(tensors[i][0]) for i in of], [], 0
        for b in nb:
            start.append(size)
            size += BLOCK * b
        fill = torch.zeros(size, dtype=torch.bool, device="cuda")
        for j, i in enumerate(of):
            fill[start[j] + tensors[i][0]:start[j] + BLOCK * nb[j]] = True
        rep = torch.tensor(nb, device="cuda")
        f = dict(of=of, start=start, n=[tensors[i][0] for i in of], size=size, dtype=dtype,
                 wd_of=[tensors[i][2] for i in of],
                 wd=torch.tensor([tensors[i][2] for i in of], device="cuda").repeat_interleave(rep),
                 block=torch.cat([torch.arange(first[i], first[i] + b, device="cuda")
                                  for i, b in zip(of, nb)]))
        f["g"] = _randn(g, size, std=2e-3, dtype=dtype).masked_fill_(fill, 0)
        p = _randn(g, size, std=0.02).masked_fill_(fill, 0)
        f["p"] = p.to(dtype)
        f["master"] = p if case["master"] and name == BF16 else None
        del p
        m = f["g"].float() * 0.3
        r = (f["g"].float().abs() * 0.7).add_(1e-3).masked_fill_(fill, 0)
        if case["bits"] == 32:
            f["m"], f["v"] = m, r.square_()
        else:
            for key, x in (("m", m), ("r", r)):
                x = x.view(-1, BLOCK)
                scale = _scale_of(x)
                f[key] = (x / scale[:, None]).to(torch.float8_e4m3fn).view(-1)
                f[key + "s"] = scale
        del m, r, fill
        s["groups"].append(f)


def prepare(case, seed):
    g = _gen(seed)
    s = dict(case=dict(case), kept={})
    op = case["op"]
    if op == "adamw":
        _prepare_adamw(case, g, s)
        return s
    E = case["E"]
    if op == "balance":
        load = torch.rand(case["layers"], E, generator=g, device="cuda")
        s["counts"] = (load.square() * 2000).to(torch.int32)
        s["bias"] = _randn(g, case["layers"], E, std=0.01)
        return s
    T, k = case["T"], case["k"]
    s["logits"] = _randn(g, T, E)
    if op == "route":
        # a bias as training leaves it: some hundred steps of the update either way
        s["bias"] = (torch.randint(-100, 101, (E,), generator=g, device="cuda").float() * 1e-3
                     if case["bias"] else None)
        return s
    sc = _score(case, s["logits"].double())
    s["idx"] = torch.topk(sc, k, dim=-1).indices.to(torch.int32).contiguous()
    w = sc.gather(1, s["idx"].long())
    w = w / w.sum(-1, keepdim=True) if case["renorm"] else w
    s["w"] = (w * case["scale"]).float().contiguous()
    s["dw"] = _randn(g, T, k, std=0.1)
    return s


# ------------------------------- the passes --------------------------------
def run(s):
    op = s["case"]["op"]
    return globals()[("_own_" if own else "_plain_") + op](s)


def _score(c, L):
    if c["score"] == "sigmoid":
        return 1.0 / (1.0 + torch.exp(-L))
    e = torch.exp(L - L.max(-1, keepdim=True).values)
    return e / e.sum(-1, keepdim=True)


def _plain_route(s):
    # 64 bits: a choice is made by the order of the values, whatever lies between them
    c = s["case"]
    T, E, k, G = c["T"], c["E"], c["k"], c["G"]
    sc = _score(c, s["logits"].double())
    q = sc if s["bias"] is None else sc + s["bias"].double()
    if c["Gk"] < G:
        best = torch.sort(q.view(T, G, E // G), dim=-1, descending=True).values
        u = best[..., :2].sum(-1) if c["top2"] else best[..., 0]
        kept = torch.sort(u, dim=-1, descending=True, stable=True).indices[:, :c["Gk"]]
        there = torch.zeros(T, G, dtype=torch.bool, device="cuda").scatter_(1, kept, True)
        q = q.masked_fill(~there.repeat_interleave(E // G, 1), -math.inf)
    idx = torch.sort(q, dim=-1, descending=True, stable=True).indices[:, :k]
    w = sc.gather(1, idx)
    if c["renorm"]:
        w = w / w.sum(-1, keepdim=True)
    return dict(idx=idx.to(torch.int32), w=(w * c["scale"]).float())


def _plain_grad(s):
    c = s["case"]
    L, idx, w, dw = s["logits"], s["idx"].long(), s["w"], s["dw"]
    a = (w * dw).sum(-1, keepdim=True)
    dl = torch.zeros_like(L)
    if c["score"] == "softmax" and not c["renorm"]:
        return dict(dlogits=_score(c, L) * (dl.scatter_(1, idx, dw * c["scale"]) - a))
    t = w * (dw - a / c["scale"]) if c["renorm"] else w * dw
    if c["score"] == "sigmoid":
        t = t / (1.0 + torch.exp(L.gather(1, idx)))
    return dict(dlogits=dl.scatter_(1, idx, t))


def _plain_balance(s):
    n = s["counts"].long()
    total, E = n.sum(-1, keepdim=True), n.shape[-1]
    s["bias"] += s["case"]["rate"] * torch.sign(total - E * n)
    return dict(bias=s["bias"],
                imbalance=(n.max(-1).values * E).float() / total[:, 0].clamp(min=1).float())


_M = 0xFFFFFFFF
_K = (0x9E3779B1, 0xD6E8FEB9, 0xA24BAED5, 0xCA5A8263)


def _fold(a, K):
    """High and low words of a 32-bit product, xor'ed (a: 32-bit values held in int64)."""
    p = (a & _M) * (K - (1 << 32) if K >= 1 << 31 else K) + ((a & _M) << 32 if K >= 1 << 31 else 0)
    return ((p >> 32) ^ p) & _M


def _random_bits(block, seed):
    """32 random bits of every element of the blocks numbered `block`."""
    x = _fold(block + _K[0], _K[1])
    x = _fold(x ^ (seed & _M), _K[2])
    x = _fold(x + (seed >> 32) + (block >> 32), _K[3])
    y = _fold(x ^ _K[0], _K[3])
    j = torch.arange(BLOCK, device=block.device) * _K[0]
    return _fold(_fold(x[:, None] + j[None, :], _K[2]) ^ y[:, None], _K[1])


def _scale_of(x):
    """2^(e - 7) where 2^e <= the largest magnitude of a block < 2^(e + 1)."""
    e = torch.frexp(x.abs().amax(-1)).exponent - 8
    return torch.ldexp(torch.ones_like(x[:, 0]), e.clamp(min=-126))


def _to_e4m3(y, u16):
    """Stochastic rounding of y (|y| < 256) to e4m3: y's neighbours below and above
    by the 16 random bits; below 2^-6, where the steps are 2^-9, with 2^-6 added."""
    a = y.abs()
    low = a < 2.0 ** -6
    z = torch.where(low, a + 2.0 ** -6, a)
    z = ((z.view(torch.int32) + (u16 * 16 + 8).to(torch.int32)) & ~0xFFFFF).view(torch.float32)
    return torch.copysign(torch.where(low, z - 2.0 ** -6, z), y)


def _plain_adamw(s):
    h, out = s["hyper"], []
    coef = torch.clamp(s["max_norm"] / (s["norm"] + 1e-6), max=1.0)
    c1, c2 = 1.0 - h["beta1"] ** h["step"], 1.0 - h["beta2"] ** h["step"]
    for f in s["groups"]:
        small = s["case"]["bits"] == 8
        g = (f["g"].float() * coef).view(-1, BLOCK)
        if small:
            m = f["m"].float().view(-1, BLOCK).mul_(f["ms"][:, None])
            v = f["r"].float().view(-1, BLOCK).mul_(f["rs"][:, None]).square_()
        else:
            m, v = f["m"].view(-1, BLOCK), f["v"].view(-1, BLOCK)
        m = m.mul_(h["beta1"]).add_(g * (1.0 - h["beta1"]))
        v = v.mul_(h["beta2"]).add_(g.square_().mul_(1.0 - h["beta2"]))
        del g
        r = torch.sqrt(v)
        p = (f["p"].float() if f["master"] is None else f["master"]).view(-1, BLOCK)
        p = p.mul_((1.0 - h["lr"] * f["wd"])[:, None])
        p.sub_((m / (r / math.sqrt(c2) + h["eps"])).mul_(h["lr"] / c1))
        whole = f["dtype"] == torch.float32 or f["master"] is not None
        if small or not whole:
            u = _random_bits(f["block"], s["seed"])
        if not whole:  # stochastic rounding to bf16 by the low 16 bits
            p = (p.view(torch.int32) + (u & 0xFFFF).to(torch.int32)) & ~0xFFFF
            p = p.view(torch.float32)
        f["p"].copy_(p.view(-1))
        if small:
            for key, x, bits in (("m", m, (u >> 8) & 0xFFFF), ("r", r, u >> 16)):
                scale = _scale_of(x)
                y = _to_e4m3(x / scale[:, None], bits)
                if key == "r":  # no root of a sum of squares becomes zero
                    y = torch.where(x > 0, y.clamp(min=2.0 ** -9), y)
                f[key].copy_(y.view(-1))
                f[key + "s"].copy_(scale)
        out.append(_updated(f))
    return out


def _updated(f):
    return {key: f[key] for key in ("p", "master", "m", "v", "r", "ms", "rs") if f.get(key) is not None}


def _own_route(s):
    from token_dispatch_grouped_fp32_gb300 import moe
    c, k = s["case"], s["kept"]
    if not k:  # what a program sets up once
        k["cfg"] = moe.config(c["T"], 8, c["E"], c["k"], 8, renormalize=c["renorm"])
        k["router"] = moe.router(c["score"], groups=c["G"], topk_groups=c["Gk"],
                                 group_score="top2" if c["top2"] else "max", weight_scale=c["scale"])
        k["idx"] = torch.empty(c["T"], c["k"], dtype=torch.int32, device="cuda")
        k["w"] = torch.empty(c["T"], c["k"], device="cuda")
    moe.moe_route_scored_from_logits(k["cfg"], k["router"], s["logits"], s["bias"], k["idx"], k["w"])
    return dict(idx=k["idx"], w=k["w"])


def _own_grad(s):
    from token_dispatch_grouped_fp32_gb300 import moe
    c, k = s["case"], s["kept"]
    if not k:
        k["cfg"] = moe.config(c["T"], 8, c["E"], c["k"], 8, renormalize=c["renorm"])
        k["router"] = moe.router(c["score"], weight_scale=c["scale"])
        k["dl"] = torch.empty_like(s["logits"])
    moe.moe_route_scored_from_logits_backward(k["cfg"], k["router"], s["logits"], s["idx"], s["w"],
                                              s["dw"], k["dl"])
    return dict(dlogits=k["dl"])


def _own_balance(s):
    from token_dispatch_grouped_fp32_gb300 import moe
    k = s["kept"]
    if not k:
        k["imbalance"] = torch.empty(s["counts"].shape[0], device="cuda")
    moe.moe_update_balance_bias(s["counts"], s["case"]["rate"], s["bias"], k["imbalance"])
    return dict(bias=s["bias"], imbalance=k["imbalance"])


def _own_adamw(s):
    from token_dispatch_grouped_fp32_gb300 import moe
    k = s["kept"]
    if not k:
        rows = {}
        small = s["case"]["bits"] == 8
        for f in s["groups"]:
            b0 = [x // BLOCK for x in f["start"]]
            for j, i in enumerate(f["of"]):
                at = slice(f["start"][j], f["start"][j] + f["n"][j])
                bl = slice(b0[j], b0[j] + _blocks(f["n"][j]))
                rows[i] = dict(param=f["p"][at], grad=f["g"][at], exp_avg=f["m"][at],
                               exp_avg_sq=f["r" if small else "v"][at],
                               exp_avg_scale=f["ms"][bl] if small else None,
                               exp_avg_sq_scale=f["rs"][bl] if small else None,
                               master=None if f["master"] is None else f["master"][at],
                               weight_decay=f["wd_of"][j])
        k["list"] = moe.adamw_list([rows[i] for i in sorted(rows)])
        k["hyper"] = moe.adamw_hyper(**s["hyper"], max_norm=s["max_norm"], seed=s["seed"],
                                     stochastic=True)
    moe.moe_adamw_step(k["list"], k["hyper"], s["norm"])
    return [_updated(f) for f in s["groups"]]


# --------------------------------- the work --------------------------------
def work(case):
    op = case["op"]
    if op == "balance":
        n = case["layers"] * case["E"]
        return dict(bytes=12 * n + 4 * case["layers"], flops=4 * n)
    if op == "adamw":
        total = flops = 0
        for n, t, _ in _tensors(case):
            es = 2 if t == BF16 else 4
            master = case["master"] and t == BF16
            total += n * (es + (8 + es if master else 2 * es))  # gradient, parameter
            total += 16 * n if case["bits"] == 32 else 4 * n + 16 * _blocks(n)
            flops += 14 * n
        return dict(bytes=total, flops=flops)
    T, E, k = case["T"], case["E"], case["k"]
    if op == "route":
        return dict(bytes=4 * T * E + 8 * T * k + (4 * E if case["bias"] else 0), flops=4 * T * E)
    read = 12 * T * k
    if case["score"] == "softmax" and not case["renorm"]:
        read += 4 * T * E
    elif case["score"] == "sigmoid":
        read += 4 * T * k
    return dict(bytes=read + 4 * T * E, flops=4 * T * k)


# ------------------------------ in 64 bits ---------------------------------
def exact(case, seed):
    s = prepare(case, seed)
    return globals()["_exact_" + case["op"]](case, s)


def _exact_route(c, s):
    T, E = c["T"], c["E"]
    L = s["logits"].double()
    sc = torch.sigmoid(L) if c["score"] == "sigmoid" else torch.softmax(L, -1)
    left = sc.clone() if s["bias"] is None else sc + s["bias"].double()[None, :]
    n = torch.arange(T, device="cuda")
    if c["Gk"] < c["G"]:
        u = left.view(T, c["G"], -1).clone()
        first = u.amax(-1)
        if c["top2"] and u.shape[-1] > 1:
            u.scatter_(-1, u.argmax(-1, keepdim=True), -math.inf)
            first = first + u.amax(-1)
        place = (first[:, None, :] > first[:, :, None]).sum(-1)  # groups before each
        left = left.view(T, c["G"], -1).masked_fill((place >= c["Gk"])[..., None], -math.inf).view(T, E)
    idx = torch.empty(T, c["k"], dtype=torch.int32, device="cuda")
    w = torch.empty(T, c["k"], dtype=torch.float64, device="cuda")
    for j in range(c["k"]):
        e = left.argmax(-1)
        idx[:, j], w[:, j] = e, sc[n, e]
        left[n, e] = -math.inf
    if c["renorm"]:
        w = torch.exp(torch.log(w) - torch.logsumexp(torch.log(w), -1, keepdim=True))
    return dict(idx=idx, w=w * c["scale"])


def _exact_grad(c, s):
    # the Jacobian of the weights, written out: dw_i/ds_j, then ds_j/dL_e
    idx, d, S = s["idx"].long(), s["dw"].double(), c["scale"]
    L = s["logits"].double()
    sc = torch.sigmoid(L) if c["score"] == "sigmoid" else torch.softmax(L, -1)
    chosen = sc.gather(1, idx)
    if c["renorm"]:
        # the weights as given (rounded to fp32) stand for the scores' shares
        share = s["w"].double() / S
        total = chosen.sum(-1, keepdim=True)
        ds = S * (d - torch.einsum("tj,tj->t", share, d)[:, None]) / total
    else:
        ds = S * d
    dl = torch.zeros_like(L)
    if c["score"] == "sigmoid":
        dl.scatter_(1, idx, ds * chosen * torch.sigmoid(-L.gather(1, idx)))
        return dict(dlogits=dl)
    dl.scatter_(1, idx, ds)
    return dict(dlogits=sc * (dl - torch.einsum("te,te->t", sc, dl)[:, None]))


def _exact_balance(c, s):
    n = s["counts"].double()
    mean = n.mean(-1, keepdim=True)
    bias = s["bias"].double()
    bias = torch.where(n < mean, bias + c["rate"], torch.where(n > mean, bias - c["rate"], bias))
    return dict(bias=bias, imbalance=n.amax(-1) / mean[:, 0].clamp(min=1e-300))


def _exact_adamw(c, s):
    h, out = s["hyper"], []
    coef = min(1.0, s["max_norm"] / (s["norm"].item() + 1e-6))
    b1, b2 = h["beta1"], h["beta2"]
    for f in s["groups"]:
        small = c["bits"] == 8
        o = dict(p=[], master=[], m=[], v=[])
        for a in range(0, f["size"], 1 << 26):
            b = min(f["size"], a + (1 << 26))
            blocks = slice(a // BLOCK, b // BLOCK)

            def wide(per_block):
                return per_block[blocks].double().repeat_interleave(BLOCK)

            g = f["g"][a:b].double() * coef
            if small:
                m = f["m"][a:b].double() * wide(f["ms"])
                v = (f["r"][a:b].double() * wide(f["rs"])) ** 2
            else:
                m, v = f["m"][a:b].double(), f["v"][a:b].double()
            m = b1 * m + (1 - b1) * g
            v = b2 * v + (1 - b2) * g * g
            p = (f["p"] if f["master"] is None else f["master"])[a:b].double()
            mh, vh = m / (1 - b1 ** h["step"]), v / (1 - b2 ** h["step"])
            p = p - h["lr"] * wide(f["wd"]) * p - h["lr"] * mh / (vh.sqrt() + h["eps"])
            o["p"].append(p)
            if not small:
                o["m"].append(m)
                o["v"].append(v)
        p = torch.cat(o["p"]) if len(o["p"]) > 1 else o["p"][0]
        # a rounded state stands for a random one of its neighbours: no value of its own
        out.append(dict(p=p, master=p if f["master"] is not None else None,
                        m=torch.cat(o["m"]) if o["m"] else None,
                        v=torch.cat(o["v"]) if o["v"] else None, r=None, ms=None, rs=None))
    return out
