"""The MoE layer's training operators, as cases that can be timed and checked.

Five operators, in the notation of include/moe.h (T tokens, d hidden size, E
experts, k experts per token, f expert width, P = T*k routed pairs):

``combine``   gradient of the weighted combine: from the output's gradient to
              the expert rows' and the routing weights' gradients
``dispatch``  gradient of the token dispatch: the rows' gradients summed back
              into token order (weighted, with the weights' gradients, where
              the routing weights act on the expert inputs)
``experts``   gradient of the grouped SwiGLU experts: rows and both weights
``route``     gradient of the router: logits, router weight, bias, tokens
``clip``      global norm of many gradient tensors and their clipped copies

``run`` computes an operator's plain form (elementary torch operations in 32
bits) or, with ``own`` set, calls the framework.  Sizes are those of the
workloads in token_dispatch_grouped_fp32_gb300/synth.py, or generic.
"""
import math
import random

import torch

own = False

BF16, F32 = "bf16", "f32"


# ------------------------------- the cases ---------------------------------
def listed():
    return [
        # one training step's output gradient through the Mixtral-shaped layer
        dict(name="combine_mixtral_4096", op="combine", T=4096, d=4096, E=8, k=2, dtype=BF16),
        # a single token (online updates, the tail of a packed batch): latency
        dict(name="combine_one_token", op="combine", T=1, d=2880, E=128, k=4, dtype=BF16),
        # the Qwen3-30B-A3B shape's batch, eight rows summed into each token
        dict(name="dispatch_qwen3_16384", op="dispatch", T=16384, d=2048, E=128, k=8, dtype=BF16,
             scale=False, zipf=True),
        # weights on the expert inputs, fp32, sizes off every tile
        dict(name="dispatch_scaled_odd_f32", op="dispatch", T=777, d=1000, E=16, k=4, dtype=F32,
             scale=True, zipf=False),
        # all expert gradients of the Mixtral-shaped layer: long reductions
        dict(name="experts_mixtral_4096", op="experts", T=4096, d=4096, E=8, k=2, f=14336,
             dtype=BF16, zipf=False),
        # many experts with about 256 rows each: weight gradients bound by their writes
        dict(name="experts_gptoss_8192", op="experts", T=8192, d=2880, E=128, k=4, f=2880,
             dtype=BF16, zipf=False),
        # a short batch routed unevenly: experts from no rows to thousands
        dict(name="experts_qwen3_zipf_2048", op="experts", T=2048, d=2048, E=128, k=8, f=768,
             dtype=BF16, zipf=True),
        # the tiny fp32 layer: fp32 throughout, latency
        dict(name="experts_tiny_f32", op="experts", T=64, d=128, E=8, k=2, f=256, dtype=F32,
             zipf=False),
        # the Qwen3 router: gradient on the chosen logits only
        dict(name="route_qwen3_16384", op="route", T=16384, d=2048, E=128, k=8, dtype=BF16,
             renorm=True, zipf=True),
        # softmax weights kept unnormalised: every logit has a gradient
        dict(name="route_mixtral_norenorm", op="route", T=4096, d=4096, E=8, k=2, dtype=BF16,
             renorm=False, zipf=False),
        # the Mixtral-shaped layer's gradients, far larger than any cache
        dict(name="clip_mixtral_layer", op="clip", layer="mixtral", dtype="mixed"),
        # hundreds of small tensors of odd sizes back to back: few bytes, many pointers
        dict(name="clip_many_small", op="clip", layer="", n=300, small=1, large=20000,
             dtype="mixed"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _width(rng, lo, hi):
    """A hidden size: one of the workloads', or an odd multiple of 8."""
    if rng.random() < 0.4:
        return rng.choice([w for w in (128, 256, 768, 2048, 2880, 4096, 7168) if lo <= w <= hi])
    return 8 * (2 * (_log(rng, lo, hi) // 16) + 1)


def draw(rng):
    op = rng.choice(["combine", "dispatch", "experts", "route", "clip"])
    if op == "clip":
        return dict(op="clip", layer="", n=_log(rng, 1, 400), small=1,
                    large=_log(rng, 10, 2_000_000), dtype=rng.choice([BF16, F32, "mixed"]))
    c = dict(op=op, T=_log(rng, 1, 16384), dtype=rng.choice([BF16, BF16, F32]))
    if op == "experts":
        c["E"] = _log(rng, 1, 128)
        c["k"] = min(c["E"], rng.randint(1, 8))
        top = 4096 if c["dtype"] == BF16 else 512  # fp32 experts: small layers
        c["d"], c["f"] = _width(rng, 64, top), _width(rng, 64, top)
        c["zipf"] = rng.random() < 0.3
        if c["dtype"] == F32:
            c["T"] = min(c["T"], 1024)
        # within the largest listed case's work and memory
        while (c["T"] > 1 and (16 * c["T"] * c["k"] * c["d"] * c["f"] > 3e12
                               or c["E"] * c["T"] * (c["d"] + 3 * c["f"]) > 3e9
                               or (c["zipf"] and 8 * c["E"] * c["T"] * c["d"] * c["f"] > 5e12))):
            c["T"] = max(1, c["T"] // 2)
        return c
    if op == "route":
        c["E"] = _log(rng, 2, 256)
        c["k"] = min(c["E"], rng.randint(1, 8))
        c["d"] = _width(rng, 64, 7168)
        # (one chosen expert with a normalised weight has no gradient at all)
        c["renorm"] = c["k"] > 1 and rng.random() < 0.6
        c["zipf"] = rng.random() < 0.3
        return c
    c["E"] = _log(rng, 1, 256)
    c["k"] = min(c["E"], rng.randint(1, 8))
    c["d"] = _width(rng, 8, 7168) if c["T"] * c["k"] > 64 else _width(rng, 64, 7168)
    if op == "dispatch":
        c["scale"] = rng.random() < 0.5
        c["zipf"] = rng.random() < 0.3
    return c


def _torch_dtype(case):
    return torch.bfloat16 if case["dtype"] == BF16 else torch.float32


# ------------------------------- the inputs --------------------------------
def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _randn(g, *shape, std=1.0, dtype=torch.float32):
    return torch.randn(*shape, generator=g, device="cuda", dtype=dtype).mul_(std)


def _logits(case, g):
    """Router logits as a layer meets them; with zipf, skewed by a per-expert offset."""
    L = _randn(g, case["T"], case["E"])
    if case.get("zipf"):
        perm = torch.randperm(case["E"], generator=g, device="cuda")
        L = L + (3.0 * (perm + 1).float().pow(-1.2))[None, :]
    return L


def _topk(L, k, renorm):
    p = torch.softmax(L.double(), -1)
    _, idx = torch.sort(L, dim=-1, descending=True, stable=True)
    idx = idx[:, :k].contiguous()
    w = p.gather(1, idx)
    if renorm:
        w = w / w.sum(-1, keepdim=True)
    return idx, w.float().contiguous()


def _dispatched(case, g):
    """idx, weights, counts, offsets, pos and src_token of a routed batch."""
    idx, w = _topk(_logits(case, g), case["k"], True)
    flat = idx.reshape(-1)
    order = torch.sort(flat, stable=True).indices
    pos = torch.empty_like(order)
    pos[order] = torch.arange(order.numel(), device="cuda")
    counts = torch.bincount(flat, minlength=case["E"])
    offsets = torch.zeros(case["E"] + 1, dtype=torch.int64, device="cuda")
    offsets[1:] = counts.cumsum(0)
    i32 = torch.int32
    return dict(idx=idx.to(i32), w=w, counts=counts.to(i32), offsets=offsets.to(i32),
                pos=pos.to(i32), src_token=(order // case["k"]).to(i32))


def _clip_tensors(case):
    """(elements, type) of every gradient tensor of a case."""
    if case["layer"]:  # gate/up, down, router weight, router bias of the Mixtral-shaped layer
        return [(8 * 4096 * 28672, BF16), (8 * 14336 * 4096, BF16), (8 * 4096, F32), (8, F32)]
    r = random.Random(case["n"] * 1000003 + case["large"])
    sizes = [_log(r, case["small"], case["large"]) for _ in range(case["n"])]
    return [(n, F32 if case["dtype"] == F32 or (case["dtype"] == "mixed" and i % 3 == 2) else BF16)
            for i, n in enumerate(sizes)]


def prepare(case, seed):
    g = _gen(seed)
    dt = _torch_dtype(case)
    s = dict(case=dict(case), kept={})
    if case["op"] == "clip":
        # gradients as views of two flat buffers, back to back, and such buffers for the copies
        tensors = _clip_tensors(case)
        flat, out, used = {}, {}, {BF16: 0, F32: 0}
        for n, t in tensors:
            used[t] += n
        for t, n in used.items():
            dtype = torch.bfloat16 if t == BF16 else torch.float32
            if n:
                flat[t] = _randn(g, n, std=2e-3, dtype=dtype)
                out[t] = torch.empty_like(flat[t])
        at = {BF16: 0, F32: 0}
        grads, outs = [], []
        for n, t in tensors:
            grads.append(flat[t][at[t]:at[t] + n])
            outs.append(out[t][at[t]:at[t] + n])
            at[t] += n
        s.update(grads=grads, outs=outs, flat_out=[out[t] for t in sorted(out)], max_norm=1e-2,
                 types=[dict(bf16=torch.bfloat16, f32=torch.float32)[t] for t in sorted(out)],
                 order=[[i for i, x in enumerate(tensors) if x[1] == t] for t in sorted(out)])
        return s
    T, d, k = case["T"], case["d"], case["k"]
    if case["op"] == "route":
        L = _logits(case, g)
        idx, w = _topk(L, k, case["renorm"])
        s.update(logits=L, idx=idx.to(torch.int32), w=w, x=_randn(g, T, d, dtype=dt),
                 Wr=_randn(g, case["E"], d, std=d ** -0.5), dw=_randn(g, T, k, std=0.1))
        return s
    s.update(_dispatched(case, g))
    P = T * k
    if case["op"] == "combine":
        s.update(dout=_randn(g, T, d, std=0.02, dtype=dt), y_perm=_randn(g, P, d, dtype=dt))
    elif case["op"] == "dispatch":
        s.update(dx_perm=_randn(g, P, d, std=0.02, dtype=dt), x=_randn(g, T, d, dtype=dt))
    else:
        f, E = case["f"], case["E"]
        x = _randn(g, T, d, dtype=dt)
        s.update(x_perm=x[s["src_token"].long()], dy_perm=_randn(g, P, d, std=0.02, dtype=dt),
                 Wgu=_randn(g, E, d, 2 * f, std=d ** -0.5, dtype=dt),
                 Wd=_randn(g, E, f, d, std=d ** -0.5, dtype=dt),
                 h_perm=torch.empty(P, f, dtype=dt, device="cuda"))
        ends = s["offsets"].tolist()
        s["cap"] = max(b - a for a, b in zip(ends, ends[1:]))  # the most rows of one expert
        for e in range(E):  # the activations that the forward pass left behind
            a, b = ends[e], ends[e + 1]
            if b > a:
                gu = (s["x_perm"][a:b] @ s["Wgu"][e]).float()
                s["h_perm"][a:b] = (gu[:, :f] * torch.sigmoid(gu[:, :f]) * gu[:, f:]).to(dt)
    return s


# ------------------------------- the passes --------------------------------
def run(s):
    op = s["case"]["op"]
    return globals()[("_own_" if own else "_plain_") + op](s)


def _plain_combine(s):
    T, k, d = s["case"]["T"], s["case"]["k"], s["case"]["d"]
    dt, pos = s["dout"].dtype, s["pos"].long()
    g = s["dout"].float()[:, None, :]
    rows = s["y_perm"].float()[pos].view(T, k, d)
    dw = (rows * g).sum(-1)
    dy = torch.empty(T * k, d, dtype=torch.float32, device="cuda")
    dy[pos] = (s["w"][:, :, None] * g).view(T * k, d)
    return dict(dy_perm=dy.to(dt), dw=dw)


def _plain_dispatch(s):
    T, k, d = s["case"]["T"], s["case"]["k"], s["case"]["d"]
    dt = s["x"].dtype
    rows = s["dx_perm"].float()[s["pos"].long()].view(T, k, d)
    if not s["case"]["scale"]:
        return dict(dx=rows.sum(1).to(dt))
    dw = (rows * s["x"].float()[:, None, :]).sum(-1)
    return dict(dx=(rows * s["w"][:, :, None]).sum(1).to(dt), dw=dw)


def _plain_experts(s):
    """Every expert's rows padded to the longest segment, batched products."""
    c = s["case"]
    E, f, cap, dt = c["E"], c["f"], s["cap"], s["x_perm"].dtype
    first, counts = s["offsets"][:-1].long(), s["counts"].long()
    slot = torch.arange(cap, device="cuda")
    there = slot[None, :] < counts[:, None]
    row = (first[:, None] + slot[None, :])[there]

    def padded(rows):
        out = torch.zeros(E, cap, rows.shape[1], dtype=torch.float32, device="cuda")
        out[there] = rows.float()[row]
        return out

    def ragged(pad):
        return pad[there].to(dt)

    x, dy, Wgu = padded(s["x_perm"]), padded(s["dy_perm"]), s["Wgu"].float()
    gu = torch.bmm(x, Wgu)
    gate, up = gu[..., :f], gu[..., f:]
    sig = 1.0 / (1.0 + torch.exp(-gate))
    dh = torch.bmm(dy, s["Wd"].float().transpose(1, 2))
    dgu = torch.cat([dh * up * sig * (1.0 + gate * (1.0 - sig)), dh * gate * sig], -1)
    del gu, gate, up, sig, dh
    dx = ragged(torch.bmm(dgu, Wgu.transpose(1, 2)))
    del Wgu
    dWgu = torch.bmm(x.transpose(1, 2), dgu).to(dt)
    del dgu, x
    dWd = torch.bmm(padded(s["h_perm"]).transpose(1, 2), dy).to(dt)
    return dict(dx_perm=dx, dWgu=dWgu, dWd=dWd)


def _plain_route(s):
    c = s["case"]
    idx, w, dw = s["idx"].long(), s["w"], s["dw"]
    inner = (w * dw).sum(-1, keepdim=True)
    dL = torch.zeros_like(s["logits"])
    if c["renorm"]:
        dL.scatter_(1, idx, w * (dw - inner))
    else:
        e = torch.exp(s["logits"] - s["logits"].max(-1, keepdim=True).values)
        p = e / e.sum(-1, keepdim=True)
        dL.scatter_(1, idx, dw)
        dL = p * (dL - inner)
    x = s["x"].float()
    return dict(dlogits=dL, dWr=dL.t() @ x, dbias=dL.sum(0), dx=(dL @ s["Wr"]).to(s["x"].dtype))


def _plain_clip(s):
    norm = torch.stack([g.float().square().sum() for g in s["grads"]]).sum().sqrt()
    coef = torch.clamp(s["max_norm"] / (norm + 1e-6), max=1.0)
    flat = [torch.cat([s["grads"][i].float() * coef for i in at]).to(t)
            for at, t in zip(s["order"], s["types"])]
    return dict(norm=norm, clipped=flat)


def _kept(s, **shapes):
    """Output and workspace buffers that a training loop allocates once."""
    if not s["kept"]:
        for name, (shape, dtype) in shapes.items():
            s["kept"][name] = torch.empty(shape, dtype=dtype, device="cuda")
    return s["kept"]


def _config(s):
    from token_dispatch_grouped_fp32_gb300 import moe
    c = s["case"]
    return moe, moe.config(c["T"], c["d"], c["E"], c["k"], c.get("f", 8), c["dtype"],
                           renormalize=c.get("renorm", True), scale_inputs=c.get("scale", False))


def _own_combine(s):
    moe, cfg = _config(s)
    k = _kept(s, dy=(s["y_perm"].shape, s["y_perm"].dtype), dw=(s["w"].shape, torch.float32))
    moe.moe_combine_backward(cfg, s["dout"], s["y_perm"], s["pos"], s["w"], k["dy"], k["dw"])
    return dict(dy_perm=k["dy"], dw=k["dw"])


def _own_dispatch(s):
    moe, cfg = _config(s)
    k = _kept(s, dx=(s["x"].shape, s["x"].dtype), dw=(s["w"].shape, torch.float32))
    if not s["case"]["scale"]:
        moe.moe_dispatch_backward(cfg, s["dx_perm"], s["pos"], None, None, k["dx"], None)
        return dict(dx=k["dx"])
    moe.moe_dispatch_backward(cfg, s["dx_perm"], s["pos"], s["w"], s["x"], k["dx"], k["dw"])
    return dict(dx=k["dx"], dw=k["dw"])


def _own_experts(s):
    moe, cfg = _config(s)
    n = moe.moe_grouped_swiglu_backward_workspace_size(cfg)
    k = _kept(s, dx=(s["x_perm"].shape, s["x_perm"].dtype), dWgu=(s["Wgu"].shape, s["Wgu"].dtype),
              dWd=(s["Wd"].shape, s["Wd"].dtype), ws=((n,), torch.uint8))
    moe.moe_grouped_swiglu_backward(cfg, s["x_perm"], s["offsets"], s["Wgu"], s["Wd"], s["h_perm"],
                                    s["dy_perm"], k["dx"], k["dWgu"], k["dWd"], k["ws"])
    return dict(dx_perm=k["dx"], dWgu=k["dWgu"], dWd=k["dWd"])


def _own_route(s):
    moe, cfg = _config(s)
    n = moe.moe_route_backward_workspace_size(cfg)
    k = _kept(s, dL=(s["logits"].shape, torch.float32), dWr=(s["Wr"].shape, torch.float32),
              db=((s["case"]["E"],), torch.float32), dx=(s["x"].shape, s["x"].dtype),
              ws=((n,), torch.uint8))
    moe.moe_route_backward(cfg, s["x"], s["Wr"], s["logits"], s["idx"], s["w"], s["dw"], None,
                           k["dL"], k["dWr"], k["db"], k["dx"], k["ws"])
    return dict(dlogits=k["dL"], dWr=k["dWr"], dbias=k["db"], dx=k["dx"])


def _own_clip(s):
    from token_dispatch_grouped_fp32_gb300 import moe
    k = s["kept"]
    if not k:
        k["list"] = moe.grad_list(s["grads"], s["outs"])
        k["ws"] = torch.empty(moe.moe_clip_grad_norm_workspace_size(), dtype=torch.uint8,
                              device="cuda")
        k["norm"] = torch.empty((), dtype=torch.float32, device="cuda")
    moe.moe_clip_grad_norm(k["list"], s["max_norm"], k["norm"], k["ws"])
    return dict(norm=k["norm"], clipped=s["flat_out"])


# --------------------------------- the work --------------------------------
def work(case):
    op, es = case["op"], 2 if case["dtype"] == BF16 else 4
    if op == "clip":
        n = sum(x * (2 if t == BF16 else 4) for x, t in _clip_tensors(case))
        return dict(bytes=2 * n, flops=n)
    T, d, k = case["T"], case["d"], case["k"]
    P = T * k
    if op == "combine":
        return dict(bytes=es * d * (T + 2 * P) + 12 * P, flops=3 * P * d)
    if op == "dispatch":
        if not case["scale"]:
            return dict(bytes=es * d * (T + P) + 4 * P, flops=P * d)
        return dict(bytes=es * d * (2 * T + P) + 12 * P, flops=4 * P * d)
    E = case["E"]
    if op == "route":
        # renormalised weights: only the chosen logits have a gradient
        n = P if case["renorm"] else T * E
        read = es * T * d + 4 * E * d + 12 * P + (0 if case["renorm"] else 4 * T * E)
        return dict(bytes=read + 4 * T * E + 4 * E * (d + 1) + es * T * d, flops=4 * n * d)
    f = case["f"]
    held = min(E, P)  # experts that can have rows: the others' weights are not read
    return dict(bytes=es * (P * (3 * d + f) + 3 * d * f * (held + E)) + 4 * (E + 1),
                flops=16 * P * d * f)


# ------------------------------ in 64 bits ---------------------------------
def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "clip":
        sums = torch.zeros((), dtype=torch.float64, device="cuda")
        for g in s["grads"]:
            for part in g.split(1 << 27):
                sums += torch.dot(part.double(), part.double())
        norm = torch.sqrt(sums)
        scale = min(1.0, s["max_norm"] / (norm.item() + 1e-6))
        flat = []
        for at in s["order"]:
            parts = [s["grads"][i].double().mul_(scale) for i in at]
            flat.append(torch.cat(parts) if len(parts) > 1 else parts[0])
        return dict(norm=norm, clipped=flat)
    T, d, k = case["T"], case["d"], case["k"]
    if op == "route":
        n = torch.arange(T, device="cuda")
        dL = torch.zeros(T, case["E"], dtype=torch.float64, device="cuda")
        w, dw = s["w"].double(), s["dw"].double()
        if case["renorm"]:  # the Jacobian of a softmax over the chosen logits
            J = torch.diag_embed(w) - w[:, :, None] * w[:, None, :]
            part = torch.einsum("tij,tj->ti", J, dw)
            for j in range(k):
                dL[n, s["idx"][:, j].long()] = part[:, j]
        else:
            p = torch.softmax(s["logits"].double(), -1)
            for j in range(k):
                e = s["idx"][:, j].long()
                dL -= (w[:, j] * dw[:, j])[:, None] * p
                dL[n, e] += p[n, e] * dw[:, j]
        return dict(dlogits=dL, dWr=torch.einsum("te,td->ed", dL, s["x"].double()),
                    dbias=torch.einsum("te->e", dL), dx=torch.einsum("te,ed->td", dL, s["Wr"].double()))
    pos = s["pos"].long().view(T, k)
    if op == "combine":
        g, dy = s["dout"].double(), torch.empty(T * k, d, dtype=torch.float64, device="cuda")
        dw = torch.empty(T, k, dtype=torch.float64, device="cuda")
        for j in range(k):
            dy[pos[:, j]] = g * s["w"][:, j:j + 1].double()
            dw[:, j] = torch.einsum("td,td->t", g, s["y_perm"][pos[:, j]].double())
        return dict(dy_perm=dy, dw=dw)
    if op == "dispatch":
        dx = torch.zeros(T, d, dtype=torch.float64, device="cuda")
        dw = torch.empty(T, k, dtype=torch.float64, device="cuda")
        for j in range(k):
            r = s["dx_perm"][pos[:, j]].double()
            dx += r * s["w"][:, j:j + 1].double() if case["scale"] else r
            dw[:, j] = torch.einsum("td,td->t", s["x"].double(), r)
        return dict(dx=dx, dw=dw) if case["scale"] else dict(dx=dx)
    f, E, ends = case["f"], case["E"], s["offsets"].tolist()
    dx = torch.zeros(T * k, d, dtype=torch.float64, device="cuda")
    dWgu = torch.zeros(E, d, 2 * f, dtype=torch.float64, device="cuda")
    dWd = torch.zeros(E, f, d, dtype=torch.float64, device="cuda")
    for e in range(E):
        a, b = ends[e], ends[e + 1]
        x, dy = s["x_perm"][a:b].double(), s["dy_perm"][a:b].double()
        W = s["Wgu"][e].double()
        gate, up = x @ W[:, :f], x @ W[:, f:]
        dh = dy @ s["Wd"][e].double().t()
        sg = torch.sigmoid(gate)
        dgate, dup = dh * up * (sg + gate * sg * (1 - sg)), dh * (gate * sg)
        dx[a:b] = dgate @ W[:, :f].t() + dup @ W[:, f:].t()
        dWgu[e, :, :f], dWgu[e, :, f:] = x.t() @ dgate, x.t() @ dup
        dWd[e] = s["h_perm"][a:b].double().t() @ dy
    return dict(dx_perm=dx, dWgu=dWgu, dWd=dWd)
