"""Plain 64-bit forward steps of the layer in torch, for the gradient tests:
their gradients come from double-precision automatic differentiation and from
central differences, never from the formulas the kernels use.  Routing (the
chosen experts) is an input: selection has no gradient."""
import torch


def weights(logits, idx, renorm):
    p = torch.softmax(logits, -1).gather(1, idx)
    return p / p.sum(-1, keepdim=True) if renorm else p


def ffn_rows(rows, offsets, Wgu, Wd):
    """y of every row of the segments [offsets[e], offsets[e+1])."""
    f = Wd.shape[1]
    out = []
    for e in range(len(offsets) - 1):
        gu = rows[offsets[e]:offsets[e + 1]] @ Wgu[e]
        g, u = gu[:, :f], gu[:, f:]
        out.append((g * torch.sigmoid(g) * u) @ Wd[e])
    return torch.cat(out)


def permute(idx, E):
    """pos [T*k], offsets [E+1] (list) and source pair of every row."""
    flat = idx.reshape(-1)
    order = torch.sort(flat, stable=True).indices
    pos = torch.empty_like(order)
    pos[order] = torch.arange(order.numel(), device=idx.device)
    counts = torch.bincount(flat, minlength=E)
    offsets = [0] + torch.cumsum(counts, 0).tolist()
    return pos, offsets, order


def layer(x, Wr, bias, Wgu, Wd, idx, renorm=True, scale_inputs=False):
    T, k = idx.shape
    logits = x @ Wr.t() + (0 if bias is None else bias)
    w = weights(logits, idx, renorm)
    pos, offsets, order = permute(idx, Wr.shape[0])
    rows = x[order // k]
    if scale_inputs:
        rows = rows * w.reshape(-1)[order][:, None]
    y = ffn_rows(rows, offsets, Wgu, Wd)[pos].view(T, k, -1)
    return y.sum(1) if scale_inputs else (w[:, :, None] * y).sum(1)


def grads(fn, inputs, out_grad):
    """Gradients of <fn(*inputs), out_grad> by automatic differentiation."""
    leaves = [t.detach().clone().requires_grad_(True) for t in inputs]
    return torch.autograd.grad((fn(*leaves) * out_grad).sum(), leaves, allow_unused=True)


def difference(fn, inputs, i, direction, out_grad, h):
    """Central difference of <fn(*inputs), out_grad> along `direction` in input i."""
    def at(s):
        args = list(inputs)
        args[i] = args[i] + s * direction
        return float((fn(*args) * out_grad).sum())
    return (at(h) - at(-h)) / (2 * h)
