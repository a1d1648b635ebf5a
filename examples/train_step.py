"""A training loop on one MoE layer: forward, loss, backward, gradient
clipping and a plain SGD step, all on one stream with no host
synchronisation inside a step.

The target is another, randomly initialised layer of the same shape; the loss
is a token's squared distance from it, averaged over the tokens.  Run on a GB300:

    python examples/train_step.py [--steps N]
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from token_dispatch_grouped_fp32_gb300 import moe, synth  # noqa: E402


def make_layer(T, d, E, k, f, seed):
    w = synth.Workload("train", T, d, E, k, f, "bf16", seed)
    inp = synth.make_inputs(w, device="cuda")
    bias = torch.zeros(E, device="cuda")
    return moe.MoELayer(inp["Wr"], inp["Wgu"], inp["Wd"], k, bias)


class Trainer:
    """fp32 master weights beside the layer's bf16 ones; every buffer of a
    step is allocated once."""

    def __init__(self, layer, lr=0.5, max_norm=1.0):
        self.layer, self.lr, self.max_norm = layer, lr, max_norm
        self.params = {"Wr": layer.Wr, "W_gate_up": layer.W_gate_up, "W_down": layer.W_down,
                       "logit_bias": layer.logit_bias}
        self.master = {n: p.float() for n, p in self.params.items()}
        self.grads = {n: torch.empty_like(p) for n, p in self.params.items()}
        # clipped in place: the list holds the buffers' addresses
        self.clip = moe.grad_list([self.grads[n] for n in self.params])
        self.clip_ws = torch.empty(moe.moe_clip_grad_norm_workspace_size(), dtype=torch.uint8,
                                   device="cuda")
        self.norm = torch.empty((), device="cuda")

    def step(self, x, target):
        out = self.layer(x)
        diff = out.float() - target.float()
        loss = diff.square().sum(-1).mean()
        dout = (diff * (2.0 / diff.shape[0])).to(out.dtype)
        self.grads["x"] = torch.empty_like(x)
        self.layer.backward(x, dout, grads=self.grads)
        moe.moe_clip_grad_norm(self.clip, self.max_norm, self.norm, self.clip_ws)
        for n, p in self.params.items():
            self.master[n].sub_(self.grads[n].float(), alpha=self.lr)
            p.copy_(self.master[n])
        return loss, self.norm


def main(steps=60, T=2048, d=256, E=16, k=4, f=256):
    teacher, student = make_layer(T, d, E, k, f, 1), make_layer(T, d, E, k, f, 2)
    trainer = Trainer(student)
    gen = torch.Generator(device="cuda").manual_seed(3)
    losses = []
    for i in range(steps):
        x = torch.randn(T, d, generator=gen, device="cuda").to(torch.bfloat16)
        target = teacher(x)
        loss, norm = trainer.step(x, target)
        losses.append(loss)
        if i % 10 == 0 or i == steps - 1:
            print(f"step {i:3d}  loss {float(loss):.3f}  gradient norm {float(norm):.4f}")
    moe.moe_last_device_error()
    return [float(v) for v in losses]


if __name__ == "__main__":
    ap = argparse.ArgumentParser()
    ap.add_argument("--steps", type=int, default=60)
    main(steps=ap.parse_args().steps)
