"""One FSDP unit that computes: the MLP half of a GPT block (layer norm, two
linear layers with a GELU between them, the residual), trained on random
targets by N virtual data-parallel ranks.

Each step gathers the unit's bf16 parameters, runs every rank's forward and
backward pass on its own tokens with the library's block operators, writes the
gradients where the reduce-scatter reads them (the rank's flat gradient), and
updates the sharded parameters with AdamW.  Between the forward and the
backward pass a rank keeps the layer norm's input and the GELU's input in 8
bits, instead of four bf16 tensors.

    python examples/train_mlp_unit.py [--d 1280] [--ffn 5120] [--tokens 4096] [--ranks 4] [--steps 10]
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

from fully_sharded_unit_gb300 import binding as B  # noqa: E402

EPS = 1e-5


class MlpUnit:
    """ln -> c_fc + GELU -> c_proj + residual, sharded over ``ranks`` (FlatParameter
    layout), with bf16 compute and gradients of ``grad_dtype``."""

    def __init__(self, d, ffn, tokens, ranks, grad_dtype="bf16", seed=0, std=0.02):
        self.d, self.ffn, self.tokens, self.ranks = d, ffn, tokens, ranks
        self.shapes = [(d,), (d,), (d, ffn), (ffn,), (ffn, d), (d,)]   # ln w, b; c_fc W, b; c_proj W, b
        self.unit = B.Unit(self.shapes, "flat", ranks, grad_dtype)
        gen = torch.Generator(device="cuda")
        gen.manual_seed(seed)
        self.init = [torch.ones(d, device="cuda"), torch.zeros(d, device="cuda"),
                     torch.empty((d, ffn), device="cuda").normal_(0, std, generator=gen), torch.zeros(ffn, device="cuda"),
                     torch.empty((ffn, d), device="cuda").normal_(0, std, generator=gen), torch.zeros(d, device="cuda")]
        self.unit.load(self.init)
        bf = torch.bfloat16
        self.gathered = torch.empty(self.unit.numel, dtype=bf, device="cuda")
        gdt = bf if grad_dtype == "bf16" else torch.float32
        self.grads = [torch.empty(self.unit.numel, dtype=gdt, device="cuda") for _ in range(ranks)]
        self.params = self._views(self.gathered)
        # one compute handle for every operator: the larger workspace of the two kinds
        weights = (self.params[2], self.params[4])   # pieces of the gathered buffer: they begin where it has them
        self.compute = B.Compute(max(B.fsdp_linear_workspace_bytes(tokens, d, ffn, weight_aligned=weights),
                                     B.fsdp_layer_norm_workspace_bytes(tokens, d)))
        self.mean, self.rstd = torch.empty(tokens, device="cuda"), torch.empty(tokens, device="cuda")
        self.wide, self.narrow = (torch.empty((tokens, n), dtype=bf, device="cuda") for n in (ffn, d))
        self.y, self.dx = (torch.empty((tokens, d), dtype=bf, device="cuda") for _ in range(2))
        # what is kept from the forward to the backward pass
        self.x8, self.z8 = B.Act8(tokens, d), B.Act8(tokens, ffn)

    def _views(self, flat):
        out, at = [], 0
        for s in self.shapes:
            n = s[0] * (s[1] if len(s) > 1 else 1)
            out.append(flat[at:at + n].view(s))
            at += n
        return out

    @property
    def kept_bytes(self):
        return self.x8.nbytes + self.z8.nbytes + 8 * self.tokens

    def forward(self, x):
        c, (lw, lb, w1, b1, w2, b2) = self.compute, self.params
        c.layer_norm_forward(x, lw, lb, EPS, self.narrow, self.mean, self.rstd, ckpt=self.x8)
        c.linear_forward(self.narrow, w1, self.wide, bias=b1, activation="gelu_tanh", preact=self.z8)
        c.linear_forward(self.wide, w2, self.y, bias=b2, residual=x)
        return self.y

    def backward(self, dy, rank):
        """The input's gradient; the parameters' go into the rank's flat gradient."""
        c, (lw, lb, w1, b1, w2, b2) = self.compute, self.params
        glw, glb, gw1, gb1, gw2, gb2 = self._views(self.grads[rank])
        h = self.wide
        c.act8_unpack(self.z8, h, activation="gelu_tanh")            # the GELU's output, recomputed
        c.linear_grad_weight(h, dy, gw2, dbias=gb2)
        c.linear_grad_input(dy, w2, h, activation="gelu_tanh", preact=self.z8)   # the GELU's input gradient
        # the normalised input, recomputed from the kept one
        x = self.dx
        c.act8_unpack(self.x8, x)
        c.layer_norm_forward(x, lw, lb, EPS, self.narrow, torch.empty_like(self.mean), torch.empty_like(self.rstd))
        c.linear_grad_weight(self.narrow, h, gw1, dbias=gb1)
        c.linear_grad_input(h, w1, self.narrow)
        c.layer_norm_backward(self.narrow, self.x8, lw, self.mean, self.rstd, self.dx, glw, glb, add=dy)
        return self.dx

    def step(self, batches, targets, hp):
        """One training step of every rank; the mean loss."""
        self.unit.allgather(self.gathered)
        total = 0.0
        for r, (x, t) in enumerate(zip(batches, targets)):
            diff = self.forward(x).float() - t.float()
            total = total + diff.square().mean()
            self.backward((diff * (2.0 / diff.numel())).to(torch.bfloat16), r)
        self.unit.reduce_scatter(self.grads)
        self.unit.adamw_step(hp)
        return total / self.ranks

    def close(self):
        status = self.compute.status() | self.unit.kernel_status()
        self.compute.close()
        self.unit.close()
        return status


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    for name, default in (("d", 1280), ("ffn", 5120), ("tokens", 4096), ("ranks", 4), ("steps", 10)):
        ap.add_argument(f"--{name}", type=int, default=default)
    a = ap.parse_args()
    m = MlpUnit(a.d, a.ffn, a.tokens, a.ranks)
    gen = torch.Generator(device="cuda")
    gen.manual_seed(1)
    batches = [torch.empty((a.tokens, a.d), device="cuda").normal_(generator=gen).to(torch.bfloat16) for _ in range(a.ranks)]
    targets = [torch.empty((a.tokens, a.d), device="cuda").normal_(generator=gen).to(torch.bfloat16) for _ in range(a.ranks)]
    hp = dict(lr=1e-3, beta1=0.9, beta2=0.999, eps=1e-8, weight_decay=0.01)
    full = a.tokens * 2 * (2 * a.d + 2 * a.ffn)
    print(f"kept between forward and backward: {m.kept_bytes / 2**20:.1f} MiB a rank ({full / 2**20:.1f} MiB as bf16)")
    m.step(batches, targets, hp)
    begin, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    losses = []
    begin.record()
    for _ in range(a.steps):
        losses.append(m.step(batches, targets, hp))
    end.record()
    torch.cuda.synchronize()
    print("loss " + " ".join(f"{v.item():.4f}" for v in losses))
    flops = a.ranks * 3 * 2 * 2 * a.tokens * a.d * a.ffn
    ms = begin.elapsed_time(end) / a.steps
    print(f"{ms:.3f} ms a step, {flops / ms / 1e9:.0f} TFLOP/s in the products")
    if m.close():
        sys.exit("a kernel gave up waiting")


if __name__ == "__main__":
    main()
