"""Trains one pre-norm residual MoE block with the library's operators:

    h -> layer_norm_forward -> moe_ffn_forward -> h + out        forward
    moe_ffn_backward -> layer_norm_backward (+ the residual path) backward
    muon_step on W1, W3, W2 of all experts, plain SGD on the rest  update

The block learns to reproduce a second, fixed block of the same shape on
random inputs.  Expert weights have fp32 masters, which muon_step updates
together with the bf16 copies that the layer reads.

    python examples/train_moe_block.py            # the benchmark layer's shape, fewer tokens
"""
from __future__ import annotations

import argparse
import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from grouped_gemm_router_gb300 import moe  # noqa: E402


class Block:
    """y = h + MoE(LN(h)) with a bf16 residual stream."""

    def __init__(self, T, D, F, E, k, gen):
        r = lambda *s: torch.randn(*s, generator=gen, device="cuda")
        self.dims, self.k = (T, D, F, E), k
        self.ln_w, self.ln_b = torch.ones(D, device="cuda"), torch.zeros(D, device="cuda")
        self.master = dict(W1=r(E, D, F) / math.sqrt(D), W3=r(E, D, F) / math.sqrt(D), W2=r(E, F, D) / math.sqrt(F))
        self.w = {n: v.bfloat16() for n, v in self.master.items()}
        self.Wg = (r(D, E) / math.sqrt(D)).bfloat16()
        self.momentum = {n: torch.zeros_like(v) for n, v in self.master.items()}
        self.ws = moe.Workspace(T, D, F, E, k, False)
        self.bws = moe.BackwardWorkspace(T, D, F, E, k, False)
        self.muon_ws = torch.empty(moe.newton_schulz_workspace_size(3 * E, D, F), dtype=torch.uint8, device="cuda")

    def forward(self, h):
        n = moe.layer_norm_forward(h, self.ln_w, bias=self.ln_b)
        out = moe.moe_ffn_forward(n["y"], self.Wg, self.w["W1"], self.w["W3"], self.w["W2"], self.k, workspace=self.ws)
        return h + out, n

    def backward(self, h, n, d):
        """Gradients for d = the gradient of h + MoE(LN(h))."""
        g = moe.moe_ffn_backward(n["y"], self.Wg, self.w["W1"], self.w["W3"], self.w["W2"], self.k, d, self.ws,
                                 bwd_workspace=self.bws)
        g.update(moe.layer_norm_backward(g["dx"], h, self.ln_w, n["mean"], n["rstd"], d_stream=d))
        return g

    def update(self, g, lr):
        names = ("W1", "W3", "W2")
        moe.muon_step([self.master[n] for n in names], [g["d" + n] for n in names], [self.momentum[n] for n in names],
                      lr=lr, weights_bf16=[self.w[n] for n in names], workspace=self.muon_ws)
        self.ln_w -= 10 * lr * g["dweight"]
        self.ln_b -= 10 * lr * g["dbias"]
        self.Wg.copy_(self.Wg.float() - 10 * lr * g["dWg"])


def train(steps=30, T=4096, D=768, F=1536, E=8, k=2, lr=0.01, seed=0, log=None):
    """Losses (mean squared error to the other block's outputs) of every step."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    teacher, student = Block(T, D, F, E, k, gen), Block(T, D, F, E, k, gen)
    losses = []
    for i in range(steps):
        h = torch.randn(T, D, generator=gen, device="cuda").bfloat16()
        target, _ = teacher.forward(h)
        y, n = student.forward(h)
        diff = y.float() - target.float()
        losses.append(float(diff.square().mean()))
        d = (diff * (2 / diff.numel())).bfloat16()
        student.update(student.backward(h, n, d), lr)
        if log:
            log(f"step {i:3d}  loss {losses[-1]:.5f}")
    if moe.device_error() != 0:
        raise RuntimeError("a device wait timed out")
    return losses


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--steps", type=int, default=30)
    ap.add_argument("--tokens", type=int, default=4096)
    a = ap.parse_args()
    train(a.steps, T=a.tokens, log=print)
