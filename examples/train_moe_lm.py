"""Trains a small language model of one pre-norm MoE block with a tied table:

    embedding_forward -> block -> layer_norm_forward -> cross_entropy_forward     forward
    cross_entropy_backward -> layer_norm_backward -> block -> embedding_backward  backward
    muon_step on the experts, plain SGD on the rest                               update

The table [V, D] is the embedding's and the head's; embedding_backward adds the
head's gradient to its own.  With --distill the model learns from the top logits
of a second, fixed model (distill_forward, distill_backward) instead of labels.
The text is a random walk over the vocabulary: each word is followed by one of
four.

    python examples/train_moe_lm.py            # the benchmark layer's shape, fewer tokens
"""
from __future__ import annotations

import argparse
import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from examples.train_moe_block import Block  # noqa: E402
from grouped_gemm_router_gb300 import moe  # noqa: E402

LOG_Z = 1e-4  # weight of the squared log of the softmax's sum


class Model:
    def __init__(self, T, D, F, E, k, V, gen):
        self.V, self.scale = V, math.sqrt(D)
        self.master = torch.randn(V, D, generator=gen, device="cuda") / math.sqrt(D)
        self.table = self.master.bfloat16()
        self.block = Block(T, D, F, E, k, gen)
        self.norm = torch.ones(D, device="cuda")
        n_teacher = 8
        self.n_teacher = n_teacher
        sizes = [moe.vocab_workspace_size(T, D, V, n, backward=b) for n in (0, n_teacher) for b in (False, True)]
        self.ws = torch.empty(max(*sizes, moe.embedding_backward_workspace_size(T, V, D)), dtype=torch.uint8, device="cuda")

    def hidden(self, ids):
        """What the head reads, and what the backward needs."""
        h0 = moe.embedding_forward(ids, self.table, scale=self.scale)
        h1, n = self.block.forward(h0)
        return moe.layer_norm_forward(h1, self.norm), (h0, n, h1)

    def backward(self, ids, f, kept, head):
        """Gradients from the head's dict(dx, dW)."""
        h0, n, h1 = kept
        top = moe.layer_norm_backward(head["dx"], h1, self.norm, f["mean"], f["rstd"], bias=False)
        g = self.block.backward(h0, n, top["dx"])
        g["dnorm"] = top["dweight"]
        g["dtable"] = moe.embedding_backward(g["dx"], ids, self.V, scale=self.scale, add=head["dW"], workspace=self.ws)
        return g

    def loss_and_gradients(self, ids, labels):
        """Mean cross entropy over the tokens with a label (plus LOG_Z times
        the mean square of log Z), and the gradients of both."""
        f, kept = self.hidden(ids)
        c = moe.cross_entropy_forward(f["y"], self.table, labels, workspace=self.ws)
        count = ((labels >= 0) & (labels < self.V)).sum().clamp(min=1)
        d_loss = torch.ones_like(c["loss"]) / count
        d_lse = 2 * LOG_Z / len(ids) * c["lse"]
        head = moe.cross_entropy_backward(d_loss, f["y"], self.table, labels, c["loss"], c["lse"], d_lse=d_lse,
                                          workspace=self.ws)
        return c["loss"].sum() / count, self.backward(ids, f, kept, head)

    def distill(self, ids, teacher_ids, teacher_logits, temperature):
        """The same from a teacher's entries for each token."""
        f, kept = self.hidden(ids)
        args = f["y"], self.table, teacher_ids, teacher_logits
        c = moe.distill_forward(*args, temperature=temperature, workspace=self.ws)
        d_loss = torch.full_like(c["loss"], temperature ** 2 / len(ids))
        head = moe.distill_backward(d_loss, *args, c["lse"], c["logits"], temperature=temperature, workspace=self.ws)
        return c["loss"].mean(), self.backward(ids, f, kept, head)

    def update(self, g, lr):
        self.block.update(g, lr)
        self.norm -= 10 * lr * g["dnorm"]
        self.master -= 10 * lr * g["dtable"]
        self.table.copy_(self.master)


def train(steps=30, T=4096, D=768, F=1536, E=8, k=2, V=20011, lr=0.01, seed=0, distill=False, log=None):
    """Losses of every step."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    model = Model(T, D, F, E, k, V, gen)
    teacher = Model(T, D, F, E, k, V, gen) if distill else None
    follows = torch.randint(0, V, (V, 4), generator=gen, device="cuda")
    losses = []
    for i in range(steps):
        ids = torch.randint(0, V, (T,), generator=gen, device="cuda")
        if teacher:
            top = (teacher.hidden(ids)[0]["y"] @ teacher.table.t()).float().topk(model.n_teacher, dim=1)
            loss, g = model.distill(ids, top.indices, top.values, 2.0)
        else:
            labels = follows[ids, torch.randint(0, 4, (T,), generator=gen, device="cuda")]
            loss, g = model.loss_and_gradients(ids, labels)
        losses.append(float(loss))
        model.update(g, lr)
        if log:
            log(f"step {i:3d}  loss {losses[-1]:.5f}")
    if moe.device_error() != 0:
        raise RuntimeError("a device wait timed out")
    return losses


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--steps", type=int, default=30)
    ap.add_argument("--tokens", type=int, default=4096)
    ap.add_argument("--distill", action="store_true")
    a = ap.parse_args()
    train(a.steps, T=a.tokens, distill=a.distill, log=print)
