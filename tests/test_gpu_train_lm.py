"""The operators together, as a language model uses them: the example runs, is
the same every time, and its gradients are those of the model in 64 bits."""
import importlib
import os
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def ex():
    from grouped_gemm_router_gb300 import build
    build.build()
    if ROOT not in sys.path:
        sys.path.insert(0, ROOT)
    return importlib.import_module("examples.train_moe_lm")


@pytest.mark.parametrize("distill", [False, True])
def test_the_example_runs(ex, distill):
    sizes = dict(steps=4, T=384, D=128, F=256, E=4, k=2, V=1003, distill=distill)
    losses = ex.train(**sizes)
    assert len(losses) == 4 and all(x == x and 0 < x < 100 for x in losses)
    assert ex.train(**sizes) == losses


def _norm64(h, w):
    mu = h.mean(1, keepdim=True)
    return (h - mu) / ((h - mu).square().mean(1, keepdim=True) + 1e-5).sqrt() * w


def _hidden64(model, ids, p, experts):
    """The model in 64 bits with the experts that the GPU's router chose."""
    b = model.block
    h0 = model.scale * p["table"][ids]
    n = _norm64(h0, b.ln_w.double()) + b.ln_b.double()
    gate = torch.softmax((n @ b.Wg.double()).gather(1, experts), 1)
    out = torch.zeros_like(h0)
    for e in range(p["W1"].shape[0]):
        y = (torch.nn.functional.silu(n @ p["W1"][e]) * (n @ p["W3"][e])) @ p["W2"][e]
        out = out + y * (gate * (experts == e)).sum(1, keepdim=True)
    return _norm64(h0 + out, model.norm.double())


@pytest.mark.parametrize("distill", [False, True])
def test_gradients_of_the_model(ex, distill):
    """Every intermediate between two operators is bf16, rounded by at most 2^-8
    of itself; on the longest way (the head's gradient, two norms, the experts'
    three products and their inputs, the stream) about eight of them add up
    with independent signs: sqrt(8) 2^-8 / sqrt(3) = 6.4e-3 of the rms, and six
    standard deviations of that are 4e-2."""
    T, D, F, E, k, V = 384, 128, 256, 4, 2, 1003
    gen = torch.Generator(device="cuda").manual_seed(3)
    model = ex.Model(T, D, F, E, k, V, gen)
    ids = torch.randint(0, V, (T,), generator=gen, device="cuda")
    labels = torch.where(torch.rand(T, generator=gen, device="cuda") < 0.1, -100,
                         torch.randint(0, V, (T,), generator=gen, device="cuda"))
    t_ids = torch.randint(-1, V, (T, 8), generator=gen, device="cuda")
    t_logits = 2 * torch.randn(T, 8, generator=gen, device="cuda")
    loss, g = model.distill(ids, t_ids, t_logits, 2.0) if distill else model.loss_and_gradients(ids, labels)
    experts = model.block.ws.views()["ids"].long()
    p = dict(table=model.table, **model.block.w)
    p = {n: v.double().requires_grad_() for n, v in p.items()}
    z = _hidden64(model, ids, p, experts) @ p["table"].t()
    if distill:
        known = t_ids >= 0
        q = torch.log_softmax(z / 2, 1).gather(1, t_ids.clamp(min=0))
        t = torch.softmax(torch.where(known, t_logits.double(), -torch.inf) / 2, 1)
        each = torch.where(known, t * (torch.log(t.clamp(min=1e-300)) - q), 0.0).sum(1)
        want, total = each.mean(), 4 * each.mean()
    else:
        known = labels >= 0
        lse = torch.logsumexp(z, 1)
        each = torch.where(known, lse - z.gather(1, labels.clamp(min=0)[:, None])[:, 0], 0.0)
        want = each.sum() / known.sum()
        total = want + ex.LOG_Z * lse.square().mean()
    total.backward()
    assert abs(float(loss.detach()) / float(want.detach()) - 1) < 2 ** -7
    for name, ref in (("dtable", p["table"].grad), ("dW1", p["W1"].grad), ("dW2", p["W2"].grad), ("dW3", p["W3"].grad)):
        rms = ref.square().mean().sqrt()
        off = (g[name].double() - ref).abs() - (4e-2 * rms + 4e-2 * ref.abs())
        assert (off <= 0).all(), f"{name}: {int((off > 0).sum())} of {off.numel()} outside"
