"""One update of the example's model against the step in 64 bits, from the
gradients that it was given: products and differences in fp32, each rounded by
2^-24 of itself, and the table is the master's rounding."""
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


def _check(got, before, grad, step):
    move = step * grad.double()
    want = before.double() - move
    assert ((got.double() - want).abs() <= 2.0 ** -23 * move.abs() + 2.0 ** -24 * 1.0001 * want.abs()).all()
    assert not torch.equal(got, before)


@pytest.mark.parametrize("distill", [False, True])
def test_one_update(ex, distill):
    T, D, V, lr = 384, 128, 1003, 0.01
    gen = torch.Generator(device="cuda").manual_seed(4)
    model = ex.Model(T, D, 256, 4, 2, V, gen)
    ids = torch.randint(0, V, (T,), generator=gen, device="cuda")
    labels = torch.randint(-1, V, (T,), generator=gen, device="cuda")
    if distill:
        t_ids = torch.randint(-1, V, (T, 8), generator=gen, device="cuda")
        _, g = model.distill(ids, t_ids, torch.randn(T, 8, generator=gen, device="cuda"), 2.0)
    else:
        _, g = model.loss_and_gradients(ids, labels)
    b = model.block
    held = [t.clone() for t in (model.master, model.norm, b.ln_w, b.ln_b)]
    experts = {n: w.clone() for n, w in b.master.items()}
    model.update(g, lr)
    for got, before, grad in zip((model.master, model.norm, b.ln_w, b.ln_b), held,
                                 (g["dtable"], g["dnorm"], g["dweight"], g["dbias"])):
        _check(got, before, grad, 10 * lr)
    assert torch.equal(model.table, model.master.bfloat16())
    for n, before in experts.items():
        assert not torch.equal(b.master[n], before) and torch.equal(b.w[n], b.master[n].bfloat16())
