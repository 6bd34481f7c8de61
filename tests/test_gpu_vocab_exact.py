"""The vocabulary product itself, through distill_forward's logits and lse, at
widths from one sum of the tensor cores to many.

Rows whose products are exact in 24 bits (one element a row, a few, whole
numbers) give exact logits: no sum of theirs is cut or rounded.  lse is off by
c = log2 e rounded, by ln 2 rounded and by two products, 2^-22 of itself, and by
2^-13 for ex2, log2 and the sums.

Dense rows of one sign: the tensor cores add 16 products at a time, and such a
step cuts at most two units of the last place of 24 bits, 2^-22 of the sum so
far.  At most 512 products are summed like that, 32 steps: 2^-17 of the sum of
magnitudes A.  The sums of up to 8192 / 512 parts are rounded to nearest:
another 16 times 2^-24."""
import numpy as np
import pytest
import torch

import _lm_ref as ref
import test_gpu_vocab_loss as base

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


@pytest.fixture(scope="module")
def moe():
    from grouped_gemm_router_gb300 import build
    build.build()
    from grouped_gemm_router_gb300 import moe as m
    yield m
    assert m.device_error() == 0


def _exact_rows(kind, T, D, V):
    g = torch.Generator(device="cuda").manual_seed(D + T)
    if kind == "whole numbers":
        x = torch.randint(-3, 4, (T, D), generator=g, device="cuda")
        W = torch.randint(-3, 4, (V, D), generator=g, device="cuda")
        return g, x.to(BF), W.to(BF)
    n = 1 if kind == "one element" else 4
    W = torch.randn(V, D, generator=g, device="cuda").to(BF)
    x = torch.zeros(T, D, device="cuda")
    at = torch.rand(T, D, generator=g, device="cuda").argsort(dim=1)[:, :n]
    if n == 4:  # W in steps of 2^-6 and whole numbers in x: 24 bits hold every sum
        W = (W.float() * 64).round().clamp(-255, 255).div(64).to(BF)
    x.scatter_(1, at, torch.randint(1, 64, (T, n), generator=g, device="cuda").float())
    return g, x.to(BF), W


@pytest.mark.parametrize("kind", ["one element", "four elements", "whole numbers"])
@pytest.mark.parametrize("T,D,V", [(70, 64, 300), (40, 512, 700), (300, 576, 257), (33, 1088, 900), (130, 2048, 513),
                                   (257, 4096, 300), (40, 8192, 1000)])
def test_exact_products(moe, kind, T, D, V):
    g, x, W = _exact_rows(kind, T, D, V)
    ids = torch.randint(0, V, (T, 9), generator=g, device="cuda")
    z = x.double() @ W.double().t()
    at = z.gather(1, ids)
    assert torch.equal(at, at.float().double())
    f = moe.distill_forward(x, W, ids, torch.zeros(T, 9, device="cuda"))
    assert torch.equal(f["logits"].double(), at)
    labels = ids[:, 0].contiguous()
    c = moe.cross_entropy_forward(x, W, labels)
    lse = torch.logsumexp(z, 1)
    tol = 2.0 ** -22 * lse.abs() + 2.0 ** -13
    for got in (f["lse"], c["lse"]):
        assert ((got.double() - lse).abs() <= tol).all(), float(((got.double() - lse).abs() / tol).max())
    # a loss adds its logit's own error, none, times the rounded factors: 2^-22 of the logit
    loss = lse - at[:, 0]
    assert ((c["loss"].double() - loss).abs() <= tol + 2.0 ** -22 * at[:, 0].abs()).all()


@pytest.mark.parametrize("T,D,V", [(33, 512, 300), (70, 1216, 257), (130, 2048, 300), (40, 8192, 300)])
def test_rows_of_one_sign(moe, T, D, V):
    g = torch.Generator(device="cuda").manual_seed(D)
    x = (torch.rand(T, D, generator=g, device="cuda") + 0.5).to(BF)
    W = ((torch.rand(V, D, generator=g, device="cuda") + 0.5) / D ** 0.5).to(BF)
    z = x.double() @ W.double().t()
    ids = torch.randint(0, V, (T, 31), generator=g, device="cuda")
    f = moe.distill_forward(x, W, ids, torch.zeros(T, 31, device="cuda"))
    off = 56 * 2.0 ** -22 + 10 * 2.0 ** -24
    at = z.gather(1, ids)
    worst = ((f["logits"].double() - at).abs() / at).max()
    assert worst <= off, float(worst)
    lse = torch.logsumexp(z, 1)
    tol = (off + 2.0 ** -22) * lse.abs() + 2.0 ** -13
    assert ((f["lse"].double() - lse).abs() <= tol).all()


@pytest.mark.parametrize("T,D,V", [(40, 576, 300), (257, 1088, 700), (130, 2048, 513), (20, 8192, 700)])
@pytest.mark.parametrize("dense", [False, True])
def test_gradients_of_sums_in_parts(moe, T, D, V, dense):
    """The gradients' bound is that of test_gpu_vocab_loss, whose 2^-13 for
    exp(z - lse) holds here: logits of a few tens."""
    g, x, W = _exact_rows("one element", T, D, V)
    if dense:
        _, x, W, _ = base._inputs(T, D, V)
    else:
        x = (x.float() / 16).to(BF)
    labels = torch.randint(-1, V + 1, (T,), generator=g, device="cuda")
    base._check_ce(moe, x, W, labels, g)
    ids, logits = base._teacher(g, T, V, 12)
    f = moe.distill_forward(x, W, ids, logits, temperature=2.0)
    dl = torch.randn(T, generator=g, device="cuda")
    got = moe.distill_backward(dl, x, W, ids, logits, f["lse"], f["logits"], temperature=2.0)
    xn, wn = base._np(x), base._np(W)
    dz = ref.distill_dz(xn, wn, ids.cpu().numpy(), base._np(logits), 2.0, base._np(dl))
    base._check_gradients(got, dz, xn, wn, "distillation")
    assert np.isfinite(dz).all()
