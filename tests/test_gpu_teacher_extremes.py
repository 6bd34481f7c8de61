"""A teacher's logits at the ends of their types.

p = softmax of the logits over temperature does not change when a constant is
taken from all of them, so rows of the type's lowest or largest value are as
good as rows of zeros; only -inf is no entry.  The probabilities are off by
2^-20 (a difference, a product, an exponential and a sum of up to 40 terms)."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def moe():
    from grouped_gemm_router_gb300 import build
    build.build()
    from grouped_gemm_router_gb300 import moe as m
    return m


def _case(T=6, D=64, V=300, K=40):
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn(T, D, generator=g, device="cuda").to(BF)
    W = (torch.randn(V, D, generator=g, device="cuda") / 8).to(BF)
    ids = torch.rand(T, V, generator=g, device="cuda").argsort(dim=1)[:, :K].contiguous()
    return x, W, ids, torch.ones(T, device="cuda")


@pytest.mark.parametrize("tau", [0.25, 0.5, 1.0, 3.0, 1e30])
@pytest.mark.parametrize("lt", [F32, BF], ids=["f32", "bf16"])
@pytest.mark.parametrize("end", [-1, 1])
def test_rows_at_the_end_of_the_type(moe, tau, lt, end):
    """All entries lowest, or all largest: the bits of a row of zeros."""
    x, W, ids, dl = _case()
    zero = torch.zeros(ids.shape, dtype=lt, device="cuda")
    far = torch.full_like(zero, end * torch.finfo(lt).max)
    a = moe.distill_forward(x, W, ids, zero, temperature=tau)
    b = moe.distill_forward(x, W, ids, far, temperature=tau)
    assert torch.isfinite(a["loss"]).all()
    assert all(torch.equal(a[n], b[n]) for n in a)
    ga = moe.distill_backward(dl, x, W, ids, zero, a["lse"], a["logits"], temperature=tau)
    gb = moe.distill_backward(dl, x, W, ids, far, b["lse"], b["logits"], temperature=tau)
    assert all(torch.equal(ga[n], gb[n]) for n in ga)
    assert tau > 1e6 or ga["dx"].any(dim=1).all()


@pytest.mark.parametrize("tau", [0.25, 0.5, 1.0, 3.0])
def test_both_ends_in_one_row(moe, tau):
    """Some entries largest, the rest lowest: those that are largest share all.
    Beside them -inf and ids outside the vocabulary are no entries, and NaN
    behind such an id is not looked at."""
    x, W, ids, dl = _case()
    most = torch.finfo(F32).max
    far = torch.full(ids.shape, -most, device="cuda")
    far[:, :5] = most
    plain = torch.full(ids.shape, -float("inf"), device="cuda")
    plain[:, :5] = 0.0
    other = ids.clone()
    other[:, 5:9] = -100
    odd = far.clone()
    odd[:, 5:9] = float("nan")
    odd[:, 9:12] = -float("inf")
    want = moe.distill_forward(x, W, ids, plain, temperature=tau)
    gw = moe.distill_backward(dl, x, W, ids, plain, want["lse"], want["logits"], temperature=tau)
    for i, l in ((ids, far), (other, odd)):
        f = moe.distill_forward(x, W, i, l, temperature=tau)
        assert torch.equal(f["loss"], want["loss"]) and torch.isfinite(f["loss"]).all()
        g = moe.distill_backward(dl, x, W, i, l, f["lse"], f["logits"], temperature=tau)
        # an entry of p = 0 has d q, formed in fp32 twice over: one rounding to bf16 apart at most
        for n in g:
            assert (g[n].float() - gw[n].float()).norm() <= 2.0 ** -8 * gw[n].float().norm()


def test_large_logits_against_64_bits(moe):
    """Logits of 1e4 to 1e5 that differ by a few: the difference is exact in
    fp32, its parts over the temperature are not."""
    x, W, ids, _ = _case()
    tau = 3.0
    g = torch.Generator(device="cuda").manual_seed(2)
    logits = 65536.0 + torch.randint(0, 64, ids.shape, generator=g, device="cuda") / 8
    f = moe.distill_forward(x, W, ids, logits, temperature=tau)
    z = x.double() @ W.double().t() / tau
    p = torch.softmax(logits.double() / tau, 1)
    loss = (p * (p.log() - z.gather(1, ids) + torch.logsumexp(z, 1)[:, None])).sum(1)
    size = float((p.log().abs() + z.gather(1, ids).abs() + torch.logsumexp(z, 1)[:, None].abs()).max())
    assert np.abs((f["loss"].double() - loss).cpu().numpy()).max() <= 2.0 ** -20 * size + 2.0 ** -13 * 2.0 ** -6


def test_both_ends_over_a_large_temperature(moe):
    """The difference of the two ends is past the type's, its part is not:
    probabilities in the ratio exp(2 max / tau)."""
    x, W, ids, dl = _case(K=2)
    tau, most = 1e38, torch.finfo(F32).max
    far = torch.tensor([most, -most], device="cuda").repeat(len(x), 1)
    near = torch.tensor([most / 1e38, -most / 1e38], device="cuda").repeat(len(x), 1)
    f = moe.distill_forward(x, W, ids, far, temperature=tau)
    p = torch.softmax(near.double(), 1)
    # the student is uniform: lse = log V, z / tau = 0
    loss = (p * p.log()).sum(1) + np.log(len(W))
    assert ((f["loss"].double() - loss).abs() <= 2.0 ** -20 * np.log(len(W)) + 2.0 ** -19).all()
