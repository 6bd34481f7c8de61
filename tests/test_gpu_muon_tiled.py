"""The Muon step of matrices with more than 128 rows, whose products are tiled
(smaller ones stay on chip), against its 64-bit definition: momentum, several
stacks and single matrices in one call, tall weights, every type of weights and
gradients.

Tolerances as in test_gpu_newton_schulz.py.  The momentum is off by the two
roundings of its sum.  The step is off by 3e-2 of the rms of the orthogonalised
update (fp16 operands: 4e-3 in the 2-norm, one element at most 8 times that),
without its bf16 rounding, since it moves the weights unrounded; the weights
add their own roundings, 4 of fp32 and with bf16 weights half a step."""
import numpy as np
import pytest
import torch

from _train_ref import muon_step

pytestmark = pytest.mark.gpu

C = (3.4445, -4.7750, 2.0315)
U = 2.0 ** -24


@pytest.fixture(scope="module")
def moe():
    from grouped_gemm_router_gb300 import build
    build.build()
    from grouped_gemm_router_gb300 import moe as m
    return m


def f64(t):
    return t.detach().double().cpu().numpy()


def _tensors(shapes, wtype, gtype, seed):
    rng = torch.Generator(device="cuda").manual_seed(seed)
    r = lambda s: torch.randn(*s, generator=rng, device="cuda")
    w = [(r(s) / 16).to(torch.bfloat16 if wtype == "bf16" else torch.float32) for s in shapes]
    g = [(1e-3 * r(s)).to(gtype) for s in shapes]
    m = [2e-3 * r(s) for s in shapes]
    low = [torch.zeros(s, dtype=torch.bfloat16, device="cuda") for s in shapes] if wtype == "f32 + copy" else None
    return w, g, m, low


def _check(moe, shapes, wtype, gtype, nesterov, seed, sampled):
    w, g, m, low = _tensors(shapes, wtype, gtype, seed)
    if low is not None:
        low[1] = None             # one stack without a copy
    before = [tuple(t.clone() for t in (a, b, c)) for a, b, c in zip(w, g, m)]
    moe.muon_step(w, g, m, lr=0.02, nesterov=nesterov, weight_decay=0.1, weights_bf16=low)
    torch.cuda.synchronize()
    assert moe.device_error() == 0
    for i, s in enumerate(shapes):
        flat = lambda t: t.reshape(-1, *s[-2:])
        n = flat(w[i]).shape[0]
        assert torch.equal(before[i][1], g[i])      # the gradients are read only
        for e in sorted({0, n - 1} if sampled else range(n)):
            w0, g0, m0 = (f64(flat(t)[e:e + 1]) for t in before[i])
            scale = 0.2 * max(s[-2:]) ** 0.5
            w1, m1 = muon_step(w0, g0, m0, 0.02, 0.95, nesterov, 0.1, scale, [C] * 5, 1e-7)
            assert (np.abs(f64(flat(m[i])[e]) - m1[0]) <= 2 * U * (np.abs(m0[0]) + np.abs(g0[0]))).all()
            o = (w0 * (1 - 0.02 * 0.1) - w1) / (0.02 * scale)
            tol = 0.02 * scale * 3e-2 * np.sqrt((o ** 2).mean()) + 4 * U * np.abs(w0)
            if wtype == "bf16":
                tol = tol + 1.01 * 2.0 ** -8 * np.abs(w1)
            assert (np.abs(f64(flat(w[i])[e]) - w1[0]) <= tol[0]).all(), (i, e)
        if low is not None and low[i] is not None:
            assert torch.equal(low[i], w[i].bfloat16())


@pytest.mark.parametrize("gtype", [torch.float32, torch.bfloat16], ids=["g f32", "g bf16"])
@pytest.mark.parametrize("wtype", ["bf16", "f32", "f32 + copy"])
@pytest.mark.parametrize("D,F", [(300, 700), (200, 333), (129, 130), (255, 1001)])
def test_stacks_of_both_orientations(moe, D, F, wtype, gtype):
    _check(moe, [(2, D, F), (3, F, D), (D, F), (F, D)], wtype, gtype, True, D, False)


@pytest.mark.parametrize("gtype", [torch.float32, torch.bfloat16], ids=["g f32", "g bf16"])
@pytest.mark.parametrize("wtype", ["bf16", "f32", "f32 + copy"])
def test_wide_tiles(moe, wtype, gtype):
    # more than two waves of narrow tiles, so 256 columns each; without Nesterov's momentum
    _check(moe, [(8, 768, 1536), (8, 768, 1536), (8, 1536, 768)], wtype, gtype, False, 7, True)


@pytest.mark.parametrize("wtype", ["bf16", "f32", "f32 + copy"])
@pytest.mark.parametrize("D,F", [(96, 200), (77, 131)])
def test_bf16_gradients_on_chip(moe, D, F, wtype):
    _check(moe, [(3, D, F), (3, F, D), (D, F)], wtype, torch.bfloat16, True, D, False)


@pytest.mark.parametrize("wtype", ["bf16", "f32 + copy"])
def test_stacks_across_the_groups(moe, wtype):
    """77 matrices, worked on 26, 26 and 25 at a time, with borders inside the
    stacks: each stack has the bits that it has in a call of its own."""
    shapes = [(20, 768, 1536), (30, 768, 1536), (27, 1536, 768)]
    w, g, m, low = _tensors(shapes, wtype, torch.float32, 3)
    copies = [tuple(t.clone() for t in (a, c)) for a, c in zip(w, m)]
    moe.muon_step(w, g, m, lr=0.02, weight_decay=0.1, weights_bf16=low)
    for i, (w1, m1) in enumerate(copies):
        low1 = None if low is None else [torch.zeros_like(low[i])]
        moe.muon_step([w1], [g[i]], [m1], lr=0.02, weight_decay=0.1, weights_bf16=low1)
        assert torch.equal(w1, w[i]) and torch.equal(m1, m[i])
        assert low is None or torch.equal(low1[0], low[i])
    torch.cuda.synchronize()
    assert moe.device_error() == 0
