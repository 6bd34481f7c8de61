"""Refusals of the Newton-Schulz and Muon entry points (no launch, no GPU),
and their 64-bit statement on the CPU."""
import ctypes

import numpy as np
import pytest

from _train_ref import muon_step, newton_schulz

FAKE = 0x100000
C = (3.4445, -4.7750, 2.0315)


@pytest.fixture(scope="module")
def N():
    from grouped_gemm_router_gb300 import build
    build.build()
    from grouped_gemm_router_gb300 import _native
    return _native


def _coeff(steps=5, bad=None):
    v = list(C) * steps
    if bad is not None:
        v[4] = bad
    return (ctypes.c_float * len(v))(*v)


def _ns(N, g=FAKE, kind=1, count=2, rows=64, cols=128, steps=5, c=None, eps=1e-7, out=FAKE, ws=FAKE, nbytes=1 << 30,
        null_c=False):
    c = None if null_c else (c or _coeff(max(steps, 1)))
    return N.lib.moe_newton_schulz(g, kind, count, rows, cols, steps, c, eps, out, ws, nbytes, None)


@pytest.mark.parametrize("bad", [dict(g=None), dict(out=None), dict(ws=None), dict(null_c=True), dict(kind=3),
                                 dict(count=-1), dict(rows=0), dict(cols=-4), dict(steps=0), dict(eps=-1.0),
                                 dict(eps=float("nan")), dict(g=FAKE + 4), dict(out=FAKE + 8), dict(ws=FAKE + 16),
                                 dict(c=_coeff(5, float("inf")))],
                         ids=lambda d: "_".join(d))
def test_newton_schulz_refusals(N, bad):
    assert _ns(N, **bad) == N.MOE_ERR_INVALID_ARG
    assert N.lib.moe_launch_count() == 0


def test_newton_schulz_limits(N):
    assert _ns(N, rows=8193) == N.MOE_ERR_UNSUPPORTED_SHAPE
    assert _ns(N, cols=8193) == N.MOE_ERR_UNSUPPORTED_SHAPE
    assert _ns(N, count=4097) == N.MOE_ERR_UNSUPPORTED_SHAPE
    assert _ns(N, steps=17) == N.MOE_ERR_UNSUPPORTED_SHAPE
    assert _ns(N, count=0) == N.MOE_OK
    size = N.lib.moe_newton_schulz_workspace_size
    assert size(2, 64, 128) == size(2, 128, 64) > 0
    assert size(0, 64, 64) == 0 and size(1, 0, 4) == 0 and size(1, 8193, 4) == 0
    assert _ns(N, nbytes=size(2, 64, 128) - 1) == N.MOE_ERR_WORKSPACE
    assert N.lib.moe_launch_count() == 0


def _muon(N, stacks=None, n=None, gt=1, wt=0, ws=FAKE, nbytes=1 << 30, params=None, **over):
    stacks = [N.MoeMatrixStack(FAKE, FAKE, FAKE, None, 2, 64, 128)] if stacks is None else stacks
    c = over.pop("c", _coeff())
    p = dict(lr=0.02, momentum=0.95, weight_decay=0.0, scale=1.0, eps=1e-7, nesterov=1, steps=5,
             coefficients=ctypes.addressof(c))
    p.update(over)
    q = N.MoeMuonParams(*(p[k] for k, _ in N.MoeMuonParams._fields_))
    arr = (N.MoeMatrixStack * max(len(stacks), 1))(*stacks)
    return N.lib.moe_muon_step(arr, len(stacks) if n is None else n, gt, wt, ctypes.byref(q), ws, nbytes, None)


def test_muon_refusals(N):
    S = lambda w=FAKE, g=FAKE, m=FAKE, b=None, count=2, rows=64, cols=128: N.MoeMatrixStack(w, g, m, b, count, rows, cols)
    bad = N.MOE_ERR_INVALID_ARG
    assert _muon(N, [S(w=None)]) == bad and _muon(N, [S(g=None)]) == bad and _muon(N, [S(m=None)]) == bad
    assert _muon(N, [S(w=FAKE + 2)]) == bad and _muon(N, [S(m=FAKE + 4)]) == bad
    assert _muon(N, [S(b=FAKE)]) == bad                                  # a copy of bf16 weights
    assert _muon(N, [S(), S(rows=64, cols=64)]) == bad                   # two shapes in one call
    assert _muon(N, [S(count=-1)]) == bad and _muon(N, [S(rows=0)]) == bad
    assert _muon(N, n=-1) == bad and _muon(N, gt=2) == bad and _muon(N, wt=2) == bad
    assert _muon(N, ws=None) == bad and _muon(N, ws=FAKE + 128) == bad
    for k in ("lr", "momentum", "weight_decay", "scale", "eps"):
        assert _muon(N, **{k: float("nan")}) == bad
    assert _muon(N, nesterov=2) == bad and _muon(N, steps=0) == bad and _muon(N, coefficients=None) == bad
    assert _muon(N, steps=17) == N.MOE_ERR_UNSUPPORTED_SHAPE
    assert _muon(N, [S(rows=9000)]) == N.MOE_ERR_UNSUPPORTED_SHAPE
    assert _muon(N, [S()] * 17) == N.MOE_ERR_UNSUPPORTED_SHAPE
    assert _muon(N, [S(count=4000), S(count=4000)]) == N.MOE_ERR_UNSUPPORTED_SHAPE
    need = N.lib.moe_newton_schulz_workspace_size(4, 64, 128)
    assert _muon(N, [S(), S(rows=128, cols=64)], nbytes=need - 1) == N.MOE_ERR_WORKSPACE
    assert _muon(N, []) == N.MOE_OK and _muon(N, [S(count=0)]) == N.MOE_OK
    assert N.lib.moe_launch_count() == 0


def test_binding_refusals(N):
    import torch
    from grouped_gemm_router_gb300 import moe
    g = torch.zeros(4, 8)
    with pytest.raises(ValueError, match="CUDA"):
        moe.newton_schulz(g)
    with pytest.raises(ValueError, match="bfloat16 or torch.float32"):
        moe.newton_schulz(g.half())
    with pytest.raises(ValueError, match="expected"):
        moe.newton_schulz(g[0])
    with pytest.raises(ValueError, match="same length"):
        moe.muon_step([g], [], [g], 0.1)
    with pytest.raises(ValueError, match="bfloat16 or torch.float32"):
        moe.muon_step([g.double()], [g], [g], 0.1)
    with pytest.raises(ValueError, match="coefficients"):
        moe._ns_coefficients([C] * 4, 5)
    assert list(moe._ns_coefficients(C, 2)) == list(moe._ns_coefficients([C, C], 2))
    assert moe.muon_step([], [], [], 0.1) is None


def test_the_definition_orthogonalises():
    """Singular vectors stay, singular values follow the scalar iteration."""
    rng = np.random.default_rng(0)
    for shape in ((6, 9), (9, 6), (5, 5)):
        g = rng.standard_normal(shape)
        u, s, vt = np.linalg.svd(g, full_matrices=False)
        t = s / np.sqrt((s ** 2).sum())
        for a, b, c in [C] * 5:
            t = a * t + b * t ** 3 + c * t ** 5
        assert np.abs(newton_schulz(g, [C] * 5, 0.0) - (u * t) @ vt).max() < 1e-12
    w, g, m = (rng.standard_normal((2, 4, 6)) for _ in range(3))
    w1, m1 = muon_step(w, g, m, 0.0, 0.9, True, 0.5, 1.0, [C] * 5, 1e-7)
    assert np.array_equal(w1, w) and np.allclose(m1, 0.9 * m + g)
