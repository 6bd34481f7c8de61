"""Layer norm's refusals (no launch, no GPU) and its formulas on the CPU."""
import ctypes

import numpy as np
import pytest

from _train_ref import layer_norm, layer_norm_grad

FAKE = 0x100000  # a 16-byte aligned address that is never dereferenced


@pytest.fixture(scope="module")
def N():
    from grouped_gemm_router_gb300 import build
    build.build()
    from grouped_gemm_router_gb300 import _native
    return _native


def _fwd(N, x=FAKE, kind=0, add=None, w=FAKE, b=None, eps=1e-5, T=4, D=64, y=FAKE, h=None, mean=FAKE, rstd=FAKE):
    return N.lib.moe_layer_norm_forward(x, kind, add, w, b, eps, T, D, y, h, mean, rstd, None)


def _bwd(N, dy=FAKE, x=FAKE, kind=0, w=FAKE, mean=FAKE, rstd=FAKE, ds=None, T=4, D=64, dx=FAKE, dw=FAKE, db=None,
         scratch=FAKE, nbytes=1 << 30):
    return N.lib.moe_layer_norm_backward(dy, x, kind, w, mean, rstd, ds, T, D, dx, dw, db, scratch, nbytes, None)


@pytest.mark.parametrize("bad", [dict(x=None), dict(w=None), dict(y=None), dict(mean=None), dict(rstd=None),
                                 dict(kind=2), dict(eps=-1.0), dict(eps=float("nan")), dict(eps=float("inf")),
                                 dict(add=FAKE), dict(h=FAKE), dict(T=-1), dict(D=0), dict(D=-8),
                                 dict(x=FAKE + 8), dict(b=FAKE + 4), dict(mean=FAKE + 4)],
                         ids=lambda d: "_".join(f"{k}={v}" for k, v in d.items()))
def test_forward_refusals(N, bad):
    assert _fwd(N, **bad) == N.MOE_ERR_INVALID_ARG
    assert N.lib.moe_launch_count() == 0


@pytest.mark.parametrize("bad", [dict(dy=None), dict(x=None), dict(w=None), dict(mean=None), dict(rstd=None),
                                 dict(dx=None), dict(dw=None), dict(scratch=None), dict(kind=-1), dict(T=-1),
                                 dict(D=0), dict(ds=FAKE + 2), dict(db=FAKE + 4), dict(scratch=FAKE + 8)],
                         ids=lambda d: "_".join(f"{k}={v}" for k, v in d.items()))
def test_backward_refusals(N, bad):
    assert _bwd(N, **bad) == N.MOE_ERR_INVALID_ARG
    assert N.lib.moe_launch_count() == 0


def test_shape_limits_and_scratch(N):
    assert _fwd(N, D=8193) == N.MOE_ERR_UNSUPPORTED_SHAPE
    assert _fwd(N, T=(1 << 24) + 1) == N.MOE_ERR_UNSUPPORTED_SHAPE
    assert _bwd(N, D=8193) == N.MOE_ERR_UNSUPPORTED_SHAPE
    assert _fwd(N, T=0) == N.MOE_OK                      # nothing to do
    size = N.lib.moe_layer_norm_backward_scratch_size
    assert size(4, 64) == 4 * 2 * 64 * 4
    assert size(1 << 20, 768) == 512 * 2 * 768 * 4       # the most partial rows
    assert size(4, 0) == 0 and size(-1, 64) == 0
    assert _bwd(N, nbytes=size(4, 64) - 1) == N.MOE_ERR_WORKSPACE
    assert N.lib.moe_launch_count() == 0


def test_binding_refuses_wrong_tensors(N):
    import torch
    from grouped_gemm_router_gb300 import moe
    x = torch.zeros(4, 64)
    w = torch.ones(64)
    with pytest.raises(ValueError, match="CUDA"):
        moe.layer_norm_forward(x, w)
    with pytest.raises(ValueError, match="bfloat16 or torch.float32"):
        moe.layer_norm_forward(x.half(), w)
    with pytest.raises(ValueError, match=r"\[T, D\]"):
        moe.layer_norm_forward(x[0], w)
    with pytest.raises(ValueError, match="CUDA"):
        moe.layer_norm_backward(x.bfloat16(), x, w, x[:, 0], x[:, 0])


def test_gradient_formula_against_differences():
    """The formula the kernels compute, against central differences of the
    forward in 64 bits: step 1e-5 leaves an error of about 1e-9."""
    rng = np.random.default_rng(0)
    x, dy, ds = (rng.standard_normal((3, 7)) for _ in range(3))
    w, b = 1 + 0.3 * rng.standard_normal(7), rng.standard_normal(7)

    def loss(x_, w_, b_):
        return (layer_norm(x_, w_, b_, 1e-3)[0] * dy).sum() + (x_ * ds).sum()

    _, mu, r = layer_norm(x, w, b, 1e-3)
    dx, dw, db = layer_norm_grad(dy, x, w, mu, r, ds)
    for got, which in ((dx, 0), (dw, 1), (db, 2)):
        for i in np.ndindex(got.shape):
            args = [x.copy(), w.copy(), b.copy()]
            args[which][i] += 1e-5
            hi = loss(*args)
            args[which][i] -= 2e-5
            assert abs((hi - loss(*args)) / 2e-5 - got[i]) < 1e-7
