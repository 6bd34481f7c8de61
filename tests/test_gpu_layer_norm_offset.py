"""Layer norm backward of rows whose mean is far from zero, against the 64-bit
definition with the mean and rstd that the kernel is given.

n = (x - mean) rstd is off by one rounding of the difference and one of the
product, 2 u of n itself, u = 2^-24, wherever the rows lie: the mean's size
does not enter.  With T <= 64 a thread adds at most one row, a block eight, and
the blocks' rows 16 and 5 levels: under 32 roundings, so 34 u sum|terms| for
the weight gradients.  dx: as in test_gpu_layer_norm.py, half a step of its
type and 70 u of its terms."""
import numpy as np
import pytest
import torch

from _train_ref import layer_norm_grad

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: U}


@pytest.fixture(scope="module")
def moe():
    from grouped_gemm_router_gb300 import build
    build.build()
    from grouped_gemm_router_gb300 import moe as m
    return m


def f64(t):
    return t.detach().double().cpu().numpy()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("mean", [0.0, 20.0, 1000.0, 30000.0])
@pytest.mark.parametrize("T,D", [(64, 64), (40, 768), (40, 1004), (40, 1008), (33, 2048), (17, 4096), (9, 8192), (9, 8190)])
def test_backward_far_from_zero(moe, T, D, mean, dtype):
    g = torch.Generator().manual_seed(T * 31 + D)
    r = lambda *s: torch.randn(*s, generator=g)
    # bf16 has 8 bits: there the spread follows the mean, or the rows would be constant
    spread = 0.5 if dtype == torch.float32 else 0.5 * max(1.0, mean / 64)
    x = (mean + spread * r(T, D)).to(dtype).cuda()
    w, dy, ds = (1 + 0.3 * r(D)).cuda(), r(T, D).bfloat16().cuda(), r(T, D).to(dtype).cuda()
    f = moe.layer_norm_forward(x, w)
    for stream in (None, ds):
        out = moe.layer_norm_backward(dy, x, w, f["mean"], f["rstd"], d_stream=stream)
        torch.cuda.synchronize()
        a = [f64(v) for v in (dy, x, w, f["mean"], f["rstd"])]
        s = None if stream is None else f64(stream)
        dx, dw, db = layer_norm_grad(*a, s)
        n, p = (a[1] - a[3][:, None]) * a[4][:, None], a[0] * a[2]
        assert (np.abs(f64(out["dweight"]) - dw) <= 34 * U * np.abs(a[0] * n).sum(0)).all()
        assert (np.abs(f64(out["dbias"]) - db) <= 34 * U * np.abs(a[0]).sum(0)).all()
        terms = a[4][:, None] * (np.abs(p) + np.abs(p).mean(1, keepdims=True)
                                 + np.abs(n) * np.abs(p * n).mean(1, keepdims=True)) + (0 if s is None else np.abs(s))
        assert (np.abs(f64(out["dx"]) - dx) <= 1.01 * HALF[dtype] * np.abs(dx) + 70 * U * terms).all()
