"""Newton-Schulz and the Muon step of matrices with one row or one column whose
last CTAs have no columns of the matrix, as views inside larger buffers: the
results are right and what lies around the matrices is neither used nor changed.

One row is a vector of norm s, and every step takes s to a s + b s^3 + c s^5.
Tolerances as for any matrix with a side under 16: the operands' fp16 rounding
at its worst, (3 |b| + 5 c) 2^-11 = 1.2e-2, beside half a bf16 step."""
import numpy as np
import pytest
import torch

from _train_ref import muon_step, newton_schulz

pytestmark = pytest.mark.gpu

C = (3.4445, -4.7750, 2.0315)
U = 2.0 ** -24
PAD = 4096  # elements on either side


@pytest.fixture(scope="module")
def moe():
    from grouped_gemm_router_gb300 import build
    build.build()
    from grouped_gemm_router_gb300 import moe as m
    return m


def f64(t):
    return t.detach().double().cpu().numpy()


def _inside(values):
    """The tensor as a view in the middle of a buffer of NaN."""
    buf = torch.full((PAD + values.numel() + PAD,), float("nan"), dtype=values.dtype, device="cuda")
    view = buf[PAD:PAD + values.numel()].view(values.shape)
    view.copy_(values)
    return buf, view


def _untouched(buf, n):
    assert torch.isnan(buf[:PAD]).all() and torch.isnan(buf[PAD + n:]).all()


# sizes with CTAs that have no columns, and neighbours without
SIZES = [513, 520, 576, 577, 1024, 1025, 1100, 1344, 1345, 1537, 1600, 1792, 1793, 2048]


@pytest.mark.parametrize("tall", [False, True], ids=["row", "column"])
@pytest.mark.parametrize("n", SIZES)
def test_newton_schulz_of_one_row(moe, n, tall):
    for count in (1, 3):
        for dtype in (torch.float32, torch.bfloat16):
            g = torch.randn(count, n, 1, generator=torch.Generator().manual_seed(n + count))
            g = (1e-3 * (g if tall else g.transpose(1, 2).contiguous())).to(dtype)
            buf, view = _inside(g)
            out, o = _inside(torch.zeros(g.shape, dtype=torch.bfloat16))
            moe.newton_schulz(view, out=o)
            torch.cuda.synchronize()
            assert moe.device_error() == 0
            _untouched(buf, g.numel())
            _untouched(out, g.numel())
            for e in range(count):
                ref = newton_schulz(f64(g[e]), [C] * 5, 1e-7)
                err = np.abs(f64(o[e]) - ref)
                assert (err <= (1.01 * 2.0 ** -8 + 1.2e-2) * np.abs(ref)).all()


@pytest.mark.parametrize("wtype", ["bf16", "f32", "f32 + copy"])
@pytest.mark.parametrize("n", [520, 1025, 1100, 1600])
def test_muon_step_of_one_row(moe, n, wtype):
    rng = torch.Generator().manual_seed(n)
    shapes = [(2, 1, n), (1, n, 1)]
    dt = torch.bfloat16 if wtype == "bf16" else torch.float32
    hosts = [((torch.randn(s, generator=rng) / 16).to(dt), 1e-3 * torch.randn(s, generator=rng),
              2e-3 * torch.randn(s, generator=rng)) for s in shapes]
    bufs = [[_inside(t) for t in h] for h in hosts]
    w, g, m = ([b[i][1] for b in bufs] for i in range(3))
    low = [_inside(torch.zeros(s, dtype=torch.bfloat16)) for s in shapes] if wtype == "f32 + copy" else None
    moe.muon_step(w, g, m, lr=0.02, weight_decay=0.1, weights_bf16=None if low is None else [v for _, v in low])
    torch.cuda.synchronize()
    assert moe.device_error() == 0
    for i, s in enumerate(shapes):
        for buf, v in bufs[i]:
            _untouched(buf, v.numel())
        w0, g0, m0 = (f64(t) for t in hosts[i])
        scale = 0.2 * n ** 0.5
        w1, m1 = muon_step(w0, g0, m0, 0.02, 0.95, True, 0.1, scale, [C] * 5, 1e-7)
        assert (np.abs(f64(m[i]) - m1) <= 2 * U * (np.abs(m0) + np.abs(g0))).all()
        o = (w0 * (1 - 0.02 * 0.1) - w1) / (0.02 * scale)
        tol = 0.02 * scale * 1.2e-2 * np.abs(o) + 4 * U * np.abs(w0)
        if wtype == "bf16":
            tol = tol + 1.01 * 2.0 ** -8 * np.abs(w1)
        assert (np.abs(f64(w[i]) - w1) <= tol).all()
        if low is not None:
            _untouched(low[i][0], low[i][1].numel())
            assert torch.equal(low[i][1], w[i].bfloat16())
