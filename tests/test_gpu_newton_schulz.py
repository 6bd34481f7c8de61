"""Newton-Schulz and the Muon step on the GPU against their 64-bit definition.

Tolerances.  The operands of the products are rounded to fp16, half a step of
2^-11 = 4.9e-4 at most, 2e-4 rms.  The last steps see X (three times), A
(three times) and B (once) with factors up to |b| s^3 + 2 |c| s^5 of about 8,
so the result is off by about 8 * 2e-4 = 1.6e-3 of its size, beside its own
bf16 rounding (2^-8 at most, 1.7e-3 rms): 4e-3 in the 2-norm, and for one
element 2^-8 of its value plus 3e-2 of the rms (over 8 times the 3.6e-3 that
the 2-norm leaves).  Matrices with a side under 16 average over too few
roundings: there the worst case counts, (3 |b| + 5 c) 2^-11 = 1.2e-2."""
import numpy as np
import pytest
import torch

from _train_ref import muon_step, newton_schulz

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


def _grad(B, rows, cols, kind, seed, dtype=torch.float32):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g)
    if kind == "full":
        x = r(B, rows, cols)
    elif kind == "few tokens":      # rank a quarter of the short side
        t = max(1, min(rows, cols) // 4)
        x = r(B, rows, t) @ r(B, t, cols)
    elif kind == "one strong":      # a few directions far above the rest
        x = 0.05 * r(B, rows, cols) + r(B, rows, 2) @ r(B, 2, cols)
    else:                           # features that never fire
        x = r(B, rows, cols)
        x[:, ::3] = 0
        x[:, :, 1::5] = 0
    return (1e-3 * x).to(dtype).cuda()


def _check(got, ref, what):
    m = min(ref.shape)
    rms = np.sqrt((ref ** 2).mean())
    err = np.abs(got - ref)
    two = np.sqrt((err ** 2).sum()) / np.sqrt((ref ** 2).sum())
    assert two <= (4e-3 if m >= 16 else 1.2e-2), (what, two)
    assert (err <= 2.0 ** -8 * 1.01 * np.abs(ref) + 3e-2 * rms).all(), (what, (err / rms).max())


SIZES = [(1, 1, 1), (2, 1, 300), (3, 5, 7), (2, 17, 40), (1, 64, 64), (4, 128, 256), (2, 129, 255), (2, 300, 300),
         (3, 1001, 363), (2, 200, 65), (1, 768, 1536), (2, 1536, 768), (1, 513, 2000), (1, 20, 8192), (70, 48, 96),
         (3, 128, 257), (2, 100, 513), (2, 600, 96), (2, 128, 1024), (1, 2048, 128), (2, 33, 2001), (2, 128, 2049), (200, 64, 64)]


@pytest.mark.parametrize("kind", ["full", "few tokens", "one strong", "dead features"])
@pytest.mark.parametrize("B,rows,cols", SIZES)
def test_newton_schulz(moe, B, rows, cols, kind):
    for dtype in (torch.float32, torch.bfloat16):
        g = _grad(B, rows, cols, kind, rows * 31 + cols, dtype)
        o = moe.newton_schulz(g)
        torch.cuda.synchronize()
        assert moe.device_error() == 0
        assert o.shape == g.shape and o.dtype == torch.bfloat16
        for e in sorted({0, B // 2, B - 1}):
            if f64(g[e]).any():
                _check(f64(o[e]), newton_schulz(f64(g[e]), [C] * 5, 1e-7), (kind, dtype, e))


@pytest.mark.parametrize("steps", [1, 2, 3, 8])
def test_steps_and_their_coefficients(moe, steps):
    cs = [C, (2.0, -1.5, 0.5), (1.875, -1.25, 0.375)]
    cs = [cs[i % 3] for i in range(steps)]
    g = _grad(2, 200, 333, "full", 3)
    o = moe.newton_schulz(g, steps=steps, coefficients=cs)
    c1 = moe.newton_schulz(g[0], steps=steps, coefficients=cs)     # a single matrix has the stack's bits
    assert torch.equal(o[0], c1)
    for e in range(2):
        _check(f64(o[e]), newton_schulz(f64(g[e]), cs, 1e-7), steps)


def test_zero_tiny_huge_and_bad_matrices(moe):
    g = _grad(6, 100, 130, "full", 4)
    ref = moe.newton_schulz(g)
    b = g.clone()
    b[1] = 0
    b[2] *= 1e-12           # far below eps: X = G / eps
    b[3] *= 1e12
    b[4, 3, 5] = float("nan")
    b[5, 99, 129] = float("-inf")
    o = moe.newton_schulz(b)
    assert torch.equal(o[0], ref[0])
    assert not o[1].any()
    small = newton_schulz(f64(b[2]), [C] * 5, 1e-7)
    assert np.abs(f64(o[2]) - small).max() <= 1e-2 * np.abs(small).max()
    _check(f64(o[3]), newton_schulz(f64(b[3]), [C] * 5, 1e-7), "huge")
    assert torch.isnan(o[4]).all() and torch.isnan(o[5]).all()


def test_transposed_input_gives_the_transposed_result(moe):
    g = _grad(2, 300, 700, "full", 6)
    a = moe.newton_schulz(g)
    b = moe.newton_schulz(g.transpose(1, 2).contiguous())
    # the norm adds its squares in another order; all else is the same
    d = (a.float() - b.transpose(1, 2).float()).abs().max()
    assert d <= 2.0 ** -7 * a.float().abs().max()


def test_repeatable_streams_graph_and_empty(moe):
    g = _grad(3, 256, 520, "full", 7)
    ref = moe.newton_schulz(g)
    for _ in range(3):
        assert torch.equal(ref, moe.newton_schulz(g))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        o = moe.newton_schulz(g)
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(ref, o)
    ws = torch.empty(moe.newton_schulz_workspace_size(3, 256, 520), dtype=torch.uint8, device="cuda")
    out = torch.empty_like(ref)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        moe.newton_schulz(g, out=out, workspace=ws)
    ws.fill_(255)             # what the workspace holds does not matter
    out.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(ref, out)
    assert moe.newton_schulz(g[:0]).shape == (0, 256, 520)


@pytest.mark.parametrize("nesterov", [True, False])
@pytest.mark.parametrize("wtype", ["bf16", "f32", "f32 + copy"])
@pytest.mark.parametrize("D,F", [(128, 256), (96, 200), (77, 131)])
def test_muon_step(moe, D, F, wtype, nesterov):
    E = 3
    shapes = [(E, D, F), (E, F, D), (D, F), (E, 40, 33)]      # two groups, a stack and single matrices
    rng = torch.Generator().manual_seed(D)
    r = lambda s: torch.randn(*s, generator=rng)
    dt = torch.bfloat16 if wtype == "bf16" else torch.float32
    w = [(r(s) / 16).to(dt).cuda() for s in shapes]
    g = [(1e-3 * r(s)).cuda() for s in shapes]
    m = [(2e-3 * r(s)).cuda() for s in shapes]
    low = None
    if wtype == "f32 + copy":
        low = [torch.empty(s, dtype=torch.bfloat16, device="cuda") if i != 1 else None for i, s in enumerate(shapes)]
    before = [(f64(a), f64(b), f64(c)) for a, b, c in zip(w, g, m)]
    moe.muon_step(w, g, m, lr=0.02, nesterov=nesterov, weight_decay=0.1, weights_bf16=low)
    torch.cuda.synchronize()
    assert moe.device_error() == 0
    for i, s in enumerate(shapes):
        w0, g0, m0 = (v.reshape(-1, *s[-2:]) for v in before[i])
        scale = 0.2 * max(s[-2:]) ** 0.5
        w1, m1 = muon_step(w0, g0, m0, 0.02, 0.95, nesterov, 0.1, scale, [C] * 5, 1e-7)
        gm = f64(m[i]).reshape(m1.shape)
        assert (np.abs(gm - m1) <= 2 * U * (np.abs(m0) + np.abs(g0))).all()
        o = (w0 * (1 - 0.02 * 0.1) - w1) / (0.02 * scale)
        rms = np.sqrt((o ** 2).mean())
        move = 0.02 * scale * 3e-2 * rms + 4 * U * np.abs(w0)
        if wtype == "bf16":
            move = move + 1.01 * 2.0 ** -8 * np.abs(w1)
        assert (np.abs(f64(w[i]).reshape(w1.shape) - w1) <= move).all()
        if low is not None and low[i] is not None:
            assert torch.equal(low[i], w[i].bfloat16())


def test_muon_step_equals_its_parts_and_leaves_a_bad_expert_alone(moe):
    """A NaN in one expert's gradient stays in that expert's weights."""
    g = _grad(4, 128, 192, "full", 12)
    w = (torch.randn(4, 128, 192, generator=torch.Generator().manual_seed(1)) / 16).cuda()
    m = torch.zeros_like(g)
    w1, m1 = w.clone(), m.clone()
    moe.muon_step([w1], [g], [m1], lr=0.1, momentum=0.5, nesterov=False, scale=1.0)
    assert torch.equal(m1, g)
    o = moe.newton_schulz(g).float()
    # the step takes the unrounded result: half a bf16 step of 0.1 o, and fp32 roundings
    assert ((w1 - (w - 0.1 * o)).abs() <= 0.1 * 1.01 * 2.0 ** -8 * o.abs() + 4 * U * w.abs() + 1e-9).all()
    b = g.clone()
    b[2, 0, 0] = float("nan")
    w2, m2 = w.clone(), m.clone()
    moe.muon_step([w2], [b], [m2], lr=0.1, momentum=0.5, nesterov=False, scale=1.0)
    keep = [0, 1, 3]
    assert torch.equal(w2[keep], w1[keep]) and torch.isnan(w2[2]).all()


def test_many_and_large_matrices(moe):
    """More than 2^31 elements: the last matrix has the bits it has alone."""
    B, rows, cols = 130, 2048, 8192
    one = _grad(1, rows, cols, "full", 13, torch.bfloat16)
    g = torch.zeros(B, rows, cols, dtype=torch.bfloat16, device="cuda")
    g[0] = one[0]
    g[-1] = one[0]
    o = moe.newton_schulz(g)
    torch.cuda.synchronize()
    assert moe.device_error() == 0
    assert torch.equal(o[0], o[-1]) and torch.equal(o[-1], moe.newton_schulz(one)[0])
    assert not o[1:-1].any()


@pytest.mark.parametrize("kind", ["full", "few tokens"])
@pytest.mark.parametrize("B,rows,cols", [(9, 129, 300), (16, 256, 1024), (38, 256, 512), (60, 250, 250), (70, 129, 131),
                                         (5, 700, 513), (4, 768, 1536), (1, 1024, 1024)])
def test_tile_widths(moe, B, rows, cols, kind):
    """One to two waves of narrow tiles, with each way of counting them, and
    the sizes just past them."""
    g = _grad(B, rows, cols, kind, 29)
    o = moe.newton_schulz(g)
    torch.cuda.synchronize()
    assert moe.device_error() == 0
    for e in range(B):
        _check(f64(o[e]), newton_schulz(f64(g[e]), [C] * 5, 1e-7), (kind, e))
