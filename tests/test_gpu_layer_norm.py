"""Layer norm on the GPU against its 64-bit definition.

Tolerances, with u = 2^-24 (half a step of fp32): a row's sums add at most 32
values one after the other in a thread and 9 levels across threads, so a mean
is off by at most 42 u mean|.|, taken as 64 u; the results then carry a few
more roundings of their own terms.  A bf16 result adds half a step, 2^-8 of
its value.  The weight gradients add at most ceil(T / rows in flight) + 8 + 64
+ 8 terms in a chain: with the T here, under 256, so 256 u sum|terms|."""
import numpy as np
import pytest
import torch

from _train_ref import layer_norm, layer_norm_grad

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


def _inputs(T, D, dtype, seed, offset=0.3, spread=1.0):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g)
    x = (spread * r(T, D) * torch.exp(0.5 * r(D)) + offset * r(D)).to(dtype).cuda()
    return dict(x=x, w=(1 + 0.3 * r(D)).cuda(), b=(0.2 * r(D)).cuda(), add=r(T, D).bfloat16().cuda(),
                dy=r(T, D).bfloat16().cuda(), ds=r(T, D).to(dtype).cuda())


SIZES = [(1, 1), (1, 64), (3, 7), (5, 8), (9, 33), (257, 128), (64, 264), (33, 520), (40, 776), (1001, 1005),
         (12, 1032), (7, 2047), (30, 2048), (5, 4100), (6, 4096), (3, 8191), (4, 8192), (5000, 768)]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("T,D", SIZES)
def test_forward(moe, T, D, dtype):
    i = _inputs(T, D, dtype, T * 10007 + D)
    for add in (None, i["add"]):
        for bias in (None, i["b"]):
            eps = 1e-5
            out = moe.layer_norm_forward(i["x"], i["w"], bias=bias, eps=eps, add=add)
            torch.cuda.synchronize()
            h = i["x"]
            if add is not None:
                h = (i["x"].float() + add.float()).to(dtype)
                assert torch.equal(out["h"], h)          # one rounding: the same bits
            assert ("h" in out) == (add is not None)
            hx, w, b = f64(h), f64(i["w"]), None if bias is None else f64(bias)
            y, mu, r = layer_norm(hx, w, b, eps)
            size = np.abs(hx).mean(axis=1)
            assert (np.abs(f64(out["mean"]) - mu) <= 64 * U * size).all()
            # the variance moves by the mean's error and by its own sum's
            assert (np.abs(f64(out["rstd"]) - r) <= r * (64 * U + 2 * (64 * U * size * r) ** 2)).all()
            tol = 2.0 ** -8 * np.abs(y) + 64 * U * (np.abs(w) * (np.abs(hx - mu[:, None]) + size[:, None]) * r[:, None]
                                                 + (0 if b is None else np.abs(b)))
            # 1.01: the half step counts from the value before its rounding
            assert (np.abs(f64(out["y"]) - y) <= 1.01 * tol).all()


def test_forward_far_offset_and_equal_rows(moe):
    # a mean 1000 times the spread: the two-pass variance keeps it
    i = _inputs(50, 768, torch.float32, 5)
    x = i["x"] * 0.5 + 1000.0
    out = moe.layer_norm_forward(x, i["w"])
    y, mu, r = layer_norm(f64(x), f64(i["w"]), None, 1e-5)
    # the mean of x is off by at most 64 u 1000 = 3.8e-3 of a spread of 0.5 before it is squared
    assert (np.abs(f64(out["rstd"]) / r - 1) <= 64 * U + (64 * U * 1000 * r) ** 2).all()
    assert (np.abs(f64(out["y"]) - y) <= 2.0 ** -8 * 1.01 * np.abs(y) + 70 * U * 1000 * r[:, None] * np.abs(f64(i["w"])) + 1e-6).all()
    # equal values: no variance, y = bias
    x = torch.full((3, 100), 2.5, device="cuda")
    w, b = torch.full((100,), 3.0, device="cuda"), torch.arange(100.0, device="cuda")
    out = moe.layer_norm_forward(x, w, bias=b, eps=1e-5)
    assert torch.equal(out["y"], b.bfloat16().expand(3, 100))
    assert torch.allclose(out["rstd"], torch.full((3,), 1e-5 ** -0.5, device="cuda"), rtol=1e-6)


def test_forward_bad_values_stay_in_their_row(moe):
    i = _inputs(40, 768, torch.float32, 6)
    ref = moe.layer_norm_forward(i["x"], i["w"], bias=i["b"])["y"]
    x = i["x"].clone()
    x[7, 3], x[20, 700] = float("nan"), float("inf")
    y = moe.layer_norm_forward(x, i["w"], bias=i["b"])["y"]
    keep = [t for t in range(40) if t not in (7, 20)]
    assert torch.equal(y[keep], ref[keep])
    assert torch.isnan(y[7]).all() and torch.isnan(y[20]).all()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("T,D", SIZES)
def test_backward(moe, T, D, dtype):
    i = _inputs(T, D, dtype, T * 20011 + D)
    f = moe.layer_norm_forward(i["x"], i["w"], bias=i["b"])
    for ds in (None, i["ds"]):
        for bias in (False, True):
            g = moe.layer_norm_backward(i["dy"], i["x"], i["w"], f["mean"], f["rstd"], bias=bias, d_stream=ds)
            torch.cuda.synchronize()
            assert g["dx"].dtype == dtype and ("dbias" in g) == bias
            dy, x, w, mu, r = (f64(v) for v in (i["dy"], i["x"], i["w"], f["mean"], f["rstd"]))
            s = None if ds is None else f64(ds)
            dx, dw, db = layer_norm_grad(dy, x, w, mu, r, s)
            n, p = (x - mu[:, None]) * r[:, None], dy * w
            terms = r[:, None] * (np.abs(p) + np.abs(p).mean(1, keepdims=True)
                                  + np.abs(n) * np.abs(p * n).mean(1, keepdims=True)) + (0 if s is None else np.abs(s))
            # n = (x - mu) r carries the rounding of the difference, 2 u |n|
            assert (np.abs(f64(g["dx"]) - dx) <= 1.01 * HALF[dtype] * np.abs(dx) + 70 * U * terms).all()
            assert (np.abs(f64(g["dweight"]) - dw) <= 256 * U * np.abs(dy * n).sum(0)).all()
            if bias:
                assert (np.abs(f64(g["dbias"]) - db) <= 256 * U * np.abs(dy).sum(0)).all()


def test_backward_is_repeatable_and_takes_no_rows(moe):
    i = _inputs(20000, 768, torch.bfloat16, 9)
    f = moe.layer_norm_forward(i["x"], i["w"])
    a = moe.layer_norm_backward(i["dy"], i["x"], i["w"], f["mean"], f["rstd"], d_stream=i["ds"])
    for _ in range(3):
        b = moe.layer_norm_backward(i["dy"], i["x"], i["w"], f["mean"], f["rstd"], d_stream=i["ds"])
        assert all(torch.equal(a[k], b[k]) for k in a)
    e = i["x"][:0]
    f = moe.layer_norm_forward(e, i["w"])
    assert f["y"].shape == (0, 768) and f["mean"].shape == (0,)
    g = moe.layer_norm_backward(i["dy"][:0], e, i["w"], f["mean"], f["rstd"])
    assert g["dx"].shape == (0, 768) and not g["dweight"].any() and not g["dbias"].any()


def test_rows_beyond_32_bit_offsets(moe):
    """2^31 and more elements: the last rows have the first rows' bits."""
    T, D = 270000, 8192
    x = torch.zeros(T, D, dtype=torch.bfloat16, device="cuda")
    i = _inputs(8, D, torch.bfloat16, 11)
    x[:8] = i["x"]
    x[-8:] = i["x"]
    out = moe.layer_norm_forward(x, i["w"], bias=i["b"])
    assert torch.equal(out["y"][:8], out["y"][-8:]) and torch.equal(out["mean"][:8], out["mean"][-8:])
    dy = torch.zeros_like(x)
    dy[:8] = i["dy"]
    dy[-8:] = i["dy"]
    g = moe.layer_norm_backward(dy, x, i["w"], out["mean"], out["rstd"])
    assert torch.equal(g["dx"][:8], g["dx"][-8:])
    r = moe.layer_norm_backward(i["dy"], i["x"], i["w"], out["mean"][:8].contiguous(), out["rstd"][:8].contiguous())
    assert torch.equal(g["dx"][:8], r["dx"])


def test_on_a_side_stream_and_in_a_graph(moe):
    i = _inputs(300, 768, torch.bfloat16, 12)
    ref = moe.layer_norm_forward(i["x"], i["w"], add=i["add"])
    gref = moe.layer_norm_backward(i["dy"], ref["h"], i["w"], ref["mean"], ref["rstd"])
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        out = moe.layer_norm_forward(i["x"], i["w"], add=i["add"])
    torch.cuda.current_stream().wait_stream(s)
    assert all(torch.equal(ref[k], out[k]) for k in ref)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = moe.layer_norm_forward(i["x"], i["w"], add=i["add"])
        g = moe.layer_norm_backward(i["dy"], out["h"], i["w"], out["mean"], out["rstd"])
    for v in (*out.values(), *g.values()):
        v.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(ref[k], out[k]) for k in ref) and all(torch.equal(gref[k], g[k]) for k in gref)
