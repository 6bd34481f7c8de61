"""Tensors that start anywhere: views into larger buffers, one element past a
16-byte boundary, have the results of aligned copies, bit for bit, and their
neighbours in the buffer stay as they are."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def moe():
    from grouped_gemm_router_gb300 import build
    build.build()
    from grouped_gemm_router_gb300 import moe as m
    return m


def _view(t):
    """t's values in a view that starts one element into a buffer of 7s."""
    buf = torch.full((t.numel() + 2,), 7, dtype=t.dtype, device="cuda")
    v = buf[1:-1].view(t.shape)
    v.copy_(t)
    assert v.data_ptr() % 16 != 0 and v.is_contiguous()
    return buf, v


def _same(a, b):
    return a.keys() == b.keys() and all(torch.equal(a[k], b[k]) for k in a)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("T,D", [(1, 1), (40, 768), (33, 1005), (0, 64)])
def test_layer_norm(moe, T, D, dtype):
    g = torch.Generator(device="cuda").manual_seed(D)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda")
    x, w, b, add, dy, ds = r(T, D).to(dtype), r(D), r(D), r(T, D).bfloat16(), r(T, D).bfloat16(), r(T, D).to(dtype)
    ref = moe.layer_norm_forward(x, w, bias=b, add=add)
    tensors = dict(x=x, weight=w, bias=b, add=add, y=torch.zeros(T, D, dtype=torch.bfloat16, device="cuda"))
    for which in (*tensors, None):           # each alone, then all
        bufs = {n: _view(t) if which in (n, None) and t.numel() else (None, t) for n, t in tensors.items()}
        out = moe.layer_norm_forward(**{n: v for n, (_, v) in bufs.items()})
        assert _same(out, ref) and out["y"] is bufs["y"][1]
        assert all(buf is None or (buf[0] == 7 and buf[-1] == 7) for buf, _ in bufs.values())
    h, mean, rstd = ref["h"], ref["mean"], ref["rstd"]
    gref = moe.layer_norm_backward(dy, h, w, mean, rstd, d_stream=ds)
    tensors = dict(dy=dy, x=h, weight=w, mean=mean, rstd=rstd, d_stream=ds)
    for which in (*tensors, None):
        args = {n: _view(t)[1] if which in (n, None) and t.numel() else t for n, t in tensors.items()}
        assert _same(moe.layer_norm_backward(**args), gref)


def test_newton_schulz(moe):
    g = torch.randn(3, 1001, 363, generator=torch.Generator(device="cuda").manual_seed(1), device="cuda")
    ref = moe.newton_schulz(g[1].clone())
    assert g[1].data_ptr() % 16 != 0
    assert torch.equal(moe.newton_schulz(g[1]), ref)
    buf, out = _view(torch.zeros_like(ref))
    assert moe.newton_schulz(g[1], out=out) is out
    assert torch.equal(out, ref) and buf[0] == 7 and buf[-1] == 7
    ws = torch.empty(moe.newton_schulz_workspace_size(1, 1001, 363) + 16, dtype=torch.uint8, device="cuda")
    with pytest.raises(ValueError, match="256-byte"):
        moe.newton_schulz(g[0], workspace=ws[16:])


def test_muon_step_moves_every_group_once(moe):
    """The second group's tensors start anywhere; a step that refused them
    after the first group had moved would move that one twice when repeated."""
    gen = torch.Generator(device="cuda").manual_seed(2)
    r = lambda s: torch.randn(*s, generator=gen, device="cuda")
    shapes = [(2, 128, 256), (2, 131, 77), (77, 131), (40, 300)]
    for which in ("weights", "grads", "momenta", "weights_bf16", None):
        t = dict(weights=[r(s) / 16 for s in shapes], grads=[1e-3 * r(s) for s in shapes],
                 momenta=[2e-3 * r(s) for s in shapes], weights_bf16=[r(s).bfloat16() for s in shapes])
        views = {n: [_view(v) if i > 0 and which in (n, None) else (None, v.clone()) for i, v in enumerate(l)]
                 for n, l in t.items()}
        moe.muon_step(lr=0.02, weight_decay=0.1, **t)
        moe.muon_step(lr=0.02, weight_decay=0.1, **{n: [v for _, v in l] for n, l in views.items()})
        for n, l in views.items():
            for (buf, v), ref in zip(l, t[n]):
                assert torch.equal(v, ref), (which, n)
                assert buf is None or (buf[0] == 7 and buf[-1] == 7)


def test_refusals_change_nothing(moe):
    """What is refused is refused before the first group moves."""
    gen = torch.Generator(device="cuda").manual_seed(3)
    r = lambda *s: torch.randn(*s, generator=gen, device="cuda")
    w, g, m = ([r(2, 128, 256), r(2, 64, 64)] for _ in range(3))
    kept = [[t.clone() for t in l] for l in (w, m)]
    ws = torch.empty(1 << 20, dtype=torch.uint8, device="cuda")
    wide = torch.zeros(1, 8193, device="cuda")
    for kw in (dict(workspace=ws[16:]), dict(workspace=ws[:256]), dict(lr=float("nan")), dict(steps=0), dict(steps=17),
               dict(grads=[g[0], g[1][:1]]), dict(momenta=[m[0], m[1].bfloat16()]), dict(grads=[g[0], g[1].transpose(1, 2)]),
               dict(weights=[w[0], wide], grads=[g[0], wide], momenta=[m[0], wide.clone()])):
        args = dict(weights=w, grads=g, momenta=m, lr=0.02)
        args.update(kw)
        with pytest.raises((ValueError, RuntimeError)):
            moe.muon_step(**args)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for l, k in zip((w, m), kept) for a, b in zip(l, k))
