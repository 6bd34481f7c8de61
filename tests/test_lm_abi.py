"""Embedding, cross entropy and distillation: refusals (no launch, no GPU) and
the formulas of their gradients against differences, on the CPU."""
import ctypes

import numpy as np
import pytest

import _lm_ref as ref

FAKE = 0x100000  # a 256-byte aligned address that is never dereferenced
BIG = 1 << 40


@pytest.fixture(scope="module")
def N():
    from grouped_gemm_router_gb300 import build
    build.build()
    from grouped_gemm_router_gb300 import _native
    return _native


def _emb(N, ids=FAKE, it=0, table=FAKE, tt=0, scale=1.0, T=4, V=10, D=64, out=FAKE, ot=0):
    return N.lib.moe_embedding_forward(ids, it, table, tt, scale, T, V, D, out, ot, None)


def _emb_bwd(N, d=FAKE, dt=0, ids=FAKE, it=0, scale=1.0, add=None, T=4, V=10, D=64, out=FAKE, ws=FAKE, n=BIG):
    return N.lib.moe_embedding_backward(d, dt, ids, it, scale, add, T, V, D, out, ws, n, None)


def _ce(N, x=FAKE, W=FAKE, y=FAKE, it=0, T=4, D=64, V=10, loss=FAKE, lse=FAKE, ws=FAKE, n=BIG):
    return N.lib.moe_cross_entropy_forward(x, W, y, it, T, D, V, loss, lse, ws, n, None)


def _ce_bwd(N, dl=FAKE, de=None, x=FAKE, W=FAKE, y=FAKE, it=0, loss=FAKE, lse=FAKE, T=4, D=64, V=10, dx=FAKE, dW=FAKE,
            ws=FAKE, n=BIG):
    return N.lib.moe_cross_entropy_backward(dl, de, x, W, y, it, loss, lse, T, D, V, dx, dW, ws, n, None)


def _teacher(N, ids=FAKE, logits=FAKE, it=0, lt=1, K=8, tau=1.0):
    return N.MoeTeacher(ids, logits, it, lt, K, tau)


def _dis(N, x=FAKE, W=FAKE, T=4, D=64, V=10, loss=FAKE, lse=FAKE, at=FAKE, ws=FAKE, n=BIG, **t):
    return N.lib.moe_distill_forward(x, W, _teacher(N, **t), T, D, V, loss, lse, at, ws, n, None)


def _dis_bwd(N, dl=FAKE, x=FAKE, W=FAKE, lse=FAKE, at=FAKE, T=4, D=64, V=10, dx=FAKE, dW=FAKE, ws=FAKE, n=BIG, **t):
    return N.lib.moe_distill_backward(dl, x, W, _teacher(N, **t), lse, at, T, D, V, dx, dW, ws, n, None)


NAN, INF = float("nan"), float("inf")
CASES = [(_emb, dict(ids=None)), (_emb, dict(table=None)), (_emb, dict(out=None)), (_emb, dict(it=2)), (_emb, dict(tt=2)),
         (_emb, dict(ot=-1)), (_emb, dict(scale=NAN)), (_emb, dict(T=-1)), (_emb, dict(V=0)), (_emb, dict(D=0)),
         (_emb, dict(ids=FAKE + 8)), (_emb, dict(out=FAKE + 2)),
         (_emb_bwd, dict(d=None)), (_emb_bwd, dict(ids=None)), (_emb_bwd, dict(out=None)), (_emb_bwd, dict(ws=None)),
         (_emb_bwd, dict(dt=3)), (_emb_bwd, dict(it=-1)), (_emb_bwd, dict(scale=INF)), (_emb_bwd, dict(add=FAKE + 2)),
         (_emb_bwd, dict(ws=FAKE + 16)), (_emb_bwd, dict(V=-1)), (_emb_bwd, dict(out=FAKE + 4)),
         (_ce, dict(x=None)), (_ce, dict(W=None)), (_ce, dict(y=None)), (_ce, dict(loss=None)), (_ce, dict(lse=None)),
         (_ce, dict(ws=None)), (_ce, dict(it=2)), (_ce, dict(T=-1)), (_ce, dict(V=0)), (_ce, dict(D=-64)),
         (_ce, dict(x=FAKE + 8)), (_ce, dict(ws=FAKE + 128)), (_ce, dict(lse=FAKE + 4)),
         (_ce_bwd, dict(dl=None)), (_ce_bwd, dict(x=None)), (_ce_bwd, dict(W=None)), (_ce_bwd, dict(y=None)),
         (_ce_bwd, dict(loss=None)), (_ce_bwd, dict(lse=None)), (_ce_bwd, dict(dx=None)), (_ce_bwd, dict(dW=None)),
         (_ce_bwd, dict(ws=None)), (_ce_bwd, dict(de=FAKE + 4)), (_ce_bwd, dict(dW=FAKE + 2)), (_ce_bwd, dict(T=0, dW=None)),
         (_dis, dict(ids=None)), (_dis, dict(logits=None)), (_dis, dict(K=0)), (_dis, dict(K=-1)), (_dis, dict(tau=0.0)),
         (_dis, dict(tau=-1.0)), (_dis, dict(tau=NAN)), (_dis, dict(tau=INF)), (_dis, dict(tau=1e-40)), (_dis, dict(it=2)),
         (_dis, dict(lt=2)), (_dis, dict(ids=FAKE + 4)), (_dis, dict(at=None)), (_dis, dict(x=None)),
         (_dis_bwd, dict(dl=None)), (_dis_bwd, dict(lse=None)), (_dis_bwd, dict(at=None)), (_dis_bwd, dict(dx=None)),
         (_dis_bwd, dict(dW=None)), (_dis_bwd, dict(K=0)), (_dis_bwd, dict(logits=FAKE + 8)), (_dis_bwd, dict(ws=None))]


@pytest.mark.parametrize("call,bad", CASES, ids=[c.__name__ + "_" + "_".join(f"{k}={v}" for k, v in b.items()) for c, b in CASES])
def test_refusals(N, call, bad):
    assert call(N, **bad) == N.MOE_ERR_INVALID_ARG
    assert N.lib.moe_launch_count() == 0


@pytest.mark.parametrize("call", [_dis, _dis_bwd])
def test_a_temperature_whose_scale_overflows_is_refused(N, call):
    """log2(e) / temperature is no finite number, though 1 / temperature is."""
    assert call(N, tau=3.5e-39) == N.MOE_ERR_INVALID_ARG


def test_missing_teacher(N):
    assert N.lib.moe_distill_forward(FAKE, FAKE, None, 4, 64, 10, FAKE, FAKE, FAKE, FAKE, BIG, None) == N.MOE_ERR_INVALID_ARG


def test_limits_and_workspaces(N):
    for call in (_emb, _emb_bwd, _ce, _ce_bwd, _dis, _dis_bwd):
        assert call(N, D=8256) == N.MOE_ERR_UNSUPPORTED_SHAPE
        assert call(N, V=N.MAX_VOCAB + 1) == N.MOE_ERR_UNSUPPORTED_SHAPE
        assert call(N, T=(1 << 24) + 1) == N.MOE_ERR_UNSUPPORTED_SHAPE
    for call in (_ce, _ce_bwd, _dis, _dis_bwd):
        assert call(N, D=96) == N.MOE_ERR_UNSUPPORTED_SHAPE
    for call in (_dis, _dis_bwd):
        assert call(N, K=N.MAX_TEACHER + 1) == N.MOE_ERR_UNSUPPORTED_SHAPE
    for call in (_emb, _ce, _dis):
        assert call(N, T=0) == N.MOE_OK          # nothing to do
    lib = N.lib
    sizes = [(_emb_bwd, lib.moe_embedding_backward_scratch_size(1001, 5003, 70), dict(D=70)),
             (_ce, lib.moe_vocab_forward_workspace_size(1001, 64, 5003, 0), {}),
             (_ce_bwd, lib.moe_vocab_backward_workspace_size(1001, 64, 5003, 0), {}),
             (_dis, lib.moe_vocab_forward_workspace_size(1001, 64, 5003, 8), {}),
             (_dis_bwd, lib.moe_vocab_backward_workspace_size(1001, 64, 5003, 8), {})]
    for call, n, kw in sizes:
        assert n > 0 and call(N, T=1001, V=5003, n=n - 1, **kw) == N.MOE_ERR_WORKSPACE
    assert lib.moe_embedding_backward_scratch_size(4, 0, 64) == 0
    for size in (lib.moe_vocab_forward_workspace_size, lib.moe_vocab_backward_workspace_size):
        assert size(4, 96, 10, 0) == 0 and size(4, 64, 10, -1) == 0 and size(4, 64, 10, N.MAX_TEACHER + 1) == 0
    # the gradient of the logits is held for a piece of the vocabulary at a time
    assert lib.moe_vocab_backward_workspace_size(1 << 18, 64, 1 << 17, 0) < 1 << 33
    assert lib.moe_launch_count() == 0


def test_binding_refuses_wrong_tensors(N):
    import torch
    from grouped_gemm_router_gb300 import moe
    x, W = torch.zeros(4, 64, dtype=torch.bfloat16), torch.zeros(10, 64, dtype=torch.bfloat16)
    ids, f = torch.zeros(4, dtype=torch.int64), torch.zeros(4)
    with pytest.raises(ValueError, match="CUDA"):
        moe.embedding_forward(ids, W)
    with pytest.raises(ValueError, match="int32 or torch.int64"):
        moe.embedding_forward(f, W)
    with pytest.raises(ValueError, match="bfloat16 or torch.float32"):
        moe.embedding_forward(ids, W.half())
    with pytest.raises(ValueError, match=r"\[V, D\]"):
        moe.embedding_forward(ids, W[0])
    with pytest.raises(ValueError, match="CUDA"):
        moe.embedding_backward(x, ids, 10)
    with pytest.raises(ValueError, match="CUDA"):
        moe.cross_entropy_forward(x, W, ids)
    with pytest.raises(ValueError, match="x must be torch.bfloat16"):
        moe.cross_entropy_forward(x.float(), W, ids)
    with pytest.raises(ValueError, match="CUDA"):
        moe.cross_entropy_backward(f, x, W, ids, f, f)
    with pytest.raises(ValueError, match="CUDA"):
        moe.distill_forward(x, W, ids[:, None], f[:, None])
    with pytest.raises(N.MoeError):
        moe.vocab_workspace_size(4, 96, 10)
    with pytest.raises(N.MoeError):
        moe.embedding_backward_workspace_size(4, 10, 8193)


def test_sizes_past_32_bits_are_refused(N, monkeypatch):
    """They are not cut to what their low halves say."""
    import torch
    from grouped_gemm_router_gb300 import moe
    big = 1 << 32
    for T, V, D in ((big + 4, 10, 64), (4, big + 10, 64), (4, 10, big + 64), (4, -10, 64)):
        with pytest.raises(N.MoeError):
            moe.embedding_backward_workspace_size(T, V, D)
        for backward in (False, True):
            with pytest.raises(N.MoeError):
                moe.vocab_workspace_size(T, D, V, backward=backward)
    with pytest.raises(N.MoeError):
        moe.vocab_workspace_size(4, 64, 10, n_teacher=big)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(FakeCuda, "data_ptr", lambda t: FAKE, raising=False)
    bf, i32, f = torch.bfloat16, torch.int32, torch.float32
    ids, y = FakeCuda((4,), i32), FakeCuda((big + 4,), i32)
    x, W = FakeCuda((4, 64), bf), FakeCuda((10, 64), bf)
    wide, many = FakeCuda((10, big + 64), bf), FakeCuda((big + 10, 64), bf)
    te, lg = FakeCuda((4, big + 8), i32), FakeCuda((4, big + 8), f)
    for call in (lambda: moe.embedding_forward(ids, wide), lambda: moe.embedding_forward(ids, many),
                 lambda: moe.embedding_forward(y, W), lambda: moe.embedding_backward(x, ids, big + 10),
                 lambda: moe.cross_entropy_forward(x, many, ids), lambda: moe.distill_forward(x, W, te, lg)):
        with pytest.raises(N.MoeError):
            call()


def _central(f, a, i, h=1e-5):
    a = a.copy()
    a[i] += h
    hi = f(a)
    a[i] -= 2 * h
    return (hi - f(a)) / (2 * h)


def test_gradients_against_differences():
    """The formulas the kernels compute, against central differences of the
    forward in 64 bits: step 1e-5 leaves an error of about 1e-9."""
    rng = np.random.default_rng(0)
    x, W = rng.standard_normal((4, 6)), rng.standard_normal((9, 6))
    dl, de = rng.standard_normal(4), rng.standard_normal(4)
    labels = np.array([3, -100, 8, 0])
    ids = np.array([[3, 5, -1], [-1, 9, -5], [0, 8, 4], [2, 2, 7]])      # one row without entries, one id twice
    lg = rng.standard_normal((4, 3))
    lg[2, 1] = -np.inf

    def ce(x_, W_):
        loss, lse = ref.cross_entropy(x_, W_, labels)
        return (loss * dl).sum() + (lse * de).sum()

    def dis(x_, W_):
        return (ref.distill(x_, W_, ids, lg, 1.7)[0] * dl).sum()

    for f, dz in ((ce, ref.cross_entropy_dz(x, W, labels, dl, de)), (dis, ref.distill_dz(x, W, ids, lg, 1.7, dl))):
        dx, dW = dz @ W, dz.T @ x
        for i in np.ndindex(x.shape):
            assert abs(_central(lambda a: f(a, W), x, i) - dx[i]) < 1e-7
        for i in np.ndindex(W.shape):
            assert abs(_central(lambda a: f(x, a), W, i) - dW[i]) < 1e-7
    assert (dz[1] == 0).all()

    toks, d_out = np.array([2, 9, 2, -1, 0]), rng.standard_normal((5, 6))
    g = ref.embedding_grad(d_out, toks, 9, 1.3)
    for i in np.ndindex(W.shape):
        assert abs(_central(lambda a: (ref.embedding(toks, a, 1.3) * d_out).sum(), W, i) - g[i]) < 1e-7


class FakeCuda:
    """What the checks look at of a CUDA tensor."""
    is_cuda = True

    def __init__(self, shape, dtype, index=0):
        import torch
        self.shape, self.dtype, self.device = torch.Size(shape), dtype, torch.device("cuda", index)

    def dim(self):
        return len(self.shape)

    def is_contiguous(self):
        return True

    def get_device(self):
        return self.device.index

    def data_ptr(self):
        raise AssertionError("used before all tensors were checked")


def _calls(moe, other, which):
    """The calls, tensor number `which` of each on device `other`."""
    import torch
    bf, f, i64, u8 = torch.bfloat16, torch.float32, torch.int64, torch.uint8

    def make(*specs):
        return [FakeCuda(s, t, other if i == which else 0) for i, (s, t) in enumerate(specs)]

    t, i = make(((10, 64), bf), ((4,), i64))
    yield 2, lambda: moe.embedding_forward(i, t)
    d, i1, add, ws = make(((4, 64), bf), ((4,), i64), ((10, 64), bf), ((1 << 24,), u8))
    yield 4, lambda: moe.embedding_backward(d, i1, 10, add=add, workspace=ws)
    x, W, y, ws1 = make(((4, 64), bf), ((10, 64), bf), ((4,), i64), ((1 << 24,), u8))
    yield 4, lambda: moe.cross_entropy_forward(x, W, y, workspace=ws1)
    x2, W2, y2, dl, lo, ls, de, ws2 = make(((4, 64), bf), ((10, 64), bf), ((4,), i64), ((4,), f), ((4,), f), ((4,), f),
                                          ((4,), f), ((1 << 24,), u8))
    yield 8, lambda: moe.cross_entropy_backward(dl, x2, W2, y2, lo, ls, d_lse=de, workspace=ws2)
    x3, W3, ti, tl, ws3 = make(((4, 64), bf), ((10, 64), bf), ((4, 8), i64), ((4, 8), f), ((1 << 24,), u8))
    yield 5, lambda: moe.distill_forward(x3, W3, ti, tl, workspace=ws3)
    x4, W4, ti4, tl4, dl4, ls4, z4, ws4 = make(((4, 64), bf), ((10, 64), bf), ((4, 8), i64), ((4, 8), f), ((4,), f), ((4,), f),
                                              ((4, 8), f), ((1 << 24,), u8))
    yield 8, lambda: moe.distill_backward(dl4, x4, W4, ti4, tl4, ls4, z4, workspace=ws4)


def test_tensors_of_another_device_are_refused(N, monkeypatch):
    import torch
    from grouped_gemm_router_gb300 import moe
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    for which in range(8):
        for n, call in _calls(moe, 1, which):
            if which < n:
                with pytest.raises(ValueError, match="cuda:1|cuda:0"):
                    call()
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 1)
    for _, call in _calls(moe, 1, 99):
        with pytest.raises(ValueError, match="current device"):
            call()


def test_small_workspaces_are_refused(N, monkeypatch):
    import torch
    from grouped_gemm_router_gb300 import moe
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(FakeCuda, "data_ptr", lambda t: FAKE, raising=False)
    monkeypatch.setattr(FakeCuda, "numel", lambda t: 128, raising=False)
    bf, u8 = torch.bfloat16, torch.uint8
    ws = FakeCuda((128,), u8)
    x, W, ids = FakeCuda((4, 64), bf), FakeCuda((10, 64), bf), FakeCuda((4,), torch.int32)
    with pytest.raises(N.MoeError):
        moe.cross_entropy_forward(x, W, ids, workspace=ws)
    with pytest.raises(N.MoeError):
        moe.embedding_backward(x, ids, 10, workspace=ws)
