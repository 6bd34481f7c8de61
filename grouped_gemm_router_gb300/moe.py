"""PyTorch-facing entry points of the MoE SwiGLU FFN forward and backward passes,
and of the operators beside them in a training step: layer norm, Newton-Schulz
orthogonalisation and the Muon step, embedding, cross entropy and distillation
over a vocabulary.

These functions only allocate outputs with torch, check shapes/dtypes, and
call the C ABI of libmoeffn.so on the current CUDA stream.  Tensor layouts:
  x [T, D] bf16, Wg [D, E] bf16, bias [E] fp32 (optional),
  W1, W3 [E, D, F] bf16, W2 [E, F, D] bf16,
  shared expert Ws1, Ws3 [D, F], Ws2 [F, D] bf16 (optional).
"""
from __future__ import annotations

import ctypes
import functools

import torch

from . import _native as N
from ._native import check, lib


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream():
    return ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)


def _need(t, name, dtype, shape=None):
    if t is None:
        return
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")


def layer_dims(x, W1, k):
    T, D = x.shape
    E, _, F = W1.shape
    return T, D, F, E, k


def workspace_size(T, D, F, E, k, shared, host_io=False) -> int:
    n = lib.moe_ffn_workspace_size(N.dims(T, D, F, E, k), int(bool(shared)), int(bool(host_io)))
    if n == 0:
        raise N.MoeError(N.MOE_ERR_UNSUPPORTED_SHAPE, "moe_ffn_workspace_size")
    return n


class Workspace:
    """Device workspace of moe_ffn_forward, with typed views of its regions
    (the layout documented in moe_ffn.h)."""

    def __init__(self, T, D, F, E, k, shared, host_io=False, device=None):
        self.dims = (T, D, F, E, k)
        self.shared = bool(shared)
        self.nbytes = workspace_size(T, D, F, E, k, shared, host_io)
        self.buf = torch.empty(self.nbytes, dtype=torch.uint8, device=device or "cuda")

    def views(self):
        T, D, F, E, k = self.dims
        S = T * k
        rows = S + (T if self.shared else 0)
        nblk = N.route_blocks(T)           # rows in use on this device
        nblk_max = (T + 15) // 16           # rows reserved (16-token blocks)
        out, off = {}, 0

        def take(name, n, dtype, shape):
            nonlocal off
            size = n * torch.tensor([], dtype=dtype).element_size()
            out[name] = self.buf[off:off + size].view(dtype).view(*shape)
            off += (size + 255) // 256 * 256

        npack = int(lib.moe_route_scratch_size(N.dims(T, D, F, E, k)))
        take("router_packed", npack, torch.uint8, (npack,))
        take("ids", S, torch.int32, (T, k))
        take("w", S, torch.float32, (T, k))
        take("hist", nblk_max * E, torch.int32, (nblk_max, E))
        out["hist"] = out["hist"][:nblk]
        take("counts", E, torch.int32, (E,))
        take("offsets", E + 1, torch.int32, (E + 1,))
        take("perm", S, torch.int32, (S,))
        take("inv", S, torch.int32, (S,))
        take("x_sorted", S * D, torch.bfloat16, (S, D))
        take("h", rows * F, torch.bfloat16, (rows, F))
        take("y", S * D, torch.bfloat16, (S, D))
        if self.shared:
            take("ys", T * D, torch.float32, (T, D))
        return out


def _options(stage_events=None, ids_in=None, weights_in=None, chained=False):
    if stage_events is None and ids_in is None and not chained:
        return None
    o = N.MoeOptions()
    o.flags = N.MOE_FFN_CHAINED if chained else 0
    for i, ev in enumerate(stage_events or []):
        if ev is None:
            continue
        handle = ev.cuda_event if hasattr(ev, "cuda_event") else int(ev)
        if not handle:
            # torch creates the CUDA event lazily, on its first record()
            ev.record()
            handle = ev.cuda_event
        o.stage_events[i] = handle
    if ids_in is not None:
        _need(ids_in, "ids_in", torch.int32)
        _need(weights_in, "weights_in", torch.float32)
        o.ids_in = ids_in.data_ptr()
        o.weights_in = weights_in.data_ptr()
    return ctypes.byref(o)


def moe_ffn_forward(x, Wg, W1, W3, W2, k, bias=None, Ws1=None, Ws3=None, Ws2=None, out=None,
                    workspace: Workspace | None = None, stage_events=None, ids_in=None,
                    weights_in=None, chained=False):
    """Forward pass of the MoE SwiGLU FFN layer; returns out [T, D] bf16.
    chained=True runs W1||W3 and W2 as one kernel with h kept on chip
    (D <= 256)."""
    T, D, F, E, k = layer_dims(x, W1, k)
    shared = Ws1 is not None
    for t, n, shp in ((x, "x", (T, D)), (Wg, "Wg", (D, E)), (W1, "W1", (E, D, F)),
                      (W3, "W3", (E, D, F)), (W2, "W2", (E, F, D)), (Ws1, "Ws1", (D, F)),
                      (Ws3, "Ws3", (D, F)), (Ws2, "Ws2", (F, D))):
        _need(t, n, torch.bfloat16, shp)
    _need(bias, "bias", torch.float32, (E,))
    if out is None:
        out = torch.empty(T, D, dtype=torch.bfloat16, device=x.device)
    if workspace is None:
        workspace = Workspace(T, D, F, E, k, shared, device=x.device)
    st = lib.moe_ffn_forward(_ptr(x), _ptr(Wg), _ptr(bias), _ptr(W1), _ptr(W3), _ptr(W2), _ptr(Ws1),
                             _ptr(Ws3), _ptr(Ws2), N.dims(T, D, F, E, k), _ptr(out),
                             _ptr(workspace.buf), workspace.nbytes,
                             _options(stage_events, ids_in, weights_in, chained), _stream())
    check(st, "moe_ffn_forward")
    return out


def moe_ffn_forward_host(x_host, Wg, W1, W3, W2, k, out_host, workspace: Workspace, bias=None,
                         Ws1=None, Ws3=None, Ws2=None, stage_events=None):
    """Forward pass with x and out in (pinned) host memory; copies are part of
    the call, enqueued on the current stream."""
    T, D, F, E, k = layer_dims(x_host, W1, k)
    if x_host.is_cuda or out_host.is_cuda:
        raise ValueError("x_host and out_host must be host tensors")
    st = lib.moe_ffn_forward_host(_ptr(x_host), _ptr(Wg), _ptr(bias), _ptr(W1), _ptr(W3), _ptr(W2),
                                  _ptr(Ws1), _ptr(Ws3), _ptr(Ws2), N.dims(T, D, F, E, k),
                                  _ptr(out_host), _ptr(workspace.buf), workspace.nbytes,
                                  _options(stage_events), _stream())
    check(st, "moe_ffn_forward_host")
    return out_host


class BackwardWorkspace:
    """Device workspace of moe_ffn_backward, with typed views of its regions
    (the layout documented in moe_ffn.h: padded sorted rows, the shared rows
    from S_pad = T*k + 64*E)."""

    def __init__(self, T, D, F, E, k, shared, device=None):
        self.dims = (T, D, F, E, k)
        self.shared = bool(shared)
        self.nbytes = int(lib.moe_ffn_backward_workspace_size(N.dims(T, D, F, E, k), int(bool(shared))))
        if self.nbytes == 0 and T > 0:
            raise N.MoeError(N.MOE_ERR_UNSUPPORTED_SHAPE, "moe_ffn_backward_workspace_size")
        self.buf = torch.empty(max(self.nbytes, 256), dtype=torch.uint8, device=device or "cuda")

    def views(self):
        T, D, F, E, k = self.dims
        S = T * k
        Sp = S + 64 * E
        rows = Sp + (T if self.shared else 0)
        out, off = {"S_pad": Sp}, 0

        def take(name, n, dtype, shape):
            nonlocal off
            size = n * torch.tensor([], dtype=dtype).element_size()
            out[name] = self.buf[off:off + size].view(dtype).view(*shape)
            off += (size + 255) // 256 * 256

        take("ybar", Sp * D, torch.bfloat16, (Sp, D))
        take("hbar", rows * F, torch.bfloat16, (rows, F))
        take("gu", rows * 2 * F, torch.bfloat16, (rows, 2 * F))
        take("h", rows * F, torch.bfloat16, (rows, F))
        take("xbar", rows * D, torch.bfloat16, (rows, D))
        take("wbar", S, torch.float32, (T, k))
        take("lbar", S, torch.float32, (T, k))
        return out


def padded_rows(counts):
    """Row of each sorted position in the backward's padded layout: group e
    starts at the sum of the earlier group sizes rounded up to 64."""
    counts = [int(c) for c in counts]
    prow0, run = [], 0
    for c in counts:
        prow0.append(run)
        run += (c + 63) // 64 * 64
    idx = []
    for e, c in enumerate(counts):
        idx.extend(range(prow0[e], prow0[e] + c))
    return idx


def moe_ffn_backward(x, Wg, W1, W3, W2, k, d_out, workspace: Workspace, Ws1=None, Ws3=None, Ws2=None,
                     bwd_workspace: BackwardWorkspace | None = None, ids_in=None, weights_in=None,
                     router=True, stage_events=None, chained=False):
    """Gradients of sum(d_out * out) for the forward call that filled
    `workspace`.  Returns dict(dx bf16 [T, D], dW1, dW3 [E, D, F], dW2 [E, F, D]
    (+ dWs1, dWs3, dWs2), and with router=True dWg [D, E], dbias [E]) fp32.
    chained: the forward call ran with chained=True (its workspace has no h)."""
    T, D, F, E, k = layer_dims(x, W1, k)
    shared = Ws1 is not None
    _need(d_out, "d_out", torch.bfloat16, (T, D))
    dev = x.device
    f32 = dict(dtype=torch.float32, device=dev)
    g = dict(dx=torch.empty(T, D, dtype=torch.bfloat16, device=dev),
             dW1=torch.empty(E, D, F, **f32), dW3=torch.empty(E, D, F, **f32), dW2=torch.empty(E, F, D, **f32))
    if shared:
        g.update(dWs1=torch.empty(D, F, **f32), dWs3=torch.empty(D, F, **f32), dWs2=torch.empty(F, D, **f32))
    if router:
        g.update(dWg=torch.empty(D, E, **f32), dbias=torch.empty(E, **f32))
    if bwd_workspace is None:
        bwd_workspace = BackwardWorkspace(T, D, F, E, k, shared, device=dev)
    st = lib.moe_ffn_backward(_ptr(x), _ptr(Wg), _ptr(W1), _ptr(W3), _ptr(W2), _ptr(Ws1), _ptr(Ws3), _ptr(Ws2),
                              _ptr(d_out), N.dims(T, D, F, E, k), _ptr(workspace.buf), workspace.nbytes,
                              _ptr(g["dx"]), _ptr(g.get("dWg")), _ptr(g.get("dbias")), _ptr(g["dW1"]),
                              _ptr(g["dW3"]), _ptr(g["dW2"]), _ptr(g.get("dWs1")), _ptr(g.get("dWs3")),
                              _ptr(g.get("dWs2")), _ptr(bwd_workspace.buf), bwd_workspace.nbytes,
                              _options(stage_events, ids_in, weights_in, chained), _stream())
    check(st, "moe_ffn_backward")
    return g


def moe_route(x, Wg, k, bias=None):
    """Router GEMM + top-k + softmax -> (ids [T,k] int32, weights [T,k] fp32,
    block_hist [ceil(T/TB), E] int32 with TB = moe_route_block_tokens(T))."""
    T, D = x.shape
    E = Wg.shape[1]
    _need(x, "x", torch.bfloat16, (T, D))
    _need(Wg, "Wg", torch.bfloat16, (D, E))
    _need(bias, "bias", torch.float32, (E,))
    ids = torch.empty(T, k, dtype=torch.int32, device=x.device)
    w = torch.empty(T, k, dtype=torch.float32, device=x.device)
    hist = torch.empty(N.route_blocks(T), E, dtype=torch.int32, device=x.device)
    d = N.dims(T, D, 64, E, k)
    nscratch = int(lib.moe_route_scratch_size(d))
    scratch = torch.empty(max(nscratch, 16), dtype=torch.uint8, device=x.device)
    st = lib.moe_route(_ptr(x), _ptr(Wg), _ptr(bias), d, _ptr(ids), _ptr(w), _ptr(hist), _ptr(scratch),
                       nscratch, _stream())
    check(st, "moe_route")
    return ids, w, hist


def moe_permute(ids, E, x=None):
    """Stable expert-grouped permutation of ids [T, k]; with x, also the
    gathered x_sorted [T*k, D]."""
    T, k = ids.shape
    _need(ids, "ids", torch.int32, (T, k))
    D = x.shape[1] if x is not None else 64
    if x is not None:
        _need(x, "x", torch.bfloat16, (T, D))
    d = N.dims(T, D, 64, E, k)
    dev = ids.device
    S = T * k
    counts = torch.empty(E, dtype=torch.int32, device=dev)
    offsets = torch.empty(E + 1, dtype=torch.int32, device=dev)
    perm = torch.empty(S, dtype=torch.int32, device=dev)
    inv = torch.empty(S, dtype=torch.int32, device=dev)
    xs = torch.empty(S, D, dtype=torch.bfloat16, device=dev) if x is not None else None
    nscratch = max(int(lib.moe_permute_scratch_size(d)), 16)
    scratch = torch.empty(nscratch, dtype=torch.uint8, device=dev)
    st = lib.moe_permute(_ptr(ids), d, _ptr(counts), _ptr(offsets), _ptr(perm), _ptr(inv), _ptr(x),
                         _ptr(xs), _ptr(scratch), nscratch, _stream())
    check(st, "moe_permute")
    return dict(counts=counts, offsets=offsets, perm=perm, inv=inv, x_sorted=xs)


def moe_grouped_swiglu(x_sorted, offsets, W1, W3, T, k, x=None, Ws1=None, Ws3=None, h=None):
    """h [T*k (+T), F] = silu(A W1[e]) * (A W3[e]) per expert group (+ shared rows)."""
    S, D = x_sorted.shape
    E, _, F = W1.shape
    shared = Ws1 is not None
    _need(x_sorted, "x_sorted", torch.bfloat16, (T * k, D))
    _need(W1, "W1", torch.bfloat16, (E, D, F))
    _need(W3, "W3", torch.bfloat16, (E, D, F))
    _need(offsets, "offsets", torch.int32, (E + 1,))
    if shared:
        _need(x, "x", torch.bfloat16, (T, D))
        _need(Ws1, "Ws1", torch.bfloat16, (D, F))
        _need(Ws3, "Ws3", torch.bfloat16, (D, F))
    rows = T * k + (T if shared else 0)
    if h is None:
        h = torch.empty(rows, F, dtype=torch.bfloat16, device=x_sorted.device)
    st = lib.moe_grouped_swiglu(_ptr(x_sorted), _ptr(x), _ptr(W1), _ptr(W3), _ptr(Ws1), _ptr(Ws3),
                                _ptr(offsets), N.dims(T, D, F, E, k), _ptr(h), _stream())
    check(st, "moe_grouped_swiglu")
    return h


def moe_grouped_down(h, offsets, W2, T, k, Ws2=None, y=None, ys=None):
    """(y [T*k, D] bf16, ys [T, D] fp32 or None): y = h W2[e] per expert
    group; with Ws2, ys = the shared rows of h times Ws2."""
    E, F, D = W2.shape
    shared = Ws2 is not None
    rows = T * k + (T if shared else 0)
    _need(h, "h", torch.bfloat16, (rows, F))
    _need(W2, "W2", torch.bfloat16, (E, F, D))
    _need(Ws2, "Ws2", torch.bfloat16, (F, D))
    _need(offsets, "offsets", torch.int32, (E + 1,))
    if y is None:
        y = torch.empty(T * k, D, dtype=torch.bfloat16, device=h.device)
    if shared and ys is None:
        ys = torch.empty(T, D, dtype=torch.float32, device=h.device)
    _need(y, "y", torch.bfloat16, (T * k, D))
    if shared:
        _need(ys, "ys", torch.float32, (T, D))
    st = lib.moe_grouped_down(_ptr(h), _ptr(W2), _ptr(Ws2), _ptr(offsets), N.dims(T, D, F, E, k),
                              _ptr(y), _ptr(ys if shared else None), _stream())
    check(st, "moe_grouped_down")
    return y, (ys if shared else None)


def moe_grouped_ffn_chained(x_sorted, offsets, W1, W3, W2, T, k, x=None, Ws1=None, Ws3=None,
                            Ws2=None, y=None, ys=None):
    """(y [T*k, D] bf16, ys [T, D] fp32 or None) = (silu(A W1[e]) * (A W3[e]))
    W2[e] per expert group (+ the shared expert's rows), in one kernel that
    never writes h (D <= 256)."""
    S, D = x_sorted.shape
    E, _, F = W1.shape
    shared = Ws1 is not None
    _need(x_sorted, "x_sorted", torch.bfloat16, (T * k, D))
    _need(W1, "W1", torch.bfloat16, (E, D, F))
    _need(W3, "W3", torch.bfloat16, (E, D, F))
    _need(W2, "W2", torch.bfloat16, (E, F, D))
    _need(offsets, "offsets", torch.int32, (E + 1,))
    if shared:
        _need(x, "x", torch.bfloat16, (T, D))
        _need(Ws1, "Ws1", torch.bfloat16, (D, F))
        _need(Ws3, "Ws3", torch.bfloat16, (D, F))
        _need(Ws2, "Ws2", torch.bfloat16, (F, D))
    if y is None:
        y = torch.empty(T * k, D, dtype=torch.bfloat16, device=x_sorted.device)
    if shared and ys is None:
        ys = torch.empty(T, D, dtype=torch.float32, device=x_sorted.device)
    _need(y, "y", torch.bfloat16, (T * k, D))
    if shared:
        _need(ys, "ys", torch.float32, (T, D))
    st = lib.moe_grouped_ffn_chained(_ptr(x_sorted), _ptr(x), _ptr(W1), _ptr(W3), _ptr(W2), _ptr(Ws1),
                                     _ptr(Ws3), _ptr(Ws2), _ptr(offsets), N.dims(T, D, F, E, k), _ptr(y),
                                     _ptr(ys if shared else None), _stream())
    check(st, "moe_grouped_ffn_chained")
    return y, (ys if shared else None)


def moe_combine(y, weights, inv, ys=None, out=None):
    """out[t] = sum_j weights[t, j] * y[inv[t*k + j]] (+ ys[t], fp32)."""
    T, k = weights.shape
    D = y.shape[1]
    _need(y, "y", torch.bfloat16, (T * k, D))
    _need(ys, "ys", torch.float32, (T, D))
    _need(weights, "weights", torch.float32, (T, k))
    _need(inv, "inv", torch.int32, (T * k,))
    if out is None:
        out = torch.empty(T, D, dtype=torch.bfloat16, device=y.device)
    E = max(k, 1)
    st = lib.moe_combine(_ptr(y), _ptr(ys), _ptr(weights), _ptr(inv), N.dims(T, D, 64, E, k),
                         _ptr(out), _stream())
    check(st, "moe_combine")
    return out


_STREAM_TYPES = {torch.bfloat16: N.MOE_BF16, torch.float32: N.MOE_FP32}
_F32 = torch.float32
_BF16 = torch.bfloat16
_empty = torch.empty
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)  # a torch without CUDA has none


def _stream_of(t):
    """The current stream of t's device, as the C ABI takes it (0.1 us where
    torch.cuda.current_stream() takes 3: these calls are a few us each)."""
    return _raw_stream(t.device.index)


def _like(t, name, dtype, shape, dev):
    """As _need for a tensor that must be there, on device number dev, without
    the copies."""
    if t.dtype is not dtype or t.shape != shape or t.get_device() != dev or not t.is_contiguous():
        _need(t, name, dtype, shape)
        raise ValueError(f"{name} is on {t.device}, the first tensor on cuda:{dev}")


def _current(t, name):
    """The number of t's device, which has to be the current one: that is where
    the C ABI launches."""
    dev, now = t.get_device(), torch.cuda.current_device()
    if dev != now:
        raise ValueError(f"{name} is on {t.device}, the current device is cuda:{now}")
    return dev


def _aligned(t):
    """t, or a copy of it where it does not start on the 16-byte boundary that
    the C ABI needs (a view into a larger tensor)."""
    return t.clone() if t is not None and t.data_ptr() & 15 else t


def _ns_workspace(t, dev):
    if t is not None:
        _like(t, "workspace", torch.uint8, t.shape, dev)
        if t.data_ptr() & 255:
            raise ValueError("workspace must start on a 256-byte boundary")


def _stream_type(x):
    """The C ABI's element type of a residual stream x."""
    kind = _STREAM_TYPES.get(x.dtype)
    if kind is None:
        raise ValueError(f"x must be torch.bfloat16 or torch.float32, got {x.dtype}")
    if x.dim() != 2:
        raise ValueError(f"x has shape {tuple(x.shape)}, expected [T, D]")
    if not x.is_cuda or not x.is_contiguous():
        _need(x, "x", x.dtype)
    return kind


def layer_norm_forward(x, weight, bias=None, eps=1e-5, add=None, y=None):
    """Layer norm of a residual stream x [T, D] (bf16 or fp32), the input of
    the MoE layer: dict(y [T, D] bf16, mean [T] fp32, rstd [T] fp32).  With
    `add` [T, D] bf16 (a sublayer's output) the stream becomes h = x + add,
    rounded to x's type, and that is what is normalised; the dict then holds
    h too.  weight, bias: [D] fp32.  Any D up to 8192.  A tensor that does not
    start on 16 bytes is copied first."""
    kind = _stream_type(x)
    dev = _current(x, "x")
    shape = x.shape
    T, D = shape
    _like(weight, "weight", _F32, (D,), dev)
    if bias is not None:
        _like(bias, "bias", _F32, (D,), dev)
    if add is not None:
        _like(add, "add", _BF16, shape, dev)
    if y is not None:
        _like(y, "y", _BF16, shape, dev)
    else:
        y = _empty(shape, dtype=_BF16, device=x.device)
    px, pw, py = x.data_ptr(), weight.data_ptr(), y.data_ptr()
    pb = None if bias is None else bias.data_ptr()
    pa = None if add is None else add.data_ptr()
    if (px | pw | py | (pb or 0) | (pa or 0)) & 15:
        out = layer_norm_forward(_aligned(x), _aligned(weight), _aligned(bias), eps, _aligned(add), _aligned(y))
        if out["y"] is not y:
            out["y"] = y.copy_(out["y"])
        return out
    mean = _empty(T, dtype=_F32, device=x.device)
    rstd = _empty(T, dtype=_F32, device=x.device)
    out = dict(y=y, mean=mean, rstd=rstd)
    h = None
    if add is not None:
        h = out["h"] = torch.empty_like(x)
    st = lib.moe_layer_norm_forward(px, kind, pa, pw, pb, eps, T, D, py, None if h is None else h.data_ptr(),
                                    mean.data_ptr(), rstd.data_ptr(), _stream_of(x))
    if st:
        check(st, "moe_layer_norm_forward")
    return out


def layer_norm_backward(dy, x, weight, mean, rstd, bias=True, d_stream=None):
    """Gradients of sum(dy * y) (+ sum(d_stream * h)) for layer_norm_forward:
    dict(dx [T, D] in x's type, dweight [D] fp32, and with bias=True dbias [D]
    fp32).  x: the rows that were normalised (the forward's h where it added);
    mean, rstd: the forward's; dy [T, D] bf16; d_stream [T, D] in x's type:
    the gradient that reaches these rows past the norm.  A tensor that does not
    start on 16 bytes is copied first."""
    kind = _stream_type(x)
    dev = _current(x, "x")
    shape = x.shape
    T, D = shape
    _like(dy, "dy", _BF16, shape, dev)
    _like(weight, "weight", _F32, (D,), dev)
    _like(mean, "mean", _F32, (T,), dev)
    _like(rstd, "rstd", _F32, (T,), dev)
    if d_stream is not None:
        _like(d_stream, "d_stream", x.dtype, shape, dev)
    pdy, px, pw, pm, pr = dy.data_ptr(), x.data_ptr(), weight.data_ptr(), mean.data_ptr(), rstd.data_ptr()
    pd = None if d_stream is None else d_stream.data_ptr()
    if (pdy | px | pw | pm | pr | (pd or 0)) & 15:
        return layer_norm_backward(*(_aligned(t) for t in (dy, x, weight, mean, rstd)), bias, _aligned(d_stream))
    dx = torch.empty_like(x)
    dweight = _empty(D, dtype=_F32, device=x.device)
    out = dict(dx=dx, dweight=dweight)
    dbias = None
    if bias:
        dbias = out["dbias"] = _empty(D, dtype=_F32, device=x.device)
    nscratch = lib.moe_layer_norm_backward_scratch_size(T, D)
    scratch = _empty(max(nscratch, 16), dtype=torch.uint8, device=x.device)
    st = lib.moe_layer_norm_backward(pdy, px, kind, pw, pm, pr, pd, T, D, dx.data_ptr(), dweight.data_ptr(),
                                     None if dbias is None else dbias.data_ptr(), scratch.data_ptr(), nscratch,
                                     _stream_of(x))
    if st:
        check(st, "moe_layer_norm_backward")
    return out


NS_COEFFICIENTS = (3.4445, -4.7750, 2.0315)


def _ns_coefficients(coefficients, steps):
    """steps x 3 C floats from one (a, b, c) for every step, or one for each."""
    c = list(coefficients)
    if c and not hasattr(c[0], "__len__"):
        c = [c] * steps
    if len(c) != steps or any(len(t) != 3 for t in c):
        raise ValueError(f"coefficients: one (a, b, c), or {steps} of them")
    return (ctypes.c_float * (3 * steps))(*(float(v) for t in c for v in t))


def newton_schulz_workspace_size(count, rows, cols) -> int:
    n = int(lib.moe_newton_schulz_workspace_size(count, rows, cols))
    if n == 0 and count > 0:
        raise N.MoeError(N.MOE_ERR_UNSUPPORTED_SHAPE, "moe_newton_schulz_workspace_size")
    return n


def newton_schulz(g, steps=5, coefficients=NS_COEFFICIENTS, eps=1e-7, out=None, workspace=None):
    """Orthogonalises each matrix of g [rows, cols] or [B, rows, cols] (bf16
    or fp32): X = G / (|G| + eps), then `steps` times
    X <- a X + (b A + c A A) X with A = X X^T (X^T X where rows > cols).
    Returns bf16 of g's shape.  coefficients: one (a, b, c) or one for each
    step.  The products take fp16 operands and fp32 sums: before its rounding
    to bf16 the result is about 1e-3 off in the 2-norm (moe_ffn.h has the
    ranges).  workspace: a uint8 CUDA tensor of newton_schulz_workspace_size
    bytes.  A g or out that does not start on 16 bytes goes through a copy."""
    kind = _STREAM_TYPES.get(g.dtype)
    if kind is None:
        raise ValueError(f"g must be torch.bfloat16 or torch.float32, got {g.dtype}")
    if g.dim() not in (2, 3):
        raise ValueError(f"g has shape {tuple(g.shape)}, expected [rows, cols] or [B, rows, cols]")
    _need(g, "g", g.dtype)
    dev = _current(g, "g")
    if out is not None:
        _like(out, "out", _BF16, g.shape, dev)
    _ns_workspace(workspace, dev)
    count = g.shape[0] if g.dim() == 3 else 1
    rows, cols = g.shape[-2:]
    c = _ns_coefficients(coefficients, steps)
    nbytes = newton_schulz_workspace_size(count, rows, cols)
    if out is None:
        out = torch.empty(g.shape, dtype=torch.bfloat16, device=g.device)
    if (g.data_ptr() | out.data_ptr()) & 15:
        o = newton_schulz(_aligned(g), steps, coefficients, eps, _aligned(out), workspace)
        return o if o is out else out.copy_(o)
    if workspace is None:
        workspace = torch.empty(max(nbytes, 256), dtype=torch.uint8, device=g.device)
    st = lib.moe_newton_schulz(g.data_ptr(), kind, count, rows, cols, steps, c, eps, out.data_ptr(),
                               workspace.data_ptr(), workspace.numel(), _stream_of(g))
    check(st, "moe_newton_schulz")
    return out


def muon_step(weights, grads, momenta, lr, momentum=0.95, nesterov=True, weight_decay=0.0, steps=5,
              coefficients=NS_COEFFICIENTS, eps=1e-7, scale=None, weights_bf16=None, workspace=None):
    """One Muon step, in place, on lists of weight matrices or stacks of them
    ([rows, cols] or [B, rows, cols]; the expert weights W1, W3, W2 as they
    are):
        m <- momentum m + g;  u = g + momentum m (nesterov) or m
        w <- (1 - lr weight_decay) w - lr scale newton_schulz(u)
    weights: all bf16, or all fp32, then with weights_bf16 (a list, entries
    may be None) the bf16 copies that the layer reads are written too; grads:
    all fp32 (as moe_ffn_backward returns them) or all bf16; momenta: fp32.
    scale: by default 0.2 sqrt(max(rows, cols)).  Matrices of the same shape
    up to transposition are worked on together, and the weights move by
    newton_schulz's result before its rounding to bf16.  workspace: a uint8
    CUDA tensor of the largest newton_schulz_workspace_size among those groups.
    Tensors that do not start on 16 bytes are updated by way of copies."""
    n = len(weights)
    low = [None] * n if weights_bf16 is None else list(weights_bf16)
    if not (len(grads) == len(momenta) == len(low) == n):
        raise ValueError("weights, grads, momenta and weights_bf16 must have the same length")
    if n == 0:
        return
    wtype, gtype = weights[0].dtype, grads[0].dtype
    for t, name in ((wtype, "weights"), (gtype, "grads")):
        if t not in _STREAM_TYPES:
            raise ValueError(f"{name} must be torch.bfloat16 or torch.float32, got {t}")
    dev = None
    for i, (w, g, m, b) in enumerate(zip(weights, grads, momenta, low)):
        if w.dim() not in (2, 3):
            raise ValueError(f"weights[{i}] has shape {tuple(w.shape)}, expected [rows, cols] or [B, rows, cols]")
        _need(w, f"weights[{i}]", wtype)
        if dev is None:
            dev = _current(w, "weights[0]")
        _like(w, f"weights[{i}]", wtype, w.shape, dev)
        _like(g, f"grads[{i}]", gtype, w.shape, dev)
        _like(m, f"momenta[{i}]", _F32, w.shape, dev)
        if b is not None:
            _like(b, f"weights_bf16[{i}]", _BF16, w.shape, dev)
            if wtype != _F32:
                raise ValueError("weights_bf16 are the copies of fp32 weights")
    _ns_workspace(workspace, dev)
    groups, copies = {}, []
    for tensors in zip(weights, grads, momenta, low):
        used = [_aligned(t) for t in tensors]
        copies += [(t, a) for t, a in zip(tensors, used) if a is not t]
        w, g, m, b = used
        rows, cols = w.shape[-2:]
        stack = N.MoeMatrixStack(w.data_ptr(), g.data_ptr(), m.data_ptr(), None if b is None else b.data_ptr(),
                                 w.shape[0] if w.dim() == 3 else 1, rows, cols)
        groups.setdefault((min(rows, cols), max(rows, cols)), []).append(stack)
    c = _ns_coefficients(coefficients, steps)
    calls = [(key, group[i:i + N.MAX_STACKS]) for key, group in groups.items()
             for i in range(0, len(group), N.MAX_STACKS)]
    sizes = [newton_schulz_workspace_size(sum(s.count for s in group), *key) for key, group in calls]
    if workspace is None:
        workspace = torch.empty(max(*sizes, 256), dtype=torch.uint8, device=weights[0].device)
    if workspace.numel() < max(sizes):
        raise N.MoeError(N.MOE_ERR_WORKSPACE, "moe_muon_step")
    stream = _stream_of(weights[0])
    for key, group in calls:
        p = N.MoeMuonParams(lr, momentum, weight_decay, 0.2 * key[1] ** 0.5 if scale is None else scale, eps,
                            int(bool(nesterov)), steps, ctypes.addressof(c))
        st = lib.moe_muon_step((N.MoeMatrixStack * len(group))(*group), len(group), _STREAM_TYPES[gtype],
                               _STREAM_TYPES[wtype], ctypes.byref(p), workspace.data_ptr(), workspace.numel(), stream)
        check(st, "moe_muon_step")
    for t, a in copies:
        t.copy_(a)


_INDEX_TYPES = {torch.int32: N.MOE_I32, torch.int64: N.MOE_I64}


def _index_type(t, name):
    kind = _INDEX_TYPES.get(t.dtype)
    if kind is None:
        raise ValueError(f"{name} must be torch.int32 or torch.int64, got {t.dtype}")
    return kind


def _float_type(t, name):
    kind = _STREAM_TYPES.get(t.dtype)
    if kind is None:
        raise ValueError(f"{name} must be torch.bfloat16 or torch.float32, got {t.dtype}")
    return kind


def _in_32_bits(where, *sizes):
    """The C ABI takes 32-bit sizes; larger ones would be cut."""
    if max(sizes) >= 1 << 31 or min(sizes) < 0:
        raise N.MoeError(N.MOE_ERR_UNSUPPORTED_SHAPE, where)


def _matrix(t, name, of):
    if t.dim() != 2:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected [{of}]")
    if not t.is_cuda or not t.is_contiguous():
        _need(t, name, t.dtype)
    return t.shape


def _buffer(workspace, nbytes, dev, device, where):
    """The caller's workspace, or one of nbytes."""
    if workspace is None:
        return torch.empty(max(nbytes, 256), dtype=torch.uint8, device=device)
    _ns_workspace(workspace, dev)
    if workspace.numel() < max(nbytes, 1):
        raise N.MoeError(N.MOE_ERR_WORKSPACE, where)
    return workspace


def embedding_forward(ids, table, scale=1.0, out_type=None):
    """out [T, D] = scale * table[ids], in out_type (by default the table's
    type): ids [T] int32 or int64, table [V, D] bf16 or fp32.  An id outside
    [0, V) gives a row of zeros.  Any D up to 8192.  A tensor that does not
    start on 16 bytes is copied first."""
    ikind, tkind = _index_type(ids, "ids"), _float_type(table, "table")
    V, D = _matrix(table, "table", "V, D")
    dev = _current(table, "table")
    if ids.dim() != 1:
        raise ValueError(f"ids has shape {tuple(ids.shape)}, expected [T]")
    _like(ids, "ids", ids.dtype, ids.shape, dev)
    out_type = table.dtype if out_type is None else out_type
    okind = _STREAM_TYPES.get(out_type)
    if okind is None:
        raise ValueError(f"out_type must be torch.bfloat16 or torch.float32, got {out_type}")
    pi, pt = ids.data_ptr(), table.data_ptr()
    if (pi | pt) & 15:
        return embedding_forward(_aligned(ids), _aligned(table), scale, out_type)
    T = ids.shape[0]
    _in_32_bits("moe_embedding_forward", T, V, D)
    out = _empty(T, D, dtype=out_type, device=table.device)
    st = lib.moe_embedding_forward(pi, ikind, pt, tkind, scale, T, V, D, out.data_ptr(), okind, _stream_of(table))
    if st:
        check(st, "moe_embedding_forward")
    return out


def embedding_backward(d_out, ids, V, scale=1.0, add=None, workspace=None):
    """Gradient of sum(d_out * embedding_forward(ids, table, scale)) in the
    table: [V, D] fp32, (add +) scale * the sums of d_out's rows by id.  d_out
    [T, D] bf16 or fp32; add [V, D] bf16: a gradient that reaches the table
    elsewhere (a tied head's dW).  The sums run in a fixed order.  workspace: a
    uint8 CUDA tensor of embedding_backward_workspace_size bytes.  A tensor that
    does not start on 16 bytes is copied first."""
    ikind, dkind = _index_type(ids, "ids"), _float_type(d_out, "d_out")
    T, D = _matrix(d_out, "d_out", "T, D")
    dev = _current(d_out, "d_out")
    _like(ids, "ids", ids.dtype, (T,), dev)
    if add is not None:
        _like(add, "add", _BF16, (V, D), dev)
    nbytes = embedding_backward_workspace_size(T, V, D)
    ws = _buffer(workspace, nbytes, dev, d_out.device, "moe_embedding_backward")
    pd, pi = d_out.data_ptr(), ids.data_ptr()
    pa = None if add is None else add.data_ptr()
    if (pd | pi | (pa or 0)) & 15:
        return embedding_backward(_aligned(d_out), _aligned(ids), V, scale, _aligned(add), ws)
    out = _empty(V, D, dtype=_F32, device=d_out.device)
    st = lib.moe_embedding_backward(pd, dkind, pi, ikind, scale, pa, T, V, D, out.data_ptr(), ws.data_ptr(),
                                    ws.numel(), _stream_of(d_out))
    if st:
        check(st, "moe_embedding_backward")
    return out


@functools.lru_cache(maxsize=1024)  # a size depends on nothing else (1 us a call)
def embedding_backward_workspace_size(T, V, D) -> int:
    _in_32_bits("moe_embedding_backward_scratch_size", T, V, D)
    n = int(lib.moe_embedding_backward_scratch_size(T, V, D))
    if n == 0 and T > 0:
        raise N.MoeError(N.MOE_ERR_UNSUPPORTED_SHAPE, "moe_embedding_backward_scratch_size")
    return n


@functools.lru_cache(maxsize=1024)
def vocab_workspace_size(T, D, V, n_teacher=0, backward=False) -> int:
    """Bytes of workspace of cross_entropy_* (n_teacher = 0) and distill_*.  A
    backward's holds the logits' gradient of a piece of the vocabulary in bf16: 2 T V
    bytes, but at most the larger of 4 GiB and 4096 T, and fp32 sums beside it."""
    name = "moe_vocab_backward_workspace_size" if backward else "moe_vocab_forward_workspace_size"
    _in_32_bits(name, T, D, V, n_teacher)
    n = int(getattr(lib, name)(T, D, V, n_teacher))
    if n == 0 and T > 0:
        raise N.MoeError(N.MOE_ERR_UNSUPPORTED_SHAPE, name)
    return n


def _head(x, W):
    """(T, D, V, device number) of the hidden states and the table."""
    if x.dtype != _BF16:
        raise ValueError(f"x must be torch.bfloat16, got {x.dtype}")
    T, D = _matrix(x, "x", "T, D")
    dev = _current(x, "x")
    if W.dim() != 2:
        raise ValueError(f"W has shape {tuple(W.shape)}, expected [V, {D}]")
    V = W.shape[0]
    _like(W, "W", _BF16, (V, D), dev)
    return T, D, V, dev


def _labels(labels, T, dev):
    kind = _index_type(labels, "labels")
    _like(labels, "labels", labels.dtype, (T,), dev)
    return kind


def cross_entropy_forward(x, W, labels, workspace=None):
    """Softmax cross entropy of the logits z = x W^T, which are never stored:
    dict(loss [T], lse [T]) fp32 with lse = log sum exp z and loss = lse -
    z[label].  x [T, D] bf16 (D a multiple of 64), W [V, D] bf16 (an embedding
    table's layout), labels [T] int32 or int64; a label outside [0, V) is a
    token without a loss: 0.  workspace: a uint8 CUDA tensor of
    vocab_workspace_size bytes.  A tensor that does not start on 16 bytes is
    copied first."""
    T, D, V, dev = _head(x, W)
    kind = _labels(labels, T, dev)
    nbytes = vocab_workspace_size(T, D, V)
    ws = _buffer(workspace, nbytes, dev, x.device, "moe_cross_entropy_forward")
    px, pw, pl = x.data_ptr(), W.data_ptr(), labels.data_ptr()
    if (px | pw | pl) & 15:
        return cross_entropy_forward(_aligned(x), _aligned(W), _aligned(labels), ws)
    loss = _empty(T, dtype=_F32, device=x.device)
    lse = _empty(T, dtype=_F32, device=x.device)
    st = lib.moe_cross_entropy_forward(px, pw, pl, kind, T, D, V, loss.data_ptr(), lse.data_ptr(), ws.data_ptr(),
                                       ws.numel(), _stream_of(x))
    if st:
        check(st, "moe_cross_entropy_forward")
    return dict(loss=loss, lse=lse)


def cross_entropy_backward(d_loss, x, W, labels, loss, lse, d_lse=None, workspace=None):
    """Gradients of sum(d_loss * loss) (+ sum(d_lse * lse), a penalty on log Z)
    for cross_entropy_forward: dict(dx [T, D], dW [V, D]) bf16.  d_loss, d_lse
    [T] fp32; loss, lse: the forward's.  The logits are computed again, by
    pieces of the vocabulary; their gradient is rounded to bf16 for the two
    products.  workspace: a uint8 CUDA tensor of vocab_workspace_size(...,
    backward=True) bytes.  A tensor that does not start on 16 bytes is copied
    first."""
    T, D, V, dev = _head(x, W)
    kind = _labels(labels, T, dev)
    for t, name in ((d_loss, "d_loss"), (loss, "loss"), (lse, "lse")):
        _like(t, name, _F32, (T,), dev)
    if d_lse is not None:
        _like(d_lse, "d_lse", _F32, (T,), dev)
    nbytes = vocab_workspace_size(T, D, V, backward=True)
    ws = _buffer(workspace, nbytes, dev, x.device, "moe_cross_entropy_backward")
    pd, px, pw, pl, po, ps = (t.data_ptr() for t in (d_loss, x, W, labels, loss, lse))
    pe = None if d_lse is None else d_lse.data_ptr()
    if (pd | px | pw | pl | po | ps | (pe or 0)) & 15:
        return cross_entropy_backward(*(_aligned(t) for t in (d_loss, x, W, labels, loss, lse, d_lse)), ws)
    dx, dW = torch.empty_like(x), torch.empty_like(W)
    st = lib.moe_cross_entropy_backward(pd, pe, px, pw, pl, kind, po, ps, T, D, V, dx.data_ptr(), dW.data_ptr(),
                                        ws.data_ptr(), ws.numel(), _stream_of(x))
    if st:
        check(st, "moe_cross_entropy_backward")
    return dict(dx=dx, dW=dW)


def _teacher(ids, logits, temperature, T, dev):
    ikind, lkind = _index_type(ids, "teacher_ids"), _float_type(logits, "teacher_logits")
    if ids.dim() != 2:
        raise ValueError(f"teacher_ids has shape {tuple(ids.shape)}, expected [{T}, K]")
    K = ids.shape[1]
    _in_32_bits("moe_teacher", K)
    _like(ids, "teacher_ids", ids.dtype, (T, K), dev)
    _like(logits, "teacher_logits", logits.dtype, (T, K), dev)
    return N.MoeTeacher(None, None, ikind, lkind, K, temperature)


def distill_forward(x, W, teacher_ids, teacher_logits, temperature=1.0, workspace=None):
    """Distillation of z = x W^T, which is never stored, from a teacher's top
    logits: with p the softmax of a token's teacher_logits / temperature among
    its K entries, dict(loss [T], lse [T], logits [T, K]) fp32, where lse = log
    sum exp(z / temperature), logits = z at the ids and loss = sum p (log p -
    logits / temperature + lse).  teacher_ids [T, K] int32 or int64 (an id
    outside [0, V) is no entry), teacher_logits [T, K] bf16 or fp32 (-inf is no
    entry), K up to 256; a token without entries has loss 0.  x, W, workspace as
    in cross_entropy_forward (vocab_workspace_size with n_teacher=K)."""
    T, D, V, dev = _head(x, W)
    te = _teacher(teacher_ids, teacher_logits, temperature, T, dev)
    nbytes = vocab_workspace_size(T, D, V, te.K)
    ws = _buffer(workspace, nbytes, dev, x.device, "moe_distill_forward")
    te.ids, te.logits = teacher_ids.data_ptr(), teacher_logits.data_ptr()
    px, pw = x.data_ptr(), W.data_ptr()
    if (px | pw | (te.ids or 0) | (te.logits or 0)) & 15:
        return distill_forward(*(_aligned(t) for t in (x, W, teacher_ids, teacher_logits)), temperature, ws)
    loss = _empty(T, dtype=_F32, device=x.device)
    lse = _empty(T, dtype=_F32, device=x.device)
    logits = _empty(T, te.K, dtype=_F32, device=x.device)
    st = lib.moe_distill_forward(px, pw, te, T, D, V, loss.data_ptr(), lse.data_ptr(), logits.data_ptr(),
                                 ws.data_ptr(), ws.numel(), _stream_of(x))
    if st:
        check(st, "moe_distill_forward")
    return dict(loss=loss, lse=lse, logits=logits)


def distill_backward(d_loss, x, W, teacher_ids, teacher_logits, lse, logits, temperature=1.0, workspace=None):
    """Gradients of sum(d_loss * loss) for distill_forward: dict(dx [T, D], dW
    [V, D]) bf16.  d_loss [T] fp32; lse, logits: the forward's; the rest as
    there and in cross_entropy_backward."""
    T, D, V, dev = _head(x, W)
    te = _teacher(teacher_ids, teacher_logits, temperature, T, dev)
    for t, name in ((d_loss, "d_loss"), (lse, "lse")):
        _like(t, name, _F32, (T,), dev)
    _like(logits, "logits", _F32, (T, te.K), dev)
    nbytes = vocab_workspace_size(T, D, V, te.K, backward=True)
    ws = _buffer(workspace, nbytes, dev, x.device, "moe_distill_backward")
    te.ids, te.logits = teacher_ids.data_ptr(), teacher_logits.data_ptr()
    pd, px, pw, ps, pz = (t.data_ptr() for t in (d_loss, x, W, lse, logits))
    if (pd | px | pw | ps | pz | (te.ids or 0) | (te.logits or 0)) & 15:
        return distill_backward(*(_aligned(t) for t in (d_loss, x, W, teacher_ids, teacher_logits, lse, logits)),
                                temperature, ws)
    dx, dW = torch.empty_like(x), torch.empty_like(W)
    st = lib.moe_distill_backward(pd, px, pw, te, ps, pz, T, D, V, dx.data_ptr(), dW.data_ptr(), ws.data_ptr(),
                                  ws.numel(), _stream_of(x))
    if st:
        check(st, "moe_distill_backward")
    return dict(dx=dx, dW=dW)


def device_error() -> int:
    return int(lib.moe_device_error())


def launch_count() -> int:
    return int(lib.moe_launch_count())
