"""The operators of a training step around the MoE layer, as they are measured.

Four operators: the layer norm in front of the MoE FFN (with the residual sum
it starts from), its backward pass, the Newton-Schulz orthogonalisation of
expert weight gradients, and the Muon update of stacks of expert weights that
is built on it.  `run` computes them in elementary torch operations in 32
bits, or through this package's entry points where `own` is true.

Sizes are those of the package's workloads (grouped_gemm_router_gb300/inputs.py):
tiny T=256 D=128 F=256 E=4, gptoss_lite T=32768 D=768 F=1536 E=8 top-2,
small_chunk T=2048 E=64 top-4, wide T=16384 D=2048 F=8192 E=16 top-2.
"""
import math

import torch

own = False

COEFFS = (3.4445, -4.7750, 2.0315)
STEPS = 5
NS_EPS = 1e-7
LN_EPS = 1e-5
LR, MOMENTUM, WEIGHT_DECAY = 0.02, 0.95, 0.01


def listed():
    return [
        # the norm before a small layer: a call bounded by its launch
        dict(name="ln_fwd_tiny", op="ln_fwd", T=256, D=128, stream="bf16", add=False, bias=True),
        # the block norm of the benchmark layer: residual sum, norm, both stored
        dict(name="ln_fwd_block", op="ln_fwd", T=32768, D=768, stream="bf16", add=True, bias=True),
        # a wide model that keeps its residual stream in fp32
        dict(name="ln_fwd_wide_f32", op="ln_fwd", T=16384, D=2048, stream="f32", add=True, bias=False),
        # a short batch of odd width (no 16-byte rows)
        dict(name="ln_bwd_odd", op="ln_bwd", T=1001, D=1005, stream="bf16", d_stream=False, bias=True),
        # the block norm's backward, with the residual path's gradient added
        dict(name="ln_bwd_block", op="ln_bwd", T=32768, D=768, stream="bf16", d_stream=True, bias=True),
        # the same for the wide fp32 stream
        dict(name="ln_bwd_wide_f32", op="ln_bwd", T=16384, D=2048, stream="f32", d_stream=True, bias=False),
        # one small stack of expert gradients: latency counts
        dict(name="ns_tiny", op="ns", B=4, rows=128, cols=256, tokens=128, grad="f32"),
        # W1's gradient of the benchmark layer
        dict(name="ns_experts", op="ns", B=8, rows=768, cols=1536, tokens=8192, grad="f32"),
        # tall, odd, bf16: no dimension is a multiple of a tile
        dict(name="ns_odd_tall", op="ns", B=3, rows=1001, cols=363, tokens=700, grad="bf16"),
        # the optimizer step of the benchmark layer: W1, W3 and W2 of 8 experts
        dict(name="muon_layer", op="muon", E=8, D=768, F=1536, tokens=8192, nesterov=True),
        # 64 experts of 128 tokens each: gradients of less than full rank
        dict(name="muon_many", op="muon", E=64, D=768, F=1536, tokens=128, nesterov=True),
        # few, large experts, F = 4 D
        dict(name="muon_wide", op="muon", E=4, D=2048, F=8192, tokens=2048, nesterov=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _size(rng, lo, hi):
    """A dimension: any, an odd multiple of 64, or a power of two."""
    v, kind = _log(rng, lo, hi), rng.randrange(3)
    return v if kind == 0 else v // 128 * 128 + 64 if kind == 1 else 1 << max(5, v.bit_length() - 1)


def draw(rng):
    op = rng.choice(("ln_fwd", "ln_bwd", "ns", "muon"))
    if op in ("ln_fwd", "ln_bwd"):
        D = min(8192, _size(rng, 48, 8192))
        T = min(_log(rng, 1, 32768), max(1, 16384 * 2048 // D))
        c = dict(op=op, T=T, D=D, stream=rng.choice(("bf16", "f32")), bias=rng.random() < 0.5)
        c["add" if op == "ln_fwd" else "d_stream"] = rng.random() < 0.5
        return c
    # the work of one matrix is bounded by the largest listed case's
    top = work(dict(op="muon", E=4, D=2048, F=8192))["flops"]
    rows, cols = _size(rng, 48, 4096), min(8192, _size(rng, 48, 8192))
    tokens = _log(rng, 16, 8192)
    one = work(dict(op="ns", B=1, rows=rows, cols=cols, grad="f32"))
    per = 3 if op == "muon" else 1
    most = int(min(64, top / one["flops"] / per, 1.2e9 / (12.0 * rows * cols * per)))
    while most < 1:
        rows, cols = rows // 2, cols // 2
        one = work(dict(op="ns", B=1, rows=rows, cols=cols, grad="f32"))
        most = int(min(64, top / one["flops"] / per, 1.2e9 / (12.0 * rows * cols * per)))
    B = _log(rng, 1, most)
    if op == "ns":
        return dict(op="ns", B=B, rows=rows, cols=cols, tokens=tokens, grad=rng.choice(("bf16", "f32")))
    return dict(op="muon", E=B, D=rows, F=cols, tokens=tokens, nesterov=rng.random() < 0.5)


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def _gradient(g, B, rows, cols, tokens):
    """Weight gradients as a layer makes them: inputs^T times output gradients
    over the tokens of an expert, features of unequal strength."""
    si = torch.exp(0.5 * _randn(g, B, rows, 1))
    so = torch.exp(0.5 * _randn(g, B, 1, cols)) * 1e-3
    return si * torch.bmm(_randn(g, B, rows, tokens), _randn(g, B, tokens, cols)) * (so / math.sqrt(tokens))


def prepare(case, seed):
    g = _gen(seed)
    op = case["op"]
    if op in ("ln_fwd", "ln_bwd"):
        T, D = case["T"], case["D"]
        dt = torch.bfloat16 if case["stream"] == "bf16" else torch.float32
        # a residual stream: features of unequal strength about a common offset
        x = (_randn(g, T, D) * torch.exp(0.5 * _randn(g, D)) + 0.3 * _randn(g, D)).to(dt)
        s = dict(op=op, x=x, weight=1 + 0.2 * _randn(g, D), bias=0.1 * _randn(g, D) if case["bias"] else None)
        if op == "ln_fwd":
            s["add"] = _randn(g, T, D).bfloat16() if case["add"] else None
            return s
        h = x.double()
        mean = h.mean(1, keepdim=True)
        s["mean"] = mean[:, 0].float()
        s["rstd"] = ((h - mean).square().mean(1) + LN_EPS).rsqrt().float()
        s["dy"] = (0.02 * _randn(g, T, D)).bfloat16()
        s["d_stream"] = (0.02 * _randn(g, T, D)).to(dt) if case["d_stream"] else None
        return s
    if op == "ns":
        grad = _gradient(g, case["B"], case["rows"], case["cols"], case["tokens"])
        return dict(op=op, g=grad.bfloat16() if case["grad"] == "bf16" else grad)
    E, D, F, t = case["E"], case["D"], case["F"], case["tokens"]
    shapes = ((E, D, F), (E, D, F), (E, F, D))
    return dict(op=op, nesterov=case["nesterov"],
                w=[(_randn(g, *s) / math.sqrt(s[1])).bfloat16() for s in shapes],
                g=[_gradient(g, *s, t) for s in shapes],
                m=[3 * _gradient(g, *s, 2 * t) for s in shapes])


# ---------------------------------------------------------------------------
# The plain forms
# ---------------------------------------------------------------------------
def _plain_ln_fwd(s):
    h = s["x"]
    if s["add"] is not None:
        h = (h.float() + s["add"].float()).to(h.dtype)
    f = h.float()
    mean = f.mean(1, keepdim=True)
    c = f - mean
    rstd = (c.square().mean(1, keepdim=True) + LN_EPS).rsqrt()
    y = c * rstd * s["weight"]
    if s["bias"] is not None:
        y = y + s["bias"]
    out = dict(y=y.bfloat16(), mean=mean[:, 0], rstd=rstd[:, 0])
    if s["add"] is not None:
        out["h"] = h
    return out


def _plain_ln_bwd(s):
    dy, rstd = s["dy"].float(), s["rstd"][:, None]
    xh = (s["x"].float() - s["mean"][:, None]) * rstd
    p = dy * s["weight"]
    dx = rstd * (p - p.mean(1, keepdim=True) - xh * (p * xh).mean(1, keepdim=True))
    if s["d_stream"] is not None:
        dx = dx + s["d_stream"].float()
    out = dict(dx=dx.to(s["x"].dtype), dweight=(dy * xh).sum(0))
    if s["bias"] is not None:
        out["dbias"] = dy.sum(0)
    return out


def _plain_ns(g):
    x = g.float()
    tall = x.shape[1] > x.shape[2]
    if tall:
        x = x.transpose(1, 2)
    x = x / (x.square().sum((1, 2), keepdim=True).sqrt() + NS_EPS)
    a, b, c = COEFFS
    for _ in range(STEPS):
        gram = x @ x.transpose(1, 2)
        x = a * x + (b * gram + c * (gram @ gram)) @ x
    return x.transpose(1, 2) if tall else x


def _plain_muon(s):
    for w, g, m in zip(s["w"], s["g"], s["m"]):
        m.mul_(MOMENTUM).add_(g)
        o = _plain_ns(g + MOMENTUM * m if s["nesterov"] else m)
        scale = 0.2 * math.sqrt(max(w.shape[1:]))
        w.copy_(w.float() * (1 - LR * WEIGHT_DECAY) - (LR * scale) * o)
    return dict(w=s["w"], m=s["m"])


def run(state):
    op = state["op"]
    if own:
        from grouped_gemm_router_gb300 import moe
        if op == "ln_fwd":
            return moe.layer_norm_forward(state["x"], state["weight"], bias=state["bias"], eps=LN_EPS, add=state["add"])
        if op == "ln_bwd":
            return moe.layer_norm_backward(state["dy"], state["x"], state["weight"], state["mean"], state["rstd"],
                                           bias=state["bias"] is not None, d_stream=state["d_stream"])
        if op == "ns":
            return moe.newton_schulz(state["g"], steps=STEPS, coefficients=COEFFS, eps=NS_EPS)
        moe.muon_step(state["w"], state["g"], state["m"], lr=LR, momentum=MOMENTUM, nesterov=state["nesterov"],
                      weight_decay=WEIGHT_DECAY, steps=STEPS, coefficients=COEFFS, eps=NS_EPS)
        return dict(w=state["w"], m=state["m"])
    if op == "ln_fwd":
        return _plain_ln_fwd(state)
    if op == "ln_bwd":
        return _plain_ln_bwd(state)
    if op == "ns":
        return _plain_ns(state["g"]).bfloat16().contiguous()
    return _plain_muon(state)


# ---------------------------------------------------------------------------
# The definitions in 64 bits
# ---------------------------------------------------------------------------
def _polar64(g):
    """The steps of Newton-Schulz on one matrix: the short side first, the
    even polynomial by Horner's rule."""
    x = g.double()
    flip = x.size(0) > x.size(1)
    x = x.t() if flip else x
    x = x / (torch.linalg.matrix_norm(x) + NS_EPS)
    eye = torch.eye(x.size(0), dtype=x.dtype, device=x.device)
    for _ in range(STEPS):
        q = torch.mm(x, x.t())
        x = torch.mm(COEFFS[0] * eye + torch.mm(q, COEFFS[1] * eye + COEFFS[2] * q), x)
    return x.t() if flip else x


def exact(case, seed):
    op = case["op"]
    s = prepare(case, seed)
    if op == "ln_fwd":
        h = s["x"]
        out = {}
        if s["add"] is not None:  # the stream is stored in its own type, and that is what is normalised
            h = (h.double() + s["add"].double()).to(h.dtype)
            out["h"] = s["x"].double() + s["add"].double()
        var, mean = torch.var_mean(h.double(), dim=1, correction=0)
        rstd = 1 / torch.sqrt(var + LN_EPS)
        y = torch.addcmul(s["bias"].double() if s["bias"] is not None else torch.zeros_like(mean[:1]),
                          (h.double() - mean[:, None]) / torch.sqrt(var + LN_EPS)[:, None], s["weight"].double())
        return dict(out, y=y, mean=mean, rstd=rstd)
    if op == "ln_bwd":
        D = case["D"]
        x, dy = s["x"].double(), s["dy"].double()
        mu, r = s["mean"].double().unsqueeze(1), s["rstd"].double().unsqueeze(1)
        n = (x - mu) * r
        gp = dy * s["weight"].double()
        dots = torch.einsum("td,td->t", gp, n).unsqueeze(1)
        dx = (gp * D - gp.sum(1, keepdim=True) - n * dots) * r / D
        if s["d_stream"] is not None:
            dx = dx + s["d_stream"].double()
        out = dict(dx=dx, dweight=torch.einsum("td,td->d", dy, n))
        if s["bias"] is not None:
            out["dbias"] = torch.einsum("td->d", dy)
        return out
    if work(case)["flops"] > 8e12:  # over 20 seconds in 64 bits
        return None
    if op == "ns":
        return torch.stack([_polar64(g) for g in s["g"]])
    ws, ms = [], []
    for w, g, m in zip(s["w"], s["g"], s["m"]):
        m1 = MOMENTUM * m.double() + g.double()
        u = MOMENTUM * m1 + g.double() if s["nesterov"] else m1
        step = LR * 0.2 * math.sqrt(max(w.shape[-1], w.shape[-2]))
        ws.append(torch.stack([(1 - LR * WEIGHT_DECAY) * w[e].double() - step * _polar64(u[e]) for e in range(w.size(0))]))
        ms.append(m1)
    return dict(w=ws, m=ms)


def work(case):
    op = case["op"]
    if op in ("ln_fwd", "ln_bwd"):
        T, D = case["T"], case["D"]
        e = 2 if case["stream"] == "bf16" else 4
        if op == "ln_fwd":  # x and y, the sum and what it adds, the two statistics
            per = e + 2 + (e + 2 if case["add"] else 0)
            return dict(bytes=T * D * per + 8 * T + 4 * D * (1 + case["bias"]), flops=8 * T * D)
        per = 2 + 2 * e + (e if case["d_stream"] else 0)
        return dict(bytes=T * D * per + 8 * T + 4 * D * (2 + case["bias"]), flops=14 * T * D)
    if op == "ns":
        count, rows, cols = case["B"], case["rows"], case["cols"]
        per = (2 if case["grad"] == "bf16" else 4) + 2
    else:  # gradient and momentum read, momentum written, weights read and written
        count, rows, cols, per = 3 * case["E"], case["D"], case["F"], 16
    m, n = min(rows, cols), max(rows, cols)
    # X X^T and its square are symmetric: half of each; then the product with X
    return dict(bytes=count * m * n * per, flops=count * STEPS * (m * (m + 1) * n + m * (m + 1) * m + 2 * m * m * n))
