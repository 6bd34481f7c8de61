"""The two ends of a language model around the MoE blocks, as they are measured.

Three operators with their gradients: the embedding lookup with scaling, the
softmax cross entropy of the unembedding product over a large vocabulary, and
the distillation of the same product from a teacher's top logits.  The last
two never keep the logits.  `run` computes them in elementary torch operations
in 32 bits, or through this package's entry points where `own` is true.

Tokens and widths are those of the package's workloads
(grouped_gemm_router_gb300/inputs.py): tiny T=256 D=128, gptoss_lite T=32768
D=768, wide T=16384 D=2048.  Vocabularies are generic: 2^13 to 2^17 entries,
and odd ones of about 5000 and 50000.
"""
import math

import torch

own = False

IGNORED = -100  # the label of a token that has no loss


def listed():
    return [
        # the token of each of a few sequences that are being decoded: latency
        dict(name="emb_fwd_few", op="emb_fwd", T=16, D=768, V=50001, table="bf16", out="bf16"),
        # the benchmark layer's batch into a bf16 residual stream
        dict(name="emb_fwd_block", op="emb_fwd", T=32768, D=768, V=50001, table="bf16", out="bf16"),
        # a short batch of odd width (no 16-byte rows), a small vocabulary
        dict(name="emb_bwd_odd", op="emb_bwd", T=1001, D=1005, V=5003, grad="bf16", add=False),
        # the benchmark layer's batch with a tied table: the head's gradient is added
        dict(name="emb_bwd_tied", op="emb_bwd", T=32768, D=768, V=50001, grad="bf16", add=True),
        # a wide model with an fp32 residual stream and a large vocabulary
        dict(name="emb_bwd_wide", op="emb_bwd", T=16384, D=2048, V=131072, grad="f32", add=False),
        # the loss of one short sequence: latency
        dict(name="ce_fwd_tiny", op="ce_fwd", T=256, D=128, V=8192),
        # the loss of the benchmark layer's batch (an evaluation pass)
        dict(name="ce_fwd_block", op="ce_fwd", T=32768, D=768, V=50001),
        # gradients of a short batch, nothing a multiple of a tile
        dict(name="ce_bwd_odd", op="ce_bwd", T=1001, D=192, V=5003, d_lse=False),
        # the training step's largest product, with the penalty on log Z
        dict(name="ce_bwd_block", op="ce_bwd", T=32768, D=768, V=50001, d_lse=True),
        # a wide model and a large vocabulary
        dict(name="ce_bwd_wide", op="ce_bwd", T=8192, D=2048, V=131072, d_lse=False),
        # few teacher entries, a small batch
        dict(name="distill_fwd_small", op="distill_fwd", T=2048, D=768, V=32768, K=8, tau=1.0),
        # a distillation step's gradients from 64 teacher entries a token
        dict(name="distill_bwd_block", op="distill_bwd", T=8192, D=768, V=50001, K=64, tau=2.0),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("emb_fwd", "emb_bwd", "ce_fwd", "ce_bwd", "distill_fwd", "distill_bwd"))
    V = _log(rng, 100, 200000)
    T = _log(rng, 1, 32768)
    if op.startswith("emb"):
        D = _log(rng, 32, 4096)
        D = D if rng.random() < 0.4 else -(-D // 64) * 64
        top = work(dict(op="emb_bwd", T=16384, D=2048, V=131072, grad="f32", add=False))["bytes"]
        pick = lambda: rng.choice(("bf16", "f32"))  # noqa: E731
        c = dict(op=op, T=T, D=D, V=V)
        c.update(dict(table=pick(), out=pick()) if op == "emb_fwd" else dict(grad=pick(), add=rng.random() < 0.4))
        # what a call that reads only some rows keeps is bounded too
        while max(work(c)["bytes"], 4 * c["V"] * D) > top:
            c["V"] = max(100, c["V"] // 2)
            c["T"] = max(1, c["T"] // 2)
        return c
    D = 64 * max(1, _log(rng, 64, 4096) // 64)
    top = work(dict(op="ce_bwd", T=8192, D=2048, V=131072, d_lse=False))["flops"]
    c = dict(op=op, T=T, D=D, V=V)
    if op == "ce_bwd":
        c["d_lse"] = rng.random() < 0.5
    if op.startswith("distill"):
        c.update(K=min(_log(rng, 1, 256), V), tau=rng.choice((0.5, 1.0, 2.0, 4.0)))
    while work(c)["flops"] > top:
        c["T"] = max(1, c["T"] // 2)
    return c


_TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def _rand(g, *shape):
    return torch.rand(*shape, generator=g, device="cuda")


def _tokens(g, n, V):
    """Tokens as text has them: frequency falls as one over the rank."""
    return (torch.exp(_rand(g, n) * math.log(V)).long() - 1).clamp(0, V - 1)


def _head(case, g):
    """Hidden states after the last norm, the table, and labels: the model
    knows some of them well (their logit stands out by up to twice ln V)."""
    T, D, V = case["T"], case["D"], case["V"]
    W = (_randn(g, V, D) / math.sqrt(D)).bfloat16()
    labels = _tokens(g, T, V)
    x = (_randn(g, T, D) + 2 * math.log(V) * _rand(g, T, 1) * W[labels].float()).bfloat16()
    return x, W, labels


def _rows(T, V):
    """Rows a chunk of which keeps a GB of 32-bit logits."""
    return max(1, min(T, (1 << 28) // V))


def prepare(case, seed):
    g = _gen(seed)
    op, T, D, V = case["op"], case["T"], case["D"], case["V"]
    s = dict(op=op, V=V)
    if op == "emb_fwd":
        s.update(ids=_tokens(g, T, V), table=(_randn(g, V, D) / math.sqrt(D)).to(_TYPES[case["table"]]),
                 scale=math.sqrt(D), out=_TYPES[case["out"]])
        return s
    if op == "emb_bwd":
        s.update(ids=_tokens(g, T, V), d_out=(1e-3 * _randn(g, T, D)).to(_TYPES[case["grad"]]), scale=math.sqrt(D))
        s["add"] = (1e-3 * _randn(g, V, D)).bfloat16() if case["add"] else None
        return s
    s["x"], s["W"], labels = _head(case, g)
    if op.startswith("ce"):
        s["labels"] = torch.where(_rand(g, T) < 0.05, IGNORED, labels)
        if op == "ce_fwd":
            return s
        parts = [_plain_ce_fwd(dict(s, x=s["x"][i:i + _rows(T, V)], labels=s["labels"][i:i + _rows(T, V)]))
                 for i in range(0, T, _rows(T, V))]
        s["loss"], s["lse"] = (torch.cat([p[n] for p in parts]) for n in ("loss", "lse"))
        n = max(1, int((s["labels"] >= 0).sum()))
        s["d_loss"] = (0.5 + _rand(g, T)) / n  # weights of the tokens, mean over them
        s["d_lse"] = 2e-4 * s["lse"] / n if case["d_lse"] else None
        return s
    K = case["K"]
    # the teacher: the student's product with noise on it, so that both agree on part of the entries
    near, ids = [], []
    for i in range(0, T, _rows(T, V)):
        z = (s["x"][i:i + _rows(T, V)] @ s["W"].t()).float()
        z += _randn(g, *z.shape)
        top = z.topk(K, dim=1)
        near.append(top.values)
        ids.append(top.indices)
    s.update(teacher_logits=torch.cat(near), teacher_ids=torch.cat(ids), tau=case["tau"])
    # a twentieth of the tokens are padding: no teacher entry
    s["teacher_ids"] = torch.where(_rand(g, T, 1) < 0.05, IGNORED, s["teacher_ids"])
    if op == "distill_fwd":
        return s
    parts = [_plain_distill_fwd(dict(s, **{n: s[n][i:i + _rows(T, V)] for n in ("x", "teacher_ids", "teacher_logits")}))
             for i in range(0, T, _rows(T, V))]
    s["lse"], s["logits"] = (torch.cat([p[n] for p in parts]) for n in ("lse", "logits"))
    s["d_loss"] = case["tau"] ** 2 * (0.5 + _rand(g, T)) / T
    return s


# ---------------------------------------------------------------------------
# The plain forms
# ---------------------------------------------------------------------------
def _known(ids, V):
    return (ids >= 0) & (ids < V)


def _plain_emb_fwd(s):
    rows = s["table"][s["ids"].clamp(0, s["V"] - 1)].float() * s["scale"]
    return torch.where(_known(s["ids"], s["V"])[:, None], rows, 0.0).to(s["out"])


def _plain_emb_bwd(s):
    d = s["d_out"].float() * s["scale"] * _known(s["ids"], s["V"])[:, None]
    out = torch.zeros(s["V"], d.shape[1], device=d.device) if s["add"] is None else s["add"].float()
    return out.index_add_(0, s["ids"].clamp(0, s["V"] - 1), d)


def _lse(z):
    m = z.amax(1, keepdim=True)
    return (m + torch.exp(z - m).sum(1, keepdim=True).log())[:, 0]


def _plain_ce_fwd(s):
    z = s["x"].float() @ s["W"].float().t()
    lse = _lse(z)
    at = z.gather(1, s["labels"].clamp(0, s["V"] - 1)[:, None])[:, 0]
    return dict(loss=torch.where(_known(s["labels"], s["V"]), lse - at, 0.0), lse=lse)


def _plain_ce_bwd(s):
    x, W = s["x"].float(), s["W"].float()
    known = _known(s["labels"], s["V"])
    d = torch.where(known, s["d_loss"], 0.0)
    p = torch.exp(x @ W.t() - s["lse"][:, None])
    p *= (d if s["d_lse"] is None else d + s["d_lse"])[:, None]
    p.scatter_add_(1, s["labels"].clamp(0, s["V"] - 1)[:, None], -d[:, None])
    return dict(dx=(p @ W).bfloat16(), dW=(p.t() @ x).bfloat16())


def _teacher(s):
    """(probabilities, their logarithms) of the teacher's entries; 0 where there is none."""
    t = torch.where(_known(s["teacher_ids"], s["V"]), s["teacher_logits"].float(), -math.inf) / s["tau"]
    m = t.amax(1, keepdim=True).clamp(min=torch.finfo(torch.float32).min)
    e = torch.exp(t - m)
    total = e.sum(1, keepdim=True)
    p = e / torch.where(total > 0, total, 1.0)
    return p, torch.where(p > 0, t - m - torch.where(total > 0, total, 1.0).log(), 0.0)


def _plain_distill_fwd(s):
    z = s["x"].float() @ s["W"].float().t()
    known = _known(s["teacher_ids"], s["V"])
    logits = torch.where(known, z.gather(1, s["teacher_ids"].clamp(0, s["V"] - 1)), 0.0)
    lse = _lse(z / s["tau"])
    p, log_p = _teacher(s)
    loss = (p * (log_p - (logits / s["tau"] - lse[:, None]))).sum(1)
    return dict(loss=loss, lse=lse, logits=logits)


def _plain_distill_bwd(s):
    x, W = s["x"].float(), s["W"].float()
    p, _ = _teacher(s)
    d = s["d_loss"] / s["tau"]
    q = torch.exp(x @ W.t() / s["tau"] - s["lse"][:, None])
    q *= (d * p.sum(1))[:, None]
    q.scatter_add_(1, s["teacher_ids"].clamp(0, s["V"] - 1), -d[:, None] * p)
    return dict(dx=(q @ W).bfloat16(), dW=(q.t() @ x).bfloat16())


def run(state):
    s, op = state, state["op"]
    if own:
        from grouped_gemm_router_gb300 import moe
        if op == "emb_fwd":
            return moe.embedding_forward(s["ids"], s["table"], scale=s["scale"], out_type=s["out"])
        if op == "emb_bwd":
            return moe.embedding_backward(s["d_out"], s["ids"], s["V"], scale=s["scale"], add=s["add"])
        if op == "ce_fwd":
            return moe.cross_entropy_forward(s["x"], s["W"], s["labels"])
        if op == "ce_bwd":
            return moe.cross_entropy_backward(s["d_loss"], s["x"], s["W"], s["labels"], s["loss"], s["lse"],
                                              d_lse=s["d_lse"])
        if op == "distill_fwd":
            return moe.distill_forward(s["x"], s["W"], s["teacher_ids"], s["teacher_logits"], temperature=s["tau"])
        return moe.distill_backward(s["d_loss"], s["x"], s["W"], s["teacher_ids"], s["teacher_logits"], s["lse"],
                                    s["logits"], temperature=s["tau"])
    return dict(emb_fwd=_plain_emb_fwd, emb_bwd=_plain_emb_bwd, ce_fwd=_plain_ce_fwd, ce_bwd=_plain_ce_bwd,
                distill_fwd=_plain_distill_fwd, distill_bwd=_plain_distill_bwd)[op](s)


# ---------------------------------------------------------------------------
# The definitions in 64 bits
# ---------------------------------------------------------------------------
def _soft_targets64(s):
    """Dense-row form of what a token is compared with: (indices, weights, 1 or 0 for the row)."""
    V = s["V"]
    if s["op"].startswith("ce"):
        ids = s["labels"].unsqueeze(1)
        w = ((ids >= 0) & (ids < V)).double()
        return ids, w
    ids = s["teacher_ids"]
    t = s["teacher_logits"].double() / s["tau"]
    t = t.masked_fill((ids < 0) | (ids >= V), -math.inf)
    return ids, torch.nan_to_num(torch.softmax(t, dim=1), nan=0.0)


def exact(case, seed):
    op, V = case["op"], case["V"]
    if work(case)["flops"] > 1.6e13:  # over 20 seconds in 64 bits
        return None
    s = prepare(case, seed)
    if op == "emb_fwd":
        return s["table"].index_select(0, s["ids"]).double().mul_(s["scale"])
    if op == "emb_bwd":
        order = torch.argsort(s["ids"], stable=True)
        tok, count = torch.unique_consecutive(s["ids"][order], return_counts=True)
        sums = torch.segment_reduce(s["d_out"].double()[order], "sum", lengths=count, axis=0, unsafe=True)
        out = torch.zeros(V, case["D"], dtype=torch.float64, device="cuda")
        out[tok] = sums * s["scale"]
        return out if s["add"] is None else out + s["add"].double()
    tau = s.get("tau", 1.0)
    W = s["W"].double()
    ids, w = _soft_targets64(s)
    got = []
    dW = torch.zeros_like(W)
    step = max(1, min(case["T"], (1 << 28) // V))
    for i in range(0, case["T"], step):
        at = slice(i, i + step)
        x, j, wj = s["x"][at].double(), ids[at], w[at]
        z = torch.mm(x, W.t()).div_(tau)
        if op.endswith("fwd"):
            lse = torch.logsumexp(z, 1)
            zj = torch.gather(z, 1, j.clamp(0, V - 1))
            cross = torch.special.xlogy(wj, wj).sum(1) + lse * wj.sum(1) - (wj * zj).sum(1)
            row = dict(loss=cross, lse=lse)
            if op == "distill_fwd":
                row["logits"] = (zj * tau).masked_fill((j < 0) | (j >= V), 0.0)
        else:
            g = s["d_loss"][at].double().unsqueeze(1) / tau
            dz = torch.softmax(z, 1) if op == "ce_bwd" else z.sub_(s["lse"][at].double().unsqueeze(1)).exp_()
            scale = g * wj.sum(1, keepdim=True)
            if op == "ce_bwd":
                if s["d_lse"] is not None:
                    scale = scale + s["d_lse"][at].double().unsqueeze(1)
            dz.mul_(scale).scatter_add_(1, j.clamp(0, V - 1), -g * wj)
            dW.addmm_(dz.t(), x)
            row = dict(dx=torch.mm(dz, W))
        got.append(row)
    out = {n: torch.cat([r[n] for r in got]) for n in got[0]}
    if op.endswith("bwd"):
        out["dW"] = dW
    return out


def _distinct(T, V):
    """About how many different tokens there are among T of _tokens: the
    frequent ones, each seen at least once, and the rare ones."""
    L = math.log(V)
    often = min(V, T / L)
    return max(1.0, min(T, V, often * (1 + math.log(V / often))))


def work(case):
    op, T, D, V = case["op"], case["T"], case["D"], case["V"]
    size = {"bf16": 2, "f32": 4}
    if op == "emb_fwd":
        return dict(bytes=int(_distinct(T, V)) * D * size[case["table"]] + T * D * size[case["out"]] + 8 * T, flops=T * D)
    if op == "emb_bwd":
        return dict(bytes=T * D * size[case["grad"]] + 8 * T + V * D * (4 + 2 * case["add"]), flops=2 * T * D)
    K = case.get("K", 0)
    io = T * D * 2 + V * D * 2 + (12 * T * K if K else 8 * T)  # hidden states, table, targets
    if op.endswith("fwd"):
        return dict(bytes=io + 8 * T + 4 * T * K, flops=2 * T * D * V)
    # the logits are not kept: their product again, then the two gradients
    return dict(bytes=io + 8 * T + 4 * T * K + T * D * 2 + V * D * 2, flops=6 * T * D * V)
