"""Cross entropy and distillation over a vocabulary on the GPU against 64-bit
statements.

Tolerances.  With A the largest sum of |x w| over a row's products, a logit is
a sum of D exact products in fp32: off by less than 2^-20 A (D 2^-24 A at
worst, and the tensor cores' sums of up to 16 products are cut, not rounded).
lse is off by that, by the 2^-22 of ex2 and log2 and by 2^-24 of each of about
a thousand sums of positive terms: 2^-20 A + 2^-13 at worst, and 2^-22 of its
size; a loss adds the error of a logit.  A gradient of the logits, dz, is
rounded to bf16 (2^-8) and off by the error of exp(z - lse) (2^-13 covers it
for A up to 64); the products' fp32 sums add less than 2^-13, and the result is
rounded once more: |dx - ref| <= (2^-8 + 2^-12) |dz| |W| + 2^-8 |ref|, the same
for dW, and 2^-126 where bf16 has only subnormal numbers."""
import numpy as np
import pytest
import torch

import _lm_ref as ref

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def moe():
    from grouped_gemm_router_gb300 import build
    build.build()
    from grouped_gemm_router_gb300 import moe as m
    yield m
    assert m.device_error() == 0


def _np(t):
    return t.detach().double().cpu().numpy()


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _inputs(T, D, V, seed=0, size=1.0):
    g = _gen(seed + T + D + V)
    W = (size * torch.randn(V, D, generator=g, device="cuda") / D ** 0.5).bfloat16()
    labels = torch.randint(-1, V + 1, (T,), generator=g, device="cuda")
    known = labels.clamp(0, V - 1)
    x = (torch.randn(T, D, generator=g, device="cuda") + 8 * torch.rand(T, 1, generator=g, device="cuda") * W[known].float()).bfloat16()
    return g, x, W, labels


def _teacher(g, T, V, K):
    ids = torch.randint(-1, V + 1, (T, K), generator=g, device="cuda")
    logits = 3 * torch.randn(T, K, generator=g, device="cuda")
    logits[torch.rand(T, K, generator=g, device="cuda") < 0.1] = -float("inf")
    if T > 2:
        ids[1] = -1                                    # a token without entries
        logits[2] = -float("inf")
    if T > 4:
        ids[3] = V - 1                                 # the same id every time
        logits[4] = torch.finfo(F32).min
        ids[4, 0], logits[4, 0] = 0, 1.0               # masked by the type's lowest value
    return ids, logits


def _close(got, want, tol, what):
    bad = np.abs(_np(got) - want) - tol
    assert np.isfinite(_np(got)).all() and (bad <= 0).all(), f"{what}: {int((bad > 0).sum())} of {bad.size}, worst by {bad.max():.3e}"


def _size(x, W):
    return (np.abs(_np(x)) @ np.abs(_np(W)).T).max()


def _check_gradients(got, dz, x, W, what, off=0.0):
    """off [T, V]: what dz may be off by besides."""
    e = (2.0 ** -8 + 2.0 ** -12) * np.abs(dz) + off
    for name, want, size in (("dx", dz @ W, e @ np.abs(W)), ("dW", dz.T @ x, e.T @ np.abs(x))):
        assert got[name].dtype == BF
        _close(got[name], want, size + 2.0 ** -8 * np.abs(want) + 2.0 ** -126, f"{what} {name}")


def _check_ce(moe, x, W, labels, g, d_lse=True):
    T = len(x)
    f = moe.cross_entropy_forward(x, W, labels)
    xn, wn, y = _np(x), _np(W), labels.cpu().numpy()
    loss, lse = ref.cross_entropy(xn, wn, y)
    tol = 2.0 ** -20 * _size(x, W) + 2.0 ** -13 + 2.0 ** -22 * np.abs(lse)
    _close(f["lse"], lse, tol, "lse")
    _close(f["loss"], loss, 2 * tol, "loss")
    dl = torch.randn(T, generator=g, device="cuda") / T
    dl[labels < 0] = float("nan")                      # not read where there is no loss
    de = torch.randn(T, generator=g, device="cuda") / T if d_lse else None
    got = moe.cross_entropy_backward(dl, x, W, labels, f["loss"], f["lse"], d_lse=de)
    dz = ref.cross_entropy_dz(xn, wn, y, np.nan_to_num(_np(dl)), None if de is None else _np(de))
    _check_gradients(got, dz, xn, wn, f"T {T} D {x.shape[1]} V {len(W)}")
    again = moe.cross_entropy_backward(dl, x, W, labels, f["loss"], f["lse"], d_lse=de)
    assert all(torch.equal(got[n], again[n]) for n in got)  # the same bits every time
    return f, got


SHAPES = [(1, 64, 1), (1, 768, 5003), (2, 64, 2), (3, 128, 63), (31, 192, 64), (33, 64, 65), (64, 320, 100), (127, 64, 128),
          (129, 128, 255), (255, 64, 256), (256, 128, 257), (257, 192, 511), (300, 768, 1000), (40, 2048, 700), (520, 64, 4100),
          (1001, 192, 5003), (20, 8192, 300)]


def test_no_gradient_whatever_a_row_holds(moe):
    """Labels that are words, rows of infinities and NaN, no gradient."""
    _, x, W, labels = _inputs(300, 128, 700)
    labels = labels.clamp(0, 699)
    x[5], x[270] = float("inf"), float("nan")
    f = moe.cross_entropy_forward(x, W, labels)
    d = torch.ones(300, device="cuda")
    d[5] = d[270] = 0
    for de in (None, torch.zeros(300, device="cuda")):
        got = moe.cross_entropy_backward(d, x, W, labels, f["loss"], f["lse"], d_lse=de)
        assert torch.isfinite(got["dx"].float()).all() and not got["dx"][[5, 270]].any()
        assert got["dx"][[4, 6, 269, 271]].any(dim=1).all()


@pytest.mark.parametrize("T,D,V", SHAPES)
@pytest.mark.parametrize("index", [torch.int64, torch.int32], ids=["i64", "i32"])
def test_cross_entropy(moe, T, D, V, index):
    g, x, W, labels = _inputs(T, D, V)
    _check_ce(moe, x, W, labels.to(index), g, d_lse=index == torch.int64)


@pytest.mark.parametrize("T,D,V", [(2000, 64, 120), (3000, 128, 1), (5000, 64, 300)])
def test_cross_entropy_of_many_tokens_and_few_words(moe, T, D, V):
    """dW's reduction over the tokens is split."""
    g, x, W, labels = _inputs(T, D, V)
    _check_ce(moe, x, W, labels, g)


def test_every_column_can_be_the_label(moe):
    T = V = 1030
    g, x, W, _ = _inputs(T, 64, V)
    _check_ce(moe, x, W, torch.arange(V, device="cuda").flip(0).contiguous(), g)


def test_no_token_has_a_loss(moe):
    _, x, W, labels = _inputs(300, 128, 700)
    labels.fill_(-100)
    f = moe.cross_entropy_forward(x, W, labels)
    assert not f["loss"].any()
    nan = torch.full((300,), float("nan"), device="cuda")
    x[5] = float("inf")                                # whatever a token without a loss holds
    got = moe.cross_entropy_backward(nan, x, W, labels, f["loss"], f["lse"])
    assert not got["dx"].any() and torch.isfinite(got["dx"].float()).all()


def test_large_and_equal_logits(moe):
    """Logits of hundreds, one of them far above the rest (loss 0, gradient
    next to 0), and rows whose logits are all the same."""
    T, D, V = 64, 128, 3000
    g, x, W, labels = _inputs(T, D, V)
    labels = labels.clamp(0, V - 1)
    x[:32] = (64 * W[labels[:32]].float()).bfloat16()
    x[32:40] = 0
    f, got = _check_ce_only_forward(moe, x, W, labels)
    assert (f["lse"][32:40] - np.log(V)).abs().max() < 1e-5
    y = labels.cpu().numpy()
    dz = ref.cross_entropy_dz(_np(x), _np(W), y, np.ones(T))
    # 1 - q at the label is a difference from 1 for any 32-bit sum of the
    # exponentials: the label's own is 1, and the 1 is in up to 64 partial sums
    # (32 of a lane's chain, 3 of the chains, 3 of the runs, 8 of the warps, and
    # as many products), each rounded by 2^-24 of it: 2^-18
    off = np.zeros_like(dz)
    off[np.arange(T), y] = 2.0 ** -18
    _check_gradients(got, dz, _np(x), _np(W), "large", off)


def _check_ce_only_forward(moe, x, W, labels):
    f = moe.cross_entropy_forward(x, W, labels)
    loss, lse = ref.cross_entropy(_np(x), _np(W), labels.cpu().numpy())
    tol = 2.0 ** -20 * _size(x, W) + 2.0 ** -13 + 2.0 ** -22 * np.abs(lse)
    _close(f["lse"], lse, tol, "lse")
    _close(f["loss"], loss, 2 * tol, "loss")
    return f, moe.cross_entropy_backward(torch.ones(len(x), device="cuda"), x, W, labels, f["loss"], f["lse"])


def test_a_token_known_well_keeps_its_gradient(moe):
    """loss about 2^-12: q - 1 at the label is far below a rounding of 1."""
    D, V = 64, 512
    W = torch.zeros(V, D, dtype=BF, device="cuda")
    W[7, 0] = 1.0
    x = torch.zeros(2, D, dtype=BF, device="cuda")
    x[:, 0] = 14.5
    labels = torch.tensor([7, 7], device="cuda")
    f, got = _check_ce_only_forward(moe, x, W, labels)
    q = float(torch.sigmoid(torch.tensor(14.5 - np.log(V - 1), dtype=torch.float64)))
    want = (q - 1) * 1.0
    assert abs(float(got["dx"][0, 0]) / want - 1) < 2.0 ** -7
    assert abs(float(got["dW"][7, 0]) / (2 * want * 14.5) - 1) < 2.0 ** -7


def test_a_row_that_is_no_number_stays_alone(moe):
    _, x, W, labels = _inputs(300, 128, 700)
    labels = labels.clamp(0, 699)
    clean = moe.cross_entropy_forward(x, W, labels)
    x[37], x[260] = float("nan"), float("inf")
    f = moe.cross_entropy_forward(x, W, labels)
    keep = torch.ones(300, dtype=torch.bool, device="cuda")
    keep[[37, 260]] = False
    for n in ("loss", "lse"):
        assert torch.equal(f[n][keep], clean[n][keep]) and not torch.isfinite(f[n][~keep]).any()


@pytest.mark.parametrize("T,D,V,K", [(1, 64, 1, 1), (3, 64, 65, 2), (5, 768, 5003, 64), (70, 128, 300, 5), (130, 192, 100, 33),
                                     (257, 64, 257, 256), (300, 128, 5003, 100), (600, 320, 1000, 31), (40, 64, 20, 256),
                                     (1001, 64, 4100, 8)])
@pytest.mark.parametrize("tau,lt,index", [(1.0, F32, torch.int64), (2.5, BF, torch.int32), (0.5, F32, torch.int32)])
def test_distillation(moe, T, D, V, K, tau, lt, index):
    g, x, W, _ = _inputs(T, D, V, seed=K)
    ids, logits = _teacher(g, T, V, K)
    ids, logits = ids.to(index), logits.to(lt)
    f = moe.distill_forward(x, W, ids, logits, temperature=tau)
    xn, wn, i, lg = _np(x), _np(W), ids.cpu().numpy(), _np(logits)
    t32 = float(np.float32(tau))
    loss, lse, at = ref.distill(xn, wn, i, lg, t32)
    a = 2.0 ** -20 * _size(x, W)
    tol = a / tau + 2.0 ** -13 + 2.0 ** -22 * np.abs(lse)
    _close(f["lse"], lse, tol, "lse")
    _close(f["logits"], at, a, "logits")
    _close(f["loss"], loss, 2 * tol + 2.0 ** -18 * (1 + np.abs(np.where(np.isfinite(lg) & (lg > -1e30), lg, 0)).max() / tau), "loss")
    if T > 2:
        assert float(f["loss"][1]) == 0 and float(f["loss"][2]) == 0
    dl = torch.randn(T, generator=g, device="cuda") / T
    got = moe.distill_backward(dl, x, W, ids, logits, f["lse"], f["logits"], temperature=tau)
    _check_gradients(got, ref.distill_dz(xn, wn, i, lg, t32, _np(dl)), xn, wn, "distillation")
    if T > 2:
        assert not got["dx"][1].any() and not got["dx"][2].any()


@pytest.mark.parametrize("T,V,K", [(300, 20000, 251), (40, 30001, 256), (520, 5003, 100), (33, 9000, 38)])
def test_logits_of_many_entries(moe, T, V, K):
    """Every run of the vocabulary finds where a row's entries begin in it."""
    D = 64
    g, x, W, _ = _inputs(T, D, V)
    ids = torch.rand(T, V, generator=g, device="cuda").argsort(dim=1)[:, :K].contiguous()
    f = moe.distill_forward(x, W, ids, torch.randn(T, K, generator=g, device="cuda"))
    z = (x.double() @ W.double().t()).gather(1, ids)
    _close(f["logits"], _np(z), 2.0 ** -20 * _size(x, W), f"logits of {K}")


def test_teacher_ids_side_by_side(moe):
    """All entries in neighbouring columns, at the edges of tiles, halves and boxes."""
    T, D, V, K = 200, 64, 1200, 64
    g, x, W, _ = _inputs(T, D, V)
    ids = (torch.arange(T, device="cuda")[:, None] * 5 + torch.randperm(K, generator=g, device="cuda")[None]) % V
    logits = torch.randn(T, K, generator=g, device="cuda")
    f = moe.distill_forward(x, W, ids, logits)
    _, _, at = ref.distill(_np(x), _np(W), ids.cpu().numpy(), _np(logits), 1.0)
    _close(f["logits"], at, 2.0 ** -20 * _size(x, W), "logits")
    dl = torch.randn(T, generator=g, device="cuda")
    got = moe.distill_backward(dl, x, W, ids, logits, f["lse"], f["logits"])
    _check_gradients(got, ref.distill_dz(_np(x), _np(W), ids.cpu().numpy(), _np(logits), 1.0, _np(dl)), _np(x), _np(W), "side by side")


def test_one_teacher_entry_is_cross_entropy(moe):
    T, D, V = 700, 192, 3001
    g, x, W, labels = _inputs(T, D, V)
    c = moe.cross_entropy_forward(x, W, labels)
    d = moe.distill_forward(x, W, labels[:, None].contiguous(), torch.randn(T, 1, generator=g, device="cuda"))
    assert torch.equal(c["lse"], d["lse"]) and torch.equal(c["loss"], d["loss"])
    dl = torch.randn(T, generator=g, device="cuda")
    a = moe.cross_entropy_backward(dl, x, W, labels, c["loss"], c["lse"])
    b = moe.distill_backward(dl, x, W, labels[:, None].contiguous(), torch.zeros(T, 1, device="cuda"), d["lse"], d["logits"])
    for n in a:  # the label's value goes two ways: expm1(-loss) and exp(z - lse) - 1
        assert (a[n].float() - b[n].float()).norm() <= 2.0 ** -8 * a[n].float().norm()


def test_no_tokens(moe):
    x, W = torch.zeros(0, 64, dtype=BF, device="cuda"), torch.ones(70, 64, dtype=BF, device="cuda")
    e, i = torch.zeros(0, device="cuda"), torch.zeros(0, dtype=torch.int64, device="cuda")
    f = moe.cross_entropy_forward(x, W, i)
    assert f["loss"].shape == (0,) and f["lse"].shape == (0,)
    got = moe.cross_entropy_backward(e, x, W, i, e, e)
    assert got["dx"].shape == (0, 64) and not got["dW"].any()
    t = moe.distill_forward(x, W, i.view(0, 1), e.view(0, 1))
    assert t["logits"].shape == (0, 1)
    assert not moe.distill_backward(e, x, W, i.view(0, 1), e.view(0, 1), e, e.view(0, 1))["dW"].any()


def test_pieces_of_the_vocabulary(moe):
    """So many tokens that the gradient of the logits is held in two pieces,
    the last a shorter one.  Rows and columns are sampled; the sums run over all."""
    T, D, V = 1 << 18, 64, 8500
    g, x, W, labels = _inputs(T, D, V)
    f = moe.cross_entropy_forward(x, W, labels)
    dl = torch.rand(T, generator=g, device="cuda") / T
    got = moe.cross_entropy_backward(dl, x, W, labels, f["loss"], f["lse"])
    assert moe.vocab_workspace_size(T, D, V, backward=True) < 2 * T * V
    Wd = W.double()
    dW = torch.zeros(V, D, dtype=torch.float64, device="cuda")
    size = torch.zeros_like(dW)
    for i in range(0, T, 1 << 15):
        s = slice(i, i + (1 << 15))
        xd, y = x[s].double(), labels[s]
        z = xd @ Wd.t()
        lse = torch.logsumexp(z, 1)
        known = (y >= 0) & (y < V)
        assert (f["lse"][s].double() - lse).abs().max() < 2.0 ** -12
        loss = torch.where(known, lse - z.gather(1, y.clamp(0, V - 1)[:, None])[:, 0], 0.0)
        assert (f["loss"][s].double() - loss).abs().max() < 2.0 ** -11
        d = torch.where(known, dl[s].double(), 0.0)
        dz = (z - lse[:, None]).exp_().mul_(d[:, None])
        dz.scatter_add_(1, y.clamp(0, V - 1)[:, None], -d[:, None])
        dW += dz.t() @ xd
        size += dz.abs().t() @ xd.abs()
        want = dz @ Wd
        tol = (2.0 ** -8 + 2.0 ** -12) * (dz.abs() @ Wd.abs()) + 2.0 ** -8 * want.abs()
        assert ((got["dx"][s].double() - want).abs() <= tol).all()
    assert ((got["dW"].double() - dW).abs() <= (2.0 ** -8 + 2.0 ** -12) * size + 2.0 ** -8 * dW.abs()).all()


def test_distillation_over_pieces(moe):
    """Teacher entries in both pieces; one entry a token is cross entropy."""
    T, D, V = 1 << 18, 64, 8500
    g, x, W, labels = _inputs(T, D, V)
    other = torch.randint(0, V, (T, 1), generator=g, device="cuda")
    ids = torch.cat([labels.clamp(0, V - 1)[:, None], other], 1)
    logits = torch.tensor([0.0, -float("inf")], device="cuda").repeat(T, 1)
    f = moe.distill_forward(x, W, ids, logits)
    c = moe.cross_entropy_forward(x, W, ids[:, 0].contiguous())
    assert torch.equal(f["lse"], c["lse"]) and torch.equal(f["loss"], c["loss"])
    dl = torch.rand(T, generator=g, device="cuda") / T
    a = moe.distill_backward(dl, x, W, ids, logits, f["lse"], f["logits"])
    b = moe.cross_entropy_backward(dl, x, W, ids[:, 0].contiguous(), c["loss"], c["lse"])
    for n in a:  # an entry of -inf has p = 0: its dz is d q, as it was; the label's value goes two ways
        assert (a[n].float() - b[n].float()).norm() <= 2.0 ** -8 * a[n].float().norm()
    even = moe.distill_forward(x, W, ids, torch.zeros(T, 2, device="cuda"))
    got = moe.distill_backward(dl, x, W, ids, torch.zeros(T, 2, device="cuda"), even["lse"], even["logits"])
    rows = torch.arange(0, T, 997, device="cuda")
    z = x[rows].double() @ W.double().t()
    dz = torch.softmax(z, 1)
    dz.scatter_add_(1, ids[rows], torch.full((len(rows), 2), -0.5, dtype=torch.float64, device="cuda"))
    dz *= dl[rows].double()[:, None]
    want = dz @ W.double()
    tol = (2.0 ** -8 + 2.0 ** -12) * (dz.abs() @ W.double().abs()) + 2.0 ** -8 * want.abs()
    assert ((got["dx"][rows].double() - want).abs() <= tol).all()


def test_views_that_start_anywhere(moe):
    g, x, W, labels = _inputs(70, 64, 300)
    ids, logits = _teacher(g, 70, 300, 5)

    def view(t):
        buf = torch.full((t.numel() + 2,), 7, dtype=t.dtype, device="cuda")
        v = buf[1:-1].view(t.shape)
        v.copy_(t)
        assert v.data_ptr() % 16
        return v

    dl, de = torch.randn(70, generator=g, device="cuda"), torch.randn(70, generator=g, device="cuda")
    f = moe.cross_entropy_forward(x, W, labels)
    b = moe.cross_entropy_backward(dl, x, W, labels, f["loss"], f["lse"], d_lse=de)
    t = moe.distill_forward(x, W, ids, logits)
    tb = moe.distill_backward(dl, x, W, ids, logits, t["lse"], t["logits"])
    vx, vW, vl = view(x), view(W), view(labels)
    f2 = moe.cross_entropy_forward(vx, vW, vl)
    b2 = moe.cross_entropy_backward(view(dl), vx, vW, vl, view(f["loss"]), view(f["lse"]), d_lse=view(de))
    t2 = moe.distill_forward(vx, vW, view(ids), view(logits))
    tb2 = moe.distill_backward(view(dl), vx, vW, view(ids), view(logits), view(t["lse"]), view(t["logits"]))
    for p, q in ((f, f2), (b, b2), (t, t2), (tb, tb2)):
        assert p.keys() == q.keys() and all(torch.equal(p[n], q[n]) for n in p)


def test_captured_and_on_streams(moe):
    """A captured forward and backward replays on new contents with one
    workspace for all; streams with workspaces of their own do not meet."""
    T, D, V, K = 300, 128, 2000, 7
    sets = []
    for seed in range(3):
        g, x, W, labels = _inputs(T, D, V, seed=seed)
        sets.append((x, W, labels, *_teacher(g, T, V, K)))
    dl = torch.ones(T, device="cuda") / T
    nbytes = max(moe.vocab_workspace_size(T, D, V, k, backward=b) for k in (0, K) for b in (False, True))

    def step(x, W, labels, ids, logits, ws=None):
        f = moe.cross_entropy_forward(x, W, labels, workspace=ws)
        b = moe.cross_entropy_backward(dl, x, W, labels, f["loss"], f["lse"], workspace=ws)
        t = moe.distill_forward(x, W, ids, logits, workspace=ws)
        tb = moe.distill_backward(dl, x, W, ids, logits, t["lse"], t["logits"], workspace=ws)
        return [*f.values(), *b.values(), *t.values(), *tb.values()]

    want = [step(*s) for s in sets]
    held = [t.clone() for t in sets[0]]
    ws = torch.empty(nbytes, dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        step(*held, ws=ws)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            got = step(*held, ws=ws)
        for st, w in zip(sets, want):
            for h, t in zip(held, st):
                h.copy_(t)
            graph.replay()
            s.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(got, w))
    streams = [torch.cuda.Stream() for _ in sets]
    torch.cuda.synchronize()
    out = []
    for q, st in zip(streams, sets):
        with torch.cuda.stream(q):
            out.append([step(*st) for _ in range(3)])
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for os, w in zip(out, want) for o in os for a, b in zip(o, w))


def test_calls_from_several_host_threads(moe):
    from concurrent.futures import ThreadPoolExecutor
    _, x, W, labels = _inputs(300, 128, 2000)
    dl = torch.ones(300, device="cuda")
    f = moe.cross_entropy_forward(x, W, labels)
    want = moe.cross_entropy_backward(dl, x, W, labels, f["loss"], f["lse"])
    torch.cuda.synchronize()

    def work(_):
        with torch.cuda.stream(torch.cuda.Stream()):
            out = []
            for _ in range(5):
                a = moe.cross_entropy_forward(x, W, labels)
                out.append((a, moe.cross_entropy_backward(dl, x, W, labels, a["loss"], a["lse"])))
            torch.cuda.current_stream().synchronize()
        return all(torch.equal(a[n], f[n]) for a, _ in out for n in f) and all(torch.equal(b[n], want[n]) for _, b in out for n in b)

    with ThreadPoolExecutor(4) as pool:
        assert all(pool.map(work, range(8)))


def test_few_tokens_and_a_large_vocabulary(moe):
    """One row of tiles: dx's reduction is split, dW's tiles are many."""
    for T, D, V in ((1, 128, 40000), (8, 704, 30001), (130, 64, 70000)):
        g, x, W, labels = _inputs(T, D, V)
        _check_ce(moe, x, W, labels, g)
        ids, logits = _teacher(g, T, V, 40)
        f = moe.distill_forward(x, W, ids, logits, temperature=2.0)
        dl = torch.randn(T, generator=g, device="cuda")
        got = moe.distill_backward(dl, x, W, ids, logits, f["lse"], f["logits"], temperature=2.0)
        _check_gradients(got, ref.distill_dz(_np(x), _np(W), ids.cpu().numpy(), _np(logits), 2.0, _np(dl)), _np(x), _np(W),
                         f"distillation {T}")


def test_neighbours_stay_as_they_are(moe):
    """Outputs of odd sizes through the C ABI, with guards behind them."""
    from grouped_gemm_router_gb300 import _native as N
    T, D, V = 33, 64, 65
    g, x, W, labels = _inputs(T, D, V)
    f = moe.cross_entropy_forward(x, W, labels)
    dl = torch.ones(T, device="cuda")
    want = moe.cross_entropy_backward(dl, x, W, labels, f["loss"], f["lse"])
    dx = torch.full((T + 8, D), 7.0, dtype=BF, device="cuda")
    dW = torch.full((V + 8, D), 7.0, dtype=BF, device="cuda")
    out = torch.full((2, T + 7), 7.0, device="cuda")
    n = max(moe.vocab_workspace_size(T, D, V, backward=b) for b in (False, True))
    ws = torch.full((n + 256,), 7, dtype=torch.uint8, device="cuda")
    s = torch.cuda.current_stream().cuda_stream
    N.check(N.lib.moe_cross_entropy_backward(dl.data_ptr(), None, x.data_ptr(), W.data_ptr(), labels.data_ptr(), 1,
                                             f["loss"].data_ptr(), f["lse"].data_ptr(), T, D, V, dx.data_ptr(), dW.data_ptr(),
                                             ws.data_ptr(), n, s), "backward")
    assert torch.equal(dx[:T], want["dx"]) and torch.equal(dW[:V], want["dW"])
    assert (dx[T:] == 7).all() and (dW[V:] == 7).all() and (ws[n:] == 7).all()
    N.check(N.lib.moe_cross_entropy_forward(x.data_ptr(), W.data_ptr(), labels.data_ptr(), 1, T, D, V, out[0].data_ptr(),
                                            out[1].data_ptr(), ws.data_ptr(), n, s), "forward")
    assert torch.equal(out[0, :T], f["loss"]) and torch.equal(out[1, :T], f["lse"])
    assert (out[:, T:] == 7).all() and (ws[n:] == 7).all()
