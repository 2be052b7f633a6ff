"""The operators on rows of logits against their plain float64 forms: every type, row stride and
alignment, masks that leave a row nothing, the type's lowest value, infinities and NaN, ties, lists of
every length, streams, graphs, offsets past 2^31 elements; gradients against the formula and against
differences of the forward calls."""
import numpy as np
import pytest

from logits_ref import EPS32, REL, grad_bound, row_distill, row_logprobs, row_logprobs_grad

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


@pytest.fixture(scope="module")
def ss():
    import fsdp_sharded_mixed_ss_gb300 as m
    return m


def _logits(rows, vocab, dtype, *, pad=0, off=0, seed=0, sigma=2.5):
    """(rows, vocab) logits with row stride vocab + pad, `off` elements past an aligned address, and their float64
    values. The padding columns hold NaN: nothing may read them."""
    g = torch.Generator(device="cuda")
    g.manual_seed(1000 * seed + rows + 7 * vocab)
    ld = vocab + pad
    buf = torch.full((rows * ld + off + 8,), float("nan"), dtype=TYPES[dtype], device="cuda")
    x = buf[off:off + rows * ld].view(rows, ld)[:, :vocab]
    z = torch.randn((rows, vocab), generator=g, device="cuda") * sigma
    z[:, :: max(1, vocab // 13)] += 6.0
    x.copy_(z)
    return x


def _same_layout(x):
    """A copy of x with its strides and 16-byte phase."""
    off = x.data_ptr() % 16 // x.element_size()
    buf = torch.zeros(off + (x.shape[0] - 1) * x.stride(0) + x.shape[1], dtype=x.dtype, device="cuda")
    y = buf.as_strided(x.shape, x.stride(), off)
    y.copy_(x)
    return y


def _np(t):
    return t.detach().double().cpu().numpy()


def _outputs(rows, k, idt=torch.int64):
    o = {n: torch.full((rows,), 77.0, device="cuda") for n in ("logprob", "entropy", "lse")}
    o["norm"] = torch.full((rows, 2), 77.0, device="cuda")
    if k:
        o["top_logprob"] = torch.full((rows, k), 77.0, device="cuda")
        o["top_id"] = torch.full((rows, k), -77, dtype=idt, device="cuda")
    return o


def _close(got, want, tol, what):
    with np.errstate(over="ignore"):  # what fp32 cannot hold is an infinity
        want = np.asarray(want, dtype=np.float32).astype(np.float64)
    got = np.asarray(got, dtype=np.float64)
    assert np.array_equal(np.isnan(got), np.isnan(want)), what
    inf = np.isinf(want)
    assert np.array_equal(got[inf], want[inf]), what
    ok = np.isfinite(want)
    err = np.abs(got[ok] - want[ok])
    tol = np.broadcast_to(tol, want.shape)[ok]
    bad = ~(err <= tol)
    assert not bad.any(), (what, float(err.max()), float((err / tol).max()))


def _check_logprobs(ss, x, tokens, k, scale=1.0, idt=torch.int64, stream=None):
    rows = x.shape[0]
    out = _outputs(rows, k, idt)
    if stream is not None:
        stream.wait_stream(torch.cuda.current_stream())
    ss.ss_token_logprobs(x, tokens, scale=scale, stream=stream, **out)
    torch.cuda.synchronize()
    X, T = _np(x), tokens.cpu().numpy()
    # the kernel's scale is fp32
    s32 = float(np.float32(scale))
    for r in range(rows):
        ref = row_logprobs(X[r], s32, int(T[r]), k)
        tol = REL + 2 * EPS32 * abs(ref["logprob"]) if np.isfinite(ref["logprob"]) else 1.0
        _close(out["logprob"][r].item(), ref["logprob"], tol, ("logprob", r))
        _close(out["entropy"][r].item(), ref["entropy"], 3 * REL * (1 + np.nan_to_num(ref["entropy"])), ("entropy", r))
        _close(out["lse"][r].item(), ref["lse"], REL + 2 * EPS32 * np.nan_to_num(abs(ref["lse"]), posinf=0), ("lse", r))
        m, s = ref["norm"]
        got = out["norm"][r].tolist()
        if not np.isnan(s):
            assert got[0] == m
        _close(got[1], s, REL * np.nan_to_num(s), ("norm", r))
        if k:
            assert out["top_id"][r].tolist() == ref["top_id"].tolist(), r
            lp = ref["top_logprob"]
            _close(_np(out["top_logprob"][r]), lp, REL + 2 * EPS32 * np.abs(np.where(np.isfinite(lp), lp, 0)), ("top", r))
    return out


SHAPES = [(1, 1), (3, 2), (2, 7), (5, 8), (4, 9), (3, 31), (2, 257), (17, 1000), (3, 4099), (6, 8192), (5, 50257),
          (1, 50257), (2, 128256), (333, 515)]


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("rows,vocab", SHAPES)
def test_logprobs_sizes(ss, rows, vocab, dtype):
    for k, pad, off, scale in [(0, 0, 0, 1.0), (1, 1, 3, 0.7), (20, 0, 1, 1.0 / 0.7), (128, 5, 0, 1.0)]:
        k = min(k, vocab)
        x = _logits(rows, vocab, dtype, pad=pad, off=off, seed=k)
        tok = torch.arange(rows, device="cuda") * 7919 % vocab
        idt = torch.int32 if k == 20 else torch.int64
        _check_logprobs(ss, x, tok.to(idt), k, scale, idt)


@pytest.mark.parametrize("rows", [1, 2, 19, 40, 77, 160, 320, 700])
def test_logprobs_row_counts(ss, rows):
    """Every way in which rows are shared out over the GPU."""
    x = _logits(rows, 20011, "bf16", pad=3, seed=5)
    tok = torch.arange(rows, device="cuda") * 131 % 20011
    _check_logprobs(ss, x, tok, 11)


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
def test_logprobs_special_rows(ss, dtype):
    lowest = torch.finfo(TYPES[dtype]).min
    big = torch.finfo(TYPES[dtype]).max
    vocab, k = 3001, 17
    x = _logits(14, vocab, dtype, pad=7, off=1)
    inf = float("inf")
    x[0] = -inf                          # nothing left
    x[1] = lowest                        # nothing left, by the type's lowest value: uniform
    x[2, 5:] = -inf                      # five tokens left, fewer than k
    x[3, :] = lowest
    x[3, 2999] = 1.5                     # one token left
    x[4, 17] = float("nan")
    x[5, 18] = inf
    x[6] = 0.0                           # all equal
    x[7] = torch.where(torch.arange(vocab, device="cuda") % 3 == 0, 0.0, -0.0).to(x.dtype)  # equal zeros
    x[8, ::2] = -inf
    x[9] = (torch.arange(vocab, device="cuda") % 5).to(x.dtype)  # many ties
    x[10] = big
    x[11] = lowest
    x[11, 7] = big
    x[12] = torch.linspace(-20, 20, vocab, device="cuda").to(x.dtype)   # ascending
    x[13] = torch.linspace(20, -20, vocab, device="cuda").to(x.dtype)   # descending
    tok = torch.tensor([3, 4, 9, 2999, 1, 2, 3000, 5, 0, 4, -1, 7, vocab, -100], device="cuda")
    _check_logprobs(ss, x, tok, k)
    _check_logprobs(ss, x, tok, 128)
    if dtype != "fp16":                  # fp16's range leaves room for it
        _check_logprobs(ss, x[:3], tok[:3], 1, 0.5)


@pytest.mark.parametrize("rows", [1, 9, 400])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_logprobs_ties_everywhere(ss, rows, dtype):
    """Rows that are all ties, or ties at the edge of the list, whatever the split of the row."""
    vocab = 50257
    x = torch.zeros((rows, vocab), dtype=TYPES[dtype], device="cuda")
    x[:, 40000:] = 1.0
    x[:, 50256] = 2.0
    x[rows // 2] = -3.0
    _check_logprobs(ss, x, torch.full((rows,), 40001, device="cuda"), 128)


@pytest.mark.parametrize("dtype,vocab,k", [("bf16", 33001, 128), ("fp16", 40007, 5), ("fp32", 16390, 64)])
def test_logprobs_many_rows(ss, dtype, vocab, k):
    """More rows than the GPU has places for, with rows among them that are masked, all ties or hold NaN."""
    rows = 1300
    x = _logits(rows, vocab, dtype, pad=3, seed=9)
    x[10] = -float("inf")
    x[11] = torch.finfo(TYPES[dtype]).min
    x[12, 7:] = -float("inf")
    x[13] = 0.0
    x[14, ::3] = -float("inf")
    x[15, 5] = float("nan")
    x[16] = (torch.arange(vocab, device="cuda") % 3).to(x.dtype)
    x[17] = torch.linspace(-9, 9, vocab, device="cuda").to(x.dtype)
    x[1299, : vocab // 2] = -float("inf")
    tok = torch.arange(rows, device="cuda") * 31 % vocab
    _check_logprobs(ss, x, tok, k)


def test_logprobs_optional_outputs(ss):
    x = _logits(6, 777, "bf16")
    tok = torch.arange(6, device="cuda")
    full = _check_logprobs(ss, x, tok, 9)
    for name in ("logprob", "entropy", "lse", "norm", "top_logprob", "top_id"):
        o = torch.full_like(full[name], 5)
        ss.ss_token_logprobs(x, tok if name in ("logprob", "top_id") else None, **{name: o})
        torch.cuda.synchronize()
        if name == "top_id":
            assert torch.equal(o, full[name])
        else:
            assert torch.allclose(o, full[name], rtol=2 * REL, atol=2 * REL), name


# ------------------------------------------------------------------ gradients

def _grad_buf(x, pad, off, fill=9.0):
    rows, vocab = x.shape
    ld = vocab + pad
    buf = torch.full((rows * ld + off + 16,), fill, dtype=x.dtype, device="cuda")
    return buf, buf[off:off + rows * ld].view(rows, ld)[:, :vocab]


def _untouched(buf, d, fill=9.0):
    d.fill_(fill)
    assert bool((buf == fill).all()), "written outside the gradient"


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("rows,vocab,pad,off,dpad,doff", [(1, 1, 0, 0, 0, 0), (3, 7, 0, 0, 0, 0), (4, 9, 1, 1, 1, 1),
                                                          (5, 1000, 0, 0, 3, 0), (3, 4099, 5, 2, 5, 2),
                                                          (3, 4099, 5, 2, 0, 1), (2, 50257, 47, 0, 47, 8),
                                                          (170, 2053, 0, 0, 0, 0), (700, 515, 1, 0, 1, 0),
                                                          (1, 128256, 0, 0, 0, 0)])
def test_logprobs_grad(ss, dtype, rows, vocab, pad, off, dpad, doff):
    k = min(8, vocab)
    scale = 0.7
    x = _logits(rows, vocab, dtype, pad=pad, off=off, seed=3)
    r = torch.arange(rows, device="cuda")
    tok = r * 7919 % vocab
    tok[rows // 2] = -1
    out = _outputs(rows, k)
    ss.ss_token_logprobs(x, tok, scale=scale, **out)
    g = torch.Generator(device="cuda")
    g.manual_seed(4)
    up = {n: torch.randn(rows, generator=g, device="cuda") for n in ("d_logprob", "d_entropy", "d_lse")}
    up["d_top_logprob"] = torch.randn((rows, k), generator=g, device="cuda")
    up["d_logprob"][rows // 2] = float("nan")        # unused: that row has no token
    buf, d = _grad_buf(x, dpad, doff)
    X, s32 = _np(x), float(np.float32(scale))
    sets = [("d_logprob",), ("d_entropy",), ("d_lse", "d_logprob"), ("d_top_logprob",), tuple(up)]
    for names in sets:
        ss.ss_token_logprobs_grad(x, out["norm"], d, tokens=tok, entropy=out["entropy"], top_id=out["top_id"],
                                  scale=scale, **{n: up[n] for n in names})
        torch.cuda.synchronize()
        got = _np(d)
        for i in range(rows):
            u = {n: float(up[n][i]) for n in names if n != "d_top_logprob"}
            if "d_top_logprob" in names:
                u["top_id"], u["d_top"] = out["top_id"][i].tolist(), up["d_top_logprob"][i].tolist()
            ref, size = row_logprobs_grad(X[i], s32, token=int(tok[i]) if "d_logprob" in names else None, **u)
            _close(got[i], ref, grad_bound(ref, size, dtype), (names, i))
    # in place: the same bits
    want = d.clone()
    ss.ss_token_logprobs_grad(x, out["norm"], x, tokens=tok, entropy=out["entropy"], top_id=out["top_id"], scale=scale,
                              **up)
    torch.cuda.synchronize()
    assert torch.equal(x, want)
    _untouched(buf, d)


def test_logprobs_grad_special_rows(ss):
    vocab = 1111
    x = _logits(9, vocab, "bf16", pad=1)
    inf = float("inf")
    x[0] = -inf
    x[1] = torch.finfo(torch.bfloat16).min
    x[2, 3:] = -inf
    x[3, 8] = float("nan")
    x[4, 9] = float("nan")                # with nothing flowing back: not read
    x[5, 9] = inf
    tok = torch.tensor([1, 2, 700, 0, 0, 1, vocab, 5, 6], device="cuda")
    out = _outputs(9, 0)
    ss.ss_token_logprobs(x, tok, **out)
    dl = torch.ones(9, device="cuda")
    dl[4] = 0.0
    dh = torch.full((9,), 0.5, device="cuda")
    dh[4] = 0.0
    buf, d = _grad_buf(x, 1, 0)
    ss.ss_token_logprobs_grad(x, out["norm"], d, tokens=tok, d_logprob=dl, entropy=out["entropy"], d_entropy=dh)
    torch.cuda.synchronize()
    X, got = _np(x), _np(d)
    for i in range(9):
        if i == 4:
            assert (got[i] == 0).all()
            continue
        ref, size = row_logprobs_grad(X[i], 1.0, token=int(tok[i]), d_logprob=1.0, d_entropy=0.5)
        _close(got[i], ref, grad_bound(ref, size, "bf16"), i)
    _untouched(buf, d)


def test_logprobs_grad_repeated_ids(ss):
    """The token among its own alternatives, and an id listed more than once: their gradients add up."""
    x = _logits(2, 600, "fp32")
    out = _outputs(2, 0)
    tok = torch.tensor([5, 7], device="cuda")
    ss.ss_token_logprobs(x, tok, **out)
    top = torch.tensor([[5, 9, 5, -1], [8, 8, 8, 7]], device="cuda")
    dt = torch.tensor([[1.0, 2.0, 3.0, float("nan")], [0.5, 0.25, -1.0, 2.0]], device="cuda")
    dl = torch.tensor([0.5, -0.25], device="cuda")
    d = torch.empty_like(x)
    ss.ss_token_logprobs_grad(x, out["norm"], d, tokens=tok, d_logprob=dl, top_id=top, d_top_logprob=dt)
    torch.cuda.synchronize()
    for i in range(2):
        ref, size = row_logprobs_grad(_np(x[i]), 1.0, token=int(tok[i]), d_logprob=float(dl[i]),
                                      top_id=top[i].tolist(), d_top=dt[i].tolist())
        _close(_np(d[i]), ref, grad_bound(ref, size, "fp32"), i)


def test_logprobs_grad_against_differences(ss):
    """Central differences of the forward outputs along random directions. The forward's error (REL) over 2h = 0.1,
    and h^2 / 6 of a third derivative that is below 10 for unit steps of these directions."""
    rows, vocab, k, h = 12, 911, 4, 0.05
    x = _logits(rows, vocab, "fp32")
    tok = torch.arange(rows, device="cuda") * 17 % vocab
    base = _outputs(rows, k)
    ss.ss_token_logprobs(x, tok, **base)
    g = torch.Generator(device="cuda")
    g.manual_seed(8)
    v = torch.randn(x.shape, generator=g, device="cuda")
    v /= v.abs().max()
    plus, minus = _outputs(rows, k), _outputs(rows, k)
    ss.ss_token_logprobs(x + h * v, tok, **plus)
    ss.ss_token_logprobs(x - h * v, tok, **minus)
    one = torch.ones(rows, device="cuda")
    tol = 2 * 3 * REL * (1 + float(base["entropy"].max())) / (2 * h) + h * h / 6 * 10
    for name, kw in [("logprob", dict(d_logprob=one)), ("entropy", dict(d_entropy=one)), ("lse", dict(d_lse=one))]:
        d = torch.empty_like(x)
        ss.ss_token_logprobs_grad(x, base["norm"], d, tokens=tok, entropy=base["entropy"], **kw)
        slope = (_np(plus[name]) - _np(minus[name])) / (2 * h)
        _close((_np(d) * _np(v)).sum(axis=1), slope, tol, name)


# ------------------------------------------------------------------ distillation

MODES = ["drop", "renorm", "bucket"]


def _tail(ss, mode):
    return {"drop": ss.SS_TAIL_DROP, "renorm": ss.SS_TAIL_RENORM, "bucket": ss.SS_TAIL_BUCKET}[mode]


def _teacher(x, k, scale, seed=0, noise=0.7, tdtype=torch.float32, idt=torch.int32):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    z = torch.nan_to_num(x.float(), nan=0.0, posinf=9.0, neginf=-30.0).clamp(-30, 30) * scale
    z = z + torch.randn(z.shape, generator=g, device="cuda") * noise
    v, i = torch.topk(z, k, dim=1)
    return i.to(idt), (v - torch.logsumexp(z, dim=1, keepdim=True)).to(tdtype)


def _check_distill(ss, x, ids, t, mode, *, scale=1.0, t_scale=1.0, weight=None, dtype="bf16", dpad=0, doff=0,
                   inplace=True):
    rows, vocab = x.shape
    loss = torch.full((rows,), 77.0, device="cuda")
    norm = torch.full((rows, 2), 77.0, device="cuda")
    tail = torch.full((rows,), 77.0, device="cuda")
    buf, d = _grad_buf(x, dpad, doff)
    kw = dict(row_weight=weight, tail=_tail(ss, mode), scale=scale, teacher_scale=t_scale)
    ss.ss_distill_topk(x, ids, t, loss, norm=norm, tail_logprob=tail, d_logits=d, **kw)
    torch.cuda.synchronize()
    X, I, T, G = _np(x), ids.cpu().numpy(), _np(t), _np(d)
    W = _np(weight) if weight is not None else np.ones(rows)
    s32, t32 = float(np.float32(scale)), float(np.float32(t_scale))
    L, P = _np(loss), _np(tail)
    bounds = []
    for r in range(rows):
        ref, lpt, g, gs, size = row_distill(X[r], s32, I[r], T[r], t32, mode, W[r])
        tol = 4 * REL * size + 1e-30
        _close(L[r], ref, tol, ("loss", mode, r))
        if not np.isnan(ref):
            _close(P[r], lpt, 2 * REL + 2 * EPS32 * np.nan_to_num(abs(lpt), posinf=0), ("tail", mode, r))
        bounds.append((g, gs, ref, tol))
        _close(G[r], g, grad_bound(g, gs, dtype), ("gradient", mode, r))
    # the loss alone
    only = torch.full((rows,), 77.0, device="cuda")
    ss.ss_distill_topk(x, ids, t, only, **kw)
    # the gradient from the saved normalisers, with an upstream gradient
    up = torch.linspace(0.5, 2.0, rows, device="cuda")
    e = torch.full_like(d, 3.0)
    ss.ss_distill_topk_grad(x, ids, t, norm, e, tail_logprob=tail, d_loss=up, **kw)
    torch.cuda.synchronize()
    E, U, O = _np(e), _np(up), _np(only)
    for r in range(rows):
        g, gs, ref, tol = bounds[r]
        _close(O[r], ref, tol, ("loss alone", mode, r))
        _close(E[r], U[r] * g, U[r] * grad_bound(g, 2 * gs, dtype) + 2.0 ** -24, ("saved gradient", mode, r))
    want = d.clone()
    _untouched(buf, d)
    if inplace:
        y = _same_layout(x)
        ss.ss_distill_topk(y, ids, t, loss, d_logits=y, **kw)
        torch.cuda.synchronize()
        assert torch.equal(y.nan_to_num(7), want.nan_to_num(7))
    return L, want


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("mode", MODES)
def test_distill_sizes(ss, dtype, mode):
    for rows, vocab, pad, off, dpad, doff, k, scale in [
            (1, 1, 0, 0, 0, 0, 1, 1.0), (3, 7, 0, 0, 0, 0, 5, 1.0), (4, 9, 1, 1, 1, 1, 9, 0.5),
            (17, 1000, 0, 0, 0, 0, 128, 1.0), (3, 4099, 5, 2, 5, 2, 16, 0.7), (3, 4099, 5, 2, 0, 1, 64, 1.0),
            (2, 50257, 47, 0, 47, 0, 32, 1.0), (200, 2053, 0, 0, 0, 0, 20, 1.0), (1, 128256, 0, 0, 0, 0, 64, 1.0),
            (5, 33001, 0, 3, 0, 3, 100, 1.0)]:
        x = _logits(rows, vocab, dtype, pad=pad, off=off, seed=k)
        idt = torch.int64 if k % 2 else torch.int32
        ids, t = _teacher(x, k, scale, seed=k, idt=idt)
        w = torch.linspace(0.25, 2.0, rows, device="cuda")
        w[rows // 2 if rows > 2 else 0] = 0.0 if rows > 2 else 1.0
        _check_distill(ss, x, ids, t, mode, scale=scale, weight=w, dtype=dtype, dpad=dpad, doff=doff)


@pytest.mark.parametrize("rows", [1, 2, 5, 20, 39, 77, 160, 500])
def test_distill_row_counts(ss, rows):
    x = _logits(rows, 20011, "bf16", pad=5, seed=2)
    ids, t = _teacher(x, 24, 1.0, seed=rows)
    _check_distill(ss, x, ids, t, "bucket", dpad=5)


@pytest.mark.parametrize("tdtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("mode", MODES)
def test_distill_teacher_types(ss, tdtype, mode):
    """A stored teacher in 16 bits (its mass may pass 1 by the rounding), at a temperature of its own."""
    x = _logits(6, 901, "fp32")
    ids, t = _teacher(x, 31, 1.0, tdtype=TYPES[tdtype])
    _check_distill(ss, x, ids, t, mode, dtype="fp32")
    if mode == "renorm":
        _check_distill(ss, x, ids, t + 5, mode, t_scale=0.5, dtype="fp32")


@pytest.mark.parametrize("mode", MODES)
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_distill_special_rows(ss, mode, dtype):
    vocab, k, inf = 1203, 12, float("inf")
    lowest = torch.finfo(TYPES[dtype]).min
    x = _logits(15, vocab, dtype, pad=5)
    ids, t = _teacher(x, k, 1.0, idt=torch.int64)
    w = torch.ones(15, device="cuda")
    x[0] = -inf                                       # nothing left of the student
    x[1] = lowest                                     # the same by the lowest value: uniform
    x[2, 7] = float("nan")
    x[3, 8] = inf
    x[4, 9] = float("nan")
    w[4] = 0.0                                        # NaN in a row that does not count
    x[5] = -inf
    x[5, ids[5]] = torch.arange(k, device="cuda").to(x.dtype)   # only the listed tokens are left
    x[6] = lowest
    x[6, ids[6]] = torch.arange(k, device="cuda").to(x.dtype)
    x[7, ids[7, 3]] = -inf                            # a listed token is masked, with mass: infinite loss
    x[8, ids[8, 2]] = -inf
    t[8, 2] = -inf                                    # a listed token is masked, without mass
    ids[9, 4:] = -1                                   # unused slots
    t[9, 4:] = float("nan")
    ids[10, :] = -5                                   # no slot used
    ids[11, 3] = vocab                                # past the vocabulary
    ids[12, 5] = ids[12, 1]                           # an id twice: the second one does not count
    ids[12, 7] = ids[12, 1]
    t[13] = -inf                                      # a teacher with no mass on its list
    t[14] = t[14] - torch.logsumexp(t[14], 0)         # all its mass on its list
    _check_distill(ss, x, ids, t, mode, weight=w, dtype=dtype, dpad=5)


def test_distill_small_tails_keep_their_digits(ss):
    """A student with 1e-6 of its mass off the list: p_t is a sum of its own terms, not 1 minus the listed mass."""
    vocab, k = 5000, 8
    x = torch.zeros((2, vocab), device="cuda")
    x += torch.linspace(-1, 1, vocab, device="cuda")
    x[:, 100:100 + k] += 22.0
    ids = torch.arange(100, 100 + k, device="cuda", dtype=torch.int32).repeat(2, 1)
    q = torch.full((2, k), 0.9 / k, device="cuda").log()
    L, _ = _check_distill(ss, x, ids, q, "bucket", dtype="fp32")
    tail = torch.empty(2, device="cuda")
    ss.ss_distill_topk(x, ids, q, tail_logprob=tail)
    want = [row_distill(_np(x[r]), 1.0, ids[r].tolist(), _np(q[r]), 1.0, "bucket", 1.0)[1] for r in range(2)]
    _close(_np(tail), np.array(want), 2 * REL, "tail")
    assert want[0] < -12


@pytest.mark.parametrize("mode", MODES)
def test_distill_grad_against_differences(ss, mode):
    rows, vocab, k, h = 10, 700, 9, 0.05
    x = _logits(rows, vocab, "fp32")
    ids, t = _teacher(x, k, 1.0)
    g = torch.Generator(device="cuda")
    g.manual_seed(11)
    v = torch.randn(x.shape, generator=g, device="cuda")
    v /= v.abs().max()
    plus, minus, loss = (torch.empty(rows, device="cuda") for _ in range(3))
    d = torch.empty_like(x)
    kw = dict(tail=_tail(ss, mode))
    ss.ss_distill_topk(x, ids, t, loss, d_logits=d, **kw)
    ss.ss_distill_topk(x + h * v, ids, t, plus, **kw)
    ss.ss_distill_topk(x - h * v, ids, t, minus, **kw)
    slope = (_np(plus) - _np(minus)) / (2 * h)
    size = max(row_distill(_np(x[r]), 1.0, ids[r].tolist(), _np(t[r]), 1.0, mode, 1.0)[4] for r in range(rows))
    _close((_np(d) * _np(v)).sum(axis=1), slope, 2 * 4 * REL * size / (2 * h) + h * h / 6 * 10, mode)


# ------------------------------------------------------------------ together, streams, graphs, size

def test_teacher_pass_feeds_the_student(ss):
    """The teacher's top alternatives are the student's list; a student equal to its teacher has no loss and, with
    the rest of the mass in the bucket, no gradient."""
    x = _logits(20, 5003, "fp32")
    tlp = torch.empty((20, 40), device="cuda")
    tid = torch.empty((20, 40), dtype=torch.int32, device="cuda")
    ss.ss_token_logprobs(x, top_logprob=tlp, top_id=tid)
    loss = torch.empty(20, device="cuda")
    d = torch.empty_like(x)
    ss.ss_distill_topk(x, tid, tlp, loss, d_logits=d)
    torch.cuda.synchronize()
    assert float(loss.abs().max()) <= 4 * REL * 8
    assert float(d.abs().max()) <= 4 * REL


def test_other_streams_and_graph_replay(ss):
    x = _logits(37, 9001, "bf16")
    ids, t = _teacher(x, 16, 1.0)
    tok = torch.arange(37, device="cuda")
    want = _check_logprobs(ss, x, tok, 16)
    wl = torch.empty(37, device="cuda")
    wd = torch.empty_like(x)
    ss.ss_distill_topk(x, ids, t, wl, d_logits=wd)
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    got = _check_logprobs(ss, x, tok, 16, stream=st)
    assert all(torch.equal(got[n], want[n]) for n in want)
    out = _outputs(37, 16)
    loss = torch.zeros(37, device="cuda")
    d = torch.zeros_like(x)
    e = torch.zeros_like(x)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ss.ss_token_logprobs(x, tok, **out)
        ss.ss_token_logprobs_grad(x, out["norm"], e, tokens=tok, d_logprob=wl)
        ss.ss_distill_topk(x, ids, t, loss, d_logits=d)
    for _ in range(2):
        for o in list(out.values()) + [loss, d, e]:
            o.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(out[n], want[n]) for n in want)
        assert torch.equal(loss, wl) and torch.equal(d, wd)
    f = torch.empty_like(x)
    ss.ss_token_logprobs_grad(x, want["norm"], f, tokens=tok, d_logprob=wl)
    torch.cuda.synchronize()
    assert torch.equal(e, f)


def test_results_do_not_change_from_call_to_call(ss):
    x = _logits(300, 30011, "bf16")
    ids, t = _teacher(x, 50, 1.0)
    tok = torch.arange(300, device="cuda")
    first = None
    for _ in range(4):
        out = _outputs(300, 50)
        loss, d = torch.empty(300, device="cuda"), torch.empty_like(x)
        ss.ss_token_logprobs(x, tok, **out)
        ss.ss_distill_topk(x, ids, t, loss, d_logits=d)
        torch.cuda.synchronize()
        got = list(out.values()) + [loss, d]
        first = first or got
        assert all(torch.equal(a, b) for a, b in zip(first, got))


def test_rows_past_2_31_elements(ss):
    """Row offsets past 2^31 elements (and bytes past 2^32): a row stride of 2^30 + 1."""
    ld, vocab, rows = (1 << 30) + 1, 5001, 4
    buf = torch.empty((rows - 1) * ld + vocab, dtype=torch.bfloat16, device="cuda")
    x = buf.as_strided((rows, vocab), (ld, 1))
    src = _logits(rows, vocab, "bf16")
    x.copy_(src)
    tok = torch.arange(rows, device="cuda")
    a, b = _outputs(rows, 9), _outputs(rows, 9)
    ss.ss_token_logprobs(x, tok, **a)
    ss.ss_token_logprobs(src, tok, **b)
    ids, t = _teacher(src, 9, 1.0)
    la, lb = torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda")
    d = torch.empty_like(src)
    ss.ss_distill_topk(src, ids, t, lb, d_logits=d)
    ss.ss_distill_topk(x, ids, t, la, d_logits=x)
    torch.cuda.synchronize()
    for n in ("logprob", "top_id"):
        assert torch.allclose(a[n].double(), b[n].double(), rtol=0, atol=2 * REL * 20)
    assert torch.allclose(la, lb, rtol=0, atol=8 * REL * 20)
    assert torch.allclose(x.float(), d.float(), rtol=2.0 ** -7, atol=6 * REL)
