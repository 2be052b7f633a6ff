"""The clipped policy loss from rows of logits against its plain float64 rows: every type, row stride and alignment,
clipped and unclipped ratios of either sign, each KL estimate, masks that leave a row nothing, infinities and NaN, rows
that carry nothing, the gradient in place and from saved values, streams, graphs, offsets past 2^31 elements."""
import numpy as np
import pytest

from logits_ref import EPS32, REL, grad_bound
from policy_ref import row_policy

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
NAMES = ("loss", "logprob", "entropy", "ratio", "kl", "d_logprob", "d_entropy")


@pytest.fixture(scope="module")
def ss():
    import fsdp_sharded_mixed_ss_gb300 as m
    return m


def _np(t):
    return t.detach().double().cpu().numpy()


def _logits(rows, vocab, dtype, *, pad=0, off=0, seed=0, sigma=2.5):
    """(rows, vocab) logits of row stride vocab + pad, `off` elements past an aligned address; NaN in the padding."""
    g = torch.Generator(device="cuda")
    g.manual_seed(1000 * seed + rows + 7 * vocab)
    ld = vocab + pad
    buf = torch.full((rows * ld + off + 8,), float("nan"), dtype=TYPES[dtype], device="cuda")
    x = buf[off:off + rows * ld].view(rows, ld)[:, :vocab]
    z = torch.randn((rows, vocab), generator=g, device="cuda") * sigma
    z[:, :: max(1, vocab // 13)] += 6.0
    x.copy_(z)
    return x


def _beside(x, pad, off, fill=9.0):
    rows, vocab = x.shape
    ld = vocab + pad
    buf = torch.full((rows * ld + off + 16,), fill, dtype=x.dtype, device="cuda")
    return buf, buf[off:off + rows * ld].view(rows, ld)[:, :vocab]


def _rows(x, scale, seed=0, idt=torch.int64):
    """Tokens, advantages of both signs, old and reference log probabilities whose ratios are on all sides of the
    borders (0.7, 0.8, 1.3, 3) and not near one."""
    rows, vocab = x.shape
    rng = np.random.default_rng(seed + rows)
    tok = rng.integers(0, vocab, rows)
    X = _np(x)
    z = np.nan_to_num(X, nan=0.0, posinf=0.0, neginf=-1e30) * scale
    top = z.max(axis=1, keepdims=True)
    lp = (z - top - np.log(np.exp(z - top).sum(axis=1, keepdims=True)))[np.arange(rows), tok]
    lp = np.maximum(lp, -1e4)
    gap = np.log(rng.choice([0.3, 0.75, 0.9, 1.0, 1.1, 1.25, 1.5, 2.5, 4.0], rows))
    f = lambda a: torch.tensor(a, dtype=torch.float32, device="cuda")  # noqa: E731
    w = rng.uniform(0.25, 2.0, rows)
    if rows > 2:
        w[rows // 2] = 0.0
    return dict(tokens=torch.tensor(tok, device="cuda").to(idt), advantage=f(rng.normal(size=rows)), old=f(lp - gap),
                ref=f(lp + rng.normal(size=rows) * 0.5), weight=f(w))


def _close(got, want, tol, what):
    with np.errstate(over="ignore"):
        want = np.asarray(want, dtype=np.float32).astype(np.float64)
    got = np.asarray(got, dtype=np.float64)
    assert np.array_equal(np.isnan(got), np.isnan(want)), (what, got, want)
    inf = np.isinf(want)
    assert np.array_equal(got[inf], want[inf]), (what, got, want)
    ok = np.isfinite(want)
    err, tol = np.abs(got[ok] - want[ok]), np.broadcast_to(tol, want.shape)[ok]
    assert (err <= tol).all(), (what, float(err.max()), float((err / tol).max()))


def _check(ss, x, r, *, dtype, scale=1.0, kind="k3", kc=0.05, ec=0.0, low=0.2, high=0.3, most=3.0, dpad=0, doff=0,
           old=True, ref=True, weight=True, inplace=True, stream=None):
    rows, vocab = x.shape
    out = {n: torch.full((rows,), 77.0, device="cuda") for n in NAMES if n != "kl" or ref}
    out["norm"] = torch.full((rows, 2), 77.0, device="cuda")
    buf, d = _beside(x, dpad, doff)
    kw = dict(old_logprob=r["old"] if old else None, ref_logprob=r["ref"] if ref else None,
              row_weight=r["weight"] if weight else None, clip_low=low, clip_high=high, clip_max=most,
              kl_kind={"k1": ss.SS_KL_K1, "k2": ss.SS_KL_K2, "k3": ss.SS_KL_K3}[kind], kl_coef=kc if ref else 0.0,
              entropy_coef=ec, scale=scale)
    if stream is not None:
        stream.wait_stream(torch.cuda.current_stream())
    ss.ss_policy_loss(x, r["tokens"], r["advantage"], d_logits=d, stream=stream, **kw, **out)
    torch.cuda.synchronize()
    f32 = lambda v: float(np.float32(v))  # noqa: E731
    one = np.float32(1)
    X, G = _np(x), _np(d)
    T, A = r["tokens"].tolist(), _np(r["advantage"])
    O, R, W = _np(r["old"]), _np(r["ref"]), _np(r["weight"])
    got = {n: _np(v) for n, v in out.items()}
    bounds = []
    for i in range(rows):
        o, b, g, gs = row_policy(X[i], f32(scale), T[i], A[i], old=O[i] if old else None, ref=R[i] if ref else None,
                                 weight=W[i] if weight else 1.0, low=float(one - (one - np.float32(low))),
                                 high=float((one + np.float32(high)) - one), most=f32(most), kind=kind,
                                 kc=f32(kc) if ref else 0.0, ec=f32(ec))
        for n in NAMES:
            if n in out:
                _close(got[n][i], o[n], b[n], (n, i))
        m, s = o["norm"]
        if not np.isnan(s):
            assert got["norm"][i, 0] == m
        _close(got["norm"][i, 1], s, REL * np.nan_to_num(s), ("norm", i))
        bound = grad_bound(g, gs, dtype) + b["flush"]
        _close(G[i], g, bound, ("gradient", i))
        bounds.append((g, bound))
    # a backward pass of its own from what the call wrote, and from the loss's call without a gradient
    alone = {n: torch.full_like(v, 55.0) for n, v in out.items()}
    ss.ss_policy_loss(x, r["tokens"], r["advantage"], **kw, **alone)
    e = torch.full_like(d, 3.0)
    ss.ss_token_logprobs_grad(x, alone["norm"], e, tokens=r["tokens"], d_logprob=alone["d_logprob"],
                              entropy=alone["entropy"], d_entropy=alone["d_entropy"], scale=scale)
    torch.cuda.synchronize()
    E = _np(e)
    for i in range(rows):
        _close(E[i], bounds[i][0], 2 * bounds[i][1], ("saved gradient", i))
    for n in out:
        assert torch.allclose(alone[n], out[n], rtol=4 * REL, atol=1e-30 + 8 * REL, equal_nan=True), n
    want = d.clone()
    d.fill_(9.0)
    assert bool((buf == 9.0).all()), "written outside the gradient"
    if inplace:
        off = x.data_ptr() % 16 // x.element_size()
        y = torch.zeros(off + (rows - 1) * x.stride(0) + vocab, dtype=x.dtype, device="cuda")
        y = y.as_strided(x.shape, x.stride(), off)
        y.copy_(x)
        again = {n: torch.full_like(v, 55.0) for n, v in out.items()}
        ss.ss_policy_loss(y, r["tokens"], r["advantage"], d_logits=y, **kw, **again)
        torch.cuda.synchronize()
        assert torch.equal(y.nan_to_num(7), want.nan_to_num(7))
    return out, want


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("rows,vocab,pad,off,dpad,doff", [
    (1, 1, 0, 0, 0, 0), (3, 2, 0, 0, 0, 0), (4, 9, 1, 1, 1, 1), (9, 31, 0, 0, 0, 0), (17, 1000, 0, 0, 0, 0),
    (3, 4099, 5, 2, 5, 2), (3, 4099, 5, 2, 0, 1), (6, 8192, 0, 0, 0, 0), (2, 50257, 47, 0, 47, 0),
    (200, 2053, 0, 0, 0, 0), (1, 128256, 0, 0, 0, 0), (5, 33001, 0, 3, 0, 3)])
def test_policy_sizes(ss, dtype, rows, vocab, pad, off, dpad, doff):
    for n, (kind, scale, ec, old, weight) in enumerate([("k3", 1.0, 0.0, True, True), ("k2", 0.7, 0.01, True, False),
                                                        ("k1", 1.25, 0.0, False, True)]):
        x = _logits(rows, vocab, dtype, pad=pad, off=off, seed=n)
        r = _rows(x, scale, seed=n, idt=torch.int32 if n == 1 else torch.int64)
        _check(ss, x, r, dtype=dtype, scale=scale, kind=kind, ec=ec, old=old, weight=weight, dpad=dpad, doff=doff)


@pytest.mark.parametrize("rows", [1, 2, 5, 20, 39, 77, 160, 320, 700])
def test_policy_row_counts(ss, rows):
    """Every way in which rows are shared out over the GPU."""
    x = _logits(rows, 20011, "bf16", pad=5, seed=2)
    _check(ss, x, _rows(x, 1.0), dtype="bf16", ec=0.02 if rows % 2 else 0.0, dpad=5)


def test_policy_long_rows(ss):
    """More columns than the blocks of a cluster take in parts of the usual size."""
    x = _logits(3, 600011, "bf16", pad=5, seed=2)
    _check(ss, x, _rows(x, 1.0), dtype="bf16", ec=0.02, weight=False)


@pytest.mark.parametrize("most", [0.0, 3.0])
def test_policy_optional_parts(ss, most):
    x = _logits(40, 777, "fp32")
    r = _rows(x, 1.0)
    for ref in (True, False):
        for ec in (0.0, -0.3):
            for kc in (0.0, -0.5):
                _check(ss, x, r, dtype="fp32", kc=kc, ec=ec, ref=ref, most=most, weight=False)
    out, _ = _check(ss, x, r, dtype="fp32", ec=0.1)
    for n in NAMES + ("norm",):
        o = torch.full_like(out[n], 5)
        ss.ss_policy_loss(x, r["tokens"], r["advantage"], old_logprob=r["old"], ref_logprob=r["ref"],
                          row_weight=r["weight"], clip_low=0.2, clip_high=0.3, clip_max=3.0, kl_coef=0.05,
                          entropy_coef=0.1, **{n: o})
        torch.cuda.synchronize()
        assert torch.allclose(o, out[n], rtol=4 * REL, atol=4 * REL), n


def test_policy_borders_are_inside(ss):
    """A ratio on a border counts as inside: 1 exactly, without an old policy, clipped to [1, 1]."""
    x = _logits(8, 500, "fp32")
    r = _rows(x, 1.0)
    _, d = _check(ss, x, r, dtype="fp32", low=0.0, high=0.0, most=0.0, old=False, ref=False, weight=False)
    assert bool((d != 0).any(dim=1).all())


def test_policy_all_clipped_rows_are_zero(ss):
    x = _logits(30, 3001, "bf16")
    r = _rows(x, 1.0)
    r["advantage"] = r["advantage"].abs() + 0.1
    r["old"] -= 3.0                                   # ratios of 6 and more
    out, d = _check(ss, x, r, dtype="bf16", ref=False)
    assert not d.any() and not out["d_logprob"].any() and bool((out["loss"] != 0).sum() == 29)


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("ec", [0.0, 0.05])
def test_policy_special_rows(ss, dtype, ec):
    vocab, inf = 1203, float("inf")
    lowest = torch.finfo(TYPES[dtype]).min
    x = _logits(16, vocab, dtype, pad=5, off=1)
    r = _rows(x, 1.0)
    tok = r["tokens"]
    x[0] = -inf                                       # nothing left
    x[1] = lowest                                     # nothing left, by the type's lowest value: uniform
    x[2, 7] = float("nan")
    x[3, 8] = inf
    x[4, 9] = float("nan")                            # NaN in a row that does not count
    r["weight"][:] = 1.0
    r["weight"][4] = 0.0
    x[5] = -inf
    x[5, 11:14] = torch.tensor([0.0, 1.0, -1.0], device="cuda").to(x.dtype)
    tok[5] = 12
    x[6, tok[6]] = -inf                               # the token itself is masked
    tok[7] = -1                                       # no token, and NaN
    x[7, 3] = float("nan")
    tok[8] = vocab                                    # past the vocabulary
    x[9] = 0.0
    x[10, ::2] = -inf
    tok[10] = 1
    x[11] = lowest
    x[11, tok[11]] = 3.0                              # the token has all the mass
    r["old"][12] = -inf                               # a ratio that is infinite
    r["advantage"][13] = 0.0
    x[14, 5] = float("nan")
    r["advantage"][14] = 0.0                          # NaN stays
    r["old"][0] = r["ref"][0] = -5.0
    for i in (1, 5, 9, 10, 11):
        r["old"][i] = r["ref"][i] = -1.5
    r["advantage"][12] = 0.5                          # clipped from above
    # k1 of a masked token is -inf, and so is its row's own term: it is left out of the rows with a KL term
    _check(ss, x, r, dtype=dtype, ec=ec, ref=False)
    keep = [i for i in range(16) if i not in (0, 6)]
    y = x[keep]
    _check(ss, y, {k: v[keep].contiguous() for k, v in r.items()}, dtype=dtype, ec=ec, kind="k3")


def test_policy_masked_token_with_kl(ss):
    """A masked token's KL term: +inf by the third estimate, -inf by the first; its gradient is
    finite with the first alone."""
    x = _logits(2, 300, "fp32")
    r = _rows(x, 1.0)
    r["weight"][:] = 1.0
    x[0, r["tokens"][0]] = -float("inf")
    x[1] = -float("inf")
    for kind, want in ((ss.SS_KL_K3, float("inf")), (ss.SS_KL_K1, -float("inf"))):
        loss, kl, d = torch.empty(2, device="cuda"), torch.empty(2, device="cuda"), torch.full_like(x, 3.0)
        ss.ss_policy_loss(x, r["tokens"], r["advantage"], loss, old_logprob=r["old"], ref_logprob=r["ref"], kl=kl,
                          kl_kind=kind, kl_coef=0.5, d_logits=d)
        torch.cuda.synchronize()
        assert kl.tolist() == [want, want] and loss.tolist() == [want, want]
        assert not d[1].any()                         # a masked-out row
        own = d[0, r["tokens"][0]].item()             # an infinite derivative times 1 - p, or a finite one
        assert np.isfinite(own) == (kind == ss.SS_KL_K1)


@pytest.mark.parametrize("offset", [0.0, 3e4, -2e6, 1e8])
def test_policy_far_from_zero(ss, offset):
    """fp32 logits far from zero, and fills and scales that take m c past 2^24."""
    x = _logits(20, 901, "fp32", sigma=8.0)
    x += offset
    r = _rows(x, 1.0)
    _check(ss, x, r, dtype="fp32", ec=0.03)
    x = _logits(12, 901, "fp32")
    x[:, 100:] = -1e10
    r = _rows(x, 40.0)
    r["tokens"] %= 100
    r["old"][:] = -2.0
    r["ref"][:] = -2.0
    X = _np(x)
    z = X * 40.0
    lp = z - z.max(axis=1, keepdims=True)
    lp = lp - np.log(np.exp(lp).sum(axis=1, keepdims=True))
    lp = lp[np.arange(12), r["tokens"].cpu().numpy()]
    r["old"] = torch.tensor(lp - 0.1, dtype=torch.float32, device="cuda")
    r["ref"] = torch.tensor(lp + 0.2, dtype=torch.float32, device="cuda")
    # |log p| reaches a few hundred: its rounding to old and ref's 32 bits is exact, and cancels
    _check(ss, x, r, dtype="fp32", scale=40.0, ec=0.03, kind="k1", kc=0.01)


def test_policy_grad_against_differences(ss):
    rows, vocab, h = 12, 700, 0.05
    x = _logits(rows, vocab, "fp32")
    r = _rows(x, 1.0)
    r["old"] = r["old"] * 0 + torch.tensor([-3.0], device="cuda")
    lp = torch.empty(rows, device="cuda")
    ss.ss_token_logprobs(x, r["tokens"], logprob=lp)
    r["old"] = lp + 0.02                              # ratios near 0.98: no border within the step
    g = torch.Generator(device="cuda")
    g.manual_seed(11)
    v = torch.randn(x.shape, generator=g, device="cuda")
    v /= v.abs().max()
    kw = dict(old_logprob=r["old"], ref_logprob=r["ref"], kl_coef=0.3, entropy_coef=0.1, clip_low=0.9, clip_high=9.0)
    plus, minus, loss, d = (*(torch.empty(rows, device="cuda") for _ in range(3)), torch.empty_like(x))
    ss.ss_policy_loss(x, r["tokens"], r["advantage"], loss, d_logits=d, **kw)
    ss.ss_policy_loss(x + h * v, r["tokens"], r["advantage"], plus, **kw)
    ss.ss_policy_loss(x - h * v, r["tokens"], r["advantage"], minus, **kw)
    slope = (_np(plus) - _np(minus)) / (2 * h)
    # two values of a few units with REL each, and the third derivative: at most 30 for ratios below 2 and
    # exp(-d) below 6 (|A| < 3: A ratio and its powers' sum, 27 of the direction's cube), over six
    size = 1.0 + float((r["advantage"].abs()).max()) + 0.3 * 6 + 0.1 * 7
    _close((_np(d) * _np(v)).sum(axis=1), slope, 2 * REL * size / h + h * h / 6 * 30, "slope")


def test_policy_streams_and_graph_replay(ss):
    x = _logits(37, 9001, "bf16")
    r = _rows(x, 1.0)
    want, wd = _check(ss, x, r, dtype="bf16", ec=0.01)
    st = torch.cuda.Stream()
    got, gd = _check(ss, x, r, dtype="bf16", ec=0.01, stream=st)
    assert torch.equal(gd, wd) and all(torch.equal(got[n], want[n]) for n in want)
    loss, d = torch.zeros(37, device="cuda"), torch.zeros_like(x)
    kw = dict(old_logprob=r["old"], ref_logprob=r["ref"], row_weight=r["weight"], clip_low=0.2, clip_high=0.3,
              clip_max=3.0, kl_coef=0.05, entropy_coef=0.01)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ss.ss_policy_loss(x, r["tokens"], r["advantage"], loss, d_logits=d, **kw)
    for _ in range(2):
        loss.zero_()
        d.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(loss, want["loss"]) and torch.equal(d, wd)


def test_policy_calls_right_behind_one_another(ss):
    """Logits written right before a call, their gradient over them read right after, without a wait in between."""
    x = _logits(90, 9001, "bf16")
    r = _rows(x, 1.0)
    kw = dict(old_logprob=r["old"], row_weight=r["weight"])
    want, loss = torch.empty_like(x), torch.empty(90, device="cuda")
    ss.ss_policy_loss(x, r["tokens"], r["advantage"], loss, d_logits=want, **kw)
    z, got = torch.empty((90, 9001), dtype=x.dtype, device="cuda"), []
    for _ in range(10):
        z.copy_(x)
        ss.ss_policy_loss(z, r["tokens"], r["advantage"], d_logits=z, **kw)
        got.append(z.clone())
        z.fill_(float("nan"))
    torch.cuda.synchronize()
    assert all(torch.equal(g, want) for g in got)


def test_policy_rows_past_2_31_elements(ss):
    """Row offsets past 2^31 elements (and bytes past 2^32): a row stride of 2^30 + 1."""
    ld, vocab, rows = (1 << 30) + 1, 5001, 4
    buf = torch.empty((rows - 1) * ld + vocab, dtype=torch.bfloat16, device="cuda")
    x = buf.as_strided((rows, vocab), (ld, 1))
    src = _logits(rows, vocab, "bf16")
    x.copy_(src)
    r = _rows(src, 1.0)
    r["weight"][:] = 1.0
    loss = torch.empty(rows, device="cuda")
    want, d = _check(ss, src, r, dtype="bf16")
    ss.ss_policy_loss(x, r["tokens"], r["advantage"], loss, old_logprob=r["old"], ref_logprob=r["ref"],
                      clip_low=0.2, clip_high=0.3, clip_max=3.0, kl_coef=0.05, d_logits=x)
    torch.cuda.synchronize()
    assert torch.allclose(loss, want["loss"], rtol=8 * REL, atol=8 * REL)
    # one rounding to bf16 of values within a few REL of one another: a step at most
    assert torch.allclose(x.float(), d.float(), rtol=2.0 ** -7, atol=6 * REL)
