"""The preference loss against its plain float64 form: pair counts and lengths from none to long, both layouts, each kind,
weights, rows outside the sequences, bad offsets, infinities and NaN; with the operators on rows of logits before and
behind it, on streams and in graphs."""
import numpy as np
import pytest

from logits_ref import REL, grad_bound, row_logprobs_grad, row_softmax
from preference_ref import preference

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def ss():
    import fsdp_sharded_mixed_ss_gb300 as m
    return m


def _np(t):
    return t.detach().double().cpu().numpy()


def _kind(ss, kind):
    return {"sigmoid": ss.SS_PREF_SIGMOID, "hinge": ss.SS_PREF_HINGE, "square": ss.SS_PREF_SQUARE}[kind]


def _batch(lengths, behind=3, before=2, seed=0, idt=torch.int64):
    rng = np.random.default_rng(seed)
    off = np.concatenate([[before], before + np.cumsum(lengths)])
    rows = int(off[-1]) + behind
    f = lambda a: torch.tensor(np.asarray(a), dtype=torch.float32, device="cuda")  # noqa: E731
    lp = -2 * rng.exponential(size=rows)
    w = rng.uniform(0.2, 2.0, rows)
    w[rng.random(rows) < 0.2] = 0.0
    return dict(lp=f(lp), ref=f(lp + 0.1 * rng.normal(size=rows)), w=f(w), off=torch.tensor(off, device="cuda").to(idt),
                pw=f(rng.uniform(0.3, 2.0, len(lengths) // 2)))


def _close(got, want, tol, what):
    with np.errstate(over="ignore"):
        want = np.asarray(want, dtype=np.float32).astype(np.float64)
    assert np.array_equal(np.isnan(got), np.isnan(want)), (what, got, want)
    inf = np.isinf(want)
    assert np.array_equal(got[inf], want[inf]), (what, got, want)
    ok = np.isfinite(want)
    err, tol = np.abs(got[ok] - want[ok]), np.broadcast_to(tol, want.shape)[ok]
    assert (err <= tol).all(), (what, float(err.max()), float((err / tol).max()))


def _check(ss, b, *, kind="sigmoid", beta=0.1, margin=0.0, smooth=0.0, average=False, halves=False, ref=True, weight=True,
           pair_weight=True, stream=None):
    rows, pairs = b["lp"].numel(), (b["off"].numel() - 1) // 2
    loss, reward = torch.full((pairs,), 77.0, device="cuda"), torch.full((pairs, 2), 77.0, device="cuda")
    d = torch.full((rows,), 55.0, device="cuda")
    kw = dict(ref_logprob=b["ref"] if ref else None, row_weight=b["w"] if weight else None,
              pair_weight=b["pw"] if pair_weight else None, kind=_kind(ss, kind), beta=beta, margin=margin,
              label_smoothing=smooth, average=average, halves=halves)
    if stream is not None:
        stream.wait_stream(torch.cuda.current_stream())
    ss.ss_preference_loss(b["lp"], b["off"], loss, reward=reward, d_logprob=d, stream=stream, **kw)
    torch.cuda.synchronize()
    f = lambda v: float(np.float32(v))  # noqa: E731
    o = preference(_np(b["lp"]), b["off"].tolist(), ref=_np(b["ref"]) if ref else None,
                   weight=_np(b["w"]) if weight else None, pair_weight=_np(b["pw"]) if pair_weight else None, kind=kind,
                   beta=f(beta), margin=f(margin), smooth=f(smooth), average=average, halves=halves)
    got = dict(loss=_np(loss), reward=_np(reward), d_logprob=_np(d))
    out = o["outside"]
    assert (got["d_logprob"][out] == 55.0).all(), "rows outside the sequences"
    _close(got["loss"], *o["loss"], "loss")
    _close(got["reward"], *o["reward"], "reward")
    _close(got["d_logprob"][~out], o["d_logprob"][0][~out], o["d_logprob"][1][~out], "gradient")
    alone = torch.empty_like(loss)
    ss.ss_preference_loss(b["lp"], b["off"], alone, **kw)
    torch.cuda.synchronize()
    assert torch.equal(alone.nan_to_num(7), loss.nan_to_num(7))
    return loss, d


LENGTHS = [[0, 0], [1, 0], [1, 1], [3, 5, 0, 2], [31, 33, 64, 1], [300, 7, 129, 600], [5000, 4000], [70000, 3],
           [200000, 150001, 0, 9], [17, 23] * 40, [100, 60] * 700]


@pytest.mark.parametrize("lengths", LENGTHS, ids=lambda v: f"{len(v)}x{max(v)}")
def test_preference_sizes(ss, lengths):
    for n, (kind, smooth, average, halves) in enumerate([("sigmoid", 0.0, False, False), ("sigmoid", 0.1, True, True),
                                                         ("square", 0.0, True, False), ("hinge", 0.0, True, True)]):
        b = _batch(lengths, seed=n, idt=torch.int32 if n % 2 else torch.int64)
        _check(ss, b, kind=kind, smooth=smooth, average=average, halves=halves, beta=0.1 if n == 0 else 1.0,
               margin=0.3 if n else 0.0, ref=n != 2, weight=n != 1, pair_weight=n != 3)


@pytest.mark.parametrize("pairs", [1, 2, 9, 40, 150, 310, 1300])
def test_preference_pair_counts(ss, pairs):
    """Every way in which pairs are shared out over the GPU, with lengths of their own."""
    rng = np.random.default_rng(pairs)
    for most in (40, 3000) if pairs > 100 else (40, 3000, 30000):
        _check(ss, _batch(rng.integers(0, most, 2 * pairs), seed=pairs))


def test_preference_long_sums_cancel(ss):
    """Half a million log ratios of nearly equal sums, without a reference: the difference keeps its digits."""
    b = _batch([500000, 500000], seed=3)
    b["lp"] = torch.round(b["lp"] * 4096) / 4096      # differences that float64 has exactly
    _check(ss, b, ref=False, weight=False, beta=1e-3)


@pytest.mark.parametrize("kind", ["sigmoid", "hinge", "square"])
def test_preference_special_values(ss, kind):
    inf, nan = float("inf"), float("nan")
    b = _batch([4, 3] * 9, before=0, behind=0)
    lp, w, pw = b["lp"], b["w"], b["pw"]
    w[:] = 1.0
    pw[:] = 1.0
    lp[0] = nan                                       # pair 0
    lp[7], w[7] = nan, 0.0                            # pair 1: not counted
    lp[14], pw[2] = nan, 0.0                          # pair 2: does not count
    lp[21] = -inf                                     # pair 3: chosen impossible
    lp[32] = -inf                                     # pair 4: rejected impossible
    lp[35] = lp[39] = -inf                            # pair 5: both, and no difference of them
    w[42:49] = 0.0                                    # pair 6: no weight at all
    lp[49] = 300.0                                    # pair 7: h far from 0
    lp[60] = 300.0                                    # pair 8
    for average in (False, True):
        _check(ss, b, kind=kind, beta=1.0, average=average)


def test_preference_bad_offsets(ss):
    """Offsets past the rows, negative or descending: NaN for their pairs, nothing else touched."""
    for off in ([0, 5, 3, 8, 12], [0, 5, 9, 12, 25], [-1, 5, 9, 12, 14], [0, 5, 9, 1 << 40, 12], [0, 2, 4, 4, -7]):
        b = _batch([5, 4, 3, 2], before=0, behind=6)
        b["off"] = torch.tensor(off, device="cuda")
        loss, _ = _check(ss, b)
        assert bool(loss.isnan().any())
        b["pw"][:] = 0.0
        loss, _ = _check(ss, b)
        assert not loss.any()


def test_preference_no_rows(ss):
    off = torch.zeros(7, dtype=torch.int32, device="cuda")
    lp = torch.empty(0, device="cuda")
    loss, d = torch.empty(3, device="cuda"), torch.empty(0, device="cuda")
    ss.ss_preference_loss(lp, off, loss, d_logprob=d, beta=1.0)
    ss.ss_preference_loss(lp, off, d_logprob=d, beta=1.0)
    torch.cuda.synchronize()
    assert np.allclose(loss.cpu().numpy(), np.log(2.0), rtol=1e-6)


@pytest.mark.parametrize("kind", ["sigmoid", "hinge", "square"])
def test_preference_grad_against_differences(ss, kind):
    b = _batch([9, 11, 30, 2, 0, 6], before=0, behind=0)
    loss, d = _check(ss, b, kind=kind, beta=0.5, margin=5.0)
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    v = torch.randn(d.shape, generator=g, device="cuda")
    h = 1.0 / 256
    plus, minus = torch.empty_like(loss), torch.empty_like(loss)
    kw = dict(ref_logprob=b["ref"], row_weight=b["w"], pair_weight=b["pw"], kind=_kind(ss, kind), beta=0.5, margin=5.0)
    ss.ss_preference_loss(b["lp"] + h * v, b["off"], plus, **kw)
    ss.ss_preference_loss(b["lp"] - h * v, b["off"], minus, **kw)
    off = b["off"].tolist()
    slope = (_np(plus) - _np(minus)) / (2 * h)
    got = np.array([(_np(d) * _np(v))[off[2 * i]:off[2 * i + 2]].sum() for i in range(3)])
    # the losses' own rounding over the step; lp + h v rounds to 2^-24 of |lp| < 20 a token; third derivatives: none but
    # the sigmoid's, 0.1 of the direction's cube (its sum over 32 tokens of weight < 2 is below 40) with beta, over six
    tol = 8 * 2.0 ** -23 * (np.abs(_np(loss)) + 1) / h + 32 * 2 * 20 * 2.0 ** -24 / h * np.abs(_np(d)).max() \
        + h * h * 0.1 * (0.5 * 40) ** 3 / 6
    assert (np.abs(got - slope) <= tol).all(), (got, slope, tol)


def test_preference_step_on_logits(ss):
    """As it is used: log probabilities of the tokens, the pairs' loss, the gradient to the logits; against float64."""
    vocab, lengths, beta = 503, [6, 4, 9, 11], 0.5
    off = torch.tensor(np.concatenate([[0], np.cumsum(lengths)]), device="cuda")
    rows = int(off[-1]) + 2
    g = torch.Generator(device="cuda")
    g.manual_seed(2)
    x = torch.randn((rows, vocab), generator=g, device="cuda") * 2
    tok = torch.randint(0, vocab, (rows,), generator=g, device="cuda")
    tok[3] = -1                                       # a position without a token
    f = lambda *s: torch.empty(*s, device="cuda")     # noqa: E731
    lp, norm, loss, d_lp, d = f(rows), f(rows, 2), f(2), torch.zeros(rows, device="cuda"), torch.empty_like(x)
    ref = -6 + torch.randn(rows, generator=g, device="cuda")
    ss.ss_token_logprobs(x, tok, logprob=lp, norm=norm)
    ss.ss_preference_loss(lp, off, loss, ref_logprob=ref, beta=beta, d_logprob=d_lp)
    ss.ss_token_logprobs_grad(x, norm, d, tokens=tok, d_logprob=d_lp)
    torch.cuda.synchronize()
    X, T = _np(x), tok.tolist()
    want = np.array([row_softmax(X[r], 1.0)[0][T[r]] if T[r] >= 0 else 0.0 for r in range(rows)])
    o = preference(want, off.tolist(), ref=_np(ref), beta=beta)
    # each log probability is within REL, so h within beta rows REL; slopes and curvatures are below 1
    _close(_np(loss), o["loss"][0], o["loss"][1] + beta * rows * REL, "loss")
    D = _np(d)
    for r in range(rows):
        up = 0.0 if o["outside"][r] else o["d_logprob"][0][r]
        grad, size = row_logprobs_grad(X[r], 1.0, token=T[r], d_logprob=up)
        more = beta * beta * rows * REL if up and T[r] >= 0 else 0.0
        _close(D[r], grad, grad_bound(grad, size, "fp32") + more, ("gradient", r))


def test_preference_streams_and_graph_replay(ss):
    b = _batch([900, 1300, 5, 2000] * 5)
    want, wd = _check(ss, b)
    loss, d = _check(ss, b, stream=torch.cuda.Stream())
    assert torch.equal(loss, want) and torch.equal(d, wd)
    loss, d = torch.zeros_like(want), torch.full_like(wd, 55.0)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ss.ss_preference_loss(b["lp"], b["off"], loss, ref_logprob=b["ref"], row_weight=b["w"], pair_weight=b["pw"],
                              d_logprob=d)
    for _ in range(2):
        loss.zero_()
        d.fill_(55.0)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(loss, want) and torch.equal(d, wd)
