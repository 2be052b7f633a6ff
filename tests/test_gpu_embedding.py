"""The embedding and its gradient against float64: types, widths, row strides and alignments, tokens that occur never, once,
in every position and across every boundary of the sums' parts, positions without a token, bases of each type and in place,
streams, graphs, offsets past 2^31 elements.

Bounds. A lookup is one product, rounded once. A sum of k rows of fp32 is within (k - 1) 2^-24 of its terms' absolute sum,
whatever its order; the scale and the base round once each, the result once more to its type."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
HALF = {"bf16": 2.0 ** -8, "fp16": 2.0 ** -11, "fp32": 2.0 ** -24}
TINY = {"bf16": 2.0 ** -133, "fp16": 2.0 ** -25, "fp32": 2.0 ** -126}


@pytest.fixture(scope="module")
def ss():
    import fsdp_sharded_mixed_ss_gb300 as m
    return m


def _rows(n, dim, dtype, *, pad=0, off=0, seed=0, fill=None):
    """(buffer, (n, dim) view of row stride dim + pad, `off` elements past an aligned address); NaN around the values, or
    `fill` everywhere."""
    g = torch.Generator(device="cuda")
    g.manual_seed(seed + n + 7 * dim)
    ld = dim + pad
    buf = torch.full((max(n, 1) * ld + off + 16,), float("nan") if fill is None else fill, dtype=TYPES[dtype],
                     device="cuda")
    x = buf[off:off + n * ld].view(n, ld)[:, :dim]
    if fill is None:
        x.copy_(torch.randn((n, dim), generator=g, device="cuda"))
    return buf, x


def _ids(n, vocab, how, seed=0, idt=torch.int64):
    rng = np.random.default_rng(seed + n)
    if how == "any":
        v = rng.integers(0, vocab, n)
    elif how == "few":                                # a handful of tokens, one of them half of all
        v = np.where(rng.random(n) < 0.5, vocab // 2, rng.integers(0, min(vocab, 5), n))
    elif how == "one":
        v = np.full(n, vocab - 1)
    elif how == "holes":                              # positions without a token, and past the table
        v = np.where(rng.random(n) < 0.3, rng.choice([-1, -100, vocab, vocab + 5, 2 ** 31 - 1], n),
                     rng.integers(0, vocab, n))
    else:
        v = np.full(n, -1)
    return torch.tensor(v, device="cuda").to(idt)


def _f64(t):
    return t.detach().double()


def _bound(want, size, count, dtype):
    """For sums of `count` rows whose terms' absolute values add to `size`."""
    return size * (count + 2) * 2.0 ** -24 + want.abs() * HALF[dtype] * (1 + 2.0 ** -8) + TINY[dtype]


# ------------------------------------------------------------------ lookup

@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("odtype", ["bf16", "fp16", "fp32"])
def test_lookup(ss, dtype, odtype):
    for n, vocab, dim, pad, off, opad, ooff, scale, idt in [
            (1, 1, 1, 0, 0, 0, 0, 1.0, torch.int64), (5, 9, 7, 0, 1, 0, 3, 0.5, torch.int32),
            (33, 100, 64, 0, 0, 0, 0, 1.0, torch.int32), (17, 50, 768, 8, 0, 16, 0, 8.0, torch.int64),
            (9, 30, 1000, 24, 0, 0, 0, 1.0, torch.int64), (40, 11, 1025, 0, 0, 3, 1, 0.3, torch.int32),
            (300, 2000, 1001, 7, 0, 7, 0, 1.0, torch.int64), (3, 5, 8192, 0, 0, 0, 0, 64.0, torch.int64)]:
        _, t = _rows(vocab, dim, dtype, pad=pad, off=off)
        buf, out = _rows(n, dim, odtype, pad=opad, off=ooff, fill=9.0)
        ids = _ids(n, vocab, "holes" if n > 4 else "any", idt=idt)
        ss.ss_embedding(t, ids, out, scale=scale)
        torch.cuda.synchronize()
        k = ids.long()
        there = ((k >= 0) & (k < vocab))[:, None]
        s32 = float(np.float32(scale))
        want = torch.where(there, _f64(t)[k.clamp(0, vocab - 1)] * s32,
                           torch.where(k[:, None] < 0, 0.0, float("nan")).double())
        got = _f64(out)
        assert torch.equal(got.isnan(), want.isnan())
        err = (got - want).abs().nan_to_num(0.0)
        # the product to fp32, then to the type
        lim = want.abs().nan_to_num(0.0) * (HALF[odtype] * (1 + 2.0 ** -8) + 2.0 ** -24) + TINY[odtype]
        assert bool((err <= lim).all())
        if scale == 1.0 and dtype == odtype:
            assert bool((err == 0).all())
        out.fill_(9.0)
        assert bool((buf == 9.0).all()), "written outside the rows"


def test_lookup_keeps_infinities_and_shapes(ss):
    t = torch.randn((20, 16), device="cuda").to(torch.bfloat16)
    t[3, 2], t[4, 5] = float("inf"), float("nan")
    ids = torch.tensor([[3, 4, 0], [1, 3, -1]], device="cuda")
    out = torch.empty((2, 3, 16), dtype=torch.bfloat16, device="cuda")
    ss.ss_embedding(t, ids, out)
    torch.cuda.synchronize()
    want = t[ids.clamp_min(0)]
    want[1, 2] = 0
    assert torch.equal(out.nan_to_num(5), want.nan_to_num(5)) and bool(out[0, 1, 5].isnan())


def test_lookup_past_2_31_elements(ss):
    """Rows past 2^31 elements of a table and of the output, by their strides."""
    ld = (1 << 30) + 8
    buf = torch.zeros(3 * ld + 64, dtype=torch.bfloat16, device="cuda")
    t = buf.as_strided((4, 64), (ld, 1))
    t.copy_(torch.randn((4, 64), device="cuda"))
    obuf = torch.zeros(3 * ld + 64, dtype=torch.bfloat16, device="cuda")
    out = obuf.as_strided((4, 64), (ld, 1))
    ss.ss_embedding(t, torch.tensor([3, 1, 0, 3], device="cuda"), out)
    torch.cuda.synchronize()
    assert torch.equal(out, t[[3, 1, 0, 3]])


# ------------------------------------------------------------------ gradient

def _workspace(ss, n, vocab, dim):
    b = ss.ss_embedding_grad_workspace(n, vocab, dim)
    return torch.full((b + 64,), 0xAB, dtype=torch.uint8, device="cuda")


def _check(ss, d, ids, vocab, *, dtype="bf16", base=None, pad=0, off=0, scale=1.0, in_place=False, stream=None):
    n, dim = d.shape
    buf, t = _rows(vocab, dim, dtype, pad=pad, off=off, fill=9.0)
    b = None
    if in_place:
        t.copy_(base)
        b = t
    elif base is not None:
        b = base
    base = None if base is None else _f64(base).clone()
    ws = _workspace(ss, n, vocab, dim)
    need = ws.numel() - 64
    if stream is not None:
        stream.wait_stream(torch.cuda.current_stream())
    ss.ss_embedding_grad(d, ids, t, ws[:need], base=b, scale=scale, stream=stream)
    torch.cuda.synchronize()
    assert bool((ws[need:] == 0xAB).all()), "written past the workspace"
    k = ids.long().view(-1)
    live = torch.nonzero((k >= 0) & (k < vocab))[:, 0]
    want = torch.zeros((vocab, dim), dtype=torch.float64, device="cuda")
    size = torch.zeros_like(want)
    s32 = float(np.float32(scale))
    want.index_add_(0, k[live], _f64(d)[live] * s32)
    size.index_add_(0, k[live], _f64(d)[live].abs() * abs(s32))
    count = torch.zeros(vocab, dtype=torch.float64, device="cuda").index_add_(
        0, k[live], torch.ones(live.numel(), dtype=torch.float64, device="cuda"))[:, None]
    if base is not None:
        want += base
        size += base.abs()
    got = _f64(t)
    assert torch.equal(got.isnan(), want.isnan())
    ok = torch.isfinite(want)
    assert torch.equal(got[~ok].nan_to_num(7), want[~ok].nan_to_num(7))
    over = ((got - want).abs() > _bound(want, size, count, dtype)) & ok
    assert not over.any(), (int(over.sum()), float((got - want)[ok].abs().max()))
    if base is not None and in_place:
        never = torch.ones(vocab, dtype=torch.bool, device="cuda")
        never[k[live]] = False
        assert torch.equal(got[never], base[never])
    result = t.clone()
    t.fill_(9.0)
    assert bool((buf == 9.0).all()), "written outside the table"
    return result


HOW = ["any", "few", "one", "holes", "none"]


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("how", HOW)
def test_grad_sizes(ss, dtype, how):
    for n, vocab, dim, dpad, doff, pad, off, odt in [
            (1, 1, 1, 0, 0, 0, 0, "fp32"), (2, 3, 5, 0, 0, 0, 0, "bf16"), (31, 7, 8, 0, 0, 0, 0, "fp16"),
            (32, 40, 64, 8, 0, 8, 0, "bf16"), (33, 40, 768, 0, 0, 0, 0, "fp16"), (64, 513, 1000, 0, 0, 24, 0, "bf16"),
            (65, 511, 1001, 3, 1, 0, 3, "fp32"), (97, 512, 1032, 0, 0, 0, 0, "fp32"), (500, 1000, 130, 6, 0, 0, 5, "bf16"),
            (1500, 50257, 40, 0, 0, 0, 0, "bf16"), (2048, 60, 264, 0, 0, 0, 0, "fp32"), (2049, 60, 264, 0, 0, 0, 0, "fp16"),
            (2500, 700, 768, 8, 0, 16, 0, "bf16"), (3001, 90, 1001, 3, 1, 0, 3, "fp32"), (2100, 64, 2056, 0, 0, 0, 0, "bf16"),
            (2200, 50, 2055, 0, 0, 1, 0, "fp32"), (9000, 300, 130, 6, 0, 0, 5, "bf16"), (20011, 3000, 24, 0, 0, 0, 0, "fp32"),
            (33001, 70, 600, 0, 0, 0, 0, "bf16")]:
        _, d = _rows(n, dim, dtype, pad=dpad, off=doff)
        ids = _ids(n, vocab, how, seed=dim, idt=torch.int32 if n % 2 else torch.int64)
        k = ids.long()
        d[(k < 0) | (k >= vocab)] = float("nan")      # not read
        _check(ss, d, ids, vocab, dtype=odt, pad=pad, off=off, scale=1.0 if n % 3 else 0.7)


@pytest.mark.parametrize("n", [1, 2, 63, 255, 256, 257, 1023, 1024, 1025, 2047, 2049, 4095, 4097, 8193, 16384, 65537, 300001])
def test_grad_position_counts(ss, n):
    """Every way in which the positions are shared out."""
    for how, vocab in (("any", 70001), ("few", 600), ("any", 17)):
        _, d = _rows(n, 16, "bf16", seed=n)
        _check(ss, d, _ids(n, vocab, how, seed=1), vocab, dtype="fp32")


@pytest.mark.parametrize("vocab", [1, 2, 255, 256, 511, 512, 513, 65535, 65536, 262143, 262144, 1 << 20, (1 << 27) + 3])
def test_grad_table_sizes(ss, vocab):
    """Every number of digits that a token has."""
    dim = 8 if vocab < 1 << 24 else 1
    _, d = _rows(3001, dim, "bf16", seed=3)
    ids = _ids(3001, vocab, "any", seed=2)
    ids[:7] = torch.tensor([0, vocab - 1, vocab // 2, vocab - 1, 0, -1, vocab], device="cuda")
    _check(ss, d, ids, vocab, dtype="bf16")


@pytest.mark.parametrize("bdt", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("n", [700, 5000])
@pytest.mark.parametrize("dim,bpad,pad,off", [(768, 0, 0, 0), (100, 4, 0, 1), (33, 0, 3, 0), (2064, 8, 0, 0)])
def test_grad_on_a_base(ss, bdt, dim, bpad, pad, off, n):
    _, d = _rows(n, dim, "bf16" if n == 700 else "fp32", seed=4)
    _, base = _rows(300, dim, bdt, pad=bpad, seed=5)
    for how in ("holes", "few"):
        ids = _ids(n, 300, how, seed=6)
        _check(ss, d, ids, 300, base=base, pad=pad, off=off, scale=0.25)
        _check(ss, d, ids, 300, base=base, pad=pad, off=off, dtype=bdt, in_place=True)
    _check(ss, d, _ids(n, 300, "none"), 300, base=base, pad=pad, off=off)


def test_grad_without_positions(ss):
    d = torch.empty((0, 48), dtype=torch.bfloat16, device="cuda")
    ids = torch.empty(0, dtype=torch.int64, device="cuda")
    _, base = _rows(30, 48, "bf16", seed=5)
    _check(ss, d, ids, 30)
    _check(ss, d, ids, 30, base=base)
    _check(ss, d, ids, 30, base=base, in_place=True)


@pytest.mark.parametrize("n,vocab", [(90, 20), (4000, 900)])
def test_grad_infinities_and_nan(ss, n, vocab):
    """They reach their own token's columns and no other."""
    _, d = _rows(n, 40, "fp32", seed=7)
    ids = _ids(n, vocab, "any", seed=8)
    d[5, 3], d[6, 4], d[70, 9] = float("nan"), float("inf"), -float("inf")
    _check(ss, d, ids, vocab, dtype="bf16")


def test_grad_is_that_of_the_lookup(ss):
    """Against differences of the lookup: <d_out, out> is linear in the table, so a step shows the whole slope."""
    vocab, dim, n, scale, h = 60, 72, 200, 0.5, 0.25
    _, t = _rows(vocab, dim, "fp32", seed=1)
    _, d = _rows(n, dim, "fp32", seed=2)
    ids = _ids(n, vocab, "holes", seed=3)
    ids = torch.where(ids >= vocab, -1, ids)
    g = _check(ss, d, ids, vocab, dtype="fp32", scale=scale)
    plus, minus = torch.empty_like(d), torch.empty_like(d)
    v = torch.randn(vocab, generator=torch.Generator(device="cuda").manual_seed(4), device="cuda", dtype=torch.float32)
    v = v[:, None].expand(vocab, dim)
    ss.ss_embedding(t + h * v, ids, plus, scale=scale)
    ss.ss_embedding(t - h * v, ids, minus, scale=scale)
    torch.cuda.synchronize()
    slope = float((_f64(d) * (_f64(plus) - _f64(minus))).sum()) / (2 * h)
    got = float((_f64(g) * _f64(v)).sum())
    # roundings of the table's steps and of the products, 2^-24 of values below 8 each, over the step
    assert abs(got - slope) <= float(_f64(d).abs().sum()) * 8 * 3 * 2.0 ** -24 / h + 1e-6


def test_grad_results_do_not_change_from_call_to_call(ss):
    _, d = _rows(5000, 200, "bf16", seed=9)
    ids = _ids(5000, 700, "few", seed=9)
    first = None
    for _ in range(4):
        got = _check(ss, d, ids, 700)
        first = got if first is None else first
        assert torch.equal(got, first)


def test_grad_streams_graphs_and_shared_workspace(ss):
    """Another stream; two captured graphs that share a workspace, replayed one behind the other."""
    sets = []
    for n, vocab in ((3000, 900), (1111, 50)):
        _, d = _rows(n, 136, "bf16", seed=n)
        ids = _ids(n, vocab, "few", seed=n)
        want = _check(ss, d, ids, vocab)
        assert torch.equal(_check(ss, d, ids, vocab, stream=torch.cuda.Stream()), want)
        sets.append((d, ids, torch.zeros((vocab, 136), dtype=torch.bfloat16, device="cuda"), want))
    ws = _workspace(ss, 3000, 900, 136)
    graphs = []
    for d, ids, t, _ in sets:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            ss.ss_embedding_grad(d, ids, t, ws)
        graphs.append(g)
    for _ in range(3):
        for (_, _, t, _), g in zip(sets, graphs):
            t.zero_()
            g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(t, want) for _, _, t, want in sets)


def test_grad_calls_right_behind_one_another(ss):
    """Calls that share a workspace, without a wait in between, their inputs written right before and overwritten right
    after, their tables read right after: sorted ones, others, in place and on a base."""
    sets = []
    for n, vocab, kind in ((5000, 3000, "none"), (1000, 2000, "base"), (4001, 500, "base"), (9000, 70, "place"),
                           (300, 40, "place")):
        _, d = _rows(n, 200, "bf16", seed=n)
        _, base = _rows(vocab, 200, "bf16", seed=vocab)
        ids = _ids(n, vocab, "few", seed=n)
        want = _check(ss, d, ids, vocab, base=None if kind == "none" else base, in_place=kind == "place")
        sets.append((n, vocab, kind, d, base, ids, want))
    ws = torch.empty(ss.ss_embedding_grad_workspace(9000, 3000, 200), dtype=torch.uint8, device="cuda")
    d = torch.empty((9000, 200), dtype=torch.bfloat16, device="cuda")
    ids = torch.empty(9000, dtype=torch.int64, device="cuda")
    b, t = (torch.empty((3000, 200), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    got = []
    for _ in range(6):
        for n, vocab, kind, src, base, tokens, _ in sets:
            d[:n].copy_(src)
            ids[:n].copy_(tokens)
            (t if kind == "place" else b)[:vocab].copy_(base)
            ss.ss_embedding_grad(d[:n], ids[:n], t[:vocab], ws,
                                 base={"none": None, "base": b[:vocab], "place": t[:vocab]}[kind])
            d.fill_(float("nan"))
            ids.fill_(3)
            b.fill_(float("nan"))
            got.append(t[:vocab].clone())
    torch.cuda.synchronize()
    for i, g in enumerate(got):
        assert torch.equal(g, sets[i % len(sets)][-1]), sets[i % len(sets)][:3]


def test_grad_on_two_streams_at_once(ss):
    """Each with a workspace of its own."""
    sets = []
    for n, vocab in ((6000, 20000), (7000, 900)):
        _, d = _rows(n, 264, "bf16", seed=n)
        ids = _ids(n, vocab, "few", seed=n)
        sets.append((d, ids, _workspace(ss, n, vocab, 264), _check(ss, d, ids, vocab), torch.cuda.Stream()))
    torch.cuda.synchronize()
    tables = [[torch.empty_like(s[3]) for _ in range(8)] for s in sets]
    for i in range(8):
        for (d, ids, ws, _, st), t in zip(sets, tables):
            ss.ss_embedding_grad(d, ids, t[i], ws, stream=st)
    torch.cuda.synchronize()
    for s, t in zip(sets, tables):
        assert all(torch.equal(x, s[3]) for x in t)


def test_grad_of_extreme_ids(ss):
    """Ids as far out as the type goes carry nothing."""
    for n in (300, 3000):
        _, d = _rows(n, 24, "bf16", seed=n)
        for idt, far in ((torch.int64, 2 ** 63 - 1), (torch.int32, 2 ** 31 - 1)):
            ids = _ids(n, 100, "any", idt=idt)
            ids[::5], ids[1::7] = far, -far - 1
            _check(ss, d, ids, 100)


def test_grad_of_many_positions_past_2_31_elements(ss):
    """The same for positions enough to be sorted."""
    n, ld = 2100, (1 << 20) + 8
    buf = torch.zeros((n - 1) * ld + 64, dtype=torch.bfloat16, device="cuda")
    d = buf.as_strided((n, 64), (ld, 1))
    _, src = _rows(n, 64, "bf16", seed=1)
    d.copy_(src)
    ids = _ids(n, 70, "any", seed=1)
    assert torch.equal(_check(ss, d, ids, 70), _check(ss, src, ids, 70))


def test_grad_past_2_31_elements(ss):
    """Rows past 2^31 elements of the gradient and of the table."""
    ld = (1 << 30) + 8
    buf = torch.zeros(3 * ld + 64, dtype=torch.bfloat16, device="cuda")
    d = buf.as_strided((4, 64), (ld, 1))
    d.copy_(torch.randn((4, 64), device="cuda"))
    tbuf = torch.zeros(3 * ld + 64, dtype=torch.bfloat16, device="cuda")
    t = tbuf.as_strided((4, 64), (ld, 1))
    ids = torch.tensor([3, 0, 3, 2], device="cuda")
    ss.ss_embedding_grad(d, ids, t, _workspace(ss, 4, 4, 64))
    torch.cuda.synchronize()
    want = torch.stack([d[1].float(), torch.zeros(64, device="cuda"), d[3].float(), d[0].float() + d[2].float()])
    assert torch.equal(t, want.to(torch.bfloat16))
