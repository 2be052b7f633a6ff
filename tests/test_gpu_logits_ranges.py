"""The operators on rows of logits over the range of their arguments: finite mask fills and other logits far from
zero, scales from the smallest to the largest, differences that pass the type's range, gradients written over their
logits. Against the plain float64 rows.

Bounds. A row's exponential 2^((x - m) c) has one rounding of its argument, 2^-24 of it, and ex2's 2^-22: terms that are
not negligible have arguments below 30, so 1.5e-6, and the adding up of at most 540 terms in a chain stays below what
is left to REL = 2e-5 (the rounding of a chain of positive terms is of both signs). That bound does not depend on how
far the logits are from zero, on the fill or on the scale, which is what these tests are about. A log probability
adds the roundings of (x - m) scale - log s, a few of its own EPS32.
"""
import numpy as np
import pytest

from logits_ref import REL, grad_bound, row_distill, row_logprobs_grad, row_softmax
from test_gpu_logits_ops import (MODES, TYPES, _check_distill, _check_logprobs, _close, _logits, _np, _outputs,
                                 _same_layout, _tail, _teacher)

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def ss():
    import fsdp_sharded_mixed_ss_gb300 as m
    return m


def _check_norms(ss, x, ids, t, mode, scale):
    """The normalisers that the distillation calls save."""
    rows = x.shape[0]
    norm = torch.full((rows, 2), 77.0, device="cuda")
    ss.ss_distill_topk(x, ids, t, norm=norm, tail=_tail(ss, mode), scale=scale)
    torch.cuda.synchronize()
    X, got, s32 = _np(x), _np(norm), float(np.float32(scale))
    for r in range(rows):
        _, m, s = row_softmax(X[r], s32)
        assert got[r, 0] == m
        _close(got[r, 1], s, REL * s, ("norm", mode, r))


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("mode", MODES)
def test_distill_sums_of_filled_rows(ss, mode, dtype):
    """Rows that a finite fill masked out are uniform: the sums keep their digits however large the fill."""
    fills = [-1e4, -1e6, -5e8, -1e9, -1.4e9, 1.4e9]
    x = _logits(len(fills), 9001, dtype, pad=3, off=1)
    ids, t = _teacher(x, 12, 1.0)
    for r, f in enumerate(fills):
        x[r] = f
    _check_norms(ss, x, ids, t, mode, 1.0)
    _check_distill(ss, x, ids, t, mode, dtype=dtype, dpad=3, doff=1)


@pytest.mark.parametrize("offset", [0.0, 1e4, -1e5, 1e6, -1e7, 1e8])
@pytest.mark.parametrize("gap", [70.0, 100.0, 3000.0])
def test_saved_gradient_of_small_tails(ss, gap, offset):
    """Unlisted mass of e^-60 and less, with logits far from zero. p / p_t is e^(z - max z - log p_t), a small number
    between large ones: relative errors of 2^-24 of |log p_t| from its own rounding, its product's with log2(e), the
    difference's, and half of that from either constant, so 4 in all; none from the logits' distance from zero."""
    vocab, k = 600, 8
    x = torch.linspace(-1.0, 1.0, vocab, device="cuda").repeat(3, 1)
    x += offset
    ids = torch.tensor([[3, 99, 100, 101, 102, 300, 301, 599]] * 3, device="cuda", dtype=torch.int32)
    x[:, ids[0].long()] = offset + gap
    t = torch.full((3, k), 0.8 / k, device="cuda").log()
    norm, tail, loss = torch.empty((3, 2), device="cuda"), torch.empty(3, device="cuda"), torch.empty(3, device="cuda")
    d, e = torch.empty_like(x), torch.empty_like(x)
    ss.ss_distill_topk(x, ids, t, loss, norm=norm, tail_logprob=tail, d_logits=d)
    ss.ss_distill_topk_grad(x, ids, t, norm, e, tail_logprob=tail)
    torch.cuda.synchronize()
    for r in range(3):
        _, lpt, g, size, _ = row_distill(_np(x[r]), 1.0, ids[r].tolist(), _np(t[r]), 1.0, "bucket", 1.0)
        assert lpt < -60
        bound = grad_bound(g, size, "fp32")
        _close(_np(d[r]), g, bound, ("fused", r))
        _close(_np(e[r]), g, bound + 4 * 2.0 ** -24 * abs(lpt) * np.abs(g), ("saved", r))


FILLS = [-1e9, -2e9, -3e9, -1e10, -1e12, -1e15, -1e20, -1e29, -1e30, -1e35, 3e9, 1e10, 1e20]
SCALES = [1.0, 0.5, 1.0 / 0.7, 10.0]


def _filled(dtype, vocab, fills, **kw):
    """For each fill a row of nothing else, one with all but ten tokens filled, one with a contiguous half filled, one
    with every third token filled, and one whose first tokens and last one are left."""
    x = _logits(5 * len(fills), vocab, dtype, **kw)
    for i, f in enumerate(fills):
        r = x[5 * i:5 * i + 5]
        keep = torch.arange(10, device="cuda") * (vocab // 11) + 3
        kept = r[1, keep].clone()
        r[0] = f
        r[1] = f
        r[1, keep] = kept
        r[2, vocab // 3:vocab // 3 + vocab // 2] = f
        r[3, ::3] = f
        r[4, 3:-1] = f
    return x


@pytest.mark.parametrize("scale", SCALES)
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_logprobs_filled_rows(ss, dtype, scale):
    x = _filled(dtype, 3001, FILLS, pad=7, off=1)
    tok = torch.arange(x.shape[0], device="cuda") * 37 % 3001
    _check_logprobs(ss, x, tok, 0, scale)
    _check_logprobs(ss, x, tok, 17, scale)


@pytest.mark.parametrize("vocab", [50257, 128256])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_logprobs_filled_rows_shared_by_blocks(ss, dtype, vocab):
    """Whole threads and blocks of a row that see fills only."""
    x = _filled(dtype, vocab, [-1e10], pad=1)
    tok = torch.arange(x.shape[0], device="cuda") * 37
    _check_logprobs(ss, x, tok, 20)
    _check_logprobs(ss, x, tok, 0, 1.0 / 0.7)


@pytest.mark.parametrize("dtype,vocab,k", [("bf16", 33001, 20), ("fp32", 16390, 50)])
def test_logprobs_filled_many_rows(ss, dtype, vocab, k):
    rows = 1000
    x = _logits(rows, vocab, dtype, pad=3, seed=9)
    fills = [-1e9, -2e9, -1e10, -1e15, -1e29]
    for i, f in enumerate(fills):
        x[10 * i, :] = f
        x[10 * i + 1, : vocab // 2] = f
        x[10 * i + 2, vocab // 2:] = f
        x[10 * i + 3, ::2] = f
        x[10 * i + 4, 50:] = f
    x[60:, -vocab // 4:] = -1e10
    _check_logprobs(ss, x, torch.arange(rows, device="cuda") * 31 % vocab, k)


@pytest.mark.parametrize("scale", [1e3, 1e5, 1e7, 1e10, 1e20])
@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
def test_logprobs_low_temperatures(ss, dtype, scale):
    """Temperatures at which a row's largest logit has all the mass, or shares it with its equals."""
    x = _logits(12, 5001, dtype, pad=1, seed=3)
    x[3] -= 40.0
    x[4] = x[4].abs() * -1.0
    x[5, 7:900:31] = x[5].max()
    x[6] = 17.25
    x[7] = 0.0
    _check_logprobs(ss, x, torch.arange(12, device="cuda") * 400, 9, scale)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("offset", [-3e2, 1e4, -1e6, 1e7, 3e7, -2e8, 4e9])
def test_logprobs_logits_far_from_zero(ss, dtype, offset):
    """Ordinary differences (as far as the type holds them) around a large offset."""
    vocab, digits = 4001, 8 if dtype == "bf16" else 24
    base = float(torch.tensor(offset, dtype=TYPES[dtype]))
    step = 2.0 ** (np.frexp(abs(base))[1] - digits)  # between neighbouring numbers of the type
    x = torch.empty((6, vocab), dtype=TYPES[dtype], device="cuda")
    g = torch.Generator(device="cuda")
    g.manual_seed(5)
    x.copy_((base + torch.randint(-6, 1, x.shape, generator=g, device="cuda").double() * step))
    for scale in (1.0, 0.25, 1.0 / step, 3.0 / step):
        _check_logprobs(ss, x, torch.arange(6, device="cuda") * 11, 5, scale)


def _check_logprobs_grad(ss, x, tok, dtype, scale):
    rows, k = x.shape[0], 4
    out = _outputs(rows, k)
    ss.ss_token_logprobs(x, tok, scale=scale, **out)
    g = torch.Generator(device="cuda")
    g.manual_seed(4)
    up = {n: torch.randn(rows, generator=g, device="cuda") for n in ("d_logprob", "d_entropy", "d_lse")}
    up["d_top_logprob"] = torch.randn((rows, k), generator=g, device="cuda")
    d = torch.full_like(x, 9.0)
    X, s32 = _np(x), float(np.float32(scale))
    for names in [("d_logprob",), ("d_entropy",), tuple(up)]:
        ss.ss_token_logprobs_grad(x, out["norm"], d, tokens=tok, entropy=out["entropy"], top_id=out["top_id"],
                                  scale=scale, **{n: up[n] for n in names})
        torch.cuda.synchronize()
        got = _np(d)
        for i in range(rows):
            u = {n: float(up[n][i]) for n in names if n != "d_top_logprob"}
            if "d_top_logprob" in names:
                u["top_id"], u["d_top"] = out["top_id"][i].tolist(), up["d_top_logprob"][i].tolist()
            ref, size = row_logprobs_grad(X[i], s32, token=int(tok[i]) if "d_logprob" in names else None, **u)
            # ex2 gives 0 for probabilities below 2^-126; log p and H near 0 are off by what the forward call's may be
            least = s32 * 2.0 ** -126 * (1e3 if "d_entropy" in names else 20.0)
            logs = 3 * REL * s32 * abs(u.get("d_entropy", 0.0)) * np.exp(row_softmax(X[i], s32)[0])
            _close(got[i], ref, grad_bound(ref, size, dtype) + least + logs, (names, i))
    y = _same_layout(x)
    ss.ss_token_logprobs_grad(y, out["norm"], y, tokens=tok, entropy=out["entropy"], top_id=out["top_id"], scale=scale,
                              **up)
    torch.cuda.synchronize()
    assert torch.equal(y, d)


@pytest.mark.parametrize("scale", SCALES)
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_logprobs_grad_filled_rows(ss, dtype, scale):
    x = _filled(dtype, 1501, FILLS, pad=3, off=2)
    _check_logprobs_grad(ss, x, torch.arange(x.shape[0], device="cuda") * 37 % 1501, dtype, scale)


@pytest.mark.parametrize("scale", [1e3, 1e5, 1e7, 1e10])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_logprobs_grad_low_temperatures(ss, dtype, scale):
    x = _logits(6, 2001, dtype, seed=3)
    x[3] -= 40.0
    x[4, 7:900:31] = x[4].max()
    x[5] = 17.25
    _check_logprobs_grad(ss, x, torch.arange(6, device="cuda") * 300, dtype, scale)


@pytest.mark.parametrize("scale", [1.0, 0.5])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("mode", MODES)
def test_distill_filled_rows(ss, mode, dtype, scale):
    x = _filled(dtype, 1203, FILLS, pad=5)
    ids, t = _teacher(x, 12, scale, idt=torch.int64)
    _check_norms(ss, x, ids, t, mode, scale)
    _check_distill(ss, x, ids, t, mode, scale=scale, dtype=dtype, dpad=5)


@pytest.mark.parametrize("dtype,vocab", [("bf16", 128256), ("fp32", 50257)])
def test_distill_filled_rows_shared_by_blocks(ss, dtype, vocab):
    x = _filled(dtype, vocab, [-1e10], pad=1)
    ids, t = _teacher(x, 64, 1.0)
    _check_norms(ss, x, ids, t, "bucket", 1.0)
    _check_distill(ss, x, ids, t, "bucket", dtype=dtype, dpad=1)


@pytest.mark.parametrize("mode", MODES)
@pytest.mark.parametrize("scale", [1e7, 1e10])
def test_distill_low_temperatures(ss, scale, mode):
    x = _logits(5, 2001, "fp32", seed=3)
    x[3] -= 40.0
    x[4] = 17.25
    ids, t = _teacher(x, 9, 1.0)
    _check_norms(ss, x, ids, t, mode, scale)
    _check_distill(ss, x, ids, t, mode, scale=scale, dtype="fp32")


@pytest.mark.parametrize("scale", [1e-30, 1e-37, 1e-38, 1e-39, 1.5e-45])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_smallest_scales(ss, dtype, scale):
    """Rows that a scale near zero makes uniform over their unmasked tokens."""
    x = _logits(4, 3001, dtype, pad=3, off=1)
    x[1, 5:2000] = -float("inf")
    x[2] = -float("inf")
    tok = torch.tensor([7, 2500, 0, 3000], device="cuda")
    _check_logprobs(ss, x, tok, 17, scale)
    _check_logprobs(ss, x, tok, 0, scale)
    ids, t = _teacher(x, 12, 1.0)
    ids[1] = torch.arange(12, device="cuda") + 2900
    for mode in MODES:
        _check_distill(ss, x, ids, t, mode, scale=scale, dtype=dtype, dpad=3, doff=1)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_differences_past_the_types_range(ss, dtype):
    """x - max x passes what the type holds, and the scale brings it back."""
    lowest, big = torch.finfo(TYPES[dtype]).min, torch.finfo(TYPES[dtype]).max
    vocab = 2003
    x = torch.full((3, vocab), lowest, dtype=TYPES[dtype], device="cuda")
    x[0, 7] = big
    x[1, ::2] = big
    x[2] = (torch.linspace(-0.99, 0.99, vocab, device="cuda", dtype=torch.float64) * big).to(x.dtype)
    tok = torch.tensor([3, 1, 0], device="cuda")
    for scale in (0.25, 0.4, 1e-20, 2e-37, 1e-37, 2e-38, 5e-39):
        _check_logprobs(ss, x, tok, 9, scale)
    ids, t = _teacher(x, 12, 1.0)
    ids[2] = torch.arange(12, device="cuda") * 150
    for mode in MODES:
        for scale in (0.25, 2e-37, 1e-37, 2e-38, 5e-39):
            _check_distill(ss, x, ids, t, mode, scale=scale, dtype=dtype)


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("mode", MODES)
def test_saved_gradient_over_its_logits(ss, mode, dtype):
    """The gradient from saved normalisers written over the logits: the same bits as apart from them, with rows in one
    part and in several, and listed tokens in every part and at both ends."""
    for rows, vocab, pad, off, k in [(3, 7, 0, 0, 5), (4, 9, 1, 1, 9), (7, 1000, 0, 3, 128), (9, 33001, 5, 3, 100),
                                     (40, 128256, 3, 1, 128), (300, 70001, 0, 0, 64)]:
        x = _logits(rows, vocab, dtype, pad=pad, off=off, seed=k)
        ids, t = _teacher(x, k, 1.0, seed=k)
        if vocab > 2 * k:  # a third of the slots over the whole row, the edges among them
            n = k // 3
            ids[:, :n] = (torch.arange(n, device="cuda") * ((vocab - 1) // (n - 1))).to(ids.dtype)
            ids[:, 0], ids[:, 1], ids[:, n - 1] = 0, vocab - 1, vocab - 2
        w = torch.linspace(0.25, 2.0, rows, device="cuda")
        w[rows // 2] = 0.0
        norm, tail, loss = (torch.empty(s, device="cuda") for s in ((rows, 2), (rows,), (rows,)))
        kw = dict(row_weight=w, tail=_tail(ss, mode))
        ss.ss_distill_topk(x, ids, t, loss, norm=norm, tail_logprob=tail, **kw)
        up = torch.linspace(0.5, 2.0, rows, device="cuda")
        up[0] = 0.0 if rows > 4 else 1.0
        kw.update(tail_logprob=tail, d_loss=up)
        apart = torch.full_like(x, 3.0)
        ss.ss_distill_topk_grad(x, ids, t, norm, apart, **kw)
        y = _same_layout(x)
        ss.ss_distill_topk_grad(y, ids, t, norm, y, **kw)
        torch.cuda.synchronize()
        assert torch.equal(y, apart), (rows, vocab)
        assert not bool(apart.isnan().any())


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("mode", MODES)
def test_losses_whose_logs_pass_the_types_range(ss, mode, dtype):
    """A listed token at the type's lowest value, and a scale that takes its log p, not its part of the loss, past what
    fp32 holds."""
    lowest, vocab, k = torch.finfo(TYPES[dtype]).min, 1203, 12
    x = _logits(4, vocab, dtype, pad=5)
    ids, t = _teacher(x, k, 1.0)
    for r in range(4):
        x[r, ids[r, 3 + r].long()] = lowest
    t = (torch.arange(k, device="cuda") * -0.3 - 2.5).repeat(4, 1)  # q of 0.08 and less, 0.3 in all
    loss, alone, d = torch.empty(4, device="cuda"), torch.empty(4, device="cuda"), torch.empty_like(x)
    for scale in (1.0 / 0.7, 2.0, 5.0):
        kw = dict(tail=_tail(ss, mode), scale=scale)
        ss.ss_distill_topk(x, ids, t, loss, d_logits=d, **kw)
        ss.ss_distill_topk(x, ids, t, alone, **kw)
        torch.cuda.synchronize()
        X, I, T, s32 = _np(x), ids.tolist(), _np(t), float(np.float32(scale))
        for r in range(4):
            ref, _, _, _, size = row_distill(X[r], s32, I[r], T[r], 1.0, mode, 1.0)
            _close([loss[r].item(), alone[r].item()], [ref, ref], 4 * REL * size, ("loss", mode, scale, r))


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("mode", MODES)
def test_distill_listed_tokens_that_are_not_numbers(ss, mode, dtype):
    """NaN or +inf at a listed token, whatever the unlisted ones are: loss, log p_t and both gradients are NaN."""
    inf, lowest = float("inf"), torch.finfo(TYPES[dtype]).min
    x = _logits(8, 1203, dtype, pad=5)
    ids, t = _teacher(x, 12, 1.0)
    for r, rest in enumerate([None, -inf, lowest, -1e4]):
        for row, value in ((r, float("nan")), (4 + r, inf)):
            if rest is not None:
                kept = x[row, ids[row].long()].clone()
                x[row] = rest
                x[row, ids[row].long()] = kept
            x[row, ids[row, 5].long()] = value
    _check_distill(ss, x, ids, t, mode, dtype=dtype, dpad=5)
    tail = torch.zeros(8, device="cuda")
    ss.ss_distill_topk(x, ids, t, tail_logprob=tail, tail=_tail(ss, mode))
    assert bool(tail.isnan().all())


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_calls_read_what_the_call_before_wrote(ss, dtype):
    """A call's kernel starts before the one ahead of it in the stream has ended: logits that the one ahead writes (a
    gradient in their place) are read after it, also where the same blocks have read them before."""
    for rows, vocab, k in [(1500, 33001, 8), (300, 20011, 0), (12, 128256, 20)]:
        x = _logits(rows, vocab, dtype, seed=2)
        ids, t = _teacher(x, 16, 1.0)
        tok = torch.arange(rows, device="cuda")
        y = x.clone()
        loss = torch.empty(rows, device="cuda")
        ss.ss_distill_topk(y, ids, t, loss, d_logits=y)
        torch.cuda.synchronize()
        want = _outputs(rows, k)
        ss.ss_token_logprobs(y, tok, scale=100.0, **want)
        torch.cuda.synchronize()
        for _ in range(5):
            z, got, first = x.clone(), _outputs(rows, k), _outputs(rows, k)
            torch.cuda.synchronize()
            ss.ss_token_logprobs(z, tok, **first)
            ss.ss_distill_topk(z, ids, t, loss, d_logits=z)
            ss.ss_token_logprobs(z, tok, scale=100.0, **got)
            torch.cuda.synchronize()
            assert all(torch.equal(got[n], want[n]) for n in want), (rows, vocab)
