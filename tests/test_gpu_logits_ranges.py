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

from logits_ref import REL, grad_bound, row_distill, row_softmax
from test_gpu_logits_ops import MODES, _check_distill, _close, _logits, _np, _tail, _teacher

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
