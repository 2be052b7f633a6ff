"""Plain float64 forms of the operators on rows of logits, one row at a time in numpy, and the
error bounds of the fp32 kernels that the tests compare with them.

Bounds. The kernels form 2^((x - m) c) with one rounding each for the difference, the product and
c = scale log2(e), and ex2.approx (2^-22 relative): with d = |x - m| c the term is within
2^-22 + 3 * 2^-24 ln 2 d of its value. The sum's terms weigh d by their share, so the mean of d is at
most log2(vocab) + 1 < 19 for the sizes here: 2.4e-7 + 2.4e-6. Adding up to 512 positive terms per
thread, 8 per warp tree and 16 over warps and blocks rounds at most 540 times, 540 * 2^-24 = 3.2e-5
at the very worst; rounding errors of both signs leave a small part of that, so REL = 2e-5 bounds
sums, and with them log s, absolutely. A log probability adds the rounding of (x - m) scale - log s.
"""
import math

import numpy as np

REL = 2e-5
EPS32 = 2.0 ** -23


def row_softmax(x, scale):
    """(log p, max x, sum) of one float64 row; log p is all -inf for a masked-out row, all NaN with NaN or +inf."""
    if np.isnan(x).any() or np.isposinf(x).any():
        return np.full_like(x, np.nan), np.nan, np.nan
    m = x.max()
    if np.isneginf(m):
        return np.full_like(x, -np.inf), -np.inf, 0.0
    d = (x - m) * scale
    s = np.exp(d).sum()
    return d - math.log(s), m, s


def row_logprobs(x, scale, token, k):
    logp, m, s = row_softmax(x, scale)
    nan, empty = np.isnan(s), s == 0
    p = np.exp(logp)
    h = np.nan if nan else (0.0 if empty else -(p[p > 0] * logp[p > 0]).sum())
    if token is None or token < 0:
        lp = 0.0
    elif token >= len(x):
        lp = np.nan
    else:
        lp = logp[token]
    lse = np.nan if nan else (-np.inf if empty else m * scale + math.log(s))
    order = np.full(k, -1) if nan else np.argsort(-(x + 0.0), kind="stable")[:k]
    top = np.full(k, np.nan) if nan else logp[order]
    return dict(logprob=lp, entropy=h, lse=lse, norm=(m, s), top_logprob=top, top_id=order)


def row_logprobs_grad(x, scale, *, token=None, d_logprob=0.0, d_entropy=0.0, d_lse=0.0, top_id=(), d_top=()):
    """(gradient, a bound on the size of the terms it is the sum of)."""
    n = len(x)
    logp, _, s = row_softmax(x, scale)
    token = -1 if token is None else token
    pairs = [(int(i), float(u)) for i, u in zip(top_id, d_top) if i >= 0]
    if token >= 0:
        pairs.append((int(token), float(d_logprob)))
    if not any(u != 0 for _, u in pairs) and d_entropy == 0 and d_lse == 0:
        return np.zeros(n), np.zeros(n)
    if s == 0:
        return np.zeros(n), np.zeros(n)
    if np.isnan(s) or any(i >= n for i, _ in pairs):
        return np.full(n, np.nan), np.zeros(n)
    p = np.exp(logp)
    lp = np.where(p > 0, logp, 0.0)
    h = -(p * lp).sum()
    total = sum(u for _, u in pairs)
    g = p * (d_lse - total) - d_entropy * p * (lp + h)
    size = p * (abs(d_lse) + sum(abs(u) for _, u in pairs) + abs(d_entropy) * (np.abs(lp) + h))
    for i, u in pairs:
        g[i] += u
        size[i] += abs(u)
    return scale * g, scale * size


def row_distill(x, scale, ids, t, t_scale, mode, weight):
    """(loss, log p_t, gradient of the loss, size of the gradient's terms, size of the loss's terms)."""
    n = len(x)
    zero = np.zeros(n)
    if weight == 0:
        return 0.0, 0.0, zero, zero, 0.0
    logp, _, s = row_softmax(x, scale)
    seen, use = set(), []
    bad = False
    for j, i in enumerate(ids):
        bad = bad or i >= n
        if 0 <= i < n and i not in seen:
            seen.add(int(i))
            use.append(j)
    ids = np.array([ids[j] for j in use], dtype=np.int64)
    lq = np.array([t[j] * t_scale for j in use], dtype=np.float64)
    nan = np.full(n, np.nan)
    if mode == "renorm" and len(use):
        m = lq.max()
        if not np.isneginf(m):
            lq = lq - (m + math.log(np.exp(lq - m).sum()))
    q = np.exp(lq)
    Q = q.sum()
    if bad or np.isnan(s) or np.isnan(Q):
        return np.nan, np.nan, nan, zero, 0.0
    qt = max(0.0, 1.0 - Q) if mode == "bucket" else 0.0
    p = np.exp(logp)
    out = np.ones(n, dtype=bool)
    out[ids] = False
    rest = logp[out]
    big = rest.max() if rest.size else -np.inf
    lpt = -np.inf
    if not np.isneginf(big) and big / math.log(2.0) > -1e4:
        lpt = big + math.log(np.exp(rest - big).sum())
    live = q > 0
    with np.errstate(invalid="ignore"):
        terms = q[live] * (lq[live] - logp[ids][live])
    loss = terms.sum()
    size = np.abs(terms).sum() + q.sum()
    if qt > 0 and not np.isneginf(lpt):
        loss += qt * (math.log(qt) - lpt)
        size += qt * (1.0 + abs(math.log(qt) - lpt)) + Q
    if s == 0:
        return weight * loss, lpt, zero, zero, abs(weight) * size
    b = Q + qt
    g = p * b
    gs = p * (Q + 1.0)
    if qt > 0 and not np.isneginf(lpt):
        ratio = np.where(out, np.exp(logp - lpt), 0.0)
        g = g - qt * ratio
        gs = gs + (qt + Q * 2e-2) * ratio  # q_t's own error is Q's, 2^-24 of 1 and a few list terms
    elif mode == "bucket":
        g = np.where(out, 0.0, g)
    g[ids] -= q
    gs[ids] += q
    k = weight * scale
    return weight * loss, lpt, k * g, abs(k) * gs, abs(weight) * size


def grad_bound(g, size, dtype):
    """Elementwise bound of a gradient's error: the sums' error on every term, and one rounding to the type."""
    b = 3 * REL * size
    if dtype == "bf16":
        return b + np.abs(g) * 2.0 ** -8 + 2.0 ** -133
    if dtype == "fp16":
        return b + np.abs(g) * 2.0 ** -11 + 2.0 ** -24
    return b + 2.0 ** -126
