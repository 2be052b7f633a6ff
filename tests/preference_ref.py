"""Plain float64 form of the preference loss, pair by pair in numpy, and bounds of the fp32 kernel's errors.

Bounds. A term w (lp - ref) rounds twice, 2^-24 each; eight of them are added in fp32 by three levels of sums, which round
each term's share three times more; the sums of pairs of fp32 above add nothing that counts. With S the sum of the terms'
absolute values a score is within 5 * 2^-24 S. The weights' sum is within 3 * 2^-24 of its own, so a mean (of weights that
are not negative) within 9 * 2^-24 S over the weights' sum, with the quotient's rounding. h is within beta times both
scores' bounds, and its own rounding. The loss follows with its slope, its derivative with its curvature; exp, log1p,
the divisions and products round at most eight times.
"""
import numpy as np

from logits_ref import EPS32


def _softplus(z):
    return np.logaddexp(0.0, z)


def preference(lp, offsets, *, ref=None, weight=None, pair_weight=None, kind="sigmoid", beta=0.1, margin=0.0, smooth=0.0,
               average=False, halves=False):
    """dict of (values, bounds) for loss, reward and d_logprob (NaN bounds nowhere; rows outside are NaN in `d`)."""
    lp = np.asarray(lp, np.float64)
    rows, pairs = len(lp), (len(offsets) - 1) // 2
    ref = np.zeros(rows) if ref is None else np.asarray(ref, np.float64)
    w = np.ones(rows) if weight is None else np.asarray(weight, np.float64)
    pw = np.ones(pairs) if pair_weight is None else np.asarray(pair_weight, np.float64)
    loss, loss_b = np.zeros(pairs), np.zeros(pairs)
    reward, reward_b = np.zeros((pairs, 2)), np.zeros((pairs, 2))
    d, d_b = np.full(rows, np.nan), np.zeros(rows)
    outside = np.ones(rows, bool)
    for i in range(pairs):
        seqs = (i, pairs + i) if halves else (2 * i, 2 * i + 1)
        spans = [(int(offsets[q]), int(offsets[q + 1])) for q in seqs]
        bad = any(a < 0 or b < a or b > rows for a, b in spans)
        if pw[i] == 0 or bad:
            if pw[i] != 0:
                loss[i], reward[i] = np.nan, np.nan
            for a, b in [] if bad else spans:
                d[a:b] = 0.0
                outside[a:b] = False
            continue
        score, err, per = [], [], []
        for a, b in spans:
            on = w[a:b] != 0
            with np.errstate(invalid="ignore"):
                t = w[a:b][on] * (lp[a:b][on] - ref[a:b][on])
            total = w[a:b][on].sum()
            p = 1.0 if not average else (1.0 / total if total != 0 else 0.0)
            score.append(t.sum() * p if len(t) else 0.0)
            err.append(((9 if average else 5) * 2.0 ** -24 * np.abs(t).sum() + 1e-37) * abs(p))
            per.append(p)
        with np.errstate(invalid="ignore"):
            h = beta * (score[0] - score[1]) - margin
        e = beta * (err[0] + err[1]) + EPS32 * abs(h) if np.isfinite(h) else 0.0  # an infinite h is that
        with np.errstate(over="ignore", invalid="ignore"):
            if kind == "sigmoid":
                s = float(np.exp(-_softplus(h)))                    # sigmoid(-h)
                value = (1 - smooth) * _softplus(-h) + (smooth * _softplus(h) if smooth else 0.0)
                slope, slope_size, curve = smooth - s, smooth + s, s * float(np.exp(-_softplus(-h)))
            elif kind == "hinge":
                value, slope, curve = max(0.0, 1.0 - h) if h == h else h, (-1.0 if h < 1 else 0.0) if h == h else h, 0.0
                slope_size = abs(slope)
            else:
                value, slope, curve = ((h - 0.5) / beta) ** 2, 2 * (h - 0.5) / beta ** 2, 2 / beta ** 2
                slope_size = abs(slope) + 2 / beta ** 2 * EPS32
        loss[i] = pw[i] * value
        slope_e = slope_size * e if e else 0.0  # (a square's slope is infinite where h is)
        loss_b[i] = abs(pw[i]) * (slope_e + curve * e * e + 8 * EPS32 * abs(value)) + 1e-37
        for k, (a, b) in enumerate(spans):
            g = (-1) ** k * pw[i] * slope * beta * per[k]
            d[a:b] = np.where(w[a:b] == 0, 0.0, w[a:b] * g)
            d_b[a:b] = np.abs(w[a:b] * pw[i] * beta * per[k]) * (curve * e + 8 * EPS32 * slope_size) + 1e-37
            outside[a:b] = False
            reward[i, k] = beta * score[k]
            reward_b[i, k] = beta * err[k] + 2 * EPS32 * abs(reward[i, k]) + 1e-37
    return dict(loss=(loss, loss_b), reward=(reward, reward_b), d_logprob=(d, d_b), outside=outside)
