"""Plain float64 form of the clipped policy loss, one row at a time in numpy, and bounds of the fp32 kernels' errors.

Bounds. A log probability is within REL of its value (logits_ref: the bound of log s; the kernels keep the rest as a
pair). ratio = exp(log p - old) then is within REL relatively, and four roundings; a KL estimate within |KL'| REL and, for
the second-order part, REL^2; its own terms round four times. The entropy is within 3 REL (1 + H). The loss adds these,
and its derivative with respect to log p is of terms A ratio and kl_coef KL' with the errors of ratio and exp(-d).
Exponentials below 2^-126 are flushed to zero, before the factors p (A + B log2 p) are applied to them: "flush" bounds
what a gradient loses to that.
"""
import math

import numpy as np

from logits_ref import EPS32, REL, row_softmax


def row_policy(x, scale, token, adv, *, old=None, ref=None, weight=1.0, low=0.2, high=0.2, most=0.0, kind="k3", kc=0.0,
               ec=0.0):
    """(outputs, their bounds, gradient, size of the gradient's terms) of one float64 row."""
    n = len(x)
    names = ("loss", "logprob", "entropy", "ratio", "kl", "d_logprob", "d_entropy")
    zero = np.zeros(n)
    if weight == 0 or token < 0:
        return dict.fromkeys(names, 0.0) | {"norm": (0.0, 0.0)}, dict.fromkeys(names + ("flush",), 0.0), zero, zero
    logp, m, s = row_softmax(x, scale)
    if np.isnan(s) or token >= n:
        o = dict.fromkeys(names, np.nan)
        if not np.isnan(s):
            p = np.exp(logp)
            o["entropy"] = -(p[p > 0] * logp[p > 0]).sum() if s else 0.0
        o["d_entropy"] = -weight * ec
        return o | {"norm": (m, s)}, dict.fromkeys(names + ("flush",), 3 * REL * 20), np.full(n, np.nan), zero
    p = np.exp(logp)
    safe = np.where(p > 0, logp, 0.0)
    h = -(p * safe).sum()
    lp = logp[token]
    with np.errstate(over="ignore", invalid="ignore"):
        ratio = math.inf if old is not None and lp - old > 709 else (1.0 if old is None else float(np.exp(lp - old)))
        lo, hi = (0.0, 1.0 + high) if adv >= 0 else (1.0 - low, most if most else math.inf)
        held = min(max(ratio, lo), hi)
        loss = -adv * held
        d_lp = -adv * ratio if lo <= ratio <= hi else 0.0
        e_loss = abs(adv) * min(ratio, 1e30) * (REL + 4 * EPS32)
        size = abs(adv) * ratio if lo <= ratio <= hi else 0.0
        kl = e_kl = 0.0
        if ref is not None:
            d = lp - ref
            back = float(np.exp(-d))
            kl = {"k1": d, "k2": d * d / 2, "k3": back + d - 1}[kind]
            dkl = {"k1": 1.0, "k2": d, "k3": 1 - back}[kind]
            e_kl = abs(dkl) * REL + REL * REL * (1 + back) + 4 * EPS32 * (abs(kl) + (kind == "k3") * min(abs(d), 1) ** 2)
            if kind == "k3" and abs(d) >= 0.5:
                e_kl += 4 * EPS32 * (abs(d) + back)
            if kc:
                loss += kc * kl
                d_lp += kc * dkl
                e_loss += abs(kc) * e_kl
                size += abs(kc) * {"k1": 1.0, "k2": abs(d) + 1, "k3": 1 + back}[kind]
    if ec:
        loss -= ec * h
    d_h = -weight * ec
    o = dict(loss=weight * loss, logprob=lp, entropy=h, ratio=ratio, kl=kl, d_logprob=weight * d_lp, d_entropy=d_h,
             norm=(m, s))
    b = dict(loss=abs(weight) * (e_loss + abs(ec) * 3 * REL * (1 + h)) + 4 * EPS32 * abs(weight * loss) + 1e-37,
             logprob=REL + EPS32 * abs(lp), entropy=3 * REL * (1 + h), ratio=ratio * (REL + 4 * EPS32), kl=e_kl + 1e-37,
             d_logprob=abs(weight) * size * (REL + 8 * EPS32) + 1e-37, d_entropy=2 * EPS32 * abs(d_h))
    b["flush"] = 2.0 ** -126 * scale * (abs(weight) * size + abs(d_h) * (126 + h))
    b = {k: float(np.nan_to_num(v, nan=1.0, posinf=1.0)) for k, v in b.items()}
    if s == 0 or (d_lp == 0 and d_h == 0):
        return o, b, zero, zero
    with np.errstate(invalid="ignore"):
        g = -p * weight * d_lp - d_h * p * (safe + h)
        gs = p * abs(weight) * size + abs(d_h) * p * (np.abs(safe) + h)
        g[token] += weight * d_lp
        gs[token] += abs(weight) * size
    return o, b, scale * g, scale * gs
