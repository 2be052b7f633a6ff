"""The clipped policy loss without a GPU: what its entry point refuses, with which status, before anything is launched,
and the plain form that the GPU tests compare with against known values and differences."""
import math

import numpy as np
import pytest

from policy_ref import row_policy

# fake, never dereferenced device addresses
X, D, T, A, B, C, E, F = (0x10000000 * i for i in range(1, 9))


@pytest.fixture(scope="module")
def ss():
    import fsdp_sharded_mixed_ss_gb300 as m
    return m


def test_policy_refusals(ss):
    def call(**kw):
        a = dict(shape=(10, 1000), dtype=ss.SS_BF16, old_logprob=B, ref_logprob=C, kl_coef=0.1, d_logits=D, stream=0)
        a.update(kw)
        ss.ss_policy_loss(a.pop("logits", X), a.pop("tokens", T), a.pop("advantage", A), a.pop("loss", E), **a)

    nan, inf = float("nan"), float("inf")
    for kw, st in [(dict(logits=0), 1), (dict(shape=(-1, 10)), 1), (dict(shape=(2, 0)), 1), (dict(ld=999), 1),
                   (dict(scale=0.0), 1), (dict(scale=nan), 1), (dict(tokens=0), 1), (dict(advantage=0), 1),
                   (dict(clip_low=-0.1), 1), (dict(clip_low=1.5), 1), (dict(clip_low=nan), 1), (dict(clip_high=-1.0), 1),
                   (dict(clip_high=inf), 1), (dict(clip_max=1.0), 1), (dict(clip_max=-2.0), 1), (dict(clip_max=inf), 1),
                   (dict(clip_max=nan), 1), (dict(kl_kind=3), 1), (dict(kl_kind=-1), 1), (dict(kl_coef=nan), 1),
                   (dict(entropy_coef=inf), 1), (dict(ref_logprob=None), 1),
                   (dict(ref_logprob=None, kl_coef=0.0, kl=F), 1), (dict(loss=None, d_logits=None), 1),
                   (dict(dtype=3), 4), (dict(idtype=2), 4), (dict(logits=X + 1), 2), (dict(tokens=T + 4), 2),
                   (dict(advantage=A + 2), 2), (dict(old_logprob=B + 1), 2), (dict(ref_logprob=C + 2), 2),
                   (dict(row_weight=F + 3), 2), (dict(loss=E + 2), 2), (dict(norm=F + 4), 2), (dict(ratio=F + 1), 2),
                   (dict(d_ld=999), 1), (dict(d_logits=X + 2), 3), (dict(d_logits=X, d_ld=1002), 3),
                   (dict(loss=A + 36), 3), (dict(entropy=E), 3), (dict(d_entropy=T + 76), 3), (dict(ld=1 << 60), 5),
                   (dict(shape=(1 << 31, 4)), 5)]:
        with pytest.raises(ss.SSError) as e:
            call(**kw)
        assert e.value.status == st, kw
    call(shape=(0, 1000))                                   # no rows: nothing to do


def test_binding_checks_tensors(ss):
    torch = pytest.importorskip("torch")
    x = torch.zeros(4, 10, dtype=torch.bfloat16)
    f, t = torch.zeros(4), torch.zeros(4, dtype=torch.int64)
    for fn, st in [(lambda: ss.ss_policy_loss(x.t(), t, f, f.clone(), stream=0), 1),
                   (lambda: ss.ss_policy_loss(x, t.short(), f, f.clone(), stream=0), 4),
                   (lambda: ss.ss_policy_loss(x, t[:3], f, f.clone(), stream=0), 1),
                   (lambda: ss.ss_policy_loss(x, t, f.half(), f.clone(), stream=0), 4),
                   (lambda: ss.ss_policy_loss(x, t, f, torch.zeros(5), stream=0), 1),
                   (lambda: ss.ss_policy_loss(x, t, f, norm=torch.zeros(4), stream=0), 1),
                   (lambda: ss.ss_policy_loss(x, t, f, d_logits=x.float(), stream=0), 4),
                   (lambda: ss.ss_policy_loss(x, t, f, f.clone(), kl_kind=2.5, stream=0), 1)]:
        with pytest.raises(ss.SSError) as e:
            fn()
        assert e.value.status == st


def test_plain_form_known_values():
    x = np.log([0.5, 0.25, 0.25])
    o, _, g, _ = row_policy(x, 1.0, 0, 2.0)                                  # ratio 1: -A, and A (p - 1[t])
    assert math.isclose(o["loss"], -2.0) and np.allclose(g, [-1.0, 0.5, 0.5])
    o, _, g, _ = row_policy(x, 1.0, 0, 2.0, old=math.log(0.25))              # ratio 2, clipped at 1.2
    assert math.isclose(o["loss"], -2.4) and not g.any() and math.isclose(o["ratio"], 2.0)
    o, _, g, _ = row_policy(x, 1.0, 0, -2.0, old=math.log(0.25), most=3.0)   # a negative one is not, below 3
    assert math.isclose(o["loss"], 4.0) and np.allclose(g, [2.0, -1.0, -1.0])
    o, _, g, _ = row_policy(x, 1.0, 0, -2.0, old=math.log(0.125), most=3.0)
    assert math.isclose(o["loss"], 6.0) and not g.any()
    o, _, _, _ = row_policy(x, 1.0, 0, 0.0, ref=math.log(0.25), kc=1.0)
    assert math.isclose(o["loss"], 0.5 + math.log(2) - 1) and o["loss"] == o["kl"]
    o, _, _, _ = row_policy(x, 1.0, 0, 0.0, ec=1.0)
    assert math.isclose(o["loss"], -1.5 * math.log(2))


@pytest.mark.parametrize("kind", ["k1", "k2", "k3"])
def test_plain_gradient_against_differences(kind):
    rng = np.random.default_rng(3)
    x, h = rng.normal(size=40) * 2, 1e-6
    lp = x * 0.7 - np.log(np.exp(x * 0.7).sum())
    for adv, gap in [(1.5, 0.1), (-1.5, 0.1), (1.5, 0.3), (-1.5, -0.3), (-1.0, 1.3)]:
        kw = dict(old=lp[5] - gap, ref=lp[5] + 0.4, weight=1.3, most=3.0, kind=kind, kc=0.3, ec=0.2)
        o, _, g, _ = row_policy(x, 0.7, 5, adv, **kw)
        for i in range(40):
            e = np.zeros(40)
            e[i] = h
            slope = (row_policy(x + e, 0.7, 5, adv, **kw)[0]["loss"] - row_policy(x - e, 0.7, 5, adv, **kw)[0]["loss"])
            assert abs(slope / (2 * h) - g[i]) < 1e-7
