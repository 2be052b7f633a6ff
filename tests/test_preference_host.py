"""The preference loss without a GPU: what its entry point refuses, with which status, before anything is launched, and the
plain form that the GPU tests compare with against known values and differences."""
import math

import numpy as np
import pytest

from preference_ref import preference

# fake, never dereferenced device addresses
L, O, R, W, P, A, B, D = (0x10000000 * i for i in range(1, 9))


@pytest.fixture(scope="module")
def ss():
    import fsdp_sharded_mixed_ss_gb300 as m
    return m


def test_preference_refusals(ss):
    def call(**kw):
        a = dict(rows=1000, pairs=10, ref_logprob=R, row_weight=W, pair_weight=P, reward=B, d_logprob=D, stream=0)
        a.update(kw)
        ss.ss_preference_loss(a.pop("logprob", L), a.pop("offsets", O), a.pop("loss", A), **a)

    nan, inf = float("nan"), float("inf")
    for kw, st in [(dict(logprob=0), 1), (dict(offsets=0), 1), (dict(rows=-1), 1), (dict(pairs=-1), 1),
                   (dict(loss=None, reward=None, d_logprob=None), 1), (dict(kind=3), 1), (dict(kind=-1), 1),
                   (dict(beta=0.0), 1), (dict(beta=-1.0), 1), (dict(beta=nan), 1), (dict(beta=inf), 1),
                   (dict(margin=nan), 1), (dict(margin=inf), 1), (dict(label_smoothing=-0.1), 1),
                   (dict(label_smoothing=1.1), 1), (dict(label_smoothing=0.1, kind=ss.SS_PREF_HINGE), 1),
                   (dict(label_smoothing=nan), 1), (dict(idtype=2), 4), (dict(pairs=1 << 28), 5), (dict(rows=1 << 61), 5),
                   (dict(logprob=L + 2), 2), (dict(offsets=O + 4), 2), (dict(ref_logprob=R + 1), 2),
                   (dict(row_weight=W + 2), 2), (dict(pair_weight=P + 2), 2), (dict(loss=A + 2), 2),
                   (dict(reward=B + 4), 2), (dict(d_logprob=D + 1), 2), (dict(d_logprob=L), 3), (dict(loss=L + 3996), 3),
                   (dict(reward=A + 32), 3), (dict(loss=O + 164), 3), (dict(d_logprob=W), 3)]:
        with pytest.raises(ss.SSError) as e:
            call(**kw)
        assert e.value.status == st, kw
    call(pairs=0)                                           # no pairs: nothing to do


def test_binding_checks_tensors(ss):
    torch = pytest.importorskip("torch")
    lp, o, f = torch.zeros(20), torch.zeros(5, dtype=torch.int64), torch.zeros(2)
    for fn, st in [(lambda: ss.ss_preference_loss(lp.half(), o, f, stream=0), 4),
                   (lambda: ss.ss_preference_loss(lp, o.short(), f, stream=0), 4),
                   (lambda: ss.ss_preference_loss(lp, o[:4], f, stream=0), 1),
                   (lambda: ss.ss_preference_loss(lp, o[:0], f, stream=0), 1),
                   (lambda: ss.ss_preference_loss(lp, o, torch.zeros(3), stream=0), 1),
                   (lambda: ss.ss_preference_loss(lp, o, reward=f, stream=0), 1),
                   (lambda: ss.ss_preference_loss(lp, o, f, row_weight=torch.zeros(19), stream=0), 1),
                   (lambda: ss.ss_preference_loss(torch.zeros(40)[::2], o, f, stream=0), 1),
                   (lambda: ss.ss_preference_loss(lp, o, f, beta="no", stream=0), 1),
                   (lambda: ss.ss_preference_loss(L, o, f, stream=0), 1)]:
        with pytest.raises(ss.SSError) as e:
            fn()
        assert e.value.status == st


def test_plain_form_known_values():
    lp, off = np.array([-1.0, -1.0, -3.0, 7.0]), [0, 2, 3]
    o = preference(lp, off, beta=1.0)                        # h = -2 + 3 = 1
    assert math.isclose(o["loss"][0][0], math.log(1 + math.exp(-1)))
    g = 1 / (1 + math.e)
    assert np.allclose(o["d_logprob"][0][:3], [-g, -g, g]) and o["outside"].tolist() == [False] * 3 + [True]
    assert np.allclose(o["reward"][0], [[-2.0, -3.0]])
    o = preference(lp, off, beta=1.0, average=True, kind="hinge", margin=0.5)   # h = -1 + 3 - 0.5
    assert o["loss"][0][0] == 0.0
    o = preference(lp, off, beta=0.5, kind="square", ref=[-1, 0, -2, 0])        # chosen -1, rejected -1: h = 0
    assert math.isclose(o["loss"][0][0], 1.0) and np.allclose(o["d_logprob"][0][:3], [-2, -2, 2])


@pytest.mark.parametrize("kind", ["sigmoid", "hinge", "square"])
@pytest.mark.parametrize("average,halves", [(False, False), (True, True)])
def test_plain_gradient_against_differences(kind, average, halves):
    rng = np.random.default_rng(1)
    off = [0, 5, 9, 9, 16]
    lp, w = -rng.exponential(size=18), rng.uniform(0.2, 2, size=18)
    w[3] = 0.0
    kw = dict(weight=w, ref=lp + rng.normal(size=18) * 0.3, pair_weight=[0.5, 2.0], kind=kind, beta=0.7, margin=0.1,
              smooth=0.2 if kind == "sigmoid" else 0.0, average=average, halves=halves)
    o = preference(lp, off, **kw)
    for i in range(18):
        e = np.zeros(18)
        e[i] = 1e-6
        slope = (preference(lp + e, off, **kw)["loss"][0].sum() - preference(lp - e, off, **kw)["loss"][0].sum()) / 2e-6
        want = o["d_logprob"][0][i]
        assert abs(slope - (0.0 if np.isnan(want) else want)) < 1e-6
