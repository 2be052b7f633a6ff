"""The operators on rows of logits without a GPU: what their entry points refuse, with which status, before
anything is launched, and the plain forms that the GPU tests compare with against known values."""
import math

import numpy as np
import pytest

from logits_ref import row_distill, row_logprobs, row_logprobs_grad

# fake, never dereferenced device addresses
X, D, T, A, B, C, E, F = (0x10000000 * i for i in range(1, 9))


@pytest.fixture(scope="module")
def ss():
    import fsdp_sharded_mixed_ss_gb300 as m
    return m


def _status(ss, fn, kw):
    with pytest.raises(ss.SSError) as e:
        fn(**kw)
    return e.value.status


def test_logprobs_refusals(ss):
    def call(**kw):
        a = dict(shape=(10, 1000), dtype=ss.SS_BF16, logprob=A, entropy=B, norm=C, top_logprob=E, top_id=F, top_k=4,
                 stream=0)
        a.update(kw)
        ss.ss_token_logprobs(a.pop("logits", X), a.pop("tokens", T), **a)

    for kw, st in [(dict(logits=0), 1), (dict(shape=(-1, 10)), 1), (dict(shape=(2, 0)), 1), (dict(ld=999), 1),
                   (dict(scale=0.0), 1), (dict(scale=-1.0), 1), (dict(scale=float("nan")), 1),
                   (dict(scale=float("inf")), 1), (dict(scale=3e38), 1), (dict(dtype=3), 4), (dict(idtype=2), 4),
                   (dict(top_k=129), 1), (dict(top_k=-1), 1), (dict(top_k=0), 1), (dict(shape=(10, 3)), 1),
                   (dict(top_logprob=None, top_id=None), 1), (dict(tokens=None), 1),
                   (dict(logprob=None, entropy=None, norm=None, top_logprob=None, top_id=None, top_k=0), 1),
                   (dict(logits=X + 1), 2), (dict(logprob=A + 2), 2), (dict(norm=C + 4), 2), (dict(top_id=F + 4), 2),
                   (dict(tokens=T + 4), 2), (dict(entropy=A + 36), 3), (dict(logprob=X + 19996), 3),
                   (dict(top_id=T + 72), 3), (dict(ld=1 << 60), 5)]:
        assert _status(ss, call, kw) == st, kw
    call(shape=(0, 1000))                                   # no rows: nothing to do


def test_logprobs_grad_refusals(ss):
    def call(**kw):
        a = dict(shape=(10, 1000), dtype=ss.SS_FP32, tokens=T, d_logprob=A, stream=0)
        a.update(kw)
        ss.ss_token_logprobs_grad(a.pop("logits", X), a.pop("norm", C), a.pop("d_logits", D), **a)

    for kw, st in [(dict(norm=None), 1), (dict(d_logits=None), 1), (dict(tokens=None), 1), (dict(d_logprob=None), 1),
                   (dict(d_entropy=B), 1), (dict(d_top_logprob=B), 1), (dict(d_top_logprob=B, top_k=3), 1),
                   (dict(d_ld=999), 1), (dict(d_logits=D + 2), 2), (dict(norm=C + 4), 2), (dict(d_logits=X + 4), 3),
                   (dict(d_logits=X, d_ld=1001), 3), (dict(d_logprob=D + 400), 3), (dict(dtype=5), 4)]:
        assert _status(ss, call, kw) == st, kw
    call(shape=(0, 1000))


def test_distill_refusals(ss):
    def call(**kw):
        a = dict(shape=(10, 1000), dtype=ss.SS_FP16, tdtype=ss.SS_FP32, idtype=ss.SS_I32, k=8, loss=A, d_logits=D,
                 stream=0)
        a.update(kw)
        ss.ss_distill_topk(a.pop("logits", X), a.pop("ids", T), a.pop("teacher", E), **a)

    for kw, st in [(dict(ids=0), 1), (dict(teacher=0), 1), (dict(k=0), 1), (dict(k=129), 1), (dict(tail=3), 1),
                   (dict(teacher_scale=0.0), 1), (dict(teacher_scale=float("inf")), 1), (dict(tdtype=None), 4),
                   (dict(idtype=7), 4), (dict(loss=None, d_logits=None), 1), (dict(shape=(10, 393217)), 5),
                   (dict(teacher=E + 2), 2), (dict(ids=T + 2), 2), (dict(row_weight=B + 1), 2),
                   (dict(norm=B + 4), 2), (dict(loss=E + 316), 3), (dict(d_logits=X + 2), 3),
                   (dict(tail_logprob=A), 3), (dict(scale=0.0), 1)]:
        assert _status(ss, call, kw) == st, kw
    call(shape=(0, 1000))

    def grad(**kw):
        a = dict(shape=(10, 1000), dtype=ss.SS_FP16, tdtype=ss.SS_FP32, idtype=ss.SS_I32, k=8, tail_logprob=B,
                 stream=0)
        a.update(kw)
        ss.ss_distill_topk_grad(X, T, E, a.pop("norm", C), a.pop("d_logits", D), **a)

    for kw, st in [(dict(norm=None), 1), (dict(d_logits=None), 1), (dict(tail_logprob=None), 1),
                   (dict(d_loss=A + 1), 2), (dict(d_loss=D), 3), (dict(tail=-1, tail_logprob=None), 1)]:
        assert _status(ss, grad, kw) == st, kw
    grad(shape=(0, 1000))


def test_binding_checks_tensors(ss):
    torch = pytest.importorskip("torch")
    x = torch.zeros(4, 10, dtype=torch.bfloat16)
    f = torch.zeros(4)
    ids = torch.zeros(4, 3, dtype=torch.int32)
    for fn, st in [(lambda: ss.ss_token_logprobs(x.t(), lse=f, stream=0), 1),
                   (lambda: ss.ss_token_logprobs(x.double(), lse=f, stream=0), 4),
                   (lambda: ss.ss_token_logprobs(x, lse=f.half(), stream=0), 4),
                   (lambda: ss.ss_token_logprobs(x, lse=torch.zeros(3), stream=0), 1),
                   (lambda: ss.ss_token_logprobs(x, lse=torch.zeros(8)[::2], stream=0), 1),
                   (lambda: ss.ss_token_logprobs(x, f, logprob=f.clone(), stream=0), 4),
                   (lambda: ss.ss_token_logprobs(x, ids[:, 0].contiguous(), logprob=f, top_id=ids.long(), stream=0), 4),
                   (lambda: ss.ss_distill_topk(x, ids, torch.zeros(4, 3), f, d_logits=x.float(), stream=0), 4),
                   (lambda: ss.ss_distill_topk(x, ids, torch.zeros(4, 3), f, d_logits=x[:, :9], stream=0), 1),
                   (lambda: ss.ss_distill_topk(x, ids, torch.zeros(4, 2), f, stream=0), 1),
                   (lambda: ss.ss_distill_topk(x, ids, torch.zeros(4, 3, dtype=torch.float64), f, stream=0), 4),
                   (lambda: ss.ss_token_logprobs(x[:1].expand(4, 10), lse=f, stream=0), 1)]:
        with pytest.raises(ss.SSError) as e:
            fn()
        assert e.value.status == st


def test_header_constants(ss):
    import os
    import re

    text = open(os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "ss.h")).read()
    for name in ("SS_MAX_TOP", "SS_MAX_DISTILL_VOCAB"):
        assert int(re.search(rf"#define {name} (\d+)", text).group(1)) == getattr(ss, name)


def test_plain_forms_known_values():
    o = row_logprobs(np.zeros(8), 1.0, 3, 2)
    assert math.isclose(o["logprob"], -math.log(8)) and math.isclose(o["entropy"], math.log(8))
    assert o["top_id"].tolist() == [0, 1]
    o = row_logprobs(np.array([0.0, math.log(3.0)]), 1.0, 1, 1)
    assert math.isclose(o["logprob"], math.log(0.75)) and math.isclose(o["lse"], math.log(4.0))
    # teacher (1/2, 1/4 listed, 1/4 left), student (1/4 each of 4): KL over (a, b, rest)
    x = np.zeros(4)
    lq = np.log([0.5, 0.25])
    loss, lpt, g, *_ = row_distill(x, 1.0, [0, 1], lq, 1.0, "bucket", 1.0)
    assert math.isclose(loss, 0.5 * math.log(2) + 0.25 * math.log(1) + 0.25 * math.log(0.5))
    assert math.isclose(lpt, math.log(0.5)) and np.allclose(g, [-0.25, 0.0, 0.125, 0.125])
    loss, _, g, *_ = row_distill(x, 1.0, [0, 1], lq, 1.0, "renorm", 1.0)
    assert math.isclose(loss, 2 / 3 * math.log(8 / 3) + 1 / 3 * math.log(4 / 3))
    assert np.allclose(g, [0.25 - 2 / 3, 0.25 - 1 / 3, 0.25, 0.25])


@pytest.mark.parametrize("mode", ["drop", "renorm", "bucket"])
def test_plain_gradients_against_differences(mode):
    rng = np.random.default_rng(3)
    x, h = rng.normal(size=40) * 2, 1e-6
    ids = [3, 9, 31]
    lq = np.log([0.4, 0.2, 0.1])
    g = row_distill(x, 0.7, ids, lq, 1.0, mode, 1.3)[2]
    gp, _ = row_logprobs_grad(x, 0.7, token=5, d_logprob=1.5, d_entropy=-0.5, d_lse=0.25, top_id=[2, 5], d_top=[1, -2])

    def both(y):
        o = row_logprobs(y, 0.7, 5, 0)
        z = y * 0.7
        lp = z - np.log(np.exp(z).sum())
        return (row_distill(y, 0.7, ids, lq, 1.0, mode, 1.3)[0],
                1.5 * o["logprob"] - 0.5 * o["entropy"] + 0.25 * o["lse"] + lp[2] - 2 * lp[5])

    for i in range(40):
        e = np.zeros(40)
        e[i] = h
        (a, b), (c, d) = both(x + e), both(x - e)
        assert abs((a - c) / (2 * h) - g[i]) < 1e-7 and abs((b - d) / (2 * h) - gp[i]) < 1e-7
