"""The embedding without a GPU: what its entry points refuse, with which status, before anything is launched."""
import os
import re

import pytest

# fake, never dereferenced device addresses
T, I, O, D, W, B = (0x100000000 * i for i in range(1, 7))


@pytest.fixture(scope="module")
def ss():
    import fsdp_sharded_mixed_ss_gb300 as m
    return m


def test_lookup_refusals(ss):
    def call(**kw):
        a = dict(shape=(1000, 64), dtype=ss.SS_BF16, out_dtype=ss.SS_FP32, n=10, stream=0)
        a.update(kw)
        ss.ss_embedding(a.pop("table", T), a.pop("ids", I), a.pop("out", O), **a)

    nan = float("nan")
    for kw, st in [(dict(table=0), 1), (dict(ids=0), 1), (dict(out=0), 1), (dict(n=-1), 1), (dict(shape=(0, 64)), 1),
                   (dict(shape=(10, 0)), 1), (dict(ld=63), 1), (dict(out_ld=63), 1), (dict(scale=nan), 1),
                   (dict(scale=float("inf")), 1), (dict(dtype=3), 4), (dict(out_dtype=-1), 4), (dict(idtype=5), 4),
                   (dict(table=T + 1), 2), (dict(ids=I + 4), 2), (dict(out=O + 2), 2),
                   (dict(shape=(1000, (1 << 24) + 1)), 5), (dict(shape=((1 << 31) - 1, 4)), 5), (dict(n=1 << 31), 5),
                   (dict(ld=1 << 60), 5), (dict(out_ld=1 << 60), 5), (dict(out=T + 127936), 3), (dict(out=I + 76), 3)]:
        with pytest.raises(ss.SSError) as e:
            call(**kw)
        assert e.value.status == st, kw
    call(n=0)                                               # no positions: nothing to do


def test_grad_refusals(ss):
    need = ss.ss_embedding_grad_workspace(10, 1000, 64)

    def call(**kw):
        a = dict(shape=(1000, 64), dtype=ss.SS_BF16, d_dtype=ss.SS_BF16, n=10, workspace_bytes=need, stream=0)
        a.update(kw)
        ss.ss_embedding_grad(a.pop("d_out", D), a.pop("ids", I), a.pop("d_table", T), a.pop("workspace", W), **a)

    nan = float("nan")
    for kw, st in [(dict(d_table=0), 1), (dict(ids=0), 1), (dict(d_out=0), 1), (dict(workspace=0), 1), (dict(n=-1), 1),
                   (dict(shape=(0, 64)), 1), (dict(ld=63), 1), (dict(d_ld=63), 1), (dict(scale=nan), 1),
                   (dict(workspace_bytes=need - 1), 1), (dict(dtype=7), 4), (dict(d_dtype=None), 4), (dict(idtype=-2), 4),
                   (dict(base=B), 4), (dict(base=B, base_dtype=ss.SS_FP32, base_ld=60), 1),
                   (dict(base=B + 2, base_dtype=ss.SS_FP32), 2), (dict(d_table=T + 1), 2), (dict(d_out=D + 1), 2),
                   (dict(ids=I + 2), 2), (dict(workspace=W + 8), 2), (dict(n=1 << 31), 5), (dict(d_ld=1 << 60), 5),
                   (dict(base=T + 2, base_dtype=ss.SS_BF16), 3), (dict(base=T, d_table=T, base_dtype=None, d_out=T), 3),
                   (dict(workspace=T), 3), (dict(ids=W), 3), (dict(d_out=T + 127998), 3)]:
        with pytest.raises(ss.SSError) as e:
            call(**kw)
        assert e.value.status == st, kw
    call(n=0, base=T)                                       # in place and no positions: nothing to do


def test_workspace_sizes(ss):
    assert ss.ss_embedding_grad_workspace(0, 10, 10) >= 0
    assert ss.ss_embedding_grad_workspace(1, 1, 1) > 0
    for bad in ((-1, 10, 10), (1 << 31, 10, 10), (5, 0, 10), (5, 10, 0), (5, 10, (1 << 24) + 1), (5, (1 << 31) - 1, 4)):
        assert ss.ss_embedding_grad_workspace(*bad) == -1
    for dim in (1, 64, 768, 4096, 8192):                    # one for n positions does for fewer
        ns = sorted({*range(200), *(int(1.01 ** i) for i in range(2160)), *range(8000, 8400), 131071, 131072})
        sizes = [ss.ss_embedding_grad_workspace(n, 1000, dim) for n in ns]
        assert sizes == sorted(sizes)


def test_binding_checks_tensors(ss):
    torch = pytest.importorskip("torch")
    t, ids, out = torch.zeros(10, 8), torch.zeros(6, dtype=torch.int64), torch.zeros(6, 8)
    w = torch.zeros(4096, dtype=torch.uint8)
    for fn, st in [(lambda: ss.ss_embedding(t.t(), ids, out, stream=0), 1),
                   (lambda: ss.ss_embedding(t.view(-1), ids, out, stream=0), 1),
                   (lambda: ss.ss_embedding(t.double(), ids, out, stream=0), 4),
                   (lambda: ss.ss_embedding(t, ids.short(), out, stream=0), 4),
                   (lambda: ss.ss_embedding(t, ids[::2], out[:3], stream=0), 1),
                   (lambda: ss.ss_embedding(t, ids, out[:5], stream=0), 1),
                   (lambda: ss.ss_embedding(t, ids, out[:, :7], stream=0), 1),
                   (lambda: ss.ss_embedding(t, ids.view(2, 3), torch.zeros(2, 3, 9)[..., :8], stream=0), 1),
                   (lambda: ss.ss_embedding(t, ids, out.long(), stream=0), 4),
                   (lambda: ss.ss_embedding_grad(out, ids, t, w, base=torch.zeros(9, 8), stream=0), 1),
                   (lambda: ss.ss_embedding_grad(out, ids, t, w[:64], stream=0), 1),
                   (lambda: ss.ss_embedding_grad(out, ids, t, None, stream=0), 1),
                   (lambda: ss.ss_embedding_grad(out, ids, t, W, stream=0), 1),
                   (lambda: ss.ss_embedding_grad(out[:1].expand(6, 8), ids, t, w, stream=0), 1)]:
        with pytest.raises(ss.SSError) as e:
            fn()
        assert e.value.status == st


def test_header_constants(ss):
    text = open(os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "ss.h")).read()
    assert int(re.search(r"#define SS_MAX_DIM (\d+)", text).group(1)) == ss.SS_MAX_DIM
    for group in (r"SS_KL_K1 = (\d), SS_KL_K2 = (\d), SS_KL_K3 = (\d)",
                  r"SS_PREF_SIGMOID = (\d), SS_PREF_HINGE = (\d), SS_PREF_SQUARE = (\d)"):
        assert re.search(group, text).groups() == ("0", "1", "2")
    assert (ss.SS_KL_K1, ss.SS_KL_K2, ss.SS_KL_K3) == (ss.SS_PREF_SIGMOID, ss.SS_PREF_HINGE, ss.SS_PREF_SQUARE) == (0, 1, 2)
