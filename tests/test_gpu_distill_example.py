"""The example that runs the operators on rows of logits together with the shard step, and one of its steps against the
plain float64 rows."""
import importlib.util
import os

import numpy as np
import pytest

from logits_ref import REL, grad_bound, row_distill

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def _example():
    spec = importlib.util.spec_from_file_location("distill_head", os.path.join(ROOT, "examples", "distill_head.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def test_distillation_learns():
    means, before, after = _example().train(steps=25, vocab=2003, dim=64, rows=128, n_ranks=3, top=16, lr=1e-2)
    assert means[-1] < 0.5 * means[0], means
    assert after > before + 1.0


def test_one_step_against_the_plain_rows():
    """The teacher's pass, the student's logits and the gradient that replaces them, as the example runs them."""
    import fsdp_sharded_mixed_ss_gb300 as ss

    ex = _example()
    dev, rows, vocab, dim, top = "cuda", 24, 1009, 32, 12
    student = ex.Head(vocab, dim, 2, dev, seed=3)
    g = torch.Generator(device=dev)
    g.manual_seed(5)
    h = torch.randn((rows, dim), generator=g, device=dev).to(torch.bfloat16)
    t = torch.randn((rows, vocab), generator=g, device=dev)
    ids = torch.empty((rows, top), dtype=torch.int32, device=dev)
    lps = torch.empty((rows, top), device=dev)
    ss.ss_token_logprobs(t, top_logprob=lps, top_id=ids)
    z = h @ student.weight.t()
    x = z.double().cpu().numpy()
    loss = torch.empty(rows, device=dev)
    ss.ss_distill_topk(z, ids, lps, loss, d_logits=z)
    torch.cuda.synchronize()
    got, lists, q = z.double().cpu().numpy(), ids.tolist(), lps.double().cpu().numpy()
    for r in range(rows):
        ref, _, grad, terms, size = row_distill(x[r], 1.0, lists[r], q[r], 1.0, "bucket", 1.0)
        assert abs(float(loss[r]) - ref) <= 4 * REL * size
        assert (np.abs(got[r] - grad) <= grad_bound(grad, terms, "bf16")).all()
