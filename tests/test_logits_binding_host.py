"""The binding of the operators on rows of logits without a GPU: addresses and tensors in one call, whatever was called
before."""
import os
import subprocess
import sys

import pytest

pytest.importorskip("torch")

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

# calls on no rows (nothing is launched); ADDRESS is never dereferenced
CALLS = {
    "logprobs": "ss.ss_token_logprobs(ADDRESS, shape=(0, 1000), dtype=ss.SS_BF16, lse=F, stream=0)",
    "logprobs_ids": "ss.ss_token_logprobs(ADDRESS, ADDRESS, idtype=ss.SS_I32, shape=(0, 1000), dtype=ss.SS_BF16,"
                    " top_id=I, top_k=4, stream=0)",
    "logprobs_grad": "ss.ss_token_logprobs_grad(ADDRESS, ADDRESS, X, shape=(0, 1000), dtype=ss.SS_BF16, d_lse=ADDRESS,"
                     " stream=0)",
    "distill": "ss.ss_distill_topk(ADDRESS, ADDRESS, T, ADDRESS, k=4, idtype=ss.SS_I32, shape=(0, 1000),"
               " dtype=ss.SS_BF16, stream=0)",
    "distill_grad": "ss.ss_distill_topk_grad(ADDRESS, ADDRESS, ADDRESS, ADDRESS, X, tail_logprob=F, k=4,"
                    " idtype=ss.SS_I32, tdtype=ss.SS_FP32, shape=(0, 1000), dtype=ss.SS_BF16, stream=0)",
}


@pytest.mark.parametrize("call", CALLS)
def test_addresses_with_tensors_in_the_first_call(call):
    code = ("import torch, fsdp_sharded_mixed_ss_gb300 as ss\n"
            "ADDRESS = 0x10000000\n"
            "F, I, T = torch.zeros(0), torch.zeros((0, 4), dtype=torch.int32), torch.zeros((0, 4))\n"
            "X = torch.zeros((0, 1000), dtype=torch.bfloat16)\n" + CALLS[call])
    p = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True)
    assert p.returncode == 0, p.stderr


def test_what_the_binding_cannot_pass_on_is_refused():
    """With the library's own error, before anything is launched."""
    import torch

    import fsdp_sharded_mixed_ss_gb300 as ss

    x = torch.zeros(4, 10, dtype=torch.bfloat16)
    f, t, ids = torch.zeros(4), torch.zeros(4, 3), torch.zeros(4, 3, dtype=torch.int32)
    at = 0x10000000
    for call in [lambda: ss.ss_token_logprobs(x[0], lse=f, stream=0),
                 lambda: ss.ss_token_logprobs(x.view(2, 2, 10), lse=f, stream=0),
                 lambda: ss.ss_token_logprobs(None, lse=f, stream=0),
                 lambda: ss.ss_token_logprobs(None, shape=(4, 10), dtype=ss.SS_BF16, lse=f, stream=0),
                 lambda: ss.ss_token_logprobs(at, lse=f, dtype=ss.SS_BF16, stream=0),
                 lambda: ss.ss_token_logprobs(at, lse=f, dtype=ss.SS_BF16, shape=(4, 1 << 70), stream=0),
                 lambda: ss.ss_token_logprobs(x, lse=f, scale=1e39, stream=0),
                 lambda: ss.ss_token_logprobs_grad(x, torch.zeros(4, 2), x[0], d_lse=f, stream=0),
                 lambda: ss.ss_distill_topk(x, None, t, f, stream=0),
                 lambda: ss.ss_distill_topk(x, None, t, f, k=3, stream=0),
                 lambda: ss.ss_distill_topk(x, ids, None, f, stream=0),
                 lambda: ss.ss_distill_topk(x, at, t, f, idtype=ss.SS_I32, stream=0),
                 lambda: ss.ss_distill_topk(x, ids, t, f, teacher_scale=1e39, stream=0),
                 lambda: ss.ss_distill_topk(x, ids, t, f, tail=1 << 40, stream=0)]:
        with pytest.raises(ss.SSError) as e:
            call()
        assert e.value.status == 1
