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
