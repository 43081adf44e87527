"""Each form of the kernels' bounded wait, alone: on a phase that nothing completes it gives up after its
limit, returns false, raises the abort flag (the clean-up wait does not), and is reported once."""

import pytest
import torch

import quantized_block_sparse_attn_b200 as qb
from quantized_block_sparse_attn_b200._binding import _ptr, _stream

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("form,abort", [(0, 1), (1, 0), (2, 1), (3, 1)])
def test_a_wait_that_runs_out(form, abort):
    L, dev = qb.lib(), torch.device("cuda:0")
    result = torch.full((3,), -1, dtype=torch.int64, device=dev)
    assert L.qbsa_check(_stream(dev)) == 0
    assert L.qbsa_wait_selftest_form(form, _ptr(result), _stream(dev)) == 0
    assert L.qbsa_check(_stream(dev)) == 4                # QBSA_ERR_TIMEOUT
    assert b"time limit" in L.qbsa_last_error()
    assert L.qbsa_check(_stream(dev)) == 0                # cleared
    done, flag, ns = result.tolist()
    assert (done, flag) == (0, abort)
    assert 1.99e9 <= ns <= 4e9                            # the limit is 2 s, a suspended poll at most about 1 ms


def test_the_context_survives():
    x = torch.ones((3, 64), dtype=torch.bfloat16, device="cuda")
    codes, scales = qb.quantize_token(x)
    qb.check()
    assert torch.all(codes == 127) and torch.allclose(scales, torch.full_like(scales, 1 / 127), rtol=2 ** -23, atol=0)
