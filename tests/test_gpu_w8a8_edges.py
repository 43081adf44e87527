"""GPU cases of the 8-bit linear layers at the ends of their ranges: magnitudes whose squares leave float32,
rows with gaps between them in large numbers, every quotient of short significands, empty tensors.

Tolerances as in test_gpu_w8a8: codes bit for bit; scales within ((terms + 10) / 2 + 6) half steps of
float32, terms = max(32, width / 1024 + 16).  A sum taken again of scaled values adds no rounding: the
scaling is by a power of two, and what it pushes below float32's range is 2^-100 of the row's sum.
"""

import pytest
import torch

import quantized_block_sparse_attn_b200 as qb
from tests.test_gpu_w8a8 import BF16, FP16, FP32, _check_tokens, _randn

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("rows,width", [(5, 1), (6, 72), (6, 1000), (6, 1031), (6, 5120), (6, 33000), (2500, 1024),
                                        (2500, 1031), (2500, 5120)])
@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("residual", [False, True])
def test_rows_up_to_the_largest_values(rows, width, dtype, residual):
    """Finite rows whose squares overflow by far: rows of the type's largest value, weights that leave the
    step small, one large value among small ones."""
    top = torch.finfo(dtype).max
    x = _randn(width, (rows, width), dtype)
    x[0] = top
    x[1] = (x[1].float() / x[1].float().abs().max() * 3e38).to(dtype)
    x[2] *= 1e25
    x[-2, width // 2] = -top
    x[-1] = -top
    res = torch.zeros_like(x) if residual else None
    for w in (torch.ones(width, dtype=FP32, device="cuda"), _randn(3, (width,), FP32).clamp_(-1, 1),
              torch.full((width,), 1e-27, device="cuda")):
        codes, scales, _ = qb.rms_norm_quant(x, w, residual=res)
        qb.check()
        _check_tokens(codes, scales, x, w, 1e-6)


@pytest.mark.parametrize("width", [1, 64, 1031, 33000])
def test_mean_and_eps_that_overflow_together(width):
    x = _randn(5, (4, width), FP32)
    x[1] = 1e19
    x[2] = 1.8e19 / width ** 0.5
    w = torch.ones(width, device="cuda")
    for eps in (3e38, 1e30, 2.0 ** -126):
        codes, scales, _ = qb.rms_norm_quant(x, w, eps)
        qb.check()
        _check_tokens(codes, scales, x, w, float(torch.tensor(eps, dtype=FP32)))
