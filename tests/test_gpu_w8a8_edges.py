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


@pytest.mark.parametrize("lead", [(0,), (0, 3), (3, 0), (2, 0, 1), (2, 1, 0)])
def test_empty_batches(lead):
    """No tokens, wherever the empty dimension stands, with outputs made and given."""
    x, w = torch.empty((*lead, 48), dtype=BF16, device="cuda"), _randn(2, (48,), BF16)
    b, sb = qb.quantize_token(_randn(1, (40, 48), BF16))
    for given in (False, True):
        kw = dict(codes=torch.empty((*lead, 48), dtype=torch.int8, device="cuda"),
                  scales=torch.empty(lead, device="cuda")) if given else {}
        c, s, h = qb.rms_norm_quant(x, w, residual=x, residual_out=torch.empty_like(x) if given else None, **kw)
        assert c.shape == x.shape and s.shape == lead and h.shape == x.shape
        c, s = qb.quantize_token(x, **kw)
        assert c.shape == x.shape and s.shape == lead
        out = torch.empty((*lead, 40), dtype=BF16, device="cuda") if given else None
        assert qb.matmul_i8(c, b, s, sb, out=out).shape == (*lead, 40)
    qb.check()
