"""GPU parity of the 8-bit linear layers (rms_norm_quant, quantize_token, matmul_i8) against the
float64 oracle, and the layer they make with the quantized attention.

Tolerances.  u = 2^-24 is half a step of float32.
- codes: equal to the float32 steps of the definition, bit for bit; and within half a code plus
  3 * 127 * u of the float64 quotient (g, a / 127 and the quotient are each rounded once).
- scale without a norm: 2 u relative (the product g and the division).  With the norm the sum of n
  squares adds at most (terms in a row of additions) * u, halved by the root; each thread adds at most
  max(32, width / 1024 + 16) squares in a row, the joins are 10 more, and the mean, eps, root and last
  division are one rounding each: bound (terms + 10) / 2 + 6.
- product: the sum is exact; its rounding to float32, the product with a_scale and the last multiply-add
  are 3 u of |product| + |bias|, then half a step of the output's type.
"""

import os
import subprocess
import sys
import threading

import numpy as np
import pytest
import torch

import quantized_block_sparse_attn_b200 as qb
from oracle import linear8

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
BF16, FP16, FP32 = torch.bfloat16, torch.float16, torch.float32


def _np(t):
    return t.double().cpu().numpy()


def _randn(seed, shape, dtype, scale=1.0):
    rng = np.random.default_rng(seed)
    return torch.from_numpy((rng.standard_normal(shape) * scale).astype(np.float32)).to(dtype).cuda()


def _check_tokens(codes, scales, h, weight=None, eps=None):
    """codes, scales against the definition for stored rows h [R, W]."""
    hn = _np(h)
    wn = None if weight is None else _np(weight)
    got = codes.cpu().numpy()
    q, _, _ = linear8.token_quotients(hn, wn)
    assert np.abs(got - q).max() <= 0.5 + 3 * 127 * U * 1.01
    assert np.array_equal(got, linear8.token_codes_f32(hn, wn))
    want = linear8.token_scales(hn, wn, eps)
    terms = max(32, hn.shape[-1] / 1024 + 16)
    bound = 2 * U if eps is None else ((terms + 10) / 2 + 6) * U
    err = np.abs(scales.double().cpu().numpy() - want)
    assert np.all(err <= bound * 1.01 * want), float((err / want).max())


WIDTHS = [1, 2, 7, 8, 9, 63, 64, 128, 250, 255, 256, 257, 511, 512, 513, 520, 1024, 1031, 2047, 2048, 4096, 5120, 8191,
          8192, 8200, 16384, 16392, 20480]


@pytest.mark.parametrize("width", WIDTHS)
@pytest.mark.parametrize("dtype,wdtype", [(BF16, BF16), (FP16, FP32), (FP32, FP32)])
def test_rms_norm_quant_widths(width, dtype, wdtype):
    rows = 5 if width > 512 else 37
    x, res = _randn(width, (rows, width), dtype), _randn(width + 1, (rows, width), dtype, 3.0)
    w = _randn(width + 2, (width,), wdtype)
    codes, scales, h = qb.rms_norm_quant(x, w, 1e-5, residual=res)
    assert codes.stride(0) % 16 == 0
    assert torch.equal(h, (x.float() + res.float()).to(dtype))
    _check_tokens(codes, scales, h, w, 1e-5)
    codes, scales, none = qb.rms_norm_quant(x, w, 1e-5)
    assert none is None
    _check_tokens(codes, scales, x, w, 1e-5)
    codes, scales = qb.quantize_token(x)
    _check_tokens(codes, scales, x)


@pytest.mark.parametrize("dtype", [BF16, FP16, FP32])
@pytest.mark.parametrize("width", [40001, 65536])
def test_rows_wider_than_registers(width, dtype):
    x, res = _randn(1, (3, width), dtype), _randn(2, (3, width), dtype)
    w = _randn(3, (width,), FP32)
    codes, scales, h = qb.rms_norm_quant(x, w, residual=res)
    _check_tokens(codes, scales, h, w, 1e-6)
    codes, scales = qb.quantize_token(x)
    _check_tokens(codes, scales, x)


@pytest.mark.parametrize("rows", [1, 2, 3, 31, 148, 1000])
def test_row_counts(rows):
    for width in (64, 96, 1280):
        x, w = _randn(rows, (rows, width), BF16), _randn(9, (width,), BF16)
        codes, scales, _ = qb.rms_norm_quant(x, w)
        _check_tokens(codes, scales, x, w, 1e-6)


@pytest.mark.parametrize("width", [128, 130, 264, 512, 513, 520, 1024, 1031, 2047, 4096, 5120, 8193, 12000, 20480, 20481])
@pytest.mark.parametrize("dtype,residual", [(BF16, True), (BF16, False), (FP16, True), (FP32, True), (FP32, False)])
def test_more_rows_than_run_at_once(width, dtype, residual):
    """Rows past one per resident CTA (streamed through shared memory), from tensors that start and end
    off a 16-byte boundary where the width is odd; with and without a norm."""
    rows = 2500 if width <= 5120 else 500
    pool = _randn(width, (rows * width + 3,), dtype)
    off = 3 if width % 8 else 0
    x = pool[off:off + rows * width].view(rows, width)
    res = _randn(width + 1, (rows, width), dtype) if residual else None
    w = _randn(width + 2, (width,), dtype)
    keep = pool.clone()
    codes, scales, h = qb.rms_norm_quant(x, w, residual=res)
    qb.check()
    assert torch.equal(pool, keep)
    if residual:
        assert torch.equal(h, (x.float() + res.float()).to(dtype))
    _check_tokens(codes, scales, h if residual else x, w, 1e-6)
    if residual:                                          # in place, and the squares of one row overflow
        if dtype != FP16:
            x[rows // 2] *= 1e30
        h = (x.float() + res.float()).to(dtype)
        codes, scales, got = qb.rms_norm_quant(x, w, residual=res, residual_out=x)
        assert got.data_ptr() == x.data_ptr() and torch.equal(x, h)
        assert torch.equal(pool[:off], keep[:off]) and torch.equal(pool[off + rows * width:], keep[off + rows * width:])
        _check_tokens(codes, scales, h, w, 1e-6)
    else:
        codes, scales = qb.quantize_token(x)
        _check_tokens(codes, scales, x)
    qb.check()


@pytest.mark.parametrize("dtype", [BF16, FP16])
def test_every_short_quotient(dtype):
    """Rows of a 16-bit type whose largest value takes every significand, with every smaller significand at
    every exponent that reaches a code: half-integer quotients among them."""
    bits = 7 if dtype == BF16 else 10
    n = 1 << bits
    tops = torch.arange(n, 2 * n, device="cuda", dtype=torch.float32)
    if dtype == FP16:
        tops = tops[::8]
    all_x = torch.cat([torch.arange(n, 2 * n, device="cuda", dtype=torch.float32) * 2.0 ** -j for j in range(9)])
    for scale in (1.0, 2.0 ** -8, 2.0 ** 5) if dtype == FP16 else (1.0, 2.0 ** -100, 2.0 ** 100):
        rows = torch.where(all_x[None] <= tops[:, None], all_x[None], torch.zeros((), device="cuda"))
        rows = (torch.cat([tops[:, None], rows], 1) * scale).to(dtype)
        codes, scales = qb.quantize_token(rows)
        _check_tokens(codes, scales, rows)


@pytest.mark.parametrize("width,off,pitch", [(64, 0, 80), (64, 1, 80), (130, 0, 136), (130, 3, 137), (1024, 8, 2048),
                                             (1024, 5, 1031), (5120, 0, 5128)])
@pytest.mark.parametrize("dtype", [BF16, FP32])
def test_strided_rows_and_what_lies_between_them(width, off, pitch, dtype):
    rows = 6
    big = _randn(7, (rows, off + pitch), dtype)
    x = big[:, off:off + width]
    r = _randn(8, (rows, off + pitch), dtype)
    res = r[:, off:off + width]
    w = _randn(10, (width,), dtype)
    hbuf = torch.full((rows + 1, off + pitch), 7.0, dtype=dtype, device="cuda")
    cbuf = torch.full((rows + 1, off + pitch), 77, dtype=torch.int8, device="cuda")
    h, codes = hbuf[:rows, off:off + width], cbuf[:rows, off:off + width]
    keep_x, keep_r = big.clone(), r.clone()
    _, scales, got = qb.rms_norm_quant(x, w, residual=res, residual_out=h, codes=codes)
    assert got.data_ptr() == h.data_ptr()
    _check_tokens(codes, scales, (x.float() + res.float()).to(dtype), w, 1e-6)
    assert torch.equal(h, (x.float() + res.float()).to(dtype))
    assert torch.equal(big, keep_x) and torch.equal(r, keep_r)
    for buf, value in ((hbuf, 7.0), (cbuf, 77)):
        outside = torch.ones_like(buf, dtype=torch.bool)
        outside[:rows, off:off + width] = False
        assert torch.all(buf[outside] == value)


@pytest.mark.parametrize("target", ["residual", "x"])
@pytest.mark.parametrize("width", [96, 1031, 5120, 33000])
def test_residual_in_place(target, width):
    x, res, w = _randn(1, (9, width), BF16), _randn(2, (9, width), BF16), _randn(3, (width,), BF16)
    want = qb.rms_norm_quant(x, w, residual=res)
    got = qb.rms_norm_quant(x, w, residual=res, residual_out=res if target == "residual" else x)
    for g, e in zip(got, want):
        assert torch.equal(g, e)


@pytest.mark.parametrize("dtype", [BF16, FP16, FP32])
@pytest.mark.parametrize("width", [72, 1000, 1031, 33000])
def test_rows_without_values_and_rows_that_are_no_numbers(width, dtype):
    x = _randn(4, (8, width), dtype)
    w = _randn(5, (width,), FP32)
    x[1] = 0
    x[2, width // 2] = float("nan")
    x[3, width - 1] = float("inf")
    x[4, 0] = float("-inf")
    x[5] = torch.finfo(dtype).tiny / 8                   # subnormal, or 0 where the type rounds it away
    x[6] = -x[0]
    bad = [2, 3, 4]
    good = [0, 1, 5, 6, 7]
    for norm in (True, False):
        codes, scales = qb.rms_norm_quant(x, w)[:2] if norm else qb.quantize_token(x)
        assert torch.all(codes[bad] == 0) and torch.all(torch.isnan(scales[bad]))
        assert torch.all(codes[1] == 0) and scales[1] == 1.0
        _check_tokens(codes[good], scales[good], x[good], w if norm else None, 1e-6 if norm else None)
        assert torch.equal(codes[6], -codes[0]) and scales[6] == scales[0]
    # a weight that is no number makes every row one
    w[width // 3] = float("nan")
    codes, scales, _ = qb.rms_norm_quant(x, w)
    assert torch.all(codes == 0) and torch.all(torch.isnan(scales))


@pytest.mark.parametrize("width", [72, 1000, 1031, 33000])
@pytest.mark.parametrize("residual", [False, True])
def test_squares_that_overflow(width, residual):
    x = _randn(6, (5, width), BF16)
    x[1] *= 1e25
    x[3] *= 1e36
    w = _randn(7, (width,), FP32, 0.5)
    res = torch.zeros_like(x) if residual else None
    codes, scales, _ = qb.rms_norm_quant(x, w, residual=res)
    _check_tokens(codes, scales, x, w, 1e-6)


def test_leading_dimensions_and_one_row():
    x, w = _randn(1, (2, 3, 40), BF16), _randn(2, (40,), BF16)
    codes, scales, h = qb.rms_norm_quant(x, w, residual=x)
    assert codes.shape == x.shape and scales.shape == (2, 3) and h.shape == x.shape
    _check_tokens(codes.reshape(6, 40), scales.reshape(6), h.reshape(6, 40), w, 1e-6)
    c1, s1, _ = qb.rms_norm_quant(x[1, 2], w)
    assert c1.shape == (40,) and s1.shape == ()
    _check_tokens(c1[None], s1[None], x[1, 2][None], w, 1e-6)
    c0, s0 = qb.quantize_token(x[:0])
    assert c0.shape == (0, 3, 40) and s0.shape == (0, 3)
    # one row for every token, by a row stride of 0
    c, s = qb.quantize_token(x[0, 0].expand(4, 40))
    _check_tokens(c, s, x[0, 0].expand(4, 40))


def test_rows_that_overlap_in_memory():
    """Windows over one buffer, by a row stride below the width (inputs only)."""
    pool = _randn(1, (40000,), BF16)
    w = _randn(2, (520,), BF16)
    for stride, rows in ((8, 3000), (3, 3000), (1, 50), (0, 5)):
        x = pool.as_strided((rows, 520), (stride, 1))
        codes, scales, _ = qb.rms_norm_quant(x, w)
        _check_tokens(codes, scales, x, w, 1e-6)
        codes, scales, h = qb.rms_norm_quant(x, w, residual=x)
        _check_tokens(codes, scales, h, w, 1e-6)
    qb.check()


@pytest.mark.parametrize("dtype,wdtype", [(BF16, FP32), (FP16, FP16), (FP32, FP32)])
@pytest.mark.parametrize("rows", [3, 2000])
def test_weight_off_a_16_byte_boundary(dtype, wdtype, rows):
    pool = _randn(3, (1100,), wdtype)
    for width in (520, 1031):
        for off in (0, 1, 2):
            x, w = _randn(4, (rows, width), dtype), pool[off:off + width]
            codes, scales, h = qb.rms_norm_quant(x, w, residual=x)
            _check_tokens(codes, scales, h, w, 1e-6)


def test_no_tokens():
    x, w = _randn(1, (4, 48), BF16), _randn(2, (48,), BF16)
    c, s, h = qb.rms_norm_quant(x[:0], w, residual=x[:0])
    assert c.shape == (0, 48) and s.shape == (0,) and h.shape == (0, 48)
    b, sb = qb.quantize_token(x)
    assert qb.matmul_i8(c, b, s, sb).shape == (0, 4)
    assert qb.matmul_i8(b, c, sb, s).shape == (4, 0)
    qb.check()


def test_more_than_2_to_31_values():
    """Row offsets past 32 bits: the last rows come out as they do alone."""
    rows, width = 66000, 32776
    x = torch.empty((rows, width), dtype=BF16, device="cuda")
    x.normal_()
    codes, scales = qb.quantize_token(x)
    for part in (x[:3], x[-5:]):
        at = 0 if part.data_ptr() == x.data_ptr() else rows - 5
        c, s = qb.quantize_token(part.clone())
        assert torch.equal(codes[at:at + len(part)], c) and torch.equal(scales[at:at + len(part)], s)
    del x
    a, b = codes[:, :64].contiguous(), codes[:width, :64].contiguous()
    sa, sb = scales, scales[:width].contiguous()
    out = qb.matmul_i8(a, b, sa, sb)
    qb.check()
    assert torch.equal(out[-5:], qb.matmul_i8(a[-5:], b, sa[-5:], sb))
    assert torch.equal(out[-300:, -1000:], qb.matmul_i8(a[-300:], b[-1000:], sa[-300:], sb[-1000:]))
    qb.check()


def test_matmul_i8_leading_dimensions():
    a, b = _codes(1, 12, 100), _codes(2, 70, 100)
    sa, sb = torch.rand(12, device="cuda"), torch.rand(70, device="cuda")
    want = qb.matmul_i8(a, b, sa, sb)
    a3 = a.as_strided((3, 4, 100), (4 * a.stride(0), a.stride(0), 1))
    assert torch.equal(qb.matmul_i8(a3, b, sa.view(3, 4), sb), want.view(3, 4, 70))
    out = torch.zeros((3, 4, 80), dtype=BF16, device="cuda")
    got = qb.matmul_i8(a3, b, sa.view(3, 4), sb, out=out[..., 5:75])
    assert torch.equal(got, want.view(3, 4, 70)) and torch.all(out[..., :5] == 0) and torch.all(out[..., 75:] == 0)
    assert torch.equal(qb.matmul_i8(a[5], b, sa[5:6], sb), want[5])
    with pytest.raises(ValueError):
        qb.matmul_i8(a3.transpose(0, 1), b, sa.view(3, 4), sb)
    qb.check()


def test_binding_refusals():
    x, w = _randn(1, (4, 64), BF16), _randn(2, (64,), BF16)
    for call in (
        lambda: qb.rms_norm_quant(x, w[:63]),
        lambda: qb.rms_norm_quant(x, w.half()),
        lambda: qb.rms_norm_quant(x, w.cpu()),
        lambda: qb.rms_norm_quant(x, w, residual=x[:3]),
        lambda: qb.rms_norm_quant(x, w, residual=x.half()),
        lambda: qb.rms_norm_quant(x, w, residual_out=x),
        lambda: qb.rms_norm_quant(x.t(), w),
        lambda: qb.rms_norm_quant(x, w, codes=torch.empty((4, 64), dtype=torch.uint8, device="cuda")),
        lambda: qb.rms_norm_quant(x, w, scales=torch.empty(3, device="cuda")),
        lambda: qb.quantize_token(torch.empty((4, 0), dtype=BF16, device="cuda")),
        lambda: qb.quantize_token(x.view(2, 2, 64).transpose(0, 1)[:, :, :32]),
    ):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(qb.QbsaError):
        qb.rms_norm_quant(x, w, 0.0)
    with pytest.raises(qb.QbsaError):
        qb.quantize_token(x, codes=torch.empty(64, dtype=torch.int8, device="cuda").expand(4, 64))
    c, s, s4 = torch.zeros((4, 64), dtype=torch.int8, device="cuda"), torch.ones(64, device="cuda"), torch.ones(4, device="cuda")
    for call in (
        lambda: qb.matmul_i8(c, c[:, :48], s4, s4),
        lambda: qb.matmul_i8(c, c, s, s4),
        lambda: qb.matmul_i8(c, c, s4, s4.double()),
        lambda: qb.matmul_i8(c, c, s4, s4, bias=s),
        lambda: qb.matmul_i8(c, c.t().contiguous().t(), s4, s4),
        lambda: qb.matmul_i8(c, c, s4, s4, out_dtype=torch.int32),
        lambda: qb.matmul_i8(c, c, s4, s4, out=torch.empty((4, 5), device="cuda")),
        lambda: qb.matmul_i8(c, c, s4, s4, out_dtype=BF16, out=torch.empty((4, 4), device="cuda")),
        lambda: qb.matmul_i8(c.cpu(), c, s4, s4),
    ):
        with pytest.raises(ValueError):
            call()
    odd = torch.zeros((4, 65), dtype=torch.int8, device="cuda")
    with pytest.raises(qb.QbsaError):
        qb.matmul_i8(odd, odd, s4, s4)


# ---------------------------------------------------------------------------------------------
# matmul_i8
# ---------------------------------------------------------------------------------------------


def _codes(seed, rows, k, low=-128):
    pitch = -(-k // 16) * 16 + 16
    rng = np.random.default_rng(seed)
    buf = torch.from_numpy(rng.integers(low, 128, (rows, pitch)).astype(np.int8)).cuda()
    return buf[:, :k]                                     # what lies beyond K is not zero


def _check_matmul(out, a, b, sa, sb, bias):
    t, want = linear8.matmul_i8(a.cpu().numpy(), b.cpu().numpy(), _np(sa), _np(sb),
                                None if bias is None else _np(bias))
    fi = torch.finfo(out.dtype)
    room = np.abs(t) + (0 if bias is None else np.abs(_np(bias)))
    bound = 3.01 * U * room
    if out.dtype != FP32:
        bound = bound + (fi.eps / 2) * (np.abs(want) + bound) + fi.smallest_normal * fi.eps / 2
    got = _np(out)
    over = np.abs(want) > fi.max * (1 - 1e-3)
    err = np.abs(got - want)
    assert np.all(err[~over] <= bound[~over]), float((err[~over] / np.maximum(bound[~over], 1e-300)).max())


def _run_matmul(seed, m, n, k, dtype, with_bias):
    rng = np.random.default_rng(seed)
    a, b = _codes(seed, m, k), _codes(seed + 1, n, k)
    sa = torch.from_numpy(rng.uniform(0.01, 0.05, m).astype(np.float32)).cuda()
    sb = torch.from_numpy(rng.uniform(1e-4, 1e-3, n).astype(np.float32)).cuda()
    bias = torch.from_numpy(rng.standard_normal(n).astype(np.float32)).cuda() if with_bias else None
    buf = torch.full((m + 2, n + 5), 9.0, dtype=dtype, device="cuda")
    out = qb.matmul_i8(a, b, sa, sb, bias=bias, out_dtype=dtype)
    qb.check()
    assert out.shape == (m, n) and out.dtype == dtype
    _check_matmul(out, a, b, sa, sb, bias)
    qb.matmul_i8(a, b, sa, sb, bias=bias, out=buf[1:m + 1, 2:n + 2])
    qb.check()
    assert torch.equal(buf[1:m + 1, 2:n + 2], out)
    buf[1:m + 1, 2:n + 2] = 9.0
    assert torch.all(buf == 9.0)


@pytest.mark.parametrize("m,n,k", [
    (1, 1, 1), (1, 64, 64), (1, 5120, 512), (2, 130, 15), (3, 128, 16), (7, 257, 17), (16, 100, 129), (17, 640, 1000),
    (31, 129, 128), (33, 31, 255), (64, 300, 2047), (65, 512, 256), (100, 1000, 640), (127, 127, 127), (128, 128, 128),
    (129, 385, 1031), (200, 1, 300), (255, 256, 512), (256, 256, 4096), (257, 511, 96), (300, 2000, 160), (513, 640, 384),
    (1000, 520, 77), (1025, 1032, 1024), (2049, 264, 640),
])
@pytest.mark.parametrize("dtype", [BF16, FP16, FP32])
def test_matmul_i8_sizes(m, n, k, dtype):
    _run_matmul(m * 7 + n, m, n, k, dtype, (m + n) % 2 == 0)


@pytest.mark.parametrize("m,n,k", [(1100, 1031, 2560), (1100, 1031, 2576), (1100, 1031, 5120), (1100, 1031, 5136),
                                   (2049, 1032, 256), (2049, 1032, 257), (2500, 640, 16), (1300, 1000, 1024)])
@pytest.mark.parametrize("dtype", [BF16, FP16, FP32])
def test_matmul_i8_many_tokens_of_short_and_long_rows(m, n, k, dtype):
    """Both numbers of epilogue warps, for outputs on and off 16-byte boundaries."""
    _run_matmul(m + n + k, m, n, k, dtype, k % 32 == 0)


@pytest.mark.parametrize("m", [1, 40, 300])
def test_matmul_i8_largest_sums(m):
    """Every code at its extreme: the sum is 2^14 K, just below 2^31 at the largest K."""
    k, n = 131071, 70
    a = torch.full((m, k + 1), -128, dtype=torch.int8, device="cuda")[:, :k]
    b = torch.full((n, k + 1), -128, dtype=torch.int8, device="cuda")[:, :k]
    b[n // 2] = 127
    one_m, one_n = torch.ones(m, device="cuda"), torch.ones(n, device="cuda")
    out = qb.matmul_i8(a, b, one_m, one_n, out_dtype=FP32)
    qb.check()
    want = torch.full((m, n), 2.0 ** 14 * k, dtype=torch.float64)
    want[:, n // 2] = -128.0 * 127 * k
    assert torch.equal(out.cpu(), want.float())


@pytest.mark.parametrize("m", [1, 24, 384])
def test_matmul_i8_scales_that_are_no_numbers(m):
    a, b = _codes(1, m, 256), _codes(2, 200, 256)
    sa, sb = torch.ones(m, device="cuda"), torch.ones(200, device="cuda")
    sa[m // 2] = float("nan")
    out = qb.matmul_i8(a, b, sa, sb)
    qb.check()
    assert torch.all(torch.isnan(out[m // 2]))
    rest = torch.arange(m) != m // 2
    assert torch.all(torch.isfinite(out[rest.cuda()]))


@pytest.mark.parametrize("m", [1, 20, 300, 3000])
def test_matmul_i8_repeats_bit_for_bit(m):
    a, b = _codes(1, m, 1536), _codes(2, 777, 1536)
    sa, sb = torch.rand(m, device="cuda") + 0.5, torch.rand(777, device="cuda")
    first = qb.matmul_i8(a, b, sa, sb, out_dtype=FP32)
    for _ in range(5):
        assert torch.equal(qb.matmul_i8(a, b, sa, sb, out_dtype=FP32), first)
    # a row alone gives what it gives in the batch
    assert torch.equal(qb.matmul_i8(a[m - 1:], b, sa[m - 1:], sb, out_dtype=FP32), first[m - 1:])
    qb.check()


# ---------------------------------------------------------------------------------------------
# as they are used
# ---------------------------------------------------------------------------------------------


class _Layer:
    """W8A8 attention layer: norm -> joint projection -> quantized block-sparse attention -> projection."""

    def __init__(self, heads, hidden):
        d = heads * 128
        self.heads = heads
        self.norm = _randn(1, (hidden,), BF16, 0.1) + 1
        self.qkv = qb.quantize_token(_randn(2, (3 * d, hidden), BF16, hidden ** -0.5))
        self.out = qb.quantize_token(_randn(3, (hidden, d), BF16, d ** -0.5))
        self.bias = _randn(4, (hidden,), FP32, 0.1)

    def __call__(self, x, residual):
        B, S, _ = x.shape
        c, s, residual = qb.rms_norm_quant(x, self.norm, residual=residual)
        qkv = qb.matmul_i8(c, self.qkv[0], s, self.qkv[1]).view(B, S, 3, self.heads, 128)
        q, k, v = (t.contiguous() for t in qkv.permute(2, 0, 3, 1, 4))
        mask = torch.ones((B, self.heads, -(-S // 128), -(-S // 128)), dtype=torch.uint8, device=x.device)
        o, _, _ = qb.qbsa_fwd(*[t for pair in zip(qb.quantize_qk(q), qb.quantize_qk(k)) for t in pair],
                              *qb.quantize_v(v), mask, 128 ** -0.5)
        o = o.permute(0, 2, 1, 3).reshape(B, S, self.heads * 128)
        c, s = qb.quantize_token(o)
        return qb.matmul_i8(c, self.out[0], s, self.out[1], bias=self.bias), residual

    def plain(self, x, residual):
        B, S, _ = x.shape
        h = x.double() + residual.double()
        y = h / torch.sqrt(h.square().mean(-1, keepdim=True) + 1e-6) * self.norm.double()
        w = self.qkv[0].double() * self.qkv[1].double()[:, None]
        q, k, v = (y @ w.t()).view(B, S, 3, self.heads, 128).permute(2, 0, 3, 1, 4)
        o = torch.softmax(q @ k.transpose(-1, -2) * 128 ** -0.5, -1) @ v
        o = o.permute(0, 2, 1, 3).reshape(B, S, -1)
        return o @ (self.out[0].double() * self.out[1].double()[:, None]).t() + self.bias.double(), h


def test_layer_around_the_quantized_attention():
    """Relative error of the layer: the codes of the normed rows are off by s / sqrt(12) with s about
    max / 127 (max about 4 sigma: 0.9 %), Q, K and V by as much again, P by E4M3's 2^-4 / sqrt(3) averaged
    over the keys, the output's codes by 0.9 %: below 5 % together."""
    layer = _Layer(4, 640)
    x, res = _randn(5, (2, 384, 640), BF16), _randn(6, (2, 384, 640), BF16)
    out, h = layer(x, res)
    qb.check()
    want, hw = layer.plain(x, res)
    assert torch.equal(h, (x.float() + res.float()).to(BF16))
    err = (out.double() - want).norm() / want.norm()
    assert err <= 0.05, float(err)


def test_layer_captured_and_replayed():
    layer = _Layer(2, 256)
    x, res = _randn(5, (1, 256, 256), BF16), _randn(6, (1, 256, 256), BF16)
    x2, res2 = _randn(7, (1, 256, 256), BF16), _randn(8, (1, 256, 256), BF16)
    want = layer(x, res)
    want2 = layer(x2, res2)
    gx, gres = x2.clone(), res2.clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        layer(gx, gres)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = layer(gx, gres)
    for i, w in ((x, want), (x2, want2), (x, want)):
        gx.copy_(i)
        gres.copy_(res if i is x else res2)
        graph.replay()
        for g, e in zip(got, w):
            assert torch.equal(g, e)
    qb.check()


def test_first_use_inside_a_capture():
    """A process whose first calls of these kernels are captured: no allocation, no set-up that a capture
    forbids."""
    script = """
import sys, torch
sys.path.insert(0, %r)
import quantized_block_sparse_attn_b200 as qb
torch.manual_seed(0)
x = torch.randn((600, 1024), device="cuda").bfloat16()
w = torch.ones(1024, device="cuda", dtype=torch.bfloat16)
b = torch.randint(-127, 128, (384, 1024), device="cuda").to(torch.int8)
sb = torch.rand(384, device="cuda")
torch.cuda.synchronize()
def run():
    c, s, h = qb.rms_norm_quant(x, w, residual=x)
    return [c, s, h] + [qb.matmul_i8(c[:m], b, s[:m], sb) for m in (1, 40, 600)]
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    got = run()
g.replay()
torch.cuda.synchronize()
for a, e in zip(got, run()):
    assert torch.equal(a, e)
qb.check()
print("captured")
""" % os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", script], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "captured" in r.stdout, r.stderr[-2000:]


def test_two_threads_at_once():
    """Calls from two host threads, each on its own stream."""
    a, b = _codes(1, 300, 1024), _codes(2, 700, 1024)
    sa, sb = torch.rand(300, device="cuda") + 0.5, torch.rand(700, device="cuda")
    x, w = _randn(3, (300, 1024), BF16), _randn(4, (1024,), BF16)
    want = (qb.matmul_i8(a, b, sa, sb), *qb.rms_norm_quant(x, w, residual=x))
    torch.cuda.synchronize()
    bad = []

    def work():
        with torch.cuda.stream(torch.cuda.Stream()):
            for _ in range(20):
                got = (qb.matmul_i8(a, b, sa, sb), *qb.rms_norm_quant(x, w, residual=x))
                torch.cuda.current_stream().synchronize()
                if not all(torch.equal(g, e) for g, e in zip(got, want)):
                    bad.append(1)
                try:
                    qb.rms_norm_quant(x, w, -1.0)
                    bad.append(2)
                except qb.QbsaError as e:
                    if "eps" not in str(e):
                        bad.append(3)

    threads = [threading.Thread(target=work) for _ in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not bad
    qb.check()


def test_streams_run_side_by_side():
    """The same layer on two streams at once: no shared scratch, so both give what one gives."""
    layer = _Layer(2, 512)
    ins = [(_randn(10 + i, (1, 512, 512), BF16), _randn(20 + i, (1, 512, 512), BF16)) for i in range(2)]
    want = [layer(*i) for i in ins]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in ins]
    got = [[], []]
    for _ in range(4):
        for k, st in enumerate(streams):
            with torch.cuda.stream(st):
                got[k].append(layer(*ins[k]))
    torch.cuda.synchronize()
    for k in range(2):
        for out in got[k]:
            for g, e in zip(out, want[k]):
                assert torch.equal(g, e)
    qb.check()
