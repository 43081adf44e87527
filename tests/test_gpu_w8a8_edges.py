"""GPU cases of the 8-bit linear layers at the ends of their ranges: magnitudes whose squares leave float32,
rows with gaps between them in large numbers, every quotient of short significands, empty tensors.

Tolerances as in test_gpu_w8a8: codes bit for bit; scales within ((terms + 10) / 2 + 6) half steps of
float32, terms = max(32, width / 1024 + 16).  A sum taken again of scaled values adds no rounding: the
scaling is by a power of two, and what it pushes below float32's range is 2^-100 of the row's sum.
"""

import numpy as np
import pytest
import torch

import quantized_block_sparse_attn_b200 as qb
from oracle import linear8
from tests.test_gpu_w8a8 import BF16, FP16, FP32, U, _check_tokens, _np, _randn

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


@pytest.mark.parametrize("rows,width", [(6, 1), (6, 72), (6, 1031), (6, 5120), (6, 33000), (2500, 1024), (2500, 1031)])
@pytest.mark.parametrize("weight", [1e12, 1e-10, 1e-25])
def test_large_rows_with_weights_far_from_one(rows, width, weight):
    """Squares that overflow next to steps from 1e35 down to 1e-14 and below."""
    for dtype in (BF16, FP32):
        x = _randn(width, (rows, width), dtype)
        x[0] = 1e20
        x[1] = (x[1].float().sign() * 1e25).to(dtype)
        x[2] = 1.8e19
        w = torch.full((width,), weight, device="cuda")
        for eps in (1e-6, 1e20, 1e36, 2e37, 3e38):
            codes, scales, _ = qb.rms_norm_quant(x, w, eps)
            qb.check()
            assert np.array_equal(codes.cpu().numpy(), linear8.token_codes_f32(_np(x), _np(w)))
            want = linear8.token_scales(_np(x), _np(w), float(torch.tensor(eps, dtype=FP32)))
            bound = ((max(32, width / 1024 + 16) + 10) / 2 + 6) * U * 1.01 * want
            # a scale below 2^-126 has steps of 2^-149: its quotient and the product with the unit, at most 1,
            # are each rounded to half of one
            assert np.all(np.abs(_np(scales) - want) <= bound + np.where(want < 2.0 ** -126, 2.0 ** -149, 0))


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


@pytest.mark.parametrize("dtype", [BF16, FP32])
def test_rows_that_interleave_or_overlap(dtype):
    """Tensors laid out at random in one buffer: a call runs where no output meets another tensor, byte by
    byte, and is refused where one does."""
    rng = np.random.default_rng(5)
    size = 2 if dtype == BF16 else 4
    w = _randn(2, (24,), FP32)
    ran = refused = 0
    for _ in range(400):
        rows, width = int(rng.integers(1, 6)), int(rng.integers(1, 25))
        same = int(rng.integers(width, 60))                 # one pitch for all of them, half of the time
        one = rng.random() < 0.5
        buf = torch.from_numpy(rng.integers(0, 8, 4096).astype(np.uint8)).cuda()
        at, held = {}, {}
        for name, item, n in (("x", size, width), ("residual", size, width), ("h", size, width), ("codes", 1, width),
                              ("scales", 4, rows)):
            pitch = n if name == "scales" else (same if one else int(rng.integers(n, 60))) * (size if one else item) // item
            count = 1 if name == "scales" else rows
            start = int(rng.integers(0, 4096 // item - pitch * count))
            if one and name != "scales" and name != "x" and rng.random() < 0.7:      # beside x, in its pitch
                start = min(4096 // item - pitch * count, int(at["x"][0] + rng.integers(0, same * size)) // item)
            at[name] = (start * item, pitch * item if count > 1 else 0, item * n, count)
            view = buf.view({"scales": FP32, "codes": torch.int8}.get(name, dtype))
            held[name] = view.as_strided((rows,) if name == "scales" else (rows, width),
                                         (1,) if name == "scales" else (pitch, 1), start)

        def bytes_of(name):
            first, pitch, length, count = at[name]
            return {first + i * pitch + j for i in range(count) for j in range(length)}

        outs = [("h", "x"), ("h", "residual"), ("h", "codes"), ("h", "scales"), ("codes", "scales"), ("codes", "x"),
                ("codes", "residual"), ("scales", "x"), ("scales", "residual")]
        in_place = {n for n in ("x", "residual") if at[n][0] == at["h"][0]}
        clash = any(bytes_of(a) & bytes_of(b) for a, b in outs if not (a == "h" and b in in_place and at[b] == at["h"]))
        x, residual = held["x"].clone(), held["residual"].clone()
        before = buf.clone()

        def call():
            return qb.rms_norm_quant(held["x"], w[:width], residual=held["residual"], residual_out=held["h"],
                                     codes=held["codes"], scales=held["scales"])

        if clash:
            with pytest.raises(qb.QbsaError):
                call()
            assert torch.equal(buf, before)
            refused += 1
        else:
            codes, scales, h = call()
            want = qb.rms_norm_quant(x, w[:width], residual=residual)
            assert torch.equal(codes, want[0]) and torch.equal(h, want[2])
            assert torch.equal(scales.view(torch.int32), want[1].view(torch.int32))
            keep = torch.ones(4096, dtype=torch.bool)
            keep[sorted(bytes_of("h") | bytes_of("codes") | bytes_of("scales"))] = False
            assert torch.equal(buf.cpu()[keep], before.cpu()[keep])
            ran += 1
    qb.check()
    assert ran >= 40 and refused >= 40


def _view(rows, width, pitch, off, dtype, seed=None, fill=None):
    """A buffer with a margin at either end, and rows of it `pitch` apart from `off` on."""
    buf = torch.full((off + rows * pitch + 40,), fill, dtype=dtype, device="cuda") if seed is None else \
        _randn(seed, (off + rows * pitch + 40,), dtype)
    return buf, buf.as_strided((rows, width), (pitch, 1), off)


def _same_outside(buf, keep, view):
    inside = torch.zeros(buf.numel(), dtype=torch.bool, device="cuda")
    inside.as_strided(view.shape, view.stride(), view.storage_offset())[...] = True
    return torch.equal(buf[~inside], keep[~inside])


@pytest.mark.parametrize("width,pitches,offs", [
    (264, (272, 280, 288, 304), (8, 16, 0, 16)),            # rows on 16-byte boundaries, with gaps
    (520, (528, 520, 1040, 528), (0, 8, 24, 32)),
    (264, (271, 269, 267, 265), (3, 5, 7, 1)),              # every row at another alignment
    (265, (265, 266, 268, 272), (0, 1, 2, 16)),
    (520, (521, 520, 523, 520), (1, 0, 4, 0)),              # one of them aligned
    (1031, (1033, 1040, 1037, 1033), (2, 9, 5, 3)),
    (1288, (1300, 1288, 1290, 1312), (6, 8, 2, 16)),
    (4099, (4101, 4111, 4100, 4112), (7, 1, 3, 5)),
    (9001, (9003, 9008, 9001, 9008), (1, 8, 0, 32)),        # four pieces per thread
])
@pytest.mark.parametrize("dtype", [BF16, FP32])
def test_many_rows_with_gaps_between_them(width, pitches, offs, dtype):
    """The streamed kernels on rows of four different pitches and offsets: values, and what lies between the
    rows and around them; the quantiser alone; the sum in place of either input."""
    rows = 2500
    xb, x = _view(rows, width, pitches[0], offs[0], dtype, seed=1)
    rb, res = _view(rows, width, pitches[1], offs[1], dtype, seed=2)
    w = _randn(3, (width,), dtype)
    hb, h = _view(rows, width, pitches[2], offs[2], dtype, fill=7.0)
    cb, codes = _view(rows, width, pitches[3], offs[3], torch.int8, fill=77)
    keep = [t.clone() for t in (xb, rb, hb, cb)]
    want = (x.float() + res.float()).to(dtype)
    _, scales, got = qb.rms_norm_quant(x, w, residual=res, residual_out=h, codes=codes)
    qb.check()
    assert got.data_ptr() == h.data_ptr() and torch.equal(h, want)
    _check_tokens(codes, scales, want, w, 1e-6)
    assert torch.equal(xb, keep[0]) and torch.equal(rb, keep[1])
    assert _same_outside(hb, keep[2], h) and _same_outside(cb, keep[3], codes)
    first = codes.clone()
    for kw in (dict(residual=None), dict(residual=res, residual_out=res), dict(residual=res, residual_out=x)):
        if kw["residual"] is not None and kw["residual_out"] is x:
            rb.copy_(keep[1])
        codes.fill_(55)
        _, s, _ = qb.rms_norm_quant(x, w, codes=codes, **kw)
        qb.check()
        if kw["residual"] is None:
            _check_tokens(codes, s, x, w, 1e-6)
        else:
            assert torch.equal(codes, first) and torch.equal(s, scales) and torch.equal(kw["residual_out"], want)
        assert _same_outside(xb, keep[0], x) and _same_outside(rb, keep[1], res) and _same_outside(cb, keep[3], codes)
    xb.copy_(keep[0])
    _, s = qb.quantize_token(x, codes=codes)
    qb.check()
    _check_tokens(codes, s, x)
    assert torch.equal(xb, keep[0]) and _same_outside(cb, keep[3], codes)


def test_columns_of_one_buffer():
    """x, the sum and the residual as columns of one buffer, many rows: outputs and inputs share 16-byte units."""
    rows, width = 2500, 527
    buf = _randn(1, (rows, 3 * width), BF16)
    keep = buf.clone()
    x, h, res = buf[:, :width], buf[:, width:2 * width], buf[:, 2 * width:]
    w = _randn(2, (width,), BF16)
    codes, scales, _ = qb.rms_norm_quant(x, w, residual=res, residual_out=h)
    qb.check()
    want = (keep[:, :width].float() + keep[:, 2 * width:].float()).to(BF16)
    assert torch.equal(h, want) and torch.equal(x, keep[:, :width]) and torch.equal(res, keep[:, 2 * width:])
    _check_tokens(codes, scales, want, w, 1e-6)


@pytest.mark.parametrize("dtype,exponents", [(FP16, (0, 5, -8, -14, -20, -24)),
                                             (BF16, (0, -100, -126, -127, -130, 88, 89, 90, 100, 119))])
def test_quotients_of_every_maximum(dtype, exponents):
    """Rows of a 16-bit type for every significand of the largest value, with every smaller significand at every
    exponent that reaches a code; at scales where the step meets 2^-126, where it passes 1.2e27 (the two ways
    of the quotient), and where the row is subnormal."""
    n = 128 if dtype == BF16 else 1024
    tops = torch.arange(n, 2 * n, device="cuda", dtype=torch.float32)
    all_x = torch.cat([tops * 2.0 ** -j for j in range(9)])
    rows = torch.where(all_x[None] <= tops[:, None], all_x[None], torch.zeros((), device="cuda"))
    rows = torch.cat([tops[:, None], rows], 1)
    for e in exponents:
        x = (rows.double() * 2.0 ** e).to(dtype)
        codes, scales = qb.quantize_token(x)
        qb.check()
        _check_tokens(codes, scales, x)
