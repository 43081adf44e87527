"""CPU checks of calls that the 8-bit linear layers have to refuse, and of some that they have to take."""

import ctypes
import types

import numpy as np
import pytest
import torch

import quantized_block_sparse_attn_b200 as qb
from quantized_block_sparse_attn_b200 import _binding


@pytest.fixture(scope="module", autouse=True)
def built():
    from quantized_block_sparse_attn_b200 import build
    build.build()


def _at(address):
    return ctypes.c_void_p(address)


def _norm(x=0x10000, xs=64, res=None, rs=0, w=0x900000, dt=0, wdt=0, rows=4, width=64, eps=1e-6, h=None, hs=0,
          codes=0x20000, cs=64, scales=0x30000):
    p = [None if a is None else _at(a) for a in (x, res, w, h, codes, scales)]
    st = qb.lib().qbsa_rms_norm_quant(p[0], xs, p[1], rs, p[2], dt, wdt, rows, width, eps, p[3], hs, p[4], cs, p[5],
                                      None)
    return st, qb.lib().qbsa_last_error().decode()


@pytest.mark.parametrize("eps", [1e-40, 1.4e-45, float(np.nextafter(np.float32(2.0 ** -126), np.float32(0)))])
def test_an_eps_that_float32_does_not_hold_in_full_is_refused(eps):
    """h^2 of h = 3e-23 is 9e-46, in float32 1.4e-45: 2 % of the norm next to an eps of 1e-44."""
    st, msg = _norm(eps=eps)
    assert st == 1 and "eps" in msg


@pytest.mark.parametrize("shape", [(0, 64), (0, 3, 64), (3, 0, 64), (3, 0, 1), (2, 1, 0, 64), (2, 0, 1, 64), (0, 0, 5)])
def test_no_rows_wherever_the_empty_dimension_stands(shape):
    t = torch.empty(shape)
    assert _binding._rows("x", t)[0] == 0
    assert _binding._rows("x", t.transpose(0, len(shape) - 2))[0] == 0
    assert _binding._rows("x", torch.empty((4, *shape[1:-1], 70))[:0, ..., 3:67])[0] == 0


def test_rows_evenly_spaced_or_refused():
    x = torch.empty((4, 6, 80))
    assert _binding._rows("x", x) == (24, 80)
    assert _binding._rows("x", x[..., 3:70]) == (24, 80)
    assert _binding._rows("x", x[:, :1]) == (4, 480)
    assert _binding._rows("x", x[:1, ::2]) == (3, 160)
    assert _binding._rows("x", x[0, 0]) == (1, 80)
    for t in (x[:, :5], x.transpose(0, 1), x[..., ::2]):
        with pytest.raises(ValueError):
            _binding._rows("x", t)


def _tensor(shape, dtype):
    """What the binding asks of a CUDA tensor before it makes the outputs, for sizes that no test allocates."""
    strides = [1]
    for n in reversed(shape[1:]):
        strides.append(strides[-1] * n)
    strides = tuple(reversed(strides))
    return types.SimpleNamespace(shape=shape, dtype=dtype, get_device=lambda: 0, stride=lambda: strides)


@pytest.mark.parametrize("size", [2 ** 31, 2 ** 32 - 5, 2 ** 32 + 64, 2 ** 33 + 1])
def test_sizes_that_a_c_int_would_take_for_others(size):
    """2^32 + 64 values of a row would be passed as 64."""
    w = _tensor((size,), torch.bfloat16)
    for call in (lambda: qb.quantize_token(_tensor((1, size), torch.bfloat16)),
                 lambda: qb.rms_norm_quant(_tensor((2, 3, size), torch.bfloat16), w)):
        with pytest.raises(qb.QbsaError, match="width"):
            call()
    i8 = torch.int8
    for m, n, k in ((size, 8, 16), (8, size, 16), (8, 8, size)):
        with pytest.raises(qb.QbsaError, match="M, N or K"):
            qb.matmul_i8(_tensor((m, k), i8), _tensor((n, k), i8), None, None)


@pytest.mark.parametrize("over", [
    dict(codes=0x10000),                                            # codes over x
    dict(codes=0x10000 + 3 * 128 + 126),                            # over the last row's last value
    dict(codes=0x10000 + 127, xs=256, cs=640, rows=9),              # pitches that differ, in row 0's last byte
    dict(scales=0x10000 + 8),
    dict(scales=0x20000 + 12),                                      # scales over codes
    dict(w=0x20000),
    dict(scales=0x900000),
    dict(res=0x40000, rs=64, h=0x40000 + 128, hs=64),               # a row further on
    dict(res=0x40000, rs=64, h=0x10000 + 2, hs=64),                 # x, one value further on
    dict(res=0x10000 + 128, rs=64, h=0x10000, hs=64),               # in place of x, and residual one row further on
    dict(res=0x40000, rs=64, h=0x20000, hs=64),                     # residual_out over codes
    dict(res=0x40000, rs=64, h=0x30000, hs=64),
    dict(res=0x40000, rs=64, h=0x900000, hs=64),
    dict(res=0x40000, rs=64, h=0x50000, hs=64, codes=0x40000 + 5),
])
def test_outputs_that_overlap(over):
    st, msg = _norm(**over)
    assert st == 1 and "overlap" in msg


@pytest.mark.parametrize("over", [dict(out=0x10000), dict(out=0x20000 + 31 * 64 + 62), dict(out=0x30000 + 60),
                                  dict(out=0x40000 + 124), dict(out=0x50000, bias=0x50000 + 16 * 64 - 4)])
def test_products_over_their_inputs(over):
    p = dict(a=0x10000, b=0x20000, sa=0x30000, sb=0x40000, bias=0x48000, out=0x50000)
    p.update(over)
    st = qb.lib().qbsa_matmul_i8(_at(p["a"]), 64, _at(p["b"]), 64, _at(p["sa"]), _at(p["sb"]), _at(p["bias"]), 16, 32,
                                 64, 0, _at(p["out"]), 32, None)
    assert st == 1 and b"overlaps" in qb.lib().qbsa_last_error()


def test_wait_selftest_refusals():
    for form, result in ((-1, 0x10000), (4, 0x10000), (0, None), (2, 0x10004)):
        assert qb.lib().qbsa_wait_selftest_form(form, result, None) == 1


@pytest.mark.parametrize("short", [True, False])
def test_calls_with_and_without_torch_s_short_names(monkeypatch, short):
    """The stream and the device come from torch's public calls where the short ones are missing; a call for
    another device than the current one makes that one current."""
    if short:
        monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda dev: 1000 + dev, raising=False)
        monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 1, raising=False)
    else:
        monkeypatch.delattr(torch._C, "_cuda_getCurrentRawStream", raising=False)
        monkeypatch.delattr(torch._C, "_cuda_getDevice", raising=False)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda dev: types.SimpleNamespace(cuda_stream=1000 + dev))
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 1)
    entered = []

    class Device:
        def __init__(self, dev):
            self.dev = dev

        def __enter__(self):
            entered.append(self.dev)

        def __exit__(self, *a):
            entered.append(None)

    monkeypatch.setattr(torch.cuda, "device", Device)
    _binding._stream_calls.cache_clear()
    try:
        seen = []
        _binding._call_on(1, lambda *a: seen.append((a, list(entered))) or 0, "x")
        _binding._call_on(3, lambda *a: seen.append((a, list(entered))) or 0, "y")
        assert seen == [(("x", 1001), []), (("y", 1003), [3])] and entered == [3, None]
        with pytest.raises(qb.QbsaError):
            _binding._call_on(1, lambda *a: 1)
    finally:
        _binding._stream_calls.cache_clear()
