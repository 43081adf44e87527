"""CPU checks of the 8-bit linear layers' entry points: refusals come before any launch, and the
oracle's own identities hold."""

import ctypes

import numpy as np
import pytest
import torch

import quantized_block_sparse_attn_b200 as qb
from oracle import linear8

FAKE = ctypes.c_void_p(0x10000)


@pytest.fixture(scope="module", autouse=True)
def built():
    from quantized_block_sparse_attn_b200 import build
    build.build()


def _norm(**over):
    a = dict(x=FAKE, xs=64, res=None, rs=0, w=FAKE, dt=0, wdt=0, rows=4, width=64, eps=1e-6, h=None, hs=0,
             codes=FAKE, cs=64, scales=FAKE)
    a.update(over)
    return qb.lib().qbsa_rms_norm_quant(a["x"], a["xs"], a["res"], a["rs"], a["w"], a["dt"], a["wdt"], a["rows"],
                                        a["width"], a["eps"], a["h"], a["hs"], a["codes"], a["cs"], a["scales"], None)


@pytest.mark.parametrize("over,status", [
    (dict(x=None), 1),
    (dict(w=None), 1),
    (dict(codes=None), 1),
    (dict(scales=None), 1),
    (dict(dt=3), 1),
    (dict(wdt=1), 1),                                     # fp16 weight of bf16 rows
    (dict(eps=0.0), 1),
    (dict(eps=-1e-6), 1),
    (dict(eps=float("nan")), 1),
    (dict(eps=float("inf")), 1),
    (dict(width=0), 1),
    (dict(rows=-1), 1),
    (dict(width=(1 << 24) + 1, xs=1 << 25, cs=1 << 25), 2),
    (dict(rows=1 << 31), 2),
    (dict(res=FAKE, rs=64), 1),                           # a residual without residual_out
    (dict(h=FAKE, hs=64), 1),
    (dict(res=FAKE, rs=64, h=ctypes.c_void_p(0x20000), hs=63), 1),
    (dict(res=FAKE, rs=128, h=FAKE, hs=64, x=ctypes.c_void_p(0x20000)), 1),   # in place, another stride
    (dict(cs=63), 1),
    (dict(xs=-64), 1),
    (dict(x=ctypes.c_void_p(0x10001)), 1),
    (dict(scales=ctypes.c_void_p(0x10002)), 1),
    (dict(w=ctypes.c_void_p(0x10002), wdt=2), 1),
])
def test_rms_norm_quant_rejects_before_launch(over, status):
    assert _norm(**over) == status, qb.lib().qbsa_last_error().decode()


def test_no_rows_is_no_work():
    assert _norm(rows=0, x=None, codes=None, scales=None) == 0
    assert qb.lib().qbsa_quantize_token(None, 0, 0, 0, 64, None, 0, None, None) == 0
    assert qb.lib().qbsa_matmul_i8(None, 0, FAKE, 64, None, FAKE, None, 0, 8, 64, 0, None, 0, None) == 0
    assert qb.lib().qbsa_matmul_i8(FAKE, 64, None, 0, FAKE, None, None, 8, 0, 64, 0, None, 0, None) == 0


@pytest.mark.parametrize("over,status", [
    (dict(x=None), 1), (dict(codes=None), 1), (dict(scales=None), 1), (dict(dt=-1), 1), (dict(width=0), 1),
    (dict(rows=-3), 1), (dict(cs=10), 1), (dict(x=ctypes.c_void_p(0x10002), dt=2), 1),
])
def test_quantize_token_rejects_before_launch(over, status):
    a = dict(x=FAKE, xs=64, dt=0, rows=4, width=64, codes=FAKE, cs=64, scales=FAKE)
    a.update(over)
    st = qb.lib().qbsa_quantize_token(a["x"], a["xs"], a["dt"], a["rows"], a["width"], a["codes"], a["cs"],
                                      a["scales"], None)
    assert st == status, qb.lib().qbsa_last_error().decode()


@pytest.mark.parametrize("over,status", [
    (dict(a=None), 1), (dict(b=None), 1), (dict(sa=None), 1), (dict(sb=None), 1), (dict(out=None), 1),
    (dict(a=ctypes.c_void_p(0x10008)), 1),
    (dict(b=ctypes.c_void_p(0x10004)), 1),
    (dict(sa=ctypes.c_void_p(0x10002)), 1),
    (dict(bias=ctypes.c_void_p(0x10001)), 1),
    (dict(out=ctypes.c_void_p(0x10001)), 1),
    (dict(lda=72), 1),                                    # not a multiple of 16
    (dict(ldb=48), 1),                                    # below K
    (dict(ldo=31), 1),
    (dict(K=0), 1),
    (dict(M=-1), 1),
    (dict(K=131072, lda=131072, ldb=131072), 2),
    (dict(M=2 ** 31 - 1), 2),
    (dict(dt=5), 1),
])
def test_matmul_i8_rejects_before_launch(over, status):
    p = dict(a=FAKE, lda=64, b=FAKE, ldb=64, sa=FAKE, sb=FAKE, bias=None, M=16, N=32, K=64, dt=0, out=FAKE, ldo=32)
    p.update(over)
    st = qb.lib().qbsa_matmul_i8(p["a"], p["lda"], p["b"], p["ldb"], p["sa"], p["sb"], p["bias"], p["M"], p["N"],
                                 p["K"], p["dt"], p["out"], p["ldo"], None)
    assert st == status, qb.lib().qbsa_last_error().decode()


def test_binding_refuses_host_tensors_and_other_types():
    x, w = torch.zeros(4, 64, dtype=torch.bfloat16), torch.ones(64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        qb.rms_norm_quant(x, w)
    with pytest.raises(ValueError):
        qb.rms_norm_quant(x.double(), w)
    with pytest.raises(ValueError):
        qb.quantize_token(x)
    with pytest.raises(ValueError):
        qb.quantize_token(x.to(torch.int32))
    c, s = torch.zeros(4, 64, dtype=torch.int8), torch.ones(4)
    with pytest.raises(ValueError):
        qb.matmul_i8(c, c, s, s)
    with pytest.raises(ValueError):
        qb.matmul_i8(c.float(), c, s, s)


def test_oracle_codes_reconstruct_within_half_a_step():
    rng = np.random.default_rng(3)
    h = rng.standard_normal((37, 129)).astype(np.float32)
    w = rng.standard_normal(129).astype(np.float32)
    q, s, _ = linear8.token_quotients(h, w)
    codes = linear8.token_codes_f32(h, w)
    # g, a / 127 and the quotient are rounded to float32: three half steps of 2^-24 on values up to 127
    assert np.abs(codes - q).max() <= 0.5 + 127 * 3 * 2.0 ** -24 * 1.01
    assert np.abs(codes).max(-1).min() == 127
    # codes * scale is the normed row, within half a code
    scale = linear8.token_scales(h, w, 1e-6)
    y = h.astype(np.float64) / np.sqrt(np.square(h.astype(np.float64)).mean(-1, keepdims=True) + 1e-6) * w
    assert np.all(np.abs(codes * scale[:, None] - y) <= 0.5001 * scale[:, None])


def test_oracle_rows_without_values():
    h = np.zeros((2, 5), np.float32)
    h[1] = 1e-44                                         # a / 127 would be 0: the step stays at 2^-126
    assert np.array_equal(linear8.token_codes_f32(h), np.zeros((2, 5), np.int8))
    assert linear8.token_scales(h)[0] == 1.0 and linear8.token_scales(h)[1] == 2.0 ** -126
    assert linear8.token_scales(h, np.ones(5), 1e-6)[0] == 1.0


def test_oracle_product_by_loops():
    rng = np.random.default_rng(4)
    a, b = rng.integers(-128, 128, (3, 7)), rng.integers(-128, 128, (2, 7))
    sa, sb, bias = rng.random(3), rng.random(2), rng.standard_normal(2)
    _, out = linear8.matmul_i8(a, b, sa, sb, bias)
    for m in range(3):
        for n in range(2):
            want = sum(int(a[m, k]) * int(b[n, k]) for k in range(7)) * sa[m] * sb[n] + bias[n]
            assert abs(out[m, n] - want) <= 1e-9 * max(1, abs(want))


@pytest.mark.parametrize("bits", [7, 10])
def test_short_quotients_by_a_reciprocal_in_two_parts(bits):
    """The kernel's quotient of 16-bit values, FMA(x, r, RN(x r_low)) with r = RN(1 / s) and
    r_low = RN(r RN(1 - s r)), equals the division RN(x / s), s = RN(a / 127), for every pair of significands
    (7 stored bits: bf16, 10: fp16) and every ratio that reaches a code; codes are equal with it."""
    f, g = np.float32, np.longdouble
    n = 1 << bits
    sig = np.arange(n, 2 * n).astype(f)
    xs = np.concatenate([sig * f(2.0 ** -j) for j in range(9)])
    assert np.finfo(g).nmant >= 63
    for a in sig[:: 1 if bits == 7 else 4]:
        s = f(a / f(127))
        r = f(f(1) / s)
        r_low = f(f(g(1) - g(s) * g(r)) * r)
        x = xs[xs <= a]
        y = (x.astype(g) * g(r) + (x * r_low).astype(g)).astype(f)     # 11 + 24 and 24 bits: exact in g
        want = x / s
        assert np.array_equal(y, want)
        assert np.array_equal(np.rint(y), np.rint(want))
    # smaller values round to 0
    assert n * 2.0 ** -8 / (n / 127) < 0.5
