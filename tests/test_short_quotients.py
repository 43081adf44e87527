"""The quantiser's quotient of 16-bit values, FMA(x, r, RN(x r_low)) with s = RN(a / 127), r = RN(1 / s) and
r_low = RN(r RN(1 - s r)), against the division RN(x / s): every pair of significands, every ratio that
reaches a code."""

import numpy as np
import pytest

F, G = np.float32, np.longdouble


def _differences(bits, exponent, limit=None):
    n = 1 << bits
    sig = np.arange(n, 2 * n).astype(F) * F(2.0 ** exponent)
    xs = np.concatenate([sig * F(2.0 ** -j) for j in range(9)])
    assert np.finfo(G).nmant >= 63
    wrong = pairs = 0
    for a in sig:
        s = max(F(a / F(127)), F(2.0 ** -126))
        if limit is not None and not s < F(limit):
            continue
        r = F(F(1) / s)
        r_low = F(F(G(1) - G(s) * G(r)) * r)
        x = xs[xs <= a]
        y = (x.astype(G) * G(r) + (x * r_low).astype(G)).astype(F)     # 11 + 24 and 24 bits: exact in G
        wrong += int((y != x / s).sum())
        pairs += len(x)
    return wrong, pairs


def test_every_pair_of_fp16():
    wrong, pairs = _differences(10, 0)
    assert wrong == 0 and pairs >= 8.9e6


@pytest.mark.parametrize("exponent", [-133, -128, -126, -125, -120, -60, 0, 60, 80, 86, 87, 88, 89])
def test_every_pair_of_bf16(exponent):
    """From steps at 2^-126 up to 1.2e27, above which the kernel divides; r_low is subnormal for some there."""
    wrong, pairs = _differences(7, exponent, limit=1.2e27)
    assert wrong == 0 and pairs >= 1e5
