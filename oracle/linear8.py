"""Plain NumPy definitions of the 8-bit linear layers: token quantisers (with and without the RMS
norm) and the INT8 product, in float64.  Test infrastructure only; shares no code with the CUDA path.

Rows h (after the residual's addition, rounded to the storage type), g = h * weight, a = max|g|,
s = max(a / 127, 2^-126) (1 if a = 0): codes = rint(g / s), scale = s / sqrt(mean(h^2) + eps)
(1 if a = 0).  `token_codes_f32` takes the same steps in float32, which fixes the codes bit for bit;
`token_quotients` gives g / s in float64, which every code has to lie next to.
"""

import numpy as np

TINY = 2.0 ** -126


def _step(a, dtype):
    s = np.maximum(a / dtype(127), dtype(TINY))
    return np.where(a == 0, dtype(1), s)


def token_quotients(h, weight=None):
    """(g / s, s, a) in float64 for rows h [..., W]."""
    g = np.asarray(h, np.float64)
    if weight is not None:
        g = g * np.asarray(weight, np.float64)
    a = np.abs(g).max(-1)
    s = _step(a, np.float64)
    return g / s[..., None], s, a


def token_codes_f32(h, weight=None):
    """int8 codes by the float32 steps of the definition (rows without NaN or infinity)."""
    g = np.asarray(h, np.float32)
    if weight is not None:
        g = g * np.asarray(weight, np.float32)
    s = _step(np.abs(g).max(-1), np.float32)
    return np.rint(g / s[..., None]).astype(np.int8)


def token_scales(h, weight=None, eps=None):
    """float64 scales; eps None: no norm."""
    _, s, a = token_quotients(h, weight)
    if eps is None:
        return s
    rms = np.sqrt(np.square(np.asarray(h, np.float64)).mean(-1) + eps)
    return np.where(a == 0, 1.0, s / rms)


def matmul_i8(a, b, a_scale, b_scale, bias=None):
    """(product in float64 before the bias, the output): [M, N]."""
    acc = np.asarray(a, np.float64) @ np.asarray(b, np.float64).T     # whole numbers below 2^53: exact
    t = acc * np.asarray(a_scale, np.float64)[:, None] * np.asarray(b_scale, np.float64)
    return t, t if bias is None else t + np.asarray(bias, np.float64)
