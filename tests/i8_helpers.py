"""The 8-bit integer operators from their definitions, in 64 bits, and bounds of their roundings (not collected)."""
from __future__ import annotations

import numpy as np

HALF = 2.0 ** -8      # a bf16 rounding, relative
ULP = 2.0 ** -24      # an fp32 rounding, relative
TINY = 2.0 ** -126    # below fp32's and bf16's normal numbers a rounding is absolute, and smaller than this


def bf16(v):
    """Nearest bf16 (ties to even) of values, as float64; through float32, as every sum here is rounded."""
    from workloads import bf16_bits_from_f32
    b = bf16_bits_from_f32(np.asarray(v, np.float32))
    return (b.astype(np.uint32) << 16).view(np.float32).astype(np.float64)


def codes(p):
    """The 8-bit codes of rows p [n, d]: nearest integers to 127 p / max|p|, ties to even.

    Exact in float64 for p with up to 16 significant bits: a quotient next to a tie is at least 1 / (2 max|p|)
    units of p's last place away from it (2^-17), or is the tie itself, which a division returns exactly."""
    m = np.abs(p).max(-1, keepdims=True)
    return np.where(m > 0, np.rint(127.0 * p / np.where(m > 0, m, 1.0)), 0.0)


def norm(x, residual, w, eps):
    """-> (h, y, codes, scale) of rows, from float64 arrays that hold bf16 values."""
    h = x if residual is None else bf16(x + residual)
    r = 1.0 / np.sqrt(np.mean(h * h, -1, keepdims=True) + eps)
    p = h * w
    return h, p * r, codes(p), (np.abs(p).max(-1, keepdims=True) * r / 127.0)[:, 0]


def activated(v, act):
    from scipy.special import erfc, expit
    if act == "silu":
        return v * expit(v)
    if act == "gelu":
        return 0.5 * v * erfc(-v / np.sqrt(2.0))
    return 0.5 * v * (1.0 + np.tanh(np.sqrt(2.0 / np.pi) * (v + 0.044715 * v ** 3)))


def product(xc, xs, wc, ws):
    """xs[m] ws[n] sum_k of int8 codes: the sums are whole numbers below 2^53."""
    return (xc.astype(np.float64) @ wc.astype(np.float64).T) * xs.astype(np.float64)[:, None] * ws.astype(np.float64)[None]


# the sum's conversion to fp32, two factors, then bf16
PRODUCT = HALF + 4 * ULP


def act_bound(act, g, x):
    """Absolute bound of act(g) x as the kernels compute it.

    silu and gelu_tanh: an exponential, a sum, a quotient, a factor and the rounding of its argument are a few fp32
    roundings each; the tanh form's argument u is a cubic, whose rounding moves the result by |2u| roundings, at most
    2 * 88 where it is not 0 or v.  gelu: erfc's argument z is rounded, which moves it by 2 z^2 roundings, at most 2 *
    88; the library's erfc is good to some units.  512 roundings are above all of these, 2^-15 of the value, far
    below bf16's 2^-8.  The plain tanh form loses 2^-53 of |v| to cancellation."""
    a = activated(g, act) * x
    return np.abs(a) * (HALF + 512 * ULP) + np.abs(g * x) * 2.0 ** -50 + TINY
