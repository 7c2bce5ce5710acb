"""The 4-bit KV pages in plain numpy, 64 bits: rows to codes and back, slab bytes,
rotation and attention.  Written from the definitions in include/lora_gemm.h (form,
place and batch of lora_kv_append / lora_kv_attention); nothing here is shared with the
library or its kernels.
"""
from __future__ import annotations

from typing import Dict, Sequence, Tuple

import numpy as np

BLOCK = 16


def bf16_round(x) -> np.ndarray:
    """float64 (through float32) to the nearest bf16 value, ties to even, as float64."""
    b = np.asarray(x, np.float32).view(np.uint32).astype(np.uint64)
    r = ((b + 0x7FFF + ((b >> 16) & 1)) >> 16).astype(np.uint32) << 16
    nan = np.isnan(np.asarray(x, np.float64))
    return np.where(nan, np.nan, r.astype(np.uint32).view(np.float32).astype(np.float64))


def bf16_bits(x) -> np.ndarray:
    """The 16 bits of values that are bf16 already."""
    return (np.asarray(x, np.float32).view(np.uint32) >> 16).astype(np.uint32)


def rotate(x: np.ndarray, pos: np.ndarray, cos_sin: np.ndarray, interleaved: bool) -> np.ndarray:
    """x [T, heads, D] with its first cos_sin.shape[1] values turned by the angles of pos [T]."""
    rot = cos_sin.shape[1]
    c = cos_sin[pos, :rot // 2].astype(np.float64)[:, None]
    s = cos_sin[pos, rot // 2:].astype(np.float64)[:, None]
    out = x.astype(np.float64).copy()
    a, b = (slice(0, rot, 2), slice(1, rot, 2)) if interleaved else (slice(0, rot // 2), slice(rot // 2, rot))
    out[..., a] = x[..., a] * c - x[..., b] * s
    out[..., b] = x[..., b] * c + x[..., a] * s
    return out


def quantise(x: np.ndarray) -> Tuple[np.ndarray, np.ndarray, np.ndarray]:
    """bf16 rows [..., D] (as float64) -> codes, step, lo."""
    lo, hi = x.min(-1), x.max(-1)
    step = bf16_round((hi - lo) / 15)
    bad = ~np.isfinite(x).all(-1)
    step = np.where(bad, np.nan, step)
    with np.errstate(all="ignore"):
        code = np.clip(np.rint((x - lo[..., None]) / step[..., None]), 0, 15)
    code = np.where((step > 0)[..., None], code, 0).astype(np.int64)
    return code, step, lo


def value(code: np.ndarray, step: np.ndarray, lo: np.ndarray) -> np.ndarray:
    return lo[..., None] + step[..., None] * code


def key_bytes(code: np.ndarray, r: int) -> Dict[int, int]:
    """Byte offset in a key slab -> value, of token r's codes [D]."""
    D = code.size
    out = {}
    for w in range(D // 8):
        word = 0
        for k in range(4):
            word |= int(code[8 * w + 2 * k]) << (4 * k) | int(code[8 * w + 2 * k + 1]) << (4 * k + 16)
        for i in range(4):
            out[r * (D // 2) + 4 * w + i] = (word >> (8 * i)) & 255
    return out


def value_bytes(code: np.ndarray, r: int) -> Dict[int, int]:
    """Byte offset in a value slab -> value, of token r's codes [D]."""
    D = code.size
    out = {}
    for i in range(16):
        for g in range(D // 64):
            unit = 0
            for k in range(4):
                unit |= int(code[i * (D // 16) + 4 * g + k]) << (4 * k)
            at = (((i * 8 + r // 2) * (D // 64) + g) * 2 + r % 2) * 2
            out[at], out[at + 1] = unit & 255, unit >> 8
    return out


def slab_bytes(D: int) -> int:
    return 8 * D + 64


def attention(q: np.ndarray, k: np.ndarray, v: np.ndarray, n_kv: int, scale: float, hidden: Sequence[int] = ()) -> np.ndarray:
    """One sequence: q [n, H, D], k and v [t, n_kv, D] (the values the cache stands for); row j sees
    tokens up to t - n + j, without those in ``hidden``; a row that sees none is zero."""
    n, H, D = q.shape
    t = k.shape[0]
    g = H // n_kv
    out = np.zeros((n, H, D))
    see = np.ones(t, bool)
    see[list(hidden)] = False
    for j in range(n):
        upto = np.nonzero(see[:max(0, t - n + j + 1)])[0]
        if upto.size == 0:
            continue
        for h in range(H):
            s = k[upto, h // g] @ q[j, h] * scale
            p = np.exp(s - s.max()) if np.isfinite(s).all() else np.full(s.shape, np.nan)
            out[j, h] = (p / p.sum()) @ v[upto, h // g]
    return out
