"""Attention over 4-bit rows in 64 bits with a bound for every output, from that output's own row
(not collected).

With p_t the softmax weights, v_t = lo_t + step_t code_t the values and out = sum p_t v_t, a kernel that
holds scores and sums in fp32 is off by no more than (u = 2^-24, half a step of fp32; Q = sum |q|;
S = the row's largest |score|)
  scores   e_t = u (scale Q (D + 16) (52 step_t + |lo_t|) + 12 S) + 2^-21 of the key's step and lo: D products
           of q with 16 + code on top of -16 sum q (at most 47 Q, D + 4 roundings), the sum of q itself
           (D / 4 + 2 roundings, times 16 step + |lo|), a few more for step, lo and the base-2 exponent, and
           exp2's own; a weight is then off by the factor 1 +- d_t, d_t = exp(e_t) - 1, the normalised
           output by sum p_t d_t |v_t - out| / (1 - sum p_t d_t)
  weights  p_t step_t rounded to bf16: 2^-8 of it, as a factor of |code_t - 8|; as two bf16 halves
           2^-16 of it, as a factor of 16 + code_t
  sums     N + 64 roundings of sums no larger than sum p_t (55 step_t + |lo_t|) + |out|
  output   rounded once: 2^-8 of it
A row's halves are two where its sequence has at most 64 query rows of a KV head, else one.
"""
from __future__ import annotations

import numpy as np

FEW_ROWS = 64
U = 2.0 ** -24


def attention_bounds(q, key, val, n_kv, scale, few=None, hidden=()):
    """One sequence: q [n, H, D]; key and val (code [t, n_kv, D], step, lo [t, n_kv]) -> (out, bound, drop),
    each [n, H, D]; drop: the output without the row's heaviest token (out where it has only one)."""
    n, H, D = q.shape
    (ck, sk, lk), (cv, sv, lv) = key, val
    t, g = ck.shape[0], H // n_kv
    if few is None:
        few = n * g <= FEW_ROWS
    out, bound, drop = (np.zeros((n, H, D)) for _ in range(3))
    seen = np.ones(t, bool)
    seen[list(hidden)] = False
    see = seen[None] & (np.arange(t)[None] <= t - n + np.arange(n)[:, None])            # [n, t]
    some = see.any(1)
    if not some.any():
        return out, bound, drop
    for h in range(H):
        kv = h // g
        k = lk[:, kv, None] + sk[:, kv, None] * ck[:, kv]
        v = lv[:, kv, None] + sv[:, kv, None] * cv[:, kv]
        qq, ss = q[some, h], see[some]
        s = np.where(ss, scale * qq @ k.T, -np.inf)
        p = np.exp(s - s.max(1, keepdims=True))
        p /= p.sum(1, keepdims=True)
        o = p @ v
        Q = np.abs(qq).sum(1)[:, None]
        S = np.abs(np.where(ss, s, 0)).max(1)[:, None]
        d = np.expm1(U * (scale * Q * (D + 16) * (52 * sk[:, kv] + np.abs(lk[:, kv]))[None] + 12 * S) + 2.0 ** -21)
        pd = p * d
        off = np.stack([(pd[i][:, None] * np.abs(v - o[i])).sum(0) for i in range(len(qq))])
        if few:
            off += 2.0 ** -16 * p @ (sv[:, kv, None] * (16 + cv[:, kv]))
        else:
            off += 2.0 ** -8 * p @ (sv[:, kv, None] * np.abs(cv[:, kv] - 8))
        off += U * (t + 64) * (p @ (55 * sv[:, kv] + np.abs(lv[:, kv])))[:, None] + U * (t + 64) * np.abs(o)
        off /= 1 - pd.sum(1, keepdims=True)
        top = p.argmax(1)
        rest = 1 - p[np.arange(len(qq)), top][:, None]
        with np.errstate(all="ignore"):
            dr = np.where(rest > 1e-12, (o - p[np.arange(len(qq)), top][:, None] * v[top]) / rest, o)
        out[some, h], bound[some, h], drop[some, h] = o, off + 2.0 ** -8 * (np.abs(o) + off) + 1e-30, dr
    return out, bound, drop


def batch_bounds(q, key, val, rows, lens, n_kv, scale, few=None, hidden=None):
    """A batch: q [T, H, D]; key, val of all sequences' tokens, one after another."""
    at, tok, parts = 0, 0, []
    for s, (n, t) in enumerate(zip(rows, lens)):
        cut = lambda c: tuple(x[tok:tok + t] for x in c)  # noqa: E731
        parts.append(attention_bounds(q[at:at + n], cut(key), cut(val), n_kv, scale, few, (hidden or {}).get(s, ())))
        at, tok = at + n, tok + t
    return tuple(np.concatenate(x) for x in zip(*parts))


def outside(got, want, bound):
    """[T, H]: rows of a head with an output outside its bound (NaN is outside)."""
    return ~(np.abs(got - want) <= bound).all(-1)


def telling(want, bound, drop):
    """The share of (row, head) pairs with tokens whose bounds tell them from all zeros, and of those whose
    heaviest token shows at all (moves an output by an eighth of the row's largest) from the row without it."""
    live = bound.any(-1)
    zero = outside(np.zeros_like(want), want, bound)[live].mean() if live.any() else 1.0
    size = np.abs(want).max(-1)
    heavy = live & (np.abs(drop - want).max(-1) > size / 8)
    return zero, outside(drop, want, bound)[heavy].mean() if heavy.any() else 1.0
