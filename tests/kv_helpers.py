"""Batches over the pool's KV pages for the KV tests (not collected)."""
from __future__ import annotations

import numpy as np

from oracle import kv_model as KV


def table_of(free, lens, npb, max_blocks):
    """[n_seqs, max_blocks, npb] pages for sequences of so many tokens, taken from ``free`` in order."""
    t = np.full((len(lens), max_blocks, npb), -1, np.int32)
    at = 0
    for s, n in enumerate(lens):
        nb = -(-n // KV.BLOCK)
        t[s, :nb] = np.asarray(free[at:at + nb * npb]).reshape(nb, npb)
        at += nb * npb
    return t


def blocks(lens):
    return sum(-(-n // KV.BLOCK) for n in lens)


def positions(rows, lens):
    """(sequence, position) of every row."""
    return [(s, t - n + j) for s, (n, t) in enumerate(zip(rows, lens)) for j in range(n)]


def cos_sin(n_pos, rot):
    f = 10000.0 ** (-np.arange(rot // 2) / (rot / 2))
    a = np.arange(n_pos)[:, None] * f
    return np.concatenate([np.cos(a), np.sin(a)], 1).astype(np.float32)


def expected_pages(pages, table, page_bytes, rows, lens, codes_k, codes_v):
    """pages [bytes] (uint8, changed) with the rows' codes and words put in; codes_* =
    (code [T, H, D], step [T, H], lo [T, H])."""
    D = codes_k[0].shape[-1]
    n_kv = codes_k[0].shape[1]
    slab = KV.slab_bytes(D)
    per = min(page_bytes // slab, 2 * n_kv)
    n_pages = pages.size // page_bytes
    for t, (s, p) in enumerate(positions(rows, lens)):
        if p < 0:
            continue
        for h in range(n_kv):
            for which, (code, step, lo) in enumerate((codes_k, codes_v)):
                i = 2 * h + which
                page = int(table[s, p // KV.BLOCK, i // per])
                if page < 0 or page >= n_pages:
                    continue
                base = page * page_bytes + (i % per) * slab
                put = (KV.value_bytes if which else KV.key_bytes)(code[t, h], p % KV.BLOCK)
                word = int(KV.bf16_bits(step[t, h])) | int(KV.bf16_bits(lo[t, h])) << 16
                for j in range(4):
                    put[8 * D + 4 * (p % KV.BLOCK) + j] = (word >> (8 * j)) & 255
                for o, b in put.items():
                    pages[base + o] = b
    return pages
