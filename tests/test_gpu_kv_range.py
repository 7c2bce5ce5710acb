"""The append's 4-bit rows over the whole range of bf16: rows whose greatest value less their least passes
what fp32 holds, rows at its ends, and tiny ones, beside ordinary rows; bytes compared exactly."""
import numpy as np
import pytest

from oracle import kv_model as KV
from tests.gpu_helpers import to_np
from tests.kv_helpers import blocks, expected_pages
from tests.test_gpu_kv import _gpu, bf16, dev, host_pages, make_batch, make_pool, say

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

MOST = float(np.uint32(0x7F7F0000).view(np.float32))    # the greatest bf16


def wide(g, T, n_kv, D):
    """bf16 rows [T, n_kv, D] of every kind, one after another."""
    x = bf16(g, T, n_kv, D)
    for t in range(T):
        for h in range(n_kv):
            r = g.uniform(-1, 1, D)
            kind = (t + 3 * h) % 6
            if kind == 0:
                x[t, h] = r * 3e38                      # a range that overflows
                x[t, h, :3] = -3e38, 3e38, 1e38
            elif kind == 1:
                x[t, h] = r * MOST                      # the whole of it
                x[t, h, -2:] = -MOST, MOST
            elif kind == 2:
                x[t, h] = 2e38 + r * 1e38               # large values, a range that fits
            elif kind == 3:
                x[t, h] = r * 2.0 ** -128               # subnormal ones
    return KV.bf16_round(x)


@pytest.mark.parametrize("D,n_kv", [(64, 3), (128, 2), (128, 32), (256, 2)])
def test_rows_of_every_range(D, n_kv):
    say("append: the whole range", D, n_kv)
    g = np.random.default_rng(D + n_kv)
    rows, lens, page = [37, 1, 20], [40, 17, 20], 2048
    pool = make_pool(page, blocks(lens) * 2 * n_kv + 5)
    b, table = make_batch(pool, 2 * n_kv, n_kv, D, rows, lens)
    k, v = wide(g, sum(rows), n_kv, D), wide(g, sum(rows), n_kv, D)
    ck, cv = KV.quantise(k), KV.quantise(v)
    assert (v.max(-1) - v.min(-1)).max() > np.finfo(np.float32).max and set(np.unique(cv[0])) == set(range(16))
    before = host_pages(pool)
    ko, vo = (torch.empty(k.shape, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    pool.kv_append(b, dev(k), dev(v), k_out=ko, v_out=vo)
    torch.cuda.synchronize()
    want = expected_pages(before, table, 2 * page, rows, lens, ck, cv)
    assert np.array_equal(host_pages(pool), want)
    with np.errstate(over="ignore"):
        for got, c in ((ko, ck), (vo, cv)):
            assert np.array_equal(to_np(got), KV.bf16_round(KV.value(*c).astype(np.float32)))
