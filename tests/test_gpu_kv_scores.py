"""KV attention where the scores lie far from zero, in every kernel: each output within the bound of its
own row (tests/kv_bounds.py), which all zeros and a lost token are outside of."""
import numpy as np
import pytest

from oracle import kv_model as KV
from tests.gpu_helpers import bits, to_np
from tests.kv_bounds import batch_bounds, outside, telling
from tests.kv_helpers import blocks
from tests.test_gpu_kv import _gpu, dev, make_batch, make_pool, say

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


def far_rows(g, T, H, n_kv, tokens, D, mean):
    """q, k, v and a scale with scores of about ``mean`` and weights of very different size."""
    q = KV.bf16_round((2 + 0.1 * g.standard_normal((T, H, D))).astype(np.float32))
    k = KV.bf16_round((np.sign(mean) * 2 + 0.1 * g.standard_normal((tokens, n_kv, D))).astype(np.float32))
    v = KV.bf16_round(g.standard_normal((tokens, n_kv, D)).astype(np.float32))
    return q, k, v, abs(mean) / (4 * D)


def attend(pool, b, table_lens, q, k, v, scale):
    """The cache of these keys and values, and the attention over it, twice."""
    import heterogeneous_adapter_gemm_amd as hg
    starts = np.concatenate([[0], np.cumsum(table_lens)]).astype(np.int32)
    n_kv, D = k.shape[1:]
    fill = hg.KvBatch(n_kv, n_kv, D, torch.from_numpy(starts).cuda(), b.ctx_len, b.page_table, int(starts[-1]))
    pool.kv_append(fill, dev(k), dev(v))
    outs = []
    for _ in range(2):
        out = torch.full(q.shape, 7.0, dtype=torch.bfloat16, device="cuda")
        pool.kv_attention(b, dev(q), out, scale=scale, workspace=pool.kv_workspace(b))
        torch.cuda.synchronize()
        outs.append(out)
    assert np.array_equal(bits(outs[0]), bits(outs[1])), "runs must agree bit for bit"
    return to_np(outs[0])


BATCHES = {
    # query heads over KV heads, rows and tokens of the sequences
    "one row": (1, 1, [1, 1], [600, 1]),
    "two rows": (2, 1, [1, 1], [600, 33]),
    "four rows": (4, 1, [1, 1], [600, 33]),
    "eight rows": (4, 1, [2, 1], [600, 33]),
    "sixteen rows": (16, 1, [1, 1], [600, 33]),
    "tiles of sixteen": (12, 1, [3, 3], [600, 3]),
    "a prompt": (2, 2, [100], [100]),                           # row 0 at position 0
    "cut tiles": (1, 1, [150], [1900]),
    "prompts and decode rows": (4, 2, [70, 1, 1], [700, 300, 2]),
    "whole tiles": (8, 8, [65] * 80, [65 + i % 3 for i in range(80)]),
}


CASES = [(name, D, mean) for name in BATCHES for D in (64, 128, 256) for mean in (-89, -150, -1000, 150, 1000)
         if name != "whole tiles" or (D == 128 and mean < 0)]


@pytest.mark.parametrize("name,D,mean", CASES)
def test_scores_far_from_zero(name, D, mean):
    H, n_kv, rows, lens = BATCHES[name]
    say("scores near", mean, name, D)
    g = np.random.default_rng(abs(mean) + D + len(rows))
    page = 512 if D == 64 else 1024 if D == 128 else 2048
    pool = make_pool(page, blocks(lens) * 2 * n_kv + 3)
    b, _ = make_batch(pool, H, n_kv, D, rows, lens)
    q, k, v, scale = far_rows(g, sum(rows), H, n_kv, sum(lens), D, mean)
    got = attend(pool, b, lens, q, k, v, scale)
    want, bound, drop = batch_bounds(q, KV.quantise(k), KV.quantise(v), rows, lens, n_kv, scale)
    zero, lost = telling(want, bound, drop)
    print(f"[parity] worst err / bound {np.nanmax(np.abs(got - want) / bound):.3f}, NaN {np.isnan(got).sum()}, "
          f"told from zero {zero:.3f}, from a lost token {lost:.3f}", flush=True)
    assert zero == 1 and lost == 1
    assert not outside(got, want, bound).any()
