"""KV attention in every kernel with a bound for each output from its own row (tests/kv_bounds.py): ordinary
batches, one row count after another, prompts beside decode rows, and rows whose scores rise, are equal, or
whose values differ very much in size.  Sequences of at most 64 query rows of a KV head keep their
weights in two bf16 halves, longer ones in one."""
import numpy as np
import pytest

from oracle import kv_model as KV
from tests.kv_bounds import FEW_ROWS, batch_bounds, outside, telling
from tests.kv_helpers import blocks
from tests.test_gpu_kv import ATTEND, _gpu, bf16, make_batch, make_pool, say
from tests.test_gpu_kv_batches import BATCHES
from tests.test_gpu_kv_scores import attend

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


def ordinary(g, T, H, n_kv, tokens, D):
    k = bf16(g, tokens, n_kv, D) + KV.bf16_round(g.standard_normal((n_kv, D)))
    return bf16(g, T, H, D, scale=1.3), KV.bf16_round(k), bf16(g, tokens, n_kv, D, scale=0.7)


def check(D, H, n_kv, page, rows, lens, q, k, v, scale=None, max_rows=None):
    pool = make_pool(page, blocks(lens) * 2 * n_kv + 3)
    b, _ = make_batch(pool, H, n_kv, D, rows, lens, max_rows=max_rows)
    scale = D ** -0.5 if scale is None else scale
    got = attend(pool, b, lens, q, k, v, scale)
    most = max(rows) if max_rows is None else max_rows
    few = True if most * H // n_kv <= FEW_ROWS else None
    want, bound, drop = batch_bounds(q, KV.quantise(k), KV.quantise(v), rows, lens, n_kv, scale, few)
    zero, lost = telling(want, bound, drop)
    print(f"[parity] worst err / bound {np.max(np.abs(got - want) / np.where(bound > 0, bound, 1e-30)):.3f}, told from zero "
          f"{zero:.3f}, from a lost token {lost:.3f}", flush=True)
    # (a rounding a token adds up to a heavy token's weight where there are very many)
    assert zero == 1 and (lost == 1 or max(lens) > 5000)
    assert not outside(got, want, bound).any()


PLAIN = [c + (None,) for c in ATTEND + BATCHES] + [
    (D, 2 * G, 2, 4096, [n, n, n], [1301, n, 33], None) for D in (64, 128, 256)
    for G, n in [(1, 1), (2, 1), (1, 2), (3, 1), (2, 4), (7, 1), (16, 1), (5, 3), (1, 17), (8, 3), (16, 4), (13, 5)]] + [
    (128, 8, 2, 1024, [37, 1, 9], [37, 500, 90], m) for m in (1, 2, 4, 16, 37, 4000)]


@pytest.mark.parametrize("case", PLAIN, ids=[f"D{c[0]}-h{c[1]}-kv{c[2]}-{len(c[4])}x{max(c[4])}-{max(c[5])}-{c[6]}" for c in PLAIN])
def test_ordinary_rows(case):
    D, H, n_kv, page, rows, lens, most = case
    say("bounds", case)
    g = np.random.default_rng(D + H + len(rows) + max(lens) + 1)
    check(D, H, n_kv, page, rows, lens, *ordinary(g, sum(rows), H, n_kv, sum(lens), D), max_rows=most)


KINDS = ["rising", "falling", "equal", "one large", "values apart"]
ROWS = [(1, [1]), (2, [1]), (4, [1]), (8, [1]), (16, [1]), (4, [9]), (2, [90]), (1, [200]), (4, [60, 1])]


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("G,rows", ROWS, ids=[f"{g}x{'+'.join(map(str, r))}" for g, r in ROWS])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_rows_of_uneven_scores_and_values(D, G, rows, kind):
    say("uneven", D, G, rows, kind)
    g = np.random.default_rng(D + G + rows[0] + KINDS.index(kind))
    lens = [700, 300][:len(rows)]
    q, k, v = ordinary(g, sum(rows), G, 1, sum(lens), D)
    at = np.concatenate([np.arange(n) for n in lens]) / 700.0
    if kind == "rising":
        q, k = q + 1, k + 5 * at[:, None, None] * D ** -0.25       # the maximum rises all the way
    elif kind == "falling":
        q, k = q + 1, k - 5 * at[:, None, None] * D ** -0.25       # the first tokens take it all
    elif kind == "equal":
        k[:] = k[0]
    elif kind == "one large":
        q = q + 1
        k[lens[0] // 2] += 20 * D ** -0.25
    else:
        v[:350] *= 2.0 ** 20
        v[350:] *= 2.0 ** -20
    q, k, v = KV.bf16_round(q), KV.bf16_round(k), KV.bf16_round(v)
    check(D, G, 1, 2048, rows, lens, q, k, v)


@pytest.mark.parametrize("G,rows", [(1, [1]), (8, [3]), (4, [60])])
def test_large_values_keep_their_room(G, rows):
    """q, k and v of up to 2^56 in size."""
    say("large values", G, rows)
    D, lens = 128, [500]
    g = np.random.default_rng(G)
    q, k, v = ordinary(g, sum(rows), G, 1, 500, D)
    assert max(np.abs(x).max() for x in (q, k, v)) < 8
    check(D, G, 1, 1024, rows, lens, q * 2.0 ** 53, k * 2.0 ** 53, v * 2.0 ** 53, scale=2.0 ** -106 * D ** -0.5)


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("G,n", [(5, 4), (4, 16), (64, 1)])
def test_up_to_64_query_rows_in_the_workspace_of_few(D, G, n):
    """The workspace of sequences of 16 query rows of a KV head, and nothing behind it touched."""
    import heterogeneous_adapter_gemm_amd as hg
    from tests.gpu_helpers import to_np
    from tests.test_gpu_kv import dev
    say("small workspace", D, G, n)
    g = np.random.default_rng(D + G)
    rows, lens = [n, 1, n], [900, 40, n]
    pool = make_pool(2048, blocks(lens) * 2 + 3)
    b, _ = make_batch(pool, G, 1, D, rows, lens)
    q, k, v = ordinary(g, sum(rows), G, 1, sum(lens), D)
    attend(pool, b, lens, q, k, v, D ** -0.5)
    few = hg.lora_kv_workspace_bytes(hg.lora_kv_batch(1, 1, D, 1, 1, 1, 1, 0, None, None, None))
    assert few < hg.lora_kv_workspace_bytes(b.c)
    ws = torch.full((few + 4096,), 255, dtype=torch.uint8, device="cuda")
    out = torch.empty(q.shape, dtype=torch.bfloat16, device="cuda")
    pool.kv_attention(b, dev(q), out, workspace=ws[:few])
    torch.cuda.synchronize()
    assert bool((ws[few:] == 255).all())
    want, bound, _ = batch_bounds(q, KV.quantise(k), KV.quantise(v), rows, lens, 1, D ** -0.5)
    assert not outside(to_np(out), want, bound).any()
