"""KV attention and append on the GPU for the batches a server makes: prompts beside decode rows, long
prompts, long contexts of few rows, hundreds of sequences, and captured calls, in 64 bits."""
import numpy as np
import pytest

from oracle import kv_model as KV
from tests.kv_helpers import blocks, expected_pages, positions
from tests.test_gpu_kv import _gpu, bf16, bits, dev, fill, make_batch, make_pool, oracle_out, say, to_np, tolerance

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


def check(D, H, n_kv, page, rows, lens, max_rows=None, seed=0, repeat=2):
    g = np.random.default_rng(seed + D + H + len(rows) + max(lens))
    pool = make_pool(page, blocks(lens) * 2 * n_kv + 3)
    b, _ = make_batch(pool, H, n_kv, D, rows, lens, max_rows=max_rows)
    k, v, (ck, cv) = fill(pool, n_kv, D, lens, g, b)
    q = bf16(g, sum(rows), H, D, scale=1.3)
    scale = D ** -0.5
    ws = pool.kv_workspace(b)
    ws.fill_(255)
    outs = []
    for _ in range(repeat):
        out = torch.full((sum(rows), H, D), 7.0, dtype=torch.bfloat16, device="cuda")
        pool.kv_attention(b, dev(q), out, workspace=ws)
        torch.cuda.synchronize()
        outs.append(out)
    assert all(np.array_equal(bits(outs[0]), bits(o)) for o in outs), "runs must agree bit for bit"
    want, got = oracle_out(q, k, v, rows, n_kv, scale), to_np(outs[0])
    tol = tolerance(want, q, k, v, ck, cv, scale, D, max(rows) * H // n_kv)
    err = np.abs(got - want)
    print(f"[parity] worst err / tolerance {np.max(err / tol):.3f}", flush=True)
    assert np.all(np.isfinite(got)) and np.all(err <= tol)
    for t, (s, p) in enumerate(positions(rows, lens)):
        if p < 0 or lens[s] == 0:
            assert not got[t].any(), "a row that sees nothing is zero"


BATCHES = [
    # D, H, n_kv, page, rows, tokens
    (64, 32, 1, 512, [1100], [1100]),                     # 35,200 query rows of one head: 275 tiles
    (128, 4, 1, 1024, [40, 1], [20000, 3]),               # two tiles whose tokens are shared by very many
    (256, 4, 2, 4096, [200, 1, 1], [200, 900, 17]),
    (64, 8, 8, 1024, [64, 1, 17, 1, 1, 130, 1, 0, 1], [64, 900, 40, 1, 16, 131, 333, 50, 2]),
    (128, 6, 2, 1024, [150, 90, 1], [150, 400, 77]),      # three query heads a KV head
    (64, 5, 1, 512, [300, 2], [310, 5]),                  # five
    (128, 32, 8, 4096, [520, 1, 1, 1], [700, 1500, 3000, 64]),
    (128, 2, 2, 1024, [129], [60]),                       # 69 rows with nothing to see
]


@pytest.mark.parametrize("case", BATCHES, ids=[f"D{c[0]}-h{c[1]}-kv{c[2]}-{len(c[4])}x{max(c[4])}-{max(c[5])}" for c in BATCHES])
def test_prompts_beside_decode_rows(case):
    say("batch", case)
    check(*case)


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("group,rows", [(1, 1), (2, 1), (1, 2), (3, 1), (4, 1), (2, 4), (7, 1), (16, 1), (5, 3)])
def test_few_rows_of_every_width(D, group, rows):
    """1 to 16 query rows of a KV head: every kernel of few rows, with cut and whole segments."""
    say("few rows", D, group, rows)
    check(D, 2 * group, 2, 4096, [rows, rows, rows], [3001, rows, 33])


@pytest.mark.parametrize("n,m", [(300, 1), (1100, 1), (520, 20)])
def test_hundreds_of_sequences(n, m):
    """More sequences than a workgroup has threads, and than four times that; every 17th has m rows, every
    fifth none."""
    say("sequences", n, m)
    g = np.random.default_rng(n)
    rows = [0 if i % 5 == 4 else m if i % 17 == 0 else 1 for i in range(n)]
    lens = [int(x) for x in g.integers(0, 70, n)]
    check(64, 2, 1, 512, rows, lens)


def test_append_to_hundreds_of_sequences():
    """Every row finds its sequence among 1,100: the pages hold what single appends of them leave."""
    D, n_kv, n = 64, 1, 1100
    say("append to 1100 sequences")
    g = np.random.default_rng(5)
    rows = [int(x) for x in g.integers(0, 3, n)]
    lens = [r + int(x) for r, x in zip(rows, g.integers(0, 40, n))]
    pool = make_pool(512, blocks(lens) * 2 + 3)
    b, table = make_batch(pool, 1, n_kv, D, rows, lens)
    before = pool.pages.view(torch.uint8).cpu().numpy().copy()
    T = sum(rows)
    k, v = bf16(g, T, n_kv, D), bf16(g, T, n_kv, D)
    ko, vo = (torch.empty((T, n_kv, D), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    pool.kv_append(b, dev(k), dev(v), k_out=ko, v_out=vo)
    torch.cuda.synchronize()
    want = expected_pages(before, table, 2 * 512, rows, lens, KV.quantise(k), KV.quantise(v))
    assert np.array_equal(pool.pages.view(torch.uint8).cpu().numpy(), want)
    for got, x in ((ko, k), (vo, v)):
        assert np.array_equal(to_np(got), KV.bf16_round(KV.value(*KV.quantise(x)).astype(np.float32)))


def test_captured_mixed_batch_follows_the_lengths():
    """A captured call over prompts and decode rows, replayed at other lengths, with the program's own
    calls between the replays."""
    D, H, n_kv, rows, top = 128, 8, 2, [33, 1, 70, 1], [600, 400, 300, 64]
    say("captured mixed batch")
    g = np.random.default_rng(23)
    pool = make_pool(1024, blocks(top) * 2 * n_kv + 3)
    b, _ = make_batch(pool, H, n_kv, D, rows, top)
    k, v, (ck, cv) = fill(pool, n_kv, D, top, g, b)
    q = bf16(g, sum(rows), H, D)
    qd, ws, ws2 = dev(q), pool.kv_workspace(b), pool.kv_workspace(b)
    out = torch.zeros((sum(rows), H, D), dtype=torch.bfloat16, device="cuda")
    own = torch.zeros_like(out)
    pool.kv_attention(b, qd, out, workspace=ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        pool.kv_attention(b, qd, out, workspace=ws)
    for lens in (top, [33, 1, 70, 0], [599, 17, 71, 64], [40, 400, 5, 1], top):
        b.ctx_len.copy_(torch.tensor(lens, dtype=torch.int32))
        graph.replay()
        torch.cuda.synchronize()
        got = out.clone()
        out.fill_(3.0)
        pool.kv_attention(b, qd, own, workspace=ws2)
        torch.cuda.synchronize()
        assert np.array_equal(bits(got), bits(own)), lens
        want = oracle_out(q, [x[:n] for x, n in zip(k, lens)], [x[:n] for x, n in zip(v, lens)], rows, n_kv, D ** -0.5)
        assert np.all(np.abs(to_np(got) - want) <= tolerance(want, q, k, v, ck, cv, D ** -0.5, D, 99)), lens
