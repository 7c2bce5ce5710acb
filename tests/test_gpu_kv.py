"""Keys and values in the pool's KV pages on the GPU (kv_append, kv_attention) against
the 64-bit oracle.

Appended bytes are compared exactly: a code is the nearest of 16 levels of a bf16 row, and
the rotation of keys is computed in 64 bits before its one rounding to bf16, so the kernel
and the oracle agree bit for bit.  Tolerance of the attention, per output:
  2^-8 |want|            the output's one rounding (half a step of bf16)
  2 e max|v|             the scores' fp32 error e (a weight is off by the factor exp(+-e), and
                         so is their sum): D + 16 roundings of 2^-24 of at most
                         scale sum|q| (32 step + |lo|)
  w                      the weights' rounding: two bf16 halves, 2^-16 of 31 steps, or (more
                         than 16 query rows a KV head) one, 2^-8 of 8 steps
  2^-20 + N 2^-24        exp2 and the fp32 sums over N tokens, relative to the largest |v|
"""
import numpy as np
import pytest

from oracle import kv_model as KV
from tests.gpu_helpers import bits, to_np
from tests.kv_helpers import blocks, cos_sin, expected_pages, positions, table_of

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    import heterogeneous_adapter_gemm_amd as hg
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    hg.library()
    yield
    torch.cuda.synchronize()


def say(*a):
    print("[case]", *a, flush=True)


def bf16(g, *shape, scale=1.0):
    """Random bf16 values as float64."""
    return KV.bf16_round(g.standard_normal(shape).astype(np.float32) * scale)


def dev(x):
    return torch.from_numpy(np.ascontiguousarray(x, dtype=np.float32)).to("cuda").to(torch.bfloat16)


def make_pool(page, n_pages, seed=0):
    import heterogeneous_adapter_gemm_amd as hg
    order = np.random.default_rng(seed).permutation(n_pages)
    pool = hg.DevicePool(hg.LORA_BF16, page, n_pages, order, 1, [512], [512], 1, 8, 64, 1)
    pool.pages.view(torch.uint8).fill_(255)
    return pool


def make_batch(pool, H, n_kv, D, rows, lens, max_blocks=None, extra_rows=0, max_rows=None):
    import heterogeneous_adapter_gemm_amd as hg
    npb = pool.kv_pages_per_block(n_kv, D)
    nb = max(1, max(-(-n // KV.BLOCK) for n in lens)) if max_blocks is None else max_blocks
    table = table_of(pool.alloc_kv(blocks(lens) * npb), lens, npb, nb)
    starts = np.concatenate([[0], np.cumsum(rows)]).astype(np.int32)
    b = hg.KvBatch(H, n_kv, D, torch.from_numpy(starts).cuda(), torch.tensor(lens, dtype=torch.int32).cuda(),
                   torch.from_numpy(table).cuda(), int(starts[-1]) + extra_rows,
                   max_rows=max(rows) if max_rows is None else max_rows)
    return b, table


def host_pages(pool):
    return pool.pages.view(torch.uint8).cpu().numpy().copy()


# ---------------------------------------------------------------- append

APPEND = [
    # D, H, n_kv, rot, interleaved, page, rows, tokens after
    (128, 8, 2, 128, False, 1024, [1, 1, 1], [1, 17, 40]),
    (128, 4, 4, 64, True, 4096, [5, 0, 33], [5, 9, 50]),
    (64, 3, 3, 64, False, 1024, [16, 1], [16, 32]),
    (64, 10, 1, 32, True, 512, [3, 2, 1, 7], [3, 18, 1, 23]),
    (64, 2, 2, 16, False, 16384, [40], [40]),
    (256, 6, 3, 256, False, 4096, [2, 19], [33, 19]),
    (256, 2, 1, 128, True, 2048, [1], [16]),
    (128, 5, 5, 0, False, 1024, [9, 1], [9, 2]),
]


@pytest.mark.parametrize("case", APPEND, ids=[f"D{c[0]}-h{c[1]}-kv{c[2]}-rot{c[3]}-p{c[5]}" for c in APPEND])
def test_append_writes_exactly_the_rows(case):
    D, H, n_kv, rot, inter, page, rows, lens = case
    say("append", case)
    g = np.random.default_rng(D + H + rot + page)
    pool = make_pool(page, blocks(lens) * 2 * n_kv + 5)
    b, table = make_batch(pool, H, n_kv, D, rows, lens)
    T = sum(rows)
    q, k, v = bf16(g, T, H, D, scale=1.5), bf16(g, T, n_kv, D), bf16(g, T, n_kv, D, scale=0.3)
    k[0, 0] = 1.25                                       # a constant row: step 0
    v[-1, -1] *= 2.0 ** 120                              # a row of large values
    v[-1, 0, 1:] *= 2.0 ** -130                          # and one of tiny ones
    v = KV.bf16_round(v)                                 # (what the device gets: subnormals have fewer bits)
    cs = cos_sin(16 * table.shape[1], rot) if rot else None
    before = host_pages(pool)
    kd, vd, qd = dev(k), dev(v), dev(q)
    k_out, v_out, q_out = torch.empty_like(kd), torch.empty_like(vd), torch.empty_like(qd)
    pool.kv_append(b, kd, vd, q=qd, q_out=q_out, k_out=k_out, v_out=v_out,
                   cos_sin=None if cs is None else torch.from_numpy(cs).cuda(), interleaved=inter)
    torch.cuda.synchronize()
    pos = np.array([p for _, p in positions(rows, lens)])
    kr = KV.bf16_round(KV.rotate(k, pos, cs, inter)) if rot else k
    ck, cv = KV.quantise(kr), KV.quantise(v)
    want = expected_pages(before, table, 2 * page, rows, lens, ck, cv)
    assert np.array_equal(host_pages(pool), want)
    assert np.array_equal(to_np(k_out), KV.bf16_round(KV.value(*ck).astype(np.float32)))
    assert np.array_equal(to_np(v_out), KV.bf16_round(KV.value(*cv).astype(np.float32)))
    # two fp32 products and their sum, then half a step of bf16
    qr = KV.rotate(q, pos, cs, inter) if rot else q
    assert np.all(np.abs(to_np(q_out) - qr) <= 2.0 ** -8 * np.abs(qr) + 3 * 2.0 ** -24 * 2 * np.abs(q).max())
    # in place, and without q or the returned rows: the same bytes
    pool.pages.view(torch.uint8).fill_(255)
    pool.kv_append(b, kd, vd, q=qd, q_out=qd, k_out=kd, v_out=vd,
                   cos_sin=None if cs is None else torch.from_numpy(cs).cuda(), interleaved=inter)
    torch.cuda.synchronize()
    assert np.array_equal(host_pages(pool), want)
    assert np.array_equal(bits(qd), bits(q_out)) and np.array_equal(bits(kd), bits(k_out))
    assert np.array_equal(bits(vd), bits(v_out))
    pool.pages.view(torch.uint8).fill_(255)
    pool.kv_append(b, dev(k), dev(v), cos_sin=None if cs is None else torch.from_numpy(cs).cuda(), interleaved=inter)
    torch.cuda.synchronize()
    assert np.array_equal(host_pages(pool), want)


def test_append_strided_rows_of_one_fused_tensor():
    """q, k and v as slices of one [T, (H + 2 n_kv) D] tensor."""
    D, H, n_kv, rows, lens = 128, 6, 2, [3, 20], [7, 20]
    say("append from a fused tensor")
    g = np.random.default_rng(4)
    pool = make_pool(1024, 64)
    b, table = make_batch(pool, H, n_kv, D, rows, lens)
    T = sum(rows)
    x = bf16(g, T, (H + 2 * n_kv) * D)
    xd = dev(x)
    q, k, v = xd[:, :H * D], xd[:, H * D:(H + n_kv) * D], xd[:, (H + n_kv) * D:]
    cs = cos_sin(16 * table.shape[1], D)
    before = host_pages(pool)
    pool.kv_append(b, k, v, q=q, q_out=q, cos_sin=torch.from_numpy(cs).cuda())
    torch.cuda.synchronize()
    x3 = x.reshape(T, H + 2 * n_kv, D)
    pos = np.array([p for _, p in positions(rows, lens)])
    kr = KV.bf16_round(KV.rotate(x3[:, H:H + n_kv], pos, cs, False))
    want = expected_pages(before, table, 2048, rows, lens, KV.quantise(kr), KV.quantise(x3[:, H + n_kv:]))
    assert np.array_equal(host_pages(pool), want)
    assert np.array_equal(to_np(xd[:, H * D:]), x[:, H * D:])     # k and v themselves stay
    with pytest.raises(ValueError):
        pool.kv_append(b, k.t(), v)
    with pytest.raises(ValueError):
        pool.kv_append(b, k[:-1], v)
    with pytest.raises(ValueError):
        pool.kv_append(b, k.float(), v)


def test_append_leaves_out_what_has_no_place():
    """Rows behind the last sequence, rows before position 0, pages outside the pool, and rows of
    infinities or NaN (which read back as NaN and spoil nothing else)."""
    D, H, n_kv, rows, lens = 64, 2, 2, [4, 3, 2], [2, 40, 30]
    say("append: rows and pages that are left out")
    g = np.random.default_rng(5)
    pool = make_pool(512, 64)
    b, table = make_batch(pool, H, n_kv, D, rows, lens, extra_rows=5)
    table[1, 2, 0] = 64           # one past the pool
    table[2, 1, 1] = -1
    b.page_table.copy_(torch.from_numpy(table))
    T = sum(rows) + 5
    k, v, q = bf16(g, T, n_kv, D), bf16(g, T, n_kv, D), bf16(g, T, H, D)
    k[5, 1, 7] = np.nan
    v[8, 0, 0] = np.inf
    v[8, 1, 3] = -np.inf
    before = host_pages(pool)
    q_out = torch.full((T, H, D), 7.0, dtype=torch.bfloat16, device="cuda")
    k_out, v_out = (torch.full((T, n_kv, D), 7.0, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    pool.kv_append(b, dev(k), dev(v), q=dev(q), q_out=q_out, k_out=k_out, v_out=v_out)
    torch.cuda.synchronize()
    ck, cv = KV.quantise(k), KV.quantise(v)
    want = expected_pages(before, table, 1024, rows, lens, ck, cv)
    got = host_pages(pool)
    # a spoilt row's lo is whatever it is: only its step has to be NaN
    slab = KV.slab_bytes(D)
    for t, (s, p) in enumerate(positions(rows, lens)):
        for h in range(n_kv):
            for which, c in enumerate((ck, cv)):
                page = int(table[s, max(p, 0) // 16, (2 * h + which) // 1]) if p >= 0 else -1
                if p >= 0 and 0 <= page < 64 and np.isnan(c[1][t, h]):
                    o = page * 1024 + 8 * D + 4 * (p % 16)
                    word = got[o:o + 4].view(np.uint32)[0]
                    assert np.isnan(np.array([word << 16], np.uint32).view(np.float32)[0])
                    want[o:o + 4] = got[o:o + 4]
    assert pool.kv_pages_per_block(n_kv, D) == 4 and slab == 576
    assert np.array_equal(got, want)
    for out, val in ((q_out, q), (k_out, KV.value(*ck)), (v_out, KV.value(*cv))):
        o = to_np(out)
        kept = [i for i, (_, p) in enumerate(positions(rows, lens)) if p >= 0]
        left = [i for i in range(T) if i not in kept]
        assert np.all(o[left] == 7.0)
        assert np.array_equal(np.isnan(o[kept]), np.isnan(val[kept]))


# ---------------------------------------------------------------- attention

def fill(pool, n_kv, D, lens, g, table_batch, scale=1.0):
    """Append every sequence's whole history; returns the values the cache stands for, per sequence."""
    import heterogeneous_adapter_gemm_amd as hg
    T = sum(lens)
    starts = np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
    b = hg.KvBatch(n_kv, n_kv, D, torch.from_numpy(starts).cuda(), table_batch.ctx_len, table_batch.page_table, T)
    k = bf16(g, T, n_kv, D, scale=scale) + KV.bf16_round(g.standard_normal((n_kv, D)))
    k, v = KV.bf16_round(k), bf16(g, T, n_kv, D, scale=0.7)
    if T:
        pool.kv_append(b, dev(k), dev(v))
    ck, cv = KV.quantise(k), KV.quantise(v)
    cut = lambda c: [KV.value(*c)[a:z] for a, z in zip(starts, starts[1:])]  # noqa: E731
    return cut(ck), cut(cv), (ck, cv)


def tolerance(want, q, k, v, ck, cv, scale, D, rows_a_head):
    """See the module's docstring; q [T, H, D], k and v lists per sequence."""
    if not any(x.size for x in k):
        return np.zeros_like(want) + 1e-30
    step_k, lo_k, step_v, lo_v = (np.nanmax(np.abs(x)) for x in (ck[1], ck[2], cv[1], cv[2]))
    n = max(x.shape[0] for x in k)
    e = scale * (D + 16) * 2.0 ** -24 * np.abs(q).sum(-1).max() * (32 * step_k + lo_k)
    vmax = lo_v + 32 * step_v
    w = 2.0 ** -16 * 31 * step_v if rows_a_head <= 16 else 2.0 ** -8 * 8 * step_v
    return 2.0 ** -8 * np.abs(want) + 2 * e * vmax + w + (2.0 ** -20 + n * 2.0 ** -24) * vmax


def oracle_out(q, k, v, rows, n_kv, scale, hidden=None):
    out, at = [], 0
    for s, n in enumerate(rows):
        out.append(KV.attention(q[at:at + n], k[s], v[s], n_kv, scale, (hidden or {}).get(s, ())))
        at += n
    return np.concatenate(out) if out else np.zeros((0,) + q.shape[1:])


ATTEND = [
    # D, H, n_kv, page, rows, tokens
    (128, 8, 2, 1024, [1, 1, 1, 1], [1, 15, 16, 17]),
    (128, 4, 4, 4096, [1, 1, 1, 1, 1], [31, 32, 33, 64, 129]),
    (64, 12, 1, 512, [3, 3, 2], [3, 40, 700]),                  # three drafted rows, one KV head: 36 query rows
    (64, 7, 7, 2048, [1, 0, 1], [5, 12, 0]),                    # no rows; no tokens
    (128, 10, 2, 1024, [4, 2], [2, 1]),                         # more rows than tokens: the first see nothing
    (256, 4, 2, 4096, [1, 2], [300, 77]),
    (128, 32, 8, 4096, [1] * 9, [1000, 1, 130, 257, 4100, 16, 511, 640, 2]),
    (128, 16, 1, 1024, [1, 1], [4097, 33]),
    (64, 40, 1, 512, [1, 1], [200, 65]),                        # 40 query rows of one token
    (128, 8, 2, 1024, [70, 1, 33], [70, 200, 300]),             # prompts and a decode row
    (64, 3, 3, 1024, [129], [400]),
    (256, 2, 1, 2048, [40, 5], [90, 5]),
    (128, 4, 4, 1024, [100], [60]),                             # 40 rows with nothing to see
    (128, 4, 2, 1024, [40], [3000]),
]


@pytest.mark.parametrize("case", ATTEND, ids=[f"D{c[0]}-h{c[1]}-kv{c[2]}-{len(c[4])}x{max(c[4])}-{max(c[5])}" for c in ATTEND])
def test_attention(case):
    D, H, n_kv, page, rows, lens = case
    say("attention", case)
    g = np.random.default_rng(D + H + len(rows) + max(lens))
    pool = make_pool(page, blocks(lens) * 2 * n_kv + 3)
    b, _ = make_batch(pool, H, n_kv, D, rows, lens)
    k, v, (ck, cv) = fill(pool, n_kv, D, lens, g, b)
    T = sum(rows)
    q = bf16(g, T, H, D, scale=1.3)
    scale = D ** -0.5
    ws = pool.kv_workspace(b)
    ws.fill_(255)
    out = torch.full((T, H, D), 7.0, dtype=torch.bfloat16, device="cuda")
    pool.kv_attention(b, dev(q), out, workspace=ws)
    out2 = torch.empty_like(out)
    pool.kv_attention(b, dev(q), out2, workspace=ws)
    torch.cuda.synchronize()
    assert np.array_equal(bits(out), bits(out2)), "two runs must agree bit for bit"
    want = oracle_out(q, k, v, rows, n_kv, scale)
    got = to_np(out)
    tol = tolerance(want, q, k, v, ck, cv, scale, D, max(rows) * H // n_kv)
    err = np.abs(got - want)
    print(f"[parity] worst err / tolerance {np.max(err / tol):.3f}, max err {err.max():.2e}", flush=True)
    assert np.all(np.isfinite(got)) and np.all(err <= tol)
    for t, (s, p) in enumerate(positions(rows, lens)):
        if p < 0 or lens[s] == 0:
            assert not got[t].any(), "a row that sees nothing is zero"


def test_attention_kernels_agree_whatever_max_rows_says():
    """max_rows too small, exact or too large chooses other kernels, the same rows."""
    D, H, n_kv, rows, lens = 128, 8, 2, [37, 1, 9], [37, 500, 90]
    say("attention under max_rows 1, 37, 4000")
    g = np.random.default_rng(12)
    pool = make_pool(1024, 512)
    b, table = make_batch(pool, H, n_kv, D, rows, lens)
    k, v, (ck, cv) = fill(pool, n_kv, D, lens, g, b)
    q = bf16(g, sum(rows), H, D)
    want = oracle_out(q, k, v, rows, n_kv, 0.1)
    import heterogeneous_adapter_gemm_amd as hg
    for most in (1, 37, 4000):
        bb = hg.KvBatch(H, n_kv, D, b.row_start, b.ctx_len, b.page_table, sum(rows), max_rows=most)
        out = torch.empty((sum(rows), H, D), dtype=torch.bfloat16, device="cuda")
        pool.kv_attention(bb, dev(q), out, scale=0.1, workspace=pool.kv_workspace(bb))
        torch.cuda.synchronize()
        assert np.all(np.abs(to_np(out) - want) <= tolerance(want, q, k, v, ck, cv, 0.1, D, 999))


def test_attention_extreme_scores_and_values():
    """Scores far apart (one token takes all the weight, and the running maximum rises late), equal
    keys, and values of very different size."""
    D, H, n_kv, lens = 128, 2, 1, [600, 600, 600]
    say("attention: extreme scores")
    import heterogeneous_adapter_gemm_amd as hg
    g = np.random.default_rng(13)
    pool = make_pool(1024, 1024)
    b, _ = make_batch(pool, H, n_kv, D, [1, 1, 1], lens)
    starts = np.array([0, 600, 1200, 1800], np.int32)
    k, v = bf16(g, 1800, 1, D), bf16(g, 1800, 1, D)
    k[:600] *= np.arange(1, 601)[:, None, None] / 20           # ever larger scores
    k[600:1200] = k[600]                                       # all the same
    v[1200:1500] *= 2.0 ** 20
    v[1500:] *= 2.0 ** -20
    k = KV.bf16_round(k)
    v = KV.bf16_round(v)
    hb = hg.KvBatch(1, 1, D, torch.from_numpy(starts).cuda(), b.ctx_len, b.page_table, 1800)
    pool.kv_append(hb, dev(k), dev(v))
    ck, cv = KV.quantise(k), KV.quantise(v)
    q = bf16(g, 3, H, D, scale=2.0)
    out = torch.empty((3, H, D), dtype=torch.bfloat16, device="cuda")
    pool.kv_attention(b, dev(q), out, scale=1.0, workspace=pool.kv_workspace(b))
    torch.cuda.synchronize()
    kk, vv = KV.value(*ck), KV.value(*cv)
    for s in range(3):
        a, z = starts[s], starts[s + 1]
        want = KV.attention(q[s:s + 1], kk[a:z], vv[a:z], 1, 1.0)
        cut = lambda c: tuple(x[a:z] for x in c)  # noqa: E731
        tol = tolerance(want, q[s:s + 1], [kk[a:z]], [vv[a:z]], cut(ck), cut(cv), 1.0, D, 2)
        assert np.all(np.abs(to_np(out)[s:s + 1] - want) <= tol), s


def test_attention_leaves_out_bad_pages_and_foreign_rows():
    """Tokens of pages outside the pool are left out; rows behind the last sequence stay; a spoilt
    cached row spoils the rows that see it and no other."""
    D, H, n_kv, rows, lens = 64, 4, 2, [1, 30, 2], [100, 60, 50]
    say("attention: bad pages, padded rows, a spoilt key")
    g = np.random.default_rng(14)
    pool = make_pool(512, 256)
    b, table = make_batch(pool, H, n_kv, D, rows, lens, extra_rows=4)
    k, v, (ck, cv) = fill(pool, n_kv, D, lens, g, b)
    bad = table.copy()
    bad[0, 3, :] = [-1, 256, -5, 2 ** 31 - 1]      # tokens 48..63 of sequence 0
    bad[1, 0, :] = 1 << 20                         # tokens 0..15 of sequence 1
    b.page_table.copy_(torch.from_numpy(bad))
    T = sum(rows) + 4
    q = bf16(g, T, H, D)
    out = torch.full((T, H, D), 7.0, dtype=torch.bfloat16, device="cuda")
    ws = pool.kv_workspace(b)
    pool.kv_attention(b, dev(q), out, workspace=ws)
    torch.cuda.synchronize()
    got = to_np(out)
    n = sum(rows)
    want = oracle_out(q[:n], k, v, rows, n_kv, 0.125, hidden={0: range(48, 64), 1: range(16)})
    assert np.all(got[n:] == 7.0)
    assert np.all(np.abs(got[:n] - want) <= tolerance(want, q[:n], k, v, ck, cv, 0.125, D, 60))
    # now token 45 of sequence 1 (row 15 of its 30) holds NaN
    b.page_table.copy_(torch.from_numpy(table))
    pool.kv_attention(b, dev(q), out, workspace=ws)
    torch.cuda.synchronize()
    clean = to_np(out)
    words = pool.pages.view(torch.int32)
    page = int(table[1, 45 // 16, 1])              # head 0's values
    words[page * 256 + 2 * D + 45 % 16] = -1
    pool.kv_attention(b, dev(q), out, workspace=ws)
    torch.cuda.synchronize()
    spoilt = to_np(out)
    hit = np.zeros((T, H), bool)
    hit[1 + 15:1 + 30, :2] = True                  # rows at positions 45.., query heads of KV head 0
    assert np.isnan(spoilt[hit]).all()
    assert np.array_equal(spoilt[~hit], clean[~hit])


def test_attention_bounds_wild_lengths():
    """Lengths past the table, negative ones and row starts past the batch stay inside the buffers."""
    D, H, n_kv = 64, 2, 1
    say("attention and append: wild lengths")
    import heterogeneous_adapter_gemm_amd as hg
    g = np.random.default_rng(15)
    pool = make_pool(512, 64)
    b, table = make_batch(pool, H, n_kv, D, [1, 1, 1], [32, 32, 32])
    k, v, _ = fill(pool, n_kv, D, [32, 32, 32], g, b)
    before = host_pages(pool)
    wild = hg.KvBatch(H, n_kv, D, torch.tensor([-3, 1, 2, 1 << 30], dtype=torch.int32, device="cuda"),
                      torch.tensor([1 << 30, -7, 32], dtype=torch.int32, device="cuda"), b.page_table, 3, max_rows=1)
    q = bf16(g, 3, H, D)
    out = torch.full((3, H, D), 7.0, dtype=torch.bfloat16, device="cuda")
    pool.kv_attention(wild, dev(q), out, scale=0.125, workspace=pool.kv_workspace(wild))
    torch.cuda.synchronize()
    got = to_np(out)
    want0 = KV.attention(q[:1], k[0], v[0], 1, 0.125)       # bounded to the table's 32 tokens
    assert np.abs(got[0] - want0[0]).max() < 0.05
    assert not got[1].any()
    want2 = KV.attention(q[2:], k[2], v[2], 1, 0.125)
    assert np.abs(got[2] - want2[0]).max() < 0.05
    pool.kv_append(wild, dev(bf16(g, 3, 1, D)), dev(bf16(g, 3, 1, D)))
    torch.cuda.synchronize()
    changed = np.nonzero((host_pages(pool) != before).reshape(64, 1024).any(1))[0]
    assert set(changed) <= {int(p) for p in table[[0, 2]].reshape(-1)}


def test_pages_past_four_gib():
    """Pages whose byte offset passes 32 bits."""
    D, H, n_kv, lens = 128, 4, 2, [50, 1]
    say("pages past 4 GiB")
    import heterogeneous_adapter_gemm_amd as hg
    page, n_pages = 1 << 20, 2600                   # 2 MiB pages, 5.2 GiB
    order = np.arange(n_pages)[::-1].copy()
    pool = hg.DevicePool(hg.LORA_BF16, page, n_pages, order, 1, [512], [512], 1, 8, 64, 1)
    b, table = make_batch(pool, H, n_kv, D, [1, 1], lens)
    assert int(table.max()) * 2 * page > 1 << 32
    g = np.random.default_rng(16)
    k, v, (ck, cv) = fill(pool, n_kv, D, lens, g, b)
    q = bf16(g, 2, H, D)
    out = torch.empty((2, H, D), dtype=torch.bfloat16, device="cuda")
    pool.kv_attention(b, dev(q), out, workspace=pool.kv_workspace(b))
    torch.cuda.synchronize()
    want = oracle_out(q, k, v, [1, 1], n_kv, D ** -0.5)
    assert np.all(np.abs(to_np(out) - want) <= tolerance(want, q, k, v, ck, cv, D ** -0.5, D, 2))


def test_captured_steps_follow_the_lengths():
    """One captured append and attention, replayed step after step: the kernels read the lengths and
    the table from device memory, so each replay appends at the new position and sees one token more."""
    D, H, n_kv, lens = 128, 8, 2, [14, 130, 1]
    say("captured decode steps")
    import heterogeneous_adapter_gemm_amd as hg
    g = np.random.default_rng(17)
    pool = make_pool(1024, 256)
    top = [n + 8 for n in lens]
    b, table = make_batch(pool, H, n_kv, D, [1, 1, 1], top)
    b.ctx_len.copy_(torch.tensor(lens, dtype=torch.int32))
    fb, _ = b, None
    k, v, _ = fill(pool, n_kv, D, lens, g, fb)
    kd, vd, qd = (torch.zeros((3, h, D), dtype=torch.bfloat16, device="cuda") for h in (n_kv, n_kv, H))
    qo, out = torch.zeros_like(qd), torch.zeros_like(qd)
    ws = pool.kv_workspace(b)
    cs_h = cos_sin(16 * table.shape[1], D)
    cs = torch.from_numpy(cs_h).cuda()

    def step():
        pool.kv_append(b, kd, vd, q=qd, q_out=qo, cos_sin=cs)
        pool.kv_attention(b, qo, out, workspace=ws)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    keep = pool.pages.clone()
    with torch.cuda.stream(side):
        step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        step()
    pool.pages.copy_(keep)
    kk, vv, now = [list(x) for x in k], [list(x) for x in v], list(lens)
    for i in range(6):
        now = [n + 1 for n in now]
        nk, nv, nq = bf16(g, 3, n_kv, D), bf16(g, 3, n_kv, D), bf16(g, 3, H, D)
        kd.copy_(dev(nk)); vd.copy_(dev(nv)); qd.copy_(dev(nq))
        b.ctx_len.copy_(torch.tensor(now, dtype=torch.int32))
        graph.replay()
        torch.cuda.synchronize()
        got, turned = to_np(out), to_np(qo)
        out.fill_(3.0)
        step()                                     # the same step run at once gives the same bits
        torch.cuda.synchronize()
        assert np.array_equal(to_np(out), got)
        pos = np.array([n - 1 for n in now])
        rk = KV.value(*KV.quantise(KV.bf16_round(KV.rotate(nk, pos, cs_h, False))))
        rv = KV.value(*KV.quantise(nv))
        for s in range(3):
            kk[s].append(rk[s]); vv[s].append(rv[s])
            want = KV.attention(turned[s:s + 1], np.array(kk[s]), np.array(vv[s]), n_kv, D ** -0.5)
            assert np.abs(got[s] - want[0]).max() <= 2.0 ** -8 * np.abs(want).max() + 1e-3, (i, s)


def test_two_streams_with_a_workspace_each():
    """Attention over one cache from two streams at once, each with its own workspace and output."""
    D, H, n_kv, lens = 128, 8, 1, [3000, 2000]
    say("two streams")
    g = np.random.default_rng(18)
    pool = make_pool(1024, 1024)
    b, _ = make_batch(pool, H, n_kv, D, [1, 1], lens)
    fill(pool, n_kv, D, lens, g, b)
    qs = [dev(bf16(g, 2, H, D)) for _ in range(2)]
    alone, ws = [], [pool.kv_workspace(b) for _ in range(2)]
    for q in qs:
        o = torch.empty_like(q)
        pool.kv_attention(b, q, o, workspace=ws[0])
        alone.append(o)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = [torch.empty_like(q) for q in qs]
    for i in range(2):
        for _ in range(8):
            pool.kv_attention(b, qs[i], outs[i], workspace=ws[i], stream=streams[i])
    torch.cuda.synchronize()
    for i in range(2):
        assert np.array_equal(bits(outs[i]), bits(alone[i]))


def test_empty_batches_and_wrong_tables():
    say("empty batches")
    import heterogeneous_adapter_gemm_amd as hg
    pool = make_pool(1024, 16)
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32, device="cuda")  # noqa: E731
    b = hg.KvBatch(4, 2, 128, i32(1), i32(0), i32(0, 3, 4), 0)
    e = torch.empty((0, 4, 128), dtype=torch.bfloat16, device="cuda")
    pool.kv_attention(b, e, e, workspace=pool.kv_workspace(b))
    pool.kv_append(b, e[:, :2], e[:, :2])
    with pytest.raises(ValueError, match="pages a block"):
        pool.kv_attention(hg.KvBatch(4, 2, 128, i32(2), i32(1), i32(1, 3, 3), 0), e, e, workspace=pool.kv_workspace(b))
    with pytest.raises(ValueError):
        hg.KvBatch(4, 2, 128, i32(2), i32(1), i32(1, 3, 4).long(), 0)
    with pytest.raises(ValueError):
        hg.KvBatch(4, 2, 128, i32(3), i32(1), i32(1, 3, 4), 0)
    with pytest.raises(ValueError, match="workspace"):
        pool.kv_attention(b, e, e)
    torch.cuda.synchronize()
