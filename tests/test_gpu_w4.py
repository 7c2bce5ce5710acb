"""The 4-bit base on the GPU (base_gemm_w4, lora_linear_w4) in 64 bits, and the attention
block of a layer served in 4 bits end to end.

Tolerance of the product, per output: half a step of bf16 (2^-8 of the value) and the fp32
sums: K terms of at most scale (16 + 15) |x| and, for the zero point, scale (16 + zero) |x|,
each with a rounding of 2^-24 on the way (a product's sum over K passes K / 32 + 32 of them).
"""
import numpy as np
import pytest

from oracle import kv_model as KV
from tests.gpu_helpers import bf16_bits, bits, to_np
from tests.kv_helpers import cos_sin
from tests.test_gpu_kv import bf16, dev, make_batch, make_pool, oracle_out, tolerance

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


def weight(g, N, K, group, std=0.02):
    """(codes, scale, zero, the weight in 64 bits, and the packed device tensors)."""
    code = g.integers(0, 16, (N, K))
    scale = (g.uniform(0.3, 1.0, (N, K // group)) * std / 4).astype(np.float16)
    zero = g.integers(0, 16, (N, K // group)).astype(np.float16)
    zero[0] = 7.5                                        # zeros need not be whole
    scale[-1] = 0
    per = lambda t: np.repeat(t.astype(np.float64), group, 1)  # noqa: E731
    w = per(scale) * (code - per(zero))
    packed = torch.from_numpy((code[:, 0::2] | code[:, 1::2] << 4).astype(np.uint8)).cuda()
    sz = torch.from_numpy(np.ascontiguousarray(np.stack([scale, zero], -1))).cuda()
    return scale, zero, w, packed, sz


def product_tolerance(want, x, scale, zero, K):
    size = 32 * float(np.abs(scale.astype(np.float64)).max())
    return 2.0 ** -8 * np.abs(want) + 2 * (K / 32 + 32) * 2.0 ** -24 * size * np.abs(x).sum(-1, keepdims=True)


SHAPES = [(1, 16, 128, 128), (1, 4096, 4096, 128), (3, 20, 256, 32), (16, 528, 1152, 64), (17, 4, 128, 32), (31, 260, 512, 128),
          (33, 1000, 640, 64), (64, 4096, 1024, 128), (65, 1004, 384, 32), (130, 516, 768, 128), (300, 272, 640, 64),
          (520, 1040, 256, 32), (48, 10244, 256, 128), (70, 10260, 384, 64), (40, 10240, 128, 32), (520, 4100, 384, 128),
          (1100, 2052, 256, 64), (129, 16388, 128, 32)]


@pytest.mark.parametrize("M,N,K,group", SHAPES)
def test_base_gemm_w4(M, N, K, group):
    import heterogeneous_adapter_gemm_amd as hg
    say("base_gemm_w4", M, N, K, group)
    g = np.random.default_rng(M + N + K + group)
    scale, zero, w, packed, sz = weight(g, N, K, group)
    x = bf16(g, M, K)
    y = torch.full((M + 1, N), 7.0, dtype=torch.bfloat16, device="cuda")
    hg.base_gemm_w4(dev(x), packed, sz, y, M, N, K, group)
    y2 = torch.empty_like(y)
    hg.base_gemm_w4(dev(x), packed, sz, y2, M, N, K, group)
    torch.cuda.synchronize()
    assert np.array_equal(bits(y)[:M], bits(y2)[:M]), "two runs must agree bit for bit"
    assert np.all(to_np(y)[M] == 7.0)
    want = x @ w.T
    err = np.abs(to_np(y)[:M] - want)
    tol = product_tolerance(want, x, scale, zero, K)
    print(f"[parity] worst err / tolerance {np.max(err / tol):.3f}", flush=True)
    assert np.all(err <= tol)


def test_base_gemm_w4_one_hot_rows_read_the_weight():
    """x of unit vectors returns W0's columns to half a step of bf16: every code and group in its place."""
    import heterogeneous_adapter_gemm_amd as hg
    for group in (32, 64, 128):
        say("one-hot rows, group", group)
        g = np.random.default_rng(group)
        N, K = 48, 256
        _, _, w, packed, sz = weight(g, N, K, group)
        y = torch.empty((K, N), dtype=torch.bfloat16, device="cuda")
        hg.base_gemm_w4(dev(np.eye(K)), packed, sz, y, K, N, K, group)
        torch.cuda.synchronize()
        # sums of 16 + code and 16 + zero are exact; their difference times scale is rounded in fp32
        assert np.all(np.abs(to_np(y) - w.T) <= 2.0 ** -8 * np.abs(w.T) + 2.0 ** -20 * np.abs(w).max())


def test_base_gemm_w4_non_finite_rows_stay_alone():
    import heterogeneous_adapter_gemm_amd as hg
    say("rows with infinities and NaN")
    g = np.random.default_rng(3)
    M, N, K = 40, 64, 256
    _, _, w, packed, sz = weight(g, N, K, 64)
    x = bf16(g, M, K)
    y0 = torch.empty((M, N), dtype=torch.bfloat16, device="cuda")
    hg.base_gemm_w4(dev(x), packed, sz, y0, M, N, K, 64)
    x[7, 3] = np.nan
    x[21, 200] = np.inf
    y1 = torch.empty_like(y0)
    hg.base_gemm_w4(dev(x), packed, sz, y1, M, N, K, 64)
    torch.cuda.synchronize()
    rest = [m for m in range(M) if m not in (7, 21)]
    assert np.array_equal(bits(y0)[rest], bits(y1)[rest])
    assert not np.isfinite(to_np(y1)[[7, 21]]).any()


def _adapters(g, pool, d_in, d_out, ranks):
    ad = {}
    for i, r in enumerate(ranks):
        A = bf16_bits((g.standard_normal((r, d_in)) * d_in ** -0.5).astype(np.float32))
        B = bf16_bits((g.standard_normal((r, d_out)) * 0.05).astype(np.float32))
        pool.page_in(i, r, 3.0 + r, A.reshape(-1), B.reshape(-1))
        f = lambda b: (b.astype(np.uint32) << 16).view(np.float32).astype(np.float64)  # noqa: E731
        ad[i] = ((3.0 + r) / r, f(A), f(B))
    return ad


def delta(x, row_ad, ad):
    out = 0.0
    for a, (gamma, A, B) in ad.items():
        out = out + (np.asarray(row_ad) == a)[:, None] * (gamma * (x @ A.T) @ B)
    return out


@pytest.mark.parametrize("lens,n_dec,group", [([], 1, 128), ([], 40, 64), ([], 64, 128), ([], 200, 32), ([130, 1, 0, 77], 45, 64),
                                              ([20], 0, 32)])
def test_lora_linear_w4(lens, n_dec, group):
    """Decode rows, prefill segments and both, over adapters of mixed ranks and rows without one
    (bit for bit base_gemm_w4's)."""
    import heterogeneous_adapter_gemm_amd as hg
    d_in, d_out, P = 1024, 1040, 512
    ranks = [16, 64, 8]
    say("lora_linear_w4", lens, n_dec, group)
    g = np.random.default_rng(len(lens) + n_dec)
    pool = hg.DevicePool(hg.LORA_BF16, P, 2048, g.permutation(2048), 1, [d_in], [d_out], 8, 64, 512, 8)
    ad = _adapters(g, pool, d_in, d_out, ranks)
    sad = [0, -1, 2, 1][:len(lens)]
    dec = g.choice([-1, 0, 1, 2], n_dec).astype(np.int32)
    row_ad = np.concatenate([np.full(n, a, np.int32) for n, a in zip(lens, sad)] + [dec])
    T = row_ad.size
    x = bf16(g, T, d_in)
    scale, zero, w, packed, sz = weight(g, d_out, d_in, group)
    slot = lambda a: -1 if a < 0 else pool.slot_of(int(a))  # noqa: E731
    plan = pool.plan(np.concatenate([[0], np.cumsum(lens)]) if lens else None, [slot(a) for a in sad] if lens else None,
                     [slot(a) for a in dec] if n_dec else None)
    for again in range(2):                       # the plan's first call uploads its index, the second finds it
        y = torch.zeros((T, d_out), dtype=torch.bfloat16, device="cuda")
        pool.linear_w4(plan, 0, 0, dev(x), packed, sz, group, y)
        torch.cuda.synchronize()
        d = delta(x, row_ad, ad)
        want = x @ w.T + d
        # the delta's bar is lora_linear's: 2e-2 of its RMS; the product's is derived above
        tol = product_tolerance(want, x, scale, zero, d_in) + 2e-2 * np.sqrt(np.mean(np.square(d)) + 1e-30)
        assert np.all(np.abs(to_np(y) - want) <= tol)
        base = torch.empty_like(y)
        hg.base_gemm_w4(dev(x), packed, sz, base, T, d_out, d_in, group)
        torch.cuda.synchronize()
        null = row_ad < 0
        assert np.array_equal(bits(y)[null], bits(base)[null])
    hg.lora_plan_destroy(plan)


def test_a_served_attention_block():
    """q, k, v projections over a 4-bit base with adapters, the append of the turned keys and the values
    to the pool that also holds the adapters, attention over them, the output projection: a prompt
    step and two decode steps, each stage in 64 bits from the bf16 values of the one before."""
    import heterogeneous_adapter_gemm_amd as hg
    D, H, n_kv, d = 128, 8, 2, 1024
    lens, page = [40, 3], 2048
    g = np.random.default_rng(21)
    d_outs = [H * D, n_kv * D, n_kv * D, d]
    pool = hg.DevicePool(hg.LORA_BF16, page, 1024, g.permutation(1024), 1, [d] * 4, d_outs, 4, 64, 64, 4)
    ads = [dict() for _ in range(4)]
    for i, r in enumerate([8, 16]):
        A = [(g.standard_normal((r, d)) * d ** -0.5).astype(np.float32) for _ in range(4)]
        B = [(g.standard_normal((r, n)) * 0.05).astype(np.float32) for n in d_outs]
        pool.page_in(i, r, 2.0 * r, np.concatenate([bf16_bits(t).reshape(-1) for t in A]),
                     np.concatenate([bf16_bits(t).reshape(-1) for t in B]))
        for j in range(4):
            ads[j][i] = (2.0, KV.bf16_round(A[j]), KV.bf16_round(B[j]))
    ws4 = [weight(g, n, d, 128, std=0.1) for n in d_outs]
    most = [n + 2 for n in lens]
    b0, table = make_batch(pool, H, n_kv, D, lens, most)
    cs = cos_sin(16 * table.shape[1], D)
    csd = torch.from_numpy(cs).cuda()
    kk, vv = [np.zeros((0, n_kv, D))] * 2, [np.zeros((0, n_kv, D))] * 2
    now = [0, 0]
    for step in range(3):
        rows = lens if step == 0 else [1, 1]
        now = [a + n for a, n in zip(now, rows)]
        T = sum(rows)
        say("served block, step", step, "rows", rows, "tokens", now)
        batch = hg.KvBatch(H, n_kv, D, torch.from_numpy(np.concatenate([[0], np.cumsum(rows)]).astype(np.int32)).cuda(),
                           torch.tensor(now, dtype=torch.int32).cuda(), b0.page_table, T, max_rows=max(rows))
        slots = [pool.slot_of(1), pool.slot_of(0)]
        plan = pool.plan([0, rows[0], T], slots) if step == 0 else pool.plan(token_slot=slots)
        row_ad = np.concatenate([np.full(rows[0], 1), np.full(rows[1], 0)])
        x = bf16(g, T, d)
        xd = dev(x)
        outs = [torch.empty((T, n), dtype=torch.bfloat16, device="cuda") for n in d_outs]

        def project(j, inp, inp_np):
            pool.linear_w4(plan, 0, j, inp, ws4[j][3], ws4[j][4], 128, outs[j])
            torch.cuda.synchronize()
            dl = delta(inp_np, row_ad, ads[j])
            want = inp_np @ ws4[j][2].T + dl
            tol = product_tolerance(want, inp_np, ws4[j][0], ws4[j][1], d) + 2e-2 * np.sqrt(np.mean(dl ** 2))
            assert np.all(np.abs(to_np(outs[j]) - want) <= tol), (step, j)

        for j in range(3):
            project(j, xd, x)
        q, k, v = (to_np(o).reshape(T, -1, D) for o in outs[:3])
        pool.kv_append(batch, outs[1], outs[2], q=outs[0], q_out=outs[0], cos_sin=csd)
        att = torch.empty((T, H, D), dtype=torch.bfloat16, device="cuda")
        pool.kv_attention(batch, outs[0], att, workspace=pool.kv_workspace(batch))
        torch.cuda.synchronize()
        pos = np.concatenate([np.arange(n - r, n) for n, r in zip(now, rows)])
        ck, cv = KV.quantise(KV.bf16_round(KV.rotate(k, pos, cs, False))), KV.quantise(v)
        kn, vn = KV.value(*ck), KV.value(*cv)
        at = np.concatenate([[0], np.cumsum(rows)])
        for s in range(2):
            kk[s] = np.concatenate([kk[s], kn[at[s]:at[s + 1]]])
            vv[s] = np.concatenate([vv[s], vn[at[s]:at[s + 1]]])
        turned = to_np(outs[0]).reshape(T, H, D)
        want = oracle_out(turned, kk, vv, rows, n_kv, D ** -0.5)
        allk, allv = KV.quantise(np.concatenate(kk)), KV.quantise(np.concatenate(vv))
        assert np.all(np.abs(to_np(att) - want) <= tolerance(want, turned, kk, vv, allk, allv, D ** -0.5, D, 99)), step
        project(3, att, to_np(att).reshape(T, H * D))
        hg.lora_plan_destroy(plan)
