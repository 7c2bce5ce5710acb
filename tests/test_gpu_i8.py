"""The 8-bit integer base on the GPU: the product, the gated product, and the product with adapters, in 64 bits."""
import numpy as np
import pytest

from tests import i8_helpers as E
from tests.gpu_helpers import bits, to_np

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


def gpu(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def matrix(g, n, k):
    """Codes over all of int8 and scales of very different rows."""
    c = g.integers(-128, 128, (n, k), dtype=np.int8)
    return c, np.exp(g.uniform(-8, -2, n)).astype(np.float32)


def exact_product(x, w):
    """On the GPU in 64 bits (sums of whole numbers below 2^53: exact)."""
    p = gpu(x[0]).double() @ gpu(w[0]).double().t().contiguous()
    return (p * gpu(x[1]).double()[:, None] * gpu(w[1]).double()).cpu().numpy()


# one row to several row blocks and column blocks of every kind of tile, K of part of a slice, part of a wave's step and
# several rings; then each of the kinds that few sizes take, and last rounds of 2, 4, 8 and 16 pieces
SHAPES = [(1, 4, 16), (1, 4096, 4096), (3, 100, 48), (16, 4160, 1040), (17, 36, 128), (16, 9000, 272), (5, 12800, 528), (32, 520, 2064),
          (30, 9000, 400), (31, 12300, 1024), (32, 16400, 640), (33, 260, 144), (64, 4096, 4096), (64, 8200, 384), (64, 10244, 2048),
          (48, 16388, 560), (64, 11008, 4112), (65, 1000, 768), (128, 4100, 656), (200, 4096, 1552), (256, 4096, 11008), (255, 7004, 352),
          (257, 64, 16), (300, 272, 656), (700, 4100, 304), (1000, 4096, 512), (2049, 8100, 272), (2961, 4096, 4096), (1100, 13000, 208),
          (1500, 11008, 336), (4100, 4360, 160), (4352, 4128, 320), (2816, 6300, 592),
          (1, 17036, 272), (33, 12316, 272), (19, 8472, 272), (8429, 72, 272), (151, 16500, 272), (206, 18732, 272),
          (342, 48388, 608), (386, 43812, 944), (391, 70364, 288), (1167, 14356, 800), (754, 21900, 560),
          (67, 6436, 272), (860, 340, 1040), (2961, 64, 528), (1000, 260, 9376), (3000, 36, 400)]


@pytest.mark.parametrize("M,N,K", SHAPES)
def test_product(M, N, K):
    import heterogeneous_adapter_gemm_amd as hg
    say("product", M, N, K)
    g = np.random.default_rng(M + 3 * N + 7 * K)
    x, w = matrix(g, M, K), matrix(g, N, K)
    want = exact_product(x, w)
    ys = []
    for _ in range(2):
        y = torch.full((M + 1, N), 7.0, dtype=torch.bfloat16, device="cuda")
        hg.base_gemm_i8(gpu(x[0]), gpu(x[1]), gpu(w[0]), gpu(w[1]), y, M, N, K)
        torch.cuda.synchronize()
        ys.append(y)
    assert torch.equal(ys[0].view(torch.int16), ys[1].view(torch.int16))
    got = to_np(ys[0])
    assert np.all(got[M] == 7.0)
    assert np.all(np.abs(got[:M] - want) <= np.abs(want) * E.PRODUCT)


GATED = [(1, 4, 16), (1, 11008, 4096), (16, 100, 48), (20, 4100, 400), (32, 2060, 2064), (64, 11008, 1040), (64, 260, 144), (64, 2052, 4096),
         (130, 1000, 768), (256, 4100, 656), (257, 132, 16), (700, 4100, 304), (1000, 2048, 512), (2049, 4060, 272), (2961, 2048, 2048),
         (1100, 6500, 208), (1500, 5504, 336), (2816, 3156, 592), (4352, 2064, 320),
         (1, 4148, 288), (17, 4216, 272), (33, 4300, 304), (34, 6264, 320), (8903, 36, 272), (163, 8552, 272),
         (1026, 8052, 608), (388, 21844, 960), (385, 35172, 288), (471, 17564, 800), (758, 10884, 560),
         (67, 6436, 272), (300, 1020, 304), (2961, 64, 528), (600, 516, 8208)]


@pytest.mark.parametrize("M,N,K", GATED)
def test_gated(M, N, K):
    import heterogeneous_adapter_gemm_amd as hg
    act = ["silu", "gelu", "gelu_tanh"][(M + N) % 3]
    say("gated", M, N, K, act)
    g = np.random.default_rng(M + 3 * N + 7 * K)
    x, wg, wu = matrix(g, M, K), matrix(g, N, K), matrix(g, N, K)
    # (gates of a size where the activations bend)
    wg[1][:] = (g.uniform(0.5, 2.0, N) / (np.exp(-5) * 73 * 73 * np.sqrt(K))).astype(np.float32)
    ge, u = exact_product(x, wg), exact_product(x, wu)
    y = torch.full((M + 1, N), 7.0, dtype=torch.bfloat16, device="cuda")
    hg.base_gated_i8(gpu(x[0]), gpu(x[1]), gpu(wg[0]), gpu(wg[1]), gpu(wu[0]), gpu(wu[1]), y, M, N, K, act=act)
    torch.cuda.synchronize()
    got = to_np(y)
    assert np.all(got[M] == 7.0)
    # the gate is 4 roundings off before the activation, which moves that by a factor of at most 2 + z^2 where the
    # result is not 0: 16 roundings for gates of up to about 14, 128 more than cover larger ones
    bound = E.act_bound(act, ge, u) + np.abs(E.activated(ge, act) * u) * 4 * 256 * E.ULP
    assert np.all(np.abs(got[:M] - E.activated(ge, act) * u) <= bound)


def test_every_tile_gives_the_same_rows():
    """The sums are exact: a row's outputs do not depend on the batch around it."""
    import heterogeneous_adapter_gemm_amd as hg
    N, K = 1028, 1040
    g = np.random.default_rng(2)
    x, w = matrix(g, 900, K), matrix(g, N, K)
    xc, xs, wc, ws = gpu(x[0]), gpu(x[1]), gpu(w[0]), gpu(w[1])
    full = torch.zeros((900, N), dtype=torch.bfloat16, device="cuda")
    hg.base_gemm_i8(xc, xs, wc, ws, full, 900, N, K)
    for M in (1, 16, 17, 32, 40, 64, 100, 256, 257, 500):
        y = torch.zeros((M, N), dtype=torch.bfloat16, device="cuda")
        hg.base_gemm_i8(xc, xs, wc, ws, y, M, N, K)
        torch.cuda.synchronize()
        assert torch.equal(y, full[:M]), M


@pytest.mark.parametrize("M", [2, 40, 300])
def test_largest_sums_and_scales_that_are_no_numbers(M):
    """The most K: sums next to int32's ends."""
    import heterogeneous_adapter_gemm_amd as hg
    N, K = 68, 131056
    assert K * 128 * 128 < 2 ** 31 <= (K + 16) * 128 * 128
    xc = torch.full((M, K), -128, dtype=torch.int8, device="cuda")
    wc = torch.full((N, K), 127, dtype=torch.int8, device="cuda")
    wc[1::2] = -128
    xs, ws = torch.full((M,), 2.0 ** -20, device="cuda"), torch.full((N,), 0.5, device="cuda")
    xs[0], ws[3] = float("nan"), float("inf")
    y = torch.zeros((M, N), dtype=torch.bfloat16, device="cuda")
    hg.base_gemm_i8(xc, xs, wc, ws, y, M, N, K)
    torch.cuda.synchronize()
    got = to_np(y)
    assert np.all(np.isnan(got[0])) and np.all(got[1:, 3] == np.inf)
    want = np.where(np.arange(N) % 2, 128.0, -127.0) * 128 * K * 2.0 ** -21
    keep = np.arange(N) != 3
    assert np.all(np.abs(got[1:][:, keep] - want[keep]) <= np.abs(want[keep]) * E.PRODUCT)


# -- with adapters ----------------------------------------------------------------------------------------------


def setup(g, d_in, d_out, ranks, P=512, max_tokens=4096):
    import heterogeneous_adapter_gemm_amd as hg
    need = sum(r * (-(-d_in // P) + -(-d_out // P)) for r in ranks)
    pool = hg.DevicePool(hg.LORA_BF16, P, need + 8, g.permutation(need + 8), 1, [d_in], [d_out], len(ranks), 64, max_tokens, 16)
    ad = []
    for i, r in enumerate(ranks):
        A, B = E.bf16(g.standard_normal((r, d_in)) * d_in ** -0.5), E.bf16(g.standard_normal((r, d_out)) * 0.05)
        pack = lambda t: (t.astype(np.float32).view(np.uint32) >> 16).astype(np.uint16).reshape(-1)  # noqa: E731
        pool.page_in(i, r, 2.0 * r + i, pack(A), pack(B))
        ad.append(((2.0 * r + i) / r, A, B))
    torch.cuda.synchronize()
    return pool, ad


def linear_want(x, xq, w, who, ad):
    """-> outputs, and a bound of their roundings."""
    y = exact_product(xq, w)
    bound = np.abs(y) * 4 * E.ULP
    K = x.shape[1]
    for a, (gamma, A, B) in enumerate(ad):
        m = np.nonzero(who == a)[0]
        if m.size:
            y[m] += gamma * (x[m] @ A.T) @ B
            # v: K products summed in fp32; gamma v enters the expand in fp32, or as two bf16 halves (2^-16), and the
            # rank's products are summed in fp32 beside the base
            size = abs(gamma) * (np.abs(x[m]) @ np.abs(A).T) @ np.abs(B)
            bound[m] += size * ((K + 80) * E.ULP + 2.0 ** -15)
    return y, bound + np.abs(y) * E.HALF + E.TINY


def rows_of(g, n, d):
    x = E.bf16(g.standard_normal((n, d)))
    s = (np.abs(x).max(1) / 127).astype(np.float32)
    return x, (E.codes(x).astype(np.int8), s)


def dev(v):
    return torch.from_numpy(np.asarray(v, np.float32)).to(torch.bfloat16).cuda()


@pytest.mark.parametrize("n,d_in,d_out,n_ad", [(1, 528, 24, 1), (5, 512, 272, 3), (16, 1040, 4360, 16), (17, 640, 264, 2), (32, 512, 8200, 6),
                                               (64, 4096, 4096, 16), (64, 512, 10248, 4), (50, 2064, 16392, 9), (65, 528, 1000, 8),
                                               (200, 1040, 1032, 5), (256, 512, 4096, 64), (300, 512, 520, 7), (1000, 784, 1032, 12),
                                               (90, 272, 8208, 7), (192, 528, 5512, 40), (130, 4096, 520, 130)])
def test_decode_rows_with_adapters(n, d_in, d_out, n_ad):
    import heterogeneous_adapter_gemm_amd as hg
    say("decode rows", n, d_in, d_out, n_ad)
    g = np.random.default_rng(n + d_out)
    pool, ad = setup(g, d_in, d_out, [64 if i % 3 == 1 else 8 + i % 5 for i in range(n_ad)])
    who = g.integers(-1, n_ad, n)
    plan = pool.plan(token_slot=[-1 if a < 0 else pool.slot_of(int(a)) for a in who])
    x, xq = rows_of(g, n, d_in)
    w = matrix(g, d_out, d_in)
    w[1][:] *= 0.02
    ys = []
    for _ in range(2):
        y = torch.full((n + 1, d_out), 7.0, dtype=torch.bfloat16, device="cuda")
        pool.linear_i8(plan, 0, 0, dev(x), gpu(xq[0]), gpu(xq[1]), gpu(w[0]), gpu(w[1]), y)
        torch.cuda.synchronize()
        ys.append(y)
    base = torch.zeros((n, d_out), dtype=torch.bfloat16, device="cuda")
    hg.base_gemm_i8(gpu(xq[0]), gpu(xq[1]), gpu(w[0]), gpu(w[1]), base, n, d_out, d_in)
    torch.cuda.synchronize()
    assert np.array_equal(bits(ys[0]), bits(ys[1]))
    want, bound = linear_want(x, xq, w, who, ad)
    got = to_np(ys[0])
    assert np.all(got[n] == 7.0) and np.all(np.abs(got[:n] - want) <= bound)
    assert np.array_equal(bits(ys[0])[:n][who < 0], bits(base)[who < 0])
    hg.lora_plan_destroy(plan)


# segments with and without an adapter, empty ones, of one row, ending inside a tile; with and without decode rows
@pytest.mark.parametrize("lens,n_dec,d_in,d_out", [([1], 0, 512, 264), ([30, 0, 7], 9, 528, 1032), ([100, 77, 1], 40, 1040, 520),
                                                   ([130, 1, 0, 77], 145, 1024, 1040), ([300, 212], 0, 512, 4104), ([64, 700, 33, 400], 192, 784, 2056),
                                                   ([1024, 900, 61], 64, 512, 4096), ([513, 1, 1, 640], 7, 4096, 1048)])
def test_prompts_with_adapters(lens, n_dec, d_in, d_out):
    prompts(lens, n_dec, d_in, d_out)


# kinds of tiles that few sizes take, and last rounds of pieces, with the expand in the epilogue
@pytest.mark.parametrize("lens,n_dec,d_in,d_out", [([100, 77, 40, 60], 12, 272, 11336), ([262], 0, 304, 16824), ([404], 0, 304, 23224),
                                                   ([70, 300, 130, 80], 8, 272, 8744), ([1000, 900, 33, 1200], 30, 608, 5224), ([130, 200, 33], 23, 960, 43680),
                                                   ([385], 0, 304, 70288), ([190, 130, 64], 68, 800, 36584), ([2000, 1500, 700, 600], 30, 560, 3416)])
def test_prompts_in_every_kind_of_tile(lens, n_dec, d_in, d_out):
    prompts(lens, n_dec, d_in, d_out)


def prompts(lens, n_dec, d_in, d_out):
    import heterogeneous_adapter_gemm_amd as hg
    say("prompts", lens, n_dec, d_in, d_out)
    g = np.random.default_rng(sum(lens) + d_out)
    ranks = [16, 64, 33, 8]
    pool, ad = setup(g, d_in, d_out, ranks, max_tokens=8192)
    sad = np.array([[0, -1, 1, 2][i % 4] for i in range(len(lens))])
    dec = g.integers(-1, len(ranks), n_dec)
    who = np.concatenate([np.repeat(sad, lens), dec])
    slot = lambda v: [-1 if a < 0 else pool.slot_of(int(a)) for a in v]  # noqa: E731
    plan = pool.plan(np.concatenate([[0], np.cumsum(lens)]), slot(sad), slot(dec))
    n = who.size
    x, xq = rows_of(g, n, d_in)
    w = matrix(g, d_out, d_in)
    w[1][:] *= 0.02
    y = torch.full((n + 1, d_out), 7.0, dtype=torch.bfloat16, device="cuda")
    pool.linear_i8(plan, 0, 0, dev(x), gpu(xq[0]), gpu(xq[1]), gpu(w[0]), gpu(w[1]), y)
    base = torch.zeros((n, d_out), dtype=torch.bfloat16, device="cuda")
    hg.base_gemm_i8(gpu(xq[0]), gpu(xq[1]), gpu(w[0]), gpu(w[1]), base, n, d_out, d_in)
    torch.cuda.synchronize()
    want, bound = linear_want(x, xq, w, who, ad)
    got = to_np(y)
    assert np.all(got[n] == 7.0) and np.all(np.abs(got[:n] - want) <= bound)
    assert np.array_equal(bits(y)[:n][who < 0], bits(base)[who < 0])
    hg.lora_plan_destroy(plan)


@pytest.mark.parametrize("n", [3, 64, 200, 600])
def test_captured_calls(n):
    """A captured layer replayed over new rows, the program's own calls between the replays, and another stream."""
    import heterogeneous_adapter_gemm_amd as hg
    say("captured", n)
    d_in, d_out = 640, 1040
    g = np.random.default_rng(n)
    pool, ad = setup(g, d_in, d_out, [16, 64, 8])
    who = g.integers(-1, 3, n)
    plan = pool.plan(token_slot=[-1 if a < 0 else pool.slot_of(int(a)) for a in who])
    w, u = matrix(g, d_out, d_in), matrix(g, d_out, d_in)
    w[1][:] *= 0.02
    wd, ud = [gpu(t) for t in w], [gpu(t) for t in u]
    xd, code, scale = dev(rows_of(g, n, d_in)[0]), torch.zeros((n, d_in), dtype=torch.int8, device="cuda"), torch.zeros(n, device="cuda")
    ys = [torch.zeros((n, d_out), dtype=torch.bfloat16, device="cuda") for _ in range(3)]

    def step():
        hg.rows_act_i8(xd, code=code, scale=scale)
        pool.linear_i8(plan, 0, 0, xd, code, scale, *wd, ys[0])
        hg.base_gemm_i8(code, scale, *wd, ys[1], n, d_out, d_in)
        hg.base_gated_i8(code, scale, *wd, *ud, ys[2], n, d_out, d_in)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    other = torch.cuda.Stream()
    for _ in range(4):
        x, xq = rows_of(g, n, d_in)
        xd.copy_(dev(x))
        graph.replay()
        torch.cuda.synchronize()
        first = [t.clone() for t in ys]
        want, bound = linear_want(x, xq, w, who, ad)
        assert np.array_equal(code.cpu().numpy(), xq[0]) and np.all(np.abs(to_np(first[0]) - want) <= bound)
        for t in ys:
            t.fill_(3.0)
        other.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(other):
            step()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(first, ys))
        assert np.array_equal(bits(ys[1])[who < 0], bits(ys[0])[who < 0])
        pool.linear_i8(plan, 0, 0, xd, code, scale, *wd, ys[0])      # (the plan's calls go on on this stream)
        torch.cuda.synchronize()
    hg.lora_plan_destroy(plan)


@pytest.mark.parametrize("n", [1, 48, 700])
def test_a_block_as_it_is_served(n):
    """Norm, gate and up with and without adapters, the gated rows, down with adapters, the next norm: each step
    against 64-bit arithmetic on the step's own inputs."""
    import heterogeneous_adapter_gemm_amd as hg
    say("block", n)
    d, f = 512, 1408
    g = np.random.default_rng(n)
    P, ranks = 512, [16, 8, 33]
    need = sum(r * 2 * (-(-d // P) + -(-f // P)) for r in ranks) * 2
    pool = hg.DevicePool(hg.LORA_BF16, P, need + 8, g.permutation(need + 8), 1, [d, d, f], [f, f, d], len(ranks), 64, 1024, 4)
    ad = [[], [], []]
    pack = lambda t: (t.astype(np.float32).view(np.uint32) >> 16).astype(np.uint16).reshape(-1)  # noqa: E731
    for i, r in enumerate(ranks):
        A = [E.bf16(g.standard_normal((r, k)) * k ** -0.5) for k in (d, d, f)]
        B = [E.bf16(g.standard_normal((r, m)) * 0.05) for m in (f, f, d)]
        pool.page_in(i, r, 2.0 * r, np.concatenate([pack(t) for t in A]), np.concatenate([pack(t) for t in B]))
        for p in range(3):
            ad[p].append((2.0, A[p], B[p]))
    torch.cuda.synchronize()
    who = g.integers(-1, 3, n)
    who[0] = 0
    plan = pool.plan(token_slot=[-1 if a < 0 else pool.slot_of(int(a)) for a in who])
    ws = []
    for m, k in ((f, d), (f, d), (d, f)):
        c = np.clip(np.rint(g.standard_normal((m, k)) * 40), -127, 127).astype(np.int8)
        ws.append((c, (g.uniform(0.5, 1.5, m) / (40 * np.sqrt(k))).astype(np.float32)))
    wd = [[gpu(t) for t in w] for w in ws]
    x, res, nw = E.bf16(g.standard_normal((n, d))), E.bf16(2 * g.standard_normal((n, d))), E.bf16(1 + 0.1 * g.standard_normal(d))
    z = lambda *s, dtype=torch.bfloat16: torch.zeros(s, dtype=dtype, device="cuda")  # noqa: E731
    s, y, c8, s8 = z(n, d), z(n, d), z(n, d, dtype=torch.int8), z(n, dtype=torch.float32)
    gate_up, a, a8, as8, down = z(2, n, f), z(n, f), z(n, f, dtype=torch.int8), z(n, dtype=torch.float32), z(n, d)
    fused, s2, y2 = z(n, f), z(n, d), z(n, d)
    hg.rows_norm_i8(dev(x), dev(nw), 1e-5, residual=dev(res), sum_out=s, y=y, code=c8, scale=s8)
    for p in range(2):
        pool.linear_i8(plan, 0, p, y, c8, s8, *wd[p], gate_up[p])
    hg.rows_act_i8(gate_up[1], gate=gate_up[0], act="silu", y=a, code=a8, scale=as8)
    pool.linear_i8(plan, 0, 2, a, a8, as8, *wd[2], down)
    hg.rows_norm_i8(down, dev(nw), 1e-5, residual=s, sum_out=s2, y=y2)
    hg.base_gated_i8(c8, s8, *wd[0], *wd[1], fused, n, f, d)
    torch.cuda.synchronize()
    h, ny, nc, nsc = E.norm(x, res, nw, 1e-5)
    assert np.array_equal(to_np(s), h) and np.array_equal(c8.cpu().numpy(), nc)
    assert np.all(np.abs(to_np(y) - ny) <= np.abs(ny) * (E.HALF + 60 * E.ULP))
    yq = (c8.cpu().numpy(), s8.cpu().numpy())
    for p in range(2):
        want, bound = linear_want(to_np(y), yq, ws[p], who, ad[p])
        assert np.all(np.abs(to_np(gate_up[p]) - want) <= bound)
    gg, uu = to_np(gate_up[0]), to_np(gate_up[1])
    assert np.all(np.abs(to_np(a) - E.activated(gg, "silu") * uu) <= E.act_bound("silu", gg, uu))
    assert np.array_equal(a8.cpu().numpy(), E.codes(to_np(a)))
    want, bound = linear_want(to_np(a), (a8.cpu().numpy(), as8.cpu().numpy()), ws[2], who, ad[2])
    assert np.all(np.abs(to_np(down) - want) <= bound)
    h2, ny2, _, _ = E.norm(to_np(down), h, nw, 1e-5)
    assert np.array_equal(to_np(s2), h2) and np.all(np.abs(to_np(y2) - ny2) <= np.abs(ny2) * (E.HALF + 60 * E.ULP))
    # rows without an adapter: the fused block is the same block, rounded once instead of three times
    ge, u = exact_product(yq, ws[0]), exact_product(yq, ws[1])
    bound = E.act_bound("silu", ge, u) + np.abs(E.activated(ge, "silu") * u) * 1024 * E.ULP
    assert np.all(np.abs(to_np(fused) - E.activated(ge, "silu") * u) <= bound)
    hg.lora_plan_destroy(plan)
