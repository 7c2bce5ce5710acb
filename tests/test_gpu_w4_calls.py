"""The 4-bit base with adapters on the GPU: every kind of decode tile with the adapters' units beside it,
captured calls and other streams, in 64 bits."""
import numpy as np
import pytest

from tests.test_gpu_kv import bf16, dev
from tests.test_gpu_w4 import _adapters, _gpu, bits, delta, product_tolerance, say, to_np, weight

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


def setup(g, d_in, d_out, ranks, n_dec, group, P=512):
    import heterogeneous_adapter_gemm_amd as hg
    need = sum(r * (-(-d_in // P) + -(-d_out // P)) for r in ranks)
    pool = hg.DevicePool(hg.LORA_BF16, P, need + 8, g.permutation(need + 8), 1, [d_in], [d_out], len(ranks), 64, 512,
                         len(ranks))
    ad = _adapters(g, pool, d_in, d_out, ranks)
    row_ad = g.integers(-1, len(ranks), n_dec).astype(np.int32)
    row_ad[:min(n_dec, len(ranks))] = np.arange(min(n_dec, len(ranks)))
    plan = pool.plan(None, None, [-1 if a < 0 else pool.slot_of(int(a)) for a in row_ad])
    return pool, ad, row_ad, plan, weight(g, d_out, d_in, group)


def bound(want, x, scale, zero, d_in, d):
    """The product's own, and the delta's: 2e-2 of its RMS, as lora_linear's."""
    return product_tolerance(want, x, scale, zero, d_in) + 2e-2 * np.sqrt(np.mean(np.square(d)) + 1e-30)


@pytest.mark.parametrize("n_dec,group,d_out,n_ad", [(1, 32, 24, 1), (5, 64, 272, 3), (16, 32, 528, 16), (17, 128, 264, 2), (31, 64, 1000, 8),
                                                    (50, 64, 10248, 4), (64, 32, 10240, 64), (64, 128, 136, 64)])
def test_decode_rows_with_adapters(n_dec, group, d_out, n_ad):
    say("decode rows", n_dec, group, d_out, n_ad)
    d_in = 512
    g = np.random.default_rng(n_dec + d_out)
    pool, ad, row_ad, plan, (scale, zero, w, packed, sz) = setup(g, d_in, d_out, [64 if i % 2 else 8 for i in range(n_ad)], n_dec, group)
    x = bf16(g, n_dec, d_in)
    ys = []
    for _ in range(2):
        y = torch.full((n_dec + 1, d_out), 7.0, dtype=torch.bfloat16, device="cuda")
        pool.linear_w4(plan, 0, 0, dev(x), packed, sz, group, y)
        torch.cuda.synchronize()
        ys.append(y)
    assert np.array_equal(bits(ys[0]), bits(ys[1])) and np.all(to_np(ys[0])[n_dec] == 7.0)
    d = delta(x, row_ad, ad)
    want = x @ w.T + d
    assert np.all(np.abs(to_np(ys[0])[:n_dec] - want) <= bound(want, x, scale, zero, d_in, d))


@pytest.mark.parametrize("n_dec", [3, 64, 200])
def test_captured_calls(n_dec):
    """A captured call replayed over new rows, the program's own calls between the replays, and one from
    another stream."""
    say("captured", n_dec)
    import heterogeneous_adapter_gemm_amd as hg
    d_in, d_out, group = 640, 1040, 128
    g = np.random.default_rng(n_dec)
    pool, ad, row_ad, plan, (scale, zero, w, packed, sz) = setup(g, d_in, d_out, [16, 64, 8], n_dec, group)
    xd = dev(bf16(g, n_dec, d_in))
    y, own, base = (torch.zeros((n_dec, d_out), dtype=torch.bfloat16, device="cuda") for _ in range(3))
    pool.linear_w4(plan, 0, 0, xd, packed, sz, group, y)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        pool.linear_w4(plan, 0, 0, xd, packed, sz, group, y)
        hg.base_gemm_w4(xd, packed, sz, base, n_dec, d_out, d_in, group)
    other = torch.cuda.Stream()
    for _ in range(4):
        x = bf16(g, n_dec, d_in)
        xd.copy_(dev(x))
        graph.replay()
        torch.cuda.synchronize()
        got, got_base = y.clone(), base.clone()
        d = delta(x, row_ad, ad)
        want = x @ w.T + d
        assert np.all(np.abs(to_np(got) - want) <= bound(want, x, scale, zero, d_in, d))
        y.fill_(3.0)
        pool.linear_w4(plan, 0, 0, xd, packed, sz, group, own)
        torch.cuda.synchronize()
        assert np.array_equal(bits(own), bits(got))
        with torch.cuda.stream(other):
            hg.base_gemm_w4(xd, packed, sz, own, n_dec, d_out, d_in, group)
        torch.cuda.synchronize()
        assert np.array_equal(bits(own), bits(got_base))
        assert np.array_equal(bits(own)[row_ad < 0], bits(got)[row_ad < 0])


@pytest.mark.parametrize("M,N,K,group", [(1100, 5636, 256, 64), (1100, 5636, 128, 128), (1290, 6660, 256, 32), (1300, 6700, 384, 128),
                                         (2050, 7684, 128, 64), (1030, 4200, 256, 64), (1030, 4200, 128, 32), (1090, 4100, 384, 128)])
def test_rounds_of_long_tiles(M, N, K, group):
    """Tiles of 128 x 128 alone (405 of them), whole ones with a last round of halves (583, 1,037), halves
    alone (297)."""
    say("long tiles", M, N, K, group)
    import heterogeneous_adapter_gemm_amd as hg
    g = np.random.default_rng(M + K)
    scale, zero, w, packed, sz = weight(g, N, K, group)
    x = bf16(g, M, K)
    y = torch.full((M + 1, N), 7.0, dtype=torch.bfloat16, device="cuda")
    hg.base_gemm_w4(dev(x), packed, sz, y, M, N, K, group)
    y2 = torch.empty_like(y)
    hg.base_gemm_w4(dev(x), packed, sz, y2, M, N, K, group)
    torch.cuda.synchronize()
    assert np.array_equal(bits(y)[:M], bits(y2)[:M]) and np.all(to_np(y)[M] == 7.0)
    want = x @ w.T
    assert np.all(np.abs(to_np(y)[:M] - want) <= product_tolerance(want, x, scale, zero, K))


@pytest.mark.parametrize("n_dec,d_out,n_ad", [(40, 1024, 3), (64, 4096, 16), (64, 7000, 40), (64, 8192, 3), (33, 8064, 8), (64, 10240, 64)])
def test_rows_without_an_adapter_are_the_base_products(n_dec, d_out, n_ad):
    """Bit for bit, whatever tiles either call takes."""
    say("rows without an adapter", n_dec, d_out, n_ad)
    import heterogeneous_adapter_gemm_amd as hg
    d_in, group = 1280, 128
    g = np.random.default_rng(n_dec + d_out)
    pool, ad, row_ad, plan, (scale, zero, w, packed, sz) = setup(g, d_in, d_out, [32] * n_ad, n_dec, group)
    none = [-1 if i % 3 == 0 else pool.slot_of(i % n_ad) for i in range(n_dec)]
    plan = pool.plan(None, None, none)
    xd = dev(bf16(g, n_dec, d_in))
    y, base = (torch.zeros((n_dec, d_out), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    pool.linear_w4(plan, 0, 0, xd, packed, sz, group, y)
    hg.base_gemm_w4(xd, packed, sz, base, n_dec, d_out, d_in, group)
    torch.cuda.synchronize()
    assert np.array_equal(bits(y)[::3], bits(base)[::3])
    assert not np.array_equal(bits(y)[1::3], bits(base)[1::3])
