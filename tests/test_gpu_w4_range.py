"""The 4-bit base at the ends of what it takes: rows of x with an infinity or NaN, in every kind of tile, and
values of up to 2^108 in size, in 64 bits."""
import numpy as np
import pytest

from tests.test_gpu_kv import bf16, dev
from tests.test_gpu_w4 import _adapters, _gpu, bits, product_tolerance, say, to_np, weight

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

SHAPES = [(1, 528, 1024, 128), (16, 260, 256, 32), (30, 516, 384, 64), (64, 4096, 256, 128), (64, 10244, 256, 64), (200, 1000, 384, 32),
          (1100, 4100, 256, 64), (1100, 5636, 128, 128)]


def product(x, packed, sz, N, K, group):
    import heterogeneous_adapter_gemm_amd as hg
    M = x.shape[0]
    y = torch.empty((M, N), dtype=torch.bfloat16, device="cuda")
    hg.base_gemm_w4(dev(x), packed, sz, y, M, N, K, group)
    torch.cuda.synchronize()
    return y


@pytest.mark.parametrize("M,N,K,group", SHAPES)
def test_rows_that_are_not_finite_are_nan_in_every_column(M, N, K, group):
    say("not finite", M, N, K, group)
    g = np.random.default_rng(M + N)
    _, _, w, packed, sz = weight(g, N, K, group)
    x = bf16(g, M, K)
    clean = product(x, packed, sz, N, K, group)
    hit = sorted({0, M // 2, M - 1})
    for i, m in enumerate(hit):
        x[m, int(g.integers(K))] = [np.inf, -np.inf, np.nan][i % 3]
    got = product(x, packed, sz, N, K, group)
    rest = [m for m in range(M) if m not in hit]
    assert np.isnan(to_np(got)[hit]).all()
    assert np.array_equal(bits(got)[rest], bits(clean)[rest])


@pytest.mark.parametrize("M,N,K,group", SHAPES)
def test_large_values_keep_their_room(M, N, K, group):
    """x of up to 2^108: group sums of 31 x stay inside fp32."""
    say("large x", M, N, K, group)
    g = np.random.default_rng(M + K)
    scale, zero, w, packed, sz = weight(g, N, K, group)
    x = bf16(g, M, K)
    assert np.abs(x).max() < 8
    x *= 2.0 ** 105
    want = x @ w.T
    assert np.all(np.abs(to_np(product(x, packed, sz, N, K, group)) - want) <= product_tolerance(want, x, scale, zero, K))


def test_rows_with_an_adapter_that_are_not_finite():
    import heterogeneous_adapter_gemm_amd as hg
    say("not finite, with adapters")
    d_in, d_out, P = 512, 520, 512
    g = np.random.default_rng(9)
    pool = hg.DevicePool(hg.LORA_BF16, P, 256, g.permutation(256), 1, [d_in], [d_out], 4, 64, 512, 4)
    _adapters(g, pool, d_in, d_out, [8, 16])
    _, _, w, packed, sz = weight(g, d_out, d_in, 64)
    for n in (5, 40, 100):
        row_ad = np.arange(n) % 3 - 1
        plan = pool.plan(None, None, [-1 if a < 0 else pool.slot_of(int(a)) for a in row_ad])
        x = bf16(g, n, d_in)
        ys = []
        for bad in (None, 0, 1):
            xx = x.copy()
            if bad is not None:
                xx[bad, 7] = np.inf
            y = torch.empty((n, d_out), dtype=torch.bfloat16, device="cuda")
            pool.linear_w4(plan, 0, 0, dev(xx), packed, sz, 64, y)
            torch.cuda.synchronize()
            ys.append(y)
            if bad is not None:
                rest = [m for m in range(n) if m != bad]
                assert np.isnan(to_np(y)[bad]).all() and np.array_equal(bits(y)[rest], bits(ys[0])[rest])
        hg.lora_plan_destroy(plan)
