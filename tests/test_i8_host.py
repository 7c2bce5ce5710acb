"""Refusals of the 8-bit integer operators, without a GPU: nothing below passes its checks on the host."""
import ctypes

import numpy as np
import pytest

import heterogeneous_adapter_gemm_amd as hg
from heterogeneous_adapter_gemm_amd import _lib
from tests import i8_helpers as E
from tests.test_kv_host import FAKE, host_pool
from tests.test_w4_devices import On

LIB = _lib.library()
EINVAL = hg.LORA_EINVAL


def norm(**kw):
    r = dict(n_rows=4, d=64, eps=1e-5, x=FAKE, weight=FAKE, residual=FAKE, sum_out=FAKE, y=FAKE, held=FAKE, code=FAKE, scale=FAKE,
             x_stride=64, residual_stride=64, sum_stride=64, y_stride=64, held_stride=64)
    r.update(kw)
    return LIB.rows_norm_i8(ctypes.byref(hg.lora_norm_rows(**r)), None), LIB.lora_last_error().decode()


def act(**kw):
    r = dict(n_rows=4, d=64, act=hg.LORA_ACT_SILU, x=FAKE, gate=FAKE, y=FAKE, held=FAKE, code=FAKE, scale=FAKE, x_stride=64,
             gate_stride=64, y_stride=64, held_stride=64)
    r.update(kw)
    return LIB.rows_act_i8(ctypes.byref(hg.lora_act_rows(**r)), None), LIB.lora_last_error().decode()


ROWS = [(dict(d=12), "multiple of 8"), (dict(d=0), "multiple of 8"), (dict(d=65544), "65536"), (dict(n_rows=-1), "rows"),
        (dict(n_rows=1 << 31), "rows"), (dict(x=None), "NULL"), (dict(x=FAKE + 8), "aligned"), (dict(x_stride=63), "aligned"),
        (dict(x_stride=56), "stride"), (dict(y=FAKE + 2), "y"), (dict(held_stride=8), "held"), (dict(code=None), "together"),
        (dict(scale=None), "together"), (dict(code=FAKE + 8), "aligned"), (dict(scale=FAKE + 2), "aligned"),
        (dict(y=None, held=None, code=None, scale=None), "no output")]


@pytest.mark.parametrize("kw,why", ROWS + [(dict(eps=0.0), "eps"), (dict(eps=-1.0), "eps"), (dict(eps=np.inf), "eps"),
                                           (dict(eps=np.nan), "eps"), (dict(weight=None), "weight"), (dict(weight=FAKE + 4), "weight"),
                                           (dict(residual=None), "residual"), (dict(residual_stride=0), "residual"),
                                           (dict(sum_stride=60), "sum_out")])
def test_norm_refusals(kw, why):
    rc, msg = norm(**kw)
    assert rc == EINVAL and why in msg


@pytest.mark.parametrize("kw,why", ROWS + [(dict(act=4), "act"), (dict(act=-1), "act"), (dict(gate=None), "gate"),
                                           (dict(act=hg.LORA_ACT_NONE), "gate"), (dict(gate_stride=32), "gate")])
def test_act_refusals(kw, why):
    rc, msg = act(**kw)
    assert rc == EINVAL and why in msg


def test_no_rows_are_no_work():
    assert norm(n_rows=0, x=None)[0] == hg.LORA_OK and act(n_rows=0, x=None)[0] == hg.LORA_OK
    assert LIB.rows_norm_i8(None, None) == EINVAL and LIB.rows_act_i8(None, None) == EINVAL
    assert LIB.base_gemm_i8(None, None, None, None, None, 0, 64, 64, None) == hg.LORA_OK
    assert LIB.base_gated_i8(None, None, None, None, None, None, hg.LORA_ACT_SILU, None, 0, 64, 64, None) == hg.LORA_OK


@pytest.mark.parametrize("M,N,K", [(-1, 64, 64), (4, 0, 64), (4, 64, 0), (4, 66, 64), (4, 64, 72), (4, 64, 131072), ((1 << 22) + 1, 64, 64),
                                   (4, (1 << 22) + 4, 64)])
def test_product_sizes(M, N, K):
    assert LIB.base_gemm_i8(FAKE, FAKE, FAKE, FAKE, FAKE, M, N, K, None) == EINVAL
    assert LIB.base_gated_i8(FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, hg.LORA_ACT_SILU, FAKE, M, N, K, None) == EINVAL


@pytest.mark.parametrize("bad", [None, FAKE + 4])
def test_product_pointers(bad):
    for i in range(5):
        p = [FAKE] * 5
        p[i] = bad
        assert LIB.base_gemm_i8(*p, 4, 64, 64, None) == EINVAL
    for i in range(7):
        p = [FAKE] * 7
        p[i] = bad
        assert LIB.base_gated_i8(*p[:6], hg.LORA_ACT_GELU, p[6], 4, 64, 64, None) == EINVAL
    for a in (hg.LORA_ACT_NONE, 4):
        assert LIB.base_gated_i8(*[FAKE] * 6, a, FAKE, 4, 64, 64, None) == EINVAL


def test_linear_refusals():
    pool = host_pool()
    plan = pool.plan(token_slot=[-1])
    call = lambda *p: LIB.lora_linear_i8(pool.pool.handle, plan.handle, 0, 0, *p, None)  # noqa: E731
    for i in (1, 2, 3, 4):
        p = [FAKE] * 6
        p[i] = None
        assert call(*p) == EINVAL and "required" in LIB.lora_last_error().decode()
    for i in (1, 2, 4):
        p = [FAKE] * 6
        p[i] = FAKE + 4
        assert call(*p) == EINVAL and "aligned" in LIB.lora_last_error().decode()
    assert call(*[FAKE] * 6) == EINVAL      # (a host-only pool)
    pool.pool.pages = On(0)
    for k in range(6):
        t = [On(0)] * 6
        t[k] = On(1)
        with pytest.raises(ValueError, match="one GPU"):
            pool.linear_i8(plan, 0, 0, *t, stream=0)


def test_rows_of_tensors_are_checked():
    torch = pytest.importorskip("torch")
    x, w = torch.zeros((4, 64), dtype=torch.bfloat16), torch.ones(64, dtype=torch.bfloat16)
    ok = dict(y=torch.zeros_like(x))
    for kw in (dict(y=torch.zeros((4, 64))), dict(y=torch.zeros((4, 72), dtype=torch.bfloat16)), dict(y=x.t()), dict(residual=x[:3], **ok),
               dict(code=torch.zeros((4, 64), dtype=torch.int8)), dict(code=torch.zeros((4, 64), dtype=torch.uint8), scale=torch.zeros(4)),
               dict(code=torch.zeros((4, 64), dtype=torch.int8), scale=torch.zeros(5)), ok):      # (and no GPU)
        with pytest.raises(ValueError):
            hg.rows_norm_i8(x, w, 1e-5, **kw)
    with pytest.raises(ValueError, match="weight"):
        hg.rows_norm_i8(x, w[:32], 1e-5, **ok)
    with pytest.raises(ValueError, match="rows"):
        hg.rows_norm_i8(x[0], w, 1e-5, **ok)
    with pytest.raises(ValueError, match="act"):
        hg.rows_act_i8(x, x, act="relu", **ok)
    with pytest.raises(ValueError, match="act"):
        hg.base_gated_i8(FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, 4, 64, 64, act="tanh")


def test_the_generators_weight():
    from workloads import make_workload
    wl = make_workload("c1")
    code, scale = wl.w0_i8()
    w = wl.w0().astype(np.float64)      # (the tiny layer's weight is fp32: the draw itself)
    assert code.dtype == np.int8 and np.all(np.abs(code).max(1) == 127)
    assert np.all(np.abs(w - scale[:, None].astype(np.float64) * code) <= 0.5 * scale[:, None] * (1 + 2.0 ** -20))


def test_packed_rows_are_the_structs():
    for packed, c in ((_lib._NORM_ROWS, hg.lora_norm_rows), (_lib._ACT_ROWS, hg.lora_act_rows)):
        v = [3, 40, 5] + list(range(1 << 40, (1 << 40) + len(c._fields_) - 3))
        assert packed.size == ctypes.sizeof(c) and packed.pack(*v) == bytes(c(*v))


def test_codes_by_whole_numbers():
    """The oracle's codes against whole-number arithmetic: p and max|p| as integers of one unit."""
    g = np.random.default_rng(5)
    for n, d in ((40, 64), (6, 1000)):
        a, b = g.integers(-255, 256, (n, d)), g.integers(128, 256, (n, d))
        a[:, 0] = 254
        a[:, 1], b[:, 1] = 127, b[:, 0]      # half of another value: a tie if that one is the greatest
        p = a * b                            # products of two 8-bit significands
        m = np.abs(p).max(1)
        got = E.codes(p.astype(np.float64) * 2.0 ** -11)
        for i in range(n):
            for j in range(d):
                q, r = divmod(127 * int(abs(p[i, j])), int(m[i]))
                q += 2 * r > m[i] or (2 * r == m[i] and q % 2)
                assert got[i, j] == (q if p[i, j] >= 0 else -q)
    assert np.array_equal(E.codes(np.zeros((2, 8))), np.zeros((2, 8)))
