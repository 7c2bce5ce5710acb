"""KV entry points and the 4-bit base without a GPU: refusals (every check comes before
any device work) and the 4-bit row form of the oracle by hand."""
import ctypes

import numpy as np
import pytest

import heterogeneous_adapter_gemm_amd as hg
from heterogeneous_adapter_gemm_amd import _lib
from oracle import kv_model as KV

FAKE = 4096   # never dereferenced: every call below fails a check on the host


def host_pool(page=1024, dtype=hg.LORA_BF16):
    return hg.DevicePool(dtype, page, 8, None, 1, [512], [512], 1, 8, 16, 1, device=None)


def batch(**kw):
    d = dict(n_heads=8, n_kv_heads=2, head_dim=128, n_seqs=3, n_rows=5, max_rows=2, max_blocks=4, reserved=0,
             row_start=FAKE, ctx_len=FAKE, page_table=FAKE)
    d.update(kw)
    return hg.lora_kv_batch(**d)


def rows(**kw):
    d = dict(k=FAKE, v=FAKE, q=FAKE, q_out=FAKE, k_out=None, v_out=None, k_stride=256, v_stride=256, q_stride=1024,
             q_out_stride=1024, k_out_stride=0, v_out_stride=0)
    d.update(kw)
    return hg.lora_kv_rows(**d)


def refused(fn, says):
    with pytest.raises(hg.LoraError) as e:
        fn()
    assert e.value.code == hg.LORA_EINVAL and says in str(e.value), str(e.value)


BAD_BATCH = [(dict(head_dim=96), "head_dim"), (dict(n_heads=7), "heads"), (dict(n_kv_heads=0), "heads"),
             (dict(n_heads=0), "heads"), (dict(n_seqs=-1), "range"), (dict(n_rows=-1), "range"),
             (dict(max_rows=-1), "range"), (dict(max_blocks=-1), "range"), (dict(max_blocks=(1 << 26) + 1), "range"),
             (dict(reserved=1), "reserved"), (dict(row_start=None), "NULL"), (dict(ctx_len=None), "NULL"),
             (dict(page_table=None), "NULL"), (dict(ctx_len=FAKE + 2), "aligned")]


@pytest.mark.parametrize("change,says", BAD_BATCH, ids=[str(list(c)[0]) + str(i) for i, (c, _) in enumerate(BAD_BATCH)])
def test_bad_batches_are_refused(change, says):
    pool = host_pool()
    b = batch(**change)
    refused(lambda: hg.lora_kv_append(pool.pool, b, rows(), stream=0), says)
    refused(lambda: hg.lora_kv_attention(pool.pool, b, FAKE, 1024, FAKE, 1024, 1.0, FAKE, 1 << 40, stream=0), says)


BAD_ROWS = [(dict(k=None), "k is NULL"), (dict(v=FAKE + 8), "aligned"), (dict(k_stride=255), "multiple of 8"),
            (dict(k_stride=248), "row stride"), (dict(q_out=None), "together"), (dict(q=None), "together"),
            (dict(q_stride=512), "row stride"), (dict(k_out=FAKE, k_out_stride=8), "row stride"),
            (dict(v_out=FAKE + 2, v_out_stride=256), "aligned")]


@pytest.mark.parametrize("change,says", BAD_ROWS, ids=[str(i) for i in range(len(BAD_ROWS))])
def test_bad_rows_are_refused(change, says):
    refused(lambda: hg.lora_kv_append(host_pool().pool, batch(), rows(**change), stream=0), says)


def test_bad_rotations_and_attention_arguments_are_refused():
    pool = host_pool()
    ap = lambda *a: hg.lora_kv_append(pool.pool, batch(), rows(), *a, stream=0)  # noqa: E731
    refused(lambda: ap(FAKE, 24, 64), "rot_dim")
    refused(lambda: ap(FAKE, 144, 64), "rot_dim")
    refused(lambda: ap(FAKE, 0, 64), "rot_dim")
    refused(lambda: ap(None, 16, 64), "rot_dim")
    refused(lambda: ap(FAKE, 128, 63), "positions")
    refused(lambda: ap(FAKE + 4, 128, 64), "aligned")
    assert _lib.library().lora_kv_append(pool.pool.handle, ctypes.byref(batch()), ctypes.byref(rows()), FAKE, 128, 64, 2,
                                         None) == hg.LORA_EINVAL
    need = hg.lora_kv_workspace_bytes(batch())
    at = lambda **k: hg.lora_kv_attention(pool.pool, batch(), *[{**dict(q=FAKE, qs=1024, out=FAKE, os=1024, scale=0.1,  # noqa: E731
                                                                         ws=FAKE, n=need), **k}[n]
                                                                 for n in ("q", "qs", "out", "os", "scale", "ws", "n")],
                                          stream=0)
    for scale in (0.0, -1.0, float("inf"), float("nan")):
        refused(lambda: at(scale=scale), "scale")
    refused(lambda: at(q=None), "q is NULL")
    refused(lambda: at(out=FAKE + 2), "aligned")
    refused(lambda: at(os=1016), "row stride")
    refused(lambda: at(ws=None), "workspace")
    refused(lambda: at(n=need - 1), "workspace")
    refused(lambda: at(), "host-only")
    refused(lambda: ap(FAKE, 128, 64), "host-only")


def test_pools_without_room_or_of_another_type_are_refused():
    refused(lambda: host_pool(512).kv_pages_per_block(2, 128), "slab")          # 1,024 bytes a page, 1,088 a slab
    refused(lambda: host_pool(dtype=hg.LORA_F32).kv_pages_per_block(2, 128), "bf16")
    # 8 KiB pages: 7 slabs of 1,088 bytes, 64 slabs of 32 heads; 16 slabs of 8 heads; one page when all fit
    assert host_pool(4096).kv_pages_per_block(32, 128) == 10
    assert host_pool(4096).kv_pages_per_block(8, 128) == 3
    assert host_pool(4096).kv_pages_per_block(1, 64) == 1
    assert host_pool(1024).kv_pages_per_block(3, 64) == 2


def test_workspace_depends_on_heads_and_rows_only():
    few, many = hg.lora_kv_workspace_bytes(batch(max_rows=4)), hg.lora_kv_workspace_bytes(batch(max_rows=5))
    assert 0 < few < many
    assert hg.lora_kv_workspace_bytes(batch(max_rows=4, n_seqs=1, n_rows=1, max_blocks=1 << 20)) == few


W4_BAD = [((4, 8, 128, 16), "group"), ((4, 8, 192, 64), "128"), ((4, 6, 128, 64), "4"), ((-1, 8, 128, 64), "sizes"),
          ((4, 0, 128, 64), "sizes"), ((4, 1 << 20, 1 << 13, 64), "2^31")]


@pytest.mark.parametrize("mnkg,says", W4_BAD, ids=[str(i) for i in range(len(W4_BAD))])
def test_base_gemm_w4_refusals(mnkg, says):
    M, N, K, G = mnkg
    refused(lambda: hg.base_gemm_w4(FAKE, FAKE, FAKE, FAKE, M, N, K, G, stream=0), says)


def test_base_gemm_w4_pointer_refusals():
    for i in range(4):
        p = [FAKE] * 4
        p[i] = None
        refused(lambda: hg.base_gemm_w4(*p, 4, 8, 128, 64, stream=0), "NULL")
        p[i] = FAKE + 8
        refused(lambda: hg.base_gemm_w4(*p, 4, 8, 128, 64, stream=0), "aligned")
    hg.base_gemm_w4(None, None, None, None, 0, 8, 128, 64, stream=0)   # no rows: a no-op
    pool = host_pool()
    plan = pool.plan(token_slot=[-1])
    refused(lambda: pool.linear_w4(plan, 0, 0, FAKE, FAKE, FAKE, 48, FAKE, stream=0), "group")
    refused(lambda: pool.linear_w4(plan, 0, 0, FAKE, None, FAKE, 64, FAKE, stream=0), "required")
    refused(lambda: pool.linear_w4(plan, 0, 0, FAKE, FAKE, FAKE, 64, FAKE, stream=0), "host-only")


def test_four_bit_rows_by_hand():
    """0 .. 15 with step 1 and lo 0 are their own codes; a constant row is exact with step 0;
    a tie goes to the even code; an infinity or NaN spoils its row only."""
    x = np.arange(16.0)[None]
    code, step, lo = KV.quantise(x)
    assert step[0] == 1 and lo[0] == 0 and np.array_equal(code[0], np.arange(16))
    code, step, lo = KV.quantise(np.full((1, 16), -3.5))
    assert step[0] == 0 and lo[0] == -3.5 and not code.any() and (KV.value(code, step, lo) == -3.5).all()
    x = np.array([[0.0, 15.0, 0.5, 1.5, 2.5] + [0.0] * 11])
    assert list(KV.quantise(x)[0][0][:5]) == [0, 15, 0, 2, 2]
    x = np.zeros((2, 16))
    x[0, 3] = np.inf
    code, step, _ = KV.quantise(x)
    assert np.isnan(step[0]) and step[1] == 0
    # word 0 of a key row holds values 0, 2, 4, 6 in its low half; unit (0, 0, 0, 1) of a value slab is token 1
    c = np.arange(64) % 16
    assert KV.key_bytes(c, 0)[0] == 0x20 and KV.key_bytes(c, 0)[2] == 0x31
    assert KV.value_bytes(c, 1)[2] == 0x10 and KV.value_bytes(c, 1)[3] == 0x32


def test_oracle_attention_by_hand():
    """Equal keys weigh every seen token the same; the row sees what the mask leaves."""
    q = np.ones((2, 2, 4))
    k = np.ones((3, 1, 4))
    v = np.arange(3.0)[:, None, None] * np.ones((3, 1, 4))
    out = KV.attention(q, k, v, 1, 0.5)
    assert np.allclose(out[0], 0.5) and np.allclose(out[1], 1.0)
    assert np.allclose(KV.attention(q, k, v, 1, 0.5, hidden=[0])[1], 1.5)
    assert not KV.attention(q, k[:1], v[:1], 1, 0.5)[0].any()       # two rows, one token: the first sees none


def test_rows_of_all_heads_stay_in_32_bits():
    """Row and tile numbers over all heads are 32-bit in the kernels: larger batches are refused."""
    pool = host_pool()
    big = dict(n_heads=1024, n_kv_heads=1, n_rows=1 << 20)
    for b in (batch(**dict(big, n_rows=(1 << 20) + 1)), batch(**dict(big, n_heads=2048))):
        refused(lambda: hg.lora_kv_append(pool.pool, b, rows(), stream=0), "2^30")
        refused(lambda: hg.lora_kv_attention(pool.pool, b, FAKE, 1 << 20, FAKE, 1 << 20, 1.0, FAKE, 1 << 40, stream=0), "2^30")
        refused(lambda: hg.lora_kv_workspace_bytes(b), "2^30")
    assert hg.lora_kv_workspace_bytes(batch(**big)) > 0


def test_w4_host_tensors_are_refused():
    import numpy as np
    import torch
    host = torch.zeros(8, 128, dtype=torch.bfloat16)
    pool = host_pool()
    plan = pool.plan(token_slot=[-1])
    for bad in (host, np.zeros((8, 128), np.float32)):
        with pytest.raises(ValueError, match="one GPU"):
            hg.base_gemm_w4(bad, FAKE, FAKE, FAKE, 8, 8, 128, 64, stream=0)
        with pytest.raises(ValueError, match="one GPU"):
            pool.linear_w4(plan, 0, 0, FAKE, FAKE, FAKE, 64, bad, stream=0)
