"""Device-memory plumbing around the C ABI.

``DevicePool`` allocates the pool's page buffer and metadata workspace with
PyTorch (the library itself never allocates device memory), pins adapter
host blobs for page-in, and forwards every operation to the library.  A
host-only pool (``device=None``) runs the allocator, tables and plans with
no GPU at all.
"""
from __future__ import annotations

from typing import Dict, Optional, Sequence

import numpy as np

from . import _lib as L


def torch_dtype(dtype: int):
    import torch
    return torch.bfloat16 if dtype == L.LORA_BF16 else torch.float32


def host_tensor(arr: np.ndarray, pin: bool = True):
    """numpy (bf16 bits as uint16, or float32) -> torch CPU tensor of the
    matching dtype, pinned (allocated pinned, not registered) when asked."""
    import torch
    a = np.ascontiguousarray(arr)
    t = torch.from_numpy(a.view(np.int16)).view(torch.bfloat16) if a.dtype == np.uint16 else torch.from_numpy(a)
    if pin:
        p = torch.empty(t.shape, dtype=t.dtype, pin_memory=True)
        p.copy_(t)
        return p
    return t


def device_tensor(arr: np.ndarray, device="cuda"):
    return host_tensor(arr, pin=False).to(device)


class KvBatch:
    """A batch over the pool's KV pages (lora_kv_batch in the C header): device int32 tensors
    row_start [n_seqs + 1], ctx_len [n_seqs] and page_table [n_seqs, max_blocks, pages per block]
    (one layer's), n_rows rows of q, k and v, at most max_rows of one sequence (None: n_rows, since the
    lengths are on the device; decode batches give it: from more than 64 query rows of a KV head on
    the kernels of prompts run beside those of few rows, and take their workspace).
    The tensors are read when the kernels run: a caller may write new lengths or pages into
    them between calls, and between replays of a captured one."""

    def __init__(self, n_heads: int, n_kv_heads: int, head_dim: int, row_start, ctx_len, page_table, n_rows: int,
                 max_rows: Optional[int] = None):
        import torch
        for name, t, dim in (("row_start", row_start, 1), ("ctx_len", ctx_len, 1), ("page_table", page_table, 3)):
            if t.dtype != torch.int32 or t.dim() != dim or not t.is_contiguous():
                raise ValueError(f"{name} must be a contiguous int32 tensor of {dim} dimension(s)")
        n_seqs = ctx_len.shape[0]
        if row_start.shape[0] != n_seqs + 1 or page_table.shape[0] != n_seqs:
            raise ValueError(f"{n_seqs} lengths, {row_start.shape[0]} row starts, {page_table.shape[0]} page tables")
        if len({row_start.device, ctx_len.device, page_table.device}) != 1:
            raise ValueError("row_start, ctx_len and page_table must be on one device")
        self.row_start, self.ctx_len, self.page_table = row_start, ctx_len, page_table
        self.device, self.index = row_start.device, row_start.get_device()
        self.pages_per_block = page_table.shape[2]
        self.n_rows = n_rows
        self.dtype, self.f32, self.cuda = torch.bfloat16, torch.float32, torch.cuda
        self.c = L.lora_kv_batch(n_heads, n_kv_heads, head_dim, n_seqs, n_rows, n_rows if max_rows is None else max_rows,
                                 page_table.shape[1], 0, row_start.data_ptr(), ctx_len.data_ptr(),
                                 page_table.data_ptr())
        self.heads = (n_heads, head_dim), (n_kv_heads, head_dim)

    def rows(self, name: str, t, kv: bool):
        """Address and row stride of t, checked to be this batch's rows of the query (or KV) heads."""
        heads, dim = self.heads[kv]
        if t.get_device() != self.index or t.dtype is not self.dtype:
            raise ValueError(f"{name} must be {self.dtype} on {self.device}")
        shape, st = t.shape, t.stride()
        if len(shape) == 3 and shape[1] == heads and shape[2] == dim:
            inner = st[2] == 1 and (heads == 1 or st[1] == dim)
        elif len(shape) == 2 and shape[1] == heads * dim:
            inner = st[1] == 1
        else:
            raise ValueError(f"{name}: shape {tuple(shape)}, not [rows, {heads}, {dim}] or [rows, {heads * dim}]")
        if shape[0] != self.n_rows or not inner:
            raise ValueError(f"{name}: {self.n_rows} rows of contiguous heads are needed")
        return t.data_ptr(), st[0] if self.n_rows > 1 else heads * dim


class DevicePool:
    def __init__(self, dtype: int, page_elems: int, num_pages: int, free_order: Optional[Sequence[int]],
                 n_layers: int, d_in: Sequence[int], d_out: Sequence[int], max_slots: int, max_rank: int,
                 max_tokens: int, max_segments: int, base_id: int = 0, device: Optional[str] = "cuda",
                 stage_bytes: int = 0, max_multi: int = 1):
        """stage_bytes > 0: a device staging area of that size for page-ins (copy engine into
        the staging area, then a scatter kernel); 0: page-ins gather over PCIe.  max_multi: most
        projections one linear_multi call takes."""
        self.dtype = dtype
        self.page_elems = page_elems
        self.num_pages = num_pages
        self.n_layers = n_layers
        self.d_in = list(d_in)
        self.d_out = list(d_out)
        self.base_id = base_id
        self.device = device
        desc, keep = L.make_desc(dtype, page_elems, num_pages, None, free_order, n_layers, d_in, d_out, max_slots,
                                 max_rank, max_tokens, max_segments, None, 0, base_id, max_multi=max_multi)
        self.pages = self.meta = self.stage = None
        if device is not None:
            import torch
            meta_bytes = L.lora_pool_meta_bytes(desc)
            self.pages = torch.empty(num_pages * page_elems, dtype=torch_dtype(dtype), device=device)
            self.meta = torch.empty(meta_bytes, dtype=torch.uint8, device=device)
            desc.pages_dev = self.pages.data_ptr()
            desc.meta_dev = self.meta.data_ptr()
            desc.meta_bytes = meta_bytes
            if stage_bytes > 0:
                self.stage = torch.empty(stage_bytes, dtype=torch.uint8, device=device)
                desc.stage_dev = self.stage.data_ptr()
                desc.stage_bytes = stage_bytes
        self.pool = L.lora_pool_create(desc, keep)
        self.pool.pages = self.pages
        self._host: Dict[int, tuple] = {}
        self._kv_pages: Dict[tuple, int] = {}

    # -- adapters ---------------------------------------------------------------
    def page_in(self, adapter_id: int, rank: int, alpha: float, A_blob: Optional[np.ndarray] = None,
                B_blob: Optional[np.ndarray] = None, stream=None, base_id: Optional[int] = None) -> int:
        base = self.base_id if base_id is None else base_id
        if self.device is None:
            return L.lora_pool_page_in(self.pool, adapter_id, rank, alpha, base, None, None, None)
        hA, hB = host_tensor(A_blob), host_tensor(B_blob)
        slot = L.lora_pool_page_in(self.pool, adapter_id, rank, alpha, base, hA, hB, stream)
        self._host[adapter_id] = (hA, hB)   # the copy reads these until it has run
        return slot

    def page_in_pinned(self, adapter_id: int, rank: int, alpha: float, hA, hB, stream=None) -> int:
        """Page in from already-pinned torch host tensors (kept alive by the caller)."""
        return L.lora_pool_page_in(self.pool, adapter_id, rank, alpha, self.base_id, hA, hB, stream)

    def page_in_pinned_batch(self, items, stream=None) -> np.ndarray:
        """Page in several adapters, layer by layer: items = [(adapter_id, rank, alpha, hA, hB)]
        with already-pinned torch host tensors (kept alive by the caller)."""
        return L.lora_pool_page_in_batch(self.pool, [(a, r, al, self.base_id, hA, hB) for a, r, al, hA, hB in items],
                                         stream)

    def page_in_batch(self, items, stream=None) -> np.ndarray:
        """items = [(adapter_id, rank, alpha, A_blob, B_blob)] from host arrays (pinned copies
        are made and kept until drop_host_copies); host-only pools take no blobs."""
        if self.device is None:
            return L.lora_pool_page_in_batch(self.pool, [(a, r, al, self.base_id, None, None)
                                                         for a, r, al, *_ in items], None)
        reqs = []
        for a, r, al, A, B in items:
            hA, hB = host_tensor(A), host_tensor(B)
            self._host[a] = (hA, hB)
            reqs.append((a, r, al, self.base_id, hA, hB))
        return L.lora_pool_page_in_batch(self.pool, reqs, stream)

    def drop_host_copies(self) -> None:
        """Forget the pinned host blobs; call after the page-in work has run."""
        self._host.clear()

    def evict(self, adapter_id: int) -> None:
        L.lora_pool_evict(self.pool, adapter_id)
        self._host.pop(adapter_id, None)

    def slot_of(self, adapter_id: int) -> int:
        return L.lora_pool_slot_of(self.pool, adapter_id)

    def slots_of(self, adapter_ids) -> np.ndarray:
        return L.lora_pool_slots_of(self.pool, adapter_ids)

    def alloc_kv(self, n: int) -> np.ndarray:
        return L.lora_pool_alloc_kv(self.pool, n)

    def free_kv(self, pages) -> None:
        L.lora_pool_free_kv(self.pool, pages)

    def page_table(self, slot: int, layer: int, proj: int):
        return L.lora_pool_page_table(self.pool, slot, layer, proj)

    def free_list(self) -> np.ndarray:
        return L.lora_pool_free_list(self.pool)

    def stats(self):
        return L.lora_pool_stats(self.pool)

    # -- batches ------------------------------------------------------------------
    def plan(self, seg_start=None, seg_slot=None, token_slot=None, stream=None) -> L.Plan:
        return L.lora_plan_create(self.pool, seg_start, seg_slot, token_slot, stream)

    def linear(self, plan: L.Plan, layer: int, proj: int, x, w0, y, stream=None) -> None:
        L.lora_linear(self.pool, plan, layer, proj, x, w0, y, stream)

    def linear_multi(self, plan: L.Plan, layer: int, projs, x, w0s, ys, stream=None) -> None:
        """Projections projs of one layer that share x, their shrinks in shared launches."""
        L.lora_linear_multi(self.pool, plan, layer, projs, x, w0s, ys, stream)

    def linear_fp8(self, plan: L.Plan, layer: int, proj: int, x, w0_code, w0_scale, y, stream=None) -> None:
        L.lora_linear_fp8(self.pool, plan, layer, proj, x, w0_code, w0_scale, y, stream)

    def linear_w4(self, plan: L.Plan, layer: int, proj: int, x, w0_code, w0_scale, group: int, y, stream=None) -> None:
        L.lora_linear_w4(self.pool, plan, layer, proj, x, w0_code, w0_scale, group, y, stream)

    def linear_i8(self, plan: L.Plan, layer: int, proj: int, x, x_code, x_scale, w0_code, w0_scale, y, stream=None) -> None:
        """x: the bf16 rows the adapters read; x_code, x_scale: the 8-bit form of them that the base reads."""
        L.lora_linear_i8(self.pool, plan, layer, proj, x, x_code, x_scale, w0_code, w0_scale, y, stream)

    # -- keys and values in the pages ----------------------------------------------
    def kv_pages_per_block(self, n_kv_heads: int, head_dim: int) -> int:
        """Pages of 16 tokens' keys and values in one layer."""
        n = self._kv_pages.get((n_kv_heads, head_dim))
        if n is None:
            n = self._kv_pages[n_kv_heads, head_dim] = L.lora_kv_pages_per_block(self.pool, n_kv_heads, head_dim)
        return n

    def kv_workspace(self, batch: KvBatch):
        """A workspace for kv_attention; calls that may overlap need one each."""
        import torch
        return torch.empty(L.lora_kv_workspace_bytes(batch.c), dtype=torch.uint8, device=batch.device)

    def _kv_call(self, batch: KvBatch, stream, call, *args) -> None:
        """call(pool, batch, *args, stream) on the batch's GPU, whichever is current."""
        if self.pages is None or batch.index != self.pages.get_device():
            raise ValueError(f"the batch is on {batch.device}, the pool on {None if self.pages is None else self.pages.device}")
        need = self.kv_pages_per_block(*batch.heads[1])
        if batch.pages_per_block != need:
            raise ValueError(f"page_table has {batch.pages_per_block} pages a block, {need} are needed")
        if stream is None:
            stream = L.current_stream(batch.index)
        cuda = batch.cuda
        if cuda.current_device() == batch.index:
            call(self.pool, batch.c, *args, stream)
        else:
            with cuda.device(batch.index):
                call(self.pool, batch.c, *args, stream)

    def kv_append(self, batch: KvBatch, k, v, q=None, q_out=None, k_out=None, v_out=None, cos_sin=None,
                  interleaved: bool = False, stream=None) -> None:
        """Append the rows' keys and values to their pages; q, k turned by cos_sin [positions, rot_dim]."""
        rows, none = batch.rows, (None, 0)
        kp, ks = rows("k", k, True)
        vp, vs = rows("v", v, True)
        qp, qs = none if q is None else rows("q", q, False)
        tp, ts = none if q_out is None else rows("q_out", q_out, False)
        kop, kos = none if k_out is None else rows("k_out", k_out, True)
        vop, vos = none if v_out is None else rows("v_out", v_out, True)
        r = L.lora_kv_rows(kp, vp, qp, tp, kop, vop, ks, vs, qs, ts, kos, vos)
        pos = rot = 0
        if cos_sin is not None:
            if cos_sin.dtype is not batch.f32 or cos_sin.dim() != 2 or not cos_sin.is_contiguous() or \
                    cos_sin.get_device() != batch.index:
                raise ValueError("cos_sin must be a contiguous float32 [positions, rot_dim] tensor on the batch's device")
            pos, rot = cos_sin.shape
            cos_sin = cos_sin.data_ptr()
        self._kv_call(batch, stream, L.lora_kv_append, r, cos_sin, rot, pos, interleaved)

    def kv_attention(self, batch: KvBatch, q, out, scale: Optional[float] = None, workspace=None, stream=None) -> None:
        """Attention of the batch's rows (q already turned) over the pages; scale None: head_dim ** -0.5."""
        if workspace is None:
            raise ValueError("kv_attention needs a workspace (kv_workspace)")
        if workspace.get_device() != batch.index or not workspace.is_contiguous():
            raise ValueError("the workspace must be contiguous and on the batch's device")
        (qp, qs), (op, os_) = batch.rows("q", q, False), batch.rows("out", out, False)
        if scale is None:
            scale = batch.heads[0][1] ** -0.5
        size = workspace.numel() * workspace.element_size()
        self._kv_call(batch, stream, L.lora_kv_attention, qp, qs, op, os_, scale, workspace.data_ptr(), size)

    def linear_decode(self, layer: int, proj: int, x, w0, y, token_slot, stream=None) -> None:
        L.lora_linear_decode(self.pool, layer, proj, x, w0, y, token_slot, stream)

    def linear_decode_noalloc(self, layer: int, proj: int, x, w0, y, token_slot, stream=None) -> None:
        L.lora_linear_decode_noalloc(self.pool, layer, proj, x, w0, y, token_slot, stream)

    def linear_prefill(self, layer: int, proj: int, x, w0, y, seg_start, seg_slot, stream=None) -> None:
        L.lora_linear_prefill(self.pool, layer, proj, x, w0, y, seg_start, seg_slot, stream)

    def set_timing(self, enable) -> None:
        """True / 1: time every call's kernels; k > 1: every k-th call; False / 0: off."""
        L.lora_pool_set_timing(self.pool, int(enable))

    def timing(self) -> Dict[str, tuple]:
        """{kernel name: (total ms, launches)} since timing was enabled."""
        return {name: L.lora_pool_timing(self.pool, k) for k, name in enumerate(L.KERNEL_NAMES)}

    def close(self) -> None:
        L.lora_pool_destroy(self.pool)


class AdapterEngine:
    """The engine layer over a DevicePool (host tier, GPU-tier LRU, look-ahead page-ins,
    admission; see lora_engine_* in the C header).

    Storage is two Python callables:
      info(adapter_id) -> (rank, alpha, base_id)
      fill(adapter_id, A, B): write the adapter's A and B blobs (layouts of page-in) into the
        flat host-cache views A and B (uint16 bf16 bits or float32, by the pool's dtype).
    An exception in either becomes a failed call (nonzero status) in the library.
    """

    def __init__(self, pool: DevicePool, info, fill, host_cache_bytes: int, max_step_tokens: int,
                 max_distinct_adapters: int, max_running: Optional[int] = None, prefetch_window: int = 64,
                 admit_in_flight: bool = True, max_wait_steps: int = 0, kv_pages_per_token: int = 0,
                 copy_stream=None):
        import ctypes
        self.pool = pool
        self.errors = errors = []   # the callbacks hold this list, not self (no reference cycle)
        elem = np.uint16 if pool.dtype == L.LORA_BF16 else np.float32
        esize = np.dtype(elem).itemsize

        def _info(_user, adapter_id, rank, alpha, base):
            try:
                r, a, b = info(int(adapter_id))
                rank[0], alpha[0], base[0] = int(r), float(a), int(b)
                return 0
            except Exception as exc:   # reported through the library's status
                errors.append(exc)
                return -1

        def _fill(_user, adapter_id, host_a, a_bytes, host_b, b_bytes):
            try:
                A = np.ctypeslib.as_array((ctypes.c_uint8 * a_bytes).from_address(host_a)).view(elem)
                B = np.ctypeslib.as_array((ctypes.c_uint8 * b_bytes).from_address(host_b)).view(elem)
                assert A.size * esize == a_bytes and B.size * esize == b_bytes
                fill(int(adapter_id), A, B)
                return 0
            except Exception as exc:
                errors.append(exc)
                return -1

        self._cb = (L.INFO_FN(_info), L.FILL_FN(_fill))
        d = L.lora_engine_desc()
        d.host_cache_bytes = int(host_cache_bytes)
        d.max_step_tokens = int(max_step_tokens)
        d.max_distinct_adapters = int(max_distinct_adapters)
        d.max_running = int(max_step_tokens if max_running is None else max_running)
        d.prefetch_window = int(prefetch_window)
        d.admit_in_flight = int(bool(admit_in_flight))
        d.max_wait_steps = int(max_wait_steps)
        d.kv_pages_per_token = int(kv_pages_per_token)
        d.info, d.fill = self._cb
        d.copy_stream = None if copy_stream is None else (copy_stream if isinstance(copy_stream, int)
                                                            else copy_stream.cuda_stream)
        self.engine = L.lora_engine_create(pool.pool, d, list(self._cb))
        self.batch = None

    def submit(self, request_id: int, adapter_id: int, prompt_tokens: int, max_new_tokens: int) -> None:
        L.lora_engine_submit(self.engine, request_id, adapter_id, prompt_tokens, max_new_tokens)

    def cancel(self, request_id: int) -> None:
        L.lora_engine_cancel(self.engine, request_id)

    def step(self, stream=None):
        """-> (batch dict with 'requests', 'adapters', 'rows' arrays added, plan or None)."""
        b, plan = L.lora_engine_step(self.engine, 0 if self.pool.device is None else stream)
        ids, ads, rows = L.lora_engine_batch_requests(self.engine, b["n_requests"])
        b.update(requests=ids, adapters=ads, rows=rows)
        self.batch = b
        return b, plan

    def step_done(self) -> None:
        L.lora_engine_step_done(self.engine)
        self.batch = None

    def row_adapter(self) -> np.ndarray:
        """Adapter id of every row of the current step's plan (-1 = none)."""
        b = self.batch
        return np.repeat(b["adapters"], b["rows"]).astype(np.int32)

    def kv_pages(self, request_id: int) -> np.ndarray:
        return L.lora_engine_kv_pages(self.engine, request_id)

    def stats(self) -> Dict[str, float]:
        return L.lora_engine_get_stats(self.engine)

    def reset_stats(self) -> None:
        L.lora_engine_reset_stats(self.engine)

    def close(self) -> None:
        L.lora_engine_destroy(self.engine)
