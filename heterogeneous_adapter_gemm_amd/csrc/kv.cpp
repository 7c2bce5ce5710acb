// Host side of the KV entry points (lora_kv_*): argument checks and launches.
// See include/lora_gemm.h for the contract of every entry point.
#include <cmath>

#include "internal.h"
#include "kv.h"
#include "lora_gemm.h"

using namespace hagemm;

namespace {

bool head_dim_ok(int32_t d) { return d == 64 || d == 128 || d == 256; }

int geometry(const lora_pool* p, int32_t kv_heads, int32_t head_dim, KvArgs* a) {
    if (!p) return set_error(LORA_EINVAL, "pool is NULL");
    const PoolPages pp = pool_pages(p);
    if (pp.dtype != LORA_BF16) return set_error(LORA_EINVAL, "the KV calls need a bf16 pool");
    if (!head_dim_ok(head_dim)) return set_error(LORA_EINVAL, "head_dim %d: 64, 128 or 256", head_dim);
    if (kv_heads < 1 || kv_heads > 4096) return set_error(LORA_EINVAL, "%d KV heads", kv_heads);
    const int64_t per_page = pp.page_bytes / kv_slab_bytes(head_dim);
    if (per_page < 1)
        return set_error(LORA_EINVAL, "a page of %lld bytes holds no slab of %d bytes (16 tokens of one head)",
                         (long long)pp.page_bytes, kv_slab_bytes(head_dim));
    a->pages = static_cast<uint8_t*>(pp.pages_dev);
    a->page_bytes = pp.page_bytes;
    a->num_pages = (int32_t)(pp.num_pages < INT32_MAX ? pp.num_pages : INT32_MAX);
    a->kv_heads = kv_heads;
    a->slabs_per_page = (int32_t)(per_page < 2 * kv_heads ? per_page : 2 * kv_heads);
    a->pages_per_block = (2 * kv_heads + a->slabs_per_page - 1) / a->slabs_per_page;
    return LORA_OK;
}

int check_sizes(const lora_kv_batch* b) {
    if (!b) return set_error(LORA_EINVAL, "batch is NULL");
    if (!head_dim_ok(b->head_dim)) return set_error(LORA_EINVAL, "head_dim %d: 64, 128 or 256", b->head_dim);
    if (b->n_kv_heads < 1 || b->n_kv_heads > 4096 || b->n_heads < 1 || b->n_heads > 65536 || b->n_heads % b->n_kv_heads)
        return set_error(LORA_EINVAL, "%d query heads over %d KV heads", b->n_heads, b->n_kv_heads);
    if (b->n_seqs < 0 || b->n_seqs > (1 << 20) || b->n_rows < 0 || b->n_rows > (1 << 22) || b->max_rows < 0 ||
        b->max_blocks < 0 || b->max_blocks > (1 << 26) || b->reserved != 0)
        return set_error(LORA_EINVAL, "n_seqs, n_rows, max_rows or max_blocks out of range, or reserved not 0");
    // (the kernels count a batch's rows of all heads in 32 bits)
    if ((int64_t)b->n_rows * b->n_heads > (int64_t(1) << 30))
        return set_error(LORA_EINVAL, "%d rows of %d heads: at most 2^30 together", b->n_rows, b->n_heads);
    return LORA_OK;
}

// *empty: nothing to do (no sequences or no rows)
int batch_args(const lora_pool* p, const lora_kv_batch* b, KvArgs* a, bool* empty) {
    int rc = check_sizes(b);
    if (rc) return rc;
    rc = geometry(p, b->n_kv_heads, b->head_dim, a);
    if (rc) return rc;
    *empty = b->n_seqs == 0 || b->n_rows == 0;
    if (*empty) return LORA_OK;
    if (!b->row_start || !b->ctx_len || (!b->page_table && b->max_blocks > 0))
        return set_error(LORA_EINVAL, "row_start, ctx_len or page_table is NULL");
    if ((uintptr_t)b->row_start % 4 || (uintptr_t)b->ctx_len % 4 || (uintptr_t)b->page_table % 4)
        return set_error(LORA_EINVAL, "row_start, ctx_len and page_table must be 4-byte aligned");
    a->heads = b->n_heads;
    a->group = b->n_heads / b->n_kv_heads;
    a->n_seqs = b->n_seqs;
    a->n_rows = b->n_rows;
    a->max_blocks = b->max_blocks;
    a->row_start = b->row_start;
    a->ctx_len = b->ctx_len;
    a->table = b->page_table;
    return LORA_OK;
}

int on_device(const KvArgs& a) {
    return a.pages ? LORA_OK : set_error(LORA_EINVAL, "host-only pool: no device work");
}

int check_rows(const char* name, const void* ptr, int64_t stride, int64_t width) {
    if (!ptr) return set_error(LORA_EINVAL, "%s is NULL", name);
    if ((uintptr_t)ptr % 16 || stride % 8) return set_error(LORA_EINVAL, "%s: 16-byte aligned rows (stride a multiple of 8)", name);
    if (stride < width || stride > (int64_t(1) << 32))
        return set_error(LORA_EINVAL, "%s: row stride %lld below %lld heads x head_dim", name, (long long)stride, (long long)width);
    return LORA_OK;
}

}  // namespace

extern "C" {

int lora_kv_pages_per_block(const lora_pool* pool, int32_t n_kv_heads, int32_t head_dim, int32_t* out) {
    KvArgs a{};
    const int rc = geometry(pool, n_kv_heads, head_dim, &a);
    if (rc) return rc;
    if (!out) return set_error(LORA_EINVAL, "out is NULL");
    *out = a.pages_per_block;
    return LORA_OK;
}

int lora_kv_workspace_bytes(const lora_kv_batch* batch, int64_t* out_bytes) {
    const int rc = check_sizes(batch);
    if (rc) return rc;
    if (!out_bytes) return set_error(LORA_EINVAL, "out_bytes is NULL");
    *out_bytes = kv_workspace_bytes(batch->head_dim, batch->n_heads / batch->n_kv_heads, batch->max_rows);
    return LORA_OK;
}

int lora_kv_append(lora_pool* pool, const lora_kv_batch* batch, const lora_kv_rows* r, const float* cos_sin,
                   int32_t rot_dim, int32_t rot_positions, int32_t interleaved, void* stream) {
    KvArgs b{};
    bool empty = false;
    int rc = batch_args(pool, batch, &b, &empty);
    if (rc) return rc;
    if (!r) return set_error(LORA_EINVAL, "rows is NULL");
    const int D = batch->head_dim;
    const int64_t kw = (int64_t)b.kv_heads * D, qw = (int64_t)batch->n_heads * D;
    if (interleaved != 0 && interleaved != 1) return set_error(LORA_EINVAL, "interleaved must be 0 or 1");
    if (cos_sin) {
        if (rot_dim < 16 || rot_dim > D || rot_dim % 16)
            return set_error(LORA_EINVAL, "rot_dim %d: a multiple of 16 up to head_dim", rot_dim);
        if ((int64_t)rot_positions < (int64_t)batch->max_blocks * kKvBlock)
            return set_error(LORA_EINVAL, "cos_sin has %d positions, the page table holds %lld tokens", rot_positions,
                             (long long)batch->max_blocks * kKvBlock);
        if ((uintptr_t)cos_sin % 16) return set_error(LORA_EINVAL, "cos_sin must be 16-byte aligned");
    } else if (rot_dim != 0) {
        return set_error(LORA_EINVAL, "rot_dim must be 0 without cos_sin");
    }
    if (empty) return on_device(b);
    if ((rc = check_rows("k", r->k, r->k_stride, kw)) || (rc = check_rows("v", r->v, r->v_stride, kw))) return rc;
    if ((r->q == nullptr) != (r->q_out == nullptr)) return set_error(LORA_EINVAL, "q and q_out go together");
    if (r->q && ((rc = check_rows("q", r->q, r->q_stride, qw)) || (rc = check_rows("q_out", r->q_out, r->q_out_stride, qw))))
        return rc;
    if (r->k_out && (rc = check_rows("k_out", r->k_out, r->k_out_stride, kw))) return rc;
    if (r->v_out && (rc = check_rows("v_out", r->v_out, r->v_out_stride, kw))) return rc;
    if ((rc = on_device(b))) return rc;
    KvAppendArgs a{r->q, r->k, r->v, r->q_out, r->k_out, r->v_out, r->q_stride, r->k_stride, r->v_stride,
                   r->q_out_stride, r->k_out_stride, r->v_out_stride, cos_sin, rot_dim, interleaved};
    const hipError_t e = launch_kv_append(D, b, a, static_cast<hipStream_t>(stream));
    if (e != hipSuccess) return set_error(LORA_EHIP, "kv append: %s", hipGetErrorString(e));
    return LORA_OK;
}

int lora_kv_attention(lora_pool* pool, const lora_kv_batch* batch, const void* q, int64_t q_stride, void* out,
                      int64_t out_stride, float scale, void* workspace, int64_t workspace_bytes, void* stream) {
    KvArgs b{};
    bool empty = false;
    int rc = batch_args(pool, batch, &b, &empty);
    if (rc) return rc;
    if (!(scale > 0.f) || !std::isfinite(scale)) return set_error(LORA_EINVAL, "scale must be positive and finite");
    if (empty) return on_device(b);
    const int64_t qw = (int64_t)batch->n_heads * batch->head_dim;
    if ((rc = check_rows("q", q, q_stride, qw)) || (rc = check_rows("out", out, out_stride, qw))) return rc;
    const int64_t need = kv_launch_bytes(batch->head_dim, b.group, batch->max_rows);
    if (!workspace || (uintptr_t)workspace % 16 || workspace_bytes < need)
        return set_error(LORA_EINVAL, "workspace: %lld bytes, 16-byte aligned", (long long)need);
    if ((rc = on_device(b))) return rc;
    const hipError_t e = launch_kv_attention(batch->head_dim, b, q, q_stride, out, out_stride, scale, batch->max_rows,
                                             workspace, static_cast<hipStream_t>(stream));
    if (e != hipSuccess) return set_error(LORA_EHIP, "kv attention: %s", hipGetErrorString(e));
    return LORA_OK;
}

}  // extern "C"
