// Declarations shared by the KV host side (kv.cpp) and its gfx950 kernels
// (kv_kernels.hip).  Not part of the public ABI.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace hagemm {

constexpr int kKvBlock = 16;   // tokens of one slab

// Bytes of one slab: 16 rows of head_dim 4-bit codes and 16 words.
constexpr int kv_slab_bytes(int head_dim) { return 8 * head_dim + 64; }

// A batch over the pool's KV pages (the C header's lora_kv_batch with the pool's part).
struct KvArgs {
    uint8_t* pages;
    int64_t page_bytes;
    int32_t num_pages;
    int32_t heads, kv_heads, group;      // group = heads / kv_heads
    int32_t n_seqs, n_rows, max_blocks;
    int32_t pages_per_block, slabs_per_page;
    const int32_t* row_start;
    const int32_t* ctx_len;
    const int32_t* table;
};

struct KvAppendArgs {
    const void *q, *k, *v;
    void *q_out, *k_out, *v_out;         // q_out NULL: no q; k_out, v_out may be NULL
    int64_t q_stride, k_stride, v_stride, q_out_stride, k_out_stride, v_out_stride;   // elements
    const float* cos_sin;                // [positions][rot]: rot / 2 cosines, then sines; NULL: no rotation
    int32_t rot, interleaved;
};

// Append workgroups that run at once, by their registers: five on each of 256 CUs (head_dim 128) or four
constexpr int64_t kv_append_blocks(int head_dim) { return 256 * (head_dim == 128 ? 5 : 4); }
constexpr int kKvRowTile = 16;           // query rows of a decode segment
// Most query rows of a KV head that go in decode segments, up to four of them: 64 requests of about 2,100
// tokens (32 heads over 8 of 128) 76 us for 109 with 8 rows each, 105 (130) with 12, 148 (146) with 16;
// eight of about 1,750 22 (33), 27 (37), 29 (37); 33 x 36 rows of one head of 64 19 (26).
constexpr int kKvFewRows = 64;
constexpr int kKvPrefillRows = 128;      // query rows of a prefill segment
// Waves that share the attention's work, as many as run at once by their registers: on each of
// 256 CUs 16 (head_dim 64), 12 (128) or 8 (256).  A prefill worker is a workgroup of four, two a CU.
constexpr int kKvPrefillWorkers = 512;
constexpr int kv_workers(int head_dim) { return 1024 * (head_dim == 64 ? 4 : head_dim == 128 ? 3 : 2); }
// A batch whose sequences may have more query rows of a KV head than that runs the kernels of many rows
// beside those of few (sequences of either kind may meet in it); the one rule for the launch and for
// the workspace that it takes.
constexpr bool kv_many_rows(int group, int max_rows) { return (int64_t)max_rows * group > kKvFewRows; }
// An entry a worker, and two partial results of a row tile of fp32 sums and (m, l) each; for a batch of
// many rows both kinds of worker's, side by side.
constexpr int64_t kv_few_bytes(int head_dim) {
    return (int64_t)kv_workers(head_dim) * (36 + 2 * kKvRowTile * (head_dim + 2) * 4);
}
constexpr int64_t kv_many_bytes(int head_dim) {
    return (int64_t)kKvPrefillWorkers * (36 + 2 * kKvPrefillRows * (head_dim + 2) * 4);
}
// What a call takes
constexpr int64_t kv_launch_bytes(int head_dim, int group, int max_rows) {
    return kv_few_bytes(head_dim) + (kv_many_rows(group, max_rows) ? kv_many_bytes(head_dim) : 0);
}
// What a caller is told to bring: from 17 query rows of a KV head on with the part of many rows, so that
// it is room enough for prompts too
static_assert(kKvRowTile <= kKvFewRows, "never less than a call takes");
constexpr int64_t kv_workspace_bytes(int head_dim, int group, int max_rows) {
    return kv_few_bytes(head_dim) + ((int64_t)max_rows * group > kKvRowTile ? kv_many_bytes(head_dim) : 0);
}

hipError_t launch_kv_append(int head_dim, const KvArgs& b, const KvAppendArgs& a, hipStream_t s);
// max_rows: the caller's bound on a sequence's rows (chooses kernels only)
hipError_t launch_kv_attention(int head_dim, const KvArgs& b, const void* q, int64_t q_stride, void* out,
                               int64_t out_stride, float scale, int32_t max_rows, void* workspace, hipStream_t s);

}  // namespace hagemm
