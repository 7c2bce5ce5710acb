// Keys and values in the pool's KV pages, 4 bits each: appending a step's rows
// (with the position rotation) and attention over them.
//
// A row x of head_dim values is held as lo + step * code, code 0..15, with one
// 32-bit word per row (bf16 step low, bf16 lo high).  16 consecutive tokens of
// one head's keys or values are one slab: 8 head_dim bytes of codes, 16 words.
// Both code layouts put the 16 x head_dim codes of a slab in the order in which
// the 64 lanes of a matrix operation want them, so that one contiguous load per
// lane fetches a lane's codes of the whole slab:
//   keys    [token][head_dim / 2 bytes]: a lane has one token and a quarter of its values;
//           in each 32-bit word of 8 values, nibble k is value 2 k, nibble k + 4 value 2 k + 1
//   values  [i = 16][token pair][4 values][token of the pair]: a lane has head_dim / 16
//           values of four consecutive tokens, two tokens side by side in each 32-bit word
// No byte is shared by two tokens' codes, so tokens can be appended one by one.
#include <algorithm>
#include <type_traits>

#include "common.h"
#include "kv.h"

namespace hagemm {
namespace {

typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));
typedef float f32x2_t __attribute__((ext_vector_type(2)));

// ---------------------------------------------------------------- sequences

// Rows and tokens of sequence s, whatever the arrays hold: rows [r0, r0 + rows) of the
// batch, len tokens in the cache, both inside their buffers.
struct KvSeq {
    int r0, rows, len;
};
__device__ __forceinline__ KvSeq kv_seq(const KvArgs& b, int s) {
    KvSeq q;
    q.r0 = min(max(b.row_start[s], 0), b.n_rows);
    q.rows = min(max(b.row_start[s + 1], q.r0), b.n_rows) - q.r0;
    q.len = min(max(b.ctx_len[s], 0), b.max_blocks * kKvBlock);
    return q;
}

// The table's entry for (sequence, block, slab); any number may stand there.
__device__ __forceinline__ const int32_t* kv_entry(const KvArgs& b, int s, int block, int slab) {
    return b.table + ((int64_t)s * b.max_blocks + block) * b.pages_per_block + slab / b.slabs_per_page;
}
__device__ __forceinline__ bool kv_page_ok(const KvArgs& b, int page) { return (uint32_t)page < (uint32_t)b.num_pages; }

// ---------------------------------------------------------------- append

__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
    return __builtin_bit_cast(uint32_t, __builtin_convertvector(f32x2_t{lo, hi}, bf16x2_t));
}
__device__ __forceinline__ u32x4 pack_row(const float (&x)[8]) {
    return u32x4{pack2(x[0], x[1]), pack2(x[2], x[3]), pack2(x[4], x[5]), pack2(x[6], x[7])};
}

// f over the N lanes (8, 16 or 32, aligned) that share a row, in every one of them
template <int N, class F>
__device__ __forceinline__ float row_reduce(float v, F f) {
    auto mov = [](float x, auto ctrl) {
        return __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(x), decltype(ctrl)::value, 0xf, 0xf, true));
    };
    v = f(v, mov(v, std::integral_constant<int, 0xB1>{}));    // quad_perm 1 0 3 2
    v = f(v, mov(v, std::integral_constant<int, 0x4E>{}));    // quad_perm 2 3 0 1
    v = f(v, mov(v, std::integral_constant<int, 0x141>{}));   // row_half_mirror
    if constexpr (N >= 16) v = f(v, mov(v, std::integral_constant<int, 0x140>{}));   // row_mirror
    if constexpr (N >= 32) v = f(v, __shfl_xor(v, 16, 64));
    return v;
}

// Rows of one head an append workgroup takes
constexpr int kv_append_rows(int head_dim) { return head_dim == 256 ? 8 : 16; }

constexpr int kSeqCache = 1024;   // row_start entries an append workgroup keeps in LDS

// One row of one head per D / 8 lanes, 8 values a lane.  A workgroup has 16 consecutive rows (8 of 256
// values) and, one after another, every blocks-th group of their heads (a head, of 64 values two), `blocks`
// workgroups sharing the rows, so that all have their share of the keys, which cost most; the next two
// groups' loads are in flight.  A slab's bytes then come from one workgroup, and meet in one L2 (one row of
// 16 heads a workgroup took 52 us for 2,286 rows of 32 + 2 x 32 heads of 128).  Query rows are turned in fp32.
// Key rows are turned in fp64 and rounded to bf16 (the key that an unquantised cache would hold) before
// they are quantised: a code then depends on the exact product only, not on how it was summed, and
// the quantisation itself works on bf16 values, whose halves, differences and quotients by
// a bf16 step are the same in any order of evaluation.
// Measured on MI355X: those 2,286 rows 37 us, 3.4 TB/s of rows and pages, about 300 vector instructions
// for 512 values of a key or value (30 us of them; its stores, or fp64, cost 2 us); 64
// decode rows of 32 + 2 x 8 heads 5 us, launch and three dependent reads.
template <int D>
__global__ __launch_bounds__(256, D == 128 ? 5 : 4) void kv_append_kernel(KvArgs b, KvAppendArgs a, int blocks) {
    constexpr int LPR = D / 8, RPB = kv_append_rows(D), HPB = 256 / LPR / RPB;
    __shared__ int rs[kSeqCache];
    const int n_cache = min(b.n_seqs + 1, kSeqCache);
    for (int i = threadIdx.x; i < n_cache; i += 256) rs[i] = b.row_start[i];
    __syncthreads();
    const int nq = a.q ? b.heads : 0;
    const int per_row = nq + 2 * b.kv_heads;
    const int c = threadIdx.x % LPR, g = threadIdx.x / LPR;
    const int groups = (per_row + HPB - 1) / HPB;
    const int t = (int)(blockIdx.x / blocks) * RPB + g % RPB;
    const int first = (int)(blockIdx.x % blocks);
    if (t >= b.n_rows) return;
    // the last sequence that starts at or before row t
    int lo = 0, hi = b.n_seqs;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        const int v = mid < n_cache ? rs[mid] : b.row_start[mid];
        if (v <= t) lo = mid; else hi = mid;
    }
    const int s = lo;
    const KvSeq sq = kv_seq(b, s);
    const int pos = sq.len - sq.rows + (t - sq.r0);
    if (t < sq.r0 || t >= sq.r0 + sq.rows || pos < 0 || pos >= b.max_blocks * kKvBlock) return;

    // this lane's angles: y is the partner's value, x -> x co + y si
    float co[8], si[8];
    const int half = a.rot >> 1;
    const bool turns = 8 * c < a.rot, second = !a.interleaved && 8 * c >= half;
    const int partner = second ? 8 * c - half : 8 * c + half;   // (pairs (i, i + rot / 2) only)
    if (turns) {
        const float* cs = a.cos_sin + (int64_t)pos * a.rot;
        if (a.interleaved) {
            const f32x4 c4 = *reinterpret_cast<const f32x4*>(cs + 4 * c);
            const f32x4 s4 = *reinterpret_cast<const f32x4*>(cs + half + 4 * c);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                co[i] = c4[i / 2];
                si[i] = i % 2 ? s4[i / 2] : -s4[i / 2];
            }
        } else {
            const int at = second ? partner : 8 * c;
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const f32x4 c4 = *reinterpret_cast<const f32x4*>(cs + at + 4 * j);
                const f32x4 s4 = *reinterpret_cast<const f32x4*>(cs + half + at + 4 * j);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    co[4 * j + i] = c4[i];
                    si[4 * j + i] = second ? s4[i] : -s4[i];
                }
            }
        }
    }

    // one head's row: kind 0 q, 1 k, 2 v; head h; its values, its partners' and its page
    struct Item {
        int kind, h, page;
        u32x4 x, y;
    };
    auto fetch = [&](int group, Item& it) {
        const int hh = HPB == 1 ? group : group * HPB + g / RPB;
        it.kind = hh >= per_row ? 3 : hh < nq ? 0 : hh < nq + b.kv_heads ? 1 : 2;
        if (it.kind == 3) return;
        it.h = it.kind == 0 ? hh : it.kind == 1 ? hh - nq : hh - nq - b.kv_heads;
        const bf16_t* src = static_cast<const bf16_t*>(it.kind == 0 ? a.q : it.kind == 1 ? a.k : a.v) +
                            t * (it.kind == 0 ? a.q_stride : it.kind == 1 ? a.k_stride : a.v_stride) + (int64_t)it.h * D;
        it.x = ld16(src + 8 * c);
        if (it.kind != 2 && turns && !a.interleaved) it.y = ld16(src + partner);
        if (it.kind != 0) it.page = *kv_entry(b, s, pos / kKvBlock, 2 * it.h + (it.kind == 2));
    };
    auto work = [&](const Item& it) {
        if (it.kind == 3) return;
        const int kind = it.kind, h = it.h;
        float x[8];
        unpack(it.x, x, bf16_t{});
        if (kind != 2 && turns) {
            float y[8];
            if (a.interleaved) {
#pragma unroll
                for (int i = 0; i < 8; ++i) y[i] = x[i ^ 1];
            } else {
                unpack(it.y, y, bf16_t{});
            }
            if (kind == 0) {
#pragma unroll
                for (int i = 0; i < 8; ++i) x[i] = x[i] * co[i] + y[i] * si[i];
            } else {
#pragma unroll
                for (int i = 0; i < 8; ++i) x[i] = (float)((double)x[i] * co[i] + (double)y[i] * si[i]);
            }
        }
        if (kind == 0) {
            st16(static_cast<bf16_t*>(a.q_out) + t * a.q_out_stride + (int64_t)h * D + 8 * c, pack_row(x));
            return;
        }
        if (kind == 1) unpack(pack_row(x), x, bf16_t{});
        // lo and step of the row; one with an infinity or NaN gets a NaN step, and reads back as NaN
        float mn = x[0], mx = x[0], bad = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            bad = fmaf(x[i], 0.f, bad);
            mn = fminf(mn, x[i]);
            mx = fmaxf(mx, x[i]);
        }
        mn = row_reduce<LPR>(mn, [](float u, float v) { return fminf(u, v); });
        mx = row_reduce<LPR>(mx, [](float u, float v) { return fmaxf(u, v); });
        bad = row_reduce<LPR>(bad, [](float u, float v) { return u + v; });
        // (halves are exact and cannot overflow: the slow way takes them where the range does)
        const uint32_t step_bits = bad == 0.f ? f32_to_bf16((mx * 0.5f - mn * 0.5f) / 7.5f) : 0x7FC0u;
        const uint32_t lo_bits = f32_to_bf16(mn);
        const float step = __uint_as_float(step_bits << 16), inv = __builtin_amdgcn_rcpf(step);
        float code[8], off = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float q = (x[i] - mn) * inv;
            code[i] = rintf(q);
            off = fmaxf(off, fabsf(q - code[i]));
            code[i] = fminf(code[i], 15.f);
        }
        // q is off by a few 2^-24: where a value is that near a border between two codes, where a
        // reciprocal or the row's range overflows (q is infinite there, and `off` leaves out its NaN) or the
        // step is 0 or NaN, by the quotient itself
        if (__ballot(!(off < 0.4999f) || !(inv < 1e30f) || !(mx - mn < INFINITY))) {
            const float half_step = step * 0.5f;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float q = rintf((x[i] * 0.5f - mn * 0.5f) / half_step);
                code[i] = half_step > 0.f ? fminf(fmaxf(q, 0.f), 15.f) : 0.f;
            }
        }
        void* back = kind == 1 ? a.k_out : a.v_out;
        if (back) {
            float z[8];
            const float base = __uint_as_float(lo_bits << 16);
#pragma unroll
            for (int i = 0; i < 8; ++i) z[i] = fmaf(step, code[i], base);
            st16(static_cast<bf16_t*>(back) + t * (kind == 1 ? a.k_out_stride : a.v_out_stride) + (int64_t)h * D + 8 * c,
                 pack_row(z));
        }
        const int slab = 2 * h + (kind == 2), r = pos % kKvBlock;
        if (!kv_page_ok(b, it.page)) return;   // a page outside the pool: the row is not kept
        uint8_t* at = b.pages + it.page * b.page_bytes + (slab % b.slabs_per_page) * kv_slab_bytes(D);
        if (kind == 1) {
            uint32_t w = 0;
#pragma unroll
            for (int k = 0; k < 4; ++k)
                w |= (uint32_t)(int)code[2 * k] << (4 * k) | (uint32_t)(int)code[2 * k + 1] << (4 * k + 16);
            *reinterpret_cast<uint32_t*>(at + r * (D / 2) + 4 * c) = w;
        } else {
            constexpr int NH = D / 64;
#pragma unroll
            for (int n = 0; n < 2; ++n) {
                uint32_t w = 0;
#pragma unroll
                for (int k = 0; k < 4; ++k) w |= (uint32_t)(int)code[4 * n + k] << (4 * k);
                const int q4 = 2 * c + n;
                *reinterpret_cast<uint16_t*>(at + (q4 / NH) * (D / 2) + (r / 2) * (D / 16) + (q4 % NH) * 4 + (r % 2) * 2) =
                    (uint16_t)w;
            }
        }
        if (c == 0) *reinterpret_cast<uint32_t*>(at + 8 * D + 4 * r) = step_bits | lo_bits << 16;
    };
    Item it[3];
    fetch(first, it[0]);
    if (first + blocks < groups) fetch(first + blocks, it[1]);
    for (int i = first; i < groups; i += 3 * blocks) {
#pragma unroll
        for (int j = 0; j < 3; ++j) {
            if (i + j * blocks >= groups) break;
            if (i + (j + 2) * blocks < groups) fetch(i + (j + 2) * blocks, it[(j + 2) % 3]);
            work(it[j]);
        }
    }
}

// ---------------------------------------------------------------- attention: the work's cut

// The work is a line of steps (32 tokens each) of all segments, one after another: a segment is
// a row tile (rb query rows of one KV head) of a sequence, its steps those of the sequence's
// tokens, tiles and heads in turn (heads innermost).  Workers (waves or workgroups) take equal
// pieces of the line, so that short and long sequences keep all of them busy alike; a segment
// that a border cuts leaves partial results, which a second launch joins.  Every workgroup
// finds its piece from the device's lengths, so the launch does not depend on them (a captured
// call follows them).
enum KvClass { kKvAll = 0, kKvFew = 1, kKvMany = 2 };   // sequences: all, of at most kKvFewRows query rows, of more

struct KvCut {
    int rb_shift, cls, workers;
};

__device__ __forceinline__ int kv_steps(int tokens) { return (tokens + 31) >> 5; }

// (row tile, head) pairs of a sequence, and steps of each (at least one: rows without a token
// have to be written too)
__device__ __forceinline__ int kv_pairs(const KvArgs& b, const KvCut& cut, const KvSeq& q) {
    const int64_t rows = (int64_t)q.rows * b.group;
    if ((cut.cls == kKvFew && rows > kKvFewRows) || (cut.cls == kKvMany && rows <= kKvFewRows)) return 0;
    return (int)((rows + (1 << cut.rb_shift) - 1) >> cut.rb_shift) * b.kv_heads;
}
__device__ __forceinline__ int kv_seg_steps(const KvSeq& q) { return max(1, kv_steps(q.len)); }

// Tiles of many rows see less the earlier their rows are, and a prompt from its first token half of
// the tokens in the mean.  So the line counts a tile's steps up to what the last tile of its band sees:
// bands of four tiles, or of more where a sequence would have more than 64 (a place on the line is
// found a band a lane).  Two steps more stand for what a tile costs beside its tokens (its q, its first
// pages, its sums).  A prompt of 2,048 rows: 97 us counting all tokens, 95 with bands, 91 with the two.
struct KvBands {
    int tiles, band;
    __device__ __forceinline__ KvBands(int pairs, int kv_heads) {
        tiles = pairs / kv_heads;
        band = 4;
        while (band * 64 < tiles) band *= 2;
    }
    __device__ __forceinline__ int end(int tile) const { return min(tiles, tile + band); }
    // steps of a tile in the band that ends before tile `end`
    __device__ __forceinline__ int steps(const KvArgs& b, const KvCut& cut, const KvSeq& q, int end) const {
        const int rows = q.rows * b.group;
        return 2 + max(1, kv_steps(q.len - q.rows + 1 + (min(rows, end << cut.rb_shift) - 1) / b.group));
    }
};

// Inclusive sums over the wave's lanes.
template <int CTRL, int ROWS_MASK>
__device__ __forceinline__ int dpp0(int v) {
    return __builtin_amdgcn_update_dpp(0, v, CTRL, ROWS_MASK, 0xf, ROWS_MASK == 0xf);
}
__device__ __forceinline__ int wave_scan(int v) {
    v += dpp0<0x111, 0xf>(v);   // row_shr 1, 2, 4, 8
    v += dpp0<0x112, 0xf>(v);
    v += dpp0<0x114, 0xf>(v);
    v += dpp0<0x118, 0xf>(v);
    v += dpp0<0x142, 0xa>(v);   // row_bcast 15, 31
    v += dpp0<0x143, 0xc>(v);
    return v;
}
template <int CTRL, int ROWS_MASK>
__device__ __forceinline__ int64_t dpp0(int64_t v) {
    const uint32_t lo = (uint32_t)dpp0<CTRL, ROWS_MASK>((int)(uint32_t)v);
    return (int64_t)((uint64_t)lo | (uint64_t)(uint32_t)dpp0<CTRL, ROWS_MASK>((int)(v >> 32)) << 32);
}
__device__ __forceinline__ int64_t wave_scan(int64_t v) {
    v += dpp0<0x111, 0xf>(v);
    v += dpp0<0x112, 0xf>(v);
    v += dpp0<0x114, 0xf>(v);
    v += dpp0<0x118, 0xf>(v);
    v += dpp0<0x142, 0xa>(v);
    v += dpp0<0x143, 0xc>(v);
    return v;
}

// The line, as a workgroup keeps it: before[i] = steps before sequence i m (m sequences a
// thread), before[256] all of them.
struct KvLine {
    int64_t before[257];
    int64_t sums[4];
};

template <bool BANDS>
__device__ __forceinline__ void kv_line(const KvArgs& b, const KvCut& cut, KvLine& line) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int m = (b.n_seqs + 255) >> 8;
    const int s0 = threadIdx.x * m, s1 = min(s0 + m, b.n_seqs);
    int64_t mine = 0;
    for (int s = s0; s < s1; ++s) {
        const KvSeq q = kv_seq(b, s);
        const int pairs = kv_pairs(b, cut, q);
        if (BANDS) {
            const KvBands n(pairs, b.kv_heads);
            for (int tile = 0, end; tile < n.tiles; tile = end) {
                end = n.end(tile);
                mine += (int64_t)(end - tile) * b.kv_heads * n.steps(b, cut, q, end);
            }
        } else {
            mine += (int64_t)pairs * kv_seg_steps(q);
        }
    }
    int64_t in = wave_scan(mine);
    if (lane == 63) line.sums[wave] = in;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < 3; ++w)
        if (w < wave) in += line.sums[w];
    line.before[threadIdx.x] = in - mine;
    if (threadIdx.x == 255) line.before[256] = in;
    __syncthreads();
}

__device__ __forceinline__ int64_t uniform64(int64_t v) {
    return (int64_t)((uint64_t)(uint32_t)__builtin_amdgcn_readfirstlane((int)(v & 0xFFFFFFFF)) |
                     (uint64_t)(uint32_t)__builtin_amdgcn_readfirstlane((int)(v >> 32)) << 32);
}

__device__ __forceinline__ int64_t lane64(int64_t v, int lane) {
    return (int64_t)((uint64_t)(uint32_t)__builtin_amdgcn_readlane((int)(v & 0xFFFFFFFF), lane) |
                     (uint64_t)(uint32_t)__builtin_amdgcn_readlane((int)(v >> 32), lane) << 32);
}

// Where a worker's piece begins: total steps in equal pieces, the first total % workers one longer.
struct KvPieces {
    int64_t size, longer;
    int workers;
    __device__ __forceinline__ KvPieces(int64_t total, int most) {
        workers = (int)min(total, (int64_t)most);
        // (at most a few thousand workers: the quotient fits a double exactly enough, then is put right)
        size = workers > 0 ? (int64_t)((double)total / workers) : 0;
        if (size * workers > total) --size;
        if (workers > 0 && total - size * workers >= workers) ++size;
        longer = total - size * workers;
    }
    __device__ __forceinline__ int64_t at(int w) const { return w * size + min((int64_t)w, longer); }
    // the worker whose piece holds step x
    __device__ __forceinline__ int holder(int64_t x) const {
        const int64_t first = longer * (size + 1);
        int w = x < first ? (int)((double)x / (double)(size + 1)) : (int)(longer + (int64_t)((double)(x - first) / (double)size));
        w = min(w, workers - 1);
        if (at(w) > x) --w;
        if (w + 1 < workers && at(w + 1) <= x) ++w;
        return w;
    }
};

// A place on the line: pair `pair` of sequence s, `off` of its `steps` steps in; pairs below `same`
// have as many.  All uniform over the wave.
template <bool BANDS>
struct KvPlace {
    int s, pair, pairs, off, steps, same;
    KvSeq q;

    __device__ __forceinline__ void band(const KvArgs& b, const KvCut& cut, int tile) {
        const KvBands n(pairs, b.kv_heads);
        const int end = n.end(tile);
        same = end * b.kv_heads;
        steps = n.steps(b, cut, q, end);
    }
    __device__ __forceinline__ void enter(const KvArgs& b, const KvCut& cut, int seq) {
        s = seq;
        q = kv_seq(b, s);
        pairs = kv_pairs(b, cut, q);
        pair = 0;
        if (BANDS) {
            band(b, cut, 0);
        } else {
            same = pairs;
            steps = kv_seg_steps(q);
        }
    }
    // pos below the line's end
    __device__ __forceinline__ void seek(const KvArgs& b, const KvCut& cut, const KvLine& line, int64_t pos) {
        const int lane = threadIdx.x & 63;
        // the last of the 256 threads' sequences that begin at or before pos
        int last = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) last += __popcll(__ballot(line.before[64 * i + lane] <= pos));
        const int m = (b.n_seqs + 255) >> 8;
        int64_t left = pos - uniform64(line.before[last - 1]);
        enter(b, cut, (last - 1) * m);
        for (;;) {
            if (BANDS) {
                // a band a lane
                const KvBands n(pairs, b.kv_heads);
                const int tile = lane * n.band, end = n.end(tile);
                const int64_t upto = wave_scan(tile < n.tiles ? (int64_t)(end - tile) * b.kv_heads * n.steps(b, cut, q, end) : 0);
                const int at = __popcll(__ballot(upto <= left));
                if (at < 64) {
                    left -= at ? lane64(upto, at - 1) : 0;
                    pair = at * n.band * b.kv_heads;
                    band(b, cut, at * n.band);
                    break;
                }
                left -= lane64(upto, 63);
            } else {
                if (left < (int64_t)pairs * steps) break;
                left -= (int64_t)pairs * steps;
            }
            enter(b, cut, s + 1);
        }
        int in = (int)((double)left / steps);
        if ((int64_t)in * steps > left) --in;
        if (left - (int64_t)in * steps >= steps) ++in;
        pair = __builtin_amdgcn_readfirstlane(pair + in);
        off = __builtin_amdgcn_readfirstlane((int)(left - (int64_t)in * steps));
    }
    // the segment after this one (one with steps must follow)
    __device__ __forceinline__ void next(const KvArgs& b, const KvCut& cut) {
        off = 0;
        if (++pair < same) return;
        if (BANDS && pair < pairs) {
            band(b, cut, pair / b.kv_heads);
            return;
        }
        do enter(b, cut, s + 1);
        while (pairs == 0);
    }
};

// ---------------------------------------------------------------- attention: one wave

// The two bf16 halves 16 + code of nibble k of both 16-bit halves of w: a nibble in the top
// four bits of bf16's seven mantissa bits counts ones above 16, so the codes need no
// conversion, only their place.  mask and ones: 0x00780078 and 0x41804180, in registers (a
// three-operand and-or takes no constants of its own).
struct CodeConst {
    uint32_t mask = 0x00780078u, ones = 0x41804180u;
    __device__ __forceinline__ CodeConst() { asm volatile("" : "+v"(mask), "+v"(ones)); }
};
__device__ __forceinline__ uint32_t code_pair(const CodeConst& c, uint32_t w, int k) {
    const uint32_t s = k == 0 ? w << 3 : k == 1 ? w >> 1 : k == 2 ? w >> 5 : w >> 9;
    return (s & c.mask) | c.ones;
}

// Over the four lanes that share a query row (lane % 16).
__device__ __forceinline__ float max_lg(float v) {
    auto a = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    v = fmaxf(__uint_as_float(a[0]), __uint_as_float(a[1]));
    a = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    return fmaxf(__uint_as_float(a[0]), __uint_as_float(a[1]));
}
__device__ __forceinline__ float sum_lg(float v) {
    auto a = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    v = __uint_as_float(a[0]) + __uint_as_float(a[1]);
    a = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    return __uint_as_float(a[0]) + __uint_as_float(a[1]);
}

// Over the two lanes that share a query row (lane % 32).
__device__ __forceinline__ float max_hg(float v) {
    const auto a = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    return fmaxf(__uint_as_float(a[0]), __uint_as_float(a[1]));
}
__device__ __forceinline__ float sum_hg(float v) {
    const auto a = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    return __uint_as_float(a[0]) + __uint_as_float(a[1]);
}

typedef float f32x16_t __attribute__((ext_vector_type(16)));
__device__ __forceinline__ f32x16_t mma32(const u32x4& a, const u32x4& b, f32x16_t c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0,
                                                   0);
}

// A wave's place for one step in LDS: the codes of two slabs of keys and two of values, then
// their words.
template <int D>
struct KvStage {
    static constexpr int kCodes = 32 * D, kBytes = kCodes + 256;
};

// Sum over the lanes of a 16-lane row that are a multiple of ROWS apart.
template <int ROWS>
__device__ __forceinline__ float sum_cols(float v) {
    auto ror = [](float x, auto n) {
        return __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(x), 0x120 + decltype(n)::value, 0xf, 0xf, true));
    };
    if constexpr (ROWS <= 8) v += ror(v, std::integral_constant<int, 8>{});
    if constexpr (ROWS <= 4) v += ror(v, std::integral_constant<int, 4>{});
    if constexpr (ROWS <= 2) v += ror(v, std::integral_constant<int, 2>{});
    if constexpr (ROWS <= 1) v += ror(v, std::integral_constant<int, 1>{});
    return v;
}
template <int ROWS>
__device__ __forceinline__ float max_cols(float v) {
    auto ror = [](float x, auto n) {
        return __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(x), 0x120 + decltype(n)::value, 0xf, 0xf, true));
    };
    if constexpr (ROWS <= 8) v = fmaxf(v, ror(v, std::integral_constant<int, 8>{}));
    if constexpr (ROWS <= 4) v = fmaxf(v, ror(v, std::integral_constant<int, 4>{}));
    if constexpr (ROWS <= 2) v = fmaxf(v, ror(v, std::integral_constant<int, 2>{}));
    if constexpr (ROWS <= 1) v = fmaxf(v, ror(v, std::integral_constant<int, 1>{}));
    return v;
}

// A wave's query rows against tokens, 32 at a time.  A matrix operation has 16 columns for
// query rows; where there are fewer rows, each takes COLS = 16 / ROWS columns, lane (li, lg) =
// (lane % 16, lane / 16) being in column li of row li % ROWS.  The columns of a row have the
// same scores and share the work on them: SUB of them take every SUB-th part of the tokens (the
// others' weights are zeros in their column), and with SPLIT each of those is a pair, one for
// either half of the weights; the columns' outputs are summed at the end.
//   scores   S^T = K Q^T: matrix operations on the codes themselves (16 + code, exact in bf16);
//            a lane gets tokens 4 lg .. 4 lg + 3 of both slabs and picks its own, then s = step *
//            (acc - 16 sum(q)) + lo * sum(q), all fp32
//   weights  p = 2^(c (s - m)); m is raised, and everything summed so far scaled down, only
//            when a score passes it by more than 8 / c (the sums' scale needs no closer bound)
//   output   O^T += V^T P'^T with P' = p step in two bf16 halves (high and the rest, so its
//            error is 2^-17) and V's codes as 16 + code; z = sum p (lo - 16 step) takes the
//            rest.  A lane gets the values 4 lg D / 16 .. + D / 4.
template <int D, int SUB, bool SPLIT>
struct KvWave {
    static constexpr int W = D / 32, NE = D / 16, COLS = SPLIT ? 2 * SUB : SUB, ROWS = 16 / COLS, NEL = 8 / SUB;
    uint32_t q[W][4];
    float qsum;
    f32x4 o[NE];
    float m, l, z;
    int limit;          // tokens this lane's row sees
    int limit_all;      // tokens every row of the tile sees
    int h, s, last_block;
    CodeConst cc;

    static __device__ __forceinline__ int row() { return (threadIdx.x & 15) % ROWS; }
    static __device__ __forceinline__ int col() { return (threadIdx.x & 15) / ROWS; }
    static __device__ __forceinline__ int part() { return SPLIT ? col() % 2 : 0; }      // 1: the weights' low half
    static __device__ __forceinline__ int sub() { return SPLIT ? col() / 2 : col(); }

    // ROWS query rows from row0 on, of one KV head of sequence seq
    __device__ __forceinline__ void load_q(const KvArgs& b, int seq, const KvSeq& sq, int head, const bf16_t* qp,
                                           int64_t stride, int row0) {
        const int lg = (threadIdx.x & 63) >> 4;
        const int rows = sq.rows * b.group;
        const int r = row0 + row();
        h = head;
        s = seq;
        last_block = (sq.len + kKvBlock - 1) / kKvBlock - 1;
        if (r < rows) {
            const bf16_t* p = qp + (int64_t)(sq.r0 + r / b.group) * stride +
                              (int64_t)(h * b.group + r % b.group) * D + lg * (D / 4);
#pragma unroll
            for (int i = 0; i < W; ++i) {
                const u32x4 v = ld16(p + 8 * i);
#pragma unroll
                for (int j = 0; j < 4; ++j) q[i][j] = v[j];
            }
        } else {
#pragma unroll
            for (int i = 0; i < W; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) q[i][j] = 0;
        }
        const int first = sq.len - sq.rows + 1;   // tokens the sequence's first row sees
        limit = r < rows ? first + r / b.group : 0;
        limit_all = first + row0 / b.group;
        m = -INFINITY;
        l = z = 0.f;
#pragma unroll
        for (int e = 0; e < NE; ++e) o[e] = f32x4{0.f, 0.f, 0.f, 0.f};
    }

    // One step: kc and vc the lane's codes of two slabs, kw and vw the words of its NEL tokens.
    __device__ __forceinline__ void step(const uint32_t (&kc)[2][W], const uint32_t (&vc)[2][W], const uint32_t (&kw)[NEL],
                                         const uint32_t (&vw)[NEL], int tok0, int bad, float c, float raise) {
        const int lg = (threadIdx.x & 63) >> 4, sb = sub();
        f32x4 sc[2];
#pragma unroll
        for (int a = 0; a < 2; ++a) {
            const float init = -16.f * qsum;
            sc[a] = f32x4{init, init, init, init};
        }
#pragma unroll
        for (int i = 0; i < W; ++i)
#pragma unroll
            for (int a = 0; a < 2; ++a) {
                u32x4 kf, qf;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    kf[j] = code_pair(cc, kc[a][i], j);
                    qf[j] = q[i][j];
                }
                sc[a] = mma_step(kf, qf, sc[a], bf16_t{});
            }
        float x[NEL], st[NEL], zp[NEL];
#pragma unroll
        for (int k = 0; k < NEL; ++k) {
            if constexpr (SUB == 1) x[k] = sc[k / 4][k % 4];
            else if constexpr (SUB == 2) x[k] = sb ? sc[1][k] : sc[0][k];
            else if constexpr (SUB == 4) x[k] = sb & 2 ? (sb & 1 ? sc[1][2 + k] : sc[1][k]) : (sb & 1 ? sc[0][2 + k] : sc[0][k]);
            else x[k] = sb & 4 ? (sb & 2 ? (sb & 1 ? sc[1][3] : sc[1][2]) : (sb & 1 ? sc[1][1] : sc[1][0]))
                               : (sb & 2 ? (sb & 1 ? sc[0][3] : sc[0][2]) : (sb & 1 ? sc[0][1] : sc[0][0]));
            x[k] = fmaf(x[k], bf16_lo(kw[k]), bf16_hi(kw[k]) * qsum);
            st[k] = bf16_lo(vw[k]);
            zp[k] = fmaf(-16.f, st[k], bf16_hi(vw[k]));
        }
        if (__builtin_expect(tok0 + 32 > limit_all || bad, 0)) {
            // tokens that a row does not see count nothing, whatever the pages hold there
#pragma unroll
            for (int k = 0; k < NEL; ++k) {
                const int a = (sb * NEL + k) / 4, tok = tok0 + 16 * a + 4 * lg + (sb * NEL + k) % 4;
                if (tok >= limit || ((bad >> a) & 1)) {
                    x[k] = -INFINITY;
                    st[k] = 0.f;
                    zp[k] = 0.f;
                }
            }
        }
        float top = x[0];
#pragma unroll
        for (int k = 1; k < NEL; ++k) top = fmaxf(top, x[k]);
        if (__ballot(top > m + raise)) {
            const float mn = fmaxf(m, max_cols<ROWS>(max_lg(top)));
            const float al = mn == -INFINITY ? 1.f : __builtin_amdgcn_exp2f(c * (m - mn));
            m = mn;
            l *= al;
            z *= al;
#pragma unroll
            for (int e = 0; e < NE; ++e)
#pragma unroll
                for (int i = 0; i < 4; ++i) o[e][i] *= al;
        }
        const float ref = m == -INFINITY ? 0.f : -c * m;
        float w[NEL];
#pragma unroll
        for (int k = 0; k < NEL; ++k) {
            const float p = __builtin_amdgcn_exp2f(fmaf(x[k], c, ref));
            l += p;
            z = fmaf(p, zp[k], z);
            w[k] = p * st[k];
        }
        // the weights' halves, at this column's tokens
        u32x4 ph{0, 0, 0, 0}, pl{0, 0, 0, 0};
        if constexpr (NEL == 1) {
            const uint32_t hi = pack2(w[0], 0.f), lo = pack2(w[0] - bf16_lo(hi), 0.f);
            const int at = 16 * (sb & 1);
            const uint32_t a = (SPLIT && part() ? lo : hi) << at, b = lo << at;
#pragma unroll
            for (int y = 0; y < 4; ++y) {
                ph[y] = sb >> 1 == y ? a : 0;
                if constexpr (!SPLIT) pl[y] = sb >> 1 == y ? b : 0;
            }
        } else {
#pragma unroll
            for (int k = 0; k < NEL; k += 2) {
                const uint32_t hi = pack2(w[k], w[k + 1]);
                const uint32_t lo = pack2(w[k] - bf16_lo(hi), w[k + 1] - bf16_hi(hi));
                const uint32_t a = SPLIT && part() ? lo : hi;
#pragma unroll
                for (int y = 0; y < 4; ++y) {
                    if (y % (NEL / 2) != k / 2) continue;
                    const bool mine = SUB == 1 || sb == y / (NEL / 2);
                    ph[y] = mine ? a : 0;
                    if constexpr (!SPLIT) pl[y] = mine ? lo : 0;
                }
            }
        }
        u32x4 vf[NE];
#pragma unroll
        for (int e = 0; e < NE; ++e) {
            constexpr int NH = W / 2;
#pragma unroll
            for (int a = 0; a < 2; ++a)
#pragma unroll
                for (int p = 0; p < 2; ++p) vf[e][2 * a + p] = code_pair(cc, vc[a][p * NH + e / 4], e % 4);
            o[e] = mma_step(vf[e], ph, o[e], bf16_t{});
            if constexpr (!SPLIT) {
                // (a block behind, so that no operation waits for the one before it)
                if (e > 0) o[e - 1] = mma_step(vf[e - 1], pl, o[e - 1], bf16_t{});
            }
        }
        if constexpr (!SPLIT) o[NE - 1] = mma_step(vf[NE - 1], pl, o[NE - 1], bf16_t{});
    }

    // Steps first .. end - 1.  Their slabs go straight to LDS, two steps ahead of the one at work
    // (lds0 and lds1 in turn), so that the loads in flight take no registers: a step is read into
    // registers as a whole, and its place given to the step after the next.
    __device__ __forceinline__ void run(const KvArgs& b, uint8_t* lds0, uint8_t* lds1, int first, int end, float c) {
        const int lane = threadIdx.x & 63, li = lane & 15, lg = lane >> 4;
        const int n = end - first;
        if (n <= 0) return;
        const float raise = 8.f / c;
        const int ks = 2 * h, vs = 2 * h + 1;
        const int64_t koff = (int64_t)(ks % b.slabs_per_page) * kv_slab_bytes(D);
        const int64_t voff = (int64_t)(vs % b.slabs_per_page) * kv_slab_bytes(D);
        constexpr int kCodes = KvStage<D>::kCodes, kLoads = kCodes / 1024 + 1;
        // lane 4 j + x: page of slab x (keys 0, 1, values 0, 1) of step j of 16
        auto pages = [&](int j0) {
            const int j = j0 + (lane >> 2), blk = 2 * (first + j) + (lane & 1);
            return j < n && blk <= last_block ? *kv_entry(b, s, blk, lane & 2 ? vs : ks) : -1;
        };
        // a lane's word of slab lg
        const int64_t word_at = (lg < 2 ? koff : voff) + 8 * D + li * 4;
        // bit a of the result: slab a has no page
        auto load = [&](int pg, int word_page, int j, uint8_t* to) {
            const uint8_t* at[4];
            int bad = 0;
#pragma unroll
            for (int x = 0; x < 4; ++x) {
                const int page = __builtin_amdgcn_readlane(pg, 4 * j + x);
                const bool ok = kv_page_ok(b, page);
                bad |= !ok << (x & 1);
                at[x] = b.pages + (ok ? page : 0) * b.page_bytes + (x < 2 ? koff : voff);
            }
            if constexpr (D == 64) {
                // two slabs a load, in order; a lane's codes of slab x are 8 bytes
#pragma unroll
                for (int i = 0; i < 2; ++i)
                    global_load_lds16((lane < 32 ? at[2 * i] : at[2 * i + 1]) + (lane & 31) * 16, to + 1024 * i);
            } else {
                // each lane its own codes, 16 bytes at a time
#pragma unroll
                for (int x = 0; x < 4; ++x)
#pragma unroll
                    for (int i = 0; i < D / 128; ++i)
                        global_load_lds16(at[x] + li * (D / 2) + lg * (D / 8) + 16 * i, to + (x * (D / 128) + i) * 1024);
            }
            global_load_lds4(b.pages + (kv_page_ok(b, word_page) ? word_page : 0) * b.page_bytes + word_at, to + kCodes);
            return bad;
        };
        // a lane's tokens in a step, as word numbers of the keys' (values') 32
        const int sb = sub(), word = (sb * NEL) / 4 * 16 + 4 * lg + (sb * NEL) % 4;
        auto read = [&](const uint8_t* from, uint32_t (&kc)[2][W], uint32_t (&vc)[2][W], uint32_t (&kw)[NEL],
                        uint32_t (&vw)[NEL]) {
#pragma unroll
            for (int x = 0; x < 4; ++x) {
                uint32_t (&d)[W] = x < 2 ? kc[x & 1] : vc[x & 1];
                if constexpr (D == 64) {
                    const u32x2 u = *reinterpret_cast<const u32x2*>(from + x * 512 + li * 32 + lg * 8);
                    d[0] = u[0];
                    d[1] = u[1];
                } else {
#pragma unroll
                    for (int i = 0; i < D / 128; ++i) {
                        const u32x4 u = ld16(from + (x * (D / 128) + i) * 1024 + lane * 16);
#pragma unroll
                        for (int y = 0; y < 4; ++y) d[4 * i + y] = u[y];
                    }
                }
            }
            const uint32_t* w = reinterpret_cast<const uint32_t*>(from + kCodes) + word;
#pragma unroll
            for (int k = 0; k < NEL; ++k) {
                kw[k] = w[k / 4 * 16 + k % 4];
                vw[k] = w[32 + k / 4 * 16 + k % 4];
            }
        };
        auto page_of_word = [&](int pg, int j) { return __builtin_amdgcn_ds_bpermute(4 * (4 * j + lg), pg); };
        int pg = pages(0), pg_next = -1;
        int bad[2];
        bad[0] = load(pg, page_of_word(pg, 0), 0, lds0);
        bad[1] = n > 1 ? load(pg, page_of_word(pg, 1), 1, lds1) : 0;
        qsum = 0.f;
#pragma unroll
        for (int i = 0; i < W; ++i)
#pragma unroll
            for (int y = 0; y < 4; ++y) qsum += bf16_lo(q[i][y]) + bf16_hi(q[i][y]);
        qsum = sum_lg(qsum);
#pragma unroll 1
        for (int j = 0; j < n; j += 2) {
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                if (j + x >= n) break;
                // this step's loads have landed (of the ones after them, the next step's alone are out)
                if (j + x + 1 < n) wait_vmcnt<kLoads>();
                else wait_vmcnt<0>();
                landed();
                uint32_t kc[2][W], vc[2][W], kw[NEL], vw[NEL];
                read(x ? lds1 : lds0, kc, vc, kw, vw);
                const int bad_now = bad[x];
                if (j + x + 2 < n) {
                    if (((j + x + 2) & 15) == 0) pg = pg_next;
                    const int wp = page_of_word(pg, (j + x + 2) & 15);
                    wait_lgkm0();   // the step is in registers: its place is free
                    if (((j + x) & 15) == 0) pg_next = pages(j + x + 16);
                    bad[x] = load(pg, wp, (j + x + 2) & 15, x ? lds1 : lds0);
                }
                step(kc, vc, kw, vw, 32 * (first + j + x), bad_now, c, raise);
            }
        }
    }

    // the sums over a row's lanes and columns
    __device__ __forceinline__ void finish() {
        if (part()) l = z = 0.f;   // (the other half's column has counted them)
        l = sum_cols<ROWS>(sum_lg(l));
        z = sum_cols<ROWS>(sum_lg(z));
#pragma unroll
        for (int e = 0; e < NE; ++e)
#pragma unroll
            for (int i = 0; i < 4; ++i) o[e][i] = sum_cols<ROWS>(o[e][i]);
    }

    // the row's results as a part: sums and (m, l)
    __device__ __forceinline__ void put_part(float* p, float* ml) const {
        const int lg = (threadIdx.x & 63) >> 4;
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int e = 0; e < NE; e += 4)
                *reinterpret_cast<f32x4*>(p + (4 * lg + i) * NE + e) =
                    f32x4{o[e][i] + z, o[e + 1][i] + z, o[e + 2][i] + z, o[e + 3][i] + z};
        if (lg == 0) {
            ml[0] = m;
            ml[1] = l;
        }
    }

    // the row's results, divided, to the output
    __device__ __forceinline__ void store(bf16_t* out) const {
        const int lg = (threadIdx.x & 63) >> 4;
        const float inv = l == 0.f ? 0.f : 1.f / l;   // a row that sees no token is zero
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int e = 0; e < NE; e += 4) {
                u32x2 v;
                v[0] = pack2((o[e][i] + z) * inv, (o[e + 1][i] + z) * inv);
                v[1] = pack2((o[e + 2][i] + z) * inv, (o[e + 3][i] + z) * inv);
                *reinterpret_cast<u32x2*>(out + (4 * lg + i) * NE + e) = v;
            }
    }
};

// What the sums of a part (of scale m, weight l) count for at scale top >= m.  A part without
// tokens has m = -inf and sums of zero; a part of NaN scores m = -inf and l = NaN.
__device__ __forceinline__ float part_factor(float m, float l, float top, float c) {
    return m == -INFINITY ? (l == 0.f ? 0.f : 1.f) : __builtin_amdgcn_exp2f(c * (m - top));
}

// Where results go: the output, or (a segment cut by a border) the workspace: an entry per
// worker and its `last` once more, then [2 workers][rb][D] sums and [2 workers][rb][2] (m, l).  A worker has at most two
// cut segments: one that began before its piece (slot 2 w) and one that ends after it (2 w + 1).
struct KvOut {
    bf16_t* out;
    int64_t stride;
    uint8_t* ws;
    int workers;    // the launch's, which place the parts
};
// The segment that begins in a worker's piece and ends after it: its parts are this worker's
// (first) to last's; where the four waves of a workgroup are all inside the segment, their
// joined part is the first one's.  last = -1: no such segment.
struct KvMerge {
    int last, row0, rows, r0, h;
    int inside0, inside1;           // workgroups [inside0, inside1) have one joined part each
    int pad;
};
static_assert(sizeof(KvMerge) == 32, "workspace layout");

__device__ __forceinline__ void put_merge(const KvOut& w, int worker, const KvMerge& e) {
    reinterpret_cast<KvMerge*>(w.ws)[worker] = e;
    reinterpret_cast<int*>(w.ws + (int64_t)w.workers * sizeof(KvMerge))[worker] = e.last;
}
__device__ __forceinline__ float* part_base(const KvOut& w) {
    return reinterpret_cast<float*>(w.ws + (int64_t)w.workers * (sizeof(KvMerge) + 4));
}
template <int D>
__device__ __forceinline__ float* part_row(const KvOut& w, int rb, int slot, int r) {
    return part_base(w) + ((int64_t)slot * rb + r) * D;
}
template <int D>
__device__ __forceinline__ float* part_ml(const KvOut& w, int rb, int slot, int r) {
    return part_base(w) + (int64_t)2 * w.workers * rb * D + ((int64_t)slot * rb + r) * 2;
}

template <int D>
__device__ __forceinline__ bf16_t* out_row(const KvArgs& b, const KvOut& w, int r0, int h, int r) {
    return w.out + (int64_t)(r0 + r / b.group) * w.stride + (int64_t)(h * b.group + r % b.group) * D;
}

// Few query rows.  Workers are waves, each with all of its piece's segments by itself; where a
// whole workgroup's piece is inside one segment its waves' sums meet in LDS, so that long
// sequences leave a part a workgroup.  Bound by reading the cache once, and by the latency of a wave's
// two steps in flight: measured on MI355X, 64 requests of about 2,050 tokens (32 heads over 8 of 128) 40 us,
// 3.6 TB/s of pages; 192 of 129 to 552 tokens, 32 KV heads with a query head each, 68 us, 4.1 TB/s; one of
// 131,071 tokens 36 us, 4 TB/s; a lone one of 1,000 tokens 7.5 us, of which 3 us are finding its piece.
template <int D, int SUB, bool SPLIT>
__device__ __forceinline__ void decode_piece(const KvArgs& b, const bf16_t* q, int64_t q_stride, const KvOut& w, float c,
                                             const KvCut& cut, int wg) {
    using Wave = KvWave<D, SUB, SPLIT>;
    constexpr int NE = D / 16, RB = Wave::ROWS;
    constexpr int kStage = KvStage<D>::kBytes, kSums = RB * (D + 4) * 4;
    // (once the steps are done, a stage holds two waves' sums)
    constexpr int kHalf = 4 * kStage > 2 * kSums ? 4 * kStage : 2 * kSums;
    __shared__ __attribute__((aligned(1024))) uint8_t stage0[kHalf];
    __shared__ __attribute__((aligned(1024))) uint8_t stage1[kHalf];
    __shared__ float sm[4][RB][3];
    __shared__ KvLine line;
    kv_line<false>(b, cut, line);
    const int lane = threadIdx.x & 63, lg = lane >> 4, row = Wave::row();
    const bool first_col = Wave::col() == 0;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int worker = 4 * wg + wave;
    const KvPieces pieces(uniform64(line.before[256]), cut.workers);
    int64_t pos = pieces.at(min(worker, pieces.workers));
    const int64_t end = pieces.at(min(worker + 1, pieces.workers));
    const int64_t wg_pos = pieces.at(min(4 * wg, pieces.workers)), wg_end = pieces.at(min(4 * wg + 4, pieces.workers));
    KvMerge entry{-1, 0, 0, 0, 0, 0, 0, 0};
    bool inside = false;
    KvPlace<false> at;
    Wave wv;
    if (wg_pos < wg_end) {
        at.seek(b, cut, line, wg_pos);
        inside = wg_pos + (at.steps - at.off) >= wg_end;
        if (inside) at.off += (int)(pos - wg_pos);
        else if (pos < end) at.seek(b, cut, line, pos);
    }
    const int64_t seg0 = pos - at.off;    // (where the first segment begins)
    while (pos < end) {
        const int h = at.pair % b.kv_heads, row0 = at.pair / b.kv_heads * RB, rows = at.q.rows * b.group;
        const int stop = (int)min((int64_t)at.steps, at.off + (end - pos));
        // steps up to the last token that the tile's last row sees
        const int seen = max(0, at.q.len - at.q.rows + 1 + (min(rows, row0 + RB) - 1) / b.group);
        wv.load_q(b, at.s, at.q, h, q, q_stride, row0);
        wv.run(b, stage0 + wave * kStage, stage1 + wave * kStage, at.off, min(kv_steps(seen), stop), c);
        wv.finish();
        const int64_t begin = pos - at.off;
        if (at.off == 0 && stop < at.steps) {
            // it begins here and is cut: its last worker is the one whose piece holds its last step
            const int64_t over = begin + at.steps;
            const int last = pieces.holder(over - 1);
            int in0 = pieces.at(4 * wg) == begin ? wg : wg + 1, in1 = last >> 2;
            if (pieces.at(min(4 * in1 + 4, pieces.workers)) == over) ++in1;
            if (in0 >= in1) in0 = in1 = (last + 4) >> 2;
            if (!(inside && begin == wg_pos && over == wg_end))
                entry = KvMerge{last, row0, min(RB, rows - row0), at.q.r0, h, in0, in1, 0};
        }
        if (inside) break;
        if (first_col && row0 + row < rows) {
            if (at.off == 0 && stop == at.steps)
                wv.store(out_row<D>(b, w, at.q.r0, h, row0 + row));
            else
                wv.put_part(part_row<D>(w, RB, 2 * worker + (at.off == 0), row), part_ml<D>(w, RB, 2 * worker + (at.off == 0), row));
        }
        pos += stop - at.off;
        if (pos < end) at.next(b, cut);
    }
    if (lane == 0) put_merge(w, worker, entry);
    if (!inside) return;

    // the four waves' sums of one segment (a wave without steps has none)
    if (pos >= end) {
        wv.m = -INFINITY;
        wv.l = wv.z = 0.f;
#pragma unroll
        for (int e = 0; e < NE; ++e) wv.o[e] = f32x4{0.f, 0.f, 0.f, 0.f};
    }
    auto sums = [&](int x, int row, int d) {
        return reinterpret_cast<float*>((x < 2 ? stage0 : stage1) + (x & 1) * kSums) + row * (D + 4) + d;
    };
    __syncthreads();   // (every wave has read its last step)
    if (first_col) {
        if (lg == 0) {
            sm[wave][row][0] = wv.m;
            sm[wave][row][1] = wv.l;
            sm[wave][row][2] = wv.z;
        }
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int e = 0; e < NE; e += 4) {
                const f32x4 v{wv.o[e][i], wv.o[e + 1][i], wv.o[e + 2][i], wv.o[e + 3][i]};
                *reinterpret_cast<f32x4*>(sums(wave, row, (4 * lg + i) * NE + e)) = v;
            }
    }
    __syncthreads();
    // 16 threads a row, D / 16 values each
    const int r = threadIdx.x >> 4, d0 = (threadIdx.x & 15) * NE;
    const int h = at.pair % b.kv_heads, row0 = at.pair / b.kv_heads * RB, rows = at.q.rows * b.group;
    if (r >= RB || row0 + r >= rows) return;
    float m = -INFINITY;
#pragma unroll
    for (int x = 0; x < 4; ++x) m = fmaxf(m, sm[x][r][0]);
    float l = 0.f, acc[NE];
#pragma unroll
    for (int e = 0; e < NE; ++e) acc[e] = 0.f;
#pragma unroll
    for (int x = 0; x < 4; ++x) {
        const float g = part_factor(sm[x][r][0], sm[x][r][1], m, c);
        l += g * sm[x][r][1];
#pragma unroll
        for (int e = 0; e < NE; ++e) acc[e] += g * (*sums(x, r, d0 + e) + sm[x][r][2]);
    }
    const int64_t begin = seg0;
    if (begin == wg_pos && begin + at.steps == wg_end) {
        const float inv = l == 0.f ? 0.f : 1.f / l;
        bf16_t* o = out_row<D>(b, w, at.q.r0, h, row0 + r) + d0;
#pragma unroll
        for (int e = 0; e < NE; e += 4) {
            u32x2 v;
            v[0] = pack2(acc[e] * inv, acc[e + 1] * inv);
            v[1] = pack2(acc[e + 2] * inv, acc[e + 3] * inv);
            *reinterpret_cast<u32x2*>(o + e) = v;
        }
    } else {
        const int slot = 2 * (4 * wg) + (begin == wg_pos);
        float* p = part_row<D>(w, RB, slot, r) + d0;
#pragma unroll
        for (int e = 0; e < NE; e += 4)
            *reinterpret_cast<f32x4*>(p + e) = f32x4{acc[e], acc[e + 1], acc[e + 2], acc[e + 3]};
        if (d0 == 0) {
            float* ml = part_ml<D>(w, RB, slot, r);
            ml[0] = m;
            ml[1] = l;
        }
    }
}

// ---------------------------------------------------------------- attention: many query rows

// Workers are workgroups: the four waves have 32 of a tile's 128 rows each and share the tokens'
// slabs, 64 tokens a stage, wave w bringing block w straight to LDS one stage ahead.  Codes are
// put in place by every wave for itself.  Bound by the vector units: of about 260 instructions for
// 32 tokens 130 put codes in place and 110 are the softmax's, 0.55 us beside 16 matrix operations of 15 ns.
// Measured on MI355X: four pieces of 512 rows behind up to 4,096 tokens (32 heads over 8 of 128) 105 us,
// 0.44 PFLOP/s, and 14 us for the sums of the cut tiles (66 MB of them written and read).
//
// 32-row matrix operations: lane (r, hg) = (lane % 32, lane / 32) holds everything of query row r:
// of 32 tokens' scores those of tokens 8 x + 4 hg .. + 3 (x 0..3), of the output as store() says.
// The weights are rounded to bf16 once here, by at most 2^-8 of a weight, as much as the output's own
// rounding and, unlike that one, with different signs from token to token (four pieces of 512 rows: 0.0024 of
// the outputs' size from the exact ones, 0.0017 of it the output's rounding); a second half, as few rows
// have it, would cost half as many matrix operations again.
// z and the sum of the rounded weights put the codes' 16 and lo in: o = sum w' (16 + code) +
// sum p (lo + 8 step) - 24 sum w', so that the rounding counts for code - 8 only.
template <int D>
struct KvRows {
    static constexpr int S = D / 16, NB = D / 32, NQ = D == 256 ? 2 : 1;
    static constexpr int kSlab = 8 * D, kCodes = 8 * kSlab, kStage = kCodes + 4 * 128 + 16;
    static constexpr int kTable = 64 * 16;   // a wave's floats of a stage's tokens
    u32x4 q[S];
    f32x16_t o[NB];
    float qsum, m, thr, l, z, s;
    int limit, limit_all;
    CodeConst cc;

    __device__ __forceinline__ void load_q(const KvArgs& b, const KvSeq& sq, int h, const bf16_t* qp, int64_t stride,
                                           int row0) {
        const int hg = (threadIdx.x & 63) >> 5, r = row0 + (threadIdx.x & 31), rows = sq.rows * b.group;
        qsum = 0.f;
        if (r < rows) {
            const bf16_t* p = qp + (int64_t)(sq.r0 + r / b.group) * stride + (int64_t)(h * b.group + r % b.group) * D +
                              hg * (D / 2);
#pragma unroll
            for (int i = 0; i < S; ++i) q[i] = ld16(p + 8 * i);
        } else {
#pragma unroll
            for (int i = 0; i < S; ++i) q[i] = u32x4{0, 0, 0, 0};
        }
#pragma unroll
        for (int i = 0; i < S; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) qsum += bf16_lo(q[i][j]) + bf16_hi(q[i][j]);
        qsum = sum_hg(qsum);
        const int first = sq.len - sq.rows + 1;
        limit = r < rows ? first + r / b.group : 0;
        limit_all = row0 < rows ? first + row0 / b.group : 0;
        m = 0.f;
        thr = -INFINITY;   // (no token yet)
        l = z = s = 0.f;
#pragma unroll
        for (int e = 0; e < NB; ++e)
#pragma unroll
            for (int i = 0; i < 16; ++i) o[e][i] = 0.f;
    }

    // Keys and values of one block to its place in a stage: keys as [i][hg][token], values as
    // [n][i] 16-byte units, the order in which the lanes read them.
    static __device__ __forceinline__ void load(const uint8_t* k, const uint8_t* v, uint8_t* stage, int block) {
        const int lane = threadIdx.x & 63;
        uint8_t* to = stage + block * 2 * kSlab;
        auto key = [](int u) { return (u & 15) * (D / 2) + ((u >> 4) & 1) * (D / 4) + (u >> 5) * 16; };
        auto val = [](int u) { return (u & 15) * (D / 2) + (u >> 4) * 16; };
        if constexpr (D == 64) {
            global_load_lds16(lane < 32 ? k + key(lane) : v + val(lane & 31), to);
        } else {
#pragma unroll
            for (int i = 0; i < D / 128; ++i) global_load_lds16(k + key(64 * i + lane), to + 1024 * i);
#pragma unroll
            for (int i = 0; i < D / 128; ++i) global_load_lds16(v + val(64 * i + lane), to + kSlab + 1024 * i);
        }
        if (lane < 32) global_load_lds4((lane < 16 ? k : v) + 8 * D + (lane & 15) * 4, stage + kCodes + block * 128);
    }

    // the floats of a stage's 64 tokens: key step and lo times c, value step, value lo + 8 step
    static __device__ __forceinline__ void table(const uint8_t* stage, f32x4* tab, float c) {
        const int lane = threadIdx.x & 63;
        const uint32_t* w = reinterpret_cast<const uint32_t*>(stage + kCodes) + (lane >> 4) * 32 + (lane & 15);
        const uint32_t kw = w[0], vw = w[16];
        const float st = bf16_lo(vw);
        tab[lane] = f32x4{bf16_lo(kw) * c, bf16_hi(kw) * c, st, fmaf(8.f, st, bf16_hi(vw))};
    }

    // 32 tokens: blocks 2 u and 2 u + 1 of a stage, the first at position tok0; bit a of bad: block
    // 2 u + a counts nothing
    __device__ __forceinline__ void step(const uint8_t* stage, const f32x4* tab, int u, int tok0, int bad) {
        const int lane = threadIdx.x & 63, lr = lane & 31, hg = lane >> 5;
        f32x16_t x;
        const float init = -16.f * qsum;
#pragma unroll
        for (int i = 0; i < 16; ++i) x[i] = init;
        const uint8_t* kp = stage + (2 * u + (lr >> 4)) * 2 * kSlab + (hg * 16 + (lr & 15)) * 16;
#pragma unroll
        for (int i = 0; i < D / 64; ++i) {
            const u32x4 w = ld16(kp + i * 512);
#pragma unroll
            for (int y = 0; y < 4; ++y) {
                const uint32_t word = w[y];
                u32x4 kf;
#pragma unroll
                for (int j = 0; j < 4; ++j) kf[j] = code_pair(cc, word, j);
                x = mma32(kf, q[4 * i + y], x);
            }
        }
        float st[16], zl[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            const f32x4 f = tab[32 * u + 8 * (i / 4) + 4 * hg + i % 4];
            x[i] = fmaf(x[i], f[0], fmaf(f[1], qsum, -m));
            st[i] = f[2];
            zl[i] = f[3];
        }
        if (__builtin_expect(tok0 + 32 > limit_all || bad, 0)) {
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                const int tok = tok0 + 8 * (i / 4) + 4 * hg + i % 4;
                if (tok >= limit || ((bad >> (i / 8)) & 1)) {
                    x[i] = -INFINITY;
                    st[i] = zl[i] = 0.f;
                }
            }
        }
        float top = x[0];
#pragma unroll
        for (int i = 1; i < 16; ++i) top = fmaxf(top, x[i]);
        if (__ballot(top > thr)) {
            float d = max_hg(top);
            const bool fresh = thr < 0.f;
            if (!(d > thr)) d = 0.f;   // (not this row, or it has no token yet)
            else thr = 8.f;
            // a row's first tokens set the scale of sums that are still zero: 2^-d of scores below -128
            // is infinite, and zero times that not a number
            const float al = fresh ? 1.f : __builtin_amdgcn_exp2f(-d);
            m += d;
            l *= al;
            z *= al;
            s *= al;
#pragma unroll
            for (int e = 0; e < NB; ++e)
#pragma unroll
                for (int i = 0; i < 16; ++i) o[e][i] *= al;
#pragma unroll
            for (int i = 0; i < 16; ++i) x[i] -= d;
        }
        u32x4 p[2];
        const bf16x2_t one = __builtin_bit_cast(bf16x2_t, 0x3F803F80u);
#pragma unroll
        for (int i = 0; i < 16; i += 2) {
            const float p0 = __builtin_amdgcn_exp2f(x[i]), p1 = __builtin_amdgcn_exp2f(x[i + 1]);
            l += p0;
            l += p1;
            z = fmaf(p0, zl[i], z);
            z = fmaf(p1, zl[i + 1], z);
            const uint32_t w = pack2(p0 * st[i], p1 * st[i + 1]);
            s = __builtin_amdgcn_fdot2_f32_bf16(__builtin_bit_cast(bf16x2_t, w), one, s, false);
            p[i / 8][i % 8 / 2] = w;
        }
#pragma unroll
        for (int a = 0; a < 2; ++a) {
            // the lane's words of block 2 u + a: token pairs 2 hg, 2 hg + 1, 4 + 2 hg, 5 + 2 hg of value
            // column lane % 16, the half of its values that lane / 16 says
            const uint8_t* vp = stage + (2 * (2 * u + a) + 1) * kSlab + (lane & 15) * 16;
            const int sel = (lane >> 4) & 1;
            uint32_t w[NQ][4];
            if constexpr (D == 64) {
#pragma unroll
                for (int n = 0; n < 2; ++n) {
                    const u32x2 v = *reinterpret_cast<const u32x2*>(vp + n * 256 + hg * 8);
                    w[0][2 * n] = v[0] >> (8 * sel);
                    w[0][2 * n + 1] = v[1] >> (8 * sel);
                }
            } else if constexpr (D == 128) {
#pragma unroll
                for (int n = 0; n < 2; ++n) {
                    const uint32_t* v = reinterpret_cast<const uint32_t*>(vp + (2 * n + hg) * 256) + sel;
                    w[0][2 * n] = v[0];
                    w[0][2 * n + 1] = v[2];
                }
            } else {
#pragma unroll
                for (int n = 0; n < 4; ++n) {
                    const uint32_t* v = reinterpret_cast<const uint32_t*>(vp + (4 * (n / 2) + 2 * hg + n % 2) * 256) + sel;
                    w[0][n] = v[0];
                    w[1][n] = v[2];
                }
            }
#pragma unroll
            for (int e = 0; e < NB; ++e) {
                u32x4 vf;
#pragma unroll
                for (int n = 0; n < 4; ++n) vf[n] = code_pair(cc, w[e / 4][n], e % 4);
                o[e] = mma32(vf, p[a], o[e]);
            }
        }
    }

    __device__ __forceinline__ void finish() {
        l = sum_hg(l);
        z = sum_hg(z) - 24.f * sum_hg(settled(s));
        if (thr < 0.f) m = -INFINITY;
    }

    // the row's values, four at a time: f(first value, values)
    template <class F>
    __device__ __forceinline__ void each4(F f) const {
        const int hg = (threadIdx.x & 63) >> 5;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int col = 8 * (i / 4) + 4 * hg + i % 4;
            if constexpr (D == 64) {
                f(col * 4, f32x4{o[0][i] + z, o[1][i] + z, o[0][i + 8] + z, o[1][i + 8] + z});
            } else {
#pragma unroll
                for (int n = 0; n < NQ; ++n)
#pragma unroll
                    for (int h = 0; h < 2; ++h)
                        f(col * (D / 16) + 8 * n + 4 * h, f32x4{o[4 * n][i + 8 * h] + z, o[4 * n + 1][i + 8 * h] + z,
                                                                o[4 * n + 2][i + 8 * h] + z, o[4 * n + 3][i + 8 * h] + z});
            }
        }
    }
};

template <int D>
__device__ __forceinline__ void prefill_piece(const KvArgs& b, const bf16_t* q, int64_t q_stride, const KvOut& w, float c,
                                              const KvCut& cut, int worker) {
    using Rows = KvRows<D>;
    constexpr int RB = kKvPrefillRows;
    __shared__ __attribute__((aligned(1024))) uint8_t stage0[Rows::kStage];
    __shared__ __attribute__((aligned(1024))) uint8_t stage1[Rows::kStage];
    __shared__ f32x4 tabs[4][64];
    __shared__ KvLine line;
    kv_line<true>(b, cut, line);
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const KvPieces pieces(uniform64(line.before[256]), cut.workers);
    int64_t pos = pieces.at(min(worker, pieces.workers));
    const int64_t end = pieces.at(min(worker + 1, pieces.workers));
    KvMerge entry{-1, 0, 0, 0, 0, 0, 0, 0};
    KvPlace<true> at;
    if (pos < end) at.seek(b, cut, line, pos);
    while (pos < end) {
        const int h = at.pair % b.kv_heads, tile0 = at.pair / b.kv_heads * RB, rows = at.q.rows * b.group;
        const int row0 = tile0 + 32 * wave, stop = (int)min((int64_t)at.steps, at.off + (end - pos));
        if (at.off == 0 && stop < at.steps) {
            const int last = pieces.holder(pos + at.steps - 1), none = (last + 4) >> 2;
            entry = KvMerge{last, tile0, min(RB, rows - tile0), at.q.r0, h, none, none, 0};
        }
        // tokens that the tile's last row sees, and the wave's
        auto sees = [&](int row) { return max(0, at.q.len - at.q.rows + 1 + row / b.group); };
        const int end_tok = min(32 * stop, sees(min(rows, tile0 + RB) - 1));
        const int wave_end = row0 < rows ? min(end_tok, sees(min(rows, row0 + 32) - 1)) : 0;
        const int first = 32 * at.off, n = (max(0, end_tok - first) + 63) / 64;
        const int ks = 2 * h, vs = 2 * h + 1;
        const int64_t koff = (int64_t)(ks % b.slabs_per_page) * kv_slab_bytes(D);
        const int64_t voff = (int64_t)(vs % b.slabs_per_page) * kv_slab_bytes(D);
        Rows r;
        r.load_q(b, at.q, h, q, q_stride, row0);
        int pk = -1, pv = -1;   // lane j: the pages of this wave's block of stage j of 64
        auto pages = [&](int j0) {
            const int blk = first / kKvBlock + 4 * (j0 + lane) + wave;
            pk = pv = -1;
            if (kKvBlock * blk < end_tok) {
                pk = *kv_entry(b, at.s, blk, ks);
                pv = *kv_entry(b, at.s, blk, vs);
            }
        };
        auto issue = [&](int j, uint8_t* stage) {
            if ((j & 63) == 0) pages(j);
            const int k = __builtin_amdgcn_readlane(pk, j & 63), v = __builtin_amdgcn_readlane(pv, j & 63);
            const bool ok = kv_page_ok(b, k) && kv_page_ok(b, v);
            Rows::load(b.pages + (ok ? k : 0) * b.page_bytes + koff, b.pages + (ok ? v : 0) * b.page_bytes + voff, stage,
                       wave);
            if (lane == 0) reinterpret_cast<int*>(stage + Rows::kCodes + 512)[wave] = !ok;
        };
        if (n > 0) issue(0, stage0);
#pragma unroll 1
        for (int j = 0; j < n; j += 2) {
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                if (j + x >= n) break;
                uint8_t* now = x ? stage1 : stage0;
                wait_vmcnt<0>();
                wait_lgkm0();
                __builtin_amdgcn_s_barrier();   // the stage is there, and every wave has done with the other
                landed();
                if (j + x + 1 < n) issue(j + x + 1, x ? stage0 : stage1);
                const int tok = first + 64 * (j + x);
                if (tok < wave_end) {
                    Rows::table(now, tabs[wave], c);
                    const u32x4 f = ld16(now + Rows::kCodes + 512);
                    const int bad = __builtin_amdgcn_readfirstlane(f[0] | f[1] << 1 | f[2] << 2 | f[3] << 3);
                    r.step(now, tabs[wave], 0, tok, bad & 3);
                    if (tok + 32 < wave_end) r.step(now, tabs[wave], 1, tok + 32, bad >> 2);
                }
            }
        }
        r.finish();
        const int rt = 32 * wave + (lane & 31);
        if (tile0 + rt < rows) {
            if (at.off == 0 && stop == at.steps) {
                bf16_t* o = out_row<D>(b, w, at.q.r0, h, tile0 + rt);
                const float inv = r.l == 0.f ? 0.f : 1.f / r.l;
                r.each4([&](int d, const f32x4& v) {
                    *reinterpret_cast<u32x2*>(o + d) = u32x2{pack2(v[0] * inv, v[1] * inv), pack2(v[2] * inv, v[3] * inv)};
                });
            } else {
                const int slot = 2 * worker + (at.off == 0);
                float* p = part_row<D>(w, RB, slot, rt);
                r.each4([&](int d, const f32x4& v) { *reinterpret_cast<f32x4*>(p + d) = v; });
                if (lane < 32) {
                    float* ml = part_ml<D>(w, RB, slot, rt);
                    ml[0] = r.m / c;   // (parts are joined at the scale of the scores)
                    ml[1] = r.l;
                }
            }
        }
        __syncthreads();   // (the stages are free)
        pos += stop - at.off;
        if (pos < end) at.next(b, cut);
    }
    if (threadIdx.x == 0) put_merge(w, worker, entry);
}

// Sums of parts at one scale.
struct KvSum {
    float m, l;
    f32x4 acc;
    __device__ __forceinline__ void add(float mo, float lo, const f32x4& ao, float c) {
        const float top = fmaxf(m, mo), f = part_factor(m, l, top, c), g = part_factor(mo, lo, top, c);
        m = top;
        l = l * f + lo * g;
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[i] = acc[i] * f + ao[i] * g;
    }
};

// Parts p0, p0 + stride, ... below n of a cut segment's row r, values d0 .. d0 + 3, eight parts'
// loads at a time.
template <int D>
__device__ __forceinline__ KvSum sum_parts(const KvOut& w, const KvMerge& e, int first, int n, int rb, int r, int d0,
                                           int p0, int stride, float c) {
    const int n0 = min(4 * e.inside0, e.last + 1) - first, n1 = n0 + e.inside1 - e.inside0;
    KvSum s{-INFINITY, 0.f, f32x4{0.f, 0.f, 0.f, 0.f}};
    for (int p = p0; p < n; p += 8 * stride) {
        f32x4 v[8];
        float mp[8], lp[8];
#pragma unroll
        for (int y = 0; y < 8; ++y) {
            const int i = p + y * stride;
            if (i >= n) continue;
            const int x = i < n0 ? first + i : i < n1 ? 4 * (e.inside0 + i - n0) : 4 * e.inside1 + i - n1;
            const int slot = 2 * x + (x == first);
            const float* ml = part_ml<D>(w, rb, slot, r);
            v[y] = *reinterpret_cast<const f32x4*>(part_row<D>(w, rb, slot, r) + d0);
            mp[y] = ml[0];
            lp[y] = ml[1];
        }
#pragma unroll
        for (int y = 0; y < 8; ++y)
            if (p + y * stride < n) s.add(mp[y], lp[y], v[y], c);
    }
    return s;
}

// The parts of the cut segments' rows, D / 4 threads a row.  Every workgroup looks through the
// workers for the cut segments and takes its share: a row a wave at a time, or, where there are
// fewer rows than workgroups, a row a workgroup.  The order of the sums is fixed.  4 to 7 us.
template <int D>
__device__ __forceinline__ void merge_list(const KvArgs& b, const KvOut& w, float c, int rb, int most_rows, int wg, int wgs) {
    constexpr int TPR = D / 4, PW = 256 / TPR, WW = 64 / TPR, kMost = kv_workers(D) / 256;
    __shared__ float sa[PW][D + 4], sm[PW], sl[PW];
    __shared__ int sums[4], list[kv_workers(D)];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int* last = reinterpret_cast<const int*>(w.ws + (int64_t)w.workers * sizeof(KvMerge));
    // this thread's workers: kMost of them, bit i of mine: the i-th has a cut segment
    uint32_t mine = 0;
#pragma unroll
    for (int i = 0; i < kMost; i += 4) {
        const int x = threadIdx.x * kMost + i;   // (the workers are a multiple of four)
        if (x < w.workers) {
            const u32x4 v = ld16(last + x);
#pragma unroll
            for (int y = 0; y < 4; ++y) mine |= (~v[y] >> 31) << (i + y);
        }
    }
    int at = wave_scan((int)__popc(mine));
    if (lane == 63) sums[wave] = at;
    __syncthreads();
    int total = 0;
#pragma unroll
    for (int x = 0; x < 4; ++x) {
        if (x < wave) at += sums[x];
        total += sums[x];
    }
    at -= __popc(mine);
    for (; mine; mine &= mine - 1) list[at++] = threadIdx.x * kMost + __ffs(mine) - 1;
    __syncthreads();
    const int items = total * most_rows;
    const bool per_wave = items > wgs;
    auto store = [&](const KvMerge& e, int r, int d0, const KvSum& s) {
        const float inv = s.l == 0.f ? 0.f : 1.f / s.l;
        u32x2 o;
        o[0] = pack2(s.acc[0] * inv, s.acc[1] * inv);
        o[1] = pack2(s.acc[2] * inv, s.acc[3] * inv);
        *reinterpret_cast<u32x2*>(out_row<D>(b, w, e.r0, e.h, e.row0 + r) + d0) = o;
    };
    const int d0 = threadIdx.x % TPR * 4;
    for (int item = per_wave ? 4 * wg + wave : wg; item < items; item += (per_wave ? 4 : 1) * wgs) {
        const int first = __builtin_amdgcn_readfirstlane(list[item / most_rows]);
        const KvMerge e = reinterpret_cast<const KvMerge*>(w.ws)[first];
        const int n0 = min(4 * e.inside0, e.last + 1) - first + e.inside1 - e.inside0;
        const int n = n0 + max(0, e.last + 1 - 4 * e.inside1);
        // (most_rows is only what the caller expects)
        for (int r = item % most_rows; r < e.rows; r += most_rows) {
            if (per_wave) {
                KvSum s = sum_parts<D>(w, e, first, n, rb, r, d0, lane / TPR, WW, c);
#pragma unroll
                for (int x = TPR; x < 64; x <<= 1) {
                    f32x4 o;
#pragma unroll
                    for (int i = 0; i < 4; ++i) o[i] = __shfl_xor(s.acc[i], x, 64);
                    const float mo = __shfl_xor(s.m, x, 64), lo = __shfl_xor(s.l, x, 64);
                    s.add(mo, lo, o, c);
                }
                if (lane < TPR) store(e, r, d0, s);
                continue;
            }
            const int pw = threadIdx.x / TPR;
            KvSum s = sum_parts<D>(w, e, first, n, rb, r, d0, pw, PW, c);
            *reinterpret_cast<f32x4*>(&sa[pw][d0]) = s.acc;
            if (d0 == 0) {
                sm[pw] = s.m;
                sl[pw] = s.l;
            }
            __syncthreads();
            if (pw == 0) {
#pragma unroll
                for (int x = 1; x < PW; ++x) s.add(sm[x], sl[x], *reinterpret_cast<const f32x4*>(&sa[x][d0]), c);
                store(e, r, d0, s);
            }
            __syncthreads();
        }
    }
}

// The same for row tiles of many rows, sixteen rows of a worker's cut segment a workgroup.  Mostly a
// segment has two or three parts and every thread sums its rows' own.  From 17 parts on the
// workgroups of its second to sixteenth worker, which have no segment of their own to join, take a
// row each, and its threads share the parts.  Bound by the bytes of the parts (four pieces of 512 rows: 14
// us), or by the latency of three dependent reads (11 us).
template <int D>
__device__ __forceinline__ void merge_tile(const KvArgs& b, const KvOut& w, float c, int rb, int worker, int chunk) {
    constexpr int TPR = D / 4, PW = 256 / TPR, RY = 16 / PW;
    __shared__ float sa[PW][D + 4], sm[PW], sl[PW];
    const int* lasts = reinterpret_cast<const int*>(w.ws + (int64_t)w.workers * sizeof(KvMerge));
    const int back = min((int)(threadIdx.x & 63), min(worker, 15));
    const int last_back = lasts[worker - back];
    const uint64_t mine = __ballot(back == 0 ? last_back >= 0 : last_back >= worker - back + 16);
    if (mine == 0) return;
    const int x = worker - __builtin_ctzll(mine);
    const KvMerge e = reinterpret_cast<const KvMerge*>(w.ws)[x];
    const int n = e.last + 1 - x;
    const int d0 = threadIdx.x % TPR * 4, pw = threadIdx.x / TPR;
    auto store = [&](int r, const KvSum& s) {
        const float inv = s.l == 0.f ? 0.f : 1.f / s.l;
        *reinterpret_cast<u32x2*>(out_row<D>(b, w, e.r0, e.h, e.row0 + r) + d0) =
            u32x2{pack2(s.acc[0] * inv, s.acc[1] * inv), pack2(s.acc[2] * inv, s.acc[3] * inv)};
    };
    if (n > 16) {
        const int r = 16 * chunk + worker - x;
        if (r >= e.rows) return;
        KvSum s = sum_parts<D>(w, e, x, n, rb, r, d0, pw, PW, c);
        *reinterpret_cast<f32x4*>(&sa[pw][d0]) = s.acc;
        if (d0 == 0) {
            sm[pw] = s.m;
            sl[pw] = s.l;
        }
        __syncthreads();
        if (pw == 0) {
#pragma unroll
            for (int i = 1; i < PW; ++i) s.add(sm[i], sl[i], *reinterpret_cast<const f32x4*>(&sa[i][d0]), c);
            store(r, s);
        }
        return;
    }
    const int r0 = 16 * chunk + pw;
    KvSum s[RY];
#pragma unroll
    for (int y = 0; y < RY; ++y) s[y] = KvSum{-INFINITY, 0.f, f32x4{0.f, 0.f, 0.f, 0.f}};
    for (int p = 0; p < n; p += 2) {
        f32x4 v[2][RY];
        float mp[2][RY], lp[2][RY];
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int y = 0; y < RY; ++y) {
                const int k = min(p + i, n - 1), slot = 2 * (x + k) + (k == 0), r = min(r0 + y * PW, e.rows - 1);
                const float* ml = part_ml<D>(w, rb, slot, r);
                v[i][y] = *reinterpret_cast<const f32x4*>(part_row<D>(w, rb, slot, r) + d0);
                mp[i][y] = ml[0];
                lp[i][y] = ml[1];
            }
#pragma unroll
        for (int i = 0; i < 2; ++i)
            if (p + i < n)
#pragma unroll
                for (int y = 0; y < RY; ++y) s[y].add(mp[i][y], lp[i][y], v[i][y], c);
    }
#pragma unroll
    for (int y = 0; y < RY; ++y)
        if (r0 + y * PW < e.rows) store(r0 + y * PW, s[y]);
}

// ---------------------------------------------------------------- attention: kernels

template <int D, int SUB, bool SPLIT>
__global__ __launch_bounds__(256, D == 64 ? 4 : D == 128 ? 3 : 2) void kv_decode_kernel(KvArgs b, const bf16_t* q, int64_t q_stride,
                                                                          KvOut w, float c, KvCut cut) {
    decode_piece<D, SUB, SPLIT>(b, q, q_stride, w, c, cut, blockIdx.x);
}

template <int D>
__global__ __launch_bounds__(256) void kv_merge_kernel(KvArgs b, KvOut w, float c, int rb, int most_rows) {
    merge_list<D>(b, w, c, rb, most_rows, blockIdx.x, gridDim.x);
}

// Batches in which sequences of few and of many rows may meet: the pieces of many rows, then those of
// few, in one launch, and then both kinds' sums.  (In turn, the few ones leave places to the others
// unevenly: 512 pieces of many rows alone took 190 us so, 112 us this way.)
struct KvBoth {
    KvOut few, many;
    KvCut few_cut, many_cut;
};

template <int D>
__global__ __launch_bounds__(256, D == 256 ? 1 : 2) void kv_mixed_kernel(KvArgs b, const bf16_t* q, int64_t q_stride, float c,
                                                                         KvBoth k) {
    const int nm = k.many.workers, i = blockIdx.x;
    if (i < nm) prefill_piece<D>(b, q, q_stride, k.many, c, k.many_cut, i);
    else decode_piece<D, 1, false>(b, q, q_stride, k.few, c, k.few_cut, i - nm);
}

constexpr int kTileChunks = kKvPrefillRows / 16;
template <int D>
__global__ __launch_bounds__(256) void kv_mixed_merge_kernel(KvArgs b, float c, KvBoth k) {
    const int nm = k.many.workers * kTileChunks, i = blockIdx.x;
    if (i < nm) merge_tile<D>(b, k.many, c, kKvPrefillRows, i / kTileChunks, i % kTileChunks);
    else merge_list<D>(b, k.few, c, kKvRowTile, kKvRowTile, i - nm, gridDim.x - nm);
}

template <int D>
hipError_t attention(const KvArgs& b, const bf16_t* q, int64_t q_stride, bf16_t* out, int64_t out_stride, float scale,
                     int32_t max_rows, void* workspace, hipStream_t s) {
    const float c = scale * 1.44269504088896341f;
    const int64_t rows = (int64_t)b.n_rows * b.group, most = (int64_t)max_rows * b.group;
    auto pairs = [&](int rb_shift) { return ((rows >> rb_shift) + b.n_seqs) * b.kv_heads; };
    auto share = [&](int rb_shift, int workers, int per_block) {
        // no more workers than steps there can be
        const int64_t n = pairs(rb_shift), steps = std::max(1, (b.max_blocks + 1) / 2);
        if (n < workers) workers = (int)std::min<int64_t>(workers, n * steps);
        return (workers + per_block - 1) / per_block * per_block;
    };
    auto merge_grid = [&](int rb_shift, int workers, int most_rows) {
        return (int)std::min<int64_t>(std::min<int64_t>(pairs(rb_shift), workers) * most_rows, 1024);
    };
    auto go = [&](int rb_shift, auto kern) {
        const KvOut w{out, out_stride, static_cast<uint8_t*>(workspace), share(rb_shift, kv_workers(D), 4)};
        hipLaunchKernelGGL(kern, dim3(w.workers / 4), dim3(256), 0, s, b, q, q_stride, w, c,
                           KvCut{rb_shift, kKvAll, w.workers});
        const int most_rows = (int)std::min<int64_t>(1 << rb_shift, std::max<int64_t>(most, 1));
        hipLaunchKernelGGL(kv_merge_kernel<D>, dim3(merge_grid(rb_shift, w.workers, most_rows)), dim3(256), 0, s, b, w, c,
                           1 << rb_shift, most_rows);
        return hipGetLastError();
    };
    static_assert(kKvRowTile == 16 && kKvPrefillRows == 128, "row tiles");
    // few rows: as many columns of a matrix operation a row as there are
    if (most <= 1) return go(0, kv_decode_kernel<D, 8, true>);
    if (most <= 2) return go(1, kv_decode_kernel<D, 4, true>);
    if (most <= 4) return go(2, kv_decode_kernel<D, 4, false>);
    if (most <= 8) return go(3, kv_decode_kernel<D, 2, false>);
    if (!kv_many_rows(b.group, max_rows)) return go(4, kv_decode_kernel<D, 1, false>);
    KvBoth k;
    k.few = KvOut{out, out_stride, static_cast<uint8_t*>(workspace), share(4, kv_workers(D), 4)};
    k.many = KvOut{out, out_stride, k.few.ws + kv_few_bytes(D), share(7, kKvPrefillWorkers, 4)};
    k.few_cut = KvCut{4, kKvFew, k.few.workers};
    k.many_cut = KvCut{7, kKvMany, k.many.workers};
    hipLaunchKernelGGL(kv_mixed_kernel<D>, dim3(k.few.workers / 4 + k.many.workers), dim3(256), 0, s, b, q, q_stride, c, k);
    const int few_merge = merge_grid(4, k.few.workers, 16);
    hipLaunchKernelGGL(kv_mixed_merge_kernel<D>, dim3(k.many.workers * kTileChunks + few_merge), dim3(256), 0, s, b, c, k);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_kv_append(int head_dim, const KvArgs& b, const KvAppendArgs& a, hipStream_t s) {
    const int64_t per_row = (a.q ? b.heads : 0) + 2 * (int64_t)b.kv_heads;
    auto go = [&](auto kern, int lanes) {
        // a workgroup for each group of heads where they are few (latency), no more than run at once where
        // there are many (2,286 rows of 32 + 2 x 32 heads of 128 37 us; neighbouring heads a workgroup 45, all
        // apart 53)
        const int rows = kv_append_rows(head_dim);
        const int64_t row_groups = (b.n_rows + rows - 1) / rows, groups = (per_row + lanes / rows - 1) / (lanes / rows);
        const int64_t blocks = std::max<int64_t>(1, std::min(groups, kv_append_blocks(head_dim) / row_groups));
        const int64_t grid = row_groups * blocks;
        if (grid > INT32_MAX) return hipErrorInvalidValue;
        hipLaunchKernelGGL(kern, dim3((unsigned)grid), dim3(256), 0, s, b, a, (int)blocks);
        return hipGetLastError();
    };
    switch (head_dim) {
        case 64: return go(kv_append_kernel<64>, 32);
        case 128: return go(kv_append_kernel<128>, 16);
        case 256: return go(kv_append_kernel<256>, 8);
    }
    return hipErrorInvalidValue;
}

hipError_t launch_kv_attention(int head_dim, const KvArgs& b, const void* q, int64_t q_stride, void* out,
                               int64_t out_stride, float scale, int32_t max_rows, void* workspace, hipStream_t s) {
    const bf16_t* qb = static_cast<const bf16_t*>(q);
    bf16_t* ob = static_cast<bf16_t*>(out);
    switch (head_dim) {
        case 64: return attention<64>(b, qb, q_stride, ob, out_stride, scale, max_rows, workspace, s);
        case 128: return attention<128>(b, qb, q_stride, ob, out_stride, scale, max_rows, workspace, s);
        case 256: return attention<256>(b, qb, q_stride, ob, out_stride, scale, max_rows, workspace, s);
    }
    return hipErrorInvalidValue;
}

}  // namespace hagemm
