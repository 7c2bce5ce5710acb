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
#include "common.h"
#include "kv.h"

namespace hagemm {
namespace {

typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));
typedef float f32x2_t __attribute__((ext_vector_type(2)));
typedef unsigned u32pair __attribute__((ext_vector_type(2)));

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

// The page of (sequence, block, slab), or -1 outside the pool.
__device__ __forceinline__ int kv_page(const KvArgs& b, int s, int block, int slab) {
    const int p = b.table[((int64_t)s * b.max_blocks + block) * b.pages_per_block + slab / b.slabs_per_page];
    return p >= 0 && p < b.num_pages ? p : -1;
}

// ---------------------------------------------------------------- append

constexpr int kSeqCache = 1024;   // row_start entries an append workgroup keeps in LDS

// One row of one head per D / 8 lanes, 8 values a lane.  Bound by reading and writing the
// rows once.  Query rows are turned in fp32 and rounded once.  Key rows are turned in fp64
// and rounded to bf16 (the key that an unquantised cache would hold) before they are
// quantised: a code then depends on the exact product only, not on how it was summed, and
// the quantisation itself works on bf16 values, whose halves, differences and quotients by
// a bf16 step are the same in any order of evaluation.
template <int D>
__global__ __launch_bounds__(256) void kv_append_kernel(KvArgs b, KvAppendArgs a) {
    constexpr int LPR = D / 8;
    __shared__ int rs[kSeqCache];
    const int n_cache = min(b.n_seqs + 1, kSeqCache);
    for (int i = threadIdx.x; i < n_cache; i += 256) rs[i] = b.row_start[i];
    __syncthreads();
    const int nq = a.q ? b.heads : 0;
    const int per_row = nq + 2 * b.kv_heads;
    const int64_t item = (int64_t)blockIdx.x * (256 / LPR) + threadIdx.x / LPR;
    const int c = threadIdx.x % LPR;
    const int64_t row64 = item / per_row;
    const bool live = row64 < b.n_rows;
    const int t = live ? (int)row64 : 0;
    const int hh = (int)(item - row64 * per_row);
    // the last sequence that starts at or before row t
    int lo = 0, hi = b.n_seqs;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        const int v = mid < n_cache ? rs[mid] : b.row_start[mid];
        if (v <= t) lo = mid; else hi = mid;
    }
    const int s = lo;
    const KvSeq q = kv_seq(b, s);
    const int pos = q.len - q.rows + (t - q.r0);
    if (!live || t < q.r0 || t >= q.r0 + q.rows || pos < 0 || pos >= b.max_blocks * kKvBlock) return;

    const int kind = hh < nq ? 0 : hh < nq + b.kv_heads ? 1 : 2;   // q, k, v
    const int h = kind == 0 ? hh : kind == 1 ? hh - nq : hh - nq - b.kv_heads;
    const bf16_t* src = static_cast<const bf16_t*>(kind == 0 ? a.q : kind == 1 ? a.k : a.v) +
                        t * (kind == 0 ? a.q_stride : kind == 1 ? a.k_stride : a.v_stride) + (int64_t)h * D;
    float x[8];
    unpack(ld16(src + 8 * c), x, bf16_t{});
    if (kind != 2 && a.rot > 0 && 8 * c < a.rot) {
        const float* cs = a.cos_sin + (int64_t)pos * a.rot;
        const int half = a.rot >> 1;
        float y[8], co[8], si[8];
        bool second = false;
        if (a.interleaved) {
            // pairs (2 i, 2 i + 1): this lane's four angles
            const f32x4 c4 = *reinterpret_cast<const f32x4*>(cs + 4 * c);
            const f32x4 s4 = *reinterpret_cast<const f32x4*>(cs + half + 4 * c);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                y[i] = x[i ^ 1];
                co[i] = c4[i / 2];
                si[i] = i % 2 ? s4[i / 2] : -s4[i / 2];
            }
        } else {
            // pairs (i, i + rot / 2): the partner's values, and this lane's eight angles
            second = 8 * c >= half;
            const int at = second ? 8 * c - half : 8 * c;
            unpack(ld16(src + (second ? at : at + half)), y, bf16_t{});
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
        if (kind == 0) {
#pragma unroll
            for (int i = 0; i < 8; ++i) x[i] = x[i] * co[i] + y[i] * si[i];
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) x[i] = (float)((double)x[i] * co[i] + (double)y[i] * si[i]);
        }
    }
    if (kind == 0) {
        st16(static_cast<bf16_t*>(a.q_out) + t * a.q_out_stride + (int64_t)h * D + 8 * c, pack(x, bf16_t{}));
        return;
    }
    const u32x4 xb = pack(x, bf16_t{});
    unpack(xb, x, bf16_t{});
    // lo and step of the row, from halves (exact), so that no finite row overflows; a row with
    // an infinity or NaN gets a NaN step, and reads back as NaN
    float mn = x[0] * 0.5f, mx = mn, bad = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        x[i] *= 0.5f;
        bad += x[i] - x[i];
        mn = fminf(mn, x[i]);
        mx = fmaxf(mx, x[i]);
    }
#pragma unroll
    for (int m = LPR / 2; m >= 1; m >>= 1) {
        mn = fminf(mn, __shfl_xor(mn, m, LPR));
        mx = fmaxf(mx, __shfl_xor(mx, m, LPR));
        bad += __shfl_xor(bad, m, LPR);
    }
    const uint32_t step_bits = bad == 0.f ? f32_to_bf16((mx - mn) / 7.5f) : 0x7FC0u;
    const uint32_t lo_bits = f32_to_bf16(mn * 2.f);
    const float step = __uint_as_float(step_bits << 16), half_step = step * 0.5f;
    int code[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float r = rintf((x[i] - mn) / half_step);
        code[i] = half_step > 0.f ? (int)fminf(fmaxf(r, 0.f), 15.f) : 0;
    }
    void* back = kind == 1 ? a.k_out : a.v_out;
    if (back) {
        float z[8];
        const float base = __uint_as_float(lo_bits << 16);
#pragma unroll
        for (int i = 0; i < 8; ++i) z[i] = base + step * (float)code[i];
        st16(static_cast<bf16_t*>(back) + t * (kind == 1 ? a.k_out_stride : a.v_out_stride) + (int64_t)h * D + 8 * c,
             pack(z, bf16_t{}));
    }
    const int slab = 2 * h + (kind == 2), r = pos % kKvBlock;
    const int page = kv_page(b, s, pos / kKvBlock, slab);
    if (page < 0) return;   // a page outside the pool: the row is not kept
    uint8_t* at = b.pages + page * b.page_bytes + (slab % b.slabs_per_page) * kv_slab_bytes(D);
    if (kind == 1) {
        uint32_t w = 0;
#pragma unroll
        for (int k = 0; k < 4; ++k) w |= (uint32_t)code[2 * k] << (4 * k) | (uint32_t)code[2 * k + 1] << (4 * k + 16);
        *reinterpret_cast<uint32_t*>(at + r * (D / 2) + 4 * c) = w;
    } else {
        constexpr int NH = D / 64;
#pragma unroll
        for (int g = 0; g < 2; ++g) {
            uint32_t w = 0;
#pragma unroll
            for (int k = 0; k < 4; ++k) w |= (uint32_t)code[4 * g + k] << (4 * k);
            const int q4 = 2 * c + g;
            *reinterpret_cast<uint16_t*>(at + (q4 / NH) * (D / 2) + (r / 2) * (D / 16) + (q4 % NH) * 4 + (r % 2) * 2) =
                (uint16_t)w;
        }
    }
    if (c == 0) *reinterpret_cast<uint32_t*>(at + 8 * D + 4 * r) = step_bits | lo_bits << 16;
}

// ---------------------------------------------------------------- attention: the work's cut

// Every workgroup finds its own piece of work from the device's lengths, so the launch does
// not depend on them (a captured call follows them).  Sequences are cut into row tiles of RB
// query rows and into parts of C steps of 32 tokens, C the same for all, so that about
// kKvUnits parts come out (but no part is shorter than min_steps).
enum KvClass { kKvAll = 0, kKvFew = 1, kKvMany = 2 };   // sequences: all, of at most kKvRowTile query rows, of more

struct KvCut {
    int rb, cls, min_steps;
};

struct KvUnit {
    int s, h, tile, part, parts, slot;   // slot: this part's (or the first part's) place in the workspace
    int steps_per_part;
    KvSeq q;
};

__device__ __forceinline__ int kv_tiles(const KvArgs& b, const KvCut& cut, const KvSeq& q) {
    const int64_t rows = (int64_t)q.rows * b.group;
    if (rows == 0 || (cut.cls == kKvFew && rows > kKvRowTile) || (cut.cls == kKvMany && rows <= kKvRowTile)) return 0;
    return (int)((rows + cut.rb - 1) / cut.rb);
}

__device__ __forceinline__ int kv_steps(int tokens) { return (tokens + 31) >> 5; }

// Unit `index` of the cut (merge: unit `index` of the row tiles, its first part's slot).
// Every thread of the 256 calls it; false past the last unit.
__device__ __forceinline__ bool kv_find(const KvArgs& b, const KvCut& cut, int64_t index, bool merge, KvUnit* u) {
    __shared__ int64_t sums[4][2];
    __shared__ int found[4];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    int64_t work = 0;
    for (int s = threadIdx.x; s < b.n_seqs; s += 256) {
        const KvSeq q = kv_seq(b, s);
        work += (int64_t)kv_tiles(b, cut, q) * kv_steps(q.len);
    }
#pragma unroll
    for (int m = 32; m >= 1; m >>= 1) work += __shfl_xor(work, m, 64);
    if (lane == 0) sums[wave][0] = work;
    if (threadIdx.x == 0) found[0] = -1;
    __syncthreads();
    work = (sums[0][0] + sums[1][0] + sums[2][0] + sums[3][0]) * b.kv_heads;
    const int64_t per = max((work + kKvUnits - 1) / kKvUnits, (int64_t)cut.min_steps);
    const int C = (int)min(per, (int64_t)(1 << 30));
    const int h = (int)(index % b.kv_heads);
    const int64_t want = index / b.kv_heads;
    int64_t base = 0, slot_base = 0;   // units and slots of the sequences before this round's
    for (int s0 = 0; s0 < b.n_seqs; s0 += 256) {
        const int s = s0 + threadIdx.x;
        KvSeq q{0, 0, 0};
        int tiles = 0, parts = 1;
        if (s < b.n_seqs) {
            q = kv_seq(b, s);
            tiles = kv_tiles(b, cut, q);
            parts = max(1, (kv_steps(q.len) + C - 1) / C);
        }
        const int64_t n = (int64_t)tiles * (merge ? 1 : parts), k = parts > 1 ? (int64_t)tiles * parts : 0;
        int64_t in = n, ik = k;   // inclusive sums over the wave, then over the workgroup
#pragma unroll
        for (int m = 1; m < 64; m <<= 1) {
            const int64_t a = __shfl_up(in, m, 64), c = __shfl_up(ik, m, 64);
            if (lane >= m) {
                in += a;
                ik += c;
            }
        }
        __syncthreads();   // (the sums of the round before have been read)
        if (lane == 63) {
            sums[wave][0] = in;
            sums[wave][1] = ik;
        }
        __syncthreads();
        int64_t all = 0, allk = 0;
#pragma unroll
        for (int w = 0; w < 4; ++w) {
            if (w < wave) {
                in += sums[w][0];
                ik += sums[w][1];
            }
            all += sums[w][0];
            allk += sums[w][1];
        }
        const int64_t mine = want - base - (in - n);
        if (mine >= 0 && mine < n) {
            found[0] = s;
            found[1] = (int)mine;
            found[2] = parts;
            found[3] = (int)((slot_base + ik - k + (merge ? mine * parts : mine)) * b.kv_heads + h);
        }
        base += all;
        slot_base += allk;
        if (want < base) break;
    }
    __syncthreads();
    if (found[0] < 0) return false;
    u->s = found[0];
    u->h = h;
    u->parts = found[2];
    u->tile = merge ? found[1] : found[1] / u->parts;
    u->part = merge ? 0 : found[1] % u->parts;
    u->slot = found[3];
    u->steps_per_part = C;
    u->q = kv_seq(b, u->s);
    return true;
}

// ---------------------------------------------------------------- attention: one wave

// The two bf16 halves 16 + code of nibble k of both 16-bit halves of w: a nibble in the top
// four bits of bf16's seven mantissa bits counts ones above 16, so the codes need no
// conversion, only their place.
__device__ __forceinline__ uint32_t code_pair(uint32_t w, int k) {
    const uint32_t s = k == 0 ? w << 3 : k == 1 ? w >> 1 : k == 2 ? w >> 5 : w >> 9;
    return (s & 0x00780078u) | 0x41804180u;
}

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

template <int W>
__device__ __forceinline__ void ld_words(const uint8_t* p, uint32_t (&o)[W]) {
    if constexpr (W == 2) {
        const u32x2 v = *reinterpret_cast<const u32x2*>(p);
        o[0] = v[0];
        o[1] = v[1];
    } else {
#pragma unroll
        for (int j = 0; j < W / 4; ++j) {
            const u32x4 v = ld16(p + 16 * j);
#pragma unroll
            for (int i = 0; i < 4; ++i) o[4 * j + i] = v[i];
        }
    }
}

// One step's keys and values of a wave: two slabs of each.
template <int D>
struct KvTile {
    static constexpr int W = D / 32;
    uint32_t k[2][W], v[2][W];
    u32x4 kw[2], vw[2];
};

// A wave's 16 query rows against tokens, 32 at a time.  Lane (li, lg) = (lane % 16, lane / 16)
// holds everything of query row li: of the scores those of tokens 4 lg .. 4 lg + 3 of both
// slabs, of the output the values 4 lg D / 16 .. + D / 4.
//   scores   S^T = K Q^T: matrix operations on the codes themselves (16 + code, exact in bf16),
//            then s = step * (acc - 16 sum(q)) + lo * sum(q), all fp32
//   weights  p = 2^(c s - m); m is raised, and everything summed so far scaled down, only
//            when a score passes it by more than 8 (the sums' scale needs no closer bound)
//   output   O^T += V^T P'^T with P' = p step in two bf16 halves (high and the rest, so its
//            error is 2^-17, below fp32 sums' worth of tokens) and V's codes as 16 + code;
//            z = sum p (lo - 16 step) takes the rest
template <int D>
struct KvWave {
    static constexpr int W = D / 32, NE = D / 16;
    uint32_t q[W][4];
    float qsum;
    f32x4 o[NE];
    float m, l, z;
    int limit;          // tokens this lane's row sees
    int limit_all;      // tokens every row of the tile sees

    __device__ __forceinline__ void load_q(const KvArgs& b, const KvUnit& u, const bf16_t* qp, int64_t stride, int row0) {
        const int lane = threadIdx.x & 63, li = lane & 15, lg = lane >> 4;
        const int rows = u.q.rows * b.group;
        const int r = row0 + li;
        qsum = 0.f;
        if (r < rows) {
            const bf16_t* p = qp + (int64_t)(u.q.r0 + r / b.group) * stride +
                              (int64_t)(u.h * b.group + r % b.group) * D + lg * (D / 4);
#pragma unroll
            for (int s = 0; s < W; ++s) {
                const u32x4 v = ld16(p + 8 * s);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    q[s][i] = v[i];
                    qsum += bf16_lo(v[i]) + bf16_hi(v[i]);
                }
            }
        } else {
#pragma unroll
            for (int s = 0; s < W; ++s)
#pragma unroll
                for (int i = 0; i < 4; ++i) q[s][i] = 0;
        }
        qsum = sum_lg(qsum);
        const int first = u.q.len - u.q.rows + 1;   // tokens the sequence's first row sees
        limit = r < rows ? first + r / b.group : 0;
        limit_all = first + row0 / b.group;
        m = -INFINITY;
        l = z = 0.f;
#pragma unroll
        for (int e = 0; e < NE; ++e) o[e] = f32x4{0.f, 0.f, 0.f, 0.f};
    }

    __device__ __forceinline__ void step(const KvTile<D>& t, int tok0, int bad, int len, float c) {
        const int lg = (threadIdx.x & 63) >> 4;
        f32x4 sc[2];
#pragma unroll
        for (int a = 0; a < 2; ++a) {
            const float init = -16.f * qsum;
            sc[a] = f32x4{init, init, init, init};
#pragma unroll
            for (int s = 0; s < W; ++s) {
                u32x4 kf, qf;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    kf[i] = code_pair(t.k[a][s], i);
                    qf[i] = q[s][i];
                }
                sc[a] = mma_step(kf, qf, sc[a], bf16_t{});
            }
        }
        float st[2][4], zp[2][4];
#pragma unroll
        for (int a = 0; a < 2; ++a)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                sc[a][i] = (sc[a][i] * bf16_lo(t.kw[a][i]) + bf16_hi(t.kw[a][i]) * qsum) * c;
                st[a][i] = bf16_lo(t.vw[a][i]);
                zp[a][i] = bf16_hi(t.vw[a][i]) - 16.f * st[a][i];
            }
        if (tok0 + 32 > limit_all || bad) {
            // tokens that a row does not see count nothing, whatever the pages hold there
#pragma unroll
            for (int a = 0; a < 2; ++a)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int tok = tok0 + 16 * a + 4 * lg + i;
                    if (tok >= limit || ((bad >> a) & 1)) {
                        sc[a][i] = -INFINITY;
                        st[a][i] = 0.f;
                        zp[a][i] = 0.f;
                    }
                }
        }
        float top = sc[0][0];
#pragma unroll
        for (int a = 0; a < 2; ++a)
#pragma unroll
            for (int i = 0; i < 4; ++i) top = fmaxf(top, sc[a][i]);
        if (__ballot(top > m + 8.f)) {
            const float mn = fmaxf(m, max_lg(top));
            const float al = mn == -INFINITY ? 1.f : __builtin_amdgcn_exp2f(m - mn);
            m = mn;
            l *= al;
            z *= al;
#pragma unroll
            for (int e = 0; e < NE; ++e)
#pragma unroll
                for (int i = 0; i < 4; ++i) o[e][i] *= al;
        }
        const float ref = m == -INFINITY ? 0.f : m;
        u32x4 ph, pl;
#pragma unroll
        for (int a = 0; a < 2; ++a)
#pragma unroll
            for (int i = 0; i < 4; i += 2) {
                const float p0 = __builtin_amdgcn_exp2f(sc[a][i] - ref), p1 = __builtin_amdgcn_exp2f(sc[a][i + 1] - ref);
                l += p0;
                l += p1;
                z = fmaf(p0, zp[a][i], z);
                z = fmaf(p1, zp[a][i + 1], z);
                const float w0 = p0 * st[a][i], w1 = p1 * st[a][i + 1];
                const uint32_t hi = pack_bf16(w0, w1);
                ph[2 * a + i / 2] = hi;
                pl[2 * a + i / 2] = pack_bf16(w0 - bf16_lo(hi), w1 - bf16_hi(hi));
            }
#pragma unroll
        for (int e = 0; e < NE; ++e) {
            constexpr int NH = W / 2;
            u32x4 vf;
#pragma unroll
            for (int a = 0; a < 2; ++a)
#pragma unroll
                for (int p = 0; p < 2; ++p) vf[2 * a + p] = code_pair(t.v[a][p * NH + e / 4], e % 4);
            o[e] = mma_step(vf, ph, o[e], bf16_t{});
            o[e] = mma_step(vf, pl, o[e], bf16_t{});
        }
    }

    // steps first, first + stride, ... below end
    __device__ __forceinline__ void run(const KvArgs& b, const KvUnit& u, int first, int end, int stride, float c) {
        const int lane = threadIdx.x & 63, li = lane & 15, lg = lane >> 4;
        const int n = end > first ? (end - first + stride - 1) / stride : 0;
        const int lane_off = li * (D / 2) + lg * (D / 8);
        const int ks = 2 * u.h, vs = 2 * u.h + 1;
        const int64_t koff = (int64_t)(ks % b.slabs_per_page) * kv_slab_bytes(D);
        const int64_t voff = (int64_t)(vs % b.slabs_per_page) * kv_slab_bytes(D);
        const int last_block = (u.q.len - 1) / kKvBlock;
        KvTile<D> t[2];
        int bad[2] = {0, 0};
        int pk = 0, pv = 0;   // lane 2 j + a: pages of slab a of step j of the 32 steps at hand
        auto pages = [&](int j0) {
            const int st = first + (j0 + (lane >> 1)) * stride;
            const int blk = 2 * st + (lane & 1);
            pk = pv = -1;
            if (j0 + (lane >> 1) < n && blk <= last_block) {
                pk = kv_page(b, u.s, blk, ks);
                pv = kv_page(b, u.s, blk, vs);
            }
        };
        auto load = [&](int j, KvTile<D>& d, int& bd) {
            bd = 0;
#pragma unroll
            for (int a = 0; a < 2; ++a) {
                const int k = __builtin_amdgcn_readlane(pk, (2 * j + a) & 63);
                const int v = __builtin_amdgcn_readlane(pv, (2 * j + a) & 63);
                if (k < 0 || v < 0) bd |= 1 << a;
                const uint8_t* kp = b.pages + max(k, 0) * b.page_bytes + koff;
                const uint8_t* vp = b.pages + max(v, 0) * b.page_bytes + voff;
                ld_words(kp + lane_off, d.k[a]);
                d.kw[a] = ld16(kp + 8 * D + 16 * lg);
                ld_words(vp + lane_off, d.v[a]);
                d.vw[a] = ld16(vp + 8 * D + 16 * lg);
            }
        };
        if (n == 0) return;
        pages(0);
        load(0, t[0], bad[0]);
        for (int j = 0; j < n; j += 2) {
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                if (j + x >= n) break;
                if (j + x + 1 < n) {
                    if (((j + x + 1) & 31) == 0) pages(j + x + 1);
                    load((j + x + 1) & 31, t[1 - x], bad[1 - x]);
                }
                step(t[x], 32 * (first + (j + x) * stride), bad[x], u.q.len, c);
            }
        }
    }

    __device__ __forceinline__ void finish() {
        l = sum_lg(l);
        z = sum_lg(z);
    }
};

// Where row r of a tile's results go: the output, or the unit's slot of the workspace.
struct KvOut {
    bf16_t* out;
    int64_t stride;
    float* part;   // [slots][RB][D], then [slots][RB][2]
};

template <int D, int RB>
__device__ __forceinline__ float* part_row(float* part, int slot, int r) {
    return part + ((int64_t)slot * RB + r) * D;
}
template <int D, int RB>
__device__ __forceinline__ float* part_ml(float* part, int slot, int r) {
    return part + (int64_t)kKvSlots * RB * D + ((int64_t)slot * RB + r) * 2;
}

// Few query rows: the four waves share a part's tokens, step by step in turn, and their sums
// meet in LDS.  Bound by reading the cache once.
template <int D>
__global__ __launch_bounds__(256) void kv_decode_kernel(KvArgs b, const bf16_t* q, int64_t q_stride, KvOut w, float c,
                                                        KvCut cut) {
    __shared__ float so[4][16][D + 4];
    __shared__ float sm[4][16][3];
    KvUnit u;
    if (!kv_find(b, cut, blockIdx.x, false, &u)) return;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, li = lane & 15, lg = lane >> 4;
    const int rows = u.q.rows * b.group, row0 = u.tile * 16;
    KvWave<D> wv;
    wv.load_q(b, u, q, q_stride, row0);
    // steps up to the last token that the tile's last row sees
    const int last = min(rows, row0 + 16) - 1;
    const int seen = max(0, u.q.len - u.q.rows + 1 + last / b.group);
    const int s0 = u.part * u.steps_per_part, s1 = min(kv_steps(seen), s0 + u.steps_per_part);
    wv.run(b, u, s0 + wave, s1, 4, c);
    wv.finish();
    if (lg == 0) {
        sm[wave][li][0] = wv.m;
        sm[wave][li][1] = wv.l;
        sm[wave][li][2] = wv.z;
    }
    constexpr int NE = D / 16;
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int e = 0; e < NE; e += 4) {
            const f32x4 v{wv.o[e][i], wv.o[e + 1][i], wv.o[e + 2][i], wv.o[e + 3][i]};
            *reinterpret_cast<f32x4*>(&so[wave][li][(4 * lg + i) * NE + e]) = v;
        }
    __syncthreads();
    // 16 threads a row, D / 16 values each
    const int r = threadIdx.x >> 4, d0 = (threadIdx.x & 15) * NE;
    if (row0 + r >= rows) return;
    float m = -INFINITY;
#pragma unroll
    for (int x = 0; x < 4; ++x) m = fmaxf(m, sm[x][r][0]);
    const float ref = m == -INFINITY ? 0.f : m;
    float l = 0.f, acc[NE];
#pragma unroll
    for (int e = 0; e < NE; ++e) acc[e] = 0.f;
#pragma unroll
    for (int x = 0; x < 4; ++x) {
        // (a wave whose tokens were all masked has m = -inf and sums of zero)
        const float f = sm[x][r][0] == -INFINITY ? (sm[x][r][1] == 0.f ? 0.f : 1.f) : __builtin_amdgcn_exp2f(sm[x][r][0] - ref);
        l += f * sm[x][r][1];
#pragma unroll
        for (int e = 0; e < NE; ++e) acc[e] += f * (so[x][r][d0 + e] + sm[x][r][2]);
    }
    if (u.parts > 1) {
        float* p = part_row<D, kKvRowTile>(w.part, u.slot, r) + d0;
#pragma unroll
        for (int e = 0; e < NE; e += 4) *reinterpret_cast<f32x4*>(p + e) = f32x4{acc[e], acc[e + 1], acc[e + 2], acc[e + 3]};
        if (d0 == 0) {
            float* ml = part_ml<D, kKvRowTile>(w.part, u.slot, r);
            ml[0] = m;
            ml[1] = l;
        }
        return;
    }
    const float inv = l == 0.f ? 0.f : 1.f / l;   // a row that sees no token is zero
    bf16_t* o = w.out + (int64_t)(u.q.r0 + (row0 + r) / b.group) * w.stride +
                (int64_t)(u.h * b.group + (row0 + r) % b.group) * D + d0;
#pragma unroll
    for (int e = 0; e < NE; e += 4) {
        u32x2 v;
        v[0] = pack_bf16(acc[e] * inv, acc[e + 1] * inv);
        v[1] = pack_bf16(acc[e + 2] * inv, acc[e + 3] * inv);
        *reinterpret_cast<u32x2*>(o + e) = v;
    }
}

// Many query rows: each of the four waves has 16 of the tile's 64 rows and goes over all the
// part's tokens.
template <int D>
__global__ __launch_bounds__(256) void kv_prefill_kernel(KvArgs b, const bf16_t* q, int64_t q_stride, KvOut w, float c,
                                                         KvCut cut) {
    KvUnit u;
    if (!kv_find(b, cut, blockIdx.x, false, &u)) return;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, li = lane & 15, lg = lane >> 4;
    const int rows = u.q.rows * b.group, row0 = u.tile * kKvPrefillRows + 16 * wave;
    if (row0 >= rows) return;
    KvWave<D> wv;
    wv.load_q(b, u, q, q_stride, row0);
    const int last = min(rows, row0 + 16) - 1;
    const int seen = max(0, u.q.len - u.q.rows + 1 + last / b.group);
    const int s0 = u.part * u.steps_per_part, s1 = min(kv_steps(seen), s0 + u.steps_per_part);
    wv.run(b, u, s0, s1, 1, c);
    wv.finish();
    const int r = row0 + li;
    if (r >= rows) return;
    constexpr int NE = D / 16;
    const int rt = 16 * wave + li;
    if (u.parts > 1) {
        float* p = part_row<D, kKvPrefillRows>(w.part, u.slot, rt);
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int e = 0; e < NE; e += 4)
                *reinterpret_cast<f32x4*>(p + (4 * lg + i) * NE + e) =
                    f32x4{wv.o[e][i] + wv.z, wv.o[e + 1][i] + wv.z, wv.o[e + 2][i] + wv.z, wv.o[e + 3][i] + wv.z};
        if (lg == 0) {
            float* ml = part_ml<D, kKvPrefillRows>(w.part, u.slot, rt);
            ml[0] = wv.m;
            ml[1] = wv.l;
        }
        return;
    }
    const float inv = wv.l == 0.f ? 0.f : 1.f / wv.l;
    bf16_t* o = w.out + (int64_t)(u.q.r0 + r / b.group) * w.stride + (int64_t)(u.h * b.group + r % b.group) * D;
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int e = 0; e < NE; e += 4) {
            u32x2 v;
            v[0] = pack_bf16((wv.o[e][i] + wv.z) * inv, (wv.o[e + 1][i] + wv.z) * inv);
            v[1] = pack_bf16((wv.o[e + 2][i] + wv.z) * inv, (wv.o[e + 3][i] + wv.z) * inv);
            *reinterpret_cast<u32x2*>(o + (4 * lg + i) * NE + e) = v;
        }
}

// The parts of a row tile, in part order.
template <int D, int RB>
__global__ __launch_bounds__(256) void kv_merge_kernel(KvArgs b, KvOut w, KvCut cut) {
    KvUnit u;
    if (!kv_find(b, cut, blockIdx.x, true, &u) || u.parts < 2) return;
    const int rows = u.q.rows * b.group, row0 = u.tile * RB;
    constexpr int TPR = D / 4;   // threads a row, four values each
    for (int r = threadIdx.x / TPR; r < RB && row0 + r < rows; r += 256 / TPR) {
        const int d0 = (threadIdx.x % TPR) * 4;
        float m = -INFINITY;
        for (int p = 0; p < u.parts; ++p) m = fmaxf(m, part_ml<D, RB>(w.part, u.slot + p * b.kv_heads, r)[0]);
        const float ref = m == -INFINITY ? 0.f : m;
        float l = 0.f;
        f32x4 acc{0.f, 0.f, 0.f, 0.f};
        for (int p = 0; p < u.parts; ++p) {
            const float* ml = part_ml<D, RB>(w.part, u.slot + p * b.kv_heads, r);
            const f32x4 v = *reinterpret_cast<const f32x4*>(part_row<D, RB>(w.part, u.slot + p * b.kv_heads, r) + d0);
            const float f = ml[0] == -INFINITY ? (ml[1] == 0.f ? 0.f : 1.f) : __builtin_amdgcn_exp2f(ml[0] - ref);
            l += f * ml[1];
#pragma unroll
            for (int i = 0; i < 4; ++i) acc[i] += f * v[i];
        }
        const float inv = l == 0.f ? 0.f : 1.f / l;
        u32x2 o;
        o[0] = pack_bf16(acc[0] * inv, acc[1] * inv);
        o[1] = pack_bf16(acc[2] * inv, acc[3] * inv);
        *reinterpret_cast<u32x2*>(w.out + (int64_t)(u.q.r0 + (row0 + r) / b.group) * w.stride +
                                  (int64_t)(u.h * b.group + (row0 + r) % b.group) * D + d0) = o;
    }
}

template <int D>
hipError_t attention(const KvArgs& b, const bf16_t* q, int64_t q_stride, bf16_t* out, int64_t out_stride, float scale,
                     int32_t max_rows, void* workspace, hipStream_t s) {
    const float c = scale * 1.44269504088896341f;
    KvOut w{out, out_stride, static_cast<float*>(workspace)};
    const int64_t rows = (int64_t)b.n_rows * b.group;
    auto go = [&](int rb, int cls, auto kern, auto merge) {
        // tiles, and parts beyond the first of each
        const int64_t tiles = (rows / rb + b.n_seqs) * b.kv_heads;
        const KvCut cut{rb, cls, 4};
        hipLaunchKernelGGL(kern, dim3((unsigned)(tiles + kKvUnits)), dim3(256), 0, s, b, q, q_stride, w, c, cut);
        // (a sequence of at most min_steps steps is never cut)
        if (b.max_blocks * kKvBlock > 32 * cut.min_steps)
            hipLaunchKernelGGL(merge, dim3((unsigned)tiles), dim3(256), 0, s, b, w, cut);
    };
    if ((int64_t)max_rows * b.group <= kKvRowTile) {
        go(kKvRowTile, kKvAll, kv_decode_kernel<D>, kv_merge_kernel<D, kKvRowTile>);
    } else {
        go(kKvRowTile, kKvFew, kv_decode_kernel<D>, kv_merge_kernel<D, kKvRowTile>);
        go(kKvPrefillRows, kKvMany, kv_prefill_kernel<D>, kv_merge_kernel<D, kKvPrefillRows>);
    }
    return hipGetLastError();
}

}  // namespace

hipError_t launch_kv_append(int head_dim, const KvArgs& b, const KvAppendArgs& a, hipStream_t s) {
    const int64_t items = (int64_t)b.n_rows * ((a.q ? b.heads : 0) + 2 * b.kv_heads);
    auto go = [&](auto kern, int per_block) {
        const int64_t grid = (items + per_block - 1) / per_block;
        if (grid > INT32_MAX) return hipErrorInvalidValue;
        hipLaunchKernelGGL(kern, dim3((unsigned)grid), dim3(256), 0, s, b, a);
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
