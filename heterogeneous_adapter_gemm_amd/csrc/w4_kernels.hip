// The shared base product with a 4-bit base weight: y[M][N] = sum_k x[m][k] *
// scale[n][k / group] * (code[n][k] - zero[n][k / group]), bf16 x, 4-bit codes
// [N][K / 2] (even k in the low half of its byte), fp16 scale and zero per
// group of 32, 64 or 128 consecutive k, fp32 accumulation.
//
// The matrix cores run bf16 on the codes themselves: a nibble put in the top
// four bits of bf16's mantissa stands for 16 + code exactly, so two codes need a
// multiplication and one and-or, and no rounding.  Per group, fp32: y += scale * acc -
// scale * (16 + zero) * sum(x): the second term is one fp32 matrix operation of
// each lane's own sum of its x.
//
// A lane of a matrix operation has a row of x (a row of codes) and its share of
// a group's k, consecutive ones: group / 4 of them where four lanes share a row
// (16-row operations), group / 2 where two do (32-row operations).
#include "bgmv_device.h"
#include "common.h"
#include "internal.h"

#include <type_traits>

namespace hagemm {
namespace {

typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef float f32x16 __attribute__((ext_vector_type(16)));

// The codes of w as bf16, 16 + code each, in their order: a byte times 2^3 + 2^15 has its low nibble in
// bits 3 to 6 and its high one in bits 19 to 22 (one instruction, the byte chosen in it).  The constants
// in registers: a three-operand and-or takes none of its own.
struct CodeConst {
    uint32_t mul = 0x8008u, mask = 0x00780078u, ones = 0x41804180u;
    __device__ __forceinline__ CodeConst() { asm volatile("" : "+v"(mul), "+v"(mask), "+v"(ones)); }
};
__device__ __forceinline__ u32x4 code_values(const CodeConst& c, uint32_t w) {
    u32x4 v;
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = (__umul24((w >> (8 * i)) & 255u, c.mul) & c.mask) | c.ones;
    return v;
}

// s plus the eight x of v
__device__ __forceinline__ float add_x(const u32x4& v, float s) {
    const bf16x2 one = __builtin_bit_cast(bf16x2, 0x3F803F80u);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t w = v[i];   // (a bit cast of v[i] itself reads v[0])
        s = __builtin_amdgcn_fdot2_f32_bf16(__builtin_bit_cast(bf16x2, w), one, s, false);
    }
    return s;
}

__device__ __forceinline__ f32x16 mma32(const u32x4& a, const u32x4& b, f32x16 c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0,
                                                   0);
}

__device__ __forceinline__ float half_lo(uint32_t w) { return (float)__builtin_bit_cast(_Float16, (uint16_t)w); }
__device__ __forceinline__ float half_hi(uint32_t w) { return (float)__builtin_bit_cast(_Float16, (uint16_t)(w >> 16)); }

// A group's scale, and what its zero point and the codes' 16 take away per unit of x.  (The scale in
// a register of its own: as a half inside a multiply-add it costs the longer instruction.)
struct Scale {
    float scale, corr;
    __device__ __forceinline__ explicit Scale(uint32_t w) {
        scale = half_lo(w);
        asm volatile("" : "+v"(scale));
        corr = -scale * (16.f + half_hi(w));
    }
};

template <int W>
__device__ __forceinline__ void ld_words(const uint8_t* p, uint32_t (&o)[W]) {
    if constexpr (W == 1) {
        o[0] = *reinterpret_cast<const uint32_t*>(p);
    } else if constexpr (W == 2) {
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

// y[m][n] = v; of a row with an adapter (its bit in raw_mask, or row_slot where that is 0) to ybase, unrounded
struct Out {
    bf16_t* y;
    float* ybase;
    const int32_t* row_slot;
    uint64_t raw_mask;
    __device__ __forceinline__ void put(int m, int n, int N, float v) const {
        const int64_t off = (int64_t)m * N + n;
        if (raw_mask ? m < 64 && raw_mask >> m & 1 : row_slot != nullptr && row_slot[m] >= 0)
            ybase[off] = v;
        else
            y[off].bits = (uint16_t)f32_to_bf16(v);
    }
    // columns n .. n + 3
    __device__ __forceinline__ void put4(int m, int n, int N, const f32x4& v) const {
        const int64_t off = (int64_t)m * N + n;
        if (raw_mask ? m < 64 && raw_mask >> m & 1 : row_slot != nullptr && row_slot[m] >= 0)
            *reinterpret_cast<f32x4*>(ybase + off) = v;
        else
            *reinterpret_cast<u32x2*>(y + off) = u32x2{pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3])};
    }
};

// ---------------------------------------------------------------- up to 16 rows

// One workgroup per 16 columns of y: its eight waves take the 128-deep pieces of K in turn (the
// codes and x of the next three in flight), and their sums meet in LDS in wave
// order.  Bound by reading the codes once; at a few microseconds, by the latency of that: one row
// 4096 -> 4096 5.9 us on MI355X, 1.5 TB/s of codes.
constexpr int kRowWaves = 8;

template <int G>
__device__ __forceinline__ void rows_tile(const bf16_t* __restrict__ x, const uint8_t* __restrict__ q,
                                          const uint32_t* __restrict__ sz, const Out& out, int M, int N, int K, int bx) {
    __shared__ float part[kRowWaves][4][64];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, li = lane & 15, lg = lane >> 4;
    const int n0 = bx * 16, n = min(n0 + li, N - 1);
    constexpr int NG = 128 / G, W = G / 32;   // groups of a piece; words (and steps) of a group a lane
    const uint8_t* qn = q + (int64_t)n * (K / 2) + lg * (G / 8);
    const uint32_t* sn = sz + (int64_t)n * (K / G);
    const bf16_t* xm = x + (int64_t)min(li, M - 1) * K + lg * (G / 4);
    const bool row = li < M;
    const CodeConst cc;
    struct Codes {
        uint32_t c[NG][W], s[NG];
    };
    struct Rows {
        u32x4 x[NG][W];
    };
    auto load = [&](int kb, Codes& p) {
#pragma unroll
        for (int g = 0; g < NG; ++g) {
            ld_words(qn + (kb + g * G) / 2, p.c[g]);
            p.s[g] = sn[kb / G + g];
        }
    };
    auto load_x = [&](int kb, Rows& p) {
#pragma unroll
        for (int g = 0; g < NG; ++g)
#pragma unroll
            for (int t = 0; t < W; ++t) {
                p.x[g][t] = u32x4{0, 0, 0, 0};
                if (row) p.x[g][t] = ld16(xm + kb + g * G + 8 * t);
            }
    };
    f32x4 acc{0.f, 0.f, 0.f, 0.f};
    constexpr int PF = 4, kStep = 128 * kRowWaves;
    Codes p[PF];
    Rows r[PF];
    const int k0 = wave * 128, last = K - 128;
#pragma unroll
    for (int i = 0; i < PF; ++i) {
        load(min(k0 + i * kStep, last), p[i]);
        load_x(min(k0 + i * kStep, last), r[i]);
    }
    for (int kb0 = k0; kb0 < K; kb0 += PF * kStep) {
#pragma unroll
        for (int i = 0; i < PF; ++i) {
            const int kb = kb0 + i * kStep;
            if (kb >= K) break;
            const Codes now = p[i];
            const Rows xr = r[i];
            if (kb + PF * kStep < K) {
                load(kb + PF * kStep, p[i]);
                load_x(kb + PF * kStep, r[i]);
            }
#pragma unroll
            for (int g = 0; g < NG; ++g) {
                const float sc = half_lo(now.s[g]), corr = -sc * (16.f + half_hi(now.s[g]));
                f32x4 d{0.f, 0.f, 0.f, 0.f};
                float xs = 0.f;
#pragma unroll
                for (int t = 0; t < W; ++t) {
                    const u32x4 v = xr.x[g][t];
                    d = mma_step(v, code_values(cc, now.c[g][t]), d, bf16_t{});
                    xs = add_x(v, xs);
                }
                acc = __builtin_amdgcn_mfma_f32_16x16x4f32(settled(xs), corr, acc, 0, 0, 0);
#pragma unroll
                for (int j = 0; j < 4; ++j) acc[j] = fmaf(sc, d[j], acc[j]);
            }
        }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) part[wave][i][lane] = acc[i];
    __syncthreads();
    if (wave < 4) {
        // wave i: rows 4 lg + i
        float v = 0.f;
#pragma unroll
        for (int w = 0; w < kRowWaves; ++w) v += part[w][wave][lane];
        const int m = 4 * lg + wave;
        if (m < M && n0 + li < N) out.put(m, n0 + li, N, v);
    }
}

// ---------------------------------------------------------------- 32-row operations

// Codes and scales of a piece of 32 NB columns, a lane's own.
template <int G, int NB>
struct W4Cols {
    static constexpr int NG = 128 / G, S = G / 16;   // groups of a piece; steps (words a lane) of a group
    struct Codes {
        uint32_t c[NB][NG][S], s[NB][NG];
    };
    const uint8_t* qn[NB];
    const uint32_t* sn[NB];

    __device__ __forceinline__ W4Cols(const uint8_t* q, const uint32_t* sz, int n0, int N, int K) {
        const int lane = threadIdx.x & 63, lr = lane & 31, hg = lane >> 5;
#pragma unroll
        for (int b = 0; b < NB; ++b) {
            const int64_t n = min(n0 + 32 * b + lr, N - 1);
            qn[b] = q + n * (K / 2) + hg * (G / 4);
            sn[b] = sz + n * (K / G);
        }
    }
    __device__ __forceinline__ void load(int kb, Codes& p) const {
#pragma unroll
        for (int b = 0; b < NB; ++b)
#pragma unroll
            for (int g = 0; g < NG; ++g) {
                ld_words(qn[b] + (kb + g * G) / 2, p.c[b][g]);
                p.s[b][g] = sn[b][kb / G + g];
            }
    }
};

// x rows in LDS: [row][16 chunks of 16 bytes], chunk i of row r in slot i ^ (r % 16), so that the
// rows of a read differ in their banks.  A wave-load fills four rows.
__device__ __forceinline__ void load_rows(const bf16_t* x, int m0, int M, int K, int kb, uint8_t* lds, int first, int count) {
    const int lane = threadIdx.x & 63;
    for (int i = 0; i < count; ++i) {
        const int r = first + 4 * i + (lane >> 4), slot = lane & 15;
        const int m = min(m0 + r, M - 1);
        global_load_lds16(x + (int64_t)m * K + kb + (slot ^ (r & 15)) * 8, lds + (first + 4 * i) * 256);
    }
}

// What a piece takes away for its zero points, one fp32 matrix operation for a pair of groups: it has
// room for two depths, a lane half each, the two halves' sums of one group or the whole sums of two.
template <int G, int NB>
struct Taken {
    static constexpr int NP = G == 32 ? 2 : 1;
    float sum[NP], corr[NP][NB];   // of this lane's row and group; of its column and group
};

// One 128-deep piece of a wave's 64 x 32 NB: acc[a][b] += rows row[a] of x (LDS at xs) times columns 32 b,
// but for the zero points; out: those of rows row[0].
template <int G, int NB>
__device__ __forceinline__ void mul_piece(const uint8_t* xs, const int (&row)[2], const typename W4Cols<G, NB>::Codes& p,
                                          const CodeConst& cc, f32x16 (&acc)[2][NB], Taken<G, NB>& out) {
    constexpr int NG = 128 / G, S = G / 16;
    const int hg = (threadIdx.x & 63) >> 5;
    float sum0 = 0.f, corr0[NB];   // (of the group before)
#pragma unroll
    for (int b = 0; b < NB; ++b) corr0[b] = 0.f;
#pragma unroll
    for (int g = 0; g < NG; ++g) {
        f32x16 d[2][NB];
        float sum = 0.f;
#pragma unroll
        for (int a = 0; a < 2; ++a)
#pragma unroll
            for (int b = 0; b < NB; ++b)
#pragma unroll
                for (int i = 0; i < 16; ++i) d[a][b][i] = 0.f;
#pragma unroll
        for (int t = 0; t < S; ++t) {
            u32x4 cf[NB];
#pragma unroll
            for (int b = 0; b < NB; ++b) cf[b] = code_values(cc, p.c[b][g][t]);
#pragma unroll
            for (int a = 0; a < 2; ++a) {
                const u32x4 v = ld16(xs + row[a] * 256 + ((g * (G / 8) + hg * S + t) ^ (row[a] & 15)) * 16);
                if (a == 0) sum = add_x(v, sum);
#pragma unroll
                for (int b = 0; b < NB; ++b) d[a][b] = mma32(v, cf[b], d[a][b]);
            }
        }
        sum = settled(sum);
        if (NG > 1 && g % 2) {
            const auto h = __builtin_amdgcn_permlane32_swap(__float_as_uint(sum0), __float_as_uint(sum), false, false);
            out.sum[g / 2] = __uint_as_float(h[0]) + __uint_as_float(h[1]);
        } else if (NG == 1) {
            out.sum[0] = sum;
        }
        sum0 = sum;
#pragma unroll
        for (int b = 0; b < NB; ++b) {
            const Scale sc(p.s[b][g]);
            out.corr[g / 2][b] = NG > 1 && hg == 0 ? corr0[b] : sc.corr;
            corr0[b] = sc.corr;
#pragma unroll
            for (int a = 0; a < 2; ++a)
#pragma unroll
                for (int i = 0; i < 16; ++i) acc[a][b][i] = fmaf(sc.scale, d[a][b][i], acc[a][b][i]);
        }
    }
}

// Row of register i of a 32 x 32 block
__device__ __forceinline__ int row32(int i) { return 8 * (i / 4) + 4 * ((threadIdx.x & 63) >> 5) + i % 4; }

// Decode batches: 32 MB rows by 32 NB columns a workgroup, its eight waves taking the 128-deep
// pieces of K in turn, in halves, each with its own place for x in LDS (two halves, the next one in
// flight) and no barrier until their sums meet there.  Two waves a SIMD, so that one's conversions run
// beside the other's matrix operations (300 vector instructions for a piece of 64 x 64, 36 matrix
// operations).  Bound by the latency of x from L2, half a step of it open, and by the tiles' number where
// they leave compute units without one: 4096 -> 11008 has 172 for 256, vector instructions issue in 38 % of a
// SIMD's cycles and matrix operations in 17 %.  Measured on MI355X, 64 rows: 4096 -> 11008 16 us, 4096 -> 4096
// 8.5 us; of the 16, 2 until the first x is there, 2 for the sums of the waves.  (Four waves with whole
// pieces took 20 us; reading a word of each column's codes four pieces ahead 20 us.)
constexpr int kDecodeWaves = 8;

template <int G, int MB, int NB>
__device__ __forceinline__ void decode_tile(const bf16_t* __restrict__ x, const uint8_t* __restrict__ q,
                                            const uint32_t* __restrict__ sz, const Out& out, int M, int N, int K, int bx,
                                            int by) {
    constexpr int kRows = 32 * MB, kStage = kRows * 128, W = kDecodeWaves;
    constexpr int GH = G < 64 ? G : 64, NG = 64 / GH, S = GH / 16;   // group's part of a half, parts of a half, steps of a part
    constexpr int kSums = MB * NB * 16 * 256;                       // a wave's sums
    constexpr int kLds = 2 * kStage > kSums ? 2 * kStage : kSums;
    __shared__ __attribute__((aligned(1024))) uint8_t lds[W * kLds];
    const int lane = threadIdx.x & 63, lr = lane & 31, hg = lane >> 5;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int n0 = bx * 32 * NB, m0 = by * kRows;
    const CodeConst cc;
    uint8_t* place = lds + wave * 2 * kStage;
    const uint8_t* qn[NB];
    const uint32_t* sn[NB];
#pragma unroll
    for (int b = 0; b < NB; ++b) {
        const int64_t c = min(n0 + 32 * b + lr, N - 1);
        qn[b] = q + c * (K / 2) + hg * (GH / 4);
        sn[b] = sz + c * (K / G);
    }
    // x: a wave-load fills eight rows of 64 values; 16-byte chunk i of row r in slot i ^ (r / 2 % 8)
    const bf16_t* xl[4 * MB];
#pragma unroll
    for (int i = 0; i < 4 * MB; ++i) {
        const int r = 8 * i + (lane >> 3);
        xl[i] = x + (int64_t)min(m0 + r, M - 1) * K + ((lane & 7) ^ ((r >> 1) & 7)) * 8;
    }
    struct Codes {
        uint32_t c[NB][NG][S], s[NB][NG];
    };
    auto issue = [&](int kb, int half, Codes& p) {
#pragma unroll
        for (int i = 0; i < 4 * MB; ++i) global_load_lds16(xl[i] + kb, place + half * kStage + i * 1024);
#pragma unroll
        for (int b = 0; b < NB; ++b)
#pragma unroll
            for (int g = 0; g < NG; ++g) {
                ld_words(qn[b] + (kb + g * GH) / 2, p.c[b][g]);
                p.s[b][g] = sn[b][(kb + g * GH) / G];
            }
    };
    f32x16 acc[MB][NB], d[MB][NB];
    float sum[MB];
#pragma unroll
    for (int a = 0; a < MB; ++a)
#pragma unroll
        for (int b = 0; b < NB; ++b)
#pragma unroll
            for (int i = 0; i < 16; ++i) acc[a][b][i] = 0.f;
    auto work = [&](int half, const Codes& p) {
        const uint8_t* xs = place + half * kStage;
#pragma unroll
        for (int g = 0; g < NG; ++g) {
            if (G <= 64 || half == 0) {
#pragma unroll
                for (int a = 0; a < MB; ++a) {
                    sum[a] = 0.f;
#pragma unroll
                    for (int b = 0; b < NB; ++b)
#pragma unroll
                        for (int i = 0; i < 16; ++i) d[a][b][i] = 0.f;
                }
            }
#pragma unroll
            for (int t = 0; t < S; ++t) {
                u32x4 cf[NB];
#pragma unroll
                for (int b = 0; b < NB; ++b) cf[b] = code_values(cc, p.c[b][g][t]);
#pragma unroll
                for (int a = 0; a < MB; ++a) {
                    const u32x4 v = ld16(xs + (32 * a + lr) * 128 + ((g * (GH / 8) + hg * S + t) ^ ((lr >> 1) & 7)) * 16);
                    sum[a] = add_x(v, sum[a]);
    #pragma unroll
                    for (int b = 0; b < NB; ++b) d[a][b] = mma32(v, cf[b], d[a][b]);
                }
            }
            if (G <= 64 || half == 1) {
#pragma unroll
                for (int a = 0; a < MB; ++a) sum[a] = settled(sum[a]);
#pragma unroll
                for (int b = 0; b < NB; ++b) {
                    const Scale sc(p.s[b][g]);
#pragma unroll
                    for (int a = 0; a < MB; ++a) {
                        acc[a][b] = __builtin_amdgcn_mfma_f32_32x32x2f32(sum[a], sc.corr, acc[a][b], 0, 0, 0);
#pragma unroll
                        for (int i = 0; i < 16; ++i) acc[a][b][i] = fmaf(sc.scale, d[a][b][i], acc[a][b][i]);
                    }
                }
            }
        }
    };
    const int n = (K / 128 - wave + W - 1) / W;   // pieces of this wave
    // (each 64 columns begin at a piece of their own, so that not all workgroups read one slice of x at
    // once; by the columns, so that every kind of tile has the same sums)
    const int shift = n > 0 ? (n0 >> 6) % n : 0;
    auto at = [&](int j) { return (wave + W * (j + shift < n ? j + shift : j + shift - n)) * 128; };
    Codes p[2];
    if (n > 0) issue(at(0), 0, p[0]);
#pragma unroll 1
    for (int j = 0; j < n; ++j) {
        const int kb = at(j);
        wait_vmcnt<0>();
        wait_lgkm0();   // (likewise the second's, a piece ago)
        issue(kb + 64, 1, p[1]);
        work(0, p[0]);
        wait_vmcnt<0>();
        wait_lgkm0();   // the first half's place has been read
        if (j + 1 < n) issue(at(j + 1), 0, p[0]);
        work(1, p[1]);
    }
    // the waves' sums: [wave][block][i][lane]
    __syncthreads();
    float* part = reinterpret_cast<float*>(lds);
#pragma unroll
    for (int a = 0; a < MB; ++a)
#pragma unroll
        for (int b = 0; b < NB; ++b)
#pragma unroll
            for (int i = 0; i < 16; ++i) part[wave * (kSums / 4) + ((a * NB + b) * 16 + i) * 64 + lane] = acc[a][b][i];
    __syncthreads();
    // four columns of a row a thread (N is a multiple of four)
#pragma unroll
    for (int e = threadIdx.x; e < MB * NB * 256; e += 64 * W) {
        const int reg = e >> 4, l4 = (e & 15) * 4, blk = reg >> 4, i = reg & 15;
        f32x4 v{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int w = 0; w < W; ++w) v += *reinterpret_cast<const f32x4*>(part + w * (kSums / 4) + reg * 64 + l4);
        const int m = m0 + 32 * (blk / NB) + 8 * (i / 4) + 4 * (l4 >> 5) + i % 4, c = n0 + 32 * (blk % NB) + (l4 & 31);
        if (m < M && c < N) out.put4(m, c, N, v);
    }
}

// One decode tile: rows (up to 16, up to 32, or blocks of 64) and columns by its kind
enum DecodeKind { kRows16, kRows32, kRows64, kRows64Wide };
template <int G, int KIND>
__device__ __forceinline__ void any_tile(const bf16_t* __restrict__ x, const uint8_t* __restrict__ q,
                                         const uint32_t* __restrict__ sz, const Out& out, int M, int N, int K, int bx, int by) {
    if constexpr (KIND == kRows16) rows_tile<G>(x, q, sz, out, M, N, K, bx);
    else if constexpr (KIND == kRows32) decode_tile<G, 1, 1>(x, q, sz, out, M, N, K, bx, by);
    else if constexpr (KIND == kRows64) decode_tile<G, 2, 1>(x, q, sz, out, M, N, K, bx, by);
    else decode_tile<G, 2, 2>(x, q, sz, out, M, N, K, bx, by);
}
constexpr int kTileThreads = 64 * kDecodeWaves;
static_assert(kRowWaves == kDecodeWaves, "one workgroup size for every kind");
constexpr int tile_rows(int kind) { return kind == kRows16 ? 16 : kind == kRows32 ? 32 : 64; }
constexpr int tile_columns(int kind) { return kind == kRows16 ? 16 : kind == kRows64Wide ? 64 : 32; }

template <int G, int KIND>
__global__ __launch_bounds__(kTileThreads, 2) void gemm_w4_decode_kernel(const bf16_t* __restrict__ x,
                                                                         const uint8_t* __restrict__ q,
                                                                         const uint32_t* __restrict__ sz, Out out, int M,
                                                                         int N, int K) {
    any_tile<G, KIND>(x, q, sz, out, M, N, K, blockIdx.x, blockIdx.y);
}

// Decode batches of up to 64 rows with adapters: the tiles, the BGMV shrink's units (two a
// workgroup) and the copy of a plan's index in one launch.  Measured on MI355X, 64 rows 4096 -> 4096, the
// whole call: 16 adapters of rank 16 15.4 us, 64 of rank 64 29.3 us (21.5 and 36.3 with a launch of their own
// for the units).
template <int G, int KIND>
__global__ __launch_bounds__(kTileThreads, 2) void gemm_w4_shrink_kernel(
    const bf16_t* __restrict__ x, const uint8_t* __restrict__ q, const uint32_t* __restrict__ sz, Out out, int M, int N, int K,
    LoraArgs a, int n_gemm, int n_cols, int n_unit, const uint32_t* __restrict__ cp_src, uint32_t* __restrict__ cp_dst, int cp_n) {
    const int b = blockIdx.x;
    if (b < n_gemm) {
        any_tile<G, KIND>(x, q, sz, out, M, N, K, b % n_cols, b / n_cols);
    } else if (b < n_gemm + n_unit) {
        const int wave = threadIdx.x >> 6;
        bgmv_shrink_unit<bf16_t, true>(a, 2 * (b - n_gemm) + wave / 4, a.lp_per_rank, a.v, wave % 4);
    } else if (threadIdx.x < 256) {
        copy_words(cp_src, cp_dst, cp_n, b - n_gemm - n_unit);
    }
}

// Long batches: 128 x 64 NB of y a workgroup, 64 x 32 NB a wave; the 128-deep pieces of x go to LDS
// once for the four waves, one piece ahead.  Bound by the vector units and the matrix cores, which
// share their issue: of 320 instructions for a piece of 64 x 64 128 put codes in place, 128 scale two
// groups' sums, 32 sum x, beside 36 matrix operations.  Measured on MI355X: 2,961 x 4096 x 4096 in groups of
// 64 143 us back to back, 0.69 PFLOP/s; 4,096 x 4096 x 11008 in groups of 128 450 us, 0.82 PFLOP/s.
template <int G, int NB>
__device__ __forceinline__ void long_tile(const bf16_t* __restrict__ x, const uint8_t* __restrict__ q,
                                          const uint32_t* __restrict__ sz, const Out& out, int M, int N, int K, int m0,
                                          int col0, uint8_t* lds0, uint8_t* lds1, float (*zs)[4][2][64]) {
    using Cols = W4Cols<G, NB>;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int n0 = col0 + (wave & 1) * 32 * NB;
    // two waves share 64 rows: either sums the x of the half that it calls its first
    const int half = 32 * (wave & 1), r0 = (wave >> 1) * 64 + half, r1 = (wave >> 1) * 64 + (half ^ 32);
    const int lane = threadIdx.x & 63, row[2] = {r0 + (lane & 31), r1 + (lane & 31)};
    const Cols cols(q, sz, n0, N, K);
    const CodeConst cc;
    f32x16 acc[2][NB];
#pragma unroll
    for (int a = 0; a < 2; ++a)
#pragma unroll
        for (int b = 0; b < NB; ++b)
#pragma unroll
            for (int i = 0; i < 16; ++i) acc[a][b][i] = 0.f;
    const int n = K / 128;
    typename Cols::Codes p[2];
    auto issue = [&](int j, uint8_t* to, typename Cols::Codes& c) {
        load_rows(x, m0, M, K, j * 128, to, 32 * wave, 8);
        cols.load(j * 128, c);
    };
    // the zero points of the piece before, its sums now there from both waves
    Taken<G, NB> taken;
    auto take = [&](int u) {
#pragma unroll
        for (int i = 0; i < taken.NP; ++i) {
            const float other = zs[u][wave ^ 1][i][lane];
#pragma unroll
            for (int b = 0; b < NB; ++b) {
                acc[0][b] = __builtin_amdgcn_mfma_f32_32x32x2f32(taken.sum[i], taken.corr[i][b], acc[0][b], 0, 0, 0);
                acc[1][b] = __builtin_amdgcn_mfma_f32_32x32x2f32(other, taken.corr[i][b], acc[1][b], 0, 0, 0);
            }
        }
    };
    issue(0, lds0, p[0]);
#pragma unroll 1
    for (int j = 0; j < n; j += 2) {
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            if (j + u >= n) break;
            wait_vmcnt<0>();
            wait_lgkm0();
            __builtin_amdgcn_s_barrier();   // every wave's rows are there, and the other place is read
            landed();
            if (j + u + 1 < n) issue(j + u + 1, u ? lds0 : lds1, p[1 - u]);
            if (j + u > 0) take(1 - u);
            mul_piece<G, NB>(u ? lds1 : lds0, row, p[u], cc, acc, taken);
#pragma unroll
            for (int i = 0; i < taken.NP; ++i) zs[u][wave][i][lane] = taken.sum[i];
        }
    }
    wait_lgkm0();
    __builtin_amdgcn_s_barrier();
    landed();
    take((n - 1) & 1);
#pragma unroll
    for (int a = 0; a < 2; ++a)
#pragma unroll
        for (int b = 0; b < NB; ++b)
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                const int m = m0 + (a ? r1 : r0) + row32(i), c = n0 + 32 * b + (threadIdx.x & 31);
                if (m < M && c < N) out.put(m, c, N, acc[a][b][i]);
            }
}

constexpr int kLongSlots = 512;   // workgroups of the long kernel that run at once

template <int G>
__global__ __launch_bounds__(256, 2) void gemm_w4_long_kernel(const bf16_t* __restrict__ x, const uint8_t* __restrict__ q,
                                                              const uint32_t* __restrict__ sz, Out out, int M, int N, int K,
                                                              int whole) {
    __shared__ __attribute__((aligned(1024))) uint8_t lds0[128 * 256];
    __shared__ __attribute__((aligned(1024))) uint8_t lds1[128 * 256];
    __shared__ float zs[2][4][2][64];
    const int row_blocks = (M + 127) / 128, col_blocks = (N + 127) / 128, b = blockIdx.x;
    const int part = b < whole ? 0 : xcd_logical(b - whole, gridDim.x - whole);
    const int lid = b < whole ? xcd_logical(b, whole) : whole + part / 2;
    // strips of four row blocks, a column block after another (a block of x has four times the bytes
    // of a block of codes: so the tiles that run at once share most of either)
    const int strip = lid / (4 * col_blocks), in = lid - strip * 4 * col_blocks, high = min(4, row_blocks - 4 * strip);
    const int m0 = (4 * strip + in % high) * 128, n0 = (in / high) * 128;
    if (b < whole) long_tile<G, 2>(x, q, sz, out, M, N, K, m0, n0, lds0, lds1, zs);
    else if (n0 + 64 * (part & 1) < N) long_tile<G, 1>(x, q, sz, out, M, N, K, m0, n0 + 64 * (part & 1), lds0, lds1, zs);
}

}  // namespace

bool gemm_w4_ok(int64_t M, int64_t N, int64_t K, int32_t group) {
    if (group != 32 && group != 64 && group != 128) return false;
    if (M < 1 || N < 1 || N % 4 || K < 128 || K % 128) return false;
    return M * K * 2 < INT32_MAX && N * K / 2 < INT32_MAX;
}

static int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }
// Blocks of 32 rows where every tile then has a compute unit of its own (each reads all of its rows' x; 64
// rows: 4096 -> 4096 8.5 us for 11.4 with blocks of 64, 11008 -> 4096 17 (24), but 4096 -> 6144 13.5 (11.6));
// `others` workgroups beside them need one too (with 40 of BGMV units 4096 -> 4096 takes 14.5 us for 12).
// Else blocks of 64, 64 columns wide where 32 would take a second round (64 rows 4096 -> 11008 17 us so, 22 with
// 32 columns; 4096 -> 4096 12 with 32 columns, 18 with 64).
static DecodeKind decode_kind(int64_t M, int64_t N, int64_t others) {
    if (M <= 16) return kRows16;
    if (M <= 32 || cdiv(M, 32) * cdiv(N, 32) + others <= 256) return kRows32;
    return cdiv(M, 64) * cdiv(N, 32) > 256 ? kRows64Wide : kRows64;
}

// f(integral_constant group, integral_constant kind)
template <typename F>
static hipError_t with_kind(int32_t group, DecodeKind kind, F&& f) {
    auto k = [&](auto g) {
        switch (kind) {
            case kRows16: return f(g, std::integral_constant<int, kRows16>{});
            case kRows32: return f(g, std::integral_constant<int, kRows32>{});
            case kRows64: return f(g, std::integral_constant<int, kRows64>{});
            default: return f(g, std::integral_constant<int, kRows64Wide>{});
        }
    };
    return group == 128  ? k(std::integral_constant<int, 128>{})
           : group == 64 ? k(std::integral_constant<int, 64>{})
                         : k(std::integral_constant<int, 32>{});
}

hipError_t launch_gemm_w4(const void* x, const void* q, const void* sz, int32_t group, void* y, int64_t M, int64_t N,
                          int64_t K, const int32_t* row_slot, float* ybase, hipStream_t s) {
    if (!gemm_w4_ok(M, N, K, group)) return hipErrorInvalidValue;
    const bf16_t* xb = static_cast<const bf16_t*>(x);
    const uint8_t* qb = static_cast<const uint8_t*>(q);
    const uint32_t* zb = static_cast<const uint32_t*>(sz);
    const Out out{static_cast<bf16_t*>(y), ybase, row_slot, 0};
    auto go = [&](auto kern, int64_t gx, int64_t gy, int threads) {
        if (gx > INT32_MAX || gy > 65535) return hipErrorInvalidValue;
        hipLaunchKernelGGL(kern, dim3((unsigned)gx, (unsigned)gy), dim3(threads), 0, s, xb, qb, zb, out, (int)M, (int)N, (int)K);
        return hipGetLastError();
    };
    const int64_t tiles = cdiv(M, 128) * cdiv(N, 128);
    // From about four rounds of the decode tiles on the long ones (4096 inputs in groups of 128: 512 x 4096 31 us
    // in decode tiles, 35 in long ones, 768 x 4096 45 (50), 300 x 11008 64 (79), 384 x 11008 75 (78), 1,024 x 4096 59
    // (54), 520 x 11008 100 (86)).
    if (M > 64 && cdiv(M, 64) * cdiv(N, 64) >= 1024) {
        // Whole tiles in rounds, and a last round that would leave most places empty as halves of 64 columns,
        // 4096 x 4096 in groups of 128: 256 tiles 54 us for 59, 384 81 (85), 448 97 (86); behind a whole round
        // 640 117 us for 131, 736 135 (135), and in groups of 64 768 171 (168).
        const int64_t rest = tiles % kLongSlots, most = tiles < kLongSlots ? kLongSlots * 3 / 4 : kLongSlots * 3 / 8;
        const int64_t whole = rest <= most ? tiles - rest : tiles;
        const int64_t grid = whole + 2 * (tiles - whole);
        if (grid > INT32_MAX) return hipErrorInvalidValue;
        auto run = [&](auto kern) {
            hipLaunchKernelGGL(kern, dim3((unsigned)grid), dim3(256), 0, s, xb, qb, zb, out, (int)M, (int)N, (int)K, (int)whole);
            return hipGetLastError();
        };
        return group == 128 ? run(gemm_w4_long_kernel<128>) : group == 64 ? run(gemm_w4_long_kernel<64>) : run(gemm_w4_long_kernel<32>);
    }
    const DecodeKind kind = decode_kind(M, N, 0);
    return with_kind(group, kind, [&](auto g, auto k) {
        return go(gemm_w4_decode_kernel<g.value, k.value>, cdiv(N, tile_columns(kind)), cdiv(M, tile_rows(kind)), kTileThreads);
    });
}

bool gemm_w4_shrink_fits(int64_t M, int64_t N, int64_t K, int32_t group, int n_su) {
    return M >= 1 && M <= 64 && n_su > 0 && gemm_w4_ok(M, N, K, group);
}

hipError_t launch_gemm_w4_shrink(const void* x, const void* q, const void* sz, int32_t group, void* y, int64_t M, int64_t N,
                                 int64_t K, const int32_t* row_slot, uint64_t raw_mask, float* ybase, const LoraArgs& a,
                                 const void* cp_src, void* cp_dst, int64_t cp_n, hipStream_t s) {
    if (!gemm_w4_shrink_fits(M, N, K, group, a.n_su) || cp_n < 0 || cp_n > INT32_MAX) return hipErrorInvalidValue;
    const Out out{static_cast<bf16_t*>(y), ybase, row_slot, raw_mask};
    const int nu = (a.n_su + 1) / 2, ncp = cp_n > 0 ? kCopyBlocks : 0;
    const DecodeKind kind = decode_kind(M, N, nu + ncp);
    const int tn = (int)cdiv(N, tile_columns(kind)), tiles = tn * (int)cdiv(M, tile_rows(kind));
    return with_kind(group, kind, [&](auto g, auto k) {
        hipLaunchKernelGGL((gemm_w4_shrink_kernel<g.value, k.value>), dim3((unsigned)(tiles + nu + ncp)), dim3(kTileThreads), 0, s,
                           static_cast<const bf16_t*>(x), static_cast<const uint8_t*>(q), static_cast<const uint32_t*>(sz), out,
                           (int)M, (int)N, (int)K, a, tiles, tn, nu, static_cast<const uint32_t*>(cp_src),
                           static_cast<uint32_t*>(cp_dst), (int)cp_n);
        return hipGetLastError();
    });
}

}  // namespace hagemm
