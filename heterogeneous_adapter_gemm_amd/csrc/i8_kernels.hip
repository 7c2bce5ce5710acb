// The shared base product in 8-bit integers (gfx950): y[m][n] = xs[m] ws[n] sum_k xc[m][k] wc[n][k], x in
// int8 codes with a scale a row, the base weight in int8 codes [N][K] with a scale an output channel.  The
// sums are exact (int32: K <= 131056, so fewer than 2^17 products of 2^14), so they do not depend on how K is split;
// each is converted to fp32 once, scaled, and rounded to bf16 once.
//
// The gated form takes two weights and writes act(g) u of the two products, unrounded until then.
//
// The integer matrix operations do twice the work of the bf16 ones per byte and instruction.  Both operands
// run along K, so a lane's 16 bytes of a row feed one 16 x 16 x 64 step; w is on the operation's M side and x on
// its N side, and a lane ends with four consecutive output columns of one row.
//
//  * i8_stream_kernel (up to 256 rows): bound by reading w once.  A workgroup of four waves holds a tile of
//    16 FM rows x 16 FN columns (gated: 8 FN of each weight); wave v takes every fourth slice of 128 K, streams
//    both operands' rows of its slices through an LDS ring of its own, and holds a whole tile of partial sums.
//    So no wave waits for another until the end, where the four partial tiles are added in LDS.
//  * i8_long_kernel (more rows): bound by the matrix operations and the feed of the tiles.  256 x 256 (or 192 x
//    256) tiles, eight waves, four stages of 64 K, fragments read one step ahead; the prefill segments'
//    expand in the epilogue.
//
// Both load straight into LDS, by buffers of a tile's own rows of one matrix: rows past M or N read as zeros, no
// offset passes 32 bits, and columns past K are asked for past the buffer's end and read as zeros too.
#include <type_traits>

#include "act_device.h"
#include "bgmv_device.h"
#include "common.h"
#include "expand_device.h"
#include "i8.h"
#include "internal.h"

namespace hagemm {
namespace {

typedef int32_t i32x4 __attribute__((ext_vector_type(4)));

__device__ __forceinline__ i32x4 mma_i8(const u32x4& a, const u32x4& b, i32x4 c) {
    return __builtin_amdgcn_mfma_i32_16x16x64_i8(__builtin_bit_cast(i32x4, a), __builtin_bit_cast(i32x4, b), c, 0, 0, 0);
}

// past the end of every buffer below (each is at most 64 rows: 8 MiB)
constexpr int kPastEnd = (int)0x80000000u;

template <typename T>
__device__ __forceinline__ const T* uniform(const T* p) {
    const uint64_t v = reinterpret_cast<uint64_t>(p);
    const uint32_t lo = __builtin_amdgcn_readfirstlane((uint32_t)v), hi = __builtin_amdgcn_readfirstlane((uint32_t)(v >> 32));
    return reinterpret_cast<const T*>(((uint64_t)hi << 32) | lo);
}

// `rows` rows of K bytes from row r0 of a matrix of `all` rows: where they start, and how many bytes exist
struct RowBuf {
    const int8_t* p;
    int bytes;
};
__device__ __forceinline__ RowBuf rows_of(const void* m, int r0, int rows, int all, int K) {
    const int have = max(0, min(rows, all - r0));
    return {uniform(static_cast<const int8_t*>(m) + (have ? (int64_t)r0 * K : 0)), __builtin_amdgcn_readfirstlane(have * K)};
}

// the four outputs of a lane: row m, columns n .. n + 3
template <int ACT>
__device__ __forceinline__ f32x4 gated(const f32x4& g, const f32x4& u) {
    f32x4 d;
#pragma unroll
    for (int i = 0; i < 4; ++i) d[i] = activate<ACT>(g[i]) * u[i];
    return d;
}

__device__ __forceinline__ f32x4 scaled(const i32x4& a, float xs, const f32x4& ws) {
    f32x4 d;
#pragma unroll
    for (int i = 0; i < 4; ++i) d[i] = (float)a[i] * xs * ws[i];
    return d;
}

__device__ __forceinline__ void put4(const I8Args& g, bool raw, int m, int n, const f32x4& d) {
    const int64_t off = (int64_t)m * g.N + n;
    if (raw) {
        *reinterpret_cast<f32x4*>(g.ybase + off) = d;
    } else {
        u32x2 o;
        o[0] = pack_bf16(d[0], d[1]);
        o[1] = pack_bf16(d[2], d[3]);
        *reinterpret_cast<u32x2*>(static_cast<bf16_t*>(g.y) + off) = o;
    }
}

// ---------------------------------------------------------------------------
// Up to 256 rows.  ACT < 0: one weight.
template <int FM_, int FN_, int S_>
struct StreamCfg {
    static constexpr int FM = FM_, FN = FN_, S = S_;
    static constexpr int R = 16 * (FM + FN);      // rows of both operands a slice
    static constexpr int STG = 4 * R * 128;       // a stage: each wave's slice
    static_assert(S * STG <= 160 * 1024, "LDS");
};

template <class C, int ACT>
__device__ __forceinline__ void i8_stream_tile(const I8Args& g, int bid, int nblocks, uint64_t raw_mask) {
    constexpr int FM = C::FM, FN = C::FN, S = C::S, STG = C::STG;
    constexpr bool GATED = ACT >= 0;
    constexpr int FO = GATED ? FN / 2 : FN;       // 16-column blocks of the output
    constexpr int LX = 2 * FM, LW = 2 * FN, L = LX + LW;   // wave-loads (8 rows of 128 B) a slice
    static_assert(!GATED || FN % 2 == 0, "both weights");
    __shared__ __attribute__((aligned(1024))) uint8_t lds0[STG];
    __shared__ __attribute__((aligned(1024))) uint8_t lds1[STG];
    __shared__ __attribute__((aligned(1024))) uint8_t lds2[S > 2 ? STG : 16];
    __shared__ __attribute__((aligned(1024))) uint8_t lds3[S > 3 ? STG : 16];
    __shared__ __attribute__((aligned(1024))) uint8_t lds4[S > 4 ? STG : 16];
    __shared__ __attribute__((aligned(1024))) uint8_t lds5[S > 5 ? STG : 16];
    __shared__ __attribute__((aligned(1024))) uint8_t lds6[S > 6 ? STG : 16];
    __shared__ __attribute__((aligned(1024))) uint8_t lds7[S > 7 ? STG : 16];
    // one array a stage, so that the compiler sees that a stage being filled is not the one being read
    auto stage = [&](int st) -> uint8_t* {
        return st == 0 ? lds0 : st == 1 ? lds1 : st == 2 ? lds2 : st == 3 ? lds3 : st == 4 ? lds4 : st == 5 ? lds5 : st == 6 ? lds6 : lds7;
    };
    const int M = g.M, N = g.N, K = g.K;
    const int row_blocks = (M + 16 * FM - 1) / (16 * FM), tiles_n = nblocks / row_blocks;
    // the row blocks of a column tile run on one XCD, one after another: they read the same slab of w
    const int lid = xcd_logical(bid, nblocks);
    const int tn = lid / row_blocks, n0 = tn * 16 * FO, m0 = (lid % row_blocks) * 16 * FM;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int li = lane & 15, lg = lane >> 4;

    const RowBuf xb = rows_of(g.x, m0, 16 * FM, M, K), wb = rows_of(g.w, n0, 16 * FO, N, K);
    const RowBuf ub = GATED ? rows_of(g.w2, n0, 16 * FO, N, K) : wb;
    // lane -> row lane / 8 of a wave-load and 16-byte slot lane % 8; slot p of row r holds chunk p ^ ((r / 2) % 4 * 2),
    // which puts eight rows' chunks c and c + 1 in distinct banks
    const int chunk = ((lane & 7) ^ (((lane >> 3) >> 1 & 3) << 1)) * 16;
    const int voff = (lane >> 3) * K + chunk;
    const int nk = (K + 127) >> 7;      // slices
    const int steps = (nk + 3) >> 2;    // each wave's
    // each column tile starts at a slice of its own, so that not all read the same part of x at once
    const int shift = (int)(((int64_t)tn * steps) / tiles_n);
    auto issue = [&](int i, uint8_t* st) {
        int at = i + shift;
        if (at >= steps) at -= steps;
        // (past a wave's steps: nothing is read)
        const int kb = i < steps ? (at * 4 + wave) * 128 : K;
        const int off = kb + chunk < K ? voff : kPastEnd;
        uint8_t* mine = st + wave * (C::R * 128);
#pragma unroll
        for (int q = 0; q < LX; ++q) buffer_load_lds16(xb.p, xb.bytes, mine + q * 1024, off + 8 * q * K, kb);
#pragma unroll
        for (int q = 0; q < LW; ++q) {
            const bool up = GATED && q >= LW / 2;
            buffer_load_lds16(up ? ub.p : wb.p, up ? ub.bytes : wb.bytes, mine + (LX + q) * 1024,
                              off + 8 * (up ? q - LW / 2 : q) * K, kb);
        }
    };

    i32x4 acc[FN][FM];
#pragma unroll
    for (int a = 0; a < FN; ++a)
#pragma unroll
        for (int b = 0; b < FM; ++b) acc[a][b] = i32x4{0, 0, 0, 0};
    const int swz = ((li >> 1) & 3) << 1;
    auto step = [&](int i, int si) {
        // the slice's loads are done; those of the S - 1 later ones may not be
        wait_vmcnt<(S - 1) * L>();
        landed();
        const uint8_t* mine = stage(si) + wave * (C::R * 128) + li * 128;
        u32x4 xf[2][FM], wf[2][FN];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int off = ((4 * h + lg) ^ swz) * 16;
#pragma unroll
            for (int b = 0; b < FM; ++b) xf[h][b] = *reinterpret_cast<const u32x4*>(mine + b * 2048 + off);
#pragma unroll
            for (int a = 0; a < FN; ++a) wf[h][a] = *reinterpret_cast<const u32x4*>(mine + (FM + a) * 2048 + off);
        }
        // the fragments are in registers before the stage is filled again
        wait_lgkm0();
        issue(i + S, stage(si));
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int a = 0; a < FN; ++a)
#pragma unroll
                for (int b = 0; b < FM; ++b) acc[a][b] = mma_i8(wf[h][a], xf[h][b], acc[a][b]);
    };
#pragma unroll
    for (int p = 0; p < S; ++p) issue(p, stage(p));
    const int full = steps - steps % S;
    for (int i = 0; i < full; i += S) {
#pragma unroll
        for (int st = 0; st < S; ++st) step(i + st, st);
    }
#pragma unroll
    for (int st = 0; st < S - 1; ++st)
        if (full + st < steps) step(full + st, st);
    wait_vmcnt<0>();   // no load may still be writing LDS

    // the partial tiles meet in LDS: wave v's blocks in array v % S, and each wave adds every fourth block
    constexpr int PART = FM * FN * 1024;
    static_assert((3 / S + 1) * PART <= STG, "partial sums");
    __syncthreads();
    {
        i32x4* part = reinterpret_cast<i32x4*>(stage(wave % S) + (wave / S) * PART);
#pragma unroll
        for (int a = 0; a < FN; ++a)
#pragma unroll
            for (int b = 0; b < FM; ++b) part[(a * FM + b) * 64 + lane] = acc[a][b];
    }
    __syncthreads();
    auto total = [&](int blk) {
        i32x4 s = {0, 0, 0, 0};
#pragma unroll
        for (int v = 0; v < 4; ++v) s += reinterpret_cast<const i32x4*>(stage(v % S) + (v / S) * PART)[blk * 64 + lane];
        return s;
    };
    for (int o = wave; o < FO * FM; o += 4) {
        const int a = o / FM, b = o - a * FM;
        const int m = m0 + b * 16 + li, n = n0 + a * 16 + 4 * lg;
        if (m >= M || n >= N) continue;
        const float xs = g.xs[m];
        f32x4 d = scaled(total(o), xs, *reinterpret_cast<const f32x4*>(g.ws + n));
        if constexpr (GATED) d = gated<ACT>(d, scaled(total(o + FO * FM), xs, *reinterpret_cast<const f32x4*>(g.ws2 + n)));
        const bool raw = g.row_slot != nullptr ? g.row_slot[m] >= 0 : m < 64 && ((raw_mask >> m) & 1) != 0;
        put4(g, raw, m, n, d);
    }
}

template <class C, int ACT>
__global__ __launch_bounds__(256, 1) void i8_stream_kernel(I8Args g) {
    i8_stream_tile<C, ACT>(g, blockIdx.x, gridDim.x, 0);
}

// Decode batches of up to 64 rows with adapters: the product's tiles, the BGMV shrink's units and the copy
// of a plan's index in one launch (blocks [0, n_gemm) are tiles, then the shrink units, then kCopyBlocks
// copying cp_n index words), as for the other bases.
template <class C>
__global__ __launch_bounds__(256, 1) void i8_stream_shrink_kernel(I8Args g, uint64_t raw_mask, LoraArgs a, int n_gemm,
                                                                  const uint32_t* __restrict__ cp_src,
                                                                  uint32_t* __restrict__ cp_dst, int cp_n) {
    const int b = blockIdx.x;
    if (b < n_gemm)
        i8_stream_tile<C, -1>(g, b, n_gemm, raw_mask);
    else if (b < n_gemm + a.n_su)
        bgmv_shrink_unit<bf16_t, true>(a, b - n_gemm);
    else
        copy_words(cp_src, cp_dst, cp_n, b - n_gemm - a.n_su);
}

// ---------------------------------------------------------------------------
// More than 256 rows.  BM x BN tiles (of w's rows: a gated tile's are BN / 2 of each weight), or pieces of the
// UNIT_M x UNIT_N ones in the last round.
template <int BM_, int BN_, int UNIT_M_, int UNIT_N_>
struct LongCfg {
    static constexpr int BM = BM_, BN = BN_, UNIT_M = UNIT_M_, UNIT_N = UNIT_N_;
};
constexpr int kLongWM = 4, kLongWN = 2, kLongWaves = kLongWM * kLongWN, kLongStages = 4;

template <class C, int ACT, bool FUSE>
__global__ __launch_bounds__(kLongWaves * 64, 1) void i8_long_kernel(I8Args g, LoraArgs seg, int tiles_m, int tiles_n, int t0,
                                                                     int count) {
    constexpr int BM = C::BM, BN = C::BN, WM = kLongWM, WN = kLongWN, NW = kLongWaves, S = kLongStages;
    constexpr int SUB_M = C::UNIT_M / BM, SUB_N = C::UNIT_N / BN, SUBS = SUB_M * SUB_N;
    constexpr bool GATED = ACT >= 0;
    constexpr int WTM = BM / WM, WTN = BN / WN, FM = WTM / 16, FN = WTN / 16;
    constexpr int RB = 64;                                // bytes of a tile row per step
    constexpr int GX = BM / 16, GW = BN / 16, NL = GX + GW, L = (NL + NW - 1) / NW;   // wave-loads of 16 rows
    constexpr int SPARE = L * NW == NL ? 0 : 1024;        // where a wave left short loads nothing
    constexpr int XB = BM * RB, STAGE = (C::UNIT_M + C::UNIT_N) * RB + SPARE;
    static_assert(SUB_M * BM == C::UNIT_M && SUB_N * BN == C::UNIT_N && WTM % 16 == 0 && WTN % 32 == 0, "tile");
    static_assert(S * STAGE <= 160 * 1024 && !(GATED && FUSE), "LDS");
    __shared__ __attribute__((aligned(1024))) uint8_t lds0[STAGE];
    __shared__ __attribute__((aligned(1024))) uint8_t lds1[STAGE];
    __shared__ __attribute__((aligned(1024))) uint8_t lds2[STAGE];
    __shared__ __attribute__((aligned(1024))) uint8_t lds3[STAGE];
    auto stage = [&](int st) -> uint8_t* { return st == 0 ? lds0 : st == 1 ? lds1 : st == 2 ? lds2 : lds3; };
    const int M = g.M, N = g.N, K = g.K;

    // tiles in groups of 8 rows of tiles, consecutive ones on one XCD: they share slices of x and w in its L2
    const int bid = blockIdx.x;
    const int t = SUBS > 1 ? t0 + bid / SUBS : t0 + xcd_logical(bid, count);
    const int group = t / (8 * tiles_n), first_m = group * 8, gm = min(tiles_m - first_m, 8);
    const int in_group = t - group * 8 * tiles_n;
    const int tm = first_m + in_group % gm, tn = in_group / gm;
    const int piece = SUBS > 1 ? bid % SUBS : 0;
    // output columns of a tile: BN, or of a gated one BN / 2
    constexpr int ON = GATED ? BN / 2 : BN, UNIT_ON = GATED ? C::UNIT_N / 2 : C::UNIT_N;
    const int m0 = tm * C::UNIT_M + (piece / SUB_N) * BM, n0 = tn * UNIT_ON + (piece % SUB_N) * ON;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wm = wave / WN, wn = wave % WN;
    const int li = lane & 15, lg = lane >> 4;

    // this wave's loads: row block b of w's side is rows 16 b .. of the tile; each wave column's WTN of them are
    // (gated) first WTN / 2 rows of the gate's weight, then as many of the other's, of the same output columns
    RowBuf buf[L];
    int at[L];
#pragma unroll
    for (int q = 0; q < L; ++q) {
        const int b = q * NW + wave;
        if (b < GX) {
            buf[q] = rows_of(g.x, m0 + 16 * b, 16, M, K);
        } else if (b < NL) {
            const int r = 16 * (b - GX), in = r % WTN;
            const bool up = GATED && in >= WTN / 2;
            const int col = GATED ? (r / WTN) * (WTN / 2) + (up ? in - WTN / 2 : in) : r;
            buf[q] = rows_of(up ? g.w2 : g.w, n0 + col, 16, N, K);
        } else {
            buf[q] = {uniform(static_cast<const int8_t*>(g.x)), 0};
        }
        at[q] = b < NL ? b * 1024 : (C::UNIT_M + C::UNIT_N) * RB;
    }
    // lane -> row lane / 4 and slot lane % 4; slot p of row r holds chunk p ^ ((r / 2) % 4): fragment reads
    // are free of bank conflicts
    const int chunk = ((lane & 3) ^ ((lane >> 3) & 3)) * 16;
    const int voff = (lane >> 2) * K + chunk;
    auto issue = [&](int j, uint8_t* st) {
        const int kb = j * RB;      // (steps past the end read nothing)
        const int off = kb + chunk < K ? voff : kPastEnd;
#pragma unroll
        for (int q = 0; q < L; ++q) buffer_load_lds16(buf[q].p, buf[q].bytes, st + at[q], off, kb);
    };

    // (int32 sums until they are scaled, in place)
    f32x4 acc[FN][FM];
#pragma unroll
    for (int a = 0; a < FN; ++a)
#pragma unroll
        for (int b = 0; b < FM; ++b) acc[a][b] = f32x4{0.f, 0.f, 0.f, 0.f};
    const int foff = (lg ^ ((li >> 1) & 3)) * 16;
    auto read_frags = [&](const uint8_t* st, u32x4 (&wf)[FN], u32x4 (&xf)[FM]) {
        const uint8_t* bx = st + (wm * WTM + li) * RB + foff;
        const uint8_t* bw = st + XB + (wn * WTN + li) * RB + foff;
#pragma unroll
        for (int b = 0; b < FM; ++b) xf[b] = *reinterpret_cast<const u32x4*>(bx + b * 16 * RB);
#pragma unroll
        for (int a = 0; a < FN; ++a) wf[a] = *reinterpret_cast<const u32x4*>(bw + a * 16 * RB);
    };
    auto mma = [&](const u32x4 (&wf)[FN], const u32x4 (&xf)[FM]) {
#pragma unroll
        for (int a = 0; a < FN; ++a)
#pragma unroll
            for (int b = 0; b < FM; ++b)
                acc[a][b] = __builtin_bit_cast(f32x4, mma_i8(wf[a], xf[b], __builtin_bit_cast(i32x4, acc[a][b])));
    };
    // Fragments of step j + 1 are read while the matrix cores work on step j; step j + S is asked for in step
    // j's stage once every wave holds step j's fragments.  Whole groups of S steps: those past the end are zeros.
    u32x4 w0[FN], x0[FM], w1[FN], x1[FM];
    const int nk = (K + RB * S - 1) / (RB * S) * S;
#pragma unroll
    for (int p = 0; p < S; ++p) issue(p, stage(p));
    wait_vmcnt<(S - 1) * L>();
    __builtin_amdgcn_s_barrier();
    read_frags(stage(0), w0, x0);
    for (int i = 0; i < nk; i += S) {
#pragma unroll
        for (int st = 0; st < S; ++st) {
            __builtin_amdgcn_sched_barrier(0);
            // this wave's loads of the next step are done, and its fragment reads of this one
            wait_vmcnt_lgkm0<(S - 2) * L>();
            // every wave's are
            __builtin_amdgcn_s_barrier();
            __builtin_amdgcn_sched_barrier(0);
            issue(i + st + S, stage(st));
            if (st % 2 == 0) {
                read_frags(stage((st + 1) % S), w1, x1);
                mma(w0, x0);
            } else {
                read_frags(stage((st + 1) % S), w0, x0);
                mma(w1, x1);
            }
            // the loads, then each fragment read followed by two matrix operations
            __builtin_amdgcn_sched_group_barrier(0x020, L, 0);
#pragma unroll
            for (int q = 0; q < FN + FM; ++q) {
                __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
                __builtin_amdgcn_sched_group_barrier(0x008, 2, 0);
            }
        }
    }
    wait_vmcnt<0>();   // no load may still be writing LDS

    // lane holds D[n = 4 lg + i][m = li] of each block
#pragma unroll
    for (int b = 0; b < FM; ++b) {
        const int m = m0 + wm * WTM + b * 16 + li;
        const float xs = m < M ? g.xs[m] : 0.f;
#pragma unroll
        for (int a = 0; a < FN; ++a) {
            const bool up = GATED && a >= FN / 2;
            const int n = n0 + (GATED ? wn * (WTN / 2) + (up ? a - FN / 2 : a) * 16 : wn * WTN + a * 16) + 4 * lg;
            const f32x4 ws = n < N ? *reinterpret_cast<const f32x4*>((up ? g.ws2 : g.ws) + n) : f32x4{0.f, 0.f, 0.f, 0.f};
            acc[a][b] = scaled(__builtin_bit_cast(i32x4, acc[a][b]), xs, ws);
        }
    }
    if constexpr (FUSE) {
        static_assert(C::UNIT_N * kExpandRow * 2 <= STAGE && C::UNIT_M * kExpandRow * 2 <= STAGE, "the expand's operands");
        expand_segments<BM, BN, WM, WN>(seg, m0, n0, N, reinterpret_cast<uint16_t*>(lds0), reinterpret_cast<uint16_t*>(lds1),
                                        reinterpret_cast<uint16_t*>(lds2), acc);
    }
#pragma unroll
    for (int b = 0; b < FM; ++b) {
        const int m = m0 + wm * WTM + b * 16 + li;
        if (m >= M) continue;
        // rows whose delta comes later (decode rows with an adapter) stay unrounded
        const bool raw = g.row_slot != nullptr && g.row_slot[m] >= 0 && (!FUSE || m >= seg.T_pre);
#pragma unroll
        for (int a = 0; a < (GATED ? FN / 2 : FN); ++a) {
            const int n = n0 + (GATED ? wn * (WTN / 2) : wn * WTN) + a * 16 + 4 * lg;
            if (n >= N) continue;
            if constexpr (GATED) put4(g, raw, m, n, gated<ACT>(acc[a][b], acc[a + FN / 2][b]));
            else put4(g, raw, m, n, acc[a][b]);
        }
    }
}

using Long256 = LongCfg<256, 256, 256, 256>;
using Long256Half = LongCfg<256, 128, 256, 256>;
using Long256Quarter = LongCfg<128, 128, 256, 256>;
using Long256Eighth = LongCfg<128, 64, 256, 256>;
using Long256Sixteenth = LongCfg<64, 64, 256, 256>;
using Long192 = LongCfg<192, 256, 192, 256>;
using Long192Half = LongCfg<192, 128, 192, 256>;

template <int ACT, bool FUSE>
hipError_t run_long(const I8Args& g, const LoraArgs& seg, hipStream_t s) {
    // Tile height 256 or 192 by the estimated time of its rounds (one workgroup a compute unit), as for the
    // bf16 base; the partial last round runs as pieces of tiles.
    const int cus = gemm_cu_count(), on = ACT >= 0 ? 128 : 256;
    auto pieces = [&](int rem) { return rem * 16 <= cus ? 16 : rem * 8 <= cus ? 8 : rem * 4 <= cus ? 4 : 2; };
    auto plan = [&](int bm, int& tm, int& tn, int& rem) {
        tm = (g.M + bm - 1) / bm;
        tn = (g.N + on - 1) / on;
        const int tiles = tm * tn;
        rem = tiles > cus ? tiles % cus : 0;
        const double f = bm == 256 ? 1.0 : 0.85;
        if (tiles <= cus) return f * (1.0 - 0.58 * (1.0 - (double)tiles / cus));
        double tail = 0.0;
        if (rem) {
            const int p = bm == 256 ? pieces(rem) : 2;
            tail = p == 2 ? (bm == 256 ? 0.5 : 0.58) * ((2 * rem + cus - 1) / cus) : 1.5 / p;
        }
        return f * (tiles / cus + tail);
    };
    int tm, tn, rem, tm2, tn2, rem2;
    const bool tall = plan(256, tm, tn, rem) <= plan(192, tm2, tn2, rem2);
    if (!tall) {
        tm = tm2;
        tn = tn2;
        rem = rem2;
    }
    const int n_main = tm * tn - rem, np = tall && rem ? pieces(rem) : 2;
    auto go = [&](auto whole, auto piece) {
        hipLaunchKernelGGL(whole, dim3(n_main), dim3(kLongWaves * 64), 0, s, g, seg, tm, tn, 0, n_main);
        if (rem) hipLaunchKernelGGL(piece, dim3(np * rem), dim3(kLongWaves * 64), 0, s, g, seg, tm, tn, n_main, rem);
    };
    if (!tall) go(i8_long_kernel<Long192, ACT, FUSE>, i8_long_kernel<Long192Half, ACT, FUSE>);
    else if (np == 16) go(i8_long_kernel<Long256, ACT, FUSE>, i8_long_kernel<Long256Sixteenth, ACT, FUSE>);
    else if (np == 8) go(i8_long_kernel<Long256, ACT, FUSE>, i8_long_kernel<Long256Eighth, ACT, FUSE>);
    else if (np == 4) go(i8_long_kernel<Long256, ACT, FUSE>, i8_long_kernel<Long256Quarter, ACT, FUSE>);
    else go(i8_long_kernel<Long256, ACT, FUSE>, i8_long_kernel<Long256Half, ACT, FUSE>);
    return hipGetLastError();
}

// Stream tiles: rows in blocks of 16, 32 or 64, and the fewest columns that leave at most a tile a compute
// unit (w then streams through all of them in one round, and x is read as seldom as that allows).
template <class Go>
void stream_shape(const I8Args& g, bool two, Go go) {
    const int cus = gemm_cu_count();
    const int fm = g.M <= 16 ? 1 : g.M <= 32 ? 2 : 4;
    const int rb = (g.M + 16 * fm - 1) / (16 * fm);
    const int blocks = (g.N + 15) / 16 * (two ? 2 : 1);   // 16-row blocks of the weights
    int fn = two ? 2 : 1;
    while (fn < 4 && (int64_t)rb * ((blocks + fn - 1) / fn) > cus) fn += two ? 2 : 1;
    go(fm, fn, (unsigned)(rb * ((blocks + fn - 1) / fn)));
}

}  // namespace

bool gemm_i8_ok(int64_t M, int64_t N, int64_t K) {
    return M >= 1 && M <= kI8MaxRows && N >= 4 && N <= kI8MaxRows && N % 4 == 0 && K >= 16 && K <= kI8MaxK && K % 16 == 0;
}

namespace {

template <int FM, int FN>
using Stream = StreamCfg<FM, FN, (FM == 1 && FN == 1) ? 8 : (FM + FN <= 5) ? 4 : (FM + FN == 6 && FM == 4) ? 3 : 2>;

template <int ACT>
hipError_t run_stream(const I8Args& g, hipStream_t s) {
    stream_shape(g, ACT >= 0, [&](int fm, int fn, unsigned grid) {
        auto go = [&](auto kern) { hipLaunchKernelGGL(kern, dim3(grid), dim3(256), 0, s, g); };
        auto by_fm = [&](auto fnc) {
            constexpr int FN = decltype(fnc)::value;
            if (fm == 1) go(i8_stream_kernel<Stream<1, FN>, ACT>);
            else if (fm == 2) go(i8_stream_kernel<Stream<2, FN>, ACT>);
            else go(i8_stream_kernel<Stream<4, FN>, ACT>);
        };
        if (fn == 2) by_fm(std::integral_constant<int, 2>{});
        else if (fn >= 4) by_fm(std::integral_constant<int, 4>{});
        else if constexpr (ACT < 0) {
            if (fn == 1) by_fm(std::integral_constant<int, 1>{});
            else by_fm(std::integral_constant<int, 3>{});
        }
    });
    return hipGetLastError();
}

}  // namespace

hipError_t launch_gemm_i8(const I8Args& g, const LoraArgs* seg, bool* fused, hipStream_t s) {
    if (fused) *fused = false;
    if (!gemm_i8_ok(g.M, g.N, g.K)) return hipErrorInvalidValue;
    if (g.M <= 256) return run_stream<-1>(g, s);
    if (seg != nullptr && seg->n_segs > 0) {
        if (fused) *fused = true;
        return run_long<-1, true>(g, *seg, s);
    }
    return run_long<-1, false>(g, LoraArgs{}, s);
}

hipError_t launch_gemm_i8_gated(const I8Args& g, int act, hipStream_t s) {
    if (!gemm_i8_ok(g.M, g.N, g.K) || g.row_slot != nullptr) return hipErrorInvalidValue;
    auto go = [&](auto actc) {
        constexpr int ACT = decltype(actc)::value;
        return g.M <= 256 ? run_stream<ACT>(g, s) : run_long<ACT, false>(g, LoraArgs{}, s);
    };
    switch (act) {
        case kActSilu: return go(std::integral_constant<int, kActSilu>{});
        case kActGelu: return go(std::integral_constant<int, kActGelu>{});
        case kActGeluTanh: return go(std::integral_constant<int, kActGeluTanh>{});
        default: return hipErrorInvalidValue;
    }
}

bool gemm_i8_shrink_fits(int64_t M, int64_t N, int64_t K, int n_su) { return M <= 64 && n_su > 0 && gemm_i8_ok(M, N, K); }

hipError_t launch_gemm_i8_shrink(const I8Args& g0, uint64_t raw_mask, const LoraArgs& a, const void* cp_src, void* cp_dst,
                                 int64_t cp_n, hipStream_t s) {
    if (!gemm_i8_shrink_fits(g0.M, g0.N, g0.K, a.n_su) || cp_n < 0 || cp_n > INT32_MAX) return hipErrorInvalidValue;
    I8Args g = g0;
    if (raw_mask != 0) g.row_slot = nullptr;
    const int ncp = cp_n > 0 ? kCopyBlocks : 0;
    stream_shape(g, false, [&](int fm, int fn, unsigned tiles) {
        auto go = [&](auto kern) {
            hipLaunchKernelGGL(kern, dim3(tiles + a.n_su + ncp), dim3(256), 0, s, g, raw_mask, a, (int)tiles,
                               static_cast<const uint32_t*>(cp_src), static_cast<uint32_t*>(cp_dst), (int)cp_n);
        };
        auto by_fm = [&](auto fnc) {
            constexpr int FN = decltype(fnc)::value;
            if (fm == 1) go(i8_stream_shrink_kernel<Stream<1, FN>>);
            else if (fm == 2) go(i8_stream_shrink_kernel<Stream<2, FN>>);
            else go(i8_stream_shrink_kernel<Stream<4, FN>>);
        };
        if (fn == 1) by_fm(std::integral_constant<int, 1>{});
        else if (fn == 2) by_fm(std::integral_constant<int, 2>{});
        else if (fn == 3) by_fm(std::integral_constant<int, 3>{});
        else by_fm(std::integral_constant<int, 4>{});
    });
    return hipGetLastError();
}

}  // namespace hagemm
