// The shared base product with a 4-bit base weight: y[M][N] = sum_k x[m][k] *
// scale[n][k / group] * (code[n][k] - zero[n][k / group]), bf16 x, 4-bit codes
// [N][K / 2] (even k in the low half of its byte), fp16 scale and zero per
// group of 32, 64 or 128 consecutive k, fp32 accumulation.
//
// The matrix cores run bf16 on the codes themselves: a nibble put in the top
// four bits of bf16's mantissa stands for 16 + code exactly, so a code needs a
// shift and one and-or, and no rounding.  Per group, fp32: y += scale * (acc -
// (16 + zero) * sum(x)), the sum of x from one more matrix operation against
// ones.
#include "common.h"
#include "internal.h"

namespace hagemm {
namespace {

// (16 + nibble k, 16 + nibble k + 4) of w as two bf16
__device__ __forceinline__ uint32_t code_pair(uint32_t w, int k) {
    const uint32_t s = k == 0 ? w << 3 : k == 1 ? w >> 1 : k == 2 ? w >> 5 : w >> 9;
    return (s & 0x00780078u) | 0x41804180u;
}

// eight consecutive x in the order of code_pair's elements: 0, 4, 1, 5, 2, 6, 3, 7
__device__ __forceinline__ u32x4 code_order(const u32x4& v) {
    return u32x4{__builtin_amdgcn_perm(v[2], v[0], 0x05040100u), __builtin_amdgcn_perm(v[2], v[0], 0x07060302u),
                 __builtin_amdgcn_perm(v[3], v[1], 0x05040100u), __builtin_amdgcn_perm(v[3], v[1], 0x07060302u)};
}

__device__ __forceinline__ float half_lo(uint32_t w) { return (float)__builtin_bit_cast(_Float16, (uint16_t)w); }
__device__ __forceinline__ float half_hi(uint32_t w) { return (float)__builtin_bit_cast(_Float16, (uint16_t)(w >> 16)); }

constexpr int kW4Waves = 4;

// One workgroup per 16 columns of y and 16 MB rows: its waves take the 128-deep pieces of K in
// turn, and their sums meet in LDS in wave order.
template <int MB, int G>
__global__ __launch_bounds__(64 * kW4Waves) void gemm_w4_kernel(const bf16_t* __restrict__ x,
                                                                const uint8_t* __restrict__ q,
                                                                const uint32_t* __restrict__ sz, bf16_t* __restrict__ y,
                                                                int M, int N, int K, const int32_t* __restrict__ row_slot,
                                                                float* __restrict__ ybase) {
    __shared__ float part[kW4Waves][MB][4][64];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, li = lane & 15, lg = lane >> 4;
    const int n0 = blockIdx.x * 16, m0 = blockIdx.y * 16 * MB;
    const int n = min(n0 + li, N - 1);
    constexpr int NG = 128 / G;
    const uint8_t* qn = q + (int64_t)n * (K / 2);
    const uint32_t* sn = sz + (int64_t)n * (K / G);
    // k of this lane's eight codes of step s: one 16-byte load a lane where a group is 128 deep
    const int kl = G == 128 ? lg * 32 : lg * 8, ks = G == 128 ? 8 : 32;
    f32x4 acc[MB];
#pragma unroll
    for (int b = 0; b < MB; ++b) acc[b] = f32x4{0.f, 0.f, 0.f, 0.f};
    const u32x4 ones{0x3F803F80u, 0x3F803F80u, 0x3F803F80u, 0x3F803F80u};
    struct Piece {
        uint32_t c[4], s[NG];
    };
    auto load = [&](int kb, Piece& p) {
        if constexpr (G == 128) {
            const u32x4 v = ld16(qn + kb / 2 + lg * 16);
#pragma unroll
            for (int i = 0; i < 4; ++i) p.c[i] = v[i];
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) p.c[i] = *reinterpret_cast<const uint32_t*>(qn + kb / 2 + i * 16 + lg * 4);
        }
#pragma unroll
        for (int g = 0; g < NG; ++g) p.s[g] = sn[kb / G + g];
    };
    auto mul = [&](int kb, const Piece& p) {
#pragma unroll
        for (int g = 0; g < NG; ++g) {
            const float sc = half_lo(p.s[g]), zr = 16.f + half_hi(p.s[g]);
            f32x4 d[MB], xs[MB];
#pragma unroll
            for (int b = 0; b < MB; ++b) d[b] = xs[b] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int t = 0; t < G / 32; ++t) {
                const int s = g * (G / 32) + t;
                u32x4 cf;
#pragma unroll
                for (int i = 0; i < 4; ++i) cf[i] = code_pair(p.c[s], i);
#pragma unroll
                for (int b = 0; b < MB; ++b) {
                    const int m = m0 + 16 * b + li;
                    u32x4 xf{0, 0, 0, 0};
                    if (m < M) xf = code_order(ld16(x + (int64_t)m * K + kb + kl + s * ks));
                    d[b] = mma_step(xf, cf, d[b], bf16_t{});
                    xs[b] = mma_step(xf, ones, xs[b], bf16_t{});
                }
            }
#pragma unroll
            for (int b = 0; b < MB; ++b)
#pragma unroll
                for (int i = 0; i < 4; ++i) acc[b][i] += sc * (d[b][i] - zr * xs[b][i]);
        }
    };
    constexpr int PF = 4;
    Piece p[PF];
    const int step = 128 * kW4Waves;
#pragma unroll
    for (int i = 0; i < PF; ++i) load(min(wave * 128 + i * step, K - 128), p[i]);
    for (int k0 = wave * 128; k0 < K; k0 += PF * step) {
#pragma unroll
        for (int i = 0; i < PF; ++i) {
            const int kb = k0 + i * step;
            if (kb < K) {
                const Piece now = p[i];
                load(min(kb + PF * step, K - 128), p[i]);
                mul(kb, now);
            }
        }
    }
#pragma unroll
    for (int b = 0; b < MB; ++b)
#pragma unroll
        for (int i = 0; i < 4; ++i) part[wave][b][i][lane] = acc[b][i];
    __syncthreads();
    for (int b = wave; b < MB; b += kW4Waves) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float v = 0.f;
#pragma unroll
            for (int w = 0; w < kW4Waves; ++w) v += part[w][b][i][lane];
            const int m = m0 + 16 * b + 4 * lg + i;
            if (m >= M || n0 + li >= N) continue;
            const int64_t off = (int64_t)m * N + n0 + li;
            if (row_slot != nullptr && row_slot[m] >= 0)
                ybase[off] = v;
            else
                y[off].bits = (uint16_t)f32_to_bf16(v);
        }
    }
}

}  // namespace

bool gemm_w4_ok(int64_t M, int64_t N, int64_t K, int32_t group) {
    if (group != 32 && group != 64 && group != 128) return false;
    if (M < 1 || N < 1 || N % 4 || K < 128 || K % 128) return false;
    return M * K * 2 < INT32_MAX && N * K / 2 < INT32_MAX;
}

hipError_t launch_gemm_w4(const void* x, const void* q, const void* sz, int32_t group, void* y, int64_t M64, int64_t N64,
                          int64_t K64, const int32_t* row_slot, float* ybase, hipStream_t s) {
    if (!gemm_w4_ok(M64, N64, K64, group)) return hipErrorInvalidValue;
    const int M = (int)M64, N = (int)N64, K = (int)K64;
    auto go = [&](auto kern, int bm) {
        hipLaunchKernelGGL(kern, dim3((N + 15) / 16, (M + bm - 1) / bm), dim3(64 * kW4Waves), 0, s,
                           static_cast<const bf16_t*>(x), static_cast<const uint8_t*>(q),
                           static_cast<const uint32_t*>(sz), static_cast<bf16_t*>(y), M, N, K, row_slot, ybase);
    };
    auto by_rows = [&](auto k1, auto k2, auto k4) {
        if (M <= 16) go(k1, 16);
        else if (M <= 32) go(k2, 32);
        else go(k4, 64);
    };
    if (group == 128) by_rows(gemm_w4_kernel<1, 128>, gemm_w4_kernel<2, 128>, gemm_w4_kernel<4, 128>);
    else if (group == 64) by_rows(gemm_w4_kernel<1, 64>, gemm_w4_kernel<2, 64>, gemm_w4_kernel<4, 64>);
    else by_rows(gemm_w4_kernel<1, 32>, gemm_w4_kernel<2, 32>, gemm_w4_kernel<4, 32>);
    return hipGetLastError();
}

}  // namespace hagemm
