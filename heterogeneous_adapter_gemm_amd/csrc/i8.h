// The 8-bit integer base: kernel arguments and launchers (i8_kernels.hip).  Internal to the library.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "internal.h"

namespace hagemm {

constexpr int64_t kI8MaxK = 131056;          // the most multiples of 16 whose sums of (-128)^2 fit int32
constexpr int64_t kI8MaxRows = 1 << 22;      // of x and of the weight: tile numbers stay inside 32 bits

// y[M][N] = xs[m] ws[n] sum_k x[m][k] w[n][k] (gated: act of it, times the same with w2, ws2).  Rows m with
// row_slot[m] >= 0 go unrounded to ybase [M][N] instead of y, for the delta kernels.
struct I8Args {
    const void* x;             // int8 codes [M][K]
    const float* xs;           // [M]
    const void *w, *w2;        // int8 codes [N][K]
    const float *ws, *ws2;     // [N]
    void* y;
    const int32_t* row_slot;
    float* ybase;
    int32_t M, N, K;
};

// N % 4 == 0, K % 16 == 0, and the sizes above
bool gemm_i8_ok(int64_t M, int64_t N, int64_t K);
// With seg (segments with adapters) the product adds their LoRA expand before rounding and sets *fused.
hipError_t launch_gemm_i8(const I8Args& g, const LoraArgs* seg, bool* fused, hipStream_t s);
hipError_t launch_gemm_i8_gated(const I8Args& g, int act, hipStream_t s);
// Decode batches (a.n_su > 0): as launch_gemm_shrink; with more than 64 rows raw_mask is 0 and row_slot names the adapter rows.
bool gemm_i8_shrink_fits(int64_t M, int64_t N, int64_t K, int n_su);
hipError_t launch_gemm_i8_shrink(const I8Args& g, uint64_t raw_mask, const LoraArgs& a, const void* cp_src, void* cp_dst,
                                 int64_t cp_n, hipStream_t s);

}  // namespace hagemm
