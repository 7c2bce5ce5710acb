// Arguments and launchers of the row kernels (rows_kernels.hip): the norm of rows and the (gated)
// rows of a projection, each with its 8-bit form.  Internal to the library.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace hagemm {

enum { kActNone = 0, kActSilu = 1, kActGelu = 2, kActGeluTanh = 3 };

// Rows of d values; strides in elements.  y, held, code and scale may be NULL (code and scale together).
struct RowsArgs {
    const void* x;
    const void* other;      // norm: the residual; act: the gate; or NULL
    const void* weight;     // norm only
    void* sum_out;          // norm with a residual: x + residual, or NULL
    void* y;
    void* held;
    int8_t* code;
    float* scale;
    int64_t x_stride, other_stride, sum_stride, y_stride, held_stride;
    int32_t n_rows, d;
    float eps;
};

constexpr int kMaxRowWidth = 65536;

hipError_t launch_rows_norm(const RowsArgs& a, hipStream_t s);
hipError_t launch_rows_act(const RowsArgs& a, int act, hipStream_t s);

}  // namespace hagemm
