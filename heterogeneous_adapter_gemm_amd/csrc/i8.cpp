// Host side of the 8-bit integer entry points that need no pool (rows_*_i8, base_*_i8): argument checks and
// launches.  See include/lora_gemm.h for the contract of every entry point.
#include "i8.h"

#include <cmath>

#include "internal.h"
#include "lora_gemm.h"
#include "rows.h"

using namespace hagemm;

namespace {

int check_row_sizes(int64_t n_rows, int32_t d) {
    if (n_rows < 0 || n_rows > INT32_MAX) return set_error(LORA_EINVAL, "%lld rows", (long long)n_rows);
    if (d < 8 || d % 8 || d > kMaxRowWidth) return set_error(LORA_EINVAL, "rows of %d values: a multiple of 8, at most %d", d, kMaxRowWidth);
    return LORA_OK;
}

// bf16 rows: 16-byte aligned, a stride that keeps them so and apart (one row's says nothing)
int check_rows(const char* name, const void* p, int64_t n, int64_t stride, int32_t d) {
    if (n == 1) stride = d;
    if ((uintptr_t)p % 16 || stride % 8) return set_error(LORA_EINVAL, "%s: 16-byte aligned rows (stride a multiple of 8)", name);
    if (stride < d || stride > (int64_t(1) << 32)) return set_error(LORA_EINVAL, "%s: row stride %lld of rows of %d", name, (long long)stride, d);
    return LORA_OK;
}

int check_form(const void* y, const void* held, const int8_t* code, const float* scale) {
    if (!y && !held && !code) return set_error(LORA_EINVAL, "no output: y, held or code is needed");
    if ((code == nullptr) != (scale == nullptr)) return set_error(LORA_EINVAL, "code and scale are given together");
    if ((uintptr_t)code % 16 || (uintptr_t)scale % 4) return set_error(LORA_EINVAL, "code must be 16-byte, scale 4-byte aligned");
    return LORA_OK;
}

#define CHECK(call)          \
    do {                     \
        const int rc_ = call; \
        if (rc_) return rc_; \
    } while (0)

int launched(hipError_t e, const char* name) {
    return e == hipSuccess ? LORA_OK : set_error(LORA_EHIP, "%s: %s", name, hipGetErrorString(e));
}

int check_product(int64_t M, int64_t N, int64_t K) {
    if (M < 0 || N < 1 || K < 1) return set_error(LORA_EINVAL, "bad sizes");
    if (N % 4 || K % 16) return set_error(LORA_EINVAL, "N must be a multiple of 4 and K of 16");
    if (M > kI8MaxRows || N > kI8MaxRows || K > kI8MaxK)
        return set_error(LORA_EINVAL, "M and N are at most %lld, K %lld", (long long)kI8MaxRows, (long long)kI8MaxK);
    return LORA_OK;
}

int check_aligned(const void* const* p, int n) {
    for (int i = 0; i < n; ++i) {
        if (!p[i]) return set_error(LORA_EINVAL, "NULL pointer");
        if ((uintptr_t)p[i] % 16) return set_error(LORA_EINVAL, "pointers must be 16-byte aligned");
    }
    return LORA_OK;
}

}  // namespace

extern "C" {

int rows_norm_i8(const lora_norm_rows* r, void* stream) {
    if (!r) return set_error(LORA_EINVAL, "rows is NULL");
    CHECK(check_row_sizes(r->n_rows, r->d));
    if (!(r->eps > 0.f) || !std::isfinite(r->eps)) return set_error(LORA_EINVAL, "eps must be positive and finite");
    if (r->n_rows == 0) return LORA_OK;
    if (!r->x || !r->weight) return set_error(LORA_EINVAL, "x or weight is NULL");
    if ((uintptr_t)r->weight % 16) return set_error(LORA_EINVAL, "weight must be 16-byte aligned");
    if (r->sum_out && !r->residual) return set_error(LORA_EINVAL, "sum_out without a residual");
    CHECK(check_rows("x", r->x, r->n_rows, r->x_stride, r->d));
    if (r->residual) CHECK(check_rows("residual", r->residual, r->n_rows, r->residual_stride, r->d));
    if (r->sum_out) CHECK(check_rows("sum_out", r->sum_out, r->n_rows, r->sum_stride, r->d));
    if (r->y) CHECK(check_rows("y", r->y, r->n_rows, r->y_stride, r->d));
    if (r->held) CHECK(check_rows("held", r->held, r->n_rows, r->held_stride, r->d));
    CHECK(check_form(r->y, r->held, r->code, r->scale));
    RowsArgs a{};
    a.x = r->x;
    a.other = r->residual;
    a.weight = r->weight;
    a.sum_out = r->sum_out;
    a.y = r->y;
    a.held = r->held;
    a.code = r->code;
    a.scale = r->scale;
    a.x_stride = r->x_stride;
    a.other_stride = r->residual_stride;
    a.sum_stride = r->sum_stride;
    a.y_stride = r->y_stride;
    a.held_stride = r->held_stride;
    a.n_rows = (int32_t)r->n_rows;
    a.d = r->d;
    a.eps = r->eps;
    return launched(launch_rows_norm(a, static_cast<hipStream_t>(stream)), "rows_norm_i8");
}

int rows_act_i8(const lora_act_rows* r, void* stream) {
    if (!r) return set_error(LORA_EINVAL, "rows is NULL");
    CHECK(check_row_sizes(r->n_rows, r->d));
    if (r->act < LORA_ACT_NONE || r->act > LORA_ACT_GELU_TANH) return set_error(LORA_EINVAL, "act %d", r->act);
    if ((r->act == LORA_ACT_NONE) != (r->gate == nullptr) && r->n_rows > 0)
        return set_error(LORA_EINVAL, "a gate goes with an activation, and none without");
    if (r->n_rows == 0) return LORA_OK;
    if (!r->x) return set_error(LORA_EINVAL, "x is NULL");
    CHECK(check_rows("x", r->x, r->n_rows, r->x_stride, r->d));
    if (r->gate) CHECK(check_rows("gate", r->gate, r->n_rows, r->gate_stride, r->d));
    if (r->y) CHECK(check_rows("y", r->y, r->n_rows, r->y_stride, r->d));
    if (r->held) CHECK(check_rows("held", r->held, r->n_rows, r->held_stride, r->d));
    CHECK(check_form(r->y, r->held, r->code, r->scale));
    RowsArgs a{};
    a.x = r->x;
    a.other = r->gate;
    a.y = r->y;
    a.held = r->held;
    a.code = r->code;
    a.scale = r->scale;
    a.x_stride = r->x_stride;
    a.other_stride = r->gate_stride;
    a.y_stride = r->y_stride;
    a.held_stride = r->held_stride;
    a.n_rows = (int32_t)r->n_rows;
    a.d = r->d;
    return launched(launch_rows_act(a, r->act, static_cast<hipStream_t>(stream)), "rows_act_i8");
}

int base_gemm_i8(const int8_t* x_code, const float* x_scale, const int8_t* w0_code, const float* w0_scale, void* y, int64_t M,
                 int64_t N, int64_t K, void* stream) {
    CHECK(check_product(M, N, K));
    if (M == 0) return LORA_OK;
    const void* p[] = {x_code, x_scale, w0_code, w0_scale, y};
    CHECK(check_aligned(p, 5));
    I8Args g{};
    g.x = x_code;
    g.xs = x_scale;
    g.w = w0_code;
    g.ws = w0_scale;
    g.y = y;
    g.M = (int32_t)M;
    g.N = (int32_t)N;
    g.K = (int32_t)K;
    return launched(launch_gemm_i8(g, nullptr, nullptr, static_cast<hipStream_t>(stream)), "base_gemm_i8");
}

int base_gated_i8(const int8_t* x_code, const float* x_scale, const int8_t* wg_code, const float* wg_scale, const int8_t* wu_code,
                  const float* wu_scale, int32_t act, void* y, int64_t M, int64_t N, int64_t K, void* stream) {
    CHECK(check_product(M, N, K));
    if (act < LORA_ACT_SILU || act > LORA_ACT_GELU_TANH) return set_error(LORA_EINVAL, "act %d", act);
    if (M == 0) return LORA_OK;
    const void* p[] = {x_code, x_scale, wg_code, wg_scale, wu_code, wu_scale, y};
    CHECK(check_aligned(p, 7));
    I8Args g{};
    g.x = x_code;
    g.xs = x_scale;
    g.w = wg_code;
    g.ws = wg_scale;
    g.w2 = wu_code;
    g.ws2 = wu_scale;
    g.y = y;
    g.M = (int32_t)M;
    g.N = (int32_t)N;
    g.K = (int32_t)K;
    return launched(launch_gemm_i8_gated(g, act, static_cast<hipStream_t>(stream)), "base_gated_i8");
}

}  // extern "C"
