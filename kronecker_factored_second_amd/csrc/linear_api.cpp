// Host side of the 8-bit linear-layer operators: argument checks, then one
// launcher call.  Nothing here allocates or throws.
#include "../../include/okls_linear.h"

#include <math.h>

#include "linear_kernels.h"

namespace {

constexpr int64_t kMaxDim = int64_t(1) << 30;
constexpr int64_t kMaxOut = int64_t(1) << 37;      // elements of a product: more than the card's memory holds
constexpr int64_t kMaxStride = int64_t(1) << 40;   // elements; keeps every byte offset inside 64 bits with room

bool dim_ok(int64_t v) { return v >= 0 && v <= kMaxDim; }
bool dtype_ok(int32_t d) { return d == OKLS_F32 || d == OKLS_BF16 || d == OKLS_F16; }
bool stride_ok(int64_t ld, int64_t cols) { return ld >= cols && ld <= kMaxStride; }
bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
uintptr_t elem(int32_t dtype) { return dtype == OKLS_F32 ? 4 : 2; }
int64_t up(int64_t v, int64_t n) { return (v + n - 1) / n * n; }

okls_status check_blocked(const okls_blocked& b, int64_t rows, int64_t cols) {
  if (b.format != OKLS_E4M3 && b.format != OKLS_E5M2) return OKLS_ERR_DTYPE;
  if (b.rows != rows || b.cols != cols) return OKLS_ERR_SHAPE;
  if (b.ld < up(cols, OKLS_BLOCK) || b.ld > kMaxStride || b.ld % 16) return OKLS_ERR_SHAPE;
  if (b.ld_scale < up(rows, 16) || b.ld_scale > kMaxStride || b.ld_scale % 16) return OKLS_ERR_SHAPE;
  if (rows == 0 || cols == 0) return OKLS_OK;
  if (b.codes == nullptr || b.scales == nullptr || !aligned(b.codes, 16) || !aligned(b.scales, 16)) return OKLS_ERR_INVALID_ARG;
  return OKLS_OK;
}

okls::Blocked device_side(const okls_blocked* b) {
  if (b == nullptr) return okls::Blocked{};
  return okls::Blocked{static_cast<uint8_t*>(b->codes), static_cast<uint8_t*>(b->scales), b->rows, b->cols, b->ld, b->ld_scale, b->format};
}

// a tensor of rows x cols elements that is read or written
bool tensor_ok(const void* p, int64_t ld, int32_t dtype, int64_t cols) {
  return p != nullptr && aligned(p, elem(dtype)) && stride_ok(ld, cols);
}

okls_status launched(hipError_t e) { return e == hipSuccess ? OKLS_OK : OKLS_ERR_HIP; }

}  // namespace

extern "C" {

okls_status okls_quantize(const void* x, int32_t x_dtype, int64_t rows, int64_t cols, int64_t ldx,
                          const float* row_factor, const void* col_factor, int32_t col_factor_dtype,
                          const okls_blocked* along_cols, const okls_blocked* along_rows, void* stream) {
  if (!dim_ok(rows) || !dim_ok(cols)) return OKLS_ERR_SHAPE;
  if (!dtype_ok(x_dtype)) return OKLS_ERR_DTYPE;
  if (along_cols == nullptr && along_rows == nullptr) return OKLS_ERR_INVALID_ARG;
  if ((row_factor == nullptr) != (col_factor == nullptr)) return OKLS_ERR_INVALID_ARG;
  if (col_factor != nullptr && !dtype_ok(col_factor_dtype)) return OKLS_ERR_DTYPE;
  if (along_cols != nullptr) if (okls_status st = check_blocked(*along_cols, rows, cols)) return st;
  if (along_rows != nullptr) if (okls_status st = check_blocked(*along_rows, cols, rows)) return st;
  if (rows == 0 || cols == 0) return OKLS_OK;
  if (!tensor_ok(x, ldx, x_dtype, cols)) return OKLS_ERR_INVALID_ARG;
  if (row_factor != nullptr && (!aligned(row_factor, 4) || !aligned(col_factor, elem(col_factor_dtype)))) return OKLS_ERR_INVALID_ARG;
  okls::QuantArgs a{x, rows, cols, ldx, row_factor, col_factor, x_dtype, col_factor_dtype, device_side(along_cols), device_side(along_rows)};
  return launched(okls::launch_quantize(a, static_cast<hipStream_t>(stream)));
}

size_t okls_scaled_matmul_workspace_size(int64_t m, int64_t n, int64_t k) {
  if (!dim_ok(m) || !dim_ok(n) || !dim_ok(k)) return 0;
  return okls::matmul_workspace(m, n, k);
}

okls_status okls_scaled_matmul(const okls_blocked* a, const okls_blocked* b, void* c, int32_t c_dtype,
                               int64_t ldc, int32_t accumulate, void* workspace, size_t ws_bytes, void* stream) {
  if (a == nullptr || b == nullptr || (accumulate != 0 && accumulate != 1)) return OKLS_ERR_INVALID_ARG;
  if (!dim_ok(a->rows) || !dim_ok(b->rows) || !dim_ok(a->cols) || a->cols != b->cols) return OKLS_ERR_SHAPE;
  if (!dtype_ok(c_dtype)) return OKLS_ERR_DTYPE;
  if (okls_status st = check_blocked(*a, a->rows, a->cols)) return st;
  if (okls_status st = check_blocked(*b, b->rows, b->cols)) return st;
  if (a->rows == 0 || b->rows == 0) return OKLS_OK;
  if (a->rows > kMaxOut / b->rows) return OKLS_ERR_SHAPE;
  if (!tensor_ok(c, ldc, c_dtype, b->rows)) return OKLS_ERR_INVALID_ARG;
  const size_t need = okls::matmul_workspace(a->rows, b->rows, a->cols);
  if (need != 0 && (workspace == nullptr || !aligned(workspace, 16) || ws_bytes < need)) return OKLS_ERR_WORKSPACE;
  okls::MatmulArgs args{device_side(a), device_side(b), c, ldc, static_cast<float*>(workspace), c_dtype, accumulate};
  return launched(okls::launch_matmul(args, static_cast<hipStream_t>(stream)));
}

okls_status okls_rms_norm(const void* x, int64_t ldx, const void* residual, int64_t ldr, int32_t dtype,
                          int64_t rows, int64_t cols, const void* weight, int32_t weight_dtype, float eps,
                          void* h, int64_t ldh, float* rstd, const okls_blocked* out, void* stream) {
  if (out == nullptr || (residual == nullptr && h != nullptr)) return OKLS_ERR_INVALID_ARG;
  if (!dim_ok(rows) || cols < 1 || cols > kMaxDim) return OKLS_ERR_SHAPE;
  if (!dtype_ok(dtype) || !dtype_ok(weight_dtype)) return OKLS_ERR_DTYPE;
  if (!(eps >= 0.0f) || isinf(eps)) return OKLS_ERR_INVALID_ARG;
  if (okls_status st = check_blocked(*out, rows, cols)) return st;
  if (rows == 0) return OKLS_OK;
  if (!tensor_ok(x, ldx, dtype, cols) || weight == nullptr || !aligned(weight, elem(weight_dtype)) ||
      rstd == nullptr || !aligned(rstd, 4)) return OKLS_ERR_INVALID_ARG;
  if (residual != nullptr && (!tensor_ok(residual, ldr, dtype, cols) || !tensor_ok(h, ldh, dtype, cols))) return OKLS_ERR_INVALID_ARG;
  okls::NormArgs a{x, residual, weight, h, rstd, rows, cols, ldx, ldr, ldh, device_side(out), eps, dtype, weight_dtype};
  return launched(okls::launch_rms_norm(a, static_cast<hipStream_t>(stream)));
}

size_t okls_rms_norm_backward_workspace_size(int64_t rows, int64_t cols) {
  if (!dim_ok(rows) || !dim_ok(cols)) return 0;
  return okls::norm_grad_workspace(rows, cols);
}

okls_status okls_rms_norm_backward(const void* dy, int64_t lddy, const void* h, int64_t ldh, const float* rstd,
                                   const void* weight, int32_t weight_dtype, const void* dh, int64_t lddh,
                                   int32_t dtype, int64_t rows, int64_t cols, void* dx, int64_t lddx,
                                   void* dweight, void* workspace, size_t ws_bytes, void* stream) {
  if (!dim_ok(rows) || cols < 1 || cols > kMaxDim) return OKLS_ERR_SHAPE;
  if (!dtype_ok(dtype) || !dtype_ok(weight_dtype)) return OKLS_ERR_DTYPE;
  if (weight == nullptr || !aligned(weight, elem(weight_dtype)) || dweight == nullptr || !aligned(dweight, elem(weight_dtype)))
    return OKLS_ERR_INVALID_ARG;
  if (rows != 0) {
    if (!tensor_ok(dy, lddy, dtype, cols) || !tensor_ok(h, ldh, dtype, cols) || !tensor_ok(dx, lddx, dtype, cols) ||
        rstd == nullptr || !aligned(rstd, 4)) return OKLS_ERR_INVALID_ARG;
    if (dh != nullptr && !tensor_ok(dh, lddh, dtype, cols)) return OKLS_ERR_INVALID_ARG;
    const size_t need = okls::norm_grad_workspace(rows, cols);
    if (need != 0 && (workspace == nullptr || !aligned(workspace, 16) || ws_bytes < need)) return OKLS_ERR_WORKSPACE;
  }
  okls::NormGradArgs a{dy, h, rstd, weight, dh, dx, dweight, static_cast<float*>(workspace), rows, cols, lddy, ldh, lddh, lddx, dtype, weight_dtype};
  return launched(okls::launch_rms_norm_backward(a, static_cast<hipStream_t>(stream)));
}

}  // extern "C"
