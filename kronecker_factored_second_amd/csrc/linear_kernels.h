// Descriptors and launchers of the 8-bit linear-layer kernels (linear_kernels.hip).
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

namespace okls {

struct Blocked {          // okls_blocked on the device side; codes == nullptr: not wanted
  uint8_t* codes;
  uint8_t* scales;
  int64_t rows, cols, ld, ld_scale;
  int32_t format;         // okls_code
};

struct QuantArgs {
  const void* x;
  int64_t rows, cols, ldx;
  const float* row_factor;
  const void* col_factor;
  int32_t x_dtype, col_dtype;
  Blocked along_cols, along_rows;
};

struct MatmulArgs {
  Blocked a, b;
  void* c;
  int64_t ldc;
  float* ws;              // partial sums of a split summed axis
  int32_t c_dtype, accumulate;
};

struct NormArgs {
  const void* x;
  const void* residual;
  const void* weight;
  void* h;
  float* rstd;
  int64_t rows, cols, ldx, ldr, ldh;
  Blocked out;
  float eps;
  int32_t dtype, weight_dtype;
};

struct NormGradArgs {
  const void* dy;
  const void* h;
  const float* rstd;
  const void* weight;
  const void* dh;
  void* dx;
  void* dweight;
  float* ws;
  int64_t rows, cols, lddy, ldh, lddh, lddx;
  int32_t dtype, weight_dtype;
};

hipError_t launch_quantize(const QuantArgs& a, hipStream_t s);
hipError_t launch_rms_norm(const NormArgs& a, hipStream_t s);
size_t norm_grad_workspace(int64_t rows, int64_t cols);
hipError_t launch_rms_norm_backward(const NormGradArgs& a, hipStream_t s);
size_t matmul_workspace(int64_t m, int64_t n, int64_t k);
hipError_t launch_matmul(const MatmulArgs& a, hipStream_t s);

}  // namespace okls
