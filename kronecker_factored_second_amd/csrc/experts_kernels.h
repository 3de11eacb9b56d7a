// Descriptors and launchers of the experts' kernels (experts_kernels.hip).
#pragma once
#include "linear_kernels.h"

namespace okls {

struct ExpertPlan {       // okls_expert_plan on the device side
  int32_t *rows, *pairs, *offsets, *counts;
  int64_t tokens;
  int32_t each, n_pairs, capacity, n_experts, align;
};

struct RowsArgs {
  ExpertPlan plan;
  const void* x;          // rows read: tokens' or sorted ones
  const void* y;          // sorted rows (combine's gradient)
  const void* weights;
  void* out;
  void* dweights;
  int64_t cols, ldx, ldy, ldo;
  int32_t dtype, weight_dtype;
};

struct ExpertMatmulArgs {
  ExpertPlan plan;
  Blocked a, b;
  void* c;
  int64_t n, ldc;
  int32_t c_dtype;
};

size_t plan_workspace(int64_t pairs, int32_t n_experts);
hipError_t launch_plan(const void* choice, bool wide, const ExpertPlan& p, int32_t* ws, hipStream_t s);
hipError_t launch_gather(const RowsArgs& a, hipStream_t s);
hipError_t launch_combine(const RowsArgs& a, hipStream_t s);
hipError_t launch_combine_backward(const RowsArgs& a, hipStream_t s);
hipError_t launch_expert_matmul(const ExpertMatmulArgs& a, hipStream_t s);
hipError_t launch_expert_weight_grad(const ExpertMatmulArgs& a, hipStream_t s);

}  // namespace okls
