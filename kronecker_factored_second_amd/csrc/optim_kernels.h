// Descriptors and launchers of the many-tensor optimizer kernels (optim_kernels.hip).
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

namespace okls {

// A launch's tensors travel in its arguments (at most 4 KB): nothing to upload,
// and a captured launch carries its own.
struct AdamTensor {
  float* p;
  const void* g;
  void* m;
  void* v;
  uint8_t* scales;
  int64_t n;
  uint32_t first;    // workgroup
  uint32_t key;      // of the rounding thresholds
};
constexpr int kAdamTensors = 64;
constexpr int kAdamChunk = 2048;   // elements a workgroup

struct AdamArgs {
  AdamTensor tensor[kAdamTensors];
  uint8_t dtype[kAdamTensors];     // of the gradients
  const float* norm;
  double max_norm;
  float beta1, rest1, beta2, rest2, eps, decay, step, unbias2;
  int32_t count;
};

struct NormTensor {
  const void* g;
  int64_t n;
  uint32_t first;    // workgroup
  int32_t dtype;
};
constexpr int kNormTensors = 128;
constexpr int kNormChunk = 32768;  // elements a workgroup

struct GradNormArgs {
  NormTensor tensor[kNormTensors];
  double* part;
  int32_t count;
};

static_assert(sizeof(AdamArgs) <= 4096 && sizeof(GradNormArgs) <= 4096, "a launch's arguments");

hipError_t launch_adamw(const AdamArgs& a, unsigned blocks, bool eight, hipStream_t s);
hipError_t launch_grad_norm(const GradNormArgs& a, unsigned blocks, hipStream_t s);
hipError_t launch_join_norm(const double* part, int64_t n, float* norm, hipStream_t s);

}  // namespace okls
