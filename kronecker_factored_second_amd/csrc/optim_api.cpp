// Host side of the many-tensor optimizer step: argument checks, then launches
// of as many tensors as a launch's arguments hold.  Nothing here allocates or throws.
#include "../../include/okls_optim.h"

#include <math.h>

#include "optim_kernels.h"

namespace {

constexpr int64_t kMaxElements = int64_t(1) << 34;
constexpr unsigned kMaxBlocks = 1u << 23;          // of a launch: fewer than 2^32 threads

bool dtype_ok(int32_t d) { return d == OKLS_F32 || d == OKLS_BF16 || d == OKLS_F16; }
bool aligned(const void* p, uintptr_t n) { return p != nullptr && (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
uintptr_t elem(int32_t dtype) { return dtype == OKLS_F32 ? 4 : 2; }
unsigned chunks(int64_t n, int64_t each) { return static_cast<unsigned>((n + each - 1) / each); }
okls_status launched(hipError_t e) { return e == hipSuccess ? OKLS_OK : OKLS_ERR_HIP; }

okls_status check_gradients(int32_t n_tensors, const okls_gradient* grads) {
  if (n_tensors < 0 || (n_tensors > 0 && grads == nullptr)) return OKLS_ERR_INVALID_ARG;
  for (int32_t i = 0; i < n_tensors; ++i) {
    if (!dtype_ok(grads[i].dtype)) return OKLS_ERR_DTYPE;
    if (grads[i].n < 0 || grads[i].n > kMaxElements) return OKLS_ERR_SHAPE;
    if (grads[i].n > 0 && !aligned(grads[i].data, elem(grads[i].dtype))) return OKLS_ERR_INVALID_ARG;
  }
  return OKLS_OK;
}

}  // namespace

extern "C" {

size_t okls_grad_norm_workspace_size(int32_t n_tensors, const okls_gradient* grads) {
  if (n_tensors < 0 || (n_tensors > 0 && grads == nullptr)) return 0;
  size_t parts = 0;
  for (int32_t i = 0; i < n_tensors; ++i)
    if (grads[i].n > 0 && grads[i].n <= kMaxElements) parts += chunks(grads[i].n, okls::kNormChunk);
  return parts * sizeof(double);
}

okls_status okls_grad_norm(int32_t n_tensors, const okls_gradient* grads, float* norm, void* workspace,
                           size_t ws_bytes, void* stream) {
  if (okls_status st = check_gradients(n_tensors, grads)) return st;
  if (!aligned(norm, 4)) return OKLS_ERR_INVALID_ARG;
  const size_t need = okls_grad_norm_workspace_size(n_tensors, grads);
  if (need != 0 && (!aligned(workspace, 8) || ws_bytes < need)) return OKLS_ERR_WORKSPACE;
  hipStream_t s = static_cast<hipStream_t>(stream);
  okls::GradNormArgs a;
  a.part = static_cast<double*>(workspace);
  a.count = 0;
  unsigned blocks = 0;
  auto flush = [&]() {
    if (a.count == 0) return OKLS_OK;
    const okls_status st = launched(okls::launch_grad_norm(a, blocks, s));
    a.part += blocks;
    a.count = 0;
    blocks = 0;
    return st;
  };
  for (int32_t i = 0; i < n_tensors; ++i) {
    if (grads[i].n == 0) continue;
    const unsigned own = chunks(grads[i].n, okls::kNormChunk);
    if (a.count == okls::kNormTensors || blocks + own > kMaxBlocks)
      if (okls_status st = flush()) return st;
    a.tensor[a.count++] = {grads[i].data, grads[i].n, blocks, grads[i].dtype};
    blocks += own;
  }
  if (okls_status st = flush()) return st;
  return launched(okls::launch_join_norm(static_cast<const double*>(workspace), static_cast<int64_t>(need / sizeof(double)), norm, s));
}

okls_status okls_adamw(const okls_adamw_config* config, int64_t t, int32_t n_tensors,
                       const okls_adamw_tensor* tensors, const float* norm, void* stream) {
  if (config == nullptr || n_tensors < 0 || (n_tensors > 0 && tensors == nullptr) || t < 1) return OKLS_ERR_INVALID_ARG;
  const okls_adamw_config& c = *config;
  if (c.moment_bits != 32 && c.moment_bits != 8) return OKLS_ERR_DTYPE;
  if (!(c.lr >= 0 && isfinite(c.lr)) || !(c.beta1 >= 0 && c.beta1 < 1) || !(c.beta2 >= 0 && c.beta2 < 1) ||
      !(c.eps >= 0 && isfinite(c.eps)) || !(c.weight_decay >= 0 && isfinite(c.weight_decay))) return OKLS_ERR_INVALID_ARG;
  if (norm != nullptr && (!aligned(norm, 4) || !(c.max_norm > 0 && isfinite(c.max_norm)))) return OKLS_ERR_INVALID_ARG;
  for (int32_t i = 0; i < n_tensors; ++i) {
    const okls_adamw_tensor& x = tensors[i];
    if (!dtype_ok(x.g_dtype)) return OKLS_ERR_DTYPE;
    if (x.n < 0 || x.n > kMaxElements) return OKLS_ERR_SHAPE;
    if ((c.moment_bits == 8) != (x.scales != nullptr) && x.n > 0) return OKLS_ERR_INVALID_ARG;
    if (x.n > 0 && (!aligned(x.p, 4) || !aligned(x.g, elem(x.g_dtype)) || !aligned(x.m, c.moment_bits / 8) ||
                    !aligned(x.v, c.moment_bits / 8))) return OKLS_ERR_INVALID_ARG;
  }
  okls::AdamArgs a;
  a.norm = norm;
  a.max_norm = c.max_norm;
  a.beta1 = static_cast<float>(c.beta1), a.rest1 = static_cast<float>(1 - c.beta1);
  a.beta2 = static_cast<float>(c.beta2), a.rest2 = static_cast<float>(1 - c.beta2);
  a.eps = static_cast<float>(c.eps);
  a.decay = static_cast<float>(1 - c.lr * c.weight_decay);
  a.step = static_cast<float>(c.lr / (1 - pow(c.beta1, static_cast<double>(t))));
  a.unbias2 = static_cast<float>(pow(1 - pow(c.beta2, static_cast<double>(t)), -0.5));
  a.count = 0;
  unsigned blocks = 0;
  auto flush = [&]() {
    if (a.count == 0) return OKLS_OK;
    const okls_status st = launched(okls::launch_adamw(a, blocks, c.moment_bits == 8, static_cast<hipStream_t>(stream)));
    a.count = 0;
    blocks = 0;
    return st;
  };
  for (int32_t i = 0; i < n_tensors; ++i) {
    const okls_adamw_tensor& x = tensors[i];
    if (x.n == 0) continue;
    const unsigned own = chunks(x.n, okls::kAdamChunk);
    if (a.count == okls::kAdamTensors || blocks + own > kMaxBlocks)
      if (okls_status st = flush()) return st;
    const uint32_t key = static_cast<uint32_t>(t) * 0x6A09E667u + static_cast<uint32_t>(i) * 0xBB67AE85u;
    a.dtype[a.count] = static_cast<uint8_t>(x.g_dtype);
    a.tensor[a.count++] = {x.p, x.g, x.m, x.v, x.scales, x.n, blocks, key};
    blocks += own;
  }
  return flush();
}

}  // extern "C"
