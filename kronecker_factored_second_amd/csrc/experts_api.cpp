// Host side of the experts' operators: argument checks, then the launchers.
// Nothing here allocates or throws.
#include "../../include/okls_experts.h"

#include "experts_kernels.h"

namespace {

constexpr int64_t kMaxDim = int64_t(1) << 30;
constexpr int64_t kMaxPairs = int64_t(1) << 28;
constexpr int64_t kMaxStride = int64_t(1) << 40;   // elements; keeps every byte offset inside 64 bits with room
constexpr int64_t kMaxOut = int64_t(1) << 37;      // elements of a product: more than the card's memory holds
constexpr int64_t kMaxTiles = int64_t(1) << 23;     // of 128 x 128, a workgroup each: fewer than 2^32 threads
constexpr int64_t kMaxCode = int64_t(1) << 24;     // bytes between a product's code rows: a tile's side spans fewer than 2^32

bool dtype_ok(int32_t d) { return d == OKLS_F32 || d == OKLS_BF16 || d == OKLS_F16; }
bool aligned(const void* p, uintptr_t n) { return p != nullptr && (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
uintptr_t elem(int32_t dtype) { return dtype == OKLS_F32 ? 4 : 2; }
int64_t up(int64_t v, int64_t n) { return (v + n - 1) / n * n; }
bool tensor_ok(const void* p, int64_t ld, int32_t dtype, int64_t cols) { return aligned(p, elem(dtype)) && ld >= cols && ld <= kMaxStride; }
okls_status launched(hipError_t e) { return e == hipSuccess ? OKLS_OK : OKLS_ERR_HIP; }

okls_status check_plan(const okls_expert_plan* p) {
  if (p == nullptr) return OKLS_ERR_INVALID_ARG;
  const int64_t rows = okls_experts_capacity(p->tokens, p->each, p->n_experts, p->align);
  if (rows < 0 || p->capacity != rows) return OKLS_ERR_SHAPE;
  if (!aligned(p->offsets, 4) || !aligned(p->counts, 4)) return OKLS_ERR_INVALID_ARG;
  if (rows > 0 && (!aligned(p->rows, 4) || !aligned(p->pairs, 4))) return OKLS_ERR_INVALID_ARG;
  return OKLS_OK;
}

okls::ExpertPlan device_side(const okls_expert_plan& p) {
  return {p.rows, p.pairs, p.offsets, p.counts, p.tokens, static_cast<int32_t>(p.each), static_cast<int32_t>(p.tokens * p.each),
          static_cast<int32_t>(p.capacity), p.n_experts, p.align};
}

okls_status check_blocked(const okls_blocked& b, int64_t rows, int64_t cols, int64_t most_ld = kMaxStride) {
  if (b.format != OKLS_E4M3 && b.format != OKLS_E5M2) return OKLS_ERR_DTYPE;
  if (b.rows != rows || b.cols != cols || rows < 0 || rows > kMaxDim || cols < 0 || cols > kMaxDim) return OKLS_ERR_SHAPE;
  if (b.ld < up(cols, OKLS_BLOCK) || b.ld > most_ld || b.ld % 16) return OKLS_ERR_SHAPE;
  if (b.ld_scale < up(rows, 16) || b.ld_scale > kMaxStride || b.ld_scale % 16) return OKLS_ERR_SHAPE;
  if (rows == 0 || cols == 0) return OKLS_OK;
  if (!aligned(b.codes, 16) || !aligned(b.scales, 16)) return OKLS_ERR_INVALID_ARG;
  return OKLS_OK;
}

okls::Blocked device_side(const okls_blocked* b) {
  if (b == nullptr) return okls::Blocked{};
  return okls::Blocked{static_cast<uint8_t*>(b->codes), static_cast<uint8_t*>(b->scales), b->rows, b->cols, b->ld, b->ld_scale, b->format};
}

}  // namespace

extern "C" {

int64_t okls_experts_capacity(int64_t tokens, int64_t each, int32_t n_experts, int32_t align) {
  if (tokens < 0 || each < 1 || tokens > kMaxPairs || each > kMaxPairs || tokens * each > kMaxPairs) return -1;
  if (n_experts < 1 || n_experts > OKLS_MAX_EXPERTS) return -1;
  if (align != 16 && align != 32 && align != 64 && align != 128) return -1;
  const int64_t pairs = tokens * each, some = pairs < n_experts ? pairs : n_experts;
  return (pairs + some * (align - 1)) / align * align;
}

size_t okls_experts_plan_workspace_size(int64_t tokens, int64_t each, int32_t n_experts) {
  if (okls_experts_capacity(tokens, each, n_experts, 16) < 0) return 0;
  return okls::plan_workspace(tokens * each, n_experts);
}

okls_status okls_experts_plan(const void* choice, int32_t choice_bits, const okls_expert_plan* plan,
                              void* workspace, size_t ws_bytes, void* stream) {
  if (okls_status st = check_plan(plan)) return st;
  if (choice_bits != 32 && choice_bits != 64) return OKLS_ERR_DTYPE;
  if (plan->tokens > 0 && !aligned(choice, choice_bits / 8)) return OKLS_ERR_INVALID_ARG;
  const size_t need = okls_experts_plan_workspace_size(plan->tokens, plan->each, plan->n_experts);
  if (need != 0 && (!aligned(workspace, 16) || ws_bytes < need)) return OKLS_ERR_WORKSPACE;
  return launched(okls::launch_plan(choice, choice_bits == 64, device_side(*plan), static_cast<int32_t*>(workspace), static_cast<hipStream_t>(stream)));
}

okls_status okls_experts_gather(const okls_expert_plan* plan, const void* x, int64_t ldx, int32_t dtype,
                                int64_t cols, void* out, int64_t ldo, void* stream) {
  if (okls_status st = check_plan(plan)) return st;
  if (!dtype_ok(dtype)) return OKLS_ERR_DTYPE;
  if (cols < 0 || cols > kMaxDim) return OKLS_ERR_SHAPE;
  if (plan->capacity == 0 || cols == 0) return OKLS_OK;
  if (!tensor_ok(x, ldx, dtype, cols) || !tensor_ok(out, ldo, dtype, cols)) return OKLS_ERR_INVALID_ARG;
  okls::RowsArgs a{device_side(*plan), x, nullptr, nullptr, out, nullptr, cols, ldx, 0, ldo, dtype, 0};
  return launched(okls::launch_gather(a, static_cast<hipStream_t>(stream)));
}

okls_status okls_experts_combine(const okls_expert_plan* plan, const void* y, int64_t ldy, int32_t dtype, int64_t cols,
                                 const void* weights, int32_t weight_dtype, void* out, int64_t ldo, void* stream) {
  if (okls_status st = check_plan(plan)) return st;
  if (!dtype_ok(dtype) || (weights != nullptr && !dtype_ok(weight_dtype))) return OKLS_ERR_DTYPE;
  if (cols < 0 || cols > kMaxDim) return OKLS_ERR_SHAPE;
  if (plan->tokens == 0 || cols == 0) return OKLS_OK;
  if (!tensor_ok(y, ldy, dtype, cols) || !tensor_ok(out, ldo, dtype, cols)) return OKLS_ERR_INVALID_ARG;
  if (weights != nullptr && !aligned(weights, elem(weight_dtype))) return OKLS_ERR_INVALID_ARG;
  okls::RowsArgs a{device_side(*plan), nullptr, y, weights, out, nullptr, cols, 0, ldy, ldo, dtype, weight_dtype};
  return launched(okls::launch_combine(a, static_cast<hipStream_t>(stream)));
}

okls_status okls_experts_combine_backward(const okls_expert_plan* plan, const void* dout, int64_t lddout, const void* y,
                                          int64_t ldy, int32_t dtype, int64_t cols, const void* weights,
                                          int32_t weight_dtype, void* dy, int64_t lddy, void* dweights, void* stream) {
  if (okls_status st = check_plan(plan)) return st;
  if (!dtype_ok(dtype) || !dtype_ok(weight_dtype)) return OKLS_ERR_DTYPE;
  if (cols < 1 || cols > kMaxDim) return OKLS_ERR_SHAPE;
  if (plan->tokens == 0) return OKLS_OK;
  if (!tensor_ok(dout, lddout, dtype, cols) || !tensor_ok(y, ldy, dtype, cols) || !tensor_ok(dy, lddy, dtype, cols)) return OKLS_ERR_INVALID_ARG;
  if (!aligned(weights, elem(weight_dtype)) || !aligned(dweights, elem(weight_dtype))) return OKLS_ERR_INVALID_ARG;
  okls::RowsArgs a{device_side(*plan), dout, y, weights, dy, dweights, cols, lddout, ldy, lddy, dtype, weight_dtype};
  return launched(okls::launch_combine_backward(a, static_cast<hipStream_t>(stream)));
}

okls_status okls_experts_quantize_rows(const okls_expert_plan* plan, const void* x, int64_t ldx, int32_t dtype,
                                       int64_t cols, int32_t gathered, const okls_blocked* along_cols,
                                       const okls_blocked* along_rows, void* stream) {
  if (okls_status st = check_plan(plan)) return st;
  if (!dtype_ok(dtype)) return OKLS_ERR_DTYPE;
  if (cols < 0 || cols > kMaxDim) return OKLS_ERR_SHAPE;
  if ((along_cols == nullptr && along_rows == nullptr) || (gathered != 0 && gathered != 1)) return OKLS_ERR_INVALID_ARG;
  const int64_t rows = plan->capacity;
  if (along_cols != nullptr) if (okls_status st = check_blocked(*along_cols, rows, cols)) return st;
  if (along_rows != nullptr) if (okls_status st = check_blocked(*along_rows, cols, rows)) return st;
  if (rows == 0 || cols == 0) return OKLS_OK;
  if (!tensor_ok(x, ldx, dtype, cols)) return OKLS_ERR_INVALID_ARG;
  okls::QuantArgs a{x, rows, cols, ldx, nullptr, nullptr, dtype, 0, device_side(along_cols), device_side(along_rows), 1, 0,
                    plan->pairs, gathered ? static_cast<int32_t>(plan->each) : 0, static_cast<int32_t>(plan->tokens * plan->each)};
  return launched(okls::launch_quantize(a, static_cast<hipStream_t>(stream)));
}

okls_status okls_experts_quantize_stack(const void* x, int32_t dtype, int32_t n_experts, int64_t stride, int64_t rows,
                                        int64_t cols, int64_t ldx, const okls_blocked* along_cols,
                                        const okls_blocked* along_rows, void* stream) {
  if (!dtype_ok(dtype)) return OKLS_ERR_DTYPE;
  if (n_experts < 1 || n_experts > OKLS_MAX_EXPERTS || rows < 0 || rows > kMaxDim || cols < 0 || cols > kMaxDim) return OKLS_ERR_SHAPE;
  if (along_cols == nullptr && along_rows == nullptr) return OKLS_ERR_INVALID_ARG;
  if (along_cols != nullptr) if (okls_status st = check_blocked(*along_cols, n_experts * up(rows, 16), cols)) return st;
  if (along_rows != nullptr) if (okls_status st = check_blocked(*along_rows, n_experts * up(cols, 16), rows)) return st;
  if (rows == 0 || cols == 0) return OKLS_OK;
  if (!tensor_ok(x, ldx, dtype, cols) || (n_experts > 1 && (stride < 0 || stride > kMaxStride))) return OKLS_ERR_INVALID_ARG;
  okls::QuantArgs a{x, rows, cols, ldx, nullptr, nullptr, dtype, 0, device_side(along_cols), device_side(along_rows), n_experts, stride, nullptr, 0, 0};
  return launched(okls::launch_quantize(a, static_cast<hipStream_t>(stream)));
}

okls_status okls_experts_matmul(const okls_expert_plan* plan, const okls_blocked* a, const okls_blocked* b, int64_t n,
                                void* c, int32_t c_dtype, int64_t ldc, void* stream) {
  if (okls_status st = check_plan(plan)) return st;
  if (a == nullptr || b == nullptr) return OKLS_ERR_INVALID_ARG;
  if (!dtype_ok(c_dtype)) return OKLS_ERR_DTYPE;
  if (n < 0 || n > kMaxDim || a->cols != b->cols) return OKLS_ERR_SHAPE;
  if (okls_status st = check_blocked(*a, plan->capacity, a->cols, kMaxCode - 16)) return st;
  if (okls_status st = check_blocked(*b, plan->n_experts * up(n, 16), a->cols, kMaxCode - 16)) return st;
  if (plan->capacity == 0 || n == 0) return OKLS_OK;
  if (!tensor_ok(c, ldc, c_dtype, n)) return OKLS_ERR_INVALID_ARG;
  if (plan->capacity > kMaxOut / n || plan->capacity / 16 > kMaxTiles * 8 / (up(n, 128) / 128)) return OKLS_ERR_SHAPE;
  okls::ExpertMatmulArgs args{device_side(*plan), device_side(a), device_side(b), c, n, ldc, c_dtype};
  return launched(okls::launch_expert_matmul(args, static_cast<hipStream_t>(stream)));
}

okls_status okls_experts_weight_grad(const okls_expert_plan* plan, const okls_blocked* a, const okls_blocked* b,
                                     void* c, int32_t c_dtype, int64_t ldc, void* stream) {
  if (okls_status st = check_plan(plan)) return st;
  if (a == nullptr || b == nullptr) return OKLS_ERR_INVALID_ARG;
  if (!dtype_ok(c_dtype)) return OKLS_ERR_DTYPE;
  if (plan->align != OKLS_BLOCK) return OKLS_ERR_UNSUPPORTED;
  if (okls_status st = check_blocked(*a, a->rows, plan->capacity, kMaxCode - 16)) return st;
  if (okls_status st = check_blocked(*b, b->rows, plan->capacity, kMaxCode - 16)) return st;
  if (a->rows == 0 || b->rows == 0) return OKLS_OK;
  if (!tensor_ok(c, ldc, c_dtype, b->rows)) return OKLS_ERR_INVALID_ARG;
  if (a->rows * plan->n_experts > kMaxOut / ldc || up(a->rows, 128) / 128 * plan->n_experts > kMaxTiles / (up(b->rows, 128) / 128)) return OKLS_ERR_SHAPE;
  okls::ExpertMatmulArgs args{device_side(*plan), device_side(a), device_side(b), c, b->rows, ldc, c_dtype};
  return launched(okls::launch_expert_weight_grad(args, static_cast<hipStream_t>(stream)));
}

}  // extern "C"
