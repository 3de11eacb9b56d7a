/*
 * okls_experts.h - C ABI of the operators around a stack of experts' matrices:
 * tokens sorted by the experts that they chose and back, and the experts' 8-bit
 * products, whose weight gradients are the G of a batched group of okls.h.
 *
 * The sorted order (okls_expert_plan).  Each of `tokens` tokens makes `each`
 * choices; choice k of token t has the number i = t each + k.  A choice outside
 * 0..n_experts - 1 is none (a dropped token).  Expert e's rows begin at
 * offsets[e] and hold its counts[e] choices in the order of their numbers; then
 * come rows without a choice up to the next multiple of `align`, where expert
 * e + 1 begins.  align 16 is what a product reads, and few rows waste least of
 * it; the weights' gradient needs 128, the 8-bit form's block, so that no block
 * of rows holds two experts.  The sizes of all tensors follow from numbers that
 * the host knows: `capacity` rows are enough for any choices, and the host never
 * waits to learn them.  Rows without a choice, up to the capacity, are zeros in
 * everything written here, except that a product's come from its operand's, which are zeros
 * if okls_experts_quantize_rows made it, and that an expert's weights that are not
 * finite give NaN in its own.
 *
 * Conventions, as in okls_linear.h: device pointers on the current device,
 * row-major with a free row stride, the caller owns every tensor and the
 * workspaces; all work is ordered on the given stream and never synchronised;
 * nothing is allocated, no memset is recorded, argument errors are returned
 * before any launch, and no call keeps anything for the next.  Sums run in a
 * fixed order: equal inputs give equal bits.  What a plan's tensors hold is
 * checked where it is used: entries outside their range count as none.
 */
#ifndef OKLS_EXPERTS_H_
#define OKLS_EXPERTS_H_

#include "okls_linear.h"

#ifdef __cplusplus
extern "C" {
#endif

#define OKLS_MAX_EXPERTS 512

typedef struct {
    int32_t* rows;      /* (tokens, each): each choice's row, -1 for none */
    int32_t* pairs;     /* (capacity): each row's choice, -1 for none */
    int32_t* offsets;   /* (n_experts + 1) */
    int32_t* counts;    /* (n_experts) */
    int64_t tokens, each;               /* tokens each <= 2^28 */
    int64_t capacity;   /* okls_experts_capacity's */
    int32_t n_experts;  /* 1..OKLS_MAX_EXPERTS */
    int32_t align;      /* 16, 32, 64 or 128 */
} okls_expert_plan;

/* The rows that any choices of these sizes fit in; -1 for sizes that are refused. */
int64_t okls_experts_capacity(int64_t tokens, int64_t each, int32_t n_experts, int32_t align);

/* Writes a plan's four tensors from the choices: (tokens, each) contiguous
 * integers of choice_bits 32 or 64.  The workspace (16-byte aligned) holds counts. */
size_t okls_experts_plan_workspace_size(int64_t tokens, int64_t each, int32_t n_experts);
okls_status okls_experts_plan(const void* choice, int32_t choice_bits, const okls_expert_plan* plan,
                              void* workspace, size_t ws_bytes, void* stream);

/* out[r] = x[pairs[r] / each] for x (tokens, cols) and out (capacity, cols) of `dtype`. */
okls_status okls_experts_gather(const okls_expert_plan* plan, const void* x, int64_t ldx, int32_t dtype,
                                int64_t cols, void* out, int64_t ldo, void* stream);

/* out[t] = sum over k of weights[t][k] y[rows[t][k]], choices without a row left
 * out, for y (capacity, cols) and out (tokens, cols) of `dtype` and contiguous weights
 * (tokens, each) of weight_dtype, or NULL for ones: the gradient of okls_experts_gather.
 * Products and sums in fp32 in k's order, rounded once. */
okls_status okls_experts_combine(const okls_expert_plan* plan, const void* y, int64_t ldy, int32_t dtype, int64_t cols,
                                 const void* weights, int32_t weight_dtype, void* out, int64_t ldo, void* stream);

/* The gradients of okls_experts_combine, from dout (tokens, cols):
 *   dy[r] = weights[i] dout[i / each], i = pairs[r];   dweights[t][k] = sum over columns dout[t] y[rows[t][k]]
 * (0 without a row); dy (capacity, cols) of `dtype`, dweights of weight_dtype. */
okls_status okls_experts_combine_backward(const okls_expert_plan* plan, const void* dout, int64_t lddout, const void* y,
                                          int64_t ldy, int32_t dtype, int64_t cols, const void* weights,
                                          int32_t weight_dtype, void* dy, int64_t lddy, void* dweights, void* stream);

/* The 8-bit form of sorted rows (capacity x cols), of their transpose, or of
 * both, as okls_quantize: rows of x (capacity, cols) as they are with gathered = 0,
 * of x (tokens, cols) at pairs[r] / each with gathered = 1.  What x holds in rows without
 * a choice is not read. */
okls_status okls_experts_quantize_rows(const okls_expert_plan* plan, const void* x, int64_t ldx, int32_t dtype,
                                       int64_t cols, int32_t gathered, const okls_blocked* along_cols,
                                       const okls_blocked* along_rows, void* stream);

/* The 8-bit forms of a stack x (n_experts, rows, cols) of matrices, `stride`
 * elements apart: along_cols holds expert e's matrix from row e up(rows, 16)
 * on (n_experts up(rows, 16) x cols), along_rows its transpose from row
 * e up(cols, 16) on; either may be NULL, not both.  Rows between are not written. */
okls_status okls_experts_quantize_stack(const void* x, int32_t dtype, int32_t n_experts, int64_t stride, int64_t rows,
                                        int64_t cols, int64_t ldx, const okls_blocked* along_cols,
                                        const okls_blocked* along_rows, void* stream);

/* c[r] = a[r] b_e^T for the rows r of each expert e: a (capacity x k) and the stack b
 * (n_experts up(n, 16) x k) in 8 bits, c (capacity, n) of c_dtype; zeros behind the last
 * expert's rows.  An expert's rows without a choice are multiplied like its others
 * (okls_experts_quantize_rows makes them zeros).  Sums as in okls_scaled_matmul. */
okls_status okls_experts_matmul(const okls_expert_plan* plan, const okls_blocked* a, const okls_blocked* b, int64_t n,
                                void* c, int32_t c_dtype, int64_t ldc, void* stream);

/* c_e = sum over the rows r of expert e of a[:, r] b[:, r]^T, zeros for an
 * expert without rows; rows without a choice are summed too, as zeros from
 * okls_experts_quantize_rows.  a (n x capacity) and b (k x capacity) in 8 bits, c
 * (n_experts, n, k) of c_dtype with row stride ldc, matrices n ldc apart.  The
 * plan's align must be 128. */
okls_status okls_experts_weight_grad(const okls_expert_plan* plan, const okls_blocked* a, const okls_blocked* b,
                                     void* c, int32_t c_dtype, int64_t ldc, void* stream);

#ifdef __cplusplus
}
#endif
#endif /* OKLS_EXPERTS_H_ */
