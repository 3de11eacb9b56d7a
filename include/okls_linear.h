/*
 * okls_linear.h - C ABI of the 8-bit linear-layer operators around the
 * preconditioner step of okls.h: what turns activations and master weights
 * into a layer's output, and the output's gradient into the gradient G that
 * okls_step reads.
 *
 * The 8-bit form of a matrix (okls_blocked).  Along its columns, the axis a
 * product sums over, every block of 128 values v of a row shares one scale
 * 2^e and holds v 2^-e rounded to nearest even in e4m3 or e5m2.  e is the
 * smallest integer >= -127 with max|v| <= F 2^e over the block's finite values
 * (F = 448 for e4m3, 57344 for e5m2), and 0 for a block with none but zeros
 * and non-finite values.  So nothing overflows, and the power of two makes
 * v 2^-e exact: each value is rounded once.  NaN stays NaN; an infinity
 * becomes NaN in e4m3, which has none, and stays in e5m2.
 *   codes:  (rows, ld) bytes, ld >= 128 ceil(cols / 128) and a multiple of 16;
 *           the columns from cols to the end of the last block are zeros.
 *   scales: (ceil(cols / 128), ld_scale) bytes, entry [b][r] = e + 127 of block
 *           b of row r; ld_scale >= rows rounded up to 16, a multiple of 16.
 * Block-major scales put the rows of one block next to each other, which is
 * how a product's tile reads them.
 *
 * Conventions, as in okls.h: device pointers on the current device, row-major,
 * the last axis contiguous and the row stride (ld*, in elements) free; the
 * caller owns every tensor and the workspaces; all work is ordered on the given
 * stream and never synchronised; nothing is allocated and no memset is
 * recorded, so every call can be captured into a HIP graph; argument errors are
 * returned before any launch.  Codes and scales must be 16-byte aligned; other
 * tensors need their element's alignment only.  No call keeps anything for the
 * next.  Sums run in a fixed order: equal inputs give equal bits.
 */
#ifndef OKLS_LINEAR_H_
#define OKLS_LINEAR_H_

#include "okls.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef enum { OKLS_E4M3 = 0, OKLS_E5M2 = 1 } okls_code;

#define OKLS_BLOCK 128

typedef struct {
    void* codes;        /* (rows, ld) bytes */
    void* scales;       /* (ceil(cols / 128), ld_scale) bytes */
    int64_t rows, cols; /* the matrix, 0..2^30 each */
    int64_t ld, ld_scale;
    int32_t format;     /* okls_code */
} okls_blocked;

/* The 8-bit form of x (rows x cols, okls_dtype x_dtype), of its transpose, or
 * of both from one read of x: `along_cols` (rows x cols, blocks along a row)
 * and `along_rows` (cols x rows, blocks along a column of x); either may be
 * NULL, not both.  With row_factor (rows, fp32) and col_factor (cols, okls_dtype
 * col_factor_dtype), both or neither, the values are
 * fl32(fl32(x row_factor) col_factor): the output of okls_rms_norm formed again
 * from h, 1/rms and the weight. */
okls_status okls_quantize(const void* x, int32_t x_dtype, int64_t rows, int64_t cols, int64_t ldx,
                          const float* row_factor, const void* col_factor, int32_t col_factor_dtype,
                          const okls_blocked* along_cols, const okls_blocked* along_rows, void* stream);

/* c = a b^T, or c += a b^T with accumulate = 1: a is m x k, b is n x k, both in
 * 8 bits and of equal cols; c is (m, n) of okls_dtype c_dtype with row stride
 * ldc.  Sums are held in fp32 and rounded once to c's type.  16-bit results take
 * the 8-bit matrix instructions, which drop what lies below 2^-13 of the largest
 * of each eight products: about 1.6e-5 of a result in norm, a hundredth of bf16's
 * own rounding, but up to 2^-10 of the sum of the products' sizes in an element
 * whose large products cancel.  fp32 results take products of the exact values,
 * whose sums round as fp32's; a value below 2^-126 may count as zero there, and
 * one of 2^128, to which the 8-bit form rounds inputs next to fp32's largest, is
 * an infinity.  A caller to whom 16-bit results drop too much takes fp32 ones and
 * casts.  k = 0 gives zeros.  The workspace (16-byte aligned) holds
 * partial sums where the summed axis is split over workgroups; it may be NULL
 * where the size is 0. */
size_t okls_scaled_matmul_workspace_size(int64_t m, int64_t n, int64_t k);
okls_status okls_scaled_matmul(const okls_blocked* a, const okls_blocked* b, void* c, int32_t c_dtype,
                               int64_t ldc, int32_t accumulate, void* workspace, size_t ws_bytes,
                               void* stream);

/* Root-mean-square norm with the residual's addition and an 8-bit output:
 *   h    = x + residual, rounded to their type (h = x where residual is NULL;
 *          then h must be NULL and nothing is written for it),
 *   rstd = (mean(h^2) + eps)^-1/2, summed in fp64 and rounded once to fp32,
 *   out  = the 8-bit form of fl32(fl32(h rstd) weight).
 * The statistics in fp64 keep the codes independent of the order of summation.
 * x, residual and h are of `dtype`; weight (cols) of weight_dtype; rstd (rows).
 * h may be x or residual (same pointer and stride): the addition in place, at
 * every width.  Nothing else that is written may overlap anything. */
okls_status okls_rms_norm(const void* x, int64_t ldx, const void* residual, int64_t ldr, int32_t dtype,
                          int64_t rows, int64_t cols, const void* weight, int32_t weight_dtype, float eps,
                          void* h, int64_t ldh, float* rstd, const okls_blocked* out, void* stream);

/* The gradient of y = h rstd weight (y's rounding to 8 bits passed straight
 * through), with g = dy weight and hat = h rstd:
 *   dx      = rstd (g - hat mean(g hat)) + dh,  the gradient of x and of the
 *             residual alike; dh, the gradient that reaches h itself, may be NULL,
 *   dweight = sum over rows of dy hat, in weight_dtype.
 * dy, h, dh and dx are of `dtype`.  dx may be dh or dy (same pointer and
 * stride), nothing else may overlap.  The workspace (16-byte aligned) holds
 * dweight's partial sums. */
size_t okls_rms_norm_backward_workspace_size(int64_t rows, int64_t cols);
okls_status okls_rms_norm_backward(const void* dy, int64_t lddy, const void* h, int64_t ldh, const float* rstd,
                                   const void* weight, int32_t weight_dtype, const void* dh, int64_t lddh,
                                   int32_t dtype, int64_t rows, int64_t cols, void* dx, int64_t lddx,
                                   void* dweight, void* workspace, size_t ws_bytes, void* stream);

#ifdef __cplusplus
}
#endif
#endif /* OKLS_LINEAR_H_ */
