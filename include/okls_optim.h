/*
 * okls_optim.h - C ABI of the optimizer step for parameters that the
 * preconditioner step of okls.h does not take (embeddings, norm weights,
 * biases, routers): AdamW over many tensors at once, with moments in 32 or in
 * 8 bits, and the norm of all gradients together that it clips them by.
 *
 * Conventions, as in okls.h: device pointers on the current device, tensors
 * contiguous, their element's alignment enough; the caller owns every tensor and
 * the workspace; the descriptors are host memory, read before the call returns.
 * All work is ordered on the given stream and never synchronised; nothing is
 * allocated and no memset is recorded, so every call can be captured into a HIP
 * graph (a replay reuses the captured t and lr); argument errors are returned
 * before any launch.  No call keeps anything for the next.  Sums run in a fixed
 * order: equal inputs give equal bits.
 */
#ifndef OKLS_OPTIM_H_
#define OKLS_OPTIM_H_

#include "okls_linear.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef struct {
    const void* data;
    int64_t n;          /* elements, 0..2^34 */
    int32_t dtype;      /* okls_dtype */
} okls_gradient;

/* norm = (sum over all tensors and elements of g^2)^1/2, squared and summed in
 * fp64 and rounded once to fp32.  0 tensors give 0.  The workspace (8-byte
 * aligned) holds partial sums. */
size_t okls_grad_norm_workspace_size(int32_t n_tensors, const okls_gradient* grads);
okls_status okls_grad_norm(int32_t n_tensors, const okls_gradient* grads, float* norm, void* workspace,
                           size_t ws_bytes, void* stream);

typedef struct {
    float* p;           /* the parameter, fp32 */
    const void* g;      /* its gradient, of g_dtype */
    void* m;            /* 32 bits: fp32 m.  8 bits: e4m3 codes of m */
    void* v;            /* 32 bits: fp32 v.  8 bits: e4m3 codes of v's root */
    uint8_t* scales;    /* 8 bits: (2, ceil(n / 128)) bytes e + 127, m's and then the root's; else NULL */
    int64_t n;          /* elements, 0..2^34 */
    int32_t g_dtype;    /* okls_dtype */
} okls_adamw_tensor;

typedef struct {
    double lr, beta1, beta2, eps, weight_decay;
    double max_norm;    /* read only with `norm` */
    int32_t moment_bits;/* 32 or 8 */
} okls_adamw_config;

/* One step t >= 1 of every tensor, in place:
 *   g <- g min(1, max_norm / (norm + 1e-6))          (only with `norm`)
 *   m <- beta1 m + (1 - beta1) g
 *   v <- beta2 v + (1 - beta2) g^2
 *   p <- (1 - lr weight_decay) p - lr / (1 - beta1^t) m / (v^1/2 / (1 - beta2^t)^1/2 + eps)
 * in fp32, the products and sums of m and v each rounded once, v's root by the
 * correctly rounded square root.  `norm`, one float on the device (okls_grad_norm's
 * result), may be NULL; where it is no finite number nothing is written at all.
 *
 * 8 bits: m and s = v^1/2 are held in e4m3 in blocks of 128 of a tensor's
 * elements, each with the power-of-two scale of okls_linear.h's 8-bit form (the root
 * takes half of v's range in exponents: e4m3's 2^18 are 2^36 of v).  The update
 * reads the old ones back, v as s^2, and takes the new ones before they are
 * rounded.  Where beta2 is 0.999 a step moves v by a thousandth, far less than
 * the 6 to 12 % between two codes: to nearest it would never move.  So a value
 * of y steps is held as floor(fl32(y + u)) steps, u in [0, 1) a multiple of
 * 2^-16 out of a hash of (t, the tensor's place in the list, the element's
 * number): each rounding is off by less than a step, up or down in proportion.
 * Roots below the smallest normal code (2^-6 of 448, 3.5e-5 of their block's
 * largest) always round up, so that a root is 0 only where it is 0 and m / s stays
 * bounded; while their block's largest root stays where it is they do not fall.  With gradients of
 * a steady size and beta2 = 0.999 a held root scatters by 15 % about v's, v is 4 % high
 * on average, and an update differs by 17 % in norm from that of moments in fp32.  NaN and infinities become NaN.
 *   hash, mod 2^32: x = (i mod 2^32) 9E3779B9h + (i / 2^32) 3C6EF372h + t 6A09E667h + place BB67AE85h,
 *   x = (x ^ x >> 16) 6A09E667h, x = (x ^ x >> 15) BB67AE85h, x = x ^ x >> 16;
 *   u = (x mod 2^16) / 2^16 for m, (x / 2^16) / 2^16 for s.
 * No tensor may overlap another. */
okls_status okls_adamw(const okls_adamw_config* config, int64_t t, int32_t n_tensors,
                       const okls_adamw_tensor* tensors, const float* norm, void* stream);

#ifdef __cplusplus
}
#endif
#endif /* OKLS_OPTIM_H_ */
