// gfx950 kernels of the optimizer step over many tensors (okls_optim.h).
//
//  adamw_kernel      AdamW with moments in fp32 or in blocks of 8 bits.
//  grad_norm_kernel  partial sums of squares of all gradients; join_norm_kernel
//                    adds them.
#include "device_common.h"
#include "optim_kernels.h"

#include "../../include/okls_optim.h"

// the definition rounds every product and sum by itself
#pragma clang fp contract(off)

namespace okls {
namespace {

// the last of `count` <= 64 tensors whose first workgroup is not behind this one: each lane looks at one
template <class T>
__device__ __forceinline__ int tensor_of(const T* t, int count, unsigned block) {
  const int lane = threadIdx.x & 63;
  return __popcll(__ballot(lane < count && t[lane < count ? lane : 0].first <= block)) - 1;
}

// What a block's scale byte stands for: 2^(byte - 127)
__device__ __forceinline__ float scale_value(uint32_t byte) { return __uint_as_float(byte == 0 ? 1u << 22 : byte << 23); }

// eight e4m3 codes as fp32
__device__ __forceinline__ void decode8(float (&v)[8], uint2 c) {
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const uint32_t w = h ? c.y : c.x;
    const auto lo = __builtin_amdgcn_cvt_pk_f32_fp8(static_cast<int>(w), false), hi = __builtin_amdgcn_cvt_pk_f32_fp8(static_cast<int>(w), true);
    v[4 * h] = lo[0], v[4 * h + 1] = lo[1], v[4 * h + 2] = hi[0], v[4 * h + 3] = hi[1];
  }
}

// The e4m3 code of x, |x| inv <= 448: y = |x| inv in steps of its size (8 to 16
// of them, fewer below the smallest normal code 2^-6), held as floor(y + u), or as
// ceil(y) below it where UP.  Codes count steps through all sizes, so 16 steps
// of one size are 8 of the next.
template <bool UP>
__device__ __forceinline__ uint32_t code_of(float x, float inv, float u) {
  const uint32_t bits = __float_as_uint(fabsf(x) * inv);
  const uint32_t size = max_u32(bits >> 23, 121u);
  const float y = __uint_as_float(bits) * __uint_as_float((257u - size) << 23);
  uint32_t k = static_cast<uint32_t>(y + u);
  if (UP && bits >> 23 < 121u) k = static_cast<uint32_t>(ceilf(y));
  uint32_t code = ((size - 121u) << 3) + k;
  code = code > 0x7eu ? 0x7eu : code;
  if (bits >= 0x7f800000u) code = 0x7fu;
  return code | (__float_as_uint(x) >> 31 << 7);
}

template <bool UP>
__device__ __forceinline__ void round8(const float (&x)[8], const uint32_t (&h)[8], uint8_t* codes, uint8_t* scale, int n) {
  uint32_t top = 0;
#pragma unroll
  for (int j = 0; j < 8; ++j) top = max_u32(top, finite_abs(x[j]));
  const uint32_t byte = scale_byte<OKLS_E4M3>(max16(top));
  const float inv = scale_inverse(byte);
  uint32_t w[2] = {0, 0};
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const uint32_t half = UP ? h[j] >> 16 : h[j] & 0xffffu;
    w[j >> 2] |= code_of<UP>(x[j], inv, static_cast<float>(half) * 0x1p-16f) << (8 * (j & 3));
  }
  if (n == 8) {
    typedef uint32_t u32x2_any __attribute__((ext_vector_type(2), aligned(1)));
    typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
    *reinterpret_cast<u32x2_any*>(codes) = u32x2{w[0], w[1]};
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (j < n) codes[j] = static_cast<uint8_t>(w[j >> 2] >> (8 * (j & 3)));
  }
  if ((threadIdx.x & 15) == 0 && n > 0) *scale = static_cast<uint8_t>(byte);
}

__device__ __forceinline__ uint2 codes_at(const uint8_t* codes, int n) {
  typedef uint32_t u32x2_any __attribute__((ext_vector_type(2), aligned(1)));
  if (n == 8) {
    const u32x2_any w = *reinterpret_cast<const u32x2_any*>(codes);
    return uint2{w[0], w[1]};
  }
  uint32_t w[2] = {0, 0};
#pragma unroll
  for (int j = 0; j < 8; ++j)
    if (j < n) w[j >> 2] |= static_cast<uint32_t>(codes[j]) << (8 * (j & 3));
  return uint2{w[0], w[1]};
}

// One thread's eight elements.  The gradient's type is known here, so that every
// load is on its way before the first is used.
template <typename G, bool EIGHT>
__device__ __forceinline__ void adamw8(const AdamArgs& a, const AdamTensor& t, int64_t i, int n, float factor) {
  float p[8], g[8], m[8], v[8], s[8];
  const int64_t blocks = (t.n + 127) >> 7, block = i >> 7;
  load8(p, t.p + i, n);
  const Raw8<G> raw = raw8(static_cast<const G*>(t.g) + i, n);
  if constexpr (EIGHT) {
    const float scale_m = n > 0 ? scale_value(t.scales[block]) : 0.0f, scale_s = n > 0 ? scale_value(t.scales[blocks + block]) : 0.0f;
    decode8(m, codes_at(static_cast<const uint8_t*>(t.m) + i, n));
    decode8(s, codes_at(static_cast<const uint8_t*>(t.v) + i, n));
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      m[j] = m[j] * scale_m;
      s[j] = s[j] * scale_s;
      v[j] = s[j] * s[j];
    }
  } else {
    load8(m, static_cast<const float*>(t.m) + i, n);
    load8(v, static_cast<const float*>(t.v) + i, n);
  }
  widen8(g, raw);
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    if (a.norm != nullptr) g[j] = g[j] * factor;
    m[j] = a.beta1 * m[j] + a.rest1 * g[j];
    v[j] = a.beta2 * v[j] + a.rest2 * g[j] * g[j];
    s[j] = __fsqrt_rn(v[j]);
    p[j] = p[j] * a.decay - a.step * (m[j] / (s[j] * a.unbias2 + a.eps));
  }
  store8(t.p + i, p, n);
  if constexpr (EIGHT) {
    uint32_t h[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const uint64_t e = static_cast<uint64_t>(i + j);
      uint32_t x = static_cast<uint32_t>(e) * 0x9E3779B9u + static_cast<uint32_t>(e >> 32) * 0x3C6EF372u + t.key;
      x = (x ^ x >> 16) * 0x6A09E667u;
      x = (x ^ x >> 15) * 0xBB67AE85u;
      h[j] = x ^ x >> 16;
      // past the tensor's end nothing joins the block's maximum
      if (j >= n) m[j] = s[j] = 0.0f;
    }
    round8<false>(m, h, static_cast<uint8_t*>(t.m) + i, t.scales + block, n);
    round8<true>(s, h, static_cast<uint8_t*>(t.v) + i, t.scales + blocks + block, n);
  } else {
    store8(static_cast<float*>(t.m) + i, m, n);
    store8(static_cast<float*>(t.v) + i, v, n);
  }
}

// 2048 elements of one tensor a workgroup, eight a thread: a block of 128 is 16
// neighbouring lanes.
template <bool EIGHT>
__global__ __launch_bounds__(256) void adamw_kernel(AdamArgs a) {
  const int at = __builtin_amdgcn_readfirstlane(tensor_of(a.tensor, a.count, blockIdx.x));
  const AdamTensor& t = a.tensor[at];
  const int64_t i = static_cast<int64_t>(blockIdx.x - t.first) * kAdamChunk + threadIdx.x * 8;
  const int n = clamp8(t.n - i);
  float factor = 1.0f;
  if (a.norm != nullptr) {
    const float norm = *a.norm;
    if (!(fabsf(norm) < __builtin_inff())) return;
    const double f = a.max_norm / (static_cast<double>(norm) + 1e-6);
    factor = static_cast<float>(f < 1.0 ? f : 1.0);
  }
  const int dtype = a.dtype[at];
  if (dtype == OKLS_F32) adamw8<float, EIGHT>(a, t, i, n, factor);
  else if (dtype == OKLS_BF16) adamw8<bf16_t, EIGHT>(a, t, i, n, factor);
  else adamw8<half_t, EIGHT>(a, t, i, n, factor);
}

template <int THREADS>
__device__ __forceinline__ double block_sum(double v) {
  __shared__ double sh[THREADS / 64];
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) v += __shfl_xor(v, o, 64);
  if ((threadIdx.x & 63) == 0) sh[threadIdx.x >> 6] = v;
  __syncthreads();
  v = 0.0;
#pragma unroll
  for (int q = 0; q < THREADS / 64; ++q) v += sh[q];
  return v;
}

// a thread's share of a chunk's squares: its type known, so that four loads are on their way at once
template <typename G>
__device__ __forceinline__ double squares(const NormTensor& t, int64_t first) {
  double sum = 0.0;
  for (int64_t i = first + threadIdx.x * 8; i < t.n && i < first + kNormChunk; i += 4 * 2048) {
    Raw8<G> g[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) g[q] = raw8(static_cast<const G*>(t.g) + i + q * 2048, clamp8(t.n - i - q * 2048));
#pragma unroll
    for (int q = 0; q < 4; ++q)
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const double v = element(g[q], j);
        sum = fma(v, v, sum);
      }
  }
  return sum;
}

__global__ __launch_bounds__(256) void grad_norm_kernel(GradNormArgs a) {
  const int half = a.count < 64 ? a.count : 64;
  int at = tensor_of(a.tensor, half, blockIdx.x);
  if (a.count > 64) at += tensor_of(a.tensor + 64, a.count - 64, blockIdx.x) + 1;
  const NormTensor& t = a.tensor[__builtin_amdgcn_readfirstlane(at)];
  const int64_t first = static_cast<int64_t>(blockIdx.x - t.first) * kNormChunk;
  double sum;
  if (t.dtype == OKLS_F32) sum = squares<float>(t, first);
  else if (t.dtype == OKLS_BF16) sum = squares<bf16_t>(t, first);
  else sum = squares<half_t>(t, first);
  sum = block_sum<256>(sum);
  if (threadIdx.x == 0) a.part[blockIdx.x] = sum;
}

__global__ __launch_bounds__(1024) void join_norm_kernel(const double* part, int64_t n, float* norm) {
  double sum = 0.0;
  for (int64_t i = threadIdx.x; i < n; i += 1024) sum += part[i];
  sum = block_sum<1024>(sum);
  if (threadIdx.x == 0) *norm = static_cast<float>(sqrt(sum));
}

}  // namespace

hipError_t launch_adamw(const AdamArgs& a, unsigned blocks, bool eight, hipStream_t s) {
  if (eight) adamw_kernel<true><<<blocks, 256, 0, s>>>(a);
  else adamw_kernel<false><<<blocks, 256, 0, s>>>(a);
  return hipGetLastError();
}

hipError_t launch_grad_norm(const GradNormArgs& a, unsigned blocks, hipStream_t s) {
  grad_norm_kernel<<<blocks, 256, 0, s>>>(a);
  return hipGetLastError();
}

hipError_t launch_join_norm(const double* part, int64_t n, float* norm, hipStream_t s) {
  join_norm_kernel<<<1, 1024, 0, s>>>(part, n, norm);
  return hipGetLastError();
}

}  // namespace okls
