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

// four e4m3 codes as fp32
__device__ __forceinline__ void decode4(float (&v)[4], uint32_t w) {
  const auto lo = __builtin_amdgcn_cvt_pk_f32_fp8(static_cast<int>(w), false), hi = __builtin_amdgcn_cvt_pk_f32_fp8(static_cast<int>(w), true);
  v[0] = lo[0], v[1] = lo[1], v[2] = hi[0], v[3] = hi[1];
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

// Four neighbouring elements at any place, the first n of them; a wave's lie side by
// side, so that each access is of whole lines, and passes the caches by where
// ONCE: nothing here is read again.
typedef uint16_t u16x4 __attribute__((ext_vector_type(4)));
typedef u16x4 u16x4_any __attribute__((aligned(2)));
typedef uint32_t u32_any __attribute__((aligned(1)));

template <typename T>
__device__ __forceinline__ void load4(float (&v)[4], const T* p, int n) {
  if (n >= 4) {
    if constexpr (sizeof(T) == 4) {
      const floatx4 x = __builtin_nontemporal_load(reinterpret_cast<const floatx4_any*>(p));
#pragma unroll
      for (int j = 0; j < 4; ++j) v[j] = x[j];
    } else {
      const u16x4 x = __builtin_nontemporal_load(reinterpret_cast<const u16x4_any*>(p));
#pragma unroll
      for (int j = 0; j < 4; ++j) v[j] = to_f32(__builtin_bit_cast(T, static_cast<uint16_t>(x[j])));
    }
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j] = j < n ? to_f32(p[j]) : 0.0f;
  }
}
__device__ __forceinline__ void store4(float* p, const float (&v)[4], int n) {
  if (n >= 4) {
    const floatx4 x = {v[0], v[1], v[2], v[3]};
    __builtin_nontemporal_store(x, reinterpret_cast<floatx4_any*>(p));
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (j < n) p[j] = v[j];
  }
}
__device__ __forceinline__ uint32_t codes4_at(const uint8_t* p, int n) {
  if (n >= 4) return __builtin_nontemporal_load(reinterpret_cast<const u32_any*>(p));
  uint32_t w = 0;
#pragma unroll
  for (int j = 0; j < 4; ++j)
    if (j < n) w |= static_cast<uint32_t>(p[j]) << (8 * j);
  return w;
}

// four values of a block of 128, which 32 neighbouring lanes hold
template <bool UP>
__device__ __forceinline__ void round4(const float (&x)[4], const uint32_t (&h)[4], uint8_t* codes, uint8_t* scale, int n) {
  uint32_t top = 0;
#pragma unroll
  for (int j = 0; j < 4; ++j) top = max_u32(top, finite_abs(x[j]));
  top = max16(top);
  top = max_u32(top, static_cast<uint32_t>(__builtin_amdgcn_ds_swizzle(static_cast<int>(top), 0x401f)));    // the lane 16 further on, or back
  const uint32_t byte = scale_byte<OKLS_E4M3>(top);
  const float inv = scale_inverse(byte);
  uint32_t w = 0;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const uint32_t half = UP ? h[j] >> 16 : h[j] & 0xffffu;
    w |= code_of<UP>(x[j], inv, static_cast<float>(half) * 0x1p-16f) << (8 * j);
  }
  if (n >= 4) {
    __builtin_nontemporal_store(w, reinterpret_cast<u32_any*>(codes));
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (j < n) codes[j] = static_cast<uint8_t>(w >> (8 * j));
  }
  if ((threadIdx.x & 31) == 0 && n > 0) *scale = static_cast<uint8_t>(byte);
}

__device__ __forceinline__ int clamp4(int64_t left) { return left >= 4 ? 4 : left > 0 ? static_cast<int>(left) : 0; }

// A thread's elements, kAdamParts times four of them.  The gradient's type is known here,
// so that every load is on its way before the first is used.
// Bound by memory: 103M elements with bf16 gradients and fp32 moments (2.68 GB) take
// 404 us, 6.6 TB/s; 92M with fp32 gradients and 8-bit moments (1.48 GB) 252 to 263, 5.6
// to 5.9 (a large copy runs at 4.7 to 5).  Eight neighbouring elements a thread, through the caches,
// took 469 and 286 us; past the caches that way, in half lines, the second took 393.
// 1024 or 4096 elements a workgroup take the second to 289 and 285.
constexpr int kAdamParts = kAdamChunk / 1024;
template <typename G, bool EIGHT>
__device__ __forceinline__ void adamw_part(const AdamArgs& a, const AdamTensor& t, int64_t first, float factor) {
  constexpr int Q = kAdamParts;
  float p[Q][4], g[Q][4], m[Q][4], v[Q][4], s[Q][4], scale_m[Q], scale_s[Q];
  uint32_t cm[Q], cs[Q];
  const int64_t blocks = (t.n + 127) >> 7;
  uint8_t *codes_m = static_cast<uint8_t*>(t.m), *codes_s = static_cast<uint8_t*>(t.v);
#pragma unroll
  for (int q = 0; q < Q; ++q) {
    const int64_t i = first + q * 1024;
    const int n = clamp4(t.n - i);
    load4(p[q], t.p + i, n);
    load4(g[q], static_cast<const G*>(t.g) + i, n);
    if constexpr (EIGHT) {
      scale_m[q] = n > 0 ? scale_value(t.scales[i >> 7]) : 0.0f;
      scale_s[q] = n > 0 ? scale_value(t.scales[blocks + (i >> 7)]) : 0.0f;
      cm[q] = codes4_at(codes_m + i, n);
      cs[q] = codes4_at(codes_s + i, n);
    } else {
      load4(m[q], static_cast<const float*>(t.m) + i, n);
      load4(v[q], static_cast<const float*>(t.v) + i, n);
    }
  }
#pragma unroll
  for (int q = 0; q < Q; ++q) {
    const int64_t i = first + q * 1024;
    const int n = clamp4(t.n - i);
    if constexpr (EIGHT) {
      decode4(m[q], cm[q]);
      decode4(s[q], cs[q]);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        m[q][j] = m[q][j] * scale_m[q];
        s[q][j] = s[q][j] * scale_s[q];
        v[q][j] = s[q][j] * s[q][j];
      }
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if (a.norm != nullptr) g[q][j] = g[q][j] * factor;
      m[q][j] = a.beta1 * m[q][j] + a.rest1 * g[q][j];
      v[q][j] = a.beta2 * v[q][j] + a.rest2 * g[q][j] * g[q][j];
      s[q][j] = __fsqrt_rn(v[q][j]);
      p[q][j] = p[q][j] * a.decay - a.step * (m[q][j] / (s[q][j] * a.unbias2 + a.eps));
    }
    store4(t.p + i, p[q], n);
    if constexpr (EIGHT) {
      uint32_t h[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint64_t e = static_cast<uint64_t>(i + j);
        uint32_t x = static_cast<uint32_t>(e) * 0x9E3779B9u + static_cast<uint32_t>(e >> 32) * 0x3C6EF372u + t.key;
        x = (x ^ x >> 16) * 0x6A09E667u;
        x = (x ^ x >> 15) * 0xBB67AE85u;
        h[j] = x ^ x >> 16;
        // past the tensor's end nothing joins the block's maximum
        if (j >= n) m[q][j] = s[q][j] = 0.0f;
      }
      round4<false>(m[q], h, codes_m + i, t.scales + (i >> 7), n);
      round4<true>(s[q], h, codes_s + i, t.scales + blocks + (i >> 7), n);
    } else {
      store4(static_cast<float*>(t.m) + i, m[q], n);
      store4(static_cast<float*>(t.v) + i, v[q], n);
    }
  }
}

// kAdamChunk elements of one tensor a workgroup.
template <bool EIGHT>
__global__ __launch_bounds__(256) void adamw_kernel(AdamArgs a) {
  const int at = __builtin_amdgcn_readfirstlane(tensor_of(a.tensor, a.count, blockIdx.x));
  const AdamTensor& t = a.tensor[at];
  const int64_t first = static_cast<int64_t>(blockIdx.x - t.first) * kAdamChunk + threadIdx.x * 4;
  float factor = 1.0f;
  if (a.norm != nullptr) {
    const float norm = *a.norm;
    if (!(fabsf(norm) < __builtin_inff())) return;
    const double f = a.max_norm / (static_cast<double>(norm) + 1e-6);
    factor = static_cast<float>(f < 1.0 ? f : 1.0);
  }
  const int dtype = a.dtype[at];
  if (dtype == OKLS_F32) adamw_part<float, EIGHT>(a, t, first, factor);
  else if (dtype == OKLS_BF16) adamw_part<bf16_t, EIGHT>(a, t, first, factor);
  else adamw_part<half_t, EIGHT>(a, t, first, factor);
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
// (with the type looked up at each load 65 us for 103M bf16 elements, now 37 behind an
// AdamW step and 57 behind work that fills the last-level cache)
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
