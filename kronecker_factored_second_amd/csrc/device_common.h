// Device helpers that the kernels of the 8-bit linear layer, of the experts and of
// the optimizer step over many tensors share: element types, wide loads and
// stores at any alignment, the 8-bit form of a block.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "../../include/okls_linear.h"

namespace okls {
namespace {

typedef _Float16 half_t;
typedef _Float16 half8_t __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float floatx4 __attribute__((ext_vector_type(4)));
typedef float floatx16 __attribute__((ext_vector_type(16)));
typedef int intx4 __attribute__((ext_vector_type(4)));
typedef int intx8 __attribute__((ext_vector_type(8)));
typedef uint16_t u16x8 __attribute__((ext_vector_type(8)));

struct bf16_t { uint16_t bits; };

__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ float to_f32(bf16_t v) { return __uint_as_float(static_cast<uint32_t>(v.bits) << 16); }
__device__ __forceinline__ float to_f32(half_t v) { return static_cast<float>(v); }

template <typename T> __device__ __forceinline__ T from_f32(float f);
template <> __device__ __forceinline__ float from_f32<float>(float f) { return f; }
template <> __device__ __forceinline__ bf16_t from_f32<bf16_t>(float f) { return bf16_t{__builtin_bit_cast(uint16_t, static_cast<__bf16>(f))}; }
template <> __device__ __forceinline__ half_t from_f32<half_t>(float f) { return static_cast<half_t>(f); }

// one element of a tensor whose type is known at run time (weights, outputs at an edge)
__device__ __forceinline__ float load_any(const void* p, int64_t i, int dtype) {
  if (dtype == OKLS_F32) return static_cast<const float*>(p)[i];
  if (dtype == OKLS_BF16) return to_f32(static_cast<const bf16_t*>(p)[i]);
  return to_f32(static_cast<const half_t*>(p)[i]);
}
__device__ __forceinline__ void store_any(void* p, int64_t i, int dtype, float v) {
  if (dtype == OKLS_F32) static_cast<float*>(p)[i] = v;
  else if (dtype == OKLS_BF16) static_cast<bf16_t*>(p)[i] = from_f32<bf16_t>(v);
  else static_cast<half_t*>(p)[i] = from_f32<half_t>(v);
}

// Eight consecutive elements as fp32; the first n of them (n <= 8) exist, the
// others are zero.  Global memory takes 16-byte accesses at any element's
// alignment, so rows that start anywhere need no path of their own.
typedef u16x8 u16x8_any __attribute__((aligned(2)));
typedef floatx4 floatx4_any __attribute__((aligned(4)));
// the eight as they lie in memory: four registers for 16-bit types
template <typename T> struct Raw8 { u16x8 v; };
template <> struct Raw8<float> { floatx4 a, b; };
template <typename T>
__device__ __forceinline__ Raw8<T> raw8(const T* p, int n) {
  Raw8<T> r{};
  if constexpr (sizeof(T) == 4) {
    if (n >= 8) {
      r.a = reinterpret_cast<const floatx4_any*>(p)[0], r.b = reinterpret_cast<const floatx4_any*>(p)[1];
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if (j < n) r.a[j] = p[j];
        if (4 + j < n) r.b[j] = p[4 + j];
      }
    }
  } else {
    if (n >= 8) {
      r.v = *reinterpret_cast<const u16x8_any*>(p);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (j < n) r.v[j] = __builtin_bit_cast(uint16_t, p[j]);
    }
  }
  return r;
}
template <typename T>
__device__ __forceinline__ float element(const Raw8<T>& r, int j) {
  if constexpr (sizeof(T) == 4) return j < 4 ? r.a[j & 3] : r.b[j & 3];
  else return to_f32(__builtin_bit_cast(T, static_cast<uint16_t>(r.v[j])));
}
template <typename T>
__device__ __forceinline__ void widen8(float (&v)[8], const Raw8<T>& r) {
#pragma unroll
  for (int j = 0; j < 8; ++j) v[j] = element(r, j);
}
template <typename T>
__device__ __forceinline__ void load8(float (&v)[8], const T* p, int n) {
  widen8(v, raw8(p, n));
}
template <typename T>
__device__ __forceinline__ void store8(T* p, const float (&v)[8], int n) {
  if (n >= 8) {
    if constexpr (sizeof(T) == 4) {
      reinterpret_cast<floatx4_any*>(p)[0] = floatx4{v[0], v[1], v[2], v[3]};
      reinterpret_cast<floatx4_any*>(p)[1] = floatx4{v[4], v[5], v[6], v[7]};
    } else {
      u16x8 a;
#pragma unroll
      for (int j = 0; j < 8; ++j) a[j] = __builtin_bit_cast(uint16_t, from_f32<T>(v[j]));
      *reinterpret_cast<u16x8_any*>(p) = a;
    }
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (j < n) p[j] = from_f32<T>(v[j]);
  }
}
__device__ __forceinline__ void load8_any(float (&v)[8], const void* p, int64_t i, int n, int dtype) {
  if (dtype == OKLS_F32) load8(v, static_cast<const float*>(p) + i, n);
  else if (dtype == OKLS_BF16) load8(v, static_cast<const bf16_t*>(p) + i, n);
  else load8(v, static_cast<const half_t*>(p) + i, n);
}

__device__ __forceinline__ int clamp8(int64_t left) { return left >= 8 ? 8 : left > 0 ? static_cast<int>(left) : 0; }

// ---------------------------------------------------------------------------
// The 8-bit form
// ---------------------------------------------------------------------------

// |v| as the bits of its float, 0 for NaN and infinities: non-negative floats
// order as their bits do, so the block maximum is an integer maximum
__device__ __forceinline__ uint32_t finite_abs(float v) {
  const uint32_t u = __float_as_uint(v) & 0x7fffffffu;
  return u >= 0x7f800000u ? 0u : u;
}
// The scale byte e + 127 of a block whose largest finite |v| has the bits
// `top`: F = 1.75 2^T (T = 8 for e4m3, 15 for e5m2), so e is top's exponent
// less T, and one more where its significand is above 1.75.  Subnormals have
// exponent field 0 and clamp with the small normal numbers at byte 0.
template <int FMT>
__device__ __forceinline__ uint32_t scale_byte(uint32_t top) {
  constexpr int T = FMT == OKLS_E4M3 ? 8 : 15;
  const int b = static_cast<int>(top >> 23) - T + ((top & 0x7fffffu) > 0x600000u ? 1 : 0);
  return top == 0 ? 127u : static_cast<uint32_t>(b > 0 ? b : 0);
}
// 2^-e: byte is at most 247, so the field 254 - byte is a normal number's
__device__ __forceinline__ float scale_inverse(uint32_t byte) { return __uint_as_float((254u - byte) << 23); }

template <int FMT>
__device__ __forceinline__ uint32_t codes4(float a, float b, float c, float d) {
  int r = 0;
  if constexpr (FMT == OKLS_E4M3) {
    r = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, r, false);
    r = __builtin_amdgcn_cvt_pk_fp8_f32(c, d, r, true);
  } else {
    r = __builtin_amdgcn_cvt_pk_bf8_f32(a, b, r, false);
    r = __builtin_amdgcn_cvt_pk_bf8_f32(c, d, r, true);
  }
  return static_cast<uint32_t>(r);
}
template <int FMT>
__device__ __forceinline__ uint2 codes8(const float (&v)[8], float inv) {
  return uint2{codes4<FMT>(v[0] * inv, v[1] * inv, v[2] * inv, v[3] * inv),
               codes4<FMT>(v[4] * inv, v[5] * inv, v[6] * inv, v[7] * inv)};
}
__device__ __forceinline__ uint32_t max_u32(uint32_t a, uint32_t b) { return a > b ? a : b; }
// the maximum over each 16 neighbouring lanes, in all of them: lane exchanges
// inside the ALU (pairs, pairs of pairs, mirrored halves, mirrored row)
__device__ __forceinline__ uint32_t max16(uint32_t v) {
  auto other = [](uint32_t x, auto ctrl) { return static_cast<uint32_t>(__builtin_amdgcn_mov_dpp(static_cast<int>(x), decltype(ctrl)::value, 0xf, 0xf, true)); };
  v = max_u32(v, other(v, std::integral_constant<int, 0xb1>{}));
  v = max_u32(v, other(v, std::integral_constant<int, 0x4e>{}));
  v = max_u32(v, other(v, std::integral_constant<int, 0x141>{}));
  return max_u32(v, other(v, std::integral_constant<int, 0x140>{}));
}

// calls go(T{}) with the element type of dtype
template <class F>
void by_type(int dtype, F go) {
  if (dtype == OKLS_F32) go(float{});
  else if (dtype == OKLS_BF16) go(bf16_t{});
  else go(half_t{});
}
int blocks_up_to(int64_t n, int most) { return static_cast<int>(n < most ? n : most); }

}  // namespace
}  // namespace okls
