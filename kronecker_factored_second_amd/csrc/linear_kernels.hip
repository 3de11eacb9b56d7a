// gfx950 kernels of the 8-bit linear-layer operators (okls_linear.h).
//
//  quantize_kernel   a 128 x 128 tile of x in registers, its 8-bit form along
//                    the rows, along the columns, or both from the one read.
//  rms_norm_kernel   residual addition, fp64 mean square, 8-bit output.
//  norm_grad_kernel  dx and partial sums of dweight; norm_dw_kernel joins them.
//  matmul kernels    c = a b^T on the scaled 8-bit matrix instructions, whose
//                    E8M0 operand scales apply the block scales for free, or
//                    on bf16 ones: tiles through LDS (matmul_tile_kernel), or
//                    straight from memory for few rows (matmul_few_kernel).
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "../../include/okls_linear.h"
#include "linear_kernels.h"

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

// One 128 x 128 tile per pass, 256 threads: thread t holds rows 8 (t / 16) + p
// and columns 8 (t % 16) + j, as they lie in memory: 16-bit types take half the
// registers, so more waves hide the loads.  A row's maximum is over 16
// neighbouring lanes, a column's over the four lane groups of a wave and,
// through LDS, the four waves.  The transposed codes go through LDS so that
// they leave as whole rows of 128 bytes.
// Bound by memory: bf16 16384 x 5632 both ways moves 371 MB in 81 us (4.6 TB/s;
// a large copy runs at 4.7), fp32 11008 x 4096 in 50 us (5.4 TB/s), one way of
// the first in 45 us (6.2 TB/s).  Held as floats, three waves a SIMD, the first
// took 110 us.  Small matrices are bound by one tile's chain of loads, maxima
// and barriers, about 7 us.
constexpr int kTileStride = 128 + 16;   // bytes; 16-byte rows that start at different banks

template <typename T, int FMT, bool FACTORS>
__global__ __launch_bounds__(256, FACTORS ? 3 : 4) void quantize_kernel(QuantArgs a) {
  __shared__ uint32_t col_top[4][128];
  __shared__ __attribute__((aligned(16))) uint8_t tile[128 * kTileStride];
  const int t = threadIdx.x, c8 = t & 15, rg = t >> 4, wave = t >> 6;
  const int64_t tiles_c = (a.cols + 127) >> 7, n_tiles = tiles_c * ((a.rows + 127) >> 7);
  const T* x = static_cast<const T*>(a.x);
  for (int64_t it = blockIdx.x; it < n_tiles; it += gridDim.x) {
    const int64_t br = it / tiles_c, bc = it - br * tiles_c;
    const int64_t r0 = br * 128 + rg * 8, c0 = bc * 128 + c8 * 8;
    const int nc = clamp8(a.cols - c0);
    Raw8<T> raw[8];
#pragma unroll
    for (int p = 0; p < 8; ++p) raw[p] = raw8(x + (r0 + p) * a.ldx + c0, r0 + p < a.rows ? nc : 0);
    float made[FACTORS ? 8 : 1][8];
    if constexpr (FACTORS) {
      float cf[8];
      load8_any(cf, a.col_factor, c0, nc, a.col_dtype);
#pragma unroll
      for (int p = 0; p < 8; ++p) {
        const float rf = r0 + p < a.rows ? a.row_factor[r0 + p] : 0.0f;
        // no value past the matrix's end, where 0 times a factor's infinity or NaN would not be 0
#pragma unroll
        for (int j = 0; j < 8; ++j) made[p][j] = j < nc && r0 + p < a.rows ? element(raw[p], j) * rf * cf[j] : 0.0f;
      }
    }
    auto value = [&](int p, int j) {
      if constexpr (FACTORS) return made[p][j];
      else return element(raw[p], j);
    };
    if (a.along_cols.codes != nullptr) {
      const Blocked& o = a.along_cols;
      uint64_t bytes = 0;
#pragma unroll
      for (int p = 0; p < 8; ++p) {
        uint32_t top = 0;
        float v[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          v[j] = value(p, j);
          top = max_u32(top, finite_abs(v[j]));
        }
        top = max16(top);
        const uint32_t byte = scale_byte<FMT>(top);
        bytes |= static_cast<uint64_t>(byte) << (8 * p);
        if (r0 + p < a.rows)
          *reinterpret_cast<uint2*>(o.codes + (r0 + p) * o.ld + c0) = codes8<FMT>(v, scale_inverse(byte));
      }
      // rows past the end have the scale of zeros; the row stride is padded to 16
      if (c8 == 0 && r0 < o.ld_scale && r0 < ((a.rows + 15) & ~int64_t(15)))
        *reinterpret_cast<uint64_t*>(o.scales + bc * o.ld_scale + r0) = bytes;
    }
    if (a.along_rows.codes != nullptr) {
      const Blocked& o = a.along_rows;
      uint32_t top[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        top[j] = 0;
#pragma unroll
        for (int p = 0; p < 8; ++p) top[j] = max_u32(top[j], finite_abs(value(p, j)));
        top[j] = max_u32(top[j], __shfl_xor(top[j], 16, 64));
        top[j] = max_u32(top[j], __shfl_xor(top[j], 32, 64));
      }
      if ((t & 63) < 16)
#pragma unroll
        for (int j = 0; j < 8; ++j) col_top[wave][c8 * 8 + j] = top[j];
      __syncthreads();
      uint64_t bytes = 0;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        uint32_t m = 0;
#pragma unroll
        for (int w = 0; w < 4; ++w) m = max_u32(m, col_top[w][c8 * 8 + j]);
        const uint32_t byte = scale_byte<FMT>(m);
        bytes |= static_cast<uint64_t>(byte) << (8 * j);
        float u[8];
#pragma unroll
        for (int p = 0; p < 8; ++p) u[p] = value(p, j);
        *reinterpret_cast<uint2*>(tile + (c8 * 8 + j) * kTileStride + rg * 8) = codes8<FMT>(u, scale_inverse(byte));
      }
      if (rg == 0 && c0 < ((a.cols + 15) & ~int64_t(15)))
        *reinterpret_cast<uint64_t*>(o.scales + br * o.ld_scale + c0) = bytes;
      __syncthreads();
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int col = q * 32 + (t >> 3), chunk = t & 7;
        if (bc * 128 + col < a.cols)
          *reinterpret_cast<uint4*>(o.codes + (bc * 128 + col) * o.ld + br * 128 + chunk * 16) =
              *reinterpret_cast<const uint4*>(tile + col * kTileStride + chunk * 16);
      }
      __syncthreads();   // the next tile writes both LDS arrays
    }
  }
}

// ---------------------------------------------------------------------------
// Norm
// ---------------------------------------------------------------------------

// A row by a wave (THR = 64, four rows a workgroup) or by a workgroup of as
// many waves as it fills, THR threads at most; its NC chunks of 8 elements a
// thread are held in registers from the one read of it.  Wider rows (NC = 0)
// are read again for the second pass.
// Bound by memory: 16384 x 2048 bf16 with the residual moves 235 MB in 47 us
// (5.0 TB/s); read twice by 256 threads it took 66.  A single token is bound
// by the launch and one chain of load, fp64 sum and store, 3.7 us.
template <int THR> constexpr int kThreads = THR > 64 ? THR : 256;

// the sum of v over a row's threads, in each of them, in a fixed order
template <int THR, typename V>
__device__ __forceinline__ V row_sum(V v, V* sh) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) v += __shfl_xor(v, o, 64);
  if constexpr (THR > 64) {
    if ((threadIdx.x & 63) == 0) sh[threadIdx.x >> 6] = v;
    __syncthreads();
    v = sh[0];
    for (int q = 1; q < static_cast<int>(blockDim.x >> 6); ++q) v += sh[q];
    __syncthreads();
  }
  return v;
}

template <typename T, int FMT, int THR, int NC>
__global__ __launch_bounds__(kThreads<THR>) void rms_norm_kernel(NormArgs a) {
  __shared__ double sh[16];
  constexpr int ROWS = THR == 64 ? 4 : 1;
  const int thr = THR == 64 ? 64 : blockDim.x, t = THR == 64 ? threadIdx.x % 64 : threadIdx.x;
  const T* x = static_cast<const T*>(a.x);
  const T* res = static_cast<const T*>(a.residual);
  T* hs = static_cast<T*>(a.h);
  const int64_t chunks = ((a.cols + 127) >> 7) * 16;   // whole blocks: past the end v = 0
  for (int64_t row = static_cast<int64_t>(blockIdx.x) * ROWS + (THR == 64 ? threadIdx.x / 64 : 0); row < a.rows; row += static_cast<int64_t>(gridDim.x) * ROWS) {
    auto read = [&](float (&v)[8], int64_t c) { load8(v, x + row * a.ldx + c * 8, clamp8(a.cols - c * 8)); };
    auto add = [&](float (&v)[8], int64_t c) {
      const int n = clamp8(a.cols - c * 8);
      float r[8];
      load8(r, res + row * a.ldr + c * 8, n);
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = to_f32(from_f32<T>(v[j] + r[j]));
      store8(hs + row * a.ldh + c * 8, v, n);
    };
    auto squares = [&](const float (&v)[8], double ss) {
#pragma unroll
      for (int j = 0; j < 8; ++j) ss = fma(static_cast<double>(v[j]), static_cast<double>(v[j]), ss);
      return ss;
    };
    auto write = [&](float (&v)[8], int64_t c, float rstd) {
      const int n = clamp8(a.cols - c * 8);
      float w[8];
      load8_any(w, a.weight, c * 8, n, a.weight_dtype);
      uint32_t top = 0;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        v[j] = j < n ? v[j] * rstd * w[j] : 0.0f;
        top = max_u32(top, finite_abs(v[j]));
      }
      top = max16(top);
      const uint32_t byte = scale_byte<FMT>(top);
      *reinterpret_cast<uint2*>(a.out.codes + row * a.out.ld + c * 8) = codes8<FMT>(v, scale_inverse(byte));
      if ((t & 15) == 0) a.out.scales[(c >> 4) * a.out.ld_scale + row] = static_cast<uint8_t>(byte);
    };
    auto rms = [&](double ss) {
      ss = row_sum<THR>(ss, sh);
      const float rstd = static_cast<float>(1.0 / sqrt(ss / static_cast<double>(a.cols) + static_cast<double>(a.eps)));
      if (t == 0) a.rstd[row] = rstd;
      return rstd;
    };
    double ss = 0.0;
    if constexpr (NC != 0) {
      float v[NC][8];
#pragma unroll
      for (int i = 0; i < NC; ++i) read(v[i], t + i * thr);      // nothing past the end
      if (res != nullptr)
#pragma unroll
        for (int i = 0; i < NC; ++i) add(v[i], t + i * thr);
#pragma unroll
      for (int i = 0; i < NC; ++i) ss = squares(v[i], ss);
      const float rstd = rms(ss);
#pragma unroll
      for (int i = 0; i < NC; ++i)
        if (t + i * thr < chunks) write(v[i], t + i * thr, rstd);
    } else {
      float v[8];
      for (int64_t c = t; c < chunks; c += thr) {
        read(v, c);
        if (res != nullptr) add(v, c);
        ss = squares(v, ss);
      }
      const float rstd = rms(ss);
      // the sum from where this thread put it: x or the residual may be the same memory
      for (int64_t c = t; c < chunks; c += thr) {
        if (res != nullptr) load8(v, hs + row * a.ldh + c * 8, clamp8(a.cols - c * 8));
        else read(v, c);
        write(v, c, rstd);
      }
    }
  }
}

constexpr int kGradBlocks = 1024;   // most workgroups of a launch, each with one row of partial sums of dweight

// The same layout.  A thread meets the same columns in every row, so dweight's
// sums stay in its registers, in fp32: ceil(rows / workgroups) terms one after
// the other, a quarter of that where a wave takes a row, so 16 in a batch of
// 16384 x 2048 and 1024 in 2^20 rows of it.  A workgroup leaves one row of
// partial sums, which norm_dw_kernel adds in fp64.
// Bound by memory: 16384 x 2048 bf16 with dh moves 268 MB in 57 us (4.7 TB/s,
// the join's 5 us included); with the sums in memory it took 172 us, with dy and
// h held as floats 99.  fp32 777 x 5121 takes 18 us for 48 MB: its partial rows,
// a third of the matrix, and the join's launch are the rest.
template <typename T, int THR, int NC>
__global__ __launch_bounds__(kThreads<THR>) void norm_grad_kernel(NormGradArgs a) {
  constexpr int ROWS = THR == 64 ? 4 : 1;
  __shared__ float sh[16];
  const int thr = THR == 64 ? 64 : blockDim.x, t = THR == 64 ? threadIdx.x % 64 : threadIdx.x;
  const T* dy = static_cast<const T*>(a.dy);
  const T* h = static_cast<const T*>(a.h);
  const T* dh = static_cast<const T*>(a.dh);
  T* dx = static_cast<T*>(a.dx);
  const int64_t chunks = (a.cols + 7) >> 3;
  float* part = a.ws + blockIdx.x * (chunks * 8);
  const float inv = 1.0f / static_cast<float>(a.cols);
  auto dot8 = [&](const float (&g)[8], const float (&u)[8], const float (&w)[8], float rstd, float dot) {
#pragma unroll
    for (int j = 0; j < 8; ++j) dot = fmaf(g[j] * w[j], u[j] * rstd, dot);
    return dot;
  };
  auto finish8 = [&](float (&g)[8], float (&u)[8], const float (&w)[8], const float (&d)[8], float (&sum)[8], float rstd, float mean, int64_t row, int64_t c, int n) {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float hat = u[j] * rstd;
      sum[j] = fmaf(g[j], hat, sum[j]);
      u[j] = fmaf(rstd, g[j] * w[j] - hat * mean, d[j]);
    }
    store8(dx + row * a.lddx + c * 8, u, n);
  };
  const int64_t step = static_cast<int64_t>(gridDim.x) * ROWS;
  if constexpr (NC != 0) {
    float sum[NC][8] = {};
    for (int64_t row = static_cast<int64_t>(blockIdx.x) * ROWS + (THR == 64 ? threadIdx.x / 64 : 0); row < a.rows; row += step) {
      // as they lie in memory, dh before the reduction too: half the registers,
      // and every load of the row on its way at once
      const float rstd = a.rstd[row];
      Raw8<T> g[NC], u[NC], d[NC];
#pragma unroll
      for (int i = 0; i < NC; ++i) {
        const int64_t c = t + i * thr;
        const int n = clamp8(a.cols - c * 8);
        g[i] = raw8(dy + row * a.lddy + c * 8, n);
        u[i] = raw8(h + row * a.ldh + c * 8, n);
        d[i] = dh != nullptr ? raw8(dh + row * a.lddh + c * 8, n) : Raw8<T>{};
      }
      float dot = 0.0f;
#pragma unroll
      for (int i = 0; i < NC; ++i) {
        const int64_t c = t + i * thr;
        float w[8], gf[8], uf[8];
        load8_any(w, a.weight, c * 8, clamp8(a.cols - c * 8), a.weight_dtype);
        widen8(gf, g[i]);
        widen8(uf, u[i]);
        dot = dot8(gf, uf, w, rstd, dot);
      }
      const float mean = row_sum<THR>(dot, sh) * inv;
#pragma unroll
      for (int i = 0; i < NC; ++i) {
        const int64_t c = t + i * thr;
        const int n = clamp8(a.cols - c * 8);
        float w[8], gf[8], uf[8], df[8];
        load8_any(w, a.weight, c * 8, n, a.weight_dtype);
        widen8(gf, g[i]);
        widen8(uf, u[i]);
        widen8(df, d[i]);
        finish8(gf, uf, w, df, sum[i], rstd, mean, row, c, n);
      }
    }
    if constexpr (ROWS > 1) {
      // the waves' sums, added in their order
      __shared__ float joined[ROWS][8][THR];
#pragma unroll
      for (int i = 0; i < NC; ++i) {
        const int me = threadIdx.x / THR;
#pragma unroll
        for (int j = 0; j < 8; ++j) joined[me][j][t] = sum[i][j];
        __syncthreads();
        for (int e = threadIdx.x; e < 8 * THR; e += 256) {
          const int64_t col = static_cast<int64_t>(i) * THR * 8 + e;
          float s = 0.0f;
#pragma unroll
          for (int q = 0; q < ROWS; ++q) s += joined[q][e & 7][e >> 3];
          if (col < chunks * 8) part[col] = s;
        }
        __syncthreads();
      }
    } else {
#pragma unroll
      for (int i = 0; i < NC; ++i)
        if (t + i * thr < chunks) store8(part + (t + i * thr) * 8, sum[i], 8);
    }
  } else {
    for (int64_t c = t; c < chunks; c += thr)
#pragma unroll
      for (int j = 0; j < 8; ++j) part[c * 8 + j] = 0.0f;
    for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
      const float rstd = a.rstd[row];
      float g[8], u[8], w[8], sum[8], dot = 0.0f;
      auto read = [&](int64_t c, int n) {
        load8(g, dy + row * a.lddy + c * 8, n);
        load8(u, h + row * a.ldh + c * 8, n);
        load8_any(w, a.weight, c * 8, n, a.weight_dtype);
      };
      for (int64_t c = t; c < chunks; c += thr) {
        read(c, clamp8(a.cols - c * 8));
        dot = dot8(g, u, w, rstd, dot);
      }
      const float mean = row_sum<THR>(dot, sh) * inv;
      for (int64_t c = t; c < chunks; c += thr) {
        const int n = clamp8(a.cols - c * 8);
        read(c, n);
        load8(sum, part + c * 8, 8);
        float d[8] = {};
        if (dh != nullptr) load8(d, dh + row * a.lddh + c * 8, n);
        finish8(g, u, w, d, sum, rstd, mean, row, c, n);
        store8(part + c * 8, sum, 8);
      }
    }
  }
}

// dweight[c] = the partial sums of column c, added in fp64: 32 groups of blocks
// in their order, then the groups in theirs
__global__ __launch_bounds__(1024) void norm_dw_kernel(const float* part, int n_parts, int64_t stride, int64_t cols, void* dweight, int dtype) {
  __shared__ double sh[32][33];
  const int c = threadIdx.x & 31, g = threadIdx.x >> 5;
  for (int64_t c0 = static_cast<int64_t>(blockIdx.x) * 32; c0 < cols; c0 += static_cast<int64_t>(gridDim.x) * 32) {
    double s = 0.0;
    if (c0 + c < cols) {
#pragma unroll 8
      for (int p = g; p < n_parts; p += 32) s += static_cast<double>(part[p * stride + c0 + c]);
    }
    sh[g][c] = s;
    __syncthreads();
    if (g == 0 && c0 + c < cols) {
      double total = 0.0;
#pragma unroll
      for (int q = 0; q < 32; ++q) total += sh[q][c];
      store_any(dweight, c0 + c, dtype, static_cast<float>(total));
    }
    __syncthreads();
  }
}

// ---------------------------------------------------------------------------
// Product
// ---------------------------------------------------------------------------

// Two ways to multiply.  The 8-bit matrix instruction runs at twice the rate
// of the 16-bit ones and applies the E8M0 scales itself, but it lines up each
// eight consecutive products on the largest of them and cuts what is below
// 2^-13 of it before the fp32 addition (measured on this card, the same in the
// unscaled instruction): about 1.6e-5 of a result in norm.  That is far below
// a 16-bit result's own rounding (1.7e-3 in bf16, 2e-4 in fp16), so 16-bit
// results take it, at the price of elements whose large products cancel: there
// up to 8 2^-13 of the sizes' sum is lost (448^2 and -448^2, each in a group of
// eight with seven products of 1, leave 0 of the 14).  A caller to whom that
// counts asks for fp32 results.  Those, which also go into the optimizer's
// factors, would lose nine bits.  They convert codes times scale to bf16, which
// holds every such value exactly (4 significant bits; a value below 2^-126,
// subnormal in fp32, may count as zero, and 2^128 is an infinity), and take the
// bf16 instruction, whose sums round as fp32's.

// cbsz / blgp of the f8f6f4 instructions: 0 e4m3, 1 e5m2 (the okls_code values)

// f(integral_constant 0), ..., f(integral_constant N - 1)
template <int N, int I = 0, class F>
__device__ __forceinline__ void for_each(F&& f) {
  if constexpr (I < N) {
    f(std::integral_constant<int, I>{});
    for_each<N, I + 1>(f);
  }
}

__device__ __forceinline__ intx8 frag(const uint8_t* p) {
  const intx4 lo = reinterpret_cast<const intx4*>(p)[0], hi = reinterpret_cast<const intx4*>(p)[1];
  return intx8{lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
}

// codes 8 s .. 8 s + 7 of a lane's, times 2^(byte - 127), in bf16
template <int F, class V>
__device__ __forceinline__ bf16x8 widen(const V& f, int s, int byte) {
  const float scale = __uint_as_float(static_cast<uint32_t>(byte) << 23);
  bf16x8 r;
#pragma unroll
  for (int q = 0; q < 2; ++q) {
    const unsigned w = static_cast<unsigned>(f[2 * s + q]);
    bf16x2 lo, hi;
    if constexpr (F == OKLS_E4M3) {
      lo = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, scale, false);
      hi = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, scale, true);
    } else {
      lo = __builtin_amdgcn_cvt_scalef32_pk_bf16_bf8(w, scale, false);
      hi = __builtin_amdgcn_cvt_scalef32_pk_bf16_bf8(w, scale, true);
    }
    r[4 * q] = lo[0], r[4 * q + 1] = lo[1], r[4 * q + 2] = hi[0], r[4 * q + 3] = hi[1];
  }
  return r;
}

#define INLINE __attribute__((always_inline))
// waits for all but the newest v vector-memory operations, other counters untouched
#define WAIT_VM(v) __builtin_amdgcn_s_waitcnt(((v) & 15) | (7 << 4) | (15 << 8) | (((v) >> 4) << 14))
#define WAIT_LDS() __builtin_amdgcn_s_waitcnt(15 | (7 << 4) | (0 << 8) | (3 << 14))

// c[0 .. 8) = v (+ c), the first n of them
template <typename T>
__device__ __forceinline__ void put8(T* c, float (&v)[8], int n, int accumulate) {
  if (accumulate) {
    float w[8];
    load8(w, c, n);
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] += w[e];
  }
  store8(c, v, n);
}

// A tile of c per workgroup.  The wave's region is GI x GJ blocks of 32 x 32;
// lane r of block row i holds row r GI + i of it, so that a lane's scale bytes
// of all its block rows are neighbours: one read each side per 128 of k.
// Codes and scales come by direct-to-LDS copies, two stages of 128 of k deep, so
// a stage has the whole of the one before to arrive in.
// Bound by the matrix cores at the clock they can hold: 8192 x 8192 x 8192 runs
// at 2.7 PFLOP/s (16-bit results; 72 % of a busy CU's cycles issue products, at
// 1.85 GHz of 2.4), 11008 x 4096 x 16384 in fp32 at 1.35-1.4 (76 %, 1.85 GHz).
// Short k pays each tile's start and its output's burst: 8191 x 5632 x 2048 runs
// at 2.1 (54 %), 176 tiles (5632 x 2048 x 8192 in fp32) leave 80 of 256 CUs
// idle, 1.0-1.15.  LDS bank conflicts are counted in one place only: 1024 cycles a
// big tile, at any k, where its 16-bit results are staged on their way out.
// A loop over tiles that let a tile's stores drain behind the next one's
// products measured the same and cost the registers of the loop.
template <int WM_, int WN_, int GI_, int GJ_>
struct Tile {
  static constexpr int WM = WM_, WN = WN_, GI = GI_, GJ = GJ_;
  static constexpr int NW = WM * WN, NT = NW * 64, RM = 32 * GI, RN = 32 * GJ, BM = WM * RM, BN = WN * RN;
  static constexpr int LA = BM / 8 / NW, LB = BN / 8 / NW;   // 1 KB copies per wave and stage
};
using TileBig = Tile<2, 4, 4, 2>;     // 256 x 256, 8 waves
using TileSmall = Tile<2, 2, 2, 2>;   // 128 x 128, 4 waves, two workgroups a CU
using TileNarrow = Tile<1, 2, 2, 2>;  // 64 x 128, 2 waves, three workgroups a CU

struct MatmulPlan {
  int tile;        // 0 none (the few-rows kernel), 1 narrow, 2 small, 3 big
  int splits;      // of the summed axis
  int tm, tn;      // tiles
};

template <int N> struct ScaleWord { using type = uint32_t; };
template <> struct ScaleWord<2> { using type = uint16_t; };

template <class C, int FA, int FB, bool F32>
__global__ __launch_bounds__(C::NT, 2) void matmul_tile_kernel(MatmulArgs a, MatmulPlan plan) {
  constexpr int GI = C::GI, GJ = C::GJ;
  constexpr int P = F32 ? 4 : 2;          // parts of a stage of 128 of k
  constexpr int FW = 16 / P;              // dwords of a lane's codes in a block row and part
  constexpr int H = GI / 2;               // block rows of a phase: a phase is half of a's block rows in one part
  __shared__ __attribute__((aligned(16))) uint8_t sA0[C::BM * 128], sA1[C::BM * 128], sB0[C::BN * 128], sB1[C::BN * 128];
  __shared__ __attribute__((aligned(16))) uint8_t e0[512], e1[512];   // scale bytes of the tile's rows, a's and from 256 on b's
  static_assert(C::BM <= 256 && C::BN <= 256, "one copy holds a side's scales");
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = wave / C::WN, wn = wave % C::WN;
  const int64_t m = a.a.rows, n = a.b.rows;

  // Workgroup w runs on XCD w % 8.  Each XCD takes a run of neighbouring tiles
  // in bands of 8 tile rows, so that the 32 or 64 it holds at a time share
  // operand rows in its L2.
  auto uniform = [](int v) { return __builtin_amdgcn_readfirstlane(v); };
  const unsigned per = plan.tm * plan.tn, total = per * plan.splits, w = blockIdx.x, x = w & 7;
  const unsigned id = x * (total >> 3) + (x < (total & 7) ? x : (total & 7)) + (w >> 3);
  const unsigned split = uniform(id / per), t = id - split * per;
  const unsigned band = uniform(t / (8u * plan.tn)), in = t - band * 8u * plan.tn;
  const unsigned high = plan.tm - band * 8 < 8 ? plan.tm - band * 8 : 8, column = uniform(in / high);
  const int64_t m0 = static_cast<int64_t>(band * 8 + in - column * high) * C::BM, n0 = static_cast<int64_t>(column) * C::BN;
  const unsigned blocks = static_cast<unsigned>((a.a.cols + 127) >> 7);
  const int k0 = uniform(blocks * split / plan.splits), nst = uniform(blocks * (split + 1) / plan.splits) - k0;

  // Copies: 8 rows of 128 bytes each.  LDS row 32 i + r of a wave's region
  // holds its row r GI + i, and 16-byte chunk c of it lies at position
  // c ^ (r / 2 % 8): 16 lanes that read one chunk of 16 consecutive r cover
  // all 64 banks.  Rows past the end read the last one; what they give is not
  // stored.
  // A side's tile spans less than 2^32 bytes (the launcher's rule), so a lane
  // keeps 32-bit offsets from a base that the whole wave shares.
  // Scale bytes: one dword a lane, even waves those of a and odd ones those of b
  // (rows padded to 16 exist; entries past them are another row's).
  const bool of_b = wave & 1;
  const int64_t ld_scale = of_b ? a.b.ld_scale : a.a.ld_scale;
  const uint8_t *baseA = a.a.codes + m0 * a.a.ld + k0 * int64_t(128), *baseB = a.b.codes + n0 * a.b.ld + k0 * int64_t(128);
  const uint8_t* baseS = (of_b ? a.b.scales + n0 : a.a.scales + m0) + k0 * ld_scale;
  uint32_t ga[C::LA], gb[C::LB];
#pragma unroll
  for (int q = 0; q < C::LA; ++q) {
    const int at = 8 * (wave + C::NW * q) + (lane >> 3), row = at / C::RM * C::RM + (at & 31) * GI + at % C::RM / 32;
    const int64_t r = m0 + row < m ? row : m - 1 - m0;
    ga[q] = static_cast<uint32_t>(r * a.a.ld) + (((lane & 7) ^ (at >> 1 & 7)) << 4);
  }
#pragma unroll
  for (int q = 0; q < C::LB; ++q) {
    const int at = 8 * (wave + C::NW * q) + (lane >> 3), row = at / C::RN * C::RN + (at & 31) * GJ + at % C::RN / 32;
    const int64_t r = n0 + row < n ? row : n - 1 - n0;
    gb[q] = static_cast<uint32_t>(r * a.b.ld) + (((lane & 7) ^ (at >> 1 & 7)) << 4);
  }
  const int64_t last = of_b ? ((n + 15) & ~int64_t(15)) - 4 - n0 : ((m + 15) & ~int64_t(15)) - 4 - m0;
  uint32_t gs = static_cast<uint32_t>(4 * lane < last ? 4 * lane : last);
  int copied = 0;
  auto copy = [&](uint8_t* dA, uint8_t* dB, uint8_t* e) INLINE {
    // opaque here, so that each stays one 32-bit register next to the uniform base
#pragma unroll
    for (int q = 0; q < C::LA; ++q) asm("" : "+v"(ga[q]));
#pragma unroll
    for (int q = 0; q < C::LB; ++q) asm("" : "+v"(gb[q]));
    asm("" : "+v"(gs));
#pragma unroll
    for (int q = 0; q < C::LA; ++q)
      __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) void*)(baseA + ga[q]),
                                       (__attribute__((address_space(3))) void*)(dA + (wave + C::NW * q) * 1024), 16, 0, 0);
#pragma unroll
    for (int q = 0; q < C::LB; ++q)
      __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) void*)(baseB + gb[q]),
                                       (__attribute__((address_space(3))) void*)(dB + (wave + C::NW * q) * 1024), 16, 0, 0);
    // every wave issues it, several to the same place with the same bytes: no branch between the products
    __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) void*)(baseS + gs),
                                     (__attribute__((address_space(3))) void*)(e + (of_b ? 256 : 0)), 4, 0, 0);
    // past the end the last stage again, into a buffer that nothing reads: no branch between the products
    const int64_t on = ++copied < nst ? 1 : 0;
    baseA += on * 128, baseB += on * 128, baseS += on * ld_scale;
  };
  const int r32 = lane & 31, half = lane >> 5;
  using WA = typename ScaleWord<GI>::type;
  using WB = typename ScaleWord<GJ>::type;

  typedef int codes_t __attribute__((ext_vector_type(FW)));
  codes_t fa[2][H], fb[2][GJ];            // codes of two phases, of two parts
  const int rowA = (wm * C::RM + r32) * 128, rowB = (wn * C::RN + r32) * 128, sw = r32 >> 1 & 7;
  int sa, sb, sa_next, sb_next;           // scale bytes of this lane's block rows
  // the codes of phase u; b's with a part's first
  auto fetch = [&](auto uc, const uint8_t* dA, const uint8_t* dB, const uint8_t* e) INLINE {
    constexpr int u = decltype(uc)::value, f = u / 2, g = u & 1;
    auto at = [&](const uint8_t* row) INLINE {
      if constexpr (FW == 4) {
        return *reinterpret_cast<const intx4*>(row + (((2 * f + half) ^ sw) << 4));
      } else {
        const intx4 lo = *reinterpret_cast<const intx4*>(row + (((4 * f + 2 * half) ^ sw) << 4));
        const intx4 hi = *reinterpret_cast<const intx4*>(row + (((4 * f + 2 * half + 1) ^ sw) << 4));
        return __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
      }
    };
    if constexpr (g == 0)
#pragma unroll
      for (int j = 0; j < GJ; ++j) fb[f & 1][j] = at(dB + rowB + j * 4096);
#pragma unroll
    for (int i = 0; i < H; ++i) fa[g][i] = at(dA + rowA + (g * H + i) * 4096);
    if constexpr (u == 0) {
      sa_next = *reinterpret_cast<const WA*>(e + wm * C::RM + r32 * GI);
      sb_next = *reinterpret_cast<const WB*>(e + 256 + wn * C::RN + r32 * GJ);
    }
  };

  floatx16 acc[GI][GJ];

  auto multiply = [&](auto uc) INLINE {
    constexpr int f = decltype(uc)::value / 2, g = decltype(uc)::value & 1;
    if constexpr (F32) {
#pragma unroll
      for (int s = 0; s < 2; ++s) {
        bf16x8 wa[H], wb[GJ];
#pragma unroll
        for (int j = 0; j < GJ; ++j) wb[j] = widen<FB>(fb[f & 1][j], s, (sb >> (8 * j)) & 255);
#pragma unroll
        for (int i = 0; i < H; ++i) wa[i] = widen<FA>(fa[g][i], s, (sa >> (8 * (g * H + i))) & 255);
#pragma unroll
        for (int i = 0; i < H; ++i)
#pragma unroll
          for (int j = 0; j < GJ; ++j)
            acc[g * H + i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(wb[j], wa[i], acc[g * H + i][j], 0, 0, 0);
      }
    } else {
      for_each<H>([&](auto ic) INLINE {
        for_each<GJ>([&](auto jc) INLINE {
          constexpr int i = decltype(ic)::value, j = decltype(jc)::value, at = g * H + i;
          acc[at][j] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(fb[f & 1][j], fa[g][i], acc[at][j], FB, FA, j, sb, at, sa);
        });
      });
    }
  };
  auto barrier = [&]() INLINE {
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
  };

  // A phase's products run while the next phase's codes come out of LDS.
  // Before the last phase of a stage every wave has taken that stage's last
  // codes, so the barrier there frees its buffer for the stage after next,
  // and the wait before it has this wave's part of the next stage in LDS.
  auto stage = [&](auto bc) INLINE {
    constexpr int b = decltype(bc)::value;
    uint8_t *hereA = b ? sA1 : sA0, *hereB = b ? sB1 : sB0, *nextA = b ? sA0 : sA1, *nextB = b ? sB0 : sB1;
    uint8_t *hereE = b ? e1 : e0, *nextE = b ? e0 : e1;
    sa = sa_next, sb = sb_next;
    for_each<2 * P>([&](auto uc) INLINE {
      constexpr int u = decltype(uc)::value;
      constexpr bool final = u == 2 * P - 1;
      if constexpr (!final) {
        fetch(std::integral_constant<int, u + 1>{}, hereA, hereB, hereE);
      } else {
        asm volatile("" ::: "memory");
        WAIT_LDS();
        WAIT_VM(0);
        barrier();
        copy(hereA, hereB, hereE);
        fetch(std::integral_constant<int, 0>{}, nextA, nextB, nextE);
      }
      multiply(uc);
      if constexpr (!F32) {
        // one product, then its share of the reads and copies
#pragma unroll
        for (int q = 0; q < H * GJ; ++q) {
          constexpr int n = H * GJ, reads = 2 * (H + (u & 1 ? GJ : 0) + final), copies = final ? C::LA + C::LB + 1 : 0;
          __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
          __builtin_amdgcn_sched_group_barrier(0x100, (reads + n - 1) / n, 0);
          __builtin_amdgcn_sched_group_barrier(0x020, (copies + n - 1) / n, 0);
        }
      }
      __builtin_amdgcn_sched_barrier(0);
    });
  };

  MatmulArgs o = a;
  const int64_t np = (n + 7) & ~int64_t(7);
  if (plan.splits > 1) {     // partial sums: (split, m, n up to a multiple of 8) in fp32
    o.ldc = np;
    o.c_dtype = OKLS_F32;
    o.accumulate = 0;
  }
  // lane l: row l % 32 of each block row, columns 8 q + 4 (l / 32) + 0..3 of
  // each block column, which lie GJ apart: 8 neighbours of a row
  static_assert(GJ == 2, "a lane's neighbours are one 16-byte store of a 16-bit result");
  auto finish = [&]() INLINE {
    if (plan.splits > 1) o.c = a.ws + split * m * np;
    const int64_t r0 = m0 + wm * C::RM, c0 = n0 + wn * C::RN;
    const bool inside = c0 + C::RN <= n;
    constexpr int S = C::RM * C::RN * 2, inB = C::BN * 128 / S;      // bytes of a wave's part; waves a buffer of b holds
    static_assert(C::NW < 8 || (4 * inB >= C::NW && C::BM == C::BN), "the buffers hold every wave's part");
    uint8_t* mine = (wave < inB ? sB0 : wave < 2 * inB ? sB1 : wave < 3 * inB ? sA0 : sA1) + wave % inB * S;
    auto rows = [&](auto* c) INLINE {
      auto* at = c + (r0 + r32 * GI) * o.ldc + c0 + 8 * half;
#pragma unroll
      for (int i = 0; i < GI; ++i) {
        if (r0 + r32 * GI + i >= m) continue;
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          float v[8];
#pragma unroll
          for (int e = 0; e < 4; ++e)
#pragma unroll
            for (int j = 0; j < GJ; ++j) v[e * GJ + j] = acc[i][j][4 * q + e];
          const int left = inside ? 8 : clamp8(n - c0 - 16 * q - 8 * half);
          put8(at + i * o.ldc + 16 * q, v, left, o.accumulate);
        }
      }
    };
    // Through LDS, so that rows leave as whole lines: straight from the lanes a
    // store would touch 32 rows.  Row 32 i + r of the wave's part of the buffers
    // holds row r GI + i (fp32: half of them at a time), its 16-byte chunks
    // spread over the banks as the codes were.
    auto staged = [&](auto* c) INLINE {
      using T = std::remove_pointer_t<decltype(c)>;
      constexpr int E = 16 / sizeof(T), CH = C::RN / E, PASSES = sizeof(T) == 4 ? 2 : 1, IP = GI / PASSES, LOG = CH == 8 ? 1 : 0;
#pragma unroll
      for (int pass = 0; pass < PASSES; ++pass) {
#pragma unroll
        for (int i = 0; i < IP; ++i)
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            __attribute__((aligned(16))) T v[8];
#pragma unroll
            for (int e = 0; e < 4; ++e)
#pragma unroll
              for (int j = 0; j < GJ; ++j) v[e * GJ + j] = from_f32<T>(acc[pass * IP + i][j][4 * q + e]);
#pragma unroll
            for (int u = 0; u < 8 / E; ++u) {
              const int chunk = ((16 * q + 8 * half) / E + u) ^ (r32 >> LOG & (CH - 1));
              *reinterpret_cast<intx4*>(mine + ((i * 32 + r32) * CH + chunk) * 16) = *reinterpret_cast<const intx4*>(&v[u * E]);
            }
          }
        WAIT_LDS();
        asm volatile("" ::: "memory");
#pragma unroll 4
        for (int t = 0; t < IP * 32 * CH / 64; ++t) {
          const int at = t * 64 + lane, row = at / CH, r = row & 31;
          const int64_t m_at = r0 + r * GI + pass * IP + (row >> 5), n_at = c0 + (at % CH ^ (r >> LOG & (CH - 1))) * E;
          const intx4 x = *reinterpret_cast<const intx4*>(mine + at * 16);
          if (m_at >= m || n_at >= n) continue;
          T* to = c + m_at * o.ldc + n_at;
          if (n_at + E <= n) {
            // past the caches, which the next workgroups' operands fill
            if constexpr (sizeof(T) == 4) __builtin_nontemporal_store(__builtin_bit_cast(floatx4, x), reinterpret_cast<floatx4_any*>(to));
            else __builtin_nontemporal_store(__builtin_bit_cast(u16x8, x), reinterpret_cast<u16x8_any*>(to));
          } else {
            __attribute__((aligned(16))) T v[E];
            *reinterpret_cast<intx4*>(v) = x;
#pragma unroll
            for (int e = 0; e < E; ++e)
              if (n_at + e < n) to[e] = v[e];
          }
        }
        WAIT_LDS();
        asm volatile("" ::: "memory");
      }
    };
    // the small tiles' few rows gain nothing by it (48 x 5120 x 13824 20.7 us
    // straight, 21.3 staged; 8191 x 5632 x 2048 in big tiles 110 and 92)
    auto write = [&](auto* c) INLINE {
      if constexpr (C::NW < 8) {
        rows(c);
      } else {
        if (o.accumulate) rows(c);
        else staged(c);
      }
    };
    if (F32 || o.c_dtype == OKLS_F32) write(static_cast<float*>(o.c));
    else if (o.c_dtype == OKLS_BF16) write(static_cast<bf16_t*>(o.c));
    else write(static_cast<half_t*>(o.c));
  };

  using I0 = std::integral_constant<int, 0>;
  using I1 = std::integral_constant<int, 1>;
  copy(sA0, sB0, e0);
  copy(sA1, sB1, e1);
#pragma unroll
  for (int i = 0; i < GI; ++i)
#pragma unroll
    for (int j = 0; j < GJ; ++j) acc[i][j] = floatx16{};
  WAIT_VM(C::LA + C::LB + 1);
  barrier();
  fetch(I0{}, sA0, sB0, e0);
  for (int st = 0; st < nst; st += 2) {
    stage(I0{});
    if (st + 1 < nst) stage(I1{});
  }
  WAIT_VM(0);              // the last copies land before the buffers are used again or given up
  if constexpr (C::NW == 8) barrier();
  finish();
}

// c = the partial sums of each element, added in the splits' order
__global__ __launch_bounds__(256) void matmul_join_kernel(MatmulArgs a, int splits) {
  const int64_t m = a.a.rows, n = a.b.rows, np = (n + 7) & ~int64_t(7);
  for (int64_t i = (blockIdx.x * 256ll + threadIdx.x) * 8; i < m * np; i += gridDim.x * 2048ll) {
    float v[8], u[8];
    load8(v, a.ws + i, 8);
    for (int s = 1; s < splits; ++s) {
      load8(u, a.ws + s * m * np + i, 8);
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] += u[e];
    }
    const int64_t row = i / np, col = i - row * np, at = row * a.ldc + col;
    const int left = clamp8(n - col);
    if (a.c_dtype == OKLS_F32) put8(static_cast<float*>(a.c) + at, v, left, a.accumulate);
    else if (a.c_dtype == OKLS_BF16) put8(static_cast<bf16_t*>(a.c) + at, v, left, a.accumulate);
    else put8(static_cast<half_t*>(a.c) + at, v, left, a.accumulate);
  }
}

// Bound by memory: one row through 11008 x 4096 (45 MB) takes 11.4 us, 4.0 TB/s
// with the launch in it.
// Few rows of a (16 TM of them a workgroup): c's columns in groups of 16 TN a workgroup,
// whose waves split the summed axis in turn and add up through LDS.  Every code
// of b is read once and straight into registers, U blocks of 128 a wave at a time.
constexpr int kFewWaves = 8;
template <int TM, int TN, int FA, int FB, bool F32>
__global__ __launch_bounds__(kFewWaves * 64) void matmul_few_kernel(MatmulArgs a) {
  constexpr int U = TM + TN <= 3 ? 4 : 2;        // blocks of k a wave has in flight
  __shared__ floatx4 part[kFewWaves][TM * TN][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t m = a.a.rows, n = a.b.rows, blocks = (a.a.cols + 127) >> 7;
  const int64_t n0 = static_cast<int64_t>(blockIdx.x) * (16 * TN), m0 = static_cast<int64_t>(blockIdx.y) * (16 * TM);
  int64_t ra[TM], rb[TN];
  const uint8_t *pa[TM], *pb[TN];
  // rows past the end read the last one; what they give is not stored
#pragma unroll
  for (int i = 0; i < TM; ++i) {
    const int64_t r = m0 + 16 * i + (lane & 15);
    ra[i] = r < m ? r : m - 1;
    pa[i] = a.a.codes + ra[i] * a.a.ld + (lane >> 4) * 32;
  }
#pragma unroll
  for (int j = 0; j < TN; ++j) {
    const int64_t r = n0 + 16 * j + (lane & 15);
    rb[j] = r < n ? r : n - 1;
    pb[j] = a.b.codes + rb[j] * a.b.ld + (lane >> 4) * 32;
  }
  floatx4 acc[TM][TN];
#pragma unroll
  for (int i = 0; i < TM; ++i)
#pragma unroll
    for (int j = 0; j < TN; ++j) acc[i][j] = floatx4{};
  auto run = [&](int64_t k, auto uc) {
    constexpr int nu = decltype(uc)::value;
    intx8 fa[nu][TM], fb[nu][TN];
    int sa[nu][TM], sb[nu][TN];
#pragma unroll
    for (int u = 0; u < nu; ++u) {
      const int64_t kb = k + u * kFewWaves;
#pragma unroll
      for (int j = 0; j < TN; ++j) {
        fb[u][j] = frag(pb[j] + kb * 128);
        sb[u][j] = a.b.scales[kb * a.b.ld_scale + rb[j]];
      }
#pragma unroll
      for (int i = 0; i < TM; ++i) {
        fa[u][i] = frag(pa[i] + kb * 128);
        sa[u][i] = a.a.scales[kb * a.a.ld_scale + ra[i]];
      }
    }
#pragma unroll
    for (int u = 0; u < nu; ++u) {
      if constexpr (F32) {
#pragma unroll
        for (int s = 0; s < 4; ++s) {
          bf16x8 wb[TN];
#pragma unroll
          for (int j = 0; j < TN; ++j) wb[j] = widen<FB>(fb[u][j], s, sb[u][j]);
#pragma unroll
          for (int i = 0; i < TM; ++i) {
            const bf16x8 wa = widen<FA>(fa[u][i], s, sa[u][i]);
#pragma unroll
            for (int j = 0; j < TN; ++j) acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(wb[j], wa, acc[i][j], 0, 0, 0);
          }
        }
      } else {
#pragma unroll
        for (int i = 0; i < TM; ++i)
#pragma unroll
          for (int j = 0; j < TN; ++j)
            acc[i][j] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(fb[u][j], fa[u][i], acc[i][j], FB, FA, 0, sb[u][j], 0, sa[u][i]);
      }
    }
  };
  int64_t k = wave;
  for (; k + (U - 1) * kFewWaves < blocks; k += U * kFewWaves) run(k, std::integral_constant<int, U>{});
  for (; k < blocks; k += kFewWaves) run(k, std::integral_constant<int, 1>{});
#pragma unroll
  for (int i = 0; i < TM; ++i)
#pragma unroll
    for (int j = 0; j < TN; ++j) part[wave][i * TN + j][lane] = acc[i][j];
  __syncthreads();
  // lane l of a block holds c[l % 16][4 (l / 16) + e]
  for (int t = threadIdx.x; t < TM * TN * 64; t += kFewWaves * 64) {
    const int blk = t >> 6, l = t & 63;
    floatx4 s = part[0][blk][l];
#pragma unroll
    for (int q = 1; q < kFewWaves; ++q) s += part[q][blk][l];
    const int64_t row = m0 + blk / TN * 16 + (l & 15), col = n0 + blk % TN * 16 + (l >> 4) * 4;
    if (row >= m) continue;
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (col + e < n) {
        const int64_t at = row * a.ldc + col + e;
        store_any(a.c, at, a.c_dtype, a.accumulate ? s[e] + load_any(a.c, at, a.c_dtype) : s[e]);
      }
  }
}

__global__ __launch_bounds__(256) void zero_kernel(void* c, int dtype, int64_t m, int64_t n, int64_t ldc) {
  for (int64_t i = blockIdx.x * 256ll + threadIdx.x; i < m * n; i += gridDim.x * 256ll) store_any(c, i / n * ldc + i % n, dtype, 0.0f);
}

// calls go(a's format, b's format, fp32 result) with compile-time values
template <class F>
void by_format(const MatmulArgs& a, F go) {
  using I0 = std::integral_constant<int, 0>;
  using I1 = std::integral_constant<int, 1>;
  auto second = [&](auto fa) {
    auto third = [&](auto fb) {
      if (a.c_dtype == OKLS_F32) go(fa, fb, std::true_type{});
      else go(fa, fb, std::false_type{});
    };
    if (a.b.format == OKLS_E4M3) third(I0{});
    else third(I1{});
  };
  if (a.a.format == OKLS_E4M3) second(I0{});
  else second(I1{});
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

hipError_t launch_quantize(const QuantArgs& a, hipStream_t s) {
  const int64_t tiles = ((a.rows + 127) / 128) * ((a.cols + 127) / 128);
  const int grid = blocks_up_to(tiles, 1 << 20);
  // the two outputs may differ in format only by two launches
  auto go = [&](const QuantArgs& q, int fmt) {
    by_type(q.x_dtype, [&](auto type) {
      using T = decltype(type);
      if (q.row_factor != nullptr) {
        if (fmt == OKLS_E4M3) quantize_kernel<T, OKLS_E4M3, true><<<grid, 256, 0, s>>>(q);
        else quantize_kernel<T, OKLS_E5M2, true><<<grid, 256, 0, s>>>(q);
      } else {
        if (fmt == OKLS_E4M3) quantize_kernel<T, OKLS_E4M3, false><<<grid, 256, 0, s>>>(q);
        else quantize_kernel<T, OKLS_E5M2, false><<<grid, 256, 0, s>>>(q);
      }
    });
  };
  if (a.along_cols.codes != nullptr && a.along_rows.codes != nullptr && a.along_cols.format != a.along_rows.format) {
    QuantArgs one = a, two = a;
    one.along_rows = Blocked{};
    two.along_cols = Blocked{};
    go(one, a.along_cols.format);
    go(two, a.along_rows.format);
  } else {
    go(a, a.along_cols.codes != nullptr ? a.along_cols.format : a.along_rows.format);
  }
  return hipGetLastError();
}

// calls go(most threads of a row, chunks of 8 a thread holds, threads of a
// workgroup).  At most two chunks: more cost the waves that hide the loads (the
// gradient of 16384 x 2048 takes 63 us with a wave a row, 56 with a workgroup;
// of 4000 x 16000 176 us with 256 threads of eight chunks, 110 with 1024 of two).
template <class F>
static void by_width(int64_t cols, F go) {
  using I0 = std::integral_constant<int, 0>;
  using I1 = std::integral_constant<int, 1>;
  using I2 = std::integral_constant<int, 2>;
  const int64_t waves = (cols + 511) / 512;        // of one chunk a lane
  const int one = static_cast<int>(waves) * 64, two = static_cast<int>((waves + 1) / 2) * 64;
  if (cols <= 512) go(std::integral_constant<int, 64>{}, I1{}, 256);
  else if (cols <= 1024) go(std::integral_constant<int, 64>{}, I2{}, 256);
  else if (cols <= 2048) go(std::integral_constant<int, 256>{}, I1{}, one);
  else if (cols <= 8192) go(std::integral_constant<int, 512>{}, I2{}, two);
  else if (cols <= 16384) go(std::integral_constant<int, 1024>{}, I2{}, two);
  else go(std::integral_constant<int, 1024>{}, I0{}, 1024);
}

hipError_t launch_rms_norm(const NormArgs& a, hipStream_t s) {
  by_type(a.dtype, [&](auto type) {
    by_width(a.cols, [&](auto thr, auto nc, int threads) {
      using T = decltype(type);
      constexpr int THR = decltype(thr)::value, NC = decltype(nc)::value;
      constexpr int rows = THR == 64 ? 4 : 1;
      const int grid = blocks_up_to((a.rows + rows - 1) / rows, 1 << 20);
      if (a.out.format == OKLS_E4M3) rms_norm_kernel<T, OKLS_E4M3, THR, NC><<<grid, threads, 0, s>>>(a);
      else rms_norm_kernel<T, OKLS_E5M2, THR, NC><<<grid, threads, 0, s>>>(a);
    });
  });
  return hipGetLastError();
}

// Workgroups of the gradient: each leaves a row of partial sums to write and
// read again, so at least two of the matrix's rows go to each, and more to the
// larger workgroups, of which fewer fill the card.
static int grad_blocks(int64_t rows, int64_t cols) {
  const int64_t each = cols <= 1024 ? 8 : 2;
  return blocks_up_to((rows + each - 1) / each, cols <= 4096 ? kGradBlocks : cols <= 8192 ? kGradBlocks / 2 : kGradBlocks / 4);
}

size_t norm_grad_workspace(int64_t rows, int64_t cols) {
  return static_cast<size_t>(grad_blocks(rows, cols)) * ((cols + 7) / 8 * 8) * 4;
}

hipError_t launch_rms_norm_backward(const NormGradArgs& a, hipStream_t s) {
  const int grid = grad_blocks(a.rows, a.cols);
  if (grid > 0) {
    by_type(a.dtype, [&](auto type) {
      by_width(a.cols, [&](auto thr, auto nc, int threads) {
        norm_grad_kernel<decltype(type), decltype(thr)::value, decltype(nc)::value><<<grid, threads, 0, s>>>(a);
      });
    });
  }
  norm_dw_kernel<<<blocks_up_to((a.cols + 31) / 32, 1 << 16), 1024, 0, s>>>(a.ws, grid, (a.cols + 7) / 8 * 8, a.cols, a.dweight, a.weight_dtype);
  return hipGetLastError();
}

// Which kernel, and into how many parts the summed axis is cut.  Measured here
// (us, 16-bit results unless fp32 is said, m x n x k):
//  - up to 16 rows straight from memory: 16 x 11008 x 4096 13.9, narrow tiles
//    15.5; more rows read a too often that way (64 x 11008 x 4096: 27.9 against
//    17.6), except where the whole weight takes no time (17 x 1024 x 1024: 3.3
//    against 6.4).
//  - the largest tile that still gives most of the 256 CUs one: 2048 x 5632 x
//    2048 is 176 big tiles, 29.8 (small 32.4); 2048 x 2048 x 2048 only 64,
//    26.9 (small 16.1); 256 x 5632 x 2048 88 small ones, 14.7 (narrow 13.2).
//    But no 256 x 256 one for at most 128 rows or columns: at least half of
//    it would lie past the end (us, big and small tiles): 48 x 50257 x 4096
//    46 and 34, fp32 83 and 54; 128 x 128256 x 4096 140 and 139, fp32 212 and
//    156; 50257 x 64 x 2048 30 and 22, fp32 51 and 33; 131072 x 128 x 2048 67
//    and 63, fp32 113 and 84.  Up to 64 rows narrow tiles would gain at some
//    sizes and lose at others: 17 x 50257 x 4096 32.4 (small 33.7), fp32 51
//    (61); 48 x 128256 x 4096 139 (122), fp32 149 (139).
//  - narrow tiles too few for the card split the sum, to about 384 workgroups,
//    where that pays: a stage of 128 takes about 0.6 us, a split sum 3 us more
//    and its partial sums' way at 5 TB/s.  48 x 5120 x 13824: 65.5 whole, 20.5
//    in 6; 256 x 5632 x 2048: 13.2 whole, 19.1 in 2.
static MatmulPlan matmul_plan(int64_t m, int64_t n, int64_t k) {
  MatmulPlan p{};
  p.splits = 1;
  if (m <= 16 || (m <= 64 && n * k <= (1 << 23))) return p;
  auto tiles = [&](int tile, int bm, int bn) {
    p.tile = tile, p.tm = static_cast<int>((m + bm - 1) / bm), p.tn = static_cast<int>((n + bn - 1) / bn);
    return static_cast<int64_t>(p.tm) * p.tn;
  };
  if (m > 128 && n > 128 && tiles(3, TileBig::BM, TileBig::BN) >= 160) return p;
  if (tiles(2, TileSmall::BM, TileSmall::BN) >= 160) return p;
  const int64_t t = tiles(1, TileNarrow::BM, TileNarrow::BN), blocks = (k + 127) / 128;
  int64_t s = (384 + t / 2) / t;
  if (s > 12) s = 12;
  if (s > blocks / 4) s = blocks / 4;
  if (s > 1 && 0.6 * static_cast<double>(blocks - blocks / s) > 3.0 + static_cast<double>(m) * n * s * 8 / 5e6) p.splits = static_cast<int>(s);
  return p;
}

size_t matmul_workspace(int64_t m, int64_t n, int64_t k) {
  if (m == 0 || n == 0 || k == 0) return 0;
  const MatmulPlan p = matmul_plan(m, n, k);
  return p.splits <= 1 ? 0 : static_cast<size_t>(p.splits) * m * ((n + 7) / 8 * 8) * 4;
}

hipError_t launch_matmul(const MatmulArgs& a, hipStream_t s) {
  const int64_t m = a.a.rows, n = a.b.rows, k = a.a.cols;
  if (k == 0) {
    if (!a.accumulate) zero_kernel<<<blocks_up_to((m * n + 255) / 256, 4096), 256, 0, s>>>(a.c, a.c_dtype, m, n, a.ldc);
    return hipGetLastError();
  }
  const MatmulPlan p = matmul_plan(m, n, k);
  // rows of codes 2^24 bytes apart leave no tile's side inside 2^32 bytes
  if (p.tile == 0 || a.a.ld >= (1 << 24) || a.b.ld >= (1 << 24)) {
    by_format(a, [&](auto fa, auto fb, auto f32) {
      constexpr int FA = decltype(fa)::value, FB = decltype(fb)::value;
      constexpr bool F32 = decltype(f32)::value;
      // parts of at most 2^21 x 2^24: a launch holds fewer than 2^32 threads and 2^16 workgroups along y
      for (int64_t m0 = 0; m0 < m; m0 += 1 << 21)
        for (int64_t n0 = 0; n0 < n; n0 += 1 << 24) {
          MatmulArgs p = a;
          p.a.codes += m0 * a.a.ld, p.a.scales += m0, p.a.rows = m - m0 < (1 << 21) ? m - m0 : 1 << 21;
          p.b.codes += n0 * a.b.ld, p.b.scales += n0, p.b.rows = n - n0 < (1 << 24) ? n - n0 : 1 << 24;
          p.c = static_cast<uint8_t*>(a.c) + (m0 * a.ldc + n0) * (F32 ? 4 : 2);
          const unsigned one = static_cast<unsigned>((p.b.rows + 15) / 16), two = static_cast<unsigned>((p.b.rows + 31) / 32);
          if (m <= 16) matmul_few_kernel<1, 1, FA, FB, F32><<<one, kFewWaves * 64, 0, s>>>(p);
          else if (m <= 32) matmul_few_kernel<2, 1, FA, FB, F32><<<one, kFewWaves * 64, 0, s>>>(p);
          else matmul_few_kernel<4, 2, FA, FB, F32><<<dim3(two, static_cast<unsigned>((p.a.rows + 63) / 64)), kFewWaves * 64, 0, s>>>(p);
        }
    });
    return hipGetLastError();
  }
  const unsigned tiles = static_cast<unsigned>(p.tm * p.tn * p.splits);
  by_format(a, [&](auto fa, auto fb, auto f32) {
    constexpr int FA = decltype(fa)::value, FB = decltype(fb)::value;
    constexpr bool F32 = decltype(f32)::value;
    if (p.tile == 3) matmul_tile_kernel<TileBig, FA, FB, F32><<<tiles, TileBig::NT, 0, s>>>(a, p);
    else if (p.tile == 2) matmul_tile_kernel<TileSmall, FA, FB, F32><<<tiles, TileSmall::NT, 0, s>>>(a, p);
    else matmul_tile_kernel<TileNarrow, FA, FB, F32><<<tiles, TileNarrow::NT, 0, s>>>(a, p);
  });
  if (p.splits > 1) matmul_join_kernel<<<blocks_up_to((m * ((n + 7) / 8) + 255) / 256, 2048), 256, 0, s>>>(a, p.splits);
  return hipGetLastError();
}

}  // namespace okls
