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
#include "device_common.h"
#include "linear_kernels.h"
#include "product_tile.h"

namespace okls {
namespace {

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

//
// Where the values come from: x as it is, with its two factors, or in the sorted
// order of experts' rows, zeros in rows without a choice.  Workgroups along y take
// a stack's matrices.
enum Source { kAsIs, kFactors, kSorted };
typedef intx4 intx4_any __attribute__((aligned(4)));

template <typename T, int FMT, int SOURCE>
__global__ __launch_bounds__(256, SOURCE == kFactors ? 3 : 4) void quantize_kernel(QuantArgs a) {
  constexpr bool FACTORS = SOURCE == kFactors;
  __shared__ uint32_t col_top[4][128];
  __shared__ __attribute__((aligned(16))) uint8_t tile[128 * kTileStride];
  const int t = threadIdx.x, c8 = t & 15, rg = t >> 4, wave = t >> 6;
  const int64_t tiles_c = (a.cols + 127) >> 7, n_tiles = tiles_c * ((a.rows + 127) >> 7);
  const T* x = static_cast<const T*>(a.x) + blockIdx.y * a.stride;
  if (gridDim.y > 1) {
    const int64_t first_c = blockIdx.y * ((a.rows + 15) & ~int64_t(15)), first_r = blockIdx.y * ((a.cols + 15) & ~int64_t(15));
    if (a.along_cols.codes != nullptr) a.along_cols.codes += first_c * a.along_cols.ld, a.along_cols.scales += first_c;
    if (a.along_rows.codes != nullptr) a.along_rows.codes += first_r * a.along_rows.ld, a.along_rows.scales += first_r;
  }
  for (int64_t it = blockIdx.x; it < n_tiles; it += gridDim.x) {
    const int64_t br = it / tiles_c, bc = it - br * tiles_c;
    const int64_t r0 = br * 128 + rg * 8, c0 = bc * 128 + c8 * 8;
    const int nc = clamp8(a.cols - c0);
    Raw8<T> raw[8];
    int pairs[SOURCE == kSorted ? 8 : 1];
    if constexpr (SOURCE == kSorted) {
      if (r0 + 8 <= a.rows) {
        const auto* at = reinterpret_cast<const intx4_any*>(a.pairs + r0);
#pragma unroll
        for (int p = 0; p < 8; ++p) pairs[p] = at[p >> 2][p & 3];
      } else {
#pragma unroll
        for (int p = 0; p < 8; ++p) pairs[p] = r0 + p < a.rows ? a.pairs[r0 + p] : -1;
      }
    }
#pragma unroll
    for (int p = 0; p < 8; ++p) {
      if constexpr (SOURCE == kSorted) {
        const int pair = pairs[p];
        const bool some = pair >= 0 && pair < a.n_pairs;
        const int64_t row = !some ? 0 : a.each > 0 ? pair / a.each : r0 + p;
        raw[p] = raw8(x + row * a.ldx + c0, some ? nc : 0);
      } else {
        raw[p] = raw8(x + (r0 + p) * a.ldx + c0, r0 + p < a.rows ? nc : 0);
      }
    }
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

// The tiles of the product (product_tile.h), or straight from memory for few rows.

struct MatmulPlan {
  int tile;        // 0 none (the few-rows kernel), 1 narrow, 2 small, 3 big
  int splits;      // of the summed axis
  int tm, tn;      // tiles
};

template <class C, int FA, int FB, bool F32>
__global__ __launch_bounds__(C::NT, 2) void matmul_tile_kernel(MatmulArgs a, MatmulPlan plan) {
  // Workgroup w runs on XCD w % 8.  Each XCD takes a run of neighbouring tiles
  // in bands of 8 tile rows, so that the 32 or 64 it holds at a time share
  // operand rows in its L2.
  auto uniform = [](int v) { return __builtin_amdgcn_readfirstlane(v); };
  const unsigned per = plan.tm * plan.tn, total = per * plan.splits, w = blockIdx.x, x = w & 7;
  const unsigned id = x * (total >> 3) + (x < (total & 7) ? x : (total & 7)) + (w >> 3);
  const unsigned split = uniform(id / per), t = id - split * per;
  const unsigned band = uniform(t / (8u * plan.tn)), in = t - band * 8u * plan.tn;
  const unsigned high = plan.tm - band * 8 < 8 ? plan.tm - band * 8 : 8, column = uniform(in / high);
  TileJob o;
  o.a_codes = a.a.codes, o.a_scales = a.a.scales, o.b_codes = a.b.codes, o.b_scales = a.b.scales;
  o.lda = a.a.ld, o.lda_scale = a.a.ld_scale, o.ldb = a.b.ld, o.ldb_scale = a.b.ld_scale;
  o.m = a.a.rows, o.n = a.b.rows;
  o.m0 = static_cast<int64_t>(band * 8 + in - column * high) * C::BM, o.n0 = static_cast<int64_t>(column) * C::BN;
  const unsigned blocks = static_cast<unsigned>((a.a.cols + 127) >> 7);
  o.k0 = uniform(blocks * split / plan.splits), o.nst = uniform(blocks * (split + 1) / plan.splits) - o.k0;
  o.c = a.c, o.ldc = a.ldc, o.c_dtype = a.c_dtype, o.accumulate = a.accumulate;
  if (plan.splits > 1) {     // partial sums: (split, m, n up to a multiple of 8) in fp32
    o.ldc = (o.n + 7) & ~int64_t(7);
    o.c = a.ws + split * o.m * o.ldc;
    o.c_dtype = OKLS_F32;
    o.accumulate = 0;
  }
  tile_product<C, FA, FB, F32>(o);
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

__device__ __forceinline__ intx8 frag(const uint8_t* p) {
  const intx4 lo = reinterpret_cast<const intx4*>(p)[0], hi = reinterpret_cast<const intx4*>(p)[1];
  return intx8{lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
}

// Bound by memory and by the loads that its waves have in flight: one row through 11008 x
// 4096 (45 MB) takes 11.4 us, 4.0 TB/s with the launch in it, of one weight; of eight in turn
// 12.4 us, 3.7 TB/s (fp32 result 13.1).  It reads its operands' fields where they
// are, in the launch's arguments: through a descriptor of 64-bit fields they took vector
// registers (62 -> 82, eight waves a SIMD -> five) and 14.7 us (fp32 14.4).
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

}  // namespace

hipError_t launch_quantize(const QuantArgs& a, hipStream_t s) {
  const int64_t tiles = ((a.rows + 127) / 128) * ((a.cols + 127) / 128);
  const dim3 grid(blocks_up_to(tiles, 1 << 20), a.batch > 1 ? a.batch : 1);
  // the two outputs may differ in format only by two launches
  auto go = [&](const QuantArgs& q, int fmt) {
    by_type(q.x_dtype, [&](auto type) {
      using T = decltype(type);
      auto from = [&](auto source) {
        constexpr int SOURCE = decltype(source)::value;
        if (fmt == OKLS_E4M3) quantize_kernel<T, OKLS_E4M3, SOURCE><<<grid, 256, 0, s>>>(q);
        else quantize_kernel<T, OKLS_E5M2, SOURCE><<<grid, 256, 0, s>>>(q);
      };
      if (q.pairs != nullptr) from(std::integral_constant<int, kSorted>{});
      else if (q.row_factor != nullptr) from(std::integral_constant<int, kFactors>{});
      else from(std::integral_constant<int, kAsIs>{});
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
    by_format(a.a.format, a.b.format, a.c_dtype, [&](auto fa, auto fb, auto f32) {
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
  by_format(a.a.format, a.b.format, a.c_dtype, [&](auto fa, auto fb, auto f32) {
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
