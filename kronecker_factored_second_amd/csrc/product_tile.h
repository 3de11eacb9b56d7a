// The product of 8-bit tiles: codes and scales through LDS into the matrix
// instructions, one tile of c a workgroup.
#pragma once
#include "device_common.h"

namespace okls {
namespace {

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

// One tile of one product c = a b^T, the same for the whole workgroup.
struct TileJob {
  const uint8_t *a_codes, *a_scales, *b_codes, *b_scales;   // of the operands' row 0
  int64_t lda, lda_scale, ldb, ldb_scale;
  int64_t m, n;           // rows of a and of b that the tile may read and c's that it may write: up to m, n
  int64_t m0, n0;         // the tile's first
  int k0, nst;            // blocks of 128 of the summed axis: the first, how many (at least one)
  void* c;
  int64_t ldc;
  int32_t c_dtype, accumulate;
};

template <int N> struct ScaleWord { using type = uint32_t; };
template <> struct ScaleWord<2> { using type = uint16_t; };

// UNEVEN: tiles that end early are common, and a wave whose rows all lie behind the end
// copies its part and leaves the products to the others.
template <class C, int FA, int FB, bool F32, bool UNEVEN = false>
__device__ __forceinline__ void tile_product(const TileJob& o) {
  constexpr int GI = C::GI, GJ = C::GJ;
  constexpr int P = F32 ? 4 : 2;          // parts of a stage of 128 of k
  constexpr int FW = 16 / P;              // dwords of a lane's codes in a block row and part
  constexpr int H = GI / 2;               // block rows of a phase: a phase is half of a's block rows in one part
  __shared__ __attribute__((aligned(16))) uint8_t sA0[C::BM * 128], sA1[C::BM * 128], sB0[C::BN * 128], sB1[C::BN * 128];
  __shared__ __attribute__((aligned(16))) uint8_t e0[512], e1[512];   // scale bytes of the tile's rows, a's and from 256 on b's
  static_assert(C::BM <= 256 && C::BN <= 256, "one copy holds a side's scales");
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = wave / C::WN, wn = wave % C::WN;
  const int64_t m = o.m, n = o.n, m0 = o.m0, n0 = o.n0;
  const int k0 = o.k0, nst = o.nst;

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
  const int64_t ld_scale = of_b ? o.ldb_scale : o.lda_scale;
  const uint8_t *baseA = o.a_codes + m0 * o.lda + k0 * int64_t(128), *baseB = o.b_codes + n0 * o.ldb + k0 * int64_t(128);
  const uint8_t* baseS = (of_b ? o.b_scales + n0 : o.a_scales + m0) + k0 * ld_scale;
  uint32_t ga[C::LA], gb[C::LB];
#pragma unroll
  for (int q = 0; q < C::LA; ++q) {
    const int at = 8 * (wave + C::NW * q) + (lane >> 3), row = at / C::RM * C::RM + (at & 31) * GI + at % C::RM / 32;
    const int64_t r = m0 + row < m ? row : m - 1 - m0;
    ga[q] = static_cast<uint32_t>(r * o.lda) + (((lane & 7) ^ (at >> 1 & 7)) << 4);
  }
#pragma unroll
  for (int q = 0; q < C::LB; ++q) {
    const int at = 8 * (wave + C::NW * q) + (lane >> 3), row = at / C::RN * C::RN + (at & 31) * GJ + at % C::RN / 32;
    const int64_t r = n0 + row < n ? row : n - 1 - n0;
    gb[q] = static_cast<uint32_t>(r * o.ldb) + (((lane & 7) ^ (at >> 1 & 7)) << 4);
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

  // lane l: row l % 32 of each block row, columns 8 q + 4 (l / 32) + 0..3 of
  // each block column, which lie GJ apart: 8 neighbours of a row
  static_assert(GJ == 2, "a lane's neighbours are one 16-byte store of a 16-bit result");
  auto finish = [&]() INLINE {
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
  if (UNEVEN && m0 + wm * C::RM >= m) {
    for (int st = 0; st < nst; ++st) {
      WAIT_VM(0);
      barrier();
      if (st & 1) copy(sA1, sB1, e1);
      else copy(sA0, sB0, e0);
    }
    WAIT_VM(0);
    if constexpr (C::NW == 8) barrier();
    return;
  }
  fetch(I0{}, sA0, sB0, e0);
  for (int st = 0; st < nst; st += 2) {
    stage(I0{});
    if (st + 1 < nst) stage(I1{});
  }
  WAIT_VM(0);              // the last copies land before the buffers are used again or given up
  if constexpr (C::NW == 8) barrier();
  finish();
}

// a product with nothing to sum
__global__ __launch_bounds__(256) void zero_kernel(void* c, int dtype, int64_t m, int64_t n, int64_t ldc) {
  for (int64_t i = blockIdx.x * 256ll + threadIdx.x; i < m * n; i += gridDim.x * 256ll) store_any(c, i / n * ldc + i % n, dtype, 0.0f);
}

// calls go(a's format, b's format, fp32 result) with compile-time values
template <class F>
void by_format(int32_t format_a, int32_t format_b, int32_t c_dtype, F go) {
  using I0 = std::integral_constant<int, 0>;
  using I1 = std::integral_constant<int, 1>;
  auto second = [&](auto fa) {
    auto third = [&](auto fb) {
      if (c_dtype == OKLS_F32) go(fa, fb, std::true_type{});
      else go(fa, fb, std::false_type{});
    };
    if (format_b == OKLS_E4M3) third(I0{});
    else third(I1{});
  };
  if (format_a == OKLS_E4M3) second(I0{});
  else second(I1{});
}

}  // namespace
}  // namespace okls
