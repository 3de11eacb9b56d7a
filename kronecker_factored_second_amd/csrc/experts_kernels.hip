// gfx950 kernels of the experts' operators (okls_experts.h).
//
//  plan_one_kernel       a stable counting sort of choices by expert in one workgroup;
//  plan_rank_kernel,     in several, ranks within each one's choices,
//  plan_place_kernel     then rows from all workgroups' counts.
//  gather_kernel         tokens' rows to the sorted order;
//  combine_kernel        back, weighted and summed: also the gradient of the first;
//  combine_backward_kernel   the gradients of the second.
//  expert_stream_kernel  the product where experts have few rows, through a ring in LDS.
//  expert_tile_kernel    the product by product_tile.h's tiles, each with its own
//                        expert's matrix; expert_rest_kernel, what whole rounds of
//                        large tiles leave over.
//  expert_weight_kernel  the weights' gradients, by the same tiles.
#include "experts_kernels.h"
#include "product_tile.h"

#include "../../include/okls_experts.h"

namespace okls {
namespace {

// ---------------------------------------------------------------------------
// The sorted order
// ---------------------------------------------------------------------------
// A stable counting sort.  A workgroup ranks groups of 4096 choices, a wave 256
// of them in turn, 64 at a time: lanes with the same expert find each other by one
// ballot for each bit of its number, the count so far is the wave's own in LDS.
// Then the counts of the waves, groups and workgroups before are added.
// Bound by latency: 65536 choices of 64 experts take two launches of 7 and 6.5 us (in
// three launches with ranks kept in memory it took 24); up to 4096 choices one
// workgroup does it all in 4 us.
constexpr int kPlanThreads = 1024, kPlanWaves = kPlanThreads / 64;
constexpr int kPlanEach = 4, kPlanGroup = kPlanThreads * kPlanEach;
constexpr int kPlanBlocks = 64;         // workgroups at most: each adds up the counts of all

template <bool WIDE>
__device__ __forceinline__ int choice_at(const void* choice, int i, int n_experts) {
  if constexpr (WIDE) {
    const int64_t e = static_cast<const int64_t*>(choice)[i];
    return e >= 0 && e < n_experts ? static_cast<int>(e) : n_experts;
  } else {
    const int e = static_cast<const int32_t*>(choice)[i];
    return e >= 0 && e < n_experts ? e : n_experts;
  }
}

// this thread's choices of a group: first + 64 q, q < kPlanEach
__device__ __forceinline__ int first_of(int group) { return group + (threadIdx.x >> 6) * (64 * kPlanEach) + (threadIdx.x & 63); }

template <bool WIDE>
__device__ __forceinline__ void read_group(const void* choice, int group, int end, int n_experts, int (&e)[kPlanEach]) {
  const int first = first_of(group);
#pragma unroll
  for (int q = 0; q < kPlanEach; ++q) e[q] = first + 64 * q < end ? choice_at<WIDE>(choice, first + 64 * q, n_experts) : n_experts;
}

// rank[q] = the number of this group's choices of the same expert before choice q;
// returns expert t's number of choices in thread t.  count: kPlanWaves x n_experts in LDS.
__device__ __forceinline__ int rank_group(const int (&e)[kPlanEach], int n_experts, int bits, int* count, int (&rank)[kPlanEach]) {
  const int t = threadIdx.x, lane = t & 63;
  int* mine = count + (t >> 6) * n_experts;
  for (int i = t; i < kPlanWaves * n_experts; i += kPlanThreads) count[i] = 0;
  __syncthreads();
#pragma unroll
  for (int q = 0; q < kPlanEach; ++q) {
    uint64_t same = ~uint64_t(0);
    for (int b = 0; b < bits; ++b) {
      const uint64_t set = __ballot(e[q] >> b & 1);
      same &= e[q] >> b & 1 ? set : ~set;
    }
    const int before = __popcll(same & ((uint64_t(1) << lane) - 1));
    const bool some = e[q] < n_experts;
    const int seen = some ? mine[e[q]] : 0;
    // every lane has read its expert's count before the group's first lane moves it
    __builtin_amdgcn_wave_barrier();
    if (some && before == 0) mine[e[q]] = seen + __popcll(same);
    __builtin_amdgcn_wave_barrier();
    rank[q] = seen + before;
  }
  __syncthreads();
  int total = 0;
  if (t < n_experts) {
    int c[kPlanWaves];
#pragma unroll
    for (int w = 0; w < kPlanWaves; ++w) c[w] = count[w * n_experts + t];
#pragma unroll
    for (int w = 0; w < kPlanWaves; ++w) {
      count[w * n_experts + t] = total;
      total += c[w];
    }
  }
  __syncthreads();
#pragma unroll
  for (int q = 0; q < kPlanEach; ++q)
    if (e[q] < n_experts) rank[q] += mine[e[q]];
  return total;
}

// the experts' first rows from their totals (thread t's): offset, n_experts + 1 in LDS; `write`: in memory too
__device__ __forceinline__ void make_offsets(int total, const ExpertPlan& p, int* offset, bool write) {
  __shared__ int waves[kPlanWaves];
  const int t = threadIdx.x, lane = t & 63;
  int room = t < p.n_experts ? (total + p.align - 1) / p.align * p.align : 0;
  const int own = room;
  for (int o = 1; o < 64; o <<= 1) {
    const int other = __shfl_up(room, o, 64);
    if (lane >= o) room += other;
  }
  if (lane == 63) waves[t >> 6] = room;
  __syncthreads();
  for (int w = 0; w < t >> 6; ++w) room += waves[w];
  if (t < p.n_experts) {
    offset[t] = room - own;
    if (t == p.n_experts - 1) offset[t + 1] = room;
    if (write) {
      p.offsets[t] = room - own;
      p.counts[t] = total;
      if (t == p.n_experts - 1) p.offsets[t + 1] = room;
    }
  }
  __syncthreads();
}

// all of it in one workgroup
template <bool WIDE>
__global__ __launch_bounds__(kPlanThreads) void plan_one_kernel(const void* choice, ExpertPlan p, int bits) {
  extern __shared__ int lds[];            // kPlanWaves x n_experts counts, n_experts + 1 offsets
  int* offset = lds + kPlanWaves * p.n_experts;
  int e[kPlanEach], rank[kPlanEach];
  read_group<WIDE>(choice, 0, p.n_pairs, p.n_experts, e);
  for (int r = threadIdx.x; r < p.capacity; r += kPlanThreads) p.pairs[r] = -1;
  const int total = rank_group(e, p.n_experts, bits, lds, rank);
  make_offsets(total, p, offset, true);
  const int first = first_of(0);
#pragma unroll
  for (int q = 0; q < kPlanEach; ++q) {
    const int i = first + 64 * q;
    if (i >= p.n_pairs) continue;
    const int row = e[q] < p.n_experts ? offset[e[q]] + rank[q] : -1;
    p.rows[i] = row;
    if (row >= 0) p.pairs[row] = i;
  }
}

// a chunk of groups a workgroup: ranks within it, and its counts (workgroup, expert)
template <bool WIDE>
__global__ __launch_bounds__(kPlanThreads) void plan_rank_kernel(const void* choice, ExpertPlan p, int bits, int chunk, int32_t* counts) {
  extern __shared__ int lds[];            // kPlanWaves x n_experts counts, n_experts of the groups before
  int* before = lds + kPlanWaves * p.n_experts;
  const int t = threadIdx.x, begin = blockIdx.x * chunk, end = min(begin + chunk, p.n_pairs);
  if (t < p.n_experts) before[t] = 0;
  for (int group = begin; group < end; group += kPlanGroup) {
    int e[kPlanEach], rank[kPlanEach];
    read_group<WIDE>(choice, group, end, p.n_experts, e);
    const int total = rank_group(e, p.n_experts, bits, lds, rank);
    const int first = first_of(group);
#pragma unroll
    for (int q = 0; q < kPlanEach; ++q)
      if (first + 64 * q < end && e[q] < p.n_experts) p.rows[first + 64 * q] = rank[q] + before[e[q]];
    __syncthreads();
    if (t < p.n_experts) before[t] += total;
  }
  if (t < p.n_experts) counts[blockIdx.x * p.n_experts + t] = before[t];
}

// Every workgroup adds up the counts of all, and those before its own; then its choices' rows.
template <bool WIDE>
__global__ __launch_bounds__(kPlanThreads) void plan_place_kernel(const void* choice, ExpertPlan p, int chunk, const int32_t* counts) {
  extern __shared__ int lds[];            // n_experts + 1 offsets, then this chunk's first rows
  int *offset = lds, *start = lds + p.n_experts + 1;
  const int t = threadIdx.x, blocks = gridDim.x, begin = blockIdx.x * chunk, end = min(begin + chunk, p.n_pairs);
  int total = 0, mine = 0;
  if (t < p.n_experts)
#pragma unroll 16
    for (int b = 0; b < blocks; ++b) {
      const int c = counts[b * p.n_experts + t];
      if (b < static_cast<int>(blockIdx.x)) mine += c;
      total += c;
    }
  make_offsets(total, p, offset, blockIdx.x == 0);
  if (t < p.n_experts) start[t] = offset[t] + mine;
  __syncthreads();
  for (int group = begin; group < end; group += kPlanGroup) {
    int e[kPlanEach], rank[kPlanEach];
    read_group<WIDE>(choice, group, end, p.n_experts, e);
    const int first = first_of(group);
#pragma unroll
    for (int q = 0; q < kPlanEach; ++q) rank[q] = first + 64 * q < end && e[q] < p.n_experts ? p.rows[first + 64 * q] : 0;
#pragma unroll
    for (int q = 0; q < kPlanEach; ++q) {
      const int i = first + 64 * q;
      if (i >= end) continue;
      const int row = e[q] < p.n_experts ? start[e[q]] + rank[q] : -1;
      p.rows[i] = row;
      if (row >= 0) p.pairs[row] = i;
    }
  }
  // rows without a choice: behind each expert's, and behind the last one
  __syncthreads();
  if (blockIdx.x == gridDim.x - 1 && t < p.n_experts) start[t] = offset[t] + total;
  __syncthreads();
  if (blockIdx.x == gridDim.x - 1)
    for (int i = t; i < p.n_experts * p.align; i += kPlanThreads) {
      const int e = i / p.align, r = start[e] + i % p.align;
      if (r < offset[e + 1]) p.pairs[r] = -1;
    }
  for (int64_t r = static_cast<int64_t>(offset[p.n_experts]) + blockIdx.x * kPlanThreads + t; r < p.capacity; r += blocks * kPlanThreads) p.pairs[r] = -1;
}

// ---------------------------------------------------------------------------
// Rows to the sorted order and back
// ---------------------------------------------------------------------------
// Tokens lead in every direction: a token's row is read (written) once for all
// its choices.  The first workgroups write the zeros of rows without a choice.
// Bound by memory.  8192 tokens of 8 choices, 2048 columns of bf16: to the sorted order
// (335 MB) 54 us, 6.2 TB/s; back (302 MB) 48 us, 6.3 TB/s; the gradient (603 MB) 121 us,
// 5.0 TB/s.  Sorted rows are read past the caches, which keep what comes next: that
// alone took there and back together from 160 to 121 us.  A wave a token, so that all
// rows' first columns were read at once, took 90 us back; zeros by a wave an expert 55 us
// for any sizes.
constexpr int kZeroGroups = 64;

// A token's choices from k0 on, at most 64 of them, a lane each: their rows, -1 for none.
__device__ __forceinline__ int rows_of(const ExpertPlan& p, int64_t token, int k0) {
  const int k = k0 + (threadIdx.x & 63);
  const int r = k < p.each ? p.rows[token * p.each + k] : -1;
  return r < p.capacity ? r : -1;
}
// their weights, 0 where there is no row: what a dropped choice's weight holds counts for nothing
__device__ __forceinline__ float weights_of(const RowsArgs& a, int64_t token, int k0, int row) {
  if (row < 0) return 0.0f;
  return a.weights != nullptr ? load_any(a.weights, token * a.plan.each + k0 + (threadIdx.x & 63), a.weight_dtype) : 1.0f;
}
__device__ __forceinline__ int at_lane(int v, int lane) { return __builtin_amdgcn_readlane(v, lane); }
__device__ __forceinline__ float at_lane(float v, int lane) { return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), lane)); }

// raw8 of what is not read again: past the caches
template <typename T>
__device__ __forceinline__ Raw8<T> raw8_once(const T* p, int n) {
  if (n < 8) return raw8(p, n);
  Raw8<T> r;
  if constexpr (sizeof(T) == 4) r.a = __builtin_nontemporal_load(reinterpret_cast<const floatx4_any*>(p)), r.b = __builtin_nontemporal_load(reinterpret_cast<const floatx4_any*>(p) + 1);
  else r.v = __builtin_nontemporal_load(reinterpret_cast<const u16x8_any*>(p));
  return r;
}

template <typename T>
__device__ __forceinline__ void put_raw8(T* p, const Raw8<T>& r, int n) {
  if (n >= 8) {
    if constexpr (sizeof(T) == 4) reinterpret_cast<floatx4_any*>(p)[0] = r.a, reinterpret_cast<floatx4_any*>(p)[1] = r.b;
    else *reinterpret_cast<u16x8_any*>(p) = r.v;
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (j < n) {
        if constexpr (sizeof(T) == 4) p[j] = j < 4 ? r.a[j & 3] : r.b[j & 3];
        else p[j] = __builtin_bit_cast(T, static_cast<uint16_t>(r.v[j]));
      }
  }
}

// zeros in the rows without a choice, by wave `wave` of `waves`
template <typename T>
__device__ __forceinline__ void zero_rows(const ExpertPlan& p, T* out, int64_t ldo, int64_t cols, int wave, int waves) {
  const int lane = threadIdx.x & 63;
  const Raw8<T> zeros{};
  auto clear = [&](int64_t r) {
    for (int64_t c = lane * 8; c < cols; c += 512) put_raw8(out + r * ldo + c, zeros, clamp8(cols - c));
  };
  // fewer than `align` rows an expert, one at a time: an expert's spread over all waves
  for (int i = wave; i < p.n_experts * p.align; i += waves) {
    const int e = i / p.align, r = max(p.offsets[e] + p.counts[e], 0) + i % p.align;
    if (r < min(p.offsets[e + 1], p.capacity)) clear(r);
  }
  for (int64_t r = static_cast<int64_t>(max(p.offsets[p.n_experts], 0)) + wave; r < p.capacity; r += waves) clear(r);
}

// What a lane holds for others (a row's number, a weight) is read from it where all
// lanes are active: loops run over the wave's columns, and lanes past the end hold 0 of them.
//
// How a launch shares out tokens and columns: `waves` of a workgroup's four stand
// side by side on one token's parts of 512 columns, 4 / waves tokens a workgroup;
// gridDim.y workgroups along a row where there are few tokens.
struct Place {
  int64_t token, step;        // the wave's first token, and from one to its next
  int64_t column, stride;     // the wave's first 512 columns, and from them to its next
};
__device__ __forceinline__ Place place(int block, int blocks, int waves) {
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), each = 4 / waves;
  const int part = blockIdx.y * waves + wave % waves;
  return {static_cast<int64_t>(block) * each + wave / waves, static_cast<int64_t>(blocks) * each,
          part * int64_t(512), static_cast<int64_t>(gridDim.y) * waves * 512};
}

template <typename T>
__global__ __launch_bounds__(256) void gather_kernel(RowsArgs a, int waves) {
  const ExpertPlan& p = a.plan;
  T* out = static_cast<T*>(a.out);
  if (blockIdx.x < kZeroGroups) {
    zero_rows(p, out, a.ldo, a.cols, (blockIdx.x * gridDim.y + blockIdx.y) * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), kZeroGroups * gridDim.y * 4);
    return;
  }
  const T* x = static_cast<const T*>(a.x);
  const Place at = place(blockIdx.x - kZeroGroups, gridDim.x - kZeroGroups, waves);
  for (int64_t t = at.token; t < p.tokens; t += at.step)
    for (int k0 = 0; k0 < p.each; k0 += 64) {
      const int row = rows_of(p, t, k0), ks = min(p.each - k0, 64);
      for (int64_t c0 = at.column; c0 < a.cols; c0 += at.stride) {
        const int64_t c = c0 + (threadIdx.x & 63) * 8;
        const int n = clamp8(a.cols - c);
        const Raw8<T> v = raw8(x + t * a.ldx + c, n);
        for (int k = 0; k < ks; ++k) {
          const int64_t r = at_lane(row, k);
          if (r >= 0) put_raw8(out + r * a.ldo + c, v, n);
        }
      }
    }
}

// G choices at a time, their rows' loads on their way together
template <typename T, int G>
__global__ __launch_bounds__(256) void combine_kernel(RowsArgs a, int waves) {
  const ExpertPlan& p = a.plan;
  const T* y = static_cast<const T*>(a.y);
  T* out = static_cast<T*>(a.out);
  const Place at = place(blockIdx.x, gridDim.x, waves);
  for (int64_t t = at.token; t < p.tokens; t += at.step) {
    int row = rows_of(p, t, 0);
    float weight = weights_of(a, t, 0, row);
    for (int64_t c0 = at.column; c0 < a.cols; c0 += at.stride) {
      const int64_t c = c0 + (threadIdx.x & 63) * 8;
      const int n = clamp8(a.cols - c);
      float s[8] = {};
      for (int k0 = 0; k0 < p.each; k0 += G) {
        if (p.each > 64 && (k0 & 63) == 0) {
          row = rows_of(p, t, k0);
          weight = weights_of(a, t, k0, row);
        }
        Raw8<T> v[G];
#pragma unroll
        for (int q = 0; q < G; ++q) {
          const int64_t r = at_lane(row, (k0 + q) & 63);
          v[q] = raw8_once(y + (r < 0 ? 0 : r) * a.ldy + c, r >= 0 ? n : 0);
        }
#pragma unroll
        for (int q = 0; q < G; ++q) {
          const float w = at_lane(weight, (k0 + q) & 63);
#pragma unroll
          for (int j = 0; j < 8; ++j) s[j] = fmaf(w, element(v[q], j), s[j]);
        }
      }
      store8(out + t * a.ldo + c, s, n);
    }
  }
}

// dy and dweights: G of a token's choices at a time, whose sums stay in registers
// and meet over a wave, and over the waves of a token in LDS.
template <typename T, int G>
__global__ __launch_bounds__(256) void combine_backward_kernel(RowsArgs a, int waves) {
  __shared__ float part[4][G];
  const ExpertPlan& p = a.plan;
  T* out = static_cast<T*>(a.out);
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
  if (blockIdx.x < kZeroGroups) {
    zero_rows(p, out, a.ldo, a.cols, blockIdx.x * 4 + wave, kZeroGroups * 4);
    return;
  }
  const T* d = static_cast<const T*>(a.x);
  const T* y = static_cast<const T*>(a.y);
  const Place at = place(blockIdx.x - kZeroGroups, gridDim.x - kZeroGroups, waves);
  // the workgroup's first token decides how often: all its waves meet at the barriers
  for (int64_t first = at.token - wave / waves; first < p.tokens; first += at.step) {
    const int64_t t = first + wave / waves;
    for (int k0 = 0; k0 < p.each; k0 += G) {
      const int row = t < p.tokens ? rows_of(p, t, k0) : -1;
      const float weight = weights_of(a, t, k0, row);
      float sum[G] = {};
      for (int64_t c0 = at.column; c0 < a.cols && t < p.tokens; c0 += at.stride) {
        const int64_t c = c0 + lane * 8;
        const int n = clamp8(a.cols - c);
        float g[8];
        load8(g, d + t * a.ldx + c, n);
        Raw8<T> v[G];
#pragma unroll
        for (int q = 0; q < G; ++q) {
          const int64_t r = at_lane(row, q);
          v[q] = raw8_once(y + (r < 0 ? 0 : r) * a.ldy + c, r >= 0 ? n : 0);
        }
#pragma unroll
        for (int q = 0; q < G; ++q) {
          const int64_t r = at_lane(row, q);
          const float w = at_lane(weight, q);
          float u[8];
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            sum[q] = fmaf(g[j], element(v[q], j), sum[q]);
            u[j] = w * g[j];
          }
          if (r >= 0) store8(out + r * a.ldo + c, u, n);
        }
      }
#pragma unroll
      for (int q = 0; q < G; ++q) {
#pragma unroll
        for (int o = 32; o > 0; o >>= 1) sum[q] += __shfl_xor(sum[q], o, 64);
        if (lane == 0) part[wave][q] = sum[q];
      }
      __syncthreads();
      if (wave % waves == 0 && lane < G && t < p.tokens && k0 + lane < p.each) {
        float s = part[wave][lane];
        for (int w = 1; w < waves; ++w) s += part[wave + w][lane];
        // without a row nothing is summed, whatever dout holds
        store_any(a.dweights, t * p.each + k0 + lane, a.weight_dtype, row >= 0 ? s : 0.0f);
      }
      __syncthreads();
    }
  }
}

// ---------------------------------------------------------------------------
// Products
// ---------------------------------------------------------------------------
// Where a workgroup's tile lies: the sorted rows are cut into tiles of BM rows,
// expert by expert.  The host knows only how many there are at most, so every wave
// counts them from the offsets, a lane an expert.
struct TileRows {
  int expert, first, end;     // its rows: first up to end, the expert's last one's
};

// rows of expert e: [first, end), inside the buffer whatever the offsets hold
__device__ __forceinline__ void expert_rows(const ExpertPlan& p, int e, int& first, int& end) {
  first = min(max(p.offsets[e], 0), p.capacity) & ~15;
  end = max(min(p.offsets[e + 1], p.capacity) & ~15, first);
}

// v summed over this lane and those before it, inside the ALU: within each 16
// lanes, then from row to row
__device__ __forceinline__ int sum_up_to(int v) {
  auto from = [](int x, auto ctrl, auto rows) { return __builtin_amdgcn_update_dpp(0, x, decltype(ctrl)::value, decltype(rows)::value, 0xf, false); };
  using All = std::integral_constant<int, 0xf>;
  v += from(v, std::integral_constant<int, 0x111>{}, All{});
  v += from(v, std::integral_constant<int, 0x112>{}, All{});
  v += from(v, std::integral_constant<int, 0x114>{}, All{});
  v += from(v, std::integral_constant<int, 0x118>{}, All{});
  v += from(v, std::integral_constant<int, 0x142>{}, std::integral_constant<int, 0xa>{});
  return v + from(v, std::integral_constant<int, 0x143>{}, std::integral_constant<int, 0xc>{});
}

// 64 experts, one a lane: its rows, and the tiles of BM rows of it and those before it
struct ExpertLanes {
  int first, end, upto;
};
template <int BM>
__device__ __forceinline__ ExpertLanes expert_lanes(const ExpertPlan& p, int e0) {
  const int e = e0 + (threadIdx.x & 63);
  ExpertLanes x{0, 0, 0};
  if (e < p.n_experts) expert_rows(p, e, x.first, x.end);
  x.upto = sum_up_to((x.end - x.first + BM - 1) / BM);
  return x;
}

// The tiles of all experts; `x` is expert_lanes of the first 64, whose offsets are read once.
template <int BM>
__device__ __forceinline__ int count_tiles(const ExpertPlan& p, ExpertLanes& x) {
  x = expert_lanes<BM>(p, 0);
  int total = __builtin_amdgcn_readlane(x.upto, 63);
  for (int e0 = 64; e0 < p.n_experts; e0 += 64) total += __builtin_amdgcn_readlane(expert_lanes<BM>(p, e0).upto, 63);
  return total;
}

// tile t < count_tiles
template <int BM>
__device__ __forceinline__ TileRows find_tile(const ExpertPlan& p, int t, ExpertLanes x) {
  TileRows r{0, 0, 0};
  int before = 0;
  for (int e0 = 0; e0 < p.n_experts; e0 += 64) {
    if (e0 != 0) {
      x = expert_lanes<BM>(p, e0);
      x.upto += before;
    }
    const int all = __builtin_amdgcn_readlane(x.upto, 63);
    if (t < all) {
      const int lane = __popcll(__ballot(x.upto <= t));     // experts that end at or before t
      const int begin = lane == 0 ? before : __builtin_amdgcn_readlane(x.upto, lane - 1);
      r.expert = e0 + lane;
      r.first = __builtin_amdgcn_readlane(x.first, lane) + (t - begin) * BM;
      r.end = __builtin_amdgcn_readlane(x.end, lane);
      break;
    }
    before = all;
  }
  return r;
}

// the most tiles of BM rows that any offsets of this plan give
int most_tiles(const ExpertPlan& p, int bm) {
  const int64_t some = p.n_pairs < p.n_experts ? p.n_pairs : p.n_experts;
  return static_cast<int>((p.capacity + some * (bm > p.align ? bm - p.align : 0)) / bm);
}

// workgroup j of n: zeros in c's rows behind the last expert's, 16 bytes at a time
__device__ __forceinline__ void zero_tail(const ExpertMatmulArgs& a, int64_t j, int64_t n) {
  typedef u16x8 zeros_any __attribute__((aligned(2)));
  const int size = a.c_dtype == OKLS_F32 ? 4 : 2, per = 16 / size;
  for (int64_t r = min(max(a.plan.offsets[a.plan.n_experts], 0), a.plan.capacity) + j; r < a.plan.capacity; r += n)
    for (int64_t c = threadIdx.x * per; c < a.n; c += static_cast<int64_t>(blockDim.x) * per) {
      if (c + per <= a.n) *reinterpret_cast<zeros_any*>(static_cast<uint8_t*>(a.c) + (r * a.ldc + c) * size) = u16x8{};
      else for (int64_t e = c; e < a.n; ++e) store_any(a.c, r * a.ldc + e, a.c_dtype, 0.0f);
    }
}

__device__ __forceinline__ TileJob expert_job(const ExpertMatmulArgs& a, const TileRows& rows) {
  TileJob o;
  const int64_t first = rows.expert * ((a.n + 15) & ~int64_t(15));
  o.a_codes = a.a.codes, o.a_scales = a.a.scales;
  o.b_codes = a.b.codes + first * a.b.ld, o.b_scales = a.b.scales + first;
  o.lda = a.a.ld, o.lda_scale = a.a.ld_scale, o.ldb = a.b.ld, o.ldb_scale = a.b.ld_scale;
  o.m = rows.end, o.n = a.n, o.m0 = rows.first;
  o.k0 = 0, o.nst = static_cast<int>((a.a.cols + 127) >> 7);
  o.c = a.c, o.ldc = a.ldc, o.c_dtype = a.c_dtype, o.accumulate = 0;
  return o;
}

constexpr int kTailGroups = 64;    // more workgroups than tiles, so that some write the zeros

// Large tiles are one workgroup a CU.  What is left over after whole rounds of all
// CUs, where it is at most half a round, goes to a launch of small tiles, four of which
// are a large one and two of which a CU holds: 16384 uneven rows x 2048 x 5632 193 ->
// 177 us.  A round of short sums costs less than the launch (64 experts, 32764 rows x
// 2816 x 1024: 157 -> 164 us), so that it is made from a summed axis of kLongSum on.
constexpr unsigned kRound = 256;
constexpr int64_t kLongSum = 4096;
__device__ __forceinline__ unsigned whole_rounds(unsigned total) {
  return total % kRound <= kRound / 2 ? total - total % kRound : total;
}

// tile t's rows, and its column of tiles: bands of 8 tile rows, column by column
template <class C>
__device__ __forceinline__ TileJob tile_job(const ExpertMatmulArgs& a, unsigned t, unsigned tm, unsigned tn, const ExpertLanes& lanes) {
  auto uniform = [](int v) { return __builtin_amdgcn_readfirstlane(v); };
  const unsigned band = uniform(t / (8u * tn)), in = t - band * 8u * tn;
  const unsigned high = tm - band * 8 < 8 ? tm - band * 8 : 8, column = uniform(in / high);
  TileJob o = expert_job(a, find_tile<C::BM>(a.plan, band * 8 + in - column * high, lanes));
  o.n0 = static_cast<int64_t>(column) * C::BN;
  return o;
}

// Bound as the plain product's tiles are where experts have many rows (16384 x 5632 x
// 2048: plain 204 us, 8 experts 187 to 191); with many experts also by their
// weights' way from memory, each of which one round of tiles reads (32764 rows x 2816 x 1024: plain
// 107 us, 64 experts 157 to 164, of 457 MB).
template <class C, int FA, int FB, bool F32>
__global__ __launch_bounds__(C::NT, 2) void expert_tile_kernel(ExpertMatmulArgs a, unsigned tn, bool rest_apart) {
  ExpertLanes lanes;
  const unsigned tm = count_tiles<C::BM>(a.plan, lanes), whole = rest_apart ? whole_rounds(tm * tn) : tm * tn, w = blockIdx.x, x = w & 7;
  if (w >= whole) return zero_tail(a, w - whole, gridDim.x - whole);
  // as in the plain product: each XCD takes a run of neighbouring tiles
  tile_product<C, FA, FB, F32, true>(tile_job<C>(a, x * (whole >> 3) + (x < (whole & 7) ? x : (whole & 7)) + (w >> 3), tm, tn, lanes));
}

template <int FA, int FB, bool F32>
__global__ __launch_bounds__(TileSmall::NT, 2) void expert_rest_kernel(ExpertMatmulArgs a, unsigned tn) {
  static_assert(TileBig::BM == 2 * TileSmall::BM && TileBig::BN == 2 * TileSmall::BN, "four small tiles are a large one");
  ExpertLanes lanes;
  const unsigned tm = count_tiles<TileBig::BM>(a.plan, lanes), total = tm * tn, t = whole_rounds(total) + (blockIdx.x >> 2);
  if (t >= total) return;
  TileJob o = tile_job<TileBig>(a, t, tm, tn, lanes);
  o.m0 += (blockIdx.x >> 1 & 1) * TileSmall::BM;
  o.n0 += (blockIdx.x & 1) * TileSmall::BN;
  if (o.m0 < o.m && o.n0 < o.n) tile_product<TileSmall, FA, FB, F32, true>(o);
}

// Few rows an expert: units of 32 rows and 64 columns, 16 a wave, an even share of
// them to each of as many workgroups as the card holds.  Bound by memory: 8 experts of
// 11008 x 4096 (364 MB) and 4 rows each take 75 to 77 us with four sets of weights in
// turn, 4.8 TB/s (reads alone reach 6.3 to 7); with one set, half of which the
// last-level cache may serve, 61 to 76 from card to card.  With one set, straight from memory into registers it took 91 to 105 us, narrow tiles, which wait
// for each stage's copies before the next, 84 to 93.  Codes and scales come by
// direct-to-LDS copies into a ring of kStages blocks of 128 of the summed axis, which runs
// on through the units: what a unit begins with is on its way while the one before
// it ends.  The weights' codes pass the caches by, as they are read once.
constexpr int kStages = 6, kStreamGroups = 512;     // two workgroups a CU
// a stage's codes, b's and then a's, and scale bytes, b's 64 and then a's 32
constexpr int kStreamScales = 64 * 128 + 32 * 128, kStreamBytes = kStreamScales + 256;

template <int FA, int FB, bool F32>
__global__ __launch_bounds__(256) void expert_stream_kernel(ExpertMatmulArgs a) {
  __shared__ __attribute__((aligned(16))) uint8_t ring[kStages * kStreamBytes];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int blocks = static_cast<int>((a.a.cols + 127) >> 7);
  const unsigned columns = static_cast<unsigned>((a.n + 63) >> 6);
  ExpertLanes lanes;
  const int tm = count_tiles<32>(a.plan, lanes);
  const uint64_t units = static_cast<uint64_t>(tm) * columns, unit = units * blockIdx.x / gridDim.x;
  const int64_t steps = static_cast<int64_t>(units * (blockIdx.x + 1) / gridDim.x - unit) * blocks;

  if (steps > 0) {
    // What is copied next.  Copies: 8 rows of 128 bytes each, two of b and one of a a wave;
    // 16-byte chunk c of row r lies at position c ^ (r / 2 % 8), so that 16
    // lanes that read one chunk of 16 rows cover all banks.  Rows past the end
    // read the last one; what they give is not stored.  Scale bytes: one copy, by every
    // wave to the same place.
    unsigned tile = static_cast<unsigned>(unit / columns), column = static_cast<unsigned>(unit - static_cast<uint64_t>(tile) * columns);
    TileRows rows = find_tile<32>(a.plan, tile, lanes);
    const int chunk = lane & 7, in = lane >> 3;
    const uint8_t *pa, *pb[2], *pe;
    const bool of_b = lane < 16;
    const int64_t step_b = a.b.ld_scale, step_a = a.a.ld_scale, step_e = of_b ? step_b : step_a;
    auto aim = [&]() INLINE {
      const int64_t first = rows.expert * ((a.n + 15) & ~int64_t(15)), c0 = column * int64_t(64);
      const int ra = wave * 8 + in;
      pa = a.a.codes + min(rows.first + ra, rows.end - 1) * a.a.ld + ((chunk ^ (ra >> 1 & 7)) << 4);
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        const int rb = (2 * wave + q) * 8 + in;
        const int64_t c = c0 + rb < a.n ? c0 + rb : a.n - 1;
        pb[q] = a.b.codes + (first + c) * a.b.ld + ((chunk ^ (rb >> 1 & 7)) << 4);
      }
      // four bytes a lane: 16 lanes of b's, 8 of a's (rows padded to 16 exist)
      const int64_t last_b = ((a.n + 15) & ~int64_t(15)) - 4, last_a = ((rows.end + 15) & ~15) - 4;
      const int64_t eb = c0 + 4 * lane < last_b ? c0 + 4 * lane : last_b, ea = rows.first + 4 * (lane - 16) < last_a ? rows.first + 4 * (lane - 16) : last_a;
      pe = of_b ? a.b.scales + first + eb : a.a.scales + (lane < 24 ? ea : rows.first);
    };
    aim();
    int block = 0;
    int64_t copied = 0;
    auto copy = [&](uint8_t* to) INLINE {
#pragma unroll
      for (int q = 0; q < 2; ++q)
        __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) void*)pb[q],
                                         (__attribute__((address_space(3))) void*)(to + (2 * wave + q) * 1024), 16, 0, 2);
      __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) void*)pa,
                                       (__attribute__((address_space(3))) void*)(to + 64 * 128 + wave * 1024), 16, 0, 0);
      __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) void*)pe,
                                       (__attribute__((address_space(3))) void*)(to + kStreamScales), 4, 0, 0);
      // past the end the last block again, into a stage that nothing reads: the same number of copies at every step
      if (++copied >= steps) return;
      if (++block < blocks) {
        pb[0] += 128, pb[1] += 128, pa += 128, pe += step_e;
        return;
      }
      block = 0;
      if (++column == columns) {
        column = 0;
        rows = find_tile<32>(a.plan, ++tile, lanes);
      }
      aim();
    };

    // Where a lane reads in a stage: two 16-byte chunks of its row of b, and of a, and their
    // scale bytes.  Both operands take chunks `quarter` and `quarter` + 4, and a sum does not care which
    // (2 quarter and the next one met in the banks).
    const int r = lane & 15, quarter = lane >> 4, sw = r >> 1 & 7;
    const uint32_t base = static_cast<uint32_t>(reinterpret_cast<uintptr_t>((__attribute__((address_space(3))) uint8_t*)ring));
    const uint32_t lo = (quarter ^ sw) << 4, hi = ((quarter + 4) ^ sw) << 4;
    const uint32_t b_lo = base + (wave * 16 + r) * 128 + lo, b_hi = b_lo - lo + hi, a_lo = base + (64 + r) * 128 + lo, a_hi = a_lo - lo + hi;
    const uint32_t b_e = base + kStreamScales + wave * 16 + r, a_e = base + kStreamScales + 64 + r;
    floatx4 acc[2] = {};
    unsigned here_tile = tile, here_column = column;
    TileRows here = rows;
    int done = 0;
    for (int q = 0; q < kStages - 1; ++q) copy(ring + q * kStreamBytes);
    int stage = 0, free = (kStages - 1) * kStreamBytes;      // byte offsets
    for (int64_t s = 0; s < steps; ++s) {
      // this wave's part of the stage is in LDS, and its reads of the last one are over; then everyone's
      WAIT_VM(4 * (kStages - 2));
      asm volatile("" ::: "memory");
      __builtin_amdgcn_s_barrier();
      asm volatile("" ::: "memory");
      copy(ring + free);
      // Read by hand: the compiler would wait for every copy under way before a read of the ring.
      intx4 bl, bh, al[2], ah[2];
      int sb, sa[2];
      asm volatile("ds_read_b128 %0, %9\n\t"
                   "ds_read_b128 %1, %10\n\t"
                   "ds_read_b128 %2, %11\n\t"
                   "ds_read_b128 %3, %12\n\t"
                   "ds_read_b128 %4, %11 offset:2048\n\t"
                   "ds_read_b128 %5, %12 offset:2048\n\t"
                   "ds_read_u8 %6, %13\n\t"
                   "ds_read_u8 %7, %14\n\t"
                   "ds_read_u8 %8, %14 offset:16\n\t"
                   "s_waitcnt lgkmcnt(0)"
                   : "=&v"(bl), "=&v"(bh), "=&v"(al[0]), "=&v"(ah[0]), "=&v"(al[1]), "=&v"(ah[1]), "=&v"(sb), "=&v"(sa[0]), "=&v"(sa[1])
                   : "v"(b_lo + stage), "v"(b_hi + stage), "v"(a_lo + stage), "v"(a_hi + stage), "v"(b_e + stage), "v"(a_e + stage)
                   : "memory");
      free = stage;
      stage = stage + kStreamBytes == kStages * kStreamBytes ? 0 : stage + kStreamBytes;
      const intx8 fb = __builtin_shufflevector(bl, bh, 0, 1, 2, 3, 4, 5, 6, 7);
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const intx8 fa = __builtin_shufflevector(al[i], ah[i], 0, 1, 2, 3, 4, 5, 6, 7);
        if constexpr (F32) {
#pragma unroll
          for (int q = 0; q < 4; ++q) acc[i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(widen<FB>(fb, q, sb), widen<FA>(fa, q, sa[i]), acc[i], 0, 0, 0);
        } else {
          acc[i] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(fb, fa, acc[i], FB, FA, 0, sb, 0, sa[i]);
        }
      }
      if (++done < blocks) continue;
      done = 0;
      // lane l of a block holds c[l % 16][4 (l / 16) + e]
      const int64_t c = here_column * int64_t(64) + wave * 16 + quarter * 4;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int row = here.first + 16 * i + r;
        if (row < here.end)
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (c + e < a.n) store_any(a.c, row * a.ldc + c + e, a.c_dtype, acc[i][e]);
        acc[i] = floatx4{};
      }
      if (++here_column == columns && s + 1 < steps) {
        here_column = 0;
        here = find_tile<32>(a.plan, ++here_tile, lanes);
      }
    }
    WAIT_VM(0);              // the last copies land before the LDS is given up
  }
  zero_tail(a, blockIdx.x, gridDim.x);
}

// The expert with the n-th most rows, so that the longest sums begin first: of up
// to 64 experts; more are taken in their own order, where each is a small part.
__device__ __forceinline__ int nth_largest(const ExpertPlan& p, int n) {
  if (p.n_experts > 64) return n;
  const int lane = threadIdx.x & 63;
  int first = 0, end = 0;
  if (lane < p.n_experts) expert_rows(p, lane, first, end);
  const int rows = lane < p.n_experts ? end - first : -1;
  int rank = 0;
  for (int e = 0; e < p.n_experts; ++e) {
    const int other = __builtin_amdgcn_readlane(rows, e);
    rank += other > rows || (other == rows && e < lane) ? 1 : 0;
  }
  return __builtin_ctzll(__ballot(rank == n && lane < p.n_experts));
}

// The weights' gradients: every expert's (n, k) tiles, summed over its blocks of 128 rows.
// Bound by the matrix cores: 32768 rows of 8 uneven experts x 5632 x 2048 in fp32 take
// 580 to 615 us, 1.23 to 1.3 PFLOP/s (the plain product 1.35; 71 % of a busy CU's cycles
// issue products).  With each expert's tiles on one XCD it took 1379 us.
template <class C, int FA, int FB, bool F32>
__global__ __launch_bounds__(C::NT, 2) void expert_weight_kernel(ExpertMatmulArgs a, unsigned tm, unsigned tn) {
  auto uniform = [](int v) { return __builtin_amdgcn_readfirstlane(v); };
  // each expert's tiles over all XCDs: experts with many tokens would fill one
  const unsigned per = tm * tn, e = nth_largest(a.plan, uniform(blockIdx.x / per)), w = blockIdx.x % per, x = w & 7;
  const unsigned t = x * (per >> 3) + (x < (per & 7) ? x : (per & 7)) + (w >> 3);
  const unsigned band = uniform(t / (8u * tn)), in = t - band * 8u * tn;
  const unsigned high = tm - band * 8 < 8 ? tm - band * 8 : 8, column = uniform(in / high);
  TileJob o;
  o.a_codes = a.a.codes, o.a_scales = a.a.scales, o.b_codes = a.b.codes, o.b_scales = a.b.scales;
  o.lda = a.a.ld, o.lda_scale = a.a.ld_scale, o.ldb = a.b.ld, o.ldb_scale = a.b.ld_scale;
  o.m = a.a.rows, o.n = a.b.rows;
  o.m0 = static_cast<int64_t>(band * 8 + in - column * high) * C::BM, o.n0 = static_cast<int64_t>(column) * C::BN;
  const int first = min(max(a.plan.offsets[e], 0), a.plan.capacity) >> 7, end = min(max(a.plan.offsets[e + 1], 0), a.plan.capacity) >> 7;
  o.k0 = uniform(first), o.nst = uniform(end) - o.k0;
  o.ldc = a.ldc, o.c_dtype = a.c_dtype, o.accumulate = 0;
  const int64_t c_first = e * o.m * o.ldc;
  o.c = static_cast<uint8_t*>(a.c) + c_first * (F32 ? 4 : 2);
  if (o.nst <= 0) {
    for (int i = threadIdx.x; i < C::BM * C::BN; i += C::NT) {
      const int64_t r = o.m0 + i / C::BN, c = o.n0 + i % C::BN;
      if (r < o.m && c < o.n) store_any(o.c, r * o.ldc + c, o.c_dtype, 0.0f);
    }
    return;
  }
  tile_product<C, FA, FB, F32>(o);
}

int bits_of(int n_experts) {
  int b = 0;
  while (1 << b <= n_experts) ++b;      // numbers up to n_experts itself: none
  return b;
}

// choices of a workgroup: whole groups, for at most kPlanBlocks workgroups
int plan_chunk(int64_t pairs) {
  return static_cast<int>(((pairs + kPlanBlocks - 1) / kPlanBlocks + kPlanGroup - 1) / kPlanGroup * kPlanGroup);
}

}  // namespace

size_t plan_workspace(int64_t pairs, int32_t n_experts) {
  if (pairs <= kPlanGroup) return 0;
  const int chunk = plan_chunk(pairs);
  return static_cast<size_t>((pairs + chunk - 1) / chunk) * n_experts * 4;
}

hipError_t launch_plan(const void* choice, bool wide, const ExpertPlan& p, int32_t* ws, hipStream_t s) {
  const int bits = bits_of(p.n_experts);
  const size_t counts = static_cast<size_t>(kPlanWaves) * p.n_experts * 4, offsets = (p.n_experts + 1) * 4;
  auto go = [&](auto w) {
    constexpr bool WIDE = decltype(w)::value;
    if (p.n_pairs <= kPlanGroup) {
      plan_one_kernel<WIDE><<<1, kPlanThreads, counts + offsets, s>>>(choice, p, bits);
      return;
    }
    const int chunk = plan_chunk(p.n_pairs), blocks = (p.n_pairs + chunk - 1) / chunk;
    plan_rank_kernel<WIDE><<<blocks, kPlanThreads, counts + offsets, s>>>(choice, p, bits, chunk, ws);
    plan_place_kernel<WIDE><<<blocks, kPlanThreads, 2 * offsets, s>>>(choice, p, chunk, ws);
  };
  if (wide) go(std::true_type{});
  else go(std::false_type{});
  return hipGetLastError();
}

// waves side by side on a token: as many parts of 512 columns as it has, up to 4.
static int side_by_side(int64_t cols) { return cols > 1024 ? 4 : cols > 512 ? 2 : 1; }

// token groups, and workgroups along a row where there are few tokens
static dim3 token_grid(const RowsArgs& a, int waves, int more) {
  const int each = 4 / waves;
  const int64_t groups = blocks_up_to((a.plan.tokens + each - 1) / each, 1 << 20), parts = (a.cols + waves * 512 - 1) / (waves * 512), want = 1024 / (groups + 1) + 1;
  return dim3(static_cast<unsigned>(groups) + more, static_cast<unsigned>(parts < want ? parts : want));
}

// calls go(choices that a wave takes at a time)
template <class F>
static void by_each(int each, F go) {
  if (each <= 2) go(std::integral_constant<int, 2>{});
  else if (each <= 4) go(std::integral_constant<int, 4>{});
  else go(std::integral_constant<int, 8>{});
}

hipError_t launch_gather(const RowsArgs& a, hipStream_t s) {
  const int waves = side_by_side(a.cols);
  by_type(a.dtype, [&](auto type) { gather_kernel<decltype(type)><<<token_grid(a, waves, kZeroGroups), 256, 0, s>>>(a, waves); });
  return hipGetLastError();
}

hipError_t launch_combine(const RowsArgs& a, hipStream_t s) {
  const int waves = side_by_side(a.cols);
  by_type(a.dtype, [&](auto type) {
    by_each(a.plan.each, [&](auto g) { combine_kernel<decltype(type), decltype(g)::value><<<token_grid(a, waves, 0), 256, 0, s>>>(a, waves); });
  });
  return hipGetLastError();
}

hipError_t launch_combine_backward(const RowsArgs& a, hipStream_t s) {
  const int waves = side_by_side(a.cols), each = 4 / waves;
  const int groups = blocks_up_to((a.plan.tokens + each - 1) / each, 1 << 20);
  by_type(a.dtype, [&](auto type) {
    by_each(a.plan.each, [&](auto g) { combine_backward_kernel<decltype(type), decltype(g)::value><<<groups + kZeroGroups, 256, 0, s>>>(a, waves); });
  });
  return hipGetLastError();
}

// Which kernel, by the rows of an expert on average; measured with four sets of
// weights in turn (us, stream / narrow / small / big tiles, 16-bit results):
//  - 8 experts of 11008 x 4096: 4 rows 75 / 84 / 98, 16 rows 81 / 86 / 98, 64 rows 189 /
//    114 / 103 / 118, 256 rows 646 / 192 / 165 / 180, 512 rows - / 298 / 263 / 228.
//  - 64 experts of 2816 x 1024: 4 rows 43 / 41 / 44, 32 rows 70 / 44 / 46 / 57, 128 rows
//    207 / 71 / 66 / 61, 512 rows - / 218 / 181 / 146.
//  - 8 experts of 2048 x 5632: 32 rows 33 / 42 / 44 / 70 (128 narrow tiles leave half of the
//    card idle; a stream's share is even), 128 rows 102 / 50 / 49 / 73, 512 rows - / 97 /
//    98 / 80.
hipError_t launch_expert_matmul(const ExpertMatmulArgs& a, hipStream_t s) {
  if (a.a.cols == 0) {
    zero_kernel<<<blocks_up_to((a.plan.capacity * a.n + 255) / 256, 4096), 256, 0, s>>>(a.c, a.c_dtype, a.plan.capacity, a.n, a.ldc);
    return hipGetLastError();
  }
  const ExpertPlan& p = a.plan;
  const int64_t some = p.n_pairs < p.n_experts ? p.n_pairs : p.n_experts, each = p.n_pairs / some;   // experts with rows, their rows on average
  // about how many tiles there are: every expert's last one is half full
  auto count = [&](int bm, int bn) { return (p.n_pairs / bm + (some + 1) / 2) * ((a.n + bn - 1) / bn); };
  by_format(a.a.format, a.b.format, a.c_dtype, [&](auto fa, auto fb, auto f32) {
    constexpr int FA = decltype(fa)::value, FB = decltype(fb)::value;
    constexpr bool F32 = decltype(f32)::value;
    auto tiles = [&](auto tile) {
      using C = decltype(tile);
      const unsigned tn = static_cast<unsigned>((a.n + C::BN - 1) / C::BN);
      expert_tile_kernel<C, FA, FB, F32><<<most_tiles(p, C::BM) * tn + kTailGroups, C::NT, 0, s>>>(a, tn, C::NW == 8 && a.a.cols >= kLongSum);
    };
    if (each <= 8 || (each <= 32 && count(64, 128) < 200)) {
      const int64_t units = most_tiles(p, 32) * ((a.n + 63) / 64);
      expert_stream_kernel<FA, FB, F32><<<blocks_up_to(units, kStreamGroups), 256, 0, s>>>(a);
    } else if (each < 64) {
      tiles(TileNarrow{});
    } else if (each < 128 || count(256, 256) < 160) {
      tiles(TileSmall{});
    } else {
      tiles(TileBig{});
      if (a.a.cols >= kLongSum) expert_rest_kernel<FA, FB, F32><<<4 * (kRound / 2), TileSmall::NT, 0, s>>>(a, static_cast<unsigned>((a.n + TileBig::BN - 1) / TileBig::BN));
    }
  });
  return hipGetLastError();
}

hipError_t launch_expert_weight_grad(const ExpertMatmulArgs& a, hipStream_t s) {
  const int64_t m = a.a.rows, n = a.b.rows;
  by_format(a.a.format, a.b.format, a.c_dtype, [&](auto fa, auto fb, auto f32) {
    constexpr int FA = decltype(fa)::value, FB = decltype(fb)::value;
    constexpr bool F32 = decltype(f32)::value;
    auto tiles = [&](auto tile) {
      using C = decltype(tile);
      const unsigned tm = static_cast<unsigned>((m + C::BM - 1) / C::BM), tn = static_cast<unsigned>((n + C::BN - 1) / C::BN);
      expert_weight_kernel<C, FA, FB, F32><<<tm * tn * a.plan.n_experts, C::NT, 0, s>>>(a, tm, tn);
    };
    // the larger tile where there are enough of them, as in the plain product
    if (m > 128 && n > 128 && ((m + 255) / 256) * ((n + 255) / 256) * a.plan.n_experts >= 160) tiles(TileBig{});
    else tiles(TileSmall{});
  });
  return hipGetLastError();
}

}  // namespace okls
