// gfx950 kernels of the experts' operators (okls_experts.h).
//
//  plan_kernel and its parts   a stable counting sort of choices by expert.
//  gather / combine kernels    tokens' rows to the sorted order and back.
//  expert tile / few kernels   the products of product_tile.h, each tile of the
//                              sorted rows with its own expert's matrix.
#include "experts_kernels.h"
#include "product_tile.h"

#include "../../include/okls_experts.h"

namespace okls {
namespace {

// ---------------------------------------------------------------------------
// The sorted order
// ---------------------------------------------------------------------------
// A stable counting sort.  Each wave ranks a run of choices of its own, 64 at a
// time: lanes with the same expert find each other by one ballot for each bit
// of its number, the count so far is the wave's own in LDS.  Then the counts of
// waves (and workgroups) before it are added.
constexpr int kPlanThreads = 1024, kPlanWaves = kPlanThreads / 64;
constexpr int kPlanOne = 16384;         // choices that one workgroup sorts alone
constexpr int kPlanChunk = 4096;        // of a workgroup otherwise, more where that would be over 1024 of them

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

// rows[i] = the number of choices of the same expert before i among this wave's
// [first, last); count[e] (LDS, the wave's own) = their number
template <bool WIDE>
__device__ void rank_wave(const void* choice, int first, int last, int n_experts, int bits, int* count, int32_t* rows) {
  const int lane = threadIdx.x & 63;
  for (int i0 = first; i0 < last; i0 += 64) {
    const int i = i0 + lane;
    const int e = i < last ? choice_at<WIDE>(choice, i, n_experts) : n_experts;
    uint64_t same = ~uint64_t(0);
    for (int b = 0; b < bits; ++b) {
      const uint64_t set = __ballot(e >> b & 1);
      same &= e >> b & 1 ? set : ~set;
    }
    const int before = __popcll(same & ((uint64_t(1) << lane) - 1));
    const int seen = e < n_experts ? count[e] : 0;
    // every lane has read its expert's count before the group's first lane moves it
    __builtin_amdgcn_wave_barrier();
    if (e < n_experts && before == 0) count[e] = seen + __popcll(same);
    __builtin_amdgcn_wave_barrier();
    if (i < last) rows[i] = seen + before;
  }
}

// each wave's counts become the counts of the waves before it; returns expert t's total in thread t
__device__ int scan_waves(int* count, int n_experts) {
  const int t = threadIdx.x;
  int total = 0;
  if (t < n_experts)
    for (int w = 0; w < kPlanWaves; ++w) {
      const int c = count[w * n_experts + t];
      count[w * n_experts + t] = total;
      total += c;
    }
  return total;
}

// offsets from the experts' totals (thread t's), in LDS (n_experts + 1) and memory
__device__ void write_offsets(int total, const ExpertPlan& p, int* offset) {
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
    p.offsets[t] = room - own;
    p.counts[t] = total;
    if (t == p.n_experts - 1) {
      offset[t + 1] = room;
      p.offsets[t + 1] = room;
    }
  }
  __syncthreads();
}

__device__ __forceinline__ int wave_run(int n) { return ((n + kPlanWaves - 1) / kPlanWaves + 63) / 64 * 64; }

// all of it in one workgroup
template <bool WIDE>
__global__ __launch_bounds__(kPlanThreads) void plan_one_kernel(const void* choice, ExpertPlan p, int bits) {
  extern __shared__ int lds[];            // kPlanWaves x n_experts counts, n_experts + 1 offsets
  int* offset = lds + kPlanWaves * p.n_experts;
  const int t = threadIdx.x, wave = t >> 6, run = wave_run(p.n_pairs);
  const int first = min(wave * run, p.n_pairs), last = min(first + run, p.n_pairs);
  for (int i = t; i < kPlanWaves * p.n_experts; i += kPlanThreads) lds[i] = 0;
  for (int r = t; r < p.capacity; r += kPlanThreads) p.pairs[r] = -1;
  __syncthreads();
  rank_wave<WIDE>(choice, first, last, p.n_experts, bits, lds + wave * p.n_experts, p.rows);
  __syncthreads();
  const int total = scan_waves(lds, p.n_experts);
  write_offsets(total, p, offset);
  for (int i = first + (t & 63); i < last; i += 64) {
    const int e = choice_at<WIDE>(choice, i, p.n_experts);
    const int row = e < p.n_experts ? offset[e] + lds[wave * p.n_experts + e] + p.rows[i] : -1;
    p.rows[i] = row;
    if (row >= 0) p.pairs[row] = i;
  }
}

// a chunk of choices a workgroup: ranks within it, and its counts (workgroup, expert)
template <bool WIDE>
__global__ __launch_bounds__(kPlanThreads) void plan_rank_kernel(const void* choice, ExpertPlan p, int bits, int chunk, int32_t* counts) {
  extern __shared__ int lds[];
  const int t = threadIdx.x, wave = t >> 6, run = wave_run(chunk);
  const int begin = blockIdx.x * chunk, end = min(begin + chunk, p.n_pairs);
  const int first = min(begin + wave * run, end), last = min(first + run, end);
  for (int i = t; i < kPlanWaves * p.n_experts; i += kPlanThreads) lds[i] = 0;
  __syncthreads();
  rank_wave<WIDE>(choice, first, last, p.n_experts, bits, lds + wave * p.n_experts, p.rows);
  __syncthreads();
  const int total = scan_waves(lds, p.n_experts);
  if (t < p.n_experts) counts[static_cast<int64_t>(blockIdx.x) * p.n_experts + t] = total;
  __syncthreads();
  for (int i = first + (t & 63); i < last; i += 64) {
    const int e = choice_at<WIDE>(choice, i, p.n_experts);
    if (e < p.n_experts) p.rows[i] += lds[wave * p.n_experts + e];
  }
}

// the workgroups' counts become the first rows of their choices
__global__ __launch_bounds__(kPlanThreads) void plan_scan_kernel(ExpertPlan p, int32_t* counts, int blocks) {
  extern __shared__ int lds[];
  const int t = threadIdx.x;
  int total = 0;
  if (t < p.n_experts)
    for (int b = 0; b < blocks; ++b) {
      int32_t& c = counts[static_cast<int64_t>(b) * p.n_experts + t];
      const int own = c;
      c = total;
      total += own;
    }
  write_offsets(total, p, lds);
  if (t < p.n_experts)
    for (int b = 0; b < blocks; ++b) counts[static_cast<int64_t>(b) * p.n_experts + t] += lds[t];
}

template <bool WIDE>
__global__ __launch_bounds__(256) void plan_place_kernel(const void* choice, ExpertPlan p, int chunk, const int32_t* counts) {
  const int n = gridDim.x * 256, t = blockIdx.x * 256 + threadIdx.x;
  for (int64_t i = t; i < p.n_pairs; i += n) {
    const int e = choice_at<WIDE>(choice, static_cast<int>(i), p.n_experts);
    const int row = e < p.n_experts ? p.rows[i] + counts[i / chunk * p.n_experts + e] : -1;
    p.rows[i] = row;
    if (row >= 0) p.pairs[row] = static_cast<int>(i);
  }
  // rows without a choice: behind each expert's, and behind the last one
  for (int e = blockIdx.x; e < p.n_experts; e += gridDim.x)
    for (int r = p.offsets[e] + p.counts[e] + threadIdx.x; r < p.offsets[e + 1]; r += 256) p.pairs[r] = -1;
  for (int64_t r = static_cast<int64_t>(p.offsets[p.n_experts]) + t; r < p.capacity; r += n) p.pairs[r] = -1;
}

// ---------------------------------------------------------------------------
// Rows to the sorted order and back
// ---------------------------------------------------------------------------
// A token's row by a wave, its parts of 512 columns by gridDim.y waves in turn.
// Tokens lead in every direction: a token's row is read (written) once for all
// its choices.  Workgroups behind the tokens' write the zeros of rows without a choice.
constexpr int kZeroGroups = 64;

// a choice's row, -1 for none; the same for the whole wave
__device__ __forceinline__ int row_of(const ExpertPlan& p, int64_t token, int k) {
  const int r = __builtin_amdgcn_readfirstlane(p.rows[token * p.each + k]);
  return r < p.capacity ? r : -1;
}

// zeros in the rows without a choice, by wave `wave` of `waves`
template <typename T>
__device__ void zero_rows(const ExpertPlan& p, T* out, int64_t ldo, int64_t cols, int wave, int waves) {
  const int lane = threadIdx.x & 63;
  const float zeros[8] = {};
  auto clear = [&](int64_t r) {
    for (int64_t c = lane * 8; c < cols; c += 512) store8(out + r * ldo + c, zeros, clamp8(cols - c));
  };
  for (int e = wave; e < p.n_experts; e += waves) {
    const int end = min(p.offsets[e + 1], p.capacity);
    for (int r = max(p.offsets[e] + p.counts[e], 0); r < end; ++r) clear(r);
  }
  for (int64_t r = static_cast<int64_t>(max(p.offsets[p.n_experts], 0)) + wave; r < p.capacity; r += waves) clear(r);
}

template <typename T>
__global__ __launch_bounds__(256) void gather_kernel(RowsArgs a, int groups) {
  const ExpertPlan& p = a.plan;
  T* out = static_cast<T*>(a.out);
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  if (static_cast<int>(blockIdx.x) >= groups) {
    const int z = ((blockIdx.x - groups) * gridDim.y + blockIdx.y) * 4 + wave;
    zero_rows(p, out, a.ldo, a.cols, z, (gridDim.x - groups) * gridDim.y * 4);
    return;
  }
  const T* x = static_cast<const T*>(a.x);
  for (int64_t t = blockIdx.x * 4 + wave; t < p.tokens; t += groups * 4)
    for (int64_t c = (blockIdx.y * 64 + lane) * 8; c < a.cols; c += gridDim.y * 512) {
      const int n = clamp8(a.cols - c);
      float v[8];
      load8(v, x + t * a.ldx + c, n);
      for (int k = 0; k < p.each; ++k) {
        const int r = row_of(p, t, k);
        if (r >= 0) store8(out + r * a.ldo + c, v, n);
      }
    }
}

template <typename T>
__global__ __launch_bounds__(256) void combine_kernel(RowsArgs a) {
  const ExpertPlan& p = a.plan;
  const T* y = static_cast<const T*>(a.y);
  T* out = static_cast<T*>(a.out);
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  for (int64_t t = blockIdx.x * 4 + wave; t < p.tokens; t += gridDim.x * 4)
    for (int64_t c = (blockIdx.y * 64 + lane) * 8; c < a.cols; c += gridDim.y * 512) {
      const int n = clamp8(a.cols - c);
      float s[8] = {};
      for (int k = 0; k < p.each; ++k) {
        const int r = row_of(p, t, k);
        if (r < 0) continue;
        const float w = a.weights != nullptr ? load_any(a.weights, t * p.each + k, a.weight_dtype) : 1.0f;
        float v[8];
        load8(v, y + r * a.ldy + c, n);
#pragma unroll
        for (int j = 0; j < 8; ++j) s[j] = fmaf(w, v[j], s[j]);
      }
      store8(out + t * a.ldo + c, s, n);
    }
}

// dy and dweights: a token's choices in groups of 4, whose sums stay in registers
template <typename T>
__global__ __launch_bounds__(256) void combine_backward_kernel(RowsArgs a, int groups) {
  const ExpertPlan& p = a.plan;
  T* out = static_cast<T*>(a.out);
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  if (static_cast<int>(blockIdx.x) >= groups) {
    zero_rows(p, out, a.ldo, a.cols, (blockIdx.x - groups) * 4 + wave, (gridDim.x - groups) * 4);
    return;
  }
  const T* d = static_cast<const T*>(a.x);
  const T* y = static_cast<const T*>(a.y);
  for (int64_t t = blockIdx.x * 4 + wave; t < p.tokens; t += groups * 4)
    for (int k0 = 0; k0 < p.each; k0 += 4) {
      int row[4];
      float w[4], sum[4] = {};
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        row[q] = k0 + q < p.each ? row_of(p, t, k0 + q) : -1;
        w[q] = row[q] >= 0 ? load_any(a.weights, t * p.each + k0 + q, a.weight_dtype) : 0.0f;
      }
      for (int64_t c = lane * 8; c < a.cols; c += 512) {
        const int n = clamp8(a.cols - c);
        float g[8];
        load8(g, d + t * a.ldx + c, n);
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          if (row[q] < 0) continue;
          float v[8];
          load8(v, y + row[q] * a.ldy + c, n);
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            sum[q] = fmaf(g[j], v[j], sum[q]);
            v[j] = w[q] * g[j];
          }
          store8(out + row[q] * a.ldo + c, v, n);
        }
      }
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        float s = sum[q];
#pragma unroll
        for (int o = 32; o > 0; o >>= 1) s += __shfl_xor(s, o, 64);
        if (lane == 0 && k0 + q < p.each) store_any(a.dweights, t * p.each + k0 + q, a.weight_dtype, s);
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

// this lane's expert's tiles, and the sum over it and the lanes before it
template <int BM>
__device__ __forceinline__ int tiles_up_to(const ExpertPlan& p, int e) {
  int n = 0;
  if (e < p.n_experts) {
    int first, end;
    expert_rows(p, e, first, end);
    n = (end - first + BM - 1) / BM;
  }
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) {
    const int other = __shfl_up(n, o, 64);
    if ((threadIdx.x & 63) >= static_cast<unsigned>(o)) n += other;
  }
  return n;
}

template <int BM>
__device__ __forceinline__ int count_tiles(const ExpertPlan& p) {
  int total = 0;
  for (int e0 = 0; e0 < p.n_experts; e0 += 64) total += __shfl(tiles_up_to<BM>(p, e0 + (threadIdx.x & 63)), 63, 64);
  return __builtin_amdgcn_readfirstlane(total);
}

// tile t < count_tiles
template <int BM>
__device__ __forceinline__ TileRows find_tile(const ExpertPlan& p, int t) {
  int before = 0;
  TileRows r{0, 0, 0};
  for (int e0 = 0; e0 < p.n_experts; e0 += 64) {
    const int upto = tiles_up_to<BM>(p, e0 + (threadIdx.x & 63)) + before, all = __shfl(upto, 63, 64);
    if (t < all) {
      const int lane = __popcll(__ballot(upto <= t));     // experts that end at or before t
      const int begin = lane == 0 ? before : __shfl(upto, lane - 1, 64);
      r.expert = __builtin_amdgcn_readfirstlane(e0 + lane);
      expert_rows(p, r.expert, r.first, r.end);
      r.first = __builtin_amdgcn_readfirstlane(r.first + (t - begin) * BM);
      r.end = __builtin_amdgcn_readfirstlane(r.end);
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

// workgroup j of n: zeros in c's rows behind the last expert's
__device__ void zero_tail(const ExpertMatmulArgs& a, int64_t j, int64_t n) {
  for (int64_t r = min(max(a.plan.offsets[a.plan.n_experts], 0), a.plan.capacity) + j; r < a.plan.capacity; r += n)
    for (int64_t c = threadIdx.x; c < a.n; c += blockDim.x) store_any(a.c, r * a.ldc + c, a.c_dtype, 0.0f);
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

template <class C, int FA, int FB, bool F32>
__global__ __launch_bounds__(C::NT, 2) void expert_tile_kernel(ExpertMatmulArgs a, unsigned tn) {
  auto uniform = [](int v) { return __builtin_amdgcn_readfirstlane(v); };
  const unsigned tm = count_tiles<C::BM>(a.plan), total = tm * tn, w = blockIdx.x, x = w & 7;
  if (w >= total) return zero_tail(a, w - total, gridDim.x - total);
  // as in the plain product: each XCD takes a run of neighbouring tiles in bands of 8 tile rows
  const unsigned t = x * (total >> 3) + (x < (total & 7) ? x : (total & 7)) + (w >> 3);
  const unsigned band = uniform(t / (8u * tn)), in = t - band * 8u * tn;
  const unsigned high = tm - band * 8 < 8 ? tm - band * 8 : 8, column = uniform(in / high);
  TileJob o = expert_job(a, find_tile<C::BM>(a.plan, band * 8 + in - column * high));
  o.n0 = static_cast<int64_t>(column) * C::BN;
  tile_product<C, FA, FB, F32>(o);
}

template <int TM, int TN, int FA, int FB, bool F32>
__global__ __launch_bounds__(kFewWaves * 64) void expert_few_kernel(ExpertMatmulArgs a) {
  const int tm = count_tiles<16 * TM>(a.plan);
  if (static_cast<int>(blockIdx.y) >= tm)
    return zero_tail(a, static_cast<int64_t>(blockIdx.y - tm) * gridDim.x + blockIdx.x, static_cast<int64_t>(gridDim.y - tm) * gridDim.x);
  TileJob o = expert_job(a, find_tile<16 * TM>(a.plan, blockIdx.y));
  o.n0 = static_cast<int64_t>(blockIdx.x) * (16 * TN);
  few_product<TM, TN, FA, FB, F32>(o);
}

// The weights' gradients: every expert's (n, k) tiles, summed over its blocks of 128 rows.
template <class C, int FA, int FB, bool F32>
__global__ __launch_bounds__(C::NT, 2) void expert_weight_kernel(ExpertMatmulArgs a, unsigned tm, unsigned tn) {
  auto uniform = [](int v) { return __builtin_amdgcn_readfirstlane(v); };
  const unsigned per = tm * tn, total = per * a.plan.n_experts, w = blockIdx.x, x = w & 7;
  const unsigned id = x * (total >> 3) + (x < (total & 7) ? x : (total & 7)) + (w >> 3);
  const unsigned e = uniform(id / per), t = id - e * per;
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

__global__ __launch_bounds__(256) void zero_matrix_kernel(void* c, int dtype, int64_t m, int64_t n, int64_t ldc) {
  for (int64_t i = blockIdx.x * 256ll + threadIdx.x; i < m * n; i += gridDim.x * 256ll) store_any(c, i / n * ldc + i % n, dtype, 0.0f);
}

int bits_of(int n_experts) {
  int b = 0;
  while (1 << b <= n_experts) ++b;      // numbers up to n_experts itself: none
  return b;
}

int plan_chunk(int64_t pairs) {
  const int64_t most = (pairs + 1023) / 1024;
  return static_cast<int>(most <= kPlanChunk ? kPlanChunk : (most + kPlanChunk - 1) / kPlanChunk * kPlanChunk);
}

}  // namespace

size_t plan_workspace(int64_t pairs, int32_t n_experts) {
  if (pairs <= kPlanOne) return 0;
  const int chunk = plan_chunk(pairs);
  return static_cast<size_t>((pairs + chunk - 1) / chunk) * n_experts * 4;
}

hipError_t launch_plan(const void* choice, bool wide, const ExpertPlan& p, int32_t* ws, hipStream_t s) {
  const int bits = bits_of(p.n_experts);
  const size_t counts = static_cast<size_t>(kPlanWaves) * p.n_experts * 4, offsets = (p.n_experts + 1) * 4;
  auto go = [&](auto w) {
    constexpr bool WIDE = decltype(w)::value;
    if (p.n_pairs <= kPlanOne) {
      plan_one_kernel<WIDE><<<1, kPlanThreads, counts + offsets, s>>>(choice, p, bits);
      return;
    }
    const int chunk = plan_chunk(p.n_pairs), blocks = (p.n_pairs + chunk - 1) / chunk;
    plan_rank_kernel<WIDE><<<blocks, kPlanThreads, counts, s>>>(choice, p, bits, chunk, ws);
    plan_scan_kernel<<<1, kPlanThreads, offsets, s>>>(p, ws, blocks);
    plan_place_kernel<WIDE><<<blocks_up_to((p.n_pairs + 255) / 256, 2048), 256, 0, s>>>(choice, p, chunk, ws);
  };
  if (wide) go(std::true_type{});
  else go(std::false_type{});
  return hipGetLastError();
}

// token groups, and parts of a row's columns where there are few tokens
static dim3 token_grid(int64_t tokens, int64_t cols, int more, int& groups) {
  groups = blocks_up_to((tokens + 3) / 4, 1 << 20);
  const int64_t parts = (cols + 511) / 512, want = 1024 / (groups + 1) + 1;
  return dim3(groups + more, static_cast<unsigned>(parts < want ? parts : want));
}

hipError_t launch_gather(const RowsArgs& a, hipStream_t s) {
  int groups;
  const dim3 grid = token_grid(a.plan.tokens, a.cols, kZeroGroups, groups);
  by_type(a.dtype, [&](auto type) { gather_kernel<decltype(type)><<<grid, 256, 0, s>>>(a, groups); });
  return hipGetLastError();
}

hipError_t launch_combine(const RowsArgs& a, hipStream_t s) {
  int groups;
  const dim3 grid = token_grid(a.plan.tokens, a.cols, 0, groups);
  by_type(a.dtype, [&](auto type) { combine_kernel<decltype(type)><<<grid, 256, 0, s>>>(a); });
  return hipGetLastError();
}

hipError_t launch_combine_backward(const RowsArgs& a, hipStream_t s) {
  const int groups = blocks_up_to((a.plan.tokens + 3) / 4, 1 << 20);
  by_type(a.dtype, [&](auto type) { combine_backward_kernel<decltype(type)><<<groups + kZeroGroups, 256, 0, s>>>(a, groups); });
  return hipGetLastError();
}

hipError_t launch_expert_matmul(const ExpertMatmulArgs& a, hipStream_t s) {
  if (a.a.cols == 0) {
    zero_matrix_kernel<<<blocks_up_to((a.plan.capacity * a.n + 255) / 256, 4096), 256, 0, s>>>(a.c, a.c_dtype, a.plan.capacity, a.n, a.ldc);
    return hipGetLastError();
  }
  const ExpertPlan& p = a.plan;
  const int64_t each = p.n_pairs / (p.n_pairs < p.n_experts ? p.n_pairs : p.n_experts);   // rows of an expert, on average
  by_format(a.a.format, a.b.format, a.c_dtype, [&](auto fa, auto fb, auto f32) {
    constexpr int FA = decltype(fa)::value, FB = decltype(fb)::value;
    constexpr bool F32 = decltype(f32)::value;
    auto tiles = [&](auto tile) {
      using C = decltype(tile);
      const unsigned tn = static_cast<unsigned>((a.n + C::BN - 1) / C::BN);
      expert_tile_kernel<C, FA, FB, F32><<<most_tiles(p, C::BM) * tn + kTailGroups, C::NT, 0, s>>>(a, tn);
    };
    if (each <= 16) expert_few_kernel<1, 1, FA, FB, F32><<<dim3(static_cast<unsigned>((a.n + 15) / 16), most_tiles(p, 16) + 1), kFewWaves * 64, 0, s>>>(a);
    else if (each <= 256) tiles(TileSmall{});
    else tiles(TileBig{});
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
    if (m > 128 && n > 128) tiles(TileBig{});
    else tiles(TileSmall{});
  });
  return hipGetLastError();
}

}  // namespace okls
