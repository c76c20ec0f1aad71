// bsq_expert.cu -- tokens sorted by expert and back.
//
// A router names topk experts for each token. Slot i = token * topk + j of those n choices becomes a
// row of a matrix in which every expert's rows are consecutive, in slot order (a stable counting
// sort), and begin at a multiple of `align` (128 puts every expert on scale tiles of its own, so
// that its rows are an operand of bsq_gemm by themselves):
//   offsets[e+1] = offsets[e] + ceil(counts[e] / align) * align,
//   position[i] = offsets[e_i] + |{i' < i: e_i' = e_i}|, slot[position[i]] = i, slot[other rows] = -1.
// An id outside [0, experts) is a dropped choice: position -1, no row.
//   gather            rows[r] = x[slot[r] / topk], zeros where slot[r] < 0
//   combine           out[t] = sum_j weights[t, j] * y[position[t, j]]  (weights 1 where there are
//                     none: the gradient of gather)
//   combine backward  dy[r] = weights[slot[r]] * dout[slot[r] / topk], zeros where slot[r] < 0;
//                     dweights[t, j] = <dout[t], y[position[t, j]]>, 0 for a dropped choice
// Nothing here uses atomics whose order could change a result. All are bound by the bytes of the
// matrices, small calls by launch latency.
#include <algorithm>
#include <type_traits>

#include "bsq.h"
#include "bsq_device.cuh"
#include "bsq_elem.cuh"
#include "bsq_internal.h"

namespace bsq {
namespace {

// ---------------------------------------------------------------- sort
// Chunks of slots, one a CTA. The CTAs need each other's counts: up to kSortCluster chunks form a
// cluster and read them from each other's shared memory, more are counted by a launch of their own
// (14336 slots of 16 experts: 7.7 us in a cluster, 13.5 us in two launches).
constexpr int kSortWarps = 8;
constexpr int kSortThreads = kSortWarps * 32;
constexpr int kSortTile = 8;             // groups of 32 slots whose ids a warp loads at once
constexpr int64_t kSortChunk = 2048;     // slots of a CTA, unless that makes more CTAs than
constexpr int64_t kSortMaxChunks = 296;  // this many, each of which reads every chunk's counts
constexpr int kSortCluster = 8;

struct SortParams {
  const void* ids;
  bool ids64;
  int32_t experts;
  int64_t slots, chunk, capacity;  // chunk: slots of a CTA, a multiple of kSortThreads
  int32_t chunks, align;
  int32_t* hist;  // [chunks][experts], more chunks than a cluster only
  int32_t *counts, *offsets, *position, *slot;
};

// The CTA's slots are cut into one consecutive range for each warp, walked in tiles of kSortTile
// groups of 32 slots; f(slot, expert or -1, peers, inside the range) is called by every lane for each
// group, peers = the lanes with the same expert. `ids` keeps the first tile, which is all of a range
// unless the slots are very many.
struct SortRange {
  int64_t begin, end;
  int ids[kSortTile];
};
__device__ __forceinline__ void load_tile(const SortParams& a, const SortRange& r, int64_t at, int (&ids)[kSortTile]) {
#pragma unroll
  for (int k = 0; k < kSortTile; ++k) {
    const int64_t i = at + 32 * k + lane_id();
    int64_t e = -1;
    if (i < r.end)
      e = a.ids64 ? __ldcg(static_cast<const long long*>(a.ids) + i) : __ldcg(static_cast<const int32_t*>(a.ids) + i);
    ids[k] = e >= 0 && e < a.experts ? static_cast<int>(e) : -1;
  }
}
template <typename F>
__device__ __forceinline__ void walk_tile(const SortRange& r, int64_t at, const int (&ids)[kSortTile], F&& f) {
#pragma unroll
  for (int k = 0; k < kSortTile; ++k) {
    const int64_t i = at + 32 * k;
    if (i >= r.end) break;
    f(i + lane_id(), ids[k], __match_any_sync(0xffffffffu, ids[k]), i + lane_id() < r.end);
  }
}
template <typename F>
__device__ __forceinline__ void for_slots(const SortParams& a, const SortRange& r, F&& f) {
  if (r.begin >= r.end) return;
  walk_tile(r, r.begin, r.ids, f);
  for (int64_t at = r.begin + 32 * kSortTile; at < r.end; at += 32 * kSortTile) {
    int ids[kSortTile];
    load_tile(a, r, at, ids);
    walk_tile(r, at, ids, f);
  }
}
__device__ __forceinline__ SortRange sort_range(const SortParams& a) {
  SortRange r;
  const int64_t begin = static_cast<int64_t>(blockIdx.x) * a.chunk, end = min(a.slots, begin + a.chunk);
  const int64_t per = a.chunk / kSortWarps;
  r.begin = begin + (threadIdx.x >> 5) * per;
  r.end = min(end, r.begin + per);
  load_tile(a, r, r.begin, r.ids);
  return r;
}
// Counts of each warp's slots, [warps][experts] in shared memory.
__device__ __forceinline__ void count_slots(const SortParams& a, const SortRange& r, int32_t* sh) {
  for (int i = threadIdx.x; i < kSortWarps * a.experts; i += kSortThreads) sh[i] = 0;
  __syncthreads();
  int32_t* mine = sh + (threadIdx.x >> 5) * a.experts;
  for_slots(a, r, [&](int64_t, int e, uint32_t peers, bool) {
    if (e >= 0 && lane_id() == static_cast<uint32_t>(__ffs(static_cast<int>(peers)) - 1)) mine[e] += __popc(peers);
    __syncwarp();
  });
  __syncthreads();
}

__global__ void __launch_bounds__(kSortThreads) expert_count_kernel(const SortParams a) {
  extern __shared__ int32_t sh[];
  // in this order: what is launched from here on starts behind everything before this kernel
  grid_dependency_wait();
  launch_dependents();
  const SortRange r = sort_range(a);
  count_slots(a, r, sh);
  for (int e = threadIdx.x; e < a.experts; e += kSortThreads) {
    int32_t s = 0;
    for (int w = 0; w < kSortWarps; ++w) s += sh[w * a.experts + e];
    a.hist[static_cast<int64_t>(blockIdx.x) * a.experts + e] = s;
  }
}

// HOW: how the other chunks' counts come -- there are none, by the cluster, or by expert_count_kernel.
enum SortHow { kOneChunk, kCluster, kCounted };

template <int HOW>
__global__ void __launch_bounds__(kSortThreads) expert_place_kernel(const SortParams a) {
  // [warps][experts] counts, then rows already taken; [experts] totals; [experts + 1] offsets
  extern __shared__ int32_t sh[];
  int32_t* total = sh + kSortWarps * a.experts;
  int32_t* offset = total + a.experts;
  __shared__ int32_t warp_sums[kSortWarps];
  const int warp = threadIdx.x >> 5;
  // expert_place_kernel<kCounted> starts behind the writers of the ids (see expert_count_kernel) and waits for
  // the counts below: 524288 slots 23 us, 45 us when it waits here
  if constexpr (HOW != kCounted) enter_stream();
  const SortRange r = sort_range(a);
  count_slots(a, r, sh);
  if constexpr (HOW == kCluster) {  // `offset` holds the chunk's own counts until all have read them
    for (int e = threadIdx.x; e < a.experts; e += kSortThreads) {
      int32_t n = 0;
      for (int w = 0; w < kSortWarps; ++w) n += sh[w * a.experts + e];
      offset[e] = n;
    }
    cluster_barrier();
  }
  if constexpr (HOW == kCounted) enter_stream();
  // totals over all chunks, and the rows that earlier chunks and warps take of each expert
  for (int e = threadIdx.x; e < a.experts; e += kSortThreads) {
    int32_t before = 0, sum = 0;
    if constexpr (HOW == kCounted) {
#pragma unroll 16
      for (int c = 0; c < a.chunks; ++c) {
        const int32_t n = a.hist[static_cast<int64_t>(c) * a.experts + e];
        sum += n;
        before += c < static_cast<int>(blockIdx.x) ? n : 0;
      }
    } else if constexpr (HOW == kCluster) {
#pragma unroll
      for (int c = 0; c < kSortCluster; ++c) {
        if (c >= a.chunks) break;
        uint32_t at;
        int32_t n;
        asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(smem_u32(offset + e)), "r"(c));
        asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(n) : "r"(at) : "memory");
        sum += n;
        before += c < static_cast<int>(blockIdx.x) ? n : 0;
      }
    } else {
      for (int w = 0; w < kSortWarps; ++w) sum += sh[w * a.experts + e];
    }
    total[e] = sum;
    int32_t run = before;
    for (int w = 0; w < kSortWarps; ++w) {
      const int32_t n = sh[w * a.experts + e];
      sh[w * a.experts + e] = run;
      run += n;
    }
  }
  if constexpr (HOW == kCluster) cluster_barrier();  // the counts in `offset` are read no more
  else __syncthreads();
  // exclusive scan of the padded totals: a run of consecutive experts for each thread
  const int per = (a.experts + kSortThreads - 1) / kSortThreads;
  const int e0 = min(a.experts, static_cast<int>(threadIdx.x) * per), e1 = min(a.experts, e0 + per);
  int32_t own = 0;
  for (int e = e0; e < e1; ++e) own += (total[e] + a.align - 1) / a.align * a.align;
  int32_t scan = own;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int32_t v = __shfl_up_sync(0xffffffffu, scan, d);
    if (lane_id() >= static_cast<uint32_t>(d)) scan += v;
  }
  if (lane_id() == 31) warp_sums[warp] = scan;
  __syncthreads();
  int32_t run = scan - own;
  for (int w = 0; w < warp; ++w) run += warp_sums[w];
  for (int e = e0; e < e1; ++e) {
    offset[e] = run;
    run += (total[e] + a.align - 1) / a.align * a.align;
  }
  if (e1 == a.experts && e0 < e1) offset[a.experts] = run;
  __syncthreads();
  if (blockIdx.x == 0) {
    for (int e = threadIdx.x; e < a.experts; e += kSortThreads) a.counts[e] = total[e];
    for (int e = threadIdx.x; e <= a.experts; e += kSortThreads) a.offsets[e] = offset[e];
  }
  int32_t* mine = sh + warp * a.experts;
  for_slots(a, r, [&](int64_t i, int e, uint32_t peers, bool in) {
    const uint32_t below = peers & ((1u << lane_id()) - 1u);
    int32_t row = -1;
    if (e >= 0) row = offset[e] + mine[e] + __popc(below);
    __syncwarp();
    if (e >= 0 && below == 0) mine[e] += __popc(peers);
    __syncwarp();
    if (in) {
      a.position[i] = row;
      if (row >= 0) a.slot[row] = static_cast<int32_t>(i);
    }
  });
  // rows of no slot: the ends of the experts' segments, and what is left of the capacity. Unsigned: the last
  // segment may end at 2^31 - 1, which a step passes.
  for (int e = blockIdx.x; e < a.experts; e += gridDim.x) {
    const uint32_t end = static_cast<uint32_t>(offset[e + 1]);
    for (uint32_t q = static_cast<uint32_t>(offset[e]) + total[e] + threadIdx.x; q < end; q += kSortThreads) a.slot[q] = -1;
  }
  for (int64_t q = offset[a.experts] + static_cast<int64_t>(blockIdx.x) * kSortThreads + threadIdx.x; q < a.capacity;
       q += static_cast<int64_t>(gridDim.x) * kSortThreads)
    a.slot[q] = -1;
}

// ---------------------------------------------------------------- rows
// Row r belongs to slot i where slot[r] = i and position[i] = r; a slot or row out of range, or a pair
// that does not agree, counts as none, so that no input reads or writes outside the matrices.
constexpr int kRowWarps = 8;
// A warp handles K choices of a token at once, and as many vectors a lane as keep 8 loads in flight.
constexpr int kLoads = 8;

struct RowParams {
  const void* src;  // gather: x; combine: y
  int64_t src_stride;
  const void* dout;
  int64_t dout_stride;
  void* dst;
  const float* weights;
  float* dweights;
  const int32_t *position, *slot;
  int64_t tokens, capacity;  // capacity: rows of the sorted matrix
  int64_t blocks;            // CTAs that clear rows of no slot, before the others
  int32_t topk, cols, nvec, clear;  // clear: rows that a clearing warp looks at, 32 at most
};

template <typename T, bool WIDE>
__device__ __forceinline__ void zero_row(T* row, int nvec) {
  Vec<T, WIDE> z;
  z.clear();
  for (int v = lane_id(); v < nvec; v += 32) z.put(row + static_cast<int64_t>(v) * Vec<T, WIDE>::kVec);
}
__device__ __forceinline__ int32_t slot_of_row(const RowParams& a, int64_t r) {
  const int32_t s = a.slot[r];
  return s >= 0 && s < a.tokens * a.topk && a.position[s] == r ? s : -1;
}
__device__ __forceinline__ int32_t row_of_slot(const RowParams& a, int64_t i) {
  const int32_t p = a.position[i];
  return p >= 0 && p < a.capacity ? p : -1;
}
// A warp clears those of its rows that have no slot: of 16 rows where few have none, of 4 where more than
// one in 16 may (7168 tokens x 2 in segments of 128: 6.9 us, 9.3 us with 16; 65536 tokens x 8 in segments of
// 16: 52 us, 63 us with 4).
template <typename T, bool WIDE>
__device__ __forceinline__ void clear_rows(const RowParams& a, int64_t r0) {
  const int64_t r = r0 + lane_id();
  const bool none = lane_id() < static_cast<uint32_t>(a.clear) && r < a.capacity && slot_of_row(a, r) < 0;
  uint32_t todo = __ballot_sync(0xffffffffu, none);
  while (todo != 0) {
    const int k = __ffs(static_cast<int>(todo)) - 1;
    todo &= todo - 1;
    zero_row<T, WIDE>(static_cast<T*>(a.dst) + (r0 + k) * a.cols, a.nvec);
  }
}

// Few rows: a warp for each.
template <typename T, bool WIDE>
__global__ void __launch_bounds__(kRowWarps * 32) expert_gather_rows_kernel(const RowParams a) {
  enter_stream();
  constexpr int VEC = Vec<T, WIDE>::kVec;
  const int64_t r = static_cast<int64_t>(blockIdx.x) * kRowWarps + (threadIdx.x >> 5);
  if (r >= a.capacity) return;
  const int32_t s = slot_of_row(a, r);
  T* out = static_cast<T*>(a.dst) + r * a.cols;
  if (s < 0) {
    zero_row<T, WIDE>(out, a.nvec);
    return;
  }
  const T* in = static_cast<const T*>(a.src) + static_cast<int64_t>(s / a.topk) * a.src_stride;
#pragma unroll 4
  for (int v = lane_id(); v < a.nvec; v += 32) {
    Vec<T, WIDE> t;
    t.load(in + static_cast<int64_t>(v) * VEC);
    t.put(out + static_cast<int64_t>(v) * VEC);
  }
}

// Many: a warp for each token and part of its row, read once and written to each of its rows; before
// them warps that clear the rows of no slot.
constexpr int kGatherVecs = 4;  // vectors a lane holds
template <typename T, bool WIDE>
__global__ void __launch_bounds__(kRowWarps * 32) expert_gather_tokens_kernel(const RowParams a) {
  enter_stream();
  constexpr int VEC = Vec<T, WIDE>::kVec;
  const int warp = threadIdx.x >> 5;
  if (blockIdx.x < a.blocks) {
    clear_rows<T, WIDE>(a, (static_cast<int64_t>(blockIdx.x) * kRowWarps + warp) * a.clear);
    return;
  }
  const int parts = (a.nvec + 32 * kGatherVecs - 1) / (32 * kGatherVecs);
  const int64_t item = (blockIdx.x - a.blocks) * kRowWarps + warp;
  const int64_t t = item / parts;
  if (t >= a.tokens) return;
  const int v0 = static_cast<int>(item - t * parts) * (32 * kGatherVecs) + lane_id();
  Vec<T, WIDE> x[kGatherVecs];
#pragma unroll
  for (int k = 0; k < kGatherVecs; ++k)
    if (v0 + 32 * k < a.nvec)
      x[k].load(static_cast<const T*>(a.src) + t * a.src_stride + static_cast<int64_t>(v0 + 32 * k) * VEC);
  for (int j0 = 0; j0 < a.topk; j0 += 32) {
    const int64_t i = t * a.topk + j0 + lane_id();
    int32_t mine = -1;
    if (j0 + static_cast<int>(lane_id()) < a.topk) {
      mine = row_of_slot(a, i);
      if (mine >= 0 && a.slot[mine] != i) mine = -1;
    }
    const int n = min(32, a.topk - j0);
    for (int j = 0; j < n; ++j) {
      const int32_t p = __shfl_sync(0xffffffffu, mine, j);
      if (p < 0) continue;
      T* out = static_cast<T*>(a.dst) + static_cast<int64_t>(p) * a.cols;
#pragma unroll
      for (int k = 0; k < kGatherVecs; ++k)
        if (v0 + 32 * k < a.nvec) x[k].put(out + static_cast<int64_t>(v0 + 32 * k) * VEC);
    }
  }
}

// A warp for each token and part of its row.
template <typename T, bool WIDE, int K>
__global__ void __launch_bounds__(kRowWarps * 32) expert_combine_kernel(const RowParams a) {
  enter_stream();
  constexpr int VEC = Vec<T, WIDE>::kVec, U = kLoads / K;
  const int parts = (a.nvec + 32 * U - 1) / (32 * U);
  const int64_t item = static_cast<int64_t>(blockIdx.x) * kRowWarps + (threadIdx.x >> 5);
  const int64_t t = item / parts;
  if (t >= a.tokens) return;
  const int v0 = static_cast<int>(item - t * parts) * (32 * U) + lane_id();
  float acc[U][VEC] = {};
  for (int j0 = 0; j0 < a.topk; j0 += K) {
    int32_t p[K];
    float w[K];
#pragma unroll
    for (int j = 0; j < K; ++j) {
      p[j] = -1;
      if (j0 + j < a.topk) p[j] = row_of_slot(a, t * a.topk + j0 + j);
    }
#pragma unroll
    for (int j = 0; j < K; ++j) w[j] = p[j] >= 0 && a.weights != nullptr ? a.weights[t * a.topk + j0 + j] : 1.0f;
    Vec<T, WIDE> y[K][U];
#pragma unroll
    for (int j = 0; j < K; ++j)
#pragma unroll
      for (int u = 0; u < U; ++u) {
        y[j][u].clear();
        if (p[j] >= 0 && v0 + 32 * u < a.nvec)
          y[j][u].load(static_cast<const T*>(a.src) + p[j] * a.src_stride + static_cast<int64_t>(v0 + 32 * u) * VEC);
      }
#pragma unroll
    for (int j = 0; j < K; ++j)
      if (p[j] >= 0) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
          float f[VEC];
          y[j][u].get(f);
#pragma unroll
          for (int e = 0; e < VEC; ++e) acc[u][e] += w[j] * f[e];
        }
      }
  }
#pragma unroll
  for (int u = 0; u < U; ++u)
    if (v0 + 32 * u < a.nvec)
      Vec<T, WIDE>::store(static_cast<T*>(a.dst) + t * a.cols + static_cast<int64_t>(v0 + 32 * u) * VEC, acc[u]);
}

// Few tokens: a warp for each slot, then for each row, cleared where it has none.
template <typename T, bool WIDE>
__global__ void __launch_bounds__(kRowWarps * 32) expert_combine_backward_slots_kernel(const RowParams a) {
  enter_stream();
  constexpr int VEC = Vec<T, WIDE>::kVec;
  const int64_t item = static_cast<int64_t>(blockIdx.x) * kRowWarps + (threadIdx.x >> 5);
  const int64_t slots = a.tokens * a.topk;
  if (item >= slots) {
    const int64_t r = item - slots;
    if (r < a.capacity && slot_of_row(a, r) < 0) zero_row<T, WIDE>(static_cast<T*>(a.dst) + r * a.cols, a.nvec);
    return;
  }
  const int32_t p = row_of_slot(a, item);
  float dot = 0.0f;
  if (p >= 0) {
    const float w = a.weights[item];
    const bool write = a.slot[p] == item;
    const T* g = static_cast<const T*>(a.dout) + item / a.topk * a.dout_stride;
    const T* y = static_cast<const T*>(a.src) + p * a.src_stride;
    T* dy = static_cast<T*>(a.dst) + static_cast<int64_t>(p) * a.cols;
#pragma unroll 4
    for (int v = lane_id(); v < a.nvec; v += 32) {
      Vec<T, WIDE> gv, yv;
      gv.load(g + static_cast<int64_t>(v) * VEC);
      yv.load(y + static_cast<int64_t>(v) * VEC);
      float gf[VEC], yf[VEC];
      gv.get(gf);
      yv.get(yf);
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        dot += gf[e] * yf[e];
        gf[e] *= w;
      }
      if (write) Vec<T, WIDE>::store(dy + static_cast<int64_t>(v) * VEC, gf);
    }
    dot = warp_sum(dot);
  }
  if (lane_id() == 0) a.dweights[item] = dot;
}

// Many: a warp for each token, which reads its row of dout once for all its choices; before them warps
// that clear the rows of no slot.
template <typename T, bool WIDE, int K>
__global__ void __launch_bounds__(kRowWarps * 32) expert_combine_backward_tokens_kernel(const RowParams a) {
  enter_stream();
  constexpr int VEC = Vec<T, WIDE>::kVec, U = kLoads / K;
  const int warp = threadIdx.x >> 5;
  if (blockIdx.x < a.blocks) {
    clear_rows<T, WIDE>(a, (static_cast<int64_t>(blockIdx.x) * kRowWarps + warp) * a.clear);
    return;
  }
  const int64_t t = (blockIdx.x - a.blocks) * kRowWarps + warp;
  if (t >= a.tokens) return;
  const T* g = static_cast<const T*>(a.dout) + t * a.dout_stride;
  for (int j0 = 0; j0 < a.topk; j0 += K) {
    int32_t p[K];
    float w[K], dot[K] = {};
    bool write[K];
#pragma unroll
    for (int j = 0; j < K; ++j) {
      p[j] = -1;
      if (j0 + j < a.topk) p[j] = row_of_slot(a, t * a.topk + j0 + j);
    }
#pragma unroll
    for (int j = 0; j < K; ++j) {
      const int64_t i = t * a.topk + j0 + j;
      w[j] = p[j] >= 0 ? a.weights[i] : 0.0f;
      write[j] = p[j] >= 0 && a.slot[p[j]] == i;
    }
    for (int v = lane_id(); v < a.nvec; v += 32 * U) {
      Vec<T, WIDE> gv[U], yv[K][U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        gv[u].clear();
        if (v + 32 * u < a.nvec) gv[u].load(g + static_cast<int64_t>(v + 32 * u) * VEC);
#pragma unroll
        for (int j = 0; j < K; ++j) {
          yv[j][u].clear();
          if (p[j] >= 0 && v + 32 * u < a.nvec)
            yv[j][u].load(static_cast<const T*>(a.src) + p[j] * a.src_stride + static_cast<int64_t>(v + 32 * u) * VEC);
        }
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        float gf[VEC];
        gv[u].get(gf);
#pragma unroll
        for (int j = 0; j < K; ++j) {
          float f[VEC];
          yv[j][u].get(f);
#pragma unroll
          for (int e = 0; e < VEC; ++e) {
            dot[j] += gf[e] * f[e];
            f[e] = gf[e] * w[j];
          }
          if (write[j] && v + 32 * u < a.nvec)
            Vec<T, WIDE>::store(static_cast<T*>(a.dst) + static_cast<int64_t>(p[j]) * a.cols +
                                    static_cast<int64_t>(v + 32 * u) * VEC, f);
        }
      }
    }
#pragma unroll
    for (int j = 0; j < K; ++j) {
      const float d = warp_sum(dot[j]);
      if (j0 + j < a.topk && lane_id() == 0) a.dweights[t * a.topk + j0 + j] = p[j] >= 0 ? d : 0.0f;
    }
  }
}

int64_t sort_chunk(int64_t slots) {
  int64_t c = kSortChunk;
  if (ceil_div(slots, c) > kSortMaxChunks) c = ceil_div(ceil_div(slots, kSortMaxChunks), kSortThreads) * kSortThreads;
  return c;
}

// The fewest choices at once that take topk in one round, 8 at most.
template <typename F>
cudaError_t by_choices(int64_t topk, F&& f) {
  if (topk <= 1) return f(std::integral_constant<int, 1>{});
  if (topk <= 2) return f(std::integral_constant<int, 2>{});
  if (topk <= 4) return f(std::integral_constant<int, 4>{});
  return f(std::integral_constant<int, 8>{});
}

template <typename F>
cudaError_t by_type(bool f32, bool wide, F&& f) {
  if (f32) return wide ? f(float{}, std::true_type{}) : f(float{}, std::false_type{});
  return wide ? f(uint16_t{}, std::true_type{}) : f(uint16_t{}, std::false_type{});
}

}  // namespace

int64_t expert_sort_workspace_bytes(int64_t slots, int64_t experts) {
  const int64_t chunks = ceil_div(slots, sort_chunk(slots));
  return chunks > kSortCluster ? chunks * experts * 4 : 0;
}

int launch_expert_sort(const void* ids, bool ids64, int64_t slots, int64_t experts, int64_t align, int64_t capacity,
                       int32_t* counts, int32_t* offsets, int32_t* position, int32_t* slot, void* workspace,
                       cudaStream_t stream, const DeviceInfo& dev) {
  SortParams a{};
  a.ids = ids, a.ids64 = ids64, a.experts = static_cast<int32_t>(experts);
  a.slots = slots, a.chunk = sort_chunk(slots), a.capacity = capacity;
  a.chunks = static_cast<int32_t>(std::max<int64_t>(1, ceil_div(slots, a.chunk)));
  a.align = static_cast<int32_t>(align);
  a.hist = static_cast<int32_t*>(workspace);
  a.counts = counts, a.offsets = offsets, a.position = position, a.slot = slot;
  const size_t count_sh = static_cast<size_t>(kSortWarps) * experts * 4;
  const size_t place_sh = count_sh + (2 * static_cast<size_t>(experts) + 1) * 4;
  static PerDevice<cudaError_t> ready;
  const int most = static_cast<int>((static_cast<size_t>(kSortWarps + 2) * BSQ_MAX_EXPERTS + 1) * 4);
  if (ready.run(dev.device, [&] {
        for (const void* k : {reinterpret_cast<const void*>(expert_count_kernel),
                              reinterpret_cast<const void*>(expert_place_kernel<kOneChunk>),
                              reinterpret_cast<const void*>(expert_place_kernel<kCluster>),
                              reinterpret_cast<const void*>(expert_place_kernel<kCounted>)}) {
          const cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, most);
          if (e != cudaSuccess) return e;
        }
        return cudaSuccess;
      }) != cudaSuccess)
    return BSQ_ERR_LAUNCH;
  const dim3 grid(static_cast<unsigned>(a.chunks));
  cudaError_t e;
  if (a.chunks == 1) {
    e = launch_in_stream(expert_place_kernel<kOneChunk>, grid, kSortThreads, place_sh, stream, 1, a);
  } else if (a.chunks <= kSortCluster) {
    e = launch_in_stream(expert_place_kernel<kCluster>, grid, kSortThreads, place_sh, stream, a.chunks, a);
  } else {
    e = launch_in_stream(expert_count_kernel, grid, kSortThreads, count_sh, stream, 1, a);
    if (e == cudaSuccess) e = launch_in_stream(expert_place_kernel<kCounted>, grid, kSortThreads, place_sh, stream, 1, a);
  }
  return e == cudaSuccess ? BSQ_OK : BSQ_ERR_LAUNCH;
}

// From this many tokens on a warp takes a token (or a part of its row) with all its choices, so that x and
// dout are read once: 16381 tokens x 2048 x 8 take 92 us to gather (162 us by rows) and 182 us backward (193 us),
// 65536 x 256 x 8 take 56 us (113 us) and 150 us (176 us). Fewer tokens would leave SMs without work; a
// warp for each row has topk times as many.
constexpr int64_t kManyTokens = 2048;

int launch_expert_gather(bool f32, const void* x, int64_t x_stride, const int32_t* position, const int32_t* slot,
                         int64_t capacity, int64_t tokens, int64_t topk, int64_t cols, void* rows, cudaStream_t stream) {
  RowParams a{};
  const int64_t es = f32 ? 4 : 2;
  a.src = x, a.src_stride = x_stride, a.dst = rows, a.position = position, a.slot = slot;
  a.tokens = tokens, a.capacity = capacity, a.topk = static_cast<int32_t>(topk), a.cols = static_cast<int32_t>(cols);
  const bool wide = wide_ok(x, x_stride * es) && wide_ok(rows, cols * es);
  a.nvec = static_cast<int32_t>(wide ? cols * es / 16 : cols);
  const bool many = tokens >= kManyTokens;
  a.clear = (capacity - tokens * topk) * 16 > capacity ? 4 : 16;
  a.blocks = many ? ceil_div(capacity, a.clear * kRowWarps) : 0;
  const int64_t grid = many ? a.blocks + ceil_div(tokens * ceil_div(a.nvec, 32 * kGatherVecs), kRowWarps)
                            : ceil_div(capacity, kRowWarps);
  if (grid > INT32_MAX) return BSQ_ERR_SHAPE;
  return by_type(f32, wide, [&](auto t, auto w) {
           using T = decltype(t);
           constexpr bool W = decltype(w)::value;
           return launch_in_stream(many ? expert_gather_tokens_kernel<T, W> : expert_gather_rows_kernel<T, W>,
                                   dim3(static_cast<unsigned>(grid)), kRowWarps * 32, 0, stream, 1, a);
         }) == cudaSuccess
             ? BSQ_OK
             : BSQ_ERR_LAUNCH;
}

int launch_expert_combine(bool f32, const void* y, int64_t y_stride, const int32_t* position, const float* weights,
                          int64_t tokens, int64_t topk, int64_t cols, int64_t capacity, void* out, cudaStream_t stream) {
  RowParams a{};
  const int64_t es = f32 ? 4 : 2;
  a.src = y, a.src_stride = y_stride, a.dst = out, a.position = position, a.weights = weights;
  a.tokens = tokens, a.capacity = capacity, a.topk = static_cast<int32_t>(topk), a.cols = static_cast<int32_t>(cols);
  const bool wide = wide_ok(y, y_stride * es) && wide_ok(out, cols * es);
  a.nvec = static_cast<int32_t>(wide ? cols * es / 16 : cols);
  const int64_t choices = topk <= 1 ? 1 : topk <= 2 ? 2 : topk <= 4 ? 4 : 8;
  const int64_t grid = ceil_div(tokens * ceil_div(a.nvec, 32 * kLoads / choices), kRowWarps);
  if (grid > INT32_MAX) return BSQ_ERR_SHAPE;
  return by_type(f32, wide, [&](auto t, auto w) {
           return by_choices(topk, [&](auto k) {
             return launch_in_stream(expert_combine_kernel<decltype(t), decltype(w)::value, decltype(k)::value>,
                                     dim3(static_cast<unsigned>(grid)), kRowWarps * 32, 0, stream, 1, a);
           });
         }) == cudaSuccess
             ? BSQ_OK
             : BSQ_ERR_LAUNCH;
}

int launch_expert_combine_backward(bool f32, const void* dout, int64_t dout_stride, const void* y, int64_t y_stride,
                                   const int32_t* position, const int32_t* slot, const float* weights, int64_t tokens,
                                   int64_t topk, int64_t cols, int64_t capacity, void* dy, float* dweights,
                                   cudaStream_t stream) {
  RowParams a{};
  const int64_t es = f32 ? 4 : 2;
  a.src = y, a.src_stride = y_stride, a.dout = dout, a.dout_stride = dout_stride, a.dst = dy;
  a.position = position, a.slot = slot, a.weights = weights, a.dweights = dweights;
  a.tokens = tokens, a.capacity = capacity, a.topk = static_cast<int32_t>(topk), a.cols = static_cast<int32_t>(cols);
  const bool wide = wide_ok(y, y_stride * es) && wide_ok(dout, dout_stride * es) && wide_ok(dy, cols * es);
  a.nvec = static_cast<int32_t>(wide ? cols * es / 16 : cols);
  const bool many = tokens >= kManyTokens;
  a.clear = (capacity - tokens * topk) * 16 > capacity ? 4 : 16;
  a.blocks = many ? ceil_div(capacity, a.clear * kRowWarps) : 0;
  const unsigned grid = static_cast<unsigned>(many ? a.blocks + ceil_div(tokens, kRowWarps)
                                                   : ceil_div(tokens * topk + capacity, kRowWarps));
  return by_type(f32, wide, [&](auto t, auto w) {
           using T = decltype(t);
           constexpr bool W = decltype(w)::value;
           if (!many)
             return launch_in_stream(expert_combine_backward_slots_kernel<T, W>, dim3(grid), kRowWarps * 32, 0, stream, 1, a);
           return by_choices(topk, [&](auto k) {
             return launch_in_stream(expert_combine_backward_tokens_kernel<T, W, decltype(k)::value>, dim3(grid),
                                     kRowWarps * 32, 0, stream, 1, a);
           });
         }) == cudaSuccess
             ? BSQ_OK
             : BSQ_ERR_LAUNCH;
}

}  // namespace bsq
