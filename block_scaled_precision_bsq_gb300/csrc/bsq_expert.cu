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
constexpr int kSortWarps = 8;
constexpr int kSortThreads = kSortWarps * 32;
constexpr int64_t kSortChunk = 2048;   // slots of a CTA, unless that makes more CTAs than
constexpr int64_t kSortMaxChunks = 296;  // this many, each of which reads every chunk's counts

struct SortParams {
  const void* ids;
  bool ids64;
  int32_t experts;
  int64_t slots, chunk, capacity;  // chunk: slots of a CTA, a multiple of kSortThreads
  int32_t chunks, align;
  int32_t* hist;  // [chunks][experts], more than one chunk only
  int32_t *counts, *offsets, *position, *slot;
};

__device__ __forceinline__ int expert_of(const SortParams& a, int64_t i, int64_t end) {
  if (i >= end) return -1;
  const int64_t e = a.ids64 ? static_cast<const int64_t*>(a.ids)[i] : static_cast<const int32_t*>(a.ids)[i];
  return e >= 0 && e < a.experts ? static_cast<int>(e) : -1;
}

// The CTA's slots are cut into one consecutive range for each warp; f(slot, expert, peers) is called
// by every lane for each group of 32 slots, peers = the lanes with the same expert.
template <typename F>
__device__ __forceinline__ void for_slots(const SortParams& a, F&& f) {
  const int64_t begin = static_cast<int64_t>(blockIdx.x) * a.chunk, end = min(a.slots, begin + a.chunk);
  const int64_t per = a.chunk / kSortWarps;
  const int64_t w0 = begin + (threadIdx.x >> 5) * per, w1 = min(end, w0 + per);
  for (int64_t i = w0; i < w1; i += 32) {
    const int e = expert_of(a, i + lane_id(), w1);
    f(i + lane_id(), e, __match_any_sync(0xffffffffu, e), i + lane_id() < w1);
  }
}

__device__ __forceinline__ void count_slots(const SortParams& a, int32_t* mine) {
  for_slots(a, [&](int64_t, int e, uint32_t peers, bool) {
    if (e >= 0 && lane_id() == static_cast<uint32_t>(__ffs(static_cast<int>(peers)) - 1)) mine[e] += __popc(peers);
    __syncwarp();
  });
}

__global__ void __launch_bounds__(kSortThreads) expert_count_kernel(const SortParams a) {
  extern __shared__ int32_t sh[];  // [warps][experts]
  for (int i = threadIdx.x; i < kSortWarps * a.experts; i += kSortThreads) sh[i] = 0;
  __syncthreads();
  count_slots(a, sh + (threadIdx.x >> 5) * a.experts);
  __syncthreads();
  for (int e = threadIdx.x; e < a.experts; e += kSortThreads) {
    int32_t s = 0;
    for (int w = 0; w < kSortWarps; ++w) s += sh[w * a.experts + e];
    a.hist[static_cast<int64_t>(blockIdx.x) * a.experts + e] = s;
  }
}

__global__ void __launch_bounds__(kSortThreads) expert_place_kernel(const SortParams a) {
  extern __shared__ int32_t sh[];  // [warps][experts] counts, then running rows; [experts] totals; [experts + 1] offsets
  int32_t* total = sh + kSortWarps * a.experts;
  int32_t* offset = total + a.experts;
  __shared__ int32_t warp_sums[kSortWarps];
  const int warp = threadIdx.x >> 5;
  for (int i = threadIdx.x; i < kSortWarps * a.experts; i += kSortThreads) sh[i] = 0;
  __syncthreads();
  count_slots(a, sh + warp * a.experts);
  __syncthreads();
  // totals over all chunks, and the rows that earlier chunks take of each expert (kept in the first
  // warp's counts, which are turned into running rows below)
  for (int e = threadIdx.x; e < a.experts; e += kSortThreads) {
    int32_t before = 0, sum = 0;
    if (a.chunks > 1) {
      for (int c = 0; c < a.chunks; ++c) {
        const int32_t n = a.hist[static_cast<int64_t>(c) * a.experts + e];
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
  __syncthreads();
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
  for_slots(a, [&](int64_t i, int e, uint32_t peers, bool in) {
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
  // rows of no slot: the ends of the experts' segments, and what is left of the capacity
  for (int e = blockIdx.x; e < a.experts; e += gridDim.x)
    for (int r = offset[e] + total[e] + threadIdx.x; r < offset[e + 1]; r += kSortThreads) a.slot[r] = -1;
  for (int64_t r = offset[a.experts] + static_cast<int64_t>(blockIdx.x) * kSortThreads + threadIdx.x; r < a.capacity;
       r += static_cast<int64_t>(gridDim.x) * kSortThreads)
    a.slot[r] = -1;
}

// ---------------------------------------------------------------- rows
constexpr int kRowWarps = 8;

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
  int32_t topk, cols, nvec;
};

template <typename T, bool WIDE>
__device__ __forceinline__ void zero_row(T* row, int nvec) {
  Vec<T, WIDE> z;
  z.clear();
  for (int v = lane_id(); v < nvec; v += 32) z.put(row + static_cast<int64_t>(v) * Vec<T, WIDE>::kVec);
}

// A warp for each row.
template <typename T, bool WIDE>
__global__ void __launch_bounds__(kRowWarps * 32) expert_gather_kernel(const RowParams a) {
  constexpr int VEC = Vec<T, WIDE>::kVec;
  const int64_t r = static_cast<int64_t>(blockIdx.x) * kRowWarps + (threadIdx.x >> 5);
  if (r >= a.capacity) return;
  const int32_t s = a.slot[r];  // a slot or row outside its range counts as none, here and below
  T* out = static_cast<T*>(a.dst) + r * a.cols;
  if (s < 0 || s >= a.tokens * a.topk) {
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

// A warp for each token and 32 vectors of its row.
template <typename T, bool WIDE>
__global__ void __launch_bounds__(kRowWarps * 32) expert_combine_kernel(const RowParams a) {
  constexpr int VEC = Vec<T, WIDE>::kVec;
  const int chunks = (a.nvec + 31) / 32;
  const int64_t item = static_cast<int64_t>(blockIdx.x) * kRowWarps + (threadIdx.x >> 5);
  const int64_t t = item / chunks;
  if (t >= a.tokens) return;
  const int v = static_cast<int>(item % chunks) * 32 + lane_id();
  if (v >= a.nvec) return;
  float acc[VEC] = {};
#pragma unroll 4
  for (int j = 0; j < a.topk; ++j) {
    const int32_t p = a.position[t * a.topk + j];
    if (p < 0 || p >= a.capacity) continue;
    const float w = a.weights != nullptr ? a.weights[t * a.topk + j] : 1.0f;
    Vec<T, WIDE> y;
    y.load(static_cast<const T*>(a.src) + p * a.src_stride + static_cast<int64_t>(v) * VEC);
    float f[VEC];
    y.get(f);
#pragma unroll
    for (int e = 0; e < VEC; ++e) acc[e] += w * f[e];
  }
  Vec<T, WIDE>::store(static_cast<T*>(a.dst) + t * a.cols + static_cast<int64_t>(v) * VEC, acc);
}

// A warp for each slot, then a warp for each row that has none.
template <typename T, bool WIDE>
__global__ void __launch_bounds__(kRowWarps * 32) expert_combine_backward_kernel(const RowParams a) {
  constexpr int VEC = Vec<T, WIDE>::kVec;
  const int64_t item = static_cast<int64_t>(blockIdx.x) * kRowWarps + (threadIdx.x >> 5);
  const int64_t slots = a.tokens * a.topk;
  if (item >= slots) {
    const int64_t r = item - slots;
    if (r < a.capacity && a.slot[r] < 0) zero_row<T, WIDE>(static_cast<T*>(a.dst) + r * a.cols, a.nvec);
    return;
  }
  const int32_t p = a.position[item];
  float dot = 0.0f;
  if (p >= 0 && p < a.capacity) {
    const float w = a.weights[item];
    const T* g = static_cast<const T*>(a.dout) + item / a.topk * a.dout_stride;
    const T* y = static_cast<const T*>(a.src) + p * a.src_stride;
    T* dy = static_cast<T*>(a.dst) + static_cast<int64_t>(p) * a.cols;
#pragma unroll 2
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
      Vec<T, WIDE>::store(dy + static_cast<int64_t>(v) * VEC, gf);
    }
    dot = warp_sum(dot);
  }
  if (lane_id() == 0) a.dweights[item] = dot;
}

int64_t sort_chunk(int64_t slots) {
  int64_t c = kSortChunk;
  if (ceil_div(slots, c) > kSortMaxChunks) c = ceil_div(ceil_div(slots, kSortMaxChunks), kSortThreads) * kSortThreads;
  return c;
}

template <typename F>
cudaError_t by_type(bool f32, bool wide, F&& f) {
  if (f32) {
    if (wide) f(float{}, std::true_type{});
    else f(float{}, std::false_type{});
  } else {
    if (wide) f(uint16_t{}, std::true_type{});
    else f(uint16_t{}, std::false_type{});
  }
  return cudaGetLastError();
}

}  // namespace

int64_t expert_sort_workspace_bytes(int64_t slots, int64_t experts) {
  const int64_t chunks = ceil_div(slots, sort_chunk(slots));
  return chunks > 1 ? chunks * experts * 4 : 0;
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
  const size_t most = (static_cast<size_t>(kSortWarps + 2) * BSQ_MAX_EXPERTS + 1) * 4;
  if (ready.run(dev.device, [&] {
        const cudaError_t e = cudaFuncSetAttribute(expert_count_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                   static_cast<int>(most));
        return e != cudaSuccess ? e
                                : cudaFuncSetAttribute(expert_place_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                       static_cast<int>(most));
      }) != cudaSuccess)
    return BSQ_ERR_LAUNCH;
  if (a.chunks > 1) expert_count_kernel<<<a.chunks, kSortThreads, count_sh, stream>>>(a);
  expert_place_kernel<<<a.chunks, kSortThreads, place_sh, stream>>>(a);
  return cudaGetLastError() == cudaSuccess ? BSQ_OK : BSQ_ERR_LAUNCH;
}

int launch_expert_gather(bool f32, const void* x, int64_t x_stride, const int32_t* slot, int64_t capacity,
                         int64_t tokens, int64_t topk, int64_t cols, void* rows, cudaStream_t stream) {
  RowParams a{};
  const int64_t es = f32 ? 4 : 2;
  a.src = x, a.src_stride = x_stride, a.dst = rows, a.slot = slot;
  a.tokens = tokens, a.capacity = capacity, a.topk = static_cast<int32_t>(topk), a.cols = static_cast<int32_t>(cols);
  const bool wide = wide_ok(x, x_stride * es) && wide_ok(rows, cols * es);
  a.nvec = static_cast<int32_t>(wide ? cols * es / 16 : cols);
  const unsigned grid = static_cast<unsigned>(ceil_div(capacity, kRowWarps));
  return by_type(f32, wide, [&](auto t, auto w) {
           expert_gather_kernel<decltype(t), decltype(w)::value><<<grid, kRowWarps * 32, 0, stream>>>(a);
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
  const int64_t grid = ceil_div(tokens * ceil_div(a.nvec, 32), kRowWarps);
  if (grid > INT32_MAX) return BSQ_ERR_SHAPE;
  return by_type(f32, wide, [&](auto t, auto w) {
           expert_combine_kernel<decltype(t), decltype(w)::value>
               <<<static_cast<unsigned>(grid), kRowWarps * 32, 0, stream>>>(a);
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
  const unsigned grid = static_cast<unsigned>(ceil_div(tokens * topk + capacity, kRowWarps));
  return by_type(f32, wide, [&](auto t, auto w) {
           expert_combine_backward_kernel<decltype(t), decltype(w)::value><<<grid, kRowWarps * 32, 0, stream>>>(a);
         }) == cudaSuccess
             ? BSQ_OK
             : BSQ_ERR_LAUNCH;
}

}  // namespace bsq
