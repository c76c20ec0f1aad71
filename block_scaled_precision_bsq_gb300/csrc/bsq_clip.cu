// bsq_clip.cu -- the norm of many gradient tensors taken together, and clipping by it.
//
//   norm = sqrt(sum over all tensors and elements of g^2), or max |g|
//   coef = max_norm / (norm + eps), 1 where norm + eps <= max_norm,  dst = coef * src for every tensor
// The tensors' addresses travel in the launch's parameters (up to kMaxItems a launch), so a call
// needs no table in device memory and can be captured into a graph. Tensors are cut into chunks,
// chunks are dealt to the CTAs in a fixed order, every CTA leaves one partial sum in the workspace
// and every CTA of the scaling kernel adds those up in the same order: no atomics, the same bits
// every time.
//
// Squares are added in fp32, 64 at most to one sum, and those sums in fp64. Where a thread's largest
// element is below 2^-50 or above 2^55, where squares would lose bits or overflow, the thread takes
// its elements again in fp64 (the rate of fp64 is far too low for all of them).
//
// Bound by HBM: the gradients are read for the norm, and read again and written for the scaling.
#include <algorithm>

#include "bsq.h"
#include "bsq_device.cuh"
#include "bsq_elem.cuh"
#include "bsq_internal.h"

namespace bsq {
namespace {

constexpr int kClipThreads = 256;
// Elements of a chunk: 64 a thread, fewer where that would leave CTAs without work. (Looking up the
// tensor of a chunk takes a chain of reads: 300M bf16 take 298 us in chunks of 16384, 309 us in 8192,
// 423 us in 4096.)
constexpr int kMinChunkLog = 11, kMaxChunkLog = 14;
constexpr int kMaxItems = 1024, kFewItems = 64;

template <int N>
struct ClipItems {
  int32_t n, chunks, chunk_log;
  const void* src[N];
  void* dst[N];
  int64_t elems[N];
  int32_t first[N + 1];  // first chunk of each tensor
  uint8_t f32[N];
};
struct ClipPartial {
  double sum;
  uint32_t amax, pad;  // largest |g| as fp32 bits: NaN above infinity above all numbers
};
struct ClipParams {
  ClipPartial* partials;  // of this launch
  const ClipPartial* all;
  int32_t num_all;
  bool inf_norm, write_norm;
  float max_norm, eps;
  float* norm;
};

template <int N>
__device__ __forceinline__ int find_item(const ClipItems<N>& it, int chunk) {
  int lo = 0, hi = it.n;  // the last item whose first chunk is not after `chunk` and that has chunks
  while (hi - lo > 1) {
    const int mid = (lo + hi) / 2;
    if (it.first[mid] <= chunk) lo = mid;
    else hi = mid;
  }
  return lo;
}

__device__ __forceinline__ uint32_t abs_bits(float v) { return __float_as_uint(v) & 0x7fffffffu; }

// vec(index) for a chunk's 16-byte vectors from element `lead` on, single(index) for the elements before
// and after.
template <typename T, typename FV, typename FS>
__device__ __forceinline__ void for_chunk(int64_t lead, int64_t n, FV&& vec, FS&& single) {
  constexpr int VEC = Vec<T, true>::kVec;
  if (lead > n) lead = n;
  const int64_t nv = (n - lead) / VEC;
#pragma unroll 4
  for (int64_t v = threadIdx.x; v < nv; v += kClipThreads) vec(lead + v * VEC);
  for (int64_t i = threadIdx.x; i < lead; i += kClipThreads) single(i);
  for (int64_t i = lead + nv * VEC + threadIdx.x; i < n; i += kClipThreads) single(i);
}
// Elements before the first one that starts a 128-byte line: a warp's vectors then fill whole lines
// (from a 16-byte boundary on, its first and last sectors are shared with other warps, and written
// by halves).
template <typename T>
__device__ __forceinline__ int64_t lead_of(const T* p) {
  return static_cast<int64_t>((128u - (static_cast<uint32_t>(reinterpret_cast<uintptr_t>(p)) & 127u)) & 127u) /
         static_cast<int64_t>(sizeof(T));
}

template <typename T>
__device__ __forceinline__ void sum_chunk(const T* p, int64_t n, double& total, uint32_t& amax) {
  constexpr int VEC = Vec<T, true>::kVec;
  const int64_t lead = lead_of(p);
  float s = 0.0f;
  uint32_t m = 0;
  for_chunk<T>(
      lead, n,
      [&](int64_t i) {
        Vec<T, true> r;
        r.load(p + i);
        float v[VEC];
        r.get(v);
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
          s += v[e] * v[e];
          m = max(m, abs_bits(v[e]));
        }
      },
      [&](int64_t i) {
        Vec<T, false> r;
        r.load(p + i);
        float v;
        r.get(&v);
        s += v * v;
        m = max(m, abs_bits(v));
      });
  amax = max(amax, m);
  constexpr uint32_t kLow = (127u - 50u) << 23, kHigh = (127u + 55u) << 23, kInf = 0x7f800000u;
  if (m != 0 && m < kInf && (m < kLow || m > kHigh)) {
    double d = 0.0;
    auto add = [&](int64_t i) {
      Vec<T, false> r;
      r.load(p + i);
      float v;
      r.get(&v);
      d += static_cast<double>(v) * static_cast<double>(v);
    };
    for_chunk<T>(
        lead, n,
        [&](int64_t i) {
          for (int e = 0; e < VEC; ++e) add(i + e);
        },
        add);
    total += d;
  } else {
    total += static_cast<double>(s);
  }
}

__device__ __forceinline__ double warp_sum(double v) {
#pragma unroll
  for (int m = 16; m > 0; m >>= 1) v += __shfl_xor_sync(0xffffffffu, v, m);
  return v;
}

// Sum and maximum over the CTA, in every thread.
__device__ __forceinline__ void cta_join(double& total, uint32_t& amax) {
  __shared__ double sums[kClipThreads / 32];
  __shared__ uint32_t maxs[kClipThreads / 32];
  total = warp_sum(total);
  amax = __reduce_max_sync(0xffffffffu, amax);
  if (lane_id() == 0) sums[threadIdx.x >> 5] = total, maxs[threadIdx.x >> 5] = amax;
  __syncthreads();
  total = 0.0;
  amax = 0;
  for (int w = 0; w < kClipThreads / 32; ++w) total += sums[w], amax = max(amax, maxs[w]);
}

template <int N>
__global__ void __launch_bounds__(kClipThreads) grad_sum_kernel(const __grid_constant__ ClipItems<N> it,
                                                                const ClipParams a) {
  enter_stream();
  double total = 0.0;
  uint32_t amax = 0;
  for (int c = blockIdx.x; c < it.chunks; c += gridDim.x) {
    const int k = find_item(it, c);
    const int64_t at = static_cast<int64_t>(c - it.first[k]) << it.chunk_log;
    const int64_t n = min(int64_t{1} << it.chunk_log, it.elems[k] - at);
    if (it.f32[k]) sum_chunk(static_cast<const float*>(it.src[k]) + at, n, total, amax);
    else sum_chunk(static_cast<const uint16_t*>(it.src[k]) + at, n, total, amax);
  }
  cta_join(total, amax);
  if (threadIdx.x == 0) a.partials[blockIdx.x] = ClipPartial{total, amax, 0u};
}

__device__ __forceinline__ float joined_norm(const ClipParams& a) {
  double total = 0.0;
  uint32_t amax = 0;
  for (int i = threadIdx.x; i < a.num_all; i += kClipThreads) {
    total += a.all[i].sum;
    amax = max(amax, a.all[i].amax);
  }
  cta_join(total, amax);
  return a.inf_norm ? __uint_as_float(amax) : static_cast<float>(sqrt(total));
}

__global__ void __launch_bounds__(kClipThreads) grad_norm_kernel(const ClipParams a) {
  enter_stream();
  const float norm = joined_norm(a);
  if (threadIdx.x == 0) *a.norm = norm;
}

// Results that nothing reads soon: first to leave L2.
__device__ __forceinline__ void store_stream(float* p, const float* v) {
  asm volatile("st.global.cs.v4.f32 [%0], {%1, %2, %3, %4};" ::"l"(p), "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3])
               : "memory");
}
__device__ __forceinline__ void store_stream(uint16_t* p, const float* v) {
  asm volatile("st.global.cs.v4.b32 [%0], {%1, %2, %3, %4};" ::"l"(p), "r"(f32x2_to_bf16x2(v[0], v[1])),
               "r"(f32x2_to_bf16x2(v[2], v[3])), "r"(f32x2_to_bf16x2(v[4], v[5])), "r"(f32x2_to_bf16x2(v[6], v[7]))
               : "memory");
}

template <typename T>
__device__ __forceinline__ void scale_chunk(const T* src, T* dst, int64_t n, float coef) {
  constexpr int VEC = Vec<T, true>::kVec;
  const int64_t lead = lead_of(dst);
  auto single = [&](int64_t i) {
    Vec<T, false> r;
    r.load(src + i);
    float v;
    r.get(&v);
    v *= coef;
    Vec<T, false>::store(dst + i, &v);
  };
  if (((reinterpret_cast<uintptr_t>(src) ^ reinterpret_cast<uintptr_t>(dst)) & 15u) != 0) {  // vectors of one are none of the other
#pragma unroll 4
    for (int64_t i = threadIdx.x; i < n; i += kClipThreads) single(i);
    return;
  }
  for_chunk<T>(
      lead, n,
      [&](int64_t i) {
        Vec<T, true> r;
        r.load(src + i);
        float v[VEC];
        r.get(v);
#pragma unroll
        for (int e = 0; e < VEC; ++e) v[e] *= coef;
        store_stream(dst + i, v);
      },
      single);
}

template <int N>
__global__ void __launch_bounds__(kClipThreads) grad_scale_kernel(const __grid_constant__ ClipItems<N> it,
                                                                  const ClipParams a) {
  enter_stream();
  const float norm = joined_norm(a);
  if (a.write_norm && blockIdx.x == 0 && threadIdx.x == 0) *a.norm = norm;
  // Compared ahead of the quotient, which has no value where both are infinite or zero. A NaN norm stays one.
  const float coef = norm + a.eps <= a.max_norm ? 1.0f : a.max_norm / (norm + a.eps);
  // backwards: what the sums read last may still lie in L2, and the results are the first to leave it
  for (int back = blockIdx.x; back < it.chunks; back += gridDim.x) {
    const int c = it.chunks - 1 - back;
    const int k = find_item(it, c);
    if (coef == 1.0f && it.src[k] == it.dst[k]) continue;  // in place and nothing to change
    const int64_t at = static_cast<int64_t>(c - it.first[k]) << it.chunk_log;
    const int64_t n = min(int64_t{1} << it.chunk_log, it.elems[k] - at);
    if (it.f32[k]) scale_chunk(static_cast<const float*>(it.src[k]) + at, static_cast<float*>(it.dst[k]) + at, n, coef);
    else scale_chunk(static_cast<const uint16_t*>(it.src[k]) + at, static_cast<uint16_t*>(it.dst[k]) + at, n, coef);
  }
}

template <int N>
int fill_items(ClipItems<N>& b, const bsq_grad_item* items, int count, int chunk_log) {
  b.n = count;
  b.chunk_log = chunk_log;
  int64_t chunks = 0;
  for (int i = 0; i < count; ++i) {
    b.src[i] = items[i].src;
    b.dst[i] = items[i].dst;
    b.elems[i] = items[i].elems;
    b.f32[i] = items[i].f32 != 0;
    b.first[i] = static_cast<int32_t>(chunks);
    chunks += ceil_div(items[i].elems, int64_t{1} << chunk_log);
    if (chunks > INT32_MAX) return BSQ_ERR_SHAPE;
  }
  b.first[count] = b.chunks = static_cast<int32_t>(chunks);
  return BSQ_OK;
}

constexpr int kCtasPerSm = 8;
int clip_grid(int chunks, int num_sms) { return std::max(1, std::min(chunks, kCtasPerSm * num_sms)); }

template <int N>
int run_items(int count, const bsq_grad_item* items, bool scale, ClipParams p, cudaStream_t stream,
              const DeviceInfo& dev) {
  ClipItems<N> b;
  const int64_t batches = std::max<int64_t>(1, ceil_div(count, N));
  ClipPartial* const base = p.partials;
  int64_t elems = 0;
  for (int i = 0; i < count; ++i) elems += items[i].elems;
  int chunk_log = kMinChunkLog;
  while (chunk_log < kMaxChunkLog && (elems >> chunk_log) > kCtasPerSm * dev.num_sms) ++chunk_log;
  for (int64_t k = 0; k < batches; ++k) {
    const int n = static_cast<int>(std::min<int64_t>(N, count - k * N));
    const int st = fill_items(b, items + k * N, n, chunk_log);
    if (st != BSQ_OK) return st;
    p.partials = base + p.num_all;
    const int grid = clip_grid(b.chunks, dev.num_sms);
    if (launch_in_stream(grad_sum_kernel<N>, dim3(static_cast<unsigned>(grid)), kClipThreads, 0, stream, 1, b, p) != cudaSuccess)
      return BSQ_ERR_LAUNCH;
    p.num_all += grid;
  }
  p.all = base;
  if (!scale || count == 0) {
    return launch_in_stream(grad_norm_kernel, dim3(1), kClipThreads, 0, stream, 1, p) == cudaSuccess ? BSQ_OK : BSQ_ERR_LAUNCH;
  }
  for (int64_t k = 0; k < batches; ++k) {
    const int n = static_cast<int>(std::min<int64_t>(N, count - k * N));
    if (batches > 1) fill_items(b, items + k * N, n, chunk_log);
    p.write_norm = k == 0;
    if (launch_in_stream(grad_scale_kernel<N>, dim3(static_cast<unsigned>(clip_grid(b.chunks, dev.num_sms))), kClipThreads, 0,
                         stream, 1, b, p) != cudaSuccess)
      return BSQ_ERR_LAUNCH;
  }
  return BSQ_OK;
}

}  // namespace

int64_t clip_workspace_bytes(int64_t count, const DeviceInfo& dev) {
  const int64_t batches = std::max<int64_t>(1, ceil_div(count, kMaxItems));
  return batches * kCtasPerSm * dev.num_sms * static_cast<int64_t>(sizeof(ClipPartial));
}

int launch_clip(int count, const bsq_grad_item* items, bool inf_norm, bool scale, float max_norm, float eps,
                void* workspace, float* norm, cudaStream_t stream, const DeviceInfo& dev) {
  ClipParams p{};
  p.partials = static_cast<ClipPartial*>(workspace);
  p.inf_norm = inf_norm, p.max_norm = max_norm, p.eps = eps, p.norm = norm;
  const int st = count <= kFewItems ? run_items<kFewItems>(count, items, scale, p, stream, dev)
                                    : run_items<kMaxItems>(count, items, scale, p, stream, dev);
  return st;
}

}  // namespace bsq
