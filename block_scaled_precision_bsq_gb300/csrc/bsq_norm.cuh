// bsq_norm.cuh -- the norms before and after a block, fused with the block's gate and the residual
// scale, forward and backward.
//
// Forward, per row (Norm is z = (v - mean) * rstd with rstd = 1 / sqrt(mean((v - mean)^2) + eps);
// the RMS norm has mean = 0):
//   n = Norm(h) * (post_weight + o) + post_bias        (n = h without a norm after the block)
//   x_out = residual_scale * x + gate * n
//   y = Norm(x_out) * (pre_weight + o) + pre_bias      (the next block's norm)
// Backward, from dx_out and dy, with z2 = Norm(x_out) and z1 = Norm(h) rebuilt from the saved
// statistics:
//   g2 = dy * (pre_weight + o),  d = dx_out + rstd2 * (g2 - mean(g2) - z2 * mean(g2 * z2))
//   dx = residual_scale * d,     g1 = d * gate * (post_weight + o)
//   dh = rstd1 * (g1 - mean(g1) - z1 * mean(g1 * z1))
//   dpre_weight = sum_r dy * z2, dpre_bias = sum_r dy
// and with A1 = sum_r d * z1, A0 = sum_r d over the rows that share a gate row,
//   dgate = (post_weight + o) * A1 + post_bias * A0,
//   dpost_weight = sum over gate rows of gate * A1, dpost_bias = sum of gate * A0,
// so four column sums (two without biases) give all five parameter gradients. (The mean(g) terms
// belong to the layer norm alone.)
//
// Both directions are bound by HBM: 4 matrices forward, 6 backward, each moved once. A row is held
// in registers by a team of 1 to 16 warps (8 to 32 elements a lane and matrix forward, 8 backward), or by
// a cluster of CTAs with 16 warps each for longer rows, so that it is read once although its statistics
// come first.
//
// This file holds what both directions use: the teams of warps that hold a row and their sums, a
// thread's columns, and how a pass over rows is cut.
#pragma once

#include <algorithm>
#include <initializer_list>

#include "bsq.h"
#include "bsq_device.cuh"
#include "bsq_elem.cuh"
#include "bsq_internal.h"

namespace bsq {
namespace {

constexpr int kMaxTeamWarps = 16;
constexpr int kMaxCluster = 16;
constexpr int kGradElems = 8;  // elements of a row in a thread of the backward pass: its column sums take registers


// ---------------------------------------------------------------- element access
// Parameters are bf16 or fp32 whatever the matrices are, and few enough to stay in L1.
template <int VEC>
__device__ __forceinline__ void load_param(const void* p, bool f32, int64_t at, float* v) {
  if (f32) {
    const float* q = static_cast<const float*>(p) + at;
    if constexpr (VEC == 1) {
      v[0] = __ldg(q);
    } else {
#pragma unroll
      for (int i = 0; i < VEC; i += 4) {
        const float4 f = __ldg(reinterpret_cast<const float4*>(q + i));
        v[i] = f.x, v[i + 1] = f.y, v[i + 2] = f.z, v[i + 3] = f.w;
      }
    }
  } else {
    const uint16_t* q = static_cast<const uint16_t*>(p) + at;
    if constexpr (VEC == 1) {
      v[0] = bf16_to_f32(__ldg(q));
    } else if constexpr (VEC == 4) {
      const uint2 w = __ldg(reinterpret_cast<const uint2*>(q));
      v[0] = __uint_as_float(w.x << 16), v[1] = __uint_as_float(w.x & 0xffff0000u);
      v[2] = __uint_as_float(w.y << 16), v[3] = __uint_as_float(w.y & 0xffff0000u);
    } else {
      Vec<uint16_t, true> t;
      t.raw = __ldg(reinterpret_cast<const uint4*>(q));
      t.get(v);
    }
  }
}
// weight + offset (1 where there is none), bias (0 where there is none)
template <int VEC>
__device__ __forceinline__ void load_weight(const void* p, bool f32, float offset, int64_t at, float* v) {
  if (p == nullptr) {
#pragma unroll
    for (int i = 0; i < VEC; ++i) v[i] = 1.0f;
    return;
  }
  load_param<VEC>(p, f32, at, v);
#pragma unroll
  for (int i = 0; i < VEC; ++i) v[i] += offset;
}

// ---------------------------------------------------------------- sums over a row
// The warps that hold one row: a team of a CTA, or all warps of a cluster. Each warp's partial sums
// go to a slot of shared memory (of every CTA of the cluster), and one barrier later every warp adds
// the slots in the same order. Two sets of slots in turn make one barrier per sum enough: a set is
// written again only behind the next sum's barrier, which every reader reaches after its reads.
template <bool CLUSTER>
struct Team {
  // 16 slots for each team (of a CTA: up to 16 teams) or each CTA of the cluster; unused ones stay 0
  static constexpr int kSlots = kMaxTeamWarps * (CLUSTER ? kMaxCluster : kMaxTeamWarps);
  float4 (*slots)[kSlots];      // [2][...]
  int warps, warp, first, bar;  // warps of the team (all CTAs), own index, first slot, named barrier
  int parity = 0;
  uint32_t ranks = 1, rank = 0;
  // publish() and collect(): barriers, their phases, and whether a wait gave up
  uint64_t* ring_bars = nullptr;
  volatile int* abort = nullptr;
  int* status = nullptr;
  uint64_t wait_ns = kWaitLimitNs;
  uint32_t phases = 0;
  bool ok = true;

  __device__ __forceinline__ void init(float4 (*s)[kSlots], int team_warps) {
    slots = s;
    const int w = threadIdx.x >> 5;
    if constexpr (CLUSTER) {
      ranks = cluster_size();
      rank = cluster_rank();
      warps = team_warps * static_cast<int>(ranks);
      warp = static_cast<int>(rank) * team_warps + w;
      first = static_cast<int>(rank) * (kMaxTeamWarps - team_warps);  // so that the slot is rank * 16 + w
      bar = 0;
    } else {
      warps = team_warps;
      warp = w % team_warps;
      first = w / team_warps * kMaxTeamWarps;
      bar = 1 + w / team_warps;
    }
    for (int i = threadIdx.x; i < 2 * kSlots; i += blockDim.x)
      slots[i / kSlots][i % kSlots] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    if constexpr (CLUSTER) cluster_barrier();
    else __syncthreads();
  }
  // index of this thread among the threads of the row, and their number
  __device__ __forceinline__ int thread() const { return warp * 32 + static_cast<int>(lane_id()); }
  __device__ __forceinline__ int threads() const { return warps * 32; }

  // v to a slot of CTA `to` of the cluster
  __device__ __forceinline__ static void store_slot(uint32_t to, const float4* slot, float4 v) {
    uint32_t remote;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(remote) : "r"(smem_u32(slot)), "r"(to));
    asm volatile("st.shared::cluster.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(remote), "f"(v.x), "f"(v.y), "f"(v.z), "f"(v.w)
                 : "memory");
  }
  // Every lane holds the warp's v: to the warp's slot, then the barrier.
  __device__ __forceinline__ void exchange(float4 v) {
    parity ^= 1;
    float4* mine = &slots[parity][first + warp];
    if constexpr (CLUSTER) {
      if (lane_id() < ranks) store_slot(lane_id(), mine, v);
      __syncwarp();
      cluster_barrier();
    } else {
      if (lane_id() == 0) *mine = v;
      __syncwarp();
      asm volatile("bar.sync %0, %1;" ::"r"(bar), "r"(warps * 32) : "memory");
    }
  }
  // The backward pass's sums through a cluster, taken in two halves around its other work: publish()
  // sends the warp's partial sums to its slot in every CTA, collect() waits until those of all warps have
  // arrived here and reads their sum into every lane. The stores carry their own completion (st.async on
  // a transaction barrier of the receiver): a cluster barrier in their place would have to order the
  // sender's other accesses too, and waits for its fetches of the rows ahead (16384 x 8192: 464 us so).
  // Two barriers and sets of slots in turn. A warp sends to a set again after its next collect(), for which
  // every warp has sent, and before that read, the sums of the set: nothing is overwritten unread.
  // FOUR values or two (v.x and v.z) share one butterfly: each of its first steps halves the number
  // of values a lane carries, so that four cost 6 shuffles instead of 20.
  template <bool FOUR>
  __device__ __forceinline__ float fold(float4 v) const {
    const bool upper = (lane_id() & 16u) != 0;
    float r;
    if constexpr (FOUR) {
      float x = upper ? v.z : v.x, y = upper ? v.w : v.y;
      x += __shfl_xor_sync(0xffffffffu, upper ? v.x : v.z, 16);
      y += __shfl_xor_sync(0xffffffffu, upper ? v.y : v.w, 16);
      const bool odd = (lane_id() & 8u) != 0;
      r = odd ? y : x;
      r += __shfl_xor_sync(0xffffffffu, odd ? x : y, 8);
    } else {
      r = upper ? v.z : v.x;
      r += __shfl_xor_sync(0xffffffffu, upper ? v.x : v.z, 16);
      r += __shfl_xor_sync(0xffffffffu, r, 8);
    }
#pragma unroll
    for (int m = 4; m > 0; m >>= 1) r += __shfl_xor_sync(0xffffffffu, r, m);
    return r;  // lanes 0-7 v.x, 8-15 v.y, 16-23 v.z, 24-31 v.w
  }
  template <bool FOUR>
  __device__ __forceinline__ void publish(float4 v) {
    const float4 all = unfold<FOUR>(fold<FOUR>(v));
    parity ^= 1;
    if (threadIdx.x == 0) mbar_arrive_expect_tx(&ring_bars[parity], static_cast<uint32_t>(warps) * 16u);
    if (lane_id() < ranks) {
      uint32_t slot, bar_at;
      asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(slot) : "r"(smem_u32(&slots[parity][first + warp])), "r"(lane_id()));
      asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(bar_at) : "r"(smem_u32(&ring_bars[parity])), "r"(lane_id()));
      asm volatile("st.async.weak.shared::cluster.mbarrier::complete_tx::bytes.v4.f32 [%0], {%1, %2, %3, %4}, [%5];" ::"r"(slot),
                   "f"(all.x), "f"(all.y), "f"(all.z), "f"(all.w), "r"(bar_at)
                   : "memory");
    }
    __syncwarp();
  }
  template <bool FOUR>
  __device__ __forceinline__ float4 unfold(float r) const {
    float4 v;
    v.x = __shfl_sync(0xffffffffu, r, 0);
    v.y = FOUR ? __shfl_sync(0xffffffffu, r, 8) : 0.0f;
    v.z = __shfl_sync(0xffffffffu, r, 16);
    v.w = FOUR ? __shfl_sync(0xffffffffu, r, 24) : 0.0f;
    return v;
  }
  template <bool FOUR>
  __device__ __forceinline__ float4 collect() {
    ok = mbar_wait_bounded_warp(&ring_bars[parity], phases >> parity & 1u, abort, status, wait_ns);
    phases ^= 1u << parity;
    if (!ok) return make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    const float* base = &slots[parity][0].x + (lane_id() >> 3) + 4 * (lane_id() & 7u);
    float r = base[0] + base[32];
    for (uint32_t k = 1; k < ranks; ++k) r += base[64 * k] + base[64 * k + 32];
#pragma unroll
    for (int m = 4; m > 0; m >>= 1) r += __shfl_xor_sync(0xffffffffu, r, m);
    return unfold<FOUR>(r);
  }
  // Sums of a and (TWO) b over the row, in every thread. Two sums share one butterfly: after its first
  // step the lower half of the warp carries a and the upper half b; the same goes for the slots.
  template <bool TWO>
  __device__ __forceinline__ float2 sum(float a, float b) {
    const bool upper = (lane_id() & 16u) != 0;
    float v;
    if constexpr (TWO) {
      v = upper ? b : a;
      v += __shfl_xor_sync(0xffffffffu, upper ? a : b, 16);
    } else {
      v = a + __shfl_xor_sync(0xffffffffu, a, 16);
    }
#pragma unroll
    for (int m = 8; m > 0; m >>= 1) v += __shfl_xor_sync(0xffffffffu, v, m);
    if (warps > 1) {
      if constexpr (CLUSTER) {
        const float v0 = __shfl_sync(0xffffffffu, v, 0), v1 = __shfl_sync(0xffffffffu, v, 16);
        exchange(make_float4(v0, v1, 0.0f, 0.0f));
      } else {
        parity ^= 1;
        float* mine = &slots[parity][first + warp].x;
        if ((lane_id() & 15u) == 0) mine[upper ? 1 : 0] = v;
        __syncwarp();
        asm volatile("bar.sync %0, %1;" ::"r"(bar), "r"(warps * 32) : "memory");
      }
      const float* base = &slots[parity][CLUSTER ? 0 : first].x + (upper ? 1 : 0) + 4 * (lane_id() & 15u);
      v = base[0];
      if constexpr (CLUSTER) {
        for (uint32_t k = 1; k < ranks; ++k) v += base[64 * k];
      }
#pragma unroll
      for (int m = 8; m > 0; m >>= 1) v += __shfl_xor_sync(0xffffffffu, v, m);
    }
    if constexpr (!TWO) return make_float2(v, 0.0f);
    return make_float2(__shfl_sync(0xffffffffu, v, 0), __shfl_sync(0xffffffffu, v, 16));
  }
};

// ---------------------------------------------------------------- a row's columns
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, uint32_t bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ uint4 load_shared16(uint32_t src) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(src)
               : "memory");
  return v;
}
__device__ __forceinline__ void load_shared_pairs(uint32_t src, f32x2& a, f32x2& b) {
  float x, y, z, w;
  asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(x), "=f"(y), "=f"(z), "=f"(w) : "r"(src) : "memory");
  a = pair(x, y), b = pair(z, w);
}
__device__ __forceinline__ void store_shared16(uint32_t dst, uint4 v) {
  asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(dst), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w)
               : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// The elements of a row that a thread holds, EPT / 2 pairs: N vectors of VEC consecutive columns, the
// i-th from column c0(i) on. Columns outside the row (lanes past its end and, with EDGE, the parts
// of the first and last vector that belong to the neighbouring rows) count as zeros with weight
// zero. How it is read:
//   kVectors  rows are whole 16-byte vectors
//   kEdges    rows begin and end inside vectors (EDGE)
//   kSingles  the matrices' rows are aligned in different ways: element by element
enum Reads { kVectors, kEdges, kSingles };

template <typename T, int EPT, int READS>
struct Columns {
  static constexpr int VEC = READS == kSingles ? 1 : 16 / static_cast<int>(sizeof(T));
  static constexpr int N = EPT / VEC;
  int first, step, cols;  // column of vector 0, distance of the next

  __device__ __forceinline__ int c0(int i) const { return first + i * step; }
  __device__ __forceinline__ bool in(int i) const { return c0(i) < cols; }
  __device__ __forceinline__ int col(int k) const { return c0(k / VEC) + k % VEC; }
  __device__ __forceinline__ bool has(int k) const {
    return READS == kEdges ? static_cast<uint32_t>(col(k)) < static_cast<uint32_t>(cols) : in(k / VEC);
  }
  // a vector with elements of neighbouring rows
  __device__ __forceinline__ bool cut(int i) const {
    return READS == kEdges && (c0(i) < 0 || (c0(i) < cols && c0(i) + VEC > cols));
  }
  // Groups of elements that are masked together: vectors, or pairs of single elements.
  static constexpr int GROUPS = VEC > 1 ? N : EPT / 2;
  __device__ __forceinline__ bool live(int i) const { return VEC > 1 ? in(i) : in(2 * i); }
  // zeros in the elements of group i outside the row
  __device__ __forceinline__ void mask(int i, f32x2* v) const {
    if constexpr (VEC == 1) {
      if (!in(2 * i)) v[0].x = 0.0f;
      if (!in(2 * i + 1)) v[0].y = 0.0f;
    } else if (cut(i)) {
#pragma unroll
      for (int e = 0; e < VEC; ++e)
        if (!has(i * VEC + e)) (e % 2 ? v[e / 2].y : v[e / 2].x) = 0.0f;
    }
  }
  // p[base + column] (bf16 or fp32) + offset, zero outside the row; `none` where there is no p
  __device__ __forceinline__ void params(const void* p, bool f32, int64_t base, float offset, float none,
                                         f32x2 (&v)[EPT / 2]) const {
    float f[EPT];
#pragma unroll
    for (int i = 0; i < N; ++i) {
      if (p == nullptr) {
#pragma unroll
        for (int e = 0; e < VEC; ++e) f[i * VEC + e] = none;
      } else if (READS == kVectors) {
        if (in(i)) load_param<VEC>(p, f32, base + c0(i), f + i * VEC);
      } else {
#pragma unroll
        for (int e = 0; e < VEC; ++e)
          if (has(i * VEC + e)) load_param<1>(p, f32, base + col(i * VEC + e), f + i * VEC + e);
      }
    }
#pragma unroll
    for (int k = 0; k < EPT; ++k) f[k] = !has(k) ? 0.0f : p != nullptr ? f[k] + offset : f[k];
#pragma unroll
    for (int k = 0; k < EPT / 2; ++k) v[k] = pair(f[2 * k], f[2 * k + 1]);
  }
  // Pairs 2 q and 2 q + 1 of the same.
  __device__ __forceinline__ void params4(const void* p, bool f32, int64_t base, float offset, float none, int q,
                                          f32x2& lo, f32x2& hi) const {
    float f[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) f[e] = none;
    if (p != nullptr) {
      if constexpr (READS == kVectors) {
        if (in(4 * q / VEC)) load_param<4>(p, f32, base + col(4 * q), f);
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (has(4 * q + e)) load_param<1>(p, f32, base + col(4 * q + e), f + e);
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) f[e] += offset;
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) f[e] = has(4 * q + e) ? f[e] : 0.0f;
    lo = pair(f[0], f[1]), hi = pair(f[2], f[3]);
  }
  // `first_at`: where the element of column `first` stands
  __device__ __forceinline__ void store(T* first_at, const f32x2 (&v)[EPT / 2]) const {
    if constexpr (READS == kSingles) {
#pragma unroll
      for (int k = 0; k < EPT; ++k)
        if (in(k)) {
          const float2 h = halves(v[k / 2]);
          Vec<T, false>::store(first_at + k * step, k % 2 ? &h.y : &h.x);
        }
    } else {
#pragma unroll
      for (int i = 0; i < N; ++i) {
        if (!in(i)) continue;
        if (!cut(i)) {
          *reinterpret_cast<uint4*>(first_at + i * step) = pack16<T>(&v[i * VEC / 2]);
        } else {
#pragma unroll
          for (int k = i * VEC; k < (i + 1) * VEC; ++k)
            if (has(k)) {
              const float2 h = halves(v[k / 2]);
              Vec<T, false>::store(first_at + i * step + k % VEC, k % 2 ? &h.y : &h.x);
            }
        }
      }
    }
  }
};


// ---------------------------------------------------------------- launches
// How a pass over rows is cut: warps of a row in a CTA, teams of a CTA, CTAs of a row.
struct RowCut {
  int reads, ept, warps, teams, cluster;  // ept: elements of a row in a thread
  int64_t classes;
  int32_t shift;
  int threads() const { return warps * teams * 32; }
};
// In how many ways rows of `cols` elements start inside a vector.
int64_t row_classes(int64_t cols, int64_t vec) {
  int64_t g = vec;
  while (cols % g != 0) g /= 2;
  return vec / g;
}
RowCut row_cut(int64_t cols, bool f32, bool wide, int64_t shift, bool forward) {
  RowCut c{};
  const int64_t vec = wide ? (f32 ? 4 : 8) : 1;
  c.classes = wide ? row_classes(cols, vec) : 1;
  c.reads = !wide ? kSingles : c.classes > 1 ? kEdges : kVectors;
  c.shift = static_cast<int32_t>(wide ? std::max<int64_t>(0, shift) : 0);
  const int64_t cover = cols + (c.classes > 1 ? vec - 1 : 0);  // a row that starts inside a vector
  c.ept = !forward || cover <= 256 ? 8 : cover <= 512 || f32 ? 16 : 32;
  c.cluster = static_cast<int>(ceil_div(cover, kMaxTeamWarps * 32 * c.ept));
  // 65530 to 65535 bf16 columns with 8 elements a thread: one vector too many for a cluster, which single elements are not
  if (c.cluster > kMaxCluster) return row_cut(cols, f32, false, 0, forward);
  c.warps = static_cast<int>(ceil_div(cover, 32 * c.ept * c.cluster));
  c.teams = c.cluster > 1 ? 1 : kMaxTeamWarps / c.warps;
  return c;
}
struct Matrix {
  const void* p;
  int64_t stride;
};
// Vectors: row r of every matrix starts at the same offset inside 16 bytes (*shift: row 0's).
bool same_offsets(std::initializer_list<Matrix> mats, int64_t cols, int64_t es, int64_t* shift) {
  *shift = -1;
  for (const Matrix& m : mats) {
    if (m.p == nullptr) continue;
    const int64_t at = static_cast<int64_t>(reinterpret_cast<uintptr_t>(m.p) & 15u) / es;
    if (*shift < 0) *shift = at;
    if (at != *shift || (m.stride - cols) % (16 / es) != 0) return false;
  }
  return true;
}

template <typename Params>
cudaError_t launch_cut(void (*kernel)(Params), const Params& a, int64_t ctas, const RowCut& c, size_t dynamic,
                       cudaStream_t stream) {
  return launch_in_stream(kernel, dim3(static_cast<unsigned>(ctas * c.cluster)), c.threads(), dynamic, stream, c.cluster, a);
}
cudaError_t allow(const void* kernel, size_t dynamic, bool cluster) {
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(dynamic));
  if (cluster && e == cudaSuccess) e = cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
  return e;
}

}  // namespace
}  // namespace bsq
