// bsq_norm.cu -- the norms before and after a block, fused with the block's gate and the residual
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
// in registers by a team of 1 to 16 warps (two 16-byte vectors a lane and matrix), or by a cluster
// of CTAs with 16 warps each for longer rows, so that it is read once although its statistics come
// first.
#include <algorithm>

#include "bsq.h"
#include "bsq_device.cuh"
#include "bsq_elem.cuh"
#include "bsq_internal.h"

namespace bsq {
namespace {

constexpr int kMaxTeamWarps = 16;
constexpr int kMaxCluster = 16;

struct NormParams {
  int64_t rows, group_rows;  // group_rows: rows that share a gate row
  int32_t cols, nvec;        // nvec: vectors (or scalars) in a row
  int32_t warps, teams;      // warps of a team in one CTA; teams of a CTA
  float eps, residual_scale, weight_offset;
  bool params_f32, post;
  const void *h, *x;
  int64_t h_stride, x_stride;
  const void *post_weight, *post_bias, *gate, *pre_weight, *pre_bias;
  void *x_out, *y;
  float4* stats;
};

// ---------------------------------------------------------------- element access
template <typename T, bool WIDE>
struct Access {
  static constexpr int kVec = Vec<T, WIDE>::kVec;
  static constexpr int kNum = WIDE ? 2 : 32 / static_cast<int>(sizeof(T));  // vectors a lane and matrix
};

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
__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ uint32_t cluster_size() {
  uint32_t r;
  asm("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_barrier() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

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
    for (int i = threadIdx.x; i < 2 * kSlots; i += blockDim.x) slots[0][i] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    if constexpr (CLUSTER) cluster_barrier();
    else __syncthreads();
  }
  // index of this thread among the threads of the row, and their number
  __device__ __forceinline__ int thread() const { return warp * 32 + static_cast<int>(lane_id()); }
  __device__ __forceinline__ int threads() const { return warps * 32; }

  // Every lane holds the warp's v: to the warp's slot, then the barrier.
  __device__ __forceinline__ void exchange(float4 v) {
    parity ^= 1;
    float4* mine = &slots[parity][first + warp];
    if constexpr (CLUSTER) {
      if (lane_id() < ranks) {
        uint32_t remote;
        asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(remote) : "r"(smem_u32(mine)), "r"(lane_id()));
        asm volatile("st.shared::cluster.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(remote), "f"(v.x), "f"(v.y), "f"(v.z),
                     "f"(v.w)
                     : "memory");
      }
      __syncwarp();
      cluster_barrier();
    } else {
      if (lane_id() == 0) *mine = v;
      asm volatile("bar.sync %0, %1;" ::"r"(bar), "r"(warps * 32) : "memory");
    }
  }
  // The backward pass's sums, taken in two halves around its other work: publish() leaves the warp's
  // partial sums in its slot behind the barrier, collect() reads the slots' sum into every lane.
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
  __device__ __forceinline__ float publish(float4 v) {
    const float r = fold<FOUR>(v);
    if (warps > 1) {
      parity ^= 1;
      if constexpr (CLUSTER) {
        const float4 all = unfold<FOUR>(r);
        parity ^= 1;
        exchange(all);
      } else {
        float* mine = &slots[parity][first + warp].x;
        if ((lane_id() & 7u) == 0) mine[lane_id() >> 3] = r;
        asm volatile("bar.sync %0, %1;" ::"r"(bar), "r"(warps * 32) : "memory");
      }
    }
    return r;
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
  __device__ __forceinline__ float4 collect(float r) const {
    if (warps > 1) {
      const float* base = &slots[parity][CLUSTER ? 0 : first].x + (lane_id() >> 3) + 4 * (lane_id() & 7u);
      r = base[0] + base[32];
      if constexpr (CLUSTER)
        for (uint32_t k = 1; k < ranks; ++k) r += base[64 * k] + base[64 * k + 32];
#pragma unroll
      for (int m = 4; m > 0; m >>= 1) r += __shfl_xor_sync(0xffffffffu, r, m);
    }
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
        asm volatile("bar.sync %0, %1;" ::"r"(bar), "r"(warps * 32) : "memory");
      }
      const float* base = &slots[parity][CLUSTER ? 0 : first].x + (upper ? 1 : 0) + 4 * (lane_id() & 15u);
      v = base[0];
      if constexpr (CLUSTER)
        for (uint32_t k = 1; k < ranks; ++k) v += base[64 * k];
#pragma unroll
      for (int m = 8; m > 0; m >>= 1) v += __shfl_xor_sync(0xffffffffu, v, m);
    }
    if constexpr (!TWO) return make_float2(v, 0.0f);
    return make_float2(__shfl_sync(0xffffffffu, v, 0), __shfl_sync(0xffffffffu, v, 16));
  }
};

// mean and 1 / sqrt(mean((v - mean)^2) + eps) of a row. The layer norm's second moment is taken
// about each warp's own mean, in a second pass over its registers, and moved to the row's mean when
// the warps join (sum of M2_w + n_w (mean_w - mean)^2): as exact as two passes over the row, with
// one exchange.
template <bool LAYER, bool CLUSTER, int N, int VEC>
__device__ __forceinline__ float2 row_stats(Team<CLUSTER>& team, const float (&v)[N][VEC], const bool (&in)[N],
                                            float n_warp, float inv_cols, float eps) {
  if constexpr (!LAYER) {
    float q = 0.0f;
#pragma unroll
    for (int i = 0; i < N; ++i)
#pragma unroll
      for (int e = 0; e < VEC; ++e) q += v[i][e] * v[i][e];
    const float2 t = team.template sum<false>(q, 0.0f);
    return make_float2(0.0f, 1.0f / sqrtf(t.x * inv_cols + eps));
  } else {
    float s = 0.0f;
#pragma unroll
    for (int i = 0; i < N; ++i)
#pragma unroll
      for (int e = 0; e < VEC; ++e) s += v[i][e];
    s = warp_sum(s);
    const float mw = n_warp > 0.0f ? s / n_warp : 0.0f;
    float q = 0.0f;
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (in[i]) {
#pragma unroll
        for (int e = 0; e < VEC; ++e) q += (v[i][e] - mw) * (v[i][e] - mw);
      }
    q = warp_sum(q);
    if (team.warps == 1) return make_float2(mw, 1.0f / sqrtf(q * inv_cols + eps));
    team.exchange(make_float4(s, q, n_warp, mw));
    float mean = 0.0f, m2 = 0.0f;
    // slots of no warp hold zeros
    const float4* slot = &team.slots[team.parity][CLUSTER ? 0 : team.first];
    const int n = CLUSTER ? static_cast<int>(team.ranks) * kMaxTeamWarps : team.warps;
    for (int i = 0; i < n; ++i) mean += slot[i].x;
    mean *= inv_cols;
    for (int i = 0; i < n; ++i) {
      const float4 p = slot[i];
      const float d = p.w - mean;
      m2 += p.y + p.z * d * d;
    }
    return make_float2(mean, 1.0f / sqrtf(m2 * inv_cols + eps));
  }
}

// ---------------------------------------------------------------- forward
template <typename T, bool WIDE, bool LAYER, bool CLUSTER>
__global__ void __launch_bounds__(kMaxTeamWarps * 32) norm_forward_kernel(const NormParams a) {
  constexpr int VEC = Access<T, WIDE>::kVec, N = Access<T, WIDE>::kNum;
  __shared__ float4 slots[2][Team<CLUSTER>::kSlots];
  Team<CLUSTER> team;
  team.init(slots, a.warps);
  const int64_t row = CLUSTER ? blockIdx.x / team.ranks
                              : static_cast<int64_t>(blockIdx.x) * a.teams + (threadIdx.x >> 5) / a.warps;
  if (row < a.rows) {
    const float inv_cols = 1.0f / static_cast<float>(a.cols);
    int col[N];
    bool in[N];
    float n_warp = 0.0f;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int v = i * team.threads() + team.thread();
      col[i] = v * VEC;
      in[i] = v < a.nvec;
      n_warp += in[i] ? static_cast<float>(VEC) : 0.0f;
    }
    if constexpr (LAYER) n_warp = warp_sum(n_warp);

    const T* x = static_cast<const T*>(a.x) + row * a.x_stride;
    Vec<T, WIDE> xr[N];
    float v[N][VEC];
    float4 st = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    if (a.h != nullptr) {
      const T* h = static_cast<const T*>(a.h) + row * a.h_stride;
      Vec<T, WIDE> hr[N];
#pragma unroll
      for (int i = 0; i < N; ++i) {
        hr[i].clear();
        xr[i].clear();
        if (in[i]) hr[i].load(h + col[i]);
        if (in[i]) xr[i].load(x + col[i]);
      }
#pragma unroll
      for (int i = 0; i < N; ++i) hr[i].get(v[i]);
      if (a.post) {
        const float2 s = row_stats<LAYER>(team, v, in, n_warp, inv_cols, a.eps);
        st.x = s.x;
        st.y = s.y;
#pragma unroll
        for (int i = 0; i < N; ++i)
          if (in[i]) {
            float w[VEC], b[VEC];
            load_weight<VEC>(a.post_weight, a.params_f32, a.weight_offset, col[i], w);
#pragma unroll
            for (int e = 0; e < VEC; ++e) b[e] = 0.0f;
            if (a.post_bias != nullptr) load_param<VEC>(a.post_bias, a.params_f32, col[i], b);
#pragma unroll
            for (int e = 0; e < VEC; ++e) v[i][e] = (v[i][e] - s.x) * s.y * w[e] + b[e];
          }
      }
      const int64_t gate_at = row / a.group_rows * a.cols;
#pragma unroll
      for (int i = 0; i < N; ++i)
        if (in[i]) {
          float xf[VEC];
          xr[i].get(xf);
          if (a.gate != nullptr) {
            float g[VEC];
            load_param<VEC>(a.gate, a.params_f32, gate_at + col[i], g);
#pragma unroll
            for (int e = 0; e < VEC; ++e) v[i][e] *= g[e];
          }
#pragma unroll
          for (int e = 0; e < VEC; ++e) v[i][e] += a.residual_scale * xf[e];
        }
    } else {
#pragma unroll
      for (int i = 0; i < N; ++i) {
        xr[i].clear();
        if (in[i]) xr[i].load(x + col[i]);
      }
#pragma unroll
      for (int i = 0; i < N; ++i) {
        xr[i].get(v[i]);
#pragma unroll
        for (int e = 0; e < VEC; ++e) v[i][e] *= a.residual_scale;
      }
    }
    if (a.x_out != nullptr) {
      T* o = static_cast<T*>(a.x_out) + row * a.cols;
#pragma unroll
      for (int i = 0; i < N; ++i)
        if (in[i]) Vec<T, WIDE>::store(o + col[i], v[i]);
    }
    if (a.y != nullptr) {
      const float2 s = row_stats<LAYER>(team, v, in, n_warp, inv_cols, a.eps);
      st.z = s.x;
      st.w = s.y;
      T* o = static_cast<T*>(a.y) + row * a.cols;
#pragma unroll
      for (int i = 0; i < N; ++i)
        if (in[i]) {
          float w[VEC], b[VEC];
          load_weight<VEC>(a.pre_weight, a.params_f32, a.weight_offset, col[i], w);
#pragma unroll
          for (int e = 0; e < VEC; ++e) b[e] = 0.0f;
          if (a.pre_bias != nullptr) load_param<VEC>(a.pre_bias, a.params_f32, col[i], b);
#pragma unroll
          for (int e = 0; e < VEC; ++e) v[i][e] = (v[i][e] - s.x) * s.y * w[e] + b[e];
          Vec<T, WIDE>::store(o + col[i], v[i]);
        }
    }
    if (a.stats != nullptr && team.thread() == 0) a.stats[row] = st;
  }
  if constexpr (CLUSTER) cluster_barrier();  // no CTA leaves while another may still write its slots
}

// ---------------------------------------------------------------- backward
// A block of rows_per_block consecutive rows is shared by `classes` CTAs (or clusters); a CTA walks
// its rows by the segments that share a gate row, its teams taking them in turn, and keeps the
// column sums in registers. A segment's A1, A0 go to slot (block + gate row) * classes + class of
// ws1 -- consecutive segments differ in block or gate row, so no two share a slot -- and the
// pre-norm's sums to slot block * classes + class of ws2.
//
// Rows whose length is no multiple of 16 bytes begin at different offsets inside a 16-byte vector,
// in a cycle of `classes` rows. A CTA takes the rows of one class alone, so that a thread's vectors
// hold the same columns in every row; the vectors at a row's two ends also hold elements of its
// neighbours, which are masked when read and not written.
//
// The rows ahead are fetched by cp.async into a ring of shared memory in which every thread reads
// only what it fetched itself: no barrier, and the loads in flight (one or two rows a team) do not
// take registers from the column sums.
// Stages of the ring: rows in flight and the one being read, within 227 KB at 512 threads.
template <typename T, int EPT>
constexpr int kRing = sizeof(T) == 4 ? 2 : 3;
constexpr int kGradElems = 8;   // elements of a matrix's row in a thread
constexpr int kGradWarps = 16;  // of a CTA; a bound of 64 registers for two such CTAs spills and is slower (16384 x 4096: 184 -> 403 us)
constexpr int kStageFloats = 4096;  // teams * cols of a CTA with several teams: 16 warps of 8 elements a lane

struct NormGradParams {
  int64_t rows, group_rows, rows_per_block;
  int32_t cols, warps, teams, classes;
  int32_t shift;  // elements from a 16-byte boundary to the first row
  float residual_scale, weight_offset;
  bool params_f32, post, sums1, sums2;
  const void *dy, *x_out, *dx_out, *h;
  int64_t dy_stride, x_out_stride, dx_out_stride, h_stride;
  const float4* stats;
  const void *post_weight, *gate, *pre_weight;
  void *dx, *dh;
  float *ws1, *ws2;  // partial sums: [slots][2][cols] each
};

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

template <typename T, int EPT, int READS>
__device__ __forceinline__ void flush_sums(const NormGradParams& a, f32x2 (&acc)[EPT / 2],
                                           const Columns<T, EPT, READS>& at, float* out, float* stage) {
  const bool join = a.teams > 1;  // teams join in order through shared memory
  float* to = join ? stage + (threadIdx.x >> 5) / a.warps * a.cols : out;
  if (join) __syncthreads();
#pragma unroll
  for (int k = 0; k < EPT; ++k)
    if (at.has(k)) {
      const float2 h = halves(acc[k / 2]);
      to[at.col(k)] = k % 2 ? h.y : h.x;
    }
  if (join) {
    __syncthreads();
    for (int c = threadIdx.x; c < a.cols; c += blockDim.x) {
      float s = 0.0f;
      for (int k = 0; k < a.teams; ++k) s += stage[k * a.cols + c];
      out[c] = s;
    }
  }
#pragma unroll
  for (int k = 0; k < EPT / 2; ++k) acc[k] = both(0.0f);
}

// One row takes three steps with a sum over the row between them:
//   A  z2, g2 from dy and x_out;              sums of g2 and g2 * z2
//   B  d from those and dx_out, dx; z1, g1;   sums of g1 and g1 * z1
//   C  dh
// A CTA takes them in turn. In a cluster, where an exchange costs a trip between SMs, an iteration
// takes step A of row i, B of row i - 1 and C of row i - 2: the sums of two rows share one exchange,
// and A, which needs none, runs while they come in (16384 x 8192: 681 us in turn, 527 us so; in one
// CTA the registers it takes cost more than it gives, 184 us in turn and 240 us so at 16384 x 4096).
// Rows outside the segment are then read as zeros and not written; a stage of the ring holds dy and
// x_out of row i, dx_out and h of row i - 1.
//
// EPT: elements a thread holds of each matrix's row. BIAS: whether A0 and dpre_bias are summed.
template <typename T, int EPT, int READS, bool LAYER, bool BIAS, bool CLUSTER>
__global__ void __launch_bounds__(kGradWarps * 32, 1) norm_backward_kernel(const NormGradParams a) {
  using Cols = Columns<T, EPT, READS>;
  constexpr int VEC = Cols::VEC, N = Cols::N, P = EPT / 2;
  constexpr bool RING = READS != kSingles;
  constexpr int kStages = kRing<T, EPT>;
  constexpr int BEHIND = CLUSTER ? 1 : 0;  // rows that dx_out and h lie behind dy and x_out
  extern __shared__ uint4 dynamic[];  // weights: [2][P / 2][threads of the team]; ring
  __shared__ float4 slots[2][Team<CLUSTER>::kSlots];
  __shared__ float stage[CLUSTER ? 1 : kStageFloats];  // [teams][cols]
  Team<CLUSTER> team;
  team.init(slots, a.warps);
  const int t = CLUSTER ? 0 : (threadIdx.x >> 5) / a.warps;
  const int64_t unit = CLUSTER ? blockIdx.x / team.ranks : blockIdx.x;
  const int64_t block = unit / a.classes;
  const int cls = static_cast<int>(unit % a.classes);
  const int lead = READS == kEdges ? static_cast<int>((a.shift + static_cast<int64_t>(cls) * a.cols) % VEC) : 0;
  const float inv_cols = 1.0f / static_cast<float>(a.cols);
  const Cols at{team.thread() * VEC - lead, team.threads() * VEC, a.cols};
  // rows and their numbers fit 32 bits; addresses advance by whole steps
  const int begin = static_cast<int>(block * a.rows_per_block);
  const int end = static_cast<int>(min(a.rows, (block + 1) * a.rows_per_block));
  const int step = a.classes * a.teams;
  const bool has[4] = {a.dy != nullptr, a.dy != nullptr, a.dx_out != nullptr, a.h != nullptr};
  // the block's rows of each matrix; offsets inside them fit 32 bits (the host sees to it)
  const T* base[4] = {static_cast<const T*>(a.dy) + begin * a.dy_stride, static_cast<const T*>(a.x_out) + begin * a.x_out_stride,
                      static_cast<const T*>(a.dx_out) + begin * a.dx_out_stride, static_cast<const T*>(a.h) + begin * a.h_stride};
  const int stride[4] = {static_cast<int>(a.dy_stride), static_cast<int>(a.x_out_stride),
                         static_cast<int>(a.dx_out_stride), static_cast<int>(a.h_stride)};
  T* const dx = static_cast<T*>(a.dx) + static_cast<int64_t>(begin) * a.cols;
  T* const dh = static_cast<T*>(a.dh) + static_cast<int64_t>(begin) * a.cols;

  // weights: this thread's pairs, 16 bytes (2 pairs) at a time
  const uint32_t team_threads = a.warps * 32;
  const uint32_t weight0 = smem_u32(dynamic) + (threadIdx.x - t * team_threads) * 16;
  const uint32_t weight_step = team_threads * 16;
  auto put_weight = [&](int which, const f32x2 (&w)[P]) {
#pragma unroll
    for (int k = 0; k < P / 2; ++k) {
      const float2 x = halves(w[2 * k]), y = halves(w[2 * k + 1]);
      store_shared16(weight0 + (which * (P / 2) + k) * weight_step,
                     make_uint4(__float_as_uint(x.x), __float_as_uint(x.y), __float_as_uint(y.x), __float_as_uint(y.y)));
    }
  };
  auto get_weight = [&](int which, f32x2 (&w)[P]) {
#pragma unroll
    for (int k = 0; k < P / 2; ++k) load_shared_pairs(weight0 + (which * (P / 2) + k) * weight_step, w[2 * k], w[2 * k + 1]);
  };
  if (t == 0) {
    f32x2 w[P];
    at.params(a.pre_weight, a.params_f32, 0, a.weight_offset, 1.0f, w);
    put_weight(0, w);
  }

  // ring: [kStages][warps][4][N][lanes] vectors; a warp's 16-byte copies land side by side (spread
  // over shared memory they read L2 sectors twice)
  const uint32_t stage_bytes = blockDim.x * (4 * N * 16);
  const uint32_t ring0 =
      smem_u32(dynamic) + P * weight_step + (threadIdx.x >> 5) * (4 * N * 512) + lane_id() * 16;
  const uint32_t ring_end = ring0 + kStages * stage_bytes;
  if constexpr (RING) {  // what is never fetched reads as zeros
#pragma unroll
    for (int s = 0; s < kStages; ++s)
#pragma unroll
      for (int m = 0; m < 4; ++m)
#pragma unroll
        for (int i = 0; i < N; ++i)
          if (!has[m] || !at.in(i)) store_shared16(ring0 + s * stage_bytes + (m * N + i) * 512, make_uint4(0, 0, 0, 0));
  }

  f32x2 a1[P] = {}, p1[P] = {};
  f32x2 a0[BIAS ? P : 1] = {}, p0[BIAS ? P : 1] = {};
  for (int seg = begin; seg < end;) {
    const int64_t group = seg / a.group_rows;
    const int seg_end = static_cast<int>(min(static_cast<int64_t>(end), (group + 1) * a.group_rows));
    if (t == 0) {  // gate * (post_weight + offset)
      f32x2 w[P];
      at.params(a.post ? a.post_weight : nullptr, a.params_f32, 0, a.weight_offset, 1.0f, w);
      if (a.gate != nullptr) {
        f32x2 g[P];
        at.params(a.gate, a.params_f32, group * a.cols, 0.0f, 1.0f, g);
#pragma unroll
        for (int k = 0; k < P; ++k) w[k] = mul2(w[k], g[k]);
      }
      put_weight(1, w);
    }
    __syncthreads();
    // this team's rows of the segment: first, first + step, ...
    const int mine = seg - begin + ((cls - (seg - begin)) % a.classes + a.classes) % a.classes;  // class's first row
    const int first = begin + mine + t * a.classes;
    const int n = first < seg_end ? (seg_end - first + step - 1) / step : 0;

    // the row to fetch next, and this thread's vector 0 of it in each matrix, as an offset from the
    // block's first row
    int ahead = 0;
    const int at_row = first - begin;
    int off[4];
#pragma unroll
    for (int m = 0; m < 4; ++m) off[m] = (m < 2 ? at_row : at_row - BEHIND * step) * stride[m] + at.first;
    auto fetch = [&](uint32_t to) {
      if constexpr (RING) {
        if (CLUSTER || ahead < n) {
          // rows outside the segment: nothing is read, zeros are written
          const uint32_t now = !CLUSTER || ahead < n ? 16 : 0;
          const uint32_t before = !CLUSTER || static_cast<uint32_t>(ahead - 1) < static_cast<uint32_t>(n) ? 16 : 0;
#pragma unroll
          for (int m = 0; m < 4; ++m) {
            if (has[m]) {
#pragma unroll
              for (int i = 0; i < N; ++i)
                if (at.in(i)) {
                  uint32_t bytes = m < 2 ? now : before;
                  // the last vector of a row stops at the row's end
                  if (READS == kEdges) bytes = min(bytes, (a.cols - at.c0(i)) * static_cast<uint32_t>(sizeof(T)));
                  cp_async16(to + (m * N + i) * 512, base[m] + (off[m] + i * at.step), bytes);
                }
            }
            off[m] += step * stride[m];
          }
        }
        ++ahead;
        cp_async_commit();
      }
    };
    // the pairs of matrix m at stage `from`, or of row k of the segment where there is no ring
    auto get = [&](uint32_t from, int m, int k, f32x2 (&v)[P]) {
      if constexpr (RING) {
#pragma unroll
        for (int i = 0; i < N; ++i) {
          unpack16<T>(load_shared16(from + (m * N + i) * 512), &v[i * VEC / 2]);
          if (at.cut(i)) {
#pragma unroll
            for (int e = i * VEC; e < (i + 1) * VEC; e += 2) {
              const float2 h = halves(v[e / 2]);
              v[e / 2] = pair(at.has(e) ? h.x : 0.0f, at.has(e + 1) ? h.y : 0.0f);
            }
          }
        }
      } else {
        float f[EPT];
        const bool live = has[m] && k >= 0 && k < n;
        const T* p = base[m] + (at_row + k * step) * static_cast<int64_t>(stride[m]);
#pragma unroll
        for (int e = 0; e < EPT; ++e) {
          Vec<T, false> r;
          r.clear();
          if (live && at.in(e)) r.load(p + at.c0(e));
          r.get(&f[e]);
        }
#pragma unroll
        for (int e = 0; e < P; ++e) v[e] = pair(f[2 * e], f[2 * e + 1]);
      }
    };
#pragma unroll
    for (int k = 0; k < kStages - 1; ++k) fetch(ring0 + k * stage_bytes);
    const float4* const stats = a.stats + first;
    float4 st_next = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    if (n > 0 && a.stats != nullptr) st_next = __ldg(stats);
    int out = at_row * a.cols + at.first;  // this thread's vector 0 of the row in the outputs
    uint32_t s = ring0, to = ring0 + (kStages - 1) * stage_bytes;  // stage to read, stage to fill
    if constexpr (!CLUSTER) {
      for (int it = 0; it < n; ++it) {
        fetch(to);
        const float4 st = st_next;
        if (it + 1 < n && a.stats != nullptr) st_next = __ldg(stats + (it + 1) * step);
        if constexpr (RING) cp_async_wait<kStages - 1>();
        f32x2 d[P], z[P], w[P];
        if (a.dy != nullptr) {
          f32x2 g[P];
          get(s, 0, it, g);
          get(s, 1, it, z);
          get_weight(0, w);
          f32x2 s0 = both(0.0f), s1 = s0;
          const f32x2 mean = both(-st.z), rstd = both(st.w);
  #pragma unroll
          for (int k = 0; k < P; ++k) {
            if (LAYER) z[k] = add2(z[k], mean);
            z[k] = mul2(z[k], rstd);
            if (BIAS) p0[k] = add2(p0[k], g[k]);
            p1[k] = fma2(g[k], z[k], p1[k]);
            g[k] = mul2(g[k], w[k]);
            if (LAYER) s0 = add2(s0, g[k]);
            s1 = fma2(g[k], z[k], s1);
          }
          const float2 sum = team.template sum<LAYER>(sum_halves(s1), LAYER ? sum_halves(s0) : 0.0f);
          const f32x2 m1 = both(-sum.x * inv_cols * st.w), m0 = both(-sum.y * inv_cols * st.w);
          get(s, 2, it, d);
  #pragma unroll
          for (int k = 0; k < P; ++k) {
            if (LAYER) d[k] = add2(d[k], m0);
            d[k] = fma2(z[k], m1, fma2(g[k], rstd, d[k]));
          }
        } else {
          get(s, 2, it, d);
        }
        if (a.dx != nullptr) {
          f32x2 o[P];
          const f32x2 scale = both(a.residual_scale);
  #pragma unroll
          for (int k = 0; k < P; ++k) o[k] = mul2(d[k], scale);
          at.store(dx + out, o);
        }
        if (a.dh != nullptr || a.sums1) {
          get(s, 3, it, z);
          get_weight(1, w);
          f32x2 s0 = both(0.0f), s1 = s0;
          const f32x2 mean = both(a.post ? -st.x : 0.0f), rstd = both(a.post ? st.y : 1.0f);
  #pragma unroll
          for (int k = 0; k < P; ++k) {
            if (LAYER) z[k] = add2(z[k], mean);
            z[k] = mul2(z[k], rstd);
            if (BIAS) a0[k] = add2(a0[k], d[k]);
            a1[k] = fma2(d[k], z[k], a1[k]);
            d[k] = mul2(d[k], w[k]);
            if (LAYER) s0 = add2(s0, d[k]);
            s1 = fma2(d[k], z[k], s1);
          }
          if (a.post) {
            const float2 sum = team.template sum<LAYER>(sum_halves(s1), LAYER ? sum_halves(s0) : 0.0f);
            const f32x2 m1 = both(-sum.x * inv_cols * st.y), m0 = both(-sum.y * inv_cols * st.y);
  #pragma unroll
            for (int k = 0; k < P; ++k) {
              d[k] = fma2(z[k], m1, mul2(d[k], rstd));
              if (LAYER) d[k] = add2(d[k], m0);
            }
          }
          if (a.dh != nullptr) at.store(dh + out, d);
        }
        out += step * a.cols;
        to = s;  // read for the last time above
        s += stage_bytes;
        if (s == ring_end) s = ring0;
      }
    } else {
      f32x2 g[P] = {}, z2[P] = {}, d[P] = {}, z1[P] = {};
      float4 st_a = make_float4(0.0f, 0.0f, 0.0f, 0.0f), st_b = st_a;
      float rstd_c = 0.0f, folded = 0.0f;
      const int iterations = n > 0 ? n + 2 : 0;
      for (int it = 0; it < iterations; ++it) {
        fetch(to);
        rstd_c = a.post ? st_b.y : 1.0f;
        st_b = st_a;
        st_a = st_next;
        st_next = it + 1 < n && a.stats != nullptr ? __ldg(stats + (it + 1) * step) : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        if constexpr (RING) cp_async_wait<kStages - 1>();
        // A
        f32x2 gn[P], zn[P], w[P];
        f32x2 s0 = both(0.0f), s1 = s0;
        get(s, 0, it, gn);
        get(s, 1, it, zn);
        get_weight(0, w);
        {
          const f32x2 mean = both(-st_a.z), rstd = both(st_a.w);
  #pragma unroll
          for (int k = 0; k < P; ++k) {
            if (LAYER) zn[k] = add2(zn[k], mean);
            zn[k] = mul2(zn[k], rstd);
            if (BIAS) p0[k] = add2(p0[k], gn[k]);
            p1[k] = fma2(gn[k], zn[k], p1[k]);
            gn[k] = mul2(gn[k], w[k]);
            if (LAYER) s0 = add2(s0, gn[k]);
            s1 = fma2(gn[k], zn[k], s1);
          }
        }
        const float4 sums = team.template collect<LAYER>(folded);  // of A's row i - 1 and B's row i - 2
        // C
        {
          const float f = a.post ? -inv_cols * rstd_c : 0.0f;
          const f32x2 m1 = both(sums.z * f), m0 = both(sums.w * f), rstd = both(rstd_c);
          if (a.dh != nullptr && it >= 2) {
  #pragma unroll
            for (int k = 0; k < P; ++k) {
              d[k] = fma2(z1[k], m1, mul2(d[k], rstd));
              if (LAYER) d[k] = add2(d[k], m0);
            }
            at.store(dh + (out - 2 * step * a.cols), d);
          }
        }
        // B
        f32x2 t0 = both(0.0f), t1 = t0;
        {
          const float f = -inv_cols * st_b.w;
          const f32x2 m1 = both(sums.x * f), m0 = both(sums.y * f), rstd = both(st_b.w);
          get(s, 2, it - 1, d);
  #pragma unroll
          for (int k = 0; k < P; ++k) {
            if (LAYER) d[k] = add2(d[k], m0);
            d[k] = fma2(z2[k], m1, fma2(g[k], rstd, d[k]));
          }
          if (a.dx != nullptr && static_cast<uint32_t>(it - 1) < static_cast<uint32_t>(n)) {
            f32x2 o[P];
            const f32x2 scale = both(a.residual_scale);
  #pragma unroll
            for (int k = 0; k < P; ++k) o[k] = mul2(d[k], scale);
            at.store(dx + (out - step * a.cols), o);
          }
        }
        {
          const f32x2 mean = both(a.post ? -st_b.x : 0.0f), rstd = both(a.post ? st_b.y : 1.0f);
          get(s, 3, it - 1, z1);
          get_weight(1, w);
  #pragma unroll
          for (int k = 0; k < P; ++k) {
            if (LAYER) z1[k] = add2(z1[k], mean);
            z1[k] = mul2(z1[k], rstd);
            if (BIAS) a0[k] = add2(a0[k], d[k]);
            a1[k] = fma2(d[k], z1[k], a1[k]);
            d[k] = mul2(d[k], w[k]);
            if (LAYER) t0 = add2(t0, d[k]);
            t1 = fma2(d[k], z1[k], t1);
            g[k] = gn[k];
            z2[k] = zn[k];
          }
        }
        folded = team.template publish<LAYER>(
            make_float4(sum_halves(s1), LAYER ? sum_halves(s0) : 0.0f, sum_halves(t1), LAYER ? sum_halves(t0) : 0.0f));
        out += step * a.cols;
        to = s;  // read for the last time above
        s += stage_bytes;
        if (s == ring_end) s = ring0;
      }
    }
    if constexpr (RING) cp_async_wait<0>();
    if (a.sums1) {
      float* sums = a.ws1 + ((block + group) * a.classes + cls) * 2 * a.cols;
      flush_sums(a, a1, at, sums, stage);
      if constexpr (BIAS) flush_sums(a, a0, at, sums + a.cols, stage);
    }
    seg = seg_end;
    if (seg < end) __syncthreads();  // the gate's weights are read no more
  }
  launch_dependents();
  if (a.sums2) {
    float* out = a.ws2 + unit * 2 * a.cols;
    flush_sums(a, p1, at, out, stage);
    if constexpr (BIAS) flush_sums(a, p0, at, out + a.cols, stage);
  }
  if constexpr (CLUSTER) cluster_barrier();  // no CTA leaves while another may still write its slots
}

// ---------------------------------------------------------------- parameter gradients
struct NormSums {
  int64_t rows, group_rows, groups, rows_per_block, units;  // units: slots of ws2
  int32_t cols, classes;
  float weight_offset;
  bool params_f32, bias;  // bias: whether A0 and dpre_bias were summed
  const void *post_weight, *post_bias, *gate;
  const float *ws1, *ws2;
  float *dpost_weight, *dpost_bias, *dgate, *dpre_weight, *dpre_bias;
};
constexpr int kSumWarps = 32;

// 32 columns a CTA (one a lane); its warps share the slots of a sum, in a fixed order. blockIdx.y: 0 the
// pre-norm's sums, 1 the post norm's and the gate's.
__global__ void __launch_bounds__(kSumWarps * 32) norm_sums_kernel(const NormSums a) {
  __shared__ float2 part[kSumWarps][32];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int c = blockIdx.x * 32 + lane;
  const bool in = c < a.cols;
  grid_dependency_wait();
  // all warps: the sum of `n` slots from `base`, returned to warp 0
  auto joined = [&](const float* base, int64_t n) {
    float2 s = make_float2(0.0f, 0.0f);
    if (in) {
#pragma unroll 8
      for (int64_t i = warp; i < n; i += kSumWarps) {
        const float* p = base + i * 2 * a.cols + c;
        s.x += p[0];
        if (a.bias) s.y += p[a.cols];
      }
    }
    __syncthreads();
    part[warp][lane] = s;
    __syncthreads();
    if (warp == 0)
      for (int w = 1; w < kSumWarps; ++w) s.x += part[w][lane].x, s.y += part[w][lane].y;
    return s;
  };
  if (blockIdx.y == 0) {
    if (a.dpre_weight == nullptr && a.dpre_bias == nullptr) return;
    const float2 s = joined(a.ws2, a.units);
    if (warp == 0 && in) {
      if (a.dpre_weight != nullptr) a.dpre_weight[c] = s.x;
      if (a.dpre_bias != nullptr) a.dpre_bias[c] = s.y;
    }
    return;
  }
  float w = 1.0f, b = 0.0f;
  if (in) {
    load_weight<1>(a.post_weight, a.params_f32, a.weight_offset, c, &w);
    if (a.post_bias != nullptr) load_param<1>(a.post_bias, a.params_f32, c, &b);
  }
  float2 total = make_float2(0.0f, 0.0f);  // of gate * (A1, A0)
  auto add_group = [&](int64_t g, float2 s) {
    float gate = 1.0f;
    if (a.gate != nullptr) load_param<1>(a.gate, a.params_f32, g * a.cols + c, &gate);
    if (a.dgate != nullptr) a.dgate[g * a.cols + c] = a.bias ? w * s.x + b * s.y : w * s.x;
    total.x += gate * s.x;
    total.y += gate * s.y;
  };
  // the slots of gate row g: those of the blocks whose rows meet it
  auto slots_of = [&](int64_t g, int64_t& n) {
    const int64_t b0 = g * a.group_rows / a.rows_per_block;
    const int64_t b1 = (min(a.rows, (g + 1) * a.group_rows) - 1) / a.rows_per_block;
    n = (b1 - b0 + 1) * a.classes;
    return a.ws1 + (b0 + g) * a.classes * 2 * a.cols;
  };
  if (a.groups < kSumWarps) {
    for (int64_t g = 0; g < a.groups; ++g) {
      int64_t n;
      const float* base = slots_of(g, n);
      const float2 s = joined(base, n);
      if (warp == 0 && in) add_group(g, s);
    }
  } else {  // a warp for each gate row
    if (in)
      for (int64_t g = warp; g < a.groups; g += kSumWarps) {
        float2 s = make_float2(0.0f, 0.0f);
        int64_t n;
        const float* base = slots_of(g, n) + c;
        for (int64_t i = 0; i < n; ++i) {
          s.x += base[i * 2 * a.cols];
          if (a.bias) s.y += base[i * 2 * a.cols + a.cols];
        }
        add_group(g, s);
      }
    __syncthreads();
    part[warp][lane] = total;
    __syncthreads();
    if (warp == 0)
      for (int k = 1; k < kSumWarps; ++k) total.x += part[k][lane].x, total.y += part[k][lane].y;
  }
  if (warp == 0 && in) {
    if (a.dpost_weight != nullptr) a.dpost_weight[c] = total.x;
    if (a.dpost_bias != nullptr) a.dpost_bias[c] = total.y;
  }
}

// ---------------------------------------------------------------- launches
struct NormShape {
  int warps, teams, cluster;  // warps of a team in a CTA, teams of a CTA, CTAs of a cluster
  int threads() const { return warps * teams * 32; }
};

// Warps for a row: as many as hold it at 32 bytes a lane and matrix; CTAs of 8 warps while a team
// fits one.
NormShape norm_shape(int64_t cols, bool f32) {
  const int64_t lane = f32 ? 8 : 16;
  int w = 1;
  while (w < kMaxTeamWarps && w * 32 * lane < cols) w *= 2;
  int c = 1;
  while (c < 8 && static_cast<int64_t>(c) * w * 32 * lane < cols) c *= 2;
  return NormShape{w, w < 8 ? 8 / w : 1, c};
}

template <typename K>
cudaError_t launch_rows(K kernel, const NormParams& a, const NormShape& s, int64_t grid, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute at[1];
  cfg.gridDim = dim3(static_cast<unsigned>(grid * s.cluster));
  cfg.blockDim = dim3(static_cast<unsigned>(s.threads()));
  cfg.stream = stream;
  if (s.cluster > 1) {
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = static_cast<unsigned>(s.cluster);
    at[0].val.clusterDim.y = 1;
    at[0].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
  }
  return cudaLaunchKernelEx(&cfg, kernel, a);
}

template <typename T, bool WIDE>
cudaError_t launch_forward(const NormParams& a, bool layer, const NormShape& s, cudaStream_t stream) {
  const int64_t grid = s.cluster > 1 ? a.rows : ceil_div(a.rows, s.teams);
  if (s.cluster > 1)
    return layer ? launch_rows(norm_forward_kernel<T, WIDE, true, true>, a, s, grid, stream)
                 : launch_rows(norm_forward_kernel<T, WIDE, false, true>, a, s, grid, stream);
  return layer ? launch_rows(norm_forward_kernel<T, WIDE, true, false>, a, s, grid, stream)
               : launch_rows(norm_forward_kernel<T, WIDE, false, false>, a, s, grid, stream);
}

// How the backward pass is cut: warps of a row in a CTA, teams of a CTA, CTAs of a row.
struct GradSplit {
  int warps, teams, cluster;
  int64_t classes, rows_per_block, blocks;
  int threads() const { return warps * teams * 32; }
  int64_t units() const { return blocks * classes; }
};
int64_t row_classes(int64_t cols, int64_t vec) {
  int64_t g = vec;
  while (cols % g != 0) g /= 2;
  return vec / g;
}
GradSplit grad_split(int64_t rows, int64_t cols, bool f32, bool wide, int num_sms) {
  GradSplit s{};
  const int64_t vec = wide ? (f32 ? 4 : 8) : 1;
  s.classes = wide ? row_classes(cols, vec) : 1;
  const int64_t cover = cols + (s.classes > 1 ? vec - 1 : 0);  // a row that starts inside a vector
  s.cluster = static_cast<int>(ceil_div(cover, kGradWarps * 32 * kGradElems));
  s.warps = static_cast<int>(ceil_div(cover, 32 * kGradElems * s.cluster));
  s.teams = s.cluster > 1 ? 1 : kGradWarps / s.warps;
  const int64_t want = std::max<int64_t>(1, num_sms / s.cluster / s.classes);  // one CTA an SM: 128 registers a thread
  const int64_t quantum = s.classes * s.teams;
  s.rows_per_block = ceil_div(ceil_div(rows, want), quantum) * quantum;
  s.blocks = ceil_div(rows, s.rows_per_block);
  return s;
}

template <typename T, int EPT, int READS, bool LAYER, bool BIAS, bool CLUSTER>
cudaError_t launch_backward(const NormGradParams& a, const GradSplit& s, cudaStream_t stream, const DeviceInfo& dev) {
  const auto kernel = norm_backward_kernel<T, EPT, READS, LAYER, BIAS, CLUSTER>;
  constexpr size_t pitch = READS != kSingles ? kRing<T, EPT> * 4 * EPT * sizeof(T) : 0;
  const size_t dynamic = pitch * s.threads() + static_cast<size_t>(s.warps) * 32 * EPT * 8;
  static PerDevice<cudaError_t> ready;
  const cudaError_t e = ready.run(dev.device, [&] {
    cudaError_t r = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         static_cast<int>((pitch + EPT * 8) * kGradWarps * 32));
    if (CLUSTER && r == cudaSuccess) r = cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    return r;
  });
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute at[1];
  cfg.gridDim = dim3(static_cast<unsigned>(s.units() * s.cluster));
  cfg.blockDim = dim3(static_cast<unsigned>(s.threads()));
  cfg.dynamicSmemBytes = dynamic;
  cfg.stream = stream;
  if (CLUSTER) {
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = static_cast<unsigned>(s.cluster);
    at[0].val.clusterDim.y = 1;
    at[0].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
  }
  return cudaLaunchKernelEx(&cfg, kernel, a);
}

template <typename T, int READS, bool LAYER, bool BIAS>
cudaError_t pick_backward(const NormGradParams& a, const GradSplit& s, cudaStream_t stream, const DeviceInfo& dev) {
  return s.cluster > 1 ? launch_backward<T, kGradElems, READS, LAYER, BIAS, true>(a, s, stream, dev)
                       : launch_backward<T, kGradElems, READS, LAYER, BIAS, false>(a, s, stream, dev);
}
// Rows that are no whole vectors take the kernels with all sums.
template <typename T>
cudaError_t pick_backward(const NormGradParams& a, int reads, bool layer, bool bias, const GradSplit& s,
                          cudaStream_t stream, const DeviceInfo& dev) {
  if (reads == kSingles)
    return layer ? pick_backward<T, kSingles, true, true>(a, s, stream, dev)
                 : pick_backward<T, kSingles, false, true>(a, s, stream, dev);
  if (reads == kEdges)
    return layer ? pick_backward<T, kEdges, true, true>(a, s, stream, dev)
                 : pick_backward<T, kEdges, false, true>(a, s, stream, dev);
  if (bias)
    return layer ? pick_backward<T, kVectors, true, true>(a, s, stream, dev)
                 : pick_backward<T, kVectors, false, true>(a, s, stream, dev);
  return layer ? pick_backward<T, kVectors, true, false>(a, s, stream, dev)
               : pick_backward<T, kVectors, false, false>(a, s, stream, dev);
}

}  // namespace

int64_t norm_workspace_floats(int64_t rows, int64_t cols, int64_t groups, bool f32, const DeviceInfo& dev) {
  if (rows <= 0) return 0;
  int64_t most = 0;  // whether the rows can be read by vectors is known at the call alone
  for (const bool wide : {false, true}) {
    const GradSplit s = grad_split(rows, cols, f32, wide, dev.num_sms);
    most = std::max(most, (2 * s.units() + groups * s.classes) * 2 * cols);
  }
  return most;
}

int launch_block_norm(const bsq_block_norm_args& g, cudaStream_t stream, const DeviceInfo&) {
  const bool f32 = (g.flags & BSQ_FLAG_SRC_F32) != 0, layer = g.kind == BSQ_NORM_LAYER;
  const int64_t es = f32 ? 4 : 2;
  const NormShape s = norm_shape(g.cols, f32);
  NormParams a{};
  a.rows = g.rows;
  a.cols = static_cast<int32_t>(g.cols);
  a.group_rows = std::max<int64_t>(1, g.rows / std::max<int64_t>(1, g.gate_groups));
  a.warps = s.warps;
  a.teams = s.teams;
  a.eps = g.eps;
  a.residual_scale = g.residual_scale;
  a.weight_offset = g.weight_offset;
  a.params_f32 = (g.flags & BSQ_FLAG_PARAMS_F32) != 0;
  a.post = (g.flags & BSQ_FLAG_POST_NORM) != 0;
  a.h = g.h, a.x = g.x, a.h_stride = g.h_stride, a.x_stride = g.x_stride;
  a.post_weight = g.post_weight, a.post_bias = g.post_bias, a.gate = g.gate;
  a.pre_weight = g.pre_weight, a.pre_bias = g.pre_bias;
  a.x_out = g.x_out, a.y = g.y, a.stats = reinterpret_cast<float4*>(g.stats);
  const int64_t rb = g.cols * es, pb = g.cols * (a.params_f32 ? 4 : 2);
  const bool wide = rb % 16 == 0 && wide_ok(g.h, g.h_stride * es) && wide_ok(g.x, g.x_stride * es) &&
                    wide_ok(g.x_out, rb) && wide_ok(g.y, rb) && wide_ok(g.post_weight, 0) && wide_ok(g.post_bias, 0) &&
                    wide_ok(g.gate, g.gate_groups > 1 ? pb : 0) && wide_ok(g.pre_weight, 0) && wide_ok(g.pre_bias, 0);
  a.nvec = static_cast<int32_t>(wide ? rb / 16 : g.cols);
  const cudaError_t e = f32 ? (wide ? launch_forward<float, true>(a, layer, s, stream)
                                    : launch_forward<float, false>(a, layer, s, stream))
                            : (wide ? launch_forward<uint16_t, true>(a, layer, s, stream)
                                    : launch_forward<uint16_t, false>(a, layer, s, stream));
  return e == cudaSuccess ? BSQ_OK : BSQ_ERR_LAUNCH;
}

int launch_block_norm_backward(const bsq_block_norm_grad_args& g, cudaStream_t stream, const DeviceInfo& dev) {
  const bool f32 = (g.flags & BSQ_FLAG_SRC_F32) != 0, layer = g.kind == BSQ_NORM_LAYER;
  const int64_t es = f32 ? 4 : 2, vec = 16 / es;
  const int64_t groups = std::max<int64_t>(1, g.gate_groups);
  NormGradParams a{};
  a.rows = g.rows;
  a.cols = static_cast<int32_t>(g.cols);
  a.group_rows = g.rows / groups;
  a.residual_scale = g.residual_scale;
  a.weight_offset = g.weight_offset;
  a.params_f32 = (g.flags & BSQ_FLAG_PARAMS_F32) != 0;
  a.post = (g.flags & BSQ_FLAG_POST_NORM) != 0;
  a.dy = g.dy, a.x_out = g.x_out, a.dx_out = g.dx_out, a.h = g.h;
  a.dy_stride = g.dy_stride, a.x_out_stride = g.x_out_stride, a.dx_out_stride = g.dx_out_stride, a.h_stride = g.h_stride;
  a.stats = reinterpret_cast<const float4*>(g.stats);
  a.post_weight = g.post_weight, a.gate = g.gate, a.pre_weight = g.pre_weight;
  a.dx = g.dx, a.dh = g.dh;
  a.sums1 = g.dpost_weight != nullptr || g.dpost_bias != nullptr || g.dgate != nullptr;
  a.sums2 = g.dpre_weight != nullptr || g.dpre_bias != nullptr;
  // Vectors: every matrix's row r starts at the same offset inside 16 bytes. Parameters are read by
  // vectors too where that offset is 0, so they have to be aligned.
  const struct { const void* p; int64_t stride; } mats[] = {{g.dy, g.dy_stride},         {g.dy ? g.x_out : nullptr, g.x_out_stride},
                                                            {g.dx_out, g.dx_out_stride}, {g.h, g.h_stride},
                                                            {g.dx, g.cols},              {g.dh, g.cols}};
  bool wide = true;
  int64_t shift = -1;
  for (const auto& m : mats) {
    if (m.p == nullptr) continue;
    const int64_t at = static_cast<int64_t>(reinterpret_cast<uintptr_t>(m.p) & 15u) / es;
    if (shift < 0) shift = at;
    wide = wide && at == shift && (m.stride - g.cols) % vec == 0;
  }
  const int64_t pb = g.cols * (a.params_f32 ? 4 : 2);
  wide = wide && (row_classes(g.cols, vec) > 1 || (shift == 0 && wide_ok(g.post_weight, 0) && wide_ok(g.pre_weight, 0) &&
                                                   wide_ok(g.gate, groups > 1 ? pb : 0)));
  GradSplit s = grad_split(g.rows, g.cols, f32, wide, dev.num_sms);
  // vectors are addressed by 32-bit offsets inside a block's rows (and up to three steps of its rows before and behind)
  int64_t widest = g.cols;
  for (const auto& m : mats)
    if (m.p != nullptr) widest = std::max(widest, m.stride);
  if (wide && (s.rows_per_block + 8 * s.classes * s.teams) * widest > INT32_MAX) {
    wide = false;
    s = grad_split(g.rows, g.cols, f32, wide, dev.num_sms);
  }
  a.shift = static_cast<int32_t>(std::max<int64_t>(0, shift));
  a.warps = s.warps;
  a.teams = s.teams;
  a.classes = static_cast<int32_t>(s.classes);
  a.rows_per_block = s.rows_per_block;
  a.ws2 = static_cast<float*>(g.workspace);
  a.ws1 = a.ws2 + s.units() * 2 * g.cols;
  // A0 is the gradient of the post bias, and part of the gate's behind one
  const int reads = !wide ? kSingles : s.classes > 1 ? kEdges : kVectors;
  const bool bias = reads != kVectors || g.dpost_bias != nullptr || g.dpre_bias != nullptr ||
                    (g.dgate != nullptr && a.post && g.post_bias != nullptr);
  cudaError_t e = f32 ? pick_backward<float>(a, reads, layer, bias, s, stream, dev)
                      : pick_backward<uint16_t>(a, reads, layer, bias, s, stream, dev);
  if (e != cudaSuccess) return BSQ_ERR_LAUNCH;
  if (a.sums1 || a.sums2) {
    NormSums n{};
    n.rows = g.rows, n.group_rows = a.group_rows, n.groups = groups;
    n.rows_per_block = s.rows_per_block, n.units = s.units(), n.cols = a.cols, n.classes = a.classes;
    n.weight_offset = g.weight_offset, n.params_f32 = a.params_f32, n.bias = bias;
    n.post_weight = a.post ? g.post_weight : nullptr, n.post_bias = a.post ? g.post_bias : nullptr, n.gate = g.gate;
    n.ws1 = a.ws1, n.ws2 = a.ws2;
    n.dpost_weight = g.dpost_weight, n.dpost_bias = g.dpost_bias, n.dgate = g.dgate;
    n.dpre_weight = g.dpre_weight, n.dpre_bias = g.dpre_bias;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute at[1];
    cfg.gridDim = dim3(static_cast<unsigned>(ceil_div(g.cols, 32)), a.sums1 ? 2 : 1);
    cfg.blockDim = dim3(kSumWarps * 32);
    cfg.stream = stream;
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    e = cudaLaunchKernelEx(&cfg, norm_sums_kernel, n);
  }
  return e == cudaSuccess ? BSQ_OK : BSQ_ERR_LAUNCH;
}

}  // namespace bsq
