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
constexpr int kMaxCluster = 8;

struct NormParams {
  int64_t rows, group_rows;  // group_rows: rows that share a gate row
  int32_t cols, nvec;        // nvec: vectors (or scalars) in a row
  int32_t warps, teams;      // warps of a team in one CTA; teams of a CTA
  float eps, residual_scale, weight_offset;
  bool params_f32, post, has_x_out;
  const void *h, *x;
  int64_t h_stride, x_stride;
  const void *post_weight, *post_bias, *gate, *pre_weight, *pre_bias;
  void *x_out, *y;
  float4* stats;
  // backward
  const void *dx_out, *dy;
  int64_t dx_out_stride, dy_stride;
  void *dx, *dh;
  int64_t rows_per_cta;
  bool sums1, sums2;  // whether A0 / A1 and dpre sums are wanted
  float *ws1, *ws2;   // partial sums: [slots][2][cols] each
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
// go to a slot of shared memory (of every CTA of the cluster), and one barrier later every thread
// adds the slots in the same order. Two sets of slots in turn make one barrier per sum enough: a
// set is written again only behind the next sum's barrier, which every reader reaches after its
// reads.
template <bool CLUSTER>
struct Team {
  float4 (*slots)[kMaxTeamWarps * kMaxCluster];  // [2][...]
  int warps, warp, first, bar;                   // warps of the team (all CTAs), own index, first slot
  int parity = 0;
  uint32_t ranks = 1, rank = 0;

  __device__ __forceinline__ void init(float4 (*s)[kMaxTeamWarps * kMaxCluster], const NormParams& a) {
    slots = s;
    const int w = threadIdx.x >> 5;
    if constexpr (CLUSTER) {
      ranks = cluster_size();
      rank = cluster_rank();
      warps = a.warps * static_cast<int>(ranks);
      warp = static_cast<int>(rank) * a.warps + w;
      first = 0;
      bar = 0;
    } else {
      warps = a.warps;
      warp = w % a.warps;
      first = w - warp;
      bar = 1 + w / a.warps;
    }
  }
  // index of this thread among the threads of the row, and their number
  __device__ __forceinline__ int thread() const { return warp * 32 + static_cast<int>(lane_id()); }
  __device__ __forceinline__ int threads() const { return warps * 32; }

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
  // Sum of two values over the row (of one where `two` is false).
  __device__ __forceinline__ float2 sum(float a, float b, bool two) {
    a = warp_sum(a);
    if (two) b = warp_sum(b);
    if (warps == 1) return make_float2(a, b);
    exchange(make_float4(a, b, 0.0f, 0.0f));
    float2 t = make_float2(0.0f, 0.0f);
    for (int i = 0; i < warps; ++i) {
      const float4 p = slots[parity][first + i];
      t.x += p.x;
      t.y += p.y;
    }
    return t;
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
    const float2 t = team.sum(q, 0.0f, false);
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
    for (int i = 0; i < team.warps; ++i) mean += team.slots[team.parity][team.first + i].x;
    mean *= inv_cols;
    for (int i = 0; i < team.warps; ++i) {
      const float4 p = team.slots[team.parity][team.first + i];
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
  __shared__ float4 slots[2][kMaxTeamWarps * kMaxCluster];
  Team<CLUSTER> team;
  team.init(slots, a);
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
// A CTA takes rows_per_cta consecutive rows and walks them by the segments that share a gate row;
// its teams take a segment's rows in turn and keep the column sums in registers. A segment's A0, A1
// go to slot (CTA + gate row) of ws1 -- consecutive segments differ in one or the other, so no two
// share a slot -- and the pre-norm's sums to slot CTA of ws2.
template <int VEC, int N, bool CLUSTER>
__device__ __forceinline__ void flush_sums(const NormParams& a, const Team<CLUSTER>& team, float (&acc)[N][VEC],
                                           const int (&col)[N], const bool (&in)[N], float* out, float* stage) {
  if (a.teams > 1) {  // teams join in order through shared memory ([teams][cols], cols <= 4096 / teams)
    const int t = (threadIdx.x >> 5) / a.warps;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < N; ++i)
#pragma unroll
      for (int e = 0; e < VEC; ++e)
        if (in[i]) stage[t * a.cols + col[i] + e] = acc[i][e];
    __syncthreads();
    for (int c = threadIdx.x; c < a.cols; c += blockDim.x) {
      float s = 0.0f;
      for (int k = 0; k < a.teams; ++k) s += stage[k * a.cols + c];
      out[c] = s;
    }
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i)
#pragma unroll
      for (int e = 0; e < VEC; ++e)
        if (in[i]) out[col[i] + e] = acc[i][e];
  }
#pragma unroll
  for (int i = 0; i < N; ++i)
#pragma unroll
    for (int e = 0; e < VEC; ++e) acc[i][e] = 0.0f;
}

template <typename T, bool WIDE, bool LAYER, bool CLUSTER>
__global__ void __launch_bounds__(kMaxTeamWarps * 32) norm_backward_kernel(const NormParams a) {
  constexpr int VEC = Access<T, WIDE>::kVec, N = Access<T, WIDE>::kNum;
  __shared__ float4 slots[2][kMaxTeamWarps * kMaxCluster];
  __shared__ float stage[4096];
  Team<CLUSTER> team;
  team.init(slots, a);
  const int t = CLUSTER ? 0 : (threadIdx.x >> 5) / a.warps;
  const int64_t cta = CLUSTER ? blockIdx.x / team.ranks : blockIdx.x;
  const float inv_cols = 1.0f / static_cast<float>(a.cols);
  int col[N];
  bool in[N];
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const int v = i * team.threads() + team.thread();
    col[i] = v * VEC;
    in[i] = v < a.nvec;
  }
  float a0[N][VEC] = {}, a1[N][VEC] = {}, p0[N][VEC] = {}, p1[N][VEC] = {};
  const int64_t begin = cta * a.rows_per_cta, end = min(a.rows, begin + a.rows_per_cta);
  for (int64_t seg = begin; seg < end;) {
    const int64_t group = seg / a.group_rows;
    const int64_t seg_end = min(end, (group + 1) * a.group_rows);
    for (int64_t row = seg + t; row < seg_end; row += a.teams) {
      const float4 st = a.stats[row];
      Vec<T, WIDE> dyr[N], xr[N], dr[N], hr[N];
      const T* dy = static_cast<const T*>(a.dy) + row * a.dy_stride;
      const T* x = static_cast<const T*>(a.x) + row * a.x_stride;
      const T* dxo = static_cast<const T*>(a.dx_out) + row * a.dx_out_stride;
      const T* h = static_cast<const T*>(a.h) + row * a.h_stride;
#pragma unroll
      for (int i = 0; i < N; ++i) {
        dyr[i].clear(), xr[i].clear(), dr[i].clear(), hr[i].clear();
        if (in[i]) {
          if (a.dy != nullptr) dyr[i].load(dy + col[i]), xr[i].load(x + col[i]);
          if (a.dx_out != nullptr) dr[i].load(dxo + col[i]);
          if (a.h != nullptr) hr[i].load(h + col[i]);
        }
      }
      float d[N][VEC];
#pragma unroll
      for (int i = 0; i < N; ++i) dr[i].get(d[i]);
      if (a.dy != nullptr) {
        float g[N][VEC], z[N][VEC];
        float s0 = 0.0f, s1 = 0.0f;
#pragma unroll
        for (int i = 0; i < N; ++i) {
          dyr[i].get(g[i]);
          xr[i].get(z[i]);
          if (in[i]) {
            float w[VEC];
            load_weight<VEC>(a.pre_weight, a.params_f32, a.weight_offset, col[i], w);
#pragma unroll
            for (int e = 0; e < VEC; ++e) {
              z[i][e] = (z[i][e] - st.z) * st.w;
              p0[i][e] += g[i][e];
              p1[i][e] += g[i][e] * z[i][e];
              g[i][e] *= w[e];
              s0 += g[i][e];
              s1 += g[i][e] * z[i][e];
            }
          }
        }
        const float2 s = team.sum(s1, s0, LAYER);
        const float m1 = s.x * inv_cols, m0 = LAYER ? s.y * inv_cols : 0.0f;
#pragma unroll
        for (int i = 0; i < N; ++i)
#pragma unroll
          for (int e = 0; e < VEC; ++e) d[i][e] += st.w * (g[i][e] - m0 - z[i][e] * m1);
      }
      if (a.dx != nullptr) {
        T* o = static_cast<T*>(a.dx) + row * a.cols;
#pragma unroll
        for (int i = 0; i < N; ++i)
          if (in[i]) {
            float f[VEC];
#pragma unroll
            for (int e = 0; e < VEC; ++e) f[e] = a.residual_scale * d[i][e];
            Vec<T, WIDE>::store(o + col[i], f);
          }
      }
      if (a.dh != nullptr || a.sums1) {
        float z[N][VEC];
        float s0 = 0.0f, s1 = 0.0f;
#pragma unroll
        for (int i = 0; i < N; ++i) {
          hr[i].get(z[i]);
          if (in[i]) {
#pragma unroll
            for (int e = 0; e < VEC; ++e) {
              if (a.post) z[i][e] = (z[i][e] - st.x) * st.y;
              a0[i][e] += d[i][e];
              a1[i][e] += d[i][e] * z[i][e];
            }
            if (a.gate != nullptr) {
              float g[VEC];
              load_param<VEC>(a.gate, a.params_f32, group * a.cols + col[i], g);
#pragma unroll
              for (int e = 0; e < VEC; ++e) d[i][e] *= g[e];
            }
            if (a.post) {
              float w[VEC];
              load_weight<VEC>(a.post_weight, a.params_f32, a.weight_offset, col[i], w);
#pragma unroll
              for (int e = 0; e < VEC; ++e) {
                d[i][e] *= w[e];
                s0 += d[i][e];
                s1 += d[i][e] * z[i][e];
              }
            }
          }
        }
        if (a.post) {
          const float2 s = team.sum(s1, s0, LAYER);
          const float m1 = s.x * inv_cols, m0 = LAYER ? s.y * inv_cols : 0.0f;
#pragma unroll
          for (int i = 0; i < N; ++i)
#pragma unroll
            for (int e = 0; e < VEC; ++e) d[i][e] = st.y * (d[i][e] - m0 - z[i][e] * m1);
        }
        if (a.dh != nullptr) {
          T* o = static_cast<T*>(a.dh) + row * a.cols;
#pragma unroll
          for (int i = 0; i < N; ++i)
            if (in[i]) Vec<T, WIDE>::store(o + col[i], d[i]);
        }
      }
    }
    if (a.sums1) {
      float* out = a.ws1 + (cta + group) * 2 * a.cols;
      flush_sums<VEC>(a, team, a1, col, in, out, stage);
      flush_sums<VEC>(a, team, a0, col, in, out + a.cols, stage);
    }
    seg = seg_end;
  }
  if (a.sums2) {
    float* out = a.ws2 + cta * 2 * a.cols;
    flush_sums<VEC>(a, team, p1, col, in, out, stage);
    flush_sums<VEC>(a, team, p0, col, in, out + a.cols, stage);
  }
  if constexpr (CLUSTER) cluster_barrier();
}

// ---------------------------------------------------------------- parameter gradients
struct NormSums {
  int64_t rows, group_rows, groups, rows_per_cta, ctas;
  int32_t cols;
  float weight_offset;
  bool params_f32;
  const void *post_weight, *post_bias, *gate;
  const float *ws1, *ws2;
  float *dpost_weight, *dpost_bias, *dgate, *dpre_weight, *dpre_bias;
};
constexpr int kSumWarps = 16;

// 32 columns a CTA (one a lane); its warps share the slots of a sum, in a fixed order.
__global__ void __launch_bounds__(kSumWarps * 32) norm_sums_kernel(const NormSums a) {
  __shared__ float2 part[kSumWarps][32];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int c = blockIdx.x * 32 + lane;
  const bool in = c < a.cols;
  // all warps: the sum of `n` slots from `base`, returned to warp 0
  auto joined = [&](const float* base, int64_t n) {
    float2 s = make_float2(0.0f, 0.0f);
    if (in) {
#pragma unroll 4
      for (int64_t i = warp; i < n; i += kSumWarps) {
        const float* p = base + i * 2 * a.cols + c;
        s.x += p[0];
        s.y += p[a.cols];
      }
    }
    __syncthreads();
    part[warp][lane] = s;
    __syncthreads();
    if (warp == 0)
      for (int w = 1; w < kSumWarps; ++w) s.x += part[w][lane].x, s.y += part[w][lane].y;
    return s;
  };
  if (a.dpre_weight != nullptr || a.dpre_bias != nullptr) {
    const float2 s = joined(a.ws2, a.ctas);
    if (warp == 0 && in) {
      if (a.dpre_weight != nullptr) a.dpre_weight[c] = s.x;
      if (a.dpre_bias != nullptr) a.dpre_bias[c] = s.y;
    }
  }
  if (a.dpost_weight == nullptr && a.dpost_bias == nullptr && a.dgate == nullptr) return;
  float w = 1.0f, b = 0.0f;
  if (in) {
    load_weight<1>(a.post_weight, a.params_f32, a.weight_offset, c, &w);
    if (a.post_bias != nullptr) load_param<1>(a.post_bias, a.params_f32, c, &b);
  }
  float2 total = make_float2(0.0f, 0.0f);  // of gate * (A1, A0)
  auto add_group = [&](int64_t g, float2 s) {
    float gate = 1.0f;
    if (a.gate != nullptr) load_param<1>(a.gate, a.params_f32, g * a.cols + c, &gate);
    if (a.dgate != nullptr) a.dgate[g * a.cols + c] = w * s.x + b * s.y;
    total.x += gate * s.x;
    total.y += gate * s.y;
  };
  // the CTAs whose rows meet gate row g, and their first slot
  auto first_cta = [&](int64_t g) { return g * a.group_rows / a.rows_per_cta; };
  auto num_ctas = [&](int64_t g) { return (g + 1) * a.group_rows - 1 < a.rows
                                              ? ((g + 1) * a.group_rows - 1) / a.rows_per_cta - first_cta(g) + 1
                                              : (a.rows - 1) / a.rows_per_cta - first_cta(g) + 1; };
  if (a.groups < kSumWarps) {
    for (int64_t g = 0; g < a.groups; ++g) {
      const float2 s = joined(a.ws1 + (first_cta(g) + g) * 2 * a.cols, num_ctas(g));
      if (warp == 0 && in) add_group(g, s);
    }
  } else {  // a warp for each gate row
    if (in)
      for (int64_t g = warp; g < a.groups; g += kSumWarps) {
        float2 s = make_float2(0.0f, 0.0f);
        const int64_t n = num_ctas(g);
        const float* base = a.ws1 + (first_cta(g) + g) * 2 * a.cols + c;
        for (int64_t i = 0; i < n; ++i) s.x += base[i * 2 * a.cols], s.y += base[i * 2 * a.cols + a.cols];
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
  while (c < kMaxCluster && static_cast<int64_t>(c) * w * 32 * lane < cols) c *= 2;
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

template <typename T, bool WIDE>
cudaError_t launch_backward(const NormParams& a, bool layer, const NormShape& s, int64_t ctas, cudaStream_t stream) {
  if (s.cluster > 1)
    return layer ? launch_rows(norm_backward_kernel<T, WIDE, true, true>, a, s, ctas, stream)
                 : launch_rows(norm_backward_kernel<T, WIDE, false, true>, a, s, ctas, stream);
  return layer ? launch_rows(norm_backward_kernel<T, WIDE, true, false>, a, s, ctas, stream)
               : launch_rows(norm_backward_kernel<T, WIDE, false, false>, a, s, ctas, stream);
}

// Rows that one CTA (or cluster) of the backward pass takes, and the number of those.
struct NormSplit {
  int64_t rows_per_cta, ctas;
};
NormSplit norm_split(int64_t rows, const NormShape& s, int num_sms) {
  const int64_t want = std::max<int64_t>(1, (s.threads() > 256 ? 1 : 2) * static_cast<int64_t>(num_sms) / s.cluster);
  const int64_t per = ceil_div(ceil_div(rows, want), s.teams) * s.teams;
  return NormSplit{per, ceil_div(rows, per)};
}

}  // namespace

int64_t norm_workspace_floats(int64_t rows, int64_t cols, int64_t groups, bool f32, const DeviceInfo& dev) {
  if (rows <= 0) return 0;
  const NormSplit p = norm_split(rows, norm_shape(cols, f32), dev.num_sms);
  return (2 * p.ctas + groups) * 2 * cols;
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
  const int64_t es = f32 ? 4 : 2;
  const NormShape s = norm_shape(g.cols, f32);
  const NormSplit p = norm_split(g.rows, s, dev.num_sms);
  const int64_t groups = std::max<int64_t>(1, g.gate_groups);
  NormParams a{};
  a.rows = g.rows;
  a.cols = static_cast<int32_t>(g.cols);
  a.group_rows = g.rows / groups;
  a.warps = s.warps;
  a.teams = s.teams;
  a.residual_scale = g.residual_scale;
  a.weight_offset = g.weight_offset;
  a.params_f32 = (g.flags & BSQ_FLAG_PARAMS_F32) != 0;
  a.post = (g.flags & BSQ_FLAG_POST_NORM) != 0;
  a.h = g.h, a.x = g.x_out, a.h_stride = g.h_stride, a.x_stride = g.x_out_stride;
  a.dx_out = g.dx_out, a.dy = g.dy, a.dx_out_stride = g.dx_out_stride, a.dy_stride = g.dy_stride;
  a.post_weight = g.post_weight, a.post_bias = g.post_bias, a.gate = g.gate;
  a.pre_weight = g.pre_weight, a.pre_bias = g.pre_bias;
  a.stats = reinterpret_cast<float4*>(const_cast<float*>(g.stats));
  a.dx = g.dx, a.dh = g.dh;
  a.rows_per_cta = p.rows_per_cta;
  a.sums1 = g.dpost_weight != nullptr || g.dpost_bias != nullptr || g.dgate != nullptr;
  a.sums2 = g.dpre_weight != nullptr || g.dpre_bias != nullptr;
  a.ws2 = static_cast<float*>(g.workspace);
  a.ws1 = a.ws2 + p.ctas * 2 * g.cols;
  const int64_t rb = g.cols * es, pb = g.cols * (a.params_f32 ? 4 : 2);
  const bool wide = rb % 16 == 0 && wide_ok(g.h, g.h_stride * es) && wide_ok(g.x_out, g.x_out_stride * es) &&
                    wide_ok(g.dx_out, g.dx_out_stride * es) && wide_ok(g.dy, g.dy_stride * es) && wide_ok(g.dx, rb) &&
                    wide_ok(g.dh, rb) && wide_ok(g.post_weight, 0) && wide_ok(g.gate, groups > 1 ? pb : 0) &&
                    wide_ok(g.pre_weight, 0);
  a.nvec = static_cast<int32_t>(wide ? rb / 16 : g.cols);
  cudaError_t e = f32 ? (wide ? launch_backward<float, true>(a, layer, s, p.ctas, stream)
                              : launch_backward<float, false>(a, layer, s, p.ctas, stream))
                      : (wide ? launch_backward<uint16_t, true>(a, layer, s, p.ctas, stream)
                              : launch_backward<uint16_t, false>(a, layer, s, p.ctas, stream));
  if (e != cudaSuccess) return BSQ_ERR_LAUNCH;
  if (a.sums1 || a.sums2) {
    NormSums n{};
    n.rows = g.rows, n.group_rows = a.group_rows, n.groups = groups;
    n.rows_per_cta = p.rows_per_cta, n.ctas = p.ctas, n.cols = a.cols;
    n.weight_offset = g.weight_offset, n.params_f32 = a.params_f32;
    n.post_weight = a.post ? g.post_weight : nullptr, n.post_bias = a.post ? g.post_bias : nullptr, n.gate = g.gate;
    n.ws1 = a.ws1, n.ws2 = a.ws2;
    n.dpost_weight = g.dpost_weight, n.dpost_bias = g.dpost_bias, n.dgate = g.dgate;
    n.dpre_weight = g.dpre_weight, n.dpre_bias = g.dpre_bias;
    norm_sums_kernel<<<static_cast<unsigned>(ceil_div(g.cols, 32)), kSumWarps * 32, 0, stream>>>(n);
    e = cudaGetLastError();
  }
  return e == cudaSuccess ? BSQ_OK : BSQ_ERR_LAUNCH;
}

}  // namespace bsq
