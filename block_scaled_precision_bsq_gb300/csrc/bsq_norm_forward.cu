// bsq_norm_forward.cu -- bsq_block_norm (the formulas stand in bsq_norm.cuh).
#include "bsq_norm.cuh"

namespace bsq {
namespace {

// Sum over the 16 lanes of a half, in each of them.
__device__ __forceinline__ float half_warp_sum(float v) {
#pragma unroll
  for (int m = 8; m > 0; m >>= 1) v += __shfl_xor_sync(0xffffffffu, v, m);
  return v;
}

// mean and 1 / sqrt(mean((v - mean)^2) + eps) of a row. The layer norm's second moment is taken
// about each warp's own mean, in a second pass over its registers, and moved to the row's mean when
// the warps join (sum of M2_w + n_w (mean_w - mean)^2): as exact as two passes over the row, with
// one exchange. v is zero outside the row; n_warp counts the warp's columns inside it, full: all.
template <bool LAYER, bool CLUSTER, typename Cols, int P>
__device__ __forceinline__ float2 row_stats(Team<CLUSTER>& team, const Cols& at, const f32x2 (&v)[P], bool full, float n_warp,
                                            float inv_n_warp, float inv_cols, float eps) {
  if constexpr (!LAYER) {
    f32x2 q = both(0.0f);
#pragma unroll
    for (int k = 0; k < P; ++k) q = fma2(v[k], v[k], q);
    const float2 t = team.template sum<false>(sum_halves(q), 0.0f);
    return make_float2(0.0f, rsqrtf(t.x * inv_cols + eps));
  } else {
    f32x2 s = both(0.0f);
#pragma unroll
    for (int k = 0; k < P; ++k) s = add2(s, v[k]);
    const float sw = warp_sum(sum_halves(s));
    const float mw = sw * inv_n_warp;
    f32x2 q = both(0.0f);
    const f32x2 minus = both(-mw);
    if (full) {
#pragma unroll
      for (int k = 0; k < P; ++k) {
        const f32x2 d = add2(v[k], minus);
        q = fma2(d, d, q);
      }
    } else {
#pragma unroll
      for (int i = 0; i < Cols::GROUPS; ++i)
        if (at.live(i)) {
          f32x2 d[P / Cols::GROUPS];
#pragma unroll
          for (int k = 0; k < P / Cols::GROUPS; ++k) d[k] = add2(v[i * (P / Cols::GROUPS) + k], minus);
          at.mask(i, d);
#pragma unroll
          for (int k = 0; k < P / Cols::GROUPS; ++k) q = fma2(d[k], d[k], q);
        }
    }
    __syncwarp();
    const float qw = warp_sum(sum_halves(q));
    if (team.warps == 1) return make_float2(mw, rsqrtf(qw * inv_cols + eps));
    team.exchange(make_float4(sw, qw, n_warp, mw));
    // a lane for each slot of a CTA, twice; slots of no warp hold zeros
    const float4* slot = &team.slots[team.parity][(CLUSTER ? 0 : team.first) + (lane_id() & 15u)];
    const uint32_t ctas = CLUSTER ? team.ranks : 1;
    float total = 0.0f, m2 = 0.0f;
    for (uint32_t k = 0; k < ctas; ++k) total += slot[k * kMaxTeamWarps].x;
    const float mean = half_warp_sum(total) * inv_cols;
    for (uint32_t k = 0; k < ctas; ++k) {
      const float4 p = slot[k * kMaxTeamWarps];
      m2 += p.y + p.z * (p.w - mean) * (p.w - mean);
    }
    m2 = half_warp_sum(m2);
    return make_float2(mean, rsqrtf(m2 * inv_cols + eps));
  }
}

// ---------------------------------------------------------------- forward
// Teams walk the rows; the rows ahead are fetched by cp.async into a ring of shared memory in which
// every thread reads only what it fetched itself, so that no barrier stands between a fetch and its
// use. A thread holds up to 32 elements of a row (16 in fp32): what a row costs whatever its length --
// shuffles, addresses, the exchange between warps -- is about 200 instructions a warp, and with 8
// elements a thread those bound the kernel (51200 x 1024 bf16: 100 us). The parameters lie in shared
// memory in fp32 where they fit beside the ring, a single gate row multiplied into the weights before
// it; else they are read through L1.
//
// Rows whose length is no multiple of 16 bytes begin at different offsets inside a 16-byte vector,
// in a cycle of `classes` rows. A CTA takes the rows of one class alone, so that a thread's vectors
// hold the same columns in every row; the vectors at a row's two ends also hold elements of its
// neighbours, which are masked when read and not written.
struct NormParams {
  int64_t group_rows;  // rows that share a gate row
  uint32_t rows, rows_per_block;
  int32_t cols, warps, teams, classes, stages;
  int32_t shift;  // elements from a 16-byte boundary to the first row
  float eps, residual_scale, weight_offset;
  bool params_f32, post;
  uint32_t staged;  // bit i: parameter array i lies in shared memory
  bool row_gates;  // the gate is read for each row, not multiplied into the weights of a segment
  const void *h, *x;
  int64_t h_stride, x_stride;
  const void *post_weight, *post_bias, *gate, *pre_weight, *pre_bias;
  void *x_out, *y;
  float4* stats;
};

template <typename T, int EPT, int READS, bool LAYER, bool CLUSTER>
__global__ void __launch_bounds__(kMaxTeamWarps * 32, 1) norm_forward_kernel(const NormParams a) {
  using Cols = Columns<T, EPT, READS>;
  constexpr int VEC = Cols::VEC, N = Cols::N, P = EPT / 2, Q = EPT / 4;
  constexpr bool RING = READS != kSingles;
  extern __shared__ uint4 dynamic[];  // weights: [up to 4][Q][threads of the team]; ring
  __shared__ float4 slots[2][Team<CLUSTER>::kSlots];
  Team<CLUSTER> team;
  team.init(slots, a.warps);
  enter_stream();
  const int t = CLUSTER ? 0 : (threadIdx.x >> 5) / a.warps;
  const uint32_t unit = CLUSTER ? blockIdx.x / team.ranks : blockIdx.x;
  const uint32_t cls = unit % a.classes;
  const int lead = READS == kEdges ? static_cast<int>((a.shift + static_cast<int64_t>(cls) * a.cols) % VEC) : 0;
  const float inv_cols = 1.0f / static_cast<float>(a.cols);
  const Cols at{team.thread() * VEC - lead, team.threads() * VEC, a.cols};
  // This team takes rows first, first + step, ... below end. Rows with gates of their own are cut into
  // blocks of consecutive rows that `classes` CTAs share; else all CTAs walk side by side, which DRAM
  // takes better (51200 x 1024: 80 us in blocks, 74 us so).
  const uint32_t strand = unit / a.classes, blocked = a.rows_per_block != 0;
  const uint32_t begin = strand * a.rows_per_block;
  const uint32_t end = blocked ? min(a.rows, begin + a.rows_per_block) : a.rows;
  const uint32_t units = (CLUSTER ? gridDim.x / team.ranks : gridDim.x) / a.classes;
  const uint32_t step = (blocked ? 1 : units) * a.teams * a.classes;
  const uint32_t first = begin + ((blocked ? 0 : strand) * a.teams + t) * a.classes + cls;
  const bool has_h = a.h != nullptr, pre = a.y != nullptr;

  // which parameters there are: post weight (and a single gate), post bias, pre weight, pre bias
  const bool scaled = has_h && ((a.post && a.post_weight != nullptr) || (a.gate != nullptr && !a.row_gates));
  const bool shifted = has_h && a.post && a.post_bias != nullptr;
  const bool scaled2 = pre && a.pre_weight != nullptr, shifted2 = pre && a.pre_bias != nullptr;
  const uint32_t team_threads = a.warps * 32;
  const uint32_t weight_step = team_threads * 16, array_step = Q * weight_step;
  const uint32_t at0 = smem_u32(dynamic) + (threadIdx.x - t * team_threads) * 16;
  const uint32_t at1 = at0 + (a.staged & 1 ? array_step : 0), at2 = at1 + (a.staged & 2 ? array_step : 0);
  const uint32_t at3 = at2 + (a.staged & 4 ? array_step : 0), arrays_end = at3 + (a.staged & 8 ? array_step : 0);
  // elements 4 q .. 4 q + 3 of parameter array 0 to 3, from global memory or as staged
  int64_t gate_at = 0;  // the segment's gate row
  auto global4 = [&](int which, int q, f32x2& lo, f32x2& hi) {
    if (which >= 2) {
      at.params4(which == 2 ? a.pre_weight : a.pre_bias, a.params_f32, 0, which == 2 ? a.weight_offset : 0.0f, 0.0f, q, lo, hi);
      return;
    }
    if (which == 0) at.params4(a.post ? a.post_weight : nullptr, a.params_f32, 0, a.weight_offset, 1.0f, q, lo, hi);
    else at.params4(a.post_bias, a.params_f32, 0, 0.0f, 0.0f, q, lo, hi);
    if (a.gate != nullptr && !a.row_gates) {
      f32x2 g0, g1;
      at.params4(a.gate, a.params_f32, gate_at, 0.0f, 1.0f, q, g0, g1);
      lo = mul2(lo, g0), hi = mul2(hi, g1);
    }
  };
  // f(q, pairs 2 q and 2 q + 1 of the array) for all q
  auto with_params = [&](int which, uint32_t from, auto&& f) {
    f32x2 lo, hi;
    if (a.staged >> which & 1) {
#pragma unroll
      for (int q = 0; q < Q; ++q) {
        load_shared_pairs(from + q * weight_step, lo, hi);
        f(q, lo, hi);
      }
    } else {
#pragma unroll
      for (int q = 0; q < Q; ++q) {
        global4(which, q, lo, hi);
        f(q, lo, hi);
      }
    }
  };

  // ring: [stages][warps][2][N][lanes] vectors; a warp's 16-byte copies land side by side
  const uint32_t stage_bytes = blockDim.x * (2 * N * 16);
  const uint32_t ring0 = arrays_end - at0 + smem_u32(dynamic) + (threadIdx.x >> 5) * (2 * N * 512) + lane_id() * 16;
  const uint32_t ring_end = ring0 + a.stages * stage_bytes;
  const T* src_h = static_cast<const T*>(a.h) + first * a.h_stride + at.first;
  const T* src_x = static_cast<const T*>(a.x) + first * a.x_stride + at.first;
  const int64_t inc_h = static_cast<int64_t>(step) * a.h_stride, inc_x = static_cast<int64_t>(step) * a.x_stride;
  uint32_t ahead = first;
  auto fetch = [&](uint32_t to) {
    if constexpr (RING) {
      if (ahead < end) {
#pragma unroll
        for (int i = 0; i < N; ++i)
          if (at.in(i)) {
            // the last vector of a row stops at the row's end
            const uint32_t bytes = READS == kEdges ? min(16, (a.cols - at.c0(i)) * static_cast<int>(sizeof(T))) : 16;
            if (has_h) cp_async16(to + i * 512, src_h + i * at.step, bytes);
            cp_async16(to + (N + i) * 512, src_x + i * at.step, bytes);
          }
        src_h += inc_h;
        src_x += inc_x;
        ahead += step;
      }
      cp_async_commit();
    }
  };
  auto get = [&](uint32_t from, int m, const void* base, int64_t stride, uint32_t row, f32x2 (&v)[P]) {
    if constexpr (RING) {
#pragma unroll
      for (int i = 0; i < N; ++i) {
        unpack16<T>(load_shared16(from + (m * N + i) * 512), &v[i * VEC / 2]);
        at.mask(i, &v[i * VEC / 2]);
      }
    } else {
      const T* p = static_cast<const T*>(base) + row * stride;
#pragma unroll
      for (int e = 0; e < P; ++e) {
        Vec<T, false> r, q;
        r.clear(), q.clear();
        if (at.in(2 * e)) r.load(p + at.c0(2 * e));
        if (at.in(2 * e + 1)) q.load(p + at.c0(2 * e + 1));
        r.get(&v[e].x), q.get(&v[e].y);
      }
    }
  };
  if constexpr (RING) {  // lanes past the row's end read zeros
    for (int s = 0; s < a.stages; ++s)
#pragma unroll
      for (int i = 0; i < 2 * N; ++i)
        if (!at.in(i % N)) store_shared16(ring0 + s * stage_bytes + i * 512, make_uint4(0, 0, 0, 0));
  }
  for (int k = 0; k < a.stages - 1; ++k) fetch(ring0 + k * stage_bytes);
  // the teams share the arrays, and the writing of them
  auto put = [&](int which, uint32_t to) {
    for (int q = t; q < Q; q += a.teams) {
      f32x2 lo, hi;
      global4(which, q, lo, hi);
      store_shared16(to + q * weight_step, make_uint4(__float_as_uint(lo.x), __float_as_uint(lo.y),
                                                      __float_as_uint(hi.x), __float_as_uint(hi.y)));
    }
  };
  if (a.staged & 4) put(2, at2);
  if (a.staged & 8) put(3, at3);
  float n_warp = 0.0f;  // the columns of this warp
#pragma unroll
  for (int k = 0; k < EPT; ++k) n_warp += at.has(k) ? 1.0f : 0.0f;
  const bool full = __all_sync(0xffffffffu, n_warp == static_cast<float>(EPT)) != 0;
  if constexpr (LAYER) n_warp = warp_sum(n_warp);
  const float inv_n_warp = n_warp > 0.0f ? 1.0f / n_warp : 0.0f;

  T* x_out = static_cast<T*>(a.x_out) + static_cast<int64_t>(first) * a.cols + at.first;
  T* y = static_cast<T*>(a.y) + static_cast<int64_t>(first) * a.cols + at.first;
  const int64_t out_step = static_cast<int64_t>(step) * a.cols;
  uint32_t s = ring0, to = ring0 + (a.stages - 1) * stage_bytes;  // stage to read, stage to fill
  uint32_t row = first;
  for (uint32_t seg = begin; seg < end;) {  // the rows that share a gate row; all where it is read for each row
    uint32_t seg_end = end;
    if (blocked) {
      const int64_t group = seg / a.group_rows;
      gate_at = group * a.cols;
      seg_end = static_cast<uint32_t>(min(static_cast<int64_t>(end), (group + 1) * a.group_rows));
    }
    if (a.staged) {
      if (seg != begin) __syncthreads();  // the last segment's weights are read no more
      if (a.staged & 1) put(0, at0);
      if (a.staged & 2) put(1, at1);
      __syncthreads();
    }
    seg = seg_end;
    for (; row < seg_end; row += step) {
      fetch(to);
      if constexpr (RING) {
        if (a.stages == 2) cp_async_wait<1>();
        else cp_async_wait<2>();
      }
      float4 st = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
      f32x2 v[P];
      if (has_h) {
        f32x2 n[P];
        get(s, 0, a.h, a.h_stride, row, n);
        if (a.post) {
          const float2 m = row_stats<LAYER>(team, at, n, full, n_warp, inv_n_warp, inv_cols, a.eps);
          st.x = m.x;
          st.y = m.y;
          const f32x2 minus = both(-m.x), rstd = both(m.y);
#pragma unroll
          for (int k = 0; k < P; ++k) {
            if (LAYER) n[k] = add2(n[k], minus);
            n[k] = mul2(n[k], rstd);
          }
        }
        if (scaled)
          with_params(0, at0, [&](int q, f32x2 lo, f32x2 hi) {
            n[2 * q] = mul2(n[2 * q], lo), n[2 * q + 1] = mul2(n[2 * q + 1], hi);
          });
        if (shifted)
          with_params(1, at1, [&](int q, f32x2 lo, f32x2 hi) {
            n[2 * q] = add2(n[2 * q], lo), n[2 * q + 1] = add2(n[2 * q + 1], hi);
          });
        if (a.row_gates) {
          const int64_t gate_row = row / a.group_rows * a.cols;
#pragma unroll
          for (int q = 0; q < Q; ++q) {
            f32x2 lo, hi;
            at.params4(a.gate, a.params_f32, gate_row, 0.0f, 1.0f, q, lo, hi);
            n[2 * q] = mul2(n[2 * q], lo), n[2 * q + 1] = mul2(n[2 * q + 1], hi);
          }
        }
        get(s, 1, a.x, a.x_stride, row, v);
        const f32x2 scale = both(a.residual_scale);
#pragma unroll
        for (int k = 0; k < P; ++k) v[k] = fma2(v[k], scale, n[k]);
        // a mean stands in columns outside the row: those count as zeros below
        if (LAYER && a.post && !full) {
#pragma unroll
          for (int i = 0; i < Cols::GROUPS; ++i) {
            if (!at.live(i)) {
#pragma unroll
              for (int k = 0; k < P / Cols::GROUPS; ++k) v[i * (P / Cols::GROUPS) + k] = both(0.0f);
            } else {
              at.mask(i, &v[i * (P / Cols::GROUPS)]);
            }
          }
        }
      } else {
        get(s, 1, a.x, a.x_stride, row, v);
        const f32x2 scale = both(a.residual_scale);
#pragma unroll
        for (int k = 0; k < P; ++k) v[k] = mul2(v[k], scale);
      }
      if (a.x_out != nullptr) at.store(x_out, v);
      if (pre) {
        const float2 m = row_stats<LAYER>(team, at, v, full, n_warp, inv_n_warp, inv_cols, a.eps);
        st.z = m.x;
        st.w = m.y;
        const f32x2 minus = both(-m.x), rstd = both(m.y);
#pragma unroll
        for (int k = 0; k < P; ++k) {
          if (LAYER) v[k] = add2(v[k], minus);
          v[k] = mul2(v[k], rstd);
        }
        if (scaled2)
          with_params(2, at2, [&](int q, f32x2 lo, f32x2 hi) {
            v[2 * q] = mul2(v[2 * q], lo), v[2 * q + 1] = mul2(v[2 * q + 1], hi);
          });
        if (shifted2)
          with_params(3, at3, [&](int q, f32x2 lo, f32x2 hi) {
            v[2 * q] = add2(v[2 * q], lo), v[2 * q + 1] = add2(v[2 * q + 1], hi);
          });
        at.store(y, v);
      }
      if (a.stats != nullptr && team.thread() == 0) a.stats[row] = st;
      x_out += out_step;
      y += out_step;
      to = s;  // read for the last time above
      s += stage_bytes;
      if (s == ring_end) s = ring0;
    }
  }
  if constexpr (RING) cp_async_wait<0>();
  if constexpr (CLUSTER) cluster_barrier();  // no CTA leaves while another may still write its slots
}

// ---------------------------------------------------------------- launches
constexpr size_t kMostDynamic = 216 * 1024;  // of 227 KB, beside the slots

template <typename T, int EPT, int READS, bool LAYER, bool CLUSTER>
cudaError_t launch_forward(NormParams a, const RowCut& c, cudaStream_t stream, const DeviceInfo& dev) {
  const auto kernel = norm_forward_kernel<T, EPT, READS, LAYER, CLUSTER>;
  static PerDevice<cudaError_t> ready;
  const cudaError_t e = ready.run(dev.device, [&] { return allow(reinterpret_cast<const void*>(kernel), kMostDynamic, CLUSTER); });
  if (e != cudaSuccess) return e;
  // A segment's gate is worth a staging of the weights where its rows keep the teams busy a few times over.
  a.row_gates = a.gate != nullptr && a.group_rows < a.rows && a.group_rows < 8 * c.teams * c.classes;
  const bool present[4] = {a.h != nullptr && ((a.post && a.post_weight != nullptr) || (a.gate != nullptr && !a.row_gates)),
                           a.h != nullptr && a.post && a.post_bias != nullptr, a.y != nullptr && a.pre_weight != nullptr,
                           a.y != nullptr && a.pre_bias != nullptr};
  const size_t stage = READS != kSingles ? static_cast<size_t>(2) * EPT * sizeof(T) * c.threads() : 0;
  const size_t array = static_cast<size_t>(4) * EPT * c.warps * 32;
  size_t weights = 0;
  for (int i = 0; i < 4; ++i)
    if (present[i] && 2 * stage + weights + array <= kMostDynamic) {
      a.staged |= 1u << i;
      weights += array;
    }
  a.stages = 3 * stage + weights <= kMostDynamic ? 3 : 2;
  const int64_t most = std::max<int64_t>(1, dev.num_sms / c.cluster / c.classes);  // one CTA an SM: 128 registers a thread
  int64_t ctas = std::min(most, ceil_div(ceil_div(a.rows, c.classes), c.teams));
  if (a.gate != nullptr && a.group_rows < a.rows && !a.row_gates) {
    const int64_t per = ceil_div(ceil_div(a.rows, most), c.classes) * c.classes;
    a.rows_per_block = static_cast<uint32_t>(per);
    ctas = ceil_div(a.rows, per);
  }
  return launch_cut(kernel, a, ctas * c.classes, c, a.stages * stage + weights, stream);
}
template <typename T, int READS, bool LAYER>
cudaError_t pick_forward(const NormParams& a, const RowCut& c, cudaStream_t stream, const DeviceInfo& dev) {
  if (c.ept == 8) return launch_forward<T, 8, READS, LAYER, false>(a, c, stream, dev);
  if constexpr (sizeof(T) == 2) {
    if (c.ept == 16) return launch_forward<T, 16, READS, LAYER, false>(a, c, stream, dev);
    return c.cluster > 1 ? launch_forward<T, 32, READS, LAYER, true>(a, c, stream, dev)
                         : launch_forward<T, 32, READS, LAYER, false>(a, c, stream, dev);
  } else {
    return c.cluster > 1 ? launch_forward<T, 16, READS, LAYER, true>(a, c, stream, dev)
                         : launch_forward<T, 16, READS, LAYER, false>(a, c, stream, dev);
  }
}
template <typename T>
cudaError_t pick_forward(const NormParams& a, bool layer, const RowCut& c, cudaStream_t stream, const DeviceInfo& dev) {
  if (c.reads == kVectors)
    return layer ? pick_forward<T, kVectors, true>(a, c, stream, dev) : pick_forward<T, kVectors, false>(a, c, stream, dev);
  if (c.reads == kEdges)
    return layer ? pick_forward<T, kEdges, true>(a, c, stream, dev) : pick_forward<T, kEdges, false>(a, c, stream, dev);
  return layer ? pick_forward<T, kSingles, true>(a, c, stream, dev) : pick_forward<T, kSingles, false>(a, c, stream, dev);
}

}  // namespace

int launch_block_norm(const bsq_block_norm_args& g, cudaStream_t stream, const DeviceInfo& dev) {
  const bool f32 = (g.flags & BSQ_FLAG_SRC_F32) != 0, layer = g.kind == BSQ_NORM_LAYER;
  const int64_t es = f32 ? 4 : 2;
  NormParams a{};
  a.rows = static_cast<uint32_t>(g.rows);
  a.cols = static_cast<int32_t>(g.cols);
  a.group_rows = g.rows / g.gate_groups;
  a.eps = g.eps;
  a.residual_scale = g.residual_scale;
  a.weight_offset = g.weight_offset;
  a.params_f32 = (g.flags & BSQ_FLAG_PARAMS_F32) != 0;
  a.post = (g.flags & BSQ_FLAG_POST_NORM) != 0;
  a.h = g.h, a.x = g.x, a.h_stride = g.h_stride, a.x_stride = g.x_stride;
  a.post_weight = g.post_weight, a.post_bias = g.post_bias, a.gate = g.gate;
  a.pre_weight = g.pre_weight, a.pre_bias = g.pre_bias;
  a.x_out = g.x_out, a.y = g.y, a.stats = reinterpret_cast<float4*>(g.stats);
  int64_t shift;
  bool wide = same_offsets({{g.h, g.h_stride}, {g.x, g.x_stride}, {g.x_out, g.cols}, {g.y, g.cols}}, g.cols, es, &shift);
  // Rows of whole vectors read their parameters by vectors too. One that is not aligned turns the call to single
  // elements, without a ring (51200 x 1024 bf16 from cold caches: 146 us, 81 us by vectors).
  const int64_t pb = g.cols * (a.params_f32 ? 4 : 2);
  wide = wide && (row_classes(g.cols, 16 / es) > 1 ||
                  (shift == 0 && wide_ok(g.post_weight, 0) && wide_ok(g.post_bias, 0) &&
                   wide_ok(g.gate, g.gate_groups > 1 ? pb : 0) && wide_ok(g.pre_weight, 0) && wide_ok(g.pre_bias, 0)));
  RowCut c = row_cut(g.cols, f32, wide, shift, true);
  if (c.cluster == 1) {
    // Few rows for an SM: as many warps for each as there is room for (one row of 4096 bf16 takes 6.0 us with
    // 4 warps, 4.2 us with 16), and no more teams in a CTA than leave every SM some.
    const int64_t for_sm = ceil_div(g.rows, dev.num_sms);
    while (c.ept > 8 && c.warps * 2 * for_sm <= kMaxTeamWarps) c.ept /= 2, c.warps *= 2;
    c.teams = static_cast<int>(std::min<int64_t>(kMaxTeamWarps / c.warps, for_sm));
  }
  a.warps = c.warps, a.teams = c.teams, a.classes = static_cast<int32_t>(c.classes), a.shift = c.shift;
  const cudaError_t e = f32 ? pick_forward<float>(a, layer, c, stream, dev) : pick_forward<uint16_t>(a, layer, c, stream, dev);
  return e == cudaSuccess ? BSQ_OK : BSQ_ERR_LAUNCH;
}

}  // namespace bsq
