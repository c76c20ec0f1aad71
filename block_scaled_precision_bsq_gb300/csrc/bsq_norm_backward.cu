// bsq_norm_backward.cu -- bsq_block_norm_backward (the formulas stand in bsq_norm.cuh).
#include "bsq_norm.cuh"

namespace bsq {
namespace {

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
template <typename T>
constexpr int kBackwardRing = sizeof(T) == 4 ? 2 : 3;
constexpr int kStageFloats = 4096;  // teams * cols of a CTA with several teams: 16 warps of 8 elements a lane

// What the column sums become, and where they lie.
struct NormSums {
  int64_t rows, group_rows, groups, rows_per_block, units;  // units: slots of ws2
  int32_t cols, classes;
  float weight_offset;
  bool params_f32, bias;  // bias: whether A0 and dpre_bias were summed
  const void *post_weight, *post_bias, *gate;
  const float *ws1, *ws2;
  float *dpost_weight, *dpost_bias, *dgate, *dpre_weight, *dpre_bias;
};

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
  int* status;
  // injected stall: the last CTA of a cluster falls silent after so many rows (-1: never); the waits' limit
  int32_t stall_after;
  uint64_t wait_ns;
  bool join;  // the CTAs form one cluster and join their sums themselves
  NormSums sums;
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

constexpr int kJoinCtas = 8;  // a joined launch: a portable cluster

// One thread's column of all parameter gradients under one gate row, from few slots (norm_sums_kernel does the
// same with a warp's share each). Other CTAs wrote them a moment ago: read past L1.
__device__ __forceinline__ void finish_column(const NormSums& a, int c) {
  const auto sums = [&](const float* ws) {
    float2 s = make_float2(0.0f, 0.0f);
#pragma unroll
    for (int i = 0; i < kJoinCtas; ++i) {
      const bool in = i < a.units;
      s.x += in ? __ldcg(ws + 2 * i * static_cast<int64_t>(a.cols) + c) : 0.0f;
      s.y += in && a.bias ? __ldcg(ws + (2 * i + 1) * static_cast<int64_t>(a.cols) + c) : 0.0f;
    }
    return s;
  };
  if (a.dpre_weight != nullptr || a.dpre_bias != nullptr) {
    const float2 s = sums(a.ws2);
    if (a.dpre_weight != nullptr) a.dpre_weight[c] = s.x;
    if (a.dpre_bias != nullptr) a.dpre_bias[c] = s.y;
  }
  if (a.dpost_weight == nullptr && a.dpost_bias == nullptr && a.dgate == nullptr) return;
  const float2 s = sums(a.ws1);
  float w, b = 0.0f, gate = 1.0f;
  load_weight<1>(a.post_weight, a.params_f32, a.weight_offset, c, &w);
  if (a.post_bias != nullptr) load_param<1>(a.post_bias, a.params_f32, c, &b);
  if (a.gate != nullptr) load_param<1>(a.gate, a.params_f32, c, &gate);
  if (a.dgate != nullptr) a.dgate[c] = a.bias ? w * s.x + b * s.y : w * s.x;
  if (a.dpost_weight != nullptr) a.dpost_weight[c] = gate * s.x;
  if (a.dpost_bias != nullptr) a.dpost_bias[c] = gate * s.y;
}

// One row takes three steps with a sum over the row between them:
//   A  z2, g2 from dy and x_out;              sums of g2 and g2 * z2
//   B  d from those and dx_out, dx; z1, g1;   sums of g1 and g1 * z1
//   C  dh
// A CTA takes them in turn. In a cluster, where an exchange costs a trip between SMs, an iteration
// takes step A of row i, B of row i - 1 and C of row i - 2: the sums of two rows share one exchange,
// and A, which needs none, runs while they come in (16384 x 8192: 681 us in turn, 344 us so; in one
// CTA the registers it takes cost more than it gives, 184 us in turn and 240 us so at 16384 x 4096).
// Rows outside the segment are then read as zeros and not written; a stage of the ring holds dy and
// x_out of row i, dx_out and h of row i - 1.
//
// BIAS: whether A0 and dpre_bias are summed.
template <typename T, int READS, bool LAYER, bool BIAS, bool CLUSTER, bool STALL>
__global__ void __launch_bounds__(kMaxTeamWarps * 32, 1) norm_backward_kernel(const NormGradParams a) {
  using Cols = Columns<T, kGradElems, READS>;
  constexpr int VEC = Cols::VEC, N = Cols::N, EPT = kGradElems, P = EPT / 2;
  constexpr bool RING = READS != kSingles;
  constexpr int kStages = kBackwardRing<T>;
  constexpr int BEHIND = CLUSTER ? 1 : 0;  // rows that dx_out and h lie behind dy and x_out
  extern __shared__ uint4 dynamic[];  // weights: [2][P / 2][threads of the team]; ring
  __shared__ float4 slots[2][Team<CLUSTER>::kSlots];
  __shared__ float stage[CLUSTER ? 1 : kStageFloats];  // [teams][cols]
  __shared__ uint64_t bars[2];
  __shared__ int abort;
  Team<CLUSTER> team;
  if constexpr (CLUSTER) {
    if (threadIdx.x == 0) {
      abort = 0;
      mbar_init(&bars[0], 1);
      mbar_init(&bars[1], 1);
      fence_mbar_init();
    }
    team.ring_bars = bars;
    team.abort = &abort;
    team.status = a.status;
    if constexpr (STALL) team.wait_ns = a.wait_ns;
  }
  team.init(slots, a.warps);
  enter_stream();
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
  // the block's rows of each matrix; offsets inside them fit 32 bits (the host sees to it), but for the reads of
  // single elements, whose rows may lie any distance apart
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
    if (t == (a.teams > 1 ? 1 : 0)) {  // gate * (post_weight + offset)
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
    // this team's rows of the segment: first, first + step, ... Unsigned, as the row behind the last may pass 2^31.
    // (Counted from the block's first row instead: 16384 x 8192 RMS with 8 gates 358 us, 343 us so.)
    const int mine = seg - begin + ((cls - (seg - begin)) % a.classes + a.classes) % a.classes;  // class's first row
    const uint32_t first = static_cast<uint32_t>(begin) + static_cast<uint32_t>(mine + t * a.classes);
    const int n = first < static_cast<uint32_t>(seg_end) ? static_cast<int>(seg_end - first + step - 1) / step : 0;

    // the row to fetch next, and this thread's vector 0 of it in each matrix, as an offset from the
    // block's first row
    int ahead = 0;
    const int at_row = static_cast<int>(first - begin);
    int off[4] = {};
    if constexpr (RING) {
#pragma unroll
      for (int m = 0; m < 4; ++m) off[m] = (m < 2 ? at_row : at_row - BEHIND * step) * stride[m] + at.first;
    }
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
          at.mask(i, &v[i * VEC / 2]);
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
      float rstd_c = 0.0f;
      const int iterations = n > 0 ? n + 2 : 0;
      int last = iterations;
      if constexpr (STALL) {
        if (team.rank + 1 == team.ranks) last = min(iterations, a.stall_after);
      }
      for (int it = 0; it < last; ++it) {
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
        // of A's row i - 1 and B's row i - 2
        const float4 sums = it > 0 ? team.template collect<LAYER>() : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        if (!team.ok) break;  // another CTA's sums never came: the status word says so
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
        if (it + 1 < iterations)
          team.template publish<LAYER>(
              make_float4(sum_halves(s1), LAYER ? sum_halves(s0) : 0.0f, sum_halves(t1), LAYER ? sum_halves(t0) : 0.0f));
        out += step * a.cols;
        to = s;  // read for the last time above
        s += stage_bytes;
        if (s == ring_end) s = ring0;
      }
      if constexpr (STALL) team.ok = team.ok && last == iterations;
    }
    if constexpr (RING) cp_async_wait<0>();
    // every warp comes here, with its sums or after a wait that gave up: the CTA leaves as one
    if (CLUSTER && __syncthreads_or(!team.ok)) break;
    if (a.sums1) {
      float* sums = a.ws1 + ((block + group) * a.classes + cls) * 2 * a.cols;
      flush_sums(a, a1, at, sums, stage);
      if constexpr (BIAS) flush_sums(a, a0, at, sums + a.cols, stage);
    }
    seg = seg_end;
    if (seg < end) __syncthreads();  // the gate's weights are read no more
  }
  if (a.sums2) {
    float* out = a.ws2 + unit * 2 * a.cols;
    flush_sums(a, p1, at, out, stage);
    if constexpr (BIAS) flush_sums(a, p0, at, out + a.cols, stage);
  }
  if constexpr (CLUSTER) {
    cluster_barrier();  // no CTA leaves while another may still write its slots
  } else if (a.join) {
    // few rows: the CTAs are one cluster, whose barrier also orders their sums in global memory
    cluster_barrier();
    for (int c = cluster_rank() * blockDim.x + threadIdx.x; c < a.cols; c += gridDim.x * blockDim.x)
      finish_column(a.sums, c);
  }
}

// ---------------------------------------------------------------- parameter gradients
constexpr int kSumWarps = 32;

// 32 columns a CTA (one a lane); its warps share the slots of a sum, in a fixed order. blockIdx.y: 0 the
// pre-norm's sums, 1 the post norm's and the gate's.
__global__ void __launch_bounds__(kSumWarps * 32) norm_sums_kernel(const NormSums a) {
  __shared__ float2 part[kSumWarps][32];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int c = blockIdx.x * 32 + lane;
  const bool in = c < a.cols;
  enter_stream();
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
  // warps for a gate row, and gate rows at once
  const int each = max(1, kSumWarps / static_cast<int>(min(a.groups, int64_t{kSumWarps}))), at_once = kSumWarps / each;
  const int share = warp % each;
  for (int64_t g0 = 0; g0 < a.groups; g0 += at_once) {
    const int64_t g = g0 + warp / each;
    const bool mine = warp / each < at_once && g < a.groups;
    float2 s = make_float2(0.0f, 0.0f);
    if (mine && in) {
      int64_t n;
      const float* base = slots_of(g, n) + c;
#pragma unroll 8
      for (int64_t i = share; i < n; i += each) {
        s.x += base[i * 2 * a.cols];
        if (a.bias) s.y += base[i * 2 * a.cols + a.cols];
      }
    }
    if (each > 1) {
      __syncthreads();
      part[warp][lane] = s;
      __syncthreads();
      if (mine && share == 0)  // warp / each < at_once: its share lies inside the warps
        for (int k = 1; k < each; ++k) s.x += part[warp + k][lane].x, s.y += part[warp + k][lane].y;
    }
    if (mine && in && share == 0) add_group(g, s);
  }
  __syncthreads();
  part[warp][lane] = total;
  __syncthreads();
  if (warp == 0)
    for (int k = 1; k < kSumWarps; ++k) total.x += part[k][lane].x, total.y += part[k][lane].y;
  if (warp == 0 && in) {
    if (a.dpost_weight != nullptr) a.dpost_weight[c] = total.x;
    if (a.dpost_bias != nullptr) a.dpost_bias[c] = total.y;
  }
}

// ---------------------------------------------------------------- launches
// The backward pass's blocks of rows: one CTA (or cluster) an SM, at 128 registers a thread; more where
// a block would pass the 32-bit offsets that dx and dh are written with (9 clusters of 16 hold all rows
// of 65536 columns).
struct GradSplit {
  int64_t rows_per_block, blocks, classes;
  int64_t units() const { return blocks * classes; }
};
// Rows around a block's own that offsets are computed for, though nothing is accessed there.
constexpr int64_t kRowsAround = 8;  // in steps of a CTA's teams and classes
bool offsets_fit(int64_t rows, int64_t width, const RowCut& c) {
  return (rows + kRowsAround * c.classes * c.teams) * width <= INT32_MAX;
}
GradSplit grad_split(int64_t rows, int64_t cols, const RowCut& c, int num_sms) {
  GradSplit s{};
  s.classes = c.classes;
  const int64_t want = std::max<int64_t>(1, num_sms / c.cluster / c.classes);
  const int64_t quantum = c.classes * c.teams;
  s.rows_per_block = ceil_div(ceil_div(rows, want), quantum) * quantum;
  if (!offsets_fit(s.rows_per_block, cols, c))
    s.rows_per_block = (INT32_MAX / cols / quantum - kRowsAround) * quantum;
  s.blocks = ceil_div(rows, s.rows_per_block);
  return s;
}

// How a call is cut. `wide`: its matrices and parameters can be read by vectors, the first row `shift`
// elements behind a 16-byte boundary; `widest`: the longest step from one row to the next of any matrix.
constexpr int64_t kManyGates = 32;
struct BackwardCut {
  RowCut rows;
  GradSplit split;
};
BackwardCut backward_cut(int64_t rows, int64_t cols, int64_t groups, bool f32, bool wide, int64_t shift, int64_t widest,
                         int num_sms) {
  BackwardCut b{};
  // A gate row has a slot of sums for each class. With many gates of fewer rows than classes most slots would hold
  // zeros: one class then, element by element (51200 x 1023 bf16, a gate for each row: 421 MB of workspace and 7.0 ms,
  // 3355 MB and 13.7 ms by vectors; 64 rows of 1001: 38 and 122 us). Not with few gates (2 rows of 1001, 2 gates: 21
  // and 15 us) or two classes (64 rows of 1020: 38 and 35 us).
  const int64_t classes = row_classes(cols, f32 ? 4 : 8);
  wide = wide && !(classes > 2 && groups >= kManyGates && rows / groups < classes);
  b.rows = row_cut(cols, f32, wide, shift, false);
  b.split = grad_split(rows, cols, b.rows, num_sms);
  // vectors are read with 32-bit offsets inside a block, single elements with 64 bits
  if (wide && !offsets_fit(b.split.rows_per_block, widest, b.rows)) {
    b.rows = row_cut(cols, f32, false, 0, false);
    b.split = grad_split(rows, cols, b.rows, num_sms);
  }
  return b;
}

template <typename T, int READS, bool LAYER, bool BIAS, bool CLUSTER, bool STALL = false>
cudaError_t launch_backward(const NormGradParams& a, const RowCut& c, int64_t units, cudaStream_t stream,
                            const DeviceInfo& dev) {
  const auto kernel = norm_backward_kernel<T, READS, LAYER, BIAS, CLUSTER, STALL>;
  constexpr size_t ring = READS != kSingles ? kBackwardRing<T> * 4 * kGradElems * sizeof(T) : 0;  // of a thread
  static PerDevice<cudaError_t> ready;
  const cudaError_t e =
      ready.run(dev.device, [&] { return allow(reinterpret_cast<const void*>(kernel), (ring + 8 * kGradElems) * kMaxTeamWarps * 32, CLUSTER); });
  if (e != cudaSuccess) return e;
  const size_t dynamic = ring * c.threads() + static_cast<size_t>(8) * kGradElems * c.warps * 32;
  if (a.join)
    return launch_in_stream(kernel, dim3(static_cast<unsigned>(units)), c.threads(), dynamic, stream,
                            static_cast<int>(units), a);
  return launch_cut(kernel, a, units, c, dynamic, stream);
}

template <typename T, int READS, bool LAYER, bool BIAS>
cudaError_t pick_backward(const NormGradParams& a, const RowCut& c, int64_t units, cudaStream_t stream,
                          const DeviceInfo& dev) {
  // An injected stall runs a second copy of the kernel, with the biases' sums, wanted or not: whatever of the stall
  // the others carried, compared in every row or only before the first, cost them 2 to 3 %.
  if (a.stall_after >= 0) return launch_backward<T, READS, LAYER, true, true, true>(a, c, units, stream, dev);
  return c.cluster > 1 ? launch_backward<T, READS, LAYER, BIAS, true>(a, c, units, stream, dev)
                       : launch_backward<T, READS, LAYER, BIAS, false>(a, c, units, stream, dev);
}
// Matrices of unlike alignment take the kernel with all sums.
template <typename T>
cudaError_t pick_backward(const NormGradParams& a, bool layer, bool bias, const RowCut& c, int64_t units,
                          cudaStream_t stream, const DeviceInfo& dev) {
  if (c.reads == kSingles)
    return layer ? pick_backward<T, kSingles, true, true>(a, c, units, stream, dev)
                 : pick_backward<T, kSingles, false, true>(a, c, units, stream, dev);
  if (c.reads == kEdges && bias)
    return layer ? pick_backward<T, kEdges, true, true>(a, c, units, stream, dev)
                 : pick_backward<T, kEdges, false, true>(a, c, units, stream, dev);
  if (c.reads == kEdges)
    return layer ? pick_backward<T, kEdges, true, false>(a, c, units, stream, dev)
                 : pick_backward<T, kEdges, false, false>(a, c, units, stream, dev);
  if (bias)
    return layer ? pick_backward<T, kVectors, true, true>(a, c, units, stream, dev)
                 : pick_backward<T, kVectors, false, true>(a, c, units, stream, dev);
  return layer ? pick_backward<T, kVectors, true, false>(a, c, units, stream, dev)
               : pick_backward<T, kVectors, false, false>(a, c, units, stream, dev);
}

}  // namespace

int64_t norm_workspace_floats(int64_t rows, int64_t cols, int64_t groups, bool f32, int num_sms) {
  if (rows <= 0) return 0;
  int64_t most = 0;  // whether the rows can be read by vectors is known at the call alone
  for (const bool wide : {false, true}) {
    const GradSplit s = backward_cut(rows, cols, groups, f32, wide, 0, cols, num_sms).split;
    most = std::max(most, (2 * s.units() + groups * s.classes) * 2 * cols);
  }
  return most;
}

NormCut norm_backward_cut(int64_t rows, int64_t cols, int64_t groups, bool f32, bool wide, int64_t widest, int num_sms) {
  const BackwardCut b = backward_cut(rows, cols, groups, f32, wide, 0, widest, num_sms);
  return {b.rows.reads != kSingles, b.rows.cluster, b.rows.warps, b.rows.teams, b.rows.classes, b.split.rows_per_block,
          b.split.blocks};
}

int launch_block_norm_backward(const bsq_block_norm_grad_args& g, cudaStream_t stream, const DeviceInfo& dev) {
  const bool f32 = (g.flags & BSQ_FLAG_SRC_F32) != 0, layer = g.kind == BSQ_NORM_LAYER;
  const int64_t es = f32 ? 4 : 2;
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
  a.status = dev.status;
  a.stall_after = -1;
  a.wait_ns = kWaitLimitNs;
  a.sums1 = g.dpost_weight != nullptr || g.dpost_bias != nullptr || g.dgate != nullptr;
  a.sums2 = g.dpre_weight != nullptr || g.dpre_bias != nullptr;
  const void* x_out = g.dy != nullptr ? g.x_out : nullptr;
  int64_t shift;
  bool wide = same_offsets({{g.dy, g.dy_stride}, {x_out, g.x_out_stride}, {g.dx_out, g.dx_out_stride}, {g.h, g.h_stride},
                            {g.dx, g.cols}, {g.dh, g.cols}}, g.cols, es, &shift);
  // Rows of whole vectors read their parameters by vectors too. One that is not aligned turns the call to single
  // elements, without a ring (from cold caches, 51200 x 1024 bf16: 621 us, 139 us by vectors; 16384 x 8192: 1711, 352).
  const int64_t pb = g.cols * (a.params_f32 ? 4 : 2);
  wide = wide && (row_classes(g.cols, 16 / es) > 1 || (shift == 0 && wide_ok(g.post_weight, 0) && wide_ok(g.pre_weight, 0) &&
                                                       wide_ok(g.gate, groups > 1 ? pb : 0)));
  const int64_t widest = std::max({g.cols, g.dy_stride, x_out != nullptr ? g.x_out_stride : 0, g.dx_out_stride, g.h_stride});
  const BackwardCut cut = backward_cut(g.rows, g.cols, groups, f32, wide, shift, widest, dev.num_sms);
  const RowCut& c = cut.rows;
  const GradSplit& s = cut.split;
  if (c.cluster > 1) {  // the kernels of one CTA a row wait on no barrier that could run out
    const StallInjection inj = take_stall(BSQ_KERNEL_NORM);
    a.stall_after = static_cast<int32_t>(std::min<int64_t>(inj.after, INT32_MAX));
    a.wait_ns = inj.limit_ns;
  }
  // No more rows than teams in 8 CTAs, and one gate row: they run as one cluster that joins its sums itself, which
  // saves the second launch (layer norm on both sides, bf16, all parameters, device time in one launch / in two:
  // 40 x 768 10.5 / 11.9 us, 128 x 64 8.1 / 9.8, 8 x 4096 15.6 / 17.5). Fewer CTAs with more rows each lose it again
  // (100 x 768 in 8 CTAs: 14.3 / 12.1), and so do more gate rows, whose sums one thread would add in turn (20 x 768
  // with 2 gates 11.7 / 11.7, with 5 18.1 / 15.4).
  a.join = (a.sums1 || a.sums2) && c.cluster == 1 && s.units() <= kJoinCtas && groups == 1;
  a.warps = c.warps, a.teams = c.teams, a.classes = static_cast<int32_t>(c.classes), a.shift = c.shift;
  a.rows_per_block = s.rows_per_block;
  a.ws2 = static_cast<float*>(g.workspace);
  a.ws1 = a.ws2 + s.units() * 2 * g.cols;
  // A0 is the gradient of the post bias, and part of the gate's behind one
  const bool bias = c.reads == kSingles || g.dpost_bias != nullptr || g.dpre_bias != nullptr ||
                    (g.dgate != nullptr && a.post && g.post_bias != nullptr);
  NormSums& n = a.sums;
  n.rows = g.rows, n.group_rows = a.group_rows, n.groups = groups;
  n.rows_per_block = s.rows_per_block, n.units = s.units(), n.cols = a.cols, n.classes = a.classes;
  n.weight_offset = g.weight_offset, n.params_f32 = a.params_f32, n.bias = bias;
  n.post_weight = a.post ? g.post_weight : nullptr, n.post_bias = a.post ? g.post_bias : nullptr, n.gate = g.gate;
  n.ws1 = a.ws1, n.ws2 = a.ws2;
  n.dpost_weight = g.dpost_weight, n.dpost_bias = g.dpost_bias, n.dgate = g.dgate;
  n.dpre_weight = g.dpre_weight, n.dpre_bias = g.dpre_bias;
  cudaError_t e = f32 ? pick_backward<float>(a, layer, bias, c, s.units(), stream, dev)
                      : pick_backward<uint16_t>(a, layer, bias, c, s.units(), stream, dev);
  if (e != cudaSuccess) return BSQ_ERR_LAUNCH;
  if ((a.sums1 || a.sums2) && !a.join) {
    const dim3 grid(static_cast<unsigned>(ceil_div(g.cols, 32)), a.sums1 ? 2 : 1);
    e = launch_in_stream(norm_sums_kernel, grid, kSumWarps * 32, 0, stream, 1, a.sums);
  }
  return e == cudaSuccess ? BSQ_OK : BSQ_ERR_LAUNCH;
}

}  // namespace bsq
