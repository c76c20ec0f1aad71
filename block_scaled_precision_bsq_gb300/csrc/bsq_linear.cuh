// bsq_linear.cuh -- block-scaled products on the 5th-generation tensor cores whose rows may be
// grouped by expert in ragged segments, with activation, residual and the activation's derivative in
// the epilogue, and the experts' weight gradients:
//   v[r, c] = alpha * sum_k Ahat[r, k] * Bhat_e[c, k] + bias_e[c],  e = the expert of row r
//   out = residual + act(v), pre = v                    (kLinPlain, kLinAct, kLinRes, kLinF32, kLinResF32)
//   out = v * act'(aux), sums[c] = sum over rows of out  (kLinGrad)
//   out_e[r, c] = alpha * sum over expert e's k of Ahat[r, k] * Bhat[c, k]        (contract)
//
// Which operand is whose. Rows come in segments of any length, columns (a layer's features) in
// multiples of 128. The 2-SM MMA has M fixed at 256 and N free in steps: so the features are the MMA's
// M side (each SM of the pair holds 128 of them) and the rows its N side, 32 to 256 at a time: a
// segment of 5 rows costs an MMA of 32 columns, not of 256 rows. The accumulator then holds the result
// transposed: a TMEM lane is a feature, a column a row, so bias and column sums are one register a thread.
//
// Windows. The rows' block scales lie in tiles of 128 rows, and the tensor cores' scale copy takes
// whole tiles. A unit of work is therefore a window of up to 256 rows that begins at a multiple of 128,
// times 256 features. A segment that begins inside a tile is computed from the tile's first row; the
// rows before it belong to another expert, cost MMA columns and are not stored. So segments need no
// alignment, and rows sorted without gaps (a few tokens while serving) are not padded to 128 each.
//
// Roles of a CTA pair as in bsq_gemm.cu: warp 0 loads by TMA into a ring, warp 1 of the leader issues scale
// copies and MMAs, the other warps drain the accumulator. Every wait is bounded.
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>
#include <type_traits>

#include "bsq_device.cuh"
#include "bsq_linear.h"

namespace bsq {
namespace {

constexpr int kFeatTile = 256;  // features of a unit (the pair's M)
constexpr int kRowTile = 256;   // most rows of a window (the MMA's N)
constexpr int kSpanBytes = 128;  // depth bytes per stage: one 128-byte swizzle span per row
constexpr int kEpiWarp0 = 2;
constexpr uint32_t kTmemAll = 512;

template <int KIND>
struct LinEpi {
  static constexpr bool kAux = KIND == kLinRes || KIND == kLinGrad || KIND == kLinResF32;
  static constexpr bool kF32 = KIND == kLinF32 || KIND == kLinResF32;
  // The activation alone is bound by its arithmetic: 16 warps. The others wait for memory and would
  // take the operand ring's shared memory for their staging.
  static constexpr int kWarps = KIND == kLinAct ? 16 : 8;
  static constexpr int kWarpCols = 4 * kRowTile / kWarps;  // rows of the window that a warp drains
  static constexpr int kChunks = kWarpCols / 32;
  static constexpr int kChunkBytes = 32 * 32 * (kF32 ? 4 : 2);
  // One staging chunk, or two that bring the auxiliary values and take the results in their places; a
  // residual's pre-activation goes through a chunk of its own.
  static constexpr int kBufs = kAux ? 2 : 1;
  static constexpr bool kOwnPre = KIND == kLinRes || KIND == kLinResF32;
  static constexpr int kBytes = kBufs * kChunkBytes + (kOwnPre ? 2048 : 0);
  static constexpr int kThreads = (kEpiWarp0 + kWarps) * 32;
};

// 512-byte scale atoms (128 rows x 4 scale columns) per stage, and values per MMA (32 bytes).
template <int FMT>
struct LinFmt {
  static constexpr int kAtoms = FMT == BSQ_NVFP4 ? 4 : FMT == BSQ_MXFP4 ? 2 : 1;
  static constexpr int kMmaDepth = FMT == BSQ_MXFP8 ? 32 : 64;
  static constexpr int kAtomDepth = FMT == BSQ_NVFP4 ? 64 : 128;
  static constexpr int kSfCols = 12 * kAtoms;  // TMEM columns of a stage's scales: 4 per atom of 128 rows
};

template <int FMT, int KIND>
struct LinSmem {
  static constexpr int kABytes = 128 * kSpanBytes;  // features
  static constexpr int kBBytes = 128 * kSpanBytes;  // rows
  static constexpr int kSfaBytes = LinFmt<FMT>::kAtoms * 512;
  static constexpr int kSfbBytes = 2 * kSfaBytes;
  static constexpr int kStageBytes = kABytes + kBBytes + kSfaBytes + kSfbBytes;
  static constexpr int kFixed = LinEpi<KIND>::kWarps * LinEpi<KIND>::kBytes + (BSQ_MAX_EXPERTS + 2) * 4 + 512;
  static constexpr int kRoom = (232448 - kFixed) / kStageBytes;
  static constexpr int kTmemRoom = (512 - kRowTile) / LinFmt<FMT>::kSfCols;
  static constexpr int S = kRoom < kTmemRoom ? (kRoom < 6 ? kRoom : 6) : (kTmemRoom < 6 ? kTmemRoom : 6);
  static constexpr int a_off = 0;
  static constexpr int b_off = a_off + S * kABytes;
  static constexpr int sfa_off = b_off + S * kBBytes;
  static constexpr int sfb_off = sfa_off + S * kSfaBytes;
  static constexpr int epi_off = sfb_off + S * kSfbBytes;
  static constexpr int bar_off = epi_off + LinEpi<KIND>::kWarps * LinEpi<KIND>::kBytes;
  static constexpr int kAuxBars = LinEpi<KIND>::kAux ? 2 * LinEpi<KIND>::kWarps : 0;
  static constexpr int kNumBars = 2 * S + 3 + kAuxBars;
  static constexpr int misc_off = bar_off + kNumBars * 8;
  static constexpr int prefix_off = misc_off + 16;
  static constexpr int total = prefix_off + (BSQ_MAX_EXPERTS + 2) * 4;
  static_assert(S >= 3 && total <= 232448, "shared memory budget");
  static_assert(epi_off % 128 == 0, "staging alignment");
};

// Instruction descriptor, as in bsq_gemm.cu but for the free N.
template <int FMT>
__device__ __forceinline__ uint32_t lin_idesc(uint32_t n, uint32_t sf_id) {
  const uint32_t t = (FMT == BSQ_MXFP8) ? 0u : 1u;
  const uint32_t ue8m0 = (FMT == BSQ_NVFP4) ? 0u : 1u;
  return (sf_id << 4) | (t << 7) | (t << 10) | ((n >> 3) << 17) | (ue8m0 << 23) | (2u << 27) | (sf_id << 29);
}

__device__ __forceinline__ void tma_load_4d_to_leader(void* smem_dst, const void* tmap, uint32_t leader_bar, int32_t c0,
                                                      int32_t c1, int32_t c2, int32_t c3, uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.4d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes.L2::cache_hint "
      "[%0], [%1, {%3, %4, %5, %6}], [%2], %7;" ::"r"(smem_u32(smem_dst)),
      "l"(reinterpret_cast<uint64_t>(tmap)), "r"(leader_bar), "r"(c0), "r"(c1), "r"(c2), "r"(c3), "l"(policy)
      : "memory");
}

// ---------------------------------------------------------------------------- activations
// exp2 and reciprocal of the special-function unit: 2^-22 relative each, below the fp32 sums' own error.
__device__ __forceinline__ float ex2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float rcp_fast(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// The normal distribution function Phi(v), and gauss = exp(-v^2 / 2): Abramowitz & Stegun, Handbook of
// Mathematical Functions, formula 7.1.26 for erfc(z), z = |v| / sqrt 2, |error| <= 1.5e-7.
__device__ __forceinline__ float normal_cdf(float v, float& gauss) {
  const float z = fabsf(v) * 0.7071067811865476f;
  const float t = rcp_fast(fmaf(0.3275911f, z, 1.0f));
  float p = fmaf(0.5f * 1.061405429f, t, 0.5f * -1.453152027f);
  p = fmaf(p, t, 0.5f * 1.421413741f);
  p = fmaf(p, t, 0.5f * -0.284496736f);
  p = fmaf(p, t, 0.5f * 0.254829592f);
  gauss = ex2_fast(z * z * -1.4426950408889634f);
  const float h = p * t * gauss;  // erfc(z) / 2
  return v >= 0.0f ? 1.0f - h : h;
}
__device__ __forceinline__ float logistic(float v) { return rcp_fast(1.0f + ex2_fast(v * -1.4426950408889634f)); }
constexpr float kTanhA = 1.5957691216057308f;             // 2 sqrt(2 / pi): (1 + tanh u) / 2 = logistic(2 u)
constexpr float kTanhB = 1.5957691216057308f * 0.044715f;

template <int ACT>
__device__ __forceinline__ float act_value(float v) {
  if constexpr (ACT == BSQ_ACT_GELU) {
    float gauss;
    return v * normal_cdf(v, gauss);
  } else if constexpr (ACT == BSQ_ACT_GELU_TANH) {
    return v * logistic(v * fmaf(kTanhB, v * v, kTanhA));
  } else if constexpr (ACT == BSQ_ACT_SILU) {
    return v * logistic(v);
  } else if constexpr (ACT == BSQ_ACT_RELU) {
    return v < 0.0f ? 0.0f : v;  // NaN stays NaN
  } else {
    return v;
  }
}
template <int ACT>
__device__ __forceinline__ float act_slope(float v) {
  if constexpr (ACT == BSQ_ACT_GELU) {
    float gauss;
    const float p = normal_cdf(v, gauss);
    return fmaf(v * 0.3989422804014327f, gauss, p);
  } else if constexpr (ACT == BSQ_ACT_GELU_TANH) {
    // past 12 the logistic is 0 or 1 to the last bit; v^2 stays finite
    const float x = fminf(fmaxf(v, -12.0f), 12.0f);
    const float s = logistic(x * fmaf(kTanhB, x * x, kTanhA));
    const float r = fmaf(x * (s - s * s), fmaf(3.0f * kTanhB, x * x, kTanhA), s);
    return v != v ? v : r;
  } else if constexpr (ACT == BSQ_ACT_SILU) {
    const float s = logistic(v);
    return s * fmaf(v, 1.0f - s, 1.0f);
  } else if constexpr (ACT == BSQ_ACT_RELU) {
    return v > 0.0f ? 1.0f : 0.0f;
  } else {
    return 1.0f;
  }
}
template <typename F>
__device__ __forceinline__ void by_activation(int act, F&& f) {
  switch (act) {
    case BSQ_ACT_GELU: f(std::integral_constant<int, BSQ_ACT_GELU>{}); break;
    case BSQ_ACT_GELU_TANH: f(std::integral_constant<int, BSQ_ACT_GELU_TANH>{}); break;
    case BSQ_ACT_SILU: f(std::integral_constant<int, BSQ_ACT_SILU>{}); break;
    case BSQ_ACT_RELU: f(std::integral_constant<int, BSQ_ACT_RELU>{}); break;
    default: break;
  }
}

// ---------------------------------------------------------------------------- units of work
struct LinArgs {
  const int32_t* counts;  // experts' rows, NULL: one segment of all rows
  const int32_t* offsets;
  const uint16_t* bias;
  const float* ga;  // NVFP4: per-tensor scales
  const float* gb;
  uint8_t* out;
  uint8_t* pre;
  float* sums;
  int* status;
  int64_t stall_after;
  uint64_t wait_ns;
  int rows, cols, depth, experts, tiles_c, mmas, act;
  int contract, aux;
};

// A window of rows times 256 features. Rows [lo, live) are computed, [live, hi) are zeros.
struct Unit {
  int w0, lo, live, hi;
  int n;        // MMA columns; 0: no product, zeros alone
  int ct, e;    // tile of features, expert
  int window;
  int mmas, kx, ka;  // MMAs along the depth, first byte and first scale atom
  int64_t row0;      // result row of row 0
};

// Expert e's segment, whatever the two arrays hold: inside [0, limit), counts inside the segment. Behind
// the last expert (e = experts): the rows of none.
__device__ __forceinline__ void segment(const LinArgs& a, int e, int limit, int& off, int& count, int& end) {
  off = min(max(a.offsets[e], 0), limit);
  end = limit;
  count = 0;
  if (e < a.experts) {
    end = min(max(a.offsets[e + 1], off), limit);
    count = min(max(a.counts[e], 0), end - off);
  }
}
__device__ __forceinline__ int windows_of(int off, int end) {
  return end > off ? (end - (off & ~127) + kRowTile - 1) / kRowTile : 0;
}

template <int FMT>
__device__ __forceinline__ Unit unit_at(const LinArgs& a, const int* prefix, int u) {
  Unit t;
  t.window = u / a.tiles_c;
  t.ct = u - t.window * a.tiles_c;
  t.e = 0;
  t.mmas = a.mmas;
  t.kx = t.ka = 0;
  t.row0 = 0;
  if (a.contract) {
    const int windows = (a.rows + kRowTile - 1) / kRowTile;
    t.e = t.window / windows;
    t.w0 = t.lo = (t.window - t.e * windows) * kRowTile;
    t.hi = min(t.w0 + kRowTile, a.rows);
    t.row0 = static_cast<int64_t>(t.e) * a.rows;
    int off, count, end;
    segment(a, t.e, a.depth, off, count, end);
    if (off & 127) {  // the scales of the depth lie in groups of 128: no product, and the caller learns of it
      if (count > 0) atomicCAS(a.status, 0, BSQ_ERR_SHAPE);
      count = 0;
    }
    t.live = count > 0 ? t.hi : t.lo;
    t.mmas = (count + LinFmt<FMT>::kMmaDepth - 1) / LinFmt<FMT>::kMmaDepth;
    t.kx = FMT == BSQ_MXFP8 ? off : off / 2;
    t.ka = off / LinFmt<FMT>::kAtomDepth;
  } else {
    int off = 0, count = a.rows, end = a.rows, first = 0;
    if (a.counts != nullptr) {
      int below = a.experts + 1;  // the last segment that does not begin behind this window
      while (below - t.e > 1) {
        const int mid = (t.e + below) >> 1;
        if (prefix[mid] <= t.window) t.e = mid;
        else below = mid;
      }
      first = prefix[t.e];
      segment(a, t.e, a.rows, off, count, end);
    }
    t.w0 = (off & ~127) + (t.window - first) * kRowTile;
    t.lo = max(t.w0, off);
    t.hi = min(t.w0 + kRowTile, end);
    t.live = min(t.hi, max(off + count, t.lo));
  }
  t.n = t.live > t.lo ? (t.live - t.w0 + 31) & ~31 : 0;
  return t;
}

// ---------------------------------------------------------------------------- the kernel
template <int FMT, int KIND>
__global__ void __launch_bounds__(LinEpi<KIND>::kThreads, 1)
    linear_kernel(const __grid_constant__ CUtensorMap mapW, const __grid_constant__ CUtensorMap mapX,
                  const __grid_constant__ CUtensorMap mapXs, const __grid_constant__ CUtensorMap mapSfw,
                  const __grid_constant__ CUtensorMap mapSfx, const __grid_constant__ CUtensorMap mapOut,
                  const __grid_constant__ CUtensorMap mapPre, const __grid_constant__ CUtensorMap mapAux,
                  const LinArgs args) {
  using E = LinEpi<KIND>;
  using L = LinSmem<FMT, KIND>;
  using P = LinFmt<FMT>;
  constexpr int S = L::S;
  extern __shared__ __align__(1024) uint8_t smem[];
  if (smem_u32(smem) & 1023u) {  // the swizzled tiles need it (uniform: all threads leave)
    if (threadIdx.x == 0) atomicCAS(args.status, 0, BSQ_ERR_LAUNCH);
    return;
  }
  uint64_t* full_bar = reinterpret_cast<uint64_t*>(smem + L::bar_off);  // leader: both CTAs' stage landed
  uint64_t* empty_bar = full_bar + S;                                   // the pair's MMAs are done with a stage
  uint64_t* tmem_full = full_bar + 2 * S;       // a unit's accumulator is complete
  uint64_t* tmem_empty = full_bar + 2 * S + 1;  // leader: both CTAs drained it
  uint64_t* drain_bar = full_bar + 2 * S + 2;
  uint64_t* aux_bar = full_bar + 2 * S + 3;     // [warp][buffer]
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(smem + L::misc_off);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + L::misc_off + 4);
  int* prefix = reinterpret_cast<int*>(smem + L::prefix_off);

  const uint32_t warp = threadIdx.x >> 5;
  const uint32_t lane = threadIdx.x & 31u;
  const uint32_t rank = cluster_rank();
  const bool leader = rank == 0;

  if (threadIdx.x == 0) {
    for (int s = 0; s < S; ++s) {
      mbar_init(&full_bar[s], 1);
      mbar_init(&empty_bar[s], 1);
    }
    mbar_init(tmem_full, 1);
    mbar_init(tmem_empty, 2 * E::kWarps);
    mbar_init(drain_bar, 1);
    for (int i = 0; i < L::kAuxBars; ++i) mbar_init(&aux_bar[i], 1);
    *abort_flag = 0;
    fence_mbar_init();
    prefetch_tmap(&mapW);
    prefetch_tmap(&mapX);
    prefetch_tmap(&mapXs);
    prefetch_tmap(&mapSfw);
    prefetch_tmap(&mapSfx);
    prefetch_tmap(&mapOut);
    if constexpr (E::kAux) prefetch_tmap(&mapAux);
  }
  if (warp == 1) {
    tmem_alloc_pair(tmem_holder, kTmemAll);
    tmem_relinquish_pair();
  }
  launch_dependents();
  grid_dependency_wait();  // inputs and outputs may belong to the previous kernel until here
  // windows ahead of each expert's first
  int num_units;
  if (args.counts != nullptr && !args.contract) {
    for (int e = threadIdx.x; e <= args.experts; e += E::kThreads) {
      int off, count, end;
      segment(args, e, args.rows, off, count, end);
      prefix[e + 1] = windows_of(off, end);
    }
    __syncthreads();
    if (warp == 0) {
      int carry = 0;
      if (lane == 0) prefix[0] = 0;
      for (int base = 0; base <= args.experts; base += 32) {
        const int i = base + static_cast<int>(lane);
        int v = i <= args.experts ? prefix[i + 1] : 0;
#pragma unroll
        for (int d = 1; d < 32; d *= 2) {
          const int o = __shfl_up_sync(0xffffffffu, v, d);
          if (static_cast<int>(lane) >= d) v += o;
        }
        v += carry;
        if (i <= args.experts) prefix[i + 1] = v;
        carry = __shfl_sync(0xffffffffu, v, 31);
      }
    }
    tc_fence_before();
    __syncthreads();
    num_units = prefix[args.experts + 1] * args.tiles_c;
  } else {
    num_units = (args.contract ? args.experts : 1) * ((args.rows + kRowTile - 1) / kRowTile) * args.tiles_c;
    tc_fence_before();
    __syncthreads();
  }
  cluster_sync_all();  // barriers of both CTAs initialised before any remote arrival
  tc_fence_after();
  const uint32_t tmem_base = *tmem_holder;
  const int first_unit = static_cast<int>(cluster_id_x());
  const int stride = static_cast<int>(num_clusters_x());

  if (warp == 0 && lane == 0) {
    // ------------------------------------------------------------------ TMA producer
    const uint64_t keep = l2_policy_evict_last();
    int stage = 0;
    uint32_t phase = 0;
    bool ok = true;
    int64_t armed = 0;
    auto produce = [&](auto stall) {
      for (int u = first_unit; u < num_units && ok; u += stride) {
        const Unit t = unit_at<FMT>(args, prefix, u);
        if (t.n == 0) continue;
        const int boxes = (t.n + 63) / 64, tiles = t.n > 128 ? 2 : 1;  // 32-row boxes of this CTA's half; scale tiles
        const uint32_t bytes = L::kABytes + L::kSfaBytes + boxes * 32 * kSpanBytes + tiles * L::kSfaBytes;
        const int x_row = t.w0 + static_cast<int>(rank) * (t.n / 2);
        const int w_row = t.ct * kFeatTile + static_cast<int>(rank) * 128;
        const int expert = args.contract ? 0 : t.e;
        const int spans = (t.mmas + 3) / 4;
        for (int s = 0; s < spans; ++s) {
          if constexpr (decltype(stall)::value) {
            if (armed == args.stall_after) {  // injected stall: no more loads, none announced
              ok = false;
              break;
            }
          }
          if (!mbar_wait_bounded(&empty_bar[stage], phase ^ 1u, abort_flag, args.status, args.wait_ns)) {
            ok = false;
            break;
          }
          if (leader) mbar_arrive_expect_tx(&full_bar[stage], 2 * bytes);
          const uint32_t bar = smem_u32(&full_bar[stage]) & ~kClusterRankBit;  // the leader's full[stage]
          const int kx = t.kx + s * kSpanBytes, ka = t.ka + s * P::kAtoms;
          tma_load_3d_to_leader(smem + L::a_off + stage * L::kABytes, &mapW, bar, kx, w_row, expert, keep);
          uint8_t* const xs = smem + L::b_off + stage * L::kBBytes;
          if (boxes == 4) {
            tma_load_2d_to_leader(xs, &mapX, bar, kx, x_row, keep);
          } else {
            for (int i = 0; i < boxes; ++i)
              tma_load_2d_to_leader(xs + i * 32 * kSpanBytes, &mapXs, bar, kx, x_row + 32 * i, keep);
          }
          tma_load_4d_to_leader(smem + L::sfa_off + stage * L::kSfaBytes, &mapSfw, bar, 0, ka,
                                2 * t.ct + static_cast<int>(rank), expert, keep);
          for (int i = 0; i < tiles; ++i)
            tma_load_3d_to_leader(smem + L::sfb_off + stage * L::kSfbBytes + i * L::kSfaBytes, &mapSfx, bar, 0, ka,
                                  (t.w0 >> 7) + i, keep);
          ++armed;
          if (++stage == S) {
            stage = 0;
            phase ^= 1u;
          }
        }
      }
    };
    if (args.stall_after < 0) produce(std::false_type{});
    else produce(std::true_type{});
    if (leader) wait_armed_stages(full_bar, S, armed, args.status, args.wait_ns);
  } else if (warp == 1 && leader) {
    // ------------------------------------------------------------------ MMA issuer
    const bool issuer = elect_one_sync();
    int stage = 0;
    uint32_t phase = 0, acc_phase = 0;
    bool ok = true;
    const uint32_t a_s0 = smem_u32(smem + L::a_off), b_s0 = smem_u32(smem + L::b_off);
    const uint32_t sfa_s0 = smem_u32(smem + L::sfa_off), sfb_s0 = smem_u32(smem + L::sfb_off);
    const uint32_t sf_t0 = tmem_base + kRowTile;
    for (int u = first_unit; u < num_units && ok; u += stride) {
      const Unit t = unit_at<FMT>(args, prefix, u);
      if (t.n == 0) continue;
      if (!mbar_wait_bounded_warp(tmem_empty, acc_phase ^ 1u, abort_flag, args.status, args.wait_ns)) break;
      acc_phase ^= 1u;
      tc_fence_after();
      const int spans = (t.mmas + 3) / 4;
      for (int s = 0; s < spans; ++s) {
        if (!mbar_wait_bounded_warp(&full_bar[stage], phase, abort_flag, args.status, args.wait_ns)) {
          ok = false;
          break;
        }
        tc_fence_after();
        const uint32_t sfa_t = sf_t0 + stage * P::kSfCols;
        const uint32_t sfb_t = sfa_t + 4 * P::kAtoms;
        const uint32_t sfa_s = sfa_s0 + stage * L::kSfaBytes;
        const uint32_t sfb_s = sfb_s0 + stage * L::kSfbBytes;
        const uint64_t adesc = smem_desc(a_s0 + stage * L::kABytes, 16, 1024, kSwizzle128B);
        const uint64_t bdesc = smem_desc(b_s0 + stage * L::kBBytes, 16, 1024, kSwizzle128B);
        if (issuer) {
#pragma unroll
          for (int i = 0; i < P::kAtoms; ++i)
            tc_cp_pair_32x128b_warpx4(sfa_t + 4 * i, smem_desc(sfa_s + 512 * i, 128, 128, kSwizzleNone));
#pragma unroll
          for (int i = 0; i < P::kAtoms; ++i)
            tc_cp_pair_32x128b_warpx4(sfb_t + 8 * i, smem_desc(sfb_s + 512 * i, 128, 128, kSwizzleNone));
          if (t.n > 128) {
#pragma unroll
            for (int i = 0; i < P::kAtoms; ++i)
              tc_cp_pair_32x128b_warpx4(sfb_t + 8 * i + 4,
                                        smem_desc(sfb_s + L::kSfaBytes + 512 * i, 128, 128, kSwizzleNone));
          }
          const int last = t.mmas - 4 * s;  // MMAs left: the depth may end inside the span
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            if (k >= last) break;
            uint32_t sfa = sfa_t, sfb = sfb_t, id = 0;
            if constexpr (FMT == BSQ_MXFP8) {
              id = k;
            } else if constexpr (FMT == BSQ_NVFP4) {
              sfa += 4 * k;
              sfb += 8 * k;
            } else {
              sfa += 4 * (k >> 1);
              sfb += 8 * (k >> 1);
              id = 2 * (k & 1);
            }
            tc_mma_pair<FMT>(tmem_base, adesc + 2 * k, bdesc + 2 * k, lin_idesc<FMT>(t.n, id), sfa, sfb,
                             (k > 0 || s > 0) ? 1u : 0u);
          }
          tc_commit_pair_mc(&empty_bar[stage], 0x3);
        }
        __syncwarp();
        if (++stage == S) {
          stage = 0;
          phase ^= 1u;
        }
      }
      if (ok && issuer) tc_commit_pair_mc(tmem_full, 0x3);
      __syncwarp();
    }
    if (issuer) tc_commit_pair(drain_bar);  // all tensor-core work ends before TMEM is released
    __syncwarp();
    mbar_wait_bounded(drain_bar, 0, nullptr, args.status, args.wait_ns);
  } else if (warp >= static_cast<uint32_t>(kEpiWarp0)) {
    // ------------------------------------------------------------------ epilogue (both CTAs)
    const uint32_t w = warp - kEpiWarp0;
    const uint32_t quad = warp & 3u;  // TMEM lanes this warp may read: 32 features
    const int c_base = static_cast<int>(w >> 2) * E::kWarpCols;
    uint8_t* const bufs = smem + L::epi_off + w * E::kBytes;
    uint8_t* const pre_buf = E::kOwnPre ? bufs + E::kBufs * E::kChunkBytes : bufs;
    uint64_t* const my_bar = aux_bar + 2 * w;
    const uint32_t tmem_empty_leader = mapa_shared(smem_u32(tmem_empty), 0);
    float alpha = 1.0f;
    if constexpr (FMT == BSQ_NVFP4) alpha = __fmul_rn(*args.ga, *args.gb);
    uint32_t acc_phase = 0, aux_phase = 0, pending = 0;

    // rows [r0, r0 + 32) of a staged chunk to `dst`: one tensor store where all rows are this unit's
    auto store = [&](const uint8_t* buf, const CUtensorMap* map, uint8_t* dst, int es, int64_t row0, int r0, int f0,
                     const Unit& t) {
      if (r0 >= t.lo && r0 + 32 <= t.hi) {
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          tma_store_2d(map, buf, f0, static_cast<int32_t>(row0 + r0));
          bulk_commit_group();
        }
      } else {
        __syncwarp();
        const int vec = 16 / es;  // values of a 16-byte piece; a row of the chunk has 2 es pieces
        for (int i = static_cast<int>(lane); i < 64 * es; i += 32) {
          const int c = i / (2 * es), piece = i % (2 * es);
          const int r = r0 + c, f = f0 + piece * vec;
          if (r >= t.lo && r < t.hi && f < args.cols)
            *reinterpret_cast<uint4*>(dst + ((row0 + r) * args.cols + f) * es) =
                *reinterpret_cast<const uint4*>(buf + c * 32 * es + piece * 16);
        }
        __syncwarp();
      }
    };

    for (int u = first_unit; u < num_units; u += stride) {
      const Unit t = unit_at<FMT>(args, prefix, u);
      const int f0 = t.ct * kFeatTile + static_cast<int>(rank) * 128 + static_cast<int>(quad) * 32;
      const int f = f0 + static_cast<int>(lane);
      const bool mine = f0 < args.cols;
      const int r_base = t.w0 + c_base;
      float bias = 0.0f;
      if (args.bias != nullptr && f < args.cols)
        bias = __uint_as_float(static_cast<uint32_t>(args.bias[static_cast<int64_t>(t.e) * args.cols + f]) << 16);
      // chunks that hold computed rows, and their auxiliary values: two of them on the way at a time
      const int j_first = max(0, (t.lo - r_base) >> 5);
      const int j_end = mine && t.n > 0 ? min(E::kChunks, (t.live - r_base + 31) >> 5) : 0;
      auto aux_load = [&](int j) {
        if constexpr (E::kAux) {
          if (args.aux && j < j_end) {
            const int b = j & 1;
            pending |= 1u << b;
            if (lane == 0) {
              mbar_arrive_expect_tx(&my_bar[b], E::kChunkBytes);
              tma_load_2d(bufs + b * E::kChunkBytes, &mapAux, &my_bar[b], f0, r_base + 32 * j);
            }
          }
        }
      };
      if constexpr (E::kAux) {
        if (lane == 0) bulk_wait_group_read<0>();  // the last unit's stores have left the chunks
        fence_proxy_async_smem();
        __syncwarp();
        aux_load(j_first);
        aux_load(j_first + 1);
      }
      uint32_t acc[E::kChunks][32];
      if (t.n > 0) {
        if (!mbar_wait_bounded(tmem_full, acc_phase, abort_flag, args.status, args.wait_ns)) break;
        acc_phase ^= 1u;
        tc_fence_after();
        __syncwarp();
#pragma unroll
        for (int j = 0; j < E::kChunks; ++j)
          if (c_base + 32 * j < t.n) tmem_ld_32x32b_x32(tmem_base + ((quad * 32u) << 16) + c_base + 32 * j, acc[j]);
        tmem_ld_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_remote(tmem_empty_leader);
      }
      float colsum = 0.0f;
      bool gone = false;
#pragma unroll
      for (int j = 0; j < E::kChunks; ++j) {
        const int r0 = r_base + 32 * j;
        if (!mine || r0 >= t.hi || r0 + 32 <= t.lo || gone) continue;
        // the chunk's values, worked on in the accumulator's registers
        uint32_t(&v)[32] = acc[j];
        const bool some = t.n > 0 && r0 < t.live;
#pragma unroll
        for (int i = 0; i < 32; ++i) v[i] = some ? __float_as_uint(fmaf(__uint_as_float(v[i]), alpha, bias)) : 0u;
        const bool whole = r0 >= t.lo && r0 + 32 <= t.live;
        auto mask = [&] {  // rows of other experts, and rows of none
          if (!whole) {
#pragma unroll
            for (int i = 0; i < 32; ++i)
              if (r0 + i < t.lo || r0 + i >= t.live) v[i] = 0u;
          }
        };
        auto put_bf16 = [&](uint8_t* buf) {
#pragma unroll
          for (int i = 0; i < 32; i += 2) {
            const __nv_bfloat162 p = __floats2bfloat162_rn(__uint_as_float(v[i]), __uint_as_float(v[i + 1]));
            const uint32_t b = *reinterpret_cast<const uint32_t*>(&p);
            *reinterpret_cast<uint16_t*>(buf + i * 64 + lane * 2) = static_cast<uint16_t>(b);
            *reinterpret_cast<uint16_t*>(buf + i * 64 + 64 + lane * 2) = static_cast<uint16_t>(b >> 16);
          }
        };
        if constexpr (KIND != kLinGrad && KIND != kLinPlain) {
          if (args.pre != nullptr) {
            mask();
            if (lane == 0) bulk_wait_group_read<0>();
            __syncwarp();
            put_bf16(pre_buf);
            store(pre_buf, &mapPre, args.pre, 2, t.row0, r0, f0, t);
          }
          by_activation(args.act, [&](auto a) {
#pragma unroll
            for (int i = 0; i < 32; ++i) v[i] = __float_as_uint(act_value<decltype(a)::value>(__uint_as_float(v[i])));
          });
        }
        uint8_t* buf = bufs;
        if constexpr (E::kAux) {
          buf = bufs + (j & 1) * E::kChunkBytes;
          if (args.aux && some) {
            if (!mbar_wait_bounded(&my_bar[j & 1], (aux_phase >> (j & 1)) & 1u, abort_flag, args.status, args.wait_ns))
              gone = true;
            gone = __any_sync(0xffffffffu, gone);
            if (gone) continue;
            aux_phase ^= 1u << (j & 1);
            pending &= ~(1u << (j & 1));
            auto aux_at = [&](int i) {
              if constexpr (E::kF32) return *reinterpret_cast<const float*>(buf + i * 128 + lane * 4);
              else return __uint_as_float(static_cast<uint32_t>(*reinterpret_cast<const uint16_t*>(buf + i * 64 + lane * 2)) << 16);
            };
            if constexpr (KIND == kLinGrad) {
              by_activation(args.act, [&](auto a) {
#pragma unroll
                for (int i = 0; i < 32; ++i)
                  v[i] = __float_as_uint(__uint_as_float(v[i]) * act_slope<decltype(a)::value>(aux_at(i)));
              });
            } else {
#pragma unroll
              for (int i = 0; i < 32; ++i) v[i] = __float_as_uint(__uint_as_float(v[i]) + aux_at(i));
            }
          }
        }
        mask();
        if constexpr (KIND == kLinGrad) {
#pragma unroll
          for (int i = 0; i < 32; ++i) colsum += __uint_as_float(v[i]);
        }
        // the chunk's values are computed while the store before it may still be reading the staging
        if (!E::kAux || !(args.aux && some)) {
          if (lane == 0) bulk_wait_group_read<0>();
        }
        __syncwarp();
        if constexpr (E::kF32) {
#pragma unroll
          for (int i = 0; i < 32; ++i) *reinterpret_cast<uint32_t*>(buf + i * 128 + lane * 4) = v[i];
        } else {
          put_bf16(buf);
        }
        store(buf, &mapOut, args.out, E::kF32 ? 4 : 2, t.row0, r0, f0, t);
        if constexpr (E::kAux) {
          if (args.aux && j + 2 < j_end && j >= j_first) {
            if (lane == 0) bulk_wait_group_read<0>();
            fence_proxy_async_smem();
            __syncwarp();
            aux_load(j + 2);
          }
        }
      }
      if (gone) break;
      if constexpr (KIND == kLinGrad) {
        if (args.sums != nullptr && f < args.cols)
          args.sums[(static_cast<int64_t>(t.window) * (kRowTile / E::kWarpCols) + (w >> 2)) * args.cols + f] = colsum;
      }
    }
    if constexpr (E::kAux) {  // loads on the way when a wait gave up must land before the CTA leaves
      for (int b = 0; b < 2; ++b)
        if (pending & (1u << b)) mbar_wait_bounded(&my_bar[b], (aux_phase >> b) & 1u, nullptr, args.status, args.wait_ns);
    }
    if (lane == 0) bulk_wait_group0();
  }

  tc_fence_before();
  __syncthreads();
  cluster_sync_all();  // neither CTA leaves while its peer may still touch its barriers or TMEM
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc_pair(tmem_base, kTmemAll);
  }
}

// ---------------------------------------------------------------------------- host side
inline bool lin_map(CUtensorMap* map, CUtensorMapDataType dt, int rank, const void* base, const cuuint64_t* dims,
                    const cuuint64_t* strides, const cuuint32_t* box, CUtensorMapSwizzle sw) {
  const EncodeTiledFn fn = encode_fn();
  const cuuint32_t estr[5] = {1, 1, 1, 1, 1};
  return fn != nullptr && fn(map, dt, rank, const_cast<void*>(base), dims, strides, box, estr,
                             CU_TENSOR_MAP_INTERLEAVE_NONE, sw, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

inline cudaLaunchConfig_t lin_config(cudaLaunchAttribute* attr, int clusters, int threads, int smem, cudaStream_t stream) {
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(2 * clusters);
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cfg;
}

template <int FMT, int KIND>
int run_linear(const LinearCall& c, cudaStream_t stream, const DeviceInfo& dev) {
  using E = LinEpi<KIND>;
  using P = LinFmt<FMT>;
  constexpr int kSmem = LinSmem<FMT, KIND>::total;
  static PerDevice<int> setup;  // per device: the shared-memory opt-in, and the clusters that fit (0 = unusable)
  const int max_clusters = setup.run(dev.device, [] {
    int n = 0;
    cudaLaunchAttribute at[2];
    cudaLaunchConfig_t cfg = lin_config(at, 1, E::kThreads, kSmem, nullptr);
    if (cudaFuncSetAttribute(linear_kernel<FMT, KIND>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem) != cudaSuccess ||
        cudaOccupancyMaxActiveClusters(&n, linear_kernel<FMT, KIND>, &cfg) != cudaSuccess) {
      cudaGetLastError();
      return 0;
    }
    return n;
  });
  if (max_clusters < 1) return BSQ_ERR_LAUNCH;

  using u64 = cuuint64_t;
  const u64 experts = static_cast<u64>(std::max<int64_t>(c.experts, 1));
  const u64 weights = c.contract ? 1 : experts;  // matrices in the columns' operand
  const u64 rows = static_cast<u64>(c.rows), cols = static_cast<u64>(c.cols);
  const u64 kb = FMT == BSQ_MXFP8 ? static_cast<u64>(c.depth) : static_cast<u64>(c.depth) / 2;
  // scale atoms along the depth: of one expert's weights, of a row of the weights' operand, of the rows' operand
  const u64 atoms = static_cast<u64>(ceil_div(c.depth / block_size(FMT), 4));
  const u64 pitch = c.stack_cols ? kb * weights : kb, atom_pitch = c.stack_cols ? atoms * weights : atoms;
  const u64 row_tiles = static_cast<u64>(ceil_div(c.rows, 128)), col_tiles = static_cast<u64>(ceil_div(c.cols, 128));
  const CUtensorMapDataType u8 = CU_TENSOR_MAP_DATA_TYPE_UINT8, u32 = CU_TENSOR_MAP_DATA_TYPE_UINT32;
  const CUtensorMapSwizzle s128 = CU_TENSOR_MAP_SWIZZLE_128B, s0 = CU_TENSOR_MAP_SWIZZLE_NONE;
  CUtensorMap mW, mX, mXs, mSfw, mSfx, mOut, mPre, mAux;
  bool ok = true;
  {
    const u64 dims[3] = {kb, cols, weights}, st[2] = {pitch, c.stack_cols ? kb : kb * cols};
    const cuuint32_t box[3] = {kSpanBytes, 128, 1};
    ok = ok && lin_map(&mW, u8, 3, c.b, dims, st, box, s128);
  }
  {
    const u64 dims[2] = {kb, rows}, st[1] = {kb};
    const cuuint32_t box[2] = {kSpanBytes, 128}, small[2] = {kSpanBytes, 32};
    ok = ok && lin_map(&mX, u8, 2, c.a, dims, st, box, s128) && lin_map(&mXs, u8, 2, c.a, dims, st, small, s128);
  }
  {
    const u64 dims[4] = {128, atoms, col_tiles, weights};
    const u64 st[3] = {512, atom_pitch * 512, (c.stack_cols ? atoms : atoms * col_tiles) * 512};
    const cuuint32_t box[4] = {128, P::kAtoms, 1, 1};
    ok = ok && lin_map(&mSfw, u32, 4, c.b_scales, dims, st, box, s0);
  }
  {
    const u64 dims[3] = {128, atoms, row_tiles}, st[2] = {512, atoms * 512};
    const cuuint32_t box[3] = {128, P::kAtoms, 1};
    ok = ok && lin_map(&mSfx, u32, 3, c.a_scales, dims, st, box, s0);
  }
  const u64 es = E::kF32 ? 4 : 2;
  const CUtensorMapDataType bf16 = CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
  const CUtensorMapDataType ot = E::kF32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : bf16;
  const cuuint32_t chunk[2] = {32, 32};
  {
    const u64 dims[2] = {cols, rows * (c.contract ? experts : 1)}, st[1] = {cols * es}, st16[1] = {cols * 2};
    ok = ok && lin_map(&mOut, ot, 2, c.out, dims, st, chunk, s0);
    mPre = mAux = mOut;
    if (c.pre != nullptr) ok = ok && lin_map(&mPre, bf16, 2, c.pre, dims, st16, chunk, s0);
  }
  if (E::kAux && c.aux != nullptr) {
    const u64 dims[2] = {cols, rows}, st[1] = {static_cast<u64>(c.aux_stride) * es};
    ok = ok && lin_map(&mAux, ot, 2, c.aux, dims, st, chunk, s0);
  }
  if (!ok) return BSQ_ERR_LAUNCH;

  LinArgs a{};
  a.counts = c.counts;
  a.offsets = c.offsets;
  a.bias = static_cast<const uint16_t*>(c.bias);
  const int64_t stacked = c.depth * static_cast<int64_t>(c.stack_cols ? weights : 1);
  a.ga = reinterpret_cast<const float*>(static_cast<const uint8_t*>(c.a_scales) + scales_body_bytes(FMT, c.rows, c.depth));
  a.gb = reinterpret_cast<const float*>(
      static_cast<const uint8_t*>(c.b_scales) +
      scales_body_bytes(FMT, c.cols * static_cast<int64_t>(c.stack_cols ? 1 : weights), stacked));
  a.out = static_cast<uint8_t*>(c.out);
  a.pre = static_cast<uint8_t*>(c.pre);
  a.sums = c.sums;
  a.status = dev.status;
  a.rows = static_cast<int>(c.rows);
  a.cols = static_cast<int>(c.cols);
  a.depth = static_cast<int>(c.depth);
  a.experts = static_cast<int>(c.experts);
  a.tiles_c = static_cast<int>(ceil_div(c.cols, kFeatTile));
  a.mmas = static_cast<int>(c.depth / P::kMmaDepth);
  a.act = c.activation;
  a.contract = c.contract ? 1 : 0;
  a.aux = E::kAux && c.aux != nullptr ? 1 : 0;
  const StallInjection inj = take_stall(BSQ_KERNEL_LINEAR);
  a.stall_after = inj.after;
  a.wait_ns = inj.limit_ns;
  const int64_t windows = ceil_div(c.rows, kRowTile) * (c.contract ? c.experts : 1) +
                          (c.counts != nullptr && !c.contract ? 2 * (c.experts + 1) : 0);
  const int clusters = static_cast<int>(std::min<int64_t>(windows * a.tiles_c, std::min(max_clusters, dev.num_sms / 2)));
  cudaLaunchAttribute at[2];
  cudaLaunchConfig_t cfg = lin_config(at, clusters, E::kThreads, kSmem, stream);
  if (cudaLaunchKernelEx(&cfg, linear_kernel<FMT, KIND>, mW, mX, mXs, mSfw, mSfx, mOut, mPre, mAux, a) != cudaSuccess)
    return BSQ_ERR_LAUNCH;
  return cudaGetLastError() == cudaSuccess ? BSQ_OK : BSQ_ERR_LAUNCH;
}

}  // namespace

template <int FMT>
int launch_linear(const LinearCall& c, cudaStream_t stream, const DeviceInfo& dev) {
  switch (c.kind) {
    case kLinPlain: return run_linear<FMT, kLinPlain>(c, stream, dev);
    case kLinAct: return run_linear<FMT, kLinAct>(c, stream, dev);
    case kLinRes: return run_linear<FMT, kLinRes>(c, stream, dev);
    case kLinGrad: return run_linear<FMT, kLinGrad>(c, stream, dev);
    case kLinF32: return run_linear<FMT, kLinF32>(c, stream, dev);
    case kLinResF32: return run_linear<FMT, kLinResF32>(c, stream, dev);
    default: return BSQ_ERR_ARG;
  }
}

}  // namespace bsq
