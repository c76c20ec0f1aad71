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
// copies and MMAs; beside them a second loader, a warp that finds the units of work ahead of the others (a search over
// the segments: 1300 cycles, a quarter of a unit's time, in each role's own path before), and the epilogue's warps.
// Every wait is bounded.
//
// What the steps brought (device time, us): experts' forward 131048 x 2048 to 1024 NVFP4, gradient through GELU
// 14336 x 1024 to 4096 MXFP8:                                        162   170
//   8 x 8 fragments and matrix stores                                155   106
//   16 warps for activations                                          -     88
//   units found ahead, two loaders                                   134    87
//   no select for each value, less arithmetic                        130    85
//   chunks of 64 rows with 16 warps                                   -     80
//   the same, all waits of a warp by a vote                          131     80
// Bounds (the same two): MMAs and scale copies alone take 99 and 45 us, without the stores 118 and 72, without the kept
// arguments as well 52; without the activation's arithmetic the second stays at 80. So it is the small rows that pass
// through the tensor copies' unit and shared memory beside the operands, 64 bytes of a row in a warp's chunk.
// Tried and left out: two pairs that share the rows' operand by multicast (134 against 131 us: 72 pairs fit, not 76),
// scale copies a stage ahead of their MMAs (138), plain stores from the staging (135, and 112 against 82 us with a kept
// argument), two staging chunks (139), chunks of 64 rows with 8 warps (143), all steps of a chunk in one pass over its
// registers (the gradient 108 us: more moves and spills).
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
constexpr int kEpiWarp0 = 4;  // the first warpgroup loads and issues, the others drain
constexpr uint32_t kTmemAll = 512;
constexpr int kUnitSlots = 4;  // units of work found ahead
constexpr int kMaxSplits = 4;  // pairs that share the depth of one unit

template <int KIND>
struct LinEpi {
  static constexpr bool kAux = KIND == kLinRes || KIND == kLinGrad || KIND == kLinResF32;
  static constexpr bool kF32 = KIND == kLinF32 || KIND == kLinResF32;
  // At launch all threads have kLaunchRegs; the first warpgroup gives up what the others then take (the sum stays
  // the same).
  static constexpr int kWarps = KIND == kLinAct || KIND == kLinGrad ? 16 : 8;
  static constexpr int kLaunchRegs = kWarps == 16 ? 96 : 168;
  static constexpr int kRoleRegs = 56, kEpiRegs = kWarps == 16 ? 104 : 224;
  static constexpr int kWarpCols = 4 * kRowTile / kWarps;  // rows of the window that a warp drains
  // A chunk is 32 rows x 32 features, or with 16 warps all 64 rows of a warp: half the waits, fences and stores.
  static constexpr int kSub = kWarps == 16 ? 2 : 1;
  static constexpr int kRows = 32 * kSub;
  static constexpr int kChunks = kWarpCols / kRows;
  static constexpr int kChunkBytes = kRows * 32 * (kF32 ? 4 : 2);
  // One staging chunk, or two that bring the auxiliary values and take the results in their places.
  static constexpr int kBufs = kAux && kChunks > 1 ? 2 : 1;
  static constexpr int kBytes = kBufs * kChunkBytes;
  static constexpr int kThreads = (kEpiWarp0 + kWarps) * 32;
  static_assert(kSub == 1 || !(kF32 || KIND == kLinRes), "chunks of 64 rows: bf16, no residual");
  static_assert(kEpiWarp0 * kRoleRegs + kWarps * kEpiRegs <= (kEpiWarp0 + kWarps) * kLaunchRegs, "register split");
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
  static constexpr int kFixed = LinEpi<KIND>::kWarps * LinEpi<KIND>::kBytes + (BSQ_MAX_EXPERTS + 4) * 4 + 1024;
  static constexpr int kRoom = (232448 - kFixed) / kStageBytes;
  static constexpr int kTmemRoom = (512 - kRowTile) / LinFmt<FMT>::kSfCols;
  static constexpr int S = kRoom < kTmemRoom ? (kRoom < 6 ? kRoom : 6) : (kTmemRoom < 6 ? kTmemRoom : 6);
  static constexpr int a_off = 0;
  static constexpr int b_off = a_off + S * kABytes;
  static constexpr int sfa_off = b_off + S * kBBytes;
  static constexpr int sfb_off = sfa_off + S * kSfaBytes;
  static constexpr int epi_off = sfb_off + S * kSfbBytes;
  static constexpr int bar_off = epi_off + LinEpi<KIND>::kWarps * LinEpi<KIND>::kBytes;
  static constexpr int kNumBars = 2 * S + 3 + 2 * kUnitSlots + 8;
  static constexpr int misc_off = (bar_off + kNumBars * 8 + 15) / 16 * 16;
  static constexpr int unit_off = misc_off + 16;
  static constexpr int prefix_off = unit_off + kUnitSlots * 48;
  static constexpr int total = prefix_off + (BSQ_MAX_EXPERTS + 4) * 4;
  static_assert(S >= 3 && total <= 232448, "shared memory budget");
  static_assert((kMaxSplits - 1) * 4 * 4096 <= S * kABytes, "the pairs' sums fit where the features' operand stood");
  static_assert(epi_off % 512 == 0, "staging chunks repeat the 64-byte swizzle's pattern");
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
__device__ __forceinline__ uint64_t rcp_pair(uint64_t x) {
  float a, b;
  f2_split(x, a, b);
  return f2(rcp_fast(a), rcp_fast(b));
}
// NaN stays NaN
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float min_nan(float a, float b) {
  float r;
  asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
// The tail Q(w) = 1 - Phi(w) of the normal distribution for two w = |v| as w's density times a polynomial: Abramowitz &
// Stegun, Handbook of Mathematical Functions, formula 7.1.26 for erfc(w / sqrt 2), |error| <= 1.5e-7 (of 2 Q). Returns
// poly and gauss = exp(-w^2 / 2), Q = -poly * gauss. Then, without cancellation and with few instructions,
//   v Phi(v) = max(v, 0) - w Q(w),   Phi(v) + v phi(v) = 1/2 + sign(v) (1/2 + w phi(w) - Q(w)).
__device__ __forceinline__ uint64_t normal_tail2(uint64_t w, uint64_t& gauss) {
  const uint64_t t = rcp_pair(f2_fma(w, f2_splat(0.3275911f * 0.7071067811865476f), f2_splat(1.0f)));
  uint64_t p = f2_fma(f2_splat(-0.5f * 1.061405429f), t, f2_splat(0.5f * 1.453152027f));
  p = f2_fma(p, t, f2_splat(-0.5f * 1.421413741f));
  p = f2_fma(p, t, f2_splat(0.5f * 0.284496736f));
  p = f2_fma(p, t, f2_splat(-0.5f * 0.254829592f));
  float a, b;
  f2_split(f2_mul(f2_mul(w, f2_splat(-0.5f * 1.4426950408889634f)), w), a, b);
  gauss = f2(ex2_fast(a), ex2_fast(b));
  return f2_mul(p, t);
}
// |v|, held below 1e18, where both tails are long zero: an infinite v gives no 0 * inf
__device__ __forceinline__ float size_of(float v) { return min_nan(fabsf(v), 1e18f); }
// 1 / (1 + exp(-v)) of two values
__device__ __forceinline__ uint64_t logistic2(uint64_t v) {
  float a, b;
  f2_split(f2_mul(v, f2_splat(-1.4426950408889634f)), a, b);
  return rcp_pair(f2_add(f2(ex2_fast(a), ex2_fast(b)), f2_splat(1.0f)));
}
constexpr float kTanhA = 1.5957691216057308f;  // 2 sqrt(2 / pi): (1 + tanh u) / 2 = logistic(2 u)
constexpr float kTanhB = 1.5957691216057308f * 0.044715f;

// act of a pair of values
template <int ACT>
__device__ __forceinline__ void act_pair(float& a, float& b) {
  const uint64_t v = f2(a, b);
  if constexpr (ACT == BSQ_ACT_GELU) {
    const uint64_t w = f2(size_of(a), size_of(b));
    uint64_t gauss;
    const uint64_t p = normal_tail2(w, gauss);
    f2_split(f2_fma(f2_mul(p, gauss), w, f2(max_nan(a, 0.0f), max_nan(b, 0.0f))), a, b);
  } else if constexpr (ACT == BSQ_ACT_GELU_TANH) {
    f2_split(f2_mul(v, logistic2(f2_mul(v, f2_fma(f2_splat(kTanhB), f2_mul(v, v), f2_splat(kTanhA))))), a, b);
  } else if constexpr (ACT == BSQ_ACT_SILU) {
    f2_split(f2_mul(v, logistic2(v)), a, b);
  } else if constexpr (ACT == BSQ_ACT_RELU) {
    a = max_nan(a, 0.0f);
    b = max_nan(b, 0.0f);
  }
}
// (a, b) times act' of (x, y)
template <int ACT>
__device__ __forceinline__ void slope_pair(float& a, float& b, float x, float y) {
  const uint64_t g = f2(a, b);
  if constexpr (ACT == BSQ_ACT_GELU) {
    const uint64_t w = f2(size_of(x), size_of(y));
    uint64_t gauss;
    const uint64_t p = normal_tail2(w, gauss);
    float s, t;  // 1/2 + (w phi - Q), which takes v's sign (-0 counts as negative: 1/2 either way)
    f2_split(f2_fma(f2_fma(w, f2_splat(0.3989422804014327f), p), gauss, f2_splat(0.5f)), s, t);
    s = __uint_as_float(__float_as_uint(s) ^ (__float_as_uint(x) & 0x80000000u));
    t = __uint_as_float(__float_as_uint(t) ^ (__float_as_uint(y) & 0x80000000u));
    f2_split(f2_mul(g, f2_add(f2(s, t), f2_splat(0.5f))), a, b);
  } else if constexpr (ACT == BSQ_ACT_GELU_TANH) {
    // past 12 the logistic is 0 or 1 to the last bit; x^2 stays finite
    const uint64_t v = f2(min_nan(max_nan(x, -12.0f), 12.0f), min_nan(max_nan(y, -12.0f), 12.0f)), v2 = f2_mul(v, v);
    const uint64_t s = logistic2(f2_mul(v, f2_fma(f2_splat(kTanhB), v2, f2_splat(kTanhA))));
    const uint64_t ds = f2_mul(s, f2_fma(s, f2_splat(-1.0f), f2_splat(1.0f)));
    const uint64_t r = f2_fma(f2_mul(v, ds), f2_fma(f2_splat(3.0f * kTanhB), v2, f2_splat(kTanhA)), s);
    f2_split(f2_mul(g, r), a, b);
  } else if constexpr (ACT == BSQ_ACT_SILU) {
    const uint64_t v = f2(x, y), s = logistic2(v);
    f2_split(f2_mul(g, f2_mul(s, f2_fma(v, f2_fma(s, f2_splat(-1.0f), f2_splat(1.0f)), f2_splat(1.0f)))), a, b);
  } else if constexpr (ACT == BSQ_ACT_RELU) {
    a *= x > 0.0f ? 1.0f : 0.0f;
    b *= y > 0.0f ? 1.0f : 0.0f;
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

// ---------------------------------------------------------------------------- fragments
// 16 lanes x 32 columns of TMEM as 8 x 8 blocks: register 4 q + 2 s + p of thread i holds lane 8 s + i / 4, column
// 8 q + 2 (i % 4) + p -- the layout of the matrix load and store below.
__device__ __forceinline__ void tmem_ld_16x256b_x4(uint32_t taddr, uint32_t* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x4.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr)
      : "memory");
}
// Four 8 x 8 blocks of 16-bit values, transposed on the way: thread 8 m + i gives the address of row i of block m.
__device__ __forceinline__ void stmatrix_trans(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(a), "r"(b),
               "r"(c), "r"(d)
               : "memory");
}
__device__ __forceinline__ void ldmatrix_trans(uint32_t addr, uint32_t& a, uint32_t& b, uint32_t& c, uint32_t& d) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(a), "=r"(b), "=r"(c), "=r"(d)
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ float bf16_lo(uint32_t x) { return __uint_as_float(x << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t x) { return __uint_as_float(x & 0xFFFF0000u); }
__device__ __forceinline__ uint32_t bf16_pair(uint32_t lo, uint32_t hi) {
  const __nv_bfloat162 p = __floats2bfloat162_rn(__uint_as_float(lo), __uint_as_float(hi));
  return *reinterpret_cast<const uint32_t*>(&p);
}

// A word into another CTA's shared memory, whose bytes complete on a barrier there.
__device__ __forceinline__ void store_remote(uint32_t addr, uint32_t v, uint32_t bar) {
  asm volatile("st.async.weak.shared::cluster.mbarrier::complete_tx::bytes.b32 [%0], %1, [%2];" ::"r"(addr), "r"(v), "r"(bar)
               : "memory");
}

// 16 bytes into shared memory, zeros where `bytes` is 0.
__device__ __forceinline__ void copy_16(uint32_t to, const void* from, int bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to), "l"(from), "r"(bytes) : "memory");
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
  int max_windows;  // more than segments that do not overlap can have; sums hold as many
  const uint8_t* aux;   // residual or kept arguments, row stride in elements; NULL: none
  int64_t aux_stride;
  int64_t bias_len, aux_len, out_len, sums_len;  // elements (index checks)
  int split_bits;  // log2 of a cluster's pairs: they share the depth of one unit (above 0: a window of up to 32 rows)
  int contract;
};

// A window of rows times 256 features. Rows [lo, live) are computed, [live, hi) are zeros.
struct Unit {
  int w0, lo, live, hi;
  int n;        // MMA columns; 0: no product, zeros alone
  int ct, e;    // tile of features, expert
  int window;
  int mmas, kx, ka;  // MMAs along the depth, first byte and first scale atom
};
static_assert(sizeof(Unit) <= 48, "a unit's slot");

__device__ __forceinline__ int offset_at(const LinArgs& a, int e) {
  return in_bounds(e >= 0 && e <= a.experts, a.status) ? a.offsets[e] : 0;
}
__device__ __forceinline__ int count_at(const LinArgs& a, int e) {
  return in_bounds(e >= 0 && e < a.experts, a.status) ? a.counts[e] : 0;
}
// Expert e's segment, whatever the two arrays hold: inside [0, limit), counts inside the segment. Behind the last
// expert (e = experts) the rows of none, and then (e = experts + 1) those ahead of all segments, [0, lead).
__device__ __forceinline__ void segment(const LinArgs& a, int e, int limit, int lead, int& off, int& count, int& end) {
  count = 0;
  if (e > a.experts) {
    off = 0;
    end = lead;
    return;
  }
  off = min(max(offset_at(a, e), 0), limit);
  end = limit;
  if (e < a.experts) {
    end = min(max(offset_at(a, e + 1), off), limit);
    count = min(max(count_at(a, e), 0), end - off);
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
  if (a.contract) {
    const int windows = (a.rows + kRowTile - 1) / kRowTile;
    t.e = t.window / windows;
    t.w0 = t.lo = (t.window - t.e * windows) * kRowTile;
    t.hi = min(t.w0 + kRowTile, a.rows);
    int off, count, end;
    segment(a, t.e, a.depth, 0, off, count, end);
    constexpr int kStep = LinFmt<FMT>::kMmaDepth;
    t.mmas = (count + kStep - 1) / kStep;
    // The scales of the depth lie in groups of 128, and the last MMA takes in whole steps of it: rows behind the segment's
    // end too, which are not this expert's (behind the operands' end it reads zeros). No product then, and the caller learns
    // of it.
    if ((off & 127) || (off + t.mmas * kStep > end && end < a.depth)) {
      if (count > 0) atomicCAS(a.status, 0, BSQ_ERR_SHAPE);
      count = t.mmas = 0;
    }
    t.live = count > 0 ? t.hi : t.lo;
    t.kx = FMT == BSQ_MXFP8 ? off : off / 2;
    t.ka = off / LinFmt<FMT>::kAtomDepth;
  } else {
    int off = 0, count = a.rows, end = a.rows, first = 0;
    if (a.counts != nullptr) {
      int below = a.experts + 2;  // the last segment that does not begin behind this window
      while (below - t.e > 1) {
        const int mid = (t.e + below) >> 1;
        if (prefix[mid] <= t.window) t.e = mid;
        else below = mid;
      }
      first = prefix[t.e];
      segment(a, t.e, a.rows, prefix[a.experts + 3], off, count, end);
    }
    t.w0 = (off & ~127) + (t.window - first) * kRowTile;
    t.lo = max(t.w0, off);
    t.hi = min(t.w0 + kRowTile, end);
    t.live = min(t.hi, max(off + count, t.lo));
  }
  t.n = t.live > t.lo ? (t.live - t.w0 + 31) & ~31 : 0;
  return t;
}

// Whether the phase has completed, without waiting.
__device__ __forceinline__ bool mbar_test(uint32_t bar_addr, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(bar_addr), "r"(parity)
      : "memory");
  return ok != 0;
}

// A warp's bounded wait, on whose outcome all its threads agree. A phase that has completed takes one test and one vote
// (experts' forward 131048 x 2048 to 1024 NVFP4 132.6 -> 131.0 us; the wide norms' backward pass, which polls for its
// peers, would lose 3 %).
__device__ __forceinline__ bool wait_warp(uint64_t* bar, uint32_t parity, volatile int* abort, int* status, uint64_t limit_ns) {
  return __all_sync(0xffffffffu, mbar_try_wait(smem_u32(bar), parity)) != 0 ||
         mbar_wait_bounded_warp(bar, parity, abort, status, limit_ns);
}

__device__ __forceinline__ void next_slot(int& slot, uint32_t& phase) {
  if (++slot == kUnitSlots) {
    slot = 0;
    phase ^= 1u;
  }
}

// ---------------------------------------------------------------------------- the kernel
template <int FMT, int KIND>
__global__ void __launch_bounds__(LinEpi<KIND>::kThreads, 1)
    linear_kernel(const __grid_constant__ CUtensorMap mapW, const __grid_constant__ CUtensorMap mapX,
                  const __grid_constant__ CUtensorMap mapXs, const __grid_constant__ CUtensorMap mapSfw,
                  const __grid_constant__ CUtensorMap mapSfx, const __grid_constant__ CUtensorMap mapOut,
                  const __grid_constant__ CUtensorMap mapPre, const LinArgs args) {
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
  uint64_t* unit_full = full_bar + 2 * S + 3;   // a unit stands in its slot
  uint64_t* unit_empty = unit_full + kUnitSlots;
  uint64_t* ready_bar = unit_empty + kUnitSlots;  // [warp] the first pair takes this pair's sums
  uint64_t* sums_bar = ready_bar + 4;             // [warp] first pair: the others' sums have come
  Unit* units = reinterpret_cast<Unit*>(smem + L::unit_off);
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(smem + L::misc_off);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + L::misc_off + 4);
  int* prefix = reinterpret_cast<int*>(smem + L::prefix_off);

  const uint32_t warp = threadIdx.x >> 5;
  const uint32_t lane = threadIdx.x & 31u;
  const uint32_t rank = cluster_rank();
  const int half = static_cast<int>(rank & 1u);  // which half of the features and of the rows' operand this CTA holds
  const int pair = static_cast<int>(rank >> 1), splits = 1 << args.split_bits;
  const bool leader = half == 0;

  if (threadIdx.x == 0) {
    for (int s = 0; s < S; ++s) {
      mbar_init(&full_bar[s], 1);
      mbar_init(&empty_bar[s], 1);
    }
    mbar_init(tmem_full, 1);
    mbar_init(tmem_empty, 2 * E::kWarps);
    mbar_init(drain_bar, 1);
    for (int i = 0; i < kUnitSlots; ++i) {
      mbar_init(&unit_full[i], 1);
      mbar_init(&unit_empty[i], 2 + (leader ? 1 : 0) + E::kWarps);  // two loaders, the issuer, the epilogue
    }
    for (int i = 0; i < 8; ++i) mbar_init(&ready_bar[i], 1);
    *abort_flag = 0;
    fence_mbar_init();
    prefetch_tmap(&mapW);
    prefetch_tmap(&mapX);
    prefetch_tmap(&mapXs);
    prefetch_tmap(&mapSfw);
    prefetch_tmap(&mapSfx);
    prefetch_tmap(&mapOut);
  }
  if (warp == 1) {
    tmem_alloc_pair(tmem_holder, kTmemAll);
    tmem_relinquish_pair();
  }
  launch_dependents();
  grid_dependency_wait();  // inputs and outputs may belong to the previous kernel until here
  // windows ahead of each segment's first; behind them the rows ahead of all segments (none: offsets begin at 0)
  int num_units;
  if (args.counts != nullptr && !args.contract) {
    int* const lead = prefix + args.experts + 3;
    for (int e = threadIdx.x; e <= args.experts; e += E::kThreads) {
      int off, count, end;
      segment(args, e, args.rows, 0, off, count, end);
      prefix[e + 1] = min(windows_of(off, end), args.max_windows);
      if (e == 0) *lead = off;
    }
    __syncthreads();
    if (*lead > 0) {  // offsets that fall may have a later segment begin ahead of the first
      __syncthreads();
      for (int e = threadIdx.x; e <= args.experts; e += E::kThreads) atomicMin(lead, max(offset_at(args, e), 0));
      __syncthreads();
    }
    if (warp == 0) {
      int carry = 0;
      if (lane == 0) {
        prefix[0] = 0;
        prefix[args.experts + 2] = windows_of(0, *lead);
      }
      __syncwarp();
      for (int base = 0; base <= args.experts + 1; base += 32) {
        const int i = base + static_cast<int>(lane);
        int v = i <= args.experts + 1 ? prefix[i + 1] : 0;
#pragma unroll
        for (int d = 1; d < 32; d *= 2) {
          const int o = __shfl_up_sync(0xffffffffu, v, d);
          if (static_cast<int>(lane) >= d) v = min(v + o, args.max_windows);
        }
        v = min(v + carry, args.max_windows);  // segments that overlap could have more: those are dropped
        if (i <= args.experts + 1) prefix[i + 1] = v;
        carry = __shfl_sync(0xffffffffu, v, 31);
      }
    }
    tc_fence_before();
    __syncthreads();
    num_units = prefix[args.experts + 2] * args.tiles_c;
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

  if (warp < static_cast<uint32_t>(kEpiWarp0)) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(E::kRoleRegs));
    if ((warp == 0 || warp == 2) && lane == 0) {
      // ------------------------------------------------------------------ TMA producers
      // Two warps, one for the features' operand and its scales and one for the rows': an issued copy costs its thread
      // about 130 cycles and a stage of the FP4 formats lasts 400 to 500.
      const bool w_side = warp == 0;
      const uint64_t keep = l2_policy_evict_last();
      int stage = 0, slot = 0;
      uint32_t phase = 0, unit_phase = 0;
      bool ok = true;
      int64_t armed = 0;
      auto produce = [&](auto stall) {
        for (int u = first_unit; u < num_units && ok; u += stride) {
          if (!mbar_wait_bounded(&unit_full[slot], unit_phase, abort_flag, args.status, args.wait_ns)) break;
          const Unit t = units[slot];
          mbar_arrive(&unit_empty[slot]);
          next_slot(slot, unit_phase);
          if (t.n == 0) continue;
          // this CTA's half of the rows in boxes of 32, or in one where it is full; all rows' scale tiles
          const int boxes = (t.n + 63) / 64, tiles = t.n > 128 ? 2 : 1;
          const uint32_t bytes = L::kABytes + L::kSfaBytes + boxes * 32 * kSpanBytes + tiles * L::kSfaBytes;
          const int x_row = t.w0 + half * (t.n / 2);
          const int w_row = t.ct * kFeatTile + half * 128;
          const int expert = args.contract ? 0 : t.e;
          const int all_spans = (t.mmas + 3) / 4, spans = all_spans * (pair + 1) >> args.split_bits;
          for (int s = all_spans * pair >> args.split_bits; s < spans; ++s) {
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
            const uint32_t bar = smem_u32(&full_bar[stage]) & ~kClusterRankBit;  // the leader's full[stage]
            const int kx = t.kx + s * kSpanBytes, ka = t.ka + s * P::kAtoms;
            if (w_side) {
              if (leader) mbar_arrive_expect_tx(&full_bar[stage], 2 * bytes);  // both warps' copies
              tma_load_3d_to_leader(smem + L::a_off + stage * L::kABytes, &mapW, bar, kx, w_row, expert, keep);
              tma_load_4d_to_leader(smem + L::sfa_off + stage * L::kSfaBytes, &mapSfw, bar, 0, ka, 2 * t.ct + half, expert,
                                    keep);
            } else {
              uint8_t* const xs = smem + L::b_off + stage * L::kBBytes;
              if (boxes == 4) {
                tma_load_2d_to_leader(xs, &mapX, bar, kx, x_row, keep);
              } else {
                for (int i = 0; i < boxes; ++i)
                  tma_load_2d_to_leader(xs + i * 32 * kSpanBytes, &mapXs, bar, kx, x_row + 32 * i, keep);
              }
              for (int i = 0; i < tiles; ++i)
                tma_load_3d_to_leader(smem + L::sfb_off + stage * L::kSfbBytes + i * L::kSfaBytes, &mapSfx, bar, 0, ka,
                                      (t.w0 >> 7) + i, keep);
            }
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
      if (leader && w_side) wait_armed_stages(full_bar, S, armed, args.status, args.wait_ns);
    } else if (warp == 3) {
      // ------------------------------------------------------------------ units of work, ahead of the other roles
      int slot = 0;
      uint32_t unit_phase = 0;
      for (int u = first_unit; u < num_units; u += stride) {
        const Unit t = unit_at<FMT>(args, prefix, u);
        if (!wait_warp(&unit_empty[slot], unit_phase ^ 1u, abort_flag, args.status, args.wait_ns)) break;
        if (lane == 0) {
          units[slot] = t;
          mbar_arrive(&unit_full[slot]);
        }
        __syncwarp();
        next_slot(slot, unit_phase);
      }
    } else if (warp == 1 && leader) {
      // ------------------------------------------------------------------ MMA issuer
      const bool issuer = elect_one_sync();
      const uint16_t pair_mask = static_cast<uint16_t>(3u << (2 * pair));
      int stage = 0, slot = 0;
      uint32_t phase = 0, acc_phase = 0, unit_phase = 0;
      bool ok = true;
      const uint32_t a_s0 = smem_u32(smem + L::a_off), b_s0 = smem_u32(smem + L::b_off);
      const uint32_t sfa_s0 = smem_u32(smem + L::sfa_off), sfb_s0 = smem_u32(smem + L::sfb_off);
      const uint32_t sf_t0 = tmem_base + kRowTile;
      for (int u = first_unit; u < num_units && ok; u += stride) {
        if (!wait_warp(&unit_full[slot], unit_phase, abort_flag, args.status, args.wait_ns)) break;
        const Unit t = units[slot];
        __syncwarp();
        if (lane == 0) mbar_arrive(&unit_empty[slot]);
        next_slot(slot, unit_phase);
        if (t.n == 0) continue;
        if (!wait_warp(tmem_empty, acc_phase ^ 1u, abort_flag, args.status, args.wait_ns)) break;
        acc_phase ^= 1u;
        tc_fence_after();
        const int all_spans = (t.mmas + 3) / 4, first = all_spans * pair >> args.split_bits;
        const int spans = all_spans * (pair + 1) >> args.split_bits;
        // whether the next stage has landed is asked before this one's instructions: the answer takes a while
        bool landed = mbar_test(smem_u32(&full_bar[stage]), phase);
        for (int s = first; s < spans; ++s) {
          if (!__all_sync(0xffffffffu, landed) &&
              !wait_warp(&full_bar[stage], phase, abort_flag, args.status, args.wait_ns)) {
            ok = false;
            break;
          }
          const int next = stage + 1 == S ? 0 : stage + 1;
          landed = s + 1 < spans && mbar_test(smem_u32(&full_bar[next]), phase ^ (next == 0 ? 1u : 0u));
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
                               (k > 0 || s > first) ? 1u : 0u);
            }
            tc_commit_pair_mc(&empty_bar[stage], pair_mask);
          }
          __syncwarp();
          if (++stage == S) {
            stage = 0;
            phase ^= 1u;
          }
        }
        if (ok && issuer) tc_commit_pair_mc(tmem_full, pair_mask);
        __syncwarp();
      }
      if (issuer) tc_commit_pair(drain_bar);  // all tensor-core work ends before TMEM is released
      __syncwarp();
      mbar_wait_bounded(drain_bar, 0, nullptr, args.status, args.wait_ns);
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(E::kEpiRegs));
    // ------------------------------------------------------------------ epilogue (both CTAs)
    const uint32_t w = warp - kEpiWarp0;
    const uint32_t quad = warp & 3u;  // TMEM lanes this warp may read: 32 features
    const int c_base = static_cast<int>(w >> 2) * E::kWarpCols;
    uint8_t* const bufs = smem + L::epi_off + w * E::kBytes;
    const uint32_t tmem_empty_leader = mapa_shared(smem_u32(tmem_empty), rank & ~1u);
    float alpha = 1.0f;
    if constexpr (FMT == BSQ_NVFP4) alpha = __fmul_rn(*args.ga, *args.gb);
    int slot = 0;
    uint32_t unit_phase = 0, acc_phase = 0;

    // A chunk is 32 rows x 32 features in 32 registers. fp32 results: a thread is a feature, a register a row.
    // bf16 results: 8 x 8 blocks (tmem_ld_16x256b_x4, features 0..15 then 16..31), which the matrix store
    // transposes into rows of 64 bytes whose 16-byte pieces the 64-byte swizzle spreads over the banks.
    // Against a feature a thread with 2-byte stores: gradient through GELU of 14336 x 4096 MXFP8 170 -> 106 us.
    auto row_of = [&](int i) {
      return E::kF32 ? i : 8 * ((i >> 2) & 3) + 2 * static_cast<int>(lane & 3u) + (i & 1);
    };
    // thread 8 m + i addresses row i (of 8 q + i) of block m in a swizzled chunk
    const uint32_t mat_row = lane & 7u, mat_off = mat_row * 64 + (((lane >> 3) ^ ((mat_row >> 1) & 3u)) << 4);

    // the rows of a staged chunk, r0 its first, to `dst`: one tensor store where all of them are this unit's
    auto store = [&](const uint8_t* buf, const CUtensorMap* map, uint8_t* dst, bool f32, int64_t row0, int r0, int f0,
                     const Unit& t) {
      if (r0 >= t.lo && r0 + E::kRows <= t.hi) {
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          tma_store_2d(map, buf, f0, static_cast<int32_t>(row0 + r0));
          bulk_commit_group();
        }
      } else {
        __syncwarp();
        const int per_row = f32 ? 8 : 4, rows_at_once = 32 / per_row;  // 16-byte pieces of a row
        const int c = static_cast<int>(lane) / per_row, piece = static_cast<int>(lane) % per_row;
        const int es = f32 ? 4 : 2, f = f0 + piece * (16 / es);
        const uint8_t* from = buf + c * 32 * es + ((E::kF32 ? piece : piece ^ ((c >> 1) & 3)) << 4);
        uint8_t* to = dst + ((row0 + r0 + c) * args.cols + f) * es;
        if (f < args.cols) {
          for (int i = 0; i < E::kRows; i += rows_at_once)
            if (r0 + c + i >= t.lo && r0 + c + i < t.hi &&
                in_bounds((row0 + r0 + c + i) * args.cols + f + 16 / es <= args.out_len, args.status))
              *reinterpret_cast<uint4*>(to + static_cast<int64_t>(i) * args.cols * es) =
                  *reinterpret_cast<const uint4*>(from + i * 32 * es);
        }
        __syncwarp();
      }
    };

    for (int u = first_unit; u < num_units; u += stride) {
      if (!wait_warp(&unit_full[slot], unit_phase, abort_flag, args.status, args.wait_ns)) break;
      const Unit t = units[slot];
      __syncwarp();
      if (lane == 0) mbar_arrive(&unit_empty[slot]);
      next_slot(slot, unit_phase);
      const int64_t row0 = args.contract ? static_cast<int64_t>(t.e) * args.rows : 0;  // result row of row 0
      const int f0 = t.ct * kFeatTile + half * 128 + static_cast<int>(quad) * 32;
      const bool mine = f0 < args.cols;
      const int r_base = t.w0 + c_base;
      // biases of this thread's features: one, or those of its four blocks
      constexpr int kOwn = E::kF32 ? 1 : 4;
      float bias[kOwn];
#pragma unroll
      for (int m = 0; m < kOwn; ++m) {
        const int f = f0 + (E::kF32 ? static_cast<int>(lane) : 8 * m + static_cast<int>(lane >> 2));
        bias[m] = 0.0f;
        // rows of none behind the last segment and ahead of the first have no expert, and no bias
        const int64_t at = static_cast<int64_t>(t.e) * args.cols + f;
        if (KIND != kLinGrad && args.bias != nullptr && t.n > 0 && f < args.cols && in_bounds(at < args.bias_len, args.status))
          bias[m] = __uint_as_float(static_cast<uint32_t>(args.bias[at]) << 16);
      }
      // chunks that hold computed rows, and their auxiliary values: two of them on the way at a time
      const int j_first = max(0, (t.lo - r_base) / E::kRows);
      const int j_end = mine && t.n > 0 && pair == 0 ? min(E::kChunks, (t.live - r_base + E::kRows - 1) / E::kRows) : 0;
      // By each thread's own copies, which need no barrier; tensor copies took the same time (gradient through GELU of
      // 14336 x 4096 MXFP8 80 us), fetching the rows into L2 a unit ahead cost 4 us.
      auto aux_load = [&](int j) {
        if constexpr (E::kAux) {
          if (args.aux != nullptr && j < j_end) {
            constexpr int es = E::kF32 ? 4 : 2, per_row = 2 * es, at_once = 32 / per_row;  // 16-byte pieces of a row
            const int c = static_cast<int>(lane) / per_row, piece = static_cast<int>(lane) % per_row;
            const int f = f0 + piece * (16 / es), first = r_base + E::kRows * j + c;
            const uint32_t to = smem_u32(bufs + (j & 1) * E::kChunkBytes) + c * 32 * es +
                                ((E::kF32 ? piece : piece ^ ((c >> 1) & 3)) << 4);
            const uint8_t* from = args.aux + (first * args.aux_stride + f) * es;
#pragma unroll
            for (int i = 0; i < E::kRows; i += at_once) {
              const bool there = f < args.cols && first + i >= t.lo && first + i < t.live &&
                                 in_bounds((first + i) * args.aux_stride + f + 16 / es <= args.aux_len, args.status);
              copy_16(to + i * 32 * es, there ? from + i * args.aux_stride * es : args.aux, there ? 16 : 0);
            }
          }
          asm volatile("cp.async.commit_group;" ::: "memory");
        }
      };
      if constexpr (E::kAux) {
        if (lane == 0) bulk_wait_group_read<0>();  // the last unit's stores have left the chunks
        __syncwarp();
        aux_load(j_first);
        if constexpr (E::kChunks > 1) aux_load(j_first + 1);
      }
      uint32_t acc[E::kWarpCols / 32][32];
      if (t.n > 0) {
        if (!wait_warp(tmem_full, acc_phase, abort_flag, args.status, args.wait_ns)) break;
        acc_phase ^= 1u;
        tc_fence_after();
#pragma unroll
        for (int j = 0; j < E::kWarpCols / 32; ++j) {
          if (c_base + 32 * j < t.n) {
            const uint32_t at = tmem_base + ((quad * 32u) << 16) + c_base + 32 * j;
            if constexpr (E::kF32) {
              tmem_ld_32x32b_x32(at, acc[j]);
            } else {
              tmem_ld_16x256b_x4(at, acc[j]);
              tmem_ld_16x256b_x4(at + (16u << 16), acc[j] + 16);
            }
          }
        }
        tmem_ld_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_remote(tmem_empty_leader);
      }
      float colsum[4] = {0.0f, 0.0f, 0.0f, 0.0f};
      if (args.split_bits > 0) {
        // The first pair adds the others' sums of the depth in their order, where its operand ring stood: its MMAs are
        // done, and a cluster has this one unit. Its four warps of the window's 32 rows say so to their peers, whose
        // stores complete on the warp's barrier.
        bool gone = false;
        if (c_base == 0 && mine && t.n > 0) {
          if (pair == 0) {
            if (lane == 0) {
              mbar_arrive_expect_tx(&sums_bar[w], (splits - 1) * 4096);
              for (int p = 1; p < splits; ++p) mbar_arrive_remote(mapa_shared(smem_u32(&ready_bar[w]), rank + 2 * p));
            }
            __syncwarp();
            gone = !wait_warp(&sums_bar[w], 0, abort_flag, args.status, args.wait_ns);
            if (!gone) {
              for (int p = 1; p < splits; ++p) {
                const uint32_t* from = reinterpret_cast<const uint32_t*>(smem + L::a_off + ((p - 1) * 4 + w) * 4096) + lane;
#pragma unroll
                for (int i = 0; i < 32; ++i)
                  acc[0][i] = __float_as_uint(__uint_as_float(acc[0][i]) + __uint_as_float(from[32 * i]));
              }
            }
          } else {
            gone = !wait_warp(&ready_bar[w], 0, abort_flag, args.status, args.wait_ns);
            if (!gone) {
              const uint32_t to = mapa_shared(smem_u32(smem + L::a_off + ((pair - 1) * 4 + w) * 4096 + lane * 4), half);
              const uint32_t bar = mapa_shared(smem_u32(&sums_bar[w]), half);
#pragma unroll
              for (int i = 0; i < 32; ++i) store_remote(to + 128 * i, acc[0][i], bar);
            }
          }
        }
        if (gone) break;
        if (pair != 0) continue;
      }
#pragma unroll
      for (int j = 0; j < E::kChunks; ++j) {
        const int r0 = r_base + E::kRows * j;
        if (!mine || r0 >= t.hi || r0 + E::kRows <= t.lo) continue;
        // the chunk's values, worked on in the accumulator's registers, in pairs: f(h, i, ..), i of the 32 rows h
        auto pairs = [&](auto&& f) {
#pragma unroll
          for (int h = 0; h < E::kSub; ++h) {
            uint32_t(&v)[32] = acc[j * E::kSub + h];
#pragma unroll
            for (int i = 0; i < 32; i += 2) {
              float a = __uint_as_float(v[i]), b = __uint_as_float(v[i + 1]);
              f(h, i, a, b);
              v[i] = __float_as_uint(a);
              v[i + 1] = __float_as_uint(b);
            }
          }
        };
        const bool some = t.n > 0 && r0 < t.live;
        if (some) {
          pairs([&](int, int i, float& a, float& b) {
            const uint64_t c = f2_splat(bias[E::kF32 ? 0 : (i >> 4) * 2 + ((i >> 1) & 1)]);
            if constexpr (FMT == BSQ_NVFP4) f2_split(f2_fma(f2(a, b), f2_splat(alpha), c), a, b);
            else if constexpr (KIND != kLinGrad) f2_split(f2_add(f2(a, b), c), a, b);
          });
        } else {
          if constexpr (!E::kF32) asm volatile("");  // a branch, not a select for each value
#pragma unroll
          for (int h = 0; h < E::kSub; ++h) {
#pragma unroll
            for (int i = 0; i < 32; ++i) acc[j * E::kSub + h][i] = 0u;
          }
        }
        const bool whole = r0 >= t.lo && r0 + E::kRows <= t.live;
        auto mask = [&] {  // rows of other experts, and rows of none
          if (!whole) {
            if constexpr (!E::kF32) asm volatile("");  // a branch, not a select for each value
#pragma unroll
            for (int h = 0; h < E::kSub; ++h) {
#pragma unroll
              for (int i = 0; i < 32; ++i) {
                const int r = r0 + 32 * h + row_of(i);
                if (r < t.lo || r >= t.live) acc[j * E::kSub + h][i] = 0u;
              }
            }
          }
        };
        auto put_bf16 = [&](uint8_t* buf) {
#pragma unroll
          for (int h = 0; h < E::kSub; ++h, buf += 2048) {
            const uint32_t(&v)[32] = acc[j * E::kSub + h];
            if constexpr (E::kF32) {
#pragma unroll
              for (int i = 0; i < 32; i += 2) {
                const uint32_t b = bf16_pair(v[i], v[i + 1]);
                *reinterpret_cast<uint16_t*>(buf + i * 64 + lane * 2) = static_cast<uint16_t>(b);
                *reinterpret_cast<uint16_t*>(buf + i * 64 + 64 + lane * 2) = static_cast<uint16_t>(b >> 16);
              }
            } else {
              const uint32_t at = smem_u32(buf) + mat_off;
#pragma unroll
              for (int q = 0; q < 4; ++q)
                stmatrix_trans(at + q * 512, bf16_pair(v[4 * q], v[4 * q + 1]), bf16_pair(v[4 * q + 2], v[4 * q + 3]),
                               bf16_pair(v[16 + 4 * q], v[17 + 4 * q]), bf16_pair(v[18 + 4 * q], v[19 + 4 * q]));
            }
          }
        };
        // the auxiliary values, which the results then take the places of
        uint8_t* const buf = bufs + (E::kAux ? (j & 1) * E::kChunkBytes : 0);
        uint32_t x[E::kAux && KIND != kLinGrad ? (E::kF32 ? 32 : 16) : 1];
        const bool aux = E::kAux && args.aux != nullptr && some;
        if constexpr (E::kAux) {
          if (aux) {
            // this chunk's copies: the next chunk's may still be on their way
            if constexpr (E::kChunks > 1) asm volatile("cp.async.wait_group 1;" ::: "memory");
            else asm volatile("cp.async.wait_group 0;" ::: "memory");
            __syncwarp();
            if constexpr (E::kF32) {
#pragma unroll
              for (int i = 0; i < 32; ++i) x[i] = *reinterpret_cast<const uint32_t*>(buf + i * 128 + lane * 4);
            } else if constexpr (KIND != kLinGrad) {
              const uint32_t at = smem_u32(buf) + mat_off;
#pragma unroll
              for (int q = 0; q < 4; ++q) ldmatrix_trans(at + q * 512, x[2 * q], x[2 * q + 1], x[8 + 2 * q], x[9 + 2 * q]);
            }
            __syncwarp();
          }
        }
        if constexpr (KIND != kLinGrad && KIND != kLinPlain) {
          if (args.pre != nullptr) {
            mask();
            if (!aux && lane == 0) bulk_wait_group_read<0>();
            __syncwarp();
            put_bf16(buf);
            store(buf, &mapPre, args.pre, false, row0, r0, f0, t);
          }
          by_activation(args.act, [&](auto k) {
            pairs([&](int, int, float& a, float& b) { act_pair<decltype(k)::value>(a, b); });
          });
        }
        if constexpr (E::kAux) {
          if (aux) {
            auto aux_of = [&](int i, float& a, float& b) {
              if constexpr (E::kF32) {
                a = __uint_as_float(x[i]);
                b = __uint_as_float(x[i + 1]);
              } else {
                a = bf16_lo(x[i >> 1]);
                b = bf16_hi(x[i >> 1]);
              }
            };
            if constexpr (KIND == kLinGrad) {
              by_activation(args.act, [&](auto k) {  // eight rows at a time: registers are short
#pragma unroll
                for (int hq = 0; hq < 4 * E::kSub; ++hq) {
                  uint32_t(&v)[32] = acc[j * E::kSub + hq / 4];
                  const int q = hq % 4;
                  uint32_t y[4];
                  ldmatrix_trans(smem_u32(buf) + mat_off + hq * 512, y[0], y[1], y[2], y[3]);
#pragma unroll
                  for (int m = 0; m < 4; ++m) {
                    const int i = (m >> 1) * 16 + 4 * q + 2 * (m & 1);
                    float a = __uint_as_float(v[i]), b = __uint_as_float(v[i + 1]);
                    slope_pair<decltype(k)::value>(a, b, bf16_lo(y[m]), bf16_hi(y[m]));
                    v[i] = __float_as_uint(a);
                    v[i + 1] = __float_as_uint(b);
                  }
                }
              });
            } else {
              pairs([&](int, int i, float& a, float& b) {
                float p, q;
                aux_of(i, p, q);
                f2_split(f2_add(f2(a, b), f2(p, q)), a, b);
              });
            }
          }
        }
        mask();
        if constexpr (KIND == kLinGrad) {
          pairs([&](int, int i, float& a, float& b) { colsum[(i >> 4) * 2 + ((i >> 1) & 1)] += a + b; });
        }
        // the chunk's values are computed while the store before it may still be reading the staging
        if ((!aux || args.pre != nullptr) && lane == 0) bulk_wait_group_read<0>();
        __syncwarp();
        if constexpr (E::kF32) {
#pragma unroll
          for (int i = 0; i < 32; ++i) *reinterpret_cast<uint32_t*>(buf + i * 128 + lane * 4) = acc[j][i];
        } else {
          put_bf16(buf);
        }
        store(buf, &mapOut, args.out, E::kF32, row0, r0, f0, t);
        if constexpr (E::kAux) {
          if constexpr (E::kChunks > 1) {
            if (lane == 0) bulk_wait_group_read<0>();
            __syncwarp();
            aux_load(j + 2);
          }
        }
      }
      if constexpr (KIND == kLinGrad) {
        if (args.sums != nullptr) {
#pragma unroll
          for (int m = 0; m < 4; ++m) {  // over the four threads that hold a feature's rows
            colsum[m] += __shfl_xor_sync(0xffffffffu, colsum[m], 1);
            colsum[m] += __shfl_xor_sync(0xffffffffu, colsum[m], 2);
            const int f = f0 + 8 * m + static_cast<int>(lane >> 2);
            const int64_t at =
                (static_cast<int64_t>(t.window) * (kRowTile / E::kWarpCols) + (w >> 2)) * args.cols + f;
            if ((lane & 3u) == 0 && f < args.cols && in_bounds(at < args.sums_len, args.status)) args.sums[at] = colsum[m];
          }
        }
      }
    }
    if constexpr (E::kAux) asm volatile("cp.async.wait_all;" ::: "memory");
    if (lane == 0) bulk_wait_group0();
  }

  if (*abort_flag && threadIdx.x == 0) {
    // some wait gave up: copies that no leader announced may still be on their way, for microseconds at most
    const uint64_t t0 = globaltimer_ns();
    for (int i = 0; i < (1 << 20) && globaltimer_ns() - t0 < 200000; ++i) {
    }
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

inline cudaLaunchConfig_t lin_config(cudaLaunchAttribute* attr, int clusters, int splits, int threads, int smem,
                                     cudaStream_t stream) {
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2 * splits;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(2 * splits * clusters);
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
  // per device: the shared-memory opt-in, and the clusters of 1, 2 and 4 pairs that fit (0 = unusable)
  struct Fit {
    int clusters[3] = {0, 0, 0};
  };
  static PerDevice<Fit> setup;
  const Fit fit = setup.run(dev.device, [] {
    Fit r;
    cudaFuncAttributes fa;  // the warpgroups' split of registers must add up to the launch's
    bool ok = cudaFuncGetAttributes(&fa, linear_kernel<FMT, KIND>) == cudaSuccess && fa.numRegs >= E::kLaunchRegs &&
              cudaFuncSetAttribute(linear_kernel<FMT, KIND>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem) ==
                  cudaSuccess;
    for (int i = 0; i < 3 && ok; ++i) {
      cudaLaunchAttribute at[2];
      cudaLaunchConfig_t cfg = lin_config(at, 1, 1 << i, E::kThreads, kSmem, nullptr);
      ok = cudaOccupancyMaxActiveClusters(&r.clusters[i], linear_kernel<FMT, KIND>, &cfg) == cudaSuccess;
    }
    if (!ok) cudaGetLastError();
    return ok ? r : Fit{};
  });
  const int max_clusters = fit.clusters[0];
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
  CUtensorMap mW, mX, mXs, mSfw, mSfx, mOut, mPre;
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
  const cuuint32_t chunk[2] = {32, E::kRows};
  const CUtensorMapSwizzle staged = E::kF32 ? s0 : CU_TENSOR_MAP_SWIZZLE_64B;
  {
    const u64 dims[2] = {cols, rows * (c.contract ? experts : 1)}, st[1] = {cols * es}, st16[1] = {cols * 2};
    ok = ok && lin_map(&mOut, ot, 2, c.out, dims, st, chunk, staged);
    mPre = mOut;
    if (c.pre != nullptr) ok = ok && lin_map(&mPre, bf16, 2, c.pre, dims, st16, chunk, staged);
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
  a.aux = E::kAux ? static_cast<const uint8_t*>(c.aux) : nullptr;
  a.aux_stride = c.aux_stride;
  const StallInjection inj = take_stall(BSQ_KERNEL_LINEAR);
  a.stall_after = inj.after;
  a.wait_ns = inj.limit_ns;
  // A segment that begins inside a tile has up to 127 + 255 rows more in windows than of its own, the rows ahead of all
  // segments up to 255: 382 (experts + 1) + 255 rows in all are fewer than 2 (experts + 1) windows.
  const int64_t windows = ceil_div(c.rows, kRowTile) * (c.contract ? c.experts : 1) +
                          (c.counts != nullptr && !c.contract ? 2 * (c.experts + 1) : 0);
  const int64_t units = windows * a.tiles_c;
  a.max_windows = static_cast<int>(windows);
  a.bias_len = c.cols * static_cast<int64_t>(experts);
  a.aux_len = (c.rows - 1) * c.aux_stride + c.cols;
  a.out_len = c.rows * c.cols * static_cast<int64_t>(c.contract ? experts : 1);
  a.sums_len = windows * (kRowTile / E::kWarpCols) * c.cols;
  // A few rows against one weight: one window, as many units as feature tiles, each bound by the stream of its weights
  // into one pair's SMs. Where that leaves half of the pairs without work, two or four pairs share a unit's depth.
  // One row, 4096 x 4096 NVFP4: 10.4 us with one pair a unit, 8.8 us with four.
  a.split_bits = 0;
  if (c.counts == nullptr && !c.contract && c.rows <= 32)
    for (int i = 1; i < 3 && units <= fit.clusters[i] && ceil_div(a.mmas, 4) >= 2 << i; ++i) a.split_bits = i;
  const int clusters =
      static_cast<int>(a.split_bits > 0 ? units : std::min<int64_t>(units, std::min(max_clusters, dev.num_sms / 2)));
  cudaLaunchAttribute at[2];
  cudaLaunchConfig_t cfg = lin_config(at, clusters, 1 << a.split_bits, E::kThreads, kSmem, stream);
  if (cudaLaunchKernelEx(&cfg, linear_kernel<FMT, KIND>, mW, mX, mXs, mSfw, mSfx, mOut, mPre, a) != cudaSuccess)
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
