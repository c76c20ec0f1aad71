// bsq_elem.cuh -- element access shared by the kernels that stream bf16 / fp32 matrices through
// registers: 16-byte vectors, or single elements where rows do not keep 16-byte alignment.
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

namespace bsq {

__device__ __forceinline__ float bf16_to_f32(uint32_t bits) { return __uint_as_float(bits << 16); }
__device__ __forceinline__ uint16_t f32_to_bf16(float v) {
  uint16_t r;
  asm("cvt.rn.bf16.f32 %0, %1;" : "=h"(r) : "f"(v));
  return r;
}
__device__ __forceinline__ uint32_t f32x2_to_bf16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
// Data read once: no place in L1.
__device__ __forceinline__ uint4 load_stream16(const void* p) {
  uint4 v;
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p)
               : "memory");
  return v;
}

// kVec elements of T: 16 bytes (WIDE) or one element. bf16 elements have T = uint16_t.
template <typename T, bool WIDE>
struct Vec;
template <>
struct Vec<uint16_t, true> {
  static constexpr int kVec = 8;
  uint4 raw;
  __device__ __forceinline__ void load(const uint16_t* p) { raw = load_stream16(p); }
  __device__ __forceinline__ void clear() { raw = make_uint4(0, 0, 0, 0); }
  __device__ __forceinline__ void get(float* v) const {
    const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = __uint_as_float(w[i] << 16);
      v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  }
  __device__ __forceinline__ void put(uint16_t* p) const { *reinterpret_cast<uint4*>(p) = raw; }
  static __device__ __forceinline__ void store(uint16_t* p, const float* v) {
    *reinterpret_cast<uint4*>(p) = make_uint4(f32x2_to_bf16x2(v[0], v[1]), f32x2_to_bf16x2(v[2], v[3]),
                                              f32x2_to_bf16x2(v[4], v[5]), f32x2_to_bf16x2(v[6], v[7]));
  }
};
template <>
struct Vec<float, true> {
  static constexpr int kVec = 4;
  uint4 raw;
  __device__ __forceinline__ void load(const float* p) { raw = load_stream16(p); }
  __device__ __forceinline__ void clear() { raw = make_uint4(0, 0, 0, 0); }
  __device__ __forceinline__ void get(float* v) const {
    v[0] = __uint_as_float(raw.x);
    v[1] = __uint_as_float(raw.y);
    v[2] = __uint_as_float(raw.z);
    v[3] = __uint_as_float(raw.w);
  }
  __device__ __forceinline__ void put(float* p) const { *reinterpret_cast<uint4*>(p) = raw; }
  static __device__ __forceinline__ void store(float* p, const float* v) {
    *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
  }
};
template <>
struct Vec<uint16_t, false> {
  static constexpr int kVec = 1;
  uint16_t raw;
  __device__ __forceinline__ void load(const uint16_t* p) { raw = *p; }
  __device__ __forceinline__ void clear() { raw = 0; }
  __device__ __forceinline__ void get(float* v) const { v[0] = bf16_to_f32(raw); }
  __device__ __forceinline__ void put(uint16_t* p) const { *p = raw; }
  static __device__ __forceinline__ void store(uint16_t* p, const float* v) { *p = f32_to_bf16(v[0]); }
};
template <>
struct Vec<float, false> {
  static constexpr int kVec = 1;
  float raw;
  __device__ __forceinline__ void load(const float* p) { raw = *p; }
  __device__ __forceinline__ void clear() { raw = 0.0f; }
  __device__ __forceinline__ void get(float* v) const { v[0] = raw; }
  __device__ __forceinline__ void put(float* p) const { *p = raw; }
  static __device__ __forceinline__ void store(float* p, const float* v) { *p = v[0]; }
};

// Pairs of fp32 values. (One 64-bit register and the packed add / multiply / fma of sm_103a took as
// long: what they save in arithmetic the moves into register pairs cost.)
struct f32x2 {
  float x, y;
};
__device__ __forceinline__ f32x2 pair(float lo, float hi) { return f32x2{lo, hi}; }
__device__ __forceinline__ float2 halves(f32x2 v) { return make_float2(v.x, v.y); }
__device__ __forceinline__ f32x2 add2(f32x2 a, f32x2 b) { return f32x2{a.x + b.x, a.y + b.y}; }
__device__ __forceinline__ f32x2 mul2(f32x2 a, f32x2 b) { return f32x2{a.x * b.x, a.y * b.y}; }
__device__ __forceinline__ f32x2 fma2(f32x2 a, f32x2 b, f32x2 c) {
  return f32x2{fmaf(a.x, b.x, c.x), fmaf(a.y, b.y, c.y)};
}
__device__ __forceinline__ f32x2 both(float v) { return pair(v, v); }
__device__ __forceinline__ float sum_halves(f32x2 v) {
  const float2 h = halves(v);
  return h.x + h.y;
}

// 16 bytes of bf16 or fp32 values as pairs, and back.
template <typename T>
__device__ __forceinline__ void unpack16(const uint4& raw, f32x2* v) {
  const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
  if constexpr (sizeof(T) == 2) {
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = pair(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u));
  } else {
    v[0] = pair(__uint_as_float(w[0]), __uint_as_float(w[1]));
    v[1] = pair(__uint_as_float(w[2]), __uint_as_float(w[3]));
  }
}
template <typename T>
__device__ __forceinline__ uint4 pack16(const f32x2* v) {
  if constexpr (sizeof(T) == 2) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 h = halves(v[i]);
      w[i] = f32x2_to_bf16x2(h.x, h.y);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
  } else {
    const float2 a = halves(v[0]), b = halves(v[1]);
    return make_uint4(__float_as_uint(a.x), __float_as_uint(a.y), __float_as_uint(b.x), __float_as_uint(b.y));
  }
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int m = 16; m > 0; m >>= 1) v += __shfl_xor_sync(0xffffffffu, v, m);
  return v;
}

__device__ __forceinline__ uint32_t cluster_size() {
  uint32_t r;
  asm("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_barrier() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// Whether vectors of 16 bytes may start every `stride_bytes` from p (true for no pointer at all).
inline bool wide_ok(const void* p, int64_t stride_bytes) {
  return p == nullptr || ((reinterpret_cast<uintptr_t>(p) | static_cast<uintptr_t>(stride_bytes)) & 15u) == 0;
}

// Programmatic dependent launch for the kernels of these files: each is launched with the attribute,
// lets the next one in the stream be launched at once and waits for the one before it ahead of its first
// access to global memory, so that launches overlap (a sort and a gather of one token: 11.3 us without).
__device__ __forceinline__ void enter_stream() {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
}
template <typename... P, typename... A>
cudaError_t launch_in_stream(void (*kernel)(P...), dim3 grid, int threads, size_t dynamic, cudaStream_t stream, int cluster,
                             const A&... args) {
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute at[2];
  cfg.gridDim = grid;
  cfg.blockDim = dim3(static_cast<unsigned>(threads));
  cfg.dynamicSmemBytes = dynamic;
  cfg.stream = stream;
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  at[1].id = cudaLaunchAttributeClusterDimension;
  at[1].val.clusterDim.x = static_cast<unsigned>(cluster);
  at[1].val.clusterDim.y = 1;
  at[1].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

}  // namespace bsq
