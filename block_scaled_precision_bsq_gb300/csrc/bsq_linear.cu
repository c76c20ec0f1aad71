// bsq_linear.cu -- entry points of the products with activation, residual and experts (bsq_linear.cuh), and
// the kernel that joins their column sums.
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>

#include "bsq_device.cuh"
#include "bsq_linear.h"

namespace bsq {

extern template int launch_linear<BSQ_MXFP8>(const LinearCall&, cudaStream_t, const DeviceInfo&);
extern template int launch_linear<BSQ_NVFP4>(const LinearCall&, cudaStream_t, const DeviceInfo&);
extern template int launch_linear<BSQ_MXFP4>(const LinearCall&, cudaStream_t, const DeviceInfo&);

namespace {

constexpr int64_t kWindow = 256;       // rows of a window (kRowTile)
constexpr int64_t kSumsPerWindow = 4;  // its column groups under kLinGrad

int launch_format(int fmt, const LinearCall& c, cudaStream_t stream, const DeviceInfo& dev) {
  switch (fmt) {
    case BSQ_MXFP8: return launch_linear<BSQ_MXFP8>(c, stream, dev);
    case BSQ_NVFP4: return launch_linear<BSQ_NVFP4>(c, stream, dev);
    case BSQ_MXFP4: return launch_linear<BSQ_MXFP4>(c, stream, dev);
    default: return BSQ_ERR_ARG;
  }
}

// dbias[e][c]: 32 columns a block, 8 threads a column take every eighth window sum, joined in a fixed order: the
// same inputs give the same bits. Expert e's windows stand behind those of the experts before it.
__global__ void __launch_bounds__(256)
    linear_sums_kernel(const float* sums, const int32_t* offsets, int rows, int max_windows, int cols, int experts,
                       float* dbias, int* status) {
  __shared__ float part[8][33];
  __shared__ int ahead[8];
  launch_dependents();
  grid_dependency_wait();
  const int e = blockIdx.y, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  int first = 0, windows = (rows + static_cast<int>(kWindow) - 1) / static_cast<int>(kWindow);
  if (offsets != nullptr) {
    auto offset_at = [&](int i) { return in_bounds(i >= 0 && i <= experts, status) ? offsets[i] : 0; };
    auto windows_of = [&](int i) {
      const int off = min(max(offset_at(i), 0), rows), end = min(max(offset_at(i + 1), off), rows);
      return end > off ? (end - (off & ~127) + static_cast<int>(kWindow) - 1) / static_cast<int>(kWindow) : 0;
    };
    int n = 0;
    for (int i = tid; i < e; i += 256) n = min(n + windows_of(i), max_windows);
    for (int d = 16; d > 0; d /= 2) n = min(n + __shfl_xor_sync(0xffffffffu, n, d), max_windows);
    if (lane == 0) ahead[warp] = n;
    __syncthreads();
    for (int i = 0; i < 8; ++i) first = min(first + ahead[i], max_windows);
    windows = min(windows_of(e), max_windows - first);  // those that segments without overlap have
  }
  const int c = blockIdx.x * 32 + lane;
  float s = 0.0f;
  if (c < cols) {
    const int64_t ahead_sums = first * kSumsPerWindow, all_sums = max_windows * kSumsPerWindow;
    const float* const own = sums + ahead_sums * cols + c;
#pragma unroll 4
    for (int i = warp; i < windows * kSumsPerWindow; i += 8) {
      if (in_bounds(ahead_sums + i < all_sums, status)) s += own[static_cast<int64_t>(i) * cols];
    }
  }
  part[warp][lane] = s;
  __syncthreads();
  if (warp == 0 && c < cols && in_bounds(e < experts, status)) {
    float total = part[0][lane];
    for (int i = 1; i < 8; ++i) total += part[i][lane];
    dbias[static_cast<int64_t>(e) * cols + c] = total;
  }
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

// What the three entry points share; BSQ_OK or the error code. The experts' weights lie one behind the other in whole
// scale tiles, hence the multiples of 128.
int check_product(int fmt, int64_t rows, int64_t cols, int64_t depth, int64_t experts, const void* a, const void* as,
                  const void* b, const void* bs, const void* out, const int32_t* counts, const int32_t* offsets) {
  if (fmt != BSQ_MXFP8 && fmt != BSQ_NVFP4 && fmt != BSQ_MXFP4) return BSQ_ERR_ARG;
  if (rows < 0 || cols <= 0 || depth < 0 || experts < 0) return BSQ_ERR_ARG;
  if (rows > INT32_MAX - 1024 || cols > INT32_MAX - 1024 || depth > INT32_MAX - 1024 || experts > BSQ_MAX_EXPERTS)
    return BSQ_ERR_SHAPE;
  if (cols % 8 != 0) return BSQ_ERR_SHAPE;
  if (rows > 0 && depth > 0 && (a == nullptr || as == nullptr || b == nullptr || bs == nullptr)) return BSQ_ERR_ARG;
  if (rows > 0 && out == nullptr) return BSQ_ERR_ARG;
  if (experts > 0 && (counts == nullptr || offsets == nullptr)) return BSQ_ERR_ARG;
  if (!aligned16(a) || !aligned16(as) || !aligned16(b) || !aligned16(bs) || !aligned16(out)) return BSQ_ERR_ALIGN;
  if (!aligned4(counts) || !aligned4(offsets)) return BSQ_ERR_ALIGN;
  return BSQ_OK;
}

int check_linear(const bsq_linear_args& a) {
  int st = check_product(a.fmt, a.rows, a.cols, a.depth, a.experts, a.A, a.A_scales, a.B, a.B_scales, a.out, a.counts,
                         a.offsets);
  if (st != BSQ_OK) return st;
  if (a.depth < 1) return BSQ_ERR_ARG;
  if (a.depth % 128 != 0 || (a.experts > 0 && a.cols % 128 != 0)) return BSQ_ERR_SHAPE;
  const int64_t e = std::max<int64_t>(a.experts, 1);
  if (e * a.cols > INT32_MAX || e * a.depth > INT32_MAX) return BSQ_ERR_SHAPE;
  if (a.activation < BSQ_ACT_NONE || a.activation > BSQ_ACT_RELU) return BSQ_ERR_ARG;
  return BSQ_OK;
}

int check_aux(const void* p, int64_t stride, int64_t cols, int64_t es) {
  if (p == nullptr) return BSQ_OK;
  // A matrix of rows of its own. The kernel would read repeated rows as well; bsq.h does not offer them, and a residual that
  // is the output could not have them.
  if (stride < cols || stride > INT32_MAX) return BSQ_ERR_SHAPE;
  return aligned16(p) && stride * es % 16 == 0 ? BSQ_OK : BSQ_ERR_ALIGN;
}

LinearCall call_of(const bsq_linear_args& a) {
  LinearCall c;
  c.activation = a.activation;
  c.stack_cols = (a.flags & BSQ_FLAG_STACK_COLS) != 0;
  c.rows = a.rows;
  c.cols = a.cols;
  c.depth = a.depth;
  c.experts = a.experts;
  c.a = a.A;
  c.a_scales = a.A_scales;
  c.b = a.B;
  c.b_scales = a.B_scales;
  c.counts = a.experts > 0 ? a.counts : nullptr;
  c.offsets = a.experts > 0 ? a.offsets : nullptr;
  c.bias = a.bias;
  c.out = a.out;
  c.pre = a.pre;
  return c;
}

}  // namespace

int64_t linear_sum_rows(int64_t rows, int64_t experts) {
  return (ceil_div(rows, kWindow) + (experts > 0 ? 2 * (experts + 1) : 0)) * kSumsPerWindow;
}

int launch_linear_sums(const LinearCall& c, float* dbias, cudaStream_t stream, const DeviceInfo& dev) {
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(ceil_div(c.cols, 32)), static_cast<unsigned>(std::max<int64_t>(c.experts, 1)));
  cfg.blockDim = dim3(256);
  cfg.stream = stream;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  if (cudaLaunchKernelEx(&cfg, linear_sums_kernel, static_cast<const float*>(c.sums), c.offsets,
                         static_cast<int>(c.rows), static_cast<int>(linear_sum_rows(c.rows, c.experts) / kSumsPerWindow),
                         static_cast<int>(c.cols), static_cast<int>(std::max<int64_t>(c.experts, 1)), dbias,
                         dev.status) != cudaSuccess)
    return BSQ_ERR_LAUNCH;
  return cudaGetLastError() == cudaSuccess ? BSQ_OK : BSQ_ERR_LAUNCH;
}

}  // namespace bsq

using bsq::record_error;

extern "C" {

int bsq_gemm_act(const bsq_linear_args* args, bsq_stream_t stream) {
  if (args == nullptr) return record_error(BSQ_ERR_ARG);
  const bsq_linear_args& a = *args;
  int st = bsq::check_linear(a);
  if (st != BSQ_OK) return record_error(st);
  if ((a.flags & ~(BSQ_FLAG_OUT_F32 | BSQ_FLAG_STACK_COLS)) || a.grad_pre != nullptr || a.dbias != nullptr)
    return record_error(BSQ_ERR_ARG);
  if (a.experts > 0 && a.residual != nullptr) return record_error(BSQ_ERR_ARG);
  const bool f32 = (a.flags & BSQ_FLAG_OUT_F32) != 0;
  st = bsq::check_aux(a.residual, a.residual_stride, a.cols, f32 ? 4 : 2);
  if (st != BSQ_OK) return record_error(st);
  if (!bsq::aligned16(a.pre) || (reinterpret_cast<uintptr_t>(a.bias) & 1u)) return record_error(BSQ_ERR_ALIGN);
  const bsq::DeviceInfo* dev = bsq::current_device();
  if (dev == nullptr) return record_error(BSQ_ERR_ARCH);
  if (a.rows == 0) return BSQ_OK;
  bsq::LinearCall c = bsq::call_of(a);
  c.aux = a.residual;
  c.aux_stride = a.residual_stride;
  if (f32) c.kind = a.residual != nullptr ? bsq::kLinResF32 : bsq::kLinF32;
  else if (a.residual != nullptr) c.kind = bsq::kLinRes;
  else c.kind = a.activation != BSQ_ACT_NONE || a.pre != nullptr ? bsq::kLinAct : bsq::kLinPlain;
  st = bsq::launch_format(a.fmt, c, reinterpret_cast<cudaStream_t>(stream), *dev);
  return st == BSQ_OK ? BSQ_OK : record_error(st);
}

size_t bsq_gemm_act_backward_workspace(int64_t rows, int64_t cols, int64_t experts) {
  if (rows < 0 || cols < 1 || experts < 0 || rows > INT32_MAX || cols > INT32_MAX || experts > BSQ_MAX_EXPERTS) return 0;
  return static_cast<size_t>(bsq::linear_sum_rows(rows, experts) * cols) * 4;
}

int bsq_gemm_act_backward(const bsq_linear_args* args, bsq_stream_t stream) {
  if (args == nullptr) return record_error(BSQ_ERR_ARG);
  const bsq_linear_args& a = *args;
  int st = bsq::check_linear(a);
  if (st != BSQ_OK) return record_error(st);
  if ((a.flags & ~BSQ_FLAG_STACK_COLS) || a.bias != nullptr || a.residual != nullptr || a.pre != nullptr)
    return record_error(BSQ_ERR_ARG);
  if (a.rows > 0 && (a.activation != BSQ_ACT_NONE) != (a.grad_pre != nullptr)) return record_error(BSQ_ERR_ARG);
  st = bsq::check_aux(a.grad_pre, a.grad_pre_stride, a.cols, 2);
  if (st != BSQ_OK) return record_error(st);
  if (!bsq::aligned4(a.dbias) || !bsq::aligned16(a.workspace)) return record_error(BSQ_ERR_ALIGN);
  if (a.dbias != nullptr && a.rows > 0 &&
      (a.workspace == nullptr || a.workspace_bytes < bsq_gemm_act_backward_workspace(a.rows, a.cols, a.experts)))
    return record_error(BSQ_ERR_ARG);
  const bsq::DeviceInfo* dev = bsq::current_device();
  if (dev == nullptr) return record_error(BSQ_ERR_ARCH);
  const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (a.rows == 0) {  // sums over no rows
    if (a.dbias != nullptr &&
        cudaMemsetAsync(a.dbias, 0, static_cast<size_t>(std::max<int64_t>(a.experts, 1) * a.cols) * 4, s) != cudaSuccess)
      return record_error(BSQ_ERR_LAUNCH);
    return BSQ_OK;
  }
  bsq::LinearCall c = bsq::call_of(a);
  c.aux = a.grad_pre;
  c.aux_stride = a.grad_pre_stride;
  c.sums = a.dbias != nullptr ? static_cast<float*>(a.workspace) : nullptr;
  c.kind = a.grad_pre != nullptr || a.dbias != nullptr ? bsq::kLinGrad : bsq::kLinPlain;
  st = bsq::launch_format(a.fmt, c, s, *dev);
  if (st == BSQ_OK && a.dbias != nullptr) st = bsq::launch_linear_sums(c, a.dbias, s, *dev);
  return st == BSQ_OK ? BSQ_OK : record_error(st);
}

int bsq_expert_gemm_wgrad(int fmt_flags, const void* dY, const void* dY_scales, const void* X, const void* X_scales,
                          const int32_t* counts, const int32_t* offsets, int64_t rows, int64_t N, int64_t K,
                          int64_t experts, void* out, bsq_stream_t stream) {
  const int fmt = fmt_flags & BSQ_FMT_MASK, flags = fmt_flags & ~BSQ_FMT_MASK;
  if (flags & ~BSQ_FLAG_OUT_F32) return record_error(BSQ_ERR_ARG);
  if (N < 1 || experts < 1) return record_error(BSQ_ERR_ARG);
  int st = bsq::check_product(fmt, N, K, rows, experts, dY, dY_scales, X, X_scales, out, counts, offsets);
  if (st != BSQ_OK) return record_error(st);
  if (rows % 32 != 0 || experts * N > INT32_MAX) return record_error(BSQ_ERR_SHAPE);
  const bsq::DeviceInfo* dev = bsq::current_device();
  if (dev == nullptr) return record_error(BSQ_ERR_ARCH);
  const bool f32 = (flags & BSQ_FLAG_OUT_F32) != 0;
  const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (rows == 0)
    return cudaMemsetAsync(out, 0, static_cast<size_t>(experts * N) * static_cast<size_t>(K) * (f32 ? 4 : 2), s) ==
                   cudaSuccess
               ? BSQ_OK
               : record_error(BSQ_ERR_LAUNCH);
  bsq::LinearCall c;
  c.kind = f32 ? bsq::kLinF32 : bsq::kLinPlain;
  c.contract = true;
  c.rows = N;
  c.cols = K;
  c.depth = rows;
  c.experts = experts;
  c.a = dY;
  c.a_scales = dY_scales;
  c.b = X;
  c.b_scales = X_scales;
  c.counts = counts;
  c.offsets = offsets;
  c.out = out;
  st = bsq::launch_format(fmt, c, s, *dev);
  return st == BSQ_OK ? BSQ_OK : record_error(st);
}

}  // extern "C"
