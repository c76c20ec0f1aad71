// bsq_linear.h -- host-side declarations of the products of bsq_linear.cuh: grouped by expert, with
// activation and residual, their gradients.
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

#include "bsq.h"
#include "bsq_internal.h"

namespace bsq {

// Epilogue kinds (bsq_linear.cuh).
enum LinearKind {
  kLinPlain = 0,   // bf16 out, bias
  kLinAct = 1,     // bf16 out, bias and activation, its argument kept if wanted
  kLinRes = 2,     // the same with a bf16 residual added
  kLinGrad = 3,    // bf16 out times the activation's derivative, column sums
  kLinF32 = 4,     // fp32 out, bias and activation
  kLinResF32 = 5   // the same with an fp32 residual added
};

// One product, arguments validated (bsq_linear.cu). out[r, c] = sum over depth of rows' operand and cols' operand.
struct LinearCall {
  int kind = kLinPlain;
  int activation = 0;     // BSQ_ACT_*
  bool contract = false;  // the weight gradient: experts are ranges of the depth
  bool stack_cols = false;  // the weights' operand has the experts side by side along its depth
  int64_t rows = 0, cols = 0, depth = 0, experts = 0;  // experts 0: one weight; contract: rows of each expert's result
  const void *a = nullptr, *a_scales = nullptr;  // rows' operand
  const void *b = nullptr, *b_scales = nullptr;  // cols' operand
  const int32_t *counts = nullptr, *offsets = nullptr;
  const void* bias = nullptr;
  const void* aux = nullptr;  // residual, or the activation's argument for its derivative
  int64_t aux_stride = 0;     // elements
  void *out = nullptr, *pre = nullptr;
  float* sums = nullptr;  // column sums of each window (workspace)
};

// The rows of window sums that a call may write (its workspace has that many rows of `cols` floats).
int64_t linear_sum_rows(int64_t rows, int64_t experts);

// One instance for each format (bsq_linear_<format>.cu).
template <int FMT>
int launch_linear(const LinearCall& c, cudaStream_t stream, const DeviceInfo& dev);

// dbias[e][c] = sum over expert e's windows of `sums` (experts 0: one sum over all), after a kLinGrad launch.
int launch_linear_sums(const LinearCall& c, float* dbias, cudaStream_t stream, const DeviceInfo& dev);

}  // namespace bsq
