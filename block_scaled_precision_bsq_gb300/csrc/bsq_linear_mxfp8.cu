// bsq_linear_mxfp8.cu -- the products of bsq_linear.cuh on MXFP8 operands (a file for each format: they compile side by side).
#include "bsq_linear.cuh"

namespace bsq {
template int launch_linear<BSQ_MXFP8>(const LinearCall&, cudaStream_t, const DeviceInfo&);
}  // namespace bsq
