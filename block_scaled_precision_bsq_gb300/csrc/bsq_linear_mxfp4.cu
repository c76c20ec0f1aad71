// bsq_linear_mxfp4.cu -- the products of bsq_linear.cuh on MXFP4 operands (a file for each format: they compile side by side).
#include "bsq_linear.cuh"

namespace bsq {
template int launch_linear<BSQ_MXFP4>(const LinearCall&, cudaStream_t, const DeviceInfo&);
}  // namespace bsq
