// k_norm_quant.cu -- all-reduce + residual + RMS norm with the output in 8 bits (e4m3) and
// fp32 scales, one per row or one per 128 elements.
#include "norm_forward.cuh"

namespace vc {

cudaError_t launch_allreduce_rmsnorm_quant(const NormArgs& a, vDataType_t dt, cudaStream_t s) {
    return a.groups == 0 ? norm_launch_q<1>(a, dt, s) : norm_launch_q<2>(a, dt, s);
}

}  // namespace vc
