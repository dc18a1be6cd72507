// k_norm.cu -- all-reduce + residual + RMS norm with the output in the data's type.
#include "norm_forward.cuh"

namespace vc {

cudaError_t launch_allreduce_rmsnorm(const NormArgs& a, vDataType_t dt, cudaStream_t s) {
    return norm_launch_q<0>(a, dt, s);
}

}  // namespace vc
