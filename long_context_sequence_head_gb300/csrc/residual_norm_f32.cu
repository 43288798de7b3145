// The fp32 kernels of the norms around a block (residual_norm.cuh).
#include "residual_norm.cuh"

namespace uly {

cudaError_t launch_residual_norm_f32(const ResidualNormParams &p, const ResidualNormPlan &q, bool bwd, cudaStream_t s)
{
    return launch_residual_norm_typed<float>(p, q, bwd, s);
}

}  // namespace uly
