// norm_fp32.cu -- the norm kernels for fp32 tensors.
#include "norm.cuh"

namespace moe {

cudaError_t launch_norm_fp32(const NormArgs& a, cudaStream_t s, bool backward) { return launch_norm_any<float>(a, s, backward); }

}  // namespace moe
