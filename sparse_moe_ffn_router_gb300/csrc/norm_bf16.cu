// norm_bf16.cu -- the norm kernels for bf16 tensors.
#include "norm.cuh"

namespace moe {

cudaError_t launch_norm_bf16(const NormArgs& a, cudaStream_t s, bool backward) { return launch_norm_any<bf16>(a, s, backward); }

}  // namespace moe
