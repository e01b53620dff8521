// norm_fp16.cu -- the norm kernels for fp16 tensors.
#include "norm.cuh"

namespace moe {

cudaError_t launch_norm_fp16(const NormArgs& a, cudaStream_t s, bool backward) { return launch_norm_any<fp16>(a, s, backward); }

}  // namespace moe
