// w4_gemm_int4.cu -- the tensor-core products of w4_gemm.cuh for MOE_W4_INT4.
#include "w4_gemm.cuh"

namespace moe {

cudaError_t launch_w4_gemm_int4(int group, int which, const W4GemmArgs& p, const CUtensorMap& b0, const CUtensorMap& b1,
                              const LayerArgs& a, cudaStream_t s) {
    return launch_w4_gemm_f<MOE_W4_INT4>(group, which, p, b0, b1, a, s);
}

}  // namespace moe
