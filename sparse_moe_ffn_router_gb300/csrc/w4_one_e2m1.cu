// w4_one_e2m1.cu -- the one-token layer kernel of w4_one.cuh for MOE_W4_E2M1.
#include "w4_one.cuh"

namespace moe {

cudaError_t w4_one_e2m1(int group, const W4OneArgs* p, cudaStream_t s) { return w4_one_f<MOE_W4_E2M1>(group, p, s); }

}  // namespace moe
