// w4_one_int4.cu -- the one-token layer kernel of w4_one.cuh for MOE_W4_INT4.
#include "w4_one.cuh"

namespace moe {

cudaError_t w4_one_int4(int group, const W4OneArgs* p, cudaStream_t s) { return w4_one_f<MOE_W4_INT4>(group, p, s); }

}  // namespace moe
