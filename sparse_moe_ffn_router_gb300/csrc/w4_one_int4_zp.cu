// w4_one_int4_zp.cu -- the one-token layer kernel of w4_one.cuh for MOE_W4_INT4_ZP.
#include "w4_one.cuh"

namespace moe {

cudaError_t w4_one_int4_zp(int group, const W4OneArgs* p, cudaStream_t s) { return w4_one_f<MOE_W4_INT4_ZP>(group, p, s); }

}  // namespace moe
