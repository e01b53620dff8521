// w4_stream_int4_zp.cu -- the streaming kernels of w4_stream.cuh for MOE_W4_INT4_ZP.
#include "w4_stream.cuh"

namespace moe {

cudaError_t launch_w4_stream_int4_zp(int group, int which, const W4StreamArgs& p, cudaStream_t s) {
    return launch_w4_stream_f<MOE_W4_INT4_ZP>(group, which, p, s);
}

}  // namespace moe
