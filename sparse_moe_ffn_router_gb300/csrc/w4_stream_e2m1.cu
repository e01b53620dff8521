// w4_stream_e2m1.cu -- the streaming kernels of w4_stream.cuh for MOE_W4_E2M1.
#include "w4_stream.cuh"

namespace moe {

cudaError_t launch_w4_stream_e2m1(int group, int which, const W4StreamArgs& p, cudaStream_t s) {
    return launch_w4_stream_f<MOE_W4_E2M1>(group, which, p, s);
}

}  // namespace moe
