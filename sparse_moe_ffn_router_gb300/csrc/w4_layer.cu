// w4_layer.cu -- launch sequences of the products on packed 4-bit weights: the linear layer and
// the experts of the MoE layer (the routing before and the combine after are the layer's own).
#include "w4_stream.cuh"

namespace moe {

cudaError_t launch_w4_stream(int format, int group, int which, const W4StreamArgs& p, cudaStream_t s) {
    switch (format) {
        case MOE_W4_INT4: return launch_w4_stream_int4(group, which, p, s);
        case MOE_W4_INT4_ZP: return launch_w4_stream_int4_zp(group, which, p, s);
        case MOE_W4_E2M1: return launch_w4_stream_e2m1(group, which, p, s);
        default: return cudaErrorInvalidValue;
    }
}

cudaError_t launch_w4_linear(const moe_w4_format& f, const W4LinearArgs& l, cudaStream_t s) {
    W4StreamArgs p = {};
    p.w = l.w;
    p.x = l.x;
    p.bias = l.bias;
    p.out = l.out;
    p.rows[0] = l.N;
    p.cols[0] = l.K;
    p.T = l.T;
    p.err = l.err;
    p.wait_ns = l.wait_ns;
    p.a.num_sms = l.num_sms;
    return launch_w4_stream(f.format, f.group, kW4Linear, p, s);
}

// Gate_up and down of the dispatched groups; Y is complete when both have run.
cudaError_t launch_w4_experts(const LayerArgs& a, const moe_w4_format& f, cudaStream_t s) {
    W4StreamArgs p = {};
    p.a = a;
    p.T = a.T;
    p.err = &a.hdr->err;
    p.wait_ns = a.wait_ns;
    p.rows[0] = 2 * a.Is; p.rows[1] = 2 * a.I;
    p.cols[0] = p.cols[1] = a.H;
    p.matrix_bytes = w4_matrix_bytes(f.format, f.group, 2 * a.I, a.H);
    cudaError_t e = launch_w4_stream(f.format, f.group, kW4Up, p, s);
    if (e != cudaSuccess) return e;
    p.rows[0] = p.rows[1] = a.H;
    p.cols[0] = a.Is; p.cols[1] = a.I;
    p.matrix_bytes = w4_matrix_bytes(f.format, f.group, a.H, a.I);
    e = launch_w4_stream(f.format, f.group, kW4Down, p, s);
    if (e != cudaSuccess) return e;
    return a.gemm ? launch_combine(a, s) : launch_combine_pdl(a, s);
}

}  // namespace moe
