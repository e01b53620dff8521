// w4_layer.cu -- launch sequences of the products on packed 4-bit weights: the linear layer and
// the experts of the MoE layer (the routing before and the combine after are the layer's own).
#include "w4_gemm.cuh"
#include "w4_one.cuh"

namespace moe {

cudaError_t launch_w4_stream(int format, int group, int which, const W4StreamArgs& p, cudaStream_t s) {
    switch (format) {
        case MOE_W4_INT4: return launch_w4_stream_int4(group, which, p, s);
        case MOE_W4_INT4_ZP: return launch_w4_stream_int4_zp(group, which, p, s);
        case MOE_W4_E2M1: return launch_w4_stream_e2m1(group, which, p, s);
        default: return cudaErrorInvalidValue;
    }
}

cudaError_t launch_w4_gemm(int format, int group, int which, const W4GemmArgs& p, const CUtensorMap& a0,
                           const CUtensorMap& a1, const LayerArgs& a, cudaStream_t s) {
    switch (format) {
        case MOE_W4_INT4: return launch_w4_gemm_int4(group, which, p, a0, a1, a, s);
        case MOE_W4_INT4_ZP: return launch_w4_gemm_int4_zp(group, which, p, a0, a1, a, s);
        case MOE_W4_E2M1: return launch_w4_gemm_e2m1(group, which, p, a0, a1, a, s);
        default: return cudaErrorInvalidValue;
    }
}

// The linear layer's path. The streaming kernel passes over the weights once for 8 tokens: about 0.04 us for
// each record of a CTA. The tensor-core kernel takes about 0.55 us for 256 rows of one column block by at most
// 128 tokens, a wave of CTAs at a time. In both the column blocks are a factor, so what decides are a CTA's
// strips: measured (2048 x 2048) 10.8 against 12.9 us at 128 tokens and 14.8 against 12.5 at 192;
// (4096 x 2048) 10.7 against 12.2 at 64 and 14.8 against 12.5 at 96; (24576 x 4096) 14.7 against 20.2 at 8 and
// 25.2 against 20.2 at 16.
static bool w4_linear_on_tensor_cores(long long T, long long N, int num_sms) {
    const long long strips = (N + kW4Strip - 1) / kW4Strip * ((T + kW4Tok - 1) / kW4Tok);
    const long long tiles = (N + kW4gRows - 1) / kW4gRows * ((T + kW4gTok - 1) / kW4gTok);
    return strips > 14 * num_sms * ((tiles + num_sms - 1) / num_sms);
}

static cudaError_t w4_linear_gemm(const moe_w4_format& f, const W4LinearArgs& l, cudaStream_t s) {
    CUtensorMap mx;
    if (!make_bf16_map(&mx, l.x, l.T, l.K, l.K, 32)) return cudaErrorInvalidValue;
    W4GemmArgs p = {};
    p.w[0] = l.w;
    p.rows[0] = l.N;
    p.cols[0] = l.K;
    p.bias = l.bias;
    p.out = l.out;
    p.T = l.T;
    p.err = l.err;
    p.wait_ns = l.wait_ns;
    LayerArgs a = {};
    a.num_sms = l.num_sms;
    return launch_w4_gemm(f.format, f.group, kW4GLinear, p, mx, mx, a, s);
}

// Gate_up and down of 256 tokens or more on the tensor cores.
static cudaError_t w4_experts_gemm(const LayerArgs& a, const moe_w4_format& f, cudaStream_t s) {
    CUtensorMap mx, mg, mh, mhs;  // the h rows are Imax apart; the columns past I (Is) of a row hold nothing
    if (!make_bf16_map(&mx, a.x, a.T, a.H, a.H, 32) || !make_bf16_map(&mg, a.x, a.T, a.H, a.H, 1) || !make_bf16_map(&mh, a.h, a.P + a.T, a.I, a.Imax, 32) ||
        !make_bf16_map(&mhs, a.h, a.P + a.T, a.Is, a.Imax, 32))
        return cudaErrorInvalidValue;
    W4GemmArgs p = {};
    p.err = &a.hdr->err;
    p.wait_ns = a.wait_ns;
    p.w[0] = reinterpret_cast<const uint8_t*>(a.gate_up);
    p.w[1] = reinterpret_cast<const uint8_t*>(a.sgu);
    p.matrix_bytes = w4_matrix_bytes(f.format, f.group, 2 * a.I, a.H);
    p.rows[0] = 2 * a.I; p.rows[1] = 2 * a.Is;
    p.cols[0] = p.cols[1] = a.H;
    cudaError_t e = launch_w4_gemm(f.format, f.group, kW4GUp, p, mg, mx, a, s);  // (gathered rows: boxes of one)
    if (e != cudaSuccess) return e;
    p.w[0] = reinterpret_cast<const uint8_t*>(a.down);
    p.w[1] = reinterpret_cast<const uint8_t*>(a.sd);
    p.matrix_bytes = w4_matrix_bytes(f.format, f.group, a.H, a.I);
    p.rows[0] = p.rows[1] = a.H;
    p.cols[0] = a.I; p.cols[1] = a.Is;
    e = launch_w4_gemm(f.format, f.group, kW4GDown, p, mh, mhs, a, s);
    if (e != cudaSuccess) return e;
    return a.K == 1 ? launch_combine_pdl(a, s) : launch_combine(a, s);  // (Y in fp32, in bf16)
}

// Strips of a block, at most: the power of two that still gives every SM four items or more of the
// call's `strips` (times token tiles). Blocks of one strip let small calls use every SM; full
// blocks spend less on each stage.
static int w4_want(long long strips, int num_sms) {
    int want = 1;
    while (want < kW4Warps && strips >= 8ll * want * num_sms) want *= 2;
    return want;
}

cudaError_t launch_w4_linear(const moe_w4_format& f, const W4LinearArgs& l, cudaStream_t s) {
    if (w4_linear_on_tensor_cores(l.T, l.N, l.num_sms)) return w4_linear_gemm(f, l, s);
    W4StreamArgs p = {};
    p.w = l.w;
    p.x = l.x;
    p.bias = l.bias;
    p.out = l.out;
    p.rows[0] = l.N;
    p.cols[0] = l.K;
    p.T = l.T;
    const long long strips = (l.N + kW4Strip - 1) / kW4Strip;
    p.b0 = p.b1 = w4_block(l.N, l.K, w4_want(strips * ((l.T + kW4Tok - 1) / kW4Tok), l.num_sms));
    p.err = l.err;
    p.wait_ns = l.wait_ns;
    p.a.num_sms = l.num_sms;
    return launch_w4_stream(f.format, f.group, kW4Linear, p, s);
}

// Gate_up and down of the dispatched groups; Y is complete when both have run.
cudaError_t launch_w4_experts(const LayerArgs& a, const moe_w4_format& f, cudaStream_t s) {
    if (a.gemm) return w4_experts_gemm(a, f, s);
    W4StreamArgs p = {};
    p.a = a;
    p.T = a.T;
    p.err = &a.hdr->err;
    p.wait_ns = a.wait_ns;
    p.rows[0] = 2 * a.Is; p.rows[1] = 2 * a.I;
    p.cols[0] = p.cols[1] = a.H;
    p.matrix_bytes = w4_matrix_bytes(f.format, f.group, 2 * a.I, a.H);
    // token tiles of the shared expert, and of the routed ones about (the routing is on the device)
    const long long ts = (a.T + kW4Tok - 1) / kW4Tok, tr = a.P < a.E ? a.P : a.E + a.P / kW4Tok;
    int want = w4_want(ts * (2 * a.Is / kW4Strip) + tr * (2 * a.I / kW4Strip), a.num_sms);
    p.b0 = w4_block(p.rows[0], a.H, want);
    p.b1 = w4_block(p.rows[1], a.H, want);
    cudaError_t e = launch_w4_stream(f.format, f.group, kW4Up, p, s);
    if (e != cudaSuccess) return e;
    p.rows[0] = p.rows[1] = a.H;
    p.cols[0] = a.Is; p.cols[1] = a.I;
    p.matrix_bytes = w4_matrix_bytes(f.format, f.group, a.H, a.I);
    want = w4_want((ts + tr) * (a.H / kW4Strip), a.num_sms);
    p.b0 = w4_block(a.H, a.Is, want);
    p.b1 = w4_block(a.H, a.I, want);
    e = launch_w4_stream(f.format, f.group, kW4Down, p, s);
    if (e != cudaSuccess) return e;
    return launch_combine_pdl(a, s);
}

static cudaError_t w4_one(int format, int group, const W4OneArgs* p, cudaStream_t s) {
    switch (format) {
        case MOE_W4_INT4: return w4_one_int4(group, p, s);
        case MOE_W4_INT4_ZP: return w4_one_int4_zp(group, p, s);
        case MOE_W4_E2M1: return w4_one_e2m1(group, p, s);
        default: return cudaErrorInvalidValue;
    }
}

// One token, strips of at most one stage (H <= 4096), h rows and sums that fit (then at least three stages do),
// one CTA per SM.
bool w4_one_supported(const LayerArgs& a, const moe_w4_format& f) {
    return a.T == 1 && a.H <= kW4StageRecs * kW4Cols && a.K <= kOneMaxK && a.Imax <= kOneMaxInner &&
           w4_one_strips(a, a.num_sms) <= kOneMaxUp && a.dlog && a.dh4 &&
           w4_one(f.format, f.group, nullptr, nullptr) == cudaSuccess;
}

// The whole layer of one token in one kernel.
cudaError_t launch_w4_one(const LayerArgs& a, const moe_w4_format& f, cudaStream_t s) {
    W4OneArgs p = {};
    p.a = a;
    p.dh = a.dh4;
    p.gu_bytes = w4_matrix_bytes(f.format, f.group, 2 * a.I, a.H);
    p.dn_bytes = w4_matrix_bytes(f.format, f.group, a.H, a.I);
    p.R = (a.H + kW4Cols - 1) / kW4Cols;
    const W4Block d = w4_block(a.H, a.Imax, kW4Warps);
    p.dwl = d.wl;
    p.drpw = d.rpw;
    p.dR = d.R;
    return w4_one(f.format, f.group, &p, s);
}

}  // namespace moe
