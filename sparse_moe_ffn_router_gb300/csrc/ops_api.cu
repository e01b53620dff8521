// ops_api.cu -- C-ABI entry points of the layer's parts (exchange, linear layers, norms): host-side
// validation, then the launches.
#include <string.h>

#include "ops.cuh"

using namespace moe;

namespace {

constexpr int32_t kMaxRows = 0x7fff0000;  // 2^31 - 2^16

bool misaligned(const void* p) { return ((uintptr_t)p & 15u) != 0; }

moe_status to_status(cudaError_t e) { return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA; }

// A buffer of a call: nothing when p is NULL.
struct Buf {
    const void* p;
    size_t n;
};

bool meets(const Buf& a, const Buf& b) {
    const uintptr_t x = (uintptr_t)a.p, y = (uintptr_t)b.p;
    return a.p && b.p && a.n && b.n && x < y + b.n && y < x + a.n;
}

// Whether a result overlaps another buffer of the call. Pairs (r, b) with r.p == b.p and r.n == b.n are allowed where
// same says so: bit j of same[i] for result i and buffer j.
template <int R, int B>
bool overlaps(const Buf (&results)[R], const Buf (&others)[B], const unsigned (&same)[R]) {
    for (int i = 0; i < R; ++i) {
        for (int j = i + 1; j < R; ++j)
            if (meets(results[i], results[j])) return true;
        for (int j = 0; j < B; ++j)
            if (meets(results[i], others[j]) &&
                !((same[i] >> j & 1u) && results[i].p == others[j].p && results[i].n == others[j].n))
                return true;
    }
    return false;
}

template <int N>
bool any_misaligned(const void* const (&p)[N]) {
    for (const void* q : p)
        if (misaligned(q)) return true;
    return false;
}

// ---- exchange

struct ExchangeCall {
    int32_t dtype, T, K, H;
    const void *tok, *rows;  // token side and row side, read (NULL: none)
    const int32_t* inv;
    const float* w;
    void* out;
    float* dots;
    bool spread, needs_tok, needs_rows, residual;
};

moe_status exchange(const ExchangeCall& c, void* stream) {
    const int b = elem_size(c.dtype);
    if (!b || c.T < 0) return MOE_ERR_INVALID_ARG;
    if (c.K < 1 || c.K > 8 || c.H < 1 || c.H > 65536 || (int64_t)c.T * c.K > kMaxRows) return MOE_ERR_UNSUPPORTED_SHAPE;
    if (c.T == 0) return MOE_OK;
    if ((c.needs_tok && !c.tok) || (c.needs_rows && !c.rows) || !c.inv || !c.out) return MOE_ERR_INVALID_ARG;
    if (any_misaligned({c.tok, c.rows, c.inv, c.w, c.out, c.dots})) return MOE_ERR_MISALIGNED;
    const size_t tok = (size_t)c.T * c.H * b, rows = tok * c.K, pairs = (size_t)c.T * c.K * 4;
    const Buf results[2] = {{c.out, c.spread ? rows : tok}, {c.dots, pairs}};
    const Buf others[4] = {{c.tok, tok}, {c.rows, rows}, {c.inv, pairs}, {c.w, pairs}};
    if (overlaps(results, others, {c.residual ? 1u : 0u, 0u})) return MOE_ERR_INVALID_ARG;
    ExchangeArgs a = {};
    a.tok = c.tok;
    a.rows = c.rows;
    a.inv = c.inv;
    a.w = c.w;
    a.out = c.out;
    a.dots = c.dots;
    a.T = c.T; a.K = c.K; a.H = c.H;
    a.num_sms = device_sms();
    return to_status(c.spread ? launch_spread(c.dtype, a, (cudaStream_t)stream) : launch_gather(c.dtype, a, (cudaStream_t)stream));
}

// ---- linear layers

bool linear_known(const moe_linear_dims* d) {
    return d && (d->dtype == MOE_BF16 || d->dtype == MOE_FP16) && d->act >= MOE_ACT_NONE && d->act <= MOE_ACT_SWIGLU && d->T >= 0;
}
bool linear_shape(const moe_linear_dims& d) {
    const int64_t most = (int64_t)1 << 40;
    return d.T <= kMaxRows && d.N >= 1 && d.N <= 1 << 20 && d.K >= 8 && d.K <= 1 << 20 && d.K % 8 == 0 && d.E >= 1 && d.E <= 256 &&
           !(d.act == MOE_ACT_SWIGLU && d.N % 32) && (int64_t)d.T * d.N < most && (int64_t)d.T * d.K < most && (int64_t)d.N * d.K < most / d.E;
}
size_t dz_bytes(const moe_linear_dims& d) { return align256((size_t)d.T * ((d.N + 7) / 8 * 8) * 2); }
size_t part_bytes(const moe_linear_dims& d) {
    const size_t rows = dz_rows(d.T, d.E);
    return align256(((d.T + rows - 1) / rows + d.E) * d.N * 4);
}

}  // namespace

extern "C" moe_status moe_sort_pairs(int32_t T, int32_t K, int32_t E, const int32_t* ids, int32_t* counts, int32_t* offsets,
                                     int32_t* perm, int32_t* inv, void* stream) {
    if (T < 0) return MOE_ERR_INVALID_ARG;
    if (K < 1 || K > 8 || E < 1 || E > 256 || (int64_t)T * K > kMaxRows) return MOE_ERR_UNSUPPORTED_SHAPE;
    if (!counts || !offsets || (T && (!ids || !perm || !inv))) return MOE_ERR_INVALID_ARG;
    if (any_misaligned({ids, counts, offsets, perm, inv})) return MOE_ERR_MISALIGNED;
    const size_t pairs = (size_t)T * K * 4;
    const Buf results[4] = {{counts, (size_t)E * 4}, {offsets, (size_t)(E + 1) * 4}, {perm, pairs}, {inv, pairs}};
    if (overlaps(results, {{ids, pairs}}, {0u, 0u, 0u, 0u})) return MOE_ERR_INVALID_ARG;
    return to_status(launch_sort_pairs(ids, counts, offsets, perm, inv, T * K, E, (cudaStream_t)stream));
}

extern "C" moe_status moe_dispatch(int32_t dtype, int32_t T, int32_t K, int32_t H, const void* x, const int32_t* inv,
                                   const float* topk_w, void* rows, void* stream) {
    return exchange({dtype, T, K, H, x, nullptr, inv, topk_w, rows, nullptr, true, true, false, false}, stream);
}

extern "C" moe_status moe_dispatch_backward(int32_t dtype, int32_t T, int32_t K, int32_t H, const void* drows, const int32_t* inv,
                                            const float* topk_w, const void* x, void* dx, float* dtopk_w, void* stream) {
    return exchange({dtype, T, K, H, dtopk_w ? x : nullptr, drows, inv, topk_w, dx, dtopk_w, false, dtopk_w != nullptr, true, false}, stream);
}

extern "C" moe_status moe_combine(int32_t dtype, int32_t T, int32_t K, int32_t H, const void* rows, const int32_t* inv,
                                  const float* topk_w, const void* residual, void* out, void* stream) {
    return exchange({dtype, T, K, H, residual, rows, inv, topk_w, out, nullptr, false, false, true, true}, stream);
}

extern "C" moe_status moe_combine_backward(int32_t dtype, int32_t T, int32_t K, int32_t H, const void* dout, const int32_t* inv,
                                           const float* topk_w, const void* rows, void* drows, float* dtopk_w, void* stream) {
    return exchange({dtype, T, K, H, dout, dtopk_w ? rows : nullptr, inv, topk_w, drows, dtopk_w, true, true, dtopk_w != nullptr, false}, stream);
}

extern "C" size_t moe_linear_workspace_size(const moe_linear_dims* d, int32_t backward) {
    if (!linear_known(d) || !linear_shape(*d)) return 0;
    return align256(sizeof(WsHeader)) + (backward ? dz_bytes(*d) + part_bytes(*d) : 0);
}

extern "C" moe_status moe_linear(const moe_linear_dims* d, const void* x, const void* w, const void* bias, const int32_t* offsets,
                                 const void* residual, void* out, void* z, void* workspace, size_t ws_bytes, void* stream) {
    if (!linear_known(d)) return MOE_ERR_INVALID_ARG;
    if (!linear_shape(*d)) return MOE_ERR_UNSUPPORTED_SHAPE;
    if (d->T == 0) return MOE_OK;
    if (!x || !w || !out || !workspace || (d->E > 1 && !offsets)) return MOE_ERR_INVALID_ARG;
    if (any_misaligned({x, w, residual, out, z, workspace}) || ((uintptr_t)bias & 1u) || ((uintptr_t)offsets & 3u)) return MOE_ERR_MISALIGNED;
    if (ws_bytes < moe_linear_workspace_size(d, 0)) return MOE_ERR_WORKSPACE_TOO_SMALL;
    const size_t T = d->T, No = d->act == MOE_ACT_SWIGLU ? d->N / 2 : d->N;
    const Buf results[3] = {{out, T * No * 2}, {z, T * d->N * 2}, {workspace, sizeof(WsHeader)}};
    const Buf others[5] = {{residual, T * No * 2}, {x, T * d->K * 2}, {w, (size_t)d->E * d->N * d->K * 2}, {bias, (size_t)d->E * d->N * 2}, {offsets, (size_t)(d->E + 1) * 4}};
    if (overlaps(results, others, {1u, 0u, 0u})) return MOE_ERR_INVALID_ARG;
    LinearArgs a = {};
    a.d = *d;
    a.x = x; a.w = w; a.bias = bias; a.offsets = offsets; a.residual = residual;
    a.out = out; a.z = z;
    a.err = &((WsHeader*)workspace)->err;
    a.wait_ns = device_wait_ns();
    a.suppress = device_suppress() == MOE_TEST_SUPPRESS_STAGE;
    a.num_sms = device_sms();
    return to_status(launch_linear(a, (cudaStream_t)stream));
}

extern "C" moe_status moe_linear_backward(const moe_linear_dims* d, const void* x, const void* w, const int32_t* offsets, const void* z,
                                          const void* dout, void* dx, void* dw, void* dbias, void* workspace, size_t ws_bytes, void* stream) {
    if (!linear_known(d)) return MOE_ERR_INVALID_ARG;
    if (!linear_shape(*d)) return MOE_ERR_UNSUPPORTED_SHAPE;
    cudaStream_t s = (cudaStream_t)stream;
    const size_t T = d->T, No = d->act == MOE_ACT_SWIGLU ? d->N / 2 : d->N, wb = (size_t)d->E * d->N * d->K * 2, bb = (size_t)d->E * d->N * 2;
    if (any_misaligned({x, w, z, dout, dx, dw, workspace}) || ((uintptr_t)dbias & 1u) || ((uintptr_t)offsets & 3u)) return MOE_ERR_MISALIGNED;
    if (T == 0) {
        cudaError_t e = cudaSuccess;
        if (dw) e = cudaMemsetAsync(dw, 0, wb, s);
        if (e == cudaSuccess && dbias) e = cudaMemsetAsync(dbias, 0, bb, s);
        return to_status(e);
    }
    if (!dout || !workspace || (dx && !w) || (dw && !x) || (d->act != MOE_ACT_NONE && !z) || (d->E > 1 && !offsets)) return MOE_ERR_INVALID_ARG;
    if (ws_bytes < moe_linear_workspace_size(d, 1)) return MOE_ERR_WORKSPACE_TOO_SMALL;
    const Buf results[4] = {{dx, T * d->K * 2}, {dw, wb}, {dbias, bb}, {workspace, moe_linear_workspace_size(d, 1)}};
    const Buf others[5] = {{dout, T * No * 2}, {z, T * d->N * 2}, {x, T * d->K * 2}, {w, wb}, {offsets, (size_t)(d->E + 1) * 4}};
    if (overlaps(results, others, {0u, 0u, 0u, 0u})) return MOE_ERR_INVALID_ARG;
    LinearArgs a = {};
    a.d = *d;
    a.x = x; a.w = w; a.offsets = offsets;
    a.z_in = z; a.dout = dout;
    a.dx = dx; a.dw = dw; a.dbias = dbias;
    char* base = (char*)workspace;
    a.err = &((WsHeader*)workspace)->err;
    a.dz = base + align256(sizeof(WsHeader));
    a.part = (float*)(base + align256(sizeof(WsHeader)) + dz_bytes(*d));
    a.wait_ns = device_wait_ns();
    a.num_sms = device_sms();
    return to_status(launch_linear_backward(a, s));
}

// ---- norms

namespace {

bool norm_known(const moe_norm_dims* d) {
    return d && elem_size(d->dtype) && d->gate >= MOE_GATE_NONE && d->gate <= MOE_GATE_FULL &&
           (d->gate_act == MOE_ACT_NONE || ((d->gate_act == MOE_ACT_SIGMOID || d->gate_act == MOE_ACT_SILU) && d->gate != MOE_GATE_NONE)) &&
           !(d->flags & ~MOE_NORM_POST) && d->T >= 0 && d->eps >= 0.f && d->eps < 3.4e38f;
}
// (T + a step of the kernels' rows stays within 32 bits)
bool norm_shape(const moe_norm_dims& d) { return d.H >= 1 && d.H <= 8192 && d.T <= kMaxRows; }
size_t gate_bytes(const moe_norm_dims& d) {
    const size_t b = elem_size(d.dtype);
    return d.gate == MOE_GATE_TOKEN ? d.T * b : d.gate == MOE_GATE_CHANNEL ? d.H * b : d.gate == MOE_GATE_FULL ? (size_t)d.T * d.H * b : 0;
}

}  // namespace

extern "C" size_t moe_norm_workspace_size(const moe_norm_dims* d) {
    if (!norm_known(d) || !norm_shape(*d)) return 0;
    return align256((size_t)norm_blocks(d->T > 0 ? d->T : 1) * 3 * d->H * 4);
}

extern "C" moe_status moe_norm_residual(const moe_norm_dims* d, const void* y, const void* residual, const void* gate,
                                        const void* gamma_post, const void* gamma_pre, void* s, void* xn, void* stream) {
    if (!norm_known(d)) return MOE_ERR_INVALID_ARG;
    if (!norm_shape(*d)) return MOE_ERR_UNSUPPORTED_SHAPE;
    if (d->T == 0) return MOE_OK;
    if (!y || (!s && !xn) || (d->gate != MOE_GATE_NONE) != (gate != nullptr) || (gamma_post && !(d->flags & MOE_NORM_POST)))
        return MOE_ERR_INVALID_ARG;
    if (any_misaligned({y, residual, gate, gamma_post, gamma_pre, s, xn})) return MOE_ERR_MISALIGNED;
    const size_t b = elem_size(d->dtype), n = (size_t)d->T * d->H * b, h = d->H * b;
    const Buf results[2] = {{s, n}, {xn, n}};
    const Buf others[5] = {{y, n}, {residual, n}, {gate, gate_bytes(*d)}, {gamma_post, h}, {gamma_pre, h}};
    // (a whole gate [T, H] is no tensor of the stream: never a result's buffer)
    if (overlaps(results, others, {3u, 3u})) return MOE_ERR_INVALID_ARG;
    NormArgs a = {};
    a.d = *d;
    a.y = y; a.residual = residual; a.gate = gate; a.gamma_post = gamma_post; a.gamma_pre = gamma_pre;
    a.s = s; a.xn = xn;
    a.num_sms = device_sms();
    return to_status(launch_norm(a, (cudaStream_t)stream, false));
}

extern "C" moe_status moe_norm_residual_backward(const moe_norm_dims* d, const void* ds, const void* dxn, const void* s,
                                                 const void* y, const void* gate, const void* gamma_post, const void* gamma_pre,
                                                 void* dresidual, void* dy, void* dgate, void* dgamma_post, void* dgamma_pre,
                                                 void* workspace, size_t ws_bytes, void* stream) {
    if (!norm_known(d)) return MOE_ERR_INVALID_ARG;
    if (!norm_shape(*d)) return MOE_ERR_UNSUPPORTED_SHAPE;
    const size_t b = elem_size(d->dtype), n = (size_t)d->T * d->H * b, h = d->H * b;
    const bool post = (d->flags & MOE_NORM_POST) != 0;
    if ((dgamma_post && !post) || (gamma_post && !post) || (dgate && d->gate == MOE_GATE_NONE)) return MOE_ERR_INVALID_ARG;
    if (any_misaligned({ds, dxn, s, y, gate, gamma_post, gamma_pre, dresidual, dy, dgate, dgamma_post, dgamma_pre, workspace})) return MOE_ERR_MISALIGNED;
    if (d->T == 0) {
        cudaError_t e = cudaSuccess;
        cudaStream_t st = (cudaStream_t)stream;
        if (dgamma_post) e = cudaMemsetAsync(dgamma_post, 0, h, st);
        if (e == cudaSuccess && dgamma_pre) e = cudaMemsetAsync(dgamma_pre, 0, h, st);
        if (e == cudaSuccess && dgate && d->gate == MOE_GATE_CHANNEL) e = cudaMemsetAsync(dgate, 0, h, st);
        return to_status(e);
    }
    if (!y || !workspace || (!ds && !dxn) || (dxn && !s) || (d->gate != MOE_GATE_NONE) != (gate != nullptr) || (dgamma_pre && !dxn))
        return MOE_ERR_INVALID_ARG;
    if (ws_bytes < moe_norm_workspace_size(d)) return MOE_ERR_WORKSPACE_TOO_SMALL;
    const Buf results[6] = {{dresidual, n}, {dy, n}, {dgate, gate_bytes(*d)}, {dgamma_post, h}, {dgamma_pre, h}, {workspace, moe_norm_workspace_size(d)}};
    const Buf others[7] = {{ds, n}, {dxn, n}, {s, n}, {y, n}, {gate, gate_bytes(*d)}, {gamma_post, h}, {gamma_pre, h}};
    if (overlaps(results, others, {15u, 15u, 0u, 0u, 0u, 0u})) return MOE_ERR_INVALID_ARG;
    NormArgs a = {};
    a.d = *d;
    a.ds = ds; a.dxn = dxn; a.s_in = s; a.y = y; a.gate = gate; a.gamma_post = gamma_post; a.gamma_pre = gamma_pre;
    a.dresidual = dresidual; a.dy = dy; a.dgate = dgate; a.dgamma_post = dgamma_post; a.dgamma_pre = dgamma_pre;
    a.part = (float*)workspace;
    a.num_sms = device_sms();
    return to_status(launch_norm(a, (cudaStream_t)stream, true));
}
