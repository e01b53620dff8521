// norm.cu -- the norms on both sides of a block, with its gate and the residual sum between them.
//
//   n    = N(y; gamma_post)  (or y)             N(v; g) = v * rsqrt(mean(v^2) + eps) * g
//   s    = residual_scale * residual + branch_scale * act(gate) * n
//   xn   = N(s; gamma_pre)                      from s before its rounding
// and the gradients of all of it. Bound by HBM: each tensor is read or written once, a row stays in
// registers between its two sums. Everything is computed in fp32 and rounded once where it is stored.
//
// Backward, for g_s = ds + (gradient through xn), r = rsqrt(mean(v^2) + eps) of each norm:
//   g_s  = ds + r_s * (dxn * gamma_pre) - s * r_s^3 * mean(dxn * gamma_pre * s)
//   dn   = branch_scale * act(gate) * g_s
//   dy   = r_y * (dn * gamma_post) - y * r_y^3 * mean(dn * gamma_post * y)
// so a row takes two rounds of sums: (s^2, y^2, dxn gamma_pre s), then (dn gamma_post y, the token
// gate's gradient). Sums over tokens (gammas, a channel gate) stay in the registers of the thread that
// owns the columns while its CTA walks its rows; each CTA writes one row of partial sums and a second
// kernel adds those in a fixed order, so gradients are the same bits on every call.
#include "ops.cuh"

namespace moe {

__device__ __forceinline__ float sigmoid(float v) { return 1.0f / (1.0f + expf(-v)); }

// act(gate) and its slope.
__device__ __forceinline__ float gate_value(int act, float g) {
    if (act == MOE_ACT_NONE) return g;
    const float p = sigmoid(g);
    return act == MOE_ACT_SIGMOID ? p : g * p;
}
__device__ __forceinline__ void gate_both(int act, float g, float& a, float& slope) {
    a = g;
    slope = 1.f;
    if (act != MOE_ACT_NONE) {
        const float p = sigmoid(g);
        a = act == MOE_ACT_SIGMOID ? p : g * p;
        slope = act == MOE_ACT_SIGMOID ? p * (1.f - p) : p * (1.f + g * (1.f - p));
    }
}

// Sums over the CTA of N values; buf is used by one call of a row only.
template <int N>
__device__ __forceinline__ void block_sum(float (&v)[N], float (*buf)[16]) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = warp_sum(v[i]);
    if (warps == 1) return;
    if (lane == 0)
#pragma unroll
        for (int i = 0; i < N; ++i) buf[i][warp] = v[i];
    __syncthreads();
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = warp_sum(lane < warps ? buf[i][lane] : 0.f);
}

template <typename T, int VE, int VPT>
__global__ void __launch_bounds__(512) k_norm(const NormArgs a) {
    typedef Vec<T, VE> V;
    __shared__ float buf[2][1][16];
    grid_dep_wait();
    grid_dep_launch();
    const moe_norm_dims& d = a.d;
    const int nv = d.H / VE;
    const int64_t row = (int64_t)blockIdx.x * nv;
    const V* py = reinterpret_cast<const V*>(a.y) + row;
    const V* pr = reinterpret_cast<const V*>(a.residual) + row;
    const V* pg = reinterpret_cast<const V*>(a.gate) + (d.gate == MOE_GATE_FULL ? row : 0);
    const bool per_column = d.gate == MOE_GATE_FULL || d.gate == MOE_GATE_CHANNEL;
    V y[VPT], r[VPT], g[VPT];
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        const int j = threadIdx.x + i * blockDim.x;
        if (j < nv) {
            y[i] = py[j];
            if (a.residual) r[i] = pr[j];
            if (per_column) g[i] = pg[j];
        }
    }
    float scale = d.branch_scale;  // of the whole row's branch
    if (d.gate == MOE_GATE_TOKEN) scale *= gate_value(d.gate_act, to_f(reinterpret_cast<const T*>(a.gate)[blockIdx.x]));
    if (d.flags & MOE_NORM_POST) {
        float sq[1] = {0.f};
#pragma unroll
        for (int i = 0; i < VPT; ++i)
            if (threadIdx.x + i * blockDim.x < nv)
#pragma unroll
                for (int e = 0; e < VE; ++e) sq[0] = fmaf(to_f(y[i].v[e]), to_f(y[i].v[e]), sq[0]);
        block_sum<1>(sq, buf[0]);
        scale *= rsqrtf(sq[0] / (float)d.H + d.eps);
    }
    const V* gp = (d.flags & MOE_NORM_POST) ? reinterpret_cast<const V*>(a.gamma_post) : nullptr;
    V* ps = reinterpret_cast<V*>(a.s) + row;
    float s[VPT][VE];
    float sq[1] = {0.f};
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        const int j = threadIdx.x + i * blockDim.x;
        if (j < nv) {
            V gm = {}, o;
            if (gp) gm = gp[j];
#pragma unroll
            for (int e = 0; e < VE; ++e) {
                float b = scale * to_f(y[i].v[e]);
                if (gp) b *= to_f(gm.v[e]);
                if (per_column) b *= gate_value(d.gate_act, to_f(g[i].v[e]));
                s[i][e] = a.residual ? fmaf(d.residual_scale, to_f(r[i].v[e]), b) : b;
                sq[0] = fmaf(s[i][e], s[i][e], sq[0]);
                o.v[e] = from_f<T>(s[i][e]);
            }
            if (a.s) ps[j] = o;
        }
    }
    if (!a.xn) return;
    block_sum<1>(sq, buf[1]);
    const float rs = rsqrtf(sq[0] / (float)d.H + d.eps);
    const V* gq = reinterpret_cast<const V*>(a.gamma_pre);
    V* px = reinterpret_cast<V*>(a.xn) + row;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        const int j = threadIdx.x + i * blockDim.x;
        if (j < nv) {
            V gm = {}, o;
            if (gq) gm = gq[j];
#pragma unroll
            for (int e = 0; e < VE; ++e) {
                float v = s[i][e] * rs;
                if (gq) v *= to_f(gm.v[e]);
                o.v[e] = from_f<T>(v);
            }
            px[j] = o;
        }
    }
}

template <typename T, int VE, int VPT>
__global__ void __launch_bounds__(512) k_norm_backward(const NormArgs a) {
    typedef Vec<T, VE> V;
    __shared__ float buf[2][2][3][16];
    grid_dep_wait();
    grid_dep_launch();
    const moe_norm_dims& d = a.d;
    const int nv = d.H / VE;
    const bool post = (d.flags & MOE_NORM_POST) != 0, pre = a.dxn != nullptr;
    const bool full = d.gate == MOE_GATE_FULL, channel = d.gate == MOE_GATE_CHANNEL, token = d.gate == MOE_GATE_TOKEN;
    float acc_post[VPT][VE], acc_pre[VPT][VE], acc_gate[VPT][VE];
#pragma unroll
    for (int i = 0; i < VPT; ++i)
#pragma unroll
        for (int e = 0; e < VE; ++e) acc_post[i][e] = acc_pre[i][e] = acc_gate[i][e] = 0.f;
    V gp[VPT], gq[VPT];
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        const int j = threadIdx.x + i * blockDim.x;
#pragma unroll
        for (int e = 0; e < VE; ++e) gp[i].v[e] = gq[i].v[e] = from_f<T>(1.f);
        if (j < nv) {
            if (post && a.gamma_post) gp[i] = reinterpret_cast<const V*>(a.gamma_post)[j];
            if (pre && a.gamma_pre) gq[i] = reinterpret_cast<const V*>(a.gamma_pre)[j];
        }
    }
    const float inv_h = 1.0f / (float)d.H;
    int turn = 0;
    for (int t = blockIdx.x; t < d.T; t += gridDim.x, turn ^= 1) {
        const int64_t row = (int64_t)t * nv;
        V y[VPT], s[VPT], ds[VPT], dx[VPT], g[VPT];
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int j = threadIdx.x + i * blockDim.x;
            if (j < nv) {
                y[i] = reinterpret_cast<const V*>(a.y)[row + j];
                if (pre) {
                    s[i] = reinterpret_cast<const V*>(a.s_in)[row + j];
                    dx[i] = reinterpret_cast<const V*>(a.dxn)[row + j];
                }
                if (a.ds) ds[i] = reinterpret_cast<const V*>(a.ds)[row + j];
                if (full || channel) g[i] = reinterpret_cast<const V*>(a.gate)[(full ? row : 0) + j];
            }
        }
        float sums[3] = {0.f, 0.f, 0.f};  // s^2, y^2, dxn gamma_pre s
#pragma unroll
        for (int i = 0; i < VPT; ++i)
            if (threadIdx.x + i * blockDim.x < nv)
#pragma unroll
                for (int e = 0; e < VE; ++e) {
                    if (post) sums[1] = fmaf(to_f(y[i].v[e]), to_f(y[i].v[e]), sums[1]);
                    if (pre) {
                        sums[0] = fmaf(to_f(s[i].v[e]), to_f(s[i].v[e]), sums[0]);
                        sums[2] = fmaf(to_f(dx[i].v[e]) * to_f(gq[i].v[e]), to_f(s[i].v[e]), sums[2]);
                    }
                }
        if (post || pre) block_sum<3>(sums, buf[turn][0]);
        const float rs = pre ? rsqrtf(sums[0] * inv_h + d.eps) : 0.f;
        const float ry = post ? rsqrtf(sums[1] * inv_h + d.eps) : 1.f;
        const float cs = pre ? rs * rs * rs * (sums[2] * inv_h) : 0.f;
        float tval = 1.f, tslope = 0.f;
        if (token) gate_both(d.gate_act, to_f(reinterpret_cast<const T*>(a.gate)[t]), tval, tslope);
        float gs[VPT][VE];
        float more[2] = {0.f, 0.f};  // dn gamma_post y, g_s n
#pragma unroll
        for (int i = 0; i < VPT; ++i)
            if (threadIdx.x + i * blockDim.x < nv)
#pragma unroll
                for (int e = 0; e < VE; ++e) {
                    float v = a.ds ? to_f(ds[i].v[e]) : 0.f;
                    if (pre) {
                        const float q = to_f(dx[i].v[e]), sv = to_f(s[i].v[e]);
                        v += rs * (q * to_f(gq[i].v[e])) - sv * cs;
                        acc_pre[i][e] = fmaf(q * sv, rs, acc_pre[i][e]);
                    }
                    gs[i][e] = v;
                    const float yv = to_f(y[i].v[e]), ga = to_f(gp[i].v[e]);
                    const float n = yv * ry * ga;  // (gamma_post is 1 and r_y is 1 without the norm)
                    float av = tval, slope = 0.f;
                    if (full || channel) gate_both(d.gate_act, to_f(g[i].v[e]), av, slope);
                    const float dn = d.branch_scale * av * v;
                    if (channel) acc_gate[i][e] = fmaf(d.branch_scale * v * n, slope, acc_gate[i][e]);
                    if (post) {
                        more[0] = fmaf(dn * ga, yv, more[0]);
                        acc_post[i][e] = fmaf(dn * yv, ry, acc_post[i][e]);
                    }
                    if (token) more[1] = fmaf(v, n, more[1]);
                }
        if (post || token) block_sum<2>(more, buf[turn][1]);
        if (token && a.dgate && threadIdx.x == 0) reinterpret_cast<T*>(a.dgate)[t] = from_f<T>(d.branch_scale * more[1] * tslope);
        const float cy = post ? ry * ry * ry * (more[0] * inv_h) : 0.f;
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int j = threadIdx.x + i * blockDim.x;
            if (j < nv) {
                V o1, o2, o3;
#pragma unroll
                for (int e = 0; e < VE; ++e) {
                    const float yv = to_f(y[i].v[e]), ga = to_f(gp[i].v[e]);
                    float av = tval, slope = 0.f;
                    if (full || channel) gate_both(d.gate_act, to_f(g[i].v[e]), av, slope);
                    const float dn = d.branch_scale * av * gs[i][e];
                    o1.v[e] = from_f<T>(d.residual_scale * gs[i][e]);
                    o2.v[e] = from_f<T>(post ? ry * (dn * ga) - yv * cy : dn);
                    if (full) o3.v[e] = from_f<T>(d.branch_scale * gs[i][e] * (yv * ry * ga) * slope);
                }
                if (a.dresidual) reinterpret_cast<V*>(a.dresidual)[row + j] = o1;
                if (a.dy) reinterpret_cast<V*>(a.dy)[row + j] = o2;
                if (full && a.dgate) reinterpret_cast<V*>(a.dgate)[row + j] = o3;
            }
        }
    }
    if (!a.part) return;
    float* part = a.part + (int64_t)blockIdx.x * 3 * d.H;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        const int j = threadIdx.x + i * blockDim.x;
        if (j < nv)
#pragma unroll
            for (int e = 0; e < VE; ++e) {
                const int h = j * VE + e;
                if (a.dgamma_post) part[h] = acc_post[i][e];
                if (a.dgamma_pre) part[d.H + h] = acc_pre[i][e];
                if (channel && a.dgate) part[2 * d.H + h] = acc_gate[i][e];
            }
    }
}

// Column sums of the row blocks' partial sums: 32 columns a CTA, eight threads a column, each an
// eighth of the blocks in order, then the eight in order.
template <typename T>
__global__ void __launch_bounds__(256) k_norm_columns(const NormArgs a, int blocks) {
    __shared__ float sm[8][33];
    grid_dep_wait();
    grid_dep_launch();
    const int which = blockIdx.y, h = blockIdx.x * 32 + threadIdx.x % 32, q = threadIdx.x / 32;
    T* out = reinterpret_cast<T*>(which == 0 ? a.dgamma_post : which == 1 ? a.dgamma_pre : a.d.gate == MOE_GATE_CHANNEL ? a.dgate : nullptr);
    if (!out) return;
    float v = 0.f;
    if (h < a.d.H) {
        const float* p = a.part + (int64_t)which * a.d.H + h;
        const int per = (blocks + 7) / 8, b1 = min(blocks, (q + 1) * per);
#pragma unroll 8
        for (int b = q * per; b < b1; ++b) v += p[(int64_t)b * 3 * a.d.H];
    }
    sm[q][threadIdx.x % 32] = v;
    __syncthreads();
    if (q == 0 && h < a.d.H) {
        v = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) v += sm[i][threadIdx.x];
        out[h] = from_f<T>(v);
    }
}

// Threads for a row and vectors for a thread: 512 threads at most, the fewest vectors that then cover the row.
static int norm_vpt(int nv) {
    int vpt = 1;
    while (vpt * 512 < nv) vpt *= 2;
    return vpt;
}
static int norm_threads(int nv, int vpt) { return max(32, ((nv + vpt - 1) / vpt + 31) / 32 * 32); }

template <typename T, int VE, int VPT>
static cudaError_t launch_norm_t(const NormArgs& a, cudaStream_t s, bool backward) {
    const int threads = norm_threads(a.d.H / VE, VPT);
    cudaError_t e;
    if (!backward) {
        MOE_LAUNCH(MOE_KERNEL_NORM, s, (e = launch_pdl(k_norm<T, VE, VPT>, dim3(a.d.T), dim3(threads), 0, s, a)));
        return e;
    }
    const int blocks = min(a.d.T, kNormBlocks);
    NormArgs b = a;
    const bool columns = a.dgamma_post || a.dgamma_pre || (a.dgate && a.d.gate == MOE_GATE_CHANNEL);
    if (!columns) b.part = nullptr;
    MOE_LAUNCH(MOE_KERNEL_NORM_BACKWARD, s, (e = launch_pdl(k_norm_backward<T, VE, VPT>, dim3(blocks), dim3(threads), 0, s, b)));
    if (e == cudaSuccess && columns)
        MOE_LAUNCH(MOE_KERNEL_NORM_BACKWARD, s, (e = launch_pdl(k_norm_columns<T>, dim3((a.d.H + 31) / 32, 3), dim3(256), 0, s, b, blocks)));
    return e;
}

template <typename T>
static cudaError_t launch_norm_any(const NormArgs& a, cudaStream_t s, bool backward) {
    constexpr int VE = 16 / (int)sizeof(T);
    if (a.d.H % VE == 0) {
        switch (norm_vpt(a.d.H / VE)) {
            case 1: return launch_norm_t<T, VE, 1>(a, s, backward);
            case 2: return launch_norm_t<T, VE, 2>(a, s, backward);
            case 4: if constexpr (VE == 4) return launch_norm_t<T, VE, 4>(a, s, backward); break;  // (H <= 8192)
        }
        return cudaErrorInvalidValue;
    }
    switch (norm_vpt(a.d.H)) {
        case 1: return launch_norm_t<T, 1, 1>(a, s, backward);
        case 2: return launch_norm_t<T, 1, 2>(a, s, backward);
        case 4: return launch_norm_t<T, 1, 4>(a, s, backward);
        case 8: return launch_norm_t<T, 1, 8>(a, s, backward);
        case 16: return launch_norm_t<T, 1, 16>(a, s, backward);
    }
    return cudaErrorInvalidValue;
}

static cudaError_t launch_norm_dtype(const NormArgs& a, cudaStream_t s, bool backward) {
    switch (a.d.dtype) {
        case MOE_BF16: return launch_norm_any<bf16>(a, s, backward);
        case MOE_FP16: return launch_norm_any<fp16>(a, s, backward);
        default: return launch_norm_any<float>(a, s, backward);
    }
}

cudaError_t launch_norm(const NormArgs& a, cudaStream_t s) { return launch_norm_dtype(a, s, false); }
cudaError_t launch_norm_backward(const NormArgs& a, cudaStream_t s) { return launch_norm_dtype(a, s, true); }

}  // namespace moe
