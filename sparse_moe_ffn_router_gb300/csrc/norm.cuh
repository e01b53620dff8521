// norm.cuh -- the norms on both sides of a block, with its gate and the residual sum between them.
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
// owns the columns while it walks its rows; each CTA writes one row of partial sums and a second
// kernel adds those in a fixed order, so gradients are the same bits on every call.
//
// A CTA is one or more groups of threads with a row each at a time (a warp where 32 vectors of 16 bytes cover the row),
// synchronised by a barrier of their own; a group loads its next row before it works on the current one, which
// is what keeps HBM busy across the two sums. A thread's 16-byte vectors are aligned in memory whatever the row
// length: the rows of a group all begin at the same place within a vector (their numbers are equal mod 8), so its columns
// stay the same from row to row, and only a row's first and last vector are moved element by element.
//
// Measured (graph replay): forward 4096 x 2048 bf16 14.3 us = 4.7 TB/s, with a whole sigmoid gate 16.7 us = 5.0 TB/s (issue slots 73 %);
// backward 4096 x 2048 36 us = 2.8 TB/s: about 660 instructions a warp and row at 0.57 a clock, two rows an SM at once, which
// the 24 column sums a thread hold to; 2051 x 1544 with a channel gate 21 us, 5 of them the second kernel.
#pragma once

#include "ops.cuh"

namespace moe {

constexpr int kNormThreads = 512;
enum { kGateRow = 0, kGateColumn = 1, kGateAll = 2 };  // none or one number a row; a channel; an element

// Of 16-bit tensors the hardware's exp and quotient do: a few 2^-22 relative against half a step of 2^-12 and up.
template <typename T>
__device__ __forceinline__ float norm_sigmoid(float v) {
    if constexpr (sizeof(T) == 2) return __fdividef(1.0f, 1.0f + __expf(-v));
    else return 1.0f / (1.0f + expf(-v));
}
// g = act(g) of N values, and their slopes.
template <typename T, int N>
__device__ __forceinline__ void gate_values(int act, float (&g)[N]) {
    if (act == MOE_ACT_SIGMOID) {
#pragma unroll
        for (int i = 0; i < N; ++i) g[i] = norm_sigmoid<T>(g[i]);
    } else if (act == MOE_ACT_SILU) {
#pragma unroll
        for (int i = 0; i < N; ++i) g[i] *= norm_sigmoid<T>(g[i]);
    }
}
template <typename T, int N>
__device__ __forceinline__ void gate_slopes(int act, float (&g)[N], float (&slope)[N]) {
    if (act == MOE_ACT_SIGMOID) {
#pragma unroll
        for (int i = 0; i < N; ++i) {
            g[i] = norm_sigmoid<T>(g[i]);
            slope[i] = g[i] * (1.f - g[i]);
        }
    } else if (act == MOE_ACT_SILU) {
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const float p = norm_sigmoid<T>(g[i]);
            slope[i] = p * (1.f + g[i] * (1.f - p));
            g[i] *= p;
        }
    } else {
#pragma unroll
        for (int i = 0; i < N; ++i) slope[i] = 1.f;
    }
}

// Where a thread's group is in its CTA, and the thread in its group.
struct NormGroup {
    int tid, threads, id, groups;  // thread of the group, its threads; group of the CTA, its groups
};
__device__ __forceinline__ NormGroup norm_group(int tpr) {
    NormGroup g;
    g.threads = tpr;
    g.id = threadIdx.x / tpr;
    g.tid = threadIdx.x - g.id * tpr;
    g.groups = blockDim.x / tpr;
    return g;
}

// Sums over the group of N values, the warps' sums in warp order. buf is this sum's alone until the group has
// passed another one.
template <int N>
__device__ __forceinline__ void group_sum(float (&v)[N], float (*buf)[20], const NormGroup& g) {
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = warp_sum(v[i]);
    if (g.threads == 32) return;
    const int warp = g.tid >> 5, warps = g.threads >> 5;
    if ((g.tid & 31) == 0)
#pragma unroll
        for (int i = 0; i < N; ++i) buf[i][warp] = v[i];
    asm volatile("bar.sync %0, %1;" ::"r"(g.id + 1), "r"(g.threads) : "memory");
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = 0.f;
#pragma unroll
    for (int w = 0; w < 20; w += 4)
        if (w < warps) {  // (places past the last warp hold zeros)
#pragma unroll
            for (int i = 0; i < N; ++i) {
                const float4 x = *reinterpret_cast<const float4*>(&buf[i][w]);
                v[i] += (x.x + x.y) + (x.z + x.w);
            }
        }
}

template <typename T>
__device__ __forceinline__ uint32_t bits_of(const T* p) {
    if constexpr (sizeof(T) == 4) return *reinterpret_cast<const uint32_t*>(p);
    else return *reinterpret_cast<const uint16_t*>(p);
}
// Columns [c, c + VE) of a row that begins at p, of which those in [0, H) exist (the others: zeros). whole: all do.
template <typename T, int VE>
__device__ __forceinline__ Raw row_get(const T* p, int c, int H, bool whole) {
    Raw r;
    if (whole) {
        const uint4 v = *reinterpret_cast<const uint4*>(p + c);
        r.w[0] = v.x; r.w[1] = v.y; r.w[2] = v.z; r.w[3] = v.w;
    } else {
        r.w[0] = r.w[1] = r.w[2] = r.w[3] = 0u;
#pragma unroll
        for (int i = 0; i < VE; ++i)
            if ((unsigned)(c + i) < (unsigned)H) r.w[i * 4 / VE] |= bits_of(p + c + i) << (VE == 8 ? 16 * (i & 1) : 0);
    }
    return r;
}
template <typename T, int VE>
__device__ __forceinline__ void row_put(T* p, int c, int H, bool whole, const Raw& r) {
    if (whole) {
        *reinterpret_cast<uint4*>(p + c) = make_uint4(r.w[0], r.w[1], r.w[2], r.w[3]);
    } else {
#pragma unroll
        for (int i = 0; i < VE; ++i)
            if ((unsigned)(c + i) < (unsigned)H) {
                if constexpr (VE == 8) reinterpret_cast<uint16_t*>(p)[c + i] = (uint16_t)(r.w[i >> 1] >> (16 * (i & 1)));
                else reinterpret_cast<uint32_t*>(p)[c + i] = r.w[i];
            }
    }
}

template <typename T, int VE, int VPT, int GATE>
__global__ void __launch_bounds__(kNormThreads, VPT == 1 ? 2 : 1) k_norm(const NormArgs a, int tpr) {
    typedef RawOf<T> R;
    __shared__ __align__(16) float bufs[16][2][2][20];
    grid_dep_wait();
    grid_dep_launch();
    const moe_norm_dims& d = a.d;
    const NormGroup g = norm_group(tpr);
    const int H = d.H, first = blockIdx.x * g.groups + g.id, step = gridDim.x * g.groups;
    constexpr bool full = GATE == kGateAll, channel = GATE == kGateColumn;
    const bool post = (d.flags & MOE_NORM_POST) != 0;
    const int mis = (int)((int64_t)first * H % VE);  // the rows' place within a vector
    int col[VPT];
    bool live[VPT], whole[VPT];
    Raw y[VPT], r[VPT], ga[VPT];
    T tg = from_f<T>(0.f);
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        col[i] = (g.tid + i * g.threads) * VE - mis;
        live[i] = col[i] < H;
        whole[i] = col[i] >= 0 && col[i] + VE <= H;
    }
    auto load = [&](int t) {
        const int64_t row = (int64_t)t * H;
#pragma unroll
        for (int i = 0; i < VPT; ++i)
            if (live[i]) {
                y[i] = row_get<T, VE>((const T*)a.y + row, col[i], H, whole[i]);
                if (a.residual) r[i] = row_get<T, VE>((const T*)a.residual + row, col[i], H, whole[i]);
                if (full) ga[i] = row_get<T, VE>((const T*)a.gate + row, col[i], H, whole[i]);
            }
        if (GATE == kGateRow && d.gate == MOE_GATE_TOKEN) tg = ((const T*)a.gate)[t];
    };
    if (first < d.T) load(first);
    // tensors [H]: in vectors where rows are aligned, else by elements
    const bool aligned = mis == 0 && H % VE == 0;
    Raw gp[VPT], gq[VPT];
    float gc[VPT][VE];  // act(gate) of a channel gate
#pragma unroll
    for (int i = 0; i < VPT; ++i)
        if (live[i]) {
            if (post && a.gamma_post) gp[i] = row_get<T, VE>((const T*)a.gamma_post, col[i], H, aligned);
            if (a.xn && a.gamma_pre) gq[i] = row_get<T, VE>((const T*)a.gamma_pre, col[i], H, aligned);
            if (channel) {
                R::values(row_get<T, VE>((const T*)a.gate, col[i], H, aligned), gc[i]);
                gate_values<T, VE>(d.gate_act, gc[i]);
            }
        }
    for (int i = g.tid; i < 80; i += g.threads) (&bufs[g.id][0][0][0])[i] = 0.f;  // (read past the last warp)
    if (g.threads > 32) asm volatile("bar.sync %0, %1;" ::"r"(g.id + 1), "r"(g.threads) : "memory");
    const float inv_h = 1.0f / (float)H;
    int turn = 0;
    for (int t = first; t < d.T; t += step, turn ^= 1) {
        const int64_t row = (int64_t)t * H;
        float scale = d.branch_scale;  // of the whole row's branch
        if (GATE == kGateRow && d.gate == MOE_GATE_TOKEN) {
            float v[1] = {to_f(tg)};
            gate_values<T, 1>(d.gate_act, v);
            scale *= v[0];
        }
        float s[VPT][VE];  // the branch without the norm's factor, then s
        float sq[1] = {0.f};
        Raw rr[VPT];
#pragma unroll
        for (int i = 0; i < VPT; ++i)
            if (live[i]) {
                float f[VE];
                rr[i] = r[i];
                R::values(y[i], s[i]);
                if (post) {
#pragma unroll
                    for (int e = 0; e < VE; ++e) sq[0] = fmaf(s[i][e], s[i][e], sq[0]);
                    if (a.gamma_post) {
                        R::values(gp[i], f);
#pragma unroll
                        for (int e = 0; e < VE; ++e) s[i][e] *= f[e];
                    }
                }
                if (full) {
                    R::values(ga[i], f);
                    gate_values<T, VE>(d.gate_act, f);
#pragma unroll
                    for (int e = 0; e < VE; ++e) s[i][e] *= f[e];
                }
                if (channel) {
#pragma unroll
                    for (int e = 0; e < VE; ++e) s[i][e] *= gc[i][e];
                }
            }
        if (t + step < d.T) load(t + step);
        if (post) {
            group_sum<1>(sq, &bufs[g.id][turn][0], g);
            scale *= rsqrtf(sq[0] * inv_h + d.eps);
        }
        sq[0] = 0.f;
#pragma unroll
        for (int i = 0; i < VPT; ++i)
            if (live[i]) {
                if (a.residual) {
                    float f[VE];
                    R::values(rr[i], f);
#pragma unroll
                    for (int e = 0; e < VE; ++e) s[i][e] = fmaf(d.residual_scale, f[e], s[i][e] * scale);
                } else {
#pragma unroll
                    for (int e = 0; e < VE; ++e) s[i][e] *= scale;
                }
#pragma unroll
                for (int e = 0; e < VE; ++e) sq[0] = fmaf(s[i][e], s[i][e], sq[0]);
                if (a.s) row_put<T, VE>((T*)a.s + row, col[i], H, whole[i], R::pack(s[i]));
            }
        if (!a.xn) continue;
        group_sum<1>(sq, &bufs[g.id][turn][1], g);
        const float rs = rsqrtf(sq[0] * inv_h + d.eps);
#pragma unroll
        for (int i = 0; i < VPT; ++i)
            if (live[i]) {
#pragma unroll
                for (int e = 0; e < VE; ++e) s[i][e] *= rs;
                if (a.gamma_pre) {
                    float f[VE];
                    R::values(gq[i], f);
#pragma unroll
                    for (int e = 0; e < VE; ++e) s[i][e] *= f[e];
                }
                row_put<T, VE>((T*)a.xn + row, col[i], H, whole[i], R::pack(s[i]));
            }
    }
}

template <typename T, int VE, int VPT, int GATE>
__global__ void __launch_bounds__(kNormThreads, 1) k_norm_backward(const NormArgs a, int tpr) {
    typedef RawOf<T> R;
    __shared__ __align__(16) float bufs[16][2][5][20];
    __shared__ float sums[VPT == 1 ? 3 : 1][VPT == 1 ? 2080 : 1];  // (several groups: rows of 256 vectors at most)
    grid_dep_wait();
    grid_dep_launch();
    const moe_norm_dims& d = a.d;
    const NormGroup g = norm_group(tpr);
    const int H = d.H, first = blockIdx.x * g.groups + g.id, step = gridDim.x * g.groups;
    constexpr bool full = GATE == kGateAll, channel = GATE == kGateColumn;
    const bool post = (d.flags & MOE_NORM_POST) != 0, pre = a.dxn != nullptr;
    const bool token = GATE == kGateRow && d.gate == MOE_GATE_TOKEN;
    const int mis = (int)((int64_t)first * H % VE);
    int col[VPT];
    bool live[VPT], whole[VPT];
    Raw y[VPT], s[VPT], ds[VPT], dx[VPT], ga[VPT];
    T tg = from_f<T>(0.f);
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        col[i] = (g.tid + i * g.threads) * VE - mis;
        live[i] = col[i] < H;
        whole[i] = col[i] >= 0 && col[i] + VE <= H;
        ds[i] = s[i] = dx[i] = Raw{{0u, 0u, 0u, 0u}};  // (of no gradient: zeros)
    }
    auto load = [&](int t) {
        const int64_t row = (int64_t)t * H;
#pragma unroll
        for (int i = 0; i < VPT; ++i)
            if (live[i]) {
                y[i] = row_get<T, VE>((const T*)a.y + row, col[i], H, whole[i]);
                if (pre) {
                    s[i] = row_get<T, VE>((const T*)a.s_in + row, col[i], H, whole[i]);
                    dx[i] = row_get<T, VE>((const T*)a.dxn + row, col[i], H, whole[i]);
                }
                if (a.ds) ds[i] = row_get<T, VE>((const T*)a.ds + row, col[i], H, whole[i]);
                if (full) ga[i] = row_get<T, VE>((const T*)a.gate + row, col[i], H, whole[i]);
            }
        if (token) tg = ((const T*)a.gate)[t];
    };
    if (first < d.T) load(first);
    const bool aligned = mis == 0 && H % VE == 0;
    float acc_post[VPT][VE], acc_pre[VPT][VE], acc_gate[VPT][VE];
    Raw gp[VPT], gq[VPT];
    float gc[VPT][VE];  // act(gate) of a channel gate
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        float one[VE];
#pragma unroll
        for (int e = 0; e < VE; ++e) {
            acc_post[i][e] = acc_pre[i][e] = acc_gate[i][e] = 0.f;
            one[e] = 1.f;
        }
        gp[i] = gq[i] = R::pack(one);
        if (live[i]) {
            if (post && a.gamma_post) gp[i] = row_get<T, VE>((const T*)a.gamma_post, col[i], H, aligned);
            if (pre && a.gamma_pre) gq[i] = row_get<T, VE>((const T*)a.gamma_pre, col[i], H, aligned);
            if (channel) {
                R::values(row_get<T, VE>((const T*)a.gate, col[i], H, aligned), gc[i]);
                gate_values<T, VE>(d.gate_act, gc[i]);
            }
        }
    }
    for (int i = g.tid; i < 200; i += g.threads) (&bufs[g.id][0][0][0])[i] = 0.f;
    if (g.threads > 32) asm volatile("bar.sync %0, %1;" ::"r"(g.id + 1), "r"(g.threads) : "memory");
    const float inv_h = 1.0f / (float)H;
    int turn = 0;
    for (int t = first; t < d.T; t += step, turn ^= 1) {
        const int64_t row = (int64_t)t * H;
        float sm[3] = {0.f, 0.f, 0.f};  // s^2, y^2, dxn gamma_pre s
#pragma unroll
        for (int i = 0; i < VPT; ++i)
            if (live[i]) {
                float yv[VE], sv[VE], q[VE], gm[VE];
                R::values(y[i], yv);
                R::values(s[i], sv);
                R::values(dx[i], q);
                R::values(gq[i], gm);
#pragma unroll
                for (int e = 0; e < VE; ++e) {
                    sm[0] = fmaf(sv[e], sv[e], sm[0]);
                    sm[1] = fmaf(yv[e], yv[e], sm[1]);
                    sm[2] = fmaf(q[e] * gm[e], sv[e], sm[2]);
                }
            }
        if (post || pre) group_sum<3>(sm, &bufs[g.id][turn][0], g);
        const float rs = pre ? rsqrtf(sm[0] * inv_h + d.eps) : 0.f;
        const float ry = post ? rsqrtf(sm[1] * inv_h + d.eps) : 1.f;
        const float cs = pre ? rs * (rs * (sm[2] * inv_h)) : 0.f;  // (r^3 by itself may leave fp32's range)
        float tval[1] = {1.f}, tslope[1] = {0.f};
        if (token) {
            tval[0] = to_f(tg);
            gate_slopes<T, 1>(d.gate_act, tval, tslope);
        }
        const float branch = d.branch_scale * tval[0];
        float gs[VPT][VE];  // dn gamma_post
        Raw yy[VPT];
        float more[2] = {0.f, 0.f};  // dn gamma_post y, g_s n
#pragma unroll
        for (int i = 0; i < VPT; ++i)
            if (live[i]) {
                float yv[VE], sv[VE], q[VE], gm[VE], v[VE], o[VE];
                yy[i] = y[i];
                R::values(s[i], sv);
                R::values(dx[i], q);
                R::values(gq[i], gm);
                R::values(ds[i], v);
#pragma unroll
                for (int e = 0; e < VE; ++e) {
                    v[e] = fmaf(rs, fmaf(-sv[e], cs, q[e] * gm[e]), v[e]);
                    acc_pre[i][e] = fmaf(q[e] * sv[e], rs, acc_pre[i][e]);
                    o[e] = d.residual_scale * v[e];
                }
                if (a.dresidual) row_put<T, VE>((T*)a.dresidual + row, col[i], H, whole[i], R::pack(o));
                R::values(y[i], yv);
                R::values(gp[i], gm);
                float ge[VE], slope[VE];
                if (full) {
                    R::values(ga[i], ge);
                    gate_slopes<T, VE>(d.gate_act, ge, slope);
                }
#pragma unroll
                for (int e = 0; e < VE; ++e) {
                    const float yn = yv[e] * ry, n = yn * gm[e];  // (gamma_post is 1 and r_y is 1 without the norm)
                    const float dn = (full ? branch * ge[e] : channel ? branch * gc[i][e] : branch) * v[e];
                    if (channel) acc_gate[i][e] = fmaf(v[e], n, acc_gate[i][e]);  // (branch and slope: once, at the end)
                    if (full) o[e] = branch * v[e] * n * slope[e];
                    if (token) more[1] = fmaf(v[e], n, more[1]);
                    acc_post[i][e] = fmaf(dn, yn, acc_post[i][e]);
                    gs[i][e] = dn * gm[e];
                    more[0] = fmaf(gs[i][e], yv[e], more[0]);
                }
                if (full && a.dgate) row_put<T, VE>((T*)a.dgate + row, col[i], H, whole[i], R::pack(o));
            }
        if (t + step < d.T) load(t + step);
        if (post || token) group_sum<2>(more, &bufs[g.id][turn][3], g);
        if (token && a.dgate && g.tid == 0) ((T*)a.dgate)[t] = from_f<T>(d.branch_scale * more[1] * tslope[0]);
        const float cy = post ? ry * (ry * (more[0] * inv_h)) : 0.f;
        if (a.dy)
#pragma unroll
            for (int i = 0; i < VPT; ++i)
                if (live[i]) {
                    float yv[VE];
                    R::values(yy[i], yv);
#pragma unroll
                    for (int e = 0; e < VE; ++e) yv[e] = post ? ry * fmaf(-yv[e], cy, gs[i][e]) : gs[i][e];
                    row_put<T, VE>((T*)a.dy + row, col[i], H, whole[i], R::pack(yv));
                }
    }
    if (!a.part) return;
    if (channel) {
#pragma unroll
        for (int i = 0; i < VPT; ++i)
            if (live[i]) {
                float ge[VE], slope[VE];
                R::values(row_get<T, VE>((const T*)a.gate, col[i], H, aligned), ge);
                gate_slopes<T, VE>(d.gate_act, ge, slope);
#pragma unroll
                for (int e = 0; e < VE; ++e) acc_gate[i][e] *= d.branch_scale * slope[e];
            }
    }
    float* part = a.part + (int64_t)blockIdx.x * 3 * H;
    if (VPT > 1 || g.groups == 1) {
#pragma unroll
        for (int i = 0; i < VPT; ++i)
#pragma unroll
            for (int e = 0; e < VE; ++e) {
                const int h = col[i] + e;
                if ((unsigned)h < (unsigned)H) {
                    part[h] = acc_post[i][e];
                    part[H + h] = acc_pre[i][e];
                    if (channel) part[2 * H + h] = acc_gate[i][e];
                }
            }
        return;
    }
    // the CTA's groups one after another: a column is another thread's in each
    for (int q = 0; q < g.groups; ++q) {
        if (q == g.id)
#pragma unroll
            for (int e = 0; e < VE; ++e) {
                const int h = col[0] + e;
                if ((unsigned)h < (unsigned)H) {
                    sums[0][h] = q ? sums[0][h] + acc_post[0][e] : acc_post[0][e];
                    sums[VPT == 1 ? 1 : 0][h] = q ? sums[VPT == 1 ? 1 : 0][h] + acc_pre[0][e] : acc_pre[0][e];
                    if (channel) sums[VPT == 1 ? 2 : 0][h] = q ? sums[VPT == 1 ? 2 : 0][h] + acc_gate[0][e] : acc_gate[0][e];
                }
            }
        __syncthreads();
    }
    for (int k = 0; k < (channel ? 3 : 2); ++k)
        for (int i = threadIdx.x; i < H; i += blockDim.x) part[k * H + i] = sums[VPT == 1 ? k : 0][i];
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

// Vectors that cover any row of H columns, wherever in a vector it begins; vectors and threads of a row.
template <typename T, int VE, int VPT, int GATE>
static cudaError_t launch_norm_t(const NormArgs& a, cudaStream_t s, bool backward, int nv) {
    const int tpr = max(32, ((nv + VPT - 1) / VPT + 31) / 32 * 32);
    int groups = VPT == 1 ? max(1, min(16, 512 / tpr)) : 1;
    while (groups > 1 && a.d.T < groups * a.num_sms) groups /= 2;  // (few rows: a CTA each)
    const int per_sm = backward || VPT > 1 ? 1 : 2;
    // rows of a group are equal mod VE
    int blocks = min((a.d.T + groups - 1) / groups, backward ? min(kNormBlocks, a.num_sms) : a.num_sms * per_sm);
    if (a.d.H % VE && blocks * groups % VE) {
        const int up = (blocks + VE - 1) / VE * VE;
        blocks = blocks < a.d.T && up <= kNormBlocks ? up : max(VE, blocks / VE * VE);
    }
    if (backward && blocks > norm_blocks(a.d.T)) return cudaErrorInvalidValue;  // (never: what the workspace holds)
    cudaError_t e;
    if (!backward) {
        MOE_LAUNCH(MOE_KERNEL_NORM, s, (e = launch_pdl(k_norm<T, VE, VPT, GATE>, dim3(blocks), dim3(tpr * groups), 0, s, a, tpr)));
        return e;
    }
    NormArgs b = a;
    const bool columns = a.dgamma_post || a.dgamma_pre || (a.dgate && a.d.gate == MOE_GATE_CHANNEL);
    if (!columns) b.part = nullptr;
    MOE_LAUNCH(MOE_KERNEL_NORM_BACKWARD, s, (e = launch_pdl(k_norm_backward<T, VE, VPT, GATE>, dim3(blocks), dim3(tpr * groups), 0, s, b, tpr)));
    if (e == cudaSuccess && columns)
        MOE_LAUNCH(MOE_KERNEL_NORM_BACKWARD, s, (e = launch_pdl(k_norm_columns<T>, dim3((a.d.H + 31) / 32, 3), dim3(256), 0, s, b, blocks)));
    return e;
}

template <typename T, int VE, int VPT>
static cudaError_t launch_norm_g(const NormArgs& a, cudaStream_t s, bool backward, int nv) {
    return a.d.gate == MOE_GATE_FULL      ? launch_norm_t<T, VE, VPT, kGateAll>(a, s, backward, nv)
           : a.d.gate == MOE_GATE_CHANNEL ? launch_norm_t<T, VE, VPT, kGateColumn>(a, s, backward, nv)
                                          : launch_norm_t<T, VE, VPT, kGateRow>(a, s, backward, nv);
}

// Vectors of a thread: the fewest with which 512 threads cover the row. (A row of 8192 columns less a few that begins inside
// a vector takes one vector more than 8192 do.)
template <typename T>
static cudaError_t launch_norm_any(const NormArgs& a, cudaStream_t s, bool backward) {
    constexpr int VE = 16 / (int)sizeof(T);
    const int nv = a.d.H % VE ? (a.d.H + 2 * VE - 2) / VE : a.d.H / VE, vpt = (nv + kNormThreads - 1) / kNormThreads;
    if (vpt == 1) return launch_norm_g<T, VE, 1>(a, s, backward, nv);
    if (vpt == 2) return launch_norm_g<T, VE, 2>(a, s, backward, nv);
    if constexpr (VE == 8)
        return launch_norm_g<T, VE, 3>(a, s, backward, nv);
    else
        return vpt <= 4 ? launch_norm_g<T, VE, 4>(a, s, backward, nv) : launch_norm_g<T, VE, 5>(a, s, backward, nv);
}

}  // namespace moe
