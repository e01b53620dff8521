// norm.cuh -- the norms on both sides of a block, with its gate and the residual sum between them.
//
//   n    = N(y; gamma_post)  (or y)             N(v; g) = v * rsqrt(mean(v^2) + eps) * g
//   s    = residual_scale * residual + branch_scale * act(gate) * n
//   xn   = N(s; gamma_pre)                      from s before its rounding
// and the gradients of all of it. Bound by HBM: each tensor is read or written once. Forward a row stays in registers between its two
// sums, as far as they go: of rows of three to five vectors a thread most kernels spill 28 to 336 bytes a thread. Backward it stays in
// shared memory, and in registers too where a thread has one vector of it (rows of 8185 fp32 and more that begin anywhere have no room
// for ds and a whole gate there: those are read from memory twice). Everything is computed in fp32 and rounded once where it is stored.
//
// Backward, for g_s = ds + (gradient through xn), r = rsqrt(mean(v^2) + eps) of each norm:
//   g_s  = ds + r_s * (dxn * gamma_pre) - s * r_s^3 * mean(dxn * gamma_pre * s)
//   dn   = branch_scale * act(gate) * g_s
//   dy   = r_y * (dn * gamma_post) - y * r_y^3 * mean(dn * gamma_post * y)
// where the last mean needs g_s at every column; but with p = dxn * gamma_pre and w = act(gate) * gamma_post * y it is
//   w . g_s = w . ds + r_s * (w . p) - r_s^3 * mean(p * s) * (w . s)
// so a row takes one round of six sums (s^2, y^2, p s, w ds, w p, w s), and the same w . g_s gives a token gate's gradient.
// Sums over tokens (gammas, a channel gate) stay in the registers of the thread that owns the columns while it walks its
// rows; each CTA writes one row of partial sums and a second kernel adds those in a fixed order, so gradients are the same
// bits on every call.
//
// A CTA is one or more groups of threads with a row each at a time (a warp where 32 vectors of 16 bytes cover the row),
// synchronised by a barrier of their own. What keeps HBM busy across the sums: forward, a group loads its next row
// into registers before it works on the current one; backward, which has up to five tensors to read, a thread copies its pieces of the next one
// to three rows into shared memory, where it alone reads them. A thread's 16-byte vectors are aligned in memory whatever the row
// length: the rows of a group all begin at the same place within a vector (their numbers are equal mod 8), so its columns
// stay the same from row to row, and only a row's first and last vector are masked when read and written element by element.
//
// Measured (graph replay): forward 4096 x 2048 bf16 14.0 us = 4.8 TB/s, 32768 x 2048 87 us = 6.2 TB/s, 4096 x 2048 with a whole sigmoid gate
// 16.0 to 16.5 us = 5.1 TB/s (issue slots 75 %), fp32 24.8 us = 5.4 TB/s; long and odd rows: 2048 x 8191 bf16 41 us = 3.3 TB/s, fp32 96 us = 2.8 TB/s,
// 2048 x 8192 fp32 63 us = 4.3 TB/s. Backward 4096 x 2048 28 us, 32768 x 2048 145 us = 5.6 TB/s, 4096 x 8192 86 us, 4096 x 2048
// fp32 37 us = 5.4 TB/s, 2048 x 8191 bf16 66, fp32 126 us: some 10 us whatever the rows for two launches, the first copies and the column sums, then issue slots.
// Tried backward: two rounds of sums and the next row in registers 37.7, 212, 155 and 60 us; 1024 threads of 64 registers that read a
// row's pieces twice instead of 512 that hold them 36.8 and 201; packed pairs of fp32 31.3 and 171 where single ones took 29.5 and 158.
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

// Zeros in place of the elements outside the row.
template <int VE>
__device__ __forceinline__ void row_mask(Raw& r, int c, int H) {
#pragma unroll
    for (int e = 0; e < VE; ++e)
        if ((unsigned)(c + e) >= (unsigned)H) r.w[e * 4 / VE] &= VE == 4 ? 0u : e & 1 ? 0x0000ffffu : 0xffff0000u;
}

template <typename T, int VE, int VPT, int GATE, bool ODD>
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
    const int mis = ODD ? (int)((int64_t)first * H % VE) : 0;  // the rows' place within a vector
    int col[VPT];
    bool live[VPT], whole[VPT];
    Raw y[VPT], r[VPT], ga[VPT];
    T tg = from_f<T>(0.f);
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        col[i] = (g.tid + i * g.threads) * VE - mis;
        live[i] = col[i] < H;
        whole[i] = !ODD || (col[i] >= 0 && col[i] + VE <= H);
    }
    const int last = d.T - VE;  // (from here on a row's last vector may reach past the tensor)
    auto load = [&](int t) {
        const int64_t row = (int64_t)t * H;
#pragma unroll
        for (int i = 0; i < VPT; ++i)
            if (live[i]) {
                const bool vec = whole[i] || t < last;
                y[i] = row_get<T, VE>((const T*)a.y + row, col[i], H, vec);
                if (a.residual) r[i] = row_get<T, VE>((const T*)a.residual + row, col[i], H, vec);
                if (full) ga[i] = row_get<T, VE>((const T*)a.gate + row, col[i], H, vec);
            }
        if (GATE == kGateRow && d.gate == MOE_GATE_TOKEN) tg = ((const T*)a.gate)[t];
    };
    if (first < d.T) load(first);
    Raw gp[VPT], gq[VPT];
    float gc[VPT][VE];  // act(gate) of a channel gate
#pragma unroll
    for (int i = 0; i < VPT; ++i)
        if (live[i]) {
            if (post && a.gamma_post) gp[i] = row_get<T, VE>((const T*)a.gamma_post, col[i], H, !ODD);
            if (a.xn && a.gamma_pre) gq[i] = row_get<T, VE>((const T*)a.gamma_pre, col[i], H, !ODD);
            if (channel) {
                R::values(row_get<T, VE>((const T*)a.gate, col[i], H, !ODD), gc[i]);
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
                if (!whole[i]) {  // (another row's elements in the same 16 bytes)
                    row_mask<VE>(y[i], col[i], H);
                    if (a.residual) row_mask<VE>(r[i], col[i], H);
                    if (full) row_mask<VE>(ga[i], col[i], H);
                }
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

// ---- backward. What a thread reads of a row it copies to shared memory itself, a few rows ahead, and reads it there twice.

// 16 bytes (the first `bytes` of them, zeros behind) on their way from global to shared memory.
__device__ __forceinline__ void copy16(uint32_t dst, const void* src, uint32_t bytes) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copies_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }
__device__ __forceinline__ Raw lds_raw(uint32_t at) {
    Raw r;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(r.w[0]), "=r"(r.w[1]), "=r"(r.w[2]), "=r"(r.w[3]) : "r"(at) : "memory");
    return r;
}
__device__ __forceinline__ void sts_raw(uint32_t at, const Raw& r) {
    asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(r.w[0]), "r"(r.w[1]), "r"(r.w[2]), "r"(r.w[3]) : "memory");
}

constexpr int kBackSums = 6;
constexpr int kBackPitch = 20;  // floats between two sums of a group: a place for each of 16 warps, 4 more against bank conflicts
// Floats that H column sums take: one more every VE.
template <int VE>
__host__ __device__ constexpr int back_columns(int H) { return H + H / VE + 1; }

// Sums over the group of six values, the same in every thread: halves of the values change lanes on the way down, so that nine exchanges
// do for all; the warps' sums meet in buf (places past the last warp hold zeros) and are added by each warp again.
__device__ __forceinline__ void back_sums(float (&v)[kBackSums], float* buf, const NormGroup& g) {
    const int lane = threadIdx.x & 31;
    float w[4], x[2], y;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float lo = v[i], hi = i < 2 ? v[4 + i] : 0.f;
        w[i] = (lane & 16 ? hi : lo) + __shfl_xor_sync(0xffffffffu, lane & 16 ? lo : hi, 16);
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) x[i] = (lane & 8 ? w[2 + i] : w[i]) + __shfl_xor_sync(0xffffffffu, lane & 8 ? w[i] : w[2 + i], 8);
    y = (lane & 4 ? x[1] : x[0]) + __shfl_xor_sync(0xffffffffu, lane & 4 ? x[0] : x[1], 4);
    y += __shfl_xor_sync(0xffffffffu, y, 2);
    y += __shfl_xor_sync(0xffffffffu, y, 1);  // lanes 4 k .. 4 k + 3 hold sum k
    if (g.threads > 32) {
        const int k = min(lane >> 2, kBackSums - 1);
        if ((lane & 3) == 0 && lane < 4 * kBackSums) buf[k * kBackPitch + (g.tid >> 5)] = y;
        asm volatile("bar.sync %0, %1;" ::"r"(g.id + 1), "r"(g.threads) : "memory");
        const float4 a = *reinterpret_cast<const float4*>(buf + k * kBackPitch + (lane & 3) * 4);
        y = (a.x + a.y) + (a.z + a.w);
        y += __shfl_xor_sync(0xffffffffu, y, 1);
        y += __shfl_xor_sync(0xffffffffu, y, 2);
    }
#pragma unroll
    for (int k = 0; k < kBackSums; ++k) v[k] = __shfl_sync(0xffffffffu, y, 4 * k);
}

// How a CTA of the backward pass uses its shared memory: a thread's constants (gammas, channel gate), its copies of rows, the
// groups' sums.
struct BackPlan {
    int tpr, groups, stages, slots;  // threads of a row, rows at once, rows on their way, tensors copied
    uint32_t ring, bufs, bytes;      // where the copies and the sums begin, all of it
};

template <typename T, int VE, int VPT, int GATE, bool ODD>
__global__ void __launch_bounds__(kNormThreads, 1)
    k_norm_backward(const NormArgs a, const BackPlan plan) {
    typedef RawOf<T> R;
    extern __shared__ __align__(16) uint8_t back_smem[];
    grid_dep_wait();
    grid_dep_launch();
    const moe_norm_dims& d = a.d;
    const NormGroup g = norm_group(plan.tpr);
    const int H = d.H, first = blockIdx.x * g.groups + g.id, step = gridDim.x * g.groups;
    constexpr bool full = GATE == kGateAll, channel = GATE == kGateColumn;
    constexpr bool kCopyAll = VPT < 5;  // (rows of 8185 fp32 and more: no room for ds and a whole gate)
    constexpr int kConsts = channel ? 2 + VE / 4 : 2;
    constexpr bool kHeld = VPT == 1;  // a row's values stay in registers from one pass over it to the other
    // A whole gate's sigmoid too where that is the long way to it (4096 x 2048 fp32 50 against 56 us), not the hardware's (bf16 40 against 38).
    constexpr bool kHeldGate = kHeld && sizeof(T) == 4;
    const bool post = (d.flags & MOE_NORM_POST) != 0, pre = a.dxn != nullptr;
    const bool token = GATE == kGateRow && d.gate == MOE_GATE_TOKEN;
    const int mis = ODD ? (int)((int64_t)first * H % VE) : 0;
    const uint32_t smem = (uint32_t)__cvta_generic_to_shared(back_smem);
    const uint32_t pieces = (uint32_t)blockDim.x * 16u;  // one of every thread
    const uint32_t consts = smem + threadIdx.x * 16u, ring = smem + plan.ring + threadIdx.x * 16u;
    float* buf = reinterpret_cast<float*>(back_smem + plan.bufs) + g.id * 2 * kBackSums * kBackPitch;
    const int slot_ds = pre ? 3 : 1, slot_gate = slot_ds + (a.ds ? 1 : 0);  // y; s and dxn; ds; a whole gate
    int col[VPT];
    bool live[VPT], whole[VPT];
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        col[i] = (g.tid + i * g.threads) * VE - mis;
        live[i] = col[i] < H;
        whole[i] = !ODD || (col[i] >= 0 && col[i] + VE <= H);
    }
    const int last = d.T - VE;  // (from here on a row's last vector may reach past the tensor)
    auto fetch = [&](int t, int stage) {
        if (t < d.T) {
#pragma unroll
            for (int i = 0; i < VPT; ++i)
                if (live[i]) {
                    // (aligned: a row's first vector may begin and its last may end in another row, whose elements are masked)
                    const int64_t at = (int64_t)t * H + col[i];
                    const uint32_t bytes = t < last ? 16u : (uint32_t)min(VE, (d.T - t) * H - col[i]) * (uint32_t)sizeof(T);
                    const uint32_t dst = ring + (uint32_t)(stage * plan.slots * VPT + i) * pieces;
                    copy16(dst, (const T*)a.y + at, bytes);
                    if (pre) {
                        copy16(dst + VPT * pieces, (const T*)a.s_in + at, bytes);
                        copy16(dst + 2 * VPT * pieces, (const T*)a.dxn + at, bytes);
                    }
                    if (kCopyAll && a.ds) copy16(dst + slot_ds * VPT * pieces, (const T*)a.ds + at, bytes);
                    if (kCopyAll && full) copy16(dst + slot_gate * VPT * pieces, (const T*)a.gate + at, bytes);
                }
        }
        copies_commit();
    };
    for (int k = 0; k < plan.stages; ++k) fetch(first + k * step, k);
    float acc_post[VPT][VE], acc_pre[VPT][VE], acc_gate[VPT][VE];
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        float one[VE];
#pragma unroll
        for (int e = 0; e < VE; ++e) one[e] = 1.f;
#pragma unroll
        for (int e = 0; e < VE; ++e) acc_post[i][e] = acc_pre[i][e] = acc_gate[i][e] = 0.f;
        Raw gp = R::pack(one), gq = gp;
        const uint32_t at = consts + (uint32_t)(i * kConsts) * pieces;
        if (live[i]) {
            if (post && a.gamma_post) gp = row_get<T, VE>((const T*)a.gamma_post, col[i], H, !ODD);
            if (pre && a.gamma_pre) gq = row_get<T, VE>((const T*)a.gamma_pre, col[i], H, !ODD);
            if (channel) {
                float gc[VE];
                R::values(row_get<T, VE>((const T*)a.gate, col[i], H, !ODD), gc);
                gate_values<T, VE>(d.gate_act, gc);
#pragma unroll
                for (int e = 0; e < VE; e += 4)
                    sts_raw(at + (2 + e / 4) * pieces, Raw{{__float_as_uint(gc[e]), __float_as_uint(gc[e + 1]), __float_as_uint(gc[e + 2]), __float_as_uint(gc[e + 3])}});
            }
        }
        sts_raw(at, gp);
        sts_raw(at + pieces, gq);
    }
    if (g.threads > 32) {
        for (int i = g.tid; i < 2 * kBackSums * kBackPitch; i += g.threads) buf[i] = 0.f;
        asm volatile("bar.sync %0, %1;" ::"r"(g.id + 1), "r"(g.threads) : "memory");
    }
    auto constant = [&](int which, int i, float (&f)[VE]) { R::values(lds_raw(consts + (uint32_t)(i * kConsts + which) * pieces), f); };
    auto channel_gate = [&](int i, float (&f)[VE]) {
#pragma unroll
        for (int e = 0; e < VE / 4; ++e) {
            const Raw r = lds_raw(consts + (uint32_t)(i * kConsts + 2 + e) * pieces);
#pragma unroll
            for (int k = 0; k < 4; ++k) f[4 * e + k] = __uint_as_float(r.w[k]);
        }
    };
    // a row's piece of the tensors (zeros outside the row): y, s, p = dxn gamma_pre, dxn s, ds
    auto gather = [&](uint32_t row, int t, int i, float (&y)[VE], float (&sv)[VE], float (&p)[VE], float (&qs)[VE], float (&ds)[VE]) {
        const uint32_t at = row + (uint32_t)i * pieces;
        Raw ry = lds_raw(at), rsv = {}, rq = {}, rd = {};
        if (pre) {
            rsv = lds_raw(at + VPT * pieces);
            rq = lds_raw(at + 2 * VPT * pieces);
        }
        if (a.ds) rd = kCopyAll ? lds_raw(at + slot_ds * VPT * pieces) : row_get<T, VE>((const T*)a.ds + (int64_t)t * H, col[i], H, whole[i]);
        if (!whole[i]) {
            row_mask<VE>(ry, col[i], H);
            row_mask<VE>(rsv, col[i], H);
            row_mask<VE>(rq, col[i], H);
            row_mask<VE>(rd, col[i], H);
        }
        R::values(ry, y);
        R::values(rd, ds);
        R::values(rsv, sv);
        if (pre) {
            float q[VE], m[VE];
            R::values(rq, q);
            constant(1, i, m);
#pragma unroll
            for (int e = 0; e < VE; ++e) {
                p[e] = q[e] * m[e];
                qs[e] = q[e] * sv[e];
            }
        } else {
#pragma unroll
            for (int e = 0; e < VE; ++e) p[e] = qs[e] = 0.f;
        }
    };
    // a whole gate's piece as it is
    auto take_gate = [&](uint32_t row, int t, int i, float (&f)[VE]) {
        Raw r = kCopyAll ? lds_raw(row + (uint32_t)(slot_gate * VPT + i) * pieces) : row_get<T, VE>((const T*)a.gate + (int64_t)t * H, col[i], H, whole[i]);
        if (!whole[i]) row_mask<VE>(r, col[i], H);
        R::values(r, f);
    };
    const float inv_h = 1.0f / (float)H;
    T tg = from_f<T>(0.f);
    if (token && first < d.T) tg = ((const T*)a.gate)[first];
    int turn = 0, stage = 0;
    for (int t = first; t < d.T; t += step, turn ^= 1) {
        const int64_t at = (int64_t)t * H;
        const uint32_t row = ring + (uint32_t)(stage * plan.slots * VPT) * pieces;
        float tval[1] = {1.f}, tslope[1] = {0.f};
        if (token) {
            tval[0] = to_f(tg);
            gate_slopes<T, 1>(d.gate_act, tval, tslope);
            if (t + step < d.T) tg = ((const T*)a.gate)[t + step];
        }
        if (plan.stages == 1) copies_wait<0>();
        else if (plan.stages == 2) copies_wait<1>();
        else copies_wait<2>();
        // with w = gate gamma_post y: s^2, y^2, p s, w ds, w p, w s
        float sm[kBackSums] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
        float y[VE], sv[VE], p[VE], qs[VE], ds[VE];
        float sig[VE];  // sigmoid of a whole gate, for the second pass
#pragma unroll
        for (int i = 0; i < VPT; ++i)
            if (live[i]) {
                gather(row, t, i, y, sv, p, qs, ds);
                float w[VE], m[VE];
                constant(0, i, m);
#pragma unroll
                for (int e = 0; e < VE; ++e) w[e] = y[e] * m[e];
                if (channel) {
                    channel_gate(i, m);
#pragma unroll
                    for (int e = 0; e < VE; ++e) w[e] *= m[e];
                }
                if (full) {
                    float g0[VE];
                    take_gate(row, t, i, g0);
                    if (d.gate_act != MOE_ACT_NONE) {
#pragma unroll
                        for (int e = 0; e < VE; ++e) {
                            const float q = norm_sigmoid<T>(g0[e]);
                            if (kHeldGate) sig[e] = q;
                            g0[e] = d.gate_act == MOE_ACT_SILU ? g0[e] * q : q;
                        }
                    }
#pragma unroll
                    for (int e = 0; e < VE; ++e) w[e] *= g0[e];
                }
#pragma unroll
                for (int e = 0; e < VE; ++e) {
                    sm[0] = fmaf(sv[e], sv[e], sm[0]);
                    sm[1] = fmaf(y[e], y[e], sm[1]);
                    sm[2] = fmaf(p[e], sv[e], sm[2]);
                    sm[3] = fmaf(w[e], ds[e], sm[3]);
                    sm[4] = fmaf(w[e], p[e], sm[4]);
                    sm[5] = fmaf(w[e], sv[e], sm[5]);
                }
            }
        back_sums(sm, buf + turn * kBackSums * kBackPitch, g);
        const float rs = pre ? rsqrtf(sm[0] * inv_h + d.eps) : 0.f;
        const float ry = post ? rsqrtf(sm[1] * inv_h + d.eps) : 1.f;
        const float cs = pre ? rs * (rs * (sm[2] * inv_h)) : 0.f;  // (r^3 by itself may leave fp32's range)
        const float wg = pre ? fmaf(rs, fmaf(-cs, sm[5], sm[4]), sm[3]) : sm[3];  // w . g_s
        const float branch = d.branch_scale * tval[0];
        const float cy = post ? ry * (ry * (branch * wg * inv_h)) : 0.f;
        if (token && a.dgate && g.tid == 0) ((T*)a.dgate)[t] = from_f<T>(d.branch_scale * (ry * wg) * tslope[0]);
#pragma unroll
        for (int i = 0; i < VPT; ++i)
            if (live[i]) {
                if (!kHeld) gather(row, t, i, y, sv, p, qs, ds);
                float v[VE], o[VE], gm[VE], dn[VE];  // v: g_s
                if (pre) {
#pragma unroll
                    for (int e = 0; e < VE; ++e) {
                        v[e] = fmaf(rs, fmaf(-sv[e], cs, p[e]), ds[e]);
                        acc_pre[i][e] = fmaf(qs[e], rs, acc_pre[i][e]);
                    }
                } else {
#pragma unroll
                    for (int e = 0; e < VE; ++e) v[e] = ds[e];
                }
                if (a.dresidual) {
#pragma unroll
                    for (int e = 0; e < VE; ++e) o[e] = d.residual_scale * v[e];
                    row_put<T, VE>((T*)a.dresidual + at, col[i], H, whole[i], R::pack(o));
                }
                constant(0, i, gm);
                float yn[VE];
#pragma unroll
                for (int e = 0; e < VE; ++e) {
                    yn[e] = y[e] * ry;
                    dn[e] = branch * v[e];
                }
                if (channel) {
                    float gc[VE];
                    channel_gate(i, gc);
#pragma unroll
                    for (int e = 0; e < VE; ++e) {
                        acc_gate[i][e] = fmaf(v[e], yn[e] * gm[e], acc_gate[i][e]);  // (branch and slope: at the end)
                        dn[e] *= gc[e];
                    }
                }
                if (full) {
                    float ge[VE], slope[VE];
                    take_gate(row, t, i, ge);
                    if (!kHeldGate) {
                        gate_slopes<T, VE>(d.gate_act, ge, slope);
                    } else {
#pragma unroll
                        for (int e = 0; e < VE; ++e) {
                            const float q = sig[e];
                            slope[e] = d.gate_act == MOE_ACT_NONE ? 1.f : d.gate_act == MOE_ACT_SILU ? q * (1.f + ge[e] * (1.f - q)) : q * (1.f - q);
                            ge[e] = d.gate_act == MOE_ACT_NONE ? ge[e] : d.gate_act == MOE_ACT_SILU ? ge[e] * q : q;
                        }
                    }
                    if (a.dgate) {
#pragma unroll
                        for (int e = 0; e < VE; ++e) o[e] = dn[e] * (yn[e] * gm[e]) * slope[e];
                        row_put<T, VE>((T*)a.dgate + at, col[i], H, whole[i], R::pack(o));
                    }
#pragma unroll
                    for (int e = 0; e < VE; ++e) dn[e] *= ge[e];
                }
#pragma unroll
                for (int e = 0; e < VE; ++e) acc_post[i][e] = fmaf(dn[e], yn[e], acc_post[i][e]);
                if (a.dy) {
                    if (post) {  // (without the norm dy is dn)
#pragma unroll
                        for (int e = 0; e < VE; ++e) dn[e] = ry * fmaf(-y[e], cy, dn[e] * gm[e]);
                    }
                    row_put<T, VE>((T*)a.dy + at, col[i], H, whole[i], R::pack(dn));
                }
            }
        fetch(t + plan.stages * step, stage);
        stage = stage + 1 == plan.stages ? 0 : stage + 1;
    }
    copies_wait<0>();
    if (!a.part) return;
    if (channel) {
#pragma unroll
        for (int i = 0; i < VPT; ++i)
            if (live[i]) {
                float ge[VE], slope[VE];
                R::values(row_get<T, VE>((const T*)a.gate, col[i], H, !ODD), ge);
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
    // the CTA's groups meet where the copies were (a column is another thread's in each), a word past every VE columns so that the
    // threads' writes lie in different banks; then a thread a column, the groups in order
    float* sums = reinterpret_cast<float*>(back_smem);
    const int kinds = channel ? 3 : 2, pitch = back_columns<VE>(H);
    __syncthreads();
#pragma unroll
    for (int e = 0; e < VE; ++e) {
        const int h = col[0] + e;
        if ((unsigned)h < (unsigned)H) {
            float* p = sums + (g.id * kinds) * pitch + h + h / VE;
            p[0] = acc_post[0][e];
            p[pitch] = acc_pre[0][e];
            if (channel) p[2 * pitch] = acc_gate[0][e];
        }
    }
    __syncthreads();
    for (int k = 0; k < kinds; ++k)
        for (int h = threadIdx.x; h < H; h += blockDim.x) {
            float v = 0.f;
            for (int q = 0; q < g.groups; ++q) v += sums[(q * kinds + k) * pitch + h + h / VE];
            part[k * H + h] = v;
        }
}

// Column sums of the row blocks' partial sums: 32 columns a CTA, 16 threads a column, each a sixteenth of the
// blocks in order, then the 16 in order.
template <typename T>
__global__ void __launch_bounds__(512) k_norm_columns(const NormArgs a, int blocks) {
    constexpr int kParts = 16;
    __shared__ float sm[kParts][33];
    grid_dep_wait();
    grid_dep_launch();
    const int which = blockIdx.y, h = blockIdx.x * 32 + threadIdx.x % 32, q = threadIdx.x / 32;
    T* out = reinterpret_cast<T*>(which == 0 ? a.dgamma_post : which == 1 ? a.dgamma_pre : a.d.gate == MOE_GATE_CHANNEL ? a.dgate : nullptr);
    if (!out) return;
    float v = 0.f;
    if (h < a.d.H) {
        const float* p = a.part + (int64_t)which * a.d.H + h;
        const int per = (blocks + kParts - 1) / kParts, b1 = min(blocks, (q + 1) * per);
        for (int b0 = q * per; b0 < b1; b0 += 10) {
            float x[10];  // on their way together
#pragma unroll
            for (int i = 0; i < 10; ++i) x[i] = b0 + i < b1 ? p[(int64_t)(b0 + i) * 3 * a.d.H] : 0.f;
#pragma unroll
            for (int i = 0; i < 10; ++i) v += x[i];
        }
    }
    sm[q][threadIdx.x % 32] = v;
    __syncthreads();
    if (q == 0 && h < a.d.H) {
        v = 0.f;
#pragma unroll
        for (int i = 0; i < kParts; ++i) v += sm[i][threadIdx.x];
        out[h] = from_f<T>(v);
    }
}

// CTAs, `most` at most; rows of a group are equal mod VE.
template <int VE>
static int norm_grid(const NormArgs& a, int groups, int most) {
    int blocks = min((a.d.T + groups - 1) / groups, most);
    if (a.d.H % VE && blocks * groups % VE) {
        const int up = (blocks + VE - 1) / VE * VE;
        blocks = blocks < a.d.T && up <= kNormBlocks ? up : max(VE, blocks / VE * VE);
    }
    return blocks;
}

// Vectors that cover any row of H columns, wherever in a vector it begins; vectors and threads of a row.
template <typename T, int VE, int VPT, int GATE, bool ODD>
static cudaError_t launch_norm_t(const NormArgs& a, cudaStream_t s, int nv) {
    const int tpr = max(32, ((nv + VPT - 1) / VPT + 31) / 32 * 32);
    int groups = VPT == 1 ? max(1, min(16, 512 / tpr)) : 1;
    while (groups > 1 && a.d.T < groups * a.num_sms) groups /= 2;  // (few rows: a CTA each)
    const int blocks = norm_grid<VE>(a, groups, a.num_sms * (VPT > 1 ? 1 : 2));
    cudaError_t e;
    MOE_LAUNCH(MOE_KERNEL_NORM, s, (e = launch_pdl(k_norm<T, VE, VPT, GATE, ODD>, dim3(blocks), dim3(tpr * groups), 0, s, a, tpr)));
    return e;
}

template <typename T, int VE, int VPT, int GATE, bool ODD>
static cudaError_t launch_norm_backward_t(const NormArgs& a, cudaStream_t s, int nv) {
    constexpr uint32_t kRoom = 227 * 1024;
    BackPlan p = {};
    p.tpr = max(32, ((nv + VPT - 1) / VPT + 31) / 32 * 32);
    // (named barriers: 15 besides the CTA's own; a warp needs none)
    p.groups = VPT == 1 ? max(1, min(p.tpr > 32 ? 8 : 16, kNormThreads / p.tpr)) : 1;
    while (p.groups > 1 && a.d.T < p.groups * a.num_sms) p.groups /= 2;  // (few rows: a CTA each)
    const int blocks = norm_grid<VE>(a, p.groups, min(kNormBlocks, a.num_sms));
    if (blocks > norm_blocks(a.d.T)) return cudaErrorInvalidValue;  // (never: what the workspace holds)
    constexpr bool kCopyAll = VPT < 5;
    const uint32_t pieces = (uint32_t)(p.tpr * p.groups * VPT) * 16u;
    p.slots = 1 + (a.dxn ? 2 : 0) + (kCopyAll && a.ds ? 1 : 0) + (kCopyAll && GATE == kGateAll ? 1 : 0);
    p.ring = pieces * (GATE == kGateColumn ? 2 + VE / 4 : 2);
    const uint32_t sums = (uint32_t)(p.groups * 2 * kBackSums * kBackPitch) * 4u;
    p.stages = (int)min(3u, (kRoom - sums - p.ring) / (pieces * p.slots));
    p.bufs = p.ring + pieces * p.slots * p.stages;
    p.bytes = max(p.bufs + sums, p.groups > 1 ? (uint32_t)(p.groups * (GATE == kGateColumn ? 3 : 2) * back_columns<VE>(a.d.H)) * 4u : 0u);
    if (p.stages < 1 || p.bytes > kRoom) return cudaErrorInvalidValue;  // (never)
    static std::atomic<bool> allowed[64];
    cudaError_t e = allow_shared(k_norm_backward<T, VE, VPT, GATE, ODD>, (int)kRoom, allowed);
    if (e != cudaSuccess) return e;
    NormArgs b = a;
    const bool columns = a.dgamma_post || a.dgamma_pre || (a.dgate && a.d.gate == MOE_GATE_CHANNEL);
    if (!columns) b.part = nullptr;
    MOE_LAUNCH(MOE_KERNEL_NORM_BACKWARD, s, (e = launch_pdl(k_norm_backward<T, VE, VPT, GATE, ODD>, dim3(blocks), dim3(p.tpr * p.groups), p.bytes, s, b, p)));
    if (e == cudaSuccess && columns)
        MOE_LAUNCH(MOE_KERNEL_NORM_BACKWARD, s, (e = launch_pdl(k_norm_columns<T>, dim3((a.d.H + 31) / 32, GATE == kGateColumn ? 3 : 2), dim3(512), 0, s, b, blocks)));
    return e;
}

template <typename T, int VE, int VPT, bool ODD>
static cudaError_t launch_norm_g(const NormArgs& a, cudaStream_t s, bool backward, int nv) {
    if (backward)
        return a.d.gate == MOE_GATE_FULL      ? launch_norm_backward_t<T, VE, VPT, kGateAll, ODD>(a, s, nv)
               : a.d.gate == MOE_GATE_CHANNEL ? launch_norm_backward_t<T, VE, VPT, kGateColumn, ODD>(a, s, nv)
                                              : launch_norm_backward_t<T, VE, VPT, kGateRow, ODD>(a, s, nv);
    return a.d.gate == MOE_GATE_FULL      ? launch_norm_t<T, VE, VPT, kGateAll, ODD>(a, s, nv)
           : a.d.gate == MOE_GATE_CHANNEL ? launch_norm_t<T, VE, VPT, kGateColumn, ODD>(a, s, nv)
                                          : launch_norm_t<T, VE, VPT, kGateRow, ODD>(a, s, nv);
}

// Vectors of a thread: the fewest with which 512 threads cover the row. ODD: rows begin anywhere in a vector. (A row of 8192 columns
// less a few then takes one vector more than 8192 do.)
template <typename T>
static cudaError_t launch_norm_any(const NormArgs& a, cudaStream_t s, bool backward) {
    constexpr int VE = 16 / (int)sizeof(T);
    if (a.d.H % VE == 0) {
        const int nv = a.d.H / VE;
        if (nv <= kNormThreads) return launch_norm_g<T, VE, 1, false>(a, s, backward, nv);
        if (nv <= 2 * kNormThreads) return launch_norm_g<T, VE, 2, false>(a, s, backward, nv);
        if constexpr (VE == 4) return launch_norm_g<T, VE, 4, false>(a, s, backward, nv);
    }
    const int nv = (a.d.H + 2 * VE - 2) / VE;
    if (nv <= kNormThreads) return launch_norm_g<T, VE, 1, true>(a, s, backward, nv);
    if (nv <= 2 * kNormThreads) return launch_norm_g<T, VE, 2, true>(a, s, backward, nv);
    return launch_norm_g<T, VE, VE == 8 ? 3 : 5, true>(a, s, backward, nv);
}

}  // namespace moe
