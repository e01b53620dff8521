// linear.cuh -- what the kernels of the linear layers share: a launch's view of its operands, the tiles and
// who takes them, activations, cluster helpers.
#pragma once

#include <type_traits>

#include "ops.cuh"
#include "sm100.cuh"
#include "tiles.h"

namespace moe {

enum { kFwd = 0, kDx = 1, kDw = 2 };

constexpr int kLinThreads = 384, kLinEpiWarp0 = 4, kLinEpiWarps = 8;
constexpr int kLinMaxE = 256;
constexpr uint32_t kLinA = 128 * 64 * 2;  // a stage's feature side
constexpr int kLinBoxRows = 32;           // token rows of one TMA box

// One launch's view of the operands.
struct LinView {
    const int32_t* offsets;
    const void *bias, *residual;
    void *out, *z;
    int T, E, N;      // token rows, experts, W's rows
    int F;            // features: contiguous extent of out
    int C;            // contraction (kFwd, kDx)
    int colw;         // columns of a tile, at most (a multiple of 16; pair kernel: of 32)
    int ftiles;
    int act;
    int vec;          // rows of out, residual and z start on 8 bytes (pair kernel: on 16)
    int boxes;        // rows of a K-major column-side TMA box
    int suppress;     // testing aid: CTA 0 never loads its first stage
    const float* part;  // kDx, kDw: column sums of chunks of `chunk` rows to add up beside the products, or NULL
    int chunk;
    void* dbias;
    uint32_t* err;
    uint64_t wait_ns;
};

struct LinTile {
    int e, f, c0, cols, row0, blocks, rows;  // expert, feature tile, first column, columns, first token row, 64-deep blocks, the expert's rows
};

__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ uint32_t cluster_size() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void cluster_sync_all() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// 16 bytes at the same shared-memory address in CTA `rank` of the cluster.
__device__ __forceinline__ float4 ld_peer(uint32_t addr, uint32_t rank) {
    float4 v;
    asm volatile(
        "{\n\t.reg .b32 a;\n\t"
        "mapa.shared::cluster.u32 a, %4, %5;\n\t"
        "ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [a];\n\t}"
        : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
        : "r"(addr), "r"(rank));
    return v;
}

// The functions of the epilogue in fp32, for results of 16 bits: exp and the quotient are the hardware's approximations,
// good to a few 2^-22 relative at the arguments that matter, far below half a step of bf16 (2^-9 and up) or fp16 (2^-12).
__device__ __forceinline__ float lin_sigmoid(float v) { return __fdividef(1.0f, 1.0f + __expf(-v)); }

// Phi(z), the normal distribution function, and e = exp(-z^2 / 2), of two values. Phi(-|z|) = e * R(t), t = 1 / (1 + 0.3 |z|): the scaled
// tail exp(z^2 / 2) * Phi(-|z|) falls smoothly from 1/2 like 1 / |z|, so it is close to a polynomial in t. R is of degree 8,
// fitted here by reweighted least squares at Chebyshev nodes for the least relative error up to |z| = 14: 6e-8, evaluated in fp32
// 4e-7. (0.5 erfc(-z / sqrt 2) by the library's erfcf: 40 us more over 4096 x 8192.)
__device__ __forceinline__ void normal_cdf(float z0, float z1, F2& cdf, F2& e) {
    const F2 z = f2(z0, z1), d = f2_fma(f2_both(0.3f), f2(fabsf(z0), fabsf(z1)), f2_both(1.0f));
    float d0, d1, x0, x1;
    f2_split(d, d0, d1);
    const F2 t = f2(__fdividef(1.0f, d0), __fdividef(1.0f, d1));
    F2 p = f2_fma(f2_both(0.0383782946f), t, f2_both(-0.169166133f));
    p = f2_fma(p, t, f2_both(0.228660107f));
    p = f2_fma(p, t, f2_both(-0.0765065104f));
    p = f2_fma(p, t, f2_both(0.142535552f));
    p = f2_fma(p, t, f2_both(0.0946835130f));
    p = f2_fma(p, t, f2_both(0.121920347f));
    p = f2_fma(p, t, f2_both(0.119487688f));
    p = f2_fma(p, t, f2_both(7.16889144e-06f));
    f2_split(f2_mul(f2_mul(z, z), f2_both(-0.5f)), x0, x1);
    e = f2(__expf(x0), __expf(x1));
    p = f2_mul(p, e);
    f2_split(p, x0, x1);
    cdf = f2(z0 < 0.f ? x0 : 1.0f - x0, z1 < 0.f ? x1 : 1.0f - x1);
}

// v = act(v) of N values: one branch, then N independent chains.
template <int N>
__device__ __forceinline__ void lin_act(int act, float (&v)[N]) {
    if (act == MOE_ACT_SILU) {
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] *= lin_sigmoid(v[i]);
    } else if (act == MOE_ACT_GELU) {
        if constexpr (N == 1) {
            F2 c, e;
            float p, unused;
            normal_cdf(v[0], v[0], c, e);
            f2_split(c, p, unused);
            v[0] *= p;
        } else {
#pragma unroll
            for (int i = 0; i + 1 < N; i += 2) {
                F2 c, e;
                normal_cdf(v[i], v[i + 1], c, e);
                f2_split(f2_mul(f2(v[i], v[i + 1]), c), v[i], v[i + 1]);
            }
        }
    } else if (act == MOE_ACT_RELU) {
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] = v[i] < 0.f ? 0.f : v[i];
    } else if (act == MOE_ACT_SIGMOID) {
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] = lin_sigmoid(v[i]);
    }
}
// d *= act'(z) of N values.
template <int N>
__device__ __forceinline__ void lin_slope(int act, const float (&z)[N], float (&d)[N]) {
    if (act == MOE_ACT_SILU) {
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const float p = lin_sigmoid(z[i]);
            d[i] *= p * (1.f + z[i] * (1.f - p));
        }
    } else if (act == MOE_ACT_GELU) {
#pragma unroll
        for (int i = 0; i + 1 < N; i += 2) {
            F2 c, e;
            normal_cdf(z[i], z[i + 1], c, e);
            const F2 slope = f2_fma(f2_mul(f2(z[i], z[i + 1]), f2_both(0.39894228f)), e, c);  // Phi + z phi
            f2_split(f2_mul(f2(d[i], d[i + 1]), slope), d[i], d[i + 1]);
        }
    } else if (act == MOE_ACT_RELU) {
#pragma unroll
        for (int i = 0; i < N; ++i) d[i] = z[i] > 0.f ? d[i] : 0.f;
    } else if (act == MOE_ACT_SIGMOID) {
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const float p = lin_sigmoid(z[i]);
            d[i] *= p * (1.f - p);
        }
    }
}

// Row boundaries of the experts and first tile of each, in shared memory; every bound is within [0, T].
template <int MODE>
__device__ void lin_tables(const LinView& a, int* off, int* start) {
    const int e = threadIdx.x;
    if (e <= a.E) {
        const int o = a.offsets ? a.offsets[e] : e ? a.T : 0;
        const int c = min(max(o, 0), a.T);
        if (c != o) atomicOr(a.err, ERR_BAD_ROUTE);
        off[e] = c;
    }
    __syncthreads();
    if (threadIdx.x < 32) {
        const int lane = threadIdx.x;
        int run = 0;
        for (int b = 0; b < a.E; b += 32) {
            const int i = b + lane;
            int n = 0;
            if (i < a.E) {
                const int rows = off[i + 1] - off[i];
                if (rows < 0) atomicOr(a.err, ERR_BAD_ROUTE);
                const int cols = MODE == kDw ? a.N : max(rows, 0);
                n = lin_tiles(cols, a.colw) * a.ftiles;
            }
            int v = n;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int y = __shfl_up_sync(0xffffffffu, v, o);
                if (lane >= o) v += y;
            }
            if (i < a.E) start[i] = run + v - n;
            run += __shfl_sync(0xffffffffu, v, 31);
        }
        if (lane == 0) start[a.E] = run;
    }
    __syncthreads();
}

// A role's way through the tiles, in increasing order: the expert it is at and that expert's tiling.
template <int MODE, int STEP>
struct LinWalk {
    int e = -1, s0 = 0, s1 = 0, n = 1, width = 0, cols = 0;
    LinTile ti;
    __device__ __forceinline__ const LinTile& to(const LinView& a, const int* off, const int* start, int t) {
        if (t >= s1 || e < 0) {
            do s1 = start[++e + 1];
            while (t >= s1);
            s0 = start[e];
            ti.e = e;
            ti.row0 = off[e];
            ti.rows = max(off[e + 1] - ti.row0, 0);
            ti.blocks = ((MODE == kDw ? ti.rows : a.C) + 63) / 64;
            cols = MODE == kDw ? a.N : ti.rows;
            n = lin_tiles(cols, a.colw);
            width = lin_width<STEP>(cols, n);
        }
        const int local = t - s0;
        ti.f = n == 1 ? local : local / n;
        ti.c0 = (local - ti.f * n) * width;
        ti.cols = min(width, cols - ti.c0);
        return ti;
    }
};

// The forward pass of at most 8 rows of one matrix, or kFewRows of several (linear_few.cu).
constexpr int kFewRows = 64;
cudaError_t launch_few(int32_t dtype, bool gated, const void* x, const void* w, const LinView& v, int num_sms, cudaStream_t s);

// Eight columns from element `at` of a tensor of `total` elements, of which n belong to the row. Where rows do not
// start on 16 bytes (VE = 1) they come as the two aligned vectors around them and are shifted into place.
template <typename T, int VE>
__device__ __forceinline__ Raw ld_cols(const T* p, int64_t at, int64_t total, int n) {
    Raw r;
    if (VE == 8) {
        const uint4 v = *reinterpret_cast<const uint4*>(p + at);
        r.w[0] = v.x; r.w[1] = v.y; r.w[2] = v.z; r.w[3] = v.w;
        return r;
    }
    const int64_t lo = at & ~(int64_t)7;
    const int m = (int)(at - lo);
    if (lo + 16 <= total) {
        const uint4 x = *reinterpret_cast<const uint4*>(p + lo), y = *reinterpret_cast<const uint4*>(p + lo + 8);
        uint32_t w[8] = {x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w};
        if (m & 4) {
#pragma unroll
            for (int i = 0; i < 6; ++i) w[i] = w[i + 2];
        }
        if (m & 2) {
#pragma unroll
            for (int i = 0; i < 5; ++i) w[i] = w[i + 1];
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) r.w[i] = __funnelshift_r(w[i], w[i + 1], 16 * (m & 1));
    } else {
        r.w[0] = r.w[1] = r.w[2] = r.w[3] = 0u;
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i < n) r.w[i >> 1] |= (uint32_t)reinterpret_cast<const uint16_t*>(p)[at + i] << (16 * (i & 1));
    }
    return r;
}

// db[e, n] of the chunks' column sums, a warp to 32 columns of an expert: the chunks of its rows in order. For `warps`
// warps, of which this is number `w`: the products' kernels have two warps to spare in every CTA.
template <typename T>
__device__ void lin_dbias(const LinView& a, const int* off, int w, int warps) {
    const int lane = threadIdx.x & 31, strips = (a.N + 31) / 32;
    for (int64_t i = w; i < (int64_t)a.E * strips; i += warps) {
        const int e = (int)(i / strips), n = (int)(i - (int64_t)e * strips) * 32 + lane;
        if (n >= a.N) continue;
        const int b0 = off[e], b1 = off[e + 1];
        float s[4] = {0.f, 0.f, 0.f, 0.f};
        if (b0 < b1) {
            const int c0 = b0 / a.chunk, c1 = (b1 - 1) / a.chunk + 1;
            const float* p = a.part + (int64_t)(c0 + e) * a.N + n;
            for (int c = c0; c < c1; c += 16, p += (int64_t)16 * a.N) {
                float v[16];  // on their way together: a strip's sums are a chain of waits (119 chunks by fours 18 us)
#pragma unroll
                for (int k = 0; k < 16; ++k) v[k] = c + k < c1 ? p[(int64_t)k * a.N] : 0.f;
#pragma unroll
                for (int k = 0; k < 16; ++k) s[k & 3] += v[k];
            }
        }
        reinterpret_cast<T*>(a.dbias)[(int64_t)e * a.N + n] = from_f<T>((s[0] + s[1]) + (s[2] + s[3]));
    }
}

// Launches of the pair kernel (linear_pair.cu); grid: CTAs, an even number.
// C: kDw, the map of its result.
cudaError_t launch_pair(int32_t dtype, int mode, bool gated, const CUtensorMap& A, const CUtensorMap& B, const CUtensorMap& C, const LinView& v,
                        int grid, cudaStream_t s);

}  // namespace moe
