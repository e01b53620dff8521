// linear.cuh -- what the kernels of the linear layers share: a launch's view of its operands, the tiles and
// who takes them, activations, cluster helpers.
#pragma once

#include <type_traits>

#include "ops.cuh"
#include "sm100.cuh"

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
        : "r"(addr), "r"(rank)
        : "memory");
    return v;
}

__device__ __forceinline__ float lin_sigmoid(float v) { return 1.0f / (1.0f + expf(-v)); }
__device__ __forceinline__ float lin_act(int act, float z) {
    switch (act) {
        case MOE_ACT_SIGMOID: return lin_sigmoid(z);
        case MOE_ACT_RELU: return z > 0.f ? z : (z != z ? z : 0.f);
        case MOE_ACT_SILU: return z * lin_sigmoid(z);
        case MOE_ACT_GELU: return 0.5f * z * erfcf(-0.70710678f * z);
        default: return z;
    }
}
__device__ __forceinline__ float lin_slope(int act, float z) {
    switch (act) {
        case MOE_ACT_SIGMOID: { const float p = lin_sigmoid(z); return p * (1.f - p); }
        case MOE_ACT_RELU: return z > 0.f ? 1.f : 0.f;
        case MOE_ACT_SILU: { const float p = lin_sigmoid(z); return p * (1.f + z * (1.f - p)); }
        case MOE_ACT_GELU: return 0.5f * erfcf(-0.70710678f * z) + z * 0.39894228f * expf(-0.5f * z * z);
        default: return 1.f;
    }
}

// Columns of each of an expert's tiles: as even as steps of STEP allow.
template <int STEP>
__device__ __forceinline__ int lin_width(int cols, int tiles) { return ((cols + tiles - 1) / tiles + STEP - 1) / STEP * STEP; }

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
                n = (cols + a.colw - 1) / a.colw * a.ftiles;
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

template <int MODE, int STEP>
__device__ __forceinline__ LinTile lin_tile(const LinView& a, const int* off, const int* start, int t) {
    int lo = 0, hi = a.E;  // start[lo] <= t < start[hi]
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (start[mid] <= t) lo = mid; else hi = mid;
    }
    LinTile r;
    r.e = lo;
    r.row0 = off[lo];
    r.rows = max(off[lo + 1] - r.row0, 0);
    const int cols = MODE == kDw ? a.N : r.rows;
    const int n = (cols + a.colw - 1) / a.colw, local = t - start[lo], width = lin_width<STEP>(cols, n);
    r.f = local / n;
    r.c0 = (local - r.f * n) * width;
    r.cols = min(width, cols - r.c0);
    r.blocks = ((MODE == kDw ? r.rows : a.C) + 63) / 64;
    return r;
}

// Launches of the pair kernel (linear_pair.cu); grid: CTAs, an even number.
cudaError_t launch_pair(int32_t dtype, int mode, bool gated, const CUtensorMap& A, const CUtensorMap& B, const LinView& v, int grid,
                        cudaStream_t s);

}  // namespace moe
