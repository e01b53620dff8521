// exchange.cu -- token rows to their experts and back.
//
//   sort      a stable counting sort of the pairs p = t * K + k by expert: counts, offsets, perm
//             (pairs in order, -1 behind the last) and inv (each pair's place, -1 for a dropped slot)
//   spread    rows[inv[p]] = (w[p]) * tok[t]            dispatch, and the backward pass of combine
//   gather    out[t] = (res[t]) + sum_k (w[p]) * rows[inv[p]]   combine, and the backward pass of dispatch
// with, on request, dots[p] = tok[t] . rows[inv[p]]: the gradient of w in either direction.
//
// All of it is bound by HBM: a token row is read once and kept in registers while its K copies are
// written, and a token's K rows are read once, side by side, and summed in fp32 in slot order, the residual last. Measured for 4096
// tokens of 2048 bf16 by 8 slots (graph replay): spread 25 us = 5.9 TB/s, with dots 49 us = 5.8 TB/s, gather into a residual 28 us = 6.0 TB/s,
// with dots 40 us = 4.2 TB/s (at 101 registers two CTAs of 256 fit an SM, so the 512 are 1.7 waves and 21 % of the warps there could be are
// active; each waits for its eight rows before it works: 27 % of the issue slots and 64 % of HBM's rate are used). Rows of 2044 (8 bytes at a
// time) 27, 61, 32, 42 us, of 2046 (4 bytes) 37, 89, 42, 83, of 2045 (elements) 45, 131, 76, 142.
// Sums and dots run in a fixed order, so results are the same bits on every call.
#include <atomic>

#include <cooperative_groups.h>

#include "ops.cuh"

namespace moe {

namespace cg = cooperative_groups;

// ---------------------------------------------------------------------------------------
// sort: one thread-block cluster of up to 16 CTAs (8 where the device has no room for 16). A CTA takes a run of pairs, each
// of its 32 warps a piece of the run. Pass one counts each warp's pairs per expert (equal ids of 32 lanes at once, by votes,
// no atomics), the counts are scanned over warps, over CTAs (read through distributed shared
// memory) and over experts, pass two writes the pairs' places. One launch and no workspace: 8 pairs 3.0 us, 32768
// pairs 7.1 (8.0 by 8 CTAs), 131072 pairs 14.4 (23.5).
constexpr int kSortWarps = 32, kSortMaxE = 256, kSortCtas = 16;

// The lanes whose expert (0 .. 255, or -1: none) is this lane's. One vote a bit: the match instruction takes one turn for each
// distinct value, and 32 lanes of 256 experts mostly are: 32768 ids took 12 us with it.
__device__ __forceinline__ unsigned same_expert(int e) {
    unsigned m = __ballot_sync(0xffffffffu, e >= 0);
#pragma unroll
    for (int b = 0; b < 8; ++b) {
        const unsigned v = __ballot_sync(0xffffffffu, (e >> b) & 1);
        m &= (e >> b) & 1 ? v : ~v;
    }
    return m;
}

__global__ void __launch_bounds__(32 * kSortWarps, 1)
    k_sort_pairs(const int32_t* __restrict__ ids, int32_t* __restrict__ counts, int32_t* __restrict__ offsets,
                 int32_t* __restrict__ perm, int32_t* __restrict__ inv, int P, int E, int seg) {
    __shared__ int cnt[kSortWarps][kSortMaxE];  // a warp's pairs of each expert, then its first place among them
    __shared__ int tot[kSortMaxE];              // this CTA's pairs of each expert
    __shared__ int base[kSortMaxE];             // first place of this CTA's pairs of each expert
    __shared__ int wsum[kSortMaxE / 32];
    __shared__ int total_s;
    cg::cluster_group cl = cg::this_cluster();
    const int rank = (int)cl.block_rank(), n = (int)cl.num_blocks();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const unsigned below = (1u << lane) - 1u;
    grid_dep_wait();
    grid_dep_launch();
    for (int e = lane; e < E; e += 32) cnt[warp][e] = 0;
    __syncwarp();
    const int64_t p0 = ((int64_t)rank * kSortWarps + warp) * seg;
    const int64_t p1 = p0 + seg < P ? p0 + seg : P;
    constexpr int kAhead = 4;  // ids loaded together; a piece of no more is ranked once and for all in the first pass
    int held[kAhead], ahead[kAhead];  // expert, pairs of the warp before it with the same one
    for (int64_t i0 = p0; i0 < p1; i0 += 32 * kAhead) {
#pragma unroll
        for (int j = 0; j < kAhead; ++j) {
            const int64_t i = i0 + 32 * j + lane;
            held[j] = i < p1 ? ids[i] : -1;
            if ((unsigned)held[j] >= (unsigned)E) held[j] = -1;
        }
#pragma unroll
        for (int j = 0; j < kAhead; ++j) {
            const unsigned m = same_expert(held[j]);
            const int before = held[j] >= 0 ? cnt[warp][held[j]] : 0;
            ahead[j] = before + __popc(m & below);
            __syncwarp();
            if (held[j] >= 0 && (m & below) == 0) cnt[warp][held[j]] = before + __popc(m);
            __syncwarp();
        }
    }
    __syncthreads();
    const int e = threadIdx.x;
    if (e < E) {
        int c[kSortWarps], sum = 0;
#pragma unroll
        for (int w = 0; w < kSortWarps; ++w) c[w] = cnt[w][e];
#pragma unroll
        for (int w = 0; w < kSortWarps; ++w) {
            cnt[w][e] = sum;
            sum += c[w];
        }
        tot[e] = sum;
    }
    if (n > 1) cl.sync();
    int all = e < E ? tot[e] : 0, before = 0;
    if (n > 1 && e < E) {
        all = 0;
        int c[kSortCtas];  // all on their way at once
#pragma unroll
        for (int r = 0; r < kSortCtas; ++r) c[r] = r < n ? cl.map_shared_rank(tot, r)[e] : 0;
#pragma unroll
        for (int r = 0; r < kSortCtas; ++r) {
            all += c[r];
            before += r < rank ? c[r] : 0;
        }
    }
    if (e < kSortMaxE) {  // exclusive scan over the experts
        int v = all;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, v, o);
            if (lane >= o) v += y;
        }
        if (lane == 31) wsum[warp] = v;
        base[e] = v - all;
    }
    __syncthreads();
    if (e < kSortMaxE) {
        int add = 0;
#pragma unroll
        for (int w = 0; w < kSortMaxE / 32; ++w) add += w < warp ? wsum[w] : 0;
        const int first = base[e] + add;
        base[e] = first + before;
        if (e == kSortMaxE - 1) total_s = first + all;
        if (rank == 0 && e < E) {
            counts[e] = all;
            offsets[e] = first;
            if (e == E - 1) offsets[E] = first + all;
        }
    }
    __syncthreads();
    const int total = total_s;
    for (int64_t i0 = p0; i0 < p1; i0 += 32 * kAhead) {
        if (seg > 32 * kAhead) {  // ranked again, from the warp's first places on
#pragma unroll
            for (int j = 0; j < kAhead; ++j) {
                const int64_t i = i0 + 32 * j + lane;
                held[j] = i < p1 ? ids[i] : -1;
                if ((unsigned)held[j] >= (unsigned)E) held[j] = -1;
            }
        }
#pragma unroll
        for (int j = 0; j < kAhead; ++j) {
            const int64_t i = i0 + 32 * j + lane;
            int at = -1;
            if (seg > 32 * kAhead) {
                const unsigned m = same_expert(held[j]);
                const int first = held[j] >= 0 ? cnt[warp][held[j]] : 0;
                if (held[j] >= 0) at = base[held[j]] + first + __popc(m & below);
                __syncwarp();
                if (held[j] >= 0 && (m & below) == 0) cnt[warp][held[j]] = first + __popc(m);
                __syncwarp();
            } else if (held[j] >= 0) {
                at = base[held[j]] + cnt[warp][held[j]] + ahead[j];
            }
            if (i < p1) {
                inv[i] = at;
                if (at >= 0) perm[at] = (int32_t)i;
                if (i >= total) perm[i] = -1;
            }
        }
    }
    if (n > 1) cl.sync();  // no CTA leaves while another may still read its counts
}

// CTAs of the largest sorting cluster that the current device holds.
static int sort_ctas() {
    static std::atomic<int> cache[64];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 8;
    int n = cache[dev].load(std::memory_order_relaxed);
    if (n) return n;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(kSortCtas);
    cfg.blockDim = dim3(32 * kSortWarps);
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = kSortCtas;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    int fits = 0;
    if (cudaFuncSetAttribute(k_sort_pairs, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) != cudaSuccess ||
        cudaOccupancyMaxActiveClusters(&fits, k_sort_pairs, &cfg) != cudaSuccess) {
        cudaGetLastError();
        fits = 0;
    }
    n = fits > 0 ? kSortCtas : 8;
    cache[dev].store(n, std::memory_order_relaxed);
    return n;
}

cudaError_t launch_sort_pairs(const int32_t* ids, int32_t* counts, int32_t* offsets, int32_t* perm, int32_t* inv, int P,
                              int E, cudaStream_t s) {
    int n = 1;
    while (n < kSortCtas && P > 1024 * n) n *= 2;
    if (n > 8) n = sort_ctas();
    const int64_t per = ((int64_t)P + n * kSortWarps - 1) / (n * kSortWarps);
    const int seg = (int)((per + 31) / 32 * 32);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(n);
    cfg.blockDim = dim3(32 * kSortWarps);
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = n;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    cudaError_t e;
    MOE_LAUNCH(MOE_KERNEL_SORT_PAIRS, s, (e = cudaLaunchKernelEx(&cfg, k_sort_pairs, ids, counts, offsets, perm, inv, P, E, seg)));
    return e;
}

// ---------------------------------------------------------------------------------------
// spread and gather. TPT threads take a token: a warp, or a CTA of 256.

constexpr int kSlots = 8;  // K, at most

// Sum over the TPT threads of a token of v[k]; thread 0 .. K - 1 of the token stores it.
template <int TPT>
__device__ __forceinline__ void store_dots(float (&v)[kSlots], float* dst, int K) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
    for (int k = 0; k < kSlots; ++k)
        if (k < K) v[k] = warp_sum(v[k]);
    if (TPT == 32) {
#pragma unroll
        for (int k = 0; k < kSlots; ++k)
            if (k < K && lane == k) dst[k] = v[k];
    } else {
        __shared__ float part[TPT / 32][kSlots];
        if (lane == 0)
#pragma unroll
            for (int k = 0; k < kSlots; ++k) part[warp][k] = v[k];
        __syncthreads();
        if ((int)threadIdx.x < K) {
            float sum = 0.f;
#pragma unroll
            for (int w = 0; w < TPT / 32; ++w) sum += part[w][threadIdx.x];
            dst[threadIdx.x] = sum;
        }
    }
}

// What a thread moves at once: 16 bytes, or what rows start on: 8, 4, one element.
template <int BYTES>
struct Words;
template <>
struct Words<8> {
    typedef uint2 type;
};
template <>
struct Words<4> {
    typedef uint32_t type;
};
template <typename T, int VE>
struct Piece {  // VE elements of fewer than 16 bytes
    typedef typename Words<VE * (int)sizeof(T)>::type type;
    static __device__ __forceinline__ type get(const T* p) { return *reinterpret_cast<const type*>(p); }
    static __device__ __forceinline__ void put(T* p, const type& r) { *reinterpret_cast<type*>(p) = r; }
    static __device__ __forceinline__ void values(const type& r, float (&f)[VE]) {
        const Vec<T, VE> v = *reinterpret_cast<const Vec<T, VE>*>(&r);
#pragma unroll
        for (int i = 0; i < VE; ++i) f[i] = to_f(v.v[i]);
    }
    static __device__ __forceinline__ type pack(const float (&f)[VE]) {
        Vec<T, VE> v;
#pragma unroll
        for (int i = 0; i < VE; ++i) v.v[i] = from_f<T>(f[i]);
        return *reinterpret_cast<const type*>(&v);
    }
};
template <typename T, int VE>
struct PieceOf16 {
    typedef Raw type;
    static __device__ __forceinline__ Raw get(const T* p) {
        const uint4 v = *reinterpret_cast<const uint4*>(p);
        return Raw{{v.x, v.y, v.z, v.w}};
    }
    static __device__ __forceinline__ void put(T* p, const Raw& r) { *reinterpret_cast<uint4*>(p) = make_uint4(r.w[0], r.w[1], r.w[2], r.w[3]); }
    static __device__ __forceinline__ void values(const Raw& r, float (&f)[VE]) { RawOf<T>::values(r, f); }
    static __device__ __forceinline__ Raw pack(const float (&f)[VE]) { return RawOf<T>::pack(f); }
};
template <>
struct Piece<bf16, 8> : PieceOf16<bf16, 8> {};
template <>
struct Piece<fp16, 8> : PieceOf16<fp16, 8> {};
template <>
struct Piece<float, 4> : PieceOf16<float, 4> {};
template <typename T>
struct Piece<T, 1> {
    typedef T type;
    static __device__ __forceinline__ T get(const T* p) { return *p; }
    static __device__ __forceinline__ void put(T* p, const T& r) { *p = r; }
    static __device__ __forceinline__ void values(const T& r, float (&f)[1]) { f[0] = to_f(r); }
    static __device__ __forceinline__ T pack(const float (&f)[1]) { return from_f<T>(f[0]); }
};

// (The residual waiting for the sum takes registers of the fourth CTA of 256 on an SM: with it 4096 x 2048 by 8 are gathered in 28.1 us,
// without 30.8 (1024 fp32 30.2 and 32.1). Pieces of one or two elements do better unbound: 42 against 48 us of 2046 bf16, 29 against 32 of 1022 fp32.)
template <typename T, int VE, int TPT, bool GATHER, bool DOTS>
__global__ void __launch_bounds__(256, TPT == 256 && GATHER && !DOTS && VE >= 4 ? 4 : 0) k_exchange(const ExchangeArgs a) {
    typedef Piece<T, VE> P;
    typedef typename P::type V;
    grid_dep_wait();
    grid_dep_launch();
    const int t = (int)(blockIdx.x * (256 / TPT) + threadIdx.x / TPT);
    if (t >= a.T) return;  // (a whole token's threads)
    const int lane = threadIdx.x % TPT;
    const int K = a.K, nv = a.H / VE;
    const int64_t pairs = (int64_t)a.T * K, p = (int64_t)t * K;
    int at[kSlots];
    float w[kSlots], dot[kSlots];
#pragma unroll
    for (int k = 0; k < kSlots; ++k) {
        at[k] = -1;
        w[k] = 1.f;
        dot[k] = 0.f;
        if (k < K) {
            at[k] = a.inv[p + k];
            if (at[k] >= pairs) at[k] = -1;  // (no place: as a dropped slot)
            if (a.w) w[k] = a.w[p + k];
        }
    }
    const T* tok = (const T*)a.tok + (int64_t)t * a.H;
    const T* rows = (const T*)a.rows;
    T* out = (T*)a.out;
    const bool scaled = a.w != nullptr;
    // The residual is added last: with it in the sum from the start every one of the K roundings would be at its size (fp32 error
    // 5.6e-8 of the result against 3.4e-8 for 6 rows of one size with it).
    const bool residual = GATHER && !DOTS && a.tok;
    for (int j = lane * VE; j < nv * VE; j += TPT * VE) {
        V x, r[kSlots];
        float xf[VE];
        if (!GATHER || a.tok) {
            x = P::get(tok + j);
            P::values(x, xf);
        }
        if (GATHER || DOTS) {
#pragma unroll
            for (int k = 0; k < kSlots; ++k)
                if (at[k] >= 0) r[k] = P::get(rows + (int64_t)at[k] * a.H + j);
        }
        float sum[VE];  // (minus zero plus anything is that thing: a token without slots keeps its residual's bits)
        if (GATHER) {
#pragma unroll
            for (int i = 0; i < VE; ++i) sum[i] = residual ? -0.f : 0.f;
        }
#pragma unroll
        for (int k = 0; k < kSlots; ++k)
            if (at[k] >= 0) {
                if (GATHER || DOTS) {
                    float f[VE];
                    P::values(r[k], f);
                    if (DOTS) {
#pragma unroll
                        for (int i = 0; i < VE; ++i) dot[k] = fmaf(xf[i], f[i], dot[k]);
                    }
                    if (GATHER) {
#pragma unroll
                        for (int i = 0; i < VE; ++i) sum[i] = fmaf(w[k], f[i], sum[i]);  // (without weights exact: times one)
                    }
                }
                if (!GATHER) {
                    V o = x;
                    if (scaled) {
                        float y[VE];
#pragma unroll
                        for (int i = 0; i < VE; ++i) y[i] = w[k] * xf[i];
                        o = P::pack(y);
                    }
                    P::put(out + (int64_t)at[k] * a.H + j, o);
                }
            }
        if (residual) {
#pragma unroll
            for (int i = 0; i < VE; ++i) sum[i] += xf[i];
        }
        if (GATHER) P::put(out + (int64_t)t * a.H + j, P::pack(sum));
    }
    if (DOTS) store_dots<TPT>(dot, a.dots + p, K);
}

template <typename T, int VE, bool GATHER, bool DOTS>
static cudaError_t launch_exchange_t(const ExchangeArgs& a, cudaStream_t s) {
    cudaError_t e;
    const int id = GATHER ? MOE_KERNEL_GATHER_ROWS : MOE_KERNEL_SPREAD_ROWS;
    // A CTA to a token where its row has 128 pieces or more, so that half of the threads at least have one: 4864 rows of 2048 bf16 by 8
    // gathered in 30 against 33 us by warps, 1003 of 1541 by elements in 10.5 against 24; of 256, 10 against 5. With dots the CTA's
    // sums cost more than they gain from 8 tokens an SM on (608 tokens 8.2 against 10.5 us, 1216 16.4 against 14.4). Shorter rows too
    // while there are few tokens, whose warps would be on a few SMs (8 tokens of 1000 bf16 by 8 1.9 against 3.9 us, 600 of 512 2.6 against
    // 2.9 and with dots 5.9 against 4.2, 1200 3.4 against 3.1).
    const bool warps = a.H / VE < 128 ? a.T >= (DOTS ? 2 : 4) * a.num_sms : DOTS && a.T >= 8 * a.num_sms;
    if (warps)
        MOE_LAUNCH(id, s, (e = launch_pdl(k_exchange<T, VE, 32, GATHER, DOTS>, dim3((a.T + 7) / 8), dim3(256), 0, s, a)));
    else
        MOE_LAUNCH(id, s, (e = launch_pdl(k_exchange<T, VE, 256, GATHER, DOTS>, dim3(a.T), dim3(256), 0, s, a)));
    return e;
}

template <typename T, bool GATHER>
static cudaError_t launch_exchange(const ExchangeArgs& a, cudaStream_t s) {
    constexpr int VE = 16 / (int)sizeof(T);
    if (a.H % VE == 0)
        return a.dots ? launch_exchange_t<T, VE, GATHER, true>(a, s) : launch_exchange_t<T, VE, GATHER, false>(a, s);
    if (a.H % (VE / 2) == 0)
        return a.dots ? launch_exchange_t<T, VE / 2, GATHER, true>(a, s) : launch_exchange_t<T, VE / 2, GATHER, false>(a, s);
    if (VE == 8 && a.H % 2 == 0)
        return a.dots ? launch_exchange_t<T, 2, GATHER, true>(a, s) : launch_exchange_t<T, 2, GATHER, false>(a, s);
    return a.dots ? launch_exchange_t<T, 1, GATHER, true>(a, s) : launch_exchange_t<T, 1, GATHER, false>(a, s);
}

cudaError_t launch_spread(int32_t dtype, const ExchangeArgs& a, cudaStream_t s) {
    return dtype == MOE_BF16 ? launch_exchange<bf16, false>(a, s) : dtype == MOE_FP16 ? launch_exchange<fp16, false>(a, s) : launch_exchange<float, false>(a, s);
}
cudaError_t launch_gather(int32_t dtype, const ExchangeArgs& a, cudaStream_t s) {
    return dtype == MOE_BF16 ? launch_exchange<bf16, true>(a, s) : dtype == MOE_FP16 ? launch_exchange<fp16, true>(a, s) : launch_exchange<float, true>(a, s);
}

}  // namespace moe
