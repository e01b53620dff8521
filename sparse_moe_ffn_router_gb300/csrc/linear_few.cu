// linear_few.cu -- the linear layers' forward pass for a handful of rows (decode): a warp to a feature.
//
// out = act(x . W_e^T + b_e) + residual. With so few rows the weights' way from HBM is all there is: a warp streams the rows
// of W of one to four features (of a gated one, gate and up) with 16-byte loads, eight of each kind on their way at once,
// and keeps the sums of up to RB rows of x in registers; x comes from L1. No tensor maps, barriers or tensor memory: a
// launch, one pass, warp sums. Rows of experts are taken one at a time: two rows of one expert read its matrix twice, the second
// time from L2. Measured: one row, 2048 x 2048 3.6 us (weights in L2), 8192 x 4096 12.3 us = 5.5 TB/s; 8 experts'
// 1024 x 2048 7.2 us = 4.7 TB/s.
#include "linear.cuh"

namespace moe {

constexpr int kFewWarps = 8, kFewBatches = kFewRows;
static_assert(32 * kFewWarps >= kLinMaxE, "an expert a thread");

template <typename T>
__device__ __forceinline__ float dot_chunk(const uint4& w, const uint4& x, float acc) {
    const T* a = reinterpret_cast<const T*>(&w);
    const T* b = reinterpret_cast<const T*>(&x);
#pragma unroll
    for (int i = 0; i < 8; ++i) acc = fmaf(to_f(a[i]), to_f(b[i]), acc);
    return acc;
}
template <>
__device__ __forceinline__ float dot_chunk<bf16>(const uint4& w, const uint4& x, float acc) { return dot8_bf16(w, x, acc); }

template <typename T, bool GATED, int RB, int FW>
__global__ void __launch_bounds__(32 * kFewWarps) k_linear_few(const T* __restrict__ x, const T* __restrict__ w, const LinView a) {
    __shared__ int list[kFewBatches][3];  // expert, first row, rows
    __shared__ int count;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    grid_dep_wait();
    grid_dep_launch();
    int batches = (a.T + RB - 1) / RB;
    if (a.offsets) {
        // one expert a thread, so that the bounds are one load's wait
        __shared__ int sums[kFewWarps];
        const int e = threadIdx.x;
        int o0 = 0, o1 = 0;
        if (e < a.E) {
            const int p0 = a.offsets[e], p1 = a.offsets[e + 1];
            o0 = min(max(p0, 0), a.T);
            o1 = min(max(p1, 0), a.T);
            if (o0 != p0 || o1 != p1 || o1 < o0) atomicOr(a.err, ERR_BAD_ROUTE);
        }
        const int mine = (max(o1 - o0, 0) + RB - 1) / RB;
        int v = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, v, o);
            if (lane >= o) v += y;
        }
        if (lane == 31) sums[warp] = v;
        __syncthreads();
        int n = 0, all = 0;
#pragma unroll
        for (int i = 0; i < kFewWarps; ++i) {
            n += i < warp ? sums[i] : 0;
            all += sums[i];
        }
        for (int i = 0; i < mine; ++i) {
            const int at = n + v - mine + i;
            if (at < kFewBatches) {  // (offsets in order give no more)
                list[at][0] = e;
                list[at][1] = o0 + i * RB;
                list[at][2] = min(o1 - o0 - i * RB, RB);
            }
        }
        if (threadIdx.x == 0) count = min(all, kFewBatches);
        __syncthreads();
        batches = count;
    }
    const int chunks = a.C / 8, per = (a.F + FW - 1) / FW;  // FW features a warp
    const int64_t items = (int64_t)batches * per;
    for (int64_t it = (int64_t)blockIdx.x * kFewWarps + warp; it < items; it += (int64_t)gridDim.x * kFewWarps) {
        const int b = (int)(it / per), f0 = (int)(it - (int64_t)b * per) * FW;
        int e = 0, row = b * RB, rows = min(a.T - row, RB);
        if (a.offsets) {
            e = list[b][0];
            row = list[b][1];
            rows = list[b][2];
        }
        const uint4* wg = reinterpret_cast<const uint4*>(w + ((int64_t)e * a.N + f0) * a.C);
        const uint4* wu = reinterpret_cast<const uint4*>(w + ((int64_t)e * a.N + a.F + f0) * a.C);  // (gated)
        const uint4* px = reinterpret_cast<const uint4*>(x + (int64_t)row * a.C);
        float s[FW][RB], u[FW][RB];
#pragma unroll
        for (int k = 0; k < FW; ++k)
#pragma unroll
            for (int r = 0; r < RB; ++r) s[k][r] = u[k][r] = 0.f;
        constexpr int U = 8 / FW;  // chunks of a feature on their way
        for (int c0 = lane; c0 < chunks; c0 += 32 * U) {
            uint4 vg[FW][U], vu[FW][U];
#pragma unroll
            for (int k = 0; k < FW; ++k)
#pragma unroll
                for (int i = 0; i < U; ++i) {
                    const int c = c0 + 32 * i;
                    if (c < chunks && f0 + k < a.F) {
                        vg[k][i] = ld_stream(wg + (int64_t)k * chunks + c);
                        if (GATED) vu[k][i] = ld_stream(wu + (int64_t)k * chunks + c);
                    }
                }
#pragma unroll
            for (int i = 0; i < U; ++i) {
                const int c = c0 + 32 * i;
                if (c < chunks) {
#pragma unroll
                    for (int r = 0; r < RB; ++r)
                        if (r < rows) {
                            const uint4 xv = ld_ro(px + (int64_t)r * chunks + c);
#pragma unroll
                            for (int k = 0; k < FW; ++k) {
                                s[k][r] = dot_chunk<T>(vg[k][i], xv, s[k][r]);
                                if (GATED) u[k][r] = dot_chunk<T>(vu[k][i], xv, u[k][r]);
                            }
                        }
                }
            }
        }
        float v = 0.f, up = 0.f;  // lane r * FW + k: row r, feature f0 + k
#pragma unroll
        for (int r = 0; r < RB; ++r)
            if (r < rows)
#pragma unroll
                for (int k = 0; k < FW; ++k) {
                    const float t = warp_sum(s[k][r]);
                    if (lane == r * FW + k) v = t;
                    if (GATED) {
                        const float t2 = warp_sum(u[k][r]);
                        if (lane == r * FW + k) up = t2;
                    }
                }
        const int f = f0 + lane % FW;
        if (lane < rows * FW && f < a.F) {
            const int64_t ro = row + lane / FW, o = ro * a.F + f, oz = ro * a.N + f;
            if (a.bias) {
                const T* bias = reinterpret_cast<const T*>(a.bias) + (int64_t)e * a.N + f;
                v += to_f(bias[0]);
                if (GATED) up += to_f(bias[a.F]);
            }
            if (a.z) {
                reinterpret_cast<T*>(a.z)[oz] = from_f<T>(v);
                if (GATED) reinterpret_cast<T*>(a.z)[oz + a.F] = from_f<T>(up);
            }
            float y[1] = {v};
            if (GATED) y[0] = v * lin_sigmoid(v) * up;
            else lin_act<1>(a.act, y);
            if (a.residual) y[0] += to_f(reinterpret_cast<const T*>(a.residual)[o]);
            reinterpret_cast<T*>(a.out)[o] = from_f<T>(y[0]);
        }
    }
}

template <typename T, bool GATED, int RB, int FW>
static cudaError_t launch_few_k(const void* x, const void* w, const LinView& v, int num_sms, cudaStream_t s) {
    const int64_t items = (int64_t)(v.offsets ? v.T : 1) * ((v.F + FW - 1) / FW), ctas = (items + kFewWarps - 1) / kFewWarps, most = (int64_t)num_sms * 8;
    return launch_pdl(k_linear_few<T, GATED, RB, FW>, dim3((unsigned)(ctas < most ? ctas : most)), dim3(32 * kFewWarps), 0, s, (const T*)x, (const T*)w, v);
}

// Rows of a batch: as the call has, experts' rows one by one. Features of a warp: as many as keep eight chunks a lane
// of the feature's row (K columns) in one go.
template <typename T, bool GATED>
static cudaError_t launch_few_t(const void* x, const void* w, const LinView& v, int num_sms, cudaStream_t s) {
    const int rb = v.offsets ? 1 : v.T, fw = v.C <= 512 ? 4 : v.C <= 1024 ? 2 : 1;
    if (rb == 1) {
        if (fw == 4) return launch_few_k<T, GATED, 1, 4>(x, w, v, num_sms, s);
        if (fw == 2) return launch_few_k<T, GATED, 1, 2>(x, w, v, num_sms, s);
        return launch_few_k<T, GATED, 1, 1>(x, w, v, num_sms, s);
    }
    if (rb <= 4) return fw > 1 ? launch_few_k<T, GATED, 4, 2>(x, w, v, num_sms, s) : launch_few_k<T, GATED, 4, 1>(x, w, v, num_sms, s);
    return fw > 1 ? launch_few_k<T, GATED, 8, 2>(x, w, v, num_sms, s) : launch_few_k<T, GATED, 8, 1>(x, w, v, num_sms, s);
}

cudaError_t launch_few(int32_t dtype, bool gated, const void* x, const void* w, const LinView& v, int num_sms, cudaStream_t s) {
    if (dtype == MOE_FP16) return gated ? launch_few_t<fp16, true>(x, w, v, num_sms, s) : launch_few_t<fp16, false>(x, w, v, num_sms, s);
    return gated ? launch_few_t<bf16, true>(x, w, v, num_sms, s) : launch_few_t<bf16, false>(x, w, v, num_sms, s);
}

}  // namespace moe
