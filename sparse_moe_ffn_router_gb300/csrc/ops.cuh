// ops.cuh -- what the exchange, norm and linear operators share: element types, vectors of them, and
// the argument blocks passed from the C-ABI entry points to the launches.
#pragma once

#include <atomic>

#include <cuda_fp16.h>

#include "launch.h"

namespace moe {

typedef __half fp16;

// Bytes of an element of moe_dtype, 0 for an unknown one.
inline int elem_size(int32_t dtype) { return dtype == MOE_BF16 || dtype == MOE_FP16 ? 2 : dtype == MOE_FP32 ? 4 : 0; }

#ifdef __CUDACC__
__device__ __forceinline__ float to_f(float v) { return v; }
__device__ __forceinline__ float to_f(bf16 v) { return __bfloat162float(v); }
__device__ __forceinline__ float to_f(fp16 v) { return __half2float(v); }
template <typename T>
__device__ __forceinline__ T from_f(float v);
template <>
__device__ __forceinline__ float from_f<float>(float v) { return v; }
template <>
__device__ __forceinline__ bf16 from_f<bf16>(float v) { return __float2bfloat16_rn(v); }
template <>
__device__ __forceinline__ fp16 from_f<fp16>(float v) { return __float2half_rn(v); }

// VE elements side by side, as one load or store moves them where their rows start on as many bytes.
template <typename T, int VE>
struct alignas(sizeof(T) * VE) Vec {
    T v[VE];
};
// Two fp32 operations in one instruction.
struct F2 {
    uint64_t v;
};
__device__ __forceinline__ F2 f2(float x, float y) {
    F2 r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r.v) : "f"(x), "f"(y));
    return r;
}
__device__ __forceinline__ void f2_split(F2 a, float& x, float& y) { asm("mov.b64 {%0, %1}, %2;" : "=f"(x), "=f"(y) : "l"(a.v)); }
__device__ __forceinline__ F2 f2_fma(F2 a, F2 b, F2 c) {
    F2 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.v) : "l"(a.v), "l"(b.v), "l"(c.v));
    return r;
}
__device__ __forceinline__ F2 f2_mul(F2 a, F2 b) {
    F2 r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
    return r;
}
__device__ __forceinline__ F2 f2_both(float x) { return f2(x, x); }

// 16 bytes of a row as they lie in memory, and their values. (Held as words: as 16-bit elements they would take twice
// the registers between the two ways of loading them.)
struct Raw {
    uint32_t w[4];
};
template <typename T>
struct RawOf;
template <>
struct RawOf<float> {
    static __device__ __forceinline__ void values(const Raw& r, float (&f)[4]) {
#pragma unroll
        for (int i = 0; i < 4; ++i) f[i] = __uint_as_float(r.w[i]);
    }
    static __device__ __forceinline__ Raw pack(const float (&f)[4]) {
        return Raw{{__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3])}};
    }
};
template <>
struct RawOf<bf16> {
    static __device__ __forceinline__ void values(const Raw& r, float (&f)[8]) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            f[2 * i] = bf_lo(r.w[i]);
            f[2 * i + 1] = bf_hi(r.w[i]);
        }
    }
    static __device__ __forceinline__ Raw pack(const float (&f)[8]) {
        return Raw{{pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]), pack_bf16x2(f[6], f[7])}};
    }
};
template <>
struct RawOf<fp16> {
    static __device__ __forceinline__ void values(const Raw& r, float (&f)[8]) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 v = __half22float2(*reinterpret_cast<const __half2*>(&r.w[i]));
            f[2 * i] = v.x;
            f[2 * i + 1] = v.y;
        }
    }
    static __device__ __forceinline__ Raw pack(const float (&f)[8]) {
        Raw r;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const __half2 h = __floats2half2_rn(f[2 * i], f[2 * i + 1]);
            r.w[i] = *reinterpret_cast<const uint32_t*>(&h);
        }
        return r;
    }
};
#endif

// Lets a kernel have `bytes` of dynamic shared memory, once for each device (done: which have it). Two host threads may make their first
// calls at the same time: then both ask for it.
template <typename Kernel>
cudaError_t allow_shared(Kernel* kernel, int bytes, std::atomic<bool> (&done)[64]) {
    int dev = 0;
    cudaGetDevice(&dev);
    const bool known = dev >= 0 && dev < 64;
    if (known && done[dev].load(std::memory_order_acquire)) return cudaSuccess;
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e == cudaSuccess && known) done[dev].store(true, std::memory_order_release);
    return e;
}

// ---- exchange (exchange.cu): tokens [T, H], rows [T * K, H], inv [T * K]
struct ExchangeArgs {
    const void* tok;       // token side, read: x, the residual, or the other factor of the dots
    const void* rows;      // row side, read
    const int32_t* inv;
    const float* w;        // [T, K] or NULL
    void* out;             // rows (spread) or tokens (gather)
    float* dots;           // [T, K] or NULL
    int T, K, H;
    int num_sms;
};
cudaError_t launch_sort_pairs(const int32_t* ids, int32_t* counts, int32_t* offsets, int32_t* perm, int32_t* inv, int P,
                              int E, cudaStream_t s);
// out[inv[t, k]] = (w) * tok[t]; dots[t, k] = tok[t] . rows[inv[t, k]]
cudaError_t launch_spread(int32_t dtype, const ExchangeArgs& a, cudaStream_t s);
// out[t] = (residual = tok when there are no dots) + sum_k (w) * rows[inv[t, k]]; dots as above
cudaError_t launch_gather(int32_t dtype, const ExchangeArgs& a, cudaStream_t s);

// ---- norm (norm.cuh)
struct NormArgs {
    moe_norm_dims d;
    const void *y, *residual, *gate, *gamma_post, *gamma_pre;
    void *s, *xn;  // forward results
    const void *s_in, *ds, *dxn;
    void *dresidual, *dy, *dgate, *dgamma_post, *dgamma_pre;
    float* part;  // [blocks, 3, H]
    int num_sms;
};
// CTAs of the backward pass over T rows, at most: one for each row or few, rounded up to 8 so that the rows of a CTA can
// begin at the same place within a vector.
constexpr int kNormBlocks = 304;
inline int64_t norm_blocks(int64_t T) { return T > kNormBlocks - 8 ? kNormBlocks : (T + 7) / 8 * 8; }
cudaError_t launch_norm_bf16(const NormArgs& a, cudaStream_t s, bool backward);
cudaError_t launch_norm_fp16(const NormArgs& a, cudaStream_t s, bool backward);
cudaError_t launch_norm_fp32(const NormArgs& a, cudaStream_t s, bool backward);
inline cudaError_t launch_norm(const NormArgs& a, cudaStream_t s, bool backward) {
    return a.d.dtype == MOE_BF16 ? launch_norm_bf16(a, s, backward) : a.d.dtype == MOE_FP16 ? launch_norm_fp16(a, s, backward) : launch_norm_fp32(a, s, backward);
}

// ---- linear (linear.cu)
struct LinearArgs {
    moe_linear_dims d;
    const void *x, *w, *bias, *residual;
    const int32_t* offsets;  // [E + 1], or NULL: all T rows are the one matrix's
    void *out, *z;           // forward results
    const void *z_in, *dout;
    void *dx, *dw, *dbias;
    void* dz;                // [T, N rounded up to 8]: gradient of the pre-activation
    float* part;             // [ceil(T / chunk) + E, N]: column sums of a chunk's rows of one expert
    int chunk;               // rows of a chunk: dz_rows or more
    uint32_t* err;
    uint64_t wait_ns;
    int num_sms;
    int suppress;            // testing aid: CTA 0 of the forward kernel never loads its first stage
};
// Rows of a chunk, at least. Of experts with a handful of rows each 4, as a CTA takes the experts in its chunk one after another (35 rows of
// 150 experts, 317 x 456: the whole backward call 37 against 87 us).
constexpr int dz_rows(int64_t T, int E) { return E > 1 && T <= 8 * (int64_t)E ? 4 : 32; }
cudaError_t launch_linear(const LinearArgs& a, cudaStream_t s);
cudaError_t launch_linear_backward(const LinearArgs& a, cudaStream_t s);
// A tensor map for TMA with 128-byte (or 64-byte) swizzle and zeros outside: dims and box innermost first, strides in
// bytes of dims 1 .. rank - 1.
bool encode_map(CUtensorMap* m, int32_t dtype, const void* base, int rank, const uint64_t* dims, const uint64_t* strides,
                const uint32_t* box, bool swizzle64 = false);

// SMs of the current device, the time limit of bounded device waits, the signal held back in tests (api.cu).
int device_sms();
uint64_t device_wait_ns();
int device_suppress();

}  // namespace moe
