// w4.cuh -- packed 4-bit weights with group scales: layout, decoding, and the warp-level product.
//
// A matrix [rows, cols] of 4-bit codes stands for w[n, k] = s[n, k / G] * v[n, k] with s in bf16
// and G = 32, 64 or 128 consecutive columns to a scale (include/moe.h, moe_w4_format):
//   INT4     v = code - 8
//   INT4_ZP  v = code - z[n, k / G]
//   E2M1     v = the 4-bit float (sign, two exponent bits, one mantissa bit)
// Every v is exact in bf16, so products v * x are exact in fp32; a group's sum over 32 columns is
// multiplied by the scale in fp32 and added to the row's fp32 sum: nothing is rounded to fewer
// bits before the output.
//
// Layout: strips of 16 rows, each a run of records of 128 columns, so a strip's weights, scales
// and zero points for any column range are one contiguous piece of memory (one bulk copy):
//   1024 bytes of codes: word [row / 8][row % 8][t][c], t, c = 0 .. 3, holds columns
//     32 c + 8 t + e, e = 0 .. 7 (even e in the low half, odd e in the high half)
//   16 x (128 / G) scales, [row][group]; for INT4_ZP then 16 x (128 / G) zero-point bytes
// The order is that of the m16n8k16 A operand: lane 4g + t reads 16 bytes of row g and 16 of row
// g + 8 (conflict-free) and holds, for each 32-column group c, the eight columns 32 c + 8 t + e as
// two MMA steps; its B operand is then eight consecutive elements of a token row. A merged
// gate_up matrix puts 8 gate rows and the 8 matching up rows into a strip, so one lane's
// accumulators hold the gate and the up value of the same feature.
#pragma once

#include <cuda_bf16.h>
#include <stdint.h>

#include "ring.cuh"

namespace moe {

constexpr int kW4Strip = 16;    // rows of a strip
constexpr int kW4Cols = 128;    // columns of a record
constexpr int kW4Codes = 1024;  // bytes of codes in a record

__host__ __device__ constexpr int w4_record_bytes(int format, int group) {
    return kW4Codes + 16 * (kW4Cols / group) * (format == MOE_W4_INT4_ZP ? 3 : 2);
}

// Bytes of one packed matrix.
__host__ __device__ inline size_t w4_matrix_bytes(int format, int group, int rows, int cols) {
    return (size_t)((rows + kW4Strip - 1) / kW4Strip) * ((cols + kW4Cols - 1) / kW4Cols) *
           w4_record_bytes(format, group);
}

#ifdef __CUDACC__

template <int FMT, int G>
struct W4Rec {
    static constexpr int kGroups = kW4Cols / G;  // groups of a row within a record
    static constexpr int kBytes = w4_record_bytes(FMT, G);
    static constexpr int kScales = kW4Codes;
    static constexpr int kZeros = kW4Codes + 32 * kGroups;
};

__device__ __forceinline__ uint32_t bf2_sub(uint32_t a, uint32_t b) {
    const __nv_bfloat162 r = __hsub2(*reinterpret_cast<__nv_bfloat162*>(&a), *reinterpret_cast<__nv_bfloat162*>(&b));
    return *reinterpret_cast<const uint32_t*>(&r);
}
__device__ __forceinline__ uint32_t bf2_mul(uint32_t a, uint32_t b) {
    const __nv_bfloat162 r = __hmul2(*reinterpret_cast<__nv_bfloat162*>(&a), *reinterpret_cast<__nv_bfloat162*>(&b));
    return *reinterpret_cast<const uint32_t*>(&r);
}

// The eight values of a word as four bf16 pairs, columns (0, 1), (2, 3), (4, 5), (6, 7); exact.
// Integer codes: 0x43 in the upper byte of a bf16 and the code in the lower bits is 128 + code;
// `bias` holds 128 + the zero point in both halves. E2M1: the three magnitude bits put at the
// lowest exponent bits and the highest mantissa bit read as the value times 2^-126 (0.5 as a
// subnormal), so one multiplication by 2^126 gives it; the packed bit order makes that two
// instructions a pair for three of the four (include/moe.h).
template <int FMT>
__device__ __forceinline__ void w4_decode(uint32_t w, uint32_t bias, uint32_t (&p)[4]) {
    if (FMT == MOE_W4_E2M1) {
        constexpr uint32_t M = 0x81c081c0u;
        p[0] = w & M;
        p[1] = (w << 3) & M;
        p[2] = (w << 6) & M;
        p[3] = ((w >> 5) & 0x01400140u) | ((w >> 3) & 0x00800080u) | ((w << 1) & 0x80008000u);
#pragma unroll
        for (int i = 0; i < 4; ++i) p[i] = bf2_mul(p[i], 0x7e807e80u);
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) p[i] = bf2_sub(((w >> (4 * i)) & 0x000f000fu) | 0x43004300u, bias);
    }
}

// One record's share of a lane: the codes, scales and zero points of rows g and g + 8, as they lie
// in shared memory.
template <int FMT, int G>
struct W4Frag {
    uint4 lo, hi;
    uint32_t s[2][W4Rec<FMT, G>::kGroups == 4 ? 2 : 1];
    uint32_t z[2];
};

template <int FMT, int G>
__device__ __forceinline__ void w4_load(uint32_t rec, int lane, W4Frag<FMT, G>& f) {
    constexpr int N = W4Rec<FMT, G>::kGroups;
    f.lo = lds128_smem(rec + (uint32_t)lane * 16u);
    f.hi = lds128_smem(rec + 512u + (uint32_t)lane * 16u);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const uint32_t row = (uint32_t)(lane >> 2) + 8u * h, at = rec + W4Rec<FMT, G>::kScales + row * (2u * N);
        if constexpr (N == 4) {
            asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(f.s[h][0]), "=r"(f.s[h][1]) : "r"(at));
        } else if constexpr (N == 2) {
            asm volatile("ld.shared.u32 %0, [%1];" : "=r"(f.s[h][0]) : "r"(at));
        } else {
            uint16_t v;
            asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(at));
            f.s[h][0] = v;
        }
        f.z[h] = 0;
        if (FMT == MOE_W4_INT4_ZP) {
            const uint32_t za = rec + W4Rec<FMT, G>::kZeros + row * N;
            if (N == 4)
                asm volatile("ld.shared.u32 %0, [%1];" : "=r"(f.z[h]) : "r"(za));
            else if (N == 2) {
                uint16_t v;
                asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(za));
                f.z[h] = v;
            } else
                asm volatile("ld.shared.u8 %0, [%1];" : "=r"(f.z[h]) : "r"(za));
        }
    }
}

template <int FMT, int G>
__device__ __forceinline__ float w4_scale(const W4Frag<FMT, G>& f, int h, int gi) {
    return (gi & 1) ? bf_hi(f.s[h][gi >> 1]) : bf_lo(f.s[h][gi >> 1]);
}
template <int FMT, int G>
__device__ __forceinline__ uint32_t w4_bias(const W4Frag<FMT, G>& f, int h, int gi) {
    if (FMT != MOE_W4_INT4_ZP) return 0x43084308u;
    return 0x43004300u | (((f.z[h] >> (8 * gi)) & 0xffu) * 0x00010001u);
}

// acc += one record (16 rows by 128 columns) times NT tiles of 8 tokens. b[n][4 c + i] are the B
// operands of lane 4g + t: token g of tile n, columns 32 c + 8 t + 2 i, + 1. acc is the m16n8
// accumulator of each tile: rows g (0, 1) and g + 8 (2, 3), tokens 2t (0, 2) and 2t + 1 (1, 3).
// Each group's sum starts at zero and is scaled in fp32.
template <int FMT, int G, int NT>
__device__ __forceinline__ void w4_mma_record(const W4Frag<FMT, G>& f, const uint32_t (&b)[NT][16], float (&acc)[NT][4]) {
    const uint32_t w0[4] = {f.lo.x, f.lo.y, f.lo.z, f.lo.w}, w1[4] = {f.hi.x, f.hi.y, f.hi.z, f.hi.w};
    float d[NT][4];
#pragma unroll
    for (int c = 0; c < 4; ++c) {
        const int gi = c * 32 / G;
        uint32_t p[4], q[4];
        w4_decode<FMT>(w0[c], w4_bias(f, 0, gi), p);
        w4_decode<FMT>(w1[c], w4_bias(f, 1, gi), q);
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            if (c * 32 % G == 0)
                mma16816_first(d[n], p[0], q[0], p[1], q[1], b[n][4 * c], b[n][4 * c + 1]);
            else
                mma16816(d[n], p[0], q[0], p[1], q[1], b[n][4 * c], b[n][4 * c + 1]);
            mma16816(d[n], p[2], q[2], p[3], q[3], b[n][4 * c + 2], b[n][4 * c + 3]);
        }
        if ((c + 1) * 32 % G == 0) {
            const float s0 = w4_scale(f, 0, gi), s1 = w4_scale(f, 1, gi);
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                acc[n][0] = fmaf(s0, d[n][0], acc[n][0]);
                acc[n][1] = fmaf(s0, d[n][1], acc[n][1]);
                acc[n][2] = fmaf(s1, d[n][2], acc[n][2]);
                acc[n][3] = fmaf(s1, d[n][3], acc[n][3]);
            }
        }
    }
}

#endif

}  // namespace moe
