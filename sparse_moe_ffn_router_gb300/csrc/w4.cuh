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
// Weight rows and token rows, at most: a row index rounded up to a tile (256 rows at most) still fits an int.
constexpr int kW4MaxRows = 0x7fffffff - 255;

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

// Packed bf16 sums and products, one instruction each (the header functions take more).
__device__ __forceinline__ uint32_t bf2_add(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("add.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
__device__ __forceinline__ uint32_t bf2_fma(uint32_t a, uint32_t b, uint32_t c) {
    uint32_t r;
    asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(a), "r"(b), "r"(c));
    return r;
}
__device__ __forceinline__ uint32_t bf2_mul(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

// The eight values of a word as four bf16 pairs, columns (0, 1), (2, 3), (4, 5), (6, 7); exact.
// Integer codes: 0x43 in the upper byte of a bf16 and the code in the lower bits is 128 + code;
// `bias` holds -(128 + the zero point) in both halves. E2M1: the three magnitude bits put at the
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
        for (int i = 0; i < 4; ++i) p[i] = bf2_add(((w >> (4 * i)) & 0x000f000fu) | 0x43004300u, bias);
    }
}

// The values as the MMA kernels use them: integer codes a quarter (kUnfold = 4 undoes it on the sums),
// which takes two shifts a word less than w4_decode. Codes 0 and 2 of a half go through 128 + code,
// times 1/4. Codes 1 and 3, in bits 4 .. 7, are read as they lie: a bf16 with only its lowest exponent
// bit and its three highest mantissa bits is linear in them (subnormals and the first binade have one
// spacing), code * 2^-129; times 2^127 that is code / 4. Every value is exact. b0, b1: -(128 + zero
// point) / 4 and -(zero point) / 4 in both halves.
template <int FMT>
struct W4Fold {
    static constexpr float kUnfold = FMT == MOE_W4_E2M1 ? 1.f : 4.f;
};
template <int FMT>
__device__ __forceinline__ void w4_decode_fold(uint32_t w, uint32_t b0, uint32_t b1, uint32_t (&p)[4]) {
    if (FMT == MOE_W4_E2M1) {
        w4_decode<FMT>(w, 0u, p);
    } else {
        const uint32_t h = w >> 8;
        p[0] = bf2_fma((w & 0x000f000fu) | 0x43004300u, 0x3e803e80u, b0);
        p[1] = bf2_fma(w & 0x00f000f0u, 0x7f007f00u, b1);
        p[2] = bf2_fma((h & 0x000f000fu) | 0x43004300u, 0x3e803e80u, b0);
        p[3] = bf2_fma(h & 0x00f000f0u, 0x7f007f00u, b1);
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

// Shared-memory loads at a register address and a constant offset (no address arithmetic a load).
template <int OFF>
__device__ __forceinline__ uint4 lds128_at(uint32_t addr) {
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4 + %5];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr), "n"(OFF) : "memory");
    return v;
}

// at: of the record + 16 * lane; meta: of the record + 2 * N * (lane / 4) (scales), zmeta: + N * (lane / 4).
template <int FMT, int G, int OFF>
__device__ __forceinline__ void w4_load_at(uint32_t at, uint32_t meta, uint32_t zmeta, W4Frag<FMT, G>& f) {
    constexpr int N = W4Rec<FMT, G>::kGroups, kS = OFF + W4Rec<FMT, G>::kScales, kZ = OFF + W4Rec<FMT, G>::kZeros;
    f.lo = lds128_at<OFF>(at);
    f.hi = lds128_at<OFF + 512>(at);
    if constexpr (N == 4) {
        asm volatile("ld.shared.v2.u32 {%0, %1}, [%2 + %3];" : "=r"(f.s[0][0]), "=r"(f.s[0][1]) : "r"(meta), "n"(kS));
        asm volatile("ld.shared.v2.u32 {%0, %1}, [%2 + %3];" : "=r"(f.s[1][0]), "=r"(f.s[1][1]) : "r"(meta), "n"(kS + 16 * N));
    } else if constexpr (N == 2) {
        asm volatile("ld.shared.u32 %0, [%1 + %2];" : "=r"(f.s[0][0]) : "r"(meta), "n"(kS));
        asm volatile("ld.shared.u32 %0, [%1 + %2];" : "=r"(f.s[1][0]) : "r"(meta), "n"(kS + 16 * N));
    } else {
        uint16_t v0, v1;
        asm volatile("ld.shared.u16 %0, [%1 + %2];" : "=h"(v0) : "r"(meta), "n"(kS));
        asm volatile("ld.shared.u16 %0, [%1 + %2];" : "=h"(v1) : "r"(meta), "n"(kS + 16 * N));
        f.s[0][0] = v0;
        f.s[1][0] = v1;
    }
    f.z[0] = f.z[1] = 0;
    if constexpr (FMT == MOE_W4_INT4_ZP) {
        if constexpr (N == 4) {
            asm volatile("ld.shared.u32 %0, [%1 + %2];" : "=r"(f.z[0]) : "r"(zmeta), "n"(kZ));
            asm volatile("ld.shared.u32 %0, [%1 + %2];" : "=r"(f.z[1]) : "r"(zmeta), "n"(kZ + 8 * N));
        } else if constexpr (N == 2) {
            uint16_t v0, v1;
            asm volatile("ld.shared.u16 %0, [%1 + %2];" : "=h"(v0) : "r"(zmeta), "n"(kZ));
            asm volatile("ld.shared.u16 %0, [%1 + %2];" : "=h"(v1) : "r"(zmeta), "n"(kZ + 8 * N));
            f.z[0] = v0;
            f.z[1] = v1;
        } else {
            asm volatile("ld.shared.u8 %0, [%1 + %2];" : "=r"(f.z[0]) : "r"(zmeta), "n"(kZ));
            asm volatile("ld.shared.u8 %0, [%1 + %2];" : "=r"(f.z[1]) : "r"(zmeta), "n"(kZ + 8 * N));
        }
    }
}

template <int FMT, int G>
__device__ __forceinline__ float w4_scale(const W4Frag<FMT, G>& f, int h, int gi) {
    return (gi & 1) ? bf_hi(f.s[h][gi >> 1]) : bf_lo(f.s[h][gi >> 1]);
}
// m16n8k16 bf16 MMAs, fp32 accumulate (not volatile: the compiler may interleave independent records).
__device__ __forceinline__ void w4_mma(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                       uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void w4_mma_first(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                             uint32_t b1) {  // onto a zero accumulator
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}

// b0 and b1 of w4_decode_fold.
template <int FMT>
__device__ __forceinline__ void w4_bias_fold(uint32_t z, int gi, uint32_t& b0, uint32_t& b1) {
    b0 = 0xc208c208u;  // -34
    b1 = 0xc000c000u;  // -2
    if (FMT == MOE_W4_INT4_ZP) {
        b0 = __byte_perm(z, 0xc2u, 0x4040u | (uint32_t)(gi << 8) | (uint32_t)gi);
        b1 = bf2_add(b0, 0x42004200u);  // + 32
    }
}

// acc += NR records (16 rows by 128 columns each) times a tile of 8 tokens, W4Fold::kUnfold times too
// small. b[r][4 c + i] are the B operands of lane 4g + t: token g, columns 32 c + 8 t + 2 i, + 1 of record
// r. acc is the m16n8 accumulator: rows g (0, 1) and g + 8 (2, 3), tokens 2t (0, 2) and 2t + 1 (1, 3).
// Each group's sum starts at zero and is scaled in fp32. The records' chains of dependent MMAs are
// interleaved, so that one fills the other's latency.
template <int FMT, int G, int NR>
__device__ __forceinline__ void w4_mma_records(const W4Frag<FMT, G> (&f)[NR], const uint32_t (&b)[NR][16], float (&acc)[4]) {
    float d[NR][4];
#pragma unroll
    for (int c = 0; c < 4; ++c) {
        const int gi = c * 32 / G;
        uint32_t p[NR][4], q[NR][4];
#pragma unroll
        for (int r = 0; r < NR; ++r) {
            const uint32_t w0 = c == 0 ? f[r].lo.x : c == 1 ? f[r].lo.y : c == 2 ? f[r].lo.z : f[r].lo.w;
            const uint32_t w1 = c == 0 ? f[r].hi.x : c == 1 ? f[r].hi.y : c == 2 ? f[r].hi.z : f[r].hi.w;
            uint32_t b00, b01, b10, b11;
            w4_bias_fold<FMT>(f[r].z[0], gi, b00, b01);
            w4_bias_fold<FMT>(f[r].z[1], gi, b10, b11);
            w4_decode_fold<FMT>(w0, b00, b01, p[r]);
            w4_decode_fold<FMT>(w1, b10, b11, q[r]);
        }
#pragma unroll
        for (int r = 0; r < NR; ++r) {
            if (c * 32 % G == 0)
                w4_mma_first(d[r], p[r][0], q[r][0], p[r][1], q[r][1], b[r][4 * c], b[r][4 * c + 1]);
            else
                w4_mma(d[r], p[r][0], q[r][0], p[r][1], q[r][1], b[r][4 * c], b[r][4 * c + 1]);
        }
#pragma unroll
        for (int r = 0; r < NR; ++r) w4_mma(d[r], p[r][2], q[r][2], p[r][3], q[r][3], b[r][4 * c + 2], b[r][4 * c + 3]);
        if ((c + 1) * 32 % G == 0) {
#pragma unroll
            for (int r = 0; r < NR; ++r) {
                const float s0 = w4_scale(f[r], 0, gi), s1 = w4_scale(f[r], 1, gi);
                acc[0] = fmaf(s0, d[r][0], acc[0]);
                acc[1] = fmaf(s0, d[r][1], acc[1]);
                acc[2] = fmaf(s1, d[r][2], acc[2]);
                acc[3] = fmaf(s1, d[r][3], acc[3]);
            }
        }
    }
}

// acc += up to two consecutive records in shared memory times a tile.
template <int FMT, int G>
__device__ __forceinline__ void w4_records(uint32_t rec, int n, const uint32_t (&b)[2][16], float (&acc)[4], int lane) {
    constexpr uint32_t N = W4Rec<FMT, G>::kGroups;
    const uint32_t at = rec + 16u * (uint32_t)lane, row = (uint32_t)lane >> 2, meta = rec + 2u * N * row, zmeta = rec + N * row;
    if (n > 1) {
        W4Frag<FMT, G> f[2];
        w4_load_at<FMT, G, 0>(at, meta, zmeta, f[0]);
        w4_load_at<FMT, G, W4Rec<FMT, G>::kBytes>(at, meta, zmeta, f[1]);
        w4_mma_records<FMT, G, 2>(f, b, acc);
    } else if (n > 0) {
        W4Frag<FMT, G> f[1];
        uint32_t b1[1][16];
        w4_load_at<FMT, G, 0>(at, meta, zmeta, f[0]);
#pragma unroll
        for (int i = 0; i < 16; ++i) b1[0][i] = b[0][i];
        w4_mma_records<FMT, G, 1>(f, b1, acc);
    }
}

#endif

}  // namespace moe
