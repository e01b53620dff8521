// w4_pack.cu -- making and reading packed 4-bit weights (layout in w4.cuh): quantising bf16
// weights, packing a checkpoint's codes, and writing packed weights out as bf16.
//
// All three pass over the data once: quantising reads 2 bytes and writes 0.52 to 0.59 bytes a weight,
// dequantising the reverse. Writing out is bound by HBM (256 matrices of 1024 x 2048: 233 us, 5.7 TB/s);
// quantising (the same bank with E2M1 codes per 32: 280 us, 4.8 TB/s; INT4 per 64: 226 us) by its ~13
// instructions a weight, so each is counted: quotients by a reciprocal and one correction step instead of
// a division, packed maxima, the hardware's E2M1 rounding, no division to find a record. A warp takes one
// record (16 rows by 128 columns): lane 4g + t holds, of rows g and g + 8, the columns 32 c + 8 t + 0 .. 7
// of every 32-column piece c -- the order of the packed words, so its codes leave as two 16-byte stores
// that the warp makes contiguous, and its weights come in 16 bytes a piece, four lanes to a
// 64-byte run of a row. A group's largest weight is a maximum over the lane's 8 values and the
// four lanes of a row (two shuffles).
#include "launch.h"
#include "w4.cuh"

namespace moe {

namespace {

struct W4PackArgs {
    const bf16* w;         // quantise: [n, rows, cols]
    bf16* out;             // dequantise: [n, rows, cols]
    const uint8_t* codes;  // pack: [n, rows, cols / 2], even column in the low nibble
    const bf16* scales;    // pack: [n, rows, cols / G]
    const uint8_t* zeros;  // pack: [n, rows, cols / G] (INT4_ZP)
    uint8_t* packed;
    int n, rows, cols, gate_up;
};

// Matrix row of strip row r.
__device__ __forceinline__ int w4_row(const W4PackArgs& a, int strip, int r) {
    if (!a.gate_up) return strip * 16 + r;
    return r < 8 ? strip * 8 + r : (a.rows >> 1) + strip * 8 + (r - 8);
}

// A code's place in its 16-bit half: i-th code (0 .. 3) of the half.
template <int FMT>
__device__ __forceinline__ uint32_t w4_place(uint32_t code, int i) {
    if (FMT != MOE_W4_E2M1) return code << (4 * i);
    const uint32_t s = code >> 3, m = code & 7u;
    if (i == 0) return (s << 15) | (m << 6);
    if (i == 1) return (s << 12) | (m << 3);
    if (i == 2) return (s << 9) | m;
    return (s << 14) | ((m >> 2) << 13) | (((m >> 1) & 1u) << 10) | ((m & 1u) << 11);
}

// Four codes of each half of a word, code i in bits 4i .. 4i+3, moved to the E2M1 packed order.
__device__ __forceinline__ uint32_t e2m1_planes(uint32_t w) {
    return ((w << 12) & 0x80008000u) | ((w << 6) & 0x01c001c0u) | ((w << 5) & 0x10001000u) | ((w >> 1) & 0x68386838u) |
           ((w >> 2) & 0x02000200u) | ((w >> 8) & 0x00070007u) | ((w >> 3) & 0x04000400u);
}

// Two E2M1 codes (nearest, halfway cases to the even code, at most 6) in a byte, lo in its low half.
__device__ __forceinline__ uint32_t e2m1_pair(float lo, float hi) {
    uint32_t r;
    asm("{\n\t.reg .b8 t;\n\tcvt.rn.satfinite.e2m1x2.f32 t, %1, %2;\n\tcvt.u32.u8 %0, t;\n\t}" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

// Maximum and minimum of packed bf16; a NaN in either operand gives NaN.
__device__ __forceinline__ uint32_t bf2_max(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
__device__ __forceinline__ uint32_t bf2_min(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("min.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

__device__ __forceinline__ void st_record(uint8_t* p, uint4 v) { *reinterpret_cast<uint4*>(p) = v; }

// Stores the scales (and zero points) of one row of a record: lane t = 0 of the row's four.
template <int FMT, int G>
__device__ __forceinline__ void st_meta(uint8_t* rec, int row, const bf16 (&s)[W4Rec<FMT, G>::kGroups],
                                        const uint32_t (&z)[W4Rec<FMT, G>::kGroups]) {
    constexpr int N = W4Rec<FMT, G>::kGroups;
    uint8_t* sp = rec + W4Rec<FMT, G>::kScales + row * (2 * N);
    uint32_t b[N], zw = 0;
#pragma unroll
    for (int i = 0; i < N; ++i) {
        b[i] = __bfloat16_as_ushort(s[i]);
        zw |= z[i] << (8 * i);
    }
    if constexpr (N == 4) {
        *reinterpret_cast<uint2*>(sp) = make_uint2(b[0] | b[1] << 16, b[2] | b[3] << 16);
        if (FMT == MOE_W4_INT4_ZP) *reinterpret_cast<uint32_t*>(rec + W4Rec<FMT, G>::kZeros + row * N) = zw;
    } else if constexpr (N == 2) {
        *reinterpret_cast<uint32_t*>(sp) = b[0] | b[1] << 16;
        if (FMT == MOE_W4_INT4_ZP) *reinterpret_cast<uint16_t*>(rec + W4Rec<FMT, G>::kZeros + row * N) = (uint16_t)zw;
    } else {
        *reinterpret_cast<uint16_t*>(sp) = (uint16_t)b[0];
        if (FMT == MOE_W4_INT4_ZP) rec[W4Rec<FMT, G>::kZeros + row * N] = (uint8_t)zw;
    }
}

// w / s for bf16 w and s, r = 1 / s to a few fp32 steps, as far as rounding the quotient to a code needs
// it. A quotient of two 8-bit mantissas is either exactly halfway between two codes or at least 1/2040
// away from that (codes are multiples of 1/2, |w / s| < 32), so an error of a few fp32 steps decides no
// code; a quotient that is exactly halfway is representable, and one correction step of the product
// w * r finds it: the remainder w - t * s is then exact, and t + remainder * r rounds to the quotient.
__device__ __forceinline__ float w4_quotient(float w, float s, float r) {
    const float t = w * r;
    return fmaf(fmaf(-t, s, w), r, t);
}

// x / D for a bf16 x >= 0, correctly rounded: the product with 1 / D and one correction step. (For D = 6, 7
// and 15 checked in exact arithmetic for every bf16; an infinity gives NaN.)
template <int D>
__device__ __forceinline__ float w4_div_const(float x) {
    constexpr float r = 1.f / D;
    const float t = __fmul_rn(x, r);
    return __fmaf_rn(__fmaf_rn(-t, (float)D, x), r, t);
}
__device__ __forceinline__ float w4_rcp(float x) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

// Walks the records of a warp: i, its 128 columns k, strip and matrix m (two divisions for all of them).
struct W4RecordWalk {
    int64_t i, m;
    int stride, k, strip, dk, ds, dm, R, S;
    __device__ __forceinline__ W4RecordWalk(const W4PackArgs& a) {
        R = (a.cols + kW4Cols - 1) / kW4Cols;
        S = (a.rows + kW4Strip - 1) / kW4Strip;
        const int first = (int)blockIdx.x * 8 + (int)(threadIdx.x >> 5);
        int m0;
        stride = (int)gridDim.x * 8;
        split(first, k, strip, m0);
        split(stride, dk, ds, dm);
        i = first;
        m = m0;
    }
    __device__ __forceinline__ void split(int n, int& k_, int& s_, int& m_) const {
        const int sg = (int)((unsigned)n / (unsigned)R);
        k_ = n - sg * R;
        m_ = (int)((unsigned)sg / (unsigned)S);
        s_ = sg - m_ * S;
    }
    __device__ __forceinline__ void next() {
        i += stride;
        m += dm;
        k += dk;
        strip += ds;
        if (k >= R) {
            k -= R;
            ++strip;
        }
        if (strip >= S) {
            strip -= S;
            ++m;
        }
    }
};

// One row of a record quantised by its four lanes. Per group: scale s = bf16(max|w| / 7) for
// INT4 (/ 6 for E2M1), or bf16(max / 15 - min / 15) over the values and 0 for INT4_ZP with zero
// point rint(-min / s); codes are the nearest value of w / s (halfway to even). A group of zeros has
// scale 0; one with a NaN or an infinity has scale NaN and codes of value 0, so every product with it
// is NaN.
template <int FMT, int G>
__device__ __forceinline__ void quantize_row(const uint4 (&v)[4], uint32_t (&words)[4], bf16 (&sc)[W4Rec<FMT, G>::kGroups], uint32_t (&zp)[W4Rec<FMT, G>::kGroups]) {
    constexpr int P = G / 32;  // 32-column pieces of a group
#pragma unroll
    for (int gi = 0; gi < 4 / P; ++gi) {
        // largest magnitude, or largest and smallest value with 0, of packed pairs
        uint32_t hi2 = 0u, lo2 = 0u;
#pragma unroll
        for (int c = gi * P; c < (gi + 1) * P; ++c) {
            const uint32_t x[4] = {v[c].x, v[c].y, v[c].z, v[c].w};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                if (FMT == MOE_W4_INT4_ZP) {
                    hi2 = bf2_max(hi2, x[j]);
                    lo2 = bf2_min(lo2, x[j]);
                } else {
                    hi2 = bf2_max(hi2, x[j] & 0x7fff7fffu);
                }
            }
        }
#pragma unroll
        for (int o = 1; o < 4; o <<= 1) {
            hi2 = bf2_max(hi2, __shfl_xor_sync(0xffffffffu, hi2, o));
            if (FMT == MOE_W4_INT4_ZP) lo2 = bf2_min(lo2, __shfl_xor_sync(0xffffffffu, lo2, o));
        }
        hi2 = bf2_max(hi2, hi2 >> 16);
        lo2 = bf2_min(lo2, lo2 >> 16);
        const float hi = bf_lo(hi2), lo = bf_lo(lo2);
        const bool bad = !(hi < INFINITY) || !(lo > -INFINITY);
        const float raw = FMT == MOE_W4_INT4_ZP ? __fadd_rn(w4_div_const<15>(hi), w4_div_const<15>(-lo))
                                                : w4_div_const<FMT == MOE_W4_INT4 ? 7 : 6>(hi);
        const bf16 sb = __float2bfloat16_rn(raw);
        const float s = __bfloat162float(sb);
        const bool use = s > 0.f && !bad;
        // (1 / s leaves the normal range below 2^-126 and above 2^126, and a subnormal scale is too coarse for
        // the quotients' bounds: such groups are divided, and clamped to the codes)
        const bool tiny = !(s >= 0x1p-120f && s <= 0x1p120f);
        const float r = use && !tiny ? w4_rcp(s) : 0.f;
        float zf = 0.f;
        if (FMT == MOE_W4_INT4_ZP && use) zf = fminf(rintf(tiny ? __fdiv_rn(-lo, s) : w4_quotient(-lo, s, r)), 15.f);
        sc[gi] = bad ? __ushort_as_bfloat16(0x7fffu) : sb;
        zp[gi] = (uint32_t)zf;
#pragma unroll
        for (int c = gi * P; c < (gi + 1) * P; ++c) {
            const uint32_t x[4] = {v[c].x, v[c].y, v[c].z, v[c].w};
            float q[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float w = (e & 1) ? bf_hi(x[e >> 1]) : bf_lo(x[e >> 1]);
                q[e] = w4_quotient(w, s, r);
            }
            if (!use || tiny) {
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const float w = (e & 1) ? bf_hi(x[e >> 1]) : bf_lo(x[e >> 1]);
                    q[e] = use ? __fdiv_rn(w, s) : 0.f;
                    if (FMT == MOE_W4_INT4) q[e] = fminf(fmaxf(q[e], -8.f), 7.f);
                    if (FMT == MOE_W4_INT4_ZP) q[e] = fminf(fmaxf(q[e], -zf), 15.f - zf);
                }
            }
            // code i of the low half is column 2i, of the high half column 2i + 1
            uint32_t w = 0;
            if (FMT == MOE_W4_E2M1) {
                w = e2m1_pair(q[0], q[2]) | e2m1_pair(q[4], q[6]) << 8 | e2m1_pair(q[1], q[3]) << 16 | e2m1_pair(q[5], q[7]) << 24;
                w = e2m1_planes(w);
            } else {
                // q + 1.5 * 2^23 rounds q to an integer (halfway to even) in the low mantissa bits
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    uint32_t m0 = __float_as_uint(q[2 * i] + 12582912.f), m1 = __float_as_uint(q[2 * i + 1] + 12582912.f);
                    if (FMT == MOE_W4_INT4) {
                        w |= ((__byte_perm(m0, m1, 0x5410) & 0x000f000fu) ^ 0x00080008u) << (4 * i);
                    } else {
                        const int z = (int)zf, b = 0x4b400000;
                        m0 = (uint32_t)min((int)m0 - b + z, 15);
                        m1 = (uint32_t)min((int)m1 - b + z, 15);
                        w |= (m0 | m1 << 16) << (4 * i);
                    }
                }
            }
            words[c] = w;
        }
    }
}

// Codes, scales and zero points of one row of a record from a checkpoint's row-major tensors.
template <int FMT, int G>
__device__ __forceinline__ void pack_row(const W4PackArgs& a, int64_t row, int k0, int t, bool live, uint32_t (&words)[4],
                         bf16 (&sc)[W4Rec<FMT, G>::kGroups], uint32_t (&zp)[W4Rec<FMT, G>::kGroups]) {
    constexpr int N = W4Rec<FMT, G>::kGroups;
#pragma unroll
    for (int c = 0; c < 4; ++c) {
        const int k = k0 + 32 * c + 8 * t;
        // eight codes in column order, four bits each; past the matrix: codes of value 0
        uint32_t in = FMT == MOE_W4_INT4 ? 0x88888888u : 0u;
        if (live && k < a.cols)
            in = *reinterpret_cast<const uint32_t*>(a.codes + row * (a.cols / 2) + k / 2);
        uint32_t w = 0;
#pragma unroll
        for (int e = 0; e < 8; ++e) w |= w4_place<FMT>((in >> (4 * e)) & 15u, e >> 1) << (16 * (e & 1));
        words[c] = w;
    }
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const int g = k0 / G + i;
        const bool in = live && g < a.cols / G;
        sc[i] = in ? a.scales[row * (a.cols / G) + g] : __float2bfloat16_rn(0.f);
        zp[i] = FMT == MOE_W4_INT4_ZP && in ? a.zeros[row * (a.cols / G) + g] & 0x7fu : 0u;
    }
}

template <int FMT, int G, bool QUANT>
__global__ void __launch_bounds__(256) k_w4_pack(W4PackArgs a, int64_t records) {
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    for (W4RecordWalk at(a); at.i < records; at.next()) {
        const int k0 = at.k * kW4Cols;
        uint8_t* rec = a.packed + (size_t)at.i * W4Rec<FMT, G>::kBytes;
        uint4 v[2][4];  // both rows' weights: all loads of a record are on their way before its first shuffle
        if (QUANT) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int row = w4_row(a, at.strip, g + 8 * h);
                const bf16* src = a.w + (at.m * a.rows + row) * a.cols + k0 + 8 * t;
#pragma unroll
                for (int c = 0; c < 4; ++c)
                    v[h][c] = row < a.rows && k0 + 32 * c + 8 * t < a.cols ? ld_stream(src + 32 * c) : make_uint4(0u, 0u, 0u, 0u);
            }
        }
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int row = w4_row(a, at.strip, g + 8 * h);
            uint32_t words[4];
            bf16 sc[W4Rec<FMT, G>::kGroups];
            uint32_t zp[W4Rec<FMT, G>::kGroups];
            if (QUANT)
                quantize_row<FMT, G>(v[h], words, sc, zp);
            else
                pack_row<FMT, G>(a, at.m * a.rows + row, k0, t, row < a.rows, words, sc, zp);
            st_record(rec + 512 * h + lane * 16, make_uint4(words[0], words[1], words[2], words[3]));
            if (t == 0) st_meta<FMT, G>(rec, g + 8 * h, sc, zp);
        }
    }
}

template <int FMT, int G>
__global__ void __launch_bounds__(256) k_w4_unpack(W4PackArgs a, int64_t records) {
    constexpr int N = W4Rec<FMT, G>::kGroups;
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    for (W4RecordWalk at(a); at.i < records; at.next()) {
        const int k0 = at.k * kW4Cols, strip = at.strip;
        const int64_t m = at.m;
        const uint8_t* rec = a.packed + (size_t)at.i * W4Rec<FMT, G>::kBytes;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int r = g + 8 * h, row = w4_row(a, strip, r);
            if (row >= a.rows) continue;
            const uint4 v = ld_stream(rec + 512 * h + lane * 16);
            const uint32_t words[4] = {v.x, v.y, v.z, v.w};
            bf16* dst = a.out + (m * a.rows + row) * a.cols + k0 + 8 * t;
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                if (k0 + 32 * c + 8 * t >= a.cols) continue;
                const int gi = c * 32 / G;
                const float s = __bfloat162float(reinterpret_cast<const bf16*>(rec + W4Rec<FMT, G>::kScales)[r * N + gi]);
                uint32_t bias = 0xc308c308u;
                if (FMT == MOE_W4_INT4_ZP) bias = 0xc300c300u | (rec[W4Rec<FMT, G>::kZeros + r * N + gi] * 0x00010001u);
                uint32_t p[4];
                w4_decode<FMT>(words[c], bias, p);
                uint4 o;  // s * v in fp32 (exact: 8 and at most 5 bits), rounded once to bf16
                o.x = pack_bf16x2(s * bf_lo(p[0]), s * bf_hi(p[0]));
                o.y = pack_bf16x2(s * bf_lo(p[1]), s * bf_hi(p[1]));
                o.z = pack_bf16x2(s * bf_lo(p[2]), s * bf_hi(p[2]));
                o.w = pack_bf16x2(s * bf_lo(p[3]), s * bf_hi(p[3]));
                *reinterpret_cast<uint4*>(dst + 32 * c) = o;
            }
        }
    }
}

// An ordinary launch after a kernel that wrote weights: it starts once that kernel is complete
// and its memory visible, and whatever the library launches next starts after it, so a layer
// call right after quantising may read the weights early (the ordering contract of moe.h).
__global__ void k_w4_settle() {}

enum { kOpQuantize, kOpPack, kOpUnpack };

template <int FMT, int G>
cudaError_t launch_pack(int op, const W4PackArgs& a, int64_t records, unsigned grid, cudaStream_t s) {
    if (op == kOpQuantize)
        MOE_LAUNCH(MOE_KERNEL_W4_PACK, s, (k_w4_pack<FMT, G, true><<<grid, 256, 0, s>>>(a, records)));
    else if (op == kOpPack)
        MOE_LAUNCH(MOE_KERNEL_W4_PACK, s, (k_w4_pack<FMT, G, false><<<grid, 256, 0, s>>>(a, records)));
    else
        MOE_LAUNCH(MOE_KERNEL_W4_PACK, s, (k_w4_unpack<FMT, G><<<grid, 256, 0, s>>>(a, records)));
    cudaError_t e = cudaGetLastError();
    if (e == cudaSuccess && op != kOpUnpack) {
        MOE_LAUNCH(MOE_KERNEL_W4_PACK, s, (k_w4_settle<<<1, 32, 0, s>>>()));
        e = cudaGetLastError();
    }
    return e;
}

cudaError_t launch(int op, int format, int group, const W4PackArgs& a, int num_sms, cudaStream_t s) {
    const int64_t records = (int64_t)a.n * ((a.rows + kW4Strip - 1) / kW4Strip) * ((a.cols + kW4Cols - 1) / kW4Cols);
    const int64_t want = (records + 7) / 8, cap = (int64_t)num_sms * 8;
    const unsigned grid = (unsigned)(want < cap ? want : cap);
#define MOE_W4_CASE(F, G) \
    if (format == F && group == G) return launch_pack<F, G>(op, a, records, grid, s)
    MOE_W4_CASE(MOE_W4_INT4, 32);
    MOE_W4_CASE(MOE_W4_INT4, 64);
    MOE_W4_CASE(MOE_W4_INT4, 128);
    MOE_W4_CASE(MOE_W4_INT4_ZP, 32);
    MOE_W4_CASE(MOE_W4_INT4_ZP, 64);
    MOE_W4_CASE(MOE_W4_INT4_ZP, 128);
    MOE_W4_CASE(MOE_W4_E2M1, 32);
    MOE_W4_CASE(MOE_W4_E2M1, 64);
    MOE_W4_CASE(MOE_W4_E2M1, 128);
#undef MOE_W4_CASE
    return cudaErrorInvalidValue;
}

}  // namespace

cudaError_t launch_w4_quantize(const moe_w4_format& f, int n, int rows, int cols, bool gate_up, const bf16* w,
                               uint8_t* packed, int num_sms, cudaStream_t s) {
    W4PackArgs a = {};
    a.w = w; a.packed = packed; a.n = n; a.rows = rows; a.cols = cols; a.gate_up = gate_up;
    return launch(kOpQuantize, f.format, f.group, a, num_sms, s);
}

cudaError_t launch_w4_pack(const moe_w4_format& f, int n, int rows, int cols, bool gate_up, const uint8_t* codes,
                           const bf16* scales, const uint8_t* zeros, uint8_t* packed, int num_sms, cudaStream_t s) {
    W4PackArgs a = {};
    a.codes = codes; a.scales = scales; a.zeros = zeros; a.packed = packed;
    a.n = n; a.rows = rows; a.cols = cols; a.gate_up = gate_up;
    return launch(kOpPack, f.format, f.group, a, num_sms, s);
}

cudaError_t launch_w4_dequantize(const moe_w4_format& f, int n, int rows, int cols, bool gate_up, const uint8_t* packed,
                                 bf16* w, int num_sms, cudaStream_t s) {
    W4PackArgs a = {};
    a.packed = const_cast<uint8_t*>(packed); a.out = w; a.n = n; a.rows = rows; a.cols = cols; a.gate_up = gate_up;
    return launch(kOpUnpack, f.format, f.group, a, num_sms, s);
}

}  // namespace moe
