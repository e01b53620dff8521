// linear_pair.cu -- the linear layers' products where there are rows enough: tiles of 256 features by up to 256
// columns on pairs of SMs.
//
// The roles and operands are those of linear.cu; here two CTAs share a tile (tcgen05 cta_group::2). Each loads
// its own 128 feature rows and half of the columns, so a 64-deep stage is 32 KB for 256 x 256 of the product's
// tile: a tensor core reads 8 KB of shared memory for 128 cycles of work and TMA writes as much, which one SM
// alone (16 KB of A and 32 KB of B a stage) cannot keep up with. The CTA of even rank issues the
// MMAs of both; its barrier of a stage counts both CTAs' copies. An expert's last rows of kDw, where they are no whole 64, have
// rows of the next expert behind them, which must not be multiplied, whatever they hold (0 x infinity would stay). The maps
// of kDw are of 64 consecutive rows from any first one, and the last block is loaded from a negative place in its 64: TMA's zeros come
// first, in both operands alike, then the rows there are, and nothing of the next expert. (Clearing the foreign rows in shared memory
// takes an order between those stores and the products that the other CTA issues. With the cluster scope that it needs, the 256
// experts' dW of 512 rows takes 194 us instead of 166, of 32768 rows 250 instead of 211; with stores of the even CTA to both 236 and 240.)
//
// Measured (graph replay, us): 4096 x 8192 x 2048 71.5 without an activation = 1922 TFLOP/s, the rate of a library product; 76 with
// GELU and bias; experts' products of 32768 rows, 256 x [1024, 2048]: forward 191 (5.7 TB/s), dx 184, dW 211 (5.8 TB/s).
//
// The epilogue reads accumulator fragments (a thread: two columns of one feature side by side), applies bias,
// activation and residual in fp32 and transposes by stmatrix, 32 columns at a time, so that what is stored is
// 16 bytes of features a lane; residual comes the same way back by ldmatrix. A warp's buffer is 2 KB, its 16-byte
// chunks swizzled so that both sides go without bank conflicts.
#include "linear.cuh"

namespace moe {

constexpr uint32_t kPairB = 128 * 64 * 2;  // half of the columns
// Stages of 32 KB, and the epilogue warps' buffers: one of 2 KB each; kDw has two, and a stage less.
constexpr int pair_stages(int mode) { return mode == kDw ? 5 : 6; }
constexpr uint32_t pair_ring(int mode) { return (uint32_t)pair_stages(mode) * (kLinA + kPairB); }
constexpr uint32_t pair_scratch(int mode) { return kLinEpiWarps * (mode == kDw ? 4096u : 2048u); }
constexpr uint32_t kPairTables = 2 * (kLinMaxE + 4) * 4;
constexpr uint32_t pair_bytes(int mode) { return 1024 + pair_ring(mode) + pair_scratch(mode) + kPairTables + 256; }

__device__ __forceinline__ uint32_t pack2(float a, float b, bf16) { return pack_bf16x2(a, b); }
__device__ __forceinline__ uint32_t pack2(float a, float b, fp16) {
    const __half2 v = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&v);
}
__device__ __forceinline__ float2 unpack2(uint32_t u, bf16) { return make_float2(bf_lo(u), bf_hi(u)); }
__device__ __forceinline__ float2 unpack2(uint32_t u, fp16) { return __half22float2(*reinterpret_cast<const __half2*>(&u)); }

// Byte of 16-byte chunk `chunk` of row `row` in a warp's buffer: rows of 64 bytes (32 features), of 32 (16 features).
__device__ __forceinline__ uint32_t at64(int row, int chunk) { return (uint32_t)(row * 64 + ((chunk ^ ((row >> 1) & 3)) << 4)); }
__device__ __forceinline__ uint32_t at32(int row, int chunk) { return (uint32_t)(row * 32 + ((chunk ^ ((row >> 2) & 1)) << 4)); }

// Rows that do not start on 16 bytes: a warp's buffer of 32 rows of kWide features to memory, a row (two of
// 16 features) at a time, lanes side by side. p: the first row's element f0 in memory, ld: elements from row to row; F: features of
// a row; rows: how many exist.
template <int kWide>
__device__ __forceinline__ uint32_t feature_at(int row, int f) { return (kWide == 16 ? at32(row, f >> 3) : at64(row, f >> 3)) + 2 * (f & 7); }
template <int kWide>
__device__ __forceinline__ void rows_out(uint32_t buf, uint16_t* p, int64_t ld, int f0, int F, int rows) {
    const int lane = threadIdx.x & 31, f = lane & (kWide - 1);
    constexpr int kAtOnce = 32 / kWide;
#pragma unroll 4
    for (int r = lane / kWide; r < rows; r += kAtOnce) {
        uint16_t v;
        asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(buf + feature_at<kWide>(r, f)) : "memory");
        if (f0 + f < F) p[(int64_t)r * ld + f] = v;
    }
}

// A warp's part of a tile: 32 accumulator lanes (q), 32 columns at a time. row0: the result's row of the tile's
// first column; fl: the CTA's first feature.
template <typename T, int MODE, bool GATED>
__device__ __forceinline__ void pair_epilogue(const LinView& a, uint32_t tmem, uint32_t buf, int q, int h, int e, int64_t row0, int fl, int cols,
                                              bool any) {
    const int lane = threadIdx.x & 31, g = lane >> 2;
    constexpr bool kFull = MODE == kFwd;
    constexpr int kWide = GATED ? 16 : 32;  // features of the warp
    const int f0 = fl + q * kWide;
    const bool vec = a.vec != 0;
    float bias[4] = {0.f, 0.f, 0.f, 0.f};  // of features g, g + 8 and g + 16, g + 24 (gated: the up rows of g, g + 8)
    if (kFull && a.bias) {
        const T* b = reinterpret_cast<const T*>(a.bias) + (int64_t)e * a.N;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int f = f0 + g + 8 * (GATED ? i & 1 : i);
            if (f < a.F) bias[i] = to_f(b[f + (GATED && i >= 2 ? a.F : 0)]);
        }
    }
    const int crow = GATED ? lane >> 1 : lane >> 2, cch = GATED ? lane & 1 : lane & 3;  // the lane's row and chunk of the result
    const int left = a.F - f0 - cch * 8;                                                // features from its chunk on
    constexpr int kRows = GATED ? 16 : 8, kRounds = 32 / kRows;
    T* out = reinterpret_cast<T*>(a.out) + (row0 + crow) * a.F + f0 + cch * 8;
    const T* res = kFull ? reinterpret_cast<const T*>(a.residual) : nullptr;
    T* z = nullptr;
    int zleft = 0;
    if (kFull && a.z) {  // rows of z hold 32 features of the warp: gated, 16 gate and the 16 up of the same features
        const int zc = lane & 3, zf = GATED ? f0 + (zc & 1) * 8 + (zc >> 1) * a.F : f0 + zc * 8;
        z = reinterpret_cast<T*>(a.z) + (row0 + (lane >> 2)) * a.N + zf;
        zleft = a.F - f0 - (GATED ? zc & 1 : zc) * 8;
    }
    for (int c = h * 32; c < cols; c += 64) {
        uint32_t r[32];  // 16 features (lanes) from 0 in r[0 .. 15], from 16 in r[16 .. 31]; each: column block b in [4 b ..]
        Raw rv[kRounds];
        if (kFull && res) {
#pragma unroll
            for (int i = 0; i < kRounds; ++i)
                if (c + crow + i * kRows < cols && left > 0) {
                    const int64_t at = (row0 + c + crow + i * kRows) * a.F + f0 + cch * 8;
                    rv[i] = vec ? ld_cols<T, 8>(res, at, 0, 8) : ld_cols<T, 1>(res, at, (int64_t)a.T * a.F, left);
                }
        }
        if (any) {
            tmem_ld_frag4(tmem + c, r);
            tmem_ld_frag4(tmem + (16u << 16) + c, r + 16);
            asm volatile("tcgen05.wait::ld.sync.aligned;"
                         : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]), "+r"(r[8]), "+r"(r[9]),
                           "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]), "+r"(r[16]), "+r"(r[17]), "+r"(r[18]),
                           "+r"(r[19]), "+r"(r[20]), "+r"(r[21]), "+r"(r[22]), "+r"(r[23]), "+r"(r[24]), "+r"(r[25]), "+r"(r[26]), "+r"(r[27]),
                           "+r"(r[28]), "+r"(r[29]), "+r"(r[30]), "+r"(r[31])::"memory");
        } else {
#pragma unroll
            for (int i = 0; i < 32; ++i) r[i] = 0u;
        }
        if (kFull && a.bias) {
#pragma unroll
            for (int i = 0; i < 32; ++i) r[i] = __float_as_uint(__uint_as_float(r[i]) + bias[(i >> 4) * 2 + ((i >> 1) & 1)]);
        }
        if (kFull && z) {
#pragma unroll
            for (int b = 0; b < 4; ++b) {
                uint32_t p[4];
#pragma unroll
                for (int m = 0; m < 4; ++m) {
                    const int i = (m >> 1) * 16 + b * 4 + (m & 1) * 2;
                    p[m] = pack2(__uint_as_float(r[i]), __uint_as_float(r[i + 1]), T());
                }
                stmatrix4_trans(buf + at64(8 * b + (lane & 7), lane >> 3), p[0], p[1], p[2], p[3]);
            }
            __syncwarp();
            if (vec) {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int row = (lane >> 2) + 8 * i;
                    const uint4 v = lds128_smem(buf + at64(row, lane & 3));
                    if (c + row < cols && zleft > 0) *reinterpret_cast<uint4*>(z + (int64_t)(c + 8 * i) * a.N) = v;
                }
            } else {  // (not gated: its rows are a multiple of 16 bytes)
                rows_out<32>(buf, reinterpret_cast<uint16_t*>(a.z) + (row0 + c) * a.N + f0, a.N, f0, a.F, min(32, cols - c));
            }
            __syncwarp();
        }
        if (kFull && res) {
#pragma unroll
            for (int i = 0; i < kRounds; ++i)
                if (c + crow + i * kRows < cols) sts128(buf + (GATED ? at32(crow + i * kRows, cch) : at64(crow + i * kRows, cch)), rv[i].w);
            __syncwarp();
        }
        // activation, residual, rounding: pairs of columns of a feature
        float v[GATED ? 16 : 32];
#pragma unroll
        for (int i = 0; i < (GATED ? 16 : 32); ++i) {
            v[i] = __uint_as_float(r[i]);
            if (GATED) v[i] *= lin_sigmoid(v[i]) * __uint_as_float(r[i + 16]);
        }
        if (kFull && !GATED) lin_act<GATED ? 16 : 32>(a.act, v);
        uint32_t p[GATED ? 8 : 16];
#pragma unroll
        for (int k = 0; k < (GATED ? 2 : 4); ++k) {  // matrices of one ldmatrix / stmatrix: gated two blocks of 16 features, else one of 32
            uint32_t rr[4];
            const uint32_t at = GATED ? at32(16 * k + 8 * (lane >> 4) + (lane & 7), (lane >> 3) & 1) : at64(8 * k + (lane & 7), lane >> 3);
            if (kFull && res) ldmatrix4_trans(buf + at, rr);
#pragma unroll
            for (int m = 0; m < 4; ++m) {
                const int i = GATED ? (2 * k + (m >> 1)) * 4 + (m & 1) * 2 : (m >> 1) * 16 + k * 4 + (m & 1) * 2;
                float v0 = v[i], v1 = v[i + 1];
                if (kFull && res) {
                    const float2 x = unpack2(rr[m], T());
                    v0 += x.x;
                    v1 += x.y;
                }
                p[k * 4 + m] = pack2(v0, v1, T());
            }
        }
        if (kFull && res) __syncwarp();
#pragma unroll
        for (int k = 0; k < (GATED ? 2 : 4); ++k) {
            const uint32_t at = GATED ? at32(16 * k + 8 * (lane >> 4) + (lane & 7), (lane >> 3) & 1) : at64(8 * k + (lane & 7), lane >> 3);
            stmatrix4_trans(buf + at, p[k * 4], p[k * 4 + 1], p[k * 4 + 2], p[k * 4 + 3]);
        }
        __syncwarp();
        if (vec) {
#pragma unroll
            for (int i = 0; i < kRounds; ++i) {
                const int row = crow + i * kRows;
                const uint4 v = lds128_smem(buf + (GATED ? at32(row, cch) : at64(row, cch)));
                if (c + row < cols && left > 0) *reinterpret_cast<uint4*>(out + (int64_t)(c + i * kRows) * a.F) = v;
            }
        } else {
            rows_out<kWide>(buf, reinterpret_cast<uint16_t*>(a.out) + (row0 + c) * a.F + f0, a.F, f0, a.F, min(32, cols - c));
        }
        __syncwarp();
    }
}

// The same of kDw: nothing is added, and a tile's rows are W's own, so a warp's 32 x 32 go out by TMA (rows and
// columns past W's are left out there), from two buffers in turn.
template <typename T>
__device__ __forceinline__ void pair_epilogue_dw(const CUtensorMap* mC, uint32_t tmem, uint32_t buf, int q, int h, int e, int c0, int fl, int cols,
                                                 bool any, int& turn) {
    const int lane = threadIdx.x & 31;
    for (int c = h * 32; c < cols; c += 64, turn ^= 1) {
        uint32_t r[32];
        if (any) {
            tmem_ld_frag4(tmem + c, r);
            tmem_ld_frag4(tmem + (16u << 16) + c, r + 16);
            asm volatile("tcgen05.wait::ld.sync.aligned;"
                         : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]), "+r"(r[8]), "+r"(r[9]),
                           "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]), "+r"(r[16]), "+r"(r[17]), "+r"(r[18]),
                           "+r"(r[19]), "+r"(r[20]), "+r"(r[21]), "+r"(r[22]), "+r"(r[23]), "+r"(r[24]), "+r"(r[25]), "+r"(r[26]), "+r"(r[27]),
                           "+r"(r[28]), "+r"(r[29]), "+r"(r[30]), "+r"(r[31])::"memory");
        } else {
#pragma unroll
            for (int i = 0; i < 32; ++i) r[i] = 0u;
        }
        const uint32_t at = buf + (uint32_t)turn * 2048u;
        if (lane == 0) tma_store_wait_read<1>();  // the store before the last has read this buffer
        __syncwarp();
#pragma unroll
        for (int b = 0; b < 4; ++b) {
            uint32_t p[4];
#pragma unroll
            for (int m = 0; m < 4; ++m) {
                const int i = (m >> 1) * 16 + b * 4 + (m & 1) * 2;
                p[m] = pack2(__uint_as_float(r[i]), __uint_as_float(r[i + 1]), T());
            }
            stmatrix4_trans(at + at64(8 * b + (lane & 7), lane >> 3), p[0], p[1], p[2], p[3]);
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
            tma_store_3d(mC, at, fl + q * 32, c0 + c, e);
            tma_store_commit();
        }
    }
}

template <typename T, int MODE, bool GATED>
__global__ void __launch_bounds__(kLinThreads, 1)
    k_linear_pair(const __grid_constant__ CUtensorMap mA, const __grid_constant__ CUtensorMap mB, const __grid_constant__ CUtensorMap mC, const LinView a) {
    constexpr int kStages = pair_stages(MODE);
    constexpr uint32_t kPairRing = pair_ring(MODE), kPairScratch = pair_scratch(MODE);
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = smem_u32(smem_raw);
    uint8_t* smem = smem_raw + (((raw + 1023u) & ~1023u) - raw);
    uint8_t* sA = smem;
    uint8_t* sB = smem + kStages * kLinA;
    uint8_t* scratch = smem + kPairRing;
    int* off = reinterpret_cast<int*>(scratch + kPairScratch);
    int* start = off + kLinMaxE + 4;
    uint64_t* full = reinterpret_cast<uint64_t*>(scratch + kPairScratch + kPairTables);  // even rank: a stage of both CTAs is ready
    uint64_t* empty = full + kStages;  // both CTAs' MMAs have read it
    uint64_t* accf = empty + kStages;
    uint64_t* acce = accf + 2;          // even rank: both CTAs' epilogues have read the accumulator
    uint64_t* mma_done = acce + 2;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(mma_done + 1);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
    volatile int* progress = abort_flag + 1;  // kDw: stages that this CTA's producer has found empty, which the longer waits go by
    static_assert((2 * kStages + 5) * 8 + 12 <= 256, "barrier area");

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = cluster_rank();
    if (threadIdx.x == 0) {
        for (int s = 0; s < kStages; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(&accf[b], 1);
            mbar_init(&acce[b], 2 * kLinEpiWarps);
        }
        mbar_init(mma_done, 1);
        *abort_flag = 0;
        *progress = 0;
        fence_mbar_init();
        tma_prefetch_desc(&mA);
        tma_prefetch_desc(&mB);
    }
    if (warp == 1) {
        tmem_alloc_pair(tmem_slot, 512);
        tmem_relinquish_pair();
    }
    tc_fence_before();
    __syncthreads();
    cluster_sync_all();  // barriers of both CTAs are ready
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    grid_dep_wait();
    grid_dep_launch();
    lin_tables<MODE>(a, off, start);
    const int total = start[a.E];
    const int step = gridDim.x / 2, first = blockIdx.x / 2;
    LinWalk<MODE, 32> walk;

    if (warp == 0) {
        // ---------------- TMA producer of this CTA's halves
        if (elect_one()) {
            int it = 0;
            for (int t = first; t < total && !*abort_flag; t += step) {
                const LinTile ti = walk.to(a, off, start, t);
                const int half = (ti.cols + 31) / 32 * 16;  // columns of this CTA
                const int c0 = ti.c0 + (int)rank * half, f = ti.f * 2 + (int)rank;
                const int boxes = MODE == kDw ? (half + 63) / 64 : (half + a.boxes - 1) / a.boxes;
                const uint32_t bytes = kLinA + (uint32_t)boxes * (MODE == kDw ? 64 : a.boxes) * 128u;
                for (int kb = 0; kb < ti.blocks; ++kb, ++it) {
                    const int s = it % kStages;
                    const uint32_t ph = (uint32_t)(it / kStages) & 1u;
                    if (!mbar_wait(&empty[s], ph ^ 1u, a.wait_ns)) {
                        atomicOr(a.err, ERR_TIMEOUT);
                        *abort_flag = 1;
                        break;
                    }
                    if (MODE == kDw) *progress = it + 1;
                    if (a.suppress && blockIdx.x == 0 && it == 0) continue;
                    uint8_t* da = sA + s * kLinA;
                    uint8_t* db = sB + s * kPairB;
                    if (rank == 0) mbar_arrive_expect_tx(&full[s], 2 * bytes);
                    const uint32_t bar = mbar_of_even(&full[s]);
                    if (MODE == kDw) {
                        const int row = ti.row0 + kb * 64, from = min(ti.rows - kb * 64 - 64, 0);
                        for (int p = 0; p < 2; ++p) tma_load_3d_pair(da + p * 8192, &mA, bar, f * 128 + p * 64, from, row);
                        for (int p = 0; p < boxes; ++p) tma_load_3d_pair(db + p * 8192, &mB, bar, c0 + p * 64, from, row);
                    } else {
                        if (MODE == kDx) {
                            for (int p = 0; p < 2; ++p) tma_load_3d_pair(da + p * 8192, &mA, bar, f * 128 + p * 64, kb * 64, ti.e);
                        } else if (GATED) {
                            tma_load_5d_pair(da, &mA, bar, kb * 64, 0, 0, f * 4, ti.e);
                        } else {
                            tma_load_3d_pair(da, &mA, bar, kb * 64, f * 128, ti.e);
                        }
                        for (int p = 0; p < boxes; ++p) tma_load_2d_pair(db + p * a.boxes * 128, &mB, bar, kb * 64, ti.row0 + c0 + p * a.boxes);
                    }
                }
            }
            // every copy this CTA issued must land before shared memory is released. (Those of the odd CTA count in the other:
            // the last product has read them by the end; where a wait ran out, a millisecond is ample.)
            if (rank == 0) {
                for (int s = 0; s < min(it, kStages); ++s)  // (its last use: number (it - 1 - s) / kStages)
                    if (!mbar_wait(&full[s], (uint32_t)((it - 1 - s) / kStages) & 1u, a.wait_ns)) atomicOr(a.err, ERR_TIMEOUT);
            }
            if (*abort_flag) {
                const uint64_t t0 = global_ns();
                while (global_ns() - t0 < 1000000u) {}
            }
        }
        __syncwarp();
    } else if (warp == 1) {
        // ---------------- MMA issuer (even rank). One lane does it all: what it spends on a stage besides the products'
        // 512 clocks is time of narrow tiles.
        if (rank == 0 && elect_one()) {
            int it = 0, local = 0;
            bool ok = true;
            const uint64_t descA = MODE == kFwd ? sdesc_kmajor_sw128(smem_u32(sA)) : sdesc_mnmajor_sw128(smem_u32(sA), 8192);
            const uint64_t descB = MODE == kDw ? sdesc_mnmajor_sw128(smem_u32(sB), 8192) : sdesc_kmajor_sw128(smem_u32(sB));
            constexpr int kStepA = MODE == kFwd ? 2 : 128, kStepB = MODE == kDw ? 128 : 2;  // 16 deeper, in 16-byte units
            for (int t = first; t < total && ok; t += step, ++local) {
                if (*abort_flag) break;
                const LinTile ti = walk.to(a, off, start, t);
                const int n32 = (ti.cols + 31) / 32 * 32;
                const uint32_t idesc = idesc_f16_f32(std::is_same<T, bf16>::value, 256, n32, MODE != kFwd, MODE == kDw);
                const int b = local & 1;
                const uint32_t d = tmem + (uint32_t)(b * 256);
                ok = mbar_wait(&acce[b], ((uint32_t)(local >> 1) & 1u) ^ 1u, a.wait_ns);
                tc_fence_after();
                for (int kb = 0; ok && kb < ti.blocks; ++kb, ++it) {
                    const int s = it % kStages;
                    ok = mbar_wait(&full[s], (uint32_t)(it / kStages) & 1u, a.wait_ns);
                    if (!ok) break;
                    tc_fence_after();
                    const uint64_t da = descA + (uint64_t)(s * (kLinA >> 4)), db = descB + (uint64_t)(s * (kPairB >> 4));
                    const int zeros = MODE == kDw ? max(4 - (ti.rows - kb * 64 + 15) / 16, 0) : 0;  // 16s without a row
#pragma unroll
                    for (int kk = 0; kk < 4; ++kk)
                        if (kk >= zeros) mma_f16_pair(d, da + kk * kStepA, db + kk * kStepB, idesc, kb != 0 || kk != zeros);
                    mma_commit_pair(&empty[s]);
                }
                if (ok && ti.blocks > 0) mma_commit_pair(&accf[b]);
                if (ok && ti.blocks == 0) {  // (no rows: zeros are written)
                    mbar_arrive_cluster(&accf[b], 0);
                    mbar_arrive_cluster(&accf[b], 1);
                }
            }
            if (!ok) {
                atomicOr(a.err, ERR_TIMEOUT);
                *abort_flag = 1;
            }
            mma_commit_pair(mma_done);
        }
        __syncwarp();
    } else if (warp >= kLinEpiWarp0) {
        // ---------------- epilogue of this CTA's features: lanes 32 q .. of the accumulator, every other 32 columns
        const int q = warp & 3, h = (warp - kLinEpiWarp0) >> 2;
        const uint32_t buf = smem_u32(scratch + (warp - kLinEpiWarp0) * (kPairScratch / kLinEpiWarps));
        int local = 0, turn = 0;
        for (int t = first; t < total; t += step, ++local) {
            const LinTile ti = walk.to(a, off, start, t);
            const int b = local & 1;
            const uint32_t use = (uint32_t)(local >> 1) & 1u;
            bool ready = false;
            if (!*abort_flag)  // (a tile's whole contraction: of kDw as long as an expert has rows, else of 2^14 stages at most)
                ready = MODE == kDw ? mbar_wait_progress(&accf[b], use, progress, a.wait_ns) : mbar_wait(&accf[b], use, a.wait_ns);
            ready = __all_sync(0xffffffffu, ready);
            if (!ready) {
                if (lane == 0) {
                    if (!*abort_flag) atomicOr(a.err, ERR_TIMEOUT);
                    *abort_flag = 1;
                }
                break;
            }
            tc_fence_after();
            const uint32_t acc = tmem + ((uint32_t)(q * 32) << 16) + (uint32_t)(b * 256);
            const int fl = (ti.f * 2 + (int)rank) * (GATED ? 64 : 128);
            if constexpr (MODE == kDw)
                pair_epilogue_dw<T>(&mC, acc, buf, q, h, ti.e, ti.c0, fl, ti.cols, ti.blocks > 0, turn);
            else
                pair_epilogue<T, MODE, GATED>(a, acc, buf, q, h, ti.e, (int64_t)ti.row0 + ti.c0, fl, ti.cols, ti.blocks > 0);
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive_cluster(&acce[b], 0);
        }
        if (MODE == kDw && lane == 0) tma_store_wait_all();
        __syncwarp();
    } else {
        if (MODE != kFwd && a.dbias) lin_dbias<T>(a, off, blockIdx.x * 2 + warp - 2, gridDim.x * 2);
        __syncwarp();
    }
    tc_fence_before();
    __syncthreads();
    // Only now, with this CTA's last tile written: from the start of the kernel the odd CTA's limit would be one of the whole call.
    if (warp == 1 && !mbar_wait(mma_done, 0, a.wait_ns) && lane == 0) atomicOr(a.err, ERR_TIMEOUT);
    __syncwarp();
    cluster_sync_all();  // neither CTA leaves while the other may still arrive on its barriers or read its tiles
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc_pair(tmem, 512);
    }
}

template <typename T, int MODE, bool GATED>
static cudaError_t launch_pair_k(const CUtensorMap& A, const CUtensorMap& B, const CUtensorMap& C, const LinView& v, int grid, cudaStream_t s) {
    static std::atomic<bool> allowed[64];
    const cudaError_t e = allow_shared(k_linear_pair<T, MODE, GATED>, (int)pair_bytes(MODE), allowed);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(kLinThreads);
    cfg.dynamicSmemBytes = pair_bytes(MODE);
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = 2;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, k_linear_pair<T, MODE, GATED>, A, B, C, v);
}

template <typename T>
static cudaError_t launch_pair_t(int mode, bool gated, const CUtensorMap& A, const CUtensorMap& B, const CUtensorMap& C, const LinView& v, int grid, cudaStream_t s) {
    if (mode == kDx) return launch_pair_k<T, kDx, false>(A, B, C, v, grid, s);
    if (mode == kDw) return launch_pair_k<T, kDw, false>(A, B, C, v, grid, s);
    return gated ? launch_pair_k<T, kFwd, true>(A, B, C, v, grid, s) : launch_pair_k<T, kFwd, false>(A, B, C, v, grid, s);
}

cudaError_t launch_pair(int32_t dtype, int mode, bool gated, const CUtensorMap& A, const CUtensorMap& B, const CUtensorMap& C, const LinView& v, int grid,
                        cudaStream_t s) {
    return dtype == MOE_FP16 ? launch_pair_t<fp16>(mode, gated, A, B, C, v, grid, s) : launch_pair_t<bf16>(mode, gated, A, B, C, v, grid, s);
}

}  // namespace moe
