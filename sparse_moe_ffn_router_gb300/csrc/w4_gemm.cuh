// w4_gemm.cuh -- the products of packed 4-bit weights with many tokens, on the 5th-generation
// tensor cores (tcgen05 + TMEM + TMA).
//
// D[128 token rows, BN weight rows] = A . B^T, both operands K-major bf16 in shared memory. A (the
// token rows, or the h rows of down) comes by TMA, or is gathered from x for a routed expert's
// gate_up. B does not exist in memory: sixteen warps read the packed records (16 rows by 128
// columns each, straight from global memory into registers, one stage ahead), decode them,
// multiply by the group scale and write bf16 into the 128-byte swizzled layout the tensor core
// reads. A weight is rounded once, to bf16(s * v): the tensor core takes bf16 operands and its
// accumulator spans all of K, so a scale per 32 to 128 columns cannot be applied behind it; the
// error is at most half a bf16 step a weight (2^-8), of the size of the roundings of h and Y.
//
// One persistent CTA per SM walks the tiles (group, N tile, M tile; the M tiles that share weights
// run back to back). A stage is 128 columns (one record): 32 KB of A, 64 KB of B at BN = 256; two
// stages, so the decoding of one overlaps the MMAs of the other: 8 MMAs of 128 x 256 x 16 are
// ~1300 cycles, the 16 records of a stage ~2400 issue slots over four schedulers. Two accumulators
// in TMEM let the epilogue of a tile overlap the next tile's MMAs. Roles:
//   warp 0     TMA producer (one lane)            warps 2-5   epilogue (TMEM lane quadrants)
//   warp 1     TMEM owner and MMA issuer           warps 6-21  decoders, and gatherers of A rows
// Decoder stores: lane 4g + t writes 16 bytes (8 columns) of row g; odd rows take the two 32-column
// pieces of a 64-column tile in the other order, which spreads the eight lanes of a store phase
// (two rows) over all banks.
#pragma once

#include "launch.h"
#include "w4.cuh"

namespace moe {

enum : int { kW4GLinear = 0, kW4GUp = 1, kW4GDown = 2 };

struct W4GemmArgs {
    const uint8_t* w[2];   // packed matrices: routed (or linear), shared
    size_t matrix_bytes;   // of one routed matrix
    int rows[2], cols[2];  // of one matrix
    const bf16* bias;      // linear
    bf16* out;             // linear [T, rows]
    int T;                 // linear: token rows
    uint32_t* err;
    uint64_t wait_ns;
};

cudaError_t launch_w4_gemm(int format, int group, int which, const W4GemmArgs& p, const CUtensorMap& a0,
                           const CUtensorMap& a1, const LayerArgs& a, int bn, cudaStream_t s);

#ifdef __CUDACC__

constexpr int kW4gM = 128, kW4gK = 128;          // token rows of a tile, columns of a stage
constexpr int kW4gStages = 2;
constexpr int kW4gDec = 16;                      // decoder warps
constexpr int kW4gThreads = 32 * (6 + kW4gDec);
constexpr uint32_t kW4gA = kW4gM * kW4gK * 2;    // bytes of a stage's A: two 64-column tiles

template <int BN>
struct W4GSmem {
    static constexpr uint32_t kB = BN * kW4gK * 2;
    static constexpr uint32_t kTiles = kW4gStages * (kW4gA + kB);
    static constexpr uint32_t kScratch = 4 * 2048;  // epilogue: per warp 32 rows of 64 bytes
    static constexpr uint32_t kBytes = 1024 + kTiles + 128 + kScratch;
};

struct W4Tile {
    int m0, n_idx, rows, a_row, src, nk;
    int out_row0;        // up: first h row of the group
    const uint8_t* w;    // the group's matrix
};

// Tile t (tiles are visited in increasing order, so the group cursor g only advances).
template <int WHICH>
__device__ __forceinline__ bool w4_find_tile(const W4GemmArgs& p, const LayerArgs& a, int t, int& g, W4Tile& ti) {
    if (WHICH == kW4GLinear) {
        const int mt = (p.T + kW4gM - 1) / kW4gM;
        ti.n_idx = t / mt;
        ti.m0 = (t - ti.n_idx * mt) * kW4gM;
        ti.rows = p.T;
        ti.a_row = 0;
        ti.src = 0;
        ti.w = p.w[0];
    } else {
        const int32_t* start = WHICH == kW4GUp ? a.up_tiles : a.dn_tiles;
        const int ng = *a.n_groups;
        while (g < ng && t >= start[g + 1]) ++g;
        if (g >= ng) return false;
        const GemmGroup G = WHICH == kW4GUp ? a.up_groups[g] : a.dn_groups[g];
        const int mt = (G.rows + kW4gM - 1) / kW4gM, local = t - start[g];
        ti.n_idx = local / mt;
        ti.m0 = (local - ti.n_idx * mt) * kW4gM;
        ti.rows = G.rows;
        ti.a_row = G.a_row0;
        ti.src = G.src;
        ti.out_row0 = G.out_row0;
        ti.w = G.src ? p.w[1] : p.w[0] + (size_t)(G.b_row0 / p.rows[0]) * p.matrix_bytes;
    }
    ti.nk = ((ti.src ? p.cols[1] : p.cols[0]) + kW4gK - 1) / kW4gK;
    return true;
}

// One record's share of a lane, from global memory.
template <int FMT, int G>
__device__ __forceinline__ void w4_load_global(const uint8_t* rec, int lane, W4Frag<FMT, G>& f) {
    constexpr int N = W4Rec<FMT, G>::kGroups;
    f.lo = ld_stream(rec + lane * 16);
    f.hi = ld_stream(rec + 512 + lane * 16);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const int row = (lane >> 2) + 8 * h;
        const uint8_t* at = rec + W4Rec<FMT, G>::kScales + row * (2 * N);
        if constexpr (N == 4) {
            const uint2 v = __ldg(reinterpret_cast<const uint2*>(at));
            f.s[h][0] = v.x;
            f.s[h][1] = v.y;
        } else if constexpr (N == 2) {
            f.s[h][0] = __ldg(reinterpret_cast<const unsigned int*>(at));
        } else {
            f.s[h][0] = __ldg(reinterpret_cast<const unsigned short*>(at));
        }
        f.z[h] = 0;
        if (FMT == MOE_W4_INT4_ZP) {
            const uint8_t* za = rec + W4Rec<FMT, G>::kZeros + row * N;
            f.z[h] = N == 4   ? __ldg(reinterpret_cast<const unsigned int*>(za))
                     : N == 2 ? __ldg(reinterpret_cast<const unsigned short*>(za))
                              : __ldg(za);
        }
    }
}

// The group's scale in both halves of a word.
template <int FMT, int G>
__device__ __forceinline__ uint32_t w4_scale2(const W4Frag<FMT, G>& f, int h, int gi) {
    return __byte_perm(f.s[h][gi >> 1], 0u, (gi & 1) ? 0x3232 : 0x1010);
}

// Writes one record as bf16 into a stage's two 64-column tiles: rows r0 + g and r1 + g (multiples
// of 8), tile stride `tile`.
template <int FMT, int G>
__device__ __forceinline__ void w4_expand(const W4Frag<FMT, G>& f, uint32_t sb, uint32_t tile, int r0, int r1, int lane) {
    const uint32_t g = (uint32_t)lane >> 2, t = (uint32_t)lane & 3u;
    const bool odd = g & 1u;
    const uint32_t w[2][4] = {{f.lo.x, f.lo.y, f.lo.z, f.lo.w}, {f.hi.x, f.hi.y, f.hi.z, f.hi.w}};
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const uint32_t row = sb + ((uint32_t)(h ? r1 : r0) + g) * 128u;
#pragma unroll
        for (int c = 0; c < 4; c += 2) {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                // even rows: piece c + i; odd rows: the other one
                const uint32_t word = odd ? w[h][c + 1 - i] : w[h][c + i];
                const int ge = (c + i) * 32 / G, go = (c + 1 - i) * 32 / G;
                const uint32_t s = ge == go ? w4_scale2(f, h, ge) : odd ? w4_scale2(f, h, go) : w4_scale2(f, h, ge);
                const uint32_t bias = ge == go ? w4_bias(f, h, ge) : odd ? w4_bias(f, h, go) : w4_bias(f, h, ge);
                uint32_t v[4];
                w4_decode<FMT>(word, bias, v);
#pragma unroll
                for (int j = 0; j < 4; ++j) v[j] = bf2_mul(v[j], s);
                const uint32_t chunk = (odd ? (uint32_t)(1 - i) : (uint32_t)i) * 4u + t;
                sts128(row + (uint32_t)(c >> 1) * tile + ((chunk ^ g) << 4), v);
            }
        }
    }
}

__device__ __forceinline__ void w4g_timeout(uint32_t* err, volatile int* abort_flag) {
    atomicOr(err, ERR_TIMEOUT);
    *abort_flag = 1;
}

template <int WHICH, int FMT, int G, int BN>
__global__ void __launch_bounds__(kW4gThreads, 1)
    k_w4_gemm(const __grid_constant__ CUtensorMap tmA0, const __grid_constant__ CUtensorMap tmA1,
              const __grid_constant__ W4GemmArgs p, const __grid_constant__ LayerArgs a) {
    constexpr int kRec = W4Rec<FMT, G>::kBytes;
    constexpr int kStrips = BN / 16;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = smem_u32(smem_raw);
    uint8_t* smem = smem_raw + (((raw + 1023u) & ~1023u) - raw);
    uint8_t* sA = smem;
    uint8_t* sB = smem + kW4gStages * kW4gA;
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + W4GSmem<BN>::kTiles);
    uint64_t* full = bars;
    uint64_t* empty = bars + kW4gStages;
    uint64_t* fullA = bars + 2 * kW4gStages;  // gathered A rows
    uint64_t* accf = bars + 3 * kW4gStages;
    uint64_t* acce = accf + 2;
    uint64_t* mma_done = acce + 2;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(mma_done + 1);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
    uint8_t* scratch = smem + W4GSmem<BN>::kTiles + 128;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint64_t limit = p.wait_ns;

    if (threadIdx.x == 0) {
        for (int s = 0; s < kW4gStages; ++s) {
            mbar_init(&full[s], 1 + kW4gDec);
            mbar_init(&empty[s], 1);
            mbar_init(&fullA[s], 32 * kW4gDec);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(&accf[b], 1);
            mbar_init(&acce[b], 4);
        }
        mbar_init(mma_done, 1);
        *abort_flag = 0;
        fence_mbar_init();
        tma_prefetch_desc(&tmA0);
        tma_prefetch_desc(&tmA1);
    }
    if (warp == 1) {
        tmem_alloc(tmem_slot, 2 * BN <= 256 ? 256 : 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    grid_dep_wait();  // the set-up above overlaps the previous kernel's end
    grid_dep_launch();
    const int total = WHICH == kW4GLinear ? ((p.T + kW4gM - 1) / kW4gM) * ((p.rows[0] + BN - 1) / BN)
                                          : (WHICH == kW4GUp ? a.up_tiles : a.dn_tiles)[*a.n_groups];

    if (warp == 0 && lane == 0) {
        // ---------------- TMA producer: A, except a routed expert's token rows
        int g = 0, it = 0;
        bool issued[kW4gStages] = {};
        uint32_t par[kW4gStages] = {};
        for (int t = blockIdx.x; t < total && !*abort_flag; t += gridDim.x) {
            W4Tile ti;
            if (!w4_find_tile<WHICH>(p, a, t, g, ti)) break;
            const CUtensorMap* mA = ti.src ? &tmA1 : &tmA0;
            for (int kb = 0; kb < ti.nk; ++kb, ++it) {
                const int s = it % kW4gStages;
                const uint32_t ph = (uint32_t)(it / kW4gStages) & 1u;
                if (!mbar_wait(&empty[s], ph ^ 1u, limit)) {
                    w4g_timeout(p.err, abort_flag);
                    break;
                }
                const bool gathered = WHICH == kW4GUp && !ti.src;
                mbar_arrive_expect_tx(&full[s], gathered ? 0u : kW4gA);
                if (!gathered) {
                    tma_load_2d(sA + s * kW4gA, mA, &full[s], kb * kW4gK, ti.a_row + ti.m0);
                    tma_load_2d(sA + s * kW4gA + kW4gA / 2, mA, &full[s], kb * kW4gK + 64, ti.a_row + ti.m0);
                }
                issued[s] = true;
                par[s] = ph;
            }
        }
        // every copy issued must land before shared memory is released
        for (int s = 0; s < kW4gStages; ++s)
            if (issued[s] && !mbar_wait(&full[s], par[s], limit)) w4g_timeout(p.err, abort_flag);
    } else if (warp == 1 && lane == 0) {
        // ---------------- MMA issuer
        constexpr uint32_t idesc = idesc_bf16_f32(kW4gM, BN);
        int g = 0, it = 0, local = 0;
        for (int t = blockIdx.x; t < total && !*abort_flag; t += gridDim.x, ++local) {
            W4Tile ti;
            if (!w4_find_tile<WHICH>(p, a, t, g, ti)) break;
            const int b = local & 1;
            if (!mbar_wait(&acce[b], ((uint32_t)(local >> 1) & 1u) ^ 1u, limit)) {
                w4g_timeout(p.err, abort_flag);
                break;
            }
            tc_fence_after();
            const uint32_t d = tmem + (uint32_t)(b * BN);
            bool ok = true;
            for (int kb = 0; kb < ti.nk; ++kb, ++it) {
                const int s = it % kW4gStages;
                const uint32_t ph = (uint32_t)(it / kW4gStages) & 1u;
                if (!mbar_wait(&full[s], ph, limit) || (WHICH == kW4GUp && !mbar_wait(&fullA[s], ph, limit))) {
                    w4g_timeout(p.err, abort_flag);
                    ok = false;
                    break;
                }
                if (WHICH == kW4GUp) fence_proxy_async_smem();  // the gathered rows
                tc_fence_after();
                const uint32_t a_addr = smem_u32(sA + s * kW4gA), b_addr = smem_u32(sB + s * W4GSmem<BN>::kB);
#pragma unroll
                for (int kk = 0; kk < kW4gK / 16; ++kk) {
                    const uint32_t o = (uint32_t)(kk & 3) * 32u;
                    mma_bf16(d, sdesc_kmajor_sw128(a_addr + (uint32_t)(kk >> 2) * (kW4gA / 2) + o),
                             sdesc_kmajor_sw128(b_addr + (uint32_t)(kk >> 2) * (W4GSmem<BN>::kB / 2) + o), idesc, (kb | kk) != 0);
                }
                mma_commit(&empty[s]);
            }
            if (!ok) break;
            mma_commit(&accf[b]);
        }
        mma_commit(mma_done);
        if (!mbar_wait(mma_done, 0, limit)) w4g_timeout(p.err, abort_flag);
    } else if (warp >= 6) {
        // ---------------- decoders: warp w takes strip w of the tile; gatherers: 8 lanes to a row's
        // 128-byte piece, rows tid / 8 and tid / 8 + 64
        const int dw = warp - 6, tid = threadIdx.x - 6 * 32;
        const uint32_t c8 = (uint32_t)(lane & 7);
        const uint64_t pol = l2_evict_last();  // each token row is read by K experts
        const int r0 = WHICH == kW4GUp ? dw * 8 : dw * 16, r1 = WHICH == kW4GUp ? BN / 2 + dw * 8 : dw * 16 + 8;
        int g = 0, it = 0, t = blockIdx.x, kb = 0;
        W4Tile ti;
        const uint8_t* rec = nullptr;  // this warp's records of the tile (NULL: none)
        auto locate = [&]() -> bool {
            if (t >= total || !w4_find_tile<WHICH>(p, a, t, g, ti)) return false;
            const int strip = ti.n_idx * kStrips + dw, strips = ((ti.src ? p.rows[1] : p.rows[0]) + 15) / 16;
            rec = dw < kStrips && strip < strips ? ti.w + (size_t)strip * ti.nk * kRec : nullptr;
            return true;
        };
        bool more = locate();
        W4Frag<FMT, G> nxt = {};
        if (more && rec) w4_load_global<FMT, G>(rec, lane, nxt);
        const bf16* arow[2] = {nullptr, nullptr};
        uint32_t live = 0;
        while (more && !*abort_flag) {
            const W4Frag<FMT, G> cur = nxt;
            const bool have = rec != nullptr, gathered = WHICH == kW4GUp && !ti.src;
            const int kcur = kb;
            if (WHICH == kW4GUp && kb == 0 && gathered) {
                live = 0;
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const int m = ti.m0 + (tid >> 3) + 64 * i;
                    arow[i] = a.x + c8 * 8;
                    if (m < ti.rows) {
                        arow[i] += (size_t)(a.perm[ti.a_row + m] / a.K) * a.H;
                        live |= 1u << i;
                    }
                }
            }
            if (++kb == ti.nk) {
                kb = 0;
                t += gridDim.x;
                more = locate();
            }
            if (more && rec) w4_load_global<FMT, G>(rec + (size_t)kb * kRec, lane, nxt);
            const int s = it % kW4gStages;
            const uint32_t ph = (uint32_t)(it / kW4gStages) & 1u;
            ++it;
            if (!__all_sync(0xffffffffu, mbar_wait(&empty[s], ph ^ 1u, limit))) {
                if (lane == 0) w4g_timeout(p.err, abort_flag);
                break;
            }
            if (WHICH == kW4GUp) {
                if (gathered) {
#pragma unroll
                    for (int j = 0; j < 2; ++j)
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            const uint32_t r = (uint32_t)(tid >> 3) + 64u * i;
                            cp_async16(smem_u32(sA + s * kW4gA) + (uint32_t)j * (kW4gA / 2) + r * 128u + ((c8 ^ (r & 7u)) << 4),
                                       arow[i] + kcur * kW4gK + 64 * j, ((live >> i) & 1u) * 16u, pol);
                        }
                    cp_async_arrive(&fullA[s]);
                } else {
                    mbar_arrive(&fullA[s]);
                }
            }
            if (have)
                w4_expand<FMT, G>(cur, smem_u32(sB + s * W4GSmem<BN>::kB), W4GSmem<BN>::kB / 2, r0, r1, lane);
            fence_proxy_async_smem();  // the tensor core reads these rows through the async proxy
            __syncwarp();
            if (lane == 0) mbar_arrive(&full[s]);
        }
        cp_async_wait_all();  // no copy may be in flight when the CTA exits
    } else if (warp >= 2) {
        // ---------------- epilogue: TMEM lanes 32 * (warp % 4) .. + 31, one accumulator row each
        const int q = warp & 3, r = q * 32 + lane;
        const uint32_t scr = smem_u32(scratch) + (uint32_t)q * 2048u;
        int g = 0, local = 0;
        for (int t = blockIdx.x; t < total && !*abort_flag; t += gridDim.x, ++local) {
            W4Tile ti;
            if (!w4_find_tile<WHICH>(p, a, t, g, ti)) break;
            const int b = local & 1, m = ti.m0 + r;
            const bool row_live = m < ti.rows;
            // the row's destination, read before the accumulator wait
            int tok = m, slot = a.K;
            float sc = 0.f;
            if (WHICH == kW4GDown && row_live) {
                if (ti.src) {
                    sc = a.sgate[m];
                } else {
                    const int pv = a.perm[ti.a_row + m];
                    tok = pv / a.K;
                    slot = pv - tok * a.K;
                    sc = a.topw[pv];
                }
            }
            if (!__all_sync(0xffffffffu, mbar_wait(&accf[b], (uint32_t)(local >> 1) & 1u, limit))) {
                if (lane == 0) w4g_timeout(p.err, abort_flag);
                break;
            }
            tc_fence_after();
            const uint32_t tb = tmem + ((uint32_t)(q * 32) << 16) + (uint32_t)(b * BN);
            if (WHICH == kW4GUp) {
                constexpr int FH = BN / 2;
                bf16* hrow = a.h + (size_t)(ti.out_row0 + m) * a.Imax + ti.n_idx * FH;
#pragma unroll 1
                for (int c = 0; c < FH / 16; ++c) {
                    uint32_t gv[16], uv[16];
                    tmem_ld16(tb + c * 16, gv);
                    tmem_ld16(tb + FH + c * 16, uv);
                    tmem_ld_wait();
                    if (row_live) {
#pragma unroll
                        for (int j = 0; j < 2; ++j) {
                            uint32_t o[4];
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                const int k = j * 8 + i * 2;
                                o[i] = pack_bf16x2(silu(__uint_as_float(gv[k])) * __uint_as_float(uv[k]),
                                                   silu(__uint_as_float(gv[k + 1])) * __uint_as_float(uv[k + 1]));
                            }
                            reinterpret_cast<uint4*>(hrow + c * 16)[j] = make_uint4(o[0], o[1], o[2], o[3]);
                        }
                    }
                }
            } else {
                // 32 columns of the warp's 32 rows at a time through shared memory (16-byte pieces
                // swizzled by row), so that a store instruction writes 8 rows x 64 contiguous bytes
                const int N = WHICH == kW4GLinear ? p.rows[0] : a.H;
                bf16* orow = WHICH == kW4GLinear ? p.out + (size_t)m * N
                                                 : a.Yb + ((size_t)tok * (a.K + 1) + slot) * a.H;
                const bool whole = (N & 7) == 0;
#pragma unroll 1
                for (int c = 0; c < BN / 32; ++c) {
                    uint32_t v[32];
                    tmem_ld32(tb + c * 32, v);
                    tmem_ld_wait();
                    const int n0 = ti.n_idx * BN + c * 32;
                    if (n0 >= N) break;
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        uint32_t o[4];
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const int k = j * 8 + i * 2;
                            float x0 = __uint_as_float(v[k]), x1 = __uint_as_float(v[k + 1]);
                            if (WHICH == kW4GDown) {
                                x0 *= sc;
                                x1 *= sc;
                            } else if (p.bias) {
                                x0 += n0 + k < N ? __bfloat162float(p.bias[n0 + k]) : 0.f;
                                x1 += n0 + k + 1 < N ? __bfloat162float(p.bias[n0 + k + 1]) : 0.f;
                            }
                            o[i] = pack_bf16x2(x0, x1);
                        }
                        sts128(scr + (uint32_t)lane * 64u + (((uint32_t)j ^ (((uint32_t)lane >> 1) & 3u)) << 4), o);
                    }
                    __syncwarp();
                    if (whole) {
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const uint32_t rr = (uint32_t)(lane >> 2) + 8u * i, pc = (uint32_t)(lane & 3);
                            const uint4 o = lds128_smem(scr + rr * 64u + ((pc ^ ((rr >> 1) & 3u)) << 4));
                            bf16* dst = reinterpret_cast<bf16*>(__shfl_sync(0xffffffffu, reinterpret_cast<uintptr_t>(orow), (int)rr));
                            if (__shfl_sync(0xffffffffu, (int)row_live, (int)rr) && n0 + (int)pc * 8 < N)
                                *reinterpret_cast<uint4*>(dst + n0 + pc * 8) = o;
                        }
                    } else {  // rows that are not 16-byte aligned: one element a lane
                        for (int rr = 0; rr < 32; ++rr) {
                            const uint32_t at = scr + (uint32_t)rr * 64u + ((((uint32_t)lane >> 3) ^ (((uint32_t)rr >> 1) & 3u)) << 4) + ((uint32_t)lane & 7u) * 2u;
                            uint16_t e;
                            asm volatile("ld.shared.u16 %0, [%1];" : "=h"(e) : "r"(at) : "memory");
                            bf16* dst = reinterpret_cast<bf16*>(__shfl_sync(0xffffffffu, reinterpret_cast<uintptr_t>(orow), rr));
                            if (__shfl_sync(0xffffffffu, (int)row_live, rr) && n0 + lane < N) dst[n0 + lane] = __ushort_as_bfloat16(e);
                        }
                    }
                    __syncwarp();
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&acce[b]);
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, 2 * BN <= 256 ? 256 : 512);
    }
}

template <int WHICH, int FMT, int G, int BN>
cudaError_t launch_w4_gemm_t(const W4GemmArgs& p, const CUtensorMap& a0, const CUtensorMap& a1, const LayerArgs& a, cudaStream_t s) {
    static bool configured[64] = {};
    int dev = 0;
    cudaGetDevice(&dev);
    if (dev < 0 || dev >= 64) dev = 0;
    constexpr int bytes = (int)W4GSmem<BN>::kBytes;
    if (!configured[dev]) {
        const cudaError_t e =
            cudaFuncSetAttribute(k_w4_gemm<WHICH, FMT, G, BN>, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
        if (e != cudaSuccess) return e;
        configured[dev] = true;
    }
    int grid = a.num_sms;
    if (WHICH == kW4GLinear) {
        const long long tiles = (long long)((p.T + kW4gM - 1) / kW4gM) * ((p.rows[0] + BN - 1) / BN);
        if (tiles < grid) grid = (int)tiles;
    }
    cudaError_t e;
    const int kernel = WHICH == kW4GLinear ? MOE_KERNEL_W4_LINEAR : WHICH == kW4GUp ? MOE_KERNEL_GATE_UP : MOE_KERNEL_DOWN;
    MOE_LAUNCH(kernel, s,
               (e = launch_pdl(k_w4_gemm<WHICH, FMT, G, BN>, dim3(grid), dim3(kW4gThreads), (size_t)bytes, s, a0, a1, p, a)));
    return e;
}

template <int FMT>
cudaError_t launch_w4_gemm_f(int group, int which, const W4GemmArgs& p, const CUtensorMap& a0, const CUtensorMap& a1,
                             const LayerArgs& a, int bn, cudaStream_t s) {
#define MOE_W4_CASE(W, G) \
    if (which == W && group == G) \
        return bn == 256 ? launch_w4_gemm_t<W, FMT, G, 256>(p, a0, a1, a, s) : launch_w4_gemm_t<W, FMT, G, 128>(p, a0, a1, a, s)
    MOE_W4_CASE(kW4GLinear, 32); MOE_W4_CASE(kW4GLinear, 64); MOE_W4_CASE(kW4GLinear, 128);
    MOE_W4_CASE(kW4GUp, 32); MOE_W4_CASE(kW4GUp, 64); MOE_W4_CASE(kW4GUp, 128);
    MOE_W4_CASE(kW4GDown, 32); MOE_W4_CASE(kW4GDown, 64); MOE_W4_CASE(kW4GDown, 128);
#undef MOE_W4_CASE
    return cudaErrorInvalidValue;
}

// One translation unit per format (compiled in parallel).
cudaError_t launch_w4_gemm_int4(int group, int which, const W4GemmArgs& p, const CUtensorMap& a0, const CUtensorMap& a1,
                                const LayerArgs& a, int bn, cudaStream_t s);
cudaError_t launch_w4_gemm_int4_zp(int group, int which, const W4GemmArgs& p, const CUtensorMap& a0, const CUtensorMap& a1,
                                   const LayerArgs& a, int bn, cudaStream_t s);
cudaError_t launch_w4_gemm_e2m1(int group, int which, const W4GemmArgs& p, const CUtensorMap& a0, const CUtensorMap& a1,
                                const LayerArgs& a, int bn, cudaStream_t s);

#endif

}  // namespace moe
