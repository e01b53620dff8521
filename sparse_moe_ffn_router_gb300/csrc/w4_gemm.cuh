// w4_gemm.cuh -- the products of packed 4-bit weights with many tokens, on the 5th-generation
// tensor cores (tcgen05 + TMEM + TMA).
//
// D[128 weight rows, N tokens] = A . B^T with the weights as the A operand in tensor memory. The bf16
// weights do not exist in memory: decoder warps read the packed records (a thread owns a weight row
// of a record: 64 bytes of codes, the columns in order), decode them, multiply by the group's scale
// and store bf16 pairs straight into TMEM (tcgen05.st, lane = weight row, column = pair of columns).
// So a weight passes through no shared memory at all: with the weights staged there as the B operand
// (the other way round) the stores, the token tiles and the MMAs' reads together came to more than the
// 128 bytes a cycle of shared memory, and the tensor cores ran at half rate. B, the token rows (h rows
// for down), K-major bf16 tiles in shared memory, comes by TMA, gathered from x four rows a copy for a
// routed expert's gate_up. A weight is rounded once, to bf16(s * v): the tensor core takes bf16 operands and
// its accumulator spans all of K, so a scale per 32 to 128 columns cannot be applied behind it; the
// error is at most half a bf16 step a weight (2^-8), of the size of the roundings of h and Y.
//
// A tile is 256 weight rows (16 strips; for gate_up 128 features) by at most 128 tokens, as two MMAs of
// 128 rows that share a stage's token rows (with 128-row tiles the token rows came from L2 twice as
// often, ~8 TB/s, and bound the kernel). The tokens of a group are split evenly over its token tiles and N
// is rounded up to 16, so a group of few tokens costs little tensor time. One persistent CTA per SM walks
// a run of tiles (group, row tile, token tile; the token tiles that share weights run back to back). TMEM:
// an accumulator of 128 columns for each row half and four A stages of 128 columns of K (64 TMEM columns
// each), two to a half. Each half has an issuer of its own: with one thread for both, its waits and commits
// were as long as the MMAs. Roles:
//   warps 0, 27 TMA producers                     warps 2-5, 6-9  epilogue (TMEM lane quadrants) of row half 0, 1
//   warps 1, 26 MMA issuers of the row halves
//   warps 10-25 decoders: four groups of four warps, group j writes A stage j, warp w lanes
//               32 (w % 4) .. + 31
//
// Measured: linear 4096 x 2048 by 4096 tokens 53 us (1.30 PFLOP/s, 0.70 of the measured cuBLAS rate; the
// tensor pipe is active 63 % of the time), the MoE layer of 4096 tokens and 256 experts 182 us in gate_up
// and 133 us in down of 380. What is left is the decoders' and the epilogue's share of the issue slots (68 %)
// and the A stages' hand-over. Neither alone gives much: a stage handed over in two halves took that layer from
// 390 to 434 us, a second accumulator for tiles of up to 64 tokens to 414; a third one for down in the place of its
// second A stages 382 against 380; accumulators read whole before anything is stored 418 (registers).
#pragma once

#include "launch.h"
#include "w4.cuh"

namespace moe {

enum : int { kW4GLinear = 0, kW4GUp = 1, kW4GDown = 2 };

constexpr int kW4gRows = 256;    // weight rows of a tile: two halves of 128
constexpr int kW4gTok = 128;     // tokens of a tile, at most
constexpr int kW4gGroups = 257;  // routed experts and the shared one, at most

struct W4GemmArgs {
    const uint8_t* w[2];   // packed matrices: routed (or linear), shared
    size_t matrix_bytes;   // of one routed matrix
    int rows[2], cols[2];  // of one matrix
    const bf16* bias;      // linear
    bf16* out;             // linear [T, rows]
    int T, tok_tiles;      // linear: token rows and their tiles
    uint32_t* err;
    uint64_t wait_ns;
};

// a0, a1: tensor maps of the token rows (linear, routed down; shared), boxes of 64 columns by 32 rows.
cudaError_t launch_w4_gemm(int format, int group, int which, const W4GemmArgs& p, const CUtensorMap& a0,
                           const CUtensorMap& a1, const LayerArgs& a, cudaStream_t s);

#ifdef __CUDACC__

constexpr int kW4gK = 128;                       // columns of a stage
constexpr int kW4gAStages = 4, kW4gBStages = 5;  // (two A stages to a row half; a sixth B stage would take the L1 that
                                                 // the records pass through: layer of 4096 tokens 388 against 380 us)
constexpr int kW4gEpi = 8, kW4gDec = 16;         // epilogue and decoder warps
constexpr int kW4gIssuer1 = 2 + kW4gEpi + kW4gDec;
constexpr int kW4gProducer1 = kW4gIssuer1 + 1;
constexpr int kW4gThreads = 32 * (kW4gProducer1 + 1);
constexpr uint32_t kW4gB = kW4gTok * kW4gK * 2;  // bytes of a B stage: two 64-column tiles
constexpr uint32_t kW4gChunk = 16 * 272;         // epilogue: 16 tokens of 128 bf16 rows
constexpr uint32_t kW4gACol = 2 * kW4gTok;       // first TMEM column of the A stages
static_assert(kW4gACol + kW4gAStages * (kW4gK / 2) <= 512, "TMEM columns");

struct W4GSmem {
    static constexpr uint32_t kTiles = kW4gBStages * kW4gB;
    static constexpr uint32_t kStage = kTiles;                   // epilogue: two chunks for each team
    static constexpr uint32_t kTok = kStage + 4 * kW4gChunk;     // down: output row and scale of each token, per epilogue warp
    static constexpr uint32_t kBars = kTok + 8 * kW4gTok * 8;
    static constexpr uint32_t kTab = kBars + 256;
    static constexpr uint32_t kBytes = 1024 + kTab + (kW4gGroups + 1) * 4 + kW4gGroups * 20 + 12;
    static_assert(kBytes <= 227 * 1024, "shared memory");
};

struct W4Tile {
    int m0, mt, n;       // first token of the tile in its group, tokens, tokens rounded up to 16
    int row0, halves;    // first weight row, row halves (1 when the second lies past the matrix)
    int b_row, src, nk;  // first B row of the group, 1: shared, stages
    int out_row0;        // up: first h row of the group
    const uint8_t* w;    // the group's matrix
};

// A group as the tiles need it (in shared memory for up and down).
struct W4Group {
    int rows, b_row, out_row;
    int matrix;      // of the routed weights; -1: the shared ones
    uint32_t tiles;  // token tiles << 8 | tokens of one
};

__host__ __device__ __forceinline__ int w4_row_tiles(int rows) { return (rows + kW4gRows - 1) / kW4gRows; }
__host__ __device__ __forceinline__ int w4_tok_tiles(int rows) { return (rows + kW4gTok - 1) / kW4gTok; }
// A tile's time, in arbitrary units: its stages, each about as long as 160 tokens' MMAs and those of its tokens.
__device__ __forceinline__ uint32_t w4_tile_cost(int cols, int per) {
    return (uint32_t)((cols + 127) / 128) * (uint32_t)(10 + (per + 15) / 16);
}

// A CTA's tiles: a run of (group, row tile, token tile), cut where the running cost passes the CTA's share of
// the whole. Every role walks the same tiles; with tiles taken in turn by all CTAs instead, finding the next
// one (a search over the groups and two divisions) was as long as a stage.
template <int WHICH>
struct W4Walk {
    const W4GemmArgs& p;
    const W4Group* groups;
    int g, i, r, tok_tiles, row_tiles, per, rows;
    uint32_t pos, hi, cost;
    W4Tile ti;

    // cost: prefix of the groups' costs (n_groups + 1); linear: none, one group of p.tok_tiles
    __device__ __forceinline__ W4Walk(const W4GemmArgs& args, const W4Group* gr, const uint32_t* prefix, int n) : p(args), groups(gr) {
        const int lane = threadIdx.x & 31;
        const uint32_t total = WHICH == kW4GLinear ? (uint32_t)(p.tok_tiles * w4_row_tiles(p.rows[0])) : prefix[n];
        pos = (uint32_t)((uint64_t)total * blockIdx.x / gridDim.x);
        hi = (uint32_t)((uint64_t)total * (blockIdx.x + 1) / gridDim.x);
        g = 0;
        if (WHICH != kW4GLinear) {
            for (int g0 = 0; g0 < n; g0 += 32)
                g += __popc(__ballot_sync(0xffffffffu, g0 + lane < n && prefix[g0 + lane + 1] <= pos));
        }
        const uint32_t first = WHICH == kW4GLinear ? 0u : prefix[g];
        group();
        const uint32_t local = (pos - first + cost - 1) / cost;  // the first tile that starts in the share
        pos = first + local * cost;
        r = (int)(local / (uint32_t)tok_tiles);
        i = (int)local - r * tok_tiles;
    }
    __device__ __forceinline__ void group() {
        if (WHICH == kW4GLinear) {
            tok_tiles = p.tok_tiles;
            rows = p.T;
            per = (int)(((unsigned)rows + (unsigned)tok_tiles - 1u) / (unsigned)tok_tiles);  // (the sum may pass 2^31)
            ti.b_row = ti.src = ti.out_row0 = 0;
            ti.w = p.w[0];
            cost = 1;
        } else {
            const W4Group G = groups[g];
            tok_tiles = (int)(G.tiles >> 8);
            per = (int)(G.tiles & 0xffu);
            rows = G.rows;
            ti.b_row = G.b_row;
            ti.out_row0 = G.out_row;
            ti.src = G.matrix < 0;
            ti.w = G.matrix < 0 ? p.w[1] : p.w[0] + (size_t)G.matrix * p.matrix_bytes;
            cost = w4_tile_cost(p.cols[ti.src], per);
        }
        row_tiles = w4_row_tiles(p.rows[ti.src]);
        ti.nk = (p.cols[ti.src] + kW4gK - 1) / kW4gK;
    }
    // The next tile into ti.
    __device__ __forceinline__ bool next() {
        if (pos >= hi) return false;
        if (r == row_tiles) {
            i = r = 0;
            ++g;
            group();
        }
        ti.m0 = i * per;
        ti.mt = min(per, rows - ti.m0);
        ti.n = (ti.mt + 15) & ~15;
        ti.row0 = r * kW4gRows;
        ti.halves = p.rows[ti.src] - ti.row0 > kW4gRows / 2 ? 2 : 1;
        pos += cost;
        if (++i == tok_tiles) {
            i = 0;
            ++r;
        }
        return true;
    }
};

// A thread's row of one record: codes [t][c], scales and zero points of its groups.
template <int FMT, int G>
struct W4Row {
    uint4 w[4];
    uint32_t s[W4Rec<FMT, G>::kGroups == 4 ? 2 : 1];
    uint32_t z;
};
template <int FMT, int G>
__device__ __forceinline__ void w4_load_row(const uint8_t* rec, int r, W4Row<FMT, G>& f) {
    constexpr int N = W4Rec<FMT, G>::kGroups;
#pragma unroll
    for (int t = 0; t < 4; ++t) f.w[t] = ld_ro(rec + r * 64 + t * 16);
    const uint8_t* at = rec + W4Rec<FMT, G>::kScales + r * (2 * N);
    if constexpr (N == 4) {
        const uint2 v = __ldg(reinterpret_cast<const uint2*>(at));
        f.s[0] = v.x;
        f.s[1] = v.y;
    } else if constexpr (N == 2) {
        f.s[0] = __ldg(reinterpret_cast<const unsigned int*>(at));
    } else {
        f.s[0] = __ldg(reinterpret_cast<const unsigned short*>(at));
    }
    f.z = 0;
    if (FMT == MOE_W4_INT4_ZP) {
        const uint8_t* za = rec + W4Rec<FMT, G>::kZeros + r * N;
        f.z = N == 4   ? __ldg(reinterpret_cast<const unsigned int*>(za))
              : N == 2 ? __ldg(reinterpret_cast<const unsigned short*>(za))
                       : __ldg(za);
    }
}

// Decodes a row's 128 weights into 64 TMEM columns of this thread's lane: bf16(s * v / kUnfold), the factor (a
// power of two) undone on the sums. (A quarter of a weight below 2^-124 is subnormal and keeps fewer bits.)
template <int FMT, int G>
__device__ __forceinline__ void w4_row_to_tmem(const W4Row<FMT, G>& f, uint32_t taddr) {
#pragma unroll
    for (int c = 0; c < 4; ++c) {
        const int gi = c * 32 / G;
        const uint32_t s = __byte_perm(f.s[gi >> 1], 0u, (gi & 1) ? 0x3232 : 0x1010);
        uint32_t b0, b1;
        w4_bias_fold<FMT>(f.z, gi, b0, b1);
        uint32_t v[16];
#pragma unroll
        for (int t = 0; t < 4; ++t) {
            const uint32_t word = c == 0 ? f.w[t].x : c == 1 ? f.w[t].y : c == 2 ? f.w[t].z : f.w[t].w;
            uint32_t q[4];
            w4_decode_fold<FMT>(word, b0, b1, q);
#pragma unroll
            for (int i = 0; i < 4; ++i) v[4 * t + i] = bf2_mul(q[i], s);
        }
        tmem_st16(taddr + 16u * (uint32_t)c, v);
    }
    tmem_st_wait();
}

// g / (1 + e^-g) by CUDA's fast exponential and division: at most ~100 fp32 steps off, far below the bf16
// step of h; where e^-g passes 2^126 it is 0 (the exact value is below 2^-119).
__device__ __forceinline__ float w4_silu(float g) { return __fdividef(g, 1.0f + __expf(-g)); }

__device__ __forceinline__ void w4g_timeout(uint32_t* err, volatile int* abort_flag) {
    atomicOr(err, ERR_TIMEOUT);
    *abort_flag = 1;
}

// Barriers of an epilogue team (four warps).
__device__ __forceinline__ void w4g_team_sync(int team) { asm volatile("bar.sync %0, 128;" ::"r"(team + 1) : "memory"); }
__device__ __forceinline__ bool w4g_team_any(int team, bool v) {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.u32 p, %1, 0;\n\t"
        "bar.red.or.pred q, %2, 128, p;\n\t"
        "selp.u32 %0, 1, 0, q;\n\t}"
        : "=r"(r)
        : "r"((uint32_t)v), "r"(team + 1)
        : "memory");
    return r != 0;
}
__device__ __forceinline__ uint2 lds64_smem(uint32_t at) {
    uint2 v;
    asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(at) : "memory");
    return v;
}

template <int WHICH, int FMT, int G>
__global__ void __launch_bounds__(kW4gThreads, 1)
    k_w4_gemm(const __grid_constant__ CUtensorMap tmB0, const __grid_constant__ CUtensorMap tmB1,
              const __grid_constant__ W4GemmArgs p, const __grid_constant__ LayerArgs a) {
    constexpr int kRec = W4Rec<FMT, G>::kBytes;
    constexpr float kUnfold = W4Fold<FMT>::kUnfold;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = smem_u32(smem_raw);
    uint8_t* smem = smem_raw + (((raw + 1023u) & ~1023u) - raw);
    uint8_t* sB = smem;
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + W4GSmem::kBars);
    uint64_t* fullB = bars;
    uint64_t* emptyB = fullB + kW4gBStages;
    uint64_t* fullA = emptyB + kW4gBStages;
    uint64_t* emptyA = fullA + kW4gAStages;
    uint64_t* accf = emptyA + kW4gAStages;
    uint64_t* acce = accf + 2;  // (an accumulator for each row half)
    uint64_t* mma_done = acce + 2;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(mma_done + 1);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
    static_assert((2 * kW4gBStages + 2 * kW4gAStages + 5) * 8 + 8 <= 256, "barriers");
    uint32_t* prefix = reinterpret_cast<uint32_t*>(smem + W4GSmem::kTab);  // of the groups' costs
    W4Group* groups = reinterpret_cast<W4Group*>(prefix + kW4gGroups + 1);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint64_t limit = p.wait_ns;

    if (threadIdx.x == 0) {
        for (int s = 0; s < kW4gBStages; ++s) {
            mbar_init(&fullB[s], 2);
            mbar_init(&emptyB[s], 2);
        }
        for (int s = 0; s < kW4gAStages; ++s) {
            mbar_init(&fullA[s], 4);
            mbar_init(&emptyA[s], 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(&accf[b], 1);
            mbar_init(&acce[b], 4);
        }
        mbar_init(mma_done, 2);
        *abort_flag = 0;
        fence_mbar_init();
        tma_prefetch_desc(&tmB0);
        tma_prefetch_desc(&tmB1);
    }
    if (warp == 1) {
        tmem_alloc(tmem_slot, 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    grid_dep_wait();  // the set-up above overlaps the previous kernel's end
    grid_dep_launch();
    int n_groups = 1;
    if (WHICH != kW4GLinear) {
        // the dispatch's groups and the prefix of their costs
        n_groups = *a.n_groups;
        if ((int)threadIdx.x < n_groups) {
            const GemmGroup G = (WHICH == kW4GUp ? a.up_groups : a.dn_groups)[threadIdx.x];
            const int tiles = w4_tok_tiles(G.rows), per = (G.rows + tiles - 1) / tiles;  // (at least 65 of several: none is empty)
            groups[threadIdx.x] = {G.rows, G.a_row0, G.out_row0, G.src ? -1 : G.b_row0 / p.rows[0], (uint32_t)tiles << 8 | (uint32_t)per};
            prefix[threadIdx.x + 1] = (uint32_t)(tiles * w4_row_tiles(p.rows[G.src ? 1 : 0])) * w4_tile_cost(p.cols[G.src ? 1 : 0], per);
        }
        __syncthreads();
        if (warp == 0) {
            uint32_t run = 0;
            for (int i0 = 0; i0 < n_groups; i0 += 32) {
                uint32_t v = i0 + lane < n_groups ? prefix[i0 + lane + 1] : 0;
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const uint32_t y = __shfl_up_sync(0xffffffffu, v, o);
                    if (lane >= o) v += y;
                }
                if (i0 + lane < n_groups) prefix[i0 + lane + 1] = run + v;
                run += __shfl_sync(0xffffffffu, v, 31);
            }
            if (lane == 0) prefix[0] = 0;
        }
        __syncthreads();
    }
    W4Walk<WHICH> walk(p, groups, prefix, n_groups);

    if (warp == 0 || warp == kW4gProducer1) {
        // ---------------- TMA producers: B, 64 columns of a stage each. A routed expert's gate_up gathers its token
        // rows from x, four a copy; a warp reads the tokens of a tile ahead, one lane issues (up to 32 copies a
        // stage: one producer for all 128 columns was as long as a stage).
        const int j = warp == 0 ? 0 : 1;
        int* tok = reinterpret_cast<int*>(smem + W4GSmem::kTok) + j * kW4gTok;
        const uint32_t toks = smem_u32(tok);
        int it = 0, pv[kW4gTok / 32] = {};
        auto find = [&]() -> bool {
            if (!walk.next()) return false;
            if (WHICH == kW4GUp && !walk.ti.src) {
#pragma unroll
                for (int i = 0; i < kW4gTok / 32; ++i)  // (rows between the tokens and N read the last token's)
                    pv[i] = a.perm[walk.ti.b_row + walk.ti.m0 + min(lane + 32 * i, walk.ti.mt - 1)];
            }
            return true;
        };
        bool more = find(), ok = true;
        while (more && ok) {
            const W4Tile ti = walk.ti;
            const bool gathered = WHICH == kW4GUp && !ti.src;
            if (gathered) {
#pragma unroll
                for (int i = 0; i < kW4gTok / 32; ++i) tok[lane + 32 * i] = pv[i] / a.K;
                __syncwarp();
            }
            more = find();
            if (elect_one()) {
                const int boxes = (ti.n + 31) / 32;
                for (int kb = 0; kb < ti.nk && !*abort_flag; ++kb, ++it) {
                    const int s = it % kW4gBStages;
                    if (!mbar_wait(&emptyB[s], ((uint32_t)(it / kW4gBStages) & 1u) ^ 1u, limit)) {
                        w4g_timeout(p.err, abort_flag);
                        break;
                    }
                    uint8_t* st = sB + s * kW4gB + j * (kW4gB / 2);
                    if (gathered) {
                        mbar_arrive_expect_tx(&fullB[s], (uint32_t)ti.n * 128u);
                        for (int r = 0; r < ti.n; r += 16) {
                            uint4 q[4];
#pragma unroll
                            for (int i = 0; i < 4; ++i) q[i] = lds128_smem(toks + 4u * (uint32_t)(r + 4 * i));
#pragma unroll
                            for (int i = 0; i < 4; ++i)
                                tma_gather4(smem_u32(st) + (uint32_t)(r + 4 * i) * 128u, &tmB0, &fullB[s], kb * kW4gK + 64 * j, (int)q[i].x,
                                            (int)q[i].y, (int)q[i].z, (int)q[i].w);
                        }
                    } else {
                        const CUtensorMap* mB = ti.src ? &tmB1 : &tmB0;
                        mbar_arrive_expect_tx(&fullB[s], (uint32_t)boxes * 4096u);
                        for (int i = 0; i < boxes; ++i)
                            tma_load_2d(st + i * 4096, mB, &fullB[s], kb * kW4gK + 64 * j, ti.b_row + ti.m0 + 32 * i);
                    }
                }
            }
            __syncwarp();
            it = (int)__reduce_max_sync(0xffffffffu, (unsigned)it);
            ok = !__any_sync(0xffffffffu, *abort_flag != 0);
        }
        // every copy issued must land before shared memory is released
        if (elect_one())
            for (int j = max(0, it - kW4gBStages); j < it; ++j)
                if (!mbar_wait(&fullB[j % kW4gBStages], (uint32_t)(j / kW4gBStages) & 1u, limit)) w4g_timeout(p.err, abort_flag);
    } else if (warp == 1 || warp == kW4gIssuer1) {
        // ---------------- MMA issuers: warp 1 the tiles' first row halves, kW4gIssuer1 the second ones
        if (elect_one()) {
            const int h = warp == 1 ? 0 : 1;
            const uint64_t desc0 = sdesc_kmajor_sw128(smem_u32(sB));
            const uint32_t d = tmem + (uint32_t)(h * kW4gTok);
            uint32_t sb = 0, pb = 0, ia = 0, pacc = 1;  // B stage and its phase, this half's A stages passed, accumulator phase
            bool ok = true;
            while (ok && walk.next() && !*abort_flag) {
                const W4Tile& ti = walk.ti;
                const uint32_t idesc = idesc_bf16_f32(kW4gRows / 2, ti.n);
                const bool mine = h < ti.halves;
                if (mine) {
                    ok = mbar_wait(&acce[h], pacc, limit);
                    pacc ^= 1u;
                }
                for (int kb = 0; kb < ti.nk && ok; ++kb) {
                    ok = mbar_wait(&fullB[sb], pb, limit);
                    if (mine) {
                        const uint32_t sa = (uint32_t)h + 2u * (ia & 1u);
                        ok = ok && mbar_wait(&fullA[sa], (ia >> 1) & 1u, limit);
                        ++ia;
                        if (!ok) break;
                        tc_fence_after();
                        const uint64_t db = desc0 + (uint64_t)(sb * (kW4gB >> 4));
                        const uint32_t acol = tmem + kW4gACol + sa * (uint32_t)(kW4gK / 2);
                        mma_bf16_ta(d, acol, db, idesc, kb != 0);
#pragma unroll
                        for (int kk = 1; kk < kW4gK / 16; ++kk)
                            mma_bf16_ta(d, acol + (uint32_t)(kk * 8), db + (uint64_t)((kk >> 2) * (kW4gB >> 5) + (kk & 3) * 2), idesc, 1u);
                        mma_commit(&emptyA[sa]);
                        mma_commit(&emptyB[sb]);
                    } else if (ok) {
                        mbar_arrive(&emptyB[sb]);
                    }
                    if (++sb == kW4gBStages) {
                        sb = 0;
                        pb ^= 1u;
                    }
                }
                if (!ok)
                    w4g_timeout(p.err, abort_flag);
                else if (mine)
                    mma_commit(&accf[h]);
            }
            mma_commit(mma_done);
            if (!mbar_wait(mma_done, 0, limit)) w4g_timeout(p.err, abort_flag);
        }
    } else if (warp >= 2 + kW4gEpi) {
        // ---------------- decoders
        const int dw = warp - 2 - kW4gEpi, grp = dw >> 2, quad = warp & 3;
        const uint32_t a0 = tmem + kW4gACol + (uint32_t)(grp * (kW4gK / 2)) + ((uint32_t)(quad * 32) << 16);
        // Group j writes A stage j: every second column block of row half j % 2. (A stage belongs to one half, so
        // that its issuer sees every phase of its barrier: tiles of one half only would let the other issuer
        // fall two phases behind.)
        const int half = grp & 1;
        int kb = grp >> 1, nk = 0;
        const uint8_t* strip = nullptr;  // this thread's strip of the tile (NULL: past the matrix)
        auto locate = [&]() -> bool {
            const W4Tile& ti = walk.ti;
            for (;;) {
                kb -= nk;
                if (!walk.next()) return false;
                nk = half < ti.halves ? ti.nk : 0;
                if (kb < nk) break;
            }
            const int i = ti.row0 / 16 + 8 * half + 2 * quad + (lane >> 4), strips = (p.rows[ti.src] + 15) / 16;
            strip = i < strips ? ti.w + (size_t)i * ti.nk * kRec : nullptr;
            return true;
        };
        W4Row<FMT, G> nxt = {};
        auto load = [&]() {
            if (strip) w4_load_row<FMT, G>(strip + kb * kRec, lane & 15, nxt);
        };
        bool more = locate();
        if (more) load();
        for (int round = 0; more && !*abort_flag; ++round) {
            const W4Row<FMT, G> cur = nxt;
            kb += 2;
            if (kb >= nk) more = locate();
            if (more) load();
            if (!__all_sync(0xffffffffu, mbar_wait(&emptyA[grp], ((uint32_t)round & 1u) ^ 1u, limit))) {
                if (lane == 0) w4g_timeout(p.err, abort_flag);
                break;
            }
            tc_fence_after();
            w4_row_to_tmem<FMT, G>(cur, a0);
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&fullA[grp]);
        }
    } else {
        // ---------------- epilogue: TMEM lanes 32 * (warp % 4) .. + 31, one weight row each; a team of
        // four warps to a row half. 16 tokens at a time pass through shared memory, where
        // a token's 128 rows (64 h values) lie together, and leave in pieces of 16 bytes: stored from
        // registers, 64 bytes a warp and token, the scattered rows of Y took longer than down's products.
        const int q = warp & 3, team = warp >= 6;
        constexpr int kPitch = WHICH == kW4GUp ? 144 : 272;  // bytes of a token: 64 or 128 values, and 16 to spread the banks
        const uint32_t stage = smem_u32(smem + W4GSmem::kStage) + (uint32_t)team * 2u * kW4gChunk;
        uint32_t* tk = reinterpret_cast<uint32_t*>(smem + W4GSmem::kTok) + (warp - 2) * 2 * kW4gTok;  // rows, scales
        const uint32_t tks = smem_u32(tk);
        // this lane's 16-byte row of a transposed store: matrix lane / 8, token lane % 8 of its block
        const uint32_t put = stage + (WHICH == kW4GUp ? (uint32_t)((((lane >> 3) & 1) * 8 + (lane & 7)) * kPitch + (q * 2 + (lane >> 4)) * 16)
                                                      : (uint32_t)(((lane >> 4) * 8 + (lane & 7)) * kPitch + q * 64 + ((lane >> 3) & 1) * 16));
        const int ldo = WHICH == kW4GUp ? a.Imax : WHICH == kW4GDown ? a.H : p.rows[0];
        bf16* const out = WHICH == kW4GUp ? a.h : WHICH == kW4GDown ? a.Yb : p.out;
        const bool bulk = WHICH != kW4GLinear || ((ldo & 7) == 0 && (reinterpret_cast<uintptr_t>(out) & 15) == 0);
        uint32_t used = 0, buf = 0;
        // One expert a token: Y stays fp32. With few slots their roundings weigh the most: with every rounding the result
        // was 1.52 times as far from the exact one as its own last rounding alone (1.41 with two experts, 1.27 with eight),
        // without Y's 1.40.
        const bool y32 = WHICH == kW4GDown && a.K == 1;
        W4Tile ti;
        const W4Tile& nx_ti = walk.ti;
        int pv[kW4gTok / 32] = {};
        // the next tile, and down's pairs of its tokens: read a tile ahead
        auto find = [&]() -> bool {
            if (!walk.next()) return false;
            if (WHICH == kW4GDown && !nx_ti.src) {
#pragma unroll
                for (int i = 0; i < kW4gTok / 32; ++i) {
                    const int m = lane + 32 * i;
                    pv[i] = m < nx_ti.mt ? a.perm[nx_ti.b_row + nx_ti.m0 + m] : 0;
                }
            }
            return true;
        };
        bool more = find(), dead = false;
        while (more && !dead) {
            ti = nx_ti;
            if (WHICH == kW4GDown) {
                // output row (token, slot) and scale of each token of the tile
                __syncwarp();  // (stores of fp32 Y may still read the last tile's)
#pragma unroll
                for (int i = 0; i < kW4gTok / 32; ++i) {
                    const int m = lane + 32 * i;
                    if (m < ti.mt) {
                        int tok = ti.m0 + m, slot = a.K;
                        float sc;
                        if (ti.src) {
                            sc = a.sgate[tok];
                        } else {
                            tok = pv[i] / a.K;
                            slot = pv[i] - tok * a.K;
                            sc = a.topw[pv[i]];
                        }
                        tk[m] = (uint32_t)(tok * (a.K + 1) + slot);
                        tk[kW4gTok + m] = __float_as_uint(kUnfold * sc);
                    }
                }
                __syncwarp();
            }
            more = find();
            const int rows = ti.src ? p.rows[1] : p.rows[0];
            if (team < ti.halves) {
                const int h = team;
                const int row0 = ti.row0 + h * (kW4gRows / 2), row = row0 + q * 32 + (lane >> 2);
                float bias[4];  // of rows row + 8 j
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    bias[j] = WHICH == kW4GLinear && p.bias && row + 8 * j < rows ? __bfloat162float(p.bias[row + 8 * j]) : 0.f;
                const int bytes = min(rows - row0, kW4gRows / 2) * (WHICH == kW4GUp ? 1 : 2);  // of a token
                if (!__all_sync(0xffffffffu, mbar_wait(&accf[h], used & 1u, limit))) {
                    if (lane == 0) w4g_timeout(p.err, abort_flag);
                    dead = true;
                }
                // the four warps of a team leave together, as they meet at its barrier
                dead = w4g_team_any(team, dead || *abort_flag);
                if (dead) break;
                ++used;
                tc_fence_after();
                const uint32_t tb = tmem + ((uint32_t)(q * 32) << 16) + (uint32_t)(h * kW4gTok);
                uint32_t nx[16];
                tmem_ld_frag2(tb, nx);
                tmem_ld_frag2(tb + (16u << 16), nx + 8);
#pragma unroll 1
                for (int c0 = 0; c0 < ti.mt; c0 += 16, buf ^= 1u) {
                    float v[16];  // [8 i + 4 b + 2 k + e]: row 16 i + 8 k + lane / 4 of the warp's 32, token 8 b + 2 (lane % 4) + e
                    tmem_ld_wait16(nx);
#pragma unroll
                    for (int c = 0; c < 16; ++c) v[c] = __uint_as_float(nx[c]);
                    if (c0 + 16 < ti.mt) {  // the next 16 tokens
                        tmem_ld_frag2(tb + (uint32_t)c0 + 16u, nx);
                        tmem_ld_frag2(tb + (16u << 16) + (uint32_t)c0 + 16u, nx + 8);
                    } else {  // the accumulator is read
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(&acce[h]);
                    }
                    if (WHICH == kW4GDown) {
#pragma unroll
                        for (int b = 0; b < 2; ++b) {
                            const uint2 e = lds64_smem(tks + (uint32_t)(kW4gTok + c0 + 8 * b + 2 * (lane & 3)) * 4u);
#pragma unroll
                            for (int j = 0; j < 4; ++j) {
                                v[8 * (j >> 1) + 4 * b + 2 * (j & 1)] *= __uint_as_float(e.x);
                                v[8 * (j >> 1) + 4 * b + 2 * (j & 1) + 1] *= __uint_as_float(e.y);
                            }
                        }
                    } else if (WHICH == kW4GLinear) {
#pragma unroll
                        for (int j = 0; j < 16; ++j) v[j] = fmaf(v[j], kUnfold, bias[2 * (j >> 3) + ((j >> 1) & 1)]);
                    }
                    if (y32) {
#pragma unroll
                        for (int j = 0; j < 16; ++j) {
                            const int m = c0 + 8 * ((j >> 2) & 1) + 2 * (lane & 3) + (j & 1), r = row + 16 * (j >> 3) + 8 * ((j >> 1) & 1);
                            if (m < ti.mt && r < rows) a.Y[(size_t)tk[m] * ldo + r] = v[j];
                        }
                        continue;
                    }
                    if (!bulk) {  // rows that are not 16-byte aligned
#pragma unroll
                        for (int j = 0; j < 16; ++j) {
                            const int m = c0 + 8 * ((j >> 2) & 1) + 2 * (lane & 3) + (j & 1), r = row + 16 * (j >> 3) + 8 * ((j >> 1) & 1);
                            if (m < ti.mt && r < rows) out[(size_t)(ti.m0 + m) * ldo + r] = __float2bfloat16_rn(v[j]);
                        }
                        continue;
                    }
                    const uint32_t at = put + buf * kW4gChunk;
                    if (WHICH == kW4GUp) {
                        // rows 0 .. 7 of a strip are gate, 8 .. 15 up: a thread holds both of a feature
                        uint32_t hv[4];
#pragma unroll
                        for (int j = 0; j < 4; ++j) {  // strip j / 2, tokens of block j % 2
                            const float* f = v + 4 * j;
                            hv[j] = pack_bf16x2(w4_silu(kUnfold * f[0]) * (kUnfold * f[2]), w4_silu(kUnfold * f[1]) * (kUnfold * f[3]));
                        }
                        stmatrix4_trans(at, hv[0], hv[1], hv[2], hv[3]);
                    } else {
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            const float* f = v + 8 * i;
                            stmatrix4_trans(at + 32u * i, pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]),
                                            pack_bf16x2(f[6], f[7]));
                        }
                    }
                    constexpr int kLanes = (kPitch - 16) / 16, kPieces = kLanes / 8;  // lanes to a token, 16 bytes each
                    const int piece = lane % kLanes;
                    bf16* dst[kPieces];
#pragma unroll
                    for (int i = 0; i < kPieces; ++i) {
                        const int m = c0 + (q * kPieces + i) * (32 / kLanes) + lane / kLanes;
                        const size_t r = WHICH == kW4GUp ? (size_t)(ti.out_row0 + ti.m0 + m)
                                         : WHICH == kW4GDown ? (size_t)tk[m] : (size_t)(ti.m0 + m);
                        dst[i] = m < ti.mt && piece * 16 < bytes ? out + r * ldo + (WHICH == kW4GUp ? row0 / 2 : row0) + piece * 8 : nullptr;
                    }
                    w4g_team_sync(team);  // (chunks alternate: the buffer is written again after the next chunk's)
                    uint4 o[kPieces];
#pragma unroll
                    for (int i = 0; i < kPieces; ++i)
                        o[i] = lds128_smem(stage + buf * kW4gChunk + (uint32_t)(((q * kPieces + i) * (32 / kLanes) + lane / kLanes) * kPitch + piece * 16));
#pragma unroll
                    for (int i = 0; i < kPieces; ++i)
                        if (dst[i]) *reinterpret_cast<uint4*>(dst[i]) = o[i];
                }
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

template <int WHICH, int FMT, int G>
cudaError_t launch_w4_gemm_t(const W4GemmArgs& args, const CUtensorMap& b0, const CUtensorMap& b1, const LayerArgs& a, cudaStream_t s) {
    static bool configured[64] = {};
    int dev = 0;
    cudaGetDevice(&dev);
    if (dev < 0 || dev >= 64) dev = 0;
    constexpr int bytes = (int)W4GSmem::kBytes;
    if (!configured[dev]) {
        const cudaError_t e =
            cudaFuncSetAttribute(k_w4_gemm<WHICH, FMT, G>, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
        if (e != cudaSuccess) return e;
        configured[dev] = true;
    }
    W4GemmArgs p = args;
    int grid = a.num_sms;
    if (WHICH == kW4GLinear) {
        // A tile's time is about that of its tokens, rounded up to 16, and of 32 more (the handshakes of a
        // stage), so more and smaller token tiles are taken where they fill the waves of CTAs better.
        const int rt = w4_row_tiles(p.rows[0]), least = w4_tok_tiles(p.T);
        long long best = 0;
        // (with many waves there is little to fill)
        const int most = (long long)least * rt <= 8LL * a.num_sms ? least + least / 2 + 1 : least;
        for (int n = least; n <= most; ++n) {
            const int per = (int)(((long long)p.T + n - 1) / n), tiles = (p.T + per - 1) / per;
            const long long cost = (((long long)tiles * rt + a.num_sms - 1) / a.num_sms) * (((per + 15) & ~15) + 32);
            if (best == 0 || cost < best) {
                best = cost;
                p.tok_tiles = tiles;
            }
        }
        if ((long long)p.tok_tiles * rt < grid) grid = p.tok_tiles * rt;
    }
    cudaError_t e;
    const int kernel = WHICH == kW4GLinear ? MOE_KERNEL_W4_LINEAR : WHICH == kW4GUp ? MOE_KERNEL_GATE_UP : MOE_KERNEL_DOWN;
    MOE_LAUNCH(kernel, s,
               (e = launch_pdl(k_w4_gemm<WHICH, FMT, G>, dim3(grid), dim3(kW4gThreads), (size_t)bytes, s, b0, b1, p, a)));
    return e;
}

template <int FMT>
cudaError_t launch_w4_gemm_f(int group, int which, const W4GemmArgs& p, const CUtensorMap& b0, const CUtensorMap& b1,
                             const LayerArgs& a, cudaStream_t s) {
#define MOE_W4_CASE(W, G) \
    if (which == W && group == G) return launch_w4_gemm_t<W, FMT, G>(p, b0, b1, a, s)
    MOE_W4_CASE(kW4GLinear, 32); MOE_W4_CASE(kW4GLinear, 64); MOE_W4_CASE(kW4GLinear, 128);
    MOE_W4_CASE(kW4GUp, 32); MOE_W4_CASE(kW4GUp, 64); MOE_W4_CASE(kW4GUp, 128);
    MOE_W4_CASE(kW4GDown, 32); MOE_W4_CASE(kW4GDown, 64); MOE_W4_CASE(kW4GDown, 128);
#undef MOE_W4_CASE
    return cudaErrorInvalidValue;
}

// One translation unit per format (compiled in parallel).
cudaError_t launch_w4_gemm_int4(int group, int which, const W4GemmArgs& p, const CUtensorMap& b0, const CUtensorMap& b1,
                                const LayerArgs& a, cudaStream_t s);
cudaError_t launch_w4_gemm_int4_zp(int group, int which, const W4GemmArgs& p, const CUtensorMap& b0, const CUtensorMap& b1,
                                   const LayerArgs& a, cudaStream_t s);
cudaError_t launch_w4_gemm_e2m1(int group, int which, const W4GemmArgs& p, const CUtensorMap& b0, const CUtensorMap& b1,
                                const LayerArgs& a, cudaStream_t s);

#endif

}  // namespace moe
