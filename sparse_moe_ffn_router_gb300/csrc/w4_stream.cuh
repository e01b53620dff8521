// w4_stream.cuh -- the weight-streaming products of packed 4-bit weights with few tokens: a linear
// layer, the experts' gate_up and the experts' down projection of the MoE layer.
//
// With few tokens each weight is used a handful of times, so the kernels are bound by reading the
// packed weights once. One persistent CTA per SM: a producer warp walks the CTA's items and copies
// each item's strips (up to 16 records, 17 to 19 KB, one contiguous 1-D TMA bulk copy) into a ring
// of shared-memory stages that keeps ~200 KB of copies in flight; eight consumer warps decode the
// codes in registers into the A operand of warp-level bf16 MMAs (16 weight rows by 8 tokens; a
// stage's 16 rows are too few for the 64/128-row tcgen05 MMA, and the decoded weights are in
// registers already), each over its share of a strip's columns with its token rows held in
// registers; two epilogue warps add the shares in a fixed order and write the results, so the
// consumers never wait for one another. Decoding, not the MMAs, is the consumers' work: about
// 1.4 (integer codes) to 1.9 (E2M1) instructions a weight and lane.
//
// Item: a block of consecutive strips of one matrix by one tile of 8 tokens. A block is as many
// strips as fill a stage (a strip of R <= 16 records is shared by W = 1, 2, 4 or 8 warps of two
// records each, so 8 / W strips to a block); a strip of more than 16 records takes ceil(R / 16)
// stages, its sums staying in the warps' registers.
#pragma once

#include "launch.h"
#include "w4.cuh"

namespace moe {

enum : int { kW4Linear = 0, kW4Up = 1, kW4Down = 2 };

// One call's operands. Group 0 is the shared expert (or the linear layer's matrix, taken first),
// group 1 the routed experts.
struct W4StreamArgs {
    LayerArgs a;        // up, down: the layer (gate_up, down, sgu, sd point to packed weights)
    const uint8_t* w;   // linear: the packed matrix
    const bf16* x;      // linear: [T, cols]
    const bf16* bias;   // linear: [rows] or NULL
    bf16* out;          // linear: [T, rows]
    int rows[2], cols[2];
    size_t matrix_bytes;  // of one routed matrix
    uint32_t* err;
    uint64_t wait_ns;
    int T;
};

struct W4Block {
    int strips, R, wl, ns, nslab, blocks;  // wl: log2 of the warps of a strip; ns: strips of a block
};

__host__ __device__ inline W4Block w4_block(int rows, int cols) {
    W4Block b;
    b.strips = (rows + kW4Strip - 1) / kW4Strip;
    b.R = (cols + kW4Cols - 1) / kW4Cols;
    const int need = ((b.R < 16 ? b.R : 16) + 1) / 2;
    b.wl = 0;
    while ((1 << b.wl) < need) ++b.wl;
    b.ns = 8 >> b.wl;
    b.nslab = (b.R + 15) / 16;
    b.blocks = (b.strips + b.ns - 1) / b.ns;
    return b;
}

cudaError_t launch_w4_stream(int format, int group, int which, const W4StreamArgs& p, cudaStream_t s);

#ifdef __CUDACC__

constexpr int kW4Tok = 8;                 // tokens per item
constexpr int kW4RedBufs = 4;             // partial-sum buffers
constexpr int kW4EpiWarps = 2;
constexpr int kW4Threads = 32 * (kWarps + 1 + kW4EpiWarps);
constexpr int kW4SmemMax = 220 * 1024;

struct W4Meta {
    int group;   // 0 shared / linear, 1 routed; -1: no more items
    int mt;      // tokens
    int row0;    // up: first h row written; down: first h row read
    int strip0;  // first strip of the block
    int key;     // the item's token set: consecutive items with one key use the same rows
    int tok[kW4Tok], slot[kW4Tok];
    float sc[kW4Tok];
};

template <int FMT, int G>
struct W4Ring {
    static constexpr int kStage = 16 * W4Rec<FMT, G>::kBytes;
    static constexpr int kRed = kW4RedBufs * kWarps * 128 * 4;
    static constexpr int kFixed = 1024 + kRed + 24 * (int)sizeof(W4Meta) + 512 + 258 * 4;
    static constexpr int kStages = (kW4SmemMax - kFixed) / kStage < 12 ? (kW4SmemMax - kFixed) / kStage : 12;
    static constexpr int kMetas = kStages + kW4RedBufs + 2;
    static_assert(kStage % 128 == 0 && kMetas <= 24 && (2 * kStages + 2 * kW4RedBufs) * 8 <= 512, "ring");
    static constexpr int kBytes = kFixed + kStages * kStage;
};

// B operands of the warp's two records from its row of the tile: elements k0 + 32 c + 8 t .. + 7 of
// each, zero past the matrix's columns (the packed weights there have scale 0, but the row's memory
// may hold anything) and for the tile's missing tokens. L2 loads (an earlier kernel wrote the rows).
__device__ __forceinline__ void w4_load_frag(uint32_t (&b)[2][1][16], const bf16* row, bool live, int rec0, int nrec, int cols,
                                             int lane) {
#pragma unroll
    for (int r = 0; r < 2; ++r)
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            const int k = (rec0 + r) * kW4Cols + 32 * c + 8 * (lane & 3);
            uint4 v = make_uint4(0u, 0u, 0u, 0u);
            if (live && r < nrec && k < cols) v = __ldcg(reinterpret_cast<const uint4*>(row + k));
            b[r][0][4 * c] = v.x; b[r][0][4 * c + 1] = v.y; b[r][0][4 * c + 2] = v.z; b[r][0][4 * c + 3] = v.w;
        }
}

template <int WHICH, int FMT, int G>
__global__ void __launch_bounds__(kW4Threads, 1) k_w4_stream(const __grid_constant__ W4StreamArgs p) {
    using Ring = W4Ring<FMT, G>;
    constexpr int kRec = W4Rec<FMT, G>::kBytes;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* base = smem_raw + (((smem_u32(smem_raw) + 127u) & ~127u) - smem_u32(smem_raw));
    uint8_t* stages = base;
    float* red = reinterpret_cast<float*>(base + Ring::kStages * Ring::kStage);
    W4Meta* metas = reinterpret_cast<W4Meta*>(reinterpret_cast<uint8_t*>(red) + Ring::kRed);
    uint64_t* full = reinterpret_cast<uint64_t*>(reinterpret_cast<uint8_t*>(metas) + 24 * sizeof(W4Meta));
    uint64_t* empty = full + Ring::kStages;
    uint64_t* rfull = empty + Ring::kStages;
    uint64_t* rempty = rfull + kW4RedBufs;
    int* tiles = reinterpret_cast<int*>(reinterpret_cast<uint8_t*>(full) + 512);
    const LayerArgs& a = p.a;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int G_ = gridDim.x, c_ = blockIdx.x;
    const uint64_t limit = p.wait_ns;
    if (threadIdx.x == 0) {
        for (int s = 0; s < Ring::kStages; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], kWarps);
        }
        for (int s = 0; s < kW4RedBufs; ++s) {
            mbar_init(&rfull[s], kWarps);
            mbar_init(&rempty[s], 1);
        }
        fence_mbar_init();
    }
    __syncthreads();
    const W4Block bg[2] = {w4_block(p.rows[0], p.cols[0]),
                           WHICH == kW4Linear ? W4Block{} : w4_block(p.rows[1], p.cols[1])};

    if (warp == kWarps) {
        // ---------------- producer
        int it = 0, item = 0;
        bool ok = true;
        // one item: its metadata, then its stages (lane 0 copies)
        auto issue = [&](int group, const uint8_t* W, int row0, int blk, int mt, int key, int tok, int slot, float sc) {
            const W4Block& b = bg[group];
            const int strip0 = blk * b.ns, ns = min(b.ns, b.strips - strip0);
            for (int slab = 0; slab < b.nslab && ok; ++slab, ++it) {
                const int s = it % Ring::kStages;
                ok = mbar_wait(&empty[s], (((uint32_t)(it / Ring::kStages)) & 1u) ^ 1u, limit);
                ok = __all_sync(0xffffffffu, ok);
                if (!ok) break;
                if (slab == 0) {
                    W4Meta& m = metas[item % Ring::kMetas];
                    if (lane < kW4Tok) {
                        m.tok[lane] = tok;
                        m.slot[lane] = slot;
                        m.sc[lane] = sc;
                    }
                    if (lane == 0) {
                        m.group = group;
                        m.mt = mt;
                        m.row0 = row0;
                        m.strip0 = strip0;
                        m.key = key;
                    }
                    __syncwarp();
                }
                if (lane == 0) {
                    const int recs = b.nslab == 1 ? ns * b.R : min(16, b.R - 16 * slab);
                    const uint32_t bytes = (uint32_t)(recs * kRec);
                    mbar_arrive_expect_tx(&full[s], bytes);
                    bulk_load(stages + (size_t)s * Ring::kStage, W + ((size_t)strip0 * b.R + 16 * slab) * kRec, bytes,
                              &full[s]);
                }
                __syncwarp();
            }
            ++item;
        };
        const int n0 = bg[0].blocks * ((p.T + kW4Tok - 1) / kW4Tok);  // group 0: (token tile, block) order
        const int i0 = (int)((long long)c_ * n0 / G_), i1 = (int)((long long)(c_ + 1) * n0 / G_);
        if (WHICH == kW4Linear) {
            grid_dep_wait();
            grid_dep_launch();
        }
        for (int i = i0; i < i1 && ok; ++i) {
            const int tile = i / bg[0].blocks, t0 = tile * kW4Tok, mt = min(kW4Tok, p.T - t0);
            const int tok = t0 + (lane < mt ? lane : 0);
            const uint8_t* W = WHICH == kW4Linear ? p.w : reinterpret_cast<const uint8_t*>(WHICH == kW4Up ? a.sgu : a.sd);
            const float sc = WHICH == kW4Down ? a.sgate[tok] : 0.f;
            issue(0, W, (WHICH == kW4Linear ? 0 : (int)a.P) + t0, i - tile * bg[0].blocks, mt, -1 - t0, tok, a.K, sc);
        }
        if (WHICH != kW4Linear) {
            if (WHICH == kW4Up) {
                grid_dep_wait();
                grid_dep_launch();  // the routing is complete: the down kernel may start
            }
            // routed items in (expert, token tile, block) order: tiles[g] = first item of group g
            const int n_act = a.hdr->n_act, blocks = bg[1].blocks;
            int run = 0;
            for (int b0 = 0; b0 < n_act; b0 += 32) {
                const int g = b0 + lane;
                int v = 0;
                if (g < n_act) v = ((a.offsets[a.act[g] + 1] - a.offsets[a.act[g]] + kW4Tok - 1) / kW4Tok) * blocks;
                int incl = v;
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const int y = __shfl_up_sync(0xffffffffu, incl, o);
                    if (lane >= o) incl += y;
                }
                if (g < n_act) tiles[g] = run + incl - v;
                run += __shfl_sync(0xffffffffu, incl, 31);
            }
            if (lane == 0) tiles[n_act] = run;
            __syncwarp();
            const int q1 = (int)((long long)(c_ + 1) * run / G_);
            int g = -1, e = 0, off = 0, cnt = 0, ctile = -1, mt = 0, tok = 0, slot = 0;
            float sc = 0.f;
            for (int q = (int)((long long)c_ * run / G_); q < q1 && ok; ++q) {
                if (g < 0 || q >= tiles[g + 1]) {
                    int lo = g < 0 ? 0 : g + 1, hi = n_act - 1;
                    while (lo < hi) {  // largest g with tiles[g] <= q
                        const int mid = (lo + hi + 1) >> 1;
                        if (tiles[mid] <= q) lo = mid; else hi = mid - 1;
                    }
                    g = lo;
                    e = a.act[g];
                    off = a.offsets[e];
                    cnt = a.offsets[e + 1] - off;
                    ctile = -1;
                }
                const int local = q - tiles[g], tile = local / blocks, h0 = off + tile * kW4Tok;
                if (tile != ctile) {
                    ctile = tile;
                    mt = min(kW4Tok, cnt - tile * kW4Tok);
                    const int pv = a.perm[h0 + (lane < mt ? lane : 0)];
                    tok = pv / a.K;
                    slot = pv - tok * a.K;
                    if (WHICH == kW4Down) sc = a.topw[pv];
                }
                const uint8_t* W = reinterpret_cast<const uint8_t*>(WHICH == kW4Up ? a.gate_up : a.down);
                issue(1, W + (size_t)e * p.matrix_bytes, h0, local - tile * blocks, mt, h0, tok, slot, sc);
            }
        }
        // the end of the items, as one more stage without copies
        if (ok) {
            const int s = it % Ring::kStages;
            ok = __all_sync(0xffffffffu, mbar_wait(&empty[s], (((uint32_t)(it / Ring::kStages)) & 1u) ^ 1u, limit));
            if (ok && lane == 0) {
                for (int j = 0; j < kW4EpiWarps; ++j) metas[(item + j) % Ring::kMetas].group = -1;
                mbar_arrive(&full[s]);
            }
        }
        if (!ok && lane == 0) atomicOr(p.err, ERR_TIMEOUT);
        // every copy issued must land before the CTA's shared memory is released (the end mark's stage
        // was free, so its last copy has landed)
        if (lane == 0)
            for (int k = 0; k < Ring::kStages - (ok ? 1 : 0) && it - 1 - k >= 0; ++k) {
                const int j = it - 1 - k;
                if (!mbar_wait(&full[j % Ring::kStages], ((uint32_t)(j / Ring::kStages)) & 1u, limit))
                    atomicOr(p.err, ERR_TIMEOUT);
            }
    } else if (warp < kWarps) {
        // ---------------- consumers
        if (WHICH != kW4Up) grid_dep_wait();  // the token rows (linear) or the h rows (down)
        if (WHICH == kW4Down) grid_dep_launch();
        uint32_t b[2][1][16];
        float acc[1][4] = {};
        int ckey = 0x7fffffff, cslab = -1, slab = 0, cgroup = -1;
        int it = 0, item = 0;
        for (;; ++it) {
            const int s = it % Ring::kStages;
            bool ok = __all_sync(0xffffffffu, mbar_wait(&full[s], ((uint32_t)(it / Ring::kStages)) & 1u, limit));
            const W4Meta& m = metas[item % Ring::kMetas];
            const int group = ok ? m.group : -1;
            const int rb = item % kW4RedBufs;
            if (group < 0) {
                // the end: passed on to each epilogue warp as one more item
                for (int j = item; j < item + kW4EpiWarps && ok; ++j) {
                    ok = mbar_wait(&rempty[j % kW4RedBufs], (((uint32_t)(j / kW4RedBufs)) & 1u) ^ 1u, limit);
                    if (ok && lane == 0) mbar_arrive(&rfull[j % kW4RedBufs]);
                }
                if (!__all_sync(0xffffffffu, ok) && lane == 0) atomicOr(p.err, ERR_TIMEOUT);
                break;
            }
            const W4Block& bk = bg[group];
            const int wl = bk.wl, sub = warp >> wl, kq = warp & ((1 << wl) - 1);
            const int Rs = bk.nslab == 1 ? bk.R : min(16, bk.R - 16 * slab);
            const int nrec = max(0, min(2, Rs - 2 * kq));
            if (m.key != ckey || slab != cslab || group != cgroup) {
                ckey = m.key;
                cslab = slab;
                cgroup = group;
                const int n = lane >> 2;
                const bool live = n < m.mt;
                const bf16* row;
                if (WHICH == kW4Linear)
                    row = p.x + (size_t)m.tok[n] * p.cols[0];
                else if (WHICH == kW4Up)
                    row = a.x + (size_t)m.tok[n] * a.H;
                else
                    row = a.h + (size_t)(m.row0 + (live ? n : 0)) * a.Imax;
                w4_load_frag(b, row, live, 16 * slab + 2 * kq, nrec, p.cols[group], lane);
            }
            if (sub < min(bk.ns, bk.strips - m.strip0)) {
                const uint32_t rec = smem_u32(stages + (size_t)s * Ring::kStage) + (uint32_t)((sub * Rs + 2 * kq) * kRec);
                if (nrec > 0) w4_mma_record<FMT, G, 1>(rec, b[0], acc, lane);
                if (nrec > 1) w4_mma_record<FMT, G, 1>(rec + kRec, b[1], acc, lane);
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&empty[s]);
            if (++slab == bk.nslab) {
                slab = 0;
                const bool free = __all_sync(0xffffffffu, mbar_wait(&rempty[rb], (((uint32_t)(item / kW4RedBufs)) & 1u) ^ 1u, limit));
                if (!free) {
                    if (lane == 0) atomicOr(p.err, ERR_TIMEOUT);
                    break;
                }
                *reinterpret_cast<float4*>(red + ((rb * kWarps + warp) * 32 + lane) * 4) =
                    make_float4(acc[0][0], acc[0][1], acc[0][2], acc[0][3]);
                acc[0][0] = acc[0][1] = acc[0][2] = acc[0][3] = 0.f;
                __syncwarp();
                if (lane == 0) mbar_arrive(&rfull[rb]);
                ++item;
            }
        }
    } else {
        // ---------------- epilogue: warp e takes items e, e + kW4EpiWarps, ...
        const int g8 = lane >> 2, t2 = 2 * (lane & 3);
        for (int item = warp - kWarps - 1;; item += kW4EpiWarps) {
            const int rb = item % kW4RedBufs;
            const bool ok = __all_sync(0xffffffffu, mbar_wait(&rfull[rb], ((uint32_t)(item / kW4RedBufs)) & 1u, limit));
            const W4Meta& m = metas[item % Ring::kMetas];
            if (!ok || m.group < 0) {
                if (!ok && lane == 0) atomicOr(p.err, ERR_TIMEOUT);
                break;
            }
            const W4Block& bk = bg[m.group];
            const int ns = min(bk.ns, bk.strips - m.strip0), mt = m.mt;
            for (int sub = 0; sub < ns; ++sub) {
                float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
                for (int k = 0; k < (1 << bk.wl); ++k) {
                    const float4 q = *reinterpret_cast<const float4*>(red + ((rb * kWarps + (sub << bk.wl) + k) * 32 + lane) * 4);
                    v.x += q.x; v.y += q.y; v.z += q.z; v.w += q.w;
                }
                const int strip = m.strip0 + sub;
                if (WHICH == kW4Up) {
                    bf16* h = a.h + (size_t)(m.row0 + t2) * a.Imax + strip * 8 + g8;
                    if (t2 < mt) h[0] = __float2bfloat16_rn(silu(v.x) * v.z);
                    if (t2 + 1 < mt) h[a.Imax] = __float2bfloat16_rn(silu(v.y) * v.w);
                } else if (WHICH == kW4Down) {
                    const int row = strip * 16 + g8;
#pragma unroll
                    for (int j = 0; j < 2; ++j)
                        if (t2 + j < mt) {
                            const size_t y = ((size_t)m.tok[t2 + j] * (a.K + 1) + m.slot[t2 + j]) * a.H + row;
                            const float sc = m.sc[t2 + j], y0 = sc * (j ? v.y : v.x), y1 = sc * (j ? v.w : v.z);
                            if (a.gemm) {
                                a.Yb[y] = __float2bfloat16_rn(y0);
                                a.Yb[y + 8] = __float2bfloat16_rn(y1);
                            } else {
                                a.Y[y] = y0;
                                a.Y[y + 8] = y1;
                            }
                        }
                } else {
                    const int N = p.rows[0], row = strip * 16 + g8;
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const int n = row + 8 * i;
                        if (n >= N) continue;
                        const float bias = p.bias ? __bfloat162float(p.bias[n]) : 0.f;
#pragma unroll
                        for (int j = 0; j < 2; ++j)
                            if (t2 + j < mt)
                                p.out[(size_t)m.tok[t2 + j] * N + n] =
                                    __float2bfloat16_rn((i ? (j ? v.w : v.z) : (j ? v.y : v.x)) + bias);
                    }
                }
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&rempty[rb]);
        }
    }
    if (WHICH == kW4Up) grid_dep_launch();
}

template <int WHICH, int FMT, int G>
cudaError_t launch_w4_stream_t(const W4StreamArgs& p, cudaStream_t s) {
    static bool configured[64] = {};
    int dev = 0;
    cudaGetDevice(&dev);
    if (dev < 0 || dev >= 64) dev = 0;
    constexpr int bytes = W4Ring<FMT, G>::kBytes;
    if (!configured[dev]) {
        const cudaError_t e =
            cudaFuncSetAttribute(k_w4_stream<WHICH, FMT, G>, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
        if (e != cudaSuccess) return e;
        configured[dev] = true;
    }
    cudaError_t e;
    const int kernel = WHICH == kW4Linear ? MOE_KERNEL_W4_LINEAR : WHICH == kW4Up ? MOE_KERNEL_GATE_UP : MOE_KERNEL_DOWN;
    MOE_LAUNCH(kernel, s,
               (e = launch_pdl(k_w4_stream<WHICH, FMT, G>, dim3(p.a.num_sms), dim3(kW4Threads), (size_t)bytes, s, p)));
    return e;
}

template <int FMT>
cudaError_t launch_w4_stream_f(int group, int which, const W4StreamArgs& p, cudaStream_t s) {
#define MOE_W4_CASE(W, G) \
    if (which == W && group == G) return launch_w4_stream_t<W, FMT, G>(p, s)
    MOE_W4_CASE(kW4Linear, 32); MOE_W4_CASE(kW4Linear, 64); MOE_W4_CASE(kW4Linear, 128);
    MOE_W4_CASE(kW4Up, 32); MOE_W4_CASE(kW4Up, 64); MOE_W4_CASE(kW4Up, 128);
    MOE_W4_CASE(kW4Down, 32); MOE_W4_CASE(kW4Down, 64); MOE_W4_CASE(kW4Down, 128);
#undef MOE_W4_CASE
    return cudaErrorInvalidValue;
}

// One translation unit per format (compiled in parallel).
cudaError_t launch_w4_stream_int4(int group, int which, const W4StreamArgs& p, cudaStream_t s);
cudaError_t launch_w4_stream_int4_zp(int group, int which, const W4StreamArgs& p, cudaStream_t s);
cudaError_t launch_w4_stream_e2m1(int group, int which, const W4StreamArgs& p, cudaStream_t s);

#endif

}  // namespace moe
