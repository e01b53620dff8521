// w4_stream.cuh -- the weight-streaming products of packed 4-bit weights with few tokens: a linear
// layer, the experts' gate_up and the experts' down projection of the MoE layer.
//
// With few tokens each weight is used a handful of times, so the kernels are bound by reading the
// packed weights once. One persistent CTA per SM: a producer warp walks the CTA's items and copies
// each item's strips (up to 32 records, 34 to 39 KB, one contiguous 1-D TMA bulk copy) into a ring
// of shared-memory stages that keeps ~180 KB of copies in flight; sixteen consumer warps decode
// the codes in registers into the A operand of warp-level bf16 MMAs (16 weight rows by 8 tokens;
// a few strips are too few rows for the 64/128-row tcgen05 MMA, and the decoded weights are in
// registers already), each over its share of a strip's columns with its token rows held in
// registers; two epilogue warps add the shares in a fixed order and write the results, so the
// consumers never wait for one another. Decoding, not the MMAs, is the consumers' work (11 to 14
// instructions for a word of eight codes), so what a stage costs besides it is kept small: one
// 16-byte word tells a consumer warp all that a stage needs as long as the token set stays.
//
// Measured: linear, one token, 24576 x 4096 E2M1 with scales per 32 columns (57 MB) 22 us from HBM, 18 from
// L2; the layer of 64 tokens (221 experts touched, INT4_ZP per 128) gate_up 60 us (235 MB, 3.9 TB/s) and
// down 43 us. Issue slots (55 to 63 % active) and the stages' hand-over bound them together: without any
// decoding gate_up takes 50 us, and a record is 165 (INT4 per 128) to 220 (E2M1 per 32) instructions.
//
// Item: a block of consecutive strips of one matrix by one tile of 8 tokens. A strip of R <= 32
// records is shared by W warps of one or two records each, so 16 / W strips fill a stage (fewer
// when that would leave SMs without items); a strip of more than 32 records takes ceil(R / 32)
// stages, its sums staying in the warps' registers.
#pragma once

#include "launch.h"
#include "w4.cuh"

namespace moe {

enum : int { kW4Linear = 0, kW4Up = 1, kW4Down = 2 };

constexpr int kW4Warps = 16;              // consumer warps
constexpr int kW4StageRecs = 32;          // records of a stage, at most
constexpr int kW4Tok = 8;                 // tokens per item

// How one matrix is cut into items.
struct W4Block {
    int strips, R;    // strips of the matrix, records of a strip
    int wl, rpw;      // log2 of the warps that share a strip, records of each
    int ns, blocks;   // strips of a block, blocks of the matrix
    int nslab;        // stages of a block
};

// want: strips of a block, at most (a power of two).
inline W4Block w4_block(int rows, int cols, int want) {
    W4Block b;
    b.strips = (rows + kW4Strip - 1) / kW4Strip;
    b.R = (cols + kW4Cols - 1) / kW4Cols;
    const int recs = b.R < kW4StageRecs ? b.R : kW4StageRecs;
    b.wl = 0;
    while ((2 << b.wl) < recs) ++b.wl;  // two records a warp
    while (b.wl < 4 && (kW4Warps >> b.wl) > want && (1 << b.wl) < recs) ++b.wl;  // down to one
    b.rpw = (1 << b.wl) >= recs ? 1 : 2;
    b.ns = kW4Warps >> b.wl;
    if (b.ns > want) b.ns = want;
    b.nslab = (b.R + kW4StageRecs - 1) / kW4StageRecs;
    b.blocks = (b.strips + b.ns - 1) / b.ns;
    return b;
}

// One call's operands. Group 0 is the shared expert (or the linear layer's matrix, taken first),
// group 1 the routed experts.
struct W4StreamArgs {
    LayerArgs a;        // up, down: the layer (gate_up, down, sgu, sd point to packed weights)
    const uint8_t* w;   // linear: the packed matrix
    const bf16* x;      // linear: [T, cols]
    const bf16* bias;   // linear: [rows] or NULL
    bf16* out;          // linear: [T, rows]
    int rows[2], cols[2];
    W4Block b0, b1;
    size_t matrix_bytes;  // of one routed matrix
    uint32_t* err;
    uint64_t wait_ns;
    int T;
};

cudaError_t launch_w4_stream(int format, int group, int which, const W4StreamArgs& p, cudaStream_t s);

#ifdef __CUDACC__

constexpr int kW4RedBufs = 4;             // partial-sum buffers
constexpr int kW4EpiWarps = 2;
constexpr int kW4Threads = 32 * (kW4Warps + 1 + kW4EpiWarps);
constexpr int kW4SmemMax = 227 * 1024;

// The token rows of an item (consecutive items mostly share them).
struct __align__(16) W4Set {
    int group;  // 0 shared / linear, 1 routed
    int mt;     // tokens
    int row0;   // up: first h row written; down: first h row read
    int pad;
    int tok[kW4Tok], slot[kW4Tok];
    float sc[kW4Tok];
};

// A stage, as the producer writes it into a ring of entries that the consumers read (an item's last stage
// into a second ring, by items, for the epilogue):
//   x  number of the token rows and column range: a new one means new rows to load
//   y  strips | records << 8 | (last stage of its item) << 16 | column range << 17; 0: no more items
//   z  first strip of the block          w  the item's W4Set
template <int FMT, int G>
struct W4Ring {
    static constexpr int kStage = kW4StageRecs * W4Rec<FMT, G>::kBytes;
    static constexpr int kRed = kW4RedBufs * kW4Warps * 128 * 4;
    static constexpr int kEnt = 16;  // entries and sets: more than the items between copy and epilogue
    static constexpr int kMaxStages = 6;
    static constexpr int oRed = 0, oEnt = oRed + kRed, oItm = oEnt + kEnt * 16, oSet = oItm + kEnt * 16, oBar = oSet + kEnt * (int)sizeof(W4Set),
                         oTab = oBar + 8 * (2 * kMaxStages + 2 * kW4RedBufs), kFixed = 128 + oTab + 260 * 10;
    static constexpr int kFit = (kW4SmemMax - kFixed) / kStage;
    static constexpr int kStages = kFit < kMaxStages ? kFit : kMaxStages;
    static_assert(kStage % 128 == 0 && kStages >= 3 && kStages + kW4RedBufs + 2 <= kEnt && oBar % 8 == 0, "ring");
    static constexpr int kBytes = kFixed + kStages * kStage;
};

// B operands of one record from a lane's token row: elements 32 c + 8 t .. + 7 from column k0, zero
// past the matrix's columns (the packed weights there have scale 0, but the row's memory may hold
// anything) and for the tile's missing tokens. L2 loads (an earlier kernel wrote the rows).
__device__ __forceinline__ void w4_load_tokens(uint32_t (&b)[16], const bf16* row, bool live, int k0, int cols, int lane) {
#pragma unroll
    for (int c = 0; c < 4; ++c) {
        const int k = k0 + 32 * c + 8 * (lane & 3);
        uint4 v = make_uint4(0u, 0u, 0u, 0u);
        if (live && k < cols) v = __ldcg(reinterpret_cast<const uint4*>(row + k));
        b[4 * c] = v.x; b[4 * c + 1] = v.y; b[4 * c + 2] = v.z; b[4 * c + 3] = v.w;
    }
}

// A cursor over a ring of N barriers: the slot, and the parity of its current round.
template <int N>
struct W4Cursor {
    uint32_t s = 0, ph = 0;
    __device__ __forceinline__ void next() {
        if (++s == (uint32_t)N) {
            s = 0;
            ph ^= 1u;
        }
    }
};

// The group of item q: the largest g with tiles[g] <= q.
__device__ __forceinline__ int w4_find(const int* tiles, int n, int q) {
    int lo = 0, hi = n - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (tiles[mid] <= q) lo = mid; else hi = mid - 1;
    }
    return lo;
}

__device__ __forceinline__ bool w4_wait(uint64_t* bar, uint32_t parity, uint64_t limit) {
    return __all_sync(0xffffffffu, mbar_wait(bar, parity, limit));
}

// As w4_wait, on a shared-window address.
__device__ __forceinline__ bool w4_wait32(uint32_t bar, uint32_t parity, uint64_t limit) {
    if (__all_sync(0xffffffffu, mbar_try_wait32(bar, parity))) return true;
    const uint64_t t0 = global_ns();
    for (;;) {
        if (__all_sync(0xffffffffu, mbar_try_wait32(bar, parity))) return true;
        if (__any_sync(0xffffffffu, global_ns() - t0 > limit)) return false;
    }
}

template <int WHICH, int FMT, int G>
__global__ void __launch_bounds__(kW4Threads, 1) k_w4_stream(const __grid_constant__ W4StreamArgs p) {
    using Ring = W4Ring<FMT, G>;
    constexpr int kRec = W4Rec<FMT, G>::kBytes;
    extern __shared__ uint8_t smem_raw[];
    // shared-window addresses throughout: arithmetic on generic pointers costs several instructions a
    // use, and a stage's bookkeeping is on every warp's critical path
    uint8_t* base = smem_raw + (((smem_u32(smem_raw) + 127u) & ~127u) - smem_u32(smem_raw));
    const uint32_t st0 = smem_u32(base), x0 = st0 + Ring::kStages * Ring::kStage;
    const uint32_t red0 = x0 + Ring::oRed, ent0 = x0 + Ring::oEnt, itm0 = x0 + Ring::oItm, full0 = x0 + Ring::oBar, empty0 = full0 + 8 * Ring::kMaxStages,
                   rfull0 = empty0 + 8 * Ring::kMaxStages, rempty0 = rfull0 + 8 * kW4RedBufs;
    uint8_t* xp = base + Ring::kStages * Ring::kStage;
    W4Set* sets = reinterpret_cast<W4Set*>(xp + Ring::oSet);
    const LayerArgs& a = p.a;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint64_t limit = p.wait_ns;
    if (threadIdx.x == 0) {
        uint64_t* bar = reinterpret_cast<uint64_t*>(xp + Ring::oBar);
        for (int s = 0; s < Ring::kMaxStages; ++s) {
            mbar_init(&bar[s], 1);
            mbar_init(&bar[Ring::kMaxStages + s], kW4Warps);
        }
        for (int s = 0; s < kW4RedBufs; ++s) {
            mbar_init(&bar[2 * Ring::kMaxStages + s], kW4Warps);
            mbar_init(&bar[2 * Ring::kMaxStages + kW4RedBufs + s], 1);
        }
        fence_mbar_init();
    }
    __syncthreads();

    if (warp == kW4Warps) {
        // ---------------- producer
        const int G_ = gridDim.x, c_ = blockIdx.x;
        W4Cursor<Ring::kStages> cur;
        int it = 0, item = 0, key = 0, nset = -1;
        bool ok = true;
        // one item: for each of its stages the copy, then (fresh: its token rows are not those of the item
        // before) the metadata, which may still have to come from memory, then the arrival that lets the
        // consumers in. rows(set): the lane's token, slot and scale.
        auto issue = [&](const W4Block& b, const uint8_t* W, int blk, bool fresh, auto rows) {
            const int strip0 = blk * b.ns, ns = min(b.ns, b.strips - strip0);
            for (int slab = 0; slab < b.nslab && ok; ++slab) {
                ok = w4_wait32(empty0 + 8u * cur.s, cur.ph ^ 1u, limit);
                if (!ok) break;
                const int recs = min(kW4StageRecs, b.R - kW4StageRecs * slab);
                const uint32_t bytes = (uint32_t)((b.nslab == 1 ? ns * recs : recs) * kRec), bar = full0 + 8u * cur.s;
                if (lane == 0) {
                    mbar_expect_tx32(bar, bytes);
                    bulk_load32(st0 + cur.s * (uint32_t)Ring::kStage, W + ((size_t)strip0 * b.R + kW4StageRecs * slab) * kRec, bytes, bar);
                }
                if (slab == 0 && fresh) {
                    ++nset;
                    rows(sets[nset & (Ring::kEnt - 1)]);
                    __syncwarp();
                }
                if (fresh || slab > 0) ++key;
                if (lane == 0) {
                    const uint32_t ent[4] = {(uint32_t)key,
                                             (uint32_t)(ns | recs << 8 | (slab == b.nslab - 1 ? 1 << 16 : 0) | slab << 17),
                                             (uint32_t)strip0, (uint32_t)(nset & (Ring::kEnt - 1))};
                    sts128(ent0 + 16u * (uint32_t)(it & (Ring::kEnt - 1)), ent);
                    if (slab == b.nslab - 1) sts128(itm0 + 16u * (uint32_t)(item & (Ring::kEnt - 1)), ent);
                    mbar_arrive32(bar);
                }
                cur.next();
                ++it;
            }
            ++item;
            if (b.nslab > 1) ++key;  // the next item starts at the first column range again
        };
        const int n0 = p.b0.blocks * ((p.T + kW4Tok - 1) / kW4Tok);  // group 0: (token tile, block) order
        const int i0 = (int)((long long)c_ * n0 / G_), i1 = (int)((long long)(c_ + 1) * n0 / G_);
        if (WHICH == kW4Linear) {
            grid_dep_wait();
            grid_dep_launch();
        }
        {
            const uint8_t* W = WHICH == kW4Linear ? p.w : reinterpret_cast<const uint8_t*>(WHICH == kW4Up ? a.sgu : a.sd);
            int tile = i0 / p.b0.blocks, blk = i0 - tile * p.b0.blocks;
            bool fresh = true;
            for (int i = i0; i < i1 && ok; ++i) {
                const int t0 = tile * kW4Tok, mt = min(kW4Tok, p.T - t0);
                issue(p.b0, W, blk, fresh, [&](W4Set& m) {
                    if (lane < kW4Tok) {
                        const int tok = t0 + (lane < mt ? lane : 0);
                        m.tok[lane] = tok;
                        m.slot[lane] = a.K;
                        m.sc[lane] = WHICH == kW4Down ? a.sgate[tok] : 0.f;
                    }
                    if (lane == 0) *reinterpret_cast<int4*>(&m) = make_int4(0, mt, (WHICH == kW4Linear ? 0 : (int)a.P) + t0, 0);
                });
                fresh = false;
                if (++blk == p.b0.blocks) {
                    blk = 0;
                    ++tile;
                    fresh = true;
                }
            }
        }
        if (WHICH != kW4Linear) {
            if (WHICH == kW4Up) {
                grid_dep_wait();
                grid_dep_launch();  // the routing is complete: the down kernel may start
            }
            // routed items in (expert, token tile, block) order: tiles[g] = first item of group g. All the
            // experts and their counts are read at once (their latencies would come one after another).
            int* tiles = reinterpret_cast<int*>(xp + Ring::oTab);
            uint32_t* groups = reinterpret_cast<uint32_t*>(tiles + 260);  // expert << 16 | first h row
            uint16_t* counts = reinterpret_cast<uint16_t*>(groups + 260);
            const int n_act = a.hdr->n_act, blocks = p.b1.blocks;
            int e8[8], o8[8], c8[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) e8[j] = 32 * j + lane < a.E ? a.act[32 * j + lane] : 0;  // (not waiting for n_act)
#pragma unroll
            for (int j = 0; j < 8; ++j) e8[j] = 32 * j + lane < n_act ? e8[j] : 0;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                o8[j] = a.offsets[e8[j]];
                c8[j] = a.offsets[e8[j] + 1];
            }
            int run = 0;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const int g = 32 * j + lane;
                c8[j] -= o8[j];
                const int v = g < n_act ? ((c8[j] + kW4Tok - 1) / kW4Tok) * blocks : 0;
                int incl = v;
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const int y = __shfl_up_sync(0xffffffffu, incl, o);
                    if (lane >= o) incl += y;
                }
                if (g < n_act) {
                    tiles[g] = run + incl - v;
                    groups[g] = (uint32_t)e8[j] << 16 | (uint32_t)o8[j];  // (fewer than 2^16 pairs below 256 tokens)
                    counts[g] = (uint16_t)c8[j];
                }
                run += __shfl_sync(0xffffffffu, incl, 31);
            }
            __syncwarp();
            const int q0 = (int)((long long)c_ * run / G_), q1 = (int)((long long)(c_ + 1) * run / G_);
            if (q0 < q1 && ok) {
                int g = w4_find(tiles, n_act, q0), tile = (q0 - tiles[g]) / blocks, blk = q0 - tiles[g] - tile * blocks;
                uint32_t eo = groups[g];
                int cnt = counts[g];
                bool fresh = true;
                const uint8_t* W0 = reinterpret_cast<const uint8_t*>(WHICH == kW4Up ? a.gate_up : a.down);
                for (int q = q0; q < q1 && ok; ++q) {
                    issue(p.b1, W0 + (size_t)(eo >> 16) * p.matrix_bytes, blk, fresh, [&](W4Set& m) {
                        const int h0 = (int)(eo & 0xffffu) + tile * kW4Tok, mt = min(kW4Tok, cnt - tile * kW4Tok);
                        if (lane < kW4Tok) {
                            const int pv = a.perm[h0 + (lane < mt ? lane : 0)], tok = pv / a.K;
                            m.tok[lane] = tok;
                            m.slot[lane] = pv - tok * a.K;
                            m.sc[lane] = WHICH == kW4Down ? a.topw[pv] : 0.f;
                        }
                        if (lane == 0) *reinterpret_cast<int4*>(&m) = make_int4(1, mt, h0, 0);
                    });
                    fresh = false;
                    if (++blk == blocks) {
                        blk = 0;
                        ++tile;
                        fresh = true;
                        if (tile * kW4Tok >= cnt && q + 1 < q1) {
                            ++g;
                            tile = 0;
                            eo = groups[g];
                            cnt = counts[g];
                        }
                    }
                }
            }
        }
        // the end of the items, as one more stage without copies
        const int issued = it;
        if (ok) {
            ok = w4_wait32(empty0 + 8u * cur.s, cur.ph ^ 1u, limit);
            if (ok && lane == 0) {
                const uint32_t ent[4] = {(uint32_t)key, 0u, 0u, 0u};
                sts128(ent0 + 16u * (uint32_t)(it & (Ring::kEnt - 1)), ent);
                for (int j = 0; j < kW4EpiWarps; ++j) sts128(itm0 + 16u * (uint32_t)((item + j) & (Ring::kEnt - 1)), ent);
                mbar_arrive32(full0 + 8u * cur.s);
            }
        }
        if (!ok && lane == 0) atomicOr(p.err, ERR_TIMEOUT);
        // every copy issued must land before the CTA's shared memory is released (the end mark's stage
        // was free, so its last copy has landed)
        uint64_t* bar = reinterpret_cast<uint64_t*>(xp + Ring::oBar);
        if (lane == 0)
            for (int k = 0; k < Ring::kStages - (ok ? 1 : 0) && issued - 1 - k >= 0; ++k) {
                const int j = issued - 1 - k;
                if (!mbar_wait(&bar[j % Ring::kStages], ((uint32_t)(j / Ring::kStages)) & 1u, limit)) atomicOr(p.err, ERR_TIMEOUT);
            }
    } else if (warp < kW4Warps) {
        // ---------------- consumers
        if (WHICH != kW4Up) grid_dep_wait();  // the token rows (linear) or the h rows (down)
        if (WHICH == kW4Down) grid_dep_launch();
        uint32_t b[2][16];
        float acc[4] = {};
        int ckey = 0, sub = 0, nrec = 0;
        uint32_t at = 0, ent = 0;  // this warp's records within a stage; the entry
        W4Cursor<Ring::kStages> cur;
        W4Cursor<kW4RedBufs> rcur;
        const uint32_t red = red0 + (uint32_t)(warp * 512 + lane * 16);
        bool ok;
        for (;;) {
            ok = w4_wait32(full0 + 8u * cur.s, cur.ph, limit);
            if (!ok) break;
            const uint4 e = lds128_smem(ent0 + ent);
            ent = (ent + 16u) & (16u * Ring::kEnt - 1u);
            const int info = (int)e.y;
            if (info == 0) break;
            if ((int)e.x != ckey) {
                ckey = (int)e.x;
                const W4Set& m = sets[e.w];
                const bool routed = m.group != 0;
                const int wl = routed ? p.b1.wl : p.b0.wl, rpw = routed ? p.b1.rpw : p.b0.rpw;
                const int recs = (info >> 8) & 0xff, kq = warp & ((1 << wl) - 1);
                sub = warp >> wl;
                nrec = max(0, min(rpw, recs - rpw * kq));
                at = (uint32_t)((sub * recs + rpw * kq) * kRec);
                if (nrec == 0) sub = kW4StageRecs;  // no share of any stage with these rows
                const int n = lane >> 2;
                const bool live = n < m.mt;
                const bf16* row;
                if (WHICH == kW4Linear)
                    row = p.x + (size_t)m.tok[n] * p.cols[0];
                else if (WHICH == kW4Up)
                    row = a.x + (size_t)m.tok[n] * a.H;
                else
                    row = a.h + (size_t)(m.row0 + (live ? n : 0)) * a.Imax;
                const int cols = routed ? p.cols[1] : p.cols[0];
                const int k0 = ((info >> 17) * kW4StageRecs + rpw * kq) * kW4Cols;
                w4_load_tokens(b[0], row, live && nrec > 0, k0, cols, lane);
                w4_load_tokens(b[1], row, live && nrec > 1, k0 + kW4Cols, cols, lane);
            }
            if (sub < (info & 0xff)) {
                const uint32_t rec = st0 + cur.s * (uint32_t)Ring::kStage + at;
                w4_records<FMT, G>(rec, nrec, b, acc, lane);
            }
            __syncwarp();
            if (lane == 0) mbar_arrive32(empty0 + 8u * cur.s);
            cur.next();
            if (info & (1 << 16)) {
                ok = w4_wait32(rempty0 + 8u * rcur.s, rcur.ph ^ 1u, limit);
                if (!ok) break;
                const uint32_t v[4] = {__float_as_uint(acc[0]), __float_as_uint(acc[1]), __float_as_uint(acc[2]),
                                       __float_as_uint(acc[3])};
                sts128(red + rcur.s * (uint32_t)(kW4Warps * 512), v);
                acc[0] = acc[1] = acc[2] = acc[3] = 0.f;
                __syncwarp();
                if (lane == 0) mbar_arrive32(rfull0 + 8u * rcur.s);
                rcur.next();
            }
        }
        // the end: passed on to each epilogue warp as one more item
        for (int j = 0; j < kW4EpiWarps && ok; ++j) {
            ok = w4_wait32(rempty0 + 8u * rcur.s, rcur.ph ^ 1u, limit);
            if (ok && lane == 0) mbar_arrive32(rfull0 + 8u * rcur.s);
            rcur.next();
        }
        if (!ok && lane == 0) atomicOr(p.err, ERR_TIMEOUT);
    } else {
        // ---------------- epilogue: warp e takes items e, e + kW4EpiWarps, ...
        const int g8 = lane >> 2, t2 = 2 * (lane & 3);
        int item = warp - kW4Warps - 1, cset = -1, wl = 0, row0 = 0;
        bool live0 = false, live1 = false;  // the lane's two tokens
        size_t o0 = 0, o1 = 0;              // their output rows
        float sc0 = 0.f, sc1 = 0.f;
        for (;; item += kW4EpiWarps) {
            const uint32_t rb = (uint32_t)item % kW4RedBufs;
            const bool ok = w4_wait32(rfull0 + 8u * rb, ((uint32_t)item / kW4RedBufs) & 1u, limit);
            const uint4 e = lds128_smem(itm0 + 16u * ((uint32_t)item & (Ring::kEnt - 1)));
            if (!ok || e.y == 0) {
                if (!ok && lane == 0) atomicOr(p.err, ERR_TIMEOUT);
                break;
            }
            const int ns = (int)(e.y & 0xffu), strip0 = (int)e.z;
            if ((int)e.w != cset) {
                cset = (int)e.w;
                const W4Set& m = sets[cset];
                wl = m.group ? p.b1.wl : p.b0.wl;
                row0 = m.row0;
                live0 = t2 < m.mt;
                live1 = t2 + 1 < m.mt;
                const int k0 = m.tok[t2], k1 = m.tok[t2 + 1];
                if (WHICH == kW4Up) {
                    o0 = (size_t)(row0 + t2) * a.Imax;
                    o1 = o0 + a.Imax;
                } else if (WHICH == kW4Down) {
                    o0 = ((size_t)k0 * (a.K + 1) + m.slot[t2]) * a.H;
                    o1 = ((size_t)k1 * (a.K + 1) + m.slot[t2 + 1]) * a.H;
                    sc0 = m.sc[t2] * W4Fold<FMT>::kUnfold;
                    sc1 = m.sc[t2 + 1] * W4Fold<FMT>::kUnfold;
                } else {
                    o0 = (size_t)k0 * p.rows[0];
                    o1 = (size_t)k1 * p.rows[0];
                }
            }
            const uint32_t r0 = red0 + rb * (uint32_t)(kW4Warps * 512) + (uint32_t)(lane * 16);
            for (int sub = 0; sub < ns; ++sub) {
                float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
                const uint32_t rs = r0 + (uint32_t)((sub << wl) * 512);
                for (int k = 0; k < (1 << wl); k += 2) {  // (at least two warps share a strip, or one)
                    const uint4 q = lds128_smem(rs + (uint32_t)(k * 512));
                    uint4 r = make_uint4(0u, 0u, 0u, 0u);
                    if (wl > 0) r = lds128_smem(rs + (uint32_t)(k * 512 + 512));
                    v.x += __uint_as_float(q.x); v.y += __uint_as_float(q.y);
                    v.z += __uint_as_float(q.z); v.w += __uint_as_float(q.w);
                    v.x += __uint_as_float(r.x); v.y += __uint_as_float(r.y);
                    v.z += __uint_as_float(r.z); v.w += __uint_as_float(r.w);
                }
                if (WHICH != kW4Down) {
                    v.x *= W4Fold<FMT>::kUnfold; v.y *= W4Fold<FMT>::kUnfold;
                    v.z *= W4Fold<FMT>::kUnfold; v.w *= W4Fold<FMT>::kUnfold;
                }
                const int strip = strip0 + sub;
                if (WHICH == kW4Up) {
                    const int f = strip * 8 + g8;
                    if (live0) a.h[o0 + f] = __float2bfloat16_rn(silu(v.x) * v.z);
                    if (live1) a.h[o1 + f] = __float2bfloat16_rn(silu(v.y) * v.w);
                } else if (WHICH == kW4Down) {
                    const int row = strip * 16 + g8;
                    if (live0) {
                        a.Y[o0 + row] = sc0 * v.x;
                        a.Y[o0 + row + 8] = sc0 * v.z;
                    }
                    if (live1) {
                        a.Y[o1 + row] = sc1 * v.y;
                        a.Y[o1 + row + 8] = sc1 * v.w;
                    }
                } else {
                    const int N = p.rows[0], n0 = strip * 16 + g8, n1 = n0 + 8;
                    const float bias0 = p.bias && n0 < N ? __bfloat162float(p.bias[n0]) : 0.f;
                    const float bias1 = p.bias && n1 < N ? __bfloat162float(p.bias[n1]) : 0.f;
                    if (live0 && n0 < N) p.out[o0 + n0] = __float2bfloat16_rn(v.x + bias0);
                    if (live1 && n0 < N) p.out[o1 + n0] = __float2bfloat16_rn(v.y + bias0);
                    if (live0 && n1 < N) p.out[o0 + n1] = __float2bfloat16_rn(v.z + bias1);
                    if (live1 && n1 < N) p.out[o1 + n1] = __float2bfloat16_rn(v.w + bias1);
                }
            }
            __syncwarp();
            if (lane == 0) mbar_arrive32(rempty0 + 8u * rb);
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
