// w4_one.cuh -- the whole MoE layer on packed 4-bit weights for one token, one persistent kernel.
//
// A decode step reads 17 MB of packed weights at the pages' shape: 2.5 us at the measured HBM rate.
// What a chain of kernels spends on launches, drained pipelines and cold starts is many times that, so
// the kernel is built for latency: one CTA per SM, every weight on its way as early as it is known,
// and as few steps as the data dependences need (scores -> routing -> h -> output). G CTAs, CTA c:
//   scores   router rows c, c + G, ... (row E is the shared gate), a warp a row;
//   routing  one warp of every CTA ranks all the scores itself;
//   gate_up  a contiguous run of strips of the shared expert (copied before the routing is known) and
//            of the routed experts; a strip's records are spread over sixteen warps, which only leave sums
//            behind; when all strips are done, a warp a strip adds them and publishes its eight h values;
//   down     output strips c, c + G, ... of the shared and every routed expert: the h rows are gathered
//            into shared memory (a warp a row), 16 / W experts' strips fill a stage, W warps to each;
//            then residual, gated shared expert and slots 0 .. K-1 are added in that order.
// Measured at the pages' shape (INT4 per 32): 14.4 to 14.6 us a layer back to back, against 28 us for the
// chain of routing, gate_up, down and combine. What bounds it is the chain of dependent steps: scores, their
// exchange, routing, the first routed weights, the h exchange, output; the weights alone are 2.5 us.
// The products are warp MMAs with one live column of eight: the weights are decoded to the A operand
// anyway, and an MMA step replaces 64 multiply-adds a lane would do on unpacked values.
// Exchanges carry a tag of the call instead of a flag or fence: 64-bit words (32-bit tag, fp32 score)
// and (32-bit tag, two bf16 h values), published with atomic exchanges at L2 and polled until all
// words needed carry this call's tag. The tag is the call's number times an odd constant, so that
// neither an earlier call's words nor other data left in the workspace is taken for this call's.
// The CTAs wait on one another, so all must be resident (one CTA per SM, checked; each waits for the
// previous grid before its first wait on a peer). Every wait is bounded: a timeout sets
// MOE_ERR_TIMEOUT and the kernel runs to its end with in-range indices.
#pragma once

#include "w4_stream.cuh"

namespace moe {

struct W4OneArgs {
    LayerArgs a;                // gate_up .. sd point to packed weights
    uint64_t* dh;               // [K + 1, Imax / 2] tagged h pairs (row K: the shared expert)
    size_t gu_bytes, dn_bytes;  // of one expert's packed matrices
    int R;                      // records of a gate_up strip
    int dwl, drpw, dR;          // down: log2 of the warps of a strip, records of each, records of the longer strip
};

constexpr int kOneMaxK = 8;
constexpr int kOneMaxUp = 24;       // gate_up strips of a CTA, at most
constexpr int kOneMaxInner = 2048;  // longest h row

// Gate_up strips that one CTA of `ctas` takes, at most.
inline int w4_one_strips(const LayerArgs& a, int ctas) {
    return (a.Is / 8 + ctas - 1) / ctas + (a.K * (a.I / 8) + ctas - 1) / ctas;
}

#ifdef __CUDACC__

constexpr int kOneThreads = 32 * (kW4Warps + 2);  // consumers, producer, router

struct W4OneRoute {
    int ids[kOneMaxK];
    float w[kOneMaxK];
    float sg;
};

template <int FMT, int G>
struct W4OneRing {
    static constexpr int kStage = kW4StageRecs * W4Rec<FMT, G>::kBytes;
    static constexpr int kPart = kOneMaxUp * kW4Warps * 16 * 4;        // [strip][warp][16]
    static constexpr int kYs = (kOneMaxK + 1) * kW4Warps * 16 * 4;     // [group][W][16], at most
    static constexpr int kFixed = 128 + kPart + kYs + 256 + 256;
};
// Shared memory: stages, h rows [K + 1][Imax] bf16 (64 bytes apart modulo 128), the token row, sums.
constexpr int w4_one_rows(int K, int Imax, int H) { return (K + 1) * (2 * Imax + 64) + 2 * H; }
template <int FMT, int G>
inline int w4_one_stages(int K, int Imax, int H) {
    static_assert((kW4SmemMax - W4OneRing<FMT, G>::kFixed - w4_one_rows(kOneMaxK, kOneMaxInner, kW4StageRecs * kW4Cols)) / W4OneRing<FMT, G>::kStage >= 3,
                  "stages beside the largest rows");
    const int n = (kW4SmemMax - W4OneRing<FMT, G>::kFixed - w4_one_rows(K, Imax, H)) / W4OneRing<FMT, G>::kStage;
    return n < 6 ? n : 6;
}

__device__ __forceinline__ void w4o_publish(uint64_t* p, uint64_t v) {
    uint64_t old;
    asm volatile("atom.exch.relaxed.gpu.global.b64 %0, [%1], %2;" : "=l"(old) : "l"(p), "l"(v) : "memory");
}
__device__ __forceinline__ uint64_t w4o_peek(const uint64_t* p) {
    uint64_t v;
    asm volatile("ld.relaxed.gpu.global.u64 %0, [%1];" : "=l"(v) : "l"(p) : "memory");
    return v;
}
__device__ __forceinline__ void w4o_peek2(const uint64_t* p, uint64_t& a, uint64_t& b) {
    asm volatile("ld.relaxed.gpu.global.v2.u64 {%0, %1}, [%2];" : "=l"(a), "=l"(b) : "l"(p) : "memory");
}

// Routing of the token by one warp from its E + 1 tagged scores (as k_decode_fused: experts by score,
// equal scores to the lower index, weights the softmax over the kept scores). Arrives on `routed` once
// the experts are known; weights and gate follow.
__device__ inline void w4o_route(const LayerArgs& a, W4OneRoute& rt, uint32_t tag, int lane, uint64_t* routed) {
    uint32_t val[9], need = 0;
#pragma unroll
    for (int j = 0; j < 9; ++j) {
        val[j] = 0u;  // a score of 0 if the wait times out
        if ((j < 8 && lane + 32 * j < a.E) || (j == 8 && lane == 0)) need |= 1u << j;
    }
    const uint64_t t0 = global_ns();
    bool timed_out = false;
    while (__any_sync(0xffffffffu, need != 0)) {
        uint64_t w[9];
#pragma unroll
        for (int j = 0; j < 9; ++j) w[j] = ((need >> j) & 1u) ? w4o_peek(a.dlog + (j < 8 ? lane + 32 * j : a.E)) : 0ull;
#pragma unroll
        for (int j = 0; j < 9; ++j)
            if (((need >> j) & 1u) && (uint32_t)(w[j] >> 32) == tag) {
                val[j] = (uint32_t)w[j];
                need &= ~(1u << j);
            }
        if (__any_sync(0xffffffffu, global_ns() - t0 > a.wait_ns)) {
            timed_out = __any_sync(0xffffffffu, need != 0);
            break;
        }
    }
    bool bad = false;
    uint32_t key[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        key[j] = 0u;
        if (lane + 32 * j < a.E) {
            float v = router_score(__uint_as_float(val[j]), a.flags);
            if (!isfinite(v)) {
                bad = true;
                v = -INFINITY;
            }
            key[j] = score_key(v);
        }
    }
    float v0, myv;
    int mye;
    warp_topk(key, a.K, lane, v0, myv, mye);
    if (lane < a.K) rt.ids[lane] = mye;
    __syncwarp();
    if (lane == 0) mbar_arrive(routed);
    const float ex = lane < a.K ? expf(myv - v0) : 0.f;
    const float s = warp_sum(ex);
    if (lane < a.K) rt.w[lane] = ex / s;
    if (lane == 0) {
        const float z = router_score(__uint_as_float(val[8]), a.flags);
        if (!isfinite(z)) bad = true;
        rt.sg = 1.0f / (1.0f + expf(-z));
        if (timed_out) atomicOr(&a.hdr->err, ERR_TIMEOUT);
    }
    if (__any_sync(0xffffffffu, bad) && lane == 0) atomicOr(&a.hdr->err, ERR_NONFINITE_SCORE);
    __syncwarp();
}

// Between gate_up and down: a warp a gate_up strip adds its sums and publishes its h values, then the h
// rows of all experts (slots, then the shared one) are gathered into shared memory, a warp a row.
template <int FMT>
__device__ __forceinline__ void w4o_exchange(const W4OneArgs& p, const W4OneRoute& rt, const float* part, uint8_t* hs, int hpitch,
                                          uint32_t tag, int n_sh, int n_up, int s0, int q0, uint32_t* err) {
    const LayerArgs& a = p.a;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, K = a.K, sr = a.I / 8;
    asm volatile("bar.sync 1, %0;" ::"n"(32 * kW4Warps) : "memory");
    // gate (lanes 0 .. 7) and up (8 .. 15) sums in warp order
    for (int i = warp; i < n_up; i += kW4Warps) {
        const bool sh = i < n_sh;
        const int q = sh ? 0 : q0 + i - n_sh, slot = sh ? K : q / sr, strip = sh ? s0 + i : q - slot * sr;
        float v = 0.f;
        if (lane < 16)
#pragma unroll
            for (int w = 0; w < kW4Warps; ++w) v += part[(i * kW4Warps + w) * 16 + lane];
        v *= W4Fold<FMT>::kUnfold;
        const float u = __shfl_down_sync(0xffffffffu, v, 8);
        const uint32_t h = __bfloat16_as_ushort(__float2bfloat16_rn(silu(v) * u));
        const uint32_t h1 = __shfl_down_sync(0xffffffffu, h, 1);
        if (lane < 8 && (lane & 1) == 0)
            w4o_publish(p.dh + (size_t)slot * (a.Imax / 2) + strip * 4 + lane / 2, ((uint64_t)tag << 32) | h1 << 16 | h);
    }
    bool ok = true;
    for (int g = warp; g <= K; g += kW4Warps) {
        const int pairs = (g == K ? a.Is : a.I) / 2;  // a multiple of 32
        const uint64_t* src = p.dh + (size_t)g * (a.Imax / 2);
        uint8_t* dst = hs + g * hpitch;
        for (int c = 0; c < pairs; c += 256) {  // four 16-byte words a lane in flight
            uint64_t v[4][2];
            uint32_t need = 0;
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (c + 64 * i + 2 * lane < pairs) need |= 1u << i;
            const uint64_t t0 = global_ns();
            while (__any_sync(0xffffffffu, need != 0)) {
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if ((need >> i) & 1u) w4o_peek2(src + c + 64 * i + 2 * lane, v[i][0], v[i][1]);
                const bool late = !ok || global_ns() - t0 > a.wait_ns;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const bool fresh = (uint32_t)(v[i][0] >> 32) == tag && (uint32_t)(v[i][1] >> 32) == tag;
                    if (((need >> i) & 1u) && (late || fresh)) {
                        if (!fresh) ok = false;
                        *reinterpret_cast<uint2*>(dst + 4 * (c + 64 * i + 2 * lane)) = make_uint2((uint32_t)v[i][0], (uint32_t)v[i][1]);
                        need &= ~(1u << i);
                    }
                }
            }
            ok = __all_sync(0xffffffffu, ok);
        }
        // tap 0: rows in dispatch order, the shared expert's last, by the last CTA: its share always holds a routed
        // strip, so its consumers have waited for weights that its producer asked for behind `routed`, and the ids are
        // complete. (Any other CTA has none where K * I / 8 is below the CTAs. Ordered by a wait for `routed` or by
        // the barrier below instead, in CTA 0, the layer took 16.2 and 16.4 us against 14.5.)
        if (blockIdx.x == gridDim.x - 1) {
            int pos = 0;
            for (int j = 0; j < K; ++j) pos += g < K && rt.ids[j] < rt.ids[g];
            __syncwarp();
            for (int c = lane; c < pairs; c += 32)
                reinterpret_cast<uint32_t*>(a.h + (size_t)(g == K ? K : pos) * a.Imax)[c] = *reinterpret_cast<uint32_t*>(dst + 4 * c);
        }
    }
    if (!ok && lane == 0) atomicOr(err, ERR_TIMEOUT);
    asm volatile("bar.sync 2, %0;" ::"n"(32 * (kW4Warps + 1)) : "memory");  // h rows in place; the router's weights too
}

template <int FMT, int G>
__global__ void __launch_bounds__(kOneThreads, 1) k_w4_one(const __grid_constant__ W4OneArgs p, int nst) {
    using Ring = W4OneRing<FMT, G>;
    constexpr int kRec = W4Rec<FMT, G>::kBytes;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* base = smem_raw + (((smem_u32(smem_raw) + 127u) & ~127u) - smem_u32(smem_raw));
    const LayerArgs& a = p.a;
    const int K = a.K, hpitch = 2 * a.Imax + 64;
    uint8_t* stages = base;
    uint8_t* hs = stages + nst * Ring::kStage;      // h rows
    uint8_t* xs = hs + (K + 1) * hpitch;            // the token row
    float* part = reinterpret_cast<float*>(xs + 2 * a.H);
    float* ys = part + kOneMaxUp * kW4Warps * 16;
    W4OneRoute& rt = *reinterpret_cast<W4OneRoute*>(ys + (kOneMaxK + 1) * kW4Warps * 16);
    uint64_t* full = reinterpret_cast<uint64_t*>(reinterpret_cast<uint8_t*>(&rt) + 256);
    uint64_t* empty = full + 6;
    uint64_t* routed = empty + 6;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int GD = gridDim.x, cta = blockIdx.x;
    const uint64_t limit = a.wait_ns;
    uint32_t* err = &a.hdr->err;
    // the kernel parameters, a word of each 64-byte line, fetched together: in the order of use their
    // constant-cache misses would come one after another
    {
        uint32_t v = 0;
        if (lane < (int)(sizeof(W4OneArgs) / 64)) v = reinterpret_cast<const uint32_t*>(&p)[16 * lane];
        asm volatile("" ::"r"(v));
    }
    if (threadIdx.x == 0) {
        for (int s = 0; s < nst; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], kW4Warps);
        }
        mbar_init(routed, 1);
        fence_mbar_init();
    }
    // every index read from the routing is in range even when a wait runs out before it is complete (a routing
    // whose own wait ran out ranks scores of 0 in the missing places)
    if (threadIdx.x < sizeof(W4OneRoute) / 4) reinterpret_cast<int*>(&rt)[threadIdx.x] = 0;
    __syncthreads();
    grid_dep_launch();  // the next kernel may be scheduled as this one's CTAs finish

    // ---- this CTA's work: gate_up strips of the shared expert, then of the routed pairs (slot, strip),
    // then the output strips
    const int ss = a.Is / 8, sr = a.I / 8;  // gate_up strips of the shared and of a routed expert
    const int s0 = cta * ss / GD, n_sh = (cta + 1) * ss / GD - s0;
    const int q0 = cta * (K * sr) / GD, n_up = n_sh + (cta + 1) * (K * sr) / GD - q0;
    const int strips_h = a.H / kW4Strip;
    const int my_strips = cta < strips_h ? (strips_h - cta + GD - 1) / GD : 0;
    const int dn = kW4Warps >> p.dwl, d_per = (K + 1 + dn - 1) / dn;  // experts of a down stage, stages of a strip

    if (warp == kW4Warps) {
        // ---------------- producer
        int st = 0, issued = 0;
        uint32_t ph = 0;
        bool ok = true;
        auto next = [&]() {
            if (++st == nst) {
                st = 0;
                ph ^= 1u;
            }
            ++issued;
        };
        auto up = [&](const uint8_t* W, int strip) {
            ok = ok && w4_wait(&empty[st], ph ^ 1u, limit);
            if (!ok) return;
            if (lane == 0) {
                const uint32_t bytes = (uint32_t)(p.R * kRec);
                mbar_arrive_expect_tx(&full[st], bytes);
                bulk_load(stages + (size_t)st * Ring::kStage, W + (size_t)strip * bytes, bytes, &full[st]);
            }
            next();
        };
        // weights only, so before the wait for the previous kernel (no more than the ring holds)
        int i = 0;
        for (; i < n_sh && i < nst; ++i) up(reinterpret_cast<const uint8_t*>(a.sgu), s0 + i);
        grid_dep_wait();
        __syncthreads();
        for (; i < n_sh; ++i) up(reinterpret_cast<const uint8_t*>(a.sgu), s0 + i);
        // (the routing's own wait is bounded by `limit`)
        if (!w4_wait(routed, 0, 4 * limit) && lane == 0) atomicOr(err, ERR_TIMEOUT);
        int slot = q0 / sr, strip = q0 - slot * sr;
        for (; i < n_up && ok; ++i) {
            up(reinterpret_cast<const uint8_t*>(a.gate_up) + (size_t)rt.ids[slot] * p.gu_bytes, strip);
            if (++strip == sr) {
                strip = 0;
                ++slot;
            }
        }
        const int Rs = (a.Is + kW4Cols - 1) / kW4Cols, Rr = (a.I + kW4Cols - 1) / kW4Cols;
        for (int o = 0; o < my_strips && ok; ++o)
            for (int g0 = 0; g0 <= K && ok; g0 += dn) {  // experts: slots 0 .. K-1, then the shared one
                const int n = min(dn, K + 1 - g0), g = g0 + lane;
                ok = w4_wait(&empty[st], ph ^ 1u, limit);
                if (!ok) break;
                if (lane == 0) mbar_arrive_expect_tx(&full[st], (uint32_t)((g0 + n > K ? (n - 1) * Rr + Rs : n * Rr) * kRec));
                __syncwarp();
                if (lane < n) {
                    const int R = g == K ? Rs : Rr;
                    const uint8_t* W = g == K ? reinterpret_cast<const uint8_t*>(a.sd)
                                              : reinterpret_cast<const uint8_t*>(a.down) + (size_t)rt.ids[g] * p.dn_bytes;
                    bulk_load(stages + (size_t)st * Ring::kStage + (size_t)(lane * p.dR) * kRec,
                              W + (size_t)(cta + o * GD) * R * kRec, (uint32_t)(R * kRec), &full[st]);
                }
                __syncwarp();
                next();
            }
        if (!ok && lane == 0) atomicOr(err, ERR_TIMEOUT);
        // every copy issued must land before the CTA's shared memory is released
        if (lane == 0)
            for (int k = 0; k < nst && issued - 1 - k >= 0; ++k) {
                const int j = issued - 1 - k;
                if (!mbar_wait(&full[j % nst], ((uint32_t)(j / nst)) & 1u, limit)) atomicOr(err, ERR_TIMEOUT);
            }
        return;
    }
    if (warp < kW4Warps && (warp & 7) == 0) {
        // this CTA's router rows towards L2, before the wait
        for (int r = cta + (warp >> 3) * GD; r <= a.E; r += 2 * GD)
            for (int i = lane; i < a.H / 64; i += 32)
                asm volatile("prefetch.global.L2 [%0];" ::"l"((r < a.E ? a.router_w + (size_t)r * a.H : a.sg) + 64 * i));
    }
    grid_dep_wait();
    const uint32_t epoch = *(volatile uint32_t*)&a.hdr->dec_epoch;
    const uint32_t sbase = *(volatile uint32_t*)&a.hdr->dec_start_base;
    const uint32_t tag = (epoch + 1u) * 0x9e3779b1u;

    if (warp > kW4Warps) {
        // ---------------- router
        __syncthreads();  // every thread has read the call's number
        if (lane == 0) red_release_add(&a.hdr->dec_start, 1u);
        w4o_route(a, rt, tag, lane, routed);
        asm volatile("bar.arrive 2, %0;" ::"n"(32 * (kW4Warps + 1)) : "memory");  // the weights and the gate are known
        if (cta == 0) {
            // the routing's results, for the workspace's taps
            int pos = 0;
            const int e = lane < K ? rt.ids[lane] : 0;
            for (int j = 0; j < K; ++j) pos += rt.ids[j] < e;
            if (lane < K) {
                a.ids[lane] = e;
                a.topw[lane] = rt.w[lane];
                a.perm[pos] = lane;
                a.inv[lane] = pos;
                a.act[pos] = e;
            }
            for (int q = lane; q <= a.E; q += 32) {
                int below = 0, cnt = 0;
                for (int j = 0; j < K; ++j) {
                    below += rt.ids[j] < q;
                    cnt += rt.ids[j] == q;
                }
                a.offsets[q] = below;
                if (q < a.E) a.counts[q] = cnt;
            }
            if (lane == 0) {
                a.sgate[0] = rt.sg;
                a.hdr->n_act = K;
                // every CTA has read the call's number once all have counted themselves in
                const uint64_t t0 = global_ns();
                while (ld_acquire(&a.hdr->dec_start) - sbase < (uint32_t)GD) {
                    if (global_ns() - t0 > limit) {
                        atomicOr(err, ERR_TIMEOUT);
                        break;
                    }
                    __nanosleep(64);
                }
                a.hdr->dec_epoch = epoch + 1u;
                a.hdr->dec_start_base = sbase + (uint32_t)GD;
            }
        }
        return;
    }

    // ---------------- consumers
    // the residual of this CTA's first output strip, read now: later its latency would come last
    float resid = 0.f;
    if (warp == 0 && my_strips > 0 && a.residual) resid = __bfloat162float(a.residual[cta * kW4Strip + (lane & 15)]);
    if (threadIdx.x < a.H / 8) *reinterpret_cast<uint4*>(xs + 16 * threadIdx.x) = ld_ro(a.x + 8 * threadIdx.x);  // H <= 4096
    if ((warp & 7) == 0) {
        // ---- scores: warps 0 and 8 take a router row each
        for (int r = cta + (warp >> 3) * GD; r <= a.E; r += 2 * GD) {
            const bf16* w = r < a.E ? a.router_w + (size_t)r * a.H : a.sg;
            float acc[2] = {0.f, 0.f};
            const int chunks = a.H / 8;
            for (int c0 = lane; c0 < chunks; c0 += 128) {
                uint4 wv[4], xv[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    wv[i] = xv[i] = make_uint4(0u, 0u, 0u, 0u);
                    if (c0 + 32 * i < chunks) {
                        wv[i] = ld_ro(w + 8 * (c0 + 32 * i));
                        xv[i] = ld_ro(a.x + 8 * (c0 + 32 * i));
                    }
                }
#pragma unroll
                for (int i = 0; i < 4; ++i) acc[i & 1] = dot8_bf16(wv[i], xv[i], acc[i & 1]);
            }
            float sc = warp_sum(acc[0] + acc[1]);
            if (lane == 0) {
                if (r < a.E && a.router_b) sc += __bfloat162float(a.router_b[r]);
                if (!(a.test_suppress == MOE_TEST_SUPPRESS_SCORE && cta == 1))
                    w4o_publish(a.dlog + r, ((uint64_t)tag << 32) | __float_as_uint(sc));
            }
        }
    }
    __syncthreads();  // the token row is in place; every thread has read the call's number

    // ---- gate_up: each warp its records of every strip, sums left in shared memory. The B operands (one
    // live column, token 0) are the same for all strips.
    const int n = lane >> 2, rpw = (p.R + kW4Warps - 1) / kW4Warps, unr = max(0, min(rpw, p.R - rpw * warp));
    uint32_t b[2][16];
    auto load_row = [&](uint32_t (&q)[16], uint32_t row, bool live, int k0, int cols) {
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            const int k = k0 + 32 * c + 8 * (lane & 3);
            uint4 v = make_uint4(0u, 0u, 0u, 0u);
            if (n == 0 && live && k < cols) v = lds128_smem(row + 2u * (uint32_t)k);
            q[4 * c] = v.x; q[4 * c + 1] = v.y; q[4 * c + 2] = v.z; q[4 * c + 3] = v.w;
        }
    };
    load_row(b[0], smem_u32(xs), unr > 0, rpw * warp * kW4Cols, a.H);
    load_row(b[1], smem_u32(xs), unr > 1, (rpw * warp + 1) * kW4Cols, a.H);
    int st = 0;
    uint32_t ph = 0;
    bool ok = true;
    for (int i = 0; i < n_up; ++i) {
        ok = ok && w4_wait(&full[st], ph, 5 * limit);  // (the producer's wait for the routing comes before)
        float acc[4] = {};
        const uint32_t rec = smem_u32(stages) + (uint32_t)(st * Ring::kStage + rpw * warp * kRec);
        w4_records<FMT, G>(rec, unr, b, acc, lane);
        __syncwarp();
        if (lane == 0) mbar_arrive(&empty[st]);
        if ((lane & 3) == 0) {
            float* q = part + (i * kW4Warps + warp) * 16 + n;
            q[0] = acc[0];
            q[8] = acc[2];
        }
        if (++st == nst) {
            st = 0;
            ph ^= 1u;
        }
    }
    w4o_exchange<FMT>(p, rt, part, hs, hpitch, tag, n_sh, n_up, s0, q0, err);

    // ---- down
    const int sub = warp >> p.dwl, kq = warp & ((1 << p.dwl) - 1), r0 = p.drpw * kq;
    for (int o = 0; o < my_strips; ++o) {
        for (int d = 0; d < d_per; ++d) {
            const int g = d * dn + sub, cols = g == K ? a.Is : a.I;
            const int nr = g <= K ? max(0, min(p.drpw, (cols + kW4Cols - 1) / kW4Cols - r0)) : 0;
            const uint32_t row = smem_u32(hs) + (uint32_t)(min(g, K) * hpitch);
            load_row(b[0], row, nr > 0, r0 * kW4Cols, cols);
            load_row(b[1], row, nr > 1, (r0 + 1) * kW4Cols, cols);
            ok = ok && w4_wait(&full[st], ph, limit);
            float acc[4] = {};
            const uint32_t rec = smem_u32(stages) + (uint32_t)(st * Ring::kStage + (sub * p.dR + r0) * kRec);
            w4_records<FMT, G>(rec, nr, b, acc, lane);
            __syncwarp();
            if (lane == 0) mbar_arrive(&empty[st]);
            if ((lane & 3) == 0 && g <= K) {
                float* q = ys + ((g << p.dwl) + kq) * 16 + n;
                q[0] = acc[0];
                q[8] = acc[2];
            }
            if (++st == nst) {
                st = 0;
                ph ^= 1u;
            }
        }
        asm volatile("bar.sync 1, %0;" ::"n"(32 * kW4Warps) : "memory");
        if (warp == 0) {
            // lane l: row l % 16 of the experts l / 16, l / 16 + 2, ...; all read before the ordered sum
            const int r16 = lane & 15, half = lane >> 4, out_row = (cta + o * GD) * kW4Strip + r16;
            constexpr int kHalf = (kOneMaxK + 2) / 2;
            float y[kHalf], all[2 * kHalf];
#pragma unroll
            for (int j = 0; j < kHalf; ++j) {
                const int e = min(2 * j + half, K);
                const float* q = ys + (e << p.dwl) * 16 + r16;
                y[j] = q[0];
                if (p.dwl > 0) y[j] += q[16];
                for (int k = 2; k < (1 << p.dwl); ++k) y[j] += q[k * 16];
                y[j] *= (e == K ? rt.sg : rt.w[e]) * W4Fold<FMT>::kUnfold;
            }
#pragma unroll
            for (int j = 0; j < kHalf; ++j) {
                const float z = __shfl_xor_sync(0xffffffffu, y[j], 16);
                all[2 * j] = half ? z : y[j];
                all[2 * j + 1] = half ? y[j] : z;
            }
            float v = o == 0 ? resid : a.residual ? __bfloat162float(a.residual[out_row]) : 0.f;
#pragma unroll
            for (int e = 0; e <= kOneMaxK; ++e)
                if (e == K) v += all[e];  // the shared expert, then slots 0 .. K-1
#pragma unroll
            for (int e = 0; e < kOneMaxK; ++e)
                if (e < K) v += all[e];
            if (half == 0) a.out[out_row] = __float2bfloat16_rn(v);
#pragma unroll
            for (int j = 0; j < kHalf; ++j)
                if (2 * j + half <= K) a.Y[(size_t)(2 * j + half) * a.H + out_row] = y[j];  // tap 1
        }
        if (o + 1 < my_strips) asm volatile("bar.sync 1, %0;" ::"n"(32 * kW4Warps) : "memory");
    }
    if (!ok && lane == 0) atomicOr(err, ERR_TIMEOUT);
}

// Whether one CTA per SM of the kernel fits on the current device (checked once per device, with the
// largest shared memory it takes).
template <int FMT, int G>
bool w4_one_fits() {
    static int fits[64] = {};  // 0 unknown, 1 yes, 2 no
    int dev = 0;
    cudaGetDevice(&dev);
    if (dev < 0 || dev >= 64) dev = 0;
    if (!fits[dev]) {
        int n = 0;
        const bool ok = cudaFuncSetAttribute(k_w4_one<FMT, G>, cudaFuncAttributeMaxDynamicSharedMemorySize, kW4SmemMax) ==
                            cudaSuccess &&
                        cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, k_w4_one<FMT, G>, kOneThreads, kW4SmemMax) ==
                            cudaSuccess &&
                        n >= 1;
        (void)cudaGetLastError();
        fits[dev] = ok ? 1 : 2;
    }
    return fits[dev] == 1;
}

template <int FMT, int G>
cudaError_t launch_w4_one_t(const W4OneArgs& p, cudaStream_t s) {
    using Ring = W4OneRing<FMT, G>;
    const int nst = w4_one_stages<FMT, G>(p.a.K, p.a.Imax, p.a.H);
    const size_t bytes = (size_t)Ring::kFixed + w4_one_rows(p.a.K, p.a.Imax, p.a.H) + (size_t)nst * Ring::kStage;
    cudaError_t e;
    MOE_LAUNCH(MOE_KERNEL_W4_FUSED, s, (e = launch_pdl(k_w4_one<FMT, G>, dim3(p.a.num_sms), dim3(kOneThreads), bytes, s, p, nst)));
    return e;
}

// p NULL: only whether the kernel fits.
template <int FMT>
cudaError_t w4_one_f(int group, const W4OneArgs* p, cudaStream_t s) {
#define MOE_W4_CASE(G) \
    if (group == G) return p ? launch_w4_one_t<FMT, G>(*p, s) : w4_one_fits<FMT, G>() ? cudaSuccess : cudaErrorNotSupported
    MOE_W4_CASE(32);
    MOE_W4_CASE(64);
    MOE_W4_CASE(128);
#undef MOE_W4_CASE
    return cudaErrorInvalidValue;
}

// One translation unit per format; p NULL asks whether the kernel fits.
cudaError_t w4_one_int4(int group, const W4OneArgs* p, cudaStream_t s);
cudaError_t w4_one_int4_zp(int group, const W4OneArgs* p, cudaStream_t s);
cudaError_t w4_one_e2m1(int group, const W4OneArgs* p, cudaStream_t s);

#endif

}  // namespace moe
