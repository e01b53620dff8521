// linear.cu -- linear layers with bias, activation and residual in the epilogue, and their gradients, for
// one weight matrix or for one to each expert's rows, on the 5th-generation tensor cores.
//
//   kFwd   out = act(x . W_e^T + b_e) + residual      D[n, t] = sum_k W_e[n, k] x[t, k]
//   kDx    dx  = dz . W_e                             D[k, t] = sum_n W_e[n, k] dz[t, n]
//   kDw    dW_e = dz_e^T . x_e                        D[k, n] = sum_t x[t, k] dz[t, n], t over expert e's rows
// with dz = act'(z) * dout from an elementwise kernel that also leaves the bias' column sums.
//
// In all three the 128 lanes of the accumulator are what is contiguous in the result, and its columns are
// the result's rows: token rows (kFwd, kDx), of which a tile takes as many as there are, in steps of
// 16, so that experts with few rows cost few columns; or W's rows (kDw). Operands are read as they
// lie in memory: K-major where the contraction is contiguous, else MN-major (W in kDx, both in kDw), so
// nothing is transposed beforehand. For swiglu a tile's 128 weight rows are 64 gate rows and the 64
// matching up rows in turns of 16, by a five-dimensional tensor map: gate and up of a feature are
// then 16 lanes apart, in one warp's reach.
//
// Three kernels: the one here, tiles of 128 features by up to 64 columns, where rows are few and the weights' way from HBM is
// what counts; pairs of SMs on 256 x 256 where they are many (linear_pair.cu); a warp to a feature for a handful of
// rows (linear_few.cu). lin_plan and few_rows below choose.
//
// Here one CTA an SM walks its share of the tiles (expert by expert, then 128 features, then columns, so tiles
// that share weights run side by side and meet in L2). Warp 0 loads by TMA into a ring of seven 64-deep stages (112 KB of
// weights on their way), warp 1 issues the MMAs into one of two accumulators in tensor memory, warps 4 - 11 write the other
// out: fp32 through shared memory, so that a lane has four features side by side. With few tiles a cluster of up to 8 CTAs takes one
// tile's contraction in parts; the parts are added in rank order through distributed shared memory. Sums are fp32 in a
// fixed order throughout. Bound by HBM: 64 tokens' 512 rows through 256 experts of 1024 x 2048, 142 us = 6.6 TB/s.
#include <atomic>

#include "linear.cuh"

namespace moe {

constexpr int kPartPitch = 132;           // floats of a column of the cluster's partial tile (4 mod 32: no bank conflicts)
constexpr int kStagePitch = 36;           // floats of a column of a warp's transposition buffer (the same)

// Columns of a tile, at most, and the ring: 16 KB of weights a stage, 112 KB on their way.
constexpr int kLinCols = 64, kLinStages = 7;
constexpr uint32_t kLinB = kLinCols * 64 * 2;
constexpr uint32_t kLinRing = kLinStages * (kLinA + kLinB);
constexpr uint32_t kLinScratch = kLinCols * kPartPitch * 4;
constexpr uint32_t kLinTables = 2 * (kLinMaxE + 4) * 4;
constexpr uint32_t kLinBytes = 1024 + kLinRing + kLinScratch + kLinTables + 256;
constexpr uint32_t kLinTmem = 2 * kLinCols;
static_assert(kLinEpiWarps * 16 * kStagePitch * 4 <= kLinScratch, "transposition buffers");

// Four consecutive features of one row of the result, from their sums v (and the up sums u).
template <typename T, bool GATED>
__device__ __forceinline__ void lin_finish(const LinView& a, int64_t row, int f, float (&v)[4], float (&u)[4], const float (&bv)[4],
                                           const float (&bu)[4]) {
    typedef Vec<T, 4> V;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[i] += bv[i];
        if (GATED) u[i] += bu[i];
    }
    T* out = reinterpret_cast<T*>(a.out) + row * a.F + f;
    const T* res = a.residual ? reinterpret_cast<const T*>(a.residual) + row * a.F + f : nullptr;
    T* z = a.z ? reinterpret_cast<T*>(a.z) + row * a.N + f : nullptr;
    float o[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) o[i] = GATED ? v[i] * lin_sigmoid(v[i]) * u[i] : v[i];
    if (!GATED) lin_act<4>(a.act, o);
    if (a.vec && f + 4 <= a.F) {
        if (res) {
            const V r = *reinterpret_cast<const V*>(res);
#pragma unroll
            for (int i = 0; i < 4; ++i) o[i] += to_f(r.v[i]);
        }
        V w;
#pragma unroll
        for (int i = 0; i < 4; ++i) w.v[i] = from_f<T>(o[i]);
        *reinterpret_cast<V*>(out) = w;
        if (z) {
#pragma unroll
            for (int i = 0; i < 4; ++i) w.v[i] = from_f<T>(v[i]);
            *reinterpret_cast<V*>(z) = w;
            if (GATED) {
#pragma unroll
                for (int i = 0; i < 4; ++i) w.v[i] = from_f<T>(u[i]);
                *reinterpret_cast<V*>(z + a.F) = w;
            }
        }
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if (f + i < a.F) {
                out[i] = from_f<T>(o[i] + (res ? to_f(res[i]) : 0.f));
                if (z) {
                    z[i] = from_f<T>(v[i]);
                    if (GATED) z[a.F + i] = from_f<T>(u[i]);
                }
            }
        }
    }
}

template <typename T>
__device__ __forceinline__ void lin_bias(const LinView& a, int e, int f, float (&b)[4]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) b[i] = a.bias && f + i < a.F ? to_f(reinterpret_cast<const T*>(a.bias)[(int64_t)e * a.N + f + i]) : 0.f;
}
template <typename T>
__device__ __forceinline__ void lin_bias_up(const LinView& a, int e, int f, float (&b)[4]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) b[i] = a.bias && f + i < a.F ? to_f(reinterpret_cast<const T*>(a.bias)[(int64_t)e * a.N + a.F + f + i]) : 0.f;
}

template <typename T, int MODE, bool GATED>
__global__ void __launch_bounds__(kLinThreads, 1)
    k_linear(const __grid_constant__ CUtensorMap mA, const __grid_constant__ CUtensorMap mB, const LinView a) {
    constexpr int kStages = kLinStages;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = smem_u32(smem_raw);
    uint8_t* smem = smem_raw + (((raw + 1023u) & ~1023u) - raw);
    uint8_t* sA = smem;
    uint8_t* sB = smem + kStages * kLinA;
    float* scratch = reinterpret_cast<float*>(smem + kLinRing);
    int* off = reinterpret_cast<int*>(smem + kLinRing + kLinScratch);
    int* start = off + kLinMaxE + 4;
    uint64_t* full = reinterpret_cast<uint64_t*>(smem + kLinRing + kLinScratch + kLinTables);
    uint64_t* empty = full + kStages;
    uint64_t* accf = empty + kStages;
    uint64_t* acce = accf + 2;
    uint64_t* mma_done = acce + 2;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(mma_done + 1);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
    volatile int* progress = abort_flag + 1;  // kDw: stages that this CTA's producer has found empty, which the longer waits go by
    static_assert((2 * kStages + 5) * 8 + 12 <= 256, "barrier area");

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = cluster_rank(), split = cluster_size();
    if (threadIdx.x == 0) {
        for (int s = 0; s < kStages; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(&accf[b], 1);
            mbar_init(&acce[b], kLinEpiWarps);
        }
        mbar_init(mma_done, 1);
        *abort_flag = 0;
        *progress = 0;
        fence_mbar_init();
        tma_prefetch_desc(&mA);
        tma_prefetch_desc(&mB);
    }
    if (warp == 1) {
        tmem_alloc(tmem_slot, kLinTmem);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    grid_dep_wait();  // everything is read from here on: operands, offsets and workspace may be the previous kernel's
    grid_dep_launch();
    lin_tables<MODE>(a, off, start);
    const int total = start[a.E];
    const int step = gridDim.x / split, first = blockIdx.x / split;
    LinWalk<MODE, 16> walk;

    if (warp == 0) {
        // ---------------- TMA producer (one lane; the warp stays together for the cluster's barriers)
        int it = 0;
        bool loads = false;
        for (int t = first; t < total; t += step) {
            if (elect_one() && !*abort_flag) {
                loads = true;
                const LinTile ti = walk.to(a, off, start, t);
                const int kb0 = (int)((int64_t)ti.blocks * rank / split), kb1 = (int)((int64_t)ti.blocks * (rank + 1) / split);
                const int boxes = MODE == kDw ? (ti.cols + 63) / 64 : (ti.cols + kLinBoxRows - 1) / kLinBoxRows;
                const uint32_t bytes = kLinA + (uint32_t)boxes * (MODE == kDw ? 64 : kLinBoxRows) * 128u;
                for (int kb = kb0; kb < kb1; ++kb, ++it) {
                    const int s = it % kStages;
                    const uint32_t ph = (uint32_t)(it / kStages) & 1u;
                    if (!mbar_wait(&empty[s], ph ^ 1u, a.wait_ns)) {
                        atomicOr(a.err, ERR_TIMEOUT);
                        *abort_flag = 1;
                        break;
                    }
                    if (MODE == kDw) *progress = it + 1;
                    if (a.suppress && blockIdx.x == 0 && it == 0) continue;
                    mbar_arrive_expect_tx(&full[s], bytes);
                    uint8_t* da = sA + s * kLinA;
                    uint8_t* db = sB + s * kLinB;
                    if (MODE == kFwd) {
                        if (GATED)
                            tma_load_5d(da, &mA, &full[s], kb * 64, 0, 0, ti.f * 4, ti.e);
                        else
                            tma_load_3d(da, &mA, &full[s], kb * 64, ti.f * 128, ti.e);
                    } else if (MODE == kDx) {
                        for (int p = 0; p < 2; ++p) tma_load_3d(da + p * 8192, &mA, &full[s], ti.f * 128 + p * 64, kb * 64, ti.e);
                    } else {
                        for (int p = 0; p < 2; ++p) tma_load_2d(da + p * 8192, &mA, &full[s], ti.f * 128 + p * 64, ti.row0 + kb * 64);
                    }
                    if (MODE == kDw)
                        for (int p = 0; p < boxes; ++p) tma_load_2d(db + p * 8192, &mB, &full[s], ti.c0 + p * 64, ti.row0 + kb * 64);
                    else
                        for (int p = 0; p < boxes; ++p)
                            tma_load_2d(db + p * (kLinBoxRows * 128), &mB, &full[s], kb * 64, ti.row0 + ti.c0 + p * kLinBoxRows);
                }
            }
            __syncwarp();
            if (split > 1) {
                cluster_sync_all();
                cluster_sync_all();
            }
        }
        // every copy this CTA issued must land before shared memory is released
        if (loads)
            for (int s = 0; s < min(it, kStages); ++s)  // (its last use: number (it - 1 - s) / kStages)
                if (!mbar_wait(&full[s], (uint32_t)((it - 1 - s) / kStages) & 1u, a.wait_ns)) atomicOr(a.err, ERR_TIMEOUT);
        __syncwarp();
    } else if (warp == 1) {
        // ---------------- MMA issuer
        int it = 0, local = 0;
        for (int t = first; t < total; t += step, ++local) {
            bool ok = !*abort_flag;
            ok = __shfl_sync(0xffffffffu, ok, 0);
            if (ok) {
                const LinTile ti = walk.to(a, off, start, t);
                const int kb0 = (int)((int64_t)ti.blocks * rank / split), kb1 = (int)((int64_t)ti.blocks * (rank + 1) / split);
                const int n16 = (ti.cols + 15) / 16 * 16;
                const uint32_t idesc = idesc_f16_f32(std::is_same<T, bf16>::value, 128, n16, MODE != kFwd, MODE == kDw);
                const int b = local & 1;
                const uint32_t use = (uint32_t)(local >> 1) & 1u;
                const uint32_t d = tmem + (uint32_t)(b * kLinCols);
                ok = mbar_wait(&acce[b], use ^ 1u, a.wait_ns);
                ok = __all_sync(0xffffffffu, ok);
                tc_fence_after();
                for (int kb = kb0; ok && kb < kb1; ++kb, ++it) {
                    const int s = it % kStages;
                    const uint32_t ph = (uint32_t)(it / kStages) & 1u;
                    ok = mbar_wait(&full[s], ph, a.wait_ns);
                    ok = __all_sync(0xffffffffu, ok);
                    if (!ok) break;
                    const uint32_t aa = smem_u32(sA + s * kLinA), bb = smem_u32(sB + s * kLinB);
                    int steps = 4;
                    if (MODE == kDw) {
                        // the expert's last block: 16 rows at a time, rows of the next expert in the last 16 set
                        // to zero in both operands (whatever they hold: 0 x infinity would stay)
                        const int left = ti.rows - kb * 64;
                        if (left < 64) {
                            steps = (left + 15) / 16;
                            if (left & 15) {
                                const int panels = 2 + (ti.cols + 63) / 64, rows = steps * 16 - left;
                                const uint32_t zero[4] = {0u, 0u, 0u, 0u};
                                for (int p = 0; p < panels; ++p) {
                                    const uint32_t at = (p < 2 ? aa + p * 8192 : bb + (p - 2) * 8192) + (uint32_t)left * 128u;
                                    for (int i = lane; i < rows * 8; i += 32) sts128(at + (uint32_t)i * 16u, zero);
                                }
                                fence_proxy_async_smem();
                                __syncwarp();
                            }
                        }
                    }
                    tc_fence_after();
                    if (elect_one()) {
                        for (int kk = 0; kk < steps; ++kk) {
                            const uint64_t da = MODE == kFwd ? sdesc_kmajor_sw128(aa + kk * 32) : sdesc_mnmajor_sw128(aa + kk * 2048, 8192);
                            const uint64_t db = MODE == kDw ? sdesc_mnmajor_sw128(bb + kk * 2048, 8192) : sdesc_kmajor_sw128(bb + kk * 32);
                            mma_bf16(d, da, db, idesc, kb != kb0 || kk != 0);
                        }
                        mma_commit(&empty[s]);
                        if (kb + 1 == kb1) mma_commit(&accf[b]);
                    }
                    __syncwarp();
                }
                if (ok && kb0 == kb1 && lane == 0) mbar_arrive(&accf[b]);  // (no rows: zeros are written)
                if (!ok && lane == 0) {
                    atomicOr(a.err, ERR_TIMEOUT);
                    *abort_flag = 1;
                }
                __syncwarp();
            }
            if (split > 1) {
                cluster_sync_all();
                cluster_sync_all();
            }
        }
        if (elect_one()) mma_commit(mma_done);
        __syncwarp();
        if (!mbar_wait(mma_done, 0, a.wait_ns) && lane == 0) atomicOr(a.err, ERR_TIMEOUT);
        __syncwarp();
    } else if (warp >= kLinEpiWarp0) {
        // ---------------- epilogue: lanes 32 q .. of the accumulator, every other 16 columns
        const int q = warp & 3, h = (warp - kLinEpiWarp0) >> 2;
        const int g = lane >> 2, tt = lane & 3;
        float* mine = scratch + (warp - kLinEpiWarp0) * 16 * kStagePitch;
        int local = 0;
        for (int t = first; t < total; t += step, ++local) {
            const LinTile ti = walk.to(a, off, start, t);
            const int kb0 = (int)((int64_t)ti.blocks * rank / split), kb1 = (int)((int64_t)ti.blocks * (rank + 1) / split);
            const int b = local & 1;
            const uint32_t use = (uint32_t)(local >> 1) & 1u;
            const int64_t row0 = MODE == kDw ? (int64_t)ti.e * a.N + ti.c0 : (int64_t)ti.row0 + ti.c0;
            // a lane's four features: those of chunk lane % 8 (gated: lane % 4) of the warp's 32 lanes
            const int f = GATED ? ti.f * 64 + q * 16 + (lane & 3) * 4 : ti.f * 128 + q * 32 + (lane & 7) * 4;
            float bv[4], bu[4];
            if (split == 1) {
                lin_bias<T>(a, ti.e, f, bv);
                if (GATED) lin_bias_up<T>(a, ti.e, f, bu);
            }
            bool ready = false;
            if (!*abort_flag)  // (a tile's whole contraction: of kDw as long as an expert has rows, else of 2^14 stages at most)
                ready = MODE == kDw ? mbar_wait_progress(&accf[b], use, progress, a.wait_ns) : mbar_wait(&accf[b], use, a.wait_ns);
            ready = __all_sync(0xffffffffu, ready);
            if (!ready && lane == 0) {
                if (!*abort_flag) atomicOr(a.err, ERR_TIMEOUT);
                *abort_flag = 1;
            }
            if (ready) {
                tc_fence_after();
                const uint32_t tb = tmem + ((uint32_t)(q * 32) << 16) + (uint32_t)(b * kLinCols);
                for (int c = h * 16; c < ti.cols; c += 32) {
                    uint32_t r[16];
                    if (kb0 < kb1) {
                        tmem_ld_frag2(tb + c, r);
                        tmem_ld_frag2(tb + (16u << 16) + c, r + 8);
                        tmem_ld_wait16(r);
                    } else {
#pragma unroll
                        for (int i = 0; i < 16; ++i) r[i] = 0u;
                    }
                    if (split > 1) {
                        float* p = scratch + c * kPartPitch + q * 32;
#pragma unroll
                        for (int i = 0; i < 16; ++i)  // register i: lane g + 8 (i / 2 % 2) + 16 (i / 8), column 8 (i / 4 % 2) + 2 tt + i % 2
                            p[(8 * ((i >> 2) & 1) + 2 * tt + (i & 1)) * kPartPitch + g + 8 * ((i >> 1) & 1) + 16 * (i >> 3)] = __uint_as_float(r[i]);
                        continue;
                    }
#pragma unroll
                    for (int i = 0; i < 16; ++i)
                        mine[(8 * ((i >> 2) & 1) + 2 * tt + (i & 1)) * kStagePitch + g + 8 * ((i >> 1) & 1) + 16 * (i >> 3)] = __uint_as_float(r[i]);
                    __syncwarp();
                    constexpr int kPer = GATED ? 8 : 4;  // columns of one round
#pragma unroll
                    for (int i = 0; i < 16 / kPer; ++i) {
                        const int col = i * kPer + lane / (32 / kPer);
                        float v[4], u[4] = {0.f, 0.f, 0.f, 0.f};
                        const float4 x = *reinterpret_cast<const float4*>(mine + col * kStagePitch + (lane & (32 / kPer - 1)) * 4);
                        v[0] = x.x; v[1] = x.y; v[2] = x.z; v[3] = x.w;
                        if (GATED) {
                            const float4 y = *reinterpret_cast<const float4*>(mine + col * kStagePitch + 16 + (lane & 3) * 4);
                            u[0] = y.x; u[1] = y.y; u[2] = y.z; u[3] = y.w;
                        }
                        if (c + col < ti.cols) lin_finish<T, GATED>(a, row0 + c + col, f, v, u, bv, bu);
                    }
                    __syncwarp();
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&acce[b]);
            }
            if (split > 1) {
                __syncwarp();
                cluster_sync_all();
                if (ready) {
                    // the tile's (column, four features) in rows of the cluster's threads; the parts in rank order
                    constexpr int kChunks = GATED ? 16 : 32;
                    const int me = (int)rank * (kLinEpiWarps * 32) + (int)threadIdx.x - kLinEpiWarp0 * 32;
                    for (int i = me; i < ti.cols * kChunks; i += (int)split * kLinEpiWarps * 32) {
                        const int col = i / kChunks, ch = i % kChunks;
                        const int at = GATED ? (ch >> 2) * 32 + (ch & 3) * 4 : ch * 4;
                        const int ff = GATED ? ti.f * 64 + ch * 4 : ti.f * 128 + ch * 4;
                        const uint32_t addr = smem_u32(scratch + col * kPartPitch + at);
                        float v[4] = {0.f, 0.f, 0.f, 0.f}, u[4] = {0.f, 0.f, 0.f, 0.f};
                        lin_bias<T>(a, ti.e, ff, bv);
                        if (GATED) lin_bias_up<T>(a, ti.e, ff, bu);
                        float4 x[8], y[8];  // all on their way at once
#pragma unroll
                        for (uint32_t r = 0; r < 8; ++r)
                            if (r < split) {
                                x[r] = ld_peer(addr, r);
                                if (GATED) y[r] = ld_peer(addr + 64, r);
                            }
#pragma unroll
                        for (uint32_t r = 0; r < 8; ++r)
                            if (r < split) {
                                v[0] += x[r].x; v[1] += x[r].y; v[2] += x[r].z; v[3] += x[r].w;
                                if (GATED) {
                                    u[0] += y[r].x; u[1] += y[r].y; u[2] += y[r].z; u[3] += y[r].w;
                                }
                            }
                        if (ff < a.F) lin_finish<T, GATED>(a, row0 + col, ff, v, u, bv, bu);
                    }
                }
                __syncwarp();
                cluster_sync_all();
            }
        }
    } else {
        if (MODE != kFwd && a.dbias) {
            lin_dbias<T>(a, off, blockIdx.x * 2 + warp - 2, gridDim.x * 2);
            __syncwarp();
        }
        if (split > 1)
            for (int t = first; t < total; t += step) {
                cluster_sync_all();
                cluster_sync_all();
            }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, kLinTmem);
    }
}

// ---------------------------------------------------------------------------------------
// dz = act'(z) * dout, and the column sums of it for the bias. Bound by HBM (32768 rows of 1024, swiglu: 28 us = 5.9 TB/s) until
// GELU's slope and the sums take the issue slots (4096 rows of 8192 with both: 43 us = 4.7 TB/s). A CTA takes a chunk of 4, 32 or 128 rows and 128
// columns (for swiglu 128 gate columns and the matching up columns); 16 threads side by side hold 8 columns
// each, 16 rows at a time. Sums are of dz before its rounding, row block by row block: those of the rows of
// expert e in chunk c go to part[c + e], a place of their own as chunks and experts follow one another. dz itself is rounded to the
// tensors' type, which the tensor cores take: dx and dW are then 1.41 times as far from 64 bits as by an fp32 dz (bf16 2.35e-3 of the norm against
// 1.66e-3, fp16 2.9e-4 against 2.1e-4); to hold the rest of it in a second matrix would double both products.

template <typename T>
__device__ __forceinline__ void st_cols(T* p, const Raw& r) { *reinterpret_cast<uint4*>(p) = make_uint4(r.w[0], r.w[1], r.w[2], r.w[3]); }

template <typename T, int VE, bool GATED>
__global__ void __launch_bounds__(256, 3) k_dz(const LinearArgs a, int pitch) {
    __shared__ int off[kLinMaxE + 1];
    __shared__ float sums[GATED ? 2 : 1][16][128];
    typedef RawOf<T> R;
    grid_dep_wait();
    grid_dep_launch();
    const int N = a.d.N, E = a.d.E, wide = GATED ? N / 2 : N;
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    const int r0 = blockIdx.x * a.chunk, r1 = min(r0 + a.chunk, a.d.T);
    const int f = blockIdx.y * 128 + tx * 8, n = min(8, wide - f);  // columns of this thread (none: n <= 0)
    const bool need_z = GATED || a.d.act != MOE_ACT_NONE;
    T* dz = reinterpret_cast<T*>(a.dz);
    const T *z = reinterpret_cast<const T*>(a.z_in), *dout = reinterpret_cast<const T*>(a.dout);
    Raw dv, zv, uv;
    auto load = [&](int r) {
        dv = ld_cols<T, VE>(dout, (int64_t)r * wide + f, (int64_t)a.d.T * wide, n);
        if (need_z) zv = ld_cols<T, VE>(z, (int64_t)r * N + f, (int64_t)a.d.T * N, n);
        if (GATED) uv = ld_cols<T, VE>(z, (int64_t)r * N + wide + f, (int64_t)a.d.T * N, n);
    };
    // whose rows they are matters to the column sums alone (rows behind the last expert's are read into nothing)
    const bool split = a.offsets && a.dbias;
    int lo = 0, hi = split ? E : 1;
    if (split) {
        for (int e = threadIdx.x; e <= E; e += 256) off[e] = min(max(a.offsets[e], 0), a.d.T);
        __syncthreads();
        while (hi - lo > 1) {  // the last expert whose rows begin at or before r0
            const int mid = (lo + hi) >> 1;
            if (off[mid] <= r0) lo = mid; else hi = mid;
        }
        hi = E;
    }
    for (int e = lo; e < hi; ++e) {
        const int b0 = split ? max(off[e], r0) : r0, b1 = split ? min(off[e + 1], r1) : r1;
        if (split && off[e] >= r1) break;
        if (b0 >= b1) continue;
        float sv[8], su[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) sv[i] = su[i] = 0.f;
        const int last = n > 0 ? b1 : b0;
        if (b0 + ty < last) load(b0 + ty);
        for (int r = b0 + ty; r < last; r += 16) {
            float d[8], v[8], u[8];
            R::values(dv, d);
            if (need_z) R::values(zv, v);
            if (GATED) R::values(uv, u);
            if (r + 16 < last) load(r + 16);  // the next row comes while this one is worked on
            const int64_t at = (int64_t)r * pitch + f;
            if (GATED) {
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const float p = lin_sigmoid(v[i]), dd = d[i];
                    d[i] = dd * u[i] * (p * (1.f + v[i] * (1.f - p)));
                    u[i] = dd * (v[i] * p);
                    su[i] += u[i];
                }
                if (dz) st_cols(dz + at + wide, R::pack(u));
            } else {
                lin_slope<8>(a.d.act, v, d);
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                if (VE == 1 && i >= n) d[i] = 0.f;  // (columns up to the pitch are zeros)
                sv[i] += d[i];
            }
            if (dz) st_cols(dz + at, R::pack(d));
        }
        if (a.dbias) {
            __syncthreads();
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                sums[0][ty][tx * 8 + i] = sv[i];
                if (GATED) sums[GATED ? 1 : 0][ty][tx * 8 + i] = su[i];
            }
            __syncthreads();
            const int half = threadIdx.x >> 7, col = threadIdx.x & 127;
            if (half < (GATED ? 2 : 1) && (int)blockIdx.y * 128 + col < wide) {
                float s = 0.f;
#pragma unroll
                for (int i = 0; i < 16; ++i) s += sums[half][i][col];
                a.part[(int64_t)((int)blockIdx.x + e) * N + half * wide + blockIdx.y * 128 + col] = s;
            }
        }
    }
}

// db alone, where no product is asked for.
template <typename T>
__global__ void __launch_bounds__(256) k_dbias(const LinView a) {
    __shared__ int off[kLinMaxE + 1];
    grid_dep_wait();
    grid_dep_launch();
    for (int e = threadIdx.x; e <= a.E; e += 256) {
        const int o = a.offsets ? a.offsets[e] : e ? a.T : 0;
        off[e] = min(max(o, 0), a.T);
        if (off[e] != o || (a.offsets && e && o < a.offsets[e - 1])) atomicOr(a.err, ERR_BAD_ROUTE);
    }
    __syncthreads();
    lin_dbias<T>(a, off, blockIdx.x * 8 + (threadIdx.x >> 5), gridDim.x * 8);
}

// ---------------------------------------------------------------------------------------
// host side

namespace {

template <typename T, int MODE, bool GATED>
cudaError_t launch_k(const CUtensorMap& A, const CUtensorMap& B, const LinView& v, int grid, int split, cudaStream_t s) {
    static std::atomic<bool> allowed[64];
    const cudaError_t e = allow_shared(k_linear<T, MODE, GATED>, (int)kLinBytes, allowed);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(kLinThreads);
    cfg.dynamicSmemBytes = kLinBytes;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = split;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = split > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, k_linear<T, MODE, GATED>, A, B, v);
}

struct LinPlan {
    bool pair;
    int colw, grid, split, width;  // columns of a tile, at most; CTAs; CTAs to a tile's contraction; columns of a tile as they are cut
};

// Clusters of `split` CTAs of the split kernel that the device holds at once (clusters lie within a GPC, so there are
// fewer than its SMs divided by their size).
template <typename T, int MODE, bool GATED>
int resident_clusters(int split, int num_sms) {
    static std::atomic<int> cache[64][3];
    int dev = 0, slot = split == 2 ? 0 : split == 4 ? 1 : 2;
    cudaGetDevice(&dev);
    if (dev < 0 || dev >= 64) return num_sms / split / 2;
    int n = cache[dev][slot].load(std::memory_order_relaxed);
    if (n) return n - 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(num_sms / split * split);
    cfg.blockDim = dim3(kLinThreads);
    cfg.dynamicSmemBytes = kLinBytes;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = split;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (cudaFuncSetAttribute(k_linear<T, MODE, GATED>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kLinBytes) != cudaSuccess ||
        cudaOccupancyMaxActiveClusters(&n, k_linear<T, MODE, GATED>, &cfg) != cudaSuccess) {
        cudaGetLastError();
        n = 0;
    }
    cache[dev][slot].store(n + 1, std::memory_order_relaxed);
    return n;
}

// Which kernel, and its tiles. groups: experts with rows, about; cols: columns of one of them, about (ragged: they are
// experts' rows); F: features (lanes) in weight rows; blocks: 64-deep steps of the contraction, about.
// Time of a 16-deep step, in clocks: on a pair, 256 features by w columns take w / 2 on the tensor cores and
// (8 KB + 32 w B) / 128 B = 64 + w / 4 through each SM's shared memory (TMA's writes and the tensor core's reads of
// its half), the more of the two up to 256 columns; one SM's 128 x 64 take 96. A wave of tiles costs its widest. With
// 64 columns or fewer the weights' way from HBM is what counts: one SM a tile, and clusters that split the contraction as long as all of them are
// resident at once (2048 x 2048, 16 tokens: clusters of 4 take 9.2 us, of 8 in two turns 15.0, one CTA a tile 12.9).
template <typename T, int MODE, bool GATED>
LinPlan lin_plan(int64_t groups, int64_t cols, bool ragged, int64_t F, int blocks, int num_sms) {
    LinPlan p = {false, kLinCols, 0, 1, 0};
    const int64_t f1 = (F + 127) / 128, f2 = (F + 255) / 256;
    const int64_t tiles = groups * f1 * ((cols + kLinCols - 1) / kLinCols);
    while (p.split < 8 && p.split * 2 <= blocks && tiles <= resident_clusters<T, MODE, GATED>(p.split * 2, num_sms)) p.split *= 2;
    // (experts' tiles are more or fewer than thought: CTAs for all that can be)
    p.grid = (int)(!ragged && tiles * p.split < num_sms ? tiles * p.split : num_sms) / p.split * p.split;
    if (cols <= kLinCols || num_sms < 2) return p;
    int64_t best = (tiles * p.split + num_sms - 1) / num_sms * 96 / p.split;
    for (int w = 256; w >= 64; w /= 2) {
        // tiles of a group's columns, twice: of experts' rows half a tile more than they fill, on average
        const int64_t n2 = ragged ? (2 * cols > w ? 2 * cols / w + 1 : 2) : 2 * ((cols + w - 1) / w);
        const int64_t width = ((2 * cols + n2 - 1) / n2 + 31) / 32 * 32, all = (groups * f2 * n2 + 1) / 2;
        const int64_t cost = (all + num_sms / 2 - 1) / (num_sms / 2) * (64 + width / 4);
        if (cost < best) {
            best = cost;
            p = {true, w, 2 * (int)(!ragged && all < num_sms / 2 ? all : num_sms / 2), 1, (int)width};
        }
    }
    return p;
}

// Rows of the pair kernel's column-side box: a CTA's half of a tile where all tiles are alike, else 32.
int pair_boxes(const LinPlan& p, bool one_group) { return one_group && p.pair ? p.width / 2 : kLinBoxRows; }

template <typename T, int MODE, bool GATED>
cudaError_t launch_plan(int32_t dtype, const LinPlan& p, const CUtensorMap& A, const CUtensorMap& B, const CUtensorMap& C, LinView v, cudaStream_t s) {
    v.colw = p.colw;
    const int per = (p.pair ? 256 : 128) / (GATED ? 2 : 1);
    v.ftiles = (v.F + per - 1) / per;
    v.vec = v.F % (p.pair ? 8 : 4) == 0;
    return p.pair ? launch_pair(dtype, MODE, GATED, A, B, C, v, p.grid, s) : launch_k<T, MODE, GATED>(A, B, v, p.grid, p.split, s);
}

// Row-major [rows, cols] with `pitch` elements between rows.
bool map_2d(CUtensorMap* m, int32_t dt, const void* p, uint64_t rows, uint64_t cols, uint64_t pitch, uint32_t box_rows) {
    const uint64_t d[2] = {cols, rows}, st[1] = {pitch * 2};
    const uint32_t b[2] = {64, box_rows};
    return encode_map(m, dt, p, 2, d, st, b);
}
// The same as 64 rows from any first one, [rows, 64, cols] whose two row strides are one and the same, for boxes of 64 that may begin
// at a negative row of the 64. (What a box then reads ends with the first row's 64th at the latest, and the kernel's with an expert's last.)
bool map_64(CUtensorMap* m, int32_t dt, const void* p, uint64_t rows, uint64_t cols, uint64_t pitch) {
    const uint64_t d[3] = {cols, 64, rows}, st[2] = {pitch * 2, pitch * 2};
    const uint32_t b[3] = {64, 64, 1};
    return encode_map(m, dt, p, 3, d, st, b);
}
// W [E, N, K].
bool map_w(CUtensorMap* m, const moe_linear_dims& d, const void* w, uint32_t box_rows) {
    const uint64_t dim[3] = {(uint64_t)d.K, (uint64_t)d.N, (uint64_t)d.E}, st[2] = {(uint64_t)d.K * 2, (uint64_t)d.N * d.K * 2};
    const uint32_t b[3] = {64, box_rows, 1};
    return encode_map(m, d.dtype, w, 3, dim, st, b);
}
// W [E, 2, I / 16, 16, K] as tiles of 64 gate and 64 up rows in turns of 16.
bool map_w_gated(CUtensorMap* m, const moe_linear_dims& d, const void* w) {
    const uint64_t K = d.K, I = d.N / 2;
    const uint64_t dim[5] = {K, 16, 2, I / 16, (uint64_t)d.E}, st[4] = {K * 2, I * K * 2, 16 * K * 2, 2 * I * K * 2};
    const uint32_t b[5] = {64, 16, 2, 4, 1};
    return encode_map(m, d.dtype, w, 5, dim, st, b);
}

LinView view_of(const LinearArgs& a) {
    LinView v = {};
    v.offsets = a.offsets;
    v.T = a.d.T;
    v.E = a.d.E;
    v.N = a.d.N;
    v.err = a.err;
    v.wait_ns = a.wait_ns;
    return v;
}

// Experts with rows, about.
int64_t groups_of(const LinearArgs& a) { return a.offsets ? (a.d.E < a.d.T ? a.d.E : a.d.T) : 1; }

// Whether the streaming kernel takes the call. One matrix: a single row always (2048 x 2048: 3.6 against 9 us, 8192 x 4096:
// 12.3 against 16.5); up to 8 while their sums, which grow with the rows, stay below the other kernel's start (2048 x 2048 by 4 rows 5.7
// against 9 us, by 8 rows 10.8 against 9.0; 8192 x 4096 by 4 rows 23 against 17). Rows of experts: each reads a matrix of
// its own, mostly, while they are no more than twice the experts (256 experts of 1024 x 2048 by 8 rows 7.2 against 17.5 us, by 64
// rows 39 against 46, by 128 rows 79 against 77; 8 experts of 2048 x 512 by 64 rows 15.7 against 7).
// (A test that holds back a stage needs a kernel that has stages.)
bool few_rows(const LinearArgs& a) {
    if (a.suppress) return false;
    if (a.offsets) return a.d.T <= kFewRows && a.d.T <= 2 * a.d.E;
    return a.d.T == 1 || (a.d.T <= 8 && (int64_t)a.d.T * a.d.N * a.d.K < 1 << 25);
}

template <typename T>
cudaError_t linear_t(const LinearArgs& a, cudaStream_t s) {
    const bool gated = a.d.act == MOE_ACT_SWIGLU;
    LinView v = view_of(a);
    v.bias = a.bias;
    v.residual = a.residual;
    v.out = a.out;
    v.z = a.z;
    v.F = gated ? a.d.N / 2 : a.d.N;
    v.C = a.d.K;
    v.act = a.d.act;
    v.suppress = a.suppress;
    cudaError_t e;
    if (few_rows(a)) {
        MOE_LAUNCH(MOE_KERNEL_LINEAR, s, (e = launch_few(a.d.dtype, gated, a.x, a.w, v, a.num_sms, s)));
        return e;
    }
    const int64_t g = groups_of(a), rows = (a.d.T + g - 1) / g;
    const int blocks = (v.C + 63) / 64;
    const bool ragged = a.offsets != nullptr;
    const LinPlan p = gated ? lin_plan<T, kFwd, true>(g, rows, ragged, a.d.N, blocks, a.num_sms) : lin_plan<T, kFwd, false>(g, rows, ragged, a.d.N, blocks, a.num_sms);
    v.boxes = pair_boxes(p, !a.offsets);
    CUtensorMap A, B;
    if (!(gated ? map_w_gated(&A, a.d, a.w) : map_w(&A, a.d, a.w, 128)) || !map_2d(&B, a.d.dtype, a.x, a.d.T, a.d.K, a.d.K, v.boxes))
        return cudaErrorInvalidValue;
    MOE_LAUNCH(MOE_KERNEL_LINEAR, s, (e = gated ? launch_plan<T, kFwd, true>(a.d.dtype, p, A, B, A, v, s) : launch_plan<T, kFwd, false>(a.d.dtype, p, A, B, A, v, s)));
    return e;
}

template <typename T, int VE, bool GATED>
cudaError_t launch_dz(const LinearArgs& a, int pitch, cudaStream_t s) {
    const int wide = GATED ? a.d.N / 2 : a.d.N;
    return launch_pdl(k_dz<T, VE, GATED>, dim3((a.d.T + a.chunk - 1) / a.chunk, (wide + 127) / 128), dim3(256), 0, s, a, pitch);
}

template <typename T>
cudaError_t linear_backward_t(const LinearArgs& in, cudaStream_t s) {
    LinearArgs a = in;
    const moe_linear_dims& d = a.d;
    const bool gated = d.act == MOE_ACT_SWIGLU, vec = d.N % 8 == 0 && (!gated || d.N % 16 == 0);
    int pitch = (d.N + 7) / 8 * 8;
    const bool plain = d.act == MOE_ACT_NONE && vec;  // dz is dout itself
    if (plain || (!a.dx && !a.dw)) a.dz = nullptr;
    cudaError_t e = cudaSuccess;
    // chunks of 128 rows where they still give every SM a CTA, else of 32 (the whole call: 16384 rows of 1024, K = 64, 61 against 79 us,
    // 2984 of 4868, K = 424, 64 against 71; 1024 of 1024 17.4 both)
    const int64_t strips = ((gated ? d.N / 2 : d.N) + 127) / 128;
    a.chunk = dz_rows(d.T, d.E);
    if (a.chunk == 32 && ((int64_t)d.T + 127) / 128 * strips >= a.num_sms) a.chunk = 128;
    if (a.dz || a.dbias) {
        MOE_LAUNCH(MOE_KERNEL_LINEAR_BACKWARD, s,
                   (e = gated ? launch_dz<T, 8, true>(a, pitch, s) : vec ? launch_dz<T, 8, false>(a, pitch, s) : launch_dz<T, 1, false>(a, pitch, s)));
        if (e != cudaSuccess) return e;
    }
    const void* dz = plain ? a.dout : a.dz;
    const int64_t g = groups_of(a);
    CUtensorMap A, B;
    LinView v = view_of(a);
    v.F = d.K;
    v.part = a.part;
    v.chunk = a.chunk;
    v.dbias = a.dbias;  // (the first of the products adds it up)
    if (a.dbias && !a.dx && !a.dw) {
        MOE_LAUNCH(MOE_KERNEL_LINEAR_BACKWARD, s, (e = launch_pdl(k_dbias<T>, dim3(a.num_sms), dim3(256), 0, s, v)));
        return e;
    }
    if (a.dx) {
        v.out = a.dx;
        v.C = d.N;
        const LinPlan p = lin_plan<T, kDx, false>(g, (d.T + g - 1) / g, a.offsets != nullptr, d.K, (v.C + 63) / 64, a.num_sms);
        v.boxes = pair_boxes(p, !a.offsets);
        if (!map_w(&A, d, a.w, 64) || !map_2d(&B, d.dtype, dz, d.T, d.N, pitch, v.boxes)) return cudaErrorInvalidValue;
        MOE_LAUNCH(MOE_KERNEL_LINEAR_BACKWARD, s, (e = launch_plan<T, kDx, false>(d.dtype, p, A, B, A, v, s)));
        if (e != cudaSuccess) return e;
        v.dbias = nullptr;
    }
    if (a.dw) {
        v.out = a.dw;
        v.C = 0;
        const LinPlan p = lin_plan<T, kDw, false>(d.E, d.N, false, d.K, (int)(((d.T + g - 1) / g + 63) / 64), a.num_sms);
        if (!(p.pair ? map_64(&A, d.dtype, a.x, d.T, d.K, d.K) && map_64(&B, d.dtype, dz, d.T, d.N, pitch)
                     : map_2d(&A, d.dtype, a.x, d.T, d.K, d.K, 64) && map_2d(&B, d.dtype, dz, d.T, d.N, pitch, 64)))
            return cudaErrorInvalidValue;
        CUtensorMap C = A;
        if (p.pair) {
            const uint64_t dim[3] = {(uint64_t)d.K, (uint64_t)d.N, (uint64_t)d.E}, st[2] = {(uint64_t)d.K * 2, (uint64_t)d.N * d.K * 2};
            const uint32_t box[3] = {32, 32, 1};
            if (!encode_map(&C, d.dtype, a.dw, 3, dim, st, box, true)) return cudaErrorInvalidValue;
        }
        MOE_LAUNCH(MOE_KERNEL_LINEAR_BACKWARD, s, (e = launch_plan<T, kDw, false>(d.dtype, p, A, B, C, v, s)));
    }
    return e;
}

}  // namespace

cudaError_t launch_linear(const LinearArgs& a, cudaStream_t s) {
    return a.d.dtype == MOE_FP16 ? linear_t<fp16>(a, s) : linear_t<bf16>(a, s);
}
cudaError_t launch_linear_backward(const LinearArgs& a, cudaStream_t s) {
    return a.d.dtype == MOE_FP16 ? linear_backward_t<fp16>(a, s) : linear_backward_t<bf16>(a, s);
}

}  // namespace moe
