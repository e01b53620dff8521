/*
 * moe.h -- C ABI of the GB300 (sm_103a) sparse Mixture-of-Experts feed-forward layer.
 *
 * The layer (per token t, "Qwen3.6-35B-A3B -- Architecture Overview", MoE FFN: 256 Experts):
 *   l      = x[t] . Wr^T (+ br)                        router scores, fp32 accumulate
 *   p      = softmax(l)                                 over the E experts
 *   ids    = the K experts of highest p, slot 0 first; equal scores go to the lower index
 *   w_k    = p[ids_k] / sum_j p[ids_j]                  renormalised to sum to 1
 *   y      = sigmoid(x[t] . ws) * S(x[t]) + sum_k w_k * X_{ids_k}(x[t])
 *   out[t] = residual[t] + y                            (residual optional)
 * where every expert is a SwiGLU network X(x) = (SiLU(x . Wg^T) * (x . Wu^T)) . Wd^T
 * (same page, Experts and Shared Expert; "Qwen3.6 35B-A3B", Blocks: SparseMoe, SwiGlu).
 *
 * Data types and layouts (bf16 = IEEE bfloat16 bit patterns; all row-major, [Out, In]
 * like `Linear` in "Qwen3.6 35B-A3B", Blocks: Linear):
 *   x, residual, out  [T, H]        bf16
 *   router_w          [E, H]        bf16       router_b [E] bf16, optional
 *   gate_up           [E, 2I, H]    bf16       rows [0,I) of each expert = gate, [I,2I) = up
 *   down              [E, H, I]     bf16
 *   shared_gate_up    [2Is, H]      bf16       same split as gate_up
 *   shared_down       [H, Is]       bf16
 *   shared_gate       [1, H]        bf16       (no bias)
 *
 * Ownership and execution. The caller owns every buffer; all pointers are device pointers
 * (16-byte aligned) unless stated otherwise. The library allocates nothing on the call
 * path: scratch lives in a caller-provided device workspace of moe_workspace_size() bytes,
 * zero-filled once before its first use (moe_workspace_init does that); the library leaves
 * it ready for the next call. Calls are asynchronous on `stream` (a cudaStream_t; NULL is
 * the legacy default stream). Argument errors are detected on the host and returned before
 * anything is launched. A workspace must not be used by two calls that may overlap in time.
 * Weights are only read. A call may start reading them (never x, residual, out or the
 * workspace) while the kernel before it on `stream` is still finishing (programmatic
 * dependent launch), so that kernel must not be one that writes the weights: after writing
 * weights on `stream`, run any other work there, or synchronize, before the call.
 * One token at the pages' layer shape (H = 2048, I = Is = 512, T = 1) runs as one grid of one
 * CTA per SM whose CTAs exchange values with one another, so it needs every SM at once:
 * kernels on other streams that hold SMs longer than the wait limit (about 1 s) make the
 * call end with MOE_ERR_TIMEOUT in the workspace's error word rather than wait for them (two such
 * calls in flight on two streams can each hold SMs that the other needs: put them on one stream).
 * Results are deterministic: the same inputs give bit-identical outputs on every call.
 */
#ifndef MOE_GB300_H
#define MOE_GB300_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* Runtime dimensions: T tokens (B*S flattened; "Qwen3.6 35B-A3B", SparseMoe.forward takes
 * [B, S, H]), H hidden width, E routed experts, K experts per token, I routed inner width,
 * Is shared inner width. Supported: T >= 0, 128 <= H <= 8192 with H % 128 == 0,
 * 1 <= K <= 8, K <= E <= 256, 64 <= I, Is <= 2048 with I % 64 == 0 and Is % 64 == 0,
 * T * (K + 1) < 2^31. T == 0 is a valid no-op.
 * flags: 0, or MOE_FLAG_BF16_SCORES; any other bit is rejected with MOE_ERR_INVALID_ARG
 * before anything runs (moe_workspace_size ignores flags). */
typedef struct {
    int32_t T, H, E, K, I, Is;
    int32_t flags;
} moe_dims;

/* bf16-typed router outputs ("Qwen3.6 35B-A3B", Blocks: SparseMoe types `gate:
 * Linear<H, Experts, T>`, `shared_expert_gate: Linear<H, 1, T>` and `ranks(logits: Tensor[R,
 * Experts; T])` with T = bf16): each router score and the shared-gate score, accumulated in
 * fp32 with the bias added, is rounded to the nearest bf16 (ties to even) before the softmax,
 * the ranking and the sigmoid. Equal rounded scores rank the lower expert index first.
 * Without the flag the fp32 scores are used unrounded. */
#define MOE_FLAG_BF16_SCORES 1

/* Pointers to one layer's weights, in device memory (moe_forward_host_experts takes gate_up
 * and down in mapped host memory instead); router_b may be NULL. */
typedef struct {
    const void* router_w;
    const void* router_b;
    const void* gate_up;
    const void* down;
    const void* shared_gate_up;
    const void* shared_down;
    const void* shared_gate;
} moe_weights;

typedef enum {
    MOE_OK = 0,
    MOE_ERR_INVALID_ARG = 1,         /* NULL pointer or negative size                       */
    MOE_ERR_UNSUPPORTED_SHAPE = 2,   /* dims outside the supported range above              */
    MOE_ERR_MISALIGNED = 3,          /* a pointer is not 16-byte aligned                    */
    MOE_ERR_WORKSPACE_TOO_SMALL = 4, /* ws_bytes < moe_workspace_size(d)                    */
    MOE_ERR_CUDA = 5,                /* a CUDA launch or runtime call failed                */
    MOE_ERR_TIMEOUT = 6,             /* a bounded device-side wait gave up                  */
    MOE_ERR_DEVICE = 7               /* a kernel flagged bad data (a non-finite score, expert offsets out of order) */
} moe_status;

/* Bytes of device workspace that moe_route / moe_forward / moe_forward_w4 need for dims d (0 if
 * d is unsupported). Host-only; never fails otherwise. (At T = 1, and at K = 1 from 256 tokens,
 * the last part is used by moe_forward_w4 alone: the other calls accept a workspace without it.) */
size_t moe_workspace_size(const moe_dims* d);

/* Zero-fill a workspace on `stream` (cudaMemsetAsync). Needed once after allocation. */
moe_status moe_workspace_init(void* workspace, size_t ws_bytes, void* stream);

/* Routing only: router scores, softmax, top-K, renormalisation, and the dispatch of the
 * (token, slot) pairs to experts ("Qwen3.6-35B-A3B -- Architecture Overview", MoE FFN: 256
 * Experts, Router; "One Token Through Qwen3.6", The Router).
 *   x        [T, H] bf16 in
 *   ids      [T, K] int32 out: expert of each slot, slot 0 = highest score
 *   topk_w   [T, K] fp32  out: renormalised routing weights (sum to 1 per token)
 *   counts   [E]    int32 out: pairs routed to each expert
 *   offsets  [E+1]  int32 out: exclusive prefix sum of counts, offsets[E] = T*K
 *   perm     [T*K]  int32 out: values t*K+k grouped by expert (ascending), tokens
 *                              ascending within an expert
 * Integer outputs are exact and reproducible; topk_w is fp32. */
moe_status moe_route(const moe_dims* d, const void* x, const moe_weights* w, int32_t* ids, float* topk_w,
                     int32_t* counts, int32_t* offsets, int32_t* perm, void* workspace, size_t ws_bytes,
                     void* stream);

/* The whole layer: out = residual + MoE(x), or MoE(x) when residual is NULL. out must not
 * overlap x; it may be the same buffer as residual. Routed and shared expert outputs are
 * summed per token in a fixed order (residual, shared, slot 0 .. K-1) in fp32 and rounded
 * to bf16 once. */
moe_status moe_forward(const moe_dims* d, const void* x, const moe_weights* w, const void* residual, void* out,
                       void* workspace, size_t ws_bytes, void* stream);

/* The layer with its token rows in HOST memory (the decode loop's view: a token's hidden
 * state arrives from the host and the layer's output goes back to it). On `stream`, in this
 * order: host_x is copied into dev_x, host_residual (when not NULL) into dev_out, moe_forward
 * runs on (dev_x, dev_out as residual or none, dev_out), and dev_out is copied into host_out.
 * Up to 1 MB of rows (T*H*2 bytes) in pinned host memory mapped into the device move by a
 * small copy kernel (MOE_KERNEL_COPY_ROWS) over the host link; pageable or larger buffers by
 * cudaMemcpyAsync (pageable ones work, but the driver stages them and may block the calling
 * thread). One token at the shape moe_forward runs in its one-token kernel, with host_x,
 * host_out and host_residual (when given) all pinned, mapped and 16-byte aligned, takes one
 * launch and no copy: that kernel reads x and the residual and writes out on the host rows
 * themselves, and dev_x / dev_out are left as they were. host_out holds the result once
 * `stream` has passed the call.
 *   host_x, host_residual, host_out  [T, H] bf16, host memory (pinned or pageable);
 *                                    host_out may be the same buffer as host_x or host_residual
 *   dev_x, dev_out                   [T, H] bf16, device memory, 16-byte aligned, disjoint
 * Errors: MOE_ERR_INVALID_ARG when host_x or host_out is NULL, a host buffer is device memory
 * or dev_x / dev_out is not device memory (cudaPointerGetAttributes, before any copy);
 * otherwise as moe_forward with x = dev_x and out = dev_out. */
moe_status moe_forward_host_io(const moe_dims* d, const void* host_x, const moe_weights* w, const void* host_residual,
                               void* host_out, void* dev_x, void* dev_out, void* workspace, size_t ws_bytes,
                               void* stream);

/* Routed experts resident in host memory ("One Token Through Qwen3.6", Where the Weights
 * Live: checkpoint on disk, system RAM, GPU memory, kernels; the routing decides which expert
 * weights a layer needs). Same layer as moe_forward, but w->gate_up and w->down point to HOST
 * memory that is pinned and mapped into the device address space (cudaHostAlloc, or
 * cudaHostRegister with mapping); every other weight, x, out, residual and the workspace are
 * device memory as for moe_forward. After the routing, one kernel copies the gate_up and down
 * rows of the experts this call touches over the host link into `shadow`, device memory of
 * moe_expert_shadow_size(d) bytes laid out like [E, 2I, H] followed by [E, H, I] bf16 (only
 * the touched experts' rows are written; the rest is left as it was), and the experts run
 * from there. One shadow can serve every layer of a model in turn.
 * Errors: MOE_ERR_INVALID_ARG when gate_up or down is not registered host memory mapped into
 * the device (checked with cudaPointerGetAttributes before any launch), when the registered
 * allocation holding gate_up or down ends before the whole [E, 2I, H] or [E, H, I] tensor
 * (checked where the driver reports the allocation's range), or shadow is NULL,
 * MOE_ERR_MISALIGNED when shadow is not 16-byte aligned, MOE_ERR_WORKSPACE_TOO_SMALL when
 * shadow_bytes < moe_expert_shadow_size(d); otherwise as moe_forward. */
size_t moe_expert_shadow_size(const moe_dims* d);
moe_status moe_forward_host_experts(const moe_dims* d, const void* x, const moe_weights* w, const void* residual,
                                    void* out, void* shadow, size_t shadow_bytes, void* workspace, size_t ws_bytes,
                                    void* stream);

/* ---- 4-bit weights with group scales -------------------------------------------------------
 * The pages' layer reads its experts' weights from HBM once per step; in 4 bits they are 3.4 to
 * 3.9 times smaller. (The pages store bf16 only; this form of the weights has no counterpart.)
 * A matrix [rows, cols] (the [Out, In] layouts above) is held as one 4-bit code per weight and,
 * for every `group` consecutive columns of a row, a bf16 scale s:
 *   w[n, k] = s[n, k / group] * v,   v = code - 8       MOE_W4_INT4
 *                                    v = code - z       MOE_W4_INT4_ZP (z: the group's zero point, 0 .. 127)
 *                                    v = sign * {0, 0.5, 1, 1.5, 2, 3, 4, 6}[code & 7]  MOE_W4_E2M1
 *                                                       (sign: bit 3 of the code)
 * group is 32, 64 or 128 and divides cols.
 * Products use v exactly and apply the scale to each group's fp32 sum in fp32. The tensor-core
 * paths multiply by s * v rounded once to bf16 (INT4, INT4_ZP: below 2^-124 to a multiple of 2^-131,
 * as the rounding is of a quarter of it): the layer from 256 tokens; the linear layer where
 * ceil(T / 8) * ceil(N / 16) is more than 14 times the SMs times the waves (tiles of 128 tokens by
 * 256 rows, an SM each).
 * Packed form (moe_w4_size bytes, 16-byte aligned): matrices one after another, each a sequence
 * of strips of 16 rows (layout MOE_W4_ROWS: rows 16j .. 16j+15; MOE_W4_GATE_UP, for the merged
 * [2I, H] tensors: gate rows 8j .. 8j+7, then the matching up rows I+8j .. I+8j+7); a strip is a
 * sequence of records of 128 columns:
 *   1024 bytes of codes: little-endian 32-bit words [r / 8][r % 8][t][c] (r the strip row, t and
 *     c = 0 .. 3); a word holds columns 32c + 8t + e, e = 0 .. 7: even e in its low half, odd e in
 *     its high half, as the (e / 2)-th code of that half. INT4, INT4_ZP: code i in bits 4i .. 4i+3.
 *     E2M1: the sign bits of codes 0 .. 3 in bits 15, 12, 9, 14 and their other three bits, high to
 *     low, in bits (8, 7, 6), (5, 4, 3), (2, 1, 0), (13, 10, 11)
 *   16 x (128 / group) scales [r][group], bf16
 *   16 x (128 / group) zero points [r][group], bytes (INT4_ZP only)
 * Rows and columns past the matrix have codes of value 0, scale 0 and zero point 0. */
typedef enum { MOE_W4_INT4 = 0, MOE_W4_INT4_ZP = 1, MOE_W4_E2M1 = 2 } moe_w4_codes;
typedef enum { MOE_W4_ROWS = 0, MOE_W4_GATE_UP = 1 } moe_w4_layout;
typedef struct {
    int32_t format; /* moe_w4_codes */
    int32_t group;  /* columns to a scale: 32, 64 or 128 */
} moe_w4_format;

/* Bytes of n packed matrices [rows, cols]; 0 when the format or shape is not supported:
 * n >= 0, 1 <= rows <= 2^31 - 256, 32 <= cols <= 65536, cols % group == 0, rows * cols < 2^40 / max(n, 1). */
size_t moe_w4_size(const moe_w4_format* f, int32_t n, int32_t rows, int32_t cols);

/* Quantises n bf16 matrices w [n, rows, cols] into packed form. Per group, in fp32 with correctly
 * rounded divisions and ties to even:
 *   INT4     s = bf16(max|w| / 7), code = clamp(rint(w / s), -8, 7) + 8
 *   INT4_ZP  over the values and 0: s = bf16(max / 15 - min / 15), z = min(rint(-min / s), 15),
 *            code = clamp(rint(w / s) + z, 0, 15)
 *   E2M1     s = bf16(max|w| / 6), code = the nearest of the format's values to w / s
 * A group whose scale rounds to 0 is stored as zeros; one that holds a NaN or an infinity gets a
 * NaN scale, so every product with it is NaN. MOE_W4_GATE_UP needs rows % 16 == 0.
 * n = 0 is a no-op. Errors: MOE_ERR_INVALID_ARG (NULL, unknown format or layout, overlapping
 * buffers), MOE_ERR_UNSUPPORTED_SHAPE, MOE_ERR_MISALIGNED, MOE_ERR_WORKSPACE_TOO_SMALL when
 * packed_bytes < moe_w4_size. A product may follow on the same stream without any other work
 * between (these calls order their writes before the early reads described above). */
moe_status moe_w4_quantize(const moe_w4_format* f, int32_t n, int32_t rows, int32_t cols, int32_t layout, const void* w,
                           void* packed, size_t packed_bytes, void* stream);

/* Packs a checkpoint's codes: codes [n, rows, cols / 2] bytes (even column in the low nibble),
 * scales [n, rows, cols / group] bf16, zeros [n, rows, cols / group] bytes (INT4_ZP only, else
 * NULL; bit 7 is ignored). Otherwise as moe_w4_quantize. */
moe_status moe_w4_pack(const moe_w4_format* f, int32_t n, int32_t rows, int32_t cols, int32_t layout, const void* codes,
                       const void* scales, const void* zeros, void* packed, size_t packed_bytes, void* stream);

/* The weights a packed form stands for: w [n, rows, cols] bf16, s * v rounded once. (moe_forward on
 * w: after other work, as the ordering rule above asks of any kernel that writes weights.) */
moe_status moe_w4_dequantize(const moe_w4_format* f, int32_t n, int32_t rows, int32_t cols, int32_t layout,
                             const void* packed, size_t packed_bytes, void* w, void* stream);

/* Linear layer on packed weights (layout MOE_W4_ROWS, one matrix [N, K]):
 *   out[t, n] = bf16( sum_k x[t, k] * w[n, k] + bias[n] )      fp32 sums in a fixed order
 *   x [T, K], bias [N] or NULL, out [T, N], all bf16 (bias 2-byte aligned); out must not overlap x.
 * T = 0 is a no-op; T <= 2^31 - 256, T * N and T * K < 2^40. The workspace (moe_w4_linear_workspace_size bytes,
 * zero-filled once by moe_workspace_init) holds the error word of moe_last_device_error; calls
 * that may overlap in time need one each. x, bias, the weights and the workspace are read after
 * the previous kernel on `stream` is complete. */
size_t moe_w4_linear_workspace_size(const moe_w4_format* f, int32_t T, int32_t N, int32_t K);
moe_status moe_w4_linear(const moe_w4_format* f, int32_t T, int32_t N, int32_t K, const void* x, const void* packed,
                         size_t packed_bytes, const void* bias, void* out, void* workspace, size_t ws_bytes,
                         void* stream);

/* moe_forward with the experts' weights packed: w->gate_up (E matrices [2I, H]) and
 * w->shared_gate_up in layout MOE_W4_GATE_UP, w->down (E matrices [H, I]) and w->shared_down in
 * layout MOE_W4_ROWS, all in format f; router_w, router_b and shared_gate are bf16 as ever. Same
 * dims (with I and Is multiples of f->group), flags, workspace (moe_workspace_size), taps
 * (moe_w4_workspace_tap: tap 1 is fp32 for any T where K = 1) and errors as moe_forward. One token
 * (H <= 4096) runs as one grid of one CTA per SM whose CTAs exchange values, with the needs stated
 * above for that. */
moe_status moe_forward_w4(const moe_dims* d, const moe_w4_format* f, const void* x, const moe_weights* w,
                          const void* residual, void* out, void* workspace, size_t ws_bytes, void* stream);

/* RMSNorm of the pre-MoE norm ("RMSNorm -> MoE FFN -> +residual", "Qwen3.6-35B-A3B --
 * Architecture Overview", Stage 2; "Qwen3.6 35B-A3B", Blocks: RmsNorm):
 *   xn[t,h] = bf16( x[t,h] / sqrt(mean_h x[t,h]^2 + eps) * gamma[h] )   (fp32 arithmetic)
 * Uses d->T and d->H only. gamma [H] bf16 may be NULL (all ones). xn must not overlap x. */
moe_status moe_rmsnorm(const moe_dims* d, const void* x, const void* gamma, float eps, void* xn, void* stream);

/* ---- Parts of the layer, with gradients -----------------------------------------------------
 * The same layer put together from parts, for training and for experts of another kind: rows to
 * their experts and back, the experts' products, and the norms around the block (the pages describe
 * the forward layer alone; these have no counterpart there). All of them are asynchronous on
 * `stream`, read every argument after the previous kernel on it is complete, allocate nothing, and
 * give the same bits on every call. Tensors are contiguous, 16-byte aligned unless stated otherwise.
 * Results that a call does not name as optional are written in full; inputs are only read. */
typedef enum { MOE_BF16 = 0, MOE_FP16 = 1, MOE_FP32 = 2 } moe_dtype;
/* Activations. GELU is z * Phi(z), Phi the normal distribution function; SWIGLU is silu(gate) * up. */
typedef enum {
    MOE_ACT_NONE = 0, MOE_ACT_RELU = 1, MOE_ACT_SILU = 2, MOE_ACT_GELU = 3, MOE_ACT_SIGMOID = 4, MOE_ACT_SWIGLU = 5
} moe_act;

/* The dispatch of given expert ids [T, K] (moe_route's, or any other router's): a stable sort of the pairs
 * p = t*K + k by expert. An id outside [0, E) drops its slot.
 *   counts [E], offsets [E+1]  pairs of each expert and their exclusive prefix sum
 *   perm [T*K]                 pairs in order of (expert, t, k); -1 from offsets[E] on
 *   inv [T*K]                  place of pair p in perm; -1 for a dropped slot
 * For ids of moe_route, counts, offsets and perm are moe_route's. 1 <= K <= 8, 1 <= E <= 256, T * K <= 2^31 - 2^16;
 * T = 0 gives zeros. A token may name an expert twice. Errors: MOE_ERR_INVALID_ARG, MOE_ERR_UNSUPPORTED_SHAPE,
 * MOE_ERR_MISALIGNED. */
moe_status moe_sort_pairs(int32_t T, int32_t K, int32_t E, const int32_t* ids, int32_t* counts, int32_t* offsets,
                          int32_t* perm, int32_t* inv, void* stream);

/* Token rows to their experts and back, weights applied on either way, and the gradients. x, out, dout, dx,
 * residual are [T, H]; rows, drows [T*K, H] in the order of perm; topk_w, dtopk_w [T, K] fp32; inv of moe_sort_pairs.
 *   moe_dispatch           rows[inv[p]] = topk_w[p] * x[t]        (topk_w NULL: the rows as they are)
 *   moe_dispatch_backward  dx[t] = sum_k topk_w[p] * drows[inv[p]];  dtopk_w[p] = x[t] . drows[inv[p]]
 *   moe_combine            out[t] = residual[t] + sum_k topk_w[p] * rows[inv[p]]   (residual, topk_w optional)
 *   moe_combine_backward   drows[inv[p]] = topk_w[p] * dout[t];      dtopk_w[p] = dout[t] . rows[inv[p]]
 * (the gradient of residual is dout). dtopk_w is optional, and x and rows of the backward calls are read for it
 * alone (NULL without it). Dropped slots give and receive nothing: their dtopk_w is 0, and rows that no pair has as
 * its place are left as they were. Sums are in fp32 in slot order, the residual last, dots in fp32, each result rounded once.
 * out may be the same buffer as residual; otherwise results overlap no input. An entry of inv that is no place
 * in [0, T*K) counts as dropped. dtype: bf16, fp16 or fp32; 1 <= K <= 8, 1 <= H <= 65536, T * K <= 2^31 - 2^16;
 * rows move fastest where H elements are a multiple of 16 bytes (then of 8, of 4). T = 0 is a no-op. */
moe_status moe_dispatch(int32_t dtype, int32_t T, int32_t K, int32_t H, const void* x, const int32_t* inv,
                        const float* topk_w, void* rows, void* stream);
moe_status moe_dispatch_backward(int32_t dtype, int32_t T, int32_t K, int32_t H, const void* drows, const int32_t* inv,
                                 const float* topk_w, const void* x, void* dx, float* dtopk_w, void* stream);
moe_status moe_combine(int32_t dtype, int32_t T, int32_t K, int32_t H, const void* rows, const int32_t* inv,
                       const float* topk_w, const void* residual, void* out, void* stream);
moe_status moe_combine_backward(int32_t dtype, int32_t T, int32_t K, int32_t H, const void* dout, const int32_t* inv,
                                const float* topk_w, const void* rows, void* drows, float* dtopk_w, void* stream);

/* Linear layers with bias, activation and residual: one matrix for all T rows (E = 1, offsets NULL), or the
 * experts' products (offsets [E+1] of moe_route or moe_sort_pairs, on the device): rows offsets[e] ..
 * offsets[e+1] - 1 of x go through matrix e.
 *   z   = x . W_e^T + bias_e           x [T, K], w [E, N, K], bias [E, N] or NULL
 *   out = act(z) + residual            out, residual [T, No]: No = N, or N/2 for SWIGLU, whose W has the gate
 *                                      rows [0, N/2) and the up rows [N/2, N) of moe_weights' gate_up
 *   z [T, N] is stored too when z is not NULL (what the backward pass reads).
 * Backward, for dout [T, No] and the z of the forward pass (NULL when act is NONE):
 *   dz = act'(z) * dout;  dx = dz . W_e;  dw_e = dz^T . x and dbias_e = sum of dz, over expert e's rows
 * (zeros for an expert without rows); the gradient of residual is dout. Each of dx, dw, dbias is optional (NULL);
 * w is read for dx alone, x for dw alone. Rows from offsets[E] on are not read into any result and are left as they were
 * in out, z and dx.
 * dtype: bf16 or fp16, all tensors. Products accumulate in fp32, bias, activation and residual are applied in fp32,
 * results are rounded once; dz is rounded to dtype before the products of the backward pass (dbias sums it before).
 * Bounds: 1 <= N <= 2^20, 8 <= K <= 2^20 with K % 8 == 0, N % 32 == 0 for SWIGLU, 1 <= E <= 256, 0 <= T <= 2^31 - 2^16,
 * T*N, T*K, E*N*K < 2^40. bias and dbias are 2-byte aligned. out may be the same buffer as residual; otherwise results
 * overlap nothing. The workspace (moe_linear_workspace_size bytes; backward: nonzero for moe_linear_backward) is
 * zero-filled once (moe_workspace_init); calls that may overlap in time need one each. Offsets that
 * fall or leave [0, T] are cut to that range and set MOE_ERR_DEVICE for moe_last_device_error; waits that run out set
 * MOE_ERR_TIMEOUT. T = 0 is a no-op for moe_linear; moe_linear_backward then writes zeros to dw and dbias. */
typedef struct {
    int32_t T, N, K, E;
    int32_t act;   /* moe_act */
    int32_t dtype; /* moe_dtype: MOE_BF16 or MOE_FP16 */
} moe_linear_dims;
size_t moe_linear_workspace_size(const moe_linear_dims* d, int32_t backward);
moe_status moe_linear(const moe_linear_dims* d, const void* x, const void* w, const void* bias, const int32_t* offsets,
                      const void* residual, void* out, void* z, void* workspace, size_t ws_bytes, void* stream);
moe_status moe_linear_backward(const moe_linear_dims* d, const void* x, const void* w, const int32_t* offsets,
                               const void* z, const void* dout, void* dx, void* dw, void* dbias, void* workspace,
                               size_t ws_bytes, void* stream);

/* The norms before and after a block with its gate and residual scale: y is a block's output, residual the stream
 * it is added to, s the stream after it, xn what the next block reads. N(v; g) = v / sqrt(mean(v^2) + eps) * g.
 *   s  = residual_scale * residual + branch_scale * act(gate) * n,   n = N(y; gamma_post) with MOE_NORM_POST, else y
 *   xn = N(s; gamma_pre)                                             (of s before its rounding)
 * y, residual, s, xn [T, H]; gamma_post, gamma_pre [H] or NULL (ones); residual may be NULL (none), and s or xn,
 * not both. gate: none, one number a token [T], one a channel [H], or one an element [T, H]; gate_act NONE,
 * SIGMOID or SILU (of the gate).
 * Backward: ds and dxn are the gradients of s and xn (either may be NULL: none), s and y the forward pass's (s is read
 * for dxn alone). Results, each optional: dresidual, dy [T, H], dgate (as gate), dgamma_post, dgamma_pre [H].
 * dgamma_pre needs dxn, dgamma_post MOE_NORM_POST, dgate a gate.
 * dtype: bf16, fp16 or fp32, all tensors; arithmetic and sums in fp32, one rounding a result. 1 <= H <= 8192,
 * 0 <= T <= 2^31 - 2^16.
 * s and xn may be the buffers of y or residual (and dresidual and dy those of ds, dxn, s or y), each as a whole; results
 * overlap nothing else. The backward workspace (moe_norm_workspace_size bytes) need not be zero-filled; calls
 * that may overlap in time need one each. T = 0 is a no-op, or writes zeros to the [H] gradients. */
typedef enum { MOE_GATE_NONE = 0, MOE_GATE_TOKEN = 1, MOE_GATE_CHANNEL = 2, MOE_GATE_FULL = 3 } moe_gate;
#define MOE_NORM_POST 1
typedef struct {
    int32_t T, H;
    int32_t dtype;    /* moe_dtype */
    int32_t gate;     /* moe_gate */
    int32_t gate_act; /* moe_act */
    int32_t flags;    /* 0 or MOE_NORM_POST */
    float eps, branch_scale, residual_scale;
} moe_norm_dims;
size_t moe_norm_workspace_size(const moe_norm_dims* d);
moe_status moe_norm_residual(const moe_norm_dims* d, const void* y, const void* residual, const void* gate,
                             const void* gamma_post, const void* gamma_pre, void* s, void* xn, void* stream);
moe_status moe_norm_residual_backward(const moe_norm_dims* d, const void* ds, const void* dxn, const void* s,
                                      const void* y, const void* gate, const void* gamma_post, const void* gamma_pre,
                                      void* dresidual, void* dy, void* dgate, void* dgamma_post, void* dgamma_pre,
                                      void* workspace, size_t ws_bytes, void* stream);

/* Synchronise `stream`, then read and clear the device error word kept in `workspace`:
 * MOE_OK, MOE_ERR_DEVICE (a kernel saw a non-finite router score, or expert offsets out of order) or MOE_ERR_TIMEOUT. */
moe_status moe_last_device_error(void* workspace, void* stream);

/* Where an intermediate lives in the workspace after moe_forward (for inspection):
 *   tap 0  h      [T*K + T, max(I,Is)] bf16: gated activations, routed rows in perm order
 *                                             then the T shared-expert rows in token order
 *   tap 1  Y      [T, K+1, H] weighted expert outputs per slot, slot K = shared; fp32
 *                 when T < 256 (weight-streaming path), bf16 from T >= 256 (tensor-core
 *                 path): bytes / (T*(K+1)*H) tells which
 *   tap 2  sgate  [T] fp32: sigmoid(x . ws)
 *   tap 3  ids    [T, K] int32      tap 4  topk_w [T, K] fp32
 * Row strides are the widths given. Returns MOE_ERR_INVALID_ARG for an unknown tap. */
moe_status moe_workspace_tap(const moe_dims* d, int tap, size_t* offset, size_t* bytes);

/* The same after moe_forward_w4. Only tap 1 differs, and only where K = 1 and T >= 256: fp32, with
 * the bytes of that. */
moe_status moe_w4_workspace_tap(const moe_dims* d, int tap, size_t* offset, size_t* bytes);

/* Load-balancing statistics of one routing call ("Qwen3.6-35B-A3B -- Architecture Overview",
 * MoE FFN: 256 Experts, Load Balancing: an auxiliary loss, coefficient 0.001, penalises uneven
 * expert utilisation across the batch). The page gives no formula; this computes, for the T
 * tokens of x, the quantities such a loss is built from and the product form that is
 * smallest under uniform routing:
 *   P[e] = (1/T) sum_t softmax(router scores of token t)[e]   (full softmax over the E scores)
 *   f[e] = (tokens routed to expert e) / (T*K)
 *   loss = 0.001 * E * sum_e f[e] * P[e]
 * P, f: [E] fp32; loss: one fp32; all device pointers (P and f 16-byte aligned), owned by the
 * caller. The routing is the same as moe_route's (and it leaves the same results in the
 * workspace). Every sum runs in a fixed order, so repeated calls give identical bits.
 * T = 0 writes zeros. Errors as moe_route. */
moe_status moe_router_stats(const moe_dims* d, const void* x, const moe_weights* w, float* P, float* f, float* loss,
                            void* workspace, size_t ws_bytes, void* stream);

/* Kernels of the layer, for moe_set_trace. */
enum {
    MOE_KERNEL_ROUTER_SCORES = 0,   /* router + shared-gate scores                 */
    MOE_KERNEL_ROUTER_TOPK = 1,     /* softmax, top-K, renormalisation             */
    MOE_KERNEL_DISPATCH_LOCAL = 2,  /* per-block expert counts and ranks           */
    MOE_KERNEL_DISPATCH_SCAN = 3,   /* offsets and block bases                     */
    MOE_KERNEL_DISPATCH_SCATTER = 4,/* dispatch permutation                        */
    MOE_KERNEL_GATE_UP = 5,         /* gate/up projections + SwiGLU, all groups    */
    MOE_KERNEL_DOWN = 6,            /* down projection + routing-weight scale      */
    /* (from T >= 256 the router scores, gate_up and down run as tensor-core GEMMs) */
    MOE_KERNEL_COMBINE = 7,         /* fixed-order sum into the residual           */
    MOE_KERNEL_RMSNORM = 8,
    MOE_KERNEL_SHARED_GATE = 9,     /* not launched: the top-K kernel scores the shared gate */
    MOE_KERNEL_GATHER = 10,         /* not launched: the gate_up GEMM gathers the token rows from x */
    MOE_KERNEL_GEMM_PLAN = 11,      /* not launched: the dispatch scan writes the GEMM tables */
    MOE_KERNEL_DECODE_FUSED = 12,   /* whole layer in one persistent kernel (T = 1) */
    MOE_KERNEL_ROUTER_STATS = 13,   /* load-balancing statistics (moe_router_stats) */
    MOE_KERNEL_FETCH_EXPERTS = 14,  /* touched experts copied from host memory (moe_forward_host_experts) */
    MOE_KERNEL_COPY_ROWS = 15,      /* token rows to or from mapped host memory (moe_forward_host_io) */
    MOE_KERNEL_W4_PACK = 16,        /* quantising, packing, dequantising 4-bit weights */
    MOE_KERNEL_W4_LINEAR = 17,      /* moe_w4_linear                                */
    MOE_KERNEL_W4_FUSED = 18,       /* whole layer on 4-bit weights in one kernel (T = 1) */
    MOE_KERNEL_SORT_PAIRS = 19,     /* moe_sort_pairs                               */
    MOE_KERNEL_SPREAD_ROWS = 20,    /* moe_dispatch, moe_combine_backward           */
    MOE_KERNEL_GATHER_ROWS = 21,    /* moe_combine, moe_dispatch_backward           */
    MOE_KERNEL_LINEAR = 22,         /* moe_linear                                   */
    MOE_KERNEL_LINEAR_BACKWARD = 23,/* moe_linear_backward, all of its kernels      */
    MOE_KERNEL_NORM = 24,           /* moe_norm_residual                            */
    MOE_KERNEL_NORM_BACKWARD = 25,  /* moe_norm_residual_backward, both its kernels */
    MOE_KERNEL_COUNT = 26
};

/* Benchmarking aid. While set, every launch of `kernel` made by this library records
 * start_events[i] on its stream just before the launch and stop_events[i] just after it,
 * i = 0, 1, ... cycling modulo n_events (cudaEvent_t handles owned by the caller), so the
 * caller can read that kernel's duration with cudaEventElapsedTime. n_events = 0 clears it.
 * Process-wide state, not thread-safe; no effect on results. */
moe_status moe_set_trace(int kernel, void* const* start_events, void* const* stop_events, int n_events);

/* Number of kernels this library has launched in this process so far. */
uint64_t moe_launch_count(void);

/* Testing aid for the bounded-wait path (the paper has no counterpart). Every wait of the
 * one-token kernel (moe_forward with T = 1 at the page's layer shape) and of the streaming
 * expert kernels (2 <= T < 256), and every wait of the kernels on 4-bit weights and of moe_linear and
 * moe_linear_backward (there counted from the last 64-deep stage of operands that was worked off: a
 * call may last as long as it is), gives up after a time limit, sets MOE_ERR_TIMEOUT in the
 * workspace's error word and lets the kernel run to its end with in-range indices; the calls
 * after a timeout need moe_workspace_init on that workspace. This sets, process-wide and for
 * the calls made after it returns:
 *   wait_ns   the time limit of those waits in nanoseconds; 0 restores the default (~1 s);
 *             at most 10 s;
 *   suppress  0 in normal use, or one signal to hold back so that a wait runs out:
 *             MOE_TEST_SUPPRESS_SCORE  CTA 1 of the one-token kernels does not publish its
 *                                      router scores (every CTA's wait for the scores runs out);
 *             MOE_TEST_SUPPRESS_STAGE  CTA 0 of moe_forward's streaming gate_up kernel (9 <= T < 256)
 *                                      never loads its first ring stage (its consumers' wait
 *                                      on the stage's mbarrier runs out); nor does that of
 *                                      moe_linear's kernel.
 * Results of calls made while a signal is held back are meaningless; no call faults, traps or
 * hangs. Returns MOE_ERR_INVALID_ARG for another suppress value or wait_ns above 10 s. Not
 * thread-safe with concurrent calls of the library. */
#define MOE_TEST_SUPPRESS_SCORE 1
#define MOE_TEST_SUPPRESS_STAGE 2
moe_status moe_test_set_wait(uint64_t wait_ns, int suppress);

/* Routing without any device allocation by the caller (the paper has no counterpart: this is
 * for callers of this library that cannot call cudaMalloc, such as a plugin whose host
 * framework owns every device allocation, an engine that reserved all of HBM up front, or a
 * latency-critical path that cannot take an allocation's synchronisation or its failure).
 * Same inputs, outputs and results as moe_route, but no workspace: its scratch is a fixed
 * 80 KiB array inside the library, held by every GPU that loads the library until the
 * process exits. Limits: T <= 64 and the scratch layout must fit (any E <= 256, K <= 8 fit);
 * larger sizes return MOE_ERR_UNSUPPORTED_SHAPE before anything is launched.
 * The first call on a device looks up the array's device address on the current device
 * (cudaGetSymbolAddress); make that first call before any stream capture. The address is
 * kept per device and context: the first call after a reset of the device looks it up again. Every call shares
 * the one array: calls that may overlap on the GPU (different streams, or devices sharing it)
 * race and must be ordered by the caller. Each call clears the part that must start at zero.
 * A non-finite router score is not reported (there is no workspace error word). */
moe_status moe_route_noalloc(const moe_dims* d, const void* x, const moe_weights* w, int32_t* ids, float* topk_w,
                             int32_t* counts, int32_t* offsets, int32_t* perm, void* stream);

/* Human-readable name of a status. Never NULL. */
const char* moe_status_string(moe_status s);

#ifdef __cplusplus
}
#endif
#endif /* MOE_GB300_H */
