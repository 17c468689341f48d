/*
 * moe.h -- C ABI of libmoe_gb300: one top-k Mixture-of-Experts FFN layer with
 * SwiGLU experts, forward and backward, on one GB300 (sm_103a).  Dropless by
 * default; optionally with a per-expert capacity (token dropping) and, for the
 * dispatch step alone, a local expert range (the "scatter & drop" that follows
 * an all-gather of every token).
 *
 * The layer (sources named by page title and section):
 *   - a trainable gate scores every expert per token; the k experts with the
 *     highest probability are chosen and their outputs summed, weighted
 *     (DisagMoE, §2.1 "混合专家（MoE）结构");
 *   - token copies are sorted by expert, then by source, so that each expert's
 *     rows are contiguous (MegaScale-MoE research digest, §3.3 under Diagram C);
 *   - the experts are SwiGLU FFNs run together as one GroupedGEMM, "one kernel
 *     for the matrix products of several experts" (digest, glossary; MegaScale-
 *     MoE paper review, §三 核心公式 and 训练流程);
 *   - forward and backward are explicit operators, not autograd (digest §3.3);
 *   - load balance may drop tokens per GPU (digest §3.2, the paragraph after
 *     Figure 7), and the all-gather path of adaptive EP drops, locally, the
 *     tokens that no local expert takes (digest §3.2, Diagram B; review §四
 *     自适应EP通信策略详解, step 2).
 *
 * Conventions shared by every entry point
 *   - Pointers named x, Wg, W1 ... and every output are DEVICE pointers owned by
 *     the caller.  The library never allocates device memory and never frees
 *     any.  Scratch space is the caller's `ws` buffer of at least
 *     moe_workspace_bytes() bytes; the layer context is the caller's `saved`
 *     buffer of moe_saved_bytes() bytes.  Every pointer must be 16-byte
 *     aligned; ws and saved must be 256-byte aligned.
 *   - Calls are asynchronous on `stream` (0 = legacy default stream); the
 *     library never synchronises except in moe_read_device_status().
 *   - All matrices are row-major and dense:
 *       x, dy, y, dx : [T, h]   bf16        Wg, dWg : [h, E] fp32    b : [E] fp32
 *       W1, W3       : [E, h, f] bf16       W2      : [E, f, h] bf16
 *       dW1, dW3     : [E, h, f] fp32       dW2     : [E, f, h] fp32
 *       topk_idx     : [T, k] int32         gates   : [T, k] fp32
 *     An assignment a = t*k + j is token t's j-th chosen expert.  A permuted
 *     row p indexes the expert-major order: rows offsets[e] .. offsets[e+1]-1
 *     belong to expert e, in ascending a.
 *   - Token dropping (dims.capacity = C > 0): expert e takes only its first C
 *     assignments in ascending a; every other assignment is dropped.  A
 *     dropped assignment has perm_dst[a] = -1, adds nothing to y and gets no
 *     gradient through the experts (its gate gradient is 0); the gates are
 *     not renormalised.  Only the offsets[E] <= T*k placed rows exist: rows
 *     p >= offsets[E] of the permuted buffers are neither written nor read.
 *     C = 0 is dropless (offsets[E] = T*k).
 *   - Gradients are written, not accumulated.  An expert that receives no
 *     token gets zero weight gradients.
 *   - Argument errors are found on the host before any launch and returned as
 *     a status; nothing is launched then.  CUDA launch errors return
 *     MOE_ERR_CUDA.  Device code never traps or prints: a kernel whose bounded
 *     wait runs out records MOE_ERR_DEVICE_TIMEOUT in the status word at the
 *     start of `ws` and returns; moe_read_device_status() reports it.  A
 *     kernel that reads an index from device memory (an expert id in
 *     topk_idx, an entry of perm_src or perm_dst, an expert offset handed in
 *     by the caller) checks it: one out of range is recorded as
 *     MOE_ERR_DEVICE_INDEX in the same status word and that element is
 *     skipped (an assignment not placed, a zero row, a slot that adds
 *     nothing), so nothing is read or written out of bounds.  The calls that
 *     take no workspace (moe_combine, moe_unpermute, moe_quantize_rows_fp8,
 *     moe_quantize_rows_fp8_block, moe_permute_noalloc, moe_block_norm_fwd)
 *     record into one status word per device that the library keeps (its
 *     address is looked up on the first such call on a device and kept until
 *     the process exits); moe_read_device_status(NULL, stream) reports that
 *     one.
 *   - Supported shapes: 1 <= k <= 8, E <= 64, T*k < 2^31, h and f multiples
 *     of 64 (the GEMMs' K blocks are 64 wide).  Calls that choose experts
 *     (moe_route, moe_layer_fwd/bwd, moe_saved_bytes) also need k <= E; the
 *     others may run on a subset of the experts (E = a local expert count).
 */
#ifndef MOE_GB300_H
#define MOE_GB300_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef struct CUstream_st* moe_stream_t;   /* == cudaStream_t */
typedef struct CUevent_st* moe_event_t;     /* == cudaEvent_t */
typedef uint16_t moe_bf16;                  /* bf16 bit pattern */

typedef enum {
  MOE_OK = 0,
  MOE_ERR_INVALID_ARG = 1,     /* null/misaligned pointer, bad dimension */
  MOE_ERR_UNSUPPORTED = 2,     /* shape outside the supported set */
  MOE_ERR_WORKSPACE = 3,       /* ws_bytes smaller than required */
  MOE_ERR_CUDA = 4,            /* a CUDA runtime/driver call failed */
  MOE_ERR_DEVICE_TIMEOUT = 5,  /* a kernel's bounded wait ran out */
  MOE_ERR_DEVICE_INDEX = 6     /* an index read on the device was out of range */
} moe_status;

typedef struct {
  int32_t T;         /* tokens */
  int32_t h;         /* hidden size */
  int32_t f;         /* expert FFN width (h_ffn) */
  int32_t E;         /* experts */
  int32_t k;         /* experts per token */
  int32_t has_bias;  /* 1: router bias b[E] is added to the logits */
  int32_t capacity;  /* 0: dropless; C > 0: at most C assignments per expert */
  int32_t sar;       /* 1: selective activation rematerialisation (see below) */
} moe_dims;

typedef enum {
  MOE_OP_ROUTE = 0,
  MOE_OP_PERMUTE = 1,
  MOE_OP_EXPERT_FFN_FWD = 2,
  MOE_OP_EXPERT_FFN_BWD = 3,
  MOE_OP_ROUTER_BWD = 4,
  MOE_OP_LAYER_FWD = 5,
  MOE_OP_LAYER_BWD = 6,
  MOE_OP_LAYER_FWD_FP8 = 7,
  MOE_OP_LAYER_BWD_FP8 = 8,
  MOE_OP_LAYER_DECODE = 9,
  MOE_OP_LAYER_DECODE_FP8 = 10,
  MOE_OP_LAYER_FWD_FP8_BLOCK = 11,
  MOE_OP_LAYER_BWD_FP8_BLOCK = 12
} moe_op;

/* Per-expert capacity for a capacity factor: ceil(factor * T * k / E), the
 * share of the T*k assignments an expert gets under perfect balance times the
 * factor (the digest's per-GPU token dropping for load balance, §3.2 after
 * Figure 7; the factor is the usual way to size it).  Returns the value for
 * dims.capacity, or -1 when T < 0, k < 1, E < 1, factor <= 0 or the result
 * does not fit an int32. */
int32_t moe_capacity_for(int32_t T, int32_t k, int32_t E, double factor);

/* Scratch bytes entry point `op` needs for `dims` (0 on invalid dims).  The
 * first 256 bytes of every workspace hold the device status word; zero the
 * workspace once before first use (or call moe_clear_device_status). */
size_t moe_workspace_bytes(const moe_dims* dims, int op);

/* Bytes of the forward->backward context that moe_layer_fwd writes into
 * `saved` and moe_layer_bwd reads: routing, dispatch maps and activations.
 *   sar = 0: the permuted token rows x_perm and all four expert activations
 *            A = X W1, B = X W3, H = silu(A)*B, O = H W2; per layer
 *            (2k + 3k f/h) T h bf16 elements.
 *   sar = 1: selective activation rematerialisation (digest §3.3 "Inter-
 *            operator overlap"; review 选择性激活重计算): only A and B, i.e.
 *            2k (f/h) T h elements -- the pages' (2kf + ...) bsh/n after SAR,
 *            against (... 2k + 3kf ...) bsh/n before, at n = 1.  The backward
 *            gathers x_perm and dy again, rebuilds H from A and B inside the
 *            FC2 dgrad, and takes the gate gradient <dy, O> as <H, dy W2^T>
 *            (the same value), so O is never needed.  H, O and x_perm then live
 *            in the forward workspace, which is not kept between the calls. */
size_t moe_saved_bytes(const moe_dims* dims);

/* Router logits l = x Wg (+ b), softmax over the E experts, top-k selection
 * (descending logit, ties to the lower expert id) and renormalisation of the
 * k probabilities: gates[t,j] = p[e_j] / sum_j' p[e_j'].  DisagMoE §2.1.
 * In: x [T,h] bf16, Wg [h,E] fp32, b [E] fp32 (ignored unless has_bias).
 * Out: topk_idx [T,k] int32, gates [T,k] fp32.  Logits accumulate in fp32. */
moe_status moe_route(const moe_dims* dims, const moe_bf16* x, const float* Wg,
                     const float* b, int32_t* topk_idx, float* gates,
                     void* ws, size_t ws_bytes, moe_stream_t stream);

/* Dispatch: per-expert histogram, exclusive scan and the stable expert-major
 * permutation (digest §3.3: sorted by expert, then by source; review §四:
 * the scatter that makes each expert's tokens contiguous).  Deterministic,
 * no atomics.
 * In: topk_idx [T,k]; x [T,h] bf16 or NULL.
 * Out: counts [E], offsets [E+1] (offsets[E] = T*k when dropless), perm_src
 * [T*k] (permuted row -> assignment; the first offsets[E] entries are
 * written), perm_dst [T*k] (assignment -> permuted row, -1 if dropped), and,
 * when x and x_perm are both non-NULL, x_perm [T*k,h] with
 * x_perm[p] = x[perm_src[p] / k] for p < offsets[E]. */
moe_status moe_permute(const moe_dims* dims, const int32_t* topk_idx,
                       const moe_bf16* x, int32_t* counts, int32_t* offsets,
                       int32_t* perm_src, int32_t* perm_dst, moe_bf16* x_perm,
                       void* ws, size_t ws_bytes, moe_stream_t stream);

/* moe_permute with no workspace argument (the pages have no counterpart; this
 * is an interface convenience).  For callers that cannot allocate device
 * memory when they dispatch, such as a runtime that owns a fixed memory
 * budget.  Same arguments
 * and outputs as moe_permute minus ws/ws_bytes.  Its scratch is a 1 MiB array
 * in the library's device memory (held by every GPU that loads the library
 * until exit), so it supports ceil(T*k / 1024) * E <= 131072 and returns
 * MOE_ERR_UNSUPPORTED beyond that.  The first call on a device looks up the
 * array's device address (a host-side runtime query).  The address is kept
 * for the life of the process: after a cudaDeviceReset, restart the
 * process before calling this again.  All calls share the array: calls that
 * overlap on the GPU race.  Index errors (an expert id out of range) go to the
 * per-device status word of the calls without a workspace.  Allocates
 * nothing. */
moe_status moe_permute_noalloc(const moe_dims* dims, const int32_t* topk_idx,
                               const moe_bf16* x, int32_t* counts,
                               int32_t* offsets, int32_t* perm_src,
                               int32_t* perm_dst, moe_bf16* x_perm,
                               moe_stream_t stream);

/* The all-gather path's local "scatter & drop" (digest §3.2, Diagram B; review
 * §四 自适应EP通信策略详解, step 2): given every token's routing, place only the
 * assignments to the local experts e_lo <= e < e_hi (0 <= e_lo < e_hi <= E),
 * each expert taking at most dims.capacity of them when that is non-zero.
 * Same outputs as moe_permute over the EL = e_hi - e_lo local experts:
 * counts [EL], offsets [EL+1] (local expert i = global e_lo + i), perm_src
 * [T*k] (first offsets[EL] entries), perm_dst [T*k] (-1 for every assignment
 * not placed here), x_perm rows p < offsets[EL] when x and x_perm are given.
 * The local rows then run through moe_expert_ffn_fwd/bwd with dims.E = EL and
 * the local experts' weights; moe_combine with this perm_dst gives the local
 * experts' share of y (the partial sum the reduce-scatter adds up).
 * Workspace: moe_workspace_bytes(dims, MOE_OP_PERMUTE). */
moe_status moe_permute_local(const moe_dims* dims, const int32_t* topk_idx,
                             int32_t e_lo, int32_t e_hi, const moe_bf16* x,
                             int32_t* counts, int32_t* offsets,
                             int32_t* perm_src, int32_t* perm_dst,
                             moe_bf16* x_perm, void* ws, size_t ws_bytes,
                             moe_stream_t stream);

/* Inverse row move: rows_assign[a] = rows_perm[perm_dst[a]] for a < T*k, a
 * zero row where perm_dst[a] = -1.  rows_perm, rows_assign: [T*k, h] bf16.
 * It undoes the expert-major order of the dispatch (digest §3.3: token copies
 * sorted by expert, then by source), taking rows back to assignment order
 * a = t*k + j.  A perm_dst entry >= T*k gives a zero row and is recorded as
 * MOE_ERR_DEVICE_INDEX in the per-device status word (no workspace; see
 * moe_read_device_status). */
moe_status moe_unpermute(const moe_dims* dims, const int32_t* perm_dst,
                         const moe_bf16* rows_perm, moe_bf16* rows_assign,
                         moe_stream_t stream);

/* Expert SwiGLU FFN as GroupedGEMMs over the expert-contiguous rows:
 * for each e and rows p of e, with X[p] = x[perm_src[p] / k]:
 *   A = X W1[e],  B = X W3[e],  H = silu(A) * B,  O = H W2[e]
 * (review §三 核心公式: SwiGLU with MoE, 3k*bsh*h_ffn multiply-adds).
 * bf16 operands, fp32 accumulation in tensor memory; A, B, H, O stored bf16
 * [T*k, f] / [T*k, h], rows p < offsets[E] only.  offsets is read on the
 * device only. */
moe_status moe_expert_ffn_fwd(const moe_dims* dims, const moe_bf16* x,
                              const int32_t* perm_src, const int32_t* offsets,
                              const moe_bf16* W1, const moe_bf16* W3,
                              const moe_bf16* W2, moe_bf16* A, moe_bf16* B,
                              moe_bf16* H, moe_bf16* O,
                              void* ws, size_t ws_bytes, moe_stream_t stream);

/* Gate-weighted combine: y[t] = sum_{j<k} gates[t,j] * O[perm_dst[t*k+j]],
 * summed in fp32 in slot order, rounded once to bf16; slots with
 * perm_dst = -1 are skipped.  Deterministic (a gather, no scatter-add).
 * DisagMoE §2.1 (weighted sum). */
moe_status moe_combine(const moe_dims* dims, const moe_bf16* O,
                       const float* gates, const int32_t* perm_dst,
                       moe_bf16* y, moe_stream_t stream);

/* Backward of the expert FFN for the loss gradient dy [T,h]:
 *   dO[p] = gates[a] * dy[t]          (a = perm_src[p], t = a / k)
 *   dg[a] = <dy[t], O[p]>             (gradient of the gate, fp32 [T*k])
 *   dH = dO W2[e]^T ; dA = dH * B * s (1 + A (1 - s)), s = sigmoid(A) ;
 *   dB = dH * silu(A)
 *   dW2[e] = H_e^T dO_e ; dW1[e] = X_e^T dA_e ; dW3[e] = X_e^T dB_e
 *   dX_perm = dA W1[e]^T + dB W3[e]^T          (fp32 [T*k, h])
 * FC2's gradients take fc2_in = H and the gradient of fc2_out (review
 * 选择性激活重计算).  A, B, H, O are moe_expert_ffn_fwd's outputs.  Rows
 * p < offsets[E] only: dg[a] is written for the placed assignments
 * a = perm_src[p] alone, and so are the dX_perm rows. */
moe_status moe_expert_ffn_bwd(const moe_dims* dims, const moe_bf16* x,
                              const moe_bf16* dy, const float* gates,
                              const int32_t* perm_src, const int32_t* offsets,
                              const moe_bf16* W1, const moe_bf16* W3,
                              const moe_bf16* W2, const moe_bf16* A,
                              const moe_bf16* B, const moe_bf16* H,
                              const moe_bf16* O, float* dX_perm, float* dg,
                              float* dW1, float* dW3, float* dW2,
                              void* ws, size_t ws_bytes, moe_stream_t stream);

/* Router backward and the token gradient:
 *   dl[t,j] = g_j (dg_j - sum_i g_i dg_i)     (softmax over the k selected),
 *             evaluated as g_j sum_i g_i (dg_j - dg_i) since sum_i g_i = 1
 *   dx[t]   = sum_j dX_perm[perm_dst[t*k+j]] + sum_j dl[t,j] Wg[:, e_j]  (bf16)
 *   dWg     = x^T dl (fp32 [h,E]; a fixed-order two-level reduction)
 * In: x, Wg, topk_idx, gates, dg [T*k], dX_perm [T*k,h] fp32, perm_src,
 * perm_dst, offsets.  A slot with perm_dst = -1 counts with dg = 0 and adds
 * no dX_perm row. */
moe_status moe_router_bwd(const moe_dims* dims, const moe_bf16* x,
                          const float* Wg, const int32_t* topk_idx,
                          const float* gates, const float* dg,
                          const float* dX_perm, const int32_t* perm_src,
                          const int32_t* perm_dst, const int32_t* offsets,
                          moe_bf16* dx, float* dWg,
                          void* ws, size_t ws_bytes, moe_stream_t stream);

/* Whole layer forward: route, permute, expert FFN, combine.  Writes y [T,h]
 * and the context `saved` (moe_saved_bytes) for moe_layer_bwd. */
moe_status moe_layer_fwd(const moe_dims* dims, const moe_bf16* x,
                         const float* Wg, const float* b, const moe_bf16* W1,
                         const moe_bf16* W3, const moe_bf16* W2, moe_bf16* y,
                         void* saved, void* ws, size_t ws_bytes,
                         moe_stream_t stream);

/* ---------------------------------------------------------------- FP8
 * FP8 training with per-token quantisation instead of per-tensor (review §三
 * 创新点 "FP8训练优化"; digest §3.4).  The expert forward matmuls run on e4m3
 * codes (tcgen05 kind::f8f6f4) with float32 scales:
 *   activations x_perm and H: one scale per row, s = amax(|row|) / 448;
 *   weights: one scale per output column of each expert (amax over the
 *   contraction dimension);
 * q = e4m3(v / s) with an IEEE float32 division and round-to-nearest-even,
 * saturating at 448; s = 1 for an all-zero row or column.  The matmul sums
 * the exact code products in fp32 and multiplies by s_row * s_col.  H is
 * quantised from its bf16 copy.  The backward is the bf16 moe_layer_bwd on
 * the activations (A, B, H, O) this forward stores.  Requires h and f to be
 * multiples of 128 (MOE_ERR_UNSUPPORTED otherwise). */

/* Bytes of a quantised-weight buffer `qw` (0 on invalid or unsupported dims). */
size_t moe_fp8_weight_bytes(const moe_dims* dims);

/* Quantises the expert weights into `qw` (256-byte aligned, caller-owned):
 *   "W13q" [E, 2f, h] e4m3, K-major: per expert, 128-row groups alternating
 *          W1 columns and W3 columns (group 2j: W1[:, 128j + r], group 2j+1:
 *          W3[:, 128j + r], r < 128; each row holds the h codes of a column);
 *   "W2q"  [E, h, f] e4m3, K-major (row n holds the f codes of W2[:, n]);
 *   "s1", "s3" [E, f] and "s2" [E, h] float32 column scales.
 * Call it after every update of W1, W3, W2; moe_fp8_weight_view(name) gives
 * each part's device address. */
moe_status moe_quantize_weights_fp8(const moe_dims* dims, const moe_bf16* W1,
                                    const moe_bf16* W3, const moe_bf16* W2,
                                    void* qw, moe_stream_t stream);
void* moe_fp8_weight_view(const moe_dims* dims, void* qw, const char* name);

/* Row quantisation on its own: for p < rows, with src = idx[p] / div (or p
 * when idx is NULL; then src_rows >= rows), q[p, :] = e4m3(in[src, :] / s[p]),
 * s[p] = amax(|in[src, :]|) / 448.  in [src_rows, n] bf16, q [rows, n] bytes,
 * scale [rows] float32; n a multiple of 16. */
moe_status moe_quantize_rows_fp8(const moe_bf16* in, int64_t rows, int32_t n,
                                 const int32_t* idx, int32_t div,
                                 int64_t src_rows, uint8_t* q, float* scale,
                                 moe_stream_t stream);

/* moe_layer_fwd with the FP8 expert forward: route, dispatch, per-token
 * quantisation of the permuted rows, FC1 (+SwiGLU) on e4m3 codes, per-token
 * quantisation of H, FC2 on e4m3 codes, combine.  Weights come only from
 * `qw` (moe_quantize_weights_fp8).  Writes y and the same `saved` context as
 * moe_layer_fwd (A, B, H, O from the FP8 matmuls), for moe_layer_bwd.
 * dims.sar = 1 is MOE_ERR_UNSUPPORTED here: the sar backward takes the gate
 * gradient <dy, O> as <H, dy W2^T>, which needs O = H W2 exactly, and this
 * O comes from the e4m3 codes of H and W2.
 * Workspace: moe_workspace_bytes(dims, MOE_OP_LAYER_FWD_FP8). */
moe_status moe_layer_fwd_fp8(const moe_dims* dims, const moe_bf16* x,
                             const float* Wg, const float* b, const void* qw,
                             moe_bf16* y, void* saved, void* ws,
                             size_t ws_bytes, moe_stream_t stream);

/* FP8 data gradient of the backward, with the same per-token reading: the
 * FC1 dgrad dX = dA W1^T + dB W3^T runs on e4m3 codes as one contraction
 * over both halves, so a row of dA and the same row of dB share one scale
 * (their amax is recorded by the FC2 dgrad's epilogue) and row n of W1[e] and
 * row n of W3[e] share one.  FC2 dgrad stays bf16: its cost is the fused
 * SwiGLU backward in its epilogue, which e4m3 operands do not shorten
 * (measured).  The weight gradients stay bf16 matmuls on the bf16 dO, dA,
 * dB.  Requires h, f multiples of 128 and dims.sar = 0.
 *
 * moe_quantize_weights_fp8_bwd writes into `qwb` (256-byte aligned,
 * moe_fp8_bwd_weight_bytes): "W1r", "W3r" [E, h, f] e4m3 (row n of W1[e] and
 * of W3[e] with one shared scale) and "s13r" [E, h] float32;
 * moe_fp8_bwd_weight_view gives each part's address.  Call it after every
 * weight update. */
size_t moe_fp8_bwd_weight_bytes(const moe_dims* dims);
moe_status moe_quantize_weights_fp8_bwd(const moe_dims* dims,
                                        const moe_bf16* W1, const moe_bf16* W3,
                                        void* qwb, moe_stream_t stream);
void* moe_fp8_bwd_weight_view(const moe_dims* dims, void* qwb,
                              const char* name);

/* moe_layer_bwd with the FP8 FC1 data gradient above, from a `saved` context
 * of moe_layer_fwd or moe_layer_fwd_fp8 (sar = 0).  W2 (bf16) feeds the FC2
 * dgrad.  Same outputs as moe_layer_bwd.  Workspace:
 * moe_workspace_bytes(dims, MOE_OP_LAYER_BWD_FP8). */
moe_status moe_layer_bwd_fp8(const moe_dims* dims, const moe_bf16* x,
                             const moe_bf16* dy, const float* Wg,
                             const moe_bf16* W2, const void* qwb,
                             const void* saved, moe_bf16* dx, float* dWg,
                             float* dW1, float* dW3, float* dW2, void* ws,
                             size_t ws_bytes, moe_stream_t stream);

/* ---------------------------------------- e4m3 with a scale for each block
 * The fine-grained form of e4m3 training and serving: a float32 scale for each
 * 1 x 128 block of an activation's row and for each 128 x 128 block of a
 * weight.  Because a weight's block is square, one copy of its codes, in the
 * weight's own layout, serves the forward and the data gradients, and weights
 * that come with such scales are used as they are.
 *   s = amax(|block|) / 448 (IEEE float32 division; 1 for a block of zeros)
 *   q = e4m3(v / s)         (the float32 quotient, to nearest even, +-448 at most)
 * A block that holds an infinity or a NaN gets a scale that is not finite, and
 * so do the results that it enters.  A block at the end of an axis that is no
 * multiple of 128 is shorter.
 *   activations [R, n]: codes uint8 [R, n], scales float [ceil(n/128), R]:
 *                       the scales of block column b of all rows together
 *   weights [E, K, N]:  codes uint8 [E, K, N], scales
 *                       float [E, ceil(K/128), ceil(N/128)]
 * Products are summed block by block: the 128 products of a block in fp32 in
 * tensor memory, then times the product of both scales and added in fp32
 * registers.  Where the product of the scales leaves float32's normal range,
 * 2^-126 to 2^128, the block's sum loses digits or is not finite.
 * No output of these calls may overlap an input, another output or ws. */

/* Rows: as moe_quantize_rows_fp8 (source row idx[p] / div, or p when idx is
 * NULL), with one scale for each block: scale[b * rows + p] is that of
 * q[p, 128 b ...].  n a multiple of 16, at most 2^31 - 512.  A source index
 * out of range gives codes 0 with scales 1 and MOE_ERR_DEVICE_INDEX in the
 * per-device status word. */
moe_status moe_quantize_rows_fp8_block(const moe_bf16* in, int64_t rows,
                                       int32_t n, const int32_t* idx,
                                       int32_t div, int64_t src_rows,
                                       uint8_t* q, float* scale,
                                       moe_stream_t stream);

/* Weights W [E, K, N] (also a single matrix, E = 1): K and N multiples of 16,
 * at most 2^31 - 512, and fewer than 2^31 blocks of 128 x 128. */
moe_status moe_quantize_weights_fp8_block(const moe_bf16* W, int32_t E,
                                          int32_t K, int32_t N, uint8_t* q,
                                          float* scale, moe_stream_t stream);

typedef struct {
  int32_t rows;     /* rows of the activations, at most 2^31 - 512 */
  int32_t K;        /* contraction, a multiple of 16, at most 2^20 */
  int32_t N;        /* output columns, a multiple of 16, at most 2^20 */
  int32_t E;        /* groups of rows (experts), at most 64 */
  int32_t trans_b;  /* 0: weights [E, K, N]; 1: [E, N, K], used transposed */
  int32_t out_f32;  /* 0: C bf16; 1: C fp32 */
} moe_gemm_dims;

/* Scratch bytes of moe_gemm_fp8_block (0 on invalid dims).  They grow with
 * rows: a workspace for the most rows serves every smaller call of the same E. */
size_t moe_gemm_workspace_bytes(const moe_gemm_dims* dims);

/* C[p] = A[p] B[e] for the rows p of each group e, offsets[e] <= p <
 * offsets[e+1] (offsets [E+1] int32 on the device, from 0; NULL with E = 1: all
 * rows).  A: aq [rows, K] with sa [ceil(K/128), rows]; B: bq with sb as above;
 * C [rows, N].  Rows p >= offsets[E] are neither read nor written.  Offsets
 * out of order or range are clamped and recorded as MOE_ERR_DEVICE_INDEX in
 * the status word of ws.
 * The same inputs give the same bits.  Calls that may run at the same time need
 * a workspace each; the first 256 bytes of ws have to be zero before its first
 * use (every call leaves them so, but for the status word; after a wait that
 * ran out the call that reads MOE_ERR_DEVICE_TIMEOUT does). */
moe_status moe_gemm_fp8_block(const moe_gemm_dims* dims, const uint8_t* aq,
                              const float* sa, const uint8_t* bq,
                              const float* sb, const int32_t* offsets, void* C,
                              void* ws, size_t ws_bytes, moe_stream_t stream);

/* A gated feed-forward block on such weights: the experts of a layer on their
 * rows, or with E = 1 and offsets NULL one dense block (a shared expert) on
 * all rows.
 *   A = x W1, B = x W3, H = silu(A) * B, y = H W2
 * with W1, W3 [E, h, f] and W2 [E, f, h] as codes and scales.  x is quantised
 * in the call; both projections, the activation, the product and H's codes
 * (from its bf16 value) come from one kernel. */
typedef struct {
  int32_t rows;     /* at most 2^31 - 512 */
  int32_t h;        /* a multiple of 64, at most 2^20 */
  int32_t f;        /* a multiple of 64, at most 2^20 */
  int32_t E;        /* groups of rows (experts), at most 64 */
  int32_t dw_bf16;  /* type of the weight gradients: 0: fp32, 1: bf16 */
} moe_ffn_dims;

/* Scratch bytes of moe_gated_ffn_fwd (backward = 0) or moe_gated_ffn_bwd
 * (backward = 1); 0 on invalid dims.  They grow with rows: a workspace for the
 * most rows serves every smaller call of the same h, f and E. */
size_t moe_ffn_workspace_bytes(const moe_ffn_dims* dims, int backward);

/* x [rows, h] bf16 (rows of expert e at offsets[e] .. offsets[e+1]-1), y
 * [rows, h] bf16.  A, B, H [rows, f] bf16 are what the backward takes; all three
 * NULL where none follows.  Rows p >= offsets[E] are neither read nor
 * written.  Offsets and ws as in moe_gemm_fp8_block: with offsets out of order
 * the groups are those of the offsets clamped into order, in every step. */
moe_status moe_gated_ffn_fwd(const moe_ffn_dims* dims, const moe_bf16* x,
                             const int32_t* offsets, const uint8_t* W1q,
                             const float* s1, const uint8_t* W3q,
                             const float* s3, const uint8_t* W2q,
                             const float* s2, moe_bf16* A, moe_bf16* B,
                             moe_bf16* H, moe_bf16* y, void* ws,
                             size_t ws_bytes, moe_stream_t stream);

/* Its backward for dy [rows, h], from the forward's x, A, B, H:
 *   dH = dy W2^T;  dA = dH * B * s (1 + A (1 - s)), dB = dH * silu(A),
 *   s = sigmoid(A);  dx = dA W1^T + dB W3^T
 *   dW1[e] = x_e^T dA_e, dW3[e] = x_e^T dB_e, dW2[e] = H_e^T dy_e
 * The data gradients run on e4m3 codes (of dy, and of dA and dB from their
 * bf16 values), the weight gradients on the bf16 x, H, dy, dA, dB.  dx
 * [rows, h] bf16 (rows p >= offsets[E] untouched); dW1, dW3 [E, h, f], dW2
 * [E, f, h] fp32 or bf16 (dims.dw_bf16), written, not accumulated, zero for
 * an expert without rows; all three NULL for weights that are not trained.
 * Offsets and ws as in moe_gemm_fp8_block. */
moe_status moe_gated_ffn_bwd(const moe_ffn_dims* dims, const moe_bf16* x,
                             const moe_bf16* dy, const int32_t* offsets,
                             const uint8_t* W1q, const float* s1,
                             const uint8_t* W3q, const float* s3,
                             const uint8_t* W2q, const float* s2,
                             const moe_bf16* A, const moe_bf16* B,
                             const moe_bf16* H, moe_bf16* dx, void* dW1,
                             void* dW3, void* dW2, void* ws, size_t ws_bytes,
                             moe_stream_t stream);

/* moe_layer_fwd and moe_layer_bwd with the experts above.  The forward writes
 * the same `saved` context as moe_layer_fwd; the backward takes one from
 * either of the two.  h and f multiples of 64, at most 2^20; dims.sar = 1
 * and more than 2^31 - 512 assignments T*k are MOE_ERR_UNSUPPORTED.
 * Workspaces: moe_workspace_bytes with
 * MOE_OP_LAYER_FWD_FP8_BLOCK and MOE_OP_LAYER_BWD_FP8_BLOCK. */
moe_status moe_layer_fwd_fp8_block(const moe_dims* dims, const moe_bf16* x,
                                   const float* Wg, const float* b,
                                   const uint8_t* W1q, const float* s1,
                                   const uint8_t* W3q, const float* s3,
                                   const uint8_t* W2q, const float* s2,
                                   moe_bf16* y, void* saved, void* ws,
                                   size_t ws_bytes, moe_stream_t stream);
moe_status moe_layer_bwd_fp8_block(const moe_dims* dims, const moe_bf16* x,
                                   const moe_bf16* dy, const float* Wg,
                                   const uint8_t* W1q, const float* s1,
                                   const uint8_t* W3q, const float* s3,
                                   const uint8_t* W2q, const float* s2,
                                   const void* saved, moe_bf16* dx, float* dWg,
                                   float* dW1, float* dW3, float* dW2, void* ws,
                                   size_t ws_bytes, moe_stream_t stream);

/* ------------------------------------------------------- a few tokens
 * The whole layer for 1 <= T <= 128 tokens, as a serving loop calls it for the
 * next token of each of its sequences.  The same mathematics as
 * moe_layer_fwd:
 *   l = x Wg (+ b);  the k largest logits (ties to the lower expert id);
 *   gates = softmax over the chosen k;
 *   y[t] = sum_j gates[t,j] (silu(x W1[e_j]) * (x W3[e_j])) W2[e_j]
 * with fp32 sums throughout; H = silu(A) * B enters FC2 as the sum of two bf16
 * values (16 bits; a row that meets an infinite weight of W2 may get NaN for
 * an infinity); A, B, the experts' outputs and the gated sum stay in fp32 until
 * y is rounded.  Only the chosen experts' weights are read, each once.  Nothing
 * is kept for a backward pass.
 *
 * In: as moe_layer_fwd.  Out: y [T,h] bf16 and, where the pointers are not
 * NULL, topk_idx [T,k] and gates [T,k].  dims.capacity > 0 drops assignments
 * as moe_layer_fwd does.  Results do not depend on how blocks are scheduled:
 * the same inputs give the same bits.
 * MOE_ERR_UNSUPPORTED: T > 128, or dims.sar = 1 (there is no context).
 * Workspace: moe_workspace_bytes(dims, MOE_OP_LAYER_DECODE).  The blocks meet
 * at counters in its first 256 bytes: all of these have to be zero before the
 * first call (every call leaves them so, but for the status word), and calls
 * that may run at the same time need a workspace each.  Where that was not
 * so, results are undefined, within bounds: an expert id or row that cannot be
 * is recorded as MOE_ERR_DEVICE_INDEX, a meeting that fails as
 * MOE_ERR_DEVICE_TIMEOUT. */
moe_status moe_layer_decode(const moe_dims* dims, const moe_bf16* x,
                            const float* Wg, const float* b,
                            const moe_bf16* W1, const moe_bf16* W3,
                            const moe_bf16* W2, moe_bf16* y,
                            int32_t* topk_idx, float* gates, void* ws,
                            size_t ws_bytes, moe_stream_t stream);

/* moe_layer_decode on e4m3 weights: `qw` as moe_quantize_weights_fp8 writes it
 * (256-byte aligned).  x is quantised with one scale for each token, H (from
 * its bf16 value) with one for each row; the products of codes are summed in
 * fp32 and multiplied by the two scales.  The activations' scales are amax times
 * the fp32 reciprocal of 448, where moe_layer_fwd_fp8 divides.  The two are an
 * ulp apart, but a bf16 row holds values exactly between two codes, which
 * that ulp decides: y is up to 0.011 apart (relative L2, layers of a few hundred
 * rows and columns).  h and f multiples of 128 (MOE_ERR_UNSUPPORTED otherwise).
 * Workspace: moe_workspace_bytes(dims, MOE_OP_LAYER_DECODE_FP8). */
moe_status moe_layer_decode_fp8(const moe_dims* dims, const moe_bf16* x,
                                const float* Wg, const float* b,
                                const void* qw, moe_bf16* y,
                                int32_t* topk_idx, float* gates, void* ws,
                                size_t ws_bytes, moe_stream_t stream);

/* The same with the scales of moe_layer_fwd_fp8 (amax / 448, a float32
 * division), for a server whose prompts go through that call: x and H get its
 * codes, and what is left between the two is that it rounds O to bf16. */
moe_status moe_layer_decode_fp8_as_fwd(const moe_dims* dims, const moe_bf16* x,
                                       const float* Wg, const float* b,
                                       const void* qw, moe_bf16* y,
                                       int32_t* topk_idx, float* gates,
                                       void* ws, size_t ws_bytes,
                                       moe_stream_t stream);

/* ------------------------------------------------- norms around the block
 * What joins the layer to its residual stream r [T,h] (bf16, or fp32 with
 * res_f32): an RMS norm of the block's output y, a gate, the residual scales,
 * and the RMS norm that feeds the next block:
 *   z     = y / rms(y) * w_post          (z = y where w_post is NULL)
 *   r_out = alpha r + beta gate * z      (rounded once to r's type)
 *   u     = r_out / rms(r_out) * w_pre   (bf16; of the stored r_out)
 * with rms(v) = sqrt(mean(v^2) + eps) over a row, all in fp32.  gate: one
 * number for each channel (fp32 [h]), for each token (fp32 [T]), or none.
 * w_post, w_pre: fp32 [h]. */
typedef enum {
  MOE_GATE_NONE = 0,
  MOE_GATE_CHANNEL = 1,  /* gate [h] */
  MOE_GATE_TOKEN = 2     /* gate [T] */
} moe_gate_kind;

typedef struct {
  int32_t T;        /* rows */
  int32_t h;        /* row length: a multiple of 8, at most 8192 */
  int32_t res_f32;  /* 1: r, r_out, dr, dr_out are fp32; 0: bf16 */
  int32_t gate;     /* moe_gate_kind */
  float eps;        /* > 0 */
  float alpha;      /* scale of the residual */
  float beta;       /* scale of the block's output */
} moe_norm_dims;

/* Scratch bytes of moe_block_norm_bwd (0 on invalid dims).  They grow with T: a
 * workspace for the most rows serves every smaller call of the same h and
 * res_f32. */
size_t moe_norm_workspace_bytes(const moe_norm_dims* dims);

/* The forward above in one pass over r and y.
 *   y NULL:      the norm before the first block: u = r / rms(r) * w_pre only.
 *                w_post and r_out must be NULL; gate, alpha, beta are unused.
 *   w_pre NULL:  the end of the last block: r_out only; u must be NULL.
 * gate is unused with MOE_GATE_NONE.  r_out may be r itself. */
moe_status moe_block_norm_fwd(const moe_norm_dims* dims, const void* r,
                              const moe_bf16* y, const float* w_post,
                              const float* gate, const float* w_pre,
                              void* r_out, moe_bf16* u, moe_stream_t stream);

/* Its backward, from the gradients du of u and dr_out of r_out's other uses
 * (NULL: none) with the same optional parts as the forward call:
 *   G    = dr_out + J_pre^T (du * w_pre),  J_pre the Jacobian of r_out / rms
 *   dr   = alpha G;   dz = beta gate * G;  dy = J_post^T (dz * w_post)
 *   dw_pre [h] = sum_t du * r_out / rms;   dw_post [h] = sum_t dz * y / rms
 *   dgate = beta G * z, summed over t (channel) or over the row (token)
 * r_out is the stored output of the forward (r where y is NULL; then
 * dr = G, and dy, dw_post, dgate must be NULL); it may be NULL without w_pre.
 * Both row norms are computed again from r_out and y: nothing is kept from
 * the forward.  dr may be dr_out itself.  Gradients are written, not
 * accumulated, and every sum has a fixed order.
 * Workspace: moe_norm_workspace_bytes(dims), 256-byte aligned. */
moe_status moe_block_norm_bwd(const moe_norm_dims* dims, const void* r_out,
                              const moe_bf16* y, const float* w_post,
                              const float* gate, const float* w_pre,
                              const moe_bf16* du, const void* dr_out, void* dr,
                              moe_bf16* dy, float* dw_post, float* dgate,
                              float* dw_pre, void* ws, size_t ws_bytes,
                              moe_stream_t stream);

/* Whole layer backward from `saved`: writes dx [T,h] bf16 and the fp32
 * gradients dWg, dW1, dW3, dW2.  The router bias gets no gradient. */
moe_status moe_layer_bwd(const moe_dims* dims, const moe_bf16* x,
                         const moe_bf16* dy, const float* Wg,
                         const moe_bf16* W1, const moe_bf16* W3,
                         const moe_bf16* W2, const void* saved, moe_bf16* dx,
                         float* dWg, float* dW1, float* dW3, float* dW2,
                         void* ws, size_t ws_bytes, moe_stream_t stream);

/* Views into a `saved` context (device pointers at fixed offsets; NULL on
 * invalid dims, and for "x_perm", "H", "O" when dims.sar = 1).  Names:
 * "topk_idx", "gates", "counts", "offsets", "perm_src", "perm_dst",
 * "x_perm", "A", "B", "H", "O". */
void* moe_saved_view(const moe_dims* dims, void* saved, const char* name);

/* Human-readable name of a status. */
const char* moe_status_string(moe_status status);

/* Synchronises `stream`, returns the status word at the start of `ws` and
 * clears it; with MOE_ERR_DEVICE_TIMEOUT it zeroes the whole 256 bytes, where
 * kernels that gave up leave what they had counted.  ws = NULL: the status word of the calls that take no workspace
 * (moe_combine, moe_unpermute, moe_quantize_rows_fp8, moe_permute_noalloc,
 * moe_quantize_rows_fp8_block, moe_block_norm_fwd) on the current device.
 * MOE_ERR_CUDA if the synchronisation itself failed. */
moe_status moe_read_device_status(void* ws, moe_stream_t stream);

/* Zeroes the 256 bytes at the start of `ws`, the status word among them
 * (asynchronous); ws = NULL: the current device's status word of the calls without a workspace. */
moe_status moe_clear_device_status(void* ws, moe_stream_t stream);

/* Failure-path self test: launches one thread that waits on an mbarrier
 * nothing will complete, with the same bounded wait the matmul pipelines use
 * but a limit of limit_us microseconds (1 .. 1000000).  The wait gives up,
 * records MOE_ERR_DEVICE_TIMEOUT in the status word at the start of `ws` and
 * the kernel returns; the context stays usable.  No fault, trap or hang. */
moe_status moe_selftest_wait_timeout(void* ws, uint32_t limit_us, moe_stream_t stream);

/* Measurement hook: while `events` is non-NULL, every kernel the library
 * launches from this host thread is followed by cudaEventRecord of the next
 * event on the launching stream (up to `capacity`).  Pass NULL to stop; the
 * return value is the number of events recorded since the previous call.
 * moe_profile_kernel_name(i) names the kernel recorded by event i. */
int moe_profile_events(moe_event_t* events, int capacity);
const char* moe_profile_kernel_name(int i);

/* Number of CUDA kernels the library has launched from the calling host
 * thread since it was loaded (a named step of the measurement hook may launch
 * more than one kernel: the router and the router weight gradient run two). */
int64_t moe_kernel_launches(void);

/* Failure-injection hook for tests: the n-th kernel launch from now on the
 * calling host thread is reported as failed (cudaErrorLaunchFailure), so the
 * entry point that made it returns MOE_ERR_CUDA at that point without
 * launching the rest of its sequence.  The kernel itself runs normally and no
 * device state is touched: the failure exists only on the host.  n <= 0
 * clears a pending injection; the hook clears itself once it fires. */
void moe_test_fail_launch_after(int n);

/* Library build string (arch, version). */
const char* moe_version(void);

#ifdef __cplusplus
}
#endif

#endif /* MOE_GB300_H */
