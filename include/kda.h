/*
 * libkda — Kimi Delta Attention (KDA) hot path for GB300 (sm_103a).
 *
 * The operation (Kimi K3 technical-report walk-through, kimi-k3-paper.pages.dev):
 *   per (sequence, head), tokens t = 1..T, state S in R^{dk x dv} (rows = key channels)
 *     S_t = (I - beta_t k_t k_t^T) Diag(exp g_t) S_{t-1} + beta_t k_t v_t^T      (section 2.2, Eq. 1)
 *     o_t = S_t^T q_t                                                        (section 2.4, Eq. 3)
 *   with a channel-wise decay exp(g_t), g_t in (-5, 0] (sections 2.3 and 3.2, Eq. 5), and
 *   an optional epilogue y_t = o_t / sqrt(mean(o_t^2) + eps) * w * sigmoid(gate_t)
 *   (section 3.3, Eq. 6: head-wise RMSNorm, then the sigmoid output gate).
 *
 * General conventions for every entry point:
 *   - All tensor pointers are caller-owned DEVICE memory, dense, row-major, in the
 *     layouts stated per argument, and 16-byte aligned (KDA_ERR_INVALID_ARG otherwise;
 *     for decode only the state pool, v and the gate logits must be).  The library never allocates device memory and
 *     never frees anything it is given.
 *   - Calls are asynchronous on `stream` (a cudaStream_t passed as void*; NULL means
 *     the legacy default stream).  The call returns after validation and launch.
 *   - Argument errors are detected synchronously on the host: nothing is launched and
 *     the corresponding status is returned.  Conditions that only the device can see
 *     (an out-of-range slot index, inconsistent cu_seqlens, a device wait that ran out)
 *     are recorded in a per-device error word read by kda_get_device_error(); the
 *     affected rows are skipped, never trapped on.
 *   - dk, dv must each be 64 or 128 and, where there is a C, C must be 64 (KDA_ERR_UNSUPPORTED otherwise).
 *   - `dtype` is the element type of q, k, v and the gate logits; `out_dtype` that of out
 *     (either may be bf16 or fp32).  bf16 prefill inputs with dk = dv = 128 run on the tcgen05
 *     tensor-core path.  fp32 inputs, and bf16 inputs with dk or dv = 64, run on a path with
 *     fp32 arithmetic whose chunk products are three-term tf32 warp MMAs (fp32-level accuracy:
 *     about 3e-5 max|err|/RMS against an fp64 reference over 8192 tokens).  The read-out is
 *     computed in fp32 and rounded once when stored in out_dtype.
 *   - Value range of the bf16 tensor-core path (prefill with dk = dv = 128): the values, the
 *     intra-chunk terms built from them (beta v, U_hat = T V, U = U_hat - W S) and the running
 *     state (h0 included) enter fp16 tensor-core operands, so each of |beta v|, |h0| and the
 *     state's entries must stay below 65504 (keep them below ~1e4 for margin; accumulation is
 *     fp32).  Past it the operand becomes inf, which reaches out and the state; the state pass
 *     tests every final state it reaches (and each checkpoint) and sets KDA_DEVERR_NONFINITE (the
 *     results are not valid; nothing traps).  Non-finite inputs set it too.  Values far below 1 (under ~6e-5 relative to the state) lose precision as fp16
 *     subnormals.  The recurrence is linear in (v, h0) jointly, so a caller with larger or tiny
 *     values can scale v and h0 by one factor and divide out and hT by it.  Keys and queries
 *     (unit norm) and the decays need no such care.  The fp32 paths have fp32 range.
 *   - Debugging: with the environment variable KDA_DEBUG_CHECKS set (any value but "" or "0";
 *     read at every call), kda_chunk_fwd*, kda_chunk_fwd_segment_map and kda_decode_* first run
 *     a check kernel over the inputs and set KDA_DEVERR_PRECONDITION when g is outside (-5, 0],
 *     beta outside [0, 1], or (decode) two requests name the same slot; kda_linear_decode_step
 *     looks for such slots too.  The check reads every
 *     g and beta once (decode: O(N^2) slot comparisons); it is off by default.
 *   - Testing: with the environment variable KDA_TEST_WAIT_TIMEOUT set (any value but "" or "0";
 *     read at every call) the prefill, kda_matmul_fp8, kda_linear_chunk_fwd and the attentions launch kernel variants
 *     whose bounded waits on work of their own CTA give up at once, so that a test can make them run
 *     out and see KDA_DEVERR_WAIT_TIMEOUT reported with the device left usable.  With the value
 *     "stall" kda_matmul_fp8, kda_linear_chunk_fwd and the attentions launch variants whose first CTA starts no work,
 *     so that its waits run out at their limit, half a second to a second.  Not for production use.
 */
#ifndef KDA_H_
#define KDA_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  KDA_OK = 0,
  KDA_ERR_INVALID_ARG = 1,   /* null pointer, negative size, inconsistent sizes          */
  KDA_ERR_UNSUPPORTED = 2,   /* dk/dv not in {64,128}, C != 64, unknown dtype, no sm_103a */
  KDA_ERR_CUDA = 3,          /* a CUDA runtime call failed (launch, attribute, sync)      */
  KDA_ERR_DEVICE = 4,        /* the device error word is non-zero (kda_get_device_error)  */
  KDA_ERR_WORKSPACE = 5      /* workspace pointer NULL or smaller than required           */
} kda_status;

typedef enum {
  KDA_DTYPE_BF16 = 0,
  KDA_DTYPE_FP32 = 1
} kda_dtype;

/* Bits of the device error word. */
#define KDA_DEVERR_BAD_SLOT     0x1u  /* a slot index outside its pool, a block outside its cache */
#define KDA_DEVERR_BAD_SEQLENS  0x2u  /* prefill: cu_seqlens not non-decreasing in [0, T]  */
#define KDA_DEVERR_WAIT_TIMEOUT 0x4u  /* a bounded device-side wait gave up                */
#define KDA_DEVERR_BAD_COUNT    0x8u  /* a number of tokens outside what its call allows     */
#define KDA_DEVERR_NONFINITE   0x10u /* tensor-core path wrote a non-finite out / state value */
#define KDA_DEVERR_PRECONDITION 0x20u /* KDA_DEBUG_CHECKS: g, beta or slot_idx broke a precondition */
#define KDA_DEVERR_NO_BLOCKS   0x40u  /* block_tables: fewer free blocks than the new tokens need */

/* Optional fused epilogue (section 3.3, Eq. 6): RMSNorm over dv per (token, head), then
 * the sigmoid output gate.  The norm is taken on the fp32 read-out before rounding.
 *   gate_logits : [rows, H, dv] in the call's dtype (rows = T_tot or N)   — required
 *   norm_weight : [dv] fp32, shared by all heads; NULL means weight 1
 *   eps         : added to mean(o^2) before the square root (typical 1e-6) */
typedef struct {
  const void* gate_logits;
  const float* norm_weight;
  float eps;
} kda_epilogue;

/* Bytes of device scratch kda_chunk_fwd needs for this problem (0 on bad arguments).
 * T has the same meaning as in kda_chunk_fwd.  The scratch holds per-chunk operands
 * of the chunkwise form (~72.5 KB per 64-token chunk and head for bf16 at dk=dv=128)
 * plus a small plan. */
size_t kda_chunk_fwd_workspace_size(int B, int64_t T, int H, int dk, int dv, int C,
                                    kda_dtype dtype);

/* Chunked prefill over a packed batch of B variable-length sequences
 * (section 2.5, Eq. 4: serial inter-chunk state pass + parallel intra-chunk term).
 *   q, k      : [T_tot, H, dk]  (dtype)      L2-normalised upstream; not re-normalised
 *   v         : [T_tot, H, dv]  (dtype)
 *   g         : [T_tot, H, dk]  fp32         log-decay; precondition g in (-5, 0]
 *   beta      : [T_tot, H]      fp32         write strength, precondition in [0, 1]
 *   h0        : [B, H, dk, dv]  fp32 or NULL (zero initial states)
 *   cu_seqlens: [B+1] int32 device token offsets (cu[0] = 0, cu[B] = T_tot, non-decreasing),
 *               or NULL meaning B sequences of exactly T tokens each
 *   out       : [T_tot, H, dv]  (out_dtype)  must not alias any input
 *   hT        : [B, H, dk, dv]  fp32 or NULL (final states not written); may alias h0
 *   T         : tokens per sequence if cu_seqlens == NULL, else T_tot
 *   C         : chunk size, must be 64.  Chunks start at each sequence's first token.
 *   epi       : NULL or the fused epilogue
 *   workspace : device scratch of at least kda_chunk_fwd_workspace_size(...) bytes,
 *               256-byte aligned; contents on entry are ignored, on exit undefined.
 * Errors: KDA_ERR_INVALID_ARG / _UNSUPPORTED / _WORKSPACE before any launch; KDA_ERR_CUDA
 * if a launch fails.  Bad cu_seqlens set KDA_DEVERR_BAD_SEQLENS and the affected
 * sequences are skipped. */
kda_status kda_chunk_fwd(const void* q, const void* k, const void* v, const float* g,
                         const float* beta, const float* h0, const int32_t* cu_seqlens,
                         void* out, float* hT, int B, int64_t T, int H, int dk, int dv, int C,
                         kda_dtype dtype, kda_dtype out_dtype, const kda_epilogue* epi,
                         void* workspace, size_t workspace_bytes, void* stream);

/* kda_chunk_fwd that also stores intermediate states for a prefix cache (section 13.9: the KDA
 * path of the prefix cache can only resume at checkpoints stored at the 512-token hash-block
 * endpoints, i.e. ckpt_chunks = 8).  Sequence b stores its fp32 state after each
 * span = 64 * ckpt_chunks of its tokens: after tokens span, 2 span, ..., floor(len_b / span) span
 * (a checkpoint at the sequence end equals hT).
 *   states      : [n_ckpt, H, dk, dv] fp32 device, 16-byte aligned, written (not read), where
 *                 n_ckpt = sum_b floor(len_b / span); sequence b's checkpoints start at index
 *                 sum_{b' < b} floor(len_b' / span), in token order
 *   ckpt_chunks : >= 1
 * Every other argument, result and error is that of kda_chunk_fwd (states == NULL or
 * ckpt_chunks < 1: KDA_ERR_INVALID_ARG). */
kda_status kda_chunk_fwd_checkpoints(const void* q, const void* k, const void* v, const float* g,
                                     const float* beta, const float* h0, const int32_t* cu_seqlens,
                                     void* out, float* hT, float* states, int64_t ckpt_chunks, int B,
                                     int64_t T, int H, int dk, int dv, int C, kda_dtype dtype,
                                     kda_dtype out_dtype, const kda_epilogue* epi, void* workspace,
                                     size_t workspace_bytes, void* stream);

/* One recurrent decode step for N requests, one token each, on a pool of fp32 states
 * updated in place (section 13.9 prefix cache: one fixed-size state per request in a
 * pooled layout; section 13.10: state update and read-out in a single fused kernel).
 *   q, k       : [N, H, dk] (dtype);  v : [N, H, dv] (dtype)
 *   g          : [N, H, dk] fp32;     beta : [N, H] fp32
 *   state_pool : [num_slots, H, dk, dv] fp32, read and written in place
 *   slot_idx   : [N] int32 device; request n uses state_pool[slot_idx[n]].  Slots must be
 *                distinct (duplicates race; not checked).  An index outside
 *                [0, num_slots) sets KDA_DEVERR_BAD_SLOT and leaves that request's out rows
 *                and every slot untouched.
 *   out        : [N, H, dv] (out_dtype)
 * Slots not named in slot_idx are never read or written. */
kda_status kda_decode_step(const void* q, const void* k, const void* v, const float* g,
                           const float* beta, float* state_pool, const int32_t* slot_idx,
                           void* out, int N, int H, int dk, int dv, int num_slots,
                           kda_dtype dtype, kda_dtype out_dtype, const kda_epilogue* epi,
                           void* stream);

/* Several tokens per request on the pooled states: the verify and accept steps of speculative
 * decoding (section 13.4: an in-place update cannot be rolled back once a draft token is
 * rejected, so verification must leave the pooled state untouched and the accepted tokens are
 * applied afterwards from their cached inputs).
 *   q, k       : [N, n_tok, H, dk] (dtype);  v : [N, n_tok, H, dv] (dtype)
 *   g          : [N, n_tok, H, dk] fp32;     beta : [N, n_tok, H] fp32
 *   gate (epi) : [N, n_tok, H, dv] (dtype)
 *   state_pool, slot_idx : as for kda_decode_step
 *   ntok_per_req : device int32 [N], tokens to apply to request n (its first ntok_per_req[n]
 *                tokens, in order), or NULL meaning all n_tok.  A value outside [0, n_tok] sets
 *                KDA_DEVERR_BAD_COUNT and that request is skipped (out and state untouched).
 *   out        : [N, n_tok, H, dv] (out_dtype); rows of tokens not applied are not written
 *   commit     : 0 = verify: the pool is only read; 1 = accept: the state of each request after
 *                its applied tokens is written back to its slot (a request with 0 tokens keeps
 *                its state).  Token t of a request sees exactly the state after its tokens < t,
 *                so outputs of a verify call and of the accepting call agree on the tokens both
 *                apply.
 * kda_decode_step(...) is kda_decode_multi(..., ntok_per_req = NULL, N, n_tok = 1, ..., commit = 1). */
kda_status kda_decode_multi(const void* q, const void* k, const void* v, const float* g,
                            const float* beta, float* state_pool, const int32_t* slot_idx,
                            const int32_t* ntok_per_req, void* out, int N, int n_tok, int H, int dk,
                            int dv, int num_slots, int commit, kda_dtype dtype, kda_dtype out_dtype,
                            const kda_epilogue* epi, void* stream);

/* Backward of the prefill recurrence (no epilogue): the gradients of
 *   L = sum_t <dout_t, o_t> + <dhT, hT>
 * with respect to q, k, v, g, beta and h0 (section 2.2 Eq. 1, section 2.4 Eq. 3; section 5.1 names
 * a KDA training kernel), to fp32 accuracy.  Two paths give the same gradients within rounding:
 * the chunkwise reverse mode of the section 2.5 / Eq. 4 chunk form (per-chunk records, serial
 * state passes over chunks, per-chunk gradients, its products as tensor-core MMAs with a
 * three-term tf32 split; used while its scratch, about 0.6 MB per (chunk, head) at dk = dv = 128,
 * stays within 48 GB), else an fp32 reverse-time sweep over the tokens with the state recomputed
 * from per-chunk checkpoints.  The environment variable
 * KDA_BACKWARD_PATH=token or =chunked forces one of them; it is read at every call, including by
 * kda_chunk_bwd_workspace_size, so query the size under the same setting.
 *   q, k, v, g, beta, h0, cu_seqlens, B, T, H, dk, dv, dtype : as for kda_chunk_fwd
 *   dout       : [T_tot, H, dv] (dtype)
 *   dhT        : [B, H, dk, dv] fp32 or NULL (zero)
 *   dq, dk_, dg: [T_tot, H, dk] fp32;  dv_ : [T_tot, H, dv] fp32;  dbeta : [T_tot, H] fp32
 *   dh0        : [B, H, dk, dv] fp32 or NULL (not written)
 *   workspace  : at least kda_chunk_bwd_workspace_size(B, T, H, dk, dv) bytes, 256-byte aligned
 * Every pointer 16-byte aligned (beta, dbeta exempt).  Errors as for kda_chunk_fwd. */
size_t kda_chunk_bwd_workspace_size(int B, int64_t T, int H, int dk, int dv);
kda_status kda_chunk_bwd(const void* q, const void* k, const void* v, const float* g,
                         const float* beta, const float* h0, const int32_t* cu_seqlens,
                         const void* dout, const float* dhT, float* dq, float* dk_, float* dv_,
                         float* dg, float* dbeta, float* dh0, int B, int64_t T, int H, int dk,
                         int dv, kda_dtype dtype, void* workspace, size_t workspace_bytes,
                         void* stream);

/* Context parallelism across devices (section 13.3.2, KCP; open-day article section 5.2).  A long
 * sequence is split into consecutive token ranges, one per device.  Over a range the state pass is
 * affine in the range's initial state: S_out = P S_in + b, with P the range's accumulated transition
 * and b its final state from a zero initial state.  Each device computes the map of its range, the
 * devices exchange these fixed-size maps (an all-gather of H * (dk*dk + dk*dv) fp32 values each),
 * each folds the maps of the ranges before its own into its initial state with kda_state_compose,
 * then runs kda_chunk_fwd on its range from that state.
 *
 * kda_chunk_fwd_segment_map: the map (P, b) of one token range of one sequence, all H heads.
 *   k, v, g, beta : the range's tokens: [T, H, dk], [T, H, dv] (dtype), [T, H, dk] fp32, [T, H] fp32
 *                   (no q: the map does not depend on it)
 *   P             : [H, dk, dk] fp32, written: S_out = P S_in + b for every initial state S_in
 *   b             : [H, dk, dv] fp32, written: the range's final state from S_in = 0
 *   workspace     : at least kda_chunk_fwd_workspace_size(1, T, H, dk, dv, C, dtype) bytes, 256-byte
 *                   aligned
 * T = 0 gives P = I and b = 0.  Supported: bf16 inputs with dk = dv = 128 (else KDA_ERR_UNSUPPORTED).
 * The range runs as one serial pass per head (two runs: from 0 and, for P, from I).
 * Other errors as for kda_chunk_fwd. */
kda_status kda_chunk_fwd_segment_map(const void* k, const void* v, const float* g, const float* beta,
                                     float* P, float* b, int64_t T, int H, int dk, int dv, int C,
                                     kda_dtype dtype, void* workspace, size_t workspace_bytes,
                                     void* stream);

/* kda_state_compose: the initial state of the range that follows n ranges with maps (P[i], b[i]),
 *   S_out = P[n-1] ( ... (P[0] S0 + b[0]) ... ) + b[n-1],
 * in fp32 on the device.
 *   P     : [n, H, dk, dk] fp32;  b : [n, H, dk, dv] fp32   (maps in token order)
 *   S0    : [H, dk, dv] fp32, or NULL for a zero state;  S_out : [H, dk, dv] fp32, may alias S0
 * n = 0 copies S0 (or writes zeros).  dk, dv in {64, 128}; all pointers 16-byte aligned device
 * memory (KDA_ERR_INVALID_ARG otherwise). */
kda_status kda_state_compose(const float* P, const float* b, const float* S0, float* S_out, int n, int H,
                             int dk, int dv, void* stream);

/* ---- Operators around a recurrent layer (serving): the 8-bit projections and the plainer linear
 * attention that models mix with KDA.  A layer runs kda_rmsnorm_quant, kda_matmul_fp8 (q, k, v),
 * kda_linear_chunk_fwd or kda_linear_decode_step, kda_rmsnorm_quant and kda_matmul_fp8 (output). */

/* RMS norm with the residual's addition and an 8-bit output with scales, for a row of D values
 *   z = x + residual,  y_ = z / sqrt(mean(z^2) + eps) * weight
 *   per block of 128 values (the last of a row may be shorter):
 *     y_scale = max(max|y_|, 1e-30) / 448,   y = y_ / y_scale rounded to e4m3
 * so that y * y_scale approximates y_.  Sum, norm and scales are fp32; the norm is taken on the
 * unrounded sum z.  A NaN or infinity in a row reaches the row's scales.
 *   x            : [rows, D] (dtype)
 *   residual     : [rows, D] (dtype) or NULL (z = x)
 *   weight       : [D] fp32 or NULL (1)
 *   residual_out : [rows, D] (dtype) or NULL; z rounded to dtype.  May be residual or x (in place);
 *                  needs a residual
 *   y            : [rows, D] e4m3 (one byte per value), the layout kda_matmul_fp8 reads
 *   y_scale      : [rows, ceil(D / 128)] fp32
 *   D            : a multiple of 16, at most 32768 (KDA_ERR_UNSUPPORTED otherwise)
 * All pointers 16-byte aligned (y_scale: 4). */
kda_status kda_rmsnorm_quant(const void* x, const void* residual, const float* weight, void* residual_out,
                             void* y, float* y_scale, int64_t rows, int D, float eps, kda_dtype dtype,
                             void* stream);

/* Matrix product of e4m3 rows with a scale for each block of 128 values:
 *   out[m][n] = sum_kb a_scale[m][kb] * b_scale[n / 128][kb] * sum_{k in block kb} a[m][k] * b[n][k]
 *   a       : [M, K] e4m3,  a_scale : [M, ceil(K / 128)] fp32          (activations)
 *   b       : [N, K] e4m3,  b_scale : [ceil(N / 128), ceil(K / 128)] fp32  (a weight, 128 x 128 blocks)
 *   out     : [M, N] (out_dtype), rounded once from fp32 sums
 *   K       : a multiple of 16; K, M, N at most 2^22
 * a, b and out 16-byte aligned, the scales 4-byte aligned.  M = 0 does nothing. */
kda_status kda_matmul_fp8(const void* a, const float* a_scale, const void* b, const float* b_scale, void* out,
                          int64_t M, int N, int K, kda_dtype out_dtype, void* stream);

/* Linear attention with one decay per head over a packed batch of B variable-length sequences:
 *   S_t = e^{g_t} S_{t-1} + k_t v_t^T,   o_t = scale * S_t^T q_t
 * (section 2.2 Eq. 1 without the erase and with a scalar decay).
 *   q, k      : [T_tot, H, dk] (dtype);  v : [T_tot, H, dv] (dtype).  A token's heads are dense; the
 *               tokens lie q_stride / k_stride / v_stride elements apart (at least a dense row, a
 *               multiple of 16 bytes), so that they can be parts of one projection's rows
 *   g         : log decay, fp32: [T_tot, H] if g_per_token, else [H] (one constant per head).  g <= 0;
 *               -infinity empties the state
 *   h0        : [B, H, dk, dv] fp32 or NULL (zero);  hT : the same or NULL (not written); may alias h0
 *   cu_seqlens: as for kda_chunk_fwd.  Offsets that do not rise from 0 to T_tot set
 *               KDA_DEVERR_BAD_SEQLENS, and nothing is written
 *   B         : at most 16384
 *   out       : [T_tot, H, dv] (out_dtype), dense; must not overlap an input
 *   T         : as for kda_chunk_fwd; T_tot at most 2^31 - 1024
 *   workspace : at least kda_linear_chunk_fwd_workspace_size(...) bytes, 256-byte aligned
 * q, k, v and the states have to be finite (a chunk's values meet in tensor-core products, where an
 * infinity times a masked zero is NaN). */
size_t kda_linear_chunk_fwd_workspace_size(int B, int64_t T, int H, int dk, int dv, kda_dtype dtype);
kda_status kda_linear_chunk_fwd(const void* q, const void* k, const void* v, const float* g, int g_per_token,
                                const float* h0, const int32_t* cu_seqlens, void* out, float* hT, int B,
                                int64_t T, int H, int dk, int dv, int64_t q_stride, int64_t k_stride,
                                int64_t v_stride, float scale, kda_dtype dtype, kda_dtype out_dtype,
                                void* workspace, size_t workspace_bytes, void* stream);

/* One token of linear attention for N requests on a pool of fp32 states, updated in place.
 *   q, k, v   : [N, H, dk] / [N, H, dv] (dtype) with row strides as in kda_linear_chunk_fwd
 *   g         : [N, H] if g_per_token, else [H], fp32
 *   state_pool, slot_idx : as for kda_decode_step (finite states, distinct slots; a bad index sets
 *               KDA_DEVERR_BAD_SLOT and leaves that request's rows and every slot untouched)
 *   out       : [N, H, dv] (out_dtype), dense */
kda_status kda_linear_decode_step(const void* q, const void* k, const void* v, const float* g, int g_per_token,
                                  float* state_pool, const int32_t* slot_idx, void* out, int N, int H, int dk,
                                  int dv, int num_slots, int64_t q_stride, int64_t k_stride, int64_t v_stride,
                                  float scale, kda_dtype dtype, kda_dtype out_dtype, void* stream);

/* ---- An attention layer over a paged cache (serving), as models mix it with recurrent layers.  The cache is a pool
 * of blocks of block_size tokens (16, 32, 64, 128 or 256), for keys and for values:
 *   k_cache, v_cache : [num_blocks, block_size, Hkv, d] bf16.  The d values of a head are dense; blocks, tokens and
 *                      heads lie cache_strides[0], [1] and [2] elements apart (both caches alike; at least d, multiples of 8),
 *                      so a layout [num_blocks, Hkv, block_size, d] is one of strides
 *   block_tables     : [N, max_blocks] int32 device; token p of request n lies in block block_tables[n][p / block_size]
 *   d in {64, 128};  H a multiple of Hkv, H / Hkv at most 128 (KDA_ERR_UNSUPPORTED otherwise).
 * A step runs kda_block_tables (once for all layers), then in each layer kda_rope_append and one of the three
 * attentions, whose `lengths` are kda_block_tables' new lengths. */

/* Block tables, slots and positions of a step, from the tokens that each request gains or loses.
 *   counts       : [N] int32, tokens that request n gains (>= 0), or the number of its last tokens that it gives up (< 0;
 *                  a request ends by giving up all)
 *   lengths      : [N] int32, tokens of each request before the step;  new_lengths: [N] int32, after it; may be lengths
 *   block_tables : [N, max_blocks] int32, updated in place: entries of blocks that new tokens need are written, all
 *                  others are left as they are (those of blocks given back too)
 *   free_ring    : [num_blocks] int32, the free blocks as a ring: entries head, head + 1, .. (modulo num_blocks).  Blocks
 *                  are taken at the head, in order of the requests, and given back behind the last, likewise
 *   free_state   : [2] int32, head and number of free blocks;  new_free_state: the same after the step; may be free_state
 *   slot_map     : [T] int32, slots (block * block_size + place in it) of the new tokens, packed in order of the requests;
 *                  -1 behind the last
 *   positions    : [T] int32, their positions in their requests; 0 behind the last
 *   cu_seqlens   : [N + 1] int32, where each request's new tokens begin
 * Blocks given back in a step are not taken in the same one.  If a request's tokens would fall below 0 or pass
 * max_blocks * block_size, or all new tokens pass T, or a state is impossible (KDA_DEVERR_BAD_COUNT), or free blocks do not
 * suffice (KDA_DEVERR_NO_BLOCKS), the step does nothing: tables, ring, lengths and state stay or are copied, the
 * slots are all -1 and the offsets 0.  A block of the tables or the ring outside [0, num_blocks) sets
 * KDA_DEVERR_BAD_SLOT; its tokens get the slot -1.
 * N at most 8192, T at most 2^30; N * max_blocks and num_blocks * block_size below 2^31.  slot_map and positions
 * 16-byte aligned, the others 4.  No two arrays overlap but those named. */
kda_status kda_block_tables(const int32_t* counts, const int32_t* lengths, int32_t* block_tables, int32_t* free_ring,
                            const int32_t* free_state, int32_t* new_lengths, int32_t* new_free_state,
                            int32_t* slot_map, int32_t* positions, int32_t* cu_seqlens, int N, int max_blocks,
                            int num_blocks, int block_size, int64_t T, void* stream);

/* Rotary positions with one or several axes, and the cache's write.  For pair i of a head's first rot values
 *   angle = positions[axis[i]][t] * inv_freq[i],  (a, b) -> (a cos - b sin, b cos + a sin)
 * the pair being values i and i + rot / 2, or 2 i and 2 i + 1 if interleaved; values from rot on are left.  Whole
 * turns are taken off in 64-bit fixed point, so positions may be as far as int32 goes, and negative: the angle is off by
 * less than 2^-25 of a turn for |inv_freq| up to 64, beyond that by |inv_freq * position| 2^-64 turns more.
 *   q, k, v   : [T, H, d], [T, Hkv, d], [T, Hkv, d] (dtype), a token's heads dense, tokens q_stride / k_stride /
 *               v_stride elements apart (as in kda_linear_chunk_fwd)
 *   inv_freq  : [rot / 2] fp64, finite, radians for each position;  axis: [rot / 2] int32 in [0, axes), or NULL (all 0)
 *   positions : [axes, T] int32
 *   slot_map  : [T] int32, as from kda_block_tables: token t's keys and values go to slot slot_map[t].  A token with -1 is
 *               skipped whole (its row of q_out too); other slots outside the cache set KDA_DEVERR_BAD_SLOT and are
 *               skipped, as are the tokens of an axis outside [0, axes).  The slots are distinct
 *   q_out     : [T, H, d] bf16, dense;  computed in fp32 and rounded once, as what goes to the cache is
 *   rot       : a multiple of 16, at most d;  axes 1 to 4
 * q, k, v, the caches and q_out 16-byte aligned, inv_freq 8, the others 4.  Nothing written may overlap an input. */
kda_status kda_rope_append(const void* q, const void* k, const void* v, const double* inv_freq, const int32_t* axis,
                           const int32_t* positions, const int32_t* slot_map, void* q_out, void* k_cache, void* v_cache,
                           int64_t T, int H, int Hkv, int d, int rot, int axes, int interleaved, int64_t q_stride,
                           int64_t k_stride, int64_t v_stride, int num_blocks, int block_size,
                           const int64_t* cache_strides, kda_dtype dtype, void* stream);

/* Attention with a sliding window and sinks, for new tokens whose keys and values are in the cache already.  The token at
 * position p of its request sees the keys j <= p with j > p - window or j < sinks:
 *   out = sum_j softmax_j(scale q . k_j) v_j        (head h reads the cache's head h / (H / Hkv))
 *   q            : [T, H, d] bf16, a token's heads dense, tokens q_stride elements apart
 *   lengths      : [N] int32, tokens of request n in the cache, its new ones included
 *   cu_seqlens   : [N + 1] int32, where each request's new tokens begin in q; they are its last ones.  Offsets that do not
 *                  rise from 0 to at most T set KDA_DEVERR_BAD_SEQLENS, and nothing is written; a request of more new
 *                  tokens than its length, or longer than max_blocks * block_size or 2^24, sets it and is skipped (in all
 *                  three calls alike, whichever kernel their sizes lead to).  Rows of out behind the last request are
 *                  left as they were
 *   window       : tokens a token sees, itself included; 0 means all.  sinks >= 0: first tokens that stay visible
 *   max_length   : no request is longer (a hint for how the work is split; 0: as long as the tables allow)
 *   out          : [T, H, d] bf16, dense; must not overlap an input
 * Keys and values of tokens that a row sees have to be finite.  What lies in the cache elsewhere may be anything, and
 * table entries of blocks that no new token sees are not read.  A block that is, outside [0, num_blocks),
 * sets KDA_DEVERR_BAD_SLOT; the rows of its request are then undefined (nothing outside the cache is read).
 * The mean number of new tokens decides how the work is done, so prompts and single tokens are faster in calls of their own.
 * Scores, softmax and sums are fp32; the weights are rounded to bf16 for their product with the values. */
kda_status kda_window_attention_fwd(const void* q, const void* k_cache, const void* v_cache, const int32_t* block_tables,
                                    const int32_t* lengths, const int32_t* cu_seqlens, void* out, int N, int64_t T,
                                    int H, int Hkv, int d, int64_t q_stride, int num_blocks, int block_size,
                                    int max_blocks, const int64_t* cache_strides, int window, int sinks,
                                    int64_t max_length, float scale, void* stream);

/* The same for one new token of each request: q, out [N, H, d], request n's token being its last (position
 * lengths[n] - 1).  A request of length 0 gets zeros; one below 0 or longer than its table or 2^24 sets KDA_DEVERR_BAD_SEQLENS and
 * is skipped. */
kda_status kda_window_attention_decode_step(const void* q, const void* k_cache, const void* v_cache,
                                            const int32_t* block_tables, const int32_t* lengths, void* out, int N, int H,
                                            int Hkv, int d, int64_t q_stride, int num_blocks, int block_size,
                                            int max_blocks, const int64_t* cache_strides, int window, int sinks,
                                            int64_t max_length, float scale, void* stream);

/* Attention of drafted tokens that form a tree, over the cache: the verify step that goes with kda_decode_multi's.
 * A request's drafted tokens lie in the cache as its last cu_seqlens[n + 1] - cu_seqlens[n] ones, behind `before` others.
 *   tree_mask : [T, mask_words] 64-bit words: bit j % 64 of word j / 64 says that the token sees drafted token j of its
 *               request (its ancestors and itself; the mask alone decides); a request drafts at most 64 * mask_words
 *               tokens (KDA_DEVERR_BAD_COUNT, and it is skipped).  Bits past a request's drafted tokens are ignored
 * A token whose mask names m drafted tokens stands at position before + m - 1 and sees, of the tokens before the drafted
 * ones, what kda_window_attention_fwd shows it there.  A token that sees nothing gets zeros.  Drafted tokens that no mask
 * names (padding) may hold anything, as what lies elsewhere in the cache may.  kda_block_tables takes back a request's last
 * tokens: accepted tokens that are not the first drafted ones have to be taken back and run again.
 * mask_words 1 to 16; tree_mask 8-byte aligned.  All else as for kda_window_attention_fwd. */
kda_status kda_tree_attention(const void* q, const void* k_cache, const void* v_cache, const int32_t* block_tables,
                              const int32_t* lengths, const int32_t* cu_seqlens, const uint64_t* tree_mask, int mask_words,
                              void* out, int N, int64_t T, int H, int Hkv, int d, int64_t q_stride, int num_blocks,
                              int block_size, int max_blocks, const int64_t* cache_strides, int window, int sinks,
                              int64_t max_length, float scale, void* stream);

/* Synchronises `stream`, then reads and clears the current device's error word into
 * *flags (KDA_DEVERR_* bits).  Returns KDA_OK, or KDA_ERR_CUDA if the sync failed. */
kda_status kda_get_device_error(void* stream, uint32_t* flags);

/* Kernel-level timing for profilers; not needed for normal use.  While enabled, each
 * internal kernel launch made by kda_chunk_fwd / kda_decode_step is bracketed by two CUDA
 * events recorded on the call's stream (a few microseconds of host overhead per launch).
 * kda_trace_collect synchronises on those events and reports, per kernel name, the number
 * of launches and their summed device time in milliseconds since the previous collect:
 *   names    : caller buffer of max_entries * 64 bytes (NUL-terminated names)
 *   launches : [max_entries];  total_ms : [max_entries];  *n_entries : entries written
 * Both return KDA_ERR_CUDA if an event call fails.  Not thread-safe against concurrent
 * enable/disable; recording itself is serialised internally. */
kda_status kda_trace_enable(int enable);
kda_status kda_trace_collect(int max_entries, char* names, int* launches, double* total_ms,
                             int* n_entries);

/* kda_chunk_fwd for callers that cannot allocate device memory.  The method itself has
 * no counterpart to this: it is an interface variant for deployment.  Callers such as
 * code running under an allocator that owns all device memory, or hosts whose execution
 * path forbids cudaMalloc, cannot provide kda_chunk_fwd's workspace; this entry point
 * takes no workspace and allocates nothing (no cudaMalloc/cudaFree, no allocating
 * library call).  Its scratch is a fixed library-owned device array of
 * kda_noalloc_scratch_bytes() bytes (64 MiB), reserved on every device that loads the
 * library until the process exits.
 *   - Arguments, layouts, results and errors are those of kda_chunk_fwd.
 *   - Problems with kda_chunk_fwd_workspace_size(...) above the scratch size return
 *     KDA_ERR_WORKSPACE before any launch.
 *   - The first call on a device looks up the array's device address (cudaGetSymbolAddress);
 *     make that first call outside any stream capture.
 *   - All calls on a device share the one array and it keeps the last call's contents
 *     (nothing in it needs to start at zero).  Calls whose GPU work overlaps in time, e.g.
 *     on two unordered streams, race on it: order them. */
kda_status kda_chunk_fwd_noalloc(const void* q, const void* k, const void* v, const float* g,
                                 const float* beta, const float* h0, const int32_t* cu_seqlens,
                                 void* out, float* hT, int B, int64_t T, int H, int dk, int dv,
                                 int C, kda_dtype dtype, kda_dtype out_dtype,
                                 const kda_epilogue* epi, void* stream);

/* Size in bytes of the library-owned scratch used by kda_chunk_fwd_noalloc. */
size_t kda_noalloc_scratch_bytes(void);

/* Static, human-readable name of a status code. */
const char* kda_status_string(kda_status status);

#ifdef __cplusplus
}
#endif
#endif /* KDA_H_ */
