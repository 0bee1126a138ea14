/*
 * gdn2.h -- C ABI of the MI355X (gfx950) Gated Delta Rule-2 token mixer.
 *
 * The operation. For every sequence n and head h, with state S (d_k x d_v, fp32) and for
 * each token t in order:
 *     alpha = exp(g_t)              per key channel, g_t = log(alpha_t) <= 0
 *     S_bar = Diag(alpha) S         decay along the key axis
 *     e = b_t * k_t,  z = w_t * v_t gated key (erase gate b, key side) and
 *                                   gated value (write gate w, value side)
 *     r = S_bar^T e                 old read with the gated key
 *     S = S_bar + k_t (z - r)^T     erase that read along k_t, write z along k_t
 *     o_t = S^T q_t                 readout from the updated state
 * This is the Gated Delta Rule-2 of "Gated DeltaNet-2: Decoupling Erase and Write in
 * Linear Attention" (reading note, §2 fast-weight objective and §3 forward pass; the
 * erase runs along k_t, as the objective's minimiser and the (I - k_t e_t^T) factor of
 * §3's backward paragraph fix). No query scale is applied: scale q beforehand if wanted.
 *
 * Conventions common to every entry point:
 *   - All tensor pointers are DEVICE pointers owned by the caller; the library never
 *     allocates, frees, synchronises, or keeps state between calls. Calls are
 *     asynchronous on `hip_stream` (a hipStream_t; NULL = the null stream).
 *   - Tensors are dense, row-major, contiguous, and 16-byte aligned.
 *   - `dtype` selects the element type of q, k, v, log_alpha, b, w and o:
 *     GDN2_BF16 (bfloat16) or GDN2_F32 (float). States are always fp32.
 *   - Arguments are validated on the host before any launch; on error nothing is
 *     launched and an error status is returned. Gate VALUES are not checked: b and w
 *     outside [0, 1] are computed as given.
 *   - Device faults surface at the caller's next synchronisation.
 *   - Numeric range: every forward entry point (chunked, training, decode) accepts any
 *     log_alpha <= 0, i.e. alpha anywhere in (0, 1], however strong the decay of a chunk
 *     or of a 16-token block; alpha below fp32 range acts as 0 (a full reset). The
 *     chunked backward has a limit of its own (see gdn2_chunk_bwd).
 */
#ifndef GDN2_H_
#define GDN2_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/*
 * Element type of q, k, v, the gates and o. Entry points take it as a plain int holding a
 * gdn2_dtype value, so that any other value is well defined on both sides of the boundary
 * and is rejected with GDN2_INVALID_ARGUMENT (an enum parameter may be assumed by the
 * compiler to hold only its enumerators, which would let it drop that check).
 */
typedef enum { GDN2_BF16 = 0, GDN2_F32 = 1 } gdn2_dtype;

enum {
  GDN2_OK = 0,
  GDN2_INVALID_ARGUMENT = 1, /* null required pointer, bad sizes, misaligned pointer */
  GDN2_UNSUPPORTED = 2,      /* head widths / dtype combination not built */
  GDN2_WORKSPACE_TOO_SMALL = 3, /* workspace_bytes below gdn2_chunk_fwd_workspace_bytes */
  GDN2_LAUNCH_FAILED = 4     /* the HIP runtime rejected a launch */
};

/*
 * Gate layouts for the *_ex entry points (bit set: that gate is one value per token and
 * head, shared by all of its channels, i.e. b = beta * 1 or w = omega * 1, the scalar-gate
 * configurations ablated in the reading note's §4). A scalar b is [..., H] in place of
 * [..., H, d_k]; a scalar w is [..., H] in place of [..., H, d_v]; same dtype, same leading
 * axes. The result equals the per-channel call with the gate broadcast over its channels.
 */
enum { GDN2_GATE_B_SCALAR = 1, GDN2_GATE_W_SCALAR = 2 };

/*
 * Chunkwise-parallel forward over whole sequences (the chunk form of the reading note's
 * §3 chunkwise-training paragraph: a per-channel cumulative decay normalises the state
 * inside a 64-token chunk, the chunk becomes an asymmetric delta recurrence, and the UT
 * transform of the Gated DeltaNet visual reading turns it into triangular-inverse and
 * matrix products). Result equals the token recurrence above up to rounding.
 *
 *   q, k, log_alpha, b : [B, T, H, d_k]   (dtype)
 *   v, w               : [B, T, H, d_v]   (dtype)
 *   initial_state      : [N, H, d_k, d_v] fp32, or NULL for a zero state
 *   o                  : [B, T, H, d_v]   (dtype), written
 *   final_state        : [N, H, d_k, d_v] fp32, or NULL (not written); may alias
 *                        initial_state (each state is read before it is overwritten)
 *   cu_seqlens         : NULL, or device int32 [N+1] offsets into the token axis of a
 *                        packed batch (then B must be 1 and T is the packed length).
 *                        Offsets must be non-decreasing with cu_seqlens[0] = 0 and
 *                        cu_seqlens[N] = T; the kernels clamp them into [0, T] so a bad
 *                        table cannot make them access memory out of bounds (its
 *                        results are then undefined).
 *   workspace          : NULL, or device scratch of at least
 *                        gdn2_chunk_fwd_workspace_bytes(...) bytes (16-byte aligned),
 *                        owned by the caller and free for the call's duration on
 *                        `hip_stream`. With a workspace the call runs the two-phase path:
 *                        one kernel computes every chunk's factors in parallel into the
 *                        workspace, a second walks the chunks of each sequence in order
 *                        (for fixed-length batches with fewer sequence x head chains than
 *                        compute units, each sequence is cut into segments that run in
 *                        parallel: a transfer pass, a scan of segment start states, then
 *                        the outputs). Without one, a single fused kernel does both per
 *                        sequence (for bf16 a kernel that prepares the next chunk's
 *                        operands while it finishes the current one).
 *                        Results agree to rounding. Ignored when
 *                        gdn2_chunk_fwd_workspace_bytes returns 0 for the dtype/widths.
 *   Without cu_seqlens, N must equal B and every sequence has length T.
 *   Supported: d_k, d_v in {64, 128} for both dtypes. GDN2_F32 runs without a workspace
 *   only: the chunk kernel for d_k = 64, and for d_k = 128, whose fp32 chunk operands do
 *   not fit the 160 KB of LDS, the token recurrence itself (one token at a time, fp32
 *   state in registers; exact to fp32 rounding, not chunk-parallel). T = 0 or N = 0 is a
 *   no-op (apart from final_state = initial).
 * Returns GDN2_OK or an error status (GDN2_WORKSPACE_TOO_SMALL when workspace_bytes is
 * below the requirement).
 */
int gdn2_chunk_fwd(const void* q, const void* k, const void* v, const void* log_alpha,
                   const void* b, const void* w, const float* initial_state, void* o,
                   float* final_state, const int32_t* cu_seqlens, int B, int T, int H,
                   int d_k, int d_v, int N, int dtype, void* workspace,
                   size_t workspace_bytes, void* hip_stream);

/*
 * gdn2_chunk_fwd with a gate layout (GDN2_GATE_* bits, 0 = per-channel gates as above):
 * scalar b and / or w are read as [B, T, H] (one value per token and head). Both the fused
 * path and the two-phase path (workspace given) support them. Any other bit gives
 * GDN2_INVALID_ARGUMENT.
 */
int gdn2_chunk_fwd_ex(const void* q, const void* k, const void* v, const void* log_alpha,
                      const void* b, const void* w, const float* initial_state, void* o,
                      float* final_state, const int32_t* cu_seqlens, int B, int T, int H,
                      int d_k, int d_v, int N, int dtype, int gate_layout, void* workspace,
                      size_t workspace_bytes, void* hip_stream);

/*
 * For callers that cannot allocate device memory (work under HIP stream capture, tight
 * serving loops, harnesses that forbid hipMalloc): gdn2_chunk_fwd_ex's two-phase path with
 * its workspace taken from a scratch array that the library holds on each device (a static
 * device array of gdn2_noalloc_scratch_bytes() = 128 MiB, resident from the library's load
 * on that device until the process ends). The call allocates and frees nothing; on its
 * first use on a device it looks up that device's scratch address (hipGetSymbolAddress).
 * The caller still passes every input and output, as for gdn2_chunk_fwd_ex (same
 * arguments without the workspace). Results equal gdn2_chunk_fwd_ex with a workspace.
 *   - Every call on one device shares that device's scratch: calls that may overlap on one
 *     device (different streams, or threads) race and must be serialised by the caller.
 *     The scratch keeps the last call's contents; nothing in it needs to start at zero.
 *   - Sizes whose workspace (gdn2_chunk_fwd_workspace_bytes for the same arguments,
 *     with or without cu_seqlens as given) exceeds the scratch give
 *     GDN2_WORKSPACE_TOO_SMALL and launch nothing; about 1.1 K tokens x heads fit per MiB
 *     at d_k = d_v = 128 (e.g. 4096 tokens x 16 heads in one sequence).
 *   - Built where the two-phase path is: GDN2_BF16 with d_k, d_v in {64, 128}
 *     (GDN2_UNSUPPORTED otherwise; the fused path of gdn2_chunk_fwd needs no workspace).
 */
int gdn2_chunk_fwd_noalloc(const void* q, const void* k, const void* v, const void* log_alpha,
                           const void* b, const void* w, const float* initial_state, void* o,
                           float* final_state, const int32_t* cu_seqlens, int B, int T, int H,
                           int d_k, int d_v, int N, int dtype, int gate_layout,
                           void* hip_stream);

/* Bytes of the per-device scratch array that gdn2_chunk_fwd_noalloc uses. */
size_t gdn2_noalloc_scratch_bytes(void);

/*
 * Device workspace, in bytes, that the two-phase path of gdn2_chunk_fwd needs for a call
 * with these sizes, with or without cu_seqlens (about 1.13 KiB per token and head at
 * d_k = d_v = 128, plus one chunk per sequence, plus (2 d_v + d_k) d_k fp32 per segment and
 * head when long sequences are cut into segments). 0 when the two-phase path is not built
 * for dtype / d_k / d_v (GDN2_BF16 with d_k, d_v in {64, 128} is) or a size is negative.
 */
size_t gdn2_chunk_fwd_workspace_bytes(int B, int T, int H, int d_k, int d_v, int N,
                                      int dtype);

/*
 * Chunkwise backward: gradients of gdn2_chunk_fwd for upstream gradients of o and of the
 * final states (the gate-aware backward of the reading note's §3: the state gradient flows
 * through the asymmetric factor Diag(alpha_t)(I - e_t k_t^T) of every token; here in chunk
 * form, with one triangular solve per chunk). Inputs and conventions as gdn2_chunk_fwd:
 *
 *   q, k, log_alpha, b, v, w, initial_state, cu_seqlens, B, T, H, d_k, d_v, N : as forward
 *   d_o               : [B, T, H, d_v] (dtype), gradient of o
 *   d_final_state     : [N, H, d_k, d_v] fp32, or NULL for zero
 *   dq, dk, dlog_alpha, db : [B, T, H, d_k] (dtype), written
 *   dv, dw            : [B, T, H, d_v] (dtype), written
 *   d_initial_state   : [N, H, d_k, d_v] fp32, or NULL (not written)
 *   range_flag        : NULL, or a device int32 that the caller clears beforehand. The call
 *                       sets it to 1 when some chunk's total decay, in some key channel,
 *                       exceeds the range of the local-gradient kernel's factors (referenced
 *                       to the middle of each channel's decay over the chunk: about 166 nats
 *                       over 64 tokens); a second kernel then recomputes those chunks'
 *                       gradients with exact pairwise decay factors, so the result is valid
 *                       for any decay either way. The second kernel reads the flag to skip
 *                       its scan when no chunk is out of range (with NULL it always scans).
 *   workspace         : required, at least gdn2_chunk_bwd_workspace_bytes(...) bytes, 16-byte
 *                       aligned, free for the call's duration on `hip_stream`.
 *   Supported: GDN2_BF16 with d_k, d_v in {64, 128}.
 * Returns GDN2_OK or an error status (GDN2_UNSUPPORTED for GDN2_F32,
 * GDN2_WORKSPACE_TOO_SMALL for a missing or short workspace).
 */
int gdn2_chunk_bwd(const void* q, const void* k, const void* v, const void* log_alpha,
                   const void* b, const void* w, const float* initial_state, const void* d_o,
                   const float* d_final_state, void* dq, void* dk, void* dv, void* dlog_alpha,
                   void* db, void* dw, float* d_initial_state, int32_t* range_flag,
                   const int32_t* cu_seqlens, int B, int T, int H, int d_k, int d_v, int N,
                   int dtype, void* workspace, size_t workspace_bytes, void* hip_stream);

/*
 * Device workspace, in bytes, that gdn2_chunk_bwd (and gdn2_chunk_fwd_train) needs for these
 * sizes, with or without cu_seqlens (about 3.7 KiB per token and head at d_k = d_v = 128, plus
 * one chunk per sequence, plus (2 d_v + d_k) d_k fp32 per segment and head when long
 * sequences are cut into segments, as for the two-phase forward); 0 where the backward is not
 * built.
 */
size_t gdn2_chunk_bwd_workspace_bytes(int B, int T, int H, int d_k, int d_v, int N,
                                      int dtype);

/*
 * gdn2_chunk_bwd with a gate layout (GDN2_GATE_* bits): a scalar b or w is read as
 * [B, T, H], and its gradient db or dw is written as [B, T, H] (the sum over the channels
 * of the per-channel gradient, since the one value is shared by all of them).
 */
int gdn2_chunk_bwd_ex(const void* q, const void* k, const void* v, const void* log_alpha,
                      const void* b, const void* w, const float* initial_state, const void* d_o,
                      const float* d_final_state, void* dq, void* dk, void* dv, void* dlog_alpha,
                      void* db, void* dw, float* d_initial_state, int32_t* range_flag,
                      const int32_t* cu_seqlens, int B, int T, int H, int d_k, int d_v, int N,
                      int dtype, int gate_layout, void* workspace, size_t workspace_bytes,
                      void* hip_stream);

/*
 * Training forward: the same result as gdn2_chunk_fwd (o, and the final state when
 * final_state is not NULL), computed by the two-phase kernels while the backward's
 * intermediates (the chunk factors, every chunk's entering state and U, and for a sequence
 * cut into segments each segment's linear map of the state) are kept in
 * `workspace`, so that gdn2_chunk_bwd_saved can skip the forward recomputation that
 * gdn2_chunk_bwd performs. Same arguments as gdn2_chunk_fwd, except that o is required and
 * workspace is required, of at least gdn2_chunk_bwd_workspace_bytes(...) bytes, and the
 * gate layout (GDN2_GATE_* bits, as for gdn2_chunk_fwd_ex) is given; bf16 only
 * (GDN2_UNSUPPORTED otherwise). The workspace stays owned by the caller and must not be
 * written until the matching gdn2_chunk_bwd_saved has run.
 */
int gdn2_chunk_fwd_train(const void* q, const void* k, const void* v, const void* log_alpha,
                         const void* b, const void* w, const float* initial_state, void* o,
                         float* final_state, const int32_t* cu_seqlens, int B, int T, int H,
                         int d_k, int d_v, int N, int dtype, int gate_layout, void* workspace,
                         size_t workspace_bytes, void* hip_stream);

/*
 * gdn2_chunk_bwd on a workspace written by gdn2_chunk_fwd_train with the same inputs,
 * initial state, cu_seqlens and sizes (the forward recomputation is skipped; nothing checks
 * that the workspace matches, and a mismatched one gives wrong gradients, never an
 * out-of-bounds access). The arguments of gdn2_chunk_bwd_ex, with its errors; the gate layout
 * must be the training forward's.
 */
int gdn2_chunk_bwd_saved(const void* q, const void* k, const void* v, const void* log_alpha,
                         const void* b, const void* w, const float* initial_state,
                         const void* d_o, const float* d_final_state, void* dq, void* dk,
                         void* dv, void* dlog_alpha, void* db, void* dw,
                         float* d_initial_state, int32_t* range_flag,
                         const int32_t* cu_seqlens, int B, int T, int H, int d_k, int d_v,
                         int N, int dtype, int gate_layout, void* workspace,
                         size_t workspace_bytes, void* hip_stream);

/*
 * The fused single-kernel path of gdn2_chunk_fwd (no workspace) with an explicit
 * value-slice width: each workgroup carries
 * `value_slice` columns of the state (16, 32, 64 or 128; a divisor of d_v; 16 only with
 * d_k = 64; at most 64 for GDN2_F32, whose d_k = 128 form has no slices). 0 selects the
 * width automatically, exactly as gdn2_chunk_fwd does. Results do not depend on the width
 * beyond rounding. Returns GDN2_UNSUPPORTED for a width that is not built.
 */
int gdn2_chunk_fwd_sliced(const void* q, const void* k, const void* v, const void* log_alpha,
                          const void* b, const void* w, const float* initial_state, void* o,
                          float* final_state, const int32_t* cu_seqlens, int B, int T, int H,
                          int d_k, int d_v, int N, int dtype, int value_slice,
                          void* hip_stream);

/*
 * One recurrent decode step for N independent sequences (the per-token procedure of
 * the reading note's §3 forward-pass paragraph; constant memory per token, the
 * abstract's decode property). The state is read once and written once in place; the
 * readout is formed from the old state as o = Diag(alpha)-decayed read of q plus
 * (q . k)(z - r), which equals S_t^T q_t.
 *
 *   q, k, log_alpha, b : [N, H, d_k]       (dtype), one token per sequence
 *   v, w               : [N, H, d_v]       (dtype)
 *   state              : [N, H, d_k, d_v]  fp32, read-modify-written in place
 *   o                  : [N, H, d_v]       (dtype), written
 *   Supported: d_k, d_v in {64, 128}, both dtypes. N = 0 is a no-op.
 * Returns GDN2_OK or an error status.
 */
int gdn2_decode_step(const void* q, const void* k, const void* v, const void* log_alpha,
                     const void* b, const void* w, float* state, void* o, int N, int H,
                     int d_k, int d_v, int dtype, void* hip_stream);

/* gdn2_decode_step with a gate layout: scalar b and / or w are [N, H]. */
int gdn2_decode_step_ex(const void* q, const void* k, const void* v, const void* log_alpha,
                        const void* b, const void* w, float* state, void* o, int N, int H,
                        int d_k, int d_v, int dtype, int gate_layout, void* hip_stream);

/*
 * L consecutive tokens for each of N sequences against a pool of recurrent states: decode
 * of a few tokens at once, or verification of draft tokens in speculative decoding (the
 * reading note's §7 names speculative decoding as the serving direction). Per (sequence,
 * head) the state of slot state_indices[n] is read once, advanced through the L tokens with
 * the decode step's arithmetic, and the state after token commit_len[n] - 1 is written back
 * to that slot (commit_len[n] = 0 leaves the slot unchanged). Outputs of all L tokens are
 * written either way.
 *
 *   q, k, log_alpha, b : [N, L, H, d_k]   (dtype)
 *   v, w               : [N, L, H, d_v]   (dtype)
 *   state_pool         : [P, H, d_k, d_v] fp32, read and (partly) written in place
 *   state_indices      : device int32 [N], the slot of each sequence; a negative or >= P
 *                        slot skips the sequence (its outputs are not written). NULL: slot n
 *                        (then P >= N is required). Two sequences must not share a slot.
 *   commit_len         : device int32 [N] in [0, L] (clamped), or NULL for L
 *   o                  : [N, L, H, d_v]   (dtype), written
 *   step_states        : NULL, or [N, L, H, d_k, d_v] fp32: the state after every token
 *                        (so that an accepted prefix can be committed without recomputing)
 *   Supported: d_k, d_v in {64, 128}, both dtypes. N = 0 or L = 0 is a no-op.
 * Returns GDN2_OK or an error status.
 */
int gdn2_decode_tokens(const void* q, const void* k, const void* v, const void* log_alpha,
                       const void* b, const void* w, float* state_pool,
                       const int32_t* state_indices, const int32_t* commit_len, void* o,
                       float* step_states, int N, int L, int H, int d_k, int d_v, int P,
                       int dtype, void* hip_stream);

/* gdn2_decode_tokens with a gate layout: scalar b and / or w are [N, L, H]. */
int gdn2_decode_tokens_ex(const void* q, const void* k, const void* v, const void* log_alpha,
                          const void* b, const void* w, float* state_pool,
                          const int32_t* state_indices, const int32_t* commit_len, void* o,
                          float* step_states, int N, int L, int H, int d_k, int d_v, int P,
                          int dtype, int gate_layout, void* hip_stream);

/*
 * Block prologue: the branches between the block's projections and the mixer (the reading
 * note's §3 block paragraph: q, k = linear -> conv -> SiLU -> L2 norm; v = linear -> conv ->
 * SiLU; per-channel decay, erase and write gates from projections of their own). One pass
 * over the six projected tensors:
 *     q = l2norm(silu(conv(xq))), k = l2norm(silu(conv(xk))), v = silu(conv(xv)),
 *     log_alpha = -decay_scale * softplus(xg), b = b_max * sigmoid(xb), w = sigmoid(xw)
 * with conv the causal depthwise convolution of width 4 over each sequence's tokens
 * (y[t, c] = sum_j conv[c, j] * x[t - 3 + j, c], zero history at every sequence start) and
 * l2norm over d_k with eps 1e-6. (Conv width, eps and the gate activations are this
 * library's readings of what the page leaves open.)
 *
 *   xq, xk, xg, xb     : [B, T, H, d_k]   (dtype) projections
 *   xv, xw             : [B, T, H, d_v]   (dtype)
 *   conv_q, conv_k     : [H * d_k, 4] fp32 taps;  conv_v : [H * d_v, 4] fp32
 *   decay_scale        : [H * d_k] fp32 (positive)
 *   b_max              : 1 nominally, 2 for the widened erase-gate range
 *   q, k, log_alpha, b : [B, T, H, d_k] (dtype), written;  v, w : [B, T, H, d_v] (dtype)
 *   cu_seqlens         : as gdn2_chunk_fwd (B = 1 when given; N = B otherwise)
 * Returns GDN2_OK or an error status.
 */
int gdn2_block_prologue(const void* xq, const void* xk, const void* xv, const void* xg,
                        const void* xb, const void* xw, const float* conv_q,
                        const float* conv_k, const float* conv_v, const float* decay_scale,
                        float b_max, void* q, void* k, void* v, void* log_alpha, void* b,
                        void* w, const int32_t* cu_seqlens, int B, int T, int H, int d_k,
                        int d_v, int N, int dtype, void* hip_stream);

/*
 * Block epilogue: the mixer output scaled by an RMSNorm with a SiLU gate (the reading note's
 * §3 block paragraph): y = o / sqrt(mean_c(o^2) + 1e-6) * weight * silu(gate), the mean over
 * d_v per (token, head).
 *
 *   o, gate, y : [rows, d_v] (dtype), rows = tokens x heads;  weight : [d_v] fp32
 * Returns GDN2_OK or an error status.
 */
int gdn2_block_epilogue(const void* o, const void* gate, const float* weight, void* y,
                        long rows, int d_v, int dtype, void* hip_stream);

/*
 * The softmax-attention layer that a hybrid stack places beside the mixer (the reading note's
 * §3 architecture paragraph: mixer, then sliding-window attention): per-head norms of queries
 * and keys with the position rotation, for training; the same pass for serving, which also
 * writes keys and values into a paged 8-bit cache; and attention over that cache.
 */

/* Flags of the norm-and-rotation entry points. */
enum {
  GDN2_ROPE_INTERLEAVED = 1, /* pairs (2i, 2i + 1) instead of (i, i + rot / 2) */
  GDN2_ROPE_NO_NORM = 2      /* rotation only: no mean square; the weights still apply */
};

/*
 * Norm of every head row of q and k and the position rotation, in one pass:
 *     n = x / sqrt(mean(x^2) + eps) * weight
 *     pair i < rot / 2, angle = position * inv_freq[i]:
 *       y_a = n_a cos - n_b sin,  y_b = n_b cos + n_a sin;   channels past rot: y = n
 * fp32 throughout, the angle reduced in fp64 (any int32 position), one rounding.
 *
 *   q, k               : [B, T, Hq, d], [B, T, Hk, d] (dtype). The rows of one token are dense;
 *                        token t (of B * T) starts at element t * q_stride / t * k_stride, so
 *                        q and k may be slices of one projection. Strides are at least H * d
 *                        and multiples of 8.
 *   q_weight, k_weight : [d] fp32, or NULL for ones
 *   positions          : device int32 [B, T], or NULL for 0 .. T - 1 in every sequence
 *   inv_freq           : device fp32 [rot / 2], radians per position (NULL when rot = 0)
 *   rot                : rotated channels, a multiple of 8 in [0, d]
 *   q_out, k_out       : dense [B, T, H, d] (dtype), written; may be q and k themselves where
 *                        those are dense
 *   Supported: d in {64, 128}, both dtypes. B * T = 0 is a no-op.
 * Returns GDN2_OK or an error status.
 */
int gdn2_qk_norm_rope(const void* q, const void* k, const float* q_weight, const float* k_weight,
                      const int32_t* positions, const float* inv_freq, void* q_out, void* k_out,
                      int B, int T, int Hq, int Hk, int d, int64_t q_stride, int64_t k_stride,
                      int rot, float eps, int flags, int dtype, void* hip_stream);

/*
 * Gradients of gdn2_qk_norm_rope: dq, dk (dense, dtype) from the dense gradients dq_out, dk_out
 * of its outputs and its inputs, and the weights' gradients [d] fp32 (each NULL where not
 * wanted; written also where the weight itself is NULL). dq may be dq_out, dk may be dk_out.
 * The sums over rows are formed in a fixed order: equal inputs give equal bits.
 *   workspace : needed where a weight gradient is: at least
 *               gdn2_qk_norm_rope_bwd_workspace_bytes(...) bytes, 16-byte aligned
 * B * T = 0 is a no-op (weight gradients are not written). Returns GDN2_OK or an error status.
 */
int gdn2_qk_norm_rope_bwd(const void* q, const void* k, const void* dq_out, const void* dk_out,
                          const float* q_weight, const float* k_weight, const int32_t* positions,
                          const float* inv_freq, void* dq, void* dk, float* dq_weight,
                          float* dk_weight, int B, int T, int Hq, int Hk, int d, int64_t q_stride,
                          int64_t k_stride, int rot, float eps, int flags, int dtype,
                          void* workspace, size_t workspace_bytes, void* hip_stream);
size_t gdn2_qk_norm_rope_bwd_workspace_bytes(int B, int T, int Hq, int Hk, int d);

/*
 * The 8-bit cache. Blocks of GDN2_CACHE_BLOCK tokens; per block and kv head one scale for the
 * keys and one for the values, a power of two s; the value held is e4m3 (OCP e4m3fn) * s.
 *   k_cache : [P, Hk, 64, d]  bytes, a key row per token
 *   v_cache : [P, Hk, d, 64]  bytes, a row per channel; token t of the block is column
 *             (t / 4 % 4) * 16 + (t / 16) * 4 + t % 4
 *   k_scale, v_scale : [P, Hk] fp32
 *   block_table : device int32 [N, max_blocks]: block b of sequence n holds its positions
 *             64 b .. 64 b + 63. An entry outside [0, P), or a position past the table, is a
 *             place that does not exist: nothing is written there, and no query sees a key or
 *             value there, whatever the pool holds elsewhere.
 *   seq_lens : device int32 [N]: tokens of every sequence, those of this call included. The
 *             new tokens of a sequence are its last ones; where it has fewer tokens than new
 *             rows, the leading rows hold no token (padding).
 * Of a block that is read, all 64 value columns must hold finite values, also where no token is:
 * a cache that starts as zeros and is written by gdn2_attn_prologue always does.
 * The new rows come as a fixed number T per sequence ([N, T, H, d]: cu_seqlens NULL, N = B) or
 * packed (cu_seqlens as for gdn2_chunk_fwd, B = 1).
 */
enum { GDN2_CACHE_BLOCK = 64 };

/*
 * Serving prologue of the attention layer: gdn2_qk_norm_rope on the new rows (position = place
 * in the sequence), queries to q_out, keys and values into the cache.
 *   A block's scale is the smallest power of two s >= 2^-64 with max|x| <= 448 s over the new
 *   rows in it, and not below its scale so far unless the block's first position is among the
 *   new rows (then what the block held is dropped: its value positions without a token are
 *   cleared). Where a scale grows, the block's older codes are rescaled (exact, but for codes
 *   that fall below e4m3's normal range). What lies behind the new tokens (dropped drafts) stays,
 *   except that values there are cleared where their scale grows to 2^120, the largest.
 *   A token whose key or value row holds a NaN, an infinity or a magnitude from 248 * 2^120 on
 *   (after norm and rotation) has a key row of NaN and a zero value row in the cache and does
 *   not count for the scales: every query of that head which attends to it comes out NaN, others
 *   are not touched.
 *   q, k, v : rows as in gdn2_qk_norm_rope, strides of their own
 *   q_out   : dense [.., Hq, d]; zeros in rows without a token (padding); rows in front of the
 *             first packed sequence and behind the last are not written; may be q where that is
 *             dense
 *   A block that this call writes must stand in the table once.
 *   Supported: GDN2_BF16, d in {64, 128}, Hq a multiple of Hk. No tokens: a no-op.
 * Returns GDN2_OK or an error status.
 */
int gdn2_attn_prologue(const void* q, const void* k, const void* v, const float* q_weight,
                       const float* k_weight, const float* inv_freq, void* q_out, void* k_cache,
                       void* v_cache, float* k_scale, float* v_scale, const int32_t* block_table,
                       const int32_t* seq_lens, const int32_t* cu_seqlens, int B, int T, int Hq,
                       int Hk, int d, int N, int P, int max_blocks, int64_t q_stride,
                       int64_t k_stride, int64_t v_stride, int rot, float eps, int flags,
                       int dtype, void* hip_stream);

/*
 * Causal attention of the new rows over the cache, which already holds their own keys and
 * values:  o_i = sum_j softmax_j(scale q_i . k_j) v_j,  j <= p_i, and j > p_i - window where
 * window > 0. Query head h reads kv head h / (Hq / Hk). A row that sees no key (padding, an
 * empty sequence, blocks that do not exist) is written as zeros; rows in front of the first packed
 * sequence and behind the last are not written.
 * Up to 32 rows (tokens of the call per sequence, or in all when packed, times Hq / Hk) the weights
 * enter the second product as two bf16 terms, and the result is off by its own rounding; above, as
 * in prompts, they are rounded once to bf16 (2.2e-3 relative in the 2-norm against 64 bits, where
 * the result's rounding alone is 1.7e-3). Sequences of few rows in a packed call may go either way.
 * The output is divided by the sum of its weights at the end, so the sum of |v| over the keys that a
 * row sees has to stay below 2^120.
 *   q, o      : dense [B, T, Hq, d] (dtype); o may be q
 *   scale     : positive and finite, usually 1 / sqrt(d)
 *   workspace : at least gdn2_cache_attention_workspace_bytes(...) bytes (0: may be NULL),
 *               16-byte aligned, free for the call's duration on `hip_stream`. A captured call
 *               uses it at every replay: two graphs that may run at once need one each.
 *   max_blocks : the key axis is cut for sequences that fill the table, as their lengths are on the
 *               device. A table several times as wide as they need makes calls of few rows or few
 *               tiles two to three times slower: pass no more columns than the longest may need.
 *   Supported: GDN2_BF16, d in {64, 128}, Hq a multiple of Hk, B * T * Hq below 2^31 - 1024. No
 *   tokens: a no-op.
 * Returns GDN2_OK or an error status.
 */
int gdn2_cache_attention(const void* q, const void* k_cache, const void* v_cache,
                         const float* k_scale, const float* v_scale, const int32_t* block_table,
                         const int32_t* seq_lens, const int32_t* cu_seqlens, void* o, int B, int T,
                         int Hq, int Hk, int d, int N, int P, int max_blocks, int window,
                         float scale, int dtype, void* workspace, size_t workspace_bytes,
                         void* hip_stream);
/* packed: whether cu_seqlens is given; the other arguments as for the call. */
size_t gdn2_cache_attention_workspace_bytes(int packed, int B, int T, int Hq, int Hk, int d, int N,
                                            int max_blocks, int window);

/*
 * What stands around the mixer in a stack: a lighter recurrent layer, the norm between layers, and
 * the verification of drafted tokens that says how many of them a pool of states commits.
 */

/*
 * The diagonal gated recurrence (the mixer's with one key channel and no erase: a state per
 * channel), over whole sequences:
 *     h_t = exp(log_alpha_t) h_{t-1} + w_t v_t,   o_t = h_t
 *
 *   v, log_alpha, w : [B, T, D] (dtype). Token t (of B * T) starts at element t * stride of its own,
 *                     its channels dense, so they may be slices of one projection; strides are at
 *                     least D, multiples of 8 and at most 2^21. w may be NULL (ones). log_alpha <= 0; -inf (a
 *                     reset) is fine.
 *   initial_state   : [N, D] fp32, or NULL for zeros
 *   o               : dense [B, T, D] (dtype), written; may be NULL where only states are wanted
 *   final_state     : [N, D] fp32, or NULL; may be initial_state
 *   states          : NULL, or gdn2_linear_recurrence_states_bytes(...) bytes: the states before
 *                     every 64th token, which the backward reads
 *   cu_seqlens      : as for gdn2_chunk_fwd, but that rows in front of the first sequence and behind the
 *                     last are allowed. They are not written.
 *   workspace       : at least gdn2_linear_recurrence_workspace_bytes(...) bytes (0: may be NULL),
 *                     16-byte aligned, free for the call's duration on `hip_stream`; calls that can
 *                     overlap, captured ones among them, need one each. Long sequences of few
 *                     channels are cut into segments that run in parallel.
 *   (With `states`, for training, rows that belong to no packed sequence are written as zeros.)
 *   Supported: D a multiple of 8, both dtypes, B * T below 2^31 - 4096, N * D / 64 below 2^23 (D
 *   rounded up to 64). A NaN or an infinity stays in its own sequence and
 *   channel, from its token on. What a decay of less than 2^-126, of one token or of several
 *   together, leaves of a state may count as nothing. T = 0 copies the initial state to the final one;
 *   N = 0 without `states` is a no-op.
 * Returns GDN2_OK or an error status.
 */
int gdn2_linear_recurrence(const void* v, const void* log_alpha, const void* w,
                           const float* initial_state, void* o, float* final_state, float* states,
                           const int32_t* cu_seqlens, int B, int T, int D, int N,
                           int64_t v_stride, int64_t g_stride, int64_t w_stride, int dtype,
                           void* workspace, size_t workspace_bytes, void* hip_stream);
/* backward: whether for gdn2_linear_recurrence_bwd; packed: whether cu_seqlens is given. */
size_t gdn2_linear_recurrence_workspace_bytes(int backward, int packed, int B, int T, int D, int N);
size_t gdn2_linear_recurrence_states_bytes(int packed, int B, int T, int D, int N);

/*
 * Gradients of gdn2_linear_recurrence: dv, dlog_alpha, dw (dense, dtype; dw only with w) and
 * d_initial_state ([N, D] fp32, or NULL) from d_o (dense), d_final_state ([N, D] fp32, or NULL for
 * zeros), the inputs and the states that the forward kept for them; workspace as for the forward. Rows that belong to no packed
 * sequence get zeros. Equal inputs give equal bits. Returns GDN2_OK or an error status.
 */
int gdn2_linear_recurrence_bwd(const void* v, const void* log_alpha, const void* w,
                               const float* states, const void* d_o, const float* d_final_state,
                               void* dv, void* dlog_alpha, void* dw, float* d_initial_state,
                               const int32_t* cu_seqlens, int B, int T, int D, int N,
                               int64_t v_stride, int64_t g_stride, int64_t w_stride, int dtype,
                               void* workspace, size_t workspace_bytes, void* hip_stream);

/*
 * L consecutive tokens of each of N sequences against a pool of states, as gdn2_decode_tokens is
 * for the mixer: v, log_alpha, w [N, L, D] with strides as above (w may be NULL), state_pool
 * [P, D] fp32, o and step_states (fp32, or NULL) dense [N, L, D]; state_indices, commit_len and
 * what they mean as there. Returns GDN2_OK or an error status.
 */
int gdn2_linear_recurrence_tokens(const void* v, const void* log_alpha, const void* w,
                                  float* state_pool, const int32_t* state_indices,
                                  const int32_t* commit_len, void* o, float* step_states, int N,
                                  int L, int D, int P, int64_t v_stride, int64_t g_stride,
                                  int64_t w_stride, int dtype, void* hip_stream);

/*
 * The norm between layers, with the residual's addition:
 *     h = x + residual   (rounded to the residual's type: the stream that the next layer adds to)
 *     y = h / sqrt(mean(h^2) + eps) * weight     (of h as it is stored; fp32 inside,
 *                                                 sums over a row fp64)
 *
 *   x        : [rows, D] (dtype), row i at element i * x_stride, channels dense
 *   residual : [rows, D] (r_dtype), r_stride likewise; or NULL: h = x, and h is not written
 *   weight   : [D] fp32
 *   y        : dense [rows, D] (dtype); with scale, e4m3 codes (bytes)
 *   h        : dense [rows, D] (r_dtype); may be residual, or x, where that is dense and of its type
 *   scale    : NULL, or fp32 [rows, D / group] (group 0: [rows], one a row): the value of a code is
 *              e4m3 * scale, with scale the smallest power of two s >= 2^-64 with max|y| <= 448 s over
 *              its group. A row with a NaN or an infinity gives NaN codes where y is NaN.
 *   group    : 0, 32, 64 or 128 channels (0 without scale); D a multiple of it
 *   Supported: D a multiple of 8 up to 16384; types bf16 with bf16, bf16 with an fp32 residual, fp32
 *   with fp32; rows below 2^23. fp32's precision where sqrt(mean(h^2) + eps) of a row lies between 2^-126
 *   and 2^126, forward and backward. rows = 0 is a no-op.
 * Returns GDN2_OK or an error status.
 */
int gdn2_residual_norm(const void* x, const void* residual, const float* weight, void* y, void* h,
                       float* scale, int64_t rows, int D, int64_t x_stride, int64_t r_stride,
                       int group, float eps, int dtype, int r_dtype, void* hip_stream);

/*
 * Gradients of gdn2_residual_norm without scale: from dy (dtype) and dh (r_dtype, or NULL for zero),
 * both dense, and h as the forward wrote it (h_stride: x itself where there was no residual),
 *     dh_total = dh + rho (u - n mean(u n)),  n = h rho,  u = dy weight
 * to dx (dtype) and, where the types differ, to dr (r_dtype; else NULL), and dweight [D] fp32. dx
 * may be dy, or dh where the types agree. Sums over rows are formed in a fixed order.
 *   workspace : at least gdn2_residual_norm_bwd_workspace_bytes(rows, D) bytes, 16-byte aligned
 * rows = 0 is a no-op (dweight is not written). Returns GDN2_OK or an error status.
 */
int gdn2_residual_norm_bwd(const void* dy, const void* dh, const void* h, const float* weight,
                           void* dx, void* dr, float* dweight, int64_t rows, int D,
                           int64_t h_stride, float eps, int dtype, int r_dtype, void* workspace,
                           size_t workspace_bytes, void* hip_stream);
size_t gdn2_residual_norm_bwd_workspace_bytes(int64_t rows, int D);

/*
 * Verification of drafted tokens from given random numbers. Sequence n has draft_len[n] drafts; p_i
 * is the target's distribution in front of draft i (p behind the last draft at i = draft_len), q_i
 * the draft's:
 *     draft i is accepted where u_i q_i(x_i) < p_i(x_i) and all before it were;  a: how many were
 *     the next token is drawn from max(p_a - q_a, 0) where draft a was rejected (from p_a where that
 *     is zero everywhere), from p_a where none was: the first j whose cumulated weight passes
 *     u_L times their sum (fp64: where the sums are not exact, a draw within some 2^-53 of the
 *     sum from a border may give the neighbouring entry)
 * Rows need not sum to one. Entries that are not positive count as zero, NaN among them.
 *
 *   target_probs : [N, L + 1, V] (dtype), dense
 *   draft_probs  : [N, L, V] (dtype), dense; or NULL: drafts that were certain (q(x_i) = 1)
 *   drafts       : device int32 [N, L]; one outside [0, V) is rejected
 *   draft_len    : device int32 [N], clamped to [0, L], or NULL for L
 *   uniforms     : fp32 [N, L + 1] in [0, 1)
 *   tokens       : int32 [N, L + 1], written: the accepted drafts, the next token, -1 behind it (the
 *                  next token itself is -1 where p_a is zero everywhere)
 *   commit_len   : int32 [N], written: a + 1. Of the L + 1 tokens that went through the target (the
 *                  last one known, then the drafts), so many are to be kept: the commit_len of
 *                  gdn2_decode_tokens and gdn2_linear_recurrence_tokens.
 *   workspace    : at least gdn2_verify_drafts_workspace_bytes(N, V) bytes, 16-byte aligned; calls
 *                  that can overlap need one each
 *   N * V / 4096 below 2^23 (V rounded up to 4096). N = 0 is a no-op. Returns GDN2_OK or an error
 *   status.
 */
int gdn2_verify_drafts(const void* target_probs, const void* draft_probs, const int32_t* drafts,
                       const int32_t* draft_len, const float* uniforms, int32_t* tokens,
                       int32_t* commit_len, int N, int L, int V, int dtype, void* workspace,
                       size_t workspace_bytes, void* hip_stream);
size_t gdn2_verify_drafts_workspace_bytes(int N, int V);

/* Human-readable text for a status code (static storage; never NULL). */
const char* gdn2_status_string(int status);

/* Library version string (static storage). */
const char* gdn2_version(void);

#ifdef __cplusplus
}
#endif

#endif /* GDN2_H_ */
