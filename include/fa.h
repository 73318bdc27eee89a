/*
 * fa.h - C ABI of the exact tiled attention library for GB300 (sm_103a).
 *
 * The library computes exact softmax attention, O = softmax(scale * Q K^T) V,
 * without ever writing an N x N matrix to device memory:
 *
 *   - the forward pass keeps a block of 128 queries on chip and streams the
 *     keys and values past it in blocks of 128 with the online softmax
 *     (running maximum m, running sum l = sum e^{s-m}, rescaled output
 *     accumulator), then writes O and one log-sum-exp L_i = m_i + log l_i per
 *     query row ("Interrogating the GPU part 5: FlashAttention", sections
 *     "How does tiling remove the traffic?" and "How can you softmax a row you
 *     never see whole?", online-softmax update equation; "LLM Flash
 *     Attention", section "End-to-end flow");
 *   - the backward pass recomputes every probability tile as
 *     P_ij = exp(S_ij - L_i) from Q, K and the saved L, and forms
 *     dV = P^T dO, dS = P o (dP - delta), dQ = scale dS K, dK = scale dS^T Q
 *     ("Interrogating the GPU part 5: FlashAttention", section "What does the
 *     backward pass do without P?", LSE equation and recompute formula).
 *
 * Conventions shared by every entry point
 * ---------------------------------------
 * Layout.  Q, K, V, O, dO, dQ, dK, dV are contiguous bf16 arrays laid out
 *   [B][H][N][d] (row-major, d fastest).  LSE and delta are contiguous fp32
 *   arrays [B][H][N].  Queries and keys share the length N.
 * Scores.  S = scale * Q K^T; LSE is in natural-log units of the scaled scores.
 * Causal.  causal = 1 hides key j from query i when j > i (top-left aligned);
 *   causal = 0 attends to all N keys.
 * Memory.  Every pointer is device memory owned by the caller; the library
 *   allocates nothing (no cudaMalloc; tensor memory is taken and released
 *   inside each thread block).  Its only state is one device status word per
 *   device, used to report a kernel that gave up waiting (FA_ERR_TIMEOUT).
 * Streams.  Calls only enqueue work on `stream` (0 = legacy default stream) and
 *   return the launch status; they do not synchronize.  A device-side timeout
 *   is reported later by fa_check_device_status.
 * Device.  Every call runs on the CURRENT device (cudaGetDevice): the caller
 *   makes the tensors' device current first.  Every tensor pointer must be
 *   device memory of that device, or managed memory; anything else (host
 *   memory, another device's memory, an address no allocation covers) gives
 *   FA_ERR_INVALID_ARG before anything is enqueued.
 * Errors.  Arguments are validated before anything is enqueued; on an error
 *   nothing runs and no output is written.  Invalid sizes, a null pointer, a
 *   pointer the current device cannot use (above) or a non-finite /
 *   non-positive scale give FA_ERR_INVALID_ARG; a pointer not on a 16-byte
 *   boundary gives FA_ERR_MISALIGNED; a head dimension other than 64 or 128
 *   gives FA_ERR_UNSUPPORTED; a failed CUDA call (including a device without
 *   sm_103a support) gives FA_ERR_CUDA.
 * Validity of the outputs.  A returned FA_OK means the work was enqueued.
 *   Every wait inside the kernels is bounded in time (fa_set_wait_limit_ns,
 *   default 10 s); a kernel whose wait runs out -- which also happens if the
 *   GPU stops running it for longer than the limit, e.g. under heavy time
 *   slicing -- stops early, leaves its outputs undefined and records
 *   FA_ERR_TIMEOUT in the device status word.  The outputs of a sequence of
 *   calls are therefore known to be valid only once fa_check_device_status
 *   has returned FA_OK after them.
 * Limits.  1 <= B, H, N; B * H < 2^31 and (ceil(N / 128) + 1) * B * H < 2^31
 *   (the kernels count 128-row blocks in 32-bit integers and address memory
 *   with 64-bit offsets, so B * H * N * d itself may exceed 2^31);
 *   fa_fwd_fp8 also needs B * H <= 65535.
 */
#ifndef FA_H_
#define FA_H_

#include <stddef.h>
#include <cuda_runtime_api.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  FA_OK = 0,
  FA_ERR_INVALID_ARG = 1,
  FA_ERR_MISALIGNED = 2,
  FA_ERR_UNSUPPORTED = 3,
  FA_ERR_CUDA = 4,
  FA_ERR_TIMEOUT = 5
} fa_status;

/*
 * Forward pass.  "Interrogating the GPU part 5: FlashAttention", sections
 * "How does tiling remove the traffic?" and "How can you softmax a row you
 * never see whole?" (online-softmax update equation), with the log-sum-exp
 * of section "What does the backward pass do without P?"; causal block
 * skipping as in "LLM Flash Attention", section "End-to-end flow".
 *
 *   q, k, v  in:  bf16 [B][H][N][d]
 *   o        out: bf16 [B][H][N][d], O = softmax(scale Q K^T) V
 *   lse      out: fp32 [B][H][N],   L_i = log sum_j exp(scale q_i . k_j)
 *   scale    finite, > 0 (1/sqrt(d) for standard attention)
 *   causal   0 or 1
 *   d        64 or 128
 */
fa_status fa_fwd(const void* q, const void* k, const void* v, void* o, float* lse, int B, int H, int N, int d,
                 float scale, int causal, cudaStream_t stream);

/*
 * FP8 forward.  "Interrogating the GPU part 5: FlashAttention", section "What
 * did FlashAttention-3 do with Hopper?" (FP8 quantised per block after a
 * random Hadamard rotation, which spreads outliers across the block);
 * "FlashAttention versions", section "FlashAttention-3 (2024)" (block-level
 * quantisation instead of one per-tensor scale).  Same result as fa_fwd up
 * to FP8 rounding, with the products on the tensor cores' E4M3 path:
 *   1. Q and K rows are rotated by R = diag(signs) H / sqrt(128) (H the
 *      Sylvester Hadamard matrix), which leaves Q K^T unchanged, and rounded
 *      to E4M3 (nearest even, saturating at +-448) with one scale per block
 *      of 128 rows of each (batch, head): scale = max|x R| / 448;
 *   2. V is rounded to E4M3 with one scale per channel of each (batch, head)
 *      over the sequence: scale = max_n |v_nc| / 448;
 *   3. the online softmax of fa_fwd runs on the dequantised scores, the
 *      probabilities are rounded to E4M3 for the P V product, and O is
 *      normalised by the sum of the rounded probabilities and multiplied by
 *      the value channel scales.  LSE uses the unrounded sum.
 *
 *   q, k, v    in:  bf16 [B][H][N][128]
 *   signs      in:  int8 [128] device array of +1 / -1 (the random signs of
 *                   the rotation; the caller draws them)
 *   o, lse     out: as for fa_fwd
 *   workspace  device scratch of ws_bytes >= fa_fwd_fp8_workspace_bytes(),
 *              16-byte aligned.  Layout (each part on a 256-byte boundary,
 *              in this order): Q R and K R in E4M3 [B][H][N][128];
 *              V^T in E4M3 [B][H][nkb][128 channels][128 keys] (keys past N
 *              zero), nkb = ceil(N / 128); query and key block scales fp32
 *              [B][H][nkb] each; value channel maxima (fp32 bits) and scales
 *              fp32 [B][H][128] each.  Its contents on entry are ignored.
 *   d          128 only (other values give FA_ERR_UNSUPPORTED)
 */
size_t fa_fwd_fp8_workspace_bytes(int B, int H, int N, int d);
fa_status fa_fwd_fp8(const void* q, const void* k, const void* v, const signed char* signs, void* o, float* lse,
                     void* workspace, size_t ws_bytes, int B, int H, int N, int d, float scale, int causal,
                     cudaStream_t stream);

/*
 * Backward preprocess: delta_i = sum_c dO_ic * O_ic, one fp32 per query row.
 * The term delta of dS = P o (dP - delta) in "Interrogating the GPU part 5:
 * FlashAttention", section "What does the backward pass do without P?"; the
 * pages do not define it, and the row sum of dO o O is its exact value
 * (sum_j P_ij dP_ij with dP = dO V^T and O = P V).
 *
 *   o, dout  in:  bf16 [B][H][N][d]
 *   delta    out: fp32 [B][H][N]
 */
fa_status fa_bwd_preprocess(const void* o, const void* dout, float* delta, int B, int H, int N, int d,
                            cudaStream_t stream);

/*
 * Bytes of device workspace fa_bwd needs: an fp32 dQ accumulator
 * [B][H][N][d], then delta and LSE*log2(e) as fp32 [B][H][Npad] each, where
 * Npad = 128 * ceil(N / 128) (every part starting on a 256-byte boundary).
 * Returns 0 for sizes fa_bwd would reject.
 */
size_t fa_bwd_workspace_bytes(int B, int H, int N, int d);

/*
 * Backward pass by recomputation.  "Interrogating the GPU part 5:
 * FlashAttention", section "What does the backward pass do without P?" (LSE
 * equation, recompute formula P_ij = exp(S_ij - L_i), dV = P^T dO,
 * dS = P o (dP - delta)); "LLM Flash Attention", section "End-to-end flow"
 * (backward paragraph).  dQ is accumulated in fp32 in the workspace and cast
 * to bf16 at the end.
 *
 *   q, k, v, o, dout  in:  bf16 [B][H][N][d]; o and lse as written by fa_fwd
 *   lse               in:  fp32 [B][H][N]
 *   dq, dk, dv        out: bf16 [B][H][N][d] (overwritten, not accumulated)
 *   workspace         device scratch of ws_bytes >= fa_bwd_workspace_bytes(),
 *                     16-byte aligned; its contents on entry are ignored
 *   scale, causal     as passed to fa_fwd
 * ws_bytes too small gives FA_ERR_INVALID_ARG.  dQ is summed with fp32
 * atomics, so it is not bitwise repeatable from run to run.
 */
fa_status fa_bwd(const void* q, const void* k, const void* v, const void* o, const void* dout, const float* lse,
                 void* dq, void* dk, void* dv, void* workspace, size_t ws_bytes, int B, int H, int N, int d,
                 float scale, int causal, cudaStream_t stream);

/*
 * Backward pass with a deterministic dQ.  Same arguments, layout, workspace
 * (ws_bytes >= fa_bwd_workspace_bytes()) and error behaviour as fa_bwd, and
 * the same dQ, dK, dV up to rounding; dQ, dK and dV are bitwise repeatable
 * from run to run on the same device.  "Interrogating the GPU part 5:
 * FlashAttention", section "What does the backward pass do without P?"
 * (recompute formula, dS = P o (dP - delta)); "LLM Flash Attention", section
 * "End-to-end flow" (each recomputed block contributes to the gradients; how
 * the contributions to dQ are summed is left open).  Here they are summed by a
 * separate pass rather than with atomics: after the key-block-major pass that
 * forms dK and dV, a query-block-major pass recomputes S = Q K^T,
 * dP = dO V^T and dS for each of its query blocks, sums dQ = scale dS K over
 * the key blocks in a fixed order in tensor memory, and writes it once.
 * This costs three more N x N x d products per head pair (the backward does
 * 7 N^2 d multiply-adds per (batch, head) instead of 5) and needs no fp32
 * atomics; the dQ accumulator part of the workspace is not used.
 */
fa_status fa_bwd_deterministic(const void* q, const void* k, const void* v, const void* o, const void* dout,
                               const float* lse, void* dq, void* dk, void* dv, void* workspace, size_t ws_bytes,
                               int B, int H, int N, int d, float scale, int causal, cudaStream_t stream);

/*
 * Backward pass with library-owned scratch.  This entry point has no
 * counterpart on the source pages; it exists for callers that cannot
 * allocate device memory when they run the backward pass -- for example a
 * plug-in inside a runtime that hands out device memory only from its own
 * arena and forbids cudaMalloc during execution, or a program that must keep
 * a fixed device-memory footprint after start-up.  It computes exactly what
 * fa_bwd computes, with the same arguments minus the workspace: the fp32 dQ
 * accumulator and delta live in a fixed array of FA_STATIC_SCRATCH_BYTES
 * compiled into the library, which every device that loads the library holds
 * until the process exits.  The call allocates nothing (no cudaMalloc, no
 * cudaFree, no allocating library routine).
 *
 * Limit: shapes whose fa_bwd_workspace_bytes(B, H, N, d) exceeds
 * FA_STATIC_SCRATCH_BYTES (72 MiB; roughly B*H*N*(d+2)*4 bytes must fit, as
 * for B=4, H=16, N=2048, d=128) return FA_ERR_INVALID_ARG and run nothing.
 * Set-up: the first call on a device looks up the array's device address on
 * that device (cudaGetSymbolAddress, with that device current) and caches it
 * for the life of the process; make that first call outside any stream
 * capture.  The cached address belongs to the device's context: after
 * cudaDeviceReset (which destroys that context and the array with it) this
 * entry point must not be called again in the same process.  Sharing: every call uses
 * the same array and the array keeps the last call's contents (each call
 * re-initialises what it reads).  Calls whose work overlaps on the GPU (on
 * different streams, or from different threads) race on the array and give
 * wrong results; calls ordered on one stream do not.
 */
#define FA_STATIC_SCRATCH_BYTES (72u * 1024u * 1024u)
fa_status fa_bwd_static_scratch(const void* q, const void* k, const void* v, const void* o, const void* dout,
                                const float* lse, void* dq, void* dk, void* dv, int B, int H, int N, int d,
                                float scale, int causal, cudaStream_t stream);

/*
 * Cross attention: queries [B][H][Nq][d] over keys and values [B][Hkv][Nk][d]
 * of another length (an encoder's states), O = softmax(scale Q K^T) V.
 * Query head h uses key/value head h / (H / Hkv); H is a multiple of Hkv.
 * There is no causal mask.  Scores, probabilities, their sums and what is joined of
 * an item cut among thread blocks are fp32; P is rounded to bf16 for P V, O once
 * at the end.
 *
 *   q        in:  bf16 [B][H][Nq][d]
 *   k, v     in:  bf16 [B][Hkv][Nk][d]
 *   key_lens in:  int32 [B] device array: request b has keys 0 .. key_lens[b]-1
 *                 (values outside [0, Nk] are taken as 0 and Nk), or null: Nk
 *                 for every request.  What K and V hold behind a request's
 *                 keys is never used, NaN and infinities included.  (Arrays of
 *                 lengths, positions, frequencies and masks, here and below,
 *                 need only their element's alignment.)
 *   o        out: bf16 [B][H][Nq][d];  lse out: fp32 [B][H][Nq].
 *                 A row without keys (or whose scores are all -inf) gives
 *                 O = 0 and LSE = -inf.
 *   workspace     device scratch of ws_bytes >= fa_cross_fwd_workspace_bytes(),
 *                 16-byte aligned, contents on entry ignored; calls that may
 *                 overlap on the GPU need one each.
 * Limits: those of fa_fwd with B * Hkv for B * H and, for N, both
 * (H / Hkv) * Nq and Nk, each at most 2^31 - 256; and
 * (ceil(Nk / 128) + 4) * B * Hkv < 2^31.  The results are the same from run to run.
 */
size_t fa_cross_fwd_workspace_bytes(int B, int H, int Hkv, int Nq, int Nk, int d);
fa_status fa_cross_fwd(const void* q, const void* k, const void* v, const int* key_lens, void* o, float* lse,
                       void* workspace, size_t ws_bytes, int B, int H, int Hkv, int Nq, int Nk, int d, float scale,
                       cudaStream_t stream);

/*
 * Backward pass of fa_cross_fwd by recomputation: P = exp(S - LSE),
 * dV = P^T dO, dS = P o (dO V^T - rowsum(dO o O)), dQ = scale dS K,
 * dK = scale dS^T Q, dK and dV summed over the query heads that share them.
 * P and dS are rounded to bf16 for the products, the gradients once at the end
 * from fp32 sums.
 *
 *   q, o, dout, lse  in:  as for fa_cross_fwd; o and lse as it wrote them
 *   dq               out: bf16 [B][H][Nq][d]
 *   dk, dv           out: bf16 [B][Hkv][Nk][d]; zero behind a request's keys
 *   workspace        as for fa_cross_fwd, of fa_cross_bwd_workspace_bytes()
 * dQ is summed with fp32 atomics, so it is not bitwise repeatable from run to
 * run; dK and dV are.
 */
size_t fa_cross_bwd_workspace_bytes(int B, int H, int Hkv, int Nq, int Nk, int d);
fa_status fa_cross_bwd(const void* q, const void* k, const void* v, const int* key_lens, const void* o,
                       const void* dout, const float* lse, void* dq, void* dk, void* dv, void* workspace,
                       size_t ws_bytes, int B, int H, int Hkv, int Nq, int Nk, int d, float scale,
                       cudaStream_t stream);

/*
 * Attention of T new tokens per request over a key/value cache that already
 * holds them: one token (T = 1), a run of tokens, or a tree of drafted ones.
 * Request b has cache_lens[b] tokens of its own in rows 0 .. cache_lens[b]-1 of
 * the cache and its drafted tokens in the rows after them, in order.  Every
 * new token sees the request's own tokens; of the drafted ones, token n sees
 * token t when bit t of draft_masks[b][n] is set (its ancestors and itself
 * in a tree), or, without masks, when t <= n.
 *
 *   q            in:  bf16 [B][H][T][d]
 *   k_cache, v_cache  in: bf16 [B][Hkv][C][d], C rows of capacity; rows behind
 *                     a request's last drafted token are never used
 *   cache_lens   in:  int32 [B] (taken into [0, C])
 *   draft_lens   in:  int32 [B], or null: request b has draft_lens[b] <= T
 *                     drafted tokens, else T; never more than fit in C rows
 *   draft_masks  in:  64-bit words [B][T], or null (each token sees the ones
 *                     before it); bits of tokens that do not exist are ignored
 *   o, lse       out: as for fa_cross_fwd; rows of tokens >= the request's
 *                     number of drafted tokens are left as they were
 *   T            any with draft_masks null; at most 64 with them
 *                (FA_ERR_UNSUPPORTED)
 *                (every row meets all drafted keys of its request, hidden ones
 *                too: a prompt of T tokens costs T x T scores, not half of them)
 *   workspace    as for fa_cross_fwd, of fa_tree_fwd_workspace_bytes()
 * The values of a drafted token meet every row of its request (with weight 0
 * where a mask hides it), so a drafted row of V with an infinity or NaN makes
 * all of them NaN.
 * Limits: those of fa_cross_fwd with T for Nq and C for Nk.
 */
size_t fa_tree_fwd_workspace_bytes(int B, int H, int Hkv, int T, int C, int d);
fa_status fa_tree_fwd(const void* q, const void* k_cache, const void* v_cache, const int* cache_lens,
                      const int* draft_lens, const unsigned long long* draft_masks, void* o, float* lse,
                      void* workspace, size_t ws_bytes, int B, int H, int Hkv, int T, int C, int d, float scale,
                      cudaStream_t stream);

/*
 * Rows of a token-major tensor, as a projection leaves them: the d values of
 * head h of token n of request b start at ptr + b batch + n token + h head
 * (elements; every stride a multiple of 8, ptr on a 16-byte boundary).
 */
typedef struct {
  void* ptr;
  long long batch, token, head;
} fa_rows;

/*
 * Head norm and rotary positions: each query and key row x becomes
 *   u = weight o x / sqrt(mean(x^2) + eps)   (norm = 1; weight null: ones)
 *   u = x                                    (norm = 0)
 * and the first rotary_dim values of u are rotated in pairs by the angle
 * position * inv_freq[i] and multiplied by `factor`:
 *   (a, b) -> factor (a cos - b sin, a sin + b cos),
 * with pairs (i, i + rotary_dim / 2) (interleaved = 0) or (2 i, 2 i + 1)
 * (interleaved = 1); values from rotary_dim on stay as they are.  Rows go from
 * token-major tensors to head-major ones, as the attention entry points read
 * them; value rows are moved along unchanged.  Angles (modulo
 * whole turns) are off by at most 2^-23 + 2^-52 |position * inv_freq| radians.
 * Arithmetic is fp32, rounded once.
 *
 *   q, k, v      in:  bf16 rows, B requests of N tokens, H heads (q) and Hkv
 *                heads (k, v); a null q, k or v (ptr null, and its output null)
 *                leaves that tensor out
 *   q_weight, k_weight  in: fp32 [d] or null
 *   inv_freq     in:  fp64 [rotary_dim / 2] (radians per position); may be null
 *                when rotary_dim is 0
 *   positions    in:  int32 [B][N], or null: starts[b] + n
 *   starts       in:  int32 [B], or null (0): row of k_out and v_out that token 0
 *                of request b goes to (its length in a cache)
 *   q_out        out: bf16 [B][H][N][d]
 *   k_out, v_out out: bf16 [B][Hkv][C][d], rows starts[b] .. starts[b] + N - 1;
 *                rows outside [0, C) are not written, other rows stay as they were
 *   rotary_dim   a multiple of 16, 0 <= rotary_dim <= d (others:
 *                FA_ERR_UNSUPPORTED); C >= N
 *   eps          finite, >= 0; factor finite
 * No input may overlap an output.
 */
fa_status fa_rope_fwd(const fa_rows* q, const fa_rows* k, const fa_rows* v, const float* q_weight,
                      const float* k_weight, const double* inv_freq, const int* positions, const int* starts,
                      void* q_out, void* k_out, void* v_out, int B, int N, int H, int Hkv, int C, int d,
                      int rotary_dim, int norm, float eps, float factor, int interleaved, cudaStream_t stream);

/*
 * Backward pass of fa_rope_fwd (with starts null and C = N).
 *
 *   q, k         in:  the forward's inputs; not read (may be null) when norm = 0
 *   dq_out, dk_out, dv_out  in: bf16 [B][H][N][d], [B][Hkv][N][d]: the gradients
 *                of its outputs, as the attention backward passes write them
 *   dq, dk, dv   out: bf16 rows like q, k, v; a null one leaves that tensor out
 *                (its gradient then null too).  The rows may overlap neither one
 *                another nor an input.
 *   dq_weight, dk_weight  out: fp32 [d], summed over all rows; may be null
 *   workspace    device scratch of ws_bytes >= fa_rope_bwd_workspace_bytes(),
 *                16-byte aligned; may be null when no weight gradient is asked for
 * The results are the same from run to run.
 */
size_t fa_rope_bwd_workspace_bytes(int B, int H, int Hkv, int N, int d);
fa_status fa_rope_bwd(const fa_rows* q, const fa_rows* k, const float* q_weight, const float* k_weight,
                      const double* inv_freq, const int* positions, const void* dq_out, const void* dk_out,
                      const void* dv_out, const fa_rows* dq, const fa_rows* dk, const fa_rows* dv, float* dq_weight,
                      float* dk_weight, void* workspace, size_t ws_bytes, int B, int N, int H, int Hkv, int d,
                      int rotary_dim, int norm, float eps, float factor, int interleaved, cudaStream_t stream);

/*
 * Self-attention in which every query sees the keys of one span:
 *   O = softmax(s) V,  s_ij = cap tanh(scale q_i . k_j / cap) - slope_h |i - j|
 * over the keys j with key_begin_i <= j < key_end_i, j <= i (causal = 1) and
 * |i - j| < window (window > 0).  Without a cap (0) the first term is scale
 * q_i . k_j, without slopes there is no second one.  Packed documents are the
 * spans from a document's first token to behind its last one, with causal = 1;
 * a prefix that is seen both ways is key_end_i = max(i + 1, prefix) with
 * causal = 0; padding has empty spans.
 * Query head h uses key/value head h / (H / Hkv); H is a multiple of Hkv.
 * Scores (the tanh included), probabilities and their sums are fp32; P is
 * rounded to bf16 for P V, O once at the end.
 *
 *   q, o, lse    as for fa_fwd;  k, v  in: bf16 [B][Hkv][N][d]
 *   key_begin, key_end  in: int32 [B][N], or null: 0 and N.  (Values outside
 *                [0, N] are taken as 0 and N.)
 *   slopes       in:  fp32 [H], or null
 *   o, lse       rows that see no key give O = 0 and LSE = -inf
 *   cap          0, or positive and at most 16384, with 4 scale / cap finite and scale / cap
 *                normal.  The tanh is off by at most 2^-21, not relative to it: scores are off by
 *                up to 2^-21 of the cap, small ones too, hence the limit.
 *   window       >= 0
 *   workspace    as for fa_cross_fwd, of fa_span_fwd_workspace_bytes()
 * Scores of pairs outside the spans have no effect, whatever they are.  Rows of V
 * meet the queries of their tile with weight 0 where they are not seen, so a row
 * of V with an infinity or NaN may make any row of O of its request and head NaN.
 * Blocks of 128 keys that no query of a tile of 128 sees are left out.
 * Limits: those of fa_fwd for H and Hkv heads.  The results are the same from run
 * to run.
 */
size_t fa_span_fwd_workspace_bytes(int B, int H, int Hkv, int N, int d);
fa_status fa_span_fwd(const void* q, const void* k, const void* v, const int* key_begin, const int* key_end,
                      const float* slopes, void* o, float* lse, void* workspace, size_t ws_bytes, int B, int H, int Hkv,
                      int N, int d, float scale, float cap, int window, int causal, cudaStream_t stream);

/*
 * Backward pass of fa_span_fwd by recomputation: P = exp(s - LSE), dV = P^T dO,
 * dS = P o (dO V^T - rowsum(dO o O)) o (1 - tanh^2), dQ = scale dS K,
 * dK = scale dS^T Q, dK and dV summed over the query heads that share them.  The
 * cap and the slopes are constants: they have no gradients here.
 *
 *   q, o, dout, lse  in:  as for fa_span_fwd; o and lse as it wrote them
 *   dq               out: bf16 [B][H][N][d];  dk, dv  out: bf16 [B][Hkv][N][d]
 *   workspace        as for fa_span_fwd, of fa_span_bwd_workspace_bytes()
 * Rows that see no key have no gradient, keys that no query sees gradients of 0.
 * Q, K, V and dO meet products with weight 0 where a pair is not seen: an infinity
 * or NaN in any row of them may make any gradient of its request NaN.
 * dQ is summed with fp32 atomics, so it is not bitwise repeatable from run to
 * run; dK and dV are.  With spans by row one thread block plans the work, in a time
 * that grows with the square of N (0.13 ms at N = 131072, 1.8 ms at 524288).
 */
size_t fa_span_bwd_workspace_bytes(int B, int H, int Hkv, int N, int d);
fa_status fa_span_bwd(const void* q, const void* k, const void* v, const int* key_begin, const int* key_end,
                      const float* slopes, const void* o, const void* dout, const float* lse, void* dq, void* dk,
                      void* dv, void* workspace, size_t ws_bytes, int B, int H, int Hkv, int N, int d, float scale,
                      float cap, int window, int causal, cudaStream_t stream);

/*
 * Keys or values of a cache in pages of page_size tokens: the d values of token t
 * of a page and head start at ptr + page page + head head + t token (elements;
 * every stride positive and a multiple of 8, ptr on a 16-byte boundary; strides of
 * dimensions of size 1 are not used).  Both [page][head][token][d] and
 * [page][token][head][d] are such caches, and so is one half of a cache that keeps
 * keys and values side by side.
 */
typedef struct {
  void* ptr;
  long long page, head, token;
} fa_pages;

/*
 * Attention of a chunk of up to T new tokens per request (one token or thousands)
 * over a cache in pages that already holds them.  Request b has cache_lens[b]
 * tokens from before; new token n is at position p = cache_lens[b] + n and sees the
 * positions j <= p, with a window > 0 those with p - j < window.  Position j of
 * request b is row j % page_size of page page_table[b][j / page_size].  Scores as
 * for fa_span_fwd: cap tanh(scale q . k / cap) - slope_h (p - j).
 *
 *   q            in:  bf16 [B][H][T][d]
 *   k_pages, v_pages  in: num_pages pages of bf16 rows
 *   page_table   in:  int32 [B][table_width]; entries of pages that hold no token
 *                which a query sees are never used.  A page may be in many
 *                requests.  Numbers outside [0, num_pages) are pages of zeros.
 *   cache_lens   in:  int32 [B] (taken into [0, C], C = table_width * page_size)
 *   chunk_lens   in:  int32 [B], or null: request b has chunk_lens[b] <= T new
 *                tokens, else T; never more than fit in C
 *   slopes       in:  fp32 [H], or null
 *   o, lse       out: as for fa_cross_fwd; rows of tokens >= the request's number
 *                of new ones are left as they were
 *   page_size    a power of two, at least 16 (others: FA_ERR_UNSUPPORTED)
 *   workspace    as for fa_cross_fwd, of fa_paged_fwd_workspace_bytes()
 * What the pages hold behind a request's last new token is never used.  The values
 * of a chunk's tokens meet the rows of the tokens before them with weight 0, so a
 * row of V with an infinity or NaN may make any row of O of its request and head
 * NaN.  The results are the same from run to run.
 * Limits: those of fa_cross_fwd with T for Nq and C for Nk.
 */
size_t fa_paged_fwd_workspace_bytes(int B, int H, int Hkv, int T, int C, int d);
fa_status fa_paged_fwd(const void* q, const fa_pages* k_pages, const fa_pages* v_pages, const int* page_table,
                       const int* cache_lens, const int* chunk_lens, const float* slopes, void* o, float* lse,
                       void* workspace, size_t ws_bytes, int B, int H, int Hkv, int T, int d, int num_pages,
                       int page_size, int table_width, float scale, float cap, int window, cudaStream_t stream);

/*
 * fa_rope_fwd for a cache in pages: the rotated keys and the values of new token n
 * of request b go to position cache_lens[b] + n of its pages (as fa_paged_fwd reads
 * them), the rotated queries to q_out.
 *
 *   q, k, v, q_weight, k_weight, inv_freq, q_out, rotary_dim, norm, eps, factor,
 *   interleaved  as for fa_rope_fwd
 *   positions    in:  int32 [B][N], or null: cache_lens[b] + n
 *   page_table, cache_lens, chunk_lens  as for fa_paged_fwd; page_table and
 *                cache_lens may be null where k and v are left out (cache_lens
 *                then counts as 0); no capacity bounds the new tokens there
 *   k_pages, v_pages  out: pages whose rows share no memory.  Rows of positions
 *                outside [0, C) and of pages outside [0, num_pages) are not
 *                written; rows of tokens >= the request's number of new ones are
 *                left as they were, in q_out too.  Where two tokens go to the same
 *                row, which of them it holds is not said.
 * No input may overlap an output.
 */
fa_status fa_rope_paged_fwd(const fa_rows* q, const fa_rows* k, const fa_rows* v, const float* q_weight,
                            const float* k_weight, const double* inv_freq, const int* positions,
                            const int* page_table, const int* cache_lens, const int* chunk_lens, void* q_out,
                            const fa_pages* k_pages, const fa_pages* v_pages, int B, int N, int H, int Hkv, int d,
                            int num_pages, int page_size, int table_width, int rotary_dim, int norm, float eps,
                            float factor, int interleaved, cudaStream_t stream);

/*
 * The entry points above from fa_cross_fwd on, with their arguments in one
 * struct (in the same order and with the same meaning), for callers whose
 * foreign function interface pays for every argument, as the Python binding's
 * does.  A null struct gives FA_ERR_INVALID_ARG.
 */
typedef struct {
  const void *q, *k, *v;
  const int* key_lens;
  void* o;
  float* lse;
  void* workspace;
  size_t ws_bytes;
  int B, H, Hkv, Nq, Nk, d;
  float scale;
  cudaStream_t stream;
} fa_cross_fwd_args;

typedef struct {
  const void *q, *k, *v;
  const int* key_lens;
  const void *o, *dout;
  const float* lse;
  void *dq, *dk, *dv, *workspace;
  size_t ws_bytes;
  int B, H, Hkv, Nq, Nk, d;
  float scale;
  cudaStream_t stream;
} fa_cross_bwd_args;

typedef struct {
  const void *q, *k_cache, *v_cache;
  const int *cache_lens, *draft_lens;
  const unsigned long long* draft_masks;
  void* o;
  float* lse;
  void* workspace;
  size_t ws_bytes;
  int B, H, Hkv, T, C, d;
  float scale;
  cudaStream_t stream;
} fa_tree_fwd_args;

typedef struct {
  fa_rows q, k, v;
  const float *q_weight, *k_weight;
  const double* inv_freq;
  const int *positions, *starts;
  void *q_out, *k_out, *v_out;
  int B, N, H, Hkv, C, d, rotary_dim, norm;
  float eps, factor;
  int interleaved;
  cudaStream_t stream;
} fa_rope_fwd_args;

typedef struct {
  fa_rows q, k;
  const float *q_weight, *k_weight;
  const double* inv_freq;
  const int* positions;
  const void *dq_out, *dk_out, *dv_out;
  fa_rows dq, dk, dv;
  float *dq_weight, *dk_weight;
  void* workspace;
  size_t ws_bytes;
  int B, N, H, Hkv, d, rotary_dim, norm;
  float eps, factor;
  int interleaved;
  cudaStream_t stream;
} fa_rope_bwd_args;

typedef struct {
  const void *q, *k, *v;
  const int *key_begin, *key_end;
  const float* slopes;
  void* o;
  float* lse;
  void* workspace;
  size_t ws_bytes;
  int B, H, Hkv, N, d;
  float scale, cap;
  int window, causal;
  cudaStream_t stream;
} fa_span_fwd_args;

typedef struct {
  const void *q, *k, *v;
  const int *key_begin, *key_end;
  const float* slopes;
  const void *o, *dout;
  const float* lse;
  void *dq, *dk, *dv, *workspace;
  size_t ws_bytes;
  int B, H, Hkv, N, d;
  float scale, cap;
  int window, causal;
  cudaStream_t stream;
} fa_span_bwd_args;

typedef struct {
  const void* q;
  fa_pages k_pages, v_pages;
  const int *page_table, *cache_lens, *chunk_lens;
  const float* slopes;
  void* o;
  float* lse;
  void* workspace;
  size_t ws_bytes;
  int B, H, Hkv, T, d, num_pages, page_size, table_width;
  float scale, cap;
  int window;
  cudaStream_t stream;
} fa_paged_fwd_args;

typedef struct {
  fa_rows q, k, v;
  const float *q_weight, *k_weight;
  const double* inv_freq;
  const int *positions, *page_table, *cache_lens, *chunk_lens;
  void* q_out;
  fa_pages k_pages, v_pages;
  int B, N, H, Hkv, d, num_pages, page_size, table_width, rotary_dim, norm;
  float eps, factor;
  int interleaved;
  cudaStream_t stream;
} fa_rope_paged_fwd_args;

fa_status fa_cross_fwd_packed(const fa_cross_fwd_args* args);
fa_status fa_cross_bwd_packed(const fa_cross_bwd_args* args);
fa_status fa_tree_fwd_packed(const fa_tree_fwd_args* args);
fa_status fa_rope_fwd_packed(const fa_rope_fwd_args* args);
fa_status fa_rope_bwd_packed(const fa_rope_bwd_args* args);
fa_status fa_span_fwd_packed(const fa_span_fwd_args* args);
fa_status fa_span_bwd_packed(const fa_span_bwd_args* args);
fa_status fa_paged_fwd_packed(const fa_paged_fwd_args* args);
fa_status fa_rope_paged_fwd_packed(const fa_rope_paged_fwd_args* args);

/*
 * Synchronizes `stream`, then returns and clears the current device's status
 * word: FA_OK, or FA_ERR_TIMEOUT if a kernel of this library gave up waiting
 * on one of its barriers since the last check (its outputs are then
 * undefined), or FA_ERR_CUDA if the synchronization itself failed.
 */
fa_status fa_check_device_status(cudaStream_t stream);

/*
 * Upper bound, in nanoseconds, on every barrier wait inside the kernels
 * launched after this call (process-wide; 0 restores the default of ten
 * seconds).  A wait that runs out makes the kernel stop early and report
 * FA_ERR_TIMEOUT through fa_check_device_status; it never traps.  Meant for
 * tests of that path.
 */
void fa_set_wait_limit_ns(unsigned long long limit_ns);

/*
 * Test hook for the timeout path.  While `enable` is nonzero, every kernel
 * launched by fa_fwd / fa_bwd (and the main kernels of fa_cross_fwd,
 * fa_cross_bwd, fa_tree_fwd, fa_span_fwd, fa_span_bwd and fa_paged_fwd) first makes its MMA-issuing thread wait on a
 * barrier that nothing ever signals; that wait runs out after the wait limit
 * (fa_set_wait_limit_ns), the kernel reports FA_ERR_TIMEOUT, drains the copies
 * it started and returns.  The outputs of the call are then undefined, as after
 * any wait that runs out: kernels that join or finish a call's parts run on
 * what is there.  Process-wide; 0 (the default) turns it off.  Nothing traps or hangs.
 */
void fa_debug_stall(int enable);

/*
 * Where fa_fwd evaluates its exponentials ("Interrogating the GPU part 5:
 * FlashAttention", section "Why did Blackwell need FlashAttention-4?": part of
 * the exponentials run in software as 2^n times a cubic in the fraction, on
 * the FMA units, the rest on the special-function unit).  soft_quarters = 0
 * (the default) computes every probability with the special-function unit's
 * ex2; 1 or 2 computes that many of every four pairs of probabilities a
 * softmax thread forms with the cubic 1 + 0.6951 f + 0.2276 f^2 + 0.0771 f^3
 * (relative error <= 1.0e-4, 20 times below a bf16 probability's rounding).
 * The results stay within the same tolerances; only the speed differs.
 * Applies to the bf16 forward launched after the call (fa_fwd_fp8 always uses
 * the special-function unit).  Process-wide.  Other values give
 * FA_ERR_INVALID_ARG and change nothing.
 */
fa_status fa_set_exp2_split(int soft_quarters);

/*
 * How fa_bwd_deterministic forms dK and dV at d = 128 ("Interrogating the GPU
 * part 5: FlashAttention", section "Why did Blackwell need FlashAttention-4?":
 * the 2-SM MMA, in which two SMs compute one product of twice the rows, each
 * reading half of the other operand from its own shared memory).  enable = 0
 * (the default): one CTA per 128-key block, as fa_bwd.  enable != 0: clusters of
 * two CTAs on adjacent key blocks, whose four products per query block
 * (S^T, dP^T, dV, dK) run as 256-row tcgen05 MMAs across the pair; the
 * results are the same up to summation order and equally bitwise repeatable.
 * d = 64 and fa_bwd are not affected.  Process-wide; applies to calls made
 * after it.
 */
void fa_set_bwd_pair_mma(int enable);

/*
 * Profiling hook.  While set, fa_fwd and fa_fwd_fp8 record fwd_start and
 * fwd_stop on their stream immediately before and after launching the
 * attention kernel (not around fa_fwd_fp8's operand preparation), and fa_bwd
 * and fa_bwd_deterministic record bwd_start and bwd_stop around the main
 * backward kernel (not around the preprocess, the final dQ cast or the
 * deterministic dQ pass), so that cudaEventElapsedTime gives the duration of
 * exactly those kernels.  The events are created and
 * owned by the caller on the device the calls run on; a null pointer disables
 * its pair.  Process-wide; call again with nulls to turn it off.
 */
void fa_set_timing_events(cudaEvent_t fwd_start, cudaEvent_t fwd_stop, cudaEvent_t bwd_start,
                          cudaEvent_t bwd_stop);

/* Static, human-readable name of a status code. */
const char* fa_status_string(fa_status status);

#ifdef __cplusplus
}
#endif

#endif /* FA_H_ */
