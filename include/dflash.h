/*
 * dflash.h — C ABI of the DFlash 2 draft-verify hot path on one GB300 GPU.
 *
 * One draft-verify cycle is four calls, in this order, on one stream:
 *
 *   dflash_lmhead_topk  two-tap conv + drafter LM head + logsumexp + top-16
 *   dflash_pair_score   context gate + low-rank bilinear scores of the
 *                       16 x 16 candidate pairs of adjacent positions
 *   dflash_path_walk    greedy or sampled walk through the K x 16 lattice
 *   dflash_verify       rejection-sampling verify, residual / bonus draw
 *
 * or two: dflash_draft (the first three in one call, with the context gate
 * computed inside the conv launch) and dflash_verify.  Where the target model
 * runs in the same program, dflash_kv_append, dflash_paged_attn and
 * dflash_sample carry its share of the cycle; dflash_kv_append_axes,
 * dflash_shared_attn, dflash_attn_mass, dflash_kv_evict and dflash_logprobs
 * do so for targets with several position axes, batches under one prompt,
 * caches of a bounded size, and answers with their probabilities.
 *
 * Sources (page title, section):
 *   "DFlash 2: Block diffusion, wearing a drafter's coat" — "Sixteen
 *     candidates per position", "A path selector", "Suffix-decay
 *     convolution", "Lossless, with conditions I did not used to state".
 *   "A 2B Drafter Made a 27B Model 3.4x Faster. Same Exact Output." —
 *     "The two fixes", "Running it", "Caveats before you rebuild your
 *     serving stack".
 *   "DFlash 2: Keep Drafting Parallel" — "What Comes Next", "A Lightweight
 *     Path Selector".
 *
 * Conventions shared by every call:
 *   - Shapes: B sequences, K drafted positions per sequence (1..16), V
 *     vocabulary, H drafter hidden size, r selector rank (1..256), C = 16
 *     candidates per position.  M = B*K rows.  All arrays are row-major and
 *     contiguous.
 *   - Every pointer argument except `seed`-like scalars is DEVICE memory
 *     owned by the caller (for example a torch CUDA tensor).  The library
 *     allocates nothing on these paths; scratch comes from the caller's
 *     workspace `ws` of at least dflash_workspace_bytes(...) bytes.
 *   - Calls are asynchronous on stream `s` (NULL = legacy default stream).
 *     Arguments are checked on the host before anything is launched; a bad
 *     argument returns DFLASH_ERR_INVALID_ARG (or _UNSUPPORTED) and
 *     launches nothing.
 *   - Problems found on the device (an index out of range, a non-finite
 *     target logit, a draft that is not among its candidates) set a sticky
 *     device error word; kernels never trap.  dflash_check() synchronises
 *     the stream, reads and clears that word and returns the matching
 *     status.
 *   - dtype (DFLASH_BF16 or DFLASH_FP32) is the storage type of the
 *     drafter-side tensors (hidden states, weights, embeddings).  All
 *     accumulation is fp32.  Scores, probabilities and target logits are
 *     fp32 whatever dtype is.
 *   - When V < 16 the candidate lists are padded with index -1 and value
 *     -inf (q = 0).
 *   - Randomness: uniforms are Philox4x32-10 (Salmon et al., SC'11) with
 *     key (seed lo, seed hi) and counter (b, t, purpose, cycle mod 2^32);
 *     purpose 0 = walk draw of position t, 1 = accept draw of position t,
 *     2 = residual / bonus draw (t = K); u = (word0 >> 8) * 2^-24.  Give
 *     each cycle a new `cycle` value.  T = 0 selects the greedy forms and
 *     ignores seed and cycle.
 */
#ifndef DFLASH_H_
#define DFLASH_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* Same type as cudaStream_t / CUstream. */
typedef struct CUstream_st* dflash_stream_t;

typedef enum {
  DFLASH_OK = 0,
  DFLASH_ERR_INVALID_ARG = 1,    /* bad pointer, size, alignment or value */
  DFLASH_ERR_UNSUPPORTED = 2,    /* valid request this build cannot run  */
  DFLASH_ERR_CUDA = 3,           /* a CUDA runtime call failed           */
  DFLASH_ERR_NONFINITE = 4,      /* device: NaN or +inf target logit     */
  DFLASH_ERR_DEVICE_TIMEOUT = 5, /* device: a bounded wait ran out       */
  DFLASH_ERR_BAD_INDEX = 6       /* device: token id outside [0, V), or a
                                    draft not among its candidates        */
} dflash_status;

typedef enum { DFLASH_BF16 = 0, DFLASH_FP32 = 1 } dflash_dtype;

#define DFLASH_CANDIDATES 16
#define DFLASH_MAX_K 16
#define DFLASH_MAX_RANK 256
#define DFLASH_MAX_SHARDS 64   /* vocabulary shards of one merge / decide */
#define DFLASH_SHARD_STATS 20  /* words per target row of shard statistics */
#define DFLASH_SHARD_PLAN 8    /* words per sequence of a shard draw plan */
#define DFLASH_MAX_AXES 4      /* position axes of dflash_kv_append_axes */
#define DFLASH_MAX_ALTERNATIVES 32  /* most likely tokens of dflash_logprobs */

/* Workspace needed by dflash_lmhead_topk (which = 0), dflash_verify
 * (which = 1), dflash_draft (which = 2) or dflash_draft_e4m3 (which = 3)
 * for these sizes, in bytes; an upper bound over both dtypes and every r.
 * Returns 0 for invalid sizes. */
size_t dflash_workspace_bytes(int which, int B, int K, int H, int V);

/*
 * Steps a1 + a2: two-tap dynamic depthwise conv, drafter LM head, online
 * logsumexp and per-position top-16.
 *
 * "Suffix-decay convolution" (drafter's coat page) and "The two fixes"
 * (2B-drafter page): each position is mixed with its predecessor,
 *     w0_t = W0 h_t,  w1_t = W1 h_t,  y_t = w0_t * h_t + w1_t * h_{t-1},
 * per channel, h_{-1} = 0 at the first block position of every sequence,
 * y rounded to dtype.  "Sixteen candidates per position" and "A Lightweight
 * Path Selector": U_t = y_t W_lm^T is the drafter's own logit; the call
 * keeps its 16 largest entries and log(sum_v exp U_t(v)) without writing
 * U_t to memory.
 *
 *   h      [B, K, H] dtype        drafter final hidden states
 *   conv_w [2H, H]   dtype        rows 0..H-1 = W0, rows H..2H-1 = W1;
 *                                 NULL skips the conv (y = h)
 *   w_lm   [V, H]    dtype        LM head
 *   topv   [B*K, 16] fp32  out    U_t of the candidates, descending
 *   topi   [B*K, 16] int32 out    their token ids (ties: lower id first)
 *   lse    [B*K]     fp32  out    logsumexp of U_t over the vocabulary
 *   ws     >= dflash_workspace_bytes(0, B, K, H, V) bytes, 256-B aligned.
 *          On return its first B*K*H elements (dtype) hold y when conv_w
 *          is not NULL.
 * Requirements: 1 <= K <= 16, B >= 1, H % 8 == 0, V >= 1; bf16 operand
 * pointers 16-byte aligned.
 */
dflash_status dflash_lmhead_topk(const void* h, const void* conv_w,
                                 const void* w_lm, int B, int K, int H,
                                 int V, dflash_dtype dt, float* topv,
                                 int32_t* topi, float* lse, void* ws,
                                 size_t ws_bytes, dflash_stream_t s);

/*
 * Step a3: context gate and low-rank bilinear pair scores.
 *
 * "A Lightweight Path Selector" (Keep Drafting Parallel page) and "A path
 * selector" (drafter's coat page): for predecessor a and current candidate
 * b of adjacent positions,
 *     S_t(a, b) = U_t(b) + < E_in(a), G(h_t) * E_out(b) >,
 *     G(h_t) = sigmoid(W_g h_t)   (gate form: this library's reading),
 * every pair scored at once, with no backbone or LM-head pass.  The
 * predecessor of position 0 is the anchor (last verified) token, so all 16
 * rows of S[b, 0] are equal.
 *
 *   topv, topi [B, K, 16]  from dflash_lmhead_topk
 *   anchor     [B] int32   last verified token of each sequence
 *   h          [B, K, H] dtype   (the same hidden states, pre-conv)
 *   w_gate     [r, H] dtype;  e_in, e_out [V, r] dtype
 *   scores     [B, K, 16, 16] fp32 out: scores[b,t,i,j] = S_t(pred_i,
 *              cand_j); -inf where either index is -1.
 * Requirements: 1 <= r <= 256, 1 <= K <= 16, H % 8 == 0; h, w_gate, e_in
 * and e_out 16-byte aligned.
 */
dflash_status dflash_pair_score(const float* topv, const int32_t* topi,
                                const int32_t* anchor, const void* h,
                                const void* w_gate, const void* e_in,
                                const void* e_out, int B, int K, int H, int V,
                                int r, dflash_dtype dt, float* scores,
                                dflash_stream_t s);

/*
 * Step a4: walk one path through the K x 16 candidate lattice.
 *
 * "A Lightweight Path Selector": starting from the verified token, greedy
 * follows the best successor; sampling draws from the scores.  With
 * prev = 0 (the anchor row) and for t = 0..K-1:
 *   T == 0: j = argmax_j scores[b,t,prev,j] (lowest j on ties), q one-hot;
 *   T >  0: w_j = exp((scores[b,t,prev,j] - max) / T), q = w / sum(w),
 *           j = the smallest j with w_0 + .. + w_j > u * sum(w),
 *           u = walk uniform (b, t);
 *   prev = j.
 *   slot  [B, K] int32 out   chosen candidate slot
 *   draft [B, K] int32 out   topi[b, t, slot]
 *   q     [B, K, 16] fp32 out the draft distribution the verifier needs
 */
dflash_status dflash_path_walk(const float* scores, const int32_t* topi,
                               int B, int K, float T, uint64_t seed,
                               uint64_t cycle, int32_t* slot, int32_t* draft,
                               float* q, dflash_stream_t s);

/*
 * Steps a1-a4 in one call: dflash_lmhead_topk, dflash_pair_score and
 * dflash_path_walk with the same arguments and outputs as those three
 * calls, in that order ("Suffix-decay convolution" and "Sixteen candidates
 * per position" of "DFlash 2: Block diffusion, wearing a drafter's coat";
 * "A Lightweight Path Selector" of "DFlash 2: Keep Drafting Parallel").
 * For bf16 storage with a conv, the context gate g_t = sigmoid(W_g h_t)
 * reads the same h tiles as the conv, so it is computed by the conv launch
 * on the tensor cores and kept in the workspace; after the LM head, one
 * launch merges its partials, scores the pairs of each position (only
 * gathering embedding rows) and walks each sequence.  Otherwise the three
 * steps run as the separate calls do.
 *   inputs   h, conv_w (may be NULL: no conv), w_lm, w_gate, e_in, e_out,
 *            anchor, sizes, dt, T, seed, cycle: as in the three calls
 *   outputs  topv, topi, lse (dflash_lmhead_topk), scores
 *            (dflash_pair_score), slot, draft, q (dflash_path_walk)
 *   ws       >= dflash_workspace_bytes(2, B, K, H, V) bytes, 256-byte
 *            aligned, caller-owned; holds y, the LM-head partials, the
 *            gate and one walk ticket per sequence.
 * Requirements: the union of the three calls' (h, w_lm, w_gate, e_in,
 * e_out, scores 16-byte aligned; H % 8 == 0; 1 <= r <= 256; T >= 0).
 * Results equal the three calls' up to the order of fp32 accumulation in
 * the gate and in the logsumexp fold: the same candidates, lse and scores
 * within fp32 rounding.
 */
dflash_status dflash_draft(const void* h, const void* conv_w, const void* w_lm,
                           const void* w_gate, const void* e_in,
                           const void* e_out, const int32_t* anchor, int B,
                           int K, int H, int V, int r, dflash_dtype dt,
                           float T, uint64_t seed, uint64_t cycle, float* topv,
                           int32_t* topi, float* lse, float* scores,
                           int32_t* slot, int32_t* draft, float* q, void* ws,
                           size_t ws_bytes, dflash_stream_t s);

/*
 * 8-bit LM head (quantized drafters: "What a block-diffusion drafter is"
 * of the 2B-drafter page and "What Comes Next" of "DFlash 2: Keep Drafting
 * Parallel" ship GGUF-quantized drafter builds; this library's 8-bit form
 * is OCP FP8 E4M3 with one fp32 scale per row, the operand type of the
 * tensor cores' kind::f8f6f4 MMA).
 *
 * dflash_quantize_e4m3_rows: x [R, H] bf16 -> codes [R, H] uint8 (E4M3:
 * bias 7, 3 mantissa bits, no infinities, 448 largest) and scale [R] fp32:
 *     scale_i = max_k |x_ik| / 448 (1 for an all-zero row),
 *     codes_ik = E4M3(x_ik / scale_i), nearest with ties to even, saturated,
 * both divisions correctly rounded fp32.  Used once on W_lm when it is
 * loaded; dflash_draft_e4m3 applies it to y every call.
 * Requirements: H % 16 == 0; x and codes 16-byte aligned.  A non-finite
 * input sets DFLASH_ERR_NONFINITE in the device error word.
 */
dflash_status dflash_quantize_e4m3_rows(const void* x, int R, int H,
                                        uint8_t* codes, float* scale,
                                        dflash_stream_t s);

/*
 * dflash_draft for bf16 storage with a conv, with the LM head on 8-bit
 * operands: the conv output y is quantized per row
 * (dflash_quantize_e4m3_rows) and U_t(v) = s_y[t] s_W[v] sum_k
 * code_y[t,k] code_W[v,k] (fp32 accumulation; the codes' products are
 * exact).  W_lm is given as codes [V, H] uint8 and row scales [V] fp32.
 * Everything else (gate, candidates, lse, scores, walk, outputs) is as in
 * dflash_draft with dt = DFLASH_BF16.
 *   ws >= dflash_workspace_bytes(3, B, K, H, V) bytes, 256-byte aligned;
 *        holds dflash_draft's workspace (its first
 *        dflash_workspace_bytes(2, B, K, H, V) bytes, with y in bf16 at
 *        offset 0), then y's codes [B*K, H] uint8, then from the next
 *        256-byte boundary y's scales [B*K] fp32.
 * Requirements: conv_w not NULL; H % 16 == 0; w_lm_codes 16-byte aligned;
 * the rest as dflash_draft.
 */
dflash_status dflash_draft_e4m3(
    const void* h, const void* conv_w, const uint8_t* w_lm_codes,
    const float* w_lm_scale, const void* w_gate, const void* e_in,
    const void* e_out, const int32_t* anchor, int B, int K, int H, int V,
    int r, float T, uint64_t seed, uint64_t cycle, float* topv,
    int32_t* topi, float* lse, float* scores, int32_t* slot, int32_t* draft,
    float* q, void* ws, size_t ws_bytes, dflash_stream_t s);

/*
 * Steps a5 + a6: rejection-sampling verify with residual or bonus draw.
 *
 * "Lossless, with conditions I did not used to state" (drafter's coat
 * page): accept a draft token x with probability min(1, p(x)/q(x)), and on
 * the first rejection resample from normalize(max(0, p - q)); the emitted
 * tokens then follow the target distribution exactly.  p_t =
 * softmax(L[b,t] / T).  For t = 0..K-1 in order, draft t is accepted iff
 * u_t * q_t(x) < p_t(x) (u_t = accept uniform (b, t)); n = the number
 * accepted before the first rejection.  If n < K the token at n is drawn
 * from max(0, p_n - q_n) (q_n zero off the candidates; p_n if that is all
 * zero); if n = K a bonus token is drawn from p_K.  A draw takes the
 * smallest token v whose running weight sum exceeds u * total (u =
 * residual uniform (b, K)).  T == 0: accept iff the draft equals
 * argmax L[b,t] (lowest id on ties) and emit argmax L[b,n].
 *
 *   target_logits [B, K+1, V] fp32   target model logits, rows 0..K
 *   draft [B, K], topi [B, K, 16], q [B, K, 16]   from the walk
 *   n_accepted [B] int32 out
 *   out_tok [B, K+1] int32 out   draft[0..n-1], the drawn token, then -1
 *   ws >= dflash_workspace_bytes(1, B, K, 0, V) bytes, 256-B aligned
 * Requirements: target_logits 16-byte aligned; T >= 0.  A NaN or +inf
 * target logit sets DFLASH_ERR_NONFINITE in the device error word.
 * Rows are read in position order, and a row after its sequence's first
 * rejection (which no result depends on) stops being read once that
 * rejection is known: a non-finite logit there may go unreported.  Rows
 * 0..n of every sequence are always read in full.
 */
dflash_status dflash_verify(const float* target_logits, const int32_t* draft,
                            const int32_t* topi, const float* q, int B, int K,
                            int V, float T, uint64_t seed, uint64_t cycle,
                            int32_t* n_accepted, int32_t* out_tok, void* ws,
                            size_t ws_bytes, dflash_stream_t s);

/*
 * One whole cycle, steps a1-a6: dflash_draft (or, with w_lm_scale,
 * dflash_draft_e4m3 with w_lm as the E4M3 codes) followed by dflash_verify
 * of its draft, topi and q, with the same arguments, outputs and results
 * as those two calls.  On the tensor-core paths (bf16 storage with a conv)
 * the conv launch also zeroes the verify's tickets, which dflash_verify
 * otherwise zeroes with a copy-engine fill of its own before its launch;
 * that fill and its gap before the verify launch cost about 4.5 us of a
 * b32k8 cycle (B = 32, K = 8, V = 151936).
 *   inputs   h, conv_w, w_lm, w_lm_scale (NULL: bf16 LM head; else w_lm
 *            holds [V, H] uint8 codes and w_lm_scale [V] fp32 scales from
 *            dflash_quantize_e4m3_rows), w_gate, e_in, e_out, anchor, the
 *            sizes, dt, T, seed, cycle: as in dflash_draft(_e4m3);
 *            target_logits [B, K+1, V] fp32 as in dflash_verify
 *   outputs  topv, topi, lse, scores, slot, draft, q (the draft call's),
 *            n_accepted, out_tok (the verify's)
 *   ws_draft >= dflash_workspace_bytes(2, ...) bytes (3 with w_lm_scale),
 *            ws_verify >= dflash_workspace_bytes(1, B, K, 0, V) bytes, both
 *            256-byte aligned and caller-owned; ws_verify's contents need
 *            no zeroing by the caller.
 * Requirements: the union of the two calls'; w_lm_scale only with
 * dt == DFLASH_BF16.  Every argument is checked before anything is
 * launched.
 */
dflash_status dflash_cycle(
    const void* h, const void* conv_w, const void* w_lm,
    const float* w_lm_scale, const void* w_gate, const void* e_in,
    const void* e_out, const int32_t* anchor, const float* target_logits,
    int B, int K, int H, int V, int r, dflash_dtype dt, float T,
    uint64_t seed, uint64_t cycle, float* topv, int32_t* topi, float* lse,
    float* scores, int32_t* slot, int32_t* draft, float* q,
    int32_t* n_accepted, int32_t* out_tok, void* ws_draft,
    size_t ws_draft_bytes, void* ws_verify, size_t ws_verify_bytes,
    dflash_stream_t s);

/*
 * dflash_verify without any caller-provided scratch, for callers that
 * cannot allocate device memory at the time they verify: serving loops whose
 * device memory belongs to another engine's allocator, code running where
 * allocation (and the synchronisation it can bring) is not allowed, and C
 * callers with no allocator of their own.  This entry point has no
 * counterpart in the pages; it exists for those callers only.
 *
 * Same arguments, checks, semantics, results and profiling stage as
 * dflash_verify, minus ws and ws_bytes.  The scratch is a fixed 4 MiB array
 * the library holds in device memory on every GPU that loads it, until the
 * process exits; sizes whose scratch, dflash_workspace_bytes(1, B, K, 0, V)
 * (about B*(K+1)*ceil(V/2048)*8 bytes), exceeds 4 MiB are refused with
 * DFLASH_ERR_UNSUPPORTED.  At V = 151936, B = 256 with K = 16 fits (2.7 MB)
 * and K = 16 fits up to B = 405; at V = 262144, B = 256 fits up to K = 14.
 * The first call on a device looks up the array's device address (so make
 * that first call before any stream capture).  All calls share the
 * array: each clears what must start at zero itself, and calls whose
 * kernels overlap on the GPU (several streams or threads on one device)
 * race on it and must be serialised by the caller.  Allocates nothing.
 */
dflash_status dflash_verify_noalloc(const float* target_logits,
                                   const int32_t* draft, const int32_t* topi,
                                   const float* q, int B, int K, int V,
                                   float T, uint64_t seed, uint64_t cycle,
                                   int32_t* n_accepted, int32_t* out_tok,
                                   dflash_stream_t s);

/*
 * The step after verify in a draft-verify loop: commit each sequence's
 * emitted tokens and hand the last one over as the next cycle's anchor.
 *
 * "What a block-diffusion drafter is" (2B-drafter page): the target
 * verifies the whole run and the matching prefix is kept; "How many tokens
 * survive": acceptance length is the mean number of draft tokens kept per
 * verification pass.  For every sequence b, with n = n_accepted[b]:
 *   tokens[b, length[b] .. length[b] + n] = out_tok[b, 0 .. n]
 *   (the n accepted drafts, then the resampled or bonus token),
 *   length[b] += n + 1, anchor[b] = out_tok[b, n];
 *   stats[0] += n (accepted drafts), stats[1] += 1 (verification passes),
 *   stats[2] += n + 1 (emitted tokens), stats[3 + n] += 1 (histogram).
 * Mean acceptance length = stats[0] / stats[1].
 *   n_accepted [B] int32, out_tok [B, K+1] int32   from dflash_verify
 *   anchor     [B] int32 in/out      the next cycle's anchor
 *   tokens     [B, capacity] int32 in/out, length [B] int32 in/out:
 *              each sequence's committed tokens; a sequence whose buffer
 *              is full keeps the tokens that fit, and the call flags
 *              DFLASH_ERR_BAD_INDEX in the device error word (length still
 *              advances, so a caller can tell how many were dropped)
 *   stats      [DFLASH_COMMIT_STATS] int64 in/out, accumulated over calls
 * All device memory, caller-owned; no workspace.  Requires 1 <= K <= 16,
 * capacity >= 1.  An n_accepted outside [0, K] is flagged as
 * DFLASH_ERR_BAD_INDEX and that sequence is left unchanged.
 */
#define DFLASH_COMMIT_STATS (3 + DFLASH_MAX_K + 1)
dflash_status dflash_commit(const int32_t* n_accepted, const int32_t* out_tok,
                            int B, int K, int32_t* anchor, int32_t* tokens,
                            int32_t* length, int capacity, int64_t* stats,
                            dflash_stream_t s);

/*
 * Selector variant: the global max-sum path through the K x 16 lattice
 * (a Viterbi walk), for T = 0.  "What Comes Next" (Keep Drafting Parallel
 * page): pairwise scoring is the simplest selector and there is room to
 * explore; the pages' own greedy walk follows the best successor instead.
 *   best_0(j) = scores[b,0,0,j],
 *   best_t(j) = max_i best_{t-1}(i) + scores[b,t,i,j]  (t = 1..K-1),
 * the path ends in the lowest j of maximal best_{K-1}(j), predecessors on
 * ties are the lowest i, sums in fp32.  Outputs as dflash_path_walk: slot,
 * draft = topi[b,t,slot], q one-hot.  scores 16-byte aligned; 1 <= K <= 16.
 * A sequence with no path of finite score flags DFLASH_ERR_BAD_INDEX.
 */
dflash_status dflash_path_viterbi(const float* scores, const int32_t* topi,
                                  int B, int K, int32_t* slot, int32_t* draft,
                                  float* q, dflash_stream_t s);

/*
 * Diagnostic of the candidate lists ("What Comes Next", Keep Drafting
 * Parallel page: recall of the 16 candidates by position, and the
 * acceptance length an oracle that always picks the right candidate among
 * them would reach).  For every drafted position (b, t), t < K:
 *   target_argmax[b,t] = the first argmax over v of target_logits[b,t,v],
 *   in_top16[b,t]      = 1 if that token is among topi[b,t,:], else 0.
 * Recall@16 at position t is the mean of in_top16[:, t]; with greedy
 * verification a perfect selector is accepted up to the first position
 * whose in_top16 is 0.  Reads the K target rows once (B*K*V*4 bytes).
 * target_logits [B, K+1, V] fp32; topi [B*K, 16]; outputs [B*K] int32.
 * A NaN / +inf logit flags DFLASH_ERR_NONFINITE.
 */
dflash_status dflash_top16_recall(const float* target_logits,
                                  const int32_t* topi, int B, int K, int V,
                                  int32_t* target_argmax, int32_t* in_top16,
                                  dflash_stream_t s);

/*
 * Vocabulary shards.  With the vocabulary split into S contiguous ranges
 * [v0, v0 + V_shard) (an LM head and target logits too large for one
 * device, or a target that is itself split by vocabulary), each shard
 * computes what depends on its range only, the shards' small summaries are
 * gathered (S x a few words per row), and a merge gives exactly what the
 * whole-vocabulary calls give: the same candidates and tokens, logsumexp
 * and probabilities within fp32 rounding of another summation order.  The
 * pages have no sharded form; the decomposition follows from the
 * definitions of the top-16, the logsumexp, the accept test and the
 * inverse CDF (each a fold over the vocabulary).  Every call runs on the
 * caller's device and stream; moving the summaries between devices (an
 * all-gather) is the caller's, and one device can run all shards in turn.
 *
 * dflash_lmhead_topk_shard: steps a1 + a2 of dflash_lmhead_topk on the
 * shard's LM-head rows w_lm_shard [V_shard, H] (the conv is recomputed on
 * every shard; it is small).  Writes the shard's partial of every row:
 *   part_v, part_i [B*K, 16]  the shard's 16 best logits and their global
 *                             ids (v0 + row of w_lm_shard), descending,
 *                             ties to the lower id, padding (-inf, -1)
 *   part_m, part_s [B*K]      the shard's max of U_t and sum exp(U_t - max)
 *   ws >= dflash_workspace_bytes(0, B, K, H, V_shard) bytes.
 * Requirements as dflash_lmhead_topk; v0 >= 0.
 */
dflash_status dflash_lmhead_topk_shard(const void* h, const void* conv_w,
                                       const void* w_lm_shard, int B, int K,
                                       int H, int V_shard, int v0,
                                       dflash_dtype dt, float* part_v,
                                       int32_t* part_i, float* part_m,
                                       float* part_s, void* ws,
                                       size_t ws_bytes, dflash_stream_t s);

/* The S shards' partials gathered in shard order (part_v, part_i
 * [S, M, 16]; part_m, part_s [S, M]; M = B*K) merged into topv, topi
 * [M, 16] and lse [M], as dflash_lmhead_topk writes them.  1 <= S <= 64. */
dflash_status dflash_topk_merge_shards(const float* part_v,
                                       const int32_t* part_i,
                                       const float* part_m,
                                       const float* part_s, int S, int M,
                                       float* topv, int32_t* topi, float* lse,
                                       dflash_stream_t s);

/*
 * Steps a5 + a6 by vocabulary shard, in three calls.
 *
 * 1. dflash_verify_shard_stats, on each shard: the shard's target logits
 *    target_shard [B, K+1, V_shard] (ids v0 .. v0 + V_shard - 1 of a
 *    vocabulary of V) -> stats [B*(K+1), DFLASH_SHARD_STATS] fp32 words,
 *    per target row: [0] the shard's max logit, [1] at T > 0 its sum of
 *    exp((x - max) / T), at T = 0 its first argmax (global id, int bits),
 *    [2..17] the logits of the row's 16 candidates the shard holds,
 *    [18] that of the draft, [19] a mask (uint bits) of which it holds
 *    (bit j: candidate j, bit 16: the draft).  The shard's segment sums
 *    stay in ws (>= dflash_workspace_bytes(1, B, K, 0, V_shard) bytes) for
 *    step 3.
 * 2. dflash_verify_shard_decide, with every shard's stats gathered in
 *    shard order ([S, B*(K+1), DFLASH_SHARD_STATS]): each row's max and Z
 *    (or argmax), the accept tests as dflash_verify takes them, n_accepted
 *    and out_tok; at T = 0 out_tok is final.  At T > 0 the token at n is
 *    drawn in step 3 (out_tok holds -1 there until then) from the plan
 *    [B, DFLASH_SHARD_PLAN]: the shard whose part of the residual (or of p)
 *    holds the draw, and the remaining mass within it.
 * 3. dflash_verify_shard_draw, on each shard (index `shard`, with its ws
 *    from step 1): the draws the plan gives to that shard, written to
 *    out_tok.  Nothing to do at T = 0.
 * Same uniforms, tests and draws as dflash_verify ("Lossless, with
 * conditions I did not used to state", drafter's coat page); the sums are
 * folded per shard, then over shards in shard order.
 */
dflash_status dflash_verify_shard_stats(const float* target_shard,
                                        const int32_t* draft,
                                        const int32_t* topi, int B, int K,
                                        int V_shard, int v0, int V, float T,
                                        float* stats, void* ws,
                                        size_t ws_bytes, dflash_stream_t s);
dflash_status dflash_verify_shard_decide(
    const float* stats, int S, const int32_t* draft, const int32_t* topi,
    const float* q, int B, int K, int V, float T, uint64_t seed,
    uint64_t cycle, int32_t* n_accepted, int32_t* out_tok, float* plan,
    dflash_stream_t s);
dflash_status dflash_verify_shard_draw(const float* target_shard,
                                       const float* plan,
                                       const int32_t* topi, const float* q,
                                       int shard, int B, int K, int V_shard,
                                       int v0, float T, int32_t* out_tok,
                                       void* ws, size_t ws_bytes,
                                       dflash_stream_t s);

/*
 * The target's side of a cycle: the tokens that go through the target model
 * before there are target logits.  The pages leave this part to the serving
 * engine ("Running it" and "Caveats before you rebuild your serving stack",
 * 2B-drafter page); these three calls are what a draft-verify loop needs
 * from it: append the block's keys and values to the cache, attend over
 * that cache with K+1 tokens per sequence, and filter or sample the logits.
 *
 * The cache holds keys and values in 8 bits (OCP FP8 E4M3, NaN never
 * stored by dflash_kv_append) in pages of `page` tokens:
 *   k_codes, v_codes [num_pages, Hkv, page, D] uint8
 *   k_scale, v_scale [num_pages, Hkv] fp32: one scale for each page and
 *                    head, a power of two of at least 2^-64; a cached value
 *                    is code * scale
 *   page_table       [B, max_pages] int32: token t of sequence b is slot
 *                    t mod page of page page_table[b, t / page]
 * page is 16, 32, 64 or 128; D is a multiple of 16 up to 256; Hq query heads
 * share Hkv key heads in groups of Hq / Hkv (query head h reads key head
 * h / (Hq / Hkv)).  Entries of page_table that no token needs are not read.
 */

/*
 * dflash_kv_append: rotate q and k by their positions, append k and v to the
 * cache.  Sequence b gets n = n_new[b] tokens (rows b*Q .. b*Q + n - 1 of q,
 * k and v) at positions pos[b] .. pos[b] + n - 1; what the cache held from
 * pos[b] on is overwritten, so the tokens that a verify rejected need no
 * clearing: append at the committed length.
 *   rotation of the first `rot` dimensions of every head by the angles whose
 *   cosines and sines row p of cos_tab, sin_tab [max_pos, rot/2] fp32 holds:
 *     (a, b) -> (a c - b s, b c + a s), the pairs (a, b) being dimensions
 *     (j, j + rot/2), or (2j, 2j + 1) if interleaved; in fp32, each product
 *     and sum rounded; rot = 0 (no tables) leaves q and k as they are
 *   scale of a page and head: the least power of two s >= 2^-64 with
 *     max |x| <= 448 s over the page's new tokens, and at least the old
 *     scale if the page holds tokens before pos[b]; where that raises the
 *     scale, the codes of those older tokens are rounded anew to it (exact
 *     but for codes that become subnormal)
 *   code = E4M3(x / s), nearest with ties to even; x is fp32 here, rounded
 *     once.
 *   q [B*Q, Hq, D], k, v [B*Q, Hkv, D] dtype, rows ld_q, ld_k, ld_v elements
 *     apart (so they can be parts of one projection's output); q may be NULL
 *     (then Hq and q_out are not used)
 *   q_out [B, Q, Hq, D] dtype out: q rotated; rows without a token are 0
 *   kv_len [B] int32 out: pos[b] + n, the length dflash_paged_attn takes;
 *     must not be pos itself
 *   n_new [B] int32, or NULL: Q tokens each
 * Requirements: D % 16 == 0, rot % 8 == 0, rot <= D, rows and pointers of q,
 * k, v, q_out aligned to four elements, the tables and codes to 16 bytes;
 * ld >= heads * D; pages that this call writes belong to one sequence each.
 * On the device: tokens beyond the page table or the angle tables, n_new
 * outside [0, Q] (all of the sequence's tokens), a negative pos (likewise) and
 * a page id outside [0, num_pages) set DFLASH_ERR_BAD_INDEX; such tokens are
 * left out.  kv_len counts none of them but those of a bad page id, which
 * dflash_paged_attn counts as zeros and flags again.  A NaN k (after its
 * rotation) or v sets DFLASH_ERR_NONFINITE and is stored as 0, an infinite one
 * sets it and is stored as the largest code.  (An infinite k is turned with its
 * partner: times a cosine or sine of 0, or against another infinity, it makes a
 * NaN.)
 */
dflash_status dflash_kv_append(
    const void* q, const void* k, const void* v, int64_t ld_q, int64_t ld_k,
    int64_t ld_v, const float* cos_tab, const float* sin_tab,
    const int32_t* pos, const int32_t* n_new, const int32_t* page_table,
    int B, int Q, int Hq, int Hkv, int D, int rot, int interleaved,
    int max_pos, int page, int num_pages, int max_pages, dflash_dtype dt,
    void* q_out, uint8_t* k_codes, uint8_t* v_codes, float* k_scale,
    float* v_scale, int32_t* kv_len, dflash_stream_t s);

/* Workspace of dflash_paged_attn for these sizes in bytes; 0 for invalid
 * sizes. */
size_t dflash_paged_attn_workspace_bytes(int B, int Q, int Hq, int Hkv, int D);

/*
 * dflash_paged_attn: softmax attention of each sequence's last tokens over
 * its cache.  Query i < q_len[b] of sequence b stands at position
 * kv_len[b] - q_len[b] + i and sees the cached tokens t
 *   causal:     t <= its own position (the verify pass, a prompt's chunk)
 *   not causal: t < kv_len[b] (a drafter's block, which sees all of itself)
 *   s_t = scale * <q, k_t>,  out = sum_t softmax(s)_t v_t,
 *   lse = ln sum_t exp(s_t).
 * A query that sees nothing, and rows i >= q_len[b], give out = 0 and
 * lse = -inf.
 *   q, out [B, Q, Hq, D] dtype; lse [B, Q, Hq] fp32 or NULL
 *   kv_len [B] int32; q_len [B] int32 or NULL (Q each)
 *   ws >= dflash_paged_attn_workspace_bytes(B, Q, Hq, Hkv, D) bytes, 256-byte
 *      aligned; its contents need no initialisation
 * With bf16 storage and D <= 128 the products run on the tensor cores: q as
 * the sum of two 8-bit numbers (all its bits, down to 2^-17 of its row's
 * largest value), the softmax weights as the sum of four E5M2 numbers (to
 * 2^-13 of themselves or 2^-25 of their row's largest, whichever is more; a
 * weight counts with its value's scale here); sums and statistics in fp32.
 * Otherwise fp32 on the CUDA cores.
 * Codes and slots past kv_len may hold anything.  Scales are powers of two
 * between 2^-64 and 2^120, as dflash_kv_append writes them.
 * Requirements: Hq % Hkv == 0, Hq / Hkv <= 64, B * Q * Hq < 2^31; q, out and
 * the codes 16-byte aligned; scale finite; fewer than 2^31 tiles of 128 tokens
 * over all sequences' page tables and key heads (with bf16).  On the device:
 * kv_len below 0 or beyond the page table, q_len outside [0, Q] and a page id
 * outside [0, num_pages) set DFLASH_ERR_BAD_INDEX (lengths are clamped, such a
 * page counts as zeros).
 */
dflash_status dflash_paged_attn(
    const void* q, const uint8_t* k_codes, const uint8_t* v_codes,
    const float* k_scale, const float* v_scale, const int32_t* page_table,
    const int32_t* kv_len, const int32_t* q_len, int B, int Q, int Hq,
    int Hkv, int D, int page, int num_pages, int max_pages, int causal,
    float scale, dflash_dtype dt, void* out, float* lse, void* ws,
    size_t ws_bytes, dflash_stream_t s);

/* Workspace of dflash_sample for these sizes in bytes; 0 for invalid sizes. */
size_t dflash_sample_workspace_bytes(int R, int V);

/*
 * dflash_sample: one token from each of R rows of logits l, with that row's
 * temperature T, top-k, top-p and min-p, from a given uniform u; and the
 * filtered logits, on which dflash_verify is lossless for the filtered
 * target distribution ("Lossless, with conditions I did not used to state",
 * drafter's coat page).  Tokens are ranked by l descending, id ascending:
 *   x_v = exp((l_v - max l) * (1 / T)) in fp32 (1 at the maximum),
 *   w_v = floor(x_v 2^44), a 64-bit integer: sums of weights are exact, so
 *         neither their order nor the launch shape can change a result
 *   top-k (0 < k): the first k tokens
 *   top-p (p < 1): of those (total weight W), the tokens whose preceding
 *         tokens weigh less than ceil(p W) (products in fp64); never none
 *   min-p (0 < m, at most 1): of those, the tokens with x_v >= m
 *   token = the smallest id whose running kept weight, in id order, exceeds
 *         floor(u W'), W' the kept tokens' weight.
 * T = 0 keeps the first maximum only.
 *   logits [R, V] dtype, rows ld elements apart; temperature [R] fp32;
 *   top_k [R] int32, top_p, min_p [R] fp32: each may be NULL (filter off);
 *   u [R] fp32 in [0, 1)
 *   token [R] int32 out; n_kept [R] int32 out or NULL: tokens kept;
 *   filtered [R, V] fp32 out or NULL: l_v if kept, else -inf
 *   ws >= dflash_sample_workspace_bytes(R, V) bytes, 256-byte aligned
 * Requirements: R >= 1, 1 <= V < 2^20 (their weights add up in 64 bits),
 * ld >= V.  A NaN (left out) or +inf logit (weight 1, every other token's 0)
 * sets DFLASH_ERR_NONFINITE, as does a row with no logit above -inf (token
 * -1, n_kept 0) or a T that is negative or not finite (taken as 0).
 */
dflash_status dflash_sample(const void* logits, int64_t ld, dflash_dtype dt,
                            const float* temperature, const int32_t* top_k,
                            const float* top_p, const float* min_p,
                            const float* u, int R, int V, int32_t* token,
                            int32_t* n_kept, float* filtered, void* ws,
                            size_t ws_bytes, dflash_stream_t s);

/*
 * dflash_kv_append_axes: dflash_kv_append with positions of their own, one to
 * DFLASH_MAX_AXES of them for each token (time, height and width of images and
 * video; with one axis, the true positions of a sequence whose cache was
 * evicted, where slots are no positions any more).  Angle j of the token in row
 * r of q and k is that of row axis_pos[axis_of[j], r] of the tables:
 *   axis_pos [axes, B*Q] int32: the positions of every row (rows without a
 *            token are not read)
 *   axis_of  [rot/2] uint8: each angle's axis, in sections or in any other
 *            order; NULL with one axis
 *   pos      [B] int32: as in dflash_kv_append the slot of the first new token,
 *            but not its position; the slots are not bounded by max_pos
 * Everything else, results included, is as there.
 * Requirements: as dflash_kv_append; rot >= 8, 1 <= axes <= DFLASH_MAX_AXES,
 * axis_of 8-byte aligned.  On the device: a position outside [0, max_pos) (the
 * nearest row is taken) and an axis_of entry of `axes` or more (axis 0 is
 * taken) set DFLASH_ERR_BAD_INDEX.
 */
dflash_status dflash_kv_append_axes(
    const void* q, const void* k, const void* v, int64_t ld_q, int64_t ld_k,
    int64_t ld_v, const float* cos_tab, const float* sin_tab,
    const int32_t* axis_pos, const uint8_t* axis_of, int axes,
    const int32_t* pos, const int32_t* n_new, const int32_t* page_table,
    int B, int Q, int Hq, int Hkv, int D, int rot, int interleaved,
    int max_pos, int page, int num_pages, int max_pages, dflash_dtype dt,
    void* q_out, uint8_t* k_codes, uint8_t* v_codes, float* k_scale,
    float* v_scale, int32_t* kv_len, dflash_stream_t s);

/* Workspace of dflash_shared_attn for these sizes in bytes; 0 for invalid
 * sizes. */
size_t dflash_shared_attn_workspace_bytes(int B, int Q, int Hq, int Hkv,
                                          int D);

/*
 * dflash_shared_attn: dflash_paged_attn for a batch whose sequences all begin
 * with the same `shared` tokens, in the same pages (one system prompt, several
 * continuations of one request).  These are read once for the rows of all
 * sequences together, each sequence's own tokens as before.  Same arguments,
 * limits and results as dflash_paged_attn, up to the roundings of another
 * order: kv_len, q_len and the positions count the shared tokens, and a query
 * sees those of them at or before its own position (all of them below
 * kv_len[b] if not causal).
 *   shared      a whole number of pages, 0 for none; the first shared / page
 *               entries of page_table are read from the first sequence's row
 *               only, whatever the other rows hold there
 *   ws >= dflash_shared_attn_workspace_bytes(B, Q, Hq, Hkv, D) bytes, 256-byte
 *      aligned; its contents need no initialisation
 * Requirements, and what is flagged on the device: as dflash_paged_attn;
 * 0 <= shared <= max_pages * page, shared % page == 0.  Sizes (the page table's
 * width among them) with which the work, counted in 128 rows times 128 tokens,
 * could pass 2^31 give DFLASH_ERR_UNSUPPORTED.
 * With bf16 and D <= 128 the tensor cores compute: q is taken as fp16 relative
 * to its row's largest value (all of bf16's bits down to 2^-28 of it), a weight
 * times its value's scale as fp16 (to 2^-11 of itself or 2^-34 of its row's
 * largest, whichever is more); sums are fp32.
 */
dflash_status dflash_shared_attn(
    const void* q, const uint8_t* k_codes, const uint8_t* v_codes,
    const float* k_scale, const float* v_scale, const int32_t* page_table,
    const int32_t* kv_len, const int32_t* q_len, int shared, int B, int Q,
    int Hq, int Hkv, int D, int page, int num_pages, int max_pages,
    int causal, float scale, dflash_dtype dt, void* out, float* lse, void* ws,
    size_t ws_bytes, dflash_stream_t s);

/*
 * dflash_attn_mass: the attention weight that each cached token gets from a
 * block of queries, added to what it has gathered before.  For every sequence
 * b, key head h and slot t with first <= t < kv_len[b]:
 *     mass[b, h, t] = (t < fresh[b] ? decay * mass[b, h, t] : 0) +
 *         sum exp(scale * <q_ij, k_t> - lse[b, i, j])
 * over the queries i < q_len[b] that see t (causal or not, as in
 * dflash_paged_attn) and the heads j of the group that reads key head h.  lse
 * is what dflash_paged_attn or dflash_shared_attn gave for these queries, so
 * the weights are the softmax's own; a query that saw nothing (lse = -inf)
 * adds nothing.  Other slots of mass are left as they are.  Called after a
 * verify with the committed lengths and q_len = n + 1, it counts the accepted
 * queries only.
 *   lse   [B, Q, Hq] fp32;  fresh [B] int32: the slots from which on there is
 *         no weight yet (the length before the block), or NULL: kv_len
 *   first slots below it are not looked at, nor pages that end below it (those
 *         that an eviction keeps anyway, for example a prefix that sequences
 *         share, whatever their rows of page_table hold there)
 *   mass  [B, Hkv] rows of fp32, ld_mass elements apart, in/out
 * Sums and weights are fp32; their order is fixed, and nothing is added
 * atomically.  (bf16 and D <= 128, the tensor cores: q as two E4M3 numbers, all
 * of bf16's bits down to 2^-14 of its row's largest value, smaller values to
 * 2^-22 of that; queries below 2^111.)
 * Requirements: as dflash_paged_attn; first >= 0, ld_mass >= 1, decay finite;
 * work that could pass 2^31 tiles of 128 rows times 128 tokens gives
 * DFLASH_ERR_UNSUPPORTED.
 * On the device: as dflash_paged_attn; a kv_len beyond ld_mass sets
 * DFLASH_ERR_BAD_INDEX too (the length is clamped).
 */
dflash_status dflash_attn_mass(
    const void* q, const uint8_t* k_codes, const float* k_scale,
    const int32_t* page_table, const int32_t* kv_len, const int32_t* q_len,
    const float* lse, const int32_t* fresh, int first, int B, int Q, int Hq,
    int Hkv, int D, int page, int num_pages, int max_pages, int causal,
    float scale, float decay, dflash_dtype dt, float* mass, int64_t ld_mass,
    dflash_stream_t s);

/* Workspace of dflash_kv_evict for these sizes in bytes; 0 for invalid
 * sizes. */
size_t dflash_kv_evict_workspace_bytes(int B, int Hkv, int page, int budget);

/*
 * dflash_kv_evict: bounds each sequence's cache to `budget` tokens, in place.
 * A sequence with n = kv_len[b] > budget keeps, in every key head for itself,
 * the slots below `sink`, those from n - recent on, and of the others the
 * budget - sink - recent of largest mass (ties: the lower slot; a NaN is below
 * all numbers and sets DFLASH_ERR_NONFINITE).  The kept tokens move to slots
 * 0 .. budget - 1 in their order; keys stay turned by the positions that they
 * were appended with, so append to such a sequence with
 * dflash_kv_append_axes.  A sequence with n <= budget stays as it is.
 *   mass     [B, Hkv] rows of fp32, ld_mass elements apart
 *   mass_out [B, Hkv] rows, ld_out apart, or NULL: the kept slots' mass in
 *            their new places [0, new_len[b]); must not overlap mass
 *   new_len  [B] int32 out: min(n, budget); must not be kv_len itself
 *   kept     [B, Hkv, budget] int32 out or NULL: the old slot of every new
 *            one, -1 from new_len[b] on
 *   codes and scales as in dflash_kv_append, in/out.  A page of which any slot
 *   changes gets the least scale that its kept tokens need (a power of two
 *   s >= 2^-64 with max |x| <= 448 s) and their codes rounded to it (exact but
 *   for codes that become subnormal); other pages, and slots from new_len[b]
 *   on, are left as they are (the latter's scale may change).
 *   ws >= dflash_kv_evict_workspace_bytes(B, Hkv, page, budget) bytes, 256-byte
 *      aligned; its contents need no initialisation
 * Pages that this call changes belong to one sequence each: with a prefix that
 * sequences share, sink covers it.  Whole pages past new_len[b] are free.
 * Requirements: sink, recent >= 0, sink + recent <= budget, 1 <= budget <=
 * 2^30, ld_mass >= 1, ld_out at least what the new lengths can be; codes
 * 16-byte aligned; scales powers of two as dflash_kv_append writes them.  On
 * the device: kv_len below 0 or beyond the page table or ld_mass sets
 * DFLASH_ERR_BAD_INDEX (clamped), as does a page id outside [0, num_pages) (its
 * tokens count as zeros; such a page is not written).
 */
dflash_status dflash_kv_evict(
    const float* mass, int64_t ld_mass, uint8_t* k_codes, uint8_t* v_codes,
    float* k_scale, float* v_scale, const int32_t* page_table,
    const int32_t* kv_len, int B, int Hkv, int D, int page, int num_pages,
    int max_pages, int budget, int sink, int recent, float* mass_out,
    int64_t ld_out, int32_t* new_len, int32_t* kept, void* ws,
    size_t ws_bytes, dflash_stream_t s);

/*
 * dflash_logprobs: what R rows of logits l say about given tokens and about
 * themselves, with x = l / T:
 *   lse     [R] ln sum_v exp(x_v)
 *   logprob [R] x_token - lse, the token's log probability
 *   rank    [R] int32: the tokens before it in the order (l descending, id
 *           ascending); 0 is the most likely
 *   entropy [R] -sum_v p_v ln p_v, p = exp(x - lse)
 *   top, top_id [R, K]: log probabilities and ids of the first K tokens in that
 *           order; where fewer than K have a logit above -inf, -inf and -1
 *   logits [R, V] dtype, rows ld elements apart; temperature [R] fp32 or NULL
 *   (1); token [R] int32 or NULL; each output may be NULL, logprob and rank
 *   are without token, top and top_id with K = 0.  A token of -1 is none: its
 *   logprob is 0, its rank -1 (so rows of dflash_verify's out_tok can be given
 *   as they are).
 * Requirements: R >= 1, 1 <= V < 2^31 - 256, ld >= V, 0 <= K <=
 * DFLASH_MAX_ALTERNATIVES.  No workspace.
 * A NaN logit counts as -inf (as a given token: logprob NaN, rank -1).  A row
 * with a +inf logit (or an x above 2.3e38, whose bits pass fp32's range) has lse =
 * +inf, one without any logit above -inf lse = -inf; both have NaN for entropy and
 * log probabilities.  Those three, and a T that is below 2^-126 or not finite
 * (taken as 1), set DFLASH_ERR_NONFINITE; a token outside [-1, V) sets
 * DFLASH_ERR_BAD_INDEX (logprob NaN, rank -1).  Finite logits, a type's lowest
 * value among them, are none of these; weights of x beyond 2^29 in size are told
 * apart as far as their rounded values differ.
 */
dflash_status dflash_logprobs(
    const void* logits, int64_t ld, dflash_dtype dt, const float* temperature,
    const int32_t* token, int R, int V, int K, float* logprob, int32_t* rank,
    float* lse, float* entropy, float* top, int32_t* top_id,
    dflash_stream_t s);

/* Philox4x32-10 of n counters (ctr [n, 4] uint32, device) under key
 * (seed lo, seed hi) into out [n, 4] uint32 (device): the generator the
 * walk and verify draw from, exposed so callers can reproduce draws. */
dflash_status dflash_philox4x32(const uint32_t* ctr, uint64_t seed,
                                uint32_t* out, int64_t n, dflash_stream_t s);

/* Per-stage timing.  While set, the library records the caller's CUDA
 * events `begin` and `end` (cudaEvent_t, created by the caller) on the
 * call's stream right before and right after it launches the kernel of
 * `stage`:
 *   0 conv, 1 LM head with top-16 / logsumexp epilogue, 2 top-16 merge,
 *   3 pair score, 4 walk, 5 verify (row pass, accept tests and draw),
 *   6 E4M3 quantization of y (dflash_draft_e4m3).
 * In dflash_draft with bf16 storage and a conv, stage 0 is the conv with
 * the context gate and stage 3 the one launch that merges, scores and
 * walks (stages 2 and 4 are not recorded).
 * Calls captured into a CUDA graph record the events as event-record
 * nodes (cudaEventRecordExternal), stamped at every replay.
 * Pass NULL for both to stop.  Process-wide host state; set it from the
 * thread that makes the calls, not while other threads call the library.
 * Returns DFLASH_ERR_INVALID_ARG for an unknown stage or a lone NULL. */
dflash_status dflash_profile_stage(int stage, void* begin, void* end);

/* Limit, in nanoseconds, of the bounded waits inside the tensor-core
 * kernels of later launches: the conv, the single-CTA LM head (one row tile,
 * B*K <= 128), dflash_paged_attn, dflash_shared_attn and dflash_attn_mass give
 * up on a wait that runs longer, stop issuing work, let their copies and MMAs
 * in flight complete, free their TMEM and set DFLASH_ERR_DEVICE_TIMEOUT in the
 * device error word (their results are then invalid).  dflash_sample's waits
 * for the copies of a row do so too (that row's token is then -1).  0 restores
 * the default of 2 s, far beyond any real wait; the CTA-pair LM head always
 * uses it.  Process-wide host state, meant for tests of that failure path
 * ("Failure detection": a wait that never completes must end in a status the
 * host reads, not a hang).
 * Always returns DFLASH_OK. */
dflash_status dflash_set_wait_limit_ns(uint64_t ns);

/* Synchronise `s`, read and clear the device error word of the current
 * device; DFLASH_OK if no kernel reported a problem since the last call. */
dflash_status dflash_check(dflash_stream_t s);

/* Static, human-readable name of a status. */
const char* dflash_status_string(dflash_status st);

#ifdef __cplusplus
}
#endif
#endif /* DFLASH_H_ */
