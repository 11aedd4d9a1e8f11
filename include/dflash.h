/*
 * dflash.h -- C ABI of the block-draft hot path (sm_100a / B200).
 *
 * One draft cycle of a one-shot block drafter in four stages:
 *   dflash_conv2tap     two-tap block-local convolution
 *   dflash_lmhead_topk  LM head over the full vocabulary fused with
 *                       log-softmax and per-position top-16 selection
 *   dflash_path_select  pair scores of neighbouring candidates + max-sum walk
 *   dflash_verify       greedy verification (accepted length, next token)
 * and the walks and verification the pages describe beside the max-sum walk:
 *   dflash_path_walk        greedy or sampled walk from the last verified token
 *   dflash_verify_rejection rejection-sampling verification against the
 *                           target's distributions
 *   dflash_ctx_table,       the pages' context-gated pair scorer: its
 *   dflash_ctx_gate,        token tables, its gate, then its scores and a
 *   dflash_ctx_walk         walk
 * and what a serving program needs around a cycle:
 *   dflash_rmsnorm,         the norm in front of the LM head (bf16, or int8
 *   dflash_rmsnorm_i8         with a scale per row)
 *   dflash_quant_i8,        weights and activations in int8, and their
 *   dflash_gemm_i8            product
 *   dflash_token_logprobs,  log-probabilities of given tokens, or of the
 *   dflash_emitted_logprobs   tokens a verification step emitted
 *
 * Sources: "DFlash 2: Keep Drafting Parallel" (the blog, read in its Chinese
 * translation) and "Inco AI's DFlash 2 lifts LLM decoding output 16-25%".
 *
 * Conventions shared by every entry point
 *   - Pointers are device pointers owned by the caller unless a parameter
 *     says "host".  The library allocates no memory and keeps no state
 *     between calls, so calls on different streams are independent.
 *   - bf16 values are passed as their 16-bit patterns (dflash_bf16).
 *   - All arrays are row-major and contiguous.  Token rows of a batch of
 *     B blocks with L drafted positions are ordered b*L + i.
 *   - `stream` is a cudaStream_t passed as void* (NULL = legacy stream).
 *     Calls only enqueue work; the return code covers host-side argument
 *     checks and launch errors.  Errors found on the device (a bounded wait
 *     that ran out, an out-of-range token index) are written with atomicCAS
 *     into `dev_status` (a device int the caller zeroes; NULL = not recorded).
 *   - Every device-side wait is bounded (default 2000 ms; the environment
 *     variable DFLASH_TIMEOUT_MS, read once per process, overrides it, and
 *     DFLASH_TIMEOUT_NS, read at every call, overrides both); a kernel that
 *     gives up records DFLASH_ERR_TIMEOUT, drains the copies and tensor-core
 *     operations it has in flight, releases its tensor memory and returns
 *     instead of hanging.  The outputs of such a call are not valid; the
 *     context stays usable for the next call.
 */
#ifndef DFLASH_H_
#define DFLASH_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef uint16_t dflash_bf16;

enum dflash_status {
  DFLASH_OK = 0,
  DFLASH_ERR_INVALID_ARG = 1,   /* null pointer, bad size, K != 16, ... */
  DFLASH_ERR_UNSUPPORTED = 2,   /* valid request this build cannot run */
  DFLASH_ERR_CUDA = 3,          /* a CUDA runtime/driver call failed */
  DFLASH_ERR_WORKSPACE = 4,     /* workspace smaller than required */
  DFLASH_ERR_TIMEOUT = 5,       /* device: a bounded wait gave up */
  DFLASH_ERR_BAD_INDEX = 6      /* device: a token index outside [0, V) */
};

/* Static text for a status code (never NULL). */
const char* dflash_status_string(int status);

/* Identity of the sources this library was compiled from: the first 16 hex
 * digits of a SHA-256 over the CUDA sources, headers and compile flags
 * (computed by the package's build script), or "unhashed" for a build made
 * without it.  Static text, never NULL; no GPU is touched.  The library's
 * own bookkeeping, not a computation of the pages, so it cites none. */
const char* dflash_build_id(void);

/*
 * Two-tap block-local convolution.
 * "DFlash 2: Keep Drafting Parallel", section "a lightweight local
 * convolution", formula Conv_k(x)_t = k_{t,0} * x_t + k_{t,1} * x_{t-1}, and
 * Figure 4: each position mixes with its predecessor inside the block; the
 * first position reads the last verified token's representation.  Here the
 * taps are the static per-channel base taps a0, a1.
 *
 *   y[b,t,c] = a0[c] * x[b,t,c] + a1[c] * x[b,t-1,c],  x[b,-1,c] = prev[b,c]
 *
 * x    [B, P, d] bf16        prev [B, d] bf16 (NULL: zeros)
 * a0   [d] bf16              a1   [d] bf16
 * y    [B, P, d] bf16 out    (fp32 arithmetic, rounded to nearest even)
 * Requires B, P, d >= 1 and d % 8 == 0 (16-byte rows); y must not overlap x.
 */
int dflash_conv2tap(const dflash_bf16* x, const dflash_bf16* prev, const dflash_bf16* a0,
                    const dflash_bf16* a1, dflash_bf16* y, int B, int P, int d, void* stream);

/*
 * Two-tap conv with content-dependent taps.
 * "DFlash 2: Keep Drafting Parallel", section "a lightweight local
 * convolution": each coefficient is a learnable base kernel plus a small
 * correction computed from the current hidden state, one correction shared
 * by every 16 channels.  With G = d / 16 and the correction projection
 * Wc [2G, d] (rows 0..G-1: tap 0, rows G..2G-1: tap 1):
 *   delta_j[b,t,g] = sum_c x[b,t,c] * Wc[j*G + g, c]
 *   y[b,t,c] = (a0[c] + delta_0[b,t,c/16]) * x[b,t,c]
 *            + (a1[c] + delta_1[b,t,c/16]) * x[b,t-1,c],  x[b,-1,:] = prev[b,:]
 * x [B,P,d], prev [B,d] (NULL: zeros), a0, a1 [d], Wc [2G,d], y [B,P,d]: bf16.
 * ws: device workspace of dflash_conv2tap_dynamic_workspace(B,P,d) bytes
 * (holds delta in fp32).  d % 16 == 0, d >= 128; all pointers 16-byte
 * aligned.  Runs the tensor-core GEMM for delta, then a streaming kernel.
 */
size_t dflash_conv2tap_dynamic_workspace(int B, int P, int d);
int dflash_conv2tap_dynamic(const dflash_bf16* x, const dflash_bf16* prev, const dflash_bf16* a0,
                            const dflash_bf16* a1, const dflash_bf16* wc, dflash_bf16* y, int B, int P, int d,
                            void* ws, size_t ws_bytes, void* stream);

/*
 * Bytes of device workspace dflash_lmhead_topk needs for these sizes
 * (0 when the sizes are invalid).
 */
size_t dflash_lmhead_topk_workspace(int M, int V, int d);

/*
 * LM head + log-softmax + top-16 per row, without writing logits to memory.
 * "DFlash 2: Keep Drafting Parallel", section "the right token is already in
 * the candidates" and Table 1 (each drafted position keeps its 16 best
 * candidates), section "a lightweight path selector" (the candidates are
 * scored without another LM-head pass).
 *
 *   z[m,v] = sum_k H[m,k] * W[v,k]     (bf16 inputs, fp32 accumulation)
 *   lse[m] = log sum_v exp(z[m,v])
 *   topk_idx[m,:]  = the 16 largest z[m,:], value descending, ties to the
 *                    lowest vocabulary index
 *   topk_logp[m,k] = z[m, topk_idx[m,k]] - lse[m]
 *
 * H [M, d] bf16, W [V, d] bf16 (both K-major, 16-byte aligned base).
 * topk_logp [M, 16] fp32 out, topk_idx [M, 16] int32 out, lse [M] fp32 out
 * (NULL: not written).  ws: device workspace of at least
 * dflash_lmhead_topk_workspace(M, V, d) bytes, 256-byte aligned; its contents
 * need no initialisation.  K must be 16, d % 8 == 0, M >= 1, V >= 16.
 * Two kernels run on `stream`: the fused GEMM + epilogue (tcgen05 / TMEM /
 * TMA) and the cross-CTA merge of the per-CTA partial lists.
 */
int dflash_lmhead_topk(const dflash_bf16* H, const dflash_bf16* W, int M, int V, int d, int K,
                       float* topk_logp, int32_t* topk_idx, float* lse, void* ws, size_t ws_bytes,
                       int* dev_status, void* stream);

/* Size of the library-owned scratch array used by dflash_lmhead_topk_static. */
#define DFLASH_STATIC_SCRATCH_BYTES (8u << 20)

/*
 * dflash_lmhead_topk without a caller workspace.  The paper has no
 * counterpart to this entry point.  For callers that cannot
 * allocate device memory when they call, e.g. code inside an allocator's own
 * hooks or engines whose device memory is all reserved up front.  Same inputs,
 * outputs and results as dflash_lmhead_topk; the partial records go to a
 * library-owned device array of DFLASH_STATIC_SCRATCH_BYTES (8 MiB), which
 * every GPU that loads the library holds until the process exits.
 *
 * Limit: dflash_lmhead_topk_workspace(M, V, d) must not exceed
 * DFLASH_STATIC_SCRATCH_BYTES, else the call returns DFLASH_ERR_UNSUPPORTED
 * (M <= 128 at V = 151,936 fits; large-M shapes generally do not).
 * The first call on each device looks up the array's device address
 * (cudaGetSymbolAddress) with that device current, so make that first call
 * before any stream capture.  The address is kept per device and CUDA
 * context: after cudaDeviceReset (a new context, the array at a new address)
 * the next call looks it up again.  Calls share the array: calls that may overlap
 * on the GPU (different streams or threads on one device) race and must be
 * serialised by the caller.  The call allocates no memory.
 */
int dflash_lmhead_topk_static(const dflash_bf16* H, const dflash_bf16* W, int M, int V, int d, int K,
                              float* topk_logp, int32_t* topk_idx, float* lse, int* dev_status,
                              void* stream);

/*
 * Diagnostic: the same GEMM path as dflash_lmhead_topk, but writing the raw
 * logits z [M, V] fp32 (row-major) instead of selecting.  Meant for small
 * shapes in tests; not part of the fused hot path.
 */
int dflash_lmhead_logits_debug(const dflash_bf16* H, const dflash_bf16* W, int M, int V, int d,
                               float* z, void* ws, size_t ws_bytes, int* dev_status, void* stream);

/*
 * Plain bf16 GEMM on the LM head's tensor-core path:
 *   C[m,n] = sum_k A[m,k] * B[n,k]      (fp32 accumulation, fp32 out)
 * A [M, K] bf16, B [N, K] bf16 (both K-major, 16-byte aligned), C [M, N] fp32
 * row-major (16-byte aligned).  K % 8 == 0, N >= 16.  Needs no workspace.
 * When M <= 128 and N is small next to the SM count, K is split across
 * CTAs whose fp32 partial sums are added into C (zeroed first on `stream`):
 * results then agree with the unsplit sum to fp32 rounding, not bit for bit
 * from run to run.  It computes the projections of the dynamic conv's tap corrections and of
 * the context-gated pair scorer ("DFlash 2: Keep Drafting Parallel",
 * sections "a lightweight local convolution" and "a lightweight path
 * selector").
 */
int dflash_gemm_bf16(const dflash_bf16* A, const dflash_bf16* B, float* C, int M, int N, int K, void* stream);

/*
 * Path selection over the candidate lists.
 * "DFlash 2: Keep Drafting Parallel", section "a lightweight path selector":
 * all adjacent candidate pairs are scored at once, then one serial walk over
 * the precomputed scores picks the path.  The pages' trained scorer is not
 * published; this entry point computes the stand-in
 *
 *   S_i[j,k] = lp[i,j] + lp[i+1,k] + e_{c_ij} . Msel . e_{c_{i+1,k}}
 *
 * and walks it with max-sum (Viterbi): delta_0 = 0,
 * delta_{i+1}[k] = max_j delta_i[j] + S_i[j,k] (ties: lowest j); the path ends
 * at argmax_k delta_{L-1}[k] (ties: lowest k).  L = 1: slot 0, score 0.
 *
 * topk_logp [B*L, 16] fp32, topk_idx [B*L, 16] int32 (values in [0, V))
 * E [V, r] bf16, Msel [r, r] bf16;  r % 8 == 0, 8 <= r <= 128; 1 <= L <= 16.
 * path_tok [B, L] int32 out; path_slot [B, L] int32 out (NULL: not written);
 * path_score [B] fp32 out (NULL: not written); pair_scores_dbg
 * [B, L-1, 16, 16] fp32 out (NULL: not written).  An index outside [0, V)
 * records DFLASH_ERR_BAD_INDEX and is read as index 0.
 */
int dflash_path_select(const float* topk_logp, const int32_t* topk_idx, const dflash_bf16* E,
                       const dflash_bf16* Msel, int B, int L, int K, int r, int V,
                       int32_t* path_tok, int32_t* path_slot, float* path_score,
                       float* pair_scores_dbg, int* dev_status, void* stream);

/*
 * dflash_path_select followed by greedy verification of the selected path,
 * in one kernel ("DFlash 2: Keep Drafting Parallel", section "a lightweight
 * path selector" and Table 1's caption): the same outputs as
 * dflash_path_select (without the pair-score dump) plus, for the chosen
 * path, accept_len [B] and next_token [B] exactly as dflash_verify defines
 * them against target [B, L+1] int32.  1 <= L <= 16.
 */
int dflash_select_verify(const float* topk_logp, const int32_t* topk_idx, const dflash_bf16* E,
                         const dflash_bf16* Msel, const int32_t* target, int B, int L, int K, int r, int V,
                         int32_t* path_tok, int32_t* path_slot, float* path_score, int32_t* accept_len,
                         int32_t* next_token, int* dev_status, void* stream);

/*
 * Vocabulary-parallel LM head: each rank owns rows [v_offset, v_offset + V)
 * of the full head and produces per-row partial records; the records of all
 * ranks, gathered in rank order, merge into the full vocabulary's top-16.
 * Same definition as dflash_lmhead_topk over the concatenated head.
 *
 * dflash_lmhead_topk_records(M, V, d): records per row P that a call with
 * this shard shape writes (0 if unsupported).  Every rank of one gather must
 * use the same P: pad a shorter rank's buffer with empty records (m = -inf,
 * s = 0, values -inf, indices 0x7fffffff), which the merge ignores.
 *
 * dflash_lmhead_topk_partial: the GEMM + online log-sum-exp + top-16 kernel
 * alone over W [V, d] (this rank's shard); writes records [M][P] into
 * `records` (dflash_lmhead_topk_workspace(M, V, d) bytes, 256-byte aligned)
 * with every vocabulary index shifted by v_offset >= 0.  A record is 36
 * 32-bit words: running max, sum of exp(z - max), 2 unused, the 16 best
 * values (descending), their 16 indices (int32 bits).
 *
 * dflash_lmhead_topk_merge: records [nrank][M][P] (16-byte aligned) ->
 * topk_logp, topk_idx [M, 16], lse [M] (nullable), exactly as
 * dflash_lmhead_topk's own merge.  K must be 16.
 */
int dflash_lmhead_topk_records(int M, int V, int d);
int dflash_lmhead_topk_partial(const dflash_bf16* H, const dflash_bf16* W, int M, int V, int d, int v_offset,
                               void* records, size_t records_bytes, int* dev_status, void* stream);
int dflash_lmhead_topk_merge(const void* records, int M, int P, int nrank, int K, float* topk_logp,
                             int32_t* topk_idx, float* lse, void* stream);

/*
 * Walk from the last verified token.
 * "DFlash 2: Keep Drafting Parallel", section "a lightweight path selector":
 * starting from the last verified token, the walk over the precomputed pair
 * scores greedily follows the best successor, or draws each successor from
 * the same scores.  With the anchor a = anchor[b] and the stand-in scores
 *   S_a[k]    = lp[b*L, k] + e_a . M . e_{c_0k}            (no unary term for a)
 *   S_i[j,k]  = lp[b*L+i, j] + lp[b*L+i+1, k] + e_{c_ij} . M . e_{c_{i+1,k}}
 * the walk picks slot s_0 from S_a and s_{i+1} from row S_i[s_i, :]:
 *   uniforms == NULL  greedy: the argmax (ties: lowest slot);
 *   otherwise         sampling: q = softmax(row / temperature) over the 16
 *                     slots, s = the smallest slot whose cumulative q exceeds
 *                     uniforms[b*L+i] (inverse CDF in slot order).
 *
 * topk_logp, topk_idx [B*L, 16] as from dflash_lmhead_topk; E [V, r] bf16,
 * Msel [r, r] bf16 (16-byte aligned); anchor [B] int32; uniforms [B, L] fp32
 * in [0, 1) or NULL; temperature > 0 (sampling only).
 * Outputs: path_tok [B, L] int32; path_slot [B, L] int32 (nullable);
 * path_score [B] fp32 (nullable; S_a[s_0] + sum_i S_i[s_i, s_{i+1}]);
 * path_q [B, L, 16] fp32 (nullable; sampling only: the distribution each slot
 * was drawn from, what dflash_verify_rejection needs as draft_q).
 * target [B, L+1] int32 (nullable): if given, the path is verified greedily
 * as dflash_verify does, into accept_len [B] and next_token [B].
 * 1 <= L <= 16, 8 <= r <= 128, r % 8 == 0.  An anchor or candidate index
 * outside [0, V) is read as 0 and records DFLASH_ERR_BAD_INDEX.
 */
int dflash_path_walk(const float* topk_logp, const int32_t* topk_idx, const dflash_bf16* E,
                     const dflash_bf16* Msel, const int32_t* anchor, const float* uniforms,
                     float temperature, int B, int L, int K, int r, int V, int32_t* path_tok,
                     int32_t* path_slot, float* path_score, float* path_q, const int32_t* target,
                     int32_t* accept_len, int32_t* next_token, int* dev_status, void* stream);

/*
 * Rejection-sampling verification of a sampled path.
 * "DFlash 2: Keep Drafting Parallel", section "a lightweight path selector",
 * and "Inco AI's DFlash 2 lifts LLM decoding output 16-25%": rejection
 * sampling restores the target's exact output distribution.  Standard
 * speculative sampling, with p_i = softmax(target_logits[b*(L+1)+i] / T) and
 * q_i = draft_q[b*L+i] (on the candidates cand_idx[b*L+i]):
 *   position i is kept while u_accept[b*L+i] * q_i[s_i] <= p_i(draft[b*L+i]);
 *   with n the first rejected position (n = L if none), accept_len[b] = n + 1
 *   and next_token[b] is drawn from max(0, p_n - q_n) (n < L) or from p_L
 *   (n = L) by inverse CDF in vocabulary order: the smallest token whose
 *   cumulative mass exceeds u_resample[b] times the total mass.
 * The draw's 8192-token slice is chosen from fp64 sums of fp32 exponentials
 * and the token inside it from fp64 exponentials; a uniform that falls within
 * about 1e-7 (relative) of a cumulative boundary may land on either side.
 *
 * target_logits [B*(L+1), V] fp32 (finite or -inf); temperature > 0 (the
 * same one the draft was sampled at); draft, draft_slot [B, L] int32 (the
 * path and its slots, as from dflash_path_walk); cand_idx [B*L, 16] int32
 * (distinct per row); draft_q [B, L, 16] fp32; u_accept [B, L] and
 * u_resample [B] fp32 uniforms in [0, 1).  accept_len, next_token [B] int32
 * out.  ws: device workspace of dflash_verify_rejection_workspace(B, L, V)
 * bytes, 16-byte aligned (the slice statistics; no initial contents needed).
 * 1 <= L <= 31, 1 <= V <= 524288.  A draft token or slot out of range
 * records DFLASH_ERR_BAD_INDEX and is clamped.
 */
size_t dflash_verify_rejection_workspace(int B, int L, int V);
int dflash_verify_rejection(const float* target_logits, float temperature, const int32_t* draft,
                            const int32_t* draft_slot, const int32_t* cand_idx, const float* draft_q,
                            const float* u_accept, const float* u_resample, int B, int L, int V,
                            int32_t* accept_len, int32_t* next_token, void* ws, size_t ws_bytes,
                            int* dev_status, void* stream);

/*
 * The pages' context-gated pair scorer, part 1: the token tables and the gate.
 * "DFlash 2: Keep Drafting Parallel", section "a lightweight path selector":
 * S_t(a, b) = U_t(b) + <A(a) (.) H(h_t), B(b)>, compact token embeddings A, B
 * matched under a context gate H.  Read here as A(a) = Pa.emb(a),
 * B(b) = Pb.emb(b), H(h_t) = sigmoid(Pg.h_t), emb(v) = Emb[v].
 *
 * A and B depend on the token alone, so they are tabulated once for the whole
 * vocabulary (whenever Emb or Pab change) and every cycle only reads rows:
 *   dflash_ctx_table: tab [V, 2e] fp32 = Emb . Pab^T -- row v holds A(v) in
 *     columns 0..e-1 and B(v) in columns e..2e-1.  Emb [V, d] bf16, Pab
 *     [2e, d] bf16 (rows 0..e-1 = Pa, e..2e-1 = Pb).
 *   dflash_ctx_gate: gate [M, e] fp32 = H . Pg^T (before the sigmoid), H
 *     [M = B*L, d] bf16 (the drafted positions' hidden states), Pg [e, d]
 *     bf16.  It needs only H, so a caller can run it on another stream
 *     while the LM head runs.
 * Both run on the library's tensor-core GEMM (dflash_gemm_bf16; its rules
 * on alignment apply).  d % 8 == 0, 16 <= e <= 1024, e % 8 == 0.
 */
int dflash_ctx_table(const dflash_bf16* Emb, const dflash_bf16* Pab, int V, int d, int e, float* tab, void* stream);
int dflash_ctx_gate(const dflash_bf16* H, const dflash_bf16* Pg, int M, int d, int e, float* gate, void* stream);

/*
 * The pages' context-gated pair scorer, part 2: scores and a walk from the
 * last verified token (same section).  Table t (0 <= t < L) scores
 *   S_t[j][k] = topk_logp[b*L+t][k] + sum_q A(pred_j)[q] sigmoid(gate[b*L+t][q]) B(c_tk)[q]
 * where pred_j is the anchor for t = 0 (every row j alike) and candidate j of
 * position t-1 otherwise (U_t enters as the log-probability: a per-position
 * constant that no walk's choice depends on).  walk: 0 = max-sum from the
 * anchor (ties: lowest slot), 1 = greedy, 2 = sampled at `temperature` with
 * one uniform per drafted position (as dflash_path_walk).
 * Inputs from dflash_lmhead_topk, dflash_ctx_table (tab [V, 2e]) and
 * dflash_ctx_gate; tab, gate 16-byte aligned.  A token index outside [0, V)
 * is read as 0 and records DFLASH_ERR_BAD_INDEX.  Outputs: path_tok [B, L]; path_slot [B, L], path_score [B]
 * (the sum of the chosen entries), path_q [B, L, 16] (sampling only) and
 * tables_dbg [B, L, 16, 16] are nullable; target [B, L+1] (nullable) adds
 * greedy verification into accept_len, next_token [B].  K must be 16.
 */
int dflash_ctx_walk(const float* topk_logp, const int32_t* topk_idx, const int32_t* anchor, const float* tab,
                    const float* gate, int B, int L, int K, int e, int V, int walk, const float* uniforms,
                    float temperature, int32_t* path_tok, int32_t* path_slot, float* path_score, float* path_q,
                    float* tables_dbg, const int32_t* target, int32_t* accept_len, int32_t* next_token,
                    int* dev_status, void* stream);

/*
 * Greedy verification.
 * "DFlash 2: Keep Drafting Parallel", Table 1 caption: the accepted length
 * includes the verifier's next token.  With n the first i where
 * draft[b,i] != target[b,i] (n = L if none):
 *   accept_len[b] = n + 1,  next_token[b] = target[b, n].
 *
 * draft [B, L] int32, target [B, L+1] int32 (the target's argmax tokens at
 * the L drafted positions and the bonus position).  accept_len [B] int32 out,
 * next_token [B] int32 out.  1 <= L <= 32.
 */
int dflash_verify(const int32_t* draft, const int32_t* target, int B, int L, int32_t* accept_len,
                  int32_t* next_token, void* stream);

/*
 * Root-mean-square norm with the residual's addition.
 * The norm that makes the LM head's input H; the paper has no counterpart to
 * this entry point (its drafter's layers are not published).  Per row m:
 *   h = bf16(x + residual)   (fp32 sum, rounded to nearest even; h = x
 *                             without a residual)
 *   r = 1 / sqrt(mean_c h[c]^2 + eps)            (fp32)
 *   y[c] = bf16(h[c] * gamma[c] * r)
 * x, residual, h, y [M, d] bf16; gamma [d] bf16; residual NULL: none, and h
 * must be NULL then; h NULL: the sum is not written.  h and y may each be the
 * same array as x or as residual (not each other); any other overlap is not
 * allowed.  A sum of squares beyond fp32's range is taken in fp64, and the
 * products h * gamma stay in range for every |gamma| < 2^64; products below
 * 2^-126 are rounded as fp32 rounds them.
 * Requires M >= 1, 8 <= d <= 32768, d % 8 == 0, eps finite and >= 1e-20,
 * 16-byte aligned pointers.
 */
int dflash_rmsnorm(const dflash_bf16* x, const dflash_bf16* residual, const dflash_bf16* gamma, float eps, int M,
                   int d, dflash_bf16* h, dflash_bf16* y, void* stream);

/*
 * The same norm with its output in int8 and one scale per row, as
 * dflash_gemm_i8 takes it (no counterpart in the paper).  With
 * a = max_c |h[c] * gamma[c]|:
 *   scale = a * r / 127,  q[c] = rint(127 * h[c] * gamma[c] / a)
 * (r cancels in q; halves round to even, decided exactly), so that
 * q * scale is the normalised row to within half a step.  q is in
 * [-127, 127].  A row with a < 2^-100 gives q = 0 and scale = 0; a row that
 * holds a NaN or an infinity (or where gamma makes one, from |gamma| of 2^64
 * on) gives q = 0 and scale = NaN, which a product taken from it carries on.
 * q [M, d] int8 (8-byte aligned), scale [M] fp32; the rest as dflash_rmsnorm.
 */
int dflash_rmsnorm_i8(const dflash_bf16* x, const dflash_bf16* residual, const dflash_bf16* gamma, float eps, int M,
                      int d, dflash_bf16* h, int8_t* q, float* scale, void* stream);

/*
 * Rows to int8 with one scale each: dflash_rmsnorm_i8 without the norm
 * (h = x, gamma = 1, r = 1; no counterpart in the paper).  Lays a weight
 * matrix out for dflash_gemm_i8 (a scale per output channel), or quantises
 * activations that are normed already.  x [M, d] bf16, q [M, d] int8,
 * scale [M] fp32; sizes and alignment as dflash_rmsnorm_i8.
 */
int dflash_quant_i8(const dflash_bf16* x, int M, int d, int8_t* q, float* scale, void* stream);

/*
 * Matrix product in 8-bit integers with a scale per token and per channel
 * (the 8-bit counterpart of dflash_gemm_bf16; none in the paper):
 *   C[m,n] = float(sum_k A[m,k] * B[n,k]) * sa[m] * sb[n]
 * The sum is exact in int32 (K <= 131071 cannot overflow it); it is rounded
 * once to fp32 and each product with a scale rounds once more, then once to
 * the output type.  Scales are used as they are (a NaN scale makes its row or
 * column NaN).
 * A [M, K], B [N, K] int8 (K-major, 16-byte aligned), sa [M], sb [N] fp32
 * (4-byte aligned), C [M, N] row-major: fp32 (c_bf16 == 0) or bf16
 * (c_bf16 == 1), aligned to its element.  M, N >= 1, 16 <= K <= 131071,
 * K % 16 == 0; C must not overlap an input.  Needs no workspace; results are
 * the same bit for bit from run to run.
 */
int dflash_gemm_i8(const int8_t* A, const float* sa, const int8_t* B, const float* sb, void* C, int c_bf16, int M,
                   int N, int K, int* dev_status, void* stream);

/*
 * Log-probabilities of given tokens, with entropy, rank and the top
 * alternatives, from logits in memory (no counterpart in the paper; a
 * serving program answers with them).  Row m, z = logits[m*ld .. m*ld + V):
 *   lse      = log sum_v exp(z[v] / T)
 *   logp     = z[t] / T - lse,  t = tokens[m]
 *   rank     = 1 + number of v with z[v] > z[t]
 *   entropy  = -sum_v p[v] log p[v],  p = exp(z / T - lse)   (nats)
 *   top_idx  = the K largest z, value descending, ties to the lowest index;
 *   top_logp = their log-probabilities
 * With K = 16 top_logp and top_idx are the candidate lists
 * dflash_path_select and the walks take.
 *
 * logits: fp32 (z_bf16 == 0) or bf16 (z_bf16 == 1) rows of V elements, ld
 * elements apart (ld >= V), aligned to the element.  -inf masks a token
 * (log-probability -inf, no entropy); in a row with nothing but -inf, lse and
 * every log-probability are -inf, the entropy is 0.  Finite masks of any size
 * are values like others (a row of nothing but one is uniform).  A row whose
 * largest value lies beyond +-1.8e8 T is read a second time.  A NaN or +inf in
 * a row makes its lse, entropy and log-probabilities NaN; a NaN counts as the
 * largest value in top_idx.
 * tokens [M] int32: a negative one marks a row that is not asked for (padding
 * of a batch): its outputs keep what they held (its logits may be read, with
 * no effect).  A token
 * >= V records DFLASH_ERR_BAD_INDEX; its row gets logp = NaN and rank = 0 and
 * the rest as usual.  tokens NULL: no tokens (every row is asked for; logp
 * and rank must be NULL).
 * logp, entropy, lse [M] fp32, rank [M] int32, top_logp [M, K] fp32, top_idx
 * [M, K] int32; every output is nullable (top_logp and top_idx: both or
 * neither; neither when K == 0).  1 <= M, 1 <= V <= 16777216,
 * 0 <= K <= min(32, V), 1e-6 <= T = temperature <= 1e6.  Log-probabilities
 * are never above 0 and entropies never below it.  Sums are fp32 within
 * a warp and fp64 across warps; results are the same bit for bit from run to
 * run.
 */
int dflash_token_logprobs(const void* logits, int z_bf16, long long ld, int M, int V, const int32_t* tokens,
                          float temperature, int K, float* logp, int32_t* rank, float* entropy, float* lse,
                          float* top_logp, int32_t* top_idx, int* dev_status, void* stream);

/*
 * dflash_token_logprobs for the tokens a verification step emits: block b's
 * rows b*(L+1) + i of target_logits (as dflash_verify_rejection takes them,
 * or bf16, or ld elements apart) with
 *   token = draft[b,i] for i < accept_len[b] - 1,
 *   token = next_token[b] for i = accept_len[b] - 1;
 * the outputs of the rows behind that keep what they held.
 * draft [B, L], accept_len, next_token [B] int32 as dflash_verify and
 * dflash_verify_rejection give them; an accept_len outside [1, L+1] records
 * DFLASH_ERR_BAD_INDEX and is clamped; a token outside [0, V) records it too,
 * its row as dflash_token_logprobs says.  Outputs [B, L+1] and [B, L+1, K].
 * 1 <= B, 1 <= L <= 32.
 */
int dflash_emitted_logprobs(const void* target_logits, int z_bf16, long long ld, int B, int L, int V,
                            const int32_t* draft, const int32_t* accept_len, const int32_t* next_token,
                            float temperature, int K, float* logp, int32_t* rank, float* entropy, float* lse,
                            float* top_logp, int32_t* top_idx, int* dev_status, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* DFLASH_H_ */
