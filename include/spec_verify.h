/*
 * spec_verify.h -- C ABI of the GB300 (sm_103a) verification step of speculative sampling.
 *
 * The operation is the target-side modified rejection sampling of
 * "Accelerating Large Language Model Decoding with Speculative Sampling"
 * (Chen et al., DeepMind), as summarised by the wikillm.com paper card:
 *   - §4.2 "Decoding transforms": the temperature transform softmax(l / T) is
 *     applied to both the target rows q and the draft rows p before anything else;
 *   - §4.2 "Modified rejection sampling" and Algorithm 2 step 3: draft token
 *     x~_t is accepted, left to right, while u_t < min(1, q(x~_t) / p(x~_t));
 *     at the first rejection one token is drawn from the normalised residual
 *     (q - p)_+ = max(0, q - p) / sum max(0, q - p), and the scan stops;
 *   - Algorithm 2 step 4 and the card's Pitfalls ("Bonus-token typo"): if all K
 *     drafts are accepted, one bonus token is drawn from the (K+1)-th target row;
 *   - the card's Pitfalls ("The residual distribution needs care"): a residual
 *     that sums to zero falls back to q itself.
 * Each sequence therefore emits between 1 and K+1 tokens (§4.2).
 *
 * Conventions the pages leave open, fixed here:
 *   - uniforms[b, t], t < K, drives the test of draft t; uniforms[b, K] drives
 *     the residual draw; uniforms[b, K+1] drives the bonus draw;
 *   - the test is strict (u < min(1, q/p)); p(x~) = 0 with q(x~) > 0 accepts,
 *     q(x~) = 0 rejects;
 *   - a draw from weights w with uniform u is the inverse CDF over ascending
 *     token id: the smallest i with w_0 + ... + w_i > u * sum(w); when no
 *     such i exists (u = 1) the largest i with w_i > 0 is taken;
 *   - -inf logits are masked entries (probability 0).
 *
 * All entry points are plain C. Pointers marked "device" must point to memory
 * of the current CUDA device; the library never allocates, frees or keeps
 * pointers between calls. Work is enqueued on `stream` (a cudaStream_t passed
 * as void*; NULL means the legacy default stream) and runs asynchronously.
 *
 * A call enqueues a memset of the workspace's control block and then either
 *   - two kernels: the streaming kernel, then the draw kernel as its
 *     programmatic dependent (launched while the streaming grid drains, and
 *     waiting on the device for it to complete); or, for calls streaming
 *     between 16 MiB and 1 GiB of logits,
 *   - one fused kernel whose CTAs take tickets: streaming work first, then the
 *     draw of each sequence, which waits on the device for that sequence's
 *     plan. The wait is bounded: after 200 ms it sets SV_DEV_TIMEOUT and the
 *     kernel winds down.
 * Make the first call on a device before capturing a stream into a CUDA graph.
 */
#ifndef SPEC_VERIFY_H_
#define SPEC_VERIFY_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* Element types. SV_E4M3 is a type of the key/value cache only. */
enum {
  SV_BF16 = 0, /* bfloat16 */
  SV_F32 = 1,  /* IEEE fp32 */
  SV_E4M3 = 2  /* 8-bit float, 4 exponent and 3 mantissa bits, largest value 448 */
};

/* Host-side return codes (no work is enqueued when one of these is returned). */
enum {
  SV_OK = 0,
  SV_ERR_NULL = 1,        /* a required pointer is NULL */
  SV_ERR_SHAPE = 2,       /* B < 0, K outside [1, 64], V outside [1, 2^31 - 1], or sizes overflow */
  SV_ERR_TEMPERATURE = 3, /* temperature not finite or not > 0 */
  SV_ERR_DTYPE = 4,       /* dtype is neither SV_BF16 nor SV_F32 */
  SV_ERR_ALIGN = 5,       /* a pointer is not aligned to its element (workspace: 256 bytes) */
  SV_ERR_WORKSPACE = 6,   /* workspace_bytes below sv_workspace_size(), or staging too small */
  SV_ERR_CUDA = 7,        /* a CUDA runtime call failed */
  SV_ERR_SCRATCH_LIMIT = 8 /* spec_verify_static: the problem needs more than its fixed scratch */
};

/* Size of the fixed device scratch array behind spec_verify_static. */
#define SV_STATIC_SCRATCH_BYTES (8u << 20)

/* Device-side status bits, OR-ed into the status word of the workspace. A
 * sequence that raises one of the first four gets out_tokens[b, :] = -1 and
 * n_accepted[b] = -1; other sequences are unaffected. */
enum {
  SV_DEV_TOKEN_RANGE = 16,   /* a draft token outside [0, V) */
  SV_DEV_NONFINITE = 32,     /* a logit row holds NaN or +inf */
  SV_DEV_EMPTY_ROW = 64,     /* a logit row is entirely -inf */
  SV_DEV_UNIFORM_RANGE = 128,/* a uniform is NaN or outside [0, 1] */
  SV_DEV_TIMEOUT = 256,      /* a bounded wait in a kernel ran out (results invalid) */
  SV_DEV_SLOT_RANGE = 512,   /* a cache slot outside the cache, other than -1 */
  SV_DEV_PAGE_RANGE = 1024,  /* a needed page outside the cache, or a context outside its page table */
  SV_DEV_NO_PAGES = 4096,    /* a request was refused: the ring has too few free pages */
  SV_DEV_SETTING = 8192,     /* a row's sampling settings are out of range */
  SV_DEV_TREE = 2048         /* a malformed tree: a parent that is not an earlier node, or a node
                                with children whose draft row lies outside the draft logits */
};

/* Bytes of device workspace spec_verify needs for this problem size; 0 for an
 * invalid size. The workspace is scratch owned by the caller; it must be
 * 256-byte aligned and must not be shared by calls in flight at the same time.
 * Pure host function: it touches no device. */
size_t sv_workspace_size(int B, int K, int V, int dtype);

/* One verification step for a batch of B independent sequences.
 *
 *   target_logits  device, [B, K+1, V] row-major, dtype; row t of sequence b is
 *                  q(. | prefix, x~_1..x~_t), t = 0..K (the target's K+1 outputs)
 *   draft_logits   device, [B, K, V] row-major, dtype; row t is p(. | prefix, x~_1..x~_t)
 *   draft_tokens   device, [B, K] int32, the drafted tokens x~ (expected in [0, V))
 *   uniforms       device, [B, K+2] fp32, expected in [0, 1)
 *   B, K, V        batch, lookahead (1..64), vocabulary (1..2^31-1)
 *   dtype          SV_BF16 or SV_F32
 *   temperature    T > 0, applied to both p and q (softmax(l / T))
 *   out_tokens     device, [B, K+1] int32 (written): accepted drafts, then the
 *                  drawn token, then -1 padding
 *   n_accepted     device, [B] int32 (written): accepted drafts per sequence, 0..K
 *   workspace      device, sv_workspace_size(B, K, V, dtype) bytes, 256-byte aligned
 *
 * Inputs are read only. Base pointers of the logits need only element
 * alignment; 16-byte aligned bases with V * sizeof(dtype) a multiple of 16
 * take the 16-byte vector-load path. Returns SV_OK once the work is enqueued, or
 * a host-side error code with nothing enqueued. B == 0 returns SV_OK at once.
 * Device-side problems are reported through sv_read_device_status(). */
int spec_verify(const void* target_logits, const void* draft_logits,
                const int32_t* draft_tokens, const float* uniforms, int B, int K, int V,
                int dtype, float temperature, int32_t* out_tokens, int32_t* n_accepted,
                void* workspace, size_t workspace_bytes, void* stream);

/* spec_verify plus intermediate values for inspection (each pointer may be NULL;
 * all are fp64 device arrays, NaN for every entry of a failed sequence):
 *   row_lse      [B, 2K+1]: log sum_i exp(l_i / T) per row, target rows 0..K
 *                first, then draft rows 0..K-1 (from the streaming pass)
 *   thresholds   [B, K]: min(1, q(x~_t)/p(x~_t)) for every t, the acceptance
 *                test's threshold (card, §4.2 "Modified rejection sampling")
 *   sample_prob  [B]: normalised weight of the drawn token in the
 *                distribution it was drawn from (residual, fallback q, or bonus q)
 *   row_max      [B, 2K+1]: max_i l_i / T per row, same row order as row_lse
 *   ratios       [B, K]: the ratio q(x~_t)/p(x~_t) itself, not clamped at 1;
 *                +inf where p(x~_t) = 0 < q(x~_t), 0 where q(x~_t) = 0
 * Every t < K gets a threshold and a ratio, also past the first rejection. */
int spec_verify_debug(const void* target_logits, const void* draft_logits,
                      const int32_t* draft_tokens, const float* uniforms, int B, int K, int V,
                      int dtype, float temperature, int32_t* out_tokens, int32_t* n_accepted,
                      void* workspace, size_t workspace_bytes, void* stream, double* row_lse,
                      double* thresholds, double* sample_prob, double* row_max,
                      double* ratios);

/* spec_verify that also records three caller-owned CUDA events (cudaEvent_t
 * passed as void*, created with timing enabled) on `stream`: `ev_start` before
 * the first kernel, `ev_stats_done` between the streaming row-statistics
 * kernel and the draw kernel (after the fused kernel, when that one runs),
 * `ev_end` after the last kernel. Elapsed times between them time the
 * streaming pass and the draw. With `ev_stats_done` set the draw kernel is an
 * ordinary launch rather than a programmatic dependent, so the pair runs back
 * to back without overlap. Any event may be NULL. */
int spec_verify_profiled(const void* target_logits, const void* draft_logits,
                         const int32_t* draft_tokens, const float* uniforms, int B, int K, int V,
                         int dtype, float temperature, int32_t* out_tokens, int32_t* n_accepted,
                         void* workspace, size_t workspace_bytes, void* stream, void* ev_start,
                         void* ev_stats_done, void* ev_end);

/* Bytes of device staging memory spec_verify_host needs (inputs and outputs). */
size_t sv_staging_size(int B, int K, int V, int dtype);

/* spec_verify on HOST buffers: copies the four inputs host -> device into
 * `staging` (device, sv_staging_size() bytes, 256-byte aligned), runs the step,
 * copies out_tokens / n_accepted back to the host buffers and synchronises
 * `stream`. Pinned host memory gives the fastest copies. Returns a host-side
 * error code, or else the device status bits of this call (0 = all ok). */
int spec_verify_host(const void* h_target_logits, const void* h_draft_logits,
                     const int32_t* h_draft_tokens, const float* h_uniforms, int B, int K,
                     int V, int dtype, float temperature, int32_t* h_out_tokens,
                     int32_t* h_n_accepted, void* staging, size_t staging_bytes,
                     void* workspace, size_t workspace_bytes, void* stream);

/* spec_verify_host without the wait: the copies and the step are enqueued on
 * `stream`, and the call returns SV_OK (or a host-side error code, with
 * nothing enqueued) at once. h_out_tokens / h_n_accepted hold the results
 * once `stream` has reached this point (cudaStreamSynchronize, or an event
 * recorded after the call); the device status bits are read with
 * sv_read_device_status(workspace, stream). The host input buffers must stay
 * unchanged until then, and pinned host memory is needed for the copies to be
 * asynchronous. A serving loop overlaps the copies of one step with the
 * kernels of the previous one by giving consecutive calls different streams,
 * staging buffers and workspaces. */
int spec_verify_host_async(const void* h_target_logits, const void* h_draft_logits,
                           const int32_t* h_draft_tokens, const float* h_uniforms, int B, int K,
                           int V, int dtype, float temperature, int32_t* h_out_tokens,
                           int32_t* h_n_accepted, void* staging, size_t staging_bytes,
                           void* workspace, size_t workspace_bytes, void* stream);

/* spec_verify for callers that cannot allocate device memory (the paper has no
 * counterpart to this; it is a property of this library only). Some callers
 * cannot provide a workspace: code running during stream capture in the global
 * or thread-local mode (where cudaMalloc is not allowed), plugins whose device
 * memory must all come from a host framework's pool, and latency-critical loops
 * where cudaMalloc may stall the device. This entry point allocates nothing and
 * takes no workspace: its scratch is one fixed array of SV_STATIC_SCRATCH_BYTES
 * (8 MiB) of device memory inside the library, which every GPU that loads the
 * library holds until the process exits.
 *
 * Arguments, layouts and results are those of spec_verify. Problems whose
 * sv_workspace_size exceeds SV_STATIC_SCRATCH_BYTES are rejected with
 * SV_ERR_SCRATCH_LIMIT and nothing is enqueued. Every call on a device shares
 * that device's array, which keeps the previous call's contents; each call
 * clears what must start at zero itself. Calls that overlap on the GPU (on
 * different streams, or from different threads) race on the array and must
 * be serialised by the caller. Outside stream capture every call looks up the
 * array's device address in the current context (cudaGetSymbolAddress); a
 * call made while `stream` is being captured reuses the address of the last
 * call on that device, so make one call outside capture first (and again
 * after cudaDeviceReset or a change of context). Device status bits are not
 * readable for these calls (there is no workspace to read them from): a
 * sequence that failed shows -1 in all its outputs and n_accepted = -1, and a
 * draw that did not complete shows -1 at position n_accepted. */
int spec_verify_static(const void* target_logits, const void* draft_logits,
                       const int32_t* draft_tokens, const float* uniforms, int B, int K, int V,
                       int dtype, float temperature, int32_t* out_tokens, int32_t* n_accepted,
                       void* stream);

/* ---------------------------------------------------------------- draft-side sampler
 *
 * Step 1 of the card's Algorithm 2: the draft model's tokens x~_t ~ p(.),
 * drawn from the transformed distribution p = softmax(l / T) ("Accelerating
 * Large Language Model Decoding with Speculative Sampling", wikillm.com paper
 * card, §4.2 "Decoding transforms", and the Pitfalls item on transformed
 * distributions): the draws that feed the verifier use the very distribution
 * the verifier's ratios and residual use. One token per row, by
 * the inverse-CDF convention above with the row's uniform; rows are
 * independent, so a caller samples one draft position for a batch per call
 * (or several positions at once when their logits are already known). */

/* Bytes of device workspace spec_draft_sample needs for N rows of V elements;
 * 0 for invalid sizes. Pure host function. */
size_t sv_sample_workspace_size(int N, int V, int dtype);

/* One token per row:
 *   logits       device, [N, V] row-major, dtype elements (element-aligned;
 *                16-byte aligned with V * sizeof(dtype) a multiple of 16 takes
 *                the 16-byte vector-load path)
 *   uniforms     device, [N] fp32: the uniform of each row's draw
 *   temperature  T > 0, finite (fp32)
 *   out_tokens   device, [N] int32: the drawn token, or -1 for a failed row
 *   sample_prob  device, [N] fp64, may be NULL: probability of the drawn token
 *   workspace    device, sv_sample_workspace_size() bytes, 256-byte aligned,
 *                caller-owned; one call at a time per workspace
 * A row fails (token -1, status bit) if it holds NaN or +inf, is entirely
 * -inf, or its uniform is NaN or outside [0, 1]; other rows are unaffected.
 * Returns SV_OK once the work is enqueued on `stream`, or a host-side error
 * code with nothing enqueued; N == 0 returns SV_OK at once. Device status bits
 * are read with sv_read_device_status(). */
int spec_draft_sample(const void* logits, const float* uniforms, int N, int V, int dtype,
                      float temperature, int32_t* out_tokens, double* sample_prob,
                      void* workspace, size_t workspace_bytes, void* stream);

/* ---------------------------------------------------------------- greedy mode
 *
 * Verification at T = 0. The paper reports greedy results but does not state
 * the rule; the card's Pitfalls ("Greedy mode is not specified") infer it by
 * applying the general rule to one-hot distributions: accept while the draft's
 * greedy token equals the target's, otherwise emit the target's greedy token.
 * Here: x~_t is accepted while it equals argmax q_t (ties go to the smallest
 * token id; -inf entries are masked); at the first mismatch j, argmax q_j is
 * emitted; if all K match, argmax q_K (the bonus token). No uniforms, no
 * temperature and no draft logits are read; the target rows are read once. */

/* Bytes of device workspace spec_verify_greedy needs; 0 for invalid sizes. */
size_t sv_greedy_workspace_size(int B, int K, int V, int dtype);

/* Greedy verification: target_logits, draft_tokens, out_tokens, n_accepted,
 * workspace and stream as for spec_verify (out_tokens holds the accepted
 * drafts, then the emitted token, then -1 padding). A sequence fails (all -1,
 * status bit) if a target row holds NaN or +inf or is entirely -inf, or a
 * draft token lies outside [0, V). Returns SV_OK once enqueued, or a host-side
 * error code with nothing enqueued; B == 0 returns SV_OK at once. */
int spec_verify_greedy(const void* target_logits, const int32_t* draft_tokens, int B, int K,
                       int V, int dtype, int32_t* out_tokens, int32_t* n_accepted,
                       void* workspace, size_t workspace_bytes, void* stream);

/* ---------------------------------------------------------------- top-k filtered verification
 *
 * The card's §4.2 "Decoding transforms": top-k is applied to both p and q,
 * and the rejection scheme then runs on the filtered distributions (the
 * Pitfalls section: the same transformed distributions are used for the
 * thresholds, the residual and the bonus draw). Each of the 2K+1 rows keeps
 * its top_k largest logits; ties go to the smaller token id and -0.0 equals
 * +0.0; the other entries count as -inf. The kept entries' softmax at
 * temperature T, the thresholds min(1, q/p), the residual max(0, q - p) and
 * the inverse-CDF draws are those of spec_verify, on the filtered rows. */

/* Bytes of device workspace spec_verify_topk needs; 0 for invalid sizes.
 * top_k >= V keeps every entry and needs sv_workspace_size(B, K, V, dtype). */
size_t sv_topk_workspace_size(int B, int K, int V, int dtype, int top_k);

/* Top-k filtered verification. Arguments as for spec_verify, plus
 *   top_k  entries kept per row: 1 <= top_k <= 256, or top_k >= V (every
 *          entry kept: the call is spec_verify's); other values return
 *          SV_ERR_SHAPE
 * Each row is reduced to its top_k entries in one pass over it (one CTA per
 * row: a running threshold and a candidate buffer in shared memory, with an
 * exact radix select over the row for adversarial orders), their softmax is
 * taken in fp64, and the verification runs on the kept (token id,
 * probability) pairs (one CTA per sequence): two kernels per call. Failures and status bits as for
 * spec_verify (a row holding +inf or NaN fails its sequence, a row whose kept
 * entries are all -inf is an empty row). Returns SV_OK once enqueued, or a
 * host-side error code with nothing enqueued; B == 0 returns SV_OK at once. */
int spec_verify_topk(const void* target_logits, const void* draft_logits,
                     const int32_t* draft_tokens, const float* uniforms, int B, int K, int V,
                     int dtype, float temperature, int top_k, int32_t* out_tokens,
                     int32_t* n_accepted, void* workspace, size_t workspace_bytes, void* stream);

/* ---------------------------------------------------------------- nucleus (top-p) filtered verification
 *
 * The card's §4.2 "Decoding transforms" with the nucleus rule on both p and
 * q: each of the 2K+1 rows keeps the shortest prefix of its entries, ordered
 * by logit (larger first, ties to the smaller token id, -0.0 equal to +0.0),
 * whose probability softmax(l / T) reaches top_p; the other entries count as
 * -inf. The filtered rows are then verified exactly as by spec_verify. */

/* Bytes of device workspace spec_verify_topp needs (spec_verify's, and one
 * 8-byte cut key per row); 0 for invalid sizes. */
size_t sv_topp_workspace_size(int B, int K, int V, int dtype);

/* Nucleus filtered verification. Arguments as for spec_verify, plus
 *   top_p        probability mass kept per row: top_p > 0; top_p >= 1 keeps
 *                every entry (the call is spec_verify's); NaN or top_p <= 0
 *                returns SV_ERR_SHAPE
 *   kept_counts  device, [B, 2K+1] int32, may be NULL: entries kept per row
 *                (target rows 0..K, then draft rows 0..K-1); V for a row that
 *                fails (NaN, +inf or all -inf), which is left as it is
 * Per row, a cut is found without a sort: mass histograms over the scaled
 * distance (m - l) / T of each entry from the row maximum, at finer and finer
 * widths, locate the cut to a bin of at most 1024 entries, whose keys are then
 * searched exactly with their masses (a bin that never gets that small, from
 * heavy ties, is resolved bit by bit over the key). Rows up to 512 KB are held
 * in the shared memory of a thread-block cluster (up to 8 CTAs per row), so
 * each row is read from memory once; longer rows are re-read per pass. Weights
 * are float-float exponentials. The cut also yields each row's kept mass, so
 * the verification (a scan kernel, then the draw) reads the rows unchanged
 * and applies each row's kept set as it loads them: sv_topp_kernels_per_call
 * kernels per call. Returns SV_OK once enqueued, or a host-side error code
 * with nothing enqueued; B == 0 returns SV_OK at once. */
int spec_verify_topp(const void* target_logits, const void* draft_logits,
                     const int32_t* draft_tokens, const float* uniforms, int B, int K, int V,
                     int dtype, float temperature, float top_p, int32_t* out_tokens,
                     int32_t* n_accepted, int32_t* kept_counts, void* workspace,
                     size_t workspace_bytes, void* stream);

/* Reads the device status word of the last call that used `workspace`: waits
 * for `stream`, then stores the OR of the SV_DEV_* bits in *status. */
int sv_read_device_status(const void* workspace, void* stream, int* status);

/* Static description of a return code or device status bit set. */
const char* sv_status_string(int status);

/* Kernels one spec_verify call over these sizes launches (for launch
 * accounting): 1 (the fused kernel) for calls streaming between 16 MiB and
 * 1 GiB; else 2 for calls whose draw needs few chunks (the streaming kernel and
 * a one-launch draw) or 3 (the streaming kernel, the draw's sum kernel and its
 * finish kernel); 0 for invalid sizes or B == 0. */
int sv_kernels_per_call(int B, int K, int V, int dtype);

/* Kernels one spec_verify_topp call with top_p < 1 over these sizes launches:
 * the cut kernel, the scan kernel and the draw (one kernel when the draw
 * needs few chunks, else two), so 3 or 4; 0 for invalid sizes or B == 0. */
int sv_topp_kernels_per_call(int B, int K, int V, int dtype);

/* Test hook: 0 (the default) chooses the kernels by size, 1 forces the kernel
 * pair, 2 forces the fused kernel. Process-wide; for tests that compare the
 * two paths. */
void sv_force_path(int path);

/* Test hook for failure detection: with `on` nonzero, calls never publish
 * their plans' release flag, so on the fused path every draw CTA's bounded
 * wait runs out (200 ms) and the call ends with SV_DEV_TIMEOUT; no GPU fault,
 * and the context stays usable. Process-wide; 0 restores normal calls. */
void sv_test_withhold_plans(int on);

/* ---------------------------------------------------------------- the scoring step's projection
 *
 * Algorithm 2 step 2 of the card: one target call scores the K+1 prefixes
 * (§4.1 "Why it works (conditional scoring)"); the verification then needs,
 * per scored row, only the statistics of the temperature transform (§4.2
 * "Decoding transforms") and the logit at the drafted token (§4.2 "Modified
 * rejection sampling"). This call fuses the model's final projection with
 * those statistics: the logits l = h W^T are formed on the tensor cores
 * (bf16 operands, fp32 accumulation) and reduced on chip, never stored.
 *
 * Bytes of device workspace sv_lmhead_stats needs; 0 for invalid sizes
 * (N < 0, V < 1, D < 8 or not a multiple of 8). Pure host function. */
size_t sv_lmhead_workspace_size(int N, int D, int V);

/* For every row n of the hidden states:
 *   hidden       device, [N, D] bf16, row-major, 16-byte aligned
 *   weight       device, [V, D] bf16, row-major, 16-byte aligned: the
 *                projection's weight, one row per token (l = h W^T)
 *   tokens       device, [N] int32: a token per row, or -1 for none
 *   temperature  T > 0, finite (fp32)
 *   row_max      device, [N] fp64 (written): max_i l_i / T
 *   lse          device, [N] fp64 (written): log sum_i exp(l_i / T)
 *   at           device, [N] fp32 (written): l at tokens[n], NaN where tokens[n]
 *                is outside [0, V)
 *   workspace    device, sv_lmhead_workspace_size() bytes, 256-byte aligned;
 *                its first 4 bytes are the device status word (read with
 *                sv_read_device_status): 32 = a row with a non-finite logit
 *                (its row_max and lse are NaN), 256 = a bounded wait ran out
 * The logits carry fp32 accumulation error: against exact arithmetic, a
 * logit differs by about 2^-24 sqrt(D) times the magnitude of the partial
 * sums. Returns SV_OK once the two kernels are enqueued on `stream`, or a
 * host-side error code with nothing enqueued; N == 0 returns SV_OK at once. */
int sv_lmhead_stats(const void* hidden, const void* weight, const int32_t* tokens, int N, int D,
                    int V, float temperature, double* row_max, double* lse, float* at,
                    void* workspace, size_t workspace_bytes, void* stream);

/* ---------------------------------------------------------------- a tree of drafted tokens
 *
 * One step of decoding with a tree of drafted tokens: queries and keys are
 * normalised and rotated (sv_qk_norm_rope), keys and values go into the paged
 * cache (sv_cache_write), the tree attends the cache (sv_tree_attention), and
 * the scored tree is verified (spec_verify_tree). The keys and values of the
 * accepted nodes then go to consecutive positions with a second sv_cache_write,
 * in which the rejected nodes' slots are -1.
 *
 * A tree of T nodes (1 <= T <= 128) is an array of T parents: parents[i] is an
 * earlier node (0 <= parents[i] < i), -1 for a node under the context, or -2 for
 * padding, which is no node; a padding node has no children.
 *
 * Norms per head and rotation by position, in one pass. For every row x of D
 * values (a head of a token): y = x / sqrt(mean(x^2) + eps) * weight, then the
 * first R values rotate in pairs, (i, i + R/2), or (2i, 2i + 1) when interleaved,
 * by the angle positions[n] * inv_freq[i]:
 *   (y0, y1) -> (y0 cos - y1 sin, y1 cos + y0 sin).
 *   q, k          device, [N, Hq, D] and [N, Hkv, D], dtype, values of a row
 *                 consecutive, token and head strides in elements; Hq or Hkv may
 *                 be 0 (its pointers may then be NULL), not both
 *   q_weight, k_weight  device, [D] dtype, or NULL for ones
 *   inv_freq      device, [R/2] fp32
 *   positions     device, [N] int32
 *   N             N * ceil((Hq + Hkv) / 16) < 2^31
 *   D, R          1 <= D <= 1024, 0 <= R <= D, R even
 *   q_out, k_out  device, written; strides as above; may be q and k themselves
 *                 (same pointer and strides), must not overlap them otherwise
 * Computed in fp32 (the angle's reduction to a fraction of a turn in 64-bit
 * integers, so that far positions lose nothing) and rounded once. 16-byte
 * aligned rows with D and R multiples of 16 (fp32: 8), D <= 512 (fp32: 256),
 * take the vector path. No workspace. Returns SV_OK once enqueued; N == 0 returns SV_OK at once. */
int sv_qk_norm_rope(const void* q, int64_t q_stride_n, int64_t q_stride_h, const void* k,
                    int64_t k_stride_n, int64_t k_stride_h, const void* q_weight,
                    const void* k_weight, const float* inv_freq, const int32_t* positions, int N,
                    int Hq, int Hkv, int D, int R, int dtype, float eps, int interleaved, void* q_out,
                    int64_t qo_stride_n, int64_t qo_stride_h, void* k_out, int64_t ko_stride_n,
                    int64_t ko_stride_h, void* stream);

/* The paged cache: k_cache and v_cache are [num_pages, Hkv, page_size, D] of
 * cache_dtype (SV_BF16 or SV_E4M3); with SV_E4M3, k_scale and v_scale are
 * [num_pages, Hkv, page_size] fp32 (else NULL). The token in slot s lies in page
 * s / page_size at offset s % page_size.
 *
 * Writes N tokens' keys and values into their slots:
 *   k, v     device, [N, Hkv, D], dtype (SV_BF16 or SV_F32), strides in elements
 *   N        N * Hkv < 2^32
 *   slots    device, [N] int64; -1 writes nothing. No slot may occur twice.
 *   status   device word, may be NULL: SV_DEV_SLOT_RANGE is OR-ed into it when a
 *            slot lies outside the cache (that token is not written). The
 *            call does not clear it.
 * SV_BF16 rounds to nearest even. SV_E4M3 stores a row of D values as
 * code = e4m3(x * (448 / a)) with the scale a / 448, a = max(max |x|, 1e-30), both
 * quotients rounded to fp32 and the code to nearest even; a row that holds NaN
 * or infinity gets a NaN scale and codes of 0, so that it reads back as NaN.
 * 1 <= D <= 1024. Returns SV_OK once enqueued; N == 0 returns SV_OK at once. */
int sv_cache_write(const void* k, int64_t k_stride_n, int64_t k_stride_h, const void* v,
                   int64_t v_stride_n, int64_t v_stride_h, const int64_t* slots, int N, int Hkv,
                   int D, int dtype, void* k_cache, void* v_cache, float* k_scale, float* v_scale,
                   int64_t num_pages, int page_size, int cache_dtype, uint32_t* status, void* stream);

/* Reads N tokens back: k_out and v_out (device, [N, Hkv, D], dtype, strides in
 * elements) get the stored values, code * scale rounded once. A slot of -1
 * gives zeros; any other slot outside the cache does too, and sets
 * SV_DEV_SLOT_RANGE in `status` as above. */
int sv_cache_read(const void* k_cache, const void* v_cache, const float* k_scale,
                  const float* v_scale, int64_t num_pages, int page_size, int cache_dtype,
                  const int64_t* slots, int N, int Hkv, int D, int dtype, void* k_out,
                  int64_t ko_stride_n, int64_t ko_stride_h, void* v_out, int64_t vo_stride_n,
                  int64_t vo_stride_h, uint32_t* status, void* stream);

/* Bytes of device workspace sv_tree_attention needs; 0 for invalid sizes.
 * Pure host function. */
size_t sv_tree_attention_workspace_size(int B, int T, int Hq, int Hkv, int D, int max_pages,
                                        int page_size);

/* Attention of B trees of T nodes over the paged cache. Sequence b has
 * ctx_lens[b] context tokens at positions 0 .. ctx_lens[b] - 1, and node i's key
 * and value lie at position ctx_lens[b] + i; position t is in page
 * page_table[b, t / page_size]. Node i attends the context, its ancestors and
 * itself: out = softmax(scale q k) v over those, query head h with key/value head
 * h / (Hq / Hkv).
 *   q           device, [B, T, Hq, D] bf16, strides in elements
 *   k_cache, v_cache, k_scale, v_scale, num_pages, page_size, cache_dtype  the cache
 *   page_table  device, [B, max_pages] int32; entries past a sequence's last node
 *               are not used
 *   ctx_lens    device, [B] int32, 0 or more
 *   parents     device, [B, T] int32, or NULL for chains (node i's parent is i - 1)
 *   out         device, [B, T, Hq, D] bf16, contiguous (written); 0 for padding
 *   workspace   device, sv_tree_attention_workspace_size() bytes, 256-byte aligned;
 *               its first 4 bytes are the device status word
 * T = 1 is the ordinary decoding step. Sums, maxima and the running output are
 * fp32. For their product with the values the weights are rounded to bf16 (2^-8 of
 * each). With an e4m3 cache and few rows (T * Hq/Hkv <= 40, D <= 128) q enters as two e4m3
 * pieces (off by 2^-19 of a row's largest value at most), and a weight times its value's
 * scale as three: off by 2^-11 of itself, or by 2^-24 of the row's largest such
 * product. Codes and scales are expected as sv_cache_write stores them (finite codes, scales up to 2^100). A
 * sequence with a malformed tree (SV_DEV_TREE), or whose context or
 * needed pages lie outside the table or the cache (SV_DEV_PAGE_RANGE), gets NaN
 * outputs; the others are unaffected. What masked positions hold, NaN included,
 * does not matter. D a multiple of 16 up to 256, page sizes of 16, 32, 64 or 128 and
 * 16-byte aligned rows take the tensor-core kernel, other shapes (D up to
 * 1024) a plain one. Returns SV_OK once enqueued; B == 0 returns SV_OK at once. */
int sv_tree_attention(const void* q, int64_t q_stride_b, int64_t q_stride_t, int64_t q_stride_h,
                      const void* k_cache, const void* v_cache, const float* k_scale,
                      const float* v_scale, int64_t num_pages, int page_size, int cache_dtype,
                      const int32_t* page_table, const int32_t* ctx_lens, const int32_t* parents,
                      int B, int T, int Hq, int Hkv, int D, int max_pages, float scale, void* out,
                      void* workspace, size_t workspace_bytes, void* stream);

/* Bytes of device workspace spec_verify_tree needs; 0 for invalid sizes (B < 0,
 * T outside [1, 128], V outside [1, 2^30]). Pure host function. */
size_t sv_tree_workspace_size(int B, int T, int V, int dtype);

/* Verification of B trees of T nodes: the modified rejection sampling of the
 * card's §4.2 with several candidates at a node. Node 0 is the root, the last
 * emitted token (parents[b, 0] is -1; every other node has a parent or is padding).
 * At the current node, the root at first, with q its target row's and p its
 * draft row's softmax(l / T), the children are tried in index order against the residual
 * r, q at first: child c of token x is accepted while u < min(1, r(x)/p(x)), and
 * becomes the current node; a rejection turns r into max(0, r - p) over its sum (a
 * sum below 2^-30, which is r = p but for rounding, leaves r). When no child is left,
 * one token is drawn from r. With each node's children drawn independently from p, the emitted
 * tokens follow the target's distribution. The tests' row sums are fp32 (about 1e-6 of a
 * ratio; spec_verify's are float-floats): a chain gives spec_verify's results but where a uniform lies within that of
 * its ratio. Draws use float-floats.
 *   target_logits  device, [B, T, V] dtype: row i is the target's at node i
 *   draft_logits   device, [R, V] dtype: the draft's rows
 *   draft_index    device, [B, T] int32: node i's row of draft_logits; read for
 *                  nodes with children only
 *   tokens         device, [B, T] int32: the nodes' tokens (the root's is not read)
 *   parents        device, [B, T] int32
 *   uniforms       device, [B, T] fp32: node i's test; the root's is the draw's
 *   out_tokens     device, [B, T] int32 (written): accepted tokens, the drawn
 *                  token, then -1
 *   out_nodes      device, [B, T] int32 (written): accepted nodes, then -1
 *   n_accepted     device, [B] int32 (written)
 * Rows of nodes that are not visited are not read. A sequence fails (all -1,
 * status bit) on a malformed tree, a token outside [0, V) or a uniform outside
 * [0, 1] of any node, and on NaN, +inf or an empty row among the visited
 * rows. Conventions and workspace as for spec_verify. */
int spec_verify_tree(const void* target_logits, const void* draft_logits, const int32_t* draft_index,
                     const int32_t* tokens, const int32_t* parents, const float* uniforms, int B, int T,
                     int V, int R, int dtype, float temperature, int32_t* out_tokens,
                     int32_t* out_nodes, int32_t* n_accepted, void* workspace, size_t workspace_bytes,
                     void* stream);

/* ---------------------------------------------------------------- drafting over a long cache
 *
 * What a draft step needs around the verification when the draft is the model itself
 * reading a part of its cache: the step's pages and slots (sv_page_plan), bounds of the
 * keys of each page (sv_page_bounds, after sv_cache_write), attention over the pages that the
 * bounds select (sv_sparse_attention), and tokens from the transformed distribution
 * (spec_filtered_sample; spec_verify_topk and spec_verify_topp verify tokens drawn with their
 * filter). Lengths stay on the device, so that a captured graph follows them. */

/* Bytes of device workspace sv_page_plan needs; 0 for B < 0. Pure host function. */
size_t sv_page_plan_workspace_size(int B);

/* The pages and slots of one step of B requests. Request b holds held[b] pages (the first
 * entries of its row of page_table) and ctx_lens[b] tokens, and new_lens[b] >= 0 tokens
 * come in behind them; new_lens[b] = -1 says that it has ended. Free pages wait in a ring:
 * state is (head, count), the pages are ring[(head + i) % capacity], i < count.
 *   - A request needs max(0, ceil((ctx + new) / page_size) - held) pages more. It is granted if
 *     it needs none, or if its need and those of the valid requests before it come to at most `count`,
 *     and if its tokens end within max_tokens; it then takes its pages from the ring in
 *     order. Nothing is taken for a request that is not granted (granted[b] = 0).
 *   - The pages of requests that have ended go behind the ring's tail, in order, and can be taken from
 *     the next call on; held_out is then 0 and granted -1. The table's entries stay as they were.
 *   - Tokens are packed by request: those of request b begin behind the sum of the max(new_lens, 0)
 *     before it, granted or not.
 *   ring         device, [capacity] int32, in and out
 *   state        device, [2] int32; state_out may be the same
 *   page_table   device, [B, max_pages] int32, in and out: only the new entries are written
 *   held         device, [B] int32; held_out may be the same
 *   slots        device, [max_tokens] int64 (written): page * page_size + offset, as
 *                sv_cache_write takes them; -1 for tokens that are not granted or not there
 *   positions, seqs  device, [max_tokens] int32 (written): the token's position and request, or -1
 *   granted      device, [B] int32 (written): new_lens, or 0
 *   workspace    device, sv_page_plan_workspace_size() bytes, 256-byte aligned
 *   status       device word, may be NULL; bits are OR-ed into it: SV_DEV_NO_PAGES and
 *                SV_DEV_SLOT_RANGE (past max_tokens) for requests that are refused, SV_DEV_PAGE_RANGE
 *                for a negative length, held outside [0, max_pages], a need outside the table, or a
 *                ring whose state is out of range or has no room for the pages that come back
 *                (none come back then)
 * Returns SV_OK once enqueued. */
int sv_page_plan(int32_t* ring, int64_t capacity, const int32_t* state, int32_t* page_table, const int32_t* held,
                 const int32_t* ctx_lens, const int32_t* new_lens, int B, int max_pages, int page_size, int max_tokens,
                 int64_t* slots, int32_t* positions, int32_t* seqs, int32_t* granted, int32_t* held_out,
                 int32_t* state_out, void* workspace, size_t workspace_bytes, uint32_t* status, void* stream);

/* Bounds of the keys of every page that holds one of the positions
 * ctx_lens[b] .. ctx_lens[b] + new_lens[b] - 1 (none for new_lens[b] <= 0), over all keys of the
 * page up to the last of those positions:
 *   codes   device, [num_pages, Hkv, 2, D] int8: the channels' minima, then their maxima
 *   scale   device, [num_pages, Hkv] fp32
 * With a = max(max |k|, 1e-30) over the page's keys of the head and up = 127 / a (rounded to fp32),
 * a minimum's code is floor(min * up), a maximum's ceil(max * up), within -127 .. 127, and
 * the scale a / 127. A page that holds NaN or infinity gets codes of 0 and the scale +inf. An
 * e4m3 key counts as code * scale rounded to fp32. No page may belong to two sequences.
 * `status` may be NULL: SV_DEV_PAGE_RANGE is OR-ed into it for lengths outside the page table (no
 * bounds are written for that sequence) and pages outside the cache. 1 <= D <= 1024. Returns
 * SV_OK once enqueued; B == 0 returns SV_OK at once. */
int sv_page_bounds(const void* k_cache, const float* k_scale, int64_t num_pages, int page_size, int cache_dtype,
                   const int32_t* page_table, const int32_t* ctx_lens, const int32_t* new_lens, int B, int Hkv,
                   int D, int max_pages, int8_t* codes, float* scale, uint32_t* status, void* stream);

/* Bytes of device workspace sv_sparse_attention needs; 0 for invalid sizes. No less for more rows, so that
 * a workspace for a batch serves smaller ones. Pure host function. */
size_t sv_sparse_attention_workspace_size(int N, int Hq, int Hkv, int D, int max_pages, int page_size, int budget);

/* Attention of N query rows over selected pages of their sequences. Row n stands at
 * positions[n] of sequence seqs[n] (n itself if seqs is NULL) and sees the keys up to and with its
 * own, in ceil((positions[n] + 1) / page_size) pages. For each key/value head it attends `budget` of
 * them, or all if there are no more: the first `sink`, the last `recent`, and those of the highest
 * scores, equal scores in page order. A head's queries q_g become codes
 * c = rint(q * (127 / a)), within -127 .. 127, and the scale s_g = a / 127, a = max(max |q_g|, 1e-30),
 * quotients and products rounded to fp32 (a head that holds NaN or infinity gets codes and a scale of
 * 0); then, in fp32 and rounded at each product,
 *   score(page) = max_g (s_g * sum_d max(c_d min_d, c_d max_d)) * scale(page)
 * with the page's codes min_d and max_d; +inf where the page's scale is, or the product is NaN. It bounds the scores of the
 * page's keys from above, to the codes' resolution, and is the same on any hardware.
 *   q            device, [N, Hq, D] bf16, strides in elements
 *   k_cache .. cache_dtype    the cache
 *   codes, bound_scale        sv_page_bounds' outputs, up to date for every page that a row sees
 *   page_table   device, [B, max_pages] int32, max_pages <= 49152
 *   positions    device, [N] int32; -1: the row is empty
 *   seqs         device, [N] int32 or NULL (then N <= B); -1: the row is empty
 *   budget, sink, recent      sink >= 0, recent >= 1, sink + recent <= budget
 *   scale        of the attention's scores, finite and > 0
 *   out          device, [N, Hq, D] bf16, contiguous (written); 0 for an empty row
 *   selected     device, [N, Hkv, budget] int32, may be NULL (written): the chosen pages' places in
 *                their sequence, ascending, then -1
 *   workspace    device, sv_sparse_attention_workspace_size() bytes, 256-byte aligned; its first
 *                4 bytes are the device status word
 * A row whose position or sequence is out of range, or one of whose pages lies outside the cache, gets NaN
 * outputs, no selected pages and SV_DEV_PAGE_RANGE; the others are unaffected.
 * With D 64 or 128, at most 8 query heads a key/value head, page_size a multiple of 16 and q and the cache on 16 bytes
 * (q's strides too), a kernel of its own attends the pages: a bf16 cache's weights are off by 2^-16 of
 * each; over an e4m3 cache q is fp16 relative to its head's largest value (off by 2^-25 of that at most), and a
 * weight times its value's scale is off by 2^-22 of itself, or by 2^-40 of the row's largest. Other shapes,
 * and their precision, are sv_tree_attention's. Codes and scales are expected as sv_cache_write stores them. Returns
 * SV_OK once enqueued; N == 0 returns SV_OK at once. */
int sv_sparse_attention(const void* q, int64_t q_stride_n, int64_t q_stride_h, const void* k_cache,
                        const void* v_cache, const float* k_scale, const float* v_scale, int64_t num_pages,
                        int page_size, int cache_dtype, const int8_t* codes, const float* bound_scale,
                        const int32_t* page_table, const int32_t* positions, const int32_t* seqs, int N, int B,
                        int Hq, int Hkv, int D, int max_pages, int budget, int sink, int recent, float scale,
                        void* out, int32_t* selected, void* workspace, size_t workspace_bytes, void* stream);

/* One token a row from the softmax of the entries that the row's settings keep, by the
 * inverse-CDF convention above. With the entries ordered by logit (larger first, ties to the
 * smaller id, -0 equal to +0) and w_i = exp((l_i - max l) / T):
 *   - top_k keeps the first top_k entries (all for top_k <= 0 or >= V);
 *   - top_p keeps the shortest prefix of those whose weight reaches top_p times theirs (all for
 *     top_p >= 1);
 *   - min_p keeps the entries of w_i >= min_p (all for min_p <= 0), the first entry always.
 * T = 0 takes the first entry, whatever the other settings.
 *   logits       device, [N, V] dtype, rows row_stride elements apart (>= V)
 *   uniforms     device, [N] fp32
 *   temperatures, top_ks, top_ps, min_ps   device, [N], a setting a row; where one is NULL the
 *                value next to it holds for all rows
 *   out_tokens   device, [N] int32 (written), -1 for a failed row
 *   out_probs    device, [N] fp32, may be NULL (written): the token's probability among the kept
 *                entries, NaN for a failed row
 *   status       device word, may be NULL; bits are OR-ed into it
 * Weights are float-float exponentials (5e-11) as whole numbers of 2^-44 of the row's largest (V above
 * 2^17: 2^(61 - ceil(log2 V))), so that no result depends on the order of a sum; smaller weights count as 0.
 * A row fails on NaN or +inf (SV_DEV_NONFINITE), with no finite entry (SV_DEV_EMPTY_ROW), on a
 * uniform outside [0, 1] (SV_DEV_UNIFORM_RANGE), and on T negative or not finite, top_p NaN or <= 0, or min_p
 * NaN or > 1 (SV_DEV_SETTING; host errors where the value holds for all rows). No workspace.
 * 1 <= V <= 2^30. Returns SV_OK once enqueued; N == 0 returns SV_OK at once. */
int spec_filtered_sample(const void* logits, int64_t row_stride, const float* uniforms, int N, int V,
                         int dtype, const float* temperatures, float temperature, const int32_t* top_ks,
                         int top_k, const float* top_ps, float top_p, const float* min_ps, float min_p,
                         int32_t* out_tokens, float* out_probs, uint32_t* status, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* SPEC_VERIFY_H_ */
