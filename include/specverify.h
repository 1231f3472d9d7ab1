/*
 * libspecverify: the verify-and-commit step of speculative decoding, on one GPU.
 *
 * Given the target model's logits for an anchor plus its draft positions, each
 * call scans every vocabulary row once on the GPU, decides how many drafts are
 * accepted, produces the correction / bonus token, and emits the KV-commit
 * index lists for the accepted positions.  Each round yields r + 1 tokens
 * (r accepted drafts plus one correction or bonus).
 *
 * Sources, cited as page title and section:
 *   [E2D] "从 EAGLE 到 DFlash 2：SGLang 与 SpecForge 的投机解码训练和推理"
 *         (tom-jerr.github.io/sglang/eagle2-in-sglang)
 *   [SGO] SGLang speculative-decoding overview (zdszero.github.io/speculative_decoding.html)
 *
 * Row convention (row-aligned verify input, [E2D] §1.1 and the verify_ids_2d
 * construction in §5.6): the target runs on [a, d1 .. dm]; row i of a request
 * carries input token verify_ids[i] (the anchor a at the request's first row)
 * and its logits give the distribution that tests verify_ids[i + 1].  The last
 * row of a request is only used for the bonus token.
 *
 * Memory and execution rules shared by every entry point:
 *   - Every array argument is a DEVICE pointer owned by the caller.  The
 *     library never allocates, never synchronises the stream and never reads
 *     device memory from the host; all work is enqueued on `stream`.
 *   - logits: [rows, ld] row-major, fp32 or bf16 (raw bits), ld >= vocab.  The
 *     base pointer must be 16-byte aligned and ld * element_size a multiple of
 *     16.  The same rules hold for q ([rows, ldq] fp32).
 *   - Host-side argument errors return a status code before anything is
 *     enqueued.  Data errors found on the device are reported per request in
 *     out->dev_status (bits below) and still produce defined outputs.
 *   - ws / ws_bytes: scratch of at least spec_verify_workspace_bytes(...)
 *     bytes, 256-byte aligned, ZERO-FILLED BEFORE ITS FIRST USE.  Every call
 *     whose kernels run to completion leaves the workspace's counter words at
 *     zero again, so a workspace can be reused by later calls on the same
 *     stream without clearing.  Calls that share a workspace must not overlap
 *     on the GPU.
 *   - Temperature: a request with temperature T samples iff 1e-30 <= T < inf;
 *     any other value (0, negative, NaN, inf) verifies that request greedily
 *     ([E2D] §6.5: greedy rows carry a one-hot q).
 *   - Uniforms are supplied by the caller in [0, 1): u_accept[row] decides the
 *     acceptance test at that row (for trees: at that node's row), u_final[b]
 *     draws the request's one correction / bonus token.
 */
#ifndef SPECVERIFY_H
#define SPECVERIFY_H

#include <stddef.h>
#include <stdint.h>

#include <cuda_runtime_api.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  SV_OK = 0,
  SV_ERR_NULL_ARG = 1,            /* a required pointer is NULL                        */
  SV_ERR_BAD_SHAPE = 2,           /* a size, stride or scalar argument is out of range */
  SV_ERR_BAD_DTYPE = 3,           /* dtype is not SV_F32 or SV_BF16                    */
  SV_ERR_MISALIGNED = 4,          /* a base pointer or row stride breaks 16-byte rule  */
  SV_ERR_UNSUPPORTED = 5,         /* a combination the library does not implement     */
  SV_ERR_WORKSPACE_TOO_SMALL = 6, /* ws is NULL, too small or not 256-byte aligned     */
  SV_ERR_CUDA = 7                 /* a CUDA launch or device query failed              */
} sv_status_t;

typedef enum { SV_F32 = 0, SV_BF16 = 1 } sv_dtype_t;

/* Per-request device status bits (out->dev_status[b], OR-ed). */
#define SV_DEV_TOKEN_RANGE 1u    /* a tested draft / child token is outside [0, vocab): it is rejected   */
#define SV_DEV_NONFINITE 2u      /* a visited row had NaN / +inf entries (ignored) or was all -inf;      */
                                 /* an all -inf row stops verification there and its token is -1          */
#define SV_DEV_BAD_TREE 4u       /* parents / sibling lists invalid: the request is verified as its root  */
#define SV_DEV_BAD_LAYOUT 8u     /* cu_seqlens range invalid: nothing committed, num_out 0, bonus -1      */
#define SV_DEV_RESIDUAL_EMPTY 16u /* residual mass was <= 0: the token was sampled from p instead         */
#define SV_DEV_DUP_SIBLING 32u   /* target-only tree: a sibling repeats a token; the repeat is skipped    */
#define SV_DEV_TIMEOUT 64u       /* a bounded wait inside a kernel gave up (never expected): this call's   */
                                 /* outputs are undefined and the workspace must be zero-filled again      */
#define SV_DEV_SLOT_RANGE 128u   /* a page id, slot or position lies outside the KV cache: it is skipped   */

/*
 * Outputs of one call (all DEVICE pointers, caller-owned).  max_len is the
 * per-request row bound of the call (chains: m + 1; ragged: max_len; trees:
 * nodes).  [E2D] §5.6.6 and §8.1 table; [SGO] "两个容易误解的工程细节".
 */
typedef struct {
  int32_t* accept_len;      /* [B] r, accepted drafts                                        */
  int32_t* num_out;         /* [B] r + 1 (= commit_lens); 0 for a bad layout                  */
  int32_t* out_tokens;      /* [B, max_len] accepted drafts then the bonus; rest -1           */
  int32_t* bonus;           /* [B] correction / bonus token (-1 when no usable row)          */
  int32_t* accept_rows;     /* [B, max_len] global logits rows committed: anchor row, then    */
                            /*   the rows of the accepted drafts / tree path; rest -1          */
  int32_t* commit_cu;       /* [B + 1] exclusive scan of num_out                              */
  int64_t* commit_src_slot; /* [rows] or NULL: row_slots[accept_rows[b][k]] at commit_cu[b]+k */
  int64_t* commit_dst_pos;  /* [rows] or NULL: seq_lens[b] + k at commit_cu[b] + k            */
  uint32_t* dev_status;     /* [B] SV_DEV_* bits                                              */
} sv_out_t;

/* Bytes of workspace needed for a call with these sizes (rows = total logits
 * rows, max_len = per-request row bound / tree nodes). */
size_t spec_verify_workspace_bytes(int64_t rows, int32_t batch, int32_t vocab, int32_t max_len);

/* Static description of a status code. */
const char* spec_verify_status_string(sv_status_t status);

/* Description of the CUDA error behind the last SV_ERR_CUDA returned on this
 * host thread ("no error" if none). */
const char* spec_verify_last_cuda_error(void);

/* Benchmark instrumentation (not needed for verification).  While set, every
 * call made from this host thread records `start` on its stream immediately
 * before its row-statistics kernel and `stop` immediately after it, so the
 * caller can time that kernel with cudaEventElapsedTime.  The events are the
 * caller's; pass NULL, NULL to stop.  Returns SV_ERR_NULL_ARG if exactly one
 * of the two is NULL. */
sv_status_t spec_verify_set_stats_events(cudaEvent_t start, cudaEvent_t stop);

/*
 * Greedy chain verification ([E2D] §1.2 first bullet; [SGO] "为什么结果不受
 * draft 影响": accept while the target argmax equals the draft, else replace
 * it with the argmax and stop).  batch requests of m drafts each: rows =
 * batch * (m + 1), request b owns rows [b*(m+1), (b+1)*(m+1)).  Argmax ties
 * resolve to the lowest index.  row_slots [rows] and seq_lens [B] (int64) are
 * only needed for commit_src_slot / commit_dst_pos.
 */
sv_status_t spec_verify_greedy_chain(const void* logits, sv_dtype_t dtype, int64_t ld, int32_t batch, int32_t m,
                                     int32_t vocab, const int32_t* verify_ids, const int64_t* row_slots,
                                     const int64_t* seq_lens, const sv_out_t* out, void* ws, size_t ws_bytes,
                                     cudaStream_t stream);

/*
 * Greedy tree verification ([SGO] "为什么结果不受 draft 影响", verify_tree_greedy;
 * [E2D] §2.4, §3.4).  Request b has `nodes` nodes (node 0 = root / anchor);
 * node i owns logits row b*nodes + i, carries token tokens[b][i] and has parent
 * parents[b][i] (-1 for the root, otherwise 0 <= parent < i).  From the root,
 * the walk moves to the first child (ascending node index, or the order of the
 * optional first_child / next_sibling lists, both [B, nodes], -1 terminated)
 * whose token equals the current row's argmax; the bonus is the argmax of the
 * last node's row.  nodes <= 1024.
 */
sv_status_t spec_verify_greedy_tree(const void* logits, sv_dtype_t dtype, int64_t ld, int32_t batch, int32_t nodes,
                                    int32_t vocab, const int32_t* tokens, const int32_t* parents,
                                    const int32_t* first_child, const int32_t* next_sibling,
                                    const int64_t* row_slots, const int64_t* seq_lens, const sv_out_t* out,
                                    void* ws, size_t ws_bytes, cudaStream_t stream);

/*
 * p/q rejection chain ([E2D] §1.2: alpha = min(1, p/q), residual
 * p' = [p - q]_+ / sum [p - q]_+; temperature-scaled softmax p = softmax(l/T),
 * §6.2).  Row j of a request accepts its draft d iff u_accept[row] * q[row][d]
 * < p_row(d); at the first rejection the correction is drawn from the residual
 * of that row, and when every draft passes the bonus is drawn from p of the
 * last row.  Draws use inverse CDF: the smallest v whose running weight sum
 * exceeds u_final[b] * S (§6.2, sample_path()).  q [rows, ldq] fp32 is the
 * proposal actually sampled from ([E2D] §5.6.1, §6.5); the last row of each
 * request is never read.  temperature [B], u_accept [rows], u_final [B] fp32.
 */
sv_status_t spec_verify_rejection_chain(const void* logits, sv_dtype_t dtype, int64_t ld, int32_t batch, int32_t m,
                                        int32_t vocab, const int32_t* verify_ids, const float* q, int64_t ldq,
                                        const float* temperature, const float* u_accept, const float* u_final,
                                        const int64_t* row_slots, const int64_t* seq_lens, const sv_out_t* out,
                                        void* ws, size_t ws_bytes, cudaStream_t stream);

/*
 * Verification by independent target sampling and prefix match ([E2D] §1.2:
 * a verification of its own, distinct from p/q rejection; the DFlash
 * inference loop: sample the target's posterior at every block position, the
 * accept length is the longest prefix where draft and sample agree, and the
 * first mismatch emits the sample).  Same layout and outputs as
 * spec_verify_rejection_chain, without q: row i's target token is drawn by
 * inverse CDF with u_sample[i] (argmax for a greedy request), draft
 * verify_ids[i + 1] is accepted iff it equals that draw, and the first
 * rejected row (or the last row when every draft is accepted) emits its own
 * draw.  No row is drawn in full except the one emitting: the statistics pass
 * also sums each row's probabilities below its draft token, and the draw
 * equals the draft iff u * Z lies in [that sum, that sum + p(draft) * Z).
 * ws: spec_verify_workspace_bytes(batch * (m + 1), batch, vocab, m + 1) bytes.
 */
sv_status_t spec_verify_sample_match_chain(const void* logits, sv_dtype_t dtype, int64_t ld, int32_t batch,
                                           int32_t m, int32_t vocab, const int32_t* verify_ids,
                                           const float* temperature, const float* u_sample, const int64_t* row_slots,
                                           const int64_t* seq_lens, const sv_out_t* out, void* ws, size_t ws_bytes,
                                           cudaStream_t stream);

/*
 * p/q rejection chain with a SPARSE q ([E2D] §6.2, §6.5: a candidate selector
 * proposes from K candidates; its q is zero outside them, and tokens outside
 * the candidates can still come out through the residual [p - q]_+).  Same
 * arguments and results as spec_verify_rejection_chain, with q replaced by
 * candidate lists: cand_ids / cand_probs [rows, ldc] (device int32 / fp32,
 * ldc >= num_cands, 1 <= num_cands <= 1024); row i's list describes the q that
 * proposed verify_ids[i + 1]: q_i(v) = the sum of cand_probs[i][c] over c with
 * cand_ids[i][c] == v.  Id -1 is padding; any other id outside [0, vocab) is
 * ignored and sets SV_DEV_TOKEN_RANGE for the request when it appears in one of
 * the request's tested rows (all rows but its last).  No dense q is read or
 * formed; the final draw of a rejected request reads that row's list in place,
 * so the lists, like every input, must stay unchanged until the call's work on
 * the stream has completed.  ws: at least
 * spec_verify_sparse_workspace_bytes(batch * (m + 1), batch, vocab, m + 1,
 * num_cands) bytes (same rules as every workspace; num_cands does not change
 * the size).
 */
size_t spec_verify_sparse_workspace_bytes(int64_t rows, int32_t batch, int32_t vocab, int32_t max_len,
                                          int32_t num_cands);

sv_status_t spec_verify_rejection_chain_sparse(const void* logits, sv_dtype_t dtype, int64_t ld, int32_t batch,
                                               int32_t m, int32_t vocab, const int32_t* verify_ids,
                                               const int32_t* cand_ids, const float* cand_probs, int32_t num_cands,
                                               int64_t ldc, const float* temperature, const float* u_accept,
                                               const float* u_final, const int64_t* row_slots,
                                               const int64_t* seq_lens, const sv_out_t* out, void* ws,
                                               size_t ws_bytes, cudaStream_t stream);

/*
 * Ragged p/q rejection ([E2D] §5.6.5: verify_lens include the anchor, compact
 * offsets, e.g. lens [4,2,6] -> [0,4,6,12]).  Request b owns rows
 * [cu_seqlens[b], cu_seqlens[b+1]) of the total_rows rows; lengths must lie in
 * [1, max_len] (length 1 = bonus only).  A request whose range is invalid gets
 * SV_DEV_BAD_LAYOUT and commits nothing.  Otherwise as the rejection chain.
 */
sv_status_t spec_verify_rejection_ragged(const void* logits, sv_dtype_t dtype, int64_t ld, int32_t batch,
                                         int64_t total_rows, int32_t max_len, int32_t vocab,
                                         const int32_t* cu_seqlens, const int32_t* verify_ids, const float* q,
                                         int64_t ldq, const float* temperature, const float* u_accept,
                                         const float* u_final, const int64_t* row_slots, const int64_t* seq_lens,
                                         const sv_out_t* out, void* ws, size_t ws_bytes, cudaStream_t stream);

/*
 * Target-only tree sampling ([SGO] "为什么结果不受 draft 影响":
 * tree_speculative_sampling_target_only uses only target probabilities, draft
 * probabilities passed as 0, thresholds default 1.0).  At node cur with
 * uniform u = u_accept[row(cur)], children are visited in order with
 * c += p_cur(token); the first child with u < c / threshold_acc or
 * p_cur(token) >= threshold_single is accepted.  A sibling repeating an
 * earlier sibling's token is skipped (SV_DEV_DUP_SIBLING).  If no child is
 * accepted the final token is drawn from p_cur with the children's tokens
 * zeroed; at a leaf, from p_leaf.  With both thresholds 1.0 the output law
 * equals the target's.  threshold_acc must be > 0 and finite.  Tree layout as
 * in spec_verify_greedy_tree.
 */
sv_status_t spec_verify_target_only_tree(const void* logits, sv_dtype_t dtype, int64_t ld, int32_t batch,
                                         int32_t nodes, int32_t vocab, const int32_t* tokens,
                                         const int32_t* parents, const int32_t* first_child,
                                         const int32_t* next_sibling, const float* temperature,
                                         float threshold_single, float threshold_acc, const float* u_accept,
                                         const float* u_final, const int64_t* row_slots, const int64_t* seq_lens,
                                         const sv_out_t* out, void* ws, size_t ws_bytes, cudaStream_t stream);

/*
 * p/q rejection chain without a caller workspace.  (The pages have no
 * counterpart: this is a deployment convenience of this library.)
 *
 * For callers that cannot provide device scratch memory — for example a plugin
 * that its host framework hands only input and output buffers, code that runs
 * after a serving engine has reserved all device memory for itself, or an
 * embedding that must not allocate at call time.  Same arguments and results as
 * spec_verify_rejection_chain, minus ws / ws_bytes: the library uses one fixed
 * scratch area of SV_NOALLOC_SCRATCH_BYTES bytes in its own device image (every
 * GPU that uses the library keeps it until the process exits) and allocates
 * nothing.  Problems whose workspace would exceed that size
 * (spec_verify_workspace_bytes(batch*(m+1), batch, vocab, m+1) >
 * SV_NOALLOC_SCRATCH_BYTES) return SV_ERR_WORKSPACE_TOO_SMALL, and argument
 * errors their status code, before anything is enqueued or any CUDA call is
 * made.  The first call in each CUDA context (on each device, and again after a
 * device reset) looks up the area's device address; make it before any stream
 * capture starts.  Every call clears the area's counter words on `stream` before
 * launching; all calls share the area, so calls that overlap on the GPU (other
 * streams or host threads) race — serialise them.
 */
#define SV_NOALLOC_SCRATCH_BYTES ((size_t)4 << 20)

sv_status_t spec_verify_rejection_chain_noalloc(const void* logits, sv_dtype_t dtype, int64_t ld, int32_t batch,
                                                int32_t m, int32_t vocab, const int32_t* verify_ids, const float* q,
                                                int64_t ldq, const float* temperature, const float* u_accept,
                                                const float* u_final, const int64_t* row_slots,
                                                const int64_t* seq_lens, const sv_out_t* out, cudaStream_t stream);

/*
 * Test and diagnostic hooks (the pages have no counterpart; not for production use).
 *
 * spec_verify_noalloc_fill_counters sets every byte of the no-allocation scratch
 * area's counter words (the words each spec_verify_rejection_chain_noalloc call
 * clears before it launches) to value & 0xff, on `stream`, in the current
 * context: a test uses it to show that a call does not depend on what an earlier
 * call left there.  Returns SV_ERR_CUDA if the area cannot be reached.
 *
 * spec_verify_set_hand_off_limit_ns(ns), ns > 0, puts the row-statistics kernel
 * of every later call, in every thread, into its expiry test: each in-CTA
 * hand-off wait gives up after ns nanoseconds, and one wait on a barrier that
 * nothing completes is sure to; the kernel then stops, waits (with the normal
 * one-second limit) for its own bulk copies still in flight, and raises the
 * workspace error word, so the call's requests report SV_DEV_TIMEOUT.  ns = 0
 * (the default) restores normal operation.  After a timed-out call, zero-fill
 * the workspace before using it again.  Always returns SV_OK.
 */
sv_status_t spec_verify_noalloc_fill_counters(uint32_t value, cudaStream_t stream);
sv_status_t spec_verify_set_hand_off_limit_ns(uint64_t ns);

/*
 * Row statistics on their own (the single pass every entry point starts
 * with; [E2D] §1.2 and §6.2: the target distribution of a row is
 * softmax(l / T), and a greedy row takes its argmax): for each of `rows`
 * rows, the maximum M (float), the lowest argmax (-1 for an all -inf row),
 * Z = sum_v exp((l_v - M)/T) with T = row_temp[row] (0 when row_temp is NULL
 * or the row is greedy), p at probe[row] (when probe and out_p are given),
 * and SV_DEV_NONFINITE in row_flags.  out_z is double.  All outputs [rows],
 * device, caller-owned; out_p / probe / row_temp may be NULL.  ws: at least
 * spec_verify_workspace_bytes(rows, 1, vocab, 1) bytes (same rules as every
 * workspace).  Argument errors (SV_ERR_NULL_ARG for a missing logits,
 * out_max, out_argmax or out_z; the logits checks of every entry point)
 * return before anything is enqueued.
 */
sv_status_t spec_verify_row_stats(const void* logits, sv_dtype_t dtype, int64_t ld, int64_t rows, int32_t vocab,
                                  const float* row_temp, const int32_t* probe, float* out_max,
                                  int32_t* out_argmax, double* out_z, float* out_p, uint32_t* row_flags,
                                  void* ws, size_t ws_bytes, cudaStream_t stream);

/*
 * DSpark verify-length scheduling ([E2D] §5.6.3 host budget, §5.6.4 device
 * allocation): how many draft rows each request verifies in the next round.
 *
 * spec_verify_dspark_budget runs on the HOST (no GPU, host pointers).  It picks
 * the extra draft budget K from historical survival scores: hist_survival[n]
 * holds one score per (request, draft position) in any order; NaN scores and
 * scores below eps are dropped, the rest sorted descending a_1 >= a_2 >= ...;
 * with N(K) = R + a_1 + ... + a_K (predicted committed tokens) and sps[M] the
 * speed (rounds per second) of a round with M target rows, M = 0 .. sps_len-1,
 *   *k_star = argmax over K with R + K < sps_len of N(K) * sps[R + K]
 * (the smaller K on ties; 0 when R >= sps_len).  Returns SV_ERR_NULL_ARG or
 * SV_ERR_BAD_SHAPE (n < 0, num_requests < 0, sps_len < 0) on bad arguments.
 *
 * spec_verify_dspark_verify_lens runs on the DEVICE.  survival [R, D] (device
 * fp32, row stride ld >= D floats) holds each request's current survival at
 * draft positions 1..D (a running product of confidences, so non-increasing
 * along a row).  Every (request r, position j) is a candidate; candidates are
 * ordered by survival descending, then position ascending, then request
 * ascending (no token id enters the order), and the first `budget` whose
 * survival is at least eps are selected (NaN orders last and is never
 * selected).  verify_lens[r] = clamp(1 + selected_r, min_len, max_len): one
 * anchor row plus the selected drafts (device int32 [R]).  ws: at least
 * spec_verify_dspark_workspace_bytes(R) bytes, zero-filled before its first
 * use; each completed call leaves it zeroed.  Host argument errors
 * (SV_ERR_NULL_ARG, SV_ERR_BAD_SHAPE for R, D or budget < 0, ld < D,
 * min_len < 1, max_len < min_len, R * D > 2^30; SV_ERR_WORKSPACE_TOO_SMALL)
 * return before anything is enqueued.
 */
size_t spec_verify_dspark_workspace_bytes(int32_t num_requests);

sv_status_t spec_verify_dspark_budget(const float* hist_survival, int64_t n, int32_t num_requests, const float* sps,
                                      int32_t sps_len, float eps, int32_t* k_star);

sv_status_t spec_verify_dspark_verify_lens(const float* survival, int32_t num_requests, int32_t num_drafts,
                                           int64_t ld, int32_t budget, int32_t min_len, int32_t max_len, float eps,
                                           int32_t* verify_lens, void* ws, size_t ws_bytes, cudaStream_t stream);

/*
 * Tree-verify inputs from parent lists ([E2D] §2.4: a flattened tree where each
 * node sees the committed history, its ancestors and itself, with position ids
 * from the path depth; §3.4: tree construction produces the mask, positions
 * and the retrieve index / next-token / next-sibling arrays of the verify walk).
 * parents [batch, nodes] (device int32): node 0 is the root (parent -1), every
 * other node's parent has a smaller index.  seq_lens [batch] (device int64,
 * may be NULL for 0): the committed length before the tree.  Outputs, all
 * device, caller-owned:
 *   positions      [batch, nodes] int64  seq_len + depth
 *   mask           [batch, nodes, nodes] uint8, mask[b][i][j] = 1 iff node j
 *                  is node i or one of its ancestors
 *   retrieve_index [batch, nodes] int32  b * nodes + i
 *   first_child    [batch, nodes] int32  lowest-index child, -1 if none
 *   next_sibling   [batch, nodes] int32  next higher-index node with the same
 *                  parent, -1 if none (the format the tree entry points accept)
 *   status         [batch] uint32        SV_DEV_BAD_TREE for an invalid parent
 *                  array (its outputs: depth 0, identity mask, -1 links)
 * 1 <= nodes <= 1024, batch <= 65535; SV_ERR_BAD_SHAPE / SV_ERR_NULL_ARG
 * before anything is enqueued.  No workspace.
 */
sv_status_t spec_verify_build_tree(const int32_t* parents, const int64_t* seq_lens, int32_t batch, int32_t nodes,
                                   int64_t* positions, uint8_t* mask, int32_t* retrieve_index,
                                   int32_t* first_child, int32_t* next_sibling, uint32_t* status,
                                   cudaStream_t stream);

/*
 * A paged KV cache, as the attention and commit calls below take it.  (The
 * pages describe verification on top of such a cache - [E2D] §2.4 the tree
 * mask over committed history and draft nodes, §5.6.6 and §8.1 the committed
 * KV slots - without fixing its layout.)
 *
 * k and v are [layers, pages, page_size, heads, head_dim] arrays with the same
 * strides (in elements); head_dim is dense, every other axis may have any
 * stride (head-major pages are a matter of strides).  Slot s is entry
 * s % page_size of page s / page_size.  Position x of request b is entry
 * x % page_size of page page_table[b * ld_table + x / page_size]; the table
 * has max_pages entries a request, so positions [0, max_pages * page_size)
 * exist.  Base pointers must be 16-byte aligned; head_dim and every stride,
 * in bytes, multiples of 16; head_dim <= 256.
 */
typedef struct {
  void* k;
  void* v;
  sv_dtype_t dtype;
  int32_t layers;
  int32_t pages;
  int32_t page_size;
  int32_t heads;
  int32_t head_dim;
  int64_t layer_stride;
  int64_t page_stride;
  int64_t slot_stride;
  int64_t head_stride;
  const int32_t* page_table; /* [batch, ld_table], device */
  int32_t max_pages;
  int64_t ld_table;
} sv_kv_cache_t;

/*
 * Attention of each request's new rows (a single decoded token, a draft chain,
 * a ragged block or a draft tree) over its committed history in the paged
 * cache and over the new rows themselves ([E2D] §2.4: each node sees the
 * committed history, its ancestors and itself).
 *
 * Request b owns rows [b * max_len, (b + 1) * max_len), or, with cu_seqlens,
 * [cu_seqlens[b], cu_seqlens[b+1]) of length 1..max_len.  Its row i has query
 * heads q[row * q_row_stride + h * q_head_stride + d] (cache dtype), h <
 * num_heads, a multiple of the cache's heads; query head h reads cache head
 * h / (num_heads / heads).  The row sees positions [0, seq_lens[b]) and, of the
 * request's own rows, row j iff mask[b][i][j] != 0 (mask: [batch, max_len,
 * max_len] uint8, the format spec_verify_build_tree writes), or j <= i when
 * mask is NULL.  The K/V of the request's rows are already in the cache, at
 * row_slots[row], or at positions seq_lens[b] + j when row_slots is NULL.
 *
 *   s_x = scale * (q . k_x)   out = sum_x softmax(s)_x v_x   lse = ln sum_x exp(s_x)
 *
 * with fp32 statistics and sums; out (cache dtype, its own row and head
 * strides, the larger at least what the other axis spans) is rounded once.
 * lse [total_rows, num_heads] fp32 may be NULL.  A row that sees nothing, or
 * only scores of -inf, has out 0 and lse -inf.  K/V of entries a row does not
 * see do not influence it, whatever they hold.
 *
 * dev_status [batch]: SV_DEV_BAD_LAYOUT for an invalid row range (the request's
 * rows are left unwritten) or a negative seq_lens[b] (taken as 0);
 * SV_DEV_SLOT_RANGE when a page, slot or position lies outside the cache (its
 * entry is not seen).  max_len * num_heads may be at most 2^24, batch at most
 * 65535.  ws: at least spec_verify_attention_workspace_bytes(...)
 * bytes, zero-filled before its first use and left zeroed where it matters by
 * every call; a workspace that served another entry point is zero-filled again.
 */
size_t spec_verify_attention_workspace_bytes(int32_t batch, int32_t max_len, int32_t num_heads, int32_t kv_heads,
                                             int32_t head_dim);

sv_status_t spec_verify_paged_attention(const void* q, int64_t q_row_stride, int64_t q_head_stride,
                                        int32_t num_heads, const sv_kv_cache_t* cache, int32_t layer, int32_t batch,
                                        int64_t total_rows, int32_t max_len, const int32_t* cu_seqlens,
                                        const int64_t* seq_lens, const int64_t* row_slots, const uint8_t* mask,
                                        float scale, void* out, int64_t out_row_stride, int64_t out_head_stride,
                                        float* lse, uint32_t* dev_status, void* ws, size_t ws_bytes,
                                        cudaStream_t stream);

/*
 * The KV move that a verification's commit lists describe ([E2D] §5.6.6,
 * §8.1): for every request b and entry e in [commit_cu[b], commit_cu[b+1]), in
 * every layer, K and V of slot commit_src_slot[e] are copied to position
 * commit_dst_pos[e] of the request.  All of a request's reads come before its
 * writes, so its sources and destinations may overlap (drafts staged in
 * place); those of different requests must not.  A request commits at most
 * max_len (<= 1024) entries, and the lists hold list_len entries.
 * Every entry of the cache must have memory of its own: SV_ERR_UNSUPPORTED when
 * an axis is repeated (a stride of 0) or its stride is less than the axes with
 * smaller ones span, and when K and V share memory (they may be interleaved).
 * dev_status [batch] (may be NULL): SV_DEV_BAD_LAYOUT when the request's range
 * is invalid (nothing is moved), SV_DEV_SLOT_RANGE when an entry's slot or
 * position lies outside the cache (that entry is not moved).
 */
sv_status_t spec_verify_kv_commit(const sv_kv_cache_t* cache, int32_t batch, int32_t max_len, int64_t list_len,
                                  const int32_t* commit_cu, const int64_t* commit_src_slot,
                                  const int64_t* commit_dst_pos, uint32_t* dev_status, cudaStream_t stream);

/*
 * Log probabilities of given tokens, with each row's entropy and its most
 * likely alternatives ([E2D] §6.2: the target distribution softmax(l / T)).
 * (What serving returns beside committed tokens, and what draft training takes
 * its loss from.)
 *
 * Output i of n describes logits row row_index[i] (row i when row_index is
 * NULL; -1 is padding, so a verification's accept_rows can be passed as it is;
 * any other index outside [0, rows) is treated as padding and flagged
 * SV_DEV_BAD_LAYOUT).  With T = row_temp[i] (1 when row_temp is NULL, or for a
 * greedy temperature: the unscaled distribution) and M the largest usable
 * logit (NaN and +inf are ignored and flagged SV_DEV_NONFINITE, as is an all
 * -inf row):
 *   row_max[i] = M,  log_z[i] = ln sum_v exp((l_v - M) / T)
 *   logprob[i][j] = (l_id - M) / T - log_z   for id = ids[i * ldi + j]
 *   entropy[i] = - sum_v p_v ln p_v
 *   top_ids / top_logprob [i][k]: the k-th most likely token, equal logits
 *     resolving to the lowest index; -1 and -inf where fewer than top_k tokens
 *     have a logit above -inf
 * logprob is 0 for id -1 (padding), -inf for a token without probability and
 * for an id outside [0, vocab) (flagged SV_DEV_TOKEN_RANGE).  A padding output
 * has logprob 0 for every id, entropy 0, row_max -inf, log_z 0, top_ids -1; an
 * all -inf row has entropy 0, row_max -inf, log_z -inf, logprob -inf.
 * entropy, row_max, log_z and flags may be NULL, as may logprob when num_ids is
 * 0 and the top arrays when top_k is 0.  num_ids <= 1024, top_k <= 64.  Sums
 * and statistics are held in fp32, joined over a row in a fixed order.
 * ws: at least spec_verify_logprobs_workspace_bytes(n, vocab, top_k) bytes,
 * zero-filled before its first use, left zeroed where it matters (zero-fill a
 * workspace that served another entry point).
 */
size_t spec_verify_logprobs_workspace_bytes(int64_t n, int32_t vocab, int32_t top_k);

sv_status_t spec_verify_token_logprobs(const void* logits, sv_dtype_t dtype, int64_t ld, int64_t rows, int32_t vocab,
                                       int64_t n, const int32_t* row_index, const int32_t* ids, int32_t num_ids,
                                       int64_t ldi, const float* row_temp, int32_t top_k, float* logprob,
                                       float* entropy, float* row_max, float* log_z, int32_t* top_ids,
                                       float* top_logprob, uint32_t* flags, void* ws, size_t ws_bytes,
                                       cudaStream_t stream);

/*
 * The gradient of spec_verify_token_logprobs (row i describing logits row i)
 * by the logits, given g_logprob [rows, num_ids], g_entropy [rows] (or NULL)
 * and g_top [rows, top_k] (or NULL), with what the forward call kept: row_max,
 * log_z, entropy (needed with g_entropy) and top_ids (needed with g_top):
 *   dlogits_v = 1/T ( sum_{j: id_j = v} g_j + sum_{k: top_k = v} gt_k - p_v G
 *                     - g_entropy p_v (ln p_v + entropy) ),  G = sum g + sum gt
 * over ids that are usable tokens; -1, ids outside [0, vocab) and tokens with
 * a NaN or +inf logit have no part in it, and neither such logits nor an all
 * -inf row receive a gradient.  dlogits [rows, ldd] has the logits' dtype (16-byte
 * aligned rows), is rounded once, and must not overlap the logits
 * (SV_ERR_UNSUPPORTED).  Either of num_ids and top_k may be 0.  No workspace.
 */
sv_status_t spec_verify_token_logprobs_backward(const void* logits, sv_dtype_t dtype, int64_t ld, int64_t rows,
                                                int32_t vocab, const int32_t* ids, int32_t num_ids, int64_t ldi,
                                                const float* row_temp, const float* row_max, const float* log_z,
                                                const float* entropy, const int32_t* top_ids, int32_t top_k,
                                                const float* g_logprob, const float* g_entropy, const float* g_top,
                                                void* dlogits, int64_t ldd, cudaStream_t stream);

/*
 * A paged KV cache held in 4 bits: 16 neighbouring columns of a head share a
 * scale, and a value is the scale times a code.  Codes are e2m1 (a sign bit,
 * and 0, 0.5, 1, 1.5, 2, 3, 4 or 6); a scale is one byte, a positive half float's
 * upper bits without the sign (five exponent bits, three of mantissa), at most
 * 10240 (larger patterns are read as that).  Values are exact in bf16 and fp32.
 *
 * data is [layers, pages, heads, block]: the block of a page and head holds K's
 * codes and V's codes ([page_size, head_dim / 2] bytes each, the even column in
 * the lower half of a byte), K's scales and V's scales ([page_size, head_dim /
 * 16] bytes each), and is padded to a multiple of 16 bytes:
 * spec_verify_packed_kv_block_bytes(page_size, head_dim), 0 for sizes that
 * have none.  head_dim is a multiple of 32, at most 256.  The strides are in
 * bytes, multiples of 16, like the base pointer.  Slots, positions and the page
 * table are those of sv_kv_cache_t.  dtype is that of the rows that go with the
 * cache: new keys and values, queries, outputs (attention takes bf16 alone).
 * Pages whose size divides 128, or is a multiple of it, are brought in block by
 * block; all others row by row, which takes attention up to six times as long.
 */
typedef struct {
  void* data;
  sv_dtype_t dtype;
  int32_t layers;
  int32_t pages;
  int32_t page_size;
  int32_t heads;
  int32_t head_dim;
  int64_t layer_stride;
  int64_t page_stride;
  int64_t head_stride;
  const int32_t* page_table; /* [batch, ld_table], device */
  int32_t max_pages;
  int64_t ld_table;
} sv_packed_kv_cache_t;

size_t spec_verify_packed_kv_block_bytes(int32_t page_size, int32_t head_dim);

/*
 * Rows of a batch and their places in a cache.  Request b owns rows [b *
 * max_len, (b + 1) * max_len), or, with cu_seqlens [batch + 1], rows
 * [cu_seqlens[b], cu_seqlens[b+1]) of total_rows, 0..max_len of them; rows of
 * no request are left alone.  Its row j lies at slot row_slots[row], or, when
 * row_slots is NULL, at position seq_lens[b] + j.
 */
typedef struct {
  int32_t batch;
  int32_t max_len;
  int64_t total_rows;
  const int32_t* cu_seqlens; /* [batch + 1] or NULL   */
  const int64_t* seq_lens;   /* [batch] or NULL       */
  const int64_t* row_slots;  /* [total_rows] or NULL  */
} sv_rows_t;

/*
 * A rotation by position: pair i < pairs of a head's columns turns by the angle
 * position * inv_freq[i].  A pair is columns (i, i + pairs), or (2 i, 2 i + 1)
 * when interleaved; columns from 2 * pairs on are left as they are.  The
 * rotated columns are also multiplied by magnitude (1 for none).  Angles are
 * reduced in more than fp32, to 2^-25 of a radian or better for inv_freq up to 1:
 * far positions, to the ends of 64 bits, lose nothing.
 */
typedef struct {
  const float* inv_freq; /* [pairs], device */
  int32_t pairs;
  int32_t interleaved;
  float magnitude;
} sv_rotation_t;

/*
 * New rows of a layer go into the cache, their keys rotated on the way, and
 * their queries are rotated beside them (what a model's layer does between its
 * projections and spec_verify_paged_attention; [E2D] §2.4: position ids come
 * from the depth in the draft tree, so they are given apart from the places).
 *
 *   (x, y) -> magnitude (x cos a - y sin a, y cos a + x sin a)   for each pair
 *
 * k and v: [rows, heads, head_dim] of the cache's dtype, q and q_out: [rows,
 * num_heads, head_dim], each with its own row and head strides in elements (rows
 * and strides multiples of 16 bytes).  positions [total_rows] (int64; NULL:
 * seq_lens[b] + j) are what rows are rotated by; rotation NULL: nothing is
 * rotated.  q NULL: only keys and values.  q_out may be q itself; any other
 * overlap of q_out with q, k, v or the cache, and of these with the cache, is
 * refused (SV_ERR_UNSUPPORTED), as are a cache whose entries share memory and
 * rows or heads of q_out that lie over one another.  seq_lens may be NULL when
 * row_slots and positions are given.
 *
 * Arithmetic is fp32, rounded once to the dtype; values are copied as they are.
 * The 4-bit cache takes the rotated values before any rounding: each group's
 * scale is the one nearest to its largest magnitude / 6, each code the one nearest
 * to its value, both half way to the even one.  Keys are rotated in twice the
 * bits of fp32 for that: the choice is that of the exact rotation wherever it is
 * further than 2^-37 (|x| + |y|) magnitude from the middle of two (inv_freq up to 1).
 * Magnitudes above 61440 are stored as 61440, a NaN as 0.  Two rows of a call must not have the same place.
 *
 * dev_status [batch] is OR-ed into (zero it first): SV_DEV_BAD_LAYOUT for an
 * invalid row range or a negative seq_lens[b] (nothing of the request is
 * written), SV_DEV_SLOT_RANGE when a row's place lies outside the cache (it is
 * not stored; its query is rotated all the same), SV_DEV_NONFINITE when a NaN
 * or an infinity went into the 4-bit cache.
 */
sv_status_t spec_verify_kv_append(const sv_kv_cache_t* cache, int32_t layer, const sv_rows_t* rows,
                                  const int64_t* positions, const sv_rotation_t* rotation, const void* k,
                                  int64_t k_row_stride, int64_t k_head_stride, const void* v, int64_t v_row_stride,
                                  int64_t v_head_stride, const void* q, int64_t q_row_stride, int64_t q_head_stride,
                                  int32_t num_heads, void* q_out, int64_t out_row_stride, int64_t out_head_stride,
                                  uint32_t* dev_status, cudaStream_t stream);

sv_status_t spec_verify_packed_kv_append(const sv_packed_kv_cache_t* cache, int32_t layer, const sv_rows_t* rows,
                                         const int64_t* positions, const sv_rotation_t* rotation, const void* k,
                                         int64_t k_row_stride, int64_t k_head_stride, const void* v,
                                         int64_t v_row_stride, int64_t v_head_stride, const void* q,
                                         int64_t q_row_stride, int64_t q_head_stride, int32_t num_heads, void* q_out,
                                         int64_t out_row_stride, int64_t out_head_stride, uint32_t* dev_status,
                                         cudaStream_t stream);

/*
 * The entries of given rows' places as they lie in the cache (of the 4-bit
 * cache: the values that they stand for), in num_layers layers from `layer` on:
 * what spec_verify_kv_append with the same rows has stored.  k and v:
 * [num_layers, rows, heads, head_dim] of the cache's dtype, with the same
 * strides in elements (head_dim dense; multiples of 16 bytes); rows, heads and
 * layers must not lie over one another, and the address ranges of k, v and the
 * cache must not meet (SV_ERR_UNSUPPORTED).  A row whose place lies outside the cache is 0.
 * dev_status [batch] is OR-ed into, with the bits of spec_verify_kv_append.
 */
sv_status_t spec_verify_kv_read(const sv_kv_cache_t* cache, int32_t layer, int32_t num_layers, const sv_rows_t* rows,
                                void* k, void* v, int64_t layer_stride, int64_t row_stride, int64_t head_stride,
                                uint32_t* dev_status, cudaStream_t stream);

sv_status_t spec_verify_packed_kv_read(const sv_packed_kv_cache_t* cache, int32_t layer, int32_t num_layers,
                                       const sv_rows_t* rows, void* k, void* v, int64_t layer_stride,
                                       int64_t row_stride, int64_t head_stride, uint32_t* dev_status,
                                       cudaStream_t stream);

/*
 * spec_verify_paged_attention over a 4-bit cache (q and out bf16), with the same arguments,
 * results and workspace.  Scores are products with the values that the cache
 * stands for; statistics and sums are fp32.
 */
sv_status_t spec_verify_packed_attention(const void* q, int64_t q_row_stride, int64_t q_head_stride,
                                         int32_t num_heads, const sv_packed_kv_cache_t* cache, int32_t layer,
                                         int32_t batch, int64_t total_rows, int32_t max_len,
                                         const int32_t* cu_seqlens, const int64_t* seq_lens, const int64_t* row_slots,
                                         const uint8_t* mask, float scale, void* out, int64_t out_row_stride,
                                         int64_t out_head_stride, float* lse, uint32_t* dev_status, void* ws,
                                         size_t ws_bytes, cudaStream_t stream);

/*
 * spec_verify_kv_commit in a 4-bit cache: codes and scales are moved as they
 * are.  SV_ERR_UNSUPPORTED when blocks share memory.
 */
sv_status_t spec_verify_packed_kv_commit(const sv_packed_kv_cache_t* cache, int32_t batch, int32_t max_len,
                                         int64_t list_len, const int32_t* commit_cu, const int64_t* commit_src_slot,
                                         const int64_t* commit_dst_pos, uint32_t* dev_status, cudaStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* SPECVERIFY_H */
