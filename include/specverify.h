/*
 * specverify.h -- C ABI of libspecverify: batched speculative-decoding
 * verification on one GB300 (sm_103a).
 *
 * Source of the method: "Accelerating Sonar through speculation"
 * (Perplexity blog), sections "Speculative decoding", "Target-Draft",
 * "EAGLE", "MTP" and "MTP schedule for a single token", and the rule of the
 * work it cites first, "Fast Inference from Transformers via Speculative
 * Decoding": accept a drafted token x with probability min(1, p(x)/q(x));
 * at the first rejection draw from norm(max(0, p - q)); after a full accept
 * draw a bonus token from the target's last row.
 *
 * Conventions shared by every call:
 *  - Every array argument is a DEVICE pointer owned by the caller, except
 *    `params`, which is a host pointer read before the call returns.  The
 *    library allocates nothing and keeps no state between calls.
 *  - Work is enqueued on `stream` (NULL = the legacy default stream) and
 *    the call returns without synchronising.  Outputs are valid once the
 *    stream reaches that point.
 *  - Host-detectable errors (NULL required pointer, bad size, unsupported
 *    combination, workspace too small) are returned synchronously and
 *    nothing is enqueued.  SPEC_ERR_CUDA reports a failed launch.
 *  - Data-dependent errors found on the device (token id outside [0, V),
 *    NaN or +inf logits, a row with no finite entry, a malformed parent
 *    array, an out-of-range accepted length) OR a SPEC_DEVERR_* bit into
 *    *dev_error (zeroed by the call first) and give that request a defined
 *    fallback result (see each call).  The library never traps.
 *  - Logit rows are contiguous: element (b, i, v) sits at
 *    ((b * rows + i) * V + v).  V need not be a multiple of 8.
 *  - Random draws use counter-based Philox4x32-10 (Salmon, Moraes, Dror,
 *    Shaw, SC'11): key = (seed lo32, seed hi32), counter = (request lo32,
 *    position lo32, purpose | round << 8, request hi32), u = (word0 >> 8) *
 *    2^-24.  Results depend only on (inputs, seed, request id, position),
 *    not on the batch size or on a request's slot in the batch: bit for bit
 *    when every row starts on a 16-byte boundary (V * element size a
 *    multiple of 16 and 16-byte aligned base pointers); otherwise rows in
 *    different slots are summed in a different order, and only decisions
 *    that sit within rounding of a threshold can differ.
 *  - Calls that overlap on the GPU must not share output or workspace
 *    buffers.
 *  - Each call makes the device that holds its logits (or hidden states)
 *    current for its own launches and puts the caller's current device
 *    back before it returns.
 *  - The linear calls, the draft-side sampler and the calls around a
 *    verification (log probabilities, distillation, cache slots, the paged
 *    cache, logit adjustment) use
 *    dependent launches:
 *    a launch may be scheduled while the kernel before it on the stream is
 *    ending, and waits for that kernel to complete before it reads or
 *    writes anything.  Stream order is kept; after any other stream
 *    operation (a copy, an event) they are ordinary launches.
 *  - spec_append_kv, spec_adjust_logits and spec_keep_path take no workspace,
 *    and their results do not depend on the batch.
 *  - spec_token_logprobs, spec_distill_topk and spec_advance_blocks take no
 *    workspace.  The same call gives the same bits every time.  Ids, ranks
 *    and error bits of a row do not depend on the other rows; its floats
 *    may differ in their last bits with R, because the number of CTAs that
 *    share a row goes by it, and with the row's alignment.
 */
#ifndef SPECVERIFY_H
#define SPECVERIFY_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* A cudaStream_t. */
typedef struct CUstream_st* spec_stream_t;

typedef enum {
    SPEC_OK = 0,
    SPEC_ERR_INVALID_ARG = 1,  /* NULL required pointer, negative size, bad params */
    SPEC_ERR_UNSUPPORTED = 2,  /* valid but not implemented (e.g. size limits) */
    SPEC_ERR_WORKSPACE = 3,    /* workspace NULL or smaller than spec_workspace_size() */
    SPEC_ERR_CUDA = 4          /* a CUDA call or kernel launch failed */
} spec_status;

/* SPEC_F16: the calls over a paged cache only. */
typedef enum { SPEC_BF16 = 0, SPEC_F32 = 1, SPEC_F16 = 2 } spec_dtype;

/* How the children of a draft-tree node were drawn from the draft model
 * (section "EAGLE": Top-K candidates per node).  The residual update after
 * a rejected child depends on it. */
typedef enum {
    SPEC_CHILD_WOR = 0,           /* sampled without replacement */
    SPEC_CHILD_IID = 1,           /* sampled with replacement */
    SPEC_CHILD_DETERMINISTIC = 2  /* the K most likely draft tokens; draft logits unused */
} spec_child_mode;

typedef enum { SPEC_OP_LINEAR = 0, SPEC_OP_TREE = 1 } spec_op;

/* What a teacher's top-K log probabilities stand for (spec_distill_topk). */
typedef enum {
    SPEC_TAIL_RENORM = 0, /* the whole teacher: renormalised over the K tokens */
    SPEC_TAIL_BUCKET = 1  /* a part of it: what is left of 1 is one bucket over all other tokens */
} spec_tail_mode;

/* Philox purposes (counter word 2, low byte). */
#define SPEC_PURPOSE_ACCEPT 1
#define SPEC_PURPOSE_RESIDUAL 2
#define SPEC_PURPOSE_BONUS 3
#define SPEC_PURPOSE_DRAFT 4

/* Bits OR-ed into *dev_error. */
#define SPEC_DEVERR_TOKEN 1      /* a draft/node token outside [0, V) */
#define SPEC_DEVERR_NONFINITE 2  /* NaN or +inf logit, or no finite logit in a row */
#define SPEC_DEVERR_PARENT 4     /* parent[] not a tree rooted at 0 with parent[i] < i, deeper than max_depth,
                                    or a node with more than 64 children */
#define SPEC_DEVERR_LENGTH 8     /* compaction: accepted length or source row out of range */
#define SPEC_DEVERR_TIMEOUT 16   /* a wait for a bulk copy ran out (2 s).  Verification, sampling:
                                    the rows it left were recomputed by the two-pass route, so
                                    the results stand.  spec_token_logprobs: the rows are
                                    refused (SPEC_DEVERR_NONFINITE is set, too).
                                    spec_distill_topk: the call's results are not to be used */
#define SPEC_DEVERR_CAPACITY 32  /* cache blocks: the free list or a request's table row ran out; a slot or a block
                                    that the cache does not have */

typedef struct {
    float temperature;  /* 0 => greedy (argmax, ties to the lowest index); > 0 => sampled */
    float top_p;        /* in (0, 1): nucleus filter on p and q; >= 1 => off */
    uint64_t seed;      /* Philox key */
    int32_t child_mode; /* spec_child_mode; tree only */
} spec_sampling_params;

/*
 * Bytes of device workspace a call needs (16-byte alignment suffices).
 * op = SPEC_OP_LINEAR: k_or_N = k.  op = SPEC_OP_TREE: k_or_N = N.
 * Returns 0 for invalid sizes.
 */
size_t spec_workspace_size(spec_op op, int B, int k_or_N, int V, spec_dtype dtype);

/*
 * Linear verification (sections "Speculative decoding" and "Target-Draft":
 * the target scores every prefix of the k drafted tokens; the longest
 * accepted prefix is kept and the target's logits after it give one more
 * token, so k drafts yield at most k+1 tokens).
 *
 *  target_logits [B, k+1, V]  row i scores the token after the prefix plus
 *                             d_1..d_i (row k: after all k drafts).
 *  draft_logits  [B, k, V]    row i is the distribution d_{i+1} was drawn
 *                             from.  Unused (may be NULL) when
 *                             temperature == 0.
 *  draft_tokens  [B, k] int32 d_1..d_k.
 *  request_ids   [B] int64 or NULL (=> b); positions [B] int64 or NULL
 *                (=> 0): drafted token i (1-based) is at position
 *                positions[b] + i; the emitted token t* at
 *                positions[b] + a + 1.
 *  params        temperature T, top_p, seed (child_mode ignored).
 *  p = filter(softmax(target / T)), q = filter(softmax(draft / T)), filter
 *  = the top-p nucleus in (logit desc, index asc) order (a token is kept
 *  when the mass before it is < top_p), renormalised.
 *  Sampled (T > 0): d_i is accepted iff u_i < p_{i-1}(d_i) / q_{i-1}(d_i)
 *  (q == 0, a token outside q's nucleus, rejects; the ratio is taken from
 *  the logits' exponents when p or q only underflows fp32, so drafts far in
 *  the tail are decided by their true ratio), u_i from purpose ACCEPT; a =
 *  number of leading
 *  accepts.  If a < k, t* is the smallest v with C(v) > u * C(V-1), C the
 *  running sum of max(0, p_a - q_a) in index order and u from purpose
 *  RESIDUAL (if that residual is all zero, of p_a instead); if a == k, the
 *  same over p_k with purpose BONUS.
 *  Greedy (T == 0): d_i is accepted iff it is the lowest-index argmax of
 *  target row i-1; t* = argmax of target row a.
 *
 *  Outputs: accepted_len [B] (a), out_tokens [B, k+1] (d_1..d_a, t*, then
 *  -1), accept_prob [B, k] = min(1, p/q) for every drafted token (greedy:
 *  1 or 0) or NULL, token_probs [B, k, 2] = (p_{i}(d_{i+1}),
 *  q_{i}(d_{i+1})) or NULL, len_hist [k+1] histogram of a over the batch
 *  (zeroed by the call) or NULL, dev_error [1] or NULL.
 *  Invalid request (bad token, non-finite row): a = 0, t* = lowest-index
 *  argmax of target row 0 over entries that are neither NaN nor +inf,
 *  accept_prob and token_probs 0.
 *  workspace: spec_workspace_size(SPEC_OP_LINEAR, B, k, V, dtype) bytes.
 *  Limits: 1 <= B, 1 <= k <= 64, 1 <= V < 2^31 / (2k+1) / B rows*V.
 */
spec_status spec_verify_linear(const void* target_logits, const void* draft_logits, spec_dtype dtype,
                               const int32_t* draft_tokens, int B, int k, int V,
                               const int64_t* request_ids, const int64_t* positions,
                               const spec_sampling_params* params,
                               int32_t* accepted_len, int32_t* out_tokens, float* accept_prob,
                               float* token_probs, int32_t* len_hist, int32_t* dev_error,
                               void* workspace, size_t workspace_bytes, spec_stream_t stream);

/*
 * Linear verification followed by the compaction of the accepted positions
 * for the next draft step, in the same launches (section "MTP": token
 * t_{i+1} is drawn from logits computed from hidden state H_i; section "MTP
 * schedule for a single token": a kernel inserts the next target tokens,
 * with no host synchronisation).  Results as spec_verify_linear followed by
 * spec_compact_accepted(hidden, B, k+1, H, accepted_len, NULL, out_tokens,
 * k+1, out_hidden, offsets, next_tokens, ...), without the compaction's own
 * launch: the launch after the row statistics takes every request's
 * decisions and the packed offsets, and each request's draw CTA copies its
 * a_b + 1 hidden rows and writes their next tokens.
 *
 *  hidden       [B, k+1, H] bf16 (2-byte elements, copied bit for bit):
 *               row i is the hidden state after the prefix plus d_1..d_i.
 *  out_hidden   [B*(k+1), H] out: row offsets[b] + r = hidden[b, r, :],
 *               r = 0..a_b (rows past offsets[B] untouched).
 *  offsets      [B+1] out: offsets[0] = 0, offsets[b+1] = offsets[b] + a_b + 1.
 *  next_tokens  [B*(k+1)] out: next_tokens[offsets[b] + r] = out_tokens[b, r].
 *  An invalid request (see spec_verify_linear) contributes its row 0 and
 *  its fallback token.  Other arguments, outputs, limits and workspace as
 *  spec_verify_linear; the vector path wants H * 2 a multiple of 16 and
 *  16-byte aligned hidden pointers (else 2-byte copies).  B * (k+1) < 2^31.
 */
spec_status spec_verify_linear_compact(const void* target_logits, const void* draft_logits, spec_dtype dtype,
                                       const int32_t* draft_tokens, int B, int k, int V,
                                       const int64_t* request_ids, const int64_t* positions,
                                       const spec_sampling_params* params, const void* hidden, int H,
                                       int32_t* accepted_len, int32_t* out_tokens, float* accept_prob,
                                       float* token_probs, int32_t* len_hist, void* out_hidden, int32_t* offsets,
                                       int32_t* next_tokens, int32_t* dev_error, void* workspace,
                                       size_t workspace_bytes, spec_stream_t stream);

/*
 * The two launch groups of spec_verify_linear (and of
 * spec_verify_linear_compact), for callers that want to time them apart or
 * start the streaming pass as soon as the logits exist.
 * spec_linear_stats_decide reads every target row (and every draft row when
 * T > 0) once, writes per-row statistics into `workspace`, and in a
 * finishing launch runs every request's accept tests: it writes
 * accepted_len, accept_prob, token_probs, len_hist and dev_error (zeroing
 * len_hist and dev_error first) and keeps each request's decision and the
 * packed offsets in the workspace.  spec_linear_draw then draws every
 * request's t* and writes out_tokens and, when hidden is not NULL, the
 * compaction outputs of spec_verify_linear_compact (hidden NULL: H,
 * out_hidden, offsets and next_tokens are ignored).  Called in that order
 * on one stream with identical inputs, params and workspace, they give
 * exactly the results of the one-call forms (which are these two calls).
 * The workspace must not be reused between them.  Arguments as above.
 */
spec_status spec_linear_stats_decide(const void* target_logits, const void* draft_logits, spec_dtype dtype,
                                     const int32_t* draft_tokens, int B, int k, int V,
                                     const int64_t* request_ids, const int64_t* positions,
                                     const spec_sampling_params* params, int32_t* accepted_len, float* accept_prob,
                                     float* token_probs, int32_t* len_hist, int32_t* dev_error, void* workspace,
                                     size_t workspace_bytes, spec_stream_t stream);
spec_status spec_linear_draw(const void* target_logits, const void* draft_logits, spec_dtype dtype,
                             const int32_t* draft_tokens, int B, int k, int V, const int64_t* request_ids,
                             const int64_t* positions, const spec_sampling_params* params, const void* hidden, int H,
                             int32_t* out_tokens, void* out_hidden, int32_t* offsets, int32_t* next_tokens,
                             const void* workspace, size_t workspace_bytes, spec_stream_t stream);

/*
 * spec_verify_linear for callers that cannot allocate device memory at the
 * point where they verify (code inside a custom allocator or memory pool,
 * code whose device memory is fixed at start-up, code that only receives
 * buffers from a host framework).  The page describes no such variant; it
 * exists for those callers only.
 *
 * Same arguments and results as spec_verify_linear, without the workspace:
 * the workspace (per-row statistics, decisions, offsets, a counter) lives in
 * a fixed array of about 2.3 MiB inside the library's device image, which
 * every GPU that loads the library keeps until the process exits.  Limits: B * (2k + 1) <= 65536 rows, else
 * SPEC_ERR_UNSUPPORTED (nothing is enqueued).  The call allocates nothing
 * (no cudaMalloc, cudaFree or allocating library routine).  The first call
 * on each device looks up the array's device address once; make that first
 * call before any stream capture.  Every call shares the one array, so
 * calls that overlap on the GPU (different streams or host threads) race on
 * it; each call clears the counter and writes every record it later reads,
 * so no state carries over.
 */
spec_status spec_verify_linear_noalloc(const void* target_logits, const void* draft_logits, spec_dtype dtype,
                                       const int32_t* draft_tokens, int B, int k, int V,
                                       const int64_t* request_ids, const int64_t* positions,
                                       const spec_sampling_params* params, int32_t* accepted_len,
                                       int32_t* out_tokens, float* accept_prob, float* token_probs,
                                       int32_t* len_hist, int32_t* dev_error, spec_stream_t stream);

/*
 * Tree verification (section "EAGLE": a static draft tree explored with the
 * Top-K candidates of every node; the longest accepted root-to-leaf path is
 * kept plus one target token).
 *
 *  target_logits [B, N, V]   row n scores the token after node n's path
 *                            (node 0 = the root, the last committed token).
 *  draft_logits  [B, N, V]   row n is the draft distribution the children of
 *                            n were drawn from; may be NULL when T == 0 or
 *                            child_mode == SPEC_CHILD_DETERMINISTIC.
 *  node_tokens   [B, N] int32 token of each node (node 0's is ignored).
 *  parent        [N] int32   parent[0] = -1, 0 <= parent[i] < i.  The
 *                            children of n are tested in increasing index
 *                            order.
 *  max_depth     depth of the deepest node (host value; checked on the
 *                device); outputs have W = max_depth + 1 columns.
 *  At node n of depth t, with P = p_n and Q = q_n: child j (0-based) with
 *  token x is accepted iff u < P(x) / Q(x) (DETERMINISTIC: u < P(x)), u from
 *  purpose ACCEPT, round j, position positions[b] + t + 1.  After a reject:
 *  P <- norm(max(0, P - Q)) (DETERMINISTIC: P with x removed, renormalised;
 *  a zero residual leaves P unchanged), and Q <- Q with x removed,
 *  renormalised (WOR) or unchanged (IID).  An accept moves to that child.
 *  A leaf draws the bonus token from p_leaf (purpose BONUS); a node whose
 *  children are all rejected draws t* from the final P (purpose RESIDUAL),
 *  both by the inverse CDF above.  Greedy: descend into the first child
 *  whose token is the lowest-index argmax of p_n, else emit that argmax.
 *
 *  Outputs: accepted_len [B] (accepted depth a), path_nodes [B, W] (0, the
 *  accepted nodes, then -1), out_tokens [B, W] (their tokens, t*, then -1),
 *  dev_error [1] or NULL.  Invalid request: a = 0, path = [0], t* = argmax
 *  of target row 0 as for the linear call.
 *  workspace: spec_workspace_size(SPEC_OP_TREE, B, N, V, dtype) bytes.
 *  Limits: 1 <= N <= 1024, max_depth < N, at most 64 children per node.
 */
spec_status spec_verify_tree(const void* target_logits, const void* draft_logits, spec_dtype dtype,
                             const int32_t* node_tokens, const int32_t* parent, int B, int N, int V,
                             int max_depth, const int64_t* request_ids, const int64_t* positions,
                             const spec_sampling_params* params, int32_t* accepted_len, int32_t* path_nodes,
                             int32_t* out_tokens, int32_t* dev_error, void* workspace, size_t workspace_bytes,
                             spec_stream_t stream);

/*
 * Tree verification with a tree of its own for every request (section
 * "EAGLE": the tree explored is fixed (EAGLE) or dynamically shaped
 * (EAGLE-2, in the page's citation); each request's tree is then its own).
 * The walk at every node is spec_verify_tree's; only the shape differs:
 *
 *  parent  [B, N] int32   row b is request b's parent array over its nodes
 *                         (parent[b, 0] = -1, 0 <= parent[b, i] < i).
 *  n_nodes [B] int32      request b has nodes 0 .. n_nodes[b]-1; its rows,
 *                         tokens and parent entries past them are not read.
 *  target_logits, draft_logits [B, N, V] and node_tokens [B, N] as for
 *  spec_verify_tree, N the largest tree; max_depth bounds every request's
 *  depth (outputs have W = max_depth + 1 columns).
 *  A request with n_nodes outside 1 .. N, or an invalid parent row, is
 *  invalid (SPEC_DEVERR_PARENT) with the defined fallback.  n_nodes NULL
 *  returns SPEC_ERR_INVALID_ARG; other host checks and limits as above.
 */
spec_status spec_verify_tree_dynamic(const void* target_logits, const void* draft_logits, spec_dtype dtype,
                                     const int32_t* node_tokens, const int32_t* parent, const int32_t* n_nodes,
                                     int B, int N, int V, int max_depth, const int64_t* request_ids,
                                     const int64_t* positions, const spec_sampling_params* params,
                                     int32_t* accepted_len, int32_t* path_nodes, int32_t* out_tokens,
                                     int32_t* dev_error, void* workspace, size_t workspace_bytes,
                                     spec_stream_t stream);

/*
 * Compaction for the next draft step (section "MTP": token t_{i+1} is drawn
 * from logits computed from hidden state H_i, so token buffers sit one step
 * left of the hidden states; section "MTP schedule for a single token": a
 * kernel inserts the next target tokens into their slots with no host
 * synchronisation).
 *
 *  hidden       [B, T, H] 2-byte elements (bf16), copied bit for bit.
 *  accepted_len [B]; out_tokens [B, W]; path_nodes [B, W] or NULL (NULL =>
 *               rows 0..a_b, the linear layout).
 *  offsets      [B+1] out: offsets[0] = 0, offsets[b+1] = offsets[b] +
 *               a_b + 1.
 *  out_hidden   [B*W, H] out: row offsets[b] + r = hidden[b, src_r, :],
 *               src_r = path_nodes[b, r] (or r), r = 0..a_b.
 *  next_tokens  [B*W] out: next_tokens[offsets[b] + r] = out_tokens[b, r]
 *               (the token that follows the hidden row it is paired with).
 *  A request with a_b outside [0, W-1], or a source row outside [0, T),
 *  contributes no rows and sets SPEC_DEVERR_LENGTH.  Rows past
 *  offsets[B] are left untouched.
 *  Limits: H * 2 bytes must be a multiple of 16 when the hidden and output
 *  pointers are 16-byte aligned for the vector path; other cases use a
 *  2-byte path.  B * W < 2^31.
 */
spec_status spec_compact_accepted(const void* hidden, int B, int T, int H, const int32_t* accepted_len,
                                  const int32_t* path_nodes, const int32_t* out_tokens, int W, void* out_hidden,
                                  int32_t* offsets, int32_t* next_tokens, int32_t* dev_error,
                                  spec_stream_t stream);

/*
 * Draft-side sampling: one token per logit row drawn from
 * filter(softmax(row / T)), the draft model's own sampling of its tokens
 * (section "Target-Draft"), done on the GPU so that a token drawn from
 * logits carried over from the previous step reaches the next draft run
 * without a host round trip (section "MTP schedule for a single token").
 *
 *  logits       [R, V] bf16 or fp32, row-major.
 *  request_ids  [R] int64 or NULL (NULL => r); positions [R] int64 or NULL
 *               (NULL => 0).  Row r draws u = Philox(seed, request_ids[r],
 *               positions[r], purpose 4 = DRAFT, round 0) and returns the
 *               smallest v with C(v) > u * C(V-1), C the running sum of the
 *               filtered probabilities in index order (the filter as in
 *               spec_verify_linear: temperature, then the exact top-p
 *               nucleus with ties at the boundary kept in index order).
 *  out_tokens   [R] int32 out.
 *  params       temperature == 0: the lowest-index maximum over entries
 *               that are neither NaN nor +inf (0 when there is none), with
 *               no error.  temperature > 0: a row holding a NaN or +inf, or
 *               no finite entry, sets SPEC_DEVERR_NONFINITE and yields that
 *               argmax.  child_mode is ignored.
 *  dev_error    [1] or NULL.
 *  Errors: SPEC_ERR_INVALID_ARG (NULL logits / out_tokens / params, R < 1,
 *  V < 1, temperature < 0 or not finite, top_p <= 0 or NaN, dtype not
 *  bf16 or fp32); SPEC_ERR_UNSUPPORTED (V above 524,280).
 */
spec_status spec_sample_rows(const void* logits, spec_dtype dtype, int R, int V, const int64_t* request_ids,
                             const int64_t* positions, const spec_sampling_params* params, int32_t* out_tokens,
                             int32_t* dev_error, spec_stream_t stream);

/*
 * Log probabilities of given tokens, with the entropy and the top
 * alternatives of every row: what a server answers with beside the emitted
 * tokens, and what a target model hands to the training of its draft
 * (spec_distill_topk).  With the target logits of a verification as
 * [B * (k+1), V] and its out_tokens as [B * (k+1)], every emitted token is
 * scored by the row that emitted it and the -1 entries cost nothing.
 *
 *  logits       R rows of V elements; row r starts row_stride * r elements
 *               after logits (row_stride >= V; rows need not be aligned).
 *  tokens       [R] int32 or NULL (no given tokens).  A row whose token is
 *               -1 is skipped and not read.
 *  temperature  T > 0: p = softmax(row / T), over the whole row.
 *  top_k        0 .. min(V, 128).
 *  logprob      [R] out: log p(token).  Over rows of many kinds it was off
 *               by 8e-7 at most (1.5e-6 at V = 524,280 where all weights
 *               are alike) or, if that is more, by its rounding; where the
 *               token holds nearly all of the row, by 1.2e-6 of its value.
 *               NULL only when tokens is NULL.
 *  rank         [R] out or NULL: 1 + the number of v before the token in
 *               (logit descending, index ascending) order.
 *  entropy      [R] out or NULL: -sum p log p, in nats.
 *  top_ids, top_logprobs  [R, top_k] out: the first top_k tokens in that
 *               order and log p of each (-inf where the logit is, or where
 *               log p is below what a float holds).
 *  A skipped row gets logprob 0, entropy 0, rank -1, top_ids -1 and
 *  top_logprobs -inf.  A token outside [0, V) other than -1
 *  (SPEC_DEVERR_TOKEN), a NaN or +inf in the row or no finite entry in it
 *  (SPEC_DEVERR_NONFINITE) gives the same, with logprob -inf.  With tokens
 *  NULL, logprob (if given) is 0 and rank -1 in every row.
 *  The waits inside are bounded (2 s): a row whose wait runs out is refused
 *  in the same way, with SPEC_DEVERR_TIMEOUT and SPEC_DEVERR_NONFINITE.
 *  R == 0 is valid and enqueues only the clearing of dev_error.
 *  Limits: V <= 524,280, top_k <= 128, T >= 2^-126 (SPEC_ERR_UNSUPPORTED
 *  otherwise).
 */
spec_status spec_token_logprobs(const void* logits, spec_dtype dtype, int R, int V, int64_t row_stride,
                                const int32_t* tokens, float temperature, int top_k, float* logprob, int32_t* rank,
                                float* entropy, int32_t* top_ids, float* top_logprobs, int32_t* dev_error,
                                spec_stream_t stream);

/*
 * Distillation of a draft model from a teacher's top-K log probabilities:
 * the loss of every row and, in the same call, its gradient.
 *
 *  student          R rows of V logits, as in spec_token_logprobs.
 *  teacher_ids      [R, K] int32: distinct tokens; -1 marks an absent entry.
 *  teacher_logprobs [R, K] float: l_j (any constant may be added under
 *                   SPEC_TAIL_RENORM); -inf counts as probability zero.
 *  weights          [R] or NULL (=> 1): a row of weight 0 is not read and
 *                   has loss 0 and gradient 0.
 *  temperature      T > 0 of the student: q = softmax(row / T).
 *  With t_j = exp(l_j), M = sum t_j and q_T = sum of q over the tokens not
 *  listed:
 *    SPEC_TAIL_RENORM: t_j <- t_j / M,  t_T = 0   (M = 0: loss 0, gradient 0)
 *    SPEC_TAIL_BUCKET: t_T = max(0, 1 - M), and 0 where q_T = 0 and 1 - M
 *                      <= 2^-16 (the rounding of the l_j)
 *    loss = sum_j t_j (log t_j - log q_j) + t_T (log t_T - log q_T), terms
 *    with t = 0 being 0, and q_T summed over the tail itself, never as
 *    1 - sum q_j.
 *  loss       [R] out, not multiplied by the weight.
 *  row_stats  [R, 8] out or NULL: what spec_distill_topk_backward needs.
 *  grad       R rows of V elements of student's type, grad_stride apart, or
 *             NULL: d(sum_r weights[r] loss[r]) / d student,
 *               listed tokens   w (S q_j - t_j) / T
 *               other tokens    w (S q_T - t_T) / T * q_v / q_T
 *             with S = sum t_j + t_T; may be student's own buffer.
 *  An id outside [0, V) other than -1, or one listed twice
 *  (SPEC_DEVERR_TOKEN), a NaN or +inf in the row or no finite entry in it,
 *  a NaN or +inf teacher value of a listed token, or under
 *  SPEC_TAIL_BUCKET an M past the range of 32 bits (SPEC_DEVERR_NONFINITE):
 *  the row has loss 0 and gradient 0.  The waits inside are bounded (2 s):
 *  after one that ran out (SPEC_DEVERR_TIMEOUT and SPEC_DEVERR_NONFINITE)
 *  the row that it was for, and those that the same CTAs would take after
 *  it, may be refused in part only: the losses and gradients of such a call
 *  are not to be used.  A listed token of t_j > 0 whose student
 *  logit is -inf makes the loss +inf; the gradient stays finite.
 *  R == 0 is valid.  Limits: 1 <= K <= 128, V <= 524,280, T >= 2^-126.
 */
spec_status spec_distill_topk(const void* student, spec_dtype dtype, int R, int V, int64_t row_stride,
                              const int32_t* teacher_ids, const float* teacher_logprobs, int K, const float* weights,
                              float temperature, spec_tail_mode tail, float* loss, float* row_stats, void* grad,
                              int64_t grad_stride, int32_t* dev_error, spec_stream_t stream);

/*
 * The gradient of spec_distill_topk for upstream gradients that are known
 * only after the losses: grad = grad_loss[r] * d loss[r] / d student, from
 * the row_stats that call wrote for the same student, teacher_ids,
 * teacher_logprobs, temperature and tail.  grad_loss [R] or NULL (=> 1); a
 * row with grad_loss 0, or one the first call skipped or refused, has
 * gradient 0 and is not read.  grad may be student's own buffer.
 */
spec_status spec_distill_topk_backward(const void* student, spec_dtype dtype, int R, int V, int64_t row_stride,
                                       const int32_t* teacher_ids, const float* teacher_logprobs, int K,
                                       const float* row_stats, const float* grad_loss, float temperature, void* grad,
                                       int64_t grad_stride, spec_stream_t stream);

/*
 * The cache slots of the next step, from the lengths of the last one: the
 * accepted tokens of a verification become part of every request's
 * sequence, requests that need them get cache blocks from a free list, and
 * every new token gets its slot.
 *
 *  seq_lens      [B] tokens of each request in the cache before the last
 *                step; accepted_len [B] a_b of that step (spec_verify_linear)
 *                or NULL: len_b = seq_lens[b] + a_b + 1 (NULL: seq_lens[b]).
 *                The last step fed its last token and the k drafts, so a_b
 *                accepted drafts leave a_b + 1 valid entries.  a_b = -1
 *                keeps the length.
 *  new_tokens    [B] n_b >= 0: tokens that the next step feeds.
 *  block_table   [B, max_blocks], rows table_stride apart, in/out: block j
 *                of request b holds its positions j * page_size ...; only
 *                the entries held[b] .. out_held[b] - 1 are written.
 *  held          [B] blocks each request has.
 *  free_blocks   the free list, a stack of *free_count <= free_capacity
 *                entries; read only.
 *  Request b needs max(held, ceil((len_b + n_b) / page_size)) blocks.  In
 *  request order, each takes what it lacks from the end of the free list:
 *  it is served iff all that it and the requests before it lack fits in
 *  *free_count.
 *  out_seq_lens [B] len_b, out_held [B], out_free_count [1]: the state for
 *  the next call; distinct from the input buffers.
 *  cu_tokens [B+1]: cu_tokens[0] = 0, cu_tokens[b+1] = cu_tokens[b] + n_b.
 *  slots     [max_tokens] int64: token i of request b is at
 *            slots[cu_tokens[b] + i] = block * page_size + offset of
 *            position len_b + i; positions [max_tokens] int32 that position
 *            (NULL: not written).  Entries past cu_tokens[B] get slot -1 and
 *            position 0.
 *  A request that is not served, or needs more than max_blocks blocks
 *  (SPEC_DEVERR_CAPACITY; it then lacks nothing in the rule above), keeps its
 *  blocks and its new tokens get slot -1.  seq_lens, held or new_tokens
 *  negative, accepted_len below -1, held above max_blocks, len_b above
 *  held * page_size or len_b + n_b above 2^31 - 1 (SPEC_DEVERR_LENGTH): the request keeps seq_lens[b] and
 *  held[b] and its new tokens (negative: none) get slot -1 and position 0.
 *  More than max_tokens new tokens set SPEC_DEVERR_LENGTH too; those past the
 *  end are not written.  A *free_count outside 0 .. free_capacity sets it
 *  and counts as 0.
 *  Limits: 1 <= B <= 16384, B * max_blocks < 2^31 (SPEC_ERR_UNSUPPORTED
 *  above), the sum of new_tokens below 2^31.
 */
spec_status spec_advance_blocks(const int32_t* seq_lens, const int32_t* accepted_len, const int32_t* new_tokens,
                                int B, int page_size, int32_t* block_table, int max_blocks, int64_t table_stride,
                                const int32_t* held, const int32_t* free_blocks, int free_capacity,
                                const int32_t* free_count, int32_t* out_seq_lens, int32_t* out_held, int32_t* out_free_count,
                                int32_t* cu_tokens, int64_t* slots, int32_t* positions, int max_tokens,
                                int32_t* dev_error, spec_stream_t stream);

/*
 * A paged cache of keys or of values: entry `place` of block j, head h,
 * begins at base + j * block_stride + place * entry_stride + h * head_stride
 * (in elements; its dim elements are contiguous), so that blocks may hold
 * [entry, head, dim] or [head, entry, dim], and keys and values may lie in one
 * buffer.  Position t of request b is entry t % page_size of block
 * block_table[b, t / page_size]; slot s is entry s % page_size of block
 * s / page_size, as spec_advance_blocks hands them out.
 */
typedef struct {
    int32_t blocks, page_size, heads, dim;
    int64_t block_stride, entry_stride, head_stride;
} spec_cache_layout;

/*
 * New tokens on their way from a model's projections into attention: heads of
 * queries and keys normalised (optional) and turned by their position, keys and
 * values stored in the tokens' cache slots.
 *
 *  q, k, v      [T, heads, dim], token t's head h at t * *_token_stride +
 *               h * *_head_stride elements (slices of one projection output
 *               count).  q NULL: only keys and values.  bf16 or fp16.
 *  q_norm, k_norm [dim] of the same type, or NULL (both or neither; k_norm
 *               alone when q is NULL): x <- x / sqrt(mean(x^2) + eps) * norm,
 *               over the head's dim elements, in 32 bits.
 *  positions    [T] int32; NULL only with rot_dim 0.
 *  inv_freq     [rot_dim / 2] fp32: pair i turns by positions[t] *
 *               inv_freq[i], (x, y) <- (x cos - y sin, y cos + x sin).  Pair i
 *               is elements (i, i + rot_dim / 2) of a head, or with
 *               `interleaved` (2i, 2i + 1); elements from rot_dim on stay.
 *               The angle is taken modulo a turn in 64-bit fixed point and
 *               rounded to 32 bits there: to 2^-25.9 turns (1e-7 radians) at
 *               any position.  In a tree, a node's position is its request's
 *               length plus its depth.
 *  slots        [T] int64 cache slots; a negative one stores nothing (its
 *               queries are still turned).  Slots are distinct: an entry named
 *               twice holds either token's values, per 8 bytes.
 *  out_q        [T, q_heads, dim] out, contiguous; may be q itself when that
 *               is contiguous.
 *  k_cache, v_cache  out: caches of one layout (heads = the kv heads).
 *  A slot of blocks * page_size or more sets SPEC_DEVERR_CAPACITY and stores
 *  nothing.  Norm, turn and rounding to the type happen once, in 32 bits.
 *  T == 0 is valid.  Limits (SPEC_ERR_UNSUPPORTED otherwise): dim a multiple
 *  of 8 up to 256, rot_dim a multiple of 8 up to dim, pointers and strides
 *  multiples of 8 bytes.
 */
spec_status spec_append_kv(const void* q, const void* k, const void* v, spec_dtype dtype, int T, int q_heads,
                           int64_t q_token_stride, int64_t q_head_stride, int64_t k_token_stride,
                           int64_t k_head_stride, int64_t v_token_stride, int64_t v_head_stride, const void* q_norm,
                           const void* k_norm, float eps, const int32_t* positions, const float* inv_freq, int rot_dim,
                           int interleaved, const int64_t* slots, void* out_q, void* k_cache, void* v_cache,
                           const spec_cache_layout* layout, int32_t* dev_error, spec_stream_t stream);

/*
 * Attention of drafted nodes over a paged cache.  Request b has seq_lens[b]
 * entries in the cache (its sequence) and behind them the entries of this
 * step's nodes, node i at position seq_lens[b] + i, all stored before the call.
 * Node n's queries see the sequence and the nodes on n's path from the root, n
 * itself included:
 *   out[b, n, h] = sum_t softmax_t(scale * q[b, n, h] . k[t, h']) v[t, h'],
 * h' = h / (q_heads / kv heads).  A linear draft is the chain (parent NULL);
 * N = 1 is a decoding step.
 *
 *  q            [B, N, q_heads, dim], strides of request, node and head in
 *               elements, heads contiguous; bf16 or fp16, as the caches.
 *  k_cache, v_cache  caches of one layout; q_heads a multiple of its heads.
 *  block_table  [B, max_blocks] int32, rows table_stride apart, as
 *               spec_advance_blocks keeps it; only the entries of positions
 *               below seq_lens[b] + n_b are read.
 *  seq_lens     [B] int32 >= 0: out_seq_lens of spec_advance_blocks.
 *  parent       NULL (node i's parent is i - 1), [N] with parent_stride 0, or
 *               [B, N] with parent_stride >= N: as in the tree verification.
 *  n_nodes      [B] int32 in 0 .. N, or NULL (N each).  Rows from n_b on have
 *               no influence and are not written.
 *  scale        > 0; scale * log2(e) finite.
 *  out          [B, N, q_heads, dim] out, contiguous; must not overlap the
 *               inputs.
 *  Entries that a node does not see have no influence on it, whatever they
 *  hold.  An entry of this step's nodes whose values are not all finite makes
 *  the whole head row of each node that sees it NaN.  Scores, softmax sums and
 *  outputs are held in 32 bits; the weights of the products with the values are
 *  rounded to the type, half a step of it each.  In fp16 small weights are off
 *  by more, by 2^-25 of the row's largest: weights of 2^-20 of it, of a long
 *  tail beside one dominant entry, by 2^-5 of themselves.
 *  A request with seq_lens[b] < 0, n_b outside 0 .. N or more positions than
 *  max_blocks blocks hold (SPEC_DEVERR_LENGTH), a parent array that is not a
 *  tree rooted at 0 with parent[i] < i (SPEC_DEVERR_PARENT), or a block outside
 *  the cache (SPEC_DEVERR_CAPACITY) gets rows of zeros (all N rows when n_b is
 *  out of range).  The waits inside are bounded (2 s): after one that ran out
 *  (SPEC_DEVERR_TIMEOUT) the call's results are not to be used.
 *  The same call gives the same bits every time; a request's floats may differ
 *  in their last bits with the other requests of its batch.
 *  workspace    spec_tree_attention_workspace() bytes on 256, for this call
 *               alone until it has completed; needs no initial value.
 *  Limits (SPEC_ERR_UNSUPPORTED): dim a multiple of 8 up to 128, N <= 1024,
 *  q_heads / heads <= 128, B <= 65,535, strides of the caches multiples of 16 bytes, caches on 16 bytes,
 *  q on 16 bytes with strides of multiples of 16 bytes.
 */
size_t spec_tree_attention_workspace(int B, int N, int q_heads, int kv_heads, int dim);
spec_status spec_tree_attention(const void* q, spec_dtype dtype, int B, int N, int q_heads, int64_t q_request_stride,
                                int64_t q_node_stride, int64_t q_head_stride, const void* k_cache, const void* v_cache,
                                const spec_cache_layout* layout, const int32_t* block_table, int max_blocks,
                                int64_t table_stride, const int32_t* seq_lens, const int32_t* parent,
                                int64_t parent_stride, const int32_t* n_nodes, float scale, void* out,
                                int32_t* dev_error, void* workspace, size_t workspace_bytes, spec_stream_t stream);

/*
 * What spec_adjust_logits does to a request's rows; every pointer is a device
 * pointer, and each group may be NULL.
 */
typedef struct {
    /* [B, history_capacity] token ids, rows history_stride apart: request b has history_lens[b] of them, the first
     * prompt_lens[b] (NULL: none) its prompt, the others its output so far, the root's token included */
    const int32_t* history;
    int64_t history_stride;
    const int32_t* history_lens;
    const int32_t* prompt_lens;
    int32_t history_capacity;
    /* token of node i, 1 <= i < R, at drafted[b * drafted_stride + i - 1]: draft_tokens [B, k] of a linear
     * verification, or node_tokens + 1 with stride N of a tree's */
    const int32_t* drafted;
    int64_t drafted_stride;
    /* as in spec_tree_attention */
    const int32_t* parent;
    int64_t parent_stride;
    const int32_t* n_nodes;
    /* [B] each */
    const float *repetition, *frequency, *presence;
    /* [B, bias_count] ids (-1: none, to fill a list up) and what is added to their logits; an id given twice gets both
     * (one id's n entries are added up in order by one thread, in n^2 steps: 0.6 ms for 300 of one id) */
    const int32_t* bias_ids;
    const float* bias_values;
    int32_t bias_count;
    /* bit v % 32 of word v / 32 of a row: token v is allowed.  Rows allowed_stride words apart, in the order of the
     * logits' rows */
    const int32_t* allowed;
    int64_t allowed_stride;
} spec_adjustments;

/*
 * Target (or draft) logits before they are verified or sampled from: penalties
 * for tokens that were said already, biases, and a grammar's mask.  Row i of
 * request b scores what follows node i, so it counts the request's history and
 * the drafted tokens on the path from the root to i:
 *   seen(v): v in the history or on the path;  c(v): times v occurs in the
 *            history from prompt_lens[b] on, and on the path
 *   y = seen ? (x > 0 ? x / repetition : x * repetition) : x
 *   y = c > 0 ? y - (frequency * c + presence) : y
 *   y = y + the sum of v's biases
 *   y = -inf where v is not allowed, whatever x is.
 * In 32 bits, rounded once; x / repetition is taken as a product with 1 /
 * repetition (off by 2^-23 of it at most) where neither leaves the range of 32
 * bits.  Where a request's penalties are 1, 0 and 0, its history and drafted
 * tokens are neither read nor checked.
 *
 *  logits, out  B * R rows of V elements, row r at r * row_stride (out:
 *               out_stride), bf16 or fp32; out may be logits itself with the
 *               same stride.  Rows from n_nodes[b] on are left as they are.
 *  A token id of the history, the path or the biases outside [0, V) (other
 *  than a bias of -1) is passed over (SPEC_DEVERR_TOKEN); history_lens[b]
 *  outside 0 .. history_capacity counts as 0, prompt_lens[b] outside
 *  0 .. history_lens[b] as the nearer end, n_nodes[b] outside 0 .. R as R
 *  (SPEC_DEVERR_LENGTH); a parent array that is not a tree (see above) makes
 *  the request's paths empty (SPEC_DEVERR_PARENT).  Infinite and NaN parameters
 *  act by the formula: a penalty on the tokens that it is for, not on others.
 *  B == 0 is valid.  Limits: V <= 524,280, R <= 1024, bias_count <= 1024,
 *  history_capacity <= 536,000,000, B <= 65,535 (SPEC_ERR_UNSUPPORTED).
 */
spec_status spec_adjust_logits(const void* logits, spec_dtype dtype, int B, int R, int V, int64_t row_stride,
                               const spec_adjustments* adjustments, void* out, int64_t out_stride,
                               int32_t* dev_error, spec_stream_t stream);

/*
 * After a tree verification: the cache entries of the accepted path move
 * together, so that the a_b + 1 valid entries that spec_advance_blocks counts on
 * are consecutive.  In every plane, the entry of node path_nodes[b, i] (position
 * seq_lens[b] + path_nodes[b, i]) moves to position seq_lens[b] + i,
 * i = 0 .. a_b.  (Entries were turned by their depth, which is i.)  Other
 * entries stay; a linear draft needs no such call.
 *
 *  planes       HOST array of n_planes device pointers, key and value caches of
 *               all layers, of one layout, none of which overlap; read before
 *               the call returns.
 *  element_size 1, 2 or 4 bytes.
 *  path_nodes   [B, W], accepted_len [B]: as the tree verification gives them,
 *               on the block_table and seq_lens of its attention.
 *  A request whose a_b is outside 0 .. W - 1, whose path is not increasing from
 *  a node >= 0 or whose positions pass its table (SPEC_DEVERR_LENGTH), or that
 *  has a block outside the cache there (SPEC_DEVERR_CAPACITY), is left as it is.
 *  Two requests must not share blocks from seq_lens[b] on.  B == 0 and
 *  n_planes == 0 are valid.  Limits: B <= 65,535, W <= 1024
 *  (SPEC_ERR_UNSUPPORTED).
 */
spec_status spec_keep_path(void* const* planes, int n_planes, int element_size, const spec_cache_layout* layout, int B,
                           int W, const int32_t* path_nodes, const int32_t* accepted_len, const int32_t* seq_lens,
                           const int32_t* block_table, int max_blocks, int64_t table_stride, int32_t* dev_error,
                           spec_stream_t stream);

/* Static, human-readable name of a status code. */
const char* spec_status_string(spec_status status);

#ifdef __cplusplus
}
#endif

#endif /* SPECVERIFY_H */
