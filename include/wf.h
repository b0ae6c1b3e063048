/*
 * wf.h - C ABI of the GB300 (sm_103a) verify-and-route library for WhiFlash
 * token-level cross-paradigm speculative decoding.
 *
 * One speculation round of WhiFlash (WhiFlash paper, arXiv 2606.07710,
 * Sec. 3.2 "Proposed Architecture"): the target model verifies the drafted
 * candidates in parallel, decoding resumes from the last accepted token, and
 * the token-level router picks the drafter for the next round (Sec. 3.3).
 * This library covers the data-parallel arithmetic of that step once the
 * target's final hidden states exist:
 *
 *   wf_lmhead_argmax  target LM head + greedy choice at every verified row
 *   wf_verify_chain   DFlash block acceptance (longest matched prefix) + bonus
 *   wf_verify_tree    EAGLE-3 tree acceptance (deepest matched root path) + bonus
 *   wf_router_mlp     neural router f_theta and the threshold decision
 *   wf_draft_topk     EAGLE-3 draft head, top-k, draft-to-target id map
 *   wf_lmhead_draft_topk  the target and draft heads in one weight sweep
 *   wf_lmhead_logprobs  log-probabilities of given tokens under the target head,
 *                     entropy, best alternatives
 *   wf_draft_distill  the draft head's loss against a teacher's top logits
 *                     (wf_draft_distill_grad: its gradients)
 *   wf_round          all of the above as one stream-ordered round
 *   wf_catchup        KV-only catch-up of the EAGLE-3 drafter after a switch
 *   wf_paged_*        a round's rows over a paged key-value cache: keys and
 *                     values in, attention, accepted rows compacted
 *   wf_pages_*        the pages' own life: reserve (copy on write), fork, trim
 *
 * Conventions shared by every call
 * - Pointers named as device buffers must be device (or managed) memory
 *   allocated by the caller; the library allocates nothing and keeps no
 *   per-call state outside the caller's workspace.  Operands the kernels copy
 *   with the tensor-memory accelerator or bulk copies (weight matrices,
 *   hidden states, backlog rows, the key / value caches, the queries of drafted
 *   rows) must be memory of the current device: a host pointer or another
 *   GPU's memory there returns WF_ERR_INVALID_ARG.
 * - bf16 tensors are passed as raw uint16 bit patterns, row-major, densely
 *   packed (row stride = number of columns), 16-byte aligned.
 * - Every call is asynchronous on `stream`: it validates its arguments on the
 *   host, enqueues kernels and returns.  Host-detectable errors (NULL
 *   pointers, sizes, alignment, workspace too small) are returned at once and
 *   nothing is enqueued.
 * - Data errors that only the device can see (a parent index outside
 *   [-1, node), a sequence longer than WF_MAX_SEQ_NODES, a draft id with no
 *   valid target id) set a sticky error word in the workspace and turn the
 *   affected outputs into -1.  The device never traps; read the word with
 *   wf_read_device_error.  Every wait inside a kernel is bounded
 *   (wf_set_wait_timeout_ns); a wait that gives up records WF_ERR_TIMEOUT.
 * - Stream order: a call reads its per-call inputs (hidden states, drafts,
 *   parents, offsets, rows, backlog) only after everything enqueued before it
 *   on `stream` has finished.  Model state — weight matrices, biases, gains,
 *   the draft-to-target map — may be fetched as soon as a kernel of the call
 *   starts, which can be while the previous kernel on the stream is still
 *   running (programmatic dependent launch): do not have work that is still
 *   in flight on the stream write it.
 * - Workspace: caller-owned device memory of at least wf_workspace_bytes()
 *   bytes, zeroed once with wf_workspace_init() before first use.  Calls
 *   leave it zeroed where that matters, so it can be reused without
 *   re-initialisation.  Calls that share a workspace must not overlap in time
 *   (use one stream, or one workspace per stream).
 */
#ifndef WF_H
#define WF_H

#include <stddef.h>
#include <stdint.h>

#if defined(__GNUC__)
#define WF_API __attribute__((visibility("default")))
#else
#define WF_API
#endif

#ifdef __cplusplus
extern "C" {
#endif

/* Same type as cudaStream_t; NULL = the legacy default stream. */
struct CUstream_st;
typedef struct CUstream_st* wf_stream_t;

typedef enum wf_status {
    WF_OK = 0,
    WF_ERR_INVALID_ARG = 1,   /* NULL pointer, bad size or alignment; nothing enqueued */
    WF_ERR_WORKSPACE = 2,     /* workspace NULL, misaligned or below wf_workspace_bytes() */
    WF_ERR_CUDA = 3,          /* a CUDA runtime call or kernel launch failed */
    WF_ERR_UNSUPPORTED = 4,   /* device is not sm_103 (GB300) or shape outside the kernels' range */
    WF_ERR_BAD_DATA = 5,      /* device-side: malformed tree / id data (see above) */
    WF_ERR_TIMEOUT = 6        /* device-side: a bounded wait gave up */
} wf_status;

/* Longest drafted sequence (nodes, not rows) a single sequence may carry. */
#define WF_MAX_SEQ_NODES 256
/* Largest k of wf_draft_topk. */
#define WF_MAX_TOPK 16

/* Human-readable name of a status code (static storage). */
WF_API const char* wf_status_string(int status);

/* Library ABI version (major * 100 + minor). */
WF_API int wf_version(void);

/*
 * Workspace size (bytes) sufficient for every call below with at most
 * P verified rows, B sequences, hidden size d, router width m, draft
 * vocabulary Vd and top-k k (pass 0 for Vd / k when the draft head is not
 * used).
 */
WF_API size_t wf_workspace_bytes(int P, int B, int d, int m, int Vd, int k);

/* Zero a workspace (asynchronously on `stream`).  Needed once before first use. */
WF_API wf_status wf_workspace_init(void* ws, size_t ws_bytes, wf_stream_t stream);

/*
 * Copy the sticky device error word out of the workspace (synchronises
 * `stream`).  *code is a wf_status (WF_OK if none), *info a call-specific
 * detail (the offending sequence index for WF_ERR_BAD_DATA).  clear != 0
 * resets the word afterwards.
 */
WF_API wf_status wf_read_device_error(void* ws, int* code, int* info, int clear, wf_stream_t stream);

/*
 * Upper bound (ns) on any single wait inside a kernel before it gives up with
 * WF_ERR_TIMEOUT (process-wide; default 2e9 = 2 s; 0 restores the default).
 * Applies to launches made after the call.
 */
WF_API void wf_set_wait_timeout_ns(uint64_t ns);

/*
 * Diagnostic for the failure path: enqueues one kernel whose single wait (an
 * mbarrier nothing ever arrives on, the same bounded wait the pipelined
 * kernels use) gives up after timeout_ns (<= 1e10) and records WF_ERR_TIMEOUT
 * in the workspace error word; the context stays usable.  No passage of the
 * pages corresponds to it.
 */
WF_API wf_status wf_probe_bounded_wait(uint64_t timeout_ns, void* ws, size_t ws_bytes, wf_stream_t stream);

/*
 * Target LM head fused with the greedy choice (WhiFlash paper Sec. 3.3.1:
 * under greedy decoding the target's next token at a verified position is
 * the argmax of its next-token distribution; Sec. 4 "Evaluation": greedy
 * decoding; vocabulary 151,936 and hidden size 2560 for Qwen3-4B per the
 * Qwen3-4B-EAGLE3 card, "Technical Specifications").
 *
 *   ids[p]      = argmax_v sum_k hidden[p,k] * W[v,k]   (lowest v on a tie)
 *   maxlogit[p] = that maximum logit (fp32), optional (NULL = not written)
 *
 * hidden   device, [P, d] bf16 bits, the target's final hidden states
 * W        device, [V, d] bf16 bits, LM-head weight (out x in)
 * P        rows, 1 <= P;  d % 8 == 0, 8 <= d <= 16384;  1 <= V < 2^31
 * ids      device, [P] int32 out
 * Logits are accumulated in fp32 on the tensor cores and never stored.
 */
WF_API wf_status wf_lmhead_argmax(const uint16_t* hidden, const uint16_t* W, int P, int d, int V,
                           int32_t* ids, float* maxlogit, void* ws, size_t ws_bytes,
                           wf_stream_t stream);

/*
 * wf_lmhead_argmax without a workspace: same inputs, outputs and result as
 * wf_lmhead_argmax, but the scratch lives in a fixed array inside the
 * library, for callers that cannot allocate device memory (a plug-in that a
 * host engine calls with only its input and output buffers, or a decode loop
 * that may not call cudaMalloc because it synchronises the device).  The
 * pages have no counterpart to this entry point; it exists for those callers.
 *
 * Limits: P <= WF_NOALLOC_MAX_ROWS (else WF_ERR_INVALID_ARG, nothing
 * enqueued).  Every loaded GPU holds the array (about 128 KB) until the
 * process exits.  All calls on a device share it: calls that overlap on the
 * GPU race, so serialise them (one stream).  The first call on a device looks
 * up the array's address and should come before any stream capture.  It
 * allocates nothing; each call clears the part of the array it uses,
 * including the array's error word: read a call's device-side status with
 * wf_noalloc_read_device_error before the next call on that device.
 */
#define WF_NOALLOC_MAX_ROWS 16384
WF_API wf_status wf_lmhead_argmax_noalloc(const uint16_t* hidden, const uint16_t* W, int P, int d, int V,
                                          int32_t* ids, float* maxlogit, wf_stream_t stream);

/*
 * The device-side status left by the last wf_lmhead_argmax_noalloc call on the
 * current device (0, or WF_ERR_TIMEOUT if one of its bounded waits gave up;
 * *info as in wf_read_device_error).  Synchronises `stream` first; clear != 0
 * resets the word.  Like the entry point above, this has no counterpart on the
 * pages.
 */
WF_API wf_status wf_noalloc_read_device_error(int* code, int* info, int clear, wf_stream_t stream);

/*
 * Runtime-informed router, WhiFlash-Entropy (paper Sec. 3.3.1): at each
 * selected row the entropy of the target's next-token distribution,
 *   H[b]     = - sum_v p_v log p_v,  p = softmax(<hidden[row_b], W_v>) (natural log)
 *   route[b] = 1 (autoregressive drafter) if H[b] > tau, else 0 (diffusion drafter)
 * computed in the same weight sweep as an LM-head argmax (the logits stay in
 * TMEM), with fp32 online softmax statistics.
 *
 * hidden device [P, d] bf16 bits; rows device [B] int32 rows of hidden, or
 * NULL for rows 0 .. B-1 (then B <= P); 1 <= B <= 256; W as for
 * wf_lmhead_argmax.  H device [B] fp32; route device [B] int32 or NULL.  A
 * row outside [0, P) sets WF_ERR_BAD_DATA and writes NaN / -1 for it.
 */
WF_API wf_status wf_lmhead_entropy(const uint16_t* hidden, int P, int d, const int32_t* rows, int B,
                                   const uint16_t* W, int V, float tau, float* H, int32_t* route, void* ws,
                                   size_t ws_bytes, wf_stream_t stream);

/*
 * DFlash block verification (paper Sec. 3.2: the parallel block returns to
 * the target for parallel verification; App. A: block size 16 for Qwen3).
 * Sequence b owns verified rows pos_off[b] .. pos_off[b+1]-1; row pos_off[b]
 * holds the last committed token, row pos_off[b]+1+j draft token j.  Its
 * drafts are draft[node_off[b] .. node_off[b+1]-1]; node count = rows - 1.
 *
 *   n_accept[b] = largest n with draft[j] == g[pos_off[b]+j] for all j < n
 *   last_pos[b] = pos_off[b] + n_accept[b]   (global row, feeds the router)
 *   bonus[b]    = g[last_pos[b]]              (the target's own next token)
 *   path[b*path_stride + j] = j for j < n, -1 otherwise (NULL = not written)
 * Tokens committed this round (the paper's acceptance length, Sec. 4
 * "Metrics") = n_accept + 1.
 *
 * g, draft, pos_off [B+1], node_off [B+1]: device int32.  Outputs: device int32 [B].
 */
WF_API wf_status wf_verify_chain(const int32_t* g, const int32_t* draft, const int32_t* pos_off,
                          const int32_t* node_off, int B, int path_stride, int32_t* n_accept,
                          int32_t* bonus, int32_t* last_pos, int32_t* path, void* ws,
                          size_t ws_bytes, wf_stream_t stream);

/*
 * EAGLE-3 tree verification (paper Sec. 3.2: the autoregressive drafter
 * produces a tree of candidates; App. A / Table 7: depth 8, top-k 10, 60
 * draft tokens).  Same row / node layout as wf_verify_chain; parent[] holds
 * sequence-local parent indices, -1 = the root, and parent[i] < i.
 *
 *   node i is accepted iff tok[i] == g[row of parent(i)] and parent(i) is
 *   accepted (the root always is); n_accept = depth of the deepest accepted
 *   node (lowest index on a tie; 0 if none); last_pos = its row (the root row
 *   if none); bonus = g[last_pos]; path = its ancestors' node ids from depth 1
 *   down, -1 padded, truncated at path_stride.
 * A parent outside [-1, i) or more than WF_MAX_SEQ_NODES nodes sets
 * WF_ERR_BAD_DATA (info = b) and writes -1 to that sequence's outputs.
 */
WF_API wf_status wf_verify_tree(const int32_t* g, const int32_t* tok, const int32_t* parent,
                         const int32_t* node_off, const int32_t* pos_off, int B, int path_stride,
                         int32_t* n_accept, int32_t* bonus, int32_t* last_pos, int32_t* path,
                         void* ws, size_t ws_bytes, wf_stream_t stream);

/*
 * Rows kept after a round (paper Sec. 3.2: decoding continues from the last
 * accepted token, so the committed positions - the root and the accepted
 * path - keep their target states and every other drafted row is dropped):
 *   acc_rows[b*(path_stride+1) + 0] = pos_off[b]                      (root)
 *   acc_rows[b*(path_stride+1) + j] = pos_off[b] + 1 + path[b*path_stride + j-1], j = 1..n_accept[b]
 *   acc_rows[...]                   = -1 after that
 *   acc_off[0] = 0, acc_off[b+1] = acc_off[b] + n_accept[b] + 1      (packed order)
 * and, if hidden_out != NULL, hidden_out[acc_off[b] + j] = hidden[acc_rows[b][j]]
 * (the hidden states the next drafting step conditions on, packed).
 * n_accept, path as returned by wf_verify_* / wf_round with the same
 * path_stride (n_accept[b] <= path_stride; a larger value is taken as
 * path_stride, -1 keeps no row); pos_off [B+1]; all device int32.
 * acc_rows [B, path_stride+1], acc_off [B+1] device int32 out; hidden [*, d],
 * hidden_out [sum(n_accept+1), d] device bf16 bits (both NULL to skip).
 */
WF_API wf_status wf_accepted_rows(const int32_t* n_accept, const int32_t* path, int path_stride,
                                  const int32_t* pos_off, int B, int32_t* acc_rows, int32_t* acc_off,
                                  const uint16_t* hidden, int d, uint16_t* hidden_out, wf_stream_t stream);

/*
 * EAGLE-3 draft-tree construction (the context-aware dynamic tree the
 * autoregressive drafter proposes; paper App. A / Table 7: depth 8, top-k 10,
 * 60 draft tokens).  Step s = 0 .. D-1 expands the frontier: frontier slot j
 * (only slot 0, the root, at s = 0) proposes k children, target ids
 * tid[b][s][j][c] and draft log-probabilities lp[b][s][j][c] <= 0 (e.g. the
 * top-k of wf_draft_topk, shifted by its log-sum-exp).  A child's score is
 * its parent's (0 at the root) plus its lp, summed in fp32.  The k best
 * children of a step (score desc, creation order asc) form the next
 * frontier, best first; the N best of all children created form the tree,
 * listed depth by depth (rank order within a depth), so parent[i] < i.
 *
 * tid device [B, D, k, k] int32, lp device [B, D, k, k] fp32 (entries of
 * unused slots at s = 0 are ignored); 1 <= k <= 16, 1 <= D <= 16,
 * 1 <= N <= k + (D-1) k^2.  Out (device, [B, N]): parent int32 (-1 = root),
 * token int32, score fp32 and depth int32 (score / depth may be NULL).  An lp
 * above 0 or not finite sets WF_ERR_BAD_DATA and writes -1 for that sequence.
 */
WF_API wf_status wf_build_tree(const int32_t* tid, const float* lp, int B, int D, int k, int N, int32_t* parent,
                               int32_t* token, float* score, int32_t* depth, void* ws, size_t ws_bytes,
                               wf_stream_t stream);

/*
 * Neural router and hardware-aware routing decision (paper Sec. 3.3.2; App. A
 * "Neural Router Architecture": h -> Linear(d, m) -> GELU -> dropout ->
 * Linear(m, 1), m = d/8 in the paper; route to the autoregressive drafter iff
 * the predicted gain exceeds tau_neural).  Dropout is the identity at
 * inference; GELU is the exact erf form.
 *
 *   z_j         = b1[j] + sum_k W1[j,k] * hidden[rows[b], k]
 *   delta_al[b] = b2 + sum_j w2[j] * GELU(z_j)
 *   route[b]    = 1 (EAGLE-3, autoregressive) if delta_al[b] > tau, else 0 (DFlash)
 *
 * hidden device [*, d] bf16 bits; rows device [B] int32 (row of each sequence,
 * e.g. last_pos of a verify call); W1 device [m, d] fp32 row-major; b1, w2
 * device [m] fp32; b2, tau host scalars.  d % 8 == 0; 1 <= m <= 65536.
 * Outputs: delta_al device [B] fp32, route device [B] int32 (either may be NULL).
 * fp32 arithmetic; the sum over j is taken in a fixed order (deterministic).
 */
WF_API wf_status wf_router_mlp(const uint16_t* hidden, const int32_t* rows, int B, int d, int m,
                        const float* W1, const float* b1, const float* w2, float b2, float tau,
                        float* delta_al, int32_t* route, void* ws, size_t ws_bytes,
                        wf_stream_t stream);

/*
 * EAGLE-3 draft head with top-k and the draft-to-target id map (Qwen3-4B-EAGLE3
 * card: fixed 32,000-id draft vocabulary, "top-k 10"; the draft vocabulary
 * cannot propose target ids outside it).
 *
 *   logits L[b,v] = sum_k x[b,k] * Wd[v,k], v < Vd
 *   for each b the k largest (logit desc, draft id asc):
 *   draft_ids[b,j] (optional), tids[b,j] = d2t[draft id], vals[b,j] = logit (fp32)
 *   lse[b] = log sum_v exp(L[b,v]) over all Vd draft ids (optional)
 *
 * lse turns the top-k logits into the draft distribution's log-probabilities,
 * vals[b,j] - lse[b], which EAGLE-3 tree construction accumulates along a
 * branch (WhiFlash paper App. A "Drafter Hyperparameters", Table 7: depth 8,
 * top-k 10, 60 draft tokens; see wf_build_tree).
 *
 * x device [B, d] bf16 bits (drafter hidden state); Wd device [Vd, d] bf16 bits;
 * d2t device [Vd] int32 absolute target ids; 1 <= k <= WF_MAX_TOPK, k <= Vd.
 * Outputs device: draft_ids / tids [B, k] int32, vals [B, k] fp32, lse [B]
 * fp32; each may be NULL, not all.  lse is fp32 (per-tile sums of e^(L - max)
 * merged in a fixed order).
 * A d2t entry < 0 sets WF_ERR_BAD_DATA (info = b) and writes -1 for that id.
 */
WF_API wf_status wf_draft_topk(const uint16_t* x, const uint16_t* Wd, const int32_t* d2t, int B, int d,
                        int Vd, int k, int32_t* draft_ids, int32_t* tids, float* vals, float* lse,
                        void* ws, size_t ws_bytes, wf_stream_t stream);

/*
 * Both heads of a round in one weight sweep: the results of wf_lmhead_argmax
 * over the P rows of hidden and of wf_draft_topk over the B rows of x (ids and
 * logits bit for bit; the log-sum-exp to fp32 rounding, its per-tile partials
 * being summed over this sweep's tiles), from one persistent launch that
 * streams Wd and W through the same pipeline (plus a small merge of the draft
 * candidates).  The pages
 * describe the two heads as separate steps (target verification, WhiFlash
 * paper Sec. 3.2; EAGLE-3 drafting, Qwen3-4B-EAGLE3 card); reading both
 * matrices in one pass is this library's scheduling, so that the smaller
 * draft matrix streams at full bandwidth instead of as a second sweep that
 * fills the GPU poorly.  No passage corresponds to the fused call itself.
 *
 * Arguments as in wf_lmhead_argmax (hidden, W, P, d, V, ids, maxlogit) and
 * wf_draft_topk (x, Wd, d2t, B, Vd, k, draft_ids, tids, vals, lse), one shared d.
 * P <= 128 and B <= 128 (one activation tile each), or P > 128 and B <= 256
 * (the paired-CTA sweep of several activation tiles, the draft rows in one
 * tile pair), else WF_ERR_UNSUPPORTED: call the two entry points.
 * Workspace: wf_workspace_bytes(P, B, d, 0, Vd, k).
 */
WF_API wf_status wf_lmhead_draft_topk(const uint16_t* hidden, const uint16_t* W, int P, int d, int V,
                               int32_t* ids, float* maxlogit, const uint16_t* x, const uint16_t* Wd,
                               const int32_t* d2t, int B, int Vd, int k, int32_t* draft_ids,
                               int32_t* tids, float* vals, float* lse, void* ws, size_t ws_bytes,
                               wf_stream_t stream);

/* Longest list of given tokens, or of a teacher's alternatives, of one row. */
#define WF_MAX_LISTED 64

/*
 * Log-probabilities under the target head: what the target gives to tokens that
 * were drafted, sampled or read, how sure it is, and its best alternatives (the
 * data that a drafter is distilled from).  The pages verify greedily and need
 * none of this; no passage corresponds to the call.  Per row p, with
 *   z_v = <hidden[p], W_v> / temperature
 *   lse[p]        = log sum_v e^(z_v)
 *   logp[p, s]    = z_(tok[p, s]) - lse[p]
 *   H[p]          = entropy of softmax(z)                       (natural log)
 *   top_ids[p, j] = the k ids of largest <hidden[p], W_v>, best first, the lower
 *                   id on a tie;  top_logp[p, j] = their z - lse[p]
 * Logits are accumulated in fp32 on the tensor cores and never stored; a given
 * token's logit has the same bits as an alternative's.  Logits and their
 * differences within a row, also divided by the temperature and times log2(e),
 * have to lie in fp32's range; what the temperature makes of them costs no digits
 * but lse's own (differences are taken first).  A row with a NaN among its logits
 * has NaN results, and a NaN is no alternative (top_ids -1).
 * A tok of -1 is a place without a token: its logp is 0.  Any other id outside
 * [0, V) sets WF_ERR_BAD_DATA (info = p) and its logp is NaN.
 * Results do not depend on timing.
 */
typedef struct wf_logprobs_args {
    const uint16_t* hidden;    /* [P, d] bf16 bits */
    const uint16_t* W;         /* [V, d] bf16 bits */
    int P, d, V;               /* 1 <= P, d % 8 == 0, 8 <= d <= 16384, 1 <= V < 2^31 - 256 */
    float temperature;         /* > 0, its reciprocal finite and > 0 */
    const int32_t* tok;        /* [P, S] or NULL */
    int S;                     /* 1 .. WF_MAX_LISTED (0 if tok is NULL) */
    int k;                     /* 0 .. WF_MAX_TOPK, at most V */
    float* logp;               /* [P, S] (with tok) */
    float* lse;                /* [P] or NULL */
    float* H;                  /* [P] or NULL */
    int32_t* top_ids;          /* [P, k] or NULL */
    float* top_logp;           /* [P, k] or NULL; with k > 0 one of the two */
} wf_logprobs_args;
/* Workspace (bytes); 0 if the shapes are out of range.  These workspaces are for
 * their own calls (with any shapes that they are large enough for). */
WF_API size_t wf_logprobs_workspace_bytes(int P, int d, int V, int S, int k);
WF_API wf_status wf_lmhead_logprobs(const wf_logprobs_args* args, void* ws, size_t ws_bytes, wf_stream_t stream);

/*
 * Distillation of the draft head (wf_draft_topk's Wd) from a teacher's top
 * logits: how far the drafter's next-token distribution is from the target's
 * decides how much of a draft is accepted.  The pages take trained drafters as
 * given; no passage corresponds to these calls.  Row n, draft ids v < Vd:
 *   z[n, v] = <x[n], Wd_v> / temperature,  q = softmax(z[n])
 *   p_j     = softmax over the row's kept alternatives of tlogit[n, j] / temperature
 *   loss[n] = sum_j p_j (log p_j - log q_(id_j))
 *   lse[n]  = log sum_v e^(z[n, v])
 * An alternative is kept if its id is not -1, has a draft id (t2d, where given)
 * and its logit is not -inf; what else the places of the others hold has no say.
 * The loss takes a row's places apart.  Where several name one draft id (as a t2d
 * that maps two target ids to it makes them) it is below KL(p || q) by what tells
 * these places apart, a constant of the teacher: the gradient is the divergence's,
 * in which their p add up.  A row without a kept alternative has loss 0 and no
 * gradient.  An id outside [0, V) (or, without t2d, [0, Vd)), or a t2d entry of Vd
 * or more, sets WF_ERR_BAD_DATA (info = n): the row's loss is NaN and it has no
 * gradient.
 * Softmax statistics and sums are fp32; z and its differences within a row have to
 * lie in fp32's range, also times log2(e).  Kept logits are rounded to fp32 one by
 * one, and so is lse: beside the row's largest, the loss read off them is off by up
 * to |z| 2^-23 a unit of p, and q in the gradients by a factor of up to
 * e^(|z| 2^-22) (|z| 10^4: 0.2 %).
 *
 * wf_draft_distill writes loss and lse and, if z is given, the z[n, v] in fp32
 * (columns from Vd, rounded up to 4, on are left as they are): 4 N Vd bytes that
 * spare the gradients a second sweep of the head.  wf_draft_distill_grad takes
 * that z and lse, the same x, Wd, teacher and temperature, and gloss[n] (the
 * derivative of what is minimised by loss[n]; NULL = 1):
 *   G[n, v] = gloss[n] / temperature (q_v - sum over j with id_j = v of p_j)
 *   dx[n]   = sum_v G[n, v] Wd_v,   dWd_v = sum_n G[n, v] x[n]
 * either output may be NULL, not both; they overlap no input.  G is rounded to
 * bf16 (up to 128 rows: to the sum of two bf16 numbers), the sums are fp32 and
 * rounded to bf16 at the end.  A row with gloss 0, or without a gradient (no kept
 * alternative, an id out of range), adds nothing as long as its x is finite.
 * Results do not depend on timing.
 */
typedef struct wf_distill_args {
    const uint16_t* x;         /* [N, d] bf16 bits, the drafter's hidden states */
    const uint16_t* Wd;        /* [Vd, d] bf16 bits */
    int N, d, Vd;              /* 1 <= N, d % 8 == 0, 8 <= d <= 16384, 1 <= Vd < 2^30 */
    const int32_t* tid;        /* [N, k] ids of the teacher's alternatives, -1 = none: target ids if t2d is given */
    const float* tlogit;       /* [N, k] their logits or log-probabilities */
    int k;                     /* 1 .. WF_MAX_LISTED */
    const int32_t* t2d;        /* [V] draft id of each target id, < 0 = none; or NULL: tid are draft ids */
    int V;                     /* (0 if t2d is NULL) */
    float temperature;         /* > 0, its reciprocal finite and > 0 */
    float* z;                  /* [N, ldz] fp32, 16-byte aligned; wf_draft_distill: or NULL */
    int64_t ldz;               /* a multiple of 4, from Vd to 2^34 */
    float* lse;                /* [N]: out of wf_draft_distill, into wf_draft_distill_grad */
    float* loss;               /* [N] (wf_draft_distill) */
    const float* gloss;        /* [N] or NULL (wf_draft_distill_grad) */
    uint16_t* dx;              /* [N, d] bf16 bits or NULL (wf_draft_distill_grad) */
    uint16_t* dWd;             /* [Vd, d] bf16 bits or NULL (wf_draft_distill_grad) */
} wf_distill_args;
/* Workspace (bytes) of both calls: 2 N Vd, and what the parts of split sums and
 * the sweep's states take; 0 if the shapes are out of range. */
WF_API size_t wf_distill_workspace_bytes(int N, int d, int Vd, int k);
WF_API wf_status wf_draft_distill(const wf_distill_args* args, void* ws, size_t ws_bytes, wf_stream_t stream);
WF_API wf_status wf_draft_distill_grad(const wf_distill_args* args, void* ws, size_t ws_bytes, wf_stream_t stream);

/*
 * One whole verify-and-route round (paper Sec. 3.2 - 3.3): LM-head argmax at
 * every verified row -> per-sequence acceptance (chain or tree by kind[b])
 * -> router on each sequence's last accepted row -> route for the next round;
 * plus, if Wd != NULL, the draft head's top-k for every sequence.  All stages
 * are stream-ordered on `stream` with no host synchronisation.  The draft
 * head shares the LM head's weight sweep (as in wf_lmhead_draft_topk) when
 * P <= 128 and B <= 128, or P > 128 and B <= 256.
 */
typedef struct wf_round_args {
    /* verified rows */
    const uint16_t* hidden;    /* [P, d] bf16 bits */
    const uint16_t* W;         /* [V, d] bf16 bits */
    int P, d, V;
    /* sequences */
    int B;
    const int32_t* pos_off;    /* [B+1] */
    const int32_t* node_off;   /* [B+1] */
    const int32_t* kind;       /* [B] 0 = DFlash chain, 1 = EAGLE-3 tree; NULL = all trees */
    const int32_t* tok;        /* [N] drafted target ids */
    const int32_t* parent;     /* [N] tree parents; ignored for chains; NULL only if kind marks all chains */
    int path_stride;           /* columns of path (0 = path not written) */
    /* router */
    int m;
    const float* W1;           /* [m, d] */
    const float* b1;           /* [m] */
    const float* w2;           /* [m] */
    float b2, tau;
    /* draft head (optional: Wd == NULL skips it) */
    const uint16_t* x;         /* [B, d] bf16 bits */
    const uint16_t* Wd;        /* [Vd, d] bf16 bits */
    const int32_t* d2t;        /* [Vd] */
    int Vd, k;
    /* outputs (device) */
    int32_t* ids;              /* [P] target argmax at every row */
    float* maxlogit;           /* [P] or NULL */
    int32_t* n_accept;         /* [B] */
    int32_t* bonus;            /* [B] */
    int32_t* last_pos;         /* [B] */
    int32_t* path;             /* [B, path_stride] or NULL */
    float* delta_al;           /* [B] */
    int32_t* route;            /* [B] */
    int32_t* draft_ids;        /* [B, k] or NULL */
    int32_t* tids;             /* [B, k] (needed if Wd != NULL) */
    float* vals;               /* [B, k] or NULL */
    /* routing policy: WF_ROUTER_NEURAL (the MLP above) or WF_ROUTER_ENTROPY
     * (WhiFlash-Entropy: route = H > tau on the target's next-token
     * distribution at the last accepted row; delta_al then receives H and
     * W1 / b1 / w2 / m are not read).  The entropy policy needs P <= 128 or
     * B <= 256. */
    int router_kind;
    float* lse;                /* [B] draft head's log-sum-exp (as in wf_draft_topk) or NULL */
} wf_round_args;

#define WF_ROUTER_NEURAL 0
#define WF_ROUTER_ENTROPY 1

WF_API wf_status wf_round(const wf_round_args* args, void* ws, size_t ws_bytes, wf_stream_t stream);

/*
 * KV-only catch-up of the autoregressive drafter (paper Sec. 3.4, "Lazy
 * Catch-up" and "KV-only Prefill"): after a switch to the EAGLE-3 drafter,
 * the tokens accepted while it was idle (its backlog) enter its KV cache in
 * one batch.  For every backlog token only the keys and values of the
 * drafter's attention layer are computed; only the final backlog token runs
 * through the attention sublayer in full, so that its state can feed the
 * next draft round.  The drafter is one Llama-style decoder layer (EAGLE3
 * card, "Technical Specifications": hidden 2560, 32 attention heads, 8 KV
 * heads; head size D = 2560 / 32 = 80).  Per backlog token j of sequence b,
 * at position pos = cache_len[b] + j:
 *   a      = u / sqrt(mean(u^2) + eps) * gamma                 (RMSNorm)
 *   Kc[b, pos] = rope(Wk a, pos),  Vc[b, pos] = Wv a            (bf16)
 * rope turns each pair (x[i], x[i + D/2]) of a head by pos * theta^(-2i/D).
 * For the final token f of each sequence (wf_catchup only):
 *   q      = rope(Wq a_f, pos_f)
 *   attn_h = softmax_t(<q_h, Kc[b, t, g]> / sqrt D) Vc[b, t, g],
 *            t < cache_len[b] + n_b, KV head g = h / (H / G)
 *   out[b] = u_f + Wo attn                                      (residual)
 * The MLP of the final token is the drafter's ordinary decode step and is not
 * part of this call.
 */
typedef struct wf_catchup_args {
    const uint16_t* u;         /* [N, din] bf16: the backlog tokens' layer inputs, sequences packed */
    const int32_t* bl_off;     /* [B+1] backlog offsets: bl_off[0] = 0, bl_off[B] = N, n_b >= 1 */
    const int32_t* cache_len;  /* [B] entries already in each sequence's caches */
    int B, N, din;             /* din % 8 == 0, 8 <= din <= 16384 */
    int H, G, D;               /* query heads, KV heads (H % G == 0, H / G <= 16), head size (D % 16 == 0, <= 128) */
    const uint16_t* gamma;     /* [din] bf16 RMSNorm gain */
    float eps, theta;          /* RMSNorm epsilon (>= 0), rotary base (> 0) */
    const uint16_t* Wq;        /* [H*D, din] bf16 (out x in) */
    const uint16_t* Wk;        /* [G*D, din] bf16 */
    const uint16_t* Wv;        /* [G*D, din] bf16 */
    const uint16_t* Wo;        /* [din, H*D] bf16 */
    uint16_t* Kc;              /* [B, cap, G*D] bf16 key cache (rotated keys), in/out */
    uint16_t* Vc;              /* [B, cap, G*D] bf16 value cache, in/out */
    int cap;                   /* cache rows per sequence; B * cap < 2^31 - 4096 */
    float* out;                /* [B, din] fp32 out (wf_catchup) */
    float* attn;               /* [B, H*D] fp32 out or NULL: the final token's attention output */
} wf_catchup_args;

/* Workspace (bytes) for wf_catchup / wf_catchup_kv with these shapes. */
WF_API size_t wf_catchup_workspace_bytes(int B, int N, int din, int H, int G, int D);

/*
 * The KV-only part alone: writes cache rows cache_len[b] .. cache_len[b] + n_b - 1
 * of every sequence and nothing else (Wq, Wo, out, attn unused).  A sequence
 * with no backlog or a backlog past `cap` sets WF_ERR_BAD_DATA (info = b)
 * and its rows past the cache are not written.
 */
WF_API wf_status wf_catchup_kv(const wf_catchup_args* args, void* ws, size_t ws_bytes, wf_stream_t stream);

/* The whole catch-up: wf_catchup_kv, then the final token's attention sublayer. */
WF_API wf_status wf_catchup(const wf_catchup_args* args, void* ws, size_t ws_bytes, wf_stream_t stream);

/* ------------------------------------------------------------------ paged cache
 * A key-value cache whose rows live in pages of page_size positions.  Position
 * t of sequence b is row t % page_size of page table[b][t / page_size], the
 * same page in every layer.  The pages describe the drafters' and the target's
 * caches as dense tensors; paging them is this library's own layout, and no
 * passage corresponds to it.  One layer of a bf16 pool under an identity table
 * is the [B, cap, G*D] cache of wf_catchup (cap = max_pages * page_size).
 *
 * A page is free when its reference count is 0.  Pages are only written
 * through sequences that hold them alone: call wf_pages_reserve for a round's
 * rows before wf_paged_append writes them.  A sequence that it could not serve
 * (added = -1) takes no part in the round: where the cache has reference
 * counts, wf_paged_append and wf_paged_compact refuse to write to a page with a
 * count above 1.
 */
#define WF_KV_BF16 0
#define WF_KV_E4M3 1   /* 8-bit values (4 exponent, 3 mantissa bits, largest 448) times an fp32 scale */
/* Most sequences of one paged cache. */
#define WF_PAGED_MAX_SEQS 4096

typedef struct wf_paged_cache {
    void* K;                   /* [layers, num_pages, page_size, G, D] bf16 bits or e4m3 bytes, 16-byte aligned */
    void* V;                   /* same */
    const float* k_scale;      /* [layers, G] fp32 > 0: key = stored value * scale (WF_KV_E4M3; NULL = 1) */
    const float* v_scale;      /* same, for the values */
    int32_t* table;            /* [B, max_pages] page of each block of positions, -1 = none */
    int32_t* ref;              /* [num_pages] sequences that hold each page (wf_pages_*; else may be NULL:
                                  no page is shared) */
    int kv_type;               /* WF_KV_BF16 or WF_KV_E4M3 */
    int layers, num_pages;     /* num_pages * page_size < 2^31 - 4096 */
    int page_size;             /* a power of two, 8 .. 1024 */
    int G, D;                  /* KV heads, head size (D % 16 == 0, 16 <= D <= 128, G * D <= 16384) */
    int B, max_pages;          /* sequences (1 .. WF_PAGED_MAX_SEQS), blocks a sequence may hold;
                                  max_pages * page_size <= 2^30 */
} wf_paged_cache;

/*
 * Workspace (bytes) of the wf_paged_* and wf_pages_* calls on a cache of B
 * sequences, G KV heads of size D, with H query heads and at most max_rows
 * rows a sequence (both only matter to wf_paged_attention).  0 if the shapes
 * are out of range.  Zero it once with wf_workspace_init, and keep it for these
 * calls (of any shapes it is large enough for): the other calls' scratch lies
 * where these keep counters.
 */
WF_API size_t wf_paged_workspace_bytes(int B, int H, int G, int D, int max_rows);

/*
 * A round's new keys and values enter the cache: row pos_off[b] + i of k and v
 * becomes position cache_len[b] + i of sequence b in `layer`.
 * k, v device, P rows of [G, D] bf16 bits, k_stride / v_stride elements from
 * row to row (a multiple of 8, from G * D to 2^30: slices of one projection's
 * output are fine); pos_off [B+1], cache_len [B] device int32.  WF_KV_E4M3
 * stores x / scale, saturated to +-448 and rounded to the nearest value (ties
 * to even; NaN stays NaN).  Rows outside [pos_off[0], pos_off[B]) may be read
 * (all P have to be readable memory) and change nothing; no other position is
 * written.  A position without a page (or past
 * max_pages), or in a page that another sequence holds too, a negative length
 * or first row sets WF_ERR_BAD_DATA (info = b) and the row is dropped.
 */
WF_API wf_status wf_paged_append(const wf_paged_cache* cache, int layer, const uint16_t* k, int64_t k_stride,
                                 const uint16_t* v, int64_t v_stride, int P, const int32_t* pos_off,
                                 const int32_t* cache_len, void* ws, size_t ws_bytes, wf_stream_t stream);

/*
 * Attention of a round's rows over the paged cache (paper Sec. 3.2: all
 * candidates of a block or tree are verified by the target in one parallel
 * pass).  Sequence b's rows pos_off[b] .. pos_off[b+1]-1 are laid out as for
 * wf_verify_*: the first holds the last committed token, row 1 + i drafted
 * node i.  Their keys and values are positions cache_len[b] + row of the cache
 * (wf_paged_append).  Row i sees every position below cache_len[b], itself,
 * and in a chain all rows before it, in a tree the first row and its
 * ancestors.  A single new token is a sequence of one row; a sequence may have
 * no row.  Per head h, g = h / (H / G):
 *   s_t    = scale <q[row, h], key_t[g]>,  t the positions the row sees
 *   out[row, h] = sum_t softmax(s)_t value_t[g]                      (bf16)
 *   lse[row, h] = log sum_t e^(s_t)                                  (fp32, natural log)
 * Scores, also times log2(e), have to lie in fp32's range; one of -inf is a
 * weight of 0.
 * A masked position never reaches a row, whatever it holds, nor does one from
 * cache_len[b] + rows on (they may be read, to the end of their page).  A row's
 * bits depend on its own sequence and on how the batch's lengths split it, not
 * on other rows' queries or on what ran before.  fp32 softmax statistics and sums; the
 * probabilities enter the product with V in the 16-bit type of the matrix
 * instruction, fp16 for WF_KV_E4M3, else bf16: rounded to one such number, for
 * max_rows = 1 over bf16 to the sum of two.  The result does not depend
 * on timing (splits of a long cache are joined in order).
 * A sequence with a parent outside [-1, i), more than max_rows rows, a
 * negative length, or a position without a page sets WF_ERR_BAD_DATA
 * (info = b) and its rows are NaN; rows outside [pos_off[0], pos_off[B]) are
 * left as they are.
 */
typedef struct wf_paged_attn_args {
    const uint16_t* q;         /* P rows of [H, D] bf16 bits, 16-byte aligned */
    int64_t q_stride;          /* elements from row to row: a multiple of 8, from H * D to 2^30 */
    int P, H;                  /* rows; query heads (H % G == 0, H / G <= 128, H * D <= 65536) */
    const int32_t* pos_off;    /* [B+1] */
    const int32_t* cache_len;  /* [B] positions before this round's rows */
    const int32_t* node_off;   /* [B+1] as for wf_verify_tree, or NULL: every sequence is a chain */
    const int32_t* kind;       /* [B] 0 = chain, 1 = tree; NULL = all trees (all chains if parent is NULL) */
    const int32_t* parent;     /* [N] sequence-local parents, or NULL: every sequence is a chain */
    int max_rows;              /* most rows of a sequence, 1 .. WF_MAX_SEQ_NODES + 1 */
    int layer;
    float scale;               /* > 0, and finite times log2(e): at most 2.35e38; e.g. 1 / sqrt(D) */
    uint16_t* out;             /* [P, H, D] bf16 bits */
    float* lse;                /* [P, H] or NULL */
} wf_paged_attn_args;
WF_API wf_status wf_paged_attention(const wf_paged_cache* cache, const wf_paged_attn_args* args, void* ws,
                                    size_t ws_bytes, wf_stream_t stream);

/*
 * Keep the committed rows of a round (paper Sec. 3.2: decoding continues from
 * the last accepted token): in every layer the accepted path's keys and values
 * move up behind the first row,
 *   position cache_len[b] + 1 + j  <-  cache_len[b] + 1 + path[b*path_stride + j],  j < n_accept[b]
 *   new_len[b] = cache_len[b] + n_accept[b] + 1
 * n_accept, path as returned by wf_verify_* / wf_round with the same
 * path_stride (0 .. WF_MAX_SEQ_NODES; an n_accept past it is taken as
 * path_stride; -1 keeps no row: new_len = cache_len).  new_len [B] device
 * int32 out, may be cache_len itself.  A path that does not increase, or a
 * first row or path row (read or written) without a page, or a row to move into
 * a page that another sequence holds too, sets WF_ERR_BAD_DATA (info = b),
 * moves nothing and writes new_len[b] = -1.
 */
WF_API wf_status wf_paged_compact(const wf_paged_cache* cache, const int32_t* n_accept, const int32_t* path,
                                  int path_stride, const int32_t* cache_len, int32_t* new_len, void* ws,
                                  size_t ws_bytes, wf_stream_t stream);

/*
 * Room for a round's rows: after the call positions cache_len[b] ..
 * cache_len[b] + (pos_off[b+1] - pos_off[b]) - 1 of every sequence lie in
 * pages that it holds alone.  In the order of the sequences (and of the blocks
 * within one), a block without a page takes the lowest-numbered free page, and
 * so does a block whose page another sequence holds too (copy on write: the
 * old page's count drops by one, and if it holds positions below cache_len[b]
 * its contents are copied, in every layer); the last holder keeps the page.
 * added [B] device int32 out (or NULL): pages taken.  If the free pages do not
 * suffice, the first sequence that does not fit and all after it get none:
 * added = -1, their blocks stay as they were.  Negative or too long lengths,
 * negative row counts and page ids out of range set WF_ERR_BAD_DATA
 * (info = b), added = -1, and leave that sequence as it was.
 */
WF_API wf_status wf_pages_reserve(const wf_paged_cache* cache, const int32_t* pos_off, const int32_t* cache_len,
                                  int32_t* added, void* ws, size_t ws_bytes, wf_stream_t stream);

/*
 * Sequence dst[i] becomes a copy of sequence src[i] (i < n) that shares its
 * pages: table entries of the blocks below cache_len[src], their counts, and
 * cache_len[dst] = cache_len[src] (in place).  No page is copied; the first
 * write to a shared one does that (wf_pages_reserve).  Refused with
 * WF_ERR_BAD_DATA (info = i), leaving both as they were: an index outside
 * [0, B), a dst that still holds a page, that is listed twice, or that is also
 * a src, a length without its pages.
 */
WF_API wf_status wf_pages_fork(const wf_paged_cache* cache, const int32_t* src, const int32_t* dst, int n,
                               int32_t* cache_len, void* ws, size_t ws_bytes, wf_stream_t stream);

/*
 * Give back the pages past each sequence's length: entries from
 * ceil(cache_len[b] / page_size) on drop one reference and become -1 (a length
 * of 0 frees the sequence).  A negative length (WF_ERR_BAD_DATA, info = b)
 * leaves the sequence as it was; a page id out of range or without a
 * reference sets the same error and the entry becomes -1.
 */
WF_API wf_status wf_pages_trim(const wf_paged_cache* cache, const int32_t* cache_len, void* ws, size_t ws_bytes,
                               wf_stream_t stream);

#ifdef __cplusplus
}
#endif
#endif /* WF_H */
