/*
 * gdn.h -- C ABI of the GB300 (sm_103a) gated delta rule chunked-prefill library.
 *
 * The operator (Gated DeltaNet, per value head, state S in R^{K x V}):
 *
 *     S_t = exp(g_t) S_{t-1} + k_t (beta_t (v_t - exp(g_t) S_{t-1}^T k_t))^T
 *     o_t = scale * S_t^T q_t
 *
 * computed chunk-parallel with chunk size GDN_CHUNK = 64.  The entry points
 * mirror the two-level API of the flash_qla 0.1.2 README (PyPI METADATA page,
 * sections "Usage / High-level API" and "Usage / Low-level API"):
 *
 *     chunk_gated_delta_rule_fwd(q, k, v, g, beta, scale, initial_state, cu_seqlens)
 *         -> (g, A, o, h, final_state)                          == gdn_fwd
 *     chunk_gated_delta_rule_bwd(q, k, v, g, beta, A, do, dht, scale, initial_state, cu_seqlens)
 *         -> (dq, dk, dv, db, dg, dh0)                          == gdn_bwd
 *
 * General conventions (every entry point):
 *  - All tensor pointers are caller-owned DEVICE memory, row-major and
 *    contiguous, 16-byte aligned.  The library never allocates device memory,
 *    never synchronises the device or the stream, and enqueues all work on
 *    the caller's `stream`.  It keeps no state between calls: concurrent calls
 *    on different streams with different workspaces are safe.
 *  - Arguments are validated on the host before anything is enqueued; a bad
 *    argument returns a status and enqueues nothing.  A failed launch returns
 *    GDN_ERR_CUDA.  Kernels that wait on an mbarrier give up after a limit.
 *    Those of gdn_fwd and gdn_bwd and their variants then record
 *    GDN_ERR_TIMEOUT in the workspace's error word, which
 *    gdn_workspace_error() reads back.  The decoding calls and linear attention
 *    have no such word: what the wait concerns is NaN in their outputs and
 *    states, and the status of the call and of later ones stays GDN_OK.
 *  - Shapes (B = batch, T = tokens per sequence, Hq = query/key heads,
 *    Hv = value heads, N = number of sequences):
 *        q, k            [B, T, Hq, K]   io dtype
 *        v, o, do, dv    [B, T, Hv, V]   io dtype
 *        dq, dk          [B, T, Hq, K]   io dtype
 *        g, g_cum, dg    [B, T, Hv]      fp32
 *        beta, dbeta     [B, T, Hv]      fp32
 *        A               [B, T, Hv, 64]  io dtype (row r of a chunk's 64x64
 *                                        matrix stored at that chunk's token r)
 *        h               [B, NC, Hv, K, V] fp32 (NC = chunks per sequence;
 *                                        varlen: [total chunks, Hv, K, V])
 *        h0, ht, dht, dh0 [N, Hv, K, V]  fp32
 *  - Grouped value heads: Hv % Hq == 0 and value head hv reads q/k head
 *    hv / (Hv / Hq).
 *  - Varlen: cu_seqlens != NULL requires B == 1; sequence s covers tokens
 *    [cu_seqlens[s], cu_seqlens[s+1]) and has its own h0 / ht; chunks never
 *    cross a sequence boundary.
 *  - Execution paths: bf16 io with K = V = 128 runs the tensor-core kernels.
 *    bf16 io with K or V = 64 runs the same kernels on zero-padded 128-wide
 *    copies that the library makes in its workspace (exact: the padded state
 *    rows and columns stay zero) and slices the outputs back.  fp32 io runs
 *    the CUDA-core kernels.
 */
#ifndef GDN_H_
#define GDN_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define GDN_CHUNK 64

typedef struct CUstream_st *gdn_stream_t; /* == cudaStream_t; NULL = legacy default stream */

typedef enum {
    GDN_OK = 0,
    GDN_ERR_INVALID_ARG = 1, /* null / misaligned pointer, bad shape, bad enum       */
    GDN_ERR_UNSUPPORTED = 2, /* valid but not implemented (e.g. K or V not 64 / 128) */
    GDN_ERR_WORKSPACE = 3,   /* workspace too small or misaligned                    */
    GDN_ERR_CUDA = 4,        /* a CUDA launch or async call failed                   */
    GDN_ERR_TIMEOUT = 5,     /* a device-side bounded wait expired (see header)      */
    GDN_ERR_TOO_LARGE = 6    /* gdn_fwd_noalloc: problem exceeds its fixed scratch     */
} gdn_status;

typedef enum { GDN_F32 = 0, GDN_BF16 = 1 } gdn_dtype;

typedef enum {
    GDN_CP_AUTO = 0,   /* exact; when the pages' trigger fires, sequences are
                          split and joined through segment transitions (gdn_fwd) */
    GDN_CP_OFF = 1,    /* one serial scan per (sequence, value head)             */
    GDN_CP_WARMUP = 2  /* approximate: segments start from a warmup state, see
                          gdn_fwd; used only when the page's trigger rule fires   */
} gdn_cp_mode;

typedef struct {
    int64_t B, T, Hq, Hv, K, V;      /* K, V in {64, 128}; Hv % Hq == 0              */
    int64_t n_seqs;                  /* = B, or number of sequences when varlen      */
    const int32_t *cu_seqlens;       /* device [n_seqs + 1] or NULL                  */
    const int32_t *cu_seqlens_host;  /* host copy of the same offsets; required iff
                                        cu_seqlens != NULL (used for launch planning) */
    gdn_dtype io_dtype;              /* dtype of q, k, v, o, A, do, dq, dk, dv       */
    float scale;                     /* output scale; K^-0.5 is the usual choice     */
    int32_t cp_mode;                 /* gdn_cp_mode                                  */
    int32_t warmup_chunks;           /* GDN_CP_WARMUP only: chunks of warmup (6..8)  */
    int32_t out_f32;                 /* checking mode, 0 or 1; see below              */
} gdn_problem;

/*
 * out_f32 = 1 with io_dtype GDN_BF16: the same kernels, in the same order,
 * write o and A (gdn_fwd) and dq, dk, dv (gdn_bwd, gdn_bwd_saved) as fp32
 * instead of rounding them to bf16; those buffers are then fp32 tensors of
 * the shapes above.  It exposes the value each kernel holds before its final
 * rounding, so that a test can hold it to an error bound tighter than one
 * bf16 rounding.  Ignored for GDN_F32 (every output is fp32 already).  The
 * forward's saved state for gdn_bwd_saved does not depend on it.
 */

/* Bytes of device workspace gdn_fwd / gdn_bwd need for this problem (0 on a
 * bad problem).  The workspace must be 256-byte aligned. */
size_t gdn_fwd_workspace_bytes(const gdn_problem *p);
size_t gdn_bwd_workspace_bytes(const gdn_problem *p);

/*
 * Forward (the README's chunk_gated_delta_rule_fwd; the high-level
 * chunk_gated_delta_rule returns (o, final_state) of this call).
 *   in : q, k, v (io dtype), g (raw log-decay, fp32, <= 0 expected), beta
 *        (fp32), h0 (nullable: zero initial state).
 *   out: o; g_cum = chunk-local inclusive cumsum of g (the README's returned
 *        `g`); A = (I + L)^{-1} per chunk, L = strict_lower(diag(beta)
 *        (D o K K^T)), D_ri = exp(g_cum_r - g_cum_i) (nullable: not written);
 *        h = state entering every chunk (nullable); final_state (nullable).
 * GDN_CP_WARMUP (the pages' sliding-window warmup, FlashQLA news page,
 * "Technical Principles"): when the trigger fires, each segment after the
 * first starts from the state obtained by running warmup_chunks chunks from a
 * zero state; the result is then approximate: the state error at a segment
 * start is at most exp(sum of g over its warmup window) * |S|_F, S the exact
 * state at the window start.  A value head whose gate sum over some warmup
 * window is above ln(1e-4) runs unsplit (exact) in that sequence.  g_cum, A
 * and h are as in the exact path; final_state comes from the last segment.
 * GDN_CP_AUTO with the trigger on (the pages' AutoCP, news page "FlashQLA's
 * core advantages"; here without approximation): the same segments; each is
 * run from a zero state and, with v = 0, from the identity, which gives its
 * contribution h_p and transition M_p (the recurrence is linear in v and S);
 * the segment starting states S_(p+1) = M_p S_p + h_p are scanned in fp32 and
 * every segment is then run from its own.  The result equals the unsplit one
 * up to rounding.
 */
gdn_status gdn_fwd(const gdn_problem *p,
                   const void *q, const void *k, const void *v,
                   const float *g, const float *beta, const float *h0,
                   void *o, float *g_cum, void *A, float *h, float *final_state,
                   void *workspace, size_t workspace_bytes, gdn_stream_t stream);

/*
 * Backward (the README's chunk_gated_delta_rule_bwd).
 *   in : q, k, v, g_cum (the forward's returned g), beta, A (the forward's A;
 *        nullable -- the backward recomputes the inverse in fp32 from k, beta
 *        and g_cum because the stored copy is rounded to the io dtype),
 *        d_o = dL/do, dht = dL/dfinal_state (nullable: zero), h0 (nullable).
 *   out: dq, dk, dv (io dtype), dbeta, dg (fp32; dg is the gradient with
 *        respect to the RAW g given to the forward), dh0 (required iff h0 !=
 *        NULL; must be NULL otherwise).
 */
gdn_status gdn_bwd(const gdn_problem *p,
                   const void *q, const void *k, const void *v,
                   const float *g_cum, const float *beta, const void *A,
                   const void *d_o, const float *dht, const float *h0,
                   void *dq, void *dk, void *dv, float *dbeta, float *dg, float *dh0,
                   void *workspace, size_t workspace_bytes, gdn_stream_t stream);

/*
 * gdn_fwd_noalloc -- gdn_fwd for callers that cannot allocate device memory
 * (no counterpart in the FlashQLA pages; this is a deployment convenience).
 * Hosts such as inference runtimes or plugin frameworks that own every device
 * allocation, code replaying a captured CUDA graph with a frozen memory pool,
 * or plain C callers without an allocator cannot provide gdn_fwd's
 * workspace.  This call takes the workspace from a file-scope __device__
 * array of GDN_NOALLOC_SCRATCH_BYTES bytes instead; it calls no cudaMalloc,
 * cudaFree or other allocating routine.  Inputs and outputs are the caller's,
 * exactly as for gdn_fwd.
 *   - Problems with gdn_fwd_workspace_bytes(p) > GDN_NOALLOC_SCRATCH_BYTES
 *     return GDN_ERR_TOO_LARGE and enqueue nothing.
 *   - Every GPU that loads the library holds the array until process exit.
 *   - All calls share the array; it keeps the last call's contents (each call
 *     rewrites what it reads and clears its error word), so calls whose GPU
 *     work overlaps -- on different streams or host threads -- race on it and
 *     must be serialised by the caller.
 *   - The array's address belongs to the CUDA context current at the call.
 *     Outside stream capture each call looks it up afresh, so a device reset
 *     or a caller-made driver context is served with its own address.  During
 *     capture the address cached for the current context by an earlier call
 *     is used: make one call in each context before any stream capture (a
 *     capture in a context never seen before returns GDN_ERR_CUDA).
 *   - What fits: the tensor-core forward needs about 33 KB per (chunk, value
 *     head), so about 1000 chunk x value-head units fit (e.g. B = 1, T = 8192,
 *     Hv = 8: 1024 units, just over; T = 4096, Hv = 8: 512 units plus the
 *     sequence split's segment states, about 30 MB, fits).
 *     gdn_fwd_workspace_bytes(p) is the exact test.
 *   - Invalid or unsupported problems return gdn_fwd's own status.
 */
#define GDN_NOALLOC_SCRATCH_BYTES (32u << 20)
gdn_status gdn_fwd_noalloc(const gdn_problem *p,
                           const void *q, const void *k, const void *v,
                           const float *g, const float *beta, const float *h0,
                           void *o, float *g_cum, void *A, float *h, float *final_state,
                           gdn_stream_t stream);
/* The error word gdn_fwd_noalloc's last call left in the shared array of the
 * current context (synchronises `stream`): GDN_OK, or GDN_ERR_TIMEOUT when a
 * device-side bounded wait of that call expired; GDN_ERR_CUDA if the array
 * cannot be reached. */
gdn_status gdn_fwd_noalloc_error(gdn_stream_t stream);

/*
 * Backward that reuses what the forward saved instead of recomputing it (the
 * save-for-backward form of gdn_bwd; no counterpart in the pages, whose
 * backward recomputes).  The forward must have run on the same problem and
 * inputs with its h output requested; `h` is that output and `fwd_workspace`
 * that call's workspace, both unchanged since.  The backward then skips its
 * A / P preparation and its state recompute (it reads the forward's operand
 * images, gate vectors and chunk-entry states) and runs only the state-
 * gradient scan and the per-chunk gradients.  Results equal gdn_bwd's up to
 * rounding, provided the forward's states were exact (cp_mode AUTO or OFF; a
 * warm-up split forward saves its approximate states, and the gradients then
 * follow those).  Arguments otherwise as gdn_bwd; the workspace must hold
 * gdn_bwd_saved_workspace_bytes(p) bytes.  For 64-wide heads the padded
 * forward's workspace holds the 128-wide states this reads (h must still be
 * passed: it marks that the forward ran with h requested).  fp32 problems
 * run gdn_bwd (h and fwd_workspace unused;
 * the workspace must then hold gdn_bwd_workspace_bytes(p), which this query
 * returns for them).
 */
size_t gdn_bwd_saved_workspace_bytes(const gdn_problem *p);
/* 1 if gdn_bwd_saved reads the forward's h and workspace for this problem
 * (bf16 io with at least one chunk), 0 if it runs gdn_bwd instead (the forward
 * then need not produce h), -1 for an invalid problem. */
int gdn_bwd_saved_uses_saved(const gdn_problem *p);
gdn_status gdn_bwd_saved(const gdn_problem *p,
                         const void *q, const void *k, const void *v,
                         const float *g_cum, const float *beta, const void *A,
                         const void *d_o, const float *dht, const float *h0,
                         const float *h, const void *fwd_workspace,
                         size_t fwd_workspace_bytes,
                         void *dq, void *dk, void *dv, float *dbeta, float *dg,
                         float *dh0, void *workspace, size_t workspace_bytes,
                         gdn_stream_t stream);

/*
 * Sequence splitting with warmup (the "AutoCP" of the FlashQLA pages: news
 * page, "FlashQLA's core advantages"; blog post, section 1).
 * gdn_cp_trigger: 1 iff the pages' rule turns splitting on for n_seqs
 *   sequences of up to seq_len tokens and n_heads value heads
 *   (n_seqs * n_heads <= 40, or <= 56 with seq_len >= 8192).
 * gdn_cp_plan: 1 iff gdn_fwd would split this problem (cp_mode GDN_CP_AUTO
 *   or GDN_CP_WARMUP, bf16 with K = V = 128, trigger on, more than one segment);
 *   then *seg_len = L = round(sqrt(N)) chunks for N chunks of the longest
 *   sequence and *n_seg = ceil(N / L).  Returns 0 otherwise, -1 on a bad problem.
 */
int gdn_cp_trigger(int64_t n_seqs, int64_t n_heads, int64_t seq_len);
int gdn_cp_plan(const gdn_problem *p, int *seg_len, int *n_seg);

/* Reads the device error word a previous gdn_fwd / gdn_bwd left in
 * `workspace` (synchronises `stream`).  Returns GDN_OK or GDN_ERR_TIMEOUT. */
gdn_status gdn_workspace_error(const void *workspace, gdn_stream_t stream);

/* Static description of a status code. */
const char *gdn_status_str(gdn_status s);

/*
 * Kernel timing (tracing; process-wide, off by default, not for concurrent
 * use from several host threads).  While enabled, every kernel the library
 * launches is bracketed by a pair of CUDA events recorded on the caller's
 * stream.  gdn_profile_read() waits for the recorded events, writes up to
 * max_entries rows (kernel name into names + i * name_stride, at most
 * name_stride - 1 characters; launch count; summed device milliseconds) and
 * clears the record.  Returns the number of rows, or -1 on a CUDA error.
 * Events are host-side objects; no device memory is allocated.
 */
void gdn_profile_enable(int on);
int gdn_profile_read(char *names, int name_stride, int *counts, double *ms, int max_entries);

/* Library version string, e.g. "gdn-gb300 0.2 sm_103a". */
const char *gdn_version(void);

/*
 * ---- Decoding ----
 *
 * Entry points for a model that generates: the state that gdn_fwd left
 * (final_state) is kept in a pool of slots and moved token by token.  They
 * need no workspace (but for gdn_beam_search) and read no offsets on the host,
 * so they can be captured in a CUDA graph.
 *
 * What a call cannot check on the host, because the numbers are on the device,
 * is checked by the kernels and never reaches memory out of range:
 *   - a state index below 0 marks an idle row: its outputs are 0, no slot is
 *     read or written;
 *   - a state index of n_slots or more, a token index of T or more, or a
 *     parent that is not an earlier node makes the row's outputs from there on
 *     NaN and leaves its slot as it was.
 * The kernels' waits for their own copies are bounded (a second).  Where one ran
 * out, the rows that it concerns have NaN for outputs and for new states.
 * Hv is at most 16383, n_seqs * Hv at most (2^31 - 1) / 2 and, for
 * gdn_reorder_states, B at most 65535 (GDN_ERR_UNSUPPORTED otherwise); o and the
 * states begin on 16-byte boundaries.
 */
typedef struct {
    int64_t batch, token, head; /* in elements; the innermost dimension is contiguous */
} gdn_strides;

typedef struct {
    int64_t B, T, Hq, Hv, K, V;    /* K, V in {64, 128}; Hv % Hq == 0                       */
    gdn_strides q, k, v, g, beta;  /* q, k [B,T,Hq,K]; v [B,T,Hv,V]; g, beta [B,T,Hv]       */
    gdn_dtype io_dtype;            /* dtype of q, k, v, o; g and beta are fp32              */
    float scale;
    int64_t n_slots, slot_stride;  /* state: [n_slots] of [Hv,K,V] fp32, slot_stride floats
                                      apart (a multiple of 4)                               */
    const int32_t *state_indices;  /* device [n_seqs] or NULL: row n has slot n             */
    int64_t n_seqs;                /* = B, or number of sequences when varlen               */
    const int32_t *cu_seqlens;     /* device [n_seqs + 1] or NULL; requires B == 1          */
    const int32_t *token_indices;  /* device [n_seqs, n_steps] or NULL, see gdn_recurrent   */
    int64_t n_steps;
} gdn_decode_problem;

/*
 * The recurrence itself, token by token:
 *     S_t = exp(g_t) S_{t-1} + k_t (beta_t (v_t - exp(g_t) S_{t-1}^T k_t))^T,  o_t = scale S_t^T q_t
 * for every row (sequence) over its T tokens, in fp32.  It reads and writes
 * each state once; meant for few tokens (gdn_fwd takes them by the chunk) and
 * right for any number.
 *   state     [n_slots, Hv, K, V] fp32, updated in place at the row's slot.  The
 *             slots of one call must differ from each other.
 *   out_state nullable [n_seqs, Hv, K, V] fp32 contiguous: row n's new state goes
 *             there instead and `state` is only read (slots may then repeat).
 *             Must not overlap `state`.
 *   token_indices: row n runs through its tokens token_indices[n][0], [1], ... up
 *             to the first negative entry instead of 0 .. T-1: the accepted path
 *             of a drafted tree, or rows of different lengths.  Not with
 *             cu_seqlens.
 *   o         [B, T, Hv, V] contiguous, or [B, n_steps, Hv, V] with token_indices
 *             (0 past a row's end).  q and o may both be NULL: only the states
 *             move.  With cu_seqlens, rows of o outside every sequence are not
 *             written; a sequence whose offsets fall or leave 0 .. T is skipped,
 *             its rows and its slot too.
 */
gdn_status gdn_recurrent(const gdn_decode_problem *p, const void *q, const void *k, const void *v,
                         const float *g, const float *beta, float *state, float *out_state, void *o,
                         gdn_stream_t stream);

/*
 * A tree of drafted tokens over a state: node t of row n is the token that
 * follows the tokens on the path from the state down to its parent,
 *     o_t = scale S_t^T q_t,  S_t = (the recurrence's step from S_parent(t)),
 * and the state itself stays as it was.  parents [B, T] (device, contiguous):
 * an earlier node of the row, or -1 for a child of the state; below -1 the
 * node is absent, and with it what hangs under it (o = 0).  T <= GDN_TREE_MAX.
 * What is not finite in a node reaches its own outputs and those of the nodes
 * under it, none of the others (fp32 and bf16).
 * After acceptance, gdn_recurrent with token_indices = the accepted path moves
 * the state.  cu_seqlens and token_indices must be NULL.
 */
#define GDN_TREE_MAX 64
gdn_status gdn_tree(const gdn_decode_problem *p, const void *q, const void *k, const void *v,
                    const float *g, const float *beta, const int32_t *parents, const float *state, void *o,
                    gdn_stream_t stream);

/*
 * One selection of a beam search.  With lse_w the logarithm of the sum of the
 * exponentials of beam w's allowed logits, candidate (w, token) has the score
 *     scores[w] + (logits[w][token] - lse_w),
 * and a finished beam has itself, with its score, as its only candidate.  The
 * n best candidates of each of the B searches come out in descending order,
 * equal ones by the lower w * vocab + token (a finished beam counts as its
 * token 0).  A logit of -inf, one whose mask byte is 0 (whatever it holds) and
 * any candidate whose score is not above -inf are never chosen; a beam with a
 * NaN or +inf among its allowed logits has no candidates.  Where fewer than n
 * are left the score is -inf, the token -1 and the parent j % W for place j.
 * The token of a finished beam is -1.
 */
typedef struct {
    int64_t B, W, vocab, n;                 /* 1 <= W, n <= GDN_BEAM_MAX; vocab <= GDN_BEAM_VOCAB_MAX */
    int64_t logits_batch, logits_beam;      /* strides in elements; the vocabulary is contiguous */
    int64_t mask_batch, mask_beam;          /* strides in bytes, 0 to share                      */
    gdn_dtype logits_dtype;
} gdn_beam_problem;
#define GDN_BEAM_MAX 64
#define GDN_BEAM_VOCAB_MAX (1 << 20)

/* Bytes of device workspace (0 on a bad problem), 256-byte aligned. */
size_t gdn_beam_search_workspace_bytes(const gdn_beam_problem *p);
/* scores [B, W] fp32, finished [B, W] bytes (nullable), mask bytes (nullable) -> out_scores fp32, out_tokens,
 * out_parents int32, all [B, n] contiguous. */
gdn_status gdn_beam_search(const gdn_beam_problem *p, const void *logits, const float *scores,
                           const uint8_t *finished, const uint8_t *mask, float *out_scores, int32_t *out_tokens,
                           int32_t *out_parents, void *workspace, size_t workspace_bytes, gdn_stream_t stream);

/*
 * The beams' states follow a selection, in place: with slot(b, i) =
 * state_indices[b * W + i] (NULL: b * W + i), for every view at once
 *     new[slot(b, i)] = old[slot(b, parents[b * W + i])]
 * Each source is read and each moved slot is written once; nothing is staged.
 * A view is one tensor of n_slots slots of slot_bytes bytes, slot_stride bytes
 * apart.  The slots of one call must differ from each other and the views must
 * not overlap.  A negative parent leaves the slot as it is; one of W or more,
 * or one whose slot is not in the pool, fills it with 0xFF bytes (NaN).
 * Views are read on the host during the call.
 */
typedef struct {
    void *data;
    int64_t slot_stride, slot_bytes;
} gdn_state_view;
gdn_status gdn_reorder_states(const gdn_state_view *views, int64_t n_views, int64_t n_slots, int64_t B, int64_t W,
                              const int32_t *parents, const int32_t *state_indices, gdn_stream_t stream);

/*
 * gdn_linear_recurrent: the same calls for linear attention,
 *     S_t = exp(g_h) S_{t-1} + k_t v_t^T,   o_t = scale S_t^T q_t,
 * whose decay is a constant of the head: g [Hv] fp32 (NULL: 0).  p->g and
 * p->beta are not read; everything else is as for gdn_recurrent.
 */
gdn_status gdn_linear_recurrent(const gdn_decode_problem *p, const void *q, const void *k, const void *v,
                                const float *g, float *state, float *out_state, void *o, gdn_stream_t stream);

/*
 * One token for each row of logits, drawn with a given random number.  Of a
 * row's allowed logits x (mask byte not 0, not -inf), best first and equal
 * ones by the lower token, the top_k first are kept; of these, with shares
 * e^(x / temperature) / sum, the fewest whose shares reach top_p; of these
 * those with at least min_p times the best one's share.  Among what is left,
 * in the order of the vocabulary, the token is the first whose running sum of
 * shares exceeds u times their sum; the log of its own part in that sum comes
 * beside it.  temperature 0: the best token, log 0.
 *   top_k of 0 and below, or above the number of tokens: all of them.  top_p of 1 and
 *   above, min_p of 0 and below: no limit; top_p of 0 and below: the best one;
 *   min_p above 1 counts as 1, u outside [0, 1) as the nearest number in it,
 *   NaN as 0.
 *   A row without a choice -- no allowed logit, a NaN or +inf among them, a
 *   temperature below 0, of +inf or NaN, a NaN for top_p or min_p -- has the
 *   token -1 and the log -inf.
 * Parameters are given for each row (fp32 or int32 [B] on the device) or, with
 * a NULL pointer, once for all rows.  Shares are whole numbers of 2^-42 of the
 * best one's: smaller ones are never drawn, and no sum depends on an order.
 *   Up to GDN_SAMPLE_ROWS_MAX rows of up to GDN_SAMPLE_VOCAB_MAX tokens; more
 * are GDN_ERR_UNSUPPORTED.
 */
typedef struct {
    int64_t B, vocab;
    int64_t logits_row, mask_row;           /* strides in elements and bytes; mask_row 0: shared */
    gdn_dtype logits_dtype;
    const float *temperatures, *top_ps, *min_ps;
    const int32_t *top_ks;
    float temperature, top_p, min_p;
    int32_t top_k;
} gdn_sample_problem;
#define GDN_SAMPLE_VOCAB_MAX (1 << 20)
#define GDN_SAMPLE_ROWS_MAX (1 << 20)

/* u [B] fp32, mask bytes (nullable) -> tokens int32 [B], logprobs fp32 [B] (nullable). */
gdn_status gdn_sample(const gdn_sample_problem *p, const void *logits, const float *u, const uint8_t *mask,
                      int32_t *tokens, float *logprobs, gdn_stream_t stream);

/*
 * ---- Linear attention over whole sequences ----
 *
 *     S_t = exp(g_h) S_{t-1} + k_t v_t^T,   o_t = scale S_t^T q_t
 *
 * with a decay that is a constant of the head, taken by the chunk of GDN_CHUNK
 * tokens, forward and backward.  Shapes, grouped value heads and sequences are
 * those of gdn_fwd, but for
 *   g [Hv] fp32 (NULL: 0), the logarithm of the decay, <= 0 expected; it has
 *     no gradient;
 *   q, k, v, d_o with strides of their own (in elements, each row of K or V values
 *     contiguous); o, dq, dk, dv are contiguous;
 *   offsets that are read on the device alone, so that nothing is needed of
 *     them on the host: a sequence whose offsets fall or leave the T tokens counts as empty.
 *     Rows of the outputs that no sequence claims become 0.
 * Neither call synchronises or allocates; both can be captured in a graph.
 * Waits of the kernels are bounded (a second); where one ran out, the outputs
 * and the states that it concerns are NaN.
 * The sequences are split over the GPU where they are few, and joined without
 * approximation, in fp32.
 * bf16 whose pointers and strides are multiples of 16 bytes above 0: the tensor
 * cores' kernels; the rest and fp32: the CUDA cores'.  A token that is not
 * finite reaches those of its own chunk before it, and all that follow it in its
 * sequence, none of another sequence.  The gradients of k, v and h0 run from the
 * last token to the first: there it reaches those of its own chunk, counted
 * from the sequence's end, and all that are before it; dq is as o.
 */
typedef struct {
    int64_t B, T, Hq, Hv, K, V;    /* K, V in {64, 128}; Hv % Hq == 0; Hv <= 16383; B T < 2^31  */
    int64_t n_seqs;                /* = B, or number of sequences when varlen                   */
    const int32_t *cu_seqlens;     /* device [n_seqs + 1] or NULL; requires B == 1              */
    gdn_dtype io_dtype;
    float scale;
    gdn_strides q, k, v, d_o;
} gdn_linear_problem;

size_t gdn_linear_fwd_workspace_bytes(const gdn_linear_problem *p);
size_t gdn_linear_bwd_workspace_bytes(const gdn_linear_problem *p);
/* h0 (nullable), final_state (nullable) [n_seqs, Hv, K, V] fp32. */
gdn_status gdn_linear_fwd(const gdn_linear_problem *p, const void *q, const void *k, const void *v, const float *g,
                          const float *h0, void *o, float *final_state, void *workspace, size_t workspace_bytes,
                          gdn_stream_t stream);
/* From d_o and dht (nullable: 0): dq, dk, dv in the io type, each nullable where it is not wanted, and dh0
 * (nullable). */
gdn_status gdn_linear_bwd(const gdn_linear_problem *p, const void *q, const void *k, const void *v, const float *g,
                          const float *h0, const void *d_o, const float *dht, void *dq, void *dk, void *dv,
                          float *dh0, void *workspace, size_t workspace_bytes, gdn_stream_t stream);

/*
 * Test aid for the bounded device-side waits (process-wide; set it only while
 * no other thread calls the library).  Problems planned after this call use
 * wait_ns as the limit of every mbarrier wait of the forward's state-chain
 * kernel (wait_ns <= 0 restores the default of one second) and, when
 * drop_load_chunk >= 0, that kernel's producer skips the k / q / operand-image
 * load of the chunk with this index in every chain.  The consumer's wait on
 * that load then expires: the kernel records GDN_ERR_TIMEOUT in the workspace
 * error word (read by gdn_workspace_error), waits for its own copies and
 * tensor-core operations in flight, frees its tensor memory and returns, and
 * the outputs of that call are incomplete.  Linear attention's tensor-core
 * kernel skips the load of that chunk in every sequence, or segment of one,
 * that it takes; its limit stays a second, and its outputs and states are NaN
 * where there was such a chunk.  Later calls on the same stream run normally.
 * gdn_debug_set_wait(0, -1) restores the defaults.
 */
void gdn_debug_set_wait(int64_t wait_ns, int32_t drop_load_chunk);

#ifdef __cplusplus
}
#endif
#endif /* GDN_H_ */
