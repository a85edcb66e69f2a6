/*
 * libspecverify: the verification sampler of speculative decoding on one
 * NVIDIA GB300 (sm_103a).
 *
 * What the library computes (page title, section):
 *   "Decodificación Especulativa y EAGLE" (Phase 10 - Lesson 25),
 *     section "El Concepto": the target scores K+1 positions in one pass; the
 *     drafted tokens are accepted or rejected left to right; a rejection
 *     draws a replacement and stops; if every draft is accepted a bonus token
 *     is drawn from the target at position K+1.
 *     section "La Regla de Exactitud": accept x_t iff r < p(x_t)/q(x_t) with
 *     r ~ U(0,1); otherwise draw from (p - q)+ / ||(p - q)+||_1 and stop.
 *     section "Caso codicioso": at temperature 0 accept iff argmax(p) = x_t,
 *     otherwise emit argmax(p) and stop.
 *   "Accelerating Sonar through speculation", section "Decodificación
 *     especulativa": n drafted tokens yield at most n+1 emitted tokens; the
 *     sampler's accepted lengths are what the scheduler reads back.
 *
 * Notation: request b in [0,B); n_b = draft_len[b] in [1,K]; T_b =
 * temperature[b]; p_{b,t} = softmax(target_logits[b,t,:] / T_b) for t <= n_b;
 * q_{b,t} = softmax(draft_logits[b,t,:] / T_b) for t < n_b.
 *
 * Readings fixed by this interface where the pages are silent:
 *   - uniforms[b,t] (t < n_b) drives the accept test at position t;
 *     uniforms[b,n_b] drives the bonus draw; uniforms_resample[b] drives the
 *     replacement draw at a rejected position.  One final draw per request.
 *   - The accept test is strict (u < p/q).  q(x) = 0 with p(x) > 0 accepts;
 *     p(x) = 0 rejects.
 *   - T_b = 0 selects the greedy rule on the raw target logits; the draft
 *     logits of that request are never read.  The same T_b divides target
 *     and draft logits.
 *   - argmax ties resolve to the lowest index.
 *   - Inverse CDF: the token is the smallest i with w_i > 0 and
 *     w_0 + ... + w_i > u * sum(w).  If rounding leaves none, the last i with
 *     w_i > 0.  A zero-weight token is never emitted.  A residual of exactly
 *     zero mass (possible only through rounding) falls back to drawing from p
 *     with the same uniform.
 *   - Rows t > n_b of the target and t >= n_b of the draft are never read.
 *   - out_tokens[b,:] = x_0 .. x_{j-1}, final token, then -1; accepted_len[b]
 *     = j in [0, n_b].
 *
 * Conventions for every call:
 *   - Ownership: every buffer is allocated and owned by the caller.  The
 *     library allocates nothing and keeps no state between calls besides
 *     what the caller's workspace holds.
 *   - Asynchrony: device calls only enqueue work on `stream` and never
 *     synchronise (except specv_read_device_status and
 *     spec_verify_sample_host, which say so).
 *   - Errors: problems visible on the host (null pointers, bad sizes,
 *     misalignment, a workspace that is too small) return a status before
 *     anything is enqueued.  Problems in the data (a draft length outside
 *     1..K, a token outside [0,V), a negative or non-finite temperature, a
 *     uniform outside [0,1), a sampled row without a finite maximum) are
 *     detected on the device: the request's accepted_len becomes -1, its
 *     out_tokens become -1, and a bit is set in the workspace's status word
 *     (specv_read_device_status).  Nothing traps.
 */
#ifndef SPECVERIFY_H
#define SPECVERIFY_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* Same object as cudaStream_t; NULL is the legacy default stream. */
typedef struct CUstream_st* specv_stream_t;

typedef enum specv_status {
  SPECV_OK = 0,
  SPECV_ERR_INVALID_ARG = 1,  /* null pointer, size out of range, misalignment */
  SPECV_ERR_UNSUPPORTED = 2,  /* shape beyond the documented limits           */
  SPECV_ERR_WORKSPACE = 3,    /* workspace or staging buffer too small         */
  SPECV_ERR_CUDA = 4,         /* a CUDA call failed                            */
  SPECV_ERR_BAD_INPUT = 5     /* the device flagged bad data (status word)     */
} specv_status;

typedef enum specv_dtype {
  SPECV_F32 = 0,   /* IEEE float32 logits                          */
  SPECV_BF16 = 1,  /* bfloat16 logits (raw 16-bit storage)          */
  SPECV_F16 = 2    /* IEEE half: the cache operators only           */
} specv_dtype;

/* Bits of the device status word. */
#define SPECV_DEV_BAD_DRAFT_LEN   0x01  /* draft_len[b] outside 1..K               */
#define SPECV_DEV_BAD_TOKEN       0x02  /* draft_tokens[b,t] outside [0,V), t<n_b  */
#define SPECV_DEV_BAD_TEMPERATURE 0x04  /* negative, NaN or infinite temperature   */
#define SPECV_DEV_BAD_UNIFORM     0x08  /* a value of uniforms[b,0..n_b] or
                                           uniforms_resample[b] outside [0,1), for
                                           greedy requests too                   */
#define SPECV_DEV_BAD_ROW         0x10  /* a row the request needs has no finite max */
#define SPECV_DEV_NO_DRAFT        0x20  /* T_b > 0 but draft_logits is NULL        */
#define SPECV_DEV_TIMEOUT         0x40  /* a bounded wait on a copy gave up        */
#define SPECV_DEV_BAD_TREE        0x80  /* a token tree whose parent of node i is not
                                           below i, or a node token outside [0,V) */
#define SPECV_DEV_BAD_CACHE       0x100 /* a cache length or page number out of range */
#define SPECV_DEV_BAD_PENALTY     0x200 /* a penalty that is not finite, or a
                                           repetition penalty not above 0         */
#define SPECV_DEV_BAD_POSITION    0x400 /* an axis number outside 0..axes-1       */
#define SPECV_DEV_BAD_BEAM        0x800 /* a beam number outside -1..W-1, or a
                                           beam's score that is NaN or +inf       */

/* Limits. */
#define SPECV_MAX_DRAFT 16      /* K <= 16                               */
#define SPECV_MAX_BATCH 65535   /* B <= 65535                            */
#define SPECV_MAX_NODES 64      /* nodes of a tree, rows of a request     */
#define SPECV_MAX_HEAD_DIM 128  /* cache operators: a multiple of 8 in 8..128 */
#define SPECV_MAX_BIAS 1024     /* biased tokens of a request             */
#define SPECV_MAX_BEAMS 64      /* beams of a request, before and after   */
#define SPECV_MAX_STATES 32     /* states of a reordering                 */
#define SPECV_MAX_CHUNK_REQUESTS 16384  /* requests of a chunk attention     */

/* Library version (major*10000 + minor*100 + patch). */
int specv_version(void);

/* Largest vocabulary supported for a dtype (2 MB rows, 342 chunks of 6 KB):
 * 1048576 for bf16, 524288 for f32. */
int specv_max_vocab(specv_dtype dtype);

/* Human-readable name of a status code (static string, never NULL). */
const char* specv_status_string(specv_status status);

/* Bytes of device workspace one call over B requests of up to K drafts of
 * a V-entry vocabulary needs: a header (status word, the residual and bonus
 * lists' lengths, which each launch sequence empties at its start), one
 * 32-byte draw record per request
 * (the residual and bonus lists), one 8-byte record per (row, 6 KB chunk),
 * the drafted tokens' logits, and one 32-byte record per (listed request,
 * 3 KB piece) holding the piece's residual sweep sums and total.  Batches
 * of more than 1024 requests run as consecutive launch sequences that share
 * it, so it is sized for at most 1024 requests.  Returns 0 for sizes out of
 * range. */
size_t specv_workspace_bytes(int B, int K, int V, specv_dtype dtype);

/* Zero a workspace on `stream` (cudaMemsetAsync).  Must run once before the
 * first call that uses the workspace; every call that completes leaves it
 * ready for the next (counters back at zero).  workspace must be 256-byte
 * aligned.  After a CUDA error inside a call, zero it again. */
specv_status specv_workspace_init(void* workspace, size_t workspace_bytes, specv_stream_t stream);

/*
 * The verification sampler.  All pointers are device pointers.
 *   target_logits     [B, K+1, V] of `dtype`, row-major, contiguous; the
 *                     base must be aligned to the element size (16-byte
 *                     alignment of every row enables bulk copies).
 *   draft_logits      [B, K, V] of `dtype`; may be NULL when every T_b is 0
 *                     (a request with T_b > 0 then fails with NO_DRAFT).
 *   draft_tokens      [B, K] int32, entries t < n_b in [0, V).
 *   draft_len         [B] int32 in 1..K, or NULL for "all K".
 *   temperature       [B] float32, >= 0 and finite; 0 selects greedy.
 *   uniforms          [B, K+1] float32 in [0,1).
 *   uniforms_resample [B] float32 in [0,1).
 *   accepted_len      [B] int32 output: j in [0, n_b], or -1 for bad data.
 *   out_tokens        [B, K+1] int32 output: accepted drafts, the final
 *                     token, then -1.
 *   workspace         specv_workspace_bytes(B, K, V, dtype) bytes, 256-byte aligned,
 *                     zeroed once with specv_workspace_init.  Calls that may
 *                     run concurrently need separate workspaces.
 *   stream            a stream of the current device (all buffers on it).
 * Enqueues four kernels on `stream` per 1024 requests (row statistics,
 * decisions, residual piece sums with the bonus draws, residual searches;
 * each as a programmatic dependent launch); no host synchronisation.
 */
specv_status spec_verify_sample(const void* target_logits, const void* draft_logits,
                                specv_dtype dtype, const int32_t* draft_tokens,
                                const int32_t* draft_len, const float* temperature,
                                const float* uniforms, const float* uniforms_resample,
                                int B, int K, int V, int32_t* accepted_len,
                                int32_t* out_tokens, void* workspace, size_t workspace_bytes,
                                specv_stream_t stream);

/*
 * Same as spec_verify_sample, and also writes per-row statistics for parity
 * checks: row_stats [B, K+1, 8] float32 (device), for the rows the request
 * needs (slots 6 and 7 only for the row of the final draw, t = accepted_len):
 *   0 max_i z^p_i (raw logit)    1 S_p = sum_i exp((z^p_i - max)/T)
 *   2 ln p(x_t)                  3 max_i z^q_i       4 S_q
 *   5 ln q(x_t)                  6 final-draw mass (below)
 *   7 the row's final-draw token (residual with uniforms_resample[b] at
 *     t < n_b, bonus with uniforms[b,n_b] at t = n_b; greedy: argmax)
 * Slot 6 is the normalised mass of the final draw's weights: sum_i (p_i - q_i)+
 * at a rejected position, sum_i p_i at the bonus position.  At T = 0 slot 0
 * is the row maximum and slot 7 the argmax for every row t <= n_b.  Unused
 * slots and rows are left untouched.
 */
specv_status spec_verify_sample_debug(const void* target_logits, const void* draft_logits,
                                      specv_dtype dtype, const int32_t* draft_tokens,
                                      const int32_t* draft_len, const float* temperature,
                                      const float* uniforms, const float* uniforms_resample,
                                      int B, int K, int V, int32_t* accepted_len,
                                      int32_t* out_tokens, void* workspace,
                                      size_t workspace_bytes, float* row_stats,
                                      specv_stream_t stream);

/* Copy the workspace's device status word to *status (host), then clear it.
 * Synchronises `stream`.  Returns SPECV_ERR_BAD_INPUT when the word was
 * non-zero, SPECV_OK when it was zero. */
specv_status specv_read_device_status(void* workspace, size_t workspace_bytes, int32_t* status,
                                      specv_stream_t stream);

/* Bytes of device staging spec_verify_sample_host needs (inputs and
 * outputs, each padded to 256 bytes).  with_draft = 0 when draft logits are
 * not passed. */
size_t specv_host_staging_bytes(int B, int K, int V, specv_dtype dtype, int with_draft);

/*
 * The sampler on HOST buffers: copies the inputs host->device into
 * `staging` (device, specv_host_staging_bytes bytes, 256-byte aligned),
 * runs spec_verify_sample, copies accepted_len and out_tokens back, and
 * synchronises `stream` before returning.  Of the logits only the rows the
 * kernels read cross the host link: a usable request's target rows
 * t <= draft_len[b] and, when temperature[b] > 0, its draft rows
 * t < draft_len[b].  Page-locked logits whose rows are a multiple of 16
 * bytes (16-byte-aligned bases) are gathered by one kernel that reads the
 * host memory through its device-visible address; other logits go as one
 * cudaMemcpyAsync per range of adjacent rows.  The other rows of `staging`
 * keep whatever they held and are never read.  draft_len and temperature are read on the host to decide
 * this, so they must be host-readable.  Every small input is copied whole.
 * Host buffers should be page-locked for asynchronous copies.  Same shapes
 * and readings as spec_verify_sample; draft_len and draft_logits may be NULL
 * as there.
 */
specv_status spec_verify_sample_host(const void* target_logits, const void* draft_logits,
                                     specv_dtype dtype, const int32_t* draft_tokens,
                                     const int32_t* draft_len, const float* temperature,
                                     const float* uniforms, const float* uniforms_resample,
                                     int B, int K, int V, int32_t* accepted_len,
                                     int32_t* out_tokens, void* staging, size_t staging_bytes,
                                     void* workspace, size_t workspace_bytes,
                                     specv_stream_t stream);

/* The launch shape the library picks for these sizes (diagnostics): out[0]
 * CTAs of the row-statistics kernel, out[1] vocabulary elements per chunk,
 * out[2] shared-memory copy slots per agent warp, out[3] chunks per row,
 * out[4] dynamic shared memory per CTA (bytes), out[5] threads per CTA
 * (32 per agent warp).  Queries the current device's occupancy; launches
 * nothing. */
specv_status specv_launch_plan(int B, int K, int V, specv_dtype dtype, int with_draft,
                               int32_t* out);

/* ------------------------------------------------------------------------
 * Steps around the verification (same conventions: device buffers, the
 * caller's workspace zeroed once with specv_workspace_init, asynchronous on
 * `stream`, data errors in the workspace's status word).
 * ---------------------------------------------------------------------- */

/* Bytes of workspace spec_sample_draft needs for R rows of V logits (0 for
 * sizes out of range). */
size_t specv_sample_workspace_bytes(int R, int V, specv_dtype dtype);

/*
 * The draft-side sampler ("Decodificación Especulativa y EAGLE", sections
 * "La Configuración de Dos Modelos" and "Desarrolla": the draft model
 * proposes each token by sampling softmax(z / T) of its logits):
 *   logits       [R, V] of `dtype`, one row per request.
 *   temperature  [R] float32 >= 0; 0 takes the row's argmax (lowest index).
 *   uniforms     [R] float32 in [0,1): tokens[r] is the smallest i with
 *                p_0 + ... + p_i > u * sum(p) and p_i > 0 (the same inverse
 *                CDF as the verification's final draws).
 *   tokens       [R] int32 output (-1 for a row flagged bad: temperature or
 *                uniform out of range, no finite maximum).
 *   workspace    specv_sample_workspace_bytes(R, V, dtype) bytes.
 *   row_stats    NULL, or [R, 8] float32: slot 0 the row maximum, 1 its
 *                normaliser sum exp((z - max)/T), 6 the drawn mass
 *                (sum of p, ~1), 7 the token; at T = 0 slots 0 and 7.
 * Enqueues two kernels per 1024 rows: the row statistics, then the
 * decisions of spec_verify_sample for requests with no drafts, whose bonus
 * draw (the sample) the decision kernel makes itself.
 */
specv_status spec_sample_draft(const void* logits, specv_dtype dtype, const float* temperature,
                               const float* uniforms, int R, int V, int32_t* tokens,
                               void* workspace, size_t workspace_bytes, float* row_stats,
                               specv_stream_t stream);

/*
 * Verification for a draft that proposes its top token ("Accelerating Sonar
 * through speculation", section "Objetivo-Borrador"): the distribution the
 * drafted token came from is the point mass q = 1{x}, so the rule of "La
 * Regla de Exactitud" accepts x_t iff u_t < p_t(x_t), and at the first
 * rejection j draws the replacement from (p_j - 1{x_j})+, i.e. from p_j with
 * x_j removed; every draft accepted draws the bonus from p_n.  No draft
 * logits.  Arguments, outputs, readings and errors as spec_verify_sample
 * without draft_logits (T = 0 is the greedy rule); workspace
 * specv_workspace_bytes(B, K, V, dtype); row_stats NULL or as
 * spec_verify_sample_debug (slots 3..5 unused; slot 6 at a rejected row is
 * 1 - p_j(x_j)).
 */
specv_status spec_verify_sample_onehot(const void* target_logits, specv_dtype dtype,
                                       const int32_t* draft_tokens, const int32_t* draft_len,
                                       const float* temperature, const float* uniforms,
                                       const float* uniforms_resample, int B, int K, int V,
                                       int32_t* accepted_len, int32_t* out_tokens,
                                       void* workspace, size_t workspace_bytes,
                                       float* row_stats, specv_stream_t stream);

/* Bytes of workspace spec_verify_tree_greedy needs (0 for sizes out of
 * range; N <= 64). */
size_t specv_tree_workspace_bytes(int B, int N, int V, specv_dtype dtype);

/*
 * Greedy verification of a token tree ("Decodificación Especulativa y EAGLE",
 * section "Verificación de Atención en Árvore"; "Accelerating Sonar through
 * speculation", section "EAGLE"): the target scores every node of a drafted
 * tree in one pass; node i is accepted iff its parent is accepted and the
 * target's argmax at the parent (lowest index) is node i's token; the root
 * (node 0, the last verified position) is always accepted.  The deepest
 * accepted node (lowest index among the deepest) ends the kept path.
 *   target_logits [B, N, V] of `dtype`: row i = the target's logits at node i.
 *   parents       [B, N] int32: parents[b,0] = -1, 0 <= parents[b,i] < i.
 *   tokens        [B, N] int32: node i's drafted token (tokens[b,0] unused).
 *   n_nodes       [B] int32 in 1..N: nodes >= n_nodes[b] are not read.
 *   accepted_len  [B] int32 output: the path's length (accepted drafts), or
 *                 -1 for a malformed tree (status SPECV_DEV_BAD_TREE) or bad
 *                 node count (SPECV_DEV_BAD_DRAFT_LEN).
 *   out_tokens    [B, N] int32 output: the path's tokens, then the argmax at
 *                 its last node, then -1.
 *   path_nodes    [B, N] int32 output: 0, then the path's node indices, then
 *                 -1 (the cache rows to keep).
 *   workspace     specv_tree_workspace_bytes(B, N, V, dtype) bytes.
 *   row_stats     NULL, or [B, N, 8] float32: slot 0 each node's maximum,
 *                 slot 7 its argmax.
 * The sampled (multi-branch) tree rule is not on the pages and not built.
 */
specv_status spec_verify_tree_greedy(const void* target_logits, specv_dtype dtype,
                                     const int32_t* parents, const int32_t* tokens,
                                     const int32_t* n_nodes, int B, int N, int V,
                                     int32_t* accepted_len, int32_t* out_tokens,
                                     int32_t* path_nodes, void* workspace,
                                     size_t workspace_bytes, float* row_stats,
                                     specv_stream_t stream);

/*
 * The post-accept insert ("Accelerating Sonar through speculation", sections
 * "Programación MTP para un solo token" and "Inferencia con decodificación
 * especulativa": a kernel writes the next step's tokens on the device, so
 * the host need not read the accepted lengths between steps).  For request
 * b with j = accepted_len[b] (as spec_verify_sample writes it):
 *   history[b, seq_lens[b] .. seq_lens[b] + j] = out_tokens[b, 0 .. j];
 *   seq_lens[b] += j + 1;  next_tokens[b] = out_tokens[b, j];
 *   cu_emitted[b + 1] = cu_emitted[b] + j + 1 (cu_emitted[0] = 0) and
 *   packed[cu_emitted[b] .. cu_emitted[b + 1]) = out_tokens[b, 0 .. j].
 * A request with j outside [0, K] emits nothing (status[b] = 1), one whose
 * history would pass L emits nothing (status[b] = 2); both keep their
 * history and length and get next_tokens[b] = -1.  status[b] = 0 otherwise.
 *   accepted_len [B], out_tokens [B, K+1], seq_lens [B] (in/out),
 *   history [B, L] (in/out), next_tokens [B], cu_emitted [B+1],
 *   packed [B*(K+1)] (only the first cu_emitted[B] written), status [B]:
 *   int32 device buffers.  One kernel of one CTA; no workspace.
 */
specv_status spec_insert_accepted(const int32_t* accepted_len, const int32_t* out_tokens, int B,
                                  int K, int32_t* seq_lens, int32_t* history, int L,
                                  int32_t* next_tokens, int32_t* cu_emitted, int32_t* packed,
                                  int32_t* status, specv_stream_t stream);

/* ------------------------------------------------------------------------
 * The target's pass over a drafted tree ("Decodificación Especulativa y
 * EAGLE", section "Verificación de Atención en Árvore": each token attends
 * to its ancestors; "Accelerating Sonar through speculation", section
 * "EAGLE"), around a paged key/value cache:
 *
 *   spec_append_nodes    norms, rotates and writes the nodes' keys and values
 *   spec_tree_attention  attends from the nodes to the cache and their paths
 *   spec_process_logits  penalties, biases and grammar masks for every node
 *   (the verification)   spec_verify_tree_greedy, spec_verify_sample, ...
 *   spec_keep_path       keeps the accepted path's cache rows
 *
 * Nodes.  A request has n_nodes[b] of N nodes; node 0 is the root (the last
 * verified token), parents[b,0] = -1 and 0 <= parents[b,i] < i.  parents =
 * NULL is a chain (node i's parent is node i-1): the K+1 positions of
 * spec_verify_sample, or with N = 1 plain decoding.  n_nodes = NULL: all N.
 * Node i lives in cache slot lens[b] + i and has position lens[b] + depth(i).
 *
 * Errors in the data.  These calls write status[b] (int32, device): 0, or
 * SPECV_DEV_* bits.  A flagged request's cache rows stay as they were, its
 * output rows (the n_nodes[b] of them, all N where n_nodes[b] itself is bad)
 * become 0 (spec_process_logits: -inf).  Rows at and behind n_nodes[b] are
 * left as they were.
 * ---------------------------------------------------------------------- */

/* A paged key/value cache.  Request b's slot s is row s % page_size of page
 * page_table[b, s / page_size].  Element (layer, page, row, head, d) of k is
 * at k + layer*layer_stride + page*page_stride + row*row_stride +
 * head*head_stride + d; v has the same strides.  Strides count elements, are
 * multiples of 8, 0 or more, and may pass 32 bits; k and v are 16-byte
 * aligned. */
typedef struct specv_cache {
  void* k;
  void* v;
  const int32_t* page_table; /* [B, max_pages], rows table_stride apart,
                                max_pages or more */
  const int32_t* lens;       /* [B]: verified tokens, 0 <= lens[b], and
                                lens[b] + n_nodes[b] <= max_pages*page_size */
  int64_t layer_stride, page_stride, row_stride, head_stride;
  int32_t layers; /* 1 but for spec_keep_path */
  int32_t pages;  /* pages in k and v: 0 <= page_table[b, .] < pages where used */
  int32_t page_size, max_pages, table_stride;
  int32_t heads;    /* key heads */
  int32_t head_dim; /* a multiple of 8, at most SPECV_MAX_HEAD_DIM */
  specv_dtype dtype; /* SPECV_BF16 or SPECV_F16 */
} specv_cache;

/* Rows [B, N, heads, head_dim] of the cache's dtype: element (b, i, h, d) is
 * at data + b*batch_stride + i*node_stride + h*head_stride + d.  data is
 * 16-byte aligned, strides are multiples of 8 elements, 0 or more. */
typedef struct specv_rows {
  void* data;
  int64_t batch_stride, node_stride, head_stride;
} specv_rows;

/*
 * Norms, rotation and append of the nodes' projections, one kernel:
 *   x <- x / sqrt(mean(x^2) + eps) * weight      (queries and keys, per head;
 *                                                 a NULL weight: no norm)
 *   (x_a, x_c) <- (x_a cos t - x_c sin t, x_c cos t + x_a sin t) * rope_scale,
 *       t = (lens[b] + depth(i)) * inv_freq[j], for j < rot_dim / 2 and
 *       (a, c) = (2j, 2j + 1) if interleaved, else (j, j + rot_dim / 2);
 *       elements d >= rot_dim keep their value.
 * Queries go to q_out, keys and values (these as they are) to the cache's
 * slots lens[b] + i.  In 32 bits, the angles in 64; rounded once, to nearest.
 *   q, k, v   [B, N, q_heads | heads | heads, head_dim] (specv_rows, of one
 *             projection or of three); q_out may be q itself, but no two of
 *             the buffers may overlap otherwise.
 *   q_weight, k_weight  [head_dim] of the cache's dtype, 16-byte aligned, or NULL.
 *   inv_freq  [rot_dim / 2] float32 (a long-context scaling is in it), or
 *             NULL with rot_dim = 0: no rotation.  rot_dim even, <= head_dim.
 * Two requests that share a page must not both write the same slot.
 */
specv_status spec_append_nodes(const specv_cache* cache, const specv_rows* q, const specv_rows* k,
                               const specv_rows* v, const int32_t* parents,
                               const int32_t* n_nodes, int B, int N, int q_heads,
                               const void* q_weight, const void* k_weight, float eps,
                               const float* inv_freq, int rot_dim, int interleaved,
                               float rope_scale, const specv_rows* q_out, int32_t* status,
                               specv_stream_t stream);

/* Bytes of workspace spec_tree_attention needs (0 for sizes out of range). */
size_t specv_attention_workspace_bytes(int B, int N, int q_heads, int kv_heads, int head_dim);

/*
 * Attention of the nodes over the cache:
 *   out[b,i,h] = sum_s softmax_s(scale q[b,i,h] . k[s, h / (q_heads/heads)]) v[s, ...]
 * over the slots s < lens[b] and s = lens[b] + a for a = i and its ancestors
 * (their rows in the cache already: spec_append_nodes).  No other slot counts,
 * whatever it holds.  Scores, maxima and sums in 32 bits; the weights are
 * rounded to the cache's dtype before the product with the values.
 *   q, out    [B, N, q_heads, head_dim]; q_heads a multiple of cache->heads.
 *   scale     > 0 and finite (1/sqrt(head_dim) as a rule).
 *   workspace specv_attention_workspace_bytes bytes, 256-byte aligned,
 *             whatever it holds.  Calls that may run at the same time need
 *             one each.
 * A wait inside the kernel that lasts two seconds gives up: then every request
 * of the call has SPECV_DEV_TIMEOUT in its status, and the rows hold anything.
 * Two kernels, the second as a programmatic dependent launch.
 */
specv_status spec_tree_attention(const specv_cache* cache, const specv_rows* q,
                                 const int32_t* parents, const int32_t* n_nodes, int B, int N,
                                 int q_heads, float scale, const specv_rows* out, int32_t* status,
                                 void* workspace, size_t workspace_bytes, specv_stream_t stream);

/*
 * Keeps the accepted path (spec_verify_tree_greedy's outputs) in the cache:
 * for j = 1 .. accepted_len[b], in every layer, keys and values,
 *   slot lens[b] + j <- slot lens[b] + path_nodes[b, j];
 *   new_lens[b] = lens[b] + accepted_len[b] + 1  (lens[b] for a flagged request).
 *   path_nodes   [B, N] int32: 0, then strictly increasing node numbers < N
 *                (else SPECV_DEV_BAD_TREE); entries behind accepted_len[b]
 *                are not read.
 *   accepted_len [B] int32 in 0..N-1 (else SPECV_DEV_BAD_DRAFT_LEN).
 *   new_lens     [B] int32 output, not cache->lens itself.
 * One kernel; no workspace.
 */
specv_status spec_keep_path(const specv_cache* cache, const int32_t* path_nodes,
                            const int32_t* accepted_len, int B, int N, int32_t* new_lens,
                            int32_t* status, specv_stream_t stream);

/*
 * Penalties, biases and grammar masks, before the verification or a sampler.
 * Row (b, i) of the logits is what the target says after node i; its text is
 * history[b, 0 .. seq_lens[b]) (as spec_insert_accepted keeps it; the root is
 * its last token) and then the tokens on the path from the root to node i.
 * With c = how often a token occurs in the text at or behind prompt_lens[b]:
 *   z <- z > 0 ? z / repetition[b] : z * repetition[b]  if the text has the token;
 *   z <- z - frequency[b] * c - presence[b] * (c > 0);
 *   z <- z + the token's bias (a token listed more than once: their sum, in
 *        the listed order);
 *   z <- -inf  if the token's bit of the mask is 0
 * in 32 bits, rounded once.  A row whose mask allows nothing becomes -inf.
 *   logits, out [B, R, V] of `dtype` (SPECV_F32 or SPECV_BF16), element (b, i, t)
 *             at b*batch_stride + i*row_stride + t (strides 0 or more); out
 *             may be logits itself (with its strides), else they do not
 *             overlap.
 *   tokens    parents != NULL: [B, R], node i's token (tokens[b,0] unused);
 *             parents == NULL (a chain): [B, R-1], the drafted tokens of
 *             spec_verify_sample.  NULL only where R = 1.
 *   n_rows    [B] in 1..R (a chain: draft_len + 1; a tree: n_nodes), or NULL.
 *   history   [B, L], rows history_stride apart; 0 <= prompt_lens[b] <=
 *             seq_lens[b] <= L (else SPECV_DEV_BAD_CACHE); prompt_lens NULL: 0.
 *   repetition, frequency, presence  [B] float32, or NULL: 1, 0, 0.
 *   bias_tokens, bias_values [B, num_bias] int32, float32, or NULL; a token
 *             below 0 is an empty place, one at or above V is flagged.
 *   allowed   [B, R, ceil(V/32)] int32, bit t % 32 of word t / 32, or NULL.
 * One kernel; no workspace.
 */
specv_status spec_process_logits(const void* logits, int64_t batch_stride, int64_t row_stride,
                                 specv_dtype dtype, int B, int R, int V, const int32_t* tokens,
                                 const int32_t* parents, const int32_t* n_rows,
                                 const int32_t* history, int64_t history_stride, int L,
                                 const int32_t* seq_lens, const int32_t* prompt_lens,
                                 const float* repetition, const float* frequency,
                                 const float* presence, const int32_t* bias_tokens,
                                 const float* bias_values, int num_bias, const int32_t* allowed,
                                 void* out, int64_t out_batch_stride, int64_t out_row_stride,
                                 int32_t* status, specv_stream_t stream);

/* ------------------------------------------------------------------------
 * Before the verification: the prompt's own pass over the paged cache, in
 * chunks of any length beside single tokens, and the drafting of a tree.
 *
 *   spec_append_chunk     norms, rotates and writes the tokens' keys and values
 *   spec_chunk_attention  attends from the tokens to the cache
 *   spec_select_beams     a tree's next level, or a beam search's next step
 *   spec_reorder_beams    moves the beams' states along
 *
 * Tokens.  The new tokens of all requests are packed: rows cu_tokens[b] ..
 * cu_tokens[b+1]-1 of T are request b's, none at all too.  Token i of request
 * b lives in cache slot lens[b] + i, which is also its position unless the
 * call is given others.  (specv_rows of packed rows: [T, heads, head_dim],
 * node_stride from token to token, batch_stride 0.)
 *
 * Errors in the data: as with the operators on a drafted tree, by request,
 * in status[b].  SPECV_DEV_BAD_DRAFT_LEN: cu_tokens falls or leaves 0..T (then
 * the request has no rows), or counts more than `longest` tokens;
 * SPECV_DEV_BAD_CACHE: lens[b] or a page out of range.  Rows of no request
 * are left as they were.
 * ---------------------------------------------------------------------- */

/*
 * Norms, rotation and append of the tokens' projections, one kernel: as
 * spec_append_nodes, for packed tokens, with
 *   t = positions[axis_of[j], i] * inv_freq[j]   (NULL positions: lens[b] + i's slot)
 * for pair j of the token in packed row i.
 *   q, k, v, q_out  [T, q_heads | heads | heads, head_dim]; q_out may be q
 *             itself, but no two of the buffers may overlap otherwise.
 *   cu_tokens [B+1] int32; no two requests' ranges may overlap.
 *   positions [axes, T] int32 of any sign, rows position_stride apart, or NULL
 *             (axes 0 or 1): a request's slots are its positions.
 *   axis_of   [rot_dim / 2] int32: the axis (time, height, width ...) by which a
 *             pair turns, 0 <= axis_of[j] < axes (else every request has
 *             SPECV_DEV_BAD_POSITION); NULL: axis 0, with axes = 1.
 * The other arguments as spec_append_nodes has them.  Two requests that share a
 * page must not both write the same slot.
 */
specv_status spec_append_chunk(const specv_cache* cache, const specv_rows* q, const specv_rows* k,
                               const specv_rows* v, const int32_t* cu_tokens, int B, int T,
                               int q_heads, const int32_t* positions, int64_t position_stride,
                               int axes, const int32_t* axis_of, const void* q_weight,
                               const void* k_weight, float eps, const float* inv_freq, int rot_dim,
                               int interleaved, float rope_scale, const specv_rows* q_out,
                               int32_t* status, specv_stream_t stream);

/* Bytes of workspace spec_chunk_attention needs (0 for sizes out of range). */
size_t specv_chunk_workspace_bytes(int longest, int q_heads, int kv_heads, int head_dim);

/*
 * Attention of the tokens over the cache.  The token at p = lens[b] + i sees
 * slot s of its request, below lens[b] + its number of tokens, iff
 *   s < prefix_lens[b]  or  p - window < s <= p,
 *   out[i,h] = sum_s softmax_s(y) v[s, h'],  h' = h / (q_heads/heads),
 *   y = cap tanh(scale q[i,h] . k[s,h'] / cap) - slopes[h] |p - s|.
 * No other slot counts, whatever it holds, and pages of which no token of the
 * call sees a slot need not exist.  Scores, maxima and sums in 32 bits; the
 * weights are rounded to the cache's dtype before the product with the values.
 *   q, out    [T, q_heads, head_dim]; q_heads a multiple of cache->heads.
 *   cu_tokens [B+1] int32; the tokens' own rows are in the cache already
 *             (spec_append_chunk).  B <= SPECV_MAX_CHUNK_REQUESTS.
 *   longest   no request has more tokens (T will do; the work is laid out
 *             for it); longest * q_heads / heads < 2^29.
 *   scale     > 0 (1/sqrt(head_dim) as a rule).
 *   cap       > 0 (and 2 scale / cap between 1e-30 and 1e30), or 0: scores are
 *             not capped.
 *   window    >= 1, or 0: no limit.
 *   prefix_lens [B] int32 >= 0 (else SPECV_DEV_BAD_CACHE), or NULL: 0.  The
 *             part of it that lens[b] and the tokens do not reach is not there.
 *   slopes    [q_heads] float32, or NULL: 0.
 *   workspace specv_chunk_workspace_bytes bytes, 256-byte aligned, whatever
 *             it holds.  Calls that may run at the same time need one each.
 * A wait inside the kernel that lasts two seconds gives up: then every request
 * of the call has SPECV_DEV_TIMEOUT in its status, and the rows hold anything.
 * Two kernels, the second as a programmatic dependent launch; one where longest is 1
 * and there is room for few slots.
 */
specv_status spec_chunk_attention(const specv_cache* cache, const specv_rows* q,
                                  const int32_t* cu_tokens, int B, int T, int longest, int q_heads,
                                  float scale, float cap, int window, const int32_t* prefix_lens,
                                  const float* slopes, const specv_rows* out, int32_t* status,
                                  void* workspace, size_t workspace_bytes, specv_stream_t stream);

/* Bytes of workspace spec_select_beams needs for sizes up to these, of both dtypes
 * (0 for sizes out of range). */
size_t specv_beam_workspace_bytes(int B, int W, int K, int V);

/*
 * The best next tokens of a request's W beams: of all (w, v)
 *   score(w, v) = scores[b,w] + logits[b,w,v] - log sum_u exp logits[b,w,u]
 * the K largest, falling, ties to the lower beam and then the lower token (within a beam
 * logits are compared: they tie where scores do, however large scores[b,w] is).  The
 * nodes of a drafted tree's next level (the beams are the last level's, scores
 * their summed log probabilities), or a beam search's step.
 *   logits    [B, W, V] of `dtype` (SPECV_F32 or SPECV_BF16), element (b, w, v)
 *             at b*batch_stride + w*row_stride + v (strides 0 or more).
 *   scores    [B, W] float32; -inf: the beam is not in play and its row not read.
 *   ended     [B, W] int32 or NULL: a beam whose text has ended (not 0) is one
 *             candidate, with the score and end_token as it is; its row is not read.
 *   out_scores [B, K] float32, tokens, beams [B, K] int32: behind the last
 *             candidate whose score, rounded to 32 bits, is above -inf: -inf, -1, -1.
 *   status    [B]: SPECV_DEV_BAD_ROW (a row has a NaN or +inf), or
 *             SPECV_DEV_BAD_BEAM (a score is one); such a request has no candidates.
 *             A row of -inf alone has none either, and is no error.
 *   W, K      1..SPECV_MAX_BEAMS.
 *   workspace specv_beam_workspace_bytes bytes for these sizes or larger ones,
 *             256-byte aligned, whatever it holds.  Calls that may run at the same time need one each.
 * A row's sum of exponentials (each within 2^-22, those of 16 entries of float32 or 32 of
 * bf16 added in 32 bits) is held in 64 bits or a pair of 32, scores are compared in 64 bits
 * and rounded once.  Two kernels, the second as a programmatic dependent
 * launch.
 */
specv_status spec_select_beams(const void* logits, int64_t batch_stride, int64_t row_stride,
                               specv_dtype dtype, int B, int W, int V, int K, const float* scores,
                               const int32_t* ended, int end_token, float* out_scores,
                               int32_t* tokens, int32_t* beams, int32_t* status, void* workspace,
                               size_t workspace_bytes, specv_stream_t stream);

/* One state of every beam: `bytes` contiguous bytes at in + b*in_batch_stride +
 * w*in_beam_stride, for w < W, and at out + b*out_batch_stride +
 * k*out_beam_stride, for k < K.  Strides count bytes, are 0 or more, those of out
 * so that no two of its places overlap. */
typedef struct specv_state {
  const void* in;
  void* out;
  int64_t in_batch_stride, in_beam_stride, out_batch_stride, out_beam_stride, bytes;
} specv_state;

/*
 * Beam k goes on from beam beams[b,k]: out[b,k] = in[b, beams[b,k]], for each of
 * num_states states, all in one call (hidden states, texts, rows of a page
 * table).  beams[b,k] = -1: an empty place, out[b,k] stays as it was.
 *   beams     [B, K] int32 in -1..W-1 (else SPECV_DEV_BAD_BEAM, and the request's
 *             states stay as they were).
 *   states    1..SPECV_MAX_STATES of them, on the host.  out may be in itself, with
 *             its strides (then every old state is read before it is overwritten);
 *             otherwise no out may overlap an in or another out (refused where both have
 *             the same strides or begin together).
 * One kernel; no workspace.
 */
specv_status spec_reorder_beams(const int32_t* beams, int B, int W, int K, const specv_state* states,
                                int num_states, int32_t* status, specv_stream_t stream);

/*
 * The sampler without any allocation, for callers that cannot allocate
 * device memory where they run it: plugin interfaces that hand the plugin
 * only the tensors it declared, serving loops that forbid cudaMalloc after
 * start-up (it can synchronise the device and fragment a fixed budget), and
 * hosts whose device memory is owned by another allocator.  The pages have
 * no counterpart; this is a packaging variant of spec_verify_sample.
 *
 * Same inputs, outputs, readings and errors as spec_verify_sample, with no
 * workspace argument: the scratch (the workspace of spec_verify_sample)
 * lives in a module-scope device array of the library of
 * SPECV_NOALLOC_SCRATCH_BYTES (4 MiB); every GPU that loads the library
 * holds it until the process exits.  Shapes whose workspace
 * (specv_workspace_bytes) exceeds it return SPECV_ERR_UNSUPPORTED.
 *   - It calls no cudaMalloc, cudaFree or allocating library routine.
 *   - Every call looks up the array's device address in the current
 *     device's context (cudaGetSymbolAddress); the first call on a device
 *     may load the library's module there, so make it before any stream
 *     capture.  `stream` must belong to the current device.
 *   - Each call zeroes the part of the array it uses (cudaMemsetAsync on
 *     `stream`), then launches the kernels.  All calls on a device share the
 *     one array: calls that may overlap on the GPU (different streams, or
 *     concurrent host threads) race and must be serialised by the caller.
 *   - The device status word is not exposed: bad data shows as
 *     accepted_len[b] = -1 and out_tokens[b,:] = -1.
 */
#define SPECV_NOALLOC_SCRATCH_BYTES (4u << 20)

specv_status spec_verify_sample_noalloc(const void* target_logits, const void* draft_logits,
                                        specv_dtype dtype, const int32_t* draft_tokens,
                                        const int32_t* draft_len, const float* temperature,
                                        const float* uniforms, const float* uniforms_resample,
                                        int B, int K, int V, int32_t* accepted_len,
                                        int32_t* out_tokens, specv_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* SPECVERIFY_H */
