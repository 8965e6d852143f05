/*
 * lsh_attn.h -- C ABI of liblsh_attn.so, LSH attention for the B200 (sm_100a)
 * and, further down, the operators of a language model around it (token table
 * and cross entropy, tokens sorted by expert).  The attention is shared-QK
 * attention restricted by random-rotation hashing, as described in "Reformer:
 * The Efficient Transformer" (arXiv 2001.04451v2):
 *   section 2 "LSH attention"     -- hash h(x) = argmax([xR; -xR]), sort by
 *                                    bucket, attend within sorted chunks;
 *   section 2 "Causal masking"    -- positions follow the same permutation,
 *                                    future positions are masked, a token may
 *                                    attend to itself only when nothing else
 *                                    is available;
 *   section 5 "Shared query-key space" -- one projection serves as query and
 *                                    key; keys are normalised;
 *   Appendix A "Multi-round attention" / "Implementation" / "Masking" --
 *                                    n_hashes independent rounds, each giving
 *                                    its own output, combined afterwards.
 *
 * Conventions shared by every call
 * --------------------------------
 *  - All tensor arguments are DEVICE pointers (cudaMalloc'd or equivalent)
 *    unless the name ends in _host.  The caller owns every buffer, including
 *    the workspace, and the library keeps no pointer after a call returns.
 *    The library allocates nothing: the stage calls and the fused call take
 *    their temporary memory from caller workspaces (sized by the
 *    *_workspace_size queries).  The two places where it holds device
 *    resources of its own are stated at their calls: lsh_attn_forward_host's
 *    streams and events, and lsh_attn_forward_noalloc's built-in scratch.
 *  - Every device pointer must be 16-byte aligned; of the token table's and
 *    the routing calls' vectors (one value per token or entry) only aligned
 *    to their values.  Tensors are dense, row-major, last dimension fastest.
 *    Outputs and workspaces share no memory with one another or with an input,
 *    unless a call says so.
 *  - `stream` is a cudaStream_t passed as void* (NULL = the legacy default
 *    stream).  All work is enqueued on it; no call synchronises the host
 *    except lsh_attn_device_check().
 *  - Arguments are checked on the host before anything is launched.  A call
 *    that returns anything but LSH_OK has launched nothing, except
 *    LSH_ERR_CUDA (a launch or copy failed part-way; lsh_attn_last_error()
 *    has the CUDA message).
 *  - Shapes (see lsh_shape): B batch, H heads, L seq_len, d d_k,
 *    n_h n_hashes, n_b n_buckets, c chunk_len.
 *  - Besides those resources, the library keeps no state between calls
 *    except one device word that records a kernel's bounded wait running out
 *    (see lsh_attn_device_check).
 */
#ifndef LSH_ATTN_H_
#define LSH_ATTN_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define LSH_ATTN_VERSION 1

#if defined(__GNUC__)
#define LSH_ATTN_API __attribute__((visibility("default")))
#else
#define LSH_ATTN_API
#endif

typedef enum lsh_status {
  LSH_OK = 0,
  LSH_ERR_INVALID_ARG = 1,     /* null/misaligned pointer, bad size or flag */
  LSH_ERR_UNSUPPORTED = 2,     /* valid request this library cannot serve  */
  LSH_ERR_WORKSPACE = 3,       /* workspace or staging buffer too small     */
  LSH_ERR_CUDA = 4,            /* a CUDA launch or copy failed              */
  LSH_ERR_DEVICE_TIMEOUT = 5   /* a kernel's bounded wait ran out           */
} lsh_status;

typedef enum lsh_dtype {
  LSH_F32 = 0,                 /* float32 qk, v, rotations, out, o_rounds   */
  LSH_BF16 = 1                 /* bfloat16 qk, v, rotations, out, o_rounds  */
} lsh_dtype;

/* lsh_shape.flags bits */
#define LSH_FLAG_PORTABLE 1u   /* use the CUDA-core kernels even where the
                                  tensor-core (tcgen05) kernels apply; for
                                  cross-checking the two kernel families   */
#define LSH_FLAG_DEDUP 2u      /* duplicate-count correction ("Reformer: The
                                  Efficient Transformer", Appendix A "Multi-
                                  round LSH attention", its "Duplicate
                                  handling" item): a key that falls in a
                                  query's window in N rounds has log N
                                  subtracted from its score in each of them,
                                  so the combined output weighs every
                                  distinct key once.  N counts the rounds r
                                  with chunk(undo_r[i]) - chunk(undo_r[j]) in
                                  {0, 1}.  Runs on the tensor-core attention
                                  for n_h <= 8 where it has a plan for the
                                  (c, d) pair, else on the CUDA-core kernel;
                                  the stage call is lsh_attn_chunked_fwd_ex. */
#define LSH_FLAG_BUCKET_MASK 4u /* bucket-equality mask (section 2 "LSH
                                  attention": a query attends only to
                                  targets in its own hash bucket): inside a
                                  window, keys whose bucket in that round
                                  differs from the query's are not attended.
                                  Runs on the tensor-core attention (on the
                                  CUDA-core kernel together with
                                  LSH_FLAG_DEDUP); the stage call is
                                  lsh_attn_chunked_fwd_ex.                 */
#define LSH_FLAG_KMEANS 8u     /* routing-style bucket assignment (the pages
                                  name online k-means for the Routing
                                  Transformer): `rotations` holds centroids
                                  [n_h, d, n_b], one set per round, and a
                                  token goes to the bucket of the centroid
                                  with the largest dot product (lowest index
                                  on ties); n_b may then be any value in
                                  [2, 32768].  bf16 with d in {64, 128} and
                                  n_b a multiple of 32 runs on the tensor-
                                  core hash kernel, other shapes on the
                                  CUDA-core one.                            */

typedef struct lsh_shape {
  int32_t batch;       /* B >= 1                                             */
  int32_t heads;       /* H >= 1                                             */
  int32_t seq_len;     /* L >= 1, < 2^31 / n_h                                */
  int32_t d_k;         /* d: 8..256, a multiple of 8                         */
  int32_t n_hashes;    /* n_h >= 1 hashing rounds                            */
  int32_t n_buckets;   /* n_b: 1, or even with 2 <= n_b <= 32768; any value
                          in [2, 32768] with LSH_FLAG_KMEANS                 */
  int32_t chunk_len;   /* c >= 1; when c does not divide L the last chunk of
                          the sorted order holds the L mod c remaining slots */
  int32_t causal;      /* 0 or 1                                             */
  int32_t dtype;       /* lsh_dtype of the floating-point tensors            */
  uint32_t flags;      /* LSH_FLAG_* bits, 0 by default                      */
} lsh_shape;

/* ---------------------------------------------------------------------- *
 * Stage 1: hash.  Section 2 "LSH attention": h(x) = argmax([xR; -xR]) with
 * a random projection R per round (Appendix A).
 *   qk        [B, H, L, d]        dtype, the shared query/key vectors.
 *   rotations [n_h, d, n_b/2]     dtype, one R per round, shared by all
 *                                 (b, h); must be NULL when n_b == 1 (every
 *                                 token then lands in bucket 0).
 *   buckets   [B, H, n_h, L]      int16 out: the argmax index in [0, n_b);
 *                                 ties go to the lowest index of [xR; -xR].
 *                                 Projections are accumulated in float32
 *                                 (exact bf16 products), so a position whose
 *                                 top two entries of [xR; -xR] are within
 *                                 float32 rounding may differ from an exact
 *                                 evaluation.
 *   inv_norm  [B, H, L]           float32 out: 1 / ||qk_i||_2, 0 for a zero row
 *                                 (the key normalisation of section 5).
 * ---------------------------------------------------------------------- */
LSH_ATTN_API lsh_status lsh_attn_hash(const lsh_shape* shape, const void* qk, const void* rotations,
                         int16_t* buckets, float* inv_norm, void* stream);

/* ---------------------------------------------------------------------- *
 * Stage 2: sort.  Section 2 / Appendix A "Implementation": per (b, h, round)
 * the positions ordered by bucket, positions increasing inside a bucket
 * (a stable sort by bucket, i.e. by the key (round, bucket, position)).
 *   buckets [B, H, n_h, L]  int16 in, values in [0, n_b).
 *   perm    [B, H, n_h, L]  int32 out: perm[.., s] = position at sorted slot s.
 *   undo    [B, H, n_h, L]  int32 out, may be NULL: undo[.., perm[.., s]] = s.
 *   counts  [B, H, n_h, n_b] int32 out, may be NULL: tokens per bucket.
 *   workspace  device memory of at least lsh_attn_sort_workspace_size()
 *              bytes (n_h * B * H * ceil(L / 2048) * n_b * 4: the per-tile
 *              bucket counts); 16-byte aligned; contents on entry ignored.
 * Bucket ids outside [0, n_b) are undefined behaviour (stage 1 never makes
 * them); the kernels do not read or write out of bounds for them.
 * A workspace smaller than the query's answer returns LSH_ERR_WORKSPACE.
 * The per-bucket counts come out of this stage, not out of stage 1: the
 * sort counts every tile of keys anyway (its first kernel), so the hash
 * needs no histogram of its own.
 * ---------------------------------------------------------------------- */
LSH_ATTN_API lsh_status lsh_attn_sort_workspace_size(const lsh_shape* shape, size_t* bytes);
LSH_ATTN_API lsh_status lsh_attn_sort(const lsh_shape* shape, const int16_t* buckets, int32_t* perm,
                         int32_t* undo, int32_t* counts, void* workspace,
                         size_t workspace_bytes, void* stream);

/* ---------------------------------------------------------------------- *
 * Stage 3: chunked attention of every round, results stored at ORIGINAL
 * positions (the unsort is folded into the store).  Section 2 "LSH
 * attention" / "Causal masking"; section 5 "Shared query-key space";
 * Appendix A "Implementation" / "Masking".  For round r, sorted slot s sits
 * in chunk k = s / c; its window is chunk k-1 (if k > 0) and chunk k.  The
 * score of query i and key j is (qk_i . qk_j) * inv_norm_j / sqrt(d); the
 * score of j == i is replaced by -1e5; with causal, j > i is excluded.
 *   qk, v       [B, H, L, d]      dtype.
 *   inv_norm    [B, H, L]         float32 (from stage 1).
 *   perm        [B, H, n_h, L]    int32 (from stage 2).
 *   o_rounds    [B, H, n_h, L, d] dtype out: softmax-weighted v per round.
 *               16-byte alignment suffices; with 32-byte alignment (every
 *               cudaMalloc'd buffer) the bf16 kernels write it in 32-byte
 *               stores, which is faster.
 *   lse_rounds  [B, H, n_h, L]    float32 out: log-sum-exp of the scores.
 * ---------------------------------------------------------------------- */
LSH_ATTN_API lsh_status lsh_attn_chunked_fwd(const lsh_shape* shape, const void* qk, const void* v,
                                const float* inv_norm, const int32_t* perm, void* o_rounds,
                                float* lse_rounds, void* stream);

/* ---------------------------------------------------------------------- *
 * Stage 3 for the variants (LSH_FLAG_DEDUP, LSH_FLAG_BUCKET_MASK, set in
 * shape->flags): as lsh_attn_chunked_fwd, plus
 *   undo    [B, H, n_h, L] int32 in, required with LSH_FLAG_DEDUP: every
 *           round's inverse permutation (the undo output of lsh_attn_sort),
 *           from which the kernel counts, for each (query, key) pair, the
 *           rounds whose window holds the pair; else may be NULL.
 *   buckets [B, H, n_h, L] int16 in, required with LSH_FLAG_BUCKET_MASK:
 *           the bucket ids of stage 1; else may be NULL.
 * ---------------------------------------------------------------------- */
LSH_ATTN_API lsh_status lsh_attn_chunked_fwd_ex(const lsh_shape* shape, const void* qk,
                                   const void* v, const float* inv_norm,
                                   const int32_t* perm, const int32_t* undo,
                                   const int16_t* buckets, void* o_rounds,
                                   float* lse_rounds, void* stream);

/* ---------------------------------------------------------------------- *
 * Stage 4: combine.  Appendix A "Multi-round attention": each round's output
 * is combined with weight exp(lse_r - LSE), LSE = logsumexp over rounds.
 *   o_rounds [B, H, n_h, L, d] dtype; lse_rounds [B, H, n_h, L] float32.
 *   out      [B, H, L, d] dtype out; lse [B, H, L] float32 out (= LSE).
 * ---------------------------------------------------------------------- */
LSH_ATTN_API lsh_status lsh_attn_combine(const lsh_shape* shape, const void* o_rounds,
                            const float* lse_rounds, void* out, float* lse, void* stream);

/* ---------------------------------------------------------------------- *
 * The whole forward pass (stages 1-4) on one stream, no host sync.
 * Produces the same out/lse as the four stage calls in sequence.
 *   workspace: device scratch of at least lsh_attn_forward_workspace_size()
 *   bytes, 256-byte aligned; its contents on entry do not matter and on
 *   return are unspecified.  Two calls in flight at once need two workspaces.
 * ---------------------------------------------------------------------- */
LSH_ATTN_API lsh_status lsh_attn_forward_workspace_size(const lsh_shape* shape, size_t* bytes);

LSH_ATTN_API lsh_status lsh_attn_forward(const lsh_shape* shape, const void* qk, const void* v,
                            const void* rotations, void* out, float* lse, void* workspace,
                            size_t workspace_bytes, void* stream);

/* ---------------------------------------------------------------------- *
 * Backward of the forward pass with the buckets and their sort held fixed
 * (the hash is piecewise constant: no gradient flows through bucket ids).
 * Gradients of `out` w.r.t. the shared qk and v for an upstream gradient
 * dout, from the multiset form of the combined output (section 2 "LSH
 * attention", Appendix A): with LSE the forward's lse output,
 *   dv_j  += exp(s_ij - LSE_i) dout_i                 over every window pair,
 *   ds_ij  = exp(s_ij - LSE_i) (dout_i . v_j - dout_i . out_i),
 * into the query and the normalised key (the self pair's -1e5 is a constant).
 *   qk, v, out, dout [B, H, L, d] dtype in; inv_norm [B, H, L] float32 and
 *   perm [B, H, n_h, L] int32 from stages 1-2; lse [B, H, L] float32 from
 *   the combine; dqk, dv [B, H, L, d] float32 out.
 *   workspace: at least lsh_attn_backward_workspace_size() bytes, 256-byte
 *   aligned.  CUDA cores with float32 atomics (the summation order, and so
 *   the last bits, can differ between runs).  The variant flags are not
 *   supported here (LSH_ERR_UNSUPPORTED).
 * ---------------------------------------------------------------------- */
LSH_ATTN_API lsh_status lsh_attn_backward_workspace_size(const lsh_shape* shape, size_t* bytes);

LSH_ATTN_API lsh_status lsh_attn_backward(const lsh_shape* shape, const void* qk, const void* v,
                             const float* inv_norm, const int32_t* perm, const void* out,
                             const float* lse, const void* dout, float* dqk, float* dv,
                             void* workspace, size_t workspace_bytes, void* stream);

/* ---------------------------------------------------------------------- *
 * The forward pass from HOST buffers: copies qk, v and rotations to the
 * device, runs the forward pass, and copies out and lse back.  The (batch,
 * head) pairs are independent, so they go in up to 8 groups through three
 * library-owned streams (copy in, compute, copy out): a group's inputs cross
 * PCIe while the previous group computes and the one before it copies back;
 * a group's qk crosses before its v, and its hash and sort start on qk alone.
 * The work starts after what is already queued on `stream`, and `stream`
 * waits for all of it, so the caller synchronises `stream` before reading
 * out_host / lse_host.  Calls on one device enqueue one at a time (a mutex
 * guards the shared streams).  Host buffers should be page-locked for the
 * copies to overlap.  On an error after the first copy was queued, `stream`
 * still waits for everything already queued (which reads and writes the
 * caller's buffers), so synchronise it before freeing them; out_host and
 * lse_host are then undefined.
 *   device_buffer: caller-owned device memory of at least
 *   lsh_attn_forward_host_device_bytes() bytes, 256-byte aligned; it holds the
 *   device copies of the inputs and outputs plus the workspace.
 * ---------------------------------------------------------------------- */
LSH_ATTN_API lsh_status lsh_attn_forward_host_device_bytes(const lsh_shape* shape, size_t* bytes);

LSH_ATTN_API lsh_status lsh_attn_forward_host(const lsh_shape* shape, const void* qk_host,
                                 const void* v_host, const void* rotations_host,
                                 void* out_host, float* lse_host, void* device_buffer,
                                 size_t device_bytes, void* stream);

/* ---------------------------------------------------------------------- *
 * The forward pass without any device allocation or caller workspace.
 * (The paper has no counterpart: this is a deployment aid of this library.)
 *
 * For callers that cannot allocate device memory: a plugin inside a host
 * framework that owns all device memory through its own pool and hands the
 * plugin only its input and output buffers, or a latency-critical path that
 * must not call cudaMalloc because it can synchronise the whole device and
 * take an unpredictable time.  Same arguments and results as
 * lsh_attn_forward, minus the workspace: the intermediates live in a scratch
 * array of LSH_ATTN_NOALLOC_SCRATCH_BYTES built into the library.
 *  - The scratch occupies that much device memory on every GPU whose
 *    context has loaded the library's device code, until the process exits.
 *    Under lazy module loading (CUDA's default, CUDA_MODULE_LOADING=LAZY)
 *    that is the GPUs where this call has run, from its first call there;
 *    with CUDA_MODULE_LOADING=EAGER it is every GPU on which the process
 *    creates a context once the library is loaded.
 *  - The first successful call on a device resolves the scratch's device
 *    address (cudaGetSymbolAddress) with that device current and keeps it;
 *    a failed lookup is retried on the next call.  Make that first call
 *    before any stream capture.
 *  - Problems whose workspace (lsh_attn_forward_workspace_size) exceeds
 *    LSH_ATTN_NOALLOC_SCRATCH_BYTES are rejected with LSH_ERR_WORKSPACE
 *    before anything is launched.
 *  - Every call on a device shares the one scratch and leaves its contents
 *    behind; nothing in it needs to start at zero.  Calls that overlap on
 *    the GPU (different streams, or different host threads, without ordering
 *    between them) race on the scratch and give wrong results: order them.
 *  - Calls no cudaMalloc, cudaFree or any other allocating routine.
 * ---------------------------------------------------------------------- */
#define LSH_ATTN_NOALLOC_SCRATCH_BYTES (64u << 20)

LSH_ATTN_API lsh_status lsh_attn_forward_noalloc(const lsh_shape* shape, const void* qk,
                                                 const void* v, const void* rotations,
                                                 void* out, float* lse, void* stream);

/* ---------------------------------------------------------------------- *
 * The token table of a language model on this attention: its lookup, the
 * lookup's gradient, and the loss against it.  (The paper computes the loss
 * of a large vocabulary in sections; the table's two ends are this library's
 * addition.)
 *   rows      n  tokens, of any number of sequences; 0 is allowed.
 *   vocab     V  rows of the table, 1 <= V <= 2^20.
 *   d_model   D  a multiple of 8 in [8, 16384].
 *   dtype     lsh_dtype of the table and of every row of D values.
 *   index_type  lsh_index_type of tokens and targets.
 *   scale     finite; see each call.
 *   flags     0 or LSH_FLAG_PORTABLE (cross entropy: CUDA cores only).
 * A token or target outside [0, V) is no error: padding (-1, say) gives a row
 * of zeros, no loss and no gradient.
 * Workspace sizes are for the current device; a workspace serves one call at
 * a time.
 * ---------------------------------------------------------------------- */
typedef enum lsh_index_type {
  LSH_I32 = 0,                 /* int32 */
  LSH_I64 = 1                  /* int64 */
} lsh_index_type;

typedef struct lsh_table {
  int64_t rows;        /* n: 0 <= n <= 2^30                                  */
  int32_t vocab;
  int32_t d_model;
  int32_t dtype;
  int32_t index_type;
  float scale;
  uint32_t flags;
} lsh_table;

/* Lookup: out[t] = scale * table[tokens[t]], a zero row for padding.
 *   tokens [n] index type; table [V, D] dtype; out [n, D] dtype out.       */
LSH_ATTN_API lsh_status lsh_attn_embed(const lsh_table* shape, const void* tokens,
                                       const void* table, void* out, void* stream);

/* Its gradient: dtable[v] = init[v] + scale * sum over tokens[t] == v of
 * dout[t], the sum in float32 and rounded once.  The tokens are sorted on the
 * device and every row of dtable is written once, without atomics: the same
 * input gives the same bits.
 *   dout [n, D] dtype; init [V, D] dtype, NULL for zeros, and may be dtable
 *   itself (the gradient is added in place); dtable [V, D] dtype out.
 *   workspace: at least lsh_attn_embed_backward_workspace_size() bytes,
 *   256-byte aligned (may be NULL when that is 0).                          */
LSH_ATTN_API lsh_status lsh_attn_embed_backward_workspace_size(const lsh_table* shape,
                                                               size_t* bytes);
LSH_ATTN_API lsh_status lsh_attn_embed_backward(const lsh_table* shape, const void* tokens,
                                                const void* dout, const void* init,
                                                void* dtable, void* workspace,
                                                size_t workspace_bytes, void* stream);

/* Softmax cross entropy of every row against the whole table, the logits
 * never stored:
 *   z_iv = scale x_i . table_v,  lse_i = log sum_v exp(z_iv),
 *   loss_i = lse_i - z_i,targets_i, and 0 for padding (lse is still given).
 * The target's exponential is kept apart from the others' sum, so that a loss
 * far below 1 keeps its digits.
 *   x [n, D] dtype; table [V, D] dtype; targets [n] index type; loss, lse
 *   [n] float32 out.
 * The rows decide which kernels run, and with them the order of the sums: up to
 * 32 float32 rows (while they fit in shared memory: 32 of D = 1600, 4 of 12800)
 * run on CUDA cores, bfloat16 and more rows on the tensor cores, more than 2^24
 * rows or LSH_FLAG_PORTABLE on the portable CUDA-core kernels.  So a row's last
 * bits may depend on how many rows stand beside it.
 * A word ruled out by a logit of -inf has no part in the sum.  But where the
 * tensor cores take float32 values, those are taken apart first, and an infinite
 * one makes every logit that it takes part in NaN.
 *   workspace: at least lsh_attn_xent_workspace_size() bytes, 256-byte
 *   aligned (may be NULL when that is 0).                                   */
LSH_ATTN_API lsh_status lsh_attn_xent_workspace_size(const lsh_table* shape, size_t* bytes);
LSH_ATTN_API lsh_status lsh_attn_xent(const lsh_table* shape, const void* x, const void* table,
                                      const void* targets, float* loss, float* lse,
                                      void* workspace, size_t workspace_bytes, void* stream);

/* Its gradients for the upstream gradient dloss [n] float32 of loss:
 *   g_iv = scale dloss_i (exp(z_iv - lse_i) - [v == targets_i]),
 *   dx_i = sum_v g_iv table_v,  dtable_v = sum_i g_iv x_i,
 * lse as the forward gave it.  Rows of padding get dx = 0 and take no part in
 * dtable, whatever x and dloss hold there and the table anywhere.
 *   dx [n, D] dtype out; dtable [V, D] dtype out.  With bfloat16, g is held in
 *   two bfloat16 values, 16 bits, for the two products; they are summed in
 *   float32 and rounded once.
 *   lse is float32, and so exp(z - lse) is off by about |lse| 2^-24 of itself.
 *   At the target, where 1 is taken from it, that error is absolute: below a loss
 *   of about |lse| 2^-24 the target's part of the gradient is rounding, its sign
 *   included.
 *   The work is that of the rows that have a target, on the tensor cores; dx of
 *   up to 128 bfloat16 rows and the CUDA-core kernels work on all rows.
 *   workspace: at least lsh_attn_xent_backward_workspace_size() bytes,
 *   256-byte aligned (may be NULL when that is 0).                          */
LSH_ATTN_API lsh_status lsh_attn_xent_backward_workspace_size(const lsh_table* shape,
                                                              size_t* bytes);
LSH_ATTN_API lsh_status lsh_attn_xent_backward(const lsh_table* shape, const void* x,
                                               const void* table, const void* targets,
                                               const float* lse, const float* dloss, void* dx,
                                               void* dtable, void* workspace,
                                               size_t workspace_bytes, void* stream);

/* ---------------------------------------------------------------------- *
 * Tokens sorted by expert and back, for a feed-forward layer whose rows are
 * routed (the routing-style assignment's counterpart outside attention).
 * Entry (t, j) is token t's j-th expert; entries are numbered t * k + j.
 *   tokens    T  0 is allowed; T * k <= 2^30.
 *   top_k     k  1..64 experts per token.
 *   n_experts E  1..1023.
 *   d_model   D  a multiple of 8 in [8, 16384].
 *   dtype     lsh_dtype of the rows; weights and their gradients are float32.
 *   index_type  lsh_index_type of the router's choice.
 * ---------------------------------------------------------------------- */
typedef struct lsh_route {
  int64_t tokens;
  int32_t top_k;
  int32_t n_experts;
  int32_t d_model;
  int32_t dtype;
  int32_t index_type;
  uint32_t flags;      /* 0                                                  */
} lsh_route;

/* The plan: entries in stable order by expert; an expert outside [0, E)
 * drops its entry (over capacity, padding), and dropped entries come last.
 * A token may name the same expert twice.
 *   experts [T, k] index type.
 *   perm    [T * k] int32 out: the entry in slot s.
 *   undo    [T, k]  int32 out: the slot of entry (t, j).
 *   offsets [E + 1] int32 out: expert e has slots offsets[e] .. offsets[e+1]-1;
 *           slots from offsets[E] on hold dropped entries.
 *   workspace: at least lsh_attn_route_sort_workspace_size() bytes, 256-byte
 *   aligned (may be NULL when that is 0).  d_model and dtype are not used.  */
LSH_ATTN_API lsh_status lsh_attn_route_sort_workspace_size(const lsh_route* shape,
                                                           size_t* bytes);
LSH_ATTN_API lsh_status lsh_attn_route_sort(const lsh_route* shape, const void* experts,
                                            int32_t* perm, int32_t* undo, int32_t* offsets,
                                            void* workspace, size_t workspace_bytes,
                                            void* stream);

/* xs[undo[t, j]] = x[t]; zero rows in the slots of dropped entries.
 *   x [T, D]; xs [T * k, D] out.                                            */
LSH_ATTN_API lsh_status lsh_attn_route_gather(const lsh_route* shape, const void* x,
                                              const int32_t* undo, const int32_t* offsets,
                                              void* xs, void* stream);

/* The gather's gradient: dx[t] = sum over kept j of dxs[undo[t, j]], summed in
 * float32 in the order of j.  Rows of dropped entries are not read.
 *   dxs [T * k, D]; dx [T, D] out.                                          */
LSH_ATTN_API lsh_status lsh_attn_route_gather_backward(const lsh_route* shape, const void* dxs,
                                                       const int32_t* undo,
                                                       const int32_t* offsets, void* dx,
                                                       void* stream);

/* out[t] = sum over kept j of weights[t, j] * y[undo[t, j]], summed in float32
 * in the order of j; a zero row for a token with no kept entry.  Rows and
 * weights of dropped entries are not read.
 *   y [T * k, D]; weights [T, k] float32; out [T, D] out.                   */
LSH_ATTN_API lsh_status lsh_attn_route_combine(const lsh_route* shape, const void* y,
                                               const float* weights, const int32_t* undo,
                                               const int32_t* offsets, void* out, void* stream);

/* The combine's gradients for dout [T, D]: dy[undo[t, j]] = weights[t, j] *
 * dout[t] and dweights[t, j] = dout[t] . y[undo[t, j]]; zero for dropped
 * entries.
 *   dy [T * k, D] out; dweights [T, k] float32 out.                         */
LSH_ATTN_API lsh_status lsh_attn_route_combine_backward(const lsh_route* shape, const void* dout,
                                                        const void* y, const float* weights,
                                                        const int32_t* undo,
                                                        const int32_t* offsets, void* dy,
                                                        float* dweights, void* stream);

/* ---------------------------------------------------------------------- *
 * Diagnostics.
 *   lsh_attn_status_string: static text for a status.
 *   lsh_attn_last_error: detail of the last failing call on this host
 *   thread (static storage, overwritten by the next failure).
 *   lsh_attn_device_check: synchronises `stream`, then reads and clears the
 *   device word that a kernel sets when one of its bounded waits runs out;
 *   returns LSH_ERR_DEVICE_TIMEOUT if it was set, LSH_ERR_CUDA if the
 *   synchronisation failed, LSH_OK otherwise.
 *   lsh_attn_version: LSH_ATTN_VERSION of the built library.
 * ---------------------------------------------------------------------- */
LSH_ATTN_API const char* lsh_attn_status_string(lsh_status status);
LSH_ATTN_API const char* lsh_attn_last_error(void);
LSH_ATTN_API lsh_status lsh_attn_device_check(void* stream);
LSH_ATTN_API int lsh_attn_version(void);

/* Number of CUDA kernels this library has launched in this process so far
 * (every stage, variant and entry point; host-side count taken at launch).
 * A diagnostic for benchmarks that report how many of their kernels ran in a
 * timed region: read it before and after.  Thread-safe; never reset. */
LSH_ATTN_API unsigned long long lsh_attn_kernel_launches(void);

/* Test hook for the failure-detection path.  Every wait inside this
 * library's tensor-core kernels is bounded (2 s); when one runs out the
 * kernel records an error word, every role of the CTA leaves its loop, work
 * already in flight is drained and the kernel returns, and
 * lsh_attn_device_check reports LSH_ERR_DEVICE_TIMEOUT.  This call sets the
 * limit, in ns, of the first wait of the tensor-core hash's MMA thread (for
 * the input tile of every CTA) for the hash launches that follow: 0 makes
 * that wait give up at once, so a test can exercise the path without any
 * fault or hang.  Returns the previous limit; pass it back to restore the
 * normal behaviour.  Process-wide; not for use while other threads launch. */
LSH_ATTN_API unsigned long long lsh_attn_test_hash_first_wait(unsigned long long ns);

/* The same for the tensor-core cross entropy: the MMA thread's first wait for
 * operands of every launch of it. */
LSH_ATTN_API unsigned long long lsh_attn_test_xent_first_wait(unsigned long long ns);

/* Test hook: the most bytes of the gradient's matrix that a piece of the
 * vocabulary may take in the cross entropy's backward (at least one tile of
 * it), for the calls and size queries that follow, so that a small case runs
 * the pieces of a large one.  Limits above the library's own change nothing.
 * Returns the previous limit.  Process-wide; not for use while other threads
 * call. */
LSH_ATTN_API unsigned long long lsh_attn_test_xent_piece_bytes(unsigned long long bytes);

#ifdef __cplusplus
}
#endif

#endif /* LSH_ATTN_H_ */
