/*
 * dsa.h -- C ABI of the DeepSeek Sparse Attention (DSA) forward pass on one
 * NVIDIA B200 (sm_100a).  Exported by libdsa.so.
 *
 * What it computes (DeepSeek-V3.2 technical-report summary, ai.flicky.cc,
 * section "DSA: внимание только к важному"):
 *
 *   lightning indexer ("Молниеносный индексатор", equation for I_{t,s}):
 *       I[t,s] = sum_{j<H_I} w[t,j] * ReLU(q_I[t,j] . k_I[s])        for s <= t
 *     with q_I and k_I in FP8 e4m3, each token carrying one positive fp32
 *     scale (q_I[t,j] = e4m3 * q_scale[t], k_I[s] = e4m3 * k_scale[s]);
 *   top-k selection and attention ("Отбор и основное внимание", equation for u_t):
 *       u_t = Attn(h_t, { c_s : I[t,s] in Top-k(I[t,:]) }),   k = 2048,
 *     MLA in MQA form: one latent KV row c_s (width d_qk) is shared by all H
 *     query heads; its leading d_v columns are the value.
 *
 * Conventions shared by every entry point:
 *   - Every pointer is caller-owned DEVICE memory, row-major and contiguous,
 *     16-byte aligned.  The library never allocates, frees or synchronises;
 *     it only enqueues kernels on `stream` (a cudaStream_t; NULL = legacy
 *     default stream).
 *   - Query i of batch b sits at sequence position t = q_offset + i and sees
 *     keys 0..t.  Keys 0..Lk-1 exist; q_offset + Lq <= Lk is required.
 *     Decode is Lq = 1, q_offset = Lk - 1; a prefill chunk is
 *     q_offset = chunk start, Lk = q_offset + Lq.
 *   - Argument and shape errors return before anything is enqueued.  A launch
 *     failure returns DSA_ERR_CUDA.  Faults inside a kernel show up at the
 *     caller's next synchronisation.  Kernels never trap: a device-side wait
 *     that exceeds its limit is recorded and reported by dsa_device_status().
 *   - Supported shapes: (H_I, d_I) in {(4, 64), (64, 128)};
 *     (H, d_qk, d_v) in {(16, 192, 128), (128, 576, 512)}; 1 <= k <= 2048;
 *     Lk < 2^31 / 16 per batch.  Anything else returns DSA_ERR_UNSUPPORTED.
 */
#ifndef DSA_H
#define DSA_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
    DSA_OK = 0,
    DSA_ERR_INVALID_ARG = 1, /* NULL pointer, negative size, misaligned pointer, q_offset+Lq > Lk */
    DSA_ERR_UNSUPPORTED = 2, /* a shape outside the supported set */
    DSA_ERR_WORKSPACE = 3,   /* workspace smaller than dsa_workspace_size() */
    DSA_ERR_CUDA = 4,        /* a CUDA runtime call or kernel launch failed */
    DSA_ERR_TIMEOUT = 5      /* a device-side wait gave up (see dsa_device_status) */
} dsa_status;

/* Inputs of the lightning indexer (equation for I_{t,s}). */
typedef struct {
    int B, Lq, Lk, q_offset;
    int H_I, d_I;            /* indexer heads and head width */
    const void *q_I;         /* e4m3 codes [B, Lq, H_I, d_I] */
    const float *q_scale;    /* fp32 [B, Lq], > 0; NULL means 1.0 */
    const void *w;           /* bf16 [B, Lq, H_I] */
    const void *k_I;         /* e4m3 codes [B, Lk, d_I] */
    const float *k_scale;    /* fp32 [B, Lk], > 0; NULL means 1.0 */
} dsa_indexer_args;

/* Inputs of the MQA / MLA-absorbed attention (equation for u_t). */
typedef struct {
    int H, d_qk, d_v;        /* query heads, latent row width, value width (d_v <= d_qk) */
    float scale;             /* softmax scale applied to q . c_s */
    const void *q;           /* bf16 [B, Lq, H, d_qk] */
    const void *kv;          /* bf16 [B, Lk, d_qk]: latent rows c_s; value = leading d_v columns */
} dsa_attn_args;

/* Which entry point dsa_workspace_size() is asked about. */
typedef enum {
    DSA_OP_TOPK = 0,
    DSA_OP_SPARSE_ATTN = 1,
    DSA_OP_FORWARD = 2,          /* dsa_forward, staged selection (the faster path) */
    DSA_OP_INDEXER_TOPK = 3,
    DSA_OP_FORWARD_LOWMEM = 4,   /* dsa_forward, fused selection (no score matrix) */
    DSA_OP_WINDOW_ATTN = 5,      /* dsa_window_attn; k = window + sinks, or INT_MAX where that is less */
    DSA_OP_SPARSE_ATTN_KV4 = 6,  /* dsa_sparse_attn_kv4 with room to unpack the cache where that is faster */
    DSA_OP_FORWARD_KV4 = 7       /* dsa_forward_kv4, staged selection and the same room */
} dsa_op;

/*
 * Indexer scores, equation for I_{t,s}.
 *   scores: fp32 [B, Lq, Lk]; scores[b,i,s] = I[q_offset+i, s] for s <= q_offset+i,
 *   and -INFINITY for s > q_offset+i.
 * Accumulation is fp32 over exact FP8 products; the per-token scales are
 * applied after the head sum (they are positive, so they commute with ReLU).
 */
dsa_status dsa_indexer_scores(const dsa_indexer_args *args, float *scores, void *stream);

/*
 * Top-k selection over indexer scores ("Отбор и основное внимание": the k
 * positions with the largest I[t,:]).
 *   scores:  fp32 [B, Lq, Lk] (only entries s <= q_offset+i are read);
 *   indices: int32 [B, Lq, k].  Row (b,i) receives the m = min(k, q_offset+i+1)
 *            positions with the largest scores, ties to the smaller position,
 *            -0.0 equal to +0.0, written in ascending position order in slots
 *            0..m-1; slots m..k-1 receive -1.
 *   workspace: may be NULL when dsa_workspace_size(DSA_OP_TOPK, ...) is 0.
 */
dsa_status dsa_topk(const float *scores, int B, int Lq, int Lk, int q_offset, int k,
                    int32_t *indices, void *workspace, size_t workspace_bytes, void *stream);

/*
 * Indexer and top-k fused: the k positions with the largest I[t,s] per row
 * (equation for I_{t,s} of "Молниеносный индексатор", then the Top-k of the
 * equation for u_t in "Отбор и основное внимание"), selected on chip as the
 * scores are produced, so the [B, Lq, Lk] score matrix is never written.
 *   indices:    int32 [B, Lq, k], exactly as dsa_topk would return for the scores
 *               of dsa_indexer_scores (ties to the smaller position, -0.0 == +0.0,
 *               ascending position order, -1 padding after min(k, t+1) slots);
 *   sel_scores: fp32 [B, Lq, k] or NULL: I[t, indices[...]] for each valid slot,
 *               -INFINITY on padding slots;
 *   workspace:  dsa_workspace_size_args(DSA_OP_INDEXER_TOPK, args, k, 0, 0) bytes
 *               (the per-row candidate lists; a few tens of MB, independent of Lk
 *               for prefill).  Its contents need not be initialised.
 */
dsa_status dsa_indexer_topk(const dsa_indexer_args *args, int k, int32_t *indices, float *sel_scores,
                            void *workspace, size_t workspace_bytes, void *stream);

/*
 * Sparse MQA attention over the selected latent rows (equation for u_t).
 *   indices: int32 [B, Lq, k]; entries outside [0, Lk) are skipped.
 *   out:     bf16 [B, Lq, H, d_v];  out[b,i,h,:] = sum_s p_s kv[b,s,:d_v],
 *            p = softmax over the selected s of scale * q[b,i,h,:] . kv[b,s,:].
 *   lse:     fp32 [B, Lq, H] or NULL; natural-log log-sum-exp of the logits
 *            (-INFINITY and out = 0 for a row with no valid entry).  A NaN in a row
 *            that a query attends to, or a logit of +INFINITY, makes its out and lse NaN.
 * Rows with B*Lq small are split over the k entries across CTAs and merged
 * (split-k); the workspace holds the partial results.
 */
dsa_status dsa_sparse_attn(const dsa_attn_args *args, int B, int Lq, int Lk,
                           const int32_t *indices, int k, void *out, float *lse,
                           void *workspace, size_t workspace_bytes, void *stream);

/*
 * dsa_sparse_attn without a workspace argument.  The pages have no counterpart
 * to this call: it is for callers that may not allocate device memory at the
 * point of the call yet still reach the split-k path (few query rows, e.g.
 * decode) -- a serving loop that committed all device memory to its own pool up
 * front, or code that must not risk the implicit device synchronisation that
 * freeing memory brings.
 *
 * Arguments, layouts, results and errors are those of dsa_sparse_attn.  The
 * split-k partials (dsa_workspace_size(DSA_OP_SPARSE_ATTN, ...) bytes; 0 when
 * B*Lq is large enough that no row is split) are kept in a fixed array of
 * DSA_NOALLOC_SCRATCH_BYTES that is part of the library's device code, so the
 * call allocates and frees nothing.  A call that needs more returns
 * DSA_ERR_WORKSPACE before launching anything.  Nothing in the array has to
 * start at zero: every partial is written before it is read.
 * Memory: the array is device memory held by every device on which it has been
 * looked up, until the process exits.  It sits in a module of its own, so with
 * the CUDA runtime's default lazy module loading only callers of this entry
 * point reserve it; with eager loading (CUDA_MODULE_LOADING=EAGER) every
 * context that loads libdsa.so does.
 * Set-up: the first call that needs the array in a CUDA context of a device
 * looks its address up (which may make the CUDA runtime load that module); the
 * address is reused until the context changes (e.g. after cudaDeviceReset).
 * Make that first call before any stream capture begins.
 * The array is shared by all calls on a device: calls whose executions overlap
 * (different streams, or host threads with no ordering between them) race on it
 * and produce wrong results.  Order them, e.g. on one stream.
 */
#define DSA_NOALLOC_SCRATCH_BYTES ((size_t)64 << 20)
dsa_status dsa_sparse_attn_noalloc(const dsa_attn_args *args, int B, int Lq, int Lk,
                                   const int32_t *indices, int k, void *out, float *lse,
                                   void *stream);

/*
 * The whole forward pass: indexer -> top-k -> sparse attention.  `iargs` and
 * `aargs` describe the same B, Lq, Lk, q_offset.
 * The selection runs one of two ways, chosen by the workspace the caller gives;
 * both produce identical indices and selected scores:
 *   staged (workspace >= dsa_workspace_size_args(DSA_OP_FORWARD, ...)): the
 *     indexer writes the causal part of the [B, Lq, Lk] fp32 score matrix into
 *     the workspace and a separate top-k kernel selects from it.  The faster
 *     path on every measured shape: the selection then runs on all SMs at full
 *     issue rate instead of competing with the indexer's epilogue.
 *   fused (workspace >= dsa_workspace_size_args(DSA_OP_FORWARD_LOWMEM, ...) but
 *     below the staged size): dsa_indexer_topk; no score matrix, a workspace of
 *     a few tens of MB, slower.
 * A workspace below both sizes is refused with DSA_ERR_WORKSPACE.
 * Short sequences (q_offset + Lq <= k): every row selects all of its positions
 * 0..t whatever the indexer says, so the pass is dense causal MLA attention (the
 * short-sequence mode of the DSA report's "Стоимость" section, where attention
 * falls back to the masked dense form): neither the indexer nor a top-k runs; the
 * attention kernel reads keys 0..t as contiguous tiles (no gathers) and writes
 * the index lists 0..t itself.
 *   indices: int32 [B, Lq, k] (as dsa_topk); out: bf16 [B, Lq, H, d_v];
 *   lse: fp32 [B, Lq, H] or NULL.
 * The workspace holds the score matrix (staged) or the candidate lists (fused),
 * then the split-k partials; its contents need not be initialised.
 */
dsa_status dsa_forward(const dsa_indexer_args *iargs, const dsa_attn_args *aargs, int k,
                       int32_t *indices, void *out, float *lse,
                       void *workspace, size_t workspace_bytes, void *stream);

/*
 * dsa_forward with two extras.
 *   sel_scores:   fp32 [B, Lq, k] or NULL: the indexer score of every selected
 *                 position (as dsa_indexer_topk), e.g. for dsa_indexer_kl_loss_selected.
 *                 When given, the indexer runs even for short sequences.
 *   stage_events: NULL, or four cudaEvent_t handles (created by the caller)
 *                 recorded on `stream` before the indexer, after the indexer,
 *                 after the top-k (on the fused path the second and third
 *                 coincide: the top-k is part of the indexer) and after the
 *                 attention (including its split-k merge).  For short sequences
 *                 without sel_scores the first three coincide (the attention
 *                 writes the index lists).
 */
dsa_status dsa_forward_timed(const dsa_indexer_args *iargs, const dsa_attn_args *aargs, int k,
                             int32_t *indices, float *sel_scores, void *out, float *lse,
                             void *workspace, size_t workspace_bytes, void *stream,
                             void *const *stage_events);

/*
 * Forward of the lightning indexer's training loss (section "Как учили
 * индексатор": the indexer learns the main attention's distribution through a
 * KL divergence; in the sparse stage only over the selected positions).
 * For query row (b,i) with the valid selected positions S (indices entries in
 * [0, Lk); others are padding):
 *   a_h[s]  = exp(scale * q[b,i,h,:] . kv[b,s,:] - lse[b,i,h])   (the attention
 *             probabilities of head h, as dsa_sparse_attn computes them);
 *   p[s]    = sum_h a_h[s] / sum_{s' in S} sum_h a_h[s']          (target, L1-normalised);
 *   kl[b,i] = sum_{s in S} p[s] * (log p[s] - log softmax_S(scores[b,i,:])[s]).
 *   args, B, Lq, Lk, indices, k: as dsa_sparse_attn (same shapes and limits);
 *   lse:    fp32 [B, Lq, H], the natural-log log-sum-exp that dsa_sparse_attn
 *           returned for the same q, kv and indices;
 *   scores: fp32 [B, Lq, Lk], the indexer scores (dsa_indexer_scores layout);
 *           only the selected entries are read, and they must be finite;
 *   target: fp32 [B, Lq, k] or NULL: p at each index slot, 0 on padding slots;
 *   kl:     fp32 [B, Lq]: the per-row loss, 0 for a row with no valid entry.
 * The reduction over rows (sum or mean) is left to the caller.  No workspace.
 */
dsa_status dsa_indexer_kl_loss(const dsa_attn_args *args, int B, int Lq, int Lk,
                               const int32_t *indices, int k, const float *lse,
                               const float *scores, float *target, float *kl, void *stream);

/*
 * dsa_indexer_kl_loss with the indexer scores given per index slot instead of as
 * a full matrix: sel_scores fp32 [B, Lq, k], sel_scores[b,i,j] = I[t, indices[b,i,j]]
 * for every valid slot j (padding slots are not read) -- what dsa_forward_timed
 * and dsa_indexer_topk return.  Everything else is dsa_indexer_kl_loss.
 */
dsa_status dsa_indexer_kl_loss_selected(const dsa_attn_args *args, int B, int Lq, int Lk,
                                        const int32_t *indices, int k, const float *lse,
                                        const float *sel_scores, float *target, float *kl, void *stream);

/*
 * Norm and position rotation of query and key heads in one pass: what makes the
 * indexer's e4m3 queries and keys, the attention's queries and the latent rows from
 * the projections' outputs.  (The pages give no formula for this step; it is the
 * ordinary norm of a head followed by the rotary embedding.)  Per head row x of D columns, in
 * fp32:
 *   z[i] = (x[i] - mean) * r * weight[i] + bias[i]  for i < norm_dim, z[i] = x[i] behind;
 *          r = 1/sqrt(mean((x - mean)^2) + eps) over the norm_dim columns; for
 *          DSA_NORM_RMS mean is 0 and there is no bias;
 *   y = z with its pairs in columns [rot_start, rot_start + 2*n_freq) turned by the
 *       angle pos * inv_freq[j]:  (a cos - b sin, b cos + a sin).  Pair j is
 *       (rot_start + j, rot_start + n_freq + j), or (rot_start + 2j, rot_start + 2j + 1)
 *       when interleaved.  The angle is reduced in 64 bits, so far positions are exact.
 * x may be a slice of a wider buffer (strides in elements, columns contiguous); a stride
 * of 0 reads the same rows again.  Nothing is recorded for a gradient: dsa_norm_rope_bwd is
 * called with the same arguments.  D, norm_dim, rot_start, the strides: multiples of 8;
 * n_freq: a multiple of 8; 8 <= D <= 1024.  B * L and B * L * H below 2^31.
 */
typedef enum { DSA_NORM_NONE = 0, DSA_NORM_RMS = 1, DSA_NORM_LAYER = 2 } dsa_norm;

typedef struct {
    int B, L, H, D;
    int64_t stride_b, stride_l, stride_h; /* of x, in elements, >= 0 */
    const void *x;             /* bf16 [B, L, H, D] by strides */
    int norm;                  /* dsa_norm */
    int norm_dim;              /* leading columns that are normalised (ignored for DSA_NORM_NONE) */
    float eps;                 /* >= 0 */
    const void *weight;        /* [norm_dim] */
    const void *bias;          /* [norm_dim] or NULL (DSA_NORM_LAYER only) */
    int weight_bf16;           /* weight and bias in bf16; 0: fp32 */
    int rot_start, n_freq;     /* n_freq = 0: no rotation */
    int interleaved;
    const float *inv_freq;     /* fp32 [n_freq], radians per position */
    const int32_t *positions;  /* int32 [B, L], or NULL: q_offset + l */
    int q_offset;
} dsa_norm_rope_args;

/*
 * scale == NULL: out is bf16 [B, L, H, D], contiguous, y rounded once.
 * Otherwise out is e4m3 [B, L, H, D] and scale fp32 [B, L], as the indexer takes them
 *   (dsa_indexer_args q_I/q_scale, or k_I/k_scale with H = 1): scale = max(amax of |y|
 *   over the token's heads, 1e-30) / 448, code = rne(y / scale), both quotients in fp32.  A
 *   token with a NaN has a NaN scale; one with an infinity has an infinite scale, zeros for its
 *   finite values and NaN codes for the infinite ones.
 * out must not overlap x.
 */
dsa_status dsa_norm_rope(const dsa_norm_rope_args *args, void *out, float *scale, void *stream);

/*
 * Gradient of the bf16 form (the e4m3 rounding passes the gradient through unchanged).
 *   dy: bf16 [B, L, H, D], contiguous; dx: bf16 [B, L, H, D], contiguous, one row for
 *   each row read (the caller adds rows that a stride of 0 repeated);
 *   dweight, dbias: fp32 [norm_dim] (dweight required unless DSA_NORM_NONE, dbias exactly
 *   when bias is given).  Sums are taken in a fixed order: the same call gives the same bits.
 *   workspace: dsa_norm_rope_bwd_workspace(args) bytes; its contents need not be initialised.
 * dx must not overlap dy or x.
 */
dsa_status dsa_norm_rope_bwd(const dsa_norm_rope_args *args, const void *dy, void *dx, float *dweight,
                             float *dbias, void *workspace, size_t workspace_bytes, void *stream);
size_t dsa_norm_rope_bwd_workspace(const dsa_norm_rope_args *args);

/*
 * The latent cache in 4 bits (2.8 times smaller than bf16 at d_qk = 576, d_v = 512).
 * Value columns are held in groups of 32 as integers q in -7..7 and one bf16 step:
 *   step = max|x| / 7 rounded up to 5 significant bits, q = rne(x / step), value = q*step,
 * which is exact in bf16.  The tail (columns behind d_v, the rotated ones) stays bf16.
 * A group with its largest magnitude below 2^-100 is stored as zeros; one with a NaN, an
 * infinity or a magnitude above 2^126 reads back as NaN.
 *   codes:  u8 [B, Lk, d_v/2].  Nibble = q + 8.  With chunk c = col/64, part p = col/16%4,
 *           word w = col/8%2 the 8 columns of a word lie in the 4 bytes (little-endian) at
 *           p*(d_v/8) + c*8 + w*4, column e = col%8 in nibble e/2 + 4*(e%2), counted from
 *           the low end;
 *   scales: bf16 [B, Lk, d_v/32], the step of group g = col/32 at (g%2)*(d_v/64) + g/2;
 *   tail:   bf16 [B, Lk, d_qk - d_v].
 * (d_qk, d_v) in {(192, 128), (576, 512)}, as the attention; B * Lk below 2^31.
 */
typedef struct {
    int B, Lk, d_qk, d_v;
    void *codes, *scales, *tail;
} dsa_kv4_cache;

/*
 * Stores kv (bf16 [B, L, d_qk]) in cache rows first .. first + L - 1 of each sequence, where
 * first is start[b] (int32 [B]) or, with start == NULL, offset.  Rows outside [0, Lk) are
 * not stored; every other cache row is left as it was.
 */
dsa_status dsa_kv4_write(const dsa_kv4_cache *cache, const void *kv, int L, const int32_t *start, int offset,
                         void *stream);
/* Reads the same rows back into kv as the values they stand for (rows outside [0, Lk): zeros). */
dsa_status dsa_kv4_read(const dsa_kv4_cache *cache, void *kv, int L, const int32_t *start, int offset,
                        void *stream);

/*
 * dsa_sparse_attn over the 4-bit cache: the same attention with c_s as the cache holds it
 * (its values are exact in bf16, so nothing is rounded on the way to the matrix product).
 *   indices, k, out, lse, limits: as dsa_sparse_attn.  Rows of the cache that no valid entry
 *   of a query names have no part in its result: they may hold anything.
 *   workspace: DSA_OP_SPARSE_ATTN bytes at least.  Where the lists name each row many times (a
 *   prefill chunk) DSA_OP_SPARSE_ATTN_KV4 asks for room for the rows in bf16 as well
 *   (B * Lk * d_qk * 2 bytes, for the call only); with it the cache is unpacked once instead
 *   of at every use.  The result is the same bit for bit.
 */
typedef struct {
    int H, d_qk, d_v;
    float scale;
    const void *q;                       /* bf16 [B, Lq, H, d_qk] */
    const void *codes, *scales, *tail;   /* dsa_kv4_cache arrays of [B, Lk, ...] */
} dsa_kv4_attn_args;
dsa_status dsa_sparse_attn_kv4(const dsa_kv4_attn_args *args, int B, int Lq, int Lk, const int32_t *indices, int k,
                               void *out, float *lse, void *workspace, size_t workspace_bytes, void *stream);

/*
 * dsa_forward with the latent rows in the 4-bit cache (the indexer's keys stay e4m3).
 *   sel_scores: as dsa_forward_timed (may be NULL); workspace: as dsa_forward (DSA_OP_FORWARD
 *   or DSA_OP_FORWARD_LOWMEM), or DSA_OP_FORWARD_KV4 with the room that dsa_sparse_attn_kv4
 *   describes, here for the first q_offset + Lq rows of each sequence, which are all that the
 *   selection can name; short sequences as there.
 */
dsa_status dsa_forward_kv4(const dsa_indexer_args *iargs, const dsa_kv4_attn_args *kargs, int k, int32_t *indices,
                           float *sel_scores, void *out, float *lse, void *workspace, size_t workspace_bytes,
                           void *stream);

/*
 * MLA attention with a sliding window and sinks, for layers without a selection (the pages
 * have no counterpart; same q, kv, out and lse as dsa_sparse_attn).
 *   Query i of sequence b sits at t = (start ? start[b] : q_offset) + i and sees the keys
 *   s with t - window < s <= t, and the first `sinks` keys s < sinks, s <= t; of either only
 *   those in [0, Lk).  start: int32 [B], sequences of different lengths (any values; a
 *   query that sees nothing gets out = 0, lse = -INFINITY).  Keys that no query sees are
 *   not read into a result: they may hold anything.
 *   1 <= window, 0 <= sinks, Lq <= Lk; without start q_offset + Lq <= Lk.
 *   workspace: dsa_workspace_size(DSA_OP_WINDOW_ATTN, B, Lq, Lk, window + sinks, H, d_v).
 */
dsa_status dsa_window_attn(const dsa_attn_args *args, int B, int Lq, int Lk, int q_offset, const int32_t *start,
                           int window, int sinks, void *out, float *lse, void *workspace, size_t workspace_bytes,
                           void *stream);

/*
 * Bytes of device workspace the entry point `op` needs for these sizes (0 = none).
 * For DSA_OP_FORWARD, DSA_OP_FORWARD_LOWMEM, DSA_OP_FORWARD_KV4 and DSA_OP_INDEXER_TOPK it assumes
 * H_I = 64, d_I = 128 and q_offset = Lk - Lq (decode, or a prefill chunk);
 * dsa_workspace_size_args gives the exact figure for any indexer arguments.
 * DSA_OP_FORWARD includes the fp32 score matrix, B * Lq * Lk * 4 bytes (4.3 GB
 * at Lq = Lk = 32768).
 */
size_t dsa_workspace_size(dsa_op op, int B, int Lq, int Lk, int k, int H, int d_v);

/* Exact workspace of `op` for these indexer arguments (pointers are not read; 0 for
 * invalid arguments).  H and d_v describe the attention (ignored for
 * DSA_OP_INDEXER_TOPK and DSA_OP_TOPK). */
size_t dsa_workspace_size_args(dsa_op op, const dsa_indexer_args *iargs, int k, int H, int d_v);

/* Human-readable name of a status code (static storage; never NULL). */
const char *dsa_status_string(dsa_status status);

/*
 * Device-side status of this library on the current device: reads (and, when
 * `clear` is non-zero, resets) the word the kernels write when a bounded wait
 * gives up.  Synchronises the device.  Returns DSA_OK or DSA_ERR_TIMEOUT
 * (DSA_ERR_CUDA if the read itself fails).
 */
dsa_status dsa_device_status(int clear);

/*
 * Self-test of the failure path: launches one CTA that waits, with a limit of
 * about `spin_limit` polls, on a barrier that nothing will ever complete, and
 * returns DSA_ERR_TIMEOUT after synchronising if (and only if) the wait gave
 * up and the kernel returned normally.  Clears the device status first and
 * afterwards.  No fault, trap or hang is involved.
 */
dsa_status dsa_selftest_wait_timeout(uint32_t spin_limit, void *stream);

/* Library version: major * 10000 + minor * 100 + patch. */
int dsa_version(void);

#ifdef __cplusplus
}
#endif

#endif /* DSA_H */
