/*
 * qsa.h -- C ABI of the QSA attention hot path for NVIDIA GB300 (sm_103a).
 *
 * The path has three steps, named after the kernels of the audit pages on
 * sparse selected attention:
 *   qsa_prep   query RMS-norm + RoPE, K/V int8 quantisation into the cache;
 *   qsa_score  head-reduced fp32 scores of every causal cache cell;
 *   qsa_attn   chunked attention over a per-token list of selected cell ids.
 *
 * Conventions shared by every entry point:
 *  - All buffer pointers in the argument structs are DEVICE pointers owned by
 *    the caller.  The library allocates nothing and keeps no state between
 *    calls; it only reads the structs during the call.
 *  - Every call is asynchronous on `stream` (a cudaStream_t passed as void*;
 *    NULL means the legacy default stream).  A QSA_OK return means the
 *    arguments were accepted and the kernels were enqueued.
 *  - Argument errors are detected on the host before anything is enqueued and
 *    are returned synchronously (QSA_ERR_INVALID_ARG, QSA_ERR_UNSUPPORTED).
 *    Argument validation makes no CUDA call.
 *  - Conditions only the device can see (an id outside [-1, cache_cells), a
 *    bounded wait that gave up) set bits (QSA_DEVERR_*) in the caller's
 *    optional device word `err` with atomicOr; read it after synchronising.
 *  - Outputs are never pre-cleared: cells a call does not define (scores
 *    beyond the causal boundary) keep whatever the caller put there.
 *  - fp16 values are passed as uint16_t bit patterns (IEEE binary16); where a
 *    call takes several types, as void* beside a qsa_dtype.
 *  - No C++ exception crosses this boundary.
 */
#ifndef QSA_H
#define QSA_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define QSA_ABI_VERSION 3

typedef enum {
    QSA_OK = 0,
    QSA_ERR_INVALID_ARG = 1,  /* null or misaligned pointer, bad size, bad dtype */
    QSA_ERR_UNSUPPORTED = 2,  /* a shape outside the built kernels (heads, head_dim, group) */
    QSA_ERR_CUDA = 3          /* a CUDA runtime call or launch failed; see qsa_last_error() */
} qsa_status;

/* Bits of the device error word. */
#define QSA_DEVERR_BAD_ID 1u   /* an id < -1 or >= cache_cells was seen and treated as padding */
#define QSA_DEVERR_TIMEOUT 2u  /* a bounded wait gave up; that launch's outputs are incomplete */
#define QSA_DEVERR_NO_PAGES 4u /* qsa_page_update: a row did not get the pages, table columns or slots it asked for */

typedef enum { QSA_F32 = 0, QSA_F16 = 1, QSA_BF16 = 2 /* paged calls only */ } qsa_dtype;

/*
 * qsa_prep -- "Round 36 Track C: qsa_prep Single-Barrier norm_rope & w == 128
 * tg_sum + qsa_score_mm Loop Unrolling", section "Summary & Decision": the
 * prep kernel normalises the query rows (RMS reduction, scale rs, weight g),
 * rotates the dims below QROT against partner tid ^ 32, and writes int8 K/V
 * codes kq, vq with their scales ksc, vsc ("round 11 track b: qsa attention
 * and score", "implementation and evaluator": four scale groups per row).
 *
 * For token t (position p = pos0 + t) and query head h, with x = q_in[t,h,:]:
 *   rs = 1/sqrt(mean(x^2) + eps);  y = (rs*x)*norm_w
 *   for i < rope_dims/2, a = p * fp32(rope_theta^(-2i/rope_dims)):
 *     y'[i] = y[i] cos a - y[i+rope_dims/2] sin a
 *     y'[i+rope_dims/2] = y[i+rope_dims/2] cos a + y[i] sin a
 *   q_out[t,h,:] = fp16_rne(y');  q_out_f32[t,h,:] = y' (if non-NULL)
 * K and V rows t are quantised into cache row pos0 + t, per group of `group`
 * dims: s = fp16_rne(fp32(amax/127)); code = s == 0 ? 0 :
 * clamp(rint_half_even(fp32(x / s)), -127, 127).  Bit-exact by definition.
 * With rope_k = 1 the key row is first rotated with the same pairs and
 * angles (no norm), in float32 steps: c = fp32(cos a), s = fp32(sin a) from
 * double-precision cos / sin, k'[i] = fp32(fp32(k[i] c) - fp32(k[i+h] s)),
 * k'[i+h] = fp32(fp32(k[i+h] c) + fp32(k[i] s)); the pages rotate only the
 * query rows, so this is an option (off = 0).
 * qbar_out: NULL, or a qsa_score workspace for these ntok tokens (at least
 * qsa_score_workspace_bytes(ntok, head_dim) bytes, 256-byte aligned) that
 * receives the score's head sum of the rotated queries: per token, fp32
 * qbar[d] = sum_h q_out_f32[t,h,d] in head order, scaled by the token's power
 * of two 2^e (see qsa_score) and stored as the fp16 pair hi = fp16(qbar 2^e),
 * lo = fp16(qbar 2^e - hi), with e after the rows; padding rows zero.  A
 * following qsa_score with workspace_holds_qbar = 1 then needs neither q nor
 * its own head-sum pass.
 *
 * Layouts (row-major, contiguous): q_in [ntok, n_q_heads, head_dim] fp32;
 * k_in, v_in [ntok, n_kv_heads, head_dim] fp32; norm_w [head_dim] fp32;
 * q_out [ntok, n_q_heads, head_dim] fp16; q_out_f32 same shape fp32 or NULL;
 * kq, vq [cache_cells, head_dim] int8; ksc, vsc [cache_cells, head_dim/group]
 * fp16.  Requires pos0 + ntok <= cache_cells.  Supported: n_kv_heads == 1,
 * head_dim == 128, group == 32, 1 <= n_q_heads <= 30, rope_dims a multiple
 * of 8 in [0, head_dim].  Float pointers and kq/vq must be 16-byte aligned.
 */
typedef struct {
    int ntok, pos0, n_q_heads, n_kv_heads, head_dim, group, rope_dims, cache_cells;
    float eps, rope_theta;
    const float *q_in, *k_in, *v_in, *norm_w;
    uint16_t *q_out;
    float *q_out_f32;
    int8_t *kq, *vq;
    uint16_t *ksc, *vsc;
    int rope_k; /* added in ABI version 2: 1 = rotate the key rows before quantising, 0 = not */
    void *qbar_out; /* added in ABI version 2: NULL or a qsa_score workspace, see above */
} qsa_prep_args;

/*
 * qsa_score -- "Round 36 Track C ..." section "Summary & Decision" (the
 * qsa_score_mm 64x64x128 tile matmul of queries against the int8 key cache)
 * and "round 11 track b: qsa attention and score", sections "implementation
 * and evaluator" and "score: valid negative result" (head-reduced output,
 * scalar dead-key tail, untouched beyond-causal cells).
 *
 *   scores[t*ld + c] = sum_h sum_g ksc[c,g] * sum_{d in g} q[t,h,d] * kq[c,d]
 * for 0 <= c <= pos0 + t; every other element of `scores` is left untouched.
 *
 * q: [ntok, n_q_heads, head_dim] in q_dtype (QSA_F32 or QSA_F16).
 * kq [cache_cells, head_dim] int8, ksc [cache_cells, head_dim/group] fp16.
 * scores: fp32, row stride ld (elements), ld >= pos0 + ntok.
 * workspace: device scratch of at least qsa_score_workspace_bytes(ntok,
 * head_dim) bytes, 256-byte aligned; the call overwrites it.  Two calls that
 * share a workspace must not run concurrently.  It holds the head sum the
 * score is computed from: with workspace_holds_qbar = 1 the caller has
 * already filled it through qsa_prep's qbar_out for the same tokens, q is
 * ignored (it may be NULL) and the head-sum pass is skipped; the scores are
 * bit-identical to those computed from the fp32 q_out_f32 of that prep.
 * max_ctas: 0 runs one persistent CTA per SM (each CTA takes all of an SM's
 * tensor memory); n > 0 runs at most n.  A caller that overlaps the score with
 * other kernels on another stream caps it so that those kernels keep the
 * remaining SMs; the scores do not depend on the cap.  Negative is rejected.
 * Range: the head sum qbar[t,:] = sum_h q[t,h,:] travels as an fp16 pair
 * hi + lo under a per-token power of two 2^e_t: e_t = 0 while the row's
 * largest |qbar| lies in [2^-4, 2^14), otherwise the row is scaled into
 * [2^13, 2^14) (|e_t| <= 120), and the scores are multiplied back by 2^-e_t.
 * Each element then carries about 22 significant bits relative to its row's
 * largest, for any finite row whose largest element is between about 2^-107
 * and the fp32 maximum; the scores meet 1e-4 * sum|terms| across that range.
 * Elements more than about 2^37 below their row's largest keep less (the fp16
 * lo part underflows), and a row with an inf or NaN gives non-finite scores,
 * as the definition does.
 * Requires pos0 + ntok <= cache_cells.  Supported: head_dim == 128,
 * group == 32, 1 <= n_q_heads <= 64.  q, kq 16-byte aligned; ksc 8-byte.
 */
typedef struct {
    int ntok, pos0, n_q_heads, head_dim, group, cache_cells;
    const void *q;
    int q_dtype;
    const int8_t *kq;
    const uint16_t *ksc;
    float *scores;
    int64_t ld;
    void *workspace;
    size_t workspace_bytes;
    unsigned int *err;
    int workspace_holds_qbar; /* added in ABI version 2: 0 or 1, see above */
    int max_ctas;             /* added in ABI version 3: 0 = one CTA per SM, n > 0 = at most n, see above */
} qsa_score_args;

/* Bytes of workspace qsa_score needs for `ntok` tokens (0 on bad input). */
size_t qsa_score_workspace_bytes(int ntok, int head_dim);

/*
 * qsa_attn -- "round 11 track b: qsa attention and score", section
 * "implementation and evaluator" (per-token selected ids, -1 padding, 64-cell
 * chunks, incomplete chunks) and "round 5 track b: cached residual norms and
 * fused mtp attention", sections "mtp attention" and "preflight / ownership"
 * (per-chunk maxima and denominators, max-first chunk merge, one value load
 * per dimension per cell shared by all query heads).
 *
 * For token t and head h, chunk c covers id slots 64c .. 64c+63; a slot is
 * valid when 0 <= id < cache_cells (ids < -1 or >= cache_cells are treated
 * as padding and set QSA_DEVERR_BAD_ID).  Head h reads KV head
 * kv = h / (n_q_heads / n_kv_heads) (the pages' mtp grid: two KV heads per
 * token, 12 query heads on each).
 *   s_j = softmax_scale * sum_g ksc[id,kv,g] * sum_{d in g} q[t,h,d] * kq[id,kv,d]
 *   m_c = max s_j, l_c = sum exp(s_j - m_c), o_c = sum exp(s_j - m_c) v_j
 *   with v_j[d] = vsc[id, kv, d/group] * vq[id, kv, d];
 *   O = sum_c exp(m_c - M) o_c / sum_c exp(m_c - M) l_c, M = max m_c;
 *   out = fp16(O), or with a gate (same section: "sigmoid gate", fp32 gates)
 *   out[t,h,d] = fp16(O[t,h,d] / (1 + exp(-gate[t,h,d]))).
 * A token with no valid slot outputs +0.
 *
 * q [ntok, n_q_heads, head_dim] fp16; kq, vq [cache_cells, n_kv_heads,
 * head_dim] int8; ksc, vsc [cache_cells, n_kv_heads, head_dim/group] fp16;
 * ids [ntok, width] int32, width a multiple of 64; out [ntok, n_q_heads,
 * head_dim] fp16; gate NULL or [ntok, n_q_heads, head_dim] fp32.
 * part: NULL, or [ntok, width/64, n_q_heads, head_dim + 2] fp32 receiving each
 * chunk's ungated (o_c[0..head_dim), m_c, l_c); an empty chunk gives
 * (0, -inf, 0).  A non-NULL part selects the split path (per-chunk kernel,
 * then a merge kernel that reads part back); NULL selects the fused
 * single-kernel path.  All pointers are device pointers owned by the caller.
 * Supported: (head_dim 128, group 32) -- the workload's shape -- or
 * (head_dim 256, group 64) -- the pages' own; n_q_heads a multiple of
 * n_kv_heads with 1..16 query heads per KV head; otherwise
 * QSA_ERR_UNSUPPORTED.  q, kq, vq, out, part 16-byte aligned; ksc, vsc
 * 8-byte; ids, gate 4-byte.
 */
typedef struct {
    int ntok, n_q_heads, n_kv_heads, head_dim, group, cache_cells, width;
    const uint16_t *q;
    const int8_t *kq, *vq;
    const uint16_t *ksc, *vsc;
    const int32_t *ids;
    float softmax_scale;
    uint16_t *out;
    float *part;
    unsigned int *err;
    const float *gate; /* added in ABI version 2 */
} qsa_attn_args;

/*
 * qsa_score_noalloc -- the pages have no counterpart to this entry point; it
 * exists for callers that cannot allocate device memory at the time they
 * score: for instance a plugin whose host engine owns all device memory and
 * forbids allocation inside its execute callback, or a serving loop that must
 * not call cudaMalloc because that call can synchronise the device and has no
 * latency bound.  It computes exactly what qsa_score computes, but instead of
 * the caller's workspace it uses a scratch array built into the library
 * (QSA_SCORE_NOALLOC_MAX_TOKENS * 516 bytes, about 4 MiB of device memory,
 * held on every GPU that loads the library until the process exits).  The
 * `workspace`, `workspace_bytes` and `workspace_holds_qbar` fields are ignored:
 * the head sum is always computed from q; `max_ctas` applies as in qsa_score.
 *
 *  - ntok above QSA_SCORE_NOALLOC_MAX_TOKENS is rejected with
 *    QSA_ERR_INVALID_ARG; nothing is enqueued.
 *  - It never allocates: no cudaMalloc, cudaFree or allocating library call.
 *  - The first call on each device looks up the scratch array's device
 *    address (cudaGetSymbolAddress) with that device current; make that
 *    first call before any stream capture.  The address is kept for the
 *    life of the process: it does not survive cudaDeviceReset(), after
 *    which this entry point must not be called on that device again.
 *  - All calls share the one array and it keeps the last call's contents.
 *    Every call rewrites what it reads, so nothing needs clearing, but two
 *    calls whose kernels overlap on the GPU (different streams without an
 *    ordering dependency, or different host threads) race on it and give
 *    wrong scores: order them on one stream or with events.
 */
#define QSA_SCORE_NOALLOC_MAX_TOKENS 8192
qsa_status qsa_score_noalloc(const qsa_score_args *args, void *stream);

/*
 * qsa_select -- the scores -> ids step between qsa_score and qsa_attn.  The
 * pages name its buffers ("Round 36 Track C ...", section "Summary &
 * Decision": scores, ids, pooled) and the decode window ("round 5 track b:
 * cached residual norms and fused mtp attention", section "mtp attention":
 * 64 sink + 256 previous local + 1 current cell) but not the rule; this is
 * the plainest reading.  For token t (p = pos0 + t):
 *   forced = {0 .. min(sink, p+1)-1} U {max(sink, p-local) .. p-1} U {p};
 *   the other causal cells c <= p are ranked by scores[t*ld + c] (float32,
 *   descending; equal scores, -0 and +0 included, rank the lower id first;
 *   a NaN ranks below every number, -inf included, NaNs among themselves by
 *   id) and the best min(p+1, budget) - |forced| of them are added (none
 *   when the forced cells alone reach the budget: they are all kept);
 *   ids[t, :] = the chosen cells ascending, then -1 up to width.
 * Deterministic and bit-exact for a given score array.
 * scores [ntok, ld] fp32: the ranked cells are read in aligned 16-byte
 * blocks, so up to three neighbouring cells on either side (within those
 * blocks) may be read too and are ignored; ids [ntok, width] int32, every
 * element written.  Both device pointers, owned by the caller, 4-byte
 * aligned.
 * Requires 1 <= budget <= width, width % 64 == 0, sink, local >= 0,
 * sink + local + 1 <= width and pos0 + ntok <= ld, else
 * QSA_ERR_INVALID_ARG; pos0 + ntok <= QSA_SELECT_MAX_CELLS (a row's top
 * digits are cached on chip), else QSA_ERR_UNSUPPORTED.  Nothing is
 * enqueued on an error.  Uses about 42 KB of shared memory per block and
 * no global scratch.
 */
#define QSA_SELECT_MAX_CELLS 32768
typedef struct {
    int ntok, pos0, width, budget, sink, local;
    const float *scores;
    int64_t ld;
    int32_t *ids;
} qsa_select_args;

qsa_status qsa_select(const qsa_select_args *args, void *stream);

/*
 * qsa_fill_ids_decode, qsa_fill_ids_even -- the per-token selected-id lists of
 * the two workload families, written on the device (ids [ntok, width] int32,
 * a device pointer owned by the caller, 4-byte aligned; every element is
 * written).  For token t at position p = pos0 + t:
 *  decode ("round 5 track b: cached residual norms and fused mtp attention",
 *  section "mtp attention": 64 sink + 256 previous local + the current
 *  cell): the cells 0 .. min(sink, p)-1, then max(sink, p-local) .. p-1,
 *  then p, ascending, then -1.  Requires sink + local + 1 <= width.
 *  even ("round 11 track b: qsa attention and score", sections "boundaries
 *  and provenance" and "implementation and evaluator": evenly spaced unique
 *  causal cells, unused slots poisoned with -1): with n = p + 1 and
 *  k = min(n, select), slot j < k holds j when k == n and
 *  floor(j (n-1) / (k-1)) otherwise (so 0 and p are always present), then
 *  -1.  Requires 2 <= select <= width.
 * Both are integer closed forms, exact.  Arguments are checked before
 * anything is enqueued (QSA_ERR_INVALID_ARG).
 */
qsa_status qsa_fill_ids_decode(int ntok, int pos0, int width, int sink, int local, int32_t *ids, void *stream);
qsa_status qsa_fill_ids_even(int ntok, int pos0, int width, int select, int32_t *ids, void *stream);

qsa_status qsa_prep(const qsa_prep_args *args, void *stream);
qsa_status qsa_score(const qsa_score_args *args, void *stream);
qsa_status qsa_attn(const qsa_attn_args *args, void *stream);

/*
 * The paged cache.  Several sequences share one pool of pages, each page
 * page_size cells of all KV heads, in the cache format of qsa_prep and
 * qsa_attn:
 *   kq, vq   int8 [n_layers, n_pages, page_size, n_kv_heads, head_dim]
 *   ksc, vsc fp16 [n_layers, n_pages, page_size, n_kv_heads, 4]
 * One layer of it is a qsa_attn cache of n_pages * page_size cells.  Cell c of
 * row r (a sequence) is pool cell
 *   page_table[r, c / page_size] * page_size + c % page_size
 * for c < seq_lens[r]; page_table is int32 [rows, max_pages], seq_lens int32
 * [rows].  A page may belong to several rows (a fork); the pages that no row
 * holds are free.
 * Supported: (head_dim 128, group 32) or (head_dim 256, group 64);
 * page_size 16, 32, 64, 128 or 256; n_pages * page_size below 2^31.
 * Outputs overlap neither each other nor the inputs, but where a call says so.
 * The page calls keep the whole state in the caller's device buffers and never
 * synchronise, so a decode loop (update, prep, attention) can be captured in a
 * graph.  The pages have no counterpart to these calls; they extend the path
 * of the pages to many sequences.
 */

/*
 * qsa_paged_prep -- the new tokens of any number of sequences: per-head RMS
 * norm of queries and keys, rotation of both, and the quantised K/V rows
 * written to their slots.
 *
 * For token t at position p = positions[t], each query and key head row x:
 *   y = (x / sqrt(mean(x^2) + eps)) * w     with w = q_norm_w / k_norm_w;
 *                                           a NULL weight leaves y = x
 *   pairs (i, j), i < rope_dims/2: (i, i + rope_dims/2), or with interleaved
 *   = 1 (2i, 2i + 1); a = p * inv_freq[i]; cos a, sin a good to 1e-6
 *   at any p:
 *     y'[i] = rope_mscale * (y[i] cos a - y[j] sin a)
 *     y'[j] = rope_mscale * (y[j] cos a + y[i] sin a)
 * dims from rope_dims on keep y.  q_out[t] = y' rounded to q_out_dtype.  Key
 * rows y' and value rows v_in are quantised per group as in qsa_prep, s =
 * fp16(max|.|/127), code = clamp(rint(./s), -127, 127), into pool cell
 * slots[t].  A group that holds a NaN, or a value beyond 127 * 65504, gets a
 * NaN or infinite scale, so that it reads back as NaN.
 * slots[t] = -1 marks a padding token: nothing of it is written, q_out included.
 * Another slot outside [0, cache_cells) is treated so too and sets
 * QSA_DEVERR_BAD_ID.  No two tokens may have the same slot.
 *
 * in_dtype (QSA_F32, QSA_F16 or QSA_BF16) is the type of q_in [ntok,
 * n_q_heads, head_dim] and k_in, v_in [ntok, n_kv_heads, head_dim]; heads are
 * contiguous, tokens are q_stride / k_stride / v_stride elements apart (so
 * the three may be views of one projection).  q_norm_w, k_norm_w fp32
 * [head_dim] or NULL; inv_freq fp32 [rope_dims/2] (non-negative and finite;
 * a context stretched by any rule comes in here), NULL with rope_dims 0;
 * positions, slots int32 [ntok], positions >= 0; q_out [ntok, n_q_heads,
 * head_dim] in q_out_dtype (QSA_F16 or QSA_BF16).
 * rope_dims is a multiple of head_dim/16 in [0, head_dim].  Inputs, weights,
 * q_out, kq and vq 16-byte aligned, token strides multiples of 16 bytes; ksc,
 * vsc 8-byte.  At most 32767 heads of each kind.
 */
typedef struct {
    int ntok, n_q_heads, n_kv_heads, head_dim, group, rope_dims, interleaved, cache_cells;
    int in_dtype, q_out_dtype;
    float eps, rope_mscale;
    const void *q_in, *k_in, *v_in;
    int64_t q_stride, k_stride, v_stride;
    const float *q_norm_w, *k_norm_w, *inv_freq;
    const int32_t *positions, *slots;
    void *q_out;
    int8_t *kq, *vq;
    uint16_t *ksc, *vsc;
    unsigned int *err;
} qsa_paged_prep_args;

/*
 * qsa_paged_gather -- cached rows read back as the values they stand for:
 *   k_out[i, h, d] = ksc[c, h, d/group] * kq[c, h, d], v_out likewise,
 * one rounding to out_dtype, for i < n_ids.  With page_table (then rows too),
 * c is cell ids[i] of row rows[i]; without, c = ids[i] is a pool cell (as
 * qsa_page_update's slots are).  ids[i] = -1 gives +0; an id < -1 or past the
 * row's table or the pool, a row outside [0, n_rows) or a table entry outside
 * the pool gives +0 and sets QSA_DEVERR_BAD_ID.
 *
 * kq, vq [cache_cells, n_kv_heads, head_dim] int8, ksc, vsc fp16 (one layer
 * of the pool); ids, rows int32 [n_ids]; page_table int32 [n_rows,
 * max_pages]; k_out, v_out [n_ids, n_kv_heads, head_dim] in out_dtype
 * (QSA_F32, QSA_F16 or QSA_BF16).  page_size is read only with page_table.
 * kq, vq, k_out, v_out 16-byte aligned; ksc, vsc 8-byte; the rest 4-byte.
 */
typedef struct {
    int n_ids, n_kv_heads, head_dim, group, cache_cells, page_size, n_rows, max_pages;
    int out_dtype;
    const int8_t *kq, *vq;
    const uint16_t *ksc, *vsc;
    const int32_t *ids, *rows, *page_table;
    void *k_out, *v_out;
    unsigned int *err;
} qsa_paged_gather_args;

/*
 * qsa_paged_attn -- attention of one new token per row of q over a whole
 * paged sequence.  Row t attends to cells 0 .. seq_lens[t]-1 of table row
 * rows[t] (rows NULL: table row t); several rows of q may read one sequence,
 * each with its own length (consecutive ones are read together where that
 * saves time: tokens of a draft window or of a chunk).  Query head h reads KV
 * head h / (n_q_heads / n_kv_heads):
 *   s_c = softmax_scale * sum_g ksc[c,g] * sum_{d in g} q[t,h,d] * kq[c,d]
 *   w_c = exp(s_c - max s);  O = sum w_c v_c / sum w_c,  v_c = vsc * vq
 *   out = O, or with a gate O / (1 + exp(-gate)), rounded to dtype
 *   lse[t,h] = max s + log(sum w_c)   (natural logarithm; lse may be NULL)
 * A row of length 0 gives out = +0 and lse = -inf; a NaN among a head's scores
 * gives NaN for both.  A length below 0 or above max_pages * page_size is cut
 * to that range, a table row outside [0, n_rows) counts as length 0, and a
 * table entry outside the pool leaves its page's cells out; each of these sets
 * QSA_DEVERR_BAD_ID.
 *
 * q, out [n_tokens, n_q_heads, head_dim] in dtype (QSA_F16 or QSA_BF16); gate
 * NULL or fp32 of that shape; lse fp32 [n_tokens, n_q_heads]; seq_lens, rows
 * int32 [n_tokens]; page_table int32 [n_rows, max_pages]; kq, vq, ksc, vsc one
 * layer of the pool.  workspace: device scratch of at least
 * qsa_paged_attn_workspace_bytes(n_q_heads, n_kv_heads, head_dim) bytes,
 * 256-byte aligned, overwritten; two calls that share one must not run
 * concurrently (graphs that replay on different streams need one each).
 * The work is divided over the cached cells of all rows, so the last bits of
 * a row's results may depend on the other rows' lengths and on max_pages (tables
 * of up to 512 cells of 128 dims or 256 of 256 are computed with more bits); the
 * same call gives the same bits.  Range: scores and sums are fp32; finite
 * scales of any size.  What a cell adds to a dim is kept to 2^-11 of itself (the
 * product of weight and V scale is one fp16 value, or two) or to 2^-24 of |code|
 * times the row's largest weight x V scale.
 * An infinite or NaN V scale makes the dims it scales NaN or infinite in the
 * rows that attend to its cell, and in no other.  An infinite or NaN K scale
 * (qsa_paged_prep leaves one for a group with such a value) makes the cell's
 * scores NaN, and with them out and lse of its KV head's query heads in the
 * rows that attend to it, and in no other.
 * Supported: n_q_heads a multiple of n_kv_heads, 1..16 query heads per KV
 * head; max_pages * page_size up to 2^30.  q, out, kq, vq 16-byte aligned; ksc, vsc, gate 8-byte; the rest 4-byte.
 */
typedef struct {
    int n_tokens, n_q_heads, n_kv_heads, head_dim, group, page_size, n_pages, n_rows, max_pages;
    int dtype;
    const void *q;
    const int8_t *kq, *vq;
    const uint16_t *ksc, *vsc;
    const int32_t *page_table, *seq_lens, *rows;
    float softmax_scale;
    const float *gate;
    void *out;
    float *lse;
    void *workspace;
    size_t workspace_bytes;
    unsigned int *err;
} qsa_paged_attn_args;

/* Bytes of workspace qsa_paged_attn needs (0 on a shape it does not support);
 * it depends on neither the batch nor the lengths. */
size_t qsa_paged_attn_workspace_bytes(int n_q_heads, int n_kv_heads, int head_dim);

/*
 * qsa_page_update -- the batch's next page table: forks, reorders, frees and
 * extends rows in one call.  New row r takes the pages of old row src[r]
 * (src NULL: r itself; -1: none, an empty row), then grows by n_new[r] tokens:
 *  - An old row that no new row takes is freed; one taken twice is forked.
 *  - Pages: if n_new[r] > 0 and the last page is partly filled and held more
 *    than once in the new table, the row gets a new page in its place and the
 *    filled cells are copied there, in all layers.  Then as many new pages as
 *    the row needs.  New pages are the pages that no new row holds, lowest
 *    number first, dealt to the rows in order.
 *  - Tokens: row r's new tokens are numbers off .. off + n_new[r] - 1 of the
 *    packed batch, off = sum of n_new of the rows before; slots[i] and
 *    positions[i] receive token i's pool cell and position.
 *  - A row grows whole or not at all.  It stays at its old length, and its
 *    tokens' slots and positions are -1, where its tokens do not fit into
 *    max_pages pages or into the n_slots entries of slots, or where it needs
 *    pages and the rows up to it have asked for more than were free.  Each
 *    sets QSA_DEVERR_NO_PAGES.
 * Outputs: page_table_out [rows, max_pages] (-1 behind a row's pages),
 * seq_lens_out [rows], refs [n_pages] (how often a page is held: 0 = free),
 * slots, positions [n_slots] (entries past the last token -1).
 * src outside [-1, n_rows_in), a length outside [0, max_pages * page_size], a
 * negative n_new and a table entry outside [0, n_pages) count as -1, the
 * nearest length, 0 and no page; each sets QSA_DEVERR_BAD_ID.
 * page_table_out and seq_lens_out may be page_table and seq_lens themselves
 * where src is NULL (then n_rows_in = n_rows), and must not overlap them
 * otherwise.  workspace: at least qsa_pages_workspace_bytes(n_rows, n_pages)
 * bytes, 256-byte aligned, overwritten; not to be shared by concurrent calls.
 * kq, vq, ksc, vsc: all layers of the pool.  kq, vq, ksc, vsc 16-byte
 * aligned, the rest 4-byte.
 */
typedef struct {
    int n_rows_in, n_rows, max_pages, n_layers, n_pages, page_size, n_kv_heads, head_dim, group, n_slots;
    const int32_t *page_table, *seq_lens, *src, *n_new;
    int8_t *kq, *vq;
    uint16_t *ksc, *vsc;
    int32_t *page_table_out, *seq_lens_out, *refs, *slots, *positions;
    void *workspace;
    size_t workspace_bytes;
    unsigned int *err;
} qsa_page_update_args;

/*
 * qsa_page_compact -- moves the held pages to the lowest page numbers.  With
 * L the number of pages that some row holds: each held page below L stays,
 * and the i-th free page below L receives the contents (all layers) of the
 * i-th held page at or above L.  Outputs: page_table_out (the rows' pages by
 * their new numbers, -1 behind them), refs [n_pages] by the new numbers,
 * page_map [n_pages] (a page's new number; -1 for a free one) and n_live [1] =
 * L.  Lengths do not change.  page_table_out may be page_table itself.
 * Lengths and entries out of range are treated as in qsa_page_update.
 * workspace and alignment as there.
 */
typedef struct {
    int n_rows, max_pages, n_layers, n_pages, page_size, n_kv_heads, head_dim, group;
    const int32_t *page_table, *seq_lens;
    int8_t *kq, *vq;
    uint16_t *ksc, *vsc;
    int32_t *page_table_out, *refs, *page_map, *n_live;
    void *workspace;
    size_t workspace_bytes;
    unsigned int *err;
} qsa_page_compact_args;

/* Bytes of workspace qsa_page_update and qsa_page_compact need (0 on bad input). */
size_t qsa_pages_workspace_bytes(int n_rows, int n_pages);

qsa_status qsa_paged_prep(const qsa_paged_prep_args *args, void *stream);
qsa_status qsa_paged_gather(const qsa_paged_gather_args *args, void *stream);
qsa_status qsa_paged_attn(const qsa_paged_attn_args *args, void *stream);
qsa_status qsa_page_update(const qsa_page_update_args *args, void *stream);
qsa_status qsa_page_compact(const qsa_page_compact_args *args, void *stream);

/*
 * qsa_check_word -- the pages have no counterpart to this call; it serves the
 * device bounds-check build of the library.  Built with QSA_CHECK=1
 * (libqsa_check.so), every kernel tests the index of its global-memory
 * accesses against the size of its buffer as the call's arguments define
 * it; an index outside sets bit 0 of a device word and that access is
 * skipped (nothing traps).  This call ORs the words of every kernel file
 * into *out (a host pointer) and clears them; it synchronises with the
 * device.  The release build returns QSA_ERR_UNSUPPORTED and writes 0.
 */
qsa_status qsa_check_word(unsigned int *out);

/* Static description of a status code. */
const char *qsa_status_str(qsa_status s);
/* Message of the last QSA_ERR_* returned on this host thread ("" if none). */
const char *qsa_last_error(void);
/* QSA_ABI_VERSION of the built library. */
int qsa_abi_version(void);

#ifdef __cplusplus
}
#endif

#endif /* QSA_H */
