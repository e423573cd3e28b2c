/*
 * hysparse.h -- C ABI of libhysparse.so, the B200 (sm_100a) hot path of the
 * HySparse hybrid block.
 *
 * Method (HySparse: A Hybrid Sparse Attention Architecture with Oracle Token
 * Selection and KV Cache Sharing, abstract; intelliparadigm write-up, sections
 * 2.1 "hybrid block", 2.2 "dual-branch sparse attention", 3.1 "cross-layer
 * sharing"): a full causal attention layer is followed by N sparse layers.
 * The full layer is the only writer of the KV cache and the "oracle" of token
 * importance; each sparse layer reuses its KV cache and its top-k key set and
 * mixes a global branch over those keys with a 128-token local window through
 * a sigmoid gate.
 *
 * Notation used below:
 *   B batch, Lq query rows, Lkv cache length, Hq query heads, Hkv KV heads,
 *   d head dim, G = Hq / Hkv (query head h reads KV head h / G),
 *   pos(i) = Lkv - Lq + i  (causal, bottom-right aligned: row i sees keys
 *   0 .. pos(i); decode is Lq = 1 with the new token at Lkv - 1, or at
 *   kv_len[b] - 1 in hysparse_block_varlen / hysparse_block_paged).
 *
 * Layouts (row-major, contiguous, every pointer 16-byte aligned):
 *   q, q_sparse[n], out, out_sparse[n]  [B][Lq][Hq][d]   (dtype of the shape)
 *   k, v                               [B][Lkv][Hkv][d]  (dtype of the shape)
 *   lse                                [B][Hq][Lq]        float, natural log
 *   scores (one row chunk)             [B][Hkv][row_count][ld_scores] float
 *   idx                                [B][Hkv][Lq][topk] int32
 *   gate_logit                         [B][Lq][Hq]        float
 *   k_win, v_win (own-window calls)    [B][lwin][Hkv][d]  (dtype of the shape),
 *                                      row r = cache position Lkv - lwin + r
 *
 * Conventions for every entry point:
 *   - All device buffers are owned by the caller (e.g. allocated by PyTorch).
 *     The library allocates no device or host memory and keeps no state
 *     between calls beyond one-time kernel attributes and each device's SM
 *     count (read once, to size grids); scratch lives in the caller's
 *     workspace `ws`.
 *   - Work is enqueued on `stream` and is asynchronous; nothing synchronises
 *     except hysparse_workspace_status.
 *   - Arguments are checked on the host before anything is launched; a
 *     non-zero return means nothing was launched and no output was touched.
 *     A failed launch returns HS_ERR_CUDA.
 *   - Supported: dtype HS_F32 with d in {64, 128}; dtype HS_BF16 with
 *     d = 128; Hq % Hkv == 0; 1 <= Hq / Hkv <= 32; Lq <= Lkv;
 *     1 <= topk <= 4096; 1 <= window <= 1024.
 *   - NaN or Inf inputs give undefined (but memory-safe) results.
 *   - One GPU per process: each kernel's one-time set-up (its shared-memory
 *     attribute) runs on the first call, on that call's device, and is not
 *     guarded against a concurrent first call; make the first call of each
 *     kind from one host thread.  Later calls may come from any thread.
 */
#ifndef HYSPARSE_H
#define HYSPARSE_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* Same type as cudaStream_t / CUstream; NULL is the legacy default stream. */
typedef struct CUstream_st *hs_stream_t;

typedef enum {
    HS_OK = 0,
    HS_ERR_INVALID_ARG = 1,   /* null or misaligned pointer, bad size, bad shape; (device) a
                                 cache length outside [1, Lkv] (mixed-length / paged decode) */
    HS_ERR_UNSUPPORTED = 2,   /* valid but not implemented (dtype/d combination) */
    HS_ERR_WORKSPACE = 3,     /* ws_bytes below hysparse_workspace_size() */
    HS_ERR_CUDA = 4,          /* a CUDA call or kernel launch failed */
    HS_ERR_INVALID_INDEX = 5, /* (device) an index list entry outside [-1, pos], or a block
                                 table entry outside the page pool (paged decode) */
    HS_ERR_TIMEOUT = 6        /* (device) a bounded wait inside a kernel gave up */
} hs_status;

/* HS_E4M3 is a page pool's type only (hs_paged_cache). */
typedef enum { HS_F32 = 0, HS_BF16 = 1, HS_E4M3 = 2 } hs_dtype;

typedef struct {
    int B, Lq, Lkv, Hq, Hkv, d;
    int dtype;    /* hs_dtype */
    float scale;  /* softmax scale on q.k; <= 0 selects 1/sqrt(d) */
} hs_shape;

/* Bytes of device workspace that hysparse_full_attn_scores,
 * hysparse_sparse_attn and hysparse_block need for this shape.  `row_chunk`
 * is the number of query rows hysparse_block scores at a time (<= 0: all Lq
 * rows); the other arguments are those of the calls.  Returns 0 for an
 * invalid shape.  The first 256 bytes of a workspace hold a status word (see
 * hysparse_workspace_status); zero them once before first use (the calls
 * only ever OR error bits into it). */
size_t hysparse_workspace_size(const hs_shape *shape, int topk, int window, int n_sparse,
                               int row_chunk);

/* The full attention layer of the hybrid block, restricted to the query rows
 * [row_begin, row_begin + row_count) of every batch element.
 *
 * Computes (HySparse abstract; write-up section 2.1, the full layer as the
 * token-importance oracle; the score is the group sum of the softmax
 * probabilities over the query heads that share a KV head):
 *   out[b,i,h]  = sum_{j <= pos(i)} softmax_j(scale * q[b,i,h].k[b,j,h/G]) v[b,j,h/G]
 *   lse[b,h,i]  = ln sum_{j <= pos(i)} exp(scale * q[b,i,h].k[b,j,h/G])
 *   scores[b,g,i-row_begin,j] = sum_{h : h/G = g} exp(scale * q.k_j - lse[b,h,i])
 *                              for j <= pos(i); entries j > pos(i) are left
 *                              unspecified and are never read by hysparse_topk.
 * `scores` may be NULL (forward pass only); otherwise ld_scores >= Lkv.
 * Only out/lse entries of the listed rows are written.  If a bounded wait
 * inside a kernel gives up (HS_ERR_TIMEOUT in the status word), the lse
 * entries of the rows and heads it could not finish are set to NaN and their
 * out and scores entries are undefined.
 * Decode (Lq == 1) uses split-K over the cache and needs `ws`.
 * Errors: HS_ERR_INVALID_ARG, HS_ERR_UNSUPPORTED, HS_ERR_WORKSPACE, HS_ERR_CUDA. */
int hysparse_full_attn_scores(const hs_shape *shape, const void *q, const void *k, const void *v,
                              void *out, float *lse, float *scores, long long ld_scores,
                              int row_begin, int row_count, void *ws, size_t ws_bytes,
                              hs_stream_t stream);

/* Per-row top-k over one chunk of importance rows (write-up section 2.2: the
 * global branch attends over the full layer's TopK indices; section 3.1: one
 * index set per row is shared by the following sparse layers).
 * For every (b, g, i) with i in [row_begin, row_begin + row_count): the
 * `topk` keys j <= pos(i) with the largest scores[b,g,i-row_begin,j], ties
 * going to the lower j.  A row with pos(i) + 1 <= topk takes all its keys.
 * The set is written to idx[b,g,i,:] in ascending key order, padded with -1.
 * Scores must be >= 0 (importance values are).  Exact and deterministic.
 * Errors: HS_ERR_INVALID_ARG, HS_ERR_CUDA. */
int hysparse_topk(const hs_shape *shape, const float *scores, long long ld_scores, int row_begin,
                  int row_count, int topk, int32_t *idx, hs_stream_t stream);

/* One sparse layer (write-up section 2.2, dual-branch sparse attention;
 * section 3.1, KV cache reuse: reads the full layer's k and v, writes no KV):
 *   Og = softmax attention of q[b,i,h] over { k_j : j in idx[b,h/G,i,:], j != -1 }
 *   Ol = softmax attention of q[b,i,h] over { k_j : max(0, pos(i)-window+1) <= j <= pos(i) }
 *   out = sigmoid(gate_logit[b,i,h]) * Og + (1 - sigmoid(gate_logit[b,i,h])) * Ol
 * The two branches may share keys; each has its own softmax.  An index list
 * with no valid entry gives Og = 0.  Index lists must hold distinct keys in
 * [0, pos(i)] (any order) padded with -1; entries outside [-1, pos(i)] are
 * skipped and reported as HS_ERR_INVALID_INDEX through the workspace status
 * word.  out_global / out_local (nullable) receive Og and Ol.
 * Decode (Lq == 1) uses split-K and needs `ws`.
 * Errors: HS_ERR_INVALID_ARG, HS_ERR_UNSUPPORTED, HS_ERR_WORKSPACE, HS_ERR_CUDA. */
int hysparse_sparse_attn(const hs_shape *shape, const void *q, const void *k, const void *v,
                         const int32_t *idx, int topk, const float *gate_logit, int window,
                         void *out, void *out_global, void *out_local, void *ws, size_t ws_bytes,
                         hs_stream_t stream);

/* One sparse layer whose local branch reads the layer's own window K/V
 * (write-up section 2.2: the global branch computes on the KV cache that the
 * full layer shares, while the local branch maintains its own 128-token
 * sliding window).  Same computation, arguments and errors as
 * hysparse_sparse_attn, except that the local branch's keys and values come
 * from k_win / v_win instead of k / v:
 *   Ol = softmax attention of q[b,i,h] over
 *        { k_win[b, j - (Lkv - lwin)] : max(0, pos(i)-window+1) <= j <= pos(i) }
 *   with values v_win at the same rows.
 * k_win, v_win  [B][lwin][Hkv][d] (dtype of the shape, caller-owned, 16-byte
 * aligned): the layer's window keys and values for cache positions
 * Lkv - lwin .. Lkv - 1 (lwin = Lkv for a prefill that projects every
 * position; lwin = window - 1 + Lq, or any length that reaches back far
 * enough, for decode against a ring of the last tokens laid out in position
 * order).  1 <= lwin <= Lkv and Lkv - lwin <= max(0, Lkv - Lq - window + 1)
 * (the buffer covers the first row's window), else HS_ERR_INVALID_ARG.
 * The global branch still reads k and v with idx.  Passing k_win = k,
 * v_win = v, lwin = Lkv gives hysparse_sparse_attn's result, bit for bit
 * when Hq / Hkv is even (with an odd ratio the plain call may choose a
 * kernel that this one does not, and the two agree to rounding). */
int hysparse_sparse_attn_own_window(const hs_shape *shape, const void *q, const void *k, const void *v,
                                    const void *k_win, const void *v_win, int lwin, const int32_t *idx, int topk,
                                    const float *gate_logit, int window, void *out, void *out_global,
                                    void *out_local, void *ws, size_t ws_bytes, hs_stream_t stream);

/* A whole hybrid block (HySparse abstract: one full layer interleaved with
 * several sparse layers; write-up section 3.1: index sharing and cache reuse):
 * the full layer over all rows (out_full, and its LSE into `lse` when not
 * NULL), its importance scores and top-k (scored `row_chunk` rows at a time
 * inside `ws`), then n_sparse sparse layers, each with its own queries and
 * gate logits, all reusing k, v and the one index set.
 * q_sparse, gate_logit and out_sparse are HOST arrays of n_sparse DEVICE
 * pointers.  idx_out (nullable) receives the index set [B][Hkv][Lq][topk];
 * when NULL it is kept in `ws`.  In decode (Lq == 1) the sparse layers run
 * as one gather launch per group of up to 16 (they share the index set and
 * the cache, so each row is read once per group); the outputs are those of
 * one hysparse_sparse_attn call per layer, bit for bit.
 * Errors: as the calls it makes. */
int hysparse_block(const hs_shape *shape, const void *q_full, const void *k, const void *v,
                   void *out_full, float *lse, int n_sparse, const void *const *q_sparse,
                   const float *const *gate_logit, void *const *out_sparse, int topk, int window,
                   int32_t *idx_out, int row_chunk, void *ws, size_t ws_bytes, hs_stream_t stream);

/* hysparse_block with every sparse layer reading its window branch from its
 * own window K/V (write-up section 2.2; the variant of
 * hysparse_sparse_attn_own_window): k_win and v_win are HOST arrays of
 * n_sparse DEVICE pointers, layer n's [B][lwin][Hkv][d] buffers for cache
 * positions Lkv - lwin .. Lkv - 1 (layouts and limits as in
 * hysparse_sparse_attn_own_window, the same lwin for every layer).  The full
 * layer, the index set and the global branches are hysparse_block's; the
 * outputs equal hysparse_sparse_attn_own_window per layer on the block's
 * index set.  Fixed-length caches only.  Errors: as hysparse_block, and
 * HS_ERR_INVALID_ARG for a missing, misaligned or too short window buffer. */
int hysparse_block_own_window(const hs_shape *shape, const void *q_full, const void *k, const void *v,
                              void *out_full, float *lse, int n_sparse, const void *const *q_sparse,
                              const float *const *gate_logit, const void *const *k_win, const void *const *v_win,
                              int lwin, void *const *out_sparse, int topk, int window, int32_t *idx_out,
                              int row_chunk, void *ws, size_t ws_bytes, hs_stream_t stream);

/* One decode step of the hybrid block over a batch whose sequences have
 * caches of different lengths (serving: every sequence decodes one token,
 * each at its own position).  Same computation, arguments and layouts as
 * hysparse_block with Lq == 1, plus
 *   kv_len  DEVICE array of B int32, 1 <= kv_len[b] <= Lkv: sequence b's
 *           cache is k[b, 0:kv_len[b]], v[b, 0:kv_len[b]] (the Lkv-row
 *           buffers hold it at their start; rows past it are never read)
 *           and its new query sits at position kv_len[b] - 1, so its full
 *           layer, scores, top-k and window branch see exactly those keys.
 * Requires Lq == 1 and the bf16, d = 128 path (else HS_ERR_UNSUPPORTED);
 * kv_len must be 4-byte aligned.  The lengths live on the device, so a value
 * outside [1, Lkv] is found there: it is clamped (nothing outside the cache
 * is read) and HS_ERR_INVALID_ARG is recorded in the workspace status word
 * (hysparse_workspace_status).  The whole batch is one row chunk.
 * Errors: as hysparse_block. */
int hysparse_block_varlen(const hs_shape *shape, const int32_t *kv_len, const void *q_full,
                          const void *k, const void *v, void *out_full, float *lse, int n_sparse,
                          const void *const *q_sparse, const float *const *gate_logit,
                          void *const *out_sparse, int topk, int window, int32_t *idx_out,
                          void *ws, size_t ws_bytes, hs_stream_t stream);

/* hysparse_block_varlen over paged caches: k_pages and v_pages are pools of
 * num_pages pages, each page_size rows of [Hkv][d] ([num_pages][page_size]
 * [Hkv][d], bf16), and sequence b's key j is row j % page_size of page
 * block_table[b * max_pages + j / page_size] (block_table: DEVICE int32,
 * B rows of max_pages entries, 4-byte aligned).  Only the entries that cover
 * keys 0 .. kv_len[b]-1 are read.  page_size is a power of two in
 * [1, 65536]; max_pages * page_size >= Lkv (shape->Lkv is the longest cache
 * any sequence may have) and num_pages * page_size < 2^31.  A table entry
 * outside [0, num_pages) is found on the device: the key is dropped and
 * HS_ERR_INVALID_INDEX recorded in the workspace status word.  The
 * workspace is the one hysparse_workspace_size gives for the shape.
 * Errors: as hysparse_block_varlen, HS_ERR_INVALID_ARG for the paging
 * arguments. */
int hysparse_block_paged(const hs_shape *shape, const int32_t *kv_len, const int32_t *block_table,
                         int page_size, int max_pages, int num_pages, const void *q_full,
                         const void *k_pages, const void *v_pages, void *out_full, float *lse,
                         int n_sparse, const void *const *q_sparse, const float *const *gate_logit,
                         void *const *out_sparse, int topk, int window, int32_t *idx_out, void *ws,
                         size_t ws_bytes, hs_stream_t stream);

/* ------------------------------------------------------------------------
 * Ragged batches and paged caches: the calls below serve prompts and chunks
 * of sequences of different lengths, packed row after row ([T][H][d], no
 * padding between sequences), next to the decode calls above, which read the
 * same pages.  (The pages of the method have no counterpart; this is the
 * serving side of their prefill / decode split.)
 *
 *   - Row strides: ld_x is the number of elements from one packed row of x to
 *     the next (>= H * d, a multiple of 16 bytes), so q, k and v may be
 *     slices of one projection's output; each row's [H][d] is contiguous.
 *   - cu_rows (DEVICE int32, B + 1 entries, ascending): rows cu_rows[b] ..
 *     cu_rows[b+1]-1 are sequence b's (none when equal).  Rows before
 *     cu_rows[0] or from cu_rows[B] on belong to no sequence: they are not
 *     read into any result and their outputs are left as they were.
 *   - The values of device arrays are checked on the device: an entry that
 *     would leave the caller's buffers is skipped or clamped and recorded in
 *     the workspace status word (HS_ERR_INVALID_ARG for lengths and
 *     positions, HS_ERR_INVALID_INDEX for block table entries), when the call
 *     has a workspace. */

/* A paged cache and the batch over it.  k_pages and v_pages are pools
 * [num_pages][page_size][Hkv][d] of cache_dtype; sequence b's position j is
 * row j % page_size of page block_table[b * max_pages + j / page_size].
 * page_size is a power of two in [1, 65536]; num_pages * page_size and
 * max_pages * page_size are below 2^31.
 * HS_E4M3 pools hold 8-bit floats (4 exponent bits, 3 mantissa bits) with one
 * scale byte per row and head in k_scale / v_scale [num_pages][Hkv][page_size]:
 * an element stands for code * 2^(byte - 127), bytes 1 to 254.  With bytes 3 to
 * 246 every such value is a bf16 number exactly.  Bytes 1 and 2 (rows whose
 * largest magnitude is at most 448 * 2^-125): values are rounded to multiples of
 * 2^-133 where rows are widened to bf16 (hysparse_cache_read to bf16, attention
 * of many rows).
 * Bytes from 247 on: codes that pass the largest float become infinity where rows
 * are widened to bf16 or fp32; attention of few rows takes them as the numbers
 * they stand for.  Byte 255 marks a row of NaN, whose codes are all NaN (0x7f or
 * 0xff, which no other row holds). */
typedef struct {
    const int32_t *cu_rows;       /* DEVICE [B + 1] */
    const int32_t *kv_len;        /* DEVICE [B]: positions in each cache, the new rows' among them */
    const int32_t *block_table;   /* DEVICE [B][max_pages] */
    int B, page_size, max_pages, num_pages;
    int cache_dtype;              /* hs_dtype */
    void *k_pages, *v_pages;
    uint8_t *k_scale, *v_scale;   /* HS_E4M3 only */
} hs_paged_cache;

/* Flags of the rotary calls. */
#define HS_ROPE_INTERLEAVED 1     /* pairs (2i, 2i+1); without it (i, i + rot/2) */
#define HS_ROPE_INVERSE 2         /* turn back: the transposed rotation, which is the gradient's */

/* Rotary positions: for every packed row t, head and pair i < rot/2, with
 * angle a = positions[t] * inv_freq[i] (in 64 bits):
 *   (x, y) -> factor * (x cos a - y sin a, y cos a + x sin a),
 * elements from rot on are copied.  q has Hq heads and k Hkv (k may be left
 * out: Hkv = 0).  dtype HS_F32 or HS_BF16; d a multiple of 8 up to 512; rot
 * even, 2 <= rot <= d; positions DEVICE int32 [T] (any sign), inv_freq DEVICE
 * double [rot/2].  out_q / out_k may be q / k themselves (same stride), else
 * they must not overlap the inputs.
 * Errors: HS_ERR_INVALID_ARG, HS_ERR_UNSUPPORTED, HS_ERR_CUDA. */
int hysparse_rope(int T, int Hq, int Hkv, int d, int dtype, const void *q, long long ld_q, const void *k,
                  long long ld_k, const int32_t *positions, const double *inv_freq, int rot, int flags, float factor,
                  void *out_q, long long ld_oq, void *out_k, long long ld_ok, hs_stream_t stream);

/* Write new keys and values into a paged cache: packed row r of sequence b
 * (of its n = cu_rows[b+1] - cu_rows[b] new rows) goes to position
 * kv_len[b] - n + (r - cu_rows[b]).  With inv_freq (else NULL) the keys are
 * turned as by hysparse_rope at those positions on the way, without a
 * rounding in between (flags: HS_ROPE_INTERLEAVED or 0).
 * k, v [T][Hkv][d] of dtype HS_F32 or HS_BF16; d a multiple of 16 up to 256.
 * HS_E4M3 pools get, per row and head, the smallest power of two 2^e with
 * max|x| <= 448 * 2^e (2^0 for a row of zeros, e >= -126) as byte e + 127 and
 * the nearest 8-bit floats (ties to even) of x / 2^e; a row with a
 * NaN becomes a row of NaN, and an infinity 448 * 2^120 (byte 247: see
 * hs_paged_cache).  Other pool types get x rounded once.  Two rows of one call must not share a pool row.
 * ws (nullable) is only used for its status word.
 * Errors: HS_ERR_INVALID_ARG, HS_ERR_UNSUPPORTED, HS_ERR_CUDA. */
int hysparse_cache_write(const hs_paged_cache *cache, int T, int Hkv, int d, int dtype, const void *k, long long ld_k,
                         const void *v, long long ld_v, const double *inv_freq, int rot, int flags, float factor,
                         void *ws, hs_stream_t stream);

/* Read rows of a paged cache back, widened and packed: row cu_rows[b] + i of
 * k, v ([total][Hkv][d] of dtype, contiguous) is position start[b] + i of
 * sequence b (start NULL: from 0 on).  cache->kv_len is not read.  A position
 * or page outside the cache leaves its output row as it was and is recorded.
 * ws (nullable) is only used for its status word.
 * Errors: HS_ERR_INVALID_ARG, HS_ERR_UNSUPPORTED, HS_ERR_CUDA. */
int hysparse_cache_read(const hs_paged_cache *cache, const int32_t *start, int total, int Hkv, int d, int dtype,
                        void *k, void *v, void *ws, hs_stream_t stream);

/* Bytes of workspace that the two attention calls below need for these
 * arguments (0 for invalid ones): 256 for the status word, and where few rows
 * face many keys, the partial results of the pieces their keys are split
 * into.  max_len 0: enough for any length.  At most 94 MB, which serve every
 * call; fewer rows can need more than many (their keys are cut into more
 * pieces), so a loop over batches of different sizes keeps one of 94 MB.
 * A workspace belongs to one call at a time: calls (or replayed graphs) that
 * may overlap on the GPU need one each.
 * Status word as in hysparse_workspace_size. */
size_t hysparse_ragged_workspace_size(int B, int T, int Hq, int Hkv, int d, int max_q, int max_len);

/* Causal attention over whole packed prompts: with sequence b's rows
 * s = cu_rows[b] .. cu_rows[b+1]-1 of q [T][Hq][d], k and v [T][Hkv][d]
 * (bf16, d = 128, Hq / Hkv <= 32):
 *   out[t,h] = sum_{s <= j <= t} softmax_j(scale * q[t,h].k[j,h/G]) v[j,h/G]
 *   lse[h,t] = ln sum_{s <= j <= t} exp(scale * q[t,h].k[j,h/G])
 * out [T][Hq][d] bf16 and lse [Hq][T] float, contiguous.  scale <= 0 selects
 * 1/sqrt(d).  max_len: the longest sequence (0: T); a longer one is recorded
 * as HS_ERR_INVALID_ARG and its rows' results are undefined.  Rows of no
 * sequence are left as they were.  Probabilities are rounded to bf16 before
 * they meet v; sums are held in fp32.  A score that is NaN or +infinity makes
 * its row's out and lse NaN.  A NaN or infinity in v[j] reaches that column
 * of the rows that see j (8-bit pools: every column), and may reach it in
 * rows of the same sequence up to 127 positions before (their probability of
 * 0 times NaN); no other row.
 * out must not overlap q, k or v.  A wait that gives up
 * (HS_ERR_TIMEOUT) marks its rows' lse with NaN.
 * ws: 256-byte aligned, hysparse_ragged_workspace_size(B, T, Hq, Hkv, d,
 * max_len, max_len) bytes.
 * Errors: HS_ERR_INVALID_ARG, HS_ERR_UNSUPPORTED, HS_ERR_WORKSPACE, HS_ERR_CUDA. */
int hysparse_packed_attn(const int32_t *cu_rows, int B, int T, int Hq, int Hkv, int d, int max_len, float scale,
                         const void *q, long long ld_q, const void *k, long long ld_k, const void *v, long long ld_v,
                         void *out, float *lse, void *ws, size_t ws_bytes, hs_stream_t stream);

/* Attention of a chunk of new tokens over a paged cache that holds them
 * already (hysparse_cache_write): sequence b's n = cu_rows[b+1] - cu_rows[b]
 * rows of q [T][Hq][d] (bf16, d = 128, Hq / Hkv <= 32) are its cache's last
 * positions; row i sees positions 0 .. kv_len[b] - n + i.  One row a sequence
 * is a decode step.  out, lse, scale, max_q (most rows of a sequence; 0: T)
 * as in hysparse_packed_attn; a row that sees nothing (kv_len[b] < n) gets
 * zeros and lse = -inf.  max_len: the longest cache (0: max_pages *
 * page_size); it only plans the work, longer ones are still right.
 * Pools of HS_BF16 or HS_E4M3.  Few rows a sequence over HS_E4M3: each product
 * of a probability and its value row's scale is off by 2^-11 of itself or 2^-32
 * of the row's largest such product (rows of zeros left out), whichever is more.
 * Only the table entries that cover
 * positions 0 .. kv_len[b]-1 are read, and nothing that lies behind
 * kv_len[b] in the last page reaches a result (NaN included).  A page outside
 * the pool drops its keys.  ws: 256-byte aligned,
 * hysparse_ragged_workspace_size(B, T, Hq, Hkv, d, max_q, the longest cache)
 * bytes.
 * Errors: as hysparse_packed_attn; HS_ERR_UNSUPPORTED for fp32 pools. */
int hysparse_chunk_attn_paged(const hs_paged_cache *cache, int T, int Hq, int Hkv, int d, int max_q, int max_len,
                              float scale, const void *q, long long ld_q, void *out, float *lse, void *ws,
                              size_t ws_bytes, hs_stream_t stream);

/* Allocation-free variant of hysparse_full_attn_scores (the pages have no
 * counterpart; this is a deployment convenience).  Same computation,
 * arguments, layouts and errors, but no workspace: its scratch lives in a
 * fixed 16 MiB device array inside the library, so callers that may not
 * allocate device memory -- a serving process that has frozen its memory
 * pool, or a plug-in host that only lends input and output buffers -- can
 * still run the full layer.  Every GPU that loads the library holds that
 * array until the process exits.
 *   - Scratch needed: 256 bytes (status word) + 8*B*Hq*Lq bytes of per-row
 *     softmax statistics, rounded up to 256; decode-shaped calls (Lq == 1,
 *     bf16) also keep their split-K partials and logit stash there, a
 *     further 4*B*Hq*Lkv + 520*B*Hq*ceil(Lkv/1024) + 768 bytes rounded up
 *     to 256.  Shapes needing more than 16 MiB return HS_ERR_WORKSPACE
 *     before anything runs (score smaller row chunks, decode smaller
 *     batches, or use hysparse_full_attn_scores).
 *   - Calls no cudaMalloc/cudaFree and allocates nothing; the caller still
 *     provides q, k, v, out, lse and (optionally) scores.
 *   - The array's device address is looked up on the first call on each
 *     device (the current device, which `stream` must belong to) and kept
 *     for the life of the process; make that first call before any stream
 *     capture, and do not use this entry point after cudaDeviceReset in the
 *     same process (the array may move).
 *   - All calls share the one array and each zeroes its status word on
 *     `stream`: calls that can overlap on the GPU (other streams, other host
 *     threads without ordering) race on it and must be serialised by the
 *     caller.
 *   - The status word cannot be read through this API.  A bounded wait that
 *     gives up inside a tensor-core kernel (HS_ERR_TIMEOUT elsewhere) leaves
 *     NaN in the lse entries of the rows and heads it could not finish; the
 *     out and scores entries of those rows are then undefined. */
int hysparse_full_attn_scores_noalloc(const hs_shape *shape, const void *q, const void *k,
                                      const void *v, void *out, float *lse, float *scores,
                                      long long ld_scores, int row_begin, int row_count,
                                      hs_stream_t stream);

/* Synchronises `stream`, reads the workspace status word (HS_OK or the
 * lowest-numbered device error recorded since it was last cleared), clears
 * it and returns it.  Returns HS_ERR_CUDA if the synchronisation fails. */
int hysparse_workspace_status(void *ws, hs_stream_t stream);

/* Diagnostic (no counterpart on the pages): L2 read bandwidth probe, the
 * denominator for kernels whose reads are served from L2 (the prefill sparse
 * layers gather K/V rows from a cache that fits in L2).  Reads the DEVICE
 * buffer `buf` (`bytes`, a multiple of 256 and >= 4096, 256-byte aligned; the
 * caller makes it L2-resident, e.g. by one untimed call first) with `blocks`
 * CTAs of 512 threads on `stream`, using L2-only loads:
 *   mode 0: streaming 16-byte reads, `passes` times over the buffer;
 *   mode 1: whole 256-byte rows at hashed positions, passes * bytes / 256
 *           rows (the access pattern of the sparse layers' row gather).
 *   modes 2 and 3: as 0 and 1, but through cp.async into shared memory
 *           (one CTA of 7 warps per SM is the intended `blocks`: the path
 *           and occupancy of the row-gather kernel); bytes >= 65536.
 * Either way passes * bytes bytes are read; time the call with events on
 * `stream`.  `sink` is a DEVICE array of at least `blocks` 64-bit words that
 * receives an XOR of what each CTA read (it keeps the loads live).
 * Errors: HS_ERR_INVALID_ARG, HS_ERR_CUDA. */
int hysparse_probe_l2_read(const void *buf, size_t bytes, int passes, int mode, int blocks,
                           unsigned long long *sink, hs_stream_t stream);

/* Diagnostic: number of CUDA kernels this library has launched in this
 * process so far (counted on the host at each launch). */
unsigned long long hysparse_launch_count(void);

/* Static text for a status code. */
const char *hysparse_status_string(int status);

/* Library version, e.g. "hysparse-b200 0.1". */
const char *hysparse_version(void);

#ifdef __cplusplus
}
#endif

#endif /* HYSPARSE_H */
