/*
 * tf_paged.h -- attention over a paged KV cache on NVIDIA B200 (sm_100a).
 *
 * Keys and values live in fixed pages of `page_size` positions drawn from
 * one shared pool; every stream reads its positions through its own row of
 * a page table.  The library provides the row write that copies new K/V rows
 * into their pages, and grouped-query attention for single-row decode,
 * draft-verify windows (causal inside the window) and chunked prompt rows.
 *
 * Sources (the TensorFold pull-request pages this library follows):
 *  - TensorFold #1620, "Kolibri-1's full layers take their K/V from pages of
 *    the core pool", opening comment:
 *      * "Pages of 512 positions": the pool and its fixed page size;
 *      * "Writes": new K/V rows are copied into the pages (tf_kv_put_rows);
 *      * "Reads": prompt rows, decode and drafted verify read keys through a
 *        page table given in the call's stream order (the tf_paged_attn_*
 *        calls);
 *    and its later comment on per-tile page lookup: a tile's page is looked
 *    up once per tile, and paging leaves the result bits unchanged.
 *  - TensorFold #2730, "an eight-row verify window", section "What this
 *    changes": a verify window is the pending token plus up to seven drafts.
 *
 * Conventions shared by every call
 * --------------------------------
 *  Layouts (all row-major, element counts, no padding):
 *    K pool, V pool  bf16  [n_pages][n_kv_heads][page_size][head_dim]  device
 *    table           int32 [n_streams][table_stride]                   device
 *    lens            int32 [n_streams]                                  device
 *    q               bf16  [n_streams][rows][n_q_heads][head_dim]       device
 *    out             fp32  [n_streams][rows][n_q_heads][head_dim]       device
 *    k_rows, v_rows  bf16  [n_streams][rows][n_kv_heads][head_dim]      device
 *
 *  (pools, q, out and rows 16-byte aligned; every array of 32-bit values
 *  4-byte aligned)
 *
 *  lens[s] counts the positions of stream s AFTER this step's rows are
 *  written.  Window row r (0 <= r < rows) sits at position
 *  lens[s] - rows + r and attends to positions 0 .. lens[s] - rows + r.
 *  Position j of stream s lives in pool page table[s][j / page_size], slot
 *  j % page_size.  Query head h reads KV head h / (n_q_heads / n_kv_heads).
 *
 *  The output is softmax(scale * q . k) weighted sum of v, accumulated in
 *  fp32 from bf16 inputs; scale is any finite number (TF_EINVAL otherwise),
 *  zero and negative ones included.  Which pool pages hold a stream's
 *  positions never changes a bit of the result: the arithmetic depends only
 *  on positions, lens, rows and the host arguments.
 *
 *  Ownership: the caller owns every buffer.  The library allocates nothing
 *  and keeps no state between calls; each call enqueues kernels on the
 *  caller's CUDA stream (`stream` is a cudaStream_t; NULL is the legacy
 *  default stream) and returns without waiting.
 *
 *  Errors: every call checks its host arguments before enqueueing anything
 *  and returns a TF_* status; on a non-zero status nothing was enqueued
 *  (TF_ECUDA: a launch failed).  lens and table are device data and are
 *  checked on the device: a stream whose length is outside
 *  [rows, min(max_len, table_stride * page_size)] is skipped and its
 *  outputs are set to NaN; a page id outside [0, n_pages) is never read.
 *  Such events set bits in the workspace's status word (tf_workspace_status).
 *  Table entries past ceil(lens[s] / page_size) are never read, and pool
 *  slots at or past lens[s] never reach an output, whatever they hold.
 *
 *  Graph capture: lens and table are read on the device, and max_len only
 *  bounds the launch, so one captured graph serves growing lengths up to
 *  max_len.
 */
#ifndef TF_PAGED_H
#define TF_PAGED_H

#include <stddef.h>
#include <stdint.h>

#if defined(__GNUC__)
#define TF_API __attribute__((visibility("default")))
#else
#define TF_API
#endif

#ifdef __cplusplus
extern "C" {
#endif

/* Status codes returned by every call. */
#define TF_OK 0
#define TF_EINVAL 1        /* a NULL or misaligned pointer, a bad size or an inconsistent shape */
#define TF_EUNSUPPORTED 2  /* a shape this library has no kernel for (head_dim, page_size) */
#define TF_ENOSPACE 3      /* the workspace (or list) is too small for the call */
#define TF_ECUDA 4         /* a CUDA launch or query failed */

/* Bits of the device-side status word (tf_workspace_status). */
#define TF_DEV_BAD_LEN 1u   /* some lens[s] outside [rows, min(max_len, table_stride*page_size)] */
#define TF_DEV_BAD_PAGE 2u  /* some table entry in use outside [0, n_pages) */
#define TF_DEV_TIMEOUT 4u   /* a pipeline wait gave up (an internal error) */
#define TF_DEV_NO_PAGE 8u   /* tf_kv_pages_grow: too few free pages (nothing was changed) */

/* The pool: K and V pages, device memory, 16-byte aligned.
 * page_size may be any positive size at every head dim (TensorFold #1620,
 * Checks, the kernel-contract bullet: the paged prompt kernel is checked
 * over pages of 512, 37 and 64); head_dim must be 128, 256 or 512.  Pages
 * that are not a multiple of 128 positions are read by tiles assembled from
 * page pieces; the results do not depend on the page size.  Head dim 256
 * calls are refused (TF_EUNSUPPORTED) for pools of more than 2^31 - 1 rows
 * (n_pages * n_kv_heads * page_size). */
typedef struct tf_kv_pool {
    void *k_pool;
    void *v_pool;
    int32_t n_pages;
    int32_t n_kv_heads;
    int32_t page_size;
    int32_t head_dim;
} tf_kv_pool;

/* The streams of one call: page table, lengths (device) and a host upper
 * bound on the lengths.  max_len <= table_stride * page_size. */
typedef struct tf_streams {
    const int32_t *table;
    int32_t table_stride;
    const int32_t *lens;
    int32_t n_streams;  /* 0: every call checks its host arguments, then does
                         * nothing and returns TF_OK (its buffers may be null) */
    int32_t max_len;
} tf_streams;

/* Row write (TensorFold #1620, opening comment, "Writes").
 * Copies `rows` new K and V rows per stream into their pages: row r of
 * stream s (k_rows[s][r][kh][:]) goes to position lens[s] - rows + r.  The
 * copy is bitwise; nothing else in the pool is touched.  A row whose
 * stream length or page id is out of range is skipped.  rows >= 1. */
TF_API int tf_kv_put_rows(const tf_kv_pool *pool, const tf_streams *streams,
                   const void *k_rows, const void *v_rows, int32_t rows,
                   void *stream);

/* Rotary positions of a layer.  Pair i (0 <= i < rotary_dim / 2) of a head is
 * dims (i, i + rotary_dim / 2), or with `adjacent` dims (2i, 2i + 1); it is
 * turned by the angle position[axis] * inv_freq[i], where axis =
 * pair_axis[i].  Dims from rotary_dim on are kept.  One axis is the rotary
 * position of text; images and video give each token a time, a height and a
 * width, and pair_axis says which pairs each of them turns (contiguous
 * sections or interleaved: any assignment). */
typedef struct tf_rope {
    const float *inv_freq;     /* device, [rotary_dim / 2] */
    const uint8_t *pair_axis;  /* host, [rotary_dim / 2], each < n_axes; NULL: all axis 0 */
    int32_t rotary_dim;        /* even, in [2, head_dim] */
    int32_t n_axes;            /* in [1, 4] */
    int32_t adjacent;          /* 0 or 1 */
} tf_rope;

/* Row write with rotary positions: turns a step's query and key rows and
 * writes keys and values into their pages, in one pass over the rows
 * (tf_kv_put_rows is the write alone).
 *  positions  device int32 [n_streams][rows][n_axes]: the rows' rotary
 *             positions, of either sign; the slot a row is written to
 *             follows lens, as in tf_kv_put_rows
 *  q          bf16, n_streams * rows rows of n_q_heads * head_dim values,
 *             q_stride elements from one to the next; q_out receives the
 *             turned rows, [n_streams][rows][n_q_heads][head_dim].  q_out may
 *             be q (with q_stride = n_q_heads * head_dim); the two must not
 *             overlap otherwise.  n_q_heads = 0: no queries (q and q_out may
 *             be null)
 *  k_rows, v_rows  likewise with n_kv_heads heads and strides of their own, so
 *             that q, k and v may be slices of one projection's output
 * Pointers are 16-byte aligned and strides are multiples of 8 elements, at
 * least the row's size.  Angles are formed in 64 bits, turned values in fp32
 * and rounded once; values and kept dims are copied bit for bit.  K/V rows
 * whose stream length or page id is out of range are skipped (their queries
 * are turned all the same); nothing else of the pool is touched.
 * Returns TF_OK, TF_EINVAL, TF_EUNSUPPORTED (head_dim) or TF_ECUDA. */
TF_API int tf_kv_put_rows_rope(const tf_kv_pool *pool, const tf_streams *streams,
                               const tf_rope *rope, const int32_t *positions,
                               const void *q, int64_t q_stride, void *q_out,
                               int32_t n_q_heads, const void *k_rows, int64_t k_stride,
                               const void *v_rows, int64_t v_stride, int32_t rows,
                               void *stream);

/* The state copy (TensorFold #1620, opening comment, "Kept states" bullet:
 * a kept state is copied by walking the slot's pages).  For every stream s
 * and position j < src->lens[s], the head_dim bf16 values of K and of V of
 * every KV head are copied bit for bit from src_pool page
 * src->table[s][j / src page_size], slot j % src page_size, to dst_pool page
 * dst_table[s][j / dst page_size], slot j % dst page_size.  Nothing else of
 * dst_pool is written.  The pools may be the same or differ in n_pages and
 * page_size; n_kv_heads and head_dim must match.  A linear buffer is a pool
 * with one page per stream (page_size >= the state's length), so keeping a
 * state (pages to linear), resuming it (linear to pages) and moving it
 * between pages are all this call.
 *  src, src_pool  as for the attention calls (src->max_len bounds every
 *                 lens[s] and sizes the launch)
 *  dst_table      device int32 [n_streams][dst_table_stride], caller-owned;
 *                 dst_table_stride * dst page_size must be >= src->max_len
 *  status         optional device uint32 (4-byte aligned): TF_DEV_BAD_LEN and
 *                 TF_DEV_BAD_PAGE are ORed in for skipped streams and pieces
 * The copied source and destination ranges must not overlap.  Returns
 * TF_OK, TF_EINVAL (bad or mismatched arguments), TF_EUNSUPPORTED (head_dim)
 * or TF_ECUDA; enqueued on `stream`. */
TF_API int tf_kv_copy_state(const tf_kv_pool *src_pool, const tf_streams *src,
                            const tf_kv_pool *dst_pool, const int32_t *dst_table,
                            int32_t dst_table_stride, uint32_t *status, void *stream);

/* Shared pages (TensorFold #1620, opening comment: a stream takes pages of
 * the core pool as it grows; the host leases them there).  The pool's
 * bookkeeping is one device array, refs[page]: how many table entries hold the
 * page, 0 for a free one.  A table entry that holds no page is -1.  A cache
 * starts with refs all 0 and its table all -1.  All calls are enqueued on
 * `stream`, keep no state elsewhere, and give results that depend on refs, the
 * tables and lens alone (pages are taken lowest id first), so they may be
 * captured and replayed.  Calls on the same refs must be ordered by the
 * caller.
 *  refs  device int32 [n_pages], 16-byte aligned; n_pages and a table's stride
 *        are at most 2^31 - 8193 (TF_EINVAL)
 * Every call takes an optional status word (device uint32, 4-byte aligned)
 * into which TF_DEV_* bits are ORed. */
typedef struct tf_kv_pages {
    int32_t *refs;
    int32_t n_pages;
    int32_t page_size;
} tf_kv_pages;

/* Fork: child row c of dst_table names the pages that hold the positions
 * [0, src_lens[parents[c]]) of its parent's row, one holder more each
 * (entries of -1, behind a sliding window, stay -1), the rest of the row is
 * -1, and dst_lens[c] is the parent's length.  parents[c] = -1 makes an empty
 * child.  One parent may have any number of children: n beams, n samples of a
 * prompt.  A reordering of beams forks into a second table and frees the
 * first.
 *  dst rows  are overwritten, not released: they hold no pages before the
 *            call.  They may be rows of src_table's memory that are no
 *            parent's; dst_lens must not overlap src_lens.
 * A parent outside [-1, n_src) or whose pages exceed either table's row makes
 * an empty child and sets TF_DEV_BAD_LEN; a page outside the pool, or one
 * that nobody holds, is left out (-1) and sets TF_DEV_BAD_PAGE. */
TF_API int tf_kv_pages_fork(const tf_kv_pages *pages, const int32_t *src_table,
                            int32_t src_stride, const int32_t *src_lens, int32_t n_src,
                            const int32_t *parents, int32_t n_dst, int32_t *dst_table,
                            int32_t dst_stride, int32_t *dst_lens, uint32_t *status,
                            void *stream);

/* Free: entries [first[s], end[s]) of row s give their pages back (one holder
 * fewer; at 0 the page is free) and hold -1.  first null: from entry 0; end
 * null: to the row's end (both null: the streams are dropped).  Rolling back
 * drafts frees the entries past the last one in use.  Entries of -1 are
 * passed over.  A first or end outside [0, table_stride] frees nothing of the
 * row and sets TF_DEV_BAD_LEN (end at or before first is an empty range);
 * a page that is outside the pool, or that nobody holds, sets
 * TF_DEV_BAD_PAGE. */
TF_API int tf_kv_pages_free(const tf_kv_pages *pages, int32_t *table, int32_t table_stride,
                            int32_t n_streams, const int32_t *first, const int32_t *end,
                            uint32_t *status, void *stream);

/* Frees the pages that a sliding window has left behind: those whose
 * positions are all at or past `sinks` and at or before lens[s] - window, so
 * that no row at position lens[s] or later sees any of them (rows already in
 * the cache might: call it after the step's attention).  window >= 1,
 * sinks >= 0. */
TF_API int tf_kv_pages_free_window(const tf_kv_pages *pages, int32_t *table,
                                   int32_t table_stride, const int32_t *lens,
                                   int32_t n_streams, int32_t window, int32_t sinks,
                                   uint32_t *status, void *stream);

/* A list of page moves: device int32 [1 + cap][4], 16-byte aligned.  Entry 0
 * is the head {moves, live pages (compact), 0, 0}; entry k >= 1 is {source
 * page or -1 (nothing to copy), destination page, positions to copy, -}.
 * tf_kv_pages_grow and _compact write it, tf_kv_pages_move performs it. */
#define TF_MOVE_BYTES 16

/* Grow: gives every position that the step's rows will be written to, lens[s]
 * - rows .. lens[s] - 1 (lens counts them already, as everywhere), a page of
 * the stream's own.  An entry of -1 gets a free page; an entry whose page
 * others hold too gets one in its place (one holder fewer for the old page)
 * and a move of the page's earlier positions (copy on write); an entry whose
 * page is the stream's own stays.  Holders are counted at the start of the
 * call: two streams that grow into the page they share both get their own.
 * A stream of length 0 is passed over; a length outside [rows, table_stride *
 * page_size] sets TF_DEV_BAD_LEN, a page outside the pool, or that nobody
 * holds, TF_DEV_BAD_PAGE, and both are left alone.  When the free pages do
 * not suffice for all streams the call changes nothing, the list is empty and
 * TF_DEV_NO_PAGE is set: read the status before the rows are written.
 *  moves, moves_bytes  the list; TF_ENOSPACE unless it can hold an entry for
 *                      every page the rows may touch: cap >= n_streams *
 *                      ((rows + page_size - 2) / page_size + 1)
 * The moves are performed (on every layer's pool) before rows are written and
 * before the next call that changes refs. */
TF_API int tf_kv_pages_grow(const tf_kv_pages *pages, int32_t *table, int32_t table_stride,
                            const int32_t *lens, int32_t n_streams, int32_t rows,
                            void *moves, size_t moves_bytes, uint32_t *status, void *stream);

/* Compact: moves the live pages to ids 0 .. n_live - 1 (the k-th live page at
 * or past n_live, in ascending order, to the k-th free one below it), and
 * makes refs and the table's entries follow.  The list's head holds the
 * number of moves and n_live, so that a caller may give the pool's tail back.
 * Every table that holds pages must be the one passed: entries elsewhere go
 * stale.
 *  moves  cap >= n_pages / 2, else TF_ENOSPACE */
TF_API int tf_kv_pages_compact(const tf_kv_pages *pages, int32_t *table, int32_t table_stride,
                               int32_t n_streams, void *moves, size_t moves_bytes,
                               uint32_t *status, void *stream);

/* Performs a list's moves on one layer's pool: for every entry the first
 * `positions` positions of the source page, K and V of every KV head, are
 * copied bit for bit to the destination page.  Entries without a source are
 * passed over, ones outside the pool set TF_DEV_BAD_PAGE.  The list stays as
 * it is. */
TF_API int tf_kv_pages_move(const tf_kv_pool *pool, const void *moves, size_t moves_bytes,
                            uint32_t *status, void *stream);

/* Workspace bytes an attention call with these arguments needs on the
 * current device (0 on a bad argument).  Follows the scratch convention of
 * the metrale page "metrale_model_arch/glm5next_dsa/select.rs": scratch is
 * owned by the caller, sized once from the largest shape it will run and
 * reused across steps (the DsaSelectScratch doc comment), and a call whose
 * plan needs more than was given fails before any launch instead of
 * overrunning it (DsaSelectScratch::fits; here TF_ENOSPACE).  The figure
 * holds for any of the attention calls with these arguments
 * (tf_paged_attn_verify_tree included) and for every call over the same pool
 * with no more n_streams and rows * n_q_heads, of any length; a call refuses
 * only what it does not fit into.  The workspace holds split-context partial
 * results and, in its first 4 bytes, the device status word, which
 * the calls only OR bits into: zero those 4 bytes once after allocating
 * (cudaMemset, or one tf_workspace_status call).  The rest needs no
 * initialisation.  One workspace may serve later calls on the same stream;
 * calls that may run concurrently need separate workspaces. */
TF_API size_t tf_paged_attn_workspace_bytes(const tf_kv_pool *pool,
                                     const tf_streams *streams,
                                     int32_t n_q_heads, int32_t rows);

/* Single-row decode (TensorFold #1620, opening comment, "Reads": decode).
 * Same as tf_paged_attn_verify with rows = 1. */
TF_API int tf_paged_attn_decode(const tf_kv_pool *pool, const tf_streams *streams,
                         const void *q, int32_t n_q_heads, float scale,
                         float *out, void *workspace, size_t workspace_bytes,
                         void *stream);

/* Draft-verify window (TensorFold #1620 "Reads": drafted verify; TensorFold
 * #2730 "What this changes": the pending token plus up to seven drafts).
 * rows in [1, 8]; row r sees positions 0 .. lens[s] - rows + r. */
TF_API int tf_paged_attn_verify(const tf_kv_pool *pool, const tf_streams *streams,
                         const void *q, int32_t n_q_heads, int32_t rows,
                         float scale, float *out, void *workspace,
                         size_t workspace_bytes, void *stream);

/* Draft-verify window whose rows form a draft tree (TensorFold #1620,
 * opening comment, first and Reads bullets: drafted verify runs through
 * "tree attention" kernels whose key groups are the 512-position pages; the
 * pages give no mask, so this reading: a window of `rows` drafted tokens,
 * laid out in order, each seeing the positions before the window and the
 * window rows named by its mask).
 *  tree_masks  device, uint8 [n_streams][rows], caller-owned, read during the
 *              call: bit c of tree_masks[s][r] set means row r of stream s
 *              sees window row c (position lens[s] - rows + c).  A draft tree
 *              gives row r its ancestors and itself; the causal window of
 *              tf_paged_attn_verify is the chain mask 2^(r+1) - 1.  Bits at or
 *              above `rows` are ignored.  A row that sees no position at all
 *              (no context before the window and an empty mask) gets NaN.
 * Everything else (arguments, layouts, results, the workspace, errors) is
 * as tf_paged_attn_verify; TF_EINVAL also when tree_masks is null (with
 * n_streams > 0).  Head dim 128
 * calls with more than 64 query rows per KV head (G * rows) read each K/V
 * tile once per 64 rows. */
TF_API int tf_paged_attn_verify_tree(const tf_kv_pool *pool, const tf_streams *streams,
                              const void *q, int32_t n_q_heads, int32_t rows,
                              const uint8_t *tree_masks, float scale, float *out,
                              void *workspace, size_t workspace_bytes, void *stream);

/* Chunked prompt rows (TensorFold #1620 "Reads": prompts through the paged
 * prompt kernels).  The same causal rule as verify for a chunk of
 * rows in [1, 4096] positions: the chunk is the last `rows` positions. */
TF_API int tf_paged_attn_prompt(const tf_kv_pool *pool, const tf_streams *streams,
                         const void *q, int32_t n_q_heads, int32_t rows,
                         float scale, float *out, void *workspace,
                         size_t workspace_bytes, void *stream);

/* Sliding-window attention with sinks: the layers of a model that see only
 * the near context (TensorFold #1620 keeps such layers in ring caches of
 * their own and pages only the full layers; here both read pages).  A row at
 * position p sees the positions j <= p with
 *     j > p - window   (the last `window` positions, its own included), or
 *     j < sinks        (the stream's first tokens, which stay visible);
 * the output is softmax(scale * q . k) weighted sum of v over them.  A row
 * always sees itself.
 *  window  >= 1; a window at or past max_len is the plain causal rule
 *  sinks   >= 0
 * rows, layouts, results and errors are those of tf_paged_attn_decode,
 * _verify (rows in [1, 8]) and _prompt (rows in [1, 4096]), for every head
 * dim, ratio of heads and page size.  Table entries and pool slots of
 * positions that no row of the call sees are never read: pages wholly behind
 * the window (tf_kv_pages_free_window) may hold -1 or belong to somebody
 * else.  A position that some rows of the call see and others do not is
 * masked by its score: its K may be anything to the others, but a V value
 * that is infinite or NaN can reach every row of the call, as in the other
 * calls.  Accuracy, relative to the output's norm: 5e-7 for up to 16 rows per KV
 * head where they run on CUDA cores and mma.sync, 3.5e-6 on the tensor cores
 * (weights kept in two bf16 parts), growing to 6e-6 for prompt rows of head dim
 * 128 over windows from 1,024 to 4,608 positions.  TF_EUNSUPPORTED for pools
 * of more than 2^31 - 1 rows (n_pages * n_kv_heads * page_size).  The workspace is sized by its own call, since a
 * window may be split over other kernels than the whole context; one
 * workspace of the larger size serves both kinds of layer in turn.  The figure
 * grows with n_streams and with rows * n_q_heads and does not depend on
 * max_len, window or sinks: taken for the largest of each, it holds for every
 * smaller call over the same pool.  A smaller workspace is TF_ENOSPACE. */
TF_API size_t tf_paged_attn_window_workspace_bytes(const tf_kv_pool *pool,
                                                   const tf_streams *streams,
                                                   int32_t n_q_heads, int32_t rows,
                                                   int32_t window, int32_t sinks);

TF_API int tf_paged_attn_decode_window(const tf_kv_pool *pool, const tf_streams *streams,
                                       const void *q, int32_t n_q_heads, int32_t window,
                                       int32_t sinks, float scale, float *out, void *workspace,
                                       size_t workspace_bytes, void *stream);

TF_API int tf_paged_attn_verify_window(const tf_kv_pool *pool, const tf_streams *streams,
                                       const void *q, int32_t n_q_heads, int32_t rows,
                                       int32_t window, int32_t sinks, float scale, float *out,
                                       void *workspace, size_t workspace_bytes, void *stream);

TF_API int tf_paged_attn_prompt_window(const tf_kv_pool *pool, const tf_streams *streams,
                                       const void *q, int32_t n_q_heads, int32_t rows,
                                       int32_t window, int32_t sinks, float scale, float *out,
                                       void *workspace, size_t workspace_bytes, void *stream);

/* Single-row decode that allocates nothing and takes no workspace.  The
 * source pages have no counterpart of this call.
 * For callers that cannot allocate device memory for a workspace: a
 * plug-in hosted by an engine that hands it only its input and output
 * buffers, or a serving loop that must not call cudaMalloc once running.
 * The split-context scratch is one static device array of 8 MiB inside
 * this library, held by every GPU that loads it until the process exits.
 * Arguments, results and errors are those of tf_paged_attn_decode, except:
 *  - TF_ENOSPACE when the call would need more than the 8 MiB of scratch
 *    (never where tf_paged_attn_workspace_bytes with rows = 1 is at most that);
 *  - the first call on each device looks the array's device address up
 *    (cudaGetSymbolAddress) with that device current; make that first call
 *    before any stream capture on the device;
 *  - every call on a device shares the one array, which keeps the last
 *    call's contents: calls whose kernels may overlap on the GPU (other
 *    streams, other host threads) race and must be serialised by the caller;
 *  - device-side status bits are not reported (streams with a bad length
 *    still get NaN outputs); use tf_paged_attn_decode to read them. */
TF_API int tf_paged_attn_decode_noalloc(const tf_kv_pool *pool,
                                        const tf_streams *streams,
                                        const void *q, int32_t n_q_heads,
                                        float scale, float *out, void *stream);

/* Reads the workspace's device status word (TF_DEV_* bits accumulated by
 * the attention calls since the last read) into *flags and clears it.
 * Synchronises `stream`.  Returns TF_OK, TF_EINVAL or TF_ECUDA.
 * The source pages have no counterpart of this call: their launchers check
 * host arguments only (the select.rs page's plan and fits), while lens and
 * table here are device data that only the kernels can check. */
TF_API int tf_workspace_status(void *workspace, uint32_t *flags, void *stream);

/* A static, human-readable name for a status code.  The select.rs page's
 * plan and fits refuse a bad shape or a short scratch with a message that
 * names what was wrong; a C caller gets the code from the call and its name
 * from here. */
TF_API const char *tf_status_str(int status);

#ifdef __cplusplus
}
#endif

#endif /* TF_PAGED_H */
