/*
 * nsa_kv4.h -- C ABI of the paged KV cache held in 4 bits: block tables and slot maps
 * built on the GPU, rows of the table forked and freed, pages compacted and copied, rows
 * of K and V written and read back, and the one-step decode that attends to the pages.
 *
 * Conventions are those of nsa_sel_attn.h: device pointers owned by the caller, calls
 * asynchronous on `stream`, arguments checked before anything is enqueued, no device
 * memory allocated, nothing aborts.  int32 arrays are 4-byte aligned.  device_status
 * (int32 in device memory, may be NULL) has bits ORed into it for what only the device
 * can see; a call that raises a bit still writes everything that is not said to be left.
 *
 * The pool: uint8 [num_pages, h_k, page_bytes], 16-byte aligned.  A page holds P =
 * page_size tokens (32, 64 or 128) of each KV head; page_bytes = P * (d + d / 8) for
 * d = head_dim (64 or 128).  The record of a (page, head) is P / 32 tiles of 32 tokens,
 * each of 32 * (d + d / 8) bytes:
 *     K codes [32][d / 2 bytes]
 *     V codes [32][d / 2 bytes]
 *     fp16 [4][32][d / 64]: K scale, K zero, V scale, V zero
 * With G = d / 64 groups of 64 dimensions, a row's codes are little-endian 32-bit words:
 * word j * G + i holds dimensions 64 i + 8 j ... 64 i + 8 j + 7, four bits each, lowest
 * first.  Code c of group i stands for c * scale[i] + zero[i].
 * Quantisation of a group x: values beyond +-65504 saturate; zero = fp16(min x), scale =
 * fp16((max x - zero) / 15), code = (x - zero) / scale to the nearest whole number, ties
 * to even, within 0 ... 15, and 0 where scale is 0.  A group that holds a NaN is stored
 * with a NaN zero: all of it reads as NaN.
 *
 * The bytes of a pool do not say its head_dim (64 tokens of d = 128 are as many as 128 of
 * d = 64): calls on one pool name the same.
 *
 * A slot is the place of one token in the pool: page * P + position within the page.
 * slot_map entries of -1 belong to no token (padding).
 */
#ifndef NSA_KV4_H
#define NSA_KV4_H

#include "nsa_sel_attn.h"

#ifdef __cplusplus
extern "C" {
#endif

/* A bit of the device status words of this header, beside those of nsa_sel_attn.h. */
enum {
    NSA_DEVERR_NO_PAGES = 8 /* the free list, the slot map or a list of copies is too short */
};

typedef struct {
    int32_t num_seqs;    /* B requests, 1 ... 16384 */
    int32_t page_size;   /* P tokens per page, >= 1 */
    int32_t table_width; /* block_table columns, >= 1; table_width * P < 2^31 */
    int32_t num_pages;   /* pages of the pool; num_pages * P < 2^31 */
    int32_t num_free;    /* entries of free_pages (nsa_page_plan) */
    int32_t max_slots;   /* entries of slot_map */
} nsa_page_dims;

/* Block tables and slot maps of one serving step.  Request b has ctx_lens[b] tokens in
 * the cache and brings new_lens[b] more (0 allowed).  In request order, each takes the
 * pages that its new tokens open, ceil((ctx + new) / P) - ceil(ctx / P), from free_pages,
 * starting at entry free_head[0]:
 *   block_table  int32 [B, table_width], updated in place: entries ceil(ctx / P) ...
 *                ceil((ctx + new) / P) - 1 of row b are written, the others left alone;
 *   slot_map     int32 [max_slots]: the slots of the new tokens, packed in request order,
 *                -1 behind the last;
 *   seq_lens     int32 [B] = ctx + new;  cu_new int32 [B + 1]: offsets of the requests'
 *                tokens in slot_map, never above max_slots;
 *   head_out     int32 [1]: free_head advanced by the pages taken.
 * seq_lens may be ctx_lens, and head_out may be free_head (a step that advances its own
 * state); other arrays do not overlap.
 * A request is refused, which leaves its row and length alone and sets its slots to -1,
 *   with NSA_DEVERR_BAD_SEQLENS: a negative length, or ctx + new > table_width * P;
 *   with NSA_DEVERR_NO_PAGES: free_pages ends before its last page, or slot_map before
 *   its last token (its tokens still count in cu_new).  Requests behind it that need
 *   pages (slots) are then refused too.
 * seq_lens of a request refused for its length is ctx held to 0 ... table_width * P.
 * A page id outside 0 ... num_pages - 1, from free_pages or from the table, sets
 * NSA_DEVERR_BAD_INDEX; its tokens' slots are -1 (and its new table entry -1). */
NSA_API nsa_status nsa_page_plan(const nsa_page_dims *dims, const int32_t *ctx_lens,
                                 const int32_t *new_lens, const int32_t *free_pages,
                                 const int32_t *free_head, int32_t *block_table,
                                 int32_t *slot_map, int32_t *seq_lens, int32_t *cu_new,
                                 int32_t *head_out, int32_t *device_status,
                                 nsa_stream_t stream);

/* Slots of tokens that the cache holds already: positions start[b] ... start[b] +
 * count[b] - 1 of each request, packed in request order into slot_map, -1 behind the
 * last; cu int32 [B + 1] gets the offsets.  Errors as above (num_free is not used). */
NSA_API nsa_status nsa_page_slots(const nsa_page_dims *dims, const int32_t *block_table,
                                  const int32_t *start, const int32_t *count,
                                  int32_t *slot_map, int32_t *cu, int32_t *device_status,
                                  nsa_stream_t stream);

/* Forks, frees and compactions.  Beside the block table and the free list (the pages free_pages[
 * free_head[0]] ... free_pages[num_free - 1] belong to nobody; the entries before them are room)
 * the caller keeps
 *   shares       int32 [num_pages]: rows that name a page beyond the first; 0 at the beginning, and
 *                nsa_page_plan, which opens pages for one row each, needs none of it.
 * A page named by a row is one of its first ceil(seq_lens / P) entries.  nsa_page_plan writes tokens
 * into a row's last page where that is partly full, so that only full pages are shared. */
typedef struct {
    int32_t num_seqs;    /* B rows of the table, 1 ... 16384 */
    int32_t page_size;   /* P tokens per page, >= 1 */
    int32_t table_width; /* block_table columns, >= 1; table_width * P < 2^31 */
    int32_t num_pages;   /* entries of shares, 0 ... 2^22 */
    int32_t num_free;    /* entries of free_pages */
    int32_t count;       /* entries of the row lists (0 ... 16384) or of the lists of copies */
} nsa_page_ops_dims;

/* Forks: row children[i] becomes a continuation of row parents[i] (int32 [count]) behind its first
 * n = fork_lens[i] tokens (fork_lens may be NULL: n = seq_lens[parents[i]]).  It gets the parent's
 * floor(n / P) full pages, whose shares grow by one, and, where n % P > 0, the next page of the free
 * list, into which (copy_src[i], copy_dst[i]) says what to copy (nsa_page_copy, for each pool that
 * the table stands for); the pair is -1 where nothing has to be.  Its length becomes n; entries
 * behind it are left alone.  What the child's row held is forgotten, not freed (nsa_page_free).
 * A parent may have several children.  head_out int32 [1], which may be free_head, gets the head
 * advanced by the pages taken.
 * A fork is refused, which leaves the child's row and length alone and its pair -1,
 *   with NSA_DEVERR_BAD_INDEX: a row outside the table, a child that is also a parent, or that an
 *                              earlier entry has named;
 *   with NSA_DEVERR_BAD_SEQLENS: a length n that is negative or beyond the parent's, or a parent's
 *                              length beyond the table;
 *   with NSA_DEVERR_NO_PAGES:  the free list ends before its page (later ones that need a page are
 *                              then refused too).
 * A page id outside 0 ... num_pages - 1, from the table or the free list, sets
 * NSA_DEVERR_BAD_INDEX: the child's entry is -1, or its pair where the copy's source is meant. */
NSA_API nsa_status nsa_page_fork(const nsa_page_ops_dims *dims, int32_t *block_table,
                                 int32_t *seq_lens, const int32_t *parents,
                                 const int32_t *children, const int32_t *fork_lens,
                                 int32_t *shares, const int32_t *free_pages,
                                 const int32_t *free_head, int32_t *copy_src, int32_t *copy_dst,
                                 int32_t *head_out, int32_t *device_status, nsa_stream_t stream);

/* Frees rows (int32 [count]): each of a row's pages loses one owner; those without another go to
 * the free list, in ascending order, into the entries just before its head (head_out, which may be
 * free_head, gets the head less their number).  The row's entries become -1, its length 0.
 * A row outside the table, and one that the list has named before, is passed over with
 * NSA_DEVERR_BAD_INDEX, a row whose length is negative or beyond the table with
 * NSA_DEVERR_BAD_SEQLENS.  Page ids outside 0 ... num_pages - 1 are passed over, and a page that more
 * rows give up than its shares count is freed once, both with NSA_DEVERR_BAD_INDEX.  Where the list
 * has too few entries before its head (or the head lies outside 0 ... num_free), the smallest ids
 * (all) are left out of it, with NSA_DEVERR_NO_PAGES. */
NSA_API nsa_status nsa_page_free(const nsa_page_ops_dims *dims, int32_t *block_table,
                                 int32_t *seq_lens, const int32_t *rows, int32_t *shares,
                                 int32_t *free_pages, const int32_t *free_head, int32_t *head_out,
                                 int32_t *device_status, nsa_stream_t stream);

/* Compacts the pool: with n pages named by the table's rows, those among them with ids from n on
 * move, in ascending order, to the ids below n that no row names, in ascending order.  copy_src and
 * copy_dst (int32 [count]) get the moves, -1 behind them; no page is the source of one and the
 * destination of another, so that nsa_page_copy may make them in any order.  table_out and shares_out,
 * which may be block_table and shares, get the new ids and counts (0 from n on); the last
 * num_pages - n entries of free_out get n ... num_pages - 1, those before are left alone; head_out
 * int32 [1] gets num_free - (num_pages - n).  Pages that no row names count as free: the old free
 * list is not read.
 * Where count is less than the moves, or num_free than num_pages - n, NSA_DEVERR_NO_PAGES is set and
 * nothing changes: table_out and shares_out get their inputs, the lists -1, free_out and head_out are
 * left alone.  count >= num_pages / 2 always suffices.
 * Page ids outside 0 ... num_pages - 1 stay, with NSA_DEVERR_BAD_INDEX; a length outside the table
 * counts as its nearest end, with NSA_DEVERR_BAD_SEQLENS. */
NSA_API nsa_status nsa_page_compact(const nsa_page_ops_dims *dims, const int32_t *block_table,
                                    const int32_t *seq_lens, const int32_t *shares,
                                    int32_t *table_out, int32_t *shares_out, int32_t *free_out,
                                    int32_t *copy_src, int32_t *copy_dst, int32_t *head_out,
                                    int32_t *device_status, nsa_stream_t stream);

/* Copies pages of a pool of num_pages records of page_bytes bytes each (all heads of a page; a
 * multiple of 16, the pool 16-byte aligned): record src[i] to record dst[i], i < count.  Pairs of
 * two -1 are skipped; others with an id outside the pool too, with NSA_DEVERR_BAD_INDEX.  A page is
 * the destination of one pair at most, and of none if it is a source: what else is left in it is
 * not defined. */
NSA_API nsa_status nsa_page_copy(int32_t num_pages, int64_t page_bytes, int32_t count, void *pool,
                                 const int32_t *src, const int32_t *dst, int32_t *device_status,
                                 nsa_stream_t stream);

typedef struct {
    int32_t num_pages; /* pages of the pool; num_pages * page_size < 2^31 */
    int32_t page_size; /* 32, 64 or 128 */
    int32_t h_k;       /* KV heads; num_pages * page_size / 32 * h_k < 2^32 */
    int32_t head_dim;  /* 64 or 128 */
    int32_t dtype;     /* nsa_dtype of k, v, q and out */
} nsa_kv4_dims;

/* Bytes of a (page, head) record, page_size * (head_dim + head_dim / 8) (host only). */
NSA_API nsa_status nsa_kv4_page_bytes(const nsa_kv4_dims *dims, size_t *bytes);

/* Quantises n rows of k and v, [n, h_k, d] with the given strides in elements (multiples
 * of 8; the last dimension contiguous; both 16-byte aligned), into the slots of slot_map
 * [n].  Slot -1 skips the row; a slot below -1 or past the pool is skipped and sets
 * NSA_DEVERR_BAD_INDEX.  A slot may appear once: what two rows leave in one slot is not
 * defined. */
NSA_API nsa_status nsa_kv4_append(const nsa_kv4_dims *dims, int32_t n, const void *k,
                                  int64_t k_token_stride, int64_t k_head_stride, const void *v,
                                  int64_t v_token_stride, int64_t v_head_stride,
                                  const int32_t *slot_map, void *pool, int32_t *device_status,
                                  nsa_stream_t stream);

/* Reads n rows back: k and v [n, h_k, d] (contiguous, 16-byte aligned) get the values of
 * the slots, rounded once to the dtype.  Rows of slot -1 are zeros, and so are those of an
 * invalid slot, which sets NSA_DEVERR_BAD_INDEX. */
NSA_API nsa_status nsa_kv4_read(const nsa_kv4_dims *dims, int32_t n, const void *pool,
                                const int32_t *slot_map, void *k, void *v,
                                int32_t *device_status, nsa_stream_t stream);

/* One-step decode over the pages: request b's new token, the last of seq_lens[b] cached
 * tokens, attends to keys of its own pages with one softmax.
 *   sel_idx      int32 [h_k, B, topk] (1 <= topk <= 32): the blocks to attend to, a block
 *                being a page (B_K = page_size), with the validity and de-duplication
 *                rules of nsa_sel_attn_decode; NULL (topk 0) attends to every block;
 *   window       > 0 keeps the keys of the last `window` tokens only; 0 keeps all;
 *   q            [B, h_q, d], out [B, h_q, d] (dtype, 16-byte aligned); h_q / h_k <= 16;
 *   lse          float32 [h_q, B], natural log, scale included;
 *   block_table  int32 [B, table_width], seq_lens int32 [B] (0 allowed: out = 0, lse =
 *                -inf).  A length that is negative or above table_width * P counts as 0
 *                or table_width * P and sets NSA_DEVERR_BAD_SEQLENS; the keys of a page id
 *                outside the pool are left out and set NSA_DEVERR_BAD_INDEX.
 *   workspace    at least nsa_kv4_decode_workspace_size bytes, 16-byte aligned (NULL when
 *                that is 0); its contents carry nothing from one call to the next.  Calls that
 *                may overlap on the GPU need workspaces of their own.
 * num_seqs * h_k * (table_width * page_size / 32 + 5), twice that for h_q / h_k > 8, has to
 * stay below 2^30 (NSA_ERR_UNSUPPORTED).
 * Rows of the pool behind a sequence's end, and tokens before its window, may hold
 * anything, NaN included. */
NSA_API nsa_status nsa_kv4_decode(const nsa_kv4_dims *dims, int32_t num_seqs, int32_t h_q,
                                  int32_t table_width, int32_t topk, int32_t window,
                                  const void *q, const void *pool, const int32_t *block_table,
                                  const int32_t *seq_lens, const int32_t *sel_idx, float scale,
                                  void *out, float *lse, int32_t *device_status, void *workspace,
                                  size_t workspace_bytes, nsa_stream_t stream);
NSA_API nsa_status nsa_kv4_decode_workspace_size(const nsa_kv4_dims *dims, int32_t num_seqs,
                                                 int32_t h_q, int32_t topk, size_t *bytes);

/* nsa_kv4_decode without a selection or a window, for a batch whose sequences share prefixes: group i
 * is sequences cu_groups[i] ... cu_groups[i + 1] - 1 (cu_groups int32 [num_groups + 1], from 0 on,
 * non-decreasing, num_seqs at most; sequences behind the last group share nothing), whose first
 * prefix_lens[i] tokens (int32 [num_groups], any number) are the same.  Every row of the table names all
 * of its sequence's pages, those of the prefix too (nsa_page_fork makes such rows).  Where it pays, the
 * prefix is read once for the group, from the pages of its first sequence that is as long as it (others
 * may have ended, nsa_page_free), and what lies behind it from each sequence's own; elsewhere (groups of
 * one, short prefixes, and batches that are small by num_seqs, h_q and table_width * P, which go
 * nsa_kv4_decode's way) each sequence reads its own pages.  A sequence that is shorter than its group's
 * prefix attends to its own pages alone.  A group is neighbouring rows of the table: a caller whose rows
 * are in another order brings table, lengths, q and outputs into it.
 *   lse is nsa_kv4_decode's within fp32's rounding.  out is as well, except that in a prefix that is shared
 * V's values are rounded to fp16 and, for bf16 outputs, the weights too, by at most 2^-11 of each, so that
 * fp16 outputs are up to 2^0.5 times their own rounding off, bf16 ones 1 % more than theirs.  Which
 * prefixes are shared depends on sizes alone (num_seqs, heads, table_width * P, a group's sequences and
 * prefix): the same sequences give other last bits in a wider table or a larger group.
 *   Arguments and errors are nsa_kv4_decode's; in addition, where the call looks for what to share, a
 * cu_groups out of order (nothing is shared then) and a prefix that is negative or above
 * table_width * P (that group shares nothing) set NSA_DEVERR_BAD_SEQLENS, and a device wait that gave
 * up NSA_DEVERR_TIMEOUT (outputs are then not defined).  num_groups is 1 ... 2^20. */
NSA_API nsa_status nsa_kv4_decode_shared(const nsa_kv4_dims *dims, int32_t num_seqs, int32_t h_q,
                                         int32_t table_width, int32_t num_groups, const void *q,
                                         const void *pool, const int32_t *block_table,
                                         const int32_t *seq_lens, const int32_t *cu_groups,
                                         const int32_t *prefix_lens, float scale, void *out,
                                         float *lse, int32_t *device_status, void *workspace,
                                         size_t workspace_bytes, nsa_stream_t stream);
NSA_API nsa_status nsa_kv4_decode_shared_workspace_size(const nsa_kv4_dims *dims, int32_t num_seqs,
                                                        int32_t h_q, int32_t num_groups,
                                                        size_t *bytes);

#ifdef __cplusplus
}
#endif

#endif /* NSA_KV4_H */
