/*
 * nsa_kv4.h -- C ABI of the paged KV cache held in 4 bits: block tables and slot maps
 * built on the GPU, rows written and read back, and the one-step decode that attends
 * to the pages.
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
    NSA_DEVERR_NO_PAGES = 8 /* nsa_page_plan: the free list or the slot map is too short */
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

#ifdef __cplusplus
}
#endif

#endif /* NSA_KV4_H */
