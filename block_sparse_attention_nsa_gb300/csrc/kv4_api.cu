// kv4_api.cu -- the C ABI of include/nsa_kv4.h: argument checks and launches.
#include <cmath>
#include <cstring>

#include "kv4.cuh"

namespace nsa {
namespace {

bool on(const void *ptr, size_t a) { return (reinterpret_cast<uintptr_t>(ptr) % a) == 0; }

nsa_status launched(cudaError_t e) { return e == cudaSuccess ? NSA_OK : NSA_ERR_CUDA; }

nsa_status check_pages(const nsa_page_dims *d) {
  if (!d) return NSA_ERR_INVALID_ARG;
  if (d->num_seqs < 1 || d->page_size < 1 || d->table_width < 1 || d->num_pages < 0 ||
      d->num_free < 0 || d->max_slots < 0)
    return NSA_ERR_INVALID_ARG;
  if (d->num_seqs > kMaxPlanSeqs) return NSA_ERR_UNSUPPORTED;
  const int64_t most = int64_t(1) << 31;
  if ((int64_t)d->table_width * d->page_size >= most || (int64_t)d->num_pages * d->page_size >= most)
    return NSA_ERR_UNSUPPORTED;
  return NSA_OK;
}

nsa_status check_kv4(const nsa_kv4_dims *d) {
  if (!d) return NSA_ERR_INVALID_ARG;
  if (d->num_pages < 0 || d->h_k < 1) return NSA_ERR_INVALID_ARG;
  if (d->dtype != NSA_BF16 && d->dtype != NSA_FP16) return NSA_ERR_UNSUPPORTED;
  if (d->head_dim != 64 && d->head_dim != 128) return NSA_ERR_UNSUPPORTED;
  if (d->page_size != 32 && d->page_size != 64 && d->page_size != 128) return NSA_ERR_UNSUPPORTED;
  const int64_t tokens = (int64_t)d->num_pages * d->page_size;
  if (tokens >= (int64_t(1) << 31) || tokens / kKv4Tile * d->h_k >= (int64_t(1) << 32))
    return NSA_ERR_UNSUPPORTED;
  return NSA_OK;
}

int log2_of(int p) { return p == 32 ? 5 : p == 64 ? 6 : 7; }

PageParams page_params(const nsa_page_dims *d) {
  PageParams p;
  std::memset(&p, 0, sizeof(p));
  p.num_seqs = d->num_seqs;
  p.page = d->page_size;
  p.width = d->table_width;
  p.num_pages = d->num_pages;
  p.num_free = d->num_free;
  p.max_slots = d->max_slots;
  return p;
}

nsa_status check_rows(const nsa_kv4_dims *d, int32_t n, const void *pool, const int32_t *slots,
                      const int32_t *status) {
  nsa_status st = check_kv4(d);
  if (st != NSA_OK) return st;
  if (n < 0) return NSA_ERR_INVALID_ARG;
  // a CTA takes eight heads' rows of 512 / d tokens (kv4_rows.cu): the grid stays below 2^30
  if ((int64_t)n * d->h_k >= (int64_t(1) << 38) / (d->head_dim / 4)) return NSA_ERR_UNSUPPORTED;
  if (n > 0 && (!slots || (d->num_pages > 0 && !pool))) return NSA_ERR_INVALID_ARG;
  if (!on(slots, 4) || !on(pool, 16) || !on(status, 4)) return NSA_ERR_INVALID_ARG;
  return NSA_OK;
}

Kv4RowParams row_params(const nsa_kv4_dims *d, int32_t n, const int32_t *slots, void *pool,
                        int32_t *status) {
  Kv4RowParams p;
  std::memset(&p, 0, sizeof(p));
  p.n = n;
  p.h_k = d->h_k;
  p.num_pages = d->num_pages;
  p.page_log2 = log2_of(d->page_size);
  p.slots = slots;
  p.pool = static_cast<uint8_t *>(pool);
  p.status = status;
  return p;
}

}  // namespace
}  // namespace nsa

using namespace nsa;

extern "C" {

nsa_status nsa_page_plan(const nsa_page_dims *dims, const int32_t *ctx_lens,
                         const int32_t *new_lens, const int32_t *free_pages,
                         const int32_t *free_head, int32_t *block_table, int32_t *slot_map,
                         int32_t *seq_lens, int32_t *cu_new, int32_t *head_out,
                         int32_t *device_status, nsa_stream_t stream) {
  nsa_status st = check_pages(dims);
  if (st != NSA_OK) return st;
  if (!ctx_lens || !new_lens || !free_head || !block_table || !seq_lens || !cu_new || !head_out ||
      (dims->num_free > 0 && !free_pages) || (dims->max_slots > 0 && !slot_map))
    return NSA_ERR_INVALID_ARG;
  for (const void *x : {(const void *)ctx_lens, (const void *)new_lens, (const void *)free_pages,
                        (const void *)free_head, (const void *)block_table, (const void *)slot_map,
                        (const void *)seq_lens, (const void *)cu_new, (const void *)head_out,
                        (const void *)device_status})
    if (!on(x, 4)) return NSA_ERR_INVALID_ARG;
  PageParams p = page_params(dims);
  p.ctx = ctx_lens;
  p.add = new_lens;
  p.free_pages = free_pages;
  p.free_head = free_head;
  p.table = block_table;
  p.slots = slot_map;
  p.seq_out = seq_lens;
  p.cu_out = cu_new;
  p.head_out = head_out;
  p.status = device_status;
  return launched(launch_pages(p, true, reinterpret_cast<cudaStream_t>(stream)));
}

nsa_status nsa_page_slots(const nsa_page_dims *dims, const int32_t *block_table,
                          const int32_t *start, const int32_t *count, int32_t *slot_map,
                          int32_t *cu, int32_t *device_status, nsa_stream_t stream) {
  nsa_status st = check_pages(dims);
  if (st != NSA_OK) return st;
  if (!block_table || !start || !count || !cu || (dims->max_slots > 0 && !slot_map))
    return NSA_ERR_INVALID_ARG;
  for (const void *x : {(const void *)block_table, (const void *)start, (const void *)count,
                        (const void *)slot_map, (const void *)cu, (const void *)device_status})
    if (!on(x, 4)) return NSA_ERR_INVALID_ARG;
  PageParams p = page_params(dims);
  p.ctx = start;
  p.add = count;
  p.table = const_cast<int32_t *>(block_table);   // only a plan writes it
  p.slots = slot_map;
  p.cu_out = cu;
  p.status = device_status;
  return launched(launch_pages(p, false, reinterpret_cast<cudaStream_t>(stream)));
}

nsa_status nsa_kv4_page_bytes(const nsa_kv4_dims *dims, size_t *bytes) {
  nsa_status st = check_kv4(dims);
  if (st != NSA_OK) return st;
  if (!bytes) return NSA_ERR_INVALID_ARG;
  *bytes = static_cast<size_t>(dims->page_size) * (dims->head_dim + dims->head_dim / 8);
  return NSA_OK;
}

nsa_status nsa_kv4_append(const nsa_kv4_dims *dims, int32_t n, const void *k,
                          int64_t k_token_stride, int64_t k_head_stride, const void *v,
                          int64_t v_token_stride, int64_t v_head_stride, const int32_t *slot_map,
                          void *pool, int32_t *device_status, nsa_stream_t stream) {
  nsa_status st = check_rows(dims, n, pool, slot_map, device_status);
  if (st != NSA_OK) return st;
  if (n > 0 && (!k || !v)) return NSA_ERR_INVALID_ARG;
  if (!on(k, 16) || !on(v, 16) || k_token_stride % 8 || k_head_stride % 8 || v_token_stride % 8 ||
      v_head_stride % 8)
    return NSA_ERR_INVALID_ARG;
  if (n == 0) return NSA_OK;
  Kv4RowParams p = row_params(dims, n, slot_map, pool, device_status);
  p.k = k;
  p.v = v;
  p.k_ts = k_token_stride;
  p.k_hs = k_head_stride;
  p.v_ts = v_token_stride;
  p.v_hs = v_head_stride;
  return launched(launch_kv4_append(dims->head_dim, dims->dtype == NSA_FP16, p,
                                    reinterpret_cast<cudaStream_t>(stream)));
}

nsa_status nsa_kv4_read(const nsa_kv4_dims *dims, int32_t n, const void *pool,
                        const int32_t *slot_map, void *k, void *v, int32_t *device_status,
                        nsa_stream_t stream) {
  nsa_status st = check_rows(dims, n, pool, slot_map, device_status);
  if (st != NSA_OK) return st;
  if (n > 0 && (!k || !v)) return NSA_ERR_INVALID_ARG;
  if (!on(k, 16) || !on(v, 16)) return NSA_ERR_INVALID_ARG;
  if (n == 0) return NSA_OK;
  Kv4RowParams p = row_params(dims, n, slot_map, const_cast<void *>(pool), device_status);
  p.k_out = k;
  p.v_out = v;
  return launched(launch_kv4_read(dims->head_dim, dims->dtype == NSA_FP16, p,
                                  reinterpret_cast<cudaStream_t>(stream)));
}

static nsa_status check_decode(const nsa_kv4_dims *dims, int32_t num_seqs, int32_t h_q,
                               int32_t topk) {
  nsa_status st = check_kv4(dims);
  if (st != NSA_OK) return st;
  if (num_seqs < 1 || h_q < 1 || topk < 0 || h_q % dims->h_k != 0) return NSA_ERR_INVALID_ARG;
  if (topk > 32 || h_q / dims->h_k > 16 || dims->h_k > 65535) return NSA_ERR_UNSUPPORTED;
  if ((int64_t)num_seqs * h_q >= (int64_t(1) << 31)) return NSA_ERR_UNSUPPORTED;
  return NSA_OK;
}

nsa_status nsa_kv4_decode_workspace_size(const nsa_kv4_dims *dims, int32_t num_seqs, int32_t h_q,
                                         int32_t topk, size_t *bytes) {
  nsa_status st = check_decode(dims, num_seqs, h_q, topk);
  if (st != NSA_OK) return st;
  if (!bytes) return NSA_ERR_INVALID_ARG;
  *bytes = kv4_decode_workspace(dims->head_dim, h_q / dims->h_k, topk > 0);
  return NSA_OK;
}

nsa_status nsa_kv4_decode(const nsa_kv4_dims *dims, int32_t num_seqs, int32_t h_q,
                          int32_t table_width, int32_t topk, int32_t window, const void *q,
                          const void *pool, const int32_t *block_table, const int32_t *seq_lens,
                          const int32_t *sel_idx, float scale, void *out, float *lse,
                          int32_t *device_status, void *workspace, size_t workspace_bytes,
                          nsa_stream_t stream) {
  nsa_status st = check_decode(dims, num_seqs, h_q, topk);
  if (st != NSA_OK) return st;
  if (table_width < 1 || window < 0 || !std::isfinite(scale)) return NSA_ERR_INVALID_ARG;
  if ((int64_t)table_width * dims->page_size >= (int64_t(1) << 31)) return NSA_ERR_UNSUPPORTED;
  if (!q || !block_table || !seq_lens || !out || !lse || (dims->num_pages > 0 && !pool) ||
      (topk > 0) != (sel_idx != nullptr))
    return NSA_ERR_INVALID_ARG;
  if (!on(q, 16) || !on(pool, 16) || !on(out, 16) || !on(workspace, 16) || !on(block_table, 4) ||
      !on(seq_lens, 4) || !on(sel_idx, 4) || !on(lse, 4) || !on(device_status, 4))
    return NSA_ERR_INVALID_ARG;
  const int g = h_q / dims->h_k;
  const size_t need = kv4_decode_workspace(dims->head_dim, g, topk > 0);
  if (need > 0 && (!workspace || workspace_bytes < need)) return NSA_ERR_WORKSPACE;
  Kv4DecodeParams p;
  std::memset(&p, 0, sizeof(p));
  p.num_seqs = num_seqs;
  p.h_q = h_q;
  p.h_k = dims->h_k;
  p.g = g;
  p.num_pages = dims->num_pages;
  p.page_log2 = log2_of(dims->page_size);
  p.width = table_width;
  p.topk = topk;
  p.window = window;
  p.scale = scale;
  p.q = q;
  p.pool = static_cast<const uint8_t *>(pool);
  p.table = block_table;
  p.lens = seq_lens;
  p.sel = sel_idx;
  p.out = out;
  p.lse = lse;
  p.status = device_status;
  p.ws = workspace;
  if (kv4_decode_tiles(p) >= (int64_t(1) << 30)) return NSA_ERR_UNSUPPORTED;
  return launched(launch_kv4_decode(dims->head_dim, dims->dtype == NSA_FP16, p,
                                    reinterpret_cast<cudaStream_t>(stream)));
}

}  // extern "C"
