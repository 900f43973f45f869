// kv4_api.cu -- the C ABI of include/nsa_kv4.h: argument checks and launches.
#include <cmath>
#include <cstring>
#include <initializer_list>

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

nsa_status check_ops(const nsa_page_ops_dims *d, bool rows) {
  if (!d) return NSA_ERR_INVALID_ARG;
  if (d->num_seqs < 1 || d->page_size < 1 || d->table_width < 1 || d->num_pages < 0 ||
      d->num_free < 0 || d->count < 0)
    return NSA_ERR_INVALID_ARG;
  if (d->num_seqs > kMaxPlanSeqs || d->num_pages > kMaxOpsPages || (rows && d->count > kMaxPlanSeqs) ||
      (int64_t)d->table_width * d->page_size >= (int64_t(1) << 31))
    return NSA_ERR_UNSUPPORTED;
  return NSA_OK;
}

PageOpsParams ops_params(const nsa_page_ops_dims *d, int32_t *status) {
  PageOpsParams p;
  std::memset(&p, 0, sizeof(p));
  p.num_seqs = d->num_seqs;
  p.page = d->page_size;
  p.width = d->table_width;
  p.num_pages = d->num_pages;
  p.num_free = d->num_free;
  p.count = d->count;
  p.status = status;
  return p;
}

// All of them there (where `needed`) and 4-byte aligned.
struct IntArg {
  const void *ptr;
  bool needed;
};
bool ints_ok(std::initializer_list<IntArg> args) {
  for (const IntArg &a : args)
    if ((a.needed && !a.ptr) || !on(a.ptr, 4)) return false;
  return true;
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

nsa_status nsa_page_fork(const nsa_page_ops_dims *dims, int32_t *block_table, int32_t *seq_lens,
                         const int32_t *parents, const int32_t *children, const int32_t *fork_lens,
                         int32_t *shares, const int32_t *free_pages, const int32_t *free_head,
                         int32_t *copy_src, int32_t *copy_dst, int32_t *head_out,
                         int32_t *device_status, nsa_stream_t stream) {
  nsa_status st = check_ops(dims, true);
  if (st != NSA_OK) return st;
  const bool any = dims->count > 0;
  if (!ints_ok({{block_table, true}, {seq_lens, true}, {parents, any}, {children, any},
                {fork_lens, false}, {shares, dims->num_pages > 0}, {free_pages, dims->num_free > 0},
                {free_head, true}, {copy_src, any}, {copy_dst, any}, {head_out, true},
                {device_status, false}}))
    return NSA_ERR_INVALID_ARG;
  PageOpsParams p = ops_params(dims, device_status);
  p.table = block_table;
  p.lens = seq_lens;
  p.rows_from = parents;
  p.rows_to = children;
  p.fork_lens = fork_lens;
  p.shares = shares;
  p.free_pages = const_cast<int32_t *>(free_pages);   // only read by a fork
  p.head_in = free_head;
  p.copy_src = copy_src;
  p.copy_dst = copy_dst;
  p.head_out = head_out;
  return launched(launch_page_op(PageOp::kFork, p, reinterpret_cast<cudaStream_t>(stream)));
}

nsa_status nsa_page_free(const nsa_page_ops_dims *dims, int32_t *block_table, int32_t *seq_lens,
                         const int32_t *rows, int32_t *shares, int32_t *free_pages,
                         const int32_t *free_head, int32_t *head_out, int32_t *device_status,
                         nsa_stream_t stream) {
  nsa_status st = check_ops(dims, true);
  if (st != NSA_OK) return st;
  if (!ints_ok({{block_table, true}, {seq_lens, true}, {rows, dims->count > 0},
                {shares, dims->num_pages > 0}, {free_pages, dims->num_free > 0}, {free_head, true},
                {head_out, true}, {device_status, false}}))
    return NSA_ERR_INVALID_ARG;
  PageOpsParams p = ops_params(dims, device_status);
  p.table = block_table;
  p.lens = seq_lens;
  p.rows_from = rows;
  p.shares = shares;
  p.free_pages = free_pages;
  p.head_in = free_head;
  p.head_out = head_out;
  return launched(launch_page_op(PageOp::kFree, p, reinterpret_cast<cudaStream_t>(stream)));
}

nsa_status nsa_page_compact(const nsa_page_ops_dims *dims, const int32_t *block_table,
                            const int32_t *seq_lens, const int32_t *shares, int32_t *table_out,
                            int32_t *shares_out, int32_t *free_out, int32_t *copy_src,
                            int32_t *copy_dst, int32_t *head_out, int32_t *device_status,
                            nsa_stream_t stream) {
  nsa_status st = check_ops(dims, false);
  if (st != NSA_OK) return st;
  const bool any = dims->count > 0, pages = dims->num_pages > 0;
  if (!ints_ok({{block_table, true}, {seq_lens, true}, {shares, pages}, {table_out, true},
                {shares_out, pages}, {free_out, dims->num_free > 0}, {copy_src, any},
                {copy_dst, any}, {head_out, true}, {device_status, false}}))
    return NSA_ERR_INVALID_ARG;
  PageOpsParams p = ops_params(dims, device_status);
  p.table_in = block_table;
  p.table = table_out;
  p.lens = const_cast<int32_t *>(seq_lens);           // only read by a compaction
  p.shares_in = shares;
  p.shares = shares_out;
  p.free_pages = free_out;
  p.copy_src = copy_src;
  p.copy_dst = copy_dst;
  p.head_out = head_out;
  return launched(launch_page_op(PageOp::kCompact, p, reinterpret_cast<cudaStream_t>(stream)));
}

nsa_status nsa_page_copy(int32_t num_pages, int64_t page_bytes, int32_t count, void *pool,
                         const int32_t *src, const int32_t *dst, int32_t *device_status,
                         nsa_stream_t stream) {
  if (num_pages < 0 || page_bytes < 1 || count < 0) return NSA_ERR_INVALID_ARG;
  if (page_bytes % 16 || page_bytes >= (int64_t(1) << 40)) return NSA_ERR_UNSUPPORTED;
  if (count == 0) return NSA_OK;
  if ((num_pages > 0 && !pool) || !on(pool, 16) ||
      !ints_ok({{src, true}, {dst, true}, {device_status, false}}))
    return NSA_ERR_INVALID_ARG;
  return launched(launch_page_copy(num_pages, page_bytes, count, pool, src, dst, device_status,
                                   reinterpret_cast<cudaStream_t>(stream)));
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

// Checks of what both decodes take, and their parameters.
static nsa_status decode_params(const nsa_kv4_dims *dims, int32_t num_seqs, int32_t h_q,
                                int32_t table_width, int32_t topk, int32_t window, const void *q,
                                const void *pool, const int32_t *block_table,
                                const int32_t *seq_lens, const int32_t *sel_idx, float scale, void *out,
                                float *lse, int32_t *device_status, void *workspace,
                                Kv4DecodeParams &p) {
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
  std::memset(&p, 0, sizeof(p));
  p.num_seqs = num_seqs;
  p.h_q = h_q;
  p.h_k = dims->h_k;
  p.g = h_q / dims->h_k;
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
  return NSA_OK;
}

nsa_status nsa_kv4_decode(const nsa_kv4_dims *dims, int32_t num_seqs, int32_t h_q,
                          int32_t table_width, int32_t topk, int32_t window, const void *q,
                          const void *pool, const int32_t *block_table, const int32_t *seq_lens,
                          const int32_t *sel_idx, float scale, void *out, float *lse,
                          int32_t *device_status, void *workspace, size_t workspace_bytes,
                          nsa_stream_t stream) {
  Kv4DecodeParams p;
  const nsa_status st =
      decode_params(dims, num_seqs, h_q, table_width, topk, window, q, pool, block_table, seq_lens,
                    sel_idx, scale, out, lse, device_status, workspace, p);
  if (st != NSA_OK) return st;
  const size_t need = kv4_decode_workspace(dims->head_dim, p.g, topk > 0);
  if (need > 0 && (!workspace || workspace_bytes < need)) return NSA_ERR_WORKSPACE;
  if (kv4_decode_tiles(p) >= (int64_t(1) << 30)) return NSA_ERR_UNSUPPORTED;
  return launched(launch_kv4_decode(dims->head_dim, dims->dtype == NSA_FP16, p,
                                    reinterpret_cast<cudaStream_t>(stream)));
}

// The workspace: what the sequences' own parts take, then the plan and the partial results.
static nsa_status check_shared(const nsa_kv4_dims *dims, int32_t num_seqs, int32_t h_q,
                               int32_t num_groups, size_t *first, size_t *bytes) {
  const nsa_status st = check_decode(dims, num_seqs, h_q, 0);
  if (st != NSA_OK) return st;
  if (num_groups < 1) return NSA_ERR_INVALID_ARG;
  if (num_groups > (1 << 20)) return NSA_ERR_UNSUPPORTED;
  *first = (kv4_decode_workspace(dims->head_dim, h_q / dims->h_k, false) + 255) / 256 * 256;
  *bytes = *first + kv4_shared_workspace(dims->head_dim, num_seqs, h_q, num_groups);
  return NSA_OK;
}

nsa_status nsa_kv4_decode_shared_workspace_size(const nsa_kv4_dims *dims, int32_t num_seqs,
                                                int32_t h_q, int32_t num_groups, size_t *bytes) {
  size_t first, all;
  const nsa_status st = check_shared(dims, num_seqs, h_q, num_groups, &first, &all);
  if (st != NSA_OK) return st;
  if (!bytes) return NSA_ERR_INVALID_ARG;
  *bytes = all;
  return NSA_OK;
}

nsa_status nsa_kv4_decode_shared(const nsa_kv4_dims *dims, int32_t num_seqs, int32_t h_q,
                                 int32_t table_width, int32_t num_groups, const void *q,
                                 const void *pool, const int32_t *block_table,
                                 const int32_t *seq_lens, const int32_t *cu_groups,
                                 const int32_t *prefix_lens, float scale, void *out, float *lse,
                                 int32_t *device_status, void *workspace, size_t workspace_bytes,
                                 nsa_stream_t stream) {
  Kv4SharedParams p;
  size_t first, need;
  nsa_status st = check_shared(dims, num_seqs, h_q, num_groups, &first, &need);
  if (st == NSA_OK)
    st = decode_params(dims, num_seqs, h_q, table_width, 0, 0, q, pool, block_table, seq_lens, nullptr,
                       scale, out, lse, device_status, workspace, p.dec);
  if (st != NSA_OK) return st;
  if (!ints_ok({{cu_groups, true}, {prefix_lens, true}})) return NSA_ERR_INVALID_ARG;
  if (!workspace || workspace_bytes < need) return NSA_ERR_WORKSPACE;
  if (kv4_decode_tiles(p.dec) >= (int64_t(1) << 30)) return NSA_ERR_UNSUPPORTED;
  p.num_groups = num_groups;
  p.cu = cu_groups;
  p.prefix = prefix_lens;
  p.ws = static_cast<uint8_t *>(workspace) + first;
  return launched(launch_kv4_shared(dims->head_dim, dims->dtype == NSA_FP16, p,
                                    reinterpret_cast<cudaStream_t>(stream)));
}

}  // extern "C"
