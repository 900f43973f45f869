// page_ops.cu -- the life of a cache's pages: rows forked and freed, the pool compacted, pages copied.
//
// State: the block table, the rows' lengths, shares[p] (rows that name page p beyond the first) and a
// free list with its head (include/nsa_kv4.h).  Counts are whole numbers, added by atomics, so no
// order shows in them; what has an order (places in the free list, lists of copies) comes from
// scans: a fork's free page is the head plus the forks before it that need one; pages that are
// freed, moved or filled are taken in ascending order from a bitmap of all pages.
//
// A few bytes per page: latency counts.  One launch of one CTA, or of a cluster of sixteen that split
// the rows (a warp a row, or a part of one) and the bitmap (a slice of pages a CTA, set through
// distributed shared memory); a cluster barrier between the steps.  Measured, caches cold: 64 rows of up to
// 128 pages forked eight times each 9 us, those 512 rows freed 12, 333 rows of up to 128 pages freed 13,
// 500 rows with 22K of 30K pages compacted 27: a third of that are marks and lookups in other CTAs'
// memory, the rest chains of dependent reads, most of them rows and lengths from HBM.  page_copy moves
// bytes, bound by HBM (238 MB of pages read and written in 70 us: 6.8 TB/s).
#include "kv4.cuh"

namespace nsa {

constexpr int kOpsThreads = 1024, kOpsWarps = kOpsThreads / 32;

// Inclusive prefix over the CTA's threads; total gets the sum.  All threads take part.
__device__ __forceinline__ int cta_incl(int x, int (&part)[kOpsWarps], int &total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  __syncthreads();                       // the totals of the call before have been read
  if (lane == 31) part[warp] = x;
  __syncthreads();
  int w = part[lane];
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, w, o);
    if (lane >= o) w += y;
  }
  total = __shfl_sync(0xffffffffu, w, 31);
  const int before = __shfl_sync(0xffffffffu, w, (warp + 31) & 31);
  return x + (warp ? before : 0);
}

// owner[r]: the first entry of list that names row r (count where none does).
__device__ __forceinline__ void first_owners(int *owner, const int32_t *list, int count, int rows) {
  for (int r = threadIdx.x; r < rows; r += kOpsThreads) owner[r] = count;
  __syncthreads();
  for (int i = threadIdx.x; i < count; i += kOpsThreads) {
    const int r = list[i];
    if (r >= 0 && r < rows) atomicMin(&owner[r], i);
  }
}

// Pages of a row of this length; a length outside the table counts as its nearest end.
__device__ __forceinline__ int row_pages(const PageOpsParams &p, int len, int32_t &err) {
  const int64_t cap = (int64_t)p.width * p.page;
  if (len < 0 || len > cap) err |= NSA_DEVERR_BAD_SEQLENS;
  const int64_t n = min((int64_t)max(len, 0), cap);
  return static_cast<int>((n + p.page - 1) / p.page);
}

__device__ __forceinline__ void report(const PageOpsParams &p, int32_t err) {
  err = __reduce_or_sync(0xffffffffu, err);
  if (err && (threadIdx.x & 31) == 0) raise(p.status, err);
}

// ---- fork -------------------------------------------------------------------------------
__global__ void __launch_bounds__(kOpsThreads) page_fork_kernel(PageOpsParams p) {
  extern __shared__ int32_t sm[];
  int *owner = sm;                         // [B] first fork into the row
  int *lens = owner + p.num_seqs;          // [count] tokens of the fork, -1: refused
  int *place = lens + p.count;             // [count] place of its page in the free list, -1: none
  uint32_t *source = reinterpret_cast<uint32_t *>(place + p.count);   // [B / 32] rows forked from
  __shared__ int part[kOpsWarps], taken;
  const int tid = threadIdx.x, lane = tid & 31, rank = blockIdx.x, ncta = gridDim.x;
  const int64_t cap = (int64_t)p.width * p.page;
  after_previous();
  for (int i = tid; i < (p.num_seqs + 31) / 32; i += kOpsThreads) source[i] = 0;
  if (tid == 0) taken = 0;
  first_owners(owner, p.rows_to, p.count, p.num_seqs);   // its barrier covers the marks' clearing
  for (int i = tid; i < p.count; i += kOpsThreads) {
    const int r = p.rows_from[i];
    if (r >= 0 && r < p.num_seqs) atomicOr(&source[r >> 5], 1u << (r & 31));
  }
  int32_t err = 0;
  const int free0 = *p.head_in;
  int avail = 0;
  if (free0 < 0 || free0 > p.num_free) err |= NSA_DEVERR_NO_PAGES;
  else avail = p.num_free - free0;
  __syncthreads();
  int used = 0;                            // pages of the forks before
  for (int i0 = 0; i0 < p.count; i0 += kOpsThreads) {
    const int i = i0 + tid;
    int n = -1;
    if (i < p.count) {
      const int from = p.rows_from[i], to = p.rows_to[i];
      const bool ok = from >= 0 && from < p.num_seqs && to >= 0 && to < p.num_seqs && owner[to] == i &&
                      !(source[to >> 5] >> (to & 31) & 1);
      if (ok) {
        const int have = p.lens[from];
        n = p.fork_lens ? p.fork_lens[i] : have;
        if (n < 0 || n > have || have > cap) {
          err |= NSA_DEVERR_BAD_SEQLENS;
          n = -1;
        }
      } else {
        err |= NSA_DEVERR_BAD_INDEX;
      }
    }
    const int need = n > 0 && n % p.page ? 1 : 0;
    int total;
    const int at = used + cta_incl(need, part, total);   // inclusive
    used += total;
    if (i < p.count) {
      if (need && at > avail) {
        err |= NSA_DEVERR_NO_PAGES;
        n = -1;
      }
      lens[i] = n;
      place[i] = need && n >= 0 ? free0 + at - 1 : -1;
      if (need && n >= 0) atomicMax(&taken, at);
    }
  }
  if (rank != 0) err = 0;                  // every CTA has seen the same
  __syncthreads();
  if (ncta > 1) asm volatile("barrier.cluster.arrive.aligned;" ::: "memory");   // the head is read
  for (int i = rank * kOpsWarps + (tid >> 5); i < p.count; i += ncta * kOpsWarps) {
    const int n = lens[i];
    int src = -1, dst = -1;
    if (n >= 0) {
      const int to = p.rows_to[i], full = n / p.page;
      const int32_t *old = p.table + (int64_t)p.rows_from[i] * p.width;
      int32_t *row = p.table + (int64_t)to * p.width;
      if (lane == 0 && place[i] >= 0) {    // the last page, in part: one of its own
        src = old[full];
        dst = p.free_pages[place[i]];
      }
      for (int j0 = 0; j0 < full; j0 += 128) {
        int pg[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) pg[u] = j0 + u * 32 + lane < full ? old[j0 + u * 32 + lane] : 0;
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          if (j0 + u * 32 + lane >= full) continue;
          const bool good = pg[u] >= 0 && pg[u] < p.num_pages;
          if (good) atomicAdd(&p.shares[pg[u]], 1);
          else err |= NSA_DEVERR_BAD_INDEX;
          row[j0 + u * 32 + lane] = good ? pg[u] : -1;
        }
      }
      if (lane == 0) {
        if (place[i] >= 0) {
          const bool from = src >= 0 && src < p.num_pages, fresh = dst >= 0 && dst < p.num_pages;
          if (!(from && fresh)) err |= NSA_DEVERR_BAD_INDEX;
          row[full] = fresh ? dst : -1;
          src = from && fresh ? src : -1;
          dst = from && fresh ? dst : -1;
        }
        p.lens[to] = n;
      }
    }
    if (lane == 0) {
      p.copy_src[i] = src;
      p.copy_dst[i] = dst;
    }
  }
  report(p, err);
  if (ncta > 1) asm volatile("barrier.cluster.wait.aligned;" ::: "memory");
  if (rank == 0 && tid == 0) *p.head_out = free0 + taken;
}

// ---- bitmaps of pages, a slice of them a CTA -----------------------------------------------
struct PageBits {
  uint32_t base;                           // shared address of the CTA's own words
  int words;                               // of a slice, at least 2
  uint32_t inv;                            // 2^32 / words, rounded up or one more
  __device__ __forceinline__ PageBits(uint32_t base_, int words_)
      : base(base_), words(words_), inv(0xffffffffu / words_ + 1) {}
  __device__ __forceinline__ uint32_t addr(int word, int offset) const {
    // the product is off by word * words at most, less than 2^32 (2^17 words of 2^22 pages in all)
    const int cta = static_cast<int>(__umulhi(word, inv));
    return in_cta(base + offset + (word - cta * words) * 4, cta);
  }
  __device__ __forceinline__ void set(int page) const {
    asm volatile("red.relaxed.cluster.shared::cluster.or.b32 [%0], %1;" ::"r"(addr(page >> 5, 0)),
                 "r"(1u << (page & 31))
                 : "memory");
  }
};
__device__ __forceinline__ uint32_t ld_cluster(uint32_t a) {
  uint32_t v;
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(a) : "memory");
  return v;
}

// Prefix counts of the CTA's words: before[w] = bits set in the slice's words ahead of w.  Returns the
// slice's bits.  All threads take part.
__device__ __forceinline__ int count_words(const uint32_t *bits, int *before, int words,
                                           int (&part)[kOpsWarps]) {
  int sum = 0;
  for (int w0 = 0; w0 < words; w0 += kOpsThreads) {
    const int w = w0 + threadIdx.x, n = w < words ? __popc(bits[w]) : 0;
    int total;
    const int incl = cta_incl(n, part, total);
    if (w < words) before[w] = sum + incl - n;
    sum += total;
  }
  return sum;
}
// Bits of the slices ahead of this one, and of all, from the CTAs' counts (one shared word each): a lane
// reads one, not each thread all of them in turn (sixteen: 4000 cycles).
__device__ __forceinline__ void cluster_counts(const int *mine, int rank, int ncta, int &ahead,
                                               int &all) {
  const int lane = threadIdx.x & 31;
  const int n = lane < ncta ? static_cast<int>(ld_cluster(in_cta(smem_u32(mine), lane))) : 0;
  ahead = __reduce_add_sync(0xffffffffu, lane < rank ? n : 0);
  all = __reduce_add_sync(0xffffffffu, n);
}

// ---- free --------------------------------------------------------------------------------
__global__ void __launch_bounds__(kOpsThreads) page_free_kernel(PageOpsParams p, int words) {
  extern __shared__ int32_t sm[];
  uint32_t *bits = reinterpret_cast<uint32_t *>(sm);   // [words] pages whose last owner went
  int *before = sm + words;                            // [words]
  int *owner = before + words;                         // [B]
  __shared__ int part[kOpsWarps], mine;
  const int tid = threadIdx.x, lane = tid & 31, rank = blockIdx.x, ncta = gridDim.x;
  const PageBits map(smem_u32(bits), words);
  for (int w = tid; w < words; w += kOpsThreads) bits[w] = 0;
  after_previous();
  constexpr int kNone = INT32_MIN;
  const int first_i = rank * kOpsWarps + (tid >> 5), step = ncta * kOpsWarps;
  int r_l = kNone, len_l = 0;
  auto look = [&](int k0) {
    const int64_t i = first_i + (int64_t)(k0 + lane) * step;
    r_l = i < p.count ? p.rows_from[i] : kNone;
    if (r_l == kNone && i < p.count) r_l = -1;
    len_l = r_l >= 0 && r_l < p.num_seqs ? p.lens[r_l] : 0;
  };
  look(0);
  const int head = *p.head_in;
  first_owners(owner, p.rows_from, p.count, p.num_seqs);
  cluster_sync();                          // every slice is clear; owner is complete
  int32_t err = 0;
  // lane k has looked up the k-th of the warp's next 32 rows
  for (int k0 = 0; first_i + (int64_t)k0 * step < p.count; k0 += 32) {
    if (k0) look(k0);
    int row_l = 0, pages_l = 0;
    if (r_l != kNone) {
      int32_t bad = 0;
      if (r_l < 0 || r_l >= p.num_seqs || owner[r_l] != first_i + (k0 + lane) * step) {
        bad = NSA_DEVERR_BAD_INDEX;
      } else {
        pages_l = row_pages(p, len_l, bad);
        row_l = r_l;
        if (!bad) p.lens[r_l] = 0;
      }
      if (bad) pages_l = 0;                // passed over: left alone
      err |= bad;
    }
    const int turns = static_cast<int>(min((int64_t)32, (p.count - first_i - (int64_t)k0 * step + step - 1) / step));
    for (int k = 0; k < turns; ++k) {
      const int pages = __shfl_sync(0xffffffffu, pages_l, k);
      int32_t *row = p.table + (int64_t)__shfl_sync(0xffffffffu, row_l, k) * p.width;
      for (int j0 = lane; j0 < pages; j0 += 128) {
        int pg[4], had[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) pg[u] = j0 + u * 32 < pages ? row[j0 + u * 32] : 0;
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          had[u] = 1;
          if (j0 + u * 32 >= pages) continue;
          if (pg[u] >= 0 && pg[u] < p.num_pages) had[u] = atomicSub(&p.shares[pg[u]], 1);
          else err |= NSA_DEVERR_BAD_INDEX;
          row[j0 + u * 32] = -1;
        }
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          if (had[u] == 0) map.set(pg[u]);
          if (had[u] < 0) err |= NSA_DEVERR_BAD_INDEX;   // more rows named it than were counted
        }
      }
    }
  }
  cluster_sync();
  const int slice = count_words(bits, before, words, part);
  if (tid == 0) mine = slice;
  cluster_sync();
  int ahead, all;
  cluster_counts(&mine, rank, ncta, ahead, all);
  const bool ordered = head >= 0 && head <= p.num_free;
  const int first = ordered ? head - all : 0;          // below 0: no room for the first ones
  if (rank == 0 && tid == 0) {
    if (first < 0 || (!ordered && all > 0)) err |= NSA_DEVERR_NO_PAGES;
    *p.head_out = ordered ? max(first, 0) : head;
  }
  for (int w = tid; w < words; w += kOpsThreads) {
    int at = first + ahead + before[w];
    for (uint32_t m = bits[w]; m; m &= m - 1, ++at) {
      const int pg = (rank * words + w) * 32 + __ffs(m) - 1;
      p.shares[pg] = 0;
      if (ordered && at >= 0) p.free_pages[at] = pg;
    }
  }
  report(p, err);
  cluster_sync();                          // no CTA leaves while its count is read
}

// ---- compact -----------------------------------------------------------------------------
// f(row, pages, first, stride) for every row and class of kChunk-sized pieces of it, a warp each: a long
// row is shared by up to kSplit warps (500 rows of up to 512 pages, 22K in all: 2.3 us of 31).  Lane k
// looks up the length of the k-th of a warp's next 32.
constexpr int kSplit = 4;
template <int kChunk, typename F>
__device__ __forceinline__ void each_row(const PageOpsParams &p, int rank, int ncta, int32_t &err, F &&f) {
  const int lane = threadIdx.x & 31, step = ncta * kOpsWarps;
  const int split = min(kSplit, (p.width + kChunk - 1) / kChunk), tasks = p.num_seqs * split;
  for (int t0 = rank * kOpsWarps + (threadIdx.x >> 5); t0 < tasks; t0 += 32 * step) {
    const int t = t0 + lane * step, part_l = t / p.num_seqs, row_l = t - part_l * p.num_seqs;
    const int pages_l = t < tasks ? row_pages(p, p.lens[row_l], err) : 0;
    const int turns = min(32, (tasks - t0 + step - 1) / step);
    for (int k = 0; k < turns; ++k)
      f(__shfl_sync(0xffffffffu, row_l, k), __shfl_sync(0xffffffffu, pages_l, k),
        __shfl_sync(0xffffffffu, part_l, k) * kChunk, split * kChunk);
  }
}

__global__ void __launch_bounds__(kOpsThreads) page_compact_kernel(PageOpsParams p, int words) {
  extern __shared__ int32_t sm[];
  uint32_t *bits = reinterpret_cast<uint32_t *>(sm);   // [words] pages in use
  int *before = sm + words;                            // [words] then: of all pages ahead
  __shared__ int part[kOpsWarps], mine;
  const int tid = threadIdx.x, lane = tid & 31, rank = blockIdx.x, ncta = gridDim.x;
  const PageBits map(smem_u32(bits), words);
  for (int w = tid; w < words; w += kOpsThreads) bits[w] = 0;
  after_previous();
  cluster_sync();
  int32_t err = 0;
  each_row<128>(p, rank, ncta, err, [&](int r, int pages, int first, int stride) {
    const int32_t *row = p.table_in + (int64_t)r * p.width;
    for (int j0 = first; j0 < pages; j0 += stride) {
      int pg[4];
#pragma unroll
      for (int u = 0; u < 4; ++u) pg[u] = j0 + u * 32 + lane < pages ? row[j0 + u * 32 + lane] : -1;
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        if (pg[u] >= 0 && pg[u] < p.num_pages) map.set(pg[u]);
        else if (j0 + u * 32 + lane < pages) err |= NSA_DEVERR_BAD_INDEX;
      }
    }
  });
  cluster_sync();
  const int slice = count_words(bits, before, words, part);
  if (tid == 0) mine = slice;
  cluster_sync();
  int ahead, live;
  cluster_counts(&mine, rank, ncta, ahead, live);
  for (int w = tid; w < words; w += kOpsThreads) before[w] += ahead;
  cluster_sync();
  // pages in use below page x (x < 32 * words * ncta)
  auto below = [&](int x) {
    const int w = x >> 5;
    return static_cast<int>(ld_cluster(map.addr(w, words * 4))) +
           __popc(ld_cluster(map.addr(w, 0)) & ((1u << (x & 31)) - 1u));
  };
  const int spare = p.num_pages - live;                // pages that end up free
  const int stay = live < p.num_pages ? below(live) : live;   // of those in use, below the new end
  const int moves = live - stay;
  const bool fits = moves <= p.count && spare <= p.num_free;
  if (!fits && rank == 0 && tid == 0) err |= NSA_DEVERR_NO_PAGES;
  const int me = rank * kOpsThreads + tid, all = ncta * kOpsThreads;
  // lists: the i-th page in use behind the end, the i-th unused one ahead of it
  if (fits) {
    for (int w = tid; w < words; w += kOpsThreads) {
      const int x0 = (rank * words + w) * 32;
      int used = before[w];                            // in use ahead of the bit at hand
      for (int k = 0; k < 32 && x0 + k < p.num_pages; ++k) {
        const int x = x0 + k;
        const bool in = bits[w] >> k & 1;
        if (x >= live && in) p.copy_src[used - stay] = x;
        if (x < live && !in) p.copy_dst[x - used] = x;
        used += in;
      }
    }
    for (int i = me; i < spare; i += all) p.free_pages[p.num_free - spare + i] = live + i;
    if (rank == 0 && tid == 0) *p.head_out = p.num_free - spare;
  }
  for (int i = me + (fits ? moves : 0); i < p.count; i += all) p.copy_src[i] = p.copy_dst[i] = -1;
  cluster_sync();                                      // the lists are complete
  // counts: a page that moves takes its own along
  for (int x = me; x < p.num_pages; x += all) {
    if (!fits) {
      if (p.shares != p.shares_in) p.shares[x] = p.shares_in[x];
      continue;
    }
    const bool in = ld_cluster(map.addr(x >> 5, 0)) >> (x & 31) & 1;
    if (x < live) {
      if (in && p.shares != p.shares_in) p.shares[x] = p.shares_in[x];
    } else {
      if (in) p.shares[p.copy_dst[below(x) - stay]] = p.shares_in[x];
      p.shares[x] = 0;
    }
  }
  const bool apart = p.table != p.table_in;
  constexpr int kAtOnce = 8;
  int32_t again = 0;                                   // reported above
  each_row<32 * kAtOnce>(p, rank, ncta, again, [&](int r, int pages, int first, int stride) {
    const int32_t *row = p.table_in + (int64_t)r * p.width;
    int32_t *out = p.table + (int64_t)r * p.width;
    const int end = apart ? p.width : pages;
    for (int j0 = first + lane; j0 < end; j0 += stride) {   // the steps of kAtOnce lookups side by side
      int pg[kAtOnce], to[kAtOnce];
#pragma unroll
      for (int u = 0; u < kAtOnce; ++u) pg[u] = j0 + 32 * u < end ? row[j0 + 32 * u] : -1;
#pragma unroll
      for (int u = 0; u < kAtOnce; ++u) {
        const bool moved = fits && j0 + 32 * u < pages && pg[u] >= live && pg[u] < p.num_pages;
        to[u] = moved ? below(pg[u]) - stay : -1;
      }
#pragma unroll
      for (int u = 0; u < kAtOnce; ++u) to[u] = to[u] >= 0 ? p.copy_dst[to[u]] : -1;
#pragma unroll
      for (int u = 0; u < kAtOnce; ++u) {
        if (to[u] >= 0) out[j0 + 32 * u] = to[u];
        else if (apart && j0 + 32 * u < end) out[j0 + 32 * u] = pg[u];
      }
    }
  });
  report(p, err);
  cluster_sync();                                      // no CTA leaves while its words are read
}

// ---- copies ------------------------------------------------------------------------------
// A CTA takes pieces of kPiece bytes at most, in turn; each warp looks 32 of them up at once, so
// that entries of -1 cost next to nothing.
constexpr int kCopyThreads = 256, kCopyEach = 4;
constexpr int kPiece = kCopyThreads * kCopyEach * 16;

__global__ void __launch_bounds__(kCopyThreads) page_copy_kernel(int num_pages, int64_t page_bytes,
                                                                 int64_t tasks, int pieces, int piece,
                                                                 uint8_t *pool, const int32_t *src,
                                                                 const int32_t *dst, int32_t *status) {
  const int tid = threadIdx.x, lane = tid & 31;
  after_previous();
  bool bad = false;
  for (int64_t t0 = blockIdx.x; t0 < tasks; t0 += 32ll * gridDim.x) {
    const int64_t t = t0 + (int64_t)lane * gridDim.x;
    int a = -1, b = -1, at = 0;
    if (t < tasks) {
      const int64_t i = t / pieces;
      a = src[i];
      b = dst[i];
      at = static_cast<int>(t - i * pieces);
      if (a != -1 || b != -1) {
        const bool ok = a >= 0 && a < num_pages && b >= 0 && b < num_pages;
        bad |= !ok;
        if (!ok) a = -1;
      }
    }
    for (uint32_t m = __ballot_sync(0xffffffffu, a >= 0); m; m &= m - 1) {
      const int k = __ffs(m) - 1;
      const int from = __shfl_sync(0xffffffffu, a, k), to = __shfl_sync(0xffffffffu, b, k);
      const int64_t off = (int64_t)__shfl_sync(0xffffffffu, at, k) * piece;
      const int size = static_cast<int>(min((int64_t)piece, page_bytes - off));
      const uint8_t *s = pool + from * page_bytes + off;
      uint8_t *d = pool + to * page_bytes + off;
      uint4 v[kCopyEach];
#pragma unroll
      for (int u = 0; u < kCopyEach; ++u)
        if ((u * kCopyThreads + tid) * 16 < size)
          v[u] = *reinterpret_cast<const uint4 *>(s + (u * kCopyThreads + tid) * 16);
#pragma unroll
      for (int u = 0; u < kCopyEach; ++u)
        if ((u * kCopyThreads + tid) * 16 < size)
          *reinterpret_cast<uint4 *>(d + (u * kCopyThreads + tid) * 16) = v[u];
    }
  }
  if (__any_sync(0xffffffffu, bad) && tid == 0) raise(status, NSA_DEVERR_BAD_INDEX);
}

// ---- launches ----------------------------------------------------------------------------
// One CTA where the rows have few entries and the pages a small bitmap, else a wide cluster.  smem(ctas):
// what the call takes, most: what the largest does.
template <typename S, typename... P, typename... A>
static cudaError_t run_op(void (*kernel)(P...), WideKernel which, int64_t entries, int num_pages, S &&smem,
                          size_t most, cudaStream_t s, A &&...args_of) {
  int ctas = 1;
  cudaError_t e = cudaSuccess;
  if (entries > 4096 || num_pages > 65536)
    e = wide_cluster(which, reinterpret_cast<const void *>(kernel), kOpsThreads, most, &ctas);
  else if (smem(1) > 40 * 1024)            // the limit is the kernel's (pages.cu)
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(most));
  if (e != cudaSuccess) return e;
  return launch_kv4(kernel, dim3(static_cast<unsigned>(ctas)), kOpsThreads, smem(ctas), ctas, s, args_of(ctas)...);
}

cudaError_t launch_page_op(PageOp op, const PageOpsParams &p, cudaStream_t s) {
  // of the largest calls, with a cluster of eight
  constexpr size_t kRows = kMaxPlanSeqs, kWords = kMaxOpsPages / 32 / 8 + 1;
  auto same = [&](int) { return p; };
  auto words = [&](int ctas) { return max(2, (p.num_pages / 32 + ctas) / ctas); };   // a word past the last page, too
  switch (op) {
    case PageOp::kFork:
      return run_op(page_fork_kernel, kWideFork, (int64_t)p.count * p.width, 0,
                    [&](int) { return 4 * (p.num_seqs + 2 * (size_t)p.count + (p.num_seqs + 31) / 32); },
                    4 * (3 * kRows + kRows / 32), s, same);
    case PageOp::kFree:
      return run_op(page_free_kernel, kWideFree, (int64_t)p.count * p.width, p.num_pages,
                    [&](int ctas) { return 8 * (size_t)words(ctas) + 4 * (size_t)p.num_seqs; },
                    8 * kWords + 4 * kRows, s, same, words);
    default:
      return run_op(page_compact_kernel, kWideCompact, (int64_t)p.num_seqs * p.width, p.num_pages,
                    [&](int ctas) { return 8 * (size_t)words(ctas); }, 8 * kWords, s, same, words);
  }
}

cudaError_t launch_page_copy(int num_pages, int64_t page_bytes, int n, void *pool, const int32_t *src,
                             const int32_t *dst, int32_t *status, cudaStream_t s) {
  int dev = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return e;
  const int64_t pieces = (page_bytes + kPiece - 1) / kPiece;
  const int piece = static_cast<int>((page_bytes / 16 + pieces - 1) / pieces * 16);   // even pieces
  const int64_t tasks = n * pieces, ctas = min(tasks, (int64_t)sms * 8);
  return launch_kv4(page_copy_kernel, dim3(static_cast<unsigned>(ctas)), kCopyThreads, 0, 1, s, num_pages,
                    page_bytes, tasks, static_cast<int>(pieces), piece, static_cast<uint8_t *>(pool),
                    src, dst, status);
}

}  // namespace nsa
