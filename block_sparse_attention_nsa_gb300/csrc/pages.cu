// pages.cu -- block tables and slot maps built on the GPU from request lengths.
//
// With P tokens a page, request b takes need_b = ceil((ctx + new) / P) - ceil(ctx / P)
// pages from a free list; two exclusive scans over the requests, of need_b and of new_b,
// give its place in the free list and in the packed slot map; every new token's slot is
// then a lookup:
//   slot = page(pos / P) * P + pos % P,   pos = ctx + its index among the new tokens,
// where the page is a free one (pos / P >= ceil(ctx / P)) or stands in the table already.
// The token that opens a page writes the table entry.
//
// A few bytes per request and slot: what counts is latency.  One launch: every CTA scans
// all requests for itself (offsets kept in shared memory, so that a slot's request is
// found there by bisection) and fills its share of the slots, four a thread at a time.  Up to 4096
// slots one CTA does it all; above, a cluster shares the slots: of eight CTAs where one turn of their
// threads is enough (32768 slots), else of sixteen, for which a call has to allow a launch first, 0.4 us
// of host time (64 decode steps 4.5 us, 1000 mixed requests with 22K slots 7.2, with sixteen too; with 40K
// 7.2 against eight's 10.1, with 312K 18.5 against 32.2; in a CUDA graph, launch included).  The outputs
// that may be the inputs' own arrays (seq_lens = ctx_lens, head_out = free_head) are written by the first
// CTA behind a cluster barrier that every CTA reaches after its last read of them.
#include <atomic>

#include "kv4.cuh"

namespace nsa {

constexpr int kPlanThreads = 1024;
constexpr int kPlanOneCta = 4096;                    // slots up to which one CTA fills the map
constexpr int kPlanEight = 8 * kPlanThreads * 4;      // and up to which eight do

__device__ __forceinline__ int64_t warp_incl(int64_t x, int lane) {
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  return x;
}

// kPlan: take pages from the free list; else the tokens are in the cache already.
template <bool kPlan>
__global__ void __launch_bounds__(kPlanThreads) page_kernel(PageParams p) {
  extern __shared__ int32_t psm[];
  int32_t *cu = psm;                        // [B + 1]
  int32_t *start = cu + p.num_seqs + 1;     // [B] first position, held to the table
  int32_t *head = start + p.num_seqs;       // [B] place in the free list, -1: refused
  __shared__ int64_t tot[2][32];
  __shared__ int taken;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int rank = blockIdx.x, ncta = gridDim.x;
  const int64_t cap = (int64_t)p.width * p.page;   // tokens that a table row can hold
  after_previous();
  int free0 = 0, avail = 0;
  int32_t err = 0;
  if (kPlan) {
    free0 = *p.free_head;
    if (free0 < 0 || free0 > p.num_free) err |= NSA_DEVERR_NO_PAGES;
    else avail = p.num_free - free0;
  }
  if (tid == 0) taken = 0;
  int64_t tok0 = 0, need0 = 0;              // tokens and pages of the earlier requests
  for (int b0 = 0; b0 < p.num_seqs; b0 += kPlanThreads) {
    const int b = b0 + tid;
    const bool in = b < p.num_seqs;
    const int c = in ? p.ctx[b] : 0, a = in ? p.add[b] : 0;
    const bool ok = c >= 0 && a >= 0 && (int64_t)c + a <= cap;
    const int n = max(a, 0);
    int64_t need = 0;
    if (kPlan && ok) need = ((int64_t)c + a + p.page - 1) / p.page - ((int64_t)c + p.page - 1) / p.page;
    int64_t ti = warp_incl(n, lane), ni = warp_incl(need, lane);
    __syncthreads();                        // the totals of the chunk before have been read
    if (lane == 31) {
      tot[0][warp] = ti;
      tot[1][warp] = ni;
    }
    __syncthreads();
    const int64_t t32 = warp_incl(tot[0][lane], lane), n32 = warp_incl(tot[1][lane], lane);
    const int64_t tb = __shfl_sync(0xffffffffu, t32, (warp + 31) & 31);
    const int64_t nb = __shfl_sync(0xffffffffu, n32, (warp + 31) & 31);
    ti += tok0 + (warp ? tb : 0);           // inclusive over all requests so far
    ni += need0 + (warp ? nb : 0);
    tok0 += __shfl_sync(0xffffffffu, t32, 31);
    need0 += __shfl_sync(0xffffffffu, n32, 31);
    if (in) {
      const bool room = n == 0 || ti <= p.max_slots;
      const bool paged = need == 0 || ni <= avail;
      if (!ok) err |= NSA_DEVERR_BAD_SEQLENS;
      if (ok && !(room && paged)) err |= NSA_DEVERR_NO_PAGES;
      const bool served = ok && room && paged;
      cu[b] = static_cast<int32_t>(min(ti - n, (int64_t)p.max_slots));
      if (b == p.num_seqs - 1) cu[b + 1] = static_cast<int32_t>(min(ti, (int64_t)p.max_slots));
      start[b] = static_cast<int32_t>(min((int64_t)max(c, 0), cap));
      head[b] = !served ? -1 : need > 0 ? free0 + static_cast<int32_t>(ni - need) : 0;
      if (served && need > 0) atomicMax(&taken, static_cast<int>(ni));
    }
  }
  if (rank == 0 && err) raise(p.status, err);
  __syncthreads();
  // every CTA has read ctx, new and the free list's head
  if (ncta > 1) asm volatile("barrier.cluster.arrive.aligned;" ::: "memory");

  const int total = cu[p.num_seqs];
  const bool wide = (reinterpret_cast<uintptr_t>(p.slots) & 15) == 0;
  bool bad = false;
  for (int64_t t0 = ((int64_t)rank * kPlanThreads + tid) * 4; t0 < p.max_slots;
       t0 += (int64_t)ncta * kPlanThreads * 4) {
    // the four tokens' pages are looked up together
    const int32_t *from[4];
    int32_t *open[4];
    uint32_t rest[4];
    int32_t out[4];
    int b = t0 < total ? upper_index(cu, p.num_seqs, static_cast<int>(t0)) : 0;
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int t = static_cast<int>(min(t0 + u, (int64_t)INT32_MAX));
      from[u] = nullptr;
      open[u] = nullptr;
      rest[u] = 0;
      if (t < total) {
        while (t >= cu[b + 1]) ++b;         // t < total = cu[B]: b stays below B
        const int h = head[b];
        const uint32_t c = start[b], pos = c + static_cast<uint32_t>(t - cu[b]);
        const uint32_t j = pos / p.page, have = (c + p.page - 1) / p.page;
        rest[u] = pos - j * p.page;
        if (h >= 0) {
          int32_t *entry = p.table + (int64_t)b * p.width + j;
          const bool fresh = kPlan && j >= have;
          from[u] = fresh ? p.free_pages + h + (j - have) : entry;
          if (fresh && rest[u] == 0) open[u] = entry;
        }
      }
    }
    int pg[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) pg[u] = from[u] ? *from[u] : -1;
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const bool good = pg[u] >= 0 && pg[u] < p.num_pages;
      if (open[u]) *open[u] = good ? pg[u] : -1;
      out[u] = good ? static_cast<int32_t>(pg[u] * p.page + rest[u]) : -1;
      bad |= from[u] && !good;
    }
    if (wide && t0 + 4 <= p.max_slots) {
      *reinterpret_cast<int4 *>(p.slots + t0) = make_int4(out[0], out[1], out[2], out[3]);
    } else {
#pragma unroll
      for (int u = 0; u < 4; ++u)
        if (t0 + u < p.max_slots) p.slots[t0 + u] = out[u];
    }
  }
  if (__any_sync(0xffffffffu, bad) && lane == 0) raise(p.status, NSA_DEVERR_BAD_INDEX);
  if (ncta > 1) asm volatile("barrier.cluster.wait.aligned;" ::: "memory");
  if (rank == 0) {
    for (int b = tid; b < p.num_seqs; b += kPlanThreads) {
      p.cu_out[b] = cu[b];
      if (kPlan) p.seq_out[b] = start[b] + (head[b] >= 0 ? cu[b + 1] - cu[b] : 0);
    }
    if (tid == 0) {
      p.cu_out[p.num_seqs] = total;
      if (kPlan) *p.head_out = free0 + taken;
    }
  }
}

cudaError_t wide_cluster(WideKernel which, const void *kernel, int threads, size_t smem, int *ctas) {
  static std::atomic<int> known[kWideKernels][64];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
  if (e == cudaSuccess) e = cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
  if (e != cudaSuccess) return e;
  const bool keep = dev >= 0 && dev < 64;
  *ctas = keep ? known[which][dev].load(std::memory_order_relaxed) : 0;
  if (*ctas) return cudaSuccess;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(kWideCluster);
  cfg.blockDim = dim3(static_cast<unsigned>(threads));
  cfg.dynamicSmemBytes = smem;
  cudaLaunchAttribute at;
  at.id = cudaLaunchAttributeClusterDimension;
  at.val.clusterDim.x = kWideCluster;
  at.val.clusterDim.y = at.val.clusterDim.z = 1;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  int clusters = 0;
  if (cudaOccupancyMaxActiveClusters(&clusters, kernel, &cfg) != cudaSuccess) {
    cudaGetLastError();                    // none, then
    clusters = 0;
  }
  *ctas = clusters > 0 ? kWideCluster : 8;
  if (keep) known[which][dev].store(*ctas, std::memory_order_relaxed);
  return cudaSuccess;
}

cudaError_t launch_pages(const PageParams &p, bool plan, cudaStream_t s) {
  auto *kernel = plan ? page_kernel<true> : page_kernel<false>;
  const size_t smem = (3 * static_cast<size_t>(p.num_seqs) + 1) * sizeof(int32_t);
  constexpr size_t kMost = (3 * static_cast<size_t>(kMaxPlanSeqs) + 1) * sizeof(int32_t);
  int ctas = 1;
  cudaError_t e = cudaSuccess;
  if (p.max_slots > kPlanEight) {
    e = wide_cluster(plan ? kWidePlan : kWideSlots, reinterpret_cast<const void *>(kernel), kPlanThreads,
                     kMost, &ctas);
  } else if (smem > 40 * 1024) {
    // the largest plan's, whatever this one's: the limit is the kernel's, and another host thread may
    // be between its own and its launch
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(kMost));
  }
  if (e != cudaSuccess) return e;
  if (p.max_slots > kPlanOneCta && p.max_slots <= kPlanEight) ctas = 8;
  return launch_kv4(kernel, dim3(ctas), kPlanThreads, smem, ctas, s, p);
}

}  // namespace nsa
