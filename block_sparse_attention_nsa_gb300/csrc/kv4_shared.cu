// kv4_shared.cu -- one-step decode over the 4-bit pages for sequences that share a prefix.
//
// The sequences of a group have the same first tokens, in the same pages.  Softmax over a sequence's
// keys splits at the prefix' end into two sums that are joined by their maxima:
//   out = (sum_prefix w v + sum_own w v) / (sum_prefix w + sum_own w),   w = exp(S - max S).
// The prefix' part is a product of all the group's query rows with the same keys, done once per 128
// rows on the tensor cores; each sequence's own part is kv4_decode.cu's, from the prefix' end on.
//
// Prefix kernel (tcgen05).  Rows of a KV head's tile are (sequence, query head) pairs, M = 128; 128
// keys a block.  The scores' sums are the tensor core's alone, as exact as fp32 products (their
// log-sum-exp is returned in fp32).  With q^ = q 2^(5 - ex), ex the exponent of a row's largest
// magnitude (in fp16 it loses 2^-30 of that), and k = c s + z in a group of dimensions,
//   q^ . k = sum_j q^_j (c_j - 8) s_hi + sum_j q^_j (c_j - 8) s_lo + Q z + 8 Q s,   Q = sum_j q^_j:
// s_hi is s without its last three bits, so that both products with c - 8 (four bits and a sign) are
// exact in fp16; Q and 8 Q are three fp16 numbers each, against z and s in 12 of the 16 columns of
// one more step; a 13th has the mask.  S = |scale| 2^(ex - 5) q^ . k.  (Codes as operands, with scales
// and zeros taken in fp32 afterwards, want both groups' accumulators apart and four numbers a key from
// shared memory for every thread: 3190 cycles for 64 keys.)
// Weights are w = 2^(S - m) 2^8 (with their factor those down to 2^-22 of the maximum are normal
// numbers in fp16).  Two roundings to fp16, of 2^-11 at most each: V's values as they are unpacked, and
// the weights, for bf16 outputs, whose own rounding is eight times as large.  For fp16 outputs, of
// the same size, W is the sum of two fp16 numbers: with W in one part the error over a long prefix
// was 1.66 times that of the output's rounding alone, with two 1.4.  Sums of weights are fp32, of
// the weights before they are rounded.
// The tensor core cuts its sums towards zero, an error of one sign that grows with its steps (8 a block, 16
// for fp16 outputs).  So its sums run over 2048 steps at most (256 blocks; 1024, 64 blocks, for fp16), and are
// added to the tile's partial rows in fp32: after 4096 blocks outputs are 1.32 (fp16) and 1.02 times (bf16)
// their own rounding off, 1.02 and 1.00 for V around 1; with one sum 5.3 and 1.07, 11.5 and 1.75, in 0 to 3 %
// less time.
// The maximum m is raised only when a score passes it by 2^4, so that most blocks rescale nothing.
//
// Roles of a CTA (one an SM, 20 warps), handing blocks on by mbarriers, every wait bounded:
//   loader       a block's record tiles by bulk copies into a ring, page by page of the table;
//   8 unpackers  codes, scales and zeros to the K and V operands (128-byte swizzle; the eight
//                dimensions of a word stay in the order 0 4 1 5 2 6 3 7 that masking gives, on both
//                sides of the product and until the output is written).  Where there is room for two
//                blocks' V, half the warps take every second block: a warp waits on the latency of
//                what it does, and has half the barriers a block (181 us to 169, 256 behind 32K);
//   MMA warp     S = Q K^T of block n + 1 into one of two score buffers, then O += W V of block n.  Q
//                and W come from tensor memory, so that only K and V are read from shared memory.
//                A step of N = 128 takes the tensor core 64 cycles (one of 64 takes 48, and only one
//                output fits beside two buffers of 128 scores); the 25 of a block took one thread
//                2800 cycles to issue, its operands moved to uniform registers each time, on a
//                scheduler that it shares with four other warps.  So the whole warp runs the loop with
//                operands the same in all lanes, and one lane issues: 212 us to 181;
//   2 x 4 softmax warps   a thread a row and half of a block's keys.  Both halves share the output
//                and so the reference m: one barrier a block tells them whether any row raises it.
//                W goes to tensor memory over the scores it came from.
// Two CTAs as a pair (D = 128, more than 128 rows a group on average): M = 256, a CTA's softmax on 128
// of the rows, and each unpacks half of a block's K and one group of V's dimensions, which the tensor
// cores of both read.  The CTA of rank 0 issues for both; arrivals on what it waits for go to its
// barriers, commits to both CTAs'.  Those arrivals release at their own CTA's scope, which the memory
// model orders for threads of that CTA alone.  They rely on this: what they report is read by nobody but
// their own SM's tensor core, and is complete before they are issued (shared memory behind each writer's
// proxy fence, tensor memory behind tcgen05.wait::st, both behind the warp's barrier).  A release at the
// cluster's scope takes about 900 cycles: 256 behind 32K 220 us in the place of 167; arrivals within each
// CTA, passed on by a warp of the second one with that release, 203.  At D = 64 half of V's dimensions
// would be half a swizzle row.
// A block takes about 2300 cycles in a pair and 3350 alone, against 1600 of the tensor core's.  Alone
// the unpackers are the longest; in a pair no role is busy all the time, each waits on the others'
// latencies.  256 sequences of 8 x 4 heads behind 32K tokens: 140 us, 981 TFLOP/s of what the formula
// wants and 1534 with the products of s_lo and the sums; the tensor pipe is busy 68 % of the time.
// Work: the line of all (tile, block) pairs, tile after tile, in equal runs, one a CTA or pair; where a
// tile is shared by runs each leaves partial rows.  kv4_join_kernel adds them and the own part.
#include <cmath>
#include <type_traits>
#include <utility>

#include "kv4.cuh"

namespace nsa {

constexpr int kShRows = 128;         // query rows of a tile
constexpr int kShKeys = 128;         // keys of a block
constexpr int kShTiles = kShKeys / kKv4Tile;
constexpr int kShThreads = 640;
constexpr int kShMaxCtas = 256;
constexpr int kShOver = 2;           // blocks that a tile's start and end count as
constexpr float kShSlack = 4.f;      // scores may exceed the reference by this much
constexpr float kShUp = 8.f;         // weights are 2^8 times 2^(S - m)
constexpr int kShQTop = 5;           // exponent of a row's largest q^
constexpr int kShMulTop = 92;        // a score's factor stays below 2^(kShMulTop + 2), scores in its unit below 2^30

// A group that shares: its first sequence and number of rows per KV head, its blocks and tiles, and
// what lies before it: counted blocks (kShOver a tile more than there are), and partial rows.  ended: the
// first sequence is shorter than the prefix.
struct ShGroup {
  int32_t seq0, rows, blocks, tiles, keys, pair0, row0, ended;
  __device__ __forceinline__ int counted() const { return blocks + kShOver; }
};
struct ShHead {
  int32_t groups, pairs, per, rows_log2;   // counted blocks; of them a CTA's (a pair's); rows of a tile
};
struct ShPlan {
  ShHead *head;
  ShGroup *groups;                   // [num_groups]
  int32_t *lo, *of;                  // [num_seqs]: first own key; group in `groups`, -1: none
  int32_t *at;                       // [num_groups]: place of a group in `groups`
  float *rec, *part;                 // records of the own parts, partial rows of the prefixes
  float2 *part_ml;
};

static int64_t up16(int64_t x) { return (x + 15) / 16 * 16; }
static int64_t partial_rows(int num_seqs, int h_q) {
  return (int64_t)kShMaxCtas * kShRows + (int64_t)num_seqs * h_q;
}
// The plan's places in a workspace, and its bytes.
static int64_t shared_layout(int d, int num_seqs, int h_q, int num_groups, uint8_t *ws, ShPlan *p) {
  int64_t at = 0;
  auto take = [&](int64_t bytes) {
    const int64_t x = at;
    at += up16(bytes);
    return ws + x;
  };
  ShPlan q;
  q.head = reinterpret_cast<ShHead *>(take(sizeof(ShHead)));
  q.groups = reinterpret_cast<ShGroup *>(take((int64_t)num_groups * sizeof(ShGroup)));
  q.lo = reinterpret_cast<int32_t *>(take(4 * (int64_t)num_seqs));
  q.of = reinterpret_cast<int32_t *>(take(4 * (int64_t)num_seqs));
  q.at = reinterpret_cast<int32_t *>(take(4 * (int64_t)num_groups));
  q.rec = reinterpret_cast<float *>(take((int64_t)num_seqs * h_q * (d + 4) * 4));
  q.part_ml = reinterpret_cast<float2 *>(take(partial_rows(num_seqs, h_q) * 8));
  q.part = reinterpret_cast<float *>(take(partial_rows(num_seqs, h_q) * d * 4));
  if (p) *p = q;
  return at;
}

// ---- the plan --------------------------------------------------------------------------
constexpr int kSetupThreads = 1024;
constexpr int kShOwnPlan = 256;      // groups up to which every CTA of the prefix kernel plans for itself

// Inclusive prefixes of three numbers over a CTA of kWarps warps; total gets the sums.
template <int kWarps>
__device__ __forceinline__ void setup_incl(int (&x)[3], int (&part)[3][32], int (&total)[3]) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
#pragma unroll
    for (int k = 0; k < 3; ++k) {
      const int y = __shfl_up_sync(0xffffffffu, x[k], o);
      if (lane >= o) x[k] += y;
    }
  }
  __syncthreads();                         // the totals of the call before have been read
  if (lane == 31)
#pragma unroll
    for (int k = 0; k < 3; ++k) part[k][warp] = x[k];
  __syncthreads();
#pragma unroll
  for (int k = 0; k < 3; ++k) {
    const int w = lane < kWarps ? part[k][lane] : 0;
    total[k] = static_cast<int>(__reduce_add_sync(0xffffffffu, w));
    x[k] += static_cast<int>(__reduce_add_sync(0xffffffffu, lane < warp ? w : 0));
  }
}

// Blocks of a prefix: without a sum past 2^31, which keys may be next to.
__device__ __forceinline__ int blocks_of(int keys) { return keys / kShKeys + (keys % kShKeys != 0); }

// Shared or not?  In units of 25 ns of an SM's time: a tile of 128 rows takes about 240 and 72 a block
// of 128 keys, one of 256 rows, of a pair, twice 240 and 50; the sequences' own passes over the prefix
// take 5 a tile of 32 keys each.
__device__ __forceinline__ bool worth_sharing(int n, int g, int keys, int rows_log2) {
  const int64_t own = (int64_t)n * (g > kK4Heads ? 2 : 1) * ((keys + 31) / 32) * 5;
  const int64_t tiles = ((int64_t)n * g + (1 << rows_log2) - 1) >> rows_log2;
  const int64_t blocks = blocks_of(keys);
  return n > 1 && own > tiles * ((1 << rows_log2) == kShRows ? 240 + 72 * blocks : 480 + 100 * blocks);
}

// By a CTA of kThreads: groups that share, in order, with what lies before each, into `groups`, and of
// every group whether it is ordered and its place there (-1: none) into `at`.  A cu_groups out of order
// shares nothing.  Returns the head (per: CTAs have equal runs, of a block at least).
template <int kThreads>
__device__ __forceinline__ ShHead make_plan(const Kv4SharedParams &p, ShGroup *groups, int32_t *at, int ctas,
                                            int rows_log2, int (&part)[3][32], int32_t &err) {
  constexpr int kWarps = kThreads / 32;
  const int cap = p.dec.width << p.dec.page_log2;
  const bool once = p.num_groups <= kThreads;                  // every thread has one group at most
  auto out_of_order = [&](int i, int a, int b) { return a < 0 || (i == 0 && a != 0) || b < a || b > p.dec.num_seqs; };
  bool ordered = true;
  if (!once) {
    bool bad = false;
    for (int i = threadIdx.x; i < p.num_groups; i += kThreads) bad |= out_of_order(i, p.cu[i], p.cu[i + 1]);
    ordered = !__syncthreads_or(bad);
  }
  int sum[3] = {0, 0, 0};                                      // groups, counted blocks, rows
  for (int i0 = 0; i0 < p.num_groups; i0 += kThreads) {
    const int i = i0 + threadIdx.x;
    int n = 0, keys = 0, a = 0, len = 0;
    bool bad = false;
    if (i < p.num_groups) {
      a = p.cu[i];
      const int b = p.cu[i + 1];
      keys = p.prefix[i];
      bad = out_of_order(i, a, b);
      n = b - a;
      if (!bad && n > 0) len = p.dec.lens[a];
    }
    if (once) ordered = !__syncthreads_or(bad);
    if (ordered && (keys < 0 || keys > cap)) err |= NSA_DEVERR_BAD_SEQLENS;
    if (!ordered || keys < 0 || keys > cap) keys = 0;
    const bool shares = keys > 0 && worth_sharing(n, p.dec.g, keys, rows_log2);
    const int r = shares ? n * p.dec.g : 0, tiles = (r + (1 << rows_log2) - 1) >> rows_log2;
    const int blocks = blocks_of(keys);
    const int mine[3] = {shares, tiles * p.dec.h_k * (blocks + kShOver), r * p.dec.h_k};
    int x[3] = {mine[0], mine[1], mine[2]}, total[3];
    setup_incl<kWarps>(x, part, total);
#pragma unroll
    for (int k = 0; k < 3; ++k) x[k] += sum[k] - mine[k];
    if (i < p.num_groups) at[i] = shares ? x[0] : -1;
    if (shares) groups[x[0]] = ShGroup{a, r, blocks, tiles, keys, x[1], x[2], len < keys};
#pragma unroll
    for (int k = 0; k < 3; ++k) sum[k] += total[k];
  }
  if (!ordered) err |= NSA_DEVERR_BAD_SEQLENS;
  __syncthreads();
  return ShHead{sum[0], sum[1], max((sum[1] + ctas - 1) / ctas, kShOver + 1), rows_log2};
}

// Sequence b's group among those that share, and its first own key.  One that ends inside the prefix
// attends to its own pages alone.
__device__ __forceinline__ void place_sequence(const Kv4SharedParams &p, const ShPlan &plan, const ShHead &head,
                                               const ShGroup *groups, const int32_t *at, int b) {
  int g = -1, lo = 0;
  if (head.groups > 0 && b < p.cu[p.num_groups]) {
    g = at[upper_index(p.cu, p.num_groups, b)];
    if (g >= 0) {
      const int keys = groups[g].keys, cap = p.dec.width << p.dec.page_log2;
      if (min(max(p.dec.lens[b], 0), cap) >= keys) lo = keys;
      else g = -1;
    }
  }
  plan.lo[b] = lo;
  plan.of[b] = g;
}

// For more groups than the prefix kernel's CTAs plan themselves.
__global__ void __launch_bounds__(kSetupThreads) kv4_share_kernel(Kv4SharedParams p, ShPlan plan, int ctas,
                                                                int rows_log2) {
  __shared__ int part[3][32];
  after_previous();
  int32_t err = 0;
  const ShHead head = make_plan<kSetupThreads>(p, plan.groups, plan.at, ctas, rows_log2, part, err);
  if (__syncthreads_or(err) && threadIdx.x == 0) raise(p.dec.status, NSA_DEVERR_BAD_SEQLENS);
  if (threadIdx.x == 0) *plan.head = head;
  for (int b = threadIdx.x; b < p.dec.num_seqs; b += kSetupThreads)
    place_sequence(p, plan, head, plan.groups, plan.at, b);
}

// ---- prefix ----------------------------------------------------------------------------
template <int D, bool kPair>
struct Sh {
  using T = Kv4Tile<D>;
  static constexpr int kG = T::kG;
  // Blocks copied ahead; K and V unpacked.  A set of unpackers uses stages of its own, phase by phase: a
  // parity tells only the last two phases apart.
  static constexpr int kSets = kPair || D == 64 ? 2 : 1;       // of unpackers, which take blocks in turn
  static constexpr int kUnpackers = 256 / kSets;
  static constexpr int kRaw = kPair ? 4 : 2, kK = 2, kV = kSets;
  static_assert(kRaw % kSets == 0 && kK % kSets == 0, "stages of its own");
  static constexpr int kKeys = kPair ? kShKeys / 2 : kShKeys;  // of a block's K, a CTA's
  static constexpr int kTiles = kKeys / kKv4Tile;
  static constexpr uint32_t kPartK = kKeys * D * 2;            // each part of K
  static constexpr uint32_t kPartV = kShKeys * (kPair ? D / 2 : D) * 2;
  // K or V of a block as it is stored: of each record tile the codes, then scales and zeros
  static constexpr uint32_t kHalfTile = T::kV + 2 * T::kArr, kRawBytes = kShTiles * kHalfTile;
  static constexpr uint32_t kOffK = 0;
  static constexpr uint32_t kOffV = kOffK + kK * 2 * kPartK;
  static constexpr uint32_t kOffZ = kOffV + kV * kPartV;       // 16 columns of z and s a stage of K
  static constexpr uint32_t kOffRaw = kOffZ + kKeys * 128;
  static constexpr uint32_t kBytes = kOffRaw + 2 * kRaw * kRawBytes + 1024;   // + alignment
  static_assert(kK <= 4, "a 128-byte row holds four stages' columns");
  static_assert(kOffV % 1024 == 0 && kOffZ % 1024 == 0 && kOffRaw % 1024 == 0, "operands' alignment");
  static_assert(kBytes <= 213 * 1024, "shared memory, with 14 KB of barriers and the plan");
  // columns of tensor memory: two blocks' scores, the output, Q, its sums
  static constexpr uint32_t kS = 0, kO = 2 * kShKeys, kQ = kO + D, kSums = kQ + D / 2;
  static constexpr uint32_t kCols = 512;
  static_assert(kSums + 8 <= kCols, "tensor memory");
};

template <int kRaw, int kK, int kV>
struct ShShared {
  uint64_t raw_full[2][kRaw], raw_empty[2][kRaw], k_full[kK], k_empty[kK], v_full[kV], v_empty[kV];   // raw: K's, V's
  uint64_t q_full, o_free, s_full[2], p_full[2], o_done;
  uint32_t seen[2][kRaw][kShTiles];            // a block's keys that exist, a bit each
  float sums[2][kShRows];                      // of each half of a row: sums of q^; of a run's weights
  float most[2][kShRows];                      // largest scores
  union {
    int top[2][kShRows];                       // largest magnitudes of q, as bits
    float all[2][kShRows];                     // sums of all runs' weights
  };
  float past[2][kShRows];                      // the partial rows' reference scores
  uint32_t tmem;
  int fail;
  int part[3][32], at[kShOwnPlan];                // of the plan
  ShGroup groups[kShOwnPlan];
};

// One tile's blocks in a CTA's run.
struct ShSpan {
  int h, tile, first, end;                     // blocks [first, end)
  int rows, part;                              // its rows, and where its partial rows lie
};
// Walks a CTA's run.
template <int kRows>                            // of a tile
struct ShWalk {
  const ShGroup *groups;
  ShGroup g;
  int group, at, stop, n_groups, cta;
  __device__ __forceinline__ ShWalk(const ShHead &hd, const ShGroup *groups_, int cta_)
      : groups(groups_), cta(cta_) {
    n_groups = hd.groups;
    at = static_cast<int>(min((int64_t)cta * hd.per, (int64_t)hd.pairs));
    stop = static_cast<int>(min((int64_t)at + hd.per, (int64_t)hd.pairs));
    group = 0;
    if (at < stop) {
      int lo = 0, hi = n_groups - 1;
      while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (groups[mid].pair0 <= at) lo = mid; else hi = mid - 1;
      }
      group = lo;
      g = groups[group];
    }
  }
  __device__ __forceinline__ bool next(ShSpan &s, int h_k) {
    while (at < stop) {
      if (at >= g.pair0 + g.tiles * h_k * g.counted()) g = groups[++group];
      const int rel = at - g.pair0, tile = rel / g.counted();   // of the group's h_k * tiles
      const int v0 = rel - tile * g.counted(), v1 = min(g.counted(), v0 + (stop - at));
      at += v1 - v0;
      s.first = max(0, v0 - kShOver);
      s.end = v1 - kShOver;
      if (s.end <= s.first) continue;
      s.h = tile / g.tiles;
      s.tile = tile - s.h * g.tiles;
      s.rows = min(kRows, g.rows - s.tile * kRows);
      s.part = cta * kRows + g.row0 + s.h * g.rows + s.tile * kRows;
      return true;
    }
    return false;
  }
};

// By a warp: the sequence whose row names a group's prefix, the first that is as long; -1: none is.
__device__ __forceinline__ int prefix_row(const Kv4DecodeParams &p, const ShGroup &g, int lane) {
  if (!g.ended) return g.seq0;
  const int n = g.rows / p.g;
  for (int i = 1; i < n; i += 32) {
    const uint32_t has = __ballot_sync(0xffffffffu, i + lane < n && p.lens[g.seq0 + i + lane] >= g.keys);
    if (has) return g.seq0 + i + __ffs(has) - 1;
  }
  return -1;
}

// Waits that give up after two seconds, once for the CTA (*fail).
__device__ __forceinline__ bool sh_wait(uint64_t *bar, uint32_t parity, int32_t *status,
                                        volatile int *fail) {
  const uint32_t addr = smem_u32(bar);
  if (mbar_try_wait(addr, parity)) return true;
  const uint64_t t0 = globaltimer_ns();
  while (true) {
    if (*fail) return false;
    if (mbar_try_wait(addr, parity)) return true;
    if (globaltimer_ns() - t0 > kWaitLimitNs) {
      *fail = 1;
      raise(status, NSA_DEVERR_TIMEOUT);
      return false;
    }
  }
}

// A warp arrives at the barrier of the CTA that issues the products, with what its threads did before (a
// pair's second CTA: see the file's head).
template <bool kPair>
__device__ __forceinline__ void warp_arrive(uint64_t *bar) {
  __syncwarp();
  if ((threadIdx.x & 31) != 0) return;
  if constexpr (kPair)
    asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(in_cta(smem_u32(bar), 0))
                 : "memory");
  else
    mbar_arrive(bar);
}

__device__ __forceinline__ void bulk_load(uint32_t dst, const void *src, uint32_t bytes, uint64_t *bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
      "l"(src), "r"(bytes), "r"(smem_u32(bar))
      : "memory");
}
// In order with the other asm statements (barriers among them), but loads may pass it: the places that
// these stores write are not read by ordinary loads.
template <int kOffset = 0>
__device__ __forceinline__ void sts128(uint32_t a, uint4 v) {
  asm volatile("st.shared.v4.b32 [%0 + %5], {%1, %2, %3, %4};" ::"r"(a), "r"(v.x), "r"(v.y), "r"(v.z),
               "r"(v.w), "n"(kOffset));
}
// Whether any of the softmax threads says so; a barrier for them all.
__device__ __forceinline__ bool any_of_256(int id, bool mine) {
  uint32_t any;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.u32 p, %1, 0;\n\t"
      "barrier.red.or.pred q, %2, 256, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}\n"
      : "=r"(any)
      : "r"(mine ? 1u : 0u), "r"(id)
      : "memory");
  return any != 0;
}

// By a whole warp, with the same operands in all lanes, so that they stay in uniform registers; the one
// with `one` issues.
template <bool kPair>
__device__ __forceinline__ void sh_mma(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t add, uint32_t one) {
  if constexpr (kPair)
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "setp.ne.b32 q, %5, 0;\n\t"
        "@q tcgen05.mma.cta_group::2.kind::f16 [%0], [%1], %2, %3, p;\n\t}\n" ::"r"(d),
        "r"(a), "l"(b), "r"(idesc), "r"(add), "r"(one)
        : "memory");
  else
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "setp.ne.b32 q, %5, 0;\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}\n" ::"r"(d),
        "r"(a), "l"(b), "r"(idesc), "r"(add), "r"(one)
        : "memory");
}

// The codes of a word less `off`, as fp16: dimensions (0, 4), (1, 5), (2, 6), (3, 7).  A code in the
// lowest bits of 1024's or in bits 4 to 7 of 64's is added to it.
__device__ __forceinline__ void code_halves(uint32_t w, float off, __half2 (&c)[4]) {
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const uint32_t x = k & 2 ? w >> 8 : w;
    const uint32_t u = k & 1 ? (x & 0x00f000f0u) | 0x54005400u : (x & 0x000f000fu) | 0x64006400u;
    c[k] = __hsub2(*reinterpret_cast<const __half2 *>(&u), __float2half2_rn((k & 1 ? 64.f : 1024.f) + off));
  }
}
template <int kOffset>
__device__ __forceinline__ void sts_halves(uint32_t a, const __half2 (&h)[4]) {
  const uint32_t *u = reinterpret_cast<const uint32_t *>(h);
  sts128<kOffset>(a, make_uint4(u[0], u[1], u[2], u[3]));
}
// V's values past fp16's largest, which the rounding of a scale can make of 65504, are held to it.
__device__ __forceinline__ __half2 held(__half2 h) {
  const __half2 top = __float2half2_rn(65504.f);
  return __hmin2_nan(__hmax2_nan(h, __hneg2(top)), top);
}
// s less its last three bits, at most 8128: eight times it fits fp16 (scales reach 8736).
__device__ __forceinline__ __half2 upper(__half2 s) {
  const uint32_t u = *reinterpret_cast<const uint32_t *>(&s) & 0xfff8fff8u;
  return __hmin2(*reinterpret_cast<const __half2 *>(&u), __float2half2_rn(8128.f));
}

// What the unpackers' thread t (of 256) brings of a block: in turn u 16 bytes, q of them, of the row of a
// key, and that row's scales or zeros (0 for a key that is not there).  All of it is loaded before any
// of it is worked on.
template <int D, int kKeys, int kThreads>       // keys of the block, or of a part of it
struct ShPiece {
  using T = Kv4Tile<D>;
  static constexpr int kG = T::kG, kChunks = T::kRow / 16, kTurns = kKeys * kChunks / kThreads;
  uint32_t w[kTurns][4];
  __half2 s[kTurns][kG], z[kTurns][kG];
  __device__ __forceinline__ static int key(int u, int t) { return (u * kThreads + t) / kChunks; }
  __device__ __forceinline__ ShPiece(const uint8_t *raw, const uint32_t (&seen)[kShTiles], int t) {
#pragma unroll
    for (int u = 0; u < kTurns; ++u) {
      const int k = key(u, t), row = k & 31, q = t % kChunks;
      const uint8_t *tile = raw + (k >> 5) * Sh<D, false>::kHalfTile;
      const uint4 x = *reinterpret_cast<const uint4 *>(tile + row * T::kRow + q * 16);
      w[u][0] = x.x;
      w[u][1] = x.y;
      w[u][2] = x.z;
      w[u][3] = x.w;
      const __half *par = reinterpret_cast<const __half *>(tile + T::kV) + row * kG;
      const bool in = seen[k >> 5] >> row & 1;
#pragma unroll
      for (int g = 0; g < kG; ++g) {
        s[u][g] = __half2half2(in ? par[g] : __ushort_as_half(0));
        z[u][g] = __half2half2(in ? par[T::kArr / 2 + g] : __ushort_as_half(0));
      }
    }
  }
  // Word 4 q + i is group i % kG's, its dimensions' chunk there (4 / kG) q + i / kG: in an operand it lies
  // at (first(t) ^ flip(i)) + step(u, i), whatever the operand's start, a multiple of 1024.
  __device__ __forceinline__ static uint32_t first(int t) {
    return sw128_offset(key(0, t), (4 / kG) * (t % kChunks), kKeys);
  }
  static constexpr uint32_t flip(int i) { return static_cast<uint32_t>(i / kG) << 4; }
  static constexpr int step(int u, int i) { return (i % kG) * kKeys * 128 + u * (kThreads / kChunks) * 128; }
};

// f(u, i) for all turns and words, with both known to the compiler.
template <typename F, int... kI>
__device__ __forceinline__ void each_word(F &&f, std::integer_sequence<int, kI...>) {
  (f(std::integral_constant<int, kI / 4>{}, std::integral_constant<int, kI % 4>{}), ...);
}

template <int D, int kKeys, int kThreads>
__device__ __forceinline__ void unpack_k(const uint8_t *raw, const uint32_t (&seen)[kShTiles], uint32_t kdst,
                                         uint32_t zdst, int stage, int t, uint32_t first) {
  using P = ShPiece<D, kKeys, kThreads>;
  constexpr int G = P::kG;
  const P p(raw, seen, t);
  __half2 hi[P::kTurns][G], lo[P::kTurns][G];
#pragma unroll
  for (int u = 0; u < P::kTurns; ++u)
#pragma unroll
    for (int g = 0; g < G; ++g) {
      hi[u][g] = upper(p.s[u][g]);
      lo[u][g] = __hsub2(p.s[u][g], hi[u][g]);
    }
  each_word([&](auto u, auto i) {
    __half2 c[4], x[4], y[4];
    code_halves(p.w[u][i], 8.f, c);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      x[k] = __hmul2(c[k], hi[u][i % G]);
      y[k] = __hmul2(c[k], lo[u][i % G]);
    }
    const uint32_t a = (kdst + first) ^ P::flip(i);
    sts_halves<P::step(u, i)>(a, x);
    sts_halves<P::step(u, i) + kKeys * D * 2>(a, y);
  }, std::make_integer_sequence<int, 4 * P::kTurns>{});
  // the first thread of a row: z z z s s s of each group; 0, or -inf: no key
  if (t % P::kChunks == 0) {
#pragma unroll
    for (int u = 0; u < P::kTurns; ++u) {
      const int key = P::key(u, t);
      uint32_t v[8] = {0u, 0u, 0u, 0u, 0u, 0u, 0u, 0u};
#pragma unroll
      for (int g = 0; g < G; ++g) {
        const __half2 zs = __lows2half2(p.z[u][g], p.s[u][g]);
        v[3 * g] = *reinterpret_cast<const uint32_t *>(&p.z[u][g]);
        v[3 * g + 1] = *reinterpret_cast<const uint32_t *>(&zs);
        v[3 * g + 2] = *reinterpret_cast<const uint32_t *>(&p.s[u][g]);
      }
      v[6] = seen[key >> 5] >> (key & 31) & 1 ? 0u : 0xfc00u;
      sts128(zdst + sw128_offset(key, 2 * stage, kKeys), make_uint4(v[0], v[1], v[2], v[3]));
      sts128(zdst + sw128_offset(key, 2 * stage + 1, kKeys), make_uint4(v[4], v[5], v[6], v[7]));
    }
  }
}

// kPair: group `rank` of the dimensions alone, every second word.
template <int D, bool kPair, int kThreads>
__device__ __forceinline__ void unpack_v(const uint8_t *raw, const uint32_t (&seen)[kShTiles], uint32_t vdst,
                                         int t, uint32_t first, int rank) {
  using P = ShPiece<D, kShKeys, kThreads>;
  constexpr int G = P::kG;
  const P p(raw, seen, t);
  if constexpr (kPair) {
    static_assert(G == 2, "a CTA of a pair has a group of V's dimensions");
    __half2 s[P::kTurns], z[P::kTurns];
    bool big = false;
#pragma unroll
    for (int u = 0; u < P::kTurns; ++u) {
      s[u] = rank ? p.s[u][G - 1] : p.s[u][0];
      z[u] = rank ? p.z[u][G - 1] : p.z[u][0];
      big |= !(fabsf(__low2float(z[u])) + 15.f * __low2float(s[u]) < 65504.f);
    }
    const bool any_big = __any_sync(0xffffffffu, big);
    each_word([&](auto u, auto i) {
      if constexpr (i % G == 0) {
        __half2 c[4];
        code_halves(rank ? p.w[u][i + 1] : p.w[u][i], 0.f, c);
#pragma unroll
        for (int k = 0; k < 4; ++k) c[k] = __hfma2(c[k], s[u], z[u]);
        if (any_big) {
#pragma unroll
          for (int k = 0; k < 4; ++k) c[k] = held(c[k]);
        }
        sts_halves<P::step(u, i)>((vdst + first) ^ P::flip(i), c);
      }
    }, std::make_integer_sequence<int, 4 * P::kTurns>{});
    return;
  }
  bool wide = false;
#pragma unroll
  for (int u = 0; u < P::kTurns; ++u)
#pragma unroll
    for (int g = 0; g < G; ++g)
      wide |= !(fabsf(__low2float(p.z[u][g])) + 15.f * __low2float(p.s[u][g]) < 65504.f);
  const bool any_wide = __any_sync(0xffffffffu, wide);
  each_word([&](auto u, auto i) {
    __half2 c[4];
    code_halves(p.w[u][i], 0.f, c);
#pragma unroll
    for (int k = 0; k < 4; ++k) c[k] = __hfma2(c[k], p.s[u][i % G], p.z[u][i % G]);
    if (any_wide) {
#pragma unroll
      for (int k = 0; k < 4; ++k) c[k] = held(c[k]);
    }
    sts_halves<P::step(u, i)>((vdst + first) ^ P::flip(i), c);
  }, std::make_integer_sequence<int, 4 * P::kTurns>{});
}

__device__ __forceinline__ float max3(float a, float b, float c) {
  float m;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(m) : "f"(a), "f"(b), "f"(c));
  return m;
}

__device__ __forceinline__ void add_scaled(float4 &a, float4 b, float f) {
  a.x = fmaf(b.x, f, a.x);
  a.y = fmaf(b.y, f, a.y);
  a.z = fmaf(b.z, f, a.z);
  a.w = fmaf(b.w, f, a.w);
}

// A number as three fp16 ones.
__device__ __forceinline__ void three_parts(float x, __half (&h)[3]) {
#pragma unroll
  for (int i = 0; i < 3; ++i) {
    h[i] = __float2half_rn(x);
    x -= __half2float(h[i]);
  }
}

template <int D, bool kFp16, bool kPair>
__global__ void __launch_bounds__(kShThreads, 1) kv4_prefix_kernel(const __grid_constant__ Kv4SharedParams sp_,
                                                                   ShPlan plan) {
  using S = Sh<D, kPair>;
  constexpr int kShRaw = S::kRaw, kShK = S::kK, kShV = S::kV, kCtas = kPair ? 2 : 1;
  constexpr int kTileRows = kShRows * kCtas;                   // of a tile, 128 of them a CTA's
  using T = Kv4Tile<D>;
  constexpr int G = S::kG;
  extern __shared__ uint8_t smem_raw[];
  __shared__ ShShared<kShRaw, kShK, kShV> sh;
  uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                              ~uintptr_t(1023));
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  volatile int *const fail = &sh.fail;
  const Kv4DecodeParams &p = sp_.dec;
  // Blocks of a run of the tensor core's sums.
  constexpr int kRun = kFp16 ? 64 : 256;
  const int rank = kPair ? blockIdx.x & 1 : 0, unit = blockIdx.x / kCtas;   // a unit walks one run
  after_previous();
  const bool own_plan = sp_.num_groups <= kShOwnPlan;
  ShHead head;
  if (own_plan) {
    // every CTA plans; the first one leaves the plan, and each a share of the sequences' places, to
    // the kernels behind
    int32_t err = 0;
    head = make_plan<kShThreads>(sp_, sh.groups, sh.at, gridDim.x / kCtas, kPair ? 8 : 7, sh.part, err);
    for (int64_t b = (int64_t)blockIdx.x * kShThreads + tid; b < p.num_seqs; b += (int64_t)gridDim.x * kShThreads)
      place_sequence(sp_, plan, head, sh.groups, sh.at, static_cast<int>(b));
    if (blockIdx.x == 0) {
      if (err) raise(p.status, err);
      if (tid == 0) *plan.head = head;
      for (int i = tid; i < head.groups; i += kShThreads) plan.groups[i] = sh.groups[i];
    }
  } else {
    head = *plan.head;
  }
  if (head.pairs <= (int64_t)unit * head.per) return;
  if (warp == 19) tmem_alloc<kPair>(&sh.tmem, S::kCols);
  if (tid == 0) {
    for (int i = 0; i < 2 * kShRaw; ++i) {
      mbar_init(&sh.raw_full[0][i], 1);
      mbar_init(&sh.raw_empty[0][i], S::kUnpackers);
    }
    for (int i = 0; i < kShK; ++i) {
      mbar_init(&sh.k_full[i], S::kUnpackers / 32 * kCtas);
      mbar_init(&sh.k_empty[i], 1);
    }
    for (int i = 0; i < kShV; ++i) {
      mbar_init(&sh.v_full[i], S::kUnpackers / 32 * kCtas);
      mbar_init(&sh.v_empty[i], 1);
    }
    mbar_init(&sh.q_full, 8 * kCtas);
    mbar_init(&sh.o_free, 8 * kCtas);
    mbar_init(&sh.o_done, 1);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sh.s_full[i], 1);
      mbar_init(&sh.p_full[i], 8 * kCtas);
    }
    sh.fail = 0;
    fence_mbar_init();
  }
  tc_fence_before();
  if constexpr (kPair) cluster_sync();
  else __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sh.tmem;
  const uint32_t sK = smem_u32(smem + S::kOffK), sV = smem_u32(smem + S::kOffV),
                 sZ = smem_u32(smem + S::kOffZ);
  uint8_t *const raw0 = smem + S::kOffRaw;
  ShWalk<kTileRows> walk(head, own_plan ? sh.groups : plan.groups, unit);
  ShSpan sp;

  if (warp == 18) {
    // ------------------------------ loader ------------------------------
    int it = 0;
    int32_t err = 0;
    while (walk.next(sp, p.h_k)) {
      const int src_row = prefix_row(p, walk.g, lane);
      const int keys = src_row < 0 ? 0 : walk.g.keys;          // 0: no sequence reads what comes of it
      const int32_t *row = p.table + (int64_t)src_row * p.width;
      const int tpl = p.page_log2 - 5, tiles_end = min((keys + kKv4Tile - 1) / kKv4Tile, sp.end * kShTiles);
      int my_page = -1;
      for (int b = sp.first; b < sp.end; ++b, ++it) {
        const int n = (b - sp.first) % (32 / kShTiles), at_tile = b * kShTiles + lane;   // record tile of the prefix
        if (n == 0) {                                          // the pages of the next 32
          my_page = -1;
          if (at_tile < tiles_end) {
            my_page = row[at_tile >> tpl];
            if (my_page < 0 || my_page >= p.num_pages) {
              my_page = -1;
              err |= NSA_DEVERR_BAD_INDEX;
            }
          }
        }
        // lane u < kShTiles brings the block's record tile u: its K, then its V
        const int pg = __shfl_sync(0xffffffffu, my_page, (n * kShTiles + lane) & 31);
        const int rs = it % kShRaw, left = at_tile < tiles_end ? keys - at_tile * kKv4Tile : 0;
        const bool there = lane < kShTiles && pg >= 0;
        const uint8_t *src = p.pool + ((((int64_t)pg * p.h_k + sp.h) << tpl) + (at_tile & ((1 << tpl) - 1))) * T::kBytes;
#pragma unroll
        for (int v = 0; v < 2; ++v) {
          // of K a CTA brings its own keys
          const int at = lane - (v ? 0 : rank * S::kTiles);
          const bool in = at >= 0 && at < (v ? kShTiles : S::kTiles), mine = there && in;
          const int tiles = __popc(__ballot_sync(0xffffffffu, mine));
          if (it >= kShRaw) sh_wait(&sh.raw_empty[v][rs], ((it / kShRaw) - 1) & 1, p.status, fail);
          __syncwarp();
          if (in) sh.seen[v][rs][at] = !mine || left <= 0 ? 0u : left >= 32 ? ~0u : (1u << left) - 1u;
          __syncwarp();
          if (lane == 0) {
            if (tiles) mbar_arrive_expect_tx(&sh.raw_full[v][rs], tiles * S::kHalfTile);
            else mbar_arrive(&sh.raw_full[v][rs]);
          }
          __syncwarp();
          if (mine) {
            const uint32_t dst = smem_u32(raw0 + (v * kShRaw + rs) * S::kRawBytes + at * S::kHalfTile);
            bulk_load(dst, src + v * T::kV, T::kV, &sh.raw_full[v][rs]);
            bulk_load(dst + T::kV, src + T::kPar + v * 2 * T::kArr, 2 * T::kArr, &sh.raw_full[v][rs]);
          }
        }
      }
    }
    err = __reduce_or_sync(0xffffffffu, err);
    if (err && lane == 0) raise(p.status, err);
    // nothing may be in flight when the CTA ends, given up or not
    if (lane < 2)
      for (int i = max(0, it - kShRaw); i < it; ++i) {
        const uint32_t bar = smem_u32(&sh.raw_full[lane][i % kShRaw]);
        const uint64_t t0 = globaltimer_ns();
        while (!mbar_try_wait(bar, (i / kShRaw) & 1) && globaltimer_ns() - t0 < kWaitLimitNs) {
        }
      }
    __syncwarp();
  } else if (warp >= 8 && warp < 16) {
    // ----------------------------- unpackers ----------------------------
    // K of a block, then its V, or with one place for V that of the block before, which the product
    // before that frees
    constexpr int kMine = S::kUnpackers;
    const int t = (tid - 256) % kMine, set = (tid - 256) / kMine;
    const uint32_t first_k = ShPiece<D, S::kKeys, kMine>::first(t), first_v = ShPiece<D, kShKeys, kMine>::first(t);
    int it = 0;
    auto k_of = [&](int i) {
      const int rs = i % kShRaw, ks = i % kShK;
      sh_wait(&sh.raw_full[0][rs], (i / kShRaw) & 1, p.status, fail);
      if (i >= kShK) sh_wait(&sh.k_empty[ks], ((i / kShK) - 1) & 1, p.status, fail);
      __syncwarp();
      unpack_k<D, S::kKeys, kMine>(raw0 + rs * S::kRawBytes, sh.seen[0][rs], sK + ks * 2 * S::kPartK, sZ, ks, t, first_k);
      fence_proxy_async_smem();
      warp_arrive<kPair>(&sh.k_full[ks]);
      mbar_arrive(&sh.raw_empty[0][rs]);
    };
    auto v_of = [&](int i) {
      const int rs = i % kShRaw, vs = i % kShV;
      sh_wait(&sh.raw_full[1][rs], (i / kShRaw) & 1, p.status, fail);
      if (i >= kShV) sh_wait(&sh.v_empty[vs], ((i / kShV) - 1) & 1, p.status, fail);
      __syncwarp();
      unpack_v<D, kPair, kMine>(raw0 + (kShRaw + rs) * S::kRawBytes, sh.seen[1][rs], sV + vs * S::kPartV, t, first_v, rank);
      fence_proxy_async_smem();
      warp_arrive<kPair>(&sh.v_full[vs]);
      mbar_arrive(&sh.raw_empty[1][rs]);
    };
    while (walk.next(sp, p.h_k))
      for (int b = sp.first; b < sp.end; ++b, ++it) {
        if (it % S::kSets != set) continue;
        k_of(it);
        if (S::kSets > 1) v_of(it);
        else if (it > 0) v_of(it - 1);
      }
    if (S::kSets == 1 && it > 0) v_of(it - 1);
    // What the last products' commits arrive at is this CTA's, in a pair from the other one too: it stays until
    // they have (a set's first warp, for the stages whose phases it has followed).
    if (t < 32) {
      auto emptied = [&](uint64_t *bars, int stages, int stage) {
        if (it > stage) sh_wait(&bars[stage], ((it - 1 - stage) / stages) & 1, p.status, fail);
      };
      for (int i = set; i < kShK; i += S::kSets) emptied(sh.k_empty, kShK, i);
      for (int i = set; i < kShV; i += S::kSets) emptied(sh.v_empty, kShV, i);
    }
  } else if (warp == 16) {
    // ----------------------------- MMA warp -----------------------------
    if (rank == 0) {
      uint32_t one;
      asm volatile("{\n\t.reg .pred q;\n\telect.sync _|q, 0xffffffff;\n\tselp.u32 %0, 1, 0, q;\n\t}\n" : "=r"(one));
      auto same = [](uint32_t x) { return __shfl_sync(0xffffffffu, x, 0); };
      const uint32_t tmem_u = same(tmem);
      constexpr uint32_t kIdS = idesc_f16(kTileRows, kShKeys, false, false, true);
      constexpr uint32_t kIdO = idesc_f16(kTileRows, D, false, true, true);
      constexpr uint32_t kHi = sdesc_hi_sw128(1024);
      const uint32_t lo_k = same(sdesc_lo_sw128(sK, 16)), lo_z = same(sdesc_lo_sw128(sZ, 16));
      const uint32_t lo_v = same(sdesc_lo_sw128(sV, kShKeys * 128));
      const uint32_t to = tmem_u + S::kO, tq = tmem_u + S::kQ, tsum = tmem_u + S::kSums;
      int it = 0;
      auto scores = [&](int i) {
        const int ks = i % kShK;
        const uint32_t ts = tmem_u + S::kS + (i & 1) * kShKeys;
        const uint32_t bk = lo_k + ks * (2 * S::kPartK >> 4), bz = lo_z + ks * (32 >> 4);
        sh_wait(&sh.k_full[ks], (i / kShK) & 1, p.status, fail);
        tc_fence_after();
        // smallest parts first: each step cuts the sum so far towards zero
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk)
          sh_mma<kPair>(ts, tq + kk * 8,
                            sdesc_join(bk + ((S::kPartK + kmajor_step(S::kKeys, kk)) >> 4), kHi), kIdS, kk > 0, one);
        sh_mma<kPair>(ts, tsum, sdesc_join(bz, kHi), kIdS, 1, one);
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk)
          sh_mma<kPair>(ts, tq + kk * 8, sdesc_join(bk + (kmajor_step(S::kKeys, kk) >> 4), kHi), kIdS, 1, one);
        if (one) mma_commit<kPair>(&sh.s_full[i & 1]);
        if (one) mma_commit<kPair>(&sh.k_empty[ks]);
      };
      auto output = [&](int i, bool add) {
        const uint32_t ts = tmem_u + S::kS + (i & 1) * kShKeys;
        const int vs = i % kShV;
        sh_wait(&sh.v_full[vs], (i / kShV) & 1, p.status, fail);
        sh_wait(&sh.p_full[i & 1], (i >> 1) & 1, p.status, fail);
        tc_fence_after();
        // weights of 32 keys lie over their scores, in fp16 the rest of them behind
#pragma unroll
        for (int part = 0; part < (kFp16 ? 2 : 1); ++part)
#pragma unroll
          for (int kk = 0; kk < kShKeys / 16; ++kk)
            sh_mma<kPair>(to, ts + (kk >> 1) * 32 + part * 16 + (kk & 1) * 8,
                              sdesc_join(lo_v + ((vs * S::kPartV + mnmajor_step(kk)) >> 4), kHi), kIdO,
                              add || part > 0 || kk > 0, one);
        if (one) mma_commit<kPair>(&sh.o_done);
        if (one) mma_commit<kPair>(&sh.v_empty[vs]);
      };
      int runs = 0;
      for (int turn = 0; walk.next(sp, p.h_k); ++turn) {
        const int nb = same(sp.end - sp.first);
        sh_wait(&sh.q_full, turn & 1, p.status, fail);
        for (int n = 0; n <= nb; ++n) {
          if (n < nb) scores(it + n);
          if (n == 0) continue;
          const bool starts = (n - 1) % kRun == 0;             // what was summed before is in the partial rows
          if (starts && runs > 0) sh_wait(&sh.o_free, (runs - 1) & 1, p.status, fail);
          runs += starts;
          output(it + n - 1, !starts);
        }
        it += nb;
      }
    }
    __syncwarp();
  } else if (warp < 8) {
    // ------------------------------ softmax -----------------------------
    const int w = warp >> 2, row = tid & 127, in_tile = row + rank * kShRows;   // row: tensor memory lane
    const uint32_t lane_off = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t to = tmem + S::kO + lane_off + w * (D / 2);
    constexpr int kHalf = D / 2;                               // dimensions of a row that are a thread's
    constexpr int kMine = kShKeys / 2;                         // keys of a block that are
    int it = 0;
    while (walk.next(sp, p.h_k)) {
      const int nb = sp.end - sp.first;
      // ---- the tile's queries ----
      const int r = sp.tile * kTileRows + in_tile;
      const bool real = in_tile < sp.rows;
      uint4 q4[kHalf / 8];
      int64_t qrow = 0;
      if (real) {
        const int b = r / p.g;
        qrow = (int64_t)(walk.g.seq0 + b) * p.h_q + sp.h * p.g + (r - b * p.g);
      }
      uint32_t top = 0;
#pragma unroll
      for (int i = 0; i < kHalf / 8; ++i) {
        q4[i] = make_uint4(0u, 0u, 0u, 0u);
        if (real)
          q4[i] = *reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(p.q) + qrow * D +
                                                   w * kHalf + i * 8);
        top = __vmaxu2(__vmaxu2(top, q4[i].x & 0x7fff7fffu), q4[i].y & 0x7fff7fffu);
        top = __vmaxu2(__vmaxu2(top, q4[i].z & 0x7fff7fffu), q4[i].w & 0x7fff7fffu);
      }
      sh.top[w][row] = max(top & 0xffffu, top >> 16);
      named_bar_sync(1, 256);
      const uint32_t big = max(sh.top[0][row], sh.top[1][row]);
      const float mag = unpack2<kFp16>(big).x;
      const int ex = max(static_cast<int>(__float_as_uint(mag) >> 23) - 127, -100);
      const float up = __uint_as_float(static_cast<uint32_t>(kShQTop - ex + 127) << 23);   // 2^(5 - ex)
      const float sgn = p.scale < 0.f ? -up : up;
      float sum = 0.f;
#pragma unroll
      for (int i = 0; i < kHalf / 8; i += 4) {
        uint32_t o[16];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float2 a = unpack2<kFp16>(q4[i + j].x), b = unpack2<kFp16>(q4[i + j].y);
          const float2 c = unpack2<kFp16>(q4[i + j].z), e = unpack2<kFp16>(q4[i + j].w);
          o[4 * j] = pack2<true>(a.x * sgn, c.x * sgn);        // dimensions 0 4, 1 5, 2 6, 3 7
          o[4 * j + 1] = pack2<true>(a.y * sgn, c.y * sgn);
          o[4 * j + 2] = pack2<true>(b.x * sgn, e.x * sgn);
          o[4 * j + 3] = pack2<true>(b.y * sgn, e.y * sgn);
          const float2 f0 = unpack2<true>(o[4 * j]), f1 = unpack2<true>(o[4 * j + 1]);
          const float2 f2 = unpack2<true>(o[4 * j + 2]), f3 = unpack2<true>(o[4 * j + 3]);
          sum += ((f0.x + f0.y) + (f1.x + f1.y)) + ((f2.x + f2.y) + (f3.x + f3.y));
        }
        tmem_st16(tmem + S::kQ + lane_off + w * (kHalf / 2) + i * 4, o);
      }
      sh.sums[w][row] = sum;
      named_bar_sync(1, 256);
      if (w == 0) {
        // Q and 8 Q of each group, in three parts each, against z and s; 1 against the mask
        float qs[2] = {sh.sums[0][row], sh.sums[1][row]};
        if (G == 1) qs[0] += qs[1];
        uint32_t o[8] = {0u, 0u, 0u, 0u, 0u, 0u, 0u, 0u};
#pragma unroll
        for (int g = 0; g < G; ++g) {
          __half a[3], b[3];
          three_parts(qs[g], a);
          three_parts(8.f * qs[g], b);
          const __half2 x = __halves2half2(a[0], a[1]), y = __halves2half2(a[2], b[0]),
                        z = __halves2half2(b[1], b[2]);
          o[3 * g] = *reinterpret_cast<const uint32_t *>(&x);
          o[3 * g + 1] = *reinterpret_cast<const uint32_t *>(&y);
          o[3 * g + 2] = *reinterpret_cast<const uint32_t *>(&z);
        }
        o[6] = 0x3c00u;
        tmem_st8(tmem + S::kSums + lane_off, o);
      }
      tmem_wait_st();
      tc_fence_before();
      warp_arrive<kPair>(&sh.q_full);
      // S = |scale| 2^(ex - 5) x, in the exponent of 2; `over` powers are left out where the factor
      // could overflow, and put back into the maximum (scores then are equal or far apart)
      const int over = max(0, static_cast<int>((__float_as_uint(p.scale) & 0x7fffffffu) >> 23) - 127 +
                                  ex - kShQTop + 2 - kShMulTop);
      // (a factor of 0 would make NaN of the mask's -inf: the least one leaves scores of 0)
      const float mul =
          fmaxf(ldexpf(fabsf(p.scale), ex - kShQTop - over) * 1.4426950408889634f, 1.17549435e-38f);
      // ---- its blocks ----
      // Differences are taken before the factor: between scores they are exact or nearly so, whatever
      // the scores' size, and weights stay within fp16 however a product rounds.
      float ref = -INFINITY, thr = -INFINITY;                  // the reference score, and when to raise it
      const float slack = __fdividef(kShSlack, mul);
      // Sums of weights: of a block's keys, of kRun blocks, of those.  One sum of all keys rounds to the same
      // side again and again where weights are alike (two keys in turn, 524288 of them: lse 7 to 9e-4 off, so
      // 2 to 4e-6).  In shared memory: fp16's threads have no register left.
      sh.all[w][row] = 0.f;
      for (int n = 0; n < nb; ++n, ++it) {
        const uint32_t ts = tmem + S::kS + (it & 1) * kShKeys + w * kMine + lane_off;
        sh_wait(&sh.s_full[it & 1], (it >> 1) & 1, p.status, fail);
        tc_fence_after();
        // twice from tensor memory, for the maximum and, 32 at a time, for the weights: 64 scores do
        // not stay in 96 registers
        float mx[2] = {-INFINITY, -INFINITY};
#pragma unroll
        for (int c = 0; c < kMine; c += 32) {
          float x[32];
          tmem_ld32(ts + c, x);
#pragma unroll
          for (int j = 0; j < 32; j += 2) mx[j >> 1 & 1] = max3(mx[j >> 1 & 1], x[j], x[j + 1]);
        }
        float m = fmaxf(mx[0], mx[1]);
        if (any_of_256(2, m > thr)) {                          // rare behind the first blocks
          sh.most[w][row] = m;
          named_bar_sync(1, 256);
          m = fmaxf(sh.most[0][row], sh.most[1][row]);
          float f = 1.f;
          if (m > thr) {
            f = ex2_approx((ref - m) * mul);                   // 0 the first time
            ref = m;
            thr = __fadd_rd(m, slack);
          }
          sh.all[w][row] *= f;
          if (n % kRun) {                                      // what the blocks before have left
            sh.sums[w][row] *= f;
            sh_wait(&sh.o_done, (it - 1) & 1, p.status, fail);
            tc_fence_after();
#pragma unroll 1
            for (int c = 0; c < kHalf; c += 16) {
              uint32_t o[16];
              tmem_ld16(to + c, o);
#pragma unroll
              for (int j = 0; j < 16; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * f);
              tmem_st16(to + c, o);
            }
          }
        }
        const float base = ref == -INFINITY ? 0.f : -ref;      // no key so far: weights of 0
        Pair sum_n(0.f, 0.f);
#pragma unroll 1
        for (int c = 0; c < kMine; c += 32) {
          float s[32];
          tmem_ld32(ts + c, s);
          uint32_t pk[16], rest[16];
#pragma unroll
          for (int j = 0; j < 32; j += 2) {
            const Pair d = Pair(s[j], s[j + 1]) + Pair(base, base);
            const float2 e = fma(d, Pair(mul, mul), Pair(kShUp, kShUp)).get();
            const float a = ex2_approx(e.x), b = ex2_approx(e.y);
            sum_n = sum_n + Pair(a, b);
            pk[j / 2] = pack2<true>(a, b);
            if (kFp16) {
              const float2 hi = unpack2<true>(pk[j / 2]);
              rest[j / 2] = pack2<true>(a - hi.x, b - hi.y);
            }
          }
          tmem_st16(ts + c, pk);                               // over the scores that have been read
          if (kFp16) tmem_st16(ts + c + 16, rest);
        }
        // every phase of o_done is waited for, one after the other: a parity tells only the last two apart
        if (it > 0) sh_wait(&sh.o_done, (it - 1) & 1, p.status, fail);
        tmem_wait_st();
        tc_fence_before();
        warp_arrive<kPair>(&sh.p_full[it & 1]);
        // (in the place of q^'s sums, which the scores waited for show to have been read)
        const float before = n % kRun ? sh.sums[w][row] : 0.f, run = before + (sum_n.get().x + sum_n.get().y);
        sh.sums[w][row] = run;
        if ((n + 1) % kRun && n + 1 < nb) continue;
        // ---- a run's sums to the partial rows ----
        sh.all[w][row] += run;
        sh_wait(&sh.o_done, it & 1, p.status, fail);
        tc_fence_after();
        constexpr float kDown = 1.f / 256.f;                   // 2^-kShUp
        const bool more = n >= kRun;                           // added to what is there, at another reference
        const float past = sh.past[w][row], f = past == -INFINITY ? 0.f : ex2_approx((past - ref) * mul);
        sh.past[w][row] = ref;
        // four dimensions of all rows, then the next four: whole lines are written
        float4 *dst = reinterpret_cast<float4 *>(plan.part) + (int64_t)sp.part * (D / 4) + in_tile;
#pragma unroll 1
        for (int c = 0; c < kHalf; c += 16) {
          uint32_t x[16];
          tmem_ld16(to + c, x);
          float o[16];
#pragma unroll
          for (int j = 0; j < 16; ++j) o[j] = __uint_as_float(x[j]) * kDown;
          if (real) {
#pragma unroll
            for (int j = 0; j < 16; j += 8) {                  // back in the order of the dimensions
              float4 *to4 = dst + (w * kHalf + c + j) / 4 * sp.rows;
              float4 u = make_float4(o[j], o[j + 2], o[j + 4], o[j + 6]);
              float4 v = make_float4(o[j + 1], o[j + 3], o[j + 5], o[j + 7]);
              if (more) {
                add_scaled(u, to4[0], f);
                add_scaled(v, to4[sp.rows], f);
              }
              to4[0] = u;
              to4[sp.rows] = v;
            }
          }
        }
        tc_fence_before();
        warp_arrive<kPair>(&sh.o_free);
      }
      // ---- the tile's sums ----
      sh.sums[w][row] = sh.all[w][row];
      named_bar_sync(1, 256);
      if (real && w == 0)
        plan.part_ml[sp.part + in_tile] =
            make_float2(ldexpf(ref * mul, over), (sh.sums[0][row] + sh.sums[1][row]) * (1.f / 256.f));
    }
  }
  tc_fence_before();
  if constexpr (kPair) cluster_sync();
  else __syncthreads();
  tc_fence_after();
  if (warp == 19) tmem_dealloc<kPair>(tmem, S::kCols);
}

// ---- join ------------------------------------------------------------------------------
// A CTA takes eight rows of a KV head (neighbouring (sequence, query head) pairs), a thread four
// dimensions of one: the parts of its sequence's own keys and, where a prefix is shared, the partial
// rows of the CTAs that its tile went through, four in flight.  kSplit threads share those partial rows.
constexpr int kJoinRows = 8;
template <int D, bool kFp16, int kSplit>
__global__ void __launch_bounds__(kJoinRows * D / 4 * kSplit) kv4_join_kernel(Kv4DecodeParams p, ShPlan plan) {
  constexpr int kEach = kJoinRows * D / 4;
  __shared__ float4 sums[kSplit > 1 ? kSplit - 1 : 1][kEach];
  __shared__ float2 mls[kSplit > 1 ? kSplit - 1 : 1][kEach];
  const int t = threadIdx.x % kEach, split = threadIdx.x / kEach;
  const int row8 = t % kJoinRows, at = t / kJoinRows;          // dimensions 4 at ...
  const int64_t rows = (int64_t)p.num_seqs * p.g, per_head = (rows + kJoinRows - 1) / kJoinRows;
  const int h = static_cast<int>(blockIdx.x / per_head);
  const int64_t want = (blockIdx.x - h * per_head) * kJoinRows + row8, i = want < rows ? want : rows - 1;
  after_previous();
  const int b = static_cast<int>(i / p.g), j = static_cast<int>(i - (int64_t)b * p.g);
  const int64_t out_row = (int64_t)b * p.h_q + h * p.g + j;
  const float *rec = plan.rec + out_row * kRecFloats<D>;
  int4 tail = make_int4(0, 0, 0, -1);
  if (split == 0) tail = *reinterpret_cast<const int4 *>(rec + D);
  const int gi = plan.of[b];
  float M = -INFINITY, l = 0.f;
  float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
  auto add = [&](const float2 (&v)[4], const float4 (&o)[4]) {
    float top = M;
#pragma unroll
    for (int u = 0; u < 4; ++u) top = fmaxf(top, v[u].x);
    const float old = l != 0.f ? ex2_approx(M - top) : 0.f;
    l *= old;
    x.x *= old;
    x.y *= old;
    x.z *= old;
    x.w *= old;
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      if (v[u].y == 0.f) continue;                             // no keys, or no part
      const float f = ex2_approx(v[u].x - top);
      l = fmaf(f, v[u].y, l);
      x.x = fmaf(f, o[u].x, x.x);
      x.y = fmaf(f, o[u].y, x.y);
      x.z = fmaf(f, o[u].z, x.z);
      x.w = fmaf(f, o[u].w, x.w);
    }
    M = top;
  };
  float2 v[4];
  float4 o[4];
  if (tail.w == 0) {
    M = __int_as_float(tail.x);
    l = __int_as_float(tail.y);
    x = *reinterpret_cast<const float4 *>(rec + 4 * at);
  } else {
    const int head = j % kK4Heads, heads = min(kK4Heads, p.g - (j - head));
    for (int k = 0; k < tail.w; k += 4) {
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        v[u] = make_float2(-INFINITY, 0.f);
        o[u] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (k + u < tail.w) {
          const float *part = part_of<D>(p, k + u == 0 ? 2 * tail.z + 1 : 2 * (tail.z + k + u));
          v[u] = *reinterpret_cast<const float2 *>(part + heads * D + 2 * head);
          const float2 *src = reinterpret_cast<const float2 *>(part + head * D + 4 * at);
          const float2 y = src[0], z = src[1];
          o[u] = make_float4(y.x, y.y, z.x, z.y);
        }
      }
      add(v, o);
    }
  }
  if (gi >= 0) {
    const ShGroup g = plan.groups[gi];
    const int per = plan.head->per, log2 = plan.head->rows_log2;
    const int r = (b - g.seq0) * p.g + j, tile = r >> log2, in = r - (tile << log2);
    const int n = min(1 << log2, g.rows - (tile << log2));
    const int t0 = g.pair0 + (h * g.tiles + tile) * g.counted() + kShOver;
    const int c0 = t0 / per, c1 = (t0 + g.blocks - 1) / per;
    const int64_t base = (int64_t)g.row0 + h * g.rows + (tile << log2);
    const float4 *parts = reinterpret_cast<const float4 *>(plan.part);
    for (int c = c0 + 4 * split; c <= c1; c += 4 * kSplit) {
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        v[u] = make_float2(-INFINITY, 0.f);
        o[u] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (c + u <= c1) {
          const int64_t k = ((int64_t)(c + u) << log2) + base;
          v[u] = plan.part_ml[k + in];
          o[u] = parts[k * (D / 4) + at * n + in];
        }
      }
      add(v, o);
    }
  }
  if constexpr (kSplit > 1) {
    if (split > 0) {
      sums[split - 1][t] = x;
      mls[split - 1][t] = make_float2(M, l);
    }
    __syncthreads();
    if (split > 0) return;
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      v[u] = u < kSplit - 1 ? mls[u][t] : make_float2(-INFINITY, 0.f);
      o[u] = u < kSplit - 1 ? sums[u][t] : make_float4(0.f, 0.f, 0.f, 0.f);
    }
    add(v, o);
  }
  if (want >= rows) return;
  const bool any = l != 0.f;                                   // a NaN sum stays one
  const float inv = any ? __fdividef(1.f, l) : 0.f;
  reinterpret_cast<uint2 *>(p.out)[out_row * (D / 4) + at] =
      make_uint2(pack2<kFp16>(x.x * inv, x.y * inv), pack2<kFp16>(x.z * inv, x.w * inv));
  if (at == 0)
    p.lse[(int64_t)(h * p.g + j) * p.num_seqs + b] = any ? (M + log2f(l)) * 0.69314718055994531f : -INFINITY;
}

// ---- launches ----------------------------------------------------------------------------
size_t kv4_shared_workspace(int d, int num_seqs, int h_q, int num_groups) {
  return static_cast<size_t>(shared_layout(d, num_seqs, h_q, num_groups, nullptr, nullptr));
}

template <int D, bool kFp16, bool kPair>
static cudaError_t run_shared(const Kv4SharedParams &p, cudaStream_t s) {
  int dev = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return e;
  ShPlan plan;
  shared_layout(D, p.dec.num_seqs, p.dec.h_q, p.num_groups, p.ws, &plan);
  const int units = (sms < kShMaxCtas ? sms : kShMaxCtas) / (kPair ? 2 : 1), ctas = units * (kPair ? 2 : 1);
  if (p.num_groups > kShOwnPlan) {
    e = launch_kv4(kv4_share_kernel, dim3(1), kSetupThreads, 0, 1, s, p, plan, units, kPair ? 8 : 7);
    if (e != cudaSuccess) return e;
  }
  auto *kernel = kv4_prefix_kernel<D, kFp16, kPair>;
  // more than half of an SM's: one CTA each, as its tensor memory allows
  constexpr int smem = Sh<D, kPair>::kBytes > 120 * 1024 ? Sh<D, kPair>::kBytes : 120 * 1024;
  e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  e = launch_kv4(kernel, dim3(static_cast<unsigned>(ctas)), kShThreads, smem, kPair ? 2 : 1, s, p, plan);
  if (e != cudaSuccess) return e;
  Kv4DecodeParams own = p.dec;
  own.lo = plan.lo;
  own.rec = plan.rec;
  e = launch_kv4_suffix(D, kFp16, own, s);
  if (e != cudaSuccess) return e;
  const int64_t rows = (int64_t)p.dec.num_seqs * p.dec.g;
  const int64_t joins = p.dec.h_k * ((rows + kJoinRows - 1) / kJoinRows);
  // Where four threads to a place fit the GPU at once, rows are few and each has many partial rows (64
  // behind 8K, 17 each: 31.8 -> 28.6 us, five prompts 27.7 -> 25.8).  Where they do not, each has a few, and
  // threads that find none cost more than they bring (256 behind 32K 170 -> 177, two documents 51 -> 53).
  constexpr int kEach = kJoinRows * D / 4;
  if (joins * kEach * 4 <= (int64_t)sms * 1024)
    return launch_kv4(kv4_join_kernel<D, kFp16, 4>, dim3(static_cast<unsigned>(joins)), kEach * 4, 0, 1, s, p.dec,
                      plan);
  return launch_kv4(kv4_join_kernel<D, kFp16, 1>, dim3(static_cast<unsigned>(joins)), kEach, 0, 1, s, p.dec, plan);
}

// A batch small enough, by the bounds that the host knows, goes the way of kv4_decode: three kernels
// that plan, share and join take about 20 us for the least of work (4 sequences behind 517 tokens: 14
// us a call against 9, 30 of up to 900: 17 against 10).  The longest sequence is taken to be as long as the
// table allows: a small batch in a wide table goes the long way.
constexpr double kShLeastUs = 20.;

cudaError_t launch_kv4_shared(int d, bool fp16, const Kv4SharedParams &p, cudaStream_t s) {
  if (kv4_decode_estimate(p.dec) < kShLeastUs) return launch_kv4_decode(d, fp16, p.dec, s);
  if (d == 64) return fp16 ? run_shared<64, true, false>(p, s) : run_shared<64, false, false>(p, s);
  // Pairs where a group has more than 128 rows on average (of 8 KV heads behind 16K: 256 rows 42 us
  // against 48, 512 61 against 72; 96 rows 39 against 35, half of the pair's rows being none)
  if ((int64_t)p.dec.num_seqs * p.dec.g > (int64_t)kShRows * p.num_groups)
    return fp16 ? run_shared<128, true, true>(p, s) : run_shared<128, false, true>(p, s);
  return fp16 ? run_shared<128, true, false>(p, s) : run_shared<128, false, false>(p, s);
}

}  // namespace nsa
