// kv4_shared.cu -- one-step decode over the 4-bit pages for sequences that share a prefix.
//
// The sequences of a group have the same first tokens, in the same pages.  Softmax over a sequence's
// keys splits at the prefix' end into two sums that are joined by their maxima:
//   out = (sum_prefix w v + sum_own w v) / (sum_prefix w + sum_own w),   w = exp(S - max S).
// The prefix' part is a product of all the group's query rows with the same keys, done once per 128
// rows on the tensor cores; each sequence's own part is kv4_decode.cu's, from the prefix' end on.
//
// Prefix kernel (tcgen05).  Rows of a KV head's tile are (sequence, query head) pairs, M = 128; 64
// keys a block.  The scores' sums are the tensor core's alone, as exact as fp32 products (their
// log-sum-exp is returned in fp32).  With q^ = q 2^(5 - ex), ex the exponent of a row's largest
// magnitude (in fp16 it loses 2^-30 of that), and k = c s + z in a group of dimensions,
//   q^ . k = sum_j q^_j (c_j - 8) s_hi + sum_j q^_j (c_j - 8) s_lo + Q z + 8 Q s,   Q = sum_j q^_j:
// s_hi is s without its last three bits, so that both products with c - 8 (four bits and a sign) are
// exact in fp16; Q and 8 Q are three fp16 numbers each, against z and s in 12 of the 16 columns of
// one more step.  S = |scale| 2^(ex - 5) q^ . k.  (Codes as operands and scales afterwards, in fp32,
// want both groups' accumulators apart and four numbers a key from shared memory for every thread:
// 3190 cycles a block, where this takes XXX.)
// Weights are w = 2^(S - m) 2^8 (with their factor those down to 2^-22 of the maximum are normal
// numbers in fp16).  Two roundings to fp16, of 2^-11 at most each: V's values as they are unpacked, and
// the weights, for bf16 outputs, whose own rounding is eight times as large.  For fp16 outputs, of
// the same size, W is the sum of two fp16 numbers: with W in one part the error over a long prefix
// was 1.66 times that of the output's rounding alone, with two 1.4.  Sums of weights are fp32, of
// the weights before they are rounded.
// The maximum m is raised only when a score passes it by 2^4, so that most blocks rescale nothing.
//
// Roles of a CTA (one an SM, 20 warps), handing blocks on by mbarriers, every wait bounded:
//   loader       a block's two record tiles by bulk copies into a ring, page by page of the table;
//   2 x 4 unpackers  codes, scales and zeros to the K and V operands (128-byte swizzle; the eight
//                dimensions of a word stay in the order 0 4 1 5 2 6 3 7 that masking gives, on both
//                sides of the product and until the output is written);
//   2 MMA threads    S = Q K^T, then O += W V, with Q and W from tensor memory: only K and V are read
//                from shared memory, whose bandwidth the two products would else fill;
//   2 x 4 softmax warps   a thread a row.
// Unpackers, MMA thread and softmax warps of either half take every other block, with a maximum, sum
// and output of their own, joined at the tile's end; while one half is between its products the
// other's run.  W goes to tensor memory over the scores it came from.
// Work: the line of all (tile, block) pairs, tile after tile, in equal runs, one a CTA; where a tile
// is shared by CTAs each leaves partial rows.  kv4_join_kernel adds them and the own part.
#include <cmath>

#include "kv4.cuh"

namespace nsa {

constexpr int kShRows = 128;         // query rows of a tile
constexpr int kShKeys = 64;          // keys of a block
// Blocks of each half (every other one of a tile) that are copied ahead, and unpacked: K's for the
// next product beside those in use; V's follow the product that frees the place.
constexpr int kShRaw = 2, kShK = 2;
constexpr int kShThreads = 640;
constexpr int kShMaxCtas = 256;
constexpr int kShOver = 8;           // blocks that a tile's start and end count as
constexpr int kSetupThreads = 1024;
constexpr float kShSlack = 4.f;      // scores may exceed the reference by this much
constexpr float kShUp = 8.f;         // weights are 2^8 times 2^(S - m)
constexpr int kShQTop = 5;           // exponent of a row's largest q^
constexpr int kShMulTop = 92;        // a score's factor stays below 2^(kShMulTop + 2), scores in its unit below 2^30

// A group that shares: its first sequence and number of rows per KV head, its blocks and tiles, and
// what lies before it: counted blocks (kShOver a tile more than there are), and partial rows.
struct ShGroup {
  int32_t seq0, rows, blocks, tiles, keys, pair0, row0, pad;
  __device__ __forceinline__ int counted() const { return blocks + kShOver; }
};
struct ShHead {
  int32_t groups, pairs, per, pad;   // counted blocks; of them a CTA's
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

// ---- setup -----------------------------------------------------------------------------
// Inclusive prefix over the CTA; total gets the sum.
__device__ __forceinline__ int setup_incl(int x, int (&part)[32], int &total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  __syncthreads();
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

// Shared or not?  In units of 25 ns of an SM's time: a tile of 128 rows takes about 240 and 24 a block
// of 64 keys; the sequences' own passes over the prefix take 5 a tile of 32 keys each.
__device__ __forceinline__ bool worth_sharing(int n, int g, int keys) {
  const int64_t own = (int64_t)n * (g > kK4Heads ? 2 : 1) * ((keys + 31) / 32) * 5;
  const int64_t tiles = ((int64_t)n * g + kShRows - 1) / kShRows;
  return n > 1 && own > tiles * (240 + 24 * (int64_t)((keys + kShKeys - 1) / kShKeys));
}

// One CTA: groups that share, in order, what lies before each, and each sequence's group and first own
// key.  A cu_groups out of order shares nothing.
constexpr int kSetupGroups = 1024;   // up to as many the groups' numbers stay in shared memory
__global__ void __launch_bounds__(kSetupThreads) kv4_share_kernel(Kv4SharedParams p, ShPlan plan, int ctas,
                                                                  int least) {
  __shared__ int part[32], s_cu[kSetupGroups + 1], s_at[kSetupGroups], s_keys[kSetupGroups];
  const int tid = threadIdx.x, cap = p.dec.width << p.dec.page_log2;
  const bool few = p.num_groups <= kSetupGroups;
  after_previous();
  int32_t err = 0;
  for (int i = tid; i < p.num_groups; i += kSetupThreads) {
    const int a = p.cu[i], b = p.cu[i + 1];
    if (a < 0 || (i == 0 && a != 0) || b < a || b > p.dec.num_seqs) err |= NSA_DEVERR_BAD_SEQLENS;
    if (few) {
      s_cu[i] = a;
      s_cu[i + 1] = b;               // the neighbour writes the same
    }
  }
  const bool ordered = !__syncthreads_or(err);
  int groups = 0, pairs = 0, rows = 0;
  for (int i0 = 0; ordered && i0 < p.num_groups; i0 += kSetupThreads) {
    const int i = i0 + tid;
    int n = 0, keys = 0, a = 0;
    if (i < p.num_groups) {
      a = p.cu[i];
      n = p.cu[i + 1] - a;
      keys = p.prefix[i];
      if (keys < 0 || keys > cap) {
        err |= NSA_DEVERR_BAD_SEQLENS;
        keys = 0;
      }
    }
    const bool shares = keys > 0 && worth_sharing(n, p.dec.g, keys);
    const int r = shares ? n * p.dec.g : 0, tiles = (r + kShRows - 1) / kShRows;
    const int blocks = (keys + kShKeys - 1) / kShKeys;
    int total;
    const int g = groups + setup_incl(shares, part, total) - shares;
    groups += total;
    const int w = tiles * p.dec.h_k * (blocks + kShOver);
    const int before = pairs + setup_incl(w, part, total) - w;
    pairs += total;
    const int row = rows + setup_incl(r * p.dec.h_k, part, total) - r * p.dec.h_k;
    rows += total;
    if (shares) plan.groups[g] = ShGroup{a, r, blocks, tiles, keys, before, row, 0};
    if (i < p.num_groups) {
      if (few) {
        s_at[i] = shares ? g : -1;
        s_keys[i] = keys;
      } else {
        plan.at[i] = shares ? g : -1;
      }
    }
  }
  if (tid == 0) *plan.head = ShHead{groups, pairs, max((pairs + ctas - 1) / ctas, least), 0};
  if (__syncthreads_or(err) && tid == 0) raise(p.dec.status, NSA_DEVERR_BAD_SEQLENS);
  for (int b = tid; b < p.dec.num_seqs; b += kSetupThreads) {
    int g = -1, lo = 0;
    if (ordered && groups > 0) {
      const int32_t *cu = few ? s_cu : p.cu;
      if (b < cu[p.num_groups]) {
        const int i = upper_index(cu, p.num_groups, b);
        g = few ? s_at[i] : plan.at[i];
        if (g >= 0) {
          const int keys = few ? s_keys[i] : plan.groups[g].keys;
          // a sequence that ends inside the prefix attends to its own pages alone
          if (min(max(p.dec.lens[b], 0), cap) >= keys) lo = keys;
          else g = -1;
        }
      }
    }
    plan.lo[b] = lo;
    plan.of[b] = g;
  }
}

// ---- prefix ----------------------------------------------------------------------------
template <int D>
struct Sh {
  using T = Kv4Tile<D>;
  static constexpr int kG = T::kG;
  static constexpr uint32_t kOperand = kShKeys * D * 2;        // V of a block, and each part of K
  static constexpr uint32_t kRawBytes = 2 * T::kBytes;
  static constexpr uint32_t kOffK = 0;
  static constexpr uint32_t kOffV = kOffK + 2 * kShK * 2 * kOperand;
  static constexpr uint32_t kOffZ = kOffV + 2 * kOperand;      // 16 columns of z and s a stage of K
  static constexpr uint32_t kOffRaw = kOffZ + kShKeys * 128;
  static constexpr uint32_t kBytes = kOffRaw + 2 * kShRaw * kRawBytes + 1024;   // + alignment
  static_assert(2 * kShK <= 4, "a 128-byte row holds four stages' columns");
  static_assert(kOffV % 1024 == 0 && kOffZ % 1024 == 0 && kOffRaw % 1024 == 0, "operands' alignment");
  static_assert(kBytes <= 226 * 1024, "shared memory");
  // columns of tensor memory: scores of both halves, outputs of both, Q, its sums
  static constexpr uint32_t kS = 0, kO = 2 * kShKeys, kQ = kO + 2 * D, kSums = kQ + D / 2;
  static constexpr uint32_t kCols = 512;
  static_assert(kSums + 8 <= kCols, "tensor memory");
};

struct ShShared {
  // of half w: stages w * kShRaw ..., w * kShK ...; of V one
  uint64_t raw_full[2 * kShRaw], raw_empty[2 * kShRaw], k_full[2 * kShK], k_empty[2 * kShK], v_full[2];
  uint64_t q_full, o_free, s_full[2], p_full[2], o_done[2];
  uint2 seen[2 * kShRaw];                      // a block's keys that exist, a bit each
  float2 ml[2][kShRows];                       // of the two halves, at a tile's end
  float sums[2][kShRows];                      // sums of q^
  int top[2][kShRows];                         // largest magnitude of a row's part, as bits
  uint32_t tmem;
  int fail;
};

// One tile's blocks in a CTA's run.
struct ShSpan {
  int h, tile, first, end;                     // blocks [first, end)
  int rows, part;                              // its rows, and where its partial rows lie
};
// Walks a CTA's run.
struct ShWalk {
  const ShGroup *groups;
  ShGroup g;
  int group, at, stop, n_groups, cta;
  __device__ __forceinline__ ShWalk(const ShPlan &plan, int cta_) : groups(plan.groups), cta(cta_) {
    const ShHead hd = *plan.head;
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
      s.rows = min(kShRows, g.rows - s.tile * kShRows);
      s.part = cta * kShRows + g.row0 + s.h * g.rows + s.tile * kShRows;
      return true;
    }
    return false;
  }
};

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

__device__ __forceinline__ void bulk_load(uint32_t dst, const void *src, uint32_t bytes, uint64_t *bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
      "l"(src), "r"(bytes), "r"(smem_u32(bar))
      : "memory");
}
__device__ __forceinline__ void sts128(uint32_t a, uint4 v) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(a), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w)
               : "memory");
}

// The codes of a word as fp16 less `off` - 1024: dimensions (0, 4), (1, 5), (2, 6), (3, 7).
__device__ __forceinline__ void code_halves(uint32_t w, __half2 off, __half2 (&c)[4]) {
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const uint32_t u = (w >> (4 * k) & 0x000f000fu) | 0x64006400u;   // 1024 + c
    c[k] = __hsub2(*reinterpret_cast<const __half2 *>(&u), off);
  }
}
__device__ __forceinline__ void sts_halves(uint32_t a, const __half2 (&h)[4]) {
  const uint32_t *u = reinterpret_cast<const uint32_t *>(h);
  sts128(a, make_uint4(u[0], u[1], u[2], u[3]));
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

// A thread's places in a block: turn u takes 16 bytes, q of them, of a key's row.
template <int D>
struct ShPlace {
  static constexpr int kChunks = Kv4Tile<D>::kRow / 16;        // 16-byte pieces of a row
  static constexpr int kTurns = kShKeys * kChunks / 128;
  int key, q, row;
  const uint8_t *tile;
  bool in;
  __device__ __forceinline__ ShPlace(const uint8_t *raw, uint2 seen, int u, int t) {
    const int i = u * 128 + t;
    key = i / kChunks;
    q = i % kChunks;
    row = key & 31;
    tile = raw + (key >> 5) * Kv4Tile<D>::kBytes;
    in = (key < 32 ? seen.x : seen.y) >> row & 1;
  }
  // entry `which` of the four arrays (K scale, K zero, V scale, V zero), 0 for a key that is not there
  __device__ __forceinline__ __half2 par(int which, int g) const {
    const __half x = reinterpret_cast<const __half *>(tile + Kv4Tile<D>::kPar + which * Kv4Tile<D>::kArr)
        [row * Kv4Tile<D>::kG + g];
    return __half2half2(in ? x : __ushort_as_half(0));
  }
  // of word 4 q + w: its group, and where its dimensions lie in an operand
  __device__ __forceinline__ uint32_t at(int w) const {
    constexpr int G = Kv4Tile<D>::kG;
    return sw128_offset(key, 8 * (w % G) + (4 / G) * q + w / G, kShKeys);
  }
};

template <int D>
__device__ __forceinline__ void unpack_k(const uint8_t *raw, uint2 seen, uint32_t kdst, uint32_t zdst,
                                         int stage, int t) {
  using T = Kv4Tile<D>;
  using P = ShPlace<D>;
  constexpr int G = T::kG;
  const __half2 off = __float2half2_rn(1032.f);
#pragma unroll
  for (int u = 0; u < P::kTurns; ++u) {
    const P p(raw, seen, u, t);
    const uint4 k4 = *reinterpret_cast<const uint4 *>(p.tile + p.row * T::kRow + p.q * 16);
    const uint32_t kw[4] = {k4.x, k4.y, k4.z, k4.w};
    __half2 hi[G], lo[G];
#pragma unroll
    for (int g = 0; g < G; ++g) {
      const __half2 s = p.par(0, g);
      hi[g] = upper(s);
      lo[g] = __hsub2(s, hi[g]);
    }
#pragma unroll
    for (int w = 0; w < 4; ++w) {
      __half2 c[4], x[4], y[4];
      code_halves(kw[w], off, c);
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        x[k] = __hmul2(c[k], hi[w % G]);
        y[k] = __hmul2(c[k], lo[w % G]);
      }
      sts_halves(kdst + p.at(w), x);
      sts_halves(kdst + Sh<D>::kOperand + p.at(w), y);
    }
  }
  if (t < kShKeys) {                                           // z z z s s s of each group; 0, or -inf: no key
    const int row = t & 31;
    const uint8_t *par = raw + (t >> 5) * T::kBytes + T::kPar;
    const bool in = (t < 32 ? seen.x : seen.y) >> row & 1;
    uint32_t v[8] = {0u, 0u, 0u, 0u, 0u, 0u, 0u, 0u};
#pragma unroll
    for (int g = 0; g < G; ++g) {
      const uint32_t s = in ? reinterpret_cast<const uint16_t *>(par)[row * G + g] : 0u;
      const uint32_t z = in ? reinterpret_cast<const uint16_t *>(par + T::kArr)[row * G + g] : 0u;
      v[3 * g] = z | z << 16;
      v[3 * g + 1] = z | s << 16;
      v[3 * g + 2] = s | s << 16;
    }
    v[6] = in ? 0u : 0xfc00u;
    sts128(zdst + sw128_offset(t, 2 * stage, kShKeys), make_uint4(v[0], v[1], v[2], v[3]));
    sts128(zdst + sw128_offset(t, 2 * stage + 1, kShKeys), make_uint4(v[4], v[5], v[6], v[7]));
  }
}

template <int D>
__device__ __forceinline__ void unpack_v(const uint8_t *raw, uint2 seen, uint32_t vdst, int t) {
  using T = Kv4Tile<D>;
  using P = ShPlace<D>;
  constexpr int G = T::kG;
  const __half2 off = __float2half2_rn(1024.f);
#pragma unroll
  for (int u = 0; u < P::kTurns; ++u) {
    const P p(raw, seen, u, t);
    const uint4 v4 = *reinterpret_cast<const uint4 *>(p.tile + T::kV + p.row * T::kRow + p.q * 16);
    const uint32_t vw[4] = {v4.x, v4.y, v4.z, v4.w};
    __half2 s[G], z[G];
    bool wide = false;
#pragma unroll
    for (int g = 0; g < G; ++g) {
      s[g] = p.par(2, g);
      z[g] = p.par(3, g);
      wide |= !(fabsf(__low2float(z[g])) + 15.f * __low2float(s[g]) < 65504.f);
    }
    const bool any_wide = __any_sync(0xffffffffu, wide);
#pragma unroll
    for (int w = 0; w < 4; ++w) {
      __half2 c[4];
      code_halves(vw[w], off, c);
#pragma unroll
      for (int k = 0; k < 4; ++k) c[k] = __hfma2(c[k], s[w % G], z[w % G]);
      if (any_wide) {
#pragma unroll
        for (int k = 0; k < 4; ++k) c[k] = held(c[k]);
      }
      sts_halves(vdst + p.at(w), c);
    }
  }
}

// A number as three fp16 ones.
__device__ __forceinline__ void three_parts(float x, __half (&h)[3]) {
#pragma unroll
  for (int i = 0; i < 3; ++i) {
    h[i] = __float2half_rn(x);
    x -= __half2float(h[i]);
  }
}

template <int D, bool kFp16>
__global__ void __launch_bounds__(kShThreads, 1) kv4_prefix_kernel(Kv4DecodeParams p, ShPlan plan) {
  using S = Sh<D>;
  using T = Kv4Tile<D>;
  constexpr int G = S::kG;
  extern __shared__ uint8_t smem_raw[];
  __shared__ ShShared sh;
  uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                              ~uintptr_t(1023));
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  volatile int *const fail = &sh.fail;
  after_previous();
  if (plan.head->pairs <= (int64_t)blockIdx.x * plan.head->per) return;   // the whole CTA
  if (warp == 19) tmem_alloc(&sh.tmem, S::kCols);
  if (tid == 0) {
    for (int i = 0; i < 2 * kShRaw; ++i) {
      mbar_init(&sh.raw_full[i], 1);
      mbar_init(&sh.raw_empty[i], 128);
    }
    for (int i = 0; i < 2 * kShK; ++i) {
      mbar_init(&sh.k_full[i], 128);
      mbar_init(&sh.k_empty[i], 1);
    }
    mbar_init(&sh.q_full, 256);
    mbar_init(&sh.o_free, 256);
    for (int w = 0; w < 2; ++w) {
      mbar_init(&sh.v_full[w], 128);
      mbar_init(&sh.s_full[w], 1);
      mbar_init(&sh.p_full[w], 128);
      mbar_init(&sh.o_done[w], 1);
    }
    sh.fail = 0;
    fence_mbar_init();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sh.tmem;
  const uint32_t sK = smem_u32(smem + S::kOffK), sV = smem_u32(smem + S::kOffV),
                 sZ = smem_u32(smem + S::kOffZ);
  uint8_t *const raw0 = smem + S::kOffRaw;
  ShWalk walk(plan, blockIdx.x);
  ShSpan sp;

  if (warp == 18) {
    // ------------------------------ loader ------------------------------
    int count[2] = {0, 0};                                     // blocks of each half
    int32_t err = 0;
    while (walk.next(sp, p.h_k)) {
      const int keys = walk.g.keys;
      const int32_t *row = p.table + (int64_t)walk.g.seq0 * p.width;
      int my_page = -1;
      for (int b = sp.first; b < sp.end; ++b) {
        const int n = (b - sp.first) & 15, w = n & 1, c = w ? count[1]++ : count[0]++;
        if (n == 0) {                                          // the pages of the next 32 tiles
          const int key = b * kShKeys + lane * 32;
          my_page = -1;
          if (key < keys && key < sp.end * kShKeys) {
            my_page = row[key >> p.page_log2];
            if (my_page < 0 || my_page >= p.num_pages) {
              my_page = -1;
              err |= NSA_DEVERR_BAD_INDEX;
            }
          }
        }
        const int pg[2] = {__shfl_sync(0xffffffffu, my_page, 2 * n),
                           __shfl_sync(0xffffffffu, my_page, 2 * n + 1)};
        const int rs = w * kShRaw + c % kShRaw;
        if (lane == 0) {
          if (c >= kShRaw) sh_wait(&sh.raw_empty[rs], ((c / kShRaw) - 1) & 1, p.status, fail);
          uint32_t seen[2], bytes = 0;
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            const int left = keys - (b * kShKeys + 32 * u);
            seen[u] = pg[u] < 0 || left <= 0 ? 0u : left >= 32 ? ~0u : (1u << left) - 1u;
            if (pg[u] >= 0) bytes += T::kBytes;
          }
          sh.seen[rs] = make_uint2(seen[0], seen[1]);
          if (bytes) mbar_arrive_expect_tx(&sh.raw_full[rs], bytes);
          else mbar_arrive(&sh.raw_full[rs]);
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            if (pg[u] < 0) continue;
            const int key = b * kShKeys + 32 * u, tpl = p.page_log2 - 5;
            const int64_t tile = (((int64_t)pg[u] * p.h_k + sp.h) << tpl) +
                                 ((key & ((1 << p.page_log2) - 1)) >> 5);
            bulk_load(smem_u32(raw0 + rs * S::kRawBytes + u * T::kBytes), p.pool + tile * T::kBytes,
                      T::kBytes, &sh.raw_full[rs]);
          }
        }
        __syncwarp();
      }
    }
    err = __reduce_or_sync(0xffffffffu, err);
    if (err && lane == 0) raise(p.status, err);
    // nothing may be in flight when the CTA ends, given up or not
    if (lane == 0)
      for (int w = 0; w < 2; ++w)
        for (int c = max(0, count[w] - kShRaw); c < count[w]; ++c) {
          const uint32_t bar = smem_u32(&sh.raw_full[w * kShRaw + c % kShRaw]);
          const uint64_t t0 = globaltimer_ns();
          while (!mbar_try_wait(bar, (c / kShRaw) & 1) && globaltimer_ns() - t0 < kWaitLimitNs) {
          }
        }
    __syncwarp();
  } else if (warp >= 8 && warp < 16) {
    // ----------------------------- unpackers ----------------------------
    const int w = (warp - 8) >> 2, t = tid & 127;
    int c = 0;                                                 // blocks of this half so far
    while (walk.next(sp, p.h_k)) {
      for (int n = w; n < sp.end - sp.first; n += 2, ++c) {
        const int rs = w * kShRaw + c % kShRaw, ks = w * kShK + c % kShK;
        sh_wait(&sh.raw_full[rs], (c / kShRaw) & 1, p.status, fail);
        if (c >= kShK) sh_wait(&sh.k_empty[ks], ((c / kShK) - 1) & 1, p.status, fail);
        __syncwarp();
        const uint2 seen = sh.seen[rs];
        const uint8_t *raw = raw0 + rs * S::kRawBytes;
        unpack_k<D>(raw, seen, sK + ks * 2 * S::kOperand, sZ, ks, t);
        fence_proxy_async_smem();
        mbar_arrive(&sh.k_full[ks]);
        if (c > 0) sh_wait(&sh.o_done[w], (c - 1) & 1, p.status, fail);
        __syncwarp();
        unpack_v<D>(raw, seen, sV + w * S::kOperand, t);
        fence_proxy_async_smem();
        mbar_arrive(&sh.v_full[w]);
        mbar_arrive(&sh.raw_empty[rs]);
      }
    }
  } else if (warp == 16 || warp == 17) {
    // ---------------------------- MMA threads ---------------------------
    if (lane == 0) {
      constexpr uint32_t kIdS = idesc_f16(kShRows, kShKeys, false, false, true);
      constexpr uint32_t kIdO = idesc_f16(kShRows, D, false, true, true);
      constexpr uint32_t kHi = sdesc_hi_sw128(1024);
      const int w = warp - 16;
      const uint32_t lo_k = sdesc_lo_sw128(sK, 16), lo_z = sdesc_lo_sw128(sZ, 16);
      const uint32_t bv = sdesc_lo_sw128(sV + w * S::kOperand, kShKeys * 128);
      const uint32_t ts = tmem + S::kS + w * kShKeys, to = tmem + S::kO + w * D;
      const uint32_t tq = tmem + S::kQ, tsum = tmem + S::kSums;
      int turn = 0, c = 0;
      for (; walk.next(sp, p.h_k); ++turn) {
        const int nb = sp.end - sp.first;
        sh_wait(&sh.q_full, turn & 1, p.status, fail);
        for (int n = w; n < nb; n += 2, ++c) {
          const int ks = w * kShK + c % kShK;
          const uint32_t bk = lo_k + ks * (2 * S::kOperand >> 4), bz = lo_z + ks * (32 >> 4);
          sh_wait(&sh.k_full[ks], (c / kShK) & 1, p.status, fail);
          tc_fence_after();
          // smallest parts first: each step cuts the sum so far towards zero
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk)
            mma_f16_ts(ts, tq + kk * 8,
                       sdesc_join(bk + ((S::kOperand + kmajor_step(kShKeys, kk)) >> 4), kHi), kIdS, kk > 0);
          mma_f16_ts(ts, tsum, sdesc_join(bz, kHi), kIdS, 1);
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk)
            mma_f16_ts(ts, tq + kk * 8, sdesc_join(bk + (kmajor_step(kShKeys, kk) >> 4), kHi), kIdS, 1);
          mma_commit(&sh.s_full[w]);
          mma_commit(&sh.k_empty[ks]);
          sh_wait(&sh.v_full[w], c & 1, p.status, fail);
          sh_wait(&sh.p_full[w], c & 1, p.status, fail);
          if (n == w && turn > 0) sh_wait(&sh.o_free, (turn - 1) & 1, p.status, fail);
          tc_fence_after();
#pragma unroll
          for (int kk = 0; kk < kShKeys / 16; ++kk)
            mma_f16_ts(to, ts + kk * 8, sdesc_join(bv + (mnmajor_step(kk) >> 4), kHi), kIdO,
                       n >= 2 || kk > 0);
          if (kFp16) {                                         // what the rounding of W has left
#pragma unroll
            for (int kk = 0; kk < kShKeys / 16; ++kk)
              mma_f16_ts(to, ts + kShKeys / 2 + kk * 8, sdesc_join(bv + (mnmajor_step(kk) >> 4), kHi),
                         kIdO, 1);
          }
          mma_commit(&sh.o_done[w]);                           // V's place is free, too
        }
      }
    }
    __syncwarp();
  } else if (warp < 8) {
    // ------------------------------ softmax -----------------------------
    const int w = warp >> 2, row = tid & 127;                  // row: tensor memory lane
    const uint32_t lane_off = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t ts = tmem + S::kS + w * kShKeys + lane_off;
    const uint32_t to = tmem + S::kO + lane_off;
    constexpr int kHalf = D / 2;                               // dimensions of a row that a thread brings
    int count = 0;
    while (walk.next(sp, p.h_k)) {
      const int nb = sp.end - sp.first;
      // ---- the tile's queries ----
      const int r = sp.tile * kShRows + row;
      const bool real = row < sp.rows;
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
      mbar_arrive(&sh.q_full);
      // S = |scale| 2^(ex - 5) x, in the exponent of 2; `over` powers are left out where the factor
      // could overflow, and put back into the maximum (scores then are equal or far apart)
      const int over = max(0, static_cast<int>((__float_as_uint(p.scale) & 0x7fffffffu) >> 23) - 127 +
                                  ex - kShQTop + 2 - kShMulTop);
      // (a factor of 0 would make NaN of the mask's -inf: the least one leaves scores of 0)
      const float mul =
          fmaxf(ldexpf(fabsf(p.scale), ex - kShQTop - over) * 1.4426950408889634f, 1.17549435e-38f);
      // ---- its blocks, every other one ----
      // Differences are taken before the factor: between scores they are exact or nearly so, whatever
      // the scores' size, and weights stay within fp16 however a product rounds.
      float ref = -INFINITY, thr = -INFINITY;                  // the reference score, and when to raise it
      const float slack = __fdividef(kShSlack, mul);
      Pair l(0.f, 0.f);
      for (int n = w; n < nb; n += 2, ++count) {
        sh_wait(&sh.s_full[w], count & 1, p.status, fail);
        tc_fence_after();
        // 32 scores at a time, once for the maximum and once for the weights: all 64 do not fit
        // beside what the rest takes of 96 registers
        float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
        for (int c = 0; c < kShKeys; c += 32) {
          float x[32];
          tmem_ld32(ts + c, x);
#pragma unroll
          for (int j = 0; j < 32; ++j) mx[j & 3] = fmaxf(mx[j & 3], x[j]);
        }
        const float m = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
        if (__any_sync(0xffffffffu, m > thr)) {
          float f = 1.f;
          if (m > thr) {
            f = ex2_approx((ref - m) * mul);                   // 0 the first time
            ref = m;
            thr = __fadd_rd(m, slack);
          }
          l = l * Pair(f, f);
          if (n >= 2) {                                        // what the blocks before have left
            sh_wait(&sh.o_done[w], (count - 1) & 1, p.status, fail);
            tc_fence_after();
#pragma unroll 1
            for (int c = 0; c < D; c += 16) {
              uint32_t o[16];
              tmem_ld16(to + w * D + c, o);
#pragma unroll
              for (int j = 0; j < 16; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * f);
              tmem_st16(to + w * D + c, o);
            }
          }
        }
        const float base = ref == -INFINITY ? 0.f : -ref;      // no key so far: weights of 0
        uint32_t rest[2][16];
#pragma unroll
        for (int c = 0; c < kShKeys; c += 32) {
          float s[32];
          tmem_ld32(ts + c, s);
          uint32_t pk[16];
#pragma unroll
          for (int j = 0; j < 32; j += 2) {
            const Pair d = Pair(s[j], s[j + 1]) + Pair(base, base);
            const float2 e = fma(d, Pair(mul, mul), Pair(kShUp, kShUp)).get();
            const float a = ex2_approx(e.x), b = ex2_approx(e.y);
            l = l + Pair(a, b);
            pk[j / 2] = pack2<true>(a, b);
            if (kFp16) {
              const float2 hi = unpack2<true>(pk[j / 2]);
              rest[c / 32][j / 2] = pack2<true>(a - hi.x, b - hi.y);
            }
          }
          tmem_st16(ts + c / 2, pk);                           // over scores that have been read
        }
        if (kFp16) {
          tmem_st16(ts + kShKeys / 2, rest[0]);
          tmem_st16(ts + kShKeys / 2 + 16, rest[1]);
        }
        tmem_wait_st();
        tc_fence_before();
        mbar_arrive(&sh.p_full[w]);
      }
      // ---- the two halves' sums ----
      if (nb > w) sh_wait(&sh.o_done[w], (count - 1) & 1, p.status, fail);
      const float2 l2 = l.get();
      sh.ml[w][row] = make_float2(ref * mul, l2.x + l2.y);
      named_bar_sync(1, 256);
      tc_fence_after();
      const float2 m0 = sh.ml[0][row];
      const float2 m1 = nb > 1 ? sh.ml[1][row] : make_float2(-INFINITY, 0.f);
      const float M = fmaxf(m0.x, m1.x);
      constexpr float kDown = 1.f / 256.f;                     // 2^-kShUp
      const float f0 = m0.y != 0.f ? ex2_approx(m0.x - M) * kDown : 0.f;
      const float f1 = m1.y != 0.f ? ex2_approx(m1.x - M) * kDown : 0.f;
      // four dimensions of all rows, then the next four: whole lines are written
      float4 *dst = reinterpret_cast<float4 *>(plan.part) + (int64_t)sp.part * (D / 4) + row;
#pragma unroll 1
      for (int c = 0; c < kHalf; c += 16) {
        uint32_t x[16], y[16];
        tmem_ld16(to + w * kHalf + c, x);
        if (nb > 1) tmem_ld16(to + D + w * kHalf + c, y);
        float o[16];
#pragma unroll
        for (int j = 0; j < 16; ++j) {
          o[j] = m0.y != 0.f ? __uint_as_float(x[j]) * f0 : 0.f;
          if (nb > 1 && m1.y != 0.f) o[j] = fmaf(__uint_as_float(y[j]), f1, o[j]);
        }
        if (real) {
#pragma unroll
          for (int j = 0; j < 16; j += 8) {                    // back in the order of the dimensions
            const int at = (w * kHalf + c + j) / 4;
            dst[at * sp.rows] = make_float4(o[j], o[j + 2], o[j + 4], o[j + 6]);
            dst[(at + 1) * sp.rows] = make_float4(o[j + 1], o[j + 3], o[j + 5], o[j + 7]);
          }
        }
      }
      if (real && w == 0)
        plan.part_ml[sp.part + row] =
            make_float2(ldexpf(M, over), f0 * m0.y + (nb > 1 ? f1 * m1.y : 0.f));
      tc_fence_before();
      mbar_arrive(&sh.o_free);
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 19) tmem_dealloc(tmem, S::kCols);
}

// ---- join ------------------------------------------------------------------------------
// A CTA takes eight rows of a KV head (neighbouring (sequence, query head) pairs), a thread four
// dimensions of one: the parts of its sequence's own keys and, where a prefix is shared, the partial
// rows of the CTAs that its tile went through, four in flight.
constexpr int kJoinRows = 8;
template <int D, bool kFp16>
__global__ void __launch_bounds__(kJoinRows * D / 4) kv4_join_kernel(Kv4DecodeParams p, ShPlan plan) {
  const int row8 = threadIdx.x % kJoinRows, at = threadIdx.x / kJoinRows;   // dimensions 4 at ...
  const int64_t rows = (int64_t)p.num_seqs * p.g, per_head = (rows + kJoinRows - 1) / kJoinRows;
  const int h = static_cast<int>(blockIdx.x / per_head);
  const int64_t i = (blockIdx.x - h * per_head) * kJoinRows + row8;
  after_previous();
  if (i >= rows) return;
  const int b = static_cast<int>(i / p.g), j = static_cast<int>(i - (int64_t)b * p.g);
  const int64_t out_row = (int64_t)b * p.h_q + h * p.g + j;
  const float *rec = plan.rec + out_row * kRecFloats<D>;
  const int4 tail = *reinterpret_cast<const int4 *>(rec + D);
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
    const int r = (b - g.seq0) * p.g + j, tile = r / kShRows, in = r - tile * kShRows;
    const int n = min(kShRows, g.rows - tile * kShRows);
    const int t0 = g.pair0 + (h * g.tiles + tile) * g.counted() + kShOver, per = plan.head->per;
    const int c0 = t0 / per, c1 = (t0 + g.blocks - 1) / per;
    const int64_t base = (int64_t)g.row0 + h * g.rows + tile * kShRows;
    const float4 *parts = reinterpret_cast<const float4 *>(plan.part);
    for (int c = c0; c <= c1; c += 4) {
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        v[u] = make_float2(-INFINITY, 0.f);
        o[u] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (c + u <= c1) {
          const int64_t k = (int64_t)(c + u) * kShRows + base;
          v[u] = plan.part_ml[k + in];
          o[u] = parts[k * (D / 4) + at * n + in];
        }
      }
      add(v, o);
    }
  }
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

template <int D, bool kFp16>
static cudaError_t run_shared(const Kv4SharedParams &p, cudaStream_t s) {
  int dev = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return e;
  ShPlan plan;
  shared_layout(D, p.dec.num_seqs, p.dec.h_q, p.num_groups, p.ws, &plan);
  const int ctas = sms < kShMaxCtas ? sms : kShMaxCtas;
  e = launch_kv4(kv4_share_kernel, dim3(1), kSetupThreads, 0, 1, s, p, plan, ctas, kShOver + 4);
  if (e != cudaSuccess) return e;
  auto *kernel = kv4_prefix_kernel<D, kFp16>;
  // more than half of an SM's: one CTA each, as its tensor memory allows
  constexpr int smem = Sh<D>::kBytes > 120 * 1024 ? Sh<D>::kBytes : 120 * 1024;
  e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  e = launch_kv4(kernel, dim3(static_cast<unsigned>(ctas)), kShThreads, smem, 1, s, p.dec, plan);
  if (e != cudaSuccess) return e;
  Kv4DecodeParams own = p.dec;
  own.lo = plan.lo;
  own.rec = plan.rec;
  e = launch_kv4_suffix(D, kFp16, own, s);
  if (e != cudaSuccess) return e;
  const int64_t rows = (int64_t)p.dec.num_seqs * p.dec.g;
  const int64_t joins = p.dec.h_k * ((rows + kJoinRows - 1) / kJoinRows);
  return launch_kv4(kv4_join_kernel<D, kFp16>, dim3(static_cast<unsigned>(joins)), kJoinRows * D / 4, 0, 1, s,
                    p.dec, plan);
}

cudaError_t launch_kv4_shared(int d, bool fp16, const Kv4SharedParams &p, cudaStream_t s) {
  if (d == 64) return fp16 ? run_shared<64, true>(p, s) : run_shared<64, false>(p, s);
  return fp16 ? run_shared<128, true>(p, s) : run_shared<128, false>(p, s);
}

}  // namespace nsa
