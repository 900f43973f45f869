// kv4_rows.cu -- rows of K and V into and out of the 4-bit pages.
//
// Per group x of 64 dimensions: zero = fp16(min x), scale = fp16((max x - zero) / 15),
// code = nearest whole number to (x - zero) / scale (ties to even) in 0 ... 15; reading
// gives code * scale + zero, rounded once.  Every value is read once and written once, so
// HBM bounds both directions: 4 d bytes of 16-bit K and V against d + d / 8 stored.
//
// Eight lanes own a group, eight dimensions each: one 16-byte access of the 16-bit row,
// three shuffles for the minimum and maximum, one 32-bit word of codes.  A warp covers K and V
// of one head, of one token at a time (two at d = 64), so that code words fill whole 32-byte
// sectors, and takes kRows consecutive tokens, whose loads it issues together.  64K tokens of 4
// heads at d = 128 (172 MB, 25.4 us at the measured 6.78 TB/s): append 40.0 us (4.3 TB/s, 76 % of
// the issue slots busy), read 30.8 us (5.6 TB/s, 77 %).
#include "kv4.cuh"

namespace nsa {

constexpr int kRowThreads = 256;
constexpr int kRows = 4;
constexpr float kHalfMax = 65504.f;

// Tokens of a warp: kRows in turn, at d = 64 two such runs side by side.
template <int D>
constexpr int kWarpTokens = kRows * 128 / D;

// A lane's place: its first token, and its group of every token.
struct RowPlace {
  int t0, h, kv, gi, j;
};
template <int D>
__device__ __forceinline__ RowPlace row_place(const Kv4RowParams &p) {
  constexpr int kG = Kv4Tile<D>::kG;
  const int lane = threadIdx.x & 31, part = lane >> 3;
  const uint64_t task = (uint64_t)blockIdx.x * (kRowThreads / 32) + (threadIdx.x >> 5);
  uint32_t tb, h;                                          // a warp has one head
  if (task >> 32) {
    tb = static_cast<uint32_t>(task / p.h_k);
    h = static_cast<uint32_t>(task - (uint64_t)tb * p.h_k);
  } else {
    tb = static_cast<uint32_t>(task) / static_cast<uint32_t>(p.h_k);
    h = static_cast<uint32_t>(task) - tb * p.h_k;
  }
  RowPlace r;
  const uint64_t t0 = (uint64_t)tb * kWarpTokens<D> + (kG == 2 ? 0 : (part >> 1) * kRows);
  r.t0 = static_cast<int>(min(t0, (uint64_t)p.n));
  r.h = h;
  r.kv = kG == 2 ? part >> 1 : part & 1;
  r.gi = kG == 2 ? part & 1 : 0;
  r.j = lane & 7;
  return r;
}

// The slots of a warp's tokens, -1 where there is none or it is not valid.
__device__ __forceinline__ void load_slots(const Kv4RowParams &p, int t0, int (&slot)[kRows]) {
  bool bad = false;
#pragma unroll
  for (int k = 0; k < kRows; ++k) {
    slot[k] = t0 + k < p.n ? p.slots[t0 + k] : -1;
    if (slot[k] < 0 || (slot[k] >> p.page_log2) >= p.num_pages) {
      bad |= slot[k] != -1;
      slot[k] = -1;
    }
  }
  if (bad && (threadIdx.x & 15) == 0) raise(p.status, NSA_DEVERR_BAD_INDEX);
}

// Offset of the tile that holds a slot of head h (tiles are counted in 32 bits: 2^32 of them
// would be 9 TB).
template <int D>
__device__ __forceinline__ int64_t slot_tile(const Kv4RowParams &p, int h, int slot) {
  const uint32_t page = static_cast<uint32_t>(slot) >> p.page_log2;
  const uint32_t in = slot & ((1 << p.page_log2) - 1);
  const uint32_t tile = ((page * p.h_k + h) << (p.page_log2 - 5)) + (in >> 5);
  return (int64_t)tile * Kv4Tile<D>::kBytes;
}

// Larger of two pairs of 16-bit floats; a NaN stays.
template <bool kFp16>
__device__ __forceinline__ uint32_t max2(uint32_t a, uint32_t b) {
  if constexpr (kFp16) {
    const __half2 m = __hmax2_nan(*reinterpret_cast<__half2 *>(&a), *reinterpret_cast<__half2 *>(&b));
    return *reinterpret_cast<const uint32_t *>(&m);
  } else {
    const __nv_bfloat162 m = __hmax2_nan(*reinterpret_cast<__nv_bfloat162 *>(&a),
                                         *reinterpret_cast<__nv_bfloat162 *>(&b));
    return *reinterpret_cast<const uint32_t *>(&m);
  }
}
template <bool kFp16>
__device__ __forceinline__ uint32_t min2(uint32_t a, uint32_t b) {
  if constexpr (kFp16) {
    const __half2 m = __hmin2_nan(*reinterpret_cast<__half2 *>(&a), *reinterpret_cast<__half2 *>(&b));
    return *reinterpret_cast<const uint32_t *>(&m);
  } else {
    const __nv_bfloat162 m = __hmin2_nan(*reinterpret_cast<__nv_bfloat162 *>(&a),
                                         *reinterpret_cast<__nv_bfloat162 *>(&b));
    return *reinterpret_cast<const uint32_t *>(&m);
  }
}
// a[i] of four, by selects.
template <typename V>
__device__ __forceinline__ V pick(const V (&a)[kRows], int i) {
  static_assert(kRows == 4, "two bits choose a row");
  return i & 2 ? (i & 1 ? a[3] : a[2]) : (i & 1 ? a[1] : a[0]);
}

// x / y for inv = 1 / y rounded: the product, corrected by its exact residual, is the correctly
// rounded quotient (Markstein, 1990).
__device__ __forceinline__ float quotient(float x, float y, float inv) {
  const float q = __fmul_rn(x, inv);
  return __fmaf_rn(__fmaf_rn(-q, y, x), inv, q);
}

// The eight codes of a lane: (x - zero) / scale to the nearest whole number, ties to even, as
// adding 1.5 * 2^23 rounds.  kHeld: held to finite x and to 0 ... 15, which most groups need
// no step for.
template <bool kFp16, bool kHeld>
__device__ __forceinline__ uint32_t code_word(const uint32_t (&w4)[4], float zero, float scale,
                                              float inv) {
  const Pair minus_zero(-zero, -zero), minus_scale(-scale, -scale), inv2(inv, inv);
  const Pair magic(12582912.f, 12582912.f);
  uint32_t word = 0;
#pragma unroll
  for (int u = 3; u >= 0; --u) {         // the lowest nibble last: each step shifts by four bits
    float2 f = unpack2<kFp16>(w4[u]);
    if (kHeld) {
      f.x = fminf(fmaxf(f.x, -kHalfMax), kHalfMax);
      f.y = fminf(fmaxf(f.y, -kHalfMax), kHalfMax);
    }
    const Pair t = Pair(f.x, f.y) + minus_zero, q0 = t * inv2;
    Pair q = fma(fma(q0, minus_scale, t), inv2, q0);   // as quotient(), two at a time
    if (kHeld) {
      const float2 g = q.get();
      q = Pair(fminf(fmaxf(g.x, 0.f), 15.f), fminf(fmaxf(g.y, 0.f), 15.f));
    }
    const float2 m = (q + magic).get();
    word = word * 16u + __float_as_uint(m.y);
    word = word * 16u + __float_as_uint(m.x);
  }
  return word - 0x4b400000u * 0x11111111u;   // less the bits of 1.5 * 2^23 in each of the eight
}

template <int D, bool kFp16>
__global__ void __launch_bounds__(kRowThreads) kv4_append_kernel(Kv4RowParams p) {
  using T = Kv4Tile<D>;
  const RowPlace r = row_place<D>(p);
  int slot[kRows];
  after_previous();
  load_slots(p, r.t0, slot);
  const int64_t ts = r.kv ? p.v_ts : p.k_ts, hs = r.kv ? p.v_hs : p.k_hs;
  const uint16_t *src = static_cast<const uint16_t *>(r.kv ? p.v : p.k) + r.t0 * ts + r.h * hs +
                        r.gi * 64 + r.j * 8;
  uint4 raw[kRows];
#pragma unroll
  for (int k = 0; k < kRows; ++k) {
    raw[k] = make_uint4(0u, 0u, 0u, 0u);
    if (slot[k] >= 0)
      raw[k] = __ldcs(reinterpret_cast<const uint4 *>(src + k * ts));
  }
  // the groups' smallest (negated) and largest values, packed
  uint32_t ends[kRows];
#pragma unroll
  for (int k = 0; k < kRows; ++k) {
    const uint32_t lo = min2<kFp16>(min2<kFp16>(raw[k].x, raw[k].y), min2<kFp16>(raw[k].z, raw[k].w));
    const uint32_t hi = max2<kFp16>(max2<kFp16>(raw[k].x, raw[k].y), max2<kFp16>(raw[k].z, raw[k].w));
    uint32_t e = max2<kFp16>(__byte_perm(lo, hi, 0x5410) ^ 0x8000u, __byte_perm(lo, hi, 0x7632) ^ 0x8000u);
#pragma unroll
    for (int o = 1; o < 8; o <<= 1) e = max2<kFp16>(e, __shfl_xor_sync(0xffffffffu, e, o));
    ends[k] = e;
  }
  // Lane j works out the zero and scale of row j % 4 for the others of its group, and stores
  // one of the two.
  const int mine = r.j & 3, my_slot = pick(slot, mine);
  const float2 e = unpack2<kFp16>(pick(ends, mine));
  const bool nan = e.x != e.x || e.y != e.y;
  const float low = -e.x, high = e.y;
  const float lo = fminf(fmaxf(low, -kHalfMax), kHalfMax);
  const float hi = fminf(fmaxf(high, -kHalfMax), kHalfMax);
  const __half zh = nan ? __ushort_as_half(0x7fff) : __float2half_rn(lo);
  const float my_zero = __half2float(zh);
  const __half sh = nan ? __ushort_as_half(0)
                        : __float2half_rn(quotient(__fsub_rn(hi, my_zero), 15.f, 1.f / 15.f));
  const float my_scale = __half2float(sh), my_inv = __frcp_rn(my_scale);
  const uint32_t both = __half_as_ushort(zh) | static_cast<uint32_t>(__half_as_ushort(sh)) << 16;
  const bool stored = my_slot >= 0;
  // no code can leave 0 ... 15 where zero is not above the smallest value and the largest
  // is not 15.5 steps above it
  const bool held = __any_sync(0xffffffffu, stored && !(my_zero <= low &&
                                                        high - my_zero < 15.4f * my_scale));
  if (stored) {
    const int row = my_slot & (kKv4Tile - 1), which = r.j >> 2;   // 0: scale, 1: zero
    *reinterpret_cast<__half *>(p.pool + slot_tile<D>(p, r.h, my_slot) + T::kPar +
                                (2 * r.kv + which) * T::kArr + (row * T::kG + r.gi) * 2) =
        which ? zh : sh;
  }
#pragma unroll
  for (int k = 0; k < kRows; ++k) {
    const int from = (threadIdx.x & 24) + k;
    const uint32_t zs = __shfl_sync(0xffffffffu, both, from);
    const float inv = __shfl_sync(0xffffffffu, my_inv, from);
    const float2 f = unpack2<true>(zs);
    const uint32_t w4[4] = {raw[k].x, raw[k].y, raw[k].z, raw[k].w};
    uint32_t word = held ? code_word<kFp16, true>(w4, f.x, f.y, inv)
                         : code_word<kFp16, false>(w4, f.x, f.y, inv);
    if (!(f.y > 0.f)) word = 0;
    if (slot[k] >= 0)
      *reinterpret_cast<uint32_t *>(p.pool + slot_tile<D>(p, r.h, slot[k]) + r.kv * T::kV +
                                    (slot[k] & (kKv4Tile - 1)) * T::kRow + (r.j * T::kG + r.gi) * 4) =
          word;
  }
}

template <int D, bool kFp16>
__global__ void __launch_bounds__(kRowThreads) kv4_read_kernel(Kv4RowParams p) {
  using T = Kv4Tile<D>;
  const RowPlace r = row_place<D>(p);
  int slot[kRows];
  after_previous();
  load_slots(p, r.t0, slot);
  uint32_t word[kRows];
  __half scale[kRows], zero[kRows];
#pragma unroll
  for (int k = 0; k < kRows; ++k) {
    word[k] = 0;
    scale[k] = zero[k] = __ushort_as_half(0);
    if (slot[k] >= 0) {
      const uint8_t *tile = p.pool + slot_tile<D>(p, r.h, slot[k]);
      const int row = slot[k] & (kKv4Tile - 1);
      word[k] = *reinterpret_cast<const uint32_t *>(tile + r.kv * T::kV + row * T::kRow +
                                                   (r.j * T::kG + r.gi) * 4);
      const __half *par = reinterpret_cast<const __half *>(tile + T::kPar + 2 * r.kv * T::kArr) +
                          row * T::kG + r.gi;
      scale[k] = *par;
      zero[k] = par[T::kArr / 2];
    }
  }
#pragma unroll
  for (int k = 0; k < kRows; ++k) {
    if (r.t0 + k >= p.n) break;
    const float s = __half2float(scale[k]), z = __half2float(zero[k]);
    // codes n and n + 4 as the low bits of two fp16s above 1024; the difference is exact
    float x[8];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const uint32_t c2 = (word[k] >> (4 * u) & 0x000f000fu) | 0x64006400u;
      const __half2 c = __hsub2(*reinterpret_cast<const __half2 *>(&c2), __float2half2_rn(1024.f));
      x[u] = fmaf(__low2float(c), s, z);   // code * scale is exact: only the sum rounds
      x[u + 4] = fmaf(__high2float(c), s, z);
    }
    uint16_t *dst = static_cast<uint16_t *>(r.kv ? p.v_out : p.k_out) +
                    ((int64_t)(r.t0 + k) * p.h_k + r.h) * D + r.gi * 64 + r.j * 8;
    __stcs(reinterpret_cast<uint4 *>(dst),
           make_uint4(pack2<kFp16>(x[0], x[1]), pack2<kFp16>(x[2], x[3]), pack2<kFp16>(x[4], x[5]),
                      pack2<kFp16>(x[6], x[7])));
  }
}

template <int D>
static cudaError_t run_rows(bool append, bool fp16, const Kv4RowParams &p, cudaStream_t s) {
  auto *kernel = append ? (fp16 ? kv4_append_kernel<D, true> : kv4_append_kernel<D, false>)
                        : (fp16 ? kv4_read_kernel<D, true> : kv4_read_kernel<D, false>);
  const int64_t warps = kRowThreads / 32;
  const int64_t tasks = ((int64_t)p.n + kWarpTokens<D> - 1) / kWarpTokens<D> * p.h_k;
  return launch_kv4(kernel, dim3(static_cast<unsigned>((tasks + warps - 1) / warps)), kRowThreads, 0,
                    1, s, p);
}

cudaError_t launch_kv4_append(int d, bool fp16, const Kv4RowParams &p, cudaStream_t s) {
  return d == 64 ? run_rows<64>(true, fp16, p, s) : run_rows<128>(true, fp16, p, s);
}
cudaError_t launch_kv4_read(int d, bool fp16, const Kv4RowParams &p, cudaStream_t s) {
  return d == 64 ? run_rows<64>(false, fp16, p, s) : run_rows<128>(false, fp16, p, s);
}

}  // namespace nsa
