// kv4_rows.cu -- rows of K and V into and out of the 4-bit pages.
//
// Per group x of 64 dimensions: zero = fp16(min x), scale = fp16((max x - zero) / 15),
// code = nearest whole number to (x - zero) / scale (ties to even) in 0 ... 15; reading
// gives code * scale + zero, rounded once.  Every value is read once and written once, so
// HBM bounds both directions: 4 d bytes of 16-bit K and V against d + d / 8 stored.
//
// Eight lanes own a group, eight dimensions each: one 16-byte access of the 16-bit row,
// three shuffles for the minimum and maximum, one 32-bit word of codes.  A warp covers
// K and V of one (token, head) at d = 128, of two at d = 64, so that its code words fill
// whole 32-byte sectors.
#include "kv4.cuh"

namespace nsa {

constexpr int kRowThreads = 256;
constexpr float kHalfMax = 65504.f;

// Where a thread's group lies: row, head, K or V, group of the row.
struct RowGroup {
  int t, h, kv, gi;
};
template <int D>
__device__ __forceinline__ RowGroup row_group(int64_t i, int h_k) {
  constexpr int kG = Kv4Tile<D>::kG;
  RowGroup r;
  r.gi = static_cast<int>(i % kG);
  r.kv = static_cast<int>(i / kG % 2);
  const int64_t th = i / (2 * kG);
  r.t = static_cast<int>(th / h_k);
  r.h = static_cast<int>(th - (int64_t)r.t * h_k);
  return r;
}

// The tile that holds a slot of head h.
template <int D>
__device__ __forceinline__ uint8_t *slot_tile(uint8_t *pool, int h_k, int page_log2, int h,
                                              int slot) {
  const int64_t page = slot >> page_log2;
  const int in = slot & ((1 << page_log2) - 1);
  return pool + ((page * h_k + h) * (int64_t)((1 << page_log2) / kKv4Tile) + in / kKv4Tile) *
                    Kv4Tile<D>::kBytes;
}

// (x - zero) / scale to the nearest whole number, ties to even, in 0 ... 15: the rounded
// product with 1 / scale is at most one off, and only next to a border; its residual
// x - zero - c * scale, exact in one fused step, says which side it is on.
__device__ __forceinline__ uint32_t code4(float x, float zero, float scale, float inv) {
  const float t = __fsub_rn(x, zero);
  const float m = __fadd_rn(__fmul_rn(t, inv), 12582912.f);   // 1.5 * 2^23: rounds to a whole number
  float c = __fsub_rn(m, 12582912.f);
  const float r = __fmaf_rn(-c, scale, t), half = 0.5f * scale;
  const bool odd = __float_as_uint(m) & 1u;
  if (fabsf(r) > half || (fabsf(r) == half && odd)) c += r > 0.f ? 1.f : -1.f;
  return static_cast<uint32_t>(fminf(fmaxf(c, 0.f), 15.f));
}

template <int D, bool kFp16>
__global__ void __launch_bounds__(kRowThreads) kv4_append_kernel(Kv4RowParams p) {
  using T = Kv4Tile<D>;
  const int lane = threadIdx.x & 31, j = lane & 7;
  const int64_t groups = (int64_t)p.n * p.h_k * 2 * T::kG;
  const int64_t i = ((int64_t)blockIdx.x * kRowThreads + threadIdx.x) >> 3;
  const bool in = i < groups;
  const RowGroup r = row_group<D>(in ? i : 0, p.h_k);
  const int slot = in ? p.slots[r.t] : -1;
  const bool good = slot >= 0 && (slot >> p.page_log2) < p.num_pages;
  if (in && slot != -1 && !good && r.h == 0 && r.kv == 0 && r.gi == 0 && j == 0)
    raise(p.status, NSA_DEVERR_BAD_INDEX);
  uint4 raw = make_uint4(0u, 0u, 0u, 0u);
  if (good) {
    const uint16_t *src = static_cast<const uint16_t *>(r.kv ? p.v : p.k) +
                          r.t * (r.kv ? p.v_ts : p.k_ts) + r.h * (r.kv ? p.v_hs : p.k_hs) +
                          r.gi * 64 + j * 8;
    raw = *reinterpret_cast<const uint4 *>(src);
  }
  const uint32_t w4[4] = {raw.x, raw.y, raw.z, raw.w};
  float x[8];
  bool nan = false;
  float lo = kHalfMax, hi = -kHalfMax;
#pragma unroll
  for (int u = 0; u < 4; ++u) {
    const float2 f = unpack2<kFp16>(w4[u]);
    x[2 * u] = f.x;
    x[2 * u + 1] = f.y;
  }
#pragma unroll
  for (int u = 0; u < 8; ++u) {
    nan |= x[u] != x[u];
    x[u] = fminf(fmaxf(x[u], -kHalfMax), kHalfMax);
    lo = fminf(lo, x[u]);
    hi = fmaxf(hi, x[u]);
  }
#pragma unroll
  for (int o = 1; o < 8; o <<= 1) {
    lo = fminf(lo, __shfl_xor_sync(0xffffffffu, lo, o));
    hi = fmaxf(hi, __shfl_xor_sync(0xffffffffu, hi, o));
  }
  nan = (__ballot_sync(0xffffffffu, nan) >> (lane & 24) & 0xffu) != 0;
  __half zh = __float2half_rn(lo);
  const float zero = __half2float(zh);
  __half sh = __float2half_rn(__fdiv_rn(__fsub_rn(hi, zero), 15.f));
  if (nan) {
    zh = __ushort_as_half(0x7fff);
    sh = __ushort_as_half(0);
  }
  const float scale = __half2float(sh), inv = scale > 0.f ? __fdiv_rn(1.f, scale) : 0.f;
  uint32_t word = 0;
  if (scale > 0.f) {
#pragma unroll
    for (int u = 0; u < 8; ++u) word |= code4(x[u], zero, scale, inv) << (4 * u);
  }
  if (good) {
    uint8_t *tile = slot_tile<D>(p.pool, p.h_k, p.page_log2, r.h, slot);
    const int row = slot & (kKv4Tile - 1);
    *reinterpret_cast<uint32_t *>(tile + r.kv * T::kV + row * T::kRow +
                                  (j * T::kG + r.gi) * 4) = word;
    if (j < 2)   // scale, zero
      *reinterpret_cast<__half *>(tile + T::kPar + (2 * r.kv + j) * T::kArr +
                                  (row * T::kG + r.gi) * 2) = j ? zh : sh;
  }
}

template <int D, bool kFp16>
__global__ void __launch_bounds__(kRowThreads) kv4_read_kernel(Kv4RowParams p) {
  using T = Kv4Tile<D>;
  const int j = threadIdx.x & 7;
  const int64_t groups = (int64_t)p.n * p.h_k * 2 * T::kG;
  const int64_t i = ((int64_t)blockIdx.x * kRowThreads + threadIdx.x) >> 3;
  if (i >= groups) return;
  const RowGroup r = row_group<D>(i, p.h_k);
  const int slot = p.slots[r.t];
  const bool good = slot >= 0 && (slot >> p.page_log2) < p.num_pages;
  uint4 out = make_uint4(0u, 0u, 0u, 0u);
  if (good) {
    const uint8_t *tile = slot_tile<D>(p.pool, p.h_k, p.page_log2, r.h, slot);
    const int row = slot & (kKv4Tile - 1);
    const uint32_t word = *reinterpret_cast<const uint32_t *>(
        tile + r.kv * T::kV + row * T::kRow + (j * T::kG + r.gi) * 4);
    const __half *par = reinterpret_cast<const __half *>(tile + T::kPar + 2 * r.kv * T::kArr) +
                        row * T::kG + r.gi;
    const float scale = __half2float(par[0]), zero = __half2float(par[T::kArr / 2]);
    float x[8];
#pragma unroll
    for (int u = 0; u < 8; ++u)   // code * scale is exact: the only fp32 rounding is the sum's
      x[u] = fmaf(static_cast<float>(word >> (4 * u) & 15u), scale, zero);
    out = make_uint4(pack2<kFp16>(x[0], x[1]), pack2<kFp16>(x[2], x[3]), pack2<kFp16>(x[4], x[5]),
                     pack2<kFp16>(x[6], x[7]));
  } else if (slot != -1 && r.h == 0 && r.kv == 0 && r.gi == 0 && j == 0) {
    raise(p.status, NSA_DEVERR_BAD_INDEX);
  }
  uint16_t *dst = static_cast<uint16_t *>(r.kv ? p.v_out : p.k_out) +
                  ((int64_t)r.t * p.h_k + r.h) * D + r.gi * 64 + j * 8;
  *reinterpret_cast<uint4 *>(dst) = out;
}

template <int D>
static unsigned row_grid(const Kv4RowParams &p) {
  const int64_t threads = (int64_t)p.n * p.h_k * 2 * Kv4Tile<D>::kG * 8;
  return static_cast<unsigned>((threads + kRowThreads - 1) / kRowThreads);
}

template <int D>
static cudaError_t run_rows(bool append, bool fp16, const Kv4RowParams &p, cudaStream_t s) {
  auto *kernel = append ? (fp16 ? kv4_append_kernel<D, true> : kv4_append_kernel<D, false>)
                        : (fp16 ? kv4_read_kernel<D, true> : kv4_read_kernel<D, false>);
  kernel<<<row_grid<D>(p), kRowThreads, 0, s>>>(p);
  return cudaGetLastError();
}

cudaError_t launch_kv4_append(int d, bool fp16, const Kv4RowParams &p, cudaStream_t s) {
  return d == 64 ? run_rows<64>(true, fp16, p, s) : run_rows<128>(true, fp16, p, s);
}
cudaError_t launch_kv4_read(int d, bool fp16, const Kv4RowParams &p, cudaStream_t s) {
  return d == 64 ? run_rows<64>(false, fp16, p, s) : run_rows<128>(false, fp16, p, s);
}

}  // namespace nsa
