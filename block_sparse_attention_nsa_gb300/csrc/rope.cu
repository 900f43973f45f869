// rope.cu -- rotary positions of queries and keys, and their gradient.
//
// Pair i of a token at position n is turned by n w_i (include/nsa_rope.h).  With w_i in 2^-64 of a
// turn, n w_i modulo 2^64 is one integer product whose upper 32 bits are n times the w_i that is held, to
// 2^-33 of a turn; the top two of them choose the quarter, the rest is the argument of sincospif within a
// quarter turn's half.  (That w_i comes from a double: off by up to about 2^-52 of itself, which n multiplies.)
//
// Every value is read once and written once: HBM bounds it.  A warp takes a token, or a share of its
// heads where tokens are few.  It works out the token's rot_dim / 2 sines and cosines once, for all
// heads of q and k, two a lane at rot_dim 128, and keeps them in shared memory; an item is 8 pairs
// of one head, two 16-byte loads and stores, the first of them loaded ahead of the position's lookup and
// the sines.  A lane has one item at a time: with four in flight, 72 registers and half as many warps
// on an SM, 64K tokens of 16 + 4 heads of 128 took 110 us a call, now 100 (671 MB: 6.7 TB/s, of a copy's
// 6.8), and 9001 tokens of 6 + 3 heads of 64 8.4, now 6.6; CTAs of 256 threads in the place of 128: 102.
#include <cmath>
#include <cstring>

#include "kv4.cuh"
#include "nsa_rope.h"

namespace nsa {

constexpr int kRopeThreads = 128;
constexpr int kRopeMaxDim = 512;

struct RopeTensor {
  const uint16_t *in;
  uint16_t *out;
  int64_t its, ihs, ots, ohs;
};
struct RopeParams {
  int n, h_q, h_k, d, rot, num_seqs, shares, passes;
  RopeTensor q, k;
  const unsigned long long *freqs;
  const int32_t *positions, *cu, *start;
  int32_t *status;
  float mscale, sign;
  bool copy_q, copy_k;              // dimensions from rot on are copied
};

// Largest s in [0, S] with cu[s] <= t, or -1, for a non-decreasing cu: 32 probes at a time.
__device__ __forceinline__ int warp_seq_of(const int32_t *cu, int num_seqs, int t, int lane) {
  int lo = -1, hi = num_seqs + 1;   // cu[lo] <= t < cu[hi], with cu[-1] = -inf, cu[S + 1] = inf
  while (hi - lo > 1) {
    const int step = (hi - lo - 1 + 31) / 32, at = lo + 1 + lane * step;
    const bool below = at < hi && cu[at] <= t;
    const int n = __popc(__ballot_sync(0xffffffffu, below));   // a prefix where cu is in order
    const int first = lo + 1;
    hi = min(hi, first + n * step);
    if (n > 0) lo = first + (n - 1) * step;
  }
  return lo;
}

// cos and sin of 2 pi phase / 2^64, times m (and the sine's sign).
__device__ __forceinline__ float2 turn_of(unsigned long long phase, float m, float sign) {
  const unsigned a = static_cast<unsigned>((phase + 0x80000000ull) >> 32);
  const unsigned q = (a + 0x20000000u) >> 30;                  // the nearest quarter
  const int r = static_cast<int>(a - (q << 30));               // within half a quarter of it
  float s, c;
  sincospif(static_cast<float>(r) * 4.656612873077393e-10f, &s, &c);   // 2^-31
  const float x = q & 1 ? s : c, y = q & 1 ? c : s;
  return make_float2((q + 1) & 2 ? -m * x : m * x, q & 2 ? -m * sign * y : m * sign * y);
}

// Item i of a token's heads: its first 16-byte chunk in the source and in the destination.
struct RopePlace {
  const uint16_t *src;
  uint16_t *dst;
};
__device__ __forceinline__ RopePlace rope_place(const RopeParams &p, int t, int head, int at) {
  const bool k = head >= p.h_q;
  const RopeTensor &x = k ? p.k : p.q;
  const int h = k ? head - p.h_q : head;
  return RopePlace{x.in + t * x.its + h * x.ihs + at, x.out + t * x.ots + h * x.ohs + at};
}

template <bool kFp16>
__device__ __forceinline__ void turn_pairs(uint32_t &a, uint32_t &b, float4 cs) {   // two pairs
  const float2 x = unpack2<kFp16>(a), y = unpack2<kFp16>(b);
  a = pack2<kFp16>(x.x * cs.x - y.x * cs.y, x.y * cs.z - y.y * cs.w);
  b = pack2<kFp16>(y.x * cs.x + x.x * cs.y, y.y * cs.z + x.y * cs.w);
}
template <bool kFp16>
__device__ __forceinline__ uint32_t turn_pair(uint32_t a, float c, float s) {
  const float2 x = unpack2<kFp16>(a);
  return pack2<kFp16>(x.x * c - x.y * s, x.y * c + x.x * s);
}

template <bool kFp16, bool kInter>
__global__ void __launch_bounds__(kRopeThreads) rope_kernel(RopeParams p) {
  extern __shared__ __align__(16) float2 turns[];              // [warps][rot / 2]
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t task = (int64_t)blockIdx.x * (kRopeThreads / 32) + warp;
  const int t = static_cast<int>(task / p.shares), share = static_cast<int>(task - (int64_t)t * p.shares);
  if (t >= p.n) return;                                        // whole warps; no barrier below
  after_previous();
  const int units = p.rot >> 4, heads = p.h_q + p.h_k;
  const int second = kInter ? 8 : p.rot >> 1;                  // from an item's first chunk to its other
  const int dh = 32 / units, du = 32 - dh * units;             // 32 items on
  const int item0 = share * p.passes * 32 + lane;
  int head = item0 / units, unit = item0 - head * units;
  const int step = kInter ? 16 : 8;                            // elements from unit to unit

  uint4 a = make_uint4(0u, 0u, 0u, 0u), b = a;
  uint16_t *dst = nullptr;
  auto load = [&]() {
    if (head >= heads) return;
    const RopePlace w = rope_place(p, t, head, unit * step);
    a = *reinterpret_cast<const uint4 *>(w.src);
    b = *reinterpret_cast<const uint4 *>(w.src + second);
    dst = w.dst;
  };
  load();

  long long pos;
  if (p.positions) {
    pos = p.positions[t];
  } else {
    const int s = warp_seq_of(p.cu, p.num_seqs, t, lane);
    if (s >= p.num_seqs && t >= p.cu[p.num_seqs]) return;      // behind the last sequence
    bool ok = s >= 0 && s < p.num_seqs;
    if (ok) {
      const int lo = p.cu[s], hi = p.cu[s + 1];
      ok = lo >= 0 && lo <= t && t < hi;
      pos = (p.start ? (long long)p.start[s] : 0ll) + t - lo;
    }
    if (!ok) {
      if (lane == 0) raise(p.status, NSA_DEVERR_BAD_SEQLENS);
      return;
    }
  }
  float2 *mine = turns + warp * (p.rot >> 1);
  for (int i = lane; i < p.rot >> 1; i += 32)
    mine[i] = turn_of(p.freqs[i] * static_cast<unsigned long long>(pos), p.mscale, p.sign);
  __syncwarp();

  for (int pass = 0;;) {
    if (head < heads) {
      const float4 *cs = reinterpret_cast<const float4 *>(mine + unit * 8);
      const float4 c0 = cs[0], c1 = cs[1], c2 = cs[2], c3 = cs[3];
      if (kInter) {
        a.x = turn_pair<kFp16>(a.x, c0.x, c0.y);
        a.y = turn_pair<kFp16>(a.y, c0.z, c0.w);
        a.z = turn_pair<kFp16>(a.z, c1.x, c1.y);
        a.w = turn_pair<kFp16>(a.w, c1.z, c1.w);
        b.x = turn_pair<kFp16>(b.x, c2.x, c2.y);
        b.y = turn_pair<kFp16>(b.y, c2.z, c2.w);
        b.z = turn_pair<kFp16>(b.z, c3.x, c3.y);
        b.w = turn_pair<kFp16>(b.w, c3.z, c3.w);
      } else {
        turn_pairs<kFp16>(a.x, b.x, c0);
        turn_pairs<kFp16>(a.y, b.y, c1);
        turn_pairs<kFp16>(a.z, b.z, c2);
        turn_pairs<kFp16>(a.w, b.w, c3);
      }
      *reinterpret_cast<uint4 *>(dst) = a;
      *reinterpret_cast<uint4 *>(dst + second) = b;
    }
    if (++pass >= p.passes) break;
    head += dh;
    unit += du;
    if (unit >= units) {
      unit -= units;
      ++head;
    }
    load();
  }
  // what is not turned
  if (!p.copy_q && !p.copy_k) return;
  const int chunks = (p.d - p.rot) >> 3, h0 = p.copy_q ? 0 : p.h_q, h1 = p.copy_k ? heads : p.h_q;
  for (int i = share * 32 + lane; i < (h1 - h0) * chunks; i += p.shares * 32) {
    const int h = i / chunks;
    const RopePlace w = rope_place(p, t, h0 + h, p.rot + (i - h * chunks) * 8);
    *reinterpret_cast<uint4 *>(w.dst) = *reinterpret_cast<const uint4 *>(w.src);
  }
}

// Warps: a token each; where tokens are fewer than the 48 warps that an SM's registers hold, on all SMs, a
// token's heads are shared between warps, each of which works out the sines for itself (to 16 warps
// only: 3000 tokens of 16 + 4 heads 12 us in the place of 8.4, 1000 5.2 in that of 4.2).
static cudaError_t launch_rope(RopeParams &p, bool fp16, bool inter, cudaStream_t s) {
  const int64_t items = (int64_t)(p.h_q + p.h_k) * (p.rot / 16);
  int dev = 0;
  const cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const int64_t passes = (items + 31) / 32, want = (int64_t)sm_count(dev) * 48;
  int64_t shares = (want + p.n - 1) / p.n;
  if (shares > passes) shares = passes;
  p.passes = static_cast<int>((passes + shares - 1) / shares);
  p.shares = static_cast<int>((passes + p.passes - 1) / p.passes);
  constexpr int kWarps = kRopeThreads / 32;
  const int64_t ctas = ((int64_t)p.n * p.shares + kWarps - 1) / kWarps;
  const size_t smem = kWarps * (p.rot / 2) * sizeof(float2);
  auto *kernel = fp16 ? (inter ? rope_kernel<true, true> : rope_kernel<true, false>)
                      : (inter ? rope_kernel<false, true> : rope_kernel<false, false>);
  return launch_kv4(kernel, dim3(static_cast<unsigned>(ctas)), kRopeThreads, smem, 1, s, p);
}

namespace {

bool on(const void *ptr, size_t a) { return (reinterpret_cast<uintptr_t>(ptr) % a) == 0; }

// Rows of d elements at multiples of two strides do not overlap.
bool apart(int64_t n, int64_t ts, int64_t h, int64_t hs, int64_t d) {
  ts = ts < 0 ? -ts : ts;
  hs = hs < 0 ? -hs : hs;
  const bool token_first = n > 1 && (h <= 1 || ts < hs);
  const int64_t n0 = token_first ? n : h, s0 = token_first ? ts : hs;   // the shorter stride
  const int64_t n1 = token_first ? h : n, s1 = token_first ? hs : ts;
  if (n0 > 1 && s0 < d) return false;
  const int64_t span = (n0 > 1 ? (n0 - 1) * s0 : 0) + d;
  return n1 <= 1 || s1 >= span;
}

struct RopeArg {
  const void *data;
  int64_t ts, hs;
};

nsa_status tensor(const nsa_rope_dims *d, int heads, const RopeArg &in, const RopeArg &out, RopeTensor &x,
                  bool &copy) {
  std::memset(&x, 0, sizeof(x));
  copy = false;
  if (heads == 0) return NSA_OK;
  if (!in.data || !out.data) return NSA_ERR_INVALID_ARG;
  for (int64_t v : {in.ts, in.hs, out.ts, out.hs}) {
    if (v % 8) return NSA_ERR_INVALID_ARG;
    if (v <= -(int64_t(1) << 40) || v >= (int64_t(1) << 40)) return NSA_ERR_UNSUPPORTED;
  }
  if (!on(in.data, 16) || !on(out.data, 16)) return NSA_ERR_INVALID_ARG;
  if (!apart(d->num_tokens, out.ts, heads, out.hs, d->head_dim)) return NSA_ERR_INVALID_ARG;
  const bool same = in.data == out.data;
  if (same && ((d->num_tokens > 1 && in.ts != out.ts) || (heads > 1 && in.hs != out.hs)))
    return NSA_ERR_INVALID_ARG;
  x.in = static_cast<const uint16_t *>(in.data);
  x.out = static_cast<uint16_t *>(const_cast<void *>(out.data));
  x.its = in.ts;
  x.ihs = in.hs;
  x.ots = out.ts;
  x.ohs = out.hs;
  copy = !same && d->rot_dim < d->head_dim;
  return NSA_OK;
}

nsa_status run_rope(const nsa_rope_dims *dims, const RopeArg &q, const RopeArg &k, const uint64_t *freqs,
                    const int32_t *positions, const int32_t *cu, const int32_t *start, float mscale,
                    float sign, const RopeArg &q_out, const RopeArg &k_out, int32_t *status,
                    nsa_stream_t stream) {
  if (!dims) return NSA_ERR_INVALID_ARG;
  const nsa_rope_dims d = *dims;
  if (d.num_tokens < 0 || d.h_q < 0 || d.h_k < 0 || d.h_q + (int64_t)d.h_k < 1 || d.head_dim < 1 ||
      d.rot_dim < 1 || d.rot_dim > d.head_dim || d.num_seqs < 0 ||
      (d.interleaved != 0 && d.interleaved != 1) || !std::isfinite(mscale))
    return NSA_ERR_INVALID_ARG;
  if (d.dtype != NSA_BF16 && d.dtype != NSA_FP16) return NSA_ERR_UNSUPPORTED;
  if (d.head_dim % 8 || d.head_dim > kRopeMaxDim || d.rot_dim % 16) return NSA_ERR_UNSUPPORTED;
  if ((int64_t)d.num_tokens * ((int64_t)d.h_q + d.h_k) >= (int64_t(1) << 31)) return NSA_ERR_UNSUPPORTED;
  if ((int64_t)d.h_q + d.h_k >= (int64_t(1) << 24)) return NSA_ERR_UNSUPPORTED;
  if (d.num_tokens == 0) return NSA_OK;
  if (!freqs || (positions != nullptr) == (cu != nullptr) || (cu != nullptr) != (d.num_seqs > 0) ||
      (start && !cu))
    return NSA_ERR_INVALID_ARG;
  if (!on(freqs, 8) || !on(positions, 4) || !on(cu, 4) || !on(start, 4) || !on(status, 4))
    return NSA_ERR_INVALID_ARG;
  RopeParams p;
  std::memset(&p, 0, sizeof(p));
  nsa_status st = tensor(&d, d.h_q, q, q_out, p.q, p.copy_q);
  if (st == NSA_OK) st = tensor(&d, d.h_k, k, k_out, p.k, p.copy_k);
  if (st != NSA_OK) return st;
  p.n = d.num_tokens;
  p.h_q = d.h_q;
  p.h_k = d.h_k;
  p.d = d.head_dim;
  p.rot = d.rot_dim;
  p.num_seqs = d.num_seqs;
  p.freqs = reinterpret_cast<const unsigned long long *>(freqs);
  p.positions = positions;
  p.cu = cu;
  p.start = start;
  p.status = status;
  p.mscale = mscale;
  p.sign = sign;
  const cudaError_t e = launch_rope(p, d.dtype == NSA_FP16, d.interleaved != 0,
                                    reinterpret_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? NSA_OK : NSA_ERR_CUDA;
}

}  // namespace
}  // namespace nsa

using namespace nsa;

extern "C" {

nsa_status nsa_rope_freqs(int32_t rot_dim, double base, int32_t scaling, double factor,
                          double trained, double low, double high, uint64_t *host_freqs) {
  if (!host_freqs || rot_dim < 2 || rot_dim % 2 || !(base > 0) || !std::isfinite(base))
    return NSA_ERR_INVALID_ARG;
  if (scaling < NSA_ROPE_PLAIN || scaling > NSA_ROPE_RAMP) return NSA_ERR_INVALID_ARG;
  if (scaling != NSA_ROPE_PLAIN && !(factor > 0 && std::isfinite(factor))) return NSA_ERR_INVALID_ARG;
  if (scaling == NSA_ROPE_BASE) {
    if (rot_dim < 4) return NSA_ERR_INVALID_ARG;
    base *= std::pow(factor, (double)rot_dim / (rot_dim - 2));
    if (!(base > 0) || !std::isfinite(base)) return NSA_ERR_INVALID_ARG;
  }
  if (scaling == NSA_ROPE_RAMP &&
      !(trained > 0 && std::isfinite(trained) && std::isfinite(low) && std::isfinite(high) && low < high))
    return NSA_ERR_INVALID_ARG;
  constexpr double kTwoPi = 6.283185307179586476925286766559;
  for (int i = 0; i < rot_dim / 2; ++i) {
    double w = std::pow(base, -2.0 * i / rot_dim);
    if (scaling == NSA_ROPE_LINEAR) w /= factor;
    if (scaling == NSA_ROPE_RAMP) {
      double c = (trained * w / kTwoPi - low) / (high - low);
      c = c < 0 ? 0 : c > 1 ? 1 : c;
      w *= c + (1 - c) / factor;
    }
    if (!std::isfinite(w)) return NSA_ERR_INVALID_ARG;
    // whole turns do not show: the fraction, in 2^-64 (1 - 2^-53 at most, so it fits)
    const double turn = w / kTwoPi, part = turn - std::floor(turn);
    host_freqs[i] = static_cast<uint64_t>(std::ldexp(part, 64));
  }
  return NSA_OK;
}

nsa_status nsa_rope(const nsa_rope_dims *dims, const void *q, int64_t q_token_stride,
                    int64_t q_head_stride, const void *k, int64_t k_token_stride,
                    int64_t k_head_stride, const uint64_t *freqs, const int32_t *positions,
                    const int32_t *cu_seqlens, const int32_t *start, float mscale, void *q_out,
                    int64_t q_out_token_stride, int64_t q_out_head_stride, void *k_out,
                    int64_t k_out_token_stride, int64_t k_out_head_stride, int32_t *device_status,
                    nsa_stream_t stream) {
  return run_rope(dims, {q, q_token_stride, q_head_stride}, {k, k_token_stride, k_head_stride}, freqs,
                  positions, cu_seqlens, start, mscale, 1.f,
                  {q_out, q_out_token_stride, q_out_head_stride},
                  {k_out, k_out_token_stride, k_out_head_stride}, device_status, stream);
}

nsa_status nsa_rope_bwd(const nsa_rope_dims *dims, const void *dq_out, int64_t dq_out_token_stride,
                        int64_t dq_out_head_stride, const void *dk_out, int64_t dk_out_token_stride,
                        int64_t dk_out_head_stride, const uint64_t *freqs, const int32_t *positions,
                        const int32_t *cu_seqlens, const int32_t *start, float mscale, void *dq,
                        int64_t dq_token_stride, int64_t dq_head_stride, void *dk,
                        int64_t dk_token_stride, int64_t dk_head_stride, int32_t *device_status,
                        nsa_stream_t stream) {
  return run_rope(dims, {dq_out, dq_out_token_stride, dq_out_head_stride},
                  {dk_out, dk_out_token_stride, dk_out_head_stride}, freqs, positions, cu_seqlens, start,
                  mscale, -1.f, {dq, dq_token_stride, dq_head_stride},
                  {dk, dk_token_stride, dk_head_stride}, device_status, stream);
}

}  // extern "C"
