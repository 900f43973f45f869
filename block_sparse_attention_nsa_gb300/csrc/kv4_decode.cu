// kv4_decode.cu -- one-step decode of attention over the 4-bit paged KV cache.
//
// Request b's new token attends, per KV head, to the kept keys i of its pages:
//   S_hi = scale * q_h . k_i,  p_hi = exp(S_hi - max S),  out_h = sum p_hi v_i / sum p_hi,
// with k_i = c * s + z per group of 64 dimensions.
//
// One CTA of eight warps per (sequence, KV head, up to eight query heads).  A tile is the 32 tokens of one record
// tile; warp w takes tiles w, w + 8, ...  Lane l owns key l for the scores (online softmax
// per head) and D / 32 consecutive dimensions of the output.  The warps' (m, l, O) are
// merged in shared memory at the end.
#include "kv4.cuh"

namespace nsa {

constexpr int kK4Warps = 8;

template <bool kFp16>
__device__ __forceinline__ float load16(const uint16_t *p) {
  const unsigned short u = *p;
  return kFp16 ? __half2float(__ushort_as_half(u)) : __uint_as_float(static_cast<uint32_t>(u) << 16);
}

template <int D, int GM, bool kFp16>
__global__ void __launch_bounds__(kK4Warps * 32) kv4_decode_kernel(Kv4DecodeParams p) {
  using T = Kv4Tile<D>;
  constexpr int E = D / 32;
  __shared__ float qs[GM * D];
  __shared__ float pw[kK4Warps][GM * 32];
  __shared__ float mg[kK4Warps][GM][D + 2];
  __shared__ int32_t kept[32];
  __shared__ int n_kept;
  const int b = blockIdx.x, h = blockIdx.y, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int head0 = blockIdx.z * GM, g = min(GM, p.g - head0), page = 1 << p.page_log2, tpl = p.page_log2 - 5;   // log2 tiles per page
  const int64_t cap = (int64_t)p.width << p.page_log2;
  const int raw = p.lens[b];
  const int len = static_cast<int>(raw < 0 ? 0 : (raw > cap ? cap : raw));
  int32_t err = raw != len ? NSA_DEVERR_BAD_SEQLENS : 0;
  const int lo = p.window > 0 && len > p.window ? len - p.window : 0;   // first key seen
  for (int i = tid; i < GM * D; i += kK4Warps * 32)
    qs[i] = i < g * D ? load16<kFp16>(static_cast<const uint16_t *>(p.q) +
                                      ((int64_t)b * p.h_q + h * p.g + head0) * D + i) * p.scale_log2
                      : 0.f;
  if (p.sel && warp == 0) {
    const int nblk = (len + page - 1) >> p.page_log2, c = len > 0 ? (len - 1) >> p.page_log2 : -1;
    const int blk = lane < p.topk ? p.sel[((int64_t)h * p.num_seqs + b) * p.topk + lane] : -1;
    if (blk < -1 || blk >= nblk) err |= lane < p.topk ? NSA_DEVERR_BAD_INDEX : 0;
    bool ok = blk >= 0 && blk <= c;
    const uint32_t same = __match_any_sync(0xffffffffu, blk);
    ok = ok && (same & ((1u << lane) - 1u)) == 0;
    const uint32_t m = __ballot_sync(0xffffffffu, ok);
    if (ok) kept[__popc(m & ((1u << lane) - 1u))] = blk;
    if (lane == 0) n_kept = __popc(m);
  }
  __syncthreads();
  const int tile0 = lo >> 5, ntiles = p.sel ? n_kept << tpl : ((len + 31) >> 5) - tile0;

  float m_run[GM], l_run[GM], o[GM][E];
#pragma unroll
  for (int hh = 0; hh < GM; ++hh) {
    m_run[hh] = -INFINITY;
    l_run[hh] = 0.f;
#pragma unroll
    for (int e = 0; e < E; ++e) o[hh][e] = 0.f;
  }
  for (int n = warp; n < ntiles; n += kK4Warps) {
    const int key0 = p.sel ? (kept[n >> tpl] << p.page_log2) + ((n & ((1 << tpl) - 1)) << 5)
                           : (tile0 + n) << 5;
    if (key0 >= len || key0 + 32 <= lo) continue;
    const int pg = p.table[(int64_t)b * p.width + (key0 >> p.page_log2)];
    if (pg < 0 || pg >= p.num_pages) {
      err |= NSA_DEVERR_BAD_INDEX;
      continue;
    }
    const uint8_t *tile = p.pool + ((((int64_t)pg * p.h_k + h) << tpl) +
                                    ((key0 & (page - 1)) >> 5)) * (int64_t)T::kBytes;
    const __half *par = reinterpret_cast<const __half *>(tile + T::kPar);
    const bool seen = key0 + lane < len && key0 + lane >= lo;
    float s[GM];
#pragma unroll
    for (int hh = 0; hh < GM; ++hh) s[hh] = 0.f;
    for (int w = 0; w < D / 8; ++w) {
      const int gi = w % T::kG, j = w / T::kG;
      const uint32_t word = *reinterpret_cast<const uint32_t *>(tile + lane * T::kRow + w * 4);
      const float sc = __half2float(par[lane * T::kG + gi]);
      const float ze = __half2float(par[(32 + lane) * T::kG + gi]);
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        const float x = fmaf(static_cast<float>(word >> (4 * u) & 15u), sc, ze);
#pragma unroll
        for (int hh = 0; hh < GM; ++hh)
          s[hh] = fmaf(qs[hh * D + gi * 64 + j * 8 + u], x, s[hh]);
      }
    }
#pragma unroll
    for (int hh = 0; hh < GM; ++hh) {
      float mx = seen ? s[hh] : -INFINITY;
#pragma unroll
      for (int off = 16; off > 0; off >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, off));
      const float m_new = fmaxf(m_run[hh], mx);
      const float alpha = ex2_approx(m_run[hh] - m_new);
      const float pv = seen ? ex2_approx(s[hh] - m_new) : 0.f;
      pw[warp][hh * 32 + lane] = pv;
      float ps = pv;
#pragma unroll
      for (int off = 16; off > 0; off >>= 1) ps += __shfl_xor_sync(0xffffffffu, ps, off);
      l_run[hh] = l_run[hh] * alpha + ps;
      m_run[hh] = m_new;
#pragma unroll
      for (int e = 0; e < E; ++e) o[hh][e] *= alpha;
    }
    __syncwarp();
    // dimensions lane * E ...: one word of the row
    const int dim = lane * E, gi = dim / 64, w = (dim % 64 / 8) * T::kG + gi;
    for (int r = max(0, lo - key0); r < min(32, len - key0); ++r) {
      const uint32_t word =
          *reinterpret_cast<const uint32_t *>(tile + T::kV + r * T::kRow + w * 4) >> (4 * (dim % 8));
      const float sc = __half2float(par[(64 + r) * T::kG + gi]);
      const float ze = __half2float(par[(96 + r) * T::kG + gi]);
#pragma unroll
      for (int e = 0; e < E; ++e) {
        const float x = fmaf(static_cast<float>(word >> (4 * e) & 15u), sc, ze);
#pragma unroll
        for (int hh = 0; hh < GM; ++hh) o[hh][e] = fmaf(pw[warp][hh * 32 + r], x, o[hh][e]);
      }
    }
    __syncwarp();
  }
  if (err) raise(p.status, err);
#pragma unroll
  for (int hh = 0; hh < GM; ++hh) {
#pragma unroll
    for (int e = 0; e < E; ++e) mg[warp][hh][lane * E + e] = o[hh][e];
    if (lane == 0) {
      mg[warp][hh][D] = m_run[hh];
      mg[warp][hh][D + 1] = l_run[hh];
    }
  }
  __syncthreads();
  for (int hh = warp; hh < g; hh += kK4Warps) {
    float M = -INFINITY, lsum = 0.f, acc[E];
    for (int w = 0; w < kK4Warps; ++w) M = fmaxf(M, mg[w][hh][D]);
#pragma unroll
    for (int e = 0; e < E; ++e) acc[e] = 0.f;
    for (int w = 0; w < kK4Warps; ++w) {
      if (mg[w][hh][D + 1] == 0.f) continue;   // a warp without keys
      const float wt = ex2_approx(mg[w][hh][D] - M);
      lsum += wt * mg[w][hh][D + 1];
#pragma unroll
      for (int e = 0; e < E; ++e) acc[e] = fmaf(wt, mg[w][hh][lane * E + e], acc[e]);
    }
    const bool any = lsum != 0.f;   // a NaN sum stays one
    const float inv = any ? 1.f / lsum : 0.f;
    uint16_t *dst =
        static_cast<uint16_t *>(p.out) + ((int64_t)b * p.h_q + h * p.g + head0 + hh) * D + lane * E;
#pragma unroll
    for (int e = 0; e < E; e += 2)
      *reinterpret_cast<uint32_t *>(dst + e) = pack2<kFp16>(acc[e] * inv, acc[e + 1] * inv);
    if (lane == 0)
      p.lse[(int64_t)(h * p.g + head0 + hh) * p.num_seqs + b] =
          any ? (M + log2f(lsum)) * 0.69314718055994531f : -INFINITY;
  }
}

size_t kv4_decode_workspace(int, int, bool) { return 0; }

template <int D, bool kFp16>
static cudaError_t run_decode4(const Kv4DecodeParams &p, cudaStream_t s) {
  const int gm = p.g <= 4 ? 4 : 8;
  auto *kernel = gm == 4 ? kv4_decode_kernel<D, 4, kFp16> : kv4_decode_kernel<D, 8, kFp16>;
  kernel<<<dim3(p.num_seqs, p.h_k, (p.g + gm - 1) / gm), kK4Warps * 32, 0, s>>>(p);
  return cudaGetLastError();
}

cudaError_t launch_kv4_decode(int d, bool fp16, const Kv4DecodeParams &p, cudaStream_t s) {
  if (d == 64) return fp16 ? run_decode4<64, true>(p, s) : run_decode4<64, false>(p, s);
  return fp16 ? run_decode4<128, true>(p, s) : run_decode4<128, false>(p, s);
}

}  // namespace nsa
