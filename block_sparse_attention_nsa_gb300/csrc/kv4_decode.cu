// kv4_decode.cu -- one-step decode of attention over the 4-bit paged KV cache.
//
// Request b's new token attends, per KV head, to the kept keys i of its pages:
//   S_hi = scale * q_h . k_i,  p_hi = exp(S_hi - max S),  out_h = sum p_hi v_i / sum p_hi,
// with k_i and v_i = c * s + z per group of 64 dimensions.  Every stored byte is read once;
// d + d / 8 bytes carry 4 d g operations, so HBM bounds a long cache if the codes become
// operands in few instructions (at 6.8 TB/s each SM gets 41 codes a clock).
//
// Tensor-core form.  Keys are the rows of m16n8k16 (mma.sync: at most 16 query heads are
// far from the 128 rows of a tcgen05 tile), heads the columns.  A code needs no
// conversion: masked out of its word as the low bits of an fp16 it IS the subnormal
// c * 2^-24 (or, at bits 4-7, 16 c * 2^-24), which the tensor core multiplies exactly.
//   scores  acc_g = sum over the group's dimensions of q^ c, exact products in fp32;
//           S = C_h (sum_g ks_g acc_g + kz_g Q_g), Q_g = sum q^ over the group, in fp32.
//           q^ is q times a power of two per head (largest magnitude in [2^14, 2^15)), so
//           that fp16 holds bf16's and fp16's values: it loses only what is 2^-38 of the
//           largest.
//   output  O_g = sum_i P'_i c_i - 8 sum_i P'_i + sum_i p_i (z_i + 8 s_i), P' = p s rounded to
//           fp16 (the one rounding: 2^-11 of a weight, on codes counted from their middle),
//           P' scaled by a power of two that follows the largest s seen.  The second term
//           takes one more product with a row of ones, the third stays in fp32.
// The softmax runs online: the reference maximum of a head is raised (and the sums
// rescaled) only when a score exceeds it by 2 in the exponent, which one vote per tile
// finds, so most tiles need no shuffles.
//
// Data.  A tile is the 32 tokens of one record tile (4608 bytes at d = 128, contiguous).
// Each warp copies its tiles into its own ring of three by cp.async, K rows in place, V
// rows reordered so that the four rows that a lane quartet reads together lie in different
// banks.  K words go to the A operand as they are; V words of two keys are joined by byte
// permutes, which puts neighbouring keys into one register.
//
// Work.  kv4_seg_kernel: a known bound on a segment's (sequence, KV head) tiles; 1 to 8
// warps share a segment, their results meet in shared memory.  kv4_long_kernel: lengths
// only the device knows; every CTA takes an equal run of the batch's tiles whatever the
// sequences' lengths, segments that cross a CTA's border leave partial results (at most
// two a CTA), and kv4_merge_kernel joins those.
#include "kv4.cuh"

namespace nsa {

constexpr int kK4Warps = 8;
constexpr int kK4Stages = 3;
constexpr int kK4MaxCtas = 320;      // CTAs of the long kernel at most
constexpr float kSlack = 2.f;        // scores may exceed the reference maximum by this much
constexpr float kPScale = 8192.f;    // P' <= 2^kSlack * kPScale < 65504

// Words of codes that a lane holds of a K row, and groups of a row.
template <int D>
struct K4 {
  using T = Kv4Tile<D>;
  static constexpr int kG = T::kG;
  static constexpr int kW = D / 32;
  static constexpr int kRing = kK4Stages * T::kBytes;
  static constexpr int kHeadPair = 2 * D + 2;   // floats of two heads' outputs in the merge area
  static constexpr int kSmem = kK4Warps * kRing;
};

// Partial results of a segment: g * (D + 2) floats: O (not divided), then m, l per head.
struct K4Split {
  int32_t seg, parts;   // parts 0: no segment of this CTA continues in the next
};

__device__ __forceinline__ void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t transpose8x8(uint32_t a) {
  uint32_t d;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
  return d;
}
__device__ __forceinline__ uint32_t lds32(uint32_t a) {
  uint32_t x;
  asm volatile("ld.shared.b32 %0, [%1];" : "=r"(x) : "r"(a));
  return x;
}
__device__ __forceinline__ float lds_half(uint32_t a) {
  unsigned short x;
  asm volatile("ld.shared.u16 %0, [%1];" : "=h"(x) : "r"(a));
  return __half2float(__ushort_as_half(x));
}
// The kG halves of row `row` of a parameter array, as floats.
template <int G>
__device__ __forceinline__ void lds_par(uint32_t arr, int row, float (&x)[G]) {
  if constexpr (G == 2) {
    const float2 f = unpack2<true>(lds32(arr + row * 4));
    x[0] = f.x;
    x[1] = f.y;
  } else {
    x[0] = lds_half(arr + row * 2);
  }
}

// The query of a segment as B operands, and its sums and scale per head of the score tile.
template <int D, int NT>
struct K4Query {
  uint32_t f[NT][K4<D>::kW][4];      // [word of the row][dims (0,4), (1,5)/16, (2,6), (3,7)/16]
  float sum[NT][2][K4<D>::kG];       // heads 2c, 2c + 1 of the lane
  float mul[NT][2];
};

template <int D, int NT>
struct K4State {
  float o[NT][K4<D>::kG][4][4];      // dims 64 gi + 8 r + 2 e (+1: 16 times), heads 2c, 2c + 1
  float ps[NT][K4<D>::kG][4];        // sum of P'
  float oz[NT][2][K4<D>::kG];        // this lane's share of sum p (z + 8 s)
  float m[NT][2], l[NT][2];          // l: this lane's share
  float vmax, rinv;                  // largest V scale allowed for, kPScale / it
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int t = 0; t < NT; ++t) {
#pragma unroll
      for (int gi = 0; gi < K4<D>::kG; ++gi)
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          ps[t][gi][x] = 0.f;
#pragma unroll
          for (int e = 0; e < 4; ++e) o[t][gi][e][x] = 0.f;
        }
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        m[t][u] = -INFINITY;
        l[t][u] = 0.f;
#pragma unroll
        for (int gi = 0; gi < K4<D>::kG; ++gi) oz[t][u][gi] = 0.f;
      }
    }
    vmax = 0.f;
    rinv = 0.f;
  }
};

// q: the segment's g rows of D.  Lane (r, c) holds head r (+ 8) and the dimensions of the K
// words that it reads.
template <int D, int NT, bool kFp16>
__device__ __forceinline__ void load_query(const uint16_t *q, int g, float scale_log2, int lane,
                                           K4Query<D, NT> &out) {
  constexpr int G = K4<D>::kG, W = K4<D>::kW;
  const int r = lane >> 2, c = lane & 3;
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    const int head = t * 8 + r;
    float x[W][8], big = 0.f, sum[G];
#pragma unroll
    for (int i = 0; i < W; ++i) {
      const int p = c * W + i, j = p / G, gi = p % G;
      uint4 raw = make_uint4(0u, 0u, 0u, 0u);
      if (head < g)
        raw = __ldg(reinterpret_cast<const uint4 *>(q + (int64_t)head * D + gi * 64 + j * 8));
      const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const float2 f = unpack2<kFp16>(w[u]);
        x[i][2 * u] = f.x;
        x[i][2 * u + 1] = f.y;
        big = fmaxf(big, fmaxf(fabsf(f.x), fabsf(f.y)));
      }
    }
    big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, 1));
    big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, 2));
    const int ex = max(static_cast<int>(__float_as_uint(big) >> 23) - 127, -100);
    const float up = __uint_as_float(static_cast<uint32_t>(14 - ex + 127) << 23);   // 2^(14 - ex)
#pragma unroll
    for (int gi = 0; gi < G; ++gi) sum[gi] = 0.f;
#pragma unroll
    for (int i = 0; i < W; ++i) {
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        x[i][u] *= up;
        sum[i % G] += x[i][u];   // word c W + i belongs to group i % G
      }
      out.f[t][i][0] = pack2<true>(x[i][0], x[i][4]);
      out.f[t][i][1] = pack2<true>(x[i][1] * 0.0625f, x[i][5] * 0.0625f);
      out.f[t][i][2] = pack2<true>(x[i][2], x[i][6]);
      out.f[t][i][3] = pack2<true>(x[i][3] * 0.0625f, x[i][7] * 0.0625f);
    }
    // acc counts in 2^-24: S = 2^(ex - 14 + 24) scale (sum ks acc + kz Q 2^-24)
    const float mul = ldexpf(scale_log2, ex + 10);
#pragma unroll
    for (int gi = 0; gi < G; ++gi) {
      sum[gi] += __shfl_xor_sync(0xffffffffu, sum[gi], 1);
      sum[gi] += __shfl_xor_sync(0xffffffffu, sum[gi], 2);
      sum[gi] *= 5.9604644775390625e-8f;
    }
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const int from = (2 * c + u) * 4;
      out.mul[t][u] = __shfl_sync(0xffffffffu, mul, from);
#pragma unroll
      for (int gi = 0; gi < G; ++gi)
        out.sum[t][u][gi] = __shfl_sync(0xffffffffu, sum[gi], from);
    }
  }
}

// Copies a record tile into a stage of the ring (cp.async, not committed here).
template <int D>
__device__ __forceinline__ void copy_tile(uint32_t stage, const uint8_t *tile, int lane) {
  using T = Kv4Tile<D>;
  const uint8_t *src = tile + lane * 16;
  if constexpr (D == 128) {
    // chunk k * 32 + lane: rows of 4 chunks
    const int kr = lane >> 2, q = lane & 3;
    const int slot = (kr >> 1) + 4 * (kr & 1);          // place of keys 2c, 2c + 1: c, c + 4
    const uint32_t vdst = stage + T::kV + slot * 64 + ((q ^ (slot & 2)) << 4);
#pragma unroll
    for (int k = 0; k < 4; ++k) cp_async16(stage + (k * 32 + lane) * 16, src + k * 512, 16u);
#pragma unroll
    for (int k = 0; k < 4; ++k) cp_async16(vdst + k * 512, src + T::kV + k * 512, 16u);
    cp_async16(stage + T::kPar + lane * 16, src + T::kPar, 16u);
  } else {
    const int kk = lane >> 1;                           // rows of 2 chunks
    const int slot = (kk & 8) + ((kk & 7) >> 1) + 4 * (kk & 1);
    const uint32_t vdst = stage + T::kV + slot * 32 + (lane & 1) * 16;
#pragma unroll
    for (int k = 0; k < 2; ++k) cp_async16(stage + (k * 32 + lane) * 16, src + k * 512, 16u);
#pragma unroll
    for (int k = 0; k < 2; ++k) cp_async16(vdst + k * 512, src + T::kV + k * 512, 16u);
    if (lane < 16) cp_async16(stage + T::kPar + lane * 16, src + T::kPar, 16u);
  }
}

// One tile: keys key0 ... key0 + 31, of which those in [lo, len) count.
template <int D, int NT>
__device__ __forceinline__ void attend_tile(uint32_t st, int key0, int lo, int len, int lane,
                                            const K4Query<D, NT> &q, K4State<D, NT> &a) {
  using T = Kv4Tile<D>;
  constexpr int G = K4<D>::kG, W = K4<D>::kW;
  const int r = lane >> 2, c = lane & 3;
  // ---- scores: rows r and r + 8 of both halves, heads 2c and 2c + 1 ----
  float s[NT][2][4];
#pragma unroll
  for (int half = 0; half < 2; ++half) {
    uint32_t w[2][W];
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const uint32_t at = st + (half * 16 + u * 8 + r) * T::kRow + c * (W * 4);
      if constexpr (W == 4)
        asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                     : "=r"(w[u][0]), "=r"(w[u][1]), "=r"(w[u][2]), "=r"(w[u][3])
                     : "r"(at));
      else
        asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(w[u][0]), "=r"(w[u][1]) : "r"(at));
    }
    float acc[NT][G][4];
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int gi = 0; gi < G; ++gi)
#pragma unroll
        for (int x = 0; x < 4; ++x) acc[t][gi][x] = 0.f;
#pragma unroll
    for (int i = 0; i < W; ++i) {
      const int gi = i % G;
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const uint32_t x = w[0][i] >> (8 * k), y = w[1][i] >> (8 * k);
#pragma unroll
        for (int t = 0; t < NT; ++t)
          mma16816(acc[t][gi], x & 0x000f000fu, y & 0x000f000fu, x & 0x00f000f0u,
                   y & 0x00f000f0u, q.f[t][i][2 * k], q.f[t][i][2 * k + 1]);
      }
    }
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      float ks[G], kz[G];
      const int row = half * 16 + u * 8 + r;
      lds_par<G>(st + T::kPar, row, ks);
      lds_par<G>(st + T::kPar + T::kArr, row, kz);
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int hd = 0; hd < 2; ++hd) {
          float x = 0.f;
#pragma unroll
          for (int gi = 0; gi < G; ++gi) {
            x = fmaf(ks[gi], acc[t][gi][2 * u + hd], x);
            x = fmaf(kz[gi], q.sum[t][hd][gi], x);
          }
          s[t][half][2 * u + hd] = x * q.mul[t][hd];
        }
    }
  }
  // ---- V scales and zeros of the lane's four rows ----
  float vs[4][G], vz[4][G];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    lds_par<G>(st + T::kPar + 2 * T::kArr, i * 8 + r, vs[i]);
    lds_par<G>(st + T::kPar + 3 * T::kArr, i * 8 + r, vz[i]);
  }
  if (key0 < lo || key0 + 32 > len) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int key = key0 + i * 8 + r;
      if (key < lo || key >= len) {   // their scales and zeros may be anything
#pragma unroll
        for (int gi = 0; gi < G; ++gi) vs[i][gi] = vz[i][gi] = 0.f;
#pragma unroll
        for (int t = 0; t < NT; ++t)
          s[t][i >> 1][(i & 1) * 2] = s[t][i >> 1][(i & 1) * 2 + 1] = -INFINITY;
      }
    }
  }
  // ---- raise the references where a score or a scale outgrew them ----
  float top[NT][2], vtop = 0.f;
  bool up = false;
#pragma unroll
  for (int t = 0; t < NT; ++t)
#pragma unroll
    for (int hd = 0; hd < 2; ++hd) {
      top[t][hd] = fmaxf(fmaxf(s[t][0][hd], s[t][0][2 + hd]), fmaxf(s[t][1][hd], s[t][1][2 + hd]));
      up |= top[t][hd] > a.m[t][hd] + kSlack;
    }
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int gi = 0; gi < G; ++gi) vtop = fmaxf(vtop, vs[i][gi]);
  up |= vtop > a.vmax;
  if (__any_sync(0xffffffffu, up)) {
#pragma unroll
    for (int o = 4; o < 32; o <<= 1) vtop = fmaxf(vtop, __shfl_xor_sync(0xffffffffu, vtop, o));
    float grow = 1.f;
    if (vtop > a.vmax) {
      const float vnew = __uint_as_float((__float_as_uint(vtop) & 0x7f800000u) + 0x00800000u);
      const float rnew = __fdiv_rn(kPScale, vnew);     // powers of two: exact
      grow = a.rinv > 0.f ? __fdiv_rn(rnew, a.rinv) : 0.f;
      a.vmax = vnew;
      a.rinv = rnew;
    }
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int hd = 0; hd < 2; ++hd) {
        float x = top[t][hd];
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, o));
        const float mnew = fmaxf(a.m[t][hd], x), alpha = ex2_approx(a.m[t][hd] - mnew);
        a.m[t][hd] = mnew;
        a.l[t][hd] *= alpha;
        const float both = alpha * grow;
#pragma unroll
        for (int gi = 0; gi < G; ++gi) {
          a.oz[t][hd][gi] *= alpha;
          a.ps[t][gi][hd] *= both;
          a.ps[t][gi][2 + hd] *= both;
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            a.o[t][gi][e][hd] *= both;
            a.o[t][gi][e][2 + hd] *= both;
          }
        }
      }
  }
  // ---- weights ----
  uint32_t pb[NT][G][2][2];   // B operands: [group][half][k rows 0-7, 8-15]
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float vsr[G], vc[G];
#pragma unroll
    for (int gi = 0; gi < G; ++gi) {
      vsr[gi] = vs[i][gi] * a.rinv;
      vc[gi] = fmaf(8.f, vs[i][gi], vz[i][gi]);
    }
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      float p[2];
#pragma unroll
      for (int hd = 0; hd < 2; ++hd) {
        p[hd] = ex2_approx(s[t][i >> 1][(i & 1) * 2 + hd] - a.m[t][hd]);
        a.l[t][hd] += p[hd];
#pragma unroll
        for (int gi = 0; gi < G; ++gi) a.oz[t][hd][gi] = fmaf(p[hd], vc[gi], a.oz[t][hd][gi]);
      }
#pragma unroll
      for (int gi = 0; gi < G; ++gi)
        pb[t][gi][i >> 1][i & 1] =
            transpose8x8(pack2<true>(p[0] * vsr[gi], p[1] * vsr[gi]));
    }
  }
  // ---- output: rows are dimensions, k the keys ----
#pragma unroll
  for (int half = 0; half < 2; ++half) {
    uint32_t w[4][G];   // keys 2c, 2c + 1, 2c + 8, 2c + 9
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t row = st + T::kV + (half * 16 + c + 4 * i) * T::kRow;
      if constexpr (G == 2)
        asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];"
                     : "=r"(w[i][0]), "=r"(w[i][1])
                     : "r"(row + ((((r >> 1) ^ (c & 2)) << 4) | ((r & 1) << 3))));
      else
        w[i][0] = lds32(row + r * 4);
    }
#pragma unroll
    for (int gi = 0; gi < G; ++gi) {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        // dims 2e, 2e + 1 of the word: byte e of the four keys' words
        const uint32_t sel = e < 2 ? 0x5410u : 0x7632u;
        const uint32_t x = __byte_perm(w[0][gi], w[1][gi], sel) >> (8 * (e & 1));
        const uint32_t y = __byte_perm(w[2][gi], w[3][gi], sel) >> (8 * (e & 1));
#pragma unroll
        for (int t = 0; t < NT; ++t)
          mma16816(a.o[t][gi][e], x & 0x000f000fu, x & 0x00f000f0u, y & 0x000f000fu,
                   y & 0x00f000f0u, pb[t][gi][half][0], pb[t][gi][half][1]);
      }
#pragma unroll
      for (int t = 0; t < NT; ++t)
        mma16816(a.ps[t][gi], 0x3c003c00u, 0x3c003c00u, 0x3c003c00u, 0x3c003c00u,
                 pb[t][gi][half][0], pb[t][gi][half][1]);
    }
  }
}

// The tiles of a segment and where they lie.
struct K4Seg {
  int b, h, len, lo;
  int first;                 // first tile (32 keys) of the segment, for a segment without selection
  const int32_t *pages;      // kept pages and their first keys (selection), in shared memory
  const int32_t *keys;
};

// Runs tiles t0, t0 + step, ... < t1 of a segment through this warp.
template <int D, int NT>
__device__ __forceinline__ void run_tiles(const Kv4DecodeParams &p, const K4Seg &sg, int t0,
                                          int t1, int step, uint32_t ring, int lane,
                                          const K4Query<D, NT> &q, K4State<D, NT> &a,
                                          int32_t &err) {
  using T = Kv4Tile<D>;
  const int count = t0 < t1 ? (t1 - t0 + step - 1) / step : 0;
  const int tpl = p.page_log2 - 5;
  const int in_page = (1 << p.page_log2) - 1;
  int my_page = -1, my_key = 0;       // of tile 32 * block + lane
  int keys[kK4Stages];                // first keys of the tiles in the ring, -1: nothing to do
  auto issue = [&](int n, int &key) {
    key = -1;
    if (n < count) {
      if ((n & 31) == 0) {            // look up the next 32 tiles' pages
        const int i = n + lane, t = t0 + i * step;
        my_page = -1;
        if (i < count) {
          if (sg.pages) {
            my_page = sg.pages[t >> tpl];
            my_key = sg.keys[t >> tpl] + ((t & ((1 << tpl) - 1)) << 5);
          } else {
            my_key = (sg.first + t) << 5;
            if (my_key < sg.len) {
              my_page = __ldg(p.table + (int64_t)sg.b * p.width + (my_key >> p.page_log2));
              if (my_page < 0 || my_page >= p.num_pages) {
                my_page = -1;
                err |= NSA_DEVERR_BAD_INDEX;
              }
            }
          }
          if (my_key >= sg.len || my_key + 32 <= sg.lo) my_page = -1;
        }
      }
      const int pg = __shfl_sync(0xffffffffu, my_page, n & 31);
      const int k0 = __shfl_sync(0xffffffffu, my_key, n & 31);
      if (pg >= 0) {
        key = k0;
        copy_tile<D>(ring + (n % kK4Stages) * T::kBytes,
                     p.pool + ((((int64_t)pg * p.h_k + sg.h) << tpl) + ((k0 & in_page) >> 5)) *
                                  (int64_t)T::kBytes,
                     lane);
      }
    }
    cp_async_commit();
  };
#pragma unroll
  for (int n = 0; n < kK4Stages - 1; ++n) issue(n, keys[n]);
  for (int n = 0; n < count; ++n) {
    issue(n + kK4Stages - 1, keys[kK4Stages - 1]);
    cp_async_wait_group<kK4Stages - 1>();
    __syncwarp();
    if (keys[0] >= 0)
      attend_tile<D, NT>(ring + (n % kK4Stages) * T::kBytes, keys[0], sg.lo, sg.len, lane, q, a);
    __syncwarp();                     // the stage is filled again in the next turn
#pragma unroll
    for (int i = 0; i + 1 < kK4Stages; ++i) keys[i] = keys[i + 1];
  }
  cp_async_wait_all();
}

// The warp's sums into its merge area (its own ring): O [head pairs], m and l per head.
template <int D, int NT>
__device__ __forceinline__ void leave_warp(float *area, float2 *ml, int lane,
                                           const K4State<D, NT> &a) {
  constexpr int G = K4<D>::kG;
  const int r = lane >> 2, c = lane & 3;
  const float back = a.rinv > 0.f ? __fdiv_rn(1.f, a.rinv) : 0.f;
  const float o24 = back * 16777216.f;
#pragma unroll
  for (int t = 0; t < NT; ++t) {
#pragma unroll
    for (int hd = 0; hd < 2; ++hd) {
      float l = a.l[t][hd], add[G];
#pragma unroll
      for (int gi = 0; gi < G; ++gi) add[gi] = a.oz[t][hd][gi];
#pragma unroll
      for (int o = 4; o < 32; o <<= 1) {
        l += __shfl_xor_sync(0xffffffffu, l, o);
#pragma unroll
        for (int gi = 0; gi < G; ++gi) add[gi] += __shfl_xor_sync(0xffffffffu, add[gi], o);
      }
      float *dst = area + (t * 4 + c) * K4<D>::kHeadPair + hd * D + 8 * r;
#pragma unroll
      for (int gi = 0; gi < G; ++gi) {
        const float base = fmaf(-8.f * back, a.ps[t][gi][hd], add[gi]);
#pragma unroll
        for (int e = 0; e < 4; ++e)
          *reinterpret_cast<float2 *>(dst + gi * 64 + 2 * e) =
              make_float2(fmaf(a.o[t][gi][e][hd], o24, base),
                          fmaf(a.o[t][gi][e][2 + hd], o24 * 0.0625f, base));
      }
      if (r == 0) ml[t * 8 + 2 * c + hd] = make_float2(a.m[t][hd], l);
    }
  }
}

// Joins the areas of `warps` warps; thread `th` of `nth`.  Writes out and lse of a whole
// segment, or a partial result to `part`.
template <int D, bool kFp16>
__device__ __forceinline__ void join_warps(const Kv4DecodeParams &p, int b, int h,
                                           const float *areas, size_t area_step, const float2 *ml,
                                           int ml_step, int warps, int th, int nth, float *part) {
  for (int i = th; i < p.g * (D / 2); i += nth) {
    const int head = i / (D / 2), dim = 2 * (i % (D / 2));
    const float *src = areas + (head >> 1) * K4<D>::kHeadPair + (head & 1) * D + dim;
    float M = -INFINITY, l = 0.f, x = 0.f, y = 0.f;
    for (int w = 0; w < warps; ++w)
      if (ml[w * ml_step + head].y != 0.f) M = fmaxf(M, ml[w * ml_step + head].x);
    for (int w = 0; w < warps; ++w) {
      const float2 v = ml[w * ml_step + head];
      if (v.y == 0.f) continue;                     // a warp without keys
      const float wt = ex2_approx(v.x - M);
      const float2 o = *reinterpret_cast<const float2 *>(src + w * area_step);
      l = fmaf(wt, v.y, l);
      x = fmaf(wt, o.x, x);
      y = fmaf(wt, o.y, y);
    }
    if (part) {
      *reinterpret_cast<float2 *>(part + head * D + dim) = make_float2(x, y);
      if (dim == 0) *reinterpret_cast<float2 *>(part + p.g * D + 2 * head) = make_float2(M, l);
    } else {
      const bool any = l != 0.f;                    // a NaN sum stays one
      const float inv = any ? 1.f / l : 0.f;
      const int64_t row = (int64_t)b * p.h_q + h * p.g + head;
      reinterpret_cast<uint32_t *>(p.out)[(row * D + dim) / 2] = pack2<kFp16>(x * inv, y * inv);
      if (dim == 0)
        p.lse[(int64_t)(h * p.g + head) * p.num_seqs + b] =
            any ? (M + log2f(l)) * 0.69314718055994531f : -INFINITY;
    }
  }
}

// Length of sequence b held to its table row, and the first key that its window shows.
__device__ __forceinline__ int seq_len(const Kv4DecodeParams &p, int b, int32_t &err) {
  const int64_t cap = (int64_t)p.width << p.page_log2;
  const int raw = __ldg(p.lens + b);
  const int len = static_cast<int>(raw < 0 ? 0 : (raw > cap ? cap : raw));
  if (raw != len) err |= NSA_DEVERR_BAD_SEQLENS;
  return len;
}
__device__ __forceinline__ int seq_lo(const Kv4DecodeParams &p, int len) {
  return p.window > 0 && len > p.window ? len - p.window : 0;
}

// One segment per kWps warps.
template <int D, int NT, bool kFp16, bool kSel>
__global__ void __launch_bounds__(kK4Warps * 32, NT == 1 ? 2 : 1)
    kv4_seg_kernel(Kv4DecodeParams p, int wps) {
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ float2 ml[kK4Warps][8 * NT];
  __shared__ int32_t kept_page[kK4Warps][32], kept_key[kK4Warps][32];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int sub = warp / wps, w = warp - sub * wps;      // segment of the CTA, warp of the segment
  const int64_t seg = (int64_t)blockIdx.x * (kK4Warps / wps) + sub;
  const bool live = seg < (int64_t)p.num_seqs * p.h_k;
  K4State<D, NT> a;
  a.clear();
  K4Seg sg = {};
  int32_t err = 0;
  if (live) {
    sg.b = static_cast<int>(seg / p.h_k);
    sg.h = static_cast<int>(seg - (int64_t)sg.b * p.h_k);
    int blk = -1;
    if (kSel && lane < p.topk)
      blk = __ldg(p.sel + ((int64_t)sg.h * p.num_seqs + sg.b) * p.topk + lane);
    sg.len = seq_len(p, sg.b, err);
    sg.lo = seq_lo(p, sg.len);
    int tiles;
    if (kSel) {
      // the kept blocks: valid, first of their value, with a page in the pool
      const int nblk = (sg.len + (1 << p.page_log2) - 1) >> p.page_log2;
      if (blk < -1 || blk >= nblk) err |= lane < p.topk ? NSA_DEVERR_BAD_INDEX : 0;
      bool ok = blk >= 0 && blk < nblk;
      const uint32_t same = __match_any_sync(0xffffffffu, blk);
      ok = ok && (same & ((1u << lane) - 1u)) == 0;
      int pg = -1;
      if (ok) {
        pg = __ldg(p.table + (int64_t)sg.b * p.width + blk);
        if (pg < 0 || pg >= p.num_pages) {
          ok = false;
          err |= NSA_DEVERR_BAD_INDEX;
        }
      }
      const uint32_t m = __ballot_sync(0xffffffffu, ok);
      if (ok) {
        const int at = __popc(m & ((1u << lane) - 1u));
        kept_page[warp][at] = pg;
        kept_key[warp][at] = blk << p.page_log2;
      }
      __syncwarp();
      sg.pages = kept_page[warp];
      sg.keys = kept_key[warp];
      tiles = __popc(m) << (p.page_log2 - 5);
    } else {
      sg.first = sg.lo >> 5;
      tiles = ((sg.len + 31) >> 5) - sg.first;
    }
    K4Query<D, NT> q;
    load_query<D, NT, kFp16>(static_cast<const uint16_t *>(p.q) +
                                 ((int64_t)sg.b * p.h_q + sg.h * p.g) * D,
                             p.g, p.scale_log2, lane, q);
    run_tiles<D, NT>(p, sg, w, tiles, wps, smem_u32(smem) + warp * K4<D>::kRing, lane, q, a, err);
    err = __reduce_or_sync(0xffffffffu, err);
    if (err && lane == 0) raise(p.status, err);
    leave_warp<D, NT>(reinterpret_cast<float *>(smem + warp * K4<D>::kRing), ml[warp], lane, a);
  }
  __syncthreads();
  if (live)
    join_warps<D, kFp16>(p, sg.b, sg.h,
                         reinterpret_cast<const float *>(smem + sub * wps * K4<D>::kRing),
                         K4<D>::kRing / 4, ml[sub * wps], 8 * NT, wps, w * 32 + lane, wps * 32,
                         nullptr);
}

// Tiles of a sequence: at least one, so that an empty one's output is written too.
__device__ __forceinline__ int seq_tiles(const Kv4DecodeParams &p, int len) {
  return max(1, ((len + 31) >> 5) - (seq_lo(p, len) >> 5));
}

__device__ __forceinline__ K4Split *splits_of(const Kv4DecodeParams &p) {
  return static_cast<K4Split *>(p.ws);
}
template <int D>
__device__ __forceinline__ float *part_of(const Kv4DecodeParams &p, int64_t i) {
  return reinterpret_cast<float *>(static_cast<uint8_t *>(p.ws) + kK4MaxCtas * sizeof(K4Split)) +
         i * (p.g * (D + 2));
}

// Equal runs of the batch's tiles (sequence, head, tile order) for every CTA.
template <int D, int NT, bool kFp16>
__global__ void __launch_bounds__(kK4Warps * 32, NT == 1 ? 2 : 1)
    kv4_long_kernel(Kv4DecodeParams p) {
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ float2 ml[kK4Warps][8 * NT];
  __shared__ int64_t wsum[kK4Warps];
  __shared__ int64_t found_base;
  __shared__ int found_b;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  // the batch's tiles, and the sequence that holds this CTA's first one
  const int per_thread = (p.num_seqs + kK4Warps * 32 - 1) / (kK4Warps * 32);
  const int b0 = min(tid * per_thread, p.num_seqs), b1 = min(b0 + per_thread, p.num_seqs);
  int32_t err = 0;
  int64_t mine = 0;
  for (int b = b0; b < b1; ++b) mine += seq_tiles(p, seq_len(p, b, err));
  int64_t incl = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t y = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += y;
  }
  if (lane == 31) wsum[warp] = incl;
  if (tid == 0) found_b = -1;
  __syncthreads();
  int64_t total = 0;
#pragma unroll
  for (int w = 0; w < kK4Warps; ++w) {
    if (w < warp) incl += wsum[w];
    total += wsum[w];
  }
  total *= p.h_k;
  // a multiple of the warps, so that no warp idles in a run
  const int64_t per = (total + (int64_t)gridDim.x * kK4Warps - 1) /
                      ((int64_t)gridDim.x * kK4Warps) * kK4Warps;
  const int64_t begin = blockIdx.x * per, end = min(begin + per, total);
  if (blockIdx.x == 0 && err) raise(p.status, err);
  err = 0;
  if (begin < end && mine > 0 && (incl - mine) * p.h_k <= begin && begin < incl * p.h_k) {
    int64_t base = (incl - mine) * p.h_k;
    for (int b = b0; b < b1; ++b) {
      const int64_t nt = (int64_t)seq_tiles(p, seq_len(p, b, err)) * p.h_k;
      if (begin < base + nt) {
        found_b = b;
        found_base = base;
        break;
      }
      base += nt;
    }
  }
  __syncthreads();
  err = 0;
  K4Split split = {0, 0};
  int b = found_b;
  int64_t base = found_base;               // first tile of (b, head 0)
  for (int64_t at = begin; at < end;) {
    int32_t ignore = 0;
    K4Seg sg = {};
    sg.b = b;
    sg.len = seq_len(p, b, ignore);
    sg.lo = seq_lo(p, sg.len);
    sg.first = sg.lo >> 5;
    const int nt = seq_tiles(p, sg.len);
    sg.h = static_cast<int>((at - base) / nt);
    const int64_t seg0 = base + (int64_t)sg.h * nt;
    const int t0 = static_cast<int>(at - seg0);
    const int t1 = static_cast<int>(min((int64_t)nt, end - seg0));
    K4State<D, NT> a;
    a.clear();
    {
      K4Query<D, NT> q;
      load_query<D, NT, kFp16>(static_cast<const uint16_t *>(p.q) +
                                   ((int64_t)sg.b * p.h_q + sg.h * p.g) * D,
                               p.g, p.scale_log2, lane, q);
      run_tiles<D, NT>(p, sg, t0 + warp, t1, kK4Warps, smem_u32(smem) + warp * K4<D>::kRing, lane,
                       q, a, err);
    }
    leave_warp<D, NT>(reinterpret_cast<float *>(smem + warp * K4<D>::kRing), ml[warp], lane, a);
    __syncthreads();
    float *part = nullptr;
    if (t0 > 0) {
      part = part_of<D>(p, 2 * (int64_t)blockIdx.x);
    } else if (t1 < nt) {
      part = part_of<D>(p, 2 * (int64_t)blockIdx.x + 1);
      split.seg = static_cast<int32_t>((int64_t)sg.b * p.h_k + sg.h);
      split.parts = static_cast<int32_t>((seg0 + nt - 1) / per - blockIdx.x + 1);
    }
    join_warps<D, kFp16>(p, sg.b, sg.h, reinterpret_cast<const float *>(smem), K4<D>::kRing / 4,
                         ml[0], 8 * NT, kK4Warps, tid, kK4Warps * 32, part);
    at = seg0 + t1;
    if (t1 == nt && sg.h == p.h_k - 1) {
      base += (int64_t)nt * p.h_k;
      ++b;
    }
    __syncthreads();                       // the areas have been read: the rings may be filled
  }
  if (tid == 0) splits_of(p)[blockIdx.x] = split;
  err = __reduce_or_sync(0xffffffffu, err);
  if (err && lane == 0) raise(p.status, err);
}

// Joins the parts of the segment that begins in CTA blockIdx.x and ends in another: its own
// second part and the following CTAs' first ones.  One CTA per (split, head).
constexpr int kMergeThreads = 256;
template <int D, bool kFp16>
__global__ void __launch_bounds__(kMergeThreads) kv4_merge_kernel(Kv4DecodeParams p) {
  __shared__ float wt[kK4MaxCtas];
  __shared__ float red[kMergeThreads / 32][2];
  __shared__ float acc[kMergeThreads];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, head = blockIdx.y;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const K4Split sp = splits_of(p)[blockIdx.x];
  if (sp.parts == 0) return;
  auto part = [&](int i) {
    return part_of<D>(p, i == 0 ? 2 * (int64_t)blockIdx.x + 1 : 2 * ((int64_t)blockIdx.x + i));
  };
  float M = -INFINITY;
  for (int i = tid; i < sp.parts; i += kMergeThreads) {
    const float2 v = *reinterpret_cast<const float2 *>(part(i) + p.g * D + 2 * head);
    if (v.y != 0.f) M = fmaxf(M, v.x);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
  if (lane == 0) red[warp][0] = M;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kMergeThreads / 32; ++w) M = fmaxf(M, red[w][0]);
  float l = 0.f;
  for (int i = tid; i < sp.parts; i += kMergeThreads) {
    const float2 v = *reinterpret_cast<const float2 *>(part(i) + p.g * D + 2 * head);
    wt[i] = v.y != 0.f ? ex2_approx(v.x - M) : 0.f;
    l = fmaf(wt[i], v.y, l);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
  if (lane == 0) red[warp][1] = l;
  __syncthreads();
  l = 0.f;
#pragma unroll
  for (int w = 0; w < kMergeThreads / 32; ++w) l += red[w][1];
  constexpr int kRows = kMergeThreads / D;
  const int dim = tid % D;
  float x = 0.f;
#pragma unroll 4
  for (int i = tid / D; i < sp.parts; i += kRows) {
    const float w = wt[i];
    if (w != 0.f) x = fmaf(w, part(i)[head * D + dim], x);
  }
  acc[tid] = x;
  __syncthreads();
  if (tid < D / 2) {
    float u = 0.f, v = 0.f;
#pragma unroll
    for (int k = 0; k < kRows; ++k) {
      u += acc[k * D + 2 * tid];
      v += acc[k * D + 2 * tid + 1];
    }
    const bool any = l != 0.f;
    const float inv = any ? 1.f / l : 0.f;
    const int b = sp.seg / p.h_k, hq = (sp.seg - b * p.h_k) * p.g + head;
    reinterpret_cast<uint32_t *>(p.out)[((int64_t)b * p.h_q + hq) * (D / 2) + tid] =
        pack2<kFp16>(u * inv, v * inv);
    if (tid == 0)
      p.lse[(int64_t)hq * p.num_seqs + b] =
          any ? (M + log2f(l)) * 0.69314718055994531f : -INFINITY;
  }
}

size_t kv4_decode_workspace(int d, int g, bool selected) {
  if (selected) return 0;
  return kK4MaxCtas * sizeof(K4Split) + 2 * (size_t)kK4MaxCtas * g * (d + 2) * sizeof(float);
}

static int sm_count() {
  static int cache[64];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 148;
  if (cache[dev] == 0) {
    int n = 0;
    cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev);
    cache[dev] = n > 0 ? n : 148;
  }
  return cache[dev];
}

template <typename K>
static cudaError_t allow_smem(K kernel, int bytes) {
  return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
}

template <int D, int NT, bool kFp16>
static cudaError_t run_decode4(const Kv4DecodeParams &p, cudaStream_t s) {
  constexpr int smem = K4<D>::kSmem;
  const int slots = sm_count() * (NT == 1 ? 2 : 1);       // CTAs resident at once
  const int64_t segs = (int64_t)p.num_seqs * p.h_k;
  // tiles that a segment has at most, as far as the host knows
  int64_t most = ((int64_t)p.width << p.page_log2) / kKv4Tile;
  if (p.window > 0) most = min(most, (int64_t)p.window / kKv4Tile + 2);
  if (p.sel) most = min(most, (int64_t)p.topk << (p.page_log2 - 5));
  if (p.sel || most <= 64) {
    // warps to a segment: as many as still fit the GPU at once, and no more than tiles
    int wps = 1;
    while (wps < kK4Warps && segs * (2 * wps) <= (int64_t)slots * kK4Warps && wps < most) wps *= 2;
    auto *kernel = p.sel ? kv4_seg_kernel<D, NT, kFp16, true> : kv4_seg_kernel<D, NT, kFp16, false>;
    cudaError_t e = allow_smem(kernel, smem);
    if (e != cudaSuccess) return e;
    const int per = kK4Warps / wps;
    kernel<<<static_cast<unsigned>((segs + per - 1) / per), kK4Warps * 32, smem, s>>>(p, wps);
    return cudaGetLastError();
  }
  auto *kernel = kv4_long_kernel<D, NT, kFp16>;
  cudaError_t e = allow_smem(kernel, smem);
  if (e != cudaSuccess) return e;
  const int ctas = min(slots, kK4MaxCtas);
  kernel<<<ctas, kK4Warps * 32, smem, s>>>(p);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(ctas, p.g);
  cfg.blockDim = dim3(kMergeThreads);
  cfg.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kv4_merge_kernel<D, kFp16>, p);
}

template <int D, bool kFp16>
static cudaError_t run_decode4_nt(const Kv4DecodeParams &p, cudaStream_t s) {
  return p.g <= 8 ? run_decode4<D, 1, kFp16>(p, s) : run_decode4<D, 2, kFp16>(p, s);
}

cudaError_t launch_kv4_decode(int d, bool fp16, const Kv4DecodeParams &p, cudaStream_t s) {
  if (d == 64) return fp16 ? run_decode4_nt<64, true>(p, s) : run_decode4_nt<64, false>(p, s);
  return fp16 ? run_decode4_nt<128, true>(p, s) : run_decode4_nt<128, false>(p, s);
}

}  // namespace nsa
