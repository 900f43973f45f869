// kv4_decode.cu -- one-step decode of attention over the 4-bit paged KV cache.
//
// Request b's new token attends, per KV head, to the kept keys i of its pages:
//   S_hi = scale * q_h . k_i,  p_hi = exp(S_hi - max S),  out_h = sum p_hi v_i / sum p_hi,
// with k_i and v_i = c * s + z per group of 64 dimensions.  Every stored byte is read once;
// d + d / 8 bytes carry 4 d g operations, so HBM bounds a long cache if the codes become
// operands in few instructions (at 6.8 TB/s each SM gets 41 codes a clock).
//
// Tensor-core form.  Keys are the rows of m16n8k16, heads the columns.  (mma.sync takes its
// operands from registers, where the codes are unpacked; a tcgen05 tile of 128 keys would want them
// written to shared or tensor memory as 16-bit numbers first, four times their bytes, for a
// tensor pipe that is at most 30 % busy as it is.)  A code needs no conversion: masked out of its
// word as the low bits of an fp16 it IS the subnormal c * 2^-24 (or, at bits 4-7, 16 c * 2^-24;
// both two bits further up, see kUp), which the tensor core multiplies exactly.
//   scores  acc_g = sum over the group's dimensions of q^ c, exact products in fp32;
//           S = C_h (sum_g ks_g acc_g + kz_g Q_g), Q_g = sum q^ over the group, in fp32.
//           q^ is q times a power of two per head (largest magnitude in [2^14, 2^15)), so
//           that fp16 holds bf16's and fp16's values: it loses only what is 2^-38 of the
//           largest (2^-34 in the half of the dimensions that is held in sixteenths).
//   output  O_g = sum_i P'_i (c_i - m) + sum_i p_i (z_i + m s_i), P' = p s scaled by a power of
//           two that follows the largest s seen; the second sum is in fp32.  For bf16 P' is
//           rounded to fp16 (2^-11 of a weight, on codes counted from their middle m = 7.5, by
//           one more product with a row of ones): below the output's own rounding, to which
//           it adds 0.4 % (64 x 8K selected: 1.4e-4 of the output beside 1.66e-3); a second part
//           took 9 % more time there (12.0 -> 13.1 us).  For fp16, whose rounding is as small, P'
//           is the sum of two fp16 numbers (2^-22), and m is 0 over a few tiles.
//           The tensor core cuts its sums towards zero, by up to 2^-24 of the largest exponent in
//           each product: an error of one sign that grows with a run, while the values that it
//           is measured by cancel.  Where it would show (K4Stream::run has the rule) a tile's
//           sums start at -m sum P', so that they end near what is left of them, and are added
//           to the warp's in fp32, rounded to nearest.  Over 288 / 1026 / 4098 tiles a warp the
//           outputs are then 1.54 / 1.64 / 1.46e-3 (bf16; 2.1 / 15 / 5.1e-3 without) and 1.92 /
//           2.13 / 2.12e-4 (fp16; 8 sum P' taken off after each tile: 2.1 / 8.3 / 17e-4) from
//           exact, their own rounding being 1.4 to 1.6e-3 and 1.8 to 2.1e-4, for 2 to 7 % of
//           bf16's time.
// The softmax runs online: the reference maximum of a head is raised (and the sums
// rescaled) only when a score exceeds it by 2 in the exponent, which one vote per tile
// finds, so most tiles need no shuffles.
//
// Data.  A tile is the 32 tokens of one record tile (4608 bytes at d = 128, contiguous).
// Each warp copies its tiles into its own ring of three by cp.async, K rows in place, V
// rows reordered so that the four rows that a lane quartet reads together lie in different
// banks.  K words go to the A operand as they are; V words of two keys are joined by byte
// permutes, which puts neighbouring keys into one register.  Each lane turns one key's V
// scales and zeros into fp32 for all, in the place of the K codes.
//
// Work.  A segment is a (sequence, KV head, up to 8 of its query heads).  kv4_seg_kernel:
// one CTA of 1 to 8 warps a segment, or a cluster of up to 8 CTAs where few segments would
// leave SMs idle, the warps taking its tiles in turn; for segments whose tiles have a bound
// that the host knows (a selection, a window, a short table).
// kv4_run_kernel: every warp takes an equal run of the batch's tiles in segment order,
// whatever the lengths, which only the device knows; a segment counts kOver tiles more than
// it has, about what starting one costs.  Segments inside a warp's run are written by that
// warp; those that cross into the next warp's are joined in the CTA, and those that cross a
// CTA's border leave partial results (at most two a CTA) for kv4_merge_kernel.
//
// Measured (d = 128, bf16): a tile costs about 530 warp instructions, its start and join
// included (567 with its sums added in fp32), and, with 12 warps on an SM, 230 to 240 cycles,
// against 198 that its bytes take at 6.78 TB/s.  64 sequences of 8K, 16 selected blocks, g = 4 (37.8
// MB): 11.9 us (three such batches in turn; behind an L2 flush 16 to 18); one of 64K in full: 17.4 us;
// eight of them (302 MB): 60.1 us, 5.03 TB/s.
#include "kv4.cuh"

namespace nsa {

// Warps that an SM holds.  At d = 128 twelve: a warp then has 168 registers instead of 128, and
// the compiler's order of a tile's loads and products gains more than the four warps lose (64 x 8K,
// 16 blocks: 12.9 -> 11.7 us; 8 x 64K in full: 59.8 -> 57.0).  At d = 64 126 registers do.
template <int D>
constexpr int kSmWarps = D == 128 ? 12 : 16;
constexpr int kK4Heads = 8;          // query heads of a segment at most
constexpr int kStages = 3;           // tiles of a warp's ring
constexpr int kOver = 4;             // tiles that a segment's start counts as
constexpr int kK4MaxCtas = 320;      // CTAs of the run kernel at most
constexpr float kSlack = 2.f;        // scores may exceed the reference maximum by this much
constexpr float kMiddle = 7.5f;      // of the codes
// Where sums need no centre.  What they lose grows with a warp's tiles and, next to what is left of
// the values, with the square root of the segment's keys: 2.6e-8 of a bf16 output times tiles *
// sqrt(keys), so that the bound below stands for 2e-4, an eighth of its rounding.
constexpr int kFewTiles = 12, kFewKeys = 2048, kFewSquare = 1 << 21;
constexpr float kPScale = 8192.f;    // P' <= 2^kSlack * kPScale < 65504
constexpr int kUp = 2;               // bits that codes are moved up by (code_pairs)
constexpr int kMulTop = 118;         // a score's factor stays below 2^(kMulTop + 2)

template <int D>
struct K4 {
  using T = Kv4Tile<D>;
  static constexpr int kG = T::kG;
  static constexpr int kW = D / 32;             // words of codes that a lane holds of a K row
  static constexpr int kHeadPair = 2 * D + 4;   // floats of two heads' outputs in an area
  static constexpr int kRing = kStages * T::kBytes;
  // A warp's results go to the ring's start; a first part that has to stay while the warp
  // goes on takes the last stage.
  static constexpr int kKept = (kStages - 1) * T::kBytes;
  static constexpr int kRunWarps = kSmWarps<D> / 2, kRunThreads = kRunWarps * 32;   // two CTAs an SM
  static_assert(kK4Heads / 2 * kHeadPair * 4 <= T::kBytes, "a stage holds an area");
};

// Where the parts of a segment that begins in CTA i and ends in another lie.
struct K4Split {
  int32_t seg, parts;   // parts 0: no segment of this CTA continues in the next
};

__device__ __forceinline__ void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
  asm(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// The same on accumulators of other registers, and on zeros.
__device__ __forceinline__ void mma16816_c(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                           uint32_t a3, uint32_t b0, uint32_t b1, Pair c01,
                                           Pair c23) {
  const float2 x = c01.get(), y = c23.get();
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%10, %11, %12, %13};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(x.x), "f"(x.y), "f"(y.x),
        "f"(y.y));
}
__device__ __forceinline__ void mma16816_0(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                           uint32_t a3, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%10, %10, %10, %10};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}
__device__ __forceinline__ uint32_t transpose8x8(uint32_t a) {
  uint32_t d;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
  return d;
}
// The kG halves of entry `i` of a parameter array, packed; and as floats.
template <int G>
__device__ __forceinline__ uint32_t lds_par(const uint8_t *arr, int i) {
  if constexpr (G == 2) return reinterpret_cast<const uint32_t *>(arr)[i];
  else return reinterpret_cast<const uint16_t *>(arr)[i];
}
template <int G>
__device__ __forceinline__ void par_floats(uint32_t u, float (&x)[G]) {
  const float2 f = unpack2<true>(u);
  x[0] = f.x;
  if constexpr (G == 2) x[1] = f.y;
}

// Codes 0, 1, 4, 5 (k = 0) or 2, 3, 6, 7 of a word of K (of V: the low or the high byte of both
// halves), in the places that the masks take.  The tensor core truncates its sums relative to the
// largest exponent, and a subnormal's leading zeros count against it: codes two bits further up
// than they lie, for one more shift a word, took a lone key's score from 1.5e-6 (fp16) and 5.6e-7
// (bf16) off to 2.4e-7 and 1.5e-7.  V's sums are all truncated the same way, so that it adds up
// where a long cache's values cancel: with weights as exact as here fp16 outputs over 64K tokens
// were 4.4e-4 off, with the two bits 1.1e-4; codes at the top of the subnormals cost 4 % of the
// time and gave little more.
__device__ __forceinline__ uint32_t code_pairs(uint32_t w, int k) {
  return k ? w >> (8 - kUp) : w << kUp;
}

// The query of a segment as B operands, and its sums and scale per head of the score tile.
template <int D>
struct K4Query {
  uint32_t f[K4<D>::kW][4];      // [word of the row][dims (0,4), (1,5)/16, (2,6), (3,7)/16]
  float sum[2][K4<D>::kG];       // sums of q^ in the raw scores' unit, heads 2c, 2c + 1 of the lane
  Pair mul;                      // raw score -> S, >= 0
};
template <int D>
struct K4RawQuery {
  uint4 w[K4<D>::kW];
};

template <int D>
struct K4State {
  float o[K4<D>::kG][4][4];      // dims 64 gi + 8 r + 2 e (+1: 16 times), heads 2c, 2c + 1
  float ps[K4<D>::kG][4];        // sum of P' (bf16)
  Pair oz[K4<D>::kG];            // this lane's share of sum p (z + m s), of both heads
  Pair minus_m, l;               // reference maximum, negated; l: this lane's share
  float thr[2];                  // score above which m is raised
  float vmax, rinv;              // largest V scale allowed for, kPScale / it
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int gi = 0; gi < K4<D>::kG; ++gi)
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        ps[gi][x] = 0.f;
#pragma unroll
        for (int e = 0; e < 4; ++e) o[gi][e][x] = 0.f;
      }
    minus_m = Pair(INFINITY, INFINITY);
    thr[0] = thr[1] = -INFINITY;
    l = Pair(0.f, 0.f);
#pragma unroll
    for (int gi = 0; gi < K4<D>::kG; ++gi) oz[gi] = Pair(0.f, 0.f);
    vmax = 0.f;
    rinv = 0.f;
  }
};

// A segment: its sequence, KV head and query heads, its keys [lo, len), its tiles.
struct K4Seg {
  int b, h, q0, g;           // q0: first query head, g: how many
  int len, lo;
  int first;                 // first tile (32 keys), without a selection
  int tiles;                 // tiles that exist
  int page, key;             // selection: lane i holds the i-th kept block's page and first key
};

// Unit u of a sequence: KV head u / parts, its query heads 8 * (u % parts) ...
__device__ __forceinline__ void set_unit(const Kv4DecodeParams &p, int u, K4Seg &sg) {
  const int parts = p.g > kK4Heads ? 2 : 1, part = parts == 2 ? u & 1 : 0;
  sg.h = parts == 2 ? u >> 1 : u;
  sg.q0 = sg.h * p.g + part * kK4Heads;
  sg.g = min(kK4Heads, p.g - part * kK4Heads);
}

// Lane (r, c) holds head r and the dimensions of the K words that it reads.
template <int D>
__device__ __forceinline__ void fetch_query(const Kv4DecodeParams &p, const K4Seg &sg, int lane,
                                            K4RawQuery<D> &raw) {
  constexpr int G = K4<D>::kG, W = K4<D>::kW;
  const int r = lane >> 2, c = lane & 3;
  const uint16_t *q =
      static_cast<const uint16_t *>(p.q) + ((int64_t)sg.b * p.h_q + sg.q0 + r) * D;
#pragma unroll
  for (int i = 0; i < W; ++i) {
    const int w = c * W + i, at = (w % G) * 64 + w / G * 8;
    raw.w[i] = make_uint4(0u, 0u, 0u, 0u);
    if (r < sg.g) raw.w[i] = *reinterpret_cast<const uint4 *>(q + at);
  }
}

// The exponent of the largest magnitude of lane (r, c)'s head r.
template <int D, bool kFp16>
__device__ __forceinline__ int query_exponent(const K4RawQuery<D> &raw) {
  uint32_t top = 0;          // magnitudes of 16-bit floats order as whole numbers
#pragma unroll
  for (int i = 0; i < K4<D>::kW; ++i) {
    const uint4 w = raw.w[i];
    top = __vmaxu2(__vmaxu2(top, w.x & 0x7fff7fffu), w.y & 0x7fff7fffu);
    top = __vmaxu2(__vmaxu2(top, w.z & 0x7fff7fffu), w.w & 0x7fff7fffu);
  }
  top = __vmaxu2(top, __shfl_xor_sync(0xffffffffu, top, 1));
  top = __vmaxu2(top, __shfl_xor_sync(0xffffffffu, top, 2));
  const float2 f = unpack2<kFp16>(top);
  return max(static_cast<int>(__float_as_uint(fmaxf(f.x, f.y)) >> 23) - 127, -100);
}

// A raw score counts in 2^-22, of a query scaled by 2^(14 - ex): S = 2^(ex + 8) |scale| raw.  A
// factor past 2^(kMulTop + 2) could overflow where S does not: `over` powers of two are left
// out of it, and of the scores, and put back into the maximum at the end.  The keys' weights do not
// miss them: what a query in fp16 keeps of such a head makes scores that are equal or differ by
// far more than 2^over times what an exponential tells apart.
__device__ __forceinline__ int score_over(float scale, int ex) {
  return max(0, static_cast<int>((__float_as_uint(scale) & 0x7fffffffu) >> 23) - 127 + ex + 10 -
                    kUp - kMulTop);
}

// Scaled by a power of two per head to a largest magnitude in [2^14, 2^15).  The sums of
// q^ come from products with rows of ones (16 for the dimensions held as sixteenths).
template <int D, bool kFp16>
__device__ __forceinline__ void make_query(const K4RawQuery<D> &raw, float scale, int lane,
                                           K4Query<D> &out) {
  constexpr int G = K4<D>::kG, W = K4<D>::kW;
  const int c = lane & 3;
  const uint32_t sign = scale < 0.f ? 0x80008000u : 0u;   // mul stays positive
  const int ex = query_exponent<D, kFp16>(raw);
  const float up = __uint_as_float(static_cast<uint32_t>(14 - ex + 127) << 23);   // 2^(14 - ex)
  const float lo = up * 0.0625f;
  float sum[G][4];
#pragma unroll
  for (int gi = 0; gi < G; ++gi)
#pragma unroll
    for (int x = 0; x < 4; ++x) sum[gi][x] = 0.f;
#pragma unroll
  for (int i = 0; i < W; ++i) {
    const float2 a = unpack2<kFp16>(raw.w[i].x ^ sign), b = unpack2<kFp16>(raw.w[i].y ^ sign);
    const float2 d = unpack2<kFp16>(raw.w[i].z ^ sign), e = unpack2<kFp16>(raw.w[i].w ^ sign);
    out.f[i][0] = pack2<true>(a.x * up, d.x * up);
    out.f[i][1] = pack2<true>(a.y * lo, d.y * lo);
    out.f[i][2] = pack2<true>(b.x * up, e.x * up);
    out.f[i][3] = pack2<true>(b.y * lo, e.y * lo);
    // word c W + i belongs to group i % G
    mma16816(sum[i % G], 0x3c003c00u, 0x3c003c00u, 0x4c004c00u, 0x4c004c00u, out.f[i][0],
             out.f[i][1]);
    mma16816(sum[i % G], 0x3c003c00u, 0x3c003c00u, 0x4c004c00u, 0x4c004c00u, out.f[i][2],
             out.f[i][3]);
  }
  const float mul = ldexpf(fabsf(scale), ex + 10 - kUp - score_over(scale, ex)) * 1.4426950408889634f;
  out.mul = Pair(__shfl_sync(0xffffffffu, mul, 8 * c), __shfl_sync(0xffffffffu, mul, 8 * c + 4));
#pragma unroll
  for (int u = 0; u < 2; ++u) {
#pragma unroll
    for (int gi = 0; gi < G; ++gi) out.sum[u][gi] = sum[gi][u] * (5.9604644775390625e-8f * (1 << kUp));
  }
}

// A lane's offsets into a tile that take more than a shift to form: where its V chunks are
// copied to and where its V words lie.  The empty asm keeps them in registers (formed again
// for every tile they cost about 15 of its instructions).
template <int D>
struct K4Lane {
  int vput, vget;
  __device__ __forceinline__ explicit K4Lane(int lane) {
    const int r = lane >> 2, c = lane & 3;
    // keys 2c and 2c + 1 go to rows c and c + 4 of their eight; at d = 128 rows with bit 1 set
    // swap their halves
    if constexpr (D == 128) {
      const int row = (r >> 1) + 4 * (r & 1);             // of key lane / 4, chunk lane % 4
      vput = row * 64 + ((c ^ (row & 2)) << 4);
      vget = c * 64 + ((((r >> 1) ^ (c & 2)) << 4) | ((r & 1) << 3));
    } else {
      const int kk = lane >> 1;                           // key lane / 2, chunk lane % 2
      vput = ((kk & 8) + ((kk & 7) >> 1) + 4 * (kk & 1)) * 32 + (lane & 1) * 16;
      vget = c * 32 + r * 4;
    }
    asm("" : "+r"(vput), "+r"(vget));
  }
};

// Copies a record tile into a stage of the ring (cp.async, not committed here).
template <int D>
__device__ __forceinline__ void copy_tile(uint32_t stage, const uint8_t *tile, int lane, int vput) {
  using T = Kv4Tile<D>;
  constexpr int kChunks = T::kV / 512;                    // per lane, of K and of V
  const uint8_t *src = tile + lane * 16;
  const uint32_t kdst = stage + lane * 16, vdst = stage + T::kV + vput;
#pragma unroll
  for (int k = 0; k < kChunks; ++k) cp_async16(kdst + k * 512, src + k * 512, 16u);
#pragma unroll
  for (int k = 0; k < kChunks; ++k) cp_async16(vdst + k * 512, src + T::kV + k * 512, 16u);
  if (D == 128 || lane < 16) cp_async16(kdst + T::kPar, src + T::kPar, 16u);
}

// The V words of a half tile: a lane's of keys 2c, 2c + 1, 2c + 8 and 2c + 9.
template <int D>
__device__ __forceinline__ void v_words(const uint8_t *st, int vget, int half,
                                        uint32_t (&w)[4][K4<D>::kG]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint8_t *at = st + Kv4Tile<D>::kV + (half * 16 + 4 * i) * Kv4Tile<D>::kRow + vget;
    if constexpr (K4<D>::kG == 2) {
      const uint2 x = *reinterpret_cast<const uint2 *>(at);
      w[i][0] = x.x; w[i][1] = x.y;
    } else {
      w[i][0] = *reinterpret_cast<const uint32_t *>(at);
    }
  }
}
// Dimensions 2e, 2e + 1 of the words of group gi: byte e of the four keys, in the masks' places.
template <int G>
__device__ __forceinline__ void v_codes(const uint32_t (&w)[4][G], int gi, int e, uint32_t &x,
                                        uint32_t &y) {
  const uint32_t sel = e < 2 ? 0x5410u : 0x7632u;
  x = code_pairs(__byte_perm(w[0][gi], w[1][gi], sel), e & 1);
  y = code_pairs(__byte_perm(w[2][gi], w[3][gi], sel), e & 1);
}

// One tile: keys key0 ... key0 + 31, of which those in [lo, len) count.
template <int D, bool kFp16>
__device__ __forceinline__ void attend_tile(uint8_t *st, int key0, int lo, int len, int lane, int vget,
                                            const K4Query<D> &q, K4State<D> &a, bool centre) {
  using T = Kv4Tile<D>;
  constexpr int G = K4<D>::kG, W = K4<D>::kW;
  const int r = lane >> 2;
  const bool ragged = key0 < lo || key0 + 32 > len;
  constexpr uint32_t kLow = 0x000f000fu << kUp, kHigh = kLow << 4;
  constexpr uint32_t kOnes = 0x3c003c00u;
  // ---- scores: rows r and r + 8 of both halves, heads 2c and 2c + 1 ----
  float s[2][4];
#pragma unroll
  for (int half = 0; half < 2; ++half) {
    uint32_t w[2][W];
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const uint8_t *at = st + (half * 16 + u * 8) * T::kRow + lane * (W * 4);
      if constexpr (W == 4) {
        const uint4 x = *reinterpret_cast<const uint4 *>(at);
        w[u][0] = x.x; w[u][1] = x.y; w[u][2] = x.z; w[u][3] = x.w;
      } else {
        const uint2 x = *reinterpret_cast<const uint2 *>(at);
        w[u][0] = x.x; w[u][1] = x.y;
      }
    }
    float acc[G][4];
#pragma unroll
    for (int i = 0; i < W; ++i)
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const uint32_t x = code_pairs(w[0][i], k), y = code_pairs(w[1][i], k);
        if (i < G && k == 0)
          mma16816_0(acc[i % G], x & kLow, y & kLow, x & kHigh, y & kHigh, q.f[i][2 * k],
                     q.f[i][2 * k + 1]);
        else
          mma16816(acc[i % G], x & kLow, y & kLow, x & kHigh, y & kHigh, q.f[i][2 * k],
                   q.f[i][2 * k + 1]);
      }
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      float ks[G], kz[G];
      par_floats<G>(lds_par<G>(st + T::kPar, half * 16 + u * 8 + r), ks);
      par_floats<G>(lds_par<G>(st + T::kPar + T::kArr, half * 16 + u * 8 + r), kz);
#pragma unroll
      for (int hd = 0; hd < 2; ++hd) {
        float x = kz[0] * q.sum[hd][0];
        if constexpr (G == 2) x = fmaf(kz[1], q.sum[hd][1], x);
#pragma unroll
        for (int gi = 0; gi < G; ++gi) x = fmaf(ks[gi], acc[gi][2 * u + hd], x);
        s[half][2 * u + hd] = x;
      }
      // rounded here: a reference rounded by itself would leave large scores' differences from
      // it as far off as they are large
      const float2 y = (Pair(s[half][2 * u], s[half][2 * u + 1]) * q.mul).get();
      s[half][2 * u] = y.x;
      s[half][2 * u + 1] = y.y;
    }
  }
  // ---- V's scales and zeros: lane's key, for everyone ----
  float vs[G], vz[G];
  par_floats<G>(lds_par<G>(st + T::kPar + 2 * T::kArr, lane), vs);
  par_floats<G>(lds_par<G>(st + T::kPar + 3 * T::kArr, lane), vz);
  if (ragged) {
    if (key0 + lane < lo || key0 + lane >= len) {   // may be anything
#pragma unroll
      for (int gi = 0; gi < G; ++gi) vs[gi] = vz[gi] = 0.f;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int key = key0 + i * 8 + r;
      if (key < lo || key >= len) s[i >> 1][(i & 1) * 2] = s[i >> 1][(i & 1) * 2 + 1] = -INFINITY;
    }
  }
  // ---- raise the references where a score or a scale outgrew them ----
  float top[2], vtop = vs[0];
  if constexpr (G == 2) vtop = fmaxf(vtop, vs[1]);
  bool up = vtop > a.vmax;
#pragma unroll
  for (int hd = 0; hd < 2; ++hd) {
    top[hd] = fmaxf(fmaxf(s[0][hd], s[0][2 + hd]), fmaxf(s[1][hd], s[1][2 + hd]));
    up |= top[hd] > a.thr[hd];
  }
  if (__any_sync(0xffffffffu, up)) {
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) vtop = fmaxf(vtop, __shfl_xor_sync(0xffffffffu, vtop, o));
    float grow = 1.f;
    if (vtop > a.vmax) {
      const float vnew = __uint_as_float((__float_as_uint(vtop) & 0x7f800000u) + 0x00800000u);
      const float rnew = __fdiv_rn(kPScale, vnew);   // powers of two: exact
      grow = a.rinv > 0.f ? __fdiv_rn(rnew, a.rinv) : 0.f;
      a.vmax = vnew;
      a.rinv = rnew;
    }
    const float2 mm = a.minus_m.get();
    float alpha[2], minus[2];
#pragma unroll
    for (int hd = 0; hd < 2; ++hd) {
      float x = top[hd];
#pragma unroll
      for (int o = 4; o < 32; o <<= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, o));
      const float old = -(hd ? mm.y : mm.x), mnew = fmaxf(old, x);
      alpha[hd] = ex2_approx(old - mnew);
      minus[hd] = -mnew;
      a.thr[hd] = __fadd_rd(mnew, kSlack);   // never more: P' has no room for another power of two
      const float both = alpha[hd] * grow;
#pragma unroll
      for (int gi = 0; gi < G; ++gi) {
        a.ps[gi][hd] *= both;
        a.ps[gi][2 + hd] *= both;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          a.o[gi][e][hd] *= both;
          a.o[gi][e][2 + hd] *= both;
        }
      }
    }
    const Pair al(alpha[0], alpha[1]);
    a.minus_m = Pair(minus[0], minus[1]);
    a.l = a.l * al;
#pragma unroll
    for (int gi = 0; gi < G; ++gi) a.oz[gi] = a.oz[gi] * al;
  }
  // over the K codes, which all have read (the vote): s / reference, z + m s
  uint8_t *const vpar = st;
  const float middle = !kFp16 || centre ? kMiddle : 0.f;
  const float unm = middle * -a.vmax * (1.f / kPScale);   // takes it off what hi leaves of P'
  if constexpr (G == 2)
    reinterpret_cast<float4 *>(vpar)[lane] =
        make_float4(vs[0] * a.rinv, vs[1] * a.rinv, fmaf(middle, vs[0], vz[0]),
                    fmaf(middle, vs[1], vz[1]));
  else
    reinterpret_cast<float2 *>(vpar)[lane] = make_float2(vs[0] * a.rinv, fmaf(middle, vs[0], vz[0]));
  __syncwarp();              // V's scales and zeros are in place
  // ---- weights ----
  uint32_t pb[G][2][2];      // B operands: [group][half][k rows 0-7, 8-15]
  uint32_t pl[G][2][2];      // what hi leaves of P' (fp16)
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 e = (Pair(s[i >> 1][(i & 1) * 2], s[i >> 1][(i & 1) * 2 + 1]) + a.minus_m).get();
    const Pair p(ex2_approx(e.x), ex2_approx(e.y));
    a.l = a.l + p;
    float vsr[G], vc[G];
    if constexpr (G == 2) {
      const float4 x = reinterpret_cast<const float4 *>(vpar)[i * 8 + r];
      vsr[0] = x.x; vsr[1] = x.y; vc[0] = x.z; vc[1] = x.w;
    } else {
      const float2 x = reinterpret_cast<const float2 *>(vpar)[i * 8 + r];
      vsr[0] = x.x; vc[0] = x.y;
    }
#pragma unroll
    for (int gi = 0; gi < G; ++gi) {
      a.oz[gi] = fma(p, Pair(vc[gi], vc[gi]), a.oz[gi]);
      const float2 w = (p * Pair(vsr[gi], vsr[gi])).get();
      const uint32_t hi = pack2<true>(w.x, w.y);
      pb[gi][i >> 1][i & 1] = transpose8x8(hi);
      if (kFp16) {
        const float2 h = unpack2<true>(hi);
        const float2 rest = make_float2(w.x - h.x, w.y - h.y);
        pl[gi][i >> 1][i & 1] = transpose8x8(pack2<true>(rest.x, rest.y));
        a.oz[gi] = fma(Pair(rest.x, rest.y), Pair(unm, unm), a.oz[gi]);
      }
    }
  }
  // ---- output: rows are dimensions, k the keys ----
  if (centre) {
    // The tile's sums start at -m sum P' and are added to the warp's, rounded to nearest.
    uint32_t w[2][4][G];
#pragma unroll
    for (int half = 0; half < 2; ++half) v_words<D>(st, vget, half, w[half]);
#pragma unroll
    for (int gi = 0; gi < G; ++gi) {
      float t[4];              // sum of P', heads 2c and 2c + 1 (twice)
      mma16816_0(t, kOnes, kOnes, kOnes, kOnes, pb[gi][0][0], pb[gi][0][1]);
      mma16816(t, kOnes, kOnes, kOnes, kOnes, pb[gi][1][0], pb[gi][1][1]);
      constexpr float kUnit = -kMiddle / (16777216.f / (1 << kUp));
      const Pair c1 = Pair(t[0], t[1]) * Pair(kUnit, kUnit);
      const Pair c16 = Pair(t[0], t[1]) * Pair(16.f * kUnit, 16.f * kUnit);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        float sum[4];
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          uint32_t x, y;
          v_codes<G>(w[half], gi, e, x, y);
          if (half == 0)
            mma16816_c(sum, x & kLow, x & kHigh, y & kLow, y & kHigh, pb[gi][0][0], pb[gi][0][1],
                       c1, c16);
          else
            mma16816(sum, x & kLow, x & kHigh, y & kLow, y & kHigh, pb[gi][1][0], pb[gi][1][1]);
          if (kFp16)
            mma16816(sum, x & kLow, x & kHigh, y & kLow, y & kHigh, pl[gi][half][0],
                     pl[gi][half][1]);
        }
        float *o = a.o[gi][e];
#pragma unroll
        for (int x = 0; x < 4; x += 2) {
          const float2 y = (Pair(o[x], o[x + 1]) + Pair(sum[x], sum[x + 1])).get();
          o[x] = y.x;
          o[x + 1] = y.y;
        }
      }
    }
    return;
  }
#pragma unroll
  for (int half = 0; half < 2; ++half) {
    uint32_t w[4][G];
    v_words<D>(st, vget, half, w);
#pragma unroll
    for (int gi = 0; gi < G; ++gi) {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        uint32_t x, y;
        v_codes<G>(w, gi, e, x, y);
        mma16816(a.o[gi][e], x & kLow, x & kHigh, y & kLow, y & kHigh, pb[gi][half][0],
                 pb[gi][half][1]);
        if (kFp16)
          mma16816(a.o[gi][e], x & kLow, x & kHigh, y & kLow, y & kHigh, pl[gi][half][0],
                   pl[gi][half][1]);
      }
      if (!kFp16) mma16816(a.ps[gi], kOnes, kOnes, kOnes, kOnes, pb[gi][half][0], pb[gi][half][1]);
    }
  }
}

// Length of sequence b held to its table row, and the first key that its window shows.
__device__ __forceinline__ int seq_len(const Kv4DecodeParams &p, int b, int32_t &err) {
  const int cap = p.width << p.page_log2;
  const int raw = p.lens[b], len = min(max(raw, 0), cap);
  if (raw != len) err |= NSA_DEVERR_BAD_SEQLENS;
  return len;
}
__device__ __forceinline__ int seq_lo(const Kv4DecodeParams &p, int len) {
  return p.window > 0 && len > p.window ? len - p.window : 0;
}

// Fills a segment's tiles.  With a selection: the kept blocks, valid, first of their value,
// with a page in the pool (64 words of scratch in shared memory bring them together).
template <bool kSel>
__device__ __forceinline__ void open_segment(const Kv4DecodeParams &p, K4Seg &sg, uint8_t *scratch,
                                             int lane, int32_t &err) {
  int blk = -1;
  if (kSel && lane < p.topk)
    blk = p.sel[((int64_t)sg.h * p.num_seqs + sg.b) * p.topk + lane];
  int32_t ignore = 0;        // reported once, where the lengths are first read
  sg.len = seq_len(p, sg.b, ignore);
  sg.lo = seq_lo(p, sg.len);
  sg.first = sg.lo >> 5;
  sg.tiles = ((sg.len + 31) >> 5) - sg.first;
  if (kSel) {
    const int nblk = (sg.len + (1 << p.page_log2) - 1) >> p.page_log2;
    if (lane < p.topk && (blk < -1 || blk >= nblk)) err |= NSA_DEVERR_BAD_INDEX;
    bool ok = blk >= 0 && blk < nblk;
    const uint32_t same = __match_any_sync(0xffffffffu, blk);
    ok = ok && (same & ((1u << lane) - 1u)) == 0;
    int pg = -1;
    if (ok) {
      pg = p.table[(int64_t)sg.b * p.width + blk];
      if (pg < 0 || pg >= p.num_pages) {
        ok = false;
        err |= NSA_DEVERR_BAD_INDEX;
      }
    }
    const uint32_t m = __ballot_sync(0xffffffffu, ok);
    int2 *list = reinterpret_cast<int2 *>(scratch);
    if (ok) list[__popc(m & ((1u << lane) - 1u))] = make_int2(pg, blk << p.page_log2);
    __syncwarp();
    const int2 mine = list[lane];
    __syncwarp();
    sg.page = mine.x;
    sg.key = mine.y;
    sg.tiles = __popc(m) << (p.page_log2 - 5);
  }
}

// Tiles t0, t0 + step, ... (count of them) of a segment through this warp's ring: all its
// stages, or those before a kept part.
template <int D, bool kFp16, bool kSel>
struct K4Stream {
  using T = Kv4Tile<D>;
  const Kv4DecodeParams &p;
  const K4Seg &sg;
  const int t0, step, count, lane;
  uint8_t *const ring;
  const bool full;                    // all stages
  const K4Lane<D> at;
  const uint8_t *my_tile;             // of tile 32 * block + lane: where it lies (null: nowhere)
  int my_key;                         // and its first key
  int put, get;                       // offsets of the stages to fill and to use next
  int keys[kStages];                  // first keys of the tiles in the ring, -1: nothing to do

  __device__ __forceinline__ K4Stream(const Kv4DecodeParams &p_, const K4Seg &sg_, int t0_,
                                      int count_, int step_, uint8_t *ring_, bool full_, int lane_)
      : p(p_), sg(sg_), t0(t0_), step(step_), count(count_), lane(lane_), ring(ring_),
        full(full_), at(lane_), my_tile(nullptr), my_key(0), put(0), get(0) {}

  __device__ __forceinline__ void next(int &stage) const {
    stage += T::kBytes;
    if (stage == (full ? kStages : kStages - 1) * T::kBytes) stage = 0;
  }
  __device__ __forceinline__ int issue(int n, int32_t &err) {
    int key = -1;
    if (n < count) {
      const int tpl = p.page_log2 - 5;
      if ((n & 31) == 0) {            // look up the next 32 tiles' pages
        const int i = n + lane, t = t0 + i * step;
        int pg = -1;
        if (kSel) {
          pg = __shfl_sync(0xffffffffu, sg.page, t >> tpl);
          my_key = __shfl_sync(0xffffffffu, sg.key, t >> tpl) + ((t & ((1 << tpl) - 1)) << 5);
          if (i >= count) pg = -1;
        } else if (i < count) {
          my_key = (sg.first + t) << 5;
          pg = p.table[(int64_t)sg.b * p.width + (my_key >> p.page_log2)];
          if (pg < 0 || pg >= p.num_pages) {
            pg = -1;
            err |= NSA_DEVERR_BAD_INDEX;
          }
        }
        if (my_key >= sg.len || my_key + 32 <= sg.lo) pg = -1;
        my_tile = pg < 0 ? nullptr
                         : p.pool + ((((int64_t)pg * p.h_k + sg.h) << tpl) +
                                     ((my_key & ((1 << p.page_log2) - 1)) >> 5)) * T::kBytes;
      }
      const uint8_t *tile = reinterpret_cast<const uint8_t *>(__shfl_sync(
          0xffffffffu, reinterpret_cast<unsigned long long>(my_tile), n & 31));
      const int k0 = __shfl_sync(0xffffffffu, my_key, n & 31);
      if (tile) {
        key = k0;
        copy_tile<D>(smem_u32(ring) + put, tile, lane, at.vput);
      }
    }
    cp_async_commit();
    next(put);
    return key;
  }
  __device__ __forceinline__ void start(int32_t &err) {
    keys[0] = issue(0, err);
    if (full) keys[1] = issue(1, err);
  }
  __device__ __forceinline__ void run(const K4Query<D> &q, K4State<D> &a, int32_t &err) {
    static_assert(kStages == 3, "two tiles ahead, or one beside a kept part");
    const bool centre = kFp16 ? count > kFewTiles || sg.tiles > kFewKeys / 32
                              : (int64_t)count * count * sg.tiles > kFewSquare;
    for (int n = 0; n < count; ++n) {
      if (full) {
        keys[2] = issue(n + 2, err);
        cp_async_wait_group<2>();
      } else {
        keys[1] = issue(n + 1, err);
        cp_async_wait_group<1>();
      }
      __syncwarp();
      if (keys[0] >= 0) attend_tile<D, kFp16>(ring + get, keys[0], sg.lo, sg.len, lane, at.vget, q, a, centre);
      __syncwarp();                   // the stage is filled again in the next turn
      next(get);
      keys[0] = keys[1];
      keys[1] = keys[2];
    }
    cp_async_wait_all();
    const float2 mul = q.mul.get();
    constexpr float kLarge = 1.f * (1ull << 59) * (1ull << 59);   // 2^kMulTop
    static_assert(kMulTop == 118, "");
    if (__any_sync(0xffffffffu, fmaxf(mul.x, mul.y) >= kLarge)) {   // powers may have been left out
      K4RawQuery<D> raw;
      fetch_query<D>(p, sg, lane, raw);
      const int over = score_over(p.scale, query_exponent<D, kFp16>(raw)), c = lane & 3;
      const float2 mm = a.minus_m.get();
      const int o0 = __shfl_sync(0xffffffffu, over, 8 * c), o1 = __shfl_sync(0xffffffffu, over, 8 * c + 4);
      a.minus_m = Pair(ldexpf(mm.x, o0), ldexpf(mm.y, o1));
    }
  }
};

// A warp's maxima, sums and zero terms, over its lanes.
template <int D>
struct K4Sums {
  float m[2], l[2], oz[2][K4<D>::kG];
  __device__ __forceinline__ explicit K4Sums(const K4State<D> &a) {
    const float2 mm = a.minus_m.get(), ll = a.l.get();
    m[0] = -mm.x;
    m[1] = -mm.y;
    l[0] = ll.x;
    l[1] = ll.y;
#pragma unroll
    for (int gi = 0; gi < K4<D>::kG; ++gi) {
      const float2 z = a.oz[gi].get();
      oz[0][gi] = z.x;
      oz[1][gi] = z.y;
    }
#pragma unroll
    for (int o = 4; o < 32; o <<= 1)
#pragma unroll
      for (int hd = 0; hd < 2; ++hd) {
        l[hd] += __shfl_xor_sync(0xffffffffu, l[hd], o);
#pragma unroll
        for (int gi = 0; gi < K4<D>::kG; ++gi)
          oz[hd][gi] += __shfl_xor_sync(0xffffffffu, oz[hd][gi], o);
      }
  }
  __device__ __forceinline__ float4 pairs() const { return make_float4(m[0], l[0], m[1], l[1]); }
};

// O times f (per head of the lane) into an area [head pairs].
template <int D, bool kFp16>
__device__ __forceinline__ void leave_out(float *area, int lane, const K4State<D> &a,
                                          const K4Sums<D> &sums, float f0, float f1) {
  constexpr int G = K4<D>::kG;
  const int r = lane >> 2, c = lane & 3;
  const float back = a.rinv > 0.f ? __fdiv_rn(1.f, a.rinv) : 0.f;   // a power of two
#pragma unroll
  for (int hd = 0; hd < 2; ++hd) {
    const float f = hd ? f1 : f0, fb = f * back, o1 = fb * (16777216.f / (1 << kUp)), o16 = o1 * 0.0625f;
    float *dst = area + c * K4<D>::kHeadPair + hd * D + 8 * r;
#pragma unroll
    for (int gi = 0; gi < G; ++gi) {
      const float z = f * sums.oz[hd][gi], base = kFp16 ? z : fmaf(-kMiddle * fb, a.ps[gi][hd], z);
#pragma unroll
      for (int e = 0; e < 4; ++e)
        *reinterpret_cast<float2 *>(dst + gi * 64 + 2 * e) = make_float2(
            fmaf(a.o[gi][e][hd], o1, base), fmaf(a.o[gi][e][2 + hd], o16, base));
    }
  }
}

// Final values of dimensions dim ... dim + 3 of query head hq.
template <int D, bool kFp16>
__device__ __forceinline__ void write_out(const Kv4DecodeParams &p, int b, int hq, int dim, float4 x,
                                          float M, float l) {
  const bool any = l != 0.f;                        // a NaN sum stays one
  const float inv = any ? __fdividef(1.f, l) : 0.f;
  const int64_t row = (int64_t)b * p.h_q + hq;
  reinterpret_cast<uint2 *>(p.out)[(row * D + dim) >> 2] =
      make_uint2(pack2<kFp16>(x.x * inv, x.y * inv), pack2<kFp16>(x.z * inv, x.w * inv));
  if (dim == 0)
    p.lse[(int64_t)hq * p.num_seqs + b] = any ? (M + log2f(l)) * 0.69314718055994531f : -INFINITY;
}

__device__ __forceinline__ uint32_t in_cta(uint32_t addr, int rank) {
  uint32_t a;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(addr), "r"(rank));
  return a;
}
__device__ __forceinline__ float4 ld_cluster4(uint32_t a) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(a)
               : "memory");
  return v;
}
__device__ __forceinline__ float2 ld_cluster2(uint32_t a) {
  float2 v;
  asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(a) : "memory");
  return v;
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// kWarps warps per segment, in one CTA; kCluster: in each of a cluster's `parts` CTAs.
template <int D, bool kFp16, bool kSel, int kWarps, bool kCluster>
__global__ void __launch_bounds__(kWarps * 32, kSmWarps<D> / kWarps)
    kv4_seg_kernel(Kv4DecodeParams p, int units, int parts) {
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ float4 ml[kWarps][kK4Heads / 2];          // m, l of two heads
  __shared__ float lsum[kWarps][kK4Heads];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  K4Seg sg = {};
  const unsigned seg = kCluster ? blockIdx.x / parts : blockIdx.x;
  const int rank = kCluster ? blockIdx.x - seg * parts : 0, step = kCluster ? parts * kWarps : kWarps;
  sg.b = static_cast<int>(seg / static_cast<unsigned>(units));
  set_unit(p, static_cast<int>(seg) - sg.b * units, sg);
  int32_t err = 0;
  after_previous();
  K4RawQuery<D> raw;
  fetch_query<D>(p, sg, lane, raw);
  open_segment<kSel>(p, sg, smem + warp * K4<D>::kRing, lane, err);
  const int first = rank * kWarps + warp;
  K4Stream<D, kFp16, kSel> st(p, sg, first, max(0, (sg.tiles - first + step - 1) / step), step,
                              smem + warp * K4<D>::kRing, true, lane);
  st.start(err);
  K4Query<D> q;
  make_query<D, kFp16>(raw, p.scale, lane, q);
  K4State<D> a;
  a.clear();
  st.run(q, a, err);
  if (tid == 0) seq_len(p, sg.b, err);
  err = __reduce_or_sync(0xffffffffu, err);
  if (err && lane == 0) raise(p.status, err);
  __shared__ float2 part_ml[kCluster ? kK4Heads : 1];
  // a CTA's own sums, where no area lies: the last stage of the first warp's ring
  float *const part = reinterpret_cast<float *>(smem + K4<D>::kKept);
  static_assert(kK4Heads * D * 4 <= Kv4Tile<D>::kBytes, "a stage holds a CTA's sums");

  // the warps agree on each head's maximum, scale their sums to it, and add up
  const int r = lane >> 2, c = lane & 3;
  const K4Sums<D> sums(a);
  if (r == 0) ml[warp][c] = sums.pairs();
  __syncthreads();
  float M0 = -INFINITY, M1 = -INFINITY;                // -inf without keys
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    const float4 v = ml[w][c];
    M0 = fmaxf(M0, v.x);
    M1 = fmaxf(M1, v.z);
  }
  const float f0 = sums.l[0] != 0.f ? ex2_approx(sums.m[0] - M0) : 0.f;
  const float f1 = sums.l[1] != 0.f ? ex2_approx(sums.m[1] - M1) : 0.f;
  if (r == 0)
    *reinterpret_cast<float2 *>(&lsum[warp][2 * c]) = make_float2(sums.l[0] * f0, sums.l[1] * f1);
  leave_out<D, kFp16>(reinterpret_cast<float *>(smem + warp * K4<D>::kRing), lane, a, sums, f0, f1);
  __syncthreads();
  for (int i = tid; i < sg.g * (D / 4); i += kWarps * 32) {
    const int head = i / (D / 4), dim = 4 * (i % (D / 4));
    const uint8_t *src = smem + ((head >> 1) * K4<D>::kHeadPair + (head & 1) * D + dim) * 4;
    float l = 0.f, M = -INFINITY;
    float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      const float4 o = *reinterpret_cast<const float4 *>(src + w * K4<D>::kRing);
      l += lsum[w][head];
      x.x += o.x;
      x.y += o.y;
      x.z += o.z;
      x.w += o.w;
    }
    if (dim == 0) {
#pragma unroll
      for (int w = 0; w < kWarps; ++w)
        M = fmaxf(M, head & 1 ? ml[w][head >> 1].z : ml[w][head >> 1].x);
    }
    if (!kCluster) {
      write_out<D, kFp16>(p, sg.b, sg.q0 + head, dim, x, M, l);
    } else {
      *reinterpret_cast<float4 *>(part + head * D + dim) = x;
      if (dim == 0) part_ml[head] = make_float2(M, l);
    }
  }
  if constexpr (kCluster) {
    // the CTAs' sums, from their shared memory, each CTA adding up a share of the outputs
    cluster_sync();
    const uint32_t mine = smem_u32(part), mine_ml = smem_u32(part_ml);
    for (int i = rank + parts * tid; i < sg.g * (D / 4); i += parts * kWarps * 32) {
      const int head = i / (D / 4), dim = 4 * (i % (D / 4));
      float2 v[8];
      float4 o[8];
      float M = -INFINITY, l = 0.f;
      float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        v[k] = make_float2(-INFINITY, 0.f);
        if (k < parts) {
          v[k] = ld_cluster2(in_cta(mine_ml + head * 8, k));
          o[k] = ld_cluster4(in_cta(mine + (head * D + dim) * 4, k));
        }
      }
#pragma unroll
      for (int k = 0; k < 8; ++k) M = fmaxf(M, v[k].x);
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        if (v[k].y == 0.f) continue;                   // a CTA without keys, or none
        const float w = ex2_approx(v[k].x - M);
        l = fmaf(w, v[k].y, l);
        x.x = fmaf(w, o[k].x, x.x);
        x.y = fmaf(w, o[k].y, x.y);
        x.z = fmaf(w, o[k].z, x.z);
        x.w = fmaf(w, o[k].w, x.w);
      }
      write_out<D, kFp16>(p, sg.b, sg.q0 + head, dim, x, M, l);
    }
    cluster_sync();                                    // no CTA leaves while it is read
  }
}

// Tiles that a sequence's segments count as: what they have, at least one, so that an empty
// one's output is written too, and kOver.
__device__ __forceinline__ int counted_tiles(const Kv4DecodeParams &p, int len) {
  return max(((len + 31) >> 5) - (seq_lo(p, len) >> 5), 1) + kOver;
}

__device__ __forceinline__ K4Split *splits_of(const Kv4DecodeParams &p) {
  return static_cast<K4Split *>(p.ws);
}
// Partial result i: O [heads][D] (not divided by l), then (m, l) per head.
__host__ __device__ constexpr int part_floats(int d, int g) {
  return (g < kK4Heads ? g : kK4Heads) * (d + 2);
}
template <int D>
__device__ __forceinline__ float *part_of(const Kv4DecodeParams &p, int i) {
  return reinterpret_cast<float *>(static_cast<uint8_t *>(p.ws) + kK4MaxCtas * sizeof(K4Split)) +
         (int64_t)i * part_floats(D, p.g);
}

__device__ __forceinline__ int warp_incl_sum(int x, int lane) {
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  return x;
}

// Equal runs of the batch's counted tiles.
template <int D, bool kFp16>
__global__ void __launch_bounds__(K4<D>::kRunThreads, 2)
    kv4_run_kernel(Kv4DecodeParams p, int units) {
  constexpr int kWarps = K4<D>::kRunWarps, kThreads = K4<D>::kRunThreads;
  extern __shared__ __align__(128) uint8_t smem[];
  // of a warp's parts ([0]: first, [1]: last): m, l of two heads; factors, l times them
  __shared__ float4 ml[2][kWarps][kK4Heads / 2];
  __shared__ float2 fac[2][kWarps][kK4Heads], top[kWarps + 1][kK4Heads / 2];
  __shared__ int pre[kThreads], wsum[kWarps], flags[kWarps];
  __shared__ int4 groups[kWarps + 1];    // of the group that warp i - 1 opens: sequence, unit, end
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, c = lane & 3;
  after_previous();
  // ---- the batch's tiles ----
  const int per_thread = (p.num_seqs + kThreads - 1) / kThreads;
  const int b0 = min(tid * per_thread, p.num_seqs), b1 = min(b0 + per_thread, p.num_seqs);
  int32_t err = 0, ignore = 0;
  int mine = 0;
  for (int b = b0; b < b1; ++b) mine += counted_tiles(p, seq_len(p, b, err));
  if (blockIdx.x == 0 && err) raise(p.status, err);
  err = 0;
  pre[tid] = warp_incl_sum(mine * units, lane);
  if (lane == 31) wsum[warp] = pre[tid];
  __syncthreads();
  int total = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) total += wsum[w];
  // the sequence that holds tile v (< total), and that sequence's first tile
  auto locate = [&](int v, int &b, int &base) {
    int w = 0, off = 0;                    // the warp whose sequences hold it, the tiles before
#pragma unroll
    for (int k = 0; k + 1 < kWarps; ++k)
      if (v >= off + wsum[w]) off += wsum[w++];
    const int x = off + pre[w * 32 + lane];
    const uint32_t before = __ballot_sync(0xffffffffu, x <= v);
    const int chunk = w * 32 + __popc(before);   // threads whose sequences lie before it
    base = before ? __shfl_sync(0xffffffffu, x, __popc(before) - 1) : off;
    b = chunk * per_thread;
    if (per_thread == 1) return;
    while (b < p.num_seqs) {               // 32 sequences at a time
      const int n = b + lane < p.num_seqs
                        ? counted_tiles(p, seq_len(p, b + lane, ignore)) * units : 0;
      const int in = warp_incl_sum(n, lane);
      const uint32_t past = __ballot_sync(0xffffffffu, v < base + in);
      const int hit = past ? __ffs(past) - 1 : 31;
      base += __shfl_sync(0xffffffffu, past ? in - n : in, hit);
      b += past ? hit : 32;
      if (past) break;
    }
  };
  // ---- this warp's run ----
  const int warps = gridDim.x * kWarps;
  const int per_warp = (total + warps - 1) / warps;
  const int per = per_warp * kWarps;                     // tiles of a CTA
  const int from = static_cast<int>(min((int64_t)blockIdx.x * per, (int64_t)total));
  const int to = from + min(per, total - from);
  int at = from + min(warp * per_warp, to - from), b = 0, base = 0;
  const int stop = at + min(per_warp, to - at);
  if (at < stop) locate(at, b, base);
  uint8_t *const ring = smem + warp * K4<D>::kRing;
  // What the run leaves for the CTA: a first part, of a segment begun before the run (and
  // whether that goes on behind it, whether it is kept in the ring's last stage), and a last
  // part, of a segment that begins in the run and goes on.
  constexpr int kFirst = 1, kLast = 2, kOn = 4, kKeep = 8;
  int left = 0;
  int unit = -1, nt = 0;
  K4State<D> a;
  while (at < stop) {
    K4Seg sg = {};
    sg.b = b;
    if (unit <= 0) nt = counted_tiles(p, seq_len(p, b, ignore));
    if (unit < 0) unit = (at - base) / nt;
    set_unit(p, unit, sg);
    const int seg0 = base + unit * nt;
    const int v0 = at - seg0, v1 = min(nt, stop - seg0);
    a.clear();
    if (v1 > kOver) {
      K4RawQuery<D> raw;
      fetch_query<D>(p, sg, lane, raw);
      open_segment<false>(p, sg, ring, lane, err);
      const int t0 = max(0, v0 - kOver), t1 = min(v1 - kOver, sg.tiles);
      K4Stream<D, kFp16, false> st(p, sg, t0, max(0, t1 - t0), 1, ring, !(left & kKeep), lane);
      st.start(err);
      K4Query<D> q;
      make_query<D, kFp16>(raw, p.scale, lane, q);
      st.run(q, a, err);
    }
    const K4Sums<D> sums(a);
    at = seg0 + v1;
    const bool goes_on = v1 < nt, first = v0 > 0;
    if (lane < 4) ml[first ? 0 : 1][warp][c] = sums.pairs();
    if (first) {
      left |= kFirst | (goes_on ? kOn : 0) | (at < stop ? kKeep : 0);
      if (warp == 0 && lane == 0) groups[0] = make_int4(b, unit, 0, 0);
      if (at < stop) leave_out<D, kFp16>(reinterpret_cast<float *>(ring + K4<D>::kKept), lane, a, sums, 1.f,
                                           1.f);
    } else if (goes_on) {                  // the run's last: stays in registers
      left |= kLast;
      if (lane == 0) groups[warp + 1] = make_int4(b, unit, seg0 + nt, 0);
    } else {
      float *area = reinterpret_cast<float *>(ring);
      leave_out<D, kFp16>(area, lane, a, sums, 1.f, 1.f);
      __syncwarp();
#pragma unroll 1
      for (int i = lane; i < sg.g * (D / 4); i += 32) {
        const int head = i / (D / 4), dim = 4 * (i % (D / 4));
        const float4 o = *reinterpret_cast<const float4 *>(
            area + (head >> 1) * K4<D>::kHeadPair + (head & 1) * D + dim);
        const float4 v = ml[1][warp][head >> 1];
        write_out<D, kFp16>(p, b, sg.q0 + head, dim, o, head & 1 ? v.z : v.x, head & 1 ? v.w : v.y);
      }
      __syncwarp();                        // read before the ring is filled again
    }
    if (++unit == units) {
      unit = 0;
      base += nt * units;
      ++b;
    }
  }
  err = __reduce_or_sync(0xffffffffu, err);
  if (err && lane == 0) raise(p.status, err);
  if (lane == 0) flags[warp] = left;
  if (tid == 0) splits_of(p)[blockIdx.x] = K4Split{0, 0};
  __syncthreads();
  // ---- join the parts of segments that cross warps ----
  // A group is a segment's parts in this CTA: the last part of warp `open` (-1: the segment
  // began in an earlier CTA) and the first parts of the warps behind it, up to the next
  // warp with a last part.
  const int fl = lane < kWarps ? flags[lane] : 0;
  const uint32_t firsts = __ballot_sync(0xffffffffu, fl & kFirst);
  const uint32_t lasts = __ballot_sync(0xffffffffu, fl & kLast);
  const uint32_t ons = __ballot_sync(0xffffffffu, fl & kOn);
  const uint32_t keeps = __ballot_sync(0xffffffffu, fl & kKeep);
  auto members = [&](int open) {           // warps whose first part belongs to the group
    const uint32_t behind = ~0u << (open + 1), next = lasts & behind;
    return firsts & behind & (next ? (next ^ (next - 1)) : ~0u);
  };
  auto opener = [&](int side) {
    const uint32_t before = lasts & ((1u << warp) - 1u);
    return side ? warp : 31 - __clz(before);
  };
#pragma unroll 1
  for (int side = 0; side < 2; ++side) {
    if (!(left & (side ? kLast : kFirst))) continue;
    const int open = opener(side), r = lane >> 2;
    const uint32_t in = members(open);
    float M0 = -INFINITY, M1 = -INFINITY;  // lane (r, c): warp r's part, heads 2c, 2c + 1
    if (r == open || (in >> r & 1)) {
      const float4 v = ml[r == open][r][c];
      M0 = v.x;
      M1 = v.z;
    }
#pragma unroll
    for (int o = 4; o < 32; o <<= 1) {
      M0 = fmaxf(M0, __shfl_xor_sync(0xffffffffu, M0, o));
      M1 = fmaxf(M1, __shfl_xor_sync(0xffffffffu, M1, o));
    }
    const float4 v = ml[side][warp][c];
    const float f0 = v.y != 0.f ? ex2_approx(v.x - M0) : 0.f;
    const float f1 = v.w != 0.f ? ex2_approx(v.z - M1) : 0.f;
    const bool kept = !side && (left & kKeep);   // left already, without its factor
    if (!kept) leave_out<D, kFp16>(reinterpret_cast<float *>(ring), lane, a, K4Sums<D>(a), f0, f1);
    if (lane < 4) {
      fac[side][warp][2 * c] = make_float2(kept ? f0 : 1.f, v.y * f0);
      fac[side][warp][2 * c + 1] = make_float2(kept ? f1 : 1.f, v.w * f1);
      top[open + 1][c] = make_float2(M0, M1);    // the same from all of the group
    }
  }
  __syncthreads();
  // Group i is the one that warp i - 1 opens.  A small one is a single warp's work.
  const bool small = min(p.g, kK4Heads) * (D / 4) <= 64;
  const int th = small ? lane : tid, nth = small ? 32 : kThreads;
#pragma unroll 1
  for (uint32_t todo = lasts << 1 | (members(-1) ? 1u : 0u); todo; todo &= todo - 1) {
    const int gr = __ffs(todo) - 1, open = gr - 1;
    if (small && gr % kWarps != warp) continue;
    const uint32_t in = members(open), all = in | (open >= 0 ? 1u << open : 0u);
    const bool on = in ? ons >> (31 - __clz(in)) & 1 : true;
    const int4 who = groups[gr];
    K4Seg sg = {};
    sg.b = who.x;
    set_unit(p, who.y, sg);
    float *part = nullptr;
    if (open < 0) part = part_of<D>(p, 2 * blockIdx.x);
    else if (on) part = part_of<D>(p, 2 * blockIdx.x + 1);
    if (open >= 0 && on && th == 0)
      splits_of(p)[blockIdx.x] = K4Split{
          sg.b * units + who.y, (who.z - 1) / per - static_cast<int>(blockIdx.x) + 1};
#pragma unroll 1
    for (int i = th; i < sg.g * (D / 4); i += nth) {
      const int head = i / (D / 4), dim = 4 * (i % (D / 4));
      const int off = ((head >> 1) * K4<D>::kHeadPair + (head & 1) * D + dim) * 4;
      float l = 0.f;
      float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 2
      for (uint32_t m = all; m; m &= m - 1) {
        const int w = __ffs(m) - 1;
        const bool fst = w != open;
        const float4 o = *reinterpret_cast<const float4 *>(
            smem + w * K4<D>::kRing + (fst && (keeps >> w & 1) ? K4<D>::kKept : 0) + off);
        const float2 f = fac[!fst][w][head];
        l += f.y;
        x.x = fmaf(f.x, o.x, x.x);
        x.y = fmaf(f.x, o.y, x.y);
        x.z = fmaf(f.x, o.z, x.z);
        x.w = fmaf(f.x, o.w, x.w);
      }
      const float2 m2 = top[gr][head >> 1];
      const float M = head & 1 ? m2.y : m2.x;
      if (part) {
        float2 *dst = reinterpret_cast<float2 *>(part + head * D + dim);
        dst[0] = make_float2(x.x, x.y);
        dst[1] = make_float2(x.z, x.w);
        if (dim == 0) *reinterpret_cast<float2 *>(part + sg.g * D + 2 * head) = make_float2(M, l);
      } else {
        write_out<D, kFp16>(p, sg.b, sg.q0 + head, dim, x, M, l);
      }
    }
  }
}

// Joins the parts of the segment that begins in CTA blockIdx.x and ends in another: its own
// second part and the following CTAs' first ones.  One CTA per (split, head): its warps take
// the parts in turn, eight in flight.
constexpr int kMergeThreads = 256;
template <int D, bool kFp16>
__global__ void __launch_bounds__(kMergeThreads) kv4_merge_kernel(Kv4DecodeParams p, int units) {
  constexpr int kWarps = kMergeThreads / 32, E = D / 32;
  __shared__ __align__(16) float acc[kWarps][D];
  __shared__ float2 wml[kWarps];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, head = blockIdx.y;
  after_previous();
  const K4Split sp = splits_of(p)[blockIdx.x];
  if (sp.parts == 0) return;
  K4Seg sg = {};
  sg.b = sp.seg / units;
  set_unit(p, sp.seg - sg.b * units, sg);
  if (head >= sg.g) return;
  float M = -INFINITY, l = 0.f, x[E];
#pragma unroll
  for (int e = 0; e < E; ++e) x[e] = 0.f;
  for (int i0 = warp; i0 < sp.parts; i0 += 8 * kWarps) {
    float2 v[8];
    float o[8][E];
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      const int i = i0 + u * kWarps;
      v[u] = make_float2(-INFINITY, 0.f);
#pragma unroll
      for (int e = 0; e < E; ++e) o[u][e] = 0.f;
      if (i < sp.parts) {
        const float *part = part_of<D>(p, i == 0 ? 2 * blockIdx.x + 1 : 2 * (blockIdx.x + i));
        v[u] = __ldcg(reinterpret_cast<const float2 *>(part + sg.g * D + 2 * head));
        const float2 *src = reinterpret_cast<const float2 *>(part + head * D + lane * E);
#pragma unroll
        for (int e = 0; e < E / 2; ++e) {
          const float2 y = __ldcg(src + e);
          o[u][2 * e] = y.x;
          o[u][2 * e + 1] = y.y;
        }
      }
    }
    float mnew = M;
#pragma unroll
    for (int u = 0; u < 8; ++u) mnew = fmaxf(mnew, v[u].x);
    const float old = l != 0.f ? ex2_approx(M - mnew) : 0.f;
    l *= old;
#pragma unroll
    for (int e = 0; e < E; ++e) x[e] *= old;
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      const float w = v[u].y != 0.f ? ex2_approx(v[u].x - mnew) : 0.f;
      l = fmaf(w, v[u].y, l);
#pragma unroll
      for (int e = 0; e < E; ++e) x[e] = fmaf(w, o[u][e], x[e]);
    }
    M = mnew;
  }
#pragma unroll
  for (int e = 0; e < E; ++e) acc[warp][lane * E + e] = x[e];
  if (lane == 0) wml[warp] = make_float2(M, l);
  __syncthreads();
  if (tid < D / 4) {
    M = -INFINITY;
    l = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) M = fmaxf(M, wml[w].x);
    float4 u = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      const float2 t = wml[w];
      const float f = t.y != 0.f ? ex2_approx(t.x - M) : 0.f;
      const float4 o = *reinterpret_cast<const float4 *>(&acc[w][4 * tid]);
      l = fmaf(f, t.y, l);
      u.x = fmaf(f, o.x, u.x);
      u.y = fmaf(f, o.y, u.y);
      u.z = fmaf(f, o.z, u.z);
      u.w = fmaf(f, o.w, u.w);
    }
    write_out<D, kFp16>(p, sg.b, sg.q0 + head, 4 * tid, u, M, l);
  }
}

// Query heads of one segment are at most kK4Heads: segments of a KV head.
static int head_parts(int g) { return g > kK4Heads ? 2 : 1; }

size_t kv4_decode_workspace(int d, int g, bool selected) {
  if (selected) return 0;
  return kK4MaxCtas * sizeof(K4Split) + 2 * (size_t)kK4MaxCtas * part_floats(d, g) * sizeof(float);
}

// Tiles of the whole batch, counted as the run kernel does, at most (its counters have 32 bits).
int64_t kv4_decode_tiles(const Kv4DecodeParams &p) {
  const int units = p.h_k * head_parts(p.g);
  return (((int64_t)p.width << p.page_log2) / kKv4Tile + 1 + kOver) * p.num_seqs * units;
}

static int sm_count(int dev) {
  static int cache[64];
  if (dev < 0 || dev >= 64) return 148;
  if (cache[dev] == 0) {
    int n = 0;
    cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev);
    cache[dev] = n > 0 ? n : 148;
  }
  return cache[dev];
}

template <int D, bool kFp16, bool kSel, int kWarps, bool kCluster = false>
static cudaError_t run_segs(const Kv4DecodeParams &p, int units, int parts, cudaStream_t s) {
  auto *kernel = kv4_seg_kernel<D, kFp16, kSel, kWarps, kCluster>;
  constexpr int smem = kWarps * K4<D>::kRing;
  const cudaError_t e =
      cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  return launch_kv4(kernel, dim3(static_cast<unsigned>(p.num_seqs) * units * parts), kWarps * 32,
                    smem, parts, s, p, units, parts);
}

// Warps to a segment: an SM holds `room` warps, and a segment's fixed cost is that of one to two
// tiles a warp, so that W warps take about waves * (1.5 + tiles / W), rounded up.  `waves` lies
// between segments / room in the GPU, which ragged lengths come near, and its next whole number,
// which equal lengths take.  More warps where two are equal: then fewer CTAs fit an SM, and they
// spread evenly.  Over 77 measured batches (160 to 2432 segments of 6 to 34 tiles, equal and
// ragged) the choice takes 3 % longer than the best W on average and 19 % at most; d = 128, W =
// 1 / 2 / 3 / 4 / 6: 256 segments of 32 tiles 23.0 / 19.3 / 17.1 / 14.5 / 11.8 us, 512 of 32 33.6 /
// 24.1 / 18.8 / 23.6 / 22.3, 800 ragged to 32 37.7 / 25.8 / 22.0 / 19.6 / 22.9, 1216 of 8 15.4 /
// 17.2 / 16.9 / 18.7 / 23.0.
template <int D>
static int seg_warps(int64_t segs, int64_t most, int sms) {
  constexpr int kRoom = kSmWarps<D>;
  int best = 1;
  double least = 0.;
  for (int w = 1; w <= kRoom / 2; ++w) {
    if (kRoom % w) continue;
    const int64_t slots = (int64_t)sms * (kRoom / w);
    const double part = static_cast<double>(segs) / static_cast<double>(slots);
    const double waves = 0.75 * (part > 1. ? part : 1.) + 0.25 * ((segs + slots - 1) / slots);
    const double t = waves * (1.5 + (most + w - 1) / w);
    if (w == 1 || t <= least) {
      best = w;
      least = t;
    }
  }
  return best;
}
// CTAs (of eight warps, or of half an SM's) to a segment: as many as the SMs hold and its tiles allow.
static int seg_ctas(int64_t segs, int64_t most, int sms) {
  int c = 1;
  while (c < 8 && segs * (2 * c) <= 2 * sms && most >= 8 * (2 * c)) c *= 2;
  return c;
}
// Segments of at most `most` tiles in CTAs of their own, or equal runs?  An SM takes about
// 0.125 us a tile; the first cost 4.2 us besides, at the bound's length on every SM, the
// second 8.9 (prefix, partial results, merge) at the true lengths.  Measured, g = 4, d = 128,
// segments / runs: 1 x 4096 tokens 6.4 / 8.5 us, 1 x 8192 8.5 / 9.7, 8 x 4096 9.2 / 13.1, 16 x 4096
// 12.8 / 16.5, 64 x 2048 18.6 / 26.2, 64 x 4096 31.3 / 38.0 (the one of these where the estimate
// takes the slower); ragged up to that length 8 x 4096 8.2 / 9.9, 64 x 2048 14.0 / 12.5, 64 x 4096
// 24.5 / 14.2.
static bool seg_better(int64_t segs, int64_t most, int ctas, int sms) {
  const int64_t on_sm = (segs * ctas + sms - 1) / sms;
  return 4.2 + 0.125 * most / ctas * on_sm < 8.9 + 0.125 * segs * most / sms;
}

template <int D, bool kFp16, bool kSel>
static cudaError_t run_decode4(const Kv4DecodeParams &p, cudaStream_t s) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const int sms = sm_count(dev), units = p.h_k * head_parts(p.g);
  // tiles that a segment has at most, as far as the host knows
  int64_t most = ((int64_t)p.width << p.page_log2) / kKv4Tile;
  if (p.window > 0) most = min(most, (int64_t)p.window / kKv4Tile + 2);
  if (kSel) most = min(most, (int64_t)p.topk << (p.page_log2 - 5));
  const int64_t segs = (int64_t)p.num_seqs * units;
  const int cluster = seg_ctas(segs, most, sms);
  if (kSel || seg_better(segs, most, cluster, sms)) {
    constexpr int kHalf = kSmWarps<D> / 2;
    if (segs * cluster <= sms) {                           // an SM for each CTA
      if (cluster == 1) return run_segs<D, kFp16, kSel, 8>(p, units, 1, s);
      return run_segs<D, kFp16, kSel, 8, true>(p, units, cluster, s);
    }
    if (cluster > 1) return run_segs<D, kFp16, kSel, kHalf, true>(p, units, cluster, s);
    const int warps = seg_warps<D>(segs, most, sms);
    if constexpr (D == 128) {
      if (warps == 3) return run_segs<D, kFp16, kSel, 3>(p, units, 1, s);
    }
    switch (warps) {
      case 1: return run_segs<D, kFp16, kSel, 1>(p, units, 1, s);
      case 2: return run_segs<D, kFp16, kSel, 2>(p, units, 1, s);
      case 4: return run_segs<D, kFp16, kSel, 4>(p, units, 1, s);
      default: return run_segs<D, kFp16, kSel, kHalf>(p, units, 1, s);
    }
  }
  const int ctas = min(sms * 2, kK4MaxCtas);               // resident at once
  auto *kernel = kv4_run_kernel<D, kFp16>;
  constexpr int threads = K4<D>::kRunThreads, smem = K4<D>::kRunWarps * K4<D>::kRing;
  e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  e = launch_kv4(kernel, dim3(ctas), threads, smem, 1, s, p, units);
  if (e != cudaSuccess) return e;
  return launch_kv4(kv4_merge_kernel<D, kFp16>, dim3(ctas, min(p.g, kK4Heads)), kMergeThreads, 0, 1,
                    s, p, units);
}

template <int D, bool kFp16>
static cudaError_t run_decode4_sel(const Kv4DecodeParams &p, cudaStream_t s) {
  return p.sel ? run_decode4<D, kFp16, true>(p, s) : run_decode4<D, kFp16, false>(p, s);
}

cudaError_t launch_kv4_decode(int d, bool fp16, const Kv4DecodeParams &p, cudaStream_t s) {
  if (d == 64) return fp16 ? run_decode4_sel<64, true>(p, s) : run_decode4_sel<64, false>(p, s);
  return fp16 ? run_decode4_sel<128, true>(p, s) : run_decode4_sel<128, false>(p, s);
}

}  // namespace nsa
