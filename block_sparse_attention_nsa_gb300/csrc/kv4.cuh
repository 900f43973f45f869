// kv4.cuh -- the 4-bit paged KV cache: record layout, launch parameters and small
// device helpers shared by pages.cu, kv4_rows.cu, kv4_decode.cu and kv4_api.cu.  The
// record is described in include/nsa_kv4.h.
#pragma once

#include "common.cuh"
#include "nsa_kv4.h"

namespace nsa {

constexpr int kMaxPlanSeqs = 16384;   // requests of one plan: their offsets stay in shared memory

struct PageParams {
  int num_seqs, page, width, num_pages, num_free, max_slots;
  const int32_t *ctx, *add;      // tokens cached, tokens brought (or start and count)
  const int32_t *free_pages, *free_head;
  int32_t *table;                // read; in a plan its new entries are written too
  int32_t *slots, *seq_out, *cu_out, *head_out;
  int32_t *status;               // may be null
};

// A (page, head) record: tiles of 32 tokens.
constexpr int kKv4Tile = 32;
template <int D>
struct Kv4Tile {
  static constexpr int kG = D / 64;                        // scale groups of a row
  static constexpr int kRow = D / 2;                       // bytes of a row's codes
  static constexpr int kV = kKv4Tile * kRow;               // offset of the V codes
  static constexpr int kPar = 2 * kV;                      // offset of the scales and zeros
  static constexpr int kArr = kKv4Tile * kG * 2;           // bytes of one of their four arrays
  static constexpr int kBytes = kPar + 4 * kArr;           // 32 * (D + D / 8)
};

struct Kv4RowParams {
  int n, h_k, num_pages, page_log2;
  const void *k, *v;                                 // append: read; strides in elements
  int64_t k_ts, k_hs, v_ts, v_hs;
  void *k_out, *v_out;                               // read: written
  const int32_t *slots;
  uint8_t *pool;
  int32_t *status;
};

struct Kv4DecodeParams {
  int num_seqs, h_q, h_k, g, num_pages, page_log2, width, topk, window;
  float scale;
  const void *q;
  const uint8_t *pool;
  const int32_t *table, *lens, *sel;                 // sel null: every block
  void *out;
  float *lse;
  int32_t *status;
  void *ws;
};

// Two fp32 operations in one instruction, each rounded to nearest.
struct Pair {
  unsigned long long v;
  __device__ __forceinline__ Pair() {}
  __device__ __forceinline__ Pair(float a, float b) {
    asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "f"(a), "f"(b));
  }
  __device__ __forceinline__ float2 get() const {
    float2 f;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(f.x), "=f"(f.y) : "l"(v));
    return f;
  }
};
__device__ __forceinline__ Pair operator+(Pair a, Pair b) {
  Pair d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d.v) : "l"(a.v), "l"(b.v));
  return d;
}
__device__ __forceinline__ Pair operator*(Pair a, Pair b) {
  Pair d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d.v) : "l"(a.v), "l"(b.v));
  return d;
}
__device__ __forceinline__ Pair fma(Pair a, Pair b, Pair c) {
  Pair d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d.v) : "l"(a.v), "l"(b.v), "l"(c.v));
  return d;
}

__device__ __forceinline__ void raise(int32_t *status, int32_t bits) {
  if (status) set_status(status, bits);
}

// Kernels of this group start while the one before them on the stream still runs (their
// launch overlaps its end) and touch no memory before it has finished.  They read with plain loads:
// what a read-only load (ld.global.nc, __ldg) takes must not change while the kernel runs, which
// for these began with the writer's end still to come, and the compiler may move one ahead of the wait.
__device__ __forceinline__ void after_previous() {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
}
template <typename... P, typename... A>
inline cudaError_t launch_kv4(void (*kernel)(P...), dim3 grid, int threads, size_t smem, int cluster,
                              cudaStream_t s, A... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(static_cast<unsigned>(threads));
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  at[1].id = cudaLaunchAttributeClusterDimension;
  at[1].val.clusterDim.x = static_cast<unsigned>(cluster);
  at[1].val.clusterDim.y = 1;
  at[1].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

cudaError_t launch_pages(const PageParams &p, bool plan, cudaStream_t s);
cudaError_t launch_kv4_append(int d, bool fp16, const Kv4RowParams &p, cudaStream_t s);
cudaError_t launch_kv4_read(int d, bool fp16, const Kv4RowParams &p, cudaStream_t s);
size_t kv4_decode_workspace(int d, int g, bool selected);
int64_t kv4_decode_tiles(const Kv4DecodeParams &p);
cudaError_t launch_kv4_decode(int d, bool fp16, const Kv4DecodeParams &p, cudaStream_t s);

}  // namespace nsa
