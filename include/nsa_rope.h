/*
 * nsa_rope.h -- C ABI of rotary positions for queries and keys, and their gradient.
 *
 * Conventions are those of nsa_sel_attn.h: device pointers owned by the caller, calls
 * asynchronous on `stream`, arguments checked before anything is enqueued, no device
 * memory allocated, nothing aborts.
 *
 * A token at position n turns pair i of its head's first rot_dim dimensions, (x, y), by the
 * angle a = n w_i, and scales it:
 *     x' = mscale (x cos a - y sin a),   y' = mscale (y cos a + x sin a),   i = 0 ... rot_dim / 2 - 1.
 * The pair is dimensions (i, i + rot_dim / 2), or (2 i, 2 i + 1) where `interleaved` is set; the
 * dimensions from rot_dim on are copied.  w_i is held as the part of a turn that one position
 * advances, in units of 2^-64: n times it, modulo 2^64, is the angle of any position that 32 bits
 * hold, without a table.  The frequency is computed in double, so that an angle is off by about
 * n w_i 2^-52: below fp32's own 2^-24 of a radian up to positions of 2^28, eight times that at 2^31 (of the
 * first pair, w_0 = 1).  Angles, sines and products are fp32; results are rounded once.
 * The gradient of a rotation is the rotation back (by -a), scaled by the same factor.
 */
#ifndef NSA_ROPE_H
#define NSA_ROPE_H

#include "nsa_sel_attn.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Frequencies w_i = base^(-2 i / rot_dim), and what a longer context makes of them. */
typedef enum {
    NSA_ROPE_PLAIN = 0,
    NSA_ROPE_LINEAR = 1,  /* w_i / factor (position interpolation: Chen et al., 2023) */
    NSA_ROPE_BASE = 2,    /* base * factor^(rot_dim / (rot_dim - 2)) in the place of base */
    NSA_ROPE_RAMP = 3     /* by parts (YaRN: Peng et al., 2023): with r = trained * w_i / (2 pi), the
                             turns of pair i over the trained length, and c = (r - low) / (high - low)
                             held to 0 ... 1:  w_i (c + (1 - c) / factor).  The factor that goes with
                             it, 0.1 ln(factor) + 1 on q and k, is mscale's. */
} nsa_rope_scaling;

/* Writes the rot_dim / 2 frequencies, in 2^-64 of a turn per position, to HOST memory (host only,
 * no CUDA call); the caller copies them to the device once.  base > 0, factor > 0, both finite;
 * trained > 0 and low < high for NSA_ROPE_RAMP, ignored otherwise; rot_dim >= 4 for NSA_ROPE_BASE. */
NSA_API nsa_status nsa_rope_freqs(int32_t rot_dim, double base, int32_t scaling, double factor,
                                  double trained, double low, double high, uint64_t *host_freqs);

typedef struct {
    int32_t num_tokens;  /* N rows of q and k, 0 allowed */
    int32_t h_q, h_k;    /* heads; one of them may be 0 (that tensor's pointers are then ignored) */
    int32_t head_dim;    /* a multiple of 8, at most 512 */
    int32_t rot_dim;     /* a multiple of 16, at most head_dim */
    int32_t interleaved; /* 0: pairs (i, i + rot_dim / 2); 1: pairs (2 i, 2 i + 1) */
    int32_t num_seqs;    /* S: sequences of cu_seqlens; 0 with `positions` */
    int32_t dtype;       /* nsa_dtype of q, k and the outputs */
} nsa_rope_dims;

/* q and k to q_out and k_out: [N, heads, head_dim] each, with a stride in elements from token to token
 * and one from head to head (multiples of 8), the last dimension contiguous, the pointer 16-byte
 * aligned.  An output may be its own input (the same pointer and strides); apart
 * from that outputs overlap neither inputs nor each other, nor do an output's own rows.
 * Positions: positions[t], int32 [N] (negative ones turn backwards); or, where it is NULL, those
 * of a packed batch: cu_seqlens int32 [num_seqs + 1], token t of sequence s has position
 * start[s] + t - cu_seqlens[s] (start int32 [num_seqs], NULL: 0).  Rows from cu_seqlens[num_seqs] on
 * are left as they are.  So are rows that a cu_seqlens that decreases or begins above 0 gives to no
 * sequence, which sets NSA_DEVERR_BAD_SEQLENS in *device_status (may be NULL).
 * freqs: uint64 [rot_dim / 2], as nsa_rope_freqs makes them, 8-byte aligned.  mscale is finite.
 * num_tokens * (h_q + h_k) has to stay below 2^31. */
NSA_API nsa_status nsa_rope(const nsa_rope_dims *dims, const void *q, int64_t q_token_stride,
                            int64_t q_head_stride, const void *k, int64_t k_token_stride,
                            int64_t k_head_stride, const uint64_t *freqs, const int32_t *positions,
                            const int32_t *cu_seqlens, const int32_t *start, float mscale,
                            void *q_out, int64_t q_out_token_stride, int64_t q_out_head_stride,
                            void *k_out, int64_t k_out_token_stride, int64_t k_out_head_stride,
                            int32_t *device_status, nsa_stream_t stream);

/* The gradient: from the gradients of q_out and k_out to those of q and k, the same rules. */
NSA_API nsa_status nsa_rope_bwd(const nsa_rope_dims *dims, const void *dq_out,
                                int64_t dq_out_token_stride, int64_t dq_out_head_stride,
                                const void *dk_out, int64_t dk_out_token_stride,
                                int64_t dk_out_head_stride, const uint64_t *freqs,
                                const int32_t *positions, const int32_t *cu_seqlens,
                                const int32_t *start, float mscale, void *dq,
                                int64_t dq_token_stride, int64_t dq_head_stride, void *dk,
                                int64_t dk_token_stride, int64_t dk_head_stride,
                                int32_t *device_status, nsa_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* NSA_ROPE_H */
