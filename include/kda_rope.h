/*
 * kda_rope.h -- norms and position rotation of queries and keys, in libkda.so.
 *
 * Between the projections and the attention of a softmax-attention layer
 * (kda_attention.h), queries and keys are normed head by head and rotated by
 * their positions.  Two calls do this in one pass over the tensors:
 *   kda_qk_norm_rope       queries and keys to tensors, or in place;
 *   kda_cache_append_rope  keys on their way into the paged cache, beside their
 *                          values, and (optionally) the queries to a tensor: all
 *                          that a serving step does between the projection and
 *                          the attention, in one launch.
 *
 * For a head's vector x, with its weight w and its token's position p:
 *     y = w x / sqrt(mean_c x_c^2 + eps)               (y = x where w is NULL)
 *     (a, b) -> (a cos t - b sin t, a sin t + b cos t),  t = 2 pi frac(p F_i / 2^64)
 * for the pairs i < rot_dim / 2 of the first rot_dim channels: channels i and
 * i + rot_dim / 2, or 2 i and 2 i + 1 where interleaved is set; the others are y.
 * All of it in fp32, rounded once to the element type; the squares are fp32's too,
 * so that a norm is for |x| below 2^60 (and above 2^-60, where eps is 0).  F_i = turns[i] is the
 * frequency in turns a position, as a 64-bit fraction of one turn: p F_i wraps
 * around a turn exactly, so that far positions are as precise as near ones.  A
 * frequency of f radians a position is F = round(f / (2 pi) * 2^64) modulo 2^64.
 *
 * Conventions: those of kda.h and kda_attention.h (q [T, H, d]; k, v [T, H_kv, d],
 * a token's heads dense, tokens *_stride elements apart).  H and H_kv need not
 * divide each other here.  A position of -1 skips its token: nothing of it is
 * read or written.  Another negative one does too, and sets KDA_DEV_BAD_POSITION.
 *
 * q_out may be q and k_out k (with the same stride); outputs may not overlap
 * anything else that a call reads or writes.
 */
#ifndef KDA_ROPE_H
#define KDA_ROPE_H

#include "kda_attention.h"

#ifdef __cplusplus
extern "C" {
#endif

/* A further bit of the device status word. */
#define KDA_DEV_BAD_POSITION 0x100u /* a position below -1 */

typedef struct kda_qk_rope_args {
    int64_t n_tokens;
    int32_t n_heads, n_kv_heads, d;
    int32_t dtype;             /* kda_dtype_t of q, k, v, the outputs and the cache */
    int32_t rot_dim;           /* 0 .. d, a multiple of 8 */
    int32_t interleaved;       /* 0: pairs (i, i + rot_dim / 2); 1: pairs (2 i, 2 i + 1) */
    float eps;                 /* finite, >= 0 */
    int32_t reserved0;         /* must be 0 */
    int64_t q_stride, k_stride, q_out_stride, k_out_stride;
    const void *q, *k;
    void *q_out, *k_out;
    const float *q_weight;     /* [d] or NULL (no norm), 16-byte aligned */
    const float *k_weight;
    const uint64_t *turns;     /* [rot_dim / 2], 16-byte aligned */
    const int32_t *positions;  /* [n_tokens] */
} kda_qk_rope_args;

kda_status_t kda_qk_norm_rope(const kda_qk_rope_args *args, void *stream);

/*
 * The same for queries, keys and values on their way into the paged cache: k goes
 * to k_cache[slot_map[t]], v is copied to v_cache[slot_map[t]].  k_out and
 * k_out_stride are ignored.  Without queries: n_heads = 0, q, q_out and q_weight
 * NULL.  A slot of -1 skips the token's key and value; another slot outside the
 * cache skips them too and sets KDA_DEV_BAD_SLOT.  The slots must be distinct.
 */
typedef struct kda_cache_append_rope_args {
    kda_qk_rope_args qk;
    const void *v;
    int64_t v_stride;
    const int32_t *slot_map;   /* [n_tokens] */
    void *k_cache, *v_cache;   /* [n_blocks, H_kv, block_size, d] */
    int64_t n_blocks;
    int32_t block_size;
    int32_t reserved0;         /* must be 0 */
} kda_cache_append_rope_args;

kda_status_t kda_cache_append_rope(const kda_cache_append_rope_args *args, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* KDA_ROPE_H */
