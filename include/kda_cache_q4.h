/*
 * kda_cache_q4.h -- a paged key/value cache held in 4 bits, in libkda.so.
 *
 * The softmax-attention layers' cache (kda_attention.h) at 4.5 bits a channel
 * instead of 16 or 32: decode attention is bound by reading its cache.
 *   kda_cache_append_q4  the step's new keys and values into the cache;
 *   kda_cache_unpack_q4  cached positions back into a full-width paged cache, for
 *                        a prompt that resumes behind them (kda_attn_prefill);
 *   kda_attn_decode_q4   decode attention over the cache, behind full-width
 *                        prefixes that groups of requests share.
 * The cache metadata is kda_cache_plan's, as for the full-width cache.
 *
 * Layout.  Of keys and of values: codes [n_blocks, H_kv, block_size, d / 2] bytes,
 * channel 2 i in the low half of byte i, 2 i + 1 in the high half; scales [n_blocks,
 * H_kv, block_size, d / 64, 2] bf16, the pair (s, m) for each group of 64 channels.
 * A channel's value is m + code * s.
 *
 * Codes of a group x, in fp32 arithmetic, rounded to nearest unless it says
 * otherwise:  m = min x, rounded down to bf16;  s = (max x - m) / 15, rounded up to
 * bf16;  code = (x - m) / s, rounded to the nearest integer, ties to even, and cut
 * to 0 .. 15 (0 where s is 0).  So x and its value are at most half a step of s
 * apart, and the roundings (m + 15 s, which can be above max x by these, is infinite
 * where it passes the type's largest number).  A group that holds an infinity or
 * NaN, or whose width or bounds leave the range of fp32 or bf16, gets s = 0 and m =
 * NaN: all of it reads as NaN.
 *
 * Conventions: those of kda.h and kda_attention.h.  All four tensors are 16-byte
 * aligned, and n_blocks * block_size * H_kv <= 2^31 - 1.
 */
#ifndef KDA_CACHE_Q4_H
#define KDA_CACHE_Q4_H

#include "kda_attention.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef struct kda_cache_q4 {
    void *k_codes, *k_scales, *v_codes, *v_scales;
    int64_t n_blocks;
    int32_t block_size;
    int32_t reserved0;          /* must be 0 */
} kda_cache_q4;

/*
 * The tokens' keys and values to their slots.  k_out and v_out (or NULL) receive
 * the values that the cache now stands for, rounded to the element type: what a
 * prompt's own attention sees if it is to see what later steps will.  They may be
 * k and v (with the same stride), and overlap nothing else.  A slot of -1 skips
 * the token; another slot outside the cache skips it too and sets
 * KDA_DEV_BAD_SLOT.  The slots must be distinct.
 */
typedef struct kda_cache_append_q4_args {
    int64_t n_tokens;
    int32_t n_kv_heads, d;
    int32_t dtype;              /* kda_dtype_t of k, v and the outputs */
    int32_t reserved0;          /* must be 0 */
    int64_t k_stride, v_stride, k_out_stride, v_out_stride;
    const void *k, *v;
    void *k_out, *v_out;        /* or NULL */
    const int32_t *slot_map;    /* [n_tokens] */
    kda_cache_q4 cache;
} kda_cache_append_q4_args;

kda_status_t kda_cache_append_q4(const kda_cache_append_q4_args *args, void *stream);

/*
 * Positions first[s] .. kv_lens[s] - 1 of each sequence (from 0 where first is
 * NULL) out of the 4-bit cache, by block_table, into the full-width cache
 * k_cache, v_cache [n_blocks, H_kv, block_size, d], by to_table, each value
 * rounded once to the element type.  Nothing else of that cache is written; the
 * rows of to_table must not share a block among the positions that are written.
 *
 * Device-visible errors: a kv_len outside [0, block_size * the shorter table row]
 * or a negative first sets KDA_DEV_BAD_SEQLENS and skips the sequence; an entry of
 * either table outside its cache sets KDA_DEV_BAD_SLOT and skips its positions.
 */
typedef struct kda_cache_unpack_q4_args {
    int32_t n_seqs;
    int32_t n_kv_heads, d;
    int32_t dtype;              /* kda_dtype_t of k_cache and v_cache */
    kda_cache_q4 cache;
    const int32_t *block_table; /* [n_seqs, table_stride] */
    const int32_t *to_table;    /* [n_seqs, to_stride] */
    int32_t table_stride, to_stride;
    const int32_t *first;       /* [n_seqs] or NULL */
    const int32_t *kv_lens;     /* [n_seqs] */
    void *k_cache, *v_cache;
    int64_t n_blocks;           /* of k_cache and v_cache */
} kda_cache_unpack_q4_args;

kda_status_t kda_cache_unpack_q4(const kda_cache_unpack_q4_args *args, void *stream);

/*
 * kda_attn_decode over a cache in 4 bits.  `base` is its argument block, with the
 * same meaning but for two things:
 *  - positions are read from `cache` (whose block_size must be base.block_size);
 *  - with groups, a group's shared positions lie in the full-width cache
 *    base.k_cache, base.v_cache (of base.n_blocks blocks), and the table's entries
 *    of those positions are blocks of that cache: a shared prompt is kept once, at
 *    full width, and read once a group, while each request's own tokens are in 4
 *    bits.  Without groups the three are ignored.
 * q and o are of base.dtype.  The keys' scores are the exact products of the codes
 * with q, accumulated in fp32, for |q| up to 2^100 and scores up to 2^27 as there.
 * bf16 q is held exactly and fp32 q in two 11-bit parts: a channel to 2^-35 (fp32:
 * 2^-39) of the largest of its 64, if that is coarser.  A weight times its value's
 * scale is held in fp16 (fp32: in two such parts) for the product with the codes:
 * 11 bits (22), or multiples of 2^-30 of the largest one so far of its head and
 * group, if those are coarser, so that values of any size may stand beside each
 * other.  The weights' sum is taken before that rounding.  Positions that a mask
 * hides never reach a result, whatever their codes and scales are.  A position
 * that is NaN makes its key group's heads NaN, or its value group's channels.
 */
typedef struct kda_attn_decode_q4_args {
    kda_attn_decode_args base;
    kda_cache_q4 cache;
} kda_attn_decode_q4_args;

/* Bytes of workspace for these sizes (those that kda_attn_decode_workspace_size
 * reads); 0 for an empty batch or invalid sizes. */
size_t kda_attn_decode_q4_workspace_size(const kda_attn_decode_q4_args *args);

kda_status_t kda_attn_decode_q4(const kda_attn_decode_q4_args *args, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* KDA_CACHE_Q4_H */
