/*
 * kda_attention.h -- the softmax-attention layers of a hybrid stack, in libkda.so.
 *
 * A hybrid stack interleaves KDA layers with full-attention layers whose cache
 * grows with every token ("Kimi K3 Tech Intro", sections 1 and 2.1: one manager
 * for the paged key/value blocks and the KDA states).  The calls here are the
 * full-attention layers' share of a serving step:
 *   kda_cache_plan      block tables, slot map and positions of one step, from
 *                       the requests' lengths, on the GPU;
 *   kda_cache_append    the step's new keys and values into the paged cache;
 *   kda_attn_prefill    causal attention over a packed batch of prompts, with
 *                       keys and values from packed tensors or from the cache;
 *   kda_attn_decode     one query token per request over the cache, with the
 *                       prefix that a group of requests shares read once.
 *
 * Conventions: those of kda.h (device pointers, the caller's buffers,
 * asynchronous on `stream`, host-visible errors before any launch, device-visible
 * ones in the status word).  q, k, v, o and the caches are 16-byte aligned; int32
 * arrays and lse need 4 bytes.  In addition:
 *  - q, o [T, H, d]; k, v [T, H_kv, d]; H a multiple of H_kv, and query head h
 *    reads key/value head h / (H / H_kv).  d in {64, 128}; H / H_kv <= 128.
 *  - The heads of one token are dense; consecutive tokens are *_stride elements
 *    apart, so that q, k and v may be slices of one fused projection's output.
 *    A stride is a multiple of 16 bytes and at least the token's own heads * d.
 *  - k_cache, v_cache [n_blocks, H_kv, block_size, d], dense; block_size in {16,
 *    32, 64, 128, 256}.  Slot number = block * block_size + offset in the block;
 *    n_blocks * block_size * H_kv <= 2^31 - 1 (the elements may exceed 2^32).
 *  - block_table [n_seqs, table_stride] int32: entry j of row s is the block of
 *    positions j * block_size .. of sequence s.  Entries past a sequence's length
 *    are not read.
 *  - q, k, v, o and the caches share one element type.  bf16: products on the
 *    tensor cores with fp32 accumulation, the softmax in fp32, its weights
 *    rounded to bf16 for the product with v (their sum is taken before that
 *    rounding), for scores |scale * q . k| up to 2^27.  fp32: fp32 throughout.
 *  - Positions that a mask hides never reach a result, whatever they hold: NaN
 *    or infinities in later tokens, other sequences, or the unwritten tail of a
 *    block change nothing.  A query row that sees no key gives zeros, and -inf
 *    as its log-sum-exp.
 *  - lse [T, H] fp32 (or NULL) receives the natural logarithm of the sum of
 *    exp(scale * q . k) over the keys that a row sees.
 *  - Results do not depend on the order in which thread blocks run.
 */
#ifndef KDA_ATTENTION_H
#define KDA_ATTENTION_H

#include "kda.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Further bits of the device status word. */
#define KDA_DEV_NO_BLOCKS 0x40u /* kda_cache_plan: the free list ran out */
#define KDA_DEV_BAD_GROUP 0x80u /* kda_attn_decode: a bad group or prefix length */

/*
 * The cache metadata of one step.  Sequence s holds cached_lens[s] tokens and
 * appends new_lens[s] (zero is allowed in both).  In order of s, each sequence
 * takes the blocks that its new tokens begin (those whose first position is a
 * new one) from free_blocks[*free_begin], free_blocks[*free_begin + 1], ... and
 * *free_end becomes the index after the last one taken.  Written:
 *   block_table[s][j]  the new entries; the others are left as they are;
 *   kv_lens[s]         cached_lens[s] + new_lens[s];
 *   cu_seqlens[s]      packed offset of s's new tokens (n_seqs + 1 entries);
 *   slot_map[t]        the cache slot of packed token t;
 *   positions[t]       its position in its sequence;
 * and slot_map[t] = positions[t] = -1 from the batch's last token up to
 * max_tokens, so that the call can be replayed at a fixed size.
 *
 * free_begin and free_end are single device integers and may not be the same
 * one.  No output may overlap an input (the lengths, free_blocks, free_begin):
 * thread blocks read all of these while others write.  Lengths are advanced by a
 * copy of kv_lens behind the call.
 *
 * Device-visible errors.  A negative length counts as zero, and a length past
 * table_stride * block_size is cut there (KDA_DEV_BAD_SEQLENS); so are tokens
 * past max_tokens, with the later cu_seqlens entries at max_tokens.  Where the
 * free list ends, the table entries and the slots of their tokens become -1 and
 * kv_lens[s] stops at the first position without a block (KDA_DEV_NO_BLOCKS).
 * A free or table entry that names a block outside the cache gives slots of -1
 * (KDA_DEV_BAD_SLOT).
 */
typedef struct kda_cache_plan_args {
    int32_t n_seqs;             /* >= 0 */
    int32_t block_size;
    int32_t table_stride;       /* entries per row of block_table, >= 1 */
    int32_t n_free;             /* entries of free_blocks */
    int64_t n_blocks;           /* blocks in the cache */
    int64_t max_tokens;         /* entries of slot_map and positions */
    const int32_t *cached_lens; /* [n_seqs] */
    const int32_t *new_lens;    /* [n_seqs] */
    const int32_t *free_blocks; /* [n_free] */
    const int32_t *free_begin;  /* [1] */
    int32_t *free_end;          /* [1] */
    int32_t *block_table;       /* [n_seqs, table_stride], read and written */
    int32_t *kv_lens;           /* [n_seqs] */
    int32_t *cu_seqlens;        /* [n_seqs + 1] */
    int32_t *slot_map;          /* [max_tokens] */
    int32_t *positions;         /* [max_tokens] */
} kda_cache_plan_args;

kda_status_t kda_cache_plan(const kda_cache_plan_args *args, void *stream);

/*
 * k_cache[slot_map[t]] = k[t] and v_cache[slot_map[t]] = v[t] for t in [0,
 * n_tokens), all H_kv heads; bit-exact.  A slot of -1 skips the token; another
 * slot outside the cache skips it too and sets KDA_DEV_BAD_SLOT.  The slots must
 * be distinct.
 */
kda_status_t kda_cache_append(int64_t n_tokens, int32_t n_kv_heads, int32_t d, int32_t dtype,
                              const void *k, int64_t k_stride, const void *v, int64_t v_stride,
                              const int32_t *slot_map, void *k_cache, void *v_cache, int64_t n_blocks,
                              int32_t block_size, void *stream);

/*
 * Causal attention over a packed batch.  Sequence s owns the query tokens
 * cu_seqlens[s] .. cu_seqlens[s + 1] - 1; they are the last ones of its K_s
 * positions, so query i sees the keys j <= K_s - (its query count) + i.
 *  - block_table == NULL: K_s is its query count, and the keys and values are the
 *    same rows of the packed k and v.
 *  - block_table != NULL: K_s = kv_lens[s], and all keys and values (the new
 *    tokens' too) are in the cache: kda_cache_append comes first.  This is how a
 *    prompt resumes behind a cached prefix.  k and v are ignored.  A sequence
 *    with more queries than positions has rows that see nothing.
 * Tokens from cu_seqlens[n_seqs] on get no output.  A decreasing cu_seqlens or
 * one past total_tokens, or a kv_len outside [0, table_stride * block_size], sets
 * KDA_DEV_BAD_SEQLENS and skips the sequence; a table entry outside the cache
 * sets KDA_DEV_BAD_SLOT, and that sequence's outputs are unspecified.
 *
 * Where the rows are too many to be cut, one thread block walks all keys of its rows,
 * and its waits run out after about a second: in bf16 that is some 2^26 keys, beyond
 * which KDA_DEV_WAIT_TIMEOUT is set and outputs are unspecified.  The same holds for
 * a shared prefix of kda_attn_decode that is not cut.
 */
typedef struct kda_attn_prefill_args {
    int32_t n_seqs;
    int32_t n_heads, n_kv_heads, d;
    int32_t dtype;             /* kda_dtype_t */
    float scale;               /* usually d^-0.5; finite */
    int64_t total_tokens;      /* rows of q, o (and k, v) */
    int64_t q_stride, k_stride, v_stride, o_stride; /* elements between tokens */
    const void *q, *k, *v;
    void *o;
    float *lse;                /* [total_tokens, H] or NULL */
    const int32_t *cu_seqlens; /* [n_seqs + 1] */
    const void *k_cache, *v_cache;
    const int32_t *block_table;
    const int32_t *kv_lens;
    int64_t n_blocks;
    int32_t block_size;
    int32_t table_stride;
    void *workspace;           /* 256-byte aligned, or NULL */
    size_t workspace_bytes;
} kda_attn_prefill_args;

/* Bytes of workspace with which kda_attn_prefill cuts the keys of few rows into
 * blocks that run side by side (only the sizes and whether block_table is NULL are
 * read); 0 where it would not, and for invalid sizes.  The workspace is optional:
 * with none, or a smaller one, every row's keys are walked by one thread block. */
size_t kda_attn_prefill_workspace_size(const kda_attn_prefill_args *args);

kda_status_t kda_attn_prefill(const kda_attn_prefill_args *args, void *stream);

/*
 * Decode attention: one query token for each sequence, over its kv_lens[s] cached
 * positions (its own new token included, so kda_cache_append comes first).
 *
 * Shared prefixes: group g holds the sequences group_start[g] ..
 * group_start[g + 1] - 1, whose first prefix_lens[g] positions (a multiple of
 * block_size) lie in the same blocks.  Those blocks are taken from the group's
 * first row of the table and read once for all of its queries.  group_start[0]
 * must be 0 and group_start[n_groups] n_seqs.  n_groups == 0: nothing is shared.
 * A group of one sequence, or a prefix of 0, is fine.
 *
 * workspace: kda_attn_decode_workspace_size bytes, for the partial results of
 * rows whose keys are split over thread blocks.
 *
 * Device-visible errors: a kv_len outside [0, table_stride * block_size] sets
 * KDA_DEV_BAD_SEQLENS and counts as 0; group bounds that decrease, leave [0,
 * n_seqs] or miss its ends, a prefix that is negative, no multiple of
 * block_size or longer than one of its members set KDA_DEV_BAD_GROUP, and the
 * outputs of that group are unspecified; a table entry outside the cache sets
 * KDA_DEV_BAD_SLOT, and the outputs of the sequences that use it are
 * unspecified.
 */
typedef struct kda_attn_decode_args {
    int32_t n_seqs;
    int32_t n_heads, n_kv_heads, d;
    int32_t dtype;
    float scale;
    int64_t q_stride, o_stride;
    const void *q;
    void *o;
    float *lse;                 /* [n_seqs, H] or NULL */
    const void *k_cache, *v_cache;
    const int32_t *block_table;
    const int32_t *kv_lens;
    int64_t n_blocks;
    int32_t block_size;
    int32_t table_stride;
    int32_t n_groups;
    int32_t reserved0;          /* must be 0 */
    const int32_t *group_start; /* [n_groups + 1] or NULL */
    const int32_t *prefix_lens; /* [n_groups] or NULL */
    void *workspace;            /* 256-byte aligned */
    size_t workspace_bytes;
} kda_attn_decode_args;

/* Bytes of workspace for these sizes (only n_seqs, n_heads, n_kv_heads, d, dtype,
 * n_groups, block_size and table_stride are read); 0 for an empty batch or invalid
 * sizes. */
size_t kda_attn_decode_workspace_size(const kda_attn_decode_args *args);

kda_status_t kda_attn_decode(const kda_attn_decode_args *args, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* KDA_ATTENTION_H */
