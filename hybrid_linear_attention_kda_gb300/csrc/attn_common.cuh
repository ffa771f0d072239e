// Shared by the softmax-attention and paged-cache kernels (not part of the C ABI).
#pragma once

#include "kda_attention.h"
#include "kda_common.cuh"

namespace kda {

// Address of the current device's status word (api.cu).
kda_status_t device_status_word(uint32_t** out);

// Lets the next kernel of the stream be scheduled beside this one; it still waits
// in griddep_wait() for this grid to complete.
__device__ __forceinline__ void griddep_launch() { asm volatile("griddepcontrol.launch_dependents;"); }

// ------------------------------------------------------------------ block scan

// Inclusive scan of one value per thread over a block of NT threads; every thread
// gets its prefix sum and the block's total.  `buf` holds NT / 32 values.
template <int NT, typename V>
__device__ __forceinline__ V block_scan(V x, V* buf, V* total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const V y = __shfl_up_sync(0xffffffffu, x, off);
        if (lane >= off) x += y;
    }
    __syncthreads();                        // the previous scan's readers are done with buf
    if (lane == 31) buf[warp] = x;
    __syncthreads();
    V before = 0, all = 0;
#pragma unroll
    for (int w = 0; w < NT / 32; ++w) {
        const V t = buf[w];
        before += w < warp ? t : 0;
        all += t;
    }
    *total = all;
    return x + before;
}

// ------------------------------------------------------------------ row tiles

// Attention rows.  The query heads of one key/value head see the same keys, so a
// tile of rows takes whole tokens with all G of those heads: row r of a tile is
// (token r / G, head r % G).  A tile of R rows therefore covers R / G tokens, and
// a tile of keys is loaded once for all of its rows.  Works the same for a prompt
// (tokens of one sequence) and for a shared prefix (the members of one group, one
// query each).
struct RowTile {
    int32_t seq;      // sequence (or group); -1: no such tile
    int32_t t0;       // first token (or member) within it
    int32_t n;        // its tokens
    int64_t row0;     // packed row of its first token
};

// The idx-th tile of `tile_tokens` tokens over the sequences cu[0] .. cu[n_seqs].
// Tiles of one sequence come last first: the later ones see more keys.  Called by
// a whole block of NT threads; bad sequences have no tiles and are flagged by the
// caller that passes report.
template <int NT>
__device__ RowTile find_tile(const int32_t* cu, int32_t n_seqs, int64_t total_tokens, int32_t tile_tokens,
                             int64_t idx, bool report, uint32_t bit, uint32_t* status) {
    __shared__ int64_t scan_buf[NT / 32];
    __shared__ RowTile found;
    if (threadIdx.x == 0) found.seq = -1;
    int64_t base = 0;
    for (int32_t s0 = 0; s0 < n_seqs; s0 += NT) {
        const int32_t s = s0 + (int32_t)threadIdx.x;
        int64_t a = 0, b = 0;
        if (s < n_seqs) {
            a = cu[s];
            b = cu[s + 1];
            if (a < 0 || b < a || b > total_tokens) {
                if (report) flag(status, bit);
                b = a;
            }
        }
        const int64_t tiles = (b - a + tile_tokens - 1) / tile_tokens;
        int64_t total;
        const int64_t incl = block_scan<NT>(tiles, scan_buf, &total) + base;
        if (idx < incl && idx >= incl - tiles) {
            found.seq = s;
            found.t0 = (int32_t)(incl - 1 - idx) * tile_tokens;
            found.n = (int32_t)(b - a);
            found.row0 = a;
        }
        base += total;
        if (base > idx && !report) break;
    }
    __syncthreads();
    return found;
}

// ------------------------------------------------------------------ launches

struct AttnTileLaunch {
    kda_attn_prefill_args a;      // q, strides, caches, ...; cu_seqlens = group_start for a shared prefix
    uint32_t* status;
    const int32_t* prefix_lens;   // shared prefixes only: keys 0 .. prefix_lens[g] of the group's first row
    // Shared prefixes, and prompts where n_split > 1: the keys are cut into n_split blocks, with partial results in
    // part_o [n_split, total_tokens, H, d] (unnormalised) and part_ml [n_split, total_tokens, H] (m, l).
    int32_t n_split;
    float split_cost;             // shared prefixes: prefix_block_tiles
    float* part_o;
    float2* part_ml;
};

// A shared prefix's keys are cut into n_split blocks, or fewer of at least sqrt(keys *
// split_cost) keys.  A block's time is its keys', and each block is one more partial
// result to join for every row of the batch, so that the sum of the two is least for
// blocks of that many; split_cost goes with the rows (prefix_split_cost).
__host__ __device__ __forceinline__ uint32_t prefix_block_tiles(uint32_t keys, uint32_t tile, uint32_t n_split, float split_cost) {
    const uint32_t even = ((keys + tile - 1) / tile + n_split - 1) / n_split;
    const uint32_t least = (uint32_t)(sqrtf((float)keys * split_cost) / (float)tile);
    return even > least ? (even > 1 ? even : 1) : (least > 1 ? least : 1);
}

// Prompt attention, and the shared-prefix part of decode attention (prefix_lens set).
constexpr int kTileKeysF32 = 64, kTileKeysBf16 = 128;                    // keys of a tile
cudaError_t launch_attn_simt(const AttnTileLaunch& p, cudaStream_t s);   // fp32
cudaError_t launch_attn_tc(const AttnTileLaunch& p, cudaStream_t s);     // bf16
inline cudaError_t launch_attn_tile(const AttnTileLaunch& p, cudaStream_t s) {
    return p.a.dtype == KDA_BF16 ? launch_attn_tc(p, s) : launch_attn_simt(p, s);
}

// Decode attention (attn_decode.cuh describes the division of work).
struct AttnDecodeLaunch {
    kda_attn_decode_args a;
    uint32_t* status;
    int32_t n_pieces;             // workers of the suffix kernel
    int32_t n_split;              // key blocks of the prefix (0: no groups)
    int32_t prefix_tile;          // keys of a tile of the prefix kernel, which the blocks are made of
    float split_cost;             // prefix_block_tiles
    float* pre_o;                 // [n_split, n_seqs, H, d] the prefix's partial results
    float2* pre_ml;               // [n_split, n_seqs, H]
    float* part_o;                // [2 * n_pieces, rows, d]: a piece's first unit, its last unit
    float2* part_ml;              // [2 * n_pieces, rows]
    int4* open;                   // [n_pieces] the unit that begins in a piece and goes on
    int2* info;                   // [n_seqs] (shared positions, all positions), where there are groups
};
// Query heads of one unit: bf16 the rows of a product.  fp32: arithmetic on rows that are
// not there costs as much, so four where no more are needed (33 sequences of up to 2000
// tokens, 4 key/value heads: four query heads each 38 us, 45 us in units of eight).
constexpr int kDecodeRowsBf16 = 16;
constexpr int decode_rows(int dtype, int G) { return dtype == KDA_BF16 ? kDecodeRowsBf16 : G <= 4 ? 4 : 8; }
// Keys of a tile.
constexpr int decode_tile(int dtype, int d) { return dtype == KDA_BF16 ? 16 : 1024 / d; }
// Tiles of the shortest piece.  Pieces share the work of a few sequences, but every piece
// of a unit is one more partial result to join, one by one: units of a few tiles are given
// a worker each (4 sequences of up to 40 tokens: 10 us, 15 us with pieces of four), long
// ones pieces of four (one sequence of 4000: 19 us, 35 us with pieces of one).
__host__ __device__ constexpr int decode_least_tiles(int64_t unit_tiles) {
    return unit_tiles < 16 ? 1 : unit_tiles < 48 ? 2 : 4;
}
constexpr int kDecodeWarps = 8, kDecodePieces = kDecodeWarps * 152;   // workers: eight warps on each of 152 SMs
cudaError_t launch_decode_info(const AttnDecodeLaunch& p, cudaStream_t s);   // p.info, where there are groups
cudaError_t launch_decode_simt(const AttnDecodeLaunch& p, cudaStream_t s);   // fp32
cudaError_t launch_decode_mma(const AttnDecodeLaunch& p, cudaStream_t s);    // bf16

// Joins a split prompt's partial results into o and lse.  Rows that no sequence wrote are those whose part_ml
// still holds the bytes kUnwritten.
constexpr int kUnwritten = 0xFF;
cudaError_t launch_prompt_join(const AttnTileLaunch& p, cudaStream_t s);

struct CachePlanLaunch {
    kda_cache_plan_args a;
    uint32_t* status;
};
cudaError_t launch_cache_plan(const CachePlanLaunch& p, cudaStream_t s);

struct CacheAppendLaunch {
    int64_t n_tokens;
    int32_t n_kv_heads, row_vecs, head_vecs;   // 16-byte pieces of one token's heads, of one head
    const void *k, *v;
    int64_t k_stride, v_stride;                // 16-byte pieces
    const int32_t* slot_map;
    void *k_cache, *v_cache;
    int64_t n_blocks;
    int32_t block_size;
    uint32_t* status;
};
cudaError_t launch_cache_append(const CacheAppendLaunch& p, cudaStream_t s);

}  // namespace kda
