// Launches of the 4-bit cache (not part of the C ABI).
#pragma once

#include "attn_common.cuh"
#include "kda_cache_q4.h"

namespace kda {

constexpr int kQ4Group = 64;                                // channels that share a scale
__host__ __device__ constexpr int q4_code_bytes(int d) { return d / 2; }                  // of a head's vector
__host__ __device__ constexpr int q4_scale_bytes(int d) { return d / kQ4Group * 4; }

struct CacheAppendQ4Launch {
    kda_cache_append_q4_args a;
    uint32_t* status;
};
cudaError_t launch_append_q4(const CacheAppendQ4Launch& p, cudaStream_t s);

struct CacheUnpackQ4Launch {
    kda_cache_unpack_q4_args a;
    uint32_t* status;
};
cudaError_t launch_unpack_q4(const CacheUnpackQ4Launch& p, cudaStream_t s);

// Decode attention over the 4-bit cache; `base` as for the full-width cache, with its k_cache,
// v_cache and n_blocks those of the shared prefixes.
struct AttnDecodeQ4Launch {
    AttnDecodeLaunch base;
    kda_cache_q4 cache;
};
constexpr int kQ4Keys = 32;                                 // keys of a tile
// Products of eight columns a unit takes: one, or two where a key/value head's query heads do
// not fit in one (fp32: two columns a head).  One sequence of 2^20 tokens, 8 key/value heads: up to
// 8 query heads each 223 us, 338 us with two columns; 16 each 338 us, 420 us with one.
__host__ __device__ constexpr int q4_columns(int dtype, int G) { return G <= (dtype == KDA_BF16 ? 8 : 4) ? 1 : 2; }
__host__ __device__ constexpr int q4_rows(int dtype, int G) { return q4_columns(dtype, G) * (dtype == KDA_BF16 ? 8 : 4); }
__host__ __device__ constexpr int q4_warps(int columns) { return columns == 1 ? 12 : 8; }   // of a thread block, one an SM
// Places on the line of pieces that a unit takes beside its tiles: its q, its first maximum, its
// result and the prefix's part of that take a worker as long as some tiles do.  512 requests of up
// to 2048 tokens, 8 heads: 161 us without, 132 us with 2, 128 us with 4, 134 us with 8; behind
// shared prefixes 228, 194, 177 and 182 us.
constexpr int kQ4Pad = 4;
cudaError_t launch_decode_q4(const AttnDecodeQ4Launch& p, cudaStream_t s);

}  // namespace kda
