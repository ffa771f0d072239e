// Launch of the norm and rotation kernels (not part of the C ABI).
#pragma once

#include "kda_common.cuh"
#include "kda_rope.h"

namespace kda {

struct RopeLaunch {
    kda_qk_rope_args a;
    bool append;                 // into the paged cache: the rest is set
    const void* v;
    int64_t v_stride;
    const int32_t* slot_map;
    void *k_cache, *v_cache;
    int64_t n_blocks;
    int32_t block_size;
    uint32_t* status;
};
cudaError_t launch_rope(const RopeLaunch& p, cudaStream_t s);

}  // namespace kda
