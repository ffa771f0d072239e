// Paged key/value cache: the metadata of one serving step, and the append.
//
// kda_cache_plan.  Sequence s with c cached tokens and t new ones owns the packed
// tokens cu[s] .. cu[s] + t - 1 at positions c .. c + t - 1, and takes the blocks
// ceil(c / B) .. ceil((c + t) / B) - 1 from the free list, behind the ones that the
// sequences before it take.  Both offsets are prefix sums over the sequences.  One
// launch: every thread block runs the (short) scan over all sequences itself and
// writes its own slice of the packed tokens, so nothing waits on another block and
// a prompt of any length is spread over the GPU.  The block that holds a cache
// block's first token writes the table entry.
//
// Bound by latency: a scan is two barriers behind the lengths' loads.  512 requests of one
// token take 3.7 us on the device, 64 prompts of up to 16384 tokens (524 k together) 6.8
// us, 0.7 TB/s of the 4.5 MB written.
#include "attn_common.cuh"

namespace kda {
namespace {

constexpr int kPlanThreads = 256;

__global__ void __launch_bounds__(kPlanThreads) cache_plan_kernel(const __grid_constant__ CachePlanLaunch p,
                                                                  int64_t slice) {
    griddep_wait();
    __shared__ int64_t scan_buf[kPlanThreads / 32];
    __shared__ int32_t s_cu[kPlanThreads + 1], s_cached[kPlanThreads];
    __shared__ int64_t s_first[kPlanThreads];
    const kda_cache_plan_args& a = p.a;
    const int tid = threadIdx.x;
    const int bs = a.block_size, shift = __ffs(bs) - 1;
    const int64_t t_lo = (int64_t)blockIdx.x * slice;
    const int64_t t_hi = t_lo + slice < a.max_tokens ? t_lo + slice : a.max_tokens;
    const int64_t cap = (int64_t)a.table_stride * bs;
    const int64_t begin = a.free_begin[0];
    int64_t tokens = 0, taken = 0;           // of the sequences before this chunk
    int chunk = 0;
    for (int32_t s0 = 0; s0 < a.n_seqs; s0 += kPlanThreads, ++chunk) {
        const bool mine = chunk % (int)gridDim.x == (int)blockIdx.x;
        const int32_t s = s0 + tid;
        int64_t c = 0, t = 0;
        bool bad = false;
        if (s < a.n_seqs) {
            c = a.cached_lens[s];
            t = a.new_lens[s];
            bad = c < 0 || t < 0;
            c = c < 0 ? 0 : c;
            t = t < 0 ? 0 : t;
            if (c > cap) c = cap, bad = true;
            if (c + t > cap) t = cap - c, bad = true;
        }
        int64_t total;
        int64_t incl = block_scan<kPlanThreads>(t, scan_buf, &total) + tokens;
        const int64_t excl = incl - t < a.max_tokens ? incl - t : a.max_tokens;
        if (incl > a.max_tokens) bad = true, incl = a.max_tokens;
        t = incl - excl;
        tokens += total;
        const int64_t have = (c + bs - 1) >> shift;
        const int64_t take = ((c + t + bs - 1) >> shift) - have;
        const int64_t first = block_scan<kPlanThreads>(take, scan_buf, &total) - take + taken + begin;
        taken += total;
        s_cu[tid] = (int32_t)excl;
        s_cached[tid] = (int32_t)c;
        s_first[tid] = first;
        if (tid == kPlanThreads - 1) s_cu[kPlanThreads] = (int32_t)incl;
        __syncthreads();
        if (mine && s < a.n_seqs) {
            if (bad) flag(p.status, KDA_DEV_BAD_SEQLENS);
            // blocks that the free list can give
            int64_t got = a.n_free - first;
            got = begin < 0 || got < 0 ? 0 : got < take ? got : take;
            int64_t kv = c + t;
            if (got < take) {
                flag(p.status, KDA_DEV_NO_BLOCKS);
                kv = (have + got) << shift;
            }
            a.kv_lens[s] = (int32_t)kv;
            a.cu_seqlens[s] = (int32_t)excl;
            if (s == a.n_seqs - 1) a.cu_seqlens[a.n_seqs] = (int32_t)incl;
        }
        // this block's packed tokens among the chunk's
        const int64_t lo = t_lo > s_cu[0] ? t_lo : s_cu[0];
        const int64_t hi = t_hi < s_cu[kPlanThreads] ? t_hi : s_cu[kPlanThreads];
        for (int64_t x = lo + tid; x < hi; x += kPlanThreads) {
            int i = 0;                       // the last sequence of the chunk that starts at or before x
#pragma unroll
            for (int step = kPlanThreads / 2; step > 0; step >>= 1)
                if (s_cu[i + step] <= x) i += step;
            const int32_t cached = s_cached[i];
            const int32_t pos = cached + (int32_t)(x - s_cu[i]);
            const int32_t j = pos >> shift, have_i = (cached + bs - 1) >> shift;
            int32_t* entry = a.block_table + (int64_t)(s0 + i) * a.table_stride + j;
            int32_t block = -1;
            bool none = false;               // the free list has ended (flagged with kv_lens)
            if (j >= have_i) {
                const int64_t f = s_first[i] + (j - have_i);
                none = begin < 0 || f >= a.n_free;
                if (!none) block = a.free_blocks[f];
            } else {
                block = *entry;
            }
            if (block < 0 || (int64_t)block >= a.n_blocks) {
                if (!none) flag(p.status, KDA_DEV_BAD_SLOT);
                block = -1;
            }
            if (j >= have_i && pos == j << shift) *entry = block;
            a.slot_map[x] = block < 0 ? -1 : (block << shift) + (pos & (bs - 1));
            a.positions[x] = pos;
        }
        __syncthreads();                     // before the next chunk rewrites the shared arrays
    }
    const int64_t total = tokens < a.max_tokens ? tokens : a.max_tokens;
    for (int64_t x = (t_lo > total ? t_lo : total) + tid; x < t_hi; x += kPlanThreads) {
        a.slot_map[x] = -1;
        a.positions[x] = -1;
    }
    if (blockIdx.x == 0 && tid == 0) {
        int64_t end = begin + taken;
        end = begin < 0 ? 0 : end < a.n_free ? end : a.n_free;
        if (begin > a.n_free) end = begin;
        a.free_end[0] = (int32_t)end;
        if (begin < 0 || begin > a.n_free) flag(p.status, KDA_DEV_NO_BLOCKS);
        if (a.n_seqs == 0) a.cu_seqlens[0] = 0;
    }
}

constexpr int kAppendThreads = 256;
constexpr int kAppendVecs = 4;

// Pure copy: 16-byte pieces, four in flight per thread.  A block takes whole tokens
// (k and v, all heads), as many as fill its threads' four pieces, at least one.  Bound by
// HBM: 32768 tokens of 8 heads, d = 128 in 43 us, 6.2 TB/s.
__global__ void __launch_bounds__(kAppendThreads) cache_append_kernel(const __grid_constant__ CacheAppendLaunch p,
                                                                      int32_t block_tokens) {
    griddep_wait();
    const int64_t t0 = (int64_t)blockIdx.x * block_tokens;
    const uint32_t row_vecs = (uint32_t)p.row_vecs, head_vecs = (uint32_t)p.head_vecs;
    const uint32_t n = 2 * row_vecs * (uint32_t)min((int64_t)block_tokens, p.n_tokens - t0);
    const uint32_t page = (uint32_t)p.block_size;
    const int64_t n_slots = p.n_blocks * p.block_size;
    for (uint32_t i0 = threadIdx.x; i0 < n; i0 += kAppendThreads * kAppendVecs) {
        float4 r[kAppendVecs];
        float4* dst[kAppendVecs];
#pragma unroll
        for (int m = 0; m < kAppendVecs; ++m) {
            const uint32_t i = i0 + m * kAppendThreads;
            dst[m] = nullptr;
            if (i >= n) continue;
            const uint32_t half = i / row_vecs, x = i - half * row_vecs;     // half: 2 * token, or that + 1 for v
            const int64_t t = t0 + (half >> 1);
            const bool is_v = half & 1;
            const int32_t slot = p.slot_map[t];
            if (slot < 0 || slot >= n_slots) {
                if (slot != -1) flag(p.status, KDA_DEV_BAD_SLOT);
                continue;
            }
            const uint32_t block = (uint32_t)slot / page, off = (uint32_t)slot - block * page;
            const uint32_t h = x / head_vecs, e = x - h * head_vecs;
            r[m] = __ldcs(static_cast<const float4*>(is_v ? p.v : p.k) + t * (is_v ? p.v_stride : p.k_stride) + x);
            dst[m] = static_cast<float4*>(is_v ? p.v_cache : p.k_cache) +
                     (((int64_t)block * p.n_kv_heads + h) * page + off) * head_vecs + e;
        }
#pragma unroll
        for (int m = 0; m < kAppendVecs; ++m)
            if (dst[m]) *dst[m] = r[m];
    }
}

}  // namespace

cudaError_t launch_cache_plan(const CachePlanLaunch& p, cudaStream_t s) {
    // slices of at least 256 tokens, at most about four blocks per SM
    int64_t slice = (p.a.max_tokens + 607) / 608;
    slice = (slice + kPlanThreads - 1) / kPlanThreads * kPlanThreads;
    slice = slice < kPlanThreads ? kPlanThreads : slice;
    const int64_t blocks = p.a.max_tokens > 0 ? (p.a.max_tokens + slice - 1) / slice : 1;
    note_launch();
    return launch_overlapped(cache_plan_kernel, dim3((unsigned)blocks), dim3(kPlanThreads), 0, s, p, slice);
}

cudaError_t launch_cache_append(const CacheAppendLaunch& p, cudaStream_t s) {
    const int32_t fit = kAppendThreads * kAppendVecs / (2 * p.row_vecs);
    // Few tokens are spread over the SMs, one to a block: 512 of 2 heads, d = 64 1.8 us, 3.2
    // us filled; 32768 of one head 5 us filled, 19 us one to a block.
    const int32_t block_tokens = fit > 1 && p.n_tokens > 2 * 152 * (int64_t)fit ? fit : 1;
    note_launch();
    return launch_overlapped(cache_append_kernel, dim3((unsigned)((p.n_tokens + block_tokens - 1) / block_tokens)),
                             dim3(kAppendThreads), 0, s, p, block_tokens);
}

}  // namespace kda
