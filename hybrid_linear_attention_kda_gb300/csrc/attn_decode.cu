// Decode attention over the paged cache for fp32 tensors, and the sequences' shared
// positions.  The division of work is described in attn_decode.cuh.  As in the bf16
// kernel a warp is a worker of its own, with a unit of four or eight query heads, a
// ring of asynchronous copies and no barrier; the products are SIMT: two or four
// lanes share a key's dot products, then every lane owns columns of the output.
//
// Bound by the cache's bytes up to two query heads a key/value head, and by arithmetic
// from four on: 33 sequences of up to 2000 tokens, 4 key/value heads, d = 128 take 33 us
// with one query head each (4 TB/s), 38 us with four, 50 us with eight; 64 sequences of
// 8192, 8/8 or 32/8 heads 0.64 ms (6.7 TB/s).
#include "async_copy.cuh"
#include "attn_decode.cuh"

namespace kda {
namespace {
using namespace decode;

// ------------------------------------------------------------------ shared positions

constexpr int kInfoThreads = 256;

// Group of sequence s (-1 when it is in none), by bisection of group_start.
__device__ int32_t group_of(const int32_t* start, int32_t n_groups, int32_t s) {
    int32_t lo = 0, hi = n_groups;               // the last g with start[g] <= s
    while (hi - lo > 1) {
        const int32_t mid = (lo + hi) / 2;
        if (start[mid] <= s) lo = mid;
        else hi = mid;
    }
    return n_groups > 0 && start[lo] <= s && s < start[lo + 1] ? lo : -1;
}

__global__ void __launch_bounds__(kInfoThreads) decode_info_kernel(const __grid_constant__ AttnDecodeLaunch p) {
    griddep_wait();
    griddep_launch();
    const kda_attn_decode_args& a = p.a;
    const int64_t cap = (int64_t)a.table_stride * a.block_size;
    const int32_t x = (int32_t)(blockIdx.x * kInfoThreads + threadIdx.x);
    if (x < a.n_groups) {
        const int32_t lo = a.group_start[x], hi = a.group_start[x + 1];
        if (lo < 0 || hi < lo || hi > a.n_seqs || (x == 0 && lo != 0) || (x == a.n_groups - 1 && hi != a.n_seqs))
            flag(p.status, KDA_DEV_BAD_GROUP);
    }
    if (x >= a.n_seqs) return;
    int64_t kv = a.kv_lens[x], shared = 0;
    if (kv < 0 || kv > cap) {
        flag(p.status, KDA_DEV_BAD_SEQLENS);
        kv = 0;
    }
    const int32_t g = group_of(a.group_start, a.n_groups, x);
    if (g >= 0) {
        shared = a.prefix_lens[g];
        if (shared < 0 || shared > cap || shared % a.block_size) shared = 0, flag(p.status, KDA_DEV_BAD_GROUP);
        if (shared > kv) flag(p.status, KDA_DEV_BAD_GROUP);
    }
    p.info[x] = make_int2((int32_t)shared, (int32_t)kv);
}

// ------------------------------------------------------------------ suffix, fp32

constexpr int kWarps = kDecodeWarps, kThreads = 32 * kWarps;
constexpr int kStages = 3;
// The maximum that weights refer to is the first tile's, and is moved when a weight
// passes kMostWeight; kLeastMaximum, the least finite number, until a row has seen a score
// above -inf: of any score above it the weight is infinite then, and moves it.
constexpr float kMostWeight = 1024.f, kLeastMaximum = -3.402823466e38f;

// A tile holds 4 KB of keys and 4 KB of values.  The 16-byte pieces of key j lie at
// piece ^ (j * lanes per key) of its row, so that eight lanes of a score (two or four
// to a key) and the lanes of a value row read distinct banks.
template <int D, int R> struct DecodeSmem {
    static constexpr int kKeys = decode_tile(KDA_FP32, D), kLanesPerKey = D / 32;
    float ring[kWarps][kStages][2][kKeys * D];
    float q[kWarps][R * D];
    float w[kWarps][kKeys * R];          // weights, key-major
};

__device__ __forceinline__ float4 load4(const float* p) { return *reinterpret_cast<const float4*>(p); }
// 16 bytes global -> shared, zeros instead when !live.
__device__ __forceinline__ void copy16(void* dst, const void* src, bool live) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"((uint32_t)__cvta_generic_to_shared(dst)),
                 "l"(__cvta_generic_to_global(src)), "r"(live ? 16 : 0)
                 : "memory");
}
template <int N> __device__ __forceinline__ void copy_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

// R query heads of a unit.
template <int D, int R>
__global__ void __launch_bounds__(kThreads, 1) decode_suffix_kernel(const __grid_constant__ AttnDecodeLaunch p) {
    using S = DecodeSmem<D, R>;
    constexpr int kKeys = S::kKeys, kLanes = S::kLanesPerKey, kPieces = D / 4, kCols = D / 32;
    extern __shared__ __align__(16) uint8_t smem_raw[];
    S& sm = *reinterpret_cast<S*>(smem_raw);
    start_after(p);
    const kda_attn_decode_args& a = p.a;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int G = a.n_heads / a.n_kv_heads, blocks = (G + R - 1) / R;
    __shared__ PieceStart at_[kWarps];
    const Line line = find_pieces<kThreads, kWarps>(p, a.n_kv_heads * blocks, kKeys, at_);
    griddep_launch();
    const int64_t piece = (int64_t)blockIdx.x * kWarps + warp;
    if (piece >= line.pieces) {
        if (lane == 0) p.open[piece] = make_int4(-1, 0, 0, 0);
        finish_empty<float, D>(p, piece, lane);
        return;
    }
    Cursor c = start(at_[warp], line, piece, a.n_kv_heads * blocks, kKeys);

    // ------------------------------------------------------------------ copies, kStages - 1 tiles ahead
    Cursor f = c;
    int32_t next_block = 0;                              // table entry of the place f
    const int page_shift = __ffs(a.block_size) - 1;
    auto look_up = [&]() {
        const int64_t key = f.info.x + f.k * kKeys;
        next_block = f.left > 0 && key < f.info.y ? a.block_table[(int64_t)f.s * a.table_stride + (key >> page_shift)] : -2;
    };
    auto fetch = [&](int stage) {
        if (f.left > 0) {
            const int64_t key = f.info.x + f.k * kKeys;
            int live = (int)max((int64_t)0, min((int64_t)kKeys, f.info.y - key));         // keys that exist
            if (live > 0 && (next_block < 0 || next_block >= a.n_blocks)) {
                flag(p.status, KDA_DEV_BAD_SLOT);
                live = 0;
            }
            const int hk = blocks == 1 ? f.u : f.u / blocks;
            const int64_t row = live > 0 ? ((int64_t)next_block * a.n_kv_heads + hk) * a.block_size + (key & (a.block_size - 1)) : 0;
            const float* ks = static_cast<const float*>(a.k_cache) + row * D;
            const float* vs = static_cast<const float*>(a.v_cache) + row * D;
#pragma unroll
            for (int i = 0; i < kKeys * kPieces / 32; ++i) {
                const int j = (i * 32 + lane) / kPieces, y = (i * 32 + lane) % kPieces;
                const int to = (j * kPieces + (y ^ (j * kLanes & 7))) * 4, from = j < live ? j * D + y * 4 : 0;
                copy16(sm.ring[warp][stage][0] + to, ks + from, j < live);
                copy16(sm.ring[warp][stage][1] + to, vs + from, j < live);
            }
            f.step(p, kKeys);
            look_up();
        }
        cp_async_commit();
    };
    look_up();
#pragma unroll
    for (int i = 0; i < kStages - 1; ++i) fetch(i);

    // ------------------------------------------------------------------ units
    const float sl = a.scale * kLog2e;
    const int my_key = lane / kLanes, my_part = lane % kLanes;
    float* q = sm.q[warp];
    float* w = sm.w[warp];
    int stage = 0;
    while (c.left > 0) {
        const int64_t k_first = c.k, k_last = c.k + c.run();
        const int32_t s = c.s;
        const int hk = c.u / blocks, rb = c.u % blocks;
        const int head0 = hk * G + rb * R, rows = min(R, G - rb * R);
        const int2 info = c.info;
        __syncwarp();                                    // the last unit's q is read
#pragma unroll
        for (int i = 4 * lane; i < R * D; i += 128) {
            float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
            if (i / D < rows) x = load4(static_cast<const float*>(a.q) + s * a.q_stride + (int64_t)head0 * D + i);
            *reinterpret_cast<float4*>(q + i) = make_float4(x.x * sl, x.y * sl, x.z * sl, x.w * sl);
        }
        float o[R][kCols], m[R], l[R];
#pragma unroll
        for (int r = 0; r < R; ++r) {
            m[r] = kLeastMaximum;
            l[r] = 0.f;
#pragma unroll
            for (int e = 0; e < kCols; ++e) o[r][e] = 0.f;
        }
        for (int64_t kt = k_first; kt < k_last; ++kt) {
            copy_wait<kStages - 2>();
            __syncwarp();                                // the tile and q are there, and the stage before is read
            fetch(stage == 0 ? kStages - 1 : stage - 1);
            const float* kb = sm.ring[warp][stage][0];
            const float* vb = sm.ring[warp][stage][1];
            stage = stage == kStages - 1 ? 0 : stage + 1;
            const bool seen = info.x + kt * kKeys + my_key < info.y;
            float x[R] = {};
#pragma unroll
            for (int i = 0; i < kPieces / kLanes; ++i) {
                const int y = i * kLanes + my_part;
                const float4 k = load4(kb + (my_key * kPieces + (y ^ (my_key * kLanes & 7))) * 4);
#pragma unroll
                for (int r = 0; r < R; ++r) {
                    const float4 z = load4(q + r * D + 4 * y);
                    x[r] = fmaf(z.w, k.w, fmaf(z.z, k.z, fmaf(z.y, k.y, fmaf(z.x, k.x, x[r]))));
                }
            }
            bool grow = false;
            float weight[R];
#pragma unroll
            for (int r = 0; r < R; ++r) {
#pragma unroll
                for (int off = 1; off < kLanes; off <<= 1) x[r] += __shfl_xor_sync(0xffffffffu, x[r], off);
                x[r] = seen ? x[r] : -CUDART_INF_F;
                weight[r] = exp2f(x[r] - m[r]);
                grow |= !(weight[r] <= kMostWeight);
            }
            if (__any_sync(0xffffffffu, grow)) {         // the first tile, and rarely later
#pragma unroll
                for (int r = 0; r < R; ++r) {
                    float mx = fmaxf(m[r], x[r]);
#pragma unroll
                    for (int off = kLanes; off < 32; off <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, off));
                    const float corr = exp2f(m[r] - mx);
                    m[r] = mx;
                    l[r] *= corr;
#pragma unroll
                    for (int e = 0; e < kCols; ++e) o[r][e] *= corr;
                    weight[r] = exp2f(x[r] - mx);
                }
            }
#pragma unroll
            for (int r = 0; r < R; ++r) l[r] += weight[r];
            if (my_part == 0)
#pragma unroll
                for (int r = 0; r < R; r += 4)
                    *reinterpret_cast<float4*>(w + my_key * R + r) = make_float4(weight[r], weight[r + 1], weight[r + 2], weight[r + 3]);
            __syncwarp();
#pragma unroll
            for (int j = 0; j < kKeys; ++j) {
                float v[kCols];
                const int y = kCols * lane / 4 ^ (j * kLanes & 7);
                if constexpr (kCols == 4) {
                    const float4 z = load4(vb + (j * kPieces + y) * 4);
                    v[0] = z.x, v[1] = z.y, v[2] = z.z, v[3] = z.w;
                } else {
                    const float2 z = *reinterpret_cast<const float2*>(vb + (j * kPieces + y) * 4 + 2 * (lane & 1));
                    v[0] = z.x, v[1] = z.y;
                }
#pragma unroll
                for (int r = 0; r < R; r += 4) {
                    const float4 z = load4(w + j * R + r);
                    const float ww[4] = {z.x, z.y, z.z, z.w};
#pragma unroll
                    for (int k = 0; k < 4; ++k)
#pragma unroll
                        for (int e = 0; e < kCols; ++e) o[r + k][e] = fmaf(ww[k], v[e], o[r + k][e]);
                }
            }
            __syncwarp();                                // the stage and the weights are read
        }
        const bool whole = k_first == 0 && k_last == c.T;
        const int n_pre = whole ? prefix_parts(p, info.x) : 0;
        if (n_pre > 0) griddep_wait();                   // the prefix's results
        const int64_t slot = part_slot(piece, k_first == 0);
        float lt[R], mt[R];
#pragma unroll
        for (int r = 0; r < R; ++r) {
            // every key's lanes hold its weight: one of them counts
            lt[r] = my_part == 0 ? l[r] : 0.f, mt[r] = m[r];
#pragma unroll
            for (int off = 16; off > 0; off >>= 1) lt[r] += __shfl_xor_sync(0xffffffffu, lt[r], off);
            if (lt[r] == 0.f) mt[r] = -CUDART_INF_F;
        }
#pragma unroll 1
        for (int i = 0; i < n_pre; ++i) {
            float2 ml[R], v[R][kCols / 2];
#pragma unroll
            for (int r = 0; r < R; ++r) {
                if (r >= rows) break;
                const int64_t pr = prefix_row(p, i, s, head0 + r);
                ml[r] = load_now2(p.pre_ml + pr);
#pragma unroll
                for (int e = 0; e < kCols / 2; ++e) v[r][e] = load_now2(p.pre_o + pr * D + kCols * lane + 2 * e);
            }
#pragma unroll
            for (int r = 0; r < R; ++r) {
                if (r >= rows) break;
                float w1, w2;
                join(mt[r], lt[r], ml[r].x, ml[r].y, w1, w2);
#pragma unroll
                for (int e = 0; e < kCols / 2; ++e) {
                    o[r][2 * e] = o[r][2 * e] * w1 + v[r][e].x * w2;
                    o[r][2 * e + 1] = o[r][2 * e + 1] * w1 + v[r][e].y * w2;
                }
            }
        }
#pragma unroll
        for (int r = 0; r < R; ++r) {
            if (r >= rows) break;
            float* out = whole ? static_cast<float*>(a.o) + s * a.o_stride + (int64_t)(head0 + r) * D : p.part_o + (slot * R + r) * D;
            const float f = !whole ? 1.f : lt[r] == 0.f ? 0.f : 1.f / lt[r];
#pragma unroll
            for (int e = 0; e < kCols; ++e) out[kCols * lane + e] = o[r][e] * f;
            if (lane == 0) {
                if (whole) write_lse(a, s, head0 + r, mt[r], lt[r]);
                else p.part_ml[slot * R + r] = make_float2(mt[r], lt[r]);
            }
        }
        if (lane == 0 && c.left == c.run()) p.open[piece] = open_unit(p, c, piece, line);
        c.next_unit(p, kKeys);
    }
    copy_wait<0>();
    finish_empty<float, D>(p, piece, lane);
}

template <int D, int R>
cudaError_t launch_t(const AttnDecodeLaunch& p, cudaStream_t s) {
    cudaError_t e = cudaFuncSetAttribute(decode_suffix_kernel<D, R>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         (int)sizeof(DecodeSmem<D, R>));
    if (e != cudaSuccess) return e;
    note_launch();
    e = launch_overlapped(decode_suffix_kernel<D, R>, dim3(p.n_pieces / kWarps), dim3(kThreads), sizeof(DecodeSmem<D, R>), s, p);
    return e == cudaSuccess ? launch_join<float, D, R>(p, s) : e;
}

}  // namespace

cudaError_t launch_decode_info(const AttnDecodeLaunch& p, cudaStream_t s) {
    const int32_t n = p.a.n_seqs > p.a.n_groups ? p.a.n_seqs : p.a.n_groups;
    note_launch();
    return launch_overlapped(decode_info_kernel, dim3((unsigned)((n + kInfoThreads - 1) / kInfoThreads)), dim3(kInfoThreads), 0,
                             s, p);
}

cudaError_t launch_decode_simt(const AttnDecodeLaunch& p, cudaStream_t s) {
    const bool few = decode_rows(KDA_FP32, p.a.n_heads / p.a.n_kv_heads) == 4;
    if (p.a.d == 128) return few ? launch_t<128, 4>(p, s) : launch_t<128, 8>(p, s);
    return few ? launch_t<64, 4>(p, s) : launch_t<64, 8>(p, s);
}

}  // namespace kda
