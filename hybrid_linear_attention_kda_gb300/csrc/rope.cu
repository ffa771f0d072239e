// Norms of queries and keys, head by head, with the position rotation, and the same on the
// way into the paged cache (include/kda_rope.h has the formulas).
//
// A head's vector is a row: d / 8 lanes with 8 channels each, as two pieces of four, so that
// both channels of every pair are in one lane: pieces j and j + rot_dim / 8 of the halves, or
// two neighbours where pairs are neighbours (and for channels behind the rotated ones).  A
// lane's four pairs are the same in all rows of a token, so that a warp forms the sines of
// its token once and walks the token's rows, several at a time: loads first, then each row's
// sum of squares over its lanes, its norm and its rotation.
#include "attn_common.cuh"
#include "rope.cuh"

namespace kda {
namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;

// Four channels of a row as they lie in memory.
template <typename T> struct Piece;
template <> struct Piece<float> {
    using Raw = float4;
    static __device__ __forceinline__ void open(const Raw& r, float* x) { x[0] = r.x, x[1] = r.y, x[2] = r.z, x[3] = r.w; }
    static __device__ __forceinline__ Raw close(const float* x) { return make_float4(x[0], x[1], x[2], x[3]); }
};
template <> struct Piece<__nv_bfloat16> {
    using Raw = uint2;
    static __device__ __forceinline__ void open(const Raw& r, float* x) {
        x[0] = __uint_as_float(r.x << 16), x[1] = __uint_as_float(r.x & 0xFFFF0000u);
        x[2] = __uint_as_float(r.y << 16), x[3] = __uint_as_float(r.y & 0xFFFF0000u);
    }
    static __device__ __forceinline__ Raw close(const float* x) {
        const __nv_bfloat162 a = __floats2bfloat162_rn(x[0], x[1]), b = __floats2bfloat162_rn(x[2], x[3]);
        return make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
    }
};

// cos and sin of 2 pi frac(position * turns / 2^64).  The product's upper 32 bits are the
// angle to 2^-32 of a turn; its nearest quarter turn is taken off in integers, so that the
// rest, at most an eighth of a turn, loses 2^-25 of itself where it becomes a float.
__device__ __forceinline__ void turn(int32_t position, uint64_t turns, float& c, float& s) {
    const uint32_t t = (uint32_t)(((uint64_t)(uint32_t)position * turns) >> 32);
    const uint32_t quarter = (t + 0x20000000u) >> 30;
    const float rest = (float)(int32_t)(t - (quarter << 30)) * 0x1p-31f;      // in half turns
    float c0, s0;
    sincospif(rest, &s0, &c0);
    c = quarter & 1 ? s0 : c0;
    s = quarter & 1 ? c0 : s0;
    if (quarter == 1 || quarter == 2) c = -c;
    if (quarter >= 2) s = -s;
}

// Warp w takes rows part * part_rows .. of token w / parts.  Rows are the query heads, then
// the key heads, then (kAppend) the value heads.
template <typename T, int D, bool kAppend>
__global__ void __launch_bounds__(kThreads) rope_kernel(const __grid_constant__ RopeLaunch p, int32_t parts, int32_t part_rows) {
    using P = Piece<T>;
    using Raw = typename P::Raw;
    constexpr int kLanes = D / 8, kRows = 32 / kLanes, kAtOnce = 4;
    griddep_wait();
    const kda_qk_rope_args& a = p.a;
    const int64_t w = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5), token = w / parts;
    if (token >= a.n_tokens) return;
    const int part = (int)(w - token * parts), lane = threadIdx.x & 31, j = lane % kLanes, own_row = lane / kLanes;
    const int32_t position = a.positions[token];
    if (position < 0) {
        if (position != -1 && lane == 0) flag(p.status, KDA_DEV_BAD_POSITION);
        return;
    }
    const int H = a.n_heads, H_kv = a.n_kv_heads, n_rows = H + (kAppend ? 2 : 1) * H_kv;
    const int lo = part * part_rows, hi = min(n_rows, lo + part_rows);

    int64_t slot_row = -1;                               // first row of the token's slot in the cache
    if (kAppend) {
        const int32_t slot = p.slot_map[token];
        if (slot >= 0 && slot < p.n_blocks * p.block_size)
            slot_row = (int64_t)(slot / p.block_size) * H_kv * p.block_size + slot % p.block_size;
        else if (slot != -1 && lane == 0)
            flag(p.status, KDA_DEV_BAD_SLOT);
    }

    const int turned = a.rot_dim / 8;                    // lanes whose channels are rotated
    const bool halves = !a.interleaved && j < turned;
    const int c0 = 4 * (halves ? j : 2 * j), c1 = halves ? c0 + a.rot_dim / 2 : c0 + 4;
    float cs[4], sn[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) cs[e] = 1.f, sn[e] = 0.f;
    if (j < turned) {
#pragma unroll
        for (int e = 0; e < 4; ++e) turn(position, a.turns[4 * j + e], cs[e], sn[e]);
    }

    const T* q = static_cast<const T*>(a.q) + token * a.q_stride;
    const T* k = static_cast<const T*>(a.k) + token * a.k_stride;
    const T* v = kAppend ? static_cast<const T*>(p.v) + token * p.v_stride : nullptr;
    for (int b = lo; b < hi; b += kRows * kAtOnce) {
        Raw raw[kAtOnce][2];
#pragma unroll
        for (int u = 0; u < kAtOnce; ++u) {
            const int r = b + u * kRows + own_row;
            raw[u][0] = raw[u][1] = Raw{};
            if (r >= hi) continue;
            const T* x = r < H ? q + (int64_t)r * D : r < H + H_kv ? k + (int64_t)(r - H) * D : v + (int64_t)(r - H - H_kv) * D;
            raw[u][0] = *reinterpret_cast<const Raw*>(x + c0);
            raw[u][1] = *reinterpret_cast<const Raw*>(x + c1);
        }
#pragma unroll
        for (int u = 0; u < kAtOnce; ++u) {
            const int r = b + u * kRows + own_row;
            const bool is_v = r >= H + H_kv;
            const float* weight = r < H ? a.q_weight : is_v ? nullptr : a.k_weight;
            float x[8];
            P::open(raw[u][0], x);
            P::open(raw[u][1], x + 4);
            if (a.q_weight || a.k_weight) {
                float sum = 0.f;
#pragma unroll
                for (int e = 0; e < 8; ++e) sum = fmaf(x[e], x[e], sum);
#pragma unroll
                for (int off = 1; off < kLanes; off <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
                if (weight) {
                    const float inv = 1.f / sqrtf(sum * (1.f / D) + a.eps);
                    const float4 w0 = *reinterpret_cast<const float4*>(weight + c0), w1 = *reinterpret_cast<const float4*>(weight + c1);
                    x[0] *= inv * w0.x, x[1] *= inv * w0.y, x[2] *= inv * w0.z, x[3] *= inv * w0.w;
                    x[4] *= inv * w1.x, x[5] *= inv * w1.y, x[6] *= inv * w1.z, x[7] *= inv * w1.w;
                }
            }
            if (!is_v) {
                if (halves) {
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const float x0 = x[e], x1 = x[4 + e];
                        x[e] = x0 * cs[e] - x1 * sn[e];
                        x[4 + e] = x0 * sn[e] + x1 * cs[e];
                    }
                } else if (j < turned) {
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const float x0 = x[2 * e], x1 = x[2 * e + 1];
                        x[2 * e] = x0 * cs[e] - x1 * sn[e];
                        x[2 * e + 1] = x0 * sn[e] + x1 * cs[e];
                    }
                }
                raw[u][0] = P::close(x);
                raw[u][1] = P::close(x + 4);
            }
            T* to = nullptr;
            if (r >= hi) {
            } else if (r < H) {
                to = static_cast<T*>(a.q_out) + token * a.q_out_stride + (int64_t)r * D;
            } else if (!kAppend) {
                to = static_cast<T*>(a.k_out) + token * a.k_out_stride + (int64_t)(r - H) * D;
            } else if (slot_row >= 0) {
                const int h = is_v ? r - H - H_kv : r - H;
                to = static_cast<T*>(is_v ? p.v_cache : p.k_cache) + (slot_row + (int64_t)h * p.block_size) * D;
            }
            if (to) {
                *reinterpret_cast<Raw*>(to + c0) = raw[u][0];
                *reinterpret_cast<Raw*>(to + c1) = raw[u][1];
            }
        }
    }
}

template <typename T, int D, bool kAppend>
cudaError_t launch_t(const RopeLaunch& p, cudaStream_t s) {
    constexpr int kBatch = 4 * (32 / (D / 8));
    const int n_rows = p.a.n_heads + (kAppend ? 2 : 1) * p.a.n_kv_heads, batches = (n_rows + kBatch - 1) / kBatch;
    // a token's rows are spread over warps until the GPU has 32 of them an SM
    int64_t parts = (152 * 32 + p.a.n_tokens - 1) / p.a.n_tokens;
    parts = parts < batches ? parts : batches;
    const int32_t part_rows = (int32_t)((batches + parts - 1) / parts) * kBatch;
    parts = (n_rows + part_rows - 1) / part_rows;
    note_launch();
    return launch_overlapped(rope_kernel<T, D, kAppend>, dim3((unsigned)((p.a.n_tokens * parts + kWarps - 1) / kWarps)),
                             dim3(kThreads), 0, s, p, (int32_t)parts, part_rows);
}

template <bool kAppend>
cudaError_t launch(const RopeLaunch& p, cudaStream_t s) {
    if (p.a.dtype == KDA_BF16) return p.a.d == 128 ? launch_t<__nv_bfloat16, 128, kAppend>(p, s) : launch_t<__nv_bfloat16, 64, kAppend>(p, s);
    return p.a.d == 128 ? launch_t<float, 128, kAppend>(p, s) : launch_t<float, 64, kAppend>(p, s);
}

}  // namespace

cudaError_t launch_rope(const RopeLaunch& p, cudaStream_t s) { return p.append ? launch<true>(p, s) : launch<false>(p, s); }

}  // namespace kda
