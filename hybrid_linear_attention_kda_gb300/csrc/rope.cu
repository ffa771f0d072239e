// Norms of queries and keys, head by head, with the position rotation, and the same on the
// way into the paged cache (include/kda_rope.h has the formulas).
//
// A head's vector is a row: d / 8 lanes with 8 channels each, as two pieces of four, so that
// both channels of every pair are in one lane: pieces j and j + rot_dim / 8 of the halves, or
// two neighbours where pairs are neighbours (and for channels behind the rotated ones).  A
// lane's four pairs are the same in all rows of a token, so that a warp forms the sines of
// its token once, with the weights in them, and walks the token's rows, several at a time: loads
// first, then each row's sum of squares over its lanes, its norm and its rotation.
//
// Bound by HBM: 32768 tokens, 32 + 8 heads, d = 128, bf16 take 111 us (6.1 TB/s), fp32 with d = 64
// 7001 tokens, 16 + 2 + 2 heads 17 us (4.3 TB/s).  512 tokens take 4.3 us: the launch and three trips to memory, the
// position, the frequencies, the rows.
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

// What a lane makes of its pairs in all rows of one kind: with the weights w and its token's
// angles, (x0, x1) -> ((w0 c) x0 - (w1 s) x1, (w0 s) x0 + (w1 c) x1), times the row's norm.
struct Turn {
    float a[4], b[4], c[4], d[4];
};
// The i-th pair's places among the lane's eight channels.
template <bool kHalves> __device__ __forceinline__ constexpr int first_of(int i) { return kHalves ? i : 2 * i; }
template <bool kHalves> __device__ __forceinline__ constexpr int second_of(int i) { return kHalves ? 4 + i : 2 * i + 1; }

// Rows lo .. hi - 1 of one kind; from and to are the lane's places in row 0, kRows rows a warp.
// Rows of a lane under way: 64 bytes (fp32 with 128: 19 us for the 7001 tokens, 92 registers).
template <typename T> constexpr int kAtOnce = 8 / (int)sizeof(T);

template <typename T, int D, bool kHalves>
__device__ __forceinline__ void turn_rows(const T* from, T* to, int64_t from_row, int64_t to_row, int lo, int hi, int c0, int c1, bool turned,
                                          const Turn& t, bool norm, float eps) {
    using P = Piece<T>;
    using Raw = typename P::Raw;
    constexpr int kLanes = D / 8, kRows = 32 / kLanes;
    for (int b = lo; b < hi; b += kRows * kAtOnce<T>) {     // (the same for all lanes)
        const int r0 = b + (threadIdx.x & 31) / kLanes;
        Raw raw[kAtOnce<T>][2];
#pragma unroll
        for (int u = 0; u < kAtOnce<T>; ++u) {
            raw[u][0] = raw[u][1] = Raw{};
            if (r0 + u * kRows < hi) {
                const T* x = from + (r0 + u * kRows) * from_row;
                raw[u][0] = *reinterpret_cast<const Raw*>(x + c0);
                raw[u][1] = *reinterpret_cast<const Raw*>(x + c1);
            }
        }
#pragma unroll
        for (int u = 0; u < kAtOnce<T>; ++u) {
            float x[8], y[8], inv = 1.f;
            P::open(raw[u][0], x);
            P::open(raw[u][1], x + 4);
            if (norm) {
                float sum = 0.f;
#pragma unroll
                for (int e = 0; e < 8; ++e) sum = fmaf(x[e], x[e], sum);
#pragma unroll
                for (int off = 1; off < kLanes; off <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
                inv = rsqrtf(fmaf(sum, 1.f / D, eps));
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float x0 = x[first_of<kHalves>(i)] * inv, x1 = x[second_of<kHalves>(i)] * inv;
                y[first_of<kHalves>(i)] = turned ? fmaf(x0, t.a[i], x1 * t.b[i]) : x0 * t.a[i];
                y[second_of<kHalves>(i)] = turned ? fmaf(x0, t.c[i], x1 * t.d[i]) : x1 * t.d[i];
            }
            if (to && r0 + u * kRows < hi) {
                T* out = to + (r0 + u * kRows) * to_row;
                *reinterpret_cast<Raw*>(out + c0) = P::close(y);
                *reinterpret_cast<Raw*>(out + c1) = P::close(y + 4);
            }
        }
    }
}

// Warp w takes rows part * part_rows .. of token w / parts.  Rows are the query heads, then
// the key heads, then (kAppend) the value heads.
template <typename T, int D, bool kHalves, bool kAppend>
__global__ void __launch_bounds__(kThreads) rope_kernel(const __grid_constant__ RopeLaunch p, int32_t parts, int32_t part_rows) {
    using Raw = typename Piece<T>::Raw;
    constexpr int kLanes = D / 8, kRows = 32 / kLanes;
    griddep_wait();
    const kda_qk_rope_args& a = p.a;
    const int64_t w = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5), token = w / parts;
    if (token >= a.n_tokens) return;
    const int part = (int)(w - token * parts), lane = threadIdx.x & 31, j = lane % kLanes;
    const int32_t position = a.positions[token];
    if (position < 0) {
        if (position != -1 && lane == 0) flag(p.status, KDA_DEV_BAD_POSITION);
        return;
    }
    const int H = a.n_heads, H_kv = a.n_kv_heads, n_rows = H + (kAppend ? 2 : 1) * H_kv;
    const int lo = part * part_rows, hi = min(n_rows, lo + part_rows);

    int64_t slot_row = -1;                               // first row of the token's slot in the cache
    if (kAppend) {
        const int32_t slot = p.slot_map[token], shift = __ffs(p.block_size) - 1;
        if (slot >= 0 && slot < p.n_blocks << shift)
            slot_row = ((int64_t)(slot >> shift) * H_kv << shift) + (slot & (p.block_size - 1));
        else if (slot != -1 && lane == 0)
            flag(p.status, KDA_DEV_BAD_SLOT);
    }

    const int turned = a.rot_dim / 8;                    // lanes whose channels are rotated
    const bool apart = kHalves && j < turned;
    const int c0 = 4 * (apart ? j : 2 * j), c1 = apart ? c0 + a.rot_dim / 2 : c0 + 4;
    float cs[4], sn[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) cs[e] = 1.f, sn[e] = 0.f;
    if (j < turned && lo < H + H_kv) {
#pragma unroll
        for (int e = 0; e < 4; ++e) turn(position, a.turns[4 * j + e], cs[e], sn[e]);
    }
    auto weighted = [&](const float* weight) {
        float w[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) w[e] = 1.f;
        if (weight) {
            Piece<float>::open(*reinterpret_cast<const float4*>(weight + c0), w);
            Piece<float>::open(*reinterpret_cast<const float4*>(weight + c1), w + 4);
        }
        Turn t;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float w0 = w[first_of<kHalves>(i)], w1 = w[second_of<kHalves>(i)];
            t.a[i] = w0 * cs[i], t.b[i] = -w1 * sn[i], t.c[i] = w0 * sn[i], t.d[i] = w1 * cs[i];
        }
        return t;
    };
    if (lo < H)
        turn_rows<T, D, kHalves>(static_cast<const T*>(a.q) + token * a.q_stride, static_cast<T*>(a.q_out) + token * a.q_out_stride, D, D, lo, min(hi, H),
                                 c0, c1, j < turned, weighted(a.q_weight), a.q_weight != nullptr, a.eps);
    if (hi > H && lo < H + H_kv) {
        T* to = nullptr;
        if (!kAppend) to = static_cast<T*>(a.k_out) + token * a.k_out_stride;
        else if (slot_row >= 0) to = static_cast<T*>(p.k_cache) + slot_row * D;
        turn_rows<T, D, kHalves>(static_cast<const T*>(a.k) + token * a.k_stride, to, D, kAppend ? (int64_t)p.block_size * D : D, max(lo - H, 0),
                                 min(hi - H, H_kv), c0, c1, j < turned, weighted(a.k_weight), a.k_weight != nullptr, a.eps);
    }
    if (kAppend && hi > H + H_kv && slot_row >= 0) {
        const T* v = static_cast<const T*>(p.v) + token * p.v_stride + 8 * j;
        T* to = static_cast<T*>(p.v_cache) + slot_row * D + 8 * j;
        const int64_t to_row = (int64_t)p.block_size * D;
#pragma unroll 2
        for (int r = max(lo - H - H_kv, 0) + lane / kLanes; r < hi - H - H_kv; r += kRows) {
            const Raw x0 = reinterpret_cast<const Raw*>(v + r * D)[0], x1 = reinterpret_cast<const Raw*>(v + r * D)[1];
            reinterpret_cast<Raw*>(to + r * to_row)[0] = x0, reinterpret_cast<Raw*>(to + r * to_row)[1] = x1;
        }
    }
}

template <typename T, int D, bool kAppend>
cudaError_t launch_t(const RopeLaunch& p, cudaStream_t s) {
    constexpr int kBatch = kAtOnce<T> * (32 / (D / 8));
    const int n_rows = p.a.n_heads + (kAppend ? 2 : 1) * p.a.n_kv_heads, batches = (n_rows + kBatch - 1) / kBatch;
    // A token's rows are spread over warps until the GPU has 32 of them an SM (bf16, 40 rows, d =
    // 128: 512 tokens 4.3 us, a warp each 6.6 us; 6000 tokens, a warp each, 25.1 us, three 28.4 us).
    int64_t parts = (152 * 32 + p.a.n_tokens - 1) / p.a.n_tokens;
    parts = parts < batches ? parts : batches;
    const int32_t part_rows = (int32_t)((batches + parts - 1) / parts) * kBatch;
    parts = (n_rows + part_rows - 1) / part_rows;
    note_launch();
    return launch_overlapped(p.a.interleaved ? rope_kernel<T, D, false, kAppend> : rope_kernel<T, D, true, kAppend>,
                             dim3((unsigned)((p.a.n_tokens * parts + kWarps - 1) / kWarps)), dim3(kThreads), 0, s, p, (int32_t)parts, part_rows);
}

template <bool kAppend>
cudaError_t launch(const RopeLaunch& p, cudaStream_t s) {
    if (p.a.dtype == KDA_BF16) return p.a.d == 128 ? launch_t<__nv_bfloat16, 128, kAppend>(p, s) : launch_t<__nv_bfloat16, 64, kAppend>(p, s);
    return p.a.d == 128 ? launch_t<float, 128, kAppend>(p, s) : launch_t<float, 64, kAppend>(p, s);
}

}  // namespace

cudaError_t launch_rope(const RopeLaunch& p, cudaStream_t s) { return p.append ? launch<true>(p, s) : launch<false>(p, s); }

}  // namespace kda
