// The 4-bit paged cache: append and read-back (include/kda_cache_q4.h has the format).
//
// The append is bound by its arithmetic: 32768 tokens of 8 heads, d = 128, bf16, with the values
// written too, take 73 us (4.2 TB/s) at 78% of the issue slots, 266 instructions a warp for 8
// channels a lane, a quarter of them for lanes whose quotient lies in the middle of two codes.
// In pairs of floats (fma.f32x2) they took 75 us.  512 tokens: 3.0 us.
//
// The read-back is bound by HBM, most of it writes: 24 sequences of up to 16384 tokens, 8 heads,
// d = 128 to bf16 take 200 us (5.9 TB/s).
#include <float.h>
#include <math_constants.h>

#include "cache_q4.cuh"

namespace kda {
namespace {

constexpr int kThreads = 256;

// x rounded to bf16 towards -inf, towards +inf (x >= 0), as a float.
__device__ __forceinline__ float bf16_down(float x) {
    const uint32_t b = __float_as_uint(x);
    return __uint_as_float((b + (b >> 31 ? 0xFFFFu : 0u)) & 0xFFFF0000u);
}
__device__ __forceinline__ float bf16_up(float x) { return __uint_as_float((__float_as_uint(x) + 0xFFFFu) & 0xFFFF0000u); }

// Eight channels as they lie in memory.
template <typename T> struct Eight;
template <> struct Eight<__nv_bfloat16> {
    uint4 r;
    __device__ __forceinline__ void open(float (&x)[8]) const {
        const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) x[2 * i] = __uint_as_float(w[i] << 16), x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
    __device__ __forceinline__ void close(const float (&x)[8]) {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const __nv_bfloat162 v = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
            w[i] = *reinterpret_cast<const uint32_t*>(&v);
        }
        r = make_uint4(w[0], w[1], w[2], w[3]);
    }
};
template <> struct Eight<float> {
    float4 r[2];
    __device__ __forceinline__ void open(float (&x)[8]) const {
        x[0] = r[0].x, x[1] = r[0].y, x[2] = r[0].z, x[3] = r[0].w;
        x[4] = r[1].x, x[5] = r[1].y, x[6] = r[1].z, x[7] = r[1].w;
    }
    __device__ __forceinline__ void close(const float (&x)[8]) {
        r[0] = make_float4(x[0], x[1], x[2], x[3]);
        r[1] = make_float4(x[4], x[5], x[6], x[7]);
    }
};

// The values of a word's codes, as T, each rounded once.  Codes become numbers as the low bits of
// 2^23, or of 128 in bf16, less that; bf16's are formed four apart and put in order.
__device__ __forceinline__ void values_of(uint32_t w, uint32_t scale, Eight<float>& out) {
    const float step = __uint_as_float(scale << 16), low = __uint_as_float(scale & 0xFFFF0000u);
    float v[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = fmaf(__uint_as_float((w >> 4 * e & 15u) | 0x4B000000u) - 8388608.f, step, low);
    out.close(v);
}
__device__ __forceinline__ void values_of(uint32_t w, uint32_t scale, Eight<__nv_bfloat16>& out) {
    const uint32_t steps = __byte_perm(scale, scale, 0x1010), lows = __byte_perm(scale, scale, 0x3232), none = 0x43004300u;
    uint32_t v[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {                            // channels e and e + 4
        const uint32_t n = (w >> 4 * e & 0x000F000Fu) | none;
        const __nv_bfloat162 r = __hfma2(__hsub2(*reinterpret_cast<const __nv_bfloat162*>(&n), *reinterpret_cast<const __nv_bfloat162*>(&none)),
                                         *reinterpret_cast<const __nv_bfloat162*>(&steps), *reinterpret_cast<const __nv_bfloat162*>(&lows));
        v[e] = *reinterpret_cast<const uint32_t*>(&r);
    }
    out.r = make_uint4(__byte_perm(v[0], v[1], 0x5410), __byte_perm(v[2], v[3], 0x5410), __byte_perm(v[0], v[1], 0x7632), __byte_perm(v[2], v[3], 0x7632));
}

__device__ __forceinline__ float min_nan(float x, float y) {
    float r;
    asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(x), "f"(y));
    return r;
}
__device__ __forceinline__ float max_nan(float x, float y) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(x), "f"(y));
    return r;
}
// The smallest and the largest of a group, eight lanes' channels; NaN where one is.  bf16 in
// pairs, and the lanes' as (smallest, - largest).
__device__ __forceinline__ void range_of(const Eight<float>&, const float (&x)[8], float& lo, float& hi) {
    lo = hi = x[0];
#pragma unroll
    for (int e = 1; e < 8; ++e) lo = min_nan(lo, x[e]), hi = max_nan(hi, x[e]);
#pragma unroll
    for (int off = 1; off < 8; off <<= 1) {
        lo = min_nan(lo, __shfl_xor_sync(0xffffffffu, lo, off));
        hi = max_nan(hi, __shfl_xor_sync(0xffffffffu, hi, off));
    }
}
__device__ __forceinline__ void range_of(const Eight<__nv_bfloat16>& v, const float (&)[8], float& lo, float& hi) {
    const __nv_bfloat162* w = reinterpret_cast<const __nv_bfloat162*>(&v.r);
    const __nv_bfloat162 a = __hmin2_nan(__hmin2_nan(w[0], w[1]), __hmin2_nan(w[2], w[3]));
    const __nv_bfloat162 b = __hmax2_nan(__hmax2_nan(w[0], w[1]), __hmax2_nan(w[2], w[3]));
    const uint32_t ab = *reinterpret_cast<const uint32_t*>(&a), bb = *reinterpret_cast<const uint32_t*>(&b) ^ 0x80008000u;
    uint32_t p = __byte_perm(ab, bb, 0x5410), q = __byte_perm(ab, bb, 0x7632);
    __nv_bfloat162 m = __hmin2_nan(*reinterpret_cast<const __nv_bfloat162*>(&p), *reinterpret_cast<const __nv_bfloat162*>(&q));
#pragma unroll
    for (int off = 1; off < 8; off <<= 1) m = __hmin2_nan(m, __shfl_xor_sync(0xffffffffu, m, off));
    lo = __low2float(m), hi = -__high2float(m);
}

constexpr float kMagic = 12582912.f;     // 1.5 * 2^23: adding it rounds to integers, which its low bits then hold

// Codes and (s, m) of a group, of which this lane has eight channels: `v` is what they are in
// memory.
//
// The definition's quotient is the correctly rounded one.  A product with 1 / s is within 2^-18
// of it, and rounds to the same integer unless it lies that near the middle of two.  Those lanes
// look at what is left of x: it lies in the middle (common in bf16: the even code is taken), or
// clearly to one side, or they divide.
template <typename T> __device__ __forceinline__ uint32_t encode(const Eight<T>& v, uint32_t& scale) {
    float x[8], lo, hi;
    v.open(x);
    range_of(v, x, lo, hi);
    float low = sizeof(T) == 2 ? lo : bf16_down(lo), step = bf16_up(__fdiv_rn(__fsub_rn(hi, low), 15.f)), by;
    const bool fine = fabsf(low) <= FLT_MAX && __fsub_rn(hi, low) <= FLT_MAX && step <= FLT_MAX;      // (no, with a NaN)
    if (!fine) low = CUDART_NAN_F, step = 0.f;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(by) : "f"(step));
    float c[8], most = 0.f;                                  // codes; how far from its integer a quotient is
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        x[e] = __fsub_rn(x[e], low);
        c[e] = fmaf(x[e], by, kMagic) - kMagic;
        most = fmaxf(most, fabsf(fmaf(x[e], by, -c[e])));
    }
    // (a tiny step's inverse is not a number to go by; nor is there a middle to be near without one)
    if (!(most <= 0.5f - 0x1p-16f) || !(step >= 0x1p-100f)) {
        bool divide = !(step >= 0x1p-100f);
        const float half = 0.5f * step, near = step * 0x1p-18f;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const float rest = fmaf(-c[e], step, x[e]), past = fabsf(rest) - half;           // both exact
            divide |= past != 0.f && fabsf(past) < near;
            const bool odd = __float_as_uint(c[e] + kMagic) & 1u;
            if (odd ? past >= 0.f : past > 0.f) c[e] += copysignf(1.f, rest);
        }
        if (divide) {
#pragma unroll
            for (int e = 0; e < 8; ++e) c[e] = step > 0.f ? fminf(rintf(__fdiv_rn(x[e], step)), 15.f) : 0.f;
        }
    }
    scale = __float_as_uint(step) >> 16 | (__float_as_uint(low) & 0xFFFF0000u);
    // four codes fit a float's integers
    const float c03 = fmaf(fmaf(fmaf(c[3], 16.f, c[2]), 16.f, c[1]), 16.f, c[0]) + kMagic, c47 = fmaf(fmaf(fmaf(c[7], 16.f, c[6]), 16.f, c[5]), 16.f, c[4]) + kMagic;
    return __byte_perm(__float_as_uint(c03), __float_as_uint(c47), 0x5410);
}

// A thread takes eight channels of a key and the same of its value, eight lanes a group.  A
// thread block takes whole tokens, all heads: block_tokens of them; `row_magic` divides by a
// token's pieces of one tensor, as ceil(2^20 / row_vecs) where a block has several tokens.
template <typename T, int D>
__global__ void __launch_bounds__(kThreads) append_q4_kernel(const __grid_constant__ CacheAppendQ4Launch p, uint32_t block_tokens, uint32_t row_magic) {
    constexpr uint32_t kHeadVecs = D / 8;
    griddep_wait();
    const kda_cache_append_q4_args& a = p.a;
    const uint32_t row_vecs = kHeadVecs * (uint32_t)a.n_kv_heads;
    const int shift = __ffs(a.cache.block_size) - 1;
    const int64_t t0 = (int64_t)blockIdx.x * block_tokens, n_slots = a.cache.n_blocks << shift;
    const uint32_t n = row_vecs * (uint32_t)min((int64_t)block_tokens, a.n_tokens - t0);
    for (uint32_t base = 0; base < n; base += kThreads) {
        const uint32_t i = base + threadIdx.x, token = block_tokens == 1 ? 0 : i * row_magic >> 20, y = i - token * row_vecs;
        const int64_t t = t0 + token;
        Eight<T> k{}, v{};
        int32_t slot = -1;
        if (i < n) {
            slot = a.slot_map[t];
            k = *reinterpret_cast<const Eight<T>*>(static_cast<const T*>(a.k) + t * a.k_stride + y * 8);
            v = *reinterpret_cast<const Eight<T>*>(static_cast<const T*>(a.v) + t * a.v_stride + y * 8);
        }
        uint32_t k_scale, v_scale;
        const uint32_t k_codes = encode(k, k_scale), v_codes = encode(v, v_scale);
        if (slot < 0 || slot >= n_slots) {
            if (slot != -1) flag(p.status, KDA_DEV_BAD_SLOT);
            continue;
        }
        const uint32_t h = y / kHeadVecs, e = y % kHeadVecs;
        // (rows are below 2^31)
        const uint64_t row = (uint32_t)(((slot >> shift) * a.n_kv_heads + h) << shift) + (slot & (a.cache.block_size - 1));
        static_cast<uint32_t*>(a.cache.k_codes)[row * kHeadVecs + e] = k_codes;
        static_cast<uint32_t*>(a.cache.v_codes)[row * kHeadVecs + e] = v_codes;
        if (e % 8 == 0) {
            static_cast<uint32_t*>(a.cache.k_scales)[row * (kHeadVecs / 8) + e / 8] = k_scale;
            static_cast<uint32_t*>(a.cache.v_scales)[row * (kHeadVecs / 8) + e / 8] = v_scale;
        }
        if (a.k_out) {
            values_of(k_codes, k_scale, k);
            *reinterpret_cast<Eight<T>*>(static_cast<T*>(a.k_out) + t * a.k_out_stride + y * 8) = k;
        }
        if (a.v_out) {
            values_of(v_codes, v_scale, v);
            *reinterpret_cast<Eight<T>*>(static_cast<T*>(a.v_out) + t * a.v_out_stride + y * 8) = v;
        }
    }
}

// ------------------------------------------------------------------ read-back

constexpr int kWarps = kThreads / 32, kRows = 16;           // an item: 16 positions of one head

// A lane's sixteen channels in stores of whole 32-byte sectors (two of 16 bytes each: 240 us for
// 24 sequences of up to 16384 tokens, 8 heads, d = 128; so: 200 us).  Such a store needs 32-byte
// alignment: caches that are aligned to 16 bytes only (`sectors` false) take two of 16.
__device__ __forceinline__ void store32(void* to, uint4 a, uint4 b, bool sectors) {
    if (sectors) {
        asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(to), "r"(a.x), "r"(a.y), "r"(a.z), "r"(a.w), "r"(b.x), "r"(b.y),
                     "r"(b.z), "r"(b.w)
                     : "memory");
    } else {
        static_cast<uint4*>(to)[0] = a, static_cast<uint4*>(to)[1] = b;
    }
}
__device__ __forceinline__ void write_sixteen(__nv_bfloat16* to, uint2 codes, uint32_t scale, bool sectors) {
    Eight<__nv_bfloat16> x, y;
    values_of(codes.x, scale, x);
    values_of(codes.y, scale, y);
    store32(to, x.r, y.r, sectors);
}
__device__ __forceinline__ void write_sixteen(float* to, uint2 codes, uint32_t scale, bool sectors) {
    Eight<float> x;
    values_of(codes.x, scale, x);
    store32(to, reinterpret_cast<const uint4*>(x.r)[0], reinterpret_cast<const uint4*>(x.r)[1], sectors);
    values_of(codes.y, scale, x);
    store32(to + 8, reinterpret_cast<const uint4*>(x.r)[0], reinterpret_cast<const uint4*>(x.r)[1], sectors);
}

// Items in the order of sequences, positions, heads, dealt to the warps in turn, so that all
// warps work side by side whatever the lengths are.  Every thread block runs the (short)
// scan over the sequences itself.
template <typename T, int D>
__global__ void __launch_bounds__(kThreads) unpack_q4_kernel(const __grid_constant__ CacheUnpackQ4Launch p) {
    griddep_wait();
    __shared__ int64_t scan_buf[kWarps];
    __shared__ int64_t s_end[kThreads];
    __shared__ int2 s_range[kThreads];                       // positions from, to
    const kda_cache_unpack_q4_args& a = p.a;
    const int tid = threadIdx.x, lane = tid & 31, bs = a.cache.block_size, shift = __ffs(bs) - 1;
    constexpr int kLanes = D / 16, kAtOnce = 32 / kLanes, kSteps = kRows / kAtOnce;    // lanes of a row, rows of a step
    const int own_row = lane / kLanes, own = lane % kLanes;
    const int64_t cap = (int64_t)min(a.table_stride, a.to_stride) * bs;
    const bool sectors = ((reinterpret_cast<uintptr_t>(a.k_cache) | reinterpret_cast<uintptr_t>(a.v_cache)) & 31u) == 0;
    const int64_t workers = (int64_t)gridDim.x * kWarps, worker = (int64_t)blockIdx.x * kWarps + (tid >> 5);
    int64_t base = 0;                                        // items of the sequences before this chunk
    for (int32_t s0 = 0; s0 < a.n_seqs; s0 += kThreads) {
        const int32_t s = s0 + tid;
        int64_t items = 0;
        int2 range = make_int2(0, 0);
        if (s < a.n_seqs) {
            const int64_t kv = a.kv_lens[s];
            const int32_t first = a.first ? a.first[s] : 0;
            if (kv < 0 || kv > cap || first < 0) {
                if (blockIdx.x == 0) flag(p.status, KDA_DEV_BAD_SEQLENS);
            } else if (first < kv) {
                range = make_int2(first, (int)kv);
                items = ((kv + kRows - 1) / kRows - first / kRows) * a.n_kv_heads;
            }
        }
        int64_t total;
        s_end[tid] = block_scan<kThreads>(items, scan_buf, &total);
        s_range[tid] = range;
        __syncthreads();
        int64_t x = worker - base % workers;                 // the chunk's items that are this warp's
        if (x < 0) x += workers;
        for (; x < total; x += workers) {
            int i = 0;                                       // the first sequence that ends behind x
#pragma unroll
            for (int step = kThreads / 2; step > 0; step >>= 1)
                if (s_end[i + step - 1] <= x) i += step;
            const int64_t rel = x - (i ? s_end[i - 1] : 0);
            const int2 r = s_range[i];
            const int32_t piece = (int32_t)(rel / a.n_kv_heads), h = (int32_t)(rel - (int64_t)piece * a.n_kv_heads);
            const int32_t pos0 = (r.x / kRows + piece) * kRows, j = pos0 >> shift;
            const int32_t from = a.block_table[(int64_t)(s0 + i) * a.table_stride + j];
            const int32_t to = a.to_table[(int64_t)(s0 + i) * a.to_stride + j];
            if (from < 0 || from >= a.cache.n_blocks || to < 0 || to >= a.n_blocks) {
                if (lane == 0) flag(p.status, KDA_DEV_BAD_SLOT);
                continue;
            }
            const int64_t src = ((int64_t)from * a.n_kv_heads + h) * bs + (pos0 & (bs - 1)) + own_row;
            const int64_t dst = ((int64_t)to * a.n_kv_heads + h) * bs + (pos0 & (bs - 1)) + own_row;
            uint2 codes[2][kSteps];
            uint32_t scale[2][kSteps];
#pragma unroll
            for (int v = 0; v < 2; ++v)
#pragma unroll
                for (int k = 0; k < kSteps; ++k) {
                    const int64_t row = src + k * kAtOnce;
                    codes[v][k] = static_cast<const uint2*>(v ? a.cache.v_codes : a.cache.k_codes)[row * kLanes + own];
                    scale[v][k] = static_cast<const uint32_t*>(v ? a.cache.v_scales : a.cache.k_scales)[row * (D / kQ4Group) + own / 4];
                }
#pragma unroll
            for (int v = 0; v < 2; ++v)
#pragma unroll
                for (int k = 0; k < kSteps; ++k) {
                    const int32_t pos = pos0 + own_row + k * kAtOnce;
                    if (pos < r.x || pos >= r.y) continue;
                    write_sixteen(static_cast<T*>(v ? a.v_cache : a.k_cache) + (dst + k * kAtOnce) * D + own * 16, codes[v][k], scale[v][k],
                                  sectors);
                }
        }
        base += total;
        __syncthreads();                                     // before the next chunk rewrites the shared arrays
    }
}

template <typename T, int D>
cudaError_t launch_unpack_t(const CacheUnpackQ4Launch& p, cudaStream_t s) {
    const int64_t cap = (int64_t)(p.a.table_stride < p.a.to_stride ? p.a.table_stride : p.a.to_stride) * p.a.cache.block_size;
    const int64_t items = (cap + kRows - 1) / kRows * p.a.n_seqs * p.a.n_kv_heads, blocks = (items + kWarps - 1) / kWarps;
    note_launch();
    return launch_overlapped(unpack_q4_kernel<T, D>, dim3((unsigned)(blocks < 152 * 8 ? blocks : 152 * 8)), dim3(kThreads), 0, s, p);
}

}  // namespace

cudaError_t launch_append_q4(const CacheAppendQ4Launch& p, cudaStream_t s) {
    // As many whole tokens as fill a block, at least one (512 tokens of one head, d = 64: 2.2 us, one
    // to a block 4.8 us; 32768: 6.2 and 178 us).
    const uint32_t row_vecs = (uint32_t)p.a.n_kv_heads * (p.a.d / 8);
    const uint32_t block_tokens = row_vecs < kThreads ? kThreads / row_vecs : 1, magic = ((1u << 20) + row_vecs - 1) / row_vecs;
    const dim3 grid((unsigned)((p.a.n_tokens + block_tokens - 1) / block_tokens));
    const bool wide = p.a.d == 128;
    note_launch();
    if (p.a.dtype == KDA_BF16)
        return launch_overlapped(wide ? append_q4_kernel<__nv_bfloat16, 128> : append_q4_kernel<__nv_bfloat16, 64>, grid, dim3(kThreads), 0, s, p, block_tokens, magic);
    return launch_overlapped(wide ? append_q4_kernel<float, 128> : append_q4_kernel<float, 64>, grid, dim3(kThreads), 0, s, p, block_tokens, magic);
}

cudaError_t launch_unpack_q4(const CacheUnpackQ4Launch& p, cudaStream_t s) {
    if (p.a.dtype == KDA_BF16) return p.a.d == 128 ? launch_unpack_t<__nv_bfloat16, 128>(p, s) : launch_unpack_t<__nv_bfloat16, 64>(p, s);
    return p.a.d == 128 ? launch_unpack_t<float, 128>(p, s) : launch_unpack_t<float, 64>(p, s);
}

}  // namespace kda
