// Decode attention over the 4-bit cache.  The division of work (a line of tiles of 16 keys,
// cut into equal pieces, a warp each, and the join) is attn_decode.cuh's.
//
// With codes n, and (s, m) of each key's group of 64 channels,
//     x_j = scale sum_g (s_jg (q_g . n_jg) + m_jg sum q_g),      p_j = 2^(x_j log2 e - max),
//     o_c = sum_j (p_j s_jg) (n_jc - 8) + sum_j p_j (m_jg + 8 s_jg)
// so that the products run on the codes themselves, and scales meet scores and weights, of
// which there are 1/64 as many.  Eight is the middle of the codes: sums of positive codes
// over many keys would be far larger than what remains of them.
//
// The products are m16n8k16 with the cache as the 16-row side, S^T = K q^T and O^T = V^T P^T,
// so that up to eight query heads cost no empty rows; units of 16 take two.  fp32 heads take
// two of the eight columns each, for the two parts that q and the weights are cut into.
//
// K: a code in an fp16 number's lowest bits is that number: the subnormals are n 2^-24, exact
// operands like any other.  A word's eight codes take four masks and a shift: at bits 4..7
// a code counts 16-fold, which q's side makes up for.  q is scaled by a power of two for the
// range of fp16.  V: 128 + n is 0x4300 | n in bf16, less 136; two keys' words are interleaved
// first, since the products add up over keys.  Weights times scales are bf16, as their range
// has no bound.
#include <cuda_fp16.h>

#include "attn_decode.cuh"
#include "cache_q4.cuh"

namespace kda {
namespace {
using namespace decode;

constexpr int kKeys = kQ4Keys;
constexpr float kMaxGrowth = 8.f;        // log2 of how far weights may exceed 1 before their maximum moves

// Per warp: a ring of tiles, each 16 keys' codes and scales of K and of V.
template <int D, int WARPS> struct Q4Smem {
    static constexpr int kCodes = kKeys * D / 2, kScales = kKeys * D / kQ4Group * 4, kTile = 2 * (kCodes + kScales);
    static constexpr int kFit = 216 * 1024 / (WARPS * kTile), kStages = kFit < 16 ? kFit : 16;
    static constexpr int kBytes = WARPS * kStages * kTile;
};

__device__ __forceinline__ uint32_t smem_u32(const void* p) { return (uint32_t)__cvta_generic_to_shared(p); }
// `bytes` of 16 bytes global -> shared, zeros behind them.
__device__ __forceinline__ void copy16(uint32_t dst, const void* src, int bytes) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(__cvta_generic_to_global(src)), "r"(bytes) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N> __device__ __forceinline__ void copy_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

__device__ __forceinline__ uint32_t lds32(uint32_t at) {
    uint32_t v;
    asm volatile("ld.shared.b32 %0, [%1];" : "=r"(v) : "r"(at) : "memory");
    return v;
}
__device__ __forceinline__ uint2 lds64(uint32_t at) {
    uint2 v;
    asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(at) : "memory");
    return v;
}
__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_bf16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// Transpose of an 8 x 8 matrix of 16-bit values, two a lane.
__device__ __forceinline__ uint32_t transpose(uint32_t x) {
    uint32_t y;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}
__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ uint32_t pack(float lo, float hi) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&v);
}
__device__ __forceinline__ uint32_t pack_half(float lo, float hi) {
    const __half2 v = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&v);
}
__device__ __forceinline__ float low_of(uint32_t x) { return __uint_as_float(x << 16); }             // bf16 pairs
__device__ __forceinline__ float high_of(uint32_t x) { return __uint_as_float(x & 0xFFFF0000u); }

// n - 8 in bf16 for the codes at bits 0..3 of both halves of x.
__device__ __forceinline__ uint32_t centred(uint32_t x) {
    const uint32_t y = (x & 0x000F000Fu) | 0x43004300u, middle = 0x43084308u;          // 128 + n, 136
    const __nv_bfloat162 v = __hsub2(*reinterpret_cast<const __nv_bfloat162*>(&y), *reinterpret_cast<const __nv_bfloat162*>(&middle));
    return *reinterpret_cast<const uint32_t*>(&v);
}

// Sixteen channels of q.
__device__ __forceinline__ void load16(const float* q, float (&x)[16]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float4 v = reinterpret_cast<const float4*>(q)[i];
        x[4 * i] = v.x, x[4 * i + 1] = v.y, x[4 * i + 2] = v.z, x[4 * i + 3] = v.w;
    }
}
__device__ __forceinline__ void load16(const __nv_bfloat16* q, float (&x)[16]) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const uint4 v = reinterpret_cast<const uint4*>(q)[i];
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int k = 0; k < 4; ++k) x[8 * i + 2 * k] = low_of(w[k]), x[8 * i + 2 * k + 1] = high_of(w[k]);
    }
}

// A unit's query heads are the columns of NT products of eight: all heads' own (bf16), or
// four heads twice, for both parts (fp32).
template <typename T, int D, int NT, int WARPS>
__global__ void __launch_bounds__(32 * WARPS, 1) decode_q4_kernel(const __grid_constant__ AttnDecodeQ4Launch launch) {
    using S = Q4Smem<D, WARPS>;
    constexpr bool kTwoParts = sizeof(T) == 4;
    constexpr int NG = D / kQ4Group, kStages = S::kStages, kColumns = kTwoParts ? 4 : 8, kRows = NT * kColumns;
    extern __shared__ __align__(128) uint8_t smem_raw[];
    const AttnDecodeLaunch& p = launch.base;
    start_after(p);
    const kda_attn_decode_args& a = p.a;
    const kda_cache_q4& cache = launch.cache;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int G = a.n_heads / a.n_kv_heads, blocks = (G + kRows - 1) / kRows;
    __shared__ PieceStart at_[WARPS];
    const Line line = find_pieces<32 * WARPS, WARPS>(p, a.n_kv_heads * blocks, kKeys, at_);
    griddep_launch();
    const int64_t piece = (int64_t)blockIdx.x * WARPS + warp;
    if (piece >= line.pieces) {
        if (lane == 0) p.open[piece] = make_int4(-1, 0, 0, 0);
        finish_empty<T, D>(p, piece, lane);
        return;
    }
    Cursor c = start(at_[warp], line, piece, a.n_kv_heads * blocks, kKeys);

    // ------------------------------------------------------------------ copies
    // The copies' own place on the line, kStages - 1 tiles ahead.  A group's 32 bytes of codes,
    // unit u = key * NG + g, lie at u ^ (u / 4 % 4): what eight lanes of a product read together
    // is in eight banks' worth of different places.
    Cursor f = c;
    const uint32_t ring = smem_u32(smem_raw) + (uint32_t)(warp * kStages * S::kTile);
    int32_t next_block = 0;                              // table entry of the place f
    const int page_shift = __ffs(a.block_size) - 1;
    auto look_up = [&]() {
        const int64_t key = f.info.x + f.k * kKeys;
        next_block = f.left > 0 && key < f.info.y ? a.block_table[(int64_t)f.s * a.table_stride + (key >> page_shift)] : -2;
    };
    auto fetch = [&](int stage) {
        if (f.left > 0) {
            const int64_t key = f.info.x + f.k * kKeys;
            int live = (int)max((int64_t)0, min((int64_t)kKeys, f.info.y - key));     // keys that exist
            if (live > 0 && (next_block < 0 || next_block >= cache.n_blocks)) {
                flag(p.status, KDA_DEV_BAD_SLOT);
                live = 0;
            }
            const int hk = blocks == 1 ? f.u : f.u / blocks;
            const int64_t row = live > 0 ? ((int64_t)next_block * a.n_kv_heads + hk) * a.block_size + (key & (a.block_size - 1)) : 0;
            const uint32_t to = ring + (uint32_t)(stage * S::kTile);
            const uint8_t* kc = static_cast<const uint8_t*>(cache.k_codes) + row * (D / 2);
            const uint8_t* vc = static_cast<const uint8_t*>(cache.v_codes) + row * (D / 2);
#pragma unroll
            for (int i = 0; i < S::kCodes / 16 / 32; ++i) {
                const int y = i * 32 + lane, u = y >> 1, bytes = u / NG < live ? 16 : 0;
                const uint32_t dst = to + (uint32_t)((u ^ (u >> 2 & 3)) * 32 + (y & 1) * 16);
                const int from = bytes ? y * 16 : 0;
                copy16(dst, kc + from, bytes);
                copy16(dst + S::kCodes, vc + from, bytes);
            }
            constexpr int kPieces = S::kScales / 16, kPieceKeys = 4 / NG;        // 16-byte pieces of the scales
            if (lane < 2 * kPieces) {
                const int y = lane % kPieces, bytes = max(0, min(16, (live - y * kPieceKeys) * NG * 4));
                const uint8_t* from = static_cast<const uint8_t*>(lane < kPieces ? cache.k_scales : cache.v_scales) + row * (NG * 4) + (bytes ? y * 16 : 0);
                copy16(to + 2 * S::kCodes + lane * 16, from, bytes);
            }
            f.step(p, kKeys);
            look_up();
        }
        copy_commit();
    };
    look_up();
#pragma unroll
    for (int i = 0; i < kStages - 1; ++i) fetch(i);

    // ------------------------------------------------------------------ units
    // Lane (n, t) of a product's operands: rows n and n + 8, columns 2 t and one more.
    const int n = lane >> 2, t = lane & 3;
    const float sc = a.scale * kLog2e;
    int stage = 0;
    while (c.left > 0) {
        const int64_t k_first = c.k, k_last = c.k + c.run();
        const int32_t s = c.s;
        const int hk = c.u / blocks, rb = c.u % blocks;
        const int head0 = hk * G + rb * kRows, rows = min(kRows, G - rb * kRows);
        const int2 info = c.info;

        // q of column n, 16 channels of each group from 64 g + 16 t, as the operands that meet
        // a word's codes: (0, 4), (1, 5) / 16, (2, 6), (3, 7) / 16.
        uint32_t q[NT][NG][2][4];
        float qsum[NT][2][NG], unscale[NT][2];           // of heads 2 t and 2 t + 1
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            const int r = nt * kColumns + n % kColumns;
            const bool live = r < rows;
            const T* qs = static_cast<const T*>(a.q) + s * a.q_stride + (int64_t)(head0 + (live ? r : 0)) * D + 16 * t;
            float x[NG][16], most = 0.f;
#pragma unroll
            for (int g = 0; g < NG; ++g) {
                load16(qs + g * kQ4Group, x[g]);
#pragma unroll
                for (int e = 0; e < 16; ++e) {
                    x[g][e] = live ? x[g][e] : 0.f;
                    most = fmaxf(most, fabsf(x[g][e]));
                }
            }
            most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, 1));
            most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, 2));
            // a power of two that brings the largest to 2^14 .. 2^15; its inverse is normal
            const int up = min(112, 14 - ((int)(__float_as_uint(most) >> 23) - 127));
            const float by = __uint_as_float((uint32_t)(up + 127) << 23);
            float undo = __uint_as_float((uint32_t)(127 - up) << 23), sum[NG];
#pragma unroll
            for (int g = 0; g < NG; ++g) {
                sum[g] = 0.f;
#pragma unroll
                for (int e = 0; e < 16; ++e) sum[g] += x[g][e], x[g][e] *= by;
                sum[g] += __shfl_xor_sync(0xffffffffu, sum[g], 1);
                sum[g] += __shfl_xor_sync(0xffffffffu, sum[g], 2);
                if (kTwoParts) {
#pragma unroll
                    for (int e = 0; e < 16; ++e) {
                        const float hi = __half2float(__float2half_rn(x[g][e]));
                        x[g][e] = n < 4 ? hi : x[g][e] - hi;
                    }
                }
#pragma unroll
                for (int w = 0; w < 2; ++w) {
                    const float* y = &x[g][8 * w];
                    q[nt][g][w][0] = pack_half(y[0], y[4]);
                    q[nt][g][w][1] = pack_half(y[1] * 0.0625f, y[5] * 0.0625f);
                    q[nt][g][w][2] = pack_half(y[2], y[6]);
                    q[nt][g][w][3] = pack_half(y[3] * 0.0625f, y[7] * 0.0625f);
                }
            }
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                unscale[nt][e] = __shfl_sync(0xffffffffu, undo, 4 * (2 * t + e));
#pragma unroll
                for (int g = 0; g < NG; ++g) qsum[nt][e][g] = __shfl_sync(0xffffffffu, sum[g], 4 * (2 * t + e)) * sc;
            }
        }

        float o[NT][NG * 4][4], m[NT][2], l[NT][2], low[NT][2][NG];      // low: sum of p (m + 8 s)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
            for (int i = 0; i < NG * 4; ++i) o[nt][i][0] = o[nt][i][1] = o[nt][i][2] = o[nt][i][3] = 0.f;
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                m[nt][e] = -CUDART_INF_F, l[nt][e] = 0.f;
#pragma unroll
                for (int g = 0; g < NG; ++g) low[nt][e][g] = 0.f;
            }
        }

        for (int64_t kt = k_first; kt < k_last; ++kt) {
            copy_wait<kStages - 2>();
            __syncwarp();                                // the tile is there, and the stage before it is read
            fetch(stage == 0 ? kStages - 1 : stage - 1);
            const uint32_t kb = ring + (uint32_t)(stage * S::kTile), vb = kb + S::kCodes, sb = vb + S::kCodes;
            stage = stage == kStages - 1 ? 0 : stage + 1;
            const int live = (int)max((int64_t)0, min((int64_t)kKeys, info.y - (info.x + kt * kKeys)));

            // scores of keys n and n + 8 (r), heads 2 t + e
            float x[NT][2][2] = {};
#pragma unroll
            for (int g = 0; g < NG; ++g) {
                uint2 w[2];
                uint32_t scale[2];
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    const int u = (n + 8 * r) * NG + g;
                    w[r] = lds64(kb + (uint32_t)((u ^ (u >> 2 & 3)) * 32 + t * 8));
                    scale[r] = lds32(sb + (uint32_t)u * 4);
                }
                float acc[NT][4] = {};
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const uint32_t w0 = h ? w[0].y : w[0].x, w1 = h ? w[1].y : w[1].x, v0 = w0 >> 8, v1 = w1 >> 8;
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) {
                        mma_f16(acc[nt], w0 & 0x000F000Fu, w1 & 0x000F000Fu, w0 & 0x00F000F0u, w1 & 0x00F000F0u, q[nt][g][h][0], q[nt][g][h][1]);
                        mma_f16(acc[nt], v0 & 0x000F000Fu, v1 & 0x000F000Fu, v0 & 0x00F000F0u, v1 & 0x00F000F0u, q[nt][g][h][2], q[nt][g][h][3]);
                    }
                }
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int r = 0; r < 2; ++r)
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            float y = acc[nt][2 * r + e];
                            if (kTwoParts) y += __shfl_xor_sync(0xffffffffu, y, 2);
                            y = y * 0x1p24f * unscale[nt][e] * sc;
                            x[nt][r][e] += fmaf(y, low_of(scale[r]), high_of(scale[r]) * qsum[nt][e][g]);
                        }
            }
            if (live < kKeys) {
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int r = 0; r < 2; ++r)
                        if (n + 8 * r >= live) x[nt][r][0] = x[nt][r][1] = -CUDART_INF_F;
            }
            bool grow = false;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const float mx = fmaxf(x[nt][0][e], x[nt][1][e]);
                    grow |= mx - m[nt][e] > kMaxGrowth;              // (false for -inf less -inf)
                }
            if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        float mx = fmaxf(x[nt][0][e], x[nt][1][e]);
#pragma unroll
                        for (int off = 4; off < 32; off <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, off));
                        mx = fmaxf(m[nt][e], mx);
                        const float w = m[nt][e] == -CUDART_INF_F ? 0.f : ex2(m[nt][e] - mx);
                        m[nt][e] = mx;
                        l[nt][e] *= w;
#pragma unroll
                        for (int g = 0; g < NG; ++g) low[nt][e][g] *= w;
#pragma unroll
                        for (int i = 0; i < NG * 4; ++i) {
                            o[nt][i][e] *= w;
                            o[nt][i][2 + e] *= w;
                        }
                    }
            }
            // weights, in place of the scores
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const float off = m[nt][e] == -CUDART_INF_F ? 0.f : m[nt][e];
#pragma unroll
                    for (int r = 0; r < 2; ++r) {
                        x[nt][r][e] = ex2(x[nt][r][e] - off);
                        l[nt][e] += x[nt][r][e];
                    }
                }
#pragma unroll
            for (int g = 0; g < NG; ++g) {
                uint32_t b[NT][2];                       // weights times scales, turned to heads n, keys 2 t, 2 t + 1 (+ 8)
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    const uint32_t scale = lds32(sb + S::kScales + (uint32_t)((n + 8 * r) * NG + g) * 4);
                    const float step = low_of(scale), mid = fmaf(8.f, step, high_of(scale));
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) {
                        float w[2];
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            low[nt][e][g] = fmaf(x[nt][r][e], mid, low[nt][e][g]);
                            w[e] = x[nt][r][e] * step;
                            if (kTwoParts) {
                                const float hi = __bfloat162float(__float2bfloat16_rn(w[e]));
                                w[e] = t < 2 ? hi : w[e] - hi;
                            }
                        }
                        b[nt][r] = transpose(pack(w[0], w[1]));
                    }
                }
                uint32_t v[2][2];                        // channels 64 g + 8 n .. of keys 2 t, 2 t + 1 (+ 8)
#pragma unroll
                for (int r = 0; r < 2; ++r)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const int u = (2 * t + e + 8 * r) * NG + g;
                        v[r][e] = lds32(vb + (uint32_t)((u ^ (u >> 2 & 3)) * 32 + n * 4));
                    }
                const uint32_t a0 = __byte_perm(v[0][0], v[0][1], 0x5410), a1 = __byte_perm(v[0][0], v[0][1], 0x7632);   // channels 0-3, 4-7
                const uint32_t c0 = __byte_perm(v[1][0], v[1][1], 0x5410), c1 = __byte_perm(v[1][0], v[1][1], 0x7632);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const uint32_t y = i < 2 ? a0 : a1, z = i < 2 ? c0 : c1;
                    const int at = 8 * (i & 1);
                    const uint32_t f0 = centred(y >> at), f1 = centred(y >> (at + 4)), f2 = centred(z >> at), f3 = centred(z >> (at + 4));
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) mma_bf16(o[nt][g * 4 + i], f0, f1, f2, f3, b[nt][0], b[nt][1]);
                }
            }
            __syncwarp();                                // all lanes have read the stage
        }

        // Lane (n, t) has channels 64 g + 8 n .. of heads 2 t + e; both parts' lanes the same.
        const bool whole = k_first == 0 && k_last == c.T;
        const int n_pre = whole ? prefix_parts(p, info.x) : 0;
        if (n_pre > 0) griddep_wait();                   // the prefix's results
        const int64_t slot = part_slot(piece, k_first == 0);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                float lt = l[nt][e], mt = m[nt][e], y[NG][8];
#pragma unroll
                for (int off = 4; off < 32; off <<= 1) lt += __shfl_xor_sync(0xffffffffu, lt, off);
#pragma unroll
                for (int g = 0; g < NG; ++g) {
                    float base = low[nt][e][g];
#pragma unroll
                    for (int off = 4; off < 32; off <<= 1) base += __shfl_xor_sync(0xffffffffu, base, off);
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        y[g][i] = o[nt][g * 4 + i / 2][(i & 1) * 2 + e];
                        if (kTwoParts) y[g][i] += __shfl_xor_sync(0xffffffffu, y[g][i], 2);
                        y[g][i] += base;
                    }
                }
                const int rr = nt * kColumns + (kTwoParts ? (2 * t + e) & 3 : 2 * t + e), head = head0 + rr;
                if (rr >= rows || (kTwoParts && t >= 2)) continue;
#pragma unroll 2
                for (int i = 0; i < n_pre; ++i) {
                    const int64_t pr = prefix_row(p, i, s, head);
                    const float2 ml = p.pre_ml[pr];
                    float w, w2;
                    join(mt, lt, ml.x, ml.y, w, w2);
#pragma unroll
                    for (int g = 0; g < NG; ++g)
#pragma unroll
                        for (int k = 0; k < 8; k += 4) {
                            const float4 v = *reinterpret_cast<const float4*>(p.pre_o + pr * D + g * kQ4Group + 8 * n + k);
                            y[g][k] = y[g][k] * w + v.x * w2;
                            y[g][k + 1] = y[g][k + 1] * w + v.y * w2;
                            y[g][k + 2] = y[g][k + 2] * w + v.z * w2;
                            y[g][k + 3] = y[g][k + 3] * w + v.w * w2;
                        }
                }
                if (whole) {
                    const float inv = lt == 0.f ? 0.f : 1.f / lt;
                    T* out = static_cast<T*>(a.o) + s * a.o_stride + (int64_t)head * D + 8 * n;
#pragma unroll
                    for (int g = 0; g < NG; ++g) {
                        if (kTwoParts) {
#pragma unroll
                            for (int k = 0; k < 8; k += 4)
                                *reinterpret_cast<float4*>(out + g * kQ4Group + k) =
                                    make_float4(y[g][k] * inv, y[g][k + 1] * inv, y[g][k + 2] * inv, y[g][k + 3] * inv);
                        } else {
                            *reinterpret_cast<uint4*>(out + g * kQ4Group) =
                                make_uint4(pack(y[g][0] * inv, y[g][1] * inv), pack(y[g][2] * inv, y[g][3] * inv),
                                           pack(y[g][4] * inv, y[g][5] * inv), pack(y[g][6] * inv, y[g][7] * inv));
                        }
                    }
                    if (n == 0) write_lse(a, s, head, mt, lt);
                } else {
                    float* out = p.part_o + (slot * kRows + rr) * D + 8 * n;
#pragma unroll
                    for (int g = 0; g < NG; ++g)
#pragma unroll
                        for (int k = 0; k < 8; k += 4)
                            *reinterpret_cast<float4*>(out + g * kQ4Group + k) = make_float4(y[g][k], y[g][k + 1], y[g][k + 2], y[g][k + 3]);
                    if (n == 0) p.part_ml[slot * kRows + rr] = make_float2(mt, lt);
                }
            }
        __syncwarp();
        if (lane == 0 && c.left == c.run()) p.open[piece] = open_unit(p, c, piece, line);
        c.next_unit(p, kKeys);
    }
    copy_wait<0>();
    finish_empty<T, D>(p, piece, lane);
}

template <typename T, int D, int NT>
cudaError_t launch_t(const AttnDecodeQ4Launch& p, cudaStream_t s) {
    constexpr int WARPS = q4_warps(NT);
    constexpr int kRows = NT * (sizeof(T) == 4 ? 4 : 8), kBytes = Q4Smem<D, WARPS>::kBytes;
    cudaError_t e = cudaFuncSetAttribute(decode_q4_kernel<T, D, NT, WARPS>, cudaFuncAttributeMaxDynamicSharedMemorySize, kBytes);
    if (e != cudaSuccess) return e;
    note_launch();
    e = launch_overlapped(decode_q4_kernel<T, D, NT, WARPS>, dim3(p.base.n_pieces / WARPS), dim3(32 * WARPS), kBytes, s, p);
    return e == cudaSuccess ? launch_join<T, D, kRows>(p.base, s) : e;
}
template <typename T, int D>
cudaError_t launch_d(const AttnDecodeQ4Launch& p, cudaStream_t s) {
    return q4_columns(p.base.a.dtype, p.base.a.n_heads / p.base.a.n_kv_heads) == 1 ? launch_t<T, D, 1>(p, s) : launch_t<T, D, 2>(p, s);
}

}  // namespace

cudaError_t launch_decode_q4(const AttnDecodeQ4Launch& p, cudaStream_t s) {
    if (p.base.a.dtype == KDA_BF16) return p.base.a.d == 128 ? launch_d<__nv_bfloat16, 128>(p, s) : launch_d<__nv_bfloat16, 64>(p, s);
    return p.base.a.d == 128 ? launch_d<float, 128>(p, s) : launch_d<float, 64>(p, s);
}

}  // namespace kda
