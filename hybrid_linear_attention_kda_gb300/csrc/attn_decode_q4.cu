// Decode attention over the 4-bit cache.  The division of work (a line of tiles of 32 keys,
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
// a code counts 16-fold, which q's side makes up for.  Each group of q is scaled by a power of two
// for the range of fp16.  (fp32 takes centred codes here too, and q's sum times m + 8 s: what the
// tensor cores cut off of larger sums would be more than fp32 loses.)
//
// V: the products add up over keys, so that a byte of codes has to meet the same byte of the
// next key: ldmatrix transposes bytes, a permutation puts 0x64 behind each, which makes 1024 +
// byte of it, and one fp16 instruction n - 8 of each of its codes.  A product's rows are the
// keys in the order in which that hands them out.  Weights times scales are rounded to fp16: 11
// bits, counted from the largest so far of each head and group (a power of two, moved like the
// weights' own maximum: unit_up).
//
// Bound, on long sequences, by the cache's bytes and the instructions that take codes apart: 321
// a warp for 16 keys of d = 128, 104 of them (by the source) masks, permutations and conversions of
// codes; the ALU and issue slots are 54% and 64% busy, DRAM 89% of the measured copy rate between
// the beginning and the end.  One sequence of 2^20 tokens, 8 key/value heads: 0.22 ms (5.4 TB/s), of
// which 23 us do not grow with the length; in bf16 it takes 0.68 ms (32 query heads).  512
// sequences of up to 2048: 128 us (4.7 TB/s).  16 query heads a key/value head: 0.34 ms, where
// twice the rows make arithmetic of it (0.42 ms in units of eight).  7 requests of up to 700
// tokens: 15 us, a chain of about ten trips to memory in two kernels.
//
// Twelve warps a block, three a scheduler, have 168 registers (one sequence of 2^20 223 us;
// sixteen with 128, 237 us).  The copies are cp.async by each warp for itself:
// a copy warp that served the others with bulk and tensor copies of 1 KB took 0.57 ms, since such
// copies leave a warp one lane at a time.
#include <cuda_fp16.h>
#include <float.h>

#include "attn_decode.cuh"
#include "cache_q4.cuh"

namespace kda {
namespace {
using namespace decode;

constexpr int kKeys = kQ4Keys;
constexpr float kMaxGrowth = 8.f;        // log2 of how far weights may exceed 1 before their maximum moves
constexpr float kMostWeight = 0x1p15f;   // times scale, in units: below fp16's largest
// A weight (up to 2^8) times the unit stays finite, so that a weight of zero gives zeros whatever
// its scale is.  (Scale times unit may not: a unit that was set by tiny scales meets a large one.)
constexpr int kMostUnit = 118;           // log2

// Per warp: a ring of tiles, each two halves of 16 keys, which may lie in two pages; codes
// of K, codes of V, scales of K, scales of V.
constexpr int kHalf = kKeys / 2;
template <int D, int WARPS> struct Q4Smem {
    static constexpr int kCodes = kKeys * D / 2, kScales = kKeys * D / kQ4Group * 4, kTile = 2 * (kCodes + kScales);
    static constexpr int kStages = 222 * 1024 / (WARPS * kTile), kBytes = WARPS * kStages * kTile;
};

__device__ __forceinline__ uint32_t smem_u32(const void* p) { return (uint32_t)__cvta_generic_to_shared(p); }
__device__ __forceinline__ void copy16(uint32_t dst, const void* src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(__cvta_generic_to_global(src)) : "memory");
}
// `bytes` of 16 bytes global -> shared, zeros behind them.
__device__ __forceinline__ void copy16(uint32_t dst, const void* src, int bytes) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(__cvta_generic_to_global(src)), "r"(bytes) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N> __device__ __forceinline__ void copy_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

// All of a half tile that is this lane's: every 16th piece of its codes, alternately from c0 and
// c1 on, and one of its scales.
template <int D>
__device__ __forceinline__ void copy_half(uint32_t c0, uint32_t c1, uint32_t sc, const uint8_t* k, const uint8_t* v, const uint8_t* from, int l16) {
    constexpr int kCodes = kKeys * D / 2;
#pragma unroll
    for (int i = 0; i < kCodes / 512; ++i) {
        copy16((i & 1 ? c1 : c0) + (i & ~1) * 256, k + i * 256);
        copy16((i & 1 ? c1 : c0) + (i & ~1) * 256 + kCodes, v + i * 256);
    }
    if (D == 128 || l16 < 8) copy16(sc, from);
}

// (What cp.async brings is there after its wait, which these loads do not pass.)
__device__ __forceinline__ uint32_t lds32(uint32_t at) {
    return *reinterpret_cast<const uint32_t*>(__cvta_shared_to_generic(at));
}
__device__ __forceinline__ uint2 lds64(uint32_t at) {
    return *reinterpret_cast<const uint2*>(__cvta_shared_to_generic(at));
}
// The scale pairs of one key.
template <int NG> __device__ __forceinline__ void load_scales(uint32_t (&scale)[2], uint32_t at) {
    if (NG == 2) {
        const uint2 v = lds64(at);
        scale[0] = v.x, scale[1] = v.y;
    } else {
        scale[0] = scale[1] = lds32(at);
    }
}
__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// The first product of a sum.
__device__ __forceinline__ void mma_f16_first(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
                 : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}
__device__ __forceinline__ void mma_bf16_k8(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t b0) {
    asm("mma.sync.aligned.m16n8k8.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5}, {%6}, {%7,%7,%7,%7};"
                 : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
                 : "r"(a0), "r"(a1), "r"(b0), "f"(0.f));
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
__device__ __forceinline__ uint32_t pack_half(float lo, float hi) {
    const __half2 v = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&v);
}
__device__ __forceinline__ float low_of(uint32_t x) { return __uint_as_float(x << 16); }             // bf16 pairs
__device__ __forceinline__ float high_of(uint32_t x) { return __uint_as_float(x & 0xFFFF0000u); }

// Two 16 x 16 blocks of bytes, transposed: r[2 i + h] holds column lane / 4 + 8 h of block i,
// rows 4 (lane % 4) .. + 3.  Lanes name the blocks' rows, 16 bytes each.
__device__ __forceinline__ void ldsm_bytes(uint32_t (&r)[4], uint32_t at) {
    asm volatile("ldmatrix.sync.aligned.m16n16.x2.trans.shared.b8 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(at)
                 : "memory");
}
// n - 8 in fp16 for the lower and the upper codes of two bytes of x (0 and 1, or 2 and 3).  With
// a byte c, 0x6400 | c is 1024 + c; without its lower code but 8 in its place, 1024 + 16 n + 8.
template <int PICK> __device__ __forceinline__ void centred(uint32_t x, uint32_t& lower, uint32_t& upper) {
    const uint32_t both = __byte_perm(x, 0x64u, PICK == 0 ? 0x4140 : 0x4342);
    const uint32_t rest = (both & 0xFFF0FFF0u) | 0x00080008u, by = 0x2C002C00u, middle = 0xD488D488u;      // 1 / 16, -72.5
    const __half2 h = *reinterpret_cast<const __half2*>(&both), r = *reinterpret_cast<const __half2*>(&rest);
    const __half2 lo = __hsub2(h, r), hi = __hfma2(r, *reinterpret_cast<const __half2*>(&by), *reinterpret_cast<const __half2*>(&middle));
    lower = *reinterpret_cast<const uint32_t*>(&lo), upper = *reinterpret_cast<const uint32_t*>(&hi);
}

// n - 8 in fp16 for the codes at bits 0..3, and at bits 4..7, of both halves of x.
__device__ __forceinline__ uint32_t centred_low(uint32_t x) {
    const uint32_t y = (x & 0x000F000Fu) | 0x64006400u, middle = 0x64086408u;                              // 1024 + n, 1032
    const __half2 v = __hsub2(*reinterpret_cast<const __half2*>(&y), *reinterpret_cast<const __half2*>(&middle));
    return *reinterpret_cast<const uint32_t*>(&v);
}
__device__ __forceinline__ uint32_t centred_high(uint32_t x) {
    const uint32_t y = (x & 0x00F000F0u) | 0x64006400u, by = 0x2C002C00u, middle = 0xD480D480u;            // 1024 + 16 n, 1 / 16, -72
    const __half2 v = __hfma2(*reinterpret_cast<const __half2*>(&y), *reinterpret_cast<const __half2*>(&by), *reinterpret_cast<const __half2*>(&middle));
    return *reinterpret_cast<const uint32_t*>(&v);
}

// x as the sum of three bf16 numbers: the i-th, nothing where i is 3.
__device__ __forceinline__ float third(float x, int i) {
    const float a = __bfloat162float(__float2bfloat16_rn(x)), b = __bfloat162float(__float2bfloat16_rn(x - a));
    return i == 0 ? a : i == 1 ? b : i == 2 ? __bfloat162float(__float2bfloat16_rn(x - a - b)) : 0.f;
}

// Sixteen channels of q as they lie in memory.
template <typename T> struct Raw16 {
    uint4 r[sizeof(T)];
    __device__ __forceinline__ void load(const T* q) {
#pragma unroll
        for (int i = 0; i < (int)sizeof(T); ++i) r[i] = reinterpret_cast<const uint4*>(q)[i];
    }
    __device__ __forceinline__ void open(float (&x)[16]) const {
#pragma unroll
        for (int i = 0; i < (int)sizeof(T); ++i) {
            const uint32_t w[4] = {r[i].x, r[i].y, r[i].z, r[i].w};
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                if (sizeof(T) == 4) x[4 * i + k] = __uint_as_float(w[k]);
                else x[(8 * i + 2 * k) & 15] = low_of(w[k]), x[(8 * i + 2 * k + 1) & 15] = high_of(w[k]);
            }
        }
    }
};

__device__ __forceinline__ void write2(float* to, float x, float y) { *reinterpret_cast<float2*>(to) = make_float2(x, y); }
__device__ __forceinline__ void write2(__nv_bfloat16* to, float x, float y) { *reinterpret_cast<__nv_bfloat162*>(to) = __floats2bfloat162_rn(x, y); }

// By how many powers of two the unit of a head's and group's weights is to move, so that the
// tile's largest weight, `most` * 2^10, lies at 2^6 .. 2^7 of it: then weights have 11 bits
// down to 2^-20 of the largest and may grow by 2^8.  Upwards only where the sums so far have
// shrunk (by `shrunk`; 0: there were none): then unit_room says how far.  The unit starts at its
// largest, where hardly a weight fits: the first one that is not zero (of a group whose first
// values have no width) moves it down.
__device__ __forceinline__ int unit_up(float most, float shrunk, float unit) {
    if (!(most > 0.f)) return 0;
    const int at = (int)(__float_as_uint(unit) >> 23) - 127;
    int up = 6 - 10 - ((int)(__float_as_uint(most) >> 23) - 127) - at;
    if (shrunk == 1.f) up = min(up, 0);
    return max(-120 - at, min(kMostUnit - at, up));                  // the unit and its inverse stay normal
}
// How far the unit may move up before a sum of magnitude `sum` is past 2^40 of it, where fp32 keeps
// less of the sum than fp16 of the weights.  2^31 keys add 2^49 at most (2^15 times a code each).
__device__ __forceinline__ int unit_room(float sum) { return max(0, 40 + 127 - (int)(__float_as_uint(sum) >> 23)); }
__device__ __forceinline__ float two_to(int i) { return __uint_as_float((uint32_t)(i + 127) << 23); }

// A worker's place on the line: unit u of sequence s at tile k of its T.  A unit takes some
// places more than it has tiles (kQ4Pad), for the time that its beginning and end take; a piece
// that ends among those holds the unit to its end, one that starts there starts with the next.
struct Place {
    int64_t left;      // of the piece from here on
    int32_t s, u, units;
    int32_t k, T;
    int2 info;

    __device__ __forceinline__ int run() const { return (int)min((int64_t)(T - k), left); }
    __device__ __forceinline__ bool whole() const { return k == 0 && left >= T; }
    __device__ __forceinline__ void next_unit(const AttnDecodeLaunch& p) {
        left -= T + kQ4Pad - k;
        k = 0;
        if (++u < units || left <= 0) return;
        u = 0;
        do {
            info = seq_info(p, ++s);
            T = (int)seq_tiles(info, kKeys);
        } while (T == 0);
    }
    __device__ __forceinline__ Place() {}
    __device__ __forceinline__ Place(const AttnDecodeLaunch& p, const PieceStart& at, int64_t length, int units_) {
        left = length, s = at.s, units = units_, info = at.info;
        T = (int)seq_tiles(info, kKeys);
        u = (int32_t)divide(at.rel, T + kQ4Pad);
        k = (int32_t)(at.rel - (int64_t)u * (T + kQ4Pad));
        if (k >= T) next_unit(p);
    }
};

// A unit's query heads are the columns of NT products of eight: all heads' own (bf16), or
// four heads twice, for both parts (fp32).
template <typename T, int D, int NT, int WARPS>
__global__ void __launch_bounds__(32 * WARPS, 1) decode_q4_kernel(const __grid_constant__ AttnDecodeQ4Launch launch) {
    using S = Q4Smem<D, WARPS>;
    constexpr bool kTwoParts = sizeof(T) == 4;
    constexpr float kUpper = kTwoParts ? 1.f : 0.0625f;  // what q's channels take that meet codes which count 16-fold
    constexpr int NG = D / kQ4Group, kStages = S::kStages, kColumns = kTwoParts ? 4 : 8, kRows = NT * kColumns;
    extern __shared__ __align__(128) uint8_t smem_raw[];
    const AttnDecodeLaunch& p = launch.base;
    start_after(p);
    const kda_attn_decode_args& a = p.a;
    const kda_cache_q4& cache = launch.cache;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int G = a.n_heads / a.n_kv_heads, blocks = (G + kRows - 1) / kRows;
    __shared__ PieceStart at_[WARPS];
    const Line line = find_pieces<32 * WARPS, WARPS>(p, a.n_kv_heads * blocks, kKeys, at_, kQ4Pad);
    griddep_launch();
    const int64_t piece = (int64_t)blockIdx.x * WARPS + warp;
    Place first;
    first.left = 0;
    if (piece < line.pieces) first = Place(p, at_[warp], line.begin(piece + 1) - line.begin(piece), a.n_kv_heads * blocks);
    if (first.left <= 0) {
        if (lane == 0) p.open[piece] = make_int4(-1, 0, 0, 0);
        finish_empty<T, D>(p, piece, lane);
        return;
    }
    // The places on the line are looked at where units begin and end: they wait in shared memory
    // meanwhile, which leaves the registers to the tiles.
    __shared__ Place here[WARPS], ahead[WARPS];
    here[warp] = ahead[warp] = first;
    __syncwarp();

    // ------------------------------------------------------------------ copies
    // The copies' own place on the line, kStages - 1 tiles ahead: cursor f at the first tile of
    // a run within one unit, f_run tiles of it to come, key f_key next.  Sixteen lanes copy a
    // half of the tile.  A group's 32 bytes of codes, unit u = key * NG + g of its half, lie at
    // u ^ (u / 4 % 4): what eight lanes of a product read together is in eight banks' worth of
    // different places.
    const uint32_t ring = smem_u32(smem_raw) + (uint32_t)(warp * kStages * S::kTile);
    const int page_shift = __ffs(a.block_size) - 1, half = lane >> 4, l16 = lane & 15;
    const int page_mask = a.block_size - 1;
    const uint32_t page_rows = (uint32_t)(a.n_kv_heads * a.block_size), n_blocks = (uint32_t)cache.n_blocks;
    int f_run, f_key, f_end;
    uint32_t f_head_row;
    const int32_t* f_row;
    // Table entries of this half's tiles, a lane each: sixteen from the present batch's first on, and
    // the sixteen behind them.
    int32_t entries = -1, entries_on = -1;
    int f_tile = 0;                                      // of the batch
    // places in shared memory: piece y = 16 i + l16 of a half's codes, and one piece of its scales
    constexpr int kPieces = S::kScales / 2 / 16, kPieceKeys = 4 / NG;
    const int scale_piece = l16 % kPieces, scale_is_v = l16 / kPieces;
    const uint32_t code0 = ring + half * (S::kCodes / 2) + (l16 >> 3) * 128 + ((l16 & 7) ^ (l16 >> 3) * (NG == 2 ? 1 : 5)) * 16;
    const uint32_t scale_to = ring + 2 * S::kCodes + scale_is_v * S::kScales + half * (S::kScales / 2) + scale_piece * 16;
    auto code_to = [&](uint32_t tile, int i) { return ((code0 + tile) ^ (NG == 2 ? 32 * i : 0)) + i * 256; };     // i: 0, 1; then 512 on
    const uint8_t* k_from = static_cast<const uint8_t*>(cache.k_codes) + l16 * 16;
    const uint8_t* v_from = static_cast<const uint8_t*>(cache.v_codes) + l16 * 16;
    const uint8_t* scale_from = static_cast<const uint8_t*>(scale_is_v ? cache.v_scales : cache.k_scales) + scale_piece * 16;
    auto look_up = [&](int ahead_by) {
        const uint32_t key = (uint32_t)f_key + (uint32_t)((ahead_by + l16) * kKeys);
        return key < (uint32_t)f_end ? f_row[key >> page_shift] : -1;
    };
    auto enter = [&](const Place& f) {
        f_run = f.run(), f_key = f.info.x + f.k * kKeys + half * kHalf, f_end = f.info.y;
        f_head_row = (uint32_t)(f.u / blocks * a.block_size);
        f_row = a.block_table + (int64_t)f.s * a.table_stride;
        f_tile = 0, entries = look_up(0), entries_on = look_up(16);
    };
    enter(ahead[warp]);
    auto fetch = [&](int stage) {
        if (f_run > 0) {
            const uint32_t to = (uint32_t)(stage * S::kTile);
            const int live = f_end - f_key;                                  // keys from here on
            const int32_t next_block = __shfl_sync(0xffffffffu, entries, (lane & 16) | f_tile);
            const bool known = (uint32_t)next_block < n_blocks;
            // (rows are below 2^31; a half lies in one page, so that those of missing keys may be named too)
            const uint32_t row = (uint32_t)next_block * page_rows + (f_head_row + (f_key & page_mask));
            if (__all_sync(0xffffffffu, known && live >= kHalf)) {
                copy_half<D>(code_to(to, 0), code_to(to, 1), scale_to + to, k_from + (uint64_t)row * (D / 2), v_from + (uint64_t)row * (D / 2),
                             scale_from + (uint64_t)row * (NG * 4), l16);
            } else {
                if (live > 0 && !known) flag(p.status, KDA_DEV_BAD_SLOT);
                const int have = known ? max(0, min(kHalf, live)) : 0;
                const uint64_t from = have > 0 ? row : 0;
#pragma unroll
                for (int i = 0; i < S::kCodes / 2 / 256; ++i) {
                    const int bytes = (i * 16 + l16) / (2 * NG) < have ? 16 : 0;
                    copy16(code_to(to, i & 1) + (i & ~1) * 256, k_from + from * (D / 2) + i * 256, bytes);
                    copy16(code_to(to, i & 1) + (i & ~1) * 256 + S::kCodes, v_from + from * (D / 2) + i * 256, bytes);
                }
                if (l16 < 2 * kPieces) copy16(scale_to + to, scale_from + from * (NG * 4), max(0, min(16, (have - scale_piece * kPieceKeys) * NG * 4)));
            }
            f_key += kKeys;
            if (--f_run == 0) {
                Place f = ahead[warp];
                f.next_unit(p);
                __syncwarp();
                ahead[warp] = f;
                __syncwarp();
                if (f.left > 0) enter(f);
            } else if (++f_tile == 16) {
                f_tile = 0, entries = entries_on, entries_on = look_up(16);
            }
        }
        copy_commit();
    };

    // ------------------------------------------------------------------ units
    // Lane (n, t) of a product's operands: rows n and n + 8, columns 2 t and one more.
    const int n = lane >> 2, t = lane & 3;
    const float sc = a.scale * kLog2e;
    // Row n + 8 r of a half's products is key own_key + 2 r.  The lane's eight bytes of its K codes
    // of group g lie at k_at(r, g), the 16 bytes that it names to ldmatrix at v0 ^ 32 g.  (The
    // tile starts at a multiple of 128 bytes, so that places are sums and exclusive ors.)
    const int own_key = 4 * (n >> 1) + (n & 1), v_key = lane & 15, v_line = v_key * NG >> 2;
    const uint32_t k0 = ring + (NG == 2 ? (n >> 1) * 256 + (((n & 1) * 4 + (t >> 1)) ^ (n & 2)) * 16
                                        : (n >> 1) * 128 + (((n & 1) * 2 + (t >> 1)) ^ (n >> 1 & 1) * 5) * 16) + (t & 1) * 8;
    const uint32_t v0 = ring + S::kCodes + v_line * 128 + ((v_key * 2 * NG + (lane >> 4) & 7) ^ (NG == 2 ? v_line & 3 : (v_line & 1) * 5)) * 16;
    const uint32_t s0 = ring + 2 * S::kCodes + own_key * NG * 4;
    auto k_at = [](uint32_t k, int r, int g) { return NG == 2 ? (k ^ (g * 32 + r * 16)) + r * 128 : k ^ r * 64; };
    int stage = 0;
    bool more = true, begun = false;
    while (more) {
        int kt, live;                                    // tiles of the unit in this piece, keys from the first one on
        const Place c = here[warp];
        kt = c.run(), live = c.info.y - (c.info.x + c.k * kKeys);

        // q of column n, 16 channels of each group from 64 g + 16 t, as the operands that meet
        // a word's codes: (0, 4), (1, 5) / 16, (2, 6), (3, 7) / 16.
        Raw16<T> raw[NT][NG];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            const int r = min(nt * kColumns + n % kColumns, min(kRows, G - c.u % blocks * kRows) - 1);
            const T* qs = static_cast<const T*>(a.q) + c.s * a.q_stride + (int64_t)(c.u / blocks * G + c.u % blocks * kRows + r) * D + 16 * t;
#pragma unroll
            for (int g = 0; g < NG; ++g) raw[nt][g].load(qs + g * kQ4Group);
        }
        if (!begun) {                                    // the first copies, while q is on its way
            begun = true;
#pragma unroll
            for (int i = 0; i < kStages - 1; ++i) fetch(i);
        }
        uint32_t q[NT][NG][2][4];
        uint32_t qsum[NT];                               // of column n, part t of three, both groups, times scale log2 e
        float unscale[NT][2][NG], sums[NT][2][NG];       // of heads 2 t and 2 t + 1, times that too; sums: fp32 only
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            const int r = nt * kColumns + n % kColumns;
            const bool is_row = r < min(kRows, G - c.u % blocks * kRows);
            float x[NG][16], undo[NG], sum[NG];
#pragma unroll
            for (int g = 0; g < NG; ++g) {
                float most = 0.f;
                raw[nt][g].open(x[g]);
#pragma unroll
                for (int e = 0; e < 16; ++e) {
                    x[g][e] = is_row ? x[g][e] : 0.f;
                    most = fmaxf(most, fabsf(x[g][e]));
                }
                most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, 1));
                most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, 2));
                // a power of two that brings the group's largest to 2^14 .. 2^15; its inverse is normal
                const int up = min(112, 14 - ((int)(__float_as_uint(most) >> 23) - 127));
                const float by = __uint_as_float((uint32_t)(up + 127) << 23);
                undo[g] = __uint_as_float((uint32_t)(127 - up) << 23);
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
                    q[nt][g][w][1] = pack_half(y[1] * kUpper, y[5] * kUpper);
                    q[nt][g][w][2] = pack_half(y[2], y[6]);
                    q[nt][g][w][3] = pack_half(y[3] * kUpper, y[7] * kUpper);
                }
            }
#pragma unroll
            for (int e = 0; e < 2; ++e)
#pragma unroll
                for (int g = 0; g < NG; ++g) {
                    unscale[nt][e][g] = __shfl_sync(0xffffffffu, undo[g], 4 * (2 * t + e)) * (kTwoParts ? 1.f : 0x1p24f) * sc;
                    if (kTwoParts) sums[nt][e][g] = __shfl_sync(0xffffffffu, sum[g], 4 * (2 * t + e)) * sc;
                }
            const float lower = third(sum[0] * sc, t), upper = NG == 2 ? third(sum[NG - 1] * sc, t) : 0.f;
            qsum[nt] = __float_as_uint(lower) >> 16 | (__float_as_uint(upper) & 0xFFFF0000u);
        }

        // o: sum of weights times codes, in units of 1 / unit; low: sum of p (m + 8 s)
        float o[NT][NG * 4][4], m[NT][2], l[NT][2], low[NT][2][NG], unit[NT][2][NG];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
            for (int i = 0; i < NG * 4; ++i) o[nt][i][0] = o[nt][i][1] = o[nt][i][2] = o[nt][i][3] = 0.f;
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                m[nt][e] = -FLT_MAX, l[nt][e] = 0.f;
#pragma unroll
                for (int g = 0; g < NG; ++g) low[nt][e][g] = 0.f, unit[nt][e][g] = two_to(kMostUnit);
            }
        }

        for (; kt > 0; --kt, live -= kKeys) {
            copy_wait<kStages - 2>();
            __syncwarp();                                // the tile is there, and the stage before it is read
            fetch(stage == 0 ? kStages - 1 : stage - 1);
            const uint32_t tile = (uint32_t)(stage * S::kTile), kb = k0 + tile, vb = v0 + tile, sb = s0 + tile;
            stage = stage == kStages - 1 ? 0 : stage + 1;

            // scores of keys own_key + 2 (r % 2) of both halves, heads 2 t + e
            float x[NT][4][2];
#pragma unroll
            for (int hf = 0; hf < 2; ++hf) {
                uint32_t scale[2][2];                    // (s, m) of both keys' groups
#pragma unroll
                for (int r = 0; r < 2; ++r) load_scales<NG>(scale[r], sb + hf * (S::kScales / 2) + r * (8 * NG));
                float y[NT][4] = {};                     // scores, as they grow; both parts' of a head, in fp32
                if (!kTwoParts) {                        // sum of m (sum q)
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
                        mma_bf16_k8(y[nt], __byte_perm(scale[0][0], scale[0][NG - 1], 0x7632), __byte_perm(scale[1][0], scale[1][NG - 1], 0x7632), qsum[nt]);
                }
#pragma unroll
                for (int g = 0; g < NG; ++g) {
                    uint2 w[2];
#pragma unroll
                    for (int r = 0; r < 2; ++r) w[r] = lds64(k_at(kb, r, g) + hf * (S::kCodes / 2));
                    float acc[NT][4];
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const uint32_t w0 = h ? w[0].y : w[0].x, w1 = h ? w[1].y : w[1].x, v0 = w0 >> 8, v1 = w1 >> 8;
                        if (kTwoParts) {                 // fp32: centred codes, and each product's sum rounded to the others'
                            const uint32_t f[2][4] = {{centred_low(w0), centred_low(w1), centred_high(w0), centred_high(w1)},
                                                      {centred_low(v0), centred_low(v1), centred_high(v0), centred_high(v1)}};
#pragma unroll
                            for (int z = 0; z < 2; ++z)
#pragma unroll
                                for (int nt = 0; nt < NT; ++nt) {
                                    float part[4];
                                    mma_f16_first(part, f[z][0], f[z][1], f[z][2], f[z][3], q[nt][g][h][2 * z], q[nt][g][h][2 * z + 1]);
#pragma unroll
                                    for (int k = 0; k < 4; ++k) acc[nt][k] = h == 0 && z == 0 ? part[k] : acc[nt][k] + part[k];
                                }
                            continue;
                        }
                        const uint32_t a0 = w0 & 0x000F000Fu, a1 = w1 & 0x000F000Fu, a2 = w0 & 0x00F000F0u, a3 = w1 & 0x00F000F0u;
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt) {
                            if (h == 0) mma_f16_first(acc[nt], a0, a1, a2, a3, q[nt][g][h][0], q[nt][g][h][1]);
                            else mma_f16(acc[nt], a0, a1, a2, a3, q[nt][g][h][0], q[nt][g][h][1]);
                            mma_f16(acc[nt], v0 & 0x000F000Fu, v1 & 0x000F000Fu, v0 & 0x00F000F0u, v1 & 0x00F000F0u, q[nt][g][h][2], q[nt][g][h][3]);
                        }
                    }
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            y[nt][k] = fmaf(acc[nt][k] * low_of(scale[k >> 1][g]), unscale[nt][k & 1][g], y[nt][k]);
                        }
                }
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        float& score = x[nt][2 * hf + (k >> 1)][k & 1];
                        score = y[nt][k];
                        if (kTwoParts) {                 // and the sum of (m + 8 s) (sum q), the codes being centred
                            score += __shfl_xor_sync(0xffffffffu, y[nt][k], 2);
#pragma unroll
                            for (int g = 0; g < NG; ++g)
                                score = fmaf(fmaf(8.f, low_of(scale[k >> 1][g]), high_of(scale[k >> 1][g])), sums[nt][k & 1][g], score);
                        }
                    }
            }
            if (live < kKeys) {
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int r = 0; r < 4; ++r)
                        if (own_key + 2 * (r & 1) + kHalf * (r >> 1) >= live) x[nt][r][0] = x[nt][r][1] = -CUDART_INF_F;
            }
            bool grow = false;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const float mx = fmaxf(fmaxf(x[nt][0][e], x[nt][1][e]), fmaxf(x[nt][2][e], x[nt][3][e]));
                    grow |= mx - m[nt][e] > kMaxGrowth;
                }
            const bool grown = __any_sync(0xffffffffu, grow);
            float shrunk[NT][2];                         // what the sums so far were multiplied by
            if (grown) {
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        float mx = fmaxf(fmaxf(x[nt][0][e], x[nt][1][e]), fmaxf(x[nt][2][e], x[nt][3][e]));
#pragma unroll
                        for (int off = 4; off < 32; off <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, off));
                        mx = fmaxf(m[nt][e], mx);
                        const float w = m[nt][e] == -FLT_MAX ? 0.f : ex2(m[nt][e] - mx);
                        shrunk[nt][e] = w;
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
                for (int e = 0; e < 2; ++e)
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        x[nt][r][e] = ex2(x[nt][r][e] - m[nt][e]);
                        l[nt][e] += x[nt][r][e];
                    }
            // weights times scales, in units, as fp16 pairs of two heads; a sum of them says whether
            // one might leave fp16's range
            uint32_t w[NT][NG][4];
            __half2 total = __float2half2_rn(0.f);
            auto weigh = [&](int nt, int g, int r, float step) {
                float y[2];
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    y[e] = x[nt][r][e] * unit[nt][e][g] * step;      // in this order: see kMostUnit
                    if (kTwoParts) {
                        const float hi = __half2float(__float2half_rn(y[e]));
                        y[e] = t < 2 ? hi : y[e] - hi;
                    }
                }
                w[nt][g][r] = pack_half(y[0], y[1]);
            };
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                uint32_t scale[2];
                load_scales<NG>(scale, sb + S::kScales + (r >> 1) * (S::kScales / 2) + (r & 1) * (8 * NG));
#pragma unroll
                for (int g = 0; g < NG; ++g) {
                    const float step = low_of(scale[g]), mid = fmaf(8.f, step, high_of(scale[g]));
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
                        for (int e = 0; e < 2; ++e) low[nt][e][g] = fmaf(x[nt][r][e], mid, low[nt][e][g]);
                        weigh(nt, g, r, step);
                        total = __hadd2(total, *reinterpret_cast<const __half2*>(&w[nt][g][r]));
                    }
                }
            }
            const bool fits = __low2float(total) <= kMostWeight && __high2float(total) <= kMostWeight;
            if (grown || __any_sync(0xffffffffu, !fits)) {
#pragma unroll
                for (int g = 0; g < NG; ++g) {
                    float step[4];
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        uint32_t scale[2];
                        load_scales<NG>(scale, sb + S::kScales + (r >> 1) * (S::kScales / 2) + (r & 1) * (8 * NG));
                        step[r] = low_of(scale[g]);
                    }
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            float most = 0.f;
#pragma unroll
                            for (int r = 0; r < 4; ++r) most = fmaxf(most, x[nt][r][e] * 0x1p-10f * step[r]);
#pragma unroll
                            for (int off = 4; off < 32; off <<= 1) most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, off));
                            float sum = 0.f;             // the largest so far of the head's lanes, both parts'
#pragma unroll
                            for (int i = 4 * g; i < 4 * g + 4; ++i) sum = fmaxf(sum, fmaxf(fabsf(o[nt][i][e]), fabsf(o[nt][i][2 + e])));
#pragma unroll
                            for (int off = kTwoParts ? 2 : 4; off < 32; off <<= 1) sum = fmaxf(sum, __shfl_xor_sync(0xffffffffu, sum, off));
                            const int up = min(unit_room(sum), unit_up(most, grown ? shrunk[nt][e] : 1.f, unit[nt][e][g]));
                            const float by = two_to(up / 2), by2 = two_to(up - up / 2);
                            unit[nt][e][g] = unit[nt][e][g] * by * by2;
#pragma unroll
                            for (int i = 4 * g; i < 4 * g + 4; ++i) {
                                o[nt][i][e] = o[nt][i][e] * by * by2;
                                o[nt][i][2 + e] = o[nt][i][2 + e] * by * by2;
                            }
                        }
#pragma unroll
                        for (int r = 0; r < 4; ++r) weigh(nt, g, r, step[r]);
                    }
                }
            }
            // The tensor cores cut what they add up off rather than round it, which over many tiles
            // would cost fp32 its last bits: there a tile's sum is formed alone, and added to o.
            float tile_o[NT][NG * 4][4];
#pragma unroll
            for (int hf = 0; hf < 2; ++hf)
#pragma unroll
                for (int g = 0; g < NG; ++g) {
                    uint32_t b[NT][2];                   // turned to heads n, rows 2 t, 2 t + 1 (+ 8)
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int r = 0; r < 2; ++r) b[nt][r] = transpose(w[nt][g][2 * hf + r]);
                    uint32_t v[4];                       // channels 64 g + 16 i + 2 n and the next, of four keys
                    ldsm_bytes(v, (vb ^ g * 32) + hf * (S::kCodes / 2));
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        uint32_t f0, f1, f2, f3;
                        centred<0>(v[i], f0, f1);
                        centred<1>(v[i], f2, f3);
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt) {
                            if (!kTwoParts) mma_f16(o[nt][g * 4 + i], f0, f1, f2, f3, b[nt][0], b[nt][1]);
                            else if (hf == 0) mma_f16_first(tile_o[nt][g * 4 + i], f0, f1, f2, f3, b[nt][0], b[nt][1]);
                            else mma_f16(tile_o[nt][g * 4 + i], f0, f1, f2, f3, b[nt][0], b[nt][1]);
                        }
                    }
                }
            if (kTwoParts) {
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int i = 0; i < NG * 4; ++i)
#pragma unroll
                        for (int k = 0; k < 4; ++k) o[nt][i][k] += tile_o[nt][i][k];
            }
            __syncwarp();                                // all lanes have read the stage
        }

        // Lane (n, t) has channels 16 i + 2 n and the next of heads 2 t + e; both parts' lanes the same.
        Place done = here[warp];
        const int32_t s = done.s;
        const int head0 = done.u / blocks * G + done.u % blocks * kRows, rows = min(kRows, G - done.u % blocks * kRows);
        const bool whole = done.whole();
        const int n_pre = whole ? prefix_parts(p, done.info.x) : 0;
        if (n_pre > 0) griddep_wait();                   // the prefix's results
        const int64_t slot = part_slot(piece, done.k == 0);
        float y[NT][2][NG * 4][2];
        int head_of[NT][2];                              // -1: nothing of this lane's to write
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
#pragma unroll
                for (int off = 4; off < 32; off <<= 1) l[nt][e] += __shfl_xor_sync(0xffffffffu, l[nt][e], off);
#pragma unroll
                for (int g = 0; g < NG; ++g) {
                    float base = low[nt][e][g];
                    const float by = 1.f / unit[nt][e][g];
#pragma unroll
                    for (int off = 4; off < 32; off <<= 1) base += __shfl_xor_sync(0xffffffffu, base, off);
#pragma unroll
                    for (int i = 4 * g; i < 4 * g + 4; ++i)
#pragma unroll
                        for (int k = 0; k < 2; ++k) {
                            float& z = y[nt][e][i][k];
                            z = o[nt][i][2 * k + e] * by;
                            if (kTwoParts) z += __shfl_xor_sync(0xffffffffu, z, 2);
                            z += base;
                        }
                }
                const int rr = nt * kColumns + ((2 * t + e) & (kColumns - 1));
                head_of[nt][e] = rr < rows && (!kTwoParts || t < 2) ? head0 + rr : -1;
            }
        for (int i = 0; i < n_pre; ++i)                  // all heads' loads of a part together
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                float2 ml[2], v[2][NG * 4];
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int64_t pr = prefix_row(p, i, s, max(head_of[nt][e], 0));
                    ml[e] = load_now2(p.pre_ml + pr);
#pragma unroll
                    for (int k = 0; k < NG * 4; ++k) v[e][k] = load_now2(p.pre_o + pr * D + 16 * k + 2 * n);
                }
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    float w, w2;
                    join(m[nt][e], l[nt][e], ml[e].x, ml[e].y, w, w2);
#pragma unroll
                    for (int k = 0; k < NG * 4; ++k) {
                        y[nt][e][k][0] = y[nt][e][k][0] * w + v[e][k].x * w2;
                        y[nt][e][k][1] = y[nt][e][k][1] * w + v[e][k].y * w2;
                    }
                }
            }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int head = head_of[nt][e];
                if (head < 0) continue;
                if (whole) {
                    const float inv = l[nt][e] == 0.f ? 0.f : 1.f / l[nt][e];
                    T* out = static_cast<T*>(a.o) + s * a.o_stride + (int64_t)head * D + 2 * n;
#pragma unroll
                    for (int k = 0; k < NG * 4; ++k) write2(out + 16 * k, y[nt][e][k][0] * inv, y[nt][e][k][1] * inv);
                    if (n == 0) write_lse(a, s, head, m[nt][e], l[nt][e]);
                } else {
                    const int64_t row = slot * kRows + (head - head0);
                    float* out = p.part_o + row * D + 2 * n;
#pragma unroll
                    for (int k = 0; k < NG * 4; ++k) write2(out + 16 * k, y[nt][e][k][0], y[nt][e][k][1]);
                    if (n == 0) p.part_ml[row] = make_float2(m[nt][e], l[nt][e]);
                }
            }
        const int64_t at = line.begin(piece + 1) - done.left;                // of tile done.k
        const bool goes_on = done.k == 0 && !whole;      // begins here and ends in a later piece: the join's
        const int4 note = goes_on ? make_int4(s, done.u, (int)line.piece_of(at + done.T - 1), prefix_parts(p, done.info.x)) : make_int4(-1, 0, 0, 0);
        done.next_unit(p);
        more = done.left > 0;
        if (lane == 0 && !more) p.open[piece] = note;
        __syncwarp();
        here[warp] = done;
        __syncwarp();
    }
    copy_wait<0>();
    finish_empty<T, D>(p, piece, lane);
}

// The join of units that several pieces share, as join_kernel does it: parts in the order of the
// prefix's blocks and then the pieces.  A row is one warp's where units have few parts (narrow).
// Where they have many (16 pieces a unit on average), a thread block's warps share a row's: every
// block counts the open units itself and takes its share of their rows.  One sequence of 2^20
// tokens: 223 us, all narrow 264 us; 512 of up to 2048: 128 us, all wide 173 us.
struct OpenRow {
    int4 open;            // sequence, unit, last piece, prefix parts
    int64_t c0;           // the piece in which the unit begins
    int r, head;          // row of the unit, query head
    int64_t parts;
    __device__ __forceinline__ OpenRow(const AttnDecodeLaunch& p, int64_t c, int row, int unit_rows) : open(p.open[c]), c0(c), r(row) {
        const int G = p.a.n_heads / p.a.n_kv_heads, blocks = (G + unit_rows - 1) / unit_rows;
        const int rb = open.y % blocks;
        head = r < G - rb * unit_rows ? open.y / blocks * G + rb * unit_rows + r : -1;
        parts = open.w + open.z - c0 + 1;
    }
};
template <typename T, int D, int ROWS, int kAtOnce>
__device__ __forceinline__ void add_row(const AttnDecodeLaunch& p, const OpenRow& x, RowSum<D>& sum, int64_t from, int64_t to, int lane) {
    sum.template add_parts<kAtOnce>(from, to, lane, [&](int64_t i, const float2*& ml, const float*& o) {
        if (i < x.open.w) {
            const int64_t at = prefix_row(p, (int)i, x.open.x, x.head);
            ml = p.pre_ml + at;
            o = p.pre_o + at * D;
        } else {
            const int64_t at = part_slot(x.c0 + i - x.open.w, i == x.open.w) * ROWS + x.r;
            ml = p.part_ml + at;
            o = p.part_o + at * D;
        }
    });
}

constexpr int kJoinThreads = 256, kJoinWarps = kJoinThreads / 32, kJoinBlocks = 304;

template <typename T, int D, int ROWS>
__global__ void __launch_bounds__(kJoinThreads) join_narrow_kernel(const __grid_constant__ AttnDecodeLaunch p, int unit_rows) {
    griddep_wait();
    const int64_t x = (int64_t)blockIdx.x * kJoinWarps + (threadIdx.x >> 5), c = x / unit_rows;
    if (c >= p.n_pieces || p.open[c].x < 0) return;
    const int lane = threadIdx.x & 31;
    const OpenRow row(p, c, (int)(x - c * unit_rows), ROWS);
    if (row.head < 0) return;
    RowSum<D> sum;
    add_row<T, D, ROWS, 4>(p, row, sum, 0, row.parts, lane);
    sum.template write<T>(p.a, row.open.x, row.head, lane);
}

template <typename T, int D, int ROWS>
__global__ void __launch_bounds__(kJoinThreads) join_wide_kernel(const __grid_constant__ AttnDecodeLaunch p, int unit_rows) {
    constexpr int kCols = D / 32;
    __shared__ int32_t scan_buf[kJoinWarps], s_piece;
    __shared__ float s_o[kJoinWarps][D];
    __shared__ float2 s_ml[kJoinWarps];
    griddep_wait();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int share = (p.n_pieces + kJoinThreads - 1) / kJoinThreads, lo = min(p.n_pieces, tid * share), hi = min(p.n_pieces, lo + share);
    int32_t mine = 0, total;
    for (int c = lo; c < hi; ++c) mine += p.open[c].x >= 0;
    const int32_t before = block_scan<kJoinThreads>(mine, scan_buf, &total) - mine;
    for (int64_t i = blockIdx.x; i < (int64_t)total * unit_rows; i += gridDim.x) {
        const int32_t unit = (int32_t)(i / unit_rows);
        __syncthreads();                                 // s_piece and the last row's parts are read
        if (unit >= before && unit < before + mine) {
            int c = lo - 1;
            for (int32_t left = unit - before; left >= 0; --left)
                while (p.open[++c].x < 0) {}
            s_piece = c;
        }
        __syncthreads();
        const OpenRow row(p, s_piece, (int)(i - (int64_t)unit * unit_rows), ROWS);
        if (row.head < 0) continue;                      // (all threads alike)
        RowSum<D> sum;
        const int64_t per = (row.parts + kJoinWarps - 1) / kJoinWarps;
        add_row<T, D, ROWS, 8>(p, row, sum, min(row.parts, warp * per), min(row.parts, (warp + 1) * per), lane);
#pragma unroll
        for (int e = 0; e < kCols; ++e) s_o[warp][lane * kCols + e] = sum.o[e];
        if (lane == 0) s_ml[warp] = make_float2(sum.m, sum.l);
        __syncthreads();
        if (warp == 0) {
            for (int w = 1; w < kJoinWarps; ++w) {
                float x[kCols];
#pragma unroll
                for (int e = 0; e < kCols; ++e) x[e] = s_o[w][lane * kCols + e];
                sum.add(s_ml[w], x);
            }
            sum.template write<T>(p.a, row.open.x, row.head, lane);
        }
    }
}

template <typename T, int D, int ROWS>
cudaError_t launch_q4_join(const AttnDecodeLaunch& p, cudaStream_t s) {
    const int G = p.a.n_heads / p.a.n_kv_heads, unit_rows = G < ROWS ? G : ROWS;
    const int64_t units = (int64_t)p.a.n_seqs * p.a.n_kv_heads * ((G + ROWS - 1) / ROWS);
    note_launch();
    if (p.n_pieces >= 16 * units)
        return launch_overlapped(join_wide_kernel<T, D, ROWS>, dim3(kJoinBlocks), dim3(kJoinThreads), 0, s, p, unit_rows);
    const int64_t rows = (int64_t)p.n_pieces * unit_rows;
    return launch_overlapped(join_narrow_kernel<T, D, ROWS>, dim3((unsigned)((rows + kJoinWarps - 1) / kJoinWarps)), dim3(kJoinThreads), 0, s, p, unit_rows);
}

template <typename T, int D, int NT>
cudaError_t launch_t(const AttnDecodeQ4Launch& p, cudaStream_t s) {
    constexpr int WARPS = q4_warps(NT);
    constexpr int kRows = NT * (sizeof(T) == 4 ? 4 : 8), kBytes = Q4Smem<D, WARPS>::kBytes;
    cudaError_t e = cudaFuncSetAttribute(decode_q4_kernel<T, D, NT, WARPS>, cudaFuncAttributeMaxDynamicSharedMemorySize, kBytes);
    if (e != cudaSuccess) return e;
    note_launch();
    e = launch_overlapped(decode_q4_kernel<T, D, NT, WARPS>, dim3(p.base.n_pieces / WARPS), dim3(32 * WARPS), kBytes, s, p);
    return e == cudaSuccess ? launch_q4_join<T, D, kRows>(p.base, s) : e;
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
