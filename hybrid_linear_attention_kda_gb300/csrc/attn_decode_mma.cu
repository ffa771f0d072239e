// Decode attention over the paged cache, bf16.  The division of work is described in
// attn_decode.cuh.
//
// A unit has up to 16 query heads, the rows of one m16n8k16 product, so the cache is
// read once for all of them: 16 rows x 4 d flops for the 4 d bytes of a key, which
// keeps the warp-level tensor instructions well below their rate (the wider tcgen05
// tiles would be seven eighths padding).  Each warp is a worker of its own: it walks
// its piece in tiles of 16 keys with its (m, l, o) in registers and its own ring of
// asynchronous copies, which run ahead across the ends of units, so that nothing in
// the kernel waits for another warp.  A page holds at least 16 keys, so that a tile
// lies in one.
//
// Bound by reading the cache once: 6.8 TB/s on one sequence of 2^20 tokens, 8 heads, d =
// 128 (0.63 ms), 5.7 TB/s on 512 sequences behind shared prefixes (0.39 ms with those).
#include "attn_decode.cuh"

namespace kda {
namespace {
using namespace decode;

constexpr int kWarps = kDecodeWarps, kThreads = 32 * kWarps, kRows = kDecodeRowsBf16, kKeys = decode_tile(KDA_BF16, 0);
constexpr float kMaxGrowth = 8.f;        // log2 of how far weights may exceed 1 before their maximum moves

template <int D> struct DecodeSmem {
    static constexpr int kTileBytes = kKeys * D * 2, kStages = 384 / D;      // 24 KB of keys and values a warp
    uint8_t ring[kWarps][kStages][2][kTileBytes];
};

__device__ __forceinline__ uint32_t smem_u32(const void* p) { return (uint32_t)__cvta_generic_to_shared(p); }
// 16 bytes global -> shared, zeros instead when !live.
__device__ __forceinline__ void copy16(uint32_t dst, const void* src, bool live) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(__cvta_generic_to_global(src)), "r"(live ? 16 : 0)
                 : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N> __device__ __forceinline__ void copy_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

__device__ __forceinline__ void ldsm(uint32_t (&r)[4], uint32_t at) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(at)
                 : "memory");
}
__device__ __forceinline__ void ldsm_t(uint32_t (&r)[4], uint32_t at) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(at)
                 : "memory");
}
__device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
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

template <int D>
__global__ void __launch_bounds__(kThreads, 1) decode_suffix_kernel(const __grid_constant__ AttnDecodeLaunch p) {
    using S = DecodeSmem<D>;
    constexpr int kChunks = D / 8, kStages = S::kStages;  // 16-byte pieces of a key
    extern __shared__ __align__(128) uint8_t smem_raw[];
    S& sm = *reinterpret_cast<S*>(smem_raw);
    start_after(p);
    const kda_attn_decode_args& a = p.a;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int G = a.n_heads / a.n_kv_heads, blocks = (G + kRows - 1) / kRows;
    __shared__ PieceStart at_[kWarps];
    const Line line = find_pieces<kThreads, kWarps>(p, a.n_kv_heads * blocks, kKeys, at_);
    griddep_launch();
    const int64_t piece = (int64_t)blockIdx.x * kWarps + warp;
    if (piece >= line.pieces) {
        if (lane == 0) p.open[piece] = make_int4(-1, 0, 0, 0);
        finish_empty<__nv_bfloat16, D>(p, piece, lane);
        return;
    }
    Cursor c = start(at_[warp], line, piece, a.n_kv_heads * blocks, kKeys);

    // ------------------------------------------------------------------ copies
    // The copies' own place on the line, kStages - 1 tiles ahead.  Chunk y of key j
    // lies at chunk y ^ (j % 8) of its row: eight keys' equal chunks in eight banks.
    Cursor f = c;
    const uint32_t ring = smem_u32(sm.ring[warp]);
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
            if (live > 0 && (next_block < 0 || next_block >= a.n_blocks)) {
                flag(p.status, KDA_DEV_BAD_SLOT);
                live = 0;
            }
            const int hk = blocks == 1 ? f.u : f.u / blocks;
            const int64_t row = live > 0 ? ((int64_t)next_block * a.n_kv_heads + hk) * a.block_size + (key & (a.block_size - 1)) : 0;
            const __nv_bfloat16* ks = static_cast<const __nv_bfloat16*>(a.k_cache) + row * D;
            const __nv_bfloat16* vs = static_cast<const __nv_bfloat16*>(a.v_cache) + row * D;
            const uint32_t kd = ring + stage * 2 * S::kTileBytes, vd = kd + S::kTileBytes;
#pragma unroll
            for (int i = 0; i < kKeys * kChunks / 32; ++i) {
                const int j = (i * 32 + lane) / kChunks, y = (i * 32 + lane) % kChunks;
                const uint32_t to = (uint32_t)(j * kChunks + (y ^ (j & 7))) * 16u;
                const int from = j < live ? j * D + y * 8 : 0;
                copy16(kd + to, ks + from, j < live);
                copy16(vd + to, vs + from, j < live);
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
    // Thread (row, column pair) of the products: rows lane / 4 and lane / 4 + 8,
    // columns 2 (lane % 4) and one more of every eight.
    const int row = lane >> 2, pair = 2 * (lane & 3);
    // addresses of the 8 x 8 blocks that this lane names to ldmatrix: K blocks (keys
    // 0-7 and 8-15) x (two chunks), V blocks (two key halves) x (two chunks)
    const int k_key = (lane & 7) + ((lane >> 4) << 3), k_chunk = (lane >> 3) & 1;
    const int v_key = lane & 15, v_chunk = lane >> 4;
    const float sc = fabsf(a.scale) * kLog2e;
    const uint32_t negate = a.scale < 0.f ? 0x80008000u : 0u;
    int stage = 0;
    while (c.left > 0) {
        const int64_t k_first = c.k, k_last = c.k + c.run();
        const int32_t s = c.s;
        const int hk = c.u / blocks, rb = c.u % blocks;
        const int head0 = hk * G + rb * kRows, rows = min(kRows, G - rb * kRows);
        const int2 info = c.info;
        uint32_t q[D / 16][4];
        {
            const __nv_bfloat16* qs = static_cast<const __nv_bfloat16*>(a.q) + s * a.q_stride + (int64_t)head0 * D;
#pragma unroll
            for (int x = 0; x < D / 16; ++x)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int r = row + 8 * (e & 1), col = 16 * x + pair + 8 * (e >> 1);
                    q[x][e] = r < rows ? *reinterpret_cast<const uint32_t*>(qs + r * D + col) ^ negate : 0u;
                }
        }
        float o[D / 8][4];
#pragma unroll
        for (int x = 0; x < D / 8; ++x) o[x][0] = o[x][1] = o[x][2] = o[x][3] = 0.f;
        float m[2] = {-CUDART_INF_F, -CUDART_INF_F}, l[2] = {0.f, 0.f};

        for (int64_t kt = k_first; kt < k_last; ++kt) {
            copy_wait<kStages - 2>();
            __syncwarp();                                // the tile is there, and the stage before it is read
            fetch(stage == 0 ? kStages - 1 : stage - 1);
            const uint32_t kb = ring + stage * 2 * S::kTileBytes, vb = kb + S::kTileBytes;
            stage = stage == kStages - 1 ? 0 : stage + 1;
            const int64_t key0 = info.x + kt * kKeys;
            const int live = (int)max((int64_t)0, min((int64_t)kKeys, info.y - key0));
            float x[2][4] = {};
#pragma unroll
            for (int d = 0; d < D / 16; ++d) {
                uint32_t b[4];
                ldsm(b, kb + (uint32_t)(k_key * kChunks + ((2 * d + k_chunk) ^ (k_key & 7))) * 16u);
                mma(x[0], q[d], b[0], b[1]);
                mma(x[1], q[d], b[2], b[3]);
            }
            // x[h][2 r + e]: row `row + 8 r`, key 8 h + pair + e
            if (live < kKeys) {
#pragma unroll
                for (int h = 0; h < 2; ++h)
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        if (8 * h + pair + (e & 1) >= live) x[h][e] = -CUDART_INF_F;
            }
            bool grow = false;
            float mn[2];
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                float mx = fmaxf(fmaxf(x[0][2 * r], x[0][2 * r + 1]), fmaxf(x[1][2 * r], x[1][2 * r + 1]));
                mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
                mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
                mn[r] = fmaxf(m[r], mx);
                grow |= (mn[r] - m[r]) * sc > kMaxGrowth || (m[r] == -CUDART_INF_F && mn[r] > m[r]);
            }
            if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    const float w = m[r] == -CUDART_INF_F ? 0.f : ex2((m[r] - mn[r]) * sc);
                    m[r] = mn[r];
                    l[r] *= w;
#pragma unroll
                    for (int y = 0; y < D / 8; ++y) {
                        o[y][2 * r] *= w;
                        o[y][2 * r + 1] *= w;
                    }
                }
            }
            uint32_t pa[4];
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                const float off = m[r] == -CUDART_INF_F ? 0.f : -m[r] * sc;
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    float w0 = ex2(fmaf(x[h][2 * r], sc, off)), w1 = ex2(fmaf(x[h][2 * r + 1], sc, off));
                    if (live < kKeys) {
                        w0 = 8 * h + pair < live ? w0 : 0.f;
                        w1 = 8 * h + pair + 1 < live ? w1 : 0.f;
                    }
                    l[r] += w0 + w1;
                    pa[r + 2 * h] = pack(w0, w1);
                }
            }
#pragma unroll
            for (int d = 0; d < D / 16; ++d) {
                uint32_t b[4];
                ldsm_t(b, vb + (uint32_t)(v_key * kChunks + ((2 * d + v_chunk) ^ (v_key & 7))) * 16u);
                mma(o[2 * d], pa, b[0], b[1]);
                mma(o[2 * d + 1], pa, b[2], b[3]);
            }
            __syncwarp();                                // all lanes have read the stage
        }

        const bool whole = k_first == 0 && k_last == c.T;
        const int n_pre = whole ? prefix_parts(p, info.x) : 0;
        if (n_pre > 0) griddep_wait();                   // the prefix's results
        const int64_t slot = part_slot(piece, k_first == 0);
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            float lt = l[r], mt = m[r] == -CUDART_INF_F ? m[r] : m[r] * sc;
            lt += __shfl_xor_sync(0xffffffffu, lt, 1);
            lt += __shfl_xor_sync(0xffffffffu, lt, 2);
            const int rr = row + 8 * r, head = head0 + rr;
            if (rr >= rows) continue;
#pragma unroll 2
            for (int i = 0; i < n_pre; ++i) {
                const int64_t pr = prefix_row(p, i, s, head);
                const float2 ml = p.pre_ml[pr];
                float w, w2;
                join(mt, lt, ml.x, ml.y, w, w2);
#pragma unroll
                for (int y = 0; y < D / 8; ++y) {
                    const float2 v = *reinterpret_cast<const float2*>(p.pre_o + pr * D + 8 * y + pair);
                    o[y][2 * r] = o[y][2 * r] * w + v.x * w2;
                    o[y][2 * r + 1] = o[y][2 * r + 1] * w + v.y * w2;
                }
            }
            if (whole) {
                const float inv = lt == 0.f ? 0.f : 1.f / lt;
                __nv_bfloat16* out = static_cast<__nv_bfloat16*>(a.o) + s * a.o_stride + (int64_t)head * D + pair;
#pragma unroll
                for (int y = 0; y < D / 8; ++y)
                    *reinterpret_cast<uint32_t*>(out + 8 * y) = pack(o[y][2 * r] * inv, o[y][2 * r + 1] * inv);
                if (pair == 0) write_lse(a, s, head, mt, lt);
            } else {
                float* out = p.part_o + (slot * kRows + rr) * D + pair;
#pragma unroll
                for (int y = 0; y < D / 8; ++y) *reinterpret_cast<float2*>(out + 8 * y) = make_float2(o[y][2 * r], o[y][2 * r + 1]);
                if (pair == 0) p.part_ml[slot * kRows + rr] = make_float2(mt, lt);
            }
        }
        __syncwarp();
        if (lane == 0 && c.left == c.run()) p.open[piece] = open_unit(p, c, piece, line);
        c.next_unit(p, kKeys);
    }
    copy_wait<0>();
    finish_empty<__nv_bfloat16, D>(p, piece, lane);
}

template <int D>
cudaError_t launch_t(const AttnDecodeLaunch& p, cudaStream_t s) {
    cudaError_t e = cudaFuncSetAttribute(decode_suffix_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         (int)sizeof(DecodeSmem<D>));
    if (e != cudaSuccess) return e;
    note_launch();
    e = launch_overlapped(decode_suffix_kernel<D>, dim3(p.n_pieces / kWarps), dim3(kThreads), sizeof(DecodeSmem<D>), s, p);
    return e == cudaSuccess ? launch_join<__nv_bfloat16, D, kRows>(p, s) : e;
}

}  // namespace

cudaError_t launch_decode_mma(const AttnDecodeLaunch& p, cudaStream_t s) {
    return p.a.d == 128 ? launch_t<128>(p, s) : launch_t<64>(p, s);
}

}  // namespace kda
