// Decode attention over the paged cache for fp32 tensors, and the sequences' shared
// positions.  The division of work is described in attn_decode.cuh; this kernel
// works on a unit of 8 query heads and tiles of 32 keys, double-buffered in shared
// memory.  Bound by reading the cache once.
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

constexpr int kThreads = 128, kRows = kDecodeRowsF32, kKeys = 32;

__device__ __forceinline__ float4 load4(const float* p) { return *reinterpret_cast<const float4*>(p); }

template <int D>
struct DecodeSmem {
    static constexpr int kPad = D + 4;
    float k[2][kKeys * kPad];
    float v[2][kKeys * kPad];
    float q[kRows * D];
    float w[kKeys * kRows];              // scores, then weights, key-major
    float corr[kRows], m[kRows], l[kRows];
    float o[kThreads / D > 1 ? kRows * D : 1];
};

template <int D>
__global__ void __launch_bounds__(kThreads) decode_suffix_kernel(const __grid_constant__ AttnDecodeLaunch p) {
    using S = DecodeSmem<D>;
    constexpr int kPad = S::kPad;
    constexpr int kParts = kThreads / D;                 // threads per output column, over the keys
    constexpr int kRowsPerThread = kRows * kKeys / kThreads;
    extern __shared__ __align__(16) uint8_t smem_raw[];
    S& sm = *reinterpret_cast<S*>(smem_raw);
    griddep_wait();
    const kda_attn_decode_args& a = p.a;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int G = a.n_heads / a.n_kv_heads, blocks = (G + kRows - 1) / kRows;
    __shared__ PieceStart at_;
    int64_t all, pieces;
    find_pieces<kThreads, 1>(p, a.n_kv_heads * blocks, kKeys, 1, &at_, all, pieces);
    griddep_launch();
    const int64_t piece = blockIdx.x;
    finish_empty<float, D>(p, (int64_t)blockIdx.x * (kThreads / 32) + warp, (int64_t)gridDim.x * (kThreads / 32), lane);
    if (piece >= pieces) {
        if (tid == 0) p.open[piece] = make_int4(-1, 0, 0, 0);
        return;
    }
    Cursor c = start(p, at_, a.n_kv_heads * blocks, kKeys);
    const float sl = a.scale * kLog2e;
    while (c.left > 0) {
        const int64_t k_first = c.k, k_last = c.k + c.run();
        const int32_t s = c.s;
        const int hk = c.u / blocks, rb = c.u % blocks;
        const int head0 = hk * G + rb * kRows, rows = min(kRows, G - rb * kRows);
        const int2 info = c.info;
        const int32_t* table = a.block_table + (int64_t)s * a.table_stride;

        auto fetch = [&](int64_t tile, int buf) {
            const int64_t base = info.x + tile * kKeys;
            for (int i = tid; i < kKeys * (D / 4); i += kThreads) {
                const int j = i / (D / 4), e = i % (D / 4) * 4;
                float* kd = sm.k[buf] + j * kPad + e;
                float* vd = sm.v[buf] + j * kPad + e;
                int32_t block = -1;
                if (base + j < info.y) {
                    block = table[(base + j) / a.block_size];
                    if (block < 0 || block >= a.n_blocks) flag(p.status, KDA_DEV_BAD_SLOT), block = -1;
                }
                if (block >= 0) {
                    const int64_t at = (((int64_t)block * a.n_kv_heads + hk) * a.block_size + (base + j) % a.block_size) * D + e;
                    cp_async16(kd, static_cast<const float*>(a.k_cache) + at);
                    cp_async16(vd, static_cast<const float*>(a.v_cache) + at);
                } else {
                    *reinterpret_cast<uint4*>(kd) = make_uint4(0, 0, 0, 0);
                    *reinterpret_cast<uint4*>(vd) = make_uint4(0, 0, 0, 0);
                }
            }
            cp_async_commit();
        };
        __syncthreads();                                 // the previous unit is finished
        fetch(k_first, 0);
        for (int i = tid; i < kRows * D; i += kThreads)
            sm.q[i] = i / D < rows ? static_cast<const float*>(a.q)[s * a.q_stride + (int64_t)head0 * D + i] * sl : 0.f;
        if (tid < kRows) sm.m[tid] = -CUDART_INF_F, sm.l[tid] = 0.f;
        float o[kRows] = {};
        const int col = tid % D, part = tid / D;
        for (int64_t kt = k_first; kt < k_last; ++kt) {
            const int buf = (int)((kt - k_first) & 1);
            cp_async_wait_all();
            __syncthreads();
            if (kt + 1 < k_last) fetch(kt + 1, buf ^ 1);
            {   // scores: thread = one key, some rows
                const int key = tid % kKeys, r0 = tid / kKeys * kRowsPerThread;
                float acc[kRowsPerThread] = {};
#pragma unroll 4
                for (int e = 0; e < D; e += 4) {
                    const float4 kx = load4(sm.k[buf] + key * kPad + e);
#pragma unroll
                    for (int r = 0; r < kRowsPerThread; ++r) {
                        const float4 qv = load4(sm.q + (r0 + r) * D + e);
                        acc[r] = fmaf(qv.w, kx.w, fmaf(qv.z, kx.z, fmaf(qv.y, kx.y, fmaf(qv.x, kx.x, acc[r]))));
                    }
                }
                const bool seen = info.x + kt * kKeys + key < info.y;
#pragma unroll
                for (int r = 0; r < kRowsPerThread; ++r) sm.w[key * kRows + r0 + r] = seen ? acc[r] : -CUDART_INF_F;
            }
            __syncthreads();
#pragma unroll
            for (int rr = 0; rr < kRows / 4; ++rr) {     // a warp's rows
                const int r = warp * (kRows / 4) + rr;
                float x = sm.w[lane * kRows + r], mx = fmaxf(sm.m[r], x);
#pragma unroll
                for (int off = 16; off > 0; off >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, off));
                const float ms = mx == -CUDART_INF_F ? 0.f : mx;
                float sum = exp2f(x - ms);
                sm.w[lane * kRows + r] = sum;
#pragma unroll
                for (int off = 16; off > 0; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
                if (lane == 0) {
                    const float corr = exp2f(sm.m[r] - ms);
                    sm.corr[r] = corr;
                    sm.l[r] = fmaf(sm.l[r], corr, sum);
                    sm.m[r] = mx;
                }
            }
            __syncthreads();
#pragma unroll
            for (int r = 0; r < kRows; ++r) o[r] *= sm.corr[r];
#pragma unroll 8
            for (int j = part; j < kKeys; j += kParts) {
                const float vx = sm.v[buf][j * kPad + col];
                const float4 w0 = load4(sm.w + j * kRows), w1 = load4(sm.w + j * kRows + 4);
                const float w[kRows] = {w0.x, w0.y, w0.z, w0.w, w1.x, w1.y, w1.z, w1.w};
#pragma unroll
                for (int r = 0; r < kRows; ++r) o[r] = fmaf(w[r], vx, o[r]);
            }
        }
        if (kParts > 1) {
            __syncthreads();
            if (part == 1)
#pragma unroll
                for (int r = 0; r < kRows; ++r) sm.o[r * D + col] = o[r];
            __syncthreads();
            if (part == 0)
#pragma unroll
                for (int r = 0; r < kRows; ++r) o[r] += sm.o[r * D + col];
        }
        if (part == 0) {
            const bool whole = k_first == 0 && k_last == c.T;
            const int n_pre = whole && info.x > 0 ? p.n_split : 0;
            const int64_t slot = part_slot(piece, k_first == 0);
#pragma unroll
            for (int r = 0; r < kRows; ++r) {
                if (r >= rows) break;
                float l = sm.l[r], m = sm.m[r], x = o[r];
                for (int i = 0; i < n_pre; ++i) {
                    const int64_t at = prefix_row(p, i, s, head0 + r);
                    const float2 ml = p.pre_ml[at];
                    float w, w2;
                    join(m, l, ml.x, ml.y, w, w2);
                    x = x * w + p.pre_o[at * D + col] * w2;
                }
                if (whole) {
                    static_cast<float*>(a.o)[s * a.o_stride + (int64_t)(head0 + r) * D + col] = l == 0.f ? 0.f : x / l;
                    if (col == 0) write_lse(a, s, head0 + r, m, l);
                } else {
                    p.part_o[(slot * kRows + r) * D + col] = x;
                    if (col == 0) p.part_ml[slot * kRows + r] = make_float2(m, l);
                }
            }
        }
        if (tid == 0 && c.left == c.run()) p.open[piece] = open_unit(c, piece, pieces, all);
        c.next_unit(p, kKeys);
    }
}

template <int D>
cudaError_t launch_t(const AttnDecodeLaunch& p, cudaStream_t s) {
    cudaError_t e = cudaFuncSetAttribute(decode_suffix_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         (int)sizeof(DecodeSmem<D>));
    if (e != cudaSuccess) return e;
    note_launch();
    e = launch_overlapped(decode_suffix_kernel<D>, dim3(p.n_pieces), dim3(kThreads), sizeof(DecodeSmem<D>), s, p);
    return e == cudaSuccess ? launch_join<float, D, kRows>(p, s) : e;
}

}  // namespace

cudaError_t launch_decode_info(const AttnDecodeLaunch& p, cudaStream_t s) {
    const int32_t n = p.a.n_seqs > p.a.n_groups ? p.a.n_seqs : p.a.n_groups;
    note_launch();
    decode_info_kernel<<<(unsigned)((n + kInfoThreads - 1) / kInfoThreads), kInfoThreads, 0, s>>>(p);
    return cudaGetLastError();
}

cudaError_t launch_decode_simt(const AttnDecodeLaunch& p, cudaStream_t s) {
    return p.a.d == 128 ? launch_t<128>(p, s) : launch_t<64>(p, s);
}

}  // namespace kda
