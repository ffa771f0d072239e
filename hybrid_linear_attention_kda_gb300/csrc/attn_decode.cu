// Decode attention over the paged cache: one query token per sequence.
//
// Three kernels after the shared prefixes' own (launched by the entry point):
//   plan    each sequence's shared and total positions, checked, and the running
//           count of suffix tiles;
//   suffix  thread block c of n_ctas takes the c-th equal piece of the line of all
//           tiles (sequence, key/value head and block of query heads, tile), so the
//           blocks finish together whatever the lengths are;
//   join    the partial results of units that were split or have a prefix:
//               m = max_p m_p,  o = sum_p 2^(m_p - m) o_p / sum_p 2^(m_p - m) l_p.
// Scores are kept times log2(e).  Bound by reading the cache once.
#include <math_constants.h>

#include "async_copy.cuh"
#include "attn_common.cuh"

namespace kda {
namespace {

constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
constexpr int kPlanThreads = 1024;

__device__ __forceinline__ int64_t div_up(int64_t a, int64_t b) { return (a + b - 1) / b; }

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

__global__ void __launch_bounds__(kPlanThreads) decode_plan_kernel(AttnDecodeLaunch p, int32_t tile_keys) {
    __shared__ int64_t scan_buf[kPlanThreads / 32];
    const kda_attn_decode_args& a = p.a;
    const int64_t cap = (int64_t)a.table_stride * a.block_size;
    for (int32_t g = threadIdx.x; g < a.n_groups; g += kPlanThreads) {
        const int32_t lo = a.group_start[g], hi = a.group_start[g + 1];
        if (lo < 0 || hi < lo || hi > a.n_seqs || (g == 0 && lo != 0) || (g == a.n_groups - 1 && hi != a.n_seqs))
            flag(p.status, KDA_DEV_BAD_GROUP);
    }
    int64_t before = 0;
    for (int32_t s0 = 0; s0 < a.n_seqs; s0 += kPlanThreads) {
        const int32_t s = s0 + (int32_t)threadIdx.x;
        int64_t tiles = 0;
        if (s < a.n_seqs) {
            int64_t kv = a.kv_lens[s], shared = 0;
            if (kv < 0 || kv > cap) {
                flag(p.status, KDA_DEV_BAD_SEQLENS);
                kv = 0;
            }
            const int32_t g = group_of(a.group_start, a.n_groups, s);
            if (g >= 0) {
                shared = a.prefix_lens[g];
                if (shared < 0 || shared > cap || shared % a.block_size) shared = 0, flag(p.status, KDA_DEV_BAD_GROUP);
                if (shared > kv) flag(p.status, KDA_DEV_BAD_GROUP);
            }
            p.info[s] = make_int2((int32_t)shared, (int32_t)kv);
            tiles = kv > shared ? div_up(kv - shared, tile_keys) : 0;
        }
        int64_t total;
        const int64_t incl = block_scan<kPlanThreads>(tiles, scan_buf, &total) + before;
        if (s < a.n_seqs) p.tiles[s + 1] = incl;
        before += total;
    }
    if (threadIdx.x == 0) p.tiles[0] = 0;
}

// The line is cut into as many pieces as there are thread blocks, but none is empty:
// piece c holds the tiles [begin(c), begin(c + 1)).
__device__ __forceinline__ int64_t n_pieces(int64_t all, int64_t n_ctas) { return all < n_ctas ? all : n_ctas; }
__device__ __forceinline__ int64_t piece_begin(int64_t all, int64_t c, int64_t n) {
    return all / n * c + all % n * c / n;
}

template <typename T> struct Tile;
template <> struct Tile<float> { static constexpr int kKeys = 32; };
template <> struct Tile<__nv_bfloat16> { static constexpr int kKeys = 64; };

constexpr int kThreads = 128, kRows = 8;

__device__ __forceinline__ float4 load4(const float* p) { return *reinterpret_cast<const float4*>(p); }

// 16 bytes of shared memory as floats.
__device__ __forceinline__ void unpack(const float* p, float (&x)[4]) {
    const float4 v = load4(p);
    x[0] = v.x, x[1] = v.y, x[2] = v.z, x[3] = v.w;
}
__device__ __forceinline__ void unpack(const __nv_bfloat16* p, float (&x)[8]) {
    const uint4 v = *reinterpret_cast<const uint4*>(p);
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        x[2 * i] = __uint_as_float(w[i] << 16);
        x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
}

template <typename T, int D>
struct DecodeSmem {
    static constexpr int kKeys = Tile<T>::kKeys, kPad = D + 16 / (int)sizeof(T);
    T k[2][kKeys * kPad];
    T v[2][kKeys * kPad];
    float q[kRows * D];
    float w[kKeys * kRows];              // scores, then weights, key-major
    float corr[kRows], m[kRows], l[kRows];
    float o[kThreads / D > 1 ? kRows * D : 1];
};

// Adds (m2, l2, o2) to (m, l, o); o is one column.
__device__ __forceinline__ void join(float& m, float& l, float& o, float m2, float l2, float o2) {
    const float mx = fmaxf(m, m2), ms = mx == -CUDART_INF_F ? 0.f : mx;
    const float w = exp2f(m - ms), w2 = exp2f(m2 - ms);
    l = l * w + l2 * w2;
    o = o * w + o2 * w2;
    m = mx;
}

// Adds the prefix's n_pre partial results of (sequence, head).
template <int D>
__device__ __forceinline__ void join_prefix(const AttnDecodeLaunch& p, int n_pre, int32_t s, int head, int col,
                                            float& m, float& l, float& o) {
    for (int i = 0; i < n_pre; ++i) {
        const int64_t at = ((int64_t)i * p.a.n_seqs + s) * p.a.n_heads + head;
        const float2 ml = p.pre_ml[at];
        join(m, l, o, ml.x, ml.y, p.pre_o[at * D + col]);
    }
}

template <typename T, int D>
__device__ __forceinline__ void write_row(const kda_attn_decode_args& a, int32_t s, int head, int col, float m, float l,
                                          float o) {
    Elem<T>::store(static_cast<T*>(a.o) + s * a.o_stride + (int64_t)head * D + col, l == 0.f ? 0.f : o / l);
    if (a.lse && col == 0) a.lse[(int64_t)s * a.n_heads + head] = l == 0.f ? -CUDART_INF_F : fmaf(m, kLn2, logf(l));
}

template <typename T, int D>
__global__ void __launch_bounds__(kThreads) decode_suffix_kernel(AttnDecodeLaunch p) {
    using S = DecodeSmem<T, D>;
    constexpr int kKeys = S::kKeys, kPad = S::kPad, kVec = 16 / (int)sizeof(T);
    constexpr int kParts = kThreads / D;                 // threads per output column, over the keys
    constexpr int kRowsPerThread = kRows * kKeys / kThreads;
    extern __shared__ __align__(16) uint8_t smem_raw[];
    S& sm = *reinterpret_cast<S*>(smem_raw);
    const kda_attn_decode_args& a = p.a;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int G = a.n_heads / a.n_kv_heads, blocks = (G + kRows - 1) / kRows;
    const int64_t U = (int64_t)a.n_kv_heads * blocks;    // units of a sequence
    const int64_t all = p.tiles[a.n_seqs] * U;
    const int64_t n = n_pieces(all, p.n_ctas);
    if (blockIdx.x >= n) return;
    int64_t at = piece_begin(all, blockIdx.x, n);
    const int64_t end = piece_begin(all, blockIdx.x + 1, n);
    int32_t s = 0;
    {
        int32_t lo = 0, hi = a.n_seqs;                   // the last s with tiles[s] * U <= at
        while (hi - lo > 1) {
            const int32_t mid = (lo + hi) / 2;
            if (p.tiles[mid] * U <= at) lo = mid;
            else hi = mid;
        }
        s = lo;
    }
    const float sl = a.scale * kLog2e;
    while (at < end) {
        while (p.tiles[s + 1] * U <= at) ++s;
        const int64_t T_s = p.tiles[s + 1] - p.tiles[s], rel = at - p.tiles[s] * U;
        const int u = (int)(rel / T_s);
        const int64_t k_first = rel % T_s, k_last = min(T_s, k_first + (end - at));   // tiles of this unit
        const int hk = u / blocks, rb = u % blocks;
        const int head0 = hk * G + rb * kRows, rows = min(kRows, G - rb * kRows);
        const int2 info = p.info[s];
        const int32_t* table = a.block_table + (int64_t)s * a.table_stride;

        auto fetch = [&](int64_t tile, int buf) {
            const int64_t base = info.x + tile * kKeys;
            for (int i = tid; i < kKeys * (D / kVec); i += kThreads) {
                const int j = i / (D / kVec), c = i % (D / kVec) * kVec;
                T* kd = sm.k[buf] + j * kPad + c;
                T* vd = sm.v[buf] + j * kPad + c;
                int32_t block = -1;
                if (base + j < info.y) {
                    block = table[(base + j) / a.block_size];
                    if (block < 0 || block >= a.n_blocks) flag(p.status, KDA_DEV_BAD_SLOT), block = -1;
                }
                if (block >= 0) {
                    const int64_t e = (((int64_t)block * a.n_kv_heads + hk) * a.block_size + (base + j) % a.block_size) * D + c;
                    cp_async16(kd, static_cast<const T*>(a.k_cache) + e);
                    cp_async16(vd, static_cast<const T*>(a.v_cache) + e);
                } else {
                    *reinterpret_cast<uint4*>(kd) = make_uint4(0, 0, 0, 0);
                    *reinterpret_cast<uint4*>(vd) = make_uint4(0, 0, 0, 0);
                }
            }
            cp_async_commit();
        };
        __syncthreads();                                 // the previous unit is finished
        fetch(k_first, 0);
        for (int i = tid; i < kRows * D; i += kThreads) {
            const int r = i / D;
            sm.q[i] = r < rows ? Elem<T>::load(static_cast<const T*>(a.q) + s * a.q_stride + (int64_t)head0 * D + i) * sl : 0.f;
        }
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
                for (int c = 0; c < D; c += kVec) {
                    float kx[kVec];
                    unpack(sm.k[buf] + key * kPad + c, kx);
#pragma unroll
                    for (int r = 0; r < kRowsPerThread; ++r)
#pragma unroll
                        for (int e = 0; e < kVec; e += 4) {
                            const float4 qv = load4(sm.q + (r0 + r) * D + c + e);
                            acc[r] = fmaf(qv.w, kx[e + 3], fmaf(qv.z, kx[e + 2], fmaf(qv.y, kx[e + 1], fmaf(qv.x, kx[e], acc[r]))));
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
                float mx = sm.m[r];
                for (int j = lane; j < kKeys; j += 32) mx = fmaxf(mx, sm.w[j * kRows + r]);
#pragma unroll
                for (int off = 16; off > 0; off >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, off));
                const float ms = mx == -CUDART_INF_F ? 0.f : mx;
                float sum = 0.f;
                for (int j = lane; j < kKeys; j += 32) {
                    const float w = exp2f(sm.w[j * kRows + r] - ms);
                    sm.w[j * kRows + r] = w;
                    sum += w;
                }
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
                const float vx = Elem<T>::load(sm.v[buf] + j * kPad + col);
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
            if (k_first == 0 && k_last == T_s) {         // the whole unit: the prefix's results join here
                const int n_pre = info.x > 0 ? p.n_split : 0;
                for (int r = 0; r < rows; ++r) {
                    float oo = 0.f, l = sm.l[r], m = sm.m[r];
#pragma unroll
                    for (int i = 0; i < kRows; ++i) oo = i == r ? o[i] : oo;
                    join_prefix<D>(p, n_pre, s, head0 + r, col, m, l, oo);
                    write_row<T, D>(a, s, head0 + r, col, m, l, oo);
                }
            } else {
                // a piece that starts inside a unit leaves slot 0, one that starts it slot 1
                const int64_t slot = 2 * (int64_t)blockIdx.x + (k_first == 0 ? 1 : 0);
#pragma unroll
                for (int r = 0; r < kRows; ++r) {
                    if (r >= rows) break;
                    p.part_o[(slot * kRows + r) * D + col] = o[r];
                    if (col == 0) p.part_ml[slot * kRows + r] = make_float2(sm.m[r], sm.l[r]);
                }
            }
        }
        at += k_last - k_first;
    }
}

// One thread block per unit; threads over the columns.
template <typename T, int D>
__global__ void __launch_bounds__(D) decode_join_kernel(AttnDecodeLaunch p) {
    const kda_attn_decode_args& a = p.a;
    const int col = threadIdx.x;
    const int G = a.n_heads / a.n_kv_heads, blocks = (G + kRows - 1) / kRows;
    const int64_t U = (int64_t)a.n_kv_heads * blocks;
    const int32_t s = (int32_t)(blockIdx.x / U);
    const int u = (int)(blockIdx.x % U), hk = u / blocks, rb = u % blocks;
    const int head0 = hk * G + rb * kRows, rows = min(kRows, G - rb * kRows);
    const int2 info = p.info[s];
    const int64_t T_s = p.tiles[s + 1] - p.tiles[s], all = p.tiles[a.n_seqs] * U;
    const int64_t lo = p.tiles[s] * U + u * T_s, hi = lo + T_s;
    int64_t c0 = 0, c1 = -1;                             // pieces that hold the unit's tiles
    if (T_s > 0) {
        const int64_t n = n_pieces(all, p.n_ctas);
        auto piece = [&](int64_t x) {                    // the piece with begin(c) <= x < begin(c + 1)
            int64_t c = (int64_t)((double)x * n / (double)all);
            c = c < 0 ? 0 : c >= n ? n - 1 : c;
            while (c > 0 && piece_begin(all, c, n) > x) --c;
            while (c + 1 < n && piece_begin(all, c + 1, n) <= x) ++c;
            return c;
        };
        c0 = piece(lo);
        c1 = piece(hi - 1);
        if (c0 == c1) return;                            // written by its piece
    }
    const int n_pre = info.x > 0 ? p.n_split : 0;
    for (int r = 0; r < rows; ++r) {
        const int head = head0 + r;
        float m = -CUDART_INF_F, l = 0.f, o = 0.f;
        join_prefix<D>(p, n_pre, s, head, col, m, l, o);
        for (int64_t c = c0; c <= c1; ++c) {
            const int64_t at = (2 * c + (c == c0 ? 1 : 0)) * kRows + r;
            const float2 ml = p.part_ml[at];
            join(m, l, o, ml.x, ml.y, p.part_o[at * D + col]);
        }
        write_row<T, D>(a, s, head, col, m, l, o);
    }
}

template <typename T, int D>
cudaError_t launch_t(const AttnDecodeLaunch& p, cudaStream_t s) {
    const kda_attn_decode_args& a = p.a;
    const cudaError_t e = cudaFuncSetAttribute(decode_suffix_kernel<T, D>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               (int)sizeof(DecodeSmem<T, D>));
    if (e != cudaSuccess) return e;
    note_launch(3);
    decode_plan_kernel<<<1, kPlanThreads, 0, s>>>(p, Tile<T>::kKeys);
    decode_suffix_kernel<T, D><<<p.n_ctas, kThreads, sizeof(DecodeSmem<T, D>), s>>>(p);
    const int G = a.n_heads / a.n_kv_heads;
    const int64_t units = (int64_t)a.n_seqs * a.n_kv_heads * ((G + kRows - 1) / kRows);
    decode_join_kernel<T, D><<<(unsigned)units, D, 0, s>>>(p);
    return cudaGetLastError();
}

}  // namespace

int attn_decode_rows(int) { return kRows; }

cudaError_t launch_attn_decode(const AttnDecodeLaunch& p, cudaStream_t s) {
    if (p.a.dtype == KDA_BF16)
        return p.a.d == 128 ? launch_t<__nv_bfloat16, 128>(p, s) : launch_t<__nv_bfloat16, 64>(p, s);
    return p.a.d == 128 ? launch_t<float, 128>(p, s) : launch_t<float, 64>(p, s);
}

}  // namespace kda
