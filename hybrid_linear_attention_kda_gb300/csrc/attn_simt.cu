// Softmax attention of row tiles for fp32 tensors, in SIMT arithmetic: prompts (causal)
// and the shared prefixes of decode attention.
//
// For the rows i of a tile and the keys j that row i sees (x_ij = scale q_i . k_j):
//     m = max_j x_ij,  l = sum_j exp(x_ij - m),  o_i = sum_j exp(x_ij - m) v_j / l
// in one pass over key tiles, with o and l rescaled whenever m grows.  Scores are
// kept times log2(e), so that exp is exp2.
//
// A thread owns 4 rows, the keys tx + 16 c of a score tile of 64 and the columns
// 4 tx + 64 c of the output.  A block's 256 threads are one group with 64 rows, or,
// where that would leave SMs idle, several groups with the same 64 / groups rows and
// every so manieth key tile each, whose results are joined at the end: the chain of
// key tiles gets as much shorter.  K is padded by 16 bytes a row, so that the 16
// threads of a row group read distinct banks; the weights reuse K's place.  Bound by
// the FP32 pipe and the shared-memory reads that feed it (eight 16-byte reads for 64
// products): 8 x 2000 tokens, 16/4 heads, d = 128 take 3.5 ms, 37 TFLOP/s.  One prompt of 512, 2 heads, d = 64 takes 20 us, 47 us with
// one group.
#include <math_constants.h>

#include "attn_common.cuh"

namespace kda {
namespace {

constexpr int kKeys = kTileKeysF32, kThreads = 256;
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

enum Mode { kPacked, kPaged, kPrefix };

template <int D> constexpr int kPad = D + 4;
template <int D> constexpr int kPPad = kKeys + 4;
constexpr int rows_of(int groups) { return 64 / groups; }
template <int D> constexpr int kGroupFloats = kKeys * kPad<D> + kKeys * D;         // one group's K and V
template <int D> constexpr size_t smem_bytes(int groups) {
    return sizeof(float) * ((size_t)rows_of(groups) * kPad<D> + (size_t)groups * kGroupFloats<D>);
}
// Most groups whose tiles fit beside each other.
template <int D> constexpr int kGroups = D == 64 ? 4 : 2;

__device__ __forceinline__ float4 load4(const float* p) { return *reinterpret_cast<const float4*>(p); }
__device__ __forceinline__ void store4(float* p, float4 x) { *reinterpret_cast<float4*>(p) = x; }

template <int D, int MODE, int GROUPS, bool SPLIT>
__global__ void __launch_bounds__(kThreads) attn_simt_kernel(const __grid_constant__ AttnTileLaunch p, int32_t Gp, int32_t chunks) {
    constexpr int kRows = rows_of(GROUPS), kGroupThreads = kThreads / GROUPS;
    griddep_wait();
    griddep_launch();
    extern __shared__ __align__(16) float smem[];
    const int tid = threadIdx.x, group = tid / kGroupThreads, gt = tid % kGroupThreads;
    const int tx = gt & 15, ty = gt >> 4;
    float* Qs = smem;
    float* Ks = Qs + kRows * kPad<D> + group * kGroupFloats<D>;
    float* Vs = Ks + kKeys * kPad<D>;
    float* Ps = Ks;
    static_assert(kPPad<D> <= kPad<D>, "the weights fit in K's place");
    // a group's own barrier
    auto group_sync = [&]() {
        if (GROUPS == 1) __syncthreads();
        else asm volatile("barrier.cta.sync %0, %1;" ::"r"(1 + group), "n"(kGroupThreads) : "memory");
    };
    const kda_attn_prefill_args& a = p.a;
    const int G = a.n_heads / a.n_kv_heads;
    const int hk = (int)(blockIdx.y / chunks), hc = (int)(blockIdx.y % chunks);
    const int head0 = hk * G + hc * Gp, gn = min(Gp, G - hc * Gp);
    const int bt = kRows / Gp;                       // tokens of a tile
    const int64_t idx = SPLIT ? blockIdx.x / p.n_split : blockIdx.x;
    const int split = SPLIT ? (int)(blockIdx.x % p.n_split) : 0;
    const bool report = MODE != kPrefix && blockIdx.x == 0 && blockIdx.y == 0;
    const RowTile rt = find_tile<kThreads>(a.cu_seqlens, a.n_seqs, a.total_tokens, bt, idx, report,
                                           KDA_DEV_BAD_SEQLENS, p.status);
    if (rt.seq < 0) return;
    const int nt = min(bt, rt.n - rt.t0);            // tokens of this tile

    // keys: row of token t sees j <= first + t
    int64_t K, first;
    const int32_t* table = nullptr;
    if (MODE == kPacked) {
        K = rt.n;
        first = 0;
    } else if (MODE == kPaged) {
        K = a.kv_lens[rt.seq];
        table = a.block_table + (int64_t)rt.seq * a.table_stride;
        if (K < 0 || K > (int64_t)a.table_stride * a.block_size) {
            if (tid == 0) flag(p.status, KDA_DEV_BAD_SEQLENS);
            return;
        }
        first = K - rt.n;
    } else {
        K = p.prefix_lens[rt.seq];
        table = a.block_table + rt.row0 * a.table_stride;
        if (K < 0 || K > (int64_t)a.table_stride * a.block_size || K % a.block_size) K = 0;   // flagged by the plan
        first = K;
    }
    int64_t k_lo = 0, k_hi = min(K, first + rt.t0 + nt);
    if (SPLIT) {
        if (MODE != kPrefix) K = max((int64_t)0, k_hi);      // the tile's keys
        const int64_t per = MODE == kPrefix ? (int64_t)prefix_block_tiles((uint32_t)K, kKeys, p.n_split, p.split_cost) * kKeys
                                            : ((K + kKeys - 1) / kKeys + p.n_split - 1) / p.n_split * kKeys;
        k_lo = min(K, split * per);
        k_hi = min(K, k_lo + per);
    }

    auto key_row = [&](int64_t j, const float*& kr, const float*& vr) -> bool {
        if (MODE == kPacked) {
            kr = static_cast<const float*>(a.k) + (rt.row0 + j) * a.k_stride + hk * D;
            vr = static_cast<const float*>(a.v) + (rt.row0 + j) * a.v_stride + hk * D;
            return true;
        }
        const int32_t block = table[j / a.block_size];
        if (block < 0 || block >= a.n_blocks) {
            flag(p.status, KDA_DEV_BAD_SLOT);
            return false;
        }
        const int64_t e = (((int64_t)block * a.n_kv_heads + hk) * a.block_size + j % a.block_size) * D;
        kr = static_cast<const float*>(a.k_cache) + e;
        vr = static_cast<const float*>(a.v_cache) + e;
        return true;
    };

    // rows past the tile's end compute on zeros and are not written
    for (int i = tid; i < kRows * (D / 4); i += kThreads) {
        const int r = i / (D / 4), c = i % (D / 4) * 4;
        const int t = r / Gp, g = r % Gp;
        float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
        if (t < nt && g < gn)
            x = load4(static_cast<const float*>(a.q) + (rt.row0 + rt.t0 + t) * a.q_stride + (head0 + g) * D + c);
        store4(Qs + r * kPad<D> + c, x);
    }

    constexpr int OC = D / 64;
    float4 o[4][OC];
    float m[4], l[4];
    int64_t lim[4];
#pragma unroll
    for (int r = 0; r < 4; ++r) {
        m[r] = -CUDART_INF_F;
        l[r] = 0.f;
        lim[r] = MODE == kPrefix ? K - 1 : first + rt.t0 + (ty * 4 + r) / Gp;
#pragma unroll
        for (int c = 0; c < OC; ++c) o[r][c] = make_float4(0.f, 0.f, 0.f, 0.f);
    }
    const float sl = a.scale * kLog2e;

    __syncthreads();                                  // Q is written
    for (int64_t k0 = k_lo + group * kKeys; k0 < k_hi; k0 += GROUPS * kKeys) {
        group_sync();                                 // the previous tile is consumed
        for (int i = gt; i < kKeys * (D / 4); i += kGroupThreads) {
            const int j = i / (D / 4), c = i % (D / 4) * 4;
            float4 kx = make_float4(0.f, 0.f, 0.f, 0.f), vx = kx;
            const float *kr, *vr;
            if (k0 + j < k_hi && key_row(k0 + j, kr, vr)) {
                kx = load4(kr + c);
                vx = load4(vr + c);
            }
            store4(Ks + j * kPad<D> + c, kx);
            store4(Vs + j * D + c, vx);
        }
        group_sync();
        float s[4][4] = {};
#pragma unroll 8
        for (int c = 0; c < D; c += 4) {
            float4 qv[4], kv[4];
#pragma unroll
            for (int r = 0; r < 4; ++r) qv[r] = load4(Qs + (ty * 4 + r) * kPad<D> + c);
#pragma unroll
            for (int j = 0; j < 4; ++j) kv[j] = load4(Ks + (tx + 16 * j) * kPad<D> + c);
#pragma unroll
            for (int r = 0; r < 4; ++r)
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    s[r][j] = fmaf(qv[r].w, kv[j].w, fmaf(qv[r].z, kv[j].z, fmaf(qv[r].y, kv[j].y, fmaf(qv[r].x, kv[j].x, s[r][j]))));
        }
        group_sync();                                 // K is read: the weights take its place
        // the tile's last key against what the tile's first token sees
        const bool masked = k0 + kKeys > (MODE == kPrefix ? k_hi : min(k_hi, first + rt.t0 + 1));
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const int64_t seen = min(lim[r] + 1, k_hi);
            float mx = m[r];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                s[r][j] = k0 + tx + 16 * j < seen ? s[r][j] * sl : -CUDART_INF_F;
                mx = fmaxf(mx, s[r][j]);
            }
#pragma unroll
            for (int off = 8; off > 0; off >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, off));
            const float ms = mx == -CUDART_INF_F ? 0.f : mx;
            const float corr = exp2f(m[r] - ms);
            float sum = 0.f;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float w = exp2f(s[r][j] - ms);
                Ps[(ty * 4 + r) * kPPad<D> + tx + 16 * j] = w;
                sum += w;
            }
#pragma unroll
            for (int off = 8; off > 0; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
            l[r] = fmaf(l[r], corr, sum);
            m[r] = mx;
#pragma unroll
            for (int c = 0; c < OC; ++c) {
                o[r][c].x *= corr;
                o[r][c].y *= corr;
                o[r][c].z *= corr;
                o[r][c].w *= corr;
            }
        }
        __syncwarp();                                 // a row's weights are written and read by one half warp
        auto product = [&](auto check) {
            constexpr bool kCheck = decltype(check)::value;
#pragma unroll 4
            for (int j = 0; j < kKeys; ++j) {
                float4 vv[OC];
#pragma unroll
                for (int c = 0; c < OC; ++c) vv[c] = load4(Vs + j * D + 4 * tx + 64 * c);
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    // a hidden value takes no part, whatever it holds (0 * NaN is NaN)
                    if (kCheck && k0 + j > lim[r]) continue;
                    const float w = Ps[(ty * 4 + r) * kPPad<D> + j];
#pragma unroll
                    for (int c = 0; c < OC; ++c) {
                        o[r][c].x = fmaf(w, vv[c].x, o[r][c].x);
                        o[r][c].y = fmaf(w, vv[c].y, o[r][c].y);
                        o[r][c].z = fmaf(w, vv[c].z, o[r][c].z);
                        o[r][c].w = fmaf(w, vv[c].w, o[r][c].w);
                    }
                }
            }
        };
        if (masked) product(std::true_type{});
        else product(std::false_type{});
    }

    if (GROUPS > 1) {
        // the other groups' results, from their tiles' places, onto the first one's
        __syncthreads();
        float* mine = Ks;                             // [row][D], then [row] (m, l)
        if (group > 0) {
#pragma unroll
            for (int r = 0; r < 4; ++r) {
#pragma unroll
                for (int c = 0; c < OC; ++c) store4(mine + (ty * 4 + r) * D + 4 * tx + 64 * c, o[r][c]);
                if (tx == 0) *reinterpret_cast<float2*>(mine + kRows * D + 2 * (ty * 4 + r)) = make_float2(m[r], l[r]);
            }
        }
        __syncthreads();
        if (group > 0) return;
        for (int x = 1; x < GROUPS; ++x) {
            const float* from = Ks + x * kGroupFloats<D>;
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const float2 ml = *reinterpret_cast<const float2*>(from + kRows * D + 2 * (ty * 4 + r));
                const float mx = fmaxf(m[r], ml.x), ms = mx == -CUDART_INF_F ? 0.f : mx;
                const float w = exp2f(m[r] - ms), w2 = exp2f(ml.x - ms);
                m[r] = mx;
                l[r] = l[r] * w + ml.y * w2;
#pragma unroll
                for (int c = 0; c < OC; ++c) {
                    const float4 z = load4(from + (ty * 4 + r) * D + 4 * tx + 64 * c);
                    o[r][c].x = o[r][c].x * w + z.x * w2;
                    o[r][c].y = o[r][c].y * w + z.y * w2;
                    o[r][c].z = o[r][c].z * w + z.z * w2;
                    o[r][c].w = o[r][c].w * w + z.w * w2;
                }
            }
        }
    }
#pragma unroll
    for (int r = 0; r < 4; ++r) {
        const int t = (ty * 4 + r) / Gp, g = (ty * 4 + r) % Gp;
        if (t >= nt || g >= gn) continue;
        const int64_t row = rt.row0 + rt.t0 + t;
        const int head = head0 + g;
        if (SPLIT) {
            const int64_t at = ((int64_t)split * a.total_tokens + row) * a.n_heads + head;
#pragma unroll
            for (int c = 0; c < OC; ++c) store4(p.part_o + at * D + 4 * tx + 64 * c, o[r][c]);
            if (tx == 0) p.part_ml[at] = make_float2(m[r], l[r]);
        } else {
            const float inv = l[r] == 0.f ? 0.f : 1.f / l[r];
            float* out = static_cast<float*>(a.o) + row * a.o_stride + (int64_t)head * D;
#pragma unroll
            for (int c = 0; c < OC; ++c)
                store4(out + 4 * tx + 64 * c, make_float4(o[r][c].x * inv, o[r][c].y * inv, o[r][c].z * inv, o[r][c].w * inv));
            if (a.lse && tx == 0) a.lse[row * a.n_heads + head] = l[r] == 0.f ? -CUDART_INF_F : fmaf(m[r], kLn2, logf(l[r]));
        }
    }
}

// Blocks of a launch with the given groups, at most.
int64_t blocks_of(const AttnTileLaunch& p, int groups, bool split, int* Gp, int* chunks) {
    const int G = p.a.n_heads / p.a.n_kv_heads, rows = rows_of(groups);
    *Gp = G < rows ? G : rows;
    *chunks = (G + *Gp - 1) / *Gp;
    return (p.a.total_tokens / (rows / *Gp) + p.a.n_seqs) * (split ? p.n_split : 1);
}

template <int D, int MODE, int GROUPS, bool SPLIT>
cudaError_t launch_g(const AttnTileLaunch& p, cudaStream_t s) {
    int32_t Gp, chunks;
    const int64_t tiles = blocks_of(p, GROUPS, SPLIT, &Gp, &chunks);
    if (tiles > (int64_t)INT32_MAX) return cudaErrorInvalidValue;
    const cudaError_t e = cudaFuncSetAttribute(attn_simt_kernel<D, MODE, GROUPS, SPLIT>,
                                               cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem_bytes<D>(GROUPS));
    if (e != cudaSuccess) return e;
    note_launch();
    return launch_overlapped(attn_simt_kernel<D, MODE, GROUPS, SPLIT>, dim3((unsigned)tiles, (unsigned)(p.a.n_kv_heads * chunks)),
                             dim3(kThreads), smem_bytes<D>(GROUPS), s, p, Gp, chunks);
}

// Several groups where the blocks of one group would keep the SMs less than one and a half
// times busy: 2 x 700 tokens, 8/2 heads, d = 128 (178 blocks) 120 us, 166 us with one group;
// 8 x 300 tokens (316 blocks) 83 us with one, 114 us with two.
template <int D, int MODE, bool SPLIT>
cudaError_t launch_t(const AttnTileLaunch& p, cudaStream_t s) {
    int Gp, chunks;
    const int64_t tiles = blocks_of(p, 1, SPLIT, &Gp, &chunks);
    return tiles * p.a.n_kv_heads * chunks <= 228 ? launch_g<D, MODE, kGroups<D>, SPLIT>(p, s)
                                                    : launch_g<D, MODE, 1, SPLIT>(p, s);
}

template <int D>
cudaError_t launch_d(const AttnTileLaunch& p, cudaStream_t s) {
    if (p.prefix_lens) return launch_t<D, kPrefix, true>(p, s);
    if (p.n_split > 1) return p.a.block_table ? launch_t<D, kPaged, true>(p, s) : launch_t<D, kPacked, true>(p, s);
    return p.a.block_table ? launch_t<D, kPaged, false>(p, s) : launch_t<D, kPacked, false>(p, s);
}

}  // namespace

cudaError_t launch_attn_simt(const AttnTileLaunch& p, cudaStream_t s) {
    return p.a.d == 128 ? launch_d<128>(p, s) : launch_d<64>(p, s);
}

}  // namespace kda
