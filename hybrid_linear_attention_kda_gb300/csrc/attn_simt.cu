// Softmax attention of row tiles for fp32 tensors, in SIMT arithmetic: prompts (causal)
// and the shared prefixes of decode attention.
//
// For the rows i of a tile and the keys j that row i sees (x_ij = scale q_i . k_j):
//     m = max_j x_ij,  l = sum_j exp(x_ij - m),  o_i = sum_j exp(x_ij - m) v_j / l
// in one pass over key tiles, with o and l rescaled whenever m grows.  Scores are
// kept times log2(e), so that exp is exp2.
//
// 256 threads own 64 rows x 64 keys, thread (ty, tx) the rows 4 ty .. 4 ty + 3, the
// keys tx + 16 c of the score tile and the columns 4 tx + 64 c of the output.  K is
// padded by 16 bytes a row, so that the 16 threads of a row group read distinct
// banks; the weights reuse K's place.  Bound by the FP32 pipe and the shared-memory
// reads that feed it.
#include <math_constants.h>

#include "attn_common.cuh"

namespace kda {
namespace {

constexpr int kRows = 64, kKeys = 64, kThreads = 256;
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

enum Mode { kPacked, kPaged, kPrefix };

template <int D> constexpr int kPad = D + 4;
template <int D> constexpr int kPPad = kKeys + 4;
template <int D> constexpr size_t smem_bytes() {
    return sizeof(float) * ((size_t)kRows * kPad<D> + (size_t)kKeys * kPad<D> + (size_t)kKeys * D);
}

__device__ __forceinline__ float4 load4(const float* p) { return *reinterpret_cast<const float4*>(p); }
__device__ __forceinline__ void store4(float* p, float4 x) { *reinterpret_cast<float4*>(p) = x; }

template <int D, int MODE>
__global__ void __launch_bounds__(kThreads) attn_simt_kernel(AttnTileLaunch p, int32_t Gp, int32_t chunks) {
    extern __shared__ __align__(16) float smem[];
    float* Qs = smem;
    float* Ks = Qs + kRows * kPad<D>;
    float* Vs = Ks + kKeys * kPad<D>;
    float* Ps = Ks;
    static_assert(kPPad<D> <= kPad<D>, "the weights fit in K's place");
    const kda_attn_prefill_args& a = p.a;
    const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4;
    const int G = a.n_heads / a.n_kv_heads;
    const int hk = (int)(blockIdx.y / chunks), hc = (int)(blockIdx.y % chunks);
    const int head0 = hk * G + hc * Gp, gn = min(Gp, G - hc * Gp);
    const int bt = kRows / Gp;                       // tokens of a tile
    const int64_t idx = MODE == kPrefix ? blockIdx.x / p.n_split : blockIdx.x;
    const int split = MODE == kPrefix ? (int)(blockIdx.x % p.n_split) : 0;
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
    if (MODE == kPrefix) {
        const int64_t per = ((K + kKeys - 1) / kKeys + p.n_split - 1) / p.n_split * kKeys;
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

    for (int64_t k0 = k_lo; k0 < k_hi; k0 += kKeys) {
        __syncthreads();                              // the previous tile is consumed (or Q is written)
        for (int i = tid; i < kKeys * (D / 4); i += kThreads) {
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
        __syncthreads();
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
        __syncthreads();                              // K is read: the weights take its place
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

#pragma unroll
    for (int r = 0; r < 4; ++r) {
        const int t = (ty * 4 + r) / Gp, g = (ty * 4 + r) % Gp;
        if (t >= nt || g >= gn) continue;
        const int64_t row = rt.row0 + rt.t0 + t;
        const int head = head0 + g;
        if (MODE == kPrefix) {
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

template <int D, int MODE>
cudaError_t launch_t(const AttnTileLaunch& p, cudaStream_t s) {
    const kda_attn_prefill_args& a = p.a;
    const int G = a.n_heads / a.n_kv_heads, Gp = G < kRows ? G : kRows, chunks = (G + Gp - 1) / Gp;
    int64_t tiles = a.total_tokens / (kRows / Gp) + a.n_seqs;
    if (MODE == kPrefix) tiles *= p.n_split;
    const cudaError_t e = cudaFuncSetAttribute(attn_simt_kernel<D, MODE>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               (int)smem_bytes<D>());
    if (e != cudaSuccess) return e;
    note_launch();
    attn_simt_kernel<D, MODE><<<dim3((unsigned)tiles, (unsigned)(a.n_kv_heads * chunks)), kThreads, smem_bytes<D>(), s>>>(
        p, Gp, chunks);
    return cudaGetLastError();
}

template <int D>
cudaError_t launch_d(const AttnTileLaunch& p, cudaStream_t s) {
    if (p.prefix_lens) return launch_t<D, kPrefix>(p, s);
    return p.a.block_table ? launch_t<D, kPaged>(p, s) : launch_t<D, kPacked>(p, s);
}

}  // namespace

cudaError_t launch_attn_simt(const AttnTileLaunch& p, cudaStream_t s) {
    return p.a.d == 128 ? launch_d<128>(p, s) : launch_d<64>(p, s);
}

}  // namespace kda
