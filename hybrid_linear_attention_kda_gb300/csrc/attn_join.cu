// Join of prompts whose keys were cut into blocks (few rows, many keys): for each row
//     m = max_p m_p,  l = sum_p 2^(m_p - m) l_p,  o = sum_p 2^(m_p - m) o_p / l
// over its n_split partial results, in order.  A warp takes a row, a lane D / 32
// columns.  Bound by its launch and a few trips to L2, about 5 us.
#include "attn_decode.cuh"

namespace kda {
namespace {

constexpr int kThreads = 256;

template <typename T, int D>
__global__ void __launch_bounds__(kThreads) prompt_join_kernel(const __grid_constant__ AttnTileLaunch p) {
    constexpr int kCols = D / 32;
    griddep_wait();
    const kda_attn_prefill_args& a = p.a;
    const int64_t rows = a.total_tokens * a.n_heads, r = ((int64_t)blockIdx.x * kThreads + threadIdx.x) / 32;
    const int lane = threadIdx.x & 31;
    if (r >= rows) return;
    if (__float_as_uint(p.part_ml[r].y) == 0x01010101u * kUnwritten) return;
    float m = -CUDART_INF_F, l = 0.f, o[kCols] = {};
#pragma unroll 4
    for (int i = 0; i < p.n_split; ++i) {
        const int64_t at = i * rows + r;
        const float2 ml = p.part_ml[at];
        if (ml.y == 0.f) continue;
        float w, w2;
        decode::join(m, l, ml.x, ml.y, w, w2);
#pragma unroll
        for (int e = 0; e < kCols; ++e) o[e] = o[e] * w + p.part_o[at * D + lane * kCols + e] * w2;
    }
    const int64_t token = r / a.n_heads, head = r - token * a.n_heads;
    const float inv = l == 0.f ? 0.f : 1.f / l;
    T* out = static_cast<T*>(a.o) + token * a.o_stride + head * D + lane * kCols;
#pragma unroll
    for (int e = 0; e < kCols; ++e) Elem<T>::store(out + e, o[e] * inv);
    if (a.lse && lane == 0) a.lse[r] = l == 0.f ? -CUDART_INF_F : fmaf(m, decode::kLn2, logf(l));
}

template <typename T, int D>
cudaError_t launch_t(const AttnTileLaunch& p, cudaStream_t s) {
    const int64_t rows = p.a.total_tokens * p.a.n_heads;
    note_launch();
    return launch_overlapped(prompt_join_kernel<T, D>, dim3((unsigned)((rows + kThreads / 32 - 1) / (kThreads / 32))),
                             dim3(kThreads), 0, s, p);
}

}  // namespace

cudaError_t launch_prompt_join(const AttnTileLaunch& p, cudaStream_t s) {
    if (p.a.dtype == KDA_BF16) return p.a.d == 128 ? launch_t<__nv_bfloat16, 128>(p, s) : launch_t<__nv_bfloat16, 64>(p, s);
    return p.a.d == 128 ? launch_t<float, 128>(p, s) : launch_t<float, 64>(p, s);
}

}  // namespace kda
