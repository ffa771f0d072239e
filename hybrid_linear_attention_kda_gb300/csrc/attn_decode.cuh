// Decode attention: the division of work, shared by the fp32 and bf16 suffix kernels.
//
// The keys that a sequence does not share (its suffix) are cut into tiles.  All
// tiles of all units (sequence, key/value head, block of query heads), in that
// order, form one line; it is cut into equal pieces, one for each thread block, so
// the blocks finish together whatever the lengths are.  A unit inside one piece is
// finished there (with its prefix's partial results); of a unit that several pieces
// share, each leaves (m, l, unnormalised o), and the join adds them up from the
// first piece to the last, behind the prefix's blocks of keys.
//
// Joining partial results:  m = max_p m_p,  o = sum_p 2^(m_p - m) o_p,  l alike;
// scores are kept times log2(e).
#pragma once

#include <math_constants.h>

#include "attn_common.cuh"

namespace kda {
namespace decode {

constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

// Shared and total positions of sequence s.  With groups the info kernel has
// written them; without, they come straight from kv_lens.
__device__ __forceinline__ int2 seq_info(const AttnDecodeLaunch& p, int32_t s) {
    if (p.a.n_groups > 0) return p.info[s];
    const int64_t kv = p.a.kv_lens[s];
    return make_int2(0, kv < 0 || kv > (int64_t)p.a.table_stride * p.a.block_size ? 0 : (int)kv);
}
__device__ __forceinline__ int64_t seq_tiles(int2 info, int tile_keys) {
    return info.y > info.x ? ((int64_t)info.y - info.x + tile_keys - 1) / tile_keys : 0;
}

// The line has as many pieces as there are thread blocks, but none is empty:
// piece c holds the tiles [begin(c), begin(c + 1)).
__device__ __forceinline__ int64_t n_pieces(int64_t all, int64_t n_ctas) { return all < n_ctas ? all : n_ctas; }
__device__ __forceinline__ int64_t piece_begin(int64_t all, int64_t c, int64_t n) {
    return all / n * c + all % n * c / n;
}

// A place on the line: unit u of sequence s, tiles k .. of its T.
struct Cursor {
    int64_t left;      // tiles of the piece from here on
    int32_t s;
    int32_t u, units;  // units of a sequence
    int64_t k, T;
    int2 info;

    __device__ __forceinline__ int64_t run() const { return T - k < left ? T - k : left; }   // tiles in this unit
    // To the next unit of the piece (left > 0 afterwards unless it was the last).
    __device__ __forceinline__ void next_unit(const AttnDecodeLaunch& p, int tile_keys) {
        left -= run();
        k = 0;
        if (++u < units || left <= 0) return;
        u = 0;
        do {
            info = seq_info(p, ++s);
            T = seq_tiles(info, tile_keys);
        } while (T == 0);
    }
};

// Start of this thread block's piece; false when it has none.  Thread i counts the
// tiles of its share of the sequences, one block scan gives the line's length and
// the thread whose share holds the piece's first tile walks it again.  Block 0
// writes the running counts that the join reads, and reports bad lengths.
template <int NT>
__device__ bool find_piece(const AttnDecodeLaunch& p, int units, int tile_keys, Cursor& c) {
    __shared__ int64_t scan_buf[NT / 32];
    __shared__ int32_t found_s;
    __shared__ int64_t found_rel;
    const int32_t n = p.a.n_seqs;
    const int32_t share = (n + NT - 1) / NT, s0 = min(n, (int32_t)threadIdx.x * share), s1 = min(n, s0 + share);
    int64_t mine = 0;
    for (int32_t s = s0; s < s1; ++s) mine += seq_tiles(seq_info(p, s), tile_keys);
    int64_t total;
    int64_t before = block_scan<NT>(mine, scan_buf, &total) - mine;
    if (blockIdx.x == 0) {
        int64_t t = before;
        for (int32_t s = s0; s < s1; ++s) {
            const int2 info = seq_info(p, s);
            if (p.a.n_groups == 0) {
                const int32_t kv = p.a.kv_lens[s];
                if (kv != info.y) flag(p.status, KDA_DEV_BAD_SEQLENS);
                p.info[s] = info;
            }
            p.tiles[s] = t;
            t += seq_tiles(info, tile_keys);
        }
        if (threadIdx.x == 0) p.tiles[n] = total;
    }
    const int64_t all = total * units, pieces = n_pieces(all, p.n_ctas);
    if ((int64_t)blockIdx.x >= pieces) return false;
    const int64_t at = piece_begin(all, blockIdx.x, pieces);
    if (before * units <= at && at < (before + mine) * units) {
        int32_t s = s0;
        for (;; ++s) {
            const int64_t t = seq_tiles(seq_info(p, s), tile_keys);
            if (at < (before + t) * units) break;
            before += t;
        }
        found_s = s;
        found_rel = at - before * units;
    }
    __syncthreads();
    c.s = found_s;
    c.units = units;
    c.info = seq_info(p, c.s);
    c.T = seq_tiles(c.info, tile_keys);
    c.u = (int32_t)(found_rel / c.T);
    c.k = found_rel % c.T;
    c.left = piece_begin(all, (int64_t)blockIdx.x + 1, pieces) - at;
    return true;
}

// Adds (m2, l2) to (m, l); the factors that the two sides' o take.
__device__ __forceinline__ void join(float& m, float& l, float m2, float l2, float& w, float& w2) {
    const float mx = fmaxf(m, m2), ms = mx == -CUDART_INF_F ? 0.f : mx;
    w = exp2f(m - ms), w2 = exp2f(m2 - ms);
    l = l * w + l2 * w2;
    m = mx;
}

__device__ __forceinline__ int64_t prefix_row(const AttnDecodeLaunch& p, int i, int32_t s, int head) {
    return ((int64_t)i * p.a.n_seqs + s) * p.a.n_heads + head;
}
__device__ __forceinline__ void write_lse(const kda_attn_decode_args& a, int32_t s, int head, float m, float l) {
    if (a.lse) a.lse[(int64_t)s * a.n_heads + head] = l == 0.f ? -CUDART_INF_F : fmaf(m, kLn2, logf(l));
}

// One thread block of four warps for each unit; a warp takes every fourth row, a
// lane D / 32 columns.
template <typename T, int D, int ROWS>
__global__ void __launch_bounds__(128) join_kernel(const __grid_constant__ AttnDecodeLaunch p) {
    constexpr int kCols = D / 32;
    griddep_wait();
    const kda_attn_decode_args& a = p.a;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int G = a.n_heads / a.n_kv_heads, blocks = (G + ROWS - 1) / ROWS;
    const int64_t U = (int64_t)a.n_kv_heads * blocks;
    const int32_t s = (int32_t)(blockIdx.x / U);
    const int u = (int)(blockIdx.x - s * U), hk = u / blocks, rb = u % blocks;
    const int head0 = hk * G + rb * ROWS, rows = min(ROWS, G - rb * ROWS);
    const int2 info = p.info[s];
    const int64_t T_s = p.tiles[s + 1] - p.tiles[s], all = p.tiles[a.n_seqs] * U;
    const int64_t lo = p.tiles[s] * U + u * T_s;
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
        c1 = piece(lo + T_s - 1);
        if (c0 == c1) return;                            // written by its piece
    }
    const int n_pre = info.x > 0 ? p.n_split : 0;
    for (int r = warp; r < rows; r += 4) {
        const int head = head0 + r;
        float m = -CUDART_INF_F, l = 0.f, o[kCols] = {};
        auto add = [&](const float2 ml, const float* src) {
            float x[kCols];
#pragma unroll
            for (int e = 0; e < kCols; ++e) x[e] = src[lane * kCols + e];
            float w, w2;
            join(m, l, ml.x, ml.y, w, w2);
#pragma unroll
            for (int e = 0; e < kCols; ++e) o[e] = o[e] * w + x[e] * w2;
        };
#pragma unroll 4
        for (int i = 0; i < n_pre; ++i) {
            const int64_t at = prefix_row(p, i, s, head);
            add(p.pre_ml[at], p.pre_o + at * D);
        }
#pragma unroll 4
        for (int64_t c = c0; c <= c1; ++c) {
            const int64_t at = (2 * c + (c == c0 ? 1 : 0)) * ROWS + r;
            add(p.part_ml[at], p.part_o + at * D);
        }
        T* out = static_cast<T*>(a.o) + s * a.o_stride + (int64_t)head * D + lane * kCols;
        const float inv = l == 0.f ? 0.f : 1.f / l;
#pragma unroll
        for (int e = 0; e < kCols; ++e) Elem<T>::store(out + e, o[e] * inv);
        if (lane == 0) write_lse(a, s, head, m, l);
    }
}

template <typename T, int D, int ROWS>
cudaError_t launch_join(const AttnDecodeLaunch& p, cudaStream_t s) {
    const int G = p.a.n_heads / p.a.n_kv_heads;
    const int64_t units = (int64_t)p.a.n_seqs * p.a.n_kv_heads * ((G + ROWS - 1) / ROWS);
    note_launch();
    return launch_overlapped(join_kernel<T, D, ROWS>, dim3((unsigned)units), dim3(128), 0, s, p);
}

}  // namespace decode
}  // namespace kda
