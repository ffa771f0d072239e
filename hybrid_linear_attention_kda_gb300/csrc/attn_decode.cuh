// Decode attention: the division of work, shared by the fp32 and bf16 suffix kernels.
//
// The keys that a sequence does not share (its suffix) are cut into tiles.  All
// tiles of all units (sequence, key/value head, block of query heads), in that
// order, form one line; it is cut into equal pieces, one for each worker (a warp),
// so that the workers finish together whatever the lengths are.  A unit inside one piece is finished there
// (with its prefix's partial results); of a unit that several pieces share, each
// leaves (m, l, unnormalised o), the piece in which it begins notes it, and the
// join adds the parts up from the first piece to the last, behind the prefix's
// blocks of keys.
//
// Joining partial results:  m = max_p m_p,  o = sum_p 2^(m_p - m) o_p,  l alike;
// scores are kept times log2(e).
#pragma once

#include <math_constants.h>

#include "attn_common.cuh"

namespace kda {
namespace decode {

constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

// The suffix kernel follows the prefix's kernel, where there are groups, and then starts
// beside it: that kernel starts when everything before it, the info kernel included,
// has completed, so only its own results are still to come.  They are waited for where
// they are joined, and by every worker before it ends, so that the join kernel follows
// both.
__device__ __forceinline__ void start_after(const AttnDecodeLaunch& p) {
    if (p.a.n_groups == 0) griddep_wait();
}

// Shared and total positions of sequence s.  With groups the info kernel has
// written them; without, they come straight from kv_lens.
__device__ __forceinline__ int2 seq_info(const AttnDecodeLaunch& p, int32_t s) {
    if (p.a.n_groups > 0) return p.info[s];
    const int64_t kv = p.a.kv_lens[s];
    return make_int2(0, kv < 0 || kv > (int64_t)p.a.table_stride * p.a.block_size ? 0 : (int)kv);
}
__device__ __forceinline__ int64_t seq_tiles(int2 info, int tile_keys) {
    return info.y > info.x ? ((uint32_t)(info.y - info.x) + (uint32_t)tile_keys - 1) / (uint32_t)tile_keys : 0;
}

// Division of counts that mostly fit 32 bits, where it takes a quarter of the time.
__device__ __forceinline__ int64_t divide(int64_t a, int64_t b) {
    return ((uint64_t)a | (uint64_t)b) >> 32 ? a / b : (int64_t)((uint32_t)a / (uint32_t)b);
}

// The line of `all` tiles has as many pieces as there are workers, or fewer of at least
// `least` tiles (decode_least_tiles).  Piece c holds the
// tiles [begin(c), begin(c + 1)); the first `more` pieces hold one tile more than the
// others.
struct Line {
    int64_t all, pieces, size, more;
    __device__ __forceinline__ Line(int64_t tiles, int64_t most, int least) : all(tiles) {
        pieces = min(most, divide(all + least - 1, least));
        size = pieces > 0 ? divide(all, pieces) : 0;
        more = all - size * pieces;
    }
    __device__ __forceinline__ int64_t begin(int64_t c) const { return c * size + min(c, more); }
    __device__ __forceinline__ int64_t piece_of(int64_t x) const {
        const int64_t long_ones = more * (size + 1);
        return x < long_ones ? divide(x, size + 1) : more + divide(x - long_ones, size);
    }
};

// A place on the line: unit u of sequence s, tiles k .. of its T.
struct Cursor {
    int64_t left;      // tiles of the piece from here on
    int32_t s;
    int32_t u, units;  // units of a sequence
    int64_t k, T;
    int2 info;

    __device__ __forceinline__ int64_t run() const { return T - k < left ? T - k : left; }   // tiles in this unit
    // One tile on.
    __device__ __forceinline__ void step(const AttnDecodeLaunch& p, int tile_keys) {
        if (k + 1 == T || left == 1) {
            next_unit(p, tile_keys);                     // (run() is 1 here)
        } else {
            ++k;
            --left;
        }
    }
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

// The pieces of a thread block of NT threads with PIECES workers: fills at[] for
// them (the caller's shared memory) and returns the line.  Thread i counts the tiles
// of its share of the sequences, one block scan gives the line's length, and the
// thread whose share holds a piece's first tile walks it again.
struct PieceStart {
    int32_t s;
    int2 info;
    int64_t rel;           // tiles past the first of s
};
template <int NT, int PIECES>
__device__ Line find_pieces(const AttnDecodeLaunch& p, int units, int tile_keys, PieceStart* at) {
    __shared__ int64_t scan_buf[NT / 32];
    const int32_t n = p.a.n_seqs;
    const int32_t share = (n + NT - 1) / NT, s0 = min(n, (int32_t)threadIdx.x * share), s1 = min(n, s0 + share);
    int64_t mine = 0;
#pragma unroll 4
    for (int32_t s = s0; s < s1; ++s) mine += seq_tiles(seq_info(p, s), tile_keys);
    int64_t total;
    const int64_t before = block_scan<NT>(mine, scan_buf, &total) - mine;
    const Line line(total * units, p.n_pieces, decode_least_tiles(divide(total, n)));
    for (int i = 0; i < PIECES; ++i) {
        const int64_t c = (int64_t)blockIdx.x * PIECES + i;
        if (c >= line.pieces) break;
        const int64_t begin = line.begin(c);
        if (before * units > begin || begin >= (before + mine) * units) continue;
        int64_t x = before;
        for (int32_t s = s0;; ++s) {
            const int2 info = seq_info(p, s);
            const int64_t t = seq_tiles(info, tile_keys);
            if (begin < (x + t) * units) {
                at[i] = PieceStart{s, info, begin - x * units};
                break;
            }
            x += t;
        }
    }
    __syncthreads();
    return line;
}

__device__ __forceinline__ Cursor start(const PieceStart& at, const Line& line, int64_t piece, int units, int tile_keys) {
    Cursor c;
    c.s = at.s;
    c.units = units;
    c.info = at.info;
    c.T = seq_tiles(at.info, tile_keys);
    c.u = (int32_t)divide(at.rel, c.T);
    c.k = at.rel - c.u * c.T;
    c.left = line.begin(piece + 1) - line.begin(piece);
    return c;
}

// What piece c leaves of a unit that it does not hold whole: slot 1 when the unit
// begins in it (then the join finds it noted in p.open), slot 0 otherwise.
__device__ __forceinline__ int64_t part_slot(int64_t c, bool begins) { return 2 * c + (begins ? 1 : 0); }

// Adds (m2, l2) to (m, l); the factors that the two sides' o take.
__device__ __forceinline__ void join(float& m, float& l, float m2, float l2, float& w, float& w2) {
    const float mx = fmaxf(m, m2), ms = mx == -CUDART_INF_F ? 0.f : mx;
    w = exp2f(m - ms), w2 = exp2f(m2 - ms);
    l = l * w + l2 * w2;
    m = mx;
}

// Blocks of keys that hold something of a shared prefix (the others' results are
// empty): as the prefix kernels cut it.
__device__ __forceinline__ int prefix_parts(const AttnDecodeLaunch& p, int shared) {
    if (shared <= 0) return 0;
    const uint32_t tiles = ((uint32_t)shared + p.prefix_tile - 1) / p.prefix_tile;
    const uint32_t per = prefix_block_tiles(shared, p.prefix_tile, p.n_split, p.split_cost);
    return (int)((tiles + per - 1) / per);
}
__device__ __forceinline__ int64_t prefix_row(const AttnDecodeLaunch& p, int i, int32_t s, int head) {
    return ((int64_t)i * p.a.n_seqs + s) * p.a.n_heads + head;
}
// Loads that are issued where they stand: a unit's end reads the prefix's results from L2,
// and among the results' stores the compiler asks for them a row at a time (53 requests of
// up to 5 fp32 tokens behind 256, 15/3 heads: 53 us, 47 us with these).
__device__ __forceinline__ float2 load_now2(const void* p) {
    float2 v;
    asm volatile("ld.global.v2.f32 {%0, %1}, [%2];" : "=f"(v.x), "=f"(v.y) : "l"(p) : "memory");
    return v;
}
__device__ __forceinline__ void write_lse(const kda_attn_decode_args& a, int32_t s, int head, float m, float l) {
    if (a.lse) a.lse[(int64_t)s * a.n_heads + head] = l == 0.f ? -CUDART_INF_F : fmaf(m, kLn2, logf(l));
}

// (m, l, o) of one row as a warp holds it, D / 32 columns a lane, and partial results
// added to it.  They come from L2, a microsecond away: four are asked for at a time.
template <int D> struct RowSum {
    static constexpr int kCols = D / 32;
    float m, l, o[kCols];

    __device__ __forceinline__ RowSum() {
        m = -CUDART_INF_F, l = 0.f;
#pragma unroll
        for (int e = 0; e < kCols; ++e) o[e] = 0.f;
    }
    __device__ __forceinline__ void add(float2 ml, const float (&x)[kCols]) {
        float w, w2;
        join(m, l, ml.x, ml.y, w, w2);
#pragma unroll
        for (int e = 0; e < kCols; ++e) o[e] = o[e] * w + x[e] * w2;
    }
    // Parts from .. to - 1 in turn; where(i, ml, o) names the i-th one's place.
    template <typename Where> __device__ __forceinline__ void add_parts(int64_t from, int64_t to, int lane, Where where) {
        constexpr int kAtOnce = 4;
        for (int64_t i = from; i < to; i += kAtOnce) {
            float2 ml[kAtOnce];
            alignas(8) float x[kAtOnce][kCols];
#pragma unroll
            for (int k = 0; k < kAtOnce; ++k) {
                ml[k] = make_float2(-CUDART_INF_F, 0.f);
#pragma unroll
                for (int e = 0; e < kCols; ++e) x[k][e] = 0.f;
                if (i + k < to) {
                    const float2* from_ml;
                    const float* from_o;
                    where(i + k, from_ml, from_o);
                    ml[k] = *from_ml;
#pragma unroll
                    for (int e = 0; e < kCols; e += 2)
                        *reinterpret_cast<float2*>(&x[k][e]) = *reinterpret_cast<const float2*>(from_o + lane * kCols + e);
                }
            }
#pragma unroll
            for (int k = 0; k < kAtOnce; ++k)
                if (i + k < to) add(ml[k], x[k]);
        }
    }
    template <typename T> __device__ __forceinline__ void write(const kda_attn_decode_args& a, int32_t s, int head, int lane) const {
        const float inv = l == 0.f ? 0.f : 1.f / l;
        T* out = static_cast<T*>(a.o) + s * a.o_stride + (int64_t)head * D + lane * kCols;
#pragma unroll
        for (int e = 0; e < kCols; ++e) Elem<T>::store(out + e, o[e] * inv);
        if (lane == 0) write_lse(a, s, head, m, l);
    }
};

// A worker's end: sequences without a suffix give zeros, or the prefix's results.  The
// heads of one sequence are spread over as many workers as there are for it.  Also
// reports bad lengths.
template <typename T, int D>
__device__ void finish_empty(const AttnDecodeLaunch& p, int64_t worker, int lane) {
    griddep_wait();
    const kda_attn_decode_args& a = p.a;
    const int n = p.n_pieces, w = (int)worker, each = max(1, n / a.n_seqs);
    const int part = a.n_seqs < n ? w / a.n_seqs : 0;
    if (part >= each) return;
    for (int32_t s = a.n_seqs < n ? w % a.n_seqs : w; s < a.n_seqs; s += n) {
        const int2 info = seq_info(p, s);
        if (a.n_groups == 0 && info.y != a.kv_lens[s] && lane == 0 && part == 0) flag(p.status, KDA_DEV_BAD_SEQLENS);
        if (info.y > info.x) continue;
        const int n_pre = prefix_parts(p, info.x);
        for (int head = part; head < a.n_heads; head += each) {
            RowSum<D> sum;
            sum.add_parts(0, n_pre, lane, [&](int64_t i, const float2*& ml, const float*& o) {
                const int64_t at = prefix_row(p, (int)i, s, head);
                ml = p.pre_ml + at;
                o = p.pre_o + at * D;
            });
            sum.template write<T>(a, s, head, lane);
        }
    }
}

constexpr int kJoinWarps = 8;

// Thread block c joins the unit that begins in piece c and ends in a later one, if
// there is one.  Its warps are spread over the unit's rows, and over its parts (the
// prefix's, then the pieces') when there are fewer rows than warps.  Bound by three
// trips to L2 and its launch: 83 requests of up to 863 tokens, 40/8 heads take 43 us with
// both kernels (47 us with the parts read one by one).
template <typename T, int D, int ROWS>
__global__ void __launch_bounds__(32 * kJoinWarps) join_kernel(const __grid_constant__ AttnDecodeLaunch p) {
    constexpr int kCols = D / 32;
    __shared__ float s_o[kJoinWarps][D];
    __shared__ float2 s_ml[kJoinWarps];
    griddep_wait();
    const kda_attn_decode_args& a = p.a;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t c0 = blockIdx.x;
    const int4 open = p.open[c0];                        // sequence (-1: none), unit, last piece, prefix parts
    if (open.x < 0) return;
    const int32_t s = open.x;
    const int n_pre = open.w;
    const int64_t parts = n_pre + open.z - c0 + 1;
    const int G = a.n_heads / a.n_kv_heads, blocks = (G + ROWS - 1) / ROWS;
    const int hk = open.y / blocks, rb = open.y % blocks;
    const int head0 = hk * G + rb * ROWS, rows = min(ROWS, G - rb * ROWS);
    const int row_warps = rows > 4 ? 8 : rows > 2 ? 4 : rows, part_warps = kJoinWarps / row_warps;
    const int r0 = warp % row_warps, pw = warp / row_warps;
    const int64_t per = (parts + part_warps - 1) / part_warps;
    for (int r = r0; r - r0 < rows; r += row_warps) {    // every warp the same number of times
        const int head = head0 + r;
        RowSum<D> sum;
        if (r < rows)
            sum.add_parts(pw * per, min(parts, (pw + 1) * per), lane, [&](int64_t i, const float2*& ml, const float*& o) {
                if (i < n_pre) {
                    const int64_t at = prefix_row(p, (int)i, s, head);
                    ml = p.pre_ml + at;
                    o = p.pre_o + at * D;
                } else {
                    const int64_t at = part_slot(c0 + i - n_pre, i == n_pre) * ROWS + r;
                    ml = p.part_ml + at;
                    o = p.part_o + at * D;
                }
            });
        if (part_warps > 1) {
            __syncthreads();
#pragma unroll
            for (int e = 0; e < kCols; ++e) s_o[warp][lane * kCols + e] = sum.o[e];
            if (lane == 0) s_ml[warp] = make_float2(sum.m, sum.l);
            __syncthreads();
            if (pw == 0)
                for (int i = 1; i < part_warps; ++i) {
                    float x[kCols];
#pragma unroll
                    for (int e = 0; e < kCols; ++e) x[e] = s_o[warp + i * row_warps][lane * kCols + e];
                    sum.add(s_ml[warp + i * row_warps], x);
                }
        }
        if (pw == 0 && r < rows) sum.template write<T>(a, s, head, lane);
    }
}

template <typename T, int D, int ROWS>
cudaError_t launch_join(const AttnDecodeLaunch& p, cudaStream_t s) {
    note_launch();
    return launch_overlapped(join_kernel<T, D, ROWS>, dim3((unsigned)p.n_pieces), dim3(32 * kJoinWarps), 0, s, p);
}

// Notes for the join whether the last unit of the piece, at cursor c, begins there
// and goes on in later pieces.
__device__ __forceinline__ int4 open_unit(const AttnDecodeLaunch& p, const Cursor& c, int64_t piece, const Line& line) {
    const int64_t rest = c.T - (c.k + c.run());          // its tiles in later pieces
    if (c.k != 0 || rest == 0) return make_int4(-1, 0, 0, 0);
    return make_int4(c.s, c.u, (int)line.piece_of(line.begin(piece + 1) + rest - 1), prefix_parts(p, c.info.x));
}

}  // namespace decode
}  // namespace kda
