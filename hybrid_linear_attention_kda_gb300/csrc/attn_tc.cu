// Softmax attention of row tiles on the tensor cores (bf16): prompts (causal) and
// the shared prefixes of decode attention.
//
// For the rows i of a tile and the keys j that row i sees, with s = q k^T:
//     m_i = max_j s_ij,  l_i = sum_j exp2(c (s_ij - m_i)),  o_i = sum_j exp2(c (s_ij - m_i)) v_j / l_i
// (c = |scale| log2(e); a negative scale negates q in the MMA descriptor), in one
// pass over tiles of 128 keys.  A thread block takes two tiles of 128 rows of one
// key/value head, so that one computes its softmax while the tensor core works on
// the other, and every key tile that is loaded serves 256 rows:
//     S_q = Q_q K^T      128 x 128 x d, both operands in shared memory, S in TMEM
//     O_q += P_q V       128 x d x 128, P (bf16) in TMEM in S's place, O in TMEM
// Roles: warps 0-3 and 4-7 the softmax of tile 0 and 1 (a thread owns a row: no
// reductions between threads), warp 8 issues the MMAs, warp 9 the TMA copies of Q
// and of K and V into a ring of stages, warps 10-11 make the values at the edge of
// what the rows see safe (below).
//
// The maximum that weights refer to is the first tile's, and is only moved when a
// half tile's weights add up to more than 2^10: until then no weight is larger, l
// and o are sums of the same weights whatever they refer to (their rounding is
// relative), and neither a maximum nor a rescaled O is needed.  A move is done by
// the rows' own threads, while no product into O is under way: for the first half of
// a tile because its scores' commit came after the last one, for the second half
// after a commit that follows the first half's product.
//
// Hidden values.  A product with P has 0 * v for hidden keys, which is NaN for an
// infinite or NaN v.  In the tiles that some row sees only a part of, warps 10-11
// therefore zero the values of keys that no row sees, and replace the non-finite
// values of the others by zero and note the first key of each column that held a
// NaN, +inf or -inf; at the end, rows that see such a key get it added.
//
// Bound by the tensor pipe: 4 d flops per (row, key) pair.  Measured on 4 x 8192
// tokens, 32 query and 8 key/value heads, d = 128: 1.48 ms, 1485 TFLOP/s.
#include <cuda.h>
#include <math_constants.h>

#include <climits>

#include "attn_common.cuh"
#include "tc05.cuh"

namespace kda {
namespace {
using namespace tc;

constexpr int kTile = 128;                    // rows of a tile, keys of a tile
constexpr int kMmaWarp = 8, kLoadWarp = 9, kGuardWarp = 10, kGuardWarps = 2;
constexpr int kThreads = 384;
// Registers a thread: 168 at launch; the softmax warps hold a whole row of scores.
// 256 * 208 + 128 * 88 <= 384 * 168.
constexpr int kSoftmaxRegs = 208, kOtherRegs = 88;
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
constexpr float kMostWeight = 1024.f;         // of a half tile, before the maximum moves
constexpr uint32_t kTmemCols = 512;           // S0 0, S1 128, O0 256, O1 384

enum Mode { kPacked, kPaged, kPrefix };

template <int D> struct Shape {
    static constexpr uint32_t kRegion = kTile * 128u;            // 128 rows x 64 columns, 128-byte swizzle
    static constexpr uint32_t kTileBytes = kRegion * (D / 64);
    static constexpr int kStages = D == 128 ? 5 : 8;
    static constexpr uint32_t kQ = 0, kRing = 2 * kTileBytes, kMisc = kRing + kStages * kTileBytes;
};

template <int D> struct Misc {
    uint64_t full[Shape<D>::kStages], empty[Shape<D>::kStages];
    uint64_t guarded[Shape<D>::kStages];
    uint64_t q_full, s_full[2], p_ready[2][2], half_done[2], o_done[2];   // p_ready: [row tile][half of the keys]
    uint32_t tslot;
    int32_t failed, poison;
    int32_t first_nan[D], first_pos[D], first_neg[D];            // first key of a column that holds such a value
};

template <int D> constexpr size_t smem_bytes() { return Shape<D>::kMisc + sizeof(Misc<D>) + 1024; }

struct Maps {
    CUtensorMap q, k, v;
};

// ------------------------------------------------------------------ PTX

__device__ __forceinline__ void tma_load_3d(void* dst, const void* tmap, int32_t x, int32_t y, int32_t z, uint64_t* bar) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::
            "r"(smem_u32(dst)),
        "l"(reinterpret_cast<uint64_t>(tmap)), "r"(x), "r"(y), "r"(z), "r"(smem_u32(bar))
        : "memory");
}
// The MMA warp runs its loop as a whole and lets one lane issue, so that the
// descriptors stay in uniform registers: issued from inside a one-lane branch, each
// MMA took 90 cycles of register moves, against 64 of the tensor pipe.
__device__ __forceinline__ uint32_t elect_one() {
    uint32_t e;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(e));
    return e;
}
// D[tmem] (+)= A[smem desc] x B[smem desc]^T, issued where `leader` is set.
__device__ __forceinline__ void mma_ss(uint32_t leader, uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                       uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p, e;\n\t"
        "setp.ne.b32 e, %0, 0;\n\t"
        "setp.ne.b32 p, %5, 0;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%1], %2, %3, %4, p;\n\t}" ::"r"(leader),
        "r"(d_tmem), "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
}
// D[tmem] (+)= A[tmem, bf16 pairs] x B[smem desc]^T.
__device__ __forceinline__ void mma_ts(uint32_t leader, uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint32_t idesc,
                                       uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p, e;\n\t"
        "setp.ne.b32 e, %0, 0;\n\t"
        "setp.ne.b32 p, %5, 0;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%1], [%2], %3, %4, p;\n\t}" ::"r"(leader),
        "r"(d_tmem), "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
}
__device__ __forceinline__ void commit(uint32_t leader, uint64_t* bar) {
    asm volatile(
        "{\n\t.reg .pred e;\n\t"
        "setp.ne.b32 e, %0, 0;\n\t"
        "@e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%1];\n\t}" ::"r"(leader),
        "r"(smem_u32(bar))
        : "memory");
}
__device__ __forceinline__ void tmem_ld32(uint32_t taddr, uint32_t* r) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, "
        "[%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
          "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
          "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(taddr));
}
__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t* r) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], "
        "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::
            "r"(taddr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
        "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]),
        "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]),
        "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
        : "memory");
}
__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// Pairs of fp32 values in one 64-bit register, for the two-wide fp32 instructions.
__device__ __forceinline__ uint64_t pair2(uint32_t lo, uint32_t hi) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "r"(lo), "r"(hi));
    return r;
}
__device__ __forceinline__ float2 unpair2(uint64_t x) {
    uint32_t lo, hi;
    asm("mov.b64 {%0, %1}, %2;" : "=r"(lo), "=r"(hi) : "l"(x));
    return make_float2(__uint_as_float(lo), __uint_as_float(hi));
}
__device__ __forceinline__ uint64_t pair2(float x) { return pair2(__float_as_uint(x), __float_as_uint(x)); }
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
template <int N> __device__ __forceinline__ void more_registers() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N)); }
template <int N> __device__ __forceinline__ void fewer_registers() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N)); }

// A place in the ring of stages, as it moves from load to load: one warp's scalar
// arithmetic between two MMAs is time that the tensor pipe waits.
struct Ring {
    uint32_t stage = 0, phase = 0;
    __device__ __forceinline__ void next(uint32_t stages) {
        if (++stage == stages) {
            stage = 0;
            phase ^= 1u;
        }
    }
};

// ------------------------------------------------------------------ the block's work

struct Work {
    RowTile rt;
    int hk, split;
    int64_t K, first;             // keys of the sequence; row of token t sees the keys j <= first + t
    int64_t k_lo, k_hi;           // keys that some row of the block sees
    int64_t all_see;              // every row sees the keys below this one
    int n_keys[2];                // key tiles of each row tile
    int tokens;                   // of a row tile
    const int32_t* table;
};

template <int MODE>
__device__ bool find_work(const AttnTileLaunch& p, Work& w) {
    const kda_attn_prefill_args& a = p.a;
    const int G = a.n_heads / a.n_kv_heads;
    const int64_t idx = blockIdx.x / a.n_kv_heads;
    w.hk = (int)(blockIdx.x - idx * a.n_kv_heads);
    w.tokens = kTile / G;
    w.split = MODE == kPrefix ? (int)(idx % p.n_split) : 0;
    w.rt = find_tile<kThreads>(a.cu_seqlens, a.n_seqs, a.total_tokens, 2 * w.tokens, MODE == kPrefix ? idx / p.n_split : idx,
                               MODE != kPrefix && blockIdx.x == 0, KDA_DEV_BAD_SEQLENS, p.status);
    if (w.rt.seq < 0) return false;
    const int64_t cap = (int64_t)a.table_stride * a.block_size;
    w.table = nullptr;
    if (MODE == kPacked) {
        w.K = w.rt.n;
        w.first = 0;
    } else if (MODE == kPaged) {
        w.K = a.kv_lens[w.rt.seq];
        w.table = a.block_table + (int64_t)w.rt.seq * a.table_stride;
        if (w.K < 0 || w.K > cap) {
            if (threadIdx.x == 0) flag(p.status, KDA_DEV_BAD_SEQLENS);
            return false;
        }
        w.first = w.K - w.rt.n;
    } else {
        w.K = p.prefix_lens[w.rt.seq];
        w.table = a.block_table + w.rt.row0 * a.table_stride;
        if (w.K < 0 || w.K > cap || w.K % a.block_size) w.K = 0;           // flagged by the decode plan
        w.first = w.K;
    }
    const int left = w.rt.n - w.rt.t0;                                     // tokens from the first one on
    if (MODE == kPrefix) {
        const int64_t per = ((w.K + kTile - 1) / kTile + p.n_split - 1) / p.n_split * kTile;
        w.k_lo = min(w.K, w.split * per);
        w.k_hi = w.all_see = min(w.K, w.k_lo + per);
        w.n_keys[0] = w.n_keys[1] = (int)((w.k_hi - w.k_lo + kTile - 1) / kTile);
    } else {
        w.k_lo = 0;
        auto seen = [&](int tokens) { return max((int64_t)0, min(w.K, w.first + w.rt.t0 + tokens)); };
        w.all_see = seen(1);
        const int64_t k0 = seen(min(left, w.tokens));
        w.k_hi = seen(min(left, 2 * w.tokens));
        w.n_keys[0] = (int)((k0 + kTile - 1) / kTile);
        w.n_keys[1] = (int)((w.k_hi + kTile - 1) / kTile);
    }
    if (left <= w.tokens) w.n_keys[1] = 0;
    return true;
}

// ------------------------------------------------------------------ kernel

template <int D, int MODE>
__global__ void __launch_bounds__(kThreads, 1)
attn_tc_kernel(const __grid_constant__ AttnTileLaunch p, const __grid_constant__ Maps maps) {
    using Sh = Shape<D>;
    constexpr int kRegions = D / 64;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    Misc<D>& ms = *reinterpret_cast<Misc<D>*>(sm + Sh::kMisc);
    const uint32_t s_base = smem_u32(sm);
    const kda_attn_prefill_args& a = p.a;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int G = a.n_heads / a.n_kv_heads;
    Work w;
    if (!find_work<MODE>(p, w)) return;

    if (warp == kMmaWarp) tmem_alloc(&ms.tslot, kTmemCols);
    if (tid == 0) {
        for (int i = 0; i < Sh::kStages; ++i) {
            mbar_init(&ms.full[i], 1);
            mbar_init(&ms.empty[i], 1 + kGuardWarps);
            mbar_init(&ms.guarded[i], 32 * kGuardWarps);
        }
        mbar_init(&ms.q_full, 1);
        for (int i = 0; i < 2; ++i) {
            mbar_init(&ms.s_full[i], 1);
            mbar_init(&ms.p_ready[i][0], 4);
            mbar_init(&ms.p_ready[i][1], 4);
            mbar_init(&ms.half_done[i], 1);
            mbar_init(&ms.o_done[i], 1);
        }
        ms.failed = 0;
        ms.poison = 0;
        fence_mbar_init();
    }
    for (int i = tid; i < D; i += kThreads) ms.first_nan[i] = ms.first_pos[i] = ms.first_neg[i] = INT_MAX;
    fence_before_sync();
    __syncthreads();
    fence_after_sync();
    constexpr uint32_t tbase = 0;                 // all of tensor memory is this block's
    auto tS = [](int q) { return tbase + 128u * q; };
    auto tO = [](int q) { return tbase + 256u + 128u * q; };
    auto waitb = [&](uint64_t* bar, uint32_t parity) -> bool {
        if (mbar_wait(bar, parity)) return true;
        atomicExch(&ms.failed, 1);
        flag(p.status, KDA_DEV_WAIT_TIMEOUT);
        return false;
    };
    // the same for a whole warp, whose lanes then agree
    auto wait_all = [&](uint64_t* bar, uint32_t parity) -> bool { return __all_sync(0xffffffffu, waitb(bar, parity)); };
    const int n_tiles = max(w.n_keys[0], w.n_keys[1]);
    // ring stage of the i-th load (K of tile j: 2 j, V of tile j: 2 j + 1) and the parity of its phase
    auto stage_of = [&](int i) { return i % Sh::kStages; };
    auto phase_of = [&](int i) { return (uint32_t)(i / Sh::kStages) & 1u; };
    // from this tile on some row sees only a part of the keys
    const int first_edge = (int)(max((int64_t)0, w.all_see - w.k_lo) / kTile);

    // the register split is made inside the branches: after a merge of the two the
    // compiler would hold everything to the smaller share
    if (warp >= kMmaWarp) {
        fewer_registers<kOtherRegs>();
        if (warp == kMmaWarp) {
            if (n_tiles > 0) {
                const uint32_t leader = elect_one();
                const uint32_t id_s = idesc_bf16(kTile, kTile, false, false) | (a.scale < 0.f ? 1u << 13 : 0u);
                const uint32_t id_o = idesc_bf16(kTile, D, false, true);
                const uint64_t d_kmajor = sdesc(0, 16, 1024), d_mnmajor = sdesc(0, Sh::kRegion, 1024);
                auto at = [](uint64_t desc, uint32_t byte) { return desc + (uint64_t)(byte >> 4); };
                auto scores = [&](int q, int stage) {
                    const uint32_t qb = s_base + Sh::kQ + q * Sh::kTileBytes, kb = s_base + Sh::kRing + stage * Sh::kTileBytes;
    #pragma unroll
                    for (int ks = 0; ks < D / 16; ++ks) {
                        const uint32_t off = (ks >> 2) * Sh::kRegion + (ks & 3) * 32;
                        mma_ss(leader, tS(q), at(d_kmajor, qb + off), at(d_kmajor, kb + off), id_s, ks > 0);
                    }
                    commit(leader, &ms.s_full[q]);
                };
                auto values = [&](int q, int half, int stage, bool first) {
                    const uint32_t vb = s_base + Sh::kRing + stage * Sh::kTileBytes;
    #pragma unroll
                    for (int ks = 4 * half; ks < 4 * half + 4; ++ks)
                        mma_ts(leader, tO(q), tS(q) + 8 * ks, at(d_mnmajor, vb + ks * 2048), id_o, !first || ks > 0);
                };
                bool ok = wait_all(&ms.q_full, 0) && wait_all(&ms.full[0], 0);
                if (ok) {
                    fence_after_sync();
                    for (int q = 0; q < 2; ++q)
                        if (w.n_keys[q] > 0) scores(q, 0);
                    commit(leader, &ms.empty[0]);
                }
                uint32_t guard_phase = 0;                         // a bit for each stage
                Ring v;
                v.next(Sh::kStages);
                // Waits for the copies stand between the MMAs of one row tile, where the
                // tensor pipe still has work.
                auto v_ready = [&](int j) -> bool {
                    if (!wait_all(&ms.full[v.stage], v.phase)) return false;
                    if (j >= first_edge) {
                        if (!wait_all(&ms.guarded[v.stage], guard_phase >> v.stage & 1)) return false;
                        guard_phase ^= 1u << v.stage;
                    }
                    return true;
                };
                ok = ok && v_ready(0);
                for (int j = 0; j < n_tiles && ok; ++j) {
                    const uint32_t vs = v.stage;
                    v.next(Sh::kStages);
                    const Ring k = v;
                    v.next(Sh::kStages);
                    const bool more = j + 1 < n_tiles;
                    if (more && !(ok = wait_all(&ms.full[k.stage], k.phase))) break;
#pragma unroll
                    for (int q = 0; q < 2; ++q) {
                        if (j < w.n_keys[q]) {
                            if (!(ok = wait_all(&ms.p_ready[q][0], j & 1))) break;
                            fence_after_sync();
                            values(q, 0, vs, j == 0);
                            commit(leader, &ms.half_done[q]);
                            if (!(ok = wait_all(&ms.p_ready[q][1], j & 1))) break;
                            fence_after_sync();
                            values(q, 1, vs, false);
                            if (j + 1 == w.n_keys[q]) commit(leader, &ms.o_done[q]);
                        }
                        if (q == 1) commit(leader, &ms.empty[vs]);
                        if (j + 1 < w.n_keys[q]) scores(q, k.stage);
                    }
                    if (ok && more) commit(leader, &ms.empty[k.stage]);
                    if (ok && more && !(ok = v_ready(j + 1))) break;
                }
                if (!ok) {
                    // let the MMAs in flight finish before shared and tensor memory go
                    commit(leader, &ms.q_full);
                    mbar_wait(&ms.q_full, 1);
                }
            }
        } else if (warp == kLoadWarp) {
            if (n_tiles > 0) {
                if (lane == 0) {
                    const int tiles = w.n_keys[1] > 0 ? 2 : 1;
                    mbar_expect_tx(&ms.q_full, (uint32_t)tiles * kRegions * (uint32_t)(w.tokens * G) * 128u);
                    for (int q = 0; q < tiles; ++q)
                        for (int c = 0; c < kRegions; ++c)
                            tma_load_3d(sm + Sh::kQ + q * Sh::kTileBytes + c * Sh::kRegion, &maps.q, 64 * c, w.hk * G,
                                        (int32_t)(w.rt.row0 + w.rt.t0 + q * w.tokens), &ms.q_full);
                }
                const int box = MODE == kPacked ? kTile : min(a.block_size, kTile);       // rows of one copy
                const int boxes = kTile / box;
                const int mine = lane / kRegions, region = lane % kRegions;               // this lane's copy
                int issued = 0;
                bool ok = true;
                Ring ring;
                for (int j = 0; j < n_tiles && ok; ++j) {
                    const int64_t k0 = w.k_lo + (int64_t)j * kTile;
                    // copies that begin beyond the last key that a row sees are left out
                    const int live = MODE == kPacked ? 1 : (int)min((int64_t)boxes, (w.k_hi - k0 + box - 1) / box);
                    int32_t row = 0;
                    if (MODE != kPacked && mine < live) {
                        const int64_t key = k0 + mine * box;
                        const int32_t block = w.table[key / a.block_size];
                        if (block < 0 || block >= a.n_blocks) {
                            flag(p.status, KDA_DEV_BAD_SLOT);
                            row = (int32_t)(a.n_blocks * a.n_kv_heads * a.block_size);     // past the end: reads zeros
                        } else {
                            row = (int32_t)((block * (int64_t)a.n_kv_heads + w.hk) * a.block_size + key % a.block_size);
                        }
                    }
                    for (int kv = 0; kv < 2 && ok; ++kv) {
                        const int i = 2 * j + kv, st = (int)ring.stage;
                        if (i >= Sh::kStages && !(ok = wait_all(&ms.empty[st], ring.phase ^ 1u))) break;
                        ring.next(Sh::kStages);
                        uint8_t* dst = sm + Sh::kRing + st * Sh::kTileBytes;
                        const void* map = kv ? &maps.v : &maps.k;
                        if (lane == 0) mbar_expect_tx(&ms.full[st], (uint32_t)(live * box) * 128u * kRegions);
                        __syncwarp();
                        if (mine < live) {
                            uint8_t* to = dst + region * Sh::kRegion + mine * box * 128;
                            if (MODE == kPacked) tma_load_3d(to, map, 64 * region, w.hk, (int32_t)(w.rt.row0 + k0), &ms.full[st]);
                            else tma_load_2d(to, map, 64 * region, row, &ms.full[st]);
                        }
                        issued = i + 1;
                    }
                }
                if (!ok) {
                    // copies in flight land before the block's shared memory goes
                    mbar_wait(&ms.q_full, 0);
                    for (int i = max(0, issued - Sh::kStages); i < issued; ++i) mbar_wait(&ms.full[stage_of(i)], phase_of(i));
                }
            }
        } else {
            const int gt = tid - 32 * kGuardWarp;
            // These warps follow every load and release its stage with the MMAs, so that
            // no barrier gets two phases ahead of their waits.
            Ring ring;
            for (int i = 0; i < 2 * n_tiles; ++i) {
                const int j = i >> 1;
                const uint32_t st = ring.stage;
                if (!wait_all(&ms.full[st], ring.phase)) break;
                ring.next(Sh::kStages);
                if (!(i & 1) || j < first_edge) {
                    if (lane == 0) mbar_arrive(&ms.empty[st]);
                    continue;
                }
                const int64_t k0 = w.k_lo + (int64_t)j * kTile;
                uint8_t* v = sm + Sh::kRing + st * Sh::kTileBytes;
                const int from = (int)max((int64_t)0, min((int64_t)kTile, w.all_see - k0));   // rows that not every row sees
                const int none = (int)max((int64_t)0, min((int64_t)kTile, w.k_hi - k0));      // rows that no row sees
                for (int x = gt; x < (kTile - from) * kRegions * 8; x += 32 * kGuardWarps) {
                    const int r = from + x / (kRegions * 8), y = x % (kRegions * 8), region = y >> 3, c = y & 7;
                    uint4* at = reinterpret_cast<uint4*>(v + region * Sh::kRegion + row64_chunk_off(r, c));
                    if (r >= none) {
                        *at = make_uint4(0, 0, 0, 0);
                        continue;
                    }
                    uint4 u = *at;
                    uint32_t* e = &u.x;
                    uint32_t hit = 0;
    #pragma unroll
                    for (int k = 0; k < 4; ++k) hit |= ((e[k] & 0x7F807F80u) + 0x00800080u) & 0x80008000u;   // exponent all ones
                    if (hit) {
                        ms.poison = 1;
                        for (int k = 0; k < 8; ++k) {
                            const uint32_t b = e[k >> 1] >> (16 * (k & 1)) & 0xFFFFu;
                            if ((b & 0x7F80u) != 0x7F80u) continue;
                            int32_t* first = b & 0x7Fu ? ms.first_nan : b & 0x8000u ? ms.first_neg : ms.first_pos;
                            atomicMin(&first[region * 64 + c * 8 + k], (int32_t)(k0 + r));
                            e[k >> 1] &= k & 1 ? 0x0000FFFFu : 0xFFFF0000u;
                        }
                        *at = u;
                    }
                }
                __threadfence_block();
                fence_async_smem();
                mbar_arrive(&ms.guarded[st]);
                __syncwarp();
                if (lane == 0) mbar_arrive(&ms.empty[st]);
            }
        }
    } else {
        // ------------------------------------------------------------------ softmax
        more_registers<kSoftmaxRegs>();
        const int q = warp >> 2;
        const int r = 32 * (warp & 3) + lane;                     // row of the tile = TMEM lane
        const uint32_t lanes = (uint32_t)(32 * (warp & 3)) << 16;
        const int t = w.rt.t0 + q * w.tokens + r / G, g = r % G;
        const bool live = r < w.tokens * G && t < w.rt.n;
        // keys that this row sees, and keys that all rows of the tile see, from k_lo on
        const int64_t seen = MODE == kPrefix ? w.k_hi : min(w.k_hi, w.first + t + 1);
        const int row_sees = (int)max((int64_t)0, seen - w.k_lo);
        const int tile_sees =
            (int)max((int64_t)0, (MODE == kPrefix ? w.k_hi : min(w.k_hi, w.first + w.rt.t0 + q * w.tokens + 1)) - w.k_lo);
        // a scale of 0 becomes the least normal number, so that a hidden score of -inf stays one
        const float c = fmaxf(fabsf(a.scale) * kLog2e, 1.17549435e-38f);
        const int n = w.n_keys[q];
        float m = -CUDART_INF_F;
        uint64_t l2 = pair2(0.f);
        bool ok = true;
        for (int j = 0; j < n; ++j) {
            if (!(ok = wait_all(&ms.s_full[q], j & 1))) break;
            fence_after_sync();
            uint32_t s[kTile];
#pragma unroll
            for (int x = 0; x < kTile; x += 32) tmem_ld32(tS(q) + lanes + x, s + x);
            tmem_wait_ld();
            if ((j + 1) * kTile > tile_sees) {
                const int visible = row_sees - j * kTile;
#pragma unroll
                for (int x = 0; x < kTile; ++x) s[x] = x < visible ? s[x] : 0xFF800000u;
            }
            auto maximum = [&]() {                                 // of the tile's scores, and m
                float top[4] = {m, m, m, m};
#pragma unroll
                for (int x = 0; x < kTile; x += 8)
#pragma unroll
                    for (int y = 0; y < 4; ++y)
                        top[y] = fmaxf(fmaxf(top[y], __uint_as_float(s[x + 2 * y])), __uint_as_float(s[x + 2 * y + 1]));
                return fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3]));
            };
            // the weights of one half of the keys, for the maximum as it stands, to P; returns their sum
            auto weights = [&](int h) -> uint64_t {
                const uint64_t off2 = pair2(m == -CUDART_INF_F ? 0.f : -m * c), c2 = pair2(c);
                uint64_t sums[2] = {pair2(0.f), pair2(0.f)};
                uint32_t w2[32];
#pragma unroll
                for (int x = 0; x < 32; ++x) {
                    const float2 y = unpair2(fma2(pair2(s[64 * h + 2 * x], s[64 * h + 2 * x + 1]), c2, off2));
                    const float p0 = ex2(y.x), p1 = ex2(y.y);
                    sums[x & 1] = add2(sums[x & 1], pair2(__float_as_uint(p0), __float_as_uint(p1)));
                    w2[x] = pack_bf16(p0, p1);
                }
                tmem_st32(tS(q) + lanes + 32 * h, w2);
                return add2(sums[0], sums[1]);
            };
            if (j == 0) m = maximum();
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                uint64_t sum = weights(h);
                const float2 both = unpair2(sum);
                const bool grow = !(both.x + both.y <= kMostWeight);
                if (__any_sync(0xffffffffu, grow)) {
                    // rare: move the maximum, rescale what was summed so far, weigh again
                    if (h == 1) ok = ok && wait_all(&ms.half_done[q], j & 1);
                    fence_after_sync();
                    const float mx = grow ? maximum() : m;         // a row's result depends on no other row
                    const float f = mx > m ? ex2((m - mx) * c) : 1.f;
                    m = mx;
                    const float2 lf = unpair2(l2);
                    l2 = pair2(__float_as_uint(lf.x * f), __float_as_uint(lf.y * f));
                    if (j > 0 || h == 1) {
#pragma unroll 1
                        for (int x = 0; x < D; x += 16) {
                            uint32_t o[16];
                            tmem_ld16(tO(q) + lanes + x, o);
                            tmem_wait_ld();
#pragma unroll
                            for (int y = 0; y < 16; ++y) o[y] = __float_as_uint(__uint_as_float(o[y]) * f);
                            tmem_st16(tO(q) + lanes + x, o);
                        }
                    }
                    tmem_wait_st();
                    sum = weights(h);
                }
                tmem_wait_st();
                fence_before_sync();
                __syncwarp();
                if (lane == 0) mbar_arrive(&ms.p_ready[q][h]);
                l2 = add2(l2, sum);
            }
        }
        const float l = unpair2(l2).x + unpair2(l2).y;
        if (ok && n > 0) ok = wait_all(&ms.o_done[q], 0);
        fence_after_sync();
        if (ok) {
            const int64_t row = w.rt.row0 + t;
            const int head = w.hk * G + g;
            const int64_t at = ((int64_t)w.split * a.total_tokens + row) * a.n_heads + head;
            const float inv = l == 0.f ? 0.f : 1.f / l;
            const bool poison = MODE != kPrefix && *(volatile int32_t*)&ms.poison;
#pragma unroll
            for (int x = 0; x < D; x += 32) {
                uint32_t o[32];
                if (n > 0) {
                    tmem_ld32(tO(q) + lanes + x, o);
                    tmem_wait_ld();
                } else {
#pragma unroll
                    for (int y = 0; y < 32; ++y) o[y] = 0u;
                }
                __syncwarp();
                if (!live) {
                } else if (MODE == kPrefix) {
                    float4* out = reinterpret_cast<float4*>(p.part_o + at * D + x);
#pragma unroll
                    for (int y = 0; y < 32; y += 4)
                        out[y / 4] = make_float4(__uint_as_float(o[y]), __uint_as_float(o[y + 1]), __uint_as_float(o[y + 2]),
                                                 __uint_as_float(o[y + 3]));
                } else {
                    if (poison) {
#pragma unroll
                        for (int y = 0; y < 32; ++y) {
                            const bool pos = seen > ms.first_pos[x + y], neg = seen > ms.first_neg[x + y];
                            float add = pos ? CUDART_INF_F : neg ? -CUDART_INF_F : 0.f;
                            if (seen > ms.first_nan[x + y] || (pos && neg)) add = CUDART_NAN_F;
                            o[y] = __float_as_uint(__uint_as_float(o[y]) + add);
                        }
                    }
                    uint4* out = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(a.o) + row * a.o_stride + (int64_t)head * D + x);
#pragma unroll
                    for (int y = 0; y < 32; y += 8) {
                        uint32_t b[4];
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            b[k] = pack_bf16(__uint_as_float(o[y + 2 * k]) * inv, __uint_as_float(o[y + 2 * k + 1]) * inv);
                        out[y / 8] = make_uint4(b[0], b[1], b[2], b[3]);
                    }
                }
                __syncwarp();
            }
            if (live) {
                const float m2 = m == -CUDART_INF_F ? m : m * c;
                if (MODE == kPrefix) p.part_ml[at] = make_float2(m2, l);
                else if (a.lse) a.lse[row * a.n_heads + head] = l == 0.f ? -CUDART_INF_F : fmaf(m2, kLn2, logf(l));
            }
        }
        fence_before_sync();
    }
    __syncthreads();
    if (warp == kMmaWarp) {
        fence_after_sync();
        tmem_dealloc(ms.tslot, kTmemCols);
    }
}

// ------------------------------------------------------------------ launch

using EncodeTiledFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                   const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                   CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiledFn encode_fn() {
    static const EncodeTiledFn fn = [] {
        void* f = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &q) == cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            return reinterpret_cast<EncodeTiledFn>(f);
        return static_cast<EncodeTiledFn>(nullptr);
    }();
    return fn;
}

// bf16 tensors in boxes of 64 columns with the 128-byte swizzle.  Every copy
// starts at column 0 or 64; rows past the end read as zero.
bool make_map(CUtensorMap* m, const void* base, uint32_t rank, const cuuint64_t* dims, const cuuint64_t* strides,
              const cuuint32_t* box) {
    const EncodeTiledFn fn = encode_fn();
    const cuuint32_t one[3] = {1, 1, 1};
    return fn && fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, rank, const_cast<void*>(base), dims, strides, box, one,
                    CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                    CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// [tokens, heads, d] with a stride between tokens, boxes of box_heads x box_tokens rows.
bool token_map(CUtensorMap* m, const void* base, int64_t tokens, int heads, int d, int64_t stride, int box_heads,
               int box_tokens) {
    const cuuint64_t dims[3] = {(cuuint64_t)d, (cuuint64_t)heads, (cuuint64_t)tokens};
    const cuuint64_t strides[2] = {(cuuint64_t)d * 2, (cuuint64_t)stride * 2};
    const cuuint32_t box[3] = {64, (cuuint32_t)box_heads, (cuuint32_t)box_tokens};
    return make_map(m, base, 3, dims, strides, box);
}

bool cache_map(CUtensorMap* m, const void* base, const kda_attn_prefill_args& a) {
    const cuuint64_t dims[2] = {(cuuint64_t)a.d, (cuuint64_t)(a.n_blocks * a.n_kv_heads * a.block_size)};
    const cuuint64_t strides[1] = {(cuuint64_t)a.d * 2};
    const cuuint32_t box[2] = {64, (cuuint32_t)(a.block_size < kTile ? a.block_size : kTile)};
    return make_map(m, base, 2, dims, strides, box);
}

template <int D, int MODE>
cudaError_t launch_t(const AttnTileLaunch& p, cudaStream_t s) {
    const kda_attn_prefill_args& a = p.a;
    const int G = a.n_heads / a.n_kv_heads, tokens = kTile / G;
    Maps maps;
    bool ok = token_map(&maps.q, a.q, a.total_tokens, a.n_heads, D, a.q_stride, G, tokens);
    if (MODE == kPacked) {
        ok = ok && token_map(&maps.k, a.k, a.total_tokens, a.n_kv_heads, D, a.k_stride, 1, kTile) &&
             token_map(&maps.v, a.v, a.total_tokens, a.n_kv_heads, D, a.v_stride, 1, kTile);
    } else {
        ok = ok && cache_map(&maps.k, a.k_cache, a) && cache_map(&maps.v, a.v_cache, a);
    }
    if (!ok) return cudaErrorInvalidValue;
    int64_t blocks = (a.total_tokens / (2 * tokens) + a.n_seqs) * a.n_kv_heads;
    if (MODE == kPrefix) blocks *= p.n_split;
    if (blocks > (int64_t)INT32_MAX) return cudaErrorInvalidValue;
    const cudaError_t e = cudaFuncSetAttribute(attn_tc_kernel<D, MODE>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               (int)smem_bytes<D>());
    if (e != cudaSuccess) return e;
    note_launch();
    attn_tc_kernel<D, MODE><<<(unsigned)blocks, kThreads, smem_bytes<D>(), s>>>(p, maps);
    return cudaGetLastError();
}

template <int D>
cudaError_t launch_d(const AttnTileLaunch& p, cudaStream_t s) {
    if (p.prefix_lens) return launch_t<D, kPrefix>(p, s);
    return p.a.block_table ? launch_t<D, kPaged>(p, s) : launch_t<D, kPacked>(p, s);
}

}  // namespace

cudaError_t launch_attn_tc(const AttnTileLaunch& p, cudaStream_t s) {
    return p.a.d == 128 ? launch_d<128>(p, s) : launch_d<64>(p, s);
}

}  // namespace kda
