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
// and of K and V into a ring of stages, warp 10 makes the values at the edge of what
// the rows see safe (below), warp 11 finds the block's next item of work.
//
// Items.  The grid has a block for each item (two row tiles of one key/value head),
// but a running block takes over the items of blocks that have not started
// (clusterlaunchcontrol), so that loads, scores and products of the next item run
// while the last one's output is written, and short and long items even out.  Every
// role walks the same items with its own running barrier phases.
//
// The maximum that weights refer to is the first tile's, and is only moved when a
// row's weights of a tile add up to more than 2^10: until then no weight is larger, l
// and o are sums of the same weights whatever they refer to (their rounding is
// relative), and neither a maximum nor a rescaled O is needed.  A move is done by the
// row's own thread: a tile's scores are committed after the last product into O.
//
// Hidden values.  A product with P has 0 * v for hidden keys, which is NaN for an
// infinite or NaN v.  In the tiles that some row sees only a part of, warp 10
// therefore zeroes the values of keys that no row sees, and replaces the non-finite
// values of the others by zero and notes the first key of each column that held a
// NaN, +inf or -inf; at the end, rows that see such a key get it added.  The notes are
// those of one item.  Before they are made anew, warp 10 waits until every softmax warp
// has counted all earlier items as read.  That wait ends whatever the roles have reached:
// a softmax warp reads its notes once its products are done, and those of earlier items
// need nothing of warp 10 that is not done before.  A barrier would not do: row tile 0
// may be past the item by then (keys that only row tile 1 sees), and row tiles may be
// two items behind, so that a phase's parity says neither.
//
// The softmax warps' tensor-memory instructions are .sync.aligned: where a branch that goes
// by the lane (a row's new maximum, a store of some rows, a wait) comes before one, a
// __syncwarp() stands between.  The masks are selects, without a branch: a __syncwarp()
// behind them made the compiler spill (4 x 8192 tokens 1.45 -> 1.51 ms).
//
// Bound by the tensor pipe where sequences are long: 4 d flops per (row, key) pair.
// Measured on 4 x 8192 tokens, 32 query and 8 key/value heads, d = 128: 1.44 ms, 1530
// TFLOP/s in a loop, under the power limit (1.33 ms in its first milliseconds).  With d =
// 64 and 16/2 heads 0.50 ms, 1100 TFLOP/s: P lies in S's place, so that a row tile's next
// scores wait for its last product, and two row tiles are too few to hide that chain at
// half the arithmetic.  Items of few tiles are bound by the steps between them, and those by
// fetching instructions: straight code that is not in the 32 KB of instruction cache
// costs 6 cycles an instruction, and a jump a trip to L2.  So what is rarely executed
// is kept in loops, and what every item executes in one place: 2880 items of one or two
// tiles (180 x 256 tokens, 16 query and 2 key/value heads, d = 64) take 95 us, and took 112
// us with the weights, the rescaling and the hidden values' repair unrolled wherever needed.
#include <cuda.h>
#include <math_constants.h>

#include <climits>

#include "attn_common.cuh"
#include "tc05.cuh"

namespace kda {
namespace {
using namespace tc;

constexpr int kTile = 128;                    // rows of a tile, keys of a tile
constexpr int kMmaWarp = 8, kLoadWarp = 9, kGuardWarp = 10;   // 11: the items
constexpr int kItemReaders = 11;              // warps that read an item: all but its own
constexpr int kThreads = 384;
// Registers a thread: 168 at launch; the softmax warps hold a whole row of scores.
// 256 * 216 + 128 * 72 <= 384 * 168.
constexpr int kSoftmaxRegs = 216, kOtherRegs = 72;
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
constexpr float kMostWeight = 1024.f;         // of a row's tile, before the maximum moves
// The maximum of a row that has seen only scores of -inf, before or after the scale: the
// first score above it gives an infinite weight, which moves it.  Near the least finite
// number, so that no score lies below; times the scale it stays finite.
constexpr float kLeastMaximum = -3e38f;
constexpr uint32_t kTmemCols = 512;           // S0 0, S1 128, O0 256, O1 384

enum Mode { kPacked, kPaged, kPrefix };

template <int D> struct Shape {
    static constexpr uint32_t kRegion = kTile * 128u;            // 128 rows x 64 columns, 128-byte swizzle
    static constexpr uint32_t kTileBytes = kRegion * (D / 64);
    static constexpr int kStages = D == 128 ? 5 : 8;
    static constexpr uint32_t kQ = 0, kRing = 2 * kTileBytes, kMisc = kRing + kStages * kTileBytes;
};

// One item of work; positions and rows of cu_seqlens fit 32 bits (a table row has fewer
// than 2^31 positions).  An item whose sequence is bad has no key tiles and no rows.
struct Item {
    int32_t n_keys0, n_keys1;     // key tiles of each row tile
    int32_t n_tiles;              // the more of the two; -1: no further items
    int32_t edge;                 // from this key tile on some row sees only a part of it
    int32_t row0;                 // packed row of the first token (or member)
    int32_t t0, n;                // first token of the item, tokens of the sequence
    int32_t hk, split;
    int32_t table_row;
    int32_t first;                // token t sees the keys j <= first + t
    int32_t k_lo, k_hi;           // keys that some row of the item sees
    int32_t all_see;              // every row sees the keys below this one
    __device__ __forceinline__ int32_t n_keys(int q) const { return q ? n_keys1 : n_keys0; }
};

template <int D> struct Misc {
    uint64_t full[Shape<D>::kStages], empty[Shape<D>::kStages];
    uint64_t guarded[Shape<D>::kStages];
    uint64_t item_full[2], item_empty[2], want, next, q_full, q_free, drained;
    uint64_t s_full[2], p_ready[2], o_done[2], o_free[2];
    alignas(16) uint4 next_block;                                 // clusterlaunchcontrol's answer
    Item item[2];
    uint32_t tslot;
    uint32_t items_read[kMmaWarp];                                // items whose notes each softmax warp is done with
    uint32_t poison;                                              // the item that the notes below belong to
    int32_t first_nan[D], first_pos[D], first_neg[D];             // first key of a column that holds such a value
};

template <int D> constexpr size_t smem_bytes() { return Shape<D>::kMisc + sizeof(Misc<D>) + 1024; }
static_assert(smem_bytes<64>() <= 227 * 1024 && smem_bytes<128>() <= 227 * 1024, "a thread block's shared memory");

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
__device__ __forceinline__ void tma_load_4d(void* dst, const void* tmap, int32_t x, int32_t y, int32_t z, int32_t w, uint64_t* bar) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], [%6];" ::
            "r"(smem_u32(dst)),
        "l"(reinterpret_cast<uint64_t>(tmap)), "r"(x), "r"(y), "r"(z), "r"(w), "r"(smem_u32(bar))
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
// A bounded wait (about a second) in few instructions: there are dozens, and outside a
// loop what one costs is mostly fetching it.
constexpr uint32_t kWaitCycles = 2000000000u;
__device__ __forceinline__ bool wait(uint64_t* bar, uint32_t parity) {
    if (mbar_test(bar, parity)) return true;
    const uint32_t t0 = (uint32_t)clock();
    while (!mbar_test(bar, parity))
        if ((uint32_t)clock() - t0 > kWaitCycles) return false;
    return true;
}
__device__ __forceinline__ uint32_t load_acquire(const uint32_t* p) {
    uint32_t x;
    asm volatile("ld.acquire.cta.shared::cta.u32 %0, [%1];" : "=r"(x) : "r"(smem_u32(p)) : "memory");
    return x;
}
__device__ __forceinline__ void store_release(uint32_t* p, uint32_t x) {
    asm volatile("st.release.cta.shared::cta.u32 [%0], %1;" ::"r"(smem_u32(p)), "r"(x) : "memory");
}
// Until a count has reached `least`, as long as wait().
__device__ __forceinline__ bool wait_count(const uint32_t* p, uint32_t least) {
    const uint32_t t0 = (uint32_t)clock();
    while (load_acquire(p) < least)
        if ((uint32_t)clock() - t0 > kWaitCycles) return false;
    return true;
}
__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// Asks for the work of a block that has not started; the answer arrives at `to` with 16 bytes on `bar`.
__device__ __forceinline__ void ask_next_block(uint4* to, uint64_t* bar) {
    asm volatile("clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes.b128 [%0], [%1];" ::"r"(smem_u32(to)),
                 "r"(smem_u32(bar))
                 : "memory");
}
// Whether the answer is a block, and its index.
__device__ __forceinline__ bool next_block(const uint4* from, uint32_t& x) {
    uint32_t taken;
    asm volatile(
        "{\n\t.reg .b128 h;\n\t.reg .pred p;\n\t"
        "ld.shared.b128 h, [%2];\n\t"
        "clusterlaunchcontrol.query_cancel.is_canceled.pred.b128 p, h;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t"
        "mov.u32 %1, 0;\n\t"
        "@p clusterlaunchcontrol.query_cancel.get_first_ctaid::x.b32.b128 %1, h;\n\t}"
        : "=r"(taken), "=r"(x)
        : "r"(smem_u32(from))
        : "memory");
    return taken;
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
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
template <int N> __device__ __forceinline__ void more_registers() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N)); }
template <int N> __device__ __forceinline__ void fewer_registers() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N)); }

// Writes 128 bytes at `byte` of each lane's row (none where row is NULL).  Four lanes trade
// their rows' 32-byte pieces, so that together they write one row at a time: a store
// instruction takes a cycle a line.  Lane x of the four puts piece x ^ y in place y; what
// comes from lane x ^ y is that row's piece x.
__device__ __forceinline__ void write_traded(uint32_t (&b)[4][8], char* row, int byte, int lane) {
#pragma unroll
    for (int bit = 1; bit < 4; bit <<= 1) {
        const bool up = lane & bit;
#pragma unroll
        for (int y = 0; y < 4; ++y)
#pragma unroll
            for (int k = 0; k < 8; ++k)
                if (!(y & bit)) {
                    const uint32_t lo = b[y][k], hi = b[y | bit][k];
                    b[y][k] = up ? hi : lo;
                    b[y | bit][k] = up ? lo : hi;
                }
    }
#pragma unroll
    for (int y = 0; y < 4; ++y) {
#pragma unroll
        for (int k = 0; k < 8; ++k)
            if (y > 0) b[y][k] = __shfl_xor_sync(0xffffffffu, b[y][k], y);
        char* to = reinterpret_cast<char*>(__shfl_xor_sync(0xffffffffu, reinterpret_cast<uint64_t>(row), y));
        if (to)
            asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(to + byte + 32 * (lane & 3)), "r"(b[y][0]),
                         "r"(b[y][1]), "r"(b[y][2]), "r"(b[y][3]), "r"(b[y][4]), "r"(b[y][5]), "r"(b[y][6]), "r"(b[y][7])
                         : "memory");
    }
}

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

// ------------------------------------------------------------------ items

// The finder's place: 32 sequences, one a lane, and the item tiles up to and with each.
struct Place {
    int32_t s0 = -32;             // the first of them
    int32_t s = 0;                // the lane's sequence
    int32_t lo = 0, hi = 0;       // and its rows
    int32_t before = 0, upto = 0; // tiles before the 32, and with the lane's own
};

// Fills `it` for grid index `block`; false when that block has nothing to do.  One
// warp; later indexes mostly lie further on, so the search goes on where the last one
// ended, mostly without a load.  Long items come first, so that the blocks end together:
// the tiles of one sequence last first, and up to 32 sequences by their positions (8
// prompts of 1 to 1024 tokens behind 256 to 4096: 116 us, 127 us unsorted; among more, the order
// makes no difference that was worth sorting).  Sequences are not interleaved: their keys
// stay in L2.  SPLIT: the keys of a tile are cut into n_split blocks, an item each.
template <int MODE, bool SPLIT>
__device__ bool find_item(const AttnTileLaunch& p, uint32_t block, Place& place, Item& it) {
    const kda_attn_prefill_args& a = p.a;
    const int lane = threadIdx.x & 31;
    const int tokens = kTile / (a.n_heads / a.n_kv_heads);
    uint32_t rest = block / (uint32_t)a.n_kv_heads;
    it.hk = (int32_t)(block - rest * a.n_kv_heads);
    it.split = 0;
    if (SPLIT) {
        const uint32_t x = rest / (uint32_t)p.n_split;
        it.split = (int32_t)(rest - x * p.n_split);
        rest = x;
    }
    const int32_t idx = (int32_t)rest;
    if (idx < place.before) place = Place{};
    uint32_t here;
    while (!(here = __ballot_sync(0xffffffffu, idx < place.upto))) {
        place.before = __shfl_sync(0xffffffffu, place.upto, 31);
        if (place.s0 + 32 >= a.n_seqs) {                                   // past the last tile, as later blocks will be
            place.upto = place.before;
            return false;
        }
        place.s0 += 32;
        place.s = place.s0 + lane;
        place.lo = place.hi = 0;
        if (place.s < a.n_seqs) {
            place.lo = a.cu_seqlens[place.s];
            place.hi = a.cu_seqlens[place.s + 1];
            if (place.lo < 0 || place.hi < place.lo || place.hi > a.total_tokens) place.hi = place.lo;
        }
        if (MODE != kPrefix && a.n_seqs > 1 && a.n_seqs <= 32) {
            const int32_t K = MODE == kPacked ? place.hi - place.lo : lane < a.n_seqs ? max(0, a.kv_lens[lane]) : 0;
            uint32_t key = (uint32_t)K / kTile * 32 + lane;                // a bitonic sort, the greatest first
#pragma unroll 1
            for (int k = 2; k <= 32; k <<= 1)
#pragma unroll 1
                for (int j = k >> 1; j > 0; j >>= 1) {
                    const uint32_t other = __shfl_xor_sync(0xffffffffu, key, j);
                    key = ((lane & j) == 0) == ((lane & k) == 0) ? max(key, other) : min(key, other);
                }
            place.s = key & 31;
            place.lo = __shfl_sync(0xffffffffu, place.lo, place.s);
            place.hi = __shfl_sync(0xffffffffu, place.hi, place.s);
        }
        int32_t upto = (int32_t)(((uint32_t)(place.hi - place.lo) + 2 * tokens - 1) / (uint32_t)(2 * tokens));
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const int32_t y = __shfl_up_sync(0xffffffffu, upto, off);
            if (lane >= off) upto += y;
        }
        place.upto = place.before + upto;
    }
    const int src = __ffs(here) - 1, seq = __shfl_sync(0xffffffffu, place.s, src);
    it.row0 = __shfl_sync(0xffffffffu, place.lo, src);
    it.n = __shfl_sync(0xffffffffu, place.hi, src) - it.row0;
    it.t0 = (__shfl_sync(0xffffffffu, place.upto, src) - 1 - idx) * 2 * tokens;
    it.table_row = MODE == kPrefix ? it.row0 : seq;
    const int64_t cap = (int64_t)a.table_stride * a.block_size;
    int32_t K;
    if (MODE == kPacked) {
        K = it.n;
    } else if (MODE == kPaged) {
        K = a.kv_lens[seq];
        if (K < 0 || K > cap) {
            if (lane == 0) flag(p.status, KDA_DEV_BAD_SEQLENS);
            return false;
        }
    } else {
        K = p.prefix_lens[seq];
        if (K < 0 || K > cap || (K & (a.block_size - 1))) K = 0;           // flagged by the decode plan
    }
    it.first = MODE == kPacked ? 0 : MODE == kPaged ? K - it.n : K;
    const int left = it.n - it.t0;                                         // tokens from the first one on
    auto tiles = [](int32_t keys) { return (int32_t)(((uint32_t)keys + kTile - 1) / kTile); };
    if (MODE == kPrefix) {
        const int64_t per = (int64_t)prefix_block_tiles(K, kTile, p.n_split, p.split_cost) * kTile;
        it.k_lo = (int32_t)min((int64_t)K, it.split * per);
        it.k_hi = it.all_see = (int32_t)min((int64_t)K, it.k_lo + per);
        it.n_keys0 = it.n_keys1 = tiles(it.k_hi - it.k_lo);
    } else {
        it.k_lo = 0;
        // (first + t0 + tokens <= K + 2 kTile, which may pass 2^31)
        auto seen = [&](int tokens) { return max(0, (int32_t)min((int64_t)K, (int64_t)it.first + it.t0 + tokens)); };
        it.all_see = seen(1);
        it.k_hi = seen(min(left, 2 * tokens));
        it.n_keys0 = tiles(seen(min(left, tokens)));
        it.n_keys1 = tiles(it.k_hi);
    }
    if (left <= tokens) it.n_keys1 = 0;
    if (MODE != kPrefix && SPLIT) {
        const int per = (int)((uint32_t)(max(it.n_keys0, it.n_keys1) + p.n_split - 1) / (uint32_t)p.n_split), from = it.split * per;
        it.k_lo = min(it.k_hi, from * kTile);
        it.k_hi = (int32_t)min((int64_t)it.k_hi, it.k_lo + (int64_t)per * kTile);
        it.n_keys0 = max(0, min(per, it.n_keys0 - from));
        it.n_keys1 = max(0, min(per, it.n_keys1 - from));
    }
    it.n_tiles = max(it.n_keys0, it.n_keys1);
    it.edge = max(0, it.all_see - it.k_lo) / kTile;
    return true;
}

// ------------------------------------------------------------------ kernel

template <int D, int MODE, bool SPLIT>
__global__ void __launch_bounds__(kThreads, 1)
attn_tc_kernel(const __grid_constant__ AttnTileLaunch p, const __grid_constant__ Maps maps) {
    using Sh = Shape<D>;
    constexpr int kRegions = D / 64;
    // Tiles of keys and values: 1024 bytes hold 8 rows x 64 columns.  Packed ones come in one
    // copy for each 64 columns; a page, in one copy of all columns, 8 rows at a time (half as
    // many copies for d = 128: with pages of 16 keys they are what bounds the kernel).
    constexpr uint32_t kColumnStep = MODE == kPacked ? Sh::kRegion : 1024u;      // to the next 64 columns
    constexpr uint32_t kRowStep = MODE == kPacked ? 1024u : 1024u * kRegions;    // to the next 8 rows
    extern __shared__ uint8_t smem_raw[];
    uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    Misc<D>& ms = *reinterpret_cast<Misc<D>*>(sm + Sh::kMisc);
    const uint32_t s_base = smem_u32(sm);
    const kda_attn_prefill_args& a = p.a;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int G = a.n_heads / a.n_kv_heads, tokens = kTile / G;
    griddep_wait();
    griddep_launch();

    if (warp == kMmaWarp) tmem_alloc(&ms.tslot, kTmemCols);
    if (tid == 0) {
        for (int i = 0; i < Sh::kStages; ++i) {
            mbar_init(&ms.full[i], 1);
            mbar_init(&ms.empty[i], 2);               // the MMAs and the guard
            mbar_init(&ms.guarded[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&ms.item_full[i], 1);
            mbar_init(&ms.item_empty[i], kItemReaders);
            mbar_init(&ms.s_full[i], 1);
            mbar_init(&ms.p_ready[i], 128);
            mbar_init(&ms.o_done[i], 1);
            mbar_init(&ms.o_free[i], 4);
        }
        mbar_init(&ms.want, 1);
        mbar_init(&ms.next, 1);
        mbar_init(&ms.q_full, 1);
        mbar_init(&ms.q_free, 1);
        mbar_init(&ms.drained, 1);
        for (int w = 0; w < kMmaWarp; ++w) ms.items_read[w] = 0;
        ms.poison = ~0u;
        fence_mbar_init();
    }
    fence_before_sync();
    __syncthreads();
    fence_after_sync();
    constexpr uint32_t tbase = 0;                 // all of tensor memory is this block's
    auto tS = [](int q) { return tbase + 128u * q; };
    auto tO = [](int q) { return tbase + 256u + 128u * q; };
    // A bounded wait of a whole warp, whose lanes then agree.  Once one runs out, the
    // roles that depend on it run out of theirs.  Between a tile's steps, where the
    // vote's time counts, lanes wait with `pass`, each for itself: one that ran out goes
    // on without waiting, to the vote at the item's end.
    bool late = false;                            // a wait ran out: flagged at the end
    auto wait_all = [&](uint64_t* bar, uint32_t parity) -> bool {
        const bool ok = __all_sync(0xffffffffu, wait(bar, parity));
        late |= !ok;
        return ok;
    };
    auto pass = [&](bool& ok, uint64_t* bar, uint32_t parity) {
        if (ok && !wait(bar, parity)) {
            late = true;
            ok = false;
        }
    };
    // The i-th item of this block, copied out of its slot; false at the end.
    auto get_item = [&](uint32_t i, Item& it) -> bool {
        if (!wait_all(&ms.item_full[i & 1], i >> 1 & 1)) return false;
        it = ms.item[i & 1];
        __syncwarp();
        if (lane == 0) mbar_arrive(&ms.item_empty[i & 1]);
        return it.n_tiles >= 0;
    };

    // the register split is made inside the branches: after a merge of the two the
    // compiler would hold everything to the smaller share
    if (warp >= kMmaWarp) {
        fewer_registers<kOtherRegs>();
        if (warp == kMmaWarp) {
            // -------------------------------------------------------------- MMAs
            const uint32_t leader = elect_one();
            const uint32_t id_s = idesc_bf16(kTile, kTile, false, false) | (a.scale < 0.f ? 1u << 13 : 0u);
            const uint32_t id_o = idesc_bf16(kTile, D, false, true);
            const uint64_t d_q = sdesc(0, 16, 1024), d_k = sdesc(0, 16, kRowStep), d_v = sdesc(0, kColumnStep, kRowStep);
            auto at = [](uint64_t desc, uint32_t byte) { return desc + (uint64_t)(byte >> 4); };
            auto scores = [&](int q, uint32_t stage) {
                const uint64_t qd = at(d_q, s_base + Sh::kQ + q * Sh::kTileBytes);
                const uint64_t kd = at(d_k, s_base + Sh::kRing + stage * Sh::kTileBytes);
#pragma unroll
                for (int ks = 0; ks < D / 16; ++ks)
                    mma_ss(leader, tS(q), at(qd, (ks >> 2) * Sh::kRegion + (ks & 3) * 32),
                           at(kd, (ks >> 2) * kColumnStep + (ks & 3) * 32), id_s, ks > 0);
                commit(leader, &ms.s_full[q]);
            };
            auto values = [&](int q, uint32_t stage, bool first) {
                const uint64_t vd = at(d_v, s_base + Sh::kRing + stage * Sh::kTileBytes);
#pragma unroll
                for (int ks = 0; ks < kTile / 16; ++ks)
                    mma_ts(leader, tO(q), tS(q) + 8 * ks, at(vd, 2 * ks * kRowStep), id_o, !first || ks > 0);
            };
            uint32_t guard_phase = 0;                             // a bit for each stage
            uint32_t p_phase = 0, o_items = 0;                    // a bit for each row tile
            Ring r;
            bool ok = true;
            Item it;
            for (uint32_t i = 0; __all_sync(0xffffffffu, ok) && get_item(i, it); ++i) {
                const int n_tiles = it.n_tiles;
                pass(ok, &ms.q_full, i & 1);
                if (n_tiles == 0) {
                    commit(leader, &ms.q_free);
                    continue;
                }
                pass(ok, &ms.full[r.stage], r.phase);
                fence_after_sync();
#pragma unroll 1
                for (int q = 0; q < 2; ++q)
                    if (it.n_keys(q) > 0) scores(q, r.stage);
                commit(leader, &ms.empty[r.stage]);
                if (n_tiles == 1) commit(leader, &ms.q_free);
                r.next(Sh::kStages);
                auto v_ready = [&](int j) {
                    pass(ok, &ms.full[r.stage], r.phase);
                    if (j >= it.edge) {
                        pass(ok, &ms.guarded[r.stage], guard_phase >> r.stage & 1);
                        guard_phase ^= 1u << r.stage;
                    }
                };
                for (int j = 0; j < n_tiles; ++j) {
                    v_ready(j);
                    const uint32_t vs = r.stage;
                    r.next(Sh::kStages);
                    const bool more = j + 1 < n_tiles;
                    if (more) pass(ok, &ms.full[r.stage], r.phase);
#pragma unroll
                    for (int q = 0; q < 2; ++q) {
                        const int n_keys = it.n_keys(q);
                        if (j < n_keys) {
                            if (j == 0) {
                                pass(ok, &ms.o_free[q], (o_items >> q & 1) ^ 1);
                                o_items ^= 1u << q;
                            }
                            pass(ok, &ms.p_ready[q], p_phase >> q & 1);
                            p_phase ^= 1u << q;
                            fence_after_sync();
                            values(q, vs, j == 0);
                            if (j + 1 == n_keys) commit(leader, &ms.o_done[q]);
                        }
                        if (q == 1) commit(leader, &ms.empty[vs]);
                        if (j + 1 < n_keys) scores(q, r.stage);
                    }
                    if (!more) break;
                    commit(leader, &ms.empty[r.stage]);
                    if (j + 2 == n_tiles) commit(leader, &ms.q_free);   // after the item's last scores
                    r.next(Sh::kStages);
                }
            }
            // the MMAs in flight finish before shared and tensor memory go
            commit(leader, &ms.drained);
            wait(&ms.drained, 0);
        } else if (warp == kLoadWarp) {
            // -------------------------------------------------------------- copies
            const int box = MODE == kPacked ? kTile : min(a.block_size, kTile);           // rows of one copy
            const int boxes = kTile / box, page_shift = MODE == kPacked ? 0 : __ffs(a.block_size) - 1;
            // this lane's copy: of its columns, or of a page
            const int mine = MODE == kPacked ? lane / kRegions : lane, region = MODE == kPacked ? lane % kRegions : 0;
            uint32_t q_loads = 0, issued = 0;
            Ring ring;
            bool ok = true;
            Item it;
            for (uint32_t i = 0; ok && get_item(i, it); ++i) {
                const int n_tiles = it.n_tiles;
                if (i > 0 && !(ok = wait_all(&ms.q_free, (i - 1) & 1))) break;
                if (lane == 0) {
                    const int tiles = it.n_keys1 > 0 ? 2 : 1;
                    mbar_expect_tx(&ms.q_full, (uint32_t)tiles * kRegions * (uint32_t)(tokens * G) * 128u);
                    for (int q = 0; q < tiles; ++q)
                        for (int c = 0; c < kRegions; ++c)
                            tma_load_3d(sm + Sh::kQ + q * Sh::kTileBytes + c * Sh::kRegion, &maps.q, 64 * c, it.hk * G,
                                        it.row0 + it.t0 + q * tokens, &ms.q_full);
                }
                q_loads = i + 1;
                const int32_t* table = MODE == kPacked ? nullptr : a.block_table + (int64_t)it.table_row * a.table_stride;
                // copies that begin beyond the last key that a row sees are left out
                auto copies = [&](int32_t k0) { return MODE == kPacked ? 1 : max(0, min(boxes, (it.k_hi - k0 + box - 1) / box)); };
                // the table's entry of this lane's page, read a tile ahead
                auto look_up = [&](int32_t k0) { return MODE != kPacked && mine < copies(k0) ? table[(k0 + mine * box) >> page_shift] : 0; };
                int32_t block = n_tiles > 0 ? look_up(it.k_lo) : 0;
                for (int j = 0; j < n_tiles && ok; ++j) {
                    const int32_t k0 = it.k_lo + j * kTile;
                    const int live = copies(k0);
                    int32_t rows8 = 0;                            // the page's place, in units of 8 rows
                    if (MODE != kPacked && mine < live) {
                        if (block < 0 || block >= a.n_blocks) {
                            flag(p.status, KDA_DEV_BAD_SLOT);
                            rows8 = (int32_t)(a.n_blocks * a.n_kv_heads * (a.block_size >> 3));     // past the end: reads zeros
                        } else {
                            rows8 = (int32_t)((block * (int64_t)a.n_kv_heads + it.hk) * (a.block_size >> 3) +
                                              ((k0 + mine * box & (a.block_size - 1)) >> 3));
                        }
                    }
                    if (j + 1 < n_tiles) block = look_up(k0 + kTile);
#pragma unroll 1
                    for (int kv = 0; kv < 2; ++kv) {
                        const uint32_t st = ring.stage;
                        if (!(ok = wait_all(&ms.empty[st], ring.phase ^ 1u))) break;
                        ring.next(Sh::kStages);
                        uint8_t* dst = sm + Sh::kRing + st * Sh::kTileBytes;
                        const void* map = kv ? &maps.v : &maps.k;
                        if (lane == 0) mbar_expect_tx(&ms.full[st], (uint32_t)(live * box) * 128u * kRegions);
                        __syncwarp();
                        if (mine < live) {
                            if (MODE == kPacked) tma_load_3d(dst + region * Sh::kRegion, map, 64 * region, it.hk, it.row0 + k0, &ms.full[st]);
                            else tma_load_4d(dst + mine * box * 2 * D, map, 0, 0, 0, rows8, &ms.full[st]);
                        }
                        ++issued;
                    }
                }
                if (lane == 0) mbar_arrive(&ms.want);             // time to claim another item
            }
            // copies in flight land before the block's shared memory goes: the last of
            // Q, and the last of every stage
            if (q_loads > 0) wait(&ms.q_full, (q_loads - 1) & 1);
            for (uint32_t i = issued < Sh::kStages ? 0 : issued - Sh::kStages; i < issued; ++i)
                wait(&ms.full[i % Sh::kStages], i / Sh::kStages & 1);
        } else if (warp == kGuardWarp) {
            // -------------------------------------------------------------- hidden values
            // This warp follows every load and releases its stage with the MMAs, so that
            // no barrier gets two phases ahead of its waits.
            Ring ring;
            bool ok = true;
            Item it;
            for (uint32_t i = 0; ok && get_item(i, it); ++i) {
                const int n_tiles = it.n_tiles, first_edge = it.edge;
                bool noted = false;
                for (int x = 0; x < 2 * n_tiles; ++x) {
                    const int j = x >> 1;
                    const uint32_t st = ring.stage;
                    if (!(ok = wait_all(&ms.full[st], ring.phase))) break;
                    ring.next(Sh::kStages);
                    if ((x & 1) && j >= first_edge) {
                        const int32_t k0 = it.k_lo + j * kTile;
                        uint8_t* v = sm + Sh::kRing + st * Sh::kTileBytes;
                        const int from = max(0, min(kTile, it.all_see - k0));             // keys that not every row sees
                        const int none = max(0, min(kTile, it.k_hi - k0));                // keys that no row sees
                        const int pieces = (kTile - from) * kRegions * 8;                 // of 16 bytes
                        auto key_of = [&](int y) { return from + y / (kRegions * 8); };
                        auto piece = [&](int y) {
                            const int z = y % (kRegions * 8);
                            const int key = key_of(y);
                            return reinterpret_cast<uint4*>(v + (z >> 3) * kColumnStep + (key >> 3) * kRowStep + row64_chunk_off(key & 7, z & 7));
                        };
                        bool hit = false;
#pragma unroll 4
                        for (int y = lane; y < pieces; y += 32) {
                            uint4* at = piece(y);
                            if (key_of(y) >= none) {
                                *at = make_uint4(0, 0, 0, 0);
                                continue;
                            }
                            const uint4 u = *at;
                            auto odd = [](uint32_t e) { return ((e & 0x7F807F80u) + 0x00800080u) & 0x80008000u; };
                            hit |= (odd(u.x) | odd(u.y) | odd(u.z) | odd(u.w)) != 0;      // an exponent of all ones
                        }
                        if (__any_sync(0xffffffffu, hit)) {
                            if (!noted) {
                                // the notes may still be read for earlier items
                                ok = __all_sync(0xffffffffu, lane >= kMmaWarp || wait_count(&ms.items_read[lane], i));
                                late |= !ok;
                                if (!ok) break;
                                for (int d = lane; d < D; d += 32) ms.first_nan[d] = ms.first_pos[d] = ms.first_neg[d] = INT_MAX;
                                __syncwarp();
                                // the item's number last: row tile 0 reads it without waiting for key tiles
                                // that it does not see, and must not take an earlier item's notes for these
                                if (lane == 0) store_release(&ms.poison, i);
                                noted = true;
                                __syncwarp();
                            }
                            for (int y = lane; y < pieces && key_of(y) < none; y += 32) {
                                uint16_t* e = reinterpret_cast<uint16_t*>(piece(y));
                                for (int k = 0; k < 8; ++k) {
                                    const uint32_t b = e[k];
                                    if ((b & 0x7F80u) != 0x7F80u) continue;
                                    int32_t* first = b & 0x7Fu ? ms.first_nan : b & 0x8000u ? ms.first_neg : ms.first_pos;
                                    atomicMin(&first[y % (kRegions * 8) * 8 + k], k0 + key_of(y));
                                    e[k] = 0;
                                }
                            }
                        }
                        __threadfence_block();
                        fence_async_smem();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(&ms.guarded[st]);
                    }
                    if (lane == 0) mbar_arrive(&ms.empty[st]);
                }
            }
        } else {
            // -------------------------------------------------------------- items
            // The next item is claimed when the last one's copies are under way, not before:
            // what a block claims early, a block that gets free first cannot have.
            Place place;
            uint32_t block = blockIdx.x;
            uint32_t i = 0;
            bool ok = true;
            for (uint32_t asked = 0;; ++asked) {
                Item it;
                if (find_item<MODE, SPLIT>(p, block, place, it)) {
                    if (!(ok = wait_all(&ms.item_empty[i & 1], (i >> 1 & 1) ^ 1))) break;
                    if (lane == 0) {
                        ms.item[i & 1] = it;
                        mbar_arrive(&ms.item_full[i & 1]);
                    }
                    if (!(ok = wait_all(&ms.want, i & 1))) break;
                    ++i;
                }
                // a shared prefix's blocks do not claim: the kernel that starts beside this one
                // waits for every block to have started
                if (MODE == kPrefix) break;
                if (lane == 0) {
                    mbar_expect_tx(&ms.next, 16);
                    ask_next_block(&ms.next_block, &ms.next);
                }
                __syncwarp();
                if (!(ok = wait_all(&ms.next, asked & 1))) break;
                const bool any = next_block(&ms.next_block, block);
                fence_async_smem();
                __syncwarp();
                if (!any) break;
            }
            if (ok && wait_all(&ms.item_empty[i & 1], (i >> 1 & 1) ^ 1) && lane == 0) {
                ms.item[i & 1].n_tiles = -1;
                mbar_arrive(&ms.item_full[i & 1]);
            }
        }
    } else {
        // ------------------------------------------------------------------ softmax
        more_registers<kSoftmaxRegs>();
        if (MODE != kPrefix && blockIdx.x == 0)
            for (int32_t s = tid; s < a.n_seqs; s += 32 * kMmaWarp) {
                const int64_t lo = a.cu_seqlens[s], hi = a.cu_seqlens[s + 1];
                if (lo < 0 || hi < lo || hi > a.total_tokens) flag(p.status, KDA_DEV_BAD_SEQLENS);
            }
        const int q = warp >> 2;
        const int r = 32 * (warp & 3) + lane;                     // row of the tile = TMEM lane
        const int r_token = r / G, g = r % G;
        const uint32_t lanes = (uint32_t)(32 * (warp & 3)) << 16;
        // a scale of 0 becomes the least normal number, so that a hidden score of -inf stays one
        const float c = fmaxf(fabsf(a.scale) * kLog2e, 1.17549435e-38f), least = kLeastMaximum / fmaxf(c, 1.f);
        // Rows that begin on 32 bytes are traded and written in whole sectors, others in 16-byte
        // pieces (720 x 64 tokens, 32/8 heads, d = 128: 200 us, and 259 us).
        const bool wide = !SPLIT && ((reinterpret_cast<uintptr_t>(a.o) | (uintptr_t)(a.o_stride * 2)) & 31u) == 0;
        uint32_t phase = 0, o_phase = 0;                          // of the tiles, of the items with tiles
        bool ok = true;
        Item it;
        for (uint32_t i = 0; __all_sync(0xffffffffu, ok) && get_item(i, it); ++i) {
            const int t = it.t0 + q * tokens + r_token;
            const bool live = r < tokens * G && t < it.n;
            // keys that this row sees, and keys that all rows of the warp see for sure.  Rows
            // past the end see none: what their scores hold is never looked at.
            const int seen = !live ? 0 : MODE == kPrefix ? it.k_hi : min(it.k_hi, it.first + t + 1);
            const int row_sees = max(0, seen - it.k_lo);
            int tile_sees = max(0, (MODE == kPrefix ? it.k_hi : min(it.k_hi, it.first + it.t0 + q * tokens + 1)) - it.k_lo);
            if (__any_sync(0xffffffffu, !live)) tile_sees = 0;
            const int n = it.n_keys(q);
            float m = least;
            uint64_t l2 = pair2(0.f);
            for (int j = 0; j < n; ++j) {
                pass(ok, &ms.s_full[q], phase);
                __syncwarp();
                phase ^= 1;
                fence_after_sync();
                uint32_t s[kTile];
#pragma unroll
                for (int x = 0; x < kTile; x += 32) tmem_ld32(tS(q) + lanes + x, s + x);
                tmem_wait_ld();
                if ((j + 1) * kTile > tile_sees) {
                    const int visible = row_sees - j * kTile;
#pragma unroll
                    for (int y = 0; y < kTile; y += 32) {
                        const uint32_t keep = visible >= y + 32 ? 0xFFFFFFFFu : visible <= y ? 0u : (1u << (visible - y)) - 1u;
#pragma unroll
                        for (int x = 0; x < 32; ++x) s[y + x] = keep & (1u << x) ? s[y + x] : 0xFF800000u;
                    }
                }
                auto maximum = [&]() {                             // of the tile's scores, and m
                    float top[4] = {m, m, m, m};
#pragma unroll
                    for (int x = 0; x < kTile; x += 8)
#pragma unroll
                        for (int y = 0; y < 4; ++y)
                            top[y] = fmaxf(fmaxf(top[y], __uint_as_float(s[x + 2 * y])), __uint_as_float(s[x + 2 * y + 1]));
                    return fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3]));
                };
                // the weights for the maximum as it stands, to P; returns their sum
                auto weights = [&]() -> uint64_t {
                    const uint64_t off2 = pair2(-m * c), c2 = pair2(c);
                    uint64_t sums[2] = {pair2(0.f), pair2(0.f)};
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        uint32_t w2[32];
#pragma unroll
                        for (int x = 0; x < 32; ++x) {
                            const float2 y = unpair2(fma2(pair2(s[64 * h + 2 * x], s[64 * h + 2 * x + 1]), c2, off2));
                            const float p0 = ex2(y.x), p1 = ex2(y.y);
                            sums[x & 1] = add2(sums[x & 1], pair2(__float_as_uint(p0), __float_as_uint(p1)));
                            w2[x] = pack_bf16(p0, p1);
                        }
                        tmem_st32(tS(q) + lanes + 32 * h, w2);
                    }
                    return add2(sums[0], sums[1]);
                };
                uint64_t sum;
                bool move = j == 0, grow = true;                   // the first tile's maximum, and the rows that want one
                for (;;) {
                    if (move) {
                        const float mx = grow ? maximum() : m;     // a row's result depends on no other row
                        const float f = mx > m ? ex2((m - mx) * c) : 1.f;
                        m = mx;
                        const float2 lf = unpair2(l2);
                        l2 = pair2(__float_as_uint(lf.x * f), __float_as_uint(lf.y * f));
                        __syncwarp();
                        // rare: rescale what was summed so far
#pragma unroll 1
                        for (int x = j == 0 ? D : 0; x < D; x += 16) {
                            uint32_t o[16];
                            tmem_ld16(tO(q) + lanes + x, o);
                            tmem_wait_ld();
#pragma unroll
                            for (int y = 0; y < 16; ++y) o[y] = __float_as_uint(__uint_as_float(o[y]) * f);
                            tmem_st16(tO(q) + lanes + x, o);
                        }
                    }
                    sum = weights();
                    if (move) break;
                    const float2 both = unpair2(sum);
                    grow = !(both.x + both.y <= kMostWeight);
                    move = __any_sync(0xffffffffu, grow);
                    if (!move) break;
                    tmem_wait_st();
                }
                l2 = add2(l2, sum);
                tmem_wait_st();
                fence_before_sync();
                mbar_arrive(&ms.p_ready[q]);
            }
            const float l = unpair2(l2).x + unpair2(l2).y;
            const float inv = l == 0.f ? 0.f : 1.f / l;
            const int64_t row = (int64_t)it.row0 + t;
            const int head = it.hk * G + g;
            const int64_t at = ((int64_t)it.split * a.total_tokens + row) * a.n_heads + head;
            if (n > 0) {
                pass(ok, &ms.o_done[q], o_phase);
                __syncwarp();
                o_phase ^= 1;
                fence_after_sync();
                if (MODE != kPrefix && __shfl_sync(0xffffffffu, load_acquire(&ms.poison), 0) == i) {
#pragma unroll 1
                    for (int x = 0; x < D; x += 16) {
                        uint32_t y[16];
                        tmem_ld16(tO(q) + lanes + x, y);
                        tmem_wait_ld();
#pragma unroll
                        for (int k = 0; k < 16; ++k) {
                            const bool pos = seen > ms.first_pos[x + k], neg = seen > ms.first_neg[x + k];
                            float add = pos ? CUDART_INF_F : neg ? -CUDART_INF_F : 0.f;
                            if (seen > ms.first_nan[x + k] || (pos && neg)) add = CUDART_NAN_F;
                            y[k] = __float_as_uint(__uint_as_float(y[k]) + add);
                        }
                        __syncwarp();
                        tmem_st16(tO(q) + lanes + x, y);
                    }
                    tmem_wait_st();
                }
            } else {                                               // no keys: zeros
                const uint32_t zero[16] = {};
                __syncwarp();
#pragma unroll 1
                for (int x = 0; x < D; x += 16) tmem_st16(tO(q) + lanes + x, zero);
                tmem_wait_st();
            }
            __syncwarp();
            if (lane == 0) store_release(&ms.items_read[warp], i + 1);
            const float m2 = l == 0.f ? -CUDART_INF_F : m * c;
            char* out = SPLIT ? reinterpret_cast<char*>(p.part_o + at * D)
                              : reinterpret_cast<char*>(static_cast<__nv_bfloat16*>(a.o) + row * a.o_stride + (int64_t)head * D);
            if (!live) out = nullptr;
            const uint64_t inv2 = pair2(inv);
#pragma unroll 1
            for (int x = 0; x < D; x += 64) {
                uint32_t o[64];
                __syncwarp();
                tmem_ld32(tO(q) + lanes + x, o);
                tmem_ld32(tO(q) + lanes + x + 32, o + 32);
                tmem_wait_ld();
                if (x + 64 == D && n > 0) {
                    fence_before_sync();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&ms.o_free[q]);
                }
                uint32_t b[4][8];
                if constexpr (SPLIT) {
#pragma unroll
                    for (int half = 0; half < 2; ++half) {
#pragma unroll
                        for (int k = 0; k < 32; ++k) b[k >> 3][k & 7] = o[32 * half + k];
                        write_traded(b, out, 4 * x + 128 * half, lane);
                    }
                } else {
#pragma unroll
                    for (int k = 0; k < 32; ++k) {
                        const float2 y = unpair2(mul2(pair2(o[2 * k], o[2 * k + 1]), inv2));
                        b[k >> 3][k & 7] = pack_bf16(y.x, y.y);
                    }
                    if (wide) {
                        write_traded(b, out, 2 * x, lane);
                    } else if (live) {
#pragma unroll
                        for (int y = 0; y < 8; ++y)
                            reinterpret_cast<uint4*>(out + 2 * x)[y] = make_uint4(b[y >> 1][4 * (y & 1)], b[y >> 1][4 * (y & 1) + 1],
                                                                                  b[y >> 1][4 * (y & 1) + 2], b[y >> 1][4 * (y & 1) + 3]);
                    }
                }
            }
            if (live) {
                if (SPLIT) p.part_ml[at] = make_float2(m2, l);
                else if (a.lse) a.lse[row * a.n_heads + head] = l == 0.f ? -CUDART_INF_F : fmaf(m2, kLn2, logf(l));
            }
            __syncwarp();
        }
        fence_before_sync();
    }
    if (late) flag(p.status, KDA_DEV_WAIT_TIMEOUT);
    __syncwarp();
    __syncthreads();
    if (warp == kMmaWarp) {
        fence_after_sync();
        tmem_dealloc(ms.tslot, kTmemCols);
    }
}

static_assert(kTile == kTileKeysBf16, "the decode join counts a prefix's tiles");

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
    const cuuint32_t one[4] = {1, 1, 1, 1};
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

// The cache's rows in eights, a page (or 128 rows of one) a box: 64 columns x 8 rows x the
// columns' 64s x the eights.
bool cache_map(CUtensorMap* m, const void* base, const kda_attn_prefill_args& a) {
    const cuuint64_t row = (cuuint64_t)a.d * 2;
    const cuuint64_t dims[4] = {64, 8, (cuuint64_t)a.d / 64, (cuuint64_t)(a.n_blocks * a.n_kv_heads * (a.block_size / 8))};
    const cuuint64_t strides[3] = {row, 128, 8 * row};
    const cuuint32_t box[4] = {64, 8, (cuuint32_t)a.d / 64, (cuuint32_t)(a.block_size < kTile ? a.block_size : kTile) / 8};
    return make_map(m, base, 4, dims, strides, box);
}

template <int D, int MODE, bool SPLIT>
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
    if (SPLIT) blocks *= p.n_split;
    if (blocks > (int64_t)INT32_MAX) return cudaErrorInvalidValue;
    const cudaError_t e = cudaFuncSetAttribute(attn_tc_kernel<D, MODE, SPLIT>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               (int)smem_bytes<D>());
    if (e != cudaSuccess) return e;
    note_launch();
    return launch_overlapped(attn_tc_kernel<D, MODE, SPLIT>, dim3((unsigned)blocks), dim3(kThreads), smem_bytes<D>(), s, p, maps);
}

template <int D>
cudaError_t launch_d(const AttnTileLaunch& p, cudaStream_t s) {
    if (p.prefix_lens) return launch_t<D, kPrefix, true>(p, s);
    if (p.n_split > 1) return p.a.block_table ? launch_t<D, kPaged, true>(p, s) : launch_t<D, kPacked, true>(p, s);
    return p.a.block_table ? launch_t<D, kPaged, false>(p, s) : launch_t<D, kPacked, false>(p, s);
}

}  // namespace

cudaError_t launch_attn_tc(const AttnTileLaunch& p, cudaStream_t s) {
    return p.a.d == 128 ? launch_d<128>(p, s) : launch_d<64>(p, s);
}

}  // namespace kda
