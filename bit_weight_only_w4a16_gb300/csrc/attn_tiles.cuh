// Tiled attention on the 5th-generation tensor cores: the kernel behind the
// prompt attention and the tree attention (which differ in what a query row may
// see, not in the arithmetic).
//
// Mathematics. For a row (query token, query head) with kept keys t:
//   s_t = c q.k_t (c = scale * log2 e),  out = sum_t 2^(s_t - m) v_t / sum_t 2^(s_t - m)
// for any m; one pass keeps m near the running maximum. m moves only when the
// maximum has grown by more than 2^8 (a weight is then at most 256, which bf16
// holds with the same relative error), so the accumulator in tensor memory is
// rarely rescaled. Weights are rounded to bf16 (relative 2^-8) for the tensor
// core's value product: the output is bf16, whose own rounding is as large. (The
// decode attention of one token carries its weights as two bf16 parts and returns
// fp32: it is bound by the stream; here a second part would be half as many
// operations more where they are the bound.) The sum of the weights, m and the
// accumulator are fp32.
//
// Rows. The G query heads of one key/value head share its keys, so a tile's 128
// rows are (token, head) pairs, 128 / G tokens with all their heads: each key
// tile serves all of them, a causal tile wastes at most 128 / G tokens of
// diagonal, and a few tokens still fill the rows.
//
// Work. A unit is one 128-key tile of one row tile. All units of a call, in
// order, are cut into equal runs, one per CTA (one CTA per SM): a CTA finishes
// the row tile its predecessor began, does whole ones, and begins another. A row
// tile that was cut leaves partial sums (accumulator, m, sum) in the scratch,
// which a second kernel merges in key order (deterministic).
//
// Tensor memory (512 columns) holds two score tiles and the accumulators: two row
// tiles share the keys at D <= 128; above, one row tile has two score tiles in
// turn, and from D = 384 on the value width is cut into two slices, each with a CTA
// of its own that forms the scores again (half as many operations more).
//
//   warp 0      tensor copies of Q, then of K and V stages through a ring
//   warp 1      issues tcgen05.mma: S = Q K^T into tensor memory, O += P V with P
//               read from tensor memory
//   warp 2      repairs V stages of edge tiles in shared memory: the rows that no
//               query row keeps become zeros (0 * NaN would poison the product)
//   warp 3      announces the run's pieces of row tiles
//   warps 4-11  softmax: scores from tensor memory, P back over them; at the end
//               of a row tile the same threads read O
//
// What bounds it (measured on GB300, clock 1.95 GHz). A unit takes the tensor core
// 8 D cycles (2048 at D = 256); the kernel takes 2790 there: each wait and
// each commit of the issuing thread leaves the tensor core about 50 and 20 cycles
// idle, the rest is the chain scores -> weights (about 1200 cycles: tensor-memory
// reads, the exchange of the maxima, 64 exponentials a thread, the store) -> product
// when it is longer than the other buffer's work. 16384 tokens, 8 heads on 1: D =
// 256 0.68 ms, 1.62 PFLOP/s, when calls lie apart (0.84 of the measured cuBLAS burst), 0.72
// ms in seconds of calls, when the power cap takes the clock to 1.74 GHz; D = 128 0.44 ms, 1.25
// PFLOP/s (the chain: with two row tiles a thread has 128 exponentials). 256 tokens after
// 130000, D = 512: 0.57-0.59 ms apart, 0.93-0.96 PFLOP/s of the operations asked for, 1.4
// of those done; 0.61 ms in seconds of calls. A long cache streams at
// 6.1 TB/s; 131072 x 512 with 16 nodes takes 84 us, of which 44 are the stream, 13
// the merge and the rest start and end.
//
// Value rows that some rows of a tile keep and others do not (the diagonal, a
// window's start, siblings in a tree) are searched for NaN and infinities as
// well: such elements become zero for the product and are added, in the
// epilogue, to exactly the rows that keep them.
#pragma once

#include "common.cuh"
#include "internal.h"

#include <cuda.h>
#include <type_traits>

namespace w4 {
namespace attn {

constexpr int kKeys = 128;      // keys per tile
constexpr int kRowsQ = 128;     // rows of one MMA tile
constexpr int kBlock = 16384;   // 128 rows x 64 dims: a block of Q or K
constexpr int kSmemBlocks = 14; // Q tiles and ring together
constexpr int kMaxSlots = 12;   // ring slots
constexpr int kPieces = 4;      // pieces in flight between the warps
// Waits give up after so many tries of 20 us: 0.7 s for what the next unit brings, 40 s
// for what lies a piece away (a whole row tile: units times 1 to 5 us; the largest keys
// and values that fit the device take about 25 s). A short wait that gives up ends all others.
constexpr int kWaitLimit = 1 << 15, kWaitPiece = 1 << 21;
constexpr int kMaxSeqs = 4096;  // sequences of a call (their tile prefix is staged in the ring's space)

template <int D>
struct Shape {
    static constexpr int DIM = D;
    static constexpr int NV = D > 256 ? 2 : 1;       // slices of the value width (tensor memory holds 256 columns of O)
    static constexpr int DV = D / NV;                // width of a slice
    static constexpr int TQ = D <= 128 ? 2 : 1;      // MMA row tiles per CTA
    static constexpr int QB = D / 64;                // blocks of a row tile's Q
    // One ring of stages in the order of use. 32 KiB where the ring then still
    // covers a copy's latency (about 1500 cycles): waiting for a stage and freeing
    // it leave the tensor core about 60 cycles without work.
    static constexpr int STAGE = D == 64 || D == 512 ? kBlock : 2 * kBlock;
    static constexpr int KB = STAGE / kBlock;             // blocks of a key stage
    static constexpr int KC = QB / KB;                    // key stages per tile
    static constexpr int VKEYS = DV <= 128 ? 128 : (D == 512 ? 32 : 64); // keys per value stage
    static constexpr int VC = kKeys / VKEYS;              // value stages per tile
    static constexpr int VBYTES = VKEYS * DV * 2;
    static constexpr int NS = (kSmemBlocks - TQ * QB) * kBlock / STAGE;  // ring slots
    static constexpr int ROWS = TQ * kRowsQ;
    static constexpr bool PAIR = TQ == 1;            // two threads per row, each with half of the keys
    static constexpr int ROW_WARPS = PAIR ? 8 : 4;   // warps that serve one MMA row tile
    static constexpr int THREADS = 12 * 32;
    // Cutting the work, a row tile counts as its units and this many more (copying
    // Q, the first scores without a product beside them, reading the accumulator)
    // when there are as many row tiles as CTAs: a run is then at least
    // 1 + TILE_COST long and holds a unit. With fewer the units alone are cut.
    // Measured (8192 tokens, 8 heads): runs of many short row tiles took a third
    // longer than the others with 3 at D = 256, as long with 4.
    static constexpr int TILE_COST = D == 256 ? 4 : (D > 256 ? 3 : 2);
    static constexpr int QBYTES = TQ * QB * kBlock;
    static constexpr size_t TILES = (size_t)QBYTES + NS * STAGE;
    static constexpr size_t SMEM = TILES + 3072;
    static_assert(VBYTES <= STAGE && VBYTES % 1024 == 0 && NS <= kMaxSlots, "ring");
    static_assert(SMEM <= 232448, "shared memory");
};

// Scratch of a call with `grid` CTAs (floats): accumulators, (m, sum) per row,
// then the integer tables.
constexpr size_t kSlotFloats = 32768; // ROWS * DV at most
inline size_t ws_need(int grid)
{
    return (size_t)2 * grid * kSlotFloats + (size_t)2 * grid * 256 * 2 + (size_t)8 * grid + 64;
}

struct Args {
    uint16_t *out;
    long long ldo; // elements between tokens
    const int32_t *cu_q, *cu_k;    // prompt: [B + 1] first query / key row of each sequence
    const int32_t *parents, *pos;  // tree: [B][N], [B]
    const int32_t *kpos;           // tree: [B][T] or null
    const uint16_t *v, *vt;        // value rows (only for the NaN / infinity path)
    long long ldv;
    float *ws_o, *ws_ml;
    int32_t *rec;   // [grid][2]: the continued row tile (0 = none, 1 = goes on, 3 = ends here); 1 = begins one
    int32_t *where; // [grid][4]: token row, tokens, key/value head, slice of the tile whose first partial CTA c holds
    int *err;
    int B, N, T; // sequences; tree: nodes, slots
    int total_q, total_k;
    int Hq, Hkv, G, D;
    int tpt; // tokens per MMA row tile: 128 / G
    int window;
    float c; // scale * log2(e)
};

struct Maps {
    CUtensorMap q, k, v, kt, vt;
};

// ------------------------------------------------------------------ PTX ----

__device__ __forceinline__ uint64_t sdesc_kmajor(uint32_t saddr)
{
    uint64_t d = (uint64_t)((saddr & 0x3FFFFu) >> 4);
    d |= (uint64_t)1 << 16;
    d |= (uint64_t)(1024 >> 4) << 32; // 8 rows x 128 B
    d |= (uint64_t)1 << 46;
    d |= (uint64_t)2 << 61; // 128-byte swizzle
    return d;
}

// The same swizzle with the other dimension contiguous: 64 dims per 128-byte
// row, `group` bytes between blocks of 64 dims, 1024 between blocks of 8 keys.
__device__ __forceinline__ uint64_t sdesc_mnmajor(uint32_t saddr, uint32_t group)
{
    uint64_t d = (uint64_t)((saddr & 0x3FFFFu) >> 4);
    d |= (uint64_t)(group >> 4) << 16;
    d |= (uint64_t)(1024 >> 4) << 32;
    d |= (uint64_t)1 << 46;
    d |= (uint64_t)2 << 61;
    return d;
}

constexpr uint32_t idesc_bf16(int n, bool b_mn)
{
    return (1u << 4) | (1u << 7) | (1u << 10) | (b_mn ? 1u << 16 : 0u) | ((uint32_t)(n >> 3) << 17) |
           ((uint32_t)(kRowsQ >> 4) << 24);
}

__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc)
{
    asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
                 "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
                 "l"(a), "l"(b), "r"(idesc), "r"(acc)
                 : "memory");
}

__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t acc)
{
    asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
                 "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
                 "r"(a), "l"(b), "r"(idesc), "r"(acc)
                 : "memory");
}

__device__ __forceinline__ void mma_commit(uint32_t bar)
{
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar)
                 : "memory");
}

__device__ __forceinline__ void tma_3d(uint32_t dst, const CUtensorMap *map, int c0, int c1, int c2, uint32_t bar)
{
    asm volatile("cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
                 " [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
                 "l"(map), "r"(c0), "r"(c1), "r"(c2), "r"(bar)
                 : "memory");
}

// One lane of the warp, in a form the compiler knows to be a single thread:
// issuing products from `lane == 0` instead took twice as long per instruction.
__device__ __forceinline__ bool elect_one()
{
    uint32_t p;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xFFFFFFFF;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
    return p != 0;
}

__device__ __forceinline__ void tc_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

#define W4_R32(v, o)                                                                                             \
    "=r"(v[o + 0]), "=r"(v[o + 1]), "=r"(v[o + 2]), "=r"(v[o + 3]), "=r"(v[o + 4]), "=r"(v[o + 5]),              \
        "=r"(v[o + 6]), "=r"(v[o + 7]), "=r"(v[o + 8]), "=r"(v[o + 9]), "=r"(v[o + 10]), "=r"(v[o + 11]),        \
        "=r"(v[o + 12]), "=r"(v[o + 13]), "=r"(v[o + 14]), "=r"(v[o + 15]), "=r"(v[o + 16]), "=r"(v[o + 17]),    \
        "=r"(v[o + 18]), "=r"(v[o + 19]), "=r"(v[o + 20]), "=r"(v[o + 21]), "=r"(v[o + 22]), "=r"(v[o + 23]),    \
        "=r"(v[o + 24]), "=r"(v[o + 25]), "=r"(v[o + 26]), "=r"(v[o + 27]), "=r"(v[o + 28]), "=r"(v[o + 29]),    \
        "=r"(v[o + 30]), "=r"(v[o + 31])
#define W4_I32(v, o)                                                                                             \
    "r"(v[o + 0]), "r"(v[o + 1]), "r"(v[o + 2]), "r"(v[o + 3]), "r"(v[o + 4]), "r"(v[o + 5]), "r"(v[o + 6]),     \
        "r"(v[o + 7]), "r"(v[o + 8]), "r"(v[o + 9]), "r"(v[o + 10]), "r"(v[o + 11]), "r"(v[o + 12]),             \
        "r"(v[o + 13]), "r"(v[o + 14]), "r"(v[o + 15]), "r"(v[o + 16]), "r"(v[o + 17]), "r"(v[o + 18]),          \
        "r"(v[o + 19]), "r"(v[o + 20]), "r"(v[o + 21]), "r"(v[o + 22]), "r"(v[o + 23]), "r"(v[o + 24]),          \
        "r"(v[o + 25]), "r"(v[o + 26]), "r"(v[o + 27]), "r"(v[o + 28]), "r"(v[o + 29]), "r"(v[o + 30]),          \
        "r"(v[o + 31])

// 32 consecutive columns of this thread's tensor-memory lane; the wait belongs to
// the same statement, so that no use of the registers can move before it.
#define W4_TLD32(v, addr)                                                                                        \
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x32.b32 "                                                       \
                 "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"                                       \
                 "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];\n\t"                  \
                 "tcgen05.wait::ld.sync.aligned;"                                                                \
                 : W4_R32(v, 0)                                                                                  \
                 : "r"(addr)                                                                                     \
                 : "memory")
// 64 columns, as two loads and one wait.
#define W4_TLD64(v, addr) \
    asm volatile(\
                 "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15," \
                 "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%64];\n\t" \
                 "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%32,%33,%34,%35,%36,%37,%38,%39,%40,%41,%42,%43,%44,%45,%46,%47," \
                 "%48,%49,%50,%51,%52,%53,%54,%55,%56,%57,%58,%59,%60,%61,%62,%63}, [%65];\n\t" \
                 "tcgen05.wait::ld.sync.aligned;" \
                 : W4_R32(v, 0), W4_R32(v, 32) \
                 : "r"(addr), "r"((addr) + 32u) \
                 : "memory")
// 16 columns.
#define W4_TST16(v, o, addr) \
    asm volatile("tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], " \
                 "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15};" ::"r"(v[o + 0]), "r"(v[o + 1]), \
                 "r"(v[o + 2]), "r"(v[o + 3]), "r"(v[o + 4]), "r"(v[o + 5]), "r"(v[o + 6]), "r"(v[o + 7]), \
                 "r"(v[o + 8]), "r"(v[o + 9]), "r"(v[o + 10]), "r"(v[o + 11]), "r"(v[o + 12]), "r"(v[o + 13]), \
                 "r"(v[o + 14]), "r"(v[o + 15]), "r"(addr) \
                 : "memory")
#define W4_TST32(v, o, addr)                                                                                     \
    asm volatile("tcgen05.st.sync.aligned.32x32b.x32.b32 [%32], "                                                \
                 "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"                                       \
                 "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31};" ::W4_I32(v, o),             \
                 "r"(addr)                                                                                       \
                 : "memory")

__device__ __forceinline__ void sts128(uint32_t a, uint4 v)
{
    asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(a), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}

__device__ __forceinline__ float ex2(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// The lowest n bits (none for n <= 0, all for n >= 32).
__device__ __forceinline__ uint32_t below(int n)
{
    return n >= 32 ? 0xFFFFFFFFu : (n <= 0 ? 0u : (1u << n) - 1u);
}

// Two fp32 rounded to bf16 (nearest even), the first in the low half.
__device__ __forceinline__ uint32_t pack2(float lo, float hi)
{
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

// ------------------------------------------------------------ the work ----

// A sequence as the kernel sees it: its query rows, its key rows, and for a row
// tile the range of keys that any of its rows keeps.
struct Seq {
    int q0, lq; // first query row, query rows
    int k0, lk; // first key row (cache row), keys (prompt: the sequence's; tree: min(pos, T))
    int off;    // prompt: position of query row 0; tree: position of depth 0
};

template <bool TREE>
__device__ __forceinline__ Seq load_seq(const Args &a, int s)
{
    Seq q;
    if (TREE) {
        q.q0 = s * a.N;
        q.lq = a.N;
        q.k0 = s * a.T;
        q.off = max(__ldg(a.pos + s), 0);
        q.lk = min(q.off, a.T);
    } else {
        // Ends are taken into the tensors first: an end before its start is an empty sequence.
        q.q0 = __ldg(a.cu_q + s);
        q.lq = q.q0 < 0 ? 0 : max(0, max(0, min(__ldg(a.cu_q + s + 1), a.total_q)) - q.q0);
        q.k0 = max(0, __ldg(a.cu_k + s));
        q.lk = max(0, max(0, min(__ldg(a.cu_k + s + 1), a.total_k)) - q.k0);
        q.off = q.lk - q.lq;
    }
    return q;
}

// First position that a window ending at position `at` holds. Positions below zero keep
// nothing, so they count as 0: the difference stays within 32 bits for every window.
__device__ __forceinline__ int window_start(int at, int window) { return max(0, max(at, 0) - window + 1); }

// First key and one past the last that any of the tokens [t0, t0 + nt) keeps.
template <bool TREE>
__device__ __forceinline__ void key_range(const Args &a, const Seq &q, int t0, int nt, int &lo, int &hi)
{
    if (TREE) {
        lo = a.window > 0 ? window_start(q.off, a.window) : 0; // depth 0 sees furthest back
        hi = q.lk;
        if (a.kpos) { // any slot may hold any position
            lo = 0;
            hi = a.T;
        }
    } else {
        lo = a.window > 0 ? window_start(q.off + t0, a.window) : 0;
        hi = min(q.lk, q.off + t0 + nt);
    }
    if (hi <= lo) {
        lo = 0;
        hi = 0;
    }
}

// Units of a row tile: its key tiles, and in a tree call one more for the tree's
// own keys; at least one, so that rows without keys are written.
template <bool TREE>
__device__ __forceinline__ int tile_units(int lo, int hi)
{
    const int n = hi > lo ? (hi + kKeys - 1) / kKeys - lo / kKeys : 0;
    return TREE ? n + 1 : max(n, 1);
}

// A piece: units [u, u1) of one row tile, as all warps see it.
struct Piece {
    int units;         // u1 - u; 0 ends the run
    int hs;            // key/value head * NV + slice of the value width
    int s;             // sequence
    int t0, nt;        // first token within the sequence, tokens
    int lo, hi;        // keys that any row keeps lie in [lo, hi)
    int n, u, u1;      // units of the row tile, of the piece
    int q0, k0;        // the sequence's first query row, first key row
    int lk, off;       // its keys; position of query row 0 (tree: of depth 0)
    int nq;            // MMA row tiles that hold any token

    __device__ __forceinline__ bool whole() const { return u == 0 && u1 == n; }
};

// Key tile of unit x of the row tile; in a tree call the tree's own keys follow
// the cache's.
template <bool TREE>
__device__ __forceinline__ bool tree_unit(const Piece &w, int x)
{
    return TREE && x == w.n - 1;
}
__device__ __forceinline__ int key0(const Piece &w, int x) { return (w.lo / kKeys + x) * kKeys; }

// A unit whose value rows need repair: keys outside [lo, hi), keys that only
// some rows keep, recorded positions, the tree's own keys.
template <bool TREE>
__device__ __forceinline__ bool edge_unit(const Args &a, const Piece &w, int x)
{
    const int k = key0(w, x);
    if (TREE) {
        if (tree_unit<TREE>(w, x) || a.kpos)
            return true;
        return k + kKeys > w.hi || k < w.lo || (a.window > 0 && k < w.lo + 64);
    }
    if (k + kKeys > w.off + w.t0 + 1 || k + kKeys > w.hi || k < w.lo) // past the first row's last key
        return true;
    return a.window > 0 && k < window_start(w.off + w.t0 + w.nt - 1, a.window); // before the last row's first key
}

// A value row's part in the product: 0 = kept by every row (or zeros already), 1 = by
// some, 2 = by none.
template <bool TREE>
__device__ __forceinline__ int key_class(const Args &a, const Piece &w, int x, int j)
{
    if (TREE) {
        // Rows past the last sequence's are past the tensor: copied as zeros.
        const int past = w.s == a.B - 1 ? 0 : 2;
        if (tree_unit<TREE>(w, x))
            return j < a.N ? 1 : past;
        const int k = key0(w, x) + j;
        if (k >= a.T)
            return past;
        const int p = a.kpos ? __ldg(a.kpos + (size_t)w.s * a.T + k) : k;
        if (p < 0 || p >= w.off)
            return 2;
        if (a.window > 0) {
            if ((long long)p <= (long long)w.off - a.window)
                return 2;
            if ((long long)p <= (long long)w.off + (a.N - 1) - a.window)
                return 1;
        }
        return 0;
    }
    const int k = key0(w, x) + j;
    if (k >= a.total_k - w.k0)
        return 0; // past the tensor
    if (k >= w.hi || k < w.lo)
        return 2;
    if (k > w.off + w.t0)
        return 1;
    if (a.window > 0 && k < window_start(w.off + w.t0 + w.nt - 1, a.window))
        return 1;
    return 0;
}

// What one row keeps.
struct RowMask {
    bool live;                // a row of the output
    int lo, hi;               // kept keys (positions) [lo, hi)
    unsigned long long nodes; // tree: ancestors or self within the window

    // A tree's absent node. Value rows are judged by what the present nodes keep, so its
    // accumulator may hold 0 * NaN: zeros are selected for it. (Where a prompt's row keeps
    // nothing, its tile's first row keeps nothing either, and every key is searched.)
    __device__ __forceinline__ bool absent() const { return nodes == 0; }
};

template <bool TREE>
__device__ __forceinline__ RowMask row_mask(const Args &a, const Piece &w, int tok, bool live)
{
    RowMask m;
    m.live = live;
    m.lo = m.hi = 0;
    m.nodes = 0;
    if (!live)
        return m;
    if (TREE) {
        const int32_t *par = a.parents + (size_t)w.s * a.N;
        int j = w.t0 + tok, d = 0, p = __ldg(par + j);
        if (p == -2) // an absent node
            return m;
        for (;; ++d) {
            if (a.window <= 0 || d < a.window)
                m.nodes |= 1ull << j;
            if (p < 0 || p >= j)
                break;
            j = p;
            p = __ldg(par + j);
        }
        m.hi = a.kpos ? w.off : w.lk;
        m.lo = a.window > 0 ? (int)min(0x7FFFFFFFll, max(0ll, (long long)w.off + d - a.window + 1)) : 0;
    } else {
        const int at = w.off + w.t0 + tok;
        m.hi = min(at + 1, w.lk);
        m.lo = a.window > 0 ? window_start(at, a.window) : 0;
    }
    return m;
}

// Adds to a stored output row (or partial) the NaN and infinite values of the
// keys that warp 2 took out of the product and that this row keeps.
template <int D, bool TREE, typename Add>
__device__ __forceinline__ void add_specials(const Args &a, const Piece &w, const RowMask &m, int kvh,
                                             int dv0, int d0, int d1, Add add)
{
#pragma unroll 1
    for (int x = w.u; x < w.u1; ++x) {
        if (!edge_unit<TREE>(a, w, x))
            continue;
        const bool tree = tree_unit<TREE>(w, x);
#pragma unroll 1
        for (int j = 0; j < kKeys; ++j) {
            if (key_class<TREE>(a, w, x, j) != 1)
                continue;
            const int k = key0(w, x) + j;
            bool kept;
            const uint16_t *row;
            if (tree) {
                kept = (m.nodes >> j) & 1;
                row = a.vt + ((size_t)(w.s * (long long)a.N + j) * a.Hkv + kvh) * D;
            } else {
                const int p = TREE && a.kpos ? __ldg(a.kpos + (size_t)w.s * a.T + k) : k;
                kept = p >= m.lo && p < m.hi;
                row = a.v + (size_t)((long long)w.k0 + k) * a.ldv + (size_t)kvh * D;
            }
            if (!kept)
                continue;
#pragma unroll 1
            for (int d = d0; d < d1; ++d) {
                const uint32_t b = row[dv0 + d];
                if ((b & 0x7F80u) == 0x7F80u)
                    add(d, __uint_as_float(b << 16));
            }
        }
    }
}

// ------------------------------------------------------------- kernel ----

struct Bars {
    unsigned long long full[kMaxSlots], edge[kMaxSlots], empty[kMaxSlots];
    unsigned long long q_full, q_empty;
    unsigned long long s_full[2], p_full[2], o_done[2], o_last[2], o_free[2], drain;
    unsigned long long pc_full[kPieces], pc_empty[kPieces];
};

// What lies behind the tiles in shared memory.
struct Shared {
    Bars bars;
    Piece piece[kPieces];
    float x[2][2][kRowsQ]; // the two threads of a row: maxima, sums ([unit parity][half][row])
    int xok[2][8];         // and whether their waits ended well ([parity][softmax warp])
    int cut[2][4], tiles;
    int special[4];        // piece whose value rows had NaN or infinities
    int warp_sums[16];
    uint32_t tmem;
    volatile int abort;
};
static_assert(sizeof(Shared) <= 3072, "shared memory");

__device__ __forceinline__ unsigned long long pack64(float lo, float hi)
{
    unsigned long long r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
    return r;
}
__device__ __forceinline__ void unpack64(unsigned long long v, float &lo, float &hi)
{
    asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
}
// Two fp32 operations in one instruction.
__device__ __forceinline__ unsigned long long fma2(unsigned long long a, unsigned long long b, unsigned long long c)
{
    unsigned long long r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ unsigned long long add2(unsigned long long a, unsigned long long b)
{
    unsigned long long r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}

// Lanes that differ in bit d of their number swap: the lower one's b for the
// upper one's a.
__device__ __forceinline__ void swap4(uint4 &a, uint4 &b, int d, bool upper)
{
    uint4 t = upper ? a : b;
    t.x = __shfl_xor_sync(0xFFFFFFFFu, t.x, d);
    t.y = __shfl_xor_sync(0xFFFFFFFFu, t.y, d);
    t.z = __shfl_xor_sync(0xFFFFFFFFu, t.z, d);
    t.w = __shfl_xor_sync(0xFFFFFFFFu, t.w, d);
    if (upper)
        a = t;
    else
        b = t;
}

template <int THREADS>
__device__ __forceinline__ long long block_scan(int v, int *warp_sums, long long &total)
{
    // Inclusive sum over the block; `total` is the sum of all. A warp's sum fits 32 bits
    // (a row tile of 2^31 keys has 2^24 units, a call below 2^31 row tiles); the sum of
    // the units of 384 such tiles does not.
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    int x = v;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int y = __shfl_up_sync(0xFFFFFFFFu, x, d);
        if (lane >= d)
            x += y;
    }
    __syncthreads();
    if (lane == 31)
        warp_sums[w] = x;
    __syncthreads();
    long long before = 0, all = 0;
#pragma unroll
    for (int i = 0; i < THREADS / 32; ++i) {
        const int t = warp_sums[i];
        before += i < w ? t : 0;
        all += t;
    }
    total = all;
    return x + before;
}

// Cuts the call's row tiles, in order of (head and slice, sequence, token), with their
// units and TILE_COST each, at equal costs: sh.cut[e] is where this CTA's run begins
// (e = 0) and ends (e = 1): tile index over all heads, sequence, tile within the
// sequence, unit. sbase: space for the first row tile of each sequence.
template <typename S, bool TREE>
__device__ __forceinline__ void plan_run(const Args &a, Shared &sh, int *sbase, int tt, int HS, int &R)
{
    if (a.B == 1) {
        R = (load_seq<TREE>(a, 0).lq + tt - 1) / tt;
        if (threadIdx.x == 0)
            sbase[0] = 0;
    }
    for (int s0 = 0; a.B > 1 && s0 < a.B; s0 += S::THREADS) {
        const int s = s0 + (int)threadIdx.x;
        const int nt = s < a.B ? (load_seq<TREE>(a, s).lq + tt - 1) / tt : 0;
        long long total;
        const int incl = (int)block_scan<S::THREADS>(nt, sh.warp_sums, total);
        if (s < a.B)
            sbase[s] = R + incl - nt;
        R += (int)total; // row tiles of the call: below 2^31
    }
    __syncthreads();
    const int extra = (long long)R * HS >= (long long)gridDim.x ? S::TILE_COST : 0;
    auto units_of = [&](int r, int &s) {
        // The last sequence that begins at or before r (empty ones begin where the next does).
        int x = 0, y = a.B - 1;
        while (x < y) {
            const int m = (x + y + 1) >> 1;
            if (sbase[m] <= r)
                x = m;
            else
                y = m - 1;
        }
        s = x;
        const Seq q = load_seq<TREE>(a, s);
        const int t0 = (r - sbase[s]) * tt;
        int lo, hi;
        key_range<TREE>(a, q, t0, min(tt, q.lq - t0), lo, hi);
        return tile_units<TREE>(lo, hi);
    };
    // Thread r of the last round of row tiles: its tile's sequence, units, cost and
    // the costs up to it. With one round they serve the second pass as well.
    int s_r = 0, n_r = 0, cost_r = 0;
    long long incl_r = 0, total_r = 0;
    auto round = [&](int r0) {
        const int r = r0 + (int)threadIdx.x;
        n_r = r < R ? units_of(r, s_r) : 0;
        cost_r = n_r > 0 ? n_r + extra : 0;
        incl_r = block_scan<S::THREADS>(cost_r, sh.warp_sums, total_r);
    };
    long long W = 0;
    for (int r0 = 0; r0 < R; r0 += S::THREADS) {
        round(r0);
        W += total_r;
    }
    const long long all = W * HS;
    long long at[2];
    int hs[2];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
        const long long ctas = max(1ll, min((long long)gridDim.x, all)); // a unit each at least
        const long long x = all * min((long long)blockIdx.x + e, ctas) / ctas;
        hs[e] = W > 0 ? (int)(x / W) : 0;
        at[e] = x - hs[e] * W;
    }
    if (threadIdx.x < 2) { // the end of the last run, until a tile claims the place
        sh.cut[threadIdx.x][0] = HS * R;
        sh.cut[threadIdx.x][3] = 0;
    }
    long long before = 0;
    for (int r0 = 0; r0 < R; r0 += S::THREADS) {
        if (R > S::THREADS)
            round(r0);
        else
            __syncthreads(); // after the defaults above
        const int r = r0 + (int)threadIdx.x;
        const long long p = before + incl_r - cost_r;
#pragma unroll
        for (int e = 0; e < 2; ++e)
            if (cost_r > 0 && hs[e] < HS && at[e] >= p && at[e] < p + cost_r) {
                sh.cut[e][0] = hs[e] * R + r;
                sh.cut[e][1] = s_r;
                sh.cut[e][2] = r - sbase[s_r];
                sh.cut[e][3] = (int)max(0ll, at[e] - p - extra);
            }
        before += total_r;
        if (max(at[0], at[1]) < before)
            break;
    }
}

template <int D, bool TREE>
__global__ void __launch_bounds__(Shape<D>::THREADS, 1)
attn_kernel(const __grid_constant__ Args a, const __grid_constant__ Maps maps)
{
    using S = Shape<D>;
    extern __shared__ __align__(1024) unsigned char smem[];
    const uint32_t q_base = smem_addr(smem);
    const uint32_t ring = q_base + S::QBYTES;
    Shared &sh = *reinterpret_cast<Shared *>(smem + S::TILES);
    Bars &bars = sh.bars;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (q_base & 1023u) { // the swizzle's atoms are 1024 bytes; there is no static shared memory before them
        if (threadIdx.x == 0)
            atomicOr(a.err, 8);
        return;
    }

    if (threadIdx.x == 0) {
        for (int i = 0; i < kMaxSlots; ++i) {
            mbar_init(smem_addr(&bars.full[i]), 1);
            mbar_init(smem_addr(&bars.edge[i]), 1); // a copied stage that warp 2 repairs before `full`
            mbar_init(smem_addr(&bars.empty[i]), 1);
        }
        mbar_init(smem_addr(&bars.q_full), 1);
        mbar_init(smem_addr(&bars.q_empty), 1);
        mbar_init(smem_addr(&bars.drain), 1);
        for (int i = 0; i < 2; ++i) {
            mbar_init(smem_addr(&bars.s_full[i]), 1);
            mbar_init(smem_addr(&bars.p_full[i]), S::ROW_WARPS);
            mbar_init(smem_addr(&bars.o_done[i]), 1); // a unit's product
            mbar_init(smem_addr(&bars.o_last[i]), 1); // a piece's last one
            mbar_init(smem_addr(&bars.o_free[i]), S::ROW_WARPS);
        }
        for (int i = 0; i < kPieces; ++i) {
            mbar_init(smem_addr(&bars.pc_full[i]), 1);
            mbar_init(smem_addr(&bars.pc_empty[i]), 3 + 8);
        }
        sh.abort = 0;
        for (int i = 0; i < 4; ++i)
            sh.special[i] = -1;
        fence_mbar_init();
    }
    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                         smem_addr(&sh.tmem)),
                     "r"(512));
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
    }
    if (threadIdx.x == 32) {
        const CUtensorMap *m = &maps.q;
        for (int i = 0; i < (TREE ? 5 : 3); ++i)
            asm volatile("prefetch.tensormap [%0];" ::"l"(m + i) : "memory");
    }
    pdl_launch_dependents();
    pdl_wait();

    // -------------------------------------------------- this CTA's run
    {
        const int tt = a.tpt * S::TQ, HS = a.Hkv * S::NV;
        int R = 0; // row tiles of a head
        if (TREE && a.B == 1) {
            // One tree: its row tiles have the same units.
            if (threadIdx.x < 2) {
                const Seq q = load_seq<TREE>(a, 0);
                int lo, hi;
                key_range<TREE>(a, q, 0, q.lq, lo, hi);
                R = (q.lq + tt - 1) / tt;
                const int extra = (long long)R * HS >= (long long)gridDim.x ? S::TILE_COST : 0;
                const long long cost = tile_units<TREE>(lo, hi) + extra, all = cost * R * HS;
                const long long ctas = min((long long)gridDim.x, all); // a unit each at least
                const long long x = all * min((long long)blockIdx.x + threadIdx.x, ctas) / ctas;
                const int tile = (int)(x / cost);
                sh.cut[threadIdx.x][0] = tile;
                sh.cut[threadIdx.x][1] = 0;
                sh.cut[threadIdx.x][2] = tile % R;
                sh.cut[threadIdx.x][3] = (int)max(0ll, x - tile * cost - extra);
            }
        } else {
            plan_run<S, TREE>(a, sh, reinterpret_cast<int *>(smem), tt, HS, R);
        }
        if (threadIdx.x == 0)
            sh.tiles = R;
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); // sbase reads before the ring's copies
        tc_fence_before();
        __syncthreads();
        tc_fence_after();
    }
    // All 512 columns: they begin at 0, which keeps the addresses constants.
    constexpr uint32_t tmem = 0;
    // S (and P over it) in columns [128 b, 128 b + 128), O_t from 256 + t * DV.
    auto s_col = [&](int b) { return tmem + 128u * (uint32_t)b; };
    auto o_col = [&](int t) { return tmem + 256u + (uint32_t)(t * S::DV); };

    auto wait = [&](unsigned long long &bar, uint32_t parity, int limit = kWaitLimit) -> bool {
        const uint32_t b = smem_addr(&bar);
        for (int i = 0; i < limit; ++i) {
            if (mbar_try_wait(b, parity, 20000u))
                return true;
            if (sh.abort)
                return false;
        }
        sh.abort = 1;
        atomicOr(a.err, 8);
        return false;
    };

    // Piece p is in sh.piece[p % kPieces] between these two.
    auto take = [&](uint32_t p) { return wait(bars.pc_full[p % kPieces], (p / kPieces) & 1, kWaitPiece); };
    auto done = [&](uint32_t p) { mbar_arrive(smem_addr(&bars.pc_empty[p % kPieces])); };

    if (warp == 0) {
        // ---------------------------------------------------- copies
        if (elect_one()) {
            uint32_t g = 0, piece = 0;    // stages, pieces so far
            uint32_t par = 0, onedge = 0; // per slot: uses of its edge barrier (parity), the last use was one
            bool ok = true;
            for (; ok; ++piece) {
                if (!(ok = take(piece)))
                    break;
                const Piece w = sh.piece[piece % kPieces];
                done(piece);
                if (w.units == 0)
                    break;
                if (piece > 0 && !(ok = wait(bars.q_empty, (piece - 1) & 1)))
                    break; // the Q copies waited for below are the previous piece's
                const int kvh = w.hs / S::NV, dv0 = (w.hs % S::NV) * S::DV;
                mbar_arrive_expect_tx(smem_addr(&bars.q_full), (uint32_t)(w.nq * S::QB * a.tpt * a.G * 128));
                for (int t = 0; t < w.nq; ++t)
                    for (int c = 0; c < S::QB; ++c)
                        tma_3d(q_base + (t * S::QB + c) * kBlock, &maps.q, 64 * c, kvh * a.G,
                               w.q0 + w.t0 + t * a.tpt, smem_addr(&bars.q_full));
                auto keys = [&](int j) {
                    const int x = w.u + j;
                    const bool tr = tree_unit<TREE>(w, x);
                    const CUtensorMap *m = tr ? &maps.kt : &maps.k;
                    const int row = tr ? w.s * a.N : w.k0 + key0(w, x);
                    for (int c = 0; c < S::KC; ++c, ++g) {
                        const uint32_t slot = g % S::NS, use = g / S::NS;
                        if (use > 0 && !wait(bars.empty[slot], (use - 1) & 1))
                            return false;
                        const uint32_t bar = smem_addr(&bars.full[slot]);
                        onedge &= ~(1u << slot);
                        mbar_arrive_expect_tx(bar, S::STAGE);
#pragma unroll
                        for (int b = 0; b < S::KB; ++b)
                            tma_3d(ring + slot * S::STAGE + b * kBlock, m, 64 * (c * S::KB + b), kvh, row, bar);
                    }
                    return true;
                };
                auto values = [&](int j) {
                    const int x = w.u + j;
                    const bool tr = tree_unit<TREE>(w, x), edge = edge_unit<TREE>(a, w, x);
                    const CUtensorMap *m = tr ? &maps.vt : &maps.v;
                    const int row = tr ? w.s * a.N : w.k0 + key0(w, x);
                    for (int c = 0; c < S::VC; ++c, ++g) {
                        const uint32_t slot = g % S::NS, use = g / S::NS;
                        if (use > 0 && !wait(bars.empty[slot], (use - 1) & 1))
                            return false;
                        const uint32_t bar = smem_addr(edge ? &bars.edge[slot] : &bars.full[slot]);
                        onedge = edge ? onedge | (1u << slot) : onedge & ~(1u << slot);
                        par ^= edge ? 1u << slot : 0u;
                        mbar_arrive_expect_tx(bar, S::VBYTES);
#pragma unroll
                        for (int b = 0; b < S::DV / 64; ++b)
                            tma_3d(ring + slot * S::STAGE + b * (S::VKEYS * 128), m, dv0 + 64 * b, kvh,
                                   row + c * S::VKEYS, bar);
                    }
                    return true;
                };
                ok = keys(0);
                for (int j = 0; ok && j < w.units; ++j) {
                    const bool more = j + 1 < w.units;
                    ok = S::PAIR ? (!more || keys(j + 1)) && values(j) : values(j) && (!more || keys(j + 1));
                }
            }
            if (!ok) {
                // Copies in flight write this CTA's shared memory: let them land.
                for (int i = 0; i < S::NS; ++i) {
                    const uint32_t uses = (g + S::NS - 1 - i) / S::NS;
                    if ((onedge >> i) & 1)
                        mbar_wait_bounded(smem_addr(&bars.edge[i]), ((par >> i) & 1) ^ 1, 64);
                    else if (uses > 0)
                        mbar_wait_bounded(smem_addr(&bars.full[i]), (uses - 1) & 1, 64);
                }
                if (piece > 0)
                    mbar_wait_bounded(smem_addr(&bars.q_full), (piece - 1) & 1, 64);
            }
        }
    } else if (warp == 1) {
        // ---------------------------------------------- tensor-core issue
        // One thread's tensor-core instructions execute in the order of their issue:
        // scores may go over weights that a product issued before them reads. Its
        // shared-memory accesses queue behind them, and the queue holds about six:
        // what the next stage needs is waited for in the middle of a stage, so that
        // there is something to issue as soon as the wait is over.
        if (elect_one()) {
            constexpr uint32_t id_s = idesc_bf16(kKeys, false), id_o = idesc_bf16(S::DV, true);
            uint32_t g = 0; // stages so far
            auto ready = [&](uint32_t i) { return wait(bars.full[i % S::NS], (i / S::NS) & 1); };
            // Scores of row tile t into buffer b from the stages i ..; `next` waits for
            // what follows; `free`: the last user of the stages.
            auto scores = [&](int t, int b, uint32_t i, bool see, bool free, auto next) {
#pragma unroll
                for (int c = 0; c < S::KC; ++c, ++i) {
                    const uint32_t slot = i % S::NS;
                    const uint64_t ad = sdesc_kmajor(q_base + (t * S::QB + c * S::KB) * kBlock);
                    const uint64_t bd = sdesc_kmajor(ring + slot * S::STAGE);
#pragma unroll
                    for (int k = 0; k < 4 * S::KB; ++k) {
                        if (k == 2 * S::KB && !(c + 1 < S::KC ? !see || ready(i + 1) : next()))
                            return false;
                        const uint32_t step = (k >> 2) * (kBlock >> 4) + 2u * (k & 3);
                        mma_ss(s_col(b), ad + step, bd + step, id_s, (c > 0 || k > 0) ? 1u : 0u);
                    }
                    if (free)
                        mma_commit(smem_addr(&bars.empty[slot]));
                }
                mma_commit(smem_addr(&bars.s_full[b]));
                return true;
            };
            // O_t (+)= P V with the weights in buffer b.
            auto product = [&](int t, int b, uint32_t i, uint32_t acc, bool see, bool free, auto next) {
#pragma unroll
                for (int c = 0; c < S::VC; ++c, ++i) {
                    const uint32_t slot = i % S::NS;
                    const uint64_t bd = sdesc_mnmajor(ring + slot * S::STAGE, S::VKEYS * 128);
#pragma unroll
                    for (int k = 0; k < S::VKEYS / 16; ++k) {
                        if (k == S::VKEYS / 32 && !(c + 1 < S::VC ? !see || ready(i + 1) : next()))
                            return false;
                        mma_ts(o_col(t), s_col(b) + (uint32_t)(c * S::VKEYS / 2 + 8 * k), bd + 128u * k, id_o,
                               c > 0 || k > 0 ? 1u : acc);
                    }
                    if (free)
                        mma_commit(smem_addr(&bars.empty[slot]));
                }
                mma_commit(smem_addr(&bars.o_done[t]));
                return true;
            };
            // The weights of a row tile's next product; at a piece's first unit the last
            // piece's accumulator has been read.
            auto weights_in = [&](int t, int b, uint32_t use, bool begin, uint32_t mine) {
                if (!wait(bars.p_full[b], use & 1) || !(!begin || mine == 0 || wait(bars.o_free[t], (mine - 1) & 1)))
                    return false;
                tc_fence_after();
                return true;
            };
            auto nothing = [] { return true; };
            auto finished = [&](int t, bool more) {
                if (!more)
                    mma_commit(smem_addr(&bars.o_last[t]));
                return true;
            };
            uint32_t n = 0, n1 = 0;        // units so far, of the second row tile
            uint32_t mine = 0, mine1 = 0;  // pieces so far, with a second row tile
            bool ok = true;
            for (uint32_t piece = 0; ok; ++piece) {
                if (!(ok = take(piece)))
                    break;
                const int units = sh.piece[piece % kPieces].units, nq = sh.piece[piece % kPieces].nq;
                done(piece);
                if (units == 0 || !(ok = wait(bars.q_full, piece & 1) && ready(g)))
                    break;
                if (S::PAIR) {
                    // Two score buffers: S(j + 1) before the product of unit j. Stages:
                    // K(0), K(1), V(0), K(2), V(1), ..., V(n - 1).
                    ok = scores(0, n & 1, g, true, true, [&] { return units == 1 || ready(g + S::KC); });
                    g += S::KC;
                    for (int j = 0; ok && j < units; ++j, ++n) {
                        const int b = n & 1;
                        auto operands = [&](uint32_t v) { return ready(v) && weights_in(0, b, n >> 1, j == 0, mine); };
                        if (j + 1 < units) {
                            ok = scores(0, b ^ 1, g, true, true, [&] { return operands(g + S::KC); });
                            g += S::KC;
                        } else {
                            ok = operands(g);
                        }
                        if (ok && (j + 2 == units || units == 1))
                            mma_commit(smem_addr(&bars.q_empty));
                        ok = ok && product(0, b, g, j > 0 ? 1u : 0u, true, true,
                                           [&] { return j + 2 >= units || ready(g + S::VC); });
                        if (j + 1 == units)
                            mma_commit(smem_addr(&bars.o_last[0]));
                        g += S::VC;
                    }
                } else {
                    // One score buffer per row tile: its product, then its next scores.
                    // Stages: K(0), V(0), K(1), V(1), ...
                    const bool two = nq == 2;
                    ok = scores(0, 0, g, true, !two, nothing) && (!two || scores(1, 1, g, false, true, nothing));
                    g += S::KC;
                    for (int j = 0; ok && j < units; ++j, ++n) {
                        const bool more = j + 1 < units;
                        const uint32_t acc = j > 0 ? 1u : 0u;
                        if (!more)
                            mma_commit(smem_addr(&bars.q_empty));
                        auto second = [&] { return !two || weights_in(1, 1, n1, j == 0, mine1); };
                        ok = ready(g) && weights_in(0, 0, n, j == 0, mine) &&
                             product(0, 0, g, acc, true, !two, [&] { return more ? ready(g + S::VC) : second(); }) &&
                             finished(0, more) &&
                             (!more || scores(0, 0, g + S::VC, true, !two, second)) &&
                             (!two || (product(1, 1, g, acc, false, true, nothing) &&
                                       (!more || scores(1, 1, g + S::VC, false, true, nothing))));
                        if (!more && two)
                            mma_commit(smem_addr(&bars.o_last[1]));
                        g += S::VC + (more ? S::KC : 0);
                        n1 += two ? 1u : 0u;
                    }
                    mine1 += two ? 1u : 0u;
                }
                ++mine;
            }
            // Every product has finished before tensor memory is freed.
            mma_commit(smem_addr(&bars.drain));
            mbar_wait_bounded(smem_addr(&bars.drain), 0, 1024);
        }
    } else if (warp == 2) {
        // ------------------------------------- value rows of edge tiles
        uint32_t base = 0, par = 0; // stages before the piece; phase of each slot's edge barrier
        int piece = 0;
        bool ok = true;
        for (; ok; ++piece) {
            ok = __all_sync(0xFFFFFFFFu, take(piece));
            if (!ok)
                break;
            const Piece w = sh.piece[piece % kPieces];
            __syncwarp();
            if (lane == 0)
                done(piece);
            const int units = w.units;
            if (units == 0)
                break;
            for (int j = 0; ok && j < units; ++j) {
                const int x = w.u + j;
                if (!edge_unit<TREE>(a, w, x))
                    continue;
                const uint32_t gv = base + (uint32_t)(j * (S::KC + S::VC) + S::KC) +
                                    (S::PAIR && j + 1 < units ? S::KC : 0);
                for (int c = 0; ok && c < S::VC; ++c) {
                    const uint32_t slot = (gv + c) % S::NS;
                    // Classes of this stage's keys: key c * VKEYS + 32 h + lane in bits 2h, 2h + 1.
                    uint32_t cls = 0;
#pragma unroll
                    for (int h = 0; h < S::VKEYS / 32; ++h)
                        cls |= (uint32_t)key_class<TREE>(a, w, x, c * S::VKEYS + 32 * h + lane) << (2 * h);
                    // Units between that are no edges pass without this warp.
                    ok = __all_sync(0xFFFFFFFFu, wait(bars.edge[slot], (par >> slot) & 1, kWaitPiece));
                    if (!ok)
                        break;
                    par ^= 1u << slot;
                    const uint32_t vb = ring + slot * S::STAGE;
                    bool found = false;
#pragma unroll
                    for (int h = 0; h < S::VKEYS / 32; ++h) {
                        const uint32_t mine = (cls >> (2 * h)) & 3u;
                        const uint32_t some = __ballot_sync(0xFFFFFFFFu, mine == 1);
                        const uint32_t none = __ballot_sync(0xFFFFFFFFu, mine == 2);
                        // Four rows at a time, eight lanes of 16 bytes each per 64 dims.
#pragma unroll 1
                        for (int r4 = 0; r4 < 32; r4 += 4) {
                            if ((((some | none) >> r4) & 0xFu) == 0)
                                continue;
                            const int rr = r4 + (lane >> 3);
                            const uint32_t p = vb + (32 * h + rr) * 128 + (lane & 7) * 16;
                            if ((none >> rr) & 1u) {
#pragma unroll
                                for (int b = 0; b < S::DV / 64; ++b)
                                    sts128(p + b * (S::VKEYS * 128), make_uint4(0, 0, 0, 0));
                            } else if ((some >> rr) & 1u) {
                                uint4 v[S::DV / 64];
#pragma unroll
                                for (int b = 0; b < S::DV / 64; ++b)
                                    v[b] = lds128(p + b * (S::VKEYS * 128));
#pragma unroll
                                for (int b = 0; b < S::DV / 64; ++b) {
                                    uint32_t *e = reinterpret_cast<uint32_t *>(&v[b]);
                                    bool bad = false;
#pragma unroll
                                    for (int i = 0; i < 4; ++i) {
                                        const bool lo = (e[i] & 0x7F80u) == 0x7F80u;
                                        const bool hi = (e[i] & 0x7F800000u) == 0x7F800000u;
                                        e[i] &= (lo ? 0xFFFF0000u : 0xFFFFFFFFu) & (hi ? 0x0000FFFFu : 0xFFFFFFFFu);
                                        bad = bad || lo || hi;
                                    }
                                    if (bad) {
                                        found = true;
                                        sts128(p + b * (S::VKEYS * 128), v[b]);
                                    }
                                }
                            }
                        }
                    }
                    if (found)
                        sh.special[piece & 3] = piece;
                    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                    __syncwarp();
                    if (lane == 0)
                        mbar_arrive(smem_addr(&bars.full[slot]));
                }
            }
            base += (uint32_t)(units * (S::KC + S::VC));
        }
    } else if (warp >= 4) {
        // ------------------------------------------------------ softmax
        // Two row tiles: a thread has a row. One row tile: two threads (warps w and
        // w + 4) have a row, 64 keys and half of the accumulator's columns each.
        const int t = S::PAIR ? 0 : (warp - 4) >> 2; // MMA row tile
        const int half = S::PAIR ? (warp - 4) >> 2 : 0;
        const int wq = warp & 3;        // tensor-memory lanes 32 wq ..
        const int row = 32 * wq + lane; // row of the MMA tile
        const uint32_t lanes = (uint32_t)(32 * wq) << 16;
        const int tok_in = row / a.G, head = row - tok_in * a.G;
        constexpr int OC = S::PAIR ? S::DV / 2 : S::DV; // accumulator columns of this thread
        uint32_t it = 0, mine = 0, piece = 0; // units, pieces of this row tile; pieces of the run
        uint32_t xs = 0;            // exchanges so far
        bool ok = true;
        // The row's two threads exchange a value, and whether their waits ended well:
        // both leave at the same exchange, so neither is left at the barrier.
        auto exchange = [&](float mine) -> float {
            const int par = xs++ & 1;
            sh.x[par][half][row] = mine;
            if (lane == 0)
                sh.xok[par][warp - 4] = ok;
            named_sync(1 + wq, 64);
            ok = ok && sh.xok[par][(warp - 4) ^ 4];
            return sh.x[par][half ^ 1][row];
        };
        for (;; ++piece) {
            ok = __all_sync(0xFFFFFFFFu, take(piece));
            if (S::PAIR)
                exchange(0.f);
            if (!ok)
                break;
            const Piece &w = sh.piece[piece % kPieces];
            const int units = w.units;
            if (units == 0)
                break;
            if (t >= w.nq) {
                __syncwarp();
                if (lane == 0)
                    done(piece);
                continue;
            }
            const int tok = t * a.tpt + tok_in;
            const RowMask rm = row_mask<TREE>(a, w, tok, tok_in < a.tpt && tok < w.nt);
            float m = -INFINITY, l = 0.f;
            for (int j = 0; j < units; ++j, ++it) {
                const int x = w.u + j, kb = key0(w, x);
                const bool tr = tree_unit<TREE>(w, x);
                const uint32_t b = S::PAIR ? (it & 1) : (uint32_t)t;
                const uint32_t ph = S::PAIR ? (it >> 1) & 1 : it & 1;
                // Kept keys of this row, one bit each; `all`: the warp keeps every key.
                uint32_t km[4];
                bool all = false;
                if (TREE && tr) {
                    km[0] = (uint32_t)rm.nodes;
                    km[1] = (uint32_t)(rm.nodes >> 32);
                    km[2] = km[3] = 0;
                } else if (TREE && a.kpos) {
                    // Recorded positions: lane i holds keys i, 32 + i, ... A key is kept by
                    // all rows, by none, or by those whose window reaches back to it.
                    const int lo = rm.hi > 0 ? rm.lo : 0x7FFFFFFF; // rm.hi = 0: an absent node
#pragma unroll
                    for (int h = 0; h < 4; ++h) {
                        const int k = kb + 32 * h + lane;
                        const int p = k < a.T ? __ldg(a.kpos + (size_t)w.s * a.T + k) : -1;
                        const bool in = p >= 0 && p < w.off;
                        const bool every = in && (a.window <= 0 || (long long)p + a.window > (long long)w.off + a.N);
                        uint32_t some = __ballot_sync(0xFFFFFFFFu, in && !every);
                        km[h] = __ballot_sync(0xFFFFFFFFu, every);
                        if (lo == 0x7FFFFFFF)
                            km[h] = 0;
                        while (some) {
                            const int i = __ffs(some) - 1;
                            some &= some - 1;
                            if (__shfl_sync(0xFFFFFFFFu, p, i) >= lo)
                                km[h] |= 1u << i;
                        }
                    }
                } else {
                    const int lo = rm.lo - kb, hi = rm.hi - kb;
                    all = __all_sync(0xFFFFFFFFu, !rm.live || (lo <= 0 && hi >= kKeys));
#pragma unroll
                    for (int h = 0; h < 4; ++h)
                        km[h] = below(hi - 32 * h) & ~below(lo - 32 * h);
                }
                ok = ok && __all_sync(0xFFFFFFFFu, wait(bars.s_full[b], ph));
                if (!S::PAIR && !ok)
                    break;
                tc_fence_after();
                const uint32_t sa = s_col(b) + lanes;
                uint32_t v[64];
                auto mask = [&](uint32_t k0, uint32_t k1) {
                    if (!all) {
#pragma unroll
                        for (int i = 0; i < 64; ++i)
                            if (!(((i < 32 ? k0 : k1) >> (i & 31)) & 1u))
                                v[i] = 0xFF800000u;
                    }
                };
                auto most = [&]() {
                    float mx[4];
#pragma unroll
                    for (int q = 0; q < 4; ++q)
                        mx[q] = fmaxf(__uint_as_float(v[q]), __uint_as_float(v[q + 4]));
#pragma unroll
                    for (int i = 8; i < 64; i += 8)
#pragma unroll
                        for (int q = 0; q < 4; ++q)
                            mx[q] = fmaxf(mx[q], fmaxf(__uint_as_float(v[i + q]), __uint_as_float(v[i + q + 4])));
                    return fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
                };
                float mt;
                if (S::PAIR) {
                    W4_TLD64(v, sa + 64u * half);
                    mask(half ? km[2] : km[0], half ? km[3] : km[1]);
                    mt = most();
                    // Also: both halves have read their scores, P may go over them.
                    mt = fmaxf(mt, exchange(mt)) * a.c;
                    if (!ok)
                        break;
                } else {
                    // 64 registers at a time: the upper half is read for the maximum, the
                    // lower half for the maximum and its weights, then the upper half again
                    // (P goes over columns that were read).
                    W4_TLD64(v, sa + 64u);
                    mask(km[2], km[3]);
                    mt = most();
                    W4_TLD64(v, sa);
                    mask(km[0], km[1]);
                    mt = fmaxf(mt, most()) * a.c;
                }
                float alpha = 1.f;
                if (rm.live && mt > m + 8.f) { // also the first kept key (m = -inf)
                    alpha = ex2(m - mt);
                    l *= alpha;
                    m = mt;
                }
                if (j > 0 && __any_sync(0xFFFFFFFFu, alpha != 1.f)) {
                    // O holds the units before this one: wait for their product. (The last
                    // one's phase is told apart: these scores were issued after the
                    // product before it, and this unit's product waits for its weights.)
                    ok = __all_sync(0xFFFFFFFFu, wait(bars.o_done[t], (it - 1) & 1));
                    if (!S::PAIR && !ok)
                        break;
                    tc_fence_after();
#pragma unroll 1
                    for (int c0 = half * OC; c0 < half * OC + OC; c0 += 32) {
                        uint32_t o[32];
                        W4_TLD32(o, o_col(t) + lanes + c0);
#pragma unroll
                        for (int i = 0; i < 32; ++i)
                            o[i] = __float_as_uint(__uint_as_float(o[i]) * alpha);
                        W4_TST32(o, 0, o_col(t) + lanes + c0);
                    }
                }
                const float mm = m == -INFINITY ? 0.f : m;
                const unsigned long long cc = pack64(a.c, a.c), nm = pack64(-mm, -mm);
                unsigned long long sum[2] = {0ull, 0ull};
                auto weights = [&](uint32_t to) {
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        uint32_t pk[16];
#pragma unroll
                        for (int i = 0; i < 16; ++i) {
                            float p0, p1;
                            unpack64(fma2(pack64(__uint_as_float(v[32 * c + 2 * i]),
                                                 __uint_as_float(v[32 * c + 2 * i + 1])),
                                          cc, nm),
                                     p0, p1);
                            p0 = ex2(p0);
                            p1 = ex2(p1);
                            sum[i & 1] = add2(sum[i & 1], pack64(p0, p1));
                            pk[i] = pack2(p0, p1);
                        }
                        W4_TST16(pk, 0, to + 16u * c);
                    }
                };
                weights(sa + 32u * half);
                if (!S::PAIR) {
                    W4_TLD64(v, sa + 64u);
                    mask(km[2], km[3]);
                    weights(sa + 32u);
                }
                float s0, s1;
                unpack64(add2(sum[0], sum[1]), s0, s1);
                l += s0 + s1;
                tc_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0)
                    mbar_arrive(smem_addr(&bars.p_full[b]));
            }
            if (!S::PAIR && !ok)
                break;
            // ------------------------------------------------- epilogue
            ok = ok && __all_sync(0xFFFFFFFFu, wait(bars.o_last[t], mine & 1));
            ++mine;
            if (S::PAIR)
                l += exchange(l);
            if (!ok)
                break;
            tc_fence_after();
            const bool whole = w.whole(), special = sh.special[piece & 3] == (int)piece;
            const int kvh = w.hs / S::NV, dv0 = (w.hs % S::NV) * S::DV;
            uint16_t *orow = a.out + (size_t)((long long)w.q0 + w.t0 + tok) * a.ldo +
                             (size_t)(kvh * a.G + head) * D + dv0;
            const int slot = 2 * (int)blockIdx.x + (w.u == 0 ? 1 : 0);
            // Partial accumulators: [slot][DV / 4][ROWS] float4.
            float4 *prow = reinterpret_cast<float4 *>(a.ws_o + (size_t)slot * kSlotFloats) + t * kRowsQ + row;
            const float f = l == 0.f ? 0.f : 1.f / l; // nothing kept: zeros
            if (whole) {
                // Four lanes exchange their rows' 16-byte parts, so that a store writes
                // 64 contiguous bytes of a row (rows 4 g + i of lanes 4 g .. 4 g + 3).
                uint16_t *to[4];
                bool live[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int src = (lane & 28) + i;
                    to[i] = reinterpret_cast<uint16_t *>(__shfl_sync(0xFFFFFFFFu, (unsigned long long)orow, src)) +
                            8 * (lane & 3);
                    live[i] = __shfl_sync(0xFFFFFFFFu, (int)rm.live, src) != 0;
                }
#pragma unroll 2
                for (int c0 = half * OC; c0 < half * OC + OC; c0 += 32) {
                    uint32_t o[32];
                    W4_TLD32(o, o_col(t) + lanes + c0);
                    if (TREE && rm.absent()) {
#pragma unroll
                        for (int i = 0; i < 32; ++i)
                            o[i] = 0u;
                    }
                    uint4 y[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        y[i].x = pack2(__uint_as_float(o[8 * i]) * f, __uint_as_float(o[8 * i + 1]) * f);
                        y[i].y = pack2(__uint_as_float(o[8 * i + 2]) * f, __uint_as_float(o[8 * i + 3]) * f);
                        y[i].z = pack2(__uint_as_float(o[8 * i + 4]) * f, __uint_as_float(o[8 * i + 5]) * f);
                        y[i].w = pack2(__uint_as_float(o[8 * i + 6]) * f, __uint_as_float(o[8 * i + 7]) * f);
                    }
#pragma unroll
                    for (int d = 1; d <= 2; d <<= 1)
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            if (!(i & d))
                                swap4(y[i], y[i ^ d], d, (lane & d) != 0);
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        if (live[i])
                            *reinterpret_cast<uint4 *>(to[i] + c0) = y[i];
                }
            } else {
#pragma unroll 1
                for (int c0 = half * OC; c0 < half * OC + OC; c0 += 32) {
                    uint32_t o[32];
                    W4_TLD32(o, o_col(t) + lanes + c0);
                    if (TREE && rm.absent()) {
#pragma unroll
                        for (int i = 0; i < 32; ++i)
                            o[i] = 0u;
                    }
                    if (rm.live) {
#pragma unroll
                        for (int i = 0; i < 32; i += 4)
                            prow[(size_t)((c0 + i) / 4) * S::ROWS] =
                                make_float4(__uint_as_float(o[i]), __uint_as_float(o[i + 1]),
                                            __uint_as_float(o[i + 2]), __uint_as_float(o[i + 3]));
                    }
                    __syncwarp();
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0)
                mbar_arrive(smem_addr(&bars.o_free[t]));
            if (!whole && rm.live && half == 0) {
                float *ml = a.ws_ml + ((size_t)slot * 256 + t * kRowsQ + row) * 2;
                ml[0] = m;
                ml[1] = l;
            }
            if (special)
                __syncwarp(); // a row's output may come from its neighbour lanes
            if (special && rm.live)
                add_specials<D, TREE>(a, w, rm, kvh, dv0, half * OC, half * OC + OC, [&](int d, float f) {
                    if (whole) {
                        const float o = __uint_as_float((uint32_t)orow[d] << 16) + f;
                        orow[d] = (uint16_t)(pack2(o, 0.f) & 0xFFFFu);
                    } else {
                        reinterpret_cast<float *>(prow + (size_t)(d / 4) * S::ROWS)[d & 3] += f;
                    }
                });
            __syncwarp();
            if (lane == 0)
                done(piece);
        }
    } else if (lane == 0) {
        // ------------- warp 3: the run's pieces, and what the merge needs to know
        const int tt = a.tpt * S::TQ;
        int cont = 0, begins = 0;
        int tile = sh.cut[0][0], s = sh.cut[0][1], i = sh.cut[0][2], u = sh.cut[0][3];
        const int end = sh.cut[1][0], end_u = sh.cut[1][3];
        uint32_t piece = 0;
        bool ok = true;
        Seq q = {};
        if (tile < end || (tile == end && u < end_u))
            q = load_seq<TREE>(a, s);
        while (ok && (tile < end || (tile == end && u < end_u))) {
            Piece w;
            w.hs = tile / sh.tiles;
            w.s = s;
            w.t0 = i * tt;
            w.nt = min(tt, q.lq - w.t0);
            key_range<TREE>(a, q, w.t0, w.nt, w.lo, w.hi);
            w.n = tile_units<TREE>(w.lo, w.hi);
            w.u = u;
            w.u1 = tile == end ? end_u : w.n;
            w.units = w.u1 - w.u;
            w.q0 = q.q0;
            w.k0 = q.k0;
            w.lk = q.lk;
            w.off = q.off;
            w.nq = S::TQ == 1 ? 1 : (w.nt > a.tpt ? 2 : 1);
            if (piece >= (uint32_t)kPieces)
                ok = wait(bars.pc_empty[piece % kPieces], (piece / kPieces - 1) & 1, kWaitPiece);
            if (!ok)
                break;
            sh.piece[piece % kPieces] = w;
            mbar_arrive(smem_addr(&bars.pc_full[piece % kPieces]));
            ++piece;
            if (w.u > 0) {
                cont = 1 | (w.u1 == w.n ? 2 : 0);
            } else if (!w.whole()) {
                begins = 1;
                int32_t *p = a.where + 4 * blockIdx.x;
                p[0] = w.q0 + w.t0;
                p[1] = w.nt;
                p[2] = w.hs / S::NV;
                p[3] = w.hs % S::NV;
            }
            u = 0;
            ++i;
            if (++tile > end || (tile == end && end_u == 0))
                break;
            while (i * tt >= q.lq) { // ends: there is another row tile
                i = 0;
                s = s + 1 < a.B ? s + 1 : 0;
                q = load_seq<TREE>(a, s);
            }
        }
        if (ok && (piece < (uint32_t)kPieces ||
                   wait(bars.pc_empty[piece % kPieces], (piece / kPieces - 1) & 1, kWaitPiece))) {
            sh.piece[piece % kPieces].units = 0;
            mbar_arrive(smem_addr(&bars.pc_full[piece % kPieces]));
        }
        a.rec[2 * blockIdx.x] = cont;
        a.rec[2 * blockIdx.x + 1] = begins;
    }

    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512));
    }
}

} // namespace attn
} // namespace w4
