// Attention of one new token of each sequence over a paged cache.
//
// Source: "Gemma 4 E2B on a 4 GB GPU with pure PyTorch" - the decode-attention
// paragraph (each cached key and value is read once for all the query heads that share
// it, the cache split into slices joined by an online softmax), for several requests
// whose caches share one pool of pages.
//
// Mathematics as in attn_tiles.cuh: out = sum_t 2^(s_t - m) v_t / sum_t 2^(s_t - m), with m
// moved only when the maximum has grown by more than 2^8. A weight goes to the value
// product as two bf16 parts (within 2^-16 of it). Sums are fp32.
//
// Why not the tiles of attn_tiles.cuh: a row tile there has 128 rows, of which one token
// with its G heads fills G, and its scores, weights and product follow one another
// through tensor memory (4700 cycles for 128 keys of 128 dims: 4.1 TB/s). Here the keys
// are the rows of a warp's products and the heads the 8 columns:
//   - a tile is 16 keys with all their dims, which one page holds (pages are multiples
//     of 16 rows): one table entry per tile, read ahead. A warp streams its tiles through
//     a ring of its own (cp.async, zeros instead of rows that are not kept), so nothing
//     in the loop waits for another warp;
//   - scores K q^T: 16 keys x 8 heads per product; their weights, transposed by movmatrix,
//     are the second operand of V^T P, whose rows are 16 dims;
//   - a query has one row of keys for all its heads, so no key is kept by some rows of a
//     tile only: what is not kept is never read.
// Work: the tiles of all (sequence, key/value head) segments, in order, cut into equal
// runs, one per block; a block's warps take turns and join their sums at a segment's end.
// A segment that was cut leaves partial sums, which a second kernel joins in a fixed order.
// Where a window or a short table keeps segments to a few tiles a warp, runs are whole
// segments and the second kernel is left out; with fewer segments than SMs a cluster of
// blocks has each, whose sums are joined through distributed shared memory.
#include "attn_launch.cuh"

namespace w4 {
namespace attn {

namespace {

constexpr int kTile = 16;

// HT: groups of 8 heads.
template <int D, int HT>
struct StepShape {
    static constexpr int W = D <= 128 || (D == 256 && HT == 1) ? 8 : 4; // warps
    static constexpr int HALF = kTile * D * 2;   // keys (or values) of a tile: a copy
    static constexpr int HS = D + 4;             // floats between heads of the joined sums (no bank twice)
    static constexpr int HEADS = 8 * HT;
    static constexpr size_t JOIN = (size_t)(W / 2) * HEADS * (HS * 4 + 8);
    // Copies in a warp's ring: what shared memory holds (3 to 12).
    static constexpr int FIT = (int)((230400 - JOIN) / ((size_t)W * HALF));
    static constexpr int ST = FIT > 12 ? 12 : FIT;
    static constexpr int RING = ST * HALF;
    static constexpr size_t SMEM = (size_t)W * RING + JOIN;
    static_assert(ST >= 3 && SMEM <= 230400, "shared memory");
};

struct StepArgs {
    Args a;
    const uint16_t *q, *k;
    long long ldq;
    int whole; // runs of whole segments
    int cs;    // blocks of a cluster, which has one segment (whole; else 1)
};

// A run's place: a segment and its kept keys.
struct Walk {
    long long base; // the run's number of the segment's first tile
    int b, h, n;    // sequence, key/value head, tiles
    int t0;         // first tile's number within the sequence
    int lo, len;    // kept keys [lo, len)
};

__device__ __forceinline__ void keys_of(const Args &a, int b, int &lo, int &len, int &n)
{
    const int l = max(0, __ldg(a.lens + b));
    lo = a.window > 0 ? window_start(l - 1, a.window) : 0;
    len = min(l, a.most_k);
    lo = min(lo, len);
    n = max(1, (len + kTile - 1) / kTile - lo / kTile); // rows without keys are written
}

__device__ __forceinline__ void step_to(const Args &a, Walk &w, long long x)
{
    while (x >= w.base + w.n) {
        w.base += w.n;
        if (++w.h == a.Hkv) {
            w.h = 0;
            ++w.b;
            keys_of(a, w.b, w.lo, w.len, w.n);
            w.t0 = w.lo / kTile;
        }
    }
}

__device__ __forceinline__ float4 ld_cluster_f32x4(uint32_t a)
{
    float4 v;
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
                 : "r"(a)
                 : "memory");
    return v;
}

// Inclusive sum over a block of W warps; `total`: all of them. 64 bits: 32 sequences of
// 2^27 tiles pass 32.
template <int W>
__device__ __forceinline__ long long run_sum(long long x, long long *warp_sums, long long &total)
{
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const long long y = __shfl_up_sync(0xFFFFFFFFu, x, d);
        if (lane >= d)
            x += y;
    }
    __syncthreads();
    if (lane == 31)
        warp_sums[w] = x;
    __syncthreads();
    long long before = 0;
    total = 0;
#pragma unroll
    for (int i = 0; i < W; ++i) {
        before += i < w ? warp_sums[i] : 0;
        total += warp_sums[i];
    }
    return x + before;
}

__device__ __forceinline__ void copy16(uint32_t dst, const void *src, bool kept)
{
    asm volatile("cp.async.cg.shared.global.L2::256B [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(kept ? 16 : 0)
                 : "memory");
}

__device__ __forceinline__ void ldsm4(uint32_t addr, uint32_t (&r)[4])
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}

__device__ __forceinline__ void ldsm4_t(uint32_t addr, uint32_t (&r)[4])
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}

__device__ __forceinline__ uint32_t transposed(uint32_t v)
{
    uint32_t r;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
    return r;
}

__device__ __forceinline__ float bf_lo(uint32_t v) { return __uint_as_float(v << 16); }
__device__ __forceinline__ float bf_hi(uint32_t v) { return __uint_as_float(v & 0xFFFF0000u); }

template <int D, int HT>
__global__ void __launch_bounds__(StepShape<D, HT>::W * 32, 1)
step_kernel(const StepArgs p)
{
    using S = StepShape<D, HT>;
    constexpr int THREADS = S::W * 32, KS = D / 16, CH = D / 8; // 16-byte pieces of a row
    extern __shared__ __align__(128) unsigned char smem[];
    __shared__ long long s_base, s_run[4], s_scan[S::W];
    __shared__ int s_seq, s_h;
    const Args &a = p.a;
    const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5, g = lane >> 2, tq = lane & 3;
    const uint32_t ring = smem_addr(smem) + w * S::RING;
    float *join = reinterpret_cast<float *>(smem + (size_t)S::W * S::RING);
    float2 *join_ml = reinterpret_cast<float2 *>(join + (size_t)(S::W / 2) * S::HEADS * S::HS); // [W / 2][HEADS]
    pdl_launch_dependents();
    pdl_wait();

    // -------------------------------------------------- this block's run
    // Its tiles [x0, x1), of them the first's segment; for runs of whole segments counted from
    // the run's own first tile, else from the call's.
    // (Through shared memory, which leaves the registers to the sums.)
    long long x0 = 0, x1 = 0, tot = 0, blocks = 1;
    const long long segments = (long long)a.B * a.Hkv;
    if (p.whole) {
        const long long block = blockIdx.x / p.cs; // with clusters there are as many as segments
        blocks = min((long long)gridDim.x / p.cs, segments);
        const long long g0 = segments * min(block, blocks) / blocks;
        const long long g1 = segments * min(block + 1, blocks) / blocks;
        if (tid == 0) {
            s_seq = (int)(g0 / a.Hkv);
            s_h = (int)(g0 % a.Hkv);
            s_base = 0;
        }
        for (long long b = g0 / a.Hkv; b * a.Hkv < g1 && g0 < g1; ++b) {
            int lo, len, n;
            keys_of(a, (int)b, lo, len, n);
            x1 += n * (min(g1, (b + 1) * a.Hkv) - max(g0, b * a.Hkv));
        }
    } else {
        // Tiles of all sequences (of one head), then the sequence in which the run begins.
        long long all = 0;
        for (int b0 = 0; b0 < a.B; b0 += THREADS) {
            int lo, len, n = 0;
            if (b0 + tid < a.B)
                keys_of(a, b0 + tid, lo, len, n);
            long long total;
            run_sum<S::W>(n, s_scan, total);
            all += total;
        }
        tot = all * a.Hkv;
        // Runs of a tile for each warp of a block, or a segment's worth, at least. (5 tokens of 4
        // positions at D = 512 in one block's run: 28 us.)
        blocks = min((long long)gridDim.x, max(tot / S::W, segments));
        x0 = tot * min((long long)blockIdx.x, blocks) / blocks;
        x1 = tot * min((long long)blockIdx.x + 1, blocks) / blocks;
        long long before = 0;
        for (int b0 = 0; b0 < a.B; b0 += THREADS) {
            int lo, len, n = 0;
            if (b0 + tid < a.B)
                keys_of(a, b0 + tid, lo, len, n);
            long long total;
            const long long incl = before + run_sum<S::W>(n, s_scan, total);
            const long long first = (incl - n) * a.Hkv; // of this sequence
            if (n > 0 && x0 >= first && x0 < incl * a.Hkv) {
                s_seq = b0 + tid;
                s_h = (int)((x0 - first) / n);
                s_base = first + (long long)s_h * n;
            }
            before += total;
            if (before * a.Hkv > x0)
                break;
        }
    }
    if (tid == 0) {
        s_run[0] = x0;
        s_run[1] = x1;
        s_run[2] = tot;
        s_run[3] = blocks;
    }
    __syncthreads();
    x0 = s_run[0];
    x1 = s_run[1];
    int begins = 0, begins_b = 0, begins_h = 0; // parts of the cut segment that this run begins, if any
    if (x0 < x1) {
        Walk c;
        c.b = s_seq;
        c.h = s_h;
        c.base = s_base;
        keys_of(a, c.b, c.lo, c.len, c.n);
        c.t0 = c.lo / kTile;
        Walk f = c; // what is copied next
        const int mine = (int)(blockIdx.x % p.cs) * S::W + w, hop = S::W * p.cs; // this warp's tiles
        long long xf = x0 + mine;

        // The next tile's page, a tile ahead of its copies.
        auto page_of = [&]() {
            int pg = -1;
            if (xf < x1) {
                step_to(a, f, xf);
                const int key = (f.t0 + (int)(xf - f.base)) * kTile;
                if (key < f.len)
                    pg = __ldg(a.table + (size_t)f.b * a.table_pages + (key >> a.page_log2));
            }
            return pg;
        };
        int pg = page_of();
        uint32_t paged = 0;   // whether the tiles copied last have a page, the newest in bit 0
        size_t at = 0;        // the tile being copied: its first row, its kept rows
        int r0 = 0, r1 = 0;
        auto rows = [&](const uint16_t *p, int slot) {
            const uint32_t to = ring + slot * S::HALF;
#pragma unroll
            for (int i = 0; i < kTile * CH / 32; ++i) {
                const int e = lane + 32 * i, r = e / CH, j = e - r * CH;
                const bool kept = r >= r0 && r < r1;
                copy16(to + r * (D * 2) + ((j ^ (r & 7)) << 4), p + at + (kept ? (size_t)r * a.row_stride : 0) + 8 * j,
                       kept);
            }
            asm volatile("cp.async.commit_group;" ::: "memory");
        };
        bool copying = false;
        // Keys of tile xf, then its values.
        auto issue_keys = [&](int slot) {
            paged <<= 1;
            copying = xf < x1;
            if (copying) {
                const int key = (f.t0 + (int)(xf - f.base)) * kTile;
                const bool have = pg >= 0 && pg < a.pages;
                paged |= have ? 1u : 0u;
                r0 = have ? f.lo - key : kTile;
                r1 = have ? f.len - key : 0;
                at = (size_t)(have ? pg : 0) * a.page_stride +
                     (size_t)(key & ((1 << a.page_log2) - 1)) * a.row_stride + (size_t)f.h * a.head_stride;
                rows(p.k, slot);
                xf += hop;
                pg = page_of();
            } else {
                asm volatile("cp.async.commit_group;" ::: "memory");
            }
        };
        auto issue_values = [&](int slot) {
            if (copying)
                rows(a.v, slot);
            else
                asm volatile("cp.async.commit_group;" ::: "memory");
        };
#pragma unroll
        for (int i = 0; i < S::ST - 1; ++i)
            (i & 1) ? issue_values(i) : issue_keys(i);
        // Copy number n + ST - 1 while copy n is worked on: the same half when ST is odd.
        auto ahead = [&](bool keys, int slot) {
            const int to = slot == 0 ? S::ST - 1 : slot - 1;
            if (keys == (S::ST % 2 == 1))
                issue_keys(to);
            else
                issue_values(to);
            asm volatile("cp.async.wait_group %0;" ::"n"(S::ST - 1) : "memory");
            __syncwarp(); // every lane's copies are in place
        };

        int slot = 0;
        long long x = x0 + mine;
        for (long long xs = x0; xs < x1;) { // segments
            step_to(a, c, xs);
            const long long end = min(x1, c.base + c.n);
            // The heads that share this key/value head: columns of the score product.
            uint32_t qb[HT][KS][2];
#pragma unroll
            for (int t = 0; t < HT; ++t) {
                const bool ok = 8 * t + g < a.G;
                const uint16_t *qp = p.q + (size_t)c.b * p.ldq + (size_t)(c.h * a.G + 8 * t + (ok ? g : 0)) * D + 2 * tq;
#pragma unroll
                for (int s = 0; s < KS; ++s) {
                    qb[t][s][0] = ok ? __ldg(reinterpret_cast<const uint32_t *>(qp + 16 * s)) : 0u;
                    qb[t][s][1] = ok ? __ldg(reinterpret_cast<const uint32_t *>(qp + 16 * s + 8)) : 0u;
                }
            }
            float o[HT][KS][4];
            float m[HT][2], l[HT][2]; // heads 8 t + 2 tq (+ 1): reference (log2 units), this lane's part of the sum
#pragma unroll
            for (int t = 0; t < HT; ++t) {
                m[t][0] = m[t][1] = -INFINITY;
                l[t][0] = l[t][1] = 0.f;
#pragma unroll
                for (int s = 0; s < KS; ++s)
                    o[t][s][0] = o[t][s][1] = o[t][s][2] = o[t][s][3] = 0.f;
            }
#pragma unroll 1
            for (; x < end; x += hop) {
                ahead(true, slot);
                const uint32_t kb = ring + slot * S::HALF;
                slot = slot == S::ST - 1 ? 0 : slot + 1;
                float sc[HT][2][4];
#pragma unroll
                for (int t = 0; t < HT; ++t)
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        sc[t][0][i] = sc[t][1][i] = 0.f;
                {
                    const int row = ((lane >> 3) & 1) * 8 + (lane & 7), up = lane >> 4;
                    const uint32_t ra = kb + row * (D * 2);
#pragma unroll
                    for (int s = 0; s < KS; ++s) {
                        uint32_t r[4];
                        ldsm4(ra + (((2 * s + up) ^ (row & 7)) << 4), r);
#pragma unroll
                        for (int t = 0; t < HT; ++t)
                            mma_16816(sc[t][s & 1], r[0], r[1], r[2], r[3], qb[t][s][0], qb[t][s][1]);
                    }
                }
                // Kept keys: rows g and g + 8 of the tile. A page that is none left zeros.
                const int key = (c.t0 + (int)(x - c.base)) * kTile;
                const bool have = (paged >> ((S::ST - 1) / 2)) & 1u;
                const bool k0 = have && key + g >= c.lo && key + g < c.len;
                const bool k1 = have && key + g + 8 >= c.lo && key + g + 8 < c.len;
                uint32_t hi[HT][2], lw[HT][2];
                bool moved = false;
                float al[HT][2];
#pragma unroll
                for (int t = 0; t < HT; ++t) {
                    float v[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        v[i] = (i < 2 ? k0 : k1) ? (sc[t][0][i] + sc[t][1][i]) * a.c : -INFINITY;
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        float mt = fmaxf(v[i], v[i + 2]);
                        mt = fmaxf(mt, __shfl_xor_sync(0xFFFFFFFFu, mt, 4));
                        mt = fmaxf(mt, __shfl_xor_sync(0xFFFFFFFFu, mt, 8));
                        mt = fmaxf(mt, __shfl_xor_sync(0xFFFFFFFFu, mt, 16));
                        al[t][i] = 1.f;
                        if (mt > m[t][i] + 8.f) { // also the first kept key (m = -inf)
                            al[t][i] = ex2(m[t][i] - mt);
                            m[t][i] = mt;
                            moved = true;
                        }
                        const float mm = m[t][i] == -INFINITY ? 0.f : m[t][i];
                        v[i] = ex2(v[i] - mm);
                        v[i + 2] = ex2(v[i + 2] - mm);
                        l[t][i] = l[t][i] * al[t][i] + (v[i] + v[i + 2]);
                    }
                    const uint32_t h0 = pack2(v[0], v[1]), h1 = pack2(v[2], v[3]);
                    hi[t][0] = transposed(h0);
                    hi[t][1] = transposed(h1);
                    lw[t][0] = transposed(pack2(v[0] - bf_lo(h0), v[1] - bf_hi(h0)));
                    lw[t][1] = transposed(pack2(v[2] - bf_lo(h1), v[3] - bf_hi(h1)));
                }
                if (__any_sync(0xFFFFFFFFu, moved)) {
#pragma unroll
                    for (int t = 0; t < HT; ++t)
#pragma unroll
                        for (int s = 0; s < KS; ++s) {
                            o[t][s][0] *= al[t][0];
                            o[t][s][1] *= al[t][1];
                            o[t][s][2] *= al[t][0];
                            o[t][s][3] *= al[t][1];
                        }
                }
                __syncwarp(); // all lanes have read the keys, whose slot the next copies go to
                ahead(false, slot);
                {
                    const int row = (lane >> 4) * 8 + (lane & 7), up = (lane >> 3) & 1;
                    const uint32_t ra = ring + slot * S::HALF + row * (D * 2);
                    slot = slot == S::ST - 1 ? 0 : slot + 1;
#pragma unroll
                    for (int s = 0; s < KS; ++s) {
                        uint32_t r[4];
                        ldsm4_t(ra + (((2 * s + up) ^ (row & 7)) << 4), r);
#pragma unroll
                        for (int t = 0; t < HT; ++t) {
                            mma_16816(o[t][s], r[0], r[1], r[2], r[3], hi[t][0], hi[t][1]);
                            mma_16816(o[t][s], r[0], r[1], r[2], r[3], lw[t][0], lw[t][1]);
                        }
                    }
                }
                __syncwarp(); // and the values
            }
            // ------------------------------------- the warps' sums joined
            // The upper half of the warps leave theirs, the lower half add them and leave the sums.
#pragma unroll
            for (int t = 0; t < HT; ++t)
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    l[t][i] += __shfl_xor_sync(0xFFFFFFFFu, l[t][i], 4);
                    l[t][i] += __shfl_xor_sync(0xFFFFFFFFu, l[t][i], 8);
                    l[t][i] += __shfl_xor_sync(0xFFFFFFFFu, l[t][i], 16);
                }
            const int u = w & (S::W / 2 - 1);
            float *own = join + (size_t)(u * S::HEADS + 2 * tq) * S::HS + g;
            auto leave = [&]() {
#pragma unroll
                for (int t = 0; t < HT; ++t) {
                    float *to = own + (size_t)8 * t * S::HS;
#pragma unroll
                    for (int s = 0; s < KS; ++s) {
                        to[16 * s] = o[t][s][0];
                        to[16 * s + S::HS] = o[t][s][1];
                        to[16 * s + 8] = o[t][s][2];
                        to[16 * s + 8 + S::HS] = o[t][s][3];
                    }
                    if (g == 0) {
                        join_ml[u * S::HEADS + 8 * t + 2 * tq] = make_float2(m[t][0], l[t][0]);
                        join_ml[u * S::HEADS + 8 * t + 2 * tq + 1] = make_float2(m[t][1], l[t][1]);
                    }
                }
            };
            if (w >= S::W / 2)
                leave();
            __syncthreads();
            if (w < S::W / 2) {
#pragma unroll
                for (int t = 0; t < HT; ++t) {
                    const float *from = own + (size_t)8 * t * S::HS;
                    float fa[2], fb[2];
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const float2 ml = join_ml[u * S::HEADS + 8 * t + 2 * tq + i];
                        const float M = fmaxf(m[t][i], ml.x);
                        fa[i] = m[t][i] == -INFINITY ? 0.f : ex2(m[t][i] - M);
                        fb[i] = ml.x == -INFINITY ? 0.f : ex2(ml.x - M);
                        m[t][i] = M;
                        l[t][i] = l[t][i] * fa[i] + ml.y * fb[i];
                    }
#pragma unroll
                    for (int s = 0; s < KS; ++s) {
                        o[t][s][0] = o[t][s][0] * fa[0] + from[16 * s] * fb[0];
                        o[t][s][1] = o[t][s][1] * fa[1] + from[16 * s + S::HS] * fb[1];
                        o[t][s][2] = o[t][s][2] * fa[0] + from[16 * s + 8] * fb[0];
                        o[t][s][3] = o[t][s][3] * fa[1] + from[16 * s + 8 + S::HS] * fb[1];
                    }
                }
                __syncwarp(); // the lanes' heads' sums have been read
                leave();
            }
            __syncthreads();
            const bool first = xs == c.base, last = end == c.base + c.n, whole = first && last;
            const int part = 2 * (int)blockIdx.x + (first ? 1 : 0);
            for (int e = tid; e < a.G * (D / 4); e += THREADS) {
                const int h = e / (D / 4), d4 = e - h * (D / 4);
                float M = -INFINITY;
#pragma unroll
                for (int v = 0; v < S::W / 2; ++v)
                    M = fmaxf(M, join_ml[v * S::HEADS + h].x);
                float L = 0.f;
                float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
                for (int v = 0; v < S::W / 2; ++v) {
                    const float2 ml = join_ml[v * S::HEADS + h];
                    const float fu = ml.x == -INFINITY ? 0.f : ex2(ml.x - M);
                    const float4 z = *reinterpret_cast<const float4 *>(join + (size_t)(v * S::HEADS + h) * S::HS + 4 * d4);
                    L = fmaf(fu, ml.y, L);
                    y.x = fmaf(fu, z.x, y.x);
                    y.y = fmaf(fu, z.y, y.y);
                    y.z = fmaf(fu, z.z, y.z);
                    y.w = fmaf(fu, z.w, y.w);
                }
                if (p.cs > 1) {
                    // The ring is done with: a cluster's block has one segment.
                    *reinterpret_cast<float4 *>(smem + ((size_t)h * D + 4 * d4) * 4) = y;
                    if (d4 == 0)
                        reinterpret_cast<float2 *>(smem + (size_t)S::HEADS * D * 4)[h] = make_float2(M, L);
                } else if (whole) {
                    const float inv = L == 0.f ? 0.f : 1.f / L; // nothing kept: zeros
                    uint2 b;
                    b.x = pack2(y.x * inv, y.y * inv);
                    b.y = pack2(y.z * inv, y.w * inv);
                    *reinterpret_cast<uint2 *>(a.out + (size_t)c.b * a.ldo + (size_t)(c.h * a.G + h) * D + 4 * d4) = b;
                } else {
                    *reinterpret_cast<float4 *>(a.ws_o + (size_t)part * kSlotFloats + (size_t)h * D + 4 * d4) = y;
                    if (d4 == 0)
                        *reinterpret_cast<float2 *>(a.ws_ml + ((size_t)part * 256 + h) * 2) = make_float2(M, L);
                }
            }
            if (p.cs > 1) {
                cluster_sync();
                const uint32_t sums = smem_addr(smem), mls = sums + S::HEADS * D * 4;
                for (int e = (int)(blockIdx.x % p.cs) * THREADS + tid; e < a.G * (D / 4); e += THREADS * p.cs) {
                    const int h = e / (D / 4), d4 = e - h * (D / 4);
                    float M = -INFINITY, L = 0.f;
                    for (int k = 0; k < p.cs; ++k)
                        M = fmaxf(M, ld_cluster_f32(map_rank(mls + 8 * h, k)));
                    float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
                    for (int k = 0; k < p.cs; ++k) {
                        const uint32_t ml = map_rank(mls + 8 * h, k);
                        const float m = ld_cluster_f32(ml), f = m == -INFINITY ? 0.f : ex2(m - M);
                        const float4 z = ld_cluster_f32x4(map_rank(sums + (h * D + 4 * d4) * 4, k));
                        L = fmaf(f, ld_cluster_f32(ml + 4), L);
                        y.x = fmaf(f, z.x, y.x);
                        y.y = fmaf(f, z.y, y.y);
                        y.z = fmaf(f, z.z, y.z);
                        y.w = fmaf(f, z.w, y.w);
                    }
                    const float inv = L == 0.f ? 0.f : 1.f / L;
                    uint2 b;
                    b.x = pack2(y.x * inv, y.y * inv);
                    b.y = pack2(y.z * inv, y.w * inv);
                    *reinterpret_cast<uint2 *>(a.out + (size_t)c.b * a.ldo + (size_t)(c.h * a.G + h) * D + 4 * d4) = b;
                }
                cluster_sync(); // this block's sums have been read
            }
            if (!whole && first) {
                // The block that has the segment's last tile: the largest one whose run begins at or before it.
                begins = (int)(((c.base + c.n) * s_run[3] - 1) / s_run[2]) - (int)blockIdx.x + 1;
                begins_b = c.b;
                begins_h = c.h;
            }
            xs = end;
            if (xs < x1)
                __syncthreads(); // the joined sums have been read
        }
        asm volatile("cp.async.wait_group 0;" ::: "memory");
    }
    if (tid == 0)
        *reinterpret_cast<int4 *>(a.rec + 4 * blockIdx.x) = make_int4(begins, begins_b, begins_h, 0);
}

// Joins the parts of the cut segments: part p of one that block c begins is slot 2 c + 1 for p = 0,
// else 2 (c + p). Block (x, y): the x-th cut segment, one head, 128 of its dims; 8 threads share a
// float4, each with every eighth part, added in the order of the threads.
constexpr int kJoinThreads = 256;

__global__ void __launch_bounds__(kJoinThreads)
step_join_kernel(const Args a, int blocks)
{
    constexpr int NW = kJoinThreads / 32, BATCH = 8;
    __shared__ int s_warp[NW], s_pick[4];
    __shared__ float s_max[NW], s_sum[NW], s_f[kJoinThreads];
    __shared__ float4 s_y[NW][32];
    pdl_wait();
    const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5;
    int4 rec = tid < blocks ? __ldcg(reinterpret_cast<const int4 *>(a.rec + 4 * tid)) : make_int4(0, 0, 0, 0);
    const uint32_t v = __ballot_sync(0xFFFFFFFFu, rec.x > 0);
    if (lane == 0)
        s_warp[w] = __popc(v);
    if (tid == 0)
        s_pick[0] = 0;
    __syncthreads();
    int before = __popc(v & ((1u << lane) - 1u));
    for (int i = 0; i < NW; ++i)
        before += i < w ? s_warp[i] : 0;
    if (rec.x > 0 && before == (int)blockIdx.x) {
        s_pick[0] = rec.x;
        s_pick[1] = tid;
        s_pick[2] = rec.y;
        s_pick[3] = rec.z;
    }
    __syncthreads();
    const int n = s_pick[0], c = s_pick[1];
    if (n == 0)
        return;
    const int per = (a.D + 127) / 128, h = (int)blockIdx.y / per, d = ((int)blockIdx.y % per) * 128 + 4 * lane;
    auto slot = [&](int p) { return (size_t)(p == 0 ? 2 * c + 1 : 2 * (c + p)); };
    auto load = [&](int p) {
        return p < n && d < a.D ? __ldcg(reinterpret_cast<const float4 *>(a.ws_o + slot(p) * kSlotFloats + (size_t)h * a.D + d))
                                : make_float4(0.f, 0.f, 0.f, 0.f);
    };
    float4 x[BATCH]; // the first parts are asked for before the weights
#pragma unroll
    for (int q = 0; q < BATCH; ++q)
        x[q] = load(w + q * NW);
    const float2 ml = tid < n ? __ldcg(reinterpret_cast<const float2 *>(a.ws_ml + (slot(tid) * 256 + h) * 2))
                              : make_float2(-INFINITY, 0.f);
    float M = ml.x;
#pragma unroll
    for (int k = 16; k; k >>= 1)
        M = fmaxf(M, __shfl_xor_sync(0xFFFFFFFFu, M, k));
    if (lane == 0)
        s_max[w] = M;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < NW; ++i)
        M = fmaxf(M, s_max[i]);
    const float f = ml.x == -INFINITY ? 0.f : ex2(ml.x - M);
    s_f[tid] = f;
    float L = f * ml.y;
#pragma unroll
    for (int k = 16; k; k >>= 1)
        L += __shfl_xor_sync(0xFFFFFFFFu, L, k);
    if (lane == 0)
        s_sum[w] = L;
    __syncthreads();
    float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int p0 = w;; p0 += BATCH * NW) {
#pragma unroll
        for (int q = 0; q < BATCH; ++q) {
            const int p = p0 + q * NW;
            const float e = p < n ? s_f[p] : 0.f;
            y.x = fmaf(x[q].x, e, y.x);
            y.y = fmaf(x[q].y, e, y.y);
            y.z = fmaf(x[q].z, e, y.z);
            y.w = fmaf(x[q].w, e, y.w);
        }
        if (p0 + BATCH * NW >= n)
            break;
#pragma unroll
        for (int q = 0; q < BATCH; ++q)
            x[q] = load(p0 + (BATCH + q) * NW);
    }
    s_y[w][lane] = y;
    __syncthreads();
    if (w == 0 && d < a.D) {
        L = 0.f;
#pragma unroll
        for (int i = 0; i < NW; ++i)
            L += s_sum[i];
#pragma unroll
        for (int i = 1; i < NW; ++i) {
            const float4 z = s_y[i][lane];
            y.x += z.x;
            y.y += z.y;
            y.z += z.z;
            y.w += z.w;
        }
        const float inv = L == 0.f ? 0.f : 1.f / L;
        uint2 b;
        b.x = pack2(y.x * inv, y.y * inv);
        b.y = pack2(y.z * inv, y.w * inv);
        *reinterpret_cast<uint2 *>(a.out + (size_t)s_pick[2] * a.ldo + (size_t)(s_pick[3] * a.G + h) * a.D + d) = b;
    }
}

template <int D, int HT>
cudaError_t launch_step(const StepArgs &p0, float *ws, int num_sms, cudaStream_t s)
{
    using S = StepShape<D, HT>;
    if (num_sms > kJoinThreads) // the join has a thread for each block's record and part
        return cudaErrorInvalidValue;
    StepArgs p = p0;
    set_scratch(p.a, ws, num_sms);
    // Keys of a segment at most, in tiles (a window may begin and end within one). Windows of 512, 8 heads,
    // D = 256, one block a segment (5 tiles a warp): 3 tokens 10.4 us whole and 9.8 cut and joined, 61 on two
    // heads of 128 8.3 and 14.4, 152 tokens 11.5 and 27. At D = 512 a tile takes a warp twice as long.
    const long long keys = p.a.window > 0 && p.a.window < p.a.most_k ? p.a.window : p.a.most_k;
    const long long tiles = (keys + kTile - 1) / kTile + 1, segments = (long long)p.a.B * p.a.Hkv;
    // Clusters while they take no more than three quarters of the SMs (the rest of a GPC may not hold one) and
    // every warp may have a tile: 3 tokens 8.7 us in clusters of 4, 10.4 in single blocks; one 8.3 and 10.3;
    // 2 of 6 heads on 2 of 384 on tables of 256 keys 7.5 and 14.3 (cut); one on a table of 3000 10.9 and 10.2 (cut).
    p.cs = 1;
    while (p.cs < 8 && segments * p.cs * 2 <= num_sms * 3 / 4 && (long long)S::W * p.cs * 2 <= tiles)
        p.cs *= 2;
    p.whole = tiles <= (D <= 256 ? 6ll : 3ll) * S::W * p.cs;
    if (!p.whole)
        p.cs = 1;
    static std::atomic<unsigned long long> set{0};
    cudaError_t e = allow_smem(step_kernel<D, HT>, S::SMEM, set);
    if (e != cudaSuccess)
        return e;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)p.cs;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(p.cs > 1 ? segments * p.cs : num_sms));
    cfg.blockDim = dim3(S::W * 32);
    cfg.dynamicSmemBytes = S::SMEM;
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = p.cs > 1 ? 2 : 1;
    e = cudaLaunchKernelEx(&cfg, step_kernel<D, HT>, p);
    if (e != cudaSuccess || p.whole)
        return e;
    cfg.gridDim = dim3((unsigned)(segments < num_sms ? segments : num_sms), (unsigned)(p.a.G * ((D + 127) / 128)));
    cfg.numAttrs = 1;
    cfg.blockDim = dim3(kJoinThreads);
    cfg.dynamicSmemBytes = 0;
    return cudaLaunchKernelEx(&cfg, step_join_kernel, p.a, num_sms);
}

} // namespace

} // namespace attn

bool step_serves(int G, int D) { return G <= 8 || (G <= 16 && D <= 256); }

cudaError_t run_attn_step(const AttnPagedArgs &p, float *ws, int num_sms, cudaStream_t s)
{
    attn::StepArgs t = {};
    t.a = attn::paged_args(p);
    t.q = p.q;
    t.k = p.k_pages;
    t.ldq = p.ldq;
    const bool one = t.a.G <= 8;
    switch (p.D) {
    case 64: return one ? attn::launch_step<64, 1>(t, ws, num_sms, s) : attn::launch_step<64, 2>(t, ws, num_sms, s);
    case 128: return one ? attn::launch_step<128, 1>(t, ws, num_sms, s) : attn::launch_step<128, 2>(t, ws, num_sms, s);
    case 256: return one ? attn::launch_step<256, 1>(t, ws, num_sms, s) : attn::launch_step<256, 2>(t, ws, num_sms, s);
    case 384: return attn::launch_step<384, 1>(t, ws, num_sms, s);
    case 512: return attn::launch_step<512, 1>(t, ws, num_sms, s);
    default: return cudaErrorNotSupported;
    }
}

} // namespace w4
