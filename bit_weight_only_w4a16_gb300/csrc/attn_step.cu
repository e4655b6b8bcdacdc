// Attention of one new token of each sequence over a paged cache.
//
// Source: "Gemma 4 E2B on a 4 GB GPU with pure PyTorch" - the decode-attention
// paragraph (each cached key and value is read once for all the query heads that share
// it, the cache split into slices joined by an online softmax), for several requests
// whose caches share one pool of pages.
//
// Mathematics as in attn_tiles.cuh: out = sum_t 2^(s_t - m) v_t / sum_t 2^(s_t - m), with m
// moved only when the maximum has grown by more than 2^8. A weight goes to the value
// product as two bf16 parts (within 2^-17 of it). Sums are fp32.
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
// A segment that was cut leaves partial sums, merged in key order by attn_merge.cu.
#include "attn_launch.cuh"

namespace w4 {
namespace attn {

namespace {

constexpr int kTile = 16;

// HT: groups of 8 heads.
template <int D, int HT>
struct StepShape {
    static constexpr int W = D <= 128 ? 8 : (D == 256 ? 4 : 2);                     // warps
    static constexpr int ST = HT == 2 ? (D == 64 ? 4 : 2) : (D == 64 ? 6 : (D == 384 ? 4 : 3)); // tiles of a warp's ring
    static constexpr int HALF = kTile * D * 2;   // keys (or values) of a tile
    static constexpr int RING = ST * 2 * HALF;   // of a warp
    static constexpr int HS = D + 4;             // floats between heads of the joined sums (no bank twice)
    static constexpr int HEADS = 8 * HT;
    static constexpr size_t JOIN = (size_t)W * HEADS * HS * 4;
    static constexpr size_t SMEM = (size_t)W * RING + JOIN + (size_t)W * HEADS * 8;
    static_assert(SMEM <= 232448 - 1024, "shared memory");
};

struct StepArgs {
    Args a;
    const uint16_t *q, *k;
    long long ldq;
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
    __shared__ long long s_base, s_scan[S::W];
    __shared__ int s_seq, s_h;
    const Args &a = p.a;
    const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5, g = lane >> 2, tq = lane & 3;
    const uint32_t ring = smem_addr(smem) + w * S::RING;
    float *join = reinterpret_cast<float *>(smem + (size_t)S::W * S::RING);
    float2 *join_ml = reinterpret_cast<float2 *>(smem + (size_t)S::W * S::RING + S::JOIN); // [W][HEADS]
    pdl_launch_dependents();
    pdl_wait();

    // -------------------------------------------------- this block's run
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
    const long long tot = all * a.Hkv;
    // A tile for each warp of a block at least.
    const long long blocks = max(1ll, min((long long)gridDim.x, tot / S::W));
    const long long x0 = tot * min((long long)blockIdx.x, blocks) / blocks;
    const long long x1 = tot * min((long long)blockIdx.x + 1, blocks) / blocks;
    long long before = 0;
    for (int b0 = 0; b0 < a.B; b0 += THREADS) {
        int lo, len, n = 0;
        if (b0 + tid < a.B)
            keys_of(a, b0 + tid, lo, len, n);
        long long total;
        const long long incl = before + run_sum<S::W>(n, s_scan, total);
        if (n > 0 && x0 < incl * a.Hkv && x0 >= (incl - n) * a.Hkv) {
            s_seq = b0 + tid;
            s_h = (int)((x0 - (incl - n) * a.Hkv) / n);
            s_base = (incl - n) * a.Hkv + (long long)s_h * n;
        }
        before += total;
        if (before * a.Hkv > x0)
            break;
    }
    __syncthreads();
    int cont = 0, begins = 0; // as in attn_tiles.cuh
    if (x0 < x1) {
        Walk c;
        c.b = s_seq;
        c.h = s_h;
        c.base = s_base;
        keys_of(a, c.b, c.lo, c.len, c.n);
        c.t0 = c.lo / kTile;
        Walk f = c; // what is copied next
        long long xf = x0 + w;

        // Tile xf into ring slot `slot`, then on to the warp's next tile.
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
        uint32_t paged = 0; // whether the tiles copied last have a page, the newest in bit 0
        auto issue = [&](int slot) {
            paged <<= 1;
            if (xf < x1) {
                const int key = (f.t0 + (int)(xf - f.base)) * kTile;
                const bool have = pg >= 0 && pg < a.pages;
                paged |= have ? 1u : 0u;
                const int r0 = have ? f.lo - key : kTile, r1 = have ? f.len - key : 0; // kept rows
                const size_t at = (size_t)(have ? pg : 0) * a.page_stride +
                                  (size_t)(key & ((1 << a.page_log2) - 1)) * a.row_stride + (size_t)f.h * a.head_stride;
                const uint32_t to = ring + slot * 2 * S::HALF;
#pragma unroll
                for (int i = 0; i < kTile * CH / 32; ++i) {
                    const int e = lane + 32 * i, r = e / CH, j = e - r * CH;
                    const bool kept = r >= r0 && r < r1;
                    const size_t from = at + (kept ? (size_t)r * a.row_stride : 0) + 8 * j;
                    const uint32_t so = to + r * (D * 2) + ((j ^ (r & 7)) << 4);
                    copy16(so, p.k + from, kept);
                    copy16(so + S::HALF, a.v + from, kept);
                }
                xf += S::W;
                pg = page_of();
            }
            asm volatile("cp.async.commit_group;" ::: "memory");
        };
#pragma unroll
        for (int i = 0; i < S::ST - 1; ++i)
            issue(i);

        int slot = 0;
        long long x = x0 + w;
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
            for (; x < end; x += S::W) {
                issue(slot == 0 ? S::ST - 1 : slot - 1);
                asm volatile("cp.async.wait_group %0;" ::"n"(S::ST - 1) : "memory");
                __syncwarp(); // every lane's copies of the tile are in place
                const uint32_t kb = ring + slot * 2 * S::HALF, vb = kb + S::HALF;
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
                const bool have = (paged >> (S::ST - 1)) & 1u;
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
                {
                    const int row = (lane >> 4) * 8 + (lane & 7), up = (lane >> 3) & 1;
                    const uint32_t ra = vb + row * (D * 2);
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
                __syncwarp(); // all lanes have read the slot that the next copies go to
            }
            // ------------------------------------- the warps' sums joined
#pragma unroll
            for (int t = 0; t < HT; ++t) {
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    float s = l[t][i];
                    s += __shfl_xor_sync(0xFFFFFFFFu, s, 4);
                    s += __shfl_xor_sync(0xFFFFFFFFu, s, 8);
                    s += __shfl_xor_sync(0xFFFFFFFFu, s, 16);
                    if (g == 0)
                        join_ml[w * S::HEADS + 8 * t + 2 * tq + i] = make_float2(m[t][i], s);
                }
                float *to = join + (size_t)(w * S::HEADS + 8 * t + 2 * tq) * S::HS + g;
#pragma unroll
                for (int s = 0; s < KS; ++s) {
                    to[16 * s] = o[t][s][0];
                    to[16 * s + S::HS] = o[t][s][1];
                    to[16 * s + 8] = o[t][s][2];
                    to[16 * s + 8 + S::HS] = o[t][s][3];
                }
            }
            __syncthreads();
            const bool first = xs == c.base, last = end == c.base + c.n, whole = first && last;
            const int part = 2 * (int)blockIdx.x + (first ? 1 : 0);
            for (int e = tid; e < a.G * (D / 4); e += THREADS) {
                const int h = e / (D / 4), d4 = e - h * (D / 4);
                float M = -INFINITY;
#pragma unroll
                for (int u = 0; u < S::W; ++u)
                    M = fmaxf(M, join_ml[u * S::HEADS + h].x);
                float L = 0.f;
                float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
                for (int u = 0; u < S::W; ++u) {
                    const float2 ml = join_ml[u * S::HEADS + h];
                    const float fu = ml.x == -INFINITY ? 0.f : ex2(ml.x - M);
                    const float4 v = *reinterpret_cast<const float4 *>(join + (size_t)(u * S::HEADS + h) * S::HS + 4 * d4);
                    L = fmaf(fu, ml.y, L);
                    y.x = fmaf(fu, v.x, y.x);
                    y.y = fmaf(fu, v.y, y.y);
                    y.z = fmaf(fu, v.z, y.z);
                    y.w = fmaf(fu, v.w, y.w);
                }
                if (whole) {
                    const float inv = L == 0.f ? 0.f : 1.f / L; // nothing kept: zeros
                    uint2 b;
                    b.x = pack2(y.x * inv, y.y * inv);
                    b.y = pack2(y.z * inv, y.w * inv);
                    *reinterpret_cast<uint2 *>(a.out + (size_t)c.b * a.ldo + (size_t)(c.h * a.G + h) * D + 4 * d4) = b;
                } else {
                    *reinterpret_cast<float4 *>(a.ws_o + (size_t)part * kSlotFloats + ((size_t)d4 * S::HEADS + h) * 4) = y;
                    if (d4 == 0)
                        *reinterpret_cast<float2 *>(a.ws_ml + ((size_t)part * 256 + h) * 2) = make_float2(M, L);
                }
            }
            if (!whole && first) {
                begins = 1;
                if (tid == 0) {
                    int32_t *at = a.where + 4 * blockIdx.x;
                    at[0] = c.b;
                    at[1] = 1;
                    at[2] = c.h;
                    at[3] = 0;
                }
            } else if (!whole) {
                cont = last ? 3 : 1;
            }
            xs = end;
            if (xs < x1)
                __syncthreads(); // the joined sums have been read
        }
        asm volatile("cp.async.wait_group 0;" ::: "memory");
    }
    if (tid == 0)
        *reinterpret_cast<int2 *>(a.rec + 2 * blockIdx.x) = make_int2(cont, begins);
}

template <int D, int HT>
cudaError_t launch_step(const StepArgs &p0, float *ws, int num_sms, cudaStream_t s)
{
    using S = StepShape<D, HT>;
    StepArgs p = p0;
    set_scratch(p.a, ws, num_sms);
    static std::atomic<unsigned long long> set{0};
    cudaError_t e = allow_smem(step_kernel<D, HT>, S::SMEM, set);
    if (e != cudaSuccess)
        return e;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(num_sms);
    cfg.blockDim = dim3(S::W * 32);
    cfg.dynamicSmemBytes = S::SMEM;
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    e = cudaLaunchKernelEx(&cfg, step_kernel<D, HT>, p);
    const long long segments = (long long)p.a.B * p.a.Hkv;
    if (e != cudaSuccess || p.a.most_k <= kTile) // a segment of one tile is never cut
        return e;
    MergeArgs g = merge_args(p.a, num_sms);
    g.rows_per_tile = S::HEADS;
    g.DV = D;
    return run_merge(g, (int)(segments < num_sms ? segments : num_sms), s);
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
