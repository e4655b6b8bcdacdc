// Low-rank adapters of many requests beside a shared projection.
//
// Mathematics. Row m has adapter i = ids[m] (none for i < 0):
//   h[m][r] = scale[i] sum_k a[i][r][k] x[m][k]            r < R <= 128
//   out[m][n] = y[m][n] + sum_r b[i][n][r] h[m][r]
// h goes to the second product as three bf16 parts, each the rounding of what those
// before it leave (within 2^-24 of h, as fp32 is): y and out are fp32, and two parts
// (2^-16) were their largest error (10^-6 of out where the sums' is 10^-7). Sums are fp32. b h
// is summed apart, small parts of all R first, and added to y once: the tensor core cuts each
// sum to a step of its own size. Errors of out for 1 row at R = 16, 61 at 64 and 4001 at 32,
// in 10^-7: products added to y 1.8, 3.6, 2.5; apart 0.4, 0.9, 2.0; small parts first 0.4, 0.6,
// 2.0 (at R = 128 2.1 -> 0.8 of 37 rows), at the same times; a plain fp32 sum 0.3, 1.4, 2.1.
//
// In both forms the second product's operands come straight from global memory: within
// 32 elements of the summed dimension a thread holds 8 consecutive ones (both operands in
// the same order), one 16-byte load for two products; and a thread's columns are twice 4
// consecutive ones (an order of the product's columns that the rows of b follow), so y is
// read and out written 64 contiguous bytes of a row at a time.
//
// Up to kGrouped rows (a decode batch, every request its own adapter): one launch. A tile
// is 16 rows of one adapter, which a block finds by ranking all rows among those of the
// same adapter, so an adapter's weights are read once for 16 of its rows. A cluster of 8
// blocks has a tile and some of the columns: each block forms h over an eighth of K, all
// sum the eighths through distributed shared memory and go on to their own columns, whose
// b and y are on their way by then. (Two dependent launches took 15 us a call for one row,
// of which the second launch was 3, and 18 for 61 rows of 12288 columns.)
//
// Above that (prompts, whose rows lie together) a tile is 64 rows in order. First kernel: x
// and a through a ring in shared memory, K split over blocks that leave partial sums of h in
// the scratch (joined by a cluster instead, 4 blocks took 19 us for 4001 x 6144 where the
// stream takes 7). A tile's adapters are shared by kTurns blocks, which take every kTurns-th (a tile
// where one prompt ends and the next begins took a block two passes, and with it the
// call; most tiles leave all turns but the first idle). Second kernel: y and b, 256
// columns a block; the partial sums are added and split once per block, through shared
// memory, with y of the first 32 rows and b on their way.
//
// Bound by y and out (8 bytes per element) for prompts, by the adapters for mixed
// batches, by latency for one token.
#include "common.cuh"
#include "internal.h"

#include <atomic>
#include <cstddef>

namespace w4 {

namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kGrouped = 512; // rows that a block ranks (two of each thread)

struct Args {
    LoraArgs p;
    float *h;          // prompts: partial sums [parts][rows of this pass][R]
    int m0, M;         // first row and rows of this pass
    int parts;         // blocks that share a tile's K
};

struct Tile {
    int row[16];                         // rows of this pass, -1 = none
    alignas(16) int ids[kGrouped];       // adapters of all rows (-1 = none, -2 = no row), read four at a time
    int cnt[kGrouped / 32], pick, rank0;
};
static_assert(offsetof(Tile, ids) % 16 == 0 && alignof(Tile) >= 16, "read four at a time");

__device__ __forceinline__ int adapter_of(const LoraArgs &p, int m)
{
    const int i = __ldg(p.ids + m);
    if (i >= p.L && p.status)
        *p.status = 1;
    return i >= 0 && i < p.L ? i : -1;
}

// Rows of tile `t` and their adapter; `none`: rows without an adapter are wanted too. -2: there is
// no such tile. A tile is led by every 16th row of an adapter, in the order of the rows.
__device__ __forceinline__ int find_tile(const Args &a, int t, bool none, Tile &s)
{
    const int tid = threadIdx.x, lane = tid & 31;
    for (int m = tid; m < kGrouped; m += kThreads)
        s.ids[m] = m < a.M ? adapter_of(a.p, a.m0 + m) : -2;
    if (tid < 16)
        s.row[tid] = -1;
    __syncthreads();
    int rank[2] = {0, 0};
    bool lead[2];
    uint32_t votes[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int m = tid + i * kThreads;
        lead[i] = false;
        if (i * kThreads < a.M) {
            // Equal ones among the rows of the warps before, then within this one's.
            const int mine = s.ids[m];
            for (int j = 0; j < (m & ~31); j += 4) {
                const int4 o = *reinterpret_cast<const int4 *>(s.ids + j);
                rank[i] += (o.x == mine) + (o.y == mine) + (o.z == mine) + (o.w == mine);
            }
            rank[i] += __popc(__match_any_sync(0xFFFFFFFFu, mine) & ((1u << lane) - 1u));
            lead[i] = mine >= (none ? -1 : 0) && rank[i] % 16 == 0;
        }
        votes[i] = __ballot_sync(0xFFFFFFFFu, lead[i]);
        if (lane == 0)
            s.cnt[m >> 5] = __popc(votes[i]);
    }
    __syncthreads();
    int total = 0;
#pragma unroll
    for (int w = 0; w < kGrouped / 32; ++w) {
        const int c = s.cnt[w];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int m = tid + i * kThreads;
            if (w == m >> 5 && lead[i] && total + __popc(votes[i] & ((1u << lane) - 1u)) == t) {
                s.pick = m;
                s.rank0 = rank[i];
            }
        }
        total += c;
    }
    __syncthreads();
    if (t >= total)
        return -2;
    const int id = s.ids[s.pick], r0 = s.rank0;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int m = tid + i * kThreads;
        if (m < a.M && s.ids[m] == id && rank[i] >= r0 && rank[i] < r0 + 16)
            s.row[rank[i] - r0] = m;
    }
    __syncthreads();
    return id;
}

constexpr int kTurns = 2;

// The adapters of 64 rows in order, found by every warp for itself: each kTurns-th from the `turn`-th on.
struct Adapters {
    int id[2];                   // of rows lane and 32 + lane; -1 = none, -2 = no row
    unsigned long long left = 0; // rows not yet taken

    __device__ __forceinline__ Adapters(const Args &a, int tile, int turn, bool none)
    {
        const int lane = threadIdx.x & 31;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int m = tile * 64 + 32 * i + lane;
            id[i] = m < a.M ? adapter_of(a.p, a.m0 + m) : -2;
            left |= (unsigned long long)__ballot_sync(0xFFFFFFFFu, id[i] >= (none ? -1 : 0)) << (32 * i);
        }
        skip(turn);
    }
    __device__ __forceinline__ void skip(int n)
    {
        unsigned long long rows;
        for (; n > 0 && left; --n)
            first(rows);
    }
    // The next adapter and its rows.
    __device__ __forceinline__ int next(unsigned long long &rows)
    {
        const int mine = first(rows);
        skip(kTurns - 1);
        return mine;
    }
    // The adapter of the first row left, and all its rows.
    __device__ __forceinline__ int first(unsigned long long &rows)
    {
        const int m = __ffsll((long long)left) - 1;
        const int a0 = __shfl_sync(0xFFFFFFFFu, id[0], m & 31), a1 = __shfl_sync(0xFFFFFFFFu, id[1], m & 31);
        const int mine = m < 32 ? a0 : a1;
        rows = (unsigned long long)__ballot_sync(0xFFFFFFFFu, id[0] == mine) |
               (unsigned long long)__ballot_sync(0xFFFFFFFFu, id[1] == mine) << 32;
        left &= ~rows;
        return mine;
    }
};

__device__ __forceinline__ uint4 ld16(const uint16_t *p, bool ok)
{
    return ok ? __ldg(reinterpret_cast<const uint4 *>(p)) : make_uint4(0, 0, 0, 0);
}

// Both products of 32 summed elements.
__device__ __forceinline__ void mma32(float (&c)[4], const uint4 &r0, const uint4 &r1, const uint4 &b)
{
    mma_16816(c, r0.x, r1.x, r0.y, r1.y, b.x, b.y);
    mma_16816(c, r0.z, r1.z, r0.w, r1.w, b.z, b.w);
}

__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }

__device__ __forceinline__ float2 ld_cluster_f32x2(uint32_t a)
{
    float2 v;
    asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(a) : "memory");
    return v;
}

// Parts of h, each the rounding of what is left.
__device__ __forceinline__ void split3(float2 v, __nv_bfloat162 (&h)[3])
{
#pragma unroll
    for (int k = 0; k < 3; ++k) {
        h[k] = __floats2bfloat162_rn(v.x, v.y);
        v.x -= __low2float(h[k]);
        v.y -= __high2float(h[k]);
    }
}

// 32 columns of b from n0 on: column c of product j is column 16 (j / 2) + 4 (c / 2) + 2 (j % 2) + c % 2.
template <int NS>
__device__ __forceinline__ void load_b(uint4 (&b)[NS][4], const LoraArgs &p, int id, int n0)
{
    const int lane = threadIdx.x & 31, g = lane >> 2, tq = lane & 3;
#pragma unroll
    for (int k = 0; k < NS; ++k)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int n = n0 + 16 * (j >> 1) + 4 * (g >> 1) + 2 * (j & 1) + (g & 1), r = 32 * k + 8 * tq;
            b[k][j] = ld16(p.b + ((size_t)id * p.N + n) * p.R + r, n < p.N && r < p.R);
        }
}

// This thread's columns of rows q = 0 (g) and 1 (g + 8): 4 tq .. and 16 + 4 tq .. of the 32. `p` at the
// first of them; in0, in1: within N.
__device__ __forceinline__ void load_y(float (&c)[4][4], int q, const float *p, bool in0, bool in1)
{
    const float4 y0 = in0 ? *reinterpret_cast<const float4 *>(p) : make_float4(0.f, 0.f, 0.f, 0.f);
    const float4 y1 = in1 ? *reinterpret_cast<const float4 *>(p + 16) : make_float4(0.f, 0.f, 0.f, 0.f);
    c[0][2 * q] = y0.x;
    c[0][2 * q + 1] = y0.y;
    c[1][2 * q] = y0.z;
    c[1][2 * q + 1] = y0.w;
    c[2][2 * q] = y1.x;
    c[2][2 * q + 1] = y1.y;
    c[3][2 * q] = y1.z;
    c[3][2 * q + 1] = y1.w;
}
__device__ __forceinline__ void store_out(float *to, const float (&c)[4][4], int q, bool in0, bool in1)
{
    if (in0)
        *reinterpret_cast<float4 *>(to) = make_float4(c[0][2 * q], c[0][2 * q + 1], c[1][2 * q], c[1][2 * q + 1]);
    if (in1)
        *reinterpret_cast<float4 *>(to + 16) = make_float4(c[2][2 * q], c[2][2 * q + 1], c[3][2 * q], c[3][2 * q + 1]);
}

constexpr int kCluster = 8;

// Both products of a tile of 16 rows. NT: products across R (R <= 8 NT). Block (cluster c of `groups`
// per tile) has the columns of warps c * 8 + rank, stepping by all of the tile's warps.
template <int NT>
__global__ void __launch_bounds__(kThreads, NT <= 8 ? 2 : 1) __cluster_dims__(kCluster, 1, 1)
lora_group_kernel(const Args a, const int groups)
{
    constexpr int NS = (NT + 3) / 4, RS = 8 * NT, HP = 32 * NS + 8; // HP: elements between rows of h
    constexpr int U = NT <= 2 ? 4 : (NT == 4 ? 2 : 1); // steps of 32 in flight
    constexpr bool EARLY = NT <= 4;                    // registers hold b beside the first product's operands
    extern __shared__ __align__(16) float part[]; // [kWarps][16][RS], then h [3][16][HP] bf16
    __nv_bfloat16 *hs = reinterpret_cast<__nv_bfloat16 *>(part + kWarps * 16 * RS);
    __shared__ Tile s;
    const LoraArgs &p = a.p;
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5, g = lane >> 2, tq = lane & 3;
    const int rank = (int)(blockIdx.x % kCluster), cl = (int)(blockIdx.x / kCluster);
    const bool copy = p.out != p.y;
    pdl_launch_dependents();
    pdl_wait();
    const int id = find_tile(a, cl / groups, copy, s);
    if (id == -2)
        return; // the whole cluster
    const int m0 = s.row[g], m1 = s.row[g + 8];
    const size_t row0 = (size_t)(a.m0 + max(m0, 0)), row1 = (size_t)(a.m0 + max(m1, 0));
    const int step = groups * kCluster * kWarps * 32;
    int n0 = (((cl % groups) * kCluster + rank) * kWarps + w) * 32;
    // The first columns' b and y are asked for before anything else.
    uint4 b[NS][4];
    float c[4][4];
    auto ask = [&](int n) {
        if (id >= 0)
            load_b<NS>(b, p, id, n);
        const bool in0 = n + 4 * tq < p.N, in1 = n + 16 + 4 * tq < p.N;
        load_y(c, 0, p.y + row0 * p.ldy + n + 4 * tq, in0 && m0 >= 0, in1 && m0 >= 0);
        load_y(c, 1, p.y + row1 * p.ldy + n + 4 * tq, in0 && m1 >= 0, in1 && m1 >= 0);
    };
    // b of all this block's columns on its way to L2 (a stretch of memory per 256 columns).
    if (id >= 0 && lane == 0 && w == 0)
        for (int n = n0; n < p.N; n += step)
            prefetch_l2_bulk(p.b + ((size_t)id * p.N + n) * p.R, (uint32_t)min(32 * kWarps, p.N - n) * p.R * 2);
    if (EARLY && n0 < p.N)
        ask(n0);
    if (id >= 0) {
        // h: this warp's steps of 32 of K.
        const int steps = p.K / 32, mine = rank * kWarps + w;
        const int s0 = (int)((long long)steps * mine / (kCluster * kWarps));
        const int s1 = (int)((long long)steps * (mine + 1) / (kCluster * kWarps));
        const uint16_t *x0 = p.x + row0 * p.ldx + 8 * tq, *x1 = p.x + row1 * p.ldx + 8 * tq;
        const uint16_t *ap = p.a + ((size_t)id * p.R + g) * p.K + 8 * tq;
        float h[NT][4];
#pragma unroll
        for (int n = 0; n < NT; ++n)
            h[n][0] = h[n][1] = h[n][2] = h[n][3] = 0.f;
#pragma unroll 1
        for (int st = s0; st < s1; st += U) {
            uint4 r0[U], r1[U], aa[U][NT];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const bool in = st + u < s1;
                r0[u] = ld16(x0 + (size_t)(st + u) * 32, in && m0 >= 0);
                r1[u] = ld16(x1 + (size_t)(st + u) * 32, in && m1 >= 0);
#pragma unroll
                for (int n = 0; n < NT; ++n)
                    aa[u][n] = ld16(ap + (size_t)n * 8 * p.K + (size_t)(st + u) * 32, in && 8 * n + g < p.R);
            }
#pragma unroll
            for (int u = 0; u < U; ++u)
#pragma unroll
                for (int n = 0; n < NT; ++n)
                    mma32(h[n], r0[u], r1[u], aa[u][n]);
        }
        float *to = part + (size_t)w * 16 * RS;
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            *reinterpret_cast<float2 *>(to + g * RS + 8 * n + 2 * tq) = make_float2(h[n][0], h[n][1]);
            *reinterpret_cast<float2 *>(to + (g + 8) * RS + 8 * n + 2 * tq) = make_float2(h[n][2], h[n][3]);
        }
        __syncthreads();
        // The warps' parts, then the blocks', in order.
        for (int e = threadIdx.x; e < 16 * RS / 2; e += kThreads) {
            float2 *f = reinterpret_cast<float2 *>(part) + e;
            float2 v = f[0];
#pragma unroll
            for (int k = 1; k < kWarps; ++k) {
                v.x += f[k * (16 * RS / 2)].x;
                v.y += f[k * (16 * RS / 2)].y;
            }
            f[0] = v;
        }
        cluster_sync();
        const float scale = p.scale ? __ldg(p.scale + id) : 1.f;
        for (int e = threadIdx.x; e < 16 * (HP / 2); e += kThreads) {
            const int i = e / (HP / 2), r = 2 * (e - i * (HP / 2));
            float2 v = make_float2(0.f, 0.f);
            if (r < RS) {
                const uint32_t at = smem_addr(part) + (uint32_t)(i * RS + r) * 4;
#pragma unroll
                for (int k = 0; k < kCluster; ++k) {
                    const float2 q = ld_cluster_f32x2(map_rank(at, k));
                    v.x += q.x;
                    v.y += q.y;
                }
                v.x *= scale;
                v.y *= scale;
            }
            __nv_bfloat162 q[3];
            split3(v, q);
#pragma unroll
            for (int k = 0; k < 3; ++k)
                *reinterpret_cast<__nv_bfloat162 *>(hs + (size_t)(k * 16 + i) * HP + r) = q[k];
        }
        __syncthreads();
        cluster_arrive(); // this block has read the others' parts
    }
    if (!EARLY && n0 < p.N)
        ask(n0);
    for (; n0 < p.N; n0 += step) {
        float d[4][4]; // b h, added to y once
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int i = 0; i < 4; ++i)
                d[j][i] = 0.f;
        if (id >= 0) {
#pragma unroll
            for (int t = 2; t >= 0; --t) // all small parts first
#pragma unroll
                for (int k = 0; k < NS; ++k) {
                    uint4 h[2];
#pragma unroll
                    for (int q = 0; q < 2; ++q)
                        h[q] = lds128(smem_addr(hs + (size_t)(t * 16 + g + 8 * q) * HP + 32 * k + 8 * tq));
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        mma32(d[j], h[0], h[1], b[k][j]);
                }
        }
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int i = 0; i < 4; ++i)
                d[j][i] = id >= 0 ? c[j][i] + d[j][i] : c[j][i]; // (without an adapter y's bits, -0 too)
        const int at = n0 + 4 * tq;
        const bool in0 = at < p.N, in1 = at + 16 < p.N;
        if (n0 + step < p.N)
            ask(n0 + step); // the next columns, ahead of the stores
        store_out(p.out + row0 * p.ldo + at, d, 0, in0 && m0 >= 0, in1 && m0 >= 0);
        store_out(p.out + row1 * p.ldo + at, d, 1, in0 && m1 >= 0, in1 && m1 >= 0);
    }
    if (id >= 0)
        cluster_wait(); // this block's part has been read
}

// Copies of 16 bytes to shared memory, zeros where !ok.
__device__ __forceinline__ void copy16(uint32_t dst, const void *src, bool ok)
{
    asm volatile("cp.async.cg.shared.global.L2::256B [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(ok ? 16 : 0)
                 : "memory");
}
__device__ __forceinline__ void ldsm4(uint32_t addr, uint32_t (&r)[4])
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}

// h of a tile of 64 rows in order. A stage is 128 elements of K: 64 rows of x and 8 NT of a, 256 bytes
// each, the 16-byte piece c of row r at c ^ (r & 7). Warp w has rows 16 (w / 2) .. and half w % 2 of a stage.
template <int NT>
struct DownShape {
    static constexpr int RS = 8 * NT;
    static constexpr int STAGE = (64 + RS) * 256;
    static constexpr int ST = NT <= 4 ? 4 : (NT == 8 ? 3 : 4); // two blocks an SM (one at NT = 16)
    static constexpr int PART = 64 * RS * 4; // over the ring's space, when it is drained
    static constexpr int SMEM = ST * STAGE > PART ? ST * STAGE : PART;
};

template <int NT>
__global__ void __launch_bounds__(kThreads, NT <= 8 ? 2 : 1)
lora_down_kernel(const Args a)
{
    using S = DownShape<NT>;
    constexpr int TR = 64, RS = S::RS, ST = S::ST;
    extern __shared__ __align__(128) unsigned char ring_[];
    float *part = reinterpret_cast<float *>(ring_); // [TR][RS]
    const LoraArgs &p = a.p;
    const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5, g = lane >> 2, tq = lane & 3;
    const int tiles = (a.M + TR - 1) / TR, part_no = (int)(blockIdx.x % a.parts);
    const int tile = (int)(blockIdx.x / a.parts) % tiles, turn = (int)(blockIdx.x / a.parts) / tiles;
    const uint32_t ring = smem_addr(ring_);
    pdl_wait();
    pdl_launch_dependents(); // what the next kernel reads early is complete
    Adapters ad(a, tile, turn, false);
    const int steps = (p.K + 127) / 128; // the last one may be short
    const int s0 = (int)((long long)steps * part_no / a.parts), s1 = (int)((long long)steps * (part_no + 1) / a.parts);
    const int wr = w >> 1, half = w & 1;
    // A thread copies piece tid % 16 of rows tid / 16, 16 further on, ...: four of x, then those of a.
    const int cr = tid >> 4, cc = tid & 15, left = a.M - (tile * TR + cr);
    const uint32_t to0 = ring + cr * 256 + ((cc ^ (cr & 7)) << 4);
    const uint16_t *px = p.x + (size_t)(a.m0 + tile * TR + cr) * p.ldx + s0 * 128 + cc * 8;

    while (ad.left) {
        unsigned long long rows;
        const int id = ad.next(rows);
        const uint16_t *pa = p.a + ((size_t)id * p.R + cr) * p.K + s0 * 128 + cc * 8;
        auto issue = [&](int i) { // stage i of this block's
            if (i < s1 - s0) {
                const uint32_t to = to0 + (i % ST) * S::STAGE;
                const bool in = (s0 + i) * 128 + cc * 8 < p.K;
                const uint16_t *x = px + i * 128, *y = pa + i * 128;
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const bool ok = in && 16 * q < left;
                    copy16(to + 16 * q * 256, ok ? x + (size_t)16 * q * p.ldx : p.x, ok);
                }
#pragma unroll
                for (int q = 0; q < (RS + 15) / 16; ++q) {
                    const int r = 16 * q + cr;
                    if (RS % 16 == 0 || r < RS) {
                        const bool ok = in && r < p.R;
                        copy16(to + (64 + 16 * q) * 256, ok ? y + (size_t)16 * q * p.K : p.a, ok);
                    }
                }
            }
            asm volatile("cp.async.commit_group;" ::: "memory");
        };
#pragma unroll
        for (int i = 0; i < ST - 1; ++i)
            issue(i);
        float c[NT][4];
#pragma unroll
        for (int n = 0; n < NT; ++n)
            c[n][0] = c[n][1] = c[n][2] = c[n][3] = 0.f;
#pragma unroll 1
        for (int st = 0; st < s1 - s0; ++st) {
            asm volatile("cp.async.wait_group %0;" ::"n"(ST - 2) : "memory");
            __syncthreads(); // the stage is in place, and the one before it has been read
            issue(st + ST - 1);
            const uint32_t xb = ring + (st % ST) * S::STAGE, ab = xb + 64 * 256;
            const int row = (lane & 7) + ((lane >> 3) & 1) * 8, up = lane >> 4; // x: rows, then halves of 16
            const int arow = (lane & 7) + (lane >> 4) * 8, aup = (lane >> 3) & 1; // a: halves of 16, then rows
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const int c0 = 8 * half + 2 * k;
                uint32_t x4[4];
                ldsm4(xb + (16 * wr + row) * 256 + (((c0 + up) ^ (row & 7)) << 4), x4);
                if (NT == 1) {
                    uint32_t b0, b1;
                    asm volatile("ldmatrix.sync.aligned.m8n8.x2.shared.b16 {%0,%1}, [%2];"
                                 : "=r"(b0), "=r"(b1)
                                 : "r"(ab + (lane & 7) * 256 + (((c0 + aup) ^ (lane & 7)) << 4))
                                 : "memory");
                    mma_16816(c[0], x4[0], x4[1], x4[2], x4[3], b0, b1);
                } else {
#pragma unroll
                    for (int n = 0; n + 1 < NT; n += 2) {
                        uint32_t b4[4];
                        ldsm4(ab + (8 * n + arow) * 256 + (((c0 + aup) ^ (arow & 7)) << 4), b4);
                        mma_16816(c[n], x4[0], x4[1], x4[2], x4[3], b4[0], b4[1]);
                        mma_16816(c[n + 1], x4[0], x4[1], x4[2], x4[3], b4[2], b4[3]);
                    }
                }
            }
        }
        asm volatile("cp.async.wait_group 0;" ::: "memory");
        __syncthreads(); // the ring's space is the parts' now
        const int i0 = 16 * wr + g, i1 = i0 + 8;
        if (half) {
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                *reinterpret_cast<float2 *>(part + i0 * RS + 8 * n + 2 * tq) = make_float2(c[n][0], c[n][1]);
                *reinterpret_cast<float2 *>(part + i1 * RS + 8 * n + 2 * tq) = make_float2(c[n][2], c[n][3]);
            }
        }
        __syncthreads();
        if (!half) {
            float *to = a.h + ((size_t)part_no * a.M + (size_t)tile * TR) * p.R + 2 * tq;
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                const float2 v0 = *reinterpret_cast<float2 *>(part + i0 * RS + 8 * n + 2 * tq);
                const float2 v1 = *reinterpret_cast<float2 *>(part + i1 * RS + 8 * n + 2 * tq);
                if (8 * n < p.R) {
                    if ((rows >> i0) & 1)
                        *reinterpret_cast<float2 *>(to + (size_t)i0 * p.R + 8 * n) = make_float2(c[n][0] + v0.x, c[n][1] + v0.y);
                    if ((rows >> i1) & 1)
                        *reinterpret_cast<float2 *>(to + (size_t)i1 * p.R + 8 * n) = make_float2(c[n][2] + v1.x, c[n][3] + v1.y);
                }
            }
        }
        __syncthreads(); // the space is the ring's again
    }
}

// out = y + b h. NS: steps of 32 across R. A warp has 32 columns of the tile's 64 rows.
template <int NS>
__global__ void __launch_bounds__(kThreads, NS == 1 ? 3 : (NS == 2 ? 2 : 1))
lora_up_kernel(const Args a)
{
    constexpr int TR = 64, RB = TR / 16, RU = 2;               // row blocks; in flight
    constexpr int HP = 32 * NS + 8;                            // elements between rows of h
    constexpr int AT = NS == 1 ? 3 : 1;                        // parts of h read together (one at a time: 29.7 us for 28.7)
    extern __shared__ __align__(16) __nv_bfloat16 hs_[];       // [3][TR][HP]
    __shared__ int s_id[TR];
    const LoraArgs &p = a.p;
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5, g = lane >> 2, tq = lane & 3;
    pdl_launch_dependents();
    const int n0 = ((int)blockIdx.y * kWarps + w) * 32, tile = (int)blockIdx.x;
    const bool in0 = n0 + 4 * tq < p.N, in1 = n0 + 16 + 4 * tq < p.N; // this thread's columns (N is a multiple of 8)
    const int m = tile * TR + g, rows = a.M - m; // this thread's first row of the pass; rows from it on
    const float *yp = p.y + (size_t)(a.m0 + m) * p.ldy + n0 + 4 * tq;
    float *op = p.out + (size_t)(a.m0 + m) * p.ldo + n0 + 4 * tq;
    int ids[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int r = tile * TR + 32 * i + lane;
        ids[i] = r < a.M ? adapter_of(p, a.m0 + r) : -2;
        if (w == 0)
            s_id[32 * i + lane] = ids[i];
    }
    int have = -2; // the adapter whose b is held
    uint4 b[NS][4];
    // h of the tile, once the first kernel has left it: partial sums added in order, scaled, in three parts.
    auto stage = [&]() {
        __syncthreads(); // the rows' adapters
        pdl_wait();
#pragma unroll 2
        for (int q = 0; q < TR * 8 * NS / kThreads; ++q) { // four elements of a row each
            const int e = q * kThreads + (int)threadIdx.x, i = e / (8 * NS), r = 4 * (e - i * 8 * NS), id = s_id[i];
            const bool ok = id >= 0 && r < p.R;
            const float *from = a.h + ((size_t)tile * TR + i) * p.R + r;
            float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
            for (int k0 = 0; k0 < a.parts; k0 += 4) {
                float4 x[4]; // in flight together
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    x[k] = ok && k0 + k < a.parts
                               ? __ldcg(reinterpret_cast<const float4 *>(from + (size_t)(k0 + k) * a.M * p.R))
                               : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    v.x += x[k].x;
                    v.y += x[k].y;
                    v.z += x[k].z;
                    v.w += x[k].w;
                }
            }
            const float f = ok && p.scale ? __ldg(p.scale + id) : 1.f;
            __nv_bfloat162 lo[3], hi[3];
            split3(make_float2(v.x * f, v.y * f), lo);
            split3(make_float2(v.z * f, v.w * f), hi);
#pragma unroll
            for (int t = 0; t < 3; ++t) {
                __nv_bfloat16 *to = hs_ + (size_t)(t * TR + i) * HP + r;
                *reinterpret_cast<__nv_bfloat162 *>(to) = lo[t];
                *reinterpret_cast<__nv_bfloat162 *>(to + 2) = hi[t];
            }
        }
        __syncthreads();
    };
#pragma unroll
    for (int rb = 0; rb < RB; rb += RU) {
        float c[RU][4][4];
#pragma unroll
        for (int u = 0; u < RU; ++u)
#pragma unroll
            for (int q = 0; q < 2; ++q) {
                const int i = (rb + u) * 16 + 8 * q;
                load_y(c[u], q, yp + (size_t)i * p.ldy, in0 && i < rows, in1 && i < rows);
            }
        if (rb == 0) {
            const int id = __shfl_sync(0xFFFFFFFFu, ids[0], 0);
            if (id >= 0) { // as a rule that of all rows
                load_b<NS>(b, p, id, n0);
                have = id;
            }
            stage();
        }
#pragma unroll
        for (int u = 0; u < RU; ++u) {
            const int i = (rb + u) * 16, from = 16 * ((rb + u) & 1);
            const int id = ids[(rb + u) >> 1]; // of lane l: row 32 ((rb + u) / 2) + l
            // The block's adapters in turn: the lanes (rows) that are left of it.
            uint32_t left = __ballot_sync(0xFFFFFFFFu, id >= 0) & (0xFFFFu << from);
            while (left) {
                const int mine = __shfl_sync(0xFFFFFFFFu, id, __ffs(left) - 1);
                const uint32_t its = __ballot_sync(0xFFFFFFFFu, id == mine) & (0xFFFFu << from);
                left &= ~its;
                if (mine != have) {
                    load_b<NS>(b, p, mine, n0);
                    have = mine;
                }
                float d[4][4]; // b h, added to y once
#pragma unroll
                for (int j = 0; j < 4; ++j)
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        d[j][k] = 0.f;
#pragma unroll
                for (int t0 = 2; t0 >= 0; t0 -= AT) // all small parts first
#pragma unroll
                    for (int k = 0; k < NS; ++k) {
                        uint4 h[AT][2];
#pragma unroll
                        for (int t = 0; t < AT; ++t)
#pragma unroll
                            for (int q = 0; q < 2; ++q)
                                h[t][q] = lds128(
                                    smem_addr(hs_ + (size_t)((t0 - t) * TR + i + 8 * q + g) * HP + 32 * k + 8 * tq));
#pragma unroll
                        for (int t = 0; t < AT; ++t)
#pragma unroll
                            for (int j = 0; j < 4; ++j)
                                mma32(d[j], h[t][0], h[t][1], b[k][j]);
                    }
                // Rows of other adapters stay as they were.
                const bool ok0 = (its >> (from + g)) & 1, ok1 = (its >> (from + g + 8)) & 1;
#pragma unroll
                for (int j = 0; j < 4; ++j)
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        c[u][j][k] = (k < 2 ? ok0 : ok1) ? c[u][j][k] + d[j][k] : c[u][j][k];
            }
#pragma unroll
            for (int q = 0; q < 2; ++q)
                store_out(op + (size_t)(i + 8 * q) * p.ldo, c[u], q, in0 && i + 8 * q < rows, in1 && i + 8 * q < rows);
        }
    }
}

// Dynamic shared memory of a kernel, once per device.
template <typename K>
cudaError_t allow(K kern, int bytes, std::atomic<unsigned long long> &set)
{
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess)
        return e;
    if (dev < 64 && ((set.load(std::memory_order_relaxed) >> dev) & 1))
        return cudaSuccess;
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e == cudaSuccess && dev < 64)
        set.fetch_or(1ull << dev, std::memory_order_relaxed);
    return e;
}

template <int NT>
cudaError_t grouped(const Args &a, int tiles, int num_sms, cudaStream_t s)
{
    constexpr int NS = (NT + 3) / 4, SMEM = kWarps * 16 * 8 * NT * 4 + 3 * 16 * (32 * NS + 8) * 2;
    static std::atomic<unsigned long long> set{0};
    cudaError_t e = allow(lora_group_kernel<NT>, SMEM, set);
    if (e != cudaSuccess)
        return e;
    // Clusters of a tile, each with a part of the columns and h formed anew: as many as the
    // columns have use for while all fit about two blocks an SM (there are fewer tiles than
    // `tiles` as a rule).
    const int most = (a.p.N + 32 * kWarps * kCluster - 1) / (32 * kWarps * kCluster);
    int groups = (5 * num_sms / 2) / (tiles * kCluster);
    groups = groups < 1 ? 1 : (groups > most ? most : groups);
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(tiles * groups * kCluster));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = SMEM;
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, lora_group_kernel<NT>, a, groups);
}

template <int NT>
cudaError_t down(const Args &a, cudaStream_t s)
{
    static std::atomic<unsigned long long> set{0};
    cudaError_t e = allow(lora_down_kernel<NT>, DownShape<NT>::SMEM, set);
    if (e != cudaSuccess)
        return e;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)((a.M + 63) / 64 * kTurns * a.parts));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = DownShape<NT>::SMEM;
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, lora_down_kernel<NT>, a);
}

template <int NT>
cudaError_t prompt(const Args &a, cudaStream_t s)
{
    constexpr int NS = (NT + 3) / 4, SMEM = 3 * 64 * (32 * NS + 8) * 2;
    cudaError_t e = down<NT>(a, s);
    if (e != cudaSuccess)
        return e;
    static std::atomic<unsigned long long> set{0};
    e = allow(lora_up_kernel<NS>, SMEM, set);
    if (e != cudaSuccess)
        return e;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)((a.M + 63) / 64), (unsigned)((a.p.N + 32 * kWarps - 1) / (32 * kWarps)));
    cfg.blockDim = dim3(kThreads);
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    cfg.dynamicSmemBytes = SMEM;
    return cudaLaunchKernelEx(&cfg, lora_up_kernel<NS>, a);
}

template <int NT>
cudaError_t pass(const Args &a, int num_sms, cudaStream_t s)
{
    if (a.M > kGrouped)
        return prompt<NT>(a, s);
    // Each adapter (and the rows without one) has at most one tile that is not full.
    const long long ids = (long long)a.p.L + 1, n = a.M / 16 + (ids < a.M ? ids : a.M);
    return grouped<NT>(a, (int)(n < a.M ? n : a.M), num_sms, s);
}

} // namespace

cudaError_t run_lora(const LoraArgs &p, float *ws, size_t ws_floats, int num_sms, cudaStream_t s)
{
    // Blocks that share a tile's K, while they fit the SMs and each has a few stages.
    const long long all = ((long long)p.M + 63) / 64;
    int parts = 1;
    while (parts < 8 && all * parts * 2 <= 2ll * num_sms && parts * 512 < p.K)
        parts *= 2;
    // Rows whose partial sums fit the scratch go in one pass (79040 at R = 128 on 152 SMs).
    const long long most = (long long)(ws_floats / ((size_t)p.R * parts)) / 64 * 64;
    for (long long m0 = 0; m0 < p.M; m0 += most) {
        Args a = {};
        a.p = p;
        a.m0 = (int)m0;
        a.M = (int)(p.M - m0 < most ? p.M - m0 : most);
        a.h = ws;
        a.parts = parts;
        const cudaError_t e = p.R <= 8    ? pass<1>(a, num_sms, s)
                              : p.R <= 16 ? pass<2>(a, num_sms, s)
                              : p.R <= 32 ? pass<4>(a, num_sms, s)
                              : p.R <= 64 ? pass<8>(a, num_sms, s)
                                          : pass<16>(a, num_sms, s);
        if (e != cudaSuccess)
            return e;
    }
    return cudaSuccess;
}

} // namespace w4
