// Low-rank adapters of many requests beside a shared projection.
//
// Mathematics. Row m has adapter i = ids[m] (none for i < 0):
//   h[m][r] = scale[i] sum_k a[i][r][k] x[m][k]            r < R <= 128
//   out[m][n] = y[m][n] + sum_r b[i][n][r] h[m][r]
// Two kernels: the first forms h, the second reads y and adds. h goes to the second
// one's tensor-core product as three bf16 parts, each the rounding of what those before
// it leave (within 2^-25 of h, as fp32 is): y and out are fp32, and two parts (2^-17)
// were their largest error (10^-6 of out where the sums' is 10^-7). Sums are fp32.
//
// Rows. A product tile is 16 rows of one adapter. Up to kGrouped rows (a decode
// batch, every request its own adapter) a block finds its tile by ranking all rows
// among those of the same adapter, so an adapter's weights are read once for 16 of
// its rows. Above that (prompts, whose rows lie together) a tile is 64 rows in
// order, and a block takes its adapters in turn.
//
// First kernel: the K dimension is split over the warps of a block and the blocks
// of a cluster, summed through distributed shared memory (in a fixed order). Second:
// a warp has 32 columns, each thread 8 consecutive ones of a row (an order of the
// product's columns that the rows of b follow), so y is read and out written 32 bytes
// at a time per thread; b and y are asked for before the first kernel has finished.
// Operands come straight from global memory: within 32 elements of the summed
// dimension a thread holds 8 consecutive ones (both operands in the same order), one
// 16-byte load for two products.
//
// Bound by y and out (8 bytes per element) for prompts, by the adapters for mixed
// batches, by latency (two dependent launches' worth) for one token.
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
    uint16_t *h;       // [3 parts][rows of this pass][R]
    int m0, M;         // first row and rows of this pass
    int parts;         // blocks of a cluster
};

template <int TR>
struct Tile {
    int row[TR];  // rows of this pass, -1 = none
    int id[TR];   // their adapter; -1 = no adapter, -2 = no row
    int list[TR]; // adapters of the tile
    int n;
    alignas(16) int ids[TR == 16 ? kGrouped : 4]; // read four at a time
    int cnt[kGrouped / 32], pick, rank0;
};

static_assert(offsetof(Tile<16>, ids) % 16 == 0 && alignof(Tile<16>) >= 16, "read four at a time");

__device__ __forceinline__ int adapter_of(const LoraArgs &p, int m)
{
    const int i = __ldg(p.ids + m);
    if (i >= p.L && p.status)
        *p.status = 1;
    return i >= 0 && i < p.L ? i : -1;
}

// Rows and adapters of tile `t`; `none`: rows without an adapter are wanted too.
// False: there is no such tile.
template <int TR>
__device__ __forceinline__ bool find_tile(const Args &a, int t, bool none, Tile<TR> &s)
{
    const int tid = threadIdx.x, lane = tid & 31;
    if (TR == 16) {
        for (int m = tid; m < kGrouped; m += kThreads)
            s.ids[m] = m < a.M ? adapter_of(a.p, a.m0 + m) : -2;
        if (tid < TR)
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
                const int mine = s.ids[m];
                const int end = min(m | 31, a.M - 1); // the warp's lanes end together
                for (int j = 0; j <= end; j += 4) {
                    const int4 o = *reinterpret_cast<const int4 *>(s.ids + j);
                    rank[i] += (j < m && o.x == mine) + (j + 1 < m && o.y == mine) + (j + 2 < m && o.z == mine) +
                               (j + 3 < m && o.w == mine);
                }
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
            return false;
        const int id = s.ids[s.pick], r0 = s.rank0;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int m = tid + i * kThreads;
            if (m < a.M && s.ids[m] == id && rank[i] >= r0 && rank[i] < r0 + 16)
                s.row[rank[i] - r0] = m;
        }
        __syncthreads();
        if (tid < TR)
            s.id[tid] = s.row[tid] >= 0 ? id : -2;
        if (tid == 0) {
            s.list[0] = id;
            s.n = 1;
        }
        __syncthreads();
        return true;
    }
    if (tid < TR) {
        const int m = t * TR + tid;
        s.row[tid] = m < a.M ? m : -1;
        s.id[tid] = m < a.M ? adapter_of(a.p, a.m0 + m) : -2;
    }
    __syncthreads();
    if (tid < 32) { // the first row of each adapter, in order
        int n = 0;
#pragma unroll
        for (int i = 0; i < TR / 32; ++i) {
            const int m = 32 * i + lane, mine = s.id[m];
            bool first = mine >= (none ? -1 : 0);
            for (int j = 0; j < m; ++j)
                first = first && s.id[j] != mine;
            const uint32_t v = __ballot_sync(0xFFFFFFFFu, first);
            if (first)
                s.list[n + __popc(v & ((1u << lane) - 1u))] = mine;
            n += __popc(v);
        }
        if (lane == 0)
            s.n = n;
    }
    __syncthreads();
    return t * TR < a.M;
}

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

// h of a tile. NT: products across R (R <= 8 NT). WK warps of a block share a tile's 16
// rows, each with a part of K.
template <int TR, int NT>
__global__ void __launch_bounds__(kThreads)
lora_down_kernel(const Args a)
{
    constexpr int WR = TR / 16, WK = kWarps / WR;
    constexpr int U = NT <= 2 ? 4 : (NT == 4 ? 3 : (NT == 8 ? 2 : 1)); // steps of 32 in flight
    constexpr int RS = 8 * NT;
    extern __shared__ __align__(16) float part[]; // [WK][TR][RS]
    __shared__ __align__(16) Tile<TR> s;
    const LoraArgs &p = a.p;
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5, g = lane >> 2, tq = lane & 3;
    const int wr = w / WK, wk = w % WK;
    const int part_no = (int)(blockIdx.x % a.parts);
    pdl_wait();
    pdl_launch_dependents(); // what the next kernel reads early is complete
    if (!find_tile<TR>(a, (int)(blockIdx.x / a.parts), false, s))
        return; // the whole cluster
    const int steps = p.K / 32, parts = a.parts * WK, mine = part_no * WK + wk;
    const int s0 = (int)((long long)steps * mine / parts), s1 = (int)((long long)steps * (mine + 1) / parts);

    for (int l = 0; l < s.n; ++l) {
        const int id = s.list[l];
        const int i0 = wr * 16 + g, i1 = i0 + 8;
        const bool ok0 = s.id[i0] == id, ok1 = s.id[i1] == id;
        if (__any_sync(0xFFFFFFFFu, ok0 || ok1)) {
            const uint16_t *x0 = p.x + (size_t)(a.m0 + (ok0 ? s.row[i0] : 0)) * p.ldx + 8 * tq;
            const uint16_t *x1 = p.x + (size_t)(a.m0 + (ok1 ? s.row[i1] : 0)) * p.ldx + 8 * tq;
            const uint16_t *ap = p.a + ((size_t)id * p.R + g) * p.K + 8 * tq;
            float c[NT][4];
#pragma unroll
            for (int n = 0; n < NT; ++n)
                c[n][0] = c[n][1] = c[n][2] = c[n][3] = 0.f;
#pragma unroll 1
            for (int st = s0; st < s1; st += U) {
                uint4 r0[U], r1[U], b[U][NT];
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    const bool in = st + u < s1;
                    r0[u] = ld16(x0 + (size_t)(st + u) * 32, in && ok0);
                    r1[u] = ld16(x1 + (size_t)(st + u) * 32, in && ok1);
#pragma unroll
                    for (int n = 0; n < NT; ++n)
                        b[u][n] = ld16(ap + (size_t)n * 8 * p.K + (size_t)(st + u) * 32, in && 8 * n + g < p.R);
                }
#pragma unroll
                for (int u = 0; u < U; ++u)
#pragma unroll
                    for (int n = 0; n < NT; ++n)
                        mma32(c[n], r0[u], r1[u], b[u][n]);
            }
            float *to = part + (size_t)wk * TR * RS;
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                *reinterpret_cast<float2 *>(to + i0 * RS + 8 * n + 2 * tq) = make_float2(c[n][0], c[n][1]);
                *reinterpret_cast<float2 *>(to + i1 * RS + 8 * n + 2 * tq) = make_float2(c[n][2], c[n][3]);
            }
        }
        __syncthreads();
        // The warps' parts, then the blocks'.
        for (int e = threadIdx.x; e < TR * RS / 2; e += kThreads) {
            if (s.id[e / (RS / 2)] != id)
                continue;
            float2 *f = reinterpret_cast<float2 *>(part) + e;
            float2 v = f[0];
#pragma unroll
            for (int k = 1; k < WK; ++k) {
                v.x += f[k * (TR * RS / 2)].x;
                v.y += f[k * (TR * RS / 2)].y;
            }
            f[0] = v;
        }
        if (a.parts > 1)
            cluster_sync();
        else
            __syncthreads();
        const float scale = p.scale ? __ldg(p.scale + id) : 1.f;
        for (int e = part_no * kThreads + threadIdx.x; e < TR * RS / 2; e += kThreads * a.parts) {
            const int i = e / (RS / 2), r = 2 * (e - i * (RS / 2));
            if (s.id[i] != id || r >= p.R)
                continue;
            float2 v = make_float2(0.f, 0.f);
            if (a.parts > 1) {
                const uint32_t at = smem_addr(part) + (uint32_t)e * 8;
                for (int k = 0; k < a.parts; ++k) {
                    const uint32_t q = map_rank(at, k);
                    v.x += ld_cluster_f32(q);
                    v.y += ld_cluster_f32(q + 4);
                }
            } else {
                v = reinterpret_cast<float2 *>(part)[e];
            }
            v.x *= scale;
            v.y *= scale;
#pragma unroll
            for (int k = 0; k < 3; ++k) {
                const __nv_bfloat162 h = __floats2bfloat162_rn(v.x, v.y);
                v.x -= __low2float(h);
                v.y -= __high2float(h);
                *reinterpret_cast<__nv_bfloat162 *>(a.h + ((size_t)k * a.M + s.row[i]) * p.R + r) = h;
            }
        }
        if (a.parts > 1)
            cluster_sync(); // before another block's reads of this one's part go stale
        else
            __syncthreads();
    }
}

// out = y + b h. NS: steps of 32 across R. A warp has 32 columns of the tile's rows.
template <int TR, int NS>
__global__ void __launch_bounds__(kThreads)
lora_up_kernel(const Args a)
{
    constexpr int RB = TR / 16, RU = RB > 1 ? 2 : 1; // row blocks; in flight
    __shared__ __align__(16) Tile<TR> s;
    const LoraArgs &p = a.p;
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5, g = lane >> 2, tq = lane & 3;
    const bool copy = p.out != p.y;
    pdl_launch_dependents();
    if (!find_tile<TR>(a, (int)blockIdx.x, copy, s)) {
        pdl_wait();
        return;
    }
    const int n0 = ((int)blockIdx.y * kWarps + w) * 32;
    const bool in = n0 + 8 * tq < p.N; // this thread's columns (N is a multiple of 8)
    bool waited = false;
    for (int l = 0; l < s.n && n0 < p.N; ++l) {
        const int id = s.list[l];
        uint4 b[NS][4];
        if (id >= 0) {
#pragma unroll
            for (int k = 0; k < NS; ++k)
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    // Column c of product j is column 8 (c / 2) + 2 j + c % 2 of the warp's 32.
                    const int n = n0 + 8 * (g >> 1) + 2 * j + (g & 1), r = 32 * k + 8 * tq;
                    b[k][j] = ld16(p.b + ((size_t)id * p.N + n) * p.R + r, n < p.N && r < p.R);
                }
        }
#pragma unroll 1
        for (int rb = 0; rb < RB; rb += RU) {
            bool ok[RU][2];
            size_t row[RU][2];
            float c[RU][4][4];
#pragma unroll
            for (int u = 0; u < RU; ++u)
#pragma unroll
                for (int q = 0; q < 2; ++q) {
                    const int i = (rb + u) * 16 + 8 * q + g;
                    ok[u][q] = s.id[i] == id;
                    row[u][q] = (size_t)(ok[u][q] ? s.row[i] : 0);
                    float4 y0 = make_float4(0.f, 0.f, 0.f, 0.f), y1 = y0;
                    if (ok[u][q] && in) {
                        const float *yp = p.y + (a.m0 + row[u][q]) * (size_t)p.ldy + n0 + 8 * tq;
                        y0 = *reinterpret_cast<const float4 *>(yp);
                        y1 = *reinterpret_cast<const float4 *>(yp + 4);
                    }
                    c[u][0][2 * q] = y0.x;
                    c[u][0][2 * q + 1] = y0.y;
                    c[u][1][2 * q] = y0.z;
                    c[u][1][2 * q + 1] = y0.w;
                    c[u][2][2 * q] = y1.x;
                    c[u][2][2 * q + 1] = y1.y;
                    c[u][3][2 * q] = y1.z;
                    c[u][3][2 * q + 1] = y1.w;
                }
            if (!waited) {
                pdl_wait();
                waited = true;
            }
            if (id >= 0) {
#pragma unroll
                for (int u = 0; u < RU; ++u)
#pragma unroll
                    for (int k = 0; k < NS; ++k) {
                        const int r = 32 * k + 8 * tq;
                        uint4 h[3][2];
#pragma unroll
                        for (int t = 0; t < 3; ++t)
#pragma unroll
                            for (int q = 0; q < 2; ++q)
                                h[t][q] = ok[u][q] && r < p.R
                                              ? __ldcg(reinterpret_cast<const uint4 *>(
                                                    a.h + ((size_t)t * a.M + row[u][q]) * p.R + r))
                                              : make_uint4(0, 0, 0, 0);
#pragma unroll
                        for (int j = 0; j < 4; ++j)
#pragma unroll
                            for (int t = 2; t >= 0; --t) // small parts first
                                mma32(c[u][j], h[t][0], h[t][1], b[k][j]);
                    }
            }
#pragma unroll
            for (int u = 0; u < RU; ++u)
#pragma unroll
                for (int q = 0; q < 2; ++q)
                    if (ok[u][q] && in) {
                        float *to = p.out + (a.m0 + row[u][q]) * (size_t)p.ldo + n0 + 8 * tq;
                        *reinterpret_cast<float4 *>(to) =
                            make_float4(c[u][0][2 * q], c[u][0][2 * q + 1], c[u][1][2 * q], c[u][1][2 * q + 1]);
                        *reinterpret_cast<float4 *>(to + 4) =
                            make_float4(c[u][2][2 * q], c[u][2][2 * q + 1], c[u][3][2 * q], c[u][3][2 * q + 1]);
                    }
        }
    }
    if (!waited)
        pdl_wait();
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

template <int TR, int NT>
cudaError_t down(Args a, int tiles, int num_sms, cudaStream_t s)
{
    constexpr int WK = kWarps / (TR / 16), SMEM = WK * TR * 8 * NT * 4;
    static std::atomic<unsigned long long> set{0};
    cudaError_t e = allow(lora_down_kernel<TR, NT>, SMEM, set);
    if (e != cudaSuccess)
        return e;
    // Blocks that share a tile: up to 8 (a portable cluster) while they are no more than
    // about two rounds of the SMs and each warp keeps a step of 32.
    a.parts = 1;
    while (a.parts < 8 && (long long)tiles * a.parts * 2 <= 4ll * num_sms && a.parts * WK * 32 < a.p.K)
        a.parts *= 2;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)a.parts;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(tiles * a.parts));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = SMEM;
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = a.parts > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, lora_down_kernel<TR, NT>, a);
}

template <int TR>
cudaError_t pass(const Args &a, int down_tiles, int up_tiles, int num_sms, cudaStream_t s)
{
    const int R = a.p.R;
    cudaError_t e;
    if (R <= 8)
        e = down<TR, 1>(a, down_tiles, num_sms, s);
    else if (R <= 16)
        e = down<TR, 2>(a, down_tiles, num_sms, s);
    else if (R <= 32)
        e = down<TR, 4>(a, down_tiles, num_sms, s);
    else if (R <= 64)
        e = down<TR, 8>(a, down_tiles, num_sms, s);
    else
        e = down<TR, 16>(a, down_tiles, num_sms, s);
    if (e != cudaSuccess)
        return e;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)up_tiles, (unsigned)((a.p.N + 32 * kWarps - 1) / (32 * kWarps)));
    cfg.blockDim = dim3(kThreads);
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (R <= 32)
        return cudaLaunchKernelEx(&cfg, lora_up_kernel<TR, 1>, a);
    if (R <= 64)
        return cudaLaunchKernelEx(&cfg, lora_up_kernel<TR, 2>, a);
    return cudaLaunchKernelEx(&cfg, lora_up_kernel<TR, 4>, a);
}

} // namespace

cudaError_t run_lora(const LoraArgs &p, float *ws, size_t ws_floats, int num_sms, cudaStream_t s)
{
    // Rows whose h fits the scratch go in one pass (53000 or so at R = 128).
    const long long most = (long long)(ws_floats * 4 / (6 * (size_t)p.R)) / 64 * 64;
    for (long long m0 = 0; m0 < p.M; m0 += most) {
        Args a = {};
        a.p = p;
        a.m0 = (int)m0;
        a.M = (int)(p.M - m0 < most ? p.M - m0 : most);
        a.h = reinterpret_cast<uint16_t *>(ws);
        cudaError_t e;
        if (a.M <= kGrouped) {
            // Each adapter has at most one tile that is not full.
            auto tiles = [&](long long ids) {
                const long long n = a.M / 16 + (ids < a.M ? ids : a.M);
                return (int)(n < a.M ? n : a.M);
            };
            e = pass<16>(a, tiles(p.L), tiles((long long)p.L + 1), num_sms, s);
        } else {
            const int tiles = (a.M + 63) / 64;
            e = pass<64>(a, tiles, tiles, num_sms, s);
        }
        if (e != cudaSuccess)
            return e;
    }
    return cudaSuccess;
}

} // namespace w4
