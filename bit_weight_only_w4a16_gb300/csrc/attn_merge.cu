// Merge of the tiled attention's partial sums.
//
// A row tile that the equal cut of the work left to several CTAs has, for each
// of them, an accumulator O_p (fp32), a reference m_p and a sum l_p per row:
//   out = sum_p O_p 2^(m_p - M) / sum_p l_p 2^(m_p - M),  M = max_p m_p,
// added in the order of the keys. Reads 4 DV bytes per row and partial, written
// shortly before by the attention kernel. 150 cut tiles of two partials each (39 MB)
// take 15 us, 152 partials of two tiles (20 MB) 13 us: finding a block's tile and its
// partials costs 2 us, so blocks are few and take many rows; a long chain is shared
// among threads instead.
#include "attn_launch.cuh"

namespace w4 {
namespace attn {

namespace {

constexpr int kThreads = 512;
constexpr int kMaxCtas = 512;
constexpr int kMaxRows = 128; // rows per block
constexpr int kBatch = 10;    // partials in flight per thread when threads share an item, 4 else

// Block (x, y): the x-th cut row tile, its rows [y rb, y rb + rb). An item is four
// columns of a row. When a block has fewer items than threads, `groups` threads
// share an item: each takes every groups-th partial, and their sums are added in
// the order of the groups.
// SHARED: such a block (one per SM, many loads per thread); else two blocks per SM.
template <bool SHARED>
__global__ void __launch_bounds__(kThreads, SHARED ? 1 : 2)
merge_kernel(const MergeArgs a)
{
    extern __shared__ float4 s_part[];  // [groups - 1][items], then weights [partials][rb]
    __shared__ int s_first, s_end, s_warp[kThreads / 32];
    __shared__ float s_inv[kMaxRows];
    pdl_wait();
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    // The CTA that begins the x-th cut tile.
    if (threadIdx.x == 0) {
        s_first = -1;
        s_end = a.ctas;
    }
    const int c = threadIdx.x; // kMaxCtas <= kThreads
    const int2 rec = c < a.ctas ? *reinterpret_cast<const int2 *>(a.rec + 2 * c) : make_int2(0, 0);
    const uint32_t v = __ballot_sync(0xFFFFFFFFu, rec.y != 0);
    if (lane == 0)
        s_warp[w] = __popc(v);
    __syncthreads();
    int before = __popc(v & ((1u << lane) - 1u));
    for (int i = 0; i < kThreads / 32; ++i)
        before += i < w ? s_warp[i] : 0;
    if (rec.y != 0 && before == (int)blockIdx.x)
        s_first = c;
    __syncthreads();
    const int first = s_first;
    if (first < 0)
        return;
    // The tile goes on in the CTAs after it up to the one that ends it.
    if (c > first && rec.x != 1)
        atomicMin(&s_end, rec.x == 3 ? c + 1 : c);
    __syncthreads();
    const int n = s_end - first, r0 = (int)blockIdx.y * a.rb;
    const int32_t *at = a.where + 4 * first;
    const int tok0 = at[0], nt = at[1], kvh = at[2], slice = at[3];
    // Partial p is slot 2 first + 1 for p = 0, else 2 (first + p).
    auto slot = [&](int p) { return p == 0 ? 2 * first + 1 : 2 * (first + p); };
    const int cols = a.DV / 4, items = a.rb * cols;
    const int groups = SHARED ? kThreads / items : 1;
    float *s_w = reinterpret_cast<float *>(s_part + (size_t)(groups - 1) * items);

    // Where item i's columns lie in a partial, and its output (null: not a row).
    const int rmask = a.rb - 1, rshift = __ffs(a.rb) - 1; // rb is a power of two
    auto offset = [&](int i) { return ((size_t)(i >> rshift) * a.rows_per_tile + r0 + (i & rmask)) * 4; };
    auto target = [&](int i) -> uint16_t * {
        const int row = r0 + (i & rmask), t = row / kRowsQ, in = row - t * kRowsQ;
        const int ti = in / a.G, tok = t * a.tpt + ti;
        if (i >= items || ti >= a.tpt || tok >= nt)
            return nullptr;
        return a.out + (size_t)(tok0 + tok) * a.ldo + (size_t)(kvh * a.G + in - ti * a.G) * a.D + slice * a.DV +
               4 * (i >> rshift);
    };
    auto load = [&](int p, size_t off) {
        return __ldcg(reinterpret_cast<const float4 *>(a.ws_o + (size_t)slot(p) * kSlotFloats + off));
    };
    auto add = [&](float4 &o, const float4 &x, float f) {
        o.x = fmaf(x.x, f, o.x);
        o.y = fmaf(x.y, f, o.y);
        o.z = fmaf(x.z, f, o.z);
        o.w = fmaf(x.w, f, o.w);
    };
    auto store = [&](uint16_t *to, const float4 &o, float f) {
        uint2 y;
        y.x = pack2(o.x * f, o.y * f);
        y.y = pack2(o.z * f, o.w * f);
        *reinterpret_cast<uint2 *>(to) = y;
    };
    // Threads that share items ask for their first partials before the weights.
    const int i = SHARED ? (int)threadIdx.x % items : 0, grp = SHARED ? (int)threadIdx.x / items : 0;
    uint16_t *to0 = SHARED && grp < groups ? target(i) : nullptr;
    const size_t off0 = offset(i);
    float4 x0[SHARED ? kBatch : 1];
    if (SHARED) {
#pragma unroll
        for (int q = 0; q < kBatch; ++q) {
            const int p = grp + q * groups;
            x0[q] = to0 && p < n ? load(p, off0) : make_float4(0.f, 0.f, 0.f, 0.f);
        }
    }
    // Weights 2^(m_p - M) and the inverse of the sum: a thread per row for a short
    // chain, a warp per row for a long one.
    auto ml_of = [&](int p, int r) {
        return __ldcg(reinterpret_cast<const float2 *>(a.ws_ml + ((size_t)slot(p) * 256 + r0 + r) * 2));
    };
    if (n <= kBatch) {
        if ((int)threadIdx.x < a.rb) {
            float2 ml[kBatch];
#pragma unroll
            for (int p = 0; p < kBatch; ++p)
                ml[p] = p < n ? ml_of(p, threadIdx.x) : make_float2(-INFINITY, 0.f);
            float M = -INFINITY, L = 0.f;
#pragma unroll
            for (int p = 0; p < kBatch; ++p)
                M = fmaxf(M, ml[p].x);
#pragma unroll
            for (int p = 0; p < kBatch; ++p) {
                const float f = ml[p].x == -INFINITY ? 0.f : ex2(ml[p].x - M);
                if (p < n)
                    s_w[p * a.rb + threadIdx.x] = f;
                L += f * ml[p].y;
            }
            s_inv[threadIdx.x] = L == 0.f ? 0.f : 1.f / L;
        }
    } else {
        for (int r = w; r < a.rb; r += kThreads / 32) {
            float M = -INFINITY, L = 0.f;
            float2 ml[kMaxCtas / 32];
#pragma unroll
            for (int q = 0; q < kMaxCtas / 32; ++q) {
                const int p = lane + 32 * q;
                ml[q] = p < n ? ml_of(p, r) : make_float2(-INFINITY, 0.f);
            }
#pragma unroll
            for (int q = 0; q < kMaxCtas / 32; ++q)
                M = fmaxf(M, ml[q].x);
            for (int d = 16; d; d >>= 1)
                M = fmaxf(M, __shfl_xor_sync(0xFFFFFFFFu, M, d));
#pragma unroll
            for (int q = 0; q < kMaxCtas / 32; ++q) {
                const int p = lane + 32 * q;
                const float f = ml[q].x == -INFINITY ? 0.f : ex2(ml[q].x - M);
                if (p < n)
                    s_w[p * a.rb + r] = f;
                L += f * ml[q].y;
            }
            for (int d = 16; d; d >>= 1)
                L += __shfl_xor_sync(0xFFFFFFFFu, L, d);
            if (lane == 0)
                s_inv[r] = L == 0.f ? 0.f : 1.f / L;
        }
    }
    __syncthreads();

    if (!SHARED) {
        for (int i = threadIdx.x; i < items; i += kThreads) {
            uint16_t *to = target(i);
            if (!to)
                continue;
            const size_t off = offset(i);
            float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
            for (int p0 = 0; p0 < n; p0 += 4) {
                float4 x[4];
#pragma unroll
                for (int q = 0; q < 4; ++q)
                    x[q] = p0 + q < n ? load(p0 + q, off) : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
                for (int q = 0; q < 4; ++q)
                    add(o, x[q], p0 + q < n ? s_w[(p0 + q) * a.rb + (i & rmask)] : 0.f);
            }
            store(to, o, s_inv[i & rmask]);
        }
        return;
    }
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    if (to0) {
        for (int p0 = grp; p0 < n; p0 += kBatch * groups) {
            float4 x[kBatch];
#pragma unroll
            for (int q = 0; q < kBatch; ++q) {
                const int p = p0 + q * groups;
                if (p0 == grp)
                    x[q] = x0[q];
                else
                    x[q] = p < n ? load(p, off0) : make_float4(0.f, 0.f, 0.f, 0.f);
            }
#pragma unroll
            for (int q = 0; q < kBatch; ++q) {
                const int p = p0 + q * groups;
                add(o, x[q], p < n ? s_w[p * a.rb + (i & rmask)] : 0.f);
            }
        }
    }
    if (grp > 0 && grp < groups)
        s_part[(grp - 1) * items + i] = o;
    __syncthreads();
    if (grp == 0 && to0) {
        for (int q = 1; q < groups; ++q)
            add(o, s_part[(q - 1) * items + i], 1.f);
        store(to0, o, s_inv[i & rmask]);
    }
}

} // namespace

cudaError_t run_merge(const MergeArgs &m0, int tiles, cudaStream_t s)
{
    MergeArgs m = m0;
    static_assert(kMaxCtas <= kThreads, "one thread per CTA");
    if (m.ctas > kMaxCtas)
        return cudaErrorInvalidValue;
    // Rows per block: about one block per SM if every tile is cut (finding the tile
    // and its partials takes a block 2 us); two rows at least (32 contiguous bytes of a
    // partial).
    m.rb = 2;
    while (m.rb < kMaxRows && (long long)tiles * (m.rows_per_tile / m.rb) > m.ctas)
        m.rb <<= 1;
    const int items = m.rb * (m.DV / 4), groups = items < kThreads ? kThreads / items : 1;
    const size_t smem = (size_t)(groups - 1) * items * sizeof(float4) + (size_t)m.ctas * m.rb * sizeof(float);
    // Once per device: up to kMaxRows weights for each CTA's partial.
    static std::atomic<unsigned long long> set{0};
    constexpr int kSmem = 16 * kThreads + 4 * kMaxRows * 256; // 136 KiB: 256 partials of 128 rows
    if (smem > (size_t)kSmem)
        return cudaErrorInvalidValue;
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess)
        return e;
    if (dev >= 64 || !((set.load(std::memory_order_relaxed) >> dev) & 1)) {
        e = cudaFuncSetAttribute(merge_kernel<false>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
        if (e == cudaSuccess)
            e = cudaFuncSetAttribute(merge_kernel<true>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
        if (e != cudaSuccess)
            return e;
        if (dev < 64)
            set.fetch_or(1ull << dev, std::memory_order_relaxed);
    }
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(tiles, m.rows_per_tile / m.rb);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return groups > 1 ? cudaLaunchKernelEx(&cfg, merge_kernel<true>, m) : cudaLaunchKernelEx(&cfg, merge_kernel<false>, m);
}

} // namespace attn

size_t attn_ws_floats(int num_sms) { return attn::ws_need(num_sms); }

} // namespace w4
