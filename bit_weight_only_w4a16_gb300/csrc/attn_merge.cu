// Merge of the tiled attention's partial sums.
//
// A row tile that the equal cut of the work left to several CTAs has, for each
// of them, an accumulator O_p (fp32), a reference m_p and a sum l_p per row:
//   out = sum_p O_p 2^(m_p - M) / sum_p l_p 2^(m_p - M),  M = max_p m_p,
// added in the order of the keys. Reads 4 DV bytes per row and partial, written
// shortly before by the attention kernel: they come from L2.
#include "attn_launch.cuh"

namespace w4 {
namespace attn {

namespace {

constexpr int kThreads = 512;
constexpr int kMaxCtas = 512;
constexpr int kMaxRows = 32; // rows per block

// Block (x, y): the x-th cut row tile, its rows [y rb, y rb + rb). An item is four
// columns of a row. When a block has fewer items than threads, `groups` threads
// share an item: each takes every groups-th partial, and their sums are added in
// the order of the groups.
__global__ void __launch_bounds__(kThreads)
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
    const int groups = items < kThreads ? kThreads / items : 1;
    float *s_w = reinterpret_cast<float *>(s_part + (size_t)(groups - 1) * items);

    // Weights 2^(m_p - M) and the inverse of the sum; one warp per row.
    for (int r = w; r < a.rb; r += kThreads / 32) {
        float M = -INFINITY, L = 0.f;
        for (int p = lane; p < n; p += 32)
            M = fmaxf(M, a.ws_ml[((size_t)slot(p) * 256 + r0 + r) * 2]);
        for (int d = 16; d; d >>= 1)
            M = fmaxf(M, __shfl_xor_sync(0xFFFFFFFFu, M, d));
        for (int p = lane; p < n; p += 32) {
            const float2 ml = *reinterpret_cast<const float2 *>(a.ws_ml + ((size_t)slot(p) * 256 + r0 + r) * 2);
            const float f = ml.x == -INFINITY ? 0.f : ex2(ml.x - M);
            s_w[p * a.rb + r] = f;
            L += f * ml.y;
        }
        for (int d = 16; d; d >>= 1)
            L += __shfl_xor_sync(0xFFFFFFFFu, L, d);
        if (lane == 0)
            s_inv[r] = L == 0.f ? 0.f : 1.f / L;
    }
    __syncthreads();

    for (int i0 = 0; i0 < items; i0 += kThreads) {
        const int i = groups > 1 ? (int)threadIdx.x % items : i0 + (int)threadIdx.x;
        const int grp = groups > 1 ? (int)threadIdx.x / items : 0;
        const bool mine = i < items && grp < groups;
        const int rr = i % a.rb, c4 = i / a.rb, row = r0 + rr;
        const int t = row / kRowsQ, in = row - t * kRowsQ;
        const int tok = t * a.tpt + in / a.G;
        const bool live = mine && in / a.G < a.tpt && tok < nt;
        float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
        if (live) {
            const size_t off = ((size_t)c4 * a.rows_per_tile + row) * 4;
#pragma unroll 8
            for (int p = grp; p < n; p += groups) {
                const float4 x = __ldcg(reinterpret_cast<const float4 *>(a.ws_o + (size_t)slot(p) * kSlotFloats + off));
                const float f = s_w[p * a.rb + rr];
                o.x = fmaf(x.x, f, o.x);
                o.y = fmaf(x.y, f, o.y);
                o.z = fmaf(x.z, f, o.z);
                o.w = fmaf(x.w, f, o.w);
            }
        }
        if (groups > 1) {
            if (mine && grp > 0)
                s_part[(grp - 1) * items + i] = o;
            __syncthreads();
            if (grp == 0)
                for (int q = 1; q < groups; ++q) {
                    const float4 x = s_part[(q - 1) * items + i];
                    o.x += x.x;
                    o.y += x.y;
                    o.z += x.z;
                    o.w += x.w;
                }
        }
        if (live && grp == 0) {
            const float f = s_inv[rr];
            uint2 y;
            y.x = pack2(o.x * f, o.y * f);
            y.y = pack2(o.z * f, o.w * f);
            *reinterpret_cast<uint2 *>(a.out + (size_t)(tok0 + tok) * a.ldo +
                                       (size_t)(kvh * a.G + in % a.G) * a.D + slice * a.DV + 4 * c4) = y;
        }
    }
}

} // namespace

cudaError_t run_merge(const MergeArgs &m0, int tiles, cudaStream_t s)
{
    MergeArgs m = m0;
    static_assert(kMaxCtas <= kThreads, "one thread per CTA");
    if (m.ctas > kMaxCtas)
        return cudaErrorInvalidValue;
    // Rows per block: about four blocks per SM if every tile is cut; two at least
    // (32 contiguous bytes of a partial).
    m.rb = 2;
    while (m.rb < kMaxRows && (long long)tiles * (m.rows_per_tile / m.rb) > 4 * m.ctas)
        m.rb <<= 1;
    const int items = m.rb * (m.DV / 4), groups = items < kThreads ? kThreads / items : 1;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(tiles, m.rows_per_tile / m.rb);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = (size_t)(groups - 1) * items * sizeof(float4) + (size_t)m.ctas * m.rb * sizeof(float);
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, merge_kernel, m);
}

} // namespace attn

size_t attn_ws_floats(int num_sms) { return attn::ws_need(num_sms); }

} // namespace w4
