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

constexpr int kThreads = 256;
constexpr int kMaxCtas = 512;

// Block (x, y): the x-th cut row tile, its rows [y rb, y rb + rb).
__global__ void __launch_bounds__(kThreads)
merge_kernel(const MergeArgs a)
{
    extern __shared__ float s_w[]; // [partials][rb] weights
    __shared__ int s_first, s_n, s_warp[kThreads / 32];
    __shared__ float s_inv[8];
    pdl_wait();
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    // The CTA that begins the x-th cut tile.
    if (threadIdx.x == 0)
        s_first = -1;
    int seen = 0;
    for (int c0 = 0; c0 < a.ctas; c0 += kThreads) {
        const int c = c0 + (int)threadIdx.x;
        const bool b = c < a.ctas && a.rec[2 * c + 1] != 0;
        const uint32_t v = __ballot_sync(0xFFFFFFFFu, b);
        __syncthreads();
        if (lane == 0)
            s_warp[w] = __popc(v);
        __syncthreads();
        int before = seen;
        for (int i = 0; i < kThreads / 32; ++i) {
            before += i < w ? s_warp[i] : 0;
            seen += s_warp[i];
        }
        if (b && before + __popc(v & ((1u << lane) - 1u)) == (int)blockIdx.x)
            s_first = c;
    }
    __syncthreads();
    const int first = s_first;
    if (first < 0)
        return;
    if (threadIdx.x == 0) {
        int n = 1;
        while (first + n < a.ctas && a.rec[2 * (first + n)] == 1)
            ++n;
        s_n = first + n < a.ctas && a.rec[2 * (first + n)] == 3 ? n + 1 : n;
    }
    __syncthreads();
    const int n = s_n, r0 = (int)blockIdx.y * a.rb;
    const int32_t *at = a.where + 4 * first;
    const int tok0 = at[0], nt = at[1], kvh = at[2], slice = at[3];
    // Partial p is slot 2 first + 1 for p = 0, else 2 (first + p).
    auto slot = [&](int p) { return p == 0 ? 2 * first + 1 : 2 * (first + p); };

    // Weights 2^(m_p - M) and the inverse of the sum; one warp per row.
    for (int r = w; r < a.rb; r += kThreads / 32) {
        float M = -INFINITY, L = 0.f;
        for (int p = lane; p < n; p += 32)
            M = fmaxf(M, a.ws_ml[((size_t)slot(p) * 256 + r0 + r) * 2]);
        for (int d = 16; d; d >>= 1)
            M = fmaxf(M, __shfl_xor_sync(0xFFFFFFFFu, M, d));
        for (int p = lane; p < n; p += 32) {
            const float *ml = a.ws_ml + ((size_t)slot(p) * 256 + r0 + r) * 2;
            const float f = ml[0] == -INFINITY ? 0.f : ex2(ml[0] - M);
            s_w[p * a.rb + r] = f;
            L += f * ml[1];
        }
        for (int d = 16; d; d >>= 1)
            L += __shfl_xor_sync(0xFFFFFFFFu, L, d);
        if (lane == 0)
            s_inv[r] = L == 0.f ? 0.f : 1.f / L;
    }
    __syncthreads();

    for (int i = threadIdx.x; i < a.rb * (a.DV / 4); i += kThreads) {
        const int rr = i % a.rb, c4 = i / a.rb, row = r0 + rr;
        const int t = row / kRowsQ, in = row - t * kRowsQ;
        const int tok = t * a.tpt + in / a.G;
        if (in / a.G >= a.tpt || tok >= nt)
            continue;
        float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
        const size_t off = ((size_t)c4 * a.rows_per_tile + row) * 4;
#pragma unroll 8
        for (int p = 0; p < n; ++p) {
            const float4 v = *reinterpret_cast<const float4 *>(a.ws_o + (size_t)slot(p) * kSlotFloats + off);
            const float f = s_w[p * a.rb + rr];
            o.x = fmaf(v.x, f, o.x);
            o.y = fmaf(v.y, f, o.y);
            o.z = fmaf(v.z, f, o.z);
            o.w = fmaf(v.w, f, o.w);
        }
        const float f = s_inv[rr];
        uint2 y;
        y.x = pack2(o.x * f, o.y * f);
        y.y = pack2(o.z * f, o.w * f);
        *reinterpret_cast<uint2 *>(a.out + (size_t)(tok0 + tok) * a.ldo +
                                   (size_t)(kvh * a.G + in % a.G) * a.D + slice * a.DV + 4 * c4) = y;
    }
}

} // namespace

cudaError_t run_merge(const MergeArgs &m0, int tiles, cudaStream_t s)
{
    MergeArgs m = m0;
    if (m.ctas > kMaxCtas)
        return cudaErrorInvalidValue;
    // Rows per block: about two blocks per SM when few tiles are cut.
    m.rb = 8;
    while (m.rb > 1 && (long long)tiles * (m.rows_per_tile / m.rb) < 2 * m.ctas)
        m.rb >>= 1;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(tiles, m.rows_per_tile / m.rb);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = (size_t)m.ctas * m.rb * sizeof(float);
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, merge_kernel, m);
}

} // namespace attn

size_t attn_ws_floats(int num_sms) { return attn::ws_need(num_sms); }

} // namespace w4
