// Norms of the query and key heads and the position rotation in one pass, and the
// store of keys and values to the pages of a cache.
//
// Source: "Gemma 4 E2B on a 4 GB GPU with pure PyTorch" - the decode-attention and
// cache paragraphs (eight query heads on one key/value head, head widths 256 and
// 512): what lies between a layer's projections (fp32, w4a16_gemv and w4a16_gemm)
// and its attention (bf16).
//
// Mathematics. For a head x of width D with weight w:
//   u = x w / sqrt(mean x^2 + eps)                    (u = x without a weight)
//   (a, b) = (u_j, u_{j + R/2}) or (u_2j, u_{2j+1}), j < R / 2
//   (a, b) -> (a cos t - b sin t, b cos t + a sin t),  t = pos * freq_j
// Elements from R on pass unturned. Norm and turn in fp32, one rounding to bf16.
//
// The angle. pos * freq_j in fp32 would be off by 2^-24 of itself: 0.008 radians at
// position 131072. Turns are counted in integers instead: freq_j / 2 pi is formed as a
// 64-bit fraction of a turn (the fp32 frequency's 24-bit significand times 2^66 / 2 pi,
// shifted), and the 64-bit product with the position drops whole turns by itself.
// Its upper 32 bits are the angle, within 2^-32 of a turn for every position.
//
// Work. A group of D / 8 lanes (32 at most) has a token and some of its heads: the
// angles are formed once and serve all of them. A lane holds both halves of four
// pairs (8 elements, two 16-byte loads of fp32), so the turn needs no exchange and
// the norm only a sum over the group's lanes. Loads of kHeads heads are in flight.
// Bound by bytes: 6 per element (fp32 in).
#include "common.cuh"
#include "internal.h"

namespace w4 {

namespace {

constexpr int kThreads = 256;

// Fraction of a turn that freq radians are, in units of 2^-64 (whole turns drop out).
// freq = m 2^e with a 24-bit m; 2^66 / (2 pi) in 64 bits is 0xA2F9836E4E44152A
// (the leading bits of 2 / pi), so the fraction is m * that, shifted by e - 2.
__device__ __forceinline__ unsigned long long turn_of(float freq)
{
    const uint32_t b = __float_as_uint(freq);
    const int ex = (int)((b >> 23) & 0xFFu);
    const unsigned long long m = (b & 0x7FFFFFu) | (ex ? 0x800000u : 0u);
    const int s = 2 - ((ex ? ex : 1) - 150); // right shift of the 128-bit product
    const unsigned long long c = 0xA2F9836E4E44152Aull;
    const unsigned long long lo = m * c, hi = __umul64hi(m, c);
    unsigned long long f;
    if (s <= 0)
        f = s > -64 ? lo << -s : 0ull;
    else if (s < 64)
        f = (lo >> s) | (hi << (64 - s));
    else
        f = s < 128 ? hi >> (s - 64) : 0ull;
    return (b >> 31) ? 0ull - f : f;
}

template <bool F32>
__device__ __forceinline__ void load4(float (&x)[4], const void *p, long long at)
{
    if (F32) {
        const float4 v = __ldcs(reinterpret_cast<const float4 *>(static_cast<const float *>(p) + at));
        x[0] = v.x;
        x[1] = v.y;
        x[2] = v.z;
        x[3] = v.w;
    } else {
        const uint2 v = __ldcs(reinterpret_cast<const uint2 *>(static_cast<const uint16_t *>(p) + at));
        x[0] = __uint_as_float(v.x << 16);
        x[1] = __uint_as_float(v.x & 0xFFFF0000u);
        x[2] = __uint_as_float(v.y << 16);
        x[3] = __uint_as_float(v.y & 0xFFFF0000u);
    }
}

__device__ __forceinline__ void store4(uint16_t *p, const float (&x)[4])
{
    uint2 v;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(v.x) : "f"(x[1]), "f"(x[0]));
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(v.y) : "f"(x[3]), "f"(x[2]));
    *reinterpret_cast<uint2 *>(p) = v;
}

// LPH lanes share a head, each with CPL chunks of 8 elements.
template <int LPH, int CPL, bool F32, bool PAGED>
__global__ void __launch_bounds__(kThreads)
qk_norm_rope_kernel(const NormRopeArgs a, const int hp, const int split)
{
    constexpr int kHeads = CPL == 1 ? 4 : 2; // heads in flight
    const int sub = threadIdx.x & (LPH - 1);
    const long long item = (long long)blockIdx.x * (kThreads / LPH) + threadIdx.x / LPH;
    const int m = (int)min(item / split, (long long)a.M - 1);
    const bool mine = item < (long long)a.M * split;
    const int h0 = (int)(item % split) * hp, H = a.Hq + (PAGED ? 2 : 1) * a.Hkv;
    const int h1 = mine ? min(h0 + hp, H) : h0;
    const int nrot = a.R / 8, nchunk = a.D / 8;

    // This lane's chunks: offsets of their two halves within a head.
    int o0[CPL], o1[CPL];
    bool has[CPL], rot[CPL];
#pragma unroll
    for (int i = 0; i < CPL; ++i) {
        const int c = sub + LPH * i;
        has[i] = c < nchunk;
        rot[i] = c < nrot;
        const bool half = rot[i] && !a.pairs;
        o0[i] = half ? 4 * c : 8 * c;
        o1[i] = half ? 4 * c + a.R / 2 : 8 * c + 4;
    }
    // Frequencies are the caller's constants: read ahead of the preceding kernel's end.
    unsigned long long turn[CPL][4];
#pragma unroll
    for (int i = 0; i < CPL; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j)
            turn[i][j] = rot[i] ? turn_of(__ldg(a.inv_freq + 4 * (sub + LPH * i) + j)) : 0ull;

    pdl_launch_dependents();
    pdl_wait();

    // The token's position, and in a paged call its place.
    int pos;
    bool row = mine, keep = false; // a row of a sequence; stored to a page
    size_t at = 0;
    if (PAGED) {
        int s = m, q0 = m, q1 = m + 1;
        if (a.cu_q) {
            // The last sequence that begins at or before row m (empty ones begin where the next does).
            int x = 0, y = a.B - 1;
            while (x < y) {
                const int mid = (x + y + 1) >> 1;
                if (__ldg(a.cu_q + mid) <= m)
                    x = mid;
                else
                    y = mid - 1;
            }
            s = x;
            q0 = __ldg(a.cu_q + s);
            q1 = min(__ldg(a.cu_q + s + 1), a.M);
            row = mine && q0 >= 0 && m >= q0 && m < q1;
        }
        pos = max(__ldg(a.lens + s), 0) - q1 + m;
        const int slot = pos >= 0 ? pos >> a.page_log2 : a.table_pages;
        int pg = -1;
        if (row && slot < a.table_pages)
            pg = __ldg(a.table + (size_t)s * a.table_pages + slot);
        keep = pg >= 0 && pg < a.pages;
        at = keep ? (size_t)pg * a.page_stride + (size_t)(pos & ((1 << a.page_log2) - 1)) * a.row_stride : 0;
        if (row && !keep && a.status && sub == 0 && h1 > a.Hq)
            *a.status = 1;
    } else {
        pos = __ldg(a.pos + m);
    }
    float cs[CPL][4], sn[CPL][4];
#pragma unroll
    for (int i = 0; i < CPL; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const unsigned long long t = (unsigned long long)(long long)pos * turn[i][j];
            sincospif((float)(int32_t)(t >> 32) * 4.656612873077393e-10f, &sn[i][j], &cs[i][j]); // 2^-31
        }

    float w[CPL][8];
    const float *wp = nullptr;
    for (int hb = h0; hb < h0 + hp; hb += kHeads) {
        float x[kHeads][CPL][8];
#pragma unroll
        for (int u = 0; u < kHeads; ++u) {
            const int h = hb + u;
            const bool live = row && h < h1;
            const int kind = h < a.Hq ? 0 : (h < a.Hq + a.Hkv ? 1 : 2);
            const void *p = kind == 0 ? a.q : (kind == 1 ? a.k : a.v);
            const long long ld = kind == 0 ? a.ldq : (kind == 1 ? a.ldk : a.ldv);
            const long long from = (long long)m * ld + (long long)(h - (kind == 0 ? 0 : (kind == 1 ? a.Hq : a.Hq + a.Hkv))) * a.D;
#pragma unroll
            for (int i = 0; i < CPL; ++i) {
                float (&lo)[4] = *reinterpret_cast<float (*)[4]>(&x[u][i][0]);
                float (&hi)[4] = *reinterpret_cast<float (*)[4]>(&x[u][i][4]);
                const bool turned = kind < 2; // values lie in order
                if (live && has[i]) {
                    load4<F32>(lo, p, from + (turned ? o0[i] : 8 * (sub + LPH * i)));
                    load4<F32>(hi, p, from + (turned ? o1[i] : 8 * (sub + LPH * i) + 4));
                } else {
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        x[u][i][j] = 0.f;
                }
            }
        }
#pragma unroll
        for (int u = 0; u < kHeads; ++u) {
            const int h = hb + u;
            const bool live = row && h < h1;
            const int kind = h < a.Hq ? 0 : (h < a.Hq + a.Hkv ? 1 : 2);
            const float *wk = kind == 0 ? a.q_weight : (kind == 1 ? a.k_weight : a.v_weight);
            float ss = 0.f;
#pragma unroll
            for (int i = 0; i < CPL; ++i)
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    ss = fmaf(x[u][i][j], x[u][i][j], ss);
#pragma unroll
            for (int d = LPH / 2; d; d >>= 1)
                ss += __shfl_xor_sync(0xFFFFFFFFu, ss, d);
            if (!live)
                continue;
            if (wk) {
                if (wk != wp) {
                    wp = wk;
#pragma unroll
                    for (int i = 0; i < CPL; ++i)
                        if (has[i]) {
                            const int c = 8 * (sub + LPH * i);
                            const float4 f0 = __ldg(reinterpret_cast<const float4 *>(wk + (kind < 2 ? o0[i] : c)));
                            const float4 f1 = __ldg(reinterpret_cast<const float4 *>(wk + (kind < 2 ? o1[i] : c + 4)));
                            w[i][0] = f0.x;
                            w[i][1] = f0.y;
                            w[i][2] = f0.z;
                            w[i][3] = f0.w;
                            w[i][4] = f1.x;
                            w[i][5] = f1.y;
                            w[i][6] = f1.z;
                            w[i][7] = f1.w;
                        }
                }
                const float r = rsqrtf(ss / (float)a.D + a.eps);
#pragma unroll
                for (int i = 0; i < CPL; ++i)
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        x[u][i][j] = has[i] ? x[u][i][j] * r * w[i][j] : 0.f;
            }
            uint16_t *to;
            if (kind == 0)
                to = a.q_out + (long long)m * a.ldqo + (long long)h * a.D;
            else if (PAGED)
                to = (kind == 1 ? a.k_pages : a.v_pages) + at + (size_t)(h - a.Hq - (kind == 1 ? 0 : a.Hkv)) * a.head_stride;
            else
                to = a.k_out + (long long)m * a.ldko + (long long)(h - a.Hq) * a.D;
            if (kind > 0 && PAGED && !keep)
                continue;
#pragma unroll
            for (int i = 0; i < CPL; ++i) {
                if (!has[i])
                    continue;
                float lo[4], hi[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    lo[j] = x[u][i][j];
                    hi[j] = x[u][i][4 + j];
                }
                int p0 = o0[i], p1 = o1[i];
                if (kind == 2) {
                    p0 = 8 * (sub + LPH * i);
                    p1 = p0 + 4;
                } else if (rot[i]) {
                    if (a.pairs) {
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            const float e = x[u][i][2 * j], o = x[u][i][2 * j + 1];
                            const float n0 = e * cs[i][j] - o * sn[i][j], n1 = o * cs[i][j] + e * sn[i][j];
                            if (j < 2) {
                                lo[2 * j] = n0;
                                lo[2 * j + 1] = n1;
                            } else {
                                hi[2 * j - 4] = n0;
                                hi[2 * j - 3] = n1;
                            }
                        }
                    } else {
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            const float e = x[u][i][j], o = x[u][i][4 + j];
                            lo[j] = e * cs[i][j] - o * sn[i][j];
                            hi[j] = o * cs[i][j] + e * sn[i][j];
                        }
                    }
                }
                store4(to + p0, lo);
                store4(to + p1, hi);
            }
        }
    }
}

template <int LPH, int CPL>
cudaError_t launch(const NormRopeArgs &a, int num_sms, cudaStream_t s)
{
    const bool paged = a.k_pages != nullptr;
    const int H = a.Hq + (paged ? 2 : 1) * a.Hkv;
    // Heads of a token are shared by more groups until there are two blocks per SM.
    constexpr int per = kThreads / LPH;
    int hp = H;
    auto blocks = [&] { return ((long long)a.M * ((H + hp - 1) / hp) + per - 1) / per; };
    while (hp > 1 && blocks() < 2ll * num_sms)
        hp = (hp + 1) / 2;
    if (blocks() > 0x7FFFFFFFll)
        return cudaErrorNotSupported;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)blocks());
    cfg.blockDim = dim3(kThreads);
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const int split = (H + hp - 1) / hp;
    auto go = [&](auto kern) { return cudaLaunchKernelEx(&cfg, kern, a, hp, split); };
    if (a.f32)
        return paged ? go(qk_norm_rope_kernel<LPH, CPL, true, true>) : go(qk_norm_rope_kernel<LPH, CPL, true, false>);
    return paged ? go(qk_norm_rope_kernel<LPH, CPL, false, true>) : go(qk_norm_rope_kernel<LPH, CPL, false, false>);
}

} // namespace

cudaError_t run_qk_norm_rope(const NormRopeArgs &a, int num_sms, cudaStream_t s)
{
    switch (a.D) {
    case 64: return launch<8, 1>(a, num_sms, s);
    case 128: return launch<16, 1>(a, num_sms, s);
    case 256: return launch<32, 1>(a, num_sms, s);
    case 384:
    case 512: return launch<32, 2>(a, num_sms, s);
    default: return cudaErrorNotSupported;
    }
}

} // namespace w4
