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
// 64-bit fraction of a turn (the fp32 frequency's 24-bit significand times 96 bits of
// 1 / 2 pi, shifted; 64 bits of it left 2^-17 of a turn at frequencies near 2^24), and the
// 64-bit product with the position drops whole turns by itself. Its upper 32 bits are the
// angle, within 2^-31 of a turn for every position and frequency below 2^24; in half turns
// as fp32 it is within 2^-26 of a turn, fp32's own step near a half turn.
//
// Work. A group of D / 8 lanes (32 at most) has a token and some of its heads; a lane holds
// both halves of four pairs (8 elements, two 16-byte loads of fp32), so the turn needs no
// exchange and the norm only a sum over the group's lanes. What is the same for all heads
// is formed once: frequencies per group, angles per token, and per token and kind of head
// the products of weight and cosine or sine, so that a head costs six operations per pair.
// (With weights, angles and addresses formed per head the kernel took 270 instructions a
// head and 32 us for 8001 tokens.) Bound by bytes: 6 per element (fp32 in).
#include "common.cuh"
#include "internal.h"

#include <type_traits>

namespace w4 {

namespace {

constexpr int kThreads = 256;

// Fraction of a turn that freq radians are, in units of 2^-64 (whole turns drop out).
// freq = m 2^e with a 24-bit m; 2^66 / (2 pi) is 0xA2F9836E4E441529.FC2757D1 (the leading
// bits of 2 / pi), so the fraction is m * that, shifted by e - 2.
__device__ __forceinline__ unsigned long long turn_of(float freq)
{
    const uint32_t b = __float_as_uint(freq);
    const int ex = (int)((b >> 23) & 0xFFu);
    const uint32_t m = (b & 0x7FFFFFu) | (ex ? 0x800000u : 0u);
    const int s = 2 - ((ex ? ex : 1) - 150); // right shift of the 128-bit product
    // In words of 32 bits, none of whose sums overflows; what is below the point loses its last word.
    const unsigned long long p0 = (unsigned long long)m * 0x4E441529u + __umulhi(m, 0xFC2757D1u);
    const unsigned long long p1 = (unsigned long long)m * 0xA2F9836Eu + (p0 >> 32);
    const unsigned long long lo = (p1 << 32) | (uint32_t)p0, hi = p1 >> 32;
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

template <int D>
struct RopeShape {
    static constexpr int CHUNKS = D / 8;                       // of 8 elements
    static constexpr int LPH = CHUNKS < 32 ? CHUNKS : 32;      // lanes of a head
    static constexpr int CPL = (CHUNKS + LPH - 1) / LPH;       // chunks of a lane
    static constexpr bool FULL = CHUNKS % LPH == 0;            // every lane has all of its chunks
    // Heads in flight, and as many ahead: what 128 registers hold (8001 tokens of 9 heads of 256: 22 us
    // with 3, 26 with 4, 24 with 2).
    static constexpr int HEADS = CPL == 1 ? 3 : 1;
};

template <int D, bool F32, bool PAGED, bool PAIRS>
__global__ void __launch_bounds__(kThreads, 2)
qk_norm_rope_kernel(const NormRopeArgs a, const int hp, const int split)
{
    using S = RopeShape<D>;
    constexpr int LPH = S::LPH, CPL = S::CPL, NH = S::HEADS, PER = kThreads / LPH;
    const int sub = threadIdx.x & (LPH - 1);
    const int H = a.Hq + (PAGED ? 2 : 1) * a.Hkv, nrot = a.R / 8;

    // This lane's chunks: offsets of their two halves within a head.
    int o0[CPL], o1[CPL];
    bool has[CPL], rot[CPL];
    float freq[CPL][4];
    unsigned long long turn[CPL][4];
    bool first = true;
    pdl_launch_dependents();
    pdl_wait();
#pragma unroll
    for (int i = 0; i < CPL; ++i) {
        const int c = sub + LPH * i;
        has[i] = S::FULL || c < S::CHUNKS;
        rot[i] = c < nrot;
        const bool half = rot[i] && !PAIRS;
        o0[i] = half ? 4 * c : 8 * c;
        o1[i] = half ? 4 * c + a.R / 2 : 8 * c + 4;
#pragma unroll
        for (int j = 0; j < 4; ++j)
            freq[i][j] = rot[i] ? __ldg(a.inv_freq + 4 * c + j) : 0.f;
    }

    const long long items = (long long)a.M * split;
    // All lanes of a warp go round together (their sums are exchanged).
    for (long long it0 = (long long)blockIdx.x * PER; it0 < items; it0 += (long long)gridDim.x * PER) {
        const long long item = it0 + threadIdx.x / LPH;
        const bool mine = item < items;
        const int m = mine ? (int)(item / split) : 0;
        const int h0 = mine ? (int)(item - (long long)m * split) * hp : 0, h1 = mine ? min(h0 + hp, H) : 0;

        // Heads h .. h + NH - 1 of the token.
        auto load = [&](float (&x)[NH][CPL][8], int hb) {
#pragma unroll
            for (int u = 0; u < NH; ++u) {
                const int h = hb + u;
                const bool isq = h < a.Hq, isk = h < a.Hq + a.Hkv;
                const void *p = isq ? a.q : (isk ? a.k : a.v);
                const long long ld = isq ? a.ldq : (isk ? a.ldk : a.ldv);
                const long long from = (long long)m * ld + (h - (isq ? 0 : (isk ? a.Hq : a.Hq + a.Hkv))) * D;
#pragma unroll
                for (int i = 0; i < CPL; ++i) {
                    if (h < h1 && has[i]) {
                        load4<F32>(*reinterpret_cast<float (*)[4]>(&x[u][i][0]), p, from + o0[i]);
                        load4<F32>(*reinterpret_cast<float (*)[4]>(&x[u][i][4]), p, from + o1[i]);
                    } else {
#pragma unroll
                        for (int j = 0; j < 8; ++j)
                            x[u][i][j] = 0.f;
                    }
                }
            }
        };
        float xa[NH][CPL][8], xb[NH][CPL][8];
        load(xa, h0);

        // The token's position, and in a paged call its place.
        int pos;
        bool row = mine, keep = false; // a row of a sequence; stored to a page
        size_t at = 0;
        if (PAGED) {
            int s = m, q1 = m + 1;
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
                const int q0 = __ldg(a.cu_q + s);
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
        if (first) { // with the first loads on their way
            first = false;
#pragma unroll
            for (int i = 0; i < CPL; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    turn[i][j] = turn_of(freq[i][j]);
        }
        float cs[CPL][4], sn[CPL][4];
#pragma unroll
        for (int i = 0; i < CPL; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const unsigned long long t = (unsigned long long)(long long)pos * turn[i][j];
                sincospif((float)(int32_t)(t >> 32) * 4.656612873077393e-10f, &sn[i][j], &cs[i][j]); // 2^-31
            }
        // Of the present kind of head: element e of pair j is multiplied by ec[j] and es[j], o by oc[j]
        // and os[j]: weight times cosine and sine (1 and 0 where nothing is turned).
        float ec[CPL][4], es[CPL][4], oc[CPL][4], os[CPL][4];
        int kind_now = -1;
        bool normed = false;
        auto process = [&](float (&x)[NH][CPL][8], int hb) {
#pragma unroll
            for (int u = 0; u < NH; ++u) {
                const int h = hb + u;
                const int kind = h < a.Hq ? 0 : (h < a.Hq + a.Hkv ? 1 : 2);
                float ss = 0.f;
#pragma unroll
                for (int i = 0; i < CPL; ++i)
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        ss = fmaf(x[u][i][j], x[u][i][j], ss);
#pragma unroll
                for (int k = LPH / 2; k; k >>= 1)
                    ss += __shfl_xor_sync(0xFFFFFFFFu, ss, k);
                if (!row || h >= h1)
                    continue;
                if (kind != kind_now) {
                    kind_now = kind;
                    const float *wk = kind == 0 ? a.q_weight : (kind == 1 ? a.k_weight : a.v_weight);
                    normed = wk != nullptr;
#pragma unroll
                    for (int i = 0; i < CPL; ++i) {
                        float4 w0 = make_float4(1.f, 1.f, 1.f, 1.f), w1 = w0;
                        if (wk && has[i]) {
                            w0 = __ldg(reinterpret_cast<const float4 *>(wk + o0[i]));
                            w1 = __ldg(reinterpret_cast<const float4 *>(wk + o1[i]));
                        }
                        const float w[8] = {w0.x, w0.y, w0.z, w0.w, w1.x, w1.y, w1.z, w1.w};
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            const float we = w[PAIRS ? 2 * j : j], wo = w[PAIRS ? 2 * j + 1 : j + 4];
                            const float c = kind < 2 ? cs[i][j] : 1.f, s = kind < 2 ? sn[i][j] : 0.f;
                            ec[i][j] = we * c;
                            es[i][j] = we * s;
                            oc[i][j] = wo * c;
                            os[i][j] = wo * s;
                        }
                    }
                }
                const float r = normed ? rsqrtf(ss * (1.f / D) + a.eps) : 1.f;
                uint16_t *to;
                if (kind == 0)
                    to = a.q_out + (long long)m * a.ldqo + h * D;
                else if (PAGED)
                    to = (kind == 1 ? a.k_pages : a.v_pages) + at + (size_t)(h - a.Hq - (kind == 1 ? 0 : a.Hkv)) * a.head_stride;
                else
                    to = a.k_out + (long long)m * a.ldko + (h - a.Hq) * D;
                if (kind > 0 && PAGED && !keep)
                    continue;
                const bool turned = kind < 2;
#pragma unroll
                for (int i = 0; i < CPL; ++i) {
                    if (!has[i])
                        continue;
                    float n[8];
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const int je = PAIRS ? 2 * j : j, jo = PAIRS ? 2 * j + 1 : j + 4;
                        const float e = x[u][i][je] * r, o = x[u][i][jo] * r;
                        // What is not turned does not meet its neighbour (0 * infinity).
                        n[je] = turned && rot[i] ? fmaf(e, ec[i][j], -(o * os[i][j])) : e * ec[i][j];
                        n[jo] = turned && rot[i] ? fmaf(e, es[i][j], o * oc[i][j]) : o * oc[i][j];
                    }
                    store4(to + o0[i], *reinterpret_cast<float (*)[4]>(&n[0]));
                    store4(to + o1[i], *reinterpret_cast<float (*)[4]>(&n[4]));
                }
            }
        };
        for (int hb = 0; hb < hp; hb += 2 * NH) {
            load(xb, h0 + hb + NH);
            process(xa, h0 + hb);
            if (hb + NH >= hp)
                break;
            load(xa, h0 + hb + 2 * NH);
            process(xb, h0 + hb + NH);
        }
    }
}

template <int D>
cudaError_t launch(const NormRopeArgs &a, int num_sms, cudaStream_t s)
{
    const bool paged = a.k_pages != nullptr;
    const int H = a.Hq + (paged ? 2 : 1) * a.Hkv;
    // Heads of a token are shared by more groups until there are two blocks per SM.
    constexpr int per = kThreads / RopeShape<D>::LPH;
    int hp = H;
    auto blocks = [&] { return ((long long)a.M * ((H + hp - 1) / hp) + per - 1) / per; };
    while (hp > 1 && blocks() < 2ll * num_sms)
        hp = (hp + 1) / 2;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(blocks() < 2ll * num_sms ? blocks() : 2ll * num_sms));
    cfg.blockDim = dim3(kThreads);
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const int split = (H + hp - 1) / hp;
    auto go = [&](auto kern) { return cudaLaunchKernelEx(&cfg, kern, a, hp, split); };
    auto pick = [&](auto f32, auto pages) {
        return a.pairs ? go(qk_norm_rope_kernel<D, f32.value, pages.value, true>)
                       : go(qk_norm_rope_kernel<D, f32.value, pages.value, false>);
    };
    using Yes = std::true_type;
    using No = std::false_type;
    if (a.f32)
        return paged ? pick(Yes{}, Yes{}) : pick(Yes{}, No{});
    return paged ? pick(No{}, Yes{}) : pick(No{}, No{});
}

} // namespace

cudaError_t run_qk_norm_rope(const NormRopeArgs &a, int num_sms, cudaStream_t s)
{
    switch (a.D) {
    case 64: return launch<64>(a, num_sms, s);
    case 128: return launch<128>(a, num_sms, s);
    case 256: return launch<256>(a, num_sms, s);
    case 384: return launch<384>(a, num_sms, s);
    case 512: return launch<512>(a, num_sms, s);
    default: return cudaErrorNotSupported;
    }
}

} // namespace w4
