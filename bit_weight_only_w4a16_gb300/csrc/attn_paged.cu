// Attention of new tokens (one of each sequence, or chunks of prompts packed one after
// another) over a paged cache; the kernel is in attn_tiles.cuh.
//
// Source: "Gemma 4 E2B on a 4 GB GPU with pure PyTorch" - the prompt-read, decode-
// attention and cache paragraphs, for several requests whose caches share one pool of
// pages.
#include "attn_launch.cuh"

namespace w4 {

cudaError_t run_attn_paged(const AttnPagedArgs &p, float *ws, int *err, int num_sms, cudaStream_t s)
{
    // One token of each sequence whose heads fit a warp's products (attn_step.cu).
    if (!p.cu_q && step_serves(p.Hq / p.Hkv, p.D))
        return run_attn_step(p, ws, num_sms, s);
    attn::Args a = attn::paged_args(p);
    a.err = err;
    const attn::Rows q = {p.q, p.total_q, p.ldq}, k = {p.k_pages, 0, 0}, v = {p.v_pages, 0, 0};
    auto run = [&](auto shape) {
        using S = decltype(shape);
        const long long tt = (long long)a.tpt * S::TQ;
        const long long tiles = (p.total_q / tt + p.B) * p.Hkv * S::NV;
        // Units of a row tile at most: its window and tokens, which may begin and end within a key tile.
        const long long keys = a.window > 0 && a.window + tt < a.most_k ? a.window + tt : a.most_k;
        const bool may_cut = (keys + attn::kKeys - 1) / attn::kKeys + 1 > attn::whole_units(p.D);
        return attn::launch<S, attn::kPaged>(a, q, k, v, k, v, tiles, may_cut, ws, num_sms, s);
    };
    switch (p.D) {
    case 64: return run(attn::Shape<64>{});
    case 128:
        // Two row tiles share the keys where products are the bound; of chunks of up to four tiles on average
        // most row tiles have no second one to share with, and one has twice the softmax threads (12 chunks, 24
        // tokens on up to 18269: 67 and 79 us; 12 of 1411 tokens on up to 929: 34 and 39; 7 of 4000 on up to
        // 9000: 301 and 250).
        return p.total_q <= 4ll * p.B * a.tpt && (long long)p.B * p.Hkv < 1ll << 26 ? run(attn::Shape<128, 1>{})
                                                                                     : run(attn::Shape<128>{});
    case 256: return run(attn::Shape<256>{});
    case 384: return run(attn::Shape<384>{});
    case 512: return run(attn::Shape<512>{});
    default: return cudaErrorNotSupported;
    }
}

} // namespace w4
