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
        const bool may_cut = a.most_k > attn::kKeys;
        return attn::launch<S::DIM, attn::kPaged>(a, q, k, v, k, v, tiles, may_cut, ws, num_sms, s);
    };
    switch (p.D) {
    case 64: return run(attn::Shape<64>{});
    case 128: return run(attn::Shape<128>{});
    case 256: return run(attn::Shape<256>{});
    case 384: return run(attn::Shape<384>{});
    case 512: return run(attn::Shape<512>{});
    default: return cudaErrorNotSupported;
    }
}

} // namespace w4
