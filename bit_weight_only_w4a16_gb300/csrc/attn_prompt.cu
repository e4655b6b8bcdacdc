// Prompt attention: causal attention of whole prompts, or chunks of them, packed
// one after another; the kernel is in attn_tiles.cuh.
//
// Source: "Gemma 4 E2B on a 4 GB GPU with pure PyTorch" - the prompt-read
// paragraph (a prompt is read in chunks, every chunk attends to the cache and
// itself) and the cache paragraph (full layers of head width 512, sliding layers
// of width 256 with a window, one key/value head under eight query heads).
#include "attn_launch.cuh"

namespace w4 {

cudaError_t run_attn_prompt(const AttnPromptArgs &p, float *ws, int *err, int num_sms, cudaStream_t s)
{
    attn::Args a = {};
    a.out = p.out;
    a.ldo = p.ldo;
    a.cu_q = p.cu_q;
    a.cu_k = p.cu_k;
    a.v = p.v;
    a.ldv = p.ldv;
    a.err = err;
    a.B = p.B;
    a.total_q = p.total_q;
    a.total_k = p.total_k;
    a.Hq = p.Hq;
    a.Hkv = p.Hkv;
    a.G = p.Hq / p.Hkv;
    a.D = p.D;
    a.tpt = attn::kRowsQ / a.G;
    a.window = p.window;
    a.c = p.scale * 1.4426950408889634f;
    const attn::Rows q = {p.q, p.total_q, p.ldq}, k = {p.k, p.total_k, p.ldk}, v = {p.v, p.total_k, p.ldv};
    auto run = [&](auto shape) {
        using S = decltype(shape);
        const long long tt = (long long)a.tpt * S::TQ;
        const long long tiles = (p.total_q / tt + p.B) * p.Hkv * S::NV;
        const bool may_cut = p.total_k > attn::kKeys;
        return attn::launch<S, attn::kPrompt>(a, q, k, v, k, v, tiles, may_cut, ws, num_sms, s);
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
