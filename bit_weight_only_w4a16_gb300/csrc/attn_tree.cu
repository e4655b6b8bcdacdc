// Attention of a tree of drafted tokens over a cache and the tree itself; the
// kernel is in attn_tiles.cuh.
//
// Source: "Gemma 4 E2B on a 4 GB GPU with pure PyTorch" - the decode-attention
// and cache paragraphs (one key/value head under eight query heads, the cache
// split over the GPU and joined by an online softmax; a ring of slots that
// records each slot's position); the drafted tokens' keys and values stay beside
// the cache until some are accepted, because a ring as long as its window has no
// slot to spare for them.
#include "attn_launch.cuh"

namespace w4 {

cudaError_t run_attn_tree(const AttnTreeArgs &p, float *ws, int *err, int num_sms, cudaStream_t s)
{
    attn::Args a = {};
    a.out = p.out;
    a.ldo = (long long)p.Hq * p.D;
    a.parents = p.parents;
    a.pos = p.pos;
    a.kpos = p.kpos;
    a.v = p.v;
    a.vt = p.v_tree;
    a.ldv = (long long)p.Hkv * p.D;
    a.err = err;
    a.B = p.B;
    a.N = p.N;
    a.T = p.T;
    a.Hq = p.Hq;
    a.Hkv = p.Hkv;
    a.G = p.Hq / p.Hkv;
    a.D = p.D;
    a.tpt = attn::kRowsQ / a.G;
    a.window = p.window;
    a.c = p.scale * 1.4426950408889634f;
    const long long rows = (long long)p.B * p.N, slots = (long long)p.B * p.T;
    const attn::Rows q = {p.q, rows, a.ldo}, k = {p.k, slots, a.ldv}, v = {p.v, slots, a.ldv};
    const attn::Rows kt = {p.k_tree, rows, a.ldv}, vt = {p.v_tree, rows, a.ldv};
    auto run = [&](auto shape) {
        using S = decltype(shape);
        const int tt = a.tpt * S::TQ;
        const long long tiles = (long long)p.B * ((p.N + tt - 1) / tt) * p.Hkv * S::NV;
        return attn::launch<S, attn::kTree>(a, q, k, v, kt, vt, tiles, true, ws, num_sms, s);
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
