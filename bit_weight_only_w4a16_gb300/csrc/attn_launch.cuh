// Host side of the tiled attention: tensor maps, the launch and the merge.
#pragma once

#include "attn_tiles.cuh"

#include <atomic>

namespace w4 {
namespace attn {

// Merges the partial sums of the row tiles that were cut (see attn_merge.cu).
struct MergeArgs {
    uint16_t *out;
    long long ldo;
    const float *ws_o, *ws_ml;
    const int32_t *rec, *where;
    int ctas; // CTAs of the attention kernel
    int rows_per_tile, D, DV, G, tpt;
    int rb; // rows per block
};
cudaError_t run_merge(const MergeArgs &m, int tiles, cudaStream_t s);

// bf16 rows [rows][heads][D], `ld` elements between rows, as boxes of 64 dims x
// `bh` heads x `br` rows in the 128-byte-swizzle layout.
inline bool encode_rows(CUtensorMap *map, const void *p, long long rows, int heads, int D, long long ld, int bh, int br)
{
    auto enc = tmap_encoder();
    if (!enc)
        return false;
    cuuint64_t dims[3] = {(cuuint64_t)D, (cuuint64_t)heads, (cuuint64_t)rows};
    cuuint64_t strides[2] = {(cuuint64_t)D * 2, (cuuint64_t)ld * 2};
    cuuint32_t box[3] = {64, (cuuint32_t)bh, (cuuint32_t)br};
    cuuint32_t es[3] = {1, 1, 1};
    return enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(p), dims, strides, box, es,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

struct Rows {
    const uint16_t *p;
    long long rows, ld;
};

// q, k, v (and for a tree the nodes' own kt, vt); a.* but the scratch is set.
// tiles: row tiles of the call at most, over all heads and value slices.
template <int D, bool TREE>
cudaError_t launch(Args a, const Rows &q, const Rows &k, const Rows &v, const Rows &kt, const Rows &vt,
                   long long tiles, bool may_cut, float *ws, int num_sms, cudaStream_t s)
{
    using S = Shape<D>;
    static_assert(S::TQ == (D <= 128 ? 2 : 1) && S::NV == (D > 256 ? 2 : 1), "as in attn_tile_tokens, attn_slices");
    Maps m;
    if (!encode_rows(&m.q, q.p, q.rows, a.Hq, D, q.ld, a.G, a.tpt) ||
        !encode_rows(&m.k, k.p, k.rows, a.Hkv, D, k.ld, 1, kKeys) ||
        !encode_rows(&m.v, v.p, v.rows, a.Hkv, D, v.ld, 1, S::VKEYS) ||
        (TREE && (!encode_rows(&m.kt, kt.p, kt.rows, a.Hkv, D, kt.ld, 1, kKeys) ||
                  !encode_rows(&m.vt, vt.p, vt.rows, a.Hkv, D, vt.ld, 1, S::VKEYS))))
        return cudaErrorInvalidValue;
    a.ws_o = ws;
    a.ws_ml = ws + (size_t)2 * num_sms * kSlotFloats;
    a.rec = reinterpret_cast<int32_t *>(a.ws_ml + (size_t)2 * num_sms * 256 * 2);
    a.where = a.rec + 2 * num_sms;

    auto kern = attn_kernel<D, TREE>;
    // Once per device: the attribute belongs to the kernel there.
    static std::atomic<unsigned long long> set{0};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess)
        return e;
    if (dev >= 64 || !((set.load(std::memory_order_relaxed) >> dev) & 1)) {
        e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)S::SMEM);
        if (e != cudaSuccess)
            return e;
        if (dev < 64)
            set.fetch_or(1ull << dev, std::memory_order_relaxed);
    }
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(num_sms);
    cfg.blockDim = dim3(S::THREADS);
    cfg.dynamicSmemBytes = S::SMEM;
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    e = cudaLaunchKernelEx(&cfg, kern, a, m);
    if (e != cudaSuccess || !may_cut)
        return e;
    MergeArgs g;
    g.out = a.out;
    g.ldo = a.ldo;
    g.ws_o = a.ws_o;
    g.ws_ml = a.ws_ml;
    g.rec = a.rec;
    g.where = a.where;
    g.ctas = num_sms;
    g.rows_per_tile = S::ROWS;
    g.D = D;
    g.DV = S::DV;
    g.G = a.G;
    g.tpt = a.tpt;
    return run_merge(g, (int)(tiles < num_sms ? tiles : num_sms), s);
}

} // namespace attn
} // namespace w4
