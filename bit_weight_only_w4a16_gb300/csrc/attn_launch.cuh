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

// Keys or values in pages: rows of a page, pages and heads lie at the call's strides.
// A box is `br` rows of a page (a multiple of 8) and `blocks` blocks of 64 dims; heads are
// so many blocks apart, which leaves the other dimensions to rows (in eights) and pages.
inline bool encode_pages(CUtensorMap *map, const void *p, const Args &a, int D, int br, int blocks)
{
    auto enc = tmap_encoder();
    if (!enc)
        return false;
    cuuint64_t dims[5] = {64, 8, (cuuint64_t)(a.Hkv - 1) * a.head_blocks + D / 64, (cuuint64_t)1 << (a.page_log2 - 3),
                          (cuuint64_t)a.pages};
    cuuint64_t strides[4] = {(cuuint64_t)a.row_stride * 2, 128, (cuuint64_t)a.row_stride * 16,
                             (cuuint64_t)a.page_stride * 2};
    cuuint32_t box[5] = {64, 8, (cuuint32_t)blocks, (cuuint32_t)br / 8, 1};
    cuuint32_t es[5] = {1, 1, 1, 1, 1};
    return enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 5, const_cast<void *>(p), dims, strides, box, es,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Partial sums' places in the scratch.
inline void set_scratch(Args &a, float *ws, int num_sms)
{
    a.ws_o = ws;
    a.ws_ml = ws + (size_t)2 * num_sms * kSlotFloats;
    a.rec = reinterpret_cast<int32_t *>(a.ws_ml + (size_t)2 * num_sms * 256 * 2);
    a.where = a.rec + 2 * num_sms;
}

// A kernel's dynamic shared memory, once per device: the attribute belongs to the kernel there.
template <typename K>
cudaError_t allow_smem(K kern, size_t bytes, std::atomic<unsigned long long> &set)
{
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess)
        return e;
    if (dev >= 64 || !((set.load(std::memory_order_relaxed) >> dev) & 1)) {
        e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
        if (e != cudaSuccess)
            return e;
        if (dev < 64)
            set.fetch_or(1ull << dev, std::memory_order_relaxed);
    }
    return cudaSuccess;
}

// What the merge takes from a call's arguments (rows_per_tile and DV are the kernel's).
inline MergeArgs merge_args(const Args &a, int num_sms)
{
    MergeArgs g = {};
    g.out = a.out;
    g.ldo = a.ldo;
    g.ws_o = a.ws_o;
    g.ws_ml = a.ws_ml;
    g.rec = a.rec;
    g.where = a.where;
    g.ctas = num_sms;
    g.D = a.D;
    g.G = a.G;
    g.tpt = a.tpt;
    return g;
}

// A paged call's arguments but its queries and the scratch.
inline Args paged_args(const AttnPagedArgs &p)
{
    Args a = {};
    a.out = p.out;
    a.ldo = p.ldo;
    a.cu_q = p.cu_q;
    a.v = p.v_pages;
    a.B = p.B;
    a.total_q = p.total_q;
    a.Hq = p.Hq;
    a.Hkv = p.Hkv;
    a.G = p.Hq / p.Hkv;
    a.D = p.D;
    a.tpt = kRowsQ / a.G;
    a.window = p.window;
    a.c = p.scale * 1.4426950408889634f;
    a.table = p.table;
    a.lens = p.lens;
    a.table_pages = p.table_pages;
    a.pages = p.pages;
    a.page_log2 = p.page_log2;
    a.most_k = p.table_pages << p.page_log2;
    a.page_stride = p.page_stride;
    a.row_stride = p.row_stride;
    a.head_stride = p.head_stride;
    a.head_blocks = (int)(p.head_stride / 64);
    return a;
}

struct Rows {
    const uint16_t *p;
    long long rows, ld;
};

// q, k, v (and for a tree the nodes' own kt, vt); a.* but the scratch is set.
// tiles: row tiles of the call at most, over all heads and value slices.
template <typename S, Kind KIND>
cudaError_t launch(Args a, const Rows &q, const Rows &k, const Rows &v, const Rows &kt, const Rows &vt,
                   long long tiles, bool may_cut, float *ws, int num_sms, cudaStream_t s)
{
    constexpr int D = S::DIM;
    static_assert(S::TQ <= (D <= 128 ? 2 : 1) && S::NV == (D > 256 ? 2 : 1), "as in attn_tile_tokens, attn_slices");
    Maps m;
    if (!encode_rows(&m.q, q.p, q.rows, a.Hq, D, q.ld, a.G, a.tpt) ||
        (KIND == kPaged
             ? !encode_pages(&m.k, k.p, a, D, min(1 << a.page_log2, kKeys), S::KB) ||
                   !encode_pages(&m.v, v.p, a, D, min(1 << a.page_log2, S::VKEYS), S::DV / 64)
             : !encode_rows(&m.k, k.p, k.rows, a.Hkv, D, k.ld, 1, kKeys) ||
                   !encode_rows(&m.v, v.p, v.rows, a.Hkv, D, v.ld, 1, S::VKEYS)) ||
        (KIND == kTree && (!encode_rows(&m.kt, kt.p, kt.rows, a.Hkv, D, kt.ld, 1, kKeys) ||
                  !encode_rows(&m.vt, vt.p, vt.rows, a.Hkv, D, vt.ld, 1, S::VKEYS))))
        return cudaErrorInvalidValue;
    set_scratch(a, ws, num_sms);

    auto kern = attn_kernel<D, KIND, S::TQ>;
    static std::atomic<unsigned long long> set{0};
    cudaError_t e = allow_smem(kern, S::SMEM, set);
    if (e != cudaSuccess)
        return e;
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
    MergeArgs g = merge_args(a, num_sms);
    g.rows_per_tile = S::ROWS;
    g.DV = S::DV;
    return run_merge(g, (int)(tiles < num_sms ? tiles : num_sms), s);
}

} // namespace attn
} // namespace w4
