// Accepted tokens' key and value rows into the caches of all layers.
//
// Source: "Gemma 4 E2B on a 4 GB GPU with pure PyTorch" - the cache paragraph
// (full layers: one slot per position; sliding layers: a ring of slots that
// records each slot's position), for the several tokens that a drafted step
// accepts at once.
//
// Row path[j] of a sequence's tree goes to position pos + j: 4 W bytes read and
// 4 W written per token and layer, a few hundred kilobytes over all layers, so the
// call is bound by its launch and two dependent reads (count, path). One block
// per layer, sequence and cache (keys, values); thread = 16 bytes, four in flight.
// 28 layers, 4 tokens of 512 bytes: 4 us on the GPU with cold caches, a call 8 us
// (host time).
#include "common.cuh"
#include "internal.h"

namespace w4 {

namespace {

constexpr int kThreads = 256;
constexpr int kInFlight = 4;

__global__ void __launch_bounds__(kThreads)
kv_commit_kernel(const KvCommitArgs a)
{
    __shared__ int s_node[64], s_slot[64];
    pdl_launch_dependents();
    pdl_wait();
    const int b = blockIdx.x % a.B, l = blockIdx.x / a.B;
    const bool first = l == 0 && blockIdx.y == 0;
    const int n = min(max(__ldg(a.count + b), 0), a.N);
    // Thread j: token j of the path; -1 = nothing to write.
    const int j = threadIdx.x;
    const long long p = j < n ? (long long)__ldg(a.pos + b) + j : 0;
    if (j < 64) {
        int node = -1, slot = -1;
        if (j < n) {
            node = __ldg(a.path + (size_t)b * a.N + j);
            const bool ok = node >= 0 && node < a.N && p >= 0 && p <= 0x7FFFFFFFll && (a.kpos || p < a.T);
            if (!ok) {
                node = -1;
                if (first && a.status)
                    *a.status = 1;
            } else {
                slot = (int)(a.kpos ? p % a.T : p);
            }
        }
        s_node[j] = node;
        s_slot[j] = slot;
    }
    __syncthreads();
    if (a.kpos && n > a.T) {
        // A short ring: the last token that is stored to a slot stays in it.
        bool later = false;
        for (int i = j + a.T; i < n; i += a.T)
            later = later || s_node[i] >= 0;
        __syncthreads();
        if (later)
            s_node[j] = -1;
        __syncthreads();
    }
    if (first && a.kpos && j < n && s_node[j] >= 0)
        a.kpos[(size_t)b * a.T + s_slot[j]] = (int32_t)p;
    const size_t lb = (size_t)l * a.B + b;
    const int w8 = a.W >> 3; // 16-byte pieces of a row
    const uint4 *src = reinterpret_cast<const uint4 *>(blockIdx.y ? a.v_tree : a.k_tree) + lb * a.N * w8;
    uint4 *dst = reinterpret_cast<uint4 *>(blockIdx.y ? a.v_cache : a.k_cache) + lb * a.T * w8;
    const long long items = (long long)n * w8;
    for (long long i0 = threadIdx.x; i0 < items; i0 += kThreads * kInFlight) {
        uint4 v[kInFlight];
        long long to[kInFlight];
#pragma unroll
        for (int q = 0; q < kInFlight; ++q) {
            const long long i = i0 + (long long)q * kThreads;
            to[q] = -1;
            if (i < items) {
                const int t = (int)(i / w8), c = (int)(i - (long long)t * w8);
                if (s_node[t] >= 0) {
                    v[q] = __ldg(src + (size_t)s_node[t] * w8 + c);
                    to[q] = (long long)s_slot[t] * w8 + c;
                }
            }
        }
#pragma unroll
        for (int q = 0; q < kInFlight; ++q)
            if (to[q] >= 0)
                dst[to[q]] = v[q];
    }
}

} // namespace

cudaError_t run_kv_commit(const KvCommitArgs &a, cudaStream_t s)
{
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(a.L * a.B), 2);
    cfg.blockDim = dim3(kThreads);
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kv_commit_kernel, a);
}

} // namespace w4
