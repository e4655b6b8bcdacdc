// Log probabilities of given tokens, entropy and the most likely alternatives
// from rows of fp32 logits (the vocabulary projection's output).
//
// Source: "Gemma 4 E2B on a 4 GB GPU with pure PyTorch" - Step 2 (the logits of
// 262144 tokens come from the 4-bit embedding). The pages pick greedily; judging
// drafted tokens needs the probabilities themselves.
//
// Mathematics, one pass: with m the running maximum of a warp,
//   s = sum e^(x - m),  u = sum e^(x - m) (x - m)
// and when m grows to m': s' = f s, u' = f (u + (m - m') s), f = e^(m - m').
//   log p(t) = (x_t - m) - log s,   entropy = log s - u / s
// (u in terms of x - m keeps the entropy's two parts small). All of it is fp32; e^y is the
// hardware's ex2 of y log2 e, whose error (2^-22 and the rounding of y log2 e) stays below
// that of the sums: log probabilities come within about 1e-7 (relative) of 64 bits.
//
// The k largest logits need no second pass over the row: the streaming blocks keep
// the maximum of every 256 logits (a chunk). The block that finishes a row last gives
// each of its threads a share of the chunks; in the order (value descending, index
// ascending) the k-th of the threads' first maxima has k - 1 logits of other chunks
// before it, so nothing behind it is among the k largest. The few chunks not behind
// it are looked at alone, while other rows' blocks still stream, and what reaches the
// bound is ranked by counting.
//
// Bound by the read of the logits: 4 V bytes a row. 256 rows of 256003 logits (262 MB)
// take 49 us with 5 alternatives, 45 us (5.8 TB/s) without: the picks of the rows that
// finish last are not hidden. One row of 262144: 9.5 us on the GPU, a chain of short
// steps (read 1.3 us, count of finished blocks 1.3, sums 0.7, bound 2, picks 3).
#include "common.cuh"
#include "internal.h"

#include <atomic>

namespace w4 {

namespace {

constexpr int kChunk = 256; // logits per chunk: two float4 per lane
constexpr int kWarps = 8;
constexpr int kBatch = 4; // chunks in flight per warp
constexpr float kLog2e = 1.4426950408889634f;
// Differences from the maximum are cut here where they are factors: 0 * -inf (a
// masked logit, or finite logits further apart than fp32 reaches) is not 0.
constexpr float kLeast = -1e30f;

// A row's counter is 0 before and after a call. A count that calls which overlapped (in
// spite of the rule) have left behind does not stay: every block first raises the counter
// to its launch's number and a count of 0, which changes nothing once one block has done
// it. A captured launch keeps the number of its capture: after a newer launch's remainder
// it is right again once a launch with a newer number has been over its rows.
constexpr int kTagShift = 16; // at most 256 blocks count

struct LogprobArgs {
    const float *x;
    long long ld;
    int V, nc, S; // logits per row, chunks per row, blocks per row
    float *cmax;  // [rows][nc]
    float *part;  // [rows][S][4]: m, s, u
    unsigned long long *left; // [rows] blocks that have finished, above kTagShift bits the call
    unsigned long long tag;   // this launch's number, larger than earlier ones'
    const int32_t *targets;
    float *logprob, *entropy, *top_logprob;
    int32_t *top_id;
    int k;
    int32_t *status;
};

// Chunk c of a row covers logits [256 c - mis, 256 c - mis + 256), where mis is
// the row's distance (in floats) from a 16-byte boundary: every interior float4
// is aligned whatever the row stride.
__device__ __forceinline__ int row_mis(const float *row)
{
    return (int)((reinterpret_cast<uintptr_t>(row) >> 2) & 3);
}

// This lane's eight logits of chunk c: elements e0 .. e0 + 3 and e0 + 128 .. e0 + 131.
__device__ __forceinline__ void load_chunk(const float *row, int mis, int V, int c, int lane, float v[8])
{
    const long long e0 = (long long)c * kChunk - mis + 4 * lane;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const long long e = e0 + 128 * h;
        if (e >= 0 && e + 4 <= V) {
            const float4 f = __ldcs(reinterpret_cast<const float4 *>(row + e));
            v[4 * h] = f.x;
            v[4 * h + 1] = f.y;
            v[4 * h + 2] = f.z;
            v[4 * h + 3] = f.w;
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                v[4 * h + i] = e + i >= 0 && e + i < V ? __ldcs(row + e + i) : -INFINITY;
        }
    }
}

__device__ __forceinline__ float ex2f(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// The block's (m, s, u) from its threads', in every thread, in a fixed order: the
// maximum first, then each thread's sums scaled once. (Merging triples pair by pair
// takes an exponential in each of the steps: 1.9 us against 1.2 for one row.)
__device__ __forceinline__ float3 block_stats(float m, float s, float u)
{
    __shared__ float sm[kWarps], ss[kWarps], su[kWarps];
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    float M = m;
#pragma unroll
    for (int d = 16; d; d >>= 1)
        M = fmaxf(M, __shfl_xor_sync(0xFFFFFFFFu, M, d));
    if (lane == 0)
        sm[w] = M;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kWarps; ++i)
        M = fmaxf(M, sm[i]);
    // A thread without finite logits has s = u = 0, or NaN.
    const float d = fmaxf(m - (M == -INFINITY ? 0.f : M), kLeast), f = ex2f(d * kLog2e);
    u = f * fmaf(d, s, u);
    s *= f;
#pragma unroll
    for (int e = 16; e; e >>= 1) {
        s += __shfl_xor_sync(0xFFFFFFFFu, s, e);
        u += __shfl_xor_sync(0xFFFFFFFFu, u, e);
    }
    if (lane == 0) {
        ss[w] = s;
        su[w] = u;
    }
    __syncthreads();
    s = ss[0];
    u = su[0];
#pragma unroll
    for (int i = 1; i < kWarps; ++i) {
        s += ss[i];
        u += su[i];
    }
    return make_float3(M, s, u);
}

// --------------------------------------------------- lists of the largest ----

// A key orders (value descending, index ascending): larger keys come first.
// Zeros of either sign are equal. 0 is below every key.
__device__ __forceinline__ unsigned long long make_key(float x, uint32_t index)
{
    const uint32_t b = __float_as_uint(x + 0.f);
    const uint32_t o = (b & 0x80000000u) ? ~b : b | 0x80000000u;
    return ((unsigned long long)o << 32) | (uint32_t)~index;
}
__device__ __forceinline__ float key_value(unsigned long long k)
{
    const uint32_t o = (uint32_t)(k >> 32);
    return __uint_as_float((o & 0x80000000u) ? o & 0x7FFFFFFFu : ~o);
}
__device__ __forceinline__ uint32_t key_index(unsigned long long k) { return ~(uint32_t)k; }

__device__ __forceinline__ unsigned long long cmp_xchg(unsigned long long k, int d, bool keep_max)
{
    const unsigned long long o = __shfl_xor_sync(0xFFFFFFFFu, k, d);
    return keep_max == (k > o) ? k : o;
}

// 32 keys, one per lane, into descending order by lane.
__device__ __forceinline__ unsigned long long sort32(unsigned long long k, int lane)
{
#pragma unroll 1
    for (int n = 2; n <= 32; n <<= 1)
#pragma unroll 1
        for (int d = n >> 1; d; d >>= 1)
            k = cmp_xchg(k, d, ((lane & d) == 0) == ((lane & n) == 0)); // n = 32: all lanes
    return k;
}

// The 32 largest of two descending lists, in descending order.
__device__ __forceinline__ unsigned long long merge32(unsigned long long list, unsigned long long other, int lane)
{
    const unsigned long long r = __shfl_sync(0xFFFFFFFFu, other, 31 - lane);
    unsigned long long k = list > r ? list : r;
#pragma unroll 1
    for (int d = 16; d; d >>= 1)
        k = cmp_xchg(k, d, (lane & d) == 0);
    return k;
}

// The block's lists into one, held by every warp: a tree of merges.
__device__ __forceinline__ unsigned long long merge_block(unsigned long long list, unsigned long long (*sl)[32],
                                                          int lane, int w)
{
#pragma unroll 1
    for (int d = kWarps / 2; d; d >>= 1) {
        __syncthreads(); // the lists of the round before have been read
        if (w >= d && w < 2 * d)
            sl[w][lane] = list;
        __syncthreads();
        if (w < d)
            list = merge32(list, sl[w + d][lane], lane);
    }
    if (w == 0)
        sl[0][lane] = list;
    __syncthreads();
    return sl[0][lane];
}

// A row's outputs from its blocks' parts and its chunk maxima; they come from other
// SMs, so they are read from L2. This code runs once a row, so what it costs a short
// call is its length: its loops stay loops.
__device__ __forceinline__ void finish_row(const LogprobArgs &a, size_t r)
{
    constexpr int kThreads = kWarps * 32, kScan = 4; // chunk maxima of a thread at a time
    __shared__ unsigned long long sl[kWarps][32], pend[kWarps][kChunk + 32];
    __shared__ unsigned long long pool[kWarps * 64];
    __shared__ int cand[32 * kScan], ncand, npool;
    const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5;
    const float *row = a.x + r * a.ld;
    const int mis = row_mis(row);

    // What the picks need first is asked for before the sums.
    const float *cmax = a.cmax + r * a.nc;
    float cm[kScan];
    auto scan = [&](int c0) {
#pragma unroll
        for (int j = 0; j < kScan; ++j) {
            const int c = c0 + j * kThreads + tid;
            cm[j] = a.k > 0 && c < a.nc ? __ldcg(cmax + c) : 0.f;
        }
    };
    scan(0);
    const int t = tid == 0 && a.logprob ? a.targets[r] : -1;
    const float xt = t >= 0 && t < a.V ? row[t] : 0.f;

    float m = -INFINITY, s = 0.f, u = 0.f;
    if (tid < a.S) { // S <= kThreads
        const float4 p = __ldcg(reinterpret_cast<const float4 *>(a.part + (r * a.S + tid) * 4));
        m = p.x;
        s = p.y;
        u = p.z;
    }
    const float3 st = block_stats(m, s, u);
    m = st.x;
    s = st.y;
    u = st.z;
    const float nan = __uint_as_float(0x7FFFFFFFu);
    const bool bad = s != s;            // a NaN or +inf among the logits
    const bool none = m == -INFINITY;   // every logit is -inf
    const float logs = bad ? nan : logf(s);
    if (tid == 0) {
        if (a.entropy)
            a.entropy[r] = bad ? nan : (none ? 0.f : logs - u / s);
        if (a.logprob) {
            float y = 0.f;
            if (t < 0 || t >= a.V) {
                if (a.status)
                    *a.status = 1;
            } else {
                y = bad ? nan : (xt == -INFINITY ? -INFINITY : (xt - m) - logs);
            }
            a.logprob[r] = y;
        }
    }
    if (a.k == 0)
        return;

    // Each thread's first chunk in the order; the k-th of those bounds the k-th logit
    // from below (k chunks have an element before it). At most k threads hold chunks
    // that are not behind the bound.
    unsigned long long first = 0;
#pragma unroll 1
    for (int c0 = 0; c0 < a.nc; c0 += kScan * kThreads) {
        if (c0)
            scan(c0);
#pragma unroll
        for (int j = 0; j < kScan; ++j) {
            const int c = c0 + j * kThreads + tid;
            const unsigned long long k = c < a.nc ? make_key(cm[j], c) : 0ull;
            first = k > first ? k : first;
        }
    }
    const unsigned long long firsts = merge_block(sort32(first, lane), sl, lane, w);
    const unsigned long long bound = __shfl_sync(0xFFFFFFFFu, firsts, a.k - 1); // 0: fewer chunks than k
    const float least = bound ? key_value(bound) : -INFINITY;

    // Those chunks' logits that reach the bound are collected, a chunk per warp at a
    // time; 32 of a warp's are merged into its list (many equal logits, else rare).
    unsigned long long list = 0;
    unsigned long long reached = 0; // its k-th: equal logits of later chunks stay out
    int n = 0; // logits collected in pend[w]
    if (tid == 0)
        npool = 0;
#pragma unroll 1
    for (int c0 = 0; c0 < a.nc; c0 += kScan * kThreads) {
        if (a.nc > kScan * kThreads)
            scan(c0);
        if (tid == 0)
            ncand = 0;
        __syncthreads();
#pragma unroll
        for (int j = 0; j < kScan; ++j) {
            const int c = c0 + j * kThreads + tid;
            if (c < a.nc && make_key(cm[j], c) >= bound) {
                const int at = atomicAdd(&ncand, 1); // in any order: the logits are ranked
                if (at < 32 * kScan) // more only if another call overwrites the maxima meanwhile
                    cand[at] = c;
            }
        }
        __syncthreads();
        const int nk = min(ncand, 32 * kScan);
        float v[8]; // the next chunk's
        int e = 0;
        auto load = [&](int i) {
            e = i < nk ? cand[i] * kChunk - mis + lane : a.V;
#pragma unroll
            for (int j = 0; j < 8; ++j)
                v[j] = e + 32 * j >= 0 && e + 32 * j < a.V ? __ldcs(row + e + 32 * j) : 0.f;
        };
        load(w);
#pragma unroll 1
        for (int i = w; i < nk; i += kWarps) {
            float x[8];
            const int ex = e;
#pragma unroll
            for (int j = 0; j < 8; ++j)
                x[j] = v[j];
            load(i + kWarps);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const int at = ex + 32 * j;
                const unsigned long long key = make_key(x[j], (uint32_t)at);
                const bool in = x[j] >= least && key > reached && at >= 0 && at < a.V;
                const uint32_t who = __ballot_sync(0xFFFFFFFFu, in);
                if (in)
                    pend[w][n + __popc(who & ((1u << lane) - 1u))] = key;
                n += __popc(who);
                if (j != 0 && j != 7)
                    continue;
                // At most 31 stay for the next chunk. After the first 32 logits too: of
                // a chunk of equal logits the others then stay out (8 sorts a chunk
                // against 1: a row of 262144 that a mask leaves three tokens takes 17 us
                // against 11 with 5 alternatives, 48 against 16 with 32).
#pragma unroll 1
                while (n >= 32) {
                    __syncwarp();
                    list = merge32(list, sort32(pend[w][n - 32 + lane], lane), lane);
                    reached = __shfl_sync(0xFFFFFFFFu, list, a.k - 1);
                    n -= 32;
                    __syncwarp();
                }
            }
        }
        __syncthreads(); // cand has been read
    }
    // What the warps have left, at most 63 each: a key's place is the number before it.
    const uint32_t held = __ballot_sync(0xFFFFFFFFu, list != 0); // the first lanes
    const int nh = __popc(held);
    int base = 0;
    if (lane == 0 && n + nh > 0)
        base = atomicAdd(&npool, n + nh);
    base = __shfl_sync(0xFFFFFFFFu, base, 0);
    if (lane < n)
        pool[base + lane] = pend[w][lane];
    if (lane < nh)
        pool[base + n + lane] = list;
    __syncthreads();
    const int np = npool;
#pragma unroll 1
    for (int i = tid; i < np || i < a.k; i += kThreads) {
        const unsigned long long key = i < np ? pool[i] : 0ull; // 0: fewer logits than k
        int place = i < np ? 0 : i;
        if (i < np) {
#pragma unroll 4
            for (int j = 0; j < np; ++j)
                place += pool[j] > key;
        }
        if (place >= a.k)
            continue;
        const float x = key_value(key);
        const size_t o = r * a.k + place;
        if (a.top_id)
            a.top_id[o] = bad || key == 0 ? -1 : (int32_t)key_index(key);
        if (a.top_logprob)
            a.top_logprob[o] = bad ? nan : (key == 0 || x == -INFINITY ? -INFINITY : (x - m) - logs);
    }
}

__global__ void __launch_bounds__(kWarps * 32)
logprob_kernel(const LogprobArgs a)
{
    pdl_launch_dependents();
    pdl_wait();
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    const float *row = a.x + (size_t)blockIdx.y * a.ld;
    const int mis = row_mis(row);
    const int c0 = (int)((long long)blockIdx.x * a.nc / a.S), c1 = (int)((long long)(blockIdx.x + 1) * a.nc / a.S);
    float *cmax = a.cmax + (size_t)blockIdx.y * a.nc;
    if (threadIdx.x == 0) // before this thread's count: the same address, so in this order
        atomicMax(a.left + blockIdx.y, a.tag << kTagShift);

    float m = -INFINITY, s = 0.f, u = 0.f; // m is the same in all lanes
    for (int cb = c0 + w; cb < c1; cb += kBatch * kWarps) {
        float v[kBatch][8];
#pragma unroll
        for (int b = 0; b < kBatch; ++b) {
            const int c = cb + b * kWarps;
            if (c < c1) {
                load_chunk(row, mis, a.V, c, lane, v[b]);
            } else {
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    v[b][i] = -INFINITY;
            }
        }
        float bm = -INFINITY;
#pragma unroll
        for (int b = 0; b < kBatch; ++b) {
            float cm = v[b][0];
#pragma unroll
            for (int i = 1; i < 8; ++i)
                cm = fmaxf(cm, v[b][i]);
            if (cm != cm)
                cm = -INFINITY; // eight NaNs: the row's sums are NaN all the same
#pragma unroll
            for (int d = 16; d; d >>= 1)
                cm = fmaxf(cm, __shfl_xor_sync(0xFFFFFFFFu, cm, d));
            if (a.k > 0 && lane == 0 && cb + b * kWarps < c1)
                cmax[cb + b * kWarps] = cm;
            bm = fmaxf(bm, cm);
        }
        if (bm > m) {
            if (m != -INFINITY) {
                const float d = fmaxf(m - bm, kLeast), f = ex2f(d * kLog2e);
                u = f * fmaf(d, s, u);
                s *= f;
            }
            m = bm;
        }
        const float ref = m == -INFINITY ? 0.f : m;
#pragma unroll
        for (int b = 0; b < kBatch; ++b)
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float d = v[b][i] - ref;
                const float e = ex2f(d * kLog2e);
                s += e;
                u = fmaf(e, fmaxf(d, kLeast), u);
            }
    }
    const float3 st = block_stats(m, s, u);
    // The block that finishes last sees all parts and chunk maxima of the row: a block's
    // are written before its count (barrier, fence), and read after all counts.
    __shared__ int s_last;
    if (threadIdx.x == 0) {
        *reinterpret_cast<float4 *>(a.part + ((size_t)blockIdx.y * a.S + blockIdx.x) * 4) =
            make_float4(st.x, st.y, st.z, 0.f);
        __threadfence();
        const int n = (int)(atomicAdd(a.left + blockIdx.y, 1ull) & ((1ull << kTagShift) - 1));
        s_last = n == a.S - 1;
        if (s_last)
            a.left[blockIdx.y] = 0;
        __threadfence();
    }
    __syncthreads();
    if (s_last)
        finish_row(a, (size_t)blockIdx.y);
}

} // namespace

cudaError_t run_logprobs(const LogprobsArgs &p, float *ws, size_t ws_floats, unsigned long long *left, int num_sms,
                         cudaStream_t s)
{
    static std::atomic<unsigned long long> launches{0};
    LogprobArgs a = {};
    a.ld = p.ld;
    a.V = p.V;
    a.nc = (p.V + 3 + kChunk - 1) / kChunk; // a row may begin three floats past a boundary
    a.k = p.k;
    a.status = p.status;
    static std::atomic<int> known{0}; // blocks per SM, the same on every device served
    int occ = known.load(std::memory_order_relaxed);
    cudaError_t e = cudaSuccess;
    if (occ == 0) {
        e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&occ, logprob_kernel, kWarps * 32, 0);
        if (e != cudaSuccess)
            return e;
        occ = occ < 1 ? 1 : occ;
        known.store(occ, std::memory_order_relaxed);
    }
    // Blocks per row: as many as fit at once (`occ` per SM), so that all stream from
    // the start to the end; for more rows than that, several waves of blocks. Measured
    // for 256 rows of 256003 logits (no alternatives): 1 block a row 74.7 us, 2 45.1,
    // 4 46.5, 5 50.9, 7 47.8.
    const long long most = (a.nc + kWarps - 1) / kWarps; // a chunk per warp at least
    const long long fit = (long long)num_sms * occ;
    long long S = p.M <= fit ? fit / p.M : (4 * fit + p.M - 1) / p.M;
    S = S < most ? S : most;
    S = S < kWarps * 32 ? S : kWarps * 32; // the last block takes a part per thread
    S = S < 1 ? 1 : S;
    a.S = (int)S;
    const size_t per_row = (size_t)a.nc + (size_t)S * 4;
    long long rows = (long long)((ws_floats - 4) / per_row); // rows of one pass
    if (rows < 1)
        return cudaErrorNotSupported; // a row's chunk maxima do not fit the scratch
    rows = rows < kLogprobRows ? rows : kLogprobRows;
    a.left = left;

    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    for (long long r0 = 0; r0 < p.M; r0 += rows) {
        const int n = (int)(p.M - r0 < rows ? p.M - r0 : rows);
        a.tag = launches.fetch_add(1, std::memory_order_relaxed) + 1;
        a.x = p.logits + (size_t)r0 * p.ld;
        a.part = ws;
        a.cmax = ws + (size_t)n * S * 4;
        a.targets = p.targets ? p.targets + r0 : nullptr;
        a.logprob = p.logprob ? p.logprob + r0 : nullptr;
        a.entropy = p.entropy ? p.entropy + r0 : nullptr;
        a.top_logprob = p.top_logprob ? p.top_logprob + (size_t)r0 * p.k : nullptr;
        a.top_id = p.top_id ? p.top_id + (size_t)r0 * p.k : nullptr;
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3((unsigned)S, n);
        cfg.blockDim = dim3(kWarps * 32);
        cfg.stream = s;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
        e = cudaLaunchKernelEx(&cfg, logprob_kernel, a);
        if (e != cudaSuccess)
            return e;
    }
    return cudaSuccess;
}

} // namespace w4
