// C ABI of libw4a16.so: argument validation, per-device set-up and dispatch.
// The declarations, with the meaning, layout, ownership and error behaviour of
// every argument, are in include/w4a16.h.
#include "../../include/w4a16.h"
#include "internal.h"

#include <atomic>
#include <cstdio>
#include <cstdlib>
#include <cstring>
#include <mutex>

namespace {

constexpr int kMaxDevices = 64;
// Argmax scratch: one 64-bit key per (x-row, CTA); 8 rows x 65536 CTAs.
constexpr size_t kKeyCapacity = 8u * 65536u;
// Prefill split-K scratch: 8 Mi fp32 partials (32 MiB).
constexpr size_t kWsFloats = 8u << 20;
// The same allocation is the scratch of the tiled attention (two partial row
// tiles per SM, about 39 MiB) and of the log probabilities.
size_t ws_capacity(int num_sms)
{
    const size_t n = w4::attn_ws_floats(num_sms);
    return n > kWsFloats ? n : kWsFloats;
}

constexpr size_t kLeftBytes = w4::kLogprobRows * sizeof(unsigned long long);

struct DeviceState {
    // Set (release) once the fields below are written; read (acquire) first.
    std::atomic<bool> ready{false};
    int num_sms = 0;
    unsigned long long *keys = nullptr;
    int *err = nullptr; // device error word written by kernels whose bounded waits ran out
    // Log probabilities: blocks of each row that have finished (zeros between calls).
    unsigned long long *left = nullptr;
    float *ws = nullptr; // prefill split-K and attention partials, ws_capacity(num_sms) floats
};

DeviceState g_dev[kMaxDevices];

std::mutex g_mu;
thread_local char g_cuda_err[256] = "";

int cuda_fail(cudaError_t e)
{
    std::snprintf(g_cuda_err, sizeof g_cuda_err, "%s: %s", cudaGetErrorName(e),
                  cudaGetErrorString(e));
    return W4_ERR_CUDA;
}

// Zeros, in place when the call returns. A stream of its own: a clear on the legacy
// stream would be ordered with neither the host nor a caller's non-blocking stream.
cudaError_t clear_now(void *p, size_t bytes)
{
    cudaStream_t s = nullptr;
    cudaError_t e = cudaStreamCreateWithFlags(&s, cudaStreamNonBlocking);
    if (e != cudaSuccess)
        return e;
    e = cudaMemsetAsync(p, 0, bytes, s);
    if (e == cudaSuccess)
        e = cudaStreamSynchronize(s);
    const cudaError_t d = cudaStreamDestroy(s);
    return e == cudaSuccess ? d : e;
}

// Set up (once) and return the state of the current device.
int device_state(DeviceState **out)
{
    int dev = -1;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) {
        cudaGetLastError();
        return W4_ERR_NO_DEVICE;
    }
    if (dev < 0 || dev >= kMaxDevices)
        return W4_ERR_NO_DEVICE;
    DeviceState &st = g_dev[dev];
    if (st.ready.load(std::memory_order_acquire)) {
        *out = &st;
        return W4_OK;
    }
    std::lock_guard<std::mutex> lk(g_mu);
    if (!st.ready.load(std::memory_order_relaxed)) {
        int major = 0, minor = 0, sms = 0;
        if (cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev) != cudaSuccess ||
            cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev) != cudaSuccess ||
            cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) {
            cudaGetLastError();
            return W4_ERR_NO_DEVICE;
        }
        if (major != 10 || minor != 3)
            return W4_ERR_NO_DEVICE; // kernels are built for sm_103a only
        void *p = nullptr;
        e = cudaMalloc(&p, kKeyCapacity * sizeof(unsigned long long) + 256);
        if (e != cudaSuccess)
            return cuda_fail(e);
        st.keys = static_cast<unsigned long long *>(p);
        st.err = reinterpret_cast<int *>(static_cast<char *>(p) + kKeyCapacity * sizeof(unsigned long long));
        e = clear_now(st.err, sizeof(int));
        if (e != cudaSuccess)
            return cuda_fail(e);
        void *w = nullptr;
        const size_t ws_bytes = ws_capacity(sms) * sizeof(float); // a multiple of 32
        e = cudaMalloc(&w, ws_bytes + kLeftBytes);
        if (e != cudaSuccess)
            return cuda_fail(e);
        st.ws = static_cast<float *>(w);
        st.left = reinterpret_cast<unsigned long long *>(static_cast<char *>(w) + ws_bytes);
        e = clear_now(st.left, kLeftBytes);
        if (e != cudaSuccess)
            return cuda_fail(e);
        st.num_sms = sms;
        // One-time lookups that plans use, done here so that a call captured
        // into a graph later makes none of them.
        w4::tmap_encoder();
        w4::m8_cluster_capacity();
        st.ready.store(true, std::memory_order_release);
    }
    *out = &st;
    return W4_OK;
}

bool aligned(const void *p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

int check_attn_args(const float *out, const uint16_t *q, const uint16_t *k, const uint16_t *v,
                    const int32_t *kpos, int window, int H, int T, int D)
{
    if (!out || !q || !k || !v)
        return W4_ERR_INVALID_ARG;
    if (H < 1 || T < 1 || D < 1 || window < 0)
        return W4_ERR_INVALID_ARG;
    if (H > 8 || D % 128 != 0 || D > 512)
        return W4_ERR_UNSUPPORTED;
    if ((long long)T * D >= (1ll << 31))
        return W4_ERR_INVALID_ARG;
    if (!aligned(q, 16) || !aligned(k, 16) || !aligned(v, 16) || !aligned(out, 4) ||
        (kpos && !aligned(kpos, 4)))
        return W4_ERR_MISALIGNED;
    return W4_OK;
}

// Rows (or slots, over all sequences) of the tiled attention calls at most: the ends of
// key tiles that begin below are 32-bit numbers too.
constexpr long long kAttnRows = 2147483647 - 1024;

// Row tiles of a tiled attention call at most; their numbers are 32-bit.
bool too_many_tiles(long long rows, int seqs, int Hq, int Hkv, int D)
{
    return rows / w4::attn_tile_tokens(Hq / Hkv, D) + seqs > 2147483647 / (w4::attn_slices(D) * (long long)Hkv);
}

// Head layout, width, window and scale of the tiled attention calls.
int check_heads(int Hq, int Hkv, int D, int window, float scale)
{
    if (Hq < 1 || Hkv < 1 || D < 1 || window < 0 || !(scale > 0.f) || !(scale <= 3.4e38f))
        return W4_ERR_INVALID_ARG;
    if (Hq % Hkv != 0)
        return W4_ERR_INVALID_ARG;
    if (Hq / Hkv > 128 || !(D == 64 || D == 128 || D == 256 || D == 384 || D == 512))
        return W4_ERR_UNSUPPORTED;
    return W4_OK;
}

int check_w4_args(const void *y, const uint16_t *x, const uint32_t *qw, const uint16_t *sc, int M,
                  int N, int K, int group)
{
    if (!y || !x || !qw || !sc)
        return W4_ERR_INVALID_ARG;
    if (M <= 0 || N <= 0 || K <= 0)
        return W4_ERR_INVALID_ARG;
    if (w4::group_shift(group) < 0)
        return W4_ERR_UNSUPPORTED;
    if (K % group != 0)
        return W4_ERR_INVALID_ARG;
    // Every flat index the kernels form stays below 2^31 words or elements.
    if ((long long)N * (K / 8) >= (1ll << 31) || (long long)M * K >= (1ll << 31) ||
        (long long)M * N >= (1ll << 31))
        return W4_ERR_INVALID_ARG;
    if (!aligned(x, 16) || !aligned(qw, 16) || !aligned(sc, 4) || !aligned(y, 4))
        return W4_ERR_MISALIGNED;
    return W4_OK;
}

// Shared memory the decode kernels need for x staging; bounded by the SM's 227 KB.
bool decode_fits(const w4::DecodePlan &p, int M, int K)
{
    return w4::decode_smem_bytes(p, M, K) <= 220 * 1024;
}

} // namespace

extern "C" {

const char *w4_status_string(int status)
{
    switch (status) {
    case W4_OK: return "W4_OK";
    case W4_ERR_INVALID_ARG: return "W4_ERR_INVALID_ARG";
    case W4_ERR_UNSUPPORTED: return "W4_ERR_UNSUPPORTED";
    case W4_ERR_MISALIGNED: return "W4_ERR_MISALIGNED";
    case W4_ERR_CUDA: return "W4_ERR_CUDA";
    case W4_ERR_NO_DEVICE: return "W4_ERR_NO_DEVICE";
    default: return "W4_ERR_UNKNOWN";
    }
}

const char *w4_last_cuda_error(void) { return g_cuda_err; }

int w4_init(void)
{
    DeviceState *st = nullptr;
    return device_state(&st);
}

int w4a16_gemv(float *y, const uint16_t *x, const uint32_t *qweight, const uint16_t *scales, int M,
               int N, int K, int group, void *stream)
{
    int rc = check_w4_args(y, x, qweight, scales, M, N, K, group);
    if (rc != W4_OK)
        return rc;
    if (M > 8)
        return W4_ERR_UNSUPPORTED;
    DeviceState *st = nullptr;
    if ((rc = device_state(&st)) != W4_OK)
        return rc;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const int lg = w4::group_shift(group);
    if (w4::vocab_supported(M, N, K, st->num_sms, lg, qweight, scales)) {
        cudaError_t e = w4::run_decode_vocab(y, x, qweight, scales, N, K, lg, nullptr, nullptr, st->err,
                                             st->num_sms, s);
        return e == cudaSuccess ? W4_OK : cuda_fail(e);
    }
    if (M == 1) {
        // Measured on GB300 in the graph-replayed sweep: the slot form first
        // (0.505 -> 0.473 ms; 1536 x 6144 3.56 -> 3.29 us, 2560 x 1536 2.23 ->
        // 2.19 us), the few-tiles-per-warp form for the shapes it cannot take
        // (K % 768 != 0: 1536 x 2048).
        const int R = w4::slab_rows_per_cta(M, N, K, st->num_sms, lg, qweight, scales);
        if (R > 0) {
            cudaError_t e = w4::run_decode_slab(R, y, x, qweight, scales, N, K, st->err, s);
            return e == cudaSuccess ? W4_OK : cuda_fail(e);
        }
        const w4::M1Plan mp = w4::plan_decode_m1(M, N, K, st->num_sms);
        if (mp.ok) {
            cudaError_t e = w4::run_decode_m1(mp, y, x, qweight, scales, N, K, lg, s);
            return e == cudaSuccess ? W4_OK : cuda_fail(e);
        }
    } else {
        const w4::Slots8Plan sp = w4::plan_slots8(M, N, K, st->num_sms, lg, qweight, scales);
        if (sp.ok) {
            cudaError_t e = w4::run_decode_slots8(sp, y, x, qweight, scales, M, N, K, nullptr, nullptr, st->err, s);
            return e == cudaSuccess ? W4_OK : cuda_fail(e);
        }
    }
    const w4::DecodePlan p = w4::plan_decode(M, N, K, st->num_sms);
    if (!decode_fits(p, M, K))
        return W4_ERR_UNSUPPORTED;
    cudaError_t e = w4::run_decode(p, y, x, qweight, scales, M, N, K, lg, nullptr, nullptr, s);
    return e == cudaSuccess ? W4_OK : cuda_fail(e);
}

int w4a16_gemm(float *y, const uint16_t *x, const uint32_t *qweight, const uint16_t *scales, int M,
               int N, int K, int group, void *stream)
{
    if (M >= 1 && M <= 8)
        return w4a16_gemv(y, x, qweight, scales, M, N, K, group, stream);
    int rc = check_w4_args(y, x, qweight, scales, M, N, K, group);
    if (rc != W4_OK)
        return rc;
    if (N % 16 != 0 || K % 64 != 0)
        return W4_ERR_UNSUPPORTED;
    DeviceState *st = nullptr;
    if ((rc = device_state(&st)) != W4_OK)
        return rc;
    const w4::PrefillPlan p = w4::plan_prefill(M, N, K, st->num_sms, kWsFloats);
    cudaError_t e = w4::run_prefill(p, y, x, qweight, scales, M, N, K, w4::group_shift(group), st->ws, st->err,
                                    static_cast<cudaStream_t>(stream));
    if (e == cudaErrorNotSupported)
        return W4_ERR_UNSUPPORTED;
    return e == cudaSuccess ? W4_OK : cuda_fail(e);
}

int w4a16_gemv_argmax(float *y, int32_t *argmax, const uint16_t *x, const uint32_t *qweight,
                      const uint16_t *scales, int M, int N, int K, int group, void *stream)
{
    int rc = check_w4_args(y, x, qweight, scales, M, N, K, group);
    if (rc != W4_OK)
        return rc;
    if (!argmax)
        return W4_ERR_INVALID_ARG;
    if (!aligned(argmax, 4))
        return W4_ERR_MISALIGNED;
    if (M > 8)
        return W4_ERR_UNSUPPORTED;
    DeviceState *st = nullptr;
    if ((rc = device_state(&st)) != W4_OK)
        return rc;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const int lg = w4::group_shift(group);
    if (w4::vocab_supported(M, N, K, st->num_sms, lg, qweight, scales)) {
        cudaError_t e = w4::run_decode_vocab(y, x, qweight, scales, N, K, lg, st->keys, argmax, st->err,
                                             st->num_sms, s);
        return e == cudaSuccess ? W4_OK : cuda_fail(e);
    }
    if (M >= 2) {
        const w4::Slots8Plan sp = w4::plan_slots8(M, N, K, st->num_sms, lg, qweight, scales);
        if (sp.ok && (size_t)M * sp.grid <= kKeyCapacity) {
            cudaError_t e = w4::run_decode_slots8(sp, y, x, qweight, scales, M, N, K, st->keys, argmax, st->err, s);
            return e == cudaSuccess ? W4_OK : cuda_fail(e);
        }
    }
    const w4::DecodePlan p = w4::plan_decode(M, N, K, st->num_sms);
    if (!decode_fits(p, M, K) || (size_t)M * p.grid > kKeyCapacity)
        return W4_ERR_UNSUPPORTED;
    cudaError_t e = w4::run_decode(p, y, x, qweight, scales, M, N, K, lg, st->keys, argmax, s);
    return e == cudaSuccess ? W4_OK : cuda_fail(e);
}

int w4_embed_gather(uint16_t *out, const int32_t *ids, const uint32_t *qtable,
                    const uint16_t *scales, int M, int N, int K, int group, int32_t *status,
                    void *stream)
{
    if (!out || !ids || !qtable || !scales)
        return W4_ERR_INVALID_ARG;
    if (M <= 0 || N <= 0 || K <= 0)
        return W4_ERR_INVALID_ARG;
    if (w4::group_shift(group) < 0)
        return W4_ERR_UNSUPPORTED;
    if (K % group != 0)
        return W4_ERR_INVALID_ARG;
    if ((long long)N * (K / 8) >= (1ll << 31) || (long long)M * K >= (1ll << 31))
        return W4_ERR_INVALID_ARG;
    if (!aligned(out, 16) || !aligned(qtable, 4) || !aligned(scales, 2) || !aligned(ids, 4) ||
        (status && !aligned(status, 4)))
        return W4_ERR_MISALIGNED;
    DeviceState *st = nullptr;
    int rc = device_state(&st);
    if (rc != W4_OK)
        return rc;
    cudaError_t e = w4::run_embed_gather(out, ids, qtable, scales, M, N, K, w4::group_shift(group), status,
                                         static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? W4_OK : cuda_fail(e);
}

int w4_device_error(int32_t *code)
{
    if (!code)
        return W4_ERR_INVALID_ARG;
    DeviceState *st = nullptr;
    int rc = device_state(&st);
    if (rc != W4_OK)
        return rc;
    cudaError_t e = cudaDeviceSynchronize();
    if (e == cudaSuccess)
        e = cudaMemcpy(code, st->err, sizeof(int32_t), cudaMemcpyDeviceToHost);
    if (e == cudaSuccess)
        e = clear_now(st->err, sizeof(int32_t));
    return e == cudaSuccess ? W4_OK : cuda_fail(e);
}

int hbm_read_probe(unsigned long long *sum, const void *buf, size_t bytes, void *stream)
{
    if (!sum || !buf || bytes == 0)
        return W4_ERR_INVALID_ARG;
    if (bytes % 16 != 0)
        return W4_ERR_INVALID_ARG;
    if (!aligned(buf, 16) || !aligned(sum, 8))
        return W4_ERR_MISALIGNED;
    DeviceState *st = nullptr;
    int rc = device_state(&st);
    if (rc != W4_OK)
        return rc;
    cudaError_t e = w4::run_read_probe(sum, buf, bytes, st->num_sms, static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? W4_OK : cuda_fail(e);
}

int w4_attn_decode(float *out, const uint16_t *q, const uint16_t *k, const uint16_t *v,
                   const int32_t *kpos, int qpos, int window, int H, int T, int D, float scale,
                   void *stream)
{
    int rc = check_attn_args(out, q, k, v, kpos, window, H, T, D);
    if (rc != W4_OK)
        return rc;
    DeviceState *st = nullptr;
    if ((rc = device_state(&st)) != W4_OK)
        return rc;
    cudaError_t e = w4::run_attn_decode(out, q, k, v, kpos, qpos, nullptr, window, H, T, D, scale, st->ws,
                                        kWsFloats, st->num_sms, static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? W4_OK : cuda_fail(e);
}

int w4a16_gemv_hadamard(float *y, int32_t *argmax, const uint16_t *x, const uint32_t *qweight,
                        const uint16_t *scales, int M, int N, int K, int group, int hblock, void *stream)
{
    int rc = check_w4_args(y, x, qweight, scales, M, N, K, group);
    if (rc != W4_OK)
        return rc;
    if (hblock < 2 || hblock > 4096 || (hblock & (hblock - 1)) != 0)
        return W4_ERR_UNSUPPORTED;
    if (K % hblock != 0)
        return W4_ERR_INVALID_ARG;
    if (M > 4)
        return W4_ERR_UNSUPPORTED;
    if (argmax && !aligned(argmax, 4))
        return W4_ERR_MISALIGNED;
    DeviceState *st = nullptr;
    if ((rc = device_state(&st)) != W4_OK)
        return rc;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    // One x-row, blocks of 256 or 512, K % 128 == 0, the shared-memory slot
    // form or the M <= 2 kernel (not the large-N forms, where the separate
    // transform overlaps the weight preload and measured faster): the decode
    // kernel forms x H itself while staging x (no transform launch, no scratch
    // rows).
    if (M == 1 && !argmax) {
        const int R = w4::slab_rows_per_cta(M, N, K, st->num_sms, w4::group_shift(group), qweight, scales, hblock);
        if (R > 0) {
            cudaError_t e = w4::run_decode_slab(R, y, x, qweight, scales, N, K, st->err, s, hblock);
            return e == cudaSuccess ? W4_OK : cuda_fail(e);
        }
    }
    if (M == 1 && (hblock == 256 || hblock == 512) && K % 128 == 0) {
        const w4::DecodePlan p = w4::plan_decode(2, N, K, st->num_sms);
        if (p.kernel == 2 && decode_fits(p, 2, K) && (!argmax || (size_t)p.grid <= kKeyCapacity)) {
            cudaError_t e = w4::run_decode(p, y, x, qweight, scales, 2, N, K, w4::group_shift(group),
                                           argmax ? st->keys : nullptr, argmax, s, true, nullptr, hblock);
            return e == cudaSuccess ? W4_OK : cuda_fail(e);
        }
    }
    // The rotated activation's (hi, lo) rows live in the split scratch.
    if ((size_t)2 * M * K * sizeof(uint16_t) > kWsFloats * sizeof(float))
        return W4_ERR_UNSUPPORTED;
    const w4::DecodePlan p = w4::plan_decode(2 * M, N, K, st->num_sms);
    if (!decode_fits(p, 2 * M, K) || (argmax && (size_t)M * p.grid > kKeyCapacity))
        return W4_ERR_UNSUPPORTED;
    uint16_t *x2 = reinterpret_cast<uint16_t *>(st->ws);
    cudaError_t e = w4::run_hadamard_split(x2, x, M, K, hblock, s);
    if (e == cudaSuccess)
        e = w4::run_decode(p, y, x2, qweight, scales, 2 * M, N, K, w4::group_shift(group),
                           argmax ? st->keys : nullptr, argmax, s, true);
    return e == cudaSuccess ? W4_OK : cuda_fail(e);
}

int w4_selftest_wait_timeout(void *stream)
{
    DeviceState *st = nullptr;
    int rc = device_state(&st);
    if (rc != W4_OK)
        return rc;
    cudaError_t e = w4::run_bounded_wait_selftest(st->err, static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? W4_OK : cuda_fail(e);
}

int w4_attn_decode_devpos(float *out, const uint16_t *q, const uint16_t *k, const uint16_t *v,
                          const int32_t *kpos, const int32_t *qpos, int window, int H, int T, int D,
                          float scale, void *stream)
{
    int rc = check_attn_args(out, q, k, v, kpos, window, H, T, D);
    if (rc != W4_OK)
        return rc;
    if (!qpos)
        return W4_ERR_INVALID_ARG;
    if (!aligned(qpos, 4))
        return W4_ERR_MISALIGNED;
    DeviceState *st = nullptr;
    if ((rc = device_state(&st)) != W4_OK)
        return rc;
    cudaError_t e = w4::run_attn_decode(out, q, k, v, kpos, 0, qpos, window, H, T, D, scale, st->ws, kWsFloats,
                                        st->num_sms, static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? W4_OK : cuda_fail(e);
}

int w4_kv_append(uint16_t *k_cache, uint16_t *v_cache, int32_t *kpos, const uint16_t *k_new,
                 const uint16_t *v_new, const int32_t *pos, int T, int D, int32_t *status, void *stream)
{
    if (!k_cache || !v_cache || !k_new || !v_new || !pos)
        return W4_ERR_INVALID_ARG;
    if (T < 1 || D < 8 || D % 8 != 0 || (long long)T * D >= (1ll << 31))
        return W4_ERR_INVALID_ARG;
    if (!aligned(k_cache, 16) || !aligned(v_cache, 16) || !aligned(k_new, 16) || !aligned(v_new, 16) ||
        !aligned(pos, 4) || (kpos && !aligned(kpos, 4)) || (status && !aligned(status, 4)))
        return W4_ERR_MISALIGNED;
    DeviceState *st = nullptr;
    int rc = device_state(&st);
    if (rc != W4_OK)
        return rc;
    cudaError_t e = w4::run_kv_append(k_cache, v_cache, kpos, k_new, v_new, pos, T, D, status,
                                      static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? W4_OK : cuda_fail(e);
}

int w4a16_gemv_argmax_forced(float *y, int32_t *argmax, const uint16_t *x, const uint32_t *qweight,
                             const uint16_t *scales, int N, int K, int group, const int32_t *forced,
                             void *stream)
{
    int rc = check_w4_args(y, x, qweight, scales, 1, N, K, group);
    if (rc != W4_OK)
        return rc;
    if (!argmax || !forced)
        return W4_ERR_INVALID_ARG;
    if (!aligned(argmax, 4) || !aligned(forced, 4))
        return W4_ERR_MISALIGNED;
    DeviceState *st = nullptr;
    if ((rc = device_state(&st)) != W4_OK)
        return rc;
    const int lg = w4::group_shift(group);
    if (w4::vocab_supported(1, N, K, st->num_sms, lg, qweight, scales)) {
        cudaError_t e = w4::run_decode_vocab(y, x, qweight, scales, N, K, lg, st->keys, argmax, st->err,
                                             st->num_sms, static_cast<cudaStream_t>(stream), forced);
        return e == cudaSuccess ? W4_OK : cuda_fail(e);
    }
    const w4::DecodePlan p = w4::plan_decode(1, N, K, st->num_sms);
    if (p.kernel == 8 || !decode_fits(p, 1, K) || (size_t)p.grid > kKeyCapacity)
        return W4_ERR_UNSUPPORTED;
    cudaError_t e = w4::run_decode(p, y, x, qweight, scales, 1, N, K, w4::group_shift(group), st->keys, argmax,
                                   static_cast<cudaStream_t>(stream), false, forced);
    return e == cudaSuccess ? W4_OK : cuda_fail(e);
}

int w4_decode_prologue(uint16_t *x_next, int32_t *tokens, int32_t *pos, const int32_t *token,
                       const uint32_t *qtable, const uint16_t *scales, int V, int K, int group, int cap,
                       int32_t *status, void *stream)
{
    if (!x_next || !pos || !token || !qtable || !scales)
        return W4_ERR_INVALID_ARG;
    if (V < 1 || K < 1 || (tokens && cap < 1))
        return W4_ERR_INVALID_ARG;
    if (w4::group_shift(group) < 0)
        return W4_ERR_UNSUPPORTED;
    if (K % group != 0 || (long long)V * (K / 8) >= (1ll << 31))
        return W4_ERR_INVALID_ARG;
    if (!aligned(x_next, 16) || !aligned(qtable, 4) || !aligned(scales, 2) || !aligned(pos, 4) ||
        !aligned(token, 4) || (tokens && !aligned(tokens, 4)) || (status && !aligned(status, 4)))
        return W4_ERR_MISALIGNED;
    DeviceState *st = nullptr;
    int rc = device_state(&st);
    if (rc != W4_OK)
        return rc;
    cudaError_t e = w4::run_decode_prologue(x_next, tokens, pos, token, qtable, scales, V, K,
                                            w4::group_shift(group), tokens ? cap : 0, status,
                                            static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? W4_OK : cuda_fail(e);
}

int w4_attn_prompt(uint16_t *out, const uint16_t *q, const uint16_t *k, const uint16_t *v, const int32_t *cu_q,
                   const int32_t *cu_k, int B, int total_q, int total_k, int Hq, int Hkv, int D, long long ldq,
                   long long ldk, long long ldv, long long ldo, int window, float scale, void *stream)
{
    if (!out || !q || !k || !v || !cu_q)
        return W4_ERR_INVALID_ARG;
    if (B < 1 || total_q < 1 || total_k < 1)
        return W4_ERR_INVALID_ARG;
    int rc = check_heads(Hq, Hkv, D, window, scale);
    if (rc != W4_OK)
        return rc;
    if (B > 4096 || total_q > kAttnRows || total_k > kAttnRows || too_many_tiles(total_q, B, Hq, Hkv, D))
        return W4_ERR_UNSUPPORTED;
    const long long wq = (long long)Hq * D, wk = (long long)Hkv * D, most = (1ll << 31) - 1;
    if (ldq < wq || ldo < wq || ldk < wk || ldv < wk || ldq > most || ldk > most || ldv > most || ldo > most)
        return W4_ERR_INVALID_ARG;
    if (ldq % 8 != 0 || ldk % 8 != 0 || ldv % 8 != 0 || ldo % 8 != 0)
        return W4_ERR_MISALIGNED;
    if (!aligned(out, 16) || !aligned(q, 16) || !aligned(k, 16) || !aligned(v, 16) || !aligned(cu_q, 4) ||
        (cu_k && !aligned(cu_k, 4)))
        return W4_ERR_MISALIGNED;
    DeviceState *st = nullptr;
    if ((rc = device_state(&st)) != W4_OK)
        return rc;
    w4::AttnPromptArgs p = {};
    p.out = out;
    p.q = q;
    p.k = k;
    p.v = v;
    p.cu_q = cu_q;
    p.cu_k = cu_k ? cu_k : cu_q;
    p.B = B;
    p.total_q = total_q;
    p.total_k = total_k;
    p.Hq = Hq;
    p.Hkv = Hkv;
    p.D = D;
    p.ldq = ldq;
    p.ldk = ldk;
    p.ldv = ldv;
    p.ldo = ldo;
    p.window = window;
    p.scale = scale;
    cudaError_t e = w4::run_attn_prompt(p, st->ws, st->err, st->num_sms, static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? W4_OK : cuda_fail(e);
}

int w4_attn_tree(uint16_t *out, const uint16_t *q, const uint16_t *k, const uint16_t *v, const int32_t *kpos,
                 const uint16_t *k_tree, const uint16_t *v_tree, const int32_t *parents, const int32_t *pos, int B,
                 int N, int T, int Hq, int Hkv, int D, int window, float scale, void *stream)
{
    if (!out || !q || !k || !v || !k_tree || !v_tree || !parents || !pos)
        return W4_ERR_INVALID_ARG;
    if (B < 1 || N < 1 || T < 1)
        return W4_ERR_INVALID_ARG;
    int rc = check_heads(Hq, Hkv, D, window, scale);
    if (rc != W4_OK)
        return rc;
    if (B > 4096 || N > 64)
        return W4_ERR_UNSUPPORTED;
    if ((long long)B * T >= (1ll << 31) || (long long)Hq * D >= (1ll << 31))
        return W4_ERR_INVALID_ARG;
    if ((long long)B * T > kAttnRows || too_many_tiles((long long)B * N, B, Hq, Hkv, D))
        return W4_ERR_UNSUPPORTED;
    if (!aligned(out, 16) || !aligned(q, 16) || !aligned(k, 16) || !aligned(v, 16) || !aligned(k_tree, 16) ||
        !aligned(v_tree, 16) || !aligned(parents, 4) || !aligned(pos, 4) || (kpos && !aligned(kpos, 4)))
        return W4_ERR_MISALIGNED;
    DeviceState *st = nullptr;
    if ((rc = device_state(&st)) != W4_OK)
        return rc;
    w4::AttnTreeArgs p = {};
    p.out = out;
    p.q = q;
    p.k = k;
    p.v = v;
    p.kpos = kpos;
    p.k_tree = k_tree;
    p.v_tree = v_tree;
    p.parents = parents;
    p.pos = pos;
    p.B = B;
    p.N = N;
    p.T = T;
    p.Hq = Hq;
    p.Hkv = Hkv;
    p.D = D;
    p.window = window;
    p.scale = scale;
    cudaError_t e = w4::run_attn_tree(p, st->ws, st->err, st->num_sms, static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? W4_OK : cuda_fail(e);
}

namespace {

// Pages of a cache: sizes, and strides that keep rows, heads and pages apart.
int check_pages(int B, int Hkv, int D, int pages, int page, int table_pages, long long page_stride,
                long long row_stride, long long head_stride)
{
    if (B < 1 || pages < 1 || page < 1 || table_pages < 1)
        return W4_ERR_INVALID_ARG;
    if (B > 4096 || page < 16 || page > 1024 || (page & (page - 1)) != 0 || (long long)table_pages * page > kAttnRows)
        return W4_ERR_UNSUPPORTED;
    struct {
        long long stride, n;
    } d[3] = {{head_stride, Hkv}, {row_stride, page}, {page_stride, pages}};
    for (int i = 0; i < 3; ++i)
        if (d[i].stride < D || d[i].stride > (1ll << 38)) // a tensor copy's strides end at 2^40 bytes
            return W4_ERR_INVALID_ARG;
    if (head_stride % 64 != 0 || row_stride % 8 != 0 || page_stride % 8 != 0)
        return W4_ERR_MISALIGNED;
    if (head_stride / 64 * Hkv >= (1ll << 31)) // a tensor copy's coordinates
        return W4_ERR_UNSUPPORTED;
    for (int i = 0; i < 2; ++i) // ascending strides
        for (int j = 0; j < 2 - i; ++j)
            if (d[j].stride > d[j + 1].stride || (d[j].stride == d[j + 1].stride && d[j].n > d[j + 1].n)) {
                const auto t = d[j];
                d[j] = d[j + 1];
                d[j + 1] = t;
            }
    double extent = D;
    for (int i = 0; i < 3; ++i) {
        if (d[i].n > 1 && (double)d[i].stride < extent)
            return W4_ERR_INVALID_ARG;
        extent += (double)d[i].stride * (double)(d[i].n - 1);
    }
    return extent < 4.6e18 ? W4_OK : W4_ERR_INVALID_ARG;
}

int log2_of(int n)
{
    int r = 0;
    while ((1 << r) < n)
        ++r;
    return r;
}

// What both norm-and-rotation calls check.
int check_norm_rope(const w4::NormRopeArgs &a, int ldv_heads)
{
    if (a.M < 1 || a.Hq < 1 || a.Hkv < 0 || a.D < 1 || a.R < 0 || !(a.eps >= 0.f) || !(a.eps <= 3.4e38f) ||
        (long long)a.Hq + 2ll * a.Hkv >= (1ll << 20))
        return W4_ERR_INVALID_ARG;
    if (!(a.D == 64 || a.D == 128 || a.D == 256 || a.D == 384 || a.D == 512) || (a.R % 8 != 0 && a.R <= a.D))
        return W4_ERR_UNSUPPORTED;
    if (a.R > a.D || (a.R > 0 && !a.inv_freq))
        return W4_ERR_INVALID_ARG;
    const long long wq = (long long)a.Hq * a.D, wk = (long long)a.Hkv * a.D, most = (1ll << 31) - 1;
    if (a.ldq < wq || a.ldqo < wq || a.ldk < wk || a.ldv < (long long)ldv_heads * a.D || a.ldko < wk || a.ldq > most ||
        a.ldqo > most || a.ldk > most || a.ldv > most || a.ldko > most)
        return W4_ERR_INVALID_ARG;
    if (a.ldq % 8 != 0 || a.ldqo % 8 != 0 || a.ldk % 8 != 0 || a.ldv % 8 != 0 || a.ldko % 8 != 0)
        return W4_ERR_MISALIGNED;
    if (!aligned(a.q_out, 16) || !aligned(a.q, 16) || !aligned(a.k, 16) || !aligned(a.v, 16) || !aligned(a.k_out, 16) ||
        !aligned(a.k_pages, 16) || !aligned(a.v_pages, 16) || !aligned(a.q_weight, 16) || !aligned(a.k_weight, 16) ||
        !aligned(a.v_weight, 16) || !aligned(a.inv_freq, 4) || !aligned(a.pos, 4) || !aligned(a.table, 4) ||
        !aligned(a.lens, 4) || !aligned(a.cu_q, 4) || !aligned(a.status, 4))
        return W4_ERR_MISALIGNED;
    return W4_OK;
}

int do_norm_rope(const w4::NormRopeArgs &a, void *stream)
{
    DeviceState *st = nullptr;
    const int rc = device_state(&st);
    if (rc != W4_OK)
        return rc;
    cudaError_t e = w4::run_qk_norm_rope(a, st->num_sms, static_cast<cudaStream_t>(stream));
    if (e == cudaErrorNotSupported)
        return W4_ERR_UNSUPPORTED;
    return e == cudaSuccess ? W4_OK : cuda_fail(e);
}

} // namespace

int w4_lora(float *out, const float *y, const uint16_t *x, const uint16_t *a, const uint16_t *b, const int32_t *ids,
            const float *scale, int M, int N, int K, int R, int L, long long ldo, long long ldy, long long ldx,
            int32_t *status, void *stream)
{
    if (!out || !y || !x || !a || !b || !ids || M < 1 || N < 1 || K < 1 || R < 1 || L < 1)
        return W4_ERR_INVALID_ARG;
    if (N % 8 != 0 || K % 32 != 0)
        return W4_ERR_INVALID_ARG;
    if (R % 8 != 0 || R > 128 || N > 1 << 23)
        return W4_ERR_UNSUPPORTED;
    const long long most = (1ll << 31) - 1;
    if (ldo < N || ldy < N || ldx < K || ldo > most || ldy > most || ldx > most || (out == y && ldo != ldy))
        return W4_ERR_INVALID_ARG;
    if (ldo % 4 != 0 || ldy % 4 != 0 || ldx % 8 != 0)
        return W4_ERR_MISALIGNED;
    if (!aligned(out, 16) || !aligned(y, 16) || !aligned(x, 16) || !aligned(a, 16) || !aligned(b, 16) ||
        !aligned(ids, 4) || !aligned(scale, 4) || !aligned(status, 4))
        return W4_ERR_MISALIGNED;
    DeviceState *st = nullptr;
    const int rc = device_state(&st);
    if (rc != W4_OK)
        return rc;
    const w4::LoraArgs p = {out, y, x, a, b, ids, scale, M, N, K, R, L, ldo, ldy, ldx, status};
    cudaError_t e = w4::run_lora(p, st->ws, ws_capacity(st->num_sms), st->num_sms, static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? W4_OK : cuda_fail(e);
}

int w4_qk_norm_rope(uint16_t *q_out, uint16_t *k_out, const void *q, const void *k, const float *q_weight,
                    const float *k_weight, const float *inv_freq, const int32_t *pos, int M, int Hq, int Hkv, int D,
                    int R, long long ldq, long long ldk, long long ldqo, long long ldko, int f32, int pairs, float eps,
                    void *stream)
{
    if (!q_out || !q || !pos || (Hkv != 0 && (!k || !k_out)))
        return W4_ERR_INVALID_ARG;
    w4::NormRopeArgs a = {};
    a.q_out = q_out;
    a.k_out = k_out;
    a.q = q;
    a.k = k;
    a.q_weight = q_weight;
    a.k_weight = k_weight;
    a.inv_freq = inv_freq;
    a.pos = pos;
    a.M = M;
    a.Hq = Hq;
    a.Hkv = Hkv;
    a.D = D;
    a.R = R;
    a.ldq = ldq;
    a.ldk = Hkv == 0 ? 0 : ldk;
    a.ldqo = ldqo;
    a.ldko = Hkv == 0 ? 0 : ldko;
    a.eps = eps;
    a.f32 = f32 != 0;
    a.pairs = pairs != 0;
    const int rc = check_norm_rope(a, 0);
    return rc == W4_OK ? do_norm_rope(a, stream) : rc;
}

int w4_qkv_paged(uint16_t *q_out, uint16_t *k_pages, uint16_t *v_pages, const void *q, const void *k, const void *v,
                 const float *q_weight, const float *k_weight, const float *v_weight, const float *inv_freq,
                 const int32_t *table, const int32_t *lens, const int32_t *cu_q, int B, int M, int Hq, int Hkv, int D,
                 int R, int pages, int page, int table_pages, long long ldq, long long ldk, long long ldv,
                 long long ldqo, long long page_stride, long long row_stride, long long head_stride, int f32,
                 int pairs, float eps, int32_t *status, void *stream)
{
    if (!q_out || !k_pages || !v_pages || !q || !k || !v || !table || !lens || Hkv < 1 || (!cu_q && M != B))
        return W4_ERR_INVALID_ARG;
    w4::NormRopeArgs a = {};
    a.q_out = q_out;
    a.k_pages = k_pages;
    a.v_pages = v_pages;
    a.q = q;
    a.k = k;
    a.v = v;
    a.q_weight = q_weight;
    a.k_weight = k_weight;
    a.v_weight = v_weight;
    a.inv_freq = inv_freq;
    a.table = table;
    a.lens = lens;
    a.cu_q = cu_q;
    a.M = M;
    a.B = B;
    a.Hq = Hq;
    a.Hkv = Hkv;
    a.D = D;
    a.R = R;
    a.pages = pages;
    a.table_pages = table_pages;
    a.ldq = ldq;
    a.ldk = ldk;
    a.ldv = ldv;
    a.ldqo = ldqo;
    a.ldko = (long long)Hkv * D; // no rows of keys
    a.page_stride = page_stride;
    a.row_stride = row_stride;
    a.head_stride = head_stride;
    a.eps = eps;
    a.f32 = f32 != 0;
    a.pairs = pairs != 0;
    a.status = status;
    int rc = check_norm_rope(a, Hkv);
    if (rc == W4_OK)
        rc = check_pages(B, Hkv, D, pages, page, table_pages, page_stride, row_stride, head_stride);
    if (rc != W4_OK)
        return rc;
    a.page_log2 = log2_of(page);
    return do_norm_rope(a, stream);
}

int w4_attn_paged(uint16_t *out, const uint16_t *q, const uint16_t *k_pages, const uint16_t *v_pages,
                  const int32_t *table, const int32_t *lens, const int32_t *cu_q, int B, int total_q, int Hq, int Hkv,
                  int D, int pages, int page, int table_pages, long long ldq, long long ldo, long long page_stride,
                  long long row_stride, long long head_stride, int window, float scale, void *stream)
{
    if (!out || !q || !k_pages || !v_pages || !table || !lens)
        return W4_ERR_INVALID_ARG;
    if (total_q < 1 || (!cu_q && total_q != B))
        return W4_ERR_INVALID_ARG;
    int rc = check_heads(Hq, Hkv, D, window, scale);
    if (rc == W4_OK)
        rc = check_pages(B, Hkv, D, pages, page, table_pages, page_stride, row_stride, head_stride);
    if (rc != W4_OK)
        return rc;
    if (total_q > kAttnRows || too_many_tiles(total_q, B, Hq, Hkv, D))
        return W4_ERR_UNSUPPORTED;
    const long long wq = (long long)Hq * D, most = (1ll << 31) - 1;
    if (ldq < wq || ldo < wq || ldq > most || ldo > most)
        return W4_ERR_INVALID_ARG;
    if (ldq % 8 != 0 || ldo % 8 != 0)
        return W4_ERR_MISALIGNED;
    if (!aligned(out, 16) || !aligned(q, 16) || !aligned(k_pages, 16) || !aligned(v_pages, 16) || !aligned(table, 4) ||
        !aligned(lens, 4) || !aligned(cu_q, 4))
        return W4_ERR_MISALIGNED;
    DeviceState *st = nullptr;
    if ((rc = device_state(&st)) != W4_OK)
        return rc;
    w4::AttnPagedArgs p = {};
    p.out = out;
    p.q = q;
    p.k_pages = k_pages;
    p.v_pages = v_pages;
    p.table = table;
    p.lens = lens;
    p.cu_q = cu_q;
    p.B = B;
    p.total_q = total_q;
    p.pages = pages;
    p.page_log2 = log2_of(page);
    p.table_pages = table_pages;
    p.Hq = Hq;
    p.Hkv = Hkv;
    p.D = D;
    p.ldq = ldq;
    p.ldo = ldo;
    p.page_stride = page_stride;
    p.row_stride = row_stride;
    p.head_stride = head_stride;
    p.window = window;
    p.scale = scale;
    cudaError_t e = w4::run_attn_paged(p, st->ws, st->err, st->num_sms, static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? W4_OK : cuda_fail(e);
}

int w4_logprobs(float *logprob, float *entropy, float *top_logprob, int32_t *top_id, const float *logits,
                const int32_t *targets, int M, int V, long long ld, int topk, int32_t *status, void *stream)
{
    if (!logits || (logprob && !targets))
        return W4_ERR_INVALID_ARG;
    if (M < 1 || V < 1 || ld < V || topk < 0)
        return W4_ERR_INVALID_ARG;
    if (topk > 32 || V > 2147483647 - 1024) // chunk ends past the row are 32-bit numbers too
        return W4_ERR_UNSUPPORTED;
    if (!aligned(logits, 4) || (targets && !aligned(targets, 4)) || (logprob && !aligned(logprob, 4)) ||
        (entropy && !aligned(entropy, 4)) || (top_logprob && !aligned(top_logprob, 4)) ||
        (top_id && !aligned(top_id, 4)) || (status && !aligned(status, 4)))
        return W4_ERR_MISALIGNED;
    if (!logprob && !entropy && (topk == 0 || (!top_logprob && !top_id)))
        return W4_ERR_INVALID_ARG; // nothing to compute
    DeviceState *st = nullptr;
    int rc = device_state(&st);
    if (rc != W4_OK)
        return rc;
    w4::LogprobsArgs p = {};
    p.logprob = logprob;
    p.entropy = entropy;
    p.top_logprob = top_logprob;
    p.top_id = top_id;
    p.logits = logits;
    p.targets = targets;
    p.M = M;
    p.V = V;
    p.ld = ld;
    p.k = top_logprob || top_id ? topk : 0;
    p.status = status;
    cudaError_t e = w4::run_logprobs(p, st->ws, ws_capacity(st->num_sms), st->left, st->num_sms,
                                     static_cast<cudaStream_t>(stream));
    if (e == cudaErrorNotSupported)
        return W4_ERR_UNSUPPORTED;
    return e == cudaSuccess ? W4_OK : cuda_fail(e);
}

int w4_kv_commit(uint16_t *k_cache, uint16_t *v_cache, int32_t *kpos, const uint16_t *k_tree,
                 const uint16_t *v_tree, const int32_t *path, const int32_t *count, const int32_t *pos, int L, int B,
                 int N, int T, int W, int32_t *status, void *stream)
{
    if (!k_cache || !v_cache || !k_tree || !v_tree || !path || !count || !pos)
        return W4_ERR_INVALID_ARG;
    if (L < 1 || B < 1 || N < 1 || T < 1 || W < 8 || W % 8 != 0 || (long long)L * B >= (1ll << 31))
        return W4_ERR_INVALID_ARG;
    if (N > 64)
        return W4_ERR_UNSUPPORTED;
    if (!aligned(k_cache, 16) || !aligned(v_cache, 16) || !aligned(k_tree, 16) || !aligned(v_tree, 16) ||
        !aligned(path, 4) || !aligned(count, 4) || !aligned(pos, 4) || (kpos && !aligned(kpos, 4)) ||
        (status && !aligned(status, 4)))
        return W4_ERR_MISALIGNED;
    DeviceState *st = nullptr;
    int rc = device_state(&st);
    if (rc != W4_OK)
        return rc;
    const w4::KvCommitArgs a = {k_cache, v_cache, kpos, k_tree, v_tree, path, count, pos, L, B, N, T, W, status};
    cudaError_t e = w4::run_kv_commit(a, static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? W4_OK : cuda_fail(e);
}

} // extern "C"
