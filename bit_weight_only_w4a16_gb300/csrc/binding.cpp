// The serving calls' usual case in native code: the same checks that the Python binding
// makes, on tensors as they are in memory, and the call of the C ABI.
//
// Why: these calls serve single tokens of many requests, and their host time is most of
// their time (the GPU is done in 4 to 10 us). Through Python a call with thirteen tensors
// took 17 us: 9 of checks, 3 of argument conversion, the rest the launch.
//
// Every function returns None for whatever is not plainly right - another type, a shape
// that does not fit, a subclass of torch.Tensor, arguments that the C call refuses (it then
// launched nothing) - and the Python code, which is complete by itself, makes the call or
// raises what is wrong with it. Any other error of the C call is raised here: a part of
// the call may have been launched, in place, and is not made a second time.
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include "../../include/w4a16.h"

#include <algorithm>
#include <cstdint>

namespace {

decltype(&w4_lora) p_lora;
decltype(&w4_qk_norm_rope) p_rope;
decltype(&w4_qkv_paged) p_qkv;
decltype(&w4_attn_paged) p_attn;

// Thrown where the Python code has to look.
struct Unusual {};

inline void need(bool ok)
{
    if (!ok)
        throw Unusual();
}

// Thrown where the C call failed; the Python function that raises it.
struct Failed {
    int status;
    const char *call;
};
PyObject *p_check;

// Makes the call. Other Python threads run meanwhile: a launch may wait for room in its
// stream's queue, whose work may wait for a host function that needs the interpreter.
template <typename F, typename... A>
void make(const char *call, F f, A... args)
{
    int status;
    Py_BEGIN_ALLOW_THREADS
    status = f(args...);
    Py_END_ALLOW_THREADS
    if (status == W4_ERR_INVALID_ARG || status == W4_ERR_UNSUPPORTED || status == W4_ERR_MISALIGNED)
        throw Unusual();
    if (status != W4_OK)
        throw Failed{status, call};
}

// A plain tensor (not a subclass) in memory.
const at::Tensor &tensor(PyObject *o)
{
    need(THPVariable_CheckExact(o));
    const at::Tensor &t = THPVariable_Unpack(o);
    need(t.defined() && t.layout() == at::kStrided && !t.is_conj() && !t.is_neg());
    return t;
}

// What a call's tensors have in common.
struct Call {
    int dev;
    cudaStream_t stream;
};

Call call_on(const at::Tensor &first, PyObject *stream)
{
    need(first.is_cuda());
    Call c;
    c.dev = first.get_device();
    need(c10::cuda::current_device() == c.dev);
    if (stream == Py_None) {
        c.stream = c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)c.dev).stream();
    } else {
        PyObject *s = PyObject_GetAttrString(stream, "cuda_stream");
        need(s != nullptr);
        c.stream = static_cast<cudaStream_t>(PyLong_AsVoidPtr(s));
        Py_DECREF(s);
        need(!PyErr_Occurred());
    }
    return c;
}

void on(const at::Tensor &t, const Call &c, at::ScalarType type)
{
    need(t.is_cuda() && t.get_device() == c.dev && t.scalar_type() == type);
}

int to_int(int64_t v)
{
    need(v >= 0 && v <= INT32_MAX);
    return (int)v;
}

int64_t number(PyObject *o)
{
    need(PyLong_Check(o));
    int over = 0;
    const long long v = PyLong_AsLongLongAndOverflow(o, &over);
    need(!over && v >= INT32_MIN && v <= INT32_MAX);
    return v;
}

float real(PyObject *o)
{
    const double v = PyFloat_AsDouble(o);
    need(!(v == -1.0 && PyErr_Occurred()));
    return (float)v;
}

// A contiguous vector of n words of this type, or null for None.
const void *words(PyObject *o, const Call &c, at::ScalarType type, int64_t n)
{
    if (o == Py_None)
        return nullptr;
    const at::Tensor &t = tensor(o);
    on(t, c, type);
    need(t.numel() == n && t.is_contiguous());
    return t.const_data_ptr();
}

const int32_t *ints(PyObject *o, const Call &c, int64_t n)
{
    return static_cast<const int32_t *>(words(o, c, at::kInt, n));
}

const float *weight(PyObject *o, const Call &c, int64_t n)
{
    const void *p = words(o, c, at::kFloat, n);
    need(!p || tensor(o).dim() == 1);
    return static_cast<const float *>(p);
}

// Rows of heads [rows][heads][D], rows strided: elements between rows.
int64_t rows_of(const at::Tensor &t, const Call &c, at::ScalarType type, int64_t rows, int64_t heads, int64_t D)
{
    on(t, c, type);
    need(t.dim() == 3 && t.size(0) == rows && t.size(1) == heads && t.size(2) == D);
    need((D == 1 || t.stride(2) == 1) && (heads == 1 || t.stride(1) == D));
    return rows > 1 ? t.stride(0) : heads * D;
}

// A matrix whose rows may be strided: elements between rows.
int64_t matrix(const at::Tensor &t, const Call &c, at::ScalarType type, int64_t rows, int64_t cols)
{
    on(t, c, type);
    need(t.dim() == 2 && t.size(0) == rows && t.size(1) == cols && (cols == 1 || t.stride(1) == 1));
    return rows > 1 ? t.stride(0) : cols;
}

// The given output, or a new one like `like` in type's place.
at::Tensor output(PyObject *o, at::IntArrayRef shape, const at::Tensor &like, at::ScalarType type)
{
    return o == Py_None ? at::empty(shape, like.options().dtype(type).requires_grad(false)) : tensor(o);
}

PyObject *give(PyObject *given, const at::Tensor &t)
{
    if (given != Py_None) {
        Py_INCREF(given);
        return given;
    }
    return THPVariable_Wrap(t);
}

struct Pool {
    uint16_t *k, *v;
    int pages, page;
    int64_t ps, rs, hs;
};

Pool pool(PyObject *ko, PyObject *vo, const Call &c, int64_t Hkv, int64_t D)
{
    const at::Tensor &k = tensor(ko), &v = tensor(vo);
    on(k, c, at::kBFloat16);
    on(v, c, at::kBFloat16);
    need(k.dim() == 4 && k.sizes() == v.sizes() && k.strides() == v.strides() && k.stride(3) == 1);
    need(k.size(2) == Hkv && k.size(3) == D);
    Pool p;
    p.k = static_cast<uint16_t *>(k.data_ptr());
    p.v = static_cast<uint16_t *>(v.data_ptr());
    p.pages = to_int(k.size(0));
    p.page = to_int(k.size(1));
    // Where there is one only, a stride that is in order.
    p.hs = Hkv > 1 ? k.stride(2) : D;
    p.rs = p.page > 1 ? k.stride(1) : D;
    p.ps = p.pages > 1 ? k.stride(0) : std::max(p.rs * p.page, p.hs * Hkv);
    return p;
}

struct Batch {
    int B, n;
    const int32_t *table, *lens, *cu;
};

Batch batch(PyObject *table, PyObject *lens, PyObject *cu, const Call &c, int64_t rows)
{
    const at::Tensor &t = tensor(table);
    need(t.dim() == 2 && lens != Py_None);
    Batch b;
    b.B = to_int(t.size(0));
    b.n = to_int(t.size(1));
    need(cu != Py_None || rows == b.B);
    b.table = ints(table, c, t.numel());
    b.lens = ints(lens, c, b.B);
    b.cu = ints(cu, c, (int64_t)b.B + 1);
    return b;
}

// (y, x, a, b, ids, scale, out, status, stream)
PyObject *lora(PyObject *const *a)
{
    const at::Tensor &y = tensor(a[0]), &x = tensor(a[1]), &la = tensor(a[2]), &lb = tensor(a[3]);
    const Call c = call_on(y, a[8]);
    need(y.dim() == 2 && la.dim() == 3 && lb.dim() == 3 && a[4] != Py_None);
    const int64_t M = y.size(0), N = y.size(1), L = la.size(0), R = la.size(1), K = la.size(2);
    on(la, c, at::kBFloat16);
    on(lb, c, at::kBFloat16);
    need(la.is_contiguous() && lb.is_contiguous() && lb.size(0) == L && lb.size(1) == N && lb.size(2) == R);
    const int64_t ldy = matrix(y, c, at::kFloat, M, N), ldx = matrix(x, c, at::kBFloat16, M, K);
    const int32_t *ids = ints(a[4], c, M);
    const float *scale = weight(a[5], c, L);
    int32_t *status = const_cast<int32_t *>(ints(a[7], c, 1));
    const int m = to_int(M), n = to_int(N), k = to_int(K), r = to_int(R), l = to_int(L);
    const at::Tensor out = output(a[6], {M, N}, y, at::kFloat);
    const int64_t ldo = matrix(out, c, at::kFloat, M, N);
    make("w4_lora", p_lora, static_cast<float *>(out.data_ptr()), static_cast<const float *>(y.const_data_ptr()),
         static_cast<const uint16_t *>(x.const_data_ptr()), static_cast<const uint16_t *>(la.const_data_ptr()),
         static_cast<const uint16_t *>(lb.const_data_ptr()), ids, scale, m, n, k, r, l, ldo, ldy, ldx, status,
         c.stream);
    return give(a[6], out);
}

bool is_f32(const at::Tensor &q)
{
    need(q.scalar_type() == at::kFloat || q.scalar_type() == at::kBFloat16);
    return q.scalar_type() == at::kFloat;
}

// Frequencies: their number twice (the turned elements).
const float *frequencies(PyObject *o, const Call &c, int &R)
{
    if (o == Py_None) {
        R = 0;
        return nullptr;
    }
    const int64_t n = tensor(o).numel();
    R = to_int(2 * n);
    return weight(o, c, n);
}

// (q, k, pos, inv_freq, q_weight, k_weight, eps, pairs, q_out, k_out, stream)
PyObject *rope(PyObject *const *a)
{
    const at::Tensor &q = tensor(a[0]);
    const Call c = call_on(q, a[10]);
    need(q.dim() == 3 && a[2] != Py_None);
    const bool f32 = is_f32(q);
    const int64_t M = q.size(0), Hq = q.size(1), D = q.size(2);
    const int64_t ldq = rows_of(q, c, q.scalar_type(), M, Hq, D);
    int R;
    const float *f = frequencies(a[3], c, R), *qw = weight(a[4], c, D), *kw = weight(a[5], c, D);
    const int32_t *pos = ints(a[2], c, M);
    const float eps = real(a[6]);
    const int pairs = PyObject_IsTrue(a[7]);
    need(pairs >= 0);
    const int m = to_int(M), hq = to_int(Hq), d = to_int(D);
    int64_t Hkv = 0, ldk = 0, ldko = 0;
    const void *kp = nullptr;
    at::Tensor ko;
    if (a[1] != Py_None) {
        const at::Tensor &k = tensor(a[1]);
        need(k.dim() == 3);
        Hkv = to_int(k.size(1));
        need(Hkv > 0);
        ldk = rows_of(k, c, q.scalar_type(), M, Hkv, D);
        kp = k.const_data_ptr();
        ko = output(a[9], {M, Hkv, D}, q, at::kBFloat16);
        ldko = rows_of(ko, c, at::kBFloat16, M, Hkv, D);
    } else {
        need(a[9] == Py_None);
    }
    const at::Tensor qo = output(a[8], {M, Hq, D}, q, at::kBFloat16);
    const int64_t ldqo = rows_of(qo, c, at::kBFloat16, M, Hq, D);
    make("w4_qk_norm_rope", p_rope, static_cast<uint16_t *>(qo.data_ptr()),
         kp ? static_cast<uint16_t *>(ko.data_ptr()) : nullptr, q.const_data_ptr(), kp, qw, kw, f, pos, m, hq,
         (int)Hkv, d, R, ldq, ldk, ldqo, ldko, f32, pairs, eps, c.stream);
    PyObject *first = give(a[8], qo);
    PyObject *second = Py_None;
    if (kp)
        second = give(a[9], ko);
    else
        Py_INCREF(second);
    PyObject *both = first && second ? PyTuple_Pack(2, first, second) : nullptr;
    Py_XDECREF(first);
    Py_XDECREF(second);
    return both;
}

// (q, k, v, k_pages, v_pages, table, lens, inv_freq, cu_q, q_weight, k_weight, v_weight, eps, pairs, q_out,
// status, stream)
PyObject *qkv(PyObject *const *a)
{
    const at::Tensor &q = tensor(a[0]), &k = tensor(a[1]), &v = tensor(a[2]);
    const Call c = call_on(q, a[16]);
    need(q.dim() == 3 && k.dim() == 3);
    const bool f32 = is_f32(q);
    const int64_t M = q.size(0), Hq = q.size(1), D = q.size(2), Hkv = k.size(1);
    const int64_t ldq = rows_of(q, c, q.scalar_type(), M, Hq, D), ldk = rows_of(k, c, q.scalar_type(), M, Hkv, D);
    const int64_t ldv = rows_of(v, c, q.scalar_type(), M, Hkv, D);
    const Pool p = pool(a[3], a[4], c, Hkv, D);
    const Batch b = batch(a[5], a[6], a[8], c, M);
    int R;
    const float *f = frequencies(a[7], c, R), *qw = weight(a[9], c, D), *kw = weight(a[10], c, D);
    const float *vw = weight(a[11], c, D);
    const float eps = real(a[12]);
    const int pairs = PyObject_IsTrue(a[13]);
    need(pairs >= 0);
    int32_t *status = const_cast<int32_t *>(ints(a[15], c, 1));
    const int m = to_int(M), hq = to_int(Hq), hkv = to_int(Hkv), d = to_int(D);
    const at::Tensor qo = output(a[14], {M, Hq, D}, q, at::kBFloat16);
    const int64_t ldqo = rows_of(qo, c, at::kBFloat16, M, Hq, D);
    make("w4_qkv_paged", p_qkv, static_cast<uint16_t *>(qo.data_ptr()), p.k, p.v, q.const_data_ptr(),
         k.const_data_ptr(), v.const_data_ptr(), qw, kw, vw, f, b.table, b.lens, b.cu, b.B, m, hq, hkv, d, R, p.pages,
         p.page, b.n, ldq, ldk, ldv, ldqo, p.ps, p.rs, p.hs, f32, pairs, eps, status, c.stream);
    return give(a[14], qo);
}

// (q, k_pages, v_pages, table, lens, cu_q, window, scale, out, stream)
PyObject *attn(PyObject *const *a)
{
    const at::Tensor &q = tensor(a[0]);
    const Call c = call_on(q, a[9]);
    need(q.dim() == 3);
    const int64_t M = q.size(0), Hq = q.size(1), D = q.size(2);
    const int64_t ldq = rows_of(q, c, at::kBFloat16, M, Hq, D);
    const at::Tensor &kp = tensor(a[1]);
    need(kp.dim() == 4);
    const int64_t Hkv = kp.size(2);
    const Pool p = pool(a[1], a[2], c, Hkv, D);
    const Batch b = batch(a[3], a[4], a[5], c, M);
    const int window = (int)number(a[6]);
    const float scale = real(a[7]);
    const int m = to_int(M), hq = to_int(Hq), hkv = to_int(Hkv), d = to_int(D);
    const at::Tensor out = output(a[8], {M, Hq, D}, q, at::kBFloat16);
    const int64_t ldo = rows_of(out, c, at::kBFloat16, M, Hq, D);
    make("w4_attn_paged", p_attn, static_cast<uint16_t *>(out.data_ptr()),
         static_cast<const uint16_t *>(q.const_data_ptr()), p.k, p.v, b.table, b.lens, b.cu, b.B, m, hq, hkv, d,
         p.pages, p.page, b.n, ldq, ldo, p.ps, p.rs, p.hs, window, scale, c.stream);
    return give(a[8], out);
}

template <PyObject *(*F)(PyObject *const *), int N>
PyObject *entry(PyObject *, PyObject *const *args, Py_ssize_t n)
{
    if (n == N) {
        try {
            return F(args);
        } catch (const Unusual &) {
        } catch (const Failed &f) {
            PyErr_Clear();
            PyObject *r = PyObject_CallFunction(p_check, "is", f.status, f.call);
            if (r) { // it raises
                Py_DECREF(r);
                PyErr_SetString(PyExc_RuntimeError, f.call);
            }
            return nullptr;
        } catch (...) { // the Python code meets it again and says what it is
        }
        PyErr_Clear();
    }
    Py_RETURN_NONE;
}

// The library's functions, by address, and at the first time the Python function that raises
// their errors (status, name).
PyObject *bind(PyObject *, PyObject *const *args, Py_ssize_t n)
{
    if (n != 5 && !(n == 4 && p_check)) {
        PyErr_SetString(PyExc_TypeError, "bind takes four addresses and a function");
        return nullptr;
    }
    void *p[4];
    for (int i = 0; i < 4; ++i) {
        p[i] = PyLong_AsVoidPtr(args[i]);
        if (PyErr_Occurred())
            return nullptr;
    }
    p_lora = reinterpret_cast<decltype(p_lora)>(p[0]);
    p_rope = reinterpret_cast<decltype(p_rope)>(p[1]);
    p_qkv = reinterpret_cast<decltype(p_qkv)>(p[2]);
    p_attn = reinterpret_cast<decltype(p_attn)>(p[3]);
    if (n == 5) {
        Py_INCREF(args[4]);
        Py_XDECREF(p_check);
        p_check = args[4];
    }
    Py_RETURN_NONE;
}

#define W4_ENTRY(f) reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)(void)>(f))
PyMethodDef methods[] = {
    {"bind", W4_ENTRY(bind), METH_FASTCALL, nullptr},
    {"lora", W4_ENTRY((entry<lora, 9>)), METH_FASTCALL, nullptr},
    {"rope", W4_ENTRY((entry<rope, 11>)), METH_FASTCALL, nullptr},
    {"qkv", W4_ENTRY((entry<qkv, 17>)), METH_FASTCALL, nullptr},
    {"attn", W4_ENTRY((entry<attn, 10>)), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

} // namespace

PyMODINIT_FUNC PyInit__binding(void) { return PyModule_Create(&module); }
