// Argument marshalling of the expert-layer calls for Python: the checks of
// binding.py's quick pass and the call of the C entry point in one step (0.4 us
// instead of 3.5 for attribute reads, tuples and ctypes, where the kernels of a
// decode step take 3 to 5).
//
// Each function answers the status of the call, or None where an operand is not
// plainly as expected; the binding then names what is wrong, or makes the call
// itself.  The entry points' addresses are handed in by bind(): this module links
// against torch alone and is optional.
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <climits>
#include <initializer_list>

#include "ar_fusion.h"

namespace {

decltype(&ar_fusion_route) g_route = nullptr;
decltype(&ar_fusion_expert_plan) g_plan = nullptr;
decltype(&ar_fusion_quant_blocks) g_quant = nullptr;
decltype(&ar_fusion_matmul_fp8) g_matmul = nullptr;
decltype(&ar_fusion_expert_matmul_fp8) g_expert_matmul = nullptr;
decltype(&ar_fusion_combine) g_combine = nullptr;

constexpr int64_t kBlock = AR_QUANT_BLOCK;

// not as expected: the caller takes the long way
struct Refused {};

void want(bool ok)
{
    if (!ok)
        throw Refused{};
}

const at::Tensor& tensor(PyObject* o)
{
    want(THPVariable_Check(o));
    return THPVariable_Unpack(o);
}

int as_int(PyObject* o)
{
    want(PyLong_Check(o));
    const long v = PyLong_AsLong(o);
    if (v == -1 && PyErr_Occurred()) {
        PyErr_Clear();
        throw Refused{};
    }
    want(v >= INT_MIN && v <= INT_MAX);
    return (int)v;
}

int extent(int64_t v)
{
    want(v >= 0 && v <= INT_MAX);
    return (int)v;
}

// enum ar_dtype of an element type
int element(const at::Tensor& t)
{
    switch (t.scalar_type()) {
    case at::kBFloat16: return AR_DT_BF16;
    case at::kHalf: return AR_DT_FP16;
    case at::kFloat: return AR_DT_FP32;
    default: throw Refused{};
    }
}

bool is_codes(const at::Tensor& t)
{
    return t.scalar_type() == at::kByte || t.scalar_type() == at::kFloat8_e4m3fn;
}

// the address of a contiguous tensor of this shape on `device`
void* at_shape(const at::Tensor& t, int device, std::initializer_list<int64_t> shape)
{
    want(t.is_cuda() && t.get_device() == device && t.is_contiguous());
    want(t.sizes() == c10::IntArrayRef(shape));
    return t.data_ptr();
}

template <class T>
T* typed(const at::Tensor& t, at::ScalarType type, int device, std::initializer_list<int64_t> shape)
{
    want(t.scalar_type() == type);
    return static_cast<T*>(at_shape(t, device, shape));
}

// the operands' device, which has to be the current one
int device_of(const at::Tensor& t)
{
    want(t.is_cuda());
    const int d = t.get_device();
    want(d == (int)c10::cuda::current_device());
    return d;
}

void* stream_of(PyObject* o, int device)
{
    if (o == Py_None)
        return c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)device).stream();
    want(PyLong_Check(o));
    void* p = PyLong_AsVoidPtr(o);
    if (!p && PyErr_Occurred()) {
        PyErr_Clear();
        throw Refused{};
    }
    return p;
}

template <class F>
PyObject* run(Py_ssize_t given, Py_ssize_t wanted, bool bound, F&& body)
{
    int rc = 0;
    try {
        want(given == wanted && bound);
        rc = body();
    } catch (...) {             // Refused, or an error of torch's on an unusual tensor
        PyErr_Clear();
        Py_RETURN_NONE;
    }
    return PyLong_FromLong(rc);
}

// the C call without the interpreter's lock, as ctypes makes it
template <class F>
int unlocked(F&& call)
{
    PyThreadState* s = PyEval_SaveThread();
    const int rc = call();
    PyEval_RestoreThread(s);
    return rc;
}

PyObject* py_route(PyObject*, PyObject* const* a, Py_ssize_t n)
{
    return run(n, 11, g_route, [&] {
        const at::Tensor &x = tensor(a[0]), &ids = tensor(a[2]);
        want(x.dim() == 2 && ids.dim() == 2);
        const int T = extent(x.size(0)), E = extent(x.size(1)), k = extent(ids.size(1));
        const int dev = device_of(x), dt = element(x);
        const void* px = at_shape(x, dev, {T, E});
        const float* bias =
            a[1] == Py_None ? nullptr : typed<float>(tensor(a[1]), at::kFloat, dev, {E});
        int32_t* pi = typed<int32_t>(ids, at::kInt, dev, {T, k});
        float* pw = typed<float>(tensor(a[3]), at::kFloat, dev, {T, k});
        const int score = as_int(a[4]), G = as_int(a[5]), keep = as_int(a[6]), gs = as_int(a[7]);
        const int renorm = PyObject_IsTrue(a[8]);
        want(renorm >= 0 && PyFloat_Check(a[9]));
        const float scale = (float)PyFloat_AS_DOUBLE(a[9]);
        void* s = stream_of(a[10], dev);
        return unlocked([&] {
            return g_route(px, T, E, dt, bias, score, G, keep, gs, k, renorm, scale, pi, pw, s);
        });
    });
}

PyObject* py_plan(PyObject*, PyObject* const* a, Py_ssize_t n)
{
    return run(n, 6, g_plan, [&] {
        const at::Tensor& ids = tensor(a[0]);
        want(ids.dim() == 2);
        const int T = extent(ids.size(0)), k = extent(ids.size(1)), E = as_int(a[1]);
        const int dev = device_of(ids);
        const int32_t* pi = typed<int32_t>(ids, at::kInt, dev, {T, k});
        int32_t* off = typed<int32_t>(tensor(a[2]), at::kInt, dev, {(int64_t)E + 1});
        int32_t* pos = typed<int32_t>(tensor(a[3]), at::kInt, dev, {T, k});
        const int first = as_int(a[4]);
        void* s = stream_of(a[5], dev);
        return unlocked([&] { return g_plan(pi, T, k, first, E, off, pos, s); });
    });
}

PyObject* py_quant(PyObject*, PyObject* const* a, Py_ssize_t n)
{
    return run(n, 7, g_quant, [&] {
        const at::Tensor &x = tensor(a[0]), &q = tensor(a[1]);
        want(x.dim() == 2 && q.dim() == 2 && is_codes(q));
        const int act = as_int(a[4]);
        const int rows = extent(x.size(0)), out = extent(q.size(0)), H = extent(q.size(1));
        const int dev = device_of(x), dt = element(x);
        const void* px = at_shape(x, dev, {rows, act == AR_ACT_SILU_MUL ? 2 * (int64_t)H : H});
        void* pq = at_shape(q, dev, {out, H});
        float* ps = typed<float>(tensor(a[2]), at::kFloat, dev, {out, (H + kBlock - 1) / kBlock});
        const int32_t *pos = nullptr, *count = nullptr;
        int copies = 1;
        if (a[3] != Py_None) {
            const at::Tensor& p = tensor(a[3]);
            want(p.dim() == 2);
            copies = extent(p.size(1));
            pos = typed<int32_t>(p, at::kInt, dev, {rows, copies});
        }
        if (a[5] != Py_None)
            count = typed<int32_t>(tensor(a[5]), at::kInt, dev, {1});
        void* s = stream_of(a[6], dev);
        return unlocked([&] {
            return g_quant(px, rows, H, dt, act, pos, copies, count, out, pq, ps, s);
        });
    });
}

PyObject* py_matmul(PyObject*, PyObject* const* a, Py_ssize_t n)
{
    return run(n, 6, g_matmul, [&] {
        const at::Tensor &x = tensor(a[0]), &b = tensor(a[2]), &o = tensor(a[4]);
        want(x.dim() == 2 && b.dim() == 2 && is_codes(x) && is_codes(b));
        const int M = extent(x.size(0)), K = extent(x.size(1)), N = extent(b.size(0));
        const int64_t kb = (K + kBlock - 1) / kBlock, nb = (N + kBlock - 1) / kBlock;
        const int dev = device_of(x), dt = element(o);
        const void *px = at_shape(x, dev, {M, K}), *pb = at_shape(b, dev, {N, K});
        const float* sa = typed<float>(tensor(a[1]), at::kFloat, dev, {M, kb});
        const float* sb = typed<float>(tensor(a[3]), at::kFloat, dev, {nb, kb});
        void* po = at_shape(o, dev, {M, N});
        void* s = stream_of(a[5], dev);
        return unlocked([&] { return g_matmul(px, sa, pb, sb, M, N, K, dt, po, s); });
    });
}

PyObject* py_expert_matmul(PyObject*, PyObject* const* a, Py_ssize_t n)
{
    return run(n, 7, g_expert_matmul, [&] {
        const at::Tensor &x = tensor(a[0]), &b = tensor(a[2]), &o = tensor(a[5]);
        want(x.dim() == 2 && b.dim() == 3 && is_codes(x) && is_codes(b));
        const int M = extent(x.size(0)), K = extent(x.size(1));
        const int E = extent(b.size(0)), N = extent(b.size(1));
        const int64_t kb = (K + kBlock - 1) / kBlock, nb = (N + kBlock - 1) / kBlock;
        const int dev = device_of(x), dt = element(o);
        const void *px = at_shape(x, dev, {M, K}), *pb = at_shape(b, dev, {E, N, K});
        const float* sa = typed<float>(tensor(a[1]), at::kFloat, dev, {M, kb});
        const float* sb = typed<float>(tensor(a[3]), at::kFloat, dev, {E, nb, kb});
        const int32_t* off = typed<int32_t>(tensor(a[4]), at::kInt, dev, {(int64_t)E + 1});
        void* po = at_shape(o, dev, {M, N});
        void* s = stream_of(a[6], dev);
        return unlocked([&] {
            return g_expert_matmul(px, sa, pb, sb, off, E, M, N, K, dt, po, s);
        });
    });
}

PyObject* py_combine(PyObject*, PyObject* const* a, Py_ssize_t n)
{
    return run(n, 6, g_combine, [&] {
        const at::Tensor &r = tensor(a[0]), &p = tensor(a[1]), &o = tensor(a[3]);
        want(r.dim() == 2 && p.dim() == 2);
        const int R = extent(r.size(0)), H = extent(r.size(1));
        const int T = extent(p.size(0)), k = extent(p.size(1));
        const int dev = device_of(r), dt = element(r);
        const void* pr = at_shape(r, dev, {R, H});
        const int32_t* pp = typed<int32_t>(p, at::kInt, dev, {T, k});
        const float* pw = typed<float>(tensor(a[2]), at::kFloat, dev, {T, k});
        void* po = typed<void>(o, r.scalar_type(), dev, {T, H});
        const void* add = a[4] == Py_None ? nullptr
                                          : typed<void>(tensor(a[4]), r.scalar_type(), dev, {T, H});
        void* s = stream_of(a[5], dev);
        return unlocked([&] { return g_combine(pr, R, pp, pw, T, k, H, dt, add, po, s); });
    });
}

template <class F>
bool take(PyObject* o, F& to)
{
    to = reinterpret_cast<F>(PyLong_AsVoidPtr(o));
    return to != nullptr;
}

PyObject* py_bind(PyObject*, PyObject* const* a, Py_ssize_t n)
{
    if (n != 6 || !take(a[0], g_route) || !take(a[1], g_plan) || !take(a[2], g_quant) ||
        !take(a[3], g_matmul) || !take(a[4], g_expert_matmul) || !take(a[5], g_combine)) {
        if (!PyErr_Occurred())
            PyErr_SetString(PyExc_ValueError, "bind takes the addresses of the six entry points");
        return nullptr;
    }
    Py_RETURN_NONE;
}

#define ARF_FAST(f) reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(f)), METH_FASTCALL
PyMethodDef g_methods[] = {
    {"bind", ARF_FAST(py_bind), "addresses of the C entry points, in the order below"},
    {"route", ARF_FAST(py_route), "ar_fusion_route"},
    {"expert_plan", ARF_FAST(py_plan), "ar_fusion_expert_plan"},
    {"quant_blocks", ARF_FAST(py_quant), "ar_fusion_quant_blocks"},
    {"matmul_fp8", ARF_FAST(py_matmul), "ar_fusion_matmul_fp8"},
    {"expert_matmul_fp8", ARF_FAST(py_expert_matmul), "ar_fusion_expert_matmul_fp8"},
    {"combine", ARF_FAST(py_combine), "ar_fusion_combine"},
    {nullptr, nullptr, 0, nullptr}};
PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_marshal", nullptr, -1, g_methods,
                        nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__marshal(void) { return PyModule_Create(&g_module); }
