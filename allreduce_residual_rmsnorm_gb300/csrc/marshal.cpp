// Argument marshalling of the expert-layer and attention-layer calls for Python: the checks of
// binding.py's quick pass and the call of the C entry point in one step (0.4 us
// instead of 3.5 for attribute reads, tuples and ctypes, where the kernels of a
// decode step take 3 to 5; 1 instead of 20 for the attention layer's many operands).
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
decltype(&ar_fusion_rope_append) g_append = nullptr;
decltype(&ar_fusion_decode_attention) g_decode = nullptr;
decltype(&ar_fusion_prompt_attention) g_prompt = nullptr;

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

// ------------------------------------------------- attention layers

// a [rows, heads, dim] tensor with a contiguous last dimension
ar_head_rows head_rows(const at::Tensor& t, at::ScalarType type, int device, int64_t rows,
                       int64_t heads, int64_t dim)
{
    want(t.scalar_type() == type && t.is_cuda() && t.get_device() == device);
    want(t.sizes() == c10::IntArrayRef({rows, heads, dim}));
    want(t.stride(2) == 1);
    return ar_head_rows{t.data_ptr(), t.stride(0), t.stride(1)};
}

at::ScalarType row_type(const at::Tensor& t)
{
    want(t.scalar_type() == at::kBFloat16 || t.scalar_type() == at::kHalf);
    return t.scalar_type();
}

// k_cache, v_cache, page_table, lengths, kv_scale
ar_kv_cache kv_cache(PyObject* const* a, PyObject* scale, at::ScalarType rows, int dev)
{
    const at::Tensor &k = tensor(a[0]), &v = tensor(a[1]), &table = tensor(a[2]);
    want(k.dim() == 4 && table.dim() == 2 && v.sizes() == k.sizes());
    ar_kv_cache c = {};
    for (const at::Tensor* t : {&k, &v}) {
        want(t->is_cuda() && t->get_device() == dev && t->stride(3) == 1);
        want(t->scalar_type() == k.scalar_type());
    }
    if (k.scalar_type() == at::kFloat8_e4m3fn) {
        c.dtype = AR_DT_E4M3;
        if (scale != Py_None)
            c.scale = typed<float>(tensor(scale), at::kFloat, dev, {2});
    } else {
        want(k.scalar_type() == rows && scale == Py_None);
        c.dtype = element(k);
    }
    c.k = k.data_ptr();
    c.v = v.data_ptr();
    c.k_page = k.stride(0), c.k_row = k.stride(1), c.k_head = k.stride(2);
    c.v_page = v.stride(0), c.v_row = v.stride(1), c.v_head = v.stride(2);
    c.pages = extent(k.size(0));
    c.page_size = extent(k.size(1));
    c.heads = extent(k.size(2));
    c.head_dim = extent(k.size(3));
    c.sequences = extent(table.size(0));
    c.max_pages = extent(table.size(1));
    c.page_table = typed<int32_t>(table, at::kInt, dev, {c.sequences, c.max_pages});
    c.lengths = typed<int32_t>(tensor(a[3]), at::kInt, dev, {c.sequences});
    return c;
}

// q, k, v, k_cache, v_cache, page_table, lengths, inv_freq, q_out, starts, positions,
// sections, interleaved, kv_scale, stream
PyObject* py_append(PyObject*, PyObject* const* a, Py_ssize_t n)
{
    return run(n, 15, g_append, [&] {
        const at::Tensor& k = tensor(a[1]);
        want(k.dim() == 3);
        const at::ScalarType type = row_type(k);
        const int dev = device_of(k), T = extent(k.size(0)), dt = element(k);
        const ar_kv_cache c = kv_cache(a + 3, a[13], type, dev);
        const ar_head_rows kr = head_rows(k, type, dev, T, c.heads, c.head_dim),
                           vr = head_rows(tensor(a[2]), type, dev, T, c.heads, c.head_dim);
        ar_head_rows q = {}, q_out = {};
        int heads = 0;
        const bool with_q = a[0] != Py_None;
        if (with_q) {
            const at::Tensor& t = tensor(a[0]);
            want(t.dim() == 3);
            heads = extent(t.size(1));
            q = head_rows(t, type, dev, T, heads, c.head_dim);
            q_out = a[8] == Py_None ? q : head_rows(tensor(a[8]), type, dev, T, heads, c.head_dim);
        } else {
            want(a[8] == Py_None);
        }
        const float* f = nullptr;
        int rot = 0;
        if (a[7] != Py_None) {
            const at::Tensor& t = tensor(a[7]);
            want(t.dim() == 1 && t.size(0) <= INT_MAX / 2);
            rot = 2 * (int)t.size(0);
            f = typed<float>(t, at::kFloat, dev, {rot / 2});
        }
        int sections[AR_MAX_AXES] = {}, axes = 1;
        const bool listed = a[11] != Py_None;
        if (listed) {
            want(PyTuple_Check(a[11]) && PyTuple_GET_SIZE(a[11]) >= 1 &&
                 PyTuple_GET_SIZE(a[11]) <= AR_MAX_AXES);
            axes = (int)PyTuple_GET_SIZE(a[11]);
            for (int i = 0; i < axes; ++i)
                sections[i] = as_int(PyTuple_GET_ITEM(a[11], i));
        }
        const int32_t *starts = nullptr, *positions = nullptr;
        if (a[9] != Py_None)
            starts = typed<int32_t>(tensor(a[9]), at::kInt, dev, {(int64_t)c.sequences + 1});
        if (a[10] != Py_None) {
            const at::Tensor& t = tensor(a[10]);
            want(t.dim() == 2 || axes == 1);
            positions = t.dim() == 2 ? typed<int32_t>(t, at::kInt, dev, {axes, T})
                                     : typed<int32_t>(t, at::kInt, dev, {T});
        }
        const int inter = PyObject_IsTrue(a[12]);
        want(inter >= 0);
        void* s = stream_of(a[14], dev);
        return unlocked([&] {
            return g_append(&c, with_q ? &q : nullptr, with_q ? &q_out : nullptr, &kr, &vr, T, heads, dt,
                            starts, positions, f, rot, listed ? sections : nullptr, axes, inter, s);
        });
    });
}

// q, k_cache, v_cache, page_table, lengths, starts (None: one row a sequence), out, workspace,
// scale, window, sinks, lse, kv_scale, stream
PyObject* py_attention(PyObject*, PyObject* const* a, Py_ssize_t n)
{
    return run(n, 14, g_decode && g_prompt, [&] {
        const at::Tensor& q = tensor(a[0]);
        want(q.dim() == 3);
        const at::ScalarType type = row_type(q);
        const int dev = device_of(q), T = extent(q.size(0)), H = extent(q.size(1)), dt = element(q);
        const ar_kv_cache c = kv_cache(a + 1, a[12], type, dev);
        const ar_head_rows qr = head_rows(q, type, dev, T, H, c.head_dim),
                           out = head_rows(tensor(a[6]), type, dev, T, H, c.head_dim);
        const bool prompt = a[5] != Py_None;
        const int32_t* starts = nullptr;
        if (prompt)
            starts = typed<int32_t>(tensor(a[5]), at::kInt, dev, {(int64_t)c.sequences + 1});
        else
            want(T == c.sequences);
        void* work = nullptr;
        size_t bytes = 0;
        if (a[7] != Py_None) {
            const at::Tensor& t = tensor(a[7]);
            want(t.is_cuda() && t.get_device() == dev && t.is_contiguous());
            work = t.data_ptr();
            bytes = t.nbytes();
        }
        want(PyFloat_Check(a[8]));
        const float scale = (float)PyFloat_AS_DOUBLE(a[8]);
        const int window = as_int(a[9]), sinks = as_int(a[10]);
        float* lse = nullptr;
        if (a[11] != Py_None)
            lse = typed<float>(tensor(a[11]), at::kFloat, dev, {T, H});
        void* s = stream_of(a[13], dev);
        return unlocked([&] {
            return prompt ? g_prompt(&c, &qr, &out, lse, starts, T, H, dt, scale, window, sinks, work,
                                     bytes, s)
                          : g_decode(&c, &qr, &out, lse, H, dt, scale, window, sinks, work, bytes, s);
        });
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
    if (n != 9 || !take(a[0], g_route) || !take(a[1], g_plan) || !take(a[2], g_quant) ||
        !take(a[3], g_matmul) || !take(a[4], g_expert_matmul) || !take(a[5], g_combine) ||
        !take(a[6], g_append) || !take(a[7], g_decode) || !take(a[8], g_prompt)) {
        if (!PyErr_Occurred())
            PyErr_SetString(PyExc_ValueError, "bind takes the addresses of the nine entry points");
        return nullptr;
    }
    Py_RETURN_NONE;
}

#define ARF_FAST(f) reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(f)), METH_FASTCALL
PyMethodDef g_methods[] = {
    {"bind", ARF_FAST(py_bind), "addresses of the C entry points: the expert layer's six, then the attention layer's"},
    {"route", ARF_FAST(py_route), "ar_fusion_route"},
    {"expert_plan", ARF_FAST(py_plan), "ar_fusion_expert_plan"},
    {"quant_blocks", ARF_FAST(py_quant), "ar_fusion_quant_blocks"},
    {"matmul_fp8", ARF_FAST(py_matmul), "ar_fusion_matmul_fp8"},
    {"expert_matmul_fp8", ARF_FAST(py_expert_matmul), "ar_fusion_expert_matmul_fp8"},
    {"combine", ARF_FAST(py_combine), "ar_fusion_combine"},
    {"rope_append", ARF_FAST(py_append), "ar_fusion_rope_append"},
    {"attention", ARF_FAST(py_attention),
     "ar_fusion_decode_attention, or with starts ar_fusion_prompt_attention"},
    {nullptr, nullptr, 0, nullptr}};
PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_marshal", nullptr, -1, g_methods,
                        nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__marshal(void) { return PyModule_Create(&g_module); }
