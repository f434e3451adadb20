// _marshal.cpp -- argument checks and calls of the smallest entry points for Python.
//
// The same work as the ctypes binding -- dtype, shape, device and layout of every tensor, the
// current stream, one C call -- without a Python object for each step: on GB300's host a routing
// call of 3 us on the device took 5.3 us to marshal through ctypes.  Every function takes its
// arguments by position (the Python wrappers hold names and defaults), raises ValueError for a
// tensor that does not fit and returns the dg_status of the call.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <c10/cuda/CUDAStream.h>
#include <dlfcn.h>
#include <torch/csrc/autograd/python_variable.h>

#include <initializer_list>
#include <string>

#include "dg.h"

namespace {

using at::ScalarType;
using at::Tensor;

decltype(&dg_quant_fp4_blockscale) g_quant;
decltype(&dg_dequant_fp4_blockscale) g_dequant;
decltype(&dg_gemv_a4w4_blockscale) g_a4w4;
decltype(&dg_moe_route) g_route;
decltype(&dg_logprobs) g_logprobs;

bool refuse(const char* name, const std::string& what)
{
    PyErr_SetString(PyExc_ValueError, (std::string(name) + ": " + what).c_str());
    return false;
}

std::string shape_text(at::IntArrayRef s)
{
    std::string t = "(";
    for (size_t i = 0; i < s.size(); ++i) t += (i ? ", " : "") + std::to_string(s[i]);
    return t + (s.size() == 1 ? ",)" : ")");
}

const Tensor* tensor(PyObject* o, const char* name)
{
    if (!THPVariable_Check(o)) {
        refuse(name, "expected a tensor");
        return nullptr;
    }
    return &THPVariable_Unpack(o);
}

// Address of a dense CUDA tensor of this dtype and shape.
bool dense(PyObject* o, const char* name, ScalarType type, std::initializer_list<int64_t> shape, void** p)
{
    const Tensor* t = tensor(o, name);
    if (!t) return false;
    const at::IntArrayRef want(shape.begin(), shape.size());
    if (t->scalar_type() != type)
        return refuse(name, std::string("dtype ") + c10::toString(t->scalar_type()) + ", expected " + c10::toString(type));
    if (t->sizes() != want)
        return refuse(name, "shape " + shape_text(t->sizes()) + ", expected " + shape_text(want));
    if (!t->is_cuda() || !t->is_contiguous()) return refuse(name, "tensors must be contiguous CUDA tensors");
    *p = t->data_ptr();
    return true;
}

bool dense_or_none(PyObject* o, const char* name, ScalarType type, std::initializer_list<int64_t> shape, void** p)
{
    *p = nullptr;
    return o == Py_None || dense(o, name, type, shape, p);
}

// Address of one fp32 on the device (None: none).
bool scalar(PyObject* o, const char* name, const float** p)
{
    *p = nullptr;
    if (o == Py_None) return true;
    const Tensor* t = tensor(o, name);
    if (!t) return false;
    if (t->scalar_type() != ScalarType::Float || t->numel() != 1) return refuse(name, "expected one torch.float32 value");
    if (!t->is_cuda()) return refuse(name, "tensors must be contiguous CUDA tensors");
    *p = static_cast<const float*>(t->data_ptr());
    return true;
}

bool two_dims(PyObject* o, const char* name, int64_t* rows, int64_t* cols)
{
    const Tensor* t = tensor(o, name);
    if (!t) return false;
    if (t->dim() != 2) return refuse(name, "shape " + shape_text(t->sizes()) + ", expected two dimensions");
    *rows = t->size(0);
    *cols = t->size(1);
    if (*rows > INT32_MAX || *cols > INT32_MAX) return refuse(name, "a dimension past 2^31 - 1");
    return true;
}

// [M, n] logits: bf16 or fp32, rows dense, any row stride.
bool logits_of(PyObject* o, const void** p, int* type, int64_t* ld, int64_t* M, int64_t* n)
{
    const Tensor* t = tensor(o, "logits");
    if (!t) return false;
    if (t->scalar_type() != ScalarType::BFloat16 && t->scalar_type() != ScalarType::Float)
        return refuse("logits", std::string("dtype ") + c10::toString(t->scalar_type()) +
                                    ", expected torch.bfloat16 or torch.float32");
    if (!two_dims(o, "logits", M, n)) return false;
    const int64_t row = t->stride(0), one = t->stride(1);
    if (!t->is_cuda() || (one != 1 && *n > 1) || (row < *n && *M > 1))
        return refuse("logits", "rows must be dense and apart, on a CUDA device");
    *p = t->data_ptr();
    *type = t->scalar_type() == ScalarType::Float ? DG_LOGITS_F32 : DG_LOGITS_BF16;
    *ld = row > *n ? row : *n;
    return true;
}

bool whole(PyObject* o, long long* v)
{
    *v = PyLong_AsLongLong(o);
    if (*v == -1 && PyErr_Occurred()) return false;
    if (*v < INT32_MIN || *v > INT32_MAX) {
        PyErr_SetString(PyExc_ValueError, "a whole number past 32 bits");
        return false;
    }
    return true;
}

// The current stream of the current device.
dg_stream_t current_stream() { return reinterpret_cast<dg_stream_t>(c10::cuda::getCurrentCUDAStream().stream()); }

bool count_args(Py_ssize_t got, Py_ssize_t want)
{
    if (got == want) return true;
    PyErr_Format(PyExc_TypeError, "%zd arguments, expected %zd", got, want);
    return false;
}

bool format_of(PyObject* o, long long* fmt)
{
    if (!whole(o, fmt)) return false;
    if (*fmt != DG_FP4_MX && *fmt != DG_FP4_NV) return refuse("fmt", "expected DG_FP4_MX or DG_FP4_NV");
    return true;
}

int64_t row_tiles(int64_t rows) { return (rows + 127) / 128; }
int64_t k_tiles(int64_t K, long long fmt) { return (K / (fmt == DG_FP4_NV ? 16 : 32) + 3) / 4; }

// No C++ exception leaves a call (a stream lookup without a usable device throws).
template <class F>
PyObject* guarded(F&& f)
{
    try {
        return f();
    } catch (const std::exception& e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
        return nullptr;
    }
}

// (x, fmt, g, q, s)
PyObject* quant(PyObject*, PyObject* const* a, Py_ssize_t n)
{
    return guarded([&]() -> PyObject* {
        int64_t M, K;
        long long fmt;
        void *x, *q, *s;
        const float* g;
        if (!count_args(n, 5) || !format_of(a[1], &fmt) || !two_dims(a[0], "x", &M, &K) ||
            !dense(a[0], "x", ScalarType::BFloat16, {M, K}, &x) || !dense(a[3], "q", ScalarType::Byte, {M, K / 2}, &q) ||
            !dense(a[4], "s", ScalarType::Byte, {row_tiles(M), k_tiles(K, fmt), 512}, &s) || !scalar(a[2], "g", &g))
            return nullptr;
        return PyLong_FromLong(g_quant(x, q, s, g, static_cast<int>(M), static_cast<int>(K), static_cast<int>(fmt), current_stream()));
    });
}

// (q, s, fmt, g, y)
PyObject* dequant(PyObject*, PyObject* const* a, Py_ssize_t n)
{
    return guarded([&]() -> PyObject* {
        int64_t M, half;
        long long fmt;
        void *q, *s, *y;
        const float* g;
        if (!count_args(n, 5) || !format_of(a[2], &fmt) || !two_dims(a[0], "q", &M, &half)) return nullptr;
        const int64_t K = 2 * half;
        if (K > INT32_MAX) {
            refuse("q", "a dimension past 2^31 - 1");
            return nullptr;
        }
        if (!dense(a[0], "q", ScalarType::Byte, {M, half}, &q) ||
            !dense(a[1], "s", ScalarType::Byte, {row_tiles(M), k_tiles(K, fmt), 512}, &s) || !scalar(a[3], "g", &g) ||
            !dense(a[4], "y", ScalarType::BFloat16, {M, K}, &y))
            return nullptr;
        return PyLong_FromLong(g_dequant(q, s, g, y, static_cast<int>(M), static_cast<int>(K), static_cast<int>(fmt), current_stream()));
    });
}

// (x, Wq, sw, fmt, gx, gw, y, ws, choice address or None)
PyObject* a4w4(PyObject*, PyObject* const* a, Py_ssize_t n)
{
    return guarded([&]() -> PyObject* {
        int64_t M, K, N, half;
        long long fmt;
        void *x, *w, *sw, *y;
        const float *gx, *gw;
        if (!count_args(n, 9) || !format_of(a[3], &fmt) || !two_dims(a[0], "x", &M, &K) ||
            !two_dims(a[1], "Wq", &N, &half) || !dense(a[0], "x", ScalarType::BFloat16, {M, K}, &x) ||
            !dense(a[1], "Wq", ScalarType::Byte, {N, K / 2}, &w) ||
            !dense(a[2], "sw", ScalarType::Byte, {row_tiles(N), k_tiles(K, fmt), 512}, &sw) ||
            !scalar(a[4], "gx", &gx) || !scalar(a[5], "gw", &gw) || !dense(a[6], "y", ScalarType::BFloat16, {M, N}, &y))
            return nullptr;
        const Tensor* ws = tensor(a[7], "ws");
        if (!ws) return nullptr;
        if (ws->scalar_type() != ScalarType::Byte || !ws->is_cuda() || !ws->is_contiguous()) {
            refuse("ws", "tensors must be contiguous CUDA tensors (torch.uint8)");
            return nullptr;
        }
        const dg_choice* choice = nullptr;
        if (a[8] != Py_None) {
            choice = static_cast<const dg_choice*>(PyLong_AsVoidPtr(a[8]));
            if (PyErr_Occurred()) return nullptr;
        }
        return PyLong_FromLong(g_a4w4(x, w, sw, gx, gw, y, static_cast<int>(M), static_cast<int>(N), static_cast<int>(K),
                                      static_cast<int>(fmt), ws->data_ptr(), static_cast<size_t>(ws->numel()), current_stream(), choice));
    });
}

// (logits, topk, score, bias, n_group, topk_group, group_top, renorm, scale, ids, w)
PyObject* route(PyObject*, PyObject* const* a, Py_ssize_t n)
{
    return guarded([&]() -> PyObject* {
        const void* x;
        int type;
        int64_t ld, M, E;
        long long v[6];
        void *bias, *ids, *w;
        if (!count_args(n, 11) || !logits_of(a[0], &x, &type, &ld, &M, &E) || !whole(a[1], &v[0]) || !whole(a[2], &v[1]) ||
            !whole(a[4], &v[2]) || !whole(a[5], &v[3]) || !whole(a[6], &v[4]))
            return nullptr;
        const int renorm = PyObject_IsTrue(a[7]);
        const double scale = PyFloat_AsDouble(a[8]);
        if (renorm < 0 || PyErr_Occurred()) return nullptr;
        if (!dense_or_none(a[3], "bias", ScalarType::Float, {E}, &bias) ||
            !dense(a[9], "ids", ScalarType::Int, {M, v[0]}, &ids) || !dense(a[10], "w", ScalarType::Float, {M, v[0]}, &w))
            return nullptr;
        const dg_route_params p = {static_cast<int32_t>(v[0]), static_cast<int32_t>(v[2]), static_cast<int32_t>(v[3]),
                                   static_cast<int32_t>(v[4]), static_cast<int32_t>(v[1]), renorm,
                                   static_cast<float>(scale)};
        return PyLong_FromLong(g_route(x, type, ld, static_cast<const float*>(bias), &p, static_cast<int32_t*>(ids),
                                       static_cast<float*>(w), static_cast<int>(M), static_cast<int>(E), current_stream()));
    });
}

// (logits, tokens, scale, n_top, logprob, rank, entropy, top_ids, top_logprobs)
PyObject* logprobs(PyObject*, PyObject* const* a, Py_ssize_t n)
{
    return guarded([&]() -> PyObject* {
        const void* x;
        int type;
        int64_t ld, M, V;
        long long top;
        void *tok, *lp, *rank, *ent, *ti, *tl;
        if (!count_args(n, 9) || !logits_of(a[0], &x, &type, &ld, &M, &V) || !whole(a[3], &top)) return nullptr;
        const double scale = PyFloat_AsDouble(a[2]);
        if (PyErr_Occurred()) return nullptr;
        if (!dense_or_none(a[1], "tokens", ScalarType::Long, {M}, &tok) ||
            !dense_or_none(a[4], "logprob", ScalarType::Float, {M}, &lp) ||
            !dense_or_none(a[5], "rank", ScalarType::Int, {M}, &rank) ||
            !dense_or_none(a[6], "entropy", ScalarType::Float, {M}, &ent) ||
            !dense_or_none(a[7], "top_ids", ScalarType::Int, {M, top}, &ti) ||
            !dense_or_none(a[8], "top_logprobs", ScalarType::Float, {M, top}, &tl))
            return nullptr;
        return PyLong_FromLong(g_logprobs(x, type, ld, static_cast<const int64_t*>(tok), static_cast<float>(scale),
                                          static_cast<int>(top), static_cast<float*>(lp), static_cast<int32_t*>(rank),
                                          static_cast<float*>(ent), static_cast<int32_t*>(ti), static_cast<float*>(tl),
                                          static_cast<int>(M), static_cast<int>(V), current_stream()));
    });
}

// (path of libdecodegemm.so): looks the entry points up.
PyObject* bind(PyObject*, PyObject* path)
{
    const char* p = PyUnicode_AsUTF8(path);
    if (!p) return nullptr;
    void* h = dlopen(p, RTLD_NOW);
    if (!h) {
        PyErr_SetString(PyExc_ImportError, dlerror());
        return nullptr;
    }
    g_quant = reinterpret_cast<decltype(g_quant)>(dlsym(h, "dg_quant_fp4_blockscale"));
    g_dequant = reinterpret_cast<decltype(g_dequant)>(dlsym(h, "dg_dequant_fp4_blockscale"));
    g_a4w4 = reinterpret_cast<decltype(g_a4w4)>(dlsym(h, "dg_gemv_a4w4_blockscale"));
    g_route = reinterpret_cast<decltype(g_route)>(dlsym(h, "dg_moe_route"));
    g_logprobs = reinterpret_cast<decltype(g_logprobs)>(dlsym(h, "dg_logprobs"));
    if (!g_quant || !g_dequant || !g_a4w4 || !g_route || !g_logprobs) {
        PyErr_SetString(PyExc_ImportError, "libdecodegemm.so lacks an entry point");
        return nullptr;
    }
    Py_RETURN_NONE;
}

PyCFunction fast(PyObject* (*f)(PyObject*, PyObject* const*, Py_ssize_t))
{
    return reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f));
}

PyMethodDef g_methods[] = {{"bind", bind, METH_O, nullptr},
                           {"quant", fast(quant), METH_FASTCALL, nullptr},
                           {"dequant", fast(dequant), METH_FASTCALL, nullptr},
                           {"a4w4", fast(a4w4), METH_FASTCALL, nullptr},
                           {"route", fast(route), METH_FASTCALL, nullptr},
                           {"logprobs", fast(logprobs), METH_FASTCALL, nullptr},
                           {nullptr, nullptr, 0, nullptr}};

PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_marshal", nullptr, -1, g_methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__marshal(void) { return PyModule_Create(&g_module); }
