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
decltype(&dg_quant_i8_rowscale) g_quant_i8;
decltype(&dg_gemv_i8_rowscale) g_i8;
decltype(&dg_moe_sort) g_sort;
decltype(&dg_moe_gather) g_gather;
decltype(&dg_moe_combine) g_combine;
decltype(&dg_moe_combine_grad) g_combine_grad;
decltype(&dg_logits_adjust) g_adjust;

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

// Rows [M, n] of any stride, dense and apart.
bool strided_rows(PyObject* o, const char* name, const void** p, int64_t* ld, int64_t* M, int64_t* n)
{
    if (!two_dims(o, name, M, n)) return false;
    const Tensor* t = &THPVariable_Unpack(o);
    const int64_t row = t->stride(0), one = t->stride(1);
    if (!t->is_cuda() || (one != 1 && *n > 1) || (row < *n && *M > 1))
        return refuse(name, "rows must be dense and apart, on a CUDA device");
    *p = t->data_ptr();
    *ld = row > *n ? row : *n;
    return true;
}

// [M, n] logits: bf16 or fp32, rows dense, any row stride.
bool logits_of(PyObject* o, const void** p, int* type, int64_t* ld, int64_t* M, int64_t* n, const char* name = "logits")
{
    const Tensor* t = tensor(o, name);
    if (!t) return false;
    if (t->scalar_type() != ScalarType::BFloat16 && t->scalar_type() != ScalarType::Float)
        return refuse(name, std::string("dtype ") + c10::toString(t->scalar_type()) +
                                    ", expected torch.bfloat16 or torch.float32");
    *type = t->scalar_type() == ScalarType::Float ? DG_LOGITS_F32 : DG_LOGITS_BF16;
    return strided_rows(o, name, p, ld, M, n);
}

// Every tensor given (None: none) is on the current device, whose stream the call takes.
bool all_here(std::initializer_list<PyObject*> tensors)
{
    const int here = c10::cuda::current_device();
    for (PyObject* o : tensors)
        if (o != Py_None && THPVariable_Unpack(o).get_device() != here) {
            PyErr_SetString(PyExc_ValueError, "a tensor is not on the current CUDA device");
            return false;
        }
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

// (x, q, s)
PyObject* quant_i8(PyObject*, PyObject* const* a, Py_ssize_t n)
{
    return guarded([&]() -> PyObject* {
        int64_t M, K;
        void *x, *q, *s;
        if (!count_args(n, 3) || !two_dims(a[0], "x", &M, &K) || !dense(a[0], "x", ScalarType::BFloat16, {M, K}, &x) ||
            !dense(a[1], "q", ScalarType::Char, {M, K}, &q) || !dense(a[2], "s", ScalarType::Float, {M}, &s) ||
            !all_here({a[0], a[1], a[2]}))
            return nullptr;
        return PyLong_FromLong(g_quant_i8(x, static_cast<int8_t*>(q), static_cast<float*>(s), static_cast<int>(M),
                                          static_cast<int>(K), current_stream()));
    });
}

// (x, Wq, sw, y, ws, choice address or None)
PyObject* i8(PyObject*, PyObject* const* a, Py_ssize_t n)
{
    return guarded([&]() -> PyObject* {
        int64_t M, K, N, kw;
        void *x, *w, *sw, *y;
        if (!count_args(n, 6) || !two_dims(a[0], "x", &M, &K) || !two_dims(a[1], "Wq", &N, &kw) ||
            !dense(a[0], "x", ScalarType::BFloat16, {M, K}, &x) || !dense(a[1], "Wq", ScalarType::Char, {N, K}, &w) ||
            !dense(a[2], "sw", ScalarType::Float, {N}, &sw) || !dense(a[3], "y", ScalarType::BFloat16, {M, N}, &y))
            return nullptr;
        const Tensor* ws = tensor(a[4], "ws");
        if (!ws) return nullptr;
        if (ws->scalar_type() != ScalarType::Byte || !ws->is_cuda() || !ws->is_contiguous()) {
            refuse("ws", "tensors must be contiguous CUDA tensors (torch.uint8)");
            return nullptr;
        }
        if (!all_here({a[0], a[1], a[2], a[3], a[4]})) return nullptr;
        const dg_choice* choice = nullptr;
        if (a[5] != Py_None) {
            choice = static_cast<const dg_choice*>(PyLong_AsVoidPtr(a[5]));
            if (PyErr_Occurred()) return nullptr;
        }
        return PyLong_FromLong(g_i8(x, static_cast<const int8_t*>(w), static_cast<const float*>(sw), y, static_cast<int>(M),
                                    static_cast<int>(N), static_cast<int>(K), ws->data_ptr(),
                                    static_cast<size_t>(ws->numel()), current_stream(), choice));
    });
}

// (ids, E, offsets, pos, slots)
PyObject* sort(PyObject*, PyObject* const* a, Py_ssize_t n)
{
    return guarded([&]() -> PyObject* {
        int64_t M, topk;
        long long E;
        void *ids, *offsets, *pos, *slots;
        if (!count_args(n, 5) || !whole(a[1], &E) || !two_dims(a[0], "ids", &M, &topk) ||
            !dense(a[0], "ids", ScalarType::Int, {M, topk}, &ids) || !dense(a[2], "offsets", ScalarType::Int, {E + 1}, &offsets) ||
            !dense(a[3], "pos", ScalarType::Int, {M, topk}, &pos) || !dense(a[4], "slots", ScalarType::Int, {M * topk}, &slots) ||
            !all_here({a[0], a[2], a[3], a[4]}))
            return nullptr;
        return PyLong_FromLong(g_sort(static_cast<const int32_t*>(ids), static_cast<int32_t*>(offsets), static_cast<int32_t*>(pos),
                                      static_cast<int32_t*>(slots), static_cast<int>(M), static_cast<int>(topk),
                                      static_cast<int>(E), current_stream()));
    });
}

// (x, pos, xs)
PyObject* gather(PyObject*, PyObject* const* a, Py_ssize_t n)
{
    return guarded([&]() -> PyObject* {
        int64_t M, K, m, topk, P, k;
        void *x, *pos, *xs;
        if (!count_args(n, 3) || !two_dims(a[0], "x", &M, &K) || !two_dims(a[1], "pos", &m, &topk) || !two_dims(a[2], "xs", &P, &k))
            return nullptr;
        const ScalarType type = THPVariable_Unpack(a[0]).scalar_type();
        if (!dense(a[0], "x", type, {M, K}, &x) || !dense(a[1], "pos", ScalarType::Int, {M, topk}, &pos) ||
            !dense(a[2], "xs", type, {P, K}, &xs) || !all_here({a[0], a[1], a[2]}))
            return nullptr;
        const int64_t bytes = K * static_cast<int64_t>(THPVariable_Unpack(a[0]).element_size());
        return PyLong_FromLong(g_gather(x, static_cast<const int32_t*>(pos), xs, static_cast<int>(M), static_cast<int>(topk),
                                        static_cast<int>(P), bytes, current_stream()));
    });
}

// (z, pos, w, y)
PyObject* combine(PyObject*, PyObject* const* a, Py_ssize_t n)
{
    return guarded([&]() -> PyObject* {
        int64_t M, N, topk, P;
        void *z, *pos, *w, *y;
        if (!count_args(n, 4) || !two_dims(a[0], "z", &P, &N) || !two_dims(a[1], "pos", &M, &topk) ||
            !dense(a[0], "z", ScalarType::BFloat16, {P, N}, &z) || !dense(a[1], "pos", ScalarType::Int, {M, topk}, &pos) ||
            !dense_or_none(a[2], "w", ScalarType::Float, {M, topk}, &w) ||
            !dense(a[3], "y", ScalarType::BFloat16, {M, N}, &y) || !all_here({a[0], a[1], a[2], a[3]}))
            return nullptr;
        return PyLong_FromLong(g_combine(z, static_cast<const int32_t*>(pos), static_cast<const float*>(w), y, static_cast<int>(M),
                                         static_cast<int>(topk), static_cast<int>(P), static_cast<int>(N), current_stream()));
    });
}

// (dy, z, pos, w, dz, dw)
PyObject* combine_grad(PyObject*, PyObject* const* a, Py_ssize_t n)
{
    return guarded([&]() -> PyObject* {
        int64_t M, N, topk, P;
        void *dy, *z, *pos, *w, *dz, *dw;
        if (!count_args(n, 6) || !two_dims(a[1], "z", &P, &N) || !two_dims(a[2], "pos", &M, &topk) ||
            !dense(a[0], "dy", ScalarType::BFloat16, {M, N}, &dy) || !dense(a[1], "z", ScalarType::BFloat16, {P, N}, &z) ||
            !dense(a[2], "pos", ScalarType::Int, {M, topk}, &pos) || !dense(a[3], "w", ScalarType::Float, {M, topk}, &w) ||
            !dense(a[4], "dz", ScalarType::BFloat16, {P, N}, &dz) || !dense(a[5], "dw", ScalarType::Float, {M, topk}, &dw) ||
            !all_here({a[0], a[1], a[2], a[3], a[4], a[5]}))
            return nullptr;
        return PyLong_FromLong(g_combine_grad(dy, z, static_cast<const int32_t*>(pos), static_cast<const float*>(w), dz,
                                              static_cast<float*>(dw), static_cast<int>(M), static_cast<int>(topk),
                                              static_cast<int>(P), static_cast<int>(N), current_stream()));
    });
}

// (logits, out, tokens, lengths, prompt_lengths, repetition, frequency, presence, bias_ids, bias, mask)
PyObject* adjust(PyObject*, PyObject* const* a, Py_ssize_t n)
{
    return guarded([&]() -> PyObject* {
        const void *x, *y, *tok = nullptr, *mask = nullptr;
        int type, otype;
        int64_t ld, ldo, M, V, mo, vo, rows, len = 0, words, nb = 0;
        dg_logits_edits e = {};
        if (!count_args(n, 11) || !logits_of(a[0], &x, &type, &ld, &M, &V) || !logits_of(a[1], &y, &otype, &ldo, &mo, &vo, "out"))
            return nullptr;
        if (otype != type || mo != M || vo != V) {
            refuse("out", "expected the logits' dtype and shape " + shape_text({M, V}));
            return nullptr;
        }
        if (a[2] != Py_None) {
            const Tensor* t = tensor(a[2], "tokens");
            if (!t) return nullptr;
            if (t->scalar_type() != ScalarType::Int) {
                refuse("tokens", "expected torch.int32");
                return nullptr;
            }
            if (!strided_rows(a[2], "tokens", &tok, &e.ld_tokens, &rows, &len)) return nullptr;
            if (rows != M) {
                refuse("tokens", "shape " + shape_text(t->sizes()) + ", expected " + std::to_string(M) + " rows");
                return nullptr;
            }
        } else {
            for (int i = 3; i < 8; ++i)
                if (a[i] != Py_None) {
                    refuse("tokens", "lengths and penalties need them");
                    return nullptr;
                }
        }
        void *lengths, *prompts, *rep, *freq, *pres, *bid = nullptr, *bias = nullptr;
        if (!dense_or_none(a[3], "lengths", ScalarType::Int, {M}, &lengths) ||
            !dense_or_none(a[4], "prompt_lengths", ScalarType::Int, {M}, &prompts) ||
            !dense_or_none(a[5], "repetition", ScalarType::Float, {M}, &rep) ||
            !dense_or_none(a[6], "frequency", ScalarType::Float, {M}, &freq) ||
            !dense_or_none(a[7], "presence", ScalarType::Float, {M}, &pres))
            return nullptr;
        if ((a[8] == Py_None) != (a[9] == Py_None)) {
            refuse("bias", "bias_ids and bias come together");
            return nullptr;
        }
        if (a[8] != Py_None && (!two_dims(a[8], "bias_ids", &rows, &nb) || !dense(a[8], "bias_ids", ScalarType::Int, {M, nb}, &bid) ||
                                !dense(a[9], "bias", ScalarType::Float, {M, nb}, &bias)))
            return nullptr;
        if (a[10] != Py_None) {
            const Tensor* t = tensor(a[10], "mask");
            if (!t) return nullptr;
            if (t->scalar_type() != ScalarType::Int) {
                refuse("mask", "expected torch.int32");
                return nullptr;
            }
            if (!strided_rows(a[10], "mask", &mask, &e.ld_mask, &rows, &words)) return nullptr;
            if (rows != M || words != (V + 31) / 32) {
                refuse("mask", "shape " + shape_text(t->sizes()) + ", expected " + shape_text({M, (V + 31) / 32}));
                return nullptr;
            }
        }
        if (!all_here({a[0], a[1], a[2], a[3], a[4], a[5], a[6], a[7], a[8], a[9], a[10]})) return nullptr;
        if (len > 0) {                                    // (lists of no entries: none)
            e.tokens = static_cast<const int32_t*>(tok);
            e.n_tokens = static_cast<int32_t>(len);
            e.lengths = static_cast<const int32_t*>(lengths);
            e.prompt_lengths = static_cast<const int32_t*>(prompts);
            e.repetition = static_cast<const float*>(rep);
            e.frequency = static_cast<const float*>(freq);
            e.presence = static_cast<const float*>(pres);
        }
        if (nb > 0) {
            e.bias_ids = static_cast<const int32_t*>(bid);
            e.bias = static_cast<const float*>(bias);
            e.n_bias = static_cast<int32_t>(nb);
        }
        e.mask = static_cast<const int32_t*>(mask);
        return PyLong_FromLong(g_adjust(x, type, ld, const_cast<void*>(y), ldo, &e, static_cast<int>(M), static_cast<int>(V),
                                        current_stream()));
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
    g_quant_i8 = reinterpret_cast<decltype(g_quant_i8)>(dlsym(h, "dg_quant_i8_rowscale"));
    g_i8 = reinterpret_cast<decltype(g_i8)>(dlsym(h, "dg_gemv_i8_rowscale"));
    g_sort = reinterpret_cast<decltype(g_sort)>(dlsym(h, "dg_moe_sort"));
    g_gather = reinterpret_cast<decltype(g_gather)>(dlsym(h, "dg_moe_gather"));
    g_combine = reinterpret_cast<decltype(g_combine)>(dlsym(h, "dg_moe_combine"));
    g_combine_grad = reinterpret_cast<decltype(g_combine_grad)>(dlsym(h, "dg_moe_combine_grad"));
    g_adjust = reinterpret_cast<decltype(g_adjust)>(dlsym(h, "dg_logits_adjust"));
    if (!g_quant || !g_dequant || !g_a4w4 || !g_route || !g_logprobs || !g_quant_i8 || !g_i8 || !g_sort || !g_gather ||
        !g_combine || !g_combine_grad || !g_adjust) {
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
                           {"quant_i8", fast(quant_i8), METH_FASTCALL, nullptr},
                           {"i8", fast(i8), METH_FASTCALL, nullptr},
                           {"sort", fast(sort), METH_FASTCALL, nullptr},
                           {"gather", fast(gather), METH_FASTCALL, nullptr},
                           {"combine", fast(combine), METH_FASTCALL, nullptr},
                           {"combine_grad", fast(combine_grad), METH_FASTCALL, nullptr},
                           {"adjust", fast(adjust), METH_FASTCALL, nullptr},
                           {nullptr, nullptr, 0, nullptr}};

PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_marshal", nullptr, -1, g_methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__marshal(void) { return PyModule_Create(&g_module); }
