// binding.cpp -- Python binding of the packed operators (argument marshalling
// only; the functions have the names and argument order of the C entry points
// without their prefix).
//
// A serving step calls these operators in every layer on a few tensors each.
// Described to the library from Python (attribute by attribute), the nine
// tensors of an append took 6 of the 11 us of a call; here they take well
// under one.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <climits>
#include <cstring>

#include "../../include/mla_decode.h"

namespace {

PyObject* g_error = nullptr;  // the package's MlaError(status, message)

void raise_status(int status, const char* message) {
    if (!g_error) {
        PyErr_SetString(PyExc_RuntimeError, message);
        return;
    }
    PyObject* e = PyObject_CallFunction(g_error, "is", status, message);
    if (e) {
        PyErr_SetObject(g_error, e);
        Py_DECREF(e);
    }
}

// The arguments of one call, taken in order; after a bad one `ok` is false, a
// Python exception is set and the rest is skipped.  The current device is asked
// for with the first tensor: what is no tensor is refused without a GPU too.
struct Args {
    PyObject* const* at;
    Py_ssize_t left;
    bool ok = true;
    int device = -1;
    mla_tensor_t desc[12];
    int used = 0;

    PyObject* next() {
        if (!ok) return nullptr;
        if (left == 0) {
            PyErr_SetString(PyExc_TypeError, "too few arguments");
            ok = false;
            return nullptr;
        }
        --left;
        return *at++;
    }
    const at::Tensor* tensor_of(PyObject* o) {
        if (!o) return nullptr;
        if (!THPVariable_Check(o)) {
            PyErr_Format(PyExc_TypeError, "a tensor expected, not %s", Py_TYPE(o)->tp_name);
            ok = false;
            return nullptr;
        }
        const at::Tensor& t = THPVariable_Unpack(o);
        if (device < 0 && t.is_cuda()) device = c10::cuda::current_device();
        if (!t.is_cuda() || t.get_device() != device) {
            raise_status(MLA_ERR_INVALID_ARG, "a tensor is not on the current CUDA device");
            ok = false;
            return nullptr;
        }
        return &t;
    }
    // NULL for None
    const mla_tensor_t* tensor() {
        PyObject* o = next();
        if (!o || o == Py_None) return nullptr;
        const at::Tensor* t = tensor_of(o);
        if (!t) return nullptr;
        if (t->dim() > 5) {
            PyErr_SetString(PyExc_ValueError, "at most 5 dims");
            ok = false;
            return nullptr;
        }
        mla_tensor_t& d = desc[used++];
        std::memset(&d, 0, sizeof d);
        d.data = t->data_ptr();
        d.ndim = static_cast<int32_t>(t->dim());
        for (int i = 0; i < d.ndim; ++i) {
            d.shape[i] = t->size(i);
            d.stride[i] = t->stride(i);
        }
        switch (t->scalar_type()) {
            case at::kBFloat16: d.dtype = MLA_DTYPE_BF16; break;
            case at::kFloat: d.dtype = MLA_DTYPE_F32; break;
            case at::kByte:
            case at::kFloat8_e4m3fn: d.dtype = MLA_DTYPE_E4M3FN; break;
            case at::kInt: d.dtype = MLA_DTYPE_I32; break;
            default: d.dtype = 0;
        }
        return &d;
    }
    // One fp32 on the device.
    const float* scale() {
        const at::Tensor* t = tensor_of(next());
        if (!t) return nullptr;
        if (t->scalar_type() != at::kFloat || t->numel() < 1) {
            raise_status(MLA_ERR_INVALID_ARG, "kv_scale: one float32 expected");
            ok = false;
            return nullptr;
        }
        return static_cast<const float*>(t->data_ptr());
    }
    float real() {
        PyObject* o = next();
        if (!o) return 0.f;
        const double v = PyFloat_AsDouble(o);
        if (v == -1.0 && PyErr_Occurred()) ok = false;
        return static_cast<float>(v);
    }
    int32_t whole() {
        PyObject* o = next();
        if (!o) return 0;
        const long v = PyLong_AsLong(o);
        if (v == -1 && PyErr_Occurred()) {
            ok = false;
        } else if (v < INT32_MIN || v > INT32_MAX) {
            PyErr_SetString(PyExc_OverflowError, "an argument does not fit 32 bits");
            ok = false;
        }
        return static_cast<int32_t>(v);
    }
    // None: the current stream; a stream object, or its raw handle.
    void* stream() {
        PyObject* o = next();
        if (!o) return nullptr;
        if (o == Py_None)
            return c10::cuda::getCurrentCUDAStream().stream();
        PyObject* handle = PyLong_Check(o) ? Py_NewRef(o) : PyObject_GetAttrString(o, "cuda_stream");
        if (!handle) {
            ok = false;
            return nullptr;
        }
        void* p = PyLong_AsVoidPtr(handle);
        Py_DECREF(handle);
        if (!p && PyErr_Occurred()) ok = false;
        return p;
    }
    bool done() {
        if (ok && left > 0) {
            PyErr_SetString(PyExc_TypeError, "too many arguments");
            ok = false;
        }
        return ok;
    }
};

PyObject* result(mla_status_t st) {
    if (st == MLA_OK) Py_RETURN_NONE;
    raise_status(st, mla_last_error());
    return nullptr;
}

// Runs `body` on the arguments; no C++ exception leaves it.
template <typename F>
PyObject* guarded(PyObject* const* args, Py_ssize_t n, F body) {
    try {
        Args a{args, n};
        return body(a);
    } catch (const std::exception& e) {
        if (!PyErr_Occurred()) PyErr_SetString(PyExc_RuntimeError, e.what());
        return nullptr;
    }
}

PyObject* append_rotated(PyObject*, PyObject* const* args, Py_ssize_t n) {
    return guarded(args, n, [](Args& a) -> PyObject* {
        const mla_tensor_t *latent = a.tensor(), *weight = a.tensor();
        const float eps = a.real();
        const mla_tensor_t* cos_sin = a.tensor();
        const int32_t interleaved = a.whole();
        const mla_tensor_t* cu = a.tensor();
        const float* scale = a.scale();
        const mla_tensor_t *table = a.tensor(), *start = a.tensor(), *cache = a.tensor(), *out = a.tensor();
        void* stream = a.stream();
        if (!a.done()) return nullptr;
        mla_status_t st;
        Py_BEGIN_ALLOW_THREADS;
        st = mla_append_rotated(latent, weight, eps, cos_sin, interleaved, cu, scale, table, start, cache, out, stream);
        Py_END_ALLOW_THREADS;
        return result(st);
    });
}

PyObject* rotate_query(PyObject*, PyObject* const* args, Py_ssize_t n) {
    return guarded(args, n, [](Args& a) -> PyObject* {
        const mla_tensor_t *q = a.tensor(), *weight = a.tensor();
        const float eps = a.real();
        const mla_tensor_t* cos_sin = a.tensor();
        const int32_t interleaved = a.whole();
        const mla_tensor_t *cu = a.tensor(), *start = a.tensor(), *nope = a.tensor(), *pe = a.tensor();
        void* stream = a.stream();
        if (!a.done()) return nullptr;
        mla_status_t st;
        Py_BEGIN_ALLOW_THREADS;
        st = mla_rotate_query(q, weight, eps, cos_sin, interleaved, cu, start, nope, pe, stream);
        Py_END_ALLOW_THREADS;
        return result(st);
    });
}

PyObject* gather_latent(PyObject*, PyObject* const* args, Py_ssize_t n) {
    return guarded(args, n, [](Args& a) -> PyObject* {
        const mla_tensor_t* cache = a.tensor();
        const float* scale = a.scale();
        const mla_tensor_t *table = a.tensor(), *cu = a.tensor(), *start = a.tensor();
        const mla_tensor_t *latent = a.tensor(), *pe = a.tensor();
        void* stream = a.stream();
        if (!a.done()) return nullptr;
        mla_status_t st;
        Py_BEGIN_ALLOW_THREADS;
        st = mla_gather_latent(cache, scale, table, cu, start, latent, pe, stream);
        Py_END_ALLOW_THREADS;
        return result(st);
    });
}

PyObject* prefill_ragged(PyObject*, PyObject* const* args, Py_ssize_t n) {
    return guarded(args, n, [](Args& a) -> PyObject* {
        const mla_tensor_t *q = a.tensor(), *kn = a.tensor(), *kp = a.tensor(), *v = a.tensor();
        const mla_tensor_t *cu_q = a.tensor(), *cu_k = a.tensor();
        const int32_t max_q = a.whole(), max_k = a.whole(), splits = a.whole();
        const float scale = a.real(), cap = a.real();
        const int32_t causal = a.whole(), window = a.whole();
        const mla_tensor_t *prefix = a.tensor(), *out = a.tensor(), *lse = a.tensor();
        void* stream = a.stream();
        if (!a.done()) return nullptr;
        mla_status_t st;
        Py_BEGIN_ALLOW_THREADS;
        st = mla_prefill_ragged(q, kn, kp, v, cu_q, cu_k, max_q, max_k, splits, scale, cap, causal, window, prefix, out,
                                lse, stream);
        Py_END_ALLOW_THREADS;
        return result(st);
    });
}

PyObject* set_error(PyObject*, PyObject* cls) {
    Py_INCREF(cls);
    Py_XSETREF(g_error, cls);
    Py_RETURN_NONE;
}

template <typename F>
PyCFunction as_function(F* f) {
    return reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f));
}

PyMethodDef kMethods[] = {
    {"append_rotated", as_function(append_rotated), METH_FASTCALL, nullptr},
    {"rotate_query", as_function(rotate_query), METH_FASTCALL, nullptr},
    {"gather_latent", as_function(gather_latent), METH_FASTCALL, nullptr},
    {"prefill_ragged", as_function(prefill_ragged), METH_FASTCALL, nullptr},
    {"set_error", set_error, METH_O, "the class that failing calls raise: MlaError(status, message)"},
    {nullptr, nullptr, 0, nullptr},
};
PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "_packed", nullptr, -1, kMethods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__packed() { return PyModule_Create(&kModule); }
