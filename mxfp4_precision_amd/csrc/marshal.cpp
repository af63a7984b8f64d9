// Python extension module: the arguments of the calls that run many times a
// step (grouped quantization and products) from Python objects to C.
//
// Of a call's host time through ctypes, 2.6 us went into 16 converted
// arguments and the checks of 8 tensors in Python, next to 3 us for the launch
// itself; a layer of experts on few rows makes six such calls in less GPU
// time than that.  Here the same conversions and checks take 0.4 us.  Only
// the usual argument is handled here (None, an int, a tensor that passes): any
// other one goes to the Python function of the ctypes binding, which converts
// it or raises its error.
//
// The module links nothing: bind() takes the addresses of the loaded
// library's entry points.

#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <cstdint>

#include "mxfp4.h"

namespace {

decltype(&mx_quantize_grouped) g_quantize_grouped;
decltype(&mx_gemm_a4w4_grouped) g_gemm_grouped;
decltype(&mx_gemm_a4w4_grouped_wgrad) g_gemm_grouped_wgrad;
PyObject *g_dptr, *g_i32ptr, *g_stream;   // the Python binding's converters
PyObject *g_quant_opts;                   // ... and its options structure
PyObject *g_int32;                        // torch.int32, once torch is imported
PyObject *s_is_cuda, *s_data_ptr, *s_dtype, *s_is_contiguous, *s_numel, *s_torch;

// Arguments of one call in order; after a failed conversion (`bad`, Python
// error set) the others return 0.
struct Args {
    PyObject *const *v;
    Py_ssize_t n, at = 0;
    bool bad = false;
    Py_buffer views[2];
    int held = 0;

    Args(PyObject *const *v_, Py_ssize_t n_) : v(v_), n(n_) {}
    ~Args() {
        while (held) PyBuffer_Release(&views[--held]);
    }
    PyObject *next() { return v[at++]; }

    uintptr_t address(PyObject *result) {   // takes the reference
        if (!result) {
            bad = true;
            return 0;
        }
        uintptr_t p = 0;
        if (result != Py_None) {
            p = (uintptr_t)PyLong_AsUnsignedLongLongMask(result);
            if (PyErr_Occurred()) bad = true;
        }
        Py_DECREF(result);
        return p;
    }
    static bool is_true(PyObject *result) {   // takes the reference; errors count as false
        const bool t = result == Py_True;
        Py_XDECREF(result);
        PyErr_Clear();
        return t;
    }
    uintptr_t tensor(PyObject *o) { return address(PyObject_CallMethodNoArgs(o, s_data_ptr)); }

    void *ptr() {
        PyObject *o = next();
        if (bad || o == Py_None) return nullptr;
        if (!PyLong_CheckExact(o) && is_true(PyObject_GetAttr(o, s_is_cuda))) return (void *)tensor(o);
        return (void *)address(PyObject_CallOneArg(g_dptr, o));
    }
    // count consecutive 32-bit integers
    const int32_t *i32ptr(int64_t count) {
        PyObject *o = next();
        if (bad || o == Py_None) return nullptr;
        if (!PyLong_CheckExact(o) && usual_i32(o, count)) return (const int32_t *)tensor(o);
        PyObject *r = nullptr, *c = PyLong_FromLongLong(count);
        if (c) r = PyObject_CallFunctionObjArgs(g_i32ptr, o, c, nullptr);
        Py_XDECREF(c);
        return (const int32_t *)address(r);
    }
    static bool usual_i32(PyObject *o, int64_t count) {
        if (!g_int32) {
            PyObject *torch = PyImport_GetModule(s_torch);
            if (torch) g_int32 = PyObject_GetAttrString(torch, "int32");
            Py_XDECREF(torch);
            PyErr_Clear();
            if (!g_int32) return false;
        }
        PyObject *t = PyObject_GetAttr(o, s_dtype);
        const bool same = t == g_int32;
        Py_XDECREF(t);
        PyErr_Clear();
        if (!same || !is_true(PyObject_GetAttr(o, s_is_cuda)) ||
            !is_true(PyObject_CallMethodNoArgs(o, s_is_contiguous)))
            return false;
        PyObject *c = PyObject_CallMethodNoArgs(o, s_numel);
        const long long have = c ? PyLong_AsLongLong(c) : -1;
        Py_XDECREF(c);
        PyErr_Clear();
        return have >= count;
    }
    int64_t i64(Py_ssize_t which) {
        if (bad) return 0;
        const long long r = PyLong_AsLongLong(v[which]);
        if (r == -1 && PyErr_Occurred()) bad = true;
        return r;
    }
    int64_t i64() { return i64(at++); }
    int i32() {
        const int64_t r = i64();
        if (!bad && r != (int)r) {
            PyErr_Format(PyExc_OverflowError, "%lld does not fit a C int", (long long)r);
            bad = true;
        }
        return (int)r;
    }
    // an mx_quant_opts of the Python binding, or None
    const mx_quant_opts *options() {
        PyObject *o = next();
        if (bad || o == Py_None) return nullptr;
        const int is = PyObject_IsInstance(o, g_quant_opts);
        if (is == 0) PyErr_Format(PyExc_TypeError, "mx_quant_opts or None is required, got %R", (PyObject *)Py_TYPE(o));
        if (is <= 0 || PyObject_GetBuffer(o, &views[held], PyBUF_SIMPLE) != 0) {
            bad = true;
            return nullptr;
        }
        return (const mx_quant_opts *)views[held++].buf;
    }
    // a handle; the Python converter takes the rest (None, streams)
    hipStream_t stream() {
        PyObject *o = next();
        if (bad) return nullptr;
        return (hipStream_t)address(PyLong_CheckExact(o) ? Py_NewRef(o) : PyObject_CallOneArg(g_stream, o));
    }
};

bool count_is(Py_ssize_t n, Py_ssize_t want) {
    if (n == want) return true;
    PyErr_Format(PyExc_TypeError, "%zd arguments expected, got %zd", want, n);
    return false;
}

template <typename F>
PyObject *run(const Args &a, F call) {
    if (a.bad) return nullptr;
    mx_status st;
    Py_BEGIN_ALLOW_THREADS
    st = call();
    Py_END_ALLOW_THREADS
    return PyLong_FromLong(st);
}

// (x, x_rows, N, ldx, row_index, M, group_ends, groups, row_opts, col_opts, layout, q_row, s_row, q_col, s_col, stream)
PyObject *quantize_grouped(PyObject *, PyObject *const *v, Py_ssize_t n) {
    if (!count_is(n, 16)) return nullptr;
    Args a(v, n);
    const void *x = a.ptr();
    const int64_t x_rows = a.i64(), N = a.i64(), ldx = a.i64();
    const int64_t M = a.i64(5);
    const int32_t *index = a.i32ptr(M);
    a.at = 6;
    const int64_t groups = a.i64(7);
    const int32_t *ends = a.i32ptr(groups);
    const int g = a.i32();
    const mx_quant_opts *ro = a.options(), *co = a.options();
    const int layout = a.i32();
    void *q = a.ptr(), *s = a.ptr(), *qc = a.ptr(), *sc = a.ptr();
    const hipStream_t st = a.stream();
    return run(a, [&] {
        return g_quantize_grouped(x, x_rows, N, ldx, index, M, ends, g, ro, co, (mx_layout)layout, q, s, qc, sc, st);
    });
}

// (M, N, K, group_ends, groups, A, A_scale, B, B_scale, layout, out_dtype, bias, C, ldc, stream)
PyObject *gemm_grouped(PyObject *, PyObject *const *v, Py_ssize_t n) {
    if (!count_is(n, 15)) return nullptr;
    Args a(v, n);
    const int64_t M = a.i64(), N = a.i64(), K = a.i64(), groups = a.i64(4);
    const int32_t *ends = a.i32ptr(groups);
    const int g = a.i32();
    const void *A = a.ptr(), *As = a.ptr(), *B = a.ptr(), *Bs = a.ptr();
    const int layout = a.i32(), dtype = a.i32();
    const void *bias = a.ptr();
    void *C = a.ptr();
    const int64_t ldc = a.i64();
    const hipStream_t st = a.stream();
    return run(a, [&] {
        return g_gemm_grouped(M, N, K, ends, g, A, As, B, Bs, (mx_layout)layout, (mx_dtype)dtype, bias, C, ldc, st);
    });
}

// (M, N, K, group_ends, groups, A, A_scale, B, B_scale, layout, out_dtype, C, ldc, group_stride, stream)
PyObject *gemm_grouped_wgrad(PyObject *, PyObject *const *v, Py_ssize_t n) {
    if (!count_is(n, 15)) return nullptr;
    Args a(v, n);
    const int64_t M = a.i64(), N = a.i64(), K = a.i64(), groups = a.i64(4);
    const int32_t *ends = a.i32ptr(groups);
    const int g = a.i32();
    const void *A = a.ptr(), *As = a.ptr(), *B = a.ptr(), *Bs = a.ptr();
    const int layout = a.i32(), dtype = a.i32();
    void *C = a.ptr();
    const int64_t ldc = a.i64(), stride = a.i64();
    const hipStream_t st = a.stream();
    return run(a, [&] {
        return g_gemm_grouped_wgrad(M, N, K, ends, g, A, As, B, Bs, (mx_layout)layout, (mx_dtype)dtype, C, ldc, stride,
                                    st);
    });
}

PyObject *bind(PyObject *, PyObject *args) {
    unsigned long long q, g, w;
    PyObject *dptr, *i32ptr, *stream, *opts;
    if (!PyArg_ParseTuple(args, "KKKOOOO", &q, &g, &w, &dptr, &i32ptr, &stream, &opts)) return nullptr;
    g_quantize_grouped = (decltype(g_quantize_grouped))(uintptr_t)q;
    g_gemm_grouped = (decltype(g_gemm_grouped))(uintptr_t)g;
    g_gemm_grouped_wgrad = (decltype(g_gemm_grouped_wgrad))(uintptr_t)w;
    Py_INCREF(dptr);
    Py_INCREF(i32ptr);
    Py_INCREF(stream);
    Py_INCREF(opts);
    g_dptr = dptr;
    g_i32ptr = i32ptr;
    g_stream = stream;
    g_quant_opts = opts;
    Py_RETURN_NONE;
}

PyMethodDef g_methods[] = {
    {"bind", bind, METH_VARARGS, nullptr},
    {"quantize_grouped", (PyCFunction)(void (*)(void))quantize_grouped, METH_FASTCALL, nullptr},
    {"gemm_grouped", (PyCFunction)(void (*)(void))gemm_grouped, METH_FASTCALL, nullptr},
    {"gemm_grouped_wgrad", (PyCFunction)(void (*)(void))gemm_grouped_wgrad, METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr},
};

PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_marshal", nullptr, -1, g_methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__marshal(void) {
    s_is_cuda = PyUnicode_InternFromString("is_cuda");
    s_data_ptr = PyUnicode_InternFromString("data_ptr");
    s_dtype = PyUnicode_InternFromString("dtype");
    s_is_contiguous = PyUnicode_InternFromString("is_contiguous");
    s_numel = PyUnicode_InternFromString("numel");
    s_torch = PyUnicode_InternFromString("torch");
    return PyModule_Create(&g_module);
}
