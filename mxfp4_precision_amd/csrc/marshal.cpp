// Python extension module: the arguments of the calls that run many times a
// step or token (grouped quantization and products, FP8 with block scales,
// expert layers for a few tokens, gradient norms) from Python objects to C.
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
decltype(&mx_quantize_fp8_b128) g_quantize_fp8_b128;
decltype(&mx_gemm_f8_b128) g_gemm_f8_b128;
decltype(&mx_linear_f8_b128) g_linear_f8_b128;
decltype(&mx_linear_f8_b128_bytes) g_linear_f8_b128_bytes;
decltype(&mx_experts_a16w4) g_experts_a16w4;
decltype(&mx_experts_a16w4_bytes) g_experts_a16w4_bytes;
decltype(&mx_grad_norm) g_grad_norm;
decltype(&mx_grad_norm_bytes) g_grad_norm_bytes;
decltype(&mx_clip_grads) g_clip_grads;
PyObject *g_dptr, *g_i32ptr, *g_f32ptr, *g_stream, *g_room;   // the Python binding's converters and checks
PyObject *g_quant_opts, *g_grad_tensor;                       // ... and its structures
PyObject *g_int32, *g_float32;                                // torch's types, once torch is imported
PyObject *s_is_cuda, *s_data_ptr, *s_dtype, *s_is_contiguous, *s_numel, *s_element_size, *s_torch, *s_type;

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
    // count consecutive 32-bit integers, or numbers
    const int32_t *i32ptr(int64_t count) { return (const int32_t *)values(count, g_int32, "int32", g_i32ptr); }
    const float *f32ptr(int64_t count) { return (const float *)values(count, g_float32, "float32", g_f32ptr); }
    uintptr_t values(int64_t count, PyObject *&type, const char *name, PyObject *convert) {
        PyObject *o = next();
        if (bad || o == Py_None) return 0;
        if (!PyLong_CheckExact(o) && usual_values(o, count, type, name)) return tensor(o);
        PyObject *r = nullptr, *c = PyLong_FromLongLong(count);
        if (c) r = PyObject_CallFunctionObjArgs(convert, o, c, nullptr);
        Py_XDECREF(c);
        return address(r);
    }
    static bool usual_values(PyObject *o, int64_t count, PyObject *&type, const char *name) {
        if (!type) {
            PyObject *torch = PyImport_GetModule(s_torch);
            if (torch) type = PyObject_GetAttrString(torch, name);
            Py_XDECREF(torch);
            PyErr_Clear();
            if (!type) return false;
        }
        PyObject *t = PyObject_GetAttr(o, s_dtype);
        const bool same = t == type;
        Py_XDECREF(t);
        PyErr_Clear();
        return same && is_true(PyObject_GetAttr(o, s_is_cuda)) && is_true(PyObject_CallMethodNoArgs(o, s_is_contiguous)) &&
               number(PyObject_CallMethodNoArgs(o, s_numel)) >= count;
    }
    static int64_t number(PyObject *result) {   // takes the reference; errors count as -1
        const long long v = result ? PyLong_AsLongLong(result) : -1;
        Py_XDECREF(result);
        PyErr_Clear();
        return v;
    }
    // a workspace; need(&bytes): its size (a status other than success is the call's to report)
    template <typename F>
    void *space(F need) {
        PyObject *o = v[at];
        size_t bytes = 0;
        if (!bad && o != Py_None && !PyLong_CheckExact(o) && need(&bytes) == MX_SUCCESS) {
            const bool usual = is_true(PyObject_GetAttr(o, s_is_cuda)) &&
                               is_true(PyObject_CallMethodNoArgs(o, s_is_contiguous)) &&
                               number(PyObject_CallMethodNoArgs(o, s_numel)) *
                                       number(PyObject_CallMethodNoArgs(o, s_element_size)) >= (int64_t)bytes;
            if (!usual) {
                PyObject *n = PyLong_FromSize_t(bytes), *r = n ? PyObject_CallFunctionObjArgs(g_room, o, n, nullptr) : nullptr;
                Py_XDECREF(n);
                Py_XDECREF(r);
                if (!r) bad = true;
            }
        }
        return ptr();
    }
    // a table of `count` gradients: an array of the binding's mx_grad_tensor, or None
    const mx_grad_tensor *grads(int64_t count) {
        PyObject *o = next();
        if (bad || o == Py_None) return nullptr;
        PyObject *type = PyObject_GetAttr((PyObject *)Py_TYPE(o), s_type);
        const bool same = type == g_grad_tensor;
        Py_XDECREF(type);
        PyErr_Clear();
        if (!same) {
            PyErr_Format(PyExc_TypeError, "an array of grad_table is required, got %R", (PyObject *)Py_TYPE(o));
            bad = true;
            return nullptr;
        }
        if (PyObject_GetBuffer(o, &views[held], PyBUF_SIMPLE) != 0) {
            bad = true;
            return nullptr;
        }
        const Py_buffer &b = views[held++];
        const int64_t have = b.len / (int64_t)sizeof(mx_grad_tensor);
        if (count > have) {
            PyErr_Format(PyExc_ValueError, "count=%lld, but the table holds %lld tensors", (long long)count, (long long)have);
            bad = true;
        }
        return (const mx_grad_tensor *)b.buf;
    }
    double f64() {
        PyObject *o = next();
        if (bad) return 0;
        const double r = PyFloat_AsDouble(o);
        if (r == -1 && PyErr_Occurred()) bad = true;
        return r;
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

// (x, M, N, ldx, row_fmt, row_opts, col_fmt, col_opts, layout, q_row, s_row, q_col, s_col, stream)
PyObject *quantize_fp8_b128(PyObject *, PyObject *const *v, Py_ssize_t n) {
    if (!count_is(n, 14)) return nullptr;
    Args a(v, n);
    const void *x = a.ptr();
    const int64_t M = a.i64(), N = a.i64(), ldx = a.i64();
    const int fr = a.i32();
    const mx_quant_opts *ro = a.options();
    const int fc = a.i32();
    const mx_quant_opts *co = a.options();
    const int layout = a.i32();
    void *q = a.ptr(), *s = a.ptr(), *qc = a.ptr(), *sc = a.ptr();
    const hipStream_t st = a.stream();
    return run(a, [&] {
        return g_quantize_fp8_b128(x, M, N, ldx, fr, ro, fc, co, (mx_layout)layout, q, s, qc, sc, st);
    });
}

// (transA, transB, M, N, K, fmt_a, A, A_scale, fmt_b, B, B_scale, layout, out_dtype, bias, C, ldc, stream)
PyObject *gemm_f8_b128(PyObject *, PyObject *const *v, Py_ssize_t n) {
    if (!count_is(n, 17)) return nullptr;
    Args a(v, n);
    const int ta = a.i32(), tb = a.i32();
    const int64_t M = a.i64(), N = a.i64(), K = a.i64();
    const int fa = a.i32();
    const void *A = a.ptr(), *As = a.ptr();
    const int fb = a.i32();
    const void *B = a.ptr(), *Bs = a.ptr();
    const int layout = a.i32(), dtype = a.i32();
    const void *bias = a.ptr();
    void *C = a.ptr();
    const int64_t ldc = a.i64();
    const hipStream_t st = a.stream();
    return run(a, [&] {
        return g_gemm_f8_b128(ta, tb, M, N, K, fa, A, As, fb, B, Bs, (mx_layout)layout, (mx_dtype)dtype, bias, C, ldc, st);
    });
}

// (M, N, K, fmt_x, x, ldx, fmt_w, W, W_scale, layout, out_dtype, bias, y, ldy, workspace, stream)
PyObject *linear_f8_b128(PyObject *, PyObject *const *v, Py_ssize_t n) {
    if (!count_is(n, 16)) return nullptr;
    Args a(v, n);
    const int64_t M = a.i64(), N = a.i64(), K = a.i64();
    const int fx = a.i32();
    const void *x = a.ptr();
    const int64_t ldx = a.i64();
    const int fw = a.i32();
    const void *W = a.ptr(), *Ws = a.ptr();
    const int layout = a.i32(), dtype = a.i32();
    const void *bias = a.ptr();
    void *y = a.ptr();
    const int64_t ldy = a.i64();
    void *ws = a.space([&](size_t *bytes) { return g_linear_f8_b128_bytes(M, K, bytes); });
    const hipStream_t st = a.stream();
    return run(a, [&] {
        return g_linear_f8_b128(M, N, K, fx, x, ldx, fw, W, Ws, (mx_layout)layout, (mx_dtype)dtype, bias, y, ldy, ws, st);
    });
}

// (tokens, K, inner, experts, topk, x, ldx, ids, weights, W1, W1_scale, W2, W2_scale, layout, out_dtype, y, ldy,
//  workspace, stream)
PyObject *experts_a16w4(PyObject *, PyObject *const *v, Py_ssize_t n) {
    if (!count_is(n, 19)) return nullptr;
    Args a(v, n);
    const int64_t tokens = a.i64(), K = a.i64(), inner = a.i64();
    const int experts = a.i32(), topk = a.i32();
    const void *x = a.ptr();
    const int64_t ldx = a.i64();
    // (sizes that the call refuses could pass 64 bits)
    const int64_t pairs = tokens >= 0 && tokens < (int64_t(1) << 31) && topk >= 0 ? tokens * topk : 0;
    const int32_t *ids = a.i32ptr(pairs);
    const float *weights = a.f32ptr(pairs);
    const void *W1 = a.ptr(), *W1s = a.ptr(), *W2 = a.ptr(), *W2s = a.ptr();
    const int layout = a.i32(), dtype = a.i32();
    void *y = a.ptr();
    const int64_t ldy = a.i64();
    void *ws = a.space([&](size_t *bytes) { return g_experts_a16w4_bytes(tokens, inner, topk, bytes); });
    const hipStream_t st = a.stream();
    return run(a, [&] {
        return g_experts_a16w4(tokens, K, inner, experts, topk, x, ldx, ids, weights, W1, W1s, W2, W2s,
                               (mx_layout)layout, (mx_dtype)dtype, y, ldy, ws, st);
    });
}

// (tensors, count, max_norm, grad_scale, workspace, info, step, stream)
PyObject *grad_norm(PyObject *, PyObject *const *v, Py_ssize_t n) {
    if (!count_is(n, 8)) return nullptr;
    Args a(v, n);
    const int64_t count = a.i64(1);
    const mx_grad_tensor *t = a.grads(count);
    a.at = 2;
    const double most = a.f64(), scale = a.f64();
    void *ws = a.space([&](size_t *bytes) { return g_grad_norm_bytes(count, bytes); });
    void *info = a.ptr(), *step = a.ptr();
    const hipStream_t st = a.stream();
    return run(a, [&] {
        return g_grad_norm(t, count, most, scale, ws, (mx_grad_norm_info *)info, (mx_adamw_step *)step, st);
    });
}

// (tensors, count, info, stream)
PyObject *clip_grads(PyObject *, PyObject *const *v, Py_ssize_t n) {
    if (!count_is(n, 4)) return nullptr;
    Args a(v, n);
    const int64_t count = a.i64(1);
    const mx_grad_tensor *t = a.grads(count);
    a.at = 2;
    const void *info = a.ptr();
    const hipStream_t st = a.stream();
    return run(a, [&] { return g_clip_grads(t, count, (const mx_grad_norm_info *)info, st); });
}

template <typename F>
void take(F &f, PyObject *addresses, Py_ssize_t i) {
    f = (F)(uintptr_t)PyLong_AsUnsignedLongLong(PyTuple_GET_ITEM(addresses, i));
}

// (addresses of the library's entry points in the order below, then the binding's converters and structures)
PyObject *bind(PyObject *, PyObject *args) {
    PyObject *f, *o[7];
    if (!PyArg_ParseTuple(args, "O!OOOOOOO", &PyTuple_Type, &f, &o[0], &o[1], &o[2], &o[3], &o[4], &o[5], &o[6]))
        return nullptr;
    if (PyTuple_GET_SIZE(f) != 12) {
        PyErr_SetString(PyExc_ValueError, "12 entry points expected");
        return nullptr;
    }
    Py_ssize_t i = 0;
    take(g_quantize_grouped, f, i++);
    take(g_gemm_grouped, f, i++);
    take(g_gemm_grouped_wgrad, f, i++);
    take(g_quantize_fp8_b128, f, i++);
    take(g_gemm_f8_b128, f, i++);
    take(g_linear_f8_b128, f, i++);
    take(g_linear_f8_b128_bytes, f, i++);
    take(g_experts_a16w4, f, i++);
    take(g_experts_a16w4_bytes, f, i++);
    take(g_grad_norm, f, i++);
    take(g_grad_norm_bytes, f, i++);
    take(g_clip_grads, f, i++);
    if (PyErr_Occurred()) return nullptr;
    PyObject **to[7] = {&g_dptr, &g_i32ptr, &g_f32ptr, &g_stream, &g_room, &g_quant_opts, &g_grad_tensor};
    for (int k = 0; k < 7; ++k) {
        Py_INCREF(o[k]);
        *to[k] = o[k];
    }
    Py_RETURN_NONE;
}

PyMethodDef g_methods[] = {
    {"bind", bind, METH_VARARGS, nullptr},
    {"quantize_grouped", (PyCFunction)(void (*)(void))quantize_grouped, METH_FASTCALL, nullptr},
    {"gemm_grouped", (PyCFunction)(void (*)(void))gemm_grouped, METH_FASTCALL, nullptr},
    {"gemm_grouped_wgrad", (PyCFunction)(void (*)(void))gemm_grouped_wgrad, METH_FASTCALL, nullptr},
    {"quantize_fp8_b128", (PyCFunction)(void (*)(void))quantize_fp8_b128, METH_FASTCALL, nullptr},
    {"gemm_f8_b128", (PyCFunction)(void (*)(void))gemm_f8_b128, METH_FASTCALL, nullptr},
    {"linear_f8_b128", (PyCFunction)(void (*)(void))linear_f8_b128, METH_FASTCALL, nullptr},
    {"experts_a16w4", (PyCFunction)(void (*)(void))experts_a16w4, METH_FASTCALL, nullptr},
    {"grad_norm", (PyCFunction)(void (*)(void))grad_norm, METH_FASTCALL, nullptr},
    {"clip_grads", (PyCFunction)(void (*)(void))clip_grads, METH_FASTCALL, nullptr},
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
    s_element_size = PyUnicode_InternFromString("element_size");
    s_torch = PyUnicode_InternFromString("torch");
    s_type = PyUnicode_InternFromString("_type_");
    return PyModule_Create(&g_module);
}
