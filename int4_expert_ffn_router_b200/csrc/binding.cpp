// binding.cpp -- the Python module behind the operators around the layer
// (coli_moe_dispatch, coli_moe_combine, coli_moe_route_backward, coli_block_norm
// and their gradients): it reads torch tensors, checks what the C ABI cannot
// see (types, shapes, devices) and calls the library. A call costs about as
// much as its launches; through ctypes, with the checks in Python, it cost
// three times that (10 us against 3 us for one launch), which is what a decoded
// token waits for.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <initializer_list>
#include <string>

#include "../../include/coli_moe.h"

namespace {

struct Refused {
    PyObject* type;
    std::string msg;
};
[[noreturn]] void value_error(const std::string& m) { throw Refused{PyExc_ValueError, m}; }
[[noreturn]] void type_error(const std::string& m) { throw Refused{PyExc_TypeError, m}; }

std::string shape_of(const at::Tensor& t) {
    std::string s = "[";
    for (int64_t i = 0; i < t.dim(); ++i) s += (i ? ", " : "") + std::to_string(t.size(i));
    return s + "]";
}

// The tensor of an argument, NULL for None.
const at::Tensor* tensor(PyObject* o, const char* name) {
    if (o == Py_None) return nullptr;
    if (!THPVariable_Check(o)) type_error(std::string(name) + " must be a torch tensor");
    const at::Tensor& t = THPVariable_Unpack(o);
    if (!t.is_cuda()) value_error(std::string(name) + " must be a CUDA tensor");
    if (t.layout() != at::kStrided) type_error(std::string(name) + " must be a dense tensor");
    if (t.is_neg()) value_error(std::string(name) + " must not be a lazily negated view");
    return &t;
}
const at::Tensor& required(PyObject* o, const char* name) {
    const at::Tensor* t = tensor(o, name);
    if (!t) type_error(std::string(name) + " must be a torch tensor");
    return *t;
}
void on_device(const at::Tensor& t, const char* name, int dev) {
    if (t.get_device() != dev) value_error(std::string(name) + " is not on cuda:" + std::to_string(dev));
}

struct Mat {
    void* p = nullptr;
    coli_dtype t = COLI_F32;
    int64_t stride = 0, rows = 0;
};
// A matrix argument [rows][cols] (rows < 0: any number), float32 or bfloat16, rows any distance apart.
Mat mat(PyObject* o, const char* name, int64_t rows, int64_t cols, int dev) {
    Mat m;
    m.stride = cols;
    const at::Tensor* t = tensor(o, name);
    if (!t) return m;
    const auto st = t->scalar_type();
    if (st == at::kFloat) m.t = COLI_F32;
    else if (st == at::kBFloat16) m.t = COLI_BF16;
    else type_error(std::string(name) + " must be float32 or bfloat16");
    if (t->dim() != 2 || t->size(1) != cols || (rows >= 0 && t->size(0) != rows))
        value_error(std::string(name) + " must have shape [" + (rows < 0 ? "*" : std::to_string(rows)) + ", " +
                    std::to_string(cols) + "], not " + shape_of(*t));
    on_device(*t, name, dev);
    if (t->stride(1) != 1 && cols > 1) value_error(std::string(name) + " must have contiguous rows");
    m.rows = t->size(0);
    m.stride = t->stride(0);
    if (m.rows <= 1 && m.stride < cols) m.stride = cols;
    m.p = t->data_ptr();
    return m;
}

// A dense array argument of `dim` sizes; NULL for None.
void* array(PyObject* o, const char* name, at::ScalarType st, int dev, int64_t a, int64_t b = -1) {
    const at::Tensor* t = tensor(o, name);
    if (!t) return nullptr;
    if (t->scalar_type() != st) type_error(std::string(name) + (st == at::kInt ? " must be int32" : " must be float32"));
    const bool shaped = b < 0 ? t->dim() == 1 && t->size(0) == a : t->dim() == 2 && t->size(0) == a && t->size(1) == b;
    if (!shaped)
        value_error(std::string(name) + " must have shape [" + std::to_string(a) + (b < 0 ? "" : ", " + std::to_string(b)) +
                    "], not " + shape_of(*t));
    on_device(*t, name, dev);
    if (!t->is_contiguous()) value_error(std::string(name) + " must be contiguous");
    return t->data_ptr();
}
float* floats(PyObject* o, const char* name, int dev, int64_t a, int64_t b = -1) {
    return static_cast<float*>(array(o, name, at::kFloat, dev, a, b));
}
int32_t* ints(PyObject* o, const char* name, int dev, int64_t a, int64_t b = -1) {
    return static_cast<int32_t*>(array(o, name, at::kInt, dev, a, b));
}

struct Work {
    void* p = nullptr;
    int64_t bytes = 0;
};
Work work_of(PyObject* o, int dev) {
    Work w;
    if (const at::Tensor* t = tensor(o, "work")) {
        on_device(*t, "work", dev);
        if (!t->is_contiguous()) value_error("work must be contiguous");
        w.p = t->data_ptr();
        w.bytes = t->numel() * (int64_t)t->element_size();
    }
    return w;
}

int64_t integer(PyObject* o, const char* name) {
    const long long v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred()) {
        PyErr_Clear();
        type_error(std::string(name) + " must be an integer");
    }
    return v;
}
int sized(int64_t v, const char* name) {  // a size that the C ABI takes as int
    if (v < 0 || v > INT32_MAX) value_error(std::string(name) + " is out of range");
    return (int)v;
}

// A stream argument: None (the current stream of `dev`), an object with cuda_stream, or a handle.
coli_stream stream_of(PyObject* o, int dev) {
    if (o == Py_None) return c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)dev).stream();
    static PyObject* name = PyUnicode_InternFromString("cuda_stream");
    PyObject* h = PyLong_Check(o) ? Py_NewRef(o) : PyObject_GetAttr(o, name);
    if (!h) {
        PyErr_Clear();
        type_error("stream must be a CUDA stream");
    }
    const unsigned long long v = PyLong_AsUnsignedLongLong(h);
    Py_DECREF(h);
    if (v == (unsigned long long)-1 && PyErr_Occurred()) {
        PyErr_Clear();
        type_error("stream must be a CUDA stream");
    }
    return reinterpret_cast<coli_stream>(v);
}

// A Block argument (its device and width: those of its arrays, None without any).
const coli_block_params* block_of(PyObject* o, const char* name, int64_t hidden, int dev) {
    if (o == Py_None) return nullptr;
    static PyObject* keys[3] = {PyUnicode_InternFromString("address"), PyUnicode_InternFromString("device"),
                                PyUnicode_InternFromString("hidden")};
    int64_t v[3] = {0, -1, -1};
    for (int i = 0; i < 3; ++i) {
        PyObject* a = PyObject_GetAttr(o, keys[i]);
        if (!a) {
            PyErr_Clear();
            type_error(std::string(name) + " must be a Block");
        }
        if (a != Py_None) v[i] = PyLong_AsLongLong(a);
        const bool none = a == Py_None;
        Py_DECREF(a);
        if (PyErr_Occurred() || (i == 0 && (none || !v[0]))) {
            PyErr_Clear();
            type_error(std::string(name) + " must be a Block");
        }
    }
    if (v[1] >= 0 && (v[1] != dev || v[2] != hidden))
        value_error(std::string(name) + "'s arrays are not [" + std::to_string(hidden) + "] on cuda:" + std::to_string(dev));
    return reinterpret_cast<const coli_block_params*>(v[0]);
}

struct Slots {
    int dev, T, K;
};
Slots slots_of(PyObject* o, const char* name) {
    const at::Tensor& t = required(o, name);
    if (t.dim() != 2) value_error(std::string(name) + " must have shape [tokens, top_k], not " + shape_of(t));
    return {(int)t.get_device(), sized(t.size(0), name), sized(t.size(1), name)};
}
int64_t width_of(const at::Tensor& t, const char* name) {
    if (t.dim() != 2) value_error(std::string(name) + " must be a matrix, not " + shape_of(t));
    return sized(t.size(1), name);
}

// A tensor argument was written: its version moves, as with torch's in-place
// operations, so that autograd notices if it had saved the values. (A tensor of
// inference mode has no version.)
void written(PyObject* o) {
    if (o == Py_None) return;
    const at::Tensor& t = THPVariable_Unpack(o);
    if (!t.is_inference()) t.unsafeGetTensorImpl()->bump_version();
}

// Runs f (which makes one library call through `call`) and returns its status
// to Python; `outs`: the arguments that it writes. Nothing within `call` may
// throw: the interpreter's lock is released there.
template <typename F>
PyObject* guarded(PyObject* const* a, Py_ssize_t given, Py_ssize_t wanted, std::initializer_list<int> outs, F f) {
    try {
        if (given != wanted) type_error("wrong number of arguments");
        const coli_status st = f();
        if (st == COLI_OK)
            for (int i : outs) written(a[i]);
        return PyLong_FromLong((long)st);
    } catch (const Refused& r) {
        PyErr_SetString(r.type, r.msg.c_str());
    } catch (const std::exception& e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
    }
    return nullptr;
}
template <typename F>
coli_status call(F f) {
    PyThreadState* s = PyEval_SaveThread();
    const coli_status st = f();
    PyEval_RestoreThread(s);
    return st;
}

#define ENTRY(name) PyObject* name(PyObject*, PyObject* const* a, Py_ssize_t n)

// ids, x, n_experts, counts, offsets, pos, slot, rows, work, stream
ENTRY(dispatch) {
    return guarded(a, n, 10, {3, 4, 5, 6, 7, 8}, [&] {
        const Slots s = slots_of(a[0], "ids");
        const int E = sized(integer(a[2], "n_experts"), "n_experts");
        const at::Tensor* x = tensor(a[1], "x");
        const int64_t H = x ? width_of(*x, "x") : 1;
        const Mat mx = mat(a[1], "x", s.T, H, s.dev), mr = mat(a[7], "rows", -1, H, s.dev);
        const Work w = work_of(a[8], s.dev);
        const int32_t* ids = ints(a[0], "ids", s.dev, s.T, s.K);
        int32_t *counts = ints(a[3], "counts", s.dev, E), *offsets = ints(a[4], "offsets", s.dev, (int64_t)E + 1);
        int32_t *pos = ints(a[5], "pos", s.dev, s.T, s.K), *slot = ints(a[6], "slot", s.dev, (int64_t)s.T * s.K);
        const coli_stream st = stream_of(a[9], s.dev);
        return call([&] {
            return coli_moe_dispatch(ids, s.T, s.K, E, mx.p, mx.t, mx.stride, (int)H, counts, offsets,
                                     pos, slot, mr.p, mr.t, mr.stride, mr.rows, w.p, w.bytes, s.dev, st);
        });
    });
}

Mat base_of(PyObject* o, const Mat& out, int64_t T, int64_t H, int dev) {
    const Mat b = mat(o, "base", T, H, dev);
    if (b.p && b.t != out.t) type_error("base must have the output's dtype");
    return b;
}

// pos, drows, dx, base, stream
ENTRY(dispatch_backward) {
    return guarded(a, n, 5, {2}, [&] {
        const Slots s = slots_of(a[0], "pos");
        const int64_t H = width_of(required(a[2], "dx"), "dx");
        required(a[1], "drows");
        const int32_t* pos = ints(a[0], "pos", s.dev, s.T, s.K);
        const Mat r = mat(a[1], "drows", -1, H, s.dev), y = mat(a[2], "dx", s.T, H, s.dev);
        const Mat b = base_of(a[3], y, s.T, H, s.dev);
        const coli_stream st = stream_of(a[4], s.dev);
        return call([&] {
            return coli_moe_dispatch_backward(pos, s.T, s.K, r.p, r.t, r.stride, r.rows, (int)H, b.p, b.stride, y.p, y.t,
                                              y.stride, s.dev, st);
        });
    });
}

// pos, weights, rows, y, base, stream
ENTRY(combine) {
    return guarded(a, n, 6, {3}, [&] {
        const Slots s = slots_of(a[0], "pos");
        const int64_t H = width_of(required(a[3], "y"), "y");
        required(a[2], "rows");
        const int32_t* pos = ints(a[0], "pos", s.dev, s.T, s.K);
        const float* w = floats(a[1], "weights", s.dev, s.T, s.K);
        const Mat r = mat(a[2], "rows", -1, H, s.dev), y = mat(a[3], "y", s.T, H, s.dev);
        const Mat b = base_of(a[4], y, s.T, H, s.dev);
        const coli_stream st = stream_of(a[5], s.dev);
        return call([&] {
            return coli_moe_combine(pos, w, s.T, s.K, r.p, r.t, r.stride, r.rows, (int)H, b.p, b.stride, y.p, y.t, y.stride,
                                    s.dev, st);
        });
    });
}

// pos, weights, dy, rows, drows, dweights, stream
ENTRY(combine_backward) {
    return guarded(a, n, 7, {4, 5}, [&] {
        const Slots s = slots_of(a[0], "pos");
        const int64_t H = width_of(required(a[2], "dy"), "dy");
        const int32_t* pos = ints(a[0], "pos", s.dev, s.T, s.K);
        const float* w = floats(a[1], "weights", s.dev, s.T, s.K);
        const Mat g = mat(a[2], "dy", s.T, H, s.dev), r = mat(a[3], "rows", -1, H, s.dev);
        const bool with_rows = a[3] != Py_None;
        const Mat d = mat(a[4], "drows", with_rows ? r.rows : -1, H, s.dev);
        if (with_rows && a[4] != Py_None && d.t != r.t) type_error("drows must have rows' dtype");
        if (!with_rows && a[5] != Py_None) value_error("dweights needs rows");
        float* dw = floats(a[5], "dweights", s.dev, s.T, s.K);
        const coli_stream st = stream_of(a[6], s.dev);
        return call([&] {
            return coli_moe_combine_backward(pos, w, s.T, s.K, g.p, g.t, g.stride, (int)H, r.p, with_rows ? r.t : d.t,
                                             r.stride, with_rows ? r.rows : d.rows, d.p, d.stride, dw, s.dev, st);
        });
    });
}

// router_w, x, ids, weights, dweights, offsets, slot, dlogits, dx, drouter_w, dbias, work, stream
ENTRY(route_backward) {
    return guarded(a, n, 13, {7, 8, 9, 10, 11}, [&] {
        const Slots s = slots_of(a[2], "ids");
        const at::Tensor& wr = required(a[0], "router_w");
        const int64_t H = width_of(wr, "router_w"), E = sized(wr.size(0), "router_w");
        const float* pw = floats(a[0], "router_w", s.dev, E, H);
        const Mat x = mat(a[1], "x", s.T, H, s.dev), dx = mat(a[8], "dx", s.T, H, s.dev);
        if (a[1] != Py_None && a[8] != Py_None && x.t != dx.t) type_error("dx must have x's dtype");
        const int32_t* ids = ints(a[2], "ids", s.dev, s.T, s.K);
        const float *w = floats(a[3], "weights", s.dev, s.T, s.K), *dw = floats(a[4], "dweights", s.dev, s.T, s.K);
        const int32_t *off = ints(a[5], "offsets", s.dev, E + 1), *slot = ints(a[6], "slot", s.dev, (int64_t)s.T * s.K);
        float *dl = floats(a[7], "dlogits", s.dev, s.T, s.K), *dwr = floats(a[9], "drouter_w", s.dev, E, H);
        float* db = floats(a[10], "dbias", s.dev, E);
        const Work work = work_of(a[11], s.dev);
        const coli_stream st = stream_of(a[12], s.dev);
        return call([&] {
            return coli_moe_route_backward(pw, (int)E, (int)H, s.K, x.p, a[1] != Py_None ? x.t : dx.t, x.stride, s.T, ids, w,
                                           dw, off, slot, dl, dx.p, dx.stride, dwr, db, work.p, work.bytes, s.dev, st);
        });
    });
}

// prev, next, x, y, x_out, n, token_gate, stream
ENTRY(block_norm) {
    return guarded(a, n, 8, {4, 5}, [&] {
        const at::Tensor& tx = required(a[2], "x");
        const int dev = (int)tx.get_device();
        const int64_t H = width_of(tx, "x");
        const int T = sized(tx.size(0), "x");
        const coli_block_params *prev = block_of(a[0], "prev", H, dev), *next = block_of(a[1], "next", H, dev);
        const Mat x = mat(a[2], "x", T, H, dev), y = mat(a[3], "y", T, H, dev), xo = mat(a[4], "x_out", T, H, dev);
        const Mat m = mat(a[5], "n", T, H, dev);
        if (a[4] != Py_None && xo.t != x.t) type_error("x_out must have x's dtype");
        const float* u = floats(a[6], "token_gate", dev, T);
        const coli_stream st = stream_of(a[7], dev);
        return call([&] {
            return coli_block_norm(prev, next, x.p, x.t, x.stride, y.p, y.t, y.stride, u, xo.p, xo.stride, m.p, m.t,
                                   m.stride, T, (int)H, dev, st);
        });
    });
}

// prev, next, x_out, y, dx_out, dn, dx, dy, dpre_gain, dpost_gain, dgate, token_gate, dtoken_gate, work, stream
ENTRY(block_norm_backward) {
    return guarded(a, n, 15, {6, 7, 8, 9, 10, 12, 13}, [&] {
        const at::Tensor& ts = required(a[2], "x_out");
        const int dev = (int)ts.get_device();
        const int64_t H = width_of(ts, "x_out");
        const int T = sized(ts.size(0), "x_out");
        const coli_block_params *prev = block_of(a[0], "prev", H, dev), *next = block_of(a[1], "next", H, dev);
        const Mat s = mat(a[2], "x_out", T, H, dev), y = mat(a[3], "y", T, H, dev), o = mat(a[4], "dx_out", T, H, dev);
        const Mat dn = mat(a[5], "dn", T, H, dev), dx = mat(a[6], "dx", T, H, dev), dy = mat(a[7], "dy", T, H, dev);
        if ((a[4] != Py_None && o.t != s.t) || (a[6] != Py_None && dx.t != s.t))
            type_error("dx_out and dx must have x_out's dtype");
        if (a[3] != Py_None && a[7] != Py_None && dy.t != y.t) type_error("dy must have y's dtype");
        float *dq = floats(a[8], "dpre_gain", dev, H), *dp = floats(a[9], "dpost_gain", dev, H);
        float *dg = floats(a[10], "dgate", dev, H), *du = floats(a[12], "dtoken_gate", dev, T);
        const float* u = floats(a[11], "token_gate", dev, T);
        const Work w = work_of(a[13], dev);
        const coli_stream st = stream_of(a[14], dev);
        return call([&] {
            return coli_block_norm_backward(prev, next, s.p, s.t, s.stride, y.p, y.t, y.stride, u, o.p, o.stride, dn.p, dn.t,
                                            dn.stride, dx.p, dx.stride, dy.p, dy.stride, dq, dp, dg, du, w.p, w.bytes, T,
                                            (int)H, dev, st);
        });
    });
}

#define METHOD(f) {#f, reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(f)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {METHOD(dispatch),       METHOD(dispatch_backward), METHOD(combine),
                         METHOD(combine_backward), METHOD(route_backward),  METHOD(block_norm),
                         METHOD(block_norm_backward), {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__binding() { return PyModule_Create(&module); }
