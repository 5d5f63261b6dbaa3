// ops_bind.cpp - argument marshalling of the operators of ampops.h for Python:
// checks tensors, takes their addresses and sizes and calls the C entry points.
//
// The smallest calls take 2.4 us on the host for the C call and its launch; the
// same checks in Python took another 2 to 6 us a call (0.3 us a tensor), here
// they take 0.3 us in all.  ops.py holds the documented functions; each passes
// its arguments on in order.  A tensor that does not fit raises ValueError
// before anything is called; the return value is the entry point's status.
// A call runs on the device of the tensor that gives it its shape, whichever is
// current, and every other tensor has to be there too (an address of another
// GPU would be a fault, not a status).
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cstring>
#include <exception>
#include <string>

#include "ampops.h"

namespace {

// The entry points, by their addresses in the library that _lib.py loaded.
struct Entries {
    decltype(&fp4_quant_mx) quant;
    decltype(&fp4_dequant_mx) dequant;
    decltype(&fp4_product_mx) product;
    decltype(&amp_layer_norm_forward) norm_forward;
    decltype(&amp_layer_norm_backward) norm_backward;
    decltype(&amp_act_forward_mx8) act_forward;
    decltype(&amp_act_backward_mx8) act_backward;
    decltype(&amp_ckpt8_save) save;
    decltype(&amp_ckpt8_restore) restore;
} g{};

struct Refused {
    std::string why;
};
[[noreturn]] void refuse(const std::string &why) { throw Refused{why}; }

std::string type_name(at::ScalarType t) { return std::string("dtype ") + c10::toString(t); }

const at::Tensor &tensor(PyObject *o, const char *what) {
    if (!THPVariable_Check(o)) refuse(std::string(what) + ": needs a tensor");
    return THPVariable_Unpack(o);
}
// Address of a contiguous GPU tensor on the call's device, of at least numel
// elements; None: NULL.
void *address(const at::Tensor &t, const char *what, int64_t numel, int64_t device) {
    if (!t.is_cuda() || !t.is_contiguous()) refuse(std::string(what) + ": needs a contiguous CUDA tensor");
    if (device >= 0 && t.get_device() != device)  // (below 0: the shape's tensor will be refused)
        refuse(std::string(what) + ": on cuda:" + std::to_string(t.get_device()) + ", the call is on cuda:" +
               std::to_string(device));
    if (t.numel() < numel)
        refuse(std::string(what) + ": " + std::to_string(t.numel()) + " elements, at least " + std::to_string(numel) +
               " needed");
    return t.data_ptr();
}
void *typed_on(PyObject *o, const char *what, int64_t numel, at::ScalarType type, int64_t device) {
    if (o == Py_None) return nullptr;
    const at::Tensor &t = tensor(o, what);
    if (t.scalar_type() != type)
        refuse(std::string(what) + ": " + type_name(t.scalar_type()) + ", expected " + c10::toString(type));
    return address(t, what, numel, device);
}
void *bytes_on(PyObject *o, const char *what, int64_t n, int64_t device) {
    if (o == Py_None) return nullptr;
    const at::Tensor &t = tensor(o, what);
    if (t.element_size() != 1)
        refuse(std::string(what) + ": " + std::to_string(t.element_size()) + "-byte elements, expected 1");
    return address(t, what, n, device);
}
amp_dtype elem(const at::Tensor &t, const char *what) {
    switch (t.scalar_type()) {
    case at::kFloat: return AMP_DT_F32;
    case at::kHalf: return AMP_DT_F16;
    case at::kBFloat16: return AMP_DT_BF16;
    default: refuse(std::string(what) + ": " + type_name(t.scalar_type()) + "; f32, f16 or bf16 is needed");
    }
}

// The matrix that gives a call its shape (the last dimension are its columns) and
// its device.
struct Matrix {
    const at::Tensor &t;
    const char *what;
    int64_t rows = 1, cols, device;
    amp_dtype type;
    Matrix(PyObject *o, const char *what_) : t(tensor(o, what_)), what(what_) {
        const auto s = t.sizes();
        if (s.empty()) refuse(std::string(what) + ": needs at least one dimension");
        cols = s.back();
        for (size_t i = 0; i + 1 < s.size(); ++i) rows *= s[i];
        type = elem(t, what);
        device = t.is_cuda() ? t.get_device() : -1;
    }
    void *p() const { return address(t, what, 0, device); }
    // the call's other tensors (None: NULL): of at least n elements of a type, or of
    // bytes; of the same type and at least its size
    void *typed(PyObject *o, const char *what, int64_t n, at::ScalarType of) const {
        return typed_on(o, what, n, of, device);
    }
    void *bytes(PyObject *o, const char *what, int64_t n) const { return bytes_on(o, what, n, device); }
    void *like(PyObject *o, const char *what) const { return typed(o, what, rows * cols, t.scalar_type()); }
};

int64_t up(int64_t v, int64_t step) { return (v + step - 1) / step; }
int64_t fp4_bytes(int64_t rows, int64_t cols) { return rows * up(cols, 32) * 16; }
int64_t fp4_scales(int64_t rows, int64_t cols) { return up(rows, 128) * up(cols, 128) * 512; }

// An 8-bit checkpoint (q, scales) or None.
struct Saved {
    void *q = nullptr, *s = nullptr;
    Saved(PyObject *o, const char *what, const Matrix &m) {
        if (o == Py_None) return;
        if (!PyTuple_Check(o) || PyTuple_GET_SIZE(o) != 2) refuse(std::string(what) + ": needs (q, scales)");
        q = m.typed(PyTuple_GET_ITEM(o, 0), what, m.rows * m.cols, at::kFloat8_e4m3fn);
        s = m.typed(PyTuple_GET_ITEM(o, 1), what, m.rows * up(m.cols, 32), at::kByte);
    }
};

// Makes a device current for a call (at no cost where it is).
struct OnDevice {
    c10::cuda::OptionalCUDAGuard guard;
    explicit OnDevice(int64_t device) {
        const auto d = static_cast<c10::DeviceIndex>(device);
        if (c10::cuda::current_device() != d) guard.set_index(d);
    }
};

// A stream object or handle; None: the current device's current stream.
amp_stream_t stream_of(PyObject *o) {
    if (o == Py_None) return c10::cuda::getCurrentCUDAStream().stream();
    PyObject *h = PyObject_HasAttrString(o, "cuda_stream") ? PyObject_GetAttrString(o, "cuda_stream") : PyNumber_Long(o);
    void *p = h ? PyLong_AsVoidPtr(h) : nullptr;
    Py_XDECREF(h);
    if (PyErr_Occurred()) {
        PyErr_Clear();
        refuse("stream: needs a stream or its handle");
    }
    return static_cast<amp_stream_t>(p);
}

// The common element type of the parameters and their gradients, each of `cols`
// elements (None ones aside; f32 if none is given).
struct Params {
    amp_dtype type = AMP_DT_F32;
    void *p[3] = {nullptr, nullptr, nullptr};
    Params(const Matrix &m, std::initializer_list<PyObject *> given) {
        const int64_t cols = m.cols;
        const at::Tensor *first = nullptr;
        int i = 0;
        for (PyObject *o : given) {
            if (o != Py_None) {
                const at::Tensor &t = tensor(o, "weight");
                if (first && t.scalar_type() != first->scalar_type())
                    refuse("weight, bias and their gradients need one dtype");
                if (t.numel() != cols)
                    refuse("weight, bias and their gradients need " + std::to_string(cols) + " elements");
                if (!first) {
                    first = &t;
                    type = elem(t, "weight");
                }
            }
        }
        for (PyObject *o : given) {
            if (o != Py_None) p[i] = address(tensor(o, "weight"), "weight", cols, m.device);
            ++i;
        }
    }
};

amp_act act_of(PyObject *o) {
    const char *s = PyUnicode_Check(o) ? PyUnicode_AsUTF8(o) : nullptr;
    if (s && !std::strcmp(s, "gelu")) return AMP_ACT_GELU;
    if (s && !std::strcmp(s, "gelu_tanh")) return AMP_ACT_GELU_TANH;
    if (s && !std::strcmp(s, "silu")) return AMP_ACT_SILU;
    PyErr_Clear();
    refuse(std::string("activation '") + (s ? s : "?") + "'; one of ['gelu', 'gelu_tanh', 'silu']");
}
double number(PyObject *o, const char *what) {
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred()) {
        PyErr_Clear();
        refuse(std::string(what) + ": needs a number");
    }
    return v;
}

// Runs one call: turns refusals and C++ exceptions into Python's, and lets other
// threads run while the entry point is in the driver.
template <class F>
PyObject *call(Py_ssize_t n, Py_ssize_t want, bool ready, F body) {
    if (n != want || !ready) {
        PyErr_SetString(PyExc_TypeError, ready ? "wrong number of arguments" : "the library is not loaded");
        return nullptr;
    }
    try {
        return PyLong_FromLong(body());
    } catch (const Refused &r) {
        PyErr_SetString(PyExc_ValueError, r.why.c_str());
    } catch (const std::exception &e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
    }
    return nullptr;
}
struct Unlocked {
    PyThreadState *s = PyEval_SaveThread();
    ~Unlocked() { PyEval_RestoreThread(s); }
};

using Args = PyObject *const *;

PyObject *quant(PyObject *, Args a, Py_ssize_t n) {  // x, q, scales, qt, scales_t, skip_if, stream
    return call(n, 7, g.quant, [&]() {
        const Matrix x(a[0], "x");
        const void *p = x.p();
        void *q = x.bytes(a[1], "q", fp4_bytes(x.rows, x.cols));
        void *s = x.bytes(a[2], "scales", fp4_scales(x.rows, x.cols));
        void *qt = x.bytes(a[3], "qt", fp4_bytes(x.cols, x.rows));
        void *st = x.bytes(a[4], "scales_t", fp4_scales(x.cols, x.rows));
        const auto *skip = static_cast<const int32_t *>(x.typed(a[5], "skip_if", 1, at::kInt));
        const OnDevice on(x.device);
        const amp_stream_t stream = stream_of(a[6]);
        Unlocked u;
        return g.quant(p, x.type, x.rows, x.cols, q, s, qt, st, skip, stream);
    });
}
PyObject *dequant(PyObject *, Args a, Py_ssize_t n) {  // q, scales, out, stream
    return call(n, 4, g.dequant, [&]() {
        const Matrix o(a[2], "out");
        void *out = o.p();
        void *q = o.bytes(a[0], "q", fp4_bytes(o.rows, o.cols));
        void *s = o.bytes(a[1], "scales", fp4_scales(o.rows, o.cols));
        const OnDevice on(o.device);
        const amp_stream_t stream = stream_of(a[3]);
        Unlocked u;
        return g.dequant(q, s, o.rows, o.cols, out, o.type, stream);
    });
}
PyObject *product(PyObject *, Args a, Py_ssize_t n) {  // a, a_scales, b, b_scales, k, out, stream
    return call(n, 7, g.product, [&]() {
        const int64_t k = PyLong_Check(a[4]) ? PyLong_AsLongLong(a[4]) : -1;
        if (k < 0 || k > (int64_t(1) << 32)) {  // sizes below are formed in 64 bits
            PyErr_Clear();
            PyObject *s = PyObject_Str(a[4]);
            const char *c = s ? PyUnicode_AsUTF8(s) : nullptr;
            const std::string why = std::string("k = ") + (c ? c : "?");
            Py_XDECREF(s);
            PyErr_Clear();
            refuse(why);
        }
        const Matrix o(a[5], "out");
        void *out = o.p();
        void *pa = o.bytes(a[0], "a", fp4_bytes(o.rows, k)), *sa = o.bytes(a[1], "a_scales", fp4_scales(o.rows, k));
        void *pb = o.bytes(a[2], "b", fp4_bytes(o.cols, k)), *sb = o.bytes(a[3], "b_scales", fp4_scales(o.cols, k));
        const OnDevice on(o.device);
        const amp_stream_t stream = stream_of(a[6]);
        Unlocked u;
        return g.product(pa, sa, pb, sb, o.rows, o.cols, k, out, o.type, stream);
    });
}
PyObject *norm_forward(PyObject *, Args a, Py_ssize_t n) {  // x, weight, bias, eps, y, mean, rstd, saved, stream
    return call(n, 9, g.norm_forward, [&]() {
        const Matrix x(a[0], "x");
        const Params w(x, {a[1], a[2]});
        const double eps = number(a[3], "eps");
        const void *p = x.p();
        void *y = x.like(a[4], "y");
        auto *mean = static_cast<float *>(x.typed(a[5], "mean", x.rows, at::kFloat));
        auto *rstd = static_cast<float *>(x.typed(a[6], "rstd", x.rows, at::kFloat));
        const Saved c(a[7], "saved", x);
        const OnDevice on(x.device);
        const amp_stream_t stream = stream_of(a[8]);
        Unlocked u;
        return g.norm_forward(p, x.type, x.rows, x.cols, w.p[0], w.p[1], w.type, eps, y, mean, rstd, c.q, c.s, stream);
    });
}
// dy, x, weight, mean, rstd, dx, dweight, dbias, workspace, saved, stream
PyObject *norm_backward(PyObject *, Args a, Py_ssize_t n) {
    return call(n, 11, g.norm_backward, [&]() {
        const Matrix dy(a[0], "dy");
        if ((a[1] == Py_None) == (a[9] == Py_None)) refuse("either x or saved");
        const Params w(dy, {a[2], a[6], a[7]});
        const void *p = dy.p(), *x = dy.like(a[1], "x");
        const auto *mean = static_cast<const float *>(dy.typed(a[3], "mean", dy.rows, at::kFloat));
        const auto *rstd = static_cast<const float *>(dy.typed(a[4], "rstd", dy.rows, at::kFloat));
        void *dx = dy.like(a[5], "dx"), *work = nullptr;
        int64_t room = 0;
        if (a[8] != Py_None) {
            const at::Tensor &t = tensor(a[8], "workspace");
            work = address(t, "workspace", 0, dy.device);
            room = t.numel() * t.element_size();
        }
        const Saved c(a[9], "saved", dy);
        const OnDevice on(dy.device);
        const amp_stream_t stream = stream_of(a[10]);
        Unlocked u;
        return g.norm_backward(p, x, dy.type, c.q, c.s, dy.rows, dy.cols, w.p[0], w.type, mean, rstd, dx, w.p[1],
                               w.p[2], work, room, stream);
    });
}
PyObject *act_forward(PyObject *, Args a, Py_ssize_t n) {  // x, kind, y, saved, up, saved_up, stream
    return call(n, 7, g.act_forward, [&]() {
        const amp_act act = act_of(a[1]);
        const Matrix x(a[0], "x");
        const void *p = x.p();
        void *y = x.like(a[2], "y"), *up_ = x.like(a[4], "up");
        const Saved c(a[3], "saved", x), cu(a[5], "saved_up", x);
        const OnDevice on(x.device);
        const amp_stream_t stream = stream_of(a[6]);
        Unlocked u;
        return g.act_forward(act, p, up_, x.type, x.rows, x.cols, y, c.q, c.s, cu.q, cu.s, stream);
    });
}
PyObject *act_backward(PyObject *, Args a, Py_ssize_t n) {  // dy, kind, saved, dx, saved_up, dup, stream
    return call(n, 7, g.act_backward, [&]() {
        const amp_act act = act_of(a[1]);
        const Matrix dy(a[0], "dy");
        const void *p = dy.p();
        const Saved c(a[2], "saved", dy), cu(a[4], "saved_up", dy);
        void *dx = dy.like(a[3], "dx"), *du = dy.like(a[5], "dup");
        const OnDevice on(dy.device);
        const amp_stream_t stream = stream_of(a[6]);
        Unlocked u;
        return g.act_backward(act, p, dy.type, dy.rows, dy.cols, c.q, c.s, cu.q, cu.s, dx, du, stream);
    });
}
PyObject *save(PyObject *, Args a, Py_ssize_t n) {  // x, q, scales, stream
    return call(n, 4, g.save, [&]() {
        const Matrix x(a[0], "x");
        const void *p = x.p();
        void *q = x.typed(a[1], "q", x.rows * x.cols, at::kFloat8_e4m3fn);
        void *s = x.typed(a[2], "scales", x.rows * up(x.cols, 32), at::kByte);
        const OnDevice on(x.device);
        const amp_stream_t stream = stream_of(a[3]);
        Unlocked u;
        return g.save(p, x.type, x.rows, x.cols, q, s, stream);
    });
}
PyObject *restore(PyObject *, Args a, Py_ssize_t n) {  // q, scales, out, stream
    return call(n, 4, g.restore, [&]() {
        const Matrix o(a[2], "out");
        void *out = o.p();
        void *q = o.typed(a[0], "q", o.rows * o.cols, at::kFloat8_e4m3fn);
        void *s = o.typed(a[1], "scales", o.rows * up(o.cols, 32), at::kByte);
        const OnDevice on(o.device);
        const amp_stream_t stream = stream_of(a[3]);
        Unlocked u;
        return g.restore(q, s, o.rows, o.cols, out, o.type, stream);
    });
}

// bind(addresses of the nine entry points, in the order of Entries)
PyObject *bind(PyObject *, Args a, Py_ssize_t n) {
    void *p[9];
    static_assert(sizeof(p) == sizeof(Entries), "entries");
    if (n != 9) {
        PyErr_SetString(PyExc_TypeError, "nine addresses");
        return nullptr;
    }
    for (int i = 0; i < 9; ++i) {
        p[i] = PyLong_AsVoidPtr(a[i]);
        if (PyErr_Occurred()) return nullptr;
    }
    std::memcpy(&g, p, sizeof p);
    Py_RETURN_NONE;
}

#define METHOD(name) \
    { #name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)(void)>(name)), METH_FASTCALL, nullptr }
PyMethodDef methods[] = {METHOD(bind), METHOD(quant), METHOD(dequant), METHOD(product), METHOD(norm_forward),
                         METHOD(norm_backward), METHOD(act_forward), METHOD(act_backward), METHOD(save),
                         METHOD(restore), {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_ops_bind", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__ops_bind(void) { return PyModule_Create(&module); }
