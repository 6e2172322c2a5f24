// seq_bind.cpp -- the part of the Python binding of the sequence operators that every call goes through: what
// a call's checks depend on as one key, its outputs, and the call itself.  A call of one token takes the device
// 5 us, and reading its tensors' shapes and strides in Python, looking a plan up by them and passing
// twenty arguments through ctypes took the host 7.
//
// The checks themselves are in _sequence.py: it makes a plan once for each key and keeps it.  Nothing here is kept from call to
// call.
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <ATen/ops/empty.h>

#include <cstdint>
#include <cstring>
#include <vector>

#include "dwseq.h"

namespace {

const at::Tensor *tensor(PyObject *o) {
    if (!THPVariable_Check(o)) {
        PyErr_Format(PyExc_TypeError, "expected a tensor, not %s", Py_TYPE(o)->tp_name);
        return nullptr;
    }
    const at::Tensor &t = THPVariable_Unpack(o);
    if (t.is_neg()) {  // its memory holds the values before torch negates them
        PyErr_SetString(PyExc_TypeError, "a tensor is negated lazily; call its resolve_neg()");
        return nullptr;
    }
    return &t;
}

// C++ exceptions end here as the Python ones that torch makes of them: no memory for an output is its OutOfMemoryError.
template <typename F> PyObject *guarded(F f) {
    HANDLE_TH_ERRORS
    return f();
    END_HANDLE_TH_ERRORS
}

// key(*tensors or None) -> bytes: shapes, strides, types and devices.
PyObject *key(PyObject *, PyObject *const *args, Py_ssize_t n) {
    return guarded([&]() -> PyObject * {
        std::vector<int64_t> k;
        k.reserve(12 * n);
        for (Py_ssize_t i = 0; i < n; ++i) {
            if (args[i] == Py_None) {
                k.push_back(-1);
                continue;
            }
            const at::Tensor *t = tensor(args[i]);
            if (!t) return nullptr;
            if (t->layout() != at::kStrided) {
                PyErr_SetString(PyExc_TypeError, "tensors must be dense");
                return nullptr;
            }
            const at::Device d = t->device();
            k.push_back(t->dim() | int64_t(t->scalar_type()) << 16 | int64_t(d.type()) << 32 | int64_t(d.index() + 1) << 48);
            for (int64_t s : t->sizes()) k.push_back(s);
            for (int64_t s : t->strides()) k.push_back(s);
        }
        return PyBytes_FromStringAndSize(reinterpret_cast<const char *>(k.data()), k.size() * sizeof(int64_t));
    });
}

at::ScalarType type_of(int64_t code) {
    switch (code) {
        case DW_F32: return at::kFloat;
        case DW_F16: return at::kHalf;
        case DW_BF16: return at::kBFloat16;
        case 3: return at::kChar;
        default: return at::kByte;
    }
}

// empty(forms, like) -> tuple of contiguous tensors on like's device.  forms: bytes of int64, for each tensor its
// type's code, dimensions and sizes.
PyObject *empty(PyObject *, PyObject *const *args, Py_ssize_t n) {
    return guarded([&]() -> PyObject * {
        if (n != 2 || !PyBytes_Check(args[0])) {
            PyErr_SetString(PyExc_TypeError, "empty(forms, like)");
            return nullptr;
        }
        const at::Tensor *like = tensor(args[1]);
        if (!like) return nullptr;
        const Py_ssize_t words = PyBytes_GET_SIZE(args[0]) / Py_ssize_t(sizeof(int64_t));
        std::vector<int64_t> f(words);
        std::memcpy(f.data(), PyBytes_AS_STRING(args[0]), words * sizeof(int64_t));
        const at::TensorOptions options = at::TensorOptions().device(like->device());
        std::vector<at::Tensor> made;
        for (Py_ssize_t i = 0; i + 1 < words && f[i + 1] >= 0 && i + 2 + f[i + 1] <= words; i += 2 + f[i + 1])
            made.push_back(at::empty(at::IntArrayRef(f.data() + i + 2, f[i + 1]), options.dtype(type_of(f[i]))));
        PyObject *out = PyTuple_New(made.size());
        if (!out) return nullptr;
        for (size_t i = 0; i < made.size(); ++i) {
            PyObject *t = THPVariable_Wrap(std::move(made[i]));
            if (!t) {
                Py_DECREF(out);
                return nullptr;
            }
            PyTuple_SET_ITEM(out, i, t);
        }
        return out;
    });
}

// A call's arguments: (numbers, tensors or None ..., number, stream).
struct Call {
    PyObject *const *args;
    Py_ssize_t tensors;
    int64_t numbers[32] = {};
    double last = 0;
    void *stream = nullptr;
    bool read(PyObject *const *a, Py_ssize_t n, Py_ssize_t want) {
        args = a + 1;
        tensors = want;
        if (n != want + 3 || !PyBytes_Check(a[0]) || PyBytes_GET_SIZE(a[0]) > Py_ssize_t(sizeof(numbers))) {
            PyErr_SetString(PyExc_TypeError, "wrong arguments");
            return false;
        }
        std::memcpy(numbers, PyBytes_AS_STRING(a[0]), PyBytes_GET_SIZE(a[0]));
        for (Py_ssize_t i = 0; i < want; ++i)
            if (args[i] != Py_None && !tensor(args[i])) return false;
        last = PyFloat_AsDouble(a[n - 2]);
        stream = PyLong_AsVoidPtr(a[n - 1]);
        return !PyErr_Occurred();
    }
    template <typename T = void> const T *in(int i) const {
        return args[i] == Py_None ? nullptr : static_cast<const T *>(THPVariable_Unpack(args[i]).const_data_ptr());
    }
    // What the call writes has a new version, as after torch's own writes in place: autograd then finds a tensor that it
    // saved before (a state that a token was added to) changed.  Inference tensors have no versions.
    template <typename T = void> T *out(int i) const {
        if (args[i] == Py_None) return nullptr;
        const at::Tensor &t = THPVariable_Unpack(args[i]);
        if (!t.is_inference()) t.unsafeGetTensorImpl()->bump_version();
        return static_cast<T *>(t.mutable_data_ptr());
    }
    size_t bytes(int i) const { return args[i] == Py_None ? 0 : THPVariable_Unpack(args[i]).nbytes(); }
};
// The call without the interpreter's lock: a full queue makes a launch wait.
template <typename F> PyObject *finish(F f) {
    int rc;
    Py_BEGIN_ALLOW_THREADS
    rc = f();
    Py_END_ALLOW_THREADS
    return PyLong_FromLong(rc);
}

// q k v log_decay state lengths o state_out workspace
PyObject *attn_fwd(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded([&]() -> PyObject * {
        Call c;
        if (!c.read(a, n, 9)) return nullptr;
        const int64_t *s = c.numbers;
        const void *q = c.in(0), *k = c.in(1), *v = c.in(2);
        const float *g = c.in<float>(3), *z = c.in<float>(4);
        const int32_t *len = c.in<int32_t>(5);
        void *o = c.out(6), *ws = c.out(8);
        float *zo = c.out<float>(7);
        const size_t bytes = c.bytes(8);
        return finish([&] {
            return decayattn_fwd(q, k, v, g, z, len, o, zo, ws, bytes, s[0], s[1], s[2], s[3], s[4], s[5], s[6], s[7], s + 9,
                                 float(c.last), int(s[8]), c.stream);
        });
    });
}

// q k v log_decay do state lengths dstate_out dq dk dv dstate workspace
PyObject *attn_bwd(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded([&]() -> PyObject * {
        Call c;
        if (!c.read(a, n, 13)) return nullptr;
        const int64_t *s = c.numbers;
        const void *q = c.in(0), *k = c.in(1), *v = c.in(2), *d = c.in(4);
        const float *g = c.in<float>(3), *z = c.in<float>(5), *dz = c.in<float>(7);
        const int32_t *len = c.in<int32_t>(6);
        void *dq = c.out(8), *dk = c.out(9), *dv = c.out(10), *ws = c.out(12);
        float *ds = c.out<float>(11);
        const size_t bytes = c.bytes(12);
        return finish([&] {
            return decayattn_bwd(q, k, v, g, d, z, len, dz, dq, dk, dv, ds, ws, bytes, s[0], s[1], s[2], s[3], s[4], s[5], s[6],
                                 s[7], s + 9, float(c.last), int(s[8]), c.stream);
        });
    });
}

// q k v log_decay state o
PyObject *attn_step(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded([&]() -> PyObject * {
        Call c;
        if (!c.read(a, n, 6)) return nullptr;
        const int64_t *s = c.numbers;
        const void *q = c.in(0), *k = c.in(1), *v = c.in(2);
        const float *g = c.in<float>(3);
        float *z = c.out<float>(4);
        void *o = c.out(5);
        return finish([&] {
            return decayattn_step(q, k, v, g, z, o, s[0], s[1], s[2], s[3], s[4], s[5], s[6], s + 9, s[7], float(c.last),
                                  int(s[8]), c.stream);
        });
    });
}

// x codes exps
PyObject *pack(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded([&]() -> PyObject * {
        Call c;
        if (!c.read(a, n, 3)) return nullptr;
        const int64_t *s = c.numbers;
        const void *x = c.in(0);
        int8_t *q = c.out<int8_t>(1), *e = c.out<int8_t>(2);
        return finish([&] { return act8_pack(x, q, e, s[0], s[1], int(s[2]), c.stream); });
    });
}

// codes exps y
PyObject *unpack(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded([&]() -> PyObject * {
        Call c;
        if (!c.read(a, n, 3)) return nullptr;
        const int64_t *s = c.numbers;
        const int8_t *q = c.in<int8_t>(0), *e = c.in<int8_t>(1);
        void *y = c.out(2);
        return finish([&] { return act8_unpack(q, e, y, s[0], s[1], int(s[2]), c.stream); });
    });
}

// x gamma beta y mean rstd codes exps workspace
PyObject *norm_fwd(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded([&]() -> PyObject * {
        Call c;
        if (!c.read(a, n, 9)) return nullptr;
        const int64_t *s = c.numbers;
        const void *x = c.in(0), *g = c.in(1), *b = c.in(2);
        void *y = c.out(3), *ws = c.out(8);
        float *m = c.out<float>(4), *r = c.out<float>(5);
        int8_t *q = c.out<int8_t>(6), *e = c.out<int8_t>(7);
        const size_t bytes = c.bytes(8);
        return finish([&] {
            return groupnorm_act_fwd(x, g, b, y, m, r, q, e, ws, bytes, s[0], s[1], s[2], s[3], float(c.last), int(s[4]),
                                     int(s[5]), c.stream);
        });
    });
}

// dy x codes exps mean rstd gamma beta dx dgamma dbeta workspace
PyObject *norm_bwd(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded([&]() -> PyObject * {
        Call c;
        if (!c.read(a, n, 12)) return nullptr;
        const int64_t *s = c.numbers;
        const void *dy = c.in(0), *x = c.in(1), *g = c.in(6), *b = c.in(7);
        const int8_t *q = c.in<int8_t>(2), *e = c.in<int8_t>(3);
        const float *m = c.in<float>(4), *r = c.in<float>(5);
        void *dx = c.out(8), *dg = c.out(9), *db = c.out(10), *ws = c.out(11);
        const size_t bytes = c.bytes(11);
        return finish([&] {
            return groupnorm_act_bwd(dy, x, q, e, m, r, g, b, dx, dg, db, ws, bytes, s[0], s[1], s[2], s[3], int(s[4]),
                                     int(s[5]), c.stream);
        });
    });
}

#define ENTRY(name) {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(name)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {ENTRY(key),  ENTRY(empty),    ENTRY(attn_fwd), ENTRY(attn_bwd),          ENTRY(attn_step), ENTRY(pack),
                         ENTRY(unpack), ENTRY(norm_fwd), ENTRY(norm_bwd), {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_seqbind", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__seqbind() { return PyModule_Create(&module); }
