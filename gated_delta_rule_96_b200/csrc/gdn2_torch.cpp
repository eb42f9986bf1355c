// The binding's native half: argument checks and marshalling of torch tensors into the C ABI of libgdn2
// (include/gdn2.h), for the calls whose kernels take a few microseconds.  A call through ctypes with a dozen
// tensors costs 20 to 30 us on the host, most of it attribute reads and argument conversions; here it is one.
//
// A CPython module without state but the library's entry points and the package's error class, both set by
// bind().  Every function checks its tensors' types, shapes, layout and device, makes their device current for
// the call and launches on the given stream or that device's current one.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/cuda/EmptyTensor.h>
#include <ATen/ops/empty.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <dlfcn.h>
#include <torch/csrc/autograd/python_variable.h>

#include <string>
#include <vector>

#include "gdn2.h"

namespace {

PyObject *g_error = nullptr;   // the package's GDN2Error

struct Library {
    decltype(&gdn2_gated_norm_fwd) gated_norm_fwd;
    decltype(&gdn2_gated_norm_bwd) gated_norm_bwd;
    decltype(&gdn2_add_norm_fwd) add_norm_fwd;
    decltype(&gdn2_add_norm_bwd) add_norm_bwd;
    decltype(&gdn2_tree_fwd) tree_fwd;
    decltype(&gdn2_recurrent_fwd) recurrent_fwd;
    decltype(&gdn2_state_copy) state_copy;
} lib;

// A refusal on its way to Python: the exception's class and text, or (type null) one that is already set.
struct Refusal {
    PyObject *type;
    std::string text;
};

std::string show(at::IntArrayRef shape) {
    std::string s = "(";
    for (size_t i = 0; i < shape.size(); ++i) s += (i ? ", " : "") + std::to_string(shape[i]);
    return s + (shape.size() == 1 ? ",)" : ")");
}

const char *show(at::ScalarType t) {
    switch (t) {
        case at::kFloat: return "float32";
        case at::kBFloat16: return "bfloat16";
        case at::kInt: return "int32";
        case at::kByte: return "uint8";
        default: return c10::toString(t);
    }
}

const at::Tensor &tensor(const char *name, PyObject *o) {
    if (!THPVariable_Check(o)) throw Refusal{PyExc_TypeError, std::string(name) + " must be a tensor"};
    return THPVariable_Unpack(o);
}

long long attribute(PyObject *o, const char *name) {
    PyObject *x = PyObject_GetAttrString(o, name);
    if (!x) throw Refusal{nullptr, ""};
    const long long v = PyLong_AsLongLong(x);
    Py_DECREF(x);
    if (v == -1 && PyErr_Occurred()) throw Refusal{nullptr, ""};
    return v;
}

// a torch.cuda.Stream
c10::cuda::CUDAStream stream_of(PyObject *o) {
    return c10::cuda::CUDAStream::unpack3(attribute(o, "stream_id"), (c10::DeviceIndex)attribute(o, "device_index"),
                                          (c10::DeviceType)attribute(o, "device_type"));
}

// The tensors of one call.  Types and shapes are checked as they come, layout and device once all are there:
// contiguous CUDA tensors on one device.
struct Call {
    struct Used {
        const char *name;
        const at::Tensor *t;
        bool contiguous;
    } used[20];
    int count = 0;

    void add(const char *name, const at::Tensor &t, bool contiguous = true) { used[count++] = {name, &t, contiguous}; }
    c10::Device device() const {
        const c10::Device d = used[0].t->device();
        for (int i = 0; i < count; ++i) {
            const Used &u = used[i];
            if (!u.t->is_cuda()) throw Refusal{PyExc_ValueError, std::string(u.name) + ": all tensors must be CUDA tensors (no CPU path)"};
            if (u.contiguous && !u.t->is_contiguous())
                throw Refusal{PyExc_ValueError, std::string(u.name) + ": all tensors must be contiguous"};
            if (u.t->device() != d)
                throw Refusal{PyExc_ValueError, std::string(u.name) + ": all tensors must be on one device (cuda:" + std::to_string(d.index()) +
                                                    " and cuda:" + std::to_string(u.t->device().index()) + " given)"};
        }
        return d;
    }
    // a tensor that must have this type and shape; None gives null where it may
    void *use(const char *name, PyObject *o, at::ScalarType type, at::IntArrayRef shape, bool optional = false) {
        if (optional && o == Py_None) return nullptr;
        const at::Tensor &t = tensor(name, o);
        if (t.scalar_type() != type)
            throw Refusal{PyExc_TypeError, std::string(name) + " must be " + show(type) + ", got " + show(t.scalar_type())};
        if (t.sizes() != shape)
            throw Refusal{PyExc_ValueError, std::string(name) + " has shape " + show(t.sizes()) + ", expected " + show(shape)};
        add(name, t);
        return t.data_ptr();
    }
    // the tensor that sets the token type
    void *tokens(const char *name, PyObject *o, int dims, int *code) {
        const at::Tensor &t = tensor(name, o);
        if (t.scalar_type() == at::kBFloat16) *code = GDN2_BF16;
        else if (t.scalar_type() == at::kFloat) *code = GDN2_F32;
        else throw Refusal{PyExc_TypeError, std::string("token tensors must be bfloat16 or float32, got ") + show(t.scalar_type())};
        if (dims ? t.dim() != dims : t.dim() < 1)
            throw Refusal{PyExc_ValueError, std::string(name) + " has shape " + show(t.sizes()) + ", expected " +
                                                (dims ? std::to_string(dims) + " dimensions" : "at least one dimension")};
        add(name, t);
        return t.data_ptr();
    }
    void *workspace(PyObject *o, size_t *bytes) {
        const at::Tensor &t = tensor("workspace", o);
        add("workspace", t);
        *bytes = t.nbytes();
        return t.data_ptr();
    }
    // one-dimensional int32 indices
    const int *index(const char *name, PyObject *o, long long *n, bool optional = false) {
        if (optional && o == Py_None) return nullptr;
        const at::Tensor &t = tensor(name, o);
        if (t.scalar_type() != at::kInt || t.dim() != 1)
            throw Refusal{PyExc_TypeError, std::string(name) + " must be a one-dimensional int32 tensor"};
        if (*n >= 0 && t.size(0) != *n)
            throw Refusal{PyExc_ValueError, std::string(name) + " has shape " + show(t.sizes()) + ", expected (" + std::to_string(*n) + ",)"};
        *n = t.size(0);
        add(name, t);
        return static_cast<const int *>(t.data_ptr());
    }
    // a state cache [slots, ...]: every slot contiguous, the slots any distance apart that keeps them apart
    float *pool(const char *name, PyObject *o, at::IntArrayRef slot, long long *stride, int *slots) {
        const at::Tensor &t = tensor(name, o);
        if (t.scalar_type() != at::kFloat) throw Refusal{PyExc_TypeError, std::string(name) + " must be float32"};
        if (t.dim() < 2 || t.sizes().slice(1) != slot)
            throw Refusal{PyExc_ValueError, std::string(name) + " has shape " + show(t.sizes()) + ", expected slots of " + show(slot)};
        add(name, t, false);
        long long floats = 1;
        for (int64_t d = t.dim() - 1; d > 0; --d) {
            if (t.size(d) != 1 && t.stride(d) != floats && t.numel() > 0)
                throw Refusal{PyExc_ValueError, std::string(name) + ": each slot of the state cache must be contiguous"};
            floats *= t.size(d);
        }
        if (t.size(0) > 1 && floats > 0 && t.stride(0) < floats)
            throw Refusal{PyExc_ValueError, std::string(name) + ": slots of the state cache must not overlap"};
        *stride = t.size(0) > 1 && floats > 0 ? t.stride(0) : floats;
        if (t.size(0) > INT32_MAX) throw Refusal{PyExc_ValueError, std::string(name) + " has too many slots"};
        *slots = (int)t.size(0);
        return static_cast<float *>(t.data_ptr());
    }
    // the call itself, on `stream` or the device's current one, with the device current and the interpreter free
    template <typename F>
    void run(const char *where, PyObject *stream, F launch) const {
        const c10::Device d = device();
        void *st;
        if (stream == Py_None) {
            st = c10::cuda::getCurrentCUDAStream(d.index()).stream();
        } else {
            const c10::cuda::CUDAStream s = stream_of(stream);
            if (s.device_index() != d.index())
                throw Refusal{PyExc_ValueError, "the stream is of cuda:" + std::to_string(s.device_index()) +
                                                    ", the tensors are on cuda:" + std::to_string(d.index())};
            st = s.stream();
        }
        int rc;
        {
            const c10::cuda::CUDAGuard guard(d);
            PyThreadState *state = PyEval_SaveThread();
            rc = launch(st);
            PyEval_RestoreThread(state);
        }
        if (rc != GDN2_OK) {
            PyObject *e = PyObject_CallFunction(g_error, "is", rc, where);
            if (e) {
                PyErr_SetObject(g_error, e);
                Py_DECREF(e);
            }
            throw Refusal{nullptr, ""};
        }
    }
};

double number(PyObject *o) {
    const double x = PyFloat_AsDouble(o);
    if (x == -1.0 && PyErr_Occurred()) throw Refusal{nullptr, ""};
    return x;
}

long long whole(PyObject *o) {
    const long long x = PyLong_AsLongLong(o);
    if (x == -1 && PyErr_Occurred()) throw Refusal{nullptr, ""};
    return x;
}

int to_int(const char *name, long long x) {
    if (x < INT32_MIN || x > INT32_MAX) throw Refusal{PyExc_ValueError, std::string(name) + " is out of range"};
    return (int)x;
}

// o if it is a tensor; where it is None a new one of `shape`, like `like` otherwise, which `made` owns.  Its memory is
// the stream's that the call runs on.
PyObject *or_new(PyObject *o, at::IntArrayRef shape, const at::Tensor &like, PyObject *stream, std::vector<PyObject *> &made) {
    if (o != Py_None) return o;
    c10::cuda::OptionalCUDAStreamGuard guard;
    if (stream != Py_None) guard.reset_stream(stream_of(stream));
    // straight from the allocator: 0.2 us an output less than a dispatched at::empty
    made.push_back(THPVariable_Wrap(like.is_cuda() ? at::Tensor(at::detail::empty_cuda(shape, like.scalar_type(), like.device(), std::nullopt))
                                                   : at::empty(shape, like.options().requires_grad(false))));
    if (!made.back()) throw Refusal{nullptr, ""};
    return made.back();
}
PyObject *or_new(PyObject *o, const at::Tensor &like, PyObject *stream, std::vector<PyObject *> &made) {
    return or_new(o, like.sizes(), like, stream, made);
}

// what a function returns: nothing where the outputs were given, the new one, or a tuple of them
PyObject *result(std::vector<PyObject *> &made) {
    if (made.empty()) Py_RETURN_NONE;
    if (made.size() == 1) {
        PyObject *o = made[0];
        made.clear();
        return o;
    }
    PyObject *t = PyTuple_New((Py_ssize_t)made.size());
    if (!t) throw Refusal{nullptr, ""};
    for (size_t i = 0; i < made.size(); ++i) PyTuple_SET_ITEM(t, (Py_ssize_t)i, made[i]);
    made.clear();
    return t;
}

// Runs `body` with the arguments and turns whatever it throws into a Python error.
template <typename Body>
PyObject *guarded(PyObject *const *a, Py_ssize_t n, Py_ssize_t want, Body body) {
    std::vector<PyObject *> made;
    try {
        if (n != want) throw Refusal{PyExc_TypeError, "wrong number of arguments"};
        return body(a, made);
    } catch (const Refusal &r) {
        if (r.type) PyErr_SetString(r.type, r.text.c_str());
    } catch (const std::exception &e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
    } catch (...) {
        PyErr_SetString(PyExc_RuntimeError, "unknown error");
    }
    for (PyObject *o : made) Py_XDECREF(o);
    return nullptr;
}

long long rows_of(const at::Tensor &t) { return t.size(-1) ? t.numel() / t.size(-1) : 0; }

// o, gate, weight, y or None, act, eps, stream
PyObject *gated_norm_fwd(PyObject *, PyObject *const *args, Py_ssize_t n) {
    return guarded(args, n, 7, [](PyObject *const *a, std::vector<PyObject *> &made) {
        Call c;
        int dt;
        const void *o = c.tokens("o", a[0], 0, &dt);
        const at::Tensor &t = THPVariable_Unpack(a[0]);
        const void *gate = c.use("gate", a[1], t.scalar_type(), t.sizes());
        const void *weight = c.use("weight", a[2], at::kFloat, t.sizes().slice(t.dim() - 1));
        void *y = c.use("y", or_new(a[3], t, a[6], made), t.scalar_type(), t.sizes());
        const int act = to_int("act", whole(a[4])), width = to_int("d_v", t.size(-1));
        const float eps = (float)number(a[5]);
        c.run("gdn2_gated_norm_fwd", a[6], [&](void *st) {
            return lib.gated_norm_fwd(o, gate, static_cast<const float *>(weight), y, rows_of(t), width, act, eps, dt, st);
        });
        return result(made);
    });
}

// o, gate, weight, dy, do, dgate, dweight (all three or none), act, eps, workspace, stream
PyObject *gated_norm_bwd(PyObject *, PyObject *const *args, Py_ssize_t n) {
    return guarded(args, n, 11, [](PyObject *const *a, std::vector<PyObject *> &made) {
        Call c;
        int dt;
        const void *o = c.tokens("o", a[0], 0, &dt);
        const at::Tensor &t = THPVariable_Unpack(a[0]);
        const auto type = t.scalar_type();
        const auto shape = t.sizes(), last = shape.slice(t.dim() - 1);
        const void *gate = c.use("gate", a[1], type, shape);
        const void *weight = c.use("weight", a[2], at::kFloat, last);
        const void *dy = c.use("dy", a[3], type, shape);
        void *d_o = c.use("do", or_new(a[4], t, a[10], made), type, shape);
        void *dgate = c.use("dgate", or_new(a[5], t, a[10], made), type, shape);
        void *dweight = c.use("dweight", or_new(a[6], THPVariable_Unpack(a[2]), a[10], made), at::kFloat, last);
        const int act = to_int("act", whole(a[7])), width = to_int("d_v", t.size(-1));
        const float eps = (float)number(a[8]);
        size_t bytes;
        void *ws = c.workspace(a[9], &bytes);
        c.run("gdn2_gated_norm_bwd", a[10], [&](void *st) {
            return lib.gated_norm_bwd(o, gate, static_cast<const float *>(weight), dy, d_o, dgate, static_cast<float *>(dweight),
                                      rows_of(t), width, act, eps, dt, ws, bytes, st);
        });
        return result(made);
    });
}

// x, residual, scale, weight, h, y, allocate (y and h), eps, stream
PyObject *add_norm_fwd(PyObject *, PyObject *const *args, Py_ssize_t n) {
    return guarded(args, n, 9, [](PyObject *const *a, std::vector<PyObject *> &made) {
        Call c;
        int dt;
        const void *x = c.tokens("x", a[0], 0, &dt);
        const at::Tensor &t = THPVariable_Unpack(a[0]);
        const auto type = t.scalar_type();
        const auto shape = t.sizes(), last = shape.slice(t.dim() - 1);
        const void *residual = c.use("residual", a[1], type, shape, true);
        const void *scale = c.use("scale", a[2], at::kFloat, last, true);
        const void *weight = c.use("weight", a[3], at::kFloat, last);
        const bool allocate = PyObject_IsTrue(a[6]) == 1;
        void *y = c.use("y", allocate ? or_new(Py_None, t, a[8], made) : a[5], type, shape);
        void *h = c.use("h", allocate ? or_new(Py_None, t, a[8], made) : a[4], type, shape, true);
        const float eps = (float)number(a[7]);
        const int width = to_int("width", t.size(-1));
        c.run("gdn2_add_norm_fwd", a[8], [&](void *st) {
            return lib.add_norm_fwd(x, residual, static_cast<const float *>(scale), static_cast<const float *>(weight), h, y,
                                    rows_of(t), to_int("width", t.size(-1)), eps, dt, st);
        });
        return result(made);
    });
}

// h, x, scale, weight, dy, dh, dresidual, dx, dscale, dweight, eps, workspace, stream, allocate (the outputs: without a
// scale dresidual and dweight alone)
PyObject *add_norm_bwd(PyObject *, PyObject *const *args, Py_ssize_t n) {
    return guarded(args, n, 14, [](PyObject *const *a, std::vector<PyObject *> &made) {
        Call c;
        int dt;
        const void *h = c.tokens("h", a[0], 0, &dt);
        const at::Tensor &t = THPVariable_Unpack(a[0]);
        const auto type = t.scalar_type();
        const auto shape = t.sizes(), last = shape.slice(t.dim() - 1);
        const void *x = c.use("x", a[1], type, shape, true);
        const void *scale = c.use("scale", a[2], at::kFloat, last, true);
        const void *weight = c.use("weight", a[3], at::kFloat, last);
        const void *dy = c.use("dy", a[4], type, shape), *dh = c.use("dh", a[5], type, shape, true);
        const bool allocate = PyObject_IsTrue(a[13]) == 1, scaled = a[2] != Py_None;
        const at::Tensor &sums = THPVariable_Unpack(a[3]);   // what the column sums are like
        const auto out = [&](int i, const at::Tensor &like, bool wanted) {
            return allocate && wanted ? or_new(Py_None, like, a[12], made) : a[i];
        };
        void *dres = c.use("dresidual", out(6, t, true), type, shape), *dx = c.use("dx", out(7, t, scaled), type, shape, true);
        void *dscale = c.use("dscale", out(8, sums, scaled), at::kFloat, last, true);
        void *dweight = c.use("dweight", out(9, sums, true), at::kFloat, last);
        const float eps = (float)number(a[10]);
        const int width = to_int("width", t.size(-1));
        size_t bytes;
        void *ws = c.workspace(a[11], &bytes);
        c.run("gdn2_add_norm_bwd", a[12], [&](void *st) {
            return lib.add_norm_bwd(h, x, static_cast<const float *>(scale), static_cast<const float *>(weight), dy, dh, dres, dx,
                                    static_cast<float *>(dscale), static_cast<float *>(dweight), rows_of(t), width, eps, dt, ws, bytes, st);
        });
        return result(made);
    });
}

// the six token tensors of a call: q, k, b, alpha [rows, H, d_k], v, w [rows, H, d_v]
struct Tokens {
    const void *q, *k, *v, *b, *w;
    const float *alpha;
    int dt;
    int rows, H, K, V;
    at::ScalarType type;

    Tokens(Call &c, PyObject *const *a) {
        q = c.tokens("q", a[0], 3, &dt);
        const at::Tensor &t = THPVariable_Unpack(a[0]), &tv = tensor("v", a[2]);
        type = t.scalar_type();
        rows = to_int("rows", t.size(0)), H = to_int("H", t.size(1)), K = to_int("d_k", t.size(2));
        if (tv.dim() != 3) throw Refusal{PyExc_ValueError, "v has shape " + show(tv.sizes()) + ", expected 3 dimensions"};
        V = to_int("d_v", tv.size(2));
        k = c.use("k", a[1], type, {rows, H, K});
        v = c.use("v", a[2], type, {rows, H, V});
        alpha = static_cast<const float *>(c.use("alpha", a[3], at::kFloat, {rows, H, K}));
        b = c.use("b", a[4], type, {rows, H, K});
        w = c.use("w", a[5], type, {rows, H, V});
    }
};

// q, k, v, alpha, b, w, S, slots, cu_nodes, parents, o or None, max_nodes, workspace, stream
PyObject *tree_fwd(PyObject *, PyObject *const *args, Py_ssize_t n) {
    return guarded(args, n, 14, [](PyObject *const *a, std::vector<PyObject *> &made) {
        Call c;
        const Tokens x(c, a);
        long long batch = -1, stride;
        const int *slots = c.index("slots", a[7], &batch);
        long long ends = batch + 1, total = x.rows;
        const int *cu = c.index("cu_nodes", a[8], &ends), *parents = c.index("parents", a[9], &total);
        int num;
        const float *S = c.pool("S", a[6], {x.H, x.K, x.V}, &stride, &num);
        void *o = c.use("o", or_new(a[10], THPVariable_Unpack(a[2]), a[13], made), x.type, {x.rows, x.H, x.V});
        const int most = to_int("max_nodes", whole(a[11])), seqs = to_int("batch", batch);
        size_t bytes;
        void *ws = c.workspace(a[12], &bytes);
        c.run("gdn2_tree_fwd", a[13], [&](void *st) {
            return lib.tree_fwd(x.q, x.k, x.v, x.alpha, x.b, x.w, S, stride, num, slots, cu, parents, o, seqs, x.H, x.rows, most, x.K, x.V,
                                x.dt, ws, bytes, st);
        });
        return result(made);
    });
}

// q, k, v, alpha, b, w, S, slots_in, slots_out, cu_tokens, index, o, allocate, workspace, stream
PyObject *recurrent_fwd(PyObject *, PyObject *const *args, Py_ssize_t n) {
    return guarded(args, n, 15, [](PyObject *const *a, std::vector<PyObject *> &made) {
        Call c;
        const Tokens x(c, a);
        long long batch = -1, stride, total = -1;
        const int *in = c.index("slots_in", a[7], &batch), *out = c.index("slots_out", a[8], &batch);
        long long ends = batch + 1;
        const int *cu = c.index("cu_tokens", a[9], &ends), *index = c.index("index", a[10], &total, true);
        if (a[10] == Py_None) total = x.rows;
        int num;
        float *S = c.pool("S", a[6], {x.H, x.K, x.V}, &stride, &num);
        PyObject *given = a[11];
        if (PyObject_IsTrue(a[12]) == 1) given = or_new(Py_None, {total, x.H, x.V}, THPVariable_Unpack(a[2]), a[14], made);
        void *o = c.use("o", given, x.type, {total, x.H, x.V}, true);
        const int seqs = to_int("batch", batch), entries = to_int("entries", total);
        size_t bytes;
        void *ws = c.workspace(a[13], &bytes);
        c.run("gdn2_recurrent_fwd", a[14], [&](void *st) {
            return lib.recurrent_fwd(x.q, x.k, x.v, x.alpha, x.b, x.w, S, stride, num, in, out, cu, index, o, seqs, x.H, entries,
                                     x.rows, x.K, x.V, x.dt, ws, bytes, st);
        });
        return result(made);
    });
}

// dst, src, dst_index, src_index, workspace, stream
PyObject *state_copy(PyObject *, PyObject *const *args, Py_ssize_t n) {
    return guarded(args, n, 6, [](PyObject *const *a, std::vector<PyObject *> &made) {
        Call c;
        const at::Tensor &d = tensor("dst", a[0]);
        if (d.dim() < 2) throw Refusal{PyExc_ValueError, "dst has shape " + show(d.sizes()) + ", expected [slots, ...]"};
        const auto slot = d.sizes().slice(1);
        long long pairs = -1, ds, ss, floats = 1;
        int dn, sn;
        const int *di = c.index("dst_index", a[2], &pairs), *si = c.index("src_index", a[3], &pairs);
        float *dst = c.pool("dst", a[0], slot, &ds, &dn);
        const float *src = c.pool("src", a[1], slot, &ss, &sn);
        for (const int64_t x : slot) floats *= x;
        const int count = to_int("pairs", pairs);
        size_t bytes;
        void *ws = c.workspace(a[4], &bytes);
        c.run("gdn2_state_copy", a[5], [&](void *st) {
            return lib.state_copy(dst, ds, dn, src, ss, sn, di, si, count, floats, ws, bytes, st);
        });
        return result(made);
    });
}

// path of libgdn2.so, error class
PyObject *bind(PyObject *, PyObject *args) {
    const char *path;
    PyObject *error;
    if (!PyArg_ParseTuple(args, "sO", &path, &error)) return nullptr;
    void *so = dlopen(path, RTLD_NOW | RTLD_LOCAL);
    if (!so) return PyErr_Format(PyExc_RuntimeError, "%s", dlerror());
#define GDN2_BIND(name)                                                                    \
    if (!(lib.name = reinterpret_cast<decltype(lib.name)>(dlsym(so, "gdn2_" #name))))      \
        return PyErr_Format(PyExc_RuntimeError, "%s has no gdn2_" #name, path);
    GDN2_BIND(gated_norm_fwd)
    GDN2_BIND(gated_norm_bwd)
    GDN2_BIND(add_norm_fwd)
    GDN2_BIND(add_norm_bwd)
    GDN2_BIND(tree_fwd)
    GDN2_BIND(recurrent_fwd)
    GDN2_BIND(state_copy)
#undef GDN2_BIND
    Py_INCREF(error);
    Py_XSETREF(g_error, error);
    Py_RETURN_NONE;
}

#define GDN2_FAST(name) {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(name)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {{"bind", bind, METH_VARARGS, nullptr},
                         GDN2_FAST(gated_norm_fwd),
                         GDN2_FAST(gated_norm_bwd),
                         GDN2_FAST(add_norm_fwd),
                         GDN2_FAST(add_norm_bwd),
                         GDN2_FAST(tree_fwd),
                         GDN2_FAST(recurrent_fwd),
                         GDN2_FAST(state_copy),
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_gdn2_torch", "Marshalling of torch tensors into libgdn2.", -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__gdn2_torch() { return PyModule_Create(&module); }
