// native.cpp -- CPython binding of the gated delta and clipping entry points (the module `_native`): checks torch
// tensors, lays out their ttt_view's and calls libttt.so, without the microseconds that the same
// marshalling takes in Python.  A call returns the entry point's ttt_status; a tensor that does not fit raises
// ValueError before anything is called.  torch is used for reading its tensors' metadata only.
#include <torch/csrc/autograd/python_variable.h>

#include <algorithm>
#include <new>
#include <string>
#include <vector>

#include "ttt.h"

namespace {

struct Refused {
    std::string why;
};

[[noreturn]] void refuse(const char* name, const std::string& why) { throw Refused{std::string(name) + " " + why}; }

const at::Tensor& tensor(PyObject* o, const char* name) {
    if (!THPVariable_Check(o)) refuse(name, "must be a tensor");
    return THPVariable_Unpack(o);
}

std::string text(std::initializer_list<int64_t> dims) {
    std::string s = "[";
    for (int64_t d : dims) s += (s.size() > 1 ? ", " : "") + std::to_string(d);
    return s + "]";
}

struct Call {
    ttt_delta_shape shape{};
    at::ScalarType type{};
    c10::Device device{c10::kCPU};

    void start(const at::Tensor& Q, const at::Tensor& V) {
        if (Q.dim() != 4 || V.dim() != 4) throw Refused{"Q, K and V must be [B][heads][N][d]"};
        if (!Q.is_cuda()) throw Refused{"Q, K and V must be CUDA tensors"};
        type = Q.scalar_type();
        device = Q.device();
        if (type == at::kBFloat16) shape.dtype = TTT_BF16;
        else if (type == at::kFloat) shape.dtype = TTT_FP32;
        else throw Refused{"Q, K and V must be bfloat16 or float32"};
        for (int64_t n : {Q.size(0), Q.size(1), Q.size(2), Q.size(3), V.size(1), V.size(3)})
            if (n > INT32_MAX) throw Refused{"a dimension exceeds 2^31 - 1"};
        shape.batch = (int)Q.size(0);
        shape.qk_heads = (int)Q.size(1);
        shape.tokens = (int)Q.size(2);
        shape.d_k = (int)Q.size(3);
        shape.heads = (int)V.size(1);
        shape.d_v = (int)V.size(3);
        if (shape.qk_heads < 1 || shape.heads % shape.qk_heads) throw Refused{"the value heads are not a multiple of the key heads"};
    }
    void like(const at::Tensor& t, const char* name, at::ScalarType want) const {
        if (t.scalar_type() != want) refuse(name, std::string("must be ") + c10::toString(want));
        if (t.device() != device) refuse(name, "must be on " + device.str());
    }
    ttt_view tokens(PyObject* o, const char* name, int heads, int width) const {
        const at::Tensor& t = tensor(o, name);
        if (t.dim() != 4 || t.size(0) != shape.batch || t.size(1) != heads || t.size(2) != shape.tokens || t.size(3) != width)
            refuse(name, "must be " + text({shape.batch, heads, shape.tokens, width}));
        like(t, name, type);
        if (width != 1 && t.stride(3) != 1) refuse(name, "must be contiguous along its last dimension");
        return ttt_view{t.data_ptr(), t.stride(0), t.stride(1), t.stride(2)};
    }
    ttt_view gates(PyObject* o, const char* name) const {
        const at::Tensor& t = tensor(o, name);
        if (t.dim() != 3 || t.size(0) != shape.batch || t.size(1) != shape.heads || t.size(2) != shape.tokens)
            refuse(name, "must be " + text({shape.batch, shape.heads, shape.tokens}));
        like(t, name, at::kFloat);
        return ttt_view{t.data_ptr(), t.stride(0), t.stride(1), t.stride(2)};
    }
    // [lead][heads][d_v][d_k] fp32, or without the leading dimension (lead 0)
    float* states(PyObject* o, const char* name, int64_t lead) const {
        if (o == Py_None) return nullptr;
        const at::Tensor& t = tensor(o, name);
        const bool fits = lead ? t.dim() == 4 && t.size(0) == lead && t.size(1) == shape.heads && t.size(2) == shape.d_v && t.size(3) == shape.d_k
                               : t.dim() == 3 && t.size(0) == shape.heads && t.size(1) == shape.d_v && t.size(2) == shape.d_k;
        if (!fits) refuse(name, "must be " + (lead ? text({lead, shape.heads, shape.d_v, shape.d_k}) : text({shape.heads, shape.d_v, shape.d_k})));
        like(t, name, at::kFloat);
        if (!t.is_contiguous()) refuse(name, "must be contiguous");
        return static_cast<float*>(t.data_ptr());
    }
    float* start_weights(PyObject* o, int* shared) const {
        *shared = 0;
        if (o == Py_None) return nullptr;
        *shared = tensor(o, "W0").dim() == 3;
        return states(o, "W0", *shared ? 0 : shape.batch);
    }
    const int* ints(PyObject* o, const char* name) const {
        if (o == Py_None) return nullptr;
        const at::Tensor& t = tensor(o, name);
        if (t.dim() != 1 || t.size(0) != shape.batch) refuse(name, "must be " + text({shape.batch}));
        like(t, name, at::kInt);
        if (!t.is_contiguous()) refuse(name, "must be contiguous");
        return static_cast<const int*>(t.data_ptr());
    }
};

struct Workspace {
    void* p = nullptr;
    size_t n = 0;
    explicit Workspace(PyObject* o) {
        if (o == Py_None) return;
        const at::Tensor& t = tensor(o, "ws");
        if (!t.is_cuda() || !t.is_contiguous()) refuse("ws", "must be a contiguous CUDA tensor");
        p = t.data_ptr();
        n = t.nbytes();
    }
};

float number(PyObject* o, const char* name) {
    const double x = PyFloat_AsDouble(o);
    if (x == -1.0 && PyErr_Occurred()) {
        PyErr_Clear();
        refuse(name, "must be a number");
    }
    return (float)x;
}

void* pointer(PyObject* o) { return PyLong_AsVoidPtr(o); }

template <class F>
PyObject* guarded(Py_ssize_t got, Py_ssize_t want, F f) {
    if (got != want) {
        PyErr_Format(PyExc_TypeError, "%zd arguments, %zd wanted", got, want);
        return nullptr;
    }
    try {
        return PyLong_FromLong(f());
    } catch (const Refused& r) {
        PyErr_SetString(PyExc_ValueError, r.why.c_str());
    } catch (const std::bad_alloc&) {
        PyErr_NoMemory();
    } catch (const std::exception& e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
    }
    return nullptr;
}

// forward(Q, K, V, G, Beta, W0, lengths, scale, Z, W1_out, ws, stream)
PyObject* forward(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded(n, 12, [&]() -> long {
        Call c;
        c.start(tensor(a[0], "Q"), tensor(a[2], "V"));
        const ttt_delta_shape& s = c.shape;
        const ttt_view q = c.tokens(a[0], "Q", s.qk_heads, s.d_k), k = c.tokens(a[1], "K", s.qk_heads, s.d_k),
                       v = c.tokens(a[2], "V", s.heads, s.d_v), g = c.gates(a[3], "G"), b = c.gates(a[4], "Beta"),
                       z = c.tokens(a[8], "Z", s.heads, s.d_v);
        int shared;
        const float* w0 = c.start_weights(a[5], &shared);
        const Workspace ws(a[10]);
        return ttt_forward_gated_delta(&q, &k, &v, &g, &b, w0, shared, c.ints(a[6], "lengths"), number(a[7], "scale"), &z,
                                       c.states(a[9], "W1_out", s.batch), &s, ws.p, ws.n, pointer(a[11]));
    });
}

// backward(Q, K, V, G, Beta, dZ, W0, dW1, lengths, scale, dQ, dK, dV, dG, dBeta, dW0, ws, stream)
PyObject* backward(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded(n, 18, [&]() -> long {
        Call c;
        c.start(tensor(a[0], "Q"), tensor(a[2], "V"));
        const ttt_delta_shape& s = c.shape;
        const ttt_view q = c.tokens(a[0], "Q", s.qk_heads, s.d_k), k = c.tokens(a[1], "K", s.qk_heads, s.d_k),
                       v = c.tokens(a[2], "V", s.heads, s.d_v), g = c.gates(a[3], "G"), b = c.gates(a[4], "Beta"),
                       dz = c.tokens(a[5], "dZ", s.heads, s.d_v), dq = c.tokens(a[10], "dQ", s.qk_heads, s.d_k),
                       dk = c.tokens(a[11], "dK", s.qk_heads, s.d_k), dv = c.tokens(a[12], "dV", s.heads, s.d_v),
                       dg = c.gates(a[13], "dG"), db = c.gates(a[14], "dBeta");
        int shared;
        const float* w0 = c.start_weights(a[6], &shared);
        if (!w0 && a[15] != Py_None) throw Refused{"dW0 needs W0"};
        float* dw0 = c.states(a[15], "dW0", shared ? 0 : s.batch);
        const Workspace ws(a[16]);
        return ttt_backward_gated_delta(&q, &k, &v, &g, &b, w0, shared, c.ints(a[8], "lengths"), number(a[9], "scale"), &dz,
                                        c.states(a[7], "dW1", s.batch), &s, ws.p, ws.n, &dq, &dk, &dv, &dg, &db, dw0, pointer(a[17]));
    });
}

// step(Q, K, V, G, Beta, W, slots, scale, Z, stream)
PyObject* step(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded(n, 10, [&]() -> long {
        Call c;
        c.start(tensor(a[0], "Q"), tensor(a[2], "V"));
        const ttt_delta_shape& s = c.shape;
        const ttt_view q = c.tokens(a[0], "Q", s.qk_heads, s.d_k), k = c.tokens(a[1], "K", s.qk_heads, s.d_k),
                       v = c.tokens(a[2], "V", s.heads, s.d_v), g = c.gates(a[3], "G"), b = c.gates(a[4], "Beta"),
                       z = c.tokens(a[8], "Z", s.heads, s.d_v);
        const at::Tensor& W = tensor(a[5], "W");
        if (W.dim() != 4 || W.size(0) < 1 || W.size(0) > INT32_MAX) throw Refused{"W must be [n_slots][heads][d_v][d_k]"};
        float* w = c.states(a[5], "W", W.size(0));
        return ttt_step_gated_delta(&q, &k, &v, &g, &b, w, (int)W.size(0), c.ints(a[6], "slots"), number(a[7], "scale"), &z, &s,
                                    pointer(a[9]));
    });
}

// workspace(backward, Q, V): bytes
PyObject* workspace(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded(n, 3, [&]() -> long {
        Call c;
        c.start(tensor(a[1], "Q"), tensor(a[2], "V"));
        return (long)ttt_gated_delta_workspace_bytes(PyObject_IsTrue(a[0]), &c.shape);
    });
}

// Whether the elements of a [B][heads][N] or [B][heads][N][d] tensor lie in the order of [B][N][heads][d], without gaps.
bool by_token(const at::Tensor& t) {
    const int64_t n = t.dim();
    if (n != 3 && n != 4) return false;
    int64_t step = 1;
    for (int64_t i : {(int64_t)3, (int64_t)1, (int64_t)2, (int64_t)0}) {       // from the innermost
        if (i >= n) continue;
        if (t.size(i) != 1 && t.stride(i) != step) return false;
        step *= t.size(i);
    }
    return true;
}

// clip(grads, out or None, max_norm, norm, ws, stream); grads, out: lists or tuples
PyObject* clip(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded(n, 6, [&]() -> long {
        if ((!PyList_Check(a[0]) && !PyTuple_Check(a[0])) || (a[1] != Py_None && !PyList_Check(a[1]) && !PyTuple_Check(a[1])))
            throw Refused{"gradients and outputs must be lists or tuples"};
        const Py_ssize_t m = PySequence_Fast_GET_SIZE(a[0]);
        if (m < 1 || m > INT32_MAX) throw Refused{"no gradients"};
        if (a[1] != Py_None && PySequence_Fast_GET_SIZE(a[1]) != m) throw Refused{"as many outputs as gradients are needed"};
        std::vector<const void*> in(m);
        std::vector<void*> out(m);
        std::vector<long long> counts(m);
        std::vector<int> types(m);
        const c10::Device device = tensor(PySequence_Fast_GET_ITEM(a[0], 0), "gradient").device();
        if (!device.is_cuda()) throw Refused{"gradients must be CUDA tensors"};
        for (Py_ssize_t i = 0; i < m; ++i) {
            const at::Tensor& g = tensor(PySequence_Fast_GET_ITEM(a[0], i), "gradient");
            const bool plain = g.is_contiguous(), tokens = by_token(g);
            if (g.device() != device || (!plain && !tokens)) throw Refused{"gradients must be tensors on one device, contiguous or laid out by token"};
            if (g.scalar_type() == at::kBFloat16) types[i] = TTT_BF16;
            else if (g.scalar_type() == at::kFloat) types[i] = TTT_FP32;
            else throw Refused{"gradients must be bfloat16 or float32"};
            in[i] = out[i] = g.data_ptr();
            counts[i] = g.numel();
            if (a[1] != Py_None) {
                const at::Tensor& o = tensor(PySequence_Fast_GET_ITEM(a[1], i), "output");
                if (o.sizes() != g.sizes() || o.scalar_type() != g.scalar_type() || o.device() != device ||
                    !((plain && o.is_contiguous()) || (tokens && by_token(o))))
                    throw Refused{"outputs must be like their gradients and laid out like them"};
                out[i] = o.data_ptr();
            }
        }
        const Workspace ws(a[4]);
        return ttt_clip_gradients(in.data(), out.data(), counts.data(), types.data(), (int)m, number(a[2], "max_norm"),
                                  static_cast<float*>(tensor(a[3], "norm").data_ptr()), ws.p, ws.n, pointer(a[5]));
    });
}

PyCFunction fast(PyObject* (*f)(PyObject*, PyObject* const*, Py_ssize_t)) { return reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f)); }

PyMethodDef methods[] = {{"forward", fast(forward), METH_FASTCALL, nullptr},
                         {"backward", fast(backward), METH_FASTCALL, nullptr},
                         {"step", fast(step), METH_FASTCALL, nullptr},
                         {"workspace", fast(workspace), METH_FASTCALL, nullptr},
                         {"clip", fast(clip), METH_FASTCALL, nullptr},
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_native", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__native() { return PyModule_Create(&module); }
