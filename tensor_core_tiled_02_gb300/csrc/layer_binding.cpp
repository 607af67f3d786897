// The layer operators on torch tensors: argument checks, output memory and the
// current stream, then one call of the C ABI (include/layer_ops.h).  layers.py
// holds the signatures and the documentation; this is its native half, because
// a call for one token runs 4 to 10 us on the GPU while the same steps in Python
// took 12 (and 0.5 a tensor for gradient clipping).  Arithmetic happens in
// libtcgemm.so only.
//
// Functions take positional arguments, refuse tensors with ValueError, and return
// their outputs, or the library's status (an int) when it is not 0.
#include <Python.h>

#include <ATen/core/grad_mode.h>
#include <ATen/ops/empty.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cstring>
#include <stdexcept>
#include <string>
#include <vector>

#include "layer_ops.h"

namespace {

// The library's entry points, handed over by bind().
struct Abi {
    decltype(&linear_forward) linear;
    decltype(&linear_backward) linear_grad;
    decltype(&linear_backward_workspace) linear_grad_ws;
    decltype(&gated_ffn_forward) gated;
    decltype(&gated_ffn_backward) gated_grad;
    decltype(&gated_ffn_backward_workspace) gated_grad_ws;
    decltype(&linear_cross_entropy) loss;
    decltype(&linear_cross_entropy_workspace) loss_ws;
    decltype(&linear_cross_entropy_backward) loss_grad;
    decltype(&linear_cross_entropy_backward_workspace) loss_grad_ws;
    decltype(&grad_clip) clip;
    decltype(&grad_clip_workspace) clip_ws;
} abi;

struct Refusal : std::runtime_error {
    using std::runtime_error::runtime_error;
};

[[noreturn]] void refuse(const std::string& why) { throw Refusal(why); }

std::string shape_of(const at::Tensor& t) {
    std::string s = "[";
    for (int64_t i = 0; i < t.dim(); ++i) s += (i ? ", " : "") + std::to_string(t.size(i));
    return s + "]";
}

const char* type_name(at::ScalarType t) { return t == at::kHalf ? "torch.float16" : t == at::kBFloat16 ? "torch.bfloat16" : "torch.float32"; }

int type_code(at::ScalarType t) {
    return t == at::kHalf ? LAYER_F16 : t == at::kBFloat16 ? LAYER_BF16 : t == at::kFloat ? LAYER_F32 : -1;
}

const at::Tensor& tensor(PyObject* o, const char* name) {
    if (!THPVariable_Check(o)) refuse(std::string(name) + " must be a tensor");
    const at::Tensor& t = THPVariable_Unpack(o);
    if (t.layout() != at::kStrided) refuse(std::string(name) + " must be a dense tensor");
    return t;
}

int64_t pitch(int64_t cols) { return (cols + 7) / 8 * 8; }

// Row stride of a matrix; a single row's is free, the library only wants it aligned.
int64_t stride_of(const at::Tensor& t, const char* name) {
    if (t.size(1) > 1 && t.stride(1) != 1) refuse(std::string(name) + "'s rows must be contiguous");
    return t.size(0) > 1 ? t.stride(0) : pitch(t.size(1));
}

// One call: the type, device and stream its first operand fixes.
struct Call {
    at::ScalarType type;
    c10::Device device;
    c10::cuda::CUDAGuard guard;
    gemm_stream_t stream;

    static const at::Tensor& checked(const at::Tensor& t, const char* name) {
        if (t.dim() != 2 || (t.scalar_type() != at::kHalf && t.scalar_type() != at::kBFloat16))
            refuse(std::string(name) + " must be a 2-D fp16 or bf16 tensor");
        return on_cuda(t, name);
    }
    static const at::Tensor& on_cuda(const at::Tensor& t, const char* name) {
        if (!t.is_cuda()) refuse(std::string(name) + " must be a CUDA tensor");
        return t;
    }
    explicit Call(const at::Tensor& t)
        : type(t.scalar_type()), device(t.device()), guard(t.device()),
          stream(c10::cuda::getCurrentCUDAStream(t.device().index()).stream()) {}

    void matrix(const at::Tensor& t, const char* name, int64_t rows, int64_t cols) const {
        if (t.scalar_type() != type) refuse(std::string(name) + " must be " + type_name(type));
        if (t.dim() != 2 || t.size(0) != rows || t.size(1) != cols)
            refuse(std::string(name) + " must be [" + std::to_string(rows) + ", " + std::to_string(cols) + "], got " + shape_of(t));
        place(t, name);
    }
    void vector(const at::Tensor& t, const char* name, int64_t n, at::ScalarType st) const {
        if (t.scalar_type() != st || t.dim() != 1 || t.size(0) != n || !t.is_contiguous())
            refuse(std::string(name) + " must be a contiguous [" + std::to_string(n) + "] tensor of its type");
        place(t, name);
    }
    void place(const at::Tensor& t, const char* name) const {
        if (t.device() != device) refuse(std::string(name) + " is on " + t.device().str() + ", not on " + device.str());
    }
    at::Tensor empty(at::IntArrayRef shape, at::ScalarType st) const {
        return at::empty(shape, at::TensorOptions().dtype(st).device(device));
    }
    // A matrix whose row stride the library takes: a multiple of 8.
    at::Tensor matrix(int64_t rows, int64_t cols) const {
        if (cols % 8 == 0) return empty({rows, cols}, type);
        return empty({rows, pitch(cols)}, type).narrow(1, 0, cols);
    }
    at::Tensor workspace(size_t bytes) const {
        return bytes ? empty({(int64_t)bytes}, at::kByte) : at::Tensor();
    }
};

// A tensor the call has written: autograd, which did not see it, must not take a copy it
// saved for unchanged.  (Inference tensors have no version.)
void wrote(const at::Tensor& t) {
    if (!t.is_inference()) t.unsafeGetTensorImpl()->bump_version();
}

void* ptr(const at::Tensor& t) { return t.defined() ? t.data_ptr() : nullptr; }
const void* cptr(PyObject* o, const char* name) { return o == Py_None ? nullptr : tensor(o, name).data_ptr(); }

PyObject* wrap(const at::Tensor& t) {
    if (!t.defined()) Py_RETURN_NONE;
    return THPVariable_Wrap(t);
}

PyObject* wrap_all(std::initializer_list<at::Tensor> ts) {
    PyObject* out = PyTuple_New((Py_ssize_t)ts.size());
    if (!out) return nullptr;
    Py_ssize_t i = 0;
    for (const at::Tensor& t : ts) {
        PyObject* o = wrap(t);
        if (!o) {
            Py_DECREF(out);
            return nullptr;
        }
        PyTuple_SET_ITEM(out, i++, o);
    }
    return out;
}

long long integer(PyObject* o) {
    const long long v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred()) {
        PyErr_Clear();
        refuse("an integer of at most 64 bits is wanted");
    }
    return v;
}

double real(PyObject* o) {
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred()) {
        PyErr_Clear();
        refuse("a number is wanted");
    }
    return v;
}

// No C++ exception leaves a function: refusals become ValueError, torch's own what torch makes
// of them (OutOfMemoryError among them).
template <typename F>
PyObject* guarded(PyObject* const* v, Py_ssize_t have, Py_ssize_t want, F&& f) {
    if (have != want) {
        PyErr_Format(PyExc_TypeError, "%zd arguments are wanted, got %zd", want, have);
        return nullptr;
    }
    if (!abi.linear) {
        PyErr_SetString(PyExc_RuntimeError, "the library is not bound");
        return nullptr;
    }
    // before the call, so that a warning turned into an error leaves everything as it was
    if (at::GradMode::is_enabled())
        for (Py_ssize_t i = 0; i < have; ++i)
            if (THPVariable_Check(v[i]) && THPVariable_Unpack(v[i]).requires_grad()) {
                if (PyErr_WarnEx(PyExc_UserWarning,
                                 "a layer operator was given a tensor that requires a gradient: it records no autograd "
                                 "graph, its gradients are those of its _backward call (torch.no_grad() says so)", 1) < 0)
                    return nullptr;
                break;
            }
    try {
        return f();
    } catch (const Refusal& e) {
        PyErr_SetString(PyExc_ValueError, e.what());
    } catch (const std::bad_alloc&) {
        PyErr_NoMemory();
    } catch (...) {
        torch::translate_exception_to_python(std::current_exception());
    }
    return nullptr;
}

// (x, w, bias, act, residual, save, out) -> y, or (y, preact)
PyObject* py_linear(PyObject*, PyObject* const* v, Py_ssize_t nargs) {
    return guarded(v, nargs, 7, [&]() -> PyObject* {
        const at::Tensor& x = Call::checked(tensor(v[0], "x"), "x");
        const at::Tensor& w = tensor(v[1], "w");
        const int64_t tokens = x.size(0), k = x.size(1);
        if (w.dim() != 2 || w.size(1) < 1 || k < 1) refuse("w must be 2-D and not empty");
        const int64_t n = w.size(1);
        const Call c(x);
        linear_args a{};
        a.ldx = stride_of(x, "x");
        c.matrix(w, "w", k, n);
        a.ldw = stride_of(w, "w");
        if (v[2] != Py_None) c.vector(tensor(v[2], "bias"), "bias", n, c.type);
        if (v[4] != Py_None) {
            const at::Tensor& r = tensor(v[4], "residual");
            c.matrix(r, "residual", tokens, n);
            a.ldr = stride_of(r, "residual");
        }
        const bool save = v[5] == Py_True;
        at::Tensor y, pre;
        if (v[6] != Py_None) {
            y = tensor(v[6], "out");
            c.matrix(y, "out", tokens, n);
            a.ldy = stride_of(y, "out");
        } else {
            y = c.matrix(tokens, n);
            a.ldy = pitch(n);
        }
        if (save) pre = c.matrix(tokens, n);
        a.x = x.data_ptr();
        a.w = w.data_ptr();
        a.bias = cptr(v[2], "bias");
        a.residual = cptr(v[4], "residual");
        a.y = y.data_ptr();
        a.preact = ptr(pre);
        a.ldp = pitch(n);
        a.tokens = tokens;
        a.k = k;
        a.n = n;
        a.dtype = type_code(c.type);
        a.act = integer(v[3]);
        const int rc = abi.linear(&a, c.stream);
        if (rc != 0) return PyLong_FromLong(rc);
        if (v[6] != Py_None) wrote(y);
        if (save) return wrap_all({y, pre});
        if (v[6] != Py_None) return Py_NewRef(v[6]);
        return wrap(y);
    });
}

// (dy, x, w, act, preact, bias) -> (dx, dw, dbias)
PyObject* py_linear_backward(PyObject*, PyObject* const* v, Py_ssize_t nargs) {
    return guarded(v, nargs, 6, [&]() -> PyObject* {
        const at::Tensor& x = Call::checked(tensor(v[1], "x"), "x");
        const at::Tensor &dy = tensor(v[0], "dy"), &w = tensor(v[2], "w");
        const int64_t tokens = x.size(0), k = x.size(1);
        if (w.dim() != 2 || w.size(1) < 1 || k < 1) refuse("w must be 2-D and not empty");
        const int64_t n = w.size(1);
        const Call c(x);
        linear_grad_args a{};
        a.act = integer(v[3]);
        a.ldx = stride_of(x, "x");
        c.matrix(w, "w", k, n);
        a.ldw = stride_of(w, "w");
        c.matrix(dy, "dy", tokens, n);
        a.lddy = stride_of(dy, "dy");
        if (a.act != LAYER_ACT_NONE) {
            if (v[4] == Py_None) refuse("preact is needed for the slope of the activation");
            const at::Tensor& pre = tensor(v[4], "preact");
            c.matrix(pre, "preact", tokens, n);
            a.ldp = stride_of(pre, "preact");
            a.preact = pre.data_ptr();
        }
        const at::Tensor dx = c.matrix(tokens, k), dw = c.matrix(k, n);
        at::Tensor dbias;
        if (v[5] == Py_True) dbias = c.empty({n}, c.type);
        a.dy = dy.data_ptr();
        a.x = x.data_ptr();
        a.w = w.data_ptr();
        a.dx = dx.data_ptr();
        a.dw = dw.data_ptr();
        a.dbias = ptr(dbias);
        a.lddx = pitch(k);
        a.lddw = pitch(n);
        a.tokens = tokens;
        a.k = k;
        a.n = n;
        a.dtype = type_code(c.type);
        size_t bytes = 0;
        int rc = abi.linear_grad_ws(&a, &bytes);
        if (rc != 0) return PyLong_FromLong(rc);
        const at::Tensor ws = c.workspace(bytes);
        a.workspace = ptr(ws);
        a.workspace_bytes = (long long)bytes;
        rc = abi.linear_grad(&a, c.stream);
        if (rc != 0) return PyLong_FromLong(rc);
        return wrap_all({dx, dw, dbias});
    });
}

struct Gated {
    int64_t tokens, dim, ffn, dim_out;
};

Gated gated_sizes(const at::Tensor& x, const at::Tensor& wg, const at::Tensor& wd) {
    const Gated g{x.size(0), x.size(1), wg.dim() == 2 ? wg.size(1) : 0, wd.dim() == 2 ? wd.size(1) : 0};
    if (g.dim < 1 || g.ffn < 1 || g.dim_out < 1) refuse("the weights must be 2-D and not empty");
    return g;
}

// (x, w_gate, w_up, w_down, act, residual, save, out) -> y, or (y, gate, up, hidden)
PyObject* py_gated_ffn(PyObject*, PyObject* const* v, Py_ssize_t nargs) {
    return guarded(v, nargs, 8, [&]() -> PyObject* {
        const at::Tensor& x = Call::checked(tensor(v[0], "x"), "x");
        const at::Tensor &wg = tensor(v[1], "w_gate"), &wu = tensor(v[2], "w_up"), &wd = tensor(v[3], "w_down");
        const Gated s = gated_sizes(x, wg, wd);
        const Call c(x);
        gated_args a{};
        a.ldx = stride_of(x, "x");
        c.matrix(wg, "w_gate", s.dim, s.ffn);
        a.ldw_gate = stride_of(wg, "w_gate");
        c.matrix(wu, "w_up", s.dim, s.ffn);
        a.ldw_up = stride_of(wu, "w_up");
        c.matrix(wd, "w_down", s.ffn, s.dim_out);
        a.ldw_down = stride_of(wd, "w_down");
        if (v[5] != Py_None) {
            const at::Tensor& r = tensor(v[5], "residual");
            c.matrix(r, "residual", s.tokens, s.dim_out);
            a.ldr = stride_of(r, "residual");
            a.residual = r.data_ptr();
        }
        const bool save = v[6] == Py_True;
        at::Tensor y, gate, up;
        if (v[7] != Py_None) {
            y = tensor(v[7], "out");
            c.matrix(y, "out", s.tokens, s.dim_out);
            a.ldy = stride_of(y, "out");
        } else {
            y = c.matrix(s.tokens, s.dim_out);
            a.ldy = pitch(s.dim_out);
        }
        const at::Tensor hidden = c.matrix(s.tokens, s.ffn);
        if (save) {
            gate = c.matrix(s.tokens, s.ffn);
            up = c.matrix(s.tokens, s.ffn);
        }
        a.x = x.data_ptr();
        a.w_gate = wg.data_ptr();
        a.w_up = wu.data_ptr();
        a.w_down = wd.data_ptr();
        a.y = y.data_ptr();
        a.hidden = hidden.data_ptr();
        a.gate = ptr(gate);
        a.up = ptr(up);
        a.ld_hidden = a.ld_gate = a.ld_up = pitch(s.ffn);
        a.tokens = s.tokens;
        a.dim = s.dim;
        a.ffn = s.ffn;
        a.dim_out = s.dim_out;
        a.dtype = type_code(c.type);
        a.act = integer(v[4]);
        const int rc = abi.gated(&a, c.stream);
        if (rc != 0) return PyLong_FromLong(rc);
        if (v[7] != Py_None) wrote(y);
        if (save) return wrap_all({y, gate, up, hidden});
        if (v[7] != Py_None) return Py_NewRef(v[7]);
        return wrap(y);
    });
}

// (dy, x, w_gate, w_up, w_down, gate, up, hidden, act) -> (dx, dw_gate, dw_up, dw_down)
PyObject* py_gated_ffn_backward(PyObject*, PyObject* const* v, Py_ssize_t nargs) {
    return guarded(v, nargs, 9, [&]() -> PyObject* {
        static const char* const names[8] = {"dy", "x", "w_gate", "w_up", "w_down", "gate", "up", "hidden"};
        const at::Tensor& x = Call::checked(tensor(v[1], "x"), "x");
        const Gated s = gated_sizes(x, tensor(v[2], "w_gate"), tensor(v[4], "w_down"));
        const Call c(x);
        const int64_t rows[8] = {s.tokens, s.tokens, s.dim, s.dim, s.ffn, s.tokens, s.tokens, s.tokens};
        const int64_t cols[8] = {s.dim_out, s.dim, s.ffn, s.ffn, s.dim_out, s.ffn, s.ffn, s.ffn};
        gated_grad_args a{};
        const void** ptrs[8] = {&a.dy, &a.x, &a.w_gate, &a.w_up, &a.w_down, &a.gate, &a.up, &a.hidden};
        long long* lds[8] = {&a.lddy, &a.ldx, &a.ldw_gate, &a.ldw_up, &a.ldw_down, &a.ld_gate, &a.ld_up, &a.ld_hidden};
        for (int i = 0; i < 8; ++i) {
            const at::Tensor& t = tensor(v[i], names[i]);
            c.matrix(t, names[i], rows[i], cols[i]);
            *lds[i] = stride_of(t, names[i]);
            *ptrs[i] = t.data_ptr();
        }
        const at::Tensor dx = c.matrix(s.tokens, s.dim), dwg = c.matrix(s.dim, s.ffn), dwu = c.matrix(s.dim, s.ffn);
        const at::Tensor dwd = c.matrix(s.ffn, s.dim_out);
        a.dx = dx.data_ptr();
        a.dw_gate = dwg.data_ptr();
        a.dw_up = dwu.data_ptr();
        a.dw_down = dwd.data_ptr();
        a.lddx = pitch(s.dim);
        a.lddw_gate = a.lddw_up = pitch(s.ffn);
        a.lddw_down = pitch(s.dim_out);
        a.tokens = s.tokens;
        a.dim = s.dim;
        a.ffn = s.ffn;
        a.dim_out = s.dim_out;
        a.dtype = type_code(c.type);
        a.act = integer(v[8]);
        size_t bytes = 0;
        int rc = abi.gated_grad_ws(&a, &bytes);
        if (rc != 0) return PyLong_FromLong(rc);
        const at::Tensor ws = c.workspace(bytes);
        a.workspace = ptr(ws);
        a.workspace_bytes = (long long)bytes;
        rc = abi.gated_grad(&a, c.stream);
        if (rc != 0) return PyLong_FromLong(rc);
        return wrap_all({dx, dwg, dwu, dwd});
    });
}

// (h, w, target, ignore_index, reduction) -> (loss, lse)
PyObject* py_loss(PyObject*, PyObject* const* v, Py_ssize_t nargs) {
    return guarded(v, nargs, 5, [&]() -> PyObject* {
        const at::Tensor& h = Call::checked(tensor(v[0], "h"), "h");
        const at::Tensor &w = tensor(v[1], "w"), &target = tensor(v[2], "target");
        if (w.dim() != 2 || w.size(0) < 1 || h.size(1) < 1) refuse("w must be [vocabulary, features] and not empty");
        const Call c(h);
        loss_args a{};
        a.tokens = h.size(0);
        a.dim = h.size(1);
        a.vocab = w.size(0);
        a.ldh = stride_of(h, "h");
        c.matrix(w, "w", a.vocab, a.dim);
        a.ldw = stride_of(w, "w");
        c.vector(target, "target (int64)", a.tokens, at::kLong);
        a.dtype = type_code(c.type);
        a.ignore_index = integer(v[3]);
        a.reduction = integer(v[4]);
        const at::Tensor loss = a.reduction == LAYER_LOSS_NONE ? c.empty({a.tokens}, at::kFloat) : c.empty({}, at::kFloat);
        const at::Tensor lse = c.empty({a.tokens}, at::kFloat);
        a.h = h.data_ptr();
        a.w = w.data_ptr();
        a.target = static_cast<const long long*>(target.data_ptr());
        a.loss = static_cast<float*>(loss.data_ptr());
        a.lse = static_cast<float*>(lse.data_ptr());
        size_t bytes = 0;
        int rc = abi.loss_ws(&a, &bytes);
        if (rc != 0) return PyLong_FromLong(rc);
        const at::Tensor ws = c.workspace(bytes);
        a.workspace = ptr(ws);
        a.workspace_bytes = (long long)bytes;
        rc = abi.loss(&a, c.stream);
        if (rc != 0) return PyLong_FromLong(rc);
        return wrap_all({loss, lse});
    });
}

// (grad_loss, h, w, target, lse, ignore_index, reduction, piece) -> (dh, dw)
PyObject* py_loss_backward(PyObject*, PyObject* const* v, Py_ssize_t nargs) {
    return guarded(v, nargs, 8, [&]() -> PyObject* {
        const at::Tensor& h = Call::checked(tensor(v[1], "h"), "h");
        const at::Tensor &grad = tensor(v[0], "grad_loss"), &w = tensor(v[2], "w");
        const at::Tensor &target = tensor(v[3], "target"), &lse = tensor(v[4], "lse");
        if (w.dim() != 2 || w.size(0) < 1 || h.size(1) < 1) refuse("w must be [vocabulary, features] and not empty");
        const Call c(h);
        loss_grad_args a{};
        a.tokens = h.size(0);
        a.dim = h.size(1);
        a.vocab = w.size(0);
        a.ldh = stride_of(h, "h");
        c.matrix(w, "w", a.vocab, a.dim);
        a.ldw = stride_of(w, "w");
        c.vector(target, "target (int64)", a.tokens, at::kLong);
        c.vector(lse, "lse (fp32)", a.tokens, at::kFloat);
        a.dtype = type_code(c.type);
        a.ignore_index = integer(v[5]);
        a.reduction = integer(v[6]);
        if (grad.scalar_type() != at::kFloat || !grad.is_contiguous() ||
            grad.numel() != (a.reduction == LAYER_LOSS_NONE ? a.tokens : 1))
            refuse("grad_loss must be contiguous fp32: one value, or [tokens] for reduction \"none\"");
        c.place(grad, "grad_loss");
        const at::Tensor dh = c.matrix(a.tokens, a.dim), dw = c.matrix(a.vocab, a.dim);
        a.h = h.data_ptr();
        a.w = w.data_ptr();
        a.target = static_cast<const long long*>(target.data_ptr());
        a.lse = static_cast<const float*>(lse.data_ptr());
        a.grad_loss = static_cast<const float*>(grad.data_ptr());
        a.dh = dh.data_ptr();
        a.dw = dw.data_ptr();
        a.lddh = a.lddw = pitch(a.dim);
        size_t bytes = 0;
        int rc = abi.loss_grad_ws(&a, integer(v[7]), &bytes);
        if (rc != 0) return PyLong_FromLong(rc);
        const at::Tensor ws = c.workspace(bytes);
        a.workspace = ptr(ws);
        a.workspace_bytes = (long long)bytes;
        rc = abi.loss_grad(&a, c.stream);
        if (rc != 0) return PyLong_FromLong(rc);
        return wrap_all({dh, dw});
    });
}

// (grads, max_norm, out, eps) -> norm; grads and out are lists
PyObject* py_clip(PyObject*, PyObject* const* v, Py_ssize_t nargs) {
    return guarded(v, nargs, 4, [&]() -> PyObject* {
        if (!PyList_Check(v[0]) || PyList_GET_SIZE(v[0]) < 1) refuse("gradients must be a list that is not empty");
        const bool in_place = v[2] == Py_None;
        const Py_ssize_t n = PyList_GET_SIZE(v[0]);
        if (!in_place && (!PyList_Check(v[2]) || PyList_GET_SIZE(v[2]) != n)) refuse("out must have as many tensors as there are gradients");
        const at::Tensor& first = Call::on_cuda(tensor(PyList_GET_ITEM(v[0], 0), "a gradient"), "a gradient");
        const Call c(first);
        std::vector<const void*> src(n);
        std::vector<void*> dst(n);
        std::vector<long long> count(n);
        std::vector<int> type(n);
        for (Py_ssize_t i = 0; i < n; ++i) {
            const at::Tensor& g = tensor(PyList_GET_ITEM(v[0], i), "a gradient");
            type[i] = type_code(g.scalar_type());
            if (type[i] < 0 || !g.is_contiguous()) refuse("gradients must be contiguous fp16, bf16 or fp32 tensors");
            c.place(g, "a gradient");
            src[i] = g.data_ptr();
            dst[i] = g.data_ptr();
            count[i] = g.numel();
            if (in_place) continue;
            const at::Tensor& o = tensor(PyList_GET_ITEM(v[2], i), "an output");
            if (o.scalar_type() != g.scalar_type() || o.numel() != count[i] || !o.is_contiguous())
                refuse("out must have the gradients' sizes and types, contiguous");
            c.place(o, "an output");
            dst[i] = o.data_ptr();
        }
        const at::Tensor norm = c.empty({}, at::kFloat);
        size_t bytes = 0;
        int rc = abi.clip_ws(n, &bytes);
        if (rc != 0) return PyLong_FromLong(rc);
        const at::Tensor ws = c.workspace(bytes);
        grad_clip_args a{};
        a.src = src.data();
        a.dst = dst.data();
        a.count = count.data();
        a.dtype = type.data();
        a.norm = static_cast<float*>(norm.data_ptr());
        a.workspace = ptr(ws);
        a.tensors = n;
        a.max_norm = real(v[1]);
        a.eps = real(v[3]);
        a.workspace_bytes = (long long)bytes;
        rc = abi.clip(&a, c.stream);
        if (rc != 0) return PyLong_FromLong(rc);
        for (Py_ssize_t i = 0; i < n; ++i) wrote(tensor(PyList_GET_ITEM(v[in_place ? 0 : 2], i), "an output"));
        return wrap(norm);
    });
}

// (address, ...) of the entry points, in Abi's order
PyObject* py_bind(PyObject*, PyObject* const* v, Py_ssize_t nargs) {
    constexpr Py_ssize_t kEntries = sizeof(Abi) / sizeof(void*);
    void* table[kEntries];
    if (nargs != kEntries) {
        PyErr_Format(PyExc_TypeError, "%zd addresses are wanted, got %zd", kEntries, nargs);
        return nullptr;
    }
    for (Py_ssize_t i = 0; i < kEntries; ++i) {
        table[i] = PyLong_AsVoidPtr(v[i]);
        if (!table[i]) {
            if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, "a null address");
            return nullptr;
        }
    }
    std::memcpy(&abi, table, sizeof(abi));
    Py_RETURN_NONE;
}

#define ENTRY(name, fn) {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(fn)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {ENTRY("bind", py_bind),
                         ENTRY("linear", py_linear),
                         ENTRY("linear_backward", py_linear_backward),
                         ENTRY("gated_ffn", py_gated_ffn),
                         ENTRY("gated_ffn_backward", py_gated_ffn_backward),
                         ENTRY("linear_cross_entropy", py_loss),
                         ENTRY("linear_cross_entropy_backward", py_loss_backward),
                         ENTRY("clip_grad_norm", py_clip),
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_layers", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__layers() { return PyModule_Create(&module); }
