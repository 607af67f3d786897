// The layer operators on torch tensors: argument checks, output memory and the
// current stream, then one call of the C ABI (include/layer_ops.h, mx_ops.h).  layers.py
// and mx.py hold the signatures and the documentation; this is their native half, because
// a call for one token runs 4 to 10 us on the GPU while the same steps in Python
// took 12 (and 0.5 a tensor for gradient clipping).  Arithmetic happens in
// libtcgemm.so only.
//
// Functions take positional arguments, refuse tensors with ValueError, and return
// their outputs, or the library's status (an int) when it is not 0.
#include <Python.h>

#include <ATen/Context.h>
#include <ATen/core/grad_mode.h>
#include <ATen/cuda/EmptyTensor.h>
#include <ATen/ops/empty.h>
#include <ATen/record_function.h>
#include <c10/core/impl/LocalDispatchKeySet.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cstring>
#include <stdexcept>
#include <string>
#include <vector>

#include "mx_ops.h"

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
    decltype(&rms_norm_forward) norm;
    decltype(&rms_norm_backward) norm_grad;
    decltype(&rms_norm_backward_workspace) norm_grad_ws;
    decltype(&mx_quantize) quantize;
    decltype(&mx_dequantize) dequantize;
    decltype(&mx_linear) mx_product;
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

// Whether someone hears of new tensors through torch's dispatcher: a dispatch mode or another
// layer above the backends, a profiler, or the filling of new memory that goes with
// deterministic algorithms.
bool dispatcher_heard() {
    const auto keys = c10::impl::tls_local_dispatch_key_set().included_ - c10::default_included_set;
    const at::Context& context = at::globalContext();
    return !keys.empty() || at::hasCallbacks() || (context.deterministicAlgorithms() && context.deterministicFillUninitializedMemory());
}

// One call: the type, device and stream its first operand fixes.
struct Call {
    at::ScalarType type;
    c10::Device device;
    c10::cuda::CUDAGuard guard;
    gemm_stream_t stream;
    bool dispatch = dispatcher_heard();

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
    // outputs of a type of their own
    Call(const at::Tensor& t, at::ScalarType out) : Call(t) { type = out; }

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
    // By way of torch's dispatcher only where someone hears it there: several of these are a good
    // part of a small call's host time (one-token norm 5.2 us so, 4.6 straight from the allocator).
    at::Tensor empty(at::IntArrayRef shape, at::ScalarType st) const {
        if (dispatch) return at::empty(shape, at::TensorOptions().dtype(st).device(device));
        return at::Tensor(at::detail::empty_cuda(shape, st, device, std::nullopt));
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

// with n >= 0: the tensors and n
PyObject* wrap_all(std::initializer_list<at::Tensor> ts, int64_t n = -1) {
    PyObject* out = PyTuple_New((Py_ssize_t)ts.size() + (n >= 0));
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
    if (n >= 0) {
        PyObject* o = PyLong_FromLongLong(n);
        if (!o) {
            Py_DECREF(out);
            return nullptr;
        }
        PyTuple_SET_ITEM(out, i, o);
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

// ---- the norm and microscaled operands ----------------------------------------------

// A microscaled matrix [rows, cols]: data [rows, bytes] and scale, tiles of 512 bytes.
struct Scaled {
    at::Tensor data, scale;
};

int64_t blocks_of(int64_t cols) { return (cols + 31) / 32; }
int64_t data_bytes(int64_t cols, int64_t format) { return blocks_of(cols) * (format == MX_E4M3 ? 32 : 16); }

Scaled new_scaled(const Call& c, int64_t rows, int64_t cols, int64_t format) {
    return {c.empty({rows, data_bytes(cols, format)}, at::kByte), c.empty({(rows + 127) / 128, (cols + 127) / 128, 32, 4, 4}, at::kByte)};
}

// One the caller hands in: sizes that fit, rows without gaps inside.  Returns its row stride.
int64_t check_scaled(const Call& c, const at::Tensor& data, const at::Tensor& scale, const char* name, int64_t rows, int64_t cols,
                     int64_t format) {
    const int64_t width = data_bytes(cols, format);
    if (data.scalar_type() != at::kByte || data.dim() != 2 || data.size(0) != rows || data.size(1) != width)
        refuse(std::string(name) + "'s data must be uint8 [" + std::to_string(rows) + ", " + std::to_string(width) + "]");
    if (data.size(1) > 1 && data.stride(1) != 1) refuse(std::string(name) + "'s rows must be contiguous");
    if (scale.scalar_type() != at::kByte || !scale.is_contiguous() || scale.numel() != (rows + 127) / 128 * ((cols + 127) / 128) * 512)
        refuse(std::string(name) + "'s scale must be contiguous uint8 [" + std::to_string((rows + 127) / 128) + ", " +
               std::to_string((cols + 127) / 128) + ", 32, 4, 4]");
    c.place(data, name);
    c.place(scale, name);
    return rows > 1 ? data.stride(0) : (width + 15) / 16 * 16;
}

int64_t checked_format(PyObject* o) {
    const int64_t f = integer(o);
    if (f != MX_E4M3 && f != MX_E2M1) refuse("format must be \"e4m3\" or \"e2m1\"");
    return f;
}

int64_t checked_cols(PyObject* o) {
    const int64_t n = integer(o);
    if (n < 0 || n > (1ll << 40)) refuse("cols must be a size");
    return n;
}

at::ScalarType type_of(PyObject* o) { return integer(o) == LAYER_BF16 ? at::kBFloat16 : at::kHalf; }

// (x, weight, residual, eps, format or None, save, out, h_out) -> (y, h or None, rstd or None),
// or with a format (data, scale, h or None, rstd or None, dim)
PyObject* py_norm(PyObject*, PyObject* const* v, Py_ssize_t nargs) {
    return guarded(v, nargs, 8, [&]() -> PyObject* {
        const at::Tensor& x = Call::checked(tensor(v[0], "x"), "x");
        const int64_t tokens = x.size(0), dim = x.size(1);
        if (dim < 1) refuse("x must have columns");
        const Call c(Call::on_cuda(x, "x"));
        rms_norm_args a{};
        a.ldx = stride_of(x, "x");
        const at::Tensor& weight = tensor(v[1], "weight");
        c.vector(weight, "weight", dim, c.type);
        const bool scaled = v[4] != Py_None;
        at::Tensor y, h, rstd;
        Scaled m;
        if (v[2] != Py_None) {
            const at::Tensor& r = tensor(v[2], "residual");
            c.matrix(r, "residual", tokens, dim);
            a.ldr = stride_of(r, "residual");
            a.residual = r.data_ptr();
            if (v[7] != Py_None) {
                h = tensor(v[7], "h_out");
                c.matrix(h, "h_out", tokens, dim);
                a.ldh = stride_of(h, "h_out");
            } else {
                h = c.matrix(tokens, dim);
                a.ldh = pitch(dim);
            }
        } else if (v[7] != Py_None) {
            refuse("h_out is x itself where there is no residual");
        }
        if (scaled) {
            a.format = checked_format(v[4]);
            m = new_scaled(c, tokens, dim, a.format);
            a.data = m.data.data_ptr();
            a.scale = m.scale.data_ptr();
            a.ldd = data_bytes(dim, a.format);
        } else if (v[6] != Py_None) {
            y = tensor(v[6], "out");
            c.matrix(y, "out", tokens, dim);
            a.ldy = stride_of(y, "out");
        } else {
            y = c.matrix(tokens, dim);
            a.ldy = pitch(dim);
        }
        if (v[5] == Py_True) rstd = c.empty({tokens}, at::kFloat);
        a.x = x.data_ptr();
        a.weight = weight.data_ptr();
        a.h = ptr(h);
        a.y = ptr(y);
        a.rstd = static_cast<float*>(ptr(rstd));
        a.tokens = tokens;
        a.dim = dim;
        a.dtype = type_code(c.type);
        a.eps = real(v[3]);
        const int rc = abi.norm(&a, c.stream);
        if (rc != 0) return PyLong_FromLong(rc);
        if (v[6] != Py_None) wrote(y);
        if (v[7] != Py_None) wrote(h);
        return scaled ? wrap_all({m.data, m.scale, h, rstd}, dim) : wrap_all({y, h, rstd});
    });
}

// (dy, h, weight, rstd, dh, out) -> (dx, dweight)
PyObject* py_norm_backward(PyObject*, PyObject* const* v, Py_ssize_t nargs) {
    return guarded(v, nargs, 6, [&]() -> PyObject* {
        const at::Tensor& h = Call::checked(tensor(v[1], "h"), "h");
        const int64_t tokens = h.size(0), dim = h.size(1);
        if (dim < 1) refuse("h must have columns");
        const Call c(h);
        rms_norm_grad_args a{};
        a.ldh = stride_of(h, "h");
        const at::Tensor &dy = tensor(v[0], "dy"), &weight = tensor(v[2], "weight"), &rstd = tensor(v[3], "rstd");
        c.matrix(dy, "dy", tokens, dim);
        a.lddy = stride_of(dy, "dy");
        c.vector(weight, "weight", dim, c.type);
        c.vector(rstd, "rstd (fp32)", tokens, at::kFloat);
        if (v[4] != Py_None) {
            const at::Tensor& dh = tensor(v[4], "dh");
            c.matrix(dh, "dh", tokens, dim);
            a.lddh = stride_of(dh, "dh");
            a.dh = dh.data_ptr();
        }
        at::Tensor dx;
        if (v[5] != Py_None) {
            dx = tensor(v[5], "out");
            c.matrix(dx, "out", tokens, dim);
            a.lddx = stride_of(dx, "out");
        } else {
            dx = c.matrix(tokens, dim);
            a.lddx = pitch(dim);
        }
        const at::Tensor dweight = c.empty({dim}, c.type);
        a.dy = dy.data_ptr();
        a.h = h.data_ptr();
        a.weight = weight.data_ptr();
        a.rstd = static_cast<const float*>(rstd.data_ptr());
        a.dx = dx.data_ptr();
        a.dweight = dweight.data_ptr();
        a.tokens = tokens;
        a.dim = dim;
        a.dtype = type_code(c.type);
        size_t bytes = 0;
        int rc = abi.norm_grad_ws(&a, &bytes);
        if (rc != 0) return PyLong_FromLong(rc);
        const at::Tensor ws = c.workspace(bytes);
        a.workspace = ptr(ws);
        a.workspace_bytes = (long long)bytes;
        rc = abi.norm_grad(&a, c.stream);
        if (rc != 0) return PyLong_FromLong(rc);
        if (v[5] != Py_None) wrote(dx);
        return wrap_all({dx, dweight});
    });
}

// (x, format, transpose) -> (data, scale, cols)
PyObject* py_quantize(PyObject*, PyObject* const* v, Py_ssize_t nargs) {
    return guarded(v, nargs, 3, [&]() -> PyObject* {
        const at::Tensor& x = Call::on_cuda(Call::checked(tensor(v[0], "x"), "x"), "x");
        const Call c(x);
        mx_quantize_args a{};
        a.rows = x.size(0);
        a.cols = x.size(1);
        a.format = checked_format(v[1]);
        a.transpose = v[2] == Py_True;
        const int64_t rows = a.transpose ? a.cols : a.rows, cols = a.transpose ? a.rows : a.cols;
        a.ldx = stride_of(x, "x");
        const Scaled m = new_scaled(c, rows, cols, a.format);
        a.x = x.data_ptr();
        a.data = m.data.data_ptr();
        a.scale = m.scale.data_ptr();
        a.ldd = data_bytes(cols, a.format);
        a.dtype = type_code(c.type);
        const int rc = abi.quantize(&a, c.stream);
        if (rc != 0) return PyLong_FromLong(rc);
        return wrap_all({m.data, m.scale}, cols);
    });
}

// (data, scale, cols, format, dtype) -> x
PyObject* py_dequantize(PyObject*, PyObject* const* v, Py_ssize_t nargs) {
    return guarded(v, nargs, 5, [&]() -> PyObject* {
        const at::Tensor &data = Call::on_cuda(tensor(v[0], "data"), "data"), &scale = tensor(v[1], "scale");
        const Call c(data, type_of(v[4]));
        mx_dequantize_args a{};
        a.rows = data.dim() == 2 ? data.size(0) : 0;
        a.cols = checked_cols(v[2]);
        a.format = checked_format(v[3]);
        a.ldd = check_scaled(c, data, scale, "a", a.rows, a.cols, a.format);
        const at::Tensor x = c.matrix(a.rows, a.cols);
        a.data = data.data_ptr();
        a.scale = scale.data_ptr();
        a.x = x.data_ptr();
        a.ldx = pitch(a.cols);
        a.dtype = type_code(c.type);
        const int rc = abi.dequantize(&a, c.stream);
        if (rc != 0) return PyLong_FromLong(rc);
        return wrap(x);
    });
}

// (x data, x scale, w data, w scale, k, format, bias, act, residual, dtype, out) -> y
PyObject* py_mx_linear(PyObject*, PyObject* const* v, Py_ssize_t nargs) {
    return guarded(v, nargs, 11, [&]() -> PyObject* {
        const at::Tensor &x = Call::on_cuda(tensor(v[0], "x"), "x"), &xs = tensor(v[1], "x"), &w = tensor(v[2], "w"), &ws = tensor(v[3], "w");
        const Call c(x, type_of(v[9]));
        mx_linear_args a{};
        a.k = checked_cols(v[4]);
        a.format = checked_format(v[5]);
        if (a.k < 1 || w.dim() != 2 || w.size(0) < 1) refuse("x and w must have columns, and w rows");
        a.tokens = x.dim() == 2 ? x.size(0) : 0;
        a.n = w.size(0);
        a.ldx = check_scaled(c, x, xs, "x", a.tokens, a.k, a.format);
        a.ldw = check_scaled(c, w, ws, "w", a.n, a.k, a.format);
        if (v[6] != Py_None) c.vector(tensor(v[6], "bias"), "bias", a.n, c.type);
        if (v[8] != Py_None) {
            const at::Tensor& r = tensor(v[8], "residual");
            c.matrix(r, "residual", a.tokens, a.n);
            a.ldr = stride_of(r, "residual");
        }
        at::Tensor y;
        if (v[10] != Py_None) {
            y = tensor(v[10], "out");
            c.matrix(y, "out", a.tokens, a.n);
            a.ldy = stride_of(y, "out");
        } else {
            y = c.matrix(a.tokens, a.n);
            a.ldy = pitch(a.n);
        }
        a.x = x.data_ptr();
        a.x_scale = xs.data_ptr();
        a.w = w.data_ptr();
        a.w_scale = ws.data_ptr();
        a.bias = cptr(v[6], "bias");
        a.residual = cptr(v[8], "residual");
        a.y = y.data_ptr();
        a.dtype = type_code(c.type);
        a.act = integer(v[7]);
        const int rc = abi.mx_product(&a, c.stream);
        if (rc != 0) return PyLong_FromLong(rc);
        if (v[10] != Py_None) {
            wrote(y);
            return Py_NewRef(v[10]);
        }
        return wrap(y);
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
                         ENTRY("rms_norm", py_norm),
                         ENTRY("rms_norm_backward", py_norm_backward),
                         ENTRY("mx_quantize", py_quantize),
                         ENTRY("mx_dequantize", py_dequantize),
                         ENTRY("mx_linear", py_mx_linear),
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_layers", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__layers() { return PyModule_Create(&module); }
