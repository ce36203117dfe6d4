// marshal.cpp -- tensor-level calls of the entry points whose kernels take a few microseconds.
//
// What ops.py does for the others -- check that tensors are contiguous CUDA tensors of the
// expected type and shape, allocate outputs that the caller did not pass, hand addresses and the
// current stream to libbitlinear.so -- costs more host time there than such a kernel runs (one
// decoded token between two blocks: 22 us in Python, of which the launch is 5).  Here it is done
// once in C++.  No arithmetic, and nothing kept from one call for the next.
#include <torch/csrc/Dtype.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <ATen/ATen.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>

#include <algorithm>
#include <vector>

#include "../../include/bitlinear.h"

namespace {

decltype(&bitlinear_workspace_bytes) p_workspace_bytes;
decltype(&bitlinear_residual_norm) p_residual_norm;
decltype(&bitlinear_residual_norm_backward) p_residual_norm_backward;
decltype(&bitlinear_grad_norm) p_grad_norm;
decltype(&bitlinear_clip_grads) p_clip_grads;
decltype(&bitlinear_quant_weight_int8) p_quant_weight_int8;
decltype(&bitlinear_linear_int8) p_linear_int8;
decltype(&bitlinear_optimizer_step_coef) p_optimizer_step_coef;
PyObject* g_raise = nullptr;   // raises the binding's error for (entry point, status)

// Interned names of the result dictionaries' keys.
struct Keys {
    PyObject *x, *h, *xq, *sx, *xdq, *r_post, *r_pre, *dx, *dy, *dpost_gain, *dpre_gain, *dgate, *norm, *coef, *grads,
        *gamma_rows, *gamma, *wq_i8, *wq_bf16, *packed;
} K;

// The result of a call under construction, and the outputs that the caller gave.  The result holds
// what the call writes and nothing else that the caller's dictionary may hold from another call.
struct Dict {
    PyObject *d = nullptr, *given = nullptr;
    explicit Dict(PyObject* out) {
        if (PyDict_Check(out)) {
            Py_INCREF(out);
            given = out;
        } else if (out != Py_None) {
            given = PyDict_New();
            if (given == nullptr) throw python_error();
            if (!PyMapping_Check(out) || PyDict_Update(given, out) != 0) {
                Py_CLEAR(given);
                PyErr_Clear();
                PyErr_Format(PyExc_TypeError, "out must be a dict of tensors, got %s", Py_TYPE(out)->tp_name);
                throw python_error();
            }
        }
        d = PyDict_New();
        if (d == nullptr) {
            Py_CLEAR(given);
            throw python_error();
        }
    }
    Dict(const Dict&) = delete;
    ~Dict() {
        Py_XDECREF(d);
        Py_XDECREF(given);
    }
    PyObject* release() {
        PyObject* r = d;
        d = nullptr;
        return r;
    }
    // The caller's output (a borrowed reference), or nullptr: none, or None.
    PyObject* find(PyObject* key) const {
        PyObject* have = given == nullptr ? nullptr : PyDict_GetItemWithError(given, key);
        if (have == nullptr && PyErr_Occurred()) throw python_error();
        return have == Py_None ? nullptr : have;
    }
    void put(PyObject* key, PyObject* o) {
        if (PyDict_SetItem(d, key, o)) throw python_error();
    }
    void set(PyObject* key, const at::Tensor& t) {
        PyObject* o = THPVariable_Wrap(t);
        if (o == nullptr) throw python_error();
        const int bad = PyDict_SetItem(d, key, o);
        Py_DECREF(o);
        if (bad) throw python_error();
    }
};

const at::Tensor& tensor(PyObject* o, const char* name) {
    TORCH_CHECK_VALUE(THPVariable_Check(o), name, " must be a tensor");
    return THPVariable_Unpack(o);
}

// A new contiguous tensor, from the caching allocator without the dispatcher (0.5 us less a tensor).
at::Tensor fresh(at::IntArrayRef shape, at::ScalarType type, at::Device dev) {
    return at::detail::empty_cuda(shape, type, dev, std::nullopt);
}

// The address of a contiguous tensor of this type, shape and device.
void* address(const at::Tensor& t, const char* name, at::ScalarType type, at::IntArrayRef shape, at::Device dev) {
    TORCH_CHECK_VALUE(t.scalar_type() == type && t.sizes() == shape && t.device() == dev && t.is_contiguous(), name,
                      " must be a contiguous ", type, " tensor of shape ", shape, " on ", dev, ", got ",
                      t.scalar_type(), " ", t.sizes(), " on ", t.device(), t.is_contiguous() ? "" : " (not contiguous)");
    return t.data_ptr();
}
void* optional(PyObject* o, const char* name, at::ScalarType type, at::IntArrayRef shape, at::Device dev) {
    return o == Py_None ? nullptr : address(tensor(o, name), name, type, shape, dev);
}

// The output `key`: the caller's (`have`), checked, or a new one.
void* output(Dict& d, PyObject* key, const char* name, at::ScalarType type, at::IntArrayRef shape, at::Device dev,
             PyObject* have) {
    if (have != nullptr && have != Py_None) {
        void* p = address(tensor(have, name), name, type, shape, dev);
        d.put(key, have);
        return p;
    }
    const at::Tensor t = fresh(shape, type, dev);
    d.set(key, t);
    return t.data_ptr();
}
void* output(Dict& d, PyObject* key, const char* name, at::ScalarType type, at::IntArrayRef shape, at::Device dev) {
    return output(d, key, name, type, shape, dev, d.find(key));
}

double number(PyObject* o) {
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred()) throw python_error();
    return v;
}
bool truth(PyObject* o) {
    const int v = PyObject_IsTrue(o);
    if (v < 0) throw python_error();
    return v != 0;
}

bl_dtype type_code(at::ScalarType t) {
    TORCH_CHECK_VALUE(t == at::kFloat || t == at::kBFloat16, "unsupported dtype ", t);
    return t == at::kFloat ? BL_F32 : BL_BF16;
}

// A call's device made current, and its current stream.
struct On {
    c10::cuda::CUDAGuard guard;
    void* stream;
    explicit On(at::Device dev) : guard(dev), stream(c10::cuda::getCurrentCUDAStream(dev.index()).stream()) {}
};

// The library call, without the interpreter's lock (a full launch queue may hold it up).
template <typename F>
bl_status unlocked(F&& f) {
    PyThreadState* state = PyEval_SaveThread();
    const bl_status st = f();
    PyEval_RestoreThread(state);
    return st;
}

bool failed(bl_status st, const char* name) {
    if (st == BL_OK) return false;
    PyObject* r = PyObject_CallFunction(g_raise, "si", name, (int)st);
    Py_XDECREF(r);
    if (!PyErr_Occurred()) PyErr_SetString(PyExc_RuntimeError, name);
    return true;
}

// A caller's workspace, or a new one of `bytes`.
void* workspace(PyObject* ws, size_t bytes, at::Device dev, at::Tensor* own, size_t* size) {
    if (ws == Py_None) {
        *own = fresh({(int64_t)bytes}, at::kByte, dev);
        *size = bytes;
        return own->data_ptr();
    }
    const at::Tensor& t = tensor(ws, "ws");
    TORCH_CHECK_VALUE(t.device() == dev && t.is_contiguous(), "ws must be a contiguous tensor on ", dev);
    *size = t.nbytes();
    return t.data_ptr();
}

void nargs_are(Py_ssize_t n, Py_ssize_t want) { TORCH_CHECK_VALUE(n == want, "expected ", want, " arguments, got ", n); }

// ------------------------------------------------------------------------------------
// residual norms
// ------------------------------------------------------------------------------------
struct Residual {
    at::Tensor x, y;
    at::Device dev = at::kCPU;
    at::ScalarType xt, yt;
    int64_t T, N;
    void *px, *py;
    bl_gate kind = BL_GATE_NONE;
    void* gate = nullptr;

    Residual(PyObject* xo, PyObject* yo, PyObject* go) : x(tensor(xo, "x")), y(tensor(yo, "y")) {
        TORCH_CHECK_VALUE(x.is_cuda() && x.dim() == 2, "x must be a CUDA tensor [T, K]");
        dev = x.device();
        xt = x.scalar_type();
        yt = y.scalar_type();
        TORCH_CHECK_VALUE((xt == at::kFloat && (yt == at::kFloat || yt == at::kBFloat16)) ||
                              (xt == at::kBFloat16 && yt == at::kBFloat16),
                          "unsupported types: residual ", xt, ", block ", yt);
        T = x.size(0);
        N = x.size(1);
        px = address(x, "x", xt, x.sizes(), dev);
        py = address(y, "y", yt, x.sizes(), dev);
        if (go == Py_None) return;
        // [T, 1] fp32: a token's; [T, K] of y's type: an element's; [1]: a scalar; [K]: a channel's
        const at::Tensor& g = tensor(go, "gate");
        if (g.dim() == 2 && g.size(1) == 1 && (N != 1 || g.scalar_type() == at::kFloat)) {
            kind = BL_GATE_TOKEN;
            gate = address(g, "gate", at::kFloat, {T, 1}, dev);
        } else if (g.dim() == 2) {
            kind = BL_GATE_ELEMENT;
            gate = address(g, "gate", yt, {T, N}, dev);
        } else if (g.dim() == 1 && g.size(0) == 1) {
            kind = BL_GATE_SCALAR;
            gate = address(g, "gate", at::kFloat, {1}, dev);
        } else {
            kind = BL_GATE_CHANNEL;
            gate = address(g, "gate", at::kFloat, {N}, dev);
        }
    }
};

// (x, y, post_norm, g_post, gate, alpha, beta, mode, g_pre, eps_post, eps_pre, want_xdq, out)
PyObject* residual_norm(PyObject*, PyObject* const* a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    nargs_are(n, 13);
    const Residual r(a[0], a[1], a[4]);
    const bool post = truth(a[2]);
    const bool quant = PyUnicode_Check(a[7]) && PyUnicode_CompareWithASCIIString(a[7], "quant") == 0;
    const bool norm = PyUnicode_Check(a[7]) && PyUnicode_CompareWithASCIIString(a[7], "norm") == 0;
    TORCH_CHECK_VALUE(quant || norm || (PyUnicode_Check(a[7]) && PyUnicode_CompareWithASCIIString(a[7], "none") == 0),
                      "mode must be 'quant', 'norm' or 'none'");
    const auto* g_post = static_cast<const float*>(optional(a[3], "g_post", at::kFloat, {r.N}, r.dev));
    const auto* g_pre = static_cast<const float*>(optional(a[8], "g_pre", at::kFloat, {r.N}, r.dev));
    const float alpha = (float)number(a[5]), beta = (float)number(a[6]);
    const float eps_post = (float)number(a[9]), eps_pre = (float)number(a[10]);
    const bool want_xdq = truth(a[11]);
    const On on(r.dev);
    Dict o(a[12]);
    const int64_t shape[2] = {r.T, r.N}, row[1] = {r.T};
    void* x = output(o, K.x, "x", r.xt, shape, r.dev);
    void* r_post = post ? output(o, K.r_post, "r_post", at::kFloat, row, r.dev) : nullptr;
    void* r_pre = quant || norm ? output(o, K.r_pre, "r_pre", at::kFloat, row, r.dev) : nullptr;
    void* h = norm ? output(o, K.h, "h", r.yt, shape, r.dev) : nullptr;
    void* xq = quant ? output(o, K.xq, "xq", at::kChar, shape, r.dev) : nullptr;
    void* sx = quant ? output(o, K.sx, "sx", at::kFloat, row, r.dev) : nullptr;
    void* xdq = quant && (want_xdq || o.find(K.xdq) != nullptr) ? output(o, K.xdq, "xdq", r.yt, shape, r.dev) : nullptr;
    if (failed(unlocked([&] { return p_residual_norm(r.px, type_code(r.xt), r.py, type_code(r.yt), r.T, r.N, post ? 1 : 0, g_post, eps_post,
                               r.kind, r.gate, alpha, beta, g_pre, eps_pre, x, (float*)r_post, (float*)r_pre, h,
                               (int8_t*)xq, (float*)sx, xdq, on.stream); }),
               "bitlinear_residual_norm"))
        return nullptr;
    return o.release();
    END_HANDLE_TH_ERRORS
}

// (dx, dh, x, y, r_post, r_pre, g_post, gate, alpha, beta, g_pre, want_dgains, want_dgate, ws, out)
PyObject* residual_norm_backward(PyObject*, PyObject* const* a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    nargs_are(n, 15);
    const Residual r(a[2], a[3], a[7]);
    const int64_t shape[2] = {r.T, r.N}, row[1] = {r.T}, col[1] = {r.N};
    const auto* dx = static_cast<const float*>(optional(a[0], "dx", at::kFloat, shape, r.dev));
    const auto* dh = static_cast<const float*>(optional(a[1], "dh", at::kFloat, shape, r.dev));
    const auto* r_post = static_cast<const float*>(optional(a[4], "r_post", at::kFloat, row, r.dev));
    const auto* r_pre = static_cast<const float*>(optional(a[5], "r_pre", at::kFloat, row, r.dev));
    const auto* g_post = static_cast<const float*>(optional(a[6], "g_post", at::kFloat, col, r.dev));
    const auto* g_pre = static_cast<const float*>(optional(a[10], "g_pre", at::kFloat, col, r.dev));
    const float alpha = (float)number(a[8]), beta = (float)number(a[9]);
    const bool gains = truth(a[11]), want_gate = truth(a[12]);
    const bool has_post = a[4] != Py_None, has_dh = a[1] != Py_None;
    TORCH_CHECK_VALUE(!has_dh || a[5] != Py_None, "dh needs r_pre");
    const On on(r.dev);
    Dict o(a[14]);
    void* dX = output(o, K.dx, "dx", at::kFloat, shape, r.dev);
    void* dY = output(o, K.dy, "dy", r.yt, shape, r.dev);
    void* dg_post = has_post && (gains || o.find(K.dpost_gain) != nullptr) ? output(o, K.dpost_gain, "dpost_gain", at::kFloat, col, r.dev) : nullptr;
    void* dg_pre = has_dh && (gains || o.find(K.dpre_gain) != nullptr) ? output(o, K.dpre_gain, "dpre_gain", at::kFloat, col, r.dev) : nullptr;
    void* dgate = nullptr;
    if (r.gate != nullptr && (want_gate || o.find(K.dgate) != nullptr)) {
        const at::Tensor& g = THPVariable_Unpack(a[7]);
        dgate = output(o, K.dgate, "dgate", g.scalar_type(), g.sizes(), r.dev);
    }
    at::Tensor own;
    size_t ws_bytes = 0;
    void* ws = nullptr;
    if (a[13] != Py_None || dg_post != nullptr || dg_pre != nullptr ||
        (dgate != nullptr && (r.kind == BL_GATE_SCALAR || r.kind == BL_GATE_CHANNEL)))
        ws = workspace(a[13], p_workspace_bytes(r.T, 16, r.N), r.dev, &own, &ws_bytes);
    if (failed(unlocked([&] { return p_residual_norm_backward(dx, dh, r.px, type_code(r.xt), r.py, type_code(r.yt), r.T, r.N,
                                        has_post ? 1 : 0, g_post, r_post, r.kind, r.gate, alpha, beta, g_pre, r_pre,
                                        (float*)dX, dY, (float*)dg_post, (float*)dg_pre, dgate, ws, ws_bytes,
                                        on.stream); }),
               "bitlinear_residual_norm_backward"))
        return nullptr;
    return o.release();
    END_HANDLE_TH_ERRORS
}

// ------------------------------------------------------------------------------------
// gradient norm and clipping
// ------------------------------------------------------------------------------------
// Bytes that a call reads or writes.  Its blocks run in any order, so what one writes no other may
// read or write; only a gradient clipped in place is both (by one thread an element).
struct Span {
    uintptr_t lo, hi;
};
bool by_start(const Span& p, const Span& q) { return p.lo < q.lo; }
// `written` must not touch one another or `read` (both are sorted here: under a microsecond for 58 tensors).
bool disjoint(std::vector<Span>& read, std::vector<Span>& written) {
    std::sort(read.begin(), read.end(), by_start);
    std::sort(written.begin(), written.end(), by_start);
    for (size_t i = 1; i < written.size(); ++i)
        if (written[i].lo < written[i - 1].hi) return false;
    // what is read may overlap: the furthest end of all that start before the written piece's end
    size_t r = 0;
    uintptr_t end = 0;
    for (const Span& w : written) {
        for (; r < read.size() && read[r].lo < w.hi; ++r) end = std::max(end, read[r].hi);
        if (end > w.lo) return false;
    }
    return true;
}

// (clip, grads, max_norm, out, norm, coef, ws)
PyObject* grads(PyObject*, PyObject* const* a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    nargs_are(n, 7);
    const bool clip = truth(a[0]);
    struct Seq {
        PyObject* s;
        Seq(PyObject* o, const char* what) : s(PySequence_Fast(o, what)) {
            if (s == nullptr) throw python_error();
        }
        ~Seq() { Py_DECREF(s); }
        Py_ssize_t size() const { return PySequence_Fast_GET_SIZE(s); }
        PyObject* at(Py_ssize_t i) const { return PySequence_Fast_GET_ITEM(s, i); }
    };
    const Seq g(a[1], "grads must be a sequence of tensors");
    // in place: the same list (an iterator is used up by the first)
    const Seq q(a[3] == Py_None ? g.s : a[3], "out must be a sequence of tensors");
    const Py_ssize_t count = g.size();
    TORCH_CHECK_VALUE(count > 0, "grads must not be empty");
    TORCH_CHECK_VALUE(q.size() == count, "out must have ", count, " tensors, got ", q.size());
    const at::Device dev = tensor(g.at(0), "grads[0]").device();
    TORCH_CHECK_VALUE(dev.is_cuda(), "grads must be CUDA tensors");
    std::vector<const void*> ptrs(count);
    std::vector<void*> outs(count);
    // a norm into new tensors writes to nothing that the caller has
    const bool look = clip || a[4] != Py_None || a[5] != Py_None || a[6] != Py_None;
    std::vector<Span> read, written;
    if (look) {
        read.reserve(count);
        written.reserve(count + 3);
    }
    auto span = [](std::vector<Span>& to, const void* p, size_t bytes) {
        if (bytes != 0) to.push_back({reinterpret_cast<uintptr_t>(p), reinterpret_cast<uintptr_t>(p) + bytes});
    };
    std::vector<int64_t> numel(count);
    std::vector<bl_dtype> types(count);
    for (Py_ssize_t i = 0; i < count; ++i) {
        const at::Tensor& t = tensor(g.at(i), "grads");
        const at::Tensor& u = a[3] == Py_None ? t : tensor(q.at(i), "out");
        TORCH_CHECK_VALUE(t.device() == dev && t.is_contiguous() && u.device() == dev && u.is_contiguous(),
                          "gradients and outputs must be contiguous CUDA tensors on one device (number ", i, ")");
        types[i] = type_code(t.scalar_type());
        TORCH_CHECK_VALUE(u.scalar_type() == t.scalar_type() && u.numel() == t.numel(),
                          "out must have the sizes and types of grads (number ", i, ")");
        ptrs[i] = t.data_ptr();
        outs[i] = u.data_ptr();
        numel[i] = t.numel();
        const size_t bytes = numel[i] * (types[i] == BL_F32 ? 4 : 2);
        if (clip) span(written, outs[i], bytes);
        if (look && (!clip || outs[i] != ptrs[i])) span(read, ptrs[i], bytes);
    }
    const On on(dev);
    Dict o(Py_None);
    const int64_t one[1] = {1};
    auto* norm = static_cast<float*>(output(o, K.norm, "norm", at::kFloat, one, dev, a[4]));
    auto* coef = static_cast<float*>(output(o, K.coef, "coef", at::kFloat, one, dev, a[5]));
    at::Tensor own;
    size_t ws_bytes = 0;
    const size_t needed = p_workspace_bytes(1, 1, 1);
    void* ws = workspace(a[6], needed, dev, &own, &ws_bytes);
    if (a[4] != Py_None) span(written, norm, 4);
    if (a[5] != Py_None) span(written, coef, 4);
    if (a[6] != Py_None) span(written, ws, std::min(ws_bytes, needed));   // no more of it is written
    if (look)
        TORCH_CHECK_VALUE(disjoint(read, written), "outputs (norm, coef, out, the workspace) must not overlap one another or a "
                                                   "gradient; only out[i] may be grads[i] itself");
    const float max_norm = (float)number(a[2]);
    if (clip) {
        if (failed(unlocked([&] { return p_clip_grads(ptrs.data(), outs.data(), numel.data(), types.data(), count, max_norm, norm, coef, ws,
                                ws_bytes, on.stream); }),
                   "bitlinear_clip_grads"))
            return nullptr;
        o.put(K.grads, q.s);
    } else if (failed(unlocked([&] { return p_grad_norm(ptrs.data(), numel.data(), types.data(), count, max_norm, norm, coef, ws, ws_bytes,
                                  on.stream); }),
                      "bitlinear_grad_norm")) {
        return nullptr;
    }
    return o.release();
    END_HANDLE_TH_ERRORS
}

// (W, dW, m, v, step, lr, beta1, beta2, eps, weight_decay, requantize, ws, out, coef)
PyObject* optimizer_step_coef(PyObject*, PyObject* const* a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    nargs_are(n, 14);
    const at::Tensor& W = tensor(a[0], "W");
    TORCH_CHECK_VALUE(W.is_cuda() && W.dim() == 2, "W must be a CUDA tensor [N, K]");
    const at::Device dev = W.device();
    const int64_t N = W.size(0), Kd = W.size(1);
    const int64_t shape[2] = {N, Kd}, one[1] = {1}, packed[2] = {N, Kd / 4};
    auto* w = static_cast<float*>(address(W, "W", at::kFloat, shape, dev));
    auto* g = static_cast<const float*>(address(tensor(a[1], "dW"), "dW", at::kFloat, shape, dev));
    auto* m = static_cast<float*>(address(tensor(a[2], "m"), "m", at::kFloat, shape, dev));
    auto* v = static_cast<float*>(address(tensor(a[3], "v"), "v", at::kFloat, shape, dev));
    auto* step = static_cast<int32_t*>(address(tensor(a[4], "step"), "step", at::kInt, one, dev));
    auto* coef = static_cast<const float*>(address(tensor(a[13], "coef"), "coef", at::kFloat, one, dev));
    float hp[5];
    for (int i = 0; i < 5; ++i) hp[i] = (float)number(a[5 + i]);
    const On on(dev);
    Dict o(a[12]);
    const bool next = truth(a[10]);
    auto want = [&](PyObject* key, const char* name, at::ScalarType type, at::IntArrayRef sh) -> void* {
        return next || o.find(key) != nullptr ? output(o, key, name, type, sh, dev) : nullptr;
    };
    auto* gamma = static_cast<float*>(want(K.gamma, "gamma", at::kFloat, one));
    auto* q = static_cast<int8_t*>(want(K.wq_i8, "wq_i8", at::kChar, shape));
    auto* b = static_cast<uint16_t*>(want(K.wq_bf16, "wq_bf16", at::kBFloat16, shape));
    auto* p = static_cast<uint8_t*>(want(K.packed, "packed", at::kByte, packed));
    at::Tensor own;
    size_t ws_bytes = 0;
    void* ws = workspace(a[11], p_workspace_bytes(1, N, 1), dev, &own, &ws_bytes);
    if (failed(unlocked([&] {
                   return p_optimizer_step_coef(w, g, m, v, N, Kd, hp[0], hp[1], hp[2], hp[3], hp[4], coef, step, q, b,
                                                p, gamma, ws, ws_bytes, on.stream);
               }),
               "bitlinear_optimizer_step_coef"))
        return nullptr;
    return o.release();
    END_HANDLE_TH_ERRORS
}

// ------------------------------------------------------------------------------------
// 8-bit linear
// ------------------------------------------------------------------------------------
// (W, want_i8, want_bf16, out)
PyObject* quant_weight_int8(PyObject*, PyObject* const* a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    nargs_are(n, 4);
    const at::Tensor& W = tensor(a[0], "W");
    TORCH_CHECK_VALUE(W.is_cuda() && W.dim() == 2, "W must be a CUDA tensor [N, K]");
    const at::Device dev = W.device();
    const void* w = address(W, "W", at::kFloat, W.sizes(), dev);
    const int64_t shape[2] = {W.size(0), W.size(1)}, row[1] = {W.size(0)};
    const On on(dev);
    Dict o(a[3]);
    void* gm = output(o, K.gamma_rows, "gamma_rows", at::kFloat, row, dev);
    auto wanted = [&](PyObject* want, PyObject* key) { return truth(want) || o.find(key) != nullptr; };
    void* q = wanted(a[1], K.wq_i8) ? output(o, K.wq_i8, "wq_i8", at::kChar, shape, dev) : nullptr;
    void* b = wanted(a[2], K.wq_bf16) ? output(o, K.wq_bf16, "wq_bf16", at::kBFloat16, shape, dev) : nullptr;
    if (failed(unlocked([&] { return p_quant_weight_int8((const float*)w, shape[0], shape[1], (int8_t*)q, (uint16_t*)b, (float*)gm, on.stream); }),
               "bitlinear_quant_weight_int8"))
        return nullptr;
    return o.release();
    END_HANDLE_TH_ERRORS
}

// (xq, sx, wq_i8, gamma_rows, out_dtype, want_acc, y, acc) -> (y, acc)
PyObject* linear_int8(PyObject*, PyObject* const* a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    nargs_are(n, 8);
    const at::Tensor &xq = tensor(a[0], "xq"), &wq = tensor(a[2], "wq_i8");
    TORCH_CHECK_VALUE(xq.is_cuda() && xq.dim() == 2, "xq must be a CUDA tensor [T, K]");
    TORCH_CHECK_VALUE(wq.dim() == 2, "wq_i8 must be a tensor [N, K]");
    const at::Device dev = xq.device();
    const int64_t T = xq.size(0), Kd = xq.size(1), N = wq.size(0);
    const void* px = address(xq, "xq", at::kChar, {T, Kd}, dev);
    const void* ps = address(tensor(a[1], "sx"), "sx", at::kFloat, {T}, dev);
    const void* pw = address(wq, "wq_i8", at::kChar, {N, Kd}, dev);
    const void* pg = address(tensor(a[3], "gamma_rows"), "gamma_rows", at::kFloat, {N}, dev);
    const On on(dev);
    at::Tensor y, acc;
    if (a[6] != Py_None) {
        y = tensor(a[6], "y");
        type_code(y.scalar_type());
        address(y, "y", y.scalar_type(), {T, N}, dev);
    } else {
        TORCH_CHECK_VALUE(THPDtype_Check(a[4]), "out_dtype must be a torch.dtype");
        const at::ScalarType t = reinterpret_cast<THPDtype*>(a[4])->scalar_type;
        type_code(t);
        y = fresh({T, N}, t, dev);
    }
    if (a[7] != Py_None) {
        acc = tensor(a[7], "acc");
        address(acc, "acc", at::kInt, {T, N}, dev);
    } else if (truth(a[5])) {
        acc = fresh({T, N}, at::kInt, dev);
    }
    if (failed(unlocked([&] { return p_linear_int8((const int8_t*)px, (const float*)ps, T, Kd, (const int8_t*)pw, (const float*)pg, N,
                             y.data_ptr(), type_code(y.scalar_type()),
                             acc.defined() ? static_cast<int32_t*>(acc.data_ptr()) : nullptr, on.stream); }),
               "bitlinear_linear_int8"))
        return nullptr;
    PyObject* both = PyTuple_New(2);
    if (both == nullptr) throw python_error();
    PyTuple_SET_ITEM(both, 0, THPVariable_Wrap(y));
    if (acc.defined()) {
        PyTuple_SET_ITEM(both, 1, THPVariable_Wrap(acc));
    } else {
        Py_INCREF(Py_None);
        PyTuple_SET_ITEM(both, 1, Py_None);
    }
    return both;
    END_HANDLE_TH_ERRORS
}

// (addresses of the entry points in the order below, raise)
PyObject* init(PyObject*, PyObject* const* a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    nargs_are(n, 9);
    void* p[8];
    for (int i = 0; i < 8; ++i) {
        p[i] = PyLong_AsVoidPtr(a[i]);
        if (p[i] == nullptr) {
            if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, "null entry point");
            return nullptr;
        }
    }
    p_workspace_bytes = reinterpret_cast<decltype(p_workspace_bytes)>(p[0]);
    p_residual_norm = reinterpret_cast<decltype(p_residual_norm)>(p[1]);
    p_residual_norm_backward = reinterpret_cast<decltype(p_residual_norm_backward)>(p[2]);
    p_grad_norm = reinterpret_cast<decltype(p_grad_norm)>(p[3]);
    p_clip_grads = reinterpret_cast<decltype(p_clip_grads)>(p[4]);
    p_quant_weight_int8 = reinterpret_cast<decltype(p_quant_weight_int8)>(p[5]);
    p_linear_int8 = reinterpret_cast<decltype(p_linear_int8)>(p[6]);
    p_optimizer_step_coef = reinterpret_cast<decltype(p_optimizer_step_coef)>(p[7]);
    Py_INCREF(a[8]);
    Py_XDECREF(g_raise);
    g_raise = a[8];
    Py_RETURN_NONE;
    END_HANDLE_TH_ERRORS
}

#define BL_METHOD(f) \
    { #f, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f)), METH_FASTCALL, nullptr }
PyMethodDef methods[] = {BL_METHOD(init), BL_METHOD(residual_norm), BL_METHOD(residual_norm_backward), BL_METHOD(grads),
                         BL_METHOD(quant_weight_int8), BL_METHOD(linear_int8),
                         BL_METHOD(optimizer_step_coef), {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_marshal", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__marshal() {
    struct {
        PyObject** at;
        const char* name;
    } keys[] = {{&K.x, "x"}, {&K.h, "h"}, {&K.xq, "xq"}, {&K.sx, "sx"}, {&K.xdq, "xdq"}, {&K.r_post, "r_post"},
                {&K.r_pre, "r_pre"}, {&K.dx, "dx"}, {&K.dy, "dy"}, {&K.dpost_gain, "dpost_gain"},
                {&K.dpre_gain, "dpre_gain"}, {&K.dgate, "dgate"}, {&K.norm, "norm"}, {&K.coef, "coef"},
                {&K.grads, "grads"}, {&K.gamma_rows, "gamma_rows"}, {&K.wq_i8, "wq_i8"}, {&K.wq_bf16, "wq_bf16"}, {&K.gamma, "gamma"},
                {&K.packed, "packed"}};
    for (auto& k : keys) {
        *k.at = PyUnicode_InternFromString(k.name);
        if (*k.at == nullptr) return nullptr;
    }
    PyObject* m = PyModule_Create(&module);
    // what build.py looks for in the file before it is loaded
    if (m != nullptr && PyModule_AddStringConstant(m, "built_for", BL_TORCH_MARK) != 0) Py_CLEAR(m);
    return m;
}
