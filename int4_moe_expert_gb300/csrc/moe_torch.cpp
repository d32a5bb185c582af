// PyTorch binding of the handle-less operators of moe.h (module _moe_torch): checks of types, shapes,
// layouts and devices, which the C side cannot see behind its pointers, allocation of the outputs on
// the call's stream, and the call.  No step of the computation runs here.  A compiled module because
// these calls are short: an argument check or an allocation from Python costs as much as a kernel of
// the smallest sizes (token lists of 8 tokens: 20 us a call from Python, of which 5 us on the GPU).
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/ATen.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cstdarg>
#include <cstdint>
#include <cstdio>
#include <initializer_list>
#include <optional>
#include <vector>

#include "moe.h"

namespace {

PyObject *g_error = nullptr;      // MoeError(status, where, message)

// raised by a failed check; the Python error is set
struct Refused {};

[[noreturn]] void refuse(const char *where, int status, const char *fmt, ...) {
    char msg[512];
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(msg, sizeof(msg), fmt, ap);
    va_end(ap);
    PyObject *e = g_error ? PyObject_CallFunction(g_error, "iss", status, where, msg) : nullptr;
    if (e) {
        PyErr_SetObject(g_error, e);
        Py_DECREF(e);
    } else if (!PyErr_Occurred()) {
        PyErr_SetString(PyExc_RuntimeError, msg);
    }
    throw Refused{};
}

using Types = std::initializer_list<at::ScalarType>;
const Types kI32 = {at::kInt}, kF32 = {at::kFloat}, kFloats = {at::kFloat, at::kHalf, at::kBFloat16},
            kF8 = {at::kFloat8_e4m3fn, at::kByte}, kMask = {at::kBool, at::kByte};

int dtype_code(at::ScalarType t) {
    return t == at::kFloat ? MOE_DTYPE_F32 : t == at::kHalf ? MOE_DTYPE_F16 : t == at::kBFloat16 ? MOE_DTYPE_BF16 : -1;
}
int64_t blocks(int64_t n) { return (n + 127) / 128; }

// One call: the device of its first tensor (which has to be the current one), its stream, and the
// checks of its arguments.
class Call {
public:
    // stream: None (the current one) or a handle
    Call(const char *where, PyObject *const *args, Py_ssize_t n, Py_ssize_t want) : where_(where) {
        if (n != want) refuse(where, MOE_ERR_INVALID, "%zd arguments, need %zd", n, want);
        if (!PyList_Check(args[0]) || PyList_GET_SIZE(args[0])) {       // a list: its first tensor
            const at::Tensor &t = tensor(PyList_Check(args[0]) ? PyList_GET_ITEM(args[0], 0) : args[0], "the first argument");
            if (!t.is_cuda()) fail("the tensors must be on a CUDA device");
            dev_ = t.get_device();
        } else {
            dev_ = c10::cuda::current_device();
        }
        if (dev_ != c10::cuda::current_device())
            fail("the tensors are on cuda:%d, the current device is cuda:%d", dev_, (int)c10::cuda::current_device());
        const auto now = c10::cuda::getCurrentCUDAStream(dev_);
        stream_ = now.stream();
        PyObject *s = args[n - 1];
        if (s != Py_None) {
            void *h = PyLong_AsVoidPtr(s);
            if (!h && PyErr_Occurred()) throw Refused{};
            if (h != (void *)stream_) {      // outputs are allocated for the stream that they are used on
                stream_ = static_cast<cudaStream_t>(h);
                guard_.emplace(h ? c10::cuda::getStreamFromExternal(stream_, dev_) : c10::cuda::getDefaultCUDAStream(dev_));
            }
        }
    }
    template <typename... A>
    [[noreturn]] void fail(const char *fmt, A... a) const { refuse(where_, MOE_ERR_INVALID, fmt, a...); }
    template <typename... A>
    [[noreturn]] void unsupported(const char *fmt, A... a) const { refuse(where_, MOE_ERR_UNSUPPORTED, fmt, a...); }

    const at::Tensor &tensor(PyObject *o, const char *name) const {
        if (!THPVariable_Check(o)) fail("%s: need a tensor", name);
        return THPVariable_Unpack(o);
    }
    const at::Tensor &dims(PyObject *o, const char *name, int64_t n) const {
        const at::Tensor &t = tensor(o, name);
        if (t.dim() != n) fail("%s: need a tensor of %d dimensions, got %d", name, (int)n, (int)t.dim());
        return t;
    }
    // on the device, of one of `types` and of `shape`, contiguous or (rows) each row so; its address
    void *need(const at::Tensor &t, const char *name, Types types, at::IntArrayRef shape, bool rows = false) const {
        bool is = false;
        for (auto s : types) is = is || t.scalar_type() == s;
        if (!is) fail("%s: its type is %s", name, at::toString(t.scalar_type()));
        if (!t.is_cuda() || t.get_device() != dev_) fail("%s: is on %s, the call on cuda:%d", name, t.device().str().c_str(), dev_);
        if (t.layout() != at::kStrided || !t.sizes().equals(shape)) {
            std::string got = "(", want = "(";
            for (auto v : t.sizes()) got += std::to_string(v) + ",";
            for (auto v : shape) want += std::to_string(v) + ",";
            fail("%s: need shape %s), got %s)", name, want.c_str(), got.c_str());
        }
        if (!t.is_contiguous() && !(rows && t.stride(-1) == 1 && t.stride(0) >= t.size(-1)))
            fail("%s: need %s", name, rows ? "contiguous rows" : "a contiguous tensor");
        return t.data_ptr();
    }
    void *need(PyObject *o, const char *name, Types types, at::IntArrayRef shape, bool rows = false) const {
        return need(tensor(o, name), name, types, shape, rows);
    }
    int32_t size(int64_t v, const char *name) const {
        if (v < 0 || v > INT32_MAX) refuse(where_, MOE_ERR_UNSUPPORTED, "%s: %lld does not fit 32 bits", name, (long long)v);
        return (int32_t)v;
    }
    int32_t integer(PyObject *o, const char *name) const {
        PyObject *i = PyBool_Check(o) ? nullptr : PyNumber_Index(o);
        if (!i) {
            PyErr_Clear();
            fail("%s: need an integer", name);
        }
        int over = 0;
        const long long v = PyLong_AsLongLongAndOverflow(i, &over);
        Py_DECREF(i);
        if (over || v < INT32_MIN || v > INT32_MAX) fail("%s: does not fit 32 bits", name);
        return (int32_t)v;
    }
    float real(PyObject *o, const char *name) const { return (float)real64(o, name); }
    double real64(PyObject *o, const char *name) const {
        const double v = PyFloat_AsDouble(o);
        if (v == -1.0 && PyErr_Occurred()) {
            PyErr_Clear();
            fail("%s: need a number", name);
        }
        return v;
    }
    bool flag(PyObject *o) const {
        const int v = PyObject_IsTrue(o);
        if (v < 0) throw Refused{};
        return v != 0;
    }
    at::Tensor empty(at::IntArrayRef shape, at::ScalarType type) const {
        return at::empty(shape, at::TensorOptions().dtype(type).device(at::Device(at::kCUDA, (c10::DeviceIndex)dev_)));
    }
    // A new tensor that the call writes whole, straight from the allocator: past the dispatcher (a norm of 4 rows,
    // five outputs: 8.8 us a call through it, 6.9 us so)
    at::Tensor fresh(at::IntArrayRef shape, at::ScalarType type) const {
        return at::Tensor(at::detail::empty_cuda(shape, type, at::Device(at::kCUDA, (c10::DeviceIndex)dev_), std::nullopt));
    }
    // out, or a new tensor of `shape` and of the asked (or the default) type
    at::Tensor output(PyObject *out, PyObject *type, at::IntArrayRef shape, at::ScalarType usual, bool rows, bool whole = false) const {
        std::optional<at::ScalarType> asked;
        if (type != Py_None) {
            if (!THPDtype_Check(type)) fail("out_dtype: need a torch.dtype");
            asked = reinterpret_cast<THPDtype *>(type)->scalar_type;
            if (dtype_code(*asked) < 0) fail("out_dtype: need float32, float16 or bfloat16");
        }
        if (out == Py_None) return whole ? fresh(shape, asked.value_or(usual)) : empty(shape, asked.value_or(usual));
        const at::Tensor &t = tensor(out, "out");
        if (asked && t.scalar_type() != *asked) fail("out is %s, out_dtype another type", at::toString(t.scalar_type()));
        need(t, "out", kFloats, shape, rows);
        return t;
    }
    static int64_t row_stride(const at::Tensor &t) { return t.size(0) > 1 ? t.stride(0) : t.size(1); }
    void *stream() const { return stream_; }
    void check(moe_status s) const {
        if (s != MOE_OK) refuse(where_, (int)s, "%s", moe_last_error());
    }

private:
    const char *where_;
    int dev_ = 0;
    cudaStream_t stream_ = nullptr;
    std::optional<c10::cuda::CUDAStreamGuard> guard_;
};

PyObject *tuple(std::initializer_list<at::Tensor> ts) {
    PyObject *r = PyTuple_New((Py_ssize_t)ts.size());
    if (!r) return nullptr;
    Py_ssize_t i = 0;
    for (const auto &t : ts) PyTuple_SET_ITEM(r, i++, THPVariable_Wrap(t));
    return r;
}

// topk_idx, n_experts, align, stream
PyObject *expert_lists(PyObject *const *a, Py_ssize_t n) {
    const Call c("moe_expert_lists", a, n, 4);
    const at::Tensor &idx = c.dims(a[0], "topk_idx", 2);
    const void *p = c.need(idx, "topk_idx", kI32, idx.sizes());
    const int32_t T = c.size(idx.size(0), "tokens"), K = c.size(idx.size(1), "top_k");
    const int32_t E = c.integer(a[1], "n_experts"), align = c.integer(a[2], "align");
    // sizes that the call refuses allocate nothing first
    const int64_t room = moe_expert_lists_rows(T, K, E, align);
    const bool ok = room >= 0 && room < (1ll << 31) && E <= 1024 && K <= 1024 && align <= 4096;
    at::Tensor counts = c.empty({ok ? E : 0}, at::kInt), off = c.empty({ok ? E + 1 : 0}, at::kInt), rows = c.empty({ok ? room : 0}, at::kInt),
               pos = c.empty(idx.sizes(), at::kInt), ws;
    const size_t need = ok ? moe_expert_lists_workspace(T, K, E) : 0;
    if (need) ws = c.empty({(int64_t)need}, at::kByte);
    c.check(moe_expert_lists(static_cast<const int32_t *>(p), T, K, E, align, counts.data_ptr<int32_t>(), off.data_ptr<int32_t>(),
                             rows.data_ptr<int32_t>(), pos.data_ptr<int32_t>(), need ? ws.data_ptr() : nullptr, need, c.stream()));
    return tuple({counts, off, rows, pos});
}

struct Balance {
    const void *x;
    int64_t ld;
    int32_t T, E, S = 1, dtype;
    const int32_t *seq = nullptr;
    const uint8_t *mask = nullptr;
    Balance(const Call &c, PyObject *logits, PyObject *seq_o, PyObject *mask_o) {
        const at::Tensor &t = c.dims(logits, "logits", 2);
        x = c.need(t, "logits", kFloats, t.sizes(), true);
        dtype = dtype_code(t.scalar_type());
        ld = Call::row_stride(t);
        T = c.size(t.size(0), "tokens");
        if (T > MOE_BALANCE_MAX_TOKENS) c.unsupported("logits: %d tokens, need %d or fewer", T, MOE_BALANCE_MAX_TOKENS);
        E = c.size(t.size(1), "experts");
        if (seq_o != Py_None) {
            const at::Tensor &s = c.dims(seq_o, "seq_offsets", 1);
            seq = static_cast<const int32_t *>(c.need(s, "seq_offsets", kI32, s.sizes()));
            if (s.size(0) < 2) c.fail("seq_offsets: need at least two entries");
            S = c.size(s.size(0) - 1, "sequences");
        }
        if (mask_o != Py_None) mask = static_cast<const uint8_t *>(c.need(mask_o, "mask", kMask, {t.size(0)}));
    }
};

// logits, topk_idx, coef, score_func, seq_offsets, mask, stream
PyObject *balance_forward(PyObject *const *a, Py_ssize_t n) {
    const Call c("moe_balance_forward", a, n, 7);
    const Balance b(c, a[0], a[4], a[5]);
    const at::Tensor &idx = c.dims(a[1], "topk_idx", 2);
    const void *p = c.need(idx, "topk_idx", kI32, {b.T, idx.size(1)});
    // sizes that the call refuses allocate nothing first
    const int32_t S = b.S <= 65535 && b.E <= 1024 ? b.S : 0;
    at::Tensor loss = c.empty({1}, at::kFloat), counts = c.empty({S, b.E}, at::kInt), sums = c.empty({S, b.E}, at::kFloat),
               tokens = c.empty({S}, at::kInt);
    const size_t need = S ? moe_balance_workspace(b.T, b.E, S) : 0;
    at::Tensor ws = c.empty({(int64_t)need}, at::kByte);
    c.check(moe_balance_forward(b.x, b.dtype, b.ld, b.T, b.E, static_cast<const int32_t *>(p), c.size(idx.size(1), "top_k"),
                                c.integer(a[3], "score_func"), c.real(a[2], "coef"), b.seq, b.S, b.mask, loss.data_ptr<float>(),
                                counts.data_ptr<int32_t>(), sums.data_ptr<float>(), tokens.data_ptr<int32_t>(), ws.data_ptr(), need,
                                c.stream()));
    return tuple({loss, counts, sums, tokens});
}

// logits, top_k, counts, tokens, coef, score_func, seq_offsets, mask, grad_loss, out, stream
PyObject *balance_backward(PyObject *const *a, Py_ssize_t n) {
    const Call c("moe_balance_backward", a, n, 11);
    const Balance b(c, a[0], a[6], a[7]);
    const void *counts = c.need(a[2], "counts", kI32, {b.S, b.E}), *tokens = c.need(a[3], "tokens", kI32, {b.S}), *g = nullptr;
    if (a[8] != Py_None) {
        const at::Tensor &t = c.tensor(a[8], "grad_loss");
        if (t.numel() != 1) c.fail("grad_loss: need one value");
        g = c.need(t, "grad_loss", kF32, t.sizes());
    }
    const at::ScalarType type = c.tensor(a[0], "logits").scalar_type();
    at::Tensor out = c.output(a[9], Py_None, {b.T, b.E}, type, true);
    if (out.scalar_type() != type) c.fail("out: its type is %s, that of logits %s", at::toString(out.scalar_type()), at::toString(type));
    c.check(moe_balance_backward(b.x, b.dtype, b.ld, b.T, b.E, c.integer(a[1], "top_k"), c.integer(a[5], "score_func"), c.real(a[4], "coef"),
                                 static_cast<const int32_t *>(counts), static_cast<const int32_t *>(tokens), b.seq, b.S, b.mask,
                                 static_cast<const float *>(g), out.data_ptr(), Call::row_stride(out), a[9] == Py_None, c.stream()));
    return THPVariable_Wrap(out);
}

// x, rows, transposed, stream
PyObject *fp8_quantize(PyObject *const *a, Py_ssize_t n) {
    const Call c("moe_fp8_quantize", a, n, 4);
    const at::Tensor &x = c.dims(a[0], "x", 2);
    const void *p = c.need(x, "x", kFloats, x.sizes(), true);
    const int64_t w = x.size(1);
    int64_t R = x.size(0);
    const int32_t *rows = nullptr;
    if (a[1] != Py_None) {
        const at::Tensor &r = c.dims(a[1], "rows", 1);
        rows = static_cast<const int32_t *>(c.need(r, "rows", kI32, r.sizes()));
        R = r.size(0);
    }
    const int both = PyObject_IsTrue(a[2]);
    if (both < 0) throw Refused{};
    const int64_t rb = blocks(R);
    at::Tensor q = c.empty({R, w}, at::kFloat8_e4m3fn), s = c.empty({blocks(w), R}, at::kFloat), qt, st;
    if (both) {
        qt = c.empty({w, rb * 128}, at::kFloat8_e4m3fn);
        st = c.empty({rb, w}, at::kFloat);
    }
    c.check(moe_fp8_quantize(p, dtype_code(x.scalar_type()), Call::row_stride(x), c.size(x.size(0), "rows of x"), c.size(w, "width"), rows,
                             c.size(R, "rows"), static_cast<uint8_t *>(q.data_ptr()), s.data_ptr<float>(),
                             both && R ? static_cast<uint8_t *>(qt.data_ptr()) : nullptr, both && R ? st.data_ptr<float>() : nullptr,
                             c.stream()));
    return both ? tuple({q, s, qt, st}) : tuple({q, s});
}

// w, transposed, stream
PyObject *fp8_quantize_weights(PyObject *const *a, Py_ssize_t n) {
    const Call c("moe_fp8_quantize_weights", a, n, 3);
    const at::Tensor &w = c.tensor(a[0], "w");
    if (w.dim() != 2 && w.dim() != 3) c.fail("w: need a tensor of 2 or 3 dimensions, got %d", (int)w.dim());
    const void *p = c.need(w, "w", kFloats, w.sizes());
    const bool lead = w.dim() == 3;
    const int64_t E = lead ? w.size(0) : 1, N = w.size(-2), K = w.size(-1);
    auto shape = [&](int64_t r, int64_t k) { return lead ? std::vector<int64_t>{E, r, k} : std::vector<int64_t>{r, k}; };
    const int both = PyObject_IsTrue(a[1]);
    if (both < 0) throw Refused{};
    at::Tensor q = c.empty(shape(N, K), at::kFloat8_e4m3fn), s = c.empty(shape(blocks(N), blocks(K)), at::kFloat), qt, st;
    if (both) {
        qt = c.empty(shape(K, N), at::kFloat8_e4m3fn);
        st = c.empty(shape(blocks(K), blocks(N)), at::kFloat);
    }
    c.check(moe_fp8_quantize_weights(p, dtype_code(w.scalar_type()), c.size(E, "E"), c.size(N, "N"), c.size(K, "K"),
                                     static_cast<uint8_t *>(q.data_ptr()), s.data_ptr<float>(),
                                     both ? static_cast<uint8_t *>(qt.data_ptr()) : nullptr, both ? st.data_ptr<float>() : nullptr, c.stream()));
    return both ? tuple({q, s, qt, st}) : tuple({q, s});
}

// x, x_scale, w, w_scale, offsets, out, out_dtype, stream
PyObject *fp8_matmul(PyObject *const *a, Py_ssize_t n) {
    const Call c("moe_fp8_matmul", a, n, 8);
    const at::Tensor &x = c.dims(a[0], "x", 2);
    const int64_t R = x.size(0), K = x.size(1), kb = blocks(K);
    const void *px = c.need(x, "x", kF8, x.sizes()), *pw, *ps, *off = nullptr;
    int64_t E = 1, N;
    if (a[4] == Py_None) {
        const at::Tensor &w = c.dims(a[2], "w", 2);
        N = w.size(0);
        pw = c.need(w, "w", kF8, {N, K});
        ps = c.need(a[3], "w_scale", kF32, {blocks(N), kb});
    } else {
        const at::Tensor &w = c.dims(a[2], "w", 3);
        E = w.size(0);
        N = w.size(1);
        pw = c.need(w, "w", kF8, {E, N, K});
        ps = c.need(a[3], "w_scale", kF32, {E, blocks(N), kb});
        off = c.need(a[4], "offsets", kI32, {E + 1});
    }
    const void *pxs = c.need(a[1], "x_scale", kF32, {kb, R});
    at::Tensor out = c.output(a[5], a[6], {R, N}, at::kBFloat16, true);
    c.check(moe_fp8_matmul(static_cast<const uint8_t *>(px), static_cast<const float *>(pxs), c.size(R, "rows"),
                           static_cast<const uint8_t *>(pw), static_cast<const float *>(ps), c.size(E, "E"), c.size(N, "N"), c.size(K, "K"),
                           static_cast<const int32_t *>(off), out.data_ptr(), dtype_code(out.scalar_type()), Call::row_stride(out), c.stream()));
    return THPVariable_Wrap(out);
}

// xt, xt_scale, dyt, dyt_scale, offsets, out, out_dtype, stream
PyObject *fp8_wgrad(PyObject *const *a, Py_ssize_t n) {
    const Call c("moe_fp8_wgrad", a, n, 8);
    const at::Tensor &xt = c.dims(a[0], "xt", 2), &dyt = c.dims(a[2], "dyt", 2);
    const int64_t K = xt.size(0), R = xt.size(1), N = dyt.size(0);
    const void *px = c.need(xt, "xt", kF8, {K, R}), *pd = c.need(dyt, "dyt", kF8, {N, R});
    const void *pxs = c.need(a[1], "xt_scale", kF32, {R / 128, K}), *pds = c.need(a[3], "dyt_scale", kF32, {R / 128, N}), *off = nullptr;
    int64_t E = 1;
    std::vector<int64_t> shape{N, K};
    if (a[4] != Py_None) {
        const at::Tensor &o = c.dims(a[4], "offsets", 1);
        off = c.need(o, "offsets", kI32, o.sizes());
        E = o.size(0) - 1;
        if (E < 1) c.fail("offsets: need at least two entries");
        shape = {E, N, K};
    }
    at::Tensor out = c.output(a[5], a[6], shape, at::kFloat, false);
    c.check(moe_fp8_wgrad(static_cast<const uint8_t *>(px), static_cast<const float *>(pxs), static_cast<const uint8_t *>(pd),
                          static_cast<const float *>(pds), c.size(R, "rows"), c.size(N, "N"), c.size(K, "K"), c.size(E, "E"),
                          static_cast<const int32_t *>(off), out.data_ptr(), dtype_code(out.scalar_type()), c.stream()));
    return THPVariable_Wrap(out);
}

// logits, top_k, bias, score_func, n_group, topk_group, norm_topk, routed_scale, mask, stream
PyObject *route_forward(PyObject *const *a, Py_ssize_t n) {
    const Call c("moe_route_forward", a, n, 10);
    const at::Tensor &x = c.dims(a[0], "logits", 2);
    const void *p = c.need(x, "logits", kFloats, x.sizes(), true);
    const int32_t T = c.size(x.size(0), "tokens"), E = c.size(x.size(1), "experts"), K = c.integer(a[1], "top_k");
    const float *bias = a[2] == Py_None ? nullptr : static_cast<const float *>(c.need(a[2], "bias", kF32, {E}));
    const uint8_t *mask = a[8] == Py_None ? nullptr : static_cast<const uint8_t *>(c.need(a[8], "mask", kMask, {T}));
    const int64_t k = K >= 1 && K <= E ? K : 0;      // sizes that the call refuses allocate nothing first
    at::Tensor idx = c.fresh({T, k}, at::kInt), w = c.fresh({T, k}, at::kFloat);
    c.check(moe_route_forward(p, dtype_code(x.scalar_type()), Call::row_stride(x), T, E, bias, K, c.integer(a[3], "score_func"),
                              c.integer(a[4], "n_group"), c.integer(a[5], "topk_group"), c.flag(a[6]), c.real(a[7], "routed_scale"), mask,
                              idx.data_ptr<int32_t>(), w.data_ptr<float>(), c.stream()));
    return tuple({idx, w});
}

// logits, topk_idx, grad_w, score_func, norm_topk, routed_scale, out, accumulate, stream
PyObject *route_backward(PyObject *const *a, Py_ssize_t n) {
    const Call c("moe_route_backward", a, n, 9);
    const at::Tensor &x = c.dims(a[0], "logits", 2), &idx = c.dims(a[1], "topk_idx", 2);
    const void *p = c.need(x, "logits", kFloats, x.sizes(), true);
    const int32_t T = c.size(x.size(0), "tokens"), E = c.size(x.size(1), "experts"), K = c.size(idx.size(1), "top_k");
    const void *pi = c.need(idx, "topk_idx", kI32, {T, K}), *pg = c.need(a[2], "grad_w", kF32, {T, K});
    const bool add = c.flag(a[7]);
    if (add && a[6] == Py_None) c.fail("accumulate: need out");
    at::Tensor out = c.output(a[6], Py_None, {T, E}, x.scalar_type(), true, true);
    if (out.scalar_type() != x.scalar_type())
        c.fail("out: its type is %s, that of logits %s", at::toString(out.scalar_type()), at::toString(x.scalar_type()));
    c.check(moe_route_backward(p, dtype_code(x.scalar_type()), Call::row_stride(x), T, E, static_cast<const int32_t *>(pi), K,
                               c.integer(a[3], "score_func"), c.flag(a[4]), c.real(a[5], "routed_scale"), static_cast<const float *>(pg),
                               out.data_ptr(), Call::row_stride(out), add, c.stream()));
    return THPVariable_Wrap(out);
}

// the norm's weight: float32 or the type of x
struct NormWeight {
    const void *p = nullptr;
    int32_t dtype = MOE_DTYPE_F32;
    NormWeight(const Call &c, PyObject *o, const at::Tensor &x) {
        if (o == Py_None) return;
        const at::Tensor &t = c.tensor(o, "weight");
        p = c.need(t, "weight", {at::kFloat, x.scalar_type()}, {x.size(1)});
        dtype = dtype_code(t.scalar_type());
    }
};

// x, residual, weight, eps, values, quantize, out, stream
PyObject *norm_forward(PyObject *const *a, Py_ssize_t n) {
    const Call c("moe_norm_forward", a, n, 8);
    const at::Tensor &x = c.dims(a[0], "x", 2);
    const void *p = c.need(x, "x", kFloats, x.sizes(), true), *res = nullptr;
    const NormWeight w(c, a[2], x);
    const bool values = c.flag(a[4]), quant = c.flag(a[5]);
    const double eps = c.real64(a[3], "eps");
    const int32_t T = c.size(x.size(0), "tokens"), H = c.size(x.size(1), "width");
    at::Tensor h = x;
    int64_t ldr = H;
    if (a[1] != Py_None) {
        const at::Tensor &r = c.tensor(a[1], "residual");
        res = c.need(r, "residual", {at::kFloat, x.scalar_type()}, x.sizes(), true);
        ldr = Call::row_stride(r);
        h = c.output(a[6], Py_None, x.sizes(), r.scalar_type(), true, true);
        if (h.scalar_type() != r.scalar_type())
            c.fail("out: its type is %s, that of residual %s", at::toString(h.scalar_type()), at::toString(r.scalar_type()));
    } else if (a[6] != Py_None) {
        c.fail("out: is the sum with a residual, and there is none");
    }
    at::Tensor y, codes, scales, rstd = c.fresh({T}, at::kFloat);
    if (values) y = c.fresh(x.sizes(), x.scalar_type());
    if (quant) {
        codes = c.fresh(x.sizes(), at::kFloat8_e4m3fn);
        scales = c.fresh({blocks(H), T}, at::kFloat);
    }
    c.check(moe_norm_forward(p, dtype_code(x.scalar_type()), Call::row_stride(x), res, dtype_code(h.scalar_type()), ldr, w.p, w.dtype, T, H, eps,
                             res ? h.data_ptr() : nullptr, Call::row_stride(h), values ? y.data_ptr() : nullptr, H, rstd.data_ptr<float>(),
                             quant && T ? static_cast<uint8_t *>(codes.data_ptr()) : nullptr, quant && T ? scales.data_ptr<float>() : nullptr,
                             c.stream()));
    return quant ? tuple({y, h, rstd, codes, scales}) : tuple({y, h, rstd});
}

// dy, h, rstd, weight, grad_h, out, stream
PyObject *norm_backward(PyObject *const *a, Py_ssize_t n) {
    const Call c("moe_norm_backward", a, n, 7);
    const at::Tensor &dy = c.dims(a[0], "dy", 2), &h = c.tensor(a[1], "h");
    const void *pd = c.need(dy, "dy", kFloats, dy.sizes(), true), *ph = c.need(h, "h", {at::kFloat, dy.scalar_type()}, dy.sizes(), true), *pg = nullptr;
    const int32_t T = c.size(dy.size(0), "tokens"), H = c.size(dy.size(1), "width");
    const void *pr = c.need(a[2], "rstd", kF32, {T});
    const NormWeight w(c, a[3], dy);
    int64_t ldg = H;
    if (a[4] != Py_None) {
        const at::Tensor &g = c.tensor(a[4], "grad_h");
        pg = c.need(g, "grad_h", {h.scalar_type()}, dy.sizes(), true);
        ldg = Call::row_stride(g);
    }
    at::Tensor out = c.output(a[5], Py_None, dy.sizes(), h.scalar_type(), true, true), dw, ws;
    if (out.scalar_type() != h.scalar_type())
        c.fail("out: its type is %s, that of h %s", at::toString(out.scalar_type()), at::toString(h.scalar_type()));
    const size_t need = w.p ? moe_norm_workspace(T, H) : 0;
    if (w.p) dw = c.fresh({H}, at::kFloat);
    if (need) ws = c.fresh({(int64_t)need}, at::kByte);
    c.check(moe_norm_backward(pd, dtype_code(dy.scalar_type()), Call::row_stride(dy), ph, dtype_code(h.scalar_type()), Call::row_stride(h),
                              static_cast<const float *>(pr), w.p, w.dtype, pg, ldg, T, H, out.data_ptr(), Call::row_stride(out),
                              w.p ? dw.data_ptr<float>() : nullptr, need ? ws.data_ptr() : nullptr, need, c.stream()));
    return tuple({out, dw});
}

struct Combine {
    const int32_t *pos;
    const float *w = nullptr;
    int32_t T, K;
    Combine(const Call &c, PyObject *pos_o, PyObject *w_o) {
        const at::Tensor &t = c.dims(pos_o, "pos", 2);
        pos = static_cast<const int32_t *>(c.need(t, "pos", kI32, t.sizes()));
        T = c.size(t.size(0), "tokens");
        K = c.size(t.size(1), "top_k");
        if (w_o != Py_None) w = static_cast<const float *>(c.need(w_o, "topk_w", kF32, {T, K}));
    }
};

// rows, pos, topk_w, add, out, out_dtype, stream
PyObject *combine_forward(PyObject *const *a, Py_ssize_t n) {
    const Call c("moe_combine_forward", a, n, 7);
    const at::Tensor &r = c.dims(a[0], "rows", 2);
    const void *p = c.need(r, "rows", kFloats, r.sizes(), true), *add = nullptr;
    const Combine q(c, a[1], a[2]);
    const int32_t R = c.size(r.size(0), "rows"), N = c.size(r.size(1), "width");
    at::Tensor out = c.output(a[4], a[5], {q.T, N}, a[3] == Py_None ? r.scalar_type() : c.tensor(a[3], "add").scalar_type(), true, true);
    int64_t ldadd = N;
    if (a[3] != Py_None) {
        const at::Tensor &t = c.tensor(a[3], "add");
        add = c.need(t, "add", {out.scalar_type()}, {q.T, N}, true);
        ldadd = Call::row_stride(t);
    }
    c.check(moe_combine_forward(p, dtype_code(r.scalar_type()), Call::row_stride(r), R, N, q.pos, q.T, q.K, q.w, add, ldadd, out.data_ptr(),
                                dtype_code(out.scalar_type()), Call::row_stride(out), c.stream()));
    return THPVariable_Wrap(out);
}

// dy, rows, pos, tokens, topk_w, out, stream
PyObject *combine_backward(PyObject *const *a, Py_ssize_t n) {
    const Call c("moe_combine_backward", a, n, 7);
    const at::Tensor &dy = c.dims(a[0], "dy", 2), &r = c.dims(a[1], "rows", 2);
    const Combine q(c, a[2], a[4]);
    const int32_t R = c.size(r.size(0), "rows"), N = c.size(r.size(1), "width");
    const void *pd = c.need(dy, "dy", kFloats, {q.T, N}, true), *pr = c.need(r, "rows", {dy.scalar_type()}, r.sizes(), true);
    const void *pt = c.need(a[3], "tokens", kI32, {R});
    at::Tensor out = c.output(a[5], Py_None, r.sizes(), r.scalar_type(), true, true), dw = c.fresh({q.T, q.K}, at::kFloat);
    if (out.scalar_type() != r.scalar_type())
        c.fail("out: its type is %s, that of rows %s", at::toString(out.scalar_type()), at::toString(r.scalar_type()));
    c.check(moe_combine_backward(pd, dtype_code(dy.scalar_type()), Call::row_stride(dy), pr, Call::row_stride(r), R, N, q.pos, q.T, q.K,
                                 static_cast<const int32_t *>(pt), q.w, out.data_ptr(), Call::row_stride(out), dw.data_ptr<float>(), c.stream()));
    return tuple({out, dw});
}

// a list of gradients: float tensors on the device whose elements lie together, in any order
struct Grads {
    std::vector<const void *> p;
    std::vector<int32_t> dtype;
    std::vector<int64_t> n;
    Grads(const Call &c, PyObject *list) {
        const Py_ssize_t count = PyList_GET_SIZE(list);
        p.reserve(count);
        dtype.reserve(count);
        n.reserve(count);
        for (Py_ssize_t i = 0; i < count; i++) {
            const at::Tensor &t = c.tensor(PyList_GET_ITEM(list, i), "grads");
            if (t.layout() != at::kStrided || !t.is_non_overlapping_and_dense()) c.fail("grads: tensor %zd has gaps between its elements", i);
            if (!t.is_cuda() || t.get_device() != c10::cuda::current_device())
                c.fail("grads: tensor %zd is on %s, the call on cuda:%d", i, t.device().str().c_str(), (int)c10::cuda::current_device());
            const int d = dtype_code(t.scalar_type());
            if (d < 0) c.fail("grads: the type of tensor %zd is %s", i, at::toString(t.scalar_type()));
            p.push_back(t.data_ptr());
            dtype.push_back(d);
            n.push_back(t.numel());
        }
    }
};

// grads, stream
PyObject *grad_norm(PyObject *const *a, Py_ssize_t n) {
    if (n < 1 || !PyList_Check(a[0])) refuse("moe_grad_norm", MOE_ERR_INVALID, "grads: need a list of tensors");
    const Call c("moe_grad_norm", a, n, 2);
    const Grads g(c, a[0]);
    at::Tensor norm = c.fresh({1}, at::kFloat);
    const size_t need = moe_grad_norm_workspace(c.size((int64_t)g.p.size(), "grads"));
    at::Tensor ws = c.fresh({(int64_t)need}, at::kByte);
    c.check(moe_grad_norm((int32_t)g.p.size(), g.p.data(), g.dtype.data(), g.n.data(), norm.data_ptr<float>(), ws.data_ptr(), need, c.stream()));
    return THPVariable_Wrap(norm);
}

// grads, norm, max_norm, out, stream
PyObject *grad_clip(PyObject *const *a, Py_ssize_t n) {
    if (n < 4 || !PyList_Check(a[0]) || (a[3] != Py_None && !PyList_Check(a[3])))
        refuse("moe_grad_clip", MOE_ERR_INVALID, "grads, out: need lists of tensors");
    const Call c("moe_grad_clip", a, n, 5);
    const Grads g(c, a[0]);
    const at::Tensor &norm = c.tensor(a[1], "norm");
    if (norm.numel() != 1) c.fail("norm: need one value");
    const void *pn = c.need(norm, "norm", kF32, norm.sizes());
    std::vector<void *> out;
    if (a[3] != Py_None) {
        const Grads o(c, a[3]);
        if (o.p.size() != g.p.size()) c.fail("out: %zu tensors, grads has %zu", o.p.size(), g.p.size());
        for (size_t i = 0; i < o.p.size(); i++) {
            const at::Tensor &s = THPVariable_Unpack(PyList_GET_ITEM(a[0], i)), &t = THPVariable_Unpack(PyList_GET_ITEM(a[3], i));
            if (s.scalar_type() != t.scalar_type() || !s.sizes().equals(t.sizes()) || !s.strides().equals(t.strides()))
                c.fail("out: tensor %zu differs from its gradient in type, shape or strides", i);
            out.push_back(const_cast<void *>(o.p[i]));
        }
    }
    c.check(moe_grad_clip(c.size((int64_t)g.p.size(), "grads"), g.p.data(), g.dtype.data(), g.n.data(), static_cast<const float *>(pn),
                          c.real(a[2], "max_norm"), a[3] != Py_None ? out.data() : nullptr, c.stream()));
    Py_RETURN_NONE;
}

template <PyObject *(*F)(PyObject *const *, Py_ssize_t)>
PyObject *entry(PyObject *, PyObject *const *args, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    try {
        return F(args, n);
    } catch (const Refused &) {
        return nullptr;
    }
    END_HANDLE_TH_ERRORS
}

PyObject *set_error(PyObject *, PyObject *cls) {
    Py_INCREF(cls);
    Py_XSETREF(g_error, cls);
    Py_RETURN_NONE;
}

#define MOE_ENTRY(f) {#f, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(entry<f>)), METH_FASTCALL, nullptr}
PyMethodDef kMethods[] = {MOE_ENTRY(expert_lists), MOE_ENTRY(balance_forward), MOE_ENTRY(balance_backward), MOE_ENTRY(fp8_quantize),
                          MOE_ENTRY(fp8_quantize_weights), MOE_ENTRY(fp8_matmul), MOE_ENTRY(fp8_wgrad), MOE_ENTRY(route_forward), MOE_ENTRY(route_backward),
                          MOE_ENTRY(norm_forward), MOE_ENTRY(norm_backward), MOE_ENTRY(combine_forward), MOE_ENTRY(combine_backward),
                          MOE_ENTRY(grad_norm), MOE_ENTRY(grad_clip),
                          {"set_error", set_error, METH_O, nullptr}, {nullptr, nullptr, 0, nullptr}};
PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "_moe_torch", nullptr, -1, kMethods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

extern "C" __attribute__((visibility("default"))) PyObject *PyInit__moe_torch() { return PyModule_Create(&kModule); }
