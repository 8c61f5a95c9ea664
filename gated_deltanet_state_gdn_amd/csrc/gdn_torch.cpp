// Native half of the Python binding of the suffix and decode operators: argument checks, output
// allocation and the call, for torch tensors.  A single-token call lasts a few microseconds on the
// GPU, and the same checks in Python cost more than that.  No computation happens here: every
// function ends in one call of the C ABI (include/gdn.h), whose address the Python side hands over.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <ATen/ops/zeros.h>
#include <c10/core/DeviceGuard.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <initializer_list>
#include <string>

#include "../../include/gdn.h"

namespace {

// A refusal: becomes GdnError(code, what).
struct Refused {
    int code;
    std::string what;
};

PyObject *g_error = nullptr, *g_raw_stream = nullptr;

typedef decltype(&gdn_conv) conv_fn;
typedef decltype(&gdn_conv_step) conv_step_fn;
typedef decltype(&gdn_ssm_scan) scan_fn;
typedef decltype(&gdn_ssm_step) ssm_step_fn;
typedef decltype(&gdn_step) step_fn;
typedef decltype(&gdn_qk_norm_rope) rope_fn;
typedef decltype(&gdn_paged_attn) attn_fn;
typedef decltype(&gdn_ssm_workspace_bytes) scan_ws_fn;
typedef decltype(&gdn_paged_workspace_bytes) attn_ws_fn;
typedef decltype(&gdn_cache_extend) extend_fn;
typedef decltype(&gdn_shared_attn) shared_fn;
typedef decltype(&gdn_sample) sample_fn;
typedef decltype(&gdn_extend_workspace_bytes) extend_ws_fn;
typedef decltype(&gdn_shared_workspace_bytes) shared_ws_fn;
typedef decltype(&gdn_sample_workspace_bytes) sample_ws_fn;
conv_fn f_conv;
conv_step_fn f_conv_step;
scan_fn f_scan;
ssm_step_fn f_ssm_step;
step_fn f_step;
rope_fn f_rope;
attn_fn f_attn;
scan_ws_fn f_scan_ws;
attn_ws_fn f_attn_ws;
extend_fn f_extend;
shared_fn f_shared;
sample_fn f_sample;
extend_ws_fn f_extend_ws;
shared_ws_fn f_shared_ws;
sample_ws_fn f_sample_ws;

const at::Tensor none;
constexpr auto F32 = at::kFloat;
constexpr auto I32 = at::kInt;
constexpr auto I64 = at::kLong;
constexpr int kFunctions = 15;   // of the C library

// The call's name and what its tensors have in common.
struct Call {
    const char *name;
    at::Device device = at::Device(at::kCPU);
    bool first = true, mixed = false;

    [[noreturn]] void refuse(int code, const char *arg, const std::string &why) const {
        throw Refused{code, std::string(name) + ": " + arg + (*arg ? " " : "") + why};
    }
    void need(bool ok, const char *why) const {
        if (!ok) refuse(GDN_ERR_SHAPE, "", why);
    }
    // A tensor argument; None is an undefined tensor.
    const at::Tensor &tensor(PyObject *o, const char *arg, bool optional = false) {
        if (o == Py_None) {
            if (!optional) refuse(GDN_ERR_NULL, arg, "is missing");
            return none;
        }
        if (!THPVariable_Check(o)) refuse(GDN_ERR_SHAPE, arg, "is not a tensor");
        const at::Tensor &t = THPVariable_Unpack(o);
        seen(t);
        return t;
    }
    void seen(const at::Tensor &t) {
        if (first) device = t.device();
        else mixed |= t.device() != device;
        first = false;
    }
    void shape(const at::Tensor &t, std::initializer_list<int64_t> want, at::ScalarType dtype, const char *arg) const {
        if (t.scalar_type() != dtype) refuse(GDN_ERR_DTYPE, arg, "has another dtype than it must have");
        if (t.sizes() != at::IntArrayRef(want)) {
            std::string s = "has another shape than (";
            for (int64_t v : want) s += std::to_string(v) + ", ";
            refuse(GDN_ERR_SHAPE, arg, s + ")");
        }
    }
    // contiguous
    void whole(const at::Tensor &t, std::initializer_list<int64_t> want, at::ScalarType dtype, const char *arg) const {
        if (!t.defined()) return;
        shape(t, want, dtype, arg);
        if (!t.is_contiguous()) refuse(GDN_ERR_ALIGN, arg, "must be contiguous");
    }
    // rows contiguous in themselves: the elements from one to the next
    int64_t rows(const at::Tensor &t, std::initializer_list<int64_t> want, at::ScalarType dtype, const char *arg) const {
        shape(t, want, dtype, arg);
        int64_t inner = 1;
        for (int64_t k = t.dim() - 1; k > 0; --k) {
            if (t.size(k) != 1 && t.stride(k) != inner) refuse(GDN_ERR_ALIGN, arg, "must have contiguous rows");
            inner *= t.size(k);
        }
        return t.size(0) > 1 ? t.stride(0) : inner;
    }
    int32_t code(const at::Tensor &t) const {
        if (t.scalar_type() == F32) return GDN_F32;
        if (t.scalar_type() == at::kBFloat16) return GDN_BF16;
        refuse(GDN_ERR_DTYPE, "", "float32 or bfloat16 wanted");
    }
    // A size as the C ABI takes it; what does not fit is refused there as a bad size.
    int32_t size32(int64_t v) const {
        if (v > 0x7fffffffLL) refuse(GDN_ERR_SHAPE, "", "a size does not fit 32 bits");
        return (int32_t)v;
    }
    // After every check of shapes: an output to allocate may be on this device only.
    void on_gpu() const {
        if (!device.is_cuda()) refuse(GDN_ERR_SHAPE, "", "tensors must be on a GPU");
        if (mixed) refuse(GDN_ERR_SHAPE, "", "tensors on different devices");
    }
    at::Tensor make(at::IntArrayRef shape, at::ScalarType dtype) const {
        return at::empty(shape, at::TensorOptions().dtype(dtype).device(device));
    }
    // Outputs in one allocation, each of which costs 1.4 us of a call of 8.
    struct Piece {
        at::Tensor &out;
        bool wanted;
        int64_t n;
        at::ScalarType dtype;
    };
    void make_pieces(std::initializer_list<Piece> pieces) const {
        int64_t bytes = 0;
        for (const Piece &p : pieces)
            if (p.wanted) bytes += (p.n * (int64_t)c10::elementSize(p.dtype) + 15) / 16 * 16;
        const at::Tensor all = make({bytes}, at::kByte);
        int64_t at_byte = 0;
        for (const Piece &p : pieces) {
            if (!p.wanted) continue;
            const int64_t size = (int64_t)c10::elementSize(p.dtype);
            p.out = at::detail::make_tensor<c10::TensorImpl>(c10::Storage(all.storage()), all.key_set(), c10::scalarTypeToTypeMeta(p.dtype));
            p.out.unsafeGetTensorImpl()->set_storage_offset(at_byte / size);
            p.out.unsafeGetTensorImpl()->set_sizes_contiguous({p.n});
            at_byte += (p.n * size + 15) / 16 * 16;
        }
    }
    at::Tensor workspace(PyObject *o, size_t bytes) const {
        if (o == Py_None) return at::zeros({(int64_t)(bytes > 256 ? bytes : 256)}, at::TensorOptions().dtype(at::kByte).device(device));
        if (!THPVariable_Check(o)) refuse(GDN_ERR_SHAPE, "ws", "is not a tensor");
        const at::Tensor &t = THPVariable_Unpack(o);
        if (t.scalar_type() != at::kByte || !t.is_contiguous() || t.device() != device)
            refuse(GDN_ERR_SHAPE, "ws", "must be a contiguous uint8 tensor on the same device");
        return t;
    }
    void *stream() const {
        PyObject *i = PyLong_FromLong(device.index());
        if (!i) throw python_error();
        PyObject *s = PyObject_CallOneArg(g_raw_stream, i);
        Py_DECREF(i);
        if (!s) throw python_error();
        void *p = PyLong_AsVoidPtr(s);
        Py_DECREF(s);
        if (!p && PyErr_Occurred()) throw python_error();
        return p;
    }
    void check(int32_t status) const {
        if (status != GDN_OK) throw Refused{status, name};
    }
};

template <class T = void>
T *ptr(const at::Tensor &t) {
    return t.defined() ? static_cast<T *>(t.data_ptr()) : nullptr;
}
bool truth(PyObject *o) {
    const int v = PyObject_IsTrue(o);
    if (v < 0) throw python_error();
    return v != 0;
}
double number(PyObject *o) {
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred()) throw python_error();
    return v;
}
int64_t integer(PyObject *o) {
    const int64_t v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred()) throw python_error();
    return v;
}
// An output argument: a tensor, True (allocate), or None / False (none).
enum class Out { given, make, none };
Out out_kind(PyObject *o) {
    return o == Py_True ? Out::make : o == Py_None || o == Py_False ? Out::none : Out::given;
}
PyObject *wrap(const at::Tensor &t) {
    if (!t.defined()) Py_RETURN_NONE;
    return THPVariable_Wrap(t);
}
// A tuple of results (takes the references).
PyObject *pack(std::initializer_list<PyObject *> items) {
    PyObject *t = PyTuple_New((Py_ssize_t)items.size());
    Py_ssize_t i = 0;
    bool ok = t != nullptr;
    for (PyObject *o : items) {
        ok = ok && o;
        if (t && o) PyTuple_SET_ITEM(t, i++, o);
        else Py_XDECREF(o);
    }
    if (!ok) {
        Py_XDECREF(t);
        throw python_error();
    }
    return t;
}

// Runs a function of (PyObject *const *args) and turns its exceptions into Python's.
template <class F>
PyObject *guarded(Py_ssize_t got, Py_ssize_t want, F f) {
    HANDLE_TH_ERRORS
    if (got != want) {
        PyErr_SetString(PyExc_TypeError, "wrong number of arguments");
        return nullptr;
    }
    try {
        return f();
    } catch (const Refused &r) {
        PyObject *e = PyObject_CallFunction(g_error, "is", r.code, r.what.c_str());
        if (e) {
            PyErr_SetObject(g_error, e);
            Py_DECREF(e);
        }
        return nullptr;
    }
    END_HANDLE_TH_ERRORS
}

// x, weight, cu, bias, state0, state_out, silu, y, ws
PyObject *conv(PyObject *, PyObject *const *v, Py_ssize_t nargs) {
    return guarded(nargs, 9, [&] {
        Call c{"gdn_conv"};
        const at::Tensor &x = c.tensor(v[0], "x"), &w = c.tensor(v[1], "weight"), &cu = c.tensor(v[2], "cu_seqlens");
        const at::Tensor &bias = c.tensor(v[3], "bias", true), &s0 = c.tensor(v[4], "state0", true);
        const int32_t dt = c.code(x);
        c.need(x.dim() == 2 && w.dim() == 2 && cu.dim() == 1 && cu.numel() > 0, "x [T, channels], weight [channels, width], cu_seqlens [n_seqs + 1]");
        const int64_t T = x.size(0), ch = x.size(1), k = w.size(1), n = cu.numel() - 1;
        const auto e = x.scalar_type();
        gdn_conv_desc d = {c.size32(n), 0, c.size32(ch), c.size32(k), dt, truth(v[6]), T, c.rows(x, {T, ch}, e, "x"), ch};
        c.whole(w, {ch, k}, F32, "weight");
        c.whole(bias, {ch}, F32, "bias");
        c.whole(cu, {n + 1}, I32, "cu_seqlens");
        c.whole(s0, {n, k - 1, ch}, e, "state0");
        at::Tensor so, y;
        const Out kind = k > 1 ? out_kind(v[5]) : Out::none;
        if (kind == Out::given) c.whole(so = c.tensor(v[5], "state_out"), {n, k - 1, ch}, e, "state_out");
        if (v[7] != Py_None) d.y_stride = c.rows(y = c.tensor(v[7], "y"), {T, ch}, e, "y");
        c.on_gpu();
        c10::DeviceGuard guard(c.device);
        if (kind == Out::make) so = c.make({n, k - 1, ch}, e);
        if (!y.defined()) y = c.make({T, ch}, e);
        const at::Tensor ws = c.workspace(v[8], 256);
        c.check(f_conv(&d, ptr(x), ptr<float>(w), ptr<float>(bias), ptr<int32_t>(cu), ptr(s0), ptr(so), ptr(y), ptr(ws),
                       ws.numel(), c.stream()));
        return pack({wrap(y), wrap(so)});
    });
}

// x, weight, state, slots, bias, silu, y, ws
PyObject *conv_step(PyObject *, PyObject *const *v, Py_ssize_t nargs) {
    return guarded(nargs, 8, [&] {
        Call c{"gdn_conv_step"};
        const at::Tensor &x = c.tensor(v[0], "x"), &w = c.tensor(v[1], "weight"), &s = c.tensor(v[2], "state");
        const at::Tensor &slots = c.tensor(v[3], "slots", true), &bias = c.tensor(v[4], "bias", true);
        const int32_t dt = c.code(x);
        c.need(x.dim() == 2 && w.dim() == 2 && s.dim() == 3, "x [rows, channels], weight [channels, width], state [n_slots, width - 1, channels]");
        const int64_t n = x.size(0), ch = x.size(1), k = w.size(1), pool = s.size(0);
        const auto e = x.scalar_type();
        gdn_conv_desc d = {c.size32(n), c.size32(pool), c.size32(ch), c.size32(k), dt, truth(v[5]), n, c.rows(x, {n, ch}, e, "x"), ch};
        c.whole(w, {ch, k}, F32, "weight");
        c.whole(bias, {ch}, F32, "bias");
        c.whole(s, {pool, k - 1, ch}, e, "state");
        c.whole(slots, {n}, I32, "slots");
        at::Tensor y;
        if (v[6] != Py_None) d.y_stride = c.rows(y = c.tensor(v[6], "y"), {n, ch}, e, "y");
        c.on_gpu();
        c10::DeviceGuard guard(c.device);
        if (!y.defined()) y = c.make({n, ch}, e);
        const at::Tensor ws = c.workspace(v[7], 256);
        c.check(f_conv_step(&d, ptr(x), ptr<float>(w), ptr<float>(bias), ptr(s), ptr<int32_t>(slots), ptr(y), ptr(ws),
                            ws.numel(), c.stream()));
        return wrap(y);
    });
}

// The tensors that both state space calls take: x, B, C, dt, A in v[0..4], D, dt_bias.
struct Ssm {
    const at::Tensor &x, &B, &C, &dt, &A, &D, &dt_bias;
    gdn_ssm_desc d = {};
    Ssm(Call &c, PyObject *const *v, PyObject *D_, PyObject *bias_)
        : x(c.tensor(v[0], "x")), B(c.tensor(v[1], "B")), C(c.tensor(v[2], "C")), dt(c.tensor(v[3], "dt")),
          A(c.tensor(v[4], "A")), D(c.tensor(D_, "D", true)), dt_bias(c.tensor(bias_, "dt_bias", true)) {
        c.need(x.dim() == 3 && B.dim() == 3, "x [T, h_v, d_v], B [T, h_qk, d_k]");
        const int64_t T = x.size(0), h = x.size(1), p = x.size(2), g = B.size(1), k = B.size(2);
        const auto e = x.scalar_type();
        d.dtype = c.code(x);
        d.h_qk = c.size32(g); d.h_v = c.size32(h); d.d_k = c.size32(k); d.d_v = c.size32(p);
        d.total_tokens = T;
        d.x_stride = c.rows(x, {T, h, p}, e, "x");
        d.b_stride = c.rows(B, {T, g, k}, e, "B");
        d.c_stride = c.rows(C, {T, g, k}, e, "C");
        d.dt_stride = c.rows(dt, {T, h}, e, "dt");
        d.y_stride = h * p;
        c.whole(A, {h}, F32, "A");
        c.whole(D, {h}, F32, "D");
        c.whole(dt_bias, {h}, F32, "dt_bias");
    }
};

// x, B, C, dt, A, cu, D, dt_bias, softplus, r, total_out_tokens, S0, S_out, y_out, cu_out, ws
PyObject *scan(PyObject *, PyObject *const *v, Py_ssize_t nargs) {
    return guarded(nargs, 16, [&] {
        Call c{"gdn_ssm_scan"};
        Ssm s(c, v, v[6], v[7]);
        gdn_ssm_desc &d = s.d;
        const at::Tensor &cu = c.tensor(v[5], "cu_seqlens"), &r = c.tensor(v[9], "r", true), &S0 = c.tensor(v[11], "S0", true);
        const at::Tensor &cu_out = c.tensor(v[14], "cu_out", true);
        c.need(cu.dim() == 1 && cu.numel() > 0, "cu_seqlens [n_seqs + 1]");
        c.need(!r.defined() || v[10] != Py_None, "r needs total_out_tokens");
        const int64_t n = cu.numel() - 1, h = d.h_v, k = d.d_k, p = d.d_v;
        const auto e = s.x.scalar_type();
        d.n_seqs = c.size32(n);
        d.softplus = truth(v[8]);
        d.total_out_tokens = v[10] == Py_None ? d.total_tokens : integer(v[10]);
        c.need(d.total_out_tokens >= 0, "total_out_tokens is negative");
        c.whole(cu, {n + 1}, I32, "cu_seqlens");
        c.whole(r, {n}, I32, "r");
        c.whole(cu_out, {n + 1}, I32, "cu_out");
        c.whole(S0, {n, h, k, p}, F32, "S0");
        at::Tensor S, y;
        if (v[12] != Py_None) c.whole(S = c.tensor(v[12], "S_out"), {n, h, k, p}, F32, "S_out");
        const Out kind = out_kind(v[13]);
        if (kind == Out::given) d.y_stride = c.rows(y = c.tensor(v[13], "y_out"), {d.total_out_tokens, h, p}, e, "y_out");
        c.on_gpu();
        c10::DeviceGuard guard(c.device);
        if (!S.defined()) S = c.make({n, h, k, p}, F32);
        if (kind == Out::make) y = c.make({d.total_out_tokens, h, p}, e);
        const at::Tensor ws = c.workspace(v[15], v[15] == Py_None ? f_scan_ws(&d) : 0);
        c.check(f_scan(&d, ptr(s.x), ptr(s.B), ptr(s.C), ptr(s.dt), ptr<float>(s.A), ptr<float>(s.dt_bias), ptr<float>(s.D),
                       ptr<int32_t>(cu), ptr<int32_t>(r), ptr<float>(S0), ptr<float>(S), ptr(y), ptr<int32_t>(cu_out),
                       ptr(ws), ws.numel(), c.stream()));
        return pack({wrap(S), wrap(y), wrap(cu_out)});
    });
}

// x, B, C, dt, A, S, slots, D, dt_bias, softplus, y, ws
PyObject *ssm_step(PyObject *, PyObject *const *v, Py_ssize_t nargs) {
    return guarded(nargs, 12, [&] {
        Call c{"gdn_ssm_step"};
        Ssm s(c, v, v[7], v[8]);
        gdn_ssm_desc &d = s.d;
        const at::Tensor &S = c.tensor(v[5], "S"), &slots = c.tensor(v[6], "slots", true);
        c.need(S.dim() == 4, "S [n_slots, h_v, d_k, d_v]");
        const int64_t n = d.total_tokens;
        const auto e = s.x.scalar_type();
        d.n_seqs = c.size32(n);
        d.n_slots = c.size32(S.size(0));
        d.softplus = truth(v[9]);
        d.total_out_tokens = n;
        c.whole(S, {S.size(0), d.h_v, d.d_k, d.d_v}, F32, "S");
        c.whole(slots, {n}, I32, "slots");
        at::Tensor y;
        if (v[10] != Py_None) d.y_stride = c.rows(y = c.tensor(v[10], "y"), {n, d.h_v, d.d_v}, e, "y");
        c.on_gpu();
        c10::DeviceGuard guard(c.device);
        if (!y.defined()) y = c.make({n, d.h_v, d.d_v}, e);
        const at::Tensor ws = c.workspace(v[11], 256);
        c.check(f_ssm_step(&d, ptr(s.x), ptr(s.B), ptr(s.C), ptr(s.dt), ptr<float>(s.A), ptr<float>(s.dt_bias), ptr<float>(s.D),
                           ptr<float>(S), ptr<int32_t>(slots), ptr(y), ptr(ws), ws.numel(), c.stream()));
        return wrap(y);
    });
}

// q, k, v, g, beta, S, slots, o, scale, f32 output, ws
PyObject *step(PyObject *, PyObject *const *v, Py_ssize_t nargs) {
    return guarded(nargs, 11, [&] {
        Call c{"gdn_step"};
        const at::Tensor &q = c.tensor(v[0], "q"), &k = c.tensor(v[1], "k"), &x = c.tensor(v[2], "v"), &g = c.tensor(v[3], "g");
        const at::Tensor &beta = c.tensor(v[4], "beta"), &S = c.tensor(v[5], "S"), &slots = c.tensor(v[6], "slots", true);
        const int32_t dt = c.code(q);
        c.need(q.dim() == 3 && x.dim() == 3 && S.dim() == 4, "q, k [rows, h_qk, d_k], v [rows, h_v, d_v], S [n_slots, h_v, d_k, d_v]");
        const int64_t n = q.size(0), hq = q.size(1), dk = q.size(2), h = x.size(1), dv = x.size(2), pool = S.size(0);
        const auto e = q.scalar_type();
        c.whole(q, {n, hq, dk}, e, "q");
        c.whole(k, {n, hq, dk}, e, "k");
        c.whole(x, {n, h, dv}, e, "v");
        c.whole(g, {n, h}, F32, "g");
        c.whole(beta, {n, h}, F32, "beta");
        c.whole(S, {pool, h, dk, dv}, F32, "S");
        c.whole(slots, {n}, I32, "slots");
        at::Tensor o;
        if (v[7] != Py_None) {
            o = c.tensor(v[7], "o");
            c.whole(o, {n, h, dv}, o.scalar_type(), "o");
        }
        const auto oe = o.defined() ? o.scalar_type() : truth(v[9]) ? F32 : e;
        gdn_desc d = {c.size32(n), c.size32(hq), c.size32(h), c.size32(dk), c.size32(dv), dt,
                      oe == F32 ? GDN_F32 : oe == at::kBFloat16 ? GDN_BF16 : -1, (float)number(v[8]), n, n};
        c.on_gpu();
        c10::DeviceGuard guard(c.device);
        if (!o.defined()) o = c.make({n, h, dv}, oe);
        const at::Tensor ws = c.workspace(v[10], 256);
        c.check(f_step(&d, ptr(q), ptr(k), ptr(x), ptr<float>(g), ptr<float>(beta), ptr<float>(S), c.size32(pool),
                       ptr<int32_t>(slots), ptr(o), ptr(ws), ws.numel(), c.stream()));
        return wrap(o);
    });
}

// What the two calls on a paged cache share.
struct Paged {
    const at::Tensor &q, &kc, &vc, &table, &cu, &kv;
    gdn_paged_desc d = {};
    int32_t holds;              // cached tokens of a row of the block table, at most 2^30
    Paged(Call &c, PyObject *q_, PyObject *kc_, PyObject *vc_, PyObject *table_, PyObject *cu_, PyObject *kv_, PyObject *max_kv)
        : q(c.tensor(q_, "q")), kc(c.tensor(kc_, "k_cache")), vc(c.tensor(vc_, "v_cache")), table(c.tensor(table_, "block_table")),
          cu(c.tensor(cu_, "cu_seqlens")), kv(c.tensor(kv_, "kv_len")) {
        c.need(q.dim() == 3 && kc.dim() == 4 && table.dim() == 2 && cu.dim() == 1 && cu.numel() > 0,
               "q [T, h_q, d], caches [n_pages, page_size, h_kv, d], block_table [n_seqs, max_pages], cu_seqlens [n_seqs + 1]");
        const int64_t n = cu.numel() - 1, dim = q.size(2), most = table.size(1);
        c.whole(cu, {n + 1}, I32, "cu_seqlens");
        c.whole(kv, {n}, I32, "kv_len");
        c.whole(table, {n, most}, I32, "block_table");
        c.need(kc.size(3) == dim, "the caches' head dim is not q's");
        c.need(kc.sizes() == vc.sizes() && kc.strides() == vc.strides(), "k_cache and v_cache differ in shape or strides");
        d.dtype = c.code(q);
        if (kc.scalar_type() != q.scalar_type() || vc.scalar_type() != q.scalar_type()) c.refuse(GDN_ERR_DTYPE, "", "the caches have q's dtype");
        if (kc.stride(3) != 1) c.refuse(GDN_ERR_ALIGN, "", "a head's cache entries must be contiguous");
        d.n_seqs = c.size32(n);
        d.h_q = c.size32(q.size(1)); d.h_kv = c.size32(kc.size(2)); d.d = c.size32(dim);
        d.page_size = c.size32(kc.size(1)); d.n_pages = c.size32(kc.size(0)); d.max_pages = c.size32(most);
        const int64_t hold = most * kc.size(1);
        int64_t bound = hold < (1 << 30) ? hold : 1 << 30;
        holds = (int32_t)bound;
        if (max_kv != Py_None) {
            const int64_t m = integer(max_kv);
            c.need(m >= 0 && m <= (1 << 30), "max_kv_len out of range");
            bound = m < hold ? m : hold;
        }
        d.max_kv_len = (int32_t)bound;
        d.total_tokens = q.size(0);
        d.scale = 1.0f / sqrtf((float)dim);
        // strides of dimensions of one element say nothing
        d.page_stride = kc.stride(0);
        d.token_stride = kc.size(1) > 1 ? kc.stride(1) : std::max(kc.stride(1), dim);
        d.head_stride = kc.size(2) > 1 ? kc.stride(2) : std::max(kc.stride(2), dim);
        d.k_stride = d.v_stride = kc.size(2) * dim;
        d.q_stride = c.rows(q, {q.size(0), q.size(1), dim}, q.scalar_type(), "q");
        d.o_stride = q.size(1) * dim;
    }
};

// q, k, v, cos_sin, k_cache, v_cache, table, cu, kv_len, q_weight, k_weight, eps, norm, interleaved, positions, q_out, max_kv, ws
PyObject *rope(PyObject *, PyObject *const *v, Py_ssize_t nargs) {
    return guarded(nargs, 18, [&] {
        Call c{"gdn_qk_norm_rope"};
        Paged p(c, v[0], v[4], v[5], v[6], v[7], v[8], v[16]);
        gdn_paged_desc &d = p.d;
        const at::Tensor &k = c.tensor(v[1], "k"), &x = c.tensor(v[2], "v"), &cs = c.tensor(v[3], "cos_sin", true);
        const at::Tensor &wq = c.tensor(v[9], "q_weight", true), &wk = c.tensor(v[10], "k_weight", true), &pos = c.tensor(v[14], "positions", true);
        const int64_t T = d.total_tokens, dim = d.d;
        const auto e = p.q.scalar_type();
        d.k_stride = c.rows(k, {T, d.h_kv, dim}, e, "k");
        d.v_stride = c.rows(x, {T, d.h_kv, dim}, e, "v");
        c.whole(wq, {dim}, F32, "q_weight");
        c.whole(wk, {dim}, F32, "k_weight");
        if (cs.defined()) {
            c.need(cs.dim() == 2, "cos_sin [positions, rot_dim]");
            d.max_pos = c.size32(cs.size(0));
            d.rot_dim = c.size32(cs.size(1));
            c.whole(cs, {cs.size(0), cs.size(1)}, F32, "cos_sin");
        }
        c.whole(pos, {T}, I32, "positions");
        d.eps = (float)number(v[11]);
        d.norm = truth(v[12]);
        d.interleaved = truth(v[13]);
        at::Tensor o;
        if (v[15] != Py_None) d.o_stride = c.rows(o = c.tensor(v[15], "q_out"), {T, d.h_q, dim}, e, "q_out");
        c.on_gpu();
        c10::DeviceGuard guard(c.device);
        if (!o.defined()) o = c.make({T, d.h_q, dim}, e);
        const at::Tensor ws = c.workspace(v[17], 256);
        c.check(f_rope(&d, ptr(p.q), ptr(k), ptr(x), ptr<float>(wq), ptr<float>(wk), ptr<float>(cs), ptr<int32_t>(p.table),
                       ptr<int32_t>(p.cu), ptr<int32_t>(p.kv), ptr<int32_t>(pos), ptr(p.kc), ptr(p.vc), ptr(o), ptr(ws),
                       ws.numel(), c.stream()));
        return wrap(o);
    });
}

// q, k_cache, v_cache, table, cu, kv_len, max_kv, scale, o, lse, ws
PyObject *attn(PyObject *, PyObject *const *v, Py_ssize_t nargs) {
    return guarded(nargs, 11, [&] {
        Call c{"gdn_paged_attn"};
        Paged p(c, v[0], v[1], v[2], v[3], v[4], v[5], v[6]);
        gdn_paged_desc &d = p.d;
        const int64_t T = d.total_tokens;
        const auto e = p.q.scalar_type();
        if (v[7] != Py_None) d.scale = (float)number(v[7]);
        at::Tensor o, lse;
        if (v[8] != Py_None) d.o_stride = c.rows(o = c.tensor(v[8], "o"), {T, d.h_q, d.d}, e, "o");
        const Out kind = out_kind(v[9]);
        if (kind == Out::given) c.whole(lse = c.tensor(v[9], "lse"), {T, d.h_q}, F32, "lse");
        c.on_gpu();
        c10::DeviceGuard guard(c.device);
        if (!o.defined()) o = c.make({T, d.h_q, d.d}, e);
        if (kind == Out::make) lse = c.make({T, d.h_q}, F32);
        const at::Tensor ws = c.workspace(v[10], v[10] == Py_None ? f_attn_ws(&d) : 0);
        c.check(f_attn(&d, ptr(p.q), ptr(p.kc), ptr(p.vc), ptr<int32_t>(p.table), ptr<int32_t>(p.cu), ptr<int32_t>(p.kv), ptr(o),
                       ptr<float>(lse), ptr(ws), ws.numel(), c.stream()));
        return lse.defined() ? pack({wrap(o), wrap(lse)}) : wrap(o);
    });
}

// A bound on a device array's values, `most` if none is given; more than the block table `holds` is as good as that.
int32_t bound(const Call &c, PyObject *o, int32_t most, int32_t holds, const char *arg) {
    if (o == Py_None) return most;
    const int64_t v = integer(o);
    if (v < 0 || v > (1 << 30)) c.refuse(GDN_ERR_SHAPE, arg, "out of range");
    return v < holds ? (int32_t)v : holds;
}

// q, k_cache, v_cache, table, cu, kv_len, cu_groups, prefix_len, max_kv, max_prefix, max_own, scale, o, lse, ws
PyObject *shared(PyObject *, PyObject *const *v, Py_ssize_t nargs) {
    return guarded(nargs, 15, [&] {
        Call c{"gdn_shared_attn"};
        Paged p(c, v[0], v[1], v[2], v[3], v[4], v[5], v[8]);
        const at::Tensor &groups = c.tensor(v[6], "cu_groups"), &prefix = c.tensor(v[7], "prefix_len");
        c.need(groups.dim() == 1 && groups.numel() > 0, "cu_groups [n_groups + 1]");
        const int64_t n = groups.numel() - 1, T = p.d.total_tokens;
        c.whole(groups, {n + 1}, I32, "cu_groups");
        c.whole(prefix, {n}, I32, "prefix_len");
        const auto e = p.q.scalar_type();
        if (v[11] != Py_None) p.d.scale = (float)number(v[11]);
        at::Tensor o, lse;
        if (v[12] != Py_None) p.d.o_stride = c.rows(o = c.tensor(v[12], "o"), {T, p.d.h_q, p.d.d}, e, "o");
        const Out kind = out_kind(v[13]);
        if (kind == Out::given) c.whole(lse = c.tensor(v[13], "lse"), {T, p.d.h_q}, F32, "lse");
        // a prefix may be longer than any kv_len, own keys may not
        const int32_t most = p.d.max_kv_len;
        gdn_shared_desc d = {p.d, c.size32(n), bound(c, v[9], most, p.holds, "max_prefix_len"), bound(c, v[10], most, most, "max_own_len")};
        c.on_gpu();
        c10::DeviceGuard guard(c.device);
        if (!o.defined()) o = c.make({T, p.d.h_q, p.d.d}, e);
        if (kind == Out::make) lse = c.make({T, p.d.h_q}, F32);
        const at::Tensor ws = c.workspace(v[14], v[14] == Py_None ? f_shared_ws(&d) : 0);
        c.check(f_shared(&d, ptr(p.q), ptr(p.kc), ptr(p.vc), ptr<int32_t>(p.table), ptr<int32_t>(p.cu), ptr<int32_t>(p.kv),
                         ptr<int32_t>(groups), ptr<int32_t>(prefix), ptr(o), ptr<float>(lse), ptr(ws), ws.numel(), c.stream()));
        return lse.defined() ? pack({wrap(o), wrap(lse)}) : wrap(o);
    });
}

// new_len, kv_len, table, free_pages, free_at, page_size, total_tokens, prefix_of, prefix_table, prefix_len, kv_out, free_out, cu, slots,
// positions, ws
PyObject *extend(PyObject *, PyObject *const *v, Py_ssize_t nargs) {
    return guarded(nargs, 16, [&] {
        Call c{"gdn_cache_extend"};
        const at::Tensor &add = c.tensor(v[0], "new_len"), &kv = c.tensor(v[1], "kv_len"), &table = c.tensor(v[2], "block_table");
        const at::Tensor &pages = c.tensor(v[3], "free_pages"), &taken = c.tensor(v[4], "free_at");
        const at::Tensor &of = c.tensor(v[7], "prefix_of", true), &pt = c.tensor(v[8], "prefix_table", true), &pl = c.tensor(v[9], "prefix_len", true);
        c.need(add.dim() == 1 && table.dim() == 2 && pages.dim() == 1, "new_len [n_seqs], block_table [n_seqs, max_pages], free_pages [n]");
        const int64_t n = add.size(0), most = table.size(1), ps = integer(v[5]), T = integer(v[6]);
        c.need(ps > 0 && T >= 0, "page_size is positive, total_tokens not negative");
        c.whole(add, {n}, I32, "new_len");
        c.whole(kv, {n}, I32, "kv_len");
        c.whole(table, {n, most}, I32, "block_table");
        c.whole(pages, {pages.size(0)}, I32, "free_pages");
        c.whole(taken, {1}, I32, "free_at");
        gdn_extend_desc d = {c.size32(n), c.size32(ps), c.size32(most), c.size32(pages.size(0)), 0, 0, T};
        if (of.defined() || pt.defined() || pl.defined()) {
            c.need(of.defined() && pt.defined() && pl.defined() && pt.dim() == 2, "prefix_of, prefix_table [n_prefixes, max_prefix_pages], prefix_len: all or none");
            d.n_prefixes = c.size32(pt.size(0));
            d.max_prefix_pages = c.size32(pt.size(1));
            c.whole(of, {n}, I32, "prefix_of");
            c.whole(pt, {pt.size(0), pt.size(1)}, I32, "prefix_table");
            c.whole(pl, {pt.size(0)}, I32, "prefix_len");
        }
        at::Tensor kvo, fo, cu, slots, pos;
        if (v[10] != Py_None) c.whole(kvo = c.tensor(v[10], "kv_out"), {n}, I32, "kv_out");
        if (v[11] != Py_None) c.whole(fo = c.tensor(v[11], "free_out"), {1}, I32, "free_out");
        if (v[12] != Py_None) c.whole(cu = c.tensor(v[12], "cu_seqlens"), {n + 1}, I32, "cu_seqlens");
        const Out sk = out_kind(v[13]), pk = out_kind(v[14]);
        if (sk == Out::given) c.whole(slots = c.tensor(v[13], "slots"), {T}, I64, "slots");
        if (pk == Out::given) c.whole(pos = c.tensor(v[14], "positions"), {T}, I32, "positions");
        c.on_gpu();
        c10::DeviceGuard guard(c.device);
        c.make_pieces({{slots, sk == Out::make, T, I64}, {pos, pk == Out::make, T, I32}, {cu, !cu.defined(), n + 1, I32},
                       {kvo, !kvo.defined(), n, I32}, {fo, !fo.defined(), 1, I32}});
        const at::Tensor ws = c.workspace(v[15], v[15] == Py_None ? f_extend_ws(d.n_seqs) : 0);
        c.check(f_extend(&d, ptr<int32_t>(add), ptr<int32_t>(kv), ptr<int32_t>(table), ptr<int32_t>(pages), ptr<int32_t>(taken),
                         ptr<int32_t>(of), ptr<int32_t>(pt), ptr<int32_t>(pl), ptr<int32_t>(kvo), ptr<int32_t>(fo), ptr<int32_t>(cu),
                         ptr<int64_t>(slots), ptr<int32_t>(pos), ptr(ws), ws.numel(), c.stream()));
        return pack({wrap(cu), wrap(kvo), wrap(fo), wrap(slots), wrap(pos)});
    });
}

// logits, u, temperature, top_k, top_p, min_p, token, logprob, ws
PyObject *sample(PyObject *, PyObject *const *v, Py_ssize_t nargs) {
    return guarded(nargs, 9, [&] {
        Call c{"gdn_sample"};
        const at::Tensor &x = c.tensor(v[0], "logits"), &u = c.tensor(v[1], "u"), &t = c.tensor(v[2], "temperature", true);
        const at::Tensor &k = c.tensor(v[3], "top_k", true), &p = c.tensor(v[4], "top_p", true), &m = c.tensor(v[5], "min_p", true);
        const int32_t dt = c.code(x);
        c.need(x.dim() == 2, "logits [rows, vocab]");
        const int64_t n = x.size(0), vocab = x.size(1);
        gdn_sample_desc d = {c.size32(n), c.size32(vocab), dt, c.rows(x, {n, vocab}, x.scalar_type(), "logits")};
        c.whole(u, {n}, F32, "u");
        c.whole(t, {n}, F32, "temperature");
        c.whole(k, {n}, I32, "top_k");
        c.whole(p, {n}, F32, "top_p");
        c.whole(m, {n}, F32, "min_p");
        at::Tensor token, lp;
        if (v[6] != Py_None) c.whole(token = c.tensor(v[6], "token"), {n}, I32, "token");
        const Out kind = out_kind(v[7]);
        if (kind == Out::given) c.whole(lp = c.tensor(v[7], "logprob"), {n}, F32, "logprob");
        c.on_gpu();
        c10::DeviceGuard guard(c.device);
        if (!token.defined()) token = c.make({n}, I32);
        if (kind == Out::make) lp = c.make({n}, F32);
        const at::Tensor ws = c.workspace(v[8], v[8] == Py_None ? f_sample_ws(&d) : 0);
        c.check(f_sample(&d, ptr(x), ptr<float>(u), ptr<float>(t), ptr<int32_t>(k), ptr<float>(p), ptr<float>(m), ptr<int32_t>(token),
                         ptr<float>(lp), ptr(ws), ws.numel(), c.stream()));
        return lp.defined() ? pack({wrap(token), wrap(lp)}) : wrap(token);
    });
}

// GdnError, the raw-stream function, and the addresses of the C functions in this order.
PyObject *bind(PyObject *, PyObject *const *v, Py_ssize_t nargs) {
    return guarded(nargs, 2 + kFunctions, [&]() -> PyObject * {
        void *f[kFunctions];
        for (int i = 0; i < kFunctions; ++i) {
            f[i] = PyLong_AsVoidPtr(v[2 + i]);
            if (!f[i]) {
                if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, "a function's address is zero");
                return nullptr;
            }
        }
        Py_INCREF(v[0]);
        Py_INCREF(v[1]);
        g_error = v[0];
        g_raw_stream = v[1];
        f_conv = (conv_fn)f[0];
        f_conv_step = (conv_step_fn)f[1];
        f_scan = (scan_fn)f[2];
        f_ssm_step = (ssm_step_fn)f[3];
        f_step = (step_fn)f[4];
        f_rope = (rope_fn)f[5];
        f_attn = (attn_fn)f[6];
        f_scan_ws = (scan_ws_fn)f[7];
        f_attn_ws = (attn_ws_fn)f[8];
        f_extend = (extend_fn)f[9];
        f_shared = (shared_fn)f[10];
        f_sample = (sample_fn)f[11];
        f_extend_ws = (extend_ws_fn)f[12];
        f_shared_ws = (shared_ws_fn)f[13];
        f_sample_ws = (sample_ws_fn)f[14];
        Py_RETURN_NONE;
    });
}

#define GDN_METHOD(name) {#name, (PyCFunction)(void (*)(void))name, METH_FASTCALL, nullptr}
PyMethodDef methods[] = {GDN_METHOD(bind), GDN_METHOD(conv), GDN_METHOD(conv_step), GDN_METHOD(scan), GDN_METHOD(ssm_step),
                         GDN_METHOD(step), GDN_METHOD(rope), GDN_METHOD(attn), GDN_METHOD(shared), GDN_METHOD(extend), GDN_METHOD(sample),
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_gdn_torch", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__gdn_torch(void) { return PyModule_Create(&module); }
