// Python binding of the operators around and beside the delta rule (module _native): checks torch tensors, allocates outputs and
// workspaces through torch, and calls the C ABI on torch's current stream.
//
// Marshalling only, like _binding.py, but without its interpreter time: a decode step's kernel takes 1.6 us, its checks in
// Python took 14 us.  The entry points of libgdn_gb300.so are handed over as addresses by init(), so this module links
// against torch alone.  Every entry turns C++ exceptions into Python ones.

#include <Python.h>

#include <ATen/ATen.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cmath>
#include <optional>
#include <string>
#include <utility>
#include <vector>

#include "../../include/gdn.h"

namespace {

// ------------------------------------------------------------------------------------------- the library's entries

#define GDN_ENTRIES(F)                                                                                          \
    F(glr_scan_fwd) F(glr_scan_bwd) F(glr_step) F(glr_workspace_size) F(gdn_qk_norm_fwd) F(gdn_qk_norm_bwd)      \
    F(gdn_qk_norm_workspace_size) F(gdn_short_conv_fwd) F(gdn_short_conv_bwd) F(gdn_short_conv_step)             \
    F(gdn_short_conv_workspace_size) F(lin_chunk_fwd) F(lin_chunk_bwd) F(lin_recurrent_step) F(lin_workspace_size) F(paged_append)      \
    F(paged_attn_step) F(paged_attn_workspace_size)
#define GDN_DECLARE(name) decltype(&::name) p_##name = nullptr;
GDN_ENTRIES(GDN_DECLARE)
PyObject* g_check = nullptr;       // _binding._check: raises GdnError for a status

struct Raised {};                  // a Python exception is set

[[noreturn]] void raise(PyObject* type, const std::string& message) {
    PyErr_SetString(type, message.c_str());
    throw Raised{};
}
[[noreturn]] void value_error(const std::string& message) { raise(PyExc_ValueError, message); }

void check(gdn_status st) {
    if (st == GDN_OK) return;
    PyObject* r = PyObject_CallFunction(g_check, "i", (int)st);
    Py_XDECREF(r);
    throw Raised{};
}
// an entry that launches: without the interpreter lock, as the driver may wait
template <typename F>
void launch(F f) {
    gdn_status st;
    Py_BEGIN_ALLOW_THREADS
    st = f();
    Py_END_ALLOW_THREADS
    check(st);
}

// ---------------------------------------------------------------------------------------------------- arguments

// The parameters of an entry, in order; the first `required` have no default.
struct Signature {
    const char* fn;
    std::vector<PyObject*> names;
    int required;
    Signature(const char* f, int r, std::initializer_list<const char*> n) : fn(f), required(r) {
        for (const char* s : n) names.push_back(PyUnicode_InternFromString(s));
    }
};
constexpr int kMaxArgs = 16;
struct Args {
    PyObject* v[kMaxArgs] = {};
    Args(const Signature& s, PyObject* const* args, Py_ssize_t nargs, PyObject* kwnames) {
        const int n = (int)s.names.size();
        if (nargs > n) raise(PyExc_TypeError, std::string(s.fn) + "() takes at most " + std::to_string(n) + " arguments");
        for (Py_ssize_t i = 0; i < nargs; ++i) v[i] = args[i];
        const Py_ssize_t kw = kwnames ? PyTuple_GET_SIZE(kwnames) : 0;
        for (Py_ssize_t i = 0; i < kw; ++i) {
            PyObject* name = PyTuple_GET_ITEM(kwnames, i);
            int at = 0;
            while (at < n && s.names[at] != name) ++at;
            if (at == n) {                       // (names are interned as a rule, not by law)
                at = 0;
                while (at < n && PyUnicode_Compare(s.names[at], name) != 0) ++at;
            }
            // (a name may be text that has no UTF-8 form: %U prints any)
            if (at == n) PyErr_Format(PyExc_TypeError, "%s() got an unexpected keyword argument '%U'", s.fn, name);
            else if (at < nargs) PyErr_Format(PyExc_TypeError, "%s() got multiple values for argument '%U'", s.fn, name);
            if (at == n || at < nargs) throw Raised{};
            v[at] = args[nargs + i];
        }
        for (int i = 0; i < s.required; ++i)
            if (!v[i]) {
                PyErr_Format(PyExc_TypeError, "%s() missing argument '%U'", s.fn, s.names[i]);
                throw Raised{};
            }
        for (int i = 0; i < n; ++i)
            if (v[i] == Py_None) v[i] = nullptr;
    }
};

bool truth(PyObject* o) {
    if (!o) return false;
    const int t = PyObject_IsTrue(o);
    if (t < 0) throw Raised{};
    return t != 0;
}

const at::Tensor& tensor(PyObject* o, const char* name) {
    if (!o || !THPVariable_Check(o)) raise(PyExc_TypeError, std::string(name) + " must be a torch.Tensor");
    return THPVariable_Unpack(o);
}

std::string text(at::IntArrayRef v) {
    std::string s = "(";
    for (size_t i = 0; i < v.size(); ++i) s += (i ? ", " : "") + std::to_string(v[i]);
    return s + ")";
}
std::string text(at::ScalarType t) { return c10::toString(t); }

gdn_dtype dtype_of(const at::Tensor& t, const char* name) {
    if (t.scalar_type() == at::kBFloat16) return GDN_BF16;
    if (t.scalar_type() == at::kFloat) return GDN_F32;
    value_error(std::string(name) + " must be float32 or bfloat16 (got " + text(t.scalar_type()) + ")");
}

void same(const at::Tensor& t, const char* name, at::IntArrayRef shape, at::ScalarType type, const at::Tensor& like) {
    if (t.sizes() != shape || t.scalar_type() != type || t.device() != like.device())
        value_error(std::string(name) + " must be " + text(type) + " of shape " + text(shape) + " on " + like.device().str() +
                    " (got " + text(t.scalar_type()) + " " + text(t.sizes()) + " on " + t.device().str() + ")");
}

// A contiguous tensor of this shape and type (none: nullptr).
void* dense(PyObject* o, const char* name, at::IntArrayRef shape, at::ScalarType type, const at::Tensor& like) {
    if (!o) return nullptr;
    const at::Tensor& t = tensor(o, name);
    same(t, name, shape, type, like);
    if (!t.is_contiguous())
        value_error(std::string(name) + " must be contiguous (strides " + text(t.strides()) + ")");
    return t.data_ptr();
}
float* dense_f32(PyObject* o, const char* name, at::IntArrayRef shape, const at::Tensor& like) {
    return static_cast<float*>(dense(o, name, shape, at::kFloat, like));
}

// The one spacing of the leading `n` dimensions of a strided tensor; `least` is what a row takes.
int64_t spacing(const at::Tensor& t, const char* name, int n, int64_t least, bool inner_ok) {
    int64_t ld = -1, rows = 1;
    bool ok = inner_ok;
    for (int i = n - 1; i >= 0; --i) {
        if (t.size(i) == 1) continue;
        if (ld < 0) ld = t.stride(i);
        else if (t.stride(i) != ld * rows) ok = false;
        rows *= t.size(i);
    }
    if (ld < 0) ld = least;
    if (!ok || ld < least)
        value_error(std::string(name) + " must have contiguous rows, evenly spaced (shape " + text(t.sizes()) + ", strides " +
                    text(t.strides()) + ")");
    return ld;
}
int64_t row_spacing(const at::Tensor& t, const char* name) {
    const int64_t D = t.size(-1);
    if (t.is_contiguous()) return D;
    return spacing(t, name, (int)t.dim() - 1, D, D == 1 || t.stride(-1) == 1);
}
// the head stride, and by reference the token stride, of a [..., H, d] tensor
int64_t head_spacing(const at::Tensor& t, const char* name, int64_t& token) {
    const int64_t H = t.size(-2), d = t.size(-1);
    if (t.is_contiguous()) {
        token = H * d;
        return d;
    }
    const int64_t hs = H > 1 ? t.stride(-2) : d;
    token = spacing(t, name, (int)t.dim() - 2, d, (d == 1 || t.stride(-1) == 1) && hs >= d);
    return hs;
}

struct Rows { void* ptr = nullptr; int64_t ld = 0; };
Rows rows(PyObject* o, const char* name, at::IntArrayRef shape, at::ScalarType type, const at::Tensor& like) {
    if (!o) return {};
    const at::Tensor& t = tensor(o, name);
    same(t, name, shape, type, like);
    return {t.data_ptr(), row_spacing(t, name)};
}

// The call's first tensor: on the current device; and the stream to launch on.  `stream` (a torch.cuda.Stream) becomes the
// current stream for the call, so that what is allocated belongs to it.
const at::Tensor& first(PyObject* o, const char* name, int dim) {
    const at::Tensor& t = tensor(o, name);
    if (dim > 0 && t.dim() != dim) value_error(std::string(name) + " must have " + std::to_string(dim) + " dimensions (got " +
                                               text(t.sizes()) + ")");
    dtype_of(t, name);
    if (!t.is_cuda()) value_error(std::string(name) + " must be a CUDA tensor");
    return t;
}
int64_t attr_int(PyObject* o, const char* name) {
    PyObject* a = PyObject_GetAttrString(o, name);
    if (!a) throw Raised{};
    const int64_t v = PyLong_AsLongLong(a);
    Py_DECREF(a);
    if (v == -1 && PyErr_Occurred()) throw Raised{};
    return v;
}
struct OnStream {
    c10::cuda::OptionalCUDAStreamGuard guard;
    void* handle;
    OnStream(PyObject* stream, const at::Tensor& x) {
        if (stream)
            guard.reset_stream(c10::cuda::CUDAStream::unpack3(attr_int(stream, "stream_id"),
                                                             (c10::DeviceIndex)attr_int(stream, "device_index"),
                                                             (c10::DeviceType)attr_int(stream, "device_type"))
                                   .unwrap());
        const auto here = c10::cuda::current_device();
        if (x.get_device() != here)
            value_error("the tensors are on cuda:" + std::to_string(x.get_device()) + ", the current device is cuda:" +
                        std::to_string((int)here));
        handle = c10::cuda::getCurrentCUDAStream(here).stream();
    }
};

at::Tensor empty(at::IntArrayRef shape, at::ScalarType type, const at::Tensor& like) {
    return at::detail::empty_cuda(shape, type, like.device(), std::nullopt);
}
// The caller's output buffer, or a new one; `keep` holds it.
void* output(PyObject* o, const char* name, at::IntArrayRef shape, at::ScalarType type, const at::Tensor& like, at::Tensor& keep) {
    if (o) {
        dense(o, name, shape, type, like);
        keep = THPVariable_Unpack(o);
    } else {
        keep = empty(shape, type, like);
    }
    return keep.data_ptr();
}
struct Workspace { void* ptr = nullptr; size_t bytes = 0; at::Tensor keep; };
Workspace workspace(PyObject* o, size_t need, const at::Tensor& like) {
    Workspace w;
    if (o) {
        const at::Tensor& t = tensor(o, "workspace");
        if (t.scalar_type() != at::kByte || t.device() != like.device() || !t.is_contiguous())
            value_error("workspace must be a contiguous uint8 tensor on " + like.device().str());
        w.keep = t;
    } else {
        if (need == 0) return w;
        w.keep = empty({(int64_t)need}, at::kByte, like);
    }
    w.ptr = w.keep.data_ptr();
    w.bytes = (size_t)w.keep.numel();
    return w;
}

struct Sequences { const int32_t* cu = nullptr; int n = 0; int64_t N = 0; };
Sequences sequences(PyObject* o, int64_t B, const at::Tensor& like) {
    if (!o) return {nullptr, 0, B};
    const at::Tensor& t = tensor(o, "cu_seqlens");
    if (t.scalar_type() != at::kInt || t.device() != like.device() || t.dim() != 1 || t.numel() < 2 || !t.is_contiguous())
        value_error("cu_seqlens must be a contiguous int32 vector of at least 2 offsets on " + like.device().str());
    return {t.data_ptr<int32_t>(), (int)(t.numel() - 1), t.numel() - 1};
}
int to_int(int64_t v, const char* what) {
    if (v > INT32_MAX) value_error(std::string(what) + " is too large (" + std::to_string(v) + ")");
    return (int)v;
}

PyObject* wrap(const at::Tensor& t) {
    if (!t.defined()) Py_RETURN_NONE;
    return THPVariable_Wrap(t);
}
PyObject* tuple_of(std::initializer_list<at::Tensor> ts) {
    PyObject* r = PyTuple_New((Py_ssize_t)ts.size());
    if (!r) throw Raised{};
    Py_ssize_t i = 0;
    for (const at::Tensor& t : ts) {
        PyObject* o = wrap(t);
        if (!o) {
            Py_DECREF(r);
            throw Raised{};
        }
        PyTuple_SET_ITEM(r, i++, o);
    }
    return r;
}
float* f32(const at::Tensor& t) { return t.defined() ? t.data_ptr<float>() : nullptr; }
void* ptr_of(const at::Tensor& t) { return t.defined() ? t.data_ptr() : nullptr; }

#define GDN_ENTRY(name) PyObject* name(PyObject*, PyObject* const* args, Py_ssize_t nargs, PyObject* kwnames)
#define GDN_BEGIN HANDLE_TH_ERRORS try {
#define GDN_END                     \
    }                               \
    catch (const Raised&) {         \
        return nullptr;             \
    }                               \
    END_HANDLE_TH_ERRORS

// ------------------------------------------------------------------------------------------- linear recurrence

struct Glr {
    Rows x, g, gi;
    float *A_log, *dt_bias;
    gdn_dtype dt, gdt;
    Glr(const at::Tensor& xt, PyObject* xo, PyObject* go, PyObject* io, PyObject* Ao, PyObject* dto) {
        const at::Tensor& gt = tensor(go, "g");
        const int64_t D = xt.size(-1);
        dt = dtype_of(xt, "x");
        gdt = dtype_of(gt, "g");
        x = rows(xo, "x", xt.sizes(), xt.scalar_type(), xt);
        g = rows(go, "g", xt.sizes(), gt.scalar_type(), xt);
        gi = rows(io, "in_gate", xt.sizes(), xt.scalar_type(), xt);
        A_log = dense_f32(Ao, "A_log", {D}, xt);
        dt_bias = dense_f32(dto, "dt_bias", {D}, xt);
    }
};

GDN_ENTRY(py_glr_scan_fwd) {
    GDN_BEGIN
    static const Signature sig("glr_scan_fwd", 2, {"x", "g", "in_gate", "A_log", "dt_bias", "normalize", "initial_state",
        "output_final_state", "cu_seqlens", "o", "final_state", "output_checkpoints", "workspace", "stream"});
    Args a(sig, args, nargs, kwnames);
    const at::Tensor& x = first(a.v[0], "x", 3);
    const Glr in(x, a.v[0], a.v[1], a.v[2], a.v[3], a.v[4]);
    const int64_t B = x.size(0), T = x.size(1), D = x.size(2);
    const Sequences s = sequences(a.v[8], B, x);
    const float* h0 = dense_f32(a.v[6], "initial_state", {s.N, D}, x);
    const int b = to_int(B, "B"), t = to_int(T, "T"), d = to_int(D, "D");
    size_t need = 0;
    check(p_glr_workspace_size(0, b, t, d, s.n, &need));
    const OnStream on(a.v[13], x);
    at::Tensor o, hT, ck;
    void* op = output(a.v[9], "o", x.sizes(), x.scalar_type(), x, o);
    if (a.v[10] || truth(a.v[7])) output(a.v[10], "final_state", {s.N, D}, at::kFloat, x, hT);
    const bool save = truth(a.v[11]), norm = truth(a.v[5]);
    if (save) ck = empty({B, (T + 63) / 64, D}, at::kFloat, x);
    const Workspace ws = workspace(a.v[12], need, x);
    launch([&] {
        return p_glr_scan_fwd(in.x.ptr, in.g.ptr, in.gi.ptr, in.A_log, in.dt_bias, norm, h0, f32(hT), s.cu, s.n, op, f32(ck), b, t, d,
                              in.x.ld, in.g.ld, in.gi.ld, in.dt, in.gdt, ws.ptr, ws.bytes, on.handle);
    });
    if (save) return tuple_of({o, hT, ck});
    return tuple_of({o, hT});
    GDN_END
}

GDN_ENTRY(py_glr_scan_bwd) {
    GDN_BEGIN
    static const Signature sig("glr_scan_bwd", 3, {"x", "g", "d_o", "in_gate", "A_log", "dt_bias", "normalize", "initial_state",
        "d_final_state", "cu_seqlens", "checkpoints", "workspace", "stream"});
    Args a(sig, args, nargs, kwnames);
    const at::Tensor& x = first(a.v[0], "x", 3);
    const Glr in(x, a.v[0], a.v[1], a.v[3], a.v[4], a.v[5]);
    const int64_t B = x.size(0), T = x.size(1), D = x.size(2);
    const Sequences s = sequences(a.v[9], B, x);
    tensor(a.v[2], "d_o");
    const void* dO = dense(a.v[2], "d_o", x.sizes(), x.scalar_type(), x);
    const float* h0 = dense_f32(a.v[7], "initial_state", {s.N, D}, x);
    const float* dhT = dense_f32(a.v[8], "d_final_state", {s.N, D}, x);
    const float* ck = dense_f32(a.v[10], "checkpoints", {B, (T + 63) / 64, D}, x);
    const int b = to_int(B, "B"), t = to_int(T, "T"), d = to_int(D, "D");
    size_t need = 0;
    check(p_glr_workspace_size(1, b, t, d, s.n, &need));
    const OnStream on(a.v[12], x);
    const bool norm = truth(a.v[6]);
    at::Tensor dx = empty(x.sizes(), x.scalar_type(), x), dg = empty(x.sizes(), in.gdt == GDN_BF16 ? at::kBFloat16 : at::kFloat, x);
    at::Tensor di, dh0, dA, ddt;
    if (in.gi.ptr || a.v[3]) di = empty(x.sizes(), x.scalar_type(), x);
    if (h0 || a.v[7]) dh0 = empty({s.N, D}, at::kFloat, x);
    if (a.v[4]) dA = empty({D}, at::kFloat, x);
    if (a.v[5]) ddt = empty({D}, at::kFloat, x);
    const Workspace ws = workspace(a.v[11], need, x);
    launch([&] {
        return p_glr_scan_bwd(in.x.ptr, in.g.ptr, in.gi.ptr, in.A_log, in.dt_bias, norm, h0, dO, dhT, s.cu, s.n, ck, ptr_of(dx), ptr_of(dg),
                              ptr_of(di), f32(dh0), f32(dA), f32(ddt), b, t, d, in.x.ld, in.g.ld, in.gi.ld, in.dt, in.gdt, ws.ptr,
                              ws.bytes, on.handle);
    });
    return tuple_of({dx, dg, di, dh0, dA, ddt});
    GDN_END
}

GDN_ENTRY(py_glr_step) {
    GDN_BEGIN
    static const Signature sig("glr_step", 3, {"x", "g", "state", "in_gate", "A_log", "dt_bias", "normalize", "state_out", "o", "stream"});
    Args a(sig, args, nargs, kwnames);
    const at::Tensor& x = first(a.v[0], "x", 2);
    const Glr in(x, a.v[0], a.v[1], a.v[3], a.v[4], a.v[5]);
    tensor(a.v[2], "state");
    float* h = dense_f32(a.v[2], "state", x.sizes(), x);
    float* h_out = a.v[7] ? dense_f32(a.v[7], "state_out", x.sizes(), x) : h;
    const int n = to_int(x.size(0), "N"), d = to_int(x.size(1), "D");
    const bool norm = truth(a.v[6]);
    const OnStream on(a.v[9], x);
    at::Tensor o;
    void* op = output(a.v[8], "o", x.sizes(), x.scalar_type(), x, o);
    launch([&] {
        return p_glr_step(in.x.ptr, in.g.ptr, in.gi.ptr, in.A_log, in.dt_bias, norm, h, h_out, op, n, d, in.x.ld, in.g.ld, in.gi.ld,
                          in.dt, in.gdt, on.handle);
    });
    return wrap(o);
    GDN_END
}

// ------------------------------------------------------------------------------------------- query/key head norm

struct Qk {
    void *q, *k;
    float *wq, *wk, *cos, *sin, eps;
    const int32_t* pos;
    gdn_norm norm;
    int n_pos = 0, rot = 0, T, Hq, Hk, d;
    bool interleaved;
    int64_t n = 1, qt, qh, kt, kh;
    gdn_dtype dt;
    // v: q_weight, k_weight, norm, eps, cos, sin, positions, interleaved
    Qk(const at::Tensor& qx, PyObject* ko, PyObject* const* v) {
        if (qx.dim() < 3) value_error("q must be a [..., heads, d] tensor");
        const at::Tensor& kx = tensor(ko, "k");
        const at::IntArrayRef lead = qx.sizes().slice(0, qx.dim() - 2);
        if (kx.dim() != qx.dim() || kx.sizes().slice(0, kx.dim() - 2) != lead || kx.size(-1) != qx.size(-1) ||
            kx.scalar_type() != qx.scalar_type() || kx.device() != qx.device())
            value_error("k must match q but for its heads: " + text(qx.scalar_type()) + " " + text(qx.sizes()) + " on " +
                        qx.device().str() + " (got " + text(kx.scalar_type()) + " " + text(kx.sizes()) + " on " + kx.device().str() + ")");
        dt = dtype_of(qx, "q");
        q = qx.data_ptr();
        k = kx.data_ptr();
        qh = head_spacing(qx, "q", qt);
        kh = head_spacing(kx, "k", kt);
        Hq = to_int(qx.size(-2), "heads");
        Hk = to_int(kx.size(-2), "heads");
        d = to_int(qx.size(-1), "d");
        for (int64_t s : lead) n *= s;
        // without positions a token's position is its index along the last leading dimension
        T = to_int(lead.back() > 0 ? lead.back() : 1, "T");
        wq = dense_f32(v[0], "q_weight", {d}, qx);
        wk = dense_f32(v[1], "k_weight", {d}, qx);
        norm = GDN_NORM_RMS;
        if (v[2]) {
            const auto is = [&](const char* n) { return PyUnicode_CompareWithASCIIString(v[2], n) == 0; };
            if (!PyUnicode_Check(v[2]) || (!is("rms") && !is("l2"))) value_error("norm must be 'rms' or 'l2'");
            if (is("l2")) norm = GDN_NORM_L2;
        }
        eps = 1e-6f;
        if (v[3]) {
            eps = (float)PyFloat_AsDouble(v[3]);
            if (PyErr_Occurred()) throw Raised{};
        }
        if (!v[4] != !v[5]) value_error("cos and sin go together");
        cos = sin = nullptr;
        if (v[4]) {
            const at::Tensor& c = tensor(v[4], "cos");
            if (c.dim() != 2) value_error("cos must be a [positions, rotary_dim / 2] tensor");
            n_pos = to_int(c.size(0), "positions");
            rot = to_int(2 * c.size(1), "rotary_dim");
            cos = dense_f32(v[4], "cos", c.sizes(), qx);
            sin = dense_f32(v[5], "sin", c.sizes(), qx);
        }
        pos = static_cast<const int32_t*>(dense(v[6], "positions", lead, at::kInt, qx));
        interleaved = truth(v[7]);
    }
};

GDN_ENTRY(py_gdn_qk_norm_fwd) {
    GDN_BEGIN
    static const Signature sig("gdn_qk_norm_fwd", 2, {"q", "k", "q_weight", "k_weight", "norm", "eps", "cos", "sin", "positions",
        "interleaved", "q_out", "k_out", "stream"});
    Args a(sig, args, nargs, kwnames);
    const at::Tensor& q = first(a.v[0], "q", 0);
    const Qk in(q, a.v[1], a.v + 2);
    const OnStream on(a.v[12], q);
    at::Tensor qo, ko;
    void* qp = output(a.v[10], "q_out", q.sizes(), q.scalar_type(), q, qo);
    void* kp = output(a.v[11], "k_out", THPVariable_Unpack(a.v[1]).sizes(), q.scalar_type(), q, ko);
    launch([&] {
        return p_gdn_qk_norm_fwd(in.q, in.k, in.wq, in.wk, in.norm, in.eps, in.cos, in.sin, in.n_pos, in.rot, in.interleaved, in.pos,
                                 qp, kp, in.n, in.T, in.Hq, in.Hk, in.d, in.qt, in.qh, in.kt, in.kh, in.dt, on.handle);
    });
    return tuple_of({qo, ko});
    GDN_END
}

GDN_ENTRY(py_gdn_qk_norm_bwd) {
    GDN_BEGIN
    static const Signature sig("gdn_qk_norm_bwd", 4, {"q", "k", "d_q_out", "d_k_out", "q_weight", "k_weight", "norm", "eps", "cos",
        "sin", "positions", "interleaved", "workspace", "stream"});
    Args a(sig, args, nargs, kwnames);
    const at::Tensor& q = first(a.v[0], "q", 0);
    const Qk in(q, a.v[1], a.v + 4);
    const at::Tensor& k = THPVariable_Unpack(a.v[1]);
    tensor(a.v[2], "d_q_out");
    tensor(a.v[3], "d_k_out");
    const void* dqo = dense(a.v[2], "d_q_out", q.sizes(), q.scalar_type(), q);
    const void* dko = dense(a.v[3], "d_k_out", k.sizes(), q.scalar_type(), q);
    size_t need = 0;
    check(p_gdn_qk_norm_workspace_size(in.n, in.Hq, in.Hk, in.d, &need));
    const OnStream on(a.v[13], q);
    at::Tensor dq = empty(q.sizes(), q.scalar_type(), q), dk = empty(k.sizes(), q.scalar_type(), q), dwq, dwk;
    if (a.v[4]) dwq = empty({in.d}, at::kFloat, q);
    if (a.v[5]) dwk = empty({in.d}, at::kFloat, q);
    const Workspace ws = workspace(a.v[12], a.v[4] || a.v[5] ? need : 0, q);
    launch([&] {
        return p_gdn_qk_norm_bwd(in.q, in.k, dqo, dko, in.wq, in.wk, in.norm, in.eps, in.cos, in.sin, in.n_pos, in.rot, in.interleaved,
                                 in.pos, ptr_of(dq), ptr_of(dk), f32(dwq), f32(dwk), in.n, in.T, in.Hq, in.Hk, in.d, in.qt, in.qh, in.kt,
                                 in.kh, in.dt, ws.ptr, ws.bytes, on.handle);
    });
    return tuple_of({dq, dk, dwq, dwk});
    GDN_END
}

// -------------------------------------------------------------------------------------------- short convolution

struct Conv {
    Rows x;
    float *w, *b;
    gdn_activation act;
    gdn_dtype dt;
    int64_t W;
    // act_given: whether the caller named an activation (None is one)
    Conv(const at::Tensor& xt, PyObject* xo, PyObject* wo, PyObject* bo, PyObject* act_o, bool act_given) {
        const int64_t D = xt.size(-1);
        dt = dtype_of(xt, "x");
        const at::Tensor& wt = tensor(wo, "weight");
        if (wt.dim() != 2) value_error("weight must be a [D, W] tensor");
        W = wt.size(1);
        w = dense_f32(wo, "weight", {D, W}, xt);
        b = dense_f32(bo, "bias", {D}, xt);
        x = rows(xo, "x", xt.sizes(), xt.scalar_type(), xt);
        act = act_given && !act_o ? GDN_ACT_NONE : GDN_ACT_SILU;
        if (act_o && (!PyUnicode_Check(act_o) || PyUnicode_CompareWithASCIIString(act_o, "silu") != 0))
            value_error("activation must be None or 'silu'");
    }
};
// whether argument `at` of the signature was passed at all
bool passed(const Signature& s, int at, Py_ssize_t nargs, PyObject* kwnames) {
    if (at < nargs) return true;
    const Py_ssize_t kw = kwnames ? PyTuple_GET_SIZE(kwnames) : 0;
    for (Py_ssize_t i = 0; i < kw; ++i)
        if (PyUnicode_Compare(PyTuple_GET_ITEM(kwnames, i), s.names[at]) == 0) return true;
    return false;
}

GDN_ENTRY(py_gdn_short_conv_fwd) {
    GDN_BEGIN
    static const Signature sig("gdn_short_conv_fwd", 2, {"x", "weight", "bias", "activation", "initial_state", "output_final_state",
        "cu_seqlens", "y", "final_state", "stream"});
    Args a(sig, args, nargs, kwnames);
    const at::Tensor& x = first(a.v[0], "x", 3);
    const Conv in(x, a.v[0], a.v[1], a.v[2], a.v[3], passed(sig, 3, nargs, kwnames));
    const int64_t B = x.size(0), T = x.size(1), D = x.size(2);
    const Sequences s = sequences(a.v[6], B, x);
    const int b = to_int(B, "B"), t = to_int(T, "T"), d = to_int(D, "D"), w = to_int(in.W, "W");
    const void* h0 = dense(a.v[4], "initial_state", {s.N, in.W - 1, D}, x.scalar_type(), x);
    const OnStream on(a.v[9], x);
    at::Tensor y, hT;
    void* yp = output(a.v[7], "y", x.sizes(), x.scalar_type(), x, y);
    if (a.v[8] || truth(a.v[5])) output(a.v[8], "final_state", {s.N, in.W - 1, D}, x.scalar_type(), x, hT);
    launch([&] {
        return p_gdn_short_conv_fwd(in.x.ptr, in.w, in.b, in.act, h0, ptr_of(hT), s.cu, s.n, yp, b, t, d, w, in.x.ld, in.dt, on.handle);
    });
    return tuple_of({y, hT});
    GDN_END
}

GDN_ENTRY(py_gdn_short_conv_bwd) {
    GDN_BEGIN
    static const Signature sig("gdn_short_conv_bwd", 3, {"x", "weight", "d_y", "bias", "activation", "initial_state", "d_final_state",
        "cu_seqlens", "workspace", "stream"});
    Args a(sig, args, nargs, kwnames);
    const at::Tensor& x = first(a.v[0], "x", 3);
    const Conv in(x, a.v[0], a.v[1], a.v[3], a.v[4], passed(sig, 4, nargs, kwnames));
    const int64_t B = x.size(0), T = x.size(1), D = x.size(2);
    const Sequences s = sequences(a.v[7], B, x);
    const int b = to_int(B, "B"), t = to_int(T, "T"), d = to_int(D, "D"), w = to_int(in.W, "W");
    tensor(a.v[2], "d_y");
    const void* dy = dense(a.v[2], "d_y", x.sizes(), x.scalar_type(), x);
    const void* h0 = dense(a.v[5], "initial_state", {s.N, in.W - 1, D}, x.scalar_type(), x);
    const void* dhT = dense(a.v[6], "d_final_state", {s.N, in.W - 1, D}, x.scalar_type(), x);
    size_t need = 0;
    check(p_gdn_short_conv_workspace_size(b, t, d, w, &need));
    const OnStream on(a.v[9], x);
    at::Tensor dx = empty(x.sizes(), x.scalar_type(), x), dw = empty({D, in.W}, at::kFloat, x), db, dh0;
    if (a.v[3]) db = empty({D}, at::kFloat, x);
    if (a.v[5]) dh0 = empty({s.N, in.W - 1, D}, x.scalar_type(), x);
    const Workspace ws = workspace(a.v[8], need, x);
    launch([&] {
        return p_gdn_short_conv_bwd(in.x.ptr, in.w, in.b, in.act, h0, dy, dhT, s.cu, s.n, ptr_of(dx), f32(dw), f32(db), ptr_of(dh0), b, t, d,
                                    w, in.x.ld, in.dt, ws.ptr, ws.bytes, on.handle);
    });
    return tuple_of({dx, dw, db, dh0});
    GDN_END
}

GDN_ENTRY(py_gdn_short_conv_step) {
    GDN_BEGIN
    static const Signature sig("gdn_short_conv_step", 3, {"x", "state", "weight", "bias", "activation", "state_out", "y", "stream"});
    Args a(sig, args, nargs, kwnames);
    const at::Tensor& x = first(a.v[0], "x", 2);
    const Conv in(x, a.v[0], a.v[2], a.v[3], a.v[4], passed(sig, 4, nargs, kwnames));
    const int64_t N = x.size(0), D = x.size(1);
    const int n = to_int(N, "N"), d = to_int(D, "D"), w = to_int(in.W, "W");
    tensor(a.v[1], "state");
    const at::IntArrayRef::value_type shape[3] = {N, in.W - 1, D};
    void* h = dense(a.v[1], "state", shape, x.scalar_type(), x);
    void* h_out = a.v[5] ? dense(a.v[5], "state_out", shape, x.scalar_type(), x) : h;
    const OnStream on(a.v[7], x);
    at::Tensor y;
    void* yp = output(a.v[6], "y", x.sizes(), x.scalar_type(), x, y);
    launch([&] {
        return p_gdn_short_conv_step(in.x.ptr, in.w, in.b, in.act, h, h_out, yp, n, d, w, in.x.ld, in.dt, on.handle);
    });
    return wrap(y);
    GDN_END
}

// ---------------------------------------------------------------------------------------------- linear attention

float number(PyObject* o, double otherwise) {
    if (!o) return (float)otherwise;
    const double x = PyFloat_AsDouble(o);
    if (x == -1.0 && PyErr_Occurred()) throw Raised{};
    return (float)x;
}

// A [..., heads, d] tensor of tokens with its strides.
struct Heads { void* ptr = nullptr; int64_t tok = 0, head = 0; };
Heads heads(PyObject* o, const char* name, at::IntArrayRef shape, at::ScalarType type, const at::Tensor& like) {
    const at::Tensor& t = tensor(o, name);
    same(t, name, shape, type, like);
    Heads h;
    h.ptr = t.data_ptr();
    h.head = head_spacing(t, name, h.tok);
    return h;
}

// q, k, v and g of the lin_ entries; v is [..., H, d_v] of `dim` dimensions.
struct Lin {
    Heads q, k, v;
    float* g;
    bool g_per_head;
    int Hk, H, dk, dv;
    float scale;
    gdn_dtype dt;
    std::vector<int64_t> q_shape;
    Lin(const at::Tensor& vt, PyObject* qo, PyObject* ko, PyObject* vo, PyObject* go, PyObject* scale_o) {
        const at::Tensor& qt = tensor(qo, "q");
        const at::Tensor& gt = tensor(go, "g");
        const int64_t dim = vt.dim();
        if (qt.dim() != dim) value_error("q must have " + std::to_string(dim) + " dimensions (got " + text(qt.sizes()) + ")");
        dt = dtype_of(vt, "v");
        q_shape.assign(vt.sizes().begin(), vt.sizes().end());
        q_shape[dim - 2] = qt.size(-2);
        q_shape[dim - 1] = qt.size(-1);
        Hk = to_int(qt.size(-2), "H_k");
        dk = to_int(qt.size(-1), "d_k");
        H = to_int(vt.size(-2), "H");
        dv = to_int(vt.size(-1), "d_v");
        v = heads(vo, "v", vt.sizes(), vt.scalar_type(), vt);
        q = heads(qo, "q", q_shape, vt.scalar_type(), vt);
        k = heads(ko, "k", q_shape, vt.scalar_type(), vt);
        g_per_head = gt.dim() == 1 && dim > 2;
        if (g_per_head) g = dense_f32(go, "g", {(int64_t)H}, vt);
        else g = dense_f32(go, "g", vt.sizes().slice(0, dim - 1), vt);
        scale = number(scale_o, 1.0 / std::sqrt((double)(dk > 0 ? dk : 1)));
    }
};

gdn_algo algo_of(PyObject* o) {
    if (!o) return GDN_ALGO_AUTO;
    if (!PyUnicode_Check(o)) raise(PyExc_TypeError, "algo must be text");
    for (const auto& [name, value] : {std::pair{"auto", GDN_ALGO_AUTO}, std::pair{"generic", GDN_ALGO_GENERIC}, std::pair{"tcgen05", GDN_ALGO_TCGEN05}})
        if (PyUnicode_CompareWithASCIIString(o, name) == 0) return value;
    value_error("algo must be 'auto', 'generic' or 'tcgen05'");
}

GDN_ENTRY(py_lin_chunk_fwd) {
    GDN_BEGIN
    static const Signature sig("lin_chunk_fwd", 4, {"q", "k", "v", "g", "scale", "initial_state", "output_final_state", "cu_seqlens",
        "algo", "o", "final_state", "workspace", "stream"});
    Args a(sig, args, nargs, kwnames);
    const at::Tensor& v = first(a.v[2], "v", 4);
    const Lin in(v, a.v[0], a.v[1], a.v[2], a.v[3], a.v[4]);
    const int64_t B = v.size(0), T = v.size(1);
    const Sequences s = sequences(a.v[7], B, v);
    const int64_t shape[4] = {s.N, in.H, in.dk, in.dv};
    const float* h0 = dense_f32(a.v[5], "initial_state", shape, v);
    const int b = to_int(B, "B"), t = to_int(T, "T");
    const gdn_algo algo = algo_of(a.v[8]);
    size_t need = 0;
    check(p_lin_workspace_size(0, b, t, in.Hk, in.H, in.dk, in.dv, s.n, &need));
    const OnStream on(a.v[12], v);
    at::Tensor o, hT;
    void* op = output(a.v[9], "o", v.sizes(), v.scalar_type(), v, o);
    if (a.v[10] || truth(a.v[6])) output(a.v[10], "final_state", shape, at::kFloat, v, hT);
    const Workspace ws = workspace(a.v[11], need, v);
    launch([&] {
        return p_lin_chunk_fwd(in.q.ptr, in.k.ptr, in.v.ptr, in.g, in.g_per_head, in.scale, h0, f32(hT), s.cu, s.n, op, b, t, in.Hk, in.H,
                               in.dk, in.dv, in.q.tok, in.q.head, in.k.tok, in.k.head, in.v.tok, in.v.head, in.dt, algo, ws.ptr,
                               ws.bytes, on.handle);
    });
    return tuple_of({o, hT});
    GDN_END
}

GDN_ENTRY(py_lin_chunk_bwd) {
    GDN_BEGIN
    static const Signature sig("lin_chunk_bwd", 5, {"q", "k", "v", "g", "d_o", "scale", "initial_state", "d_final_state", "cu_seqlens",
        "algo", "workspace", "stream"});
    Args a(sig, args, nargs, kwnames);
    const at::Tensor& v = first(a.v[2], "v", 4);
    const Lin in(v, a.v[0], a.v[1], a.v[2], a.v[3], a.v[5]);
    const int64_t B = v.size(0), T = v.size(1);
    const Sequences s = sequences(a.v[8], B, v);
    const int64_t shape[4] = {s.N, in.H, in.dk, in.dv};
    tensor(a.v[4], "d_o");
    const void* dO = dense(a.v[4], "d_o", v.sizes(), v.scalar_type(), v);
    const float* h0 = dense_f32(a.v[6], "initial_state", shape, v);
    const float* dhT = dense_f32(a.v[7], "d_final_state", shape, v);
    const int b = to_int(B, "B"), t = to_int(T, "T");
    const gdn_algo algo = algo_of(a.v[9]);
    size_t need = 0;
    check(p_lin_workspace_size(1, b, t, in.Hk, in.H, in.dk, in.dv, s.n, &need));
    const OnStream on(a.v[11], v);
    at::Tensor dq = empty(in.q_shape, v.scalar_type(), v), dk = empty(in.q_shape, v.scalar_type(), v);
    at::Tensor dv = empty(v.sizes(), v.scalar_type(), v), dg, dh0;
    if (in.g_per_head) dg = empty({(int64_t)in.H}, at::kFloat, v);
    else dg = empty(v.sizes().slice(0, 3), at::kFloat, v);
    if (a.v[6]) dh0 = empty(shape, at::kFloat, v);
    const Workspace ws = workspace(a.v[10], need, v);
    launch([&] {
        return p_lin_chunk_bwd(in.q.ptr, in.k.ptr, in.v.ptr, in.g, in.g_per_head, in.scale, h0, dO, dhT, s.cu, s.n, ptr_of(dq), ptr_of(dk),
                               ptr_of(dv), f32(dg), f32(dh0), b, t, in.Hk, in.H, in.dk, in.dv, in.q.tok, in.q.head, in.k.tok, in.k.head,
                               in.v.tok, in.v.head, in.dt, algo, ws.ptr, ws.bytes, on.handle);
    });
    return tuple_of({dq, dk, dv, dg, dh0});
    GDN_END
}

GDN_ENTRY(py_lin_recurrent_step) {
    GDN_BEGIN
    static const Signature sig("lin_recurrent_step", 5, {"q", "k", "v", "g", "state", "scale", "state_out", "o", "stream"});
    Args a(sig, args, nargs, kwnames);
    const at::Tensor& v = first(a.v[2], "v", 3);
    const Lin in(v, a.v[0], a.v[1], a.v[2], a.v[3], a.v[5]);
    const int64_t shape[4] = {v.size(0), in.H, in.dk, in.dv};
    tensor(a.v[4], "state");
    float* h = dense_f32(a.v[4], "state", shape, v);
    float* h_out = a.v[6] ? dense_f32(a.v[6], "state_out", shape, v) : h;
    const int n = to_int(v.size(0), "N");
    const OnStream on(a.v[8], v);
    at::Tensor o;
    void* op = output(a.v[7], "o", v.sizes(), v.scalar_type(), v, o);
    launch([&] {
        return p_lin_recurrent_step(in.q.ptr, in.k.ptr, in.v.ptr, in.g, in.g_per_head, in.scale, h, h_out, op, n, in.Hk, in.H, in.dk, in.dv,
                                    in.q.tok, in.q.head, in.k.tok, in.k.head, in.v.tok, in.v.head, in.dt, on.handle);
    });
    return wrap(o);
    GDN_END
}

// --------------------------------------------------------------------------------------------------- paged cache

gdn_paged_side paged_side(const at::Tensor& t, const char* name) {
    const int64_t d = t.size(3);
    if (d > 1 && t.stride(3) != 1) value_error(std::string(name) + " must have contiguous channels (strides " + text(t.strides()) + ")");
    gdn_paged_side s;
    s.data = t.data_ptr();
    // (a dimension of one has a stride of no meaning)
    s.page_stride = t.size(0) > 1 ? t.stride(0) : d;
    s.slot_stride = t.size(1) > 1 ? t.stride(1) : d;
    s.head_stride = t.size(2) > 1 ? t.stride(2) : d;
    return s;
}

gdn_paged_cache paged_cache(const at::Tensor& like, PyObject* ko, PyObject* vo, PyObject* to, PyObject* lo) {
    const at::Tensor& k = tensor(ko, "k_cache");
    const at::Tensor& v = tensor(vo, "v_cache");
    const at::Tensor& table = tensor(to, "block_table");
    const at::Tensor& lengths = tensor(lo, "lengths");
    if (k.dim() != 4) value_error("k_cache must be [n_pages, page_size, H_k, d] (got " + text(k.sizes()) + ")");
    same(k, "k_cache", k.sizes(), like.scalar_type(), like);
    same(v, "v_cache", k.sizes(), like.scalar_type(), like);
    if (lengths.dim() != 1 || lengths.scalar_type() != at::kInt || lengths.device() != like.device() || !lengths.is_contiguous())
        value_error("lengths must be a contiguous int32 vector on " + like.device().str());
    if (table.dim() != 2 || table.scalar_type() != at::kInt || table.device() != like.device() || table.size(0) != lengths.size(0) ||
        (table.size(1) > 1 && table.stride(1) != 1))
        value_error("block_table must be int32 of shape (" + std::to_string(lengths.size(0)) + ", max_pages) with contiguous rows on " +
                    like.device().str() + " (got " + text(table.scalar_type()) + " " + text(table.sizes()) + ")");
    gdn_paged_cache c{};
    c.k = paged_side(k, "k_cache");
    c.v = paged_side(v, "v_cache");
    c.block_table = table.numel() ? table.data_ptr<int32_t>() : nullptr;
    c.lengths = lengths.data_ptr<int32_t>();
    c.table_stride = table.size(0) > 1 ? table.stride(0) : table.size(1);
    c.N = to_int(lengths.size(0), "N");
    c.max_pages = to_int(table.size(1), "max_pages");
    c.n_pages = to_int(k.size(0), "n_pages");
    c.page_size = to_int(k.size(1), "page_size");
    c.H_k = to_int(k.size(2), "H_k");
    c.d = to_int(k.size(3), "d");
    c.dtype = dtype_of(k, "k_cache");
    return c;
}

GDN_ENTRY(py_paged_append) {
    GDN_BEGIN
    static const Signature sig("paged_append", 6, {"k", "v", "k_cache", "v_cache", "block_table", "lengths", "q", "cu_seqlens", "cos",
        "sin", "interleaved", "q_out", "stream"});
    Args a(sig, args, nargs, kwnames);
    const at::Tensor& k = first(a.v[0], "k", 3);
    const gdn_paged_cache c = paged_cache(k, a.v[2], a.v[3], a.v[4], a.v[5]);
    const int64_t n = k.size(0), shape[3] = {n, c.H_k, c.d};
    const Heads kh = heads(a.v[0], "k", shape, k.scalar_type(), k), vh = heads(a.v[1], "v", shape, k.scalar_type(), k);
    Heads qh;
    int64_t q_shape[3] = {n, 0, c.d};
    if (a.v[6]) {
        const at::Tensor& q = tensor(a.v[6], "q");
        if (q.dim() != 3) value_error("q must have 3 dimensions (got " + text(q.sizes()) + ")");
        q_shape[1] = q.size(1);
        qh = heads(a.v[6], "q", q_shape, k.scalar_type(), k);
    } else if (a.v[11]) {
        value_error("q_out is given without q");
    }
    const Sequences s = sequences(a.v[7], c.N, k);
    if (s.cu && s.n != c.N)
        value_error("cu_seqlens must have one offset more than lengths (got " + std::to_string(s.n + 1) + " for " + std::to_string(c.N) +
                    " sequences)");
    int64_t n_pos = 0, half = 0;
    const float *cos = nullptr, *sin = nullptr;
    if (!a.v[8] != !a.v[9]) value_error("cos and sin go together");
    if (a.v[8]) {
        const at::Tensor& t = tensor(a.v[8], "cos");
        if (t.dim() != 2) value_error("cos must be [positions, rotary_dim / 2] (got " + text(t.sizes()) + ")");
        n_pos = t.size(0);
        half = t.size(1);
        cos = dense_f32(a.v[8], "cos", t.sizes(), k);
        sin = dense_f32(a.v[9], "sin", t.sizes(), k);
    }
    const int np = to_int(n_pos, "positions"), rot = to_int(2 * half, "rotary_dim"), hq = to_int(q_shape[1], "H_q");
    const bool interleaved = truth(a.v[10]);
    const OnStream on(a.v[12], k);
    at::Tensor qo;
    void* qp = a.v[6] ? output(a.v[11], "q_out", q_shape, k.scalar_type(), k, qo) : nullptr;
    launch([&] {
        return p_paged_append(kh.ptr, vh.ptr, qh.ptr, &c, s.cu, cos, sin, np, rot, interleaved, qp, n, hq, kh.tok, kh.head, vh.tok, vh.head,
                              qh.tok, qh.head, on.handle);
    });
    return wrap(qo);
    GDN_END
}

GDN_ENTRY(py_paged_attn_step) {
    GDN_BEGIN
    static const Signature sig("paged_attn_step", 5, {"q", "k_cache", "v_cache", "block_table", "lengths", "scale", "o", "output_lse",
        "workspace", "stream"});
    Args a(sig, args, nargs, kwnames);
    const at::Tensor& q = first(a.v[0], "q", 3);
    const gdn_paged_cache c = paged_cache(q, a.v[1], a.v[2], a.v[3], a.v[4]);
    const int64_t shape[3] = {c.N, q.size(1), c.d};
    const Heads qh = heads(a.v[0], "q", shape, q.scalar_type(), q);
    const int hq = to_int(q.size(1), "H_q");
    const float scale = number(a.v[5], 1.0 / std::sqrt((double)c.d));
    size_t need = 0;
    check(p_paged_attn_workspace_size(c.N, hq, c.H_k, c.d, c.max_pages, c.page_size, &need));
    const bool with_lse = truth(a.v[7]);
    const OnStream on(a.v[9], q);
    at::Tensor o, lse;
    void* op = output(a.v[6], "o", shape, q.scalar_type(), q, o);
    if (with_lse) lse = empty({(int64_t)c.N, (int64_t)hq}, at::kFloat, q);
    const Workspace ws = workspace(a.v[8], need, q);
    launch([&] { return p_paged_attn_step(qh.ptr, &c, scale, op, f32(lse), hq, qh.tok, qh.head, ws.ptr, ws.bytes, on.handle); });
    if (with_lse) return tuple_of({o, lse});
    return wrap(o);
    GDN_END
}

// ------------------------------------------------------------------------------------------------------- module

// (row stride) of a [..., D] tensor, (token stride, head stride) of a [..., H, d] one: what the entries pass on
GDN_ENTRY(py_spacing) {
    GDN_BEGIN
    static const Signature sig("spacing", 1, {"t", "heads"});
    Args a(sig, args, nargs, kwnames);
    const at::Tensor& t = tensor(a.v[0], "t");
    if (!truth(a.v[1])) return Py_BuildValue("(L)", (long long)row_spacing(t, "t"));
    int64_t token = 0;
    const int64_t head = head_spacing(t, "t", token);
    return Py_BuildValue("(LL)", (long long)token, (long long)head);
    GDN_END
}

// init(check, {name: address})
PyObject* py_init(PyObject*, PyObject* const* args, Py_ssize_t nargs) {
    if (nargs != 2 || !PyDict_Check(args[1])) {
        PyErr_SetString(PyExc_TypeError, "init(check, addresses)");
        return nullptr;
    }
#define GDN_BIND(name)                                                                     \
    {                                                                                      \
        PyObject* v = PyDict_GetItemString(args[1], #name);                                \
        void* p = v ? PyLong_AsVoidPtr(v) : nullptr;                                       \
        if (!p) {                                                                          \
            if (!PyErr_Occurred()) PyErr_SetString(PyExc_KeyError, #name);                 \
            return nullptr;                                                                \
        }                                                                                  \
        p_##name = reinterpret_cast<decltype(&::name)>(p);                                 \
    }
    GDN_ENTRIES(GDN_BIND)
    Py_INCREF(args[0]);
    Py_XSETREF(g_check, args[0]);
    Py_RETURN_NONE;
}

#define GDN_METHOD(name, doc) \
    {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(py_##name)), METH_FASTCALL | METH_KEYWORDS, doc}
PyMethodDef methods[] = {
    GDN_METHOD(glr_scan_fwd,
        "glr_scan_fwd(x, g, in_gate=None, A_log=None, dt_bias=None, normalize=False, initial_state=None, "
        "output_final_state=False, cu_seqlens=None, o=None, final_state=None, output_checkpoints=False, workspace=None, "
        "stream=None)\n--\n\n"
        "Gated linear recurrence h_t = a_t h_{t-1} + u_t over whole sequences (C ABI glr_scan_fwd).\n\n"
        "x, g and in_gate [B, T, D]: log a = g, or -exp(A_log) softplus(g + dt_bias) with A_log; u = s sigmoid(in_gate) x\n"
        "with s = sqrt(1 - a^2) under normalize.  g is fp32 or x's type; states are [N, D] fp32.  Packed sequences:\n"
        "cu_seqlens (int32, B = 1).  Returns (o in x's type, final_state or None), and with output_checkpoints the\n"
        "[B, ceil(T / 64), D] fp32 states that glr_scan_bwd takes."),
    GDN_METHOD(glr_scan_bwd,
        "glr_scan_bwd(x, g, d_o, in_gate=None, A_log=None, dt_bias=None, normalize=False, initial_state=None, "
        "d_final_state=None, cu_seqlens=None, checkpoints=None, workspace=None, stream=None)\n--\n\n"
        "Gradients of <d_o, o> + <d_final_state, final_state> through glr_scan_fwd (C ABI glr_scan_bwd).\n\n"
        "checkpoints are the forward's; without them they are computed again.  Returns (dx, dg, din_gate,\n"
        "d_initial_state, dA_log, ddt_bias), with None where the input is None; token gradients in their tensor's type,\n"
        "the others fp32."),
    GDN_METHOD(glr_step,
        "glr_step(x, g, state, in_gate=None, A_log=None, dt_bias=None, normalize=False, state_out=None, o=None, "
        "stream=None)\n--\n\n"
        "One decode token of the gated linear recurrence for N sequences (C ABI glr_step); returns o [N, D].\n\n"
        "state [N, D] fp32 is updated in place, or kept when state_out is given, which then takes the new state."),
    GDN_METHOD(gdn_qk_norm_fwd,
        "gdn_qk_norm_fwd(q, k, q_weight=None, k_weight=None, norm='rms', eps=1e-6, cos=None, sin=None, positions=None, "
        "interleaved=False, q_out=None, k_out=None, stream=None)\n--\n\n"
        "Norm of every query and key head, with the position rotation in the same pass (C ABI gdn_qk_norm_fwd).\n\n"
        "q [..., H_q, d] and k [..., H_k, d] of the same leading shape ([B, T] or [N]).  norm is 'rms' (mean of squares) or\n"
        "'l2' (unit length); weights [d] fp32.  cos, sin [positions, rotary_dim / 2] fp32 turn the first rotary_dim\n"
        "channels, pairs (m, m + rotary_dim / 2) or (2m, 2m + 1) when interleaved; positions int32 of the leading shape, or\n"
        "None: the index along its last dimension.  Returns (q_out, k_out), contiguous."),
    GDN_METHOD(gdn_qk_norm_bwd,
        "gdn_qk_norm_bwd(q, k, d_q_out, d_k_out, q_weight=None, k_weight=None, norm='rms', eps=1e-6, cos=None, sin=None, "
        "positions=None, interleaved=False, workspace=None, stream=None)\n--\n\n"
        "Gradients through gdn_qk_norm_fwd (C ABI gdn_qk_norm_bwd): (dq, dk, dq_weight or None, dk_weight or None).\n\n"
        "d_q_out and d_k_out are contiguous, in q's type, as are dq and dk; the weights' gradients are fp32."),
    GDN_METHOD(gdn_short_conv_fwd,
        "gdn_short_conv_fwd(x, weight, bias=None, activation='silu', initial_state=None, output_final_state=False, "
        "cu_seqlens=None, y=None, final_state=None, stream=None)\n--\n\n"
        "Causal depthwise convolution of the last W tokens, with its activation (C ABI gdn_short_conv_fwd).\n\n"
        "x [B, T, D]; weight [D, W] (W = 2, 3, 4) and bias [D] fp32, the last tap on the current token; activation 'silu'\n"
        "or None.  States [N, W - 1, D] in x's type are the last W - 1 inputs, oldest first.  Returns (y, final_state or\n"
        "None)."),
    GDN_METHOD(gdn_short_conv_bwd,
        "gdn_short_conv_bwd(x, weight, d_y, bias=None, activation='silu', initial_state=None, d_final_state=None, "
        "cu_seqlens=None, workspace=None, stream=None)\n--\n\n"
        "Gradients of <d_y, y> + <d_final_state, final_state> through gdn_short_conv_fwd (C ABI gdn_short_conv_bwd).\n\n"
        "Returns (dx, dweight, dbias, d_initial_state), the last two None where their input is None; dx and\n"
        "d_initial_state in x's type, the others fp32."),
    GDN_METHOD(gdn_short_conv_step,
        "gdn_short_conv_step(x, state, weight, bias=None, activation='silu', state_out=None, y=None, stream=None)\n--\n\n"
        "One decode token of the short convolution for N sequences (C ABI gdn_short_conv_step); returns y [N, D].\n\n"
        "state [N, W - 1, D] in x's type moves up by the token in place, or is kept when state_out is given."),
    GDN_METHOD(lin_chunk_fwd,
        "lin_chunk_fwd(q, k, v, g, scale=None, initial_state=None, output_final_state=False, cu_seqlens=None, algo='auto', o=None, "
        "final_state=None, workspace=None, stream=None)\n--\n\n"
        "Linear attention with a decay for each head, S_t = exp(g_t) S_{t-1} + k_t v_t^T, o_t = scale S_t^T q_t, over whole\n"
        "sequences (C ABI lin_chunk_fwd).\n\n"
        "q, k [B, T, H_k, d_k] and v [B, T, H, d_v] in bf16 or fp32, H a multiple of H_k; g fp32, log decays [B, T, H] or [H];\n"
        "states [N, H, d_k, d_v] fp32; scale d_k ** -0.5.  Packed sequences: cu_seqlens (int32, B = 1).  Returns (o in v's type,\n"
        "final_state or None)."),
    GDN_METHOD(lin_chunk_bwd,
        "lin_chunk_bwd(q, k, v, g, d_o, scale=None, initial_state=None, d_final_state=None, cu_seqlens=None, algo='auto', "
        "workspace=None, stream=None)\n--\n\n"
        "Gradients of <d_o, o> + <d_final_state, final_state> through lin_chunk_fwd (C ABI lin_chunk_bwd).\n\n"
        "Returns (dq, dk, dv, dg, d_initial_state or None); token gradients in their tensor's type, dg (of g's shape) and\n"
        "d_initial_state fp32.  A key head's dq and dk sum those of its value heads."),
    GDN_METHOD(lin_recurrent_step,
        "lin_recurrent_step(q, k, v, g, state, scale=None, state_out=None, o=None, stream=None)\n--\n\n"
        "One decode token of linear attention for N sequences (C ABI lin_recurrent_step); returns o [N, H, d_v].\n\n"
        "q, k [N, H_k, d_k], v [N, H, d_v], g [N, H] or [H].  state [N, H, d_k, d_v] fp32 is updated in place, or kept when\n"
        "state_out is given, which then takes the new state."),
    GDN_METHOD(paged_append,
        "paged_append(k, v, k_cache, v_cache, block_table, lengths, q=None, cu_seqlens=None, cos=None, sin=None, interleaved=False, "
        "q_out=None, stream=None)\n--\n\n"
        "Write new tokens' keys and values into a paged cache, keys (and q) turned by their position on the way (C ABI\n"
        "paged_append).\n\n"
        "k, v [n, H_k, d], q [n, H_q, d]; k_cache, v_cache [n_pages, page_size, H_k, d] at any strides with contiguous channels;\n"
        "block_table [N, max_pages] and lengths [N] int32, the lengths with the new tokens.  One token for each sequence, or\n"
        "cu_seqlens [N + 1].  cos, sin [positions, rotary_dim / 2] fp32, pairs as in gdn_qk_norm_fwd.  Returns the turned q,\n"
        "contiguous, or None."),
    GDN_METHOD(paged_attn_step,
        "paged_attn_step(q, k_cache, v_cache, block_table, lengths, scale=None, o=None, output_lse=False, workspace=None, "
        "stream=None)\n--\n\n"
        "Softmax attention of one new token for each sequence over a paged cache (C ABI paged_attn_step); returns o [N, H_q, d],\n"
        "and with output_lse the log of the softmax's sum [N, H_q] fp32.\n\n"
        "q [N, H_q, d], H_q a multiple of H_k; the cache as in paged_append; scale d ** -0.5.  A sequence of length 0 has o = 0\n"
        "and lse = -inf.  Work is divided by the table's width: cut it to the longest sequence, block_table[:, :pages]."),
    GDN_METHOD(spacing, "spacing(t, heads=False)\n--\n\nThe strides that the entries pass on for a strided tensor."),
    {"init", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(py_init)), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_native", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__native() { return PyModule_Create(&module); }
