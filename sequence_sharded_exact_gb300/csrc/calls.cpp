// calls.cpp -- the Python side of the operators around a key/value cache, compiled: the argument checks, the outputs'
// and workspaces' allocation and the call into libringattn for what a serving step calls over and over.
//
// Each function does what its namesake in binding.py does, for arguments that pass all of that one's checks, on the
// current stream; for any others, and where the library refuses the call, it returns None having enqueued nothing, and
// binding.py, which then runs, names the reason.  What it saves is the host's time per call, which is all the time of a small
// one: the attention of five drafted tokens over a short cache takes 9 us on the GPU and took 24 us of checks,
// allocations and argument conversion.
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/autograd/python_variable.h>

#include "../../include/ringattn.h"

namespace {

decltype(&ring_attn_qk_norm_rope) norm_rope = nullptr;
decltype(&ring_attn_qk_norm_rope_bwd) norm_rope_bwd = nullptr;
decltype(&ring_attn_qk_norm_rope_bwd_workspace_size) norm_rope_bwd_workspace = nullptr;
decltype(&ring_attn_cache_write) write_cache = nullptr;
decltype(&ring_attn_cache_read) read_cache = nullptr;
decltype(&ring_attn_tree_fwd) tree = nullptr;
decltype(&ring_attn_tree_fwd_workspace_size) tree_workspace = nullptr;
decltype(&ring_attn_qk_rope_axes) rope_axes = nullptr;
decltype(&ring_attn_tree_window_fwd) tree_window = nullptr;
decltype(&ring_attn_window_fwd) window_forward = nullptr;
decltype(&ring_attn_window_fwd_workspace_size) window_forward_workspace = nullptr;
decltype(&ring_attn_window_bwd) window_backward = nullptr;
decltype(&ring_attn_window_bwd_workspace_size) window_backward_workspace = nullptr;

using at::ScalarType;
using at::Tensor;
using Sizes = std::initializer_list<int64_t>;

struct Misfit {};  // the Python path takes over

// A plain tensor (no subclass that dispatches to Python).
const Tensor& tensor(PyObject* o)
{
    if (!THPVariable_Check(o)) throw Misfit{};
    const Tensor& t = THPVariable_Unpack(o);
    if (t.unsafeGetTensorImpl()->is_python_dispatch() || t.layout() != at::kStrided) throw Misfit{};
    return t;
}

struct Call {
    at::Device device;
    c10::cuda::CUDAGuard guard;
    explicit Call(const Tensor& t) : device(t.device()), guard(check(t)) {}
    static at::Device check(const Tensor& t)
    {
        if (!t.is_cuda()) throw Misfit{};
        return t.device();
    }
    void* stream() const { return c10::cuda::getCurrentCUDAStream(device.index()).stream(); }

    bool fits(const Tensor& t, at::IntArrayRef shape, ScalarType dtype) const
    {
        return t.scalar_type() == dtype && t.device() == device && t.sizes() == shape;
    }
    // A contiguous tensor of this device, shape and dtype.
    void* dense(PyObject* o, at::IntArrayRef shape, ScalarType dtype) const
    {
        const Tensor& t = tensor(o);
        if (!fits(t, shape, dtype) || !t.is_contiguous()) throw Misfit{};
        return t.data_ptr();
    }
    void* optional(PyObject* o, at::IntArrayRef shape, ScalarType dtype) const { return o == Py_None ? nullptr : dense(o, shape, dtype); }
    // The caller's output, checked, or a new one.
    Tensor output(PyObject* o, at::IntArrayRef shape, ScalarType dtype) const
    {
        if (o == Py_None) return at::empty(shape, at::TensorOptions().dtype(dtype).device(device));
        dense(o, shape, dtype);
        return THPVariable_Unpack(o);
    }
    Tensor workspace(PyObject* o, int64_t need) const
    {
        if (o == Py_None) return at::empty({need}, at::TensorOptions().dtype(at::kByte).device(device));
        const Tensor& t = tensor(o);
        if (t.scalar_type() != at::kByte || t.device() != device || !t.is_contiguous() || t.numel() < need) throw Misfit{};
        return t;
    }
    // A tensor read by strides (batch, head, row), null if it is contiguous; the library checks them.
    struct Rows {
        const void* p;
        long long strides[3];
        bool dense;
        const long long* given() const { return dense ? nullptr : strides; }
    };
    Rows rows(const Tensor& t, at::IntArrayRef shape, ScalarType dtype) const
    {
        if (!fits(t, shape, dtype)) throw Misfit{};
        Rows r{t.data_ptr(), {0, 0, 0}, t.is_contiguous()};
        if (!r.dense) {
            if (t.stride(3) != 1) throw Misfit{};
            for (int i = 0; i < 3; ++i) r.strides[i] = t.stride(i);
        }
        return r;
    }
};

int small(int64_t v)
{
    if (v < 0 || v > 0x7fffffff) throw Misfit{};
    return (int)v;
}

int code_of(ScalarType t)
{
    if (t == at::kFloat) return RA_F32;
    if (t == at::kBFloat16) return RA_BF16;
    throw Misfit{};
}

int whole_number(PyObject* o)
{
    if (!PyLong_CheckExact(o)) throw Misfit{};
    int overflow = 0;
    const long long v = PyLong_AsLongLongAndOverflow(o, &overflow);
    if (overflow || v < INT_MIN || v > INT_MAX) throw Misfit{};
    return (int)v;
}

double real_number(PyObject* o)
{
    if (!PyFloat_CheckExact(o)) throw Misfit{};
    return PyFloat_AS_DOUBLE(o);
}

int layout_code(PyObject* o)
{
    if (!PyUnicode_CheckExact(o)) throw Misfit{};
    if (PyUnicode_CompareWithASCIIString(o, "contiguous") == 0) return 0;
    if (PyUnicode_CompareWithASCIIString(o, "zigzag") == 0) return 1;
    if (PyUnicode_CompareWithASCIIString(o, "striped") == 0) return 2;
    throw Misfit{};
}

void four(const Tensor& t)
{
    if (t.dim() != 4) throw Misfit{};
}

struct CacheArgs {
    void *k, *v, *ke, *ve;
    int cap, code;
    CacheArgs(const Call& c, PyObject* o, int64_t B, int64_t Hkv, int64_t d, ScalarType dtype)
    {
        if (!PyTuple_Check(o) || PyTuple_GET_SIZE(o) != 4) throw Misfit{};
        const Tensor& t = tensor(PyTuple_GET_ITEM(o, 0));
        four(t);
        cap = small(t.size(2));
        const ScalarType kind = t.scalar_type();
        const bool quant = kind == at::kFloat8_e4m3fn;
        if (!quant && kind != dtype) throw Misfit{};
        code = quant ? RA_E4M3 : code_of(kind);
        const Sizes shape = {B, Hkv, cap, d}, rows = {B, Hkv, cap};
        k = c.dense(PyTuple_GET_ITEM(o, 0), shape, kind);
        v = c.dense(PyTuple_GET_ITEM(o, 1), shape, kind);
        ke = quant ? c.dense(PyTuple_GET_ITEM(o, 2), rows, at::kByte) : nullptr;
        ve = quant ? c.dense(PyTuple_GET_ITEM(o, 3), rows, at::kByte) : nullptr;
    }
};

void accept(ra_status st)
{
    if (st != RA_OK) throw Misfit{};
}

PyObject* pair_of(Tensor a, Tensor b)
{
    PyObject* x = THPVariable_Wrap(std::move(a));
    PyObject* y = x ? THPVariable_Wrap(std::move(b)) : nullptr;
    PyObject* r = y ? PyTuple_Pack(2, x, y) : nullptr;
    Py_XDECREF(x);
    Py_XDECREF(y);
    return r;
}

// Runs f; None for whatever the Python path has to answer.
template <typename F>
PyObject* answer(Py_ssize_t given, Py_ssize_t expected, F f)
{
    if (given != expected) {
        PyErr_Format(PyExc_TypeError, "expected %zd arguments, not %zd", expected, given);
        return nullptr;
    }
    try {
        return f();
    } catch (const Misfit&) {
    } catch (const std::exception&) {
    }
    Py_RETURN_NONE;
}

// q, cache, lens, mask, ntok, out_dtype, out, lse, workspace, and through a window: window, sinks, positions
PyObject* attend(PyObject* const* a, Py_ssize_t n, Py_ssize_t expected)
{
    return answer(n, expected, [&]() -> PyObject* {
        const Tensor& q = tensor(a[0]);
        four(q);
        const Call c(q);
        const int64_t B = q.size(0), H = q.size(1), T = q.size(2), d = q.size(3);
        const ScalarType dt = q.scalar_type();
        const int code = code_of(dt);
        const void* qp = c.dense(a[0], {B, H, T, d}, dt);
        if (!PyTuple_Check(a[1]) || PyTuple_GET_SIZE(a[1]) != 4) throw Misfit{};
        const Tensor& k = tensor(PyTuple_GET_ITEM(a[1], 0));
        four(k);
        const int64_t Hkv = k.size(1);
        const CacheArgs cache(c, a[1], B, Hkv, d, dt);
        ScalarType odt = dt;
        if (a[5] != Py_None) {
            if (!THPDtype_Check(a[5])) throw Misfit{};
            odt = reinterpret_cast<THPDtype*>(a[5])->scalar_type;
            if (odt != dt && odt != at::kFloat) throw Misfit{};
        }
        const auto* lens = static_cast<const int*>(c.dense(a[2], {B}, at::kInt));
        const auto* ntok = static_cast<const int*>(c.optional(a[4], {B}, at::kInt));
        const unsigned char* mask = nullptr;
        int batched = 0;
        if (a[3] != Py_None) {
            const Tensor& m = tensor(a[3]);
            batched = m.dim() == 3;
            mask = static_cast<const unsigned char*>(batched ? c.dense(a[3], {B, T, T}, at::kBool) : c.dense(a[3], {T, T}, at::kBool));
        }
        const int b = small(B), h = small(H), hk = small(Hkv), t = small(T), dd = small(d);
        const size_t need = tree_workspace(b, h, hk, t, dd, cache.cap, code, cache.code);
        if (need == 0) throw Misfit{};
        Tensor out = c.output(a[6], {B, H, T, d}, odt), lse = c.output(a[7], {B, H, T}, at::kFloat);
        const Tensor ws = c.workspace(a[8], (int64_t)need);
        if (expected == 9) {
            accept(tree(qp, cache.k, cache.v, cache.ke, cache.ve, lens, ntok, mask, batched, out.data_ptr(), static_cast<float*>(lse.data_ptr()),
                        ws.data_ptr(), (size_t)ws.numel(), b, h, hk, t, dd, cache.cap, code, cache.code, code_of(odt), c.stream()));
        } else {
            const auto* pos = static_cast<const int*>(c.optional(a[11], {B, T}, at::kInt));
            accept(tree_window(qp, cache.k, cache.v, cache.ke, cache.ve, lens, ntok, mask, batched, pos, out.data_ptr(),
                               static_cast<float*>(lse.data_ptr()), ws.data_ptr(), (size_t)ws.numel(), b, h, hk, t, dd, cache.cap,
                               whole_number(a[9]), whole_number(a[10]), code, cache.code, code_of(odt), c.stream()));
        }
        return pair_of(std::move(out), std::move(lse));
    });
}

PyObject* py_tree_fwd(PyObject*, PyObject* const* a, Py_ssize_t n) { return attend(a, n, 9); }
PyObject* py_tree_window_fwd(PyObject*, PyObject* const* a, Py_ssize_t n) { return attend(a, n, 12); }

// cache, k, v, lens, ntok
PyObject* py_cache_write(PyObject*, PyObject* const* a, Py_ssize_t n)
{
    return answer(n, 5, [&]() -> PyObject* {
        const Tensor &k = tensor(a[1]), &v = tensor(a[2]);
        four(k);
        const Call c(k);
        const int64_t B = k.size(0), Hkv = k.size(1), T = k.size(2), d = k.size(3);
        const ScalarType dt = k.scalar_type();
        const int code = code_of(dt);
        const Call::Rows kr = c.rows(k, {B, Hkv, T, d}, dt), vr = c.rows(v, {B, Hkv, T, d}, dt);
        const CacheArgs cache(c, a[0], B, Hkv, d, dt);
        const auto* lens = static_cast<const int*>(c.optional(a[3], {B}, at::kInt));
        const auto* ntok = static_cast<const int*>(c.optional(a[4], {B}, at::kInt));
        accept(write_cache(kr.p, kr.given(), vr.p, vr.given(), cache.k, cache.v, cache.ke, cache.ve, lens, ntok, small(B), small(Hkv), small(T),
                           small(d), cache.cap, code, cache.code, c.stream()));
        Py_RETURN_TRUE;
    });
}

// cache, rows, row0, dtype, k, v
PyObject* py_cache_read(PyObject*, PyObject* const* a, Py_ssize_t n)
{
    return answer(n, 6, [&]() -> PyObject* {
        if (!PyTuple_Check(a[0]) || PyTuple_GET_SIZE(a[0]) != 4 || !THPDtype_Check(a[3])) throw Misfit{};
        const Tensor& t = tensor(PyTuple_GET_ITEM(a[0], 0));
        four(t);
        const Call c(t);
        const int64_t B = t.size(0), Hkv = t.size(1), d = t.size(3);
        const ScalarType dt = reinterpret_cast<THPDtype*>(a[3])->scalar_type;
        const int code = code_of(dt), rows = whole_number(a[1]), row0 = whole_number(a[2]);
        const CacheArgs cache(c, a[0], B, Hkv, d, dt);
        if (rows < 1 || row0 < 0 || row0 > cache.cap || rows > cache.cap - row0) throw Misfit{};
        Tensor k = c.output(a[4], {B, Hkv, rows, d}, dt), v = c.output(a[5], {B, Hkv, rows, d}, dt);
        accept(read_cache(cache.k, cache.v, cache.ke, cache.ve, k.data_ptr(), v.data_ptr(), small(B), small(Hkv), row0, rows, small(d),
                          cache.cap, code, cache.code, c.stream()));
        return pair_of(std::move(k), std::move(v));
    });
}

// What the forward and the backward share: q, k, wq, wk, then n_shards, layout, base, eps, shard, positions.
struct NormRopeArgs {
    int64_t B, H, Hkv, rows, d;
    ScalarType dt;
    int code, L, n, which, layout;
    double base, eps;
    const int* positions;
    Call::Rows q, k;
    const float *wq, *wk;
    NormRopeArgs(const Call& c, PyObject* const* a, PyObject* const* s)
    {
        const Tensor &tq = tensor(a[0]), &tk = tensor(a[1]);
        four(tk);
        B = tq.size(0), H = tq.size(1), rows = tq.size(2), d = tq.size(3), Hkv = tk.size(1);
        dt = tq.scalar_type();
        code = code_of(dt);
        q = c.rows(tq, {B, H, rows, d}, dt);
        k = c.rows(tk, {B, Hkv, rows, d}, dt);
        wq = static_cast<const float*>(c.dense(a[2], {d}, at::kFloat));
        wk = static_cast<const float*>(c.dense(a[3], {d}, at::kFloat));
        n = whole_number(s[0]);
        layout = layout_code(s[1]);
        base = real_number(s[2]);
        eps = real_number(s[3]);
        positions = static_cast<const int*>(c.optional(s[5], {B, rows}, at::kInt));
        which = -1;
        int64_t all = rows;
        if (positions) {
            if (s[4] != Py_None || n != 1) throw Misfit{};
            layout = 0;
        } else if (s[4] != Py_None) {
            which = whole_number(s[4]);
            if (which < 0 || which >= n) throw Misfit{};
            all = rows * n;
        }
        L = small(all);
    }
};

// q, k, wq, wk, n_shards, layout, base, eps, shard, positions, q_out, k_out
PyObject* py_norm_rope(PyObject*, PyObject* const* a, Py_ssize_t n)
{
    return answer(n, 12, [&]() -> PyObject* {
        const Tensor& q = tensor(a[0]);
        four(q);
        const Call c(q);
        const NormRopeArgs s(c, a, a + 4);
        Tensor qo = c.output(a[10], {s.B, s.H, s.rows, s.d}, s.dt), ko = c.output(a[11], {s.B, s.Hkv, s.rows, s.d}, s.dt);
        accept(norm_rope(s.q.p, s.q.given(), s.k.p, s.k.given(), s.wq, s.wk, qo.data_ptr(), ko.data_ptr(), small(s.B), small(s.H), small(s.Hkv),
                         s.L, small(s.d), s.n, s.which, s.layout, s.code, s.base, s.eps, s.positions, c.stream()));
        return pair_of(std::move(qo), std::move(ko));
    });
}

// q, k, wq, wk, dq_out, dk_out, n_shards, layout, base, eps, shard, positions, dq, dk, workspace
PyObject* py_norm_rope_bwd(PyObject*, PyObject* const* a, Py_ssize_t n)
{
    return answer(n, 15, [&]() -> PyObject* {
        const Tensor& q = tensor(a[0]);
        four(q);
        const Call c(q);
        const NormRopeArgs s(c, a, a + 6);
        const int64_t qs[4] = {s.B, s.H, s.rows, s.d}, ks[4] = {s.B, s.Hkv, s.rows, s.d};
        const void *gq = c.dense(a[4], qs, s.dt), *gk = c.dense(a[5], ks, s.dt);
        Tensor dq = c.output(a[12], qs, s.dt), dk = c.output(a[13], ks, s.dt);
        Tensor dwq = c.output(Py_None, {s.d}, at::kFloat), dwk = c.output(Py_None, {s.d}, at::kFloat);
        const Tensor ws = c.workspace(a[14], (int64_t)norm_rope_bwd_workspace(small(s.d)));
        accept(norm_rope_bwd(s.q.p, s.q.given(), s.k.p, s.k.given(), s.wq, s.wk, gq, gk, dq.data_ptr(), dk.data_ptr(),
                             static_cast<float*>(dwq.data_ptr()), static_cast<float*>(dwk.data_ptr()), ws.data_ptr(), (size_t)ws.numel(),
                             small(s.B), small(s.H), small(s.Hkv), s.L, small(s.d), s.n, s.which, s.layout, s.code, s.base, s.eps, s.positions,
                             c.stream()));
        PyObject* t[4] = {THPVariable_Wrap(std::move(dq)), THPVariable_Wrap(std::move(dk)), THPVariable_Wrap(std::move(dwq)),
                          THPVariable_Wrap(std::move(dwk))};
        PyObject* r = t[0] && t[1] && t[2] && t[3] ? PyTuple_Pack(4, t[0], t[1], t[2], t[3]) : nullptr;
        for (PyObject* o : t) Py_XDECREF(o);
        return r;
    });
}

// q, k, positions, sections, wq, wk, base, eps, spectrum, q_out, k_out
PyObject* py_rope_axes(PyObject*, PyObject* const* a, Py_ssize_t n)
{
    return answer(n, 11, [&]() -> PyObject* {
        const Tensor &q = tensor(a[0]), &k = tensor(a[1]);
        four(q);
        four(k);
        const Call c(q);
        const int64_t B = q.size(0), H = q.size(1), rows = q.size(2), d = q.size(3), Hkv = k.size(1);
        const ScalarType dt = q.scalar_type();
        const int code = code_of(dt);
        const Call::Rows qr = c.rows(q, {B, H, rows, d}, dt), kr = c.rows(k, {B, Hkv, rows, d}, dt);
        if (!PyTuple_CheckExact(a[3])) throw Misfit{};
        const Py_ssize_t axes = PyTuple_GET_SIZE(a[3]);
        if (axes < 1 || axes > 4) throw Misfit{};
        int sections[4];
        for (Py_ssize_t i = 0; i < axes; ++i) sections[i] = whole_number(PyTuple_GET_ITEM(a[3], i));
        const auto* pos = static_cast<const int*>(c.dense(a[2], {axes, B, rows}, at::kInt));
        const auto* wq = static_cast<const float*>(c.optional(a[4], {d}, at::kFloat));
        const auto* wk = static_cast<const float*>(c.optional(a[5], {d}, at::kFloat));
        if ((wq == nullptr) != (wk == nullptr)) throw Misfit{};
        const double base = real_number(a[6]), eps = real_number(a[7]);
        if (!PyUnicode_CheckExact(a[8])) throw Misfit{};
        const bool whole = PyUnicode_CompareWithASCIIString(a[8], "whole") == 0;
        if (!whole && PyUnicode_CompareWithASCIIString(a[8], "axis") != 0) throw Misfit{};
        Tensor qo = c.output(a[9], {B, H, rows, d}, dt), ko = c.output(a[10], {B, Hkv, rows, d}, dt);
        accept(rope_axes(qr.p, qr.given(), kr.p, kr.given(), wq, wk, qo.data_ptr(), ko.data_ptr(), small(B), small(H), small(Hkv), small(rows),
                         small(d), (int)axes, sections, whole ? RA_SPECTRUM_WHOLE : RA_SPECTRUM_AXIS, code, base, eps, pos, c.stream()));
        return pair_of(std::move(qo), std::move(ko));
    });
}

// What window_fwd and window_bwd share: q, k, v, and n_shards, window, sinks, causal, layout.
struct WindowCall {
    int B, H, Hkv, L, d, n, window, sinks, causal, layout, code;
    ScalarType dt;
    const void *q, *k, *v;
    WindowCall(const Call& c, PyObject* const* a, PyObject* const* how)
    {
        const Tensor &tq = tensor(a[0]), &tk = tensor(a[1]);
        four(tk);
        B = small(tq.size(0)), H = small(tq.size(1)), L = small(tq.size(2)), d = small(tq.size(3)), Hkv = small(tk.size(1));
        dt = tq.scalar_type();
        code = code_of(dt);
        q = c.dense(a[0], {B, H, L, d}, dt);
        k = c.dense(a[1], {B, Hkv, L, d}, dt);
        v = c.dense(a[2], {B, Hkv, L, d}, dt);
        n = whole_number(how[0]);
        window = whole_number(how[1]);
        sinks = whole_number(how[2]);
        if (!PyBool_Check(how[3])) throw Misfit{};
        causal = how[3] == Py_True;
        layout = layout_code(how[4]);
    }
};

// q, k, v, n_shards, window, sinks, causal, layout, out_dtype, out, lse, workspace
PyObject* py_window_fwd(PyObject*, PyObject* const* a, Py_ssize_t n)
{
    return answer(n, 12, [&]() -> PyObject* {
        const Tensor& q = tensor(a[0]);
        four(q);
        const Call c(q);
        const WindowCall w(c, a, a + 3);
        ScalarType odt = w.dt;
        if (a[8] != Py_None) {
            if (!THPDtype_Check(a[8])) throw Misfit{};
            odt = reinterpret_cast<THPDtype*>(a[8])->scalar_type;
            if (odt != w.dt && odt != at::kFloat) throw Misfit{};
        }
        Tensor out = c.output(a[9], {w.B, w.H, w.L, w.d}, odt), lse = c.output(a[10], {w.B, w.H, w.L}, at::kFloat);
        const Tensor ws = c.workspace(a[11], (int64_t)window_forward_workspace(w.B, w.H, w.Hkv, w.L, w.d, w.n, w.layout, w.code));
        accept(window_forward(w.q, w.k, w.v, out.data_ptr(), static_cast<float*>(lse.data_ptr()), ws.data_ptr(), (size_t)ws.numel(), w.B, w.H,
                              w.Hkv, w.L, w.d, w.n, w.window, w.sinks, w.causal, w.layout, w.code, code_of(odt), c.stream()));
        return pair_of(std::move(out), std::move(lse));
    });
}

// q, k, v, out, lse, dout, n_shards, window, sinks, causal, layout, grad_dtype, dq, dk, dv, workspace
PyObject* py_window_bwd(PyObject*, PyObject* const* a, Py_ssize_t n)
{
    return answer(n, 16, [&]() -> PyObject* {
        const Tensor& q = tensor(a[0]);
        four(q);
        const Call c(q);
        const WindowCall w(c, a, a + 6);
        const int64_t qs[4] = {w.B, w.H, w.L, w.d}, ks[4] = {w.B, w.Hkv, w.L, w.d};
        const ScalarType odt = tensor(a[3]).scalar_type();
        if (odt != w.dt && odt != at::kFloat) throw Misfit{};
        const void *out = c.dense(a[3], qs, odt), *dout = c.dense(a[5], qs, w.dt);
        const auto* lse = static_cast<const float*>(c.dense(a[4], {w.B, w.H, w.L}, at::kFloat));
        if (!THPDtype_Check(a[11])) throw Misfit{};
        const ScalarType gdt = reinterpret_cast<THPDtype*>(a[11])->scalar_type;
        const int grad = code_of(gdt);
        Tensor dq = c.output(a[12], qs, gdt), dk = c.output(a[13], ks, gdt), dv = c.output(a[14], ks, gdt);
        const size_t need = window_backward_workspace(w.B, w.H, w.Hkv, w.L, w.d, w.n, w.window, w.sinks, w.causal, w.layout, w.code);
        if (need == 0) throw Misfit{};
        const Tensor ws = c.workspace(a[15], (int64_t)need);
        accept(window_backward(w.q, w.k, w.v, out, lse, dout, dq.data_ptr(), dk.data_ptr(), dv.data_ptr(), ws.data_ptr(), (size_t)ws.numel(), w.B,
                               w.H, w.Hkv, w.L, w.d, w.n, w.window, w.sinks, w.causal, w.layout, w.code, code_of(odt), grad, c.stream()));
        PyObject* t[3] = {THPVariable_Wrap(std::move(dq)), THPVariable_Wrap(std::move(dk)), THPVariable_Wrap(std::move(dv))};
        PyObject* r = t[0] && t[1] && t[2] ? PyTuple_Pack(3, t[0], t[1], t[2]) : nullptr;
        for (PyObject* o : t) Py_XDECREF(o);
        return r;
    });
}

// bind(address, ...): the library's functions, in the order of the pointers above.
PyObject* py_bind(PyObject*, PyObject* const* a, Py_ssize_t n)
{
    void** to[] = {reinterpret_cast<void**>(&norm_rope), reinterpret_cast<void**>(&norm_rope_bwd),
                   reinterpret_cast<void**>(&norm_rope_bwd_workspace), reinterpret_cast<void**>(&write_cache),
                   reinterpret_cast<void**>(&read_cache), reinterpret_cast<void**>(&tree), reinterpret_cast<void**>(&tree_workspace),
                   reinterpret_cast<void**>(&rope_axes), reinterpret_cast<void**>(&tree_window),
                   reinterpret_cast<void**>(&window_forward), reinterpret_cast<void**>(&window_forward_workspace),
                   reinterpret_cast<void**>(&window_backward), reinterpret_cast<void**>(&window_backward_workspace)};
    if (n != (Py_ssize_t)(sizeof(to) / sizeof(to[0]))) {
        PyErr_SetString(PyExc_TypeError, "one address for each function");
        return nullptr;
    }
    for (Py_ssize_t i = 0; i < n; ++i) {
        void* p = PyLong_AsVoidPtr(a[i]);
        if (!p) {
            if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, "null address");
            return nullptr;
        }
        *to[i] = p;
    }
    Py_RETURN_NONE;
}

#define FAST(f) reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(f)), METH_FASTCALL
PyMethodDef methods[] = {{"bind", FAST(py_bind), nullptr},
                         {"tree_fwd", FAST(py_tree_fwd), nullptr},
                         {"tree_window_fwd", FAST(py_tree_window_fwd), nullptr},
                         {"cache_write", FAST(py_cache_write), nullptr},
                         {"cache_read", FAST(py_cache_read), nullptr},
                         {"qk_norm_rope", FAST(py_norm_rope), nullptr},
                         {"qk_norm_rope_bwd", FAST(py_norm_rope_bwd), nullptr},
                         {"qk_rope_axes", FAST(py_rope_axes), nullptr},
                         {"window_fwd", FAST(py_window_fwd), nullptr},
                         {"window_bwd", FAST(py_window_bwd), nullptr},
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_calls", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__calls() { return PyModule_Create(&module); }
