// calls.cpp -- the binding's calls of the linear, mixture-of-experts and
// attention layers, marshalled in C++ (the Python module quantized_weight_prefill_amd._calls).
//
// At decode sizes these kernels take a few microseconds, and checking and
// marshalling their arguments in Python took longer than that (13.9 us a call
// of the one-token linear layer, 8.2 with the checks pared down, against 6 us
// of GPU time).  Each function here takes the common call -- tensors of the
// right kind on the current device, its current stream, no caller's
// workspace -- and returns its result; for any other call it returns None
// before doing anything, and the Python code next to it checks the arguments
// one by one, names what is wrong, or makes the call itself.  A status from
// the library comes back as an int.  Nothing is computed here.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/core/LegacyTypeDispatch.h>
#include <ATen/ops/as_strided.h>
#include <ATen/ops/empty.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cmath>
#include <cstdint>
#include <exception>

#include "qgemm.h"

namespace {

PyObject *g_device = nullptr, *g_stream = nullptr;  // torch's current device index, and its current stream's pointer

struct Bad {};  // not the common call

long long integer(PyObject *o)
{
    const long long v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred()) {
        PyErr_Clear();
        throw Bad{};
    }
    return v;
}

const at::Tensor &tensor(PyObject *o)
{
    if (!THPVariable_Check(o)) throw Bad{};
    return THPVariable_Unpack(o);
}

// The tensor's data when it is contiguous on GPU `index`; None is null.
void *data(PyObject *o, int index)
{
    if (o == Py_None) return nullptr;
    const at::Tensor &t = tensor(o);
    if (!t.is_cuda() || t.get_device() != index || !t.is_contiguous()) throw Bad{};
    return t.data_ptr();
}

// ... and of this type and shape.
void *data(PyObject *o, int index, at::ScalarType type, at::IntArrayRef shape)
{
    if (o == Py_None) return nullptr;
    const at::Tensor &t = tensor(o);
    if (t.scalar_type() != type || t.sizes() != shape) throw Bad{};
    return data(o, index);
}

int half_type(const at::Tensor &t)
{
    if (t.scalar_type() == at::kHalf) return QGEMM_F16;
    if (t.scalar_type() == at::kBFloat16) return QGEMM_BF16;
    throw Bad{};
}

// The current stream of GPU `index`, which must be the current device.
void *stream_of(int index)
{
    PyObject *d = PyObject_CallNoArgs(g_device);
    if (!d) throw Bad{};
    const long current = PyLong_AsLong(d);
    Py_DECREF(d);
    if (current != index) throw Bad{};
    PyObject *i = PyLong_FromLong(index);
    PyObject *s = i ? PyObject_CallOneArg(g_stream, i) : nullptr;
    Py_XDECREF(i);
    if (!s) throw Bad{};
    void *p = PyLong_AsVoidPtr(s);
    Py_DECREF(s);
    return p;
}

size_t packed(int fmt, int64_t N, int64_t K, int64_t group, int has_zp)
{
    size_t n = 0;
    if (fmt == QGEMM_FMT_Q4K) n = qgemm_q4k_packed_bytes(N, K);
    else if (fmt == QGEMM_FMT_Q6K) n = qgemm_q6k_packed_bytes(N, K);
    else if (fmt == QGEMM_FMT_W4A16 && group != 0) n = qgemm_w4a16_packed_bytes(N, K, group, has_zp);
    if (n == 0) throw Bad{};
    return n;
}

// Bytes of E weights of `each`, where they can be counted at all: a product
// that wraps around would pass for a small one.
size_t of_experts(int64_t E, size_t each)
{
    if (each > SIZE_MAX / (size_t)E) throw Bad{};
    return (size_t)E * each;
}

void holds(PyObject *w, size_t need)
{
    if (tensor(w).nbytes() < need) throw Bad{};
}

// The caller's `out` (`bytes` from `y`) shares memory with an input, of n
// bytes: not a call for here.
void apart(const void *y, size_t bytes, const void *p, size_t n)
{
    const uintptr_t a = (uintptr_t)y, b = (uintptr_t)p;
    if (p && a < b + n && b < a + bytes) throw Bad{};
}

// The body of a function: its result, None for an uncommon call, or the
// library's status when that is not QGEMM_OK.
template <class F>
PyObject *guarded(F body)
{
    const at::AutoDispatchBelowADInplaceOrView below;  // nothing here is differentiable
    try {
        return body();
    } catch (const Bad &) {
        PyErr_Clear();
        Py_RETURN_NONE;
    } catch (...) {  // torch's own, an allocation that fails among them
        torch::translate_exception_to_python(std::current_exception());
        return nullptr;
    }
}

PyObject *wrap_or_status(int st, const at::Tensor &t) { return st == QGEMM_OK ? THPVariable_Wrap(t) : PyLong_FromLong(st); }

// linear(format, layout, x, wp, M, N, K, bias, residual, act, gated, group,
// has_zp, rung, out, out_layout)
PyObject *linear(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    return guarded([&]() -> PyObject * {
        if (n != 16) throw Bad{};
        const at::Tensor &x = tensor(a[2]);
        const int index = x.get_device(), dtype = half_type(x), fmt = (int)integer(a[0]), xl = (int)integer(a[1]);
        const int64_t M = integer(a[4]), N = integer(a[5]), K = integer(a[6]), group = integer(a[11]);
        const int act = (int)integer(a[9]), gated = PyObject_IsTrue(a[10]), zp = PyObject_IsTrue(a[12]);
        const int rung = (int)integer(a[13]), yl = (int)integer(a[15]);
        if (M < 1 || N < 1 || N > INT32_MAX / 2 || gated < 0 || zp < 0) throw Bad{};
        const int64_t nt = gated ? 2 * N : N;
        const at::ScalarType type = x.scalar_type();
        const void *xp = data(a[2], index), *wp = data(a[3], index);
        const void *bp = data(a[7], index, type, {nt}), *rp = data(a[8], index, type, {M, N});
        const size_t wb = packed(fmt, nt, K, group, zp);
        holds(a[3], wb);
        const int64_t flat = (int64_t)(qgemm_xf_bytes(M, N) / 2);
        if (yl != QGEMM_X_ROW && (yl != QGEMM_X_FRAG || flat == 0)) throw Bad{};
        const int64_t rows[2] = {M, N}, frag[1] = {flat};
        const at::IntArrayRef shape = yl == QGEMM_X_ROW ? at::IntArrayRef(rows, 2) : at::IntArrayRef(frag, 1);
        void *yp = data(a[14], index, type, shape);
        if (yp) {
            const size_t yb = tensor(a[14]).nbytes();
            apart(yp, yb, xp, xl == QGEMM_X_FRAG ? qgemm_xf_bytes(M, K) : (size_t)(2 * M * K));
            apart(yp, yb, wp, wb);
            apart(yp, yb, bp, (size_t)(2 * nt));
            if (yl == QGEMM_X_FRAG || yp != rp) apart(yp, yb, rp, (size_t)(2 * M * N));
        }
        void *s = stream_of(index);
        const at::Tensor y = yp ? tensor(a[14]) : at::empty(shape, x.options());
        if (!yp) yp = y.data_ptr();
        const size_t need = qgemm_linear_workspace_bytes(fmt, rung, xl, M, N, K, gated, dtype);
        at::Tensor ws;
        if (need) ws = at::empty({(int64_t)need}, x.options().dtype(at::kByte));
        int st;
        Py_BEGIN_ALLOW_THREADS
        st = qgemm_linear(fmt, rung, xl, xp, wp, bp, rp, yp, yl, M, N, K, group, zp, act, gated, dtype,
                          need ? ws.data_ptr() : nullptr, need, s);
        Py_END_ALLOW_THREADS
        return wrap_or_status(st, y);
    });
}

PyObject *tuple_of(std::initializer_list<at::Tensor> ts)
{
    PyObject *t = PyTuple_New((Py_ssize_t)ts.size());
    if (!t) return nullptr;
    Py_ssize_t i = 0;
    for (const at::Tensor &v : ts) PyTuple_SET_ITEM(t, i++, THPVariable_Wrap(v));
    return t;
}

// moe_route(logits, top_k, score, renorm, scale)
PyObject *moe_route(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    return guarded([&]() -> PyObject * {
        if (n != 5) throw Bad{};
        const at::Tensor &l = tensor(a[0]);
        if (l.dim() != 2) throw Bad{};
        const int index = l.get_device(), lt = l.scalar_type() == at::kFloat ? QGEMM_F32 : half_type(l);
        const void *lp = data(a[0], index);
        const int64_t T = l.size(0), E = l.size(1), k = integer(a[1]);
        const int score = (int)integer(a[2]), renorm = PyObject_IsTrue(a[3]);
        const double scale = PyFloat_AsDouble(a[4]);
        if (T < 1 || k < 1 || k > E || k > 64 || renorm < 0 || (scale == -1.0 && PyErr_Occurred())) throw Bad{};
        void *s = stream_of(index);
        // one allocation for the three integer results, one for the weights
        const int64_t P = T * k;
        const at::Tensor buf = at::empty({2 * P + E + 1}, l.options().dtype(at::kInt));
        const at::Tensor w = at::empty({T, k}, l.options().dtype(at::kFloat));
        int *p = buf.data_ptr<int>();
        int st;
        Py_BEGIN_ALLOW_THREADS
        st = qgemm_moe_route(lp, lt, T, E, k, score, renorm, (float)scale, p, w.data_ptr<float>(), p + 2 * P, p + P, s);
        Py_END_ALLOW_THREADS
        if (st != QGEMM_OK) return PyLong_FromLong(st);
        return tuple_of({buf.as_strided({T, k}, {k, 1}, 0), w, buf.as_strided({E + 1}, {1}, 2 * P),
                         buf.as_strided({P}, {1}, P)});
    });
}

// moe_group(ids, E)
PyObject *moe_group(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    return guarded([&]() -> PyObject * {
        if (n != 2) throw Bad{};
        const at::Tensor &ids = tensor(a[0]);
        if (ids.dim() != 2 || ids.scalar_type() != at::kInt) throw Bad{};
        const int index = ids.get_device();
        const void *ip = data(a[0], index);
        const int64_t T = ids.size(0), k = ids.size(1), E = integer(a[1]);
        if (T < 1 || E < 1 || E > QGEMM_MOE_MAX_EXPERTS) throw Bad{};
        void *s = stream_of(index);
        const at::Tensor offs = at::empty({E + 1}, ids.options()), rows = at::empty({T * k}, ids.options());
        int st;
        Py_BEGIN_ALLOW_THREADS
        st = qgemm_moe_group((const int32_t *)ip, T, E, k, offs.data_ptr<int>(), rows.data_ptr<int>(), s);
        Py_END_ALLOW_THREADS
        return st == QGEMM_OK ? tuple_of({offs, rows}) : PyLong_FromLong(st);
    });
}

// moe(format_up, format_down, x, w_up, w_down, weights, offsets, rows, inter,
// group, has_zp, act, residual, out)
PyObject *moe(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    return guarded([&]() -> PyObject * {
        if (n != 14) throw Bad{};
        const at::Tensor &x = tensor(a[2]), &w = tensor(a[5]);
        if (x.dim() != 2 || w.dim() != 2) throw Bad{};
        const int index = x.get_device(), dtype = half_type(x), fu = (int)integer(a[0]), fd = (int)integer(a[1]);
        const int64_t T = x.size(0), H = x.size(1), k = w.size(1), E = tensor(a[6]).numel() - 1;
        const int64_t inter = integer(a[8]), group = integer(a[9]);
        const int zp = PyObject_IsTrue(a[10]), act = (int)integer(a[11]);
        if (T < 1 || E < 1 || inter < 1 || inter > INT32_MAX / 2 || zp < 0) throw Bad{};
        const void *xp = data(a[2], index), *up = data(a[3], index), *dp = data(a[4], index);
        const void *wt = data(a[5], index, at::kFloat, {T, k}), *op = data(a[6], index, at::kInt, {E + 1});
        const void *rp = data(a[7], index, at::kInt, {T * k}), *res = data(a[12], index, x.scalar_type(), {T, H});
        const size_t ub = of_experts(E, packed(fu, 2 * inter, H, group, zp));
        const size_t db = of_experts(E, packed(fd, H, inter, group, zp));
        holds(a[3], ub);
        holds(a[4], db);
        void *yp = data(a[13], index, x.scalar_type(), {T, H});
        if (yp) {
            const size_t yb = (size_t)(2 * T * H);
            if (yp != xp) apart(yp, yb, xp, yb);
            if (yp != res) apart(yp, yb, res, yb);
            apart(yp, yb, up, ub);
            apart(yp, yb, dp, db);
            apart(yp, yb, wt, (size_t)(4 * T * k));
            apart(yp, yb, op, (size_t)(4 * (E + 1)));
            apart(yp, yb, rp, (size_t)(4 * T * k));
        }
        const size_t need = qgemm_moe_workspace_bytes(T, k, H, inter);
        if (need == 0) throw Bad{};
        void *s = stream_of(index);
        const at::Tensor y = yp ? tensor(a[13]) : at::empty({T, H}, x.options());
        if (!yp) yp = y.data_ptr();
        const at::Tensor ws = at::empty({(int64_t)need}, x.options().dtype(at::kByte));
        int st;
        Py_BEGIN_ALLOW_THREADS
        st = qgemm_moe(fu, fd, xp, up, dp, (const float *)wt, (const int32_t *)op, (const int32_t *)rp, res, yp, T, k, E,
                       H, inter, group, zp, act, dtype, ws.data_ptr(), need, s);
        Py_END_ALLOW_THREADS
        return wrap_or_status(st, y);
    });
}

// Rows of heads [T][heads][head_dim], each row's heads side by side.
struct Rows {
    const void *p = nullptr;
    int64_t T = 0, heads = 0, D = 0, stride = 0;
    size_t span() const { return (size_t)(2 * ((T - 1) * stride + heads * D)); }
};

Rows rows(PyObject *o, int index, at::ScalarType type)
{
    const at::Tensor &t = tensor(o);
    if (t.dim() != 3 || !t.is_cuda() || t.get_device() != index || t.scalar_type() != type) throw Bad{};
    Rows r{nullptr, t.size(0), t.size(1), t.size(2), 0};
    if (r.T < 1 || r.heads < 1 || r.D < 1 || t.stride(2) != 1 || (r.heads > 1 && t.stride(1) != r.D)) throw Bad{};
    r.stride = r.T > 1 ? t.stride(0) : r.heads * r.D;
    r.p = t.data_ptr();
    return r;
}

float real(PyObject *o)
{
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred()) throw Bad{};
    return (float)v;
}

// The rotation's table and positions, and the norm: what qk_norm_rope and
// kv_append share.
struct Turn {
    const float *rope = nullptr;
    int64_t lines = 0, rot = 0;
    const int32_t *positions = nullptr;
    float eps = -1.0f;
    int interleaved = 0;
};

Turn turn(PyObject *rope, PyObject *positions, PyObject *eps, PyObject *interleaved, int64_t T, int index)
{
    Turn t;
    if (rope != Py_None) {
        const at::Tensor &r = tensor(rope);
        if (r.dim() != 2 || r.scalar_type() != at::kFloat) throw Bad{};
        t.rope = (const float *)data(rope, index);
        t.lines = r.size(0);
        t.rot = r.size(1);
    }
    t.positions = (const int32_t *)data(positions, index, at::kInt, {T});
    if (eps != Py_None) t.eps = real(eps);
    t.interleaved = PyObject_IsTrue(interleaved);
    if (t.interleaved < 0) throw Bad{};
    return t;
}

// A cache and its sequences.
struct Cache {
    uint8_t *p = nullptr;
    int64_t pages = 0, page = 0, width = 0, S = 0;
    const int32_t *tables = nullptr, *lens = nullptr, *offsets = nullptr;
    size_t bytes = 0;
};

Cache cache_of(PyObject *cache, PyObject *tables, PyObject *lens, PyObject *offsets, int64_t T, int64_t kv_heads, int64_t D,
               int index)
{
    const at::Tensor &c = tensor(cache), &tb = tensor(tables);
    if (c.dim() != 2 || c.scalar_type() != at::kByte || tb.dim() != 2 || lens == Py_None) throw Bad{};
    if (kv_heads < 1 || kv_heads > 65536 || (D != 64 && D != 128)) throw Bad{};  // their product divides below: never 0
    Cache r;
    r.p = (uint8_t *)data(cache, index);
    r.bytes = c.nbytes();
    r.pages = c.size(0);
    r.page = c.size(1) * 16 / (20 * kv_heads * D);
    if (r.page < 1 || qgemm_kv_page_bytes(kv_heads, D, r.page) != (size_t)c.size(1)) throw Bad{};
    r.S = tb.size(0);
    r.width = tb.size(1);
    r.tables = (const int32_t *)data(tables, index, at::kInt, {r.S, r.width});
    r.lens = (const int32_t *)data(lens, index, at::kInt, {r.S});
    r.offsets = (const int32_t *)data(offsets, index, at::kInt, {r.S + 1});
    if (r.S < 1 || (!r.offsets && r.S != T)) throw Bad{};
    return r;
}

// qk_norm_rope(q, k, rope, positions, q_weight, k_weight, eps, interleaved)
PyObject *qk_norm_rope(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    return guarded([&]() -> PyObject * {
        if (n != 8) throw Bad{};
        const at::Tensor &x = tensor(a[0]);
        const int index = x.get_device(), dtype = half_type(x);
        const Rows q = rows(a[0], index, x.scalar_type());
        Rows k;
        if (a[1] != Py_None) {
            k = rows(a[1], index, x.scalar_type());
            if (k.T != q.T || k.D != q.D) throw Bad{};
        }
        const Turn t = turn(a[2], a[3], a[6], a[7], q.T, index);
        if (t.rope && !t.positions) throw Bad{};
        const float *wq = (const float *)data(a[4], index, at::kFloat, {q.D});
        const float *wk = (const float *)data(a[5], index, at::kFloat, {q.D});
        void *s = stream_of(index);
        const at::Tensor yq = at::empty({q.T, q.heads, q.D}, x.options());
        at::Tensor yk;
        if (k.p) yk = at::empty({k.T, k.heads, k.D}, x.options());
        int st;
        Py_BEGIN_ALLOW_THREADS
        st = qgemm_qk_norm_rope(q.p, q.stride, k.p, k.stride, wq, wk, t.rope, t.lines, t.rot, t.interleaved, t.positions, t.eps,
                                yq.data_ptr(), q.heads * q.D, k.p ? yk.data_ptr() : nullptr, k.heads * q.D, q.T, q.heads, k.heads,
                                q.D, dtype, s);
        Py_END_ALLOW_THREADS
        if (st != QGEMM_OK) return PyLong_FromLong(st);
        if (k.p) return tuple_of({yq, yk});
        PyObject *y = THPVariable_Wrap(yq), *both = y ? PyTuple_Pack(2, y, Py_None) : nullptr;
        Py_XDECREF(y);
        return both;
    });
}

// kv_append(cache, k, v, tables, lens, offsets, rope, positions, k_weight,
// eps, interleaved, q, q_weight): the queries' result, or True without any
PyObject *kv_append(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    return guarded([&]() -> PyObject * {
        if (n != 13) throw Bad{};
        const at::Tensor &x = tensor(a[1]);
        const int index = x.get_device(), dtype = half_type(x);
        const Rows k = rows(a[1], index, x.scalar_type()), v = rows(a[2], index, x.scalar_type());
        if (v.T != k.T || v.heads != k.heads || v.D != k.D) throw Bad{};
        const Cache c = cache_of(a[0], a[3], a[4], a[5], k.T, k.heads, k.D, index);
        const Turn t = turn(a[6], a[7], a[9], a[10], k.T, index);
        const float *wk = (const float *)data(a[8], index, at::kFloat, {k.D});
        const float *wq = (const float *)data(a[12], index, at::kFloat, {k.D});
        Rows q;
        if (a[11] != Py_None) {
            q = rows(a[11], index, x.scalar_type());
            if (q.T != k.T || q.D != k.D) throw Bad{};
            apart(c.p, c.bytes, q.p, q.span());
        }
        apart(c.p, c.bytes, k.p, k.span());
        apart(c.p, c.bytes, v.p, v.span());
        apart(c.p, c.bytes, c.tables, (size_t)(4 * c.S * c.width));
        apart(c.p, c.bytes, c.lens, (size_t)(4 * c.S));
        apart(c.p, c.bytes, c.offsets, (size_t)(4 * (c.S + 1)));
        apart(c.p, c.bytes, t.rope, (size_t)(4 * t.lines * t.rot));
        apart(c.p, c.bytes, t.positions, (size_t)(4 * k.T));
        apart(c.p, c.bytes, wk, (size_t)(4 * k.D));
        apart(c.p, c.bytes, wq, (size_t)(4 * k.D));
        void *s = stream_of(index);
        at::Tensor y;
        if (q.p) y = at::empty({q.T, q.heads, q.D}, x.options());
        int st;
        Py_BEGIN_ALLOW_THREADS
        st = qgemm_kv_append(c.p, c.pages, c.page, c.tables, c.width, c.lens, c.offsets, c.S, k.p, k.stride, v.p, v.stride, wk,
                             t.rope, t.lines, t.rot, t.interleaved, t.positions, t.eps, q.p, q.stride, wq,
                             q.p ? y.data_ptr() : nullptr, q.heads * q.D, k.T, q.heads, k.heads, k.D, dtype | QGEMM_ZERO_REST, s);
        Py_END_ALLOW_THREADS
        if (st != QGEMM_OK) return PyLong_FromLong(st);
        if (q.p) return THPVariable_Wrap(y);
        Py_RETURN_TRUE;
    });
}

// kv_read(cache, tables, lens, T, kv_heads, head_dim, offsets, type)
PyObject *kv_read(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    return guarded([&]() -> PyObject * {
        if (n != 8) throw Bad{};
        const at::Tensor &x = tensor(a[0]);
        const int index = x.get_device();
        const int64_t T = integer(a[3]), H = integer(a[4]), D = integer(a[5]), type = integer(a[7]);
        if (T < 1 || D < 1 || (type != QGEMM_F16 && type != QGEMM_BF16 && type != QGEMM_F32)) throw Bad{};
        const Cache c = cache_of(a[0], a[1], a[2], a[6], T, H, D, index);
        void *s = stream_of(index);
        const at::TensorOptions o = x.options().dtype(type == QGEMM_F16 ? at::kHalf : type == QGEMM_BF16 ? at::kBFloat16 : at::kFloat);
        const at::Tensor k = at::empty({T, H, D}, o), v = at::empty({T, H, D}, o);
        int st;
        Py_BEGIN_ALLOW_THREADS
        st = qgemm_kv_read(c.p, c.pages, c.page, c.tables, c.width, c.lens, c.offsets, c.S, k.data_ptr(), v.data_ptr(), T, H, D,
                           (int)type, s);
        Py_END_ALLOW_THREADS
        return st == QGEMM_OK ? tuple_of({k, v}) : PyLong_FromLong(st);
    });
}

// kv_attention(q, cache, tables, lens, kv_heads, offsets, scale, window,
// max_len, out)
PyObject *kv_attention(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    return guarded([&]() -> PyObject * {
        if (n != 10) throw Bad{};
        const at::Tensor &x = tensor(a[0]);
        const int index = x.get_device(), dtype = half_type(x);
        const Rows q = rows(a[0], index, x.scalar_type());
        const int64_t H = integer(a[4]), window = integer(a[7]), max_len = integer(a[8]);
        const Cache c = cache_of(a[1], a[2], a[3], a[5], q.T, H, q.D, index);
        const float scale = a[6] == Py_None ? (float)(1.0 / std::sqrt((double)q.D)) : real(a[6]);
        const int64_t all = c.width * c.page;
        if (max_len < 0) throw Bad{};
        void *yp = data(a[9], index, x.scalar_type(), {q.T, q.heads, q.D});
        if (yp) {
            const size_t yb = tensor(a[9]).nbytes();
            apart(yp, yb, q.p, q.span());
            apart(yp, yb, c.p, c.bytes);
            apart(yp, yb, c.tables, (size_t)(4 * c.S * c.width));
            apart(yp, yb, c.lens, (size_t)(4 * c.S));
            apart(yp, yb, c.offsets, (size_t)(4 * (c.S + 1)));
        }
        void *s = stream_of(index);
        const at::Tensor y = yp ? tensor(a[9]) : at::empty({q.T, q.heads, q.D}, x.options());
        const size_t need = qgemm_kv_attention_workspace_bytes(q.T, c.S, q.heads, H, q.D, max_len && max_len < all ? max_len : all,
                                                               c.offsets != nullptr);
        at::Tensor ws;
        if (need) ws = at::empty({(int64_t)need}, x.options().dtype(at::kByte));
        int st;
        Py_BEGIN_ALLOW_THREADS
        st = qgemm_kv_attention(q.p, q.stride, c.p, c.pages, c.page, c.tables, c.width, c.lens, c.offsets, c.S, y.data_ptr(), q.T,
                                q.heads, H, q.D, window, scale, max_len, yp ? dtype : dtype | QGEMM_ZERO_REST, need ? ws.data_ptr() : nullptr,
                                need, s);
        Py_END_ALLOW_THREADS
        return wrap_or_status(st, y);
    });
}

// bind(current_device, current_stream): torch's queries, as callables
PyObject *bind(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    if (n != 2) {
        PyErr_SetString(PyExc_TypeError, "bind takes two callables");
        return nullptr;
    }
    Py_INCREF(a[0]);
    Py_INCREF(a[1]);
    Py_XSETREF(g_device, a[0]);
    Py_XSETREF(g_stream, a[1]);
    Py_RETURN_NONE;
}

PyMethodDef methods[] = {
    {"bind", (PyCFunction)(void (*)(void))bind, METH_FASTCALL, nullptr},
    {"linear", (PyCFunction)(void (*)(void))linear, METH_FASTCALL, nullptr},
    {"moe_route", (PyCFunction)(void (*)(void))moe_route, METH_FASTCALL, nullptr},
    {"moe_group", (PyCFunction)(void (*)(void))moe_group, METH_FASTCALL, nullptr},
    {"moe", (PyCFunction)(void (*)(void))moe, METH_FASTCALL, nullptr},
    {"qk_norm_rope", (PyCFunction)(void (*)(void))qk_norm_rope, METH_FASTCALL, nullptr},
    {"kv_append", (PyCFunction)(void (*)(void))kv_append, METH_FASTCALL, nullptr},
    {"kv_read", (PyCFunction)(void (*)(void))kv_read, METH_FASTCALL, nullptr},
    {"kv_attention", (PyCFunction)(void (*)(void))kv_attention, METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr},
};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_calls", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__calls(void) { return PyModule_Create(&module); }
