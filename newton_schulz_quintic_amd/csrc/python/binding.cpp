// Python binding of the training-step operators: the module _binding, whose
// functions carry the C entry points' names and take torch tensors. Argument
// marshalling only (addresses, sizes, strides, types; what is wrong with them is
// raised as TypeError, ValueError or NSError), done here because a short
// operator's kernel takes 4 us: marshalled in Python a call took 7 to 11 us.
//
// Every tensor must be on the current GPU. Work goes to `stream` (default:
// torch's current one) without waiting for it. Tensors that torch allocated on
// another stream are the caller's to order and to record on it. Autograd records
// nothing of a call; the versions of the tensors that it writes move on.

#include <Python.h>

#include <ATen/core/Tensor.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cstring>
#include <initializer_list>
#include <string>

#include "ns.h"

namespace {

struct Raised {};   // a Python exception is set

[[noreturn]] void raise(PyObject *type, const std::string &message) {
    PyErr_SetString(type, message.c_str());
    throw Raised{};
}

// Kept for the life of the module.
PyObject *g_ns_error = nullptr, *g_new_workspace = nullptr, *g_raw_stream = nullptr, *g_get_device = nullptr;
PyObject *g_str_device = nullptr, *g_str_cuda_stream = nullptr;

void check(ns_status status) {
    if (status == NS_OK) return;
    PyObject *e = PyObject_CallFunction(g_ns_error, "is", (int)status, ns_last_error());
    if (e) {
        PyErr_SetObject(g_ns_error, e);
        Py_DECREF(e);
    }
    throw Raised{};
}

std::string text(const at::Tensor &t) {
    std::string s = "(";
    for (int64_t i = 0; i < t.dim(); ++i) s += (i ? ", " : "") + std::to_string(t.size(i));
    return s + ")";
}
std::string text(std::initializer_list<int64_t> shape) {
    std::string s = "(";
    bool first = true;
    for (int64_t n : shape) {
        s += (first ? "" : ", ") + std::to_string(n);
        first = false;
    }
    return s + ")";
}
std::string text(at::ScalarType t) { return std::string("torch.") + c10::toString(t); }

// ---------------------------------------------------------------------------
// arguments
// ---------------------------------------------------------------------------

constexpr int kMaxArgs = 20;

// A function's parameters in order, `required` of them without a default.
struct Signature {
    const char *function;
    int count, required;
    const char *names[kMaxArgs];
    PyObject *interned[kMaxArgs];
};

struct Args {
    const Signature &sig;
    PyObject *v[kMaxArgs] = {};

    Args(Signature &s, PyObject *const *args, Py_ssize_t n, PyObject *kwnames) : sig(s) {
        if (n > s.count)
            raise(PyExc_TypeError, std::string(s.function) + "() takes at most " + std::to_string(s.count) + " arguments");
        for (Py_ssize_t i = 0; i < n; ++i) v[i] = args[i];
        const Py_ssize_t named = kwnames ? PyTuple_GET_SIZE(kwnames) : 0;
        for (Py_ssize_t j = 0; j < named; ++j) {
            PyObject *key = PyTuple_GET_ITEM(kwnames, j);
            int at = -1;
            for (int i = 0; i < s.count && at < 0; ++i)
                if (s.interned[i] == key) at = i;
            for (int i = 0; i < s.count && at < 0; ++i)   // a key that was not interned
                if (PyUnicode_Compare(s.interned[i], key) == 0) at = i;
            const char *name = PyUnicode_AsUTF8(key);
            if (!name) throw Raised{};
            if (at < 0) raise(PyExc_TypeError, std::string(s.function) + "() got an unexpected keyword argument '" + name + "'");
            if (v[at]) raise(PyExc_TypeError, std::string(s.function) + "() got multiple values for argument '" + name + "'");
            v[at] = args[n + j];
        }
        for (int i = 0; i < s.required; ++i)
            if (!v[i]) raise(PyExc_TypeError, std::string(s.function) + "() missing argument '" + s.names[i] + "'");
        for (int i = 0; i < s.count; ++i)
            if (!v[i]) v[i] = Py_None;
    }

    const at::Tensor *tensor(int i) const {
        if (v[i] == Py_None) return nullptr;
        if (!THPVariable_Check(v[i])) raise(PyExc_TypeError, std::string(sig.names[i]) + " must be a tensor");
        return &THPVariable_Unpack(v[i]);
    }
    const at::Tensor &must(int i) const {
        const at::Tensor *t = tensor(i);
        if (!t) raise(PyExc_ValueError, std::string(sig.names[i]) + " is required");
        return *t;
    }
    double number(int i, double otherwise) const {
        if (v[i] == Py_None) return otherwise;
        const double x = PyFloat_AsDouble(v[i]);
        if (x == -1.0 && PyErr_Occurred()) throw Raised{};
        return x;
    }
    int64_t integer(int i) const {
        const long long x = PyLong_AsLongLong(v[i]);
        if (x == -1 && PyErr_Occurred()) throw Raised{};
        return x;
    }
    bool flag(int i) const {
        if (v[i] == Py_None) return false;
        const int x = PyObject_IsTrue(v[i]);
        if (x < 0) throw Raised{};
        return x;
    }
    // Checks that the tensors among arguments [0, n) are on the current GPU; returns its index.
    int64_t device(int n) const {
        int64_t here = -1;
        for (int i = 0; i < n; ++i) {
            if (v[i] == Py_None || !THPVariable_Check(v[i])) continue;
            const at::Tensor &t = THPVariable_Unpack(v[i]);
            const int64_t at = t.is_cuda() ? t.get_device() : -1;
            if (here < 0 && at >= 0) {
                PyObject *d = PyObject_CallNoArgs(g_get_device);
                if (!d) throw Raised{};
                here = PyLong_AsLongLong(d);
                Py_DECREF(d);
            }
            if (at < 0 || at != here)
                raise(PyExc_ValueError, std::string(sig.names[i]) + " is on " + t.device().str() + ", not on the current GPU");
        }
        return here;
    }
    void *stream(int i, int64_t device) const {
        PyObject *s;
        if (v[i] == Py_None) {
            PyObject *d = PyLong_FromLongLong(device < 0 ? 0 : device);
            if (!d) throw Raised{};
            s = PyObject_CallOneArg(g_raw_stream, d);
            Py_DECREF(d);
        } else if (PyLong_Check(v[i])) {
            s = Py_NewRef(v[i]);
        } else {
            s = PyObject_GetAttr(v[i], g_str_cuda_stream);
        }
        if (!s) throw Raised{};
        const unsigned long long h = PyLong_AsUnsignedLongLong(s);
        Py_DECREF(s);
        if (h == (unsigned long long)-1 && PyErr_Occurred()) throw Raised{};
        return reinterpret_cast<void *>(h);
    }
};

ns_dtype code(const at::Tensor &t, const char *name) {
    if (t.scalar_type() == at::kBFloat16) return NS_BF16;
    if (t.scalar_type() == at::kFloat) return NS_F32;
    raise(PyExc_TypeError, std::string(name) + ": unsupported dtype " + text(t.scalar_type()));
}

int32_t int_bytes(const at::Tensor &t, const char *name) {
    if (t.scalar_type() == at::kInt) return 4;
    if (t.scalar_type() == at::kLong) return 8;
    raise(PyExc_TypeError, std::string(name) + " must be int32 or int64, not " + text(t.scalar_type()));
}

void want_type(const at::Tensor &t, const char *name, at::ScalarType type) {
    if (t.scalar_type() != type)
        raise(PyExc_TypeError, std::string(name) + " must be " + text(type) + ", not " + text(t.scalar_type()));
}

// A contiguous tensor of one shape and type; its address (NULL for None).
template <typename P>
P *array(const at::Tensor *t, const char *name, std::initializer_list<int64_t> shape, at::ScalarType type) {
    if (!t) return nullptr;
    want_type(*t, name, type);
    if (t->sizes() != at::IntArrayRef(shape) || !t->is_contiguous())
        raise(PyExc_ValueError, std::string(name) + " must be contiguous and of shape " + text(shape) + ", not " + text(*t));
    return static_cast<P *>(t->data_ptr());
}

// A (rows, cols) tensor whose rows are contiguous; its row stride.
int64_t row_stride(const at::Tensor &t, const char *name, int64_t rows, int64_t cols, at::ScalarType type) {
    want_type(t, name, type);
    if (t.dim() != 2 || t.size(0) != rows || t.size(1) != cols)
        raise(PyExc_ValueError, std::string(name) + " must have shape " + text({rows, cols}) + ", not " + text(t));
    if (t.stride(1) != 1 && cols > 1 && rows) raise(PyExc_ValueError, std::string("each row of ") + name + " must be contiguous");
    return rows > 1 ? t.stride(0) : std::max<int64_t>(cols, 1);
}

// The caller's workspace, or a new one of the size that `size` gives (the
// library checks that of a given one). A new reference.
template <typename Size>
PyObject *workspace(PyObject *given, const Size &size, PyObject *like, PyObject *stream, void **p, size_t *bytes) {
    PyObject *w;
    if (given == Py_None) {
        size_t need = 0;
        check(size(&need));
        PyObject *device = PyObject_GetAttr(like, g_str_device);
        if (!device) throw Raised{};
        w = PyObject_CallFunction(g_new_workspace, "nOO", (Py_ssize_t)need, device, stream);
        Py_DECREF(device);
        if (!w) throw Raised{};
    } else {
        w = Py_NewRef(given);
    }
    if (!THPVariable_Check(w)) {
        Py_DECREF(w);
        raise(PyExc_TypeError, "workspace must be a tensor");
    }
    const at::Tensor &t = THPVariable_Unpack(w);
    if (t.scalar_type() != at::kByte || !t.is_contiguous()) {
        Py_DECREF(w);
        raise(PyExc_ValueError, "workspace must be a contiguous uint8 tensor");
    }
    *p = t.data_ptr();
    *bytes = (size_t)t.numel();
    return w;
}

// Tells autograd that a call has written these: a backward pass that saved one of them, written in place, then says so.
void wrote(std::initializer_list<const at::Tensor *> outputs) {
    for (const at::Tensor *t : outputs)
        if (t && !t->is_inference()) t->unsafeGetTensorImpl()->bump_version();
}

// Drops a reference on the way out, unless it is given away.
struct Held {
    PyObject *o;
    ~Held() { Py_XDECREF(o); }
    PyObject *give() {
        PyObject *r = o;
        o = nullptr;
        return r;
    }
};

template <typename F> PyObject *guarded(const F &f) {
    try {
        return f();
    } catch (const Raised &) {
        return nullptr;
    } catch (const std::exception &e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
        return nullptr;
    }
}

// ---------------------------------------------------------------------------
// queries and keys
// ---------------------------------------------------------------------------

// A (batch, seq, heads, head_dim) or (seq, heads, head_dim) tensor with contiguous heads, like `of`.
ns_heads heads(const at::Tensor *t, const char *name, const at::Tensor *of, const char *of_name) {
    if (!t != !of) raise(PyExc_ValueError, std::string(name) + " goes with " + of_name + ": give both or neither");
    if (!t) return ns_heads{nullptr, 0, 0, 0, 0};
    if (t->scalar_type() != of->scalar_type() || t->sizes() != of->sizes())
        raise(PyExc_ValueError, std::string(name) + " must have shape " + text(*of) + " and dtype " + text(of->scalar_type()) +
                                    ", not " + text(*t) + ", " + text(t->scalar_type()));
    const int64_t n = t->dim();
    if (t->stride(n - 1) != 1 && t->size(n - 1) > 1 && t->numel())
        raise(PyExc_ValueError, std::string("each head of ") + name + " must be contiguous");
    return ns_heads{t->data_ptr(), n == 4 ? t->stride(0) : 0, t->stride(n - 3), t->stride(n - 2), (int32_t)t->size(n - 2)};
}

// What the forward and the backward call share.
struct HeadArgs {
    int64_t batch, seq;
    int32_t dim;
    ns_dtype dtype, w_dtype = NS_F32;
    ns_heads q, k;
    const void *wq = nullptr, *wk = nullptr, *pos = nullptr;
    const float *cos = nullptr, *sin = nullptr;
    int64_t rows = 0, pos_stride = 0;
    int32_t rope = 0, pos_bytes = 4;

    HeadArgs(const at::Tensor *tq, const at::Tensor *tk, const at::Tensor *qw, const at::Tensor *kw, const at::Tensor *c,
             const at::Tensor *s, const at::Tensor *p) {
        const at::Tensor *first = tq ? tq : tk;
        if (!first) raise(PyExc_ValueError, "q or k is required");
        dtype = code(*first, tq ? "q" : "k");
        const int64_t n = first->dim();
        if (n != 3 && n != 4) raise(PyExc_ValueError, "q and k must be (batch, seq, heads, head_dim) or (seq, heads, head_dim)");
        batch = n == 4 ? first->size(0) : 1;
        seq = first->size(n - 3);
        dim = (int32_t)std::min<int64_t>(first->size(n - 1), INT32_MAX);
        if (tq && tk &&
            (tk->scalar_type() != tq->scalar_type() || tk->dim() != n || tk->size(0) != tq->size(0) ||
             tk->size(n - 3) != seq || tk->size(n - 1) != tq->size(n - 1)))
            raise(PyExc_ValueError, "q and k must share dtype, batch, seq and head_dim");
        q = heads(tq, "q", tq, "q");
        k = heads(tk, "k", tk, "k");
        if (const at::Tensor *w = qw ? qw : kw) {
            w_dtype = code(*w, "weights");
            for (const at::Tensor *x : {qw, kw})
                if (x && (x->scalar_type() != w->scalar_type() || x->dim() != 1 || x->size(0) != dim || !x->is_contiguous()))
                    raise(PyExc_ValueError, "weights must share one dtype and be contiguous of shape " + text({dim}));
            wq = qw ? qw->data_ptr() : nullptr;
            wk = kw ? kw->data_ptr() : nullptr;
        }
        if (!c != !s) raise(PyExc_ValueError, "cos and sin go together");
        if (c) {
            if (c->dim() != 2) raise(PyExc_ValueError, "cos and sin must be (positions, rope_dim / 2)");
            rows = c->size(0);
            rope = (int32_t)std::min<int64_t>(2 * c->size(1), INT32_MAX - 1);
            cos = array<float>(c, "cos", {rows, c->size(1)}, at::kFloat);
            sin = array<float>(s, "sin", {rows, c->size(1)}, at::kFloat);
        }
        if (p) {
            pos_bytes = int_bytes(*p, "pos");
            const int64_t last = p->dim() - 1;   // one row for all sequences (a stride of 0), or a row each
            if (last < 0 || last > 1 || p->size(last) != seq || (last == 1 && p->size(0) != batch && p->size(0) != 1))
                raise(PyExc_ValueError, "pos must have shape " + text({seq}) + ", " + text({1, seq}) + " or " + text({batch, seq}) +
                                            ", not " + text(*p));
            if (p->stride(last) != 1 && seq > 1 && batch) raise(PyExc_ValueError, "pos must have contiguous rows");
            if (last == 1 && p->size(0) > 1) pos_stride = p->stride(0);
            pos = p->data_ptr();
        }
    }
};

Signature s_norm_rope = {"ns_qk_norm_rope", 12, 4,
                         {"q", "k", "q_out", "k_out", "q_weight", "k_weight", "cos", "sin", "pos", "eps", "interleaved", "stream"}};
PyObject *norm_rope(PyObject *, PyObject *const *args, Py_ssize_t n, PyObject *kw) {
    return guarded([&]() -> PyObject * {
        const Args a(s_norm_rope, args, n, kw);
        const int64_t device = a.device(9);
        const at::Tensor *q = a.tensor(0), *k = a.tensor(1);
        const HeadArgs h(q, k, a.tensor(4), a.tensor(5), a.tensor(6), a.tensor(7), a.tensor(8));
        const ns_heads oq = heads(a.tensor(2), "q_out", q, "q"), ok = heads(a.tensor(3), "k_out", k, "k");
        check(ns_qk_norm_rope(h.batch, h.seq, h.dim, h.dtype, &h.q, &h.k, h.wq, h.wk, h.w_dtype, (float)a.number(9, 1e-6),
                              h.cos, h.sin, h.rows, h.rope, a.flag(10), h.pos, h.pos_bytes, h.pos_stride, &oq, &ok,
                              a.stream(11, device)));
        wrote({a.tensor(2), a.tensor(3)});
        Py_RETURN_NONE;
    });
}

Signature s_norm_rope_backward = {"ns_qk_norm_rope_backward", 17, 6,
                                  {"q", "k", "dq_out", "dk_out", "dq", "dk", "dq_weight", "dk_weight", "q_weight",
                                   "k_weight", "cos", "sin", "pos", "eps", "interleaved", "workspace", "stream"}};
PyObject *norm_rope_backward(PyObject *, PyObject *const *args, Py_ssize_t n, PyObject *kw) {
    return guarded([&]() -> PyObject * {
        const Args a(s_norm_rope_backward, args, n, kw);
        const int64_t device = a.device(16);
        const at::Tensor *q = a.tensor(0), *k = a.tensor(1);
        const HeadArgs h(q, k, a.tensor(8), a.tensor(9), a.tensor(10), a.tensor(11), a.tensor(12));
        const ns_heads gq = heads(a.tensor(2), "dq_out", q, "q"), gk = heads(a.tensor(3), "dk_out", k, "k");
        const ns_heads oq = heads(a.tensor(4), "dq", q, "q"), ok = heads(a.tensor(5), "dk", k, "k");
        float *wq = array<float>(a.tensor(6), "dq_weight", {h.dim}, at::kFloat);
        float *wk = array<float>(a.tensor(7), "dk_weight", {h.dim}, at::kFloat);
        void *p = nullptr;
        size_t bytes = 0;
        Held ws{nullptr};
        if (wq || wk || a.v[15] != Py_None)
            ws.o = workspace(a.v[15], [&](size_t *need) { return ns_qk_norm_rope_workspace_bytes(h.batch, h.seq, h.dim, need); },
                             q ? a.v[0] : a.v[1], a.v[16], &p, &bytes);
        check(ns_qk_norm_rope_backward(h.batch, h.seq, h.dim, h.dtype, &h.q, &h.k, &gq, &gk, h.wq, h.wk, h.w_dtype,
                                       (float)a.number(13, 1e-6), h.cos, h.sin, h.rows, h.rope, a.flag(14), h.pos,
                                       h.pos_bytes, h.pos_stride, &oq, &ok, wq, wk, p, bytes, a.stream(16, device)));
        wrote({a.tensor(4), a.tensor(5), a.tensor(6), a.tensor(7)});
        if (ws.o) return ws.give();
        Py_RETURN_NONE;
    });
}

// ---------------------------------------------------------------------------
// tokens by expert
// ---------------------------------------------------------------------------

Signature s_moe_sort = {"ns_moe_sort", 7, 5,
                        {"expert_ids", "num_experts", "offsets", "slot_of_row", "row_of_slot", "workspace", "stream"}};
PyObject *moe_sort(PyObject *, PyObject *const *args, Py_ssize_t n, PyObject *kw) {
    return guarded([&]() -> PyObject * {
        const Args a(s_moe_sort, args, n, kw);
        const int64_t device = a.device(6);
        const at::Tensor &ids = a.must(0);
        if (ids.dim() != 2) raise(PyExc_ValueError, "expert_ids must be (tokens, top_k)");
        const int64_t t = ids.size(0), k = ids.size(1), e = a.integer(1);
        const int32_t id_bytes = int_bytes(ids, "expert_ids");
        const int64_t ld = row_stride(ids, "expert_ids", t, k, ids.scalar_type());
        if (k > INT32_MAX || e > INT32_MAX - 1 || e < 0) raise(PyExc_ValueError, "num_experts or top_k out of range");
        a.must(2), a.must(3), a.must(4);
        int32_t *offsets = array<int32_t>(a.tensor(2), "offsets", {e + 1}, at::kInt);
        int32_t *slot_of_row = array<int32_t>(a.tensor(3), "slot_of_row", {t * k}, at::kInt);
        int32_t *row_of_slot = array<int32_t>(a.tensor(4), "row_of_slot", {t, k}, at::kInt);
        void *p;
        size_t bytes;
        Held ws{workspace(a.v[5], [&](size_t *need) { return ns_moe_sort_workspace_bytes(t, (int32_t)k, (int32_t)e, need); },
                          a.v[0], a.v[6], &p, &bytes)};
        check(ns_moe_sort(t, (int32_t)k, (int32_t)e, ids.data_ptr(), id_bytes, ld, offsets, slot_of_row, row_of_slot, p, bytes,
                          a.stream(6, device)));
        wrote({a.tensor(2), a.tensor(3), a.tensor(4)});
        return ws.give();
    });
}

// Sizes of a call on token rows `tok`, and the map's address.
struct RowCall {
    int64_t t, hidden;
    int32_t k, h;
    ns_dtype dtype;
    at::ScalarType type;
    const int32_t *rows;
    RowCall(const at::Tensor &tok, const char *name, const at::Tensor &map) : type(tok.scalar_type()) {
        if (map.dim() != 2) raise(PyExc_ValueError, "row_of_slot must be (tokens, top_k)");
        if (tok.dim() != 2) raise(PyExc_ValueError, std::string(name) + " must be (tokens, hidden)");
        t = map.size(0);
        hidden = tok.size(1);
        if (map.size(1) > INT32_MAX || hidden > INT32_MAX) raise(PyExc_ValueError, "top_k or hidden out of range");
        k = (int32_t)map.size(1);
        h = (int32_t)hidden;
        dtype = code(tok, name);
        rows = array<int32_t>(&map, "row_of_slot", {t, map.size(1)}, at::kInt);
    }
    int64_t token_rows(const at::Tensor &x, const char *name) const { return row_stride(x, name, t, hidden, type); }
    int64_t sorted_rows(const at::Tensor &x, const char *name) const { return row_stride(x, name, t * k, hidden, type); }
};

Signature s_moe_dispatch = {"ns_moe_dispatch", 4, 3, {"x", "row_of_slot", "xs", "stream"}};
PyObject *moe_dispatch(PyObject *, PyObject *const *args, Py_ssize_t n, PyObject *kw) {
    return guarded([&]() -> PyObject * {
        const Args a(s_moe_dispatch, args, n, kw);
        const int64_t device = a.device(3);
        const at::Tensor &x = a.must(0), &xs = a.must(2);
        const RowCall c(x, "x", a.must(1));
        const int64_t ld = c.token_rows(x, "x"), out_ld = c.sorted_rows(xs, "xs");
        check(ns_moe_dispatch(c.t, c.k, c.h, c.dtype, x.data_ptr(), ld, c.rows, xs.data_ptr(), out_ld, a.stream(3, device)));
        wrote({&xs});
        Py_RETURN_NONE;
    });
}

Signature s_moe_dispatch_backward = {"ns_moe_dispatch_backward", 4, 3, {"dxs", "row_of_slot", "dx", "stream"}};
PyObject *moe_dispatch_backward(PyObject *, PyObject *const *args, Py_ssize_t n, PyObject *kw) {
    return guarded([&]() -> PyObject * {
        const Args a(s_moe_dispatch_backward, args, n, kw);
        const int64_t device = a.device(3);
        const at::Tensor &dxs = a.must(0), &dx = a.must(2);
        const RowCall c(dx, "dx", a.must(1));
        const int64_t ld = c.sorted_rows(dxs, "dxs"), out_ld = c.token_rows(dx, "dx");
        check(ns_moe_dispatch_backward(c.t, c.k, c.h, c.dtype, dxs.data_ptr(), ld, c.rows, dx.data_ptr(), out_ld,
                                       a.stream(3, device)));
        wrote({&dx});
        Py_RETURN_NONE;
    });
}

Signature s_moe_combine = {"ns_moe_combine", 5, 4, {"y", "row_of_slot", "weights", "out", "stream"}};
PyObject *moe_combine(PyObject *, PyObject *const *args, Py_ssize_t n, PyObject *kw) {
    return guarded([&]() -> PyObject * {
        const Args a(s_moe_combine, args, n, kw);
        const int64_t device = a.device(4);
        const at::Tensor &y = a.must(0), &out = a.must(3);
        const RowCall c(out, "out", a.must(1));
        const int64_t ld = c.sorted_rows(y, "y"), out_ld = c.token_rows(out, "out");
        const float *w = array<float>(a.tensor(2), "weights", {c.t, c.k}, at::kFloat);
        check(ns_moe_combine(c.t, c.k, c.h, c.dtype, y.data_ptr(), ld, c.rows, w, out.data_ptr(), out_ld, a.stream(4, device)));
        wrote({&out});
        Py_RETURN_NONE;
    });
}

Signature s_moe_combine_backward = {"ns_moe_combine_backward", 7, 6,
                                    {"dout", "y", "row_of_slot", "weights", "dy", "dweights", "stream"}};
PyObject *moe_combine_backward(PyObject *, PyObject *const *args, Py_ssize_t n, PyObject *kw) {
    return guarded([&]() -> PyObject * {
        const Args a(s_moe_combine_backward, args, n, kw);
        const int64_t device = a.device(6);
        const at::Tensor &dout = a.must(0), &y = a.must(1), &dy = a.must(4);
        const RowCall c(dout, "dout", a.must(2));
        a.must(3), a.must(5);
        const int64_t dout_ld = c.token_rows(dout, "dout"), y_ld = c.sorted_rows(y, "y"), dy_ld = c.sorted_rows(dy, "dy");
        const float *w = array<float>(a.tensor(3), "weights", {c.t, c.k}, at::kFloat);
        float *dw = array<float>(a.tensor(5), "dweights", {c.t, c.k}, at::kFloat);
        check(ns_moe_combine_backward(c.t, c.k, c.h, c.dtype, dout.data_ptr(), dout_ld, y.data_ptr(), y_ld, c.rows, w,
                                      dy.data_ptr(), dy_ld, dw, a.stream(6, device)));
        wrote({&dy, a.tensor(5)});
        Py_RETURN_NONE;
    });
}

// ---------------------------------------------------------------------------
// distillation
// ---------------------------------------------------------------------------

struct DistillCall {
    int64_t rows, vocab, ld;
    int32_t v, k, id_bytes;
    ns_dtype dtype, t_dtype;
    at::ScalarType type;
    const float *teacher_lse;
    DistillCall(const at::Tensor &z, const at::Tensor &ids, const at::Tensor &teacher, const at::Tensor *lse)
        : type(z.scalar_type()) {
        if (z.dim() != 2 || ids.dim() != 2) raise(PyExc_ValueError, "logits must be (rows, vocab) and ids (rows, top_k)");
        rows = z.size(0);
        vocab = z.size(1);
        if (vocab > INT32_MAX || ids.size(1) > INT32_MAX) raise(PyExc_ValueError, "vocab or top_k out of range");
        v = (int32_t)vocab;
        k = (int32_t)ids.size(1);
        dtype = code(z, "logits");
        ld = row_stride(z, "logits", rows, vocab, type);
        id_bytes = int_bytes(ids, "ids");
        if (ids.size(0) != rows || !ids.is_contiguous())
            raise(PyExc_ValueError, "ids must be contiguous of shape (" + std::to_string(rows) + ", top_k)");
        t_dtype = code(teacher, "teacher");
        if (teacher.sizes() != ids.sizes() || !teacher.is_contiguous())
            raise(PyExc_ValueError, "teacher must be contiguous and shaped like ids");
        teacher_lse = array<float>(lse, "teacher_lse", {rows}, at::kFloat);
    }
};

Signature s_distill = {"ns_distill_topk", 12, 5,
                       {"logits", "ids", "teacher", "loss", "lse", "teacher_lse", "rest_lse", "temperature", "grad_loss",
                        "dlogits", "workspace", "stream"}};
PyObject *distill(PyObject *, PyObject *const *args, Py_ssize_t n, PyObject *kw) {
    return guarded([&]() -> PyObject * {
        const Args a(s_distill, args, n, kw);
        const int64_t device = a.device(11);
        const at::Tensor &z = a.must(0), &ids = a.must(1), &teacher = a.must(2);
        const at::Tensor *dz = a.tensor(9), *rest = a.tensor(6), *g = a.tensor(8);
        const DistillCall c(z, ids, teacher, a.tensor(5));
        if (!dz != !g) raise(PyExc_ValueError, "dlogits and grad_loss go together");
        if (!rest != !c.teacher_lse && c.rows) raise(PyExc_ValueError, "rest_lse and teacher_lse go together");
        a.must(3), a.must(4);
        float *loss = array<float>(a.tensor(3), "loss", {c.rows}, at::kFloat);
        float *lse = array<float>(a.tensor(4), "lse", {c.rows}, at::kFloat);
        float *rest_lse = array<float>(rest, "rest_lse", {c.rows}, at::kFloat);
        const float *grad = array<float>(g, "grad_loss", {c.rows}, at::kFloat);
        const int64_t dld = dz ? row_stride(*dz, "dlogits", c.rows, c.vocab, c.type) : 0;
        void *p;
        size_t bytes;
        Held ws{workspace(a.v[10], [&](size_t *need) { return ns_distill_workspace_bytes(c.rows, c.v, c.k, need); }, a.v[0],
                          a.v[11], &p, &bytes)};
        check(ns_distill_topk(c.rows, c.v, c.k, c.dtype, z.data_ptr(), c.ld, ids.data_ptr(), c.id_bytes, teacher.data_ptr(),
                              c.t_dtype, c.teacher_lse, (float)a.number(7, 1.0), grad, loss, lse, rest_lse,
                              dz ? dz->data_ptr() : nullptr, dld, p, bytes, a.stream(11, device)));
        wrote({a.tensor(3), a.tensor(4), rest, dz});
        return ws.give();
    });
}

Signature s_distill_backward = {"ns_distill_topk_backward", 10, 6,
                                {"logits", "ids", "teacher", "lse", "grad_loss", "dlogits", "teacher_lse", "rest_lse",
                                 "temperature", "stream"}};
PyObject *distill_backward(PyObject *, PyObject *const *args, Py_ssize_t n, PyObject *kw) {
    return guarded([&]() -> PyObject * {
        const Args a(s_distill_backward, args, n, kw);
        const int64_t device = a.device(8);
        const at::Tensor &z = a.must(0), &ids = a.must(1), &teacher = a.must(2), &dz = a.must(5);
        const DistillCall c(z, ids, teacher, a.tensor(6));
        const at::Tensor *rest = a.tensor(7);
        if (!rest != !c.teacher_lse && c.rows) raise(PyExc_ValueError, "rest_lse and teacher_lse go together");
        a.must(3), a.must(4);
        const float *lse = array<float>(a.tensor(3), "lse", {c.rows}, at::kFloat);
        const float *rest_lse = array<float>(rest, "rest_lse", {c.rows}, at::kFloat);
        const float *grad = array<float>(a.tensor(4), "grad_loss", {c.rows}, at::kFloat);
        const int64_t dld = row_stride(dz, "dlogits", c.rows, c.vocab, c.type);
        check(ns_distill_topk_backward(c.rows, c.v, c.k, c.dtype, z.data_ptr(), c.ld, ids.data_ptr(), c.id_bytes,
                                       teacher.data_ptr(), c.t_dtype, c.teacher_lse, (float)a.number(8, 1.0), lse, rest_lse,
                                       grad, dz.data_ptr(), dld, a.stream(9, device)));
        wrote({&dz});
        Py_RETURN_NONE;
    });
}

// ---------------------------------------------------------------------------
// module
// ---------------------------------------------------------------------------

#define NSQ_METHOD(name, function, doc)                                                                           \
    {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(function)), METH_FASTCALL | METH_KEYWORDS, \
     PyDoc_STR(doc)}

PyMethodDef methods[] = {
    NSQ_METHOD("ns_qk_norm_rope", norm_rope,
               "ns_qk_norm_rope(q, k, q_out, k_out, q_weight=None, k_weight=None, cos=None, sin=None, pos=None, "
               "eps=1e-06, interleaved=False, stream=None)\n--\n\n"
               "RMS norm of each head of q and k, its weight and the position rotation (see ns.h).\n\n"
               "q, k: (batch, seq, heads, head_dim) or (seq, heads, head_dim) views with contiguous heads, bf16 or f32;\n"
               "k (or q) and its output may be None. cos, sin: (positions, rope_dim / 2) f32, or None for no rotation.\n"
               "pos: (seq,), (1, seq) or (batch, seq) int32 or int64 with contiguous rows, or None for 0, 1, ... Outputs may be\n"
               "the inputs."),
    NSQ_METHOD("ns_qk_norm_rope_backward", norm_rope_backward,
               "ns_qk_norm_rope_backward(q, k, dq_out, dk_out, dq, dk, dq_weight=None, dk_weight=None, q_weight=None, "
               "k_weight=None, cos=None, sin=None, pos=None, eps=1e-06, interleaved=False, workspace=None, stream=None)\n--\n\n"
               "Gradient of ns_qk_norm_rope (see ns.h): q and k are the forward's inputs, dq_weight and dk_weight\n"
               "(head_dim) f32 or None. Returns the workspace (None if neither weight gradient is wanted and none given)."),
    NSQ_METHOD("ns_moe_sort", moe_sort,
               "ns_moe_sort(expert_ids, num_experts, offsets, slot_of_row, row_of_slot, workspace=None, stream=None)\n--\n\n"
               "Rows of the tokens' choices sorted by expert (see ns.h).\n\n"
               "expert_ids: (tokens, top_k) int32 or int64 with contiguous choices; ids outside [0, num_experts) are\n"
               "dropped. offsets (num_experts + 1), slot_of_row (tokens * top_k) and row_of_slot (tokens, top_k): int32\n"
               "outputs. Returns the workspace."),
    NSQ_METHOD("ns_moe_dispatch", moe_dispatch,
               "ns_moe_dispatch(x, row_of_slot, xs, stream=None)\n--\n\n"
               "xs[row_of_slot[t, k]] = x[t] (see ns.h): x (tokens, hidden), xs (tokens * top_k, hidden), rows contiguous."),
    NSQ_METHOD("ns_moe_dispatch_backward", moe_dispatch_backward,
               "ns_moe_dispatch_backward(dxs, row_of_slot, dx, stream=None)\n--\n\n"
               "dx[t] = sum over k of dxs[row_of_slot[t, k]] (see ns.h)."),
    NSQ_METHOD("ns_moe_combine", moe_combine,
               "ns_moe_combine(y, row_of_slot, weights, out, stream=None)\n--\n\n"
               "out[t] = sum over k of weights[t, k] * y[row_of_slot[t, k]] (see ns.h); weights (tokens, top_k) f32 or None."),
    NSQ_METHOD("ns_moe_combine_backward", moe_combine_backward,
               "ns_moe_combine_backward(dout, y, row_of_slot, weights, dy, dweights, stream=None)\n--\n\n"
               "Gradient of ns_moe_combine (see ns.h): dy like y (or y itself), dweights (tokens, top_k) f32."),
    NSQ_METHOD("ns_distill_topk", distill,
               "ns_distill_topk(logits, ids, teacher, loss, lse, teacher_lse=None, rest_lse=None, temperature=1.0, "
               "grad_loss=None, dlogits=None, workspace=None, stream=None)\n--\n\n"
               "Loss against a teacher's top logits and, with grad_loss and dlogits, its gradient in the same pass\n"
               "(see ns.h).\n\n"
               "logits: (rows, vocab) with contiguous rows; ids (rows, top_k) int32 or int64; teacher (rows, top_k) bf16 or\n"
               "f32; loss, lse, rest_lse, teacher_lse, grad_loss: (rows,) f32. dlogits may be logits. Returns the workspace."),
    NSQ_METHOD("ns_distill_topk_backward", distill_backward,
               "ns_distill_topk_backward(logits, ids, teacher, lse, grad_loss, dlogits, teacher_lse=None, rest_lse=None, "
               "temperature=1.0, stream=None)\n--\n\n"
               "Gradient of ns_distill_topk by itself, from the lse (and rest_lse) it gave (see ns.h)."),
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_binding", "Training-step operators of the library. Autograd records nothing of a call (see the\n"
                      "example's autograd functions); the versions of the tensors that a call writes move on.", -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

bool import_name(const char *from, const char *name, PyObject **to) {
    PyObject *m = PyImport_ImportModule(from);
    if (!m) return false;
    *to = PyObject_GetAttrString(m, name);
    Py_DECREF(m);
    return *to != nullptr;
}

}  // namespace

PyMODINIT_FUNC PyInit__binding() {
    if (!import_name("newton_schulz_quintic_amd._lib", "NSError", &g_ns_error) ||
        !import_name("newton_schulz_quintic_amd._lib", "_new_workspace", &g_new_workspace) ||
        !import_name("torch._C", "_cuda_getCurrentRawStream", &g_raw_stream) ||
        !import_name("torch.cuda", "current_device", &g_get_device))
        return nullptr;
    g_str_device = PyUnicode_InternFromString("device");
    g_str_cuda_stream = PyUnicode_InternFromString("cuda_stream");
    for (Signature *s : {&s_norm_rope, &s_norm_rope_backward, &s_moe_sort, &s_moe_dispatch, &s_moe_dispatch_backward,
                         &s_moe_combine, &s_moe_combine_backward, &s_distill, &s_distill_backward})
        for (int i = 0; i < s->count; ++i) {
            s->interned[i] = PyUnicode_InternFromString(s->names[i]);
            if (!s->interned[i]) return nullptr;
        }
    if (!g_str_device || !g_str_cuda_stream) return nullptr;
    return PyModule_Create(&module);
}
