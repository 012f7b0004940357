// The torch conveniences' checks and marshalling for the operators between a
// block's products, as a Python extension module.  A decode step makes these
// calls one after the other on rows of a few kilobytes; spelled out in Python,
// a call's checks take two to three times as long as the kernel it launches
// (append of one token: 7 us of 11; here 1 us).
//
// Every function checks types, shapes, strides and devices, forms the C call's
// arguments and makes it through the address it was given at setup(), so the
// module serves whatever build of the library the package has loaded.  It
// returns the call's status.  No C++ exception leaves it.
#define PY_SSIZE_T_CLEAN
#include <torch/csrc/autograd/python_variable.h>

#include <exception>
#include <stdexcept>

#include "q4_0.h"

namespace {

struct Entries {
    decltype(&q4_0_kv_append) append;
    decltype(&q4_0_attention) attention;
    decltype(&q4_0_residual_norm) norm;
    decltype(&q4_0_kv_append8) append8;
    decltype(&q4_0_attention8) attention8;
    decltype(&q4_0_kv_read8) read8;
    decltype(&q4_0_embed) embed;
    decltype(&q4_0_verify) verify;
    PyObject *raw_stream;  // device index -> handle of torch's current stream
} g;

// An error set for Python: the message's exception type with it.
struct Refused : std::runtime_error {
    PyObject *type;
    Refused(PyObject *t, const std::string &m) : std::runtime_error(m), type(t) {}
};
struct Raised {};  // Python's own error is set already

[[noreturn]] void bad_value(const std::string &m) { throw Refused(PyExc_ValueError, m); }
[[noreturn]] void bad_type(const std::string &m) { throw Refused(PyExc_TypeError, m); }

std::string text(at::IntArrayRef s) {
    std::string r = "(";
    for (size_t i = 0; i < s.size(); ++i) r += (i ? ", " : "") + std::to_string(s[i]);
    return r + ")";
}

const at::Tensor *tensor(PyObject *o, const char *name, bool optional = false) {
    if (optional && o == Py_None) return nullptr;
    if (!THPVariable_Check(o)) bad_type(std::string(name) + " must be a tensor");
    return &THPVariable_Unpack(o);
}

int dtype_code(const at::Tensor &t, const char *name) {
    if (t.scalar_type() == at::kFloat) return Q4_0_F32;
    if (t.scalar_type() == at::kHalf) return Q4_0_F16;
    bad_type(std::string(name) + " must be float32 or float16, not " +
             c10::toString(t.scalar_type()));
}

// The address of a dense tensor of one type and shape.
void *dense(const at::Tensor &t, const char *name, at::ScalarType type, at::IntArrayRef shape) {
    if (t.scalar_type() != type)
        bad_type(std::string(name) + " must be " + c10::toString(type) + ", not " +
                 c10::toString(t.scalar_type()));
    if (t.sizes() != shape)
        bad_value(std::string(name) + " must have shape " + text(shape) + ", not " +
                  text(t.sizes()));
    if (!t.is_contiguous()) bad_value(std::string(name) + " must be contiguous");
    return t.data_ptr();
}

// Row stride of [n, width] or [n, heads, dim] rows: dense within a row, any
// distance between rows.
int64_t rows(const at::Tensor &t, const char *name, int64_t n, int64_t width) {
    const auto s = t.sizes(), d = t.strides();
    int64_t w;
    bool ok;
    if (s.size() == 2) {
        w = s[1];
        ok = d[1] == 1 || w <= 1;
    } else if (s.size() == 3) {
        w = s[1] * s[2];
        ok = (d[2] == 1 || s[2] <= 1) && (d[1] == s[2] || s[1] <= 1);
    } else {
        bad_value(std::string(name) + " must have two or three dimensions");
    }
    if (!ok) bad_value(std::string(name) + "'s rows must be dense");
    if (s[0] != n || w != width)
        bad_value(std::string(name) + " has shape " + text(s) + ", which does not fit the call");
    return n > 1 ? d[0] : w;
}

// All of a call's tensors are on one GPU: its index.
template <size_t N> int device(const at::Tensor *const (&ts)[N]) {
    int dev = -1;
    for (const at::Tensor *t : ts) {
        if (!t) continue;
        if (!t->is_cuda()) bad_value("every tensor of the call must be on a GPU");
        const int d = t->get_device();
        if (dev >= 0 && d != dev) bad_value("the call's tensors are on different GPUs");
        dev = d;
    }
    return dev;
}

void *stream_of(PyObject *stream, int dev) {
    if (stream != Py_None) {
        void *p = PyLong_AsVoidPtr(stream);
        if (!p && PyErr_Occurred()) throw Raised();
        return p;
    }
    PyObject *arg = PyLong_FromLong(dev);
    if (!arg) throw Raised();
    PyObject *r = PyObject_CallOneArg(g.raw_stream, arg);
    Py_DECREF(arg);
    if (!r) throw Raised();
    void *p = PyLong_AsVoidPtr(r);
    Py_DECREF(r);
    if (!p && PyErr_Occurred()) throw Raised();
    return p;
}

int64_t integer(PyObject *o) {
    const int64_t v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred()) throw Raised();
    return v;
}

float number(PyObject *o) {
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred()) throw Raised();
    return (float)v;
}

template <typename F> PyObject *guarded(F body) {
    try {
        return body();
    } catch (const Raised &) {
    } catch (const Refused &e) {
        PyErr_SetString(e.type, e.what());
    } catch (const std::exception &e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
    }
    return nullptr;
}

void want(Py_ssize_t have, Py_ssize_t need) {
    if (have != need) bad_type("wrong number of arguments");
}

// ---- descriptors ------------------------------------------------------------
// Objects that hold a descriptor of q4_0.h and the tensors behind it.  What a
// tensor holds may be replaced at any time (Module.to gives its parameters new
// memory), so every use forms the descriptor again from the tensors.
struct Cache {
    PyObject_HEAD
    q4_0_kv_cache c;
    PyObject *k, *v;
};
struct Cache8 {
    PyObject_HEAD
    q4_0_kv_cache8 c;
    PyObject *k, *v, *k_scale, *v_scale;
};
struct Rotary {
    PyObject_HEAD
    q4_0_rotary r;
    int64_t norm_dim;  // of the weights; 0 without
    int device;        // of its tensors; -1 without any, -2 on no GPU
    PyObject *inv_freq, *q_norm, *k_norm;
};
PyTypeObject *g_cache_type, *g_cache8_type, *g_rotary_type;

q4_0_kv_cache read_cache(PyObject *ko, PyObject *vo) {
    const at::Tensor *k = tensor(ko, "k"), *v = tensor(vo, "v");
    const auto s = k->sizes();
    if (s.size() != 4) bad_value("k must be [pages, heads, page_size, dim], not " + text(s));
    // (a call divides by dim before the C entry sees it)
    for (const int64_t d : s)
        if (d < 1) bad_value("a cache has no empty dimension: " + text(s));
    void *kp = dense(*k, "k", at::kHalf, s), *vp = dense(*v, "v", at::kHalf, s);
    if (k->device() != v->device()) bad_value("k and v are on different devices");
    return {kp, vp, s[0], s[1], s[2], s[3]};
}

q4_0_kv_cache8 read_cache8(PyObject *ko, PyObject *vo, PyObject *kso, PyObject *vso) {
    const at::Tensor *k = tensor(ko, "k"), *v = tensor(vo, "v"), *ks = tensor(kso, "k_scale"),
                     *vs = tensor(vso, "v_scale");
    const auto s = k->sizes();
    if (s.size() != 4) bad_value("k must be [pages, heads, page_size, dim], not " + text(s));
    for (const int64_t d : s)
        if (d < 1) bad_value("a cache has no empty dimension: " + text(s));
    void *kp = dense(*k, "k", at::kChar, s), *vp = dense(*v, "v", at::kChar, s);
    void *ksp = dense(*ks, "k_scale", at::kFloat, s.slice(0, 3)),
         *vsp = dense(*vs, "v_scale", at::kFloat, s.slice(0, 3));
    if (k->device() != v->device() || k->device() != ks->device() || k->device() != vs->device())
        bad_value("the cache's tensors are on different devices");
    return {kp, vp, (float *)ksp, (float *)vsp, s[0], s[1], s[2], s[3]};
}

// inv_freq, q_norm and k_norm into `o`'s fields; the rest of it stays.
void read_rotary(Rotary &o, PyObject *inv_freq, PyObject *q_norm, PyObject *k_norm) {
    int dev = -1;
    const auto take = [&](PyObject *t, const char *name, int64_t &length) -> const float * {
        const at::Tensor *x = tensor(t, name, true);
        if (!x) return nullptr;
        if (x->dim() != 1) bad_value(std::string(name) + " must have one dimension");
        const float *p = (const float *)dense(*x, name, at::kFloat, x->sizes());
        const int d = x->is_cuda() ? x->get_device() : -2;
        if (dev != -1 && d != dev) bad_value("the rotation's tensors are on different devices");
        dev = d;
        length = x->size(0);
        return p;
    };
    int64_t half = 0, ql = 0, kl = 0;
    o.r.inv_freq = take(inv_freq, "inv_freq", half);
    o.r.rot_dim = 2 * half;
    o.r.q_norm = take(q_norm, "q_norm", ql);
    o.r.k_norm = take(k_norm, "k_norm", kl);
    if (ql && kl && ql != kl) bad_value("q_norm and k_norm have different lengths");
    o.norm_dim = ql ? ql : kl;
    o.device = dev;
}

void refresh(Cache &c) { c.c = read_cache(c.k, c.v); }
void refresh(Cache8 &c) { c.c = read_cache8(c.k, c.v, c.k_scale, c.v_scale); }
void refresh(Rotary &r) { read_rotary(r, r.inv_freq, r.q_norm, r.k_norm); }

template <typename T> void drop(PyObject *self, std::initializer_list<PyObject **> held) {
    for (PyObject **p : held) Py_CLEAR(*p);
    PyTypeObject *type = Py_TYPE(self);
    type->tp_free(self);
    Py_DECREF(type);
}
void cache_free(PyObject *self) {
    Cache *c = (Cache *)self;
    drop<Cache>(self, {&c->k, &c->v});
}
void cache8_free(PyObject *self) {
    Cache8 *c = (Cache8 *)self;
    drop<Cache8>(self, {&c->k, &c->v, &c->k_scale, &c->v_scale});
}
void rotary_free(PyObject *self) {
    Rotary *r = (Rotary *)self;
    drop<Rotary>(self, {&r->inv_freq, &r->q_norm, &r->k_norm});
}

template <typename C> PyObject *cache_address(PyObject *self, void *) {
    return guarded([&]() -> PyObject * {
        refresh(*(C *)self);
        return PyLong_FromVoidPtr(&((C *)self)->c);
    });
}
template <typename C> PyObject *cache_field(PyObject *self, void *at) {
    return guarded([&]() -> PyObject * {
        refresh(*(C *)self);
        return PyLong_FromLongLong(*(int64_t *)((char *)&((C *)self)->c + (size_t)at));
    });
}
PyObject *rotary_address(PyObject *self, void *) {
    return guarded([&]() -> PyObject * {
        refresh(*(Rotary *)self);
        return PyLong_FromVoidPtr(&((Rotary *)self)->r);
    });
}
#define CACHE_FIELDS(C, D)                                                                    \
    {                                                                                         \
        {"address", cache_address<C>, nullptr, "address of the descriptor", nullptr},         \
        {"pages", cache_field<C>, nullptr, nullptr, (void *)offsetof(D, pages)},              \
        {"heads", cache_field<C>, nullptr, nullptr, (void *)offsetof(D, heads)},              \
        {"page_size", cache_field<C>, nullptr, nullptr, (void *)offsetof(D, page_size)},      \
        {"dim", cache_field<C>, nullptr, nullptr, (void *)offsetof(D, dim)},                  \
        {nullptr, nullptr, nullptr, nullptr, nullptr}                                         \
    }
PyGetSetDef cache_fields[] = CACHE_FIELDS(Cache, q4_0_kv_cache);
PyGetSetDef cache8_fields[] = CACHE_FIELDS(Cache8, q4_0_kv_cache8);
PyGetSetDef rotary_fields[] = {
    {"address", rotary_address, nullptr, "address of the descriptor", nullptr},
    {nullptr, nullptr, nullptr, nullptr, nullptr}};
PyType_Slot cache_slots[] = {{Py_tp_dealloc, (void *)cache_free},
                             {Py_tp_getset, cache_fields},
                             {Py_tp_doc, (void *)"A paged cache's descriptor."},
                             {0, nullptr}};
PyType_Slot cache8_slots[] = {{Py_tp_dealloc, (void *)cache8_free},
                              {Py_tp_getset, cache8_fields},
                              {Py_tp_doc, (void *)"An 8-bit paged cache's descriptor."},
                              {0, nullptr}};
PyType_Slot rotary_slots[] = {{Py_tp_dealloc, (void *)rotary_free},
                              {Py_tp_getset, rotary_fields},
                              {Py_tp_doc, (void *)"A rotation's descriptor."},
                              {0, nullptr}};
// made by the functions below only: without them the fields would be empty
constexpr unsigned kTypeFlags = Py_TPFLAGS_DEFAULT | Py_TPFLAGS_DISALLOW_INSTANTIATION;
PyType_Spec cache_spec = {"gemm_q4_amd.KvCache", sizeof(Cache), 0, kTypeFlags, cache_slots};
PyType_Spec cache8_spec = {"gemm_q4_amd.KvCache8", sizeof(Cache8), 0, kTypeFlags, cache8_slots};
PyType_Spec rotary_spec = {"gemm_q4_amd.Rotary", sizeof(Rotary), 0, kTypeFlags, rotary_slots};

PyObject *held(PyObject *o) {
    Py_INCREF(o);
    return o;
}

PyObject *make_cache(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded([&]() -> PyObject * {
        want(n, 2);
        const q4_0_kv_cache read = read_cache(a[0], a[1]);
        Cache *c = (Cache *)g_cache_type->tp_alloc(g_cache_type, 0);
        if (!c) throw Raised();
        c->c = read;
        c->k = held(a[0]);
        c->v = held(a[1]);
        return (PyObject *)c;
    });
}

// k, v, k_scale, v_scale
PyObject *make_cache8(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded([&]() -> PyObject * {
        want(n, 4);
        const q4_0_kv_cache8 read = read_cache8(a[0], a[1], a[2], a[3]);
        Cache8 *c = (Cache8 *)g_cache8_type->tp_alloc(g_cache8_type, 0);
        if (!c) throw Raised();
        c->c = read;
        c->k = held(a[0]);
        c->v = held(a[1]);
        c->k_scale = held(a[2]);
        c->v_scale = held(a[3]);
        return (PyObject *)c;
    });
}

PyObject *is_cache8(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded([&]() -> PyObject * {
        want(n, 1);
        return PyBool_FromLong(PyObject_TypeCheck(a[0], g_cache8_type));
    });
}

// inv_freq, interleaved, amplitude, q_norm, k_norm, eps, weight_offset
PyObject *make_rotary(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded([&]() -> PyObject * {
        want(n, 7);
        Rotary read = {};
        read_rotary(read, a[0], a[3], a[4]);
        const int inter = PyObject_IsTrue(a[1]);
        if (inter < 0) throw Raised();
        read.r.interleaved = inter;
        read.r.amplitude = number(a[2]);
        read.r.eps = number(a[5]);
        read.r.weight_offset = number(a[6]);
        Rotary *o = (Rotary *)g_rotary_type->tp_alloc(g_rotary_type, 0);
        if (!o) throw Raised();
        o->r = read.r;
        o->norm_dim = read.norm_dim;
        o->device = read.device;
        o->inv_freq = held(a[0]);
        o->q_norm = held(a[3]);
        o->k_norm = held(a[4]);
        return (PyObject *)o;
    });
}

// A call's cache, of either kind.
struct AnyCache {
    const q4_0_kv_cache *c16;
    const q4_0_kv_cache8 *c8;
    int64_t heads, dim;
    const at::Tensor *k;
};
AnyCache cache_of(PyObject *o) {
    if (PyObject_TypeCheck(o, g_cache_type)) {
        Cache &c = *(Cache *)o;
        refresh(c);
        return {&c.c, nullptr, c.c.heads, c.c.dim, &THPVariable_Unpack(c.k)};
    }
    if (!PyObject_TypeCheck(o, g_cache8_type))
        bad_type("cache must come from kv_cache() or kv_cache8()");
    Cache8 &c = *(Cache8 *)o;
    refresh(c);
    return {nullptr, &c.c, c.c.heads, c.c.dim, &THPVariable_Unpack(c.k)};
}

// ---- calls ------------------------------------------------------------------
// cache, rot, q, k, v, positions, slots, q_out, stream
PyObject *call_append(PyObject *, PyObject *const *a, Py_ssize_t nargs) {
    return guarded([&]() -> PyObject * {
        want(nargs, 9);
        const AnyCache c = cache_of(a[0]);
        const Rotary *rot = nullptr;
        if (a[1] != Py_None) {
            if (!PyObject_TypeCheck(a[1], g_rotary_type)) bad_type("rot must come from rotary()");
            refresh(*(Rotary *)a[1]);
            rot = (const Rotary *)a[1];
        }
        const at::Tensor *q = tensor(a[2], "q", true), *k = tensor(a[3], "k"),
                         *v = tensor(a[4], "v"), *pos = tensor(a[5], "positions", true),
                         *slots = tensor(a[6], "slots"), *out = tensor(a[7], "q_out", !q);
        const int code = dtype_code(*k, "k");
        if (v->scalar_type() != k->scalar_type() || (q && q->scalar_type() != k->scalar_type()))
            bad_type("q, k and v must have one type");
        const int64_t n = k->dim() ? k->size(0) : 0, dim = c.dim, width = c.heads * dim;
        if (rot && rot->norm_dim && rot->norm_dim != dim)
            bad_value("norm weights of " + std::to_string(rot->norm_dim) +
                      " do not fit heads of " + std::to_string(dim));
        const int64_t ks = rows(*k, "k", n, width), vs = rows(*v, "v", n, width);
        int64_t qs = 0, heads = 0;
        int qcode = 0;
        if (q) {
            heads = q->dim() == 3 ? q->size(1) : (q->dim() == 2 ? q->size(1) / dim : 0);
            qs = rows(*q, "q", n, heads * dim);
            qcode = dtype_code(*out, "q_out");
            dense(*out, "q_out", out->scalar_type(), {n, heads, dim});
        }
        const void *pp = pos ? dense(*pos, "positions", at::kInt, {n}) : nullptr;
        const void *sp = dense(*slots, "slots", at::kLong, {n});
        const at::Tensor *all[] = {q,     k,  v, pos, slots, q ? out : nullptr, c.k};
        const int dev = device(all);
        if (rot && rot->device != -1 && rot->device != dev)
            bad_value("the rotation's tensors are not on the call's GPU");
        const auto call = [&](auto *entry, auto *cache) {
            return entry(
                cache, rot ? &rot->r : nullptr, q ? q->data_ptr() : nullptr, qs, k->data_ptr(),
                ks, v->data_ptr(), vs, code, q ? out->data_ptr() : nullptr, qcode, heads,
                (const int32_t *)pp, (const int64_t *)sp, n, stream_of(a[8], dev));
        };
        return PyLong_FromLong(c.c8 ? call(g.append8, c.c8) : call(g.append, c.c16));
    });
}

// cache, q, q_start, kv_len, table, window, sinks, scale, y, ws, stream
PyObject *call_attention(PyObject *, PyObject *const *a, Py_ssize_t nargs) {
    return guarded([&]() -> PyObject * {
        want(nargs, 11);
        const AnyCache c = cache_of(a[0]);
        const at::Tensor *q = tensor(a[1], "q"), *start = tensor(a[2], "q_start"),
                         *len = tensor(a[3], "kv_len"), *table = tensor(a[4], "table"),
                         *y = tensor(a[8], "y"), *ws = tensor(a[9], "ws", true);
        if (q->dim() != 3 || q->size(2) != c.dim)
            bad_value("q must be [n, heads, " + std::to_string(c.dim) + "], not " +
                      text(q->sizes()));
        const int code = dtype_code(*q, "q");
        const int64_t n = q->size(0), heads = q->size(1);
        const int64_t qs = rows(*q, "q", n, heads * c.dim);
        const int64_t batch = len->dim() ? len->size(0) : 0;
        const int64_t width = table->dim() == 2 ? table->size(1) : 0;
        const void *sp = dense(*start, "q_start", at::kInt, {batch + 1});
        const void *lp = dense(*len, "kv_len", at::kInt, {batch});
        const void *tp = dense(*table, "table", at::kInt, {batch, width});
        void *yp = dense(*y, "y", q->scalar_type(), {n, heads, c.dim});
        if (ws && !ws->is_contiguous()) bad_value("ws must be contiguous");
        const at::Tensor *all[] = {q, start, len, table, y, ws, c.k};
        const int dev = device(all);
        const auto call = [&](auto *entry, auto *cache) {
            return entry(cache, q->data_ptr(), qs, code, heads, yp, n, (const int32_t *)sp,
                         (const int32_t *)lp, (const int32_t *)tp, width, batch, integer(a[5]),
                         integer(a[6]), number(a[7]), ws ? ws->data_ptr() : nullptr,
                         ws ? ws->nbytes() : 0, stream_of(a[10], dev));
        };
        return PyLong_FromLong(c.c8 ? call(g.attention8, c.c8) : call(g.attention, c.c16));
    });
}

// h, b, pre, post, gate, alpha, eps, weight_offset, h_out, y, stream
PyObject *call_norm(PyObject *, PyObject *const *a, Py_ssize_t nargs) {
    return guarded([&]() -> PyObject * {
        want(nargs, 11);
        const at::Tensor *h = tensor(a[0], "h"), *b = tensor(a[1], "b", true),
                         *pre = tensor(a[2], "pre", true), *post = tensor(a[3], "post", true),
                         *gate = tensor(a[4], "gate", true), *out = tensor(a[8], "h_out", !b),
                         *y = tensor(a[9], "y", !pre);
        if (h->scalar_type() != at::kFloat)
            bad_type(std::string("h must be float32, not ") + c10::toString(h->scalar_type()));
        if (h->dim() != 2) bad_value("h must be [n, dim], not " + text(h->sizes()));
        const int64_t n = h->size(0), dim = h->size(1), hs = rows(*h, "h", n, dim);
        int64_t bs = 0, ys = 0, grow = 0, gcol = 0;
        int bcode = 0, ycode = 0;
        if (b) {
            bs = rows(*b, "b", n, dim);
            bcode = dtype_code(*b, "b");
            if (out->scalar_type() != at::kFloat) bad_type("h_out must be float32");
            if (rows(*out, "h_out", n, dim) != hs) bad_value("h_out must have h's row stride");
            if (gate) {
                if (gate->scalar_type() != at::kFloat) bad_type("gate must be float32");
                if (gate->dim() != 2 || (gate->size(0) != 1 && gate->size(0) != n) ||
                    (gate->size(1) != 1 && gate->size(1) != dim))
                    bad_value("gate must be [n, dim], [n, 1] or [1, dim], not " +
                              text(gate->sizes()));
                grow = gate->size(0) > 1 ? gate->stride(0) : 0;
                gcol = gate->size(1) > 1 ? gate->stride(1) : 0;
            }
        }
        if (pre) {
            dense(*pre, "pre", at::kFloat, {dim});
            ys = rows(*y, "y", n, dim);
            ycode = dtype_code(*y, "y");
        }
        if (post) dense(*post, "post", at::kFloat, {dim});
        const at::Tensor *all[] = {h, b, pre, post, gate, b ? out : nullptr, pre ? y : nullptr};
        const int dev = device(all);
        const auto f = [](const at::Tensor *t) { return t ? (float *)t->data_ptr() : nullptr; };
        return PyLong_FromLong(g.norm(
            b ? b->data_ptr() : nullptr, bcode, bs, f(post), f(gate), grow, gcol, number(a[5]),
            f(h), b ? f(out) : nullptr, hs, f(pre), number(a[7]), number(a[6]),
            pre ? y->data_ptr() : nullptr, ycode, ys, n, dim, stream_of(a[10], dev)));
    });
}

// cache, slots, k, v, stream
PyObject *call_read(PyObject *, PyObject *const *a, Py_ssize_t nargs) {
    return guarded([&]() -> PyObject * {
        want(nargs, 5);
        const AnyCache c = cache_of(a[0]);
        if (!c.c8) bad_type("cache must come from kv_cache8()");
        const at::Tensor *slots = tensor(a[1], "slots"), *k = tensor(a[2], "k"),
                         *v = tensor(a[3], "v");
        const int64_t n = slots->dim() ? slots->size(0) : 0;
        const void *sp = dense(*slots, "slots", at::kLong, {n});
        const int code = dtype_code(*k, "k");
        void *kp = dense(*k, "k", k->scalar_type(), {n, c.heads, c.dim});
        void *vp = dense(*v, "v", k->scalar_type(), {n, c.heads, c.dim});
        const at::Tensor *all[] = {slots, k, v, c.k};
        const int dev = device(all);
        return PyLong_FromLong(
            g.read8(c.c8, (const int64_t *)sp, n, kp, vp, code, stream_of(a[4], dev)));
    });
}

// packed, tokens, out, in, scale, pre, eps, weight_offset, h, y, stream
PyObject *call_embed(PyObject *, PyObject *const *a, Py_ssize_t nargs) {
    return guarded([&]() -> PyObject * {
        want(nargs, 11);
        const at::Tensor *packed = tensor(a[0], "packed"), *tokens = tensor(a[1], "tokens"),
                         *pre = tensor(a[5], "pre", true), *h = tensor(a[8], "h"),
                         *y = tensor(a[9], "y", !pre);
        const int64_t out = integer(a[2]), in = integer(a[3]);
        const int64_t n = tokens->dim() ? tokens->size(0) : 0;
        const void *tp = dense(*tokens, "tokens", at::kInt, {n});
        const int64_t rows = (out + 15) / 16 * 16, groups = (in / 32 + 3) / 4;
        if (packed->scalar_type() != at::kByte || !packed->is_contiguous())
            bad_type("packed must be dense bytes");
        // (sizes the C entry refuses are left to it)
        if (out > 0 && in > 0 && out <= Q4_0_MAX_OUT && in <= Q4_0_MAX_IN &&
            packed->numel() < rows * groups * 72)
            bad_value("packed holds " + std::to_string(packed->numel()) + " bytes, fewer than " +
                      std::to_string(rows * groups * 72));
        float *hp = (float *)dense(*h, "h", at::kFloat, {n, in}), *wp = nullptr;
        void *yp = nullptr;
        int code = 0;
        if (pre) {
            wp = (float *)dense(*pre, "pre", at::kFloat, {in});
            code = dtype_code(*y, "y");
            yp = dense(*y, "y", y->scalar_type(), {n, in});
        }
        const at::Tensor *all[] = {packed, tokens, h, pre, pre ? y : nullptr};
        const int dev = device(all);
        return PyLong_FromLong(g.embed(packed->data_ptr(), (const int32_t *)tp, n, out, in,
                                       number(a[4]), hp, wp, number(a[7]), number(a[6]), yp, code,
                                       stream_of(a[10], dev)));
    });
}

// logits, tokens, q_start, uniform, drafted, temperature, accepted, following, ws, stream
PyObject *call_verify(PyObject *, PyObject *const *a, Py_ssize_t nargs) {
    return guarded([&]() -> PyObject * {
        want(nargs, 10);
        const at::Tensor *logits = tensor(a[0], "logits"), *tokens = tensor(a[1], "tokens"),
                         *start = tensor(a[2], "q_start"), *uni = tensor(a[3], "uniform"),
                         *drafted = tensor(a[4], "draft_logits", true),
                         *heat = tensor(a[5], "temperature", true),
                         *acc = tensor(a[6], "accepted"), *next = tensor(a[7], "following"),
                         *ws = tensor(a[8], "ws", true);
        if (logits->dim() != 2) bad_value("logits must be [n, vocab], not " + text(logits->sizes()));
        const int code = dtype_code(*logits, "logits");
        const int64_t n = logits->size(0), vocab = logits->size(1);
        const int64_t stride = rows(*logits, "logits", n, vocab);
        int64_t dstride = 0;
        if (drafted) {
            if (drafted->scalar_type() != logits->scalar_type())
                bad_type("logits and draft_logits must have one type");
            dstride = rows(*drafted, "draft_logits", n, vocab);
        }
        const int64_t batch = start->dim() && start->size(0) ? start->size(0) - 1 : 0;
        const void *sp = dense(*start, "q_start", at::kInt, {batch + 1});
        const void *tp = dense(*tokens, "tokens", at::kInt, {n});
        const void *up = dense(*uni, "uniform", at::kFloat, {n, 2});
        const void *hp = heat ? dense(*heat, "temperature", at::kFloat, {batch}) : nullptr;
        void *ap = dense(*acc, "accepted", at::kInt, {batch});
        void *np = dense(*next, "following", at::kInt, {batch});
        if (ws && !ws->is_contiguous()) bad_value("ws must be contiguous");
        const at::Tensor *all[] = {logits, tokens, start, uni, drafted, heat, acc, next, ws};
        const int dev = device(all);
        return PyLong_FromLong(g.verify(
            logits->data_ptr(), stride, drafted ? drafted->data_ptr() : nullptr, dstride, code,
            vocab, (const int32_t *)tp, (const int32_t *)sp, n, batch, (const float *)hp,
            (const float *)up, (int32_t *)ap, (int32_t *)np, ws ? ws->data_ptr() : nullptr,
            ws ? ws->nbytes() : 0, stream_of(a[9], dev)));
    });
}

// Addresses of the entries in the order of Entries, and the function that gives a
// device's current stream.
PyObject *setup(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded([&]() -> PyObject * {
        want(n, 9);
        void *entries[8];
        for (int i = 0; i < 8; ++i) entries[i] = PyLong_AsVoidPtr(a[i]);
        if (PyErr_Occurred()) throw Raised();
        g = {(decltype(g.append))entries[0],  (decltype(g.attention))entries[1],
             (decltype(g.norm))entries[2],    (decltype(g.append8))entries[3],
             (decltype(g.attention8))entries[4], (decltype(g.read8))entries[5],
             (decltype(g.embed))entries[6],   (decltype(g.verify))entries[7],
             held(a[8])};
        return held(Py_None);
    });
}

#define FAST(name, fn) {name, (PyCFunction)(void (*)(void))fn, METH_FASTCALL, nullptr}
PyMethodDef methods[] = {FAST("setup", setup),
                         FAST("kv_cache", make_cache),
                         FAST("kv_cache8", make_cache8),
                         FAST("is_cache8", is_cache8),
                         FAST("rotary", make_rotary),
                         FAST("kv_append", call_append),
                         FAST("attention", call_attention),
                         FAST("residual_norm", call_norm),
                         FAST("kv_read", call_read),
                         FAST("embed", call_embed),
                         FAST("verify", call_verify),
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_bind",
                      "Checks and marshalling of the block operators' torch conveniences.", -1,
                      methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__bind(void) {
    g_cache_type = (PyTypeObject *)PyType_FromSpec(&cache_spec);
    g_cache8_type = (PyTypeObject *)PyType_FromSpec(&cache8_spec);
    g_rotary_type = (PyTypeObject *)PyType_FromSpec(&rotary_spec);
    if (!g_cache_type || !g_cache8_type || !g_rotary_type) return nullptr;
    PyObject *m = PyModule_Create(&module);
    if (m && PyModule_AddStringConstant(m, "torch_version", Q4_0_TORCH_VERSION) < 0) Py_CLEAR(m);
    return m;
}
