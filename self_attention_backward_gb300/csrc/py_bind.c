/* py_bind.c -- argument marshalling of the window attention family for Python.
 *
 * The same work as binding.py's ctypes calls (tensor attributes to pointers, sizes
 * and strides, their checks, the C entry point), in C: the calls of a decoding step
 * take a few microseconds on the GPU, and written in Python their marshalling took
 * more than twice that.  No arithmetic and no CUDA here; the entry points' addresses
 * come from binding.py, which loads the CUDA library.
 *
 * Functions return their outputs (None in the place of an output argument: a new
 * tensor like its input), or the entry point's status if it is not 0, or OTHER_DEVICE
 * when the tensors' device is not the current one (binding.py switches and calls
 * again), OTHER_STREAM when a kept workspace is not of the current stream; arguments that do not fit together raise ValueError.
 */
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include "psa_attn.h"

#define OTHER_DEVICE 1000
#define OTHER_STREAM 1001

static PyObject *s_data_ptr, *s_stride, *s_shape, *s_dtype, *s_get_device;   /* attribute names */
static PyObject *s_device, *kw_make;                                         /* a tensor's device, ("dtype", "device") */
static PyObject *t_f32, *t_bf16, *t_i32, *t_u8, *f_device, *f_stream, *f_like, *f_empty;   /* torch's own */

static int (*p_rope)(const psa_rope_plan*, const psa_attn_view*, const psa_attn_view*, int, const psa_attn_view*,
                     const psa_attn_view*, int, int, int, const int*, long long, long long, int, int, void*);
static int (*p_fwd)(const psa_win_shape*, const psa_attn_view*, const psa_attn_view*, const psa_attn_view*,
                    const psa_attn_view*, float*, const int*, const int*, int, void*);
static int (*p_bwd)(const psa_win_shape*, const psa_attn_view*, const psa_attn_view*, const psa_attn_view*,
                    const psa_attn_view*, const float*, const psa_attn_view*, const psa_attn_view*, const psa_attn_view*,
                    const psa_attn_view*, const int*, const int*, void*, size_t, int, void*);
static size_t (*p_bwd_bytes)(const psa_win_shape*);
static int (*p_append)(const psa_win_cache*, const psa_attn_view*, const psa_attn_view*, int, const int*, const int*,
                       const psa_rope_plan*, const int*, long long, long long, void*);
static int (*p_decode)(const psa_win_cache*, const psa_attn_view*, const psa_attn_view*, float*, int, const int*, float,
                       void*, size_t, void*);
static int (*p_store)(const psa_win_cache*, const psa_win_scales*, const psa_attn_view*, const psa_attn_view*, int, const int*,
                      long long, int, const int*, const int*, const psa_rope_plan*, const int*, long long, long long, int,
                      void*);
static int (*p_read)(const psa_win_cache*, const psa_win_scales*, const psa_attn_view*, const psa_attn_view*, int, const int*,
                     const int*, int, void*);
static int (*p_decode_any)(const psa_win_cache*, const psa_win_scales*, const psa_attn_view*, const psa_attn_view*, float*, int,
                           const int*, float, void*, size_t, int, void*);
static int (*p_tree)(const psa_win_cache*, const psa_win_scales*, const psa_attn_view*, const psa_attn_view*,
                     const psa_attn_view*, const psa_attn_view*, float*, int, int, const int*, long long, const int*,
                     const int*, float, void*, size_t, int, int, void*);
static size_t (*p_decode_any_bytes)(const psa_win_cache*, int, int);
static size_t (*p_tree_bytes)(const psa_win_cache*, int, int, int);

enum { T_F32 = PSA_F32, T_BF16 = PSA_BF16, T_I32 = 100, T_OTHER = 101 };

/* What a torch tensor says of itself. */
typedef struct {
    const char* name;
    void* p;
    int nd, dtype, dev;
    long long n[4], s[4];
} Ten;

static int bad(const char* fmt, const char* a, const char* b) {
    PyErr_Format(PyExc_ValueError, fmt, a, b);
    return 0;
}

static int ints(PyObject* t, int nd, long long* to) {
    for (int i = 0; i < nd; ++i) {
        to[i] = PyLong_AsLongLong(PyTuple_GET_ITEM(t, i));
        if (to[i] == -1 && PyErr_Occurred()) return 0;
    }
    return 1;
}
static int as_int(PyObject* o, long long* to) {
    if (!o) return 0;
    *to = PyLong_AsLongLong(o);
    Py_DECREF(o);
    return !(*to == -1 && PyErr_Occurred());
}

/* Reads tensor o of nd dimensions (0: any up to 4). */
static int get(PyObject* o, const char* name, int nd, Ten* t) {
    long long v;
    t->name = name;
    PyObject* shape = PyObject_GetAttr(o, s_shape);
    if (!shape) return 0;
    int ok = PyTuple_Check(shape) && PyTuple_GET_SIZE(shape) <= 4;
    if (ok) {
        t->nd = (int)PyTuple_GET_SIZE(shape);
        ok = ints(shape, t->nd, t->n);
    } else {
        bad("%s has too many dimensions%s", name, "");
    }
    Py_DECREF(shape);
    if (!ok) return 0;
    if (nd && t->nd != nd) {
        PyErr_Format(PyExc_ValueError, "%s has to have %d dimensions, not %d", name, nd, t->nd);
        return 0;
    }
    PyObject* stride = PyObject_CallMethodNoArgs(o, s_stride);
    if (!stride) return 0;
    ok = PyTuple_Check(stride) && PyTuple_GET_SIZE(stride) == t->nd && ints(stride, t->nd, t->s);
    Py_DECREF(stride);
    if (!ok) return PyErr_Occurred() ? 0 : bad("%s has no strides%s", name, "");
    if (!as_int(PyObject_CallMethodNoArgs(o, s_get_device), &v)) return 0;
    t->dev = (int)v;
    if (v < 0) return bad("tensors have to be on a CUDA device: %s is not%s", name, "");
    PyObject* p = PyObject_CallMethodNoArgs(o, s_data_ptr);
    if (!p) return 0;
    t->p = (void*)(uintptr_t)PyLong_AsUnsignedLongLong(p);
    Py_DECREF(p);
    if (PyErr_Occurred()) return 0;
    PyObject* dt = PyObject_GetAttr(o, s_dtype);
    if (!dt) return 0;
    t->dtype = dt == t_bf16 ? T_BF16 : dt == t_f32 ? T_F32 : dt == t_i32 ? T_I32 : T_OTHER;
    Py_DECREF(dt);
    return 1;
}
/* A floating tensor; with `like`, of its dtype and device. */
static int get_data(PyObject* o, const char* name, int nd, const Ten* like, Ten* t) {
    if (!get(o, name, nd, t)) return 0;
    if (t->dtype != T_F32 && t->dtype != T_BF16) return bad("%s has to be fp32 or bf16%s", name, "");
    if (like && (t->dtype != like->dtype || t->dev != like->dev))
        return bad("%s and %s differ in dtype or device", like->name, name);
    return 1;
}
static int same_shape(const Ten* a, const Ten* b) {
    if (a->nd != b->nd) return bad("%s has to be shaped like %s", b->name, a->name);
    for (int i = 0; i < a->nd; ++i)
        if (a->n[i] != b->n[i]) return bad("%s has to be shaped like %s", b->name, a->name);
    return 1;
}
static int dense(const Ten* t) {
    long long want = 1;
    for (int i = 0; i < t->nd; ++i)
        if (t->n[i] == 0) return 1;
    for (int i = t->nd - 1; i >= 0; --i) {
        if (t->n[i] != 1 && t->s[i] != want) return 0;
        want *= t->n[i];
    }
    return 1;
}
/* int32 [n], contiguous, or None (NULL). */
static int get_lens(PyObject* o, const char* name, const Ten* like, long long n, const int** to) {
    Ten t;
    *to = NULL;
    if (o == Py_None) return 1;
    if (!get(o, name, 0, &t)) return 0;
    if (t.dtype != T_I32 || t.nd != 1 || t.n[0] != n || t.dev != like->dev || !dense(&t))
        return bad("%s has to be a contiguous int32 tensor [B] on the device of %s", name, like->name);
    *to = (const int*)t.p;
    return 1;
}
/* fp32, contiguous, of the first `nd` dimensions of q. */
static int get_lse(PyObject* o, const Ten* q, int nd, float** to) {
    Ten t;
    if (!get(o, "lse", 0, &t)) return 0;
    int ok = t.dtype == T_F32 && t.nd == nd && t.dev == q->dev && dense(&t);
    for (int i = 0; ok && i < nd; ++i) ok = t.n[i] == q->n[i];
    if (!ok) return bad("lse has to be a contiguous fp32 tensor [B, heads%s] on the device of %s", nd == 3 ? ", Nq" : "", q->name);
    *to = (float*)t.p;
    return 1;
}
/* int32 positions [axes, B, N], [axes, 1, N] or [axes, N]. */
static int get_pos(PyObject* o, const Ten* like, long long axes, long long B, long long N, const int** p, long long* sa,
                   long long* sb) {
    Ten t;
    if (!get(o, "pos", 0, &t)) return 0;
    int ok = t.dtype == T_I32 && t.dev == like->dev && (t.nd == 2 || t.nd == 3) && t.n[0] == axes && t.n[t.nd - 1] == N &&
             (t.nd == 2 || t.n[1] == B || t.n[1] == 1) && (N <= 1 || t.s[t.nd - 1] == 1);
    if (!ok) {
        PyErr_Format(PyExc_ValueError,
                     "pos has to be an int32 tensor [%lld, %lld, %lld] or [%lld, %lld], contiguous along the rows, on the "
                     "device of %s", axes, B, N, axes, N, like->name);
        return 0;
    }
    *p = (const int*)t.p;
    *sa = t.s[0];
    *sb = t.nd == 3 && t.n[1] > 1 ? t.s[1] : 0;
    return 1;
}

/* An int32 table [B, n], [1, n] or [n] (one row for all sequences), contiguous along its rows; *n is given, or
 * -1 and found.  None: NULL. */
static int get_table(PyObject* o, const char* name, const Ten* like, long long B, long long* n, const int** p, long long* stride) {
    Ten t;
    *p = NULL;
    *stride = 0;
    if (o == Py_None) return 1;
    if (!get(o, name, 0, &t)) return 0;
    const long long cols = t.nd ? t.n[t.nd - 1] : 0;
    const int ok = t.dtype == T_I32 && t.dev == like->dev && (t.nd == 1 || (t.nd == 2 && (t.n[0] == B || t.n[0] == 1))) &&
                   (*n < 0 || cols == *n) && (cols <= 1 || t.s[t.nd - 1] == 1);
    if (!ok)
        return bad("%s has to be an int32 tensor [B, n] or [n], contiguous along its rows, on the device of %s", name, like->name);
    *n = cols;
    *p = (const int*)t.p;
    if (t.nd == 2 && t.n[0] > 1) *stride = t.s[0];
    return 1;
}

/* A new tensor like `o`, whose attributes are `t`. */
static PyObject* make_like(PyObject* o, const char* name, const Ten* t, Ten* to) {
    PyObject* r = PyObject_CallOneArg(f_like, o);
    if (!r) return NULL;
    *to = *t;
    to->name = name;
    int ok = 1;
    if (!dense(t)) {                                 /* else its strides are t's */
        PyObject* stride = PyObject_CallMethodNoArgs(r, s_stride);
        ok = stride && PyTuple_Check(stride) && PyTuple_GET_SIZE(stride) == t->nd && ints(stride, t->nd, to->s);
        Py_XDECREF(stride);
    }
    PyObject* p = ok ? PyObject_CallMethodNoArgs(r, s_data_ptr) : NULL;
    if (p) {
        to->p = (void*)(uintptr_t)PyLong_AsUnsignedLongLong(p);
        Py_DECREF(p);
    }
    if (!p || PyErr_Occurred()) {
        if (!PyErr_Occurred()) bad("%s cannot be made%s", name, "");
        Py_DECREF(r);
        return NULL;
    }
    return r;
}
/* A new contiguous tensor on the device of tensor `on`, its size given as a tuple or a number (stolen). */
static PyObject* make(PyObject* size, PyObject* dtype, PyObject* on, void** data) {
    if (!size) return NULL;
    PyObject *dev = PyObject_GetAttr(on, s_device), *r = NULL;
    if (dev) {
        PyObject* args[3] = {size, dtype, dev};
        r = PyObject_Vectorcall(f_empty, args, 1, kw_make);
        Py_DECREF(dev);
    }
    Py_DECREF(size);
    PyObject* p = r ? PyObject_CallMethodNoArgs(r, s_data_ptr) : NULL;
    if (p) {
        *data = (void*)(uintptr_t)PyLong_AsUnsignedLongLong(p);
        Py_DECREF(p);
    }
    if (!p || PyErr_Occurred()) {
        Py_XDECREF(r);
        return NULL;
    }
    return r;
}
/* The output argument `a`, shaped like `like` (attributes t), or a new one: a new reference. */
static PyObject* output(PyObject* a, const char* name, int nd, PyObject* like, const Ten* t, Ten* to) {
    if (a == Py_None) return make_like(like, name, t, to);
    if (!get_data(a, name, nd, t, to) || !same_shape(t, to)) return NULL;
    return Py_NewRef(a);
}

static psa_attn_view view(const Ten* t) {
    psa_attn_view v = {t->p, t->s[0], t->s[1], t->s[2], t->s[3]};
    return v;
}
static int fits(const Ten* t, int from, int to) {   /* sizes that an int holds */
    for (int i = from; i < to; ++i)
        if (t->n[i] > 0x7fffffffll) return bad("%s is too large%s", t->name, "");
    return 1;
}

/* rc = the entry point's status, without the interpreter's lock: a launch may have to wait
 * for room in the stream's queue. */
#define CALL(expr)              \
    do {                        \
        Py_BEGIN_ALLOW_THREADS  \
        rc = (int)(expr);       \
        Py_END_ALLOW_THREADS    \
    } while (0)

/* What a function returns: its n outputs (stolen; NULL in one's place after an error), or the
 * status. */
static PyObject* result(int rc, int n, PyObject* const* out) {
    int ok = rc == 0;
    for (int i = 0; i < n; ++i) ok = ok && out[i];
    PyObject* r = NULL;
    if (ok && n == 1) return out[0];
    if (ok) r = n == 2 ? PyTuple_Pack(2, out[0], out[1]) : PyTuple_Pack(3, out[0], out[1], out[2]);
    else if (!PyErr_Occurred()) r = PyLong_FromLong(rc);
    for (int i = 0; i < n; ++i) Py_XDECREF(out[i]);
    return r;
}

/* result() of one output, which an error since it was made takes back. */
static PyObject* call_result(int rc, PyObject** out) {
    if (PyErr_Occurred()) Py_CLEAR(out[0]);
    return result(rc, 1, out);
}

/* 1: *stream is the device's current stream; 0: an error; -1: another device is current. */
static int on_device(int dev, void** stream) {
    long long cur, st;
    if (!as_int(PyObject_CallNoArgs(f_device), &cur)) return 0;
    if (cur != dev) return -1;
    PyObject* d = PyLong_FromLong(dev);
    if (!d) return 0;
    PyObject* r = PyObject_CallOneArg(f_stream, d);
    Py_DECREF(d);
    if (!as_int(r, &st)) return 0;
    *stream = (void*)(intptr_t)st;
    return 1;
}
#define ON_DEVICE(dev, stream)                       \
    do {                                             \
        const int on = on_device(dev, &(stream));    \
        if (on == 0) return NULL;                    \
        if (on < 0) return PyLong_FromLong(OTHER_DEVICE); \
    } while (0)

/* init(f32, bf16, i32, u8, current device, current raw stream, empty_like, empty, addresses of the twelve entry points) */
static PyObject* init(PyObject* self, PyObject* a) {
    unsigned long long f[12];
    if (!PyArg_ParseTuple(a, "OOOOOOOOKKKKKKKKKKKK", &t_f32, &t_bf16, &t_i32, &t_u8, &f_device, &f_stream, &f_like, &f_empty, &f[0],
                          &f[1], &f[2], &f[3], &f[4], &f[5], &f[6], &f[7], &f[8], &f[9], &f[10], &f[11]))
        return NULL;
    Py_INCREF(t_f32), Py_INCREF(t_bf16), Py_INCREF(t_i32), Py_INCREF(t_u8);
    Py_INCREF(f_device), Py_INCREF(f_stream), Py_INCREF(f_like), Py_INCREF(f_empty);
    *(void**)&p_rope = (void*)(uintptr_t)f[0];
    *(void**)&p_fwd = (void*)(uintptr_t)f[1];
    *(void**)&p_bwd = (void*)(uintptr_t)f[2];
    *(void**)&p_bwd_bytes = (void*)(uintptr_t)f[3];
    *(void**)&p_append = (void*)(uintptr_t)f[4];
    *(void**)&p_decode = (void*)(uintptr_t)f[5];
    *(void**)&p_store = (void*)(uintptr_t)f[6];
    *(void**)&p_read = (void*)(uintptr_t)f[7];
    *(void**)&p_decode_any = (void*)(uintptr_t)f[8];
    *(void**)&p_tree = (void*)(uintptr_t)f[9];
    *(void**)&p_decode_any_bytes = (void*)(uintptr_t)f[10];
    *(void**)&p_tree_bytes = (void*)(uintptr_t)f[11];
    Py_RETURN_NONE;
}

/* rope(plan address, q, pos, k or None, inverse, out or None, out_k or None): out, or out and out_k */
static PyObject* rope(PyObject* self, PyObject* const* a, Py_ssize_t na) {
    if (na != 7) return PyErr_Format(PyExc_TypeError, "rope takes 7 arguments");
    const psa_rope_plan* plan = (const psa_rope_plan*)PyLong_AsVoidPtr(a[0]);
    if (!plan) return PyErr_Occurred() ? NULL : PyErr_Format(PyExc_ValueError, "no plan");
    Ten q, o, k, ok;
    const int two = a[3] != Py_None;
    const int* pos;
    long long sa, sb;
    if (!get_data(a[1], "q", 4, NULL, &q) || !fits(&q, 0, 3)) return NULL;
    if (q.n[3] != plan->head_dim) return bad("q's features are not the plan's%s%s", "", ""), NULL;
    if (!get_pos(a[2], &q, plan->n_axes, q.n[0], q.n[2], &pos, &sa, &sb)) return NULL;
    if (two) {
        if (!get_data(a[3], "k", 4, &q, &k) || !fits(&k, 1, 2)) return NULL;
        if (k.n[0] != q.n[0] || k.n[2] != q.n[2] || k.n[3] != q.n[3]) return bad("k and q do not fit together%s%s", "", ""), NULL;
    }
    const int inverse = PyObject_IsTrue(a[4]);
    if (inverse < 0) return NULL;
    void* st;
    ON_DEVICE(q.dev, st);
    int rc = 0;
    PyObject* out[2] = {output(a[5], "out", 4, a[1], &q, &o), NULL};
    if (out[0] && two) out[1] = output(a[6], "out_k", 4, a[3], &k, &ok);
    if (out[0] && (!two || out[1])) {
        const psa_attn_view vq = view(&q), vo = view(&o);
        psa_attn_view vk, vok;
        if (two) vk = view(&k), vok = view(&ok);
        CALL(p_rope(plan, &vq, &vo, (int)q.n[1], two ? &vk : NULL, two ? &vok : NULL, two ? (int)k.n[1] : 0, (int)q.n[0],
                    (int)q.n[2], pos, sa, sb, inverse, q.dtype, st));
    }
    return result(rc, 1 + two, out);
}

/* q, k, v and the mask to a problem. */
static int get_shape(PyObject* const* a, Ten* q, Ten* k, Ten* v, psa_win_shape* s) {
    if (!get_data(a[0], "q", 4, NULL, q) || !get_data(a[1], "k", 4, q, k) || !get_data(a[2], "v", 4, q, v) ||
        !same_shape(k, v) || !fits(q, 0, 4) || !fits(k, 1, 3))
        return 0;
    if (k->n[0] != q->n[0] || k->n[3] != q->n[3]) return bad("k, v and q do not fit together%s%s", "", "");
    const double scale = PyFloat_AsDouble(a[3]);
    if (PyErr_Occurred()) return 0;
    int overflow;
    const long long w = PyLong_AsLongLongAndOverflow(a[4], &overflow), n = PyLong_AsLongLong(a[5]);
    if (PyErr_Occurred()) return 0;
    s->B = (int)q->n[0], s->q_heads = (int)q->n[1], s->kv_heads = (int)k->n[1], s->Nq = (int)q->n[2], s->Nk = (int)k->n[2];
    s->head_dim = (int)q->n[3];
    /* what an int does not hold is larger than every sequence */
    s->window = overflow > 0 || w > 0x7fffffffll ? 0x7fffffff : overflow < 0 || w < 0 ? -1 : (int)w;
    s->sinks = n > 0x7fffffffll ? 0x7fffffff : n < 0 ? -1 : (int)n;
    s->scale = (float)scale;
    s->dtype = q->dtype;
    return 1;
}

/* win_fwd(q, k, v, scale, window, sinks, q_lens, kv_lens, out or None, lse or None, algo): out, lse */
static PyObject* win_fwd(PyObject* self, PyObject* const* a, Py_ssize_t na) {
    if (na != 11) return PyErr_Format(PyExc_TypeError, "win_fwd takes 11 arguments");
    Ten q, k, v, o;
    psa_win_shape s;
    const int *ql, *kl;
    float* lse = NULL;
    if (!get_shape(a, &q, &k, &v, &s) || !get_lens(a[6], "q_lens", &q, q.n[0], &ql) ||
        !get_lens(a[7], "kv_lens", &q, q.n[0], &kl) || (a[9] != Py_None && !get_lse(a[9], &q, 3, &lse)))
        return NULL;
    const long algo = PyLong_AsLong(a[10]);
    if (PyErr_Occurred()) return NULL;
    void* st;
    ON_DEVICE(q.dev, st);
    int rc = 0;
    PyObject* out[2] = {output(a[8], "out", 4, a[0], &q, &o), NULL};
    if (out[0])
        out[1] = a[9] != Py_None ? Py_NewRef(a[9]) : make(Py_BuildValue("(LLL)", q.n[0], q.n[1], q.n[2]), t_f32, a[0], (void**)&lse);
    if (out[1]) {
        const psa_attn_view vq = view(&q), vk = view(&k), vv = view(&v), vo = view(&o);
        CALL(p_fwd(&s, &vq, &vk, &vv, &vo, lse, ql, kl, (int)algo, st));
    }
    return result(rc, 2, out);
}

/* win_bwd_bytes(q, k, v, scale, window, sinks): workspace bytes */
static PyObject* win_bwd_bytes(PyObject* self, PyObject* const* a, Py_ssize_t na) {
    if (na != 6) return PyErr_Format(PyExc_TypeError, "win_bwd_bytes takes 6 arguments");
    Ten q, k, v;
    psa_win_shape s;
    if (!get_shape(a, &q, &k, &v, &s)) return NULL;
    return PyLong_FromSize_t(p_bwd_bytes(&s));
}

/* win_bwd(q, k, v, scale, window, sinks, q_lens, kv_lens, o, lse, do, dq, dk, dv, workspace, algo): dq, dk, dv;
 * dq, dk, dv, workspace: or None */
static PyObject* win_bwd(PyObject* self, PyObject* const* a, Py_ssize_t na) {
    if (na != 16) return PyErr_Format(PyExc_TypeError, "win_bwd takes 16 arguments");
    Ten q, k, v, o, d, dq, dk, dv, ws = {0};
    psa_win_shape s;
    const int *ql, *kl;
    float* lse;
    if (!get_shape(a, &q, &k, &v, &s) || !get_data(a[8], "o", 4, &q, &o) || !same_shape(&q, &o) ||
        !get_data(a[10], "do", 4, &q, &d) || !same_shape(&q, &d) || !get_lens(a[6], "q_lens", &q, q.n[0], &ql) ||
        !get_lens(a[7], "kv_lens", &q, q.n[0], &kl) || !get_lse(a[9], &q, 3, &lse))
        return NULL;
    const int have = a[14] != Py_None;
    if (have) {
        if (!get(a[14], "workspace", 1, &ws)) return NULL;
        if (ws.dev != q.dev || !dense(&ws)) return bad("the workspace is not on the tensors' device%s%s", "", ""), NULL;
    }
    const long algo = PyLong_AsLong(a[15]);
    if (PyErr_Occurred()) return NULL;
    void* st;
    ON_DEVICE(q.dev, st);
    int rc = 0;
    PyObject *out[3] = {output(a[11], "dq", 4, a[0], &q, &dq), NULL, NULL}, *tmp = NULL;
    if (out[0]) out[1] = output(a[12], "dk", 4, a[1], &k, &dk);
    if (out[1]) out[2] = output(a[13], "dv", 4, a[2], &v, &dv);
    if (out[2] && !have) {                           /* freed after the launch, in the stream's order */
        ws.n[0] = (long long)p_bwd_bytes(&s);
        if (ws.n[0] && !(tmp = make(PyLong_FromLongLong(ws.n[0]), t_u8, a[0], &ws.p))) Py_CLEAR(out[2]);
    }
    if (out[2]) {
        const psa_attn_view vq = view(&q), vk = view(&k), vv = view(&v), vo = view(&o), vd = view(&d), vdq = view(&dq),
                            vdk = view(&dk), vdv = view(&dv);
        CALL(p_bwd(&s, &vq, &vk, &vv, &vo, lse, &vd, &vdq, &vdk, &vdv, ql, kl, ws.p, (size_t)ws.n[0], (int)algo, st));
    }
    Py_XDECREF(tmp);
    return result(rc, 3, out);
}

/* append(cache address, its device, k_new, v_new, start, n_new or None, plan address or 0, pos or None): the status */
static PyObject* append(PyObject* self, PyObject* const* a, Py_ssize_t na) {
    if (na != 8) return PyErr_Format(PyExc_TypeError, "append takes 8 arguments");
    const psa_win_cache* c = (const psa_win_cache*)PyLong_AsVoidPtr(a[0]);
    const psa_rope_plan* plan = (const psa_rope_plan*)PyLong_AsVoidPtr(a[6]);
    const long dev = PyLong_AsLong(a[1]);
    if (PyErr_Occurred()) return NULL;
    Ten k, v, like = {"the cache", NULL, 4, c->dtype, (int)dev, {0}, {0}};
    const int *start, *n_new, *pos = NULL;
    long long sa = 0, sb = 0;
    if (!get_data(a[2], "k_new", 4, &like, &k) || !get_data(a[3], "v_new", 4, &like, &v) || !same_shape(&k, &v) || !fits(&k, 2, 3))
        return NULL;
    if (k.n[0] != c->B || k.n[1] != c->kv_heads || k.n[3] != c->head_dim)
        return bad("k_new and v_new have to be [B, Hkv, T, d] of the cache%s%s", "", ""), NULL;
    if (!get_lens(a[4], "start", &like, c->B, &start) || !get_lens(a[5], "n_new", &like, c->B, &n_new)) return NULL;
    if (!plan != (a[7] == Py_None)) return bad("plan and pos are given together or not at all%s%s", "", ""), NULL;
    if (plan && !get_pos(a[7], &like, plan->n_axes, c->B, k.n[2], &pos, &sa, &sb)) return NULL;
    void* st;
    ON_DEVICE(dev, st);
    const psa_attn_view vk = view(&k), vv = view(&v);
    int rc;
    CALL(p_append(c, &vk, &vv, (int)k.n[2], start, n_new, plan, pos, sa, sb, st));
    return PyLong_FromLong(rc);
}

/* decode(cache address, its device, q, lens, scale, out or None, lse or None, workspace or None, its bytes, its stream):
 * out */
static PyObject* decode(PyObject* self, PyObject* const* a, Py_ssize_t na) {
    if (na != 10) return PyErr_Format(PyExc_TypeError, "decode takes 10 arguments");
    const psa_win_cache* c = (const psa_win_cache*)PyLong_AsVoidPtr(a[0]);
    const long dev = PyLong_AsLong(a[1]);
    const double scale = PyFloat_AsDouble(a[4]);
    if (PyErr_Occurred()) return NULL;
    Ten q, o, ws = {0}, like = {"the cache", NULL, 4, c->dtype, (int)dev, {0}, {0}};
    const int* lens;
    float* lse = NULL;
    if (!get_data(a[2], "q", 3, &like, &q) || !fits(&q, 1, 2)) return NULL;
    if (q.n[0] != c->B || q.n[2] != c->head_dim) return bad("q has to be [B, Hq, d] of the cache%s%s", "", ""), NULL;
    if (a[3] == Py_None) return bad("lens is missing%s%s", "", ""), NULL;
    if (!get_lens(a[3], "lens", &like, c->B, &lens)) return NULL;
    if (a[6] != Py_None && !get_lse(a[6], &q, 2, &lse)) return NULL;
    const int have = a[7] != Py_None;
    if (have && !get(a[7], "workspace", 1, &ws)) return NULL;
    const size_t bytes = PyLong_AsSize_t(a[8]);
    void* const ws_stream = PyLong_AsVoidPtr(a[9]);
    if (PyErr_Occurred()) return NULL;
    void* st;
    ON_DEVICE(dev, st);
    if (have && st != ws_stream) return PyLong_FromLong(OTHER_STREAM);
    int rc = 0;
    PyObject* out[1] = {output(a[5], "out", 3, a[2], &q, &o)};
    if (out[0]) {
        const psa_attn_view vq = {q.p, q.s[0], q.s[1], 0, q.s[2]}, vo = {o.p, o.s[0], o.s[1], 0, o.s[2]};
        CALL(p_decode(c, &vq, &vo, lse, (int)q.n[1], lens, (float)scale, have ? ws.p : NULL, bytes, st));
    }
    return result(rc, 1, out);
}

/* k_new and v_new (names kn, vn) to a cache of any type: their type is the cache's, or any to an 8-bit one. */
static int get_new(PyObject* ko, PyObject* vo, const psa_win_cache* c, long dev, Ten* k, Ten* v) {
    if (!get_data(ko, "k_new", 4, NULL, k) || !get_data(vo, "v_new", 4, k, v) || !same_shape(k, v) || !fits(k, 2, 3)) return 0;
    if (k->dev != dev || (c->dtype != PSA_E4M3 && k->dtype != c->dtype))
        return bad("%s and %s differ in dtype or device", "the cache", "k_new");
    if (k->n[0] != c->B || k->n[1] != c->kv_heads || k->n[3] != c->head_dim)
        return bad("k_new and v_new have to be [B, Hkv, T, d] of the cache%s%s", "", "");
    return 1;
}

/* store(cache address, scales address or 0, device, k_new, v_new, start, n_new or None, plan address or 0, pos or None,
 * rows or None): the status */
static PyObject* store(PyObject* self, PyObject* const* a, Py_ssize_t na) {
    if (na != 10) return PyErr_Format(PyExc_TypeError, "store takes 10 arguments");
    const psa_win_cache* c = (const psa_win_cache*)PyLong_AsVoidPtr(a[0]);
    const psa_win_scales* sc = (const psa_win_scales*)PyLong_AsVoidPtr(a[1]);
    const long dev = PyLong_AsLong(a[2]);
    const psa_rope_plan* plan = (const psa_rope_plan*)PyLong_AsVoidPtr(a[7]);
    if (PyErr_Occurred()) return NULL;
    Ten k, v;
    const int *start, *n_new, *rows, *pos = NULL;
    long long sa = 0, sb = 0, R = -1, stride;
    if (!get_new(a[3], a[4], c, dev, &k, &v)) return NULL;
    if (!get_lens(a[5], "start", &k, c->B, &start) || !get_lens(a[6], "n_new", &k, c->B, &n_new)) return NULL;
    if (!plan != (a[8] == Py_None)) return bad("plan and pos are given together or not at all%s%s", "", ""), NULL;
    if (plan && !get_pos(a[8], &k, plan->n_axes, c->B, k.n[2], &pos, &sa, &sb)) return NULL;
    if (!get_table(a[9], "rows", &k, c->B, &R, &rows, &stride)) return NULL;
    if (a[9] == Py_None) R = k.n[2];
    if (R > 0x7fffffffll) return bad("%s is too large%s", "rows", ""), NULL;
    if (R == 0) return PyLong_FromLong(0);
    void* st;
    ON_DEVICE(dev, st);
    const psa_attn_view vk = view(&k), vv = view(&v);
    int rc;
    CALL(p_store(c, sc, &vk, &vv, (int)k.n[2], rows, stride, (int)R, start, n_new, plan, pos, sa, sb, k.dtype, st));
    return PyLong_FromLong(rc);
}

/* read(cache address, scales address or 0, device, the cache's k, first, n, lens, dtype, k or None, v or None): k, v */
static PyObject* read_back(PyObject* self, PyObject* const* a, Py_ssize_t na) {
    if (na != 10) return PyErr_Format(PyExc_TypeError, "read_back takes 10 arguments");
    const psa_win_cache* c = (const psa_win_cache*)PyLong_AsVoidPtr(a[0]);
    const psa_win_scales* sc = (const psa_win_scales*)PyLong_AsVoidPtr(a[1]);
    const long dev = PyLong_AsLong(a[2]);
    const long long n = PyLong_AsLongLong(a[5]);
    if (PyErr_Occurred()) return NULL;
    if (n < 0 || n > 0x7fffffffll) return bad("%s has to be 0 to 2^31 - 1%s", "n", ""), NULL;
    const int dtype = a[7] == t_f32 ? T_F32 : a[7] == t_bf16 ? T_BF16 : T_OTHER;
    if (dtype == T_OTHER) return bad("%s has to be fp32 or bf16%s", "dtype", ""), NULL;
    Ten o[2], like = {"the cache", NULL, 4, dtype, (int)dev, {0}, {0}};
    const int *first, *lens;
    if (a[4] == Py_None || a[6] == Py_None) return bad("first or lens is missing%s%s", "", ""), NULL;
    if (!get_lens(a[4], "first", &like, c->B, &first) || !get_lens(a[6], "lens", &like, c->B, &lens)) return NULL;
    void* st;
    ON_DEVICE(dev, st);
    int rc = 0;
    PyObject* out[2] = {NULL, NULL};
    for (int i = 0; i < 2; ++i) {
        const char* name = i ? "out_v" : "out_k";
        const long long want[4] = {c->B, c->kv_heads, n, c->head_dim};
        if (a[8 + i] != Py_None) {
            if (!get_data(a[8 + i], name, 4, &like, &o[i])) break;
            int same = 1;
            for (int e = 0; e < 4; ++e) same = same && o[i].n[e] == want[e];
            if (!same) {
                bad("%s has to be [B, Hkv, n, d] of the cache%s", name, "");
                break;
            }
            out[i] = Py_NewRef(a[8 + i]);
        } else {
            out[i] = make(Py_BuildValue("(LLLL)", want[0], want[1], want[2], want[3]), a[7], a[3], &o[i].p);
            if (!out[i]) break;
            o[i].s[3] = 1, o[i].s[2] = want[3], o[i].s[1] = want[2] * want[3], o[i].s[0] = want[1] * o[i].s[1];
        }
    }
    if (out[0] && out[1]) {
        const psa_attn_view vk = view(&o[0]), vv = view(&o[1]);
        CALL(p_read(c, sc, &vk, &vv, (int)n, first, lens, dtype, st));
    }
    return result(rc, 2, out);
}

/* A workspace of `n` bytes for one call, to be freed after its launch, in the stream's order: what many
 * caches' calls need is then one piece of memory a stream, and that of a captured call is its graph's.  NULL
 * and no error: none is needed. */
static PyObject* call_workspace(size_t n, PyObject* on, void** data) {
    *data = NULL;
    return n ? make(PyLong_FromSize_t(n), t_u8, on, data) : NULL;
}

/* decode_any(cache address, scales address, device, q, lens, scale, out or None, lse or None): out */
static PyObject* decode_any(PyObject* self, PyObject* const* a, Py_ssize_t na) {
    if (na != 8) return PyErr_Format(PyExc_TypeError, "decode_any takes 8 arguments");
    const psa_win_cache* c = (const psa_win_cache*)PyLong_AsVoidPtr(a[0]);
    const psa_win_scales* sc = (const psa_win_scales*)PyLong_AsVoidPtr(a[1]);
    const long dev = PyLong_AsLong(a[2]);
    const double scale = PyFloat_AsDouble(a[5]);
    if (PyErr_Occurred()) return NULL;
    Ten q, o;
    const int* lens;
    float* lse = NULL;
    void *ws, *st;
    if (!get_data(a[3], "q", 3, NULL, &q) || !fits(&q, 1, 2)) return NULL;
    if (q.dev != dev || (c->dtype != PSA_E4M3 && q.dtype != c->dtype))
        return bad("%s and %s differ in dtype or device", "the cache", "q"), NULL;
    if (q.n[0] != c->B || q.n[2] != c->head_dim) return bad("q has to be [B, Hq, d] of the cache%s%s", "", ""), NULL;
    if (a[4] == Py_None) return bad("lens is missing%s%s", "", ""), NULL;
    if (!get_lens(a[4], "lens", &q, c->B, &lens) || (a[7] != Py_None && !get_lse(a[7], &q, 2, &lse))) return NULL;
    ON_DEVICE(dev, st);
    int rc = 0;
    const size_t bytes = p_decode_any_bytes(c, (int)q.n[1], q.dtype);
    PyObject *out[1] = {output(a[6], "out", 3, a[3], &q, &o)}, *tmp = out[0] ? call_workspace(bytes, a[3], &ws) : NULL;
    if (out[0] && !PyErr_Occurred()) {
        const psa_attn_view vq = {q.p, q.s[0], q.s[1], 0, q.s[2]}, vo = {o.p, o.s[0], o.s[1], 0, o.s[2]};
        CALL(p_decode_any(c, sc, &vq, &vo, lse, (int)q.n[1], lens, (float)scale, ws, bytes, q.dtype, st));
    }
    Py_XDECREF(tmp);
    return call_result(rc, out);
}

/* tree(cache address, scales address or 0, device, q, k_new, v_new, lens, scale, parents or None, n_new or None, out or
 * None, lse or None, algo): out */
static PyObject* tree(PyObject* self, PyObject* const* a, Py_ssize_t na) {
    if (na != 13) return PyErr_Format(PyExc_TypeError, "tree takes 13 arguments");
    const psa_win_cache* c = (const psa_win_cache*)PyLong_AsVoidPtr(a[0]);
    const psa_win_scales* sc = (const psa_win_scales*)PyLong_AsVoidPtr(a[1]);
    const long dev = PyLong_AsLong(a[2]), algo = PyLong_AsLong(a[12]);
    const double scale = PyFloat_AsDouble(a[7]);
    if (PyErr_Occurred()) return NULL;
    Ten q, k, v, o;
    const int *lens, *parents, *n_new;
    long long stride, T;
    float* lse = NULL;
    void *ws, *st;
    if (!get_new(a[4], a[5], c, dev, &k, &v)) return NULL;
    if (!get_data(a[3], "q", 4, &k, &q) || !fits(&q, 1, 2)) return NULL;
    if (q.n[0] != c->B || q.n[2] != k.n[2] || q.n[3] != c->head_dim)
        return bad("q has to be [B, Hq, T, d] of the cache and of k_new%s%s", "", ""), NULL;
    T = k.n[2];
    if (a[6] == Py_None) return bad("lens is missing%s%s", "", ""), NULL;
    if (!get_lens(a[6], "lens", &q, c->B, &lens) || !get_table(a[8], "parents", &q, c->B, &T, &parents, &stride) ||
        !get_lens(a[9], "n_new", &q, c->B, &n_new) || (a[11] != Py_None && !get_lse(a[11], &q, 3, &lse)))
        return NULL;
    ON_DEVICE(dev, st);
    int rc = 0;
    const size_t bytes = p_tree_bytes(c, (int)q.n[1], (int)q.n[2], q.dtype);
    PyObject *out[1] = {output(a[10], "out", 4, a[3], &q, &o)}, *tmp = out[0] ? call_workspace(bytes, a[3], &ws) : NULL;
    if (out[0] && !PyErr_Occurred()) {
        const psa_attn_view vq = view(&q), vk = view(&k), vv = view(&v), vo = view(&o);
        CALL(p_tree(c, sc, &vq, &vk, &vv, &vo, lse, (int)q.n[1], (int)k.n[2], parents, stride, n_new, lens, (float)scale, ws,
                    bytes, (int)algo, q.dtype, st));
    }
    Py_XDECREF(tmp);
    return call_result(rc, out);
}

#define FAST(name) {#name, (PyCFunction)(void (*)(void))name, METH_FASTCALL, NULL}
static PyMethodDef methods[] = {{"init", init, METH_VARARGS, NULL}, FAST(rope), FAST(win_fwd), FAST(win_bwd_bytes),
                                FAST(win_bwd), FAST(append), FAST(decode), FAST(store), FAST(read_back),
                                FAST(decode_any), FAST(tree), {NULL, NULL, 0, NULL}};
static struct PyModuleDef module = {PyModuleDef_HEAD_INIT, "_psa_bind", NULL, -1, methods};

PyMODINIT_FUNC PyInit__psa_bind(void) {
    s_data_ptr = PyUnicode_InternFromString("data_ptr");
    s_stride = PyUnicode_InternFromString("stride");
    s_shape = PyUnicode_InternFromString("shape");
    s_dtype = PyUnicode_InternFromString("dtype");
    s_get_device = PyUnicode_InternFromString("get_device");
    s_device = PyUnicode_InternFromString("device");
    kw_make = Py_BuildValue("(ss)", "dtype", "device");
    if (!s_data_ptr || !s_stride || !s_shape || !s_dtype || !s_get_device || !s_device || !kw_make) return NULL;
    PyObject* m = PyModule_Create(&module);
    if (m && (PyModule_AddIntConstant(m, "OTHER_DEVICE", OTHER_DEVICE) < 0 ||
              PyModule_AddIntConstant(m, "OTHER_STREAM", OTHER_STREAM) < 0)) {
        Py_DECREF(m);
        return NULL;
    }
    return m;
}
