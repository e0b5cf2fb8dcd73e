// The paged calls as a CPython extension: argument marshalling and output
// allocation without the interpreter, for calls that are made once per layer and
// decoding step and take less time on the GPU than a dozen attribute reads in
// Python (measured on the Grace host: 19 us an attention call through ctypes).
//
// Each function takes the case that a program normally makes — tensors of the
// right types, shapes and strides on the current device, on its current stream —
// and answers None for anything else; the binding (fm.py) then goes its own way, with
// the same library call behind full checks and their errors.
#include <torch/csrc/autograd/python_variable.h>

#include <initializer_list>

#include <ATen/ops/empty.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>

#include "fm.h"

namespace {

decltype(&fm_paged_plan) g_plan;
decltype(&fm_paged_append) g_append;
decltype(&fm_attn_paged) g_attn;
decltype(&fm_rope) g_rope;
decltype(&fm_paged_append_rope) g_append_rope;
decltype(&fm_paged_weights) g_weights;
decltype(&fm_paged_evict) g_evict;
decltype(&fm_paged_release) g_release;
decltype(&fm_verify_drafts) g_verify;

// Tensor of an argument, or null.
const at::Tensor *tensor(PyObject *o) { return THPVariable_Check(o) ? &THPVariable_Unpack(o) : nullptr; }

// Address of a contiguous CUDA tensor of that type on device dev with n elements
// (any number if n < 0), or null.
void *flat(PyObject *o, at::ScalarType type, int dev, int64_t n = -1, int dims = -1)
{
    const at::Tensor *t = tensor(o);
    if (!t || !t->is_cuda() || t->get_device() != dev || t->scalar_type() != type || !t->is_contiguous()) return nullptr;
    if ((n >= 0 && t->numel() != n) || (dims >= 0 && t->dim() != dims)) return nullptr;
    return t->data_ptr();
}

// The current device if tensor t is on it, else -1.
int device_of(const at::Tensor *t)
{
    if (!t || !t->is_cuda()) return -1;
    const int dev = t->get_device();
    return dev == c10::cuda::current_device() ? dev : -1;
}

fm_stream_t stream_of(int dev) { return (fm_stream_t)c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)dev).stream(); }

// (scaled: whether the descales of an e4m3 cache are looked for.)
bool cache_of(PyObject *ko, PyObject *vo, PyObject *kdo, PyObject *vdo, int dev, fm_paged_cache *c, bool scaled = true)
{
    const at::Tensor *k = tensor(ko), *v = tensor(vo);
    if (!k || !v || !k->is_cuda() || !v->is_cuda() || k->get_device() != dev || v->get_device() != dev) return false;
    const at::ScalarType type = k->scalar_type();
    if (v->scalar_type() != type || k->dim() != 4 || v->sizes() != k->sizes() || k->stride(3) != 1 || v->stride(3) != 1) return false;
    c->k_descale = c->v_descale = nullptr;
    c->dtype = FM_DT_BF16;
    if (type != at::kBFloat16) {
        if (type != at::kByte && type != at::kFloat8_e4m3fn) return false;
        c->dtype = FM_DT_E4M3;
        c->k_descale = scaled ? (const float *)flat(kdo, at::kFloat, dev, 1) : nullptr;
        c->v_descale = scaled ? (const float *)flat(vdo, at::kFloat, dev, 1) : nullptr;
        if (scaled && (!c->k_descale || !c->v_descale)) return false;
    }
    for (int i = 0; i < 4; ++i)
        if (k->size(i) > INT32_MAX) return false;
    c->k = k->data_ptr();
    c->v = v->data_ptr();
    const int64_t d = k->size(3);
    int64_t *ks[3] = {&c->k_page, &c->k_head, &c->k_tok}, *vs[3] = {&c->v_page, &c->v_head, &c->v_tok};
    for (int i = 0; i < 3; ++i) {           // the stride of a dimension of size one is never used
        *ks[i] = k->size(i) > 1 ? k->stride(i) : d;
        *vs[i] = v->size(i) > 1 ? v->stride(i) : d;
    }
    c->num_pages = (int32_t)k->size(0);
    c->Hkv = (int32_t)k->size(1);
    c->page_size = (int32_t)k->size(2);
    c->d = (int32_t)d;
    return true;
}

// bf16 rows [T, H, d] with any token and head strides.
bool rows_of(const at::Tensor *t, int dev, int64_t H, int64_t d, int64_t *tok, int64_t *head)
{
    if (!t || !t->is_cuda() || t->get_device() != dev || t->scalar_type() != at::kBFloat16 || t->dim() != 3 || t->size(1) != H ||
        t->size(2) != d || t->stride(2) != 1 || t->size(0) > INT32_MAX)
        return false;
    *tok = t->size(0) > 1 ? t->stride(0) : d;
    *head = H > 1 ? t->stride(1) : d;
    return true;
}

PyObject *none() { Py_RETURN_NONE; }

// bind(plan, append, attn, rope, append_rope, weights, evict, release, verify): addresses of the library's functions.
PyObject *bind(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    if (n != 9) {
        PyErr_SetString(PyExc_TypeError, "bind(plan, append, attn, rope, append_rope, weights, evict, release, verify)");
        return nullptr;
    }
    g_plan = (decltype(g_plan))PyLong_AsVoidPtr(a[0]);
    g_append = (decltype(g_append))PyLong_AsVoidPtr(a[1]);
    g_attn = (decltype(g_attn))PyLong_AsVoidPtr(a[2]);
    g_rope = (decltype(g_rope))PyLong_AsVoidPtr(a[3]);
    g_append_rope = (decltype(g_append_rope))PyLong_AsVoidPtr(a[4]);
    g_weights = (decltype(g_weights))PyLong_AsVoidPtr(a[5]);
    g_evict = (decltype(g_evict))PyLong_AsVoidPtr(a[6]);
    g_release = (decltype(g_release))PyLong_AsVoidPtr(a[7]);
    g_verify = (decltype(g_verify))PyLong_AsVoidPtr(a[8]);
    if (PyErr_Occurred()) return nullptr;
    return none();
}

const fm_paged_step *step_of(PyObject *o)
{
    const void *p = PyLong_AsVoidPtr(o);
    if (!p) PyErr_Clear();
    return (const fm_paged_step *)p;
}

// plan(step, ctx, new, table, seq, cu, slots, positions, plan, status, free, head, next): status code or None.
PyObject *plan(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    if (n != 13) return none();
    const fm_paged_step *s = step_of(a[0]);
    const int dev = device_of(tensor(a[1]));
    if (!s || dev < 0) return none();
    const int64_t R = s->requests, T = s->max_tokens;
    const auto i32 = at::kInt;
    void *ctx = flat(a[1], i32, dev, R, 1), *fresh = flat(a[2], i32, dev, R, 1), *table = flat(a[3], i32, dev, R * s->max_pages, 2),
         *seq = flat(a[4], i32, dev, R, 1), *cu = flat(a[5], i32, dev, R + 1, 1), *slots = flat(a[6], at::kLong, dev, T, 1),
         *pos = flat(a[7], i32, dev, T, 1), *buf = flat(a[8], at::kByte, dev), *status = flat(a[9], i32, dev, 1, 1);
    if (!ctx || !fresh || !table || !seq || !cu || !slots || !pos || !buf || !status || tensor(a[3])->size(0) != R) return none();
    void *pages = nullptr, *head = nullptr, *next = nullptr;
    int n_free = 0;
    if (a[10] != Py_None) {
        pages = flat(a[10], i32, dev, -1, 1);
        head = flat(a[11], i32, dev, 1, 1);
        next = flat(a[12], i32, dev, 1, 1);
        if (!pages || !head || !next || tensor(a[10])->numel() > INT32_MAX) return none();
        n_free = (int)tensor(a[10])->numel();
    }
    return PyLong_FromLong(g_plan(s, (const int32_t *)ctx, (const int32_t *)fresh, (int32_t *)table, (const int32_t *)pages, n_free,
                                  (const int32_t *)head, (int32_t *)next, (int32_t *)seq, (int32_t *)cu, (int64_t *)slots, (int32_t *)pos,
                                  buf, (size_t)tensor(a[8])->numel(), (int32_t *)status, stream_of(dev)));
}

// append(k, v, slots, k_cache, v_cache, status, k_descale, v_descale): status code or None.
PyObject *append(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    if (n != 8) return none();
    const at::Tensor *k = tensor(a[0]), *v = tensor(a[1]), *slots = tensor(a[2]);
    const int dev = device_of(k);
    fm_paged_cache c;
    int64_t kt, kh, vt, vh;
    if (dev < 0 || !cache_of(a[3], a[4], a[6], a[7], dev, &c) || !rows_of(k, dev, c.Hkv, c.d, &kt, &kh) || !rows_of(v, dev, c.Hkv, c.d, &vt, &vh))
        return none();
    const void *at = flat(a[2], at::kLong, dev, -1, 1);
    void *status = flat(a[5], at::kInt, dev, 1, 1);
    if (!at || !status || v->size(0) != k->size(0) || slots->numel() < k->size(0) || k->size(0) == 0) return none();
    return PyLong_FromLong(g_append(k->data_ptr(), kt, kh, v->data_ptr(), vt, vh, (const int64_t *)at, (int)k->size(0), &c, (int32_t *)status,
                                    stream_of(dev)));
}

// attend(step, q, k_cache, v_cache, table, plan, scale, fp32 output, status, k_descale, v_descale): (o, lse), status code or None.
PyObject *attend(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    if (n != 11) return none();
    const fm_paged_step *s = step_of(a[0]);
    const at::Tensor *q = tensor(a[1]);
    const int dev = device_of(q);
    fm_paged_cache c;
    int64_t qt, qh;
    if (!s || dev < 0 || !cache_of(a[2], a[3], a[9], a[10], dev, &c) || !rows_of(q, dev, s->Hq, s->d, &qt, &qh)) return none();
    void *table = flat(a[4], at::kInt, dev, (int64_t)s->requests * s->max_pages, 2), *buf = flat(a[5], at::kByte, dev),
         *status = flat(a[8], at::kInt, dev, 1, 1);
    const double scale = PyFloat_Check(a[6]) ? PyFloat_AS_DOUBLE(a[6]) : -1.0;
    if (!table || !buf || !status || scale <= 0 || tensor(a[4])->size(0) != s->requests || q->size(0) == 0) return none();
    const bool f32 = a[7] == Py_True;
    const auto opt = at::TensorOptions().device(q->device());
    at::Tensor o = at::empty(q->sizes(), opt.dtype(f32 ? at::kFloat : at::kBFloat16));
    at::Tensor lse = at::empty({q->size(0), q->size(1)}, opt.dtype(at::kFloat));
    const fm_status st = g_attn(s, q->data_ptr(), qt, qh, (int)q->size(0), &c, (const int32_t *)table, buf, (size_t)tensor(a[5])->numel(),
                                (float)scale, o.data_ptr(), f32 ? FM_DT_F32 : FM_DT_BF16, (float *)lse.data_ptr(), (int32_t *)status,
                                stream_of(dev));
    if (st != FM_OK) return PyLong_FromLong(st);
    PyObject *po = THPVariable_Wrap(std::move(o)), *pl = THPVariable_Wrap(std::move(lse));
    if (!po || !pl) {
        Py_XDECREF(po);
        Py_XDECREF(pl);
        return nullptr;
    }
    PyObject *r = PyTuple_Pack(2, po, pl);
    Py_DECREF(po);
    Py_DECREF(pl);
    return r;
}

// A tensor like `like` in shape, of that type, newly allocated; or `given` if it is not None and is one, contiguous, on dev.
bool out_like(PyObject *given, const at::Tensor &like, at::ScalarType type, int dev, at::Tensor *out)
{
    if (given == Py_None) {
        *out = at::empty(like.sizes(), at::TensorOptions().device(like.device()).dtype(type));
        return true;
    }
    const at::Tensor *t = tensor(given);
    if (!t || !flat(given, type, dev) || t->sizes() != like.sizes()) return false;
    *out = *t;
    return true;
}

// A Rotary's table, by its address, if the tensor of its turns is on dev.
const fm_rotary *rotary_of(PyObject *o, PyObject *turns, int dev)
{
    const fm_rotary *r = (const fm_rotary *)PyLong_AsVoidPtr(o);
    if (!r) {
        PyErr_Clear();
        return nullptr;
    }
    const at::Tensor *t = tensor(turns);
    return t && t->is_cuda() && t->get_device() == dev && t->data_ptr() == r->turns ? r : nullptr;
}

// fp32 pool of weights [num_pages, Hkv, page_size] beside a key cache.
float *pool_of(PyObject *o, const at::Tensor &k, int dev)
{
    const at::Tensor *t = tensor(o);
    if (!t || t->dim() != 3 || t->size(0) != k.size(0) || t->size(1) != k.size(1) || t->size(2) != k.size(2)) return nullptr;
    return (float *)flat(o, at::kFloat, dev);
}

// The strides of a [B, H, N, d] tensor, or of rows [T, H, d] as one batch; those of dimensions of size one are never used.
bool batch_of(const at::Tensor &t, int64_t *B, int64_t *H, int64_t *N, fm_strides *s)
{
    const int64_t dims = t.dim();
    if ((dims != 3 && dims != 4) || t.stride(dims - 1) != 1) return false;
    *B = dims == 4 ? t.size(0) : 1;
    *H = t.size(1);
    *N = t.size(dims == 4 ? 2 : 0);
    s->batch = *B > 1 ? t.stride(0) : 0;
    s->head = *H > 1 ? t.stride(1) : 0;
    s->tok = *N > 1 ? t.stride(dims == 4 ? 2 : 0) : 0;
    return *B <= INT32_MAX && *H <= INT32_MAX && *N <= INT32_MAX;
}

int float_of(const at::Tensor &t) { return t.scalar_type() == at::kBFloat16 ? FM_DT_BF16 : t.scalar_type() == at::kFloat ? FM_DT_F32 : -1; }

// rope(x, positions, table, turns, out, fp32 output (None: x's type), inverse): the result, status code or None.
PyObject *rope(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    if (n != 7) return none();
    const at::Tensor *x = tensor(a[0]), *pos = tensor(a[1]);
    const int dev = device_of(x);
    if (dev < 0 || !pos || x->numel() == 0 || float_of(*x) < 0) return none();
    int64_t B, H, N, Bo, Ho, No;
    fm_strides xs, ys;
    if (!batch_of(*x, &B, &H, &N, &xs)) return none();
    const fm_rotary *r = rotary_of(a[2], a[3], dev);
    const void *p = flat(a[1], at::kInt, dev);
    const bool own = pos->dim() == 2 && x->dim() == 4;        // positions of every sequence of the batch
    if (!r || !p || (own ? pos->size(0) != B || pos->size(1) != N : pos->dim() != 1 || pos->size(0) != N)) return none();
    const at::ScalarType type = a[5] == Py_None ? x->scalar_type() : a[5] == Py_True ? at::kFloat : at::kBFloat16;
    at::Tensor y;
    if (a[4] == Py_None) {
        y = at::empty(x->sizes(), x->options().dtype(type));
    } else {
        const at::Tensor *t = tensor(a[4]);
        if (!t || !t->is_cuda() || t->get_device() != dev || t->sizes() != x->sizes() || (a[5] != Py_None && t->scalar_type() != type)) return none();
        y = *t;
    }
    if (float_of(y) < 0 || !batch_of(y, &Bo, &Ho, &No, &ys)) return none();
    // (In each function the result is wrapped before the call, so that nothing that fails behind it makes the call twice.)
    PyObject *res = THPVariable_Wrap(y);
    if (!res) return nullptr;
    const fm_status st = g_rope(x->data_ptr(), float_of(*x), xs, (const int32_t *)p, own ? N : 0, (int)B, (int)H, (int)N, (int)x->size(x->dim() - 1), r,
                                a[6] == Py_True, y.data_ptr(), float_of(y), ys, stream_of(dev));
    if (st == FM_OK) return res;
    Py_DECREF(res);
    return PyLong_FromLong(st);
}

// append_rope(q, k, v, slots, positions, table, turns, k_cache, v_cache, status, q_out, k_descale, v_descale): the turned q, status
// code or None.
PyObject *append_rope(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    if (n != 13) return none();
    const at::Tensor *q = tensor(a[0]), *k = tensor(a[1]), *v = tensor(a[2]), *slots = tensor(a[3]), *pos = tensor(a[4]);
    const int dev = device_of(q);
    fm_paged_cache c;
    int64_t qt, qh, kt, kh, vt, vh, ot, oh;
    if (dev < 0 || q->dim() != 3 || !cache_of(a[7], a[8], a[11], a[12], dev, &c) || !rows_of(q, dev, q->size(1), c.d, &qt, &qh) ||
        !rows_of(k, dev, c.Hkv, c.d, &kt, &kh) || !rows_of(v, dev, c.Hkv, c.d, &vt, &vh))
        return none();
    const int64_t T = q->size(0);
    const void *at = flat(a[3], at::kLong, dev, -1, 1), *p = flat(a[4], at::kInt, dev, -1, 1);
    void *status = flat(a[9], at::kInt, dev, 1, 1);
    const fm_rotary *r = rotary_of(a[5], a[6], dev);
    if (!at || !p || !status || !r || T == 0 || k->size(0) != T || v->size(0) != T || slots->numel() < T || pos->numel() < T || q->size(1) > INT32_MAX)
        return none();
    at::Tensor o;
    if (a[10] == Py_None) {
        o = at::empty(q->sizes(), q->options());
    } else {
        const at::Tensor *t = tensor(a[10]);
        if (!t || t->sizes() != q->sizes()) return none();
        o = *t;
    }
    if (!rows_of(&o, dev, q->size(1), c.d, &ot, &oh)) return none();
    PyObject *res = THPVariable_Wrap(o);
    if (!res) return nullptr;
    const fm_status st = g_append_rope(q->data_ptr(), qt, qh, (int)q->size(1), k->data_ptr(), kt, kh, v->data_ptr(), vt, vh, (const int64_t *)at,
                                       (const int32_t *)p, (int)T, r, &c, o.data_ptr(), ot, oh, (int32_t *)status, stream_of(dev));
    if (st == FM_OK) return res;
    Py_DECREF(res);
    return PyLong_FromLong(st);
}

// weigh(step, q, lse, k_cache, table, plan, scale, weights, status, k_descale): status code or None.
PyObject *weigh(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    if (n != 10) return none();
    const fm_paged_step *s = step_of(a[0]);
    const at::Tensor *q = tensor(a[1]), *z = tensor(a[2]);
    const int dev = device_of(q);
    fm_paged_cache c;
    int64_t qt, qh;
    if (!s || dev < 0 || !cache_of(a[3], a[3], a[9], a[9], dev, &c) || !rows_of(q, dev, s->Hq, s->d, &qt, &qh)) return none();
    const void *lse = flat(a[2], at::kFloat, dev, q->size(0) * s->Hq, 2), *table = flat(a[4], at::kInt, dev, (int64_t)s->requests * s->max_pages, 2);
    void *buf = flat(a[5], at::kByte, dev), *status = flat(a[8], at::kInt, dev, 1, 1);
    float *pool = pool_of(a[7], *tensor(a[3]), dev);
    const double scale = PyFloat_Check(a[6]) ? PyFloat_AS_DOUBLE(a[6]) : -1.0;
    if (!lse || z->size(1) != s->Hq || !table || !buf || !status || !pool || scale <= 0 || tensor(a[4])->size(0) != s->requests || q->size(0) == 0)
        return none();
    return PyLong_FromLong(g_weights(s, q->data_ptr(), qt, qh, (int)q->size(0), &c, (const int32_t *)table, buf, (size_t)tensor(a[5])->numel(), (float)scale,
                                     (const float *)lse, pool, (int32_t *)status, stream_of(dev)));
}

// A C int that a Python int holds.
bool int_of(PyObject *o, int *x)
{
    int over = 0;
    const long v = PyLong_Check(o) ? PyLong_AsLongAndOverflow(o, &over) : (over = 1, 0);
    if (over || v > INT32_MAX || v < INT32_MIN) return false;
    *x = (int)v;
    return true;
}

// evict(lens, table, k_cache, v_cache, weights, budget, status, recent, sink, kept, new_lens): the new lengths, status code or None.
PyObject *evict(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    if (n != 11) return none();
    const at::Tensor *lens = tensor(a[0]), *table = tensor(a[1]);
    const int dev = device_of(lens);
    fm_paged_cache c;
    int budget, recent, sink;
    if (dev < 0 || !int_of(a[5], &budget) || !int_of(a[7], &recent) || !int_of(a[8], &sink) || budget <= 0 ||
        !cache_of(a[2], a[3], nullptr, nullptr, dev, &c, false))
        return none();
    const int64_t R = lens->dim() == 1 ? lens->size(0) : -1;
    const void *at = flat(a[0], at::kInt, dev, R, 1), *pages = flat(a[1], at::kInt, dev, -1, 2);
    void *status = flat(a[6], at::kInt, dev, 1, 1);
    float *pool = pool_of(a[4], *tensor(a[2]), dev);
    c.k_descale = c.v_descale = pool;         // any address: codes are moved as they are
    if (R <= 0 || R > INT32_MAX || !at || !pages || !status || !pool || table->size(0) != R || table->size(1) > INT32_MAX) return none();
    at::Tensor kept, now;
    if (a[9] == Py_None) {
        kept = at::empty({R, c.Hkv, budget}, lens->options());
    } else {
        const at::Tensor *t = tensor(a[9]);
        if (!t || !flat(a[9], at::kInt, dev, R * c.Hkv * budget, 3) || t->size(0) != R || t->size(1) != c.Hkv) return none();
        kept = *t;
    }
    if (!out_like(a[10], *lens, at::kInt, dev, &now)) return none();
    PyObject *res = THPVariable_Wrap(now);
    if (!res) return nullptr;
    const fm_status st = g_evict(&c, (int)R, (int)table->size(1), (const int32_t *)at, (const int32_t *)pages, pool, budget, recent, sink,
                                 (int32_t *)kept.data_ptr(), (int32_t *)now.data_ptr(), (int32_t *)status, stream_of(dev));
    if (st == FM_OK) return res;
    Py_DECREF(res);
    return PyLong_FromLong(st);
}

// A tuple of new references, which are taken; null where one is missing.
PyObject *tuple_of(std::initializer_list<PyObject *> xs)
{
    PyObject *r = PyTuple_New((Py_ssize_t)xs.size());
    bool all = r != nullptr;
    Py_ssize_t i = 0;
    for (PyObject *x : xs) {
        all = all && x;
        if (r) PyTuple_SET_ITEM(r, i++, x);
        else Py_XDECREF(x);
    }
    if (!all) Py_CLEAR(r);
    return r;
}

// release(held, lens, table, page_size, num_pages, free, head, status, free_next, seq_lens): (seq_lens, free_next), status code or None.
PyObject *release(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    if (n != 10 || a[5] == Py_None) return none();
    const at::Tensor *held = tensor(a[0]), *table = tensor(a[2]), *pages = tensor(a[5]), *head = tensor(a[6]);
    const int dev = device_of(held);
    int page_size, num_pages;
    if (dev < 0 || held->dim() != 1 || !int_of(a[3], &page_size) || !int_of(a[4], &num_pages)) return none();
    const int64_t R = held->size(0);
    const auto i32 = at::kInt;
    const void *h = flat(a[0], i32, dev, R, 1), *l = flat(a[1], i32, dev, R, 1), *t = flat(a[2], i32, dev, -1, 2), *hd = flat(a[6], i32, dev, 1, 1);
    void *free = flat(a[5], i32, dev, -1, 1), *status = flat(a[7], i32, dev, 1, 1);
    if (R <= 0 || R > INT32_MAX || !h || !l || !t || !free || !hd || !status || table->size(0) != R || table->size(1) > INT32_MAX || pages->numel() > INT32_MAX)
        return none();
    at::Tensor next, seq;
    if (!out_like(a[8], *head, i32, dev, &next) || !out_like(a[9], *held, i32, dev, &seq)) return none();
    PyObject *res = tuple_of({THPVariable_Wrap(seq), THPVariable_Wrap(next)});
    if (!res) return nullptr;
    const fm_status st = g_release((int)R, (int)table->size(1), num_pages, page_size, (const int32_t *)h, (const int32_t *)l, (const int32_t *)t, (int32_t *)free,
                                   (int)pages->numel(), (const int32_t *)hd, (int32_t *)next.data_ptr(), (int32_t *)seq.data_ptr(), (int32_t *)status, stream_of(dev));
    if (st == FM_OK) return res;
    Py_DECREF(res);
    return PyLong_FromLong(st);
}

// verify(target, draft, tokens, u_accept, u_sample, cu, seq, status, out, n_out, new_lens): (out, n_out, new_lens), status code or None.
PyObject *verify(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    if (n != 11) return none();
    const at::Tensor *p = tensor(a[0]), *q = tensor(a[1]), *seq = tensor(a[6]);
    const int dev = device_of(p);
    if (dev < 0 || p->dim() != 2 || p->size(0) == 0 || p->size(1) == 0 || float_of(*p) < 0 || p->stride(1) != 1 || !seq || seq->dim() != 1) return none();
    const int64_t T = p->size(0), V = p->size(1), R = seq->size(0);
    if (a[1] != Py_None && (!q || !q->is_cuda() || q->get_device() != dev || q->sizes() != p->sizes() || q->scalar_type() != p->scalar_type() || q->stride(1) != 1))
        return none();
    const auto i32 = at::kInt;
    const void *tok = flat(a[2], i32, dev, T, 1), *ua = flat(a[3], at::kFloat, dev, T, 1), *us = flat(a[4], at::kFloat, dev, R, 1), *cu = flat(a[5], i32, dev, R + 1, 1),
               *len = flat(a[6], i32, dev, R, 1);
    void *status = flat(a[7], i32, dev, 1, 1);
    if (R <= 0 || R > INT32_MAX || T > INT32_MAX || V > INT32_MAX || !tok || !ua || !us || !cu || !len || !status) return none();
    at::Tensor out, count, now;
    if (!out_like(a[8], *tensor(a[2]), i32, dev, &out) || !out_like(a[9], *seq, i32, dev, &count) || !out_like(a[10], *seq, i32, dev, &now)) return none();
    PyObject *res = tuple_of({THPVariable_Wrap(out), THPVariable_Wrap(count), THPVariable_Wrap(now)});
    if (!res) return nullptr;
    const fm_status st = g_verify(p->data_ptr(), T > 1 ? p->stride(0) : V, q ? q->data_ptr() : nullptr, q && T > 1 ? q->stride(0) : V, float_of(*p), (int)V, (int)T,
                                  (const int32_t *)tok, (const float *)ua, (const float *)us, (const int32_t *)cu, (const int32_t *)len, (int)R,
                                  (int32_t *)out.data_ptr(), (int32_t *)count.data_ptr(), (int32_t *)now.data_ptr(), (int32_t *)status, stream_of(dev));
    if (st == FM_OK) return res;
    Py_DECREF(res);
    return PyLong_FromLong(st);
}

// No exception of torch's (a tensor without storage, a failing CUDA call) leaves a
// function: the other way meets it again and raises it.
template <PyObject *(*F)(PyObject *, PyObject *const *, Py_ssize_t)>
PyObject *guarded(PyObject *self, PyObject *const *a, Py_ssize_t n)
{
    try {
        return F(self, a, n);
    } catch (...) {
        PyErr_Clear();
        return none();
    }
}

PyMethodDef methods[] = {{"bind", (PyCFunction)(void (*)(void))bind, METH_FASTCALL, nullptr},
                         {"plan", (PyCFunction)(void (*)(void))guarded<plan>, METH_FASTCALL, nullptr},
                         {"append", (PyCFunction)(void (*)(void))guarded<append>, METH_FASTCALL, nullptr},
                         {"attend", (PyCFunction)(void (*)(void))guarded<attend>, METH_FASTCALL, nullptr},
                         {"rope", (PyCFunction)(void (*)(void))guarded<rope>, METH_FASTCALL, nullptr},
                         {"append_rope", (PyCFunction)(void (*)(void))guarded<append_rope>, METH_FASTCALL, nullptr},
                         {"weigh", (PyCFunction)(void (*)(void))guarded<weigh>, METH_FASTCALL, nullptr},
                         {"evict", (PyCFunction)(void (*)(void))guarded<evict>, METH_FASTCALL, nullptr},
                         {"release", (PyCFunction)(void (*)(void))guarded<release>, METH_FASTCALL, nullptr},
                         {"verify", (PyCFunction)(void (*)(void))guarded<verify>, METH_FASTCALL, nullptr},
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_fm_call", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__fm_call(void) { return PyModule_Create(&module); }
