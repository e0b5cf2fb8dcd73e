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

#include <ATen/ops/empty.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>

#include "fm.h"

namespace {

decltype(&fm_paged_plan) g_plan;
decltype(&fm_paged_append) g_append;
decltype(&fm_attn_paged) g_attn;

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

bool cache_of(PyObject *ko, PyObject *vo, PyObject *kdo, PyObject *vdo, int dev, fm_paged_cache *c)
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
        c->k_descale = (const float *)flat(kdo, at::kFloat, dev, 1);
        c->v_descale = (const float *)flat(vdo, at::kFloat, dev, 1);
        if (!c->k_descale || !c->v_descale) return false;
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

// bind(plan, append, attn): addresses of the library's functions.
PyObject *bind(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    if (n != 3) {
        PyErr_SetString(PyExc_TypeError, "bind(plan, append, attn)");
        return nullptr;
    }
    g_plan = (decltype(g_plan))PyLong_AsVoidPtr(a[0]);
    g_append = (decltype(g_append))PyLong_AsVoidPtr(a[1]);
    g_attn = (decltype(g_attn))PyLong_AsVoidPtr(a[2]);
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
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_fm_call", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__fm_call(void) { return PyModule_Create(&module); }
