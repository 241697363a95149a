// The attention and cache helpers of __init__.py for their plain calls: GPU
// tensors of the right types and shapes, the current stream, the helpers' own
// workspace.  Each checks its arguments, allocates its results and calls the
// C ABI, as the Python form does, in 3 to 6 us of host time instead of 15 to
// 20 (the kernels of a decode step take about as long).  Whatever is not
// plain, wrong arguments among it, returns None: the Python form then does
// the call or says what is wrong.
#include <Python.h>

#include <ATen/ATen.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cmath>

#include "../../include/cfp32.h"

namespace {

// The library's entry points (from the library that the package has loaded),
// and two Python callables: the current raw stream of a device index, and the
// helpers' workspace of (bytes, device index, raw stream), None where it has to
// be allocated first (which the Python form does).  From that callable's return
// to the end of a call no other thread runs Python, and the buffer is held, so
// two threads' launches over one workspace follow each other.
struct Api {
    decltype(&cfp32_attention_prompt_workspace_bytes) prompt_ws;
    decltype(&cfp32_attention_prompt) prompt;
    decltype(&cfp32_attention_decode_workspace_bytes) decode_ws;
    decltype(&cfp32_attention_decode) decode;
    decltype(&cfp32_cache_reserve) reserve;
    decltype(&cfp32_cache_append) append;
    decltype(&cfp32_cache_fork_workspace_bytes) fork_ws;
    decltype(&cfp32_cache_fork) fork;
    decltype(&cfp32_cache_free) free;
    decltype(&cfp32_cache_compact_workspace_bytes) compact_ws;
    decltype(&cfp32_cache_compact) compact;
} api;
PyObject *raw_stream, *scratch;

const at::Tensor *tensor(PyObject *o) { return THPVariable_Check(o) ? &THPVariable_Unpack(o) : nullptr; }

struct View {
    char *p;
    int64_t s0, s1;
};

// [n0, n1, D] with contiguous D.
bool heads(const at::Tensor *t, at::ScalarType type, c10::Device dev, View &v)
{
    if (!t || t->scalar_type() != type || t->device() != dev || t->dim() != 3) return false;
    if (t->stride(2) != 1 && t->size(2) > 1) return false;
    v = {(char *)t->data_ptr(), t->stride(0), t->stride(1)};
    return true;
}

struct PoolView {
    char *p;
    int64_t page, head, tok;
};
bool pool(const at::Tensor *t, at::ScalarType type, c10::Device dev, PoolView &v)
{
    if (!t || t->scalar_type() != type || t->device() != dev || t->dim() != 4) return false;
    if (t->stride(3) != 1 && t->size(3) > 1) return false;
    v = {(char *)t->data_ptr(), t->stride(0), t->stride(1), t->stride(2)};
    return true;
}

bool ints(const at::Tensor *t, c10::Device dev, int dim, int32_t *&p)
{
    if (!t || t->scalar_type() != at::kInt || t->device() != dev || t->dim() != dim) return false;
    if (t->stride(dim - 1) != 1 && t->size(dim - 1) > 1) return false;
    p = (int32_t *)t->data_ptr();
    return true;
}

int64_t ld(const at::Tensor &t) { return std::max(t.size(0) > 1 ? t.stride(0) : 0, t.size(1)); }

at::Tensor empty(at::IntArrayRef size, at::ScalarType type, c10::Device dev)
{
    return at::empty(size, at::TensorOptions().dtype(type).device(dev));
}

// The current stream; false with a Python error set.
bool stream_of(c10::Device dev, void *&st, PyObject *&st_obj)
{
    PyObject *i = PyLong_FromLong(dev.index());
    st_obj = i ? PyObject_CallOneArg(raw_stream, i) : nullptr;
    Py_XDECREF(i);
    if (!st_obj) return false;
    st = PyLong_AsVoidPtr(st_obj);
    return !(st == nullptr && PyErr_Occurred());
}

struct Call {
    void *stream = nullptr, *ws = nullptr;  // ws null: refused by the C ABI where one is needed
    PyObject *st_obj = nullptr, *buffer = nullptr;
    ~Call()
    {
        Py_XDECREF(st_obj);
        Py_XDECREF(buffer);
    }
    bool ready(c10::Device dev, size_t need)
    {
        if (!stream_of(dev, stream, st_obj)) return false;
        if (!need) return true;
        buffer = PyObject_CallFunction(scratch, "niO", (Py_ssize_t)need, (int)dev.index(), st_obj);
        if (!buffer) return false;
        const at::Tensor *t = tensor(buffer);
        if (t) ws = t->data_ptr();
        return true;
    }
};

PyObject *none() { Py_RETURN_NONE; }

bool kv_type(const at::Tensor &t, int &kv)
{
    kv = t.scalar_type() == at::kHalf ? CFP32_KV_F16 : CFP32_KV_F32;
    return t.scalar_type() == at::kHalf || t.scalar_type() == at::kFloat;
}

bool scale_of(PyObject *o, int64_t D, double &scale)
{
    if (o == Py_None) scale = 1.0 / std::sqrt((double)D);
    else if (PyFloat_CheckExact(o)) scale = PyFloat_AS_DOUBLE(o);
    else return false;
    return true;
}

// C++ exceptions (an allocation that fails) become Python errors.
template <PyObject *(*F)(PyObject *const *)>
PyObject *guarded(PyObject *, PyObject *const *args, Py_ssize_t n, Py_ssize_t want)
{
    if (n != want) return none();
    try {
        return F(args);
    } catch (const c10::OutOfMemoryError &e) {
        return none();  // the Python form raises it as torch does
    } catch (const std::exception &e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
        return nullptr;
    }
}

PyObject *tuple_of(std::initializer_list<at::Tensor> ts)
{
    PyObject *r = PyTuple_New((Py_ssize_t)ts.size());
    Py_ssize_t i = 0;
    if (r)
        for (const at::Tensor &t : ts) PyTuple_SET_ITEM(r, i++, THPVariable_Wrap(t));
    return r;
}

// (q, k, v, cu_q, cu_k or None, causal, scale or None, out or None)
PyObject *prompt(PyObject *const *a)
{
    const at::Tensor *q = tensor(a[0]), *k = tensor(a[1]), *v = tensor(a[2]), *cq = tensor(a[3]);
    const at::Tensor *ck = a[4] == Py_None ? cq : tensor(a[4]), *out = a[7] == Py_None ? nullptr : tensor(a[7]);
    if (!q || !k || !v || !cq || !ck || !q->is_cuda() || (a[7] != Py_None && !out)) return none();
    const c10::Device dev = q->device();
    int kv;
    View vq, vk, vv, vo;
    int32_t *pq, *pk;
    double scale;
    if (!kv_type(*k, kv) || !heads(q, at::kFloat, dev, vq) || !heads(k, k->scalar_type(), dev, vk) ||
        !heads(v, k->scalar_type(), dev, vv) || !ints(cq, dev, 1, pq) || !ints(ck, dev, 1, pk))
        return none();
    const int64_t Tq = q->size(0), Hq = q->size(1), D = q->size(2), Tk = k->size(0), Hkv = k->size(1), S = cq->size(0) - 1;
    if (D == 0 || k->size(2) != D || v->sizes() != k->sizes() || Hkv == 0 || Hq % Hkv || S < 0 || ck->size(0) != S + 1 ||
        !scale_of(a[6], D, scale) || !PyBool_Check(a[5]))
        return none();
    const at::Tensor o = out ? *out : empty(q->sizes(), at::kFloat, dev);
    if (o.sizes() != q->sizes() || !heads(&o, at::kFloat, dev, vo)) return none();
    Call c;
    const size_t need = api.prompt_ws(S, Tk, Hkv, D, kv);
    if (!c.ready(dev, need)) return nullptr;
    if (api.prompt((const float *)vq.p, vq.s0, vq.s1, vk.p, vk.s0, vk.s1, vv.p, vv.s0, vv.s1, kv, pq, pk, (float *)vo.p, vo.s0,
                   vo.s1, S, Tq, Tk, Hq, Hkv, D, a[5] == Py_True, scale, c.ws, need, c.stream) != CFP32_OK)
        return none();
    return THPVariable_Wrap(o);
}

// (q, k_pages, v_pages, table, lens, shared_pages, scale or None, out or None)
PyObject *decode(PyObject *const *a)
{
    const at::Tensor *q = tensor(a[0]), *k = tensor(a[1]), *v = tensor(a[2]), *table = tensor(a[3]), *lens = tensor(a[4]);
    const at::Tensor *out = a[7] == Py_None ? nullptr : tensor(a[7]);
    if (!q || !k || !v || !table || !lens || !q->is_cuda() || (a[7] != Py_None && !out) || !PyLong_CheckExact(a[5])) return none();
    const c10::Device dev = q->device();
    int kv;
    View vq, vo;
    PoolView pk, pv;
    int32_t *pt, *pl;
    double scale;
    const int64_t shared = PyLong_AsLongLong(a[5]);
    if (shared == -1 && PyErr_Occurred()) {
        PyErr_Clear();
        return none();
    }
    if (!kv_type(*k, kv) || !heads(q, at::kFloat, dev, vq) || !pool(k, k->scalar_type(), dev, pk) ||
        !pool(v, k->scalar_type(), dev, pv) || !ints(table, dev, 2, pt) || !ints(lens, dev, 1, pl))
        return none();
    const int64_t B = q->size(0), Hq = q->size(1), D = q->size(2), P = k->size(0), Hkv = k->size(1), page = k->size(2),
                  W = table->size(1);
    if (D == 0 || k->size(3) != D || v->sizes() != k->sizes() || Hkv == 0 || Hq % Hkv || table->size(0) != B ||
        lens->size(0) != B || !scale_of(a[6], D, scale))
        return none();
    const at::Tensor o = out ? *out : empty(q->sizes(), at::kFloat, dev);
    if (o.sizes() != q->sizes() || !heads(&o, at::kFloat, dev, vo)) return none();
    Call c;
    const size_t need = api.decode_ws(B, Hq, Hkv, D, W, page, shared, kv);
    if (!c.ready(dev, need)) return nullptr;
    if (api.decode((const float *)vq.p, vq.s0, vq.s1, pk.p, pk.page, pk.head, pk.tok, pv.p, pv.page, pv.head, pv.tok, kv, P, page,
                   pt, ld(*table), W, pl, shared, (float *)vo.p, vo.s0, vo.s1, B, Hq, Hkv, D, scale, c.ws, need, c.stream) != CFP32_OK)
        return none();
    return THPVariable_Wrap(o);
}

// (table, lens, refs, cu, page)
PyObject *reserve(PyObject *const *a)
{
    const at::Tensor *table = tensor(a[0]), *lens = tensor(a[1]), *refs = tensor(a[2]), *cu = tensor(a[3]);
    if (!table || !table->is_cuda() || !PyLong_CheckExact(a[4])) return none();
    const c10::Device dev = table->device();
    int32_t *pt, *pl, *pr, *pc;
    if (!ints(table, dev, 2, pt) || !ints(lens, dev, 1, pl) || !ints(refs, dev, 1, pr) || !ints(cu, dev, 1, pc)) return none();
    const int64_t S = table->size(0), W = table->size(1), P = refs->size(0), page = PyLong_AsLongLong(a[4]);
    if (page == -1 && PyErr_Occurred()) {
        PyErr_Clear();
        return none();
    }
    if (lens->size(0) != S || cu->size(0) != S + 1) return none();
    const at::Tensor to = empty({S, W}, at::kInt, dev), ro = empty({P}, at::kInt, dev);
    Call c;
    if (!c.ready(dev, 0)) return nullptr;
    if (api.reserve(pt, ld(*table), pl, pc, pr, (int32_t *)to.data_ptr(), ld(to), (int32_t *)ro.data_ptr(), nullptr, S, W, P, page,
                    c.stream) != CFP32_OK)
        return none();
    return tuple_of({to, ro});
}

// (k, v, cu, k_pages, v_pages, table, lens)
PyObject *append(PyObject *const *a)
{
    const at::Tensor *k = tensor(a[0]), *v = tensor(a[1]), *cu = tensor(a[2]), *kp = tensor(a[3]), *vp = tensor(a[4]),
                     *table = tensor(a[5]), *lens = tensor(a[6]);
    if (!k || !v || !kp || !vp || !table || !lens || !cu || !kp->is_cuda()) return none();
    const c10::Device dev = kp->device();
    int kv;
    View vk, vv;
    PoolView pk, pv;
    int32_t *pt, *pl, *pc;
    if (!kv_type(*kp, kv) || !heads(k, at::kFloat, dev, vk) || !heads(v, at::kFloat, dev, vv) ||
        !pool(kp, kp->scalar_type(), dev, pk) || !pool(vp, kp->scalar_type(), dev, pv) || !ints(table, dev, 2, pt) ||
        !ints(lens, dev, 1, pl) || !ints(cu, dev, 1, pc))
        return none();
    const int64_t P = kp->size(0), Hkv = kp->size(1), page = kp->size(2), D = kp->size(3), S = table->size(0), W = table->size(1);
    if (vp->sizes() != kp->sizes() || k->sizes() != v->sizes() || k->size(1) != Hkv || k->size(2) != D || lens->size(0) != S ||
        cu->size(0) != S + 1)
        return none();
    const at::Tensor lo = empty({S}, at::kInt, dev);
    Call c;
    if (!c.ready(dev, 0)) return nullptr;
    if (api.append((const float *)vk.p, vk.s0, vk.s1, (const float *)vv.p, vv.s0, vv.s1, pc, pl, (int32_t *)lo.data_ptr(), pk.p, pk.page,
                   pk.head, pk.tok, pv.p, pv.page, pv.head, pv.tok, kv, P, page, pt, ld(*table), S, W, k->size(0), Hkv, D,
                   c.stream) != CFP32_OK)
        return none();
    return THPVariable_Wrap(lo);
}

// (k_pages, v_pages, table, lens, refs, parents)
PyObject *fork(PyObject *const *a)
{
    const at::Tensor *kp = tensor(a[0]), *vp = tensor(a[1]), *table = tensor(a[2]), *lens = tensor(a[3]), *refs = tensor(a[4]),
                     *parents = tensor(a[5]);
    if (!kp || !kp->is_cuda()) return none();
    const c10::Device dev = kp->device();
    int kv;
    PoolView pk, pv;
    int32_t *pt, *pl, *pr, *pp;
    if (!kv_type(*kp, kv) || !pool(kp, kp->scalar_type(), dev, pk) || !pool(vp, kp->scalar_type(), dev, pv) ||
        !ints(table, dev, 2, pt) || !ints(lens, dev, 1, pl) || !ints(refs, dev, 1, pr) || !ints(parents, dev, 1, pp))
        return none();
    const int64_t P = kp->size(0), Hkv = kp->size(1), page = kp->size(2), D = kp->size(3), S = table->size(0), W = table->size(1),
                  C = parents->size(0);
    if (vp->sizes() != kp->sizes() || lens->size(0) != S || refs->size(0) != P) return none();
    const at::Tensor to = empty({C, W}, at::kInt, dev), lo = empty({C}, at::kInt, dev), ro = empty({P}, at::kInt, dev);
    Call c;
    const size_t need = api.fork_ws(C);
    if (!c.ready(dev, need)) return nullptr;
    if (api.fork(pk.p, pk.page, pk.head, pk.tok, pv.p, pv.page, pv.head, pv.tok, kv, P, page, Hkv, D, pt, ld(*table), pl, pr, pp,
                 (int32_t *)to.data_ptr(), W, (int32_t *)lo.data_ptr(), (int32_t *)ro.data_ptr(), nullptr, S, W, C, c.ws, need,
                 c.stream) != CFP32_OK)
        return none();
    return tuple_of({to, ro, lo});
}

// (rows, refs)
PyObject *free_pages(PyObject *const *a)
{
    const at::Tensor *rows = tensor(a[0]), *refs = tensor(a[1]);
    if (!refs || !refs->is_cuda()) return none();
    const c10::Device dev = refs->device();
    int32_t *pw, *pr;
    if (!ints(rows, dev, 2, pw) || !ints(refs, dev, 1, pr)) return none();
    const at::Tensor ro = empty(refs->sizes(), at::kInt, dev);
    Call c;
    if (!c.ready(dev, 0)) return nullptr;
    if (api.free(pw, ld(*rows), pr, (int32_t *)ro.data_ptr(), rows->size(0), rows->size(1), refs->size(0), c.stream) != CFP32_OK)
        return none();
    return THPVariable_Wrap(ro);
}

// (k_pages, v_pages, table, refs)
PyObject *compact(PyObject *const *a)
{
    const at::Tensor *kp = tensor(a[0]), *vp = tensor(a[1]), *table = tensor(a[2]), *refs = tensor(a[3]);
    if (!kp || !kp->is_cuda()) return none();
    const c10::Device dev = kp->device();
    int kv;
    PoolView pk, pv;
    int32_t *pt, *pr;
    if (!kv_type(*kp, kv) || !pool(kp, kp->scalar_type(), dev, pk) || !pool(vp, kp->scalar_type(), dev, pv) ||
        !ints(table, dev, 2, pt) || !ints(refs, dev, 1, pr))
        return none();
    const int64_t P = kp->size(0), Hkv = kp->size(1), page = kp->size(2), D = kp->size(3), S = table->size(0), W = table->size(1);
    if (vp->sizes() != kp->sizes() || refs->size(0) != P) return none();
    const at::Tensor to = empty({S, W}, at::kInt, dev), ro = empty({P}, at::kInt, dev), live = empty({1}, at::kInt, dev);
    Call c;
    const size_t need = api.compact_ws(P);
    if (!c.ready(dev, need)) return nullptr;
    if (api.compact(pk.p, pk.page, pk.head, pk.tok, pv.p, pv.page, pv.head, pv.tok, kv, P, page, Hkv, D, pt, ld(*table), pr,
                    (int32_t *)to.data_ptr(), ld(to), (int32_t *)ro.data_ptr(), (int32_t *)live.data_ptr(), S, W, c.ws, need,
                    c.stream) != CFP32_OK)
        return none();
    return tuple_of({to, ro, live});
}

// (entry points' addresses in Api's order, raw_stream, scratch)
PyObject *bind(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    constexpr Py_ssize_t count = sizeof(Api) / sizeof(void *);
    if (n != 3 || !PyTuple_Check(a[0]) || PyTuple_GET_SIZE(a[0]) != count) {
        PyErr_SetString(PyExc_TypeError, "bind: wrong arguments");
        return nullptr;
    }
    void *p[count];
    for (Py_ssize_t i = 0; i < count; ++i) {
        p[i] = PyLong_AsVoidPtr(PyTuple_GET_ITEM(a[0], i));
        if (!p[i]) {
            if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, "bind: a null entry point");
            return nullptr;
        }
    }
    memcpy(&api, p, sizeof api);
    Py_INCREF(a[1]);
    Py_INCREF(a[2]);
    Py_XSETREF(raw_stream, a[1]);
    Py_XSETREF(scratch, a[2]);
    Py_RETURN_NONE;
}

#define CFP32_HELPER(NAME, FUNC, N)                                               \
    PyObject *NAME##_call(PyObject *m, PyObject *const *a, Py_ssize_t n) { return guarded<FUNC>(m, a, n, N); }
CFP32_HELPER(prompt, prompt, 8)
CFP32_HELPER(decode, decode, 8)
CFP32_HELPER(reserve, reserve, 5)
CFP32_HELPER(append, append, 7)
CFP32_HELPER(fork, fork, 6)
CFP32_HELPER(free, free_pages, 2)
CFP32_HELPER(compact, compact, 4)
#undef CFP32_HELPER

#define CFP32_METHOD(NAME, FUNC) {NAME, (PyCFunction)(void (*)(void))FUNC, METH_FASTCALL, nullptr}
PyMethodDef methods[] = {CFP32_METHOD("bind", bind),
                         CFP32_METHOD("attention_prompt", prompt_call),
                         CFP32_METHOD("attention_decode", decode_call),
                         CFP32_METHOD("cache_reserve", reserve_call),
                         CFP32_METHOD("cache_append", append_call),
                         CFP32_METHOD("cache_fork", fork_call),
                         CFP32_METHOD("cache_free", free_call),
                         CFP32_METHOD("cache_compact", compact_call),
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_helpers", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__helpers(void) { return PyModule_Create(&module); }
