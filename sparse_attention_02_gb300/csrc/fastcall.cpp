/* The calls of the Python binding that go out once per layer and token, with
 * their argument checks in C: on a few tokens the interpreter's own checks and
 * the marshalling of twenty arguments take the host longer than the kernels
 * take the GPU (a decode step's cache append: 10.6 us of host time in Python).
 *
 * Tensors are read through PyTorch's own C++ headers (their attributes asked for
 * in Python take 0.4 us a tensor, and a call has up to ten).
 *
 * Every function takes the arguments of the binding's function of that name,
 * in order, and either makes the call, returning the library's status, or
 * returns NotImplemented without having done anything, where an argument is
 * not plainly what the call needs; the Python form then finds out what is
 * wrong and says so, or makes the call itself.
 */
#define PY_SSIZE_T_CLEAN
#include <Python.h>
#include <dlfcn.h>
#include <stdint.h>
#include <torch/csrc/autograd/python_variable.h>

#include "../../include/dsa.h"

namespace {

PyObject *s_cuda_stream;
PyObject *get_device_fn, *get_stream_fn;               /* current device, its raw stream */
PyObject *alloc_fn, *free_fn;                          /* PyTorch's allocator: address of (bytes, stream), its release */

decltype(&dsa_rmsnorm) f_rmsnorm;
decltype(&dsa_rmsnorm_backward) f_rmsnorm_backward;
decltype(&dsa_rmsnorm_backward_workspace_size) f_rmsnorm_backward_ws;
decltype(&dsa_cache_append) f_cache_append;
decltype(&dsa_rope_queries) f_rope_queries;
decltype(&dsa_index_rope_backward) f_index_rope_backward;
decltype(&dsa_mla_decode_paged) f_mla_decode;
decltype(&dsa_mla_decode_workspace_size) f_mla_decode_ws;

/* An address as whatever the library takes it for. */
struct Address {
    void *v = nullptr;
    template <typename T> operator T *() const { return static_cast<T *>(v); }
};

/* What is known of a tensor argument. */
struct Arg {
    int nd = 0;
    int64_t dim[3] = {}, stride[3] = {};
    bool contiguous = false;
    int dtype = 0; /* DSA_BF16, DSA_FP32, or one of the below */
    Address p;
};
enum { K_FP64 = 10, K_INT32, K_UINT8, K_ANY /* bf16 or fp32 */ };

/* What t is; false where it is not a plain tensor of the device with up to 3 dimensions and the type. */
bool look(PyObject *t, long cur, int want, Arg *a)
{
    if (!THPVariable_Check(t))
        return false;
    const at::Tensor &v = THPVariable_Unpack(t);
    switch (v.scalar_type()) {
    case at::kBFloat16: a->dtype = DSA_BF16; break;
    case at::kFloat: a->dtype = DSA_FP32; break;
    case at::kDouble: a->dtype = K_FP64; break;
    case at::kInt: a->dtype = K_INT32; break;
    case at::kByte: a->dtype = K_UINT8; break;
    default: return false;
    }
    if (want == K_ANY ? (a->dtype != DSA_BF16 && a->dtype != DSA_FP32) : a->dtype != want)
        return false;
    if (!v.is_cuda() || v.layout() != at::kStrided || v.get_device() != cur || v.dim() > 3)
        return false;
    a->nd = (int)v.dim();
    for (int i = 0; i < a->nd; ++i) {
        a->dim[i] = v.size(i);
        a->stride[i] = v.stride(i);
    }
    a->contiguous = v.is_contiguous();
    a->p.v = v.data_ptr(); /* throws, or is null, where there is no memory behind it */
    return a->p.v || v.numel() == 0;
}

int64_t as_int(PyObject *o, int *ok)
{
    int64_t v = o ? PyLong_AsLongLong(o) : -1;
    if (!o || (v == -1 && PyErr_Occurred()))
        *ok = 0;
    Py_XDECREF(o);
    return v;
}

/* A contiguous tensor of the shape (n1, n2 < 0: fewer dimensions). */
int at(PyObject *t, long cur, int want, int64_t n0, int64_t n1, int64_t n2, Arg *a)
{
    return look(t, cur, want, a) && a->nd == 1 + (n1 >= 0) + (n2 >= 0) && a->dim[0] == n0 && (n1 < 0 || a->dim[1] == n1) &&
           (n2 < 0 || a->dim[2] == n2) && a->contiguous;
}

/* A 2-D tensor whose rows may be apart; *ld is their distance. */
int at_rows(PyObject *t, long cur, int want, int64_t n0, int64_t n1, Arg *a, int64_t *ld)
{
    if (!look(t, cur, want, a) || a->nd != 2 || a->dim[0] != n0 || a->dim[1] != n1)
        return 0;
    *ld = n0 > 1 ? a->stride[0] : n1;
    return (n1 == 1 || a->stride[1] == 1) && *ld >= n1;
}

/* Device, and the stream of the call: stream's, or the device's current one. */
int where(PyObject *stream, long *cur, dsa_stream_t *s)
{
    int ok = 1;
    *cur = (long)as_int(PyObject_CallNoArgs(get_device_fn), &ok);
    if (!ok)
        return 0;
    PyObject *v;
    if (stream == Py_None) {
        PyObject *c = PyLong_FromLong(*cur);
        v = c ? PyObject_CallOneArg(get_stream_fn, c) : NULL;
        Py_XDECREF(c);
    } else {
        v = PyObject_GetAttr(stream, s_cuda_stream);
    }
    *s = (dsa_stream_t)(uintptr_t)as_int(v, &ok);
    return ok;
}

/* Workspace of `need` bytes: the caller's, or one of PyTorch's allocator on the call's stream, to be given back
 * (release) once the call is enqueued: what the allocator hands out next on that stream runs after it.  A tensor
 * for it would take the host as long as the rest of a small call (517 x 1111 norm backward: 11.3 us, 6.2 without). */
int workspace(PyObject *ws, dsa_stream_t stream, long cur, size_t need, void **p, size_t *bytes, PyObject **keep)
{
    Arg a;
    int ok = 1;
    *keep = NULL;
    *p = NULL;
    *bytes = 0;
    if (ws != Py_None) {
        if (!look(ws, cur, K_UINT8, &a) || a.nd != 1 || !a.contiguous)
            return 0;
        *p = a.p;
        *bytes = (size_t)a.dim[0];
        return 1;
    }
    if (!need)
        return 1;
    *keep = PyObject_CallFunction(alloc_fn, "nK", (Py_ssize_t)need, (unsigned long long)(uintptr_t)stream);
    if (!*keep)
        return 0;
    Py_INCREF(*keep);
    *p = (void *)(uintptr_t)as_int(*keep, &ok);
    *bytes = need;
    return ok;
}

void release(PyObject *keep)
{
    if (!keep)
        return;
    PyObject *done = PyObject_CallOneArg(free_fn, keep);
    if (!done)
        PyErr_Clear();
    Py_XDECREF(done);
    Py_DECREF(keep);
}

/* Numbers: plain Python ones only. */
int number(PyObject *o, double *v)
{
    if (!PyFloat_Check(o) && !PyLong_Check(o))
        return 0;
    *v = PyFloat_AsDouble(o);
    return !(*v == -1.0 && PyErr_Occurred());
}

int integer(PyObject *o, int *v)
{
    if (!PyLong_Check(o))
        return 0;
    long x = PyLong_AsLong(o);
    *v = (int)x;
    return x >= INT32_MIN && x <= INT32_MAX && !PyErr_Occurred();
}

PyObject *not_plain(PyObject *keep)
{
    PyErr_Clear();
    release(keep);
    Py_RETURN_NOTIMPLEMENTED;
}

#define FITS(n) ((n) <= INT32_MAX)

/* The library's call, with other Python threads free to run. */
#define CALL(rc, expr)                                                                                                              \
    do {                                                                                                                            \
        Py_BEGIN_ALLOW_THREADS rc = (expr);                                                                                         \
        Py_END_ALLOW_THREADS                                                                                                        \
    } while (0)

/* x, weight, eps, out, residual, residual_out, codes, scale, block, scale_mode, stream */
PyObject *py_rmsnorm(PyObject *const *v, Py_ssize_t n)
{
    long cur;
    dsa_stream_t st;
    Arg x, w, o, r, h, c, s;
    int64_t ldx, ldo = 0, ldr = 0, ldh = 0;
    double eps;
    int block, mode;
    if (n != 11 || !where(v[10], &cur, &st) || !number(v[2], &eps) || !integer(v[8], &block) || !integer(v[9], &mode) ||
        !look(v[0], cur, K_ANY, &x) || x.nd != 2 || !FITS(x.dim[1]))
        return not_plain(NULL);
    const int64_t rows = x.dim[0], cols = x.dim[1];
    ldx = rows > 1 ? x.stride[0] : cols;
    if ((cols != 1 && x.stride[1] != 1) || ldx < cols || !at(v[1], cur, K_ANY, cols, -1, -1, &w) ||
        (v[3] != Py_None && !at_rows(v[3], cur, x.dtype, rows, cols, &o, &ldo)) ||
        (v[4] != Py_None && !at_rows(v[4], cur, x.dtype, rows, cols, &r, &ldr)) ||
        (v[5] != Py_None && !at_rows(v[5], cur, x.dtype, rows, cols, &h, &ldh)) ||
        (v[6] != Py_None && !at(v[6], cur, K_UINT8, rows, cols, -1, &c)))
        return not_plain(NULL);
    if (v[7] != Py_None) {
        const int64_t parts = block > 0 ? (cols + block - 1) / block : 1;
        if (!look(v[7], cur, DSA_FP32, &s) || s.dim[0] != rows || !s.contiguous ||
            !((s.nd == 2 && s.dim[1] == parts) || (s.nd == 1 && parts == 1)))
            return not_plain(NULL);
    }
    int rc;
    CALL(rc, f_rmsnorm(x.p, ldx, r.p, ldr, w.p, rows, (int)cols, x.dtype, w.dtype, (float)eps, h.p, ldh, o.p, ldo,
                                     c.p, s.p, block, mode, st));
    return PyLong_FromLong(rc);
}

/* dy, h, weight, eps, dx, dweight, dres, workspace, stream */
PyObject *py_rmsnorm_backward(PyObject *const *v, Py_ssize_t n)
{
    long cur;
    dsa_stream_t st;
    Arg dy, h, w, dx, dw, e;
    double eps;
    void *ws;
    size_t bytes;
    PyObject *keep = NULL;
    if (n != 9 || !where(v[8], &cur, &st) || !number(v[3], &eps) || !look(v[1], cur, K_ANY, &h) || h.nd != 2 ||
        !FITS(h.dim[1]) || !h.contiguous)
        return not_plain(NULL);
    const int64_t rows = h.dim[0], cols = h.dim[1];
    if (!at(v[0], cur, h.dtype, rows, cols, -1, &dy) || !at(v[2], cur, K_ANY, cols, -1, -1, &w) ||
        !at(v[4], cur, h.dtype, rows, cols, -1, &dx) || !at(v[5], cur, DSA_FP32, cols, -1, -1, &dw) ||
        (v[6] != Py_None && !at(v[6], cur, h.dtype, rows, cols, -1, &e)) ||
        !workspace(v[7], st, cur, v[7] == Py_None ? f_rmsnorm_backward_ws(rows, (int)cols) : 0, &ws, &bytes, &keep))
        return not_plain(keep);
    int rc;
    CALL(rc, f_rmsnorm_backward(dy.p, h.p, w.p, e.p, rows, (int)cols, h.dtype, w.dtype, (float)eps, dx.p, dw.p, ws, bytes, st));
    release(keep);
    return PyLong_FromLong(rc);
}

/* pos, block_table, inv_freq, kv, kv_pool, kI, k8_pool, ks_pool, seq, kv_weight, eps, scale_mode, stream */
PyObject *py_cache_append(PyObject *const *v, Py_ssize_t n)
{
    long cur;
    dsa_stream_t st;
    Arg pos, bt, fr, kv, kp, k, k8, ks, seq, w;
    int64_t ld = 0, ldI = 0;
    double eps;
    int mode;
    const int with_kv = n == 13 && v[3] != Py_None, with_k = n == 13 && v[5] != Py_None;
    if (n != 13 || (!with_kv && !with_k) || !where(v[12], &cur, &st) || !number(v[10], &eps) || !integer(v[11], &mode) ||
        !look(v[0], cur, K_INT32, &pos) || pos.nd != 1 || !FITS(pos.dim[0]) || !pos.contiguous ||
        !look(v[1], cur, K_INT32, &bt) || bt.nd != 2 || !FITS(bt.dim[0]) || !FITS(bt.dim[1]) || !bt.contiguous ||
        !at(v[2], cur, K_FP64, 32, -1, -1, &fr))
        return not_plain(NULL);
    const int64_t T = pos.dim[0];
    int64_t pages = 0, page = 0;
    if (with_kv) {
        if (!at_rows(v[3], cur, DSA_BF16, T, 576, &kv, &ld) || !look(v[4], cur, DSA_BF16, &kp) || kp.nd != 3 ||
            kp.dim[2] != 576 || !kp.contiguous || (v[9] != Py_None && !at(v[9], cur, K_ANY, 512, -1, -1, &w)))
            return not_plain(NULL);
        pages = kp.dim[0], page = kp.dim[1];
    }
    if (with_k) {
        if (!at_rows(v[5], cur, K_ANY, T, 128, &k, &ldI) || !look(v[6], cur, K_UINT8, &k8) || k8.nd != 3 || k8.dim[2] != 128 ||
            !k8.contiguous || (with_kv && (k8.dim[0] != pages || k8.dim[1] != page)))
            return not_plain(NULL);
        pages = k8.dim[0], page = k8.dim[1];
        if (!at(v[7], cur, DSA_FP32, pages, page, -1, &ks))
            return not_plain(NULL);
    }
    if (!FITS(pages) || !FITS(page) || (v[8] != Py_None && !at(v[8], cur, K_INT32, T, -1, -1, &seq)))
        return not_plain(NULL);
    int rc;
    CALL(rc, f_cache_append(pos.p, seq.p, (int)T, bt.p, (int)bt.dim[0], (int)bt.dim[1], (int)pages, (int)page, fr.p,
                                          kv.p, ld, w.p, w.dtype, (float)eps, kp.p, k.p, ldI, k.dtype, mode, k8.p, ks.p, st));
    return PyLong_FromLong(rc);
}

/* pos, inv_freq, q_rope, q, qI, q8, q_scale, scale_mode, stream */
PyObject *py_rope_queries(PyObject *const *v, Py_ssize_t n)
{
    long cur;
    dsa_stream_t st;
    Arg pos, fr, r, q, qi, q8, s;
    int64_t H = 0, HI = 0;
    int mode;
    const int with_r = n == 9 && v[2] != Py_None, with_i = n == 9 && v[4] != Py_None;
    if (n != 9 || (!with_r && !with_i) || !where(v[8], &cur, &st) || !integer(v[7], &mode) || !look(v[0], cur, K_INT32, &pos) ||
        pos.nd != 1 || !FITS(pos.dim[0]) || !pos.contiguous || !at(v[1], cur, K_FP64, 32, -1, -1, &fr))
        return not_plain(NULL);
    const int64_t T = pos.dim[0];
    if (with_r) {
        if (!look(v[2], cur, DSA_BF16, &r) || r.nd != 3 || r.dim[0] != T || r.dim[2] != 64 || r.stride[2] != 1)
            return not_plain(NULL);
        H = r.dim[1];
        if (!FITS(H) || !at(v[3], cur, DSA_BF16, T, H, 576, &q))
            return not_plain(NULL);
    }
    if (with_i) {
        if (!look(v[4], cur, K_ANY, &qi) || qi.nd != 3 || qi.dim[0] != T || qi.dim[2] != 128 || !qi.contiguous)
            return not_plain(NULL);
        HI = qi.dim[1];
        if (!FITS(HI) || !at(v[5], cur, K_UINT8, T, HI, 128, &q8) || !at(v[6], cur, DSA_FP32, T, -1, -1, &s))
            return not_plain(NULL);
    }
    int rc;
    CALL(rc, f_rope_queries(pos.p, fr.p, (int)T, r.p, T > 1 ? r.stride[0] : 0, H > 1 ? r.stride[1] : 0, (int)H, q.p,
                                          qi.p, (int)HI, with_i ? qi.dtype : DSA_BF16, mode, q8.p, s.p, st));
    return PyLong_FromLong(rc);
}

/* g, pos, inv_freq, dx, stream */
PyObject *py_index_rope_backward(PyObject *const *v, Py_ssize_t n)
{
    long cur;
    dsa_stream_t st;
    Arg g, pos, fr, dx;
    if (n != 5 || !where(v[4], &cur, &st) || !look(v[0], cur, DSA_FP32, &g) || g.nd < 2 || g.dim[g.nd - 1] != 128 ||
        !FITS(g.dim[0]) || !FITS(g.dim[1]) || !g.contiguous || !at(v[1], cur, K_INT32, g.dim[0], -1, -1, &pos) ||
        !at(v[2], cur, K_FP64, 32, -1, -1, &fr) || !at(v[3], cur, K_ANY, g.dim[0], g.dim[1], g.nd == 3 ? 128 : -1, &dx))
        return not_plain(NULL);
    int rc;
    CALL(rc, f_index_rope_backward(g.p, pos.p, fr.p, (int)g.dim[0], g.nd == 3 ? (int)g.dim[1] : 1, dx.p, dx.dtype, st));
    return PyLong_FromLong(rc);
}

/* q, kv_pool, block_table, ctx_len, sm_scale, out, lse, workspace, stream */
PyObject *py_mla_decode_paged(PyObject *const *v, Py_ssize_t n)
{
    long cur;
    dsa_stream_t st;
    Arg q, kv, bt, ctx, out, lse;
    double scale;
    void *ws;
    size_t bytes;
    PyObject *keep = NULL;
    if (n != 9 || !where(v[8], &cur, &st) || !number(v[4], &scale) || !look(v[0], cur, DSA_BF16, &q) || q.nd != 3 ||
        q.dim[2] != 576 || !FITS(q.dim[0]) || !FITS(q.dim[1]) || !q.contiguous || !look(v[1], cur, DSA_BF16, &kv) ||
        kv.nd != 3 || kv.dim[2] != 576 || !FITS(kv.dim[0]) || !FITS(kv.dim[1]) || !kv.contiguous ||
        !look(v[2], cur, K_INT32, &bt) || bt.nd != 2 || bt.dim[0] != q.dim[0] || !FITS(bt.dim[1]) || !bt.contiguous ||
        !at(v[3], cur, K_INT32, q.dim[0], -1, -1, &ctx) || !at(v[5], cur, DSA_BF16, q.dim[0], q.dim[1], 512, &out) ||
        !at(v[6], cur, DSA_FP32, q.dim[0], q.dim[1], -1, &lse) ||
        !workspace(v[7], st, cur, v[7] == Py_None ? f_mla_decode_ws((int)q.dim[0], (int)q.dim[1]) : 0, &ws, &bytes, &keep))
        return not_plain(keep);
    int rc;
    CALL(rc, f_mla_decode(q.p, kv.p, (int)kv.dim[0], (int)kv.dim[1], bt.p, (int)bt.dim[1], ctx.p, (int)q.dim[0],
                                (int)q.dim[1], (float)scale, out.p, lse.p, ws, bytes, st));
    release(keep);
    return PyLong_FromLong(rc);
}

/* init(path of the library, current device, raw stream of a device, alloc(bytes, stream), free(address)) */
PyObject *py_init(PyObject *, PyObject *args)
{
    const char *path;
    if (!PyArg_ParseTuple(args, "sOOOO", &path, &get_device_fn, &get_stream_fn, &alloc_fn, &free_fn))
        return NULL;
    void *lib = dlopen(path, RTLD_NOW | RTLD_LOCAL);
    if (!lib) {
        PyErr_SetString(PyExc_RuntimeError, dlerror());
        return NULL;
    }
    f_rmsnorm = (decltype(f_rmsnorm))dlsym(lib, "dsa_rmsnorm");
    f_rmsnorm_backward = (decltype(f_rmsnorm_backward))dlsym(lib, "dsa_rmsnorm_backward");
    f_rmsnorm_backward_ws = (decltype(f_rmsnorm_backward_ws))dlsym(lib, "dsa_rmsnorm_backward_workspace_size");
    f_cache_append = (decltype(f_cache_append))dlsym(lib, "dsa_cache_append");
    f_rope_queries = (decltype(f_rope_queries))dlsym(lib, "dsa_rope_queries");
    f_index_rope_backward = (decltype(f_index_rope_backward))dlsym(lib, "dsa_index_rope_backward");
    f_mla_decode = (decltype(f_mla_decode))dlsym(lib, "dsa_mla_decode_paged");
    f_mla_decode_ws = (decltype(f_mla_decode_ws))dlsym(lib, "dsa_mla_decode_workspace_size");
    if (!f_rmsnorm || !f_rmsnorm_backward || !f_rmsnorm_backward_ws || !f_cache_append || !f_rope_queries || !f_index_rope_backward ||
        !f_mla_decode || !f_mla_decode_ws) {
        PyErr_SetString(PyExc_RuntimeError, "the library lacks an entry point");
        return NULL;
    }
    PyObject *kept[] = {get_device_fn, get_stream_fn, alloc_fn, free_fn};
    for (size_t i = 0; i < sizeof kept / sizeof *kept; ++i)
        Py_INCREF(kept[i]);
    Py_RETURN_NONE;
}

/* What PyTorch throws leaves the call to the Python form, which then raises it. */
template <PyObject *(*F)(PyObject *const *, Py_ssize_t)> PyObject *entry(PyObject *, PyObject *const *v, Py_ssize_t n)
{
    try {
        return F(v, n);
    } catch (...) {
        return not_plain(NULL);
    }
}

#define FAST(name) {#name, (PyCFunction)(void (*)(void))entry<py_##name>, METH_FASTCALL, NULL}
PyMethodDef methods[] = {FAST(rmsnorm),
                                FAST(rmsnorm_backward),
                                FAST(cache_append),
                                FAST(rope_queries),
                                FAST(index_rope_backward),
                                FAST(mla_decode_paged),
                                {"init", py_init, METH_VARARGS, NULL},
                                {NULL, NULL, 0, NULL}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_fastcall", NULL, -1, methods, NULL, NULL, NULL, NULL};

} // namespace

PyMODINIT_FUNC PyInit__fastcall(void)
{
    s_cuda_stream = PyUnicode_InternFromString("cuda_stream");
    return PyModule_Create(&module);
}
