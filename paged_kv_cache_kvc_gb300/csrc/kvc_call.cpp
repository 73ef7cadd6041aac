// CPython module `_kvc_call`: argument checks and marshalling of the rotary write and of attention with
// modified scores, for the Python binding.  A decode step's smallest calls take a few microseconds on the
// GPU; checking nine tensors and filling a C call through ctypes took 16 on the host.  Here a call reads the
// tensors' headers directly and takes about 5, most of it the launch.
//
// Every function takes its arguments by position, raises ValueError for a tensor that is not what the call
// takes, and returns the library's status.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cmath>

#include "../../include/kvc.h"

namespace {

struct Bad {};   // a Python error is set

// Other Python threads run while a launch is under way.
struct Unlocked {
    PyThreadState *state = PyEval_SaveThread();
    ~Unlocked() { PyEval_RestoreThread(state); }
};

[[noreturn]] void fail(const char *name, const char *what)
{
    PyErr_Format(PyExc_ValueError, "%s %s", name, what);
    throw Bad{};
}

const at::Tensor *tensor(PyObject *o, at::ScalarType type, int64_t device, const char *name, bool optional = false)
{
    if (o == Py_None) {
        if (optional) return nullptr;
        fail(name, "is required");
    }
    if (!THPVariable_Check(o)) fail(name, "must be a CUDA tensor");
    const at::Tensor &t = THPVariable_Unpack(o);
    if (!t.is_cuda()) fail(name, "must be a CUDA tensor");
    if (t.scalar_type() != type) {
        PyErr_Format(PyExc_ValueError, "%s must be %s, got %s", name, at::toString(type), at::toString(t.scalar_type()));
        throw Bad{};
    }
    if (t.get_device() != device) {
        PyErr_Format(PyExc_ValueError, "%s is on cuda:%d, the pool on cuda:%d", name, static_cast<int>(t.get_device()),
                     static_cast<int>(device));
        throw Bad{};
    }
    return &t;
}

// A contiguous tensor of the given shape (-1: any size).
template <size_t N>
const at::Tensor *shaped(PyObject *o, at::ScalarType type, int64_t device, const int64_t (&shape)[N], const char *name,
                         bool optional = false)
{
    const at::Tensor *t = tensor(o, type, device, name, optional);
    if (!t) return nullptr;
    bool ok = t->dim() == static_cast<int64_t>(N);
    for (size_t i = 0; ok && i < N; ++i) ok = shape[i] < 0 || t->size(i) == shape[i];
    if (!ok) fail(name, "has the wrong shape");
    if (!t->is_contiguous()) fail(name, "must be contiguous");
    return t;
}

void *ptr(const at::Tensor *t) { return t ? t->data_ptr() : nullptr; }

// bf16 [rows][heads][d]: rows may be strided, a row's heads must be contiguous.
struct Rows {
    void *data = nullptr;
    int64_t stride = 0;
    int64_t heads = 0;
};

Rows head_rows(PyObject *o, int64_t device, int64_t rows, int64_t heads, int64_t d, const char *name)
{
    const at::Tensor *t = tensor(o, at::kBFloat16, device, name);
    if (t->dim() != 3 || t->size(0) != rows || (heads >= 0 && t->size(1) != heads) || t->size(2) != d)
        fail(name, "has the wrong shape");
    Rows r;
    r.heads = t->size(1);
    if (t->numel() > 0 && (t->stride(2) != 1 || (r.heads > 1 && t->stride(1) != d)))
        fail(name, "must have a row's heads contiguous");
    r.data = t->data_ptr();
    r.stride = rows > 1 ? t->stride(0) : r.heads * d;
    return r;
}

int64_t integer(PyObject *o, const char *name)
{
    const long long v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred()) {
        PyErr_Clear();
        fail(name, "must be an integer");
    }
    return v;
}

int32_t int32(PyObject *o, const char *name)
{
    const int64_t v = integer(o, name);
    if (v != static_cast<int32_t>(v)) fail(name, "is out of range");
    return static_cast<int32_t>(v);
}

// What a call needs of its pool: (handle, device, head_dim, num_kv_heads), a tuple that the Pool keeps.
struct PoolArgs {
    kvc_pool *pool;
    int64_t device, d, heads;
};

PoolArgs pool_args(PyObject *o)
{
    if (!PyTuple_CheckExact(o) || PyTuple_GET_SIZE(o) != 4) fail("pool", "must be an open Pool");
    PoolArgs p;
    p.pool = reinterpret_cast<kvc_pool *>(PyLong_AsVoidPtr(PyTuple_GET_ITEM(o, 0)));
    if (PyErr_Occurred()) throw Bad{};
    if (!p.pool) fail("pool", "is closed");
    p.device = integer(PyTuple_GET_ITEM(o, 1), "device");
    p.d = integer(PyTuple_GET_ITEM(o, 2), "head_dim");
    p.heads = integer(PyTuple_GET_ITEM(o, 3), "num_kv_heads");
    return p;
}

// The given stream (an integer handle), or torch's current stream of the pool's device.
void *stream_of(PyObject *o, const PoolArgs &p)
{
    if (o == Py_None) return c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(p.device)).stream();
    void *s = PyLong_AsVoidPtr(o);
    if (PyErr_Occurred()) throw Bad{};
    return s;
}

void count(Py_ssize_t n, Py_ssize_t want)
{
    if (n != want) {
        PyErr_Format(PyExc_TypeError, "%zd arguments, %zd wanted", n, want);
        throw Bad{};
    }
}

// (rotary_dim, interleaved, inv_freq, q_norm, k_norm, eps)
kvc_rope rope_of(PyObject *o, const PoolArgs &p)
{
    if (!PyTuple_CheckExact(o) || PyTuple_GET_SIZE(o) != 6) fail("rope", "must be a Rope");
    kvc_rope r{};
    r.rotary_dim = int32(PyTuple_GET_ITEM(o, 0), "rotary_dim");
    r.interleaved = int32(PyTuple_GET_ITEM(o, 1), "interleaved");
    r.inv_freq = static_cast<const float *>(ptr(shaped(PyTuple_GET_ITEM(o, 2), at::kFloat, p.device, {r.rotary_dim / 2}, "inv_freq", true)));
    r.q_norm = ptr(shaped(PyTuple_GET_ITEM(o, 3), at::kBFloat16, p.device, {p.d}, "q_norm", true));
    r.k_norm = ptr(shaped(PyTuple_GET_ITEM(o, 4), at::kBFloat16, p.device, {p.d}, "k_norm", true));
    r.norm_eps = static_cast<float>(PyFloat_AsDouble(PyTuple_GET_ITEM(o, 5)));
    if (PyErr_Occurred()) throw Bad{};
    return r;
}

// (pool, layer, block_tables, start, cu or None, q or None, k, v, q_out or None, rope, stream)
long rope_write(PyObject *const *a, Py_ssize_t n)
{
    count(n, 11);
    const PoolArgs p = pool_args(a[0]);
    const int32_t layer = int32(a[1], "layer");
    const at::Tensor *bt = shaped(a[2], at::kInt, p.device, {-1, -1}, "block_tables");
    const int64_t B = bt->size(0);
    const at::Tensor *start = shaped(a[3], at::kInt, p.device, {B}, "seq_lens / start_pos");
    const at::Tensor *cu = shaped(a[4], at::kInt, p.device, {B + 1}, "cu_tokens", true);
    const at::Tensor *kt = tensor(a[6], at::kBFloat16, p.device, "k");
    const int64_t rows = cu ? (kt->dim() > 0 ? kt->size(0) : 0) : B;
    const Rows k = head_rows(a[6], p.device, rows, p.heads, p.d, "k");
    const Rows v = head_rows(a[7], p.device, rows, p.heads, p.d, "v");
    if ((a[5] == Py_None) != (a[8] == Py_None)) fail("q and q_out", "go together");
    Rows q;
    void *q_out = nullptr;
    if (a[5] != Py_None) {
        q = head_rows(a[5], p.device, rows, -1, p.d, "q");
        q_out = ptr(shaped(a[8], at::kBFloat16, p.device, {rows, q.heads, p.d}, "q_out"));
    }
    const kvc_rope rope = rope_of(a[9], p);
    void *s = stream_of(a[10], p);
    const int32_t mb = static_cast<int32_t>(bt->size(1)), b32 = static_cast<int32_t>(B), hq = static_cast<int32_t>(q.heads);
    const int32_t *table = static_cast<const int32_t *>(ptr(bt)), *st = static_cast<const int32_t *>(ptr(start));
    const Unlocked unlocked;
    if (!cu)
        return kvc_rope_append(p.pool, layer, table, mb, st, b32, q.data, q.stride, hq, k.data, k.stride, v.data, v.stride,
                               &rope, q_out, s);
    return kvc_rope_write_tokens(p.pool, layer, table, mb, st, static_cast<const int32_t *>(ptr(cu)), b32, rows, q.data,
                                 q.stride, hq, k.data, k.stride, v.data, v.stride, &rope, q_out, s);
}

struct ModArgs {
    const at::Tensor *q, *out, *lse, *ws;
    kvc_score_mod mod;
    bool has_mod;
    float scale;
};

// q, out, lse or None, (softcap, window, sink, prefix, alibi or None, doc_start or None) or None, scale or None,
// workspace or None
ModArgs mod_args(const PoolArgs &p, PyObject *q, PyObject *out, PyObject *lse, PyObject *mod, PyObject *scale, PyObject *ws)
{
    ModArgs m{};
    m.q = shaped(q, at::kBFloat16, p.device, {-1, -1, p.d}, "q");
    const int64_t n = m.q->size(0), h = m.q->size(1);
    m.out = shaped(out, at::kBFloat16, p.device, {n, h, p.d}, "out");
    m.lse = shaped(lse, at::kFloat, p.device, {n, h}, "lse", true);
    m.has_mod = mod != Py_None;
    if (m.has_mod) {
        if (!PyTuple_CheckExact(mod) || PyTuple_GET_SIZE(mod) != 6) fail("mod", "must be a ScoreMod");
        m.mod.softcap = static_cast<float>(PyFloat_AsDouble(PyTuple_GET_ITEM(mod, 0)));
        m.mod.window = int32(PyTuple_GET_ITEM(mod, 1), "window");
        m.mod.sink = int32(PyTuple_GET_ITEM(mod, 2), "sink");
        m.mod.prefix = int32(PyTuple_GET_ITEM(mod, 3), "prefix");
        m.mod.alibi = static_cast<const float *>(ptr(shaped(PyTuple_GET_ITEM(mod, 4), at::kFloat, p.device, {h}, "alibi", true)));
        m.mod.doc_start = static_cast<const int32_t *>(ptr(shaped(PyTuple_GET_ITEM(mod, 5), at::kInt, p.device, {n}, "doc_start", true)));
    }
    m.scale = scale == Py_None ? static_cast<float>(1.0 / std::sqrt(static_cast<double>(p.d)))
                               : static_cast<float>(PyFloat_AsDouble(scale));
    if (PyErr_Occurred()) throw Bad{};
    m.ws = shaped(ws, at::kByte, p.device, {-1}, "workspace", true);
    return m;
}

// (pool, layer, q, block_tables, seq_lens, out, lse, mod, scale, workspace, stream)
long decode_attn_mod(PyObject *const *a, Py_ssize_t n)
{
    count(n, 11);
    const PoolArgs p = pool_args(a[0]);
    const int32_t layer = int32(a[1], "layer");
    const ModArgs m = mod_args(p, a[2], a[5], a[6], a[7], a[8], a[9]);
    const int64_t B = m.q->size(0);
    const at::Tensor *bt = shaped(a[3], at::kInt, p.device, {B, -1}, "block_tables");
    const at::Tensor *lens = shaped(a[4], at::kInt, p.device, {B}, "seq_lens");
    void *s = stream_of(a[10], p);
    const Unlocked unlocked;
    return kvc_decode_attn_mod(p.pool, layer, ptr(m.q), static_cast<int32_t>(m.q->size(1)), static_cast<const int32_t *>(ptr(bt)),
                               static_cast<int32_t>(bt->size(1)), static_cast<const int32_t *>(ptr(lens)),
                               static_cast<int32_t>(B), m.has_mod ? &m.mod : nullptr, ptr(m.out),
                               static_cast<float *>(ptr(m.lse)), m.scale, ptr(m.ws), m.ws ? m.ws->numel() : 0, s);
}

// (pool, layer, q, block_table_row, q_start, out, lse, mod, scale, workspace, stream)
long prefill_attn_mod(PyObject *const *a, Py_ssize_t n)
{
    count(n, 11);
    const PoolArgs p = pool_args(a[0]);
    const int32_t layer = int32(a[1], "layer");
    const ModArgs m = mod_args(p, a[2], a[5], a[6], a[7], a[8], a[9]);
    const at::Tensor *row = shaped(a[3], at::kInt, p.device, {-1}, "block_table_row");
    const int32_t q_start = int32(a[4], "q_start");
    const int64_t n_q = m.q->size(0);
    if (n_q > 0x7FFFFFFF) fail("q", "has too many rows");
    void *s = stream_of(a[10], p);
    const Unlocked unlocked;
    return kvc_prefill_attn_mod(p.pool, layer, ptr(m.q), static_cast<int32_t>(n_q), static_cast<int32_t>(m.q->size(1)),
                                static_cast<const int32_t *>(ptr(row)), static_cast<int32_t>(row->size(0)), q_start,
                                m.has_mod ? &m.mod : nullptr, ptr(m.out), static_cast<float *>(ptr(m.lse)), m.scale,
                                ptr(m.ws), m.ws ? m.ws->numel() : 0, s);
}

template <long (*F)(PyObject *const *, Py_ssize_t)>
PyObject *entry(PyObject *, PyObject *const *args, Py_ssize_t n)
{
    try {
        return PyLong_FromLong(F(args, n));
    } catch (const Bad &) {
        return nullptr;
    } catch (const std::exception &e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
        return nullptr;
    }
}

template <long (*F)(PyObject *const *, Py_ssize_t)>
PyMethodDef method(const char *name)
{
    return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&entry<F>)), METH_FASTCALL, nullptr};
}

PyMethodDef methods[] = {method<rope_write>("rope_write"), method<decode_attn_mod>("decode_attn_mod"),
                         method<prefill_attn_mod>("prefill_attn_mod"), {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_kvc_call", "Argument marshalling of the kvc binding.", -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__kvc_call(void) { return PyModule_Create(&module); }
