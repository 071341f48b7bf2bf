// binding.cpp -- torch tensors to the C ABI, for the calls of a decode step.
//
// A decode step makes a handful of calls that take a few microseconds each on
// the GPU, so their marshalling counts: checked and converted in Python with
// ctypes a call took 15 to 20 microseconds of host time, here one or two.
// The functions take the arguments of the Python functions of the same names
// (_abi.py documents them), raise TypeError and ValueError for tensors of the
// wrong kind, and return the C ABI's status.  The library itself is loaded by
// path (attach), so this module holds no second copy of it.
#include <Python.h>

#include <dlfcn.h>

#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include "../../include/tf_paged.h"

namespace {

// ---- the library's entry points ------------------------------------------------

#define TF_CALLS(X)                                                                                \
    X(tf_paged_attn_decode_window)                                                                 \
    X(tf_paged_attn_verify_window)                                                                 \
    X(tf_paged_attn_prompt_window)                                                                 \
    X(tf_kv_put_rows_rope)                                                                         \
    X(tf_kv_pages_fork)                                                                            \
    X(tf_kv_pages_free)                                                                            \
    X(tf_kv_pages_free_window)                                                                     \
    X(tf_kv_pages_grow)                                                                            \
    X(tf_kv_pages_compact)                                                                         \
    X(tf_kv_pages_move)

struct Calls {
#define X(name) decltype(&::name) name = nullptr;
    TF_CALLS(X)
#undef X
} lib;

// Thrown after a Python exception was set.
struct PyError {};

[[noreturn]] void fail(PyObject *type, const char *fmt, const char *name)
{
    PyErr_Format(type, fmt, name);
    throw PyError{};
}

// ---- arguments -------------------------------------------------------------------

const at::Tensor &tensor_of(PyObject *o, const char *name)
{
    if (!THPVariable_Check(o))
        fail(PyExc_TypeError, "%s must be a tensor", name);
    return THPVariable_Unpack(o);
}

const char *type_name(at::ScalarType t)
{
    return t == at::kInt ? "torch.int32" : t == at::kFloat ? "torch.float32" : "torch.bfloat16";
}

// A tensor of the given type and dims (any strides).
const at::Tensor &need_strided(PyObject *o, at::ScalarType type, int64_t dims, const char *name)
{
    const at::Tensor &t = tensor_of(o, name);
    if (t.scalar_type() != type || t.dim() != dims) {
        PyErr_Format(PyExc_TypeError, "%s must be a %s tensor with %d dims", name, type_name(type), (int)dims);
        throw PyError{};
    }
    return t;
}

const at::Tensor &need(PyObject *o, at::ScalarType type, int64_t dims, const char *name)
{
    const at::Tensor &t = need_strided(o, type, dims, name);
    if (!t.is_contiguous())
        fail(PyExc_ValueError, "%s must be contiguous", name);
    return t;
}

void must(bool ok, const char *what)
{
    if (!ok)
        fail(PyExc_ValueError, "%s", what);
}

int32_t int_of(PyObject *o, const char *name)
{
    const long long v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred())
        throw PyError{};
    if (v < INT32_MIN || v > INT32_MAX)
        fail(PyExc_OverflowError, "%s does not fit 32 bits", name);
    return (int32_t)v;
}

float float_of(PyObject *o)
{
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred())
        throw PyError{};
    return (float)v;
}

// The tensors of a call are on the current CUDA device (the kernels run
// there); checked last, after their types and shapes.
struct Devices {
    const at::Tensor *seen[16];
    const char *names[16];
    int n = 0;
    void on(const at::Tensor &t, const char *name)
    {
        seen[n] = &t;
        names[n++] = name;
    }
    void check() const
    {
        int current = -1;
        for (int i = 0; i < n; ++i) {
            if (seen[i]->numel() == 0)
                continue;  // never read
            if (!seen[i]->is_cuda())
                fail(PyExc_ValueError, "%s must be on the GPU", names[i]);
            if (current < 0)
                current = c10::cuda::current_device();
            if (seen[i]->device().index() != current)
                fail(PyExc_ValueError, "%s is not on the current device", names[i]);
        }
    }
};

// The call's stream, once everything else about its arguments is known to be
// right (None: torch's current stream).
void *stream_of(const Devices &dev, PyObject *o)
{
    dev.check();
    if (o == Py_None)
        return c10::cuda::getCurrentCUDAStream().stream();
    if (PyLong_Check(o)) {
        void *s = PyLong_AsVoidPtr(o);
        if (PyErr_Occurred())
            throw PyError{};
        return s;
    }
    PyObject *handle = PyObject_GetAttrString(o, "cuda_stream");
    if (!handle)
        throw PyError{};
    void *s = PyLong_AsVoidPtr(handle);
    Py_DECREF(handle);
    if (PyErr_Occurred())
        throw PyError{};
    return s;
}

tf_kv_pool pool_of(PyObject *k, PyObject *v, Devices &dev)
{
    const at::Tensor &kp = need(k, at::kBFloat16, 4, "k_pool"), &vp = need(v, at::kBFloat16, 4, "v_pool");
    must(kp.sizes() == vp.sizes(), "k_pool and v_pool differ in shape");
    for (int i = 0; i < 4; ++i)
        must(kp.size(i) <= INT32_MAX, "k_pool is too large");
    dev.on(kp, "k_pool");
    dev.on(vp, "v_pool");
    return {kp.data_ptr(), vp.data_ptr(), (int32_t)kp.size(0), (int32_t)kp.size(1), (int32_t)kp.size(2),
            (int32_t)kp.size(3)};
}

struct Table {
    int32_t *data;
    int32_t rows, stride;
};

Table table_of(PyObject *o, const char *name, Devices &dev)
{
    const at::Tensor &t = need(o, at::kInt, 2, name);
    must(t.size(0) <= INT32_MAX && t.size(1) <= INT32_MAX, "the table is too large");
    dev.on(t, name);
    return {(int32_t *)t.data_ptr(), (int32_t)t.size(0), (int32_t)t.size(1)};
}

// One int32 per row; None: null.
int32_t *row_ints(PyObject *o, int64_t n, const char *name, Devices &dev)
{
    if (o == Py_None)
        return nullptr;
    const at::Tensor &t = need(o, at::kInt, 1, name);
    if (t.size(0) != n)
        fail(PyExc_ValueError, "%s must have one element per row", name);
    dev.on(t, name);
    return (int32_t *)t.data_ptr();
}

tf_streams streams_of(PyObject *table, PyObject *lens, PyObject *max_len, Devices &dev)
{
    const Table t = table_of(table, "table", dev);
    return {t.data, t.stride, row_ints(lens, t.rows, "lens", dev), t.rows, int_of(max_len, "max_len")};
}

tf_kv_pages pages_of(PyObject *refs, PyObject *page_size, Devices &dev)
{
    const at::Tensor &r = need(refs, at::kInt, 1, "refs");
    must(r.size(0) <= INT32_MAX, "refs is too large");
    dev.on(r, "refs");
    return {(int32_t *)r.data_ptr(), (int32_t)r.size(0), int_of(page_size, "page_size")};
}

uint32_t *status_of(PyObject *o, Devices &dev)
{
    if (o == Py_None)
        return nullptr;
    const at::Tensor &t = tensor_of(o, "status");
    if (t.scalar_type() != at::kInt || t.numel() < 1)
        fail(PyExc_TypeError, "%s must be an int32 tensor", "status");
    dev.on(t, "status");
    return (uint32_t *)t.data_ptr();
}

struct Moves {
    void *data;
    size_t bytes;
};

Moves moves_of(PyObject *o, Devices &dev)
{
    const at::Tensor &t = need(o, at::kInt, 2, "moves");
    must(t.size(1) == 4, "moves must be [1 + cap][4]");
    dev.on(t, "moves");
    return {t.data_ptr(), (size_t)t.size(0) * TF_MOVE_BYTES};
}

// Step rows [S][W][heads][d], which may be slices of a wider projection
// output: heads and dims dense, rows evenly apart.
struct Rows {
    void *data;
    int64_t stride;
};

Rows rows_of(const at::Tensor &t, int64_t S, int64_t W, int64_t heads, int64_t d, const char *name, Devices &dev)
{
    if (t.size(0) != S || t.size(1) != W || t.size(2) != heads || t.size(3) != d)
        fail(PyExc_ValueError, "%s must be [n_streams][rows][heads][head_dim]", name);
    const int64_t row = W > 1 ? t.stride(1) : S > 1 ? t.stride(0) : heads * d;
    if ((d > 1 && t.stride(3) != 1) || (heads > 1 && t.stride(2) != d) ||
        (W > 1 && S > 1 && t.stride(0) != W * row))
        fail(PyExc_ValueError, "%s: heads and dims must be dense and rows evenly spaced", name);
    dev.on(t, name);
    return {t.data_ptr(), row};
}

// ---- the calls ------------------------------------------------------------------

// Lets other Python threads run while the library enqueues a call's kernels, as
// ctypes does: a launch waits while the stream's queue is full, and a host
// function in that queue may need the interpreter.
struct NoGil {
    PyThreadState *const state = PyEval_SaveThread();
    ~NoGil() { PyEval_RestoreThread(state); }
};

// Runs f(args) with the number of arguments checked and exceptions kept out of
// the interpreter.
template <Py_ssize_t N, class F>
PyObject *guarded(PyObject *const *args, Py_ssize_t n, F f)
{
    if (n != N) {
        PyErr_Format(PyExc_TypeError, "%zd arguments expected", N);
        return nullptr;
    }
    try {
        const int rc = f(args);
        return PyLong_FromLong(rc);
    } catch (const PyError &) {
        return nullptr;
    } catch (const std::exception &e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
        return nullptr;
    }
}

// kind 0: decode, 1: verify, 2: prompt.  (k_pool, v_pool, table, lens, q,
// window, sinks, scale, out, workspace, max_len, stream)
template <int kind>
PyObject *attn_window(PyObject *, PyObject *const *args, Py_ssize_t n)
{
    return guarded<12>(args, n, [](PyObject *const *a) {
        Devices dev;
        const at::Tensor &q = need(a[4], at::kBFloat16, 4, "q"), &out = need(a[8], at::kFloat, 4, "out");
        must(kind != 0 || q.size(1) == 1, "decode takes one row per stream");
        must(out.sizes() == q.sizes(), "out must have q's shape");
        const at::Tensor &ws = tensor_of(a[9], "workspace");
        must(ws.is_contiguous(), "workspace must be contiguous");
        const tf_kv_pool pool = pool_of(a[0], a[1], dev);
        const tf_streams st = streams_of(a[2], a[3], a[10], dev);
        must(q.size(0) == st.n_streams && q.size(3) == pool.head_dim, "q must be [n_streams][rows][heads][head_dim]");
        must(q.size(1) <= INT32_MAX && q.size(2) <= INT32_MAX, "q is too large");
        dev.on(q, "q");
        dev.on(out, "out");
        dev.on(ws, "workspace");
        const int32_t rows = (int32_t)q.size(1), heads = (int32_t)q.size(2);
        const int32_t window = int_of(a[5], "window"), sinks = int_of(a[6], "sinks");
        const float scale = float_of(a[7]);
        void *stream = stream_of(dev, a[11]);
        const void *qp = q.data_ptr();
        float *o = (float *)out.data_ptr();
        void *w = ws.data_ptr();
        const size_t w_bytes = ws.nbytes();
        NoGil no_gil;
        if (kind == 0)
            return lib.tf_paged_attn_decode_window(&pool, &st, qp, heads, window, sinks, scale, o, w, w_bytes, stream);
        return (kind == 1 ? lib.tf_paged_attn_verify_window : lib.tf_paged_attn_prompt_window)(
            &pool, &st, qp, heads, rows, window, sinks, scale, o, w, w_bytes, stream);
    });
}

// (k_pool, v_pool, table, lens, q or None, k_rows, v_rows, positions, the
// rope's inv_freq, address of the tf_rope, max_len, q_out or None, stream)
PyObject *put_rows_rope(PyObject *, PyObject *const *args, Py_ssize_t n)
{
    return guarded<13>(args, n, [](PyObject *const *a) {
        Devices dev;
        const auto *rope = (const tf_rope *)PyLong_AsVoidPtr(a[9]);
        if (PyErr_Occurred())
            throw PyError{};
        must(rope != nullptr, "the rope has no address");
        const at::Tensor &pos = need(a[7], at::kInt, 3, "positions");
        const at::Tensor &k = need_strided(a[5], at::kBFloat16, 4, "k_rows"),
                         &v = need_strided(a[6], at::kBFloat16, 4, "v_rows");
        const tf_kv_pool pool = pool_of(a[0], a[1], dev);
        const tf_streams st = streams_of(a[2], a[3], a[10], dev);
        must(pos.size(0) == st.n_streams && pos.size(2) == rope->n_axes,
             "positions must be [n_streams][rows][n_axes]");
        const int64_t W = pos.size(1);
        must(W <= INT32_MAX, "too many rows");
        Rows q{nullptr, 0};
        int32_t heads = 0;
        void *q_out = nullptr;
        if (a[4] != Py_None) {
            const at::Tensor &t = need_strided(a[4], at::kBFloat16, 4, "q");
            must(t.size(2) <= INT32_MAX, "q is too large");
            heads = (int32_t)t.size(2);
            q = rows_of(t, st.n_streams, W, heads, pool.head_dim, "q", dev);
            const at::Tensor &o = need(a[11], at::kBFloat16, 4, "q_out");
            must(o.sizes() == t.sizes(), "q_out must have q's shape");
            dev.on(o, "q_out");
            q_out = o.data_ptr();
        }
        const Rows kr = rows_of(k, st.n_streams, W, pool.n_kv_heads, pool.head_dim, "k_rows", dev);
        const Rows vr = rows_of(v, st.n_streams, W, pool.n_kv_heads, pool.head_dim, "v_rows", dev);
        dev.on(pos, "positions");
        const at::Tensor &freq = need(a[8], at::kFloat, 1, "inv_freq");
        must(freq.data_ptr() == rope->inv_freq, "the rope's inv_freq has moved");
        dev.on(freq, "inv_freq");
        void *stream = stream_of(dev, a[12]);
        const auto *position = (const int32_t *)pos.data_ptr();
        NoGil no_gil;
        return lib.tf_kv_put_rows_rope(&pool, &st, rope, position, q.data, q.stride, q_out, heads, kr.data,
                                       kr.stride, vr.data, vr.stride, (int32_t)W, stream);
    });
}

// (refs, page_size, src_table, src_lens, parents, dst_table, dst_lens, status, stream)
PyObject *pages_fork(PyObject *, PyObject *const *args, Py_ssize_t n)
{
    return guarded<9>(args, n, [](PyObject *const *a) {
        Devices dev;
        const tf_kv_pages pg = pages_of(a[0], a[1], dev);
        const Table src = table_of(a[2], "src_table", dev), dst = table_of(a[5], "dst_table", dev);
        const int32_t *lens = row_ints(a[3], src.rows, "src_lens", dev);
        const int32_t *parents = row_ints(a[4], dst.rows, "parents", dev);
        int32_t *dst_lens = row_ints(a[6], dst.rows, "dst_lens", dev);
        uint32_t *status = status_of(a[7], dev);
        void *stream = stream_of(dev, a[8]);
        NoGil no_gil;
        return lib.tf_kv_pages_fork(&pg, src.data, src.stride, lens, src.rows, parents, dst.rows, dst.data, dst.stride,
                                    dst_lens, status, stream);
    });
}

// (refs, page_size, table, first, end, status, stream)
PyObject *pages_free(PyObject *, PyObject *const *args, Py_ssize_t n)
{
    return guarded<7>(args, n, [](PyObject *const *a) {
        Devices dev;
        const tf_kv_pages pg = pages_of(a[0], a[1], dev);
        const Table t = table_of(a[2], "table", dev);
        const int32_t *first = row_ints(a[3], t.rows, "first", dev), *end = row_ints(a[4], t.rows, "end", dev);
        uint32_t *status = status_of(a[5], dev);
        void *stream = stream_of(dev, a[6]);
        NoGil no_gil;
        return lib.tf_kv_pages_free(&pg, t.data, t.stride, t.rows, first, end, status, stream);
    });
}

// (refs, page_size, table, lens, window, sinks, status, stream)
PyObject *pages_free_window(PyObject *, PyObject *const *args, Py_ssize_t n)
{
    return guarded<8>(args, n, [](PyObject *const *a) {
        Devices dev;
        const tf_kv_pages pg = pages_of(a[0], a[1], dev);
        const Table t = table_of(a[2], "table", dev);
        const int32_t *lens = row_ints(a[3], t.rows, "lens", dev);
        const int32_t window = int_of(a[4], "window"), sinks = int_of(a[5], "sinks");
        uint32_t *status = status_of(a[6], dev);
        void *stream = stream_of(dev, a[7]);
        NoGil no_gil;
        return lib.tf_kv_pages_free_window(&pg, t.data, t.stride, lens, t.rows, window, sinks, status, stream);
    });
}

// (refs, page_size, table, lens, rows, moves, status, stream)
PyObject *pages_grow(PyObject *, PyObject *const *args, Py_ssize_t n)
{
    return guarded<8>(args, n, [](PyObject *const *a) {
        Devices dev;
        const tf_kv_pages pg = pages_of(a[0], a[1], dev);
        const Table t = table_of(a[2], "table", dev);
        const int32_t *lens = row_ints(a[3], t.rows, "lens", dev);
        const Moves m = moves_of(a[5], dev);
        const int32_t rows = int_of(a[4], "rows");
        uint32_t *status = status_of(a[6], dev);
        void *stream = stream_of(dev, a[7]);
        NoGil no_gil;
        return lib.tf_kv_pages_grow(&pg, t.data, t.stride, lens, t.rows, rows, m.data, m.bytes, status, stream);
    });
}

// (refs, page_size, table, moves, status, stream)
PyObject *pages_compact(PyObject *, PyObject *const *args, Py_ssize_t n)
{
    return guarded<6>(args, n, [](PyObject *const *a) {
        Devices dev;
        const tf_kv_pages pg = pages_of(a[0], a[1], dev);
        const Table t = table_of(a[2], "table", dev);
        const Moves m = moves_of(a[3], dev);
        uint32_t *status = status_of(a[4], dev);
        void *stream = stream_of(dev, a[5]);
        NoGil no_gil;
        return lib.tf_kv_pages_compact(&pg, t.data, t.stride, t.rows, m.data, m.bytes, status, stream);
    });
}

// (k_pool, v_pool, moves, status, stream)
PyObject *pages_move(PyObject *, PyObject *const *args, Py_ssize_t n)
{
    return guarded<5>(args, n, [](PyObject *const *a) {
        Devices dev;
        const tf_kv_pool pool = pool_of(a[0], a[1], dev);
        const Moves m = moves_of(a[2], dev);
        uint32_t *status = status_of(a[3], dev);
        void *stream = stream_of(dev, a[4]);
        NoGil no_gil;
        return lib.tf_kv_pages_move(&pool, m.data, m.bytes, status, stream);
    });
}

// (path of the library)
PyObject *attach(PyObject *, PyObject *path)
{
    const char *p = PyUnicode_AsUTF8(path);
    if (!p)
        return nullptr;
    void *h = dlopen(p, RTLD_NOW | RTLD_LOCAL);
    if (!h) {
        PyErr_SetString(PyExc_ImportError, dlerror());
        return nullptr;
    }
#define X(name)                                                                                    \
    lib.name = (decltype(lib.name))dlsym(h, #name);                                                \
    if (!lib.name) {                                                                               \
        PyErr_SetString(PyExc_ImportError, "the library lacks " #name);                            \
        return nullptr;                                                                            \
    }
    TF_CALLS(X)
#undef X
    Py_RETURN_NONE;
}

#define FAST(name) reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(name)), METH_FASTCALL, nullptr

PyMethodDef methods[] = {
    {"attach", attach, METH_O, nullptr},
    {"tf_paged_attn_decode_window", FAST(attn_window<0>)},
    {"tf_paged_attn_verify_window", FAST(attn_window<1>)},
    {"tf_paged_attn_prompt_window", FAST(attn_window<2>)},
    {"tf_kv_put_rows_rope", FAST(put_rows_rope)},
    {"tf_kv_pages_fork", FAST(pages_fork)},
    {"tf_kv_pages_free", FAST(pages_free)},
    {"tf_kv_pages_free_window", FAST(pages_free_window)},
    {"tf_kv_pages_grow", FAST(pages_grow)},
    {"tf_kv_pages_compact", FAST(pages_compact)},
    {"tf_kv_pages_move", FAST(pages_move)},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__binding(void) { return PyModule_Create(&module); }
