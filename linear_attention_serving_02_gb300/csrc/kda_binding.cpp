// Python binding of the latent-attention and page entry points of include/kda.h: checks of
// tensors, allocation of outputs and scratch with torch, and the call. A decode step makes a
// handful of these calls, each of a few microseconds on the GPU, so the checks are compiled:
// through ctypes a call of 28 arguments cost 20 us on the host, of which the launch was 4.
//
// kda.py wraps each function with its documented signature; here all arguments are positional.
// Every tensor must be on the device of the first one; the call is made with that device
// current, on its current stream.

#include <Python.h>

#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <vector>

#include "kda.h"

namespace {

PyObject *g_error = nullptr;  // kda.KdaError

// raise KdaError(fn, rc); for use as `return fail(...)`
PyObject *fail(const char *fn, int rc) {
    PyObject *e = PyObject_CallFunction(g_error, "si", fn, rc);
    if (e) {
        PyErr_SetObject(g_error, e);
        Py_DECREF(e);
    }
    return nullptr;
}

const at::Tensor &tensor(PyObject *o, const char *name) {
    TORCH_CHECK_TYPE(THPVariable_Check(o), name, " must be a tensor");
    return THPVariable_Unpack(o);
}

// Type, rank and place of a tensor, and that its last `tail` dimensions are dense.
const at::Tensor &need(PyObject *o, const char *name, at::ScalarType type, int64_t dim, int64_t tail, int dev) {
    const at::Tensor &t = tensor(o, name);
    TORCH_CHECK_TYPE(t.scalar_type() == type, name, " must be ", type, ", got ", t.scalar_type());
    TORCH_CHECK_VALUE(t.dim() == dim, name, " must have ", dim, " dimensions, got ", t.dim());
    TORCH_CHECK_VALUE(t.is_cuda(), name, " must be a CUDA tensor");
    TORCH_CHECK_VALUE(dev < 0 || t.device().index() == dev, name, " must be on cuda:", dev, ", got ", t.device());
    int64_t want = 1;
    for (int64_t d = dim - 1; d >= dim - tail; --d) {
        TORCH_CHECK_VALUE(t.size(d) <= 1 || t.stride(d) == want, name, " must be dense in its last ", tail, " dimensions");
        want *= t.size(d);
    }
    return t;
}
void shape(const at::Tensor &t, const char *name, std::initializer_list<int64_t> want) {
    TORCH_CHECK_VALUE(t.sizes() == at::IntArrayRef(want), name, " must be ", at::IntArrayRef(want), ", got ", t.sizes());
}
constexpr at::ScalarType kBf = at::kBFloat16, kF = at::kFloat, kI = at::kInt;

const int32_t *ints(PyObject *o, const char *name, int64_t n, int dev) {
    const at::Tensor &t = need(o, name, kI, 1, 1, dev);
    TORCH_CHECK_VALUE(t.size(0) == n, name, " must have ", n, " entries, got ", t.size(0));
    return static_cast<const int32_t *>(t.const_data_ptr());
}
int32_t *status_word(PyObject *o, int dev) {
    if (o == Py_None) return nullptr;
    const at::Tensor &t = need(o, "status", kI, 1, 1, dev);
    TORCH_CHECK_VALUE(t.size(0) >= 1, "status must hold one int32");
    return static_cast<int32_t *>(t.data_ptr());
}
const uint16_t *bf(const at::Tensor &t) { return static_cast<const uint16_t *>(t.const_data_ptr()); }
uint16_t *bf_out(const at::Tensor &t) { return static_cast<uint16_t *>(t.data_ptr()); }
const float *f32(const at::Tensor &t) { return static_cast<const float *>(t.const_data_ptr()); }

int64_t whole(PyObject *o, const char *name) {
    const long long v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred()) {
        PyErr_Clear();
        TORCH_CHECK_TYPE(false, name, " must be a whole number that fits 64 bits");
    }
    return v;
}
int32_t whole32(PyObject *o, const char *name) {
    const int64_t v = whole(o, name);
    TORCH_CHECK_VALUE(v >= INT32_MIN && v <= INT32_MAX, name, " does not fit 32 bits");
    return (int32_t)v;
}
float real(PyObject *o, const char *name) {
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred()) {
        PyErr_Clear();
        TORCH_CHECK_TYPE(false, name, " must be a number");
    }
    return (float)v;
}
bool truth(PyObject *o, const char *name) {
    const int v = PyObject_IsTrue(o);
    if (v < 0) {
        PyErr_Clear();
        TORCH_CHECK_TYPE(false, name, " must be a truth value");
    }
    return v != 0;
}
int32_t extent(int64_t v, const char *what) {
    TORCH_CHECK_VALUE(v <= INT32_MAX, what, " does not fit 32 bits");
    return (int32_t)v;
}

struct Cache {
    const at::Tensor *t;
    int64_t stride;
    int32_t pages, size, max_pages;
    const int32_t *table;
};
Cache paged(PyObject *cache, PyObject *page_table, int64_t seqs, int dev) {
    Cache c;
    c.t = &need(cache, "cache", kBf, 3, 2, dev);
    TORCH_CHECK_VALUE(c.t->size(2) == KDA_MLA_ROW, "cache must be [num_pages, page_size, ", KDA_MLA_ROW, "]");
    const at::Tensor &table = need(page_table, "page_table", kI, 2, 2, c.t->device().index());
    TORCH_CHECK_VALUE(table.size(0) == seqs, "page_table must have a row for each of ", seqs, " sequences");
    c.pages = extent(c.t->size(0), "the number of pages");
    c.size = extent(c.t->size(1), "the page size");
    c.stride = c.pages > 1 ? c.t->stride(0) : (int64_t)c.size * KDA_MLA_ROW;
    c.max_pages = extent(table.size(1), "the page table");
    c.table = static_cast<const int32_t *>(table.const_data_ptr());
    return c;
}
int64_t row_stride(const at::Tensor &t, int64_t least) { return t.size(0) > 1 ? t.stride(0) : least; }
void *stream_of(int dev) { return c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)dev).stream(); }

// a new dense tensor, without the way through the dispatcher that at::empty takes
at::Tensor fresh(at::IntArrayRef sizes, at::ScalarType type, int dev) {
    return at::Tensor(at::detail::empty_cuda(sizes, type, c10::Device(c10::kCUDA, (c10::DeviceIndex)dev), std::nullopt));
}

bool args(Py_ssize_t n, Py_ssize_t want, const char *fn) {
    if (n == want) return true;
    PyErr_Format(PyExc_TypeError, "%s takes %zd arguments, got %zd", fn, want, n);
    return false;
}

PyObject *mla_append(PyObject *, PyObject *const *a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    if (!args(n, 13, "mla_append")) return nullptr;
    const at::Tensor &c = need(a[0], "c", kBf, 2, 1, -1);
    const int dev = c.device().index();
    const c10::cuda::CUDAGuard guard((c10::DeviceIndex)dev);
    const int64_t T = c.size(0);
    shape(c, "c", {T, KDA_MLA_LATENT});
    const at::Tensor &k_pe = need(a[1], "k_pe", kBf, 2, 1, dev);
    shape(k_pe, "k_pe", {T, KDA_MLA_POS});
    const at::Tensor &lens = need(a[4], "cache_lens", kI, 1, 1, dev);
    const int64_t N = lens.size(0);
    const Cache cache = paged(a[2], a[3], N, dev);
    const int32_t *cu = a[5] == Py_None ? nullptr : ints(a[5], "cu_seqlens", N + 1, dev);
    const float *norm_w = nullptr, *rope = nullptr;
    int32_t rope_len = 0;
    if (a[6] != Py_None) {
        const at::Tensor &w = need(a[6], "norm_w", kF, 1, 1, dev);
        shape(w, "norm_w", {KDA_MLA_LATENT});
        norm_w = f32(w);
    }
    if (a[8] != Py_None) {
        const at::Tensor &r = need(a[8], "rope", kF, 2, 2, dev);
        shape(r, "rope", {r.size(0), KDA_MLA_POS});
        rope = f32(r);
        rope_len = extent(r.size(0), "rope");
    }
    at::Tensor q_out;
    const uint16_t *qp = nullptr;
    uint16_t *qo = nullptr;
    int64_t qs[2] = {0, 0}, qos[2] = {0, 0};
    int32_t H = 0;
    if (a[10] != Py_None) {
        TORCH_CHECK_VALUE(rope != nullptr, "q_pe is only rotated: it needs rope");
        const at::Tensor &q = need(a[10], "q_pe", kBf, 3, 1, dev);
        H = extent(q.size(1), "the number of heads");
        shape(q, "q_pe", {T, H, KDA_MLA_POS});
        q_out = a[11] == Py_None ? fresh({T, H, KDA_MLA_POS}, kBf, dev) : need(a[11], "q_out", kBf, 3, 1, dev);
        shape(q_out, "q_out", {T, H, KDA_MLA_POS});
        qp = bf(q);
        qo = bf_out(q_out);
        // the stride of a dimension of one says nothing
        auto stride = [](const at::Tensor &t, int d) { return t.size(d) > 1 ? t.stride(d) : (int64_t)KDA_MLA_POS; };
        qs[0] = stride(q, 0), qs[1] = stride(q, 1);
        qos[0] = stride(q_out, 0), qos[1] = stride(q_out, 1);
    } else {
        TORCH_CHECK_VALUE(a[11] == Py_None, "q_out needs q_pe");
    }
    const int rc = kda_mla_append(bf(c), row_stride(c, KDA_MLA_LATENT), bf(k_pe), row_stride(k_pe, KDA_MLA_POS), norm_w,
                                  real(a[7], "eps"), rope, rope_len, truth(a[9], "rope_interleaved"), qp, qs[0], qs[1],
                                  qo, qos[0], qos[1], H, cu, static_cast<const int32_t *>(lens.const_data_ptr()),
                                  cache.table, cache.max_pages, bf_out(*cache.t), cache.stride, cache.pages, cache.size,
                                  T, extent(N, "the number of sequences"), status_word(a[12], dev), stream_of(dev));
    if (rc != KDA_OK) return fail("kda_mla_append", rc);
    if (!qo && !q_out.defined()) Py_RETURN_NONE;
    return a[11] == Py_None ? THPVariable_Wrap(std::move(q_out)) : Py_NewRef(a[11]);
    END_HANDLE_TH_ERRORS
}

PyObject *mla_gather(PyObject *, PyObject *const *a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    if (!args(n, 6, "mla_gather")) return nullptr;
    const at::Tensor &first = need(a[0], "cache", kBf, 3, 2, -1);
    const int dev = first.device().index();
    const c10::cuda::CUDAGuard guard((c10::DeviceIndex)dev);
    const int64_t N = need(a[1], "page_table", kI, 2, 2, dev).size(0), T = whole(a[3], "total_rows");
    const Cache cache = paged(a[0], a[1], N, dev);
    const int32_t *cu = ints(a[2], "cu_seqlens", N + 1, dev);
    TORCH_CHECK_VALUE(T >= 0, "total_rows must not be negative");
    at::Tensor out = a[4] == Py_None ? fresh({T, KDA_MLA_ROW}, kBf, dev) : need(a[4], "out", kBf, 2, 2, dev);
    shape(out, "out", {T, KDA_MLA_ROW});
    const int rc = kda_mla_gather(bf(first), cache.stride, cache.pages, cache.size, cu, cache.table, cache.max_pages,
                                  bf_out(out), T, extent(N, "the number of sequences"), status_word(a[5], dev), stream_of(dev));
    if (rc != KDA_OK) return fail("kda_mla_gather", rc);
    return a[4] == Py_None ? THPVariable_Wrap(std::move(out)) : Py_NewRef(a[4]);
    END_HANDLE_TH_ERRORS
}

// (a, b) as a Python pair: the caller's own objects where it gave them
PyObject *pair(at::Tensor &&a, PyObject *given_a, at::Tensor &&b, PyObject *given_b) {
    PyObject *x = given_a == Py_None ? THPVariable_Wrap(std::move(a)) : Py_NewRef(given_a);
    PyObject *y = given_b == Py_None ? THPVariable_Wrap(std::move(b)) : Py_NewRef(given_b);
    PyObject *t = x && y ? PyTuple_Pack(2, x, y) : nullptr;
    Py_XDECREF(x);
    Py_XDECREF(y);
    return t;
}

PyObject *mla_prefill(PyObject *, PyObject *const *a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    if (!args(n, 10, "mla_prefill")) return nullptr;
    const at::Tensor &q = need(a[0], "q", kBf, 3, 3, -1);
    const int dev = q.device().index();
    const c10::cuda::CUDAGuard guard((c10::DeviceIndex)dev);
    const int64_t Tq = q.size(0), H = q.size(1);
    shape(q, "q", {Tq, H, KDA_MLA_QK});
    const at::Tensor &kv = need(a[1], "kv", kBf, 3, 3, dev), &k_pe = need(a[2], "k_pe", kBf, 2, 1, dev);
    const int64_t Tk = kv.size(0);
    shape(kv, "kv", {Tk, H, 2 * KDA_MLA_NOPE});
    shape(k_pe, "k_pe", {Tk, KDA_MLA_POS});
    const at::Tensor &cu_q = need(a[3], "cu_seqlens_q", kI, 1, 1, dev);
    const int64_t N = cu_q.size(0) - 1;
    TORCH_CHECK_VALUE(N >= 0, "cu_seqlens_q must hold num_seqs + 1 offsets");
    const int32_t *cu_k = ints(a[4], "cu_seqlens_k", N + 1, dev);
    at::Tensor o = a[7] == Py_None ? fresh({Tq, H, KDA_MLA_NOPE}, kBf, dev) : need(a[7], "o", kBf, 3, 3, dev);
    at::Tensor lse = a[8] == Py_None ? fresh({Tq, H}, kF, dev) : need(a[8], "lse", kF, 2, 2, dev);
    shape(o, "o", {Tq, H, KDA_MLA_NOPE});
    shape(lse, "lse", {Tq, H});
    const int rc = kda_mla_prefill(bf(q), bf(kv), bf(k_pe), row_stride(k_pe, KDA_MLA_POS),
                                   static_cast<const int32_t *>(cu_q.const_data_ptr()), cu_k, Tq, Tk,
                                   extent(N, "the number of sequences"), extent(H, "the number of heads"),
                                   truth(a[6], "causal"), real(a[5], "scale"), bf_out(o),
                                   static_cast<float *>(lse.data_ptr()), status_word(a[9], dev), stream_of(dev));
    if (rc != KDA_OK) return fail("kda_mla_prefill", rc);
    return pair(std::move(o), a[7], std::move(lse), a[8]);
    END_HANDLE_TH_ERRORS
}

PyObject *mla_decode(PyObject *, PyObject *const *a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    if (!args(n, 11, "mla_decode")) return nullptr;
    const at::Tensor &q_lat = need(a[0], "q_lat", kBf, 3, 3, -1);
    const int dev = q_lat.device().index();
    const c10::cuda::CUDAGuard guard((c10::DeviceIndex)dev);
    const at::Tensor &lens = need(a[4], "cache_lens", kI, 1, 1, dev);
    const int64_t N = lens.size(0), rows = q_lat.size(0), H = q_lat.size(1);
    const int32_t m = whole32(a[6], "num_tokens");
    TORCH_CHECK_VALUE(m >= 0 && rows == N * m, "q_lat has ", rows, " rows, expected num_seqs * num_tokens = ", N, " * ", m);
    shape(q_lat, "q_lat", {rows, H, KDA_MLA_LATENT});
    const at::Tensor &q_pe = need(a[1], "q_pe", kBf, 3, 3, dev);
    shape(q_pe, "q_pe", {rows, H, KDA_MLA_POS});
    const Cache cache = paged(a[2], a[3], N, dev);
    at::Tensor o = a[7] == Py_None ? fresh({rows, H, KDA_MLA_LATENT}, kBf, dev) : need(a[7], "o", kBf, 3, 3, dev);
    at::Tensor lse = a[8] == Py_None ? fresh({rows, H}, kF, dev) : need(a[8], "lse", kF, 2, 2, dev);
    shape(o, "o", {rows, H, KDA_MLA_LATENT});
    shape(lse, "lse", {rows, H});
    const int32_t n32 = extent(N, "the number of sequences"), h32 = extent(H, "the number of heads");
    at::Tensor ws;
    if (a[9] == Py_None) {
        ws = fresh({(int64_t)kda_mla_decode_workspace_size(n32, h32, m)}, at::kByte, dev);
    } else {
        ws = tensor(a[9], "workspace");
        TORCH_CHECK_VALUE(ws.is_cuda() && ws.device().index() == dev && ws.is_contiguous(),
                          "workspace must be contiguous and on cuda:", dev);
    }
    const int rc = kda_mla_decode(bf(q_lat), bf(q_pe), bf(*cache.t), cache.stride, cache.pages, cache.size, cache.table,
                                  cache.max_pages, static_cast<const int32_t *>(lens.const_data_ptr()), n32, h32, m,
                                  real(a[5], "scale"), bf_out(o), static_cast<float *>(lse.data_ptr()), ws.data_ptr(),
                                  ws.nbytes(), status_word(a[10], dev), stream_of(dev));
    if (rc != KDA_OK) return fail("kda_mla_decode", rc);
    return pair(std::move(o), a[7], std::move(lse), a[8]);
    END_HANDLE_TH_ERRORS
}

// Page ids: a list or tuple of whole numbers, or a contiguous 1-D CPU int32 tensor.
struct Ids {
    std::vector<int32_t> own;
    const int32_t *p;
    int64_t n;
    bool fits = true;  // false: an id is negative or past 32 bits
    Ids(PyObject *o, const char *name) {
        if (PyList_CheckExact(o) || PyTuple_CheckExact(o)) {
            n = PySequence_Fast_GET_SIZE(o);
            own.resize((size_t)n);
            for (int64_t i = 0; i < n; ++i) {
                PyObject *item = PySequence_Fast_GET_ITEM(o, i);
                int over = 0;
                const long long v = PyLong_Check(item) ? PyLong_AsLongLongAndOverflow(item, &over) : index(item, name, &over);
                fits = fits && !over && v >= 0 && v <= INT32_MAX;
                own[(size_t)i] = (int32_t)v;
                TORCH_CHECK_VALUE(PySequence_Fast_GET_SIZE(o) == n, name, " changed its length");  // by an item's __index__
            }
            p = own.data();
        } else {
            const at::Tensor &t = tensor(o, name);
            TORCH_CHECK_VALUE(t.device().is_cpu() && t.scalar_type() == kI && t.dim() == 1 && t.is_contiguous(), name,
                              " must be a contiguous 1-D CPU int32 tensor");
            p = static_cast<const int32_t *>(t.const_data_ptr());
            n = t.size(0);
        }
    }
    static long long index(PyObject *item, const char *name, int *over) {
        Py_INCREF(item);  // its own code runs: the list's reference may go
        PyObject *i = PyNumber_Index(item);
        Py_DECREF(item);
        if (!i) {
            PyErr_Clear();
            TORCH_CHECK_TYPE(false, name, " must hold whole numbers");
        }
        const long long v = PyLong_AsLongLongAndOverflow(i, over);
        Py_DECREF(i);
        return v;
    }
};

PyObject *pages_copy(PyObject *, PyObject *const *a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    if (!args(n, 3, "pages_copy")) return nullptr;
    const at::Tensor &pool = tensor(a[0], "pool");
    const Ids src(a[1], "src"), dst(a[2], "dst");
    TORCH_CHECK_VALUE(pool.is_cuda() && pool.dim() >= 3, "pool must be a CUDA tensor [layers, pages, ...]");
    const int dev = pool.device().index();
    const c10::cuda::CUDAGuard guard((c10::DeviceIndex)dev);
    int64_t page = 1;
    for (int64_t d = pool.dim() - 1; d >= 2; --d) {
        TORCH_CHECK_VALUE(pool.size(d) <= 1 || pool.stride(d) == page, "pool must be dense within a page");
        page *= pool.size(d);
    }
    TORCH_CHECK_VALUE(src.n == dst.n, "src and dst must have the same length");
    if (!src.fits || !dst.fits) return fail("kda_pages_copy", KDA_ERR_PAGES);
    const int64_t es = pool.element_size(), layers = pool.size(0), pages = pool.size(1), bytes = page * es;
    const int64_t page_stride = pages > 1 ? pool.stride(1) * es : bytes;
    const int64_t layer_stride = layers > 1 ? pool.stride(0) * es : page_stride * pages;
    const int rc = kda_pages_copy(pool.data_ptr(), page_stride, bytes, extent(pages, "the number of pages"), layer_stride,
                                  extent(layers, "the number of layers"), src.p, dst.p, extent(src.n, "the list"), stream_of(dev));
    if (rc != KDA_OK) return fail("kda_pages_copy", rc);
    return Py_NewRef(a[0]);
    END_HANDLE_TH_ERRORS
}

PyObject *set_error(PyObject *, PyObject *cls) {
    Py_XSETREF(g_error, Py_NewRef(cls));
    Py_RETURN_NONE;
}

PyCFunction fast(PyObject *(*f)(PyObject *, PyObject *const *, Py_ssize_t)) {
    return reinterpret_cast<PyCFunction>(reinterpret_cast<void *>(f));
}
PyMethodDef g_methods[] = {{"mla_append", fast(mla_append), METH_FASTCALL, nullptr},
                           {"mla_gather", fast(mla_gather), METH_FASTCALL, nullptr},
                           {"mla_prefill", fast(mla_prefill), METH_FASTCALL, nullptr},
                           {"mla_decode", fast(mla_decode), METH_FASTCALL, nullptr},
                           {"pages_copy", fast(pages_copy), METH_FASTCALL, nullptr},
                           {"set_error", set_error, METH_O, nullptr},
                           {nullptr, nullptr, 0, nullptr}};
PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_kda_binding", nullptr, -1, g_methods};

}  // namespace

PyMODINIT_FUNC PyInit__kda_binding() { return PyModule_Create(&g_module); }
