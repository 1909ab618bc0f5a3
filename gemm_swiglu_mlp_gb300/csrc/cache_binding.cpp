// The Python side of the paged-cache entry points (include/swiglu.h), natively:
// argument checks, device and stream, output buffers and the C ABI call.
//
// Small ones of these calls take 2 to 16 microseconds of GPU time in a serving step,
// several a layer. Checked and marshalled in Python they took the host 10.6 (plan),
// 7.4 (write), 13 (accept) and 18 (attention, which is two launches), so a step
// waited for its host; here they take 2.8, 2.0, 3.8 and 10.3, launches included.
// The module holds no operator: it calls the functions of libswiglu_gb300.so,
// whose addresses cache.py gives it.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/ops/empty.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <cuda_runtime_api.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <map>
#include <optional>
#include <utility>

#include "swiglu.h"

namespace {

using at::Tensor;

decltype(&swiglu_cache_plan) g_plan;
decltype(&swiglu_cache_write) g_write;
decltype(&swiglu_tree_attention_workspace_bytes) g_attend_bytes;
decltype(&swiglu_tree_attention) g_attend;
decltype(&swiglu_cache_accept) g_accept;
PyObject *g_error;       // SwigluError
PyObject *g_workspace;   // (device index, bytes, stream or None) -> uint8 tensor

// A check failed and a Python exception is set.
struct Refused {};

[[noreturn]] void refuse(PyObject *type, const char *format, const char *name, const char *more = "",
                         long long a = 0, long long b = 0) {
    PyErr_Format(type, format, name, more, a, b);
    throw Refused{};
}

const Tensor &cuda_tensor(PyObject *o, const char *name, int index) {
    if (!THPVariable_Check(o) || !THPVariable_Unpack(o).is_cuda())
        refuse(PyExc_TypeError, "%s must be a CUDA tensor", name);
    const Tensor &t = THPVariable_Unpack(o);
    if (index >= 0 && t.get_device() != index)
        refuse(PyExc_ValueError, "%s must be on the same device as the others%s", name);
    return t;
}
const Tensor &cuda_tensor(PyObject *o, const char *name, at::ScalarType type, int index) {
    const Tensor &t = cuda_tensor(o, name, index);
    if (t.scalar_type() != type)
        refuse(PyExc_TypeError, "%s must be %s, not another type", name, c10::toString(type));
    return t;
}

// A contiguous vector of n values (n < 0: any).
const Tensor &vector(PyObject *o, const char *name, int64_t n, int index) {
    const Tensor &t = cuda_tensor(o, name, at::kInt, index);
    if (t.dim() != 1 || (n >= 0 && t.size(0) != n) || !t.is_contiguous())
        refuse(PyExc_ValueError, "%s must be a contiguous vector of %s%lld values", name,
               n < 0 ? "any number, not " : "", n < 0 ? t.numel() : n);
    return t;
}

// A contiguous matrix of `rows` rows and at least one column.
const Tensor &matrix(PyObject *o, const char *name, int64_t rows, int index,
                     at::ScalarType type = at::kInt) {
    const Tensor &t = cuda_tensor(o, name, type, index);
    if (t.dim() != 2 || t.size(0) != rows || t.size(1) < 1 || !t.is_contiguous())
        refuse(PyExc_ValueError, "%s must be contiguous, [%s%lld, at least 1]", name, "", rows);
    return t;
}

// A block table; without requests its columns do not matter.
int64_t table_columns(PyObject *o, int64_t rows, int index, void **data) {
    if (rows == 0) {
        const Tensor &t = cuda_tensor(o, "block_table", at::kInt, index);
        if (t.dim() != 2 || t.size(0) != 0)
            refuse(PyExc_ValueError, "%s must be [0, any]%s", "block_table");
        *data = nullptr;
        return 1;
    }
    const Tensor &t = matrix(o, "block_table", rows, index);
    *data = t.data_ptr();
    return t.size(1);
}

// [tokens, heads, dim] BF16 rows: the last dimension contiguous, the others'
// strides multiples of 8 (tokens or heads < 0: any).
const Tensor &rows(PyObject *o, const char *name, int64_t tokens, int64_t heads, int64_t dim,
                   int index) {
    const Tensor &t = cuda_tensor(o, name, at::kBFloat16, index);
    if (t.dim() != 3 || t.size(2) != dim || (heads >= 0 && t.size(1) != heads) ||
        (tokens >= 0 && t.size(0) != tokens))
        refuse(PyExc_ValueError, "%s must be [tokens, heads, head size]%s like the others: %lld heads"
               " or %lld values a row do not fit", name, "", t.dim() == 3 ? t.size(1) : -1,
               t.dim() == 3 ? t.size(2) : -1);
    if (t.stride(2) != 1 || ((t.stride(0) | t.stride(1)) & 7))
        refuse(PyExc_ValueError, "%s must have a contiguous last dimension and strides that are "
               "multiples of 8%s", name);
    return t;
}

// A pair of caches [layers (if allowed), pages, kv heads, page size, head size].
struct Caches {
    void *k, *v;
    int64_t layers, pages, heads, page_size, dim;
    int index;
};
Caches caches(PyObject *ko, PyObject *vo, bool layered) {
    const Tensor &k = cuda_tensor(ko, "k_cache", at::kBFloat16, -1);
    const int index = k.get_device();
    const Tensor &v = cuda_tensor(vo, "v_cache", at::kBFloat16, index);
    const int64_t d = k.dim();
    if ((d != 4 && !(layered && d == 5)) || !k.is_contiguous())
        refuse(PyExc_ValueError, "%s must be contiguous, [%spages, kv heads, page size, head size]",
               "k_cache", layered ? "(layers,) " : "");
    if (!v.is_contiguous() || v.sizes() != k.sizes())
        refuse(PyExc_ValueError, "%s must be contiguous and of k_cache's shape%s", "v_cache");
    return {k.data_ptr(), v.data_ptr(), d == 5 ? k.size(0) : 1, k.size(d - 4), k.size(d - 3),
            k.size(d - 2), k.size(d - 1), index};
}

// Handle of the given torch.cuda.Stream, or of the current one.
void *stream_of(PyObject *stream, int index) {
    if (stream == Py_None) return c10::cuda::getCurrentCUDAStream(index).stream();
    PyObject *h = PyObject_GetAttrString(stream, "cuda_stream");
    if (!h) throw Refused{};
    void *p = PyLong_AsVoidPtr(h);
    Py_DECREF(h);
    if (!p && PyErr_Occurred()) throw Refused{};
    return p;
}

bool capturing(void *stream) {
    cudaStreamCaptureStatus status = cudaStreamCaptureStatusNone;
    if (cudaStreamIsCapturing(static_cast<cudaStream_t>(stream), &status) != cudaSuccess) {
        cudaGetLastError();   // (of a stream that no call may use now: its launch reports it)
        return true;
    }
    return status != cudaStreamCaptureStatusNone;
}

int64_t integer(PyObject *o) {
    const long long v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred()) throw Refused{};
    return v;
}

void done(int status, const char *entry) {
    if (status == SWIGLU_OK) return;
    PyObject *e = PyObject_CallFunction(g_error, "is", status, entry);
    if (e) {
        PyErr_SetObject(g_error, e);
        Py_DECREF(e);
    }
    throw Refused{};
}

bool count_is(Py_ssize_t got, Py_ssize_t want) {
    if (got == want) return true;
    PyErr_Format(PyExc_TypeError, "expected %zd arguments, got %zd", want, got);
    return false;
}

#define GUARDED_BEGIN HANDLE_TH_ERRORS try {
#define GUARDED_END                 \
    }                               \
    catch (const Refused &) {       \
        return nullptr;             \
    }                               \
    END_HANDLE_TH_ERRORS

// plan(ctx_lens, new_lens, pages_held, block_table, free_pages, page_size,
//      max_tokens, parents, free_head, query_start, slots, positions,
//      pages_held_out, counts, mask, stream); the outputs are tensors that exist
PyObject *plan(PyObject *, PyObject *const *a, Py_ssize_t n) {
    GUARDED_BEGIN
    if (!count_is(n, 16)) return nullptr;
    const Tensor &ctx = vector(a[0], "ctx_lens", -1, -1);
    const int index = ctx.get_device();
    const int64_t R = ctx.size(0), T = integer(a[6]);
    const Tensor &fresh = vector(a[1], "new_lens", R, index);
    const Tensor &held = vector(a[2], "pages_held", R, index);
    void *table = nullptr;
    const int64_t max_pages = table_columns(a[3], R, index, &table);
    const Tensor &free_pages = vector(a[4], "free_pages", -1, index);
    const Tensor *parents = a[7] == Py_None ? nullptr : &matrix(a[7], "parents", R, index);
    const Tensor *head = a[8] == Py_None ? nullptr : &vector(a[8], "free_head", 1, index);
    const Tensor &start = vector(a[9], "out.query_start", R + 1, index);
    const Tensor &slots = vector(a[10], "out.slots", T, index);
    const Tensor &positions = vector(a[11], "out.positions", T, index);
    const Tensor &held_out = vector(a[12], "out.pages_held", R, index);
    const Tensor &counts = vector(a[13], "out.counts", 3, index);
    const int64_t width = parents ? parents->size(1) : 0;
    void *mask = nullptr;
    if ((a[14] == Py_None) != !parents)
        refuse(PyExc_ValueError, "%s goes with parents: both or neither%s", "out.mask");
    if (parents && T > 0) {
        const Tensor &m = matrix(a[14], "out.mask", T, index, at::kLong);
        if (m.size(1) != (width + 63) / 64)
            refuse(PyExc_ValueError, "%s must have %s%lld words a token", "out.mask", "",
                   (width + 63) / 64);
        mask = m.data_ptr();
    }
    const c10::cuda::CUDAGuard guard(static_cast<c10::DeviceIndex>(index));
    done(g_plan(static_cast<int32_t *>(ctx.data_ptr()), static_cast<int32_t *>(fresh.data_ptr()),
                static_cast<int32_t *>(held.data_ptr()), static_cast<int32_t *>(table), R, max_pages,
                static_cast<int32_t *>(free_pages.data_ptr()), free_pages.size(0),
                head ? static_cast<int32_t *>(head->data_ptr()) : nullptr, integer(a[5]),
                parents ? static_cast<int32_t *>(parents->data_ptr()) : nullptr, width, T,
                static_cast<int32_t *>(start.data_ptr()), static_cast<int32_t *>(slots.data_ptr()),
                static_cast<int32_t *>(positions.data_ptr()),
                static_cast<int32_t *>(held_out.data_ptr()),
                static_cast<int32_t *>(counts.data_ptr()), static_cast<int64_t *>(mask),
                stream_of(a[15], index)),
         "swiglu_cache_plan");
    Py_RETURN_NONE;
    GUARDED_END
}

// write(k, v, slots, k_cache, v_cache, stream)
PyObject *write(PyObject *, PyObject *const *a, Py_ssize_t n) {
    GUARDED_BEGIN
    if (!count_is(n, 6)) return nullptr;
    const Caches c = caches(a[3], a[4], false);
    const Tensor &k = rows(a[0], "k", -1, c.heads, c.dim, c.index);
    const int64_t T = k.size(0);
    const Tensor &v = rows(a[1], "v", T, c.heads, c.dim, c.index);
    const Tensor &slots = vector(a[2], "slots", T, c.index);
    const c10::cuda::CUDAGuard guard(static_cast<c10::DeviceIndex>(c.index));
    done(g_write(k.data_ptr(), v.data_ptr(), T, c.heads, c.dim, k.stride(0), k.stride(1),
                 v.stride(0), v.stride(1), static_cast<int32_t *>(slots.data_ptr()), c.k, c.v,
                 c.pages, c.page_size, stream_of(a[5], c.index)),
         "swiglu_cache_write");
    Py_RETURN_NONE;
    GUARDED_END
}

// One attention workspace per (device, stream), made by cache.py and grown on
// demand; kept to the process's end. No captured call uses it: a graph holds the
// address, which growing would leave to the allocator, and may be replayed on
// another stream beside this one's calls. Apart from the other entry points'
// workspaces, whose counters have to stay as they are between calls.
using Workspaces = std::map<std::pair<int, void *>, Tensor>;
Workspaces &workspaces() {
    static Workspaces *all = new Workspaces;   // (not destroyed after CUDA at exit)
    return *all;
}

// attend(q, k_cache, v_cache, block_table, ctx_lens, query_start, mask, scale,
//        out, workspace, stream) -> out
PyObject *attend(PyObject *, PyObject *const *a, Py_ssize_t n) {
    GUARDED_BEGIN
    if (!count_is(n, 11)) return nullptr;
    const Caches c = caches(a[1], a[2], false);
    const Tensor &q = rows(a[0], "q", -1, -1, c.dim, c.index);
    const int64_t T = q.size(0), heads = q.size(1);
    if (c.heads < 1 || heads % c.heads)
        refuse(PyExc_ValueError, "%s heads must be a multiple of the kv heads%s (%lld of %lld)", "q",
               "", heads, c.heads);
    const Tensor &ctx = vector(a[4], "ctx_lens", -1, c.index);
    const int64_t R = ctx.size(0);
    void *table = nullptr;
    const int64_t max_pages = table_columns(a[3], R, c.index, &table);
    const Tensor &start = vector(a[5], "query_start", R + 1, c.index);
    const Tensor *mask = nullptr;
    if (a[6] != Py_None) mask = &matrix(a[6], "mask", T, c.index, at::kLong);
    double scale = 1.0;
    if (a[7] == Py_None) {
        scale = c.dim == 128 ? 0.08838834764831845 : c.dim == 64 ? 0.125 : 1.0;   // 1/sqrt(dim)
    } else {
        scale = PyFloat_AsDouble(a[7]);
        if (scale == -1.0 && PyErr_Occurred()) return nullptr;
    }
    const c10::cuda::CUDAGuard guard(static_cast<c10::DeviceIndex>(c.index));
    Tensor made;
    const Tensor *out = &made;
    if (a[8] == Py_None) {
        made = at::empty({T, heads, c.dim}, q.options());
    } else {
        out = &cuda_tensor(a[8], "out", at::kBFloat16, c.index);
        if (out->dim() != 3 || out->size(0) != T || out->size(1) != heads ||
            out->size(2) != c.dim || !out->is_contiguous())
            refuse(PyExc_ValueError, "%s must be contiguous and of q's shape%s", "out");
    }
    void *stream = stream_of(a[10], c.index);
    const size_t need = g_attend_bytes(T, heads, c.heads, c.dim);
    void *ws = nullptr;
    size_t ws_bytes = 0;
    Tensor captured;   // a captured call's: the graph's pool has it back after this call's launches
    if (a[9] != Py_None) {
        const Tensor &w = cuda_tensor(a[9], "workspace", c.index);
        if (!w.is_contiguous())
            refuse(PyExc_ValueError, "%s must be contiguous%s", "workspace");
        ws = w.data_ptr();
        ws_bytes = w.nbytes();
    } else if (need) {
        Tensor &w = capturing(stream) ? captured : workspaces()[{c.index, stream}];
        if (!w.defined() || w.nbytes() < need) {
            PyObject *o = PyObject_CallFunction(g_workspace, "inO", c.index,
                                                static_cast<Py_ssize_t>(need), a[10]);
            if (!o) return nullptr;
            w = THPVariable_Unpack(o);
            Py_DECREF(o);
        }
        ws = w.data_ptr();
        ws_bytes = w.nbytes();
    }
    done(g_attend(q.data_ptr(), q.stride(0), q.stride(1), c.k, c.v, c.pages, c.page_size,
                  static_cast<int32_t *>(table), R, max_pages, static_cast<int32_t *>(ctx.data_ptr()),
                  static_cast<int32_t *>(start.data_ptr()),
                  mask ? static_cast<int64_t *>(mask->data_ptr()) : nullptr,
                  mask ? mask->size(1) : 0, static_cast<float>(scale), out->data_ptr(), T, heads,
                  c.heads, c.dim, ws, ws_bytes, stream),
         "swiglu_tree_attention");
    if (a[8] == Py_None) return THPVariable_Wrap(std::move(made));
    return Py_NewRef(a[8]);
    GUARDED_END
}

// accept(k_cache, v_cache, block_table, ctx_lens, paths, path_lens, stream) -> new ctx_lens
PyObject *accept(PyObject *, PyObject *const *a, Py_ssize_t n) {
    GUARDED_BEGIN
    if (!count_is(n, 7)) return nullptr;
    const Caches c = caches(a[0], a[1], true);
    const Tensor &ctx = vector(a[3], "ctx_lens", -1, c.index);
    const int64_t R = ctx.size(0);
    void *table = nullptr;
    const int64_t max_pages = table_columns(a[2], R, c.index, &table);
    const Tensor &lens = vector(a[5], "path_lens", R, c.index);
    void *paths = nullptr;
    int64_t width = 0;
    if (R) {
        const Tensor &p = matrix(a[4], "paths", R, c.index);
        paths = p.data_ptr();
        width = p.size(1);
    }
    const c10::cuda::CUDAGuard guard(static_cast<c10::DeviceIndex>(c.index));
    Tensor out = at::empty({R}, ctx.options());
    done(g_accept(c.k, c.v, c.layers, c.pages, c.heads, c.page_size, c.dim,
                  static_cast<int32_t *>(table), R, max_pages, static_cast<int32_t *>(ctx.data_ptr()),
                  static_cast<int32_t *>(paths), width, static_cast<int32_t *>(lens.data_ptr()),
                  static_cast<int32_t *>(out.data_ptr()), stream_of(a[6], c.index)),
         "swiglu_cache_accept");
    return THPVariable_Wrap(std::move(out));
    GUARDED_END
}

// connect(plan, write, workspace_bytes, attend, accept, SwigluError, workspace):
// the library's functions as addresses
PyObject *connect(PyObject *, PyObject *const *a, Py_ssize_t n) {
    if (!count_is(n, 7)) return nullptr;
    void *p[5];
    for (int i = 0; i < 5; ++i) {
        p[i] = PyLong_AsVoidPtr(a[i]);
        if (!p[i]) {
            if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, "a function has no address");
            return nullptr;
        }
    }
    g_plan = reinterpret_cast<decltype(g_plan)>(p[0]);
    g_write = reinterpret_cast<decltype(g_write)>(p[1]);
    g_attend_bytes = reinterpret_cast<decltype(g_attend_bytes)>(p[2]);
    g_attend = reinterpret_cast<decltype(g_attend)>(p[3]);
    g_accept = reinterpret_cast<decltype(g_accept)>(p[4]);
    Py_XDECREF(g_error);
    Py_XDECREF(g_workspace);
    g_error = Py_NewRef(a[5]);
    g_workspace = Py_NewRef(a[6]);
    Py_RETURN_NONE;
}

#define FAST(f) reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f)), METH_FASTCALL, ""
PyMethodDef g_methods[] = {{"connect", FAST(connect)}, {"plan", FAST(plan)},
                           {"write", FAST(write)},     {"attend", FAST(attend)},
                           {"accept", FAST(accept)},   {nullptr, nullptr, 0, nullptr}};
PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_cache_binding", nullptr, -1, g_methods,
                        nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__cache_binding(void) { return PyModule_Create(&g_module); }
