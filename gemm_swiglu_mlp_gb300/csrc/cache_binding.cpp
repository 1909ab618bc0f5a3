// The Python side of the paged-cache entry points and of the decode step's others
// (include/swiglu.h), natively: argument checks, device and stream, output buffers
// and the C ABI call.
//
// Small ones of these calls take 2 to 16 microseconds of GPU time in a serving step,
// several a layer. Checked and marshalled in Python they took the host 10.6 (plan),
// 7.4 (write), 13 (accept) and 18 (attention, which is two launches), so a step
// waited for its host; here they take 2.8, 2.0, 3.8 and 10.3, launches included.
// The module holds no operator: it calls the functions of libswiglu_gb300.so,
// whose addresses cache.py gives it. Python functions: cache.py and step.py.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/EmptyTensor.h>
#include <ATen/ops/empty.h>
#include <c10/cuda/CUDACachingAllocator.h>
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
decltype(&swiglu_head_rotate) g_rotate;
decltype(&swiglu_head_rotate_write) g_rotate_write;
decltype(&swiglu_verify_drafts) g_verify;
decltype(&swiglu_up_forward_q4) g_up_q4;
decltype(&swiglu_down_forward_q4) g_down_q4;
decltype(&swiglu_mlp_forward_q4) g_mlp_q4;
decltype(&swiglu_up_q4_workspace_bytes) g_up_q4_bytes, g_down_q4_bytes, g_mlp_q4_bytes;
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

// What the two rotations share: q and k, frequencies, weights, and q's output.
struct Rotation {
    const Tensor *q, *k, *positions;
    const float *inv_freq;
    int64_t T, q_heads, kv_heads, dim, freqs;
    void *q_weight, *k_weight;
    int index;
};
void *head_weight(PyObject *o, const char *name, int64_t dim, int index) {
    if (o == Py_None) return nullptr;
    const Tensor &w = cuda_tensor(o, name, at::kBFloat16, index);
    if (w.dim() != 1 || w.size(0) != dim || !w.is_contiguous())
        refuse(PyExc_ValueError, "%s must be a contiguous vector of %s%lld values", name, "", dim);
    return w.data_ptr();
}
Rotation rotation(PyObject *q, PyObject *k, PyObject *positions, PyObject *inv_freq,
                  PyObject *q_weight, PyObject *k_weight) {
    Rotation r{};
    const Tensor &qt = cuda_tensor(q, "q", at::kBFloat16, -1);
    r.index = qt.get_device();
    r.dim = qt.dim() == 3 ? qt.size(2) : -1;
    r.q = &rows(q, "q", -1, -1, r.dim, r.index);
    r.T = r.q->size(0);
    r.q_heads = r.q->size(1);
    r.k = &rows(k, "k", r.T, -1, r.dim, r.index);
    r.kv_heads = r.k->size(1);
    r.positions = &vector(positions, "positions", r.T, r.index);
    if (inv_freq != Py_None) {
        const Tensor &f = cuda_tensor(inv_freq, "inv_freq", at::kFloat, r.index);
        if (f.dim() != 1 || !f.is_contiguous())
            refuse(PyExc_ValueError, "%s must be a contiguous vector%s", "inv_freq");
        r.freqs = f.size(0);
        r.inv_freq = r.freqs ? static_cast<const float *>(f.data_ptr()) : nullptr;
    }
    r.q_weight = head_weight(q_weight, "q_weight", r.dim, r.index);
    r.k_weight = head_weight(k_weight, "k_weight", r.dim, r.index);
    return r;
}
const Tensor &made_or_given(PyObject *o, const char *name, const Tensor &like, Tensor *made) {
    if (o != Py_None)
        return rows(o, name, like.size(0), like.size(1), like.size(2), like.get_device());
    *made = at::empty(like.sizes(), like.options().memory_format(at::MemoryFormat::Contiguous));
    return *made;
}
double number(PyObject *o) {
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred()) throw Refused{};
    return v;
}
bool truth(PyObject *o) {
    const int v = PyObject_IsTrue(o);
    if (v < 0) throw Refused{};
    return v != 0;
}

// rotate(q, k, positions, inv_freq, q_weight, k_weight, eps, interleaved, q_out, k_out, stream)
//   -> (q_out, k_out)
PyObject *rotate(PyObject *, PyObject *const *a, Py_ssize_t n) {
    GUARDED_BEGIN
    if (!count_is(n, 11)) return nullptr;
    const Rotation r = rotation(a[0], a[1], a[2], a[3], a[4], a[5]);
    const float eps = static_cast<float>(number(a[6]));
    const bool interleaved = truth(a[7]);
    const c10::cuda::CUDAGuard guard(static_cast<c10::DeviceIndex>(r.index));
    Tensor made_q, made_k;
    const Tensor &qo = made_or_given(a[8], "q_out", *r.q, &made_q);
    const Tensor &ko = made_or_given(a[9], "k_out", *r.k, &made_k);
    done(g_rotate(r.q->data_ptr(), r.q->stride(0), r.q->stride(1), r.k->data_ptr(), r.k->stride(0),
                  r.k->stride(1), static_cast<int32_t *>(r.positions->data_ptr()), r.T, r.q_heads,
                  r.kv_heads, r.dim, r.inv_freq, r.freqs, interleaved, r.q_weight, r.k_weight, eps,
                  qo.data_ptr(), qo.stride(0), qo.stride(1), ko.data_ptr(), ko.stride(0),
                  ko.stride(1), stream_of(a[10], r.index)),
         "swiglu_head_rotate");
    PyObject *q = made_q.defined() ? THPVariable_Wrap(std::move(made_q)) : Py_NewRef(a[8]);
    PyObject *k = made_k.defined() ? THPVariable_Wrap(std::move(made_k)) : Py_NewRef(a[9]);
    return Py_BuildValue("(NN)", q, k);
    GUARDED_END
}

// rotate_write(q, k, v, positions, inv_freq, slots, k_cache, v_cache, q_weight, k_weight, eps,
//              interleaved, q_out, stream) -> q_out
PyObject *rotate_write(PyObject *, PyObject *const *a, Py_ssize_t n) {
    GUARDED_BEGIN
    if (!count_is(n, 14)) return nullptr;
    const Rotation r = rotation(a[0], a[1], a[3], a[4], a[8], a[9]);
    const Caches c = caches(a[6], a[7], false);
    if (c.index != r.index || c.heads != r.kv_heads || c.dim != r.dim)
        refuse(PyExc_ValueError, "%s must be on q's device and have k's heads%s: %lld of %lld values",
               "k_cache", "", c.heads, c.dim);
    const Tensor &v = rows(a[2], "v", r.T, r.kv_heads, r.dim, r.index);
    const Tensor &slots = vector(a[5], "slots", r.T, r.index);
    const float eps = static_cast<float>(number(a[10]));
    const bool interleaved = truth(a[11]);
    const c10::cuda::CUDAGuard guard(static_cast<c10::DeviceIndex>(r.index));
    Tensor made;
    const Tensor &qo = made_or_given(a[12], "q_out", *r.q, &made);
    done(g_rotate_write(r.q->data_ptr(), r.q->stride(0), r.q->stride(1), r.k->data_ptr(),
                        r.k->stride(0), r.k->stride(1), v.data_ptr(), v.stride(0), v.stride(1),
                        static_cast<int32_t *>(r.positions->data_ptr()),
                        static_cast<int32_t *>(slots.data_ptr()), r.T, r.q_heads, r.kv_heads, r.dim,
                        r.inv_freq, r.freqs, interleaved, r.q_weight, r.k_weight, eps, qo.data_ptr(),
                        qo.stride(0), qo.stride(1), c.k, c.v, c.pages, c.page_size,
                        stream_of(a[13], r.index)),
         "swiglu_head_rotate_write");
    return made.defined() ? THPVariable_Wrap(std::move(made)) : Py_NewRef(a[12]);
    GUARDED_END
}

// A [rows, vocab] table of probabilities: the last dimension contiguous.
const Tensor &probabilities(PyObject *o, const char *name, at::ScalarType type, int64_t rows,
                            int64_t vocab, int index) {
    const Tensor &t = cuda_tensor(o, name, type, index);
    if (t.dim() != 2 || t.size(0) != rows || t.size(1) < 1 || (vocab >= 0 && t.size(1) != vocab) ||
        (t.stride(1) != 1 && t.size(1) > 1))
        refuse(PyExc_ValueError, "%s must be [%s%lld, vocabulary] with a contiguous last dimension",
               name, "", rows);
    return t;
}
// (a single row's stride may be anything)
int64_t row_stride(const Tensor &t) { return t.size(0) > 1 ? t.stride(0) : t.size(1); }

// A new contiguous int32 tensor on the current device, in memory of its own (so that a caller may
// resize it), straight from the allocator: a greedy verification with three of them takes the
// host 4.7 to 5.1 us, with one allocation cut into three 4.5 to 5.5.
Tensor new_i32(at::IntArrayRef sizes) {
    return Tensor(at::detail::empty_generic(sizes, c10::cuda::CUDACachingAllocator::get(),
                                            c10::DispatchKeySet(c10::DispatchKey::CUDA), at::kInt,
                                            std::nullopt));
}

// verify(tokens, query_start, target, parents, draft, uniform, width, paths, path_lens,
//        next_tokens, stream) -> (paths, path_lens, next_tokens)
PyObject *verify(PyObject *, PyObject *const *a, Py_ssize_t n) {
    GUARDED_BEGIN
    if (!count_is(n, 11)) return nullptr;
    const Tensor &tokens = vector(a[0], "tokens", -1, -1);
    const int index = tokens.get_device();
    const int64_t T = tokens.size(0);
    const Tensor &start = vector(a[1], "query_start", -1, index);
    const int64_t R = start.size(0) - 1;
    if (R < 0) refuse(PyExc_ValueError, "%s must have a value for every request and one more%s",
                      "query_start");
    int64_t width = -1;
    void *parents = nullptr;
    if (a[3] != Py_None) {
        const Tensor &p = cuda_tensor(a[3], "parents", at::kInt, index);
        if (p.dim() != 2 || p.size(0) != R || p.size(1) < 1 || !p.is_contiguous())
            refuse(PyExc_ValueError, "%s must be contiguous, [%s%lld, at least 1]", "parents", "", R);
        parents = p.data_ptr();
        width = p.size(1);
    }
    if (a[6] == Py_None) {
        if (width < 0)
            refuse(PyExc_ValueError, "%s must be given for chains (no parents)%s", "width");
    } else {
        const int64_t w = integer(a[6]);
        if (w < 1 || (width >= 0 && w != width))
            refuse(PyExc_ValueError, "%s must be positive, and the parents' columns if there are "
                   "any%s, not %lld", "width", "", w);
        width = w;
    }
    const Tensor &any = cuda_tensor(a[2], "target", index);
    const bool greedy = any.scalar_type() == at::kInt;
    const Tensor *target = nullptr, *draft = nullptr, *uniform = nullptr;
    if (greedy) {
        target = &vector(a[2], "target", T, index);
        if (a[4] != Py_None || a[5] != Py_None)
            refuse(PyExc_ValueError, "%s and uniform do not go with a target of tokens%s", "draft");
    } else {
        if (any.scalar_type() != at::kFloat && any.scalar_type() != at::kBFloat16)
            refuse(PyExc_TypeError, "%s must be float32, bfloat16 or int32 (greedy tokens)%s",
                   "target");
        target = &probabilities(a[2], "target", any.scalar_type(), T, -1, index);
        if (a[4] != Py_None)
            draft = &probabilities(a[4], "draft", any.scalar_type(), T, target->size(1), index);
        const Tensor &u = cuda_tensor(a[5], "uniform", at::kFloat, index);
        if (u.dim() != 1 || u.size(0) != T || !u.is_contiguous())
            refuse(PyExc_ValueError, "%s must be a contiguous vector of %s%lld values", "uniform", "",
                   T);
        uniform = &u;
    }
    const c10::cuda::CUDAGuard guard(static_cast<c10::DeviceIndex>(index));
    Tensor made[3];
    void *out[3];
    static const char *const names[3] = {"out.paths", "out.path_lens", "out.next_tokens"};
    for (int i = 0; i < 3; ++i) {
        if (a[7 + i] == Py_None) {
            made[i] = i ? new_i32({R}) : new_i32({R, width});
            out[i] = made[i].data_ptr();
            continue;
        }
        const Tensor &t = cuda_tensor(a[7 + i], names[i], at::kInt, index);
        if (t.dim() != (i ? 1 : 2) || t.size(0) != R || (!i && t.size(1) != width) ||
            !t.is_contiguous())
            refuse(PyExc_ValueError, "%s must be contiguous, one row a request%s (%lld)", names[i], "",
                   R);
        out[i] = t.data_ptr();
    }
    done(g_verify(static_cast<int32_t *>(tokens.data_ptr()), T,
                  static_cast<int32_t *>(start.data_ptr()), R, static_cast<int32_t *>(parents), width,
                  target->data_ptr(), greedy ? 0 : row_stride(*target),
                  greedy ? SWIGLU_TARGET_TOKENS
                         : any.scalar_type() == at::kFloat ? SWIGLU_TARGET_FP32 : SWIGLU_TARGET_BF16,
                  draft ? draft->data_ptr() : nullptr, draft ? row_stride(*draft) : 0,
                  greedy ? 0 : target->size(1),
                  uniform ? static_cast<float *>(uniform->data_ptr()) : nullptr,
                  static_cast<int32_t *>(out[0]), static_cast<int32_t *>(out[1]),
                  static_cast<int32_t *>(out[2]), stream_of(a[10], index)),
         "swiglu_verify_drafts");
    PyObject *o[3];
    for (int i = 0; i < 3; ++i)
        o[i] = made[i].defined() ? THPVariable_Wrap(std::move(made[i])) : Py_NewRef(a[7 + i]);
    return Py_BuildValue("(NNN)", o[0], o[1], o[2]);
    GUARDED_END
}

// A weight of 4-bit codes [columns, length / 2] bytes and its scales [groups, columns].
struct Codes {
    void *codes, *scales;
    int64_t columns;
};
Codes q4_weight(PyObject *q, PyObject *s, const char *name, const char *scale_name, int64_t columns,
                int64_t length, int64_t group, int index) {
    const Tensor &c = cuda_tensor(q, name, at::kByte, index);
    if (c.dim() != 2 || length % 2 || c.size(1) != length / 2 ||
        (columns >= 0 && c.size(0) != columns) || !c.is_contiguous())
        refuse(PyExc_ValueError, "%s must be contiguous bytes, [columns, %s%lld]: two codes each",
               name, "", length / 2);
    const Tensor &t = cuda_tensor(s, scale_name, at::kBFloat16, index);
    if (t.dim() != 2 || t.size(0) != (length + group - 1) / group || t.size(1) != c.size(0) ||
        !t.is_contiguous())
        refuse(PyExc_ValueError, "%s must be contiguous, [%s%lld, %lld]: a group's in a row",
               scale_name, "", (length + group - 1) / group, c.size(0));
    return {c.data_ptr(), t.data_ptr(), c.size(0)};
}
int64_t q4_group(PyObject *o) {
    const int64_t g = integer(o);
    if (g != 32 && g != 64 && g != 128)
        refuse(PyExc_ValueError, "%s must be 32, 64 or 128%s, not %lld", "group", "", g);
    return g;
}
const Tensor &q4_rows(PyObject *o, const char *name, int64_t rows, int64_t columns, int index) {
    const Tensor &t = cuda_tensor(o, name, at::kBFloat16, index);
    if (t.dim() != 2 || (rows >= 0 && t.size(0) != rows) || (columns >= 0 && t.size(1) != columns) ||
        !t.is_contiguous())
        refuse(PyExc_ValueError, "%s must be a contiguous matrix%s of %lld rows", name, "",
               rows >= 0 ? rows : t.dim() == 2 ? t.size(0) : -1);
    return t;
}
const Tensor &q4_out(PyObject *o, const char *name, const Tensor &like, int64_t columns,
                     Tensor *made) {
    if (o != Py_None) return q4_rows(o, name, like.size(0), columns, like.get_device());
    *made = at::empty({like.size(0), columns}, like.options());
    return *made;
}

// The caller's workspace, or one of this call's own where one is used: from the current
// stream's memory (under capture, of the graph's pool), which may be given out again behind it.
struct Scratch {
    Tensor made;
    void *p = nullptr;
    size_t bytes = 0;
    Scratch(PyObject *o, size_t need, const Tensor &like) {
        if (o != Py_None) {
            const Tensor &w = cuda_tensor(o, "workspace", like.get_device());
            if (!w.is_contiguous()) refuse(PyExc_ValueError, "%s must be contiguous%s", "workspace");
            p = w.data_ptr();
            bytes = w.nbytes();
        } else if (need) {
            made = at::empty({static_cast<int64_t>(need)}, like.options().dtype(at::kByte));
            p = made.data_ptr();
            bytes = need;
        }
    }
};

// up_q4(A, Q1, S1, Q2, S2, group, Y, workspace, stream) -> Y
PyObject *up_q4(PyObject *, PyObject *const *a, Py_ssize_t n) {
    GUARDED_BEGIN
    if (!count_is(n, 9)) return nullptr;
    const Tensor &A = q4_rows(a[0], "A", -1, -1, -1);
    const int index = A.get_device();
    const int64_t M = A.size(0), K = A.size(1), group = q4_group(a[5]);
    const Codes w1 = q4_weight(a[1], a[2], "Q1", "S1", -1, K, group, index);
    const Codes w2 = q4_weight(a[3], a[4], "Q2", "S2", w1.columns, K, group, index);
    const c10::cuda::CUDAGuard guard(static_cast<c10::DeviceIndex>(index));
    Tensor made;
    const Tensor &Y = q4_out(a[6], "Y", A, w1.columns, &made);
    const Scratch ws(a[7], g_up_q4_bytes(M, w1.columns, K, group), A);
    done(g_up_q4(A.data_ptr(), w1.codes, w1.scales, w2.codes, w2.scales, Y.data_ptr(), M, w1.columns,
                 K, group, ws.p, ws.bytes, stream_of(a[8], index)),
         "swiglu_up_forward_q4");
    return made.defined() ? THPVariable_Wrap(std::move(made)) : Py_NewRef(a[6]);
    GUARDED_END
}

// down_q4(Y, Q3, S3, group, out, workspace, stream) -> out
PyObject *down_q4(PyObject *, PyObject *const *a, Py_ssize_t n) {
    GUARDED_BEGIN
    if (!count_is(n, 7)) return nullptr;
    const Tensor &Y = q4_rows(a[0], "Y", -1, -1, -1);
    const int index = Y.get_device();
    const int64_t M = Y.size(0), N = Y.size(1), group = q4_group(a[3]);
    const Codes w3 = q4_weight(a[1], a[2], "Q3", "S3", -1, N, group, index);
    const c10::cuda::CUDAGuard guard(static_cast<c10::DeviceIndex>(index));
    Tensor made;
    const Tensor &out = q4_out(a[4], "out", Y, w3.columns, &made);
    const Scratch ws(a[5], g_down_q4_bytes(M, N, w3.columns, group), Y);
    done(g_down_q4(Y.data_ptr(), w3.codes, w3.scales, out.data_ptr(), M, N, w3.columns, group, ws.p,
                   ws.bytes, stream_of(a[6], index)),
         "swiglu_down_forward_q4");
    return made.defined() ? THPVariable_Wrap(std::move(made)) : Py_NewRef(a[4]);
    GUARDED_END
}

// mlp_q4(A, Q1, S1, Q2, S2, Q3, S3, group, Y, out, workspace, stream) -> out
PyObject *mlp_q4(PyObject *, PyObject *const *a, Py_ssize_t n) {
    GUARDED_BEGIN
    if (!count_is(n, 12)) return nullptr;
    const Tensor &A = q4_rows(a[0], "A", -1, -1, -1);
    const int index = A.get_device();
    const int64_t M = A.size(0), K = A.size(1), group = q4_group(a[7]);
    const Codes w1 = q4_weight(a[1], a[2], "Q1", "S1", -1, K, group, index);
    const Codes w2 = q4_weight(a[3], a[4], "Q2", "S2", w1.columns, K, group, index);
    const Codes w3 = q4_weight(a[5], a[6], "Q3", "S3", K, w1.columns, group, index);
    const c10::cuda::CUDAGuard guard(static_cast<c10::DeviceIndex>(index));
    Tensor made_y, made;
    const Tensor &Y = q4_out(a[8], "Y", A, w1.columns, &made_y);
    const Tensor &out = q4_out(a[9], "out", A, K, &made);
    const Scratch ws(a[10], g_mlp_q4_bytes(M, w1.columns, K, group), A);
    done(g_mlp_q4(A.data_ptr(), w1.codes, w1.scales, w2.codes, w2.scales, w3.codes, w3.scales,
                  Y.data_ptr(), out.data_ptr(), M, w1.columns, K, group, ws.p, ws.bytes,
                  stream_of(a[11], index)),
         "swiglu_mlp_forward_q4");
    return made.defined() ? THPVariable_Wrap(std::move(made)) : Py_NewRef(a[9]);
    GUARDED_END
}

// connect(plan, write, workspace_bytes, attend, accept, rotate, rotate_write, verify, up_q4,
// down_q4, mlp_q4, their workspace_bytes, SwigluError, workspace): the library's functions as
// addresses
PyObject *connect(PyObject *, PyObject *const *a, Py_ssize_t n) {
    constexpr int kFunctions = 14;
    if (!count_is(n, kFunctions + 2)) return nullptr;
    void *p[kFunctions];
    for (int i = 0; i < kFunctions; ++i) {
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
    g_rotate = reinterpret_cast<decltype(g_rotate)>(p[5]);
    g_rotate_write = reinterpret_cast<decltype(g_rotate_write)>(p[6]);
    g_verify = reinterpret_cast<decltype(g_verify)>(p[7]);
    g_up_q4 = reinterpret_cast<decltype(g_up_q4)>(p[8]);
    g_down_q4 = reinterpret_cast<decltype(g_down_q4)>(p[9]);
    g_mlp_q4 = reinterpret_cast<decltype(g_mlp_q4)>(p[10]);
    g_up_q4_bytes = reinterpret_cast<decltype(g_up_q4_bytes)>(p[11]);
    g_down_q4_bytes = reinterpret_cast<decltype(g_down_q4_bytes)>(p[12]);
    g_mlp_q4_bytes = reinterpret_cast<decltype(g_mlp_q4_bytes)>(p[13]);
    Py_XDECREF(g_error);
    Py_XDECREF(g_workspace);
    g_error = Py_NewRef(a[kFunctions]);
    g_workspace = Py_NewRef(a[kFunctions + 1]);
    Py_RETURN_NONE;
}

#define FAST(f) reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f)), METH_FASTCALL, ""
PyMethodDef g_methods[] = {{"connect", FAST(connect)}, {"plan", FAST(plan)},
                           {"write", FAST(write)},     {"attend", FAST(attend)},
                           {"accept", FAST(accept)},   {"rotate", FAST(rotate)},
                           {"rotate_write", FAST(rotate_write)},
                           {"verify", FAST(verify)},   {"up_q4", FAST(up_q4)},
                           {"down_q4", FAST(down_q4)}, {"mlp_q4", FAST(mlp_q4)},
                           {nullptr, nullptr, 0, nullptr}};
PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_cache_binding", nullptr, -1, g_methods,
                        nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__cache_binding(void) { return PyModule_Create(&g_module); }
