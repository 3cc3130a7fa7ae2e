// Marshalling of the serving calls (serving.py, prompt.py) for the usual case, in C: every tensor a plain,
// contiguous one of the expected type and shape on the current device.  A small call is bound by the
// host, and Python's checks and ctypes' argument conversion are most of its 7 to 14 us.
//
// Each function takes the Python call's arguments in order and returns its result, or False where
// anything is not as usual; the Python call then goes its own way, which handles strides and other devices
// and raises what is to be raised.  The library's functions are given by address, so this module links
// only torch and nothing of it computes.
#include <Python.h>

#include <ATen/ops/empty.h>
#include <c10/core/impl/VirtualGuardImpl.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <climits>
#include <cmath>

#include "kda.h"

namespace {

PyObject* g_raw_stream = nullptr;  // device index -> handle of its current stream
PyObject* g_check = nullptr;       // status -> raises

decltype(&kda_cache_append) f_append;
decltype(&kda_paged_decode) f_decode;
decltype(&kda_paged_decode_workspace) f_decode_ws;
decltype(&kda_cache_fork) f_fork;
decltype(&kda_cache_free) f_free;
decltype(&kda_cache_reserve) f_reserve;
decltype(&kda_cache_compact) f_compact;
decltype(&kda_cache_workspace_size) f_cache_ws;
decltype(&kda_pages_copy) f_copy;
decltype(&kda_beam_select) f_select;
decltype(&kda_beam_select_workspace) f_select_ws;
decltype(&kda_beam_reorder) f_reorder;
decltype(&kda_rotary) f_rotary;
decltype(&kda_rotary_append) f_place;
decltype(&kda_paged_prefill) f_prefill;
decltype(&kda_paged_prefill_workspace) f_prefill_ws;
decltype(&kda_token_logprobs) f_logprobs;
decltype(&kda_token_logprobs_workspace) f_logprobs_ws;
decltype(&kda_token_logprobs_grad) f_logprobs_grad;

using at::Tensor;
constexpr auto kI32 = at::kInt;

// the tensor behind a plain contiguous GPU argument of that type and number of axes, or nullptr
const Tensor* plain(PyObject* o, at::ScalarType type, int dim, int dev) {
    if (!THPVariable_CheckExact(o)) return nullptr;
    const Tensor& t = THPVariable_Unpack(o);
    if (!t.is_cuda() || t.device().index() != dev || t.scalar_type() != type || (dim >= 0 && t.dim() != dim) ||
        !t.is_contiguous())
        return nullptr;
    return &t;
}

// device of a plain GPU tensor if it is the current one, else -1
int device_of(PyObject* o) {
    if (!THPVariable_CheckExact(o)) return -1;
    const Tensor& t = THPVariable_Unpack(o);
    if (!t.is_cuda()) return -1;
    const int dev = t.device().index();
    return c10::impl::VirtualGuardImpl(c10::DeviceType::CUDA).getDevice().index() == dev ? dev : -1;
}

int code_of(PyObject* o) {
    const auto t = THPVariable_Unpack(o).scalar_type();
    return t == at::kFloat ? KDA_F32 : t == at::kBFloat16 ? KDA_BF16 : -1;
}

bool small(int64_t x) { return x >= INT32_MIN && x <= INT32_MAX; }

// an int argument that fits 32 bits
bool int_of(PyObject* o, int32_t& x) {
    if (!PyLong_CheckExact(o)) return false;
    int over = 0;
    const long y = PyLong_AsLongAndOverflow(o, &over);
    if (over || !small(y)) return false;
    x = (int32_t)y;
    return true;
}

// the current stream's handle; false with a Python error set
bool stream_of(int dev, void*& s) {
    PyObject* i = PyLong_FromLong(dev);
    PyObject* r = i ? PyObject_CallOneArg(g_raw_stream, i) : nullptr;
    Py_XDECREF(i);
    if (!r) return false;
    s = PyLong_AsVoidPtr(r);
    Py_DECREF(r);
    return !(s == nullptr && PyErr_Occurred());
}

// true for KDA_OK; else false with the Python error of the status set
bool passed(int status) {
    if (status == KDA_OK) return true;
    PyObject* r = PyObject_CallFunction(g_check, "i", status);
    if (r) {
        Py_DECREF(r);
        PyErr_SetString(PyExc_RuntimeError, "library call failed");
    }
    return false;
}

Tensor fresh(at::IntArrayRef shape, at::ScalarType type, const Tensor& like) {
    return at::empty(shape, like.options().dtype(type));
}

// The caller's workspace if it is a plain byte tensor of at least `need` bytes, else a new one;
// false for an argument that is not usual.
bool workspace_of(PyObject* o, size_t need, int dev, const Tensor& like, Tensor& keep, void*& p, size_t& bytes) {
    if (need == (size_t)-1) return false;
    if (o != Py_None) {
        const Tensor* t = plain(o, at::kByte, -1, dev);
        if (!t) return false;
        if ((size_t)t->numel() >= need) {
            p = t->data_ptr();
            bytes = (size_t)t->numel();
            return true;
        }
    }
    p = nullptr;
    bytes = need;
    if (need) {
        keep = fresh({(int64_t)need}, at::kByte, like);
        p = keep.data_ptr();
    }
    return true;
}

// an optional output: the given plain tensor of that shape, or a new one
bool output_of(PyObject* o, at::IntArrayRef shape, at::ScalarType type, int dev, const Tensor& like, Tensor& out) {
    if (o == Py_None) {
        out = fresh(shape, type, like);
        return true;
    }
    const Tensor* t = plain(o, type, (int)shape.size(), dev);
    if (!t || t->sizes() != shape) return false;
    out = *t;
    return true;
}

// Marks a tensor as modified in place, for autograd (inference tensors have no version).
void written(const Tensor& t) {
    if (!t.is_inference()) t.unsafeGetTensorImpl()->bump_version();
}

#define KDA_USUAL(cond) \
    if (!(cond)) Py_RETURN_FALSE
#define KDA_CALL(status_expr)            \
    void* stream = nullptr;              \
    if (!stream_of(dev, stream)) return nullptr; \
    int status;                          \
    Py_BEGIN_ALLOW_THREADS               \
    status = (status_expr);              \
    Py_END_ALLOW_THREADS                 \
    if (!passed(status)) return nullptr

PyObject* pair(Tensor a, Tensor b) {
    PyObject* x = THPVariable_Wrap(std::move(a));
    PyObject* y = THPVariable_Wrap(std::move(b));
    PyObject* r = x && y ? PyTuple_Pack(2, x, y) : nullptr;
    Py_XDECREF(x);
    Py_XDECREF(y);
    return r;
}

// k, v, k_pages, v_pages, page_table, start, cu_seqlens
PyObject* cache_append(PyObject*, PyObject* const* a, Py_ssize_t n_args) {
    HANDLE_TH_ERRORS
    KDA_USUAL(n_args == 7);
    const int dev = device_of(a[0]);
    KDA_USUAL(dev >= 0);
    const int code = code_of(a[0]);
    KDA_USUAL(code >= 0);
    const auto type = THPVariable_Unpack(a[0]).scalar_type();
    const Tensor *k = plain(a[0], type, 3, dev), *v = plain(a[1], type, 3, dev), *kp = plain(a[2], type, 4, dev),
                 *vp = plain(a[3], type, 4, dev), *table = plain(a[4], kI32, 2, dev), *start = plain(a[5], kI32, 1, dev);
    KDA_USUAL(k && v && kp && vp && table && start);
    KDA_USUAL(k->sizes() == v->sizes() && kp->sizes() == vp->sizes() && kp->size(1) == k->size(1) &&
              kp->size(3) == k->size(2) && start->size(0) == table->size(0));
    const Tensor* cu = nullptr;
    if (a[6] != Py_None) {
        cu = plain(a[6], kI32, 1, dev);
        KDA_USUAL(cu && cu->size(0) == table->size(0) + 1);
    }
    KDA_USUAL(small(k->numel() / (k->size(2) ? k->size(2) : 1)) && small(kp->size(0)) && small(kp->size(2)) &&
              small(table->size(0)) && small(table->size(1)));
    KDA_CALL(f_append(k->data_ptr(), v->data_ptr(), k->stride(0), v->stride(0),
                      cu ? static_cast<const int32_t*>(cu->data_ptr()) : nullptr,
                      static_cast<const int32_t*>(start->data_ptr()), (int32_t)table->size(0), k->size(0),
                      kp->data_ptr(), vp->data_ptr(), kp->stride(0), vp->stride(0), (int32_t)kp->size(0),
                      (int32_t)kp->size(2), static_cast<const int32_t*>(table->data_ptr()), table->stride(0),
                      (int32_t)table->size(1), (int32_t)k->size(1), (int32_t)k->size(2), code, stream));
    Py_RETURN_NONE;
    END_HANDLE_TH_ERRORS
}

// q, k_pages, v_pages, page_table, lengths, scale, window, sinks, max_length, out, lse, workspace
PyObject* paged_decode(PyObject*, PyObject* const* a, Py_ssize_t n_args) {
    HANDLE_TH_ERRORS
    KDA_USUAL(n_args == 12);
    const int dev = device_of(a[0]);
    KDA_USUAL(dev >= 0);
    const int code = code_of(a[0]);
    KDA_USUAL(code >= 0);
    const auto type = THPVariable_Unpack(a[0]).scalar_type();
    const Tensor *q = plain(a[0], type, 3, dev), *kp = plain(a[1], type, 4, dev), *vp = plain(a[2], type, 4, dev),
                 *table = plain(a[3], kI32, 2, dev), *lengths = plain(a[4], kI32, 1, dev);
    KDA_USUAL(q && kp && vp && table && lengths);
    const int64_t N = q->size(0), Hq = q->size(1), d = q->size(2), P = table->size(1), page = kp->size(2);
    KDA_USUAL(kp->sizes() == vp->sizes() && kp->size(3) == d && table->size(0) == N && lengths->size(0) == N);
    KDA_USUAL(small(N) && small(Hq) && small(d) && small(P) && small(page) && small(kp->size(0)) &&
              small(kp->size(1)) && small(P * page));
    int32_t window, sinks, most = (int32_t)(P * page);
    KDA_USUAL(int_of(a[6], window) && int_of(a[7], sinks));
    if (a[8] != Py_None) {
        int32_t bound;
        KDA_USUAL(int_of(a[8], bound) && bound > 0);
        most = bound < most ? bound : most;
    }
    double scale = 0.;
    if (a[5] != Py_None) {
        KDA_USUAL(PyFloat_CheckExact(a[5]));
        scale = PyFloat_AS_DOUBLE(a[5]);
    } else {
        scale = d > 0 ? std::pow((double)d, -0.5) : 0.;
    }
    const size_t need = f_decode_ws((int32_t)N, (int32_t)Hq, (int32_t)kp->size(1), (int32_t)d, code, most, window, sinks);
    Tensor keep, out, lse;
    void* ws;
    size_t ws_bytes;
    KDA_USUAL(workspace_of(a[11], need, dev, *q, keep, ws, ws_bytes));
    KDA_USUAL(output_of(a[9], q->sizes(), at::kFloat, dev, *q, out));
    const bool want = a[10] != Py_None && a[10] != Py_False;
    if (want) KDA_USUAL(output_of(a[10] == Py_True ? Py_None : a[10], {N, Hq}, at::kFloat, dev, *q, lse));
    KDA_CALL(f_decode(q->data_ptr(), q->stride(0), kp->data_ptr(), vp->data_ptr(), kp->stride(0), vp->stride(0),
                      (int32_t)kp->size(0), (int32_t)page, static_cast<const int32_t*>(table->data_ptr()),
                      table->stride(0), (int32_t)P, static_cast<const int32_t*>(lengths->data_ptr()), (int32_t)N,
                      (int32_t)Hq, (int32_t)kp->size(1), (int32_t)d, code, (float)scale, window, sinks, most,
                      static_cast<float*>(out.data_ptr()), want ? static_cast<float*>(lse.data_ptr()) : nullptr, ws,
                      ws_bytes, stream));
    return want ? pair(std::move(out), std::move(lse)) : THPVariable_Wrap(std::move(out));
    END_HANDLE_TH_ERRORS
}

int32_t* ints(const Tensor& t) { return static_cast<int32_t*>(t.data_ptr()); }

// page_table, lengths, refcount, parents, table_out, lengths_out
PyObject* cache_fork(PyObject*, PyObject* const* a, Py_ssize_t n_args) {
    HANDLE_TH_ERRORS
    KDA_USUAL(n_args == 6);
    const int dev = device_of(a[0]);
    KDA_USUAL(dev >= 0);
    const Tensor *table = plain(a[0], kI32, 2, dev), *lengths = plain(a[1], kI32, 1, dev),
                 *refs = plain(a[2], kI32, 1, dev), *parents = plain(a[3], kI32, 1, dev);
    KDA_USUAL(table && lengths && refs && parents);
    const int64_t N = table->size(0), P = table->size(1), M = parents->size(0);
    KDA_USUAL(lengths->size(0) == N && small(N) && small(P) && small(M) && small(refs->size(0)));
    Tensor out, lengths_out;
    KDA_USUAL(output_of(a[4], {M, P}, kI32, dev, *table, out) && output_of(a[5], {M}, kI32, dev, *table, lengths_out));
    KDA_CALL(f_fork(ints(*table), table->stride(0), ints(*lengths), (int32_t)N, (int32_t)P, ints(*refs),
                    (int32_t)refs->size(0), ints(*parents), (int32_t)M, ints(out), out.stride(0), ints(lengths_out),
                    stream));
    return pair(std::move(out), std::move(lengths_out));
    END_HANDLE_TH_ERRORS
}

// page_table, lengths, refcount, rows
PyObject* cache_free(PyObject*, PyObject* const* a, Py_ssize_t n_args) {
    HANDLE_TH_ERRORS
    KDA_USUAL(n_args == 4);
    const int dev = device_of(a[0]);
    KDA_USUAL(dev >= 0);
    const Tensor *table = plain(a[0], kI32, 2, dev), *lengths = plain(a[1], kI32, 1, dev),
                 *refs = plain(a[2], kI32, 1, dev), *rows = plain(a[3], kI32, 1, dev);
    KDA_USUAL(table && lengths && refs && rows);
    const int64_t N = table->size(0), P = table->size(1);
    KDA_USUAL(lengths->size(0) == N && small(N) && small(P) && small(rows->size(0)) && small(refs->size(0)));
    KDA_CALL(f_free(ints(*table), table->stride(0), ints(*lengths), (int32_t)N, (int32_t)P, ints(*refs),
                    (int32_t)refs->size(0), ints(*rows), (int32_t)rows->size(0), stream));
    Py_RETURN_NONE;
    END_HANDLE_TH_ERRORS
}

// page_table, lengths, refcount, new_tokens, page_size, copies, granted, workspace
PyObject* cache_reserve(PyObject*, PyObject* const* a, Py_ssize_t n_args) {
    HANDLE_TH_ERRORS
    KDA_USUAL(n_args == 8);
    const int dev = device_of(a[0]);
    KDA_USUAL(dev >= 0);
    const Tensor *table = plain(a[0], kI32, 2, dev), *lengths = plain(a[1], kI32, 1, dev),
                 *refs = plain(a[2], kI32, 1, dev), *add = plain(a[3], kI32, 1, dev);
    int32_t page;
    KDA_USUAL(table && lengths && refs && add && int_of(a[4], page));
    const int64_t N = table->size(0), P = table->size(1);
    KDA_USUAL(lengths->size(0) == N && add->size(0) == N && small(N) && small(P) && small(refs->size(0)));
    Tensor keep, copies, granted;
    void* ws;
    size_t ws_bytes;
    KDA_USUAL(workspace_of(a[7], f_cache_ws((int32_t)N, (int32_t)refs->size(0)), dev, *table, keep, ws, ws_bytes));
    KDA_USUAL(output_of(a[5], {N, 2}, kI32, dev, *table, copies) && output_of(a[6], {N}, kI32, dev, *table, granted));
    KDA_CALL(f_reserve(ints(*table), table->stride(0), ints(*lengths), (int32_t)N, (int32_t)P, ints(*refs),
                       (int32_t)refs->size(0), page, ints(*add), ints(copies), ints(granted), ws, ws_bytes, stream));
    return pair(std::move(copies), std::move(granted));
    END_HANDLE_TH_ERRORS
}

// page_table, refcount, table_out, refcount_out, moves, workspace
PyObject* cache_compact(PyObject*, PyObject* const* a, Py_ssize_t n_args) {
    HANDLE_TH_ERRORS
    KDA_USUAL(n_args == 6);
    const int dev = device_of(a[0]);
    KDA_USUAL(dev >= 0);
    const Tensor *table = plain(a[0], kI32, 2, dev), *refs = plain(a[1], kI32, 1, dev);
    KDA_USUAL(table && refs);
    const int64_t N = table->size(0), P = table->size(1), pages = refs->size(0);
    KDA_USUAL(small(N) && small(P) && small(pages));
    Tensor keep, out, refs_out, moves;
    void* ws;
    size_t ws_bytes;
    KDA_USUAL(workspace_of(a[5], f_cache_ws((int32_t)N, (int32_t)pages), dev, *table, keep, ws, ws_bytes));
    KDA_USUAL(output_of(a[2], {N, P}, kI32, dev, *table, out) && output_of(a[3], {pages}, kI32, dev, *table, refs_out) &&
              output_of(a[4], {pages / 2, 2}, kI32, dev, *table, moves));
    KDA_CALL(f_compact(ints(*table), table->stride(0), (int32_t)N, (int32_t)P, ints(*refs), (int32_t)pages, ints(out),
                       out.stride(0), ints(refs_out), ints(moves), ws, ws_bytes, stream));
    PyObject* x = THPVariable_Wrap(std::move(out));
    PyObject* y = THPVariable_Wrap(std::move(refs_out));
    PyObject* z = THPVariable_Wrap(std::move(moves));
    PyObject* r = x && y && z ? PyTuple_Pack(3, x, y, z) : nullptr;
    Py_XDECREF(x);
    Py_XDECREF(y);
    Py_XDECREF(z);
    return r;
    END_HANDLE_TH_ERRORS
}

constexpr Py_ssize_t kMost = 64;  // buffers of a list

// The buffers of a list (or a single tensor): contiguous, `rows` rows each; false where not usual.
bool buffers_of(PyObject* o, int dev, int64_t rows, int least_dim, void** base, int64_t* bytes, int32_t& count) {
    PyObject* one[1] = {o};
    PyObject** item = one;
    Py_ssize_t n = 1;
    if (PyList_CheckExact(o)) {
        n = PyList_GET_SIZE(o);
        item = &PyList_GET_ITEM(o, 0);
    } else if (PyTuple_CheckExact(o)) {
        n = PyTuple_GET_SIZE(o);
        item = &PyTuple_GET_ITEM(o, 0);
    }
    if (n < 1 || n > kMost) return false;
    for (Py_ssize_t i = 0; i < n; ++i) {
        if (!THPVariable_CheckExact(item[i])) return false;
        const Tensor& t = THPVariable_Unpack(item[i]);
        if (!t.is_cuda() || t.device().index() != dev || t.dim() < least_dim || !t.is_contiguous() || t.size(0) != rows)
            return false;
        base[i] = t.data_ptr();
        bytes[i] = rows ? t.numel() / rows * (int64_t)t.element_size() : 0;
    }
    count = (int32_t)n;
    return true;
}

PyObject* first_of(PyObject* o) {
    if (PyList_CheckExact(o)) return PyList_GET_SIZE(o) ? PyList_GET_ITEM(o, 0) : o;
    if (PyTuple_CheckExact(o)) return PyTuple_GET_SIZE(o) ? PyTuple_GET_ITEM(o, 0) : o;
    return o;
}

// pools, pairs
PyObject* pages_copy(PyObject*, PyObject* const* a, Py_ssize_t n_args) {
    HANDLE_TH_ERRORS
    KDA_USUAL(n_args == 2);
    PyObject* first = first_of(a[0]);
    const int dev = device_of(first);
    KDA_USUAL(dev >= 0 && THPVariable_Unpack(first).dim() > 1);
    const int64_t pages = THPVariable_Unpack(first).size(0);
    const Tensor* pairs = plain(a[1], kI32, 2, dev);
    void* base[kMost];
    int64_t bytes[kMost];
    int32_t n;
    KDA_USUAL(pairs && pairs->size(1) == 2 && small(pages) && buffers_of(a[0], dev, pages, 2, base, bytes, n));
    KDA_CALL(f_copy(base, bytes, bytes, n, (int32_t)pages, ints(*pairs), pairs->size(0), stream));
    Py_RETURN_NONE;
    END_HANDLE_TH_ERRORS
}

// states, parents
PyObject* beam_reorder(PyObject*, PyObject* const* a, Py_ssize_t n_args) {
    HANDLE_TH_ERRORS
    KDA_USUAL(n_args == 2);
    const int dev = device_of(first_of(a[0]));
    KDA_USUAL(dev >= 0);
    const Tensor* parents = plain(a[1], kI32, 2, dev);
    KDA_USUAL(parents && small(parents->size(0)) && small(parents->size(1)));
    void* base[kMost];
    int64_t bytes[kMost];
    int32_t n;
    KDA_USUAL(buffers_of(a[0], dev, parents->size(0) * parents->size(1), 1, base, bytes, n));
    KDA_CALL(f_reorder(base, bytes, n, ints(*parents), (int32_t)parents->size(0), (int32_t)parents->size(1), stream));
    Py_RETURN_NONE;
    END_HANDLE_TH_ERRORS
}

// logits, scores, n_out, finished, eos, workspace
PyObject* beam_select(PyObject*, PyObject* const* a, Py_ssize_t n_args) {
    HANDLE_TH_ERRORS
    KDA_USUAL(n_args == 6);
    const int dev = device_of(a[0]);
    KDA_USUAL(dev >= 0);
    const int code = code_of(a[0]);
    KDA_USUAL(code >= 0);
    const Tensor *logits = plain(a[0], THPVariable_Unpack(a[0]).scalar_type(), 3, dev),
                 *scores = plain(a[1], at::kFloat, 2, dev);
    KDA_USUAL(logits && scores);
    const int64_t B = logits->size(0), K = logits->size(1), V = logits->size(2);
    KDA_USUAL(scores->size(0) == B && scores->size(1) == K && small(B) && small(K) && small(V));
    int32_t n_out = (int32_t)K, eos;
    KDA_USUAL((a[2] == Py_None || int_of(a[2], n_out)) && n_out > 0 && int_of(a[4], eos));
    const Tensor* finished = nullptr;
    Tensor over, keep;
    if (a[3] != Py_None) {
        KDA_USUAL(THPVariable_CheckExact(a[3]));
        const auto type = THPVariable_Unpack(a[3]).scalar_type();
        KDA_USUAL(type == at::kByte || type == at::kBool);
        finished = plain(a[3], type, 2, dev);
        KDA_USUAL(finished && finished->sizes() == scores->sizes());
        over = fresh({B, n_out}, type, *logits);
    }
    void* ws;
    size_t ws_bytes;
    KDA_USUAL(workspace_of(a[5], f_select_ws((int32_t)B, (int32_t)K, (int32_t)V, n_out), dev, *logits, keep, ws, ws_bytes));
    Tensor best = fresh({B, n_out}, at::kFloat, *logits), parents = fresh({B, n_out}, kI32, *logits),
           tokens = fresh({B, n_out}, kI32, *logits);
    KDA_CALL(f_select(logits->data_ptr(), V, static_cast<const float*>(scores->data_ptr()),
                      finished ? static_cast<const uint8_t*>(finished->data_ptr()) : nullptr, (int32_t)B, (int32_t)K,
                      (int32_t)V, n_out, eos, code, static_cast<float*>(best.data_ptr()), ints(parents), ints(tokens),
                      finished ? static_cast<uint8_t*>(over.data_ptr()) : nullptr, ws, ws_bytes, stream));
    PyObject* r = PyTuple_New(4);
    if (!r) return nullptr;
    PyTuple_SET_ITEM(r, 0, THPVariable_Wrap(std::move(best)));
    PyTuple_SET_ITEM(r, 1, THPVariable_Wrap(std::move(parents)));
    PyTuple_SET_ITEM(r, 2, THPVariable_Wrap(std::move(tokens)));
    if (finished) {
        PyTuple_SET_ITEM(r, 3, THPVariable_Wrap(std::move(over)));
    } else {
        Py_INCREF(Py_None);
        PyTuple_SET_ITEM(r, 3, Py_None);
    }
    return r;
    END_HANDLE_TH_ERRORS
}

// "half" or "interleaved"
bool layout_of(PyObject* o, int32_t& x) {
    if (!PyUnicode_CheckExact(o)) return false;
    if (PyUnicode_CompareWithASCIIString(o, "half") == 0) x = KDA_ROTARY_HALVES;
    else if (PyUnicode_CompareWithASCIIString(o, "interleaved") == 0) x = KDA_ROTARY_INTERLEAVED;
    else return false;
    return true;
}

// q, k, positions, freqs, layout, amplitude, inverse, q_out, k_out
PyObject* rotary(PyObject*, PyObject* const* a, Py_ssize_t n_args) {
    HANDLE_TH_ERRORS
    KDA_USUAL(n_args == 9);
    const int dev = device_of(a[0]);
    KDA_USUAL(dev >= 0);
    const int code = code_of(a[0]);
    KDA_USUAL(code >= 0);
    const auto type = THPVariable_Unpack(a[0]).scalar_type();
    const Tensor *q = plain(a[0], type, 3, dev), *positions = plain(a[2], kI32, 1, dev),
                 *freqs = plain(a[3], at::kDouble, 1, dev);
    int32_t layout;
    KDA_USUAL(q && positions && freqs && layout_of(a[4], layout) && PyFloat_CheckExact(a[5]) && PyBool_Check(a[6]));
    const int64_t T = q->size(0), d = q->size(2);
    KDA_USUAL(positions->size(0) == T && freqs->size(0) > 0 && 2 * freqs->size(0) <= d && small(T) &&
              small(q->size(1)) && small(d));
    const Tensor* k = nullptr;
    if (a[1] != Py_None) {
        k = plain(a[1], type, 3, dev);
        KDA_USUAL(k && k->size(0) == T && k->size(2) == d && small(k->size(1)));
    } else {
        KDA_USUAL(a[8] == Py_None);
    }
    Tensor qo, ko;
    KDA_USUAL(output_of(a[7], q->sizes(), type, dev, *q, qo) && (!k || output_of(a[8], k->sizes(), type, dev, *k, ko)));
    KDA_CALL(f_rotary(q->data_ptr(), q->stride(0), k ? k->data_ptr() : nullptr, k ? k->stride(0) : 0,
                      static_cast<const int32_t*>(positions->data_ptr()), static_cast<const double*>(freqs->data_ptr()),
                      T, (int32_t)q->size(1), k ? (int32_t)k->size(1) : 0, (int32_t)d, (int32_t)(2 * freqs->size(0)),
                      layout, (float)PyFloat_AS_DOUBLE(a[5]), a[6] == Py_True, code, qo.data_ptr(), qo.stride(0),
                      k ? ko.data_ptr() : nullptr, k ? ko.stride(0) : 0, stream));
    written(qo);
    if (k) written(ko);
    if (k) return pair(std::move(qo), std::move(ko));
    PyObject* x = THPVariable_Wrap(std::move(qo));
    PyObject* r = x ? PyTuple_Pack(2, x, Py_None) : nullptr;
    Py_XDECREF(x);
    return r;
    END_HANDLE_TH_ERRORS
}

// q, k, v, k_pages, v_pages, page_table, start, freqs, cu_seqlens, layout, amplitude, q_out
PyObject* rotary_append(PyObject*, PyObject* const* a, Py_ssize_t n_args) {
    HANDLE_TH_ERRORS
    KDA_USUAL(n_args == 12);
    const int dev = device_of(a[0]);
    KDA_USUAL(dev >= 0);
    const int code = code_of(a[0]);
    KDA_USUAL(code >= 0);
    const auto type = THPVariable_Unpack(a[0]).scalar_type();
    const Tensor *q = plain(a[0], type, 3, dev), *k = plain(a[1], type, 3, dev), *v = plain(a[2], type, 3, dev),
                 *kp = plain(a[3], type, 4, dev), *vp = plain(a[4], type, 4, dev), *table = plain(a[5], kI32, 2, dev),
                 *start = plain(a[6], kI32, 1, dev), *freqs = plain(a[7], at::kDouble, 1, dev);
    int32_t layout;
    KDA_USUAL(q && k && v && kp && vp && table && start && freqs && layout_of(a[9], layout) && PyFloat_CheckExact(a[10]));
    const int64_t T = q->size(0), d = q->size(2), N = table->size(0);
    KDA_USUAL(k->sizes() == v->sizes() && k->size(0) == T && k->size(2) == d && kp->sizes() == vp->sizes() &&
              kp->size(1) == k->size(1) && kp->size(3) == d && start->size(0) == N && freqs->size(0) > 0 &&
              2 * freqs->size(0) <= d);
    KDA_USUAL(small(T) && small(q->size(1)) && small(k->size(1)) && small(d) && small(kp->size(0)) &&
              small(kp->size(2)) && small(N) && small(table->size(1)));
    const Tensor* cu = nullptr;
    if (a[8] != Py_None) {
        cu = plain(a[8], kI32, 1, dev);
        KDA_USUAL(cu && cu->size(0) == N + 1);
    }
    Tensor qo;
    KDA_USUAL(output_of(a[11], q->sizes(), type, dev, *q, qo));
    KDA_CALL(f_place(q->data_ptr(), q->stride(0), k->data_ptr(), k->stride(0), v->data_ptr(), v->stride(0),
                     cu ? static_cast<const int32_t*>(cu->data_ptr()) : nullptr,
                     static_cast<const int32_t*>(start->data_ptr()), (int32_t)N, T,
                     static_cast<const double*>(freqs->data_ptr()), (int32_t)(2 * freqs->size(0)), layout,
                     (float)PyFloat_AS_DOUBLE(a[10]), qo.data_ptr(), qo.stride(0), kp->data_ptr(), vp->data_ptr(),
                     kp->stride(0), vp->stride(0), (int32_t)kp->size(0), (int32_t)kp->size(2),
                     static_cast<const int32_t*>(table->data_ptr()), table->stride(0), (int32_t)table->size(1),
                     (int32_t)q->size(1), (int32_t)k->size(1), (int32_t)d, code, stream));
    written(qo);
    written(*kp);
    written(*vp);
    return THPVariable_Wrap(std::move(qo));
    END_HANDLE_TH_ERRORS
}

// q, k_pages, v_pages, page_table, lengths, cu_seqlens, scale, window, sinks, max_length, out, lse, workspace
PyObject* paged_prefill(PyObject*, PyObject* const* a, Py_ssize_t n_args) {
    HANDLE_TH_ERRORS
    KDA_USUAL(n_args == 13);
    const int dev = device_of(a[0]);
    KDA_USUAL(dev >= 0);
    const int code = code_of(a[0]);
    KDA_USUAL(code >= 0);
    const auto type = THPVariable_Unpack(a[0]).scalar_type();
    const Tensor *q = plain(a[0], type, 3, dev), *kp = plain(a[1], type, 4, dev), *vp = plain(a[2], type, 4, dev),
                 *table = plain(a[3], kI32, 2, dev), *lengths = plain(a[4], kI32, 1, dev), *cu = plain(a[5], kI32, 1, dev);
    KDA_USUAL(q && kp && vp && table && lengths && cu);
    const int64_t T = q->size(0), Hq = q->size(1), d = q->size(2), N = table->size(0), P = table->size(1),
                  page = kp->size(2);
    KDA_USUAL(kp->sizes() == vp->sizes() && kp->size(3) == d && lengths->size(0) == N && cu->size(0) == N + 1);
    KDA_USUAL(small(T) && small(N) && small(Hq) && small(d) && small(P) && small(page) && small(kp->size(0)) &&
              small(kp->size(1)) && small(P * page));
    int32_t window, sinks, most = (int32_t)(P * page);
    KDA_USUAL(int_of(a[7], window) && int_of(a[8], sinks));
    if (a[9] != Py_None) {
        int32_t bound;
        KDA_USUAL(int_of(a[9], bound) && bound > 0);
        most = bound < most ? bound : most;
    }
    double scale = 0.;
    if (a[6] != Py_None) {
        KDA_USUAL(PyFloat_CheckExact(a[6]));
        scale = PyFloat_AS_DOUBLE(a[6]);
    } else {
        scale = d > 0 ? std::pow((double)d, -0.5) : 0.;
    }
    const size_t need =
        f_prefill_ws((int32_t)N, T, (int32_t)Hq, (int32_t)kp->size(1), (int32_t)d, code, most, window, sinks);
    Tensor keep, out, lse;
    void* ws;
    size_t ws_bytes;
    KDA_USUAL(workspace_of(a[12], need, dev, *q, keep, ws, ws_bytes));
    KDA_USUAL(output_of(a[10], q->sizes(), type, dev, *q, out));
    const bool want = a[11] != Py_None && a[11] != Py_False;
    if (want) KDA_USUAL(output_of(a[11] == Py_True ? Py_None : a[11], {T, Hq}, at::kFloat, dev, *q, lse));
    KDA_CALL(f_prefill(q->data_ptr(), q->stride(0), kp->data_ptr(), vp->data_ptr(), kp->stride(0), vp->stride(0),
                       (int32_t)kp->size(0), (int32_t)page, ints(*table), table->stride(0), (int32_t)P, ints(*lengths),
                       ints(*cu), (int32_t)N, T, (int32_t)Hq, (int32_t)kp->size(1), (int32_t)d, code, (float)scale,
                       window, sinks, most, out.data_ptr(), want ? static_cast<float*>(lse.data_ptr()) : nullptr, ws,
                       ws_bytes, stream));
    written(out);
    if (want) written(lse);
    return want ? pair(std::move(out), std::move(lse)) : THPVariable_Wrap(std::move(out));
    END_HANDLE_TH_ERRORS
}

// An optional plain contiguous [rows] argument; false for any other.
bool optional_of(PyObject* o, at::ScalarType type, int64_t rows, int dev, const void*& p) {
    p = nullptr;
    if (o == Py_None) return true;
    const Tensor* t = plain(o, type, 1, dev);
    if (!t || t->size(0) != rows) return false;
    p = t->data_ptr();
    return true;
}

// logits, tokens, top, entropy, workspace
PyObject* token_logprobs(PyObject*, PyObject* const* a, Py_ssize_t n_args) {
    HANDLE_TH_ERRORS
    KDA_USUAL(n_args == 5);
    const int dev = device_of(a[0]);
    KDA_USUAL(dev >= 0);
    const int code = code_of(a[0]);
    KDA_USUAL(code >= 0);
    const Tensor* x = plain(a[0], THPVariable_Unpack(a[0]).scalar_type(), 2, dev);
    int32_t top;
    KDA_USUAL(x && int_of(a[2], top) && top >= 0 && PyBool_Check(a[3]) && small(x->size(1)) && top <= x->size(1));
    const int64_t R = x->size(0), V = x->size(1);
    const bool want = a[3] == Py_True;
    const void* tokens;
    KDA_USUAL(optional_of(a[1], kI32, R, dev, tokens));
    Tensor keep;
    void* ws;
    size_t ws_bytes;
    KDA_USUAL(workspace_of(a[4], f_logprobs_ws(R, (int32_t)V, top), dev, *x, keep, ws, ws_bytes));
    const bool given = a[1] != Py_None;
    Tensor lp, lse = fresh({R}, at::kFloat, *x), ent, best, which;
    if (given) lp = fresh({R}, at::kFloat, *x);
    if (want) ent = fresh({R}, at::kFloat, *x);
    if (top) {
        best = fresh({R, top}, at::kFloat, *x);
        which = fresh({R, top}, kI32, *x);
    }
    auto floats = [](Tensor& t) { return t.defined() ? static_cast<float*>(t.data_ptr()) : nullptr; };
    KDA_CALL(f_logprobs(x->data_ptr(), x->stride(0), static_cast<const int32_t*>(tokens), R, (int32_t)V, top, code,
                        floats(lp), floats(lse), floats(ent), floats(best), top ? ints(which) : nullptr, ws, ws_bytes,
                        stream));
    PyObject* r = PyTuple_New(5);
    if (!r) return nullptr;
    Tensor* out[5] = {&lp, &lse, &ent, &best, &which};
    for (int i = 0; i < 5; ++i) {
        PyObject* o = Py_None;
        if (out[i]->defined()) o = THPVariable_Wrap(std::move(*out[i]));
        else Py_INCREF(o);
        if (!o) {
            Py_DECREF(r);
            return nullptr;
        }
        PyTuple_SET_ITEM(r, i, o);
    }
    return r;
    END_HANDLE_TH_ERRORS
}

// logits, tokens, lse, d_logprobs, d_lse, entropy, d_entropy, out
PyObject* token_logprobs_grad(PyObject*, PyObject* const* a, Py_ssize_t n_args) {
    HANDLE_TH_ERRORS
    KDA_USUAL(n_args == 8);
    const int dev = device_of(a[0]);
    KDA_USUAL(dev >= 0);
    const int code = code_of(a[0]);
    KDA_USUAL(code >= 0);
    const auto type = THPVariable_Unpack(a[0]).scalar_type();
    const Tensor* x = plain(a[0], type, 2, dev);
    KDA_USUAL(x && small(x->size(1)) && a[2] != Py_None);
    const int64_t R = x->size(0);
    KDA_USUAL((a[3] == Py_None || a[1] != Py_None) && (a[6] == Py_None || a[5] != Py_None));
    const void *tokens, *lse, *d_lp, *d_lse, *ent, *d_ent;
    KDA_USUAL(optional_of(a[1], kI32, R, dev, tokens) && optional_of(a[2], at::kFloat, R, dev, lse) &&
              optional_of(a[3], at::kFloat, R, dev, d_lp) && optional_of(a[4], at::kFloat, R, dev, d_lse) &&
              optional_of(a[5], at::kFloat, R, dev, ent) && optional_of(a[6], at::kFloat, R, dev, d_ent));
    Tensor out;
    KDA_USUAL(output_of(a[7], x->sizes(), type, dev, *x, out));
    auto floats = [](const void* p) { return static_cast<const float*>(p); };
    KDA_CALL(f_logprobs_grad(x->data_ptr(), x->stride(0), static_cast<const int32_t*>(tokens), floats(lse), floats(ent),
                             floats(d_lp), floats(d_lse), floats(d_ent), R, (int32_t)x->size(1), code, out.data_ptr(),
                             out.stride(0), stream));
    written(out);
    return THPVariable_Wrap(std::move(out));
    END_HANDLE_TH_ERRORS
}

// setup(raw_stream, check, {name: address})
template <typename F>
bool address(PyObject* d, const char* name, F& f) {
    PyObject* o = PyDict_GetItemString(d, name);  // borrowed
    void* p = o ? PyLong_AsVoidPtr(o) : nullptr;
    if (!p) {
        if (!PyErr_Occurred()) PyErr_Format(PyExc_ValueError, "no address of %s", name);
        return false;
    }
    f = reinterpret_cast<F>(p);
    return true;
}

PyObject* setup(PyObject*, PyObject* args) {
    PyObject *raw, *check, *d;
    if (!PyArg_ParseTuple(args, "OOO!", &raw, &check, &PyDict_Type, &d)) return nullptr;
    if (!address(d, "kda_cache_append", f_append) || !address(d, "kda_paged_decode", f_decode) ||
        !address(d, "kda_paged_decode_workspace", f_decode_ws) || !address(d, "kda_cache_fork", f_fork) ||
        !address(d, "kda_cache_free", f_free) || !address(d, "kda_cache_reserve", f_reserve) ||
        !address(d, "kda_cache_compact", f_compact) || !address(d, "kda_cache_workspace_size", f_cache_ws) ||
        !address(d, "kda_pages_copy", f_copy) || !address(d, "kda_beam_select", f_select) ||
        !address(d, "kda_beam_select_workspace", f_select_ws) || !address(d, "kda_beam_reorder", f_reorder) ||
        !address(d, "kda_rotary", f_rotary) || !address(d, "kda_rotary_append", f_place) ||
        !address(d, "kda_paged_prefill", f_prefill) ||
        !address(d, "kda_paged_prefill_workspace", f_prefill_ws) ||
        !address(d, "kda_token_logprobs", f_logprobs) ||
        !address(d, "kda_token_logprobs_workspace", f_logprobs_ws) ||
        !address(d, "kda_token_logprobs_grad", f_logprobs_grad))
        return nullptr;
    Py_INCREF(raw);
    Py_INCREF(check);
    Py_XSETREF(g_raw_stream, raw);
    Py_XSETREF(g_check, check);
    Py_RETURN_NONE;
}

#define KDA_FN(name) {#name, (PyCFunction)(void*)name, METH_FASTCALL, nullptr}
PyMethodDef methods[] = {KDA_FN(cache_append),  KDA_FN(paged_decode),  KDA_FN(cache_fork), KDA_FN(cache_free),
                         KDA_FN(cache_reserve), KDA_FN(cache_compact), KDA_FN(pages_copy), KDA_FN(beam_select),
                         KDA_FN(beam_reorder),  KDA_FN(rotary),        KDA_FN(rotary_append),
                         KDA_FN(paged_prefill), KDA_FN(token_logprobs), KDA_FN(token_logprobs_grad),
                         {"setup", setup, METH_VARARGS, nullptr},      {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_kda_marshal", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

#define KDA_TEXT_(x) #x
#define KDA_TEXT(x) KDA_TEXT_(x)

// The versions that the module was built for: it is used with these only.
PyMODINIT_FUNC PyInit__kda_marshal(void) {
    PyObject* m = PyModule_Create(&module);
    if (m && (PyModule_AddStringConstant(m, "torch_version", KDA_TORCH_VERSION) < 0 ||
              PyModule_AddStringConstant(m, "python_version",
                                         KDA_TEXT(PY_MAJOR_VERSION) "." KDA_TEXT(PY_MINOR_VERSION)) < 0)) {
        Py_DECREF(m);
        return nullptr;
    }
    return m;
}
