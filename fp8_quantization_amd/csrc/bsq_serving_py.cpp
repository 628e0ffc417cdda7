// bsq_serving_py.cpp -- the Python binding of libbsq_serving as a CPython
// extension (module _serving).  Argument marshalling only, like the package's
// ctypes binding; native because a decode step calls these operators for a
// few microseconds of GPU work each, and checking their eight to ten tensors
// attribute by attribute from Python took 18 to 30 us a call.
//
// Every function takes its arguments by position; serving.py gives them names
// and defaults.  A tensor of a wrong dtype, device or layout raises TypeError,
// one of a wrong size BsqError (the class handed to `init`), before anything
// runs.
#include <ATen/hip/impl/HIPStreamMasqueradingAsCUDA.h>
#include <c10/core/DeviceGuard.h>
#include <c10/core/StreamGuard.h>
#include <c10/hip/HIPFunctions.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>
#include <torch/torch.h>

#include <cstdarg>
#include <cstdio>
#include <string>

#include "bsq_serving.h"

namespace {

PyObject* g_bsq_error = nullptr;

struct Refused {
    int status;                      // 0: TypeError
    std::string what;
};
[[noreturn]] void refuse(int status, const char* fmt, ...) {
    char buf[512];
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(buf, sizeof(buf), fmt, ap);
    va_end(ap);
    throw Refused{status, buf};
}

void check(int status) {
    if (status != BSQ_OK) throw Refused{status, bsq_serving_last_error()};
}
int64_t size_of(int64_t n) {
    if (n < 0) throw Refused{BSQ_ERR_INVALID_ARG, bsq_serving_last_error()};
    return n;
}

// The arguments of a call, taken in order.
struct Args {
    PyObject* const* p;
    Py_ssize_t n, i = 0;
    PyObject* next() {
        if (i >= n) refuse(0, "too few arguments");
        return p[i++];
    }
    int64_t integer(const char* name) {
        const int64_t v = PyLong_AsLongLong(next());
        if (v == -1 && PyErr_Occurred()) {
            PyErr_Clear();
            refuse(0, "%s must be an integer", name);
        }
        return v;
    }
    double number(const char* name) {
        const double v = PyFloat_AsDouble(next());
        if (v == -1.0 && PyErr_Occurred()) {
            PyErr_Clear();
            refuse(0, "%s must be a number", name);
        }
        return v;
    }
    // null: None
    const at::Tensor* tensor(const char* name, bool optional = false) {
        return unpack(next(), name, optional);
    }
    const at::Tensor* unpack(PyObject* o, const char* name, bool optional = false) {
        if (optional && o == Py_None) return nullptr;
        if (!THPVariable_Check(o)) refuse(0, "%s must be a GPU tensor", name);
        const at::Tensor& t = THPVariable_Unpack(o);
        if (!t.is_cuda()) refuse(0, "%s must be a GPU tensor", name);
        if (device.has_value() && t.device() != *device)
            refuse(0, "%s is on %s, other tensors on %s", name, t.device().str().c_str(),
                   device->str().c_str());
        device = t.device();
        return &t;
    }
    std::optional<at::Device> device;
};

// The stream of a call (an object with cuda_stream, or None for the current one).  It is torch's
// current stream as long as this lives, so whatever the call allocates belongs to it: its memory
// has been used by earlier work of that stream alone, and goes to later work of it alone.  With
// memory of the caller's stream the kernels could overwrite what that stream is still reading.
// The tensors' device is the current one meanwhile: launched with another current, kernels on a
// device's default stream would run on that other one.
struct CallStream {
    void* raw;
    explicit CallStream(Args& a) {
        PyObject* o = a.next();
        if (c10::hip::current_device() != a.device->index()) device.reset_device(*a.device);
        const auto now = at::hip::getCurrentHIPStreamMasqueradingAsCUDA(a.device->index());
        raw = now.stream();
        if (o == Py_None) return;
        PyObject* attr = PyObject_GetAttrString(o, "cuda_stream");
        if (!attr) {
            PyErr_Clear();
            refuse(0, "stream must be a torch.cuda.Stream");
        }
        void* given = PyLong_AsVoidPtr(attr);
        Py_DECREF(attr);
        if (!given && PyErr_Occurred()) {
            PyErr_Clear();
            refuse(0, "stream must be a torch.cuda.Stream");
        }
        if (given == raw) return;
        raw = given;
        caller = now.unwrap();
        guard.reset_stream(at::hip::getStreamFromExternalMasqueradingAsCUDA(
            static_cast<hipStream_t>(given), a.device->index()).unwrap());
    }
    // An output for the caller; one that the call allocated itself (`own`) will be used by the
    // caller's stream too, so its memory must not go to this one's work before that is done.
    PyObject* give(const at::Tensor& t, const at::Tensor& own) const {
        if (caller && own.defined()) own.record_stream(*caller);
        return THPVariable_Wrap(t);
    }

private:
    std::optional<c10::Stream> caller;   // the caller's stream, where it is another
    c10::OptionalDeviceGuard device;
    c10::OptionalStreamGuard guard;
};

// Whether the dimensions after the first lie without gaps.
bool dense_rows(const at::Tensor& t) {
    int64_t want = 1;
    for (int64_t d = t.dim() - 1; d > 0; --d) {
        if (t.size(d) > 1 && t.stride(d) != want) return false;
        want *= t.size(d);
    }
    return true;
}
int64_t row_stride(const at::Tensor& t) {
    if (t.size(0) > 1) return t.stride(0);
    int64_t n = 1;
    for (int64_t d = 1; d < t.dim(); ++d) n *= t.size(d);
    return n;
}

const at::Tensor& vec(const at::Tensor* t, const char* name, at::ScalarType dtype, int64_t n,
                      bool exact) {
    const bool fits = t->scalar_type() == dtype ||
                      (dtype == at::kUInt32 && t->scalar_type() == at::kInt);
    if (!fits || !t->is_contiguous() || t->dim() != 1)
        refuse(0, "%s must be a contiguous 1-D GPU tensor of dtype %s", name,
               dtype == at::kUInt32 ? "uint32 or int32" : c10::toString(dtype));
    if (t->numel() < n || (exact && t->numel() != n))
        refuse(BSQ_ERR_INVALID_ARG, "%s has %lld entries; it must have %s%lld", name,
               (long long)t->numel(), exact ? "" : "at least ", (long long)n);
    return *t;
}

// A 2-D tensor of exactly rows x cols without gaps.
void* matrix(const at::Tensor* t, const char* name, at::ScalarType dtype, int64_t rows,
             int64_t cols) {
    if (t->scalar_type() != dtype || t->dim() != 2 || !t->is_contiguous())
        refuse(0, "%s must be a contiguous 2-D GPU tensor of dtype %s", name,
               c10::toString(dtype));
    if (t->size(0) < rows || t->size(1) != cols)
        refuse(BSQ_ERR_INVALID_ARG, "%s is [%lld, %lld]; it must be [%lld, %lld]", name,
               (long long)t->size(0), (long long)t->size(1), (long long)rows, (long long)cols);
    return t->data_ptr();
}

// Rows of BF16, dense within a row.
const at::Tensor& rows_of(const at::Tensor* t, const char* name, int64_t dims) {
    if (t->scalar_type() != at::kBFloat16 || t->dim() != dims || !dense_rows(*t))
        refuse(0, "%s must be a %lld-D bfloat16 GPU tensor, contiguous within a row", name,
               (long long)dims);
    return *t;
}

bsq_kv_cache cache_of(Args& a) {
    static const char* const names[4] = {"k_codes", "v_codes", "k_scales", "v_scales"};
    static const int64_t dims[4] = {5, 4, 2, 2};
    PyObject* o = a.next();
    if (!PyTuple_Check(o) || PyTuple_GET_SIZE(o) != 4) refuse(0, "cache must be a KvCache");
    const at::Tensor* t[4];
    for (int i = 0; i < 4; ++i) {
        t[i] = a.unpack(PyTuple_GET_ITEM(o, i), names[i]);
        if (t[i]->scalar_type() != at::kByte || t[i]->dim() != dims[i] || !dense_rows(*t[i]))
            refuse(0, "%s must be a %lld-D uint8 GPU tensor, contiguous within a page", names[i],
                   (long long)dims[i]);
    }
    const int64_t P = t[0]->size(0), H = t[0]->size(1), D = 16 * t[0]->size(2);
    bool fits = t[0]->size(3) == BSQ_KV_PAGE && t[0]->size(4) == 16 && t[1]->size(2) == D &&
                t[1]->size(3) == BSQ_KV_PAGE && D <= 0x7FFFFFFF && H <= 0x7FFFFFFF;
    for (int i = 1; i < 4; ++i) fits = fits && t[i]->size(0) == P && t[i]->size(1) == H;
    if (!fits) refuse(BSQ_ERR_INVALID_ARG, "the tensors' shapes are no cache's");
    if (P > 1 && (t[0]->stride(0) != t[1]->stride(0) || t[2]->stride(0) != t[3]->stride(0)))
        refuse(0, "k and v must have the same stride from a page to the next");
    bsq_kv_cache c;
    c.k_codes = t[0]->data_ptr();
    c.v_codes = t[1]->data_ptr();
    c.k_scales = static_cast<uint8_t*>(t[2]->data_ptr());
    c.v_scales = static_cast<uint8_t*>(t[3]->data_ptr());
    c.num_pages = P;
    c.page_stride = row_stride(*t[0]);
    c.scale_stride = row_stride(*t[2]);
    c.num_heads = (int32_t)H;
    c.head_dim = (int32_t)D;
    return c;
}

// block_table and kv_lens.
struct Table {
    int32_t* p;
    int32_t* lens;
    int64_t stride, pages, seqs;
};
int32_t* table_rows(const at::Tensor& t, const char* name, int64_t* stride) {
    if (t.scalar_type() != at::kInt || t.dim() != 2 || !dense_rows(t))
        refuse(0, "%s must be a 2-D row-major int32 GPU tensor", name);
    *stride = row_stride(t);
    return static_cast<int32_t*>(t.data_ptr());
}
Table table_of(Args& a) {
    Table r;
    const at::Tensor& t = *a.tensor("block_table");
    r.p = table_rows(t, "block_table", &r.stride);
    r.seqs = t.size(0);
    r.pages = t.size(1);
    r.lens = static_cast<int32_t*>(vec(a.tensor("kv_lens"), "kv_lens", at::kInt, r.seqs, true).data_ptr());
    return r;
}

at::Tensor empty(at::IntArrayRef shape, at::ScalarType dtype, const at::Device& device) {
    return at::empty(shape, at::TensorOptions().dtype(dtype).device(device));
}

// Workspace of a call: the caller's, or an allocation that the call's stream owns (a CallStream
// lives), given back at the call's end to later work of that stream.
struct Workspace {
    at::Tensor own;
    void* p = nullptr;
    int64_t bytes = 0;
    Workspace(Args& a, const at::Tensor* given, int64_t need) {
        if (given) {
            if (given->scalar_type() != at::kByte || !given->is_contiguous())
                refuse(0, "workspace must be a contiguous uint8 GPU tensor");
            p = given->data_ptr();
            bytes = given->numel();
        } else if (need > 0) {
            own = empty({need}, at::kByte, *a.device);
            p = own.data_ptr();
            bytes = need;
        }
    }
};

template <PyObject* (*F)(Args&)>
PyObject* entry(PyObject*, PyObject* const* args, Py_ssize_t n) {
    try {
        Args a{args, n};
        return F(a);
    } catch (const Refused& r) {
        if (r.status == 0 || !g_bsq_error) {
            PyErr_SetString(PyExc_TypeError, r.what.c_str());
        } else if (PyObject* e = PyObject_CallFunction(g_bsq_error, "is", r.status, r.what.c_str())) {
            PyErr_SetObject(g_bsq_error, e);
            Py_DECREF(e);
        }
    } catch (...) {                  // torch's own: its Python class (OutOfMemoryError)
        torch::translate_exception_to_python(std::current_exception());
    }
    return nullptr;
}

PyObject* none() { Py_RETURN_NONE; }

PyObject* init(Args& a) {
    Py_XDECREF(g_bsq_error);
    g_bsq_error = a.next();
    Py_INCREF(g_bsq_error);
    return none();
}

// cache, k, v, row_offsets, kv_lens <- block_table first: (block_table, kv_lens), max_new, stream
PyObject* append(Args& a) {
    const bsq_kv_cache c = cache_of(a);
    const at::Tensor& k = rows_of(a.tensor("k"), "k", 3);
    const at::Tensor& v = rows_of(a.tensor("v"), "v", 3);
    const at::Tensor* offsets = a.tensor("row_offsets");
    const Table t = table_of(a);
    const int64_t max_new = a.integer("max_new");
    const CallStream stream(a);
    vec(offsets, "row_offsets", at::kUInt32, t.seqs + 1, true);
    for (const at::Tensor* x : {&k, &v})
        if (x->size(1) != c.num_heads || x->size(2) != c.head_dim || x->size(0) != k.size(0))
            refuse(BSQ_ERR_INVALID_ARG, "k and v must be [rows, %d, %d], as many rows each",
                   c.num_heads, c.head_dim);
    check(kv_cache_append(&c, k.data_ptr(), row_stride(k), v.data_ptr(), row_stride(v),
                          static_cast<uint32_t*>(offsets->data_ptr()), t.lens, t.p, t.stride, t.pages,
                          t.seqs, k.size(0), max_new, stream.raw));
    return none();
}

// q, cache, row_offsets, block_table, kv_lens, max_q, max_kv, scale, window, out, lse, want_lse,
// workspace, stream -> (out, lse or None)
PyObject* attention(Args& a) {
    const at::Tensor& q = rows_of(a.tensor("q"), "q", 3);
    const bsq_kv_cache c = cache_of(a);
    const at::Tensor* offsets = a.tensor("row_offsets");
    const Table t = table_of(a);
    const int64_t max_q = a.integer("max_q"), max_kv = a.integer("max_kv");
    const double scale = a.number("scale");
    const int64_t window = a.integer("window");
    const at::Tensor* out = a.tensor("out", true);
    const at::Tensor* lse = a.tensor("lse", true);
    const bool want_lse = a.integer("return_lse") != 0;
    const at::Tensor* given = a.tensor("workspace", true);
    const CallStream stream(a);
    const int64_t R = q.size(0), Hq = q.size(1), D = q.size(2);
    if (D != c.head_dim)
        refuse(BSQ_ERR_INVALID_ARG, "q is %lld wide, the cache's heads %d", (long long)D, c.head_dim);
    vec(offsets, "row_offsets", at::kUInt32, t.seqs + 1, true);
    at::Tensor new_out, new_lse;
    if (out) {
        rows_of(out, "out", 3);
        if (out->size(0) < R || out->size(1) != Hq || out->size(2) != D)
            refuse(BSQ_ERR_INVALID_ARG, "out must be [%lld, %lld, %lld]", (long long)R, (long long)Hq,
                   (long long)D);
    } else {
        new_out = empty({R, Hq, D}, at::kBFloat16, *a.device);
        out = &new_out;
    }
    if (lse) {
        matrix(lse, "lse", at::kFloat, R, Hq);
    } else if (want_lse) {
        new_lse = empty({R, Hq}, at::kFloat, *a.device);
        lse = &new_lse;
    }
    const int64_t need = size_of(kv_cache_attention_workspace(c.num_heads, D, Hq, t.seqs, R, max_q,
                                                              max_kv, window));
    const Workspace ws(a, need ? given : nullptr, need);
    check(kv_cache_attention(&c, q.data_ptr(), row_stride(q), Hq,
                             static_cast<uint32_t*>(offsets->data_ptr()), t.lens, t.p, t.stride,
                             t.pages, t.seqs, R, max_q, max_kv, (float)scale, window,
                             out->data_ptr(), row_stride(*out),
                             lse ? static_cast<float*>(lse->data_ptr()) : nullptr, ws.p, ws.bytes,
                             stream.raw));
    PyObject* o = stream.give(*out, new_out);
    PyObject* l = lse ? stream.give(*lse, new_lse) : none();
    PyObject* r = o && l ? PyTuple_Pack(2, o, l) : nullptr;
    Py_XDECREF(o);
    Py_XDECREF(l);
    return r;
}

// cache, src, dst, stream
PyObject* pages_copy(Args& a) {
    const bsq_kv_cache c = cache_of(a);
    const at::Tensor* src = a.tensor("src");
    const int64_t n = src->numel();
    const int32_t* s = vec(src, "src", at::kInt, n, true).data_ptr<int32_t>();
    const int32_t* d = vec(a.tensor("dst"), "dst", at::kInt, n, true).data_ptr<int32_t>();
    const CallStream stream(a);
    check(kv_pages_copy(&c, s, d, n, stream.raw));
    return none();
}

const at::Tensor* status_of(const at::Tensor* given, int64_t n, at::Tensor& own, Args& a) {
    if (given) {
        vec(given, "status", at::kInt, n, true);
        return given;
    }
    own = empty({n}, at::kInt, *a.device);
    return &own;
}

// block_table, kv_lens, refcounts, slots, add_tokens, status, stream -> status
PyObject* pages_reserve(Args& a) {
    const Table t = table_of(a);
    const at::Tensor& refs = vec(a.tensor("refcounts"), "refcounts", at::kInt, 0, false);
    const at::Tensor* slots = a.tensor("slots");
    const int64_t n = slots->numel();
    vec(slots, "slots", at::kInt, n, true);
    const at::Tensor& add = vec(a.tensor("add_tokens"), "add_tokens", at::kInt, n, true);
    const at::Tensor* given = a.tensor("status", true);
    const CallStream stream(a);
    at::Tensor own;
    const at::Tensor* status = status_of(given, n, own, a);
    check(kv_pages_reserve(t.p, t.stride, t.pages, t.seqs, t.lens, refs.data_ptr<int32_t>(),
                           refs.numel(), slots->data_ptr<int32_t>(), add.data_ptr<int32_t>(), n,
                           status->data_ptr<int32_t>(), stream.raw));
    return stream.give(*status, own);
}

// cache, block_table, kv_lens, refcounts, parents, children, status, stream -> status
PyObject* pages_fork(Args& a) {
    const bsq_kv_cache c = cache_of(a);
    const Table t = table_of(a);
    const at::Tensor& refs = vec(a.tensor("refcounts"), "refcounts", at::kInt, c.num_pages, true);
    const at::Tensor* parents = a.tensor("parents");
    const int64_t n = parents->numel();
    vec(parents, "parents", at::kInt, n, true);
    const at::Tensor& children = vec(a.tensor("children"), "children", at::kInt, n, true);
    const at::Tensor* given = a.tensor("status", true);
    const CallStream stream(a);
    at::Tensor own;
    const at::Tensor* status = status_of(given, n, own, a);
    check(kv_pages_fork(&c, t.p, t.stride, t.pages, t.seqs, t.lens, refs.data_ptr<int32_t>(),
                        parents->data_ptr<int32_t>(), children.data_ptr<int32_t>(), n,
                        status->data_ptr<int32_t>(), stream.raw));
    return stream.give(*status, own);
}

// block_table, kv_lens, refcounts, slots, stream
PyObject* pages_free(Args& a) {
    const Table t = table_of(a);
    const at::Tensor& refs = vec(a.tensor("refcounts"), "refcounts", at::kInt, 0, false);
    const at::Tensor& slots = vec(a.tensor("slots"), "slots", at::kInt, 0, false);
    const CallStream stream(a);
    check(kv_pages_free(t.p, t.stride, t.pages, t.seqs, t.lens, refs.data_ptr<int32_t>(), refs.numel(),
                        slots.data_ptr<int32_t>(), slots.numel(), stream.raw));
    return none();
}

// cache, block_table, kv_lens, refcounts, table_out, refcounts_out, num_live, workspace, stream
// -> (table, refcounts, num_live)
PyObject* pages_compact(Args& a) {
    const bsq_kv_cache c = cache_of(a);
    const Table t = table_of(a);
    const at::Tensor& refs = vec(a.tensor("refcounts"), "refcounts", at::kInt, c.num_pages, true);
    const at::Tensor* table = a.tensor("table_out", true);
    const at::Tensor* counts = a.tensor("refcounts_out", true);
    const at::Tensor* live = a.tensor("num_live", true);
    const at::Tensor* given = a.tensor("workspace", true);
    const CallStream stream(a);
    at::Tensor new_table, new_counts, new_live;
    if (!table) {
        new_table = empty({t.seqs, t.pages}, at::kInt, *a.device);
        table = &new_table;
    }
    int64_t stride;
    int32_t* rows = table_rows(*table, "table_out", &stride);
    if (table->size(0) != t.seqs || table->size(1) != t.pages)
        refuse(BSQ_ERR_INVALID_ARG, "table_out must be [%lld, %lld], as block_table",
               (long long)t.seqs, (long long)t.pages);
    if (!counts) {
        new_counts = empty({c.num_pages}, at::kInt, *a.device);
        counts = &new_counts;
    }
    vec(counts, "refcounts_out", at::kInt, c.num_pages, true);
    if (!live) {
        new_live = empty({1}, at::kInt, *a.device);
        live = &new_live;
    }
    vec(live, "num_live", at::kInt, 1, false);
    const Workspace ws(a, given, size_of(kv_pages_compact_workspace(c.num_pages)));
    check(kv_pages_compact(&c, t.p, t.stride, t.pages, t.seqs, t.lens, refs.data_ptr<int32_t>(), rows,
                           stride, counts->data_ptr<int32_t>(), live->data_ptr<int32_t>(), ws.p,
                           ws.bytes, stream.raw));
    PyObject* o[3] = {stream.give(*table, new_table), stream.give(*counts, new_counts),
                      stream.give(*live, new_live)};
    PyObject* r = o[0] && o[1] && o[2] ? PyTuple_Pack(3, o[0], o[1], o[2]) : nullptr;
    for (PyObject* x : o) Py_XDECREF(x);
    return r;
}

// x, format, w13_codes, w13_scales, w2_codes, w2_scales, num_experts, topk, router_logits,
// topk_ids, topk_weights, renormalize, out, workspace, stream -> (out, ids, weights)
PyObject* moe(Args& a) {
    const at::Tensor& x = rows_of(a.tensor("x"), "x", 2);
    const int fmt = (int)a.integer("format");
    if (fmt != BSQ_MXFP4 && fmt != BSQ_MXFP8)
        refuse(BSQ_ERR_UNSUPPORTED, "format %d is not provided (MXFP4 or MXFP8 weights)", fmt);
    const at::Tensor* w13 = a.tensor("w13_codes");
    const at::Tensor* w13s = a.tensor("w13_scales");
    const at::Tensor* w2 = a.tensor("w2_codes");
    const at::Tensor* w2s = a.tensor("w2_scales");
    const int64_t E = a.integer("num_experts"), k = a.integer("topk");
    const at::Tensor* logits = a.tensor("router_logits", true);
    const at::Tensor* ids = a.tensor("topk_ids", true);
    const at::Tensor* weights = a.tensor("topk_weights", true);
    const int64_t renormalize = a.integer("renormalize");
    const at::Tensor* out = a.tensor("out", true);
    const at::Tensor* given = a.tensor("workspace", true);
    const CallStream stream(a);
    const int64_t T = x.size(0), H = x.size(1);
    if (w13->dim() != 2 || E < 1 || w13->size(0) % (2 * E) != 0)
        refuse(BSQ_ERR_INVALID_ARG,
               "w13_codes must hold num_experts * 2 * inter rows, num_experts >= 1");
    const int64_t I = w13->size(0) / (2 * E);
    if (H % 128 != 0 || I % 128 != 0)
        refuse(BSQ_ERR_INVALID_ARG, "hidden=%lld and inter=%lld must be multiples of 128",
               (long long)H, (long long)I);
    if (k < 1) refuse(BSQ_ERR_INVALID_ARG, "topk=%lld must be at least 1", (long long)k);
    auto width = [&](int64_t K) { return fmt == BSQ_MXFP8 ? K : K / 2; };
    auto records = [](int64_t K) { return (K + 511) / 512 * 256; };
    matrix(w13, "w13_codes", at::kByte, 2 * E * I, width(H));
    matrix(w13s, "w13_scales", at::kByte, 2 * E * I / 16, records(H));
    matrix(w2, "w2_codes", at::kByte, E * H, width(I));
    matrix(w2s, "w2_scales", at::kByte, E * H / 16, records(I));
    at::Tensor new_out, new_ids, new_weights;
    if (out) {
        rows_of(out, "out", 2);
        if (out->size(0) < T || out->size(1) != H)
            refuse(BSQ_ERR_INVALID_ARG, "out must be [%lld, %lld]", (long long)T, (long long)H);
    } else {
        new_out = empty({T, H}, at::kBFloat16, *a.device);
        out = &new_out;
    }
    if (logits) {
        matrix(logits, "router_logits", at::kFloat, T, E);
        if (!ids) {
            new_ids = empty({T, k}, at::kInt, *a.device);
            ids = &new_ids;
        }
        if (!weights) {
            new_weights = empty({T, k}, at::kFloat, *a.device);
            weights = &new_weights;
        }
    } else if (!ids || !weights) {
        refuse(BSQ_ERR_INVALID_ARG, "give router_logits, or topk_ids and topk_weights");
    }
    matrix(ids, "topk_ids", at::kInt, T, k);
    matrix(weights, "topk_weights", at::kFloat, T, k);
    // sizes that the workspace refuses are refused by the call, with its message
    const int64_t need = moe_few_tokens_workspace(T, H, I, k);
    const Workspace ws(a, given, need < 0 ? 0 : need);
    check(moe_few_tokens(fmt, x.data_ptr(), row_stride(x), T, H, I, E, k, w13->data_ptr(),
                         w13s->data_ptr(), w2->data_ptr(), w2s->data_ptr(),
                         logits ? logits->data_ptr<float>() : nullptr, (int)renormalize,
                         ids->data_ptr<int32_t>(), weights->data_ptr<float>(), out->data_ptr(),
                         row_stride(*out), ws.p, ws.bytes, stream.raw));
    PyObject* o[3] = {stream.give(*out, new_out), stream.give(*ids, new_ids),
                      stream.give(*weights, new_weights)};
    PyObject* r = o[0] && o[1] && o[2] ? PyTuple_Pack(3, o[0], o[1], o[2]) : nullptr;
    for (PyObject* p : o) Py_XDECREF(p);
    return r;
}

#define ENTRY(name, fn) {name, (PyCFunction)(void (*)(void))entry<fn>, METH_FASTCALL, nullptr}
PyMethodDef g_methods[] = {ENTRY("init", init),
                           ENTRY("append", append),
                           ENTRY("attention", attention),
                           ENTRY("pages_copy", pages_copy),
                           ENTRY("pages_reserve", pages_reserve),
                           ENTRY("pages_fork", pages_fork),
                           ENTRY("pages_free", pages_free),
                           ENTRY("pages_compact", pages_compact),
                           ENTRY("moe", moe),
                           {nullptr, nullptr, 0, nullptr}};
PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_serving", nullptr, -1, g_methods,
                        nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__serving() { return PyModule_Create(&g_module); }
