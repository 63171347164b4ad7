// serve_ext.cpp - argument marshalling of the serving operators for Python
// (serving.py): checks that tensors live on the current CUDA device with the
// documented type and layout, passes their addresses and the stream to the C
// entry points of include/tfserve.h, and returns their status.  Nothing is
// computed here; it is compiled because a decode step's calls are shorter than
// a dozen attribute look-ups of a tensor from Python (13-25 us a call, of which
// the library's own host work is 3-5).
#include <Python.h>

#include <ATen/ATen.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include "../../include/tfserve.h"

namespace {

struct Raised {};  // a Python error is set

[[noreturn]] void raise(PyObject *type, const char *name, const char *what) {
    PyErr_Format(type, "%s %s", name, what);
    throw Raised{};
}

enum Kind { kBf16, kI32, kU8, kF32, kStatus, kOut, kLogits };

bool is_kind(at::ScalarType t, Kind k) {
    switch (k) {
        case kBf16: return t == at::kBFloat16 || t == at::kShort || t == at::kUInt16;
        case kI32: return t == at::kInt;
        case kU8: return t == at::kByte;
        case kF32: return t == at::kFloat;
        case kStatus: return t == at::kInt || t == at::kUInt32;
        case kOut: return t == at::kFloat || t == at::kBFloat16;
        case kLogits: return t == at::kFloat || t == at::kBFloat16 || t == at::kShort || t == at::kUInt16;
    }
    return false;
}

// A tensor argument: on the current device, of a documented type and, unless
// `strided`, contiguous.
struct Arg {
    const at::Tensor *t;
    void *p;
    Arg(PyObject *o, const char *name, Kind kind, int &device, bool strided = false) {
        if (!THPVariable_Check(o)) raise(PyExc_TypeError, name, "must be a torch.Tensor");
        t = &THPVariable_Unpack(o);
        if (!t->is_cuda()) raise(PyExc_ValueError, name, "must be on a CUDA device");
        if (device < 0) device = c10::cuda::current_device();  // (there is one: a tensor lives on it)
        if (t->get_device() != device) raise(PyExc_ValueError, name, "must be on the current CUDA device");
        if (!is_kind(t->scalar_type(), kind)) raise(PyExc_TypeError, name, "has a dtype the call does not take");
        if (!strided && !t->is_contiguous()) raise(PyExc_ValueError, name, "must be contiguous");
        p = t->numel() ? t->data_ptr() : nullptr;
    }
    int64_t n() const { return t->numel(); }
    int64_t dim(int i) const { return t->size(i); }
    bool shape(std::initializer_list<int64_t> s) const {
        return t->dim() == (int64_t)s.size() && std::equal(s.begin(), s.end(), t->sizes().begin());
    }
};

int32_t len32(int64_t n);
void must(bool ok, const char *what);

// Entries of a segment table.
int32_t entries(const Arg &a, const char *what) {
    must(a.n() % 5 == 0, what);
    return len32(a.n() / 5);
}

void must(bool ok, const char *what) {
    if (ok) return;
    PyErr_SetString(PyExc_ValueError, what);
    throw Raised{};
}

// A host table: None, or int32 numbers in a C-contiguous buffer, as many as the
// device table it copies (anything else numpy can read is converted first).
struct Table {
    Py_buffer view{};
    PyObject *own = nullptr;
    const int32_t *p = nullptr;
    Table(PyObject *o, const char *name, int64_t n) {
        if (o == Py_None) return;
        if (!take(o)) {
            PyErr_Clear();
            PyObject *np = PyImport_ImportModule("numpy");
            if (!np) throw Raised{};
            own = PyObject_CallMethod(np, "ascontiguousarray", "Os", o, "int32");
            Py_DECREF(np);
            if (!own) throw Raised{};
            if (!take(own)) {
                Py_CLEAR(own);
                raise(PyExc_TypeError, name, "is not a table of int32 numbers");
            }
        }
        if (view.len != n * 4) {
            drop();
            raise(PyExc_ValueError, name, "and the device table it copies differ in length");
        }
        p = static_cast<const int32_t *>(view.buf);
    }
    ~Table() { drop(); }
    Table(const Table &) = delete;
    Table &operator=(const Table &) = delete;

  private:
    bool take(PyObject *o) {
        if (PyObject_GetBuffer(o, &view, PyBUF_C_CONTIGUOUS | PyBUF_FORMAT) != 0) {
            view.obj = nullptr;
            return false;
        }
        if (view.itemsize == 4 && view.format && view.format[0] == 'i' && !view.format[1]) return true;
        PyBuffer_Release(&view);
        view.obj = nullptr;
        return false;
    }
    void drop() {
        if (view.obj) PyBuffer_Release(&view);
        view.obj = nullptr;
        Py_CLEAR(own);
    }
};

const tf_q8_cache *cache_of(PyObject *address) {
    const tf_q8_cache *c = static_cast<const tf_q8_cache *>(PyLong_AsVoidPtr(address));
    if (!c) {
        if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, "the cache has no address");
        throw Raised{};
    }
    return c;
}

tf_stream_t stream_of(PyObject *o, int device) {
    if (o == Py_None) return reinterpret_cast<tf_stream_t>(c10::cuda::getCurrentCUDAStream(device).stream());
    void *p = PyLong_AsVoidPtr(o);
    if (PyErr_Occurred()) throw Raised{};
    return static_cast<tf_stream_t>(p);
}

int32_t i32(PyObject *o) {
    const long v = PyLong_AsLong(o);
    if (v == -1 && PyErr_Occurred()) throw Raised{};
    if (v > INT32_MAX || v < INT32_MIN) {
        PyErr_SetString(PyExc_OverflowError, "an integer argument is past 32 bits");
        throw Raised{};
    }
    return (int32_t)v;
}
int32_t len32(int64_t n) {
    if (n > INT32_MAX) {
        PyErr_SetString(PyExc_ValueError, "a tensor has more elements than the call takes");
        throw Raised{};
    }
    return (int32_t)n;
}
float f32(PyObject *o) {
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred()) throw Raised{};
    return (float)v;
}
int out_type(const Arg &a) { return a.t->scalar_type() == at::kBFloat16 ? TF_OUT_BF16 : TF_OUT_F32; }

// Runs `f`, turning what it throws into a Python error; its status otherwise.
template <typename F>
PyObject *guarded(Py_ssize_t got, Py_ssize_t want, F &&f) {
    if (got != want) {
        PyErr_SetString(PyExc_TypeError, "wrong number of arguments");
        return nullptr;
    }
    try {
        return PyLong_FromLong((long)f());
    } catch (const Raised &) {
    } catch (const std::exception &e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
    }
    return nullptr;
}

using Args = PyObject *const *;

// (k_rows, v_rows, cache, page_table, segs, status, segs_host, page_table_host, stream)
PyObject *kv_append(PyObject *, Args a, Py_ssize_t n) {
    return guarded(n, 9, [&]() {
        int dev = -1;  // the current device, once a tensor has been seen
        const tf_q8_cache *c = cache_of(a[2]);
        const Arg k(a[0], "k_rows", kBf16, dev), v(a[1], "v_rows", kBf16, dev);
        must(k.t->dim() == 3 && k.shape({k.dim(0), c->n_kv_heads, c->head_dim}) && v.t->sizes() == k.t->sizes(),
             "rows / cache shapes disagree");
        const Arg pt(a[3], "page_table", kI32, dev), sg(a[4], "segs", kI32, dev), st(a[5], "status", kStatus, dev);
        const Table sh(a[6], "segs_host", sg.n()), ph(a[7], "page_table_host", pt.n());
        return tf_kv_append_q8(k.p, v.p, len32(k.dim(0)), c, (const int32_t *)pt.p, len32(pt.n()),
                               (const tf_seg *)sg.p, entries(sg, "segs must hold five numbers an entry"), (const tf_seg *)sh.p, ph.p, (uint32_t *)st.p,
                               stream_of(a[8], dev));
    });
}

// (cache, page_table, segs, k_pool, v_pool, dst_page_table, status, segs_host, page_table_host, dst_host, stream)
PyObject *kv_read(PyObject *, Args a, Py_ssize_t n) {
    return guarded(n, 11, [&]() {
        int dev = -1;  // the current device, once a tensor has been seen
        const tf_q8_cache *c = cache_of(a[0]);
        const Arg k(a[3], "k_pool", kBf16, dev), v(a[4], "v_pool", kBf16, dev);
        must(k.t->dim() == 4 && k.shape({k.dim(0), c->n_kv_heads, c->page_size, c->head_dim}) &&
                 v.t->sizes() == k.t->sizes(),
             "pool / cache shapes disagree");
        const Arg pt(a[1], "page_table", kI32, dev), sg(a[2], "segs", kI32, dev), dt(a[5], "dst_page_table", kI32, dev),
            st(a[6], "status", kStatus, dev);
        must(dt.n() == pt.n(), "page_table and dst_page_table differ in length");
        const Table sh(a[7], "segs_host", sg.n()), ph(a[8], "page_table_host", pt.n()),
            dh(a[9], "dst_page_table_host", dt.n());
        return tf_kv_read_q8(c, (const int32_t *)pt.p, len32(pt.n()), (const tf_seg *)sg.p, entries(sg, "segs must hold five numbers an entry"),
                             (const tf_seg *)sh.p, ph.p, k.p, v.p, len32(k.dim(0)), (const int32_t *)dt.p, dh.p,
                             (uint32_t *)st.p, stream_of(a[10], dev));
    });
}

// (q, cache, page_table, segs, scale, full, split_keys, n_splits_max, workspace, out, flags, status, segs_host,
//  page_table_host, stream)
PyObject *attn_q8(PyObject *, Args a, Py_ssize_t n) {
    return guarded(n, 15, [&]() {
        int dev = -1;  // the current device, once a tensor has been seen
        const tf_q8_cache *c = cache_of(a[1]);
        const Arg q(a[0], "q", kBf16, dev), out(a[9], "out", kOut, dev), fl(a[10], "flags", kU8, dev);
        must(q.t->dim() == 3 && q.dim(2) == c->head_dim && out.t->sizes() == q.t->sizes() &&
                 fl.shape({q.dim(0), q.dim(1)}),
             "q / cache / out / flags shapes disagree");
        const Arg pt(a[2], "page_table", kI32, dev), sg(a[3], "segs", kI32, dev), ws(a[8], "workspace", kU8, dev),
            st(a[11], "status", kStatus, dev);
        const Table sh(a[12], "segs_host", sg.n()), ph(a[13], "page_table_host", pt.n());
        const int full = PyObject_IsTrue(a[5]);
        if (full < 0) throw Raised{};
        return tf_paged_attn_q8(q.p, len32(q.dim(0)), len32(q.dim(1)), c, (const int32_t *)pt.p, len32(pt.n()),
                                (const tf_seg *)sg.p, entries(sg, "segs must hold five numbers an entry"), (const tf_seg *)sh.p, ph.p, f32(a[4]), full,
                                i32(a[6]), i32(a[7]), ws.p, (size_t)ws.n(), out.p, out_type(out), (uint8_t *)fl.p,
                                (uint32_t *)st.p, stream_of(a[14], dev));
    });
}

// (q, k_pool, v_pool, page_table, prefixes, segs, scale, split_keys, n_prefix_splits, n_splits_max, workspace, out,
//  flags, status, prefixes_host, segs_host, page_table_host, stream)
PyObject *attn_shared(PyObject *, Args a, Py_ssize_t n) {
    return guarded(n, 18, [&]() {
        int dev = -1;  // the current device, once a tensor has been seen
        const Arg q(a[0], "q", kBf16, dev), k(a[1], "k_pool", kBf16, dev), v(a[2], "v_pool", kBf16, dev),
            out(a[11], "out", kOut, dev), fl(a[12], "flags", kU8, dev);
        must(q.t->dim() == 3 && k.t->dim() == 4 && k.dim(3) == q.dim(2) && v.t->sizes() == k.t->sizes() &&
                 out.t->sizes() == q.t->sizes() && fl.shape({q.dim(0), q.dim(1)}),
             "q / pool / out / flags shapes disagree");
        const Arg pt(a[3], "page_table", kI32, dev), pre(a[4], "prefixes", kI32, dev), sg(a[5], "segs", kI32, dev),
            ws(a[10], "workspace", kU8, dev), st(a[13], "status", kStatus, dev);
        const Table xh(a[14], "prefixes_host", pre.n()), sh(a[15], "segs_host", sg.n()),
            ph(a[16], "page_table_host", pt.n());
        return tf_paged_attn_shared(q.p, len32(q.dim(0)), len32(q.dim(1)), k.p, v.p, len32(k.dim(0)), len32(k.dim(2)),
                                    len32(k.dim(1)), len32(k.dim(3)), (const int32_t *)pt.p, len32(pt.n()),
                                    (const tf_seg *)pre.p, entries(pre, "prefixes must hold five numbers an entry"), (const tf_seg *)xh.p,
                                    (const tf_seg *)sg.p, entries(sg, "segs must hold five numbers an entry"), (const tf_seg *)sh.p, ph.p, f32(a[6]),
                                    i32(a[7]), i32(a[8]), i32(a[9]), ws.p, (size_t)ws.n(), out.p, out_type(out),
                                    (uint8_t *)fl.p, (uint32_t *)st.p, stream_of(a[17], dev));
    });
}

// (logits, tokens, scale, n_cols, token_logprobs, entropy, lse, top_ids, top_logprobs, flags, status, stream)
PyObject *logprob(PyObject *, Args a, Py_ssize_t n) {
    return guarded(n, 12, [&]() {
        int dev = -1;  // the current device, once a tensor has been seen
        const Arg x(a[0], "logits", kLogits, dev, true);
        must(x.t->dim() == 2 && (x.dim(1) <= 1 || x.t->stride(1) == 1), "logits must be 2-D with unit column stride");
        const int64_t rows = x.dim(0), cols = x.dim(1), ld = rows > 1 ? x.t->stride(0) : cols;
        const int32_t nc = a[3] == Py_None ? len32(cols) : i32(a[3]);
        must(nc <= cols, "n_cols is past the logits' columns");
        const Arg tok(a[1], "tokens", kI32, dev), tl(a[4], "token_logprobs", kF32, dev);
        must(tok.t->dim() == 2 && tok.dim(0) == rows && tl.t->sizes() == tok.t->sizes(),
             "tokens and token_logprobs must be [rows][n_tokens]");
        const Arg fl(a[9], "flags", kU8, dev), st(a[10], "status", kStatus, dev);
        float *ent = nullptr, *lse = nullptr, *tops = nullptr;
        int32_t *ids = nullptr, k = 0;
        const char *per_row = "entropy, lse and flags must have a value a row";
        must(fl.n() == rows, per_row);
        if (a[5] != Py_None) {
            const Arg e(a[5], "entropy", kF32, dev);
            must(e.n() == rows, per_row);
            ent = (float *)e.p;
        }
        if (a[6] != Py_None) {
            const Arg l(a[6], "lse", kF32, dev);
            must(l.n() == rows, per_row);
            lse = (float *)l.p;
        }
        const char *top = "top_ids and top_logprobs must be [rows][top_k], both or neither";
        must((a[7] == Py_None) == (a[8] == Py_None), top);
        if (a[7] != Py_None) {
            const Arg i(a[7], "top_ids", kI32, dev), t(a[8], "top_logprobs", kF32, dev);
            must(i.t->dim() == 2 && i.dim(0) == rows && t.t->sizes() == i.t->sizes(), top);
            k = len32(i.dim(1));
            ids = (int32_t *)i.p;
            tops = (float *)t.p;
        }
        return tf_logprob_rows(x.p, x.t->scalar_type() == at::kFloat ? TF_OUT_F32 : TF_OUT_BF16, len32(rows), nc, ld,
                               f32(a[2]), (const int32_t *)tok.p, len32(tok.dim(1)), (float *)tl.p, ent, lse, k, ids,
                               tops, (uint8_t *)fl.p, (uint32_t *)st.p, stream_of(a[11], dev));
    });
}

#define FAST(f) reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)(void)>(f)), METH_FASTCALL
PyMethodDef methods[] = {{"kv_append_q8", FAST(kv_append), nullptr},   {"kv_read_q8", FAST(kv_read), nullptr},
                         {"paged_attn_q8", FAST(attn_q8), nullptr},    {"paged_attn_shared", FAST(attn_shared), nullptr},
                         {"logprob_rows", FAST(logprob), nullptr},     {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_serve", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__serve() { return PyModule_Create(&module); }
