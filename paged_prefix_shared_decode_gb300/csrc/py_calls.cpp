// Python module _calls: the argument checks and the calls of the small, often
// repeated entry points, without an interpreted line per argument.  (With the
// checks in Python and the call through ctypes a sparse attention over ten
// tensors took 9.7 us of host time, here 2.8; a beam selection with its
// reorder 14.6, here 6.6.)  Every function checks its tensors' type, shape,
// device and layout, raises ValueError where one does not fit, and KvpError
// where the library refuses; None is a null pointer and an int an address that
// is not checked.  Signatures and documentation stand in the package, which
// binds the library's functions and calls these with positional arguments.
#include <torch/csrc/autograd/python_variable.h>

#include <cstring>
#include <initializer_list>
#include <numeric>
#include <string>
#include <vector>

#include "../../include/kvp.h"

namespace {

struct Raised {};                    // a Python error is set

[[noreturn]] void value_error(const std::string &what) {
    PyErr_SetString(PyExc_ValueError, what.c_str());
    throw Raised{};
}

// What the package binds: its error, torch's device and stream, the library.
PyObject *g_error = nullptr, *g_device = nullptr, *g_stream = nullptr;
struct Lib {                         // (in the order of the module's `functions`)
    decltype(&::seq_append_rope) append_rope;
    decltype(&::seq_reorder) reorder;
    decltype(&::kvp_pool_shape) pool_shape;
    decltype(&::kvp_pool_head_dim) pool_head_dim;
    decltype(&::kvp_page_bounds) bounds;
    decltype(&::kvp_page_scores) scores;
    decltype(&::kvp_page_select) select;
    decltype(&::paged_sparse_attention) sparse;
    decltype(&::kvp_beam_select) beam;
    decltype(&::kvp_state_reorder) state;
} g_lib;

const char *type_name(at::ScalarType t) {
    switch (t) {
        case at::kFloat: return "torch.float32";
        case at::kBFloat16: return "torch.bfloat16";
        case at::kHalf: return "torch.float16";
        case at::kInt: return "torch.int32";
        case at::kLong: return "torch.int64";
        case at::kByte: return "torch.uint8";
        case at::kBool: return "torch.bool";
        default: return c10::toString(t);
    }
}

std::string shape_text(c10::IntArrayRef s) {
    std::string r = "(";
    for (size_t i = 0; i < s.size(); ++i) r += (i ? ", " : "") + std::to_string(s[i]);
    return r + (s.size() == 1 ? ",)" : ")");
}

const at::Tensor &tensor(const char *name, PyObject *x) {
    if (!THPVariable_Check(x)) value_error(std::string(name) + ": expected a tensor, got " + Py_TYPE(x)->tp_name);
    return THPVariable_Unpack(x);
}

int64_t integer(const char *name, PyObject *x) {
    PyObject *i = PyNumber_Index(x);
    if (!i) throw Raised{};
    const long long v = PyLong_AsLongLong(i);
    Py_DECREF(i);
    if (v == -1 && PyErr_Occurred()) {
        PyErr_Clear();
        value_error(std::string(name) + ": out of range");
    }
    return v;
}
int32_t integer32(const char *name, PyObject *x) {
    const int64_t v = integer(name, x);
    if (v < INT32_MIN || v > INT32_MAX) value_error(std::string(name) + ": out of range");
    return (int32_t)v;
}

void *address(PyObject *x) {          // None or an int address
    if (x == Py_None) return nullptr;
    void *p = PyLong_AsVoidPtr(x);
    if (!p && PyErr_Occurred()) throw Raised{};
    return p;
}

// The device that is current, and the stream (None: torch's current one).
struct Here {
    int device = 0;                   // (before CUDA is in use no tensor is on it)
    void *stream = nullptr;

    explicit Here(PyObject *given) {
        PyObject *d = PyObject_CallNoArgs(g_device);
        if (d) {
            device = (int)PyLong_AsLong(d);
            if (given == Py_None) {
                PyObject *s = PyObject_CallOneArg(g_stream, d);
                Py_DECREF(d);
                if (!s) throw Raised{};
                stream = PyLong_AsVoidPtr(s);
                Py_DECREF(s);
                return;
            }
            Py_DECREF(d);
        } else {
            PyErr_Clear();
        }
        if (given == Py_None) return;
        if (PyLong_Check(given)) {
            stream = address(given);
            return;
        }
        PyObject *s = PyObject_GetAttrString(given, "cuda_stream");
        if (!s) throw Raised{};
        stream = PyLong_AsVoidPtr(s);
        Py_DECREF(s);
        if (!stream && PyErr_Occurred()) throw Raised{};
    }

    // Device address of a tensor argument of the given type and shape.
    void *arg(const char *name, PyObject *x, at::ScalarType type, c10::IntArrayRef shape) const {
        if (x == Py_None || PyLong_Check(x)) return address(x);
        const at::Tensor &t = tensor(name, x);
        if (t.scalar_type() != type)
            value_error(std::string(name) + ": expected " + type_name(type) + ", got " + type_name(t.scalar_type()));
        if (t.sizes() != shape)
            value_error(std::string(name) + ": expected shape " + shape_text(shape) + ", got " + shape_text(t.sizes()));
        if (!t.is_cuda() || t.get_device() != device)
            value_error(std::string(name) + ": on " + t.device().str() + ", expected a tensor on the current device, cuda:" +
                        std::to_string(device));
        if (!t.is_contiguous()) value_error(std::string(name) + ": expected a contiguous tensor");
        return t.data_ptr();
    }
    void *arg(const char *name, PyObject *x, at::ScalarType type, std::initializer_list<int64_t> shape) const {
        return arg(name, x, type, c10::IntArrayRef(shape.begin(), shape.size()));
    }
};

// Size of a tensor's dimension, from the back if negative.
int64_t size_of(const char *name, PyObject *x, int64_t dim) {
    const at::Tensor &t = tensor(name, x);
    if (dim < 0) dim += t.dim();
    if (dim < 0 || dim >= t.dim()) value_error(std::string(name) + ": too few dimensions, shape " + shape_text(t.sizes()));
    return t.size(dim);
}

// A structure of the binding (ctypes), by its bytes.
template <class T>
T structure(const char *name, PyObject *x) {
    Py_buffer b;
    if (PyObject_GetBuffer(x, &b, PyBUF_SIMPLE) != 0) throw Raised{};
    T r;
    const bool fits = b.len == (Py_ssize_t)sizeof(T);
    if (fits) std::memcpy(&r, b.buf, sizeof(T));
    PyBuffer_Release(&b);
    if (!fits) value_error(std::string(name) + ": not the structure that the call takes");
    return r;
}

// Host integers of a list, an array or any sequence.
std::vector<int32_t> integers(const char *name, PyObject *x) {
    std::vector<int32_t> r;
    if (!PyList_Check(x) && PyObject_CheckBuffer(x)) {
        Py_buffer b;
        if (PyObject_GetBuffer(x, &b, PyBUF_FORMAT | PyBUF_C_CONTIGUOUS) == 0) {
            const std::string f = b.format ? b.format : "B";
            const bool is32 = f == "i" && b.itemsize == 4, is64 = (f == "l" || f == "q") && b.itemsize == 8;
            if (b.ndim == 1 && (is32 || is64)) {
                const Py_ssize_t n = b.len / b.itemsize;
                r.resize(n);
                bool fits = true;
                for (Py_ssize_t i = 0; i < n; ++i) {
                    const int64_t v = is32 ? static_cast<const int32_t *>(b.buf)[i] : static_cast<const int64_t *>(b.buf)[i];
                    fits &= v >= INT32_MIN && v <= INT32_MAX;
                    r[i] = (int32_t)v;
                }
                PyBuffer_Release(&b);
                if (!fits) value_error(std::string(name) + ": out of range");
                return r;
            }
            const int dims = b.ndim;
            PyBuffer_Release(&b);
            if (dims != 1) value_error(std::string(name) + ": expected one dimension");
        } else {
            PyErr_Clear();
        }
    }
    PyObject *s = PySequence_Fast(x, "expected a sequence of integers");
    if (!s) throw Raised{};
    const Py_ssize_t n = PySequence_Fast_GET_SIZE(s);
    r.reserve(n);
    try {
        for (Py_ssize_t i = 0; i < n; ++i) r.push_back(integer32(name, PySequence_Fast_GET_ITEM(s, i)));
    } catch (...) {
        Py_DECREF(s);
        throw;
    }
    Py_DECREF(s);
    return r;
}

// The library's call without the interpreter's lock; KvpError unless it is OK.
template <class Call>
void run(const char *what, Call call) {
    int rc;
    Py_BEGIN_ALLOW_THREADS;
    rc = call();
    Py_END_ALLOW_THREADS;
    if (rc == KVP_OK) return;
    PyObject *e = PyObject_CallFunction(g_error, "is", rc, what);
    if (e) {
        PyErr_SetObject(g_error, e);
        Py_DECREF(e);
    }
    throw Raised{};
}

// A batch held on the device.
struct Batch {
    int32_t S, MB;
    const int32_t *tables, *lens, *start;

    Batch(const Here &at, PyObject *t, PyObject *l, PyObject *q_start) {
        S = (int32_t)size_of("seq_lens", l, 0);
        MB = 0;
        tables = nullptr;
        if (t) {
            MB = (int32_t)size_of("block_tables", t, -1);
            tables = static_cast<int32_t *>(at.arg("block_tables", t, at::kInt, {S, MB}));
        }
        lens = static_cast<int32_t *>(at.arg("seq_lens", l, at::kInt, {S}));
        start = q_start ? static_cast<int32_t *>(at.arg("q_start", q_start, at::kInt, {S + 1})) : nullptr;
    }
};

void f_append_rope(PyObject *const *a) {
    kvp_pool *pool = static_cast<kvp_pool *>(address(a[0]));
    const std::vector<int32_t> seqs = integers("seqs", a[1]), ntoks = integers("ntoks", a[2]);
    if (seqs.size() != ntoks.size())
        value_error("ntoks: expected " + std::to_string(seqs.size()) + " entries, got " + std::to_string(ntoks.size()));
    const kvp_rope_desc rope = structure<kvp_rope_desc>("rope", a[5]);
    const Here at(a[9]);
    const int64_t T = std::accumulate(ntoks.begin(), ntoks.end(), int64_t{0});
    void *k = nullptr, *v = nullptr, *q = nullptr, *q_out = nullptr;
    int32_t *positions = nullptr, hq = 0;
    if (T != 0) {
        int32_t layers = 0, heads = 0, d = 0;
        run("kvp_pool_shape", [&] { return g_lib.pool_shape(pool, &layers, &heads); });
        run("kvp_pool_head_dim", [&] { return g_lib.pool_head_dim(pool, &d); });
        k = at.arg("k", a[3], at::kBFloat16, {layers, T, heads, d});
        v = at.arg("v", a[4], at::kBFloat16, {layers, T, heads, d});
        positions = static_cast<int32_t *>(at.arg("positions", a[6], at::kInt, {T}));
        if (a[7] != Py_None) {
            hq = (int32_t)size_of("q", a[7], -2);
            q = at.arg("q", a[7], at::kBFloat16, {layers, T, hq, d});
            q_out = at.arg("q_out", a[8], at::kBFloat16, {layers, T, hq, d});
        }
    }
    run("seq_append_rope", [&] {
        return g_lib.append_rope(pool, (int32_t)seqs.size(), seqs.data(), ntoks.data(), k, v, &rope, positions, q, q_out, hq,
                                 at.stream);
    });
}

void f_reorder(PyObject *const *a) {
    const std::vector<int32_t> dst = integers("dst", a[1]), src = integers("src", a[2]);
    if (dst.size() != src.size())
        value_error("src: expected " + std::to_string(dst.size()) + " entries, got " + std::to_string(src.size()));
    kvp_pool *pool = static_cast<kvp_pool *>(address(a[0]));
    run("seq_reorder", [&] { return g_lib.reorder(pool, dst.data(), src.data(), (int32_t)dst.size()); });
}

void f_bounds(PyObject *const *a) {
    const kvp_attn_desc d = structure<kvp_attn_desc>("desc", a[4]);
    const Here at(a[6]);
    const Batch b(at, a[1], a[2], nullptr);
    void *k = at.arg("k_pool", a[0], at::kBFloat16, {d.num_layers, d.num_blocks, d.num_kv_heads, d.block_size, d.head_dim});
    void *out = at.arg("bounds", a[5], at::kBFloat16, {d.num_layers, d.num_blocks, d.num_kv_heads, 2, d.head_dim});
    const int32_t n_new = integer32("n_new", a[3]);
    run("kvp_page_bounds", [&] { return g_lib.bounds(k, b.tables, b.lens, b.S, b.MB, n_new, &d, out, at.stream); });
}

void f_scores(PyObject *const *a) {
    const kvp_attn_desc d = structure<kvp_attn_desc>("desc", a[5]);
    const Here at(a[7]);
    const Batch b(at, a[3], a[4], a[1]);
    const int64_t T = size_of("q", a[0], 1), stride = size_of("scores", a[6], -1);
    void *q = at.arg("q", a[0], at::kBFloat16, {d.num_layers, T, d.num_q_heads, d.head_dim});
    void *bounds = at.arg("bounds", a[2], at::kBFloat16, {d.num_layers, d.num_blocks, d.num_kv_heads, 2, d.head_dim});
    float *out = static_cast<float *>(at.arg("scores", a[6], at::kFloat, {d.num_layers, T, d.num_kv_heads, stride}));
    run("kvp_page_scores", [&] {
        return g_lib.scores(q, b.start, (int32_t)T, bounds, b.tables, b.lens, b.S, b.MB, &d, out, stride, at.stream);
    });
}

void f_select(PyObject *const *a) {
    const kvp_attn_desc d = structure<kvp_attn_desc>("desc", a[3]);
    const Here at(a[8]);
    const Batch b(at, nullptr, a[2], a[1]);
    const int64_t T = size_of("scores", a[0], 1), stride = size_of("scores", a[0], -1), budget = size_of("selected", a[6], -1);
    float *scores = static_cast<float *>(at.arg("scores", a[0], at::kFloat, {d.num_layers, T, d.num_kv_heads, stride}));
    int32_t *out = static_cast<int32_t *>(at.arg("selected", a[6], at::kInt, {d.num_layers, T, d.num_kv_heads, budget}));
    const int32_t sink = integer32("n_sink", a[4]), recent = integer32("n_recent", a[5]);
    const int32_t MB = a[7] == Py_None ? (int32_t)stride : integer32("max_blocks", a[7]);
    run("kvp_page_select", [&] {
        return g_lib.select(scores, stride, b.start, (int32_t)T, b.lens, b.S, MB, &d, (int32_t)budget, sink, recent, out,
                            at.stream);
    });
}

void f_sparse(PyObject *const *a) {
    const kvp_attn_desc d = structure<kvp_attn_desc>("desc", a[7]);
    const Here at(a[10]);
    const Batch b(at, a[4], a[5], a[1]);
    const int64_t T = size_of("q", a[0], 1), budget = size_of("selected", a[6], -1);
    const int64_t wide[4] = {d.num_layers, T, d.num_q_heads, d.head_dim};
    const int64_t pool[5] = {d.num_layers, d.num_blocks, d.num_kv_heads, d.block_size, d.head_dim};
    void *q = at.arg("q", a[0], at::kBFloat16, c10::IntArrayRef(wide, 4));
    void *k = at.arg("k_pool", a[2], at::kBFloat16, c10::IntArrayRef(pool, 5));
    void *v = at.arg("v_pool", a[3], at::kBFloat16, c10::IntArrayRef(pool, 5));
    int32_t *sel = static_cast<int32_t *>(at.arg("selected", a[6], at::kInt, {d.num_layers, T, d.num_kv_heads, budget}));
    void *out = at.arg("out", a[8], at::kBFloat16, c10::IntArrayRef(wide, 4));
    float *lse = static_cast<float *>(at.arg("lse", a[9], at::kFloat, c10::IntArrayRef(wide, 3)));
    run("paged_sparse_attention", [&] {
        return g_lib.sparse(q, b.start, (int32_t)T, k, v, b.tables, b.lens, b.S, b.MB, sel, (int32_t)budget, &d, out, lse,
                            at.stream);
    });
}

void f_beam(PyObject *const *a) {
    const Here at(a[9]);
    // the workspace: a tensor that has what ws_bytes says (None: all of it), or an
    // address of ws_bytes
    int64_t bytes = a[8] == Py_None ? -1 : integer("ws_bytes", a[8]);
    if (a[8] != Py_None && bytes < 0) value_error("ws_bytes: out of range");
    const at::Tensor *room = THPVariable_Check(a[7]) ? &THPVariable_Unpack(a[7]) : nullptr;
    if (room) {
        const int64_t has = (int64_t)room->nbytes();
        if (bytes > has)
            value_error("ws_bytes: " + std::to_string(bytes) + ", but the workspace has " + std::to_string(has));
        if (bytes < 0) bytes = has;
    } else if (bytes < 0) {
        value_error("ws_bytes: needed where the workspace is no tensor");
    }
    const at::Tensor &x = tensor("logits", a[0]);
    const at::ScalarType type = x.scalar_type();
    const int kind = type == at::kFloat ? KVP_F32 : type == at::kBFloat16 ? KVP_BF16 : type == at::kHalf ? KVP_F16 : -1;
    if (kind < 0 || !x.is_cuda() || x.get_device() != at.device)
        value_error("logits: expected float32, bfloat16 or float16 on cuda:" + std::to_string(at.device) + ", got " +
                    type_name(type) + " on " + x.device().str());
    if (x.dim() != 3) value_error("logits: expected three dimensions, got shape " + shape_text(x.sizes()));
    const int64_t G = x.size(0), B = x.size(1), V = x.size(2);
    const int64_t row = B > 1 ? x.stride(1) : G > 1 ? x.stride(0) : V;
    if ((V > 1 && x.stride(2) != 1) || (G > 1 && x.stride(0) != B * row))
        value_error("logits: expected evenly spaced contiguous rows, got strides " + shape_text(x.strides()));
    if (G > INT32_MAX || B > INT32_MAX || V > INT32_MAX) value_error("logits: too large, shape " + shape_text(x.sizes()));
    uint8_t *finished = nullptr;
    if (a[2] != Py_None) {
        const at::ScalarType t = tensor("finished", a[2]).scalar_type();
        if (t != at::kBool && t != at::kByte)
            value_error(std::string("finished: expected bool or uint8, got ") + type_name(t));
        finished = static_cast<uint8_t *>(at.arg("finished", a[2], t, {G, B}));
    }
    const int64_t n = size_of("out_scores", a[4], -1);
    float *cum = static_cast<float *>(at.arg("scores", a[1], at::kFloat, {G, B}));
    float *best = static_cast<float *>(at.arg("out_scores", a[4], at::kFloat, {G, n}));
    int32_t *rows = static_cast<int32_t *>(at.arg("out_rows", a[5], at::kInt, {G, n}));
    int32_t *tokens = static_cast<int32_t *>(at.arg("out_tokens", a[6], at::kInt, {G, n}));
    void *ws = room ? at.arg("workspace", a[7], room->scalar_type(), room->sizes()) : address(a[7]);
    const int32_t pad = integer32("pad_token", a[3]);
    const void *logits = x.data_ptr();
    run("kvp_beam_select", [&] {
        return g_lib.beam(logits, kind, row, cum, finished, pad, (int32_t)G, (int32_t)B, (int32_t)V, (int32_t)n, best, rows,
                          tokens, ws, (size_t)bytes, at.stream);
    });
}

void f_state(PyObject *const *a) {
    const Here at(a[4]);
    const at::Tensor &src = tensor("src", a[0]);
    const at::Tensor &index = tensor("index", a[2]);
    int64_t dim = integer("dim", a[3]);
    if (dim < 0) dim += src.dim();
    if (dim < 0 || dim >= src.dim()) value_error("dim: no such dimension of shape " + shape_text(src.sizes()));
    const int64_t n_src = src.size(dim), n_dst = size_of("dst", a[1], dim);
    if (index.numel() != n_dst)
        value_error("index: expected " + std::to_string(n_dst) + " entries, got " + std::to_string(index.numel()));
    int64_t outer = 1, row = (int64_t)src.element_size();
    for (int64_t i = 0; i < dim; ++i) outer *= src.size(i);
    for (int64_t i = dim + 1; i < src.dim(); ++i) row *= src.size(i);
    std::vector<int64_t> want = src.sizes().vec();
    want[dim] = n_dst;
    if (n_src > INT32_MAX || n_dst > INT32_MAX) value_error("src: too many rows");
    void *from = at.arg("src", a[0], src.scalar_type(), src.sizes());
    void *to = at.arg("dst", a[1], src.scalar_type(), c10::IntArrayRef(want));
    const int32_t *at_rows = static_cast<int32_t *>(at.arg("index", a[2], at::kInt, index.sizes()));
    run("kvp_state_reorder",
        [&] { return g_lib.state(from, to, at_rows, outer, (int32_t)n_src, (int32_t)n_dst, row, at.stream); });
}

template <void (*F)(PyObject *const *), int N>
PyObject *entry(PyObject *, PyObject *const *args, Py_ssize_t n) {
    if (n != N) {
        PyErr_Format(PyExc_TypeError, "expected %d arguments, got %zd", N, n);
        return nullptr;
    }
    try {
        F(args);
        Py_RETURN_NONE;
    } catch (const Raised &) {
    } catch (const std::bad_alloc &) {
        PyErr_NoMemory();
    } catch (const std::exception &e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
    }
    return nullptr;
}

// bind(KvpError, device function, stream function, addresses in Lib's order)
PyObject *bind(PyObject *, PyObject *const *args, Py_ssize_t n) {
    constexpr int kFunctions = sizeof(Lib) / sizeof(void *);
    if (n != 3 + kFunctions) {
        PyErr_SetString(PyExc_TypeError, "bind: wrong number of arguments");
        return nullptr;
    }
    void *f[kFunctions];
    for (int i = 0; i < kFunctions; ++i) {
        f[i] = PyLong_AsVoidPtr(args[3 + i]);
        if (!f[i]) {
            if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, "bind: a null address");
            return nullptr;
        }
    }
    std::memcpy(&g_lib, f, sizeof f);
    // (kept for the process: nothing unbinds them)
    PyObject **to[3] = {&g_error, &g_device, &g_stream};
    for (int i = 0; i < 3; ++i) {
        Py_INCREF(args[i]);
        Py_XSETREF(*to[i], args[i]);
    }
    Py_RETURN_NONE;
}

#define KVP_ENTRY(name, f, n) {name, (PyCFunction)(void (*)(void))entry<f, n>, METH_FASTCALL, nullptr}
PyMethodDef methods[] = {
    {"bind", (PyCFunction)(void (*)(void))bind, METH_FASTCALL, nullptr},
    KVP_ENTRY("seq_append_rope", f_append_rope, 10),
    KVP_ENTRY("seq_reorder", f_reorder, 3),
    KVP_ENTRY("kvp_page_bounds", f_bounds, 7),
    KVP_ENTRY("kvp_page_scores", f_scores, 8),
    KVP_ENTRY("kvp_page_select", f_select, 9),
    KVP_ENTRY("paged_sparse_attention", f_sparse, 11),
    KVP_ENTRY("kvp_beam_select", f_beam, 10),
    KVP_ENTRY("kvp_state_reorder", f_state, 5),
    {nullptr, nullptr, 0, nullptr},
};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_calls", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__calls(void) {
    PyObject *m = PyModule_Create(&module);
    PyObject *f = Py_BuildValue("(ssssssssss)", "seq_append_rope", "seq_reorder", "kvp_pool_shape", "kvp_pool_head_dim",
                                "kvp_page_bounds", "kvp_page_scores", "kvp_page_select", "paged_sparse_attention",
                                "kvp_beam_select", "kvp_state_reorder");
    if (!m || !f || PyModule_AddObjectRef(m, "functions", f) != 0 ||
        PyModule_AddStringConstant(m, "torch_version", KVP_TORCH_VERSION) != 0)
        Py_CLEAR(m);
    Py_XDECREF(f);
    return m;
}
