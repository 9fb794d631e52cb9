// bind.cpp -- the Python calls of the target-pass operators (include/dspark.h).
//
// They run once per layer or per cycle, some on inputs so small that the host's
// share is the whole time: through ctypes, checking thirteen tensors and making
// five cost 24 us around a kernel of 3.  This module (6 us) does the same checks and
// allocations on the tensors themselves and calls the same C entry points; it
// holds no state and none of the operators' arithmetic.
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cmath>
#include <exception>
#include <initializer_list>

#include "../../include/dspark.h"

namespace {

PyObject *g_error = nullptr;          // the package's DSparkError
PyObject *g_out_of_memory = nullptr;  // torch.OutOfMemoryError

struct Raised {};  // a Python exception is set

[[noreturn]] void raise(PyObject *type, const char *fmt, const char *name) {
    PyErr_Format(type, fmt, name);
    throw Raised{};
}

const at::Tensor &tensor(const char *name, PyObject *o) {
    if (!THPVariable_Check(o)) raise(PyExc_TypeError, "%s is not a tensor", name);
    return THPVariable_Unpack(o);
}

const char *type_name(at::ScalarType t) { return c10::toString(t); }

void check_type(const char *name, const at::Tensor &t, at::ScalarType dt) {
    if (t.scalar_type() == dt) return;
    PyErr_Format(PyExc_TypeError, "%s is %s, expected %s", name, type_name(t.scalar_type()), type_name(dt));
    throw Raised{};
}

// The GPU that a call runs on: every tensor of the call is on it.
struct Gpu {
    c10::Device device;
    explicit Gpu(const char *name, const at::Tensor &t) : device(t.device()) {
        if (!t.is_cuda()) raise(PyExc_ValueError, "dspark tensors must live on the GPU: %s does not", name);
    }

    void check(const char *name, const at::Tensor &t) const {
        if (!t.is_cuda()) raise(PyExc_ValueError, "dspark tensors must live on the GPU: %s does not", name);
        if (t.device() != device) raise(PyExc_ValueError, "%s is on another GPU than the other tensors", name);
    }

    // address of a contiguous tensor of this element type (and shape)
    void *want(const char *name, PyObject *o, at::ScalarType dt) const {
        const at::Tensor &t = tensor(name, o);
        check_type(name, t, dt);
        check(name, t);
        if (!t.is_contiguous()) raise(PyExc_ValueError, "dspark tensors must be contiguous: %s is not", name);
        return t.data_ptr();
    }
    void *want(const char *name, PyObject *o, at::ScalarType dt, std::initializer_list<int64_t> shape) const {
        const at::Tensor &t = tensor(name, o);
        check_type(name, t, dt);
        if (t.sizes() != at::IntArrayRef(shape)) raise(PyExc_ValueError, "%s has another shape than expected", name);
        return want(name, o, dt);
    }
    void *maybe(const char *name, PyObject *o, at::ScalarType dt) const { return o == Py_None ? nullptr : want(name, o, dt); }
    void *maybe(const char *name, PyObject *o, at::ScalarType dt, std::initializer_list<int64_t> shape) const {
        return o == Py_None ? nullptr : want(name, o, dt, shape);
    }

    // a [N, H, D] view whose D elements are adjacent
    const void *heads(const char *name, PyObject *o, at::ScalarType dt, std::initializer_list<int64_t> shape, int64_t *row,
                      int64_t *head) const {
        const at::Tensor &t = tensor(name, o);
        check(name, t);
        check_type(name, t, dt);
        if (t.sizes() != at::IntArrayRef(shape)) raise(PyExc_ValueError, "%s has another shape than expected", name);
        if (t.stride(2) != 1 && t.size(2) > 1) raise(PyExc_ValueError, "the elements of a head of %s must be adjacent", name);
        *row = t.stride(0);
        *head = t.stride(1);
        return t.data_ptr();
    }

    at::Tensor empty(at::ScalarType dt, std::initializer_list<int64_t> shape) const {
        return at::detail::empty_cuda(at::IntArrayRef(shape), dt, device, std::nullopt);
    }
    dspark_stream_t stream() const {
        return reinterpret_cast<dspark_stream_t>(c10::cuda::getCurrentCUDAStream(device.index()).stream());
    }
};

int32_t dtype_code(const char *name, const at::Tensor &t) {
    if (t.scalar_type() == at::kBFloat16) return DSPARK_BF16;
    if (t.scalar_type() == at::kFloat) return DSPARK_F32;
    PyErr_Format(PyExc_TypeError, "unsupported element type %s of %s", type_name(t.scalar_type()), name);
    throw Raised{};
}

const at::Tensor &dims(const char *name, PyObject *o, int64_t n) {
    const at::Tensor &t = tensor(name, o);
    if (t.dim() != n) raise(PyExc_ValueError, "%s has another number of dimensions than expected", name);
    return t;
}

int32_t small(const char *name, int64_t v) {
    if (v < INT32_MIN || v > INT32_MAX) raise(PyExc_ValueError, "%s is beyond 32 bits", name);
    return (int32_t)v;
}

int32_t integer(const char *name, PyObject *o) {
    const long long v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred()) throw Raised{};
    return small(name, v);
}

void check(int rc) {
    if (rc == DSPARK_OK) return;
    PyObject *e = PyObject_CallFunction(g_error, "is", rc, dspark_last_error());
    if (e) {
        PyErr_SetObject(g_error, e);
        Py_DECREF(e);
    }
    throw Raised{};
}

// A new dict, or the caller's.
struct Outputs {
    PyObject *dict;
    bool own;
    explicit Outputs(PyObject *given) : dict(given), own(given == Py_None) {
        if (own) {
            dict = PyDict_New();
            if (!dict) throw Raised{};
        } else if (!PyDict_Check(given)) {
            raise(PyExc_TypeError, "%s is not a dict", "out");
        }
    }
    Outputs(const Outputs &) = delete;
    ~Outputs() {
        if (own) Py_XDECREF(dict);
    }
    // address of output `name`: the caller's, or one made for the call
    void *get(const Gpu &gpu, const char *name, at::ScalarType dt, std::initializer_list<int64_t> shape, bool optional = false) {
        if (!own) {
            PyObject *o = PyDict_GetItemString(dict, name);
            if (!o || o == Py_None) {
                if (optional) return nullptr;
                raise(PyExc_KeyError, "%s", name);
            }
            return gpu.want(name, o, dt, shape);
        }
        return add(name, gpu.empty(dt, shape));
    }
    // the same for heads: the caller's may be a view whose D elements are adjacent
    void *heads(const Gpu &gpu, const char *name, at::ScalarType dt, std::initializer_list<int64_t> shape, int64_t *row, int64_t *head) {
        if (!own) {
            PyObject *o = PyDict_GetItemString(dict, name);
            if (!o || o == Py_None) raise(PyExc_KeyError, "%s", name);
            return const_cast<void *>(gpu.heads(name, o, dt, shape, row, head));
        }
        const int64_t *n = shape.begin();
        *row = n[1] * n[2];
        *head = n[2];
        return add(name, gpu.empty(dt, shape));
    }
    struct Part {
        const char *name;
        int64_t n;
        int32_t **at;
    };
    // int32 vectors in one allocation, each on a 256-byte boundary: the allocator is what
    // a call with small outputs costs most
    void get_together(const Gpu &gpu, std::initializer_list<Part> parts) {
        if (!own) {
            for (const Part &p : parts) *p.at = static_cast<int32_t *>(get(gpu, p.name, at::kInt, {p.n}));
            return;
        }
        int64_t all = 0;
        for (const Part &p : parts) all += (p.n + 63) / 64 * 64;
        const at::Tensor whole = gpu.empty(at::kInt, {all});
        int64_t from = 0;
        for (const Part &p : parts) {
            at::Tensor t = at::detail::make_tensor<c10::TensorImpl>(c10::Storage(whole.storage()), whole.key_set(), whole.dtype());
            t.unsafeGetTensorImpl()->set_storage_offset(from);
            t.unsafeGetTensorImpl()->set_sizes_contiguous({p.n});
            *p.at = static_cast<int32_t *>(add(p.name, std::move(t)));
            from += (p.n + 63) / 64 * 64;
        }
    }
    void *add(const char *name, at::Tensor t) {
        void *at = t.data_ptr();
        PyObject *o = THPVariable_Wrap(std::move(t));
        const int rc = o ? PyDict_SetItemString(dict, name, o) : -1;
        Py_XDECREF(o);
        if (rc < 0) throw Raised{};
        return at;
    }
    PyObject *take() {
        if (!own) Py_INCREF(dict);
        own = false;
        return dict;
    }
};

constexpr at::ScalarType I32 = at::kInt, I64 = at::kLong, F32 = at::kFloat;
int32_t *i32(void *p) { return static_cast<int32_t *>(p); }
float *f32(void *p) { return static_cast<float *>(p); }

void count_args(Py_ssize_t got, Py_ssize_t want) {
    if (got != want) raise(PyExc_TypeError, "%s", "wrong number of arguments");
}

// lens rows table held free n_free page N parents max_rows out err
PyObject *page_map(PyObject *const *x, Py_ssize_t n) {
    count_args(n, 12);
    const at::Tensor &table = dims("table", x[2], 2), &free = dims("free", x[4], 1);
    const Gpu gpu("table", table);
    const c10::cuda::CUDAGuard guard(gpu.device);
    const int64_t R = table.size(0);
    dspark_page_map_args a{};
    a.R = small("R", R);
    a.page = integer("page", x[6]);
    a.n_pages = small("n_pages", free.size(0));
    a.max_pages = small("max_pages", table.size(1));
    a.N = integer("N", x[7]);
    if (a.N < 0) raise(PyExc_ValueError, "%s is negative", "N");
    if (x[8] != Py_None) {
        const int32_t rows = x[9] == Py_None ? 0 : integer("max_rows", x[9]);
        if (rows < 1) raise(PyExc_ValueError, "trees need %s", "max_rows");
        a.W = (int32_t)(((int64_t)rows + 63) / 64);
        a.n_parents = small("parents", tensor("parents", x[8]).numel());
        a.parents = i32(gpu.want("parents", x[8], I32));
    }
    a.len = i32(gpu.want("lens", x[0], I32, {R}));
    a.rows = i32(gpu.want("rows", x[1], I32, {R}));
    a.table = i32(gpu.want("table", x[2], I32));
    a.held = i32(gpu.want("held", x[3], I32, {R}));
    a.free_list = i32(gpu.want("free", x[4], I32));
    a.n_free = i32(gpu.want("n_free", x[5], I32, {1}));
    a.err = i32(gpu.maybe("err", x[11], I32));
    Outputs out(x[10]);
    // what the next call reads apart from what the cycle does, so that it keeps no more alive
    out.get_together(gpu, {{"held", R, &a.held_out}, {"n_free", 1, &a.n_free_out}});
    out.get_together(gpu, {{"row_start", R + 1, &a.row_start}, {"slot", a.N, &a.slot}, {"pos", a.N, &a.pos}});
    if (a.parents) a.mask = static_cast<uint64_t *>(out.get(gpu, "mask", I64, {a.N, a.W}));
    check(dspark_page_map(&a, gpu.stream()));
    return out.take();
}

// k v slot k_cache v_cache err
PyObject *cache_store(PyObject *const *x, Py_ssize_t n) {
    count_args(n, 6);
    const at::Tensor &cache = dims("k_cache", x[3], 4), &k = dims("k", x[0], 3);
    const Gpu gpu("k_cache", cache);
    const c10::cuda::CUDAGuard guard(gpu.device);
    const at::ScalarType dt = cache.scalar_type();
    const int64_t N = k.size(0), pages = cache.size(0), H = cache.size(1), page = cache.size(2), D = cache.size(3);
    dspark_cache_store_args a{};
    a.N = small("N", N), a.H = small("H", H), a.D = small("D", D), a.page = small("page", page), a.n_pages = small("n_pages", pages);
    a.dtype = dtype_code("k_cache", cache);
    dims("v", x[1], 3);
    a.k = gpu.heads("k", x[0], dt, {N, H, D}, &a.k_row, &a.k_head);
    a.v = gpu.heads("v", x[1], dt, {N, H, D}, &a.v_row, &a.v_head);
    a.slot = i32(gpu.want("slot", x[2], I32, {N}));
    a.k_cache = gpu.want("k_cache", x[3], dt);
    a.v_cache = gpu.want("v_cache", x[4], dt, {pages, H, page, D});
    a.err = i32(gpu.maybe("err", x[5], I32));
    check(dspark_cache_store(&a, gpu.stream()));
    Py_RETURN_NONE;
}

float number(PyObject *o) {
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred()) throw Raised{};
    return (float)v;
}

// q k v pos freq q_weight k_weight eps interleaved slot k_cache v_cache out err
PyObject *rope_store(PyObject *const *x, Py_ssize_t n) {
    count_args(n, 14);
    const bool queries = x[0] != Py_None, keys = x[1] != Py_None, cached = x[9] != Py_None;
    if (!queries && !keys) raise(PyExc_ValueError, "%s", "neither queries nor keys are given");
    const at::Tensor &first = dims(queries ? "q" : "k", x[queries ? 0 : 1], 3);
    const Gpu gpu(queries ? "q" : "k", first);
    const c10::cuda::CUDAGuard guard(gpu.device);
    const at::ScalarType dt = first.scalar_type();
    const int64_t N = first.size(0), D = first.size(2);
    dspark_rope_store_args a{};
    a.N = small("N", N), a.D = small("D", D);
    a.dtype = dtype_code(queries ? "q" : "k", first);
    a.eps = number(x[7]);
    a.interleaved = PyObject_IsTrue(x[8]);
    if (a.interleaved < 0) throw Raised{};
    a.pos = i32(gpu.want("pos", x[3], I32, {N}));
    a.rot = small("rot", 2 * dims("freq", x[4], 1).size(0));
    a.freq = f32(gpu.want("freq", x[4], F32));
    a.q_weight = gpu.maybe("q_weight", x[5], dt, {D});
    a.k_weight = gpu.maybe("k_weight", x[6], dt, {D});
    a.err = i32(gpu.maybe("err", x[13], I32));
    if (queries) {
        a.Hq = small("Hq", first.size(1));
        a.q = gpu.heads("q", x[0], dt, {N, a.Hq, D}, &a.q_row, &a.q_head);
    }
    if (keys) {
        a.H = small("H", dims("k", x[1], 3).size(1));
        a.k = gpu.heads("k", x[1], dt, {N, a.H, D}, &a.k_row, &a.k_head);
    }
    if (cached) {
        if (!keys) raise(PyExc_ValueError, "%s", "slots are given without keys");
        const at::Tensor &cache = dims("k_cache", x[10], 4);
        dims("v", x[2], 3);
        a.v = gpu.heads("v", x[2], dt, {N, a.H, D}, &a.v_row, &a.v_head);
        a.slot = i32(gpu.want("slot", x[9], I32, {N}));
        const int64_t pages = cache.size(0), page = cache.size(2);
        a.page = small("page", page), a.n_pages = small("n_pages", pages);
        a.k_cache = gpu.want("k_cache", x[10], dt, {pages, a.H, page, D});
        a.v_cache = gpu.want("v_cache", x[11], dt, {pages, a.H, page, D});
    } else if (x[10] != Py_None || x[11] != Py_None) {
        raise(PyExc_ValueError, "%s", "caches are given without slots");
    }
    Outputs out(x[12]);
    if (queries) a.q_out = out.heads(gpu, "q", dt, {N, a.Hq, D}, &a.q_out_row, &a.q_out_head);
    if (keys && !cached) a.k_out = out.heads(gpu, "k", dt, {N, a.H, D}, &a.k_out_row, &a.k_out_head);
    check(dspark_rope_store(&a, gpu.stream()));
    return out.take();
}

// tokens of a page of a cache in 4 bits [n_pages, H, page * D * 9 / 16]
int64_t page_of(const char *name, const at::Tensor &cache, int64_t D) {
    if (D < 16 || D % 16 || cache.size(2) % (D / 16 * 9)) raise(PyExc_ValueError, "pages of %s are not whole tokens of this head size", name);
    return cache.size(2) / (D / 16 * 9);
}

// k v slot k_cache v_cache values out err
PyObject *cache_store4(PyObject *const *x, Py_ssize_t n) {
    count_args(n, 8);
    const at::Tensor &cache = dims("k_cache", x[3], 3), &k = dims("k", x[0], 3);
    const Gpu gpu("k_cache", cache);
    const c10::cuda::CUDAGuard guard(gpu.device);
    const at::ScalarType dt = k.scalar_type();
    const int64_t N = k.size(0), pages = cache.size(0), H = cache.size(1), D = k.size(2);
    dspark_cache_store4_args a{};
    a.N = small("N", N), a.H = small("H", H), a.D = small("D", D), a.n_pages = small("n_pages", pages);
    a.page = small("page", page_of("k_cache", cache, D));
    a.dtype = dtype_code("k", k);
    dims("v", x[1], 3);
    a.k = gpu.heads("k", x[0], dt, {N, H, D}, &a.k_row, &a.k_head);
    a.v = gpu.heads("v", x[1], dt, {N, H, D}, &a.v_row, &a.v_head);
    a.slot = i32(gpu.want("slot", x[2], I32, {N}));
    a.k_cache = static_cast<uint8_t *>(gpu.want("k_cache", x[3], at::kByte));
    a.v_cache = static_cast<uint8_t *>(gpu.want("v_cache", x[4], at::kByte, {pages, H, cache.size(2)}));
    a.err = i32(gpu.maybe("err", x[7], I32));
    const int values = PyObject_IsTrue(x[5]);
    if (values < 0) throw Raised{};
    if (!values && x[6] == Py_None) {
        check(dspark_cache_store4(&a, gpu.stream()));
        Py_RETURN_NONE;
    }
    Outputs out(x[6]);
    a.k_out = out.get(gpu, "k", dt, {N, H, D});
    a.v_out = out.get(gpu, "v", dt, {N, H, D});
    check(dspark_cache_store4(&a, gpu.stream()));
    return out.take();
}

// q k_cache v_cache table lens row_start mask scale max_rows out ws err; size_only: the
// workspace's bytes and no call; four: caches in 4 bits
PyObject *tree_attention_as(PyObject *const *x, Py_ssize_t n, bool size_only, bool four) {
    count_args(n, 12);
    const at::Tensor &cache = dims("k_cache", x[1], four ? 3 : 4), &q = dims("q", x[0], 3), &table = dims("table", x[3], 2);
    const Gpu gpu("k_cache", cache);
    const c10::cuda::CUDAGuard guard(gpu.device);
    const at::ScalarType dt = four ? q.scalar_type() : cache.scalar_type(), held = four ? at::kByte : dt;
    const int64_t N = q.size(0), Hq = q.size(1), R = table.size(0);
    const int64_t pages = cache.size(0), H = cache.size(1), D = four ? q.size(2) : cache.size(3);
    const int64_t page = four ? page_of("k_cache", cache, D) : cache.size(2);
    dspark_tree_attention_args a{};
    a.R = small("R", R), a.N = small("N", N), a.Hq = small("Hq", Hq), a.H = small("H", H), a.D = small("D", D);
    a.page = small("page", page), a.n_pages = small("n_pages", pages), a.max_pages = small("max_pages", table.size(1));
    a.dtype = four ? dtype_code("q", q) : dtype_code("k_cache", cache);
    a.max_rows = integer("max_rows", x[8]);
    if (x[7] != Py_None) a.scale = number(x[7]);
    else a.scale = D > 0 ? (float)(1.0 / std::sqrt((double)D)) : 1.f;
    a.q = gpu.heads("q", x[0], dt, {N, Hq, D}, &a.q_row, &a.q_head);
    a.k_cache = gpu.want("k_cache", x[1], held);
    a.v_cache = four ? gpu.want("v_cache", x[2], held, {pages, H, cache.size(2)}) : gpu.want("v_cache", x[2], held, {pages, H, page, D});
    a.table = i32(gpu.want("table", x[3], I32));
    a.len = i32(gpu.want("lens", x[4], I32, {R}));
    a.row_start = i32(gpu.want("row_start", x[5], I32, {R + 1}));
    if (x[6] != Py_None) {
        a.W = small("W", dims("mask", x[6], 2).size(1));
        a.mask = static_cast<uint64_t *>(gpu.want("mask", x[6], I64, {N, a.W}));
    }
    a.err = i32(gpu.maybe("err", x[11], I32));
    const size_t bytes = four ? dspark_tree_attention4_workspace_size(&a) : dspark_tree_attention_workspace_size(&a);
    if (size_only) return PyLong_FromSize_t(bytes);
    Outputs out(x[9]);
    a.out = out.get(gpu, "out", dt, {N, Hq, D});
    a.lse = f32(out.get(gpu, "lse", F32, {N, Hq}, true));
    at::Tensor own;
    void *ws = nullptr;
    if (x[10] == Py_None) {
        own = gpu.empty(at::kByte, {(int64_t)(bytes ? bytes : 256)});
        ws = own.data_ptr();
    } else {
        const at::Tensor &t = tensor("ws", x[10]);
        gpu.check("ws", t);
        if (!t.is_contiguous() || t.nbytes() < bytes) {
            PyErr_Format(PyExc_ValueError, "workspace of %zu bytes, need %zu adjacent ones", t.nbytes(), bytes);
            throw Raised{};
        }
        ws = t.data_ptr();
    }
    check(four ? dspark_tree_attention4(&a, ws, gpu.stream()) : dspark_tree_attention(&a, ws, gpu.stream()));
    return out.take();
}
PyObject *tree_attention(PyObject *const *x, Py_ssize_t n) { return tree_attention_as(x, n, false, false); }
PyObject *tree_attention_workspace_size(PyObject *const *x, Py_ssize_t n) { return tree_attention_as(x, n, true, false); }
PyObject *tree_attention4(PyObject *const *x, Py_ssize_t n) { return tree_attention_as(x, n, false, true); }
PyObject *tree_attention4_workspace_size(PyObject *const *x, Py_ssize_t n) { return tree_attention_as(x, n, true, true); }

// T row_start tok mask hist hist_len prompt_len rep freq pres bias_start bias_id bias_val allow allow_row out err
PyObject *logit_rules(PyObject *const *x, Py_ssize_t n) {
    count_args(n, 17);
    const at::Tensor &T = dims("T", x[0], 2);
    const Gpu gpu("T", T);
    const c10::cuda::CUDAGuard guard(gpu.device);
    const at::ScalarType dt = T.scalar_type();
    const int64_t N = T.size(0), V = T.size(1), R = dims("row_start", x[1], 1).size(0) - 1;
    dspark_logit_rules_args a{};
    a.R = small("R", R), a.N = small("N", N), a.V = small("V", V);
    a.dtype = dtype_code("T", T);
    a.T = gpu.want("T", x[0], dt);
    a.row_start = i32(gpu.want("row_start", x[1], I32));
    a.tok = i32(gpu.maybe("tok", x[2], I32, {N}));
    if (x[3] != Py_None) {
        a.W = small("W", dims("mask", x[3], 2).size(1));
        a.mask = static_cast<uint64_t *>(gpu.want("mask", x[3], I64, {N, a.W}));
    }
    if (x[4] != Py_None) {
        a.max_hist = small("max_hist", dims("hist", x[4], 2).size(1));
        a.hist = i32(gpu.want("hist", x[4], I32, {R, a.max_hist}));
    }
    a.hist_len = i32(gpu.maybe("hist_len", x[5], I32, {R}));
    a.prompt_len = i32(gpu.maybe("prompt_len", x[6], I32, {R}));
    a.rep = f32(gpu.maybe("rep", x[7], F32, {R}));
    a.freq = f32(gpu.maybe("freq", x[8], F32, {R}));
    a.pres = f32(gpu.maybe("pres", x[9], F32, {R}));
    a.bias_start = i32(gpu.maybe("bias_start", x[10], I32, {R + 1}));
    if (x[11] != Py_None) {
        a.n_bias = small("n_bias", dims("bias_id", x[11], 1).size(0));
        a.bias_id = i32(gpu.want("bias_id", x[11], I32));
    }
    a.bias_val = f32(gpu.maybe("bias_val", x[12], F32, {a.n_bias}));
    if (x[13] != Py_None) {
        a.n_allow = small("n_allow", dims("allow", x[13], 2).size(0));
        a.allow = reinterpret_cast<uint32_t *>(gpu.want("allow", x[13], I32, {a.n_allow, (V + 31) / 32}));
    }
    a.allow_row = i32(gpu.maybe("allow_row", x[14], I32, {N}));
    a.err = i32(gpu.maybe("err", x[16], I32));
    if (x[15] != Py_None) {
        a.out = gpu.want("out", x[15], dt, {N, V});
        check(dspark_logit_rules(&a, gpu.stream()));
        Py_INCREF(x[15]);
        return x[15];
    }
    at::Tensor out = gpu.empty(dt, {N, V});
    a.out = out.data_ptr();
    check(dspark_logit_rules(&a, gpu.stream()));
    return THPVariable_Wrap(std::move(out));
}

// no C++ exception leaves the module
template <PyObject *(*F)(PyObject *const *, Py_ssize_t)>
PyObject *call(PyObject *, PyObject *const *x, Py_ssize_t n) {
    try {
        return F(x, n);
    } catch (const Raised &) {
        return nullptr;
    } catch (const c10::OutOfMemoryError &e) {
        PyErr_SetString(g_out_of_memory, e.what_without_backtrace());
    } catch (const std::exception &e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
    } catch (...) {
        PyErr_SetString(PyExc_RuntimeError, "unknown C++ exception");
    }
    return nullptr;
}

// the exceptions to raise: DSparkError, torch.OutOfMemoryError
PyObject *set_errors(PyObject *const *x, Py_ssize_t n) {
    count_args(n, 2);
    Py_INCREF(x[0]);
    Py_XSETREF(g_error, x[0]);
    Py_INCREF(x[1]);
    Py_XSETREF(g_out_of_memory, x[1]);
    Py_RETURN_NONE;
}

template <PyObject *(*F)(PyObject *const *, Py_ssize_t)>
constexpr PyMethodDef method(const char *name) {
    return PyMethodDef{name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&call<F>)), METH_FASTCALL, nullptr};
}

PyMethodDef g_methods[] = {method<page_map>("page_map"),
                           method<cache_store>("cache_store"),
                           method<tree_attention>("tree_attention"),
                           method<tree_attention_workspace_size>("tree_attention_workspace_size"),
                           method<rope_store>("rope_store"),
                           method<cache_store4>("cache_store4"),
                           method<tree_attention4>("tree_attention4"),
                           method<tree_attention4_workspace_size>("tree_attention4_workspace_size"),
                           method<logit_rules>("logit_rules"),
                           method<set_errors>("set_errors"),
                           {nullptr, nullptr, 0, nullptr}};

PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_dspark_bind", nullptr, -1, g_methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__dspark_bind(void) { return PyModule_Create(&g_module); }
