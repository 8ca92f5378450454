// Python binding of the drafted step's calls (paged_kv_rope_append,
// paged_attention_tree, paged_kv_tree_commit) and of those of a cache within a
// budget (paged_kv_norm_rope_append, paged_attention_decode_weights,
// paged_attention_prefill_weights, paged_kv_evict): argument checks and marshalling
// only, as in ops.py, in C++.
//
// Each of these calls takes a dozen tensors, and checking and unpacking them
// from Python through ctypes took 22 to 30 us a call on the Grace cores, ten
// times what their smallest kernels take.  The functions here are called
// positionally by ops.py, which documents them.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <initializer_list>
#include <string>

#include "paged_kv.h"

namespace {

struct Failed {};  // a Python error is set

[[noreturn]] void fail(PyObject* type, const std::string& what) {
    PyErr_SetString(type, what.c_str());
    throw Failed();
}

const char* dtype_name(at::ScalarType t) {
    switch (t) {
        case at::kHalf: return "torch.float16";
        case at::kInt: return "torch.int32";
        case at::kLong: return "torch.int64";
        case at::kFloat: return "torch.float32";
        case at::kByte: return "torch.uint8";
        default: return c10::toString(t);
    }
}

std::string shape_of(c10::IntArrayRef s) {
    std::string r = "(";
    for (size_t i = 0; i < s.size(); ++i) r += (i ? ", " : "") + std::to_string(s[i]);
    return r + (s.size() == 1 ? ",)" : ")");
}

// The call's tensors share one device, the first one's.
struct Call {
    c10::DeviceIndex device = -1;
    const char* first = nullptr;

    const at::Tensor& tensor(PyObject* o, const char* name) {
        if (!THPVariable_Check(o)) fail(PyExc_TypeError, std::string(name) + " must be a torch.Tensor");
        const at::Tensor& t = THPVariable_Unpack(o);
        if (!t.is_cuda()) fail(PyExc_ValueError, std::string(name) + " must be on a CUDA device");
        const c10::DeviceIndex d = t.get_device();
        if (device < 0) {
            device = d;
            first = name;
        } else if (d != device) {
            fail(PyExc_ValueError, std::string(name) + " is on cuda:" + std::to_string(d) + ", " + first +
                                       " on cuda:" + std::to_string(device));
        }
        return t;
    }
    const at::Tensor& need(PyObject* o, const char* name, at::ScalarType dtype, int64_t ndim) {
        const at::Tensor& t = tensor(o, name);
        if (t.scalar_type() != dtype)
            fail(PyExc_TypeError, std::string(name) + " must be " + dtype_name(dtype) + ", got " + dtype_name(t.scalar_type()));
        if (t.dim() != ndim)
            fail(PyExc_ValueError, std::string(name) + " must have " + std::to_string(ndim) + " dims, got " + shape_of(t.sizes()));
        if (!t.is_contiguous()) fail(PyExc_ValueError, std::string(name) + " must be contiguous");
        return t;
    }
    // Data of an optional tensor (None: null).
    void* optional(PyObject* o, const char* name, at::ScalarType dtype, int64_t ndim) {
        return o == Py_None ? nullptr : need(o, name, dtype, ndim).data_ptr();
    }
    // fp16 [tokens][heads][dim]; only the tokens may be strided.
    const at::Tensor& tokens(PyObject* o, const char* name, int64_t heads, int64_t dim, int64_t* stride) {
        const at::Tensor& t = tensor(o, name);
        if (t.scalar_type() != at::kHalf)
            fail(PyExc_TypeError, std::string(name) + " must be torch.float16, got " + dtype_name(t.scalar_type()));
        if (t.dim() != 3 || t.size(1) != heads || t.size(2) != dim)
            fail(PyExc_ValueError, std::string(name) + " must be [tokens][" + std::to_string(heads) + "][" +
                                       std::to_string(dim) + "], got " + shape_of(t.sizes()));
        if (t.numel() && ((dim > 1 && t.stride(2) != 1) || (heads > 1 && t.stride(1) != dim)))
            fail(PyExc_ValueError, std::string(name) + "'s heads and dims must be contiguous");
        *stride = t.size(0) > 1 ? t.stride(0) : heads * dim;  // the stride of a single token means nothing
        return t;
    }
};

void need_shape(const at::Tensor& t, const char* name, std::initializer_list<int64_t> shape) {
    const c10::IntArrayRef want(shape.begin(), shape.size());
    if (t.sizes() != want)
        fail(PyExc_ValueError, std::string(name) + " must have shape " + shape_of(want) + ", got " + shape_of(t.sizes()));
}

int to_int(PyObject* o) {
    const long v = PyLong_AsLong(o);
    if (v == -1 && PyErr_Occurred()) throw Failed();
    if (v > INT_MAX || v < INT_MIN) fail(PyExc_OverflowError, "integer argument does not fit 32 bits");
    return (int)v;
}

float to_float(PyObject* o) {
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred()) throw Failed();
    return (float)v;
}

// None: the device's current stream; else a torch stream or a raw handle.
cudaStream_t to_stream(PyObject* o, c10::DeviceIndex device) {
    if (o == Py_None) return c10::cuda::getCurrentCUDAStream(device).stream();
    PyObject* raw = PyObject_GetAttrString(o, "cuda_stream");
    if (!raw) {
        PyErr_Clear();
        raw = Py_NewRef(o);
    }
    PyObject* index = PyNumber_Index(raw);
    Py_DECREF(raw);
    if (!index) throw Failed();
    void* p = PyLong_AsVoidPtr(index);
    Py_DECREF(index);
    if (!p && PyErr_Occurred()) throw Failed();
    return static_cast<cudaStream_t>(p);
}

// Sizes that pass 32 bits stop here, so no int below is cut short.
int narrow(int64_t v, const char* what) {
    if (v > INT_MAX) fail(PyExc_ValueError, std::string(what) + " does not fit 32 bits");
    return (int)v;
}

struct Pools {
    void *k, *v;
    const float *ks, *vs;
    int64_t nb, bs, hk, d;
};

// Both pools fp16 without scales, or both E4M3 codes with both scales.
Pools need_pools(Call& c, PyObject* ko, PyObject* vo, PyObject* kso, PyObject* vso) {
    if ((kso == Py_None) != (vso == Py_None)) fail(PyExc_ValueError, "k_scale and v_scale go together");
    const bool fp8 = kso != Py_None;
    const at::Tensor& k = c.need(ko, "k_pool", fp8 ? at::kByte : at::kHalf, 4);
    const at::Tensor& v = c.need(vo, "v_pool", fp8 ? at::kByte : at::kHalf, 4);
    need_shape(v, "v_pool", {k.size(0), k.size(1), k.size(2), k.size(3)});
    Pools p{k.data_ptr(), v.data_ptr(), nullptr, nullptr, k.size(0), k.size(1), k.size(2), k.size(3)};
    if (fp8) {
        const at::Tensor& ks = c.need(kso, "k_scale", at::kFloat, 1);
        const at::Tensor& vs = c.need(vso, "v_scale", at::kFloat, 1);
        need_shape(ks, "k_scale", {p.hk});
        need_shape(vs, "v_scale", {p.hk});
        p.ks = static_cast<const float*>(ks.data_ptr());
        p.vs = static_cast<const float*>(vs.data_ptr());
    }
    return p;
}

struct Rows {
    const int32_t *tables, *seq_lens, *q_start;
    int64_t rows, mbpr;
};

Rows need_rows(Call& c, PyObject* to, PyObject* so, PyObject* qo) {
    const at::Tensor& t = c.need(to, "block_tables", at::kInt, 2);
    const at::Tensor& s = c.need(so, "seq_lens", at::kInt, 1);
    const at::Tensor& q = c.need(qo, "q_start", at::kInt, 1);
    const int64_t rows = s.size(0);
    if (t.size(0) != rows) fail(PyExc_ValueError, "block_tables must have a row per seq_len");
    if (q.size(0) != rows + 1) fail(PyExc_ValueError, "q_start must have rows + 1 entries");
    return {static_cast<const int32_t*>(t.data_ptr()), static_cast<const int32_t*>(s.data_ptr()),
            static_cast<const int32_t*>(q.data_ptr()), rows, t.size(1)};
}

template <class F>
PyObject* guarded(const char* name, Py_ssize_t got, Py_ssize_t want, F&& body) {
    if (got != want) {
        PyErr_Format(PyExc_TypeError, "%s takes %zd arguments, got %zd", name, want, got);
        return nullptr;
    }
    try {
        return PyLong_FromLong(body());
    } catch (const Failed&) {
        return nullptr;
    } catch (const std::exception& e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
        return nullptr;
    }
}

// The arguments that the rotary appends share, a[0 .. 17], checked and unpacked; norms
// (a[18 .. 20]: q_weight, k_weight, eps) where `norm`.
int append_rotated(PyObject* const* a, bool norm) {
    Call c;
    const Pools p = need_pools(c, a[0], a[1], a[14], a[15]);
    const Rows r = need_rows(c, a[2], a[3], a[4]);
    int64_t sk = 0, sv = 0, sq = 0, hq = 0;
    const at::Tensor& k = c.tokens(a[5], "k_new", p.hk, p.d, &sk);
    const at::Tensor& v = c.tokens(a[6], "v_new", p.hk, p.d, &sv);
    const int64_t total = k.size(0);
    need_shape(v, "v_new", {total, p.hk, p.d});
    const at::Tensor& rates = c.need(a[7], "rates", at::kLong, 1);
    if ((a[10] == Py_None) != (a[11] == Py_None)) fail(PyExc_ValueError, "q and q_out go together");
    void *q = nullptr, *q_out = nullptr;
    if (a[10] != Py_None) {
        const at::Tensor& o = c.need(a[11], "q_out", at::kHalf, 3);
        hq = o.size(1);
        need_shape(o, "q_out", {total, hq, p.d});
        const at::Tensor& x = c.tokens(a[10], "q", hq, p.d, &sq);
        need_shape(x, "q", {total, hq, p.d});
        q = x.data_ptr();
        q_out = o.data_ptr();
    }
    const int32_t* pos = nullptr;
    if (a[12] != Py_None) {
        const at::Tensor& x = c.need(a[12], "rope_positions", at::kInt, 1);
        need_shape(x, "rope_positions", {total});
        pos = static_cast<const int32_t*>(x.data_ptr());
    }
    const void *qw = nullptr, *kw = nullptr;
    if (norm) {
        if (hq && a[18] == Py_None) fail(PyExc_ValueError, "q_weight goes with q");
        if (a[18] != Py_None) {
            const at::Tensor& x = c.need(a[18], "q_weight", at::kHalf, 1);
            need_shape(x, "q_weight", {p.d});
            qw = x.data_ptr();
        }
        const at::Tensor& x = c.need(a[19], "k_weight", at::kHalf, 1);
        need_shape(x, "k_weight", {p.d});
        kw = x.data_ptr();
    }
    auto* err = static_cast<int32_t*>(c.optional(a[16], "dev_err", at::kInt, 1));
    const c10::cuda::OptionalCUDAGuard guard(c10::Device(c10::kCUDA, c.device));
    const auto* turns = static_cast<const uint64_t*>(rates.data_ptr());
    const int rows = narrow(r.rows, "rows"), tokens = narrow(total, "tokens"), heads = narrow(hq, "q heads"),
              hk = narrow(p.hk, "kv heads"), d = narrow(p.d, "head_dim"), rot = narrow(2 * rates.size(0), "rot_dim"),
              layout = to_int(a[9]), bs = narrow(p.bs, "block_size"), mbpr = narrow(r.mbpr, "block_tables"),
              nb = narrow(p.nb, "blocks"), most = to_int(a[8]);
    const float mscale = to_float(a[13]);
    const cudaStream_t stream = to_stream(a[17], c.device);
    if (norm)
        return paged_kv_norm_rope_append(q_out, p.k, p.v, p.ks, p.vs, r.tables, r.seq_lens, r.q_start, pos, turns, q,
                                         k.data_ptr(), v.data_ptr(), qw, kw, to_float(a[20]), sq, sk, sv, rows,
                                         tokens, heads, hk, d, rot, layout, mscale, bs, mbpr, nb, most, err, stream);
    return paged_kv_rope_append(q_out, p.k, p.v, p.ks, p.vs, r.tables, r.seq_lens, r.q_start, pos, turns, q,
                                k.data_ptr(), v.data_ptr(), sq, sk, sv, rows, tokens, heads, hk, d, rot, layout,
                                mscale, bs, mbpr, nb, most, err, stream);
}

PyObject* rope_append(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded("rope_append", n, 18, [&]() -> int { return append_rotated(a, false); });
}

PyObject* norm_rope_append(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded("norm_rope_append", n, 21, [&]() -> int { return append_rotated(a, true); });
}

PyObject* tree_attention(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded("tree_attention", n, 15, [&]() -> int {
        Call c;
        const at::Tensor& out = c.need(a[0], "out", at::kHalf, 3);
        const at::Tensor& q = c.need(a[1], "q", at::kHalf, 3);
        need_shape(out, "out", {q.size(0), q.size(1), q.size(2)});
        const Pools p = need_pools(c, a[2], a[3], a[11], a[12]);
        const Rows r = need_rows(c, a[4], a[5], a[6]);
        const at::Tensor& ws = c.need(a[9], "workspace", at::kByte, 1);
        if (p.d != q.size(2))
            fail(PyExc_ValueError, "q has head_dim " + std::to_string(q.size(2)) + ", the pools " + std::to_string(p.d));
        const uint32_t* mask = nullptr;
        int64_t words = 0;
        if (a[10] != Py_None) {
            const at::Tensor& m = c.need(a[10], "mask", at::kInt, 2);
            words = m.size(1);
            need_shape(m, "mask", {q.size(0), words});
            mask = static_cast<const uint32_t*>(m.data_ptr());
        }
        auto* err = static_cast<int32_t*>(c.optional(a[13], "dev_err", at::kInt, 1));
        const c10::cuda::OptionalCUDAGuard guard(c10::Device(c10::kCUDA, c.device));
        return paged_attention_tree(
            out.data_ptr(), q.data_ptr(), p.k, p.v, p.ks, p.vs, r.tables, r.seq_lens, r.q_start, mask,
            narrow(words, "mask words"), narrow(r.rows, "rows"), narrow(q.size(0), "tokens"),
            narrow(q.size(1), "q heads"), narrow(p.hk, "kv heads"), narrow(p.d, "head_dim"),
            narrow(p.bs, "block_size"), to_float(a[7]), narrow(r.mbpr, "block_tables"), narrow(p.nb, "blocks"),
            to_int(a[8]), ws.data_ptr(), (size_t)ws.numel(), err, to_stream(a[14], c.device));
    });
}

PyObject* tree_commit(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded("tree_commit", n, 11, [&]() -> int {
        Call c;
        const at::Tensor& k0 = c.tensor(a[0], "k_pool");
        const at::ScalarType dt = k0.scalar_type();
        if (dt != at::kHalf && dt != at::kByte)
            fail(PyExc_TypeError, std::string("k_pool must be torch.float16 or torch.uint8, got ") + dtype_name(dt));
        const int64_t nd = k0.dim() == 5 ? 5 : 4;
        const at::Tensor& k = c.need(a[0], "k_pool", dt, nd);
        const at::Tensor& v = c.need(a[1], "v_pool", dt, nd);
        if (v.sizes() != k.sizes())
            fail(PyExc_ValueError, "v_pool must have shape " + shape_of(k.sizes()) + ", got " + shape_of(v.sizes()));
        const Rows r = need_rows(c, a[2], a[3], a[4]);
        const at::Tensor& path = c.need(a[5], "path", at::kInt, 2);
        const at::Tensor& lens = c.need(a[6], "path_lens", at::kInt, 1);
        if (path.size(0) != r.rows || lens.size(0) != r.rows)
            fail(PyExc_ValueError, "path and path_lens must have a row per seq_len");
        int32_t* fresh = nullptr;
        if (a[8] != Py_None) {
            const at::Tensor& x = c.need(a[8], "new_seq_lens", at::kInt, 1);
            need_shape(x, "new_seq_lens", {r.rows});
            fresh = static_cast<int32_t*>(x.data_ptr());
        }
        auto* err = static_cast<int32_t*>(c.optional(a[9], "dev_err", at::kInt, 1));
        const c10::cuda::OptionalCUDAGuard guard(c10::Device(c10::kCUDA, c.device));
        return paged_kv_tree_commit(
            k.data_ptr(), v.data_ptr(), r.tables, r.seq_lens, r.q_start, static_cast<const int32_t*>(path.data_ptr()),
            static_cast<const int32_t*>(lens.data_ptr()), fresh, nd == 5 ? narrow(k.size(0), "layers") : 1,
            narrow(r.rows, "rows"), narrow(path.size(1), "path"), narrow(k.size(nd - 2), "kv heads"),
            narrow(k.size(nd - 1), "head_dim"), dt == at::kHalf ? 2 : 1, narrow(k.size(nd - 3), "block_size"),
            narrow(r.mbpr, "block_tables"), narrow(k.size(nd - 4), "blocks"), to_int(a[7]), err,
            to_stream(a[10], c.device));
    });
}

// Running sums float [rows][heads][stride].
float* need_weights(Call& c, PyObject* o, int64_t rows, int64_t heads, int64_t* stride) {
    const at::Tensor& w = c.need(o, "weights", at::kFloat, 3);
    *stride = w.size(2);
    need_shape(w, "weights", {rows, heads, *stride});
    return static_cast<float*>(w.data_ptr());
}

PyObject* decode_weights(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded("decode_weights", n, 14, [&]() -> int {
        Call c;
        const at::Tensor& out = c.need(a[0], "out", at::kHalf, 3);
        const at::Tensor& q = c.need(a[2], "q", at::kHalf, 3);
        need_shape(out, "out", {q.size(0), q.size(1), q.size(2)});
        const Pools p = need_pools(c, a[3], a[4], a[10], a[11]);
        const at::Tensor& tables = c.need(a[5], "block_tables", at::kInt, 2);
        const at::Tensor& lens = c.need(a[6], "seq_lens", at::kInt, 1);
        const int64_t rows = q.size(0);
        need_shape(lens, "seq_lens", {rows});
        if (tables.size(0) != rows) fail(PyExc_ValueError, "block_tables must have a row per seq_len");
        if (p.d != q.size(2))
            fail(PyExc_ValueError, "q has head_dim " + std::to_string(q.size(2)) + ", the pools " + std::to_string(p.d));
        int64_t stride = 0;
        float* w = need_weights(c, a[1], rows, p.hk, &stride);
        const at::Tensor& ws = c.need(a[9], "workspace", at::kByte, 1);
        auto* err = static_cast<int32_t*>(c.optional(a[12], "dev_err", at::kInt, 1));
        const c10::cuda::OptionalCUDAGuard guard(c10::Device(c10::kCUDA, c.device));
        return paged_attention_decode_weights(
            out.data_ptr(), w, q.data_ptr(), p.k, p.v, p.ks, p.vs, static_cast<const int32_t*>(tables.data_ptr()),
            static_cast<const int32_t*>(lens.data_ptr()), narrow(rows, "rows"), narrow(q.size(1), "q heads"),
            narrow(p.hk, "kv heads"), narrow(p.d, "head_dim"), narrow(p.bs, "block_size"), to_float(a[7]),
            narrow(tables.size(1), "block_tables"), narrow(p.nb, "blocks"), to_int(a[8]), stride, ws.data_ptr(),
            (size_t)ws.numel(), err, to_stream(a[13], c.device));
    });
}

PyObject* prefill_weights(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded("prefill_weights", n, 13, [&]() -> int {
        Call c;
        const at::Tensor& q = c.need(a[1], "q", at::kHalf, 3);
        const bool fp8 = a[10] != Py_None;
        const at::Tensor& k = c.need(a[2], "k_pool", fp8 ? at::kByte : at::kHalf, 4);
        const int64_t hk = k.size(2), d = k.size(3);
        if (d != q.size(2))
            fail(PyExc_ValueError, "q has head_dim " + std::to_string(q.size(2)) + ", the pool " + std::to_string(d));
        const float* ks = nullptr;
        if (fp8) {
            const at::Tensor& x = c.need(a[10], "k_scale", at::kFloat, 1);
            need_shape(x, "k_scale", {hk});
            ks = static_cast<const float*>(x.data_ptr());
        }
        const Rows r = need_rows(c, a[3], a[4], a[5]);
        int64_t stride = 0;
        float* w = need_weights(c, a[0], r.rows, hk, &stride);
        const at::Tensor& ws = c.need(a[8], "workspace", at::kByte, 1);
        const int window = a[9] == Py_None ? INT_MAX : to_int(a[9]);
        auto* err = static_cast<int32_t*>(c.optional(a[11], "dev_err", at::kInt, 1));
        const c10::cuda::OptionalCUDAGuard guard(c10::Device(c10::kCUDA, c.device));
        return paged_attention_prefill_weights(
            w, q.data_ptr(), k.data_ptr(), ks, r.tables, r.seq_lens, r.q_start, narrow(r.rows, "rows"),
            narrow(q.size(0), "tokens"), narrow(q.size(1), "q heads"), narrow(hk, "kv heads"), narrow(d, "head_dim"),
            narrow(k.size(1), "block_size"), to_float(a[6]), window, narrow(r.mbpr, "block_tables"),
            narrow(k.size(0), "blocks"), to_int(a[7]), stride, ws.data_ptr(), (size_t)ws.numel(), err,
            to_stream(a[12], c.device));
    });
}

PyObject* evict(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded("evict", n, 17, [&]() -> int {
        Call c;
        const at::Tensor& k0 = c.tensor(a[0], "k_pool");
        const at::ScalarType dt = k0.scalar_type();
        if (dt != at::kHalf && dt != at::kByte)
            fail(PyExc_TypeError, std::string("k_pool must be torch.float16 or torch.uint8, got ") + dtype_name(dt));
        const int64_t nd = k0.dim() == 5 ? 5 : 4;
        const at::Tensor& k = c.need(a[0], "k_pool", dt, nd);
        const at::Tensor& v = c.need(a[1], "v_pool", dt, nd);
        if (v.sizes() != k.sizes())
            fail(PyExc_ValueError, "v_pool must have shape " + shape_of(k.sizes()) + ", got " + shape_of(v.sizes()));
        const at::Tensor& tables = c.need(a[2], "block_tables", at::kInt, 2);
        const at::Tensor& lens = c.need(a[3], "seq_lens", at::kInt, 1);
        const int64_t rows = lens.size(0), layers = nd == 5 ? k.size(0) : 1, hk = k.size(nd - 2);
        if (tables.size(0) != rows) fail(PyExc_ValueError, "block_tables must have a row per seq_len");
        // one layer's lists, or every layer's
        const at::Tensor& w = c.need(a[4], "weights", at::kFloat, nd - 1);
        const at::Tensor& pos = c.need(a[5], "token_pos", at::kInt, nd - 1);
        const int64_t stride = w.size(nd - 2);
        if ((nd == 5 && w.size(0) != layers) || w.size(nd - 4) != rows || w.size(nd - 3) != hk)
            fail(PyExc_ValueError, std::string("weights must be ") + (nd == 5 ? "[layers]" : "") +
                                       "[rows][kv_heads][stride], got " + shape_of(w.sizes()));
        auto same = [&](const at::Tensor& t, const char* name) {
            if (t.sizes() != w.sizes())
                fail(PyExc_ValueError, std::string(name) + " must have shape " + shape_of(w.sizes()) + ", got " + shape_of(t.sizes()));
        };
        same(pos, "token_pos");
        auto per_row = [&](PyObject* o, const char* name) -> int32_t* {
            if (o == Py_None) return nullptr;
            const at::Tensor& x = c.need(o, name, at::kInt, 1);
            need_shape(x, name, {rows});
            return static_cast<int32_t*>(x.data_ptr());
        };
        const int32_t* tracked = per_row(a[10], "tracked");
        const int32_t* next = per_row(a[11], "next_pos");
        if ((a[12] == Py_None) != (a[13] == Py_None)) fail(PyExc_ValueError, "weights_out and token_pos_out go together");
        float* w_out = static_cast<float*>(w.data_ptr());
        int32_t* pos_out = static_cast<int32_t*>(pos.data_ptr());
        if (a[12] != Py_None) {
            const at::Tensor& wo = c.need(a[12], "weights_out", at::kFloat, nd - 1);
            const at::Tensor& po = c.need(a[13], "token_pos_out", at::kInt, nd - 1);
            same(wo, "weights_out");
            same(po, "token_pos_out");
            w_out = static_cast<float*>(wo.data_ptr());
            pos_out = static_cast<int32_t*>(po.data_ptr());
        }
        int32_t* fresh = per_row(a[14], "new_seq_lens");
        auto* err = static_cast<int32_t*>(c.optional(a[15], "dev_err", at::kInt, 1));
        const c10::cuda::OptionalCUDAGuard guard(c10::Device(c10::kCUDA, c.device));
        return paged_kv_evict(
            k.data_ptr(), v.data_ptr(), static_cast<const int32_t*>(tables.data_ptr()),
            static_cast<const int32_t*>(lens.data_ptr()), static_cast<const float*>(w.data_ptr()),
            static_cast<const int32_t*>(pos.data_ptr()), tracked, next, w_out, pos_out, fresh, narrow(layers, "layers"),
            narrow(rows, "rows"), narrow(hk, "kv heads"), narrow(k.size(nd - 1), "head_dim"), dt == at::kHalf ? 2 : 1,
            narrow(k.size(nd - 3), "block_size"), narrow(tables.size(1), "block_tables"), narrow(k.size(nd - 4), "blocks"),
            to_int(a[7]), stride, to_int(a[6]), to_int(a[8]), to_int(a[9]), err, to_stream(a[16], c.device));
    });
}

template <class F>
PyCFunction as_function(F f) {
    return reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(f));
}

PyMethodDef methods[] = {
    {"rope_append", as_function(rope_append), METH_FASTCALL, nullptr},
    {"norm_rope_append", as_function(norm_rope_append), METH_FASTCALL, nullptr},
    {"tree_attention", as_function(tree_attention), METH_FASTCALL, nullptr},
    {"tree_commit", as_function(tree_commit), METH_FASTCALL, nullptr},
    {"decode_weights", as_function(decode_weights), METH_FASTCALL, nullptr},
    {"prefill_weights", as_function(prefill_weights), METH_FASTCALL, nullptr},
    {"evict", as_function(evict), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr},
};

PyModuleDef module_def = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__binding(void) { return PyModule_Create(&module_def); }
