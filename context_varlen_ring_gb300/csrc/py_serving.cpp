// py_serving.cpp -- the Python module `_serving`: argument checks, output
// allocation and the calls into libra.so for rotary positions, the cache
// append, paged attention, its keys' weights, eviction and the gated delta rule.
//
// These calls are made once a layer and decoding step, where the kernels take
// a few microseconds: the same checks in Python took 40 to 50 us a call on a
// Grace core, ten times the kernels' time.  Only torch's C++ tensor access is
// used; the work is in the library's C entries.
#include <Python.h>

#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/DynamicTypes.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cmath>
#include <string>
#include <vector>

#include "../../include/ra.h"

namespace {

struct Raised {};  // a Python exception is set

[[noreturn]] void raise(PyObject *type, const std::string &msg) {
    PyErr_SetString(type, msg.c_str());
    throw Raised{};
}
[[noreturn]] void value_error(const std::string &msg) { raise(PyExc_ValueError, msg); }

void check(ra_status st, const char *where) {
    if (st == RA_OK) return;
    PyObject *mod = PyImport_ImportModule("context_varlen_ring_gb300._lib");
    if (!mod) throw Raised{};
    PyObject *type = PyObject_GetAttrString(mod, "RaError");
    Py_DECREF(mod);
    if (!type) throw Raised{};
    PyObject *err = PyObject_CallFunction(type, "iss", (int)st, where, ra_last_error());
    if (err) PyErr_SetObject(type, err);
    Py_XDECREF(err);
    Py_DECREF(type);
    throw Raised{};
}

const at::Tensor &tensor(PyObject *o, const char *name) {
    if (!THPVariable_Check(o)) raise(PyExc_TypeError, std::string(name) + " must be a tensor");
    return THPVariable_Unpack(o);
}

int dtype_code(const at::Tensor &t) {
    if (t.scalar_type() == at::kBFloat16) return RA_BF16;
    if (t.scalar_type() == at::kFloat) return RA_FP32;
    raise(PyExc_TypeError, std::string("unsupported dtype ") + c10::toString(t.scalar_type()));
}

// A [T, H, d] tensor whose rows of H * d elements are contiguous; the row stride.
int64_t rows(const at::Tensor &x, const char *name, const at::Tensor *like = nullptr) {
    if (x.dim() != 3) value_error(std::string(name) + " must be [T, heads, d]");
    if (!x.is_cuda()) value_error("tensors must be on a CUDA device");
    if (like && (x.get_device() != like->get_device() || x.scalar_type() != like->scalar_type()))
        value_error(std::string(name) + " must have the device and dtype of the other tensors");
    const int64_t T = x.size(0), H = x.size(1), d = x.size(2);
    if ((d > 1 && x.stride(2) != 1) || (H > 1 && x.stride(1) != d))
        value_error(std::string(name) + ": the heads of a token must be contiguous");
    return T > 1 ? x.stride(0) : H * d;
}

const int32_t *index(const at::Tensor &x, const char *name, int64_t device) {
    if (x.scalar_type() != at::kInt) raise(PyExc_TypeError, std::string(name) + " must be int32");
    if (!x.is_cuda() || x.get_device() != device || !x.is_contiguous())
        value_error(std::string(name) + " must be a contiguous tensor on the device of the data");
    return static_cast<const int32_t *>(x.data_ptr());
}

// A host array of n values: a CPU tensor or anything with a buffer (numpy).
template <typename E>
struct Host {
    at::Tensor held;
    Py_buffer buf{};
    bool has_buf = false;
    const E *p = nullptr;
    int64_t n = 0;
    void take(PyObject *o, at::ScalarType type, const char *name) {
        if (THPVariable_Check(o)) {
            held = THPVariable_Unpack(o);
            if (held.scalar_type() != type || !held.is_contiguous() || !held.device().is_cpu())
                held = held.detach().to(at::kCPU, type).contiguous();
            if (held.dim() != 1) value_error(std::string(name) + " must be [n_pairs]");
            p = static_cast<const E *>(held.data_ptr());
            n = held.numel();
            return;
        }
        if (PyObject_GetBuffer(o, &buf, PyBUF_C_CONTIGUOUS | PyBUF_FORMAT) != 0) throw Raised{};
        has_buf = true;
        const char want = sizeof(E) == 8 ? 'd' : 'B';
        if (buf.ndim != 1 || buf.itemsize != (Py_ssize_t)sizeof(E) || !buf.format || buf.format[0] != want)
            value_error(std::string(name) + " must be [n_pairs] of " + (want == 'd' ? "float64" : "uint8"));
        p = static_cast<const E *>(buf.buf);
        n = buf.len / buf.itemsize;
    }
    ~Host() {
        if (has_buf) PyBuffer_Release(&buf);
    }
};

struct RopeArg {
    Host<double> freq;
    Host<uint8_t> axes;
    ra_rope c{};
    const int32_t *pos = nullptr;
    RopeArg(PyObject *pos_o, PyObject *freq_o, PyObject *axes_o, PyObject *adjacent, int64_t T, int64_t device) {
        freq.take(freq_o, at::kDouble, "inv_freq");
        if (axes_o != Py_None) {
            axes.take(axes_o, at::kByte, "axes");
            if (axes.n != freq.n) value_error("inv_freq and axes must be [n_pairs]");
        }
        const at::Tensor &ps = tensor(pos_o, "pos");
        pos = index(ps, "pos", device);
        if ((ps.dim() != 1 && ps.dim() != 2) || ps.size(-1) != T) value_error("pos must be [T] or [axes, T]");
        const int adj = PyObject_IsTrue(adjacent);
        if (adj < 0) throw Raised{};
        if (freq.n > 1 << 20) value_error("too many pairs");
        c = ra_rope{freq.p, axes.p, (int32_t)freq.n, ps.dim() == 2 ? (int32_t)ps.size(0) : 1, adj};
    }
};

struct On {  // the tensors' device is current, and their stream
    c10::cuda::CUDAGuard guard;
    void *stream;
    explicit On(int64_t device)
        : guard((c10::DeviceIndex)device),
          stream(c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)device).stream()) {}
};

// A new tensor straight from the allocator (the dispatcher's way there takes 0.5 us more).
at::Tensor fresh(at::IntArrayRef sizes, at::ScalarType type, const at::Tensor &like) {
    return at::Tensor(at::detail::empty_cuda(sizes, type, like.device(), std::nullopt));
}

at::Tensor output(PyObject *o, const at::Tensor &like, const char *name) {
    if (o == Py_None) return fresh(like.sizes(), like.scalar_type(), like);
    const at::Tensor &x = tensor(o, name);
    if (x.sizes() != like.sizes()) value_error(std::string(name) + " must have the shape of its input");
    return x;
}

ra_paged_kv paged(const at::Tensor &k, const at::Tensor &v) {
    if (k.dim() != 4 || v.sizes() != k.sizes()) value_error("k_cache and v_cache must be [pages, page_size, Hkv, d] alike");
    if (!k.is_cuda() || !v.is_cuda() || v.get_device() != k.get_device() || v.scalar_type() != k.scalar_type())
        value_error("k_cache and v_cache must be on one CUDA device, of one dtype");
    int64_t st[3];
    for (int i = 0; i < 3; ++i) {  // a dimension of one element has no stride that matters
        st[i] = k.size(i) == 1 ? 0 : k.stride(i);
        if (st[i] != (v.size(i) == 1 ? 0 : v.stride(i))) value_error("k_cache and v_cache must have the same strides");
    }
    if (k.size(3) > 1 && (k.stride(3) != 1 || v.stride(3) != 1)) value_error("the caches' heads must be contiguous");
    if (k.size(1) > INT32_MAX || k.size(2) > INT32_MAX || k.size(3) > INT32_MAX) value_error("bad cache shape");
    return ra_paged_kv{k.data_ptr(), v.data_ptr(), k.size(0), st[0], st[1], st[2],
                       (int32_t)k.size(1), (int32_t)k.size(2), (int32_t)k.size(3), dtype_code(k)};
}

struct Segments {
    const int32_t *table, *cu, *lens;
    int64_t width;
    int B;
    Segments(PyObject *table_o, PyObject *cu_o, PyObject *lens_o, int64_t device) {
        const at::Tensor &t = tensor(table_o, "page_table"), &c = tensor(cu_o, "cu_seqlens"),
                         &l = tensor(lens_o, "kv_lens");
        table = index(t, "page_table", device);
        cu = index(c, "cu_seqlens", device);
        lens = index(l, "kv_lens", device);
        if (t.dim() != 2 || t.size(0) != l.numel() || c.numel() != l.numel() + 1 || l.numel() > INT32_MAX)
            value_error("page_table [B, width], cu_seqlens [B + 1] and kv_lens [B] must agree");
        width = t.size(1);
        B = (int)l.numel();
    }
};

PyObject *pair(at::Tensor a, at::Tensor b) {
    PyObject *x = THPVariable_Wrap(std::move(a));
    PyObject *y = b.defined() ? THPVariable_Wrap(std::move(b)) : Py_NewRef(Py_None);
    PyObject *t = x && y ? PyTuple_Pack(2, x, y) : nullptr;
    Py_XDECREF(x);
    Py_XDECREF(y);
    return t;
}

void arity(Py_ssize_t n, Py_ssize_t want) {
    if (n != want) raise(PyExc_TypeError, "wrong number of arguments");
}

int int_of(int64_t v, const char *name) {
    if (v > INT32_MAX) value_error(std::string(name) + " is too large");
    return (int)v;
}

// (backward, q, k, pos, inv_freq, axes, adjacent, q_out, k_out)
PyObject *rope(PyObject *const *a, Py_ssize_t n) {
    arity(n, 9);
    const bool bwd = a[0] == Py_True;
    const at::Tensor &q = tensor(a[1], "q");
    const int64_t qs = rows(q, "q");
    const int64_t T = q.size(0), d = q.size(2), dev = q.get_device();
    const int dt = dtype_code(q);
    int64_t ks = 0, kos = 0;
    int hk = 0;
    const void *kp = nullptr;
    if (a[2] != Py_None) {
        const at::Tensor &k = tensor(a[2], "k");
        ks = rows(k, "k", &q);
        if (k.size(0) != T || k.size(2) != d) value_error("k must have q's tokens and head size");
        hk = int_of(k.size(1), "k");
        kp = k.data_ptr();
    } else if (a[8] != Py_None) {
        value_error("k_out without k");
    }
    RopeArg r(a[3], a[4], a[5], a[6], T, dev);
    On on(dev);
    at::Tensor qo = output(a[7], q, "q_out"), ko;
    const int64_t qos = rows(qo, "q_out", &q);
    if (a[2] != Py_None) {
        ko = output(a[8], THPVariable_Unpack(a[2]), "k_out");
        kos = rows(ko, "k_out", &q);
    }
    check((bwd ? ra_rope_bwd : ra_rope_fwd)(q.data_ptr(), kp, qo.data_ptr(), ko.defined() ? ko.data_ptr() : nullptr, dt,
                                            T, int_of(q.size(1), "q"), hk, int_of(d, "d"), qs, ks, qos, kos, r.pos,
                                            &r.c, on.stream),
          bwd ? "ra_rope_bwd" : "ra_rope_fwd");
    return pair(std::move(qo), std::move(ko));
}

// (k, v, k_cache, v_cache, page_table, cu_seqlens, kv_lens, q, pos, inv_freq, axes, adjacent, q_out)
PyObject *append(PyObject *const *a, Py_ssize_t n) {
    arity(n, 13);
    const at::Tensor &k = tensor(a[0], "k"), &v = tensor(a[1], "v");
    const int64_t ks = rows(k, "k"), vs = rows(v, "v", &k), T = k.size(0), d = k.size(2), dev = k.get_device();
    const at::Tensor &kc = tensor(a[2], "k_cache"), &vc = tensor(a[3], "v_cache");
    const ra_paged_kv cache = paged(kc, vc);
    if (v.sizes() != k.sizes() || k.size(1) != cache.Hkv || d != cache.d)
        value_error("k and v must be [T, Hkv, d] with the cache's heads");
    if (kc.get_device() != dev || kc.scalar_type() != k.scalar_type())
        value_error("the cache must have the device and dtype of k");
    const Segments s(a[4], a[5], a[6], dev);
    const bool has_q = a[7] != Py_None;
    if (!has_q && a[12] != Py_None) value_error("q_out without q");
    const bool turn = a[9] != Py_None;
    if (turn && a[8] == Py_None) value_error("inv_freq without pos");
    int64_t qs = 0, qos = 0;
    int hq = 0;
    const void *qp = nullptr;
    if (has_q) {
        const at::Tensor &q = tensor(a[7], "q");
        qs = rows(q, "q", &k);
        if (q.size(0) != T || q.size(2) != d) value_error("q must have k's tokens and head size");
        hq = int_of(q.size(1), "q");
        qp = q.data_ptr();
    }
    On on(dev);
    at::Tensor qo;
    if (has_q) {
        qo = output(a[12], THPVariable_Unpack(a[7]), "q_out");
        qos = rows(qo, "q_out", &k);
    }
    auto call = [&](const int32_t *pos, const ra_rope *r) {
        check(ra_kv_cache_append(k.data_ptr(), v.data_ptr(), ks, vs, T, &cache, s.table, s.width, s.cu, s.lens, s.B, qp,
                                 qo.defined() ? qo.data_ptr() : nullptr, hq, qs, qos, pos, r, on.stream),
              "ra_kv_cache_append");
    };
    if (turn) {
        const RopeArg r(a[8], a[9], a[10], a[11], T, dev);
        call(r.pos, &r.c);
    } else {
        call(nullptr, nullptr);
    }
    return qo.defined() ? THPVariable_Wrap(std::move(qo)) : Py_NewRef(Py_None);
}

// (q, k_cache, v_cache, page_table, cu_seqlens_q, kv_lens, prefix_table, prefix_lens, prefix_groups, causal, scale,
//  max_q_len, out, lse, out_dtype, workspace)
PyObject *attn(PyObject *const *a, Py_ssize_t n) {
    arity(n, 16);
    const at::Tensor &q = tensor(a[0], "q");
    const int64_t qs = rows(q, "q"), T = q.size(0), d = q.size(2), dev = q.get_device();
    const int hq = int_of(q.size(1), "q");
    const at::Tensor &kc = tensor(a[1], "k_cache"), &vc = tensor(a[2], "v_cache");
    const ra_paged_kv cache = paged(kc, vc);
    if (kc.get_device() != dev || kc.scalar_type() != q.scalar_type() || cache.d != d)
        value_error("the cache must have the device, dtype and head size of q");
    const Segments s(a[3], a[4], a[5], dev);
    const bool some = a[6] != Py_None || a[7] != Py_None || a[8] != Py_None;
    if (some && (a[6] == Py_None || a[7] == Py_None || a[8] == Py_None))
        value_error("prefix_table, prefix_lens and prefix_groups go together");
    const Segments *pre = nullptr;
    alignas(Segments) char room[sizeof(Segments)];
    if (some) pre = new (room) Segments(a[6], a[8], a[7], dev);
    const int causal = PyObject_IsTrue(a[9]);
    if (causal < 0) throw Raised{};
    double scale = 1.0 / std::sqrt((double)d);
    if (a[10] != Py_None) {
        scale = PyFloat_AsDouble(a[10]);
        if (scale == -1.0 && PyErr_Occurred()) throw Raised{};
    }
    long long most = 0;
    if (a[11] != Py_None) {
        most = PyLong_AsLongLong(a[11]);
        if (most == -1 && PyErr_Occurred()) throw Raised{};
        most = std::min<long long>(std::max<long long>(most, 0), INT32_MAX);
    }
    at::ScalarType ot = q.scalar_type();
    const bool has_type = a[14] != Py_None;
    if (has_type) {
        if (!THPDtype_Check(a[14])) raise(PyExc_TypeError, "out_dtype must be a torch.dtype");
        ot = reinterpret_cast<THPDtype *>(a[14])->scalar_type;
    }
    On on(dev);
    at::Tensor out, lse, ws;
    if (a[12] == Py_None) {
        out = fresh(q.sizes(), ot, q);
    } else {
        out = tensor(a[12], "out");
        if (out.sizes() != q.sizes() || !out.is_contiguous() || !out.is_cuda() || out.get_device() != dev)
            value_error("out must be a contiguous [T, Hq, d] tensor on q's device");
        if (has_type && out.scalar_type() != ot) value_error("out does not have out_dtype");
    }
    if (a[13] == Py_None) {
        lse = fresh({hq, T}, at::kFloat, q);
    } else {
        lse = tensor(a[13], "lse");
        if (lse.dim() != 2 || lse.size(0) != hq || lse.size(1) != T || !lse.is_contiguous() || !lse.is_cuda() ||
            lse.get_device() != dev || lse.scalar_type() != at::kFloat)
            value_error("lse must be a contiguous fp32 [Hq, T] tensor on q's device");
    }
    const int groups = pre ? pre->B : 0;
    if (a[15] == Py_None) {
        const size_t need = ra_paged_attn_workspace_bytes(T, s.B, groups, hq, cache.Hkv, (int)d, cache.dtype, (int)most);
        ws = fresh({(int64_t)std::max<size_t>(need, 256)}, at::kByte, q);
    } else {
        ws = tensor(a[15], "workspace");
        if (!ws.is_contiguous() || !ws.is_cuda() || ws.get_device() != dev)
            value_error("workspace must be a contiguous tensor on q's device");
    }
    check(ra_paged_attn_fwd(q.data_ptr(), qs, T, hq, &cache, s.table, s.width, s.cu, s.lens, s.B,
                            pre ? pre->table : nullptr, pre ? pre->width : 0, pre ? pre->lens : nullptr,
                            pre ? pre->cu : nullptr, groups, causal, (int)most, (float)scale, out.data_ptr(),
                            dtype_code(out), static_cast<float *>(lse.data_ptr()), ws.data_ptr(), ws.nbytes(),
                            on.stream),
          "ra_paged_attn_fwd");
    return pair(std::move(out), std::move(lse));
}

// Weights [pages, page_size, Hkv] of a cache's keys.
ra_paged_weights paged_weights(const at::Tensor &w, const ra_paged_kv &cache, int64_t dev) {
    if (w.scalar_type() != at::kFloat) raise(PyExc_TypeError, "weights must be float32");
    if (w.dim() != 3 || w.size(0) != cache.n_pages || w.size(1) != cache.page_size || w.size(2) != cache.Hkv)
        value_error("weights must be [pages, page_size, Hkv] of the cache");
    if (!w.is_cuda() || w.get_device() != dev) value_error("weights must be on the device of the cache");
    return ra_paged_weights{static_cast<float *>(w.data_ptr()), w.stride(0), w.stride(1), w.stride(2)};
}

// (q, k_cache, page_table, cu_seqlens_q, kv_lens, lse, weights, prefix_table, prefix_lens, prefix_groups, causal, scale,
//  max_q_len)
PyObject *key_weights(PyObject *const *a, Py_ssize_t n) {
    arity(n, 13);
    const at::Tensor &q = tensor(a[0], "q");
    const int64_t qs = rows(q, "q"), T = q.size(0), d = q.size(2), dev = q.get_device();
    const int hq = int_of(q.size(1), "q");
    const at::Tensor &kc = tensor(a[1], "k_cache"), &lse = tensor(a[5], "lse"), &w = tensor(a[6], "weights");
    const ra_paged_kv cache = paged(kc, kc);
    if (kc.get_device() != dev || kc.scalar_type() != q.scalar_type() || cache.d != d)
        value_error("the cache must have the device, dtype and head size of q");
    const ra_paged_weights pw = paged_weights(w, cache, dev);
    if (lse.dim() != 2 || lse.size(0) != hq || lse.size(1) != T || !lse.is_contiguous() || !lse.is_cuda() ||
        lse.get_device() != dev || lse.scalar_type() != at::kFloat)
        value_error("lse must be a contiguous fp32 [Hq, T] tensor on q's device");
    const Segments s(a[2], a[3], a[4], dev);
    const bool some = a[7] != Py_None || a[8] != Py_None || a[9] != Py_None;
    if (some && (a[7] == Py_None || a[8] == Py_None || a[9] == Py_None))
        value_error("prefix_table, prefix_lens and prefix_groups go together");
    const Segments *pre = nullptr;
    alignas(Segments) char room[sizeof(Segments)];
    if (some) pre = new (room) Segments(a[7], a[9], a[8], dev);
    const int causal = PyObject_IsTrue(a[10]);
    if (causal < 0) throw Raised{};
    double scale = 1.0 / std::sqrt((double)d);
    if (a[11] != Py_None) {
        scale = PyFloat_AsDouble(a[11]);
        if (scale == -1.0 && PyErr_Occurred()) throw Raised{};
    }
    long long most = 0;
    if (a[12] != Py_None) {
        most = PyLong_AsLongLong(a[12]);
        if (most == -1 && PyErr_Occurred()) throw Raised{};
        most = std::min<long long>(std::max<long long>(most, 0), INT32_MAX);
    }
    On on(dev);
    check(ra_paged_attn_key_weights(q.data_ptr(), qs, T, hq, &cache, &pw, s.table, s.width, s.cu, s.lens, s.B,
                                    pre ? pre->table : nullptr, pre ? pre->width : 0, pre ? pre->lens : nullptr,
                                    pre ? pre->cu : nullptr, pre ? pre->B : 0, causal, (int)most, (float)scale,
                                    static_cast<const float *>(lse.data_ptr()), on.stream),
          "ra_paged_attn_key_weights");
    return Py_NewRef(a[6]);
}

// (k_cache, v_cache, weights, page_table, kv_lens, keep, keep_lens, sinks, recent, per_head, out_table, new_lens, kept)
PyObject *evict(PyObject *const *a, Py_ssize_t n) {
    arity(n, 13);
    const at::Tensor &kc = tensor(a[0], "k_cache"), &vc = tensor(a[1], "v_cache");
    const ra_paged_kv cache = paged(kc, vc);
    const int64_t dev = kc.get_device();
    const ra_paged_weights pw = paged_weights(tensor(a[2], "weights"), cache, dev);
    const at::Tensor &table = tensor(a[3], "page_table"), &lens = tensor(a[4], "kv_lens");
    const int32_t *tp = index(table, "page_table", dev), *lp = index(lens, "kv_lens", dev);
    if (table.dim() != 2 || lens.dim() != 1 || table.size(0) != lens.numel() || lens.numel() > INT32_MAX)
        value_error("page_table [B, width] and kv_lens [B] must agree");
    const int B = (int)lens.numel();
    long long num[3];
    const char *names[3] = {"keep", "sinks", "recent"};
    PyObject *const given[3] = {a[5], a[7], a[8]};
    for (int i = 0; i < 3; ++i) {
        num[i] = PyLong_AsLongLong(given[i]);
        if (num[i] == -1 && PyErr_Occurred()) throw Raised{};
        if (num[i] < 0 || num[i] > INT32_MAX) value_error(std::string(names[i]) + " must be in [0, 2^31)");
    }
    const int32_t *each = nullptr, *op = nullptr;
    int64_t ow = 0;
    if (a[6] != Py_None) {
        const at::Tensor &x = tensor(a[6], "keep_lens");
        each = index(x, "keep_lens", dev);
        if (x.dim() != 1 || x.numel() != B) value_error("keep_lens must be [B]");
    }
    const int per_head = PyObject_IsTrue(a[9]);
    if (per_head < 0) throw Raised{};
    if (a[10] != Py_None) {
        const at::Tensor &x = tensor(a[10], "out_table");
        op = index(x, "out_table", dev);
        if (x.dim() != 2 || x.size(0) != B) value_error("out_table must be [B, width]");
        ow = x.size(1);
        static const int32_t none = 0;
        if (!op) op = &none;  // (no entries: nothing is read, nothing is kept)
    }
    On on(dev);
    at::Tensor left, kept;
    const int64_t H = per_head ? cache.Hkv : 1;
    if (a[11] == Py_None) {
        left = fresh({B}, at::kInt, kc);
    } else {
        left = tensor(a[11], "new_lens");
        index(left, "new_lens", dev);
        if (left.dim() != 1 || left.numel() != B) value_error("new_lens must be [B]");
    }
    if (a[12] == Py_None) {
        kept = fresh({B, H, num[0]}, at::kInt, kc);
    } else {
        kept = tensor(a[12], "kept");
        index(kept, "kept", dev);
        if (kept.dim() != 3 || kept.size(0) != B || kept.size(1) != H || kept.size(2) != num[0])
            value_error("kept must be [B, Hkv (1 without per_head), keep]");
    }
    check(ra_kv_cache_evict(&cache, &pw, tp, table.size(1), lp, B, (int)num[0], each, (int)num[1], (int)num[2], per_head, op,
                            ow, static_cast<int32_t *>(left.data_ptr()), static_cast<int32_t *>(kept.data_ptr()),
                            on.stream),
          "ra_kv_cache_evict");
    return pair(std::move(left), std::move(kept));
}

// The gated delta rule's inputs: q, k [T, Hk, dk], v [T, Hv, dv], g, beta fp32 [T, Hv].
struct DeltaArg {
    ra_delta c{};
    int64_t dev;
    const at::Tensor &q, &k, &v;
    DeltaArg(PyObject *q_o, PyObject *k_o, PyObject *v_o, PyObject *g_o, PyObject *b_o, PyObject *scale_o)
        : q(tensor(q_o, "q")), k(tensor(k_o, "k")), v(tensor(v_o, "v")) {
        c.q_stride = rows(q, "q");
        dev = q.get_device();
        c.k_stride = rows(k, "k", &q);
        c.v_stride = rows(v, "v", &q);
        if (k.sizes() != q.sizes() || v.size(0) != q.size(0))
            value_error("q and k must be [T, Hk, dk] and v [T, Hv, dv] of the same tokens");
        c.T = q.size(0);
        c.Hk = int_of(q.size(1), "q");
        c.Hv = int_of(v.size(1), "v");
        c.dk = int_of(q.size(2), "q");
        c.dv = int_of(v.size(2), "v");
        c.dtype = dtype_code(q);
        c.q = q.data_ptr();
        c.k = k.data_ptr();
        c.v = v.data_ptr();
        c.g = gate(g_o, "g");
        c.beta = gate(b_o, "beta");
        double scale = 1.0 / std::sqrt((double)c.dk);
        if (scale_o != Py_None) {
            scale = PyFloat_AsDouble(scale_o);
            if (scale == -1.0 && PyErr_Occurred()) throw Raised{};
        }
        c.scale = (float)scale;
    }
    const float *gate(PyObject *o, const char *name) {
        const at::Tensor &x = tensor(o, name);
        if (x.scalar_type() != at::kFloat) raise(PyExc_TypeError, std::string(name) + " must be float32");
        if (x.dim() != 2 || x.size(0) != c.T || x.size(1) != c.Hv || !x.is_contiguous() || !x.is_cuda() ||
            x.get_device() != dev)
            value_error(std::string(name) + " must be a contiguous [T, Hv] tensor on the device of q");
        return static_cast<const float *>(x.data_ptr());
    }
    // fp32 [n, Hv, dk, dv] (n < 0: any number)
    float *states(const at::Tensor &x, const char *name, int64_t n) {
        if (x.scalar_type() != at::kFloat) raise(PyExc_TypeError, std::string(name) + " must be float32");
        if (x.dim() != 4 || (n >= 0 && x.size(0) != n) || x.size(1) != c.Hv || x.size(2) != c.dk || x.size(3) != c.dv ||
            !x.is_contiguous() || !x.is_cuda() || x.get_device() != dev)
            value_error(std::string(name) + " must be a contiguous [states, Hv, dk, dv] tensor on the device of q");
        return static_cast<float *>(x.data_ptr());
    }
    void segments(PyObject *cu_o) {
        const at::Tensor &cu = tensor(cu_o, "cu_seqlens");
        c.cu_seqlens = index(cu, "cu_seqlens", dev);
        if (cu.dim() != 1 || cu.numel() < 1 || cu.numel() > INT32_MAX) value_error("cu_seqlens must be [N + 1]");
        c.N = (int)cu.numel() - 1;
    }
    // slots [N], into a pool of n states
    void places(PyObject *slots_o, int64_t n) {
        c.n_slots = n;
        if (slots_o == Py_None) {
            if (n != c.N) value_error("without slots there must be one state for each sequence");
            return;
        }
        const at::Tensor &s = tensor(slots_o, "slots");
        c.slots = index(s, "slots", dev);
        if (s.dim() != 1 || s.numel() != c.N) value_error("slots must be [N], one for each sequence");
    }
};

at::Tensor scratch(PyObject *o, const DeltaArg &d, int bwd) {
    if (o == Py_None) {
        const size_t need = ra_delta_rule_workspace_bytes(d.c.T, d.c.N, d.c.Hk, d.c.Hv, d.c.dk, d.c.dv, d.c.dtype, bwd);
        return fresh({(int64_t)std::max<size_t>(need, 256)}, at::kByte, d.q);
    }
    const at::Tensor &ws = tensor(o, "workspace");
    if (!ws.is_contiguous() || !ws.is_cuda() || ws.get_device() != d.dev)
        value_error("workspace must be a contiguous tensor on q's device");
    return ws;
}

// (q, k, v, g, beta, cu_seqlens, state, slots, state_out, final_state, scale, out, workspace)
PyObject *delta_fwd(PyObject *const *a, Py_ssize_t n) {
    arity(n, 13);
    DeltaArg d(a[0], a[1], a[2], a[3], a[4], a[10]);
    d.segments(a[5]);
    const int want = PyObject_IsTrue(a[9]);
    if (want < 0) throw Raised{};
    On on(d.dev);
    at::Tensor out, last;
    int64_t pool = -1;
    if (a[6] != Py_None) {
        const at::Tensor &s = tensor(a[6], "state");
        d.c.state = d.states(s, "state", -1);
        pool = s.size(0);
    }
    if (a[8] != Py_None) {
        last = tensor(a[8], "state_out");
        d.states(last, "state_out", pool);
        pool = last.size(0);
    } else if (want) {
        if (a[7] != Py_None) value_error("final states at slots need state_out (it may be state)");
        if (pool >= 0 && pool != d.c.N) value_error("without slots there must be one state for each sequence");
        last = fresh({d.c.N, d.c.Hv, d.c.dk, d.c.dv}, at::kFloat, d.q);
        pool = d.c.N;
    }
    if (pool >= 0)
        d.places(a[7], pool);
    else if (a[7] != Py_None)
        value_error("slots without state or state_out");
    if (a[11] == Py_None) {
        out = fresh(d.v.sizes(), d.q.scalar_type(), d.q);
    } else {
        out = tensor(a[11], "out");
        if (out.sizes() != d.v.sizes() || !out.is_contiguous() || !out.is_cuda() || out.get_device() != d.dev ||
            out.scalar_type() != d.q.scalar_type())
            value_error("out must be a contiguous [T, Hv, dv] tensor of q's dtype and device");
    }
    const at::Tensor ws = scratch(a[12], d, 0);
    check(ra_delta_rule_fwd(&d.c, out.data_ptr(), last.defined() ? static_cast<float *>(last.data_ptr()) : nullptr,
                            ws.data_ptr(), ws.nbytes(), on.stream),
          "ra_delta_rule_fwd");
    return pair(std::move(out), std::move(last));
}

// (dout, q, k, v, g, beta, cu_seqlens, state, slots, dstate, scale, workspace)
PyObject *delta_bwd(PyObject *const *a, Py_ssize_t n) {
    arity(n, 12);
    DeltaArg d(a[1], a[2], a[3], a[4], a[5], a[10]);
    d.segments(a[6]);
    const at::Tensor &dout = tensor(a[0], "dout");
    const int64_t stride = rows(dout, "dout", &d.q);
    if (dout.sizes() != d.v.sizes()) value_error("dout must be [T, Hv, dv]");
    On on(d.dev);
    at::Tensor g[6];
    float *last = nullptr;
    if (a[7] != Py_None) {
        const at::Tensor &s = tensor(a[7], "state");
        d.c.state = d.states(s, "state", -1);
        d.places(a[8], s.size(0));
        g[5] = fresh({d.c.N, d.c.Hv, d.c.dk, d.c.dv}, at::kFloat, d.q);
    } else if (a[8] != Py_None) {
        value_error("slots without state");
    }
    if (a[9] != Py_None) last = d.states(tensor(a[9], "dstate"), "dstate", d.c.N);
    const auto type = d.q.scalar_type();
    g[0] = fresh(d.q.sizes(), type, d.q);
    g[1] = fresh(d.q.sizes(), type, d.q);
    g[2] = fresh(d.v.sizes(), type, d.q);
    g[3] = fresh({d.c.T, d.c.Hv}, at::kFloat, d.q);
    g[4] = fresh({d.c.T, d.c.Hv}, at::kFloat, d.q);
    const at::Tensor ws = scratch(a[11], d, 1);
    check(ra_delta_rule_bwd(&d.c, dout.data_ptr(), stride, last, g[0].data_ptr(), g[1].data_ptr(), g[2].data_ptr(),
                            static_cast<float *>(g[3].data_ptr()), static_cast<float *>(g[4].data_ptr()),
                            g[5].defined() ? static_cast<float *>(g[5].data_ptr()) : nullptr, ws.data_ptr(), ws.nbytes(),
                            on.stream),
          "ra_delta_rule_bwd");
    PyObject *t = PyTuple_New(6);
    if (!t) throw Raised{};
    for (int i = 0; i < 6; ++i) {
        PyObject *x = g[i].defined() ? THPVariable_Wrap(std::move(g[i])) : Py_NewRef(Py_None);
        if (!x) {
            Py_DECREF(t);
            throw Raised{};
        }
        PyTuple_SET_ITEM(t, i, x);
    }
    return t;
}

// (q, k, v, g, beta, state, slots, scale, out)
PyObject *delta_step(PyObject *const *a, Py_ssize_t n) {
    arity(n, 9);
    DeltaArg d(a[0], a[1], a[2], a[3], a[4], a[7]);
    if (d.c.T > INT32_MAX) value_error("too many sequences");
    d.c.N = (int)d.c.T;
    const at::Tensor &s = tensor(a[5], "state");
    float *state = d.states(s, "state", -1);
    d.places(a[6], s.size(0));
    On on(d.dev);
    at::Tensor out;
    if (a[8] == Py_None) {
        out = fresh(d.v.sizes(), d.q.scalar_type(), d.q);
    } else {
        out = tensor(a[8], "out");
        if (out.sizes() != d.v.sizes() || !out.is_contiguous() || !out.is_cuda() || out.get_device() != d.dev ||
            out.scalar_type() != d.q.scalar_type())
            value_error("out must be a contiguous [B, Hv, dv] tensor of q's dtype and device");
    }
    check(ra_delta_rule_step(&d.c, state, out.data_ptr(), on.stream), "ra_delta_rule_step");
    return THPVariable_Wrap(std::move(out));
}

template <PyObject *(*F)(PyObject *const *, Py_ssize_t)>
PyObject *entry(PyObject *, PyObject *const *args, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    try {
        return F(args, n);
    } catch (const Raised &) {
        return nullptr;
    }
    END_HANDLE_TH_ERRORS
}

PyMethodDef methods[] = {
    {"rope", (PyCFunction)(void *)entry<rope>, METH_FASTCALL, nullptr},
    {"append", (PyCFunction)(void *)entry<append>, METH_FASTCALL, nullptr},
    {"attn", (PyCFunction)(void *)entry<attn>, METH_FASTCALL, nullptr},
    {"key_weights", (PyCFunction)(void *)entry<key_weights>, METH_FASTCALL, nullptr},
    {"evict", (PyCFunction)(void *)entry<evict>, METH_FASTCALL, nullptr},
    {"delta_fwd", (PyCFunction)(void *)entry<delta_fwd>, METH_FASTCALL, nullptr},
    {"delta_bwd", (PyCFunction)(void *)entry<delta_bwd>, METH_FASTCALL, nullptr},
    {"delta_step", (PyCFunction)(void *)entry<delta_step>, METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_serving", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__serving(void) { return PyModule_Create(&module); }
