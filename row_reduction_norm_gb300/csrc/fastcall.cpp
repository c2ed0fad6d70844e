// fastcall.cpp -- the Python calls of the rotary, append, dropout, embedding,
// log probability and clipping operators without Python's own cost: a CPython
// module that takes torch tensors, makes the checks of api.py on them, and calls
// the C ABI on the current stream.
//
// These kernels take two microseconds for a decode step while the checks, the
// argument conversion and the allocations of a call through Python objects and
// ctypes take seven to thirty.  Each function here takes what the api.py
// function of its name takes, by position; it returns that function's result,
// or None when anything about the arguments is out of the ordinary (a stream
// given, another device current, a wrong shape or type, a tensor subclass):
// api.py then goes its own way, which is also where every refusal is worded.
// A status of the C ABI other than RMSNORM_OK comes back as an int.
//
// Nothing is computed and nothing is kept here; the C ABI's addresses are
// handed over once by bind().
//
// Arguments are read with the interpreter's lock held; allocations and the C
// ABI's calls are made without it, as torch's and ctypes' are: either may block
// (a full launch queue, an allocator's own lock), and what they wait for may
// need another Python thread.
#include <Python.h>

#include <ATen/ATen.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/core/Allocator.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cstring>
#include <vector>

#include "rmsnorm.h"

namespace {

decltype(&rmsnorm_qk_rope_fwd) qk_rope_fwd;
decltype(&rmsnorm_qk_rope_bwd) qk_rope_bwd;
decltype(&rmsnorm_qk_rope_bwd_workspace_bytes) qk_rope_bwd_workspace_bytes;
decltype(&rmsnorm_qkv_append) qkv_append_fn;
decltype(&rmsnorm_dropout_fwd) dropout_fwd;
decltype(&rmsnorm_bwd) norm_bwd;
decltype(&rmsnorm_bwd_workspace_bytes) bwd_workspace_bytes;
decltype(&rmsnorm_dropout_bwd) dropout_bwd;
decltype(&rmsnorm_embedding_fwd) embedding_fwd;
decltype(&rmsnorm_embedding_bwd) embedding_bwd;
decltype(&rmsnorm_embedding_bwd_workspace_bytes) embedding_bwd_workspace_bytes;
decltype(&rmsnorm_logprobs_fwd) logprobs_fwd;
decltype(&rmsnorm_logprobs_bwd) logprobs_bwd;
decltype(&rmsnorm_grad_norm) norm_of_grads;
decltype(&rmsnorm_clip_grads) clip_grads;
decltype(&rmsnorm_grad_norm_workspace_bytes) grad_norm_workspace_bytes;

// Thrown (and caught in this file) to leave a call to api.py.
struct Elsewhere {};

void need(bool ok) {
    if (!ok) throw Elsewhere();
}

const at::Tensor &tensor(PyObject *o) {
    need(THPVariable_CheckExact(o));
    const at::Tensor &t = THPVariable_Unpack(o);
    need(t.defined() && t.is_cuda() && t.layout() == at::kStrided);
    return t;
}

int64_t whole(PyObject *o) {
    need(PyLong_CheckExact(o));
    int over = 0;
    const long long v = PyLong_AsLongLongAndOverflow(o, &over);
    need(over == 0);
    return (int64_t)v;
}

int32_t count(PyObject *o) {
    const int64_t v = whole(o);
    need(v >= 0 && v <= INT32_MAX);
    return (int32_t)v;
}

float real(PyObject *o) {
    if (PyFloat_CheckExact(o)) return (float)PyFloat_AS_DOUBLE(o);
    return (float)whole(o);
}

bool truth(PyObject *o) {
    need(o == Py_True || o == Py_False);
    return o == Py_True;
}

int code_of(const at::Tensor &t) {
    if (t.scalar_type() == at::kBFloat16) return RMSNORM_BF16;
    need(t.scalar_type() == at::kFloat);
    return RMSNORM_F32;
}

// The device of the call, which has to be the current one.
struct Where {
    int dev;
    explicit Where(const at::Tensor &t) : dev(t.get_device()) { need(dev >= 0 && c10::cuda::current_device() == dev); }
    rmsnorm_stream_t stream() const {
        return reinterpret_cast<rmsnorm_stream_t>(c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)dev).stream());
    }
    void same(const at::Tensor &t, at::ScalarType type) const {
        need(t.get_device() == dev && t.scalar_type() == type);
    }
};

// Address of a contiguous [size] tensor, or NULL for None.
void *vector(PyObject *o, int64_t size, at::ScalarType type, const Where &w) {
    if (o == Py_None) return nullptr;
    const at::Tensor &t = tensor(o);
    w.same(t, type);
    need(t.dim() == 1 && t.size(0) == size && (size <= 1 || t.stride(0) == 1));
    return t.data_ptr();
}

// Token stride of a [tokens, >= width] tensor of packed heads.
int64_t head_rows(const at::Tensor &t, int64_t width, int64_t tokens, at::ScalarType type, const Where &w) {
    w.same(t, type);
    need(t.dim() == 2 && t.size(0) == tokens && t.size(1) >= width && (t.stride(1) == 1 || t.size(1) <= 1));
    const int64_t s = t.stride(0), n = t.size(1);
    return tokens > 1 || s > n ? s : n;
}

void *like(const at::Tensor &t, const at::Tensor &x, const Where &w) {
    w.same(t, x.scalar_type());
    need(t.sizes() == x.sizes() && t.is_contiguous());
    return t.data_ptr();
}

void rope_arg(rmsnorm_rope_t *r, PyObject *positions, PyObject *inv_freq, PyObject *sections, PyObject *interleaved,
              int64_t tokens, int64_t head_dim, const Where &w) {
    std::memset(r, 0, sizeof(*r));
    const at::Tensor &f = tensor(inv_freq);
    const int64_t pairs = f.numel();
    need(pairs >= 1 && pairs <= head_dim / 2);
    r->inv_freq = static_cast<const float *>(vector(inv_freq, pairs, at::kFloat, w));
    if (sections == Py_None) {
        r->axes = 1;
        r->section[0] = (int32_t)pairs;
    } else {
        need(PyList_CheckExact(sections) || PyTuple_CheckExact(sections));
        const Py_ssize_t axes = PySequence_Fast_GET_SIZE(sections);
        need(axes >= 1 && axes <= 4);
        int64_t sum = 0;
        for (Py_ssize_t a = 0; a < axes; ++a) {
            r->section[a] = count(PySequence_Fast_GET_ITEM(sections, a));
            sum += r->section[a];
        }
        need(sum == pairs);
        r->axes = (int32_t)axes;
    }
    r->rot_dim = (int32_t)(2 * pairs);
    r->interleaved = truth(interleaved);
    r->position_bytes = 4;
    if (positions != Py_None) {
        const at::Tensor &p = tensor(positions);
        need(p.get_device() == w.dev && (p.scalar_type() == at::kLong || p.scalar_type() == at::kInt));
        if (p.dim() == 1) need(r->axes == 1 && p.size(0) == tokens);
        else need(p.dim() == 2 && p.size(0) == r->axes && p.size(1) == tokens);
        need(tokens <= 1 || p.stride(p.dim() - 1) == 1);
        r->positions = p.data_ptr();
        r->position_bytes = p.scalar_type() == at::kLong ? 8 : 4;
        if (r->axes > 1) r->position_stride = tokens > 1 || p.stride(0) > tokens ? p.stride(0) : tokens;
    }
}

// A tensor of x's type and device, uninitialised.  Straight from the allocator
// of the current stream: through the dispatcher an allocation takes 1.5 us on
// the host, nearly a launch (the norm's gradient with a weight 7.7 -> 6.0 us of
// host time a call, with the workspace's memory alone in place of a tensor).
at::Tensor fresh_of(at::IntArrayRef size, at::ScalarType type, const at::Tensor &x) {
    return at::Tensor(at::detail::empty_cuda(size, type, x.device(), std::nullopt));
}
at::Tensor fresh(at::IntArrayRef size, const at::Tensor &x) { return fresh_of(size, x.scalar_type(), x); }

// Part of a tensor's memory as a tensor of its own, `first` elements of 4 bytes
// from its start: small outputs of one call share an allocation (five of their
// own take 4 us of host time, five of these 1).
at::Tensor part_of(const at::Tensor &all, int64_t first, at::IntArrayRef size, at::ScalarType type) {
    at::Tensor t = at::detail::make_tensor<c10::TensorImpl>(c10::Storage(all.storage()),
                                                            c10::DispatchKeySet(c10::DispatchKey::CUDA),
                                                            c10::scalarTypeToTypeMeta(type));
    t.unsafeGetTensorImpl()->set_sizes_contiguous(size);
    t.unsafeGetTensorImpl()->set_storage_offset(first);
    return t;
}

// A workspace given, or made without the lock (memory of the current stream,
// handed back when the call is over and used again only behind it).
struct Workspace {
    c10::DataPtr made;
    void *at = nullptr;
    int64_t bytes = 0;
    void given(PyObject *o, int64_t n, const Where &w) {
        bytes = n;
        if (o == Py_None) return;
        const at::Tensor &t = tensor(o);
        need(t.get_device() == w.dev && t.is_contiguous() && t.numel() * (int64_t)t.element_size() >= n);
        at = t.data_ptr();
    }
    void make() {
        if (bytes == 0 || at != nullptr) return;
        made = c10::GetAllocator(c10::kCUDA)->allocate((size_t)bytes);
        at = made.get();
    }
};

// A span without the interpreter's lock.  No Python object is touched in it;
// an exception takes the lock back on its way out.
class Unlocked {
    PyThreadState *state;

public:
    Unlocked() : state(PyEval_SaveThread()) {}
    ~Unlocked() { PyEval_RestoreThread(state); }
    Unlocked(const Unlocked &) = delete;
    Unlocked &operator=(const Unlocked &) = delete;
};

// An output given, or made without the lock.
struct Output {
    PyObject *object;
    at::Tensor made;
    void *at = nullptr;
    explicit Output(PyObject *o) : object(o) {}
    bool given() const { return object != Py_None; }
    void make(at::IntArrayRef size, const at::Tensor &x) {
        if (given()) return;
        made = fresh(size, x);
        at = made.data_ptr();
    }
    PyObject *result() const {
        if (!given()) return THPVariable_Wrap(made);
        Py_INCREF(object);
        return object;
    }
};

PyObject *status_of(int st) { return PyLong_FromLong(st); }

PyObject *wrap_or_none(const at::Tensor &t) {
    if (t.defined()) return THPVariable_Wrap(t);
    Py_RETURN_NONE;
}

// Runs a call; what it leaves to api.py comes back as None.
template <typename F>
PyObject *guarded(F f) {
    try {
        return f();
    } catch (const Elsewhere &) {
        Py_RETURN_NONE;
    } catch (const std::exception &e) {   // an allocation that failed
        PyErr_Clear();
        Py_RETURN_NONE;
    }
}

// (qkv, q_heads, k_heads, head_dim, positions, inv_freq, q_w, k_w, eps, weight_bias, norm, sections, interleaved, out)
PyObject *qk_norm_rope(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded([&]() -> PyObject * {
        need(n == 14 && qk_rope_fwd != nullptr);
        const at::Tensor x = tensor(a[0]);
        void *from = x.data_ptr();
        const int code = code_of(x);
        const Where w(x);
        const int32_t q = count(a[1]), k = count(a[2]);
        const int64_t d = whole(a[3]), tokens = x.dim() == 2 ? x.size(0) : -1, width = ((int64_t)q + k) * d;
        const int64_t xs = head_rows(x, width, tokens, x.scalar_type(), w);
        void *qw = vector(a[6], d, x.scalar_type(), w), *kw = vector(a[7], d, x.scalar_type(), w);
        rmsnorm_rope_t rope;
        need(a[4] != Py_None);
        rope_arg(&rope, a[4], a[5], a[11], a[12], tokens, d, w);
        const float bias = real(a[9]), eps = real(a[8]);
        const int norm = truth(a[10]);
        Output y(a[13]);
        int64_t ys = width;
        if (y.given()) {
            const at::Tensor &o = tensor(a[13]);
            ys = head_rows(o, width, tokens, x.scalar_type(), w);
            y.at = o.data_ptr();
        }
        int st;
        {
            const Unlocked span;
            y.make({tokens, width}, x);
            st = qk_rope_fwd(from, y.at, tokens, xs, ys, q, k, d, qw, kw, bias, eps, norm, &rope, code, w.stream());
        }
        return st == RMSNORM_OK ? y.result() : status_of(st);
    });
}

// (dout, qkv, q_heads, k_heads, head_dim, positions, inv_freq, q_w, k_w, eps, weight_bias, norm, sections, interleaved,
//  out, workspace)
PyObject *qk_norm_rope_backward(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded([&]() -> PyObject * {
        need(n == 16 && qk_rope_bwd != nullptr);
        const at::Tensor g = tensor(a[0]);
        void *from = g.data_ptr();
        const int code = code_of(g);
        const Where w(g);
        const int32_t q = count(a[2]), k = count(a[3]);
        const int64_t d = whole(a[4]), tokens = g.dim() == 2 ? g.size(0) : -1, width = ((int64_t)q + k) * d;
        const int64_t gs = head_rows(g, width, tokens, g.scalar_type(), w);
        const bool norm = truth(a[11]);
        need(!norm || a[1] != Py_None);
        void *x = nullptr;
        int64_t xs = width;
        if (a[1] != Py_None) {
            const at::Tensor &t = tensor(a[1]);
            xs = head_rows(t, width, tokens, g.scalar_type(), w);
            x = t.data_ptr();
        }
        void *qw = vector(a[7], d, g.scalar_type(), w), *kw = vector(a[8], d, g.scalar_type(), w);
        rmsnorm_rope_t rope;
        need(a[5] != Py_None);
        rope_arg(&rope, a[5], a[6], a[12], a[13], tokens, d, w);
        const float bias = real(a[10]), eps = real(a[9]);
        Output y(a[14]);
        int64_t ys = width;
        if (y.given()) {
            const at::Tensor &o = tensor(a[14]);
            ys = head_rows(o, width, tokens, g.scalar_type(), w);
            y.at = o.data_ptr();
        }
        at::Tensor dq, dk;
        Workspace ws;
        const bool weights = qw != nullptr && kw != nullptr;
        if (weights) {
            const int64_t bytes = qk_rope_bwd_workspace_bytes(d);
            need(bytes > 0);
            ws.given(a[15], bytes, w);
        }
        int st;
        {
            const Unlocked span;
            y.make({tokens, width}, g);
            if (weights) {
                dq = fresh({d}, g);
                dk = fresh({d}, g);
                ws.make();
            }
            st = qk_rope_bwd(from, x, y.at, tokens, gs, xs, ys, q, k, d, qw, kw, weights ? dq.data_ptr() : nullptr,
                             weights ? dk.data_ptr() : nullptr, bias, eps, norm, &rope, code, ws.at,
                             (uint64_t)ws.bytes, w.stream());
        }
        if (st != RMSNORM_OK) return status_of(st);
        return Py_BuildValue("(NNN)", y.result(), wrap_or_none(dq), wrap_or_none(dk));
    });
}

// (qkv, k_cache, v_cache, page_table, cu_tokens, cache_lens, q_heads, kv_heads, head_dim, inv_freq, positions, q_w, k_w,
//  eps, weight_bias, norm, sections, interleaved, k_scale, v_scale, q_out, dropped)
PyObject *qkv_append(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded([&]() -> PyObject * {
        need(n == 22 && qkv_append_fn != nullptr);
        const at::Tensor x = tensor(a[0]);
        void *from = x.data_ptr();
        const int code = code_of(x);
        const Where w(x);
        const int32_t q = count(a[6]), kv_heads = count(a[7]);
        need(q > 0);
        const int64_t d = whole(a[8]), tokens = x.dim() == 2 ? x.size(0) : -1;
        const int64_t xs = head_rows(x, ((int64_t)q + 2 * (int64_t)kv_heads) * d, tokens, x.scalar_type(), w);
        void *qw = vector(a[11], d, x.scalar_type(), w), *kw = vector(a[12], d, x.scalar_type(), w);
        rmsnorm_rope_t rope;
        rope_arg(&rope, a[10], a[9], a[16], a[17], tokens, d, w);
        const at::Tensor &kc = tensor(a[1]), &vc = tensor(a[2]), &table = tensor(a[3]);
        const at::ScalarType held = kc.scalar_type();
        need(held == x.scalar_type() || held == at::kFloat8_e4m3fn);
        w.same(kc, held);
        w.same(vc, held);
        need(kc.dim() == 4 && kc.size(2) == kv_heads && kc.size(3) == d && kc.stride(3) == 1 &&
             vc.sizes() == kc.sizes() && vc.strides() == kc.strides());
        w.same(table, at::kInt);
        need(table.dim() == 2 && (table.stride(1) == 1 || table.size(1) <= 1));
        const int64_t seqs = table.size(0), max_pages = table.size(1);
        need(seqs <= INT32_MAX && max_pages <= INT32_MAX && kc.size(0) <= INT32_MAX && kc.size(1) <= INT32_MAX);
        rmsnorm_paged_kv_t kv;
        std::memset(&kv, 0, sizeof(kv));
        kv.k_cache = kc.data_ptr();
        kv.v_cache = vc.data_ptr();
        kv.page_table = static_cast<const int32_t *>(table.data_ptr());
        need(a[4] != Py_None && a[5] != Py_None);
        kv.cu_tokens = static_cast<const int32_t *>(vector(a[4], seqs + 1, at::kInt, w));
        kv.cache_lens = static_cast<const int32_t *>(vector(a[5], seqs, at::kInt, w));
        kv.dropped = static_cast<int32_t *>(vector(a[21], 1, at::kInt, w));
        kv.page_table_stride = seqs > 1 || table.stride(0) > max_pages ? table.stride(0) : max_pages;
        kv.page_stride = kc.size(0) > 1 ? kc.stride(0) : 0;
        kv.row_stride = kc.size(1) > 1 ? kc.stride(1) : 0;
        kv.head_stride = kc.size(2) > 1 ? kc.stride(2) : 0;
        kv.seqs = (int32_t)seqs;
        kv.max_pages = (int32_t)max_pages;
        kv.num_pages = (int32_t)kc.size(0);
        kv.page_size = (int32_t)kc.size(1);
        kv.cache_dtype = held == at::kFloat8_e4m3fn ? (int)RMSNORM_E4M3 : code;
        kv.k_scale = real(a[18]);
        kv.v_scale = real(a[19]);
        const float bias = real(a[14]), eps = real(a[13]);
        const int norm = truth(a[15]);
        Output y(a[20]);
        int64_t ys = (int64_t)q * d;
        if (y.given()) {
            const at::Tensor &o = tensor(a[20]);
            ys = head_rows(o, ys, tokens, x.scalar_type(), w);
            y.at = o.data_ptr();
        }
        int st;
        {
            const Unlocked span;
            y.make({tokens, (int64_t)q * d}, x);
            st = qkv_append_fn(from, y.at, tokens, xs, ys, q, kv_heads, d, qw, kw, bias, eps, norm, &rope, &kv, code,
                               w.stream());
        }
        return st == RMSNORM_OK ? y.result() : status_of(st);
    });
}

struct Rows {
    int64_t rows, hidden;
    explicit Rows(const at::Tensor &t) {
        need(t.dim() >= 1 && t.size(-1) >= 1 && t.is_contiguous());
        hidden = t.size(-1);
        rows = t.numel() / hidden;
    }
};

const uint64_t *rng_of(PyObject *o, float p, const Where &w) {
    if (o == Py_None) {
        need(p == 0.f);
        return nullptr;
    }
    return static_cast<const uint64_t *>(vector(o, 2, at::kLong, w));
}

// (x, residual, p, rng, w, eps, weight_bias, out, residual_out)
PyObject *rms_norm_dropout(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded([&]() -> PyObject * {
        need(n == 9 && dropout_fwd != nullptr);
        const at::Tensor x = tensor(a[0]);
        void *from = x.data_ptr();
        const int code = code_of(x);
        const Where w(x);
        const Rows r(x);
        const void *res = like(tensor(a[1]), x, w);
        const float p = real(a[2]);
        const uint64_t *rng = rng_of(a[3], p, w);
        void *weight = vector(a[4], r.hidden, x.scalar_type(), w);
        const float eps = real(a[5]), bias = real(a[6]);
        Output y(a[7]), h(a[8]);
        if (y.given()) y.at = like(tensor(a[7]), x, w);
        if (h.given()) h.at = like(tensor(a[8]), x, w);
        int st;
        {
            const Unlocked span;
            y.make(x.sizes(), x);
            h.make(x.sizes(), x);
            st = dropout_fwd(from, res, weight, y.at, h.at, r.rows, r.hidden, eps, bias, p, rng, code, w.stream());
        }
        if (st != RMSNORM_OK) return status_of(st);
        return Py_BuildValue("(NN)", y.result(), h.result());
    });
}

// What the two gradients of the norm share: dw and the workspace, with a weight.
struct Backward {
    const at::Tensor dy;
    int code;
    Where w;
    Rows r;
    void *from, *h, *weight, *dh;
    at::Tensor dw;
    void *dw_at = nullptr;
    Workspace ws;
    Backward(PyObject *dy_, PyObject *h_, PyObject *w_, PyObject *dh_, PyObject *workspace)
        : dy(tensor(dy_)), code(code_of(dy)), w(dy), r(dy), from(dy.data_ptr()), h(like(tensor(h_), dy, w)),
          weight(vector(w_, r.hidden, dy.scalar_type(), w)), dh(dh_ == Py_None ? nullptr : like(tensor(dh_), dy, w)) {
        if (weight == nullptr) return;
        const int64_t bytes = bwd_workspace_bytes(r.rows, r.hidden, code);
        need(bytes > 0);
        ws.given(workspace, bytes, w);
    }
    void make() {   // without the lock
        if (weight == nullptr) return;
        dw = fresh({r.hidden}, dy);
        dw_at = dw.data_ptr();
        ws.make();
    }
};

// (dy, h, w, dresidual_out, eps, weight_bias, out, workspace)
PyObject *rms_norm_backward(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded([&]() -> PyObject * {
        need(n == 8 && norm_bwd != nullptr);
        Backward b(a[0], a[1], a[2], a[3], a[7]);
        const float eps = real(a[4]), bias = real(a[5]);
        Output dx(a[6]);
        if (dx.given()) dx.at = like(tensor(a[6]), b.dy, b.w);
        int st;
        {
            const Unlocked span;
            b.make();
            dx.make(b.dy.sizes(), b.dy);
            st = norm_bwd(b.from, b.h, b.weight, b.dh, dx.at, b.dw_at, b.r.rows, b.r.hidden, eps, bias, b.code, b.ws.at,
                          (uint64_t)b.ws.bytes, b.w.stream());
        }
        if (st != RMSNORM_OK) return status_of(st);
        return Py_BuildValue("(NN)", dx.result(), wrap_or_none(b.dw));
    });
}

// (dy, h, p, rng, w, dresidual_out, eps, weight_bias, dresidual, dx, workspace)
PyObject *rms_norm_dropout_backward(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded([&]() -> PyObject * {
        need(n == 11 && dropout_bwd != nullptr);
        Backward b(a[0], a[1], a[4], a[5], a[10]);
        const float p = real(a[2]), eps = real(a[6]), bias = real(a[7]);
        const uint64_t *rng = rng_of(a[3], p, b.w);
        Output dres(a[8]), dx(a[9]);
        if (dres.given()) dres.at = like(tensor(a[8]), b.dy, b.w);
        if (dx.given()) dx.at = like(tensor(a[9]), b.dy, b.w);
        int st;
        {
            const Unlocked span;
            b.make();
            dres.make(b.dy.sizes(), b.dy);
            dx.make(b.dy.sizes(), b.dy);
            st = dropout_bwd(b.from, b.h, b.weight, b.dh, dres.at, dx.at, b.dw_at, b.r.rows, b.r.hidden, eps, bias, p,
                             rng, b.code, b.ws.at, (uint64_t)b.ws.bytes, b.w.stream());
        }
        if (st != RMSNORM_OK) return status_of(st);
        return Py_BuildValue("(NNN)", dres.result(), dx.result(), wrap_or_none(b.dw));
    });
}

// Contiguous token ids, of the shape given or of any.
struct Ids {
    void *at = nullptr;
    int bytes = 4;
    Ids(PyObject *o, const int64_t *rows, const Where &w) {
        const at::Tensor &t = tensor(o);
        need(t.get_device() == w.dev && (t.scalar_type() == at::kLong || t.scalar_type() == at::kInt) && t.is_contiguous());
        if (rows != nullptr) need(t.dim() == 1 && t.size(0) == *rows);
        at = t.data_ptr();
        bytes = t.scalar_type() == at::kLong ? 8 : 4;
    }
    Ids() = default;
};

// Row stride of a 2-D tensor.
int64_t row_stride(const at::Tensor &t) {
    need(t.dim() == 2 && t.size(1) >= 1 && (t.stride(1) == 1 || t.size(1) == 1));
    return t.size(0) > 1 || t.stride(0) > t.size(1) ? t.stride(0) : t.size(1);
}

// (tokens, table, scale, out)
PyObject *embedding(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded([&]() -> PyObject * {
        need(n == 4 && embedding_fwd != nullptr);
        const at::Tensor table = tensor(a[1]), tokens = tensor(a[0]);
        const int code = code_of(table);
        const Where w(table);
        const int64_t stride = row_stride(table), vocab = table.size(0), width = table.size(1), count = tokens.numel();
        const Ids ids(a[0], nullptr, w);
        const float scale = real(a[2]);
        c10::SmallVector<int64_t, 6> shape(tokens.sizes().begin(), tokens.sizes().end());
        shape.push_back(width);
        Output y(a[3]);
        if (y.given()) {
            const at::Tensor &o = tensor(a[3]);
            w.same(o, table.scalar_type());
            need(o.sizes() == at::IntArrayRef(shape) && o.is_contiguous());
            y.at = o.data_ptr();
        }
        int st;
        {
            const Unlocked span;
            y.make(shape, table);
            st = embedding_fwd(ids.at, ids.bytes, table.data_ptr(), y.at, count, vocab, width, stride, scale, code,
                               w.stream());
        }
        return st == RMSNORM_OK ? y.result() : status_of(st);
    });
}

// (dout, tokens, vocab, scale, out, accumulate, workspace)
PyObject *embedding_backward(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded([&]() -> PyObject * {
        need(n == 7 && embedding_bwd != nullptr);
        const at::Tensor dy = tensor(a[0]), tokens = tensor(a[1]);
        const int code = code_of(dy);
        const Where w(dy);
        const Rows r(dy);
        const Ids ids(a[1], nullptr, w);
        need(tokens.sizes() == dy.sizes().slice(0, dy.dim() - 1));
        const int64_t vocab = whole(a[2]);
        need(vocab >= 1);
        const float scale = real(a[3]);
        const bool add = truth(a[5]);
        Output d(a[4]);
        int64_t stride = r.hidden;
        int held = code;
        if (d.given()) {
            const at::Tensor &o = tensor(a[4]);
            held = code_of(o);
            need(o.get_device() == w.dev && (held == code || held == RMSNORM_F32) && o.dim() == 2 && o.size(0) == vocab &&
                 o.size(1) == r.hidden);
            stride = row_stride(o);
            d.at = o.data_ptr();
        } else {
            need(!add);
        }
        Workspace ws;
        const int64_t bytes = embedding_bwd_workspace_bytes(r.rows, vocab, r.hidden);
        need(bytes > 0);
        ws.given(a[6], bytes, w);
        int st;
        {
            const Unlocked span;
            d.make({vocab, r.hidden}, dy);
            ws.make();
            st = embedding_bwd(dy.data_ptr(), ids.at, ids.bytes, d.at, r.rows, vocab, r.hidden, stride, scale, add, code,
                               held, ws.at, (uint64_t)ws.bytes, w.stream());
        }
        return st == RMSNORM_OK ? d.result() : status_of(st);
    });
}

float *floats(const at::Tensor &t) { return t.defined() ? static_cast<float *>(t.data_ptr()) : nullptr; }

// (logits, tokens, temperature, top, entropy)
PyObject *token_logprobs(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded([&]() -> PyObject * {
        need(n == 5 && logprobs_fwd != nullptr);
        const at::Tensor x = tensor(a[0]);
        const int code = code_of(x);
        const Where w(x);
        const int64_t stride = row_stride(x), rows = x.size(0), vocab = x.size(1);
        const bool given = a[1] != Py_None;
        const Ids ids = given ? Ids(a[1], &rows, w) : Ids();
        const float temperature = real(a[2]);
        const int32_t top = count(a[3]);
        need(top <= 32 && top <= vocab);
        const bool entropy = truth(a[4]);
        at::Tensor lp, stats, ent, top_lp, top_ids;
        int st;
        {
            const Unlocked span;
            const int64_t many = rows * (2 + (given ? 1 : 0) + (entropy ? 1 : 0) + 2 * (int64_t)top);
            const at::Tensor all = fresh_of({many}, at::kFloat, x);
            int64_t next = 2 * rows;
            stats = part_of(all, 0, {rows, 2}, at::kFloat);
            auto take = [&](at::IntArrayRef size, int64_t n, at::ScalarType type) {
                next += n;
                return part_of(all, next - n, size, type);
            };
            if (given) lp = take({rows}, rows, at::kFloat);
            if (entropy) ent = take({rows}, rows, at::kFloat);
            if (top > 0) {
                top_lp = take({rows, top}, rows * top, at::kFloat);
                top_ids = take({rows, top}, rows * top, at::kInt);
            }
            st = logprobs_fwd(x.data_ptr(), ids.at, ids.bytes, floats(lp), floats(stats), floats(ent), floats(top_lp),
                              top > 0 ? static_cast<int32_t *>(top_ids.data_ptr()) : nullptr, rows, vocab, stride, top,
                              temperature, code, w.stream());
        }
        if (st != RMSNORM_OK) return status_of(st);
        return Py_BuildValue("(NNNNN)", wrap_or_none(lp), wrap_or_none(stats), wrap_or_none(ent), wrap_or_none(top_lp),
                             wrap_or_none(top_ids));
    });
}

// (logits, tokens, stats, dlogprobs, entropy, dentropy, temperature, out)
PyObject *token_logprobs_backward(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded([&]() -> PyObject * {
        need(n == 8 && logprobs_bwd != nullptr);
        const at::Tensor x = tensor(a[0]);
        const int code = code_of(x);
        const Where w(x);
        const int64_t stride = row_stride(x), rows = x.size(0), vocab = x.size(1);
        const Ids ids = a[1] != Py_None ? Ids(a[1], &rows, w) : Ids();
        const at::Tensor &stats = tensor(a[2]);
        w.same(stats, at::kFloat);
        need(stats.dim() == 2 && stats.size(0) == rows && stats.size(1) == 2 && stats.is_contiguous());
        const float *of = static_cast<const float *>(stats.data_ptr());
        const float *dlp = static_cast<const float *>(vector(a[3], rows, at::kFloat, w));
        const float *ent = static_cast<const float *>(vector(a[4], rows, at::kFloat, w));
        const float *dent = static_cast<const float *>(vector(a[5], rows, at::kFloat, w));
        need((dlp == nullptr || ids.at != nullptr) && (dent == nullptr || ent != nullptr));
        const float temperature = real(a[6]);
        Output d(a[7]);
        int64_t dstride = vocab;
        if (d.given()) {
            const at::Tensor &o = tensor(a[7]);
            w.same(o, x.scalar_type());
            need(o.sizes() == x.sizes());
            dstride = row_stride(o);
            d.at = o.data_ptr();
        }
        int st;
        {
            const Unlocked span;
            d.make({rows, vocab}, x);
            st = logprobs_bwd(x.data_ptr(), ids.at, ids.bytes, of, dlp, ent, dent, d.at, rows, vocab, stride, dstride,
                              temperature, code, w.stream());
        }
        return st == RMSNORM_OK ? d.result() : status_of(st);
    });
}

// (grads, max_norm or None for the norm alone, out, workspace)
PyObject *clip_grad_norm(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded([&]() -> PyObject * {
        need(n == 4 && clip_grads != nullptr);
        need(PyList_CheckExact(a[0]) || PyTuple_CheckExact(a[0]));
        need(a[2] == Py_None || PyList_CheckExact(a[2]) || PyTuple_CheckExact(a[2]));
        const Py_ssize_t many = PySequence_Fast_GET_SIZE(a[0]);
        need(a[2] == Py_None || PySequence_Fast_GET_SIZE(a[2]) == many);
        std::vector<rmsnorm_grad_t> grads;
        std::vector<at::Tensor> held;   // the lists may change while the lock is not held
        grads.reserve(many);
        held.reserve(2 * many);
        for (Py_ssize_t i = 0; i < many; ++i) {
            PyObject *of = PySequence_Fast_GET_ITEM(a[0], i);
            if (of == Py_None) continue;
            const at::Tensor &g = tensor(of);
            need(g.is_contiguous() && (held.empty() || g.get_device() == held[0].get_device()));
            rmsnorm_grad_t e;
            std::memset(&e, 0, sizeof(e));
            e.grad = g.data_ptr();
            e.out = g.data_ptr();
            e.count = g.numel();
            e.dtype = code_of(g);
            held.push_back(g);
            if (a[2] != Py_None) {
                const at::Tensor &o = tensor(PySequence_Fast_GET_ITEM(a[2], i));
                need(o.get_device() == g.get_device() && o.scalar_type() == g.scalar_type() && o.sizes() == g.sizes() &&
                     o.is_contiguous());
                e.out = o.data_ptr();
                held.push_back(o);
            }
            grads.push_back(e);
        }
        need(!held.empty());
        const Where w(held[0]);
        const bool clip = a[1] != Py_None;
        const float most = clip ? real(a[1]) : 0.f;
        Workspace ws;
        ws.given(a[3], grad_norm_workspace_bytes(), w);
        at::Tensor norm;
        int st;
        {
            const Unlocked span;
            norm = fresh_of({1}, at::kFloat, held[0]);
            ws.make();
            st = clip ? clip_grads(grads.data(), (int64_t)grads.size(), most, floats(norm), ws.at, (uint64_t)ws.bytes,
                                   w.stream())
                      : norm_of_grads(grads.data(), (int64_t)grads.size(), floats(norm), ws.at, (uint64_t)ws.bytes,
                                      w.stream());
        }
        return st == RMSNORM_OK ? THPVariable_Wrap(norm) : status_of(st);
    });
}

// Addresses of the C ABI's functions, in the order below.
PyObject *bind(PyObject *, PyObject *const *a, Py_ssize_t n) {
    void *const to[] = {&qk_rope_fwd, &qk_rope_bwd, &qk_rope_bwd_workspace_bytes, &qkv_append_fn, &dropout_fwd, &norm_bwd,
                        &bwd_workspace_bytes, &dropout_bwd, &embedding_fwd, &embedding_bwd,
                        &embedding_bwd_workspace_bytes, &logprobs_fwd, &logprobs_bwd, &norm_of_grads, &clip_grads,
                        &grad_norm_workspace_bytes};
    constexpr int kMany = sizeof(to) / sizeof(to[0]);
    void *at[kMany];
    if (n != kMany) {
        PyErr_Format(PyExc_TypeError, "bind takes %d addresses", kMany);
        return nullptr;
    }
    for (int i = 0; i < kMany; ++i) {
        at[i] = PyLong_AsVoidPtr(a[i]);
        if (PyErr_Occurred()) return nullptr;
    }
    for (int i = 0; i < kMany; ++i) std::memcpy(to[i], &at[i], sizeof(void *));
    Py_RETURN_NONE;
}

#define ENTRY(f) {#f, reinterpret_cast<PyCFunction>(reinterpret_cast<void *>(&f)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {ENTRY(bind), ENTRY(qk_norm_rope), ENTRY(qk_norm_rope_backward), ENTRY(qkv_append),
                         ENTRY(rms_norm_dropout), ENTRY(rms_norm_backward), ENTRY(rms_norm_dropout_backward),
                         ENTRY(embedding), ENTRY(embedding_backward), ENTRY(token_logprobs),
                         ENTRY(token_logprobs_backward), ENTRY(clip_grad_norm), {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_fastcall", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__fastcall() { return PyModule_Create(&module); }
