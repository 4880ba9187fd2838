// torch_binding.cpp -- the short way from torch tensors to libfd for the calls
// that a serving loop makes once a layer and step: append_kv_norm, evict_kv,
// PagedDecoder.decode_weights, DiffDecoder, CrossDecoder and PrefixDecoder.  A call's arguments are checked
// and its outputs allocated here instead of in Python, which took 15 to 25 us
// of host time a call around 4 us of launches.
//
// Marshalling only.  Every function returns None where anything is not as the
// ordinary case has it (another type, shape, layout or device, a stream given,
// a call that libfd refuses): the Python binding then takes the call from the
// start, so that its checks, messages and errors are the ones there are.  A call
// that failed otherwise may have launched some of its kernels; it is not made
// again, and FdError is raised here.
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <initializer_list>

#include "../../include/fd_api.h"

namespace {

decltype(&fd_append_kv_norm) g_append = nullptr;
decltype(&fd_evict_kv) g_evict = nullptr;
decltype(&fd_decode_paged_weights) g_weights = nullptr;
decltype(&fd_decode_paged_diff) g_diff = nullptr;
decltype(&fd_cross_paged) g_cross = nullptr;
decltype(&fd_decode_paged_prefix) g_prefix = nullptr;

PyObject *g_error = nullptr;  // FdError

// Thrown where the call is not the ordinary case.
struct Other {};

// Thrown where the call failed in or after its launches.
struct Failed {
    fd_status status;
};

at::ScalarType torch_type(int t) {
    switch (t) {
    case FD_F16: return at::kHalf;
    case FD_BF16: return at::kBFloat16;
    case FD_E4M3: return at::kFloat8_e4m3fn;
    case FD_F32: return at::kFloat;
    }
    throw Other();
}

fd_dtype fd_type(at::ScalarType t) {
    switch (t) {
    case at::kHalf: return FD_F16;
    case at::kBFloat16: return FD_BF16;
    case at::kFloat8_e4m3fn: return FD_E4M3;
    case at::kFloat: return FD_F32;
    default: throw Other();
    }
}

// The tensors of one call: all on one device, which is the current one.
class Call {
  public:
    // A plain strided tensor (no subclass).
    const at::Tensor &tensor(PyObject *o) {
        if (!THPVariable_CheckExact(o)) throw Other();
        const at::Tensor &t = THPVariable_Unpack(o);
        if (t.layout() != at::kStrided || !t.is_cuda()) throw Other();
        const int d = t.get_device();
        if (device_ < 0) device_ = d;
        if (d != device_) throw Other();
        return t;
    }
    const at::Tensor &dense(PyObject *o, at::ScalarType type, std::initializer_list<int64_t> shape) {
        const at::Tensor &t = tensor(o);
        if (t.scalar_type() != type || t.sizes() != at::IntArrayRef(shape) || !t.is_contiguous()) throw Other();
        return t;
    }
    template <typename T = void>
    T *data(PyObject *o, at::ScalarType type, std::initializer_list<int64_t> shape) {
        return static_cast<T *>(dense(o, type, shape).data_ptr());
    }
    // None: a null pointer.
    template <typename T = void>
    T *maybe(PyObject *o, at::ScalarType type, std::initializer_list<int64_t> shape) {
        return o == Py_None ? nullptr : data<T>(o, type, shape);
    }
    int32_t *status(PyObject *o) {
        if (o == Py_None) return nullptr;
        const at::Tensor &t = tensor(o);
        if (t.scalar_type() != at::kInt || t.numel() < 1 || !t.is_contiguous()) throw Other();
        return static_cast<int32_t *>(t.data_ptr());
    }
    // Memory of any type, and its bytes.
    void *bytes(PyObject *o, size_t *n) {
        const at::Tensor &t = tensor(o);
        if (!t.is_contiguous()) throw Other();
        *n = t.nbytes();
        return t.data_ptr();
    }
    // [lead..., heads, D] with contiguous heads and its tokens at one stride.
    const void *rows(PyObject *o, at::ScalarType type, at::IntArrayRef shape, long long *stride) {
        const at::Tensor &t = tensor(o);
        if (t.scalar_type() != type || t.sizes() != shape) throw Other();
        const int64_t n = t.dim(), D = shape[n - 1], heads = shape[n - 2];
        const at::IntArrayRef st = t.strides();
        if (st[n - 1] != 1 || (heads > 1 && st[n - 2] != D)) throw Other();
        int64_t count = 1, step = heads * D;
        for (int64_t i = n - 3; i >= 0; --i) {
            if (shape[i] == 1) continue;
            if (count == 1) step = st[i];
            else if (st[i] != count * step) throw Other();
            count *= shape[i];
        }
        if (step < heads * D || step % 8) throw Other();
        *stride = step;
        return t.data_ptr();
    }
    at::Tensor make(at::IntArrayRef shape, at::ScalarType type) const {
        return at::empty(shape, at::TensorOptions().dtype(type).device(at::kCUDA, (c10::DeviceIndex)device_));
    }
    // The current stream of the tensors' device, which has to be current.
    void *stream() const {
        if (device_ < 0 || c10::cuda::current_device() != device_) throw Other();
        return c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)device_).stream();
    }

  private:
    int device_ = -1;
};

long long as_int(PyObject *o) {
    if (!PyLong_CheckExact(o)) throw Other();
    const long long v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred()) throw Other();
    if (v < INT32_MIN || v > INT32_MAX) throw Other();
    return v;
}

bool as_bool(PyObject *o) {
    const int v = PyObject_IsTrue(o);
    if (v < 0) throw Other();
    return v != 0;
}

float as_float(PyObject *o) {
    if (!PyFloat_CheckExact(o) && !PyLong_CheckExact(o)) throw Other();
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred()) throw Other();
    return (float)v;
}

const fd_plan_t *as_plan(PyObject *o) {
    void *p = PyLong_AsVoidPtr(o);
    if (!p) throw Other();
    return static_cast<const fd_plan_t *>(p);
}

// Run a libfd entry point without the interpreter's lock.  The three statuses
// of a refusal come before anything is launched.
template <typename F>
void run(F &&f) {
    fd_status r;
    Py_BEGIN_ALLOW_THREADS
    r = f();
    Py_END_ALLOW_THREADS
    if (r == FD_ERR_INVALID_ARG || r == FD_ERR_UNSUPPORTED || r == FD_ERR_WORKSPACE_TOO_SMALL) throw Other();
    if (r != FD_OK) throw Failed{r};
}

PyObject *wrap(const at::Tensor &t) { return THPVariable_Wrap(t); }

// An output: the given tensor, or a new one.
struct Output {
    at::Tensor made;
    PyObject *given = nullptr;
    void *ptr = nullptr;
    PyObject *object() const {  // a new reference
        if (given) {
            Py_INCREF(given);
            return given;
        }
        return wrap(made);
    }
};

Output output(Call &c, PyObject *o, at::IntArrayRef shape, at::ScalarType type) {
    Output r;
    if (o != Py_None) {
        const at::Tensor &t = c.tensor(o);
        if (t.scalar_type() != type || t.sizes() != shape || !t.is_contiguous()) throw Other();
        r.given = o;
        r.ptr = t.data_ptr();
    } else {
        r.made = c.make(shape, type);
        r.ptr = r.made.data_ptr();
    }
    return r;
}

PyObject *tuple_of(std::initializer_list<PyObject *> items) {
    PyObject *t = PyTuple_New((Py_ssize_t)items.size());
    Py_ssize_t i = 0;
    for (PyObject *o : items) PyTuple_SET_ITEM(t, i++, o);
    return t;
}

struct Pools {
    void *k, *v;
    const float *ks, *vs;
};

Pools pools(Call &c, const fd_problem &p, PyObject *k, PyObject *v, PyObject *ks, PyObject *vs) {
    const at::ScalarType kv = torch_type(p.kv_dtype);
    Pools r;
    r.k = c.data(k, kv, {p.num_pages, p.page_size, p.Hkv, p.D});
    r.v = c.data(v, kv, {p.num_pages, p.page_size, p.Hkv, p.D});
    r.ks = c.maybe<const float>(ks, at::kFloat, {p.num_pages, p.Hkv});
    r.vs = c.maybe<const float>(vs, at::kFloat, {p.num_pages, p.Hkv});
    return r;
}

// Sizes and types of the pools and of the block table.
fd_problem problem_of(Call &c, PyObject *k_pages, PyObject *block_table) {
    const at::Tensor &kp = c.tensor(k_pages), &bt = c.tensor(block_table);
    if (kp.dim() != 4 || bt.dim() != 2) throw Other();
    for (int i = 0; i < 4; ++i)
        if (kp.size(i) > INT32_MAX) throw Other();
    if (bt.size(0) > INT32_MAX || bt.size(1) > INT32_MAX) throw Other();
    fd_problem p;
    p.B = (int)bt.size(0);
    p.max_blocks_per_seq = (int)bt.size(1);
    p.num_pages = (int)kp.size(0);
    p.page_size = (int)kp.size(1);
    p.Hq = p.Hkv = (int)kp.size(2);
    p.D = (int)kp.size(3);
    p.kv_dtype = fd_type(kp.scalar_type());
    p.q_dtype = p.out_dtype = p.kv_dtype == FD_E4M3 ? FD_BF16 : p.kv_dtype;
    return p;
}

// q, k_new, v_new, k_pages, v_pages, block_table, seq_lens, q_weight, k_weight,
// eps, cos, sin, interleaved, positions, new_lens, k_scale, v_scale, q_out, status
PyObject *append(PyObject *const *a) {
    Call c;
    fd_problem p = problem_of(c, a[3], a[5]);
    const at::Tensor &k = c.tensor(a[1]);
    const int64_t nd = k.dim();
    if ((nd != 3 && nd != 4) || k.size(0) != p.B) throw Other();
    const at::ScalarType act = k.scalar_type();
    p.q_dtype = p.out_dtype = fd_type(act);
    fd_norm_append n = {};
    n.tokens = nd == 4 ? (int)k.size(1) : 1;
    const int64_t kshape[4] = {p.B, n.tokens, p.Hkv, p.D}, kshape3[3] = {p.B, p.Hkv, p.D};
    const at::IntArrayRef ks = nd == 4 ? at::IntArrayRef(kshape, 4) : at::IntArrayRef(kshape3, 3);
    n.k_new = c.rows(a[1], act, ks, &n.k_stride);
    n.v_new = c.rows(a[2], act, ks, &n.v_stride);
    Output qo;
    if (a[0] != Py_None) {
        const at::Tensor &q = c.tensor(a[0]);
        if (q.dim() != nd) throw Other();
        p.Hq = (int)q.size(nd - 2);
        const int64_t qshape[4] = {p.B, n.tokens, p.Hq, p.D}, qshape3[3] = {p.B, p.Hq, p.D};
        const at::IntArrayRef qs = nd == 4 ? at::IntArrayRef(qshape, 4) : at::IntArrayRef(qshape3, 3);
        n.q = c.rows(a[0], act, qs, &n.q_stride);
        if (a[17] != Py_None) {
            qo.given = a[17];
            n.q_out = const_cast<void *>(c.rows(a[17], act, qs, &n.q_out_stride));
        } else {
            qo.made = c.make(qs, act);
            n.q_out = qo.made.data_ptr();
            n.q_out_stride = (long long)p.Hq * p.D;
        }
    } else if (a[17] != Py_None) {
        throw Other();
    }
    n.weight_dtype = p.q_dtype;
    PyObject *w = a[7] != Py_None ? a[7] : a[8];
    if (w != Py_None) {
        const at::ScalarType wt = c.tensor(w).scalar_type() == at::kFloat ? at::kFloat : act;
        n.q_weight = c.maybe(a[7], wt, {p.D});
        n.k_weight = c.maybe(a[8], wt, {p.D});
        n.weight_dtype = fd_type(wt);
    }
    n.eps = as_float(a[9]);
    if (a[10] != Py_None || a[11] != Py_None) {
        if (a[10] == Py_None) throw Other();
        const at::Tensor &cs = c.tensor(a[10]);
        if (cs.dim() != 2 || cs.size(0) > INT32_MAX || cs.size(1) > p.D) throw Other();
        n.max_pos = (int)cs.size(0);
        n.rotary_dim = 2 * (int)cs.size(1);
        n.rotary_cos = c.data<const float>(a[10], at::kFloat, {cs.size(0), cs.size(1)});
        n.rotary_sin = c.data<const float>(a[11], at::kFloat, {cs.size(0), cs.size(1)});
        n.interleaved = as_bool(a[12]);
    }
    n.positions = c.maybe<const int32_t>(a[13], at::kInt, {p.B});
    n.new_lens = c.maybe<const int32_t>(a[14], at::kInt, {p.B});
    const Pools pl = pools(c, p, a[3], a[4], a[15], a[16]);
    const int32_t *bt = c.data<const int32_t>(a[5], at::kInt, {p.B, p.max_blocks_per_seq});
    const int32_t *sl = c.data<const int32_t>(a[6], at::kInt, {p.B});
    int32_t *status = c.status(a[18]);
    void *stream = c.stream();
    run([&] { return g_append(&p, &n, pl.k, pl.v, pl.ks, pl.vs, bt, sl, status, stream); });
    // (q_out,): q_out may be None itself
    if (a[0] == Py_None) {
        Py_INCREF(Py_None);
        return tuple_of({Py_None});
    }
    return tuple_of({qo.object()});
}

// k_pages, v_pages, block_table, seq_lens, weights, budget, sinks, recent,
// dst_table, weights_out, k_scale, v_scale, status
PyObject *evict(PyObject *const *a) {
    Call c;
    const fd_problem p = problem_of(c, a[0], a[2]);
    const Pools pl = pools(c, p, a[0], a[1], a[10], a[11]);
    const int32_t *bt = c.data<const int32_t>(a[2], at::kInt, {p.B, p.max_blocks_per_seq});
    const int32_t *sl = c.data<const int32_t>(a[3], at::kInt, {p.B});
    const at::Tensor &wt = c.tensor(a[4]);
    if (wt.dim() != 3 || wt.size(2) < 1 || wt.size(2) > INT32_MAX) throw Other();
    const int64_t room = wt.size(2);
    const float *w = c.data<const float>(a[4], at::kFloat, {p.B, p.Hkv, room});
    const int budget = (int)as_int(a[5]), sinks = (int)as_int(a[6]), recent = (int)as_int(a[7]);
    if (budget < 1) throw Other();
    const int32_t *dst = c.maybe<const int32_t>(a[8], at::kInt, {p.B, p.max_blocks_per_seq});
    float *wo = c.maybe<float>(a[9], at::kFloat, {p.B, p.Hkv, room});
    int32_t *status = c.status(a[12]);
    void *stream = c.stream();
    const at::Tensor lens = c.make({p.B}, at::kInt), kept = c.make({p.B, p.Hkv, budget}, at::kInt);
    run([&] {
        return g_evict(&p, pl.k, pl.v, pl.ks, pl.vs, bt, sl, w, wo, (int)room, budget, sinks, recent, dst,
                       static_cast<int32_t *>(lens.data_ptr()), static_cast<int32_t *>(kept.data_ptr()), status, stream);
    });
    return tuple_of({wrap(lens), wrap(kept)});
}

// The shapes a decoder's tensors have: [B, tail] or, with several query tokens,
// [B, q_len, tail].
struct Shape {
    int64_t d[5];
    int n = 0;
    Shape(const fd_plan_t &pl, std::initializer_list<int64_t> tail) {
        d[n++] = pl.kv_rows;
        if (pl.q_len > 1) d[n++] = pl.q_len;
        for (int64_t t : tail) d[n++] = t;
    }
    operator at::IntArrayRef() const { return at::IntArrayRef(d, n); }
};

const void *query(Call &c, const fd_plan_t &pl, PyObject *o, int64_t heads) {
    const at::Tensor &t = c.tensor(o);
    if (t.scalar_type() != torch_type(pl.problem.q_dtype) || t.sizes() != at::IntArrayRef(Shape(pl, {heads, pl.problem.D})) ||
        !t.is_contiguous())
        throw Other();
    return t.data_ptr();
}

// plan, q, k_pages, v_pages, block_table, seq_lens, weights, weights_out,
// k_scale, v_scale, out, lse, want_lse, workspace, weights_workspace, status
PyObject *weights(PyObject *const *a) {
    Call c;
    const fd_plan_t &pl = *as_plan(a[0]);
    const fd_problem &p = pl.problem;  // its B counts query rows
    if (pl.row_fold != (pl.q_len > 1 ? pl.q_len : 1)) throw Other();
    const void *q = query(c, pl, a[1], p.Hq);
    const Pools po = pools(c, p, a[2], a[3], a[8], a[9]);
    const int32_t *bt = c.data<const int32_t>(a[4], at::kInt, {pl.kv_rows, p.max_blocks_per_seq});
    const int32_t *sl = c.data<const int32_t>(a[5], at::kInt, {pl.kv_rows});
    PyObject *to = a[7] != Py_None ? a[7] : a[6];
    if (to == Py_None) throw Other();
    const at::Tensor &wt = c.tensor(to);
    if (wt.dim() != 3 || wt.size(2) < 1 || wt.size(2) > INT32_MAX) throw Other();
    float *wo = c.data<float>(to, at::kFloat, {pl.kv_rows, p.Hkv, wt.size(2)});
    const float *wi = c.maybe<const float>(a[6], at::kFloat, {pl.kv_rows, p.Hkv, wt.size(2)});
    size_t ws_bytes = 0, ww_bytes = 0;
    void *ws = c.bytes(a[13], &ws_bytes), *ww = c.bytes(a[14], &ww_bytes);
    int32_t *status = c.status(a[15]);
    void *stream = c.stream();
    const bool want_lse = a[11] != Py_None || as_bool(a[12]);
    const Output out = output(c, a[10], Shape(pl, {p.Hq, p.D}), torch_type(p.out_dtype));
    Output lse;
    if (want_lse) lse = output(c, a[11], Shape(pl, {p.Hq}), at::kFloat);
    const int room = (int)wt.size(2);
    run([&] {
        return g_weights(&pl, q, po.k, po.v, po.ks, po.vs, bt, sl, out.ptr, static_cast<float *>(lse.ptr), wi, wo, room, ws,
                         ws_bytes, ww, ww_bytes, status, stream);
    });
    PyObject *l = want_lse ? lse.object() : Py_None;
    if (!want_lse) Py_INCREF(Py_None);
    Py_INCREF(to);
    return tuple_of({out.object(), l, to});
}

// plan, q, k_pages, v_pages, block_table, seq_lens, lam, norm_weight, eps,
// out_scale, k_scale, v_scale, out, lse, want_lse, workspace, status
PyObject *diff(PyObject *const *a) {
    Call c;
    const fd_plan_t &pl = *as_plan(a[0]);
    const fd_problem &p = pl.problem;  // two query rows a head; its B counts query rows
    const int heads = p.Hq / 2;
    if (pl.row_fold != (pl.q_len > 1 ? pl.q_len : 1)) throw Other();
    const void *q = query(c, pl, a[1], heads);
    const Pools po = pools(c, p, a[2], a[3], a[10], a[11]);
    const int32_t *bt = c.data<const int32_t>(a[4], at::kInt, {pl.kv_rows, p.max_blocks_per_seq});
    const int32_t *sl = c.data<const int32_t>(a[5], at::kInt, {pl.kv_rows});
    const float *lam = c.data<const float>(a[6], at::kFloat, {heads});
    const void *nw = nullptr;
    fd_dtype wt = FD_F32;
    if (a[7] != Py_None) {
        const at::ScalarType t = c.tensor(a[7]).scalar_type() == at::kFloat ? at::kFloat : torch_type(p.q_dtype);
        nw = c.data(a[7], t, {p.D});
        wt = fd_type(t);
    }
    const float eps = as_float(a[8]), scale = as_float(a[9]);
    size_t ws_bytes = 0;
    void *ws = c.bytes(a[15], &ws_bytes);
    int32_t *status = c.status(a[16]);
    void *stream = c.stream();
    const bool want_lse = a[13] != Py_None || as_bool(a[14]);
    const Output out = output(c, a[12], Shape(pl, {heads, p.D}), torch_type(p.out_dtype));
    Output lse;
    if (want_lse) lse = output(c, a[13], Shape(pl, {heads, 2}), at::kFloat);
    run([&] {
        return g_diff(&pl, q, po.k, po.v, po.ks, po.vs, bt, sl, lam, nw, wt, eps, scale, out.ptr,
                      static_cast<float *>(lse.ptr), ws, ws_bytes, status, stream);
    });
    PyObject *l = want_lse ? lse.object() : Py_None;
    if (!want_lse) Py_INCREF(Py_None);
    return tuple_of({out.object(), l});
}

// plan, q, k_pages, v_pages, block_table, kv_lens, q_lens, k_scale, v_scale,
// out, lse, want_lse, workspace, status
PyObject *cross(PyObject *const *a) {
    Call c;
    const void *at = PyLong_AsVoidPtr(a[0]);
    if (!at) throw Other();
    const fd_cross_plan_t &pl = *static_cast<const fd_cross_plan_t *>(at);
    const fd_problem &p = pl.problem;
    const bool flat = pl.tokens == 1 && c.tensor(a[1]).dim() == 3;
    const int64_t s4[4] = {pl.seqs, pl.tokens, p.Hq, p.D}, s3[3] = {pl.seqs, p.Hq, p.D};
    const at::IntArrayRef shape = flat ? at::IntArrayRef(s3, 3) : at::IntArrayRef(s4, 4);
    long long stride = 0;
    const void *q = c.rows(a[1], torch_type(p.q_dtype), shape, &stride);
    const Pools po = pools(c, p, a[2], a[3], a[7], a[8]);
    const int32_t *bt = c.data<const int32_t>(a[4], at::kInt, {pl.kv_rows, p.max_blocks_per_seq});
    const int32_t *kl = c.data<const int32_t>(a[5], at::kInt, {pl.kv_rows});
    const int32_t *ql = c.maybe<const int32_t>(a[6], at::kInt, {pl.seqs});
    size_t ws_bytes = 0;
    void *ws = c.bytes(a[12], &ws_bytes);
    int32_t *status = c.status(a[13]);
    void *stream = c.stream();
    const bool want_lse = a[10] != Py_None || as_bool(a[11]);
    const Output out = output(c, a[9], shape, torch_type(p.out_dtype));
    Output lse;
    if (want_lse) lse = output(c, a[10], shape.slice(0, shape.size() - 1), at::kFloat);
    run([&] {
        return g_cross(&pl, q, stride, ql, po.k, po.v, po.ks, po.vs, bt, kl, out.ptr, static_cast<float *>(lse.ptr), ws,
                       ws_bytes, status, stream);
    });
    PyObject *l = want_lse ? lse.object() : Py_None;
    if (!want_lse) Py_INCREF(Py_None);
    return tuple_of({out.object(), l});
}

// plan, q, k_pages, v_pages, prefix_table, prefix_lens, members, offsets,
// block_table, seq_lens, k_scale, v_scale, out, lse, want_lse, workspace, status
PyObject *prefix(PyObject *const *a) {
    Call c;
    const void *at = PyLong_AsVoidPtr(a[0]);
    if (!at) throw Other();
    const fd_prefix_plan_t &pp = *static_cast<const fd_prefix_plan_t *>(at);
    const fd_plan_t &pl = pp.own;
    const fd_problem &p = pp.shared.problem;  // its block table is the prefixes'
    const void *q = query(c, pl, a[1], p.Hq);
    const Pools po = pools(c, p, a[2], a[3], a[10], a[11]);
    const int32_t *pt = c.data<const int32_t>(a[4], at::kInt, {pp.prefixes, p.max_blocks_per_seq});
    const int32_t *ln = c.data<const int32_t>(a[5], at::kInt, {pp.prefixes});
    const int32_t *mb = c.data<const int32_t>(a[6], at::kInt, {pp.shared.seqs});
    const int32_t *of = c.data<const int32_t>(a[7], at::kInt, {pp.prefixes + 1});
    const int32_t *bt = c.data<const int32_t>(a[8], at::kInt, {pl.kv_rows, pl.problem.max_blocks_per_seq});
    const int32_t *sl = c.data<const int32_t>(a[9], at::kInt, {pl.kv_rows});
    size_t ws_bytes = 0;
    void *ws = c.bytes(a[15], &ws_bytes);
    int32_t *status = c.status(a[16]);
    void *stream = c.stream();
    const bool want_lse = a[13] != Py_None || as_bool(a[14]);
    const Output out = output(c, a[12], Shape(pl, {p.Hq, p.D}), torch_type(p.out_dtype));
    Output lse;
    if (want_lse) lse = output(c, a[13], Shape(pl, {p.Hq}), at::kFloat);
    run([&] {
        return g_prefix(&pp, q, po.k, po.v, po.ks, po.vs, pt, ln, mb, of, bt, sl, out.ptr, static_cast<float *>(lse.ptr),
                        ws, ws_bytes, status, stream);
    });
    PyObject *l = want_lse ? lse.object() : Py_None;
    if (!want_lse) Py_INCREF(Py_None);
    return tuple_of({out.object(), l});
}

PyObject *raise(fd_status status, const char *what) {
    PyObject *e = PyObject_CallFunction(g_error, "is", (int)status, what);
    if (e) {
        PyErr_SetObject(g_error, e);
        Py_DECREF(e);
    }
    return nullptr;
}

constexpr char kAppend[] = "fd_append_kv_norm", kEvict[] = "fd_evict_kv", kWeights[] = "fd_decode_paged_weights",
               kDiff[] = "fd_decode_paged_diff", kCross[] = "fd_cross_paged", kPrefix[] = "fd_decode_paged_prefix";

template <PyObject *(*F)(PyObject *const *), Py_ssize_t N, const char *NAME>
PyObject *entry(PyObject *, PyObject *const *args, Py_ssize_t n) {
    if (n == N) {
        try {
            return F(args);
        } catch (const Failed &f) {
            return raise(f.status, NAME);
        } catch (...) {
        }
    }
    PyErr_Clear();
    Py_RETURN_NONE;
}

PyObject *init(PyObject *, PyObject *args) {
    unsigned long long f[4];
    PyObject *error;
    if (!PyArg_ParseTuple(args, "KKKKO", &f[0], &f[1], &f[2], &f[3], &error)) return nullptr;
    Py_INCREF(error);
    Py_XDECREF(g_error);
    g_error = error;
    g_append = reinterpret_cast<decltype(g_append)>(f[0]);
    g_evict = reinterpret_cast<decltype(g_evict)>(f[1]);
    g_weights = reinterpret_cast<decltype(g_weights)>(f[2]);
    g_diff = reinterpret_cast<decltype(g_diff)>(f[3]);
    Py_RETURN_NONE;
}

PyObject *init_shared(PyObject *, PyObject *args) {
    unsigned long long f[2];
    if (!PyArg_ParseTuple(args, "KK", &f[0], &f[1])) return nullptr;
    g_cross = reinterpret_cast<decltype(g_cross)>(f[0]);
    g_prefix = reinterpret_cast<decltype(g_prefix)>(f[1]);
    Py_RETURN_NONE;
}

#define FD_FAST(name, f, n, what) \
    {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&entry<f, n, what>)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {{"init", init, METH_VARARGS, "addresses of libfd's entry points and the error class"},
                         {"init_shared", init_shared, METH_VARARGS, "addresses of fd_cross_paged and fd_decode_paged_prefix"},
                         FD_FAST("append_kv_norm", append, 19, kAppend),
                         FD_FAST("evict_kv", evict, 13, kEvict),
                         FD_FAST("decode_weights", weights, 16, kWeights),
                         FD_FAST("decode_diff", diff, 17, kDiff),
                         FD_FAST("cross", cross, 14, kCross),
                         FD_FAST("decode_prefix", prefix, 17, kPrefix),
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_fd_torch", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__fd_torch() { return PyModule_Create(&module); }
