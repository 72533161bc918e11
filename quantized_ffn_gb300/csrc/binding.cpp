// binding.cpp -- the Python binding of the 8-bit, sorting, bf16 and adapter entry points as
// a native module: it checks each tensor's type, shape, place and contiguity, makes
// the outputs that are not given, and calls the C ABI on the current (or given)
// stream.  A small call is bound by what the host does: the sort, dispatch and
// combine of one token take 6.5 us on the GPU, and 8.7 to 9.6 us of host time from
// here (26 us by ctypes and checks in Python).  No computation happens here.
//
// The C functions' addresses are given once by zffn.py (bind), so that there is one
// loader of the library.
#include <Python.h>

#include <ATen/ops/empty.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <optional>
#include <sstream>
#include <stdexcept>
#include <string>

#include "zffn.h"

namespace {

struct Api {
    decltype(&zffn_fp8_quantize) quantize;
    decltype(&zffn_fp8_dequant) dequant;
    decltype(&zffn_fp8_matmul) matmul;
    decltype(&zffn_fp8_experts) experts;
    decltype(&zffn_moe_sort) sort;
    decltype(&zffn_moe_dispatch) dispatch;
    decltype(&zffn_moe_combine) combine;
    decltype(&zffn_moe_combine_grad) combine_grad;
    decltype(&zffn_moe_swiglu_fp8) swiglu;
    decltype(&zffn_bf16_matmul) bf16_matmul;
    decltype(&zffn_bf16_matmul_grad_w) bf16_matmul_grad_w;
    decltype(&zffn_swiglu) plain_swiglu;
    decltype(&zffn_swiglu_grad) plain_swiglu_grad;
    decltype(&zffn_lora_add) lora_add;
    decltype(&zffn_lora_grad) lora_grad;
    decltype(&zffn_lora_work_bytes) lora_work_bytes;
} api{};
PyObject *g_fail = nullptr;   // (status, name) -> raises ZffnError

using Sizes = at::IntArrayRef;
using at::ScalarType;
constexpr ScalarType kF32 = at::kFloat, kBF16 = at::kBFloat16, kI32 = at::kInt, kF8 = at::kFloat8_e4m3fn, kU8 = at::kByte;

struct ValueError : std::runtime_error {
    using std::runtime_error::runtime_error;
};
struct Raised {};             // a Python exception is set

std::string shape_text(Sizes s) {
    std::ostringstream o;
    o << '(';
    for (size_t i = 0; i < s.size(); ++i) o << (i ? ", " : "") << s[i];
    o << (s.size() == 1 ? ",)" : ")");
    return o.str();
}

const at::Tensor &tensor(PyObject *o, const char *name) {
    if (!THPVariable_Check(o)) throw ValueError(std::string(name) + " must be a tensor");
    return THPVariable_Unpack(o);
}

// The current device (asked for once a call: entry() forgets it): the library's
// workspace, its error word and the launches are of this one.
thread_local int t_device = -1;
int current_device() {
    if (t_device < 0) t_device = c10::cuda::current_device();
    return t_device;
}
void on_device(int64_t device, const char *name) {
    if (device != current_device())
        throw ValueError(std::string(name) + " must be on the current device, cuda:" + std::to_string(current_device()) + ", got cuda:" +
                         std::to_string(device));
}

void *place(const at::Tensor &t, const char *name) {
    if (!t.is_cuda()) throw ValueError(std::string(name) + " must be a CUDA tensor");
    on_device(t.get_device(), name);
    if (!t.is_contiguous()) throw ValueError(std::string(name) + " must be contiguous");
    return const_cast<void *>(t.const_data_ptr());
}

// Address of a contiguous CUDA tensor of this type and shape.
void *ptr(const at::Tensor &t, const char *name, ScalarType type, Sizes shape) {
    if (t.sizes() != shape)
        throw ValueError(std::string(name) + " must have shape " + shape_text(shape) + ", got " + shape_text(t.sizes()));
    if (t.scalar_type() != type)
        throw ValueError(std::string(name) + " must be " + at::toString(type) + ", got " + at::toString(t.scalar_type()));
    return place(t, name);
}
void *ptr(PyObject *o, const char *name, ScalarType type, Sizes shape) { return ptr(tensor(o, name), name, type, shape); }
float *f32(PyObject *o, const char *name, Sizes shape) { return static_cast<float *>(ptr(o, name, kF32, shape)); }
int32_t *i32(PyObject *o, const char *name, Sizes shape) { return static_cast<int32_t *>(ptr(o, name, kI32, shape)); }
// e4m3 bytes, as float8_e4m3fn or uint8
void *f8(PyObject *o, const char *name, Sizes shape) {
    const at::Tensor &t = tensor(o, name);
    return ptr(t, name, t.scalar_type() == kU8 ? kU8 : kF8, shape);
}
int dtype_of(const at::Tensor &t, const char *name) {
    if (t.scalar_type() == kF32) return ZFFN_DT_F32;
    if (t.scalar_type() == kBF16) return ZFFN_DT_BF16;
    throw ValueError(std::string(name) + " must be torch.float32 or torch.bfloat16, got " + at::toString(t.scalar_type()));
}
ScalarType type_of(PyObject *dtype) {
    if (!THPDtype_Check(dtype)) throw ValueError("dtype must be a torch.dtype");
    return reinterpret_cast<THPDtype *>(dtype)->scalar_type;
}
void dims(const at::Tensor &t, const char *name, int n) {
    if (t.dim() != n) throw ValueError(std::string(name) + " must have " + std::to_string(n) + " dimensions, got " + shape_text(t.sizes()));
}

// The stream of a call: the given one, else the current one.  While it lives a given
// stream is the current one, so that the outputs made for the call come from that
// stream's memory (a block that another stream has let go of may still be written by
// kernels there).
struct Stream {
    std::optional<c10::cuda::CUDAStreamGuard> guard;
    void *s;
    explicit Stream(PyObject *stream) {
        if (stream == Py_None) {
            s = c10::cuda::getCurrentCUDAStream().stream();
            return;
        }
        PyObject *h = PyObject_GetAttrString(stream, "cuda_stream");
        if (!h) throw Raised{};
        s = PyLong_AsVoidPtr(h);
        Py_DECREF(h);
        if (PyErr_Occurred()) throw Raised{};
        if (PyObject *d = PyObject_GetAttrString(stream, "device_index")) {
            const long device = PyLong_AsLong(d);
            Py_DECREF(d);
            if (PyErr_Occurred()) throw Raised{};
            on_device(device, "stream");
        } else {
            PyErr_Clear();   // (a bare handle: the current device's)
        }
        guard.emplace(c10::cuda::getStreamFromExternal(static_cast<cudaStream_t>(s), current_device()));
    }
};

// The given output, or a new one like `like` (kept alive in `made`).
struct Output {
    at::Tensor made;
    PyObject *given;
    const at::Tensor &t;
    Output(PyObject *o, const char *name, Sizes shape, ScalarType type, const at::Tensor &like)
        : made(o == Py_None ? at::empty(shape, like.options().dtype(type)) : at::Tensor()),
          given(o == Py_None ? nullptr : o), t(given ? tensor(o, name) : made) {}
    explicit Output(at::Tensor m) : made(std::move(m)), given(nullptr), t(made) {}
    Output(const Output &) = delete;   // (t refers to made)
    PyObject *object() const {
        if (!given) return THPVariable_Wrap(made);
        Py_INCREF(given);
        return given;
    }
};

// A contiguous part of a tensor's memory, from element `at` on.
at::Tensor part(const at::Tensor &of, int64_t at, Sizes shape) {
    at::Tensor t = at::detail::make_tensor<c10::TensorImpl>(c10::Storage(of.storage()), of.key_set(), of.dtype());
    t.unsafeGetTensorImpl()->set_storage_offset(at);
    t.unsafeGetTensorImpl()->set_sizes_contiguous(shape);
    return t;
}

template <typename F>
void call(const char *name, F f) {
    zffn_status st;
    Py_BEGIN_ALLOW_THREADS
    st = f();
    Py_END_ALLOW_THREADS
    if (st == ZFFN_OK) return;
    Py_XDECREF(PyObject_CallFunction(g_fail, "is", (int)st, name));
    throw Raised{};
}

int64_t blocks(int64_t n) { return (n + 127) / 128; }
int to_int(PyObject *o) {
    const long v = PyLong_AsLong(o);
    if (v == -1 && PyErr_Occurred()) throw Raised{};
    if (v < INT32_MIN || v > INT32_MAX) throw ValueError("an integer argument is out of range");
    return (int)v;
}
int narrow(int64_t v, const char *name) {
    if (v > INT32_MAX) throw ValueError(std::string(name) + " is too large");
    return (int)v;
}
PyObject *pair(PyObject *a, PyObject *b) {
    PyObject *t = a && b ? PyTuple_New(2) : nullptr;
    if (!t) {
        Py_XDECREF(a);
        Py_XDECREF(b);
        throw Raised{};
    }
    PyTuple_SET_ITEM(t, 0, a);
    PyTuple_SET_ITEM(t, 1, b);
    return t;
}
PyObject *plan_item(PyObject *plan, int i) {
    if (!PyTuple_Check(plan) || PyTuple_GET_SIZE(plan) != 3) throw ValueError("plan must be a MoePlan");
    return PyTuple_GET_ITEM(plan, i);
}

// (x, block_rows, q, scale, stream) -> (q, scale)
PyObject *fp8_quantize(PyObject *const *a) {
    const at::Tensor &x = tensor(a[0], "x");
    dims(x, "x", 2);
    const int block_rows = to_int(a[1]);
    if (block_rows != 1 && block_rows != 128) throw ValueError("block_rows must be 1 or 128");
    const int64_t R = x.size(0), C = x.size(1);
    const int dtype = dtype_of(x, "x");
    const void *px = place(x, "x");
    const int64_t sc[2] = {(R + block_rows - 1) / block_rows, blocks(C)};
    const Stream on(a[4]);
    Output q(a[2], "q", x.sizes(), kF8, x), s(a[3], "scale", sc, kF32, x);
    void *pq = ptr(q.t, "q", q.t.scalar_type() == kU8 ? kU8 : kF8, x.sizes());
    float *ps = static_cast<float *>(ptr(s.t, "scale", kF32, sc));
    call("zffn_fp8_quantize", [&] { return api.quantize(dtype, px, pq, ps, R, C, block_rows, on.s); });
    return pair(q.object(), s.object());
}

// (q, scale, block_rows, out, stream) -> out
PyObject *fp8_dequant(PyObject *const *a) {
    const at::Tensor &q = tensor(a[0], "q");
    dims(q, "q", 2);
    const int block_rows = to_int(a[2]);
    if (block_rows != 1 && block_rows != 128) throw ValueError("block_rows must be 1 or 128");
    const int64_t R = q.size(0), C = q.size(1);
    const int64_t sc[2] = {(R + block_rows - 1) / block_rows, blocks(C)};
    const void *pq = f8(a[0], "q", q.sizes());
    const float *ps = f32(a[1], "scale", sc);
    const Stream on(a[4]);
    Output out(a[3], "out", q.sizes(), kF32, q);
    float *po = static_cast<float *>(ptr(out.t, "out", kF32, q.sizes()));
    call("zffn_fp8_dequant", [&] { return api.dequant(pq, ps, po, R, C, block_rows, on.s); });
    return out.object();
}

// (a, a_scale, w, w_scale, offsets, y, dtype, stream) -> y
PyObject *fp8_matmul(PyObject *const *a) {
    const at::Tensor &x = tensor(a[0], "a"), &w = tensor(a[2], "w");
    const bool grouped = a[4] != Py_None;
    dims(x, "a", 2);
    dims(w, "w", grouped ? 3 : 2);
    const int64_t M = x.size(0), K = x.size(1), N = w.size(-2), E = grouped ? w.size(0) : 1;
    const int64_t ws[3] = {E, N, K}, ss[3] = {E, blocks(N), blocks(K)}, as[2] = {M, blocks(K)}, ys[2] = {M, N}, os[1] = {E + 1};
    const int skip = grouped ? 0 : 1;
    const void *px = f8(a[0], "a", x.sizes());
    const float *pxs = f32(a[1], "a_scale", as);
    const void *pw = f8(a[2], "w", Sizes(ws + skip, 3 - skip));
    const float *pws = f32(a[3], "w_scale", Sizes(ss + skip, 3 - skip));
    const int32_t *po = grouped ? i32(a[4], "offsets", os) : nullptr;
    const Stream on(a[7]);
    Output y(a[5], "y", ys, a[5] == Py_None ? type_of(a[6]) : kF32, x);
    const int yd = dtype_of(y.t, "y");
    void *py = ptr(y.t, "y", y.t.scalar_type(), ys);
    const int m = narrow(M, "M"), n = narrow(N, "N"), k = narrow(K, "K"), e = narrow(E, "E");
    call("zffn_fp8_matmul", [&] { return api.matmul(px, pxs, pw, pws, po, yd, py, m, n, k, e, on.s); });
    return y.object();
}

// the stacked (or single) gate, up and down weights at a[0 .. 5]
struct Experts {
    const void *wg, *wu, *wd;
    const float *sg, *su, *sd;
    int64_t E, I;
    Experts(PyObject *const *a, bool stacked, int64_t H) {
        const at::Tensor &g = tensor(a[0], "Wg");
        dims(g, "Wg", stacked ? 3 : 2);
        E = stacked ? g.size(0) : 1;
        I = g.size(-2);
        const int skip = stacked ? 0 : 1;
        const int64_t up[3] = {E, I, H}, down[3] = {E, H, I}, su_[3] = {E, blocks(I), blocks(H)}, sd_[3] = {E, blocks(H), blocks(I)};
        auto cut = [&](const int64_t *s) { return Sizes(s + skip, 3 - skip); };
        wg = f8(a[0], "Wg", cut(up));
        sg = f32(a[1], "sg", cut(su_));
        wu = f8(a[2], "Wu", cut(up));
        su = f32(a[3], "su", cut(su_));
        wd = f8(a[4], "Wd", cut(down));
        sd = f32(a[5], "sd", cut(sd_));
    }
};

// (a, a_scale, Wg, sg, Wu, su, Wd, sd, offsets, y, dtype, stream) -> y
PyObject *fp8_experts(PyObject *const *a) {
    const at::Tensor &x = tensor(a[0], "a");
    dims(x, "a", 2);
    const bool grouped = a[8] != Py_None;
    const int64_t P = x.size(0), H = x.size(1);
    const Experts w(a + 2, grouped, H);
    const int64_t as[2] = {P, blocks(H)}, os[1] = {w.E + 1};
    const void *px = f8(a[0], "a", x.sizes());
    const float *pxs = f32(a[1], "a_scale", as);
    const int32_t *po = grouped ? i32(a[8], "offsets", os) : nullptr;
    const Stream on(a[11]);
    Output y(a[9], "y", x.sizes(), a[9] == Py_None ? type_of(a[10]) : kF32, x);
    const int yd = dtype_of(y.t, "y");
    void *py = ptr(y.t, "y", y.t.scalar_type(), x.sizes());
    const int p = narrow(P, "P"), h = narrow(H, "H"), i = narrow(w.I, "I"), e = narrow(w.E, "E");
    call("zffn_fp8_experts", [&] { return api.experts(px, pxs, po, w.wg, w.sg, w.wu, w.su, w.wd, w.sd, yd, py, p, h, i, e, on.s); });
    return y.object();
}

// (expert_ids, E, plan, stream) -> (row_slot, slot_row, offsets)
PyObject *moe_sort(PyObject *const *a) {
    const at::Tensor &ids = tensor(a[0], "expert_ids");
    dims(ids, "expert_ids", 2);
    const int64_t T = ids.size(0), k = ids.size(1);
    const int E = to_int(a[1]);
    const int64_t rs[1] = {T * k}, os[1] = {E < 0 ? 0 : (int64_t)E + 1};
    const int32_t *pi = i32(a[0], "expert_ids", ids.sizes());
    const bool given = a[2] != Py_None;
    const Stream on(a[3]);
    // (a new plan is one allocation: each costs 1.2 us of host time, where the sort of one
    // token takes 3 us on the GPU)
    const int64_t P = T * k, each = (P + 3) / 4 * 4;
    const at::Tensor all = given ? at::Tensor() : at::empty({2 * each + os[0]}, ids.options());
    const Output row_slot = given ? Output(plan_item(a[2], 0), "row_slot", rs, kI32, ids) : Output(part(all, 0, rs));
    const Output slot_row = given ? Output(plan_item(a[2], 1), "slot_row", ids.sizes(), kI32, ids) : Output(part(all, each, ids.sizes()));
    const Output offsets = given ? Output(plan_item(a[2], 2), "offsets", os, kI32, ids) : Output(part(all, 2 * each, os));
    int32_t *pr = static_cast<int32_t *>(ptr(row_slot.t, "row_slot", kI32, rs)),
            *ps = static_cast<int32_t *>(ptr(slot_row.t, "slot_row", kI32, ids.sizes())),
            *po = static_cast<int32_t *>(ptr(offsets.t, "offsets", kI32, os));
    const int t = narrow(T, "T"), kk = narrow(k, "top_k");
    call("zffn_moe_sort", [&] { return api.sort(pi, pr, ps, po, t, E, kk, on.s); });
    PyObject *out = PyTuple_New(3);
    if (!out) throw Raised{};
    const Output *items[3] = {&row_slot, &slot_row, &offsets};
    for (int i = 0; i < 3; ++i) {
        PyObject *o = items[i]->object();
        if (!o) {
            Py_DECREF(out);
            throw Raised{};
        }
        PyTuple_SET_ITEM(out, i, o);
    }
    return out;
}

// a plan's slot_row, and its T and top_k
const at::Tensor &slots(PyObject *plan) {
    const at::Tensor &s = tensor(plan_item(plan, 1), "slot_row");
    dims(s, "slot_row", 2);
    return s;
}

// (x, plan, scale, out, scale_out, stream) -> out, or (out, scale_out)
PyObject *moe_dispatch(PyObject *const *a) {
    const at::Tensor &x = tensor(a[0], "x"), &s = slots(a[1]);
    dims(x, "x", 2);
    const int64_t T = x.size(0), H = x.size(1), k = s.size(1), P = T * k;
    const int64_t rs[1] = {P}, ss[2] = {T, k}, xs[2] = {P, H};
    const void *px = place(x, "x");
    const int32_t *pr = i32(plan_item(a[1], 0), "row_slot", rs), *ps = i32(plan_item(a[1], 1), "slot_row", ss);
    const Stream on(a[5]);
    Output out(a[3], "out", xs, x.scalar_type(), x);
    void *po = ptr(out.t, "out", x.scalar_type(), xs);
    const int t = narrow(T, "T"), kk = narrow(k, "top_k");
    const int64_t bytes = H * (int64_t)x.element_size();
    if (a[2] == Py_None) {
        call("zffn_moe_dispatch", [&] { return api.dispatch(px, bytes, nullptr, 0, pr, ps, po, nullptr, t, kk, on.s); });
        return out.object();
    }
    const at::Tensor &sc = tensor(a[2], "scale");
    dims(sc, "scale", 2);
    const int64_t C = sc.size(1), cs[2] = {T, C}, cos[2] = {P, C};
    const float *pc = f32(a[2], "scale", cs);
    Output sout(a[4], "scale_out", cos, kF32, x);
    float *pco = static_cast<float *>(ptr(sout.t, "scale_out", kF32, cos));
    call("zffn_moe_dispatch", [&] { return api.dispatch(px, bytes, pc, C, pr, ps, po, pco, t, kk, on.s); });
    return pair(out.object(), sout.object());
}

// (rows, plan, weights, y, accumulate, stream) -> y
PyObject *moe_combine(PyObject *const *a) {
    const at::Tensor &r = tensor(a[0], "rows"), &s = slots(a[1]);
    dims(r, "rows", 2);
    const int64_t T = s.size(0), k = s.size(1), H = r.size(1), rs[2] = {T * k, H}, ys[2] = {T, H};
    const int accumulate = PyObject_IsTrue(a[4]);
    if (accumulate < 0) throw Raised{};
    if (accumulate && a[3] == Py_None) throw ValueError("accumulate=True needs y");
    const int dtype = dtype_of(r, "rows");
    const void *pr = ptr(r, "rows", r.scalar_type(), rs);
    const int32_t *ps = i32(plan_item(a[1], 1), "slot_row", s.sizes());
    const float *pw = a[2] == Py_None ? nullptr : f32(a[2], "weights", s.sizes());
    const Stream on(a[5]);
    Output y(a[3], "y", ys, kF32, r);
    float *py = static_cast<float *>(ptr(y.t, "y", kF32, ys));
    const int t = narrow(T, "T"), h = narrow(H, "H"), kk = narrow(k, "top_k");
    call("zffn_moe_combine", [&] { return api.combine(dtype, pr, ps, pw, py, t, h, kk, accumulate, on.s); });
    return y.object();
}

// (dy, rows, plan, weights, drows, dweights, stream) -> (drows, dweights)
PyObject *moe_combine_grad(PyObject *const *a) {
    const at::Tensor &r = tensor(a[1], "rows"), &s = slots(a[2]);
    dims(r, "rows", 2);
    const int64_t T = s.size(0), k = s.size(1), H = r.size(1), rs[2] = {T * k, H}, ys[2] = {T, H}, ns[1] = {T * k};
    const int dtype = dtype_of(r, "rows");
    const float *pd = f32(a[0], "dy", ys);
    const void *pr = ptr(r, "rows", r.scalar_type(), rs);
    const int32_t *pn = i32(plan_item(a[2], 0), "row_slot", ns), *ps = i32(plan_item(a[2], 1), "slot_row", s.sizes());
    const float *pw = f32(a[3], "weights", s.sizes());
    const Stream on(a[6]);
    Output dr(a[4], "drows", rs, r.scalar_type(), r), dw(a[5], "dweights", s.sizes(), kF32, r);
    void *pdr = ptr(dr.t, "drows", r.scalar_type(), rs);
    float *pdw = static_cast<float *>(ptr(dw.t, "dweights", kF32, s.sizes()));
    const int t = narrow(T, "T"), h = narrow(H, "H"), kk = narrow(k, "top_k");
    call("zffn_moe_combine_grad", [&] { return api.combine_grad(dtype, pd, pr, pn, ps, pw, pdr, pdw, t, h, kk, on.s); });
    return pair(dr.object(), dw.object());
}

// (x, expert_ids, expert_weights, Wg, sg, Wu, su, Wd, sd, y, accumulate, stream) -> y
PyObject *moe_swiglu_fp8(PyObject *const *a) {
    const at::Tensor &x = tensor(a[0], "x"), &ids = tensor(a[1], "expert_ids");
    dims(x, "x", 2);
    dims(ids, "expert_ids", 2);
    const int64_t T = x.size(0), H = x.size(1), k = ids.size(1), ss[2] = {T, k};
    const int accumulate = PyObject_IsTrue(a[10]);
    if (accumulate < 0) throw Raised{};
    if (accumulate && a[9] == Py_None) throw ValueError("accumulate=True needs y");
    const Experts w(a + 3, true, H);
    const void *px = ptr(x, "x", kBF16, x.sizes());
    const int32_t *pi = i32(a[1], "expert_ids", ss);
    const float *pw = f32(a[2], "expert_weights", ss);
    const Stream on(a[11]);
    Output y(a[9], "y", x.sizes(), kF32, x);
    float *py = static_cast<float *>(ptr(y.t, "y", kF32, x.sizes()));
    const int t = narrow(T, "T"), h = narrow(H, "H"), i = narrow(w.I, "I"), e = narrow(w.E, "E"), kk = narrow(k, "top_k");
    call("zffn_moe_swiglu_fp8", [&] { return api.swiglu(px, pi, pw, w.wg, w.sg, w.wu, w.su, w.wd, w.sd, py, t, h, i, e, kk, accumulate, on.s); });
    return y.object();
}

// An output that may be given: its type is the given one's, else `type`.
ScalarType given_type(PyObject *o, const char *name, ScalarType type) {
    return o == Py_None ? type : tensor(o, name).scalar_type();
}

// (a, w, offsets, transposed, y, dtype, stream) -> y
PyObject *bf16_matmul(PyObject *const *a) {
    const at::Tensor &x = tensor(a[0], "a"), &w = tensor(a[1], "w");
    const bool grouped = a[2] != Py_None;
    const int transposed = PyObject_IsTrue(a[3]);
    if (transposed < 0) throw Raised{};
    dims(x, "a", 2);
    dims(w, "w", grouped ? 3 : 2);
    const int64_t M = x.size(0), K = x.size(1), N = w.size(transposed ? -1 : -2), E = grouped ? w.size(0) : 1;
    const int64_t ws[3] = {E, transposed ? K : N, transposed ? N : K}, ys[2] = {M, N}, os[1] = {E + 1};
    const int skip = grouped ? 0 : 1;
    const void *px = ptr(x, "a", kBF16, x.sizes());
    const void *pw = ptr(w, "w", kBF16, Sizes(ws + skip, 3 - skip));
    const int32_t *po = grouped ? i32(a[2], "offsets", os) : nullptr;
    const Stream on(a[6]);
    Output y(a[4], "y", ys, given_type(a[4], "y", type_of(a[5])), x);
    const int yd = dtype_of(y.t, "y");
    void *py = ptr(y.t, "y", y.t.scalar_type(), ys);
    const int m = narrow(M, "M"), n = narrow(N, "N"), k = narrow(K, "K"), e = narrow(E, "E");
    call("zffn_bf16_matmul", [&] { return api.bf16_matmul(px, pw, po, transposed, yd, py, m, n, k, e, on.s); });
    return y.object();
}

// (dy, a, offsets, dw, dtype, stream) -> dw
PyObject *bf16_matmul_grad_w(PyObject *const *a) {
    const at::Tensor &d = tensor(a[0], "dy"), &x = tensor(a[1], "a");
    dims(d, "dy", 2);
    dims(x, "a", 2);
    const bool grouped = a[2] != Py_None;
    const int64_t M = x.size(0), K = x.size(1), N = d.size(1), ds[2] = {M, N};
    int64_t E = 1;
    if (grouped) {
        const at::Tensor &o = tensor(a[2], "offsets");
        dims(o, "offsets", 1);
        E = o.size(0) - 1;
        if (E < 1) throw ValueError("offsets must have shape (E + 1,)");
    }
    const int64_t ws[3] = {E, N, K}, os[1] = {E + 1};
    const int skip = grouped ? 0 : 1;
    const void *pd = ptr(d, "dy", kBF16, ds), *px = ptr(x, "a", kBF16, x.sizes());
    const int32_t *po = grouped ? i32(a[2], "offsets", os) : nullptr;
    const Stream on(a[5]);
    Output dw(a[3], "dw", Sizes(ws + skip, 3 - skip), given_type(a[3], "dw", type_of(a[4])), x);
    const int wd = dtype_of(dw.t, "dw");
    void *pw = ptr(dw.t, "dw", dw.t.scalar_type(), Sizes(ws + skip, 3 - skip));
    const int m = narrow(M, "M"), n = narrow(N, "N"), k = narrow(K, "K"), e = narrow(E, "E");
    call("zffn_bf16_matmul_grad_w", [&] { return api.bf16_matmul_grad_w(pd, px, po, wd, pw, m, n, k, e, on.s); });
    return dw.object();
}

// (gu, h, stream) -> h
PyObject *swiglu(PyObject *const *a) {
    const at::Tensor &gu = tensor(a[0], "gu");
    dims(gu, "gu", 2);
    if (gu.size(1) % 2) throw ValueError("gu must have an even number of columns");
    const int64_t R = gu.size(0), I = gu.size(1) / 2, hs[2] = {R, I};
    const int dtype = dtype_of(gu, "gu");
    const void *pg = place(gu, "gu");
    const Stream on(a[2]);
    Output h(a[1], "h", hs, gu.scalar_type(), gu);
    void *ph = ptr(h.t, "h", gu.scalar_type(), hs);
    call("zffn_swiglu", [&] { return api.plain_swiglu(dtype, pg, ph, R, I, on.s); });
    return h.object();
}

// (dh, gu, dgu, stream) -> dgu
PyObject *swiglu_grad(PyObject *const *a) {
    const at::Tensor &gu = tensor(a[1], "gu");
    dims(gu, "gu", 2);
    if (gu.size(1) % 2) throw ValueError("gu must have an even number of columns");
    const int64_t R = gu.size(0), I = gu.size(1) / 2, hs[2] = {R, I};
    const int dtype = dtype_of(gu, "gu");
    const void *pg = place(gu, "gu"), *pd = ptr(a[0], "dh", gu.scalar_type(), hs);
    const Stream on(a[3]);
    Output out(a[2], "dgu", gu.sizes(), gu.scalar_type(), gu);
    void *po = ptr(out.t, "dgu", gu.scalar_type(), gu.sizes());
    call("zffn_swiglu_grad", [&] { return api.plain_swiglu_grad(dtype, pd, pg, po, R, I, on.s); });
    return out.object();
}

// What both adapter calls check: x [T, K], A [L, r, K], B [L, N, r], the plan of top_k = 1, the scales.
struct Lora {
    int64_t T, K, L, r, N;
    const void *x, *A, *B;
    const int32_t *row_slot, *slot_row, *offsets;
    const float *scale;
    Lora(PyObject *x_, PyObject *A_, PyObject *B_, PyObject *plan, PyObject *scale_) {
        const at::Tensor &tx = tensor(x_, "x"), &ta = tensor(A_, "A"), &tb = tensor(B_, "B");
        dims(tx, "x", 2);
        dims(ta, "A", 3);
        dims(tb, "B", 3);
        T = tx.size(0), K = tx.size(1), L = ta.size(0), r = ta.size(1), N = tb.size(1);
        const int64_t as[3] = {L, r, K}, bs[3] = {L, N, r}, rs[1] = {T}, ss[2] = {T, 1}, os[1] = {L + 1}, ls[1] = {L};
        x = ptr(tx, "x", kBF16, tx.sizes());
        A = ptr(ta, "A", kBF16, as);
        B = ptr(tb, "B", kBF16, bs);
        row_slot = i32(plan_item(plan, 0), "row_slot", rs);
        slot_row = i32(plan_item(plan, 1), "slot_row", ss);
        offsets = i32(plan_item(plan, 2), "offsets", os);
        scale = scale_ == Py_None ? nullptr : f32(scale_, "scale", ls);
        narrow(T, "T"), narrow(K, "K"), narrow(L, "L"), narrow(r, "r"), narrow(N, "N");
    }
};

// What a call works in, from the current stream's memory.
struct Work {
    at::Tensor t;
    void *at = nullptr;
    Work(const Lora &p, int backward, const at::Tensor &like) {
        if (const size_t bytes = api.lora_work_bytes((int)p.T, (int)p.r, (int)p.L, backward)) {
            t = at::empty({(int64_t)bytes}, like.options().dtype(kU8));
            at = t.data_ptr();
        }
    }
};

// (x, A, B, plan, scale, base, out, v, dtype, stream) -> (out, v)
PyObject *lora_add(PyObject *const *a) {
    const Lora p(a[0], a[1], a[2], a[3], a[4]);
    const at::Tensor &x = tensor(a[0], "x");
    const int64_t os[2] = {p.T, p.N}, vs[2] = {p.T, p.r};
    const ScalarType type = given_type(a[5], "base", given_type(a[6], "out", type_of(a[8])));
    const void *pb = a[5] == Py_None ? nullptr : ptr(a[5], "base", type, os);
    const Stream on(a[9]);
    Output out(a[6], "out", os, type, x), v(a[7], "v", vs, kF32, x);
    const int dtype = dtype_of(out.t, "out");
    void *po = ptr(out.t, "out", type, os);
    float *pv = static_cast<float *>(ptr(v.t, "v", kF32, vs));
    const Work work(p, 0, x);
    call("zffn_lora_add", [&] {
        return api.lora_add(p.x, p.A, p.B, p.scale, p.row_slot, p.slot_row, p.offsets, dtype, pb, po, pv, work.at, (int)p.T, (int)p.N, (int)p.K, (int)p.r,
                            (int)p.L, on.s);
    });
    return pair(out.object(), v.object());
}

// (dy, x, v, A, B, plan, scale, base, dx, dA, dB, dtype, stream) -> (dx, dA, dB)
PyObject *lora_grad(PyObject *const *a) {
    const Lora p(a[1], a[3], a[4], a[5], a[6]);
    const at::Tensor &x = tensor(a[1], "x"), &tA = tensor(a[3], "A"), &tB = tensor(a[4], "B");
    const int64_t ds[2] = {p.T, p.N}, vs[2] = {p.T, p.r};
    const void *pd = ptr(a[0], "dy", kBF16, ds);
    const float *pv = f32(a[2], "v", vs);
    const ScalarType type = given_type(a[7], "base", given_type(a[8], "dx", type_of(a[11])));
    const ScalarType wtype = given_type(a[9], "dA", given_type(a[10], "dB", type_of(a[11])));
    const void *pb = a[7] == Py_None ? nullptr : ptr(a[7], "base", type, x.sizes());
    const Stream on(a[12]);
    Output dx(a[8], "dx", x.sizes(), type, x), dA(a[9], "dA", tA.sizes(), wtype, x), dB(a[10], "dB", tB.sizes(), wtype, x);
    const Output dv(Py_None, "dv", vs, kF32, x);
    const int xd = dtype_of(dx.t, "dx"), wd = dtype_of(dA.t, "dA");
    void *px = ptr(dx.t, "dx", type, x.sizes()), *pA = ptr(dA.t, "dA", wtype, tA.sizes()), *pB = ptr(dB.t, "dB", wtype, tB.sizes());
    float *pdv = static_cast<float *>(ptr(dv.t, "dv", kF32, vs));
    const Work work(p, 1, x);
    call("zffn_lora_grad", [&] {
        return api.lora_grad(pd, p.x, pv, p.A, p.B, p.scale, p.row_slot, p.slot_row, p.offsets, xd, pb, px, wd, pA, pB, pdv, work.at, (int)p.T, (int)p.N,
                             (int)p.K, (int)p.r, (int)p.L, on.s);
    });
    PyObject *out = PyTuple_New(3);
    if (!out) throw Raised{};
    const Output *items[3] = {&dx, &dA, &dB};
    for (int i = 0; i < 3; ++i) {
        PyObject *o = items[i]->object();
        if (!o) {
            Py_DECREF(out);
            throw Raised{};
        }
        PyTuple_SET_ITEM(out, i, o);
    }
    return out;
}

template <PyObject *(*F)(PyObject *const *), int N>
PyObject *entry(PyObject *, PyObject *const *args, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    if (n != N) {
        PyErr_Format(PyExc_TypeError, "%d arguments expected, got %zd", N, n);
        return nullptr;
    }
    t_device = -1;
    try {
        return F(args);
    } catch (const ValueError &e) {
        PyErr_SetString(PyExc_ValueError, e.what());
    } catch (const Raised &) {
        if (!PyErr_Occurred()) PyErr_SetString(PyExc_RuntimeError, "the call failed");
    }
    return nullptr;
    END_HANDLE_TH_ERRORS
}

// bind(fail, address of each function in Api's order)
PyObject *bind(PyObject *, PyObject *const *args, Py_ssize_t n) {
    constexpr Py_ssize_t count = sizeof(Api) / sizeof(void *);
    if (n != count + 1) {
        PyErr_SetString(PyExc_TypeError, "bind takes a callable and the functions' addresses");
        return nullptr;
    }
    void *p[count];
    for (Py_ssize_t i = 0; i < count; ++i) {
        p[i] = PyLong_AsVoidPtr(args[i + 1]);
        if (PyErr_Occurred()) return nullptr;
    }
    static_assert(sizeof(p) == sizeof(api), "one address for each function");
    memcpy(&api, p, sizeof(api));
    Py_INCREF(args[0]);
    Py_XSETREF(g_fail, args[0]);
    Py_RETURN_NONE;
}

#define ENTRY(f, n) {#f, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(entry<f, n>)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {
    ENTRY(fp8_quantize, 5), ENTRY(fp8_dequant, 5), ENTRY(fp8_matmul, 8), ENTRY(fp8_experts, 12), ENTRY(moe_sort, 4),
    ENTRY(moe_dispatch, 6), ENTRY(moe_combine, 6), ENTRY(moe_combine_grad, 7), ENTRY(moe_swiglu_fp8, 12),
    ENTRY(bf16_matmul, 7), ENTRY(bf16_matmul_grad_w, 6), ENTRY(swiglu, 3), ENTRY(swiglu_grad, 4), ENTRY(lora_add, 10), ENTRY(lora_grad, 13),
    {"bind", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(bind)), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_zffn_native", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__zffn_native() {
    return PyModule_Create(&module);
}
