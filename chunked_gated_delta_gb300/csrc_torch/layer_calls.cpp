// layer_calls.cpp -- the Python calls of the served layer's operators (step,
// rms_norm, linear): argument checks, output allocation and the C-ABI call.
//
// A decode step makes these calls once per layer and token, at a few
// microseconds of kernel time each.  Checked and marshalled in Python they take
// 9 to 14 us of host time on the Grace cores; here they take 2.2 to 5.0, by
// the outputs that they allocate; the launch itself is most of 2.  The module is
// plain CPython API on torch's tensors; binding.py holds the documented functions
// that call it.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cmath>
#include <cstring>
#include <optional>
#include <string>

#include "../../include/kda.h"

namespace {

PyObject* g_error = nullptr;  // KdaError

struct Refused {  // a Python exception to raise: its type and text
    PyObject* type;
    std::string text;
};
[[noreturn]] void refuse(std::string text) { throw Refused{PyExc_TypeError, std::move(text)}; }
inline void need(bool ok, const char* text) {
    if (!ok) refuse(text);
}

const at::Tensor& tensor(PyObject* o, const char* name) {
    if (!THPVariable_Check(o)) refuse(std::string(name) + " must be a tensor");
    return THPVariable_Unpack(o);
}
const at::Tensor* optional(PyObject* o, const char* name) { return o == Py_None ? nullptr : &tensor(o, name); }
void* address(const at::Tensor* t) { return t ? t->data_ptr() : nullptr; }

bool same_shape(const at::Tensor& t, std::initializer_list<int64_t> shape) {
    return t.sizes() == at::IntArrayRef(shape.begin(), shape.size());
}

// A tensor of another GPU would reach the kernel as an address of this one.
void need_one_device(const at::Tensor& first, std::initializer_list<const at::Tensor*> others) {
    for (const at::Tensor* t : others)
        need(!t || t->device() == first.device(), "all tensors must be on one device");
}

// Elements between consecutive token rows of [B, T, ...] (0: contiguous).
int64_t token_stride(const char* name, const at::Tensor& t) {
    if (t.is_contiguous()) return 0;
    int64_t inner = 1;
    for (int64_t i = t.dim() - 1; i >= 2; --i) {
        if (t.size(i) != 1 && t.stride(i) != inner)
            refuse(std::string(name) + ": the heads of a token must be contiguous");
        inner *= t.size(i);
    }
    const int64_t B = t.size(0), T = t.size(1);
    if (B * T <= 1) return 0;
    const int64_t step = T > 1 ? t.stride(1) : t.stride(0);
    if (step < inner || (B > 1 && t.stride(0) != T * step))
        refuse(std::string(name) + ": token rows must be equally spaced over [B, T] and not overlap");
    return step;
}

// Elements between consecutive rows of [..., dim] (0: contiguous).
int64_t row_stride(const char* name, const at::Tensor& t, int64_t dim) {
    if (t.is_contiguous()) return 0;
    if (dim != 1 && t.stride(-1) != 1) refuse(std::string(name) + ": the elements of a row must be contiguous");
    int64_t step = -1, rows = 1;
    for (int64_t i = t.dim() - 2; i >= 0; --i) {
        if (t.size(i) == 1) continue;
        if (step < 0) step = t.stride(i);
        else if (t.stride(i) != step * rows) refuse(std::string(name) + ": rows must be equally spaced");
        rows *= t.size(i);
    }
    if (step >= 0 && step < dim) refuse(std::string(name) + ": rows must not overlap");
    return step < 0 ? 0 : step;
}

int dtype_code(at::ScalarType t) {
    switch (t) {
    case at::kBFloat16: return KDA_DTYPE_BF16;
    case at::kHalf: return KDA_DTYPE_F16;
    case at::kFloat: return KDA_DTYPE_F32;
    case at::kFloat8_e4m3fn: return KDA_DTYPE_E4M3;
    default: return -1;
    }
}
bool dtype_arg(PyObject* o, at::ScalarType* t) {
    if (o == Py_None) return false;
    if (!THPDtype_Check(o)) refuse("out_dtype must be a torch.dtype");
    *t = reinterpret_cast<THPDtype*>(o)->scalar_type;
    return true;
}

// torch's allocator without its dispatcher (half of the 1.5 us that an output costs).
at::Tensor empty(at::IntArrayRef shape, at::ScalarType dtype, const at::Tensor& like) {
    return at::Tensor(at::detail::empty_cuda(shape, dtype, like.device(), std::nullopt));
}

// The device of a call and the stream that it runs on (the caller's, or the current
// one).  While this lives both are the current ones, so outputs are allocated for
// the stream that writes them: memory freed with work still pending on another
// stream is not given to this one, nor an output that is dropped to another.
class Place {
  public:
    Place(PyObject* stream, const at::Tensor& t) : device_(checked(stream, t)) {
        if (stream == Py_None) {
            stream_ = c10::cuda::getCurrentCUDAStream(t.get_device()).stream();
            return;
        }
        PyObject* handle = PyObject_GetAttrString(stream, "cuda_stream");
        if (!handle) throw Refused{nullptr, ""};
        stream_ = static_cast<cudaStream_t>(PyLong_AsVoidPtr(handle));
        Py_DECREF(handle);
        if (PyErr_Occurred()) throw Refused{nullptr, ""};
        given_.emplace(c10::cuda::getStreamFromExternal(stream_, t.get_device()));
    }
    void* stream() const { return stream_; }

  private:
    static c10::Device checked(PyObject* stream, const at::Tensor& t) {
        if (stream != Py_None && PyObject_HasAttrString(stream, "device_index")) {  // (torch's streams have it)
            PyObject* index = PyObject_GetAttrString(stream, "device_index");
            if (!index) throw Refused{nullptr, ""};
            const long i = PyLong_AsLong(index);
            Py_DECREF(index);
            if (PyErr_Occurred()) throw Refused{nullptr, ""};
            need(i == t.get_device(), "stream must be of the tensors' device");
        }
        return t.device();
    }
    c10::cuda::CUDAGuard device_;
    std::optional<c10::cuda::CUDAStreamGuard> given_;
    cudaStream_t stream_;
};
double number(PyObject* o) {
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred()) throw Refused{nullptr, ""};
    return v;
}

void check(kda_status rc, const char* where) {
    if (rc == KDA_OK) return;
    if (g_error) {
        PyObject* e = PyObject_CallFunction(g_error, "is", (int)rc, where);
        if (e) {
            PyErr_SetObject(g_error, e);
            Py_DECREF(e);
        }
        throw Refused{nullptr, ""};
    }
    throw Refused{PyExc_RuntimeError, std::string(where) + ": status " + std::to_string((int)rc)};
}

// Runs one call; a C++ exception becomes the Python one.
template <typename F>
PyObject* guarded(Py_ssize_t got, Py_ssize_t want, F call) {
    try {
        if (got != want) throw Refused{PyExc_TypeError, "wrong number of arguments"};
        return call();
    } catch (const Refused& r) {
        if (r.type) PyErr_SetString(r.type, r.text.c_str());
    } catch (const std::exception& e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
    } catch (...) {
        PyErr_SetString(PyExc_RuntimeError, "unknown C++ exception");
    }
    return nullptr;
}
PyObject* kept(PyObject* given, at::Tensor&& made) {
    if (given != Py_None) {
        Py_INCREF(given);
        return given;
    }
    return THPVariable_Wrap(std::move(made));
}
int32_t* status_word(const at::Tensor* t) {
    need(!t || (t->scalar_type() == at::kInt && t->is_cuda() && t->numel() >= 1), "status must be a CUDA int32 tensor");
    return static_cast<int32_t*>(address(t));
}

// q, k, v, g, beta, state, slots, scale, cu_seqlens, out, status, stream, beta_logits
PyObject* call_step(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded(n, 13, [&]() -> PyObject* {
        const at::Tensor &q = tensor(a[0], "q"), &k = tensor(a[1], "k"), &v = tensor(a[2], "v"), &g = tensor(a[3], "g"),
                         &beta = tensor(a[4], "beta"), &state = tensor(a[5], "state");
        const at::Tensor *slots = optional(a[6], "slots"), *cu = optional(a[8], "cu_seqlens"),
                         *out = optional(a[9], "out"), *status = optional(a[10], "status");
        const at::ScalarType io = q.scalar_type();
        need(io == at::kBFloat16 || io == at::kHalf, "q must be bf16 or fp16");
        need(q.dim() == 4 && k.sizes() == q.sizes() && v.dim() == 4 && v.size(0) == q.size(0) && v.size(1) == q.size(1),
             "q and k are [B,T,Hqk,K], v is [B,T,H,V]");
        const int64_t B = q.size(0), T = q.size(1), Hqk = q.size(2), K = q.size(3), H = v.size(2), V = v.size(3);
        need(k.scalar_type() == io && v.scalar_type() == io && beta.scalar_type() == io && g.scalar_type() == at::kFloat,
             "k, v and beta have q's dtype, g is float32");
        need(same_shape(g, {B, T, H, K}) && same_shape(beta, {B, T, H}), "g is [B,T,H,K], beta is [B,T,H]");
        const bool s16 = state.scalar_type() == at::kBFloat16;
        need((s16 || state.scalar_type() == at::kFloat) && state.is_contiguous() && state.dim() == 4 &&
                 same_shape(state, {state.size(0), H, K, V}),
             "state must be a contiguous float32 or bfloat16 tensor [num_slots,H,K,V]");
        need(state.size(0) <= INT32_MAX && B <= INT32_MAX && T <= INT32_MAX && H <= INT32_MAX, "sizes beyond 32 bits");
        int64_t N = 0;
        if (cu) {
            N = cu->numel() - 1;
            need(cu->scalar_type() == at::kInt && cu->is_cuda() && cu->is_contiguous() && N >= 1 && N <= INT32_MAX,
                 "cu_seqlens must be a contiguous CUDA int32 tensor [N+1]");
        }
        need(!slots || (slots->scalar_type() == at::kInt && slots->is_cuda() && slots->is_contiguous() &&
                        slots->numel() == (cu ? N : B)),
             "slots must be a contiguous CUDA int32 tensor, one per sequence");
        need(q.is_cuda() && k.is_cuda() && v.is_cuda() && g.is_cuda() && beta.is_cuda() && state.is_cuda(),
             "step takes CUDA tensors");
        need(!out || (out->scalar_type() == io && out->sizes() == v.sizes() && out->is_cuda() && out->is_contiguous()),
             "out must be a contiguous CUDA tensor of v's shape and dtype");
        need_one_device(q, {&k, &v, &g, &beta, &state, slots, cu, out, status});
        kda_step_opts o{};
        o.io_dtype = io == at::kHalf ? KDA_IO_F16 : KDA_IO_BF16;
        o.state_dtype = s16 ? KDA_STATE_BF16 : KDA_STATE_F32;
        const int logits = PyObject_IsTrue(a[12]);
        if (logits < 0) throw Refused{nullptr, ""};
        o.beta_logits = logits;
        o.qk_heads = Hqk == H ? 0 : (int32_t)Hqk;
        need(Hqk > 0 || H == 0, "q and k have no heads");
        o.num_slots = (int32_t)state.size(0);
        o.q_stride = token_stride("q", q);
        o.k_stride = token_stride("k", k);
        o.v_stride = token_stride("v", v);
        o.g_stride = token_stride("g", g);
        o.beta_stride = token_stride("beta", beta);
        const kda_dims d{(int32_t)B, (int32_t)T, (int32_t)H, (int32_t)K, (int32_t)V, (int32_t)N};
        const float scale = a[7] == Py_None ? 1.f / std::sqrt((float)K) : (float)number(a[7]);
        const Place place(a[11], q);
        at::Tensor made;
        if (!out) made = empty(v.sizes(), io, q);
        check(kda_step(q.data_ptr(), k.data_ptr(), v.data_ptr(), static_cast<const float*>(g.data_ptr()),
                       beta.data_ptr(), scale, state.data_ptr(), static_cast<const int32_t*>(address(slots)),
                       static_cast<const int32_t*>(address(cu)), out ? out->data_ptr() : made.data_ptr(), &d, &o,
                       status_word(status), place.stream()),
              "kda_step");
        return kept(a[9], std::move(made));
    });
}

// x, weight, residual, eps, out_dtype, out, residual_out, stream
PyObject* call_rms_norm(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded(n, 8, [&]() -> PyObject* {
        const at::Tensor& x = tensor(a[0], "x");
        const at::Tensor *weight = optional(a[1], "weight"), *residual = optional(a[2], "residual"),
                         *out = optional(a[5], "out"), *sum = optional(a[6], "residual_out");
        const at::ScalarType io = x.scalar_type();
        need(dtype_code(io) >= 0 && io != at::kFloat8_e4m3fn && x.dim() >= 1 && x.is_cuda(),
             "x must be a CUDA tensor of bf16, fp16 or fp32");
        at::ScalarType to = io;
        dtype_arg(a[4], &to);
        need(to == io || to == at::kFloat || to == at::kFloat8_e4m3fn,
             "out_dtype must be x's dtype, float32 or float8_e4m3fn");
        const int64_t dim = x.size(-1);
        need(!residual || (residual->scalar_type() == io && residual->sizes() == x.sizes() && residual->is_cuda()),
             "residual must be a CUDA tensor of x's shape and dtype");
        need(!weight || ((weight->scalar_type() == io || weight->scalar_type() == at::kFloat) &&
                         same_shape(*weight, {dim}) && weight->is_cuda() && weight->is_contiguous()),
             "weight must be a contiguous CUDA tensor [dim] of x's dtype or float32");
        need(!sum || (sum->scalar_type() == io && sum->sizes() == x.sizes() && sum->is_cuda()),
             "residual_out must be a CUDA tensor of x's shape and dtype");
        need(!out || (out->scalar_type() == to && out->sizes() == x.sizes() && out->is_cuda() && out->is_contiguous()),
             "out must be a contiguous CUDA tensor of x's shape and out_dtype");
        need_one_device(x, {weight, residual, out, sum});
        kda_norm_opts o{};
        o.io_dtype = dtype_code(io);
        o.out_dtype = dtype_code(to);
        o.weight_f32 = weight && weight->scalar_type() == at::kFloat;
        o.eps = (float)number(a[3]);
        o.x_stride = row_stride("x", x, dim);
        o.residual_stride = residual ? row_stride("residual", *residual, dim) : 0;
        o.sum_stride = sum ? row_stride("residual_out", *sum, dim) : 0;
        const Place place(a[7], x);
        at::Tensor made, made_sum, scale;
        if (!out) made = empty(x.sizes(), to, x);
        if (residual && !sum) made_sum = empty(x.sizes(), io, x);
        if (to == at::kFloat8_e4m3fn) scale = empty(x.sizes().slice(0, x.dim() - 1), at::kFloat, x);
        const bool with_sum = residual || sum;
        check(kda_rms_norm(x.data_ptr(), address(residual), address(weight), out ? out->data_ptr() : made.data_ptr(),
                           scale.defined() ? static_cast<float*>(scale.data_ptr()) : nullptr,
                           sum ? sum->data_ptr() : made_sum.defined() ? made_sum.data_ptr() : nullptr,
                           dim ? x.numel() / dim : 0, dim, &o, place.stream()),
              "kda_rms_norm");
        PyObject* y = kept(a[5], std::move(made));
        PyObject* ys = scale.defined() ? THPVariable_Wrap(std::move(scale)) : (Py_INCREF(Py_None), Py_None);
        PyObject* s = with_sum ? kept(a[6], std::move(made_sum)) : (Py_INCREF(Py_None), Py_None);
        PyObject* all = y && ys && s ? PyTuple_Pack(3, y, ys, s) : nullptr;
        Py_XDECREF(y);
        Py_XDECREF(ys);
        Py_XDECREF(s);
        return all;
    });
}

int activation(PyObject* o) {
    if (o == Py_None) return KDA_ACT_NONE;
    const char* name = PyUnicode_Check(o) ? PyUnicode_AsUTF8(o) : nullptr;
    static constexpr const char* kNames[] = {"none", "silu", "gelu", "sigmoid", "logsigmoid"};
    for (int i = 0; name && i < 5; ++i)
        if (!strcmp(name, kNames[i])) return i;
    PyErr_Clear();
    throw Refused{PyExc_ValueError, "act must be one of gelu, logsigmoid, none, sigmoid, silu"};
}

// x, w, bias, act, residual, x_scale, w_scale, out_dtype, out, status, stream
PyObject* call_linear(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded(n, 11, [&]() -> PyObject* {
        const at::Tensor &x = tensor(a[0], "x"), &w = tensor(a[1], "w");
        const at::Tensor *bias = optional(a[2], "bias"), *residual = optional(a[4], "residual"),
                         *xs = optional(a[5], "x_scale"), *ws = optional(a[6], "w_scale"), *out = optional(a[8], "out"),
                         *status = optional(a[9], "status");
        const at::ScalarType io = x.scalar_type();
        const bool f8 = io == at::kFloat8_e4m3fn;
        need((io == at::kBFloat16 || io == at::kHalf || f8) && w.scalar_type() == io && x.is_cuda() && w.is_cuda(),
             "x and w must be CUDA tensors of one dtype: bf16, fp16 or float8_e4m3fn");
        at::ScalarType to = f8 ? at::kBFloat16 : io;
        dtype_arg(a[7], &to);
        need(to == at::kBFloat16 || to == at::kHalf || to == at::kFloat, "out_dtype must be bf16, fp16 or float32");
        kda_linear_opts o{};
        o.act = activation(a[3]);
        need(x.dim() >= 1 && w.dim() == 2 && x.size(-1) == w.size(1), "x is [..., K], w is [N, K]");
        const int64_t N = w.size(0), K = w.size(1);
        c10::DimVector shape(x.sizes().begin(), x.sizes().end());
        shape.back() = N;
        const at::IntArrayRef lead(shape.data(), shape.size() - 1);
        if (f8)
            need(xs && ws && xs->sizes() == lead && same_shape(*ws, {N}) && xs->scalar_type() == at::kFloat &&
                     ws->scalar_type() == at::kFloat && xs->is_cuda() && ws->is_cuda() && xs->is_contiguous() &&
                     ws->is_contiguous(),
                 "float8 operands take contiguous CUDA float32 x_scale [...] and w_scale [N]");
        else
            need(!xs && !ws, "x_scale and w_scale go with float8 operands only");
        need(!bias || (bias->scalar_type() == at::kFloat && same_shape(*bias, {N}) && bias->is_cuda() &&
                       bias->is_contiguous()),
             "bias must be a contiguous CUDA float32 tensor [N]");
        need(!residual || (residual->scalar_type() == to && residual->sizes() == at::IntArrayRef(shape) &&
                           residual->is_cuda()),
             "residual must be a CUDA tensor [..., N] of out_dtype");
        need(!out || (out->scalar_type() == to && out->sizes() == at::IntArrayRef(shape) && out->is_cuda()),
             "out must be a CUDA tensor [..., N] of out_dtype");
        need_one_device(x, {&w, bias, residual, xs, ws, out, status});
        o.io_dtype = dtype_code(io);
        o.out_dtype = dtype_code(to);
        o.x_stride = row_stride("x", x, K);
        o.w_stride = row_stride("w", w, K);
        o.residual_stride = residual ? row_stride("residual", *residual, N) : 0;
        o.y_stride = out ? row_stride("out", *out, N) : 0;
        const Place place(a[10], x);
        at::Tensor made;
        if (!out) made = empty(shape, to, x);
        check(kda_linear(x.data_ptr(), w.data_ptr(), static_cast<const float*>(address(bias)), address(residual),
                         static_cast<const float*>(address(xs)), static_cast<const float*>(address(ws)),
                         out ? out->data_ptr() : made.data_ptr(), K ? x.numel() / K : 0, N, K, &o, status_word(status),
                         place.stream()),
              "kda_linear");
        return kept(a[8], std::move(made));
    });
}

// KdaError, called as KdaError(code, where)
PyObject* set_error(PyObject*, PyObject* type) {
    Py_INCREF(type);
    Py_XDECREF(g_error);
    g_error = type;
    Py_RETURN_NONE;
}

PyMethodDef kMethods[] = {
    {"step", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(call_step)), METH_FASTCALL, nullptr},
    {"rms_norm", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(call_rms_norm)), METH_FASTCALL, nullptr},
    {"linear", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(call_linear)), METH_FASTCALL, nullptr},
    {"set_error", set_error, METH_O, nullptr},
    {nullptr, nullptr, 0, nullptr},
};
PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "_layer_calls", nullptr, -1, kMethods};

}  // namespace

PyMODINIT_FUNC PyInit__layer_calls() { return PyModule_Create(&kModule); }
