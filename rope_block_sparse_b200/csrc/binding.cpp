// The prompt side's calls over torch tensors, for the Python layer (h3a.py):
// checks, fresh outputs, the tensors' device and its current stream, then the
// C ABI.  A single-token step's kernels take two to ten microseconds; the same
// work in Python and ctypes took the host 14 to 19 a call, here it takes 3.9 to
// 4.6 (packed_attention) and 5.1 (rope, residual_rmsnorm).  Every function is
// positional and returns new or given tensors; wrong arguments raise ValueError, a
// status other than H3A_OK the H3AError of h3a.py.
#include <ATen/core/Tensor.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cstring>
#include <string>

#include "h3a.h"

namespace {

// An argument that is refused; what() goes into the ValueError.
struct Refused {
    std::string why;
};
// A status other than H3A_OK.
struct Failed {
    const char* call;
    h3a_status status;
};

PyObject* g_error = nullptr;  // H3AError(call, status, detail)

const at::Tensor& tensor(PyObject* o, const char* name) {
    if (!THPVariable_Check(o)) throw Refused{std::string(name) + " must be a torch.Tensor"};
    return THPVariable_Unpack(o);
}

// None stands for an undefined tensor.
const at::Tensor& maybe(PyObject* o, const char* name) {
    static const at::Tensor none;
    return o == Py_None ? none : tensor(o, name);
}

void require(bool ok, const char* name, const char* what) {
    if (!ok) throw Refused{std::string(name) + " " + what};
}

// A bf16 / fp16 CUDA tensor of `dims` dimensions whose last one is contiguous.
h3a_dtype check_rows(const at::Tensor& t, const char* name, int dims) {
    const auto type = t.scalar_type();
    if (type != at::kBFloat16 && type != at::kHalf)
        throw Refused{std::string(name) + " must be bfloat16 or float16, got " + c10::toString(type)};
    require(t.is_cuda(), name, "must be on a CUDA device (libh3a has no CPU path)");
    if (t.dim() != dims || (t.stride(dims - 1) != 1 && t.size(dims - 1) > 1))
        throw Refused{std::string(name) + " must have " + std::to_string(dims) + " dimensions, the last one contiguous"};
    // the descriptors hold them in 32 bits
    for (int i = 1; i < dims; ++i) require(t.size(i) <= INT32_MAX, name, "has a dimension of 2^31 or more");
    return type == at::kHalf ? H3A_FP16 : H3A_BF16;
}

void check_like(const at::Tensor& t, const char* name, int dims, const at::Tensor& first) {
    check_rows(t, name, dims);
    require(t.scalar_type() == first.scalar_type() && t.device() == first.device(), name,
            "must have the element type and device of the first tensor");
}

const int32_t* check_index(const at::Tensor& t, const char* name, int64_t n, const at::Tensor& first) {
    if (t.scalar_type() != at::kInt || t.dim() != 1 || t.size(0) != n || !t.is_contiguous() || t.device() != first.device())
        throw Refused{std::string(name) + " must be a contiguous int32 [" + std::to_string(n) + "] tensor on " +
                      first.device().str()};
    return t.const_data_ptr<int32_t>();
}

at::Tensor fresh(at::IntArrayRef sizes, at::ScalarType type, const at::Tensor& like) {
    return at::Tensor(at::detail::empty_cuda(sizes, type, like.device(), std::nullopt));
}

h3a_stream_t stream_of(const at::Tensor& t) {
    return reinterpret_cast<h3a_stream_t>(c10::cuda::getCurrentCUDAStream(t.device().index()).stream());
}

// Runs a call of the C ABI without the interpreter's lock.
template <typename F>
void launch(const char* name, F&& call) {
    h3a_status status;
    Py_BEGIN_ALLOW_THREADS;
    status = call();
    Py_END_ALLOW_THREADS;
    if (status != H3A_OK) throw Failed{name, status};
}

bool truth(PyObject* o) {
    const int v = PyObject_IsTrue(o);
    if (v < 0) throw Refused{""};
    return v != 0;
}
double number(PyObject* o) {
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred()) throw Refused{""};
    return v;
}
// As fp32; what fp32 rounds to zero is not meant as the zero that turns a number off.
float number32(PyObject* o, const char* name) {
    const double v = number(o);
    const float f = static_cast<float>(v);
    require(f != 0.0f || v == 0.0, name, "is so small that it would be zero in fp32");
    return f;
}
int64_t whole(PyObject* o) {
    PyObject* i = PyNumber_Index(o);  // no fractions
    if (i == nullptr) throw Refused{""};
    const int64_t v = PyLong_AsLongLong(i);
    Py_DECREF(i);
    if (v == -1 && PyErr_Occurred()) throw Refused{""};
    return v;
}

PyObject* wrap(const at::Tensor& t) {
    if (!t.defined()) Py_RETURN_NONE;
    return THPVariable_Wrap(t);
}
// A tuple of tensors (None where undefined).
template <typename... T>
PyObject* tuple_of(const T&... t) {
    PyObject* items[] = {wrap(t)...};
    PyObject* r = PyTuple_New(sizeof...(T));
    for (size_t i = 0; i < sizeof...(T); ++i) {
        if (r == nullptr || items[i] == nullptr) {
            Py_XDECREF(r);
            return nullptr;
        }
        PyTuple_SET_ITEM(r, i, items[i]);
    }
    return r;
}

// Runs a function's body; its exceptions become Python's.
template <typename F>
PyObject* guarded(Py_ssize_t given, Py_ssize_t wanted, F&& body) {
    if (given != wanted) {
        PyErr_Format(PyExc_TypeError, "expected %zd arguments, got %zd", wanted, given);
        return nullptr;
    }
    try {
        return body();
    } catch (const Refused& e) {
        if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, e.why.c_str());
    } catch (const Failed& e) {
        if (g_error == nullptr) {
            PyErr_Format(PyExc_RuntimeError, "%s failed: %s", e.call, h3a_status_string(e.status));
        } else {
            PyObject* x = PyObject_CallFunction(g_error, "sis", e.call, static_cast<int>(e.status),
                                                e.status == H3A_ERR_CUDA ? h3a_last_cuda_error_string() : "");
            if (x != nullptr) {
                PyErr_SetObject(g_error, x);
                Py_DECREF(x);
            }
        }
    } catch (const std::exception& e) {  // out of memory and the like, from torch
        if (!PyErr_Occurred()) PyErr_SetString(PyExc_RuntimeError, e.what());
    }
    return nullptr;
}

h3a_heads_desc heads_desc(const at::Tensor& x, const at::Tensor& y) {
    return {static_cast<int32_t>(x.size(1)), static_cast<int32_t>(x.size(2)), x.stride(0), x.stride(1), y.stride(0), y.stride(1)};
}

// rope(q, k, positions, plan, inverse, q_out, k_out): outputs None for fresh ones
PyObject* rope(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded(n, 7, [&]() -> PyObject* {
        const at::Tensor &q = tensor(a[0], "q"), &k = maybe(a[1], "k"), &positions = tensor(a[2], "positions");
        at::Tensor yq = maybe(a[5], "out"), yk = maybe(a[6], "out");
        const bool given = yq.defined() || yk.defined();
        require(!given || (yq.defined() && yk.defined() == k.defined()), "out", "must hold a tensor for q, and one for k exactly where k is given");
        const h3a_dtype dtype = check_rows(q, "q", 3);
        const int64_t tokens = q.size(0);
        const int32_t* at_positions = check_index(positions, "positions", tokens, q);
        if (k.defined()) {
            check_like(k, "k", 3, q);
            if (k.size(0) != tokens || k.size(2) != q.size(2)) throw Refused{"q and k must have the same tokens and head_dim"};
        }
        Py_buffer plan;
        if (PyObject_GetBuffer(a[3], &plan, PyBUF_SIMPLE) != 0) throw Refused{""};
        h3a_rope_plan p;
        const bool fits = plan.len == static_cast<Py_ssize_t>(sizeof(p));
        if (fits) std::memcpy(&p, plan.buf, sizeof(p));
        PyBuffer_Release(&plan);
        require(fits, "plan", "must be what rope_plan() returns");
        const bool inverse = truth(a[4]);
        const c10::cuda::CUDAGuard guard(q.device());
        if (!given) {
            yq = fresh(q.sizes(), q.scalar_type(), q);
            if (k.defined()) yk = fresh(k.sizes(), q.scalar_type(), q);
        }
        check_like(yq, "out", 3, q);
        require(yq.sizes() == q.sizes(), "out", "must have the shapes of q and k");
        h3a_heads_desc dq = heads_desc(q, yq), dk{};
        if (k.defined()) {
            check_like(yk, "out", 3, q);
            require(yk.sizes() == k.sizes(), "out", "must have the shapes of q and k");
            dk = heads_desc(k, yk);
        }
        const h3a_stream_t st = stream_of(q);
        launch("h3a_rope", [&]() {
            return h3a_rope(q.const_data_ptr(), yq.mutable_data_ptr(), &dq, k.defined() ? k.const_data_ptr() : nullptr,
                            k.defined() ? yk.mutable_data_ptr() : nullptr, k.defined() ? &dk : nullptr, dtype, at_positions, tokens,
                            &p, inverse, st);
        });
        return tuple_of(yq, yk);
    });
}

// residual_rmsnorm(x, f, gamma, eps, scales, h, y, s): scales 0, 1, 2 (h3a_scales);
// h, y and s all None for fresh outputs
PyObject* residual_rmsnorm(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded(n, 8, [&]() -> PyObject* {
        const at::Tensor &x = tensor(a[0], "x"), &f = maybe(a[1], "f"), &gamma = tensor(a[2], "gamma");
        const float eps = number32(a[3], "eps");
        const int64_t scales = whole(a[4]);
        at::Tensor h = maybe(a[5], "h"), y = maybe(a[6], "y"), s = maybe(a[7], "scales");
        const bool given = h.defined() || y.defined() || s.defined();
        require(!given || (y.defined() && h.defined() == f.defined() && s.defined() == (scales != H3A_SCALES_NONE)), "out",
                "must hold a tensor for y, for h exactly where f is given and for the scales exactly where y is scaled");
        const h3a_dtype dtype = check_rows(x, "x", 2);
        const int64_t rows = x.size(0), width = x.size(1);
        if (f.defined()) {
            check_like(f, "f", 2, x);
            require(f.sizes() == x.sizes(), "f", "must match x");
        }
        require(gamma.scalar_type() == at::kFloat && gamma.dim() == 1 && gamma.size(0) == width && gamma.is_contiguous() &&
                    gamma.device() == x.device(),
                "gamma", "must be a contiguous fp32 [C] tensor on x's device");
        const auto y_type = scales == H3A_SCALES_NONE ? x.scalar_type() : at::kFloat8_e4m3fn;
        const int64_t groups = (width + H3A_SCALE_GROUP - 1) / H3A_SCALE_GROUP;
        const c10::cuda::CUDAGuard guard(x.device());
        if (!given) {
            if (f.defined()) h = fresh(x.sizes(), x.scalar_type(), x);
            y = fresh(x.sizes(), y_type, x);
            if (scales == H3A_SCALES_ROW) s = fresh({rows}, at::kFloat, x);
            if (scales == H3A_SCALES_GROUP) s = fresh({rows, groups}, at::kFloat, x);
        } else {
            if (f.defined()) {
                check_like(h, "h", 2, x);
                require(h.sizes() == x.sizes(), "h", "must match x");
            }
            require(y.scalar_type() == y_type && y.sizes() == x.sizes() && (width <= 1 || y.stride(1) == 1) && y.device() == x.device(), "y",
                    "must have x's shape, rows contiguous, and x's type or, with scales, float8_e4m3fn");
            if (scales != H3A_SCALES_NONE)
                require(s.scalar_type() == at::kFloat && s.is_contiguous() && s.device() == x.device() &&
                            (scales == H3A_SCALES_ROW ? s.dim() == 1 && s.size(0) == rows
                                                      : s.dim() == 2 && s.size(0) == rows && s.size(1) == groups),
                        "scales", "must be a contiguous fp32 [rows] (row) or [rows, ceil(C / 128)] (group) tensor");
        }
        // a single row is not stepped: any stride
        auto step = [&](const at::Tensor& t) { return t.defined() && rows > 1 ? t.stride(0) : width; };
        const h3a_stream_t st = stream_of(x);
        launch("h3a_residual_rmsnorm", [&]() {
            return h3a_residual_rmsnorm(x.const_data_ptr(), step(x), f.defined() ? f.const_data_ptr() : nullptr, step(f),
                                        gamma.const_data_ptr<float>(), rows, static_cast<int32_t>(width), dtype, eps,
                                        static_cast<h3a_scales>(scales), h.defined() ? h.mutable_data_ptr() : nullptr, step(h),
                                        y.mutable_data_ptr(), step(y), s.defined() ? s.mutable_data_ptr<float>() : nullptr, st);
        });
        return tuple_of(h, y, s);
    });
}

// packed_attention(q, k, v, starts_q, starts_k, max_q, max_k, lengths_k, causal,
// scale, return_lse, workspace, out): lengths_k, workspace and out may be None
PyObject* packed_attention(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded(n, 13, [&]() -> PyObject* {
        const at::Tensor &q = tensor(a[0], "q"), &k = tensor(a[1], "k"), &v = tensor(a[2], "v");
        const at::Tensor &starts_q = tensor(a[3], "starts_q"), &starts_k = tensor(a[4], "starts_k"), &lengths = maybe(a[7], "lengths_k");
        h3a_packed_desc d{};
        d.scale = number32(a[9], "scale");
        d.dtype = check_rows(q, "q", 3);
        check_like(k, "k", 3, q);
        check_like(v, "v", 3, q);
        if (k.sizes() != v.sizes() || k.size(2) != q.size(2)) throw Refused{"k and v must have one shape, and q's head_dim"};
        const int64_t seqs = starts_q.dim() == 1 ? starts_q.size(0) - 1 : 0;
        const int32_t* sq = check_index(starts_q, "starts_q", seqs + 1, q);
        const int32_t* sk = check_index(starts_k, "starts_k", seqs + 1, q);
        const int32_t* lk = lengths.defined() ? check_index(lengths, "lengths_k", seqs, q) : nullptr;
        d.max_q = whole(a[5]), d.max_k = whole(a[6]);
        d.causal = truth(a[8]);
        const bool with_lse = truth(a[10]);
        const c10::cuda::CUDAGuard guard(q.device());
        at::Tensor workspace = maybe(a[11], "workspace"), out = maybe(a[12], "out"), lse;
        if (!out.defined()) {
            out = fresh(q.sizes(), q.scalar_type(), q);
        } else {
            check_like(out, "out", 3, q);
            require(out.sizes() == q.sizes(), "out", "must have q's shape");
        }
        d.seqs = static_cast<int32_t>(seqs);
        d.heads = static_cast<int32_t>(q.size(1)), d.kv_heads = static_cast<int32_t>(k.size(1)), d.head_dim = static_cast<int32_t>(q.size(2));
        d.total_q = q.size(0), d.total_k = k.size(0);
        d.q_stride_n = q.stride(0), d.q_stride_h = q.stride(1), d.k_stride_n = k.stride(0), d.k_stride_h = k.stride(1);
        d.v_stride_n = v.stride(0), d.v_stride_h = v.stride(1), d.o_stride_n = out.stride(0), d.o_stride_h = out.stride(1);
        size_t room = 0;
        if (!workspace.defined()) {
            const h3a_status status = h3a_packed_attention_workspace_size(&d, &room);
            if (status != H3A_OK) throw Failed{"h3a_packed_attention", status};
            if (room > 0) workspace = fresh({static_cast<int64_t>(room)}, at::kByte, q);
        } else {
            require(workspace.is_contiguous() && workspace.device() == q.device(), "workspace",
                    "must be a contiguous tensor on q's device");
            room = workspace.nbytes();
        }
        if (with_lse) lse = fresh({q.size(0), q.size(1)}, at::kFloat, q);
        const h3a_stream_t st = stream_of(q);
        launch("h3a_packed_attention", [&]() {
            return h3a_packed_attention(q.const_data_ptr(), k.const_data_ptr(), v.const_data_ptr(), &d, sq, sk, lk, out.mutable_data_ptr(),
                                        with_lse ? lse.mutable_data_ptr<float>() : nullptr,
                                        workspace.defined() ? workspace.mutable_data_ptr() : nullptr, room, st);
        });
        return with_lse ? tuple_of(out, lse) : wrap(out);
    });
}

// set_error(H3AError)
PyObject* set_error(PyObject*, PyObject* type) {
    Py_INCREF(type);
    Py_XSETREF(g_error, type);
    Py_RETURN_NONE;
}

PyMethodDef kMethods[] = {
    {"rope", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(rope)), METH_FASTCALL, nullptr},
    {"residual_rmsnorm", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(residual_rmsnorm)), METH_FASTCALL, nullptr},
    {"packed_attention", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(packed_attention)), METH_FASTCALL, nullptr},
    {"set_error", set_error, METH_O, nullptr},
    {nullptr, nullptr, 0, nullptr},
};

PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, kMethods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__binding() { return PyModule_Create(&kModule); }
