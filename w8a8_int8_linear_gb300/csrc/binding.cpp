// The Python calls of the operators between the Linears (operators.py): checks
// of tensors, allocation of outputs, and the C ABI call on the current stream.
// The kernels of single tokens take 4 to 12 us; the same steps written in Python
// and called through ctypes took the host 13 to 18 us a call, here 4 to 5.
//
// Every function gets its arguments by position and returns its result, or the
// library's status as an int where that is not W8A8_OK.
#include <Python.h>

#include <ATen/ATen.h>
#include <c10/core/GradMode.h>
#include <c10/cuda/CUDAGraphsC10Utils.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cmath>
#include <map>
#include <string>
#include <utility>

#include "../../include/w8a8.h"

namespace {

using at::ScalarType;
using at::Tensor;

struct Refused {
    PyObject* type;  // null: the Python error is already set
    std::string text;
};
[[noreturn]] void type_error(const std::string& text) { throw Refused{PyExc_TypeError, text}; }
[[noreturn]] void value_error(const std::string& text) { throw Refused{PyExc_ValueError, text}; }

std::string name_of(ScalarType t) {
    switch (t) {
        case ScalarType::BFloat16: return "torch.bfloat16";
        case ScalarType::Half: return "torch.float16";
        case ScalarType::Float: return "torch.float32";
        case ScalarType::Double: return "torch.float64";
        case ScalarType::Char: return "torch.int8";
        case ScalarType::Int: return "torch.int32";
        case ScalarType::Long: return "torch.int64";
        default: return c10::toString(t);
    }
}

bool none(PyObject* o) { return o == Py_None; }

const Tensor& tensor(PyObject* o, const char* name) {
    if (!THPVariable_Check(o)) type_error(std::string(name) + " must be a torch.Tensor");
    return THPVariable_Unpack(o);
}
double number(PyObject* o) {
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred()) throw Refused{nullptr, ""};
    return v;
}
int64_t integer(PyObject* o) {
    const long long v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred()) throw Refused{nullptr, ""};
    return v;
}
bool truth(PyObject* o) {
    const int v = PyObject_IsTrue(o);
    if (v < 0) throw Refused{nullptr, ""};
    return v != 0;
}

// An argument that may be a tensor, by its place.
struct Argument {
    int at;
    const char* name;
    bool written = false;  // by the call, where it is given
};

// The kernels run on the GPU of the first tensor; the others must be on it too
// (what is no CUDA tensor at all is refused by name later on).  What is written
// in place has no gradient: autograd would give that of the value before.
template <size_t N>
void check_arguments(PyObject* const* a, const Argument (&arguments)[N]) {
    const Argument* first = nullptr;
    c10::Device device(c10::kCUDA);
    for (const Argument& g : arguments) {
        if (!THPVariable_Check(a[g.at])) continue;
        const Tensor& t = THPVariable_Unpack(a[g.at]);
        if (g.written && t.requires_grad() && c10::GradMode::is_enabled())
            value_error(std::string(g.name) + " requires a gradient and cannot be written in place: detach it, or call "
                        "under torch.no_grad()");
        if (!t.is_cuda()) continue;
        if (!first) {
            first = &g;
            device = t.device();
        } else if (t.device() != device) {
            value_error(std::string(g.name) + " is on " + t.device().str() + ", " + first->name + " on " + device.str());
        }
    }
}

// Autograd learns that they were written, so that a backward pass which needs a
// value from before says so (tensors made in inference mode have no version).
template <size_t N>
void bump_written(PyObject* const* a, const Argument (&arguments)[N]) {
    for (const Argument& g : arguments) {
        if (!g.written || none(a[g.at])) continue;
        const Tensor& t = THPVariable_Unpack(a[g.at]);
        if (!t.is_inference()) t.unsafeGetTensorImpl()->bump_version();
    }
}

w8a8_dtype dtype_of(ScalarType t) {
    return t == ScalarType::BFloat16 ? W8A8_BF16 : t == ScalarType::Half ? W8A8_FP16 : W8A8_FP32;
}

Tensor empty(at::IntArrayRef shape, ScalarType type, const Tensor& like) {
    return at::empty(shape, like.options().dtype(type));
}

// A [tokens, heads, dim] tensor on the GPU, 16-bit (of `type` where given), dense
// in its last dimension.  A dimension of one row has no stride of its own and
// gets the row length.
struct Heads {
    void* ptr;
    int64_t tokens, heads, dim, token, head;
};
Heads heads(const Tensor& t, const char* name, const ScalarType* type = nullptr) {
    const std::string n(name);
    if (type && t.scalar_type() != *type) type_error(n + " must be " + name_of(*type) + ", got " + name_of(t.scalar_type()));
    if (!type && t.scalar_type() != ScalarType::BFloat16 && t.scalar_type() != ScalarType::Half)
        type_error(n + " must be torch.bfloat16 or torch.float16, got " + name_of(t.scalar_type()));
    if (!t.is_cuda()) value_error(n + " must be a CUDA tensor");
    if (t.dim() != 3) value_error(n + " must be [tokens, heads, dim]");
    const auto size = t.sizes(), stride = t.strides();
    if (stride[2] != 1 && size[2] != 1) value_error(n + " must be dense in its last dimension");
    return {t.data_ptr(), size[0], size[1], size[2], size[0] != 1 ? stride[0] : size[1] * size[2],
            size[1] != 1 ? stride[1] : size[2]};
}

// `out` [tokens, heads, dim] as given (of `of`'s shape), or new.
Heads output(PyObject* o, const char* name, const Tensor& of, const Heads& h, ScalarType type, Tensor& out) {
    if (none(o)) {
        out = empty({h.tokens, h.heads, h.dim}, type, of);
        return {out.data_ptr(), h.tokens, h.heads, h.dim, h.heads * h.dim, h.dim};
    }
    out = tensor(o, name);
    const Heads r = heads(out, name, &type);
    if (r.tokens != h.tokens || r.heads != h.heads || r.dim != h.dim)
        value_error(std::string(name) + " must have the shape of its input");
    return r;
}

// A dense vector of n values on the GPU.
template <typename T = void>
const T* indices(PyObject* o, ScalarType type, int64_t n, const char* name) {
    if (!THPVariable_Check(o) || THPVariable_Unpack(o).scalar_type() != type)
        type_error(std::string(name) + " must be a " + name_of(type) + " tensor");
    const Tensor& t = THPVariable_Unpack(o);
    if (!t.is_cuda() || t.dim() != 1 || t.numel() != n || !t.is_contiguous())
        value_error(std::string(name) + " must be a dense CUDA tensor of " + std::to_string(n) + " values");
    return static_cast<const T*>(t.data_ptr());
}

PyObject* wrap(const Tensor& t) {
    if (!t.defined()) Py_RETURN_NONE;
    return THPVariable_Wrap(t);
}
PyObject* status(w8a8_status s) { return PyLong_FromLong(s); }

// A new workspace, its counters zeroed on the current stream.
Tensor new_workspace(const Tensor& like) {
    Tensor ws = at::empty({static_cast<int64_t>(w8a8_attention_workspace_size())}, like.options().dtype(ScalarType::Byte));
    ws.narrow(0, 0, static_cast<int64_t>(w8a8_attention_workspace_zeroed())).zero_();
    return ws;
}

// One per stream; a captured call gets its own, zeroed by every replay.
Tensor workspace_of(const Tensor& like, cudaStream_t stream) {
    if (c10::cuda::currentStreamCaptureStatusMayInitCtx() != c10::cuda::CaptureStatus::None) return new_workspace(like);
    // not freed at exit, when the CUDA context may be gone before it
    static auto* all = new std::map<std::pair<int, cudaStream_t>, Tensor>;
    Tensor& ws = (*all)[{like.get_device(), stream}];
    if (!ws.defined()) ws = new_workspace(like);
    return ws;
}

// Q, K, V, cu_q, cu_k, k_lens, batch, causal, scale, out, lse, workspace
PyObject* attention(PyObject* const* a) {
    static constexpr Argument arguments[] = {{0, "Q"}, {1, "K"}, {2, "V"}, {3, "cu_q"}, {4, "cu_k"}, {5, "k_lens"},
                                             {9, "out", true}, {11, "workspace"}};
    check_arguments(a, arguments);
    Tensor q = tensor(a[0], "Q"), k = tensor(a[1], "K"), v = tensor(a[2], "V");
    Heads hq = heads(q, "Q");
    const ScalarType type = q.scalar_type();
    Heads hk = heads(k, "K", &type), hv = heads(v, "V", &type);
    if (!(hq.token && hq.head && hk.token && hk.head && hv.token && hv.head)) {  // a broadcast dimension is laid out
        q = q.contiguous(), k = k.contiguous(), v = v.contiguous();
        hq = heads(q, "Q"), hk = heads(k, "K"), hv = heads(v, "V");
    }
    if (hk.dim != hq.dim || k.sizes() != v.sizes())
        value_error("K and V must be [keys, KV heads, dim] with the queries' dim");
    int64_t batch = 0;
    if (!none(a[3]))
        batch = tensor(a[3], "cu_q").numel() - 1;
    else if (!none(a[4]))
        batch = tensor(a[4], "cu_k").numel() - 1;
    else
        batch = integer(a[6]);
    const auto* cu_q = none(a[3]) ? nullptr : indices<int32_t>(a[3], ScalarType::Int, batch + 1, "cu_q");
    const auto* cu_k = none(a[4]) ? nullptr : indices<int32_t>(a[4], ScalarType::Int, batch + 1, "cu_k");
    const auto* k_lens = none(a[5]) ? nullptr : indices<int32_t>(a[5], ScalarType::Int, batch, "k_lens");
    const double scale = none(a[8]) ? 1.0 / std::sqrt(static_cast<double>(hq.dim)) : number(a[8]);
    const c10::cuda::CUDAGuard guard(q.device());
    Tensor out, lse;
    const Heads ho = output(a[9], "out", q, hq, type, out);
    if (truth(a[10])) lse = empty({hq.tokens, hq.heads}, ScalarType::Float, q);
    const cudaStream_t stream = c10::cuda::getCurrentCUDAStream().stream();
    const Tensor ws = none(a[11]) ? workspace_of(q, stream) : tensor(a[11], "workspace");
    if (!ws.is_cuda() || !ws.is_contiguous()) value_error("workspace must be a dense CUDA tensor");
    const w8a8_status s = w8a8_attention(
        hq.ptr, hk.ptr, hv.ptr, ho.ptr, lse.defined() ? static_cast<float*>(lse.data_ptr()) : nullptr, cu_q, cu_k, k_lens,
        dtype_of(type), batch, hq.tokens, hk.tokens, hq.heads, hk.heads, hq.dim, hq.token, hq.head, hk.token, hk.head,
        hv.token, hv.head, ho.token, ho.head, static_cast<float>(scale), truth(a[7]), ws.data_ptr(), ws.nbytes(), stream);
    if (s != W8A8_OK) return status(s);
    bump_written(a, arguments);
    if (!lse.defined()) return wrap(out);
    return Py_BuildValue("(NN)", wrap(out), wrap(lse));
}

struct Turns {
    const int64_t* positions;
    const double* freqs;
    int64_t rot;
};
Turns turns(PyObject* positions, PyObject* freqs, int64_t tokens) {
    Turns r;
    r.positions = indices<int64_t>(positions, ScalarType::Long, tokens, "positions");
    const int64_t pairs = tensor(freqs, "freqs").numel();
    r.freqs = indices<double>(freqs, ScalarType::Double, pairs, "freqs");
    r.rot = 2 * pairs;
    return r;
}

// Q, K, positions, freqs, layout, amplitude, inverse, q_out, k_out
PyObject* rotary(PyObject* const* a) {
    static constexpr Argument arguments[] = {{0, "Q"}, {1, "K"}, {2, "positions"}, {3, "freqs"}, {7, "q_out", true},
                                             {8, "k_out", true}};
    check_arguments(a, arguments);
    const Tensor& q = tensor(a[0], "Q");
    const Heads hq = heads(q, "Q");
    const ScalarType type = q.scalar_type();
    Heads hk = {}, ko = {};
    Tensor q_out, k_out;
    if (!none(a[1])) {
        hk = heads(tensor(a[1], "K"), "K", &type);
        if (hk.tokens != hq.tokens || hk.dim != hq.dim) value_error("K must have the tokens and the dim of Q");
    }
    const Turns tu = turns(a[2], a[3], hq.tokens);
    const c10::cuda::CUDAGuard guard(q.device());
    if (!none(a[1])) ko = output(a[8], "k_out", q, hk, type, k_out);
    const Heads qo = output(a[7], "q_out", q, hq, type, q_out);
    const w8a8_status s = w8a8_rotary(
        hq.ptr, hk.ptr, qo.ptr, ko.ptr, dtype_of(type), hq.tokens, hq.heads, hk.heads, hq.dim, tu.rot, hq.token, hq.head,
        hk.token, hk.head, qo.token, qo.head, ko.token, ko.head, tu.positions, tu.freqs, static_cast<float>(number(a[5])),
        static_cast<w8a8_rotary_layout>(integer(a[4])), truth(a[6]), c10::cuda::getCurrentCUDAStream().stream());
    if (s != W8A8_OK) return status(s);
    bump_written(a, arguments);
    return Py_BuildValue("(NN)", wrap(q_out), wrap(k_out));
}

// Q, K, V, positions, freqs, k_cache, v_cache, slots, layout, amplitude, q_out
PyObject* rotary_append(PyObject* const* a) {
    static constexpr Argument arguments[] = {{0, "Q"}, {1, "K"}, {2, "V"}, {3, "positions"}, {4, "freqs"},
                                             {5, "k_cache", true}, {6, "v_cache", true}, {7, "slots"},
                                             {10, "q_out", true}};
    check_arguments(a, arguments);
    const Tensor& q = tensor(a[0], "Q");
    const Heads hq = heads(q, "Q");
    const ScalarType type = q.scalar_type();
    const Tensor &k = tensor(a[1], "K"), &v = tensor(a[2], "V");
    const Tensor &kc = tensor(a[5], "k_cache"), &vc = tensor(a[6], "v_cache");
    const Heads hk = heads(k, "K", &type), hv = heads(v, "V", &type);
    const Heads ck = heads(kc, "k_cache", &type), cv = heads(vc, "v_cache", &type);
    if (hk.tokens != hq.tokens || hk.dim != hq.dim) value_error("K must have the tokens and the dim of Q");
    if (k.sizes() != v.sizes() || ck.heads != hk.heads || ck.dim != hk.dim || kc.sizes() != vc.sizes())
        value_error("V must have the shape of K, and both caches its heads and dim");
    const Turns tu = turns(a[3], a[4], hq.tokens);
    const auto* slots = indices<int64_t>(a[7], ScalarType::Long, hq.tokens, "slots");
    const c10::cuda::CUDAGuard guard(q.device());
    Tensor q_out;
    const Heads qo = output(a[10], "q_out", q, hq, type, q_out);
    const w8a8_status s = w8a8_rotary_append(
        hq.ptr, hk.ptr, hv.ptr, qo.ptr, ck.ptr, cv.ptr, dtype_of(type), hq.tokens, hq.heads, hk.heads, hq.dim, tu.rot,
        ck.tokens, hq.token, hq.head, hk.token, hk.head, hv.token, hv.head, qo.token, qo.head, ck.token, ck.head, cv.token,
        cv.head, tu.positions, slots, tu.freqs, static_cast<float>(number(a[9])),
        static_cast<w8a8_rotary_layout>(integer(a[8])), c10::cuda::getCurrentCUDAStream().stream());
    if (s != W8A8_OK) return status(s);
    bump_written(a, arguments);
    return wrap(q_out);
}

// A dense CUDA tensor of the given type and shape; null for None.
void* dense(PyObject* o, const char* name, ScalarType type, at::IntArrayRef shape) {
    if (none(o)) return nullptr;
    const Tensor& t = tensor(o, name);
    if (t.scalar_type() != type)
        type_error(std::string(name) + " must be " + name_of(type) + ", got " + name_of(t.scalar_type()));
    if (!t.is_cuda() || !t.is_contiguous() || t.sizes() != shape)
        value_error(std::string(name) + " must be a dense CUDA tensor of shape " + c10::str(shape));
    return t.data_ptr();
}

// X, B, gamma, beta, eps, kind, alpha, gate, branch_gamma, mod_scale, mod_shift,
// rows_per_group, h_out, image, codes, y
PyObject* residual_norm_quant(PyObject* const* a) {
    static constexpr Argument arguments[] = {{0, "X"}, {1, "B"}, {2, "gamma"}, {3, "beta"}, {7, "gate"},
                                             {8, "branch_gamma"}, {9, "mod_scale"}, {10, "mod_shift"},
                                             {12, "h_out", true}};
    check_arguments(a, arguments);
    if (!THPVariable_Check(a[0]) || THPVariable_Unpack(a[0]).dim() != 2) value_error("X must be a [rows, width] tensor");
    const Tensor& x = THPVariable_Unpack(a[0]);
    const ScalarType type = x.scalar_type(), bf16 = ScalarType::BFloat16;
    if (type != bf16 && type != ScalarType::Float)
        type_error("X must be torch.bfloat16 or torch.float32, got " + name_of(type));
    const int64_t m = x.size(0), k = x.size(1), per = integer(a[11]);
    const at::IntArrayRef shape = x.sizes();
    const void* px = dense(a[0], "X", type, shape);
    if (none(a[1])) type_error("B must be a torch.Tensor");
    const void* pb = dense(a[1], "B", bf16, shape);
    const void* gamma = dense(a[2], "gamma", bf16, {k});
    const void* beta = dense(a[3], "beta", bf16, {k});
    const void* branch_gamma = dense(a[8], "branch_gamma", bf16, {k});
    // [groups, k] or [k], parts of one wider tensor: they share their row stride
    const void* mod[3] = {};
    int64_t stride = 0;
    bool strided = false;
    static const char* const names[3] = {"gate", "mod_scale", "mod_shift"};
    PyObject* const given[3] = {a[7], a[9], a[10]};
    for (int i = 0; i < 3; ++i) {
        if (none(given[i])) continue;
        const std::string n(names[i]);
        if (!THPVariable_Check(given[i])) type_error(n + " must be a torch.bfloat16 CUDA tensor");
        const Tensor& t = THPVariable_Unpack(given[i]);
        if (t.scalar_type() != bf16 || !t.is_cuda()) type_error(n + " must be a torch.bfloat16 CUDA tensor");
        const int64_t d = t.dim();
        if (d < 1 || d > 2 || t.size(d - 1) != k || (k != 1 && t.stride(d - 1) != 1))
            value_error(n + " must be [groups, " + std::to_string(k) + "], dense in its last dimension");
        const int64_t groups = d == 1 ? 1 : t.size(0);
        if (per > 0 ? groups < m / per + (m % per != 0) : m > 0 && !(groups == 1 && per == 0))
            value_error(n + " has " + std::to_string(groups) + " rows of " + std::to_string(per) +
                        " tokens each, too few for " + std::to_string(m) + " tokens");
        if (per && m > per) {  // a single row serves every token, and its stride is not used
            const int64_t s = d == 1 ? k : t.stride(0);
            if (strided && s != stride) value_error("gate, mod_scale and mod_shift must have the same row stride");
            stride = s;
            strided = true;
        }
        mod[i] = t.data_ptr();
    }
    const c10::cuda::CUDAGuard guard(x.device());
    Tensor h, image, codes, y, sx;
    void* ph = dense(a[12], "h_out", type, shape);
    if (none(a[12])) {
        h = empty(shape, type, x);
        ph = h.data_ptr();
    } else {
        h = THPVariable_Unpack(a[12]);
    }
    if (truth(a[13])) image = empty(shape, bf16, x);
    if (truth(a[14])) codes = empty(shape, ScalarType::Char, x);
    if (truth(a[15])) y = empty(shape, bf16, x);
    if (image.defined() || codes.defined()) sx = empty({m}, ScalarType::Float, x);
    const auto at_ = [](const Tensor& t) { return t.defined() ? t.data_ptr() : nullptr; };
    const w8a8_status s = w8a8_residual_norm_quant(
        px, pb, ph, dtype_of(type), branch_gamma, gamma, beta, mod[0], mod[1], mod[2], stride, per,
        static_cast<float>(number(a[6])), static_cast<float>(number(a[4])), static_cast<w8a8_norm_kind>(integer(a[5])), m,
        k, at_(y), static_cast<int8_t*>(at_(codes)), at_(image), static_cast<float*>(at_(sx)),
        c10::cuda::getCurrentCUDAStream().stream());
    if (s != W8A8_OK) return status(s);
    bump_written(a, arguments);
    return Py_BuildValue("(NNNNN)", wrap(h), wrap(image), wrap(sx), wrap(codes), wrap(y));
}

template <PyObject* (*F)(PyObject* const*), int N>
PyObject* call(PyObject*, PyObject* const* args, Py_ssize_t n) {
    if (n != N) {
        PyErr_Format(PyExc_TypeError, "expected %d arguments, got %zd", N, n);
        return nullptr;
    }
    try {
        return F(args);
    } catch (const Refused& r) {
        if (r.type) PyErr_SetString(r.type, r.text.c_str());
    } catch (const c10::OutOfMemoryError& e) {
        PyObject* torch = PyImport_ImportModule("torch");
        PyObject* type = torch ? PyObject_GetAttrString(torch, "OutOfMemoryError") : nullptr;
        if (type) PyErr_SetString(type, e.what_without_backtrace());  // else the error is set
        Py_XDECREF(type);
        Py_XDECREF(torch);
    } catch (const c10::Error& e) {
        PyErr_SetString(PyExc_RuntimeError, e.what_without_backtrace());
    } catch (const std::exception& e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
    }
    return nullptr;
}

#define W8A8_CALL(name, n) \
    {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(call<name, n>)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {W8A8_CALL(attention, 12), W8A8_CALL(rotary, 9), W8A8_CALL(rotary_append, 11),
                         W8A8_CALL(residual_norm_quant, 16), {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "w8a8_binding", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit_w8a8_binding() { return PyModule_Create(&module); }
