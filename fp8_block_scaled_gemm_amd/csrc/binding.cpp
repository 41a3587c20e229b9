// Python entry to the operators of include/dg_ops.h: checks torch tensors,
// allocates outputs and workspaces that the caller did not give from torch's
// caching allocator, and calls the C ABI.  These calls run a few microseconds
// on the GPU, and checking ten tensors in Python took as long; here it takes
// about one (one row with adapters: 14.4 -> 6.8 us of host time per call).
//
// Each function takes positional arguments only (the wrappers in __init__.py
// give them their names and defaults), the raw stream last, and returns its
// outputs, or the C call's status as an int when that is not DG_OK.  Checks
// raise TypeError or ValueError, like the other functions of the package.
#include <Python.h>

#include <ATen/ATen.h>
#include <c10/core/GradMode.h>
#include <torch/csrc/autograd/python_variable.h>

#include <sstream>
#include <stdexcept>
#include <string>

#include "dg_ops.h"
#include "on_device.h"

namespace {

struct Bad {
    PyObject* kind;  // borrowed: an exception class
    std::string text;
};

// Thrown when a Python error is already set.
struct PythonError {};

std::string shape_text(at::IntArrayRef s) {
    std::ostringstream o;
    o << "(";
    for (size_t i = 0; i < s.size(); ++i) o << (i ? ", " : "") << s[i];
    o << (s.size() == 1 ? ",)" : ")");
    return o.str();
}

const at::Tensor& tensor(PyObject* o, const char* what) {
    if (!THPVariable_Check(o)) throw Bad{PyExc_TypeError, std::string(what) + " must be a torch.Tensor"};
    return THPVariable_Unpack(o);
}

// A GPU tensor of n dimensions, from which the call's sizes are read.
const at::Tensor& sized(PyObject* o, const char* what, int64_t n) {
    const at::Tensor& t = tensor(o, what);
    if (t.dim() != n)
        throw Bad{PyExc_ValueError, std::string(what) + " must have " + std::to_string(n) +
                                        " dimensions, got shape " + shape_text(t.sizes())};
    if (!t.is_cuda()) throw Bad{PyExc_ValueError, std::string(what) + " must be on the GPU"};
    return t;
}

bool one_of(at::ScalarType t, std::initializer_list<at::ScalarType> types) {
    for (at::ScalarType a : types)
        if (a == t) return true;
    return false;
}

// The data pointer of a contiguous tensor of one of these types, of this
// shape, on this GPU.
void* pointer(const at::Tensor& t, const char* what, std::initializer_list<at::ScalarType> types,
              std::initializer_list<int64_t> shape, at::Device dev) {
    if (!t.is_cuda()) throw Bad{PyExc_ValueError, std::string(what) + " must be on the GPU"};
    if (!t.is_contiguous()) throw Bad{PyExc_ValueError, std::string(what) + " must be contiguous"};
    if (!one_of(t.scalar_type(), types))
        throw Bad{PyExc_TypeError, std::string(what) + " must be " + at::toString(*types.begin()) + ", got " +
                                       at::toString(t.scalar_type())};
    if (t.sizes() != at::IntArrayRef(shape.begin(), shape.size()))
        throw Bad{PyExc_ValueError, std::string(what) + " must have shape " +
                                        shape_text(at::IntArrayRef(shape.begin(), shape.size())) + ", got " +
                                        shape_text(t.sizes())};
    if (t.device() != dev)
        throw Bad{PyExc_ValueError, "all tensors of a call must be on one device, got " + dev.str() + " and " +
                                        t.device().str()};
    return t.data_ptr();
}

void* pointer(PyObject* o, const char* what, std::initializer_list<at::ScalarType> types,
              std::initializer_list<int64_t> shape, at::Device dev) {
    return pointer(tensor(o, what), what, types, shape, dev);
}

#define DG_CODES {at::kByte, at::kFloat8_e4m3fn}
#define DG_BITS {at::kBFloat16, at::kUInt16, at::kShort}

int64_t integer(PyObject* o) {
    const long long v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred()) throw PythonError{};
    return v;
}

float number(PyObject* o) {
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred()) throw PythonError{};
    return (float)v;
}

at::Tensor given_or_new(PyObject* o, const char* what, at::IntArrayRef shape, at::ScalarType type, at::Device dev) {
    if (o == Py_None) {
        for (int64_t n : shape)
            if (n < 0) throw Bad{PyExc_ValueError, std::string(what) + " cannot have shape " + shape_text(shape)};
        return at::empty(shape, at::TensorOptions().dtype(type).device(dev));
    }
    return tensor(o, what);
}

// The caller's workspace, or a new one.  It may be dropped once the call is
// enqueued: the allocator hands it out again on the same stream only.
at::Tensor workspace(PyObject* o, int64_t bytes, at::Device dev) {
    if (o == Py_None) return at::empty({std::max<int64_t>(bytes, 16)}, at::TensorOptions().dtype(at::kByte).device(dev));
    const at::Tensor& t = tensor(o, "workspace");
    if (t.scalar_type() != at::kByte || t.dim() != 1 || t.device() != dev || !t.is_contiguous())
        throw Bad{PyExc_ValueError, "workspace must be a contiguous one-dimensional uint8 tensor on the call's device"};
    return t;
}

// The interpreter lock is given up while the library enqueues: a launch waits
// where the stream's queue is full, and other threads (one of which may be what
// the stream waits for) go on meanwhile.
struct Unlocked {
    PyThreadState* const state = PyEval_SaveThread();
    Unlocked() = default;
    Unlocked(const Unlocked&) = delete;
    Unlocked& operator=(const Unlocked&) = delete;
    ~Unlocked() { PyEval_RestoreThread(state); }
};

template <class F>
dg_status unlocked(F call) {
    const Unlocked on;
    return call();
}

void* stream_of(PyObject* o) { return reinterpret_cast<void*>((uintptr_t)integer(o)); }

// A function's body behind Python's calling convention: argument count and
// exceptions.
template <Py_ssize_t kArgs, class F>
PyObject* guarded(PyObject* const* a, Py_ssize_t n, F body) {
    if (n != kArgs) {
        PyErr_Format(PyExc_TypeError, "expected %zd arguments, got %zd", kArgs, n);
        return nullptr;
    }
    try {
        return body(a);
    } catch (const Bad& e) {
        PyErr_SetString(e.kind, e.text.c_str());
    } catch (const PythonError&) {
    } catch (const std::exception& e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
    }
    return nullptr;
}

// logits, k, ids, weights, bias, n_group, topk_group, scoring, renormalize, scale, stream
PyObject* moe_topk(PyObject*, PyObject* const* args, Py_ssize_t n) {
    return guarded<11>(args, n, [](PyObject* const* a) -> PyObject* {
        const at::Tensor& x = sized(a[0], "logits", 2);
        const int64_t T = x.size(0), E = x.size(1), k = integer(a[1]);
        const at::Device dev = x.device();
        const bool bf16 = x.scalar_type() == at::kBFloat16;
        void* const px = pointer(x, "logits", {at::kFloat, at::kBFloat16}, {T, E}, dev);
        void* const pb = a[4] == Py_None ? nullptr : pointer(a[4], "bias", {at::kFloat}, {E}, dev);
        const at::Tensor ids = given_or_new(a[2], "ids", {T, k}, at::kInt, dev);
        const at::Tensor weights = given_or_new(a[3], "weights", {T, k}, at::kFloat, dev);
        int32_t* const pi = (int32_t*)pointer(ids, "ids", {at::kInt}, {T, k}, dev);
        float* const pw = (float*)pointer(weights, "weights", {at::kFloat}, {T, k}, dev);
        const int64_t groups = integer(a[5]), kept = integer(a[6]);
        const int scoring = (int)integer(a[7]), renormalize = (int)integer(a[8]);
        const float scale = number(a[9]);
        void* const stream = stream_of(a[10]);
        const OnDevice on(dev.index());
        const dg_status s = unlocked([&] {
            return bf16 ? dg_moe_topk_bf16((const uint16_t*)px, (const float*)pb, pi, pw, T, E, k, groups, kept, scoring,
                                           renormalize, scale, stream)
                        : dg_moe_topk((const float*)px, (const float*)pb, pi, pw, T, E, k, groups, kept, scoring,
                                      renormalize, scale, stream);
        });
        if (s != DG_OK) return PyLong_FromLong(s);
        PyObject* const out = PyTuple_New(2);
        if (out == nullptr) return nullptr;
        PyTuple_SET_ITEM(out, 0, a[2] == Py_None ? THPVariable_Wrap(ids) : Py_NewRef(a[2]));
        PyTuple_SET_ITEM(out, 1, a[3] == Py_None ? THPVariable_Wrap(weights) : Py_NewRef(a[3]));
        return out;
    });
}

// logits, ids, grad_weights, grad_logits, scoring, renormalize, scale, stream
PyObject* moe_topk_backward(PyObject*, PyObject* const* args, Py_ssize_t n) {
    return guarded<8>(args, n, [](PyObject* const* a) -> PyObject* {
        const at::Tensor& x = sized(a[0], "logits", 2);
        const int64_t T = x.size(0), E = x.size(1), k = sized(a[1], "ids", 2).size(1);
        const at::Device dev = x.device();
        const bool bf16 = x.scalar_type() == at::kBFloat16;
        void* const px = pointer(x, "logits", {at::kFloat, at::kBFloat16}, {T, E}, dev);
        const int32_t* const pi = (const int32_t*)pointer(a[1], "ids", {at::kInt}, {T, k}, dev);
        const float* const pg = (const float*)pointer(a[2], "grad_weights", {at::kFloat}, {T, k}, dev);
        const at::Tensor out = given_or_new(a[3], "grad_logits", {T, E}, x.scalar_type(), dev);
        void* const po = pointer(out, "grad_logits", {x.scalar_type()}, {T, E}, dev);
        const int scoring = (int)integer(a[4]), renormalize = (int)integer(a[5]);
        const float scale = number(a[6]);
        void* const stream = stream_of(a[7]);
        const OnDevice on(dev.index());
        const dg_status s = unlocked([&] {
            return bf16 ? dg_moe_topk_backward_bf16((const uint16_t*)px, pi, pg, (uint16_t*)po, T, E, k, scoring,
                                                    renormalize, scale, stream)
                        : dg_moe_topk_backward((const float*)px, pi, pg, (float*)po, T, E, k, scoring, renormalize, scale,
                                               stream);
        });
        if (s != DG_OK) return PyLong_FromLong(s);
        return a[3] == Py_None ? THPVariable_Wrap(out) : Py_NewRef(a[3]);
    });
}

int64_t e8m0_pitch(int64_t kb) { return (kb + 3) / 4 * 4; }

// e8m0, x, sx, ids, weights, w13, s13, w2, s2, y, workspace, stream
PyObject* moe_mlp(PyObject*, PyObject* const* args, Py_ssize_t n) {
    return guarded<12>(args, n, [](PyObject* const* a) -> PyObject* {
        const bool e8 = a[0] == Py_True;
        const at::Tensor& x = sized(a[1], "x", 2);
        const int64_t T = x.size(0), H = x.size(1), k = sized(a[3], "ids", 2).size(1);
        const at::Tensor& w2 = sized(a[7], "w2", 3);
        const int64_t E = w2.size(0), I = w2.size(2);
        const at::Device dev = x.device();
        const at::ScalarType st = e8 ? at::kByte : at::kFloat;
        const int64_t kh = e8 ? e8m0_pitch(H / 128) : H / 128, ki = e8 ? e8m0_pitch(I / 128) : I / 128;
        const auto* px = (const uint8_t*)pointer(x, "x", DG_CODES, {T, H}, dev);
        const void* const psx = pointer(a[2], "sx", {st}, {T, kh}, dev);
        const auto* pi = (const int32_t*)pointer(a[3], "ids", {at::kInt}, {T, k}, dev);
        const auto* pw = (const float*)pointer(a[4], "weights", {at::kFloat}, {T, k}, dev);
        const auto* p13 = (const uint8_t*)pointer(a[5], "w13", DG_CODES, {E, 2 * I, H}, dev);
        const void* const ps13 = pointer(a[6], "s13", {st}, {E, (2 * I + 127) / 128, kh}, dev);
        const auto* p2 = (const uint8_t*)pointer(w2, "w2", DG_CODES, {E, H, I}, dev);
        const void* const ps2 = pointer(a[8], "s2", {st}, {E, (H + 127) / 128, ki}, dev);
        const at::Tensor y = given_or_new(a[9], "y", {T, H}, at::kBFloat16, dev);
        auto* py = (uint16_t*)pointer(y, "y", DG_BITS, {T, H}, dev);
        int64_t bytes = 0;
        dg_status s = dg_moe_mlp_fp8_workspace(T, k, E, H, I, &bytes);
        if (s != DG_OK) return PyLong_FromLong(s);
        const at::Tensor ws = workspace(a[10], bytes, dev);
        void* const pws = ws.data_ptr();
        void* const stream = stream_of(a[11]);
        const OnDevice on(dev.index());
        s = unlocked([&] {
            return e8 ? dg_moe_mlp_fp8_e8m0(px, (const uint8_t*)psx, pi, pw, p13, (const uint8_t*)ps13, p2,
                                            (const uint8_t*)ps2, py, T, k, E, H, I, pws, ws.numel(), stream)
                      : dg_moe_mlp_fp8(px, (const float*)psx, pi, pw, p13, (const float*)ps13, p2, (const float*)ps2, py,
                                       T, k, E, H, I, pws, ws.numel(), stream);
        });
        if (s != DG_OK) return PyLong_FromLong(s);
        return a[9] == Py_None ? THPVariable_Wrap(y) : Py_NewRef(a[9]);
    });
}

// e8m0, A, sa, B, sb, D, x, lora_a, lora_b, ids, scaling, workspace, stream
PyObject* gemm_lora(PyObject*, PyObject* const* args, Py_ssize_t n) {
    return guarded<13>(args, n, [](PyObject* const* a) -> PyObject* {
        const bool e8 = a[0] == Py_True;
        const at::Tensor& A = sized(a[1], "A", 2);
        const at::Tensor& B = sized(a[3], "B", 2);
        const at::Tensor& la = sized(a[7], "lora_a", 3);
        const int64_t M = A.size(0), K = A.size(1), N = B.size(0), L = la.size(0), R = la.size(1);
        const at::Device dev = A.device();
        const at::ScalarType st = e8 ? at::kByte : at::kFloat;
        const int64_t kb = e8 ? e8m0_pitch(K / 128) : K / 128;
        const auto* pA = (const uint8_t*)pointer(A, "A", DG_CODES, {M, K}, dev);
        const void* const psa = pointer(a[2], "sa", {st}, {M, kb}, dev);
        const auto* pB = (const uint8_t*)pointer(B, "B", DG_CODES, {N, K}, dev);
        const void* const psb = pointer(a[4], "sb", {st}, {(N + 127) / 128, kb}, dev);
        auto* pD = (uint16_t*)pointer(a[5], "D", DG_BITS, {M, N}, dev);
        const auto* px = (const uint16_t*)pointer(a[6], "x", {at::kBFloat16}, {M, K}, dev);
        const auto* pa = (const uint16_t*)pointer(la, "lora_a", {at::kBFloat16}, {L, R, K}, dev);
        const auto* pb = (const uint16_t*)pointer(a[8], "lora_b", {at::kBFloat16}, {L, N, R}, dev);
        const auto* pi = (const int32_t*)pointer(a[9], "ids", {at::kInt}, {M}, dev);
        const auto* ps = (const float*)pointer(a[10], "scaling", {at::kFloat}, {L}, dev);
        int64_t bytes = 0;
        dg_status s = dg_fp8_gemm_nt_lora_workspace(M, N, K, L, R, &bytes);
        if (s != DG_OK) return PyLong_FromLong(s);
        const at::Tensor ws = workspace(a[11], bytes, dev);
        void* const pws = ws.data_ptr();
        void* const stream = stream_of(a[12]);
        const OnDevice on(dev.index());
        s = unlocked([&] {
            return e8 ? dg_fp8_gemm_nt_lora_e8m0(pA, (const uint8_t*)psa, pB, (const uint8_t*)psb, pD, px, pa, pb, pi, ps,
                                                 M, N, K, L, R, pws, ws.numel(), stream)
                      : dg_fp8_gemm_nt_lora(pA, (const float*)psa, pB, (const float*)psb, pD, px, pa, pb, pi, ps, M, N, K,
                                            L, R, pws, ws.numel(), stream);
        });
        if (s != DG_OK) return PyLong_FromLong(s);
        return Py_NewRef(a[5]);
    });
}

// Whether gradients are recorded and any of the arguments is a tensor that requires one.
PyObject* wants_grad(PyObject*, PyObject* const* a, Py_ssize_t n) {
    if (c10::GradMode::is_enabled())
        for (Py_ssize_t i = 0; i < n; ++i)
            if (THPVariable_Check(a[i]) && THPVariable_Unpack(a[i]).requires_grad()) Py_RETURN_TRUE;
    Py_RETURN_FALSE;
}

#define DG_METHOD(name) {#name, (PyCFunction)(void (*)())name, METH_FASTCALL, nullptr}
PyMethodDef methods[] = {DG_METHOD(moe_topk), DG_METHOD(moe_topk_backward), DG_METHOD(moe_mlp), DG_METHOD(gemm_lora),
                         DG_METHOD(wants_grad),
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__binding() { return PyModule_Create(&module); }
