// Python entry to the operators of include/dg_ops.h, dg_experts.h and
// dg_int8.h: checks torch tensors,
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
#include <ATen/core/LegacyTypeDispatch.h>
#include <c10/core/AutogradState.h>
#include <c10/core/GradMode.h>
#include <torch/csrc/autograd/python_variable.h>

#include <sstream>
#include <stdexcept>
#include <string>
#include <utility>

#include "dg_experts.h"
#include "dg_int8.h"
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

// A tensor that the caller gave and the call wrote.  Its version goes up, so that
// a recorded graph that saved it before refuses to go back with other values.
PyObject* written(PyObject* given) {
    const at::Tensor& t = THPVariable_Unpack(given);
    if (!t.is_inference()) t.unsafeGetTensorImpl()->bump_version();
    return Py_NewRef(given);
}

// The tensor that a caller gave, or the new one.
PyObject* returned(PyObject* given, const at::Tensor& t) {
    return given == Py_None ? THPVariable_Wrap(t) : written(given);
}

// A tuple of the calls' outputs; `given` are the arguments they came as.
PyObject* returned(std::initializer_list<std::pair<PyObject*, const at::Tensor*>> outs) {
    PyObject* const tuple = PyTuple_New((Py_ssize_t)outs.size());
    if (tuple == nullptr) return nullptr;
    Py_ssize_t i = 0;
    for (const auto& o : outs) PyTuple_SET_ITEM(tuple, i++, returned(o.first, *o.second));
    return tuple;
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
        return returned({{a[2], &ids}, {a[3], &weights}});
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
        return returned(a[3], out);
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
        return returned(a[9], y);
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
        return written(a[5]);
    });
}

// A pointer that may be left out: None.
void* pointer_or_null(PyObject* o, const char* what, std::initializer_list<at::ScalarType> types,
                      std::initializer_list<int64_t> shape, at::Device dev) {
    return o == Py_None ? nullptr : pointer(o, what, types, shape, dev);
}

// The plan of a sort: sizes, outputs that were given or are new, workspace.
struct Plan {
    int64_t T, k, E, M;
    at::Tensor rows, layout, offsets, ws;
    const int32_t* ids;
    int32_t *prows, *playout, *poffsets;
    dg_status status;

    // `held`: the buffer for the sorted rows, or None
    Plan(PyObject* o, PyObject* experts, PyObject* rows_, PyObject* layout_, PyObject* offsets_, PyObject* held,
         PyObject* workspace_) {
        const at::Tensor& t = sized(o, "ids", 2);
        const at::Device dev = t.device();
        T = t.size(0), k = t.size(1), E = integer(experts), M = 0;
        int64_t bytes = 0;
        if ((status = dg_moe_sort_rows(T, k, E, &M)) != DG_OK) return;
        if ((status = dg_moe_sort_workspace(T, k, E, &bytes)) != DG_OK) return;
        if (layout_ != Py_None)
            M = sized(layout_, "layout", 1).size(0);
        else if (held != Py_None)
            M = sized(held, "the rows' buffer", 2).size(0);
        ids = (const int32_t*)pointer(t, "ids", {at::kInt}, {T, k}, dev);
        if (rows_ == Py_None && layout_ == Py_None && offsets_ == Py_None) {
            // one allocation for the three: each takes longer than a kernel for
            // few tokens can spare (one token: 8.8 -> 6.2 us of host time)
            const int64_t at_rows = M, at_offsets = M + (T * k + 3) / 4 * 4;
            const at::Tensor all = at::empty({at_offsets + E + 1}, at::TensorOptions().dtype(at::kInt).device(dev));
            const at::AutoDispatchBelowADInplaceOrView plain;
            layout = all.as_strided({M}, {1}, 0);
            rows = all.as_strided({T, k}, {k, 1}, at_rows);
            offsets = all.as_strided({E + 1}, {1}, at_offsets);
        } else {
            rows = given_or_new(rows_, "rows", {T, k}, at::kInt, dev);
            layout = given_or_new(layout_, "layout", {M}, at::kInt, dev);
            offsets = given_or_new(offsets_, "offsets", {E + 1}, at::kInt, dev);
        }
        prows = (int32_t*)pointer(rows, "rows", {at::kInt}, {T, k}, dev);
        playout = (int32_t*)pointer(layout, "layout", {at::kInt}, {M}, dev);
        poffsets = (int32_t*)pointer(offsets, "offsets", {at::kInt}, {E + 1}, dev);
        if (bytes > 0 || workspace_ != Py_None) ws = workspace(workspace_, bytes, dev);
    }
    void* scratch() const { return ws.defined() ? ws.data_ptr() : nullptr; }
    int64_t scratch_bytes() const { return ws.defined() ? ws.numel() : 0; }
};

// ids, E, rows, layout, offsets, workspace, stream
PyObject* moe_sort(PyObject*, PyObject* const* args, Py_ssize_t n) {
    return guarded<7>(args, n, [](PyObject* const* a) -> PyObject* {
        const Plan p(a[0], a[1], a[2], a[3], a[4], Py_None, a[5]);
        if (p.status != DG_OK) return PyLong_FromLong(p.status);
        void* const stream = stream_of(a[6]);
        void* const pws = p.scratch();
        const OnDevice on(p.rows.device().index());
        const dg_status s = unlocked([&] {
            return dg_moe_sort(p.ids, p.prows, p.playout, p.poffsets, p.T, p.k, p.E, p.M, pws, p.scratch_bytes(), stream);
        });
        if (s != DG_OK) return PyLong_FromLong(s);
        return returned({{a[2], &p.rows}, {a[3], &p.layout}, {a[4], &p.offsets}});
    });
}

// How the rows of a dispatch or gate call are held, as __init__.py numbers them.
enum Held { kBf16 = 0, kFp8 = 1, kFp8E8 = 2, kInt8 = 3 };

// The codes or rows [M][width] and the scales of a call, given or new.
struct Rows {
    at::Tensor q, s;
    void *pq, *ps;

    Rows(int held, PyObject* q_, PyObject* s_, const char* name, int64_t M, int64_t width, at::Device dev) : ps(nullptr) {
        const int64_t kb = width / 128;
        const at::ScalarType qt = held == kBf16 ? at::kBFloat16 : held == kInt8 ? at::kChar : at::kByte;
        q = given_or_new(q_, name, {M, width}, qt, dev);
        if (held == kBf16) {
            pq = pointer(q, name, DG_BITS, {M, width}, dev);
            return;
        }
        pq = held == kInt8 ? pointer(q, name, {at::kChar}, {M, width}, dev) : pointer(q, name, DG_CODES, {M, width}, dev);
        if (held == kInt8) {
            s = given_or_new(s_, "s", {M}, at::kFloat, dev);
            ps = pointer(s, "s", {at::kFloat}, {M}, dev);
        } else if (held == kFp8) {
            s = given_or_new(s_, "s", {M, kb}, at::kFloat, dev);
            ps = pointer(s, "s", {at::kFloat}, {M, kb}, dev);
        } else {
            const int64_t pitch = e8m0_pitch(kb);
            s = given_or_new(s_, "s", {M, pitch}, at::kByte, dev);
            if (s_ == Py_None && pitch != kb) s.zero_();  // the padding bytes, which no kernel writes
            ps = pointer(s, "s", {at::kByte}, {M, pitch}, dev);
        }
    }
};

// held, x, ids, E, q, s, rows, layout, offsets, workspace, stream
PyObject* moe_dispatch(PyObject*, PyObject* const* args, Py_ssize_t n) {
    return guarded<11>(args, n, [](PyObject* const* a) -> PyObject* {
        const int held = (int)integer(a[0]);
        const at::Tensor& x = sized(a[1], "x", 2);
        const int64_t H = x.size(1);
        const at::Device dev = x.device();
        const Plan p(a[2], a[3], a[6], a[7], a[8], a[4], a[9]);
        if (p.status != DG_OK) return PyLong_FromLong(p.status);
        const auto* px = (const uint16_t*)pointer(x, "x", {at::kBFloat16}, {p.T, H}, dev);
        pointer(a[2], "ids", {at::kInt}, {p.T, p.k}, dev);  // on x's device
        const OnDevice on(dev.index());
        const Rows r(held, a[4], a[5], held == kBf16 ? "out" : "q", p.M, H, dev);
        void* const stream = stream_of(a[10]);
        void* const pws = p.scratch();
        const dg_status s = unlocked([&] {
            switch (held) {
                case kBf16:
                    return dg_moe_dispatch(px, p.ids, (uint16_t*)r.pq, p.prows, p.playout, p.poffsets, p.T, p.k, p.E, H, p.M,
                                           pws, p.scratch_bytes(), stream);
                case kFp8:
                    return dg_moe_dispatch_fp8(px, p.ids, (uint8_t*)r.pq, (float*)r.ps, p.prows, p.playout, p.poffsets, p.T,
                                               p.k, p.E, H, p.M, pws, p.scratch_bytes(), stream);
                case kFp8E8:
                    return dg_moe_dispatch_fp8_e8m0(px, p.ids, (uint8_t*)r.pq, (uint8_t*)r.ps, p.prows, p.playout,
                                                    p.poffsets, p.T, p.k, p.E, H, p.M, pws, p.scratch_bytes(), stream);
                default:
                    return dg_moe_dispatch_int8(px, p.ids, (int8_t*)r.pq, (float*)r.ps, p.prows, p.playout, p.poffsets, p.T,
                                                p.k, p.E, H, p.M, pws, p.scratch_bytes(), stream);
            }
        });
        if (s != DG_OK) return PyLong_FromLong(s);
        if (held == kBf16) return returned({{a[4], &r.q}, {a[6], &p.rows}, {a[7], &p.layout}, {a[8], &p.offsets}});
        return returned({{a[4], &r.q}, {a[5], &r.s}, {a[6], &p.rows}, {a[7], &p.layout}, {a[8], &p.offsets}});
    });
}

// y, rows, weights, out, stream
PyObject* moe_unpermute(PyObject*, PyObject* const* args, Py_ssize_t n) {
    return guarded<5>(args, n, [](PyObject* const* a) -> PyObject* {
        const at::Tensor& y = sized(a[0], "y", 2);
        const at::Tensor& rows = sized(a[1], "rows", 2);
        const int64_t M = y.size(0), H = y.size(1), T = rows.size(0), k = rows.size(1);
        const at::Device dev = y.device();
        const auto* py = (const uint16_t*)pointer(y, "y", {at::kBFloat16}, {M, H}, dev);
        const auto* pr = (const int32_t*)pointer(rows, "rows", {at::kInt}, {T, k}, dev);
        const auto* pw = (const float*)pointer_or_null(a[2], "weights", {at::kFloat}, {T, k}, dev);
        const at::Tensor out = given_or_new(a[3], "out", {T, H}, at::kBFloat16, dev);
        auto* po = (uint16_t*)pointer(out, "out", DG_BITS, {T, H}, dev);
        void* const stream = stream_of(a[4]);
        const OnDevice on(dev.index());
        const dg_status s = unlocked([&] { return dg_moe_unpermute(py, pr, pw, po, T, k, H, M, stream); });
        if (s != DG_OK) return PyLong_FromLong(s);
        return returned(a[3], out);
    });
}

// grad, y (an int: its rows, where the weights' gradient is not wanted), rows, weights, layout, grad_y,
// grad_weights, want_y, want_weights, stream
PyObject* moe_unpermute_backward(PyObject*, PyObject* const* args, Py_ssize_t n) {
    return guarded<10>(args, n, [](PyObject* const* a) -> PyObject* {
        const at::Tensor& g = sized(a[0], "grad", 2);
        const bool rows_only = PyLong_Check(a[1]);
        const at::Tensor& rows = sized(a[2], "rows", 2);
        const int64_t T = g.size(0), H = g.size(1), k = rows.size(1);
        const int64_t M = rows_only ? integer(a[1]) : sized(a[1], "y", 2).size(0);
        const at::Device dev = g.device();
        const bool want_y = a[7] == Py_True, want_w = a[8] == Py_True;
        const auto* pg = (const uint16_t*)pointer(g, "grad", {at::kBFloat16}, {T, H}, dev);
        const auto* py =
            rows_only ? nullptr : (const uint16_t*)pointer(a[1], "y", {at::kBFloat16}, {M, H}, dev);
        const auto* pr = (const int32_t*)pointer(rows, "rows", {at::kInt}, {T, k}, dev);
        const auto* pw = (const float*)pointer_or_null(a[3], "weights", {at::kFloat}, {T, k}, dev);
        const auto* pl = (const int32_t*)pointer_or_null(a[4], "layout", {at::kInt}, {M}, dev);
        const OnDevice on(dev.index());
        at::Tensor gy, gw;
        uint16_t* pgy = nullptr;
        float* pgw = nullptr;
        if (want_y) {
            gy = given_or_new(a[5], "grad_y", {M, H}, at::kBFloat16, dev);
            pgy = (uint16_t*)pointer(gy, "grad_y", DG_BITS, {M, H}, dev);
            if (a[5] == Py_None && pl == nullptr) gy.zero_();  // which rows are padding is not known
        }
        if (want_w) {
            gw = given_or_new(a[6], "grad_weights", {T, k}, at::kFloat, dev);
            pgw = (float*)pointer(gw, "grad_weights", {at::kFloat}, {T, k}, dev);
        }
        void* const stream = stream_of(a[9]);
        const dg_status s = unlocked([&] { return dg_moe_unpermute_backward(pg, py, pr, pw, pl, pgy, pgw, T, k, H, M, stream); });
        if (s != DG_OK) return PyLong_FromLong(s);
        PyObject* const out = PyTuple_New(2);
        if (out == nullptr) return nullptr;
        PyTuple_SET_ITEM(out, 0, want_y ? returned(a[5], gy) : Py_NewRef(Py_None));
        PyTuple_SET_ITEM(out, 1, want_w ? returned(a[6], gw) : Py_NewRef(Py_None));
        return out;
    });
}

// held, z, layout, q, s, stream
PyObject* swiglu(PyObject*, PyObject* const* args, Py_ssize_t n) {
    return guarded<6>(args, n, [](PyObject* const* a) -> PyObject* {
        const int held = (int)integer(a[0]);
        const at::Tensor& z = sized(a[1], "z", 2);
        const int64_t M = z.size(0), I = z.size(1) / 2;
        const at::Device dev = z.device();
        const auto* pz = (const uint16_t*)pointer(z, "z", {at::kBFloat16}, {M, 2 * I}, dev);
        const auto* pl = (const int32_t*)pointer_or_null(a[2], "layout", {at::kInt}, {M}, dev);
        const OnDevice on(dev.index());
        const Rows r(held, a[3], a[4], held == kBf16 ? "h" : "q", M, I, dev);
        void* const stream = stream_of(a[5]);
        const dg_status s = unlocked([&] {
            switch (held) {
                case kBf16: return dg_swiglu(pz, pl, (uint16_t*)r.pq, M, I, stream);
                case kFp8: return dg_swiglu_quantize_fp8(pz, pl, (uint8_t*)r.pq, (float*)r.ps, M, I, stream);
                case kFp8E8: return dg_swiglu_quantize_fp8_e8m0(pz, pl, (uint8_t*)r.pq, (uint8_t*)r.ps, M, I, stream);
                default: return dg_swiglu_quantize_int8(pz, pl, (int8_t*)r.pq, (float*)r.ps, M, I, stream);
            }
        });
        if (s != DG_OK) return PyLong_FromLong(s);
        if (held == kBf16) return returned(a[3], r.q);
        return returned({{a[3], &r.q}, {a[4], &r.s}});
    });
}

// z, grad_h, layout, grad_z, stream
PyObject* swiglu_backward(PyObject*, PyObject* const* args, Py_ssize_t n) {
    return guarded<5>(args, n, [](PyObject* const* a) -> PyObject* {
        const at::Tensor& z = sized(a[0], "z", 2);
        const int64_t M = z.size(0), I = z.size(1) / 2;
        const at::Device dev = z.device();
        const auto* pz = (const uint16_t*)pointer(z, "z", {at::kBFloat16}, {M, 2 * I}, dev);
        const auto* pg = (const uint16_t*)pointer(a[1], "grad_h", {at::kBFloat16}, {M, I}, dev);
        const auto* pl = (const int32_t*)pointer_or_null(a[2], "layout", {at::kInt}, {M}, dev);
        const at::Tensor out = given_or_new(a[3], "grad_z", {M, 2 * I}, at::kBFloat16, dev);
        auto* po = (uint16_t*)pointer(out, "grad_z", DG_BITS, {M, 2 * I}, dev);
        void* const stream = stream_of(a[4]);
        const OnDevice on(dev.index());
        const dg_status s = unlocked([&] { return dg_swiglu_backward(pz, pg, pl, po, M, I, stream); });
        if (s != DG_OK) return PyLong_FromLong(s);
        return returned(a[3], out);
    });
}

// A, sa, B, sb, D, grouped_layout (None: dense), stream
PyObject* int8_gemm(PyObject*, PyObject* const* args, Py_ssize_t n) {
    return guarded<7>(args, n, [](PyObject* const* a) -> PyObject* {
        const bool grouped = a[5] != Py_None;
        const at::Tensor& A = sized(a[0], "A", 2);
        const at::Tensor& B = sized(a[2], "B", grouped ? 3 : 2);
        const int64_t M = A.size(0), K = A.size(1), G = grouped ? B.size(0) : 1, N = B.size(grouped ? 1 : 0);
        const at::Device dev = A.device();
        const auto* pA = (const int8_t*)pointer(A, "A", {at::kChar}, {M, K}, dev);
        const auto* psa = (const float*)pointer(a[1], "sa", {at::kFloat}, {M}, dev);
        const auto* pB = (const int8_t*)(grouped ? pointer(B, "B", {at::kChar}, {G, N, K}, dev)
                                                 : pointer(B, "B", {at::kChar}, {N, K}, dev));
        const auto* psb = (const float*)(grouped ? pointer(a[3], "sb", {at::kFloat}, {G, N}, dev)
                                                 : pointer(a[3], "sb", {at::kFloat}, {N}, dev));
        auto* pD = (uint16_t*)pointer(a[4], "D", DG_BITS, {M, N}, dev);
        const auto* pl = (const int32_t*)pointer_or_null(a[5], "grouped_layout", {at::kInt}, {M}, dev);
        void* const stream = stream_of(a[6]);
        const OnDevice on(dev.index());
        const dg_status s = unlocked([&] {
            return grouped ? dg_int8_gemm_grouped_contiguous(pA, psa, pB, psb, pD, pl, M, N, K, G, stream)
                           : dg_int8_gemm_nt(pA, psa, pB, psb, pD, M, N, K, stream);
        });
        if (s != DG_OK) return PyLong_FromLong(s);
        return written(a[4]);
    });
}

// x, q, s, stream
PyObject* quantize_int8(PyObject*, PyObject* const* args, Py_ssize_t n) {
    return guarded<4>(args, n, [](PyObject* const* a) -> PyObject* {
        const at::Tensor& x = sized(a[0], "x", 2);
        const int64_t M = x.size(0), K = x.size(1);
        const at::Device dev = x.device();
        const bool bf16 = x.scalar_type() == at::kBFloat16;
        const void* const px = pointer(x, "x", {at::kFloat, at::kBFloat16}, {M, K}, dev);
        const Rows r(kInt8, a[1], a[2], "q", M, K, dev);
        void* const stream = stream_of(a[3]);
        const OnDevice on(dev.index());
        const dg_status s = unlocked([&] {
            return bf16 ? dg_quantize_int8_per_row_bf16((const uint16_t*)px, M, K, (int8_t*)r.pq, (float*)r.ps, stream)
                        : dg_quantize_int8_per_row((const float*)px, M, K, (int8_t*)r.pq, (float*)r.ps, stream);
        });
        if (s != DG_OK) return PyLong_FromLong(s);
        return returned({{a[1], &r.q}, {a[2], &r.s}});
    });
}

// Whether any of the arguments is a tensor that requires a gradient where those
// are recorded, or carries a forward-mode tangent, which the calls' functions
// refuse (a plain call would drop it).
PyObject* wants_grad(PyObject*, PyObject* const* a, Py_ssize_t n) {
    const bool backward = c10::GradMode::is_enabled(), forward = c10::AutogradState::get_tls_state().get_fw_grad_mode();
    for (Py_ssize_t i = 0; i < n; ++i) {
        if (!THPVariable_Check(a[i])) continue;
        const at::Tensor& t = THPVariable_Unpack(a[i]);
        if ((backward && t.requires_grad()) || (forward && t._fw_grad(0).defined())) Py_RETURN_TRUE;
    }
    Py_RETURN_FALSE;
}

#define DG_METHOD(name) {#name, (PyCFunction)(void (*)())name, METH_FASTCALL, nullptr}
PyMethodDef methods[] = {DG_METHOD(moe_topk), DG_METHOD(moe_topk_backward), DG_METHOD(moe_mlp), DG_METHOD(gemm_lora),
                         DG_METHOD(wants_grad), DG_METHOD(moe_sort), DG_METHOD(moe_dispatch), DG_METHOD(moe_unpermute),
                         DG_METHOD(moe_unpermute_backward), DG_METHOD(swiglu), DG_METHOD(swiglu_backward),
                         DG_METHOD(int8_gemm), DG_METHOD(quantize_int8),
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__binding() { return PyModule_Create(&module); }
