// kla_binding.cpp -- Python binding of the mixer operators (kla_gated_scan_*,
// kla_rotary_forward, kla_qk_norm_rotary_* of include/kla.h) as a CPython
// extension: argument checks, the tensors that a call returns, the stream, and
// one call of the C ABI.  A decode step or a short batch takes the GPU one to
// four microseconds; marshalling it in Python took six to seventeen.
//
// Work goes to `stream` (None: the current stream of the tensors' device), and
// what a call allocates belongs to that stream, whichever one is current.  Other
// Python threads run while it allocates and launches: an allocation may wait for
// the device, a launch waits where the stream's queue is full.
#include "kla.h"

#include <ATen/ATen.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <array>
#include <exception>
#include <optional>
#include <sstream>
#include <string>

namespace {

using at::Tensor;

PyObject *g_error = nullptr;  // KlaError(status, name of the call)

// A Python exception, thrown through the C++ frames of a call.
struct Refused : std::exception {};
[[noreturn]] void refuse(PyObject *type, const std::string &what) {
    PyErr_SetString(type, what.c_str());
    throw Refused();
}

template <typename... A>
std::string text(const A &...a) {
    std::ostringstream s;
    (s << ... << a);
    return s.str();
}
std::string dtype_name(at::ScalarType t) {
    PyObject *o = PyObject_Str(reinterpret_cast<PyObject *>(torch::getTHPDtype(t)));
    std::string s = o ? PyUnicode_AsUTF8(o) : "?";
    Py_XDECREF(o);
    return s;
}

// Python's lock, let go of while this lives.
struct Unlocked {
    PyThreadState *state = PyEval_SaveThread();
    ~Unlocked() { PyEval_RestoreThread(state); }
};

const Tensor &tensor(PyObject *o, const char *name) {
    if (!THPVariable_Check(o)) refuse(PyExc_TypeError, text(name, " must be a tensor"));
    return THPVariable_Unpack(o);
}

// What the tensors of a call have in common: their device.
struct Place {
    c10::Device device;
    explicit Place(const Tensor &t) : device(t.device()) {}

    void here(const char *name, const Tensor &t) const {
        if (t.device() != device)
            refuse(PyExc_ValueError, text(name, " must be on the device of the other tensors; it is on ", t.device()));
    }
    // The address of a dense tensor of this shape and type.
    void *dense(const char *name, const Tensor &t, at::IntArrayRef shape, at::ScalarType type) const {
        if (t.sizes() != shape) refuse(PyExc_ValueError, text(name, " must be ", shape, ", got ", t.sizes()));
        if (t.scalar_type() != type)
            refuse(PyExc_TypeError, text(name, " must be ", dtype_name(type), ", got ", dtype_name(t.scalar_type())));
        here(name, t);
        if (!t.is_contiguous()) refuse(PyExc_ValueError, text(name, " must be contiguous"));
        return t.data_ptr();
    }
    // The same of an argument that may be None (null).
    void *maybe(const char *name, PyObject *o, at::IntArrayRef shape, at::ScalarType type) const {
        return o == Py_None ? nullptr : dense(name, tensor(o, name), shape, type);
    }
    Tensor empty(at::IntArrayRef shape, at::ScalarType type) const {
        return at::empty(shape, at::TensorOptions().dtype(type).device(device));
    }
};

// The device and stream of a call, current while it lasts.
struct Enqueue {
    std::optional<c10::cuda::CUDAStreamGuard> other;
    std::optional<c10::cuda::CUDAGuard> device;
    cudaStream_t handle = nullptr;

    Enqueue(const Place &at, PyObject *stream) {
        if (!at.device.is_cuda()) refuse(PyExc_ValueError, "tensors must be on a CUDA device");
        if (stream != Py_None) {
            auto field = [&](const char *name) -> int64_t {
                PyObject *o = PyObject_GetAttrString(stream, name);
                if (!o) throw Refused();
                const int64_t v = PyLong_AsLongLong(o);
                Py_DECREF(o);
                if (v == -1 && PyErr_Occurred()) throw Refused();
                return v;
            };
            const auto s = c10::cuda::CUDAStream::unpack3(field("stream_id"), (c10::DeviceIndex)field("device_index"),
                                                          (c10::DeviceType)field("device_type"));
            if (s.device() != at.device)
                refuse(PyExc_ValueError, text("the stream is on ", s.device(), ", the tensors on ", at.device));
            other.emplace(s);
            handle = s.stream();
        } else {
            if (c10::cuda::current_device() != at.device.index()) device.emplace(at.device);
            handle = c10::cuda::getCurrentCUDAStream(at.device.index()).stream();
        }
    }
};

void check(kla_status_t status, const char *name) {
    if (status == KLA_OK) return;
    PyObject *e = PyObject_CallFunction(g_error, "is", (int)status, name);
    if (e) PyErr_SetObject(g_error, e);
    Py_XDECREF(e);
    throw Refused();
}

// The part of a call that allocates and launches, without Python's lock.
template <typename F>
void enqueue(const char *name, F part) {
    kla_status_t status;
    {
        const Unlocked others;
        status = part();
    }
    check(status, name);
}

kla_dtype_t code_of(const Tensor &t) {
    if (t.scalar_type() == at::kFloat) return KLA_F32;
    if (t.scalar_type() == at::kBFloat16) return KLA_BF16;
    refuse(PyExc_TypeError, text("inputs must be float32 or bfloat16, got ", dtype_name(t.scalar_type())));
}

// The gate layout of f for states of `shape` ([.., H, N]).
kla_gate_t gate_of(const Tensor &f, at::IntArrayRef shape) {
    if (f.sizes() == shape) return KLA_GATE_CHANNEL;
    if (f.sizes() == shape.slice(0, shape.size() - 1)) return KLA_GATE_HEAD;
    refuse(PyExc_ValueError, text("f must be ", shape, " (a gate per channel) or ", shape.slice(0, shape.size() - 1),
                                  " (shared by a head), got ", f.sizes()));
}

bool truth(PyObject *o) {
    const int t = PyObject_IsTrue(o);
    if (t < 0) throw Refused();
    return t != 0;
}
int64_t integer(PyObject *o) {
    const int64_t v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred()) throw Refused();
    return v;
}
float real(PyObject *o) {
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred()) throw Refused();
    return (float)v;
}

PyObject *wrap(const Tensor &t) {
    if (t.defined()) return THPVariable_Wrap(t);
    Py_RETURN_NONE;
}
template <typename... T>
PyObject *tuple(const T &...t) {
    PyObject *o = PyTuple_New(sizeof...(T));
    if (!o) throw Refused();
    Py_ssize_t i = 0;
    ((PyTuple_SET_ITEM(o, i++, wrap(t))), ...);
    return o;
}
// A given tensor was written: autograd counts versions, and refuses to use what
// it saved from before (such as the states that a view of them steps on from).
void written(PyObject *o) {
    const Tensor &t = THPVariable_Unpack(o);
    if (!t.is_inference()) t.unsafeGetTensorImpl()->bump_version();
}
// The argument itself where it was given, else the new tensor.
PyObject *given_or(PyObject *o, const Tensor &t) {
    if (o == Py_None) return wrap(t);
    written(o);
    Py_INCREF(o);
    return o;
}
void *address(const Tensor &t) { return t.defined() ? t.data_ptr() : nullptr; }

// A caller's workspace, or a new one.
struct Workspace {
    Tensor own;
    void *p = nullptr;
    size_t bytes = 0;
    Workspace(const Place &at, PyObject *given) {
        if (given == Py_None) return;
        const Tensor &t = tensor(given, "workspace");
        p = at.dense("workspace", t, t.sizes(), t.scalar_type());
        bytes = t.nbytes();
    }
    // A new one of `need` bytes (0: none, or there is a given one).
    void have(const Place &at, size_t need) {
        if (need == 0) return;
        own = at.empty({(int64_t)need}, at::kByte);
        p = own.data_ptr();
        bytes = need;
    }
};

// ---- the gated recurrence ----------------------------------------------------
// (f, x, h0, out, stream)
PyObject *gated_scan_forward(PyObject *const *a) {
    const Tensor &f = tensor(a[0], "f"), &x = tensor(a[1], "x");
    const auto s = x.sizes();
    if (s.size() != 4) refuse(PyExc_ValueError, "x must be [B, T, H, N]");
    const kla_dtype_t code = code_of(x);
    if (f.scalar_type() != x.scalar_type()) refuse(PyExc_TypeError, "f and x must share one dtype");
    const kla_gate_t gate = gate_of(f, s);
    const Place at(x);
    const void *pf = at.dense("f", f, f.sizes(), x.scalar_type()), *px = at.dense("x", x, s, x.scalar_type());
    const void *h0 = at.maybe("h0", a[2], {s[0], s[2], s[3]}, at::kFloat);
    void *ph = at.maybe("out", a[3], s, at::kFloat);
    const Enqueue on(at, a[4]);
    Tensor h;
    enqueue("kla_gated_scan_forward", [&] {
        if (a[3] == Py_None) {
            h = at.empty(s, at::kFloat);
            ph = h.data_ptr();
        }
        return kla_gated_scan_forward(pf, px, code, gate, static_cast<const float *>(h0), static_cast<float *>(ph), s[0],
                                      s[1], s[2], s[3], on.handle);
    });
    return given_or(a[3], h);
}

// (f, x, h_state, out, stream)
PyObject *gated_scan_step(PyObject *const *a) {
    const Tensor &f = tensor(a[0], "f"), &x = tensor(a[1], "x");
    const auto s = x.sizes();
    if (s.size() != 3) refuse(PyExc_ValueError, "x must be [B, H, N]");
    const kla_dtype_t code = code_of(x);
    if (f.scalar_type() != x.scalar_type()) refuse(PyExc_TypeError, "f and x must share one dtype");
    const kla_gate_t gate = gate_of(f, s);
    const Place at(x);
    const void *pf = at.dense("f", f, f.sizes(), x.scalar_type()), *px = at.dense("x", x, s, x.scalar_type());
    void *h = at.dense("h_state", tensor(a[2], "h_state"), s, at::kFloat);
    PyObject *out = a[3] == Py_None ? a[2] : a[3];
    void *ph = a[3] == Py_None ? h : at.dense("out", tensor(a[3], "out"), s, at::kFloat);
    const Enqueue on(at, a[4]);
    enqueue("kla_gated_scan_step", [&] {
        return kla_gated_scan_step(pf, px, code, gate, static_cast<const float *>(h), static_cast<float *>(ph), s[0], s[1],
                                   s[2], on.handle);
    });
    return given_or(out, Tensor());
}

// (f, h, g_h, h0, three of want, workspace, stream)
PyObject *gated_scan_backward(PyObject *const *a) {
    const Tensor &f = tensor(a[0], "f"), &h = tensor(a[1], "h");
    const auto s = h.sizes();
    if (s.size() != 4) refuse(PyExc_ValueError, "h must be the forward output, [B, T, H, N]");
    const kla_gate_t gate = gate_of(f, s);
    const kla_dtype_t code = code_of(f);
    const Place at(h);
    const void *pf = at.dense("f", f, f.sizes(), f.scalar_type()), *ph = at.dense("h", h, s, at::kFloat);
    const void *pg = at.dense("g_h", tensor(a[2], "g_h"), s, at::kFloat);
    const void *h0 = at.maybe("h0", a[3], {s[0], s[2], s[3]}, at::kFloat);
    const bool want[3] = {truth(a[4]), truth(a[5]), truth(a[6])};
    size_t need = 0;
    if (want[0] && a[7] == Py_None)
        check(kla_gated_scan_backward_workspace_size(s[0], s[1], s[2], s[3], code, gate, &need),
              "kla_gated_scan_backward_workspace_size");
    const Enqueue on(at, a[8]);
    Workspace room(at, a[7]);
    Tensor gf, gx, gh0;
    enqueue("kla_gated_scan_backward", [&] {
        room.have(at, need);
        if (want[0]) gf = at.empty(f.sizes(), f.scalar_type());
        if (want[1]) gx = at.empty(s, f.scalar_type());
        if (want[2]) gh0 = at.empty({s[0], s[2], s[3]}, at::kFloat);
        return kla_gated_scan_backward(pf, code, gate, static_cast<const float *>(h0), static_cast<const float *>(ph),
                                       static_cast<const float *>(pg), address(gf), address(gx),
                                       static_cast<float *>(address(gh0)), s[0], s[1], s[2], s[3], room.p, room.bytes,
                                       on.handle);
    });
    return tuple(gf, gx, gh0);
}

// ---- rotation and norm ---------------------------------------------------------
// The strides of [B, T, H, D] rows.
std::array<int64_t, 3> strides_of(const char *name, const Tensor &t) {
    const auto st = t.strides();
    if (st[3] != 1 && t.size(3) > 1) refuse(PyExc_ValueError, text("the last axis of ", name, " must be contiguous"));
    return {st[0], st[1], st[2]};
}

struct Rotation {
    const double *freq = nullptr;
    int64_t rot = 0;
    const int64_t *positions = nullptr;
    int64_t stride = 0;

    Rotation(const Place &at, int64_t B, int64_t T, int64_t D, PyObject *inv_freq, PyObject *pos) {
        if (inv_freq == Py_None) {
            if (pos != Py_None) refuse(PyExc_ValueError, "positions need inv_freq");
            return;
        }
        const Tensor &f = tensor(inv_freq, "inv_freq");
        if (f.dim() != 1 || 2 * f.size(0) > D)
            refuse(PyExc_ValueError, text("inv_freq must be [rot_dim / 2] with rot_dim at most ", D, ", got ", f.sizes()));
        freq = static_cast<const double *>(at.dense("inv_freq", f, f.sizes(), at::kDouble));
        rot = 2 * f.size(0);
        if (pos == Py_None) return;
        const Tensor &p = tensor(pos, "positions");
        if (p.scalar_type() != at::kLong)
            refuse(PyExc_TypeError, text("positions must be torch.int64, got ", dtype_name(p.scalar_type())));
        at.here("positions", p);
        const bool each = p.dim() == 2 && p.size(0) == B && p.size(1) == T;
        if (!each && !(p.dim() == 1 && p.size(0) == T))
            refuse(PyExc_ValueError, text("positions must be [", B, ", ", T, "] or [", T, "], got ", p.sizes()));
        if (T > 1 && p.stride(-1) != 1) refuse(PyExc_ValueError, "the last axis of positions must be contiguous");
        positions = static_cast<const int64_t *>(p.data_ptr());
        stride = each && B > 1 ? p.stride(0) : 0;
    }
};

// (x, inv_freq, positions, position0, interleaved, scale, inverse, out, stream)
PyObject *rotary_forward(PyObject *const *a) {
    const Tensor &x = tensor(a[0], "x");
    const auto s = x.sizes();
    if (s.size() != 4) refuse(PyExc_ValueError, "x must be [B, T, H, D]");
    const kla_dtype_t code = code_of(x);
    const auto strides = strides_of("x", x);
    const Place at(x);
    const Rotation r(at, s[0], s[1], s[3], a[1], a[2]);
    void *py = at.maybe("out", a[7], s, x.scalar_type());
    const int64_t position0 = integer(a[3]);
    const bool interleaved = truth(a[4]), inverse = truth(a[6]);
    const float scale = real(a[5]);
    const Enqueue on(at, a[8]);
    Tensor y;
    enqueue("kla_rotary_forward", [&] {
        if (a[7] == Py_None) {
            y = at.empty(s, x.scalar_type());
            py = y.data_ptr();
        }
        return kla_rotary_forward(x.data_ptr(), strides.data(), code, r.freq, r.rot, interleaved, scale, inverse,
                                  r.positions, r.stride, position0, py, s[0], s[1], s[2], s[3], on.handle);
    });
    return given_or(a[7], y);
}

// The inputs that the two passes of QK-Norm share: (q, k, q_weight, k_weight,
// inv_freq, positions, position0, eps, interleaved, scale, ...)
struct QK {
    const Tensor &q, &k;
    Place at;
    kla_dtype_t code;
    std::array<int64_t, 3> qs, ks;
    const float *qw, *kw;
    Rotation r;
    int64_t position0;
    float eps, scale;
    int interleaved;

    static const Tensor &shaped(const Tensor &q, const Tensor &k) {
        if (q.dim() != 4 || k.dim() != 4 || q.size(0) != k.size(0) || q.size(1) != k.size(1) || q.size(3) != k.size(3))
            refuse(PyExc_ValueError, "q must be [B, T, Hq, D] and k [B, T, Hk, D]");
        if (k.scalar_type() != q.scalar_type())
            refuse(PyExc_TypeError,
                   text("k must be ", dtype_name(q.scalar_type()), ", got ", dtype_name(k.scalar_type())));
        return q;
    }
    explicit QK(PyObject *const *a)
        : q(shaped(tensor(a[0], "q"), tensor(a[1], "k"))), k(tensor(a[1], "k")), at(q), code(code_of(q)),
          qs(strides_of("q", q)), ks(strides_of("k", k)),
          qw(static_cast<const float *>(at.maybe("q_weight", a[2], {q.size(3)}, at::kFloat))),
          kw(static_cast<const float *>(at.maybe("k_weight", a[3], {q.size(3)}, at::kFloat))),
          r(at, q.size(0), q.size(1), q.size(3), a[4], a[5]), position0(integer(a[6])), eps(real(a[7])),
          scale(real(a[9])), interleaved(truth(a[8])) {
        at.here("k", k);
    }
};

// (the ten of QK, q_out, k_out, stream)
PyObject *qk_norm_rotary_forward(PyObject *const *a) {
    const QK c(a);
    const auto type = c.q.scalar_type();
    void *pq = c.at.maybe("out", a[10], c.q.sizes(), type), *pk = c.at.maybe("out", a[11], c.k.sizes(), type);
    const Enqueue on(c.at, a[12]);
    Tensor yq, yk;
    enqueue("kla_qk_norm_rotary_forward", [&] {
        if (a[10] == Py_None) {
            yq = c.at.empty(c.q.sizes(), type);
            pq = yq.data_ptr();
        }
        if (a[11] == Py_None) {
            yk = c.at.empty(c.k.sizes(), type);
            pk = yk.data_ptr();
        }
        return kla_qk_norm_rotary_forward(c.q.data_ptr(), c.qs.data(), c.k.data_ptr(), c.ks.data(), c.code, c.qw, c.kw,
                                          c.eps, c.r.freq, c.r.rot, c.interleaved, c.scale, c.r.positions, c.r.stride,
                                          c.position0, pq, pk, c.q.size(0), c.q.size(1), c.q.size(2), c.k.size(2),
                                          c.q.size(3), on.handle);
    });
    PyObject *o = PyTuple_New(2);
    if (!o) throw Refused();
    PyTuple_SET_ITEM(o, 0, given_or(a[10], yq));
    PyTuple_SET_ITEM(o, 1, given_or(a[11], yk));
    return o;
}

// (the ten of QK, g_q, g_k, four of want, workspace, stream)
PyObject *qk_norm_rotary_backward(PyObject *const *a) {
    const QK c(a);
    const auto type = c.q.scalar_type();
    const void *gq = c.at.maybe("g_q", a[10], c.q.sizes(), type), *gk = c.at.maybe("g_k", a[11], c.k.sizes(), type);
    const bool has_q = a[10] != Py_None, has_k = a[11] != Py_None;
    const bool want[4] = {truth(a[12]) && has_q, truth(a[13]) && has_k, truth(a[14]) && has_q && c.qw,
                          truth(a[15]) && has_k && c.kw};
    const int64_t D = c.q.size(3);
    const Enqueue on(c.at, a[17]);
    size_t need = 0;  // it depends on the current device
    if ((want[2] || want[3]) && a[16] == Py_None)
        check(kla_qk_norm_rotary_backward_workspace_size(c.q.size(2), c.k.size(2), D, &need),
              "kla_qk_norm_rotary_backward_workspace_size");
    Workspace room(c.at, a[16]);
    Tensor dq, dk, dqw, dkw;
    enqueue("kla_qk_norm_rotary_backward", [&] {
        room.have(c.at, need);
        if (want[0]) dq = c.at.empty(c.q.sizes(), type);
        if (want[1]) dk = c.at.empty(c.k.sizes(), type);
        if (want[2]) dqw = c.at.empty({D}, at::kFloat);
        if (want[3]) dkw = c.at.empty({D}, at::kFloat);
        return kla_qk_norm_rotary_backward(c.q.data_ptr(), c.qs.data(), c.k.data_ptr(), c.ks.data(), c.code, c.qw, c.kw,
                                           c.eps, c.r.freq, c.r.rot, c.interleaved, c.scale, c.r.positions, c.r.stride,
                                           c.position0, gq, gk, address(dq), address(dk),
                                           static_cast<float *>(address(dqw)), static_cast<float *>(address(dkw)),
                                           c.q.size(0), c.q.size(1), c.q.size(2), c.k.size(2), D, room.p, room.bytes,
                                           on.handle);
    });
    return tuple(dq, dk, dqw, dkw);
}

// Entry of a function of exactly N arguments: no C++ exception leaves it.
template <PyObject *(*F)(PyObject *const *), int N>
PyObject *entry(PyObject *, PyObject *const *args, Py_ssize_t n) {
    if (n != N) {
        PyErr_Format(PyExc_TypeError, "takes %d arguments, got %zd", N, n);
        return nullptr;
    }
    try {
        return F(args);
    } catch (const Refused &) {  // the Python error is set
    } catch (...) {
        torch::translate_exception_to_python(std::current_exception());
    }
    return nullptr;
}

PyObject *set_error(PyObject *, PyObject *type) {
    Py_INCREF(type);
    Py_XDECREF(g_error);
    g_error = type;
    Py_RETURN_NONE;
}

#define KLA_ENTRY(name, n) {#name, reinterpret_cast<PyCFunction>(entry<name, n>), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {
    KLA_ENTRY(gated_scan_forward, 5),
    KLA_ENTRY(gated_scan_step, 5),
    KLA_ENTRY(gated_scan_backward, 9),
    KLA_ENTRY(rotary_forward, 9),
    KLA_ENTRY(qk_norm_rotary_forward, 13),
    KLA_ENTRY(qk_norm_rotary_backward, 18),
    {"set_error", set_error, METH_O, nullptr},
    {nullptr, nullptr, 0, nullptr},
};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_mixer", "Binding of the mixer operators.", -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

// The torch and Python that this was built for, between zeros: found by the
// build without loading it.
const char g_built_for[] = "\0" KLA_BUILT_FOR;

}  // namespace

PyMODINIT_FUNC PyInit__mixer() {
    PyObject *m = PyModule_Create(&module);
    if (m && PyModule_AddStringConstant(m, "built_for", g_built_for + 1) < 0) {
        Py_DECREF(m);
        return nullptr;
    }
    return m;
}
