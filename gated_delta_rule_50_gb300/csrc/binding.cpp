// binding.cpp -- the Python side of the decoding entry points of include/gdn.h, as an extension module.
//
// A decoding call works for a few microseconds on the GPU, and marshalling it through ctypes took three times as
// long: reading some forty properties of the tensors one Python attribute at a time.  Here they are read from the
// tensors themselves.  Everything else is as in the ctypes binding: checks, PyTorch memory and the current stream,
// one C call.
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/core/grad_mode.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/core/AutogradState.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cmath>
#include <initializer_list>
#include <limits>
#include <sstream>
#include <string>
#include <vector>

#include "gdn.h"

namespace {

using at::Tensor;

PyObject *g_error = nullptr, *g_no_memory = nullptr;  // the package's GdnError, torch.OutOfMemoryError

struct Raise {
    PyObject *type;
    std::string text;
};
[[noreturn]] void value_error(const std::string &text) { throw Raise{PyExc_ValueError, text}; }
[[noreturn]] void type_error(const std::string &text) { throw Raise{PyExc_TypeError, text}; }
struct Failed {  // a status of the library
    int status;
    const char *where;
};

template <typename F> PyObject *guarded(F f) {
    try {
        return f();
    } catch (const Raise &r) {
        PyErr_SetString(r.type, r.text.c_str());
    } catch (const Failed &s) {
        if (PyObject *e = PyObject_CallFunction(g_error, "is", s.status, s.where)) {
            PyErr_SetObject(g_error, e);
            Py_DECREF(e);
        }
    } catch (const c10::OutOfMemoryError &e) {
        PyErr_SetString(g_no_memory, e.what_without_backtrace());
    } catch (const c10::Error &e) {
        PyErr_SetString(PyExc_RuntimeError, e.what_without_backtrace());
    } catch (const std::exception &e) {
        if (!PyErr_Occurred()) PyErr_SetString(PyExc_RuntimeError, e.what());
    }
    return nullptr;
}

std::string text_of(at::IntArrayRef s) {
    std::ostringstream o;
    o << '(';
    for (size_t i = 0; i < s.size(); ++i) o << (i ? ", " : "") << s[i];
    o << (s.size() == 1 ? ",)" : ")");
    return o.str();
}

Tensor tensor(PyObject *o, const char *name) {
    if (!THPVariable_Check(o)) type_error(std::string(name) + " must be a tensor, got " + Py_TYPE(o)->tp_name);
    return THPVariable_Unpack(o);
}
Tensor optional(PyObject *o, const char *name) { return o == Py_None ? Tensor() : tensor(o, name); }
template <typename T = void> T *ptr(const Tensor &t) { return t.defined() ? static_cast<T *>(t.data_ptr()) : nullptr; }

void on_cuda(const Tensor &t, const char *name) {
    if (!t.is_cuda()) value_error(std::string(name) + " must be a CUDA tensor (no CPU path)");
}
void on_device(const Tensor &t, const char *name, at::Device dev) {
    if (t.device() != dev) value_error(std::string(name) + " must be on " + dev.str() + ", got " + t.device().str());
}
void shaped(const Tensor &t, const char *name, at::IntArrayRef shape, at::Device dev) {
    if (t.sizes() != shape) value_error(std::string(name) + " must have shape " + text_of(shape) + ", got " + text_of(t.sizes()));
    on_device(t, name, dev);
}
// Device indices as contiguous int32.  What needs more bits stays out of range, above or below: no slot, token or node
// has such a number (see reorder for pools of more than 2^31 slots).
Tensor ints(const Tensor &t, const char *name, at::IntArrayRef shape, at::Device dev) {
    if (!t.defined()) return t;
    shaped(t, name, shape, dev);
    if (t.scalar_type() == at::kInt) return t.contiguous();
    if (!at::isIntegralType(t.scalar_type(), false))
        type_error(std::string(name) + " must hold integers, got " + toString(t.scalar_type()));
    if (t.element_size() < 4) return t.to(at::kInt).contiguous();
    Tensor wide = t.to(at::kLong);
    constexpr int64_t least = std::numeric_limits<int32_t>::min(), most = std::numeric_limits<int32_t>::max();
    if (t.scalar_type() == at::kUInt64) wide = wide.masked_fill(wide.lt(0), most);  // past 2^63
    return wide.clamp(at::Scalar(least), at::Scalar(most)).to(at::kInt).contiguous();
}
bool slots_contiguous(const Tensor &t) {  // every t[i]
    int64_t expected = 1;
    for (int64_t d = t.dim() - 1; d > 0; --d) {
        if (t.size(d) != 1 && t.stride(d) != expected) return t.numel() == 0;
        expected *= t.size(d);
    }
    return true;
}
Tensor inner_contiguous(const Tensor &t) { return t.stride(t.dim() - 1) == 1 ? t : t.contiguous(); }
gdn_dtype io_dtype(const Tensor &t, const char *what) {
    if (t.scalar_type() == at::kBFloat16) return GDN_BF16;
    if (t.scalar_type() == at::kFloat) return GDN_F32;
    type_error(std::string("unsupported ") + what + " dtype " + toString(t.scalar_type()) + " (bfloat16 or float32)");
}
gdn_stream_t stream_of(at::Device dev) { return reinterpret_cast<gdn_stream_t>(c10::cuda::getCurrentCUDAStream(dev.index()).stream()); }
void check(gdn_status s, const char *where) {
    if (s != GDN_OK) throw Failed{(int)s, where};
}
gdn_strides strides_of(const Tensor &t) { return {t.stride(0), t.stride(1), t.stride(2)}; }

// Nothing here has a derivative, in either direction: what would drop one is refused
void no_derivative(std::initializer_list<const Tensor *> tensors) {
    const bool backward = at::GradMode::is_enabled(), forward = c10::AutogradState::get_tls_state().get_fw_grad_mode();
    for (const Tensor *t : tensors) {
        if (!t->defined()) continue;
        if (backward && t->requires_grad())
            value_error("the decoding operators have no backward: call them under torch.no_grad(), or train through "
                        "chunk_gated_delta_rule");
        if (forward && t->_fw_grad(0).defined()) value_error("the decoding operators take no forward-mode tangents");
    }
}
// A new version of a tensor that a kernel writes in place, as autograd counts them
void written(const Tensor &t) {
    if (!t.is_inference()) t.unsafeGetTensorImpl()->bump_version();
}

// What the two state operators share: checks, the layouts that the kernels read, the problem
struct Decode {
    Tensor q, k, v, g, beta, state;
    gdn_decode_problem p{};
    at::Device dev = at::kCPU;

    Decode(PyObject *const *a) {
        q = optional(a[0], "q"), k = tensor(a[1], "k"), v = tensor(a[2], "v"), g = tensor(a[3], "g"), beta = tensor(a[4], "beta");
        state = tensor(a[5], "state");
        on_cuda(k, "k");
        dev = k.device();
        if (k.dim() != 4 || v.dim() != 4) value_error("k and v must have four dimensions: [B, T, heads, width]");
        p.B = k.size(0), p.T = k.size(1), p.Hq = k.size(2), p.K = k.size(3), p.Hv = v.size(2), p.V = v.size(3);
        p.io_dtype = io_dtype(k, "io");
        if (q.defined()) shaped(q, "q", k.sizes(), dev);
        shaped(v, "v", {p.B, p.T, p.Hv, p.V}, dev);
        shaped(g, "g", {p.B, p.T, p.Hv}, dev);
        shaped(beta, "beta", {p.B, p.T, p.Hv}, dev);
        if (v.scalar_type() != k.scalar_type() || (q.defined() && q.scalar_type() != k.scalar_type()))
            type_error("q, k and v must have one dtype");
        no_derivative({&q, &k, &v, &g, &beta, &state});
        if (state.dim() != 4 || state.size(1) != p.Hv || state.size(2) != p.K || state.size(3) != p.V)
            value_error("state must have shape (slots, " + std::to_string(p.Hv) + ", " + std::to_string(p.K) + ", " +
                        std::to_string(p.V) + "), got " + text_of(state.sizes()));
        if (state.scalar_type() != at::kFloat) type_error(std::string("state must be float32, got ") + toString(state.scalar_type()));
        on_device(state, "state", dev);
        if (!slots_contiguous(state)) value_error("every slot of state must be contiguous");
        k = inner_contiguous(k), v = inner_contiguous(v);
        if (q.defined()) q = inner_contiguous(q), p.q = strides_of(q);
        if (g.scalar_type() != at::kFloat) g = g.to(at::kFloat);
        if (beta.scalar_type() != at::kFloat) beta = beta.to(at::kFloat);
        p.k = strides_of(k), p.v = strides_of(v), p.g = strides_of(g), p.beta = strides_of(beta);
        p.scale = a[6] == Py_None ? (float)std::pow((double)p.K, -0.5) : (float)PyFloat_AsDouble(a[6]);
        if (PyErr_Occurred()) throw std::runtime_error("scale");
        p.n_slots = state.size(0), p.slot_stride = state.stride(0);
        p.n_seqs = p.B;
    }
    Tensor out(int64_t rows, int64_t steps) const {
        return at::detail::empty_cuda({rows, steps, p.Hv, p.V}, k.scalar_type(), dev, std::nullopt);
    }
};

bool arguments(Py_ssize_t got, Py_ssize_t wanted) {
    if (got == wanted) return true;
    PyErr_Format(PyExc_TypeError, "expected %zd arguments, got %zd", wanted, got);
    return false;
}

// (q, k, v, g, beta, state, scale, state_indices, cu_seqlens, token_indices, out_state) -> o or None
PyObject *recurrent(PyObject *, PyObject *const *a, Py_ssize_t n) {
    if (!arguments(n, 11)) return nullptr;
    return guarded([&]() -> PyObject * {
        Decode d(a);
        gdn_decode_problem &p = d.p;
        Tensor cu = optional(a[8], "cu_seqlens"), list = optional(a[9], "token_indices"), out_state = optional(a[10], "out_state");
        int64_t steps = p.T;
        if (cu.defined()) {
            if (p.B != 1) value_error("cu_seqlens needs B = 1");
            if (list.defined()) value_error("token_indices and cu_seqlens exclude each other");
            if (cu.dim() != 1 || cu.size(0) < 1) value_error("cu_seqlens must have one dimension and at least one entry");
            cu = ints(cu, "cu_seqlens", cu.sizes(), d.dev);
            p.n_seqs = cu.size(0) - 1;
            p.cu_seqlens = ptr<int32_t>(cu);
        }
        if (list.defined()) {
            if (list.dim() != 2) value_error("token_indices must have two dimensions");
            steps = p.n_steps = list.size(1);
            list = ints(list, "token_indices", {p.B, steps}, d.dev);
            p.token_indices = ptr<int32_t>(list);
        }
        const Tensor slots = ints(optional(a[7], "state_indices"), "state_indices", {p.n_seqs}, d.dev);
        p.state_indices = ptr<int32_t>(slots);
        if (out_state.defined()) {
            shaped(out_state, "out_state", {p.n_seqs, p.Hv, p.K, p.V}, d.dev);
            if (out_state.scalar_type() != at::kFloat || !out_state.is_contiguous())
                value_error("out_state must be contiguous float32");
            no_derivative({&out_state});
        }
        const c10::cuda::CUDAGuard guard(d.dev);
        Tensor o;
        if (d.q.defined()) o = d.out(p.B, steps);
        if (cu.defined() && o.defined()) o.zero_();  // the kernel writes the sequences' rows alone
        check(gdn_recurrent(&p, ptr(d.q), ptr(d.k), ptr(d.v), ptr<float>(d.g), ptr<float>(d.beta), ptr<float>(d.state),
                            ptr<float>(out_state), ptr(o), stream_of(d.dev)),
              "gdn_recurrent");
        written(out_state.defined() ? out_state : d.state);
        if (!o.defined()) Py_RETURN_NONE;
        return THPVariable_Wrap(o);
    });
}

// (q, k, v, g, beta, state, scale, state_indices, parents) -> o
PyObject *tree(PyObject *, PyObject *const *a, Py_ssize_t n) {
    if (!arguments(n, 9)) return nullptr;
    return guarded([&]() -> PyObject * {
        if (a[0] == Py_None) value_error("q must be given");
        Decode d(a);
        gdn_decode_problem &p = d.p;
        const Tensor slots = ints(optional(a[7], "state_indices"), "state_indices", {p.B}, d.dev);
        const Tensor parents = ints(tensor(a[8], "parents"), "parents", {p.B, p.T}, d.dev);
        p.state_indices = ptr<int32_t>(slots);
        const c10::cuda::CUDAGuard guard(d.dev);
        const Tensor o = d.out(p.B, p.T);
        check(gdn_tree(&p, ptr(d.q), ptr(d.k), ptr(d.v), ptr<float>(d.g), ptr<float>(d.beta), ptr<int32_t>(parents),
                       ptr<float>(d.state), ptr(o), stream_of(d.dev)),
              "gdn_tree");
        return THPVariable_Wrap(o);
    });
}

// (logits, scores, finished, mask, num_candidates, workspace) -> (scores, tokens, parents)
PyObject *beam(PyObject *, PyObject *const *a, Py_ssize_t n_args) {
    if (!arguments(n_args, 6)) return nullptr;
    return guarded([&]() -> PyObject * {
        Tensor logits = tensor(a[0], "logits"), scores = tensor(a[1], "scores"), finished = optional(a[2], "finished"),
               mask = optional(a[3], "mask"), workspace = optional(a[5], "workspace");
        on_cuda(logits, "logits");
        const at::Device dev = logits.device();
        if (logits.dim() != 3) value_error("logits must have three dimensions: [B, W, vocab]");
        gdn_beam_problem p{};
        p.B = logits.size(0), p.W = logits.size(1), p.vocab = logits.size(2);
        p.logits_dtype = io_dtype(logits, "logits");
        p.n = a[4] == Py_None ? p.W : PyLong_AsLongLong(a[4]);
        if (PyErr_Occurred()) throw std::runtime_error("num_candidates");
        if (p.n < 1 || p.n > GDN_BEAM_MAX || p.W < 1 || p.W > GDN_BEAM_MAX)
            value_error("beams and candidates must be 1 to " + std::to_string(GDN_BEAM_MAX));
        shaped(scores, "scores", {p.B, p.W}, dev);
        no_derivative({&logits, &scores});
        if (scores.scalar_type() != at::kFloat) type_error(std::string("scores must be float32, got ") + toString(scores.scalar_type()));
        logits = inner_contiguous(logits);
        p.logits_batch = logits.stride(0), p.logits_beam = logits.stride(1);
        scores = scores.contiguous();
        if (finished.defined()) {
            shaped(finished, "finished", {p.B, p.W}, dev);
            if (finished.scalar_type() != at::kBool) type_error(std::string("finished must be bool, got ") + toString(finished.scalar_type()));
            finished = finished.contiguous();
        }
        if (mask.defined()) {
            if (mask.scalar_type() != at::kBool) type_error(std::string("mask must be bool, got ") + toString(mask.scalar_type()));
            on_device(mask, "mask", dev);
            if (mask.sizes() != logits.sizes()) {
                try {
                    mask = mask.expand(logits.sizes());
                } catch (const c10::Error &) {
                    value_error("mask must be broadcastable to " + text_of(logits.sizes()) + ", got " + text_of(mask.sizes()));
                }
            }
            mask = inner_contiguous(mask);
            p.mask_batch = mask.stride(0), p.mask_beam = mask.stride(1);
        }
        const size_t need = gdn_beam_search_workspace_bytes(&p);
        if (need == 0) throw Failed{GDN_ERR_UNSUPPORTED, "gdn_beam_search"};
        const c10::cuda::CUDAGuard guard(dev);
        if (workspace.defined()) on_device(workspace, "workspace", dev);
        if (!workspace.defined() || !workspace.is_contiguous() || workspace.nbytes() < need)
            workspace = at::detail::empty_cuda({(int64_t)need}, at::kByte, dev, std::nullopt);
        const Tensor out = at::detail::empty_cuda({p.B, p.n}, at::kFloat, dev, std::nullopt);
        const Tensor tokens = at::detail::empty_cuda({p.B, p.n}, at::kInt, dev, std::nullopt);
        const Tensor parents = at::detail::empty_cuda({p.B, p.n}, at::kInt, dev, std::nullopt);
        check(gdn_beam_search(&p, ptr(logits), ptr<float>(scores), ptr<uint8_t>(finished), ptr<uint8_t>(mask), ptr<float>(out),
                              ptr<int32_t>(tokens), ptr<int32_t>(parents), ptr(workspace), workspace.nbytes(), stream_of(dev)),
              "gdn_beam_search");
        PyObject *s = THPVariable_Wrap(out), *t = THPVariable_Wrap(tokens), *r = THPVariable_Wrap(parents);
        return Py_BuildValue("(NNN)", s, t, r);
    });
}

// (states, parents, state_indices) -> None
PyObject *reorder(PyObject *, PyObject *const *a, Py_ssize_t n_args) {
    if (!arguments(n_args, 3)) return nullptr;
    return guarded([&]() -> PyObject * {
        std::vector<Tensor> states;
        if (THPVariable_Check(a[0])) {
            states.push_back(THPVariable_Unpack(a[0]));
        } else {
            PyObject *list = PySequence_Fast(a[0], "states must be a tensor or a sequence of tensors");
            if (!list) throw std::runtime_error("states");
            try {
                for (Py_ssize_t i = 0; i < PySequence_Fast_GET_SIZE(list); ++i)
                    states.push_back(tensor(PySequence_Fast_GET_ITEM(list, i), "states"));
            } catch (...) {
                Py_DECREF(list);
                throw;
            }
            Py_DECREF(list);
        }
        if (states.empty()) Py_RETURN_NONE;
        on_cuda(states[0], "states");
        const at::Device dev = states[0].device();
        Tensor parents = tensor(a[1], "parents");
        if (parents.dim() != 2) value_error("parents must have two dimensions: [B, W]");
        const int64_t B = parents.size(0), W = parents.size(1);
        if (W < 1 || W > GDN_BEAM_MAX) value_error("beams must be 1 to " + std::to_string(GDN_BEAM_MAX));
        parents = ints(parents, "parents", {B, W}, dev);
        const Tensor given = optional(a[2], "state_indices"), indices = ints(given, "state_indices", {B, W}, dev);
        std::vector<gdn_state_view> views;
        views.reserve(states.size());
        int64_t slots = 0;
        for (const Tensor &s : states) {
            if (s.dim() < 1) value_error("all states must have the same number of slots");
            if (views.empty()) slots = s.size(0);
            if (s.size(0) != slots) value_error("all states must have the same number of slots");
            on_device(s, "states", dev);
            no_derivative({&s});
            if (!slots_contiguous(s)) value_error("every slot of a state must be contiguous");
            const int64_t size = (int64_t)s.element_size();
            views.push_back({s.data_ptr(), s.stride(0) * size, slots ? s.numel() / slots * size : 0});
        }
        if (slots > std::numeric_limits<int32_t>::max() && given.defined() && given.scalar_type() != at::kInt)
            value_error("a pool of more than 2^31 - 1 slots takes int32 state_indices");
        const c10::cuda::CUDAGuard guard(dev);
        check(gdn_reorder_states(views.data(), (int64_t)views.size(), slots, B, W, ptr<int32_t>(parents), ptr<int32_t>(indices),
                                 stream_of(dev)),
              "gdn_reorder_states");
        for (const Tensor &s : states) written(s);
        Py_RETURN_NONE;
    });
}

// (GdnError, torch.OutOfMemoryError)
PyObject *set_errors(PyObject *, PyObject *const *a, Py_ssize_t n_args) {
    if (!arguments(n_args, 2)) return nullptr;
    Py_INCREF(a[0]), Py_INCREF(a[1]);
    Py_XDECREF(g_error), Py_XDECREF(g_no_memory);
    g_error = a[0], g_no_memory = a[1];
    Py_RETURN_NONE;
}

PyMethodDef methods[] = {
    {"recurrent", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(recurrent)), METH_FASTCALL, nullptr},
    {"tree", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(tree)), METH_FASTCALL, nullptr},
    {"beam", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(beam)), METH_FASTCALL, nullptr},
    {"reorder", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(reorder)), METH_FASTCALL, nullptr},
    {"set_errors", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(set_errors)), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_gdn_decode", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__gdn_decode(void) { return PyModule_Create(&module); }
