// binding.cpp -- the Python side of the decoding entry points of include/gdn.h and of those of linear attention, as an
// extension module.
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

#include <algorithm>
#include <cmath>
#include <initializer_list>
#include <limits>
#include <sstream>
#include <string>
#include <type_traits>
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
                        "chunk_gated_delta_rule or chunk_linear_attention");
        if (forward && t->_fw_grad(0).defined()) value_error("the decoding operators take no forward-mode tangents");
    }
}
// The calls below the autograd function of linear attention: a derivative is not dropped either
void below_autograd(std::initializer_list<const Tensor *> tensors) {
    const bool backward = at::GradMode::is_enabled(), forward = c10::AutogradState::get_tls_state().get_fw_grad_mode();
    for (const Tensor *t : tensors) {
        if (!t->defined()) continue;
        if (backward && t->requires_grad()) value_error("chunk_linear_attention_fwd and _bwd have no derivative: call chunk_linear_attention");
        if (forward && t->_fw_grad(0).defined()) value_error("linear attention takes no forward-mode tangents");
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

    // a: q, k, v, g, beta, state, scale; without the delta rule beta is None and g, which may be, has one value per head
    Decode(PyObject *const *a, bool delta = true) {
        q = optional(a[0], "q"), k = tensor(a[1], "k"), v = tensor(a[2], "v");
        g = delta ? tensor(a[3], "g") : optional(a[3], "g"), beta = delta ? tensor(a[4], "beta") : Tensor();
        state = tensor(a[5], "state");
        on_cuda(k, "k");
        dev = k.device();
        if (k.dim() != 4 || v.dim() != 4) value_error("k and v must have four dimensions: [B, T, heads, width]");
        p.B = k.size(0), p.T = k.size(1), p.Hq = k.size(2), p.K = k.size(3), p.Hv = v.size(2), p.V = v.size(3);
        p.io_dtype = io_dtype(k, "io");
        if (q.defined()) shaped(q, "q", k.sizes(), dev);
        shaped(v, "v", {p.B, p.T, p.Hv, p.V}, dev);
        if (delta) {
            shaped(g, "g", {p.B, p.T, p.Hv}, dev);
            shaped(beta, "beta", {p.B, p.T, p.Hv}, dev);
        } else if (g.defined()) {
            shaped(g, "g", {p.Hv}, dev);
            if (c10::isComplexType(g.scalar_type())) type_error("g must hold real numbers");
        }
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
        if (g.defined() && g.scalar_type() != at::kFloat) g = g.to(at::kFloat);
        p.k = strides_of(k), p.v = strides_of(v);
        if (delta) {
            if (beta.scalar_type() != at::kFloat) beta = beta.to(at::kFloat);
            p.g = strides_of(g), p.beta = strides_of(beta);
        } else if (g.defined()) {
            g = g.contiguous();
        }
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
PyObject *step(PyObject *const *a, Py_ssize_t n, bool delta) {
    if (!arguments(n, 11)) return nullptr;
    return guarded([&]() -> PyObject * {
        Decode d(a, delta);
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
        if (delta)
            check(gdn_recurrent(&p, ptr(d.q), ptr(d.k), ptr(d.v), ptr<float>(d.g), ptr<float>(d.beta), ptr<float>(d.state),
                                ptr<float>(out_state), ptr(o), stream_of(d.dev)),
                  "gdn_recurrent");
        else
            check(gdn_linear_recurrent(&p, ptr(d.q), ptr(d.k), ptr(d.v), ptr<float>(d.g), ptr<float>(d.state),
                                       ptr<float>(out_state), ptr(o), stream_of(d.dev)),
                  "gdn_linear_recurrent");
        written(out_state.defined() ? out_state : d.state);
        if (!o.defined()) Py_RETURN_NONE;
        return THPVariable_Wrap(o);
    });
}

PyObject *recurrent(PyObject *, PyObject *const *a, Py_ssize_t n) { return step(a, n, true); }
PyObject *linear_recurrent(PyObject *, PyObject *const *a, Py_ssize_t n) { return step(a, n, false); }

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

// What the forward and the backward of linear attention share: checks, layouts, the problem
struct Linear {
    Tensor q, k, v, g, h0, cu;
    gdn_linear_problem p{};
    at::Device dev = at::kCPU;

    // a: q, k, v, g, scale, initial_state, cu_seqlens
    Linear(PyObject *const *a) {
        q = tensor(a[0], "q"), k = tensor(a[1], "k"), v = tensor(a[2], "v"), g = optional(a[3], "g");
        h0 = optional(a[5], "initial_state"), cu = optional(a[6], "cu_seqlens");
        below_autograd({&q, &k, &v, &g, &h0});
        on_cuda(q, "q");
        dev = q.device();
        if (q.dim() != 4 || v.dim() != 4) value_error("q and v must have four dimensions: [B, T, heads, width]");
        p.B = q.size(0), p.T = q.size(1), p.Hq = q.size(2), p.K = q.size(3), p.Hv = v.size(2), p.V = v.size(3);
        p.io_dtype = io_dtype(q, "io");
        shaped(k, "k", q.sizes(), dev);
        shaped(v, "v", {p.B, p.T, p.Hv, p.V}, dev);
        if (k.scalar_type() != q.scalar_type() || v.scalar_type() != q.scalar_type()) type_error("q, k and v must have one dtype");
        q = mappable(q), k = mappable(k), v = mappable(v);
        p.q = strides_of(q), p.k = strides_of(k), p.v = strides_of(v);
        if (g.defined()) {
            shaped(g, "g", {p.Hv}, dev);
            if (c10::isComplexType(g.scalar_type())) type_error("g must hold real numbers");
            if (g.scalar_type() != at::kFloat) g = g.to(at::kFloat);
            g = g.contiguous();
        }
        p.scale = a[4] == Py_None ? (float)std::pow((double)p.K, -0.5) : (float)PyFloat_AsDouble(a[4]);
        if (PyErr_Occurred()) throw std::runtime_error("scale");
        p.n_seqs = p.B;
        if (cu.defined()) {
            if (p.B != 1) value_error("cu_seqlens needs B = 1");
            if (cu.dim() != 1 || cu.size(0) < 1) value_error("cu_seqlens must have one dimension and at least one entry");
            cu = ints(cu, "cu_seqlens", cu.sizes(), dev);
            p.n_seqs = cu.size(0) - 1;
            p.cu_seqlens = ptr<int32_t>(cu);
        }
        h0 = state(h0, "initial_state");
    }
    // As it is where the tensor cores' kernel can take it (rows on 16-byte boundaries, none shared), else a copy
    static Tensor mappable(const Tensor &t) {
        bool ok = t.stride(3) == 1;
        if (t.scalar_type() == at::kBFloat16) {
            ok = ok && (reinterpret_cast<uintptr_t>(t.data_ptr()) & 15) == 0;
            for (int d = 0; d < 3; ++d) ok = ok && (t.size(d) <= 1 || (t.stride(d) > 0 && t.stride(d) % 8 == 0));
        }
        return ok ? t : t.clone(at::MemoryFormat::Contiguous);
    }
    Tensor state(const Tensor &t, const char *name) const {
        if (!t.defined()) return t;
        shaped(t, name, {p.n_seqs, p.Hv, p.K, p.V}, dev);
        if (t.scalar_type() != at::kFloat) type_error(std::string(name) + " must be float32, got " + toString(t.scalar_type()));
        const Tensor c = t.contiguous();
        return (reinterpret_cast<uintptr_t>(c.data_ptr()) & 15) == 0 ? c : c.clone();
    }
    Tensor new_state() const { return at::detail::empty_cuda({p.n_seqs, p.Hv, p.K, p.V}, at::kFloat, dev, std::nullopt); }
    Tensor workspace(size_t bytes, const char *where) const {
        if (bytes == 0) throw Failed{GDN_ERR_UNSUPPORTED, where};
        return at::detail::empty_cuda({(int64_t)bytes}, at::kByte, dev, std::nullopt);
    }
};

// (q, k, v, g, scale, initial_state, cu_seqlens, output_final_state) -> (o, final_state or None)
PyObject *linear_fwd(PyObject *, PyObject *const *a, Py_ssize_t n) {
    if (!arguments(n, 8)) return nullptr;
    return guarded([&]() -> PyObject * {
        Linear x(a);
        const int wanted = PyObject_IsTrue(a[7]);
        if (wanted < 0) throw std::runtime_error("output_final_state");
        const c10::cuda::CUDAGuard guard(x.dev);
        const Tensor ws = x.workspace(gdn_linear_fwd_workspace_bytes(&x.p), "gdn_linear_fwd");
        const Tensor o = at::detail::empty_cuda({x.p.B, x.p.T, x.p.Hv, x.p.V}, x.q.scalar_type(), x.dev, std::nullopt);
        const Tensor end = wanted ? x.new_state() : Tensor();
        check(gdn_linear_fwd(&x.p, ptr(x.q), ptr(x.k), ptr(x.v), ptr<float>(x.g), ptr<float>(x.h0), ptr(o), ptr<float>(end),
                             ptr(ws), ws.nbytes(), stream_of(x.dev)),
              "gdn_linear_fwd");
        PyObject *first = THPVariable_Wrap(o), *second = Py_None;
        if (wanted) second = THPVariable_Wrap(end);
        else Py_INCREF(Py_None);
        return Py_BuildValue("(NN)", first, second);
    });
}

// (q, k, v, g, scale, initial_state, cu_seqlens, do, dht, wanted) -> (dq, dk, dv, dh0), None for each whose bit of `wanted` is 0
PyObject *linear_bwd(PyObject *, PyObject *const *a, Py_ssize_t n) {
    if (!arguments(n, 10)) return nullptr;
    return guarded([&]() -> PyObject * {
        Linear x(a);
        Tensor d_o = tensor(a[7], "do");
        shaped(d_o, "do", {x.p.B, x.p.T, x.p.Hv, x.p.V}, x.dev);
        if (d_o.scalar_type() != x.q.scalar_type()) type_error("do must have the dtype of q, k and v");
        d_o = Linear::mappable(d_o);
        x.p.d_o = strides_of(d_o);
        const Tensor dht = x.state(optional(a[8], "dht"), "dht");
        below_autograd({&d_o, &dht});
        const long wanted = PyLong_AsLong(a[9]);
        if (PyErr_Occurred()) throw std::runtime_error("wanted");
        const c10::cuda::CUDAGuard guard(x.dev);
        const Tensor ws = x.workspace(gdn_linear_bwd_workspace_bytes(&x.p), "gdn_linear_bwd");
        Tensor out[4];
        for (int i = 0; i < 3; ++i)
            if (wanted >> i & 1)
                out[i] = at::detail::empty_cuda(i < 2 ? x.q.sizes() : x.v.sizes(), x.q.scalar_type(), x.dev, std::nullopt);
        if (wanted >> 3 & 1) out[3] = x.new_state();
        check(gdn_linear_bwd(&x.p, ptr(x.q), ptr(x.k), ptr(x.v), ptr<float>(x.g), ptr<float>(x.h0), ptr(d_o), ptr<float>(dht),
                             ptr(out[0]), ptr(out[1]), ptr(out[2]), ptr<float>(out[3]), ptr(ws), ws.nbytes(), stream_of(x.dev)),
              "gdn_linear_bwd");
        PyObject *r[4];
        for (int i = 0; i < 4; ++i) {
            r[i] = out[i].defined() ? THPVariable_Wrap(out[i]) : Py_None;
            if (!out[i].defined()) Py_INCREF(Py_None);
        }
        return Py_BuildValue("(NNNN)", r[0], r[1], r[2], r[3]);
    });
}

// A parameter of every row: a number, or a tensor of one for each row
template <typename T> Tensor per_row(PyObject *o, const char *name, T none, T *one, int64_t B, at::Device dev) {
    *one = none;
    if (o == Py_None) return Tensor();
    if (!THPVariable_Check(o)) {
        if constexpr (std::is_same_v<T, float>) {
            *one = (float)PyFloat_AsDouble(o);
        } else {
            const long long k = PyLong_AsLongLong(o);
            *one = (T)std::min<long long>(std::max<long long>(k, std::numeric_limits<T>::min()), std::numeric_limits<T>::max());
        }
        if (PyErr_Occurred()) throw std::runtime_error(name);
        return Tensor();
    }
    const Tensor t = THPVariable_Unpack(o);
    if constexpr (std::is_same_v<T, float>) {
        shaped(t, name, {B}, dev);
        if (!at::isFloatingType(t.scalar_type())) type_error(std::string(name) + " must hold floating-point numbers, got " + toString(t.scalar_type()));
        return t.to(at::kFloat).contiguous();
    } else {
        return ints(t, name, {B}, dev);
    }
}

// (logits, random, temperature, top_k, top_p, min_p, mask) -> (tokens, logprobs)
PyObject *sample(PyObject *, PyObject *const *a, Py_ssize_t n) {
    if (!arguments(n, 7)) return nullptr;
    return guarded([&]() -> PyObject * {
        Tensor logits = tensor(a[0], "logits"), u = tensor(a[1], "random"), mask = optional(a[6], "mask");
        on_cuda(logits, "logits");
        const at::Device dev = logits.device();
        if (logits.dim() != 2) value_error("logits must have two dimensions: [B, vocab]");
        gdn_sample_problem p{};
        p.B = logits.size(0), p.vocab = logits.size(1);
        p.logits_dtype = io_dtype(logits, "logits");
        if (p.vocab < 1 || p.vocab > GDN_SAMPLE_VOCAB_MAX)
            value_error("the vocabulary must have 1 to " + std::to_string(GDN_SAMPLE_VOCAB_MAX) + " tokens");
        shaped(u, "random", {p.B}, dev);
        if (u.scalar_type() != at::kFloat) type_error(std::string("random must be float32, got ") + toString(u.scalar_type()));
        no_derivative({&logits, &u});
        logits = inner_contiguous(logits), u = u.contiguous();
        p.logits_row = logits.stride(0);
        const Tensor heat = per_row<float>(a[2], "temperature", 1.f, &p.temperature, p.B, dev);
        const Tensor top_k = per_row<int32_t>(a[3], "top_k", 0, &p.top_k, p.B, dev);
        const Tensor top_p = per_row<float>(a[4], "top_p", 1.f, &p.top_p, p.B, dev);
        const Tensor min_p = per_row<float>(a[5], "min_p", 0.f, &p.min_p, p.B, dev);
        no_derivative({&heat, &top_p, &min_p});
        p.temperatures = ptr<float>(heat), p.top_ks = ptr<int32_t>(top_k), p.top_ps = ptr<float>(top_p), p.min_ps = ptr<float>(min_p);
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
            p.mask_row = mask.stride(0);
        }
        const c10::cuda::CUDAGuard guard(dev);
        const Tensor tokens = at::detail::empty_cuda({p.B}, at::kInt, dev, std::nullopt);
        const Tensor logprobs = at::detail::empty_cuda({p.B}, at::kFloat, dev, std::nullopt);
        check(gdn_sample(&p, ptr(logits), ptr<float>(u), ptr<uint8_t>(mask), ptr<int32_t>(tokens), ptr<float>(logprobs), stream_of(dev)),
              "gdn_sample");
        PyObject *t = THPVariable_Wrap(tokens), *l = THPVariable_Wrap(logprobs);
        return Py_BuildValue("(NN)", t, l);
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
    {"linear_recurrent", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(linear_recurrent)), METH_FASTCALL, nullptr},
    {"linear_fwd", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(linear_fwd)), METH_FASTCALL, nullptr},
    {"linear_bwd", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(linear_bwd)), METH_FASTCALL, nullptr},
    {"sample", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(sample)), METH_FASTCALL, nullptr},
    {"set_errors", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(set_errors)), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_gdn_decode", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__gdn_decode(void) { return PyModule_Create(&module); }
