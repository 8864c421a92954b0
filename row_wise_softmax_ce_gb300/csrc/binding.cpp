// binding.cpp -- the objectives' and the choices' calls for PyTorch tensors: the checks, the
// outputs and the current stream, then the C ABI of libcerows.so. Marshalling
// only, as the ctypes functions beside it are; it exists because these calls are
// also made on batches whose kernels take a few microseconds, where checking
// and allocating from Python took several times that (policy_step on 64 x 1000:
// 26 us a call through ctypes).
//
// Each function takes its arguments by position (the Python functions of the
// package give them names and defaults) and returns its tensors, or the status
// of a refused call as an int. A bad argument raises TypeError or ValueError.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <algorithm>
#include <initializer_list>
#include <string>

#include "ce_rows.h"

namespace {

struct Refused {
    PyObject *type;
    std::string text;
};
struct Raised {};  // a Python error is set already

PyObject *out_of_memory = nullptr;  // torch.OutOfMemoryError

[[noreturn]] void type_error(const std::string &text) { throw Refused{PyExc_TypeError, text}; }
[[noreturn]] void value_error(const std::string &text) { throw Refused{PyExc_ValueError, text}; }

const at::Tensor &tensor(PyObject *o, const char *name) {
    if (!THPVariable_Check(o)) type_error(std::string(name) + " must be a torch.Tensor");
    return THPVariable_Unpack(o);
}

double number(PyObject *o) {
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred()) throw Raised{};
    return v;
}

std::string where(const at::Device &d) { return d.str(); }

// Logits of f32, bf16 or f16, [rows, cols] with contiguous rows.
struct Logits {
    const at::Tensor &t;
    int dtype;
    int64_t rows, vocab, stride;
};

Logits logits_of(PyObject *o, PyObject *vocab_o) {
    if (!THPVariable_Check(o)) type_error("logits must be a float32, bfloat16 or float16 torch.Tensor");
    const at::Tensor &t = THPVariable_Unpack(o);
    int dtype;
    switch (t.scalar_type()) {
    case at::kFloat: dtype = CE_F32; break;
    case at::kBFloat16: dtype = CE_BF16; break;
    case at::kHalf: dtype = CE_F16; break;
    default: type_error("logits must be a float32, bfloat16 or float16 torch.Tensor");
    }
    if (!t.is_cuda()) value_error("logits must be on a CUDA device");
    if (t.dim() != 2) value_error("logits must be 2-D [rows, cols]");
    const int64_t rows = t.size(0), cols = t.size(1);
    if (rows > 0 && cols > 1 && t.stride(1) != 1) value_error("each row of logits must be contiguous (stride(1) == 1)");
    int64_t vocab = cols;
    if (vocab_o != Py_None) {
        vocab = PyLong_AsLongLong(vocab_o);
        if (vocab == -1 && PyErr_Occurred()) throw Raised{};
    }
    if (vocab < 1 || vocab > cols)
        value_error("need 1 <= vocab <= logits.shape[1] (vocab=" + std::to_string(vocab) + ", cols=" + std::to_string(cols) + ")");
    int64_t stride = cols;
    if (rows > 1) {
        stride = t.stride(0);
        if (stride < vocab) value_error("rows of logits overlap (stride(0) < vocab)");
    }
    return Logits{t, dtype, rows, vocab, stride};
}

const int64_t *labels_of(PyObject *o, const Logits &x) {
    const at::Tensor &t = tensor(o, "labels");
    if (t.scalar_type() != at::kLong || t.dim() != 1 || t.size(0) != x.rows)
        value_error("labels must be int64 [rows=" + std::to_string(x.rows) + "]");
    if (t.device() != x.t.device() || !t.is_contiguous()) value_error("labels must be contiguous and on the logits' device");
    return t.const_data_ptr<int64_t>();
}

// A contiguous f32 [n] tensor's values; null for None.
float *f32_of(PyObject *o, int64_t n, const Logits &x, const char *name) {
    if (o == Py_None) return nullptr;
    const at::Tensor &t = tensor(o, name);
    if (t.scalar_type() != at::kFloat || t.dim() != 1 || t.size(0) != n || t.device() != x.t.device() || !t.is_contiguous())
        value_error(std::string(name) + " must be a contiguous float32 tensor [" + std::to_string(n) + "] on " +
                    where(x.t.device()));
    return static_cast<float *>(t.data_ptr());
}

// The gradient: the caller's [rows, >= vocab] tensor of the logits' type with
// contiguous rows, checked (None: allocated dense later).
void check_grad(PyObject *o, const Logits &x, at::Tensor *grad, int64_t *stride) {
    *stride = x.vocab;
    if (o == Py_None) return;
    const at::Tensor &t = tensor(o, "grad");
    if (t.scalar_type() != x.t.scalar_type() || t.device() != x.t.device() || t.dim() != 2 || t.size(0) != x.rows ||
        t.size(1) < x.vocab || (x.rows > 0 && t.size(1) > 1 && t.stride(1) != 1))
        value_error("grad must be a tensor of the logits' type, [rows=" + std::to_string(x.rows) + ", >= " +
                    std::to_string(x.vocab) + "] with contiguous rows, on " + where(x.t.device()));
    if (x.rows > 1) {
        *stride = t.stride(0);
        if (*stride < x.vocab) value_error("rows of grad overlap (stride(0) < vocab)");
    }
    *grad = t;
}

// An optional output: not wanted (False), allocated (True) or the caller's tensor.
struct Wanted {
    bool any;
    at::Tensor t;
};
Wanted wanted(PyObject *o, const Logits &x, const char *name) {
    if (o == Py_False || o == Py_None) return {false, {}};
    if (o == Py_True) return {true, {}};
    f32_of(o, x.rows, x, name);
    return {true, THPVariable_Unpack(o)};
}

// Other threads' Python runs while memory is allocated and kernels are launched.
struct WithoutGil {
    PyThreadState *state = PyEval_SaveThread();
    ~WithoutGil() { PyEval_RestoreThread(state); }
};

// Uninitialised device memory from PyTorch's allocator, without the dispatcher
// (four to six outputs a call: policy step 64 x 1000 11.5 -> 10.5 us on the
// host). empty_cuda is not part of PyTorch's public interface; it is there, with
// these arguments, in 2.9 and 2.11, and a version without it fails to compile.
at::Tensor empty(const Logits &x, at::IntArrayRef sizes, at::ScalarType type) {
    return at::detail::empty_cuda(sizes, type, x.t.device(), std::nullopt);
}
at::Tensor f32(const Logits &x, at::IntArrayRef sizes) { return empty(x, sizes, at::kFloat); }
float *data(const at::Tensor &t) { return t.defined() ? static_cast<float *>(t.data_ptr()) : nullptr; }
ce_stream_t stream_of(const Logits &x) {
    return reinterpret_cast<ce_stream_t>(c10::cuda::getCurrentCUDAStream(x.t.device().index()).stream());
}

// Tells autograd that a call wrote to a tensor of the caller's, as an in-place
// operation of PyTorch does: a backward pass that saved it raises an error
// instead of reading what is there now. Inference tensors keep no version.
// `given` is a tensor that was checked, or None, True or False (a tensor check of
// those goes through Python's isinstance).
void written(int status, PyObject *given) {
    if (status != CE_OK || given == Py_None || given == Py_True || given == Py_False) return;
    const at::Tensor &t = THPVariable_Unpack(given);
    if (!t.is_inference()) t.unsafeGetTensorImpl()->bump_version();
}

// The tensors as a tuple (None for one that was not wanted), or the status.
PyObject *result(int status, std::initializer_list<at::Tensor> tensors) {
    if (status != CE_OK) return PyLong_FromLong(status);
    PyObject *tuple = PyTuple_New(static_cast<Py_ssize_t>(tensors.size()));
    if (!tuple) throw Raised{};
    Py_ssize_t i = 0;
    for (const at::Tensor &t : tensors) {
        PyObject *o = t.defined() ? THPVariable_Wrap(t) : Py_NewRef(Py_None);
        if (!o) {
            Py_DECREF(tuple);
            throw Raised{};
        }
        PyTuple_SET_ITEM(tuple, i++, o);
    }
    return tuple;
}

// logp_rows(logits, labels, weights, temperature, vocab, entropy, out)
PyObject *logp(PyObject *const *a) {
    const Logits x = logits_of(a[0], a[4]);
    const int64_t *labels = labels_of(a[1], x);
    const float *w = f32_of(a[2], x.rows, x, "weights");
    const double temperature = number(a[3]);
    Wanted ent = wanted(a[5], x, "entropy");
    at::Tensor out;
    if (f32_of(a[6], x.rows, x, "out") || a[6] != Py_None) out = THPVariable_Unpack(a[6]);
    int st;
    {
        WithoutGil nogil;
        c10::cuda::CUDAGuard guard(x.t.device());
        if (!out.defined()) out = f32(x, {x.rows});
        if (ent.any && !ent.t.defined()) ent.t = f32(x, {x.rows});
        st = logp_rows(x.t.data_ptr(), x.dtype, x.rows, x.vocab, x.stride, labels, w, temperature, data(out),
                       data(ent.t), stream_of(x));
    }
    written(st, a[5]);
    written(st, a[6]);
    return result(st, {out, ent.t});
}

// policy(step, logits, labels, old_logp, advantages, scale, ref_logp, weights, clip_low,
//        clip_high, kl_coef, entropy_coef, temperature, vocab, entropy, grad)
PyObject *policy(PyObject *const *a) {
    const bool step = a[0] == Py_True;
    const Logits x = logits_of(a[1], a[13]);
    const int64_t *labels = labels_of(a[2], x);
    if (a[3] == Py_None || a[4] == Py_None) value_error("old_logp and advantages are needed");
    const float *old = f32_of(a[3], x.rows, x, "old_logp"), *adv = f32_of(a[4], x.rows, x, "advantages");
    const float *ref = f32_of(a[6], x.rows, x, "ref_logp"), *w = f32_of(a[7], x.rows, x, "weights");
    const ce_policy par = {number(a[5]), number(a[12]), number(a[8]), number(a[9]), number(a[10]), number(a[11])};
    if (par.kl_coef != 0.0 && a[6] == Py_None) value_error("kl_coef needs ref_logp");
    Wanted ent = wanted(a[14], x, "entropy");
    at::Tensor grad, loss, rows, lp;
    int64_t grad_stride = 0;
    if (step) check_grad(a[15], x, &grad, &grad_stride);
    int st;
    {
        WithoutGil nogil;
        c10::cuda::CUDAGuard guard(x.t.device());
        if (ent.any && !ent.t.defined()) ent.t = f32(x, {x.rows});
        rows = f32(x, {x.rows});
        lp = f32(x, {x.rows});
        loss = f32(x, {});
        if (step) {
            if (!grad.defined()) grad = empty(x, {x.rows, x.vocab}, x.t.scalar_type());
            st = policy_step(x.t.data_ptr(), x.dtype, x.rows, x.vocab, x.stride, labels, old, adv, ref, w, &par,
                             grad.data_ptr(), grad_stride, data(rows), data(lp), data(ent.t), data(loss), stream_of(x));
        } else {
            st = policy_loss(x.t.data_ptr(), x.dtype, x.rows, x.vocab, x.stride, labels, old, adv, ref, w, &par,
                             data(rows), data(lp), data(ent.t), data(loss), stream_of(x));
        }
    }
    written(st, a[14]);
    written(st, a[15]);
    return step ? result(st, {grad, loss, rows, lp, ent.t}) : result(st, {loss, rows, lp, ent.t});
}

// preference(step, logits, labels, offsets, scale, ref_logp, weights, kind, beta, label_smoothing,
//            margin, average, temperature, vocab, grad)
PyObject *preference(PyObject *const *a) {
    const bool step = a[0] == Py_True;
    const Logits x = logits_of(a[1], a[13]);
    const int64_t *labels = labels_of(a[2], x);
    const at::Tensor &offsets = tensor(a[3], "offsets");
    if (offsets.scalar_type() != at::kLong || offsets.dim() != 1 || offsets.size(0) % 2 != 1 ||
        offsets.device() != x.t.device() || !offsets.is_contiguous())
        value_error("offsets must be a contiguous int64 tensor [2 * pairs + 1] on the logits' device");
    const int64_t pairs = offsets.size(0) / 2;
    const float *ref = f32_of(a[5], 2 * pairs, x, "ref_logp"), *w = f32_of(a[6], x.rows, x, "weights");
    const long kind = PyLong_AsLong(a[7]);
    if (kind == -1 && PyErr_Occurred()) throw Raised{};
    const int average = PyObject_IsTrue(a[11]);
    if (average < 0) throw Raised{};
    const ce_preference par = {number(a[4]),  number(a[12]),          number(a[8]), number(a[9]),
                               number(a[10]), static_cast<int>(kind), average};
    at::Tensor grad, loss, pair_losses, seq, lp, work;
    int64_t grad_stride = 0;
    if (step) check_grad(a[14], x, &grad, &grad_stride);
    int st;
    {
        WithoutGil nogil;
        c10::cuda::CUDAGuard guard(x.t.device());
        lp = f32(x, {x.rows});
        seq = f32(x, {2 * pairs});
        pair_losses = f32(x, {pairs});
        loss = f32(x, {});
        work = f32(x, {4 * (step ? x.rows + 1 : 1)});
        if (step) {
            if (!grad.defined()) grad = empty(x, {x.rows, x.vocab}, x.t.scalar_type());
            st = preference_step(x.t.data_ptr(), x.dtype, x.rows, x.vocab, x.stride, labels, w,
                                 offsets.const_data_ptr<int64_t>(), pairs, ref, &par, grad.data_ptr(), grad_stride,
                                 data(lp), data(seq), data(pair_losses), data(loss), work.data_ptr(), stream_of(x));
        } else {
            st = preference_loss(x.t.data_ptr(), x.dtype, x.rows, x.vocab, x.stride, labels, w,
                                 offsets.const_data_ptr<int64_t>(), pairs, ref, &par, data(lp), data(seq),
                                 data(pair_losses), data(loss), work.data_ptr(), stream_of(x));
        }
    }
    written(st, a[14]);
    return step ? result(st, {grad, loss, pair_losses, seq, lp}) : result(st, {loss, pair_losses, seq, lp});
}

// -- the choices made from a row's softmax

// A contiguous tensor of the given type and sizes on the logits' device.
const at::Tensor &shaped(PyObject *o, at::ScalarType type, const char *type_name, at::IntArrayRef sizes, const Logits &x,
                         const char *name) {
    const at::Tensor &t = tensor(o, name);
    if (t.scalar_type() != type || t.sizes() != sizes || t.device() != x.t.device() || !t.is_contiguous()) {
        std::string shape;
        for (int64_t n : sizes) shape += (shape.empty() ? "" : ", ") + std::to_string(n);
        value_error(std::string(name) + " must be a contiguous " + type_name + " tensor [" + shape + "] on " +
                    where(x.t.device()));
    }
    return t;
}

// A temperature: a number, or an f32 tensor with one for every row.
struct Temperature {
    double all = 1.0;
    const float *rows = nullptr;
};
Temperature temperature_of(PyObject *o, const Logits &x) {
    if (!THPVariable_Check(o)) return {number(o), nullptr};
    return {1.0, f32_of(o, x.rows, x, "temperature")};
}

at::Tensor i64(const Logits &x, at::IntArrayRef sizes) { return empty(x, sizes, at::kLong); }
int64_t *longs(const at::Tensor &t) { return t.defined() ? static_cast<int64_t *>(t.data_ptr()) : nullptr; }

// The work buffer of a choice (requests < 0: of a sampling).
at::Tensor scratch(const Logits &x, int64_t requests) {
    return empty(x, {std::max<int64_t>(16, choice_work(x.dtype, x.rows, x.vocab, requests))}, at::kByte);
}

// sample(logits, uniforms, temperature, vocab, logp, out)
PyObject *sample(PyObject *const *a) {
    const Logits x = logits_of(a[0], a[3]);
    const float *u = shaped(a[1], at::kFloat, "float32", {x.rows}, x, "uniforms").const_data_ptr<float>();
    const Temperature t = temperature_of(a[2], x);
    Wanted lp = wanted(a[4], x, "logp");
    at::Tensor out;
    if (a[5] != Py_None) out = shaped(a[5], at::kLong, "int64", {x.rows}, x, "out");
    int st;
    {
        WithoutGil nogil;
        c10::cuda::CUDAGuard guard(x.t.device());
        if (!out.defined()) out = i64(x, {x.rows});
        if (lp.any && !lp.t.defined()) lp.t = f32(x, {x.rows});
        const at::Tensor work = scratch(x, -1);
        st = sample_rows(x.t.data_ptr(), x.dtype, x.rows, x.vocab, x.stride, u, t.all, t.rows, longs(out), data(lp.t),
                         work.data_ptr(), stream_of(x));
    }
    written(st, a[4]);
    written(st, a[5]);
    return result(st, {out, lp.t});
}

// verify(logits, drafts, offsets, uniforms, draft_logits, temperature, vocab, logp)
PyObject *verify(PyObject *const *a) {
    const Logits x = logits_of(a[0], a[6]);
    const int64_t *drafts = shaped(a[1], at::kLong, "int64", {x.rows}, x, "drafts").const_data_ptr<int64_t>();
    const at::Tensor &offsets = tensor(a[2], "offsets");
    if (offsets.scalar_type() != at::kLong || offsets.dim() != 1 || offsets.size(0) < 1 ||
        offsets.device() != x.t.device() || !offsets.is_contiguous())
        value_error("offsets must be a contiguous int64 tensor [requests + 1] on the logits' device");
    const int64_t requests = offsets.size(0) - 1;
    const float *u = shaped(a[3], at::kFloat, "float32", {x.rows, 2}, x, "uniforms").const_data_ptr<float>();
    const void *draft_logits = nullptr;
    int64_t draft_stride = 0;
    if (a[4] != Py_None) {
        const at::Tensor &q = tensor(a[4], "draft_logits");
        if (q.scalar_type() != x.t.scalar_type() || q.device() != x.t.device() || q.dim() != 2 || q.size(0) != x.rows ||
            q.size(1) < x.vocab || (x.rows > 0 && q.size(1) > 1 && q.stride(1) != 1))
            value_error("draft_logits must be a tensor of the logits' type, [rows=" + std::to_string(x.rows) + ", >= " +
                        std::to_string(x.vocab) + "] with contiguous rows, on " + where(x.t.device()));
        draft_logits = q.data_ptr();
        draft_stride = x.rows > 1 ? q.stride(0) : x.vocab;
        if (draft_stride < x.vocab) value_error("rows of draft_logits overlap (stride(0) < vocab)");
    }
    const Temperature t = temperature_of(a[5], x);
    Wanted lp = wanted(a[7], x, "logp");
    at::Tensor accepted, tokens, work;
    int st;
    {
        WithoutGil nogil;
        c10::cuda::CUDAGuard guard(x.t.device());
        accepted = i64(x, {requests});
        tokens = i64(x, {x.rows});
        work = scratch(x, requests);
        if (lp.any && !lp.t.defined()) lp.t = f32(x, {x.rows});
        st = verify_drafts(x.t.data_ptr(), x.dtype, x.rows, x.vocab, x.stride, drafts, draft_logits, draft_stride,
                           offsets.const_data_ptr<int64_t>(), requests, u, t.all, t.rows, longs(accepted),
                           longs(tokens), data(lp.t), work.data_ptr(), stream_of(x));
    }
    written(st, a[7]);
    return result(st, {accepted, tokens, lp.t});
}

int int_of(PyObject *o) {
    const long v = PyLong_AsLong(o);
    if (v == -1 && PyErr_Occurred()) throw Raised{};
    return v < INT32_MIN ? INT32_MIN : v > INT32_MAX ? INT32_MAX : static_cast<int>(v);
}

bool truth_of(PyObject *o) {
    const int v = PyObject_IsTrue(o);
    if (v < 0) throw Raised{};
    return v != 0;
}

// route(logits, k, score, bias, groups, top_groups, group_top, renormalise, scale, weights, counts)
PyObject *route(PyObject *const *a) {
    const Logits x = logits_of(a[0], Py_None);
    const ce_route par = {int_of(a[2]), int_of(a[1]), int_of(a[4]), int_of(a[5]), int_of(a[6]), truth_of(a[7]), number(a[8])};
    const float *bias = f32_of(a[3], x.vocab, x, "bias"), *w = f32_of(a[9], x.rows, x, "weights");
    const bool count = truth_of(a[10]);
    const int64_t k = par.k > 0 && par.k <= x.vocab ? par.k : 0;  // else refused
    at::Tensor chosen, gates, counts;
    int st;
    {
        WithoutGil nogil;
        c10::cuda::CUDAGuard guard(x.t.device());
        chosen = i64(x, {x.rows, k});
        gates = f32(x, {x.rows, k});
        if (count) counts = i64(x, {x.vocab});
        st = route_rows(x.t.data_ptr(), x.dtype, x.rows, x.vocab, x.stride, &par, bias, w, longs(chosen), data(gates),
                        longs(counts), stream_of(x));
    }
    return result(st, {chosen, gates, counts});
}

// route_grad(logits, chosen, gates_grad, score, renormalise, scale, weights, grad)
PyObject *route_gradient(PyObject *const *a) {
    const Logits x = logits_of(a[0], Py_None);
    const at::Tensor &c = tensor(a[1], "chosen");
    if (c.dim() != 2) value_error("chosen must be int64 [rows, k]");
    const int64_t k = c.size(1);
    const int64_t *chosen = shaped(a[1], at::kLong, "int64", {x.rows, k}, x, "chosen").const_data_ptr<int64_t>();
    const float *g = shaped(a[2], at::kFloat, "float32", {x.rows, k}, x, "gates_grad").const_data_ptr<float>();
    const ce_route par = {int_of(a[3]), static_cast<int>(k > 1024 ? 1025 : k), 1, 1, 1, truth_of(a[4]), number(a[5])};
    const float *w = f32_of(a[6], x.rows, x, "weights");
    at::Tensor grad;
    int64_t grad_stride = 0;
    check_grad(a[7], x, &grad, &grad_stride);
    int st;
    {
        WithoutGil nogil;
        c10::cuda::CUDAGuard guard(x.t.device());
        if (!grad.defined()) grad = empty(x, {x.rows, x.vocab}, x.t.scalar_type());
        st = route_grad(x.t.data_ptr(), x.dtype, x.rows, x.vocab, x.stride, &par, w, chosen, g, grad.data_ptr(),
                        grad_stride, stream_of(x));
    }
    written(st, a[7]);
    return result(st, {grad});
}

// One entry point: the number of arguments, and every C++ exception as a Python error.
template <PyObject *(*kFn)(PyObject *const *), Py_ssize_t kArgs>
PyObject *entry(PyObject *, PyObject *const *args, Py_ssize_t n) {
    if (n != kArgs) {
        PyErr_Format(PyExc_TypeError, "%zd arguments are wanted, not %zd", kArgs, n);
        return nullptr;
    }
    try {
        return kFn(args);
    } catch (const Refused &r) {
        PyErr_SetString(r.type, r.text.c_str());
    } catch (const Raised &) {
    } catch (const c10::OutOfMemoryError &e) {
        PyErr_SetString(out_of_memory, e.what_without_backtrace());
    } catch (const c10::Error &e) {
        PyErr_SetString(PyExc_RuntimeError, e.what_without_backtrace());
    } catch (const std::exception &e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
    } catch (...) {
        PyErr_SetString(PyExc_RuntimeError, "unknown C++ exception");
    }
    return nullptr;
}

template <PyObject *(*kFn)(PyObject *const *), Py_ssize_t kArgs>
PyCFunction fast() {
    return reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&entry<kFn, kArgs>));
}

PyMethodDef methods[] = {
    {"logp_rows", fast<logp, 7>(), METH_FASTCALL, nullptr},
    {"policy", fast<policy, 16>(), METH_FASTCALL, nullptr},
    {"preference", fast<preference, 15>(), METH_FASTCALL, nullptr},
    {"sample", fast<sample, 6>(), METH_FASTCALL, nullptr},
    {"verify", fast<verify, 8>(), METH_FASTCALL, nullptr},
    {"route", fast<route, 11>(), METH_FASTCALL, nullptr},
    {"route_grad", fast<route_gradient, 8>(), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr},
};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__binding(void) {
    PyObject *torch = PyImport_ImportModule("torch");
    if (!torch) return nullptr;
    out_of_memory = PyObject_GetAttrString(torch, "OutOfMemoryError");
    Py_DECREF(torch);
    return out_of_memory ? PyModule_Create(&module) : nullptr;
}
