// binding.cpp -- the calls of recurrent_nn_amd/lm.py on torch tensors, made in
// one step where everything is as it should be.
//
// For a few microseconds of kernel the interpreter's share counts: looking at
// a tensor's shape, strides, type and device from Python, and allocating one,
// take longer than the launch.  Each function here checks its tensors,
// allocates the outputs and the workspace, and calls the C entry point; where
// a tensor is of another kind, shape, type or device than the call needs (or
// on another device than the current one) it returns None and does nothing:
// the caller then does the same steps itself, and says what is wrong.  Returns
// the outputs as a tuple, or the C status where that is not RNN_OK.
#include "binding_common.h"

namespace {

// The entry points of the library that the interpreter has loaded.
struct Entries {
    decltype(&rnn_conv_run) conv;
    decltype(&rnn_scan_workspace_size) scan_size;
    decltype(&rnn_scan_run) scan;
    decltype(&rnn_quantize_rows) quantize;
    decltype(&rnn_quant_workspace_size) project_size;
    decltype(&rnn_quant_project) project;
    decltype(&rnn_scores_workspace_size) scores_size;
    decltype(&rnn_token_scores) scores;
} lib;

// x, weight, bias, silu, state, lens, out, state_out
PyObject *conv(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    return plain_call(a, n, 10, [&](const Call &c) {
        const at::Tensor &x = *c.tensor(a[0]), &weight = *c.tensor(a[1]);
        need(x.dim() == 3 && weight.dim() == 2);
        Call::last_contiguous(x);
        const int64_t b = x.size(0), t = x.size(1), d = x.size(2), k = weight.size(1);
        c.dense(a[1], at::kFloat, {d, k}, false);
        const at::Tensor *bias = c.dense(a[2], at::kFloat, {d});
        const at::Tensor *state = c.dense(a[4], x.scalar_type(), {b, k - 1, d});
        const at::Tensor *lens = c.dense(a[5], at::kInt, {b});
        const at::Tensor *out = c.rows(a[6], x.scalar_type(), x.sizes(), true);
        const at::Tensor *state_out = c.dense(a[7], x.scalar_type(), {b, k - 1, d});
        need(k >= 1);
        const int32_t type = type_of(x.scalar_type());
        const at::Tensor y = out ? *out : at::empty({b, t, d}, x.options());
        const at::Tensor h = state_out ? *state_out : at::empty({b, k - 1, d}, x.options());
        const rnn_conv_desc desc{b, t, d, x.stride(0), x.stride(1), y.stride(0), y.stride(1),
                                 (int32_t)k, truth(a[3]), type};
        const int status = without_gil(lib.conv, &desc, c.stream, x.data_ptr(),
                                       (const float *)weight.data_ptr(), (const float *)ptr(bias),
                                       ptr(state), (const int32_t *)ptr(lens), y.data_ptr(),
                                       h.data_ptr());
        return results(status, {y, h});
    });
}

// x, dt, A, B, C, D, z, dt_bias, dt_softplus, state, lens, out, state_out
PyObject *scan(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    return plain_call(a, n, 15, [&](const Call &c) {
        const at::Tensor &x = *c.tensor(a[0]), &B = *c.tensor(a[3]);
        need(x.dim() == 3 && (B.dim() == 3 || B.dim() == 4));
        Call::last_contiguous(x);
        const at::ScalarType kind = x.scalar_type();
        const int32_t type = type_of(kind);
        const int64_t b = x.size(0), t = x.size(1), d = x.size(2), s = B.size(-1);
        const bool grouped = B.dim() == 4;
        const int64_t groups = grouped ? B.size(2) : 1;
        need(B.scalar_type() == kind && B.size(0) == b && B.size(1) == t);
        Call::last_contiguous(B);
        const at::Tensor &dt = *c.rows(a[1], kind, x.sizes(), false);
        const at::Tensor &C = *c.rows(a[4], kind, B.sizes(), false);
        const at::Tensor &A = *c.dense(a[2], at::kFloat, {d, s}, false);
        const at::Tensor *D = c.dense(a[5], at::kFloat, {d});
        const at::Tensor *z = c.rows(a[6], kind, x.sizes(), true);
        const at::Tensor *bias = c.dense(a[7], at::kFloat, {d});
        const at::Tensor *state = c.dense(a[9], at::kFloat, {b, d, s});
        const at::Tensor *lens = c.dense(a[10], at::kInt, {b});
        const at::Tensor *out = c.rows(a[11], kind, x.sizes(), true);
        const at::Tensor *state_out = c.dense(a[12], at::kFloat, {b, d, s});
        const at::Tensor y = out ? *out : at::empty({b, t, d}, x.options());
        const at::Tensor h = state_out ? *state_out : at::empty({b, d, s}, A.options());
        const rnn_scan_desc desc{b, t, d, s, groups, x.stride(0), x.stride(1), dt.stride(0), dt.stride(1),
                                 z ? z->stride(0) : 0, z ? z->stride(1) : 0, y.stride(0), y.stride(1),
                                 B.stride(0), B.stride(1), grouped ? B.stride(2) : 0,
                                 C.stride(0), C.stride(1), grouped ? C.stride(2) : 0,
                                 type, truth(a[8])};
        size_t size = 0;
        int status = lib.scan_size(&desc, &size);
        if (status != RNN_OK)
            return results(status, {});
        const at::Tensor ws = bytes(x, size);
        status = without_gil(lib.scan, &desc, c.stream, size ? ws.data_ptr() : nullptr, size,
                             x.data_ptr(), dt.data_ptr(), (const float *)A.data_ptr(), B.data_ptr(),
                             C.data_ptr(), (const float *)ptr(D), ptr(z), (const float *)ptr(bias),
                             (const float *)ptr(state), (const int32_t *)ptr(lens), y.data_ptr(),
                             (float *)h.data_ptr());
        return results(status, {y, h});
    });
}

// x
PyObject *quantize(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    return plain_call(a, n, 3, [&](const Call &c) {
        const at::Tensor &x = *c.tensor(a[0]);
        need(x.dim() == 2);
        Call::last_contiguous(x);
        const int32_t type = type_of(x.scalar_type());
        const int64_t rows = x.size(0), cols = x.size(1), pitch = (cols + 127) / 128 * 128;
        const at::Tensor q = at::empty({rows, pitch}, x.options().dtype(at::kChar));
        const at::Tensor scale = at::empty({rows}, x.options().dtype(at::kFloat));
        const int status = without_gil(lib.quantize, c.stream, rows, cols, type, x.data_ptr(),
                                       x.stride(0), (int8_t *)q.data_ptr(), pitch,
                                       (float *)scale.data_ptr());
        return results(status, {pitch == cols ? q : q.narrow(1, 0, cols), scale});
    });
}

// 8-bit rows, readable in whole 16-byte pieces.
void eight_bit(const at::Tensor &t)
{
    need(t.scalar_type() == at::kChar && t.dim() == 2);
    Call::last_contiguous(t);
    need(t.size(0) == 0 || t.stride(0) == t.size(1) ||
         (int64_t)t.storage().nbytes() >= t.storage_offset() + (t.size(0) - 1) * t.stride(0) +
                                              (t.size(1) + 15) / 16 * 16);
}

// x, w, w_scale, bias, x_scale, out_dtype, out
PyObject *project(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    return plain_call(a, n, 9, [&](const Call &c) {
        const at::Tensor &x = *c.tensor(a[0]), &w = *c.tensor(a[1]);
        const bool eight = x.scalar_type() == at::kChar;
        need(x.dim() == 2 && eight == (a[4] != Py_None));
        Call::last_contiguous(x);
        eight_bit(w);
        const int64_t rows = x.size(0), cols = x.size(1), outs = w.size(0);
        need(w.size(1) == cols);
        const int32_t x_type = eight ? (int32_t)RNN_DTYPE_I8 : type_of(x.scalar_type());
        if (eight)
            eight_bit(x);
        const at::Tensor &w_scale = *c.dense(a[2], at::kFloat, {outs}, false);
        const at::Tensor *bias = c.dense(a[3], at::kFloat, {outs});
        const at::Tensor *x_scale = c.dense(a[4], at::kFloat, {rows});
        const at::Tensor *out = c.tensor(a[6], true);
        at::ScalarType kind = out ? out->scalar_type() : eight ? at::kFloat : x.scalar_type();
        if (a[5] != Py_None) {
            need(THPDtype_Check(a[5]));
            kind = ((THPDtype *)a[5])->scalar_type;
        }
        const int32_t y_type = type_of(kind);
        const int64_t shape[2] = {rows, outs};
        c.rows(a[6], kind, shape, true);
        const at::Tensor y = out ? *out : at::empty(shape, x.options().dtype(kind));
        const rnn_quant_desc desc{rows, cols, outs, x.stride(0), w.stride(0), y.stride(0), x_type, y_type};
        size_t size = 0;
        int status = lib.project_size(&desc, &size);
        if (status != RNN_OK)
            return results(status, {});
        const at::Tensor ws = bytes(x, size);
        status = without_gil(lib.project, &desc, c.stream, size ? ws.data_ptr() : nullptr, size,
                             x.data_ptr(), (const float *)ptr(x_scale), (const int8_t *)w.data_ptr(),
                             (const float *)w_scale.data_ptr(), (const float *)ptr(bias), y.data_ptr());
        return results(status, {y});
    });
}

// logits, tokens, top
PyObject *scores(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    return plain_call(a, n, 5, [&](const Call &c) {
        const at::Tensor &x = *c.tensor(a[0]);
        need(x.dim() == 2 && PyLong_Check(a[2]));
        Call::last_contiguous(x);
        const int64_t rows = x.size(0), vocab = x.size(1), top = PyLong_AsLongLong(a[2]);
        if (PyErr_Occurred())
            PyErr_Clear();
        need(top >= 0 && top <= RNN_SCORES_MAX_TOP && vocab > 0);
        const at::Tensor *tokens = c.tensor(a[1], true);
        const bool narrow = tokens && tokens->scalar_type() == at::kInt;
        c.dense(a[1], narrow ? at::kInt : at::kLong, {rows});
        const rnn_scores_desc desc{rows, vocab, x.stride(0), type_of(x.scalar_type()), narrow ? 4 : 8,
                                   (int32_t)top};
        size_t size = 0;
        int status = lib.scores_size(&desc, &size);
        if (status != RNN_OK)
            return results(status, {});
        const auto real = x.options().dtype(at::kFloat), whole = x.options().dtype(at::kInt);
        const at::Tensor ws = bytes(x, size);
        at::Tensor logprob, rank;
        if (tokens) {
            logprob = at::empty({rows}, real);
            rank = at::empty({rows}, whole);
        }
        const at::Tensor entropy = at::empty({rows}, real);
        const at::Tensor top_logprobs = at::empty({rows, top}, real), top_ids = at::empty({rows, top}, whole);
        status = without_gil(lib.scores, &desc, c.stream, size ? ws.data_ptr() : nullptr, size,
                             x.data_ptr(), ptr(tokens), tokens ? (float *)logprob.data_ptr() : nullptr,
                             (float *)entropy.data_ptr(), tokens ? (int32_t *)rank.data_ptr() : nullptr,
                             (float *)top_logprobs.data_ptr(), (int32_t *)top_ids.data_ptr());
        return results(status, {logprob, entropy, rank, top_logprobs, top_ids});
    });
}

// bind(address of each entry point, in the order of Entries)
PyObject *bind(PyObject *, PyObject *const *a, Py_ssize_t n) { return bind_entries(lib, a, n); }

template <class F> constexpr PyCFunction method(F f) { return (PyCFunction)(void (*)(void))f; }

PyMethodDef methods[] = {
    {"bind", method(bind), METH_FASTCALL, nullptr},
    {"conv", method(conv), METH_FASTCALL, nullptr},
    {"scan", method(scan), METH_FASTCALL, nullptr},
    {"quantize", method(quantize), METH_FASTCALL, nullptr},
    {"project", method(project), METH_FASTCALL, nullptr},
    {"scores", method(scores), METH_FASTCALL, nullptr},
    {"bind_delta", method(bind_delta), METH_FASTCALL, nullptr},
    {"delta", method(delta_call), METH_FASTCALL, nullptr},
    {"norm", method(norm_call), METH_FASTCALL, nullptr},
    {"beam", method(beam_call), METH_FASTCALL, nullptr},
    {"reorder", method(reorder_call), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__binding() { return PyModule_Create(&module); }
