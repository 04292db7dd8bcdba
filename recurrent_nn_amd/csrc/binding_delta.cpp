// binding_delta.cpp -- the calls of recurrent_nn_amd/delta.py on torch tensors,
// made in one step where everything is as it should be (as binding.cpp).
#include "binding_common.h"

#include <cmath>

namespace {

struct Entries {
    decltype(&rnn_delta_workspace_size) delta_size;
    decltype(&rnn_delta_run) delta;
    decltype(&rnn_gated_norm) norm;
    decltype(&rnn_beam_workspace_size) beam_size;
    decltype(&rnn_beam_select) beam;
    decltype(&rnn_reorder_states) reorder;
} lib;

double number(PyObject *o)
{
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred())
        throw python_error();
    return v;
}

// A whole number that is one already (no subclass, no object with __index__).
int64_t whole(PyObject *o)
{
    need(PyLong_CheckExact(o));
    const int64_t v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred()) {
        PyErr_Clear();
        throw NotPlain{};
    }
    return v;
}

}  // namespace

PyObject *bind_delta(PyObject *, PyObject *const *a, Py_ssize_t n) { return bind_entries(lib, a, n); }

// q, k, v, beta, g, A, dt_bias, beta_sigmoid, normalize, scale, state, lens, out, state_out
PyObject *delta_call(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    return plain_call(a, n, 16, [&](const Call &c) {
        const at::Tensor &q = *c.tensor(a[0]), &k = *c.tensor(a[1]), &v = *c.tensor(a[2]);
        need(q.dim() == 4 && v.dim() == 4);
        Call::last_contiguous(q);
        const at::ScalarType kind = q.scalar_type();
        const int32_t type = type_of(kind);
        const int64_t b = q.size(0), t = q.size(1), kh = q.size(2), dk = q.size(3), h = v.size(2),
                      dv = v.size(3);
        c.rows(a[1], kind, q.sizes(), false);
        need(v.scalar_type() == kind && v.size(0) == b && v.size(1) == t);
        Call::last_contiguous(v);
        const at::Tensor &beta = *c.tensor(a[3]);
        const at::ScalarType gate = beta.scalar_type();
        need(gate == at::kFloat || gate == kind);
        const int64_t gates[3] = {b, t, h};
        c.rows(a[3], gate, gates, false);
        const at::Tensor *g = c.rows(a[4], gate, gates, true);
        const at::Tensor *A = c.dense(a[5], at::kFloat, {h});
        const at::Tensor *bias = c.dense(a[6], at::kFloat, {h});
        const at::Tensor *state = c.dense(a[10], at::kFloat, {b, h, dk, dv});
        const at::Tensor *lens = c.dense(a[11], at::kInt, {b});
        const at::Tensor *out = c.rows(a[12], kind, v.sizes(), true);
        const at::Tensor *state_out = c.dense(a[13], at::kFloat, {b, h, dk, dv});
        need(dk >= 1);
        const float scale = a[9] == Py_None ? (float)(1.0 / std::sqrt((double)dk)) : (float)number(a[9]);
        const bool sigmoid = truth(a[7]), normalize = truth(a[8]);
        const at::Tensor o = out ? *out : at::empty({b, t, h, dv}, q.options());
        const at::Tensor s = state_out ? *state_out
                                       : at::empty({b, h, dk, dv}, q.options().dtype(at::kFloat));
        const rnn_delta_desc desc{b, t, kh, h, dk, dv, q.stride(0), q.stride(1), q.stride(2),
                                  k.stride(0), k.stride(1), k.stride(2), v.stride(0), v.stride(1),
                                  v.stride(2), o.stride(0), o.stride(1), o.stride(2), beta.stride(0),
                                  beta.stride(1), g ? g->stride(0) : 0, g ? g->stride(1) : 0, type,
                                  type_of(gate), normalize, sigmoid, scale};
        size_t size = 0;
        int status = lib.delta_size(&desc, &size);
        if (status != RNN_OK)
            return results(status, {});
        const at::Tensor ws = bytes(q, size);
        status = without_gil(lib.delta, &desc, c.stream, size ? ws.data_ptr() : nullptr, size,
                             q.data_ptr(), k.data_ptr(), v.data_ptr(), beta.data_ptr(), ptr(g),
                             (const float *)ptr(A), (const float *)ptr(bias), (const float *)ptr(state),
                             (const int32_t *)ptr(lens), o.data_ptr(), (float *)s.data_ptr());
        return results(status, {o, s});
    });
}

// x, weight, z, gate_first, eps, out
PyObject *norm_call(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    return plain_call(a, n, 8, [&](const Call &c) {
        const at::Tensor &x = *c.tensor(a[0]), &w = *c.tensor(a[1]);
        const int64_t dims = x.dim();
        need(dims == 2 || dims == 3);
        Call::last_contiguous(x);
        const at::ScalarType kind = x.scalar_type();
        const int64_t rows = x.size(0), groups = dims == 3 ? x.size(1) : 1, dim = x.size(-1);
        if (w.dim() == 1)
            c.dense(a[1], at::kFloat, {dim}, false);
        else
            c.dense(a[1], at::kFloat, {groups, dim}, false);
        const at::Tensor *z = c.rows(a[2], kind, x.sizes(), true);
        const at::Tensor *out = c.rows(a[5], kind, x.sizes(), true);
        const bool first = truth(a[3]);
        const float eps = (float)number(a[4]);
        const int32_t type = type_of(kind);
        const at::Tensor y = out ? *out : at::empty(x.sizes(), x.options());
        const auto group = [&](const at::Tensor *t) { return t && dims == 3 ? t->stride(1) : 0; };
        const rnn_norm_desc desc{rows, groups, dim, x.stride(0), group(&x), z ? z->stride(0) : 0, group(z),
                                 y.stride(0), group(&y), w.dim() == 1 ? 0 : dim, type, first, eps};
        const int status = without_gil(lib.norm, &desc, c.stream, x.data_ptr(), (const float *)w.data_ptr(),
                                       ptr(z), y.data_ptr());
        return results(status, {y});
    });
}

// logits, scores, keep, finished, eos
PyObject *beam_call(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    return plain_call(a, n, 7, [&](const Call &c) {
        const at::Tensor &x = *c.tensor(a[0]);
        need(x.dim() == 3);
        Call::last_contiguous(x);
        const int64_t b = x.size(0), beams = x.size(1), vocab = x.size(2);
        const int64_t keep = a[2] == Py_None ? beams : whole(a[2]);
        const at::Tensor &scores = *c.dense(a[1], at::kFloat, {b, beams}, false);
        const at::Tensor *finished = c.tensor(a[3], true);
        const int64_t eos = finished ? whole(a[4]) : 0;
        if (finished)
            c.dense(a[3], finished->scalar_type() == at::kByte ? at::kByte : at::kBool, {b, beams});
        need(keep >= 1 && keep <= RNN_BEAM_MAX);
        const rnn_beam_desc desc{b, beams, vocab, x.stride(0), x.stride(1), type_of(x.scalar_type()),
                                 (int32_t)keep, eos};
        size_t size = 0;
        int status = lib.beam_size(&desc, &size);
        if (status != RNN_OK)
            return results(status, {});
        const at::Tensor ws = bytes(x, size);
        const auto ids = x.options().dtype(at::kInt);
        const at::Tensor values = at::empty({b, keep}, x.options().dtype(at::kFloat));
        const at::Tensor tokens = at::empty({b, keep}, ids), parents = at::empty({b, keep}, ids);
        status = without_gil(lib.beam, &desc, c.stream, size ? ws.data_ptr() : nullptr, size, x.data_ptr(),
                             (const float *)scores.data_ptr(), (const uint8_t *)ptr(finished),
                             (float *)values.data_ptr(), (int32_t *)tokens.data_ptr(),
                             (int32_t *)parents.data_ptr());
        return results(status, {values, tokens, parents});
    });
}

// states (a list), parents, dim (a whole number), out (a list or None): a list
PyObject *reorder_call(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    return plain_call(a, n, 6, [&](const Call &c) -> PyObject * {
        need(PyList_CheckExact(a[0]) && (a[3] == Py_None || PyList_CheckExact(a[3])));
        const at::Tensor &parents = *c.tensor(a[1]);
        need(parents.scalar_type() == at::kInt && parents.dim() == 2 && parents.is_contiguous());
        const int64_t dim = whole(a[2]), batch = parents.size(0), keep = parents.size(1);
        const Py_ssize_t count = PyList_GET_SIZE(a[0]);
        need(batch > 0 && dim >= 0 && count > 0 && (a[3] == Py_None || PyList_GET_SIZE(a[3]) == count));
        std::vector<rnn_reorder_item> items;
        std::vector<at::Tensor> outs;
        items.reserve(count);
        outs.reserve(count);
        int64_t beams = 0;
        for (Py_ssize_t i = 0; i < count; ++i) {
            const at::Tensor &x = *c.tensor(PyList_GET_ITEM(a[0], i));
            need(x.is_contiguous() && dim < x.dim() && x.size(dim) % batch == 0);
            if (i == 0)
                beams = x.size(dim) / batch;
            need(beams > 0 && x.size(dim) == batch * beams);
            int64_t outer = 1, inner = (int64_t)x.element_size();
            for (int64_t d = 0; d < x.dim(); ++d)
                (d < dim ? outer : inner) *= d == dim ? 1 : x.size(d);
            at::DimVector sizes(x.sizes());
            sizes[dim] = batch * keep;
            if (a[3] == Py_None) {
                outs.push_back(at::empty(sizes, x.options()));
            } else {
                const at::Tensor &o = *c.tensor(PyList_GET_ITEM(a[3], i));
                need(o.is_contiguous() && o.scalar_type() == x.scalar_type() && o.sizes() == at::IntArrayRef(sizes));
                outs.push_back(o);
            }
            items.push_back({x.data_ptr(), outs.back().data_ptr(), outer, inner});
        }
        const int status = without_gil(lib.reorder, c.stream, batch, beams, keep,
                                       (const int32_t *)parents.data_ptr(),
                                       (const rnn_reorder_item *)items.data(), (int64_t)count);
        if (status != RNN_OK)
            return PyLong_FromLong(status);
        PyObject *list = PyList_New(count);
        if (!list)
            return nullptr;
        for (Py_ssize_t i = 0; i < count; ++i) {
            PyObject *o = THPVariable_Wrap(outs[i]);
            if (!o) {
                Py_DECREF(list);
                return nullptr;
            }
            PyList_SET_ITEM(list, i, o);
        }
        return list;
    });
}
