// model_bind.cpp -- the Python side of include/gemm_model.h: checks of tensor
// arguments, allocation of results and workspaces, and the call, as functions
// of positional arguments for model.py (which documents them).
#include "bind.hpp"
#include "gemm_model.h"

namespace {

float number(PyObject *o) {
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred()) throw python_error();
    return (float)v;
}

// A contiguous tensor of a shape on device dev.
void *packed(const Tensor &t, const char *name, int dev, at::ScalarType dt, at::IntArrayRef size) {
    held(t, name, dev);
    if (t.scalar_type() != dt)
        fail(PyExc_TypeError, "%s has dtype %s, must be %s", name, dtype_name(t.scalar_type()), dtype_name(dt));
    if (t.sizes() != size || !t.is_contiguous()) {
        std::string want = "(";
        for (size_t i = 0; i < size.size(); ++i) want += (i ? ", " : "") + std::to_string(size[i]);
        fail(PyExc_ValueError, "%s has shape %s, must be contiguous of shape %s)", name, shape(t).c_str(), want.c_str());
    }
    return t.data_ptr();
}

// 32 or 64, from an integer tensor.
int bits(const Tensor &t, const char *name) {
    if (t.scalar_type() != at::kInt && t.scalar_type() != at::kLong)
        fail(PyExc_TypeError, "%s has dtype %s, must be int32 or int64", name, dtype_name(t.scalar_type()));
    return t.scalar_type() == at::kLong ? 64 : 32;
}

// ---- losses of the output head --------------------------------------------------

// x and w of the arguments; the device.
int head(gemm_head_args &a, const Tensor &x, const Tensor &w) {
    a.type = float_type(x, "x");
    const int dev = on_device(x, "x");
    a.ldx = rows(x, "x", dev);
    a.tokens = x.size(0);
    a.hidden = x.size(1);
    if (w.dim() != 2 || w.size(1) != a.hidden)
        fail(PyExc_ValueError, "w has shape %s, must be (vocabulary, %lld)", shape(w).c_str(), (long long)a.hidden);
    a.vocab = w.size(0);
    a.w = packed(w, "w", dev, x.scalar_type(), w.sizes());
    a.x = x.data_ptr();
    return dev;
}

struct Saved {
    Tensor lse, picked, ids, weights, mass;
    gemm_head_saved s = {};
    void of(int dev, int64_t T, int64_t k, bool teacher) {
        s.lse = (float *)packed(lse, "saved", dev, at::kFloat, {T});
        if (!teacher) {
            s.picked = (float *)packed(picked, "saved", dev, at::kFloat, {T});
            return;
        }
        s.picked = (float *)packed(picked, "saved", dev, at::kFloat, {T, k});
        s.ids = (int32_t *)packed(ids, "saved", dev, at::kInt, {T, k});
        s.weights = (float *)packed(weights, "saved", dev, at::kFloat, {T, k});
        s.mass = (float *)packed(mass, "saved", dev, at::kFloat, {T});
    }
};

Tensor head_loss(const gemm_head_args &a, const Saved &s, const Tensor &x, int dev) {
    const int64_t need = gemm_head_workspace(&a, 0);
    if (need < 0) check(gemm_head_loss(&a, nullptr, nullptr, nullptr, 0, nullptr));
    const Tensor loss = fresh({a.tokens}, at::kFloat, x.device()), ws = fresh({need}, at::kByte, x.device());
    check(gemm_head_loss(&a, (float *)loss.data_ptr(), &s.s, ws.data_ptr(), need, stream_of(dev)));
    return loss;
}

PyObject *head_backward(const gemm_head_args &a, const Saved &s, const Tensor &d_loss, const Tensor &x, bool need_dx,
                        bool need_dw, int dev) {
    const float *d = (const float *)packed(d_loss, "d_loss", dev, at::kFloat, {a.tokens});
    const int64_t need = gemm_head_workspace(&a, 1);
    if (need < 0) check(gemm_head_backward(&a, nullptr, nullptr, nullptr, nullptr, nullptr, 0, nullptr));
    const Tensor ws = fresh({need}, at::kByte, x.device());
    Tensor dx, dw;
    if (need_dx) dx = fresh({a.tokens, a.hidden}, x.scalar_type(), x.device());
    if (need_dw) dw = fresh({a.vocab, a.hidden}, x.scalar_type(), x.device());
    check(gemm_head_backward(&a, d, &s.s, ptr(dx), ptr(dw), ws.data_ptr(), need, stream_of(dev)));
    return tuple({dx, dw});
}

Tensor labels(gemm_head_args &a, PyObject *const *v, int dev) {
    const Tensor targets = needed(v[0], "targets");
    a.target_bits = bits(targets, "targets");
    a.targets = packed(targets, "targets", dev, targets.scalar_type(), {a.tokens});
    a.ignore_index = integer(v[1]);
    a.scale = number(v[2]);
    a.z_loss = number(v[3]);
    return targets;
}

// (x, w, targets, ignore_index, scale, z_loss) -> (loss, lse, picked)
PyObject *cross_entropy(PyObject *, Args v, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    count(n, 6);
    const Tensor x = needed(v[0], "x"), w = needed(v[1], "w");
    gemm_head_args a = {};
    const int dev = head(a, x, w);
    const Tensor targets = labels(a, v + 2, dev);
    Saved s;
    s.lse = fresh({a.tokens}, at::kFloat, x.device());
    s.picked = fresh({a.tokens}, at::kFloat, x.device());
    s.of(dev, a.tokens, 1, false);
    const Tensor loss = head_loss(a, s, x, dev);
    return tuple({loss, s.lse, s.picked});
    END_HANDLE_TH_ERRORS
}

// (d_loss, x, w, lse, picked, targets, ignore_index, scale, z_loss, need_dx, need_dw) -> (dx, dw)
PyObject *cross_entropy_backward(PyObject *, Args v, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    count(n, 11);
    const Tensor d_loss = needed(v[0], "d_loss"), x = needed(v[1], "x"), w = needed(v[2], "w");
    gemm_head_args a = {};
    const int dev = head(a, x, w);
    Saved s;
    s.lse = needed(v[3], "saved");
    s.picked = needed(v[4], "saved");
    s.of(dev, a.tokens, 1, false);
    const Tensor targets = labels(a, v + 5, dev);
    return head_backward(a, s, d_loss, x, v[9] == Py_True, v[10] == Py_True, dev);
    END_HANDLE_TH_ERRORS
}

// (x, w, ids, logits, temperature, scale) -> (loss, lse, picked, ids, weights, mass)
PyObject *distillation(PyObject *, Args v, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    count(n, 6);
    const Tensor x = needed(v[0], "x"), w = needed(v[1], "w"), ids = needed(v[2], "teacher_ids"),
                 logits = needed(v[3], "teacher_logits");
    gemm_head_args a = {};
    const int dev = head(a, x, w);
    if (ids.dim() != 2 || ids.size(0) != a.tokens || ids.size(1) < 1)
        fail(PyExc_ValueError, "teacher_ids has shape %s, must be (%lld, entries)", shape(ids).c_str(),
             (long long)a.tokens);
    const int64_t T = a.tokens, k = ids.size(1);
    if (k > GEMM_HEAD_MAX_ENTRIES)
        fail(PyExc_ValueError, "teacher_ids has %lld entries a token, at most %d", (long long)k, GEMM_HEAD_MAX_ENTRIES);
    a.entries = (int32_t)k;
    a.teacher_ids = (const int32_t *)packed(ids, "teacher_ids", dev, at::kInt, {T, k});
    a.teacher_type = float_type(logits, "teacher_logits");
    a.ld_teacher = rows(logits, "teacher_logits", dev, logits.scalar_type(), T, k);
    a.teacher_logits = logits.data_ptr();
    a.temperature = number(v[4]);
    a.scale = number(v[5]);
    Saved s;
    s.lse = fresh({T}, at::kFloat, x.device());
    s.mass = fresh({T}, at::kFloat, x.device());
    s.picked = fresh({T, k}, at::kFloat, x.device());
    s.weights = fresh({T, k}, at::kFloat, x.device());
    s.ids = fresh({T, k}, at::kInt, x.device());
    s.of(dev, T, k, true);
    const Tensor loss = head_loss(a, s, x, dev);
    return tuple({loss, s.lse, s.picked, s.ids, s.weights, s.mass});
    END_HANDLE_TH_ERRORS
}

// (d_loss, x, w, lse, picked, ids, weights, mass, temperature, scale, need_dx, need_dw) -> (dx, dw)
PyObject *distillation_backward(PyObject *, Args v, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    count(n, 12);
    const Tensor d_loss = needed(v[0], "d_loss"), x = needed(v[1], "x"), w = needed(v[2], "w");
    gemm_head_args a = {};
    const int dev = head(a, x, w);
    Saved s;
    s.lse = needed(v[3], "saved");
    s.picked = needed(v[4], "saved");
    s.ids = needed(v[5], "saved");
    s.weights = needed(v[6], "saved");
    s.mass = needed(v[7], "saved");
    if (s.ids.dim() != 2 || s.ids.size(1) < 1 || s.ids.size(1) > GEMM_HEAD_MAX_ENTRIES)
        fail(PyExc_ValueError, "saved must be what linear_distillation returned for these tokens");
    a.entries = (int32_t)s.ids.size(1);
    s.of(dev, a.tokens, a.entries, true);
    a.temperature = number(v[8]);
    a.scale = number(v[9]);
    return head_backward(a, s, d_loss, x, v[10] == Py_True, v[11] == Py_True, dev);
    END_HANDLE_TH_ERRORS
}

// ---- tokens by expert --------------------------------------------------------------

// (ids, experts) -> (offsets, row_of)
PyObject *expert_sort(PyObject *, Args v, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    count(n, 2);
    const Tensor ids = needed(v[0], "ids");
    const int64_t E = integer(v[1]);
    if (E < 1 || E > GEMM_EXPERT_MAX_EXPERTS)
        fail(PyExc_ValueError, "experts must be 1 to %d, is %lld", GEMM_EXPERT_MAX_EXPERTS, (long long)E);
    const int id_bits = bits(ids, "ids"), dev = on_device(ids, "ids");
    if (ids.dim() != 2 || ids.size(1) < 1)
        fail(PyExc_ValueError, "ids has shape %s, must be (tokens, top_k)", shape(ids).c_str());
    const int64_t T = ids.size(0), k = ids.size(1);
    if (k >= 1LL << 31 || (T > 0 && k > ((1LL << 31) - 1) / T))
        fail(PyExc_ValueError, "ids of shape %s are 2^31 slots or more", shape(ids).c_str());
    const void *p = packed(ids, "ids", dev, ids.scalar_type(), {T, k});
    const Tensor offsets = fresh({E + 1}, at::kInt, ids.device()), row_of = fresh({T, k}, at::kInt, ids.device());
    const int64_t need = gemm_expert_sort_workspace(T, (int32_t)k, (int32_t)E);
    Tensor ws;
    if (need > 0) ws = fresh({need}, at::kByte, ids.device());
    check(gemm_expert_sort(p, id_bits, T, (int32_t)k, (int32_t)E, (int32_t *)offsets.data_ptr(),
                           (int32_t *)row_of.data_ptr(), ptr(ws), need, stream_of(dev)));
    return tuple({offsets, row_of});
    END_HANDLE_TH_ERRORS
}

// A sort's results.
struct Order {
    const int32_t *offsets, *row_of;
    int32_t experts, top_k;
    int64_t T;
    Order(const Tensor &o, const Tensor &r, int dev) {
        if (o.dim() != 1 || o.size(0) < 2 || o.size(0) > GEMM_EXPERT_MAX_EXPERTS + 1 || r.dim() != 2 || r.size(1) < 1)
            fail(PyExc_ValueError, "order must be what expert_sort returned");
        T = r.size(0);
        top_k = (int32_t)r.size(1);
        experts = (int32_t)o.size(0) - 1;
        offsets = (const int32_t *)packed(o, "the order's offsets", dev, at::kInt, o.sizes());
        row_of = (const int32_t *)packed(r, "the order's row_of", dev, at::kInt, r.sizes());
    }
};

// (x, offsets, row_of) -> rows
PyObject *expert_gather(PyObject *, Args v, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    count(n, 3);
    const Tensor x = needed(v[0], "x"), offsets = needed(v[1], "order"), row_of = needed(v[2], "order");
    const gemm_dtype type = float_type(x, "x");
    const int dev = on_device(x, "x");
    const Order o(offsets, row_of, dev);
    const int64_t ld = rows(x, "x", dev, x.scalar_type(), o.T, x.dim() == 2 ? x.size(1) : 0), H = x.size(1);
    const Tensor out = fresh({o.T * o.top_k, H}, x.scalar_type(), x.device());
    check(gemm_expert_gather(type, x.data_ptr(), ld, out.data_ptr(), H, o.T, H, o.top_k, o.experts, o.offsets,
                             o.row_of, stream_of(dev)));
    return wrap(out);
    END_HANDLE_TH_ERRORS
}

// (rows, offsets, row_of, weights?) -> out
PyObject *expert_combine(PyObject *, Args v, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    count(n, 4);
    const Tensor y = needed(v[0], "rows"), offsets = needed(v[1], "order"), row_of = needed(v[2], "order"),
                 weights = tensor(v[3], "weights");
    const gemm_dtype type = float_type(y, "rows");
    const int dev = on_device(y, "rows");
    const Order o(offsets, row_of, dev);
    const int64_t ld = rows(y, "rows", dev, y.scalar_type(), o.T * o.top_k, y.dim() == 2 ? y.size(1) : 0);
    const int64_t H = y.size(1);
    const float *w =
        weights.defined() ? (const float *)packed(weights, "weights", dev, at::kFloat, {o.T, o.top_k}) : nullptr;
    const Tensor out = fresh({o.T, H}, y.scalar_type(), y.device());
    check(gemm_expert_combine(type, y.data_ptr(), ld, w, out.data_ptr(), H, o.T, H, o.top_k, o.experts, o.offsets,
                              o.row_of, stream_of(dev)));
    return wrap(out);
    END_HANDLE_TH_ERRORS
}

// (d_out, rows, offsets, row_of, weights) -> (d_rows, d_weights)
PyObject *expert_combine_backward(PyObject *, Args v, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    count(n, 5);
    const Tensor d = needed(v[0], "d_out"), y = needed(v[1], "rows"), offsets = needed(v[2], "order"),
                 row_of = needed(v[3], "order"), weights = tensor(v[4], "weights");
    const gemm_dtype type = float_type(d, "d_out");
    const int dev = on_device(d, "d_out");
    const Order o(offsets, row_of, dev);
    const int64_t ld_d = rows(d, "d_out", dev, d.scalar_type(), o.T, d.dim() == 2 ? d.size(1) : 0), H = d.size(1);
    const int64_t ld = rows(y, "rows", dev, d.scalar_type(), o.T * o.top_k, H);
    const float *w =
        weights.defined() ? (const float *)packed(weights, "weights", dev, at::kFloat, {o.T, o.top_k}) : nullptr;
    const Tensor d_rows = fresh({o.T * o.top_k, H}, d.scalar_type(), d.device());
    Tensor d_weights;
    if (weights.defined()) d_weights = fresh({o.T, o.top_k}, at::kFloat, d.device());
    check(gemm_expert_combine_backward(type, d.data_ptr(), ld_d, y.data_ptr(), ld, w, d_rows.data_ptr(), H,
                                       (float *)ptr(d_weights), o.T, H, o.top_k, o.experts, o.offsets, o.row_of,
                                       stream_of(dev)));
    return tuple({d_rows, d_weights});
    END_HANDLE_TH_ERRORS
}

PyMethodDef methods[] = {FAST("cross_entropy", cross_entropy), FAST("cross_entropy_backward", cross_entropy_backward),
                         FAST("distillation", distillation), FAST("distillation_backward", distillation_backward),
                         FAST("expert_sort", expert_sort), FAST("expert_gather", expert_gather),
                         FAST("expert_combine", expert_combine),
                         FAST("expert_combine_backward", expert_combine_backward), {"set_check", set_check, METH_O, nullptr},
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_model", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__model() { return PyModule_Create(&module); }
