// block_bind.cpp -- the Python side of include/gemm_block.h: checks of tensor
// arguments, allocation of results and workspaces, and the call, as functions
// of positional arguments for block.py (which documents them). In C++ because
// a call of this kind is shorter than its marshalling in Python: one token's
// norms took 11.7 us a pass through ctypes, of which 4 are the kernel's.
#include "bind.hpp"
#include "gemm_block.h"

namespace {

// ---- MXFP4 ------------------------------------------------------------------------

// (x, rows?, columns?) -> codes and scales of either form, None where not asked for
PyObject *quantize(PyObject *, Args v, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    count(n, 3);
    const Tensor x = needed(v[0], "x");
    const gemm_dtype type = float_type(x, "x");
    const int dev = on_device(x, "x");
    const int64_t ld = rows(x, "x", dev), R = x.size(0), C = x.size(1);
    Tensor rc, rs, cc, cs;
    const auto pair = [&](int64_t n, int64_t k, Tensor &codes, Tensor &scales) {
        const int64_t kp = gemm_mx4_padded(k);
        codes = fresh({n, kp / 2}, at::kByte, x.device());
        scales = fresh({n, kp / 32}, at::kByte, x.device());
    };
    if (v[1] == Py_True) pair(R, C, rc, rs);
    if (v[2] == Py_True) pair(C, R, cc, cs);
    check(gemm_mx4_quantize(x.data_ptr(), type, R, C, ld, (uint8_t *)ptr(rc), (uint8_t *)ptr(rs),
                            (uint8_t *)ptr(cc), (uint8_t *)ptr(cs), stream_of(dev)));
    return tuple({rc, rs, cc, cs});
    END_HANDLE_TH_ERRORS
}

// (codes, scales, k, dtype) -> values
PyObject *dequantize(PyObject *, Args v, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    count(n, 4);
    const Tensor codes = needed(v[0], "codes"), scales = needed(v[1], "scales");
    const int64_t k = integer(v[2]);
    if (!THPDtype_Check(v[3])) fail(PyExc_TypeError, "dtype must be a torch dtype");
    const at::ScalarType dt = reinterpret_cast<THPDtype *>(v[3])->scalar_type;
    if (dt != at::kFloat && dt != at::kHalf && dt != at::kBFloat16)
        fail(PyExc_TypeError, "dtype %s must be float32, float16 or bfloat16", dtype_name(dt));
    const int dev = on_device(codes, "codes");
    on_device(scales, "scales");
    std::vector<int64_t> size(codes.sizes().begin(), codes.sizes().end());
    size.back() = k;
    int64_t lead = 1;
    for (size_t i = 0; i + 1 < size.size(); ++i) lead *= size[i];
    const Tensor out = fresh(size, dt, codes.device());
    check(gemm_mx4_dequantize((const uint8_t *)codes.data_ptr(), (const uint8_t *)scales.data_ptr(), lead, k,
                              out.data_ptr(), dt == at::kFloat ? GEMM_F32 : dt == at::kHalf ? GEMM_F16 : GEMM_BF16,
                              k, stream_of(dev)));
    return wrap(out);
    END_HANDLE_TH_ERRORS
}

// (plan, x, codes, scales, N, K, bias, out) -> y
PyObject *linear(PyObject *, Args v, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    count(n, 8);
    void *plan = PyLong_AsVoidPtr(v[0]);
    const Tensor x = needed(v[1], "x"), codes = needed(v[2], "weight"), scales = needed(v[3], "weight"),
                 bias = tensor(v[6], "bias");
    Tensor out = tensor(v[7], "out");
    const int64_t N = integer(v[4]), K = integer(v[5]);
    const gemm_dtype type = float_type(x, "x");
    const int dev = on_device(x, "x");
    held(codes, "the weight's codes", dev);
    held(scales, "the weight's scales", dev);
    const int64_t ld = rows(x, "x", dev), M = x.size(0);
    if (x.size(1) != K)
        fail(PyExc_ValueError, "x has %lld columns, the weight %lld", (long long)x.size(1), (long long)K);
    const void *b = vector(bias, "bias", dev, at::kBFloat16, N);
    const int64_t need = gemm_mx4_linear_workspace(M, K);
    Tensor ws;
    if (need > 0) ws = fresh({need}, at::kByte, x.device());
    if (!out.defined()) out = fresh({M, N}, at::kBFloat16, x.device());
    else if (rows(out, "out", dev, at::kBFloat16, M, N) != N) fail(PyExc_ValueError, "out must be contiguous");
    check(gemm_mx4_linear((gemm_plan_t)plan, x.data_ptr(), type, ld, (const uint8_t *)codes.data_ptr(),
                          (const uint8_t *)scales.data_ptr(), b, out.data_ptr(), M, N, K, ptr(ws), need,
                          stream_of(dev)));
    return wrap(out);
    END_HANDLE_TH_ERRORS
}

// (plan, dy, x, codes, scales, N, K, need_dx, need_dw) -> (dx, dw)
PyObject *linear_backward(PyObject *, Args v, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    count(n, 9);
    void *plan = PyLong_AsVoidPtr(v[0]);
    const bool need_dx = v[7] == Py_True, need_dw = v[8] == Py_True;
    const Tensor dy = needed(v[1], "dy"), x = need_dw ? needed(v[2], "x") : Tensor(), codes = tensor(v[3], "weight_t"),
                 scales = tensor(v[4], "weight_t");
    const int64_t N = integer(v[5]), K = integer(v[6]);
    const gemm_dtype type = float_type(dy, "dy");
    const int dev = on_device(dy, "dy");
    if (need_dx) {
        held(needed(v[3], "weight_t"), "weight_t's codes", dev);
        held(needed(v[4], "weight_t"), "weight_t's scales", dev);
    }
    const int64_t ld = rows(dy, "dy", dev), M = dy.size(0);
    if (dy.size(1) != N)
        fail(PyExc_ValueError, "dy has %lld columns, the weight %lld rows", (long long)dy.size(1), (long long)N);
    const int64_t ldx = need_dw ? rows(x, "x", dev, dy.scalar_type(), M, K) : 0;
    const int64_t need = gemm_mx4_linear_backward_workspace(M, N, K);
    const Tensor ws = fresh({need}, at::kByte, dy.device());
    Tensor dx, dw;
    if (need_dx) dx = fresh({M, K}, at::kBFloat16, dy.device());
    if (need_dw) dw = fresh({N, K}, at::kBFloat16, dy.device());
    check(gemm_mx4_linear_backward((gemm_plan_t)plan, dy.data_ptr(), ld, ptr(x), ldx, type,
                                   need_dx ? (const uint8_t *)ptr(codes) : nullptr,
                                   need_dx ? (const uint8_t *)ptr(scales) : nullptr, ptr(dx), ptr(dw), M, N, K,
                                   ws.data_ptr(), need, stream_of(dev)));
    return tuple({dx, dw});
    END_HANDLE_TH_ERRORS
}

// ---- mixture of experts ---------------------------------------------------------------

// (desc, x, row_mask, out, routing?, workspace, router) -> (out, ids, probs); the
// router stands for all that desc points to
PyObject *moe(PyObject *, Args v, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    count(n, 7);
    const gemm_moe_desc *d = (const gemm_moe_desc *)PyLong_AsVoidPtr(v[0]);
    const Tensor x = needed(v[1], "x"), ws = needed(v[5], "workspace");
    Tensor mask = tensor(v[2], "row_mask"), out = tensor(v[3], "out"), ids, probs;
    const bool routing = v[4] == Py_True;
    const at::ScalarType dt = d->type == GEMM_F16 ? at::kHalf : at::kBFloat16;
    const int dev = on_device(x, "x");
    held(needed(v[6], "router"), "the layer", dev);
    held(ws, "workspace", dev);
    const int64_t ldx = rows(x, "x", dev, dt), T = x.size(0), H = x.size(1);
    if (H != d->hidden)
        fail(PyExc_ValueError, "x has %lld columns, the layer %lld", (long long)H, (long long)d->hidden);
    const void *m = vector(mask, "row_mask", dev, mask.defined() && mask.scalar_type() == at::kBool ? at::kBool : at::kByte, T);
    int64_t ldo = H;
    if (!out.defined()) out = fresh({T, H}, dt, x.device());
    else ldo = rows(out, "out", dev, dt, T, H);
    if (routing) {
        ids = fresh({T, d->top_k}, at::kInt, x.device());
        probs = fresh({T, d->top_k}, at::kFloat, x.device());
    }
    check(gemm_moe_forward(d, x.data_ptr(), ldx, (const uint8_t *)m, out.data_ptr(), ldo, (int32_t *)ptr(ids),
                           (float *)ptr(probs), T, ws.data_ptr(), ws.numel(), stream_of(dev)));
    return tuple({out, ids, probs});
    END_HANDLE_TH_ERRORS
}

// ---- norms around a block ---------------------------------------------------------------

int64_t gate_rows(const Tensor &gate, int dev, at::ScalarType dt, int64_t T, int64_t H, int64_t &ld) {
    if (!gate.defined()) {
        ld = 0;
        return 0;
    }
    ld = rows(gate, "gate", dev, dt);
    const int64_t g = gate.size(0);
    if (gate.size(1) != H || (T > 0 && (g == 0 || T % g)))
        fail(PyExc_ValueError, "gate has shape %s: its rows must divide %lld rows of %lld columns",
                                shape(gate).c_str(), (long long)T, (long long)H);
    return g;
}

// (block, residual, w_post, gate, scale, w_next, eps, act) -> (out, next, saved)
PyObject *norm(PyObject *, Args v, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    count(n, 8);
    const Tensor block = tensor(v[0], "block"), residual = needed(v[1], "residual"), w_post = tensor(v[2], "w_post"),
                 gate = tensor(v[3], "gate"), scale = tensor(v[4], "scale"), w_next = tensor(v[5], "w_next");
    gemm_norm_args a = {};
    a.eps = (float)PyFloat_AsDouble(v[6]);
    if (PyErr_Occurred()) throw python_error();
    a.gate_act = (gemm_epilogue)integer(v[7]);
    a.type = float_type(residual, "residual");
    const int dev = on_device(residual, "residual");
    const at::ScalarType dt = residual.scalar_type();
    a.ld_residual = rows(residual, "residual", dev);
    const int64_t T = residual.size(0), H = residual.size(1);
    a.rows = T;
    a.cols = H;
    if (block.defined()) a.ld_block = rows(block, "block", dev, dt, T, H);
    a.gate_rows = gate_rows(gate, dev, dt, T, H, a.ld_gate);
    a.w_post = vector(w_post, "w_post", dev, dt, H);
    a.scale = vector(scale, "scale", dev, dt, H);
    a.w_next = vector(w_next, "w_next", dev, dt, H);
    const Tensor saved = fresh({2, T}, at::kFloat, residual.device());
    const Tensor out = block.defined() ? fresh({T, H}, dt, residual.device()) : residual;
    const Tensor next = w_next.defined() ? fresh({T, H}, dt, residual.device()) : Tensor();
    a.block = ptr(block);
    a.residual = residual.data_ptr();
    a.gate = ptr(gate);
    a.out = block.defined() ? out.data_ptr() : nullptr;
    a.next = ptr(next);
    a.ld_out = a.ld_next = H;
    a.rstd_post = (float *)saved.data_ptr();
    a.rstd_next = a.rstd_post + T;
    check(gemm_norm_residual(&a, stream_of(dev)));
    return tuple({out, next, saved});
    END_HANDLE_TH_ERRORS
}

// (d_out, d_next, block, out, saved, w_post, gate, scale, w_next, act) ->
// (d_block, d_residual, d_gate, d_scale, d_w_post, d_w_next)
PyObject *norm_backward(PyObject *, Args v, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    count(n, 10);
    const Tensor d_out = tensor(v[0], "d_out"), d_next = tensor(v[1], "d_next"), block = tensor(v[2], "block"),
                 out = needed(v[3], "out"), saved = needed(v[4], "saved"), w_post = tensor(v[5], "w_post"),
                 gate = tensor(v[6], "gate"), scale = tensor(v[7], "scale"), w_next = tensor(v[8], "w_next");
    gemm_norm_backward_args a = {};
    a.gate_act = (gemm_epilogue)integer(v[9]);
    a.type = float_type(out, "out");
    const int dev = on_device(out, "out");
    const at::ScalarType dt = out.scalar_type();
    a.ld_out = rows(out, "out", dev);
    const int64_t T = out.size(0), H = out.size(1);
    a.rows = T;
    a.cols = H;
    if (d_next.defined() != w_next.defined()) fail(PyExc_ValueError, "d_next and w_next go together");
    if (saved.scalar_type() != at::kFloat || saved.dim() != 2 || saved.size(0) != 2 || saved.size(1) != T ||
        !saved.is_contiguous())
        fail(PyExc_ValueError, "saved must be what norm_residual returned for these rows");
    on_device(saved, "saved");
    if (block.defined()) a.ld_block = rows(block, "block", dev, dt, T, H);
    if (d_out.defined()) a.ld_d_out = rows(d_out, "d_out", dev, dt, T, H);
    if (d_next.defined()) a.ld_d_next = rows(d_next, "d_next", dev, dt, T, H);
    a.gate_rows = gate_rows(gate, dev, dt, T, H, a.ld_gate);
    a.w_post = vector(w_post, "w_post", dev, dt, H);
    a.scale = vector(scale, "scale", dev, dt, H);
    a.w_next = vector(w_next, "w_next", dev, dt, H);
    a.d_out = ptr(d_out);
    a.d_next = ptr(d_next);
    a.block = ptr(block);
    a.out = out.data_ptr();
    a.gate = ptr(gate);
    a.rstd_post = (const float *)saved.data_ptr();
    a.rstd_next = a.rstd_post + T;
    const at::Device device = out.device();
    const int64_t need = gemm_norm_backward_workspace(&a);
    if (need < 0) check(gemm_norm_residual_backward(&a, stream_of(dev)));
    const Tensor d_residual = fresh({T, H}, dt, device), ws = fresh({need}, at::kByte, device);
    Tensor d_block, d_gate, d_scale, d_w_post, d_w_next;
    if (block.defined()) d_block = fresh({T, H}, dt, device);
    if (gate.defined()) d_gate = fresh({a.gate_rows, H}, dt, device);
    if (scale.defined()) d_scale = fresh({H}, dt, device);
    if (w_post.defined()) d_w_post = fresh({H}, dt, device);
    if (w_next.defined()) d_w_next = fresh({H}, dt, device);
    a.d_block = ptr(d_block);
    a.d_residual = d_residual.data_ptr();
    a.ld_d_block = a.ld_d_residual = H;
    a.d_gate = ptr(d_gate);
    a.d_scale = ptr(d_scale);
    a.d_w_post = ptr(d_w_post);
    a.d_w_next = ptr(d_w_next);
    a.workspace = ws.data_ptr();
    a.workspace_bytes = need;
    check(gemm_norm_residual_backward(&a, stream_of(dev)));
    return tuple({d_block, d_residual, d_gate, d_scale, d_w_post, d_w_next});
    END_HANDLE_TH_ERRORS
}

PyMethodDef methods[] = {FAST("quantize", quantize), FAST("dequantize", dequantize), FAST("linear", linear),
                         FAST("linear_backward", linear_backward), FAST("moe", moe), FAST("norm", norm),
                         FAST("norm_backward", norm_backward), {"set_check", set_check, METH_O, nullptr},
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_block", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__block() { return PyModule_Create(&module); }
