// block_api.cpp -- the C ABI declared in include/gemm_block.h: argument checks,
// workspace layouts and launches of the feed-forward block's operators. Every
// check is made before anything is enqueued.
#include "block.hpp"

using namespace mg;

namespace {

bool is_float(gemm_dtype t) { return t == GEMM_F32 || t == GEMM_F16 || t == GEMM_BF16; }
int64_t size_of(gemm_dtype t) { return t == GEMM_F32 ? 4 : 2; }
int64_t align16(int64_t n) { return (n + 15) / 16 * 16; }
bool misaligned(const void *p, unsigned n) { return reinterpret_cast<uintptr_t>(p) % n != 0; }
long long ll(int64_t v) { return (long long)v; }

constexpr int64_t kMaxDim = 1LL << 31;   // rows and columns stay below
constexpr int64_t kMaxElems = 1LL << 46;

gemm_status launched(hipError_t e, const char *what) {
    if (e == hipSuccess) return api_ok();
    return api_fail(GEMM_HIP_ERROR, "%s: launch failed: %s (%d)", what, hipGetErrorString(e), (int)e);
}

// A matrix argument: sizes, leading dimension, pointer (needed unless empty).
gemm_status check_matrix(const char *what, const char *name, const void *p, gemm_dtype type,
                         int64_t rows, int64_t cols, int64_t ld) {
    if (!is_float(type))
        return api_fail(GEMM_UNSUPPORTED, "%s: %s must be F32, F16 or BF16", what, name);
    if (rows < 0 || cols < 0)
        return api_fail(GEMM_INVALID_ARG, "%s: negative size %lld x %lld of %s", what, ll(rows),
                        ll(cols), name);
    if (rows >= kMaxDim || cols >= kMaxDim)
        return api_fail(GEMM_UNSUPPORTED, "%s: %s has a dimension of 2^31 or more", what, name);
    if (rows == 0 || cols == 0) return GEMM_OK;
    if (!p) return api_fail(GEMM_INVALID_ARG, "%s: %s is NULL", what, name);
    if (rows > 1 && ld < cols)
        return api_fail(GEMM_INVALID_ARG, "%s: leading dimension %lld of %s is below its %lld columns",
                        what, ll(ld), name, ll(cols));
    if (ld > kMaxElems / rows)
        return api_fail(GEMM_UNSUPPORTED, "%s: %s spans more than 2^46 elements", what, name);
    if (misaligned(p, (unsigned)size_of(type)))
        return api_fail(GEMM_INVALID_ARG, "%s: %s is not aligned to its element", what, name);
    return GEMM_OK;
}

gemm_status check_vector(const char *what, const char *name, const void *p, gemm_dtype type) {
    if (p && misaligned(p, (unsigned)size_of(type)))
        return api_fail(GEMM_INVALID_ARG, "%s: %s is not aligned to its element", what, name);
    return GEMM_OK;
}

// A packed MXFP4 matrix (needed unless empty).
gemm_status check_mx4(const char *what, const char *name, const uint8_t *codes,
                      const uint8_t *scales, int64_t rows, int64_t k) {
    if (rows == 0 || k == 0) return GEMM_OK;
    if (!codes || !scales)
        return api_fail(GEMM_INVALID_ARG, "%s: codes or scales of %s are NULL", what, name);
    if (misaligned(codes, 16) || misaligned(scales, 8))
        return api_fail(GEMM_INVALID_ARG, "%s: %s needs 16-byte aligned codes and 8-byte aligned scales",
                        what, name);
    return GEMM_OK;
}

gemm_status check_workspace(const char *what, const void *p, int64_t have, int64_t need) {
    if (need <= 0) return GEMM_OK;
    if (!p || have < need)
        return api_fail(GEMM_INVALID_ARG, "%s: workspace of %lld bytes, needs %lld", what,
                        p ? ll(have) : 0LL, ll(need));
    if (misaligned(p, 16))
        return api_fail(GEMM_INVALID_ARG, "%s: workspace is not 16-byte aligned", what);
    return GEMM_OK;
}

gemm_status check_plan(const char *what, gemm_plan_t plan, PlanInfo *pi) {
    if (!plan_info(plan, pi)) return api_fail(GEMM_NOT_INITIALIZED, "%s: invalid plan handle", what);
    if (!pi->mxf4_tn)
        return api_fail(GEMM_UNSUPPORTED, "%s: needs an F4_E2M1 plan with A RowMajor, B ColumnMajor "
                        "and C RowMajor", what);
    return GEMM_OK;
}

int64_t codes_bytes(int64_t rows, int64_t k) { return rows * (mx4_kp(k) / 2); }
int64_t scales_bytes(int64_t rows, int64_t k) { return rows * (mx4_kp(k) / 32); }
int64_t mx4_bytes(int64_t rows, int64_t k) {
    return align16(codes_bytes(rows, k)) + align16(scales_bytes(rows, k));
}

#define CHECK(expr)                          \
    do {                                     \
        const gemm_status st_ = (expr);      \
        if (st_ != GEMM_OK) return st_;      \
    } while (0)

// A packed matrix's place in a workspace.
struct Packed {
    uint8_t *codes, *scales;
};
Packed carve(char *&p, int64_t rows, int64_t k) {
    Packed q;
    q.codes = reinterpret_cast<uint8_t *>(p);
    q.scales = q.codes + align16(codes_bytes(rows, k));
    p += mx4_bytes(rows, k);
    return q;
}

}  // namespace

extern "C" {

int64_t gemm_mx4_padded(int64_t k) { return k > 0 ? mx4_kp(k) : 0; }

gemm_status gemm_mx4_quantize(const void *x, gemm_dtype x_type, int64_t rows, int64_t cols,
                              int64_t ld, uint8_t *row_codes, uint8_t *row_scales,
                              uint8_t *col_codes, uint8_t *col_scales, void *stream) {
    const char *what = "gemm_mx4_quantize";
    CHECK(check_matrix(what, "x", x, x_type, rows, cols, ld));
    if (!row_codes != !row_scales || !col_codes != !col_scales)
        return api_fail(GEMM_INVALID_ARG, "%s: codes and scales go together", what);
    if (rows == 0 || cols == 0) return api_ok();
    if (!row_codes && !col_codes)
        return api_fail(GEMM_INVALID_ARG, "%s: neither direction is asked for", what);
    if (row_codes) CHECK(check_mx4(what, "the row form", row_codes, row_scales, rows, cols));
    if (col_codes) CHECK(check_mx4(what, "the column form", col_codes, col_scales, cols, rows));
    return launched(launch_mx4_quantize(x_type,
                                        {x, rows, cols, ld, row_codes, row_scales, col_codes, col_scales},
                                        nullptr, static_cast<hipStream_t>(stream)),
                    what);
}

gemm_status gemm_mx4_dequantize(const uint8_t *codes, const uint8_t *scales, int64_t rows,
                                int64_t k, void *out, gemm_dtype out_type, int64_t ld,
                                void *stream) {
    const char *what = "gemm_mx4_dequantize";
    CHECK(check_matrix(what, "out", out, out_type, rows, k, ld));
    CHECK(check_mx4(what, "the matrix", codes, scales, rows, k));
    if (rows == 0 || k == 0) return api_ok();
    return launched(launch_mx4_dequantize(codes, scales, rows, k, out, out_type, ld,
                                          static_cast<hipStream_t>(stream)),
                    what);
}

int64_t gemm_mx4_linear_workspace(int64_t M, int64_t K) {
    return M > 0 && K > 0 && !mx4_in_kernel(M, K) ? mx4_bytes(M, K) : 0;
}

gemm_status gemm_mx4_linear(gemm_plan_t plan, const void *x, gemm_dtype x_type, int64_t ldx,
                            const uint8_t *w_codes, const uint8_t *w_scales, const void *bias,
                            void *y, int64_t M, int64_t N, int64_t K, void *workspace,
                            int64_t workspace_bytes, void *stream) {
    const char *what = "gemm_mx4_linear";
    PlanInfo pi;
    CHECK(check_plan(what, plan, &pi));
    CHECK(check_matrix(what, "x", x, x_type, M, K, ldx));
    CHECK(check_matrix(what, "y", y, GEMM_BF16, M, N, N));
    CHECK(check_mx4(what, "the weight", w_codes, w_scales, N, K));
    CHECK(check_vector(what, "bias", bias, GEMM_BF16));
    if (M == 0 || N == 0) return api_ok();
    CHECK(check_workspace(what, workspace, workspace_bytes, gemm_mx4_linear_workspace(M, K)));
    CHECK(plan_on_device(plan));
    const hipStream_t st = static_cast<hipStream_t>(stream);
    Packed q = {nullptr, nullptr};
    if (K > 0 && !mx4_in_kernel(M, K)) {
        char *p = static_cast<char *>(workspace);
        q = carve(p, M, K);
        CHECK(launched(launch_mx4_quantize(x_type, {x, M, K, ldx, q.codes, q.scales, nullptr, nullptr}, nullptr, st),
                       what));
    }
    if (K > 0 && mx4_is_few(M, K))
        return launched(launch_mx4_few(x, x_type, ldx, q.codes, q.scales, w_codes, w_scales, bias, y, M, N, K,
                                       pi.act, st),
                        what);
    return gemm_plan_run_mx(plan, q.codes, w_codes, nullptr, y, bias, M, N, gemm_mx4_padded(K), 1.0f,
                            0.0f, q.scales, w_scales, stream);
}

int64_t gemm_mx4_linear_backward_workspace(int64_t M, int64_t N, int64_t K) {
    if (M <= 0 || N <= 0 || K <= 0) return 0;
    return mx4_bytes(M, N) + mx4_bytes(N, M) + mx4_bytes(K, M);
}

gemm_status gemm_mx4_linear_backward(gemm_plan_t plan, const void *dy, int64_t ld_dy,
                                     const void *x, int64_t ldx, gemm_dtype type,
                                     const uint8_t *wt_codes, const uint8_t *wt_scales, void *dx,
                                     void *dw, int64_t M, int64_t N, int64_t K, void *workspace,
                                     int64_t workspace_bytes, void *stream) {
    const char *what = "gemm_mx4_linear_backward";
    PlanInfo pi;
    CHECK(check_plan(what, plan, &pi));
    if (pi.act != GEMM_EPI_LINEAR)
        return api_fail(GEMM_UNSUPPORTED, "%s: needs a plan with the LINEAR epilogue", what);
    CHECK(check_matrix(what, "dy", dy, type, M, N, ld_dy));
    if (dw) CHECK(check_matrix(what, "x", x, type, M, K, ldx));
    if (M < 0 || N < 0 || K < 0 || K >= kMaxDim)
        return api_fail(GEMM_INVALID_ARG, "%s: bad size M=%lld N=%lld K=%lld", what, ll(M), ll(N), ll(K));
    if (dx) {
        CHECK(check_matrix(what, "dx", dx, GEMM_BF16, M, K, K));
        CHECK(check_mx4(what, "the weight", wt_codes, wt_scales, K, N));
    }
    if (dw) CHECK(check_matrix(what, "dw", dw, GEMM_BF16, N, K, K));
    if (!dx && !dw) return api_ok();
    CHECK(check_workspace(what, workspace, workspace_bytes,
                          gemm_mx4_linear_backward_workspace(M, N, K)));
    CHECK(plan_on_device(plan));
    const hipStream_t st = static_cast<hipStream_t>(stream);
    char *p = static_cast<char *>(workspace);
    Packed rows = {nullptr, nullptr}, cols = rows, xc = rows;
    if (M > 0 && N > 0 && K > 0) {
        rows = carve(p, M, N);
        cols = carve(p, N, M);
        xc = carve(p, K, M);
        const Mx4Quant q = {dy, M, N, ld_dy, dx ? rows.codes : nullptr, dx ? rows.scales : nullptr,
                            dw ? cols.codes : nullptr, dw ? cols.scales : nullptr},
                       qx = {x, M, K, ldx, nullptr, nullptr, xc.codes, xc.scales};
        CHECK(launched(launch_mx4_quantize(type, q, dw ? &qx : nullptr, st), what));
    }
    if (dx && M > 0 && K > 0)
        CHECK(gemm_plan_run_mx(plan, rows.codes, wt_codes, nullptr, dx, nullptr, M, K,
                               gemm_mx4_padded(N), 1.0f, 0.0f, rows.scales, wt_scales, stream));
    if (dw && N > 0 && K > 0)
        CHECK(gemm_plan_run_mx(plan, cols.codes, xc.codes, nullptr, dw, nullptr, N, K,
                               gemm_mx4_padded(M), 1.0f, 0.0f, cols.scales, xc.scales, stream));
    return api_ok();
}

// ---- mixture of experts -------------------------------------------------------------

static gemm_status check_moe(const char *what, const gemm_moe_desc *d, int64_t tokens) {
    if (!d) return api_fail(GEMM_INVALID_ARG, "%s: desc is NULL", what);
    if (d->hidden < 0 || d->inner < 0 || tokens < 0 || d->experts < 1 || d->top_k < 1)
        return api_fail(GEMM_INVALID_ARG, "%s: bad size hidden=%lld inner=%lld tokens=%lld experts=%d "
                        "top_k=%d", what, ll(d->hidden), ll(d->inner), ll(tokens), (int)d->experts,
                        (int)d->top_k);
    if (d->top_k > d->experts)
        return api_fail(GEMM_INVALID_ARG, "%s: top_k = %d of %d experts", what, (int)d->top_k,
                        (int)d->experts);
    if (d->experts > GEMM_MOE_MAX_EXPERTS || d->top_k > GEMM_MOE_MAX_TOP_K)
        return api_fail(GEMM_UNSUPPORTED, "%s: more than %d experts or top_k above %d", what,
                        GEMM_MOE_MAX_EXPERTS, GEMM_MOE_MAX_TOP_K);
    if (tokens > GEMM_MOE_MAX_TOKENS)
        return api_fail(GEMM_UNSUPPORTED, "%s: %lld tokens, at most %d a call%s", what, ll(tokens),
                        GEMM_MOE_MAX_TOKENS, d->weight_type == GEMM_F4_E2M1
                            ? " (more are calls of their own)"
                            : " (many more are grouped_gemm_run's case, or calls of their own)");
    if (d->hidden > GEMM_MOE_MAX_SIZE || d->inner > GEMM_MOE_MAX_SIZE)
        return api_fail(GEMM_UNSUPPORTED, "%s: hidden or inner above %d", what, GEMM_MOE_MAX_SIZE);
    if (d->type != GEMM_F16 && d->type != GEMM_BF16)
        return api_fail(GEMM_UNSUPPORTED, "%s: type must be F16 or BF16", what);
    if (d->weight_type != d->type && !(d->weight_type == GEMM_F4_E2M1 && d->type == GEMM_BF16))
        return api_fail(GEMM_UNSUPPORTED, "%s: weights must have the type of x, or F4_E2M1 with BF16", what);
    return GEMM_OK;
}

int64_t gemm_moe_state_bytes(const gemm_moe_desc *desc) {
    if (check_moe("gemm_moe_state_bytes", desc, 0) != GEMM_OK) return -1;
    return moe_state_bytes(desc->hidden);
}

int64_t gemm_moe_workspace(const gemm_moe_desc *desc, int64_t tokens) {
    if (check_moe("gemm_moe_workspace", desc, tokens) != GEMM_OK) return -1;
    return moe_layout(desc->hidden, desc->inner, desc->experts, desc->top_k, (int)tokens,
                      desc->type == GEMM_F16).total;
}

gemm_status gemm_moe_forward(const gemm_moe_desc *d, const void *x, int64_t ldx,
                             const uint8_t *row_mask, void *out, int64_t ld_out, int32_t *ids,
                             float *probs, int64_t tokens, void *workspace,
                             int64_t workspace_bytes, void *stream) {
    const char *what = "gemm_moe_forward";
    CHECK(check_moe(what, d, tokens));
    CHECK(check_matrix(what, "x", x, d->type, tokens, d->hidden, ldx));
    CHECK(check_matrix(what, "out", out, d->type, tokens, d->hidden, ld_out));
    if (misaligned(ids, 4) || misaligned(probs, 4))
        return api_fail(GEMM_INVALID_ARG, "%s: ids or probs are not 4-byte aligned", what);
    if (tokens == 0) return api_ok();
    if (tokens > 1 && ldx > ((1LL << 31) - 1) / 2 / tokens)
        return api_fail(GEMM_UNSUPPORTED, "%s: x spans 2^31 bytes or more", what);
    if (d->hidden > 0) {
        CHECK(check_matrix(what, "router", d->router, d->type, d->experts, d->hidden, d->hidden));
        if (d->inner > 0) {
            if (d->weight_type == GEMM_F4_E2M1) {
                CHECK(check_mx4(what, "up", static_cast<const uint8_t *>(d->up), d->up_scales,
                                d->experts, d->hidden));
                CHECK(check_mx4(what, "down", static_cast<const uint8_t *>(d->down), d->down_scales,
                                d->experts, d->inner));
            } else {
                CHECK(check_matrix(what, "up", d->up, d->type, 2 * d->inner, d->hidden, d->hidden));
                CHECK(check_matrix(what, "down", d->down, d->type, d->hidden, d->inner, d->inner));
            }
        }
    }
    const int64_t need = gemm_moe_workspace(d, tokens);
    CHECK(check_workspace(what, workspace, workspace_bytes, need));
    MoeArgs a;
    a.H = d->hidden;
    a.I = d->inner;
    a.ldx = ldx;
    a.ldo = ld_out;
    a.T = (int)tokens;
    a.E = d->experts;
    a.k = d->top_k;
    a.renorm = d->renormalize != 0;
    a.x = x;
    a.router = d->router;
    a.up = d->up;
    a.down = d->down;
    a.up_s = d->up_scales;
    a.down_s = d->down_scales;
    a.mask = row_mask;
    a.out = out;
    a.ids = ids;
    a.probs = probs;
    a.ws = static_cast<char *>(workspace);
    return launched(launch_moe(d->type, d->weight_type, a, static_cast<hipStream_t>(stream)), what);
}

// ---- norms ------------------------------------------------------------------------------

static gemm_status check_norm_shape(const char *what, gemm_dtype type, gemm_epilogue act,
                                    int64_t rows, int64_t cols, const void *gate, int64_t gate_rows,
                                    int64_t ld_gate) {
    if (!is_float(type)) return api_fail(GEMM_UNSUPPORTED, "%s: type must be F32, F16 or BF16", what);
    if (rows < 0 || cols < 0)
        return api_fail(GEMM_INVALID_ARG, "%s: negative size %lld x %lld", what, ll(rows), ll(cols));
    if (rows >= kMaxDim) return api_fail(GEMM_UNSUPPORTED, "%s: 2^31 rows or more", what);
    if (cols > GEMM_NORM_MAX_COLS)
        return api_fail(GEMM_UNSUPPORTED, "%s: %lld columns, at most %d", what, ll(cols),
                        GEMM_NORM_MAX_COLS);
    if (act != GEMM_EPI_LINEAR && act != GEMM_EPI_SIGMOID)
        return api_fail(GEMM_UNSUPPORTED, "%s: gate_act must be LINEAR or SIGMOID", what);
    if (gate) {
        if (gate_rows < 0 || (rows > 0 && (gate_rows < 1 || rows % gate_rows != 0)))
            return api_fail(GEMM_INVALID_ARG, "%s: %lld gate rows do not divide %lld rows", what,
                            ll(gate_rows), ll(rows));
        CHECK(check_matrix(what, "gate", gate, type, gate_rows, cols, ld_gate));
    }
    return GEMM_OK;
}

gemm_status gemm_norm_residual(const gemm_norm_args *p, void *stream) {
    const char *what = "gemm_norm_residual";
    if (!p) return api_fail(GEMM_INVALID_ARG, "%s: args is NULL", what);
    gemm_norm_args a = *p;
    CHECK(check_norm_shape(what, a.type, a.gate_act, a.rows, a.cols, a.gate, a.gate_rows, a.ld_gate));
    if (a.rows == 0 || a.cols == 0) return api_ok();   // an empty tensor's pointer may be NULL
    if (!a.block && (a.w_post || a.gate || a.scale))
        return api_fail(GEMM_INVALID_ARG, "%s: w_post, gate and scale belong to a block", what);
    if (!a.block && !a.w_next)
        return api_fail(GEMM_INVALID_ARG, "%s: neither a block nor a next norm", what);
    CHECK(check_matrix(what, "residual", a.residual, a.type, a.rows, a.cols, a.ld_residual));
    if (a.block) {
        CHECK(check_matrix(what, "block", a.block, a.type, a.rows, a.cols, a.ld_block));
        CHECK(check_matrix(what, "out", a.out, a.type, a.rows, a.cols, a.ld_out));
    }
    if (a.w_next) CHECK(check_matrix(what, "next", a.next, a.type, a.rows, a.cols, a.ld_next));
    CHECK(check_vector(what, "w_post", a.w_post, a.type));
    CHECK(check_vector(what, "scale", a.scale, a.type));
    CHECK(check_vector(what, "w_next", a.w_next, a.type));
    if (misaligned(a.rstd_post, 4) || misaligned(a.rstd_next, 4))
        return api_fail(GEMM_INVALID_ARG, "%s: rstd is not 4-byte aligned", what);
    return launched(launch_norm_forward(a, static_cast<hipStream_t>(stream)), what);
}

static gemm_status check_norm_backward(const char *what, const gemm_norm_backward_args *p) {
    if (!p) return api_fail(GEMM_INVALID_ARG, "%s: args is NULL", what);
    const gemm_norm_backward_args &a = *p;
    CHECK(check_norm_shape(what, a.type, a.gate_act, a.rows, a.cols, a.gate, a.gate_rows, a.ld_gate));
    return GEMM_OK;
}

int64_t gemm_norm_backward_workspace(const gemm_norm_backward_args *p) {
    if (check_norm_backward("gemm_norm_backward_workspace", p) != GEMM_OK) return -1;
    const NormCut c = norm_cut(p->rows, p->cols, p->gate ? p->gate_rows : 1);
    return align16(c.parts * (c.chunks > 1 ? 4 : 3) * p->cols * 4);
}

gemm_status gemm_norm_residual_backward(const gemm_norm_backward_args *p, void *stream) {
    const char *what = "gemm_norm_residual_backward";
    CHECK(check_norm_backward(what, p));
    const gemm_norm_backward_args &a = *p;
    if (!a.block && a.rows > 0 && a.cols > 0 && (a.w_post || a.gate || a.scale || a.d_block))
        return api_fail(GEMM_INVALID_ARG, "%s: w_post, gate, scale and d_block belong to a block", what);
    if ((a.d_w_post && !a.w_post) || (a.d_gate && !a.gate) || (a.d_scale && !a.scale) ||
        (a.d_w_next && !a.w_next))
        return api_fail(GEMM_INVALID_ARG, "%s: a gradient of a tensor that is not there", what);
    if (!a.d_next != !a.w_next && a.rows > 0 && a.cols > 0)
        return api_fail(GEMM_INVALID_ARG, "%s: d_next and w_next go together", what);
    if (a.d_out) CHECK(check_matrix(what, "d_out", a.d_out, a.type, a.rows, a.cols, a.ld_d_out));
    CHECK(check_matrix(what, "d_residual", a.d_residual, a.type, a.rows, a.cols, a.ld_d_residual));
    if (a.w_next) {
        CHECK(check_matrix(what, "d_next", a.d_next, a.type, a.rows, a.cols, a.ld_d_next));
        CHECK(check_matrix(what, "out", a.out, a.type, a.rows, a.cols, a.ld_out));
    }
    if (a.block) {
        CHECK(check_matrix(what, "block", a.block, a.type, a.rows, a.cols, a.ld_block));
        CHECK(check_matrix(what, "d_block", a.d_block, a.type, a.rows, a.cols, a.ld_d_block));
    }
    const struct {
        const char *name;
        const void *p;
    } vecs[] = {{"w_post", a.w_post}, {"scale", a.scale}, {"w_next", a.w_next}, {"d_gate", a.d_gate},
                {"d_scale", a.d_scale}, {"d_w_post", a.d_w_post}, {"d_w_next", a.d_w_next}};
    for (const auto &v : vecs) CHECK(check_vector(what, v.name, v.p, a.type));
    if (a.rows > 0 && a.cols > 0 &&
        ((a.w_next && !a.rstd_next) || (a.w_post && !a.rstd_post) || misaligned(a.rstd_next, 4) ||
         misaligned(a.rstd_post, 4)))
        return api_fail(GEMM_INVALID_ARG, "%s: rstd_post or rstd_next is missing or misaligned", what);
    if (a.cols == 0) return api_ok();
    CHECK(check_workspace(what, a.workspace, a.workspace_bytes, gemm_norm_backward_workspace(p)));
    return launched(launch_norm_backward(a, static_cast<hipStream_t>(stream)), what);
}

}  // extern "C"
