// extern "C" entry points of the dense operators (declared in
// include/rvqmoe.h): argument checks, workspace layout, kernel dispatch.
// Host code only.
#include <math.h>

#include "arg_check.cuh"

using namespace rvq;

namespace {

bool dense_shape(int32_t n, int32_t rows, int32_t cols) {
    return n >= 1 && rows >= 8 && cols >= 8 && rows % 8 == 0 && cols % 8 == 0 && n <= kMaxDim &&
           rows <= kMaxDim && cols <= kMaxDim;
}

rvq_status check_dense_shape(const char *who, int32_t n, int32_t rows, int32_t cols, int act,
                             rvq_dtype dt) {
    CHECK_ARG(dense_shape(n, rows, cols),
              "%s: n %d, rows %d, cols %d (n >= 1; rows and cols multiples of 8)", who, n, rows,
              cols);
    CHECK_ARG(act >= MOE_ACT_NONE && act <= MOE_ACT_GELU_TANH, "%s: activation %d", who, act);
    CHECK_ARG(dtype16(dt), "%s: dtype %d (bf16 or fp16)", who, (int)dt);
    return RVQ_OK;
}

// Workspace: status | partial sums of split products | and for a gradient dp
// 16-bit [mats][n][rows] | bias partials.  The calls' products run one after
// another and share the partial sums' place.
struct WsPlan {
    size_t off_partial, off_dp, off_part, total;
};

DenseJob product_of(int mode, int32_t M, int32_t N, int32_t K, int a_t, int b_t) {
    DenseJob j = {};
    j.mode = mode;
    j.M = M;
    j.N = N;
    j.K = K;
    j.a_t = a_t;
    j.b_t = b_t;
    return j;
}

// The products of a call, by their sizes: the forward's, or dx and dw.
DenseJob forward_product(int mats, int32_t n, int32_t rows, int32_t cols) {
    return product_of(mats == 2 ? DG_GATED : DG_PLAIN, n, rows, cols, 0, 0);
}
DenseJob dx_product(int mats, int32_t n, int32_t rows, int32_t cols) {
    return product_of(mats == 2 ? DG_SUM_K : DG_PLAIN, n, cols, rows, 0, 1);
}
DenseJob dw_product(int mats, int32_t n, int32_t rows, int32_t cols) {
    return product_of(mats == 2 ? DG_PAIR_M : DG_PLAIN, rows, cols, n, 1, 1);
}

WsPlan plan_ws(int mats, int32_t n, int32_t rows, int32_t cols, bool backward) {
    WsPlan P = {};
    P.off_partial = RVQ_WS_STATUS_BYTES;
    if (!backward) {
        P.total = up256(P.off_partial +
                        dense_gemm_partial_bytes(forward_product(mats, n, rows, cols)));
        return P;
    }
    const size_t dx = dense_gemm_partial_bytes(dx_product(mats, n, rows, cols));
    const size_t dw = dense_gemm_partial_bytes(dw_product(mats, n, rows, cols));
    P.off_dp = up256(P.off_partial + (dx > dw ? dx : dw));
    P.off_part = up256(P.off_dp + (size_t)mats * n * rows * 2);
    P.total = up256(P.off_part + (size_t)dense_bwd_chunks(n) * mats * rows * 4);
    return P;
}

// a gradient's workspace serves the forward call too
size_t ws_bytes_of(int mats, int32_t n, int32_t rows, int32_t cols, int32_t backward) {
    if (!dense_shape(n, rows, cols)) return 0;
    const size_t f = plan_ws(mats, n, rows, cols, false).total;
    const size_t b = backward ? plan_ws(mats, n, rows, cols, true).total : 0;
    return f > b ? f : b;
}

}  // namespace

extern "C" {

size_t moe_linear_workspace_bytes(int32_t n, int32_t rows, int32_t cols, int32_t backward) {
    return ws_bytes_of(1, n, rows, cols, backward);
}

size_t moe_gated_linear_workspace_bytes(int32_t n, int32_t rows, int32_t cols, int32_t backward) {
    return ws_bytes_of(2, n, rows, cols, backward);
}

rvq_status moe_linear(const void *x_dev, int64_t ldx, const void *w_dev, int64_t ldw,
                      const void *bias_dev, rvq_dtype dt, int32_t n, int32_t rows, int32_t cols,
                      moe_act act, float alpha, const void *residual_dev, rvq_dtype rdt,
                      int64_t ldr, void *out_dev, rvq_dtype odt, int64_t ldo, float *pre_dev,
                      void *ws_dev, size_t ws_bytes, rvq_stream_t stream) {
    const char *who = "moe_linear";
    RVQ_TRY(check_dense_shape(who, n, rows, cols, (int)act, dt));
    RVQ_TRY(check_matrix(who, "x", x_dev, ldx, cols));
    RVQ_TRY(check_matrix(who, "w", w_dev, ldw, cols));
    CHECK_ARG(dtype_any(odt), "%s: out dtype %d", who, (int)odt);
    RVQ_TRY(check_matrix(who, "out", out_dev, ldo, rows));
    if (residual_dev) {
        CHECK_ARG(dtype_any(rdt), "%s: residual dtype %d", who, (int)rdt);
        RVQ_TRY(check_matrix(who, "residual", residual_dev, ldr, rows));
    }
    CHECK_ALIGN(bias_dev, who, "bias");
    CHECK_ALIGN(pre_dev, who, "pre");
    const size_t oe = elem_bytes(odt);
    const Span o = {out_dev, ldo, n, rows, oe}, pre = {pre_dev, rows, n, rows, 4};
    const Span in[] = {{x_dev, ldx, n, cols, 2}, {w_dev, ldw, rows, cols, 2},
                       vector(bias_dev, rows, 2)};
    const Span res = {residual_dev, ldr, n, rows, elem_bytes(rdt)};
    CHECK_ARG(all_apart({o, pre}, in) && apart(pre, res), "%s: out or pre overlaps another matrix",
              who);
    CHECK_ARG((residual_dev == out_dev && rdt == odt && ldr == ldo) ||
                  apart(o, res),
              "%s: out overlaps the residual with another type, place or pitch", who);
    RVQ_TRY(check_ws(who, ws_dev, ws_bytes, ws_bytes_of(1, n, rows, cols, 0)));
    DenseJob j = {};
    j.mode = DG_PLAIN;
    j.M = n;
    j.N = rows;
    j.K = cols;
    j.a[0] = x_dev;
    j.lda = ldx;
    j.b[0] = w_dev;
    j.ldb = ldw;
    j.dt = (int)dt;
    j.bias[0] = bias_dev;
    j.act = (int)act;
    j.alpha = alpha;
    j.residual = residual_dev;
    j.rdt = (int)rdt;
    j.ldr = ldr;
    j.out[0] = out_dev;
    j.odt = (int)odt;
    j.ldo = ldo;
    j.pre[0] = pre_dev;
    j.status = (uint32_t *)ws_dev;
    j.partial = (float *)((uint8_t *)ws_dev + RVQ_WS_STATUS_BYTES);
    return launch_dense_gemm(j, (cudaStream_t)stream);
}

rvq_status moe_gated_linear(const void *x_dev, int64_t ldx, const void *wg_dev,
                            const void *wu_dev, int64_t ldw, const void *bg_dev,
                            const void *bu_dev, rvq_dtype dt, int32_t n, int32_t rows,
                            int32_t cols, moe_act act, void *out_dev, int64_t ldo, float *pre_dev,
                            void *ws_dev, size_t ws_bytes, rvq_stream_t stream) {
    const char *who = "moe_gated_linear";
    RVQ_TRY(check_dense_shape(who, n, rows, cols, (int)act, dt));
    RVQ_TRY(check_matrix(who, "x", x_dev, ldx, cols));
    RVQ_TRY(check_matrix(who, "wg", wg_dev, ldw, cols));
    RVQ_TRY(check_matrix(who, "wu", wu_dev, ldw, cols));
    RVQ_TRY(check_matrix(who, "out", out_dev, ldo, rows));
    CHECK_ALIGN(bg_dev, who, "bg");
    CHECK_ALIGN(bu_dev, who, "bu");
    CHECK_ALIGN(pre_dev, who, "pre");
    const Span out[] = {{out_dev, ldo, n, rows, 2}, {pre_dev, rows, n, rows, 4},
                        {pre_dev ? pre_dev + (size_t)n * rows : nullptr, rows, n, rows, 4}};
    const Span in[] = {{x_dev, ldx, n, cols, 2}, {wg_dev, ldw, rows, cols, 2},
                       {wu_dev, ldw, rows, cols, 2}, vector(bg_dev, rows, 2),
                       vector(bu_dev, rows, 2)};
    CHECK_ARG(all_apart(out, in), "%s: out or pre overlaps another matrix", who);
    RVQ_TRY(check_ws(who, ws_dev, ws_bytes, ws_bytes_of(2, n, rows, cols, 0)));
    DenseJob j = {};
    j.mode = DG_GATED;
    j.M = n;
    j.N = rows;
    j.K = cols;
    j.a[0] = x_dev;
    j.lda = ldx;
    j.b[0] = wg_dev;
    j.b[1] = wu_dev;
    j.ldb = ldw;
    j.dt = (int)dt;
    j.bias[0] = bg_dev;
    j.bias[1] = bu_dev;
    j.act = (int)act;
    j.alpha = 1.f;
    j.out[0] = out_dev;
    j.odt = (int)dt;
    j.ldo = ldo;
    j.pre[0] = pre_dev;
    j.pre[1] = pre_dev ? pre_dev + (size_t)n * rows : nullptr;
    j.status = (uint32_t *)ws_dev;
    j.partial = (float *)((uint8_t *)ws_dev + RVQ_WS_STATUS_BYTES);
    return launch_dense_gemm(j, (cudaStream_t)stream);
}

rvq_status moe_linear_backward(const void *dout_dev, int64_t lddo, const void *x_dev, int64_t ldx,
                               const void *w_dev, int64_t ldw, const float *pre_dev, rvq_dtype dt,
                               int32_t n, int32_t rows, int32_t cols, moe_act act, float alpha,
                               void *dx_dev, int64_t lddx, void *dw_dev, int64_t lddw,
                               void *dbias_dev, void *ws_dev, size_t ws_bytes,
                               rvq_stream_t stream) {
    const char *who = "moe_linear_backward";
    RVQ_TRY(check_dense_shape(who, n, rows, cols, (int)act, dt));
    RVQ_TRY(check_matrix(who, "dout", dout_dev, lddo, rows));
    CHECK_ARG(dx_dev || dw_dev || dbias_dev, "%s: no gradient is wanted", who);
    CHECK_ARG(act == MOE_ACT_NONE || pre_dev, "%s: activation %d needs pre", who, (int)act);
    if (dx_dev) {
        RVQ_TRY(check_matrix(who, "w", w_dev, ldw, cols));
        RVQ_TRY(check_matrix(who, "dx", dx_dev, lddx, cols));
    }
    if (dw_dev) {
        RVQ_TRY(check_matrix(who, "x", x_dev, ldx, cols));
        RVQ_TRY(check_matrix(who, "dw", dw_dev, lddw, cols));
    }
    CHECK_ALIGN(dbias_dev, who, "dbias");
    CHECK_ALIGN(pre_dev, who, "pre");
    // The products of dx and dw may run in one launch, the bias sums beside either.
    const Span out[] = {{dx_dev, lddx, n, cols, 2}, {dw_dev, lddw, rows, cols, 2},
                        vector(dbias_dev, rows, 2)};
    const Span in[] = {{dx_dev || dw_dev ? dout_dev : nullptr, lddo, n, rows, 2},
                       {dx_dev ? w_dev : nullptr, ldw, rows, cols, 2},
                       {dw_dev ? x_dev : nullptr, ldx, n, cols, 2}};
    CHECK_ARG(all_apart(out, in), "%s: a gradient overlaps an input or another gradient", who);
    RVQ_TRY(check_ws(who, ws_dev, ws_bytes, ws_bytes_of(1, n, rows, cols, 1)));
    const WsPlan P = plan_ws(1, n, rows, cols, true);
    uint8_t *ws = (uint8_t *)ws_dev;
    cudaStream_t st = (cudaStream_t)stream;
    // without an activation the products read dout itself (alpha goes into
    // their epilogues), so nothing is rounded on the way
    const bool direct = act == MOE_ACT_NONE;
    BiasSums sums = {};
    if (!direct || dbias_dev) {
        DenseBwdJob b = {};
        b.mats = 1;
        b.n = n;
        b.rows = rows;
        b.act = (int)act;
        b.alpha = alpha;
        b.dout = dout_dev;
        b.ldd = lddo;
        b.dt = (int)dt;
        b.pre[0] = direct ? nullptr : pre_dev;
        b.dp[0] = (direct || !(dx_dev || dw_dev)) ? nullptr : ws + P.off_dp;
        b.dbias[0] = dbias_dev;
        b.part = (float *)(ws + P.off_part);
        RVQ_TRY(launch_dense_bwd(b, st));
        sums = bias_sums_of(b);
    }
    DenseJob j = {};
    j.mode = DG_PLAIN;
    j.dt = (int)dt;
    j.alpha = direct ? alpha : 1.f;
    j.odt = (int)dt;
    j.a[0] = direct ? dout_dev : ws + P.off_dp;
    j.lda = direct ? lddo : rows;
    j.status = (uint32_t *)ws_dev;
    j.partial = (float *)(ws + P.off_partial);
    j.b_t = 1;
    // dx: [n][rows] x [rows][cols]; dw: [n][rows]^T x [n][cols]
    DenseJob w = j;
    j.M = n;
    j.N = cols;
    j.K = rows;
    j.b[0] = w_dev;
    j.ldb = ldw;
    j.out[0] = dx_dev;
    j.ldo = lddx;
    w.a_t = 1;
    w.M = rows;
    w.N = cols;
    w.K = n;
    w.b[0] = x_dev;
    w.ldb = ldx;
    w.out[0] = dw_dev;
    w.ldo = lddw;
    return launch_dense_gemm_two(j, w, sums, st);
}

rvq_status moe_gated_linear_backward(const void *dout_dev, int64_t lddo, const void *x_dev,
                                     int64_t ldx, const void *wg_dev, const void *wu_dev,
                                     int64_t ldw, const float *pre_dev, rvq_dtype dt, int32_t n,
                                     int32_t rows, int32_t cols, moe_act act, void *dx_dev,
                                     int64_t lddx, void *dwg_dev, void *dwu_dev, int64_t lddw,
                                     void *dbg_dev, void *dbu_dev, void *ws_dev, size_t ws_bytes,
                                     rvq_stream_t stream) {
    const char *who = "moe_gated_linear_backward";
    RVQ_TRY(check_dense_shape(who, n, rows, cols, (int)act, dt));
    RVQ_TRY(check_matrix(who, "dout", dout_dev, lddo, rows));
    CHECK_ARG(dx_dev || dwg_dev || dbg_dev || dbu_dev, "%s: no gradient is wanted", who);
    CHECK_ARG((dwg_dev == nullptr) == (dwu_dev == nullptr), "%s: dwg and dwu go together", who);
    CHECK_ARG(pre_dev, "%s: null pre", who);
    CHECK_ALIGN(pre_dev, who, "pre");
    CHECK_ALIGN(dbg_dev, who, "dbg");
    CHECK_ALIGN(dbu_dev, who, "dbu");
    if (dx_dev) {
        RVQ_TRY(check_matrix(who, "wg", wg_dev, ldw, cols));
        RVQ_TRY(check_matrix(who, "wu", wu_dev, ldw, cols));
        RVQ_TRY(check_matrix(who, "dx", dx_dev, lddx, cols));
    }
    if (dwg_dev) {
        RVQ_TRY(check_matrix(who, "x", x_dev, ldx, cols));
        RVQ_TRY(check_matrix(who, "dwg", dwg_dev, lddw, cols));
        RVQ_TRY(check_matrix(who, "dwu", dwu_dev, lddw, cols));
    }
    // As in moe_linear_backward; dout is read before the products.
    const Span out[] = {{dx_dev, lddx, n, cols, 2}, {dwg_dev, lddw, rows, cols, 2},
                        {dwu_dev, lddw, rows, cols, 2}, vector(dbg_dev, rows, 2),
                        vector(dbu_dev, rows, 2)};
    const Span in[] = {{dx_dev ? wg_dev : nullptr, ldw, rows, cols, 2},
                       {dx_dev ? wu_dev : nullptr, ldw, rows, cols, 2},
                       {dwg_dev ? x_dev : nullptr, ldx, n, cols, 2}};
    CHECK_ARG(all_apart(out, in), "%s: a gradient overlaps an input or another gradient", who);
    RVQ_TRY(check_ws(who, ws_dev, ws_bytes, ws_bytes_of(2, n, rows, cols, 1)));
    const WsPlan P = plan_ws(2, n, rows, cols, true);
    uint8_t *ws = (uint8_t *)ws_dev;
    cudaStream_t st = (cudaStream_t)stream;
    const size_t plane = (size_t)n * rows;
    const bool products = dx_dev || dwg_dev;
    DenseBwdJob b = {};
    b.mats = 2;
    b.n = n;
    b.rows = rows;
    b.act = (int)act;
    b.alpha = 1.f;
    b.dout = dout_dev;
    b.ldd = lddo;
    b.dt = (int)dt;
    b.pre[0] = pre_dev;
    b.pre[1] = pre_dev + plane;
    b.dp[0] = products ? ws + P.off_dp : nullptr;
    b.dp[1] = products ? ws + P.off_dp + plane * 2 : nullptr;
    b.dbias[0] = dbg_dev;
    b.dbias[1] = dbu_dev;
    b.part = (float *)(ws + P.off_part);
    RVQ_TRY(launch_dense_bwd(b, st));
    DenseJob j = {};
    j.dt = (int)dt;
    j.alpha = 1.f;
    j.odt = (int)dt;
    j.a[0] = b.dp[0];
    j.a[1] = b.dp[1];
    j.lda = rows;
    j.b_t = 1;
    j.status = (uint32_t *)ws_dev;
    j.partial = (float *)(ws + P.off_partial);
    DenseJob w = j;
    j.mode = DG_SUM_K;
    j.M = n;
    j.N = cols;
    j.K = rows;
    j.b[0] = wg_dev;
    j.b[1] = wu_dev;
    j.ldb = ldw;
    j.out[0] = dx_dev;
    j.ldo = lddx;
    w.mode = DG_PAIR_M;
    w.a_t = 1;
    w.M = rows;
    w.N = cols;
    w.K = n;
    w.b[0] = x_dev;
    w.ldb = ldx;
    w.out[0] = dwg_dev;
    w.out[1] = dwu_dev;
    w.ldo = lddw;
    return launch_dense_gemm_two(j, w, bias_sums_of(b), st);
}

rvq_status rvq_selftest_dense_plan(int32_t gated, int32_t backward, int32_t n, int32_t rows,
                                   int32_t cols, int32_t out[7]) {
    const char *who = "rvq_selftest_dense_plan";
    CHECK_ARG(dense_shape(n, rows, cols) && out, "%s: n %d, rows %d, cols %d, out %p", who, n, rows,
              cols, (void *)out);
    const int mats = gated ? 2 : 1;
    int32_t plan[7];
    if (backward) {
        const DenseJob dw = dw_product(mats, n, rows, cols);
        dense_plan_of(dx_product(mats, n, rows, cols), &dw, plan);
    } else {
        dense_plan_of(forward_product(mats, n, rows, cols), nullptr, plan);
    }
    for (int i = 0; i < 7; ++i) out[i] = plan[i];
    return RVQ_OK;
}

// ---------------------------------------------------------------- norm join

rvq_status moe_norm_join(const void *h_dev, rvq_dtype hdt, const void *y_dev, rvq_dtype ydt,
                         int32_t n, int32_t d, float alpha, const void *gate_dev,
                         moe_gate gate_kind, rvq_dtype gdt, int32_t post_norm,
                         const void *w_post_dev, const void *w_pre_dev, rvq_dtype wdt, float eps,
                         void *h_out_dev, void *xn_dev, rvq_dtype xdt, float *rstd_dev,
                         rvq_stream_t stream) {
    const char *who = "moe_norm_join";
    RVQ_TRY(check_join(who, h_dev, hdt, y_dev, ydt, n, d, gate_dev, (int)gate_kind, gdt, post_norm,
                       w_post_dev, w_pre_dev, wdt, xdt));
    CHECK_ARG(eps >= 0.f && isfinite(eps), "%s: eps %g", who, (double)eps);
    CHECK_ARG(h_out_dev || xn_dev, "%s: neither h_out nor xn is wanted", who);
    CHECK_ALIGN(h_out_dev, who, "h_out");
    CHECK_ALIGN(xn_dev, who, "xn");
    CHECK_ALIGN(rstd_dev, who, "rstd");
    const JoinSpan in[] = {{h_dev, hdt, n, d}, {y_dev, ydt, n, d},
                           gate_span(gate_dev, gdt, (int)gate_kind, n, d),
                           {w_post_dev, wdt, 1, d}, {w_pre_dev, wdt, 1, d}};
    CHECK_ARG(join_outputs_ok(in, {h_out_dev, hdt, n, d}, {xn_dev, xdt, n, d},
                              {rstd_dev, RVQ_F32, 2, n}),
              "%s: an output overlaps an input of another type or place, or another output", who);
    JoinJob j = {};
    j.n = n;
    j.d = d;
    j.eps = eps;
    j.alpha = alpha;
    j.h = h_dev;
    j.hdt = (int)hdt;
    j.y = y_dev;
    j.ydt = (int)ydt;
    j.gate = gate_dev;
    j.gate_kind = (int)gate_kind;
    j.gdt = (int)gdt;
    j.post_norm = post_norm != 0;
    j.w_post = w_post_dev;
    j.w_pre = w_pre_dev;
    j.wdt = (int)wdt;
    j.h_out = h_out_dev;
    j.xn = xn_dev;
    j.xdt = (int)xdt;
    j.rstd = rstd_dev;
    return launch_norm_join(j, (cudaStream_t)stream);
}

static size_t join_part_bytes(int32_t n, int32_t d) {
    return (size_t)join_bwd_slots(n, d) * ((size_t)3 * d + 1) * 4;
}

size_t moe_norm_join_workspace_bytes(int32_t n, int32_t d) {
    if (n < 1 || n > kMaxDim || d < 8 || d % 8 != 0 || d > kJoinMaxD) return 0;
    return up256(RVQ_WS_STATUS_BYTES + join_part_bytes(n, d));
}

rvq_status moe_norm_join_backward(const void *dh_out_dev, const void *dxn_dev, rvq_dtype xdt,
                                  const void *h_dev, rvq_dtype hdt, const void *y_dev,
                                  rvq_dtype ydt, int32_t n, int32_t d, float alpha,
                                  const void *gate_dev, moe_gate gate_kind, rvq_dtype gdt,
                                  int32_t post_norm, const void *w_post_dev,
                                  const void *w_pre_dev, rvq_dtype wdt, const float *rstd_dev,
                                  void *dh_dev, void *dy_dev, void *dgate_dev, void *dw_post_dev,
                                  void *dw_pre_dev, void *ws_dev, size_t ws_bytes,
                                  rvq_stream_t stream) {
    const char *who = "moe_norm_join_backward";
    RVQ_TRY(check_join(who, h_dev, hdt, y_dev, ydt, n, d, gate_dev, (int)gate_kind, gdt, post_norm,
                       w_post_dev, w_pre_dev, wdt, xdt));
    CHECK_ARG(dh_out_dev || dxn_dev, "%s: neither dh_out nor dxn is given", who);
    CHECK_ARG(dh_dev || dy_dev || dgate_dev || dw_post_dev || dw_pre_dev,
              "%s: no gradient is wanted", who);
    CHECK_ARG(rstd_dev, "%s: null rstd", who);
    CHECK_ARG(!dgate_dev || gate_dev, "%s: dgate without a gate", who);
    CHECK_ARG(!dh_dev || h_dev, "%s: dh without h", who);
    CHECK_ARG(!dw_post_dev || post_norm, "%s: dw_post without post_norm", who);
    CHECK_ARG(!dw_pre_dev || dxn_dev, "%s: dw_pre without dxn", who);
    const void *al[] = {dh_out_dev, dxn_dev, rstd_dev, dh_dev, dy_dev, dgate_dev, dw_post_dev,
                        dw_pre_dev};
    static const char *const names[] = {"dh_out", "dxn", "rstd", "dh", "dy", "dgate", "dw_post",
                                        "dw_pre"};
    for (int i = 0; i < 8; ++i) CHECK_ALIGN(al[i], who, names[i]);
    // dgate per row and dh, dy are written while other blocks read their rows; the
    // gains' and the other gates' gradients after the last row.
    const JoinSpan gate = gate_span(gate_dev, gdt, (int)gate_kind, n, d);
    const JoinSpan out[] = {{dh_dev, hdt, n, d}, {dy_dev, ydt, n, d},
                            gate_span(dgate_dev, gdt, (int)gate_kind, n, d),
                            {dw_post_dev, wdt, 1, d}, {dw_pre_dev, wdt, 1, d}};
    const JoinSpan in[] = {{h_dev, hdt, n, d}, {y_dev, ydt, n, d}, gate, {dh_out_dev, hdt, n, d},
                           {dxn_dev, xdt, n, d}, {rstd_dev, RVQ_F32, 2, n},
                           {w_post_dev, wdt, 1, d}, {w_pre_dev, wdt, 1, d}};
    const bool gate_rows = gate_kind == MOE_GATE_TOKEN || gate_kind == MOE_GATE_FULL;
    bool ok = true;
    for (int o = 0; o < 5; ++o) {
        for (int i = 0; i < o; ++i) ok = ok && apart(out[o], out[i]);
        if (o > 2 || (o == 2 && !gate_rows)) continue;
        for (int i = 0; i < 8; ++i) ok = ok && (i < 5 ? same_or_apart(out[o], in[i])
                                                      : apart(out[o], in[i]));
    }
    CHECK_ARG(ok, "%s: a gradient overlaps an input of another type or place, or another gradient",
              who);
    RVQ_TRY(check_ws(who, ws_dev, ws_bytes, moe_norm_join_workspace_bytes(n, d)));
    JoinJob j = {};
    j.n = n;
    j.d = d;
    j.alpha = alpha;
    j.h = h_dev;
    j.hdt = (int)hdt;
    j.y = y_dev;
    j.ydt = (int)ydt;
    j.gate = gate_dev;
    j.gate_kind = (int)gate_kind;
    j.gdt = (int)gdt;
    j.post_norm = post_norm != 0;
    j.w_post = w_post_dev;
    j.w_pre = w_pre_dev;
    j.wdt = (int)wdt;
    j.xdt = (int)xdt;
    j.rstd = const_cast<float *>(rstd_dev);
    j.dh_out = dh_out_dev;
    j.dxn = dxn_dev;
    j.dh = dh_dev;
    j.dy = dy_dev;
    j.dgate = dgate_dev;
    j.dw_post = dw_post_dev;
    j.dw_pre = dw_pre_dev;
    j.part = (float *)((uint8_t *)ws_dev + RVQ_WS_STATUS_BYTES);
    j.slots = join_bwd_slots(n, d);
    return launch_norm_join_bwd(j, (cudaStream_t)stream);
}

}  // extern "C"
