// extern "C" entry points of the microscaled operators (declared in
// include/rvqmoe.h): argument checks, kernel dispatch.  Host code only.
#include <math.h>

#include "arg_check.cuh"
#include "mx_tc.cuh"

using namespace rvq;

namespace {

bool mx_shape(int32_t rows, int32_t cols) {
    // 2^31 - 1 words of scales: more than the device's memory holds
    return rows >= 1 && rows <= kMaxDim && cols >= 8 && cols % 8 == 0 && cols <= kMaxDim &&
           (int64_t)rows * mx_tiles(cols) <= 0x7fffffff;
}
bool mx_format(int f) { return f == MOE_MX_F8 || f == MOE_MX_F4; }

size_t code_bytes(int fmt, int32_t rows, int32_t cols) {
    return (size_t)mx_pitch(fmt, cols) * (size_t)rows;
}
size_t scale_bytes(int32_t rows, int32_t cols) {
    return (size_t)mx_tiles(rows) * (size_t)mx_tiles(cols) * kMxTileBytes;
}

rvq_status check_mx_shape(const char *who, int32_t rows, int32_t cols) {
    CHECK_ARG(mx_shape(rows, cols), "%s: %d x %d (at least 1 x 8, columns a multiple of 8)", who,
              rows, cols);
    return RVQ_OK;
}

// A microscaled matrix: not NULL, its codes and scales on 32 bytes (the tensor maps
// of the products need it).
rvq_status check_mx(const char *who, const char *what, const void *codes, const void *scales,
                    int fmt) {
    CHECK_ARG(codes != nullptr && scales != nullptr, "%s: null %s", who, what);
    CHECK_ARG(mx_format(fmt), "%s: format %d of %s", who, fmt, what);
    if ((((uintptr_t)codes | (uintptr_t)scales) & 31u) != 0) {
        set_error("%s: %s: codes %p or scales %p not 32-byte aligned", who, what, codes, scales);
        return RVQ_EALIGN;
    }
    return RVQ_OK;
}

Span codes_of(const void *p, int fmt, int32_t rows, int32_t cols) {
    const int32_t unit = fmt == MOE_MX_F8 ? kMxTile : kMxTile / 2;
    return {p, unit, rows * mx_tiles(cols), unit, 1};
}
Span scales_of(const void *p, int32_t rows, int32_t cols) {
    return {p, kMxTileBytes, (int32_t)(mx_tiles(rows) * mx_tiles(cols)), kMxTileBytes, 1};
}

bool mx_product_shape(int32_t n, int32_t rows, int32_t cols) {
    return mx_shape(n, cols) && mx_shape(rows, cols) && rows >= 8 && rows % 8 == 0 &&
           mx_shape(n, rows);
}

rvq_status check_mx_product(const char *who, int32_t n, int32_t rows, int32_t cols, int act) {
    CHECK_ARG(mx_product_shape(n, rows, cols),
              "%s: n %d, rows %d, cols %d (n >= 1; rows and cols multiples of 8)", who, n, rows,
              cols);
    CHECK_ARG(act >= MOE_ACT_NONE && act <= MOE_ACT_GELU_TANH, "%s: activation %d", who, act);
    return RVQ_OK;
}

MxJob mx_job(int mats, int32_t n, int32_t rows, int32_t cols, const uint8_t *x, const uint8_t *xs,
             int xfmt, int wfmt, int act, void *ws) {
    MxJob j = {};
    j.mats = mats;
    j.n = n;
    j.rows = rows;
    j.cols = cols;
    j.x = x;
    j.xs = xs;
    j.xfmt = xfmt;
    j.wfmt = wfmt;
    j.act = act;
    j.status = (uint32_t *)ws;
    return j;
}

}  // namespace

extern "C" {

size_t moe_mx_code_bytes(moe_mx fmt, int32_t rows, int32_t cols) {
    return mx_shape(rows, cols) && mx_format((int)fmt) ? code_bytes((int)fmt, rows, cols) : 0;
}

size_t moe_mx_scale_bytes(int32_t rows, int32_t cols) {
    return mx_shape(rows, cols) ? scale_bytes(rows, cols) : 0;
}

rvq_status moe_mx_quantize(const void *x_dev, int64_t ldx, rvq_dtype xdt, int32_t rows,
                           int32_t cols, moe_mx fmt, uint8_t *codes_dev, uint8_t *scales_dev,
                           rvq_stream_t stream) {
    const char *who = "moe_mx_quantize";
    RVQ_TRY(check_mx_shape(who, rows, cols));
    CHECK_ARG(dtype_any(xdt), "%s: dtype %d", who, (int)xdt);
    RVQ_TRY(check_matrix(who, "x", x_dev, ldx, cols));
    RVQ_TRY(check_mx(who, "output", codes_dev, scales_dev, (int)fmt));
    const Span in[] = {{x_dev, ldx, rows, cols, elem_bytes(xdt)}};
    CHECK_ARG(all_apart({codes_of(codes_dev, (int)fmt, rows, cols),
                         scales_of(scales_dev, rows, cols)}, in),
              "%s: codes or scales overlap x or each other", who);
    return launch_mx_quantize({x_dev, ldx, (int)xdt, rows, cols, (int)fmt, codes_dev, scales_dev},
                              (cudaStream_t)stream);
}

rvq_status moe_mx_dequantize(const uint8_t *codes_dev, const uint8_t *scales_dev, moe_mx fmt,
                             int32_t rows, int32_t cols, void *out_dev, rvq_dtype odt, int64_t ldo,
                             rvq_stream_t stream) {
    const char *who = "moe_mx_dequantize";
    RVQ_TRY(check_mx_shape(who, rows, cols));
    RVQ_TRY(check_mx(who, "input", codes_dev, scales_dev, (int)fmt));
    CHECK_ARG(dtype_any(odt), "%s: dtype %d", who, (int)odt);
    RVQ_TRY(check_matrix(who, "out", out_dev, ldo, cols));
    const Span out[] = {{out_dev, ldo, rows, cols, elem_bytes(odt)}};
    const Span in[] = {codes_of(codes_dev, (int)fmt, rows, cols),
                       scales_of(scales_dev, rows, cols)};
    CHECK_ARG(all_apart(out, in), "%s: out overlaps the codes or scales", who);
    return launch_mx_dequantize({codes_dev, scales_dev, rows, cols, (int)fmt, out_dev, ldo, (int)odt},
                                (cudaStream_t)stream);
}

size_t moe_mx_linear_workspace_bytes(int32_t n, int32_t rows, int32_t cols) {
    return mx_product_shape(n, rows, cols) ? RVQ_WS_STATUS_BYTES : 0;
}

size_t moe_mx_gated_linear_workspace_bytes(int32_t n, int32_t rows, int32_t cols) {
    return moe_mx_linear_workspace_bytes(n, rows, cols);
}

rvq_status moe_mx_linear(const uint8_t *x_dev, const uint8_t *x_scales_dev, moe_mx xfmt,
                         const uint8_t *w_dev, const uint8_t *w_scales_dev, moe_mx wfmt,
                         const float *bias_dev, int32_t n, int32_t rows, int32_t cols, moe_act act,
                         float alpha, const void *residual_dev, rvq_dtype rdt, int64_t ldr,
                         void *out_dev, rvq_dtype odt, int64_t ldo, void *ws_dev, size_t ws_bytes,
                         rvq_stream_t stream) {
    const char *who = "moe_mx_linear";
    RVQ_TRY(check_mx_product(who, n, rows, cols, (int)act));
    RVQ_TRY(check_mx(who, "x", x_dev, x_scales_dev, (int)xfmt));
    RVQ_TRY(check_mx(who, "w", w_dev, w_scales_dev, (int)wfmt));
    CHECK_ARG(dtype_any(odt), "%s: out dtype %d", who, (int)odt);
    RVQ_TRY(check_matrix(who, "out", out_dev, ldo, rows));
    if (residual_dev) {
        CHECK_ARG(dtype_any(rdt), "%s: residual dtype %d", who, (int)rdt);
        RVQ_TRY(check_matrix(who, "residual", residual_dev, ldr, rows));
    }
    CHECK_ALIGN(bias_dev, who, "bias");
    const Span out[] = {{out_dev, ldo, n, rows, elem_bytes(odt)}};
    const Span in[] = {codes_of(x_dev, (int)xfmt, n, cols), scales_of(x_scales_dev, n, cols),
                       codes_of(w_dev, (int)wfmt, rows, cols), scales_of(w_scales_dev, rows, cols),
                       vector(bias_dev, rows, 4)};
    CHECK_ARG(all_apart(out, in), "%s: out overlaps an input", who);
    CHECK_ARG((residual_dev == out_dev && rdt == odt && ldr == ldo) ||
                  apart(out[0], {residual_dev, ldr, n, rows, elem_bytes(rdt)}),
              "%s: out overlaps the residual with another type, place or pitch", who);
    RVQ_TRY(check_ws(who, ws_dev, ws_bytes, moe_mx_linear_workspace_bytes(n, rows, cols)));
    MxJob j = mx_job(1, n, rows, cols, x_dev, x_scales_dev, (int)xfmt, (int)wfmt, (int)act, ws_dev);
    j.w[0] = w_dev;
    j.ws[0] = w_scales_dev;
    j.bias[0] = bias_dev;
    j.alpha = alpha;
    j.residual = residual_dev;
    j.rdt = (int)rdt;
    j.ldr = ldr;
    j.out = out_dev;
    j.odt = (int)odt;
    j.ldo = ldo;
    return launch_mx_product(j, (cudaStream_t)stream);
}

rvq_status moe_mx_gated_linear(const uint8_t *x_dev, const uint8_t *x_scales_dev, moe_mx xfmt,
                               const uint8_t *wg_dev, const uint8_t *wg_scales_dev,
                               const uint8_t *wu_dev, const uint8_t *wu_scales_dev, moe_mx wfmt,
                               const float *bg_dev, const float *bu_dev, int32_t n, int32_t rows,
                               int32_t cols, moe_act act, void *out_dev, rvq_dtype odt, int64_t ldo,
                               uint8_t *codes_dev, uint8_t *scales_dev, moe_mx ofmt, void *ws_dev,
                               size_t ws_bytes, rvq_stream_t stream) {
    const char *who = "moe_mx_gated_linear";
    RVQ_TRY(check_mx_product(who, n, rows, cols, (int)act));
    RVQ_TRY(check_mx(who, "x", x_dev, x_scales_dev, (int)xfmt));
    RVQ_TRY(check_mx(who, "wg", wg_dev, wg_scales_dev, (int)wfmt));
    RVQ_TRY(check_mx(who, "wu", wu_dev, wu_scales_dev, (int)wfmt));
    CHECK_ARG((out_dev != nullptr) != (codes_dev != nullptr || scales_dev != nullptr),
              "%s: either out or codes and scales", who);
    if (out_dev) {
        CHECK_ARG(dtype_any(odt), "%s: out dtype %d", who, (int)odt);
        RVQ_TRY(check_matrix(who, "out", out_dev, ldo, rows));
    } else {
        RVQ_TRY(check_mx(who, "output", codes_dev, scales_dev, (int)ofmt));
    }
    CHECK_ALIGN(bg_dev, who, "bg");
    CHECK_ALIGN(bu_dev, who, "bu");
    const Span out[] = {{out_dev, ldo, n, rows, elem_bytes(odt)},
                        codes_of(codes_dev, (int)ofmt, n, rows), scales_of(scales_dev, n, rows)};
    const Span in[] = {codes_of(x_dev, (int)xfmt, n, cols), scales_of(x_scales_dev, n, cols),
                       codes_of(wg_dev, (int)wfmt, rows, cols), scales_of(wg_scales_dev, rows, cols),
                       codes_of(wu_dev, (int)wfmt, rows, cols), scales_of(wu_scales_dev, rows, cols),
                       vector(bg_dev, rows, 4), vector(bu_dev, rows, 4)};
    CHECK_ARG(all_apart(out, in), "%s: an output overlaps an input or another output", who);
    RVQ_TRY(check_ws(who, ws_dev, ws_bytes, moe_mx_gated_linear_workspace_bytes(n, rows, cols)));
    MxJob j = mx_job(2, n, rows, cols, x_dev, x_scales_dev, (int)xfmt, (int)wfmt, (int)act, ws_dev);
    j.w[0] = wg_dev;
    j.w[1] = wu_dev;
    j.ws[0] = wg_scales_dev;
    j.ws[1] = wu_scales_dev;
    j.bias[0] = bg_dev;
    j.bias[1] = bu_dev;
    j.alpha = 1.f;
    j.out = out_dev;
    j.odt = (int)odt;
    j.ldo = ldo;
    j.codes = codes_dev;
    j.scales = scales_dev;
    j.ofmt = (int)ofmt;
    return launch_mx_product(j, (cudaStream_t)stream);
}

rvq_status rvq_selftest_mx_plan(int32_t gated, moe_mx xfmt, moe_mx wfmt, int32_t n, int32_t rows,
                                int32_t cols, int32_t out[2]) {
    const char *who = "rvq_selftest_mx_plan";
    CHECK_ARG(mx_product_shape(n, rows, cols) && mx_format((int)xfmt) && mx_format((int)wfmt) && out,
              "%s: n %d, rows %d, cols %d, formats %d and %d, out %p", who, n, rows, cols, (int)xfmt,
              (int)wfmt, (void *)out);
    const MxJob j = mx_job(gated ? 2 : 1, n, rows, cols, nullptr, nullptr, (int)xfmt, (int)wfmt, 0,
                           nullptr);
    const bool tiles = mx_by_tiles(j);
    out[0] = tiles ? MOE_WAY_TILES : MOE_WAY_STREAM;
    out[1] = tiles ? 1 : plan_mx_stream(j).split;
    return RVQ_OK;
}

rvq_status moe_norm_join_mx(const void *h_dev, rvq_dtype hdt, const void *y_dev, rvq_dtype ydt,
                            int32_t n, int32_t d, float alpha, const void *gate_dev,
                            moe_gate gate_kind, rvq_dtype gdt, int32_t post_norm,
                            const void *w_post_dev, const void *w_pre_dev, rvq_dtype wdt, float eps,
                            void *h_out_dev, void *xn_dev, rvq_dtype xdt, moe_mx fmt,
                            uint8_t *codes_dev, uint8_t *scales_dev, float *rstd_dev,
                            rvq_stream_t stream) {
    const char *who = "moe_norm_join_mx";
    RVQ_TRY(check_join(who, h_dev, hdt, y_dev, ydt, n, d, gate_dev, (int)gate_kind, gdt, post_norm,
                       w_post_dev, w_pre_dev, wdt, xdt));
    CHECK_ARG(eps >= 0.f && isfinite(eps), "%s: eps %g", who, (double)eps);
    RVQ_TRY(check_mx(who, "output", codes_dev, scales_dev, (int)fmt));
    CHECK_ALIGN(h_out_dev, who, "h_out");
    CHECK_ALIGN(xn_dev, who, "xn");
    CHECK_ALIGN(rstd_dev, who, "rstd");
    const JoinSpan spans[] = {{h_dev, hdt, n, d}, {y_dev, ydt, n, d},
                              gate_span(gate_dev, gdt, (int)gate_kind, n, d),
                              {w_post_dev, wdt, 1, d}, {w_pre_dev, wdt, 1, d}};
    CHECK_ARG(join_outputs_ok(spans, {h_out_dev, hdt, n, d}, {xn_dev, xdt, n, d},
                              {rstd_dev, RVQ_F32, 2, n}),
              "%s: an output overlaps an input of another type or place, or another output", who);
    const Span mx[] = {codes_of(codes_dev, (int)fmt, n, d),
                       scales_of(scales_dev, n, d)};
    Span others[8];
    const JoinSpan outs[] = {{h_out_dev, hdt, n, d}, {xn_dev, xdt, n, d}, {rstd_dev, RVQ_F32, 2, n}};
    for (int i = 0; i < 5; ++i) others[i] = span_of(spans[i]);
    for (int i = 0; i < 3; ++i) others[5 + i] = span_of(outs[i]);
    CHECK_ARG(all_apart(mx, others), "%s: codes or scales overlap another matrix", who);
    MxJoinJob job = {};
    JoinJob &j = job.join;
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
    job.fmt = (int)fmt;
    job.codes = codes_dev;
    job.scales = scales_dev;
    return launch_mx_join(job, (cudaStream_t)stream);
}

}  // extern "C"
