// Argument checks shared by the host side of the dense and the microscaled operators
// (dense_api.cu, mx_api.cu).
#pragma once

#include "dense.cuh"

#define CHECK_ARG(cond, ...)          \
    do {                              \
        if (!(cond)) {                \
            set_error(__VA_ARGS__);   \
            return RVQ_EINVAL;        \
        }                             \
    } while (0)
#define CHECK_ALIGN(p, who, what)                                                          \
    do {                                                                                   \
        if (((uintptr_t)(p) & 15u) != 0) {                                                 \
            set_error("%s: %s %p is not 16-byte aligned", who, what, (const void *)(p));   \
            return RVQ_EALIGN;                                                             \
        }                                                                                  \
    } while (0)

namespace rvq {

constexpr int64_t kMaxLd = (int64_t)1 << 36;  // a tensor map's row pitch is below 2^40 bytes
constexpr int32_t kMaxDim = (1 << 24) - 256;  // 65535 blocks of 256 columns

inline size_t up256(size_t v) { return (v + 255) / 256 * 256; }

inline bool dtype16(rvq_dtype t) { return t == RVQ_BF16 || t == RVQ_F16; }
inline bool dtype_any(rvq_dtype t) { return t == RVQ_F32 || dtype16(t); }
inline size_t elem_bytes(rvq_dtype t) { return t == RVQ_F32 ? 4 : 2; }

// A row-major matrix: not NULL, 16-byte aligned, pitch >= columns and a
// multiple of 8 elements.
inline rvq_status check_matrix(const char *who, const char *what, const void *p, int64_t ld,
                        int32_t cols) {
    CHECK_ARG(p != nullptr, "%s: null %s", who, what);
    CHECK_ARG(ld >= cols && ld % 8 == 0 && ld < kMaxLd,
              "%s: %s row pitch %lld for %d columns (>= columns, a multiple of 8)", who, what,
              (long long)ld, cols);
    CHECK_ALIGN(p, who, what);
    return RVQ_OK;
}

inline rvq_status check_ws(const char *who, const void *ws, size_t bytes, size_t need) {
    CHECK_ARG(ws != nullptr && ((uintptr_t)ws & 255u) == 0,
              "%s: workspace must be 256-byte aligned and not null", who);
    if (bytes < need) {
        set_error("%s: workspace %zu < %zu bytes", who, bytes, need);
        return RVQ_ENOMEM;
    }
    return RVQ_OK;
}

// Two row-major matrices do not overlap.
inline bool disjoint(const void *a, int64_t lda, int32_t ra, int32_t ca, size_t ea, const void *b,
              int64_t ldb, int32_t rb, int32_t cb, size_t eb) {
    if (a == nullptr || b == nullptr) return true;
    const uintptr_t a0 = (uintptr_t)a, b0 = (uintptr_t)b;
    const uintptr_t a1 = a0 + ((uint64_t)(ra - 1) * (uint64_t)lda + (uint64_t)ca) * ea;
    const uintptr_t b1 = b0 + ((uint64_t)(rb - 1) * (uint64_t)ldb + (uint64_t)cb) * eb;
    if (a1 <= b0 || b1 <= a0) return true;
    // of one row pitch, in different columns: parts of one wider matrix
    const uint64_t wa = (uint64_t)ca * ea, wb = (uint64_t)cb * eb;
    const uint64_t pa = (uint64_t)lda * ea, pb = (uint64_t)ldb * eb;
    const uint64_t pitch = ra > 1 ? pa : pb;
    if ((ra > 1 && rb > 1 && pa != pb) || pitch == 0) return false;
    const uint64_t at = b0 >= a0 ? (b0 - a0) % pitch : (pitch - (a0 - b0) % pitch) % pitch;
    return at >= wa && at + wb <= pitch;
}

// A row-major matrix, or (vector()) contiguous values; NULL: absent.
struct Span {
    const void *p;
    int64_t ld;
    int32_t rows, cols;
    size_t e;
};

inline Span vector(const void *p, int32_t n, size_t e) { return {p, n, 1, n, e}; }

inline bool apart(const Span &a, const Span &b) {
    return disjoint(a.p, a.ld, a.rows, a.cols, a.e, b.p, b.ld, b.rows, b.cols, b.e);
}

// Outputs that one launch may write while it reads the inputs: none overlaps an
// input or another output.
template <int O, int I>
bool all_apart(const Span (&out)[O], const Span (&in)[I]) {
    for (int o = 0; o < O; ++o) {
        for (int i = 0; i < I; ++i)
            if (!apart(out[o], in[i])) return false;
        for (int i = 0; i < o; ++i)
            if (!apart(out[o], out[i])) return false;
    }
    return true;
}

// ---------------------------------------------------------------- norm join

inline rvq_status check_join(const char *who, const void *h, rvq_dtype hdt, const void *y,
                             rvq_dtype ydt, int32_t n, int32_t d, const void *gate, int kind,
                             rvq_dtype gdt, int32_t post_norm, const void *w_post,
                             const void *w_pre, rvq_dtype wdt, rvq_dtype xdt) {
    CHECK_ARG(n >= 1 && n <= kMaxDim && d >= 8 && d % 8 == 0 && d <= kJoinMaxD,
              "%s: n %d, d %d (n from 1 to 2^24 - 256; d a multiple of 8, at most %d)", who, n, d,
              kJoinMaxD);
    CHECK_ARG(dtype_any(hdt) && dtype_any(ydt) && dtype_any(gdt) && dtype_any(wdt) &&
                  dtype_any(xdt),
              "%s: dtypes %d, %d, %d, %d, %d", who, (int)hdt, (int)ydt, (int)gdt, (int)wdt,
              (int)xdt);
    CHECK_ARG(y != nullptr, "%s: null y", who);
    CHECK_ARG(kind >= MOE_GATE_NONE && kind <= MOE_GATE_FULL && (kind == MOE_GATE_NONE) == !gate,
              "%s: gate kind %d %s a gate", who, kind, gate ? "with" : "without");
    CHECK_ARG(post_norm || !w_post, "%s: w_post without post_norm", who);
    CHECK_ALIGN(h, who, "h");
    CHECK_ALIGN(y, who, "y");
    CHECK_ALIGN(gate, who, "gate");
    CHECK_ALIGN(w_post, who, "w_post");
    CHECK_ALIGN(w_pre, who, "w_pre");
    return RVQ_OK;
}

// A tensor of the join: n rows of d values, or values over tokens or channels
// (len); kept apart from others, or over rows of its own type.
struct JoinSpan {
    const void *p;
    rvq_dtype dt;
    int32_t rows, cols;
};

inline bool apart(const JoinSpan &a, const JoinSpan &b) {
    return disjoint(a.p, a.cols, a.rows, a.cols, elem_bytes(a.dt), b.p, b.cols, b.rows, b.cols,
                    elem_bytes(b.dt));
}

// Every block reads its rows before it writes them: an output may take the place of
// rows of the same type.
inline bool same_or_apart(const JoinSpan &a, const JoinSpan &b) {
    return (a.p == b.p && a.dt == b.dt && a.rows == b.rows && a.cols == b.cols) || apart(a, b);
}

inline JoinSpan gate_span(const void *p, rvq_dtype dt, int kind, int32_t n, int32_t d) {
    return {p, dt, kind == MOE_GATE_TOKEN || kind == MOE_GATE_FULL ? n : 1,
            kind == MOE_GATE_CHANNEL || kind == MOE_GATE_FULL ? d : 1};
}

inline Span span_of(const JoinSpan &s) {
    return {s.p, s.cols, s.rows, s.cols, elem_bytes(s.dt)};
}

// in: h, y, the gate, w_post, w_pre.  h_out and xn may take the place of h, y or a full
// gate; otherwise the outputs overlap nothing.
inline bool join_outputs_ok(const JoinSpan (&in)[5], const JoinSpan &h_out, const JoinSpan &xn,
                            const JoinSpan &rstd) {
    bool ok = apart(h_out, xn) && apart(h_out, rstd) && apart(xn, rstd);
    for (int i = 0; i < 5; ++i) {
        const bool rows = i < 3 && in[i].rows == xn.rows && in[i].cols == xn.cols;
        for (const JoinSpan *o : {&h_out, &xn})
            ok = ok && (rows ? same_or_apart(*o, in[i]) : apart(*o, in[i]));
        ok = ok && apart(rstd, in[i]);
    }
    return ok;
}

}  // namespace rvq
