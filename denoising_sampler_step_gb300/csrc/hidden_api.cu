// The C entry points of the hidden stream (embedding lookup, norm, head): argument checks and launches.
// Declarations and contracts are in include/dgsamp.h.
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>
#include <initializer_list>

#include "dg_internal.h"
#include "hidden.cuh"

namespace dg {
namespace {

constexpr int64_t kMaxRows = 1LL << 28, kMaxVocab = 0x7ffffff0LL, kMaxWidth = 1LL << 30;
// rows * ld stays below this, so that offsets in bytes fit 64 bits
constexpr int64_t kMaxElements = 1LL << 56;

bool known(int32_t dtype, bool codes = false) {
    return dtype == DG_F32 || dtype == DG_BF16 || (codes && dtype == DG_E4M3);
}

// A matrix [rows, d]: its type, stride, size and the alignment of its entries.
dg_status check_rows(const char *what, const char *name, const Rows &m, int64_t rows, int64_t d, bool codes = false) {
    if (!known(m.dtype, codes)) return fail(DG_ERR_INVALID_ARG, "%s: unknown dtype %d of %s", what, m.dtype, name);
    if (m.ld < d) return fail(DG_ERR_INVALID_ARG, "%s: the row stride of %s is below %lld", what, name, (long long)d);
    if (rows > 0 && !m.p) return fail(DG_ERR_INVALID_ARG, "%s: %s is NULL", what, name);
    if (m.ld > kMaxElements / (rows + 1)) return fail(DG_ERR_UNSUPPORTED, "%s: %s is too large", what, name);
    if (reinterpret_cast<uintptr_t>(m.p) % entry_size(m.dtype) != 0)
        return fail(DG_ERR_UNSUPPORTED, "%s: %s is not aligned to its entries", what, name);
    return DG_OK;
}

// Memory from lo to hi, of a matrix only the first `width` bytes of every `pitch`.
struct Span {
    uintptr_t lo, hi, pitch = 0, width = 0;
};
Span span(const Rows &m, int64_t rows, int64_t d) {
    const uintptr_t lo = reinterpret_cast<uintptr_t>(m.p);
    if (!m.p || rows < 1) return {lo, lo};
    const int64_t size = entry_size(m.dtype);
    return {lo, lo + (uintptr_t)(((rows - 1) * m.ld + d) * size), (uintptr_t)(m.ld * size), (uintptr_t)(d * size)};
}
Span span(const void *p, int64_t bytes) {
    const uintptr_t lo = reinterpret_cast<uintptr_t>(p);
    return {lo, lo + (p ? (uintptr_t)bytes : 0)};
}
bool meet(const Span &a, const Span &b) {
    if (!(a.lo < b.hi && b.lo < a.hi)) return false;
    if (a.pitch == 0 || a.pitch != b.pitch) return true;
    // columns of one buffer: b's may lie in what a leaves of each row
    const uintptr_t off = b.lo >= a.lo ? (b.lo - a.lo) % a.pitch : a.pitch - 1 - (a.lo - b.lo - 1) % a.pitch;
    return off < a.width || off + b.width > a.pitch;
}

// Whether `out` may stand where `in` does: apart, or exactly in its place.
bool apart_or_same(const Rows &out, const Rows &in, int64_t rows, int64_t d) {
    if (out.p == in.p && out.dtype == in.dtype && (out.ld == in.ld || rows <= 1)) return true;
    return !meet(span(out, rows, d), span(in, rows, d));
}

dg_status overlap(const char *what, const char *out, const char *in) {
    return fail(DG_ERR_INVALID_ARG, "%s: %s overlaps %s", what, out, in);
}

dg_status check_slice(const char *what, int64_t V, int64_t s, int64_t e, int64_t rows_pad, int64_t R, int64_t d,
                      const int32_t *token) {
    if (R < 0 || d < 1 || V < 1) return fail(DG_ERR_INVALID_ARG, "%s: need R >= 0, d >= 1 and V >= 1", what);
    if (s < 0 || e < s || e > V)
        return fail(DG_ERR_INVALID_ARG, "%s: slice [%lld, %lld) is reversed or outside the vocabulary", what,
                    (long long)s, (long long)e);
    if (e - s > rows_pad)
        return fail(DG_ERR_INVALID_ARG, "%s: the slice has %lld vocabulary entries but the shard only %lld rows", what,
                    (long long)(e - s), (long long)rows_pad);
    if (V > kMaxVocab || R > kMaxRows || d >= kMaxWidth) return fail(DG_ERR_UNSUPPORTED, "%s: V, R or d too large", what);
    if (R > 0 && !token) return fail(DG_ERR_INVALID_ARG, "%s: token is NULL", what);
    return DG_OK;
}

dg_status check_norm(const char *what, int64_t R, int64_t d, const void *weight, int32_t weight_dtype, float offset) {
    if (R < 0 || d < 1) return fail(DG_ERR_INVALID_ARG, "%s: need R >= 0 and d >= 1", what);
    if (R > kMaxRows) return fail(DG_ERR_UNSUPPORTED, "%s: R too large", what);
    if (d > kMaxNormWidth)
        return fail(DG_ERR_UNSUPPORTED, "%s: d = %lld is above %lld", what, (long long)d, (long long)kMaxNormWidth);
    if (!std::isfinite(offset)) return fail(DG_ERR_INVALID_ARG, "%s: weight_offset must be finite", what);
    if (weight && !known(weight_dtype))
        return fail(DG_ERR_INVALID_ARG, "%s: unknown dtype %d of weight", what, weight_dtype);
    if (weight && reinterpret_cast<uintptr_t>(weight) % entry_size(weight_dtype) != 0)
        return fail(DG_ERR_UNSUPPORTED, "%s: weight is not aligned to its entries", what);
    return DG_OK;
}

// Vectors of four-byte entries.
dg_status check_vectors(const char *what, std::initializer_list<const void *> vectors) {
    for (const void *v : vectors)
        if (reinterpret_cast<uintptr_t>(v) & 3)
            return fail(DG_ERR_UNSUPPORTED, "%s: a vector of tokens, scales or statistics is not 4-byte aligned", what);
    return DG_OK;
}

dg_status check_workspace(const char *what, const void *workspace, size_t bytes, size_t need) {
    if (!workspace || bytes < need)
        return fail(DG_ERR_INVALID_ARG, "%s: workspace of %zu bytes is below the %zu needed", what,
                    workspace ? bytes : (size_t)0, need);
    if (!aligned16(workspace)) return fail(DG_ERR_UNSUPPORTED, "%s: workspace must be 16-byte aligned", what);
    return DG_OK;
}

#define DG_TRY(call)                        \
    do {                                    \
        const dg_status st_ = (call);       \
        if (st_ != DG_OK) return st_;       \
    } while (0)

}  // namespace
}  // namespace dg

using namespace dg;

extern "C" {

dg_status dg_token_embed(const void *table, int32_t dtype, const float *scale, int64_t V, int64_t vocab_start,
                         int64_t vocab_end, int64_t rows_pad, int64_t ldw, int64_t d, const int32_t *token,
                         int64_t R, float gamma, void *out, int32_t out_dtype, int64_t ldo, dg_stream_t stream) {
    t_last_error[0] = 0;
    const char *what = "token embed";
    DG_TRY(check_slice(what, V, vocab_start, vocab_end, rows_pad, R, d, token));
    const int64_t rows = vocab_end - vocab_start;
    const EmbedRows a{Rows{const_cast<void *>(table), ldw, dtype}, scale, V, vocab_start, vocab_end, R, d, token, gamma,
                      Rows{out, ldo, out_dtype}, false};
    DG_TRY(check_rows(what, "table", a.table, R > 0 ? rows : 0, d, true));
    DG_TRY(check_rows(what, "out", a.rows, R, d));
    if (R == 0) return DG_OK;
    if ((dtype == DG_E4M3) != (scale != nullptr) && rows > 0)
        return fail(DG_ERR_INVALID_ARG, "%s: scale goes with E4M3 codes, and with them alone", what);
    DG_TRY(check_vectors(what, {token, scale}));
    if (meet(span(a.rows, R, d), span(a.table, rows, d))) return overlap(what, "out", "table");
    if (meet(span(a.rows, R, d), span(token, 4 * R))) return overlap(what, "out", "token");
    if (meet(span(a.rows, R, d), span(scale, 4 * rows))) return overlap(what, "out", "scale");
    const cudaError_t e = launch_token_embed(a, (cudaStream_t)stream);
    return e == cudaSuccess ? DG_OK : cuda_fail(e, what);
}

size_t dg_token_embed_backward_workspace_size(int64_t R, int64_t vocab_len, int64_t d) {
    if (R < 1 || R > kMaxRows || vocab_len < 0 || vocab_len > kMaxVocab || d < 1 || d >= kMaxWidth) return 0;
    return token_embed_backward_bytes(R, d);
}

dg_status dg_token_embed_backward(const void *grad, int32_t dtype, int64_t R, int64_t d, int64_t ldg,
                                  const int32_t *token, int64_t V, int64_t vocab_start, int64_t vocab_end,
                                  float gamma, void *grad_table, int32_t table_dtype, int64_t rows_pad, int64_t ldt,
                                  int32_t accumulate, void *workspace, size_t workspace_bytes, dg_stream_t stream) {
    t_last_error[0] = 0;
    const char *what = "token embed backward";
    DG_TRY(check_slice(what, V, vocab_start, vocab_end, rows_pad, R, d, token));
    const int64_t rows = vocab_end - vocab_start;
    const EmbedRows a{Rows{grad_table, ldt, table_dtype}, nullptr, V, vocab_start, vocab_end, R, d, token, gamma,
                      Rows{const_cast<void *>(grad), ldg, dtype}, accumulate != 0};
    DG_TRY(check_rows(what, "grad_table", a.table, rows, d));
    DG_TRY(check_rows(what, "grad", a.rows, R, d));
    if (rows == 0 || (R == 0 && a.accumulate)) return DG_OK;
    DG_TRY(check_vectors(what, {token}));
    if (R > 0) {
        DG_TRY(check_workspace(what, workspace, workspace_bytes, token_embed_backward_bytes(R, d)));
        const Span t = span(a.table, rows, d), w = span(workspace, (int64_t)workspace_bytes);
        if (meet(t, span(a.rows, R, d))) return overlap(what, "grad_table", "grad");
        if (meet(t, span(token, 4 * R))) return overlap(what, "grad_table", "token");
        if (meet(w, t) || meet(w, span(a.rows, R, d)) || meet(w, span(token, 4 * R)))
            return overlap(what, "workspace", "another argument");
    }
    const cudaError_t e = launch_token_embed_backward(a, workspace, (cudaStream_t)stream);
    return e == cudaSuccess ? DG_OK : cuda_fail(e, what);
}

dg_status dg_rms_norm(const void *x, int32_t dtype, int64_t R, int64_t d, int64_t ldx, const void *residual,
                      int32_t residual_dtype, int64_t ldr, const void *weight, int32_t weight_dtype,
                      float weight_offset, float eps, void *hidden, int32_t hidden_dtype, int64_t ldh, void *out,
                      int32_t out_dtype, int64_t ldo, float *out_scale, float *rstd, dg_stream_t stream) {
    t_last_error[0] = 0;
    const char *what = "rms norm";
    DG_TRY(check_norm(what, R, d, weight, weight_dtype, weight_offset));
    if (!(eps >= 0.0f) || !std::isfinite(eps))
        return fail(DG_ERR_INVALID_ARG, "%s: eps must not be negative, and finite", what);
    const NormRows a{Rows{const_cast<void *>(x), ldx, dtype}, Rows{const_cast<void *>(residual), ldr, residual_dtype},
                     Rows{hidden, ldh, hidden_dtype}, Rows{out, ldo, out_dtype}, out_scale, rstd, weight, weight_dtype,
                     weight_offset, eps, R, d};
    DG_TRY(check_rows(what, "x", a.x, R, d));
    if (residual) DG_TRY(check_rows(what, "residual", a.residual, R, d));
    if (hidden) DG_TRY(check_rows(what, "hidden", a.hidden, R, d));
    DG_TRY(check_rows(what, "out", a.out, R, d, true));
    if (R == 0) return DG_OK;
    if ((out_dtype == DG_E4M3) != (out_scale != nullptr))
        return fail(DG_ERR_INVALID_ARG, "%s: out_scale goes with E4M3 codes, and with them alone", what);
    DG_TRY(check_vectors(what, {out_scale, rstd}));
    if (!apart_or_same(a.out, a.x, R, d)) return overlap(what, "out", "x without replacing it");
    if (residual && !apart_or_same(a.out, a.residual, R, d)) return overlap(what, "out", "residual without replacing it");
    const Span so = span(a.out, R, d), sh = span(a.hidden, R, d);
    if (hidden) {
        if (!apart_or_same(a.hidden, a.x, R, d)) return overlap(what, "hidden", "x without replacing it");
        if (residual && !apart_or_same(a.hidden, a.residual, R, d))
            return overlap(what, "hidden", "residual without replacing it");
        if (meet(so, sh)) return overlap(what, "out", "hidden");
    }
    const Span sw = span(weight, weight ? d * entry_size(weight_dtype) : 0);
    if (meet(so, sw) || meet(sh, sw)) return overlap(what, "an output", "weight");
    const Span rows[] = {span(out_scale, 4 * R), span(rstd, 4 * R)};
    for (const Span &v : rows)
        if (meet(v, so) || meet(v, sh) || meet(v, sw) || meet(v, span(a.x, R, d)) || meet(v, span(a.residual, R, d)))
            return overlap(what, "out_scale or rstd", "another argument");
    if (meet(rows[0], rows[1])) return overlap(what, "out_scale", "rstd");
    const cudaError_t e = launch_rms_norm(a, (cudaStream_t)stream);
    return e == cudaSuccess ? DG_OK : cuda_fail(e, what);
}

size_t dg_rms_norm_backward_workspace_size(int64_t R, int64_t d) {
    if (R < 1 || R > kMaxRows || d < 1 || d > kMaxNormWidth) return 0;
    return rms_norm_backward_bytes(R, d);
}

dg_status dg_rms_norm_backward(const void *grad, int32_t dtype, int64_t R, int64_t d, int64_t ldg,
                               const void *hidden, int32_t hidden_dtype, int64_t ldh, const float *rstd,
                               const void *weight, int32_t weight_dtype, float weight_offset,
                               const void *grad_hidden, int32_t grad_hidden_dtype, int64_t ldu, void *grad_x,
                               int64_t ldx, void *grad_weight, void *workspace, size_t workspace_bytes,
                               dg_stream_t stream) {
    t_last_error[0] = 0;
    const char *what = "rms norm backward";
    DG_TRY(check_norm(what, R, d, weight, weight_dtype, weight_offset));
    const NormBackRows a{Rows{const_cast<void *>(grad), ldg, dtype}, Rows{const_cast<void *>(hidden), ldh, hidden_dtype},
                         Rows{const_cast<void *>(grad_hidden), ldu, grad_hidden_dtype}, Rows{grad_x, ldx, hidden_dtype},
                         rstd, weight, weight_dtype, weight_offset, grad_weight, R, d};
    DG_TRY(check_rows(what, "grad", a.grad, R, d));
    DG_TRY(check_rows(what, "hidden", a.hidden, R, d));
    if (grad_hidden) DG_TRY(check_rows(what, "grad_hidden", a.grad_hidden, R, d));
    DG_TRY(check_rows(what, "grad_x", a.grad_x, R, d));
    if (R > 0 && !rstd) return fail(DG_ERR_INVALID_ARG, "%s: rstd is NULL", what);
    if (grad_weight && !weight) return fail(DG_ERR_INVALID_ARG, "%s: grad_weight without a weight", what);
    if (grad_weight && reinterpret_cast<uintptr_t>(grad_weight) % entry_size(weight_dtype) != 0)
        return fail(DG_ERR_UNSUPPORTED, "%s: grad_weight is not aligned to its entries", what);
    if (R == 0 && !grad_weight) return DG_OK;
    DG_TRY(check_vectors(what, {rstd}));
    const Span sx = span(a.grad_x, R, d), sw = span(grad_weight, grad_weight ? d * entry_size(weight_dtype) : 0);
    const Span in[] = {span(a.grad, R, d), span(a.hidden, R, d), span(a.grad_hidden, R, d), span(rstd, 4 * R),
                       span(weight, weight ? d * entry_size(weight_dtype) : 0)};
    if (R > 0) {
        if (!apart_or_same(a.grad_x, a.grad, R, d)) return overlap(what, "grad_x", "grad without replacing it");
        if (!apart_or_same(a.grad_x, a.hidden, R, d)) return overlap(what, "grad_x", "hidden without replacing it");
        if (grad_hidden && !apart_or_same(a.grad_x, a.grad_hidden, R, d))
            return overlap(what, "grad_x", "grad_hidden without replacing it");
        if (meet(sx, in[3])) return overlap(what, "grad_x", "rstd");
        if (meet(sx, in[4]) || meet(sx, sw)) return overlap(what, "grad_x", "weight or grad_weight");
    }
    for (const Span &v : in)
        if (meet(sw, v)) return overlap(what, "grad_weight", "another argument");
    if (grad_weight && R > 0) {
        DG_TRY(check_workspace(what, workspace, workspace_bytes, rms_norm_backward_bytes(R, d)));
        const Span ws = span(workspace, (int64_t)workspace_bytes);
        for (const Span &v : in)
            if (meet(ws, v)) return overlap(what, "workspace", "another argument");
        if (meet(ws, sx) || meet(ws, sw)) return overlap(what, "workspace", "another argument");
    }
    const cudaError_t e = launch_rms_norm_backward(a, workspace, (cudaStream_t)stream);
    return e == cudaSuccess ? DG_OK : cuda_fail(e, what);
}

dg_status dg_head_e4m3(const uint8_t *X, int64_t ldx, const float *x_scale, int64_t R, int64_t d, const uint8_t *Q,
                       const float *scale, int64_t V, int64_t ldq, void *logits, int32_t dtype, int64_t ldl,
                       dg_stream_t stream) {
    t_last_error[0] = 0;
    const char *what = "head";
    if (R < 0 || d < 1 || V < 1) return fail(DG_ERR_INVALID_ARG, "%s: need R >= 0, d >= 1 and V >= 1", what);
    if (R > kMaxRows || V > (1LL << 30) || d >= (1LL << 24)) return fail(DG_ERR_UNSUPPORTED, "%s: R, V or d too large", what);
    const Rows x{const_cast<uint8_t *>(X), ldx, DG_E4M3}, q{const_cast<uint8_t *>(Q), ldq, DG_E4M3}, l{logits, ldl, dtype};
    DG_TRY(check_rows(what, "X", x, R, d, true));
    DG_TRY(check_rows(what, "Q", q, R > 0 ? V : 0, d, true));
    DG_TRY(check_rows(what, "logits", l, R, V));
    if (R == 0) return DG_OK;
    if (!x_scale || !scale) return fail(DG_ERR_INVALID_ARG, "%s: a scale is NULL", what);
    if (!aligned16(X) || !aligned16(Q) || (ldx & 15) || (ldq & 15))
        return fail(DG_ERR_UNSUPPORTED, "%s: rows of codes must start on 16-byte boundaries: pad the row stride to a "
                    "multiple of 16 (d stays; columns at d and past it are not read)", what);
    if (!aligned16(logits) || (ldl * entry_size(dtype)) % 16 != 0)
        return fail(DG_ERR_UNSUPPORTED, "%s: logits rows must start on 16-byte boundaries: pad the row stride to a "
                    "multiple of %d elements", what, 16 / entry_size(dtype));
    DG_TRY(check_vectors(what, {x_scale, scale}));
    if (ldx >= (1LL << 40) || ldq >= (1LL << 40)) return fail(DG_ERR_UNSUPPORTED, "%s: a row stride is too large", what);
    const Span sl = span(l, R, V);
    if (meet(sl, span(x, R, d)) || meet(sl, span(q, V, d)) || meet(sl, span(x_scale, 4 * R)) || meet(sl, span(scale, 4 * V)))
        return overlap(what, "logits", "an input");
    const char *msg = what;
    const cudaError_t e = launch_head_e4m3(X, ldx, x_scale, R, d, Q, ldq, scale, V, logits, dtype, ldl,
                                           (cudaStream_t)stream, &msg);
    return e == cudaSuccess ? DG_OK : cuda_fail(e, msg);
}

}  // extern "C"
