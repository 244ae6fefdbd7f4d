// The C entry points of the losses and of the top logits: argument checks and launches.
// Declarations and contracts are in include/dgsamp.h.
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "dg_internal.h"
#include "row_loss.cuh"

namespace dg {
namespace {

// R * ld stays below this, so that offsets in bytes fit 64 bits.
constexpr int64_t kMaxElements = 1LL << 56;

// The rules every call of this part has in common.
dg_status check_rows(const char *what, const void *logits, int32_t dtype, int64_t R, int64_t V, int64_t ldl,
                     float temperature) {
    if (dtype != DG_F32 && dtype != DG_BF16) return fail(DG_ERR_INVALID_ARG, "%s: unknown dtype %d", what, dtype);
    if (R < 0 || V < 1 || ldl < V) return fail(DG_ERR_INVALID_ARG, "%s: need R >= 0, V >= 1, ldl >= V", what);
    if (!(temperature > 0.0f) || !(temperature < INFINITY))
        return fail(DG_ERR_INVALID_ARG, "%s: temperature must be positive and finite", what);
    if (R > 0 && !logits) return fail(DG_ERR_INVALID_ARG, "%s: logits is NULL", what);
    if (V > 0x7ffffff0LL || R > (1LL << 28) || ldl > kMaxElements / (R + 1))
        return fail(DG_ERR_UNSUPPORTED, "%s: V, R or ldl too large", what);
    if (R > 0 && (!aligned16(logits) || (ldl * element_size(dtype)) % 16 != 0))
        return fail(DG_ERR_UNSUPPORTED,
                    "%s: logits rows must start on 16-byte boundaries: pad the row stride to a multiple of %d "
                    "elements (V stays; columns at V and past it are not read)",
                    what, 16 / element_size(dtype));
    return DG_OK;
}

// The gradient's place: beside the logits, or exactly on them.
dg_status check_grad(const char *what, const void *logits, int32_t dtype, int64_t R, int64_t V, int64_t ldl,
                     const void *grad, int64_t ldg) {
    const int64_t size = element_size(dtype);
    if (!grad) return fail(DG_ERR_INVALID_ARG, "%s: grad is NULL", what);
    if (ldg < V) return fail(DG_ERR_INVALID_ARG, "%s: need ldg >= V", what);
    if (ldg > kMaxElements / (R + 1)) return fail(DG_ERR_UNSUPPORTED, "%s: ldg too large", what);
    if (!aligned16(grad) || (ldg * size) % 16 != 0)
        return fail(DG_ERR_UNSUPPORTED,
                    "%s: grad rows must start on 16-byte boundaries: pad the row stride to a multiple of %d elements",
                    what, 16 / element_size(dtype));
    if (grad == logits && (ldg == ldl || R <= 1)) return DG_OK;
    const uintptr_t x0 = reinterpret_cast<uintptr_t>(logits), g0 = reinterpret_cast<uintptr_t>(grad);
    const uintptr_t x1 = x0 + (uintptr_t)(((R - 1) * ldl + V) * size);
    const uintptr_t g1 = g0 + (uintptr_t)(((R - 1) * ldg + V) * size);
    if (g0 < x1 && x0 < g1)
        return fail(DG_ERR_INVALID_ARG, "%s: grad overlaps the logits without replacing them", what);
    return DG_OK;
}

dg_status check_workspace(const char *what, const RowLossArgs &a, RowLossHead head, RowLossPass pass,
                          const void *workspace, size_t workspace_bytes) {
    if (!takes_workspace(a.V, element_size(a.dtype), head, pass)) return DG_OK;
    const size_t need = row_loss_workspace_bytes(a.R, a.V, a.dtype);
    if (!workspace || workspace_bytes < need)
        return fail(DG_ERR_INVALID_ARG, "%s: workspace of %zu bytes is below the %zu needed", what, workspace_bytes,
                    need);
    if (!aligned16(workspace)) return fail(DG_ERR_UNSUPPORTED, "%s: workspace must be 16-byte aligned", what);
    return DG_OK;
}

dg_status check_teacher(const char *what, int64_t R, const int32_t *indices, const float *teacher, int32_t K,
                        int64_t ldk) {
    if (K < 1 || ldk < K) return fail(DG_ERR_INVALID_ARG, "%s: need K >= 1 and ldk >= K", what);
    if (K > kMaxTopK) return fail(DG_ERR_UNSUPPORTED, "%s: K = %d is above %d", what, K, kMaxTopK);
    if (ldk > (1LL << 31)) return fail(DG_ERR_UNSUPPORTED, "%s: ldk too large", what);
    if (R > 0 && (!indices || !teacher)) return fail(DG_ERR_INVALID_ARG, "%s: indices or teacher is NULL", what);
    return DG_OK;
}

RowLossArgs row_args(const void *logits, int32_t dtype, int64_t R, int64_t V, int64_t ldl, float temperature,
                     const float *weight, void *grad, int64_t ldg) {
    RowLossArgs a{};
    a.logits = logits;
    a.dtype = dtype;
    a.R = R;
    a.V = V;
    a.ldl = ldl;
    a.T = temperature;
    a.weight = weight;
    a.grad = grad;
    a.ldg = ldg;
    return a;
}

dg_status run(const char *what, const RowLossArgs &a, RowLossHead head, RowLossPass pass, void *workspace,
              size_t workspace_bytes, dg_stream_t stream, bool chained = false) {
    const dg_status st = check_workspace(what, a, head, pass, workspace, workspace_bytes);
    if (st != DG_OK) return st;
    const cudaError_t e = launch_row_loss(a, head, pass, workspace, (cudaStream_t)stream, chained);
    return e == cudaSuccess ? DG_OK : cuda_fail(e, what);
}

}  // namespace
}  // namespace dg

using namespace dg;

extern "C" {

size_t dg_row_topk_workspace_size(int64_t R, int64_t V, int32_t K, int32_t dtype) {
    if (R < 1 || R > (1LL << 28) || V < 1 || V > 0x7ffffff0LL || K < 1 || K > kMaxTopK || K > V ||
        (dtype != DG_F32 && dtype != DG_BF16))
        return 0;
    return row_topk_workspace_bytes(R, V, K, dtype);
}

size_t dg_row_loss_workspace_size(int64_t R, int64_t V, int32_t dtype) {
    if (R < 1 || R > (1LL << 28) || V < 1 || V > 0x7ffffff0LL || (dtype != DG_F32 && dtype != DG_BF16)) return 0;
    return row_loss_workspace_bytes(R, V, dtype);
}

int32_t dg_row_loss_needs_workspace(int64_t V, int32_t dtype) {
    return V >= 1 && V <= 0x7ffffff0LL && (dtype == DG_F32 || dtype == DG_BF16) &&
           takes_workspace(V, element_size(dtype), kHeadToken, kPassForward);
}

dg_status dg_row_topk(const void *logits, int32_t dtype, int64_t R, int64_t V, int64_t ldl, int32_t K,
                      float temperature, float *values, int32_t *indices, int64_t ldk, float *lse, void *workspace,
                      size_t workspace_bytes, dg_stream_t stream) {
    t_last_error[0] = 0;
    const char *what = "row topk";
    dg_status st = check_rows(what, logits, dtype, R, V, ldl, temperature);
    if (st != DG_OK) return st;
    if (K < 1 || K > V || ldk < K) return fail(DG_ERR_INVALID_ARG, "%s: need 1 <= K <= V and ldk >= K", what);
    if (K > kMaxTopK) return fail(DG_ERR_UNSUPPORTED, "%s: K = %d is above %d", what, K, kMaxTopK);
    if (ldk > (1LL << 31)) return fail(DG_ERR_UNSUPPORTED, "%s: ldk too large", what);
    if (!row_topk_fits(R, V, dtype)) return fail(DG_ERR_UNSUPPORTED, "%s: more than 16 TiB of rows", what);
    if (R == 0) return DG_OK;
    if (!values || !indices) return fail(DG_ERR_INVALID_ARG, "%s: an output pointer is NULL", what);
    const size_t need = row_topk_workspace_bytes(R, V, K, dtype);
    if (need == 0) return fail(DG_ERR_CUDA, "%s: no CUDA device", what);
    if (!workspace || workspace_bytes < need)
        return fail(DG_ERR_INVALID_ARG, "%s: workspace of %zu bytes is below the %zu needed", what, workspace_bytes,
                    need);
    if (!aligned16(workspace)) return fail(DG_ERR_UNSUPPORTED, "%s: workspace must be 16-byte aligned", what);
    const RowTopKArgs a{logits, ldl, dtype, R, V, K, temperature, values, indices, ldk, lse};
    const cudaError_t e = launch_row_topk(a, workspace, (cudaStream_t)stream);
    return e == cudaSuccess ? DG_OK : cuda_fail(e, what);
}

dg_status dg_token_logp(const void *logits, int32_t dtype, int64_t R, int64_t V, int64_t ldl, const int32_t *token,
                        float temperature, const float *weight, float *logp, float *lse, void *workspace,
                        size_t workspace_bytes, dg_stream_t stream) {
    t_last_error[0] = 0;
    const char *what = "token logp";
    dg_status st = check_rows(what, logits, dtype, R, V, ldl, temperature);
    if (st != DG_OK || R == 0) return st;
    if (!token) return fail(DG_ERR_INVALID_ARG, "%s: token is NULL", what);
    RowLossArgs a = row_args(logits, dtype, R, V, ldl, temperature, weight, nullptr, 0);
    a.token = token;
    a.logp = logp;
    a.lse = lse;
    return run(what, a, kHeadToken, kPassForward, workspace, workspace_bytes, stream);
}

dg_status dg_token_logp_backward(const void *logits, int32_t dtype, int64_t R, int64_t V, int64_t ldl,
                                 const int32_t *token, float temperature, const float *lse, const float *dlogp,
                                 const float *weight, void *grad, int64_t ldg, void *workspace,
                                 size_t workspace_bytes, dg_stream_t stream) {
    t_last_error[0] = 0;
    const char *what = "token logp backward";
    dg_status st = check_rows(what, logits, dtype, R, V, ldl, temperature);
    if (st != DG_OK || R == 0) return st;
    if (!token || !lse || !dlogp) return fail(DG_ERR_INVALID_ARG, "%s: token, lse or dlogp is NULL", what);
    st = check_grad(what, logits, dtype, R, V, ldl, grad, ldg);
    if (st != DG_OK) return st;
    RowLossArgs a = row_args(logits, dtype, R, V, ldl, temperature, weight, grad, ldg);
    a.token = token;
    a.lse = const_cast<float *>(lse);
    a.dlogp = const_cast<float *>(dlogp);
    return run(what, a, kHeadToken, kPassBackward, workspace, workspace_bytes, stream);
}

dg_status dg_distill_loss(const void *logits, int32_t dtype, int64_t R, int64_t V, int64_t ldl,
                          const int32_t *indices, const float *teacher, int32_t K, int64_t ldk,
                          const float *teacher_lse, float temperature, const float *weight, float *loss, float *lse,
                          float *tail_logp, void *grad, int64_t ldg, void *workspace, size_t workspace_bytes,
                          dg_stream_t stream) {
    t_last_error[0] = 0;
    const char *what = "distill loss";
    dg_status st = check_rows(what, logits, dtype, R, V, ldl, temperature);
    if (st == DG_OK) st = check_teacher(what, R, indices, teacher, K, ldk);
    if (st != DG_OK || R == 0) return st;
    if (grad) st = check_grad(what, logits, dtype, R, V, ldl, grad, ldg);
    if (st != DG_OK) return st;
    RowLossArgs a = row_args(logits, dtype, R, V, ldl, temperature, weight, grad, ldg);
    a.indices = indices;
    a.teacher = teacher;
    a.K = K;
    a.ldk = ldk;
    a.teacher_lse = teacher_lse;
    a.loss = loss;
    a.lse = lse;
    a.tail_logp = teacher_lse ? tail_logp : nullptr;
    return run(what, a, kHeadDistill, grad ? kPassStep : kPassForward, workspace, workspace_bytes, stream);
}

dg_status dg_distill_loss_backward(const void *logits, int32_t dtype, int64_t R, int64_t V, int64_t ldl,
                                   const int32_t *indices, const float *teacher, int32_t K, int64_t ldk,
                                   const float *teacher_lse, float temperature, const float *lse,
                                   const float *tail_logp, const float *dloss, void *grad, int64_t ldg,
                                   void *workspace, size_t workspace_bytes, dg_stream_t stream) {
    t_last_error[0] = 0;
    const char *what = "distill loss backward";
    dg_status st = check_rows(what, logits, dtype, R, V, ldl, temperature);
    if (st == DG_OK) st = check_teacher(what, R, indices, teacher, K, ldk);
    if (st != DG_OK || R == 0) return st;
    if (!lse) return fail(DG_ERR_INVALID_ARG, "%s: lse is NULL", what);
    if (teacher_lse && !tail_logp)
        return fail(DG_ERR_INVALID_ARG, "%s: teacher_lse needs the forward call's tail_logp", what);
    st = check_grad(what, logits, dtype, R, V, ldl, grad, ldg);
    if (st != DG_OK) return st;
    RowLossArgs a = row_args(logits, dtype, R, V, ldl, temperature, dloss, grad, ldg);
    a.indices = indices;
    a.teacher = teacher;
    a.K = K;
    a.ldk = ldk;
    a.teacher_lse = teacher_lse;
    a.lse = const_cast<float *>(lse);
    a.tail_logp = const_cast<float *>(tail_logp);
    return run(what, a, kHeadDistill, kPassBackward, workspace, workspace_bytes, stream);
}

dg_status dg_policy_loss(const void *logits, int32_t dtype, int64_t R, int64_t V, int64_t ldl, const int32_t *token,
                         const float *old_logp, const float *ref_logp, const float *advantage, float temperature,
                         float clip_low, float clip_high, float kl_coef, const float *weight, float *loss,
                         float *logp, float *lse, float *kl, uint8_t *clipped, float *dlogp, void *grad, int64_t ldg,
                         void *workspace, size_t workspace_bytes, dg_stream_t stream) {
    t_last_error[0] = 0;
    const char *what = "policy loss";
    dg_status st = check_rows(what, logits, dtype, R, V, ldl, temperature);
    if (st != DG_OK) return st;
    if (!(clip_low >= 0.0f && clip_low <= 1.0f) || !(clip_high >= 0.0f && clip_high < INFINITY) ||
        !(kl_coef >= 0.0f && kl_coef < INFINITY))
        return fail(DG_ERR_INVALID_ARG, "%s: need 0 <= clip_low <= 1, clip_high >= 0, kl_coef >= 0, finite", what);
    if (R == 0) return DG_OK;
    if (!token || !old_logp || !advantage)
        return fail(DG_ERR_INVALID_ARG, "%s: token, old_logp or advantage is NULL", what);
    if (grad) st = check_grad(what, logits, dtype, R, V, ldl, grad, ldg);
    if (st != DG_OK) return st;
    RowLossArgs a = row_args(logits, dtype, R, V, ldl, temperature, weight, grad, ldg);
    a.policy = true;
    a.token = token;
    a.old_logp = old_logp;
    a.ref_logp = ref_logp;
    a.advantage = advantage;
    a.clip_low = clip_low;
    a.clip_high = clip_high;
    a.kl_coef = kl_coef;
    a.loss = loss;
    a.logp = logp;
    a.lse = lse;
    a.kl = kl;
    a.clipped = clipped;
    a.dlogp = dlogp;
    return run(what, a, kHeadToken, grad ? kPassStep : kPassForward, workspace, workspace_bytes, stream);
}

dg_status dg_preference_loss(const void *logits, int32_t dtype, int64_t R, int64_t V, int64_t ldl,
                             const int32_t *token, const float *ref_logp, const int32_t *seq_start, int32_t P,
                             float beta, float label_smoothing, float temperature, const float *weight,
                             const float *pair_weight, float *loss, float *log_ratio, float *logp, float *lse,
                             float *dlogp, void *grad, int64_t ldg, void *workspace, size_t workspace_bytes,
                             dg_stream_t stream) {
    t_last_error[0] = 0;
    const char *what = "preference loss";
    dg_status st = check_rows(what, logits, dtype, R, V, ldl, temperature);
    if (st != DG_OK) return st;
    if (P < 0 || !std::isfinite(beta) || !(label_smoothing >= 0.0f && label_smoothing < 1.0f))
        return fail(DG_ERR_INVALID_ARG, "%s: need P >= 0, a finite beta and 0 <= label_smoothing < 1", what);
    if (P > (1 << 28)) return fail(DG_ERR_UNSUPPORTED, "%s: P too large", what);
    if (R > 0 && (!token || !logp || !lse || !dlogp))
        return fail(DG_ERR_INVALID_ARG, "%s: token, logp, lse or dlogp is NULL", what);
    if (P > 0 && (!seq_start || !loss)) return fail(DG_ERR_INVALID_ARG, "%s: seq_start or loss is NULL", what);
    if (R > 0 && grad) st = check_grad(what, logits, dtype, R, V, ldl, grad, ldg);
    if (st != DG_OK) return st;
    RowLossArgs a = row_args(logits, dtype, R, V, ldl, temperature, weight, nullptr, 0);
    a.token = token;
    a.logp = logp;
    a.lse = lse;
    a.dlogp = dlogp;
    a.keep_low = P > 0;  // until the pairs' kernel has added it up; without pairs 0
    if (R > 0) st = run(what, a, kHeadToken, kPassForward, workspace, workspace_bytes, stream);
    if (st != DG_OK) return st;
    if (P > 0) {
        const PairLossArgs pa{logp, ref_logp, weight,          token,       seq_start, R, V, P,
                              beta, label_smoothing, pair_weight, loss, log_ratio, dlogp};
        const cudaError_t e = launch_pair_loss(pa, (cudaStream_t)stream);
        if (e != cudaSuccess) return cuda_fail(e, "preference loss: pairs");
    }
    if (R == 0 || !grad) return DG_OK;
    a.weight = nullptr;  // dlogp holds it
    a.grad = grad;
    a.ldg = ldg;
    return run(what, a, kHeadToken, kPassBackward, workspace, workspace_bytes, stream, P > 0);
}

}  // extern "C"
