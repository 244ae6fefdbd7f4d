// Losses on rows of full-vocabulary logits: what the host code and the kernel share.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include <cfloat>
#include <cmath>

#include "../../include/dgsamp.h"
#include "row_loss_plan.h"

namespace dg {

inline int element_size(int dtype) { return dtype == DG_BF16 ? 2 : 4; }

// log2(e) / T.  One float's rounding of it, up to 2^-24, puts a row's log-sum-exp off by that times its
// mean (m - x) / T, and every row's in the same direction, which a sequence's sum of log-probabilities
// shows.  So where such sums are taken, sums of exponentials take it as two floats, hi rounded down, so
// that -inf times either is -inf.  One float is enough where it is too small by 2^-27 to 2^-26, as at
// T = 1: that makes up for most of the hardware's error (row_loss.cu), and saves one operation in six.
struct Scale {
    float hi, lo;
};
inline bool two_floats(float T, Scale *s) {
    const double c = 1.4426950408889634074 / (double)T;
    s->hi = (float)c;
    s->lo = 0.0f;
    const double low = (c - (double)s->hi) / c * (1 << 27);
    if (low >= 1.0 && low <= 2.0) return false;
    if ((double)s->hi > c) s->hi = nextafterf(s->hi, 0.0f);
    s->lo = (float)(c - (double)s->hi);
    return s->lo > 0.0f;
}

struct RowLossArgs {
    const void *logits;  // [R, ldl] fp32 or bf16
    int64_t ldl;
    int dtype;  // dg_dtype, of logits and grad
    int64_t R, V;
    float T;              // temperature
    Scale scale;          // filled in for the kernels that take it
    const float *weight;  // [R] or NULL (1): a row of weight 0 is not read, its outputs are 0
    void *grad;           // [R, ldg] or NULL
    int64_t ldg;
    float *lse;           // [R]: written forward, read backward
    float *loss;          // [R] or NULL
    // kHeadToken
    const int32_t *token;    // [R]; a negative token leaves the row out like weight 0
    bool policy;             // the clipped policy loss; else the log-probability alone
    bool keep_low;           // and then dlogp is what the log-probability's rounding left
    const float *old_logp, *ref_logp, *advantage;
    float clip_low, clip_high, kl_coef;
    float *logp, *kl;
    uint8_t *clipped;
    float *dlogp;  // [R] dloss/dlogp: written forward, read backward (then the coefficient is dlogp * weight)
    // kHeadDistill
    const int32_t *indices;  // [R, ldk]; a negative index leaves the entry out
    const float *teacher;    // [R, ldk]
    int64_t ldk;
    int K;
    const float *teacher_lse;  // [R] or NULL (renormalise over the K entries)
    float *tail_logp;          // [R] ln p_0 with teacher_lse: written forward, read backward
};

size_t row_loss_workspace_bytes(int64_t R, int64_t V, int dtype);
// Takes the workspace where takes_workspace says so, and refuses to start without one there.
// chained: the kernel before it on the stream is one of row_loss.cu's.
cudaError_t launch_row_loss(const RowLossArgs &a, RowLossHead head, RowLossPass pass, void *workspace,
                            cudaStream_t stream, bool chained = false);

// Preference loss of P pairs from the rows' log-probabilities: losses, log ratios, dlogp.
struct PairLossArgs {
    const float *logp, *ref_logp;  // ref_logp may be NULL (0)
    const float *weight;           // [R] or NULL
    const int32_t *token;
    const int32_t *seq_start;      // [2P + 1]
    int64_t R, V;
    int32_t P;
    float beta, label_smoothing;
    const float *pair_weight;  // [P] or NULL
    float *loss, *log_ratio, *dlogp;
};
cudaError_t launch_pair_loss(const PairLossArgs &a, cudaStream_t stream);

// The K largest logits of each row (row_topk.cu).
struct RowTopKArgs {
    const void *logits;
    int64_t ldl;
    int dtype;
    int64_t R, V;
    int K;
    float T;
    float *values;
    int32_t *indices;
    int64_t ldk;
    float *lse;  // [R] or NULL
};
// Whether the rows' 8 KB units can be counted in 32 bits (16 TiB of logits).
bool row_topk_fits(int64_t R, int64_t V, int dtype);
size_t row_topk_workspace_bytes(int64_t R, int64_t V, int K, int dtype);
cudaError_t launch_row_topk(const RowTopKArgs &a, void *workspace, cudaStream_t stream);

}  // namespace dg
