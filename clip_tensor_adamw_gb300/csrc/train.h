// What the operators' host side (train_api.cpp) and kernels (logits.cu, packed.cu, wgrad.cu) share: the arguments of a
// launch, already checked, and the launch functions. Each returns a cudaError_t as int.
#pragma once

#include <cstdint>

#include "mica_train.h"

namespace mica {

struct LogitRows {
    const void* z;
    const void* targets;
    int64_t rows;
    int64_t ld;
    int32_t vocab;
    int32_t dtype;
    int32_t wide_targets;  // int64 targets
    float inv_t;           // 1 / temperature
    double wide_inv_t;
    // log2(e) / temperature, rounded, and as a_hi + a_lo with a_lo > 0: exp((z - origin) / temperature) =
    // 2^((z - origin) * (a_hi + a_lo))
    float a, a_hi, a_lo;
};

// A row's softmax statistics: the logit that its weights are counted from (the largest; -inf: nothing but that in the row),
// and 1 over their sum.
struct RowStat {
    float origin;
    float inv_sum;
};

struct PolicyTerms {
    const float* old_logps;
    const float* advantages;
    const float* ref_logps;  // or null
    const float* weights;    // or null
    float lo, hi, kl_coef, inv_denom;
    float grad_factor;  // grad_scale / (denom * temperature)
};

// logps, and where not null entropies, of every row; without entropies also, where not null, what rounding took from the
// logps, and the softmax statistics
int launch_row_logps(const LogitRows& L, float* logps, float* rest_logps, float* entropy, RowStat* stat, void* stream);
// dz = coef * ((j == target) - p): coef[row] * factor given, the softmax computed here
int launch_row_softmax_grad(const LogitRows& L, const float* coef, float factor, void* dz, int64_t ld_d, void* stream);
// the same with the coefficient of the policy loss, from the log-probability found on the way (also written)
int launch_row_policy_grad(const LogitRows& L, const PolicyTerms& P, float* logps, void* dz, int64_t ld_d, void* stream);
// the same with the softmax statistics and the whole coefficient given
int launch_row_grad(const LogitRows& L, const RowStat* stat, const float* coef, void* dz, int64_t ld_d, void* stream);
int launch_policy_sums(const LogitRows& L, const PolicyTerms& P, const float* logps, float* stats, void* stream);

struct PairTerms {
    const int32_t* cu_seqlens;
    const float* ref_logps;  // or null
    int32_t pairs;
    int32_t kind;
    int32_t length_norm;
    float beta, smoothing;
    float grad_factor;  // grad_scale / (pairs * temperature)
};
// loss, rewards (or null) and, where coef is not null, each row's coefficient, from the logps and their rests; sums: 6 * pairs
// floats of workspace
int launch_pairs(const LogitRows& L, const PairTerms& P, const float* logps, const float* rest, float* sums, float* loss,
                 float* rewards, float* coef, void* stream);

int launch_act_pack(const void* x, int64_t ld_x, const mica_packed& p, int32_t act, bool gated, void* y, int64_t ld_y,
                    void* stream);
int launch_act_unpack(const mica_packed& p, void* x, int64_t ld_x, void* stream);
int launch_act_grad(const mica_packed& p, int32_t act, bool gated, const void* dy, int64_t ld_dy, int32_t dtype, void* dx,
                    int64_t ld_dx, void* stream);

struct Wgrad {
    mica_packed x;
    const void* dy;
    int64_t ld_dy;
    int32_t dy_dtype;
    int32_t dw_dtype;
    int64_t n;
    const void* add;
    int64_t ld_add;
    void* dw;
    int64_t ld_dw;
};
// The status words of these kernels' bounded waits, as read_device_status (plan.h); 0, and nothing is copied, in a process
// that has launched none of them.
int read_logits_status(unsigned int* status);
int read_wgrad_status(unsigned int* status);

int64_t wgrad_workspace(int64_t tokens, int64_t features, int64_t n, const void* dy, int64_t ld_dy, int sms);
int launch_wgrad(const Wgrad& w, void* workspace, int sms, void* stream);

}  // namespace mica
