// The C ABI of include/mica_train.h: host-side validation and the launches of the loss operators and the 8-bit
// activation checkpoints.
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>
#include <limits>

#include "checks.h"
#include "host.h"
#include "mica_train.h"
#include "plan.h"
#include "train.h"

namespace mica {
namespace {

mica_status check_logits(const mica_logits* z, LogitRows* L) {
    if (!z) return fail(MICA_ERR_NULL, "the logits are NULL");
    if (!is_type(z->dtype)) return fail(MICA_ERR_DTYPE, "logits must be float32, float16 or bfloat16");
    if (z->target_bytes != 4 && z->target_bytes != 8) return fail(MICA_ERR_DTYPE, "targets must be int32 or int64");
    if (!std::isfinite(z->temperature) || !(z->temperature > 0.0))
        return fail(MICA_ERR_HYPER, "temperature %g is not finite and > 0", z->temperature);
    if (!(z->temperature >= 1e-30 && z->temperature <= 1e30))
        return fail(MICA_ERR_HYPER, "temperature %g is outside [1e-30, 1e30]", z->temperature);
    const double a = 1.4426950408889634074 / z->temperature;
    float a_hi = (float)a;  // the largest float32 below a, so that the rest is positive
    if (a_hi >= a) a_hi = std::nextafter(a_hi, 0.0f);
    const float a_lo = std::fmax((float)(a - a_hi), std::numeric_limits<float>::denorm_min());
    MICA_TRY(check_extent(z->rows, z->vocab, 1, "logits"));
    MICA_TRY(check_stride(z->ld, 0, z->rows, z->vocab, "logits"));
    *L = LogitRows{z->logits, z->targets, z->rows, z->ld, (int32_t)z->vocab, z->dtype, z->target_bytes == 8,
                   (float)(1.0 / z->temperature), 1.0 / z->temperature, (float)a, a_hi, a_lo};
    return MICA_OK;
}

mica_status add_logits(const mica_logits* z, Buffers* b) {
    MICA_TRY(b->matrix(z->logits, z->rows, z->vocab, z->ld, bytes_of(z->dtype), bytes_of(z->dtype), false, "logits"));
    return b->vec(z->targets, z->rows, (size_t)z->target_bytes, false, "targets");
}

// dlogits: the logits' type; in place when it is the logits' buffer with their stride
mica_status add_dlogits(const mica_logits* z, void* d, int64_t ld_d, Buffers* b) {
    const size_t es = bytes_of(z->dtype);
    if (d && d == z->logits && ld_d == z->ld) b->in_place(d);
    return b->matrix(d, z->rows, z->vocab, ld_d, es, es, true, "dlogits");
}

size_t round16(size_t n) { return (n + 15) / 16 * 16; }

mica_status check_packed(const mica_packed* p, const char* what) {
    if (!p) return fail(MICA_ERR_NULL, "%s is NULL", what);
    if (!is_type(p->dtype)) return fail(MICA_ERR_DTYPE, "%s: the source's type must be float32, float16 or bfloat16", what);
    MICA_TRY(check_extent(p->rows, p->cols, 0, what));
    MICA_TRY(check_stride(p->ld, p->cols, p->rows, p->cols, "codes"));
    MICA_TRY(check_stride(p->ld_s, (p->cols + 31) / 32, p->rows, p->cols, "steps"));
    if (p->ld % 32) return fail(MICA_ERR_COUNT, "codes: the row stride %lld is not a multiple of 32", (long long)p->ld);
    if (p->ld_s % 4) return fail(MICA_ERR_COUNT, "steps: the row stride %lld is not a multiple of 4", (long long)p->ld_s);
    return MICA_OK;
}

mica_status add_packed(const mica_packed* p, bool written, Buffers* b) {
    const int64_t blocks = (p->cols + 31) / 32;
    MICA_TRY(b->matrix(p->codes, p->rows, blocks * 32, p->ld, 1, 16, written, "codes"));
    // (four steps are read at a time; only a row's blocks are written)
    return b->matrix(p->steps, p->rows, written ? blocks : (blocks + 3) / 4 * 4, p->ld_s, 1, 4, written, "steps");
}

mica_status check_act(const mica_packed* p, int32_t act, int32_t gated, int32_t least) {
    if (act < least || act > MICA_ACT_RELU) return fail(MICA_ERR_HYPER, "act %d is not an activation this call takes", act);
    if (gated && act == MICA_ACT_NONE) return fail(MICA_ERR_HYPER, "a gated unit needs an activation function");
    if (gated && p->cols % 64)
        return fail(MICA_ERR_COUNT, "a gated unit's %lld columns are not twice a multiple of 32", (long long)p->cols);
    return MICA_OK;
}

}  // namespace
}  // namespace mica

using namespace mica;

extern "C" mica_status mica_token_logps(const mica_logits* z, float* logps, float* entropy, void* stream) {
    LogitRows L;
    MICA_TRY(check_logits(z, &L));
    if (z->rows == 0) return ok();
    int dev = 0;
    MICA_TRY(current_device(&dev));
    Buffers b(dev);
    MICA_TRY(add_logits(z, &b));
    MICA_TRY(b.vec(logps, z->rows, 4, true, "logps"));
    if (entropy) MICA_TRY(b.vec(entropy, z->rows, 4, true, "entropy"));
    MICA_TRY(b.disjoint());
    return after_launch(launch_row_logps(L, logps, nullptr, entropy, nullptr, stream), stream, "token log-probabilities launch");
}

extern "C" mica_status mica_token_logps_grad(const mica_logits* z, const float* dlogps, void* dlogits, int64_t ld_d,
                                             void* stream) {
    LogitRows L;
    MICA_TRY(check_logits(z, &L));
    MICA_TRY(check_stride(ld_d, z->vocab, z->rows, z->vocab, "dlogits"));
    if (z->rows == 0) return ok();
    int dev = 0;
    MICA_TRY(current_device(&dev));
    Buffers b(dev);
    MICA_TRY(add_logits(z, &b));
    MICA_TRY(b.vec(dlogps, z->rows, 4, false, "dlogps"));
    MICA_TRY(add_dlogits(z, dlogits, ld_d, &b));
    MICA_TRY(b.disjoint());
    return after_launch(launch_row_softmax_grad(L, dlogps, L.inv_t, dlogits, ld_d, stream), stream,
                        "log-probabilities' gradient launch");
}

// workspace: three floats per sequence | a RowStat, the rest of a log-probability and a coefficient per row
extern "C" int64_t mica_preference_workspace(int64_t rows, int32_t pairs) {
    if (rows < 0 || rows > MICA_MAX_ROWS || pairs < 0 || pairs > (1 << 24)) return 0;
    return (int64_t)((size_t)pairs * 6 * sizeof(float) + round16((size_t)rows * (sizeof(RowStat) + 2 * sizeof(float))));
}

extern "C" mica_status mica_preference_loss(const mica_logits* z, const int32_t* cu_seqlens, int32_t pairs,
                                            const float* ref_logps, const mica_preference_hp* hp, float* loss,
                                            float* rewards, float* logps, void* dlogits, int64_t ld_d, void* workspace,
                                            int64_t workspace_bytes, void* stream) {
    LogitRows L;
    MICA_TRY(check_logits(z, &L));
    if (!hp) return fail(MICA_ERR_NULL, "hp is NULL");
    if (pairs < 0 || pairs > (1 << 24)) return fail(MICA_ERR_COUNT, "pairs = %d is outside [0, 2^24]", pairs);
    if (!std::isfinite(hp->beta) || !(hp->beta > 0.0)) return fail(MICA_ERR_HYPER, "beta %g is not finite and > 0", hp->beta);
    if (hp->kind < MICA_PREF_SIGMOID || hp->kind > MICA_PREF_IPO)
        return fail(MICA_ERR_HYPER, "kind %d is not a preference loss", hp->kind);
    if (!(hp->label_smoothing >= 0.0 && hp->label_smoothing < 1.0))
        return fail(MICA_ERR_HYPER, "label_smoothing %g is outside [0, 1)", hp->label_smoothing);
    if (hp->label_smoothing != 0.0 && hp->kind != MICA_PREF_SIGMOID)
        return fail(MICA_ERR_HYPER, "label_smoothing goes with the sigmoid loss only");
    if (!std::isfinite(hp->grad_scale)) return fail(MICA_ERR_HYPER, "grad_scale %g is not finite", hp->grad_scale);
    if (hp->flags & ~MICA_PREF_LENGTH_NORM) return fail(MICA_ERR_HYPER, "unknown flags 0x%x", hp->flags);
    if (dlogits) MICA_TRY(check_stride(ld_d, z->vocab, z->rows, z->vocab, "dlogits"));
    const int64_t need = mica_preference_workspace(z->rows, pairs);
    if (need && !workspace) return fail(MICA_ERR_NULL, "workspace is NULL");
    if (workspace_bytes < need)
        return fail(MICA_ERR_COUNT, "the workspace has %lld bytes of %lld", (long long)workspace_bytes, (long long)need);
    int dev = 0;
    MICA_TRY(current_device(&dev));
    Buffers b(dev);
    MICA_TRY(add_logits(z, &b));
    MICA_TRY(b.vec(cu_seqlens, pairs ? 2 * (int64_t)pairs + 1 : 0, 4, false, "cu_seqlens"));
    if (ref_logps) MICA_TRY(b.vec(ref_logps, z->rows, 4, false, "ref_logps"));
    MICA_TRY(b.vec(loss, 1, 4, true, "loss"));
    if (rewards) MICA_TRY(b.vec(rewards, 2 * (int64_t)pairs, 4, true, "rewards"));
    MICA_TRY(b.vec(logps, z->rows, 4, true, "logps"));
    if (dlogits) MICA_TRY(add_dlogits(z, dlogits, ld_d, &b));
    MICA_TRY(b.matrix(workspace, 1, need, need, 1, 16, true, "workspace"));
    MICA_TRY(b.disjoint());

    float* sums = static_cast<float*>(workspace);
    RowStat* stat = reinterpret_cast<RowStat*>(sums + 6 * (size_t)pairs);
    float* rest = reinterpret_cast<float*>(stat + z->rows);
    float* coef = rest + z->rows;
    const PairTerms P{cu_seqlens, ref_logps, pairs, hp->kind, (hp->flags & MICA_PREF_LENGTH_NORM) != 0,
                      (float)hp->beta, (float)hp->label_smoothing,
                      pairs ? (float)(hp->grad_scale / pairs / z->temperature) : 0.0f};
    if (z->rows)
        MICA_TRY(after_launch(launch_row_logps(L, logps, rest, nullptr, dlogits ? stat : nullptr, stream), stream,
                              "log-probabilities launch"));
    MICA_TRY(after_launch(launch_pairs(L, P, logps, rest, sums, loss, rewards, dlogits ? coef : nullptr, stream), stream,
                          "preference pairs launch"));
    if (!dlogits || z->rows == 0) return ok();
    return after_launch(launch_row_grad(L, stat, coef, dlogits, ld_d, stream), stream, "preference gradient launch");
}

extern "C" mica_status mica_policy_loss(const mica_logits* z, const float* old_logps, const float* advantages,
                                        const float* ref_logps, const float* weights, const mica_policy_hp* hp,
                                        float* stats, float* logps, void* dlogits, int64_t ld_d, void* stream) {
    LogitRows L;
    MICA_TRY(check_logits(z, &L));
    if (!hp) return fail(MICA_ERR_NULL, "hp is NULL");
    if (!(hp->clip_low >= 0.0 && hp->clip_low <= 1.0))
        return fail(MICA_ERR_HYPER, "clip_low %g is outside [0, 1]", hp->clip_low);
    if (!(hp->clip_high >= 0.0)) return fail(MICA_ERR_HYPER, "clip_high %g is not >= 0", hp->clip_high);
    if (!std::isfinite(hp->kl_coef) || hp->kl_coef < 0.0)
        return fail(MICA_ERR_HYPER, "kl_coef %g is not finite and >= 0", hp->kl_coef);
    if (!std::isfinite(hp->denom) || !(hp->denom > 0.0)) return fail(MICA_ERR_HYPER, "denom %g is not finite and > 0", hp->denom);
    if (!std::isfinite(hp->grad_scale)) return fail(MICA_ERR_HYPER, "grad_scale %g is not finite", hp->grad_scale);
    if (dlogits) MICA_TRY(check_stride(ld_d, z->vocab, z->rows, z->vocab, "dlogits"));
    int dev = 0;
    MICA_TRY(current_device(&dev));
    Buffers b(dev);
    MICA_TRY(add_logits(z, &b));
    MICA_TRY(b.vec(old_logps, z->rows, 4, false, "old_logps"));
    MICA_TRY(b.vec(advantages, z->rows, 4, false, "advantages"));
    if (ref_logps) MICA_TRY(b.vec(ref_logps, z->rows, 4, false, "ref_logps"));
    if (weights) MICA_TRY(b.vec(weights, z->rows, 4, false, "weights"));
    MICA_TRY(b.vec(stats, 4, 4, true, "stats"));
    MICA_TRY(b.vec(logps, z->rows, 4, true, "logps"));
    if (dlogits) MICA_TRY(add_dlogits(z, dlogits, ld_d, &b));
    MICA_TRY(b.disjoint());

    const PolicyTerms P{old_logps, advantages, ref_logps, weights, (float)(1.0 - hp->clip_low),
                        (float)(1.0 + hp->clip_high), (float)hp->kl_coef, (float)(1.0 / hp->denom),
                        (float)(hp->grad_scale / hp->denom / z->temperature)};
    if (z->rows)
        MICA_TRY(after_launch(dlogits ? launch_row_policy_grad(L, P, logps, dlogits, ld_d, stream)
                                      : launch_row_logps(L, logps, nullptr, nullptr, nullptr, stream),
                              stream, "policy loss launch"));
    return after_launch(launch_policy_sums(L, P, logps, stats, stream), stream, "policy sums launch");
}

extern "C" mica_status mica_act_pack(const void* x, int64_t ld_x, const mica_packed* p, int32_t act, int32_t gated, void* y,
                                     int64_t ld_y, void* stream) {
    MICA_TRY(check_packed(p, "the checkpoint"));
    MICA_TRY(check_act(p, act, gated, MICA_ACT_NONE));
    const int64_t out = gated ? p->cols / 2 : p->cols;
    const size_t es = bytes_of(p->dtype);
    MICA_TRY(check_stride(ld_x, 0, p->rows, p->cols, "x"));
    if (act != MICA_ACT_NONE) MICA_TRY(check_stride(ld_y, out, p->rows, out, "y"));
    else if (y) return fail(MICA_ERR_HYPER, "y is given without an activation function");
    if (p->rows == 0 || p->cols == 0) return ok();
    int dev = 0;
    MICA_TRY(current_device(&dev));
    Buffers b(dev);
    MICA_TRY(b.matrix(x, p->rows, p->cols, ld_x, es, es, false, "x"));
    MICA_TRY(add_packed(p, true, &b));
    if (act != MICA_ACT_NONE) MICA_TRY(b.matrix(y, p->rows, out, ld_y, es, es, true, "y"));
    MICA_TRY(b.disjoint());
    return after_launch(launch_act_pack(x, ld_x, *p, act, gated != 0, y, ld_y, stream), stream, "activation pack launch");
}

extern "C" mica_status mica_act_unpack(const mica_packed* p, void* x, int64_t ld_x, void* stream) {
    MICA_TRY(check_packed(p, "the checkpoint"));
    MICA_TRY(check_stride(ld_x, p->cols, p->rows, p->cols, "x"));
    if (p->rows == 0 || p->cols == 0) return ok();
    int dev = 0;
    MICA_TRY(current_device(&dev));
    Buffers b(dev);
    MICA_TRY(add_packed(p, false, &b));
    MICA_TRY(b.matrix(x, p->rows, p->cols, ld_x, bytes_of(p->dtype), bytes_of(p->dtype), true, "x"));
    MICA_TRY(b.disjoint());
    return after_launch(launch_act_unpack(*p, x, ld_x, stream), stream, "activation unpack launch");
}

extern "C" mica_status mica_act_grad(const mica_packed* p, int32_t act, int32_t gated, const void* dy, int64_t ld_dy,
                                     int32_t dtype, void* dx, int64_t ld_dx, void* stream) {
    MICA_TRY(check_packed(p, "the checkpoint"));
    MICA_TRY(check_act(p, act, gated, MICA_ACT_GELU_TANH));
    if (!is_type(dtype)) return fail(MICA_ERR_DTYPE, "dy must be float32, float16 or bfloat16");
    const int64_t in = gated ? p->cols / 2 : p->cols;
    MICA_TRY(check_stride(ld_dy, 0, p->rows, in, "dy"));
    MICA_TRY(check_stride(ld_dx, p->cols, p->rows, p->cols, "dx"));
    if (p->rows == 0 || p->cols == 0) return ok();
    int dev = 0;
    MICA_TRY(current_device(&dev));
    Buffers b(dev);
    MICA_TRY(add_packed(p, false, &b));
    MICA_TRY(b.matrix(dy, p->rows, in, ld_dy, bytes_of(dtype), bytes_of(dtype), false, "dy"));
    MICA_TRY(b.matrix(dx, p->rows, p->cols, ld_dx, bytes_of(dtype), bytes_of(dtype), true, "dx"));
    if (!gated && dx == dy && ld_dx == ld_dy) b.in_place(dx);
    MICA_TRY(b.disjoint());
    return after_launch(launch_act_grad(*p, act, gated != 0, dy, ld_dy, dtype, dx, ld_dx, stream), stream,
                        "activation gradient launch");
}

extern "C" int64_t mica_packed_wgrad_workspace(const mica_packed* x, const void* dy, int64_t ld_dy, int64_t n) {
    int dev = 0;
    if (check_packed(x, "the checkpoint") != MICA_OK || n < 0 || n > MICA_MAX_COLS ||
        check_stride(n, n, x->cols, n, "dw") != MICA_OK || current_device(&dev) != MICA_OK)
        return 0;
    return wgrad_workspace(x->rows, x->cols, n, dy, ld_dy, sm_count(dev));
}

extern "C" mica_status mica_packed_wgrad(const mica_packed* x, const void* dy, int64_t ld_dy, int32_t dy_dtype, int64_t n,
                                         const void* add, int64_t ld_add, void* dw, int64_t ld_dw, int32_t dw_dtype,
                                         void* workspace, int64_t workspace_bytes, void* stream) {
    MICA_TRY(check_packed(x, "the checkpoint"));
    if (dy_dtype != MICA_BF16 && dy_dtype != MICA_F16) return fail(MICA_ERR_DTYPE, "dy must be bfloat16 or float16");
    if (dy_dtype == MICA_F16 && x->dtype != MICA_F16)
        return fail(MICA_ERR_DTYPE, "a float16 dy needs the checkpoint of a float16 activation");
    if (!is_type(dw_dtype)) return fail(MICA_ERR_DTYPE, "dw must be float32, float16 or bfloat16");
    MICA_TRY(check_extent(x->rows, n, 0, "dy"));
    MICA_TRY(check_stride(ld_dy, 0, x->rows, n, "dy"));
    MICA_TRY(check_stride(ld_dw, n, x->cols, n, "dw"));
    if (add) MICA_TRY(check_stride(ld_add, 0, x->cols, n, "add"));
    if (x->cols == 0 || n == 0) return ok();
    int dev = 0;
    MICA_TRY(current_device(&dev));
    const int sms = sm_count(dev);
    const int64_t need = wgrad_workspace(x->rows, x->cols, n, dy, ld_dy, sms);
    if (need && !workspace) return fail(MICA_ERR_NULL, "workspace is NULL");
    if (workspace_bytes < need)
        return fail(MICA_ERR_COUNT, "the workspace has %lld bytes of %lld", (long long)workspace_bytes, (long long)need);
    const size_t es = bytes_of(dw_dtype);
    Buffers b(dev);
    MICA_TRY(add_packed(x, false, &b));
    MICA_TRY(b.matrix(dy, x->rows, n, ld_dy, 2, 2, false, "dy"));
    if (add) MICA_TRY(b.matrix(add, x->cols, n, ld_add, es, es, false, "add"));
    MICA_TRY(b.matrix(dw, x->cols, n, ld_dw, es, es, true, "dw"));
    if (add == dw && ld_add == ld_dw) b.in_place(dw);
    MICA_TRY(b.matrix(workspace, 1, need, need, 1, 16, true, "workspace"));
    MICA_TRY(b.disjoint());
    const Wgrad w{*x, dy, ld_dy, dy_dtype, dw_dtype, n, add, ld_add, dw, ld_dw};
    return after_launch(launch_wgrad(w, workspace, sms, stream), stream, "weight gradient launch");
}
