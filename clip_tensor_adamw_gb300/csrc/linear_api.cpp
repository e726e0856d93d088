// The C ABI of the losses from hidden states (include/mica_train.h): host-side validation and launches.
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "checks.h"
#include "linear.h"

namespace mica {
namespace {

mica_status check_linear(const mica_linear* l, Linear* L) {
    if (!l) return fail(MICA_ERR_NULL, "the hidden states are NULL");
    if (l->dtype != MICA_F16 && l->dtype != MICA_BF16)
        return fail(MICA_ERR_DTYPE, "hidden states and embedding must be float16 or bfloat16");
    if (l->target_bytes != 4 && l->target_bytes != 8) return fail(MICA_ERR_DTYPE, "targets must be int32 or int64");
    if (!(l->temperature >= 0x1p-20 && l->temperature <= 0x1p20))
        return fail(MICA_ERR_HYPER, "temperature %g is outside [2^-20, 2^20]", l->temperature);
    MICA_TRY(check_extent(l->rows, l->vocab, 1, "the vocabulary"));
    if (l->features < 1 || l->features > MICA_MAX_FEATURES)
        return fail(MICA_ERR_COUNT, "%lld features are outside [1, 2^16]", (long long)l->features);
    MICA_TRY(check_stride(l->ld_h, 0, l->rows, l->features, "h"));
    MICA_TRY(check_stride(l->ld_w, 0, l->vocab, l->features, "w"));
    *L = Linear{l->h, l->w, l->targets, l->rows, l->ld_h, l->ld_w, (int32_t)l->features, (int32_t)l->vocab, l->dtype,
                l->target_bytes == 8, l->temperature};
    return MICA_OK;
}

mica_status check_grads(const mica_linear* l, const mica_linear_grads* g, LinearGrad* G) {
    *G = LinearGrad{g->dh, g->ld_dh, g->dw, g->ld_dw, g->dw_dtype, g->add, g->ld_add};
    // (without rows dh has no elements, and may be NULL for that)
    if (!g->dh && !g->dw && l->rows > 0) return fail(MICA_ERR_NULL, "neither dh nor dw is given");
    if (g->dh) MICA_TRY(check_stride(g->ld_dh, l->features, l->rows, l->features, "dh"));
    if (!g->dw) {
        if (g->add) return fail(MICA_ERR_NULL, "add is given without dw");
        return MICA_OK;
    }
    if (!is_type(g->dw_dtype)) return fail(MICA_ERR_DTYPE, "dw must be float32, float16 or bfloat16");
    MICA_TRY(check_stride(g->ld_dw, l->features, l->vocab, l->features, "dw"));
    if (g->add) MICA_TRY(check_stride(g->ld_add, 0, l->vocab, l->features, "add"));
    return MICA_OK;
}

mica_status add_inputs(const mica_linear* l, Buffers* b) {
    MICA_TRY(b->matrix(l->h, l->rows, l->features, l->ld_h, 2, 2, false, "h"));
    MICA_TRY(b->matrix(l->w, l->vocab, l->features, l->ld_w, 2, 2, false, "w"));
    return b->vec(l->targets, l->rows, (size_t)l->target_bytes, false, "targets");
}

mica_status add_grads(const mica_linear* l, const mica_linear_grads* g, Buffers* b) {
    if (g->dh) MICA_TRY(b->matrix(g->dh, l->rows, l->features, g->ld_dh, 2, 2, true, "dh"));
    if (!g->dw) return MICA_OK;
    const size_t es = bytes_of(g->dw_dtype);
    if (g->add) MICA_TRY(b->matrix(g->add, l->vocab, l->features, g->ld_add, es, es, false, "add"));
    MICA_TRY(b->matrix(g->dw, l->vocab, l->features, g->ld_dw, es, es, true, "dw"));
    if (g->add == g->dw && g->ld_add == g->ld_dw) b->in_place(g->dw);
    return MICA_OK;
}

mica_status add_workspace(void* workspace, int64_t bytes, int64_t need, Buffers* b) {
    if (need && !workspace) return fail(MICA_ERR_NULL, "workspace is NULL");
    if (bytes < need)
        return fail(MICA_ERR_COUNT, "the workspace has %lld bytes of %lld", (long long)bytes, (long long)need);
    return b->matrix(workspace, 1, need, need, 1, 16, true, "workspace");
}

}  // namespace
}  // namespace mica

using namespace mica;

extern "C" int64_t mica_linear_logps_workspace(const mica_linear* l) {
    Linear L;
    return check_linear(l, &L) == MICA_OK ? linear_logps_workspace(L) : 0;
}

extern "C" mica_status mica_linear_logps(const mica_linear* l, float* logps, float* lse, void* workspace,
                                         int64_t workspace_bytes, void* stream) {
    Linear L;
    MICA_TRY(check_linear(l, &L));
    if (l->rows == 0) return ok();
    int dev = 0;
    MICA_TRY(current_device(&dev));
    Buffers b(dev);
    MICA_TRY(add_inputs(l, &b));
    MICA_TRY(b.vec(logps, l->rows, 4, true, "logps"));
    if (lse) MICA_TRY(b.vec(lse, l->rows, 4, true, "lse"));
    MICA_TRY(add_workspace(workspace, workspace_bytes, linear_logps_workspace(L), &b));
    MICA_TRY(b.disjoint());
    return after_launch(launch_linear_logps(L, logps, lse, workspace, sm_count(dev), stream), stream,
                        "log-probabilities from hidden states launch");
}

extern "C" int64_t mica_linear_grad_workspace(const mica_linear* l, const mica_linear_grads* g) {
    Linear L;
    LinearGrad G;
    int dev = 0;
    if (check_linear(l, &L) != MICA_OK || !g || check_grads(l, g, &G) != MICA_OK || (!G.dh && !G.dw)) return 0;
    if (current_device(&dev) != MICA_OK) return 0;
    return linear_grad_workspace(L, G, sm_count(dev));
}

extern "C" mica_status mica_linear_logps_grad(const mica_linear* l, const float* lse, const float* dlogps,
                                              const mica_linear_grads* g, void* workspace, int64_t workspace_bytes,
                                              void* stream) {
    Linear L;
    LinearGrad G;
    MICA_TRY(check_linear(l, &L));
    if (!g) return fail(MICA_ERR_NULL, "the gradients are NULL");
    MICA_TRY(check_grads(l, g, &G));
    if (!G.dh && !G.dw) return ok();
    int dev = 0;
    MICA_TRY(current_device(&dev));
    const int sms = sm_count(dev);
    Buffers b(dev);
    MICA_TRY(add_inputs(l, &b));
    MICA_TRY(b.vec(lse, l->rows, 4, false, "lse"));
    MICA_TRY(b.vec(dlogps, l->rows, 4, false, "dlogps"));
    MICA_TRY(add_grads(l, g, &b));
    MICA_TRY(add_workspace(workspace, workspace_bytes, linear_grad_workspace(L, G, sms), &b));
    MICA_TRY(b.disjoint());
    return after_launch(launch_linear_grad(L, lse, dlogps, G, workspace, sms, stream), stream,
                        "gradients of log-probabilities from hidden states launch");
}

extern "C" int64_t mica_linear_cross_entropy_workspace(const mica_linear* l, const mica_linear_grads* g) {
    Linear L;
    LinearGrad G{};
    int dev = 0;
    if (check_linear(l, &L) != MICA_OK || (g && check_grads(l, g, &G) != MICA_OK) || current_device(&dev) != MICA_OK) return 0;
    return linear_ce_workspace(L, G, sm_count(dev));
}

extern "C" mica_status mica_linear_cross_entropy(const mica_linear* l, const mica_cross_entropy_hp* hp, float* loss,
                                                 float* logps, const mica_linear_grads* g, void* workspace,
                                                 int64_t workspace_bytes, void* stream) {
    Linear L;
    LinearGrad G{};
    MICA_TRY(check_linear(l, &L));
    if (!hp) return fail(MICA_ERR_NULL, "hp is NULL");
    if (!std::isfinite(hp->denom) || hp->denom < 0.0) return fail(MICA_ERR_HYPER, "denom %g is not finite and >= 0", hp->denom);
    if (hp->denom != 0.0 && (hp->denom < 1e-30 || hp->denom > 1e30))
        return fail(MICA_ERR_HYPER, "denom %g is outside [1e-30, 1e30]", hp->denom);
    if (!std::isfinite(hp->grad_scale)) return fail(MICA_ERR_HYPER, "grad_scale %g is not finite", hp->grad_scale);
    if (g) MICA_TRY(check_grads(l, g, &G));
    int dev = 0;
    MICA_TRY(current_device(&dev));
    const int sms = sm_count(dev);
    Buffers b(dev);
    MICA_TRY(add_inputs(l, &b));
    MICA_TRY(b.vec(loss, 1, 4, true, "loss"));
    MICA_TRY(b.vec(logps, l->rows, 4, true, "logps"));
    if (g) MICA_TRY(add_grads(l, g, &b));
    MICA_TRY(add_workspace(workspace, workspace_bytes, linear_ce_workspace(L, G, sms), &b));
    MICA_TRY(b.disjoint());
    return after_launch(launch_linear_ce(L, hp->denom, hp->grad_scale, loss, logps, G, workspace, sms, stream), stream,
                        "cross entropy from hidden states launch");
}
