// What the host side (linear_api.cpp) and the kernels (linear.cu) of the losses from hidden states share: the arguments of a
// launch, already checked, and the launch functions. Each returns a cudaError_t as int.
#pragma once

#include <cstdint>

#include "mica_train.h"

namespace mica {

struct Linear {
    const void* h;
    const void* w;
    const void* targets;
    int64_t rows, ld_h, ld_w;
    int32_t features, vocab;
    int32_t dtype;         // MICA_F16 or MICA_BF16
    int32_t wide_targets;  // int64 targets
    double temperature;
};

struct LinearGrad {
    void* dh;  // or null
    int64_t ld_dh;
    void* dw;  // or null
    int64_t ld_dw;
    int32_t dw_dtype;
    const void* add;  // or null
    int64_t ld_add;
};

int64_t linear_logps_workspace(const Linear& L);
// lse may be null
int launch_linear_logps(const Linear& L, float* logps, float* lse, void* workspace, int sms, void* stream);

int64_t linear_grad_workspace(const Linear& L, const LinearGrad& G, int sms);
int launch_linear_grad(const Linear& L, const float* lse, const float* dlogps, const LinearGrad& G, void* workspace, int sms,
                       void* stream);

int64_t linear_ce_workspace(const Linear& L, const LinearGrad& G, int sms);
// denom: 0 for the scored rows' number; the gradients are those of grad_scale * loss, and none are taken where G has none
int launch_linear_ce(const Linear& L, double denom, double grad_scale, float* loss, float* logps, const LinearGrad& G,
                     void* workspace, int sms, void* stream);

int read_linear_status(unsigned int* status);

}  // namespace mica
