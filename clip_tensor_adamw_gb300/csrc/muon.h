// What the host side (muon_api.cpp) and the kernels (muon.cu) of the orthogonalised step share.
#pragma once

#include <cstdint>

#include "mica_muon.h"

namespace mica {

// A checked call: mica_orthogonalize (x, out) or mica_muon_steps (g, m, w).
struct Muon {
    const int64_t* rows;
    const int64_t* cols;
    int32_t count;
    const void* const* in;  // x, or g
    int32_t in_dtype;
    float* const* m;        // null: mica_orthogonalize
    void* const* out;       // out, or w
    int32_t out_dtype;      // MICA_F32 for w
    const mica_newton_schulz* ns;
    mica_muon_hp hp;
    const float* d_factor;
};

int64_t muon_workspace(const int64_t* rows, const int64_t* cols, int32_t T, uint32_t flags);
// returns a cudaError_t
int launch_muon(const Muon& c, void* workspace, int sms, void* stream);
int read_muon_status(unsigned int* status);

}  // namespace mica
