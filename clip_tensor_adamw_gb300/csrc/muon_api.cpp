// The C ABI of the orthogonalised optimizer step (include/mica_muon.h): host-side validation and launches.
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <new>
#include <vector>

#include "checks.h"
#include "muon.h"

namespace mica {
namespace {

constexpr int32_t kMostListed = 1 << 20;

mica_status check_sizes(const int64_t* rows, const int64_t* cols, int32_t T) {
    if (T < 0 || T > kMostListed) return fail(MICA_ERR_COUNT, "T = %d is outside [0, 2^20]", T);
    if (T > 0 && (!rows || !cols)) return fail(MICA_ERR_NULL, "rows or cols is NULL");
    for (int32_t k = 0; k < T; ++k)
        if (rows[k] < 0 || rows[k] > MICA_MAX_SIDE || cols[k] < 0 || cols[k] > MICA_MAX_SIDE)
            return fail(MICA_ERR_COUNT, "matrix %d is %lld x %lld: sides must be in [0, 2^17]", k, (long long)rows[k],
                        (long long)cols[k]);
    return MICA_OK;
}

// The largest that |q(u)| and sqrt(u) |q(u)|, q = a + b u + c u^2, come to over u in [0, top^2]: at an end, or where the
// derivative is 0, b + 2 c u = 0 for the one and a + 3 b u + 5 c u^2 = 0 for the other.
struct Peaks {
    double factor = 0.0, value = 0.0;
};
Peaks peaks_of(const double* coefficients, double top) {
    const double a = coefficients[0], b = coefficients[1], c = coefficients[2], end = top * top;
    Peaks p;
    const auto at = [&](double u) {
        if (!(u >= 0.0 && u <= end)) return;  // (or no number: the derivative has no such root)
        const double q = std::fabs(a + u * (b + u * c));
        p.factor = std::max(p.factor, q);
        p.value = std::max(p.value, std::sqrt(u) * q);
    };
    at(0.0);
    at(end);
    at(-b / (2.0 * c));
    const double square = 9.0 * b * b - 20.0 * a * c;
    if (square >= 0.0) {
        const double w = -0.5 * (3.0 * b + std::copysign(std::sqrt(square), b));
        at(w / (5.0 * c));
        at(a / w);
    }
    return p;
}

// Follows the largest singular value that each step can leave: what the products hold in binary16 (x, x x^T and the
// polynomial of it, 2^10 times) must stay within its range.
mica_status check_iteration(const mica_newton_schulz* ns) {
    if (!ns) return fail(MICA_ERR_NULL, "the iteration is NULL");
    if (ns->flags & ~MICA_NS_PRECISE) return fail(MICA_ERR_HYPER, "unknown flags 0x%x of the iteration", ns->flags);
    if (!(ns->eps >= 1e-30 && ns->eps <= 1.0)) return fail(MICA_ERR_HYPER, "eps %g is outside [1e-30, 1]", ns->eps);
    if (ns->steps < 1 || ns->steps > MICA_MAX_NS_STEPS)
        return fail(MICA_ERR_HYPER, "steps = %d is outside [1, %d]", ns->steps, MICA_MAX_NS_STEPS);
    if (!ns->coefficients) return fail(MICA_ERR_NULL, "coefficients is NULL");
    constexpr double kMost = 32.0, kMostCoefficient = 1e30;
    double top = 1.0;
    for (int s = 0; s < ns->steps; ++s) {
        const double* c = ns->coefficients + 3 * s;
        for (int i = 0; i < 3; ++i)
            if (!(std::fabs(c[i]) <= kMostCoefficient))
                return fail(MICA_ERR_HYPER, "step %d's coefficient %g is not within 1e30", s, c[i]);
        const Peaks p = peaks_of(c, top);
        if (!(p.factor <= kMost && p.value * p.value <= kMost))
            return fail(MICA_ERR_HYPER, "step %d's polynomial reaches %g: it must stay below %g", s,
                        std::max(p.factor, p.value * p.value), kMost);
        top = p.value;
    }
    return MICA_OK;
}

// Every matrix of every list of a call: device memory, and what is written overlaps nothing else.
class Lists {
  public:
    explicit Lists(int device) : device_(device) {}

    // but: where not null, a list whose k-th entry is the same memory and is not counted twice
    mica_status add(const void* const* p, const int64_t* rows, const int64_t* cols, int32_t T, size_t elem, bool written,
                    const char* name, const void* const* but = nullptr) {
        if (T > 0 && !p) return fail(MICA_ERR_NULL, "%s is NULL", name);
        for (int32_t k = 0; k < T; ++k) {
            const size_t bytes = (size_t)rows[k] * (size_t)cols[k] * elem;
            if (bytes == 0) continue;
            if (!p[k]) return fail(MICA_ERR_NULL, "%s[%d] is NULL", name, k);
            const mica_status s = check_device_span(p[k], bytes, elem, device_, name, k);
            if (s != MICA_OK) return s;
            if (but && but[k] == p[k]) continue;
            const uintptr_t lo = reinterpret_cast<uintptr_t>(p[k]);
            spans_.push_back(Span{lo, lo + bytes, written, name, k});
        }
        return MICA_OK;
    }
    mica_status add(const void* p, size_t bytes, size_t align, bool written, const char* name) {
        if (bytes == 0) return MICA_OK;
        if (!p) return fail(MICA_ERR_NULL, "%s is NULL", name);
        const mica_status s = check_device_span(p, bytes, align, device_, name, 0);
        if (s != MICA_OK) return s;
        const uintptr_t lo = reinterpret_cast<uintptr_t>(p);
        spans_.push_back(Span{lo, lo + bytes, written, name, 0});
        return MICA_OK;
    }

    mica_status disjoint() {
        std::sort(spans_.begin(), spans_.end(), [](const Span& a, const Span& b) { return a.lo < b.lo; });
        const Span *any = nullptr, *written = nullptr;  // of those before, the ones that reach furthest
        for (const Span& s : spans_) {
            const Span* hit = written && written->hi > s.lo ? written : s.written && any && any->hi > s.lo ? any : nullptr;
            if (hit) return fail(MICA_ERR_OVERLAP, "%s[%d] overlaps %s[%d]", s.name, s.k, hit->name, hit->k);
            if (!any || s.hi > any->hi) any = &s;
            if (s.written && (!written || s.hi > written->hi)) written = &s;
        }
        return MICA_OK;
    }

  private:
    struct Span {
        uintptr_t lo, hi;
        bool written;
        const char* name;
        int32_t k;
    };
    int device_;
    std::vector<Span> spans_;
};

bool all_empty(const int64_t* rows, const int64_t* cols, int32_t T) {
    for (int32_t k = 0; k < T; ++k)
        if (rows[k] && cols[k]) return false;
    return true;
}

mica_status check_workspace(void* workspace, int64_t bytes, int64_t need, Lists* lists) {
    if (need && !workspace) return fail(MICA_ERR_NULL, "workspace is NULL");
    if (bytes < need)
        return fail(MICA_ERR_COUNT, "the workspace has %lld bytes of %lld", (long long)bytes, (long long)need);
    return lists->add(workspace, (size_t)need, 16, true, "workspace");
}

mica_status orthogonalize(const void* const* x, void* const* out, const int64_t* rows, const int64_t* cols, int32_t T,
                          int32_t x_dtype, int32_t out_dtype, const mica_newton_schulz* ns, void* workspace,
                          int64_t workspace_bytes, void* stream) {
    MICA_TRY(check_sizes(rows, cols, T));
    if (!is_type(x_dtype)) return fail(MICA_ERR_DTYPE, "x must be float32, float16 or bfloat16");
    if (out_dtype != MICA_F16 && out_dtype != MICA_BF16) return fail(MICA_ERR_DTYPE, "out must be float16 or bfloat16");
    MICA_TRY(check_iteration(ns));
    if (all_empty(rows, cols, T)) return ok();
    int dev = 0;
    MICA_TRY(current_device(&dev));
    Lists lists(dev);
    MICA_TRY(lists.add(out, rows, cols, T, 2, true, "out"));
    MICA_TRY(lists.add(x, rows, cols, T, bytes_of(x_dtype), false, "x", x_dtype == out_dtype ? out : nullptr));
    MICA_TRY(check_workspace(workspace, workspace_bytes, muon_workspace(rows, cols, T, ns->flags), &lists));
    MICA_TRY(lists.disjoint());
    const Muon c{rows, cols, T, x, x_dtype, nullptr, out, out_dtype, ns, mica_muon_hp{}, nullptr};
    return after_launch(launch_muon(c, workspace, sm_count(dev), stream), stream, "orthogonalisation launch");
}

mica_status muon_steps(float* const* w, void* const* g, float* const* m, const int64_t* rows, const int64_t* cols, int32_t T,
                       int32_t g_dtype, const mica_muon_hp* hp, const mica_newton_schulz* ns, const float* d_factor,
                       void* workspace, int64_t workspace_bytes, void* stream) {
    MICA_TRY(check_sizes(rows, cols, T));
    if (g_dtype != MICA_F32 && g_dtype != MICA_F16) return fail(MICA_ERR_DTYPE, "g must be float32 or float16");
    if (!hp) return fail(MICA_ERR_NULL, "hp is NULL");
    if (!std::isfinite(hp->lr) || hp->lr < 0.0) return fail(MICA_ERR_HYPER, "lr %g is not finite and >= 0", hp->lr);
    if (!(hp->momentum >= 0.0 && hp->momentum < 1.0))
        return fail(MICA_ERR_HYPER, "momentum %g is outside [0, 1)", hp->momentum);
    if (!std::isfinite(hp->weight_decay) || hp->weight_decay < 0.0)
        return fail(MICA_ERR_HYPER, "weight_decay %g is not finite and >= 0", hp->weight_decay);
    if (hp->adjust < MICA_MUON_PLAIN || hp->adjust > MICA_MUON_MATCH_RMS)
        return fail(MICA_ERR_HYPER, "adjust %d is none of the adjustments", hp->adjust);
    if (hp->flags & ~MICA_STEP_SKIP_NONFINITE) return fail(MICA_ERR_HYPER, "unknown flags 0x%x", hp->flags);
    MICA_TRY(check_iteration(ns));
    if (all_empty(rows, cols, T)) return ok();
    int dev = 0;
    MICA_TRY(current_device(&dev));
    Lists lists(dev);
    MICA_TRY(lists.add(reinterpret_cast<const void* const*>(w), rows, cols, T, 4, true, "w"));
    MICA_TRY(lists.add(g, rows, cols, T, bytes_of(g_dtype), hp->zero_grad != 0, "g"));
    MICA_TRY(lists.add(reinterpret_cast<const void* const*>(m), rows, cols, T, 4, true, "m"));
    if (d_factor) MICA_TRY(lists.add(d_factor, 4, 4, false, "d_factor"));
    MICA_TRY(check_workspace(workspace, workspace_bytes, muon_workspace(rows, cols, T, ns->flags), &lists));
    MICA_TRY(lists.disjoint());
    const Muon c{rows, cols, T, const_cast<const void* const*>(g), g_dtype, m, reinterpret_cast<void* const*>(w), MICA_F32,
                 ns, *hp, d_factor};
    return after_launch(launch_muon(c, workspace, sm_count(dev), stream), stream, "orthogonalised step launch");
}

}  // namespace
}  // namespace mica

using namespace mica;

extern "C" int64_t mica_newton_schulz_workspace(const int64_t* rows, const int64_t* cols, int32_t T, uint32_t flags) {
    try {
        return check_sizes(rows, cols, T) == MICA_OK ? muon_workspace(rows, cols, T, flags) : 0;
    } catch (const std::bad_alloc&) {
        return 0;
    }
}

extern "C" mica_status mica_orthogonalize(const void* const* x, void* const* out, const int64_t* rows, const int64_t* cols,
                                          int32_t T, int32_t x_dtype, int32_t out_dtype, const mica_newton_schulz* ns,
                                          void* workspace, int64_t workspace_bytes, void* stream) {
    try {
        return orthogonalize(x, out, rows, cols, T, x_dtype, out_dtype, ns, workspace, workspace_bytes, stream);
    } catch (const std::bad_alloc&) {
        return fail(MICA_ERR_NOMEM, "out of host memory");
    }
}

extern "C" mica_status mica_muon_steps(float* const* w, void* const* g, float* const* m, const int64_t* rows,
                                       const int64_t* cols, int32_t T, int32_t g_dtype, const mica_muon_hp* hp,
                                       const mica_newton_schulz* ns, const float* d_factor, void* workspace,
                                       int64_t workspace_bytes, void* stream) {
    try {
        return muon_steps(w, g, m, rows, cols, T, g_dtype, hp, ns, d_factor, workspace, workspace_bytes, stream);
    } catch (const std::bad_alloc&) {
        return fail(MICA_ERR_NOMEM, "out of host memory");
    }
}
