/*
 * mica_muon: the optimizer step whose update is orthogonalised (momentum, Newton-Schulz products, decoupled decay), on one
 * GB300 (sm_103a), as a C ABI of the same library as mica_optim.h. It stands beside mica_adamw_steps for a model's weight
 * matrices (embeddings, output layers and vectors stay with AdamW) and takes the same device-resident clip factor.
 *
 *   mica_orthogonalize   a list of matrices, each replaced by its Newton-Schulz iterate
 *   mica_muon_steps      the whole step over a list of weight matrices
 *
 * Conventions, where they differ from mica_optim.h's (ownership, streams, validation before anything is queued, error
 * details, MICA_SYNC_DEBUG and mica_sync are the same):
 *   - A matrix is rows[k] x cols[k] contiguous elements; sides in [0, MICA_MAX_SIDE] (one with a side of 0 is skipped).
 *   - Nothing is allocated and no table is cached: what a call needs is the caller's workspace, whose contents need not be
 *     set and are not read by a later call. Every call can be captured into a CUDA graph.
 *   - Results do not depend on the order in which CTAs run: no floating-point atomics. The same list gives the same bits. In
 *     another list a matrix's may differ in the last places of its float32 sums: where a list has too few tiles for the GPU,
 *     a long sum is split in parts, by the list's sizes and the number of SMs.
 */
#ifndef MICA_MUON_H
#define MICA_MUON_H

#include "mica_optim.h"
#include "mica_train.h" /* MICA_BF16 */

#ifdef __cplusplus
extern "C" {
#endif

#define MICA_MAX_SIDE ((int64_t)1 << 17)
#define MICA_MAX_NS_STEPS 16

/*
 * The iteration: x = u / (|u| + eps), |u| the Frobenius norm; then, `steps` times, with G the smaller of x x^T and x^T x,
 *   x = a x + (b G + c G^2) x     (G on the side that it fits)
 * where step s takes (a, b, c) = coefficients[3 s .. 3 s + 2]. So each singular value t of x becomes a t + b t^3 + c t^5, and
 * the singular vectors stay. For all singular values that can occur, |u| being 1 at first, the polynomials'
 * values must be at most sqrt(32) in size, and those of a + b t^2 + c t^4 at most 32 (MICA_ERR_HYPER otherwise).
 * x, G and the polynomial of G are held in binary16 between the products (scaled by 2^10; products are exact and summed in
 * float32), which takes a result some 2^-9 to 2^-10 of its norm off; directions whose singular values in u are a thousand
 * times below the largest get correspondingly less accurate. With MICA_NS_PRECISE, and always for matrices whose smaller side
 * is at most 256 (whose products are short), they are held in pairs of binary16, at three times the operations, for results
 * some 2^-19 off before they are rounded to out's type. A zero matrix gives zeros; a matrix with an infinity or a NaN gives NaNs.
 */
#define MICA_NS_PRECISE 1u
typedef struct {
    const double* coefficients; /* host, 3 * steps, at most 1e30 in size */
    double eps;                 /* [1e-30, 1] */
    int32_t steps;              /* [1, MICA_MAX_NS_STEPS] */
    uint32_t flags;             /* MICA_NS_PRECISE or 0 */
} mica_newton_schulz;

/* The workspace of both calls for a list of these sizes and the iteration's flags, in bytes (the pointer 16-byte aligned).
 * A list is taken in batches of at most 8 shapes, 256 matrices and 128 M elements (or one larger matrix), and the largest
 * batch's is needed: some 4 bytes an element and 4 bytes x the smaller side squared, twice that for matrices held in pairs,
 * and, for lists so small that long sums are split, 256 KB for each part, at most 24 MB. */
MICA_API int64_t mica_newton_schulz_workspace(const int64_t* rows, const int64_t* cols, int32_t T, uint32_t flags);

/*
 * out[k] = the iterate of x[k]. x: MICA_F32, MICA_F16 or MICA_BF16; out: MICA_F16 or MICA_BF16; out[k] may be x[k] where
 * their types are the same.
 * Errors: NULL / COUNT (also a workspace too small) / DTYPE / HYPER / ADDRESS / OVERLAP / DEVICE / CUDA.
 */
MICA_API mica_status mica_orthogonalize(const void* const* x, void* const* out, const int64_t* rows, const int64_t* cols,
                                        int32_t T, int32_t x_dtype, int32_t out_dtype, const mica_newton_schulz* ns,
                                        void* workspace, int64_t workspace_bytes, void* stream);

/* mica_muon_hp.adjust: what the learning rate of a rows x cols matrix is multiplied by
 *   MICA_MUON_PLAIN      1
 *   MICA_MUON_ORIGINAL   sqrt(max(1, rows / cols))
 *   MICA_MUON_MATCH_RMS  0.2 sqrt(max(rows, cols)): updates about as large as AdamW's */
enum { MICA_MUON_PLAIN = 0, MICA_MUON_ORIGINAL = 1, MICA_MUON_MATCH_RMS = 2 };

typedef struct {
    double lr;           /* finite, >= 0 */
    double momentum;     /* [0, 1) */
    double weight_decay; /* finite, >= 0 */
    int32_t nesterov;
    int32_t adjust;
    int32_t zero_grad;   /* g is zeroed once it has been read */
    uint32_t flags;      /* MICA_STEP_SKIP_NONFINITE or 0 */
} mica_muon_hp;

/*
 * One step over T weight matrices, in place, with f = *d_factor (1 when NULL):
 *   gh = f g;  m = m + (1 - momentum) (gh - m);  u = nesterov ? gh + momentum (m - gh) : m
 *   w = w (1 - lr weight_decay) - lr adjust(rows, cols) O(u)
 * O the Newton-Schulz iterate. w, m: float32; g: MICA_F32 or MICA_F16. MICA_STEP_SKIP_NONFINITE leaves w and m as they are
 * when f is not > 0 (g is still zeroed when asked).
 * Errors: as mica_orthogonalize.
 */
MICA_API mica_status mica_muon_steps(float* const* w, void* const* g, float* const* m, const int64_t* rows,
                                     const int64_t* cols, int32_t T, int32_t g_dtype, const mica_muon_hp* hp,
                                     const mica_newton_schulz* ns, const float* d_factor, void* workspace,
                                     int64_t workspace_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* MICA_MUON_H */
