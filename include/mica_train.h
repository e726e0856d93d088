/*
 * mica_train: the operators of a fine-tuning step that stand before the optimizer step of mica_optim.h, on one GB300
 * (sm_103a), as a C ABI of the same library: losses over a language model's logits with the gradient of the logits,
 * and activation checkpoints in 8 bits with the backward passes that read them. The weight gradients that
 * mica_packed_wgrad writes are of the types that mica_clip_grad_norms and mica_adamw_steps take.
 *
 *   mica_token_logps        log-probabilities (and entropies) of given tokens
 *   mica_token_logps_grad   the gradient of the logits, given that of the log-probabilities (any loss over them)
 *   mica_preference_loss    a preference loss over pairs of packed sequences, and the gradient of the logits
 *   mica_policy_loss        a clipped policy loss with a KL term, and the gradient of the logits
 *   mica_act_pack           an activation's checkpoint in 8 bits, and the activation function's value
 *   mica_act_unpack         the values a checkpoint stands for
 *   mica_act_grad           an activation function's backward pass from a checkpoint
 *   mica_packed_wgrad       a linear layer's weight gradient from its input's checkpoint
 *   mica_linear_logps       log-probabilities of given tokens from hidden states and an output embedding, logits not stored
 *   mica_linear_logps_grad  the gradients of both, given that of the log-probabilities (any loss over them)
 *   mica_linear_cross_entropy  softmax cross entropy from hidden states, with both gradients
 *
 * Conventions, where they differ from mica_optim.h's (ownership, streams, validation before anything is queued, error
 * details, MICA_SYNC_DEBUG and mica_sync are the same):
 *   - Matrices are device pointers with a row stride in elements (`ld`); the elements of a row are contiguous. Every
 *     alignment to the element is taken. Only rows * ld spans are checked: [p, p + ((rows-1)*ld + cols)) has to lie in
 *     p's allocation (MICA_ERR_ADDRESS); one of more than 2^44 elements is MICA_ERR_COUNT whatever p is.
 *   - Nothing is allocated and no table is cached. What a call needs besides its outputs is the caller's workspace,
 *     whose size a call of its own gives; its contents need not be set and are not read by a later call.
 *   - Results do not depend on the order in which CTAs run: no floating-point atomics.
 *   - Every call can be captured into a CUDA graph.
 *   - Sums, maxima and statistics are held in float32, pairs of float32 or float64; results are rounded once, to nearest-even.
 *   - Where the inputs give an infinity or a NaN, the formula's value comes out, never an error.
 */
#ifndef MICA_TRAIN_H
#define MICA_TRAIN_H

#include "mica_optim.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Element types of logits and activations: MICA_F32 and MICA_F16 (mica_optim.h), and bfloat16. */
#define MICA_BF16 4

/* The largest extents: rows (tokens) and columns (vocabulary, features) of a matrix. Offsets are 64-bit. */
#define MICA_MAX_ROWS ((int64_t)1 << 30)
#define MICA_MAX_COLS ((int64_t)1 << 24)

/*
 * A matrix of logits and the token scored in each row: row t holds z = logits[t*ld .. t*ld + vocab). With
 * x = z / temperature and the target y = targets[t]:  logp = x[y] - log sum_j exp(x[j]).
 *   - target < 0: the row does not count. It is not read; its log-probability and entropy are 0, and its gradient
 *     row is zeros, whatever it holds.
 *   - target >= vocab: the log-probability is NaN (nothing out of range is read), and so is the row's gradient unless
 *     its coefficient is 0.
 *   - a logit of -inf is a banned token (probability 0); a row with nothing else gives NaN, as 0/0 does.
 *   - ld may be anything >= 0 (0: every row the same) as long as the matrix is only read.
 */
typedef struct {
    const void* logits;
    const void* targets;  /* [rows], int32 or int64 */
    int64_t rows;         /* [0, MICA_MAX_ROWS] */
    int64_t vocab;        /* [1, MICA_MAX_COLS] */
    int64_t ld;
    double temperature;   /* [1e-30, 1e30] */
    int32_t dtype;        /* MICA_F32, MICA_F16 or MICA_BF16 */
    int32_t target_bytes; /* 4 or 8 */
} mica_logits;

/*
 * Log-probabilities of the rows' targets, logps[rows] float32, and, when entropy is not NULL, the entropies
 * -sum_j p_j log p_j of the rows' distributions, float32. One read of the logits.
 * Errors: NULL / COUNT / DTYPE / HYPER (temperature) / ADDRESS / OVERLAP / DEVICE / CUDA.
 */
MICA_API mica_status mica_token_logps(const mica_logits* z, float* logps, float* entropy, void* stream);

/*
 * dlogits[t][j] = dlogps[t] / temperature * ((j == target) - p_j), p the row's softmax of z / temperature; a row whose
 * target is negative or whose dlogps is 0 gets zeros. dlogits: the logits' type, row stride ld_d >= vocab; it may be
 * the logits' own buffer with ld_d == ld (in place), and otherwise must not overlap it. One read and one write.
 * Errors: as mica_token_logps.
 */
MICA_API mica_status mica_token_logps_grad(const mica_logits* z, const float* dlogps, void* dlogits, int64_t ld_d,
                                           void* stream);

/* mica_preference_hp.kind: the loss of a pair, with d = (chosen's sum) - (rejected's sum) and h = beta * d
 *   MICA_PREF_SIGMOID  -(1 - eps) log sigmoid(h) - eps log sigmoid(-h), eps = label_smoothing
 *   MICA_PREF_HINGE    max(0, 1 - h) (its slope at h == 1 is 0)
 *   MICA_PREF_IPO      (d - 1 / (2 beta))^2 */
enum { MICA_PREF_SIGMOID = 0, MICA_PREF_HINGE = 1, MICA_PREF_IPO = 2 };
#define MICA_PREF_LENGTH_NORM 1u /* a sequence's sum is divided by its number of scored tokens (at least 1) */

typedef struct {
    double beta;            /* finite, > 0 */
    double label_smoothing; /* [0, 1); MICA_PREF_SIGMOID only, 0 otherwise */
    double grad_scale;      /* finite: the gradient is that of grad_scale * loss (a loss scale) */
    int32_t kind;
    uint32_t flags;
} mica_preference_hp;

/*
 * A preference loss over `pairs` pairs of sequences packed into the rows of z: sequence s is rows
 * cu_seqlens[s] .. cu_seqlens[s+1] - 1, pair p is sequences 2p (chosen) and 2p + 1 (rejected). A sequence's sum is that
 * of logp - ref_logps over its scored rows (target >= 0); one without such rows has the sum 0. ref_logps: [rows], the
 * reference policy's log-probabilities (mica_token_logps), or NULL for zeros; those of rows that do not count are not
 * used. cu_seqlens: 2 * pairs + 1 device int32, non-decreasing; bounds outside [0, rows] are clamped to it and a
 * sequence that ends before it starts is empty. Rows in no sequence get zero gradients, whatever their targets.
 *   *loss     = the mean over pairs (0 when there are none)
 *   rewards   [2 * pairs]: beta times the sequences' sums, or NULL
 *   logps     [rows]: the policy's log-probabilities
 *   dlogits   the gradient of grad_scale * loss, as in mica_token_logps_grad; NULL for the loss alone
 * workspace: mica_preference_workspace(rows, pairs) bytes, 16-byte aligned.
 * A sequence's log-ratios are summed unrounded, in pairs of float32 (some 45 bits). 0 <= pairs <= 2^24.
 * Errors: NULL / COUNT (also a workspace too small) / DTYPE / HYPER / ADDRESS / OVERLAP / DEVICE / CUDA.
 */
MICA_API mica_status mica_preference_loss(const mica_logits* z, const int32_t* cu_seqlens, int32_t pairs,
                                          const float* ref_logps, const mica_preference_hp* hp, float* loss,
                                          float* rewards, float* logps, void* dlogits, int64_t ld_d, void* workspace,
                                          int64_t workspace_bytes, void* stream);
MICA_API int64_t mica_preference_workspace(int64_t rows, int32_t pairs);

typedef struct {
    double clip_low;   /* [0, 1]: the ratio's lower bound is 1 - clip_low */
    double clip_high;  /* >= 0 (may be infinite): its upper bound is 1 + clip_high */
    double kl_coef;    /* finite, >= 0 */
    double denom;      /* finite, > 0: what the sums over tokens are divided by, e.g. the tokens scored in the step */
    double grad_scale; /* finite */
} mica_policy_hp;

/*
 * A clipped policy loss with a KL term, token by token. For each row with target >= 0, with r = exp(logp - old_logps),
 * A = advantages, q = ref_logps - logp and w = weights (1 when NULL):
 *   l  = -min(r A, clamp(r, 1 - clip_low, 1 + clip_high) A)
 *   kl = exp(q) - q - 1                       (0 when ref_logps is NULL)
 *   loss = sum w (l + kl_coef * kl) / denom
 * The gradient of l is that of the smaller of the two products (of r A where they are equal).
 *   stats   4 float32: the loss, sum w l / denom, sum w kl / denom, and sum w [clipped] / denom, where a token is
 *           clipped when the clamped product is the smaller
 *   logps   [rows]
 *   dlogits the gradient of grad_scale * loss, as in mica_token_logps_grad; NULL for the loss alone
 * old_logps, advantages, ref_logps and weights are [rows] float32; those of rows that do not count are not used. The
 * sums are taken in pairs of float32 (some 45 bits). No workspace.
 * Errors: as mica_preference_loss.
 */
MICA_API mica_status mica_policy_loss(const mica_logits* z, const float* old_logps, const float* advantages,
                                      const float* ref_logps, const float* weights, const mica_policy_hp* hp,
                                      float* stats, float* logps, void* dlogits, int64_t ld_d, void* stream);

/*
 * An activation's checkpoint in 8 bits: a matrix of rows x cols values as signed codes q with one power-of-two step for
 * each block of 32 columns of a row (the last block may be short): the value is q * 2^e. A block's e is the smallest
 * integer with max|x| / 2^e < 127.5, but at least -126, or -24 when dtype is MICA_F16 (binary16 values are multiples
 * of 2^-24), and q is x / 2^e rounded to nearest, ties to even, but at most so that q * 2^e is finite in the source's
 * type (|q| <= 63 at its top exponent, for blocks that reach 63.5/64 of its range). So a value is off by at most half a
 * step (under 1/127 of its block's largest; in those blocks by up to a whole step), and, having 7 significant bits, is exact in the
 * source's type and in bfloat16: what reads a checkpoint rounds nothing. A block that holds an infinity or a NaN
 * stands for NaNs, so that a step that overflowed shows in the gradients.
 *   codes   int8 [rows][ld], 16-byte aligned, ld a multiple of 32 and >= cols; the last block's codes past cols
 *           are 0
 *   steps   uint8 [rows][ld_s], 4-byte aligned, ld_s a multiple of 4 and >= ceil(cols / 32): e + 127; 255 for NaNs. The
 *           entries past the last block are not written and not used (but read: the last row has all of a multiple of 4).
 *   dtype   the source's type, MICA_F32, MICA_F16 or MICA_BF16
 */
typedef struct {
    void* codes;
    void* steps;
    int64_t rows;  /* [0, MICA_MAX_ROWS] */
    int64_t cols;  /* [0, MICA_MAX_COLS] */
    int64_t ld;
    int64_t ld_s;
    int32_t dtype;
    int32_t reserved; /* 0 */
} mica_packed;

/* Activation functions: none (the checkpoint alone), GELU in its tanh form, GELU by erf, SiLU and ReLU. A gated unit
 * takes 2F columns and gives F: y[j] = act(x[j]) * x[F + j]; F must be a multiple of 32. */
enum { MICA_ACT_NONE = 0, MICA_ACT_GELU_TANH = 1, MICA_ACT_GELU = 2, MICA_ACT_SILU = 3, MICA_ACT_RELU = 4 };

/*
 * Packs x (p->dtype, rows x cols, row stride ld_x) into p's buffers and, when act is not MICA_ACT_NONE, writes y, the
 * activation function's value at x (not at the checkpoint's rounded values), of x's type: rows x cols, or rows x
 * cols / 2 when gated. y is NULL when act is MICA_ACT_NONE. One read of x.
 * Errors: NULL / COUNT / DTYPE / HYPER (act) / ADDRESS / OVERLAP / DEVICE / CUDA.
 */
MICA_API mica_status mica_act_pack(const void* x, int64_t ld_x, const mica_packed* p, int32_t act, int32_t gated, void* y,
                                   int64_t ld_y, void* stream);

/* The checkpoint's values, exactly, in its source's type: x, rows x cols, row stride ld_x. Errors: as mica_act_pack. */
MICA_API mica_status mica_act_unpack(const mica_packed* p, void* x, int64_t ld_x, void* stream);

/*
 * The backward pass of an activation function (not MICA_ACT_NONE) from its input's checkpoint, at the checkpoint's
 * values x: dx[j] = dy[j] * act'(x[j]), or, gated, dx[j] = dy[j] * x[F+j] * act'(x[j]) and
 * dx[F+j] = dy[j] * act(x[j]). dy (rows x cols, or cols / 2 when gated) and dx (rows x cols) are of type dtype, computed
 * in float32. Where not gated, dx may be dy's own buffer with the same row stride. ReLU's slope at 0 is 0.
 * Errors: as mica_act_pack.
 */
MICA_API mica_status mica_act_grad(const mica_packed* p, int32_t act, int32_t gated, const void* dy, int64_t ld_dy,
                                   int32_t dtype, void* dx, int64_t ld_dx, void* stream);

/*
 * The weight gradient of a linear layer y = x W from its input's checkpoint (rows = tokens, cols = features in):
 *   dw[i][j] = add[i][j] + sum_t x[t][i] * dy[t][j]
 * dy: tokens x n, row stride ld_dy, of type dy_dtype: MICA_BF16 (any checkpoint), or MICA_F16 (one of a binary16
 * source). dw: features x n, row stride ld_dw, MICA_F32, MICA_F16 or MICA_BF16; add: the same type with row stride
 * ld_add, NULL for zeros, or dw itself (accumulation in place). The products are exact and summed in float32, add is
 * added in float32, and the result is rounded once. No tokens: dw = add. workspace: mica_packed_wgrad_workspace bytes
 * for the same arguments, 16-byte aligned (it may be 0 bytes, and NULL then): sums of parts, at most 20 MB, and a
 * copy of a dy whose rows are not 16-byte aligned (as large as dy: tokens x n elements, n rounded up to a multiple of 8).
 * Errors: NULL / COUNT / DTYPE / ADDRESS / OVERLAP / DEVICE / CUDA.
 */
MICA_API mica_status mica_packed_wgrad(const mica_packed* x, const void* dy, int64_t ld_dy, int32_t dy_dtype, int64_t n,
                                       const void* add, int64_t ld_add, void* dw, int64_t ld_dw, int32_t dw_dtype,
                                       void* workspace, int64_t workspace_bytes, void* stream);
MICA_API int64_t mica_packed_wgrad_workspace(const mica_packed* x, const void* dy, int64_t ld_dy, int64_t n);

/*
 * Hidden states, an output embedding and the token scored in each row: row t's logits are
 * z[j] = sum_k h[t*ld_h + k] * w[j*ld_w + k] / temperature, j < vocab. They are never stored. Rows are taken in pieces, and
 * the workspaces hold, for a piece of P rows:
 *   - 2 P vocab bytes with gradients: the logits' gradient in 16 bits (or, in cross entropy, what it is a multiple of). P is
 *     at most 2^29 / vocab, rounded down to a multiple of 256, but no fewer than 256: so all rows up to 1 GB of it (8,192 rows
 *     of 50,257 tokens: 824 MB), pieces of up to 1 GB beyond, and 256 rows where those take more (8.6 GB at 2^24 tokens)
 *   - P vocab / 16 bytes in the forward pass (mica_linear_logps, cross entropy): maxima and sums. There P is at most 16,384
 *     and 2^32 / vocab, rounded as above: 256 MB
 *   - 2 P features bytes, the rows that count gathered; as much again in cross entropy with gradients of MICA_BF16
 * and further
 *   - 2 vocab features bytes, a copy of w, where its rows do not begin at multiples of 16 bytes or overlap
 *   - 40 MB for each of dh and dw, sums of parts; 4 vocab features bytes more where there are several pieces and dw is of 16 bits
 *   - some 4 bytes a row and 40 a row of a piece
 *
 *   - the products are exact and summed in float32; maxima and sums over the vocabulary are float32
 *   - target < 0: the row does not count. It is not read; its log-probability is 0 and its gradient zeros, whatever it
 *     holds. Rows that do not count cost next to nothing
 *   - target >= vocab: the log-probability is NaN (nothing out of range is read), and so are the gradients that the row
 *     takes part in, unless its coefficient is 0
 *   - h and w have the same type, MICA_F16 or MICA_BF16, any alignment and row stride
 */
typedef struct {
    const void* h;        /* rows x features */
    const void* w;        /* vocab x features, as an embedding's table or a linear layer's [out][in] */
    const void* targets;  /* [rows], int32 or int64 */
    int64_t rows;         /* [0, MICA_MAX_ROWS] */
    int64_t features;     /* [1, MICA_MAX_FEATURES] */
    int64_t vocab;        /* [1, MICA_MAX_COLS] */
    int64_t ld_h, ld_w;
    double temperature;   /* [2^-20, 2^20] */
    int32_t dtype;        /* MICA_F16 or MICA_BF16 */
    int32_t target_bytes; /* 4 or 8 */
} mica_linear;
#define MICA_MAX_FEATURES ((int64_t)1 << 16)

/*
 * Log-probabilities of the rows' targets, logps[rows] float32, and, when lse is not NULL, lse[rows] float32: the logarithm of
 * the sum of exp of the row's logits (0 where the row does not count). workspace: mica_linear_logps_workspace bytes for the
 * same argument, 16-byte aligned.
 * Errors: NULL / COUNT (also a workspace too small) / DTYPE / HYPER (temperature) / ADDRESS / OVERLAP / DEVICE / CUDA.
 */
MICA_API mica_status mica_linear_logps(const mica_linear* l, float* logps, float* lse, void* workspace,
                                       int64_t workspace_bytes, void* stream);
MICA_API int64_t mica_linear_logps_workspace(const mica_linear* l);

/*
 * Where the gradients go: dh (rows x features, of h's type) and dw (vocab x features, MICA_F32, MICA_F16 or MICA_BF16), one
 * or both (without rows dh may be NULL too); dw = add + the gradient, where add is of dw's type, NULL for zeros, or dw itself
 * (accumulation in place).
 * The gradient of the logits is rounded to h's type (scaled, in binary16, so that its largest finite row uses the whole
 * range), as the tensor cores take it; sums are float32 and rounded once. So before its own rounding an element is off by up
 * to 2^-8 (bfloat16) or 2^-11 (binary16) of the terms that it sums up, whatever dw's type: dw by 0.9e-3 to 1.7e-3, or 1.3e-4
 * to 2.1e-4, of its norm. mica_linear_cross_entropy rounds up to three times in bfloat16, but once where a row's target is, so
 * that it comes to 1.7e-3 of the norm as well, and up to 3 x 2^-8 of an element's terms; in binary16 its target's elements are
 * exact where the target is unlikely (1.4e-4).
 */
typedef struct {
    void* dh;
    void* dw;
    const void* add;
    int64_t ld_dh, ld_dw, ld_add;
    int32_t dw_dtype;
    int32_t reserved; /* 0 */
} mica_linear_grads;

/*
 * The gradients given that of the log-probabilities, dlogps[rows] float32, and lse[rows] as mica_linear_logps gives it: with
 * d[t][j] = dlogps[t] / temperature * ((j == target) - exp(z[t][j] - lse[t])), dh = d w and dw = add + d^T h. A row whose
 * target is negative or whose dlogps is 0 does not count: its dh is zeros. workspace: mica_linear_grad_workspace bytes for
 * the same arguments, 16-byte aligned.
 * Errors: as mica_linear_logps.
 */
MICA_API mica_status mica_linear_logps_grad(const mica_linear* l, const float* lse, const float* dlogps,
                                            const mica_linear_grads* g, void* workspace, int64_t workspace_bytes,
                                            void* stream);
MICA_API int64_t mica_linear_grad_workspace(const mica_linear* l, const mica_linear_grads* g);

typedef struct {
    double denom;      /* >= 0, finite: what the sum over rows is divided by; 0: the number of rows that count */
    double grad_scale; /* finite; 0: every row's coefficient is 0, its logits' gradient zeros whatever its target is */
} mica_cross_entropy_hp;

/*
 * Softmax cross entropy: *loss = -(sum of logps over the rows that count) / denom (0 when none count), logps[rows], and the
 * gradients of grad_scale * loss where g is not NULL. workspace: mica_linear_cross_entropy_workspace bytes.
 * Errors: as mica_linear_logps.
 */
MICA_API mica_status mica_linear_cross_entropy(const mica_linear* l, const mica_cross_entropy_hp* hp, float* loss,
                                               float* logps, const mica_linear_grads* g, void* workspace,
                                               int64_t workspace_bytes, void* stream);
MICA_API int64_t mica_linear_cross_entropy_workspace(const mica_linear* l, const mica_linear_grads* g);

#ifdef __cplusplus
}
#endif

#endif /* MICA_TRAIN_H */
