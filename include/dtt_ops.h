/*
 * dtt_ops.h -- operators on what a rank owns between a reduce-scatter and an all-gather: the
 * residual's addition with a root-mean-square norm or a layer norm (bf16, f32 or 8-bit output) and
 * their backward passes, tokens' rows sorted by expert and back, the orthogonalisation of a momentum
 * update by Newton-Schulz products, and AdamW over the tensors of the rank's share.
 *
 * The conventions of dtt.h hold: DTT_OK or a negative DTT_E* code with dtt_last_error(), device
 * pointers in the current device's context, the caller's streams and buffers.  Nothing here
 * allocates device memory: where an operator needs a workspace the caller passes one (and keeps
 * it to one stream at a time, or orders the streams).  Every call is asynchronous on `stream`, makes
 * no device-wide synchronisation and can be captured into a CUDA graph once dtt_preload has run.
 * A tensor is rows of contiguous elements, `pitch` bytes apart, at any alignment its element type
 * allows; rows that are 16-byte aligned throughout take the faster paths.  Inputs may be read in whole
 * aligned 16-byte words (no allocation ends within one); outputs are written exactly.
 *
 * Run them between rounds, not in one: their kernels take nearly all shared memory and registers
 * of an SM, and large orthogonalisations every SM at once, while a round's copiers hold theirs from
 * the round's start (an early copier, from the round before on) until it is done.  An operator that
 * a round in progress waits for, as its producer or before it on its stream, may not get to run
 * beside the copiers, and the round then ends by its time limit.  No call checks this.
 */
#ifndef DTT_OPS_H
#define DTT_OPS_H

#include "dtt.h"

#ifdef __cplusplus
extern "C" {
#endif

/* An 8-bit output type beside DTT_BF16 and DTT_F32: 4 exponent and 3 mantissa bits, finite up to
 * 448, no infinities. */
enum { DTT_E4M3 = 3 };

/* ---------------------------------------------------------------------------------------- */
/* Residual addition and root-mean-square norm                                                */
/* ---------------------------------------------------------------------------------------- */

/* For each row:
 *     h_c = x_c + residual_c             (f32; h = x without a residual)
 *     s   = 1 / sqrt(mean_c h_c^2 + eps) (f32, over the unrounded h)
 *     y_c = h_c s weight_c               (weight NULL: 1)
 * residual_out = h, rounded once to its type; rstd = s.  With y_dtype DTT_E4M3 the row is cut into
 * groups of `group` columns (0: the whole row; the last group holds what is left) and
 *     scale = max(max_c |y_c| / 448, 2^-100) (to an ulp),
 *     y stored = e4m3(y_c / scale), the f32 quotient to the nearest code, ties to even,
 * so y_c ~ stored * scale, and a group of zeros gives zeros.  NaN anywhere in a row makes the
 * row's rstd, scales and outputs NaN; a row whose sum of squares overflows f32 has rstd 0.  Should one
 * of the kernels' bounded waits for a row ever run out, that row and the rows its CTA takes after it are NaN, in
 * residual_out, dx and dweight too. */
typedef struct dtt_rmsnorm_desc {
    uint32_t x_dtype;        /* x and, in the backward pass, dy: DTT_BF16 or DTT_F32 */
    uint32_t residual_dtype; /* residual, residual_out; backward: h, dres and dx: DTT_BF16 or DTT_F32 */
    uint32_t weight_dtype;   /* DTT_BF16 or DTT_F32 */
    uint32_t y_dtype;        /* DTT_BF16, DTT_F32 or DTT_E4M3 */
    uint32_t group;          /* DTT_E4M3: columns per scale, 0 (one per row), 32, 64 or 128; else 0 */
    float eps;               /* finite, >= 0 */
    uint64_t cols;           /* 1 .. 2^24 */
} dtt_rmsnorm_desc;

/* rows x cols elements (rows 0: nothing is read or written).  The same call gives the same bits; a row of
 * another call may differ in the last bits where the number of rows, the alignments or the absence of
 * an argument choose another form, whose sums run in another order.
 *  - residual, residual_out, rstd may be NULL; residual_out may be residual itself (the same
 *    pointer and pitch), otherwise no output overlaps an input or another output.
 *  - scales: device f32 [rows][ceil(cols / group)] (group 0: [rows]), needed for DTT_E4M3 and
 *    NULL otherwise.
 * Errors: DTT_EINVAL (a bad desc; a missing or misaligned pointer; a pitch smaller than a row, or
 * no multiple of its element), DTT_ECUDA. */
int dtt_rmsnorm_forward(const dtt_rmsnorm_desc* desc, uint64_t rows, const void* x, uint64_t x_pitch,
                        const void* residual, uint64_t residual_pitch, const void* weight,
                        void* residual_out, uint64_t residual_out_pitch, void* y, uint64_t y_pitch,
                        float* scales, float* rstd, cudaStream_t stream);

/* The backward pass, from the forward's saved h (residual_out, or x where there was no residual) and
 * rstd:  with n_c = h_c rstd and m = mean_c(dy_c weight_c n_c) of each row,
 *     dx_c = rstd (dy_c weight_c - n_c m) + dres_c      (the gradient of x and of residual alike)
 *     dweight_c = sum over rows of dy_c n_c             (f32)
 * dres is the gradient that reaches residual_out from its other readers (NULL: none).  An 8-bit
 * y passes its gradient straight through.  Sums are f32 in an order that depends on the sizes
 * and alignments alone, so the same call gives the same bits.  rows 0: dweight is zeroed, nothing else.
 *  - dweight may be NULL (not computed; workspace is then unused and may be NULL); a NULL weight
 *    (1 everywhere) needs dweight NULL.  dx may be dres itself; no other overlap.
 *  - workspace: dtt_rmsnorm_workspace's bytes, 16-byte aligned.
 * y_dtype and group are not used.  Errors: as dtt_rmsnorm_forward, and DTT_EINVAL for a workspace
 * that is missing or short. */
int dtt_rmsnorm_backward(const dtt_rmsnorm_desc* desc, uint64_t rows, const void* dy, uint64_t dy_pitch,
                         const void* h, uint64_t h_pitch, const void* weight, const float* rstd,
                         const void* dres, uint64_t dres_pitch, void* dx, uint64_t dx_pitch,
                         float* dweight, void* workspace, uint64_t workspace_bytes, cudaStream_t stream);

/* Bytes of dtt_rmsnorm_backward's workspace, for any number of rows.  Errors: DTT_EINVAL. */
int dtt_rmsnorm_workspace(const dtt_rmsnorm_desc* desc, uint64_t* bytes);

/* ---------------------------------------------------------------------------------------- */
/* Residual addition and layer norm                                                           */
/* ---------------------------------------------------------------------------------------- */

/* For each row, all as above but
 *     mean = mean_c h_c,   s = 1 / sqrt(mean_c (h_c - mean)^2 + eps)     (f32, over the unrounded h, the mean first)
 *     y_c  = (h_c - mean) s weight_c + bias_c                            (weight NULL: 1, bias NULL: 0)
 * weight_dtype is the bias's too.  A row whose squares about the mean overflow f32 has rstd 0; one whose sum does has an
 * infinite mean and NaN in y. */
typedef dtt_rmsnorm_desc dtt_layernorm_desc;

/* As dtt_rmsnorm_forward, with the bias, and the mean ([rows] f32, or NULL) beside rstd. */
int dtt_layernorm_forward(const dtt_layernorm_desc* desc, uint64_t rows, const void* x, uint64_t x_pitch,
                          const void* residual, uint64_t residual_pitch, const void* weight, const void* bias,
                          void* residual_out, uint64_t residual_out_pitch, void* y, uint64_t y_pitch,
                          float* scales, float* mean, float* rstd, cudaStream_t stream);

/* As dtt_rmsnorm_backward, from the forward's mean and rstd:  with n_c = (h_c - mean) rstd, g_c = dy_c weight_c,
 *     dx_c = rstd (g_c - mean_c(g_c) - n_c mean_c(g_c n_c)) + dres_c
 *     dweight_c = sum over rows of dy_c n_c,  dbias_c = sum over rows of dy_c      (f32)
 * dweight and dbias may each be NULL (both: workspace is unused).  rows 0: those that are given are zeroed.
 *  - workspace: dtt_layernorm_workspace's bytes, 16-byte aligned. */
int dtt_layernorm_backward(const dtt_layernorm_desc* desc, uint64_t rows, const void* dy, uint64_t dy_pitch,
                           const void* h, uint64_t h_pitch, const void* weight, const float* mean, const float* rstd,
                           const void* dres, uint64_t dres_pitch, void* dx, uint64_t dx_pitch, float* dweight,
                           float* dbias, void* workspace, uint64_t workspace_bytes, cudaStream_t stream);

/* Bytes of dtt_layernorm_backward's workspace, for any number of rows.  Errors: DTT_EINVAL. */
int dtt_layernorm_workspace(const dtt_layernorm_desc* desc, uint64_t* bytes);

/* ---------------------------------------------------------------------------------------- */
/* Orthogonalising an update by Newton-Schulz products                                        */
/* ---------------------------------------------------------------------------------------- */

/* For each of `batch` matrices G of rows x cols:
 *     u  = G                          without momentum
 *     M <- mu M + G, u = M            with momentum (M is updated in place)
 *     M <- mu M + G, u = G + mu M     with nesterov (M the new one)
 *     X  = u / (|u|_F + eps), transposed where rows > cols
 *     `steps` times, with step k's coefficients (a, b, c):
 *         A = X X^T;  X <- a X + (b A + c A A) X
 *     out = scale X (transposed back), rounded to bf16.
 * Each step maps every singular value s of X to a s + b s^3 + c s^5 and keeps the singular
 * vectors.  The products run on the tensor cores with f16 operands and f32 sums; X itself is held
 * in 32 bits (two f16 halves, 22 significant bits), because a rounded iterate's noise in the
 * directions that u lacks would grow by a (3.44 with the usual coefficients) in every step.  A is
 * rounded to f16, and b A + c A A to two f16 terms where the smaller side is 128 at most (256 for
 * most shapes), to one beyond.  Five usual steps end 1.7e-3 to 2.6e-3 of the result's norm off 64 bits,
 * of which the bf16 output's own rounding is 1.66e-3; a matrix with a handful of singular values, all
 * where a step is steep, up to 1e-2.
 * |u|^2 is summed in f32: where it overflows (|u| of 1.8e19 or more) the result is zeros, and elements below
 * 1e-19 add nothing to it (eps has to be well above what |u| is then).  Elements of X below 2^-36 are 0, as
 * all are where eps is 1e10 times |u|.  A NaN or an infinity makes its matrix NaN, and no other of the batch.
 * Large matrices run as one cooperative launch over all SMs: it begins when they are free. */
#define DTT_ORTHO_MAX_STEPS 32

typedef struct dtt_ortho_desc {
    uint32_t x_dtype;        /* G: DTT_BF16 or DTT_F32 */
    uint32_t batch;          /* >= 1 */
    uint64_t rows, cols;     /* each 1 .. 65536 */
    uint32_t steps;          /* 1 .. DTT_ORTHO_MAX_STEPS */
    uint32_t momentum;       /* 0: u = G; 1: M is an argument of every call */
    uint32_t nesterov;       /* with momentum: 1: u = G + mu M */
    float mu;                /* finite; used with momentum */
    float eps;               /* finite, > 0 */
    float scale;             /* finite */
    float coeffs[DTT_ORTHO_MAX_STEPS][3];   /* (a, b, c) of each step.  They must keep the iterate
                                within f16: with p_k(s) = a s + b s^3 + c s^5 and bound_0 = 1,
                                bound_{k+1} = max over s in [0, bound_k] of |p_k(s)| stays <= 16, and
                                |b| bound_k^2 + |c| bound_k^4 <= 1024 (DTT_EINVAL otherwise) */
} dtt_ortho_desc;

typedef struct dtt_ortho dtt_ortho;

/* Bytes of the workspace that a desc needs.  Errors: DTT_EINVAL (a bad desc). */
int dtt_ortho_workspace(const dtt_ortho_desc* desc, uint64_t* bytes);

/* A handle: the desc, checked, and the tensor maps of its workspace, which the caller owns, keeps
 * until the handle's last call has finished on the GPU, and gives to no other handle meanwhile
 * (device, 256-byte aligned, workspace_bytes long).  Calls on one handle share the workspace: run
 * them on one stream, or order the streams.
 * Errors: DTT_EINVAL (also a workspace that is short or misaligned), DTT_ENOMEM, DTT_ECUDA. */
int dtt_ortho_create(const dtt_ortho_desc* desc, void* workspace, uint64_t workspace_bytes, dtt_ortho** out);

/* Run it.  x, momentum (f32; NULL exactly where the desc has none) and out (bf16): matrix i starts
 * i * stride bytes after the first, rows `pitch` bytes apart; the matrices follow one another, or their rows
 * alternate.  No output overlaps an input.
 * err: device uint32, incremented where a bounded internal wait gives up (0 after a clean run;
 * otherwise the outputs are unspecified, the call has ended all the same, and the next one is as ever).
 * Errors: DTT_EINVAL (pointers, alignment to the element, pitches, strides), DTT_ECUDA. */
int dtt_ortho_run(dtt_ortho* o, const void* x, uint64_t x_pitch, uint64_t x_stride, float* momentum,
                  uint64_t momentum_pitch, uint64_t momentum_stride, void* out, uint64_t out_pitch,
                  uint64_t out_stride, uint32_t* err, cudaStream_t stream);

/* Release the handle (the workspace stays the caller's). */
void dtt_ortho_destroy(dtt_ortho* o);

/* ---------------------------------------------------------------------------------------- */
/* Tokens' rows sorted by expert, and back                                                     */
/* ---------------------------------------------------------------------------------------- */

/* Expert parallelism between an all-gather and a reduce-scatter: a rank that holds experts first .. first + experts - 1
 * sorts the gathered tokens' rows by expert, runs its experts' products on them, and adds the results, weighted, to
 * its partial sum for every token.  A pair (t, j) is token t's choice j of top_k. */
typedef struct dtt_experts_desc {
    uint32_t experts;        /* of this rank: 1 .. 1024 */
    uint32_t first;          /* the id of the first one: below 2^31 */
    uint32_t top_k;          /* choices of a token: 1 .. 32 */
    uint32_t align;          /* an expert's rows are filled up to a multiple of this: 1 .. 65536 */
} dtt_experts_desc;

/* Where each pair's row goes.  ids: device [tokens][top_k] of 4 or 8 bytes; an id that is not one of this rank's experts
 * (another rank's, a negative one: no choice) has no row here.  An id may come twice in a token.
 *     offsets[0] = 0, offsets[e + 1] = offsets[e] + counts[e] rounded up to a multiple of align,
 *     position[t][j] = offsets[e] + the number of pairs before (t, j), token by token, with the same expert e,
 * or -1 for a pair without a row here.  position: int32 [tokens][top_k], offsets: int32 [experts + 1], counts: int32
 * [experts].  Rows from max_rows on do not exist: pairs that would go there get -1 too, and offsets and counts end
 * there.  tokens top_k + experts (align - 1) rows are always enough.  The result is the same every time.
 *  - workspace: dtt_experts_workspace's bytes, 16-byte aligned; calls that share it run in order.
 * tokens 0: offsets and counts are zeroed.  tokens top_k + experts align and max_rows are below 2^31.
 * Errors: DTT_EINVAL, DTT_ECUDA; so below. */
int dtt_experts_route(const dtt_experts_desc* desc, uint64_t tokens, const void* ids, uint32_t id_bytes, uint64_t max_rows,
                      int32_t* position, int32_t* offsets, int32_t* counts, void* workspace, uint64_t workspace_bytes,
                      cudaStream_t stream);

/* Bytes of dtt_experts_route's workspace, for any number of tokens. */
int dtt_experts_workspace(const dtt_experts_desc* desc, uint64_t* bytes);

/* rows[position[t][j]] = x[t], and zeros in the rows that fill an expert's up (so that products over them add nothing);
 * rows from offsets[experts] on are left as they were.  Rows are moved as they are, row_bytes (1 .. 2^26) of any
 * type; with scales, scale_count f32 a row, row_scales[position[t][j]] = scales[t] the same way (NULL both: none;
 * those of 0 tokens or of 0 rows may be NULL by themselves, as x and rows then may).
 * position, offsets, counts: dtt_experts_route's for the same desc; a position is looked at before it is used (one
 * that is not below max_rows has no row), two equal ones leave either row.  No output overlaps an input. */
int dtt_experts_dispatch(const dtt_experts_desc* desc, uint64_t tokens, const int32_t* position, const int32_t* offsets,
                         const int32_t* counts, const void* x, uint64_t x_pitch, uint64_t row_bytes, void* rows,
                         uint64_t rows_pitch, uint64_t max_rows, const float* scales, uint64_t scales_pitch,
                         uint64_t scale_count, float* row_scales, uint64_t row_scales_pitch, cudaStream_t stream);

/* out[t] = sum over j of weights[t][j] rows[position[t][j]], of the pairs that have a row, in f32 in j's order, rounded once;
 * a token without any gets zeros.  weights: f32 [tokens][top_k], NULL: 1, which is the dispatch's gradient (rows: the
 * gradient of its rows, out: that of x).  Rows that no pair goes to are not read.  rows, out: bf16 or f32. */
int dtt_experts_combine(const dtt_experts_desc* desc, uint64_t tokens, uint64_t cols, const int32_t* position, const void* rows,
                        uint32_t rows_dtype, uint64_t rows_pitch, uint64_t max_rows, const float* weights, void* out,
                        uint32_t out_dtype, uint64_t out_pitch, cudaStream_t stream);

/* The combination's gradients:
 *     drows[position[t][j]] = weights[t][j] dout[t]                  (rounded once to the rows' type)
 *     dweights[t][j] = sum over c of dout[t][c] rows[position[t][j]][c]   (f32; 0 for a pair without a row)
 * and zeros in the rows of drows that fill an expert's up; those from offsets[experts] on are left as they were.
 * dweights may be NULL (rows is then not read).  dout, and rows and drows: bf16 or f32.  The same call gives
 * the same bits.  drows may be rows itself, with one pitch, where dweights is NULL; no other overlap. */
int dtt_experts_combine_backward(const dtt_experts_desc* desc, uint64_t tokens, uint64_t cols, const int32_t* position,
                                 const int32_t* offsets, const int32_t* counts, const void* dout, uint32_t dout_dtype,
                                 uint64_t dout_pitch, const void* rows, uint32_t rows_dtype, uint64_t rows_pitch,
                                 uint64_t max_rows, const float* weights, void* drows, uint64_t drows_pitch,
                                 float* dweights, cudaStream_t stream);

/* ---------------------------------------------------------------------------------------- */
/* AdamW over the tensors of a rank's share                                                    */
/* ---------------------------------------------------------------------------------------- */

/* For each element of each tensor, in f32, at step t (1, 2, ...) with the rate lr:
 *     g = grad_scale grad
 *     m <- beta1 m + (1 - beta1) g
 *     v <- beta2 v + (1 - beta2) g^2
 *     p <- p - lr weight_decay p - lr / (1 - beta1^t) m / (sqrt(v) / sqrt(1 - beta2^t) + eps)
 *     copy = p, rounded to bf16 (where there is one: the all-gather's part of the new weights)
 * States: DTT_F32, m and v as they are; or DTT_E4M3: m and sqrt(v) in codes of 8 bits, with one f32 scale for
 * each DTT_ADAMW_BLOCK elements of a tensor (the last block holds what is left),
 *     scale = max(max |x| / 448, 2^-100) over the block (to an ulp),  code = e4m3(x / scale) (x / scale to a few ulp),
 * but a root above zero has the code 2^-9 at least, since the next step divides by it, and a block's largest is
 * rounded at random as the formula's products and sums, each rounded to f32 by itself, leave it.  The step itself uses the
 * new m and v before they are rounded.  All states zero, their scales too, is the start.
 * stochastic = 0: codes and bf16 weights are rounded to nearest.  1: up, away from zero, with the probability of
 * what lies below, so that small changes that nearest would lose each time add up on average; a copy stays
 * rounded to nearest.  The random numbers are a function of seed, step, the tensor's number in the list and the
 * element's in the tensor alone: with mix(x) = { x ^= x >> 16; x *= 0x85A308D3; x ^= x >> 15; x *= 0xB7E15163;
 * x ^= x >> 16 } on 32 bits and r = mix(i 0x9E3779B9 + (i >> 32) 0x2E1B2139 + mix(mix(mix(seed) + t) + tensor)),
 * m is rounded by r's high 16 bits, sqrt(v) by its low 16, p by the high 16 of r 0x2E1B2139.  They take the
 * place of the highest 16 of the bits that are cut off.
 * The same call on the same values gives the same bits.  v and its root are f32, a subnormal v (gradients below 1e-18 or
 * so) with the digits that are left there, and with 8-bit states all of them down to 2^-150: (1 - beta2) g^2 below 2^-150
 * adds nothing to v; gradients above 1e19 make it infinite and the step zero.  NaN in a gradient makes its element's p, m and v NaN, with
 * 8-bit states its block's from the next step on; so does an infinity there. */
#define DTT_ADAMW_BLOCK 128

typedef struct dtt_adamw_desc {
    uint32_t param_dtype;    /* DTT_BF16 or DTT_F32 */
    uint32_t grad_dtype;     /* DTT_BF16 or DTT_F32 */
    uint32_t state_dtype;    /* DTT_F32 or DTT_E4M3 */
    uint32_t stochastic;     /* 0 or 1 */
    double beta1, beta2;     /* each in [0, 1) */
    float eps;               /* finite, 2^-100 or more */
    uint32_t seed;           /* used with stochastic */
} dtt_adamw_desc;

/* One tensor: n contiguous elements at any alignment that their types allow.  Those whose param, grad, m, v and copy are
 * all 16-byte aligned at the same element (8-bit states: at the first) take the fast path. */
typedef struct dtt_adamw_tensor {
    void* param;
    const void* grad;
    void* m;                 /* states: f32, or codes */
    void* v;
    float* m_scales;         /* 8-bit states: [ceil(n / DTT_ADAMW_BLOCK)]; f32: NULL */
    float* v_scales;
    void* copy;              /* bf16, or NULL; with f32 weights alone */
    uint64_t n;              /* 0 .. 2^40 - 1; 0: nothing is read or written, pointers may be NULL */
    float weight_decay;      /* finite */
    uint32_t reserved;       /* 0 */
} dtt_adamw_tensor;

typedef struct dtt_adamw dtt_adamw;

/* A handle: the desc and the list of tensors, checked and kept on the host (it holds no device memory).  The
 * buffers stay the caller's; none that is written overlaps another one, or a gradient (gradients may one another), which is
 * refused for the list's own: a tensor comes once.
 * Errors: DTT_EINVAL, DTT_ENOMEM, DTT_ECUDA. */
int dtt_adamw_create(const dtt_adamw_desc* desc, const dtt_adamw_tensor* tensors, uint32_t count, dtt_adamw** out);

/* One step over all tensors.
 *  - grads: NULL, or this step's gradients in the list's order (those of empty tensors are not looked at), which overlap
 *    nothing that is written.
 *  - lr_dev: device f32, read when the kernels run; lr is then not used.  NULL: lr, which must be finite.
 *  - step_dev: device uint32, the steps made so far, which the call counts up first: what a graph that is
 *    replayed needs.  step is then not used.  NULL: step, 1 or more.
 *  - grad_scale: device f32 that gradients are multiplied by (clipping, a loss scale), or NULL: 1.
 * Calls that share a handle may run on any streams as far as their buffers allow.  Errors: DTT_EINVAL, DTT_ECUDA. */
int dtt_adamw_run(dtt_adamw* o, const void* const* grads, float lr, uint32_t step, const float* lr_dev,
                  uint32_t* step_dev, const float* grad_scale, cudaStream_t stream);

/* Release the handle. */
void dtt_adamw_destroy(dtt_adamw* o);

#ifdef __cplusplus
}
#endif

#endif /* DTT_OPS_H */
