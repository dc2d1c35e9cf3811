/*
 * dtt_ops.h -- operators on the block of rows that a rank owns between a reduce-scatter and an
 * all-gather: the residual's addition with a root-mean-square norm (bf16, f32 or 8-bit output),
 * its backward pass, and the orthogonalisation of a momentum update by Newton-Schulz products.
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

#ifdef __cplusplus
}
#endif

#endif /* DTT_OPS_H */
