/*
 * ptored_step.h -- C ABI of the operators that a training or serving step of a
 * tensor-parallel model runs next to the cross-rank reduction and the block
 * boundary, on one MI355X (gfx950): the boundary of a model with layer norm,
 * the column-parallel half of a gated feed-forward block, and the clipping of
 * gradients by their global norm.
 *
 * Notation, matrices (ptored_rows), status codes, element types, streams, the
 * order of argument checks and what counts as an overlap are those of
 * ptored_block.h; matrices start at any element, and `ld` is any pitch of at
 * least the columns: gate and up may be the halves of one buffer.  Everything is
 * computed in binary32 or more from the first load to the stores, and each
 * output is rounded once, but for what a call says.  Results do not vary from
 * run to run.
 */
#ifndef PTORED_STEP_H
#define PTORED_STEP_H

#include "ptored_block.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ---------------------------------------------------------------- layer norm
 *
 *     x' = x + y_0 + ... + y_{N-1}                the N ranks' partial outputs
 *     m  = mean_d(x'),  r = 1/sqrt(mean_d((x' - m)^2) + eps)
 *     z  = (x' - m) r w + b
 * A row whose variance passes binary32's range has r = 0.
 */
typedef struct ptored_layer_norm_params {
    int64_t rows, cols;   /* T, D; D <= PTORED_BLOCK_MAX_COLS */
    const void* weight;   /* w [D], or NULL: ones */
    const void* bias;     /* b [D], or NULL: zeros; not read by the backward pass */
    float eps;            /* >= 0; not read by the backward pass */
    int32_t dtype;        /* F32, BF16 or F16: activations */
    int32_t weight_dtype; /* F32 or `dtype`: weight, bias and their gradients */
} ptored_layer_norm_params;

/*
 * ptored_layer_norm -- the boundary, forward.
 *
 * parts  HOST array of nranks DEVICE pointers, T x D each with pitch part_ld,
 *        0 <= nranks <= PTORED_MAX_RANKS.  With none, x' = x.
 * x is required; x_out (x'), z, mean (m [T]) and rstd (r [T]) may be NULL.  An
 * output may be exactly an input matrix of the same pitch (of any pitch, if T
 * is 1); every other overlap of an output is rejected.
 */
int ptored_layer_norm(const void* const* parts, int nranks, int64_t part_ld,
                      const ptored_layer_norm_params* params, ptored_rows x, ptored_rows x_out,
                      ptored_rows z, float* mean, float* rstd, hipStream_t stream);

/*
 * ptored_layer_norm_backward -- gradients of the boundary:
 *     xh = (x' - m) r,  u = dz w
 *     dx = dx_out + r (u - mean_d(u) - xh mean_d(u xh))
 *     dw = sum_t dz xh,  db = sum_t dz
 * dz, x_out (x'), mean and rstd are required; dx_out (the gradient that reaches
 * x' past z) may be NULL: none.  dx is the gradient of x and of every rank's
 * partial; dx, dweight and dbias may be NULL.  dx may be dz, dx_out or x_out
 * itself.  Zero rows give zero gradients.  The workspace has
 * ptored_layer_norm_backward_workspace bytes and is 16-byte aligned; without
 * dweight and dbias none is needed.
 */
int ptored_layer_norm_backward(const ptored_layer_norm_params* params, ptored_rows dz,
                               ptored_rows dx_out, ptored_rows x_out, const float* mean,
                               const float* rstd, ptored_rows dx, void* dweight, void* dbias,
                               void* workspace, int64_t workspace_bytes, hipStream_t stream);

/* Bytes of workspace for weights' gradients of such a call (no HIP call). */
int ptored_layer_norm_backward_workspace(int64_t rows, int64_t cols, int64_t* bytes);

/* ---------------------------------------------------------------- gated feed-forward
 *
 *     g = x Wg^T,  u = x Wu^T,  y = f(g) u
 * with x T x D, both weights F x D, and g, u, y T x F.  Products of 16-bit
 * types are exact, sums in binary32; f takes g as summed.  Products of F32 may be
 * taken as those of each operand's exact sum of three bfloat16, of which those
 * below 2^-21 of the whole are left out, and what an operand holds below 2^-133 is;
 * then an infinite operand gives NaN where binary32 gives an infinity.
 */
typedef enum ptored_activation {
    PTORED_SILU = 0,     /* f(g) = g / (1 + exp(-g)) */
    PTORED_GELU = 1,     /* f(g) = g (1 + erf(g / sqrt(2))) / 2 */
    PTORED_GELU_TANH = 2 /* f(g) = g (1 + tanh(sqrt(2/pi) (g + 0.044715 g^3))) / 2 */
} ptored_activation;

/* Longest rows (D and F) and largest pitch of the matrices that its products read,
 * in bytes; more is UNSUPPORTED.  dg and du alone are not products. */
#define PTORED_FFN_MAX_PITCH (1 << 22)

typedef struct ptored_ffn_params {
    int64_t rows, cols, wide; /* T, D, F */
    int32_t dtype;            /* F32, BF16 or F16 */
    int32_t activation;       /* ptored_activation */
} ptored_ffn_params;

/*
 * ptored_gated_ffn -- y, and with `gate` and `up` (data NULL: not wanted) also
 * g and u, each rounded to dtype, for the backward pass.  Outputs overlap
 * nothing.  Zero columns give zeros.
 */
int ptored_gated_ffn(const ptored_ffn_params* params, ptored_rows x, ptored_rows w_gate,
                     ptored_rows w_up, ptored_rows y, ptored_rows gate, ptored_rows up,
                     void* workspace, int64_t workspace_bytes, hipStream_t stream);

/* Bytes of workspace (16-byte aligned) that such a forward pass needs; 0 but where
 * few tokens meet few features (no HIP call). */
int ptored_gated_ffn_workspace(int64_t rows, int64_t cols, int64_t wide, int dtype, int64_t* bytes);

/* Buffers of the backward pass. */
typedef struct ptored_ffn_grad_io {
    ptored_rows dy;        /* gradient of y, T x F */
    ptored_rows gate, up;  /* g and u as the forward pass kept them */
    ptored_rows dgate, dup; /* T x F, required; each may be exactly dy, gate or up */
    ptored_rows x;         /* needed with dw_gate or dw_up */
    ptored_rows w_gate, w_up; /* needed with dx */
    ptored_rows dx;        /* T x D, or NULL: not wanted */
    ptored_rows dw_gate, dw_up; /* F x D of dw_dtype, or NULL: not wanted */
    int32_t dw_dtype;      /* F32 or dtype */
    int32_t accumulate;    /* nonzero: weight gradients are added to what is there */
    void* workspace;       /* ptored_gated_ffn_backward_workspace bytes, 16-byte aligned */
    int64_t workspace_bytes;
} ptored_ffn_grad_io;

/*
 * ptored_gated_ffn_backward -- gradients:
 *     dg = dy u f'(g),  du = dy f(g)
 *     dx = dg Wg + du Wu,  dWg = dg^T x,  dWu = du^T x  (+ what is there, with accumulate)
 * dg and du are rounded to dtype as they are stored, and the products take
 * them as stored: the matrix instructions' operands have that type.
 */
int ptored_gated_ffn_backward(const ptored_ffn_params* params, const ptored_ffn_grad_io* io,
                              hipStream_t stream);

/* Bytes of workspace that such a backward pass needs with any of the gradients;
 * often 0 (no HIP call). */
int ptored_gated_ffn_backward_workspace(int64_t rows, int64_t cols, int64_t wide, int dtype,
                                        int64_t* bytes);

/* ---------------------------------------------------------------- gradient clipping */

/* One gradient: rows x cols elements, contiguous where rows is 1 (fewer than 2^40;
 * of several rows fewer than 2^31, their pitches at most 2^27; more is
 * UNSUPPORTED). */
typedef struct ptored_grad {
    const void* data;
    void* out;      /* where the scaled gradient goes; may be data itself */
    int64_t rows, cols;
    int64_t ld, out_ld; /* pitches in elements; not read where rows is 1 */
    int32_t dtype;     /* F32, BF16 or F16 */
    int32_t out_dtype; /* dtype or F32 */
} ptored_grad;

/*
 * ptored_grad_norm -- norm[0] = sqrt(sum of all elements' squares), summed in
 * binary64 and rounded to binary32.  `grads` is a HOST array, read during the
 * call only; out fields are not read.  No gradients give 0; a NaN or an infinity
 * passes through.  A gradient may be listed twice and then counts twice.
 */
int ptored_grad_norm(const ptored_grad* grads, int64_t count, float* norm, void* workspace,
                     int64_t workspace_bytes, hipStream_t stream);

/*
 * ptored_grad_scale -- out = data c for every gradient, with c = max_norm /
 * norm[0] where norm[0] > max_norm, 1 where it is not, and NaN where it is NaN.
 * `norm` is a DEVICE pointer, read when the kernels run: it may be what an
 * all-reduce of several ranks' norms left.  c is rounded to binary32 and every
 * product once to out_dtype.  max_norm >= 0 (infinity: c = 1).  An out is its
 * data exactly (type and pitch too) or overlaps no gradient's data or out;
 * column slices of one buffer do not overlap.
 */
int ptored_grad_scale(const ptored_grad* grads, int64_t count, const float* norm, float max_norm,
                      void* workspace, int64_t workspace_bytes, hipStream_t stream);

/* ptored_grad_clip -- both: the norm into norm[0], and the gradients scaled by
 * it as ptored_grad_scale scales them. */
int ptored_grad_clip(const ptored_grad* grads, int64_t count, float max_norm, float* norm,
                     void* workspace, int64_t workspace_bytes, hipStream_t stream);

/* Bytes of workspace (16-byte aligned) of each of the three calls for these
 * gradients (no HIP call; only shapes and types are read). */
int ptored_grad_norm_workspace(const ptored_grad* grads, int64_t count, int64_t* bytes);

#ifdef __cplusplus
}
#endif

#endif /* PTORED_STEP_H */
