/*
 * ptored_block.h -- C ABI of the block-boundary operators that follow the
 * cross-rank reduction in a tensor-parallel model, on one MI355X (gfx950),
 * and of the 8-bit activation checkpoints that a training step keeps.
 *
 * Notation: T rows (tokens), D columns (channels), all buffers row-major with
 * unit column stride; `ld` is a row pitch in elements (bytes for the packed
 * checkpoints).  Any alignment that the element type itself has is accepted,
 * and any pitch of at least the columns.
 *
 * The block boundary:
 *     h  = y_0 + ... + y_{N-1}                    the N ranks' partial outputs
 *     p  = h r1 (w1 + o),  r1 = 1/sqrt(mean_d(h^2) + eps)   (no w1: p = h)
 *     x' = beta x + alpha g p                               (no gate: g = 1)
 *     z  = x' r2 (w2 + o), r2 = 1/sqrt(mean_d(x'^2) + eps)  (no w2: no z)
 * computed in binary32 from the first load to the stores: sums of squares and
 * the fold (ascending rank) included; each output is rounded once.  A row
 * whose mean square passes binary32's range has r = 0, as the formula gives
 * in binary32.
 *
 * The 8-bit form of a T x D activation: 32 consecutive elements of a row (the
 * last block of a row may be shorter) share a power of two 2^E, the smallest
 * E in [-120, 127] for which rint(amax 2^(6-E)) <= 127.  q = rint(v 2^(6-E))
 * (ties to even; at E = 127 limited to +-127) is kept as int8, E + 127 as one
 * byte; the value kept is q 2^(E-6), off by at most 2^(E-7) (2^(E-6) at
 * E = 127), and exact in bfloat16.  A block that holds an infinity or a NaN
 * keeps scale byte 255 and stands for NaN throughout.
 *
 * Status codes, element types and the stream rules are those of ptored.h:
 * every call is asynchronous on `stream`, allocates nothing, synchronises
 * nothing, can be captured in a graph, and checks its arguments before any
 * HIP call in the order INVALID_ARG (counts, null pointers, shapes),
 * UNSUPPORTED (types, i32 among them, or more than PTORED_BLOCK_MAX_COLS
 * columns), INVALID_ARG (the workspace, alignment), OVERLAP.  Buffers overlap
 * where they share a byte: two column ranges of one matrix do not, nor does a
 * buffer in the gaps between a matrix's rows.  Of two matrices in rows of
 * different pitches, both with gaps, it is their spans that count, from the
 * first byte to the last.  Zero rows or columns are no error.
 * Results do not vary from run to run.
 */
#ifndef PTORED_BLOCK_H
#define PTORED_BLOCK_H

#include "ptored.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Most columns of the norm operators (a row stays in registers). */
#define PTORED_BLOCK_MAX_COLS 16384
/* Elements of a row that share one scale byte of a packed checkpoint. */
#define PTORED_CHECKPOINT_BLOCK 32

/* A T x D matrix of elements; data may be NULL where a call says so. */
typedef struct ptored_rows {
    void* data;
    int64_t ld; /* elements from one row to the next */
} ptored_rows;

/* A T x D matrix in 8 bits: T x D int8 and T x ceil(D/32) scale bytes. */
typedef struct ptored_checkpoint {
    void* q;
    int64_t q_ld; /* bytes from one row of q to the next, >= D */
    void* scales;
    int64_t scales_ld; /* bytes, >= ceil(D/32) */
} ptored_checkpoint;

/* What the forward and the backward pass share. */
typedef struct ptored_block_params {
    int64_t rows, cols; /* T, D */
    const void* post_weight; /* w1 [D], or NULL: no norm after the block */
    const void* pre_weight;  /* w2 [D], or NULL: no norm before the next block */
    ptored_rows gate; /* g: gate_rows x D of `dtype`, or data NULL: no gate */
    int64_t gate_rows; /* divides rows; row t takes gate row t / (rows / gate_rows).
                          Not read without a gate */
    float weight_offset;  /* o, added to both weights (1: weights kept as offsets from 1) */
    float branch_scale;   /* alpha */
    float residual_scale; /* beta */
    float eps;            /* >= 0; not read by the backward pass */
    int32_t dtype;        /* F32, BF16 or F16: activations and gate */
    int32_t weight_dtype; /* F32 or `dtype`: both weights and their gradients */
} ptored_block_params;

/* Buffers of the forward pass.  Any output may be NULL. */
typedef struct ptored_block_io {
    ptored_rows x;     /* residual stream, required */
    ptored_rows x_out; /* x'; may be x itself */
    ptored_rows z;     /* needs pre_weight */
    ptored_rows h;     /* the fold, for the backward pass; may be parts[r] */
    float* post_rstd;  /* r1 [T], needs post_weight */
    float* pre_rstd;   /* r2 [T], needs pre_weight */
    /* 8-bit forms of h, x' and z as rounded to `dtype` (q NULL: not wanted) */
    ptored_checkpoint h_kept, x_kept, z_kept;
} ptored_block_io;

/*
 * ptored_block_norm -- the block boundary, forward.
 *
 * parts  HOST array of nranks DEVICE pointers, T x D each with pitch part_ld,
 *        0 <= nranks <= PTORED_MAX_RANKS.  With none, x' = beta x (the norm
 *        before the first block): post_weight, gate, h and h_kept must be
 *        absent.
 * An output may be exactly an input matrix of the same pitch (of any pitch, if
 * T is 1); every other overlap of an output is rejected.
 */
int ptored_block_norm(const void* const* parts, int nranks, int64_t part_ld,
                      const ptored_block_params* params, const ptored_block_io* io,
                      hipStream_t stream);

/* Buffers of the backward pass. */
typedef struct ptored_block_grad_io {
    ptored_rows dz;     /* gradient of z; required with pre_weight, absent without */
    ptored_rows dx_out; /* gradient that reaches x' past z; NULL: none (then dz is needed) */
    /* activations of the forward pass, both in `dtype` or both packed:
     * x' is needed with pre_weight, h with post_weight or dgate */
    ptored_rows x_out, h;
    ptored_checkpoint x_kept, h_kept;
    const float* post_rstd; /* needed with post_weight */
    const float* pre_rstd;  /* needed with pre_weight */
    ptored_rows dx; /* gradient of x; may be dz, dx_out, x_out or h itself; or NULL */
    ptored_rows dh; /* gradient of h, and of every rank's partial; likewise */
    ptored_rows dgate; /* gate_rows x D; NULL: not wanted */
    void* dpost_weight; /* [D] of weight_dtype; NULL: not wanted */
    void* dpre_weight;  /* [D] of weight_dtype; NULL: not wanted */
    void* workspace; /* ptored_block_norm_backward_workspace bytes, 16-byte aligned */
    int64_t workspace_bytes;
} ptored_block_grad_io;

/*
 * ptored_block_norm_backward -- gradients of the block boundary:
 *     xh = x' r2,  u = dz (w2 + o),  s = dx_out + r2 (u - xh mean_d(u xh))
 *     dx = beta s,   dw2 = sum_t dz xh
 *     hh = h r1,  e = alpha g s,  v = e (w1 + o)
 *     dh = r1 (v - hh mean_d(v hh))   (no w1: dh = e),   dw1 = sum_t e hh
 *     dg = sum of alpha p s over the rows that share the gate row
 * in binary32, each output rounded once.  Zero rows give zero gradients.
 */
int ptored_block_norm_backward(const ptored_block_params* params,
                               const ptored_block_grad_io* io, hipStream_t stream);

/* Bytes of workspace that the backward pass of such a call needs (no HIP
 * call); gate_rows 0 without a gate. */
int ptored_block_norm_backward_workspace(int64_t rows, int64_t cols, int64_t gate_rows,
                                         int64_t* bytes);

/* ptored_checkpoint_pack -- the 8-bit form of x (T x D of `dtype`). */
int ptored_checkpoint_pack(ptored_rows x, int64_t rows, int64_t cols, int dtype,
                           ptored_checkpoint kept, hipStream_t stream);

/* ptored_checkpoint_unpack -- out = the values kept, rounded to `dtype`
 * (exact for F32 and BF16; F16 overflows to infinity past 65504). */
int ptored_checkpoint_unpack(ptored_checkpoint kept, int64_t rows, int64_t cols, int dtype,
                             ptored_rows out, hipStream_t stream);

/*
 * ptored_checkpoint_wgrad -- a projection's weight gradient from its packed
 * input: dw[o, i] = sum_t dy[t, o] x[t, i] (+ dw[o, i] with accumulate),
 * products exact and sums in binary32, rounded once to dw_dtype (of F32, a dy
 * below 2^-110 is cut to a multiple of 2^-133 first).  dy is rows x outs of
 * `dtype`; x is rows x cols; dw is outs x cols of dw_dtype, F32 or `dtype`.  Zero
 * rows give zeros (or leave dw, with accumulate).
 */
int ptored_checkpoint_wgrad(ptored_rows dy, ptored_checkpoint x, int64_t rows, int64_t outs,
                            int64_t cols, int dtype, ptored_rows dw, int dw_dtype,
                            int accumulate, void* workspace, int64_t workspace_bytes,
                            hipStream_t stream);

/* Bytes of workspace that such a weight gradient needs; often 0 (no HIP call). */
int ptored_checkpoint_wgrad_workspace(int64_t rows, int64_t outs, int64_t cols, int dtype,
                                      int64_t* bytes);

#ifdef __cplusplus
}
#endif

#endif /* PTORED_BLOCK_H */
