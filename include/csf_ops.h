/*
 * csf_ops.h -- C ABI of the expert-layer operators in libcsf.so: what a
 * caller of csf_decode runs on either side of the decoded scales.
 *
 *   csf_rms_norm       residual addition, root-mean-square norm and
 *                      quantisation of a layer's input, in one pass
 *   csf_route          top-k router: expert choice, weights, and the slots
 *                      grouped by expert (expert_start, as csf_decode takes it)
 *   csf_expert_matmul  block-scaled product of quantised rows with the FP4
 *                      weights of the experts that own them; the weight
 *                      scales are a CSF_LAYOUT_BLOCKED workspace of csf_decode;
 *                      bias, activation (plain or gated), row weight, residual
 *                      and output quantisation in the epilogue
 *
 * The conventions of csf.h hold: device pointers owned by the caller, calls
 * asynchronous on `stream`, no allocation, no host synchronisation, argument
 * and launch errors as a csf_status, data errors as CSF_DEV_ERR_* bits OR-ed
 * into the optional device word `error_word`.  Arguments are checked on the
 * host before any CUDA call; a pointer off the alignment of its element is
 * CSF_ERR_ARG.
 */
#ifndef CSF_OPS_H
#define CSF_OPS_H

#include "csf.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Element types of plain tensors. */
typedef enum { CSF_BF16 = 0, CSF_F16 = 1, CSF_F32 = 2 } csf_dtype;

/* Quantised rows.  A row of `cols` values is held as codes and one scale byte
 * per block of values; columns past `cols` up to the next multiple of 32 are
 * coded 0.
 *   CSF_ROWS_NVFP4  E2M1 codes, two a byte (even column in the low nibble);
 *                   a UE4M3 scale per 16 columns; value = code * scale *
 *                   tensor scale.
 *   CSF_ROWS_MXFP8  E4M3 codes, one a byte; a UE8M0 scale (2^(byte - 127),
 *                   255 = NaN) per 32 columns; value = code * scale.
 * Scale rows are row-major, `scale_stride` bytes apart (a multiple of 16);
 * bytes past the row's blocks are 0 up to the next multiple of 16.
 * How a block of values v with largest magnitude m becomes codes:
 *   NVFP4: scale = m / (6 * tensor scale) rounded to UE4M3 (ties to even,
 *          at most 448); code = v / (scale * tensor scale) rounded to E2M1
 *          (ties to even, saturating); 0 where the scale rounds to 0.
 *   MXFP8: scale = the smallest power of two with m <= 448 * scale (2^-127 at
 *          least); code = v / scale rounded to E4M3 (ties to even).
 * A block that holds an infinity or a NaN gets a NaN scale (0x7F, 255). */
typedef enum { CSF_ROWS_NVFP4 = 0, CSF_ROWS_MXFP8 = 1 } csf_rows_kind;

typedef struct {
    int32_t kind;              /* csf_rows_kind */
    int32_t cols;              /* values per row, >= 1 */
    int64_t rows;              /* >= 0 */
    uint8_t *codes;            /* 16-byte aligned */
    int64_t code_stride;       /* bytes between rows, a multiple of 16 */
    uint8_t *scales;           /* 16-byte aligned */
    int64_t scale_stride;      /* bytes between rows, a multiple of 16 */
    const float *tensor_scale; /* NVFP4 output: device scalar, 2^-117 .. 2^125 (its products with scales
                                  are normal numbers), NULL = 1; not read elsewhere */
} csf_rows;

/*
 * h = x + residual (in 32 bits); sum_out = h rounded to the type of x;
 * y = h / sqrt(mean(h^2) + eps) * weight, quantised to `out`.  The norm is of
 * the unrounded h, over the whole range of finite h: squares past float32's
 * range are summed scaled.  An infinite h makes its own y NaN and the row's
 * others 0, a NaN all of them NaN.
 */
typedef struct {
    const void *x;          /* [rows][cols] of dtype, row stride x_stride elements */
    int64_t x_stride;
    const void *residual;   /* optional, same type; NULL: h = x */
    int64_t residual_stride;
    void *sum_out;          /* optional [rows][cols] of dtype; may be `residual` or `x` itself */
    int64_t sum_stride;
    const void *weight;     /* [cols] of dtype */
    int32_t dtype;          /* csf_dtype of x, residual, sum_out and weight */
    float eps;
    csf_rows out;           /* kind, rows, cols and destination */
} csf_rms_norm_args;

/*
 * One launch.  Any alignment of x, residual, sum_out and weight to their
 * element; rows of 16-byte aligned addresses and widths load wide.
 * Errors: CSF_ERR_ARG (NULL, misaligned or short strides, unknown kind or
 * type), CSF_ERR_CUDA.
 */
csf_status csf_rms_norm(const csf_rms_norm_args *a, void *stream);

/*
 * Top-k router.  Per token the k largest logits in descending order, ties to
 * the lower expert; NaN counts as larger than every number.  A logit of -inf
 * switches the expert off for the token: where fewer than k are left, the
 * rest of ids and slots is -1 and of weights 0.
 *   weights: softmax over all experts (renormalize = 0) or over the chosen
 *   ones (1), in 32 bits.
 *   expert_start[e]: number of chosen (token, expert) pairs with an expert
 *   below e; slots are numbered by expert, then by token.  rows[slot] is the
 *   slot's token (-1 for slots at or past expert_start[experts]);
 *   slots[token][j] the slot of choice j.
 * Deterministic: the slot order depends on the logits alone.
 */
typedef struct {
    const void *logits;    /* [tokens][experts] of dtype, row stride logits_stride elements */
    int64_t logits_stride;
    int32_t dtype;         /* csf_dtype */
    int32_t tokens;        /* >= 0; tokens * k < 2^31 */
    int32_t experts;       /* 1 .. 1024 */
    int32_t k;             /* 1 .. min(32, experts) */
    int32_t renormalize;
    int32_t *ids;          /* [tokens][k] */
    float *weights;        /* [tokens][k] */
    int32_t *expert_start; /* [experts + 1] */
    int32_t *rows;         /* [tokens * k] */
    int32_t *slots;        /* [tokens][k] */
    void *scratch;         /* device, 16-byte aligned, csf_route_scratch_bytes(); NULL if that is 0 */
    size_t scratch_bytes;
} csf_route_args;

/* Scratch bytes of csf_route (0 for up to 512 tokens).  Host only. */
size_t csf_route_scratch_bytes(int32_t tokens, int32_t experts);

/* One launch for up to 512 tokens, else three.  Errors: CSF_ERR_ARG,
 * CSF_ERR_SIZE (scratch), CSF_ERR_UNSUPPORTED (experts or k beyond the
 * limits), CSF_ERR_CUDA. */
csf_status csf_route(const csf_route_args *a, void *stream);

typedef enum { CSF_ACT_NONE = 0, CSF_ACT_RELU = 1, CSF_ACT_SILU = 2, CSF_ACT_GELU_TANH = 3 } csf_act;

/*
 * For slot s of expert e (expert_start[e] <= s < expert_start[e+1]) and x row
 * r = rows[s] (or s):
 *   p[n] = alpha[e] * sum_k x[r][k] * w[e][n][k] + bias[e][n]
 *   plain:  y[n] = act(p[n]),                   0 <= n < N
 *   gated:  y[n] = act(p[n]) * p[N/2 + n],      0 <= n < N/2
 *   out[s][n] = y[n] * row_scale[s] + residual[s][n]
 * with x and w as the values they stand for without their tensor scales
 * (alpha carries the product of those).  x NVFP4 goes with w NVFP4, x MXFP8
 * with w MXFP4.  Sums in 32 bits, a matrix step (64 columns NVFP4, 32 MXFP8)
 * at a time, each of which may be off by a unit in the last place of what it
 * holds: a sum is within (K / 32 + 4) 2^-23 of sum_k |x w|.  SiLU and GELU are
 * within 2^-20 of their value, GELU with 2^-21 |z| more, z the argument of its
 * exponential.  Slots at or past expert_start[E] are not written; with an
 * expert_start that is out of order or range, none is.  A row index out of
 * range stands for row 0.
 */
typedef struct {
    csf_rows x;              /* rows x cols (= K); K a multiple of 32 (NVFP4) or 128 (MXFP8) */
    const int32_t *rows;     /* optional [slots]: the x row of each slot */
    int64_t slots;           /* >= 0, < 2^31; rows NULL: slots <= x.rows */
    int32_t experts;         /* E, 1 .. 8192 */
    int32_t n;               /* N weight rows per expert; gated: a multiple of 256 */
    const uint8_t *w;        /* [E][N][K/2] E2M1 codes, even column in the low nibble; 32-byte aligned */
    const uint8_t *w_scales; /* E stacks of N x K/16 (K/32) scales in CSF_LAYOUT_BLOCKED; 16-byte aligned */
    const void *expert_start;/* [E+1]; NULL: E must be 1 and owns every slot */
    int32_t expert_start_is_int64;
    const float *alpha;      /* optional [E] */
    const void *bias;        /* optional [E][N] of bias_dtype */
    int32_t bias_dtype;
    int32_t act;             /* csf_act */
    int32_t gated;
    const float *row_scale;  /* optional [slots] */
    const void *residual;    /* optional [slots][F] of residual_dtype, F = N or N/2 */
    int64_t residual_stride; /* elements */
    int32_t residual_dtype;
    int32_t out_dtype;       /* plain output: csf_dtype; read when out != NULL */
    void *out;               /* plain output [slots][F], row stride out_stride elements; or NULL: */
    int64_t out_stride;
    csf_rows out_rows;       /* quantised output: kind, cols = F, rows = slots (see csf_rows) */
    uint32_t *error_word;    /* optional: CSF_DEV_ERR_CORRUPT (a row index or expert_start out of range),
                                CSF_DEV_ERR_TIMEOUT (a bounded wait gave up; the output is incomplete) */
} csf_expert_matmul_args;

/* One launch.  Errors: CSF_ERR_ARG, CSF_ERR_UNSUPPORTED (K or N off the
 * multiples above or within 512 of 2^31, E > 8192), CSF_ERR_CUDA. */
csf_status csf_expert_matmul(const csf_expert_matmul_args *a, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* CSF_OPS_H */
