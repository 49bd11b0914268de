/*
 * csf_layer.h -- C ABI of the operators that carry an expert layer's tokens
 * and its 8-bit products, in libcsf.so beside those of csf_ops.h:
 *
 *   csf_fp8_matmul    product of FP8 rows with E4M3 weights that have a scale
 *                     for each block of 128 x 128: dense layers and experts
 *                     beside the FP4 ones, and the gradient of their input
 *   csf_dispatch      rows to their experts' slots, as they are or quantised;
 *                     without slots, the quantiser of a product's input
 *   csf_combine       a token's rows back from its slots, with the router's
 *                     weights; without weights, the gradient of csf_dispatch
 *   csf_combine_grad  the gradient of csf_combine: of the slots' rows and of
 *                     the weights
 *   csf_route_grad    the gradient of csf_route: from the weights' to the
 *                     logits'
 *
 * The conventions of csf.h and csf_ops.h hold: device pointers owned by the
 * caller, calls asynchronous on `stream`, no allocation, no host
 * synchronisation, argument and launch errors as a csf_status, data errors as
 * CSF_DEV_ERR_* bits OR-ed into the optional device word `error_word`.
 * Arguments are checked on the host before any CUDA call; a pointer off the
 * alignment of its element is CSF_ERR_ARG.  Results do not depend on the
 * order in which a launch's blocks run.
 */
#ifndef CSF_LAYER_H
#define CSF_LAYER_H

#include "csf_ops.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * For slot s of expert e (expert_start[e] <= s < expert_start[e+1]) and x row
 * r = rows[s] (or s), with xs and ws the block scales, b the blocks of 128 of
 * the summed index:
 *   p[f] = sum_b xs[r][b] ws[e][f / 128][b] sum_{k in b} x[r][k] w[e][f][k] + bias[e][f]
 *   transposed:
 *   p[f] = sum_b xs[r][b] ws[e][b][f / 128] sum_{n in b} x[r][n] w[e][n][f] + bias[e][f]
 *   plain:  y[f] = act(p[f])
 *   gated:  y[f] = act(p[f]) * p[N/2 + f], 0 <= f < N/2; not with transposed
 *   out[s][f] = y[f] * row_scale[s] + residual[s][f]
 * Sums in 32 bits, within (depth / 32 + 4) 2^-23 of sum |x w| of the values
 * where xs ws, which is formed first, is a normal float32 number or 0.
 * SiLU and GELU are as csf_expert_matmul's.  Slots at or past expert_start[E]
 * are not written; with an expert_start that is out of order or range, none
 * is.  A row index out of range stands for row 0.
 */
typedef struct {
    csf_rows x;              /* CSF_ROWS_FP8, cols = the summed length: K, or N transposed */
    const int32_t *rows;     /* optional [slots]: the x row of each slot */
    int64_t slots;           /* >= 0, < 2^31; rows NULL: slots <= x.rows */
    int32_t experts;         /* E, 1 .. 8192 */
    int32_t n, k;            /* w's rows and columns per expert; k a multiple of 16, transposed: n too; gated: n of 256 */
    int32_t transposed;
    const uint8_t *w;        /* [E][N][K] E4M3, 16-byte aligned */
    const float *w_scales;   /* [E][ceil(N / 128)][ceil(K / 128)] */
    const void *expert_start;/* [E+1]; NULL: E must be 1 and owns every slot */
    int32_t expert_start_is_int64;
    int32_t bias_dtype;
    const void *bias;        /* optional [E][N] ([E][K] transposed) of bias_dtype */
    int32_t act;             /* csf_act */
    int32_t gated;
    const float *row_scale;  /* optional [slots] */
    const void *residual;    /* optional [slots][F] of residual_dtype */
    int64_t residual_stride; /* elements */
    int32_t residual_dtype;
    int32_t out_dtype;       /* plain output: csf_dtype; read when out != NULL */
    void *out;               /* plain output [slots][F], row stride out_stride elements; or NULL: */
    int64_t out_stride;
    csf_rows out_rows;       /* FP8 rows, cols = F, rows = slots */
    uint32_t *error_word;    /* optional: CSF_DEV_ERR_CORRUPT (a row index or expert_start out of range),
                                CSF_DEV_ERR_TIMEOUT (a bounded wait gave up; the output is incomplete) */
} csf_fp8_matmul_args;

/* One launch.  Errors: CSF_ERR_ARG, CSF_ERR_UNSUPPORTED (k, n off the
 * multiples above or within 512 of 2^31, E > 8192), CSF_ERR_CUDA. */
csf_status csf_fp8_matmul(const csf_fp8_matmul_args *a, void *stream);

/*
 * out[slots[t][j]] = x[t], rounded to the output's type or quantised as
 * csf_rows says.  Slots of -1 are choices that fell away; others outside
 * [0, out_count) are not written and set CSF_DEV_ERR_CORRUPT.  Output rows
 * that no slot names are left as they were.  Each slot belongs to one choice,
 * as csf_route numbers them: a row that two choices name, of one token or of
 * two, may hold parts of both, and codes of one with scales of the other.
 * Without slots out[t] = x[t].
 */
typedef struct {
    const void *x;           /* [tokens][cols] of dtype, row stride x_stride elements */
    int64_t x_stride;
    int32_t dtype;           /* csf_dtype */
    int32_t tokens;          /* >= 0 */
    int32_t cols;            /* 1 .. 2^24 */
    int32_t k;               /* slots per token, 1 .. 1024; read when slots != NULL */
    const int32_t *slots;    /* optional [tokens][k] */
    int64_t out_count;       /* output rows; without slots: tokens */
    void *out;               /* plain output [out_count][cols], row stride out_stride elements; or NULL: */
    int64_t out_stride;
    int32_t out_dtype;
    csf_rows out_rows;       /* quantised output: kind, cols, rows = out_count */
    uint32_t *error_word;    /* optional */
} csf_dispatch_args;

/* One launch.  Errors: CSF_ERR_ARG, CSF_ERR_UNSUPPORTED (cols, k), CSF_ERR_CUDA. */
csf_status csf_dispatch(const csf_dispatch_args *a, void *stream);

/*
 * out[t] = sum_j weights[t][j] * y[slots[t][j]] + residual[t], summed in 32
 * bits in the order of j, the residual last.  Slots of -1 add nothing,
 * whatever their weight; others outside [0, y_rows) add nothing and set
 * CSF_DEV_ERR_CORRUPT.  Without weights they are 1.  `out` may be `residual`.
 */
typedef struct {
    const void *y;           /* [y_rows][cols] of y_dtype, row stride y_stride elements */
    int64_t y_stride, y_rows;
    int32_t y_dtype;
    int32_t tokens;          /* >= 0 */
    int32_t cols;            /* 1 .. 2^24 */
    int32_t k;               /* 1 .. 1024 */
    const int32_t *slots;    /* [tokens][k] */
    const float *weights;    /* optional [tokens][k] */
    const void *residual;    /* optional [tokens][cols] of residual_dtype */
    int64_t residual_stride;
    int32_t residual_dtype, out_dtype;
    void *out;               /* [tokens][cols] of out_dtype */
    int64_t out_stride;
    uint32_t *error_word;    /* optional */
} csf_combine_args;

/* One launch.  Errors: CSF_ERR_ARG, CSF_ERR_UNSUPPORTED (cols, k), CSF_ERR_CUDA. */
csf_status csf_combine(const csf_combine_args *a, void *stream);

/*
 * The gradient of csf_combine for g = d out:
 *   dy[slots[t][j]]   = weights[t][j] * g[t], rounded or quantised
 *   dweights[t][j]    = sum_c g[t][c] * y[slots[t][j]][c], in 32 bits
 * (that of the residual is g itself).  Either may be left out.  Choices of
 * slot -1 have dweights 0 and write no dy, those out of range likewise and
 * set CSF_DEV_ERR_CORRUPT; rows of dy that no slot names are left as they
 * were.  Each slot belongs to one choice, as csf_route numbers them.
 */
typedef struct {
    const void *g;           /* [tokens][cols] of g_dtype, row stride g_stride elements */
    int64_t g_stride;
    const void *y;           /* [slot_rows][cols] of y_dtype; read for dweights */
    int64_t y_stride;
    int64_t slot_rows;       /* rows of y and dy */
    int32_t g_dtype, y_dtype;
    int32_t tokens;          /* >= 0 */
    int32_t cols;            /* 1 .. 2^24 */
    int32_t k;               /* 1 .. 1024 */
    int32_t dy_dtype;
    const int32_t *slots;    /* [tokens][k] */
    const float *weights;    /* optional [tokens][k]: 1 without */
    void *dy;                /* plain [slot_rows][cols] of dy_dtype; or NULL: */
    int64_t dy_stride;
    csf_rows dy_rows;        /* quantised: kind, cols, rows = slot_rows; codes NULL: no dy */
    float *dweights;         /* optional [tokens][k] */
    uint32_t *error_word;    /* optional */
} csf_combine_grad_args;

/* One launch.  Errors: CSF_ERR_ARG, CSF_ERR_UNSUPPORTED (cols, k), CSF_ERR_CUDA. */
csf_status csf_combine_grad(const csf_combine_grad_args *a, void *stream);

/*
 * The gradient of csf_route's weights w for its logits, with d = dweights:
 *   renormalize: dlogits[ids[j]] = w_j (d_j - sum_i w_i d_i), 0 elsewhere
 *   else:        dlogits[e] = sum_{j: ids[j] = e} w_j d_j - p_e sum_i w_i d_i,
 *                p the softmax over all experts (0 for logits of -inf)
 * in 32 bits.  The choice of experts is taken as fixed.  Ids outside
 * [0, experts) are choices that fell away; a token without any gets zeros.
 */
typedef struct {
    const void *logits;      /* [tokens][experts] of dtype; not read (may be NULL) with renormalize */
    int64_t logits_stride;
    void *dlogits;           /* [tokens][experts] of dtype, row stride dlogits_stride elements; may be logits */
    int64_t dlogits_stride;
    int32_t dtype;           /* csf_dtype of both */
    int32_t tokens;          /* >= 0 */
    int32_t experts;         /* 1 .. 1024 */
    int32_t k;               /* 1 .. min(32, experts) */
    const int32_t *ids;      /* [tokens][k] */
    const float *weights;    /* [tokens][k] */
    const float *dweights;   /* [tokens][k] */
    int32_t renormalize;     /* as the call of csf_route */
} csf_route_grad_args;

/* One launch.  Errors: CSF_ERR_ARG, CSF_ERR_UNSUPPORTED (experts or k beyond the limits), CSF_ERR_CUDA. */
csf_status csf_route_grad(const csf_route_grad_args *a, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* CSF_LAYER_H */
