// Rows to their experts' slots and back (csf_dispatch, csf_combine) and the
// gradient of the way back (csf_combine_grad).
//
// All three are bound by memory, so each goes by tokens: a token's row is read
// once, whether it is written to k slots (and quantised once for them), added
// up from k slots, or both multiplied with k slots' rows and written to k
// others.  A thread has 8 columns at a time, 16 bytes of 16-bit rows (16 on the
// way to slots: 16 bytes of codes); a warp's lanes are neighbours, so that a
// row's pieces are whole lines wherever the row lies.
//
// Measured: 8192 bfloat16 tokens of 2048 to 8 slots each in FP8 29.7 us
// (5.8 TB/s; filling what is written takes no less), 4095 tokens of 5120 added
// up from 8 slots with a residual 68 us (6.2 TB/s, 0.91 of the measured copy),
// the gradient of 3001 of 1600 with 6 choices 23.5 us (5.3 TB/s).  The quantiser
// alone is bound by instructions: 16384 bfloat16 rows of 5120 to FP8 / MXFP8 /
// NVFP4 49 / 45 / 55 us, 43.7 / 36.7 / 49.3 M warp instructions, 72 to 77% of the
// issue slots (an NVFP4 scale, its inverse and its conversion are for 16 columns,
// an FP8 one's for 128).
#include <algorithm>

#include "csf_elem.cuh"
#include "csf_internal.cuh"
#include "csf_layer.h"

namespace csfk {
namespace {

constexpr int kPlain = -1;           // a kernel's output: plain rows, or a csf_rows_kind
constexpr int kMaxSlots = 1024, kMaxCols = 1 << 24;
constexpr int kRowThreads = 256;

// How a block's threads lie over rows: `lanes` a row (a multiple of 16, the
// lanes of the widest scale block, or of 32), `per_block` rows.
struct Span {
    int32_t tokens, cols, chunks;    // chunks: 8-column pieces of the row padded to 32
    int32_t lanes, per_block;
};

// The fewest rounds of up to 256 threads of `width` columns, evenly; short
// rows share a block.
Span span_of(int32_t tokens, int32_t cols, int least_lanes, int width = 8) {
    Span s;
    s.tokens = tokens;
    s.cols = cols;
    s.chunks = (int32_t)(round_up(cols, 32) / 8);
    const int pieces = s.chunks * 8 / width, rounds = (pieces + kRowThreads - 1) / kRowThreads;
    const int each = (pieces + rounds - 1) / rounds;
    s.lanes = (int32_t)round_up(each, each <= least_lanes ? least_lanes : 32);
    s.per_block = kRowThreads / s.lanes;
    return s;
}

unsigned blocks_of(const Span &s) { return (unsigned)(((int64_t)s.tokens + s.per_block - 1) / s.per_block); }

// Blocks of a launch whose rows need nothing of one another's columns: where
// the tokens alone make few, a row's rounds are blocks too (one token of 5120,
// 8 choices: 5.1 us in one block).
dim3 grid_of(const Span &s, int width) {
    const int pieces = s.chunks * 8 / width, rounds = (pieces + s.lanes - 1) / s.lanes;
    const unsigned blocks = blocks_of(s);
    return dim3(blocks, (int)blocks < sm_count() ? (unsigned)std::min(rounds, 64) : 1u);
}

struct DispatchParams {
    Span span;
    const void *x;
    int64_t x_stride;            // elements
    int32_t wide_x, wide_out;
    const int32_t *slots;        // null: row t goes to row t
    int32_t k, out_dtype;
    int64_t out_count;
    char *out;
    int64_t out_stride;          // bytes
    uint8_t *scales;
    int64_t scale_stride;
    const float *tensor_scale;
    uint32_t *err;
};

__device__ __forceinline__ int64_t row_bytes(int64_t row, int64_t stride, int dtype) {
    return row * stride * (dtype == CSF_F32 ? 4 : 2);
}

// DTYPE: csf_dtype of x; KIND: what comes out.
template <int DTYPE, int KIND>
__global__ void __launch_bounds__(kRowThreads) dispatch_kernel(const __grid_constant__ DispatchParams p) {
    const int nth = threadIdx.x / p.span.lanes, tid = threadIdx.x - nth * p.span.lanes;
    const int64_t t = (int64_t)blockIdx.x * p.span.per_block + nth;
    const bool live = t < p.span.tokens;
    const char *x = static_cast<const char *>(p.x) + row_bytes(live ? t : 0, p.x_stride, DTYPE);
    const int32_t *slots = p.slots ? p.slots + t * p.k : nullptr;
    const int k = p.slots ? p.k : 1;
    const float g = KIND == CSF_ROWS_NVFP4 && p.tensor_scale ? *p.tensor_scale : 1.f;
    const int pieces = p.span.chunks >> 1;       // of 16 columns
    bool bad = false;
    for (int c0 = blockIdx.y * p.span.lanes; c0 < pieces; c0 += gridDim.y * p.span.lanes) {
        const int c = c0 + tid;
        elem::Raw r[2];
        quant::Coded q[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) r[h] = elem::load(x, c * 16 + 8 * h, live ? p.span.cols : 0, DTYPE, p.wide_x);
        if constexpr (KIND == kPlain) {
            if (p.out_dtype != DTYPE) {
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    float y[8];
                    elem::to_floats(y, r[h], DTYPE);
                    r[h] = elem::from_floats(y, p.out_dtype);
                }
            }
        } else {
            float y[2][8];
#pragma unroll
            for (int h = 0; h < 2; ++h) elem::to_floats(y[h], r[h], DTYPE);
            const uint32_t m = quant::block_amax16<KIND>(y);
#pragma unroll
            for (int h = 0; h < 2; ++h) q[h] = quant::encode8<KIND>(y[h], m, g);
        }
        if (!live || c * 16 >= (KIND == kPlain ? p.span.cols : p.span.chunks * 8)) continue;
#pragma unroll 8
        for (int j = 0; j < k; ++j) {
            const int64_t s = slots ? __ldg(slots + j) : t;
            if (s < 0 || s >= p.out_count) {
                bad |= s != -1;
                continue;
            }
            char *out = p.out + s * p.out_stride;
            if constexpr (KIND == kPlain) {
#pragma unroll
                for (int h = 0; h < 2; ++h)
                    if (c * 16 + 8 * h < p.span.cols) elem::store(out, c * 16 + 8 * h, p.span.cols, r[h], p.out_dtype, p.wide_out);
            } else {
                uint8_t *scales = p.scales + s * p.scale_stride;
                quant::put16<KIND>(q, reinterpret_cast<uint8_t *>(out), scales, c);
                const int blocks = quant::scale_bytes<KIND>(p.span.chunks);
                for (int i = c; i < ((blocks + 15) & ~15) - blocks; i += pieces) scales[blocks + i] = 0;
            }
        }
    }
    if (bad && p.err) atomicOr(p.err, CSF_DEV_ERR_CORRUPT);
}

struct CombineParams {
    Span span;
    const void *y, *residual;
    void *out;
    int64_t y_stride, y_rows, residual_stride, out_stride;   // elements
    const int32_t *slots;
    const float *weights;
    int32_t k, residual_dtype, out_dtype;
    int32_t wide_y, wide_residual, wide_out;
    uint32_t *err;
};

// A token's choices, 32 at a time, one a lane of each of its warps: their
// rows, their weights, and which of them have a row.
struct Choices {
    int32_t slot;
    float weight;
    uint32_t on;      // lanes with a row

    __device__ __forceinline__ void load(const int32_t *slots, const float *weights, int64_t first, int left, int64_t rows, int lane, bool &bad) {
        const int32_t s = lane < left ? __ldg(slots + first + lane) : -1;
        const bool is = s >= 0 && s < rows;
        bad |= !is && s != -1;
        slot = s;
        weight = is && weights ? __ldg(weights + first + lane) : 1.f;
        on = __ballot_sync(0xFFFFFFFFu, is);
    }
};

// DTYPE: csf_dtype of y.  WIDE: every row of y in whole 16-byte pieces.
template <int DTYPE, bool WIDE>
__global__ void __launch_bounds__(kRowThreads) combine_kernel(const __grid_constant__ CombineParams p) {
    constexpr int kBatch = DTYPE == CSF_F32 ? 4 : 8;      // rows under way at once
    const int lane = threadIdx.x & 31, nth = threadIdx.x / p.span.lanes, tid = threadIdx.x - nth * p.span.lanes;
    const int64_t t = (int64_t)blockIdx.x * p.span.per_block + nth;
    if (t >= p.span.tokens) return;
    bool bad = false;
    Choices ch;
    ch.load(p.slots, p.weights, t * p.k, p.k, p.y_rows, lane, bad);
    for (int c0 = blockIdx.y * p.span.lanes; c0 * 8 < p.span.cols; c0 += gridDim.y * p.span.lanes) {
        const int c = c0 + tid;
        const bool live = c * 8 < p.span.cols;
        elem::Raw res;
        if (p.residual && live)
            res = elem::load(static_cast<const char *>(p.residual) + row_bytes(t, p.residual_stride, p.residual_dtype), c * 8,
                             p.span.cols, p.residual_dtype, p.wide_residual);
        float sum[8] = {};
        for (int j0 = 0; j0 < p.k; j0 += 32) {
            if (p.k > 32) ch.load(p.slots, p.weights, t * p.k + j0, p.k - j0, p.y_rows, lane, bad);
            for (int b = 0; b < min(32, p.k - j0); b += kBatch) {
                elem::Raw r[kBatch];
#pragma unroll
                for (int j = 0; j < kBatch; ++j) {
                    r[j].a = r[j].b = make_uint4(0, 0, 0, 0);
                    if (!(ch.on >> (b + j) & 1)) continue;       // alike in the warp
                    const char *row = static_cast<const char *>(p.y) + row_bytes(__shfl_sync(0xFFFFFFFFu, ch.slot, b + j), p.y_stride, DTYPE);
                    if constexpr (WIDE) {
                        if (live) {
                            const uint4 *at = reinterpret_cast<const uint4 *>(row) + (size_t)c * (DTYPE == CSF_F32 ? 2 : 1);
                            r[j].a = __ldg(at);
                            if (DTYPE == CSF_F32) r[j].b = __ldg(at + 1);
                        }
                    } else {
                        r[j] = elem::load(row, c * 8, p.span.cols, DTYPE, p.wide_y);
                    }
                }
#pragma unroll
                for (int j = 0; j < kBatch; ++j) {
                    if (!(ch.on >> (b + j) & 1)) continue;
                    const float w = __shfl_sync(0xFFFFFFFFu, ch.weight, b + j);
                    float y[8];
                    elem::to_floats(y, r[j], DTYPE);
#pragma unroll
                    for (int i = 0; i < 8; ++i) sum[i] = fmaf(w, y[i], sum[i]);
                }
            }
        }
        if (!live) continue;
        if (p.residual) {
            float y[8];
            elem::to_floats(y, res, p.residual_dtype);
#pragma unroll
            for (int i = 0; i < 8; ++i) sum[i] += y[i];
        }
        elem::store(static_cast<char *>(p.out) + row_bytes(t, p.out_stride, p.out_dtype), c * 8, p.span.cols,
                    elem::from_floats(sum, p.out_dtype), p.out_dtype, p.wide_out);
    }
    if (bad && p.err) atomicOr(p.err, CSF_DEV_ERR_CORRUPT);
}

struct CombineGradParams {
    Span span;
    const void *g, *y;
    int64_t g_stride, y_stride;      // elements
    int64_t slot_rows;
    const int32_t *slots;
    const float *weights;
    float *dweights;
    char *dy;                        // null: none
    int64_t dy_stride;               // bytes
    uint8_t *scales;
    int64_t scale_stride;
    const float *tensor_scale;
    int32_t k, g_dtype, dy_dtype;
    int32_t wide_g, wide_y, wide_dy;
    uint32_t *err;
};

// The products of g with the slots' rows are summed by thread over its
// columns, then over a warp's lanes, then over the row's warps in order.
// DTYPE: csf_dtype of g and y (WIDE: in whole 16-byte pieces) or of y; KIND:
// what dy is.
template <int DTYPE, int KIND, bool WIDE>
__global__ void __launch_bounds__(kRowThreads) combine_grad_kernel(const __grid_constant__ CombineGradParams p) {
    constexpr int kBatch = DTYPE == CSF_F32 ? 4 : 8;      // choices at a time
    __shared__ float part[kRowThreads / 32][kBatch];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int nth = threadIdx.x / p.span.lanes, tid = threadIdx.x - nth * p.span.lanes;
    const int warps = p.span.lanes >> 5;                  // of a row
    const int64_t t = (int64_t)blockIdx.x * p.span.per_block + nth;
    const bool live = t < p.span.tokens;
    const int g_dtype = WIDE ? DTYPE : p.g_dtype;
    const char *g_row = static_cast<const char *>(p.g) + row_bytes(live ? t : 0, p.g_stride, g_dtype);
    const float ts = KIND == CSF_ROWS_NVFP4 && p.tensor_scale ? *p.tensor_scale : 1.f;
    const bool products = p.dweights != nullptr;
    bool bad = false;
    for (int j0 = 0; j0 < p.k; j0 += 32) {
        Choices ch;
        ch.load(p.slots, p.weights, t * p.k + j0, live ? p.k - j0 : 0, p.slot_rows, lane, bad);
        // choices without a row have no product
        if (products && live && tid < 32 && j0 + lane < p.k && !(ch.on >> lane & 1)) p.dweights[t * p.k + j0 + lane] = 0.f;
        for (int b = 0; b < min(32, p.k - j0); b += kBatch) {
            float sum[kBatch] = {};
            for (int c0 = 0; c0 < p.span.chunks; c0 += p.span.lanes) {
                const int c = c0 + tid;
                const bool in = c * 8 < p.span.cols;
                auto fetch = [&](const char *row, int dtype, bool wide) {
                    if constexpr (WIDE) {
                        elem::Raw r;
                        r.a = r.b = make_uint4(0, 0, 0, 0);
                        if (in) {
                            const uint4 *at = reinterpret_cast<const uint4 *>(row) + (size_t)c * (DTYPE == CSF_F32 ? 2 : 1);
                            r.a = __ldg(at);
                            if (DTYPE == CSF_F32) r.b = __ldg(at + 1);
                        }
                        return r;
                    } else {
                        return elem::load(row, c * 8, p.span.cols, dtype, wide);
                    }
                };
                elem::Raw gr = {make_uint4(0, 0, 0, 0), make_uint4(0, 0, 0, 0)}, yr[kBatch];
                if (live) gr = fetch(g_row, g_dtype, p.wide_g);
                if (products) {
#pragma unroll
                    for (int j = 0; j < kBatch; ++j) {
                        yr[j].a = yr[j].b = make_uint4(0, 0, 0, 0);
                        if (ch.on >> (b + j) & 1)       // alike in the warp
                            yr[j] = fetch(static_cast<const char *>(p.y) + row_bytes(__shfl_sync(0xFFFFFFFFu, ch.slot, b + j), p.y_stride, DTYPE), DTYPE, p.wide_y);
                    }
                }
                float g[8];
                elem::to_floats(g, gr, g_dtype);
                uint32_t amax = 0;
                if constexpr (KIND != kPlain) amax = quant::block_amax<KIND>(g);
#pragma unroll
                for (int j = 0; j < kBatch; ++j) {
                    if (!(ch.on >> (b + j) & 1)) continue;
                    float y[8];
                    if (products) {
                        elem::to_floats(y, yr[j], DTYPE);
                        if (in) {
#pragma unroll
                            for (int i = 0; i < 8; ++i) sum[j] = fmaf(g[i], y[i], sum[j]);
                        }
                    }
                    if (!p.dy) continue;
                    const float w = __shfl_sync(0xFFFFFFFFu, ch.weight, b + j);
                    const int64_t slot = __shfl_sync(0xFFFFFFFFu, ch.slot, b + j);
#pragma unroll
                    for (int i = 0; i < 8; ++i) y[i] = w * g[i];
                    char *out = p.dy + slot * p.dy_stride;
                    if constexpr (KIND == kPlain) {
                        if (in) elem::store(out, c * 8, p.span.cols, elem::from_floats(y, p.dy_dtype), p.dy_dtype, p.wide_dy);
                    } else {
                        // the largest of the rounded products is the rounded product of the largest
                        const uint32_t m = __float_as_uint(w * __uint_as_float(amax)) & 0x7FFFFFFFu;
                        uint8_t *scales = p.scales + slot * p.scale_stride;
                        if (c < p.span.chunks) quant::put8<KIND>(quant::encode8<KIND>(y, m, ts), reinterpret_cast<uint8_t *>(out), scales, c);
                        const int blocks = quant::scale_bytes<KIND>(p.span.chunks);
                        if (c < ((blocks + 15) & ~15) - blocks) scales[blocks + c] = 0;
                    }
                }
            }
            if (!products) continue;
#pragma unroll
            for (int j = 0; j < kBatch; ++j) {
#pragma unroll
                for (int d = 16; d > 0; d >>= 1) sum[j] += __shfl_xor_sync(0xFFFFFFFFu, sum[j], d);
                if (warps == 1) {
                    if (lane == 0 && (ch.on >> (b + j) & 1)) p.dweights[t * p.k + j0 + b + j] = sum[j];
                } else if (lane == j) {
                    part[warp][j] = sum[j];
                }
            }
            if (warps > 1) {
                __syncthreads();
                if (tid < kBatch && (ch.on >> (b + tid) & 1)) {
                    float total = 0.f;
                    for (int i = 0; i < warps; ++i) total += part[nth * warps + i][tid];
                    p.dweights[t * p.k + j0 + b + tid] = total;
                }
                __syncthreads();
            }
        }
    }
    if (bad && p.err) atomicOr(p.err, CSF_DEV_ERR_CORRUPT);
}

template <int DTYPE>
void launch_dispatch(const DispatchParams &p, int kind, cudaStream_t s) {
    const dim3 grid = grid_of(p.span, 16);
    const unsigned threads = (unsigned)(p.span.lanes * p.span.per_block);
    switch (kind) {
        case kPlain: dispatch_kernel<DTYPE, kPlain><<<grid, threads, 0, s>>>(p); break;
        case CSF_ROWS_NVFP4: dispatch_kernel<DTYPE, CSF_ROWS_NVFP4><<<grid, threads, 0, s>>>(p); break;
        case CSF_ROWS_MXFP8: dispatch_kernel<DTYPE, CSF_ROWS_MXFP8><<<grid, threads, 0, s>>>(p); break;
        default: dispatch_kernel<DTYPE, CSF_ROWS_FP8><<<grid, threads, 0, s>>>(p); break;
    }
}

template <int DTYPE, bool WIDE>
void launch_combine_grad(const CombineGradParams &p, int kind, cudaStream_t s) {
    const unsigned grid = blocks_of(p.span), threads = (unsigned)(p.span.lanes * p.span.per_block);
    switch (kind) {
        case kPlain: combine_grad_kernel<DTYPE, kPlain, WIDE><<<grid, threads, 0, s>>>(p); break;
        case CSF_ROWS_NVFP4: combine_grad_kernel<DTYPE, CSF_ROWS_NVFP4, WIDE><<<grid, threads, 0, s>>>(p); break;
        case CSF_ROWS_MXFP8: combine_grad_kernel<DTYPE, CSF_ROWS_MXFP8, WIDE><<<grid, threads, 0, s>>>(p); break;
        default: combine_grad_kernel<DTYPE, CSF_ROWS_FP8, WIDE><<<grid, threads, 0, s>>>(p); break;
    }
}

template <int DTYPE>
void launch_combine_grad(const CombineGradParams &p, int kind, cudaStream_t s) {
    const bool wide = p.wide_g && (!p.dweights || p.wide_y) && p.g_dtype == DTYPE && p.span.cols % 8 == 0;
    if (wide) launch_combine_grad<DTYPE, true>(p, kind, s);
    else launch_combine_grad<DTYPE, false>(p, kind, s);
}

template <int DTYPE>
void launch_combine(const CombineParams &p, cudaStream_t s) {
    const dim3 grid = grid_of(p.span, 8);
    const unsigned threads = (unsigned)(p.span.lanes * p.span.per_block);
    if (p.wide_y && p.span.cols % 8 == 0) combine_kernel<DTYPE, true><<<grid, threads, 0, s>>>(p);
    else combine_kernel<DTYPE, false><<<grid, threads, 0, s>>>(p);
}

// A plain matrix that a call needs.
bool matrix_ok(const void *p, int64_t stride, int32_t dtype, int32_t cols) {
    return p && dtype_known(dtype) && stride >= cols && aligned_to(p, dtype_bytes(dtype));
}

csf_status launched() {
    if (cudaGetLastError() == cudaSuccess) return CSF_OK;
    return CSF_ERR_CUDA;
}

}  // namespace
}  // namespace csfk

using namespace csfk;

extern "C" csf_status csf_dispatch(const csf_dispatch_args *a, void *stream) {
    if (!a || a->tokens < 0 || a->cols < 1 || a->out_count < 0 || !dtype_known(a->dtype)) return CSF_ERR_ARG;
    if (a->slots && a->k < 1) return CSF_ERR_ARG;
    if (!a->slots && a->out_count != a->tokens) return CSF_ERR_ARG;
    if (a->cols > kMaxCols || (a->slots && a->k > kMaxSlots)) return CSF_ERR_UNSUPPORTED;
    if (a->tokens == 0) return CSF_OK;
    if (!a->out && (!rows_valid(a->out_rows, true) || a->out_rows.cols != a->cols || a->out_rows.rows != a->out_count ||
                    !aligned_to(a->out_rows.tensor_scale, 4)))
        return CSF_ERR_ARG;
    if (!matrix_ok(a->x, a->x_stride, a->dtype, a->cols) || !aligned_to(a->slots, 4) || !aligned_to(a->error_word, 4)) return CSF_ERR_ARG;
    if (a->out && !matrix_ok(a->out, a->out_stride, a->out_dtype, a->cols)) return CSF_ERR_ARG;
    DispatchParams p = {};
    p.span = span_of(a->tokens, a->cols, 16, 16);
    p.x = a->x;
    p.x_stride = a->x_stride;
    p.wide_x = wide_rows(a->x, a->x_stride, a->dtype);
    p.slots = a->slots;
    p.k = a->k;
    p.out_count = a->out_count;
    p.err = a->error_word;
    int kind = kPlain;
    if (a->out) {
        p.out = static_cast<char *>(a->out);
        p.out_dtype = a->out_dtype;
        p.out_stride = a->out_stride * (int64_t)dtype_bytes(a->out_dtype);
        p.wide_out = wide_rows(a->out, a->out_stride, a->out_dtype);
    } else {
        kind = a->out_rows.kind;
        p.out = reinterpret_cast<char *>(a->out_rows.codes);
        p.out_stride = a->out_rows.code_stride;
        p.scales = a->out_rows.scales;
        p.scale_stride = a->out_rows.scale_stride;
        p.tensor_scale = a->out_rows.tensor_scale;
    }
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (a->dtype == CSF_BF16) launch_dispatch<CSF_BF16>(p, kind, s);
    else if (a->dtype == CSF_F16) launch_dispatch<CSF_F16>(p, kind, s);
    else launch_dispatch<CSF_F32>(p, kind, s);
    return launched();
}

extern "C" csf_status csf_combine(const csf_combine_args *a, void *stream) {
    if (!a || a->tokens < 0 || a->cols < 1 || a->k < 1 || a->y_rows < 0 || !dtype_known(a->y_dtype) || !dtype_known(a->out_dtype)) return CSF_ERR_ARG;
    if (a->cols > kMaxCols || a->k > kMaxSlots) return CSF_ERR_UNSUPPORTED;
    if (a->tokens == 0) return CSF_OK;
    if (a->y_rows > 0 && !matrix_ok(a->y, a->y_stride, a->y_dtype, a->cols)) return CSF_ERR_ARG;
    if (!matrix_ok(a->out, a->out_stride, a->out_dtype, a->cols)) return CSF_ERR_ARG;
    if (a->residual && !matrix_ok(a->residual, a->residual_stride, a->residual_dtype, a->cols)) return CSF_ERR_ARG;
    if (!a->slots || !aligned_to(a->slots, 4) || !aligned_to(a->weights, 4) || !aligned_to(a->error_word, 4)) return CSF_ERR_ARG;
    CombineParams p = {};
    p.span = span_of(a->tokens, a->cols, 32);
    p.y = a->y;
    p.y_stride = a->y_stride;
    p.y_rows = a->y_rows;
    p.wide_y = wide_rows(a->y, a->y_stride, a->y_dtype);
    p.residual = a->residual;
    p.residual_stride = a->residual_stride;
    p.residual_dtype = a->residual_dtype;
    p.wide_residual = wide_rows(a->residual, a->residual_stride, a->residual_dtype);
    p.out = a->out;
    p.out_stride = a->out_stride;
    p.out_dtype = a->out_dtype;
    p.wide_out = wide_rows(a->out, a->out_stride, a->out_dtype);
    p.slots = a->slots;
    p.weights = a->weights;
    p.k = a->k;
    p.err = a->error_word;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (a->y_dtype == CSF_BF16) launch_combine<CSF_BF16>(p, s);
    else if (a->y_dtype == CSF_F16) launch_combine<CSF_F16>(p, s);
    else launch_combine<CSF_F32>(p, s);
    return launched();
}

extern "C" csf_status csf_combine_grad(const csf_combine_grad_args *a, void *stream) {
    if (!a || a->tokens < 0 || a->cols < 1 || a->k < 1 || a->slot_rows < 0 || !dtype_known(a->g_dtype)) return CSF_ERR_ARG;
    if (a->cols > kMaxCols || a->k > kMaxSlots) return CSF_ERR_UNSUPPORTED;
    const bool quantised = !a->dy && a->dy_rows.codes;
    if (quantised && (!rows_valid(a->dy_rows, true) || a->dy_rows.cols != a->cols || a->dy_rows.rows != a->slot_rows ||
                      !aligned_to(a->dy_rows.tensor_scale, 4)))
        return CSF_ERR_ARG;
    if (a->tokens == 0) return CSF_OK;
    if (!matrix_ok(a->g, a->g_stride, a->g_dtype, a->cols)) return CSF_ERR_ARG;
    if (a->dy && !matrix_ok(a->dy, a->dy_stride, a->dy_dtype, a->cols)) return CSF_ERR_ARG;
    if (a->dweights && (!dtype_known(a->y_dtype) || (a->slot_rows > 0 && !matrix_ok(a->y, a->y_stride, a->y_dtype, a->cols)))) return CSF_ERR_ARG;
    if (!a->slots || !aligned_to(a->slots, 4) || !aligned_to(a->weights, 4) || !aligned_to(a->dweights, 4) || !aligned_to(a->error_word, 4))
        return CSF_ERR_ARG;
    if (!a->dy && !quantised && !a->dweights) return CSF_OK;
    CombineGradParams p = {};
    p.span = span_of(a->tokens, a->cols, 32);
    // A warp a token where there are enough of them: nothing waits for another
    // warp's part of the products (3001 tokens of 1600, 6 choices: 26 us, 34 a
    // block a token).
    const int warps = (int)std::max<int64_t>(1, 16ll * sm_count() / a->tokens);
    if (warps * 32 < p.span.lanes) p.span.lanes = warps * 32, p.span.per_block = kRowThreads / p.span.lanes;
    p.g = a->g;
    p.g_stride = a->g_stride;
    p.g_dtype = a->g_dtype;
    p.wide_g = wide_rows(a->g, a->g_stride, a->g_dtype);
    p.dweights = a->dweights;
    int y_dtype = a->g_dtype;        // not read
    if (a->dweights) {
        y_dtype = a->y_dtype;
        p.y = a->y;
        p.y_stride = a->y_stride;
        p.wide_y = wide_rows(a->y, a->y_stride, a->y_dtype);
    }
    p.slot_rows = a->slot_rows;
    p.slots = a->slots;
    p.weights = a->weights;
    p.k = a->k;
    p.err = a->error_word;
    int kind = kPlain;
    if (a->dy) {
        p.dy = static_cast<char *>(a->dy);
        p.dy_dtype = a->dy_dtype;
        p.dy_stride = a->dy_stride * (int64_t)dtype_bytes(a->dy_dtype);
        p.wide_dy = wide_rows(a->dy, a->dy_stride, a->dy_dtype);
    } else if (quantised) {
        kind = a->dy_rows.kind;
        p.dy = reinterpret_cast<char *>(a->dy_rows.codes);
        p.dy_stride = a->dy_rows.code_stride;
        p.scales = a->dy_rows.scales;
        p.scale_stride = a->dy_rows.scale_stride;
        p.tensor_scale = a->dy_rows.tensor_scale;
    }
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (y_dtype == CSF_BF16) launch_combine_grad<CSF_BF16>(p, kind, s);
    else if (y_dtype == CSF_F16) launch_combine_grad<CSF_F16>(p, kind, s);
    else launch_combine_grad<CSF_F32>(p, kind, s);
    return launched();
}
