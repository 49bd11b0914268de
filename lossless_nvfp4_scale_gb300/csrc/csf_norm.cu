// Residual addition, root-mean-square norm and quantisation in one pass
// (csf_rms_norm): y = h * rsqrt(mean(h^2) + eps) * weight, h = x + residual.
//
// Bound by memory: a row is read once and stays in registers, in chunks of 8
// columns a thread, while its sum of squares is formed and the next row is
// under way; then the chunks are scaled, the block maxima come from shuffles
// between the 16 (128 columns, FP8), 4 (32, MXFP8) or 2 (16, NVFP4) threads of
// a block, and codes and scales leave.  Rows too wide for the registers are
// read twice.  16384 bfloat16 rows of 5120 with a residual to MXFP8: 99 us,
// 5.96 TB/s (0.88 of the measured copy); 127 us with a block a row, whose
// loads wait for its reduction.
#include <algorithm>
#include <atomic>

#include "csf_internal.cuh"
#include "csf_quant.cuh"

namespace csfk {
namespace {

constexpr int kNormMaxThreads = 1024;

// Mean squares from kLeastMean up to infinity are taken as they are: what
// underflows below them does not count.  Smaller rows are taken 2^96 times
// larger (their values are below 2^-38, rows having 2^24 at most), others
// 2^80 times smaller (values below 2^48), so that their squares and sums stay
// in range.  (What loses bits by the latter is below 2^-46 in a row whose mean
// square is above 2^104: below 2^-98 in the result.)
constexpr float kLeastMean = 0x1p-100f, kUp = 0x1p96f, kDown = 0x1p-80f;

// Where the registers are full (rows loaded ahead by a whole block) such rows
// are marked and done when the block's others are: 16384 rows of 5120 to NVFP4
// take 86 us so, 85 without and 97 with a branch for them in the loop.  Else
// they are done at once.  The mark is an NVFP4 row's first scale (UE4M3, a
// byte below 0x80) or an MXFP8 or FP8 row's first code (the conversion's NaN
// is 0x7F).
constexpr uint8_t kAgain = 0xFF;

struct NormParams {
    const void *x, *residual, *weight;
    void *sum;
    int64_t x_stride, residual_stride, sum_stride;   // elements
    uint8_t *codes, *scales;
    int64_t code_stride, scale_stride;
    const float *tensor_scale;
    int64_t rows;
    int32_t cols, chunks;        // chunks: 8-column pieces of the padded row
    float eps, inv_cols;
    int32_t wide_x, wide_residual, wide_sum, wide_weight;   // 16-byte accesses allowed
};

template <typename T> struct Elem;
template <> struct Elem<__nv_bfloat16> {
    static __device__ float to(__nv_bfloat16 v) { return __bfloat162float(v); }
    static __device__ __nv_bfloat16 from(float v) { return __float2bfloat16_rn(v); }
};
template <> struct Elem<__half> {
    static __device__ float to(__half v) { return __half2float(v); }
    static __device__ __half from(float v) { return __float2half_rn(v); }
};
template <> struct Elem<float> {
    static __device__ float to(float v) { return v; }
    static __device__ float from(float v) { return v; }
};

// Columns c .. c+7 of a row, 0 past its end.
template <typename T>
__device__ __forceinline__ void load8(float (&v)[8], const T *row, int c, int cols, bool wide) {
    if (wide && c + 8 <= cols) {
        union { uint4 q[sizeof(T) / 2]; T e[8]; } u;
#pragma unroll
        for (int i = 0; i < (int)(sizeof(T) / 2); ++i) u.q[i] = reinterpret_cast<const uint4 *>(row + c)[i];
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = Elem<T>::to(u.e[i]);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = c + i < cols ? Elem<T>::to(row[c + i]) : 0.f;
    }
}

template <typename T>
__device__ __forceinline__ void store8(const float (&v)[8], T *row, int c, int cols, bool wide) {
    if (wide && c + 8 <= cols) {
        union { uint4 q[sizeof(T) / 2]; T e[8]; } u;
#pragma unroll
        for (int i = 0; i < 8; ++i) u.e[i] = Elem<T>::from(v[i]);
#pragma unroll
        for (int i = 0; i < (int)(sizeof(T) / 2); ++i) reinterpret_cast<uint4 *>(row + c)[i] = u.q[i];
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (c + i < cols) row[c + i] = Elem<T>::from(v[i]);
    }
}

// h of one chunk: x + residual.
template <typename T>
__device__ __forceinline__ void load_h(float (&h)[8], const NormParams &p, int64_t row, int c) {
    load8(h, static_cast<const T *>(p.x) + row * p.x_stride, c, p.cols, p.wide_x);
    if (p.residual) {
        float r[8];
        load8(r, static_cast<const T *>(p.residual) + row * p.residual_stride, c, p.cols, p.wide_residual);
#pragma unroll
        for (int i = 0; i < 8; ++i) h[i] += r[i];
    }
}

// 8 elements as stored.
template <typename T>
struct Raw {
    union { uint4 q[sizeof(T) / 2]; T e[8]; };
};

template <typename T>
__device__ __forceinline__ void load_raw(Raw<T> &r, const T *at) {
#pragma unroll
    for (int i = 0; i < (int)(sizeof(T) / 2); ++i) r.q[i] = reinterpret_cast<const uint4 *>(at)[i];
}

// Threads of a block that loads ahead: what it holds of 32-bit rows takes
// more than the 64 registers that 1024 threads leave.
template <typename T>
__host__ __device__ constexpr int max_ahead() {
    return sizeof(T) == 4 ? 512 : kNormMaxThreads;
}

// A row's sum over its block or warp; `part` holds the warps' sums.
template <bool WARP>
__device__ __forceinline__ float add_up(float sum, float (&part)[32]) {
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, d);
    if constexpr (!WARP) {
        const int lane = threadIdx.x & 31;
        if (lane == 0) part[threadIdx.x >> 5] = sum;
        __syncthreads();
        sum = lane < (int)(blockDim.x >> 5) ? part[lane] : 0.f;
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, d);
    }
    return sum;
}

// Whether a mean square can be taken as it is.
__device__ __forceinline__ bool in_range(float mean) { return mean >= kLeastMean && mean < __int_as_float(0x7F800000); }

// Mean square (plus eps) of a row that is read twice, of h times k.
template <typename T, bool WARP>
__device__ __forceinline__ float mean_of_row(const NormParams &p, int64_t row, float k, int tid, int threads, float (&part)[32]) {
    float sum = 0.f;
    for (int c = tid; c < p.chunks; c += threads) {
        float h[8];
        load_h<T>(h, p, row, c * 8);
#pragma unroll
        for (int i = 0; i < 8; ++i) sum = fmaf(h[i] * k, h[i] * k, sum);
    }
    return add_up<WARP>(sum, part) * p.inv_cols + p.eps * k * k;
}

// A row that is read twice, its values any finite numbers.  (Rows of 20000
// take 1 to 4% longer with the factor k.)
template <typename T, int KIND, bool WARP>
__device__ __forceinline__ void whole_row(const NormParams &p, int64_t row, int tid, int threads, float g, float (&part)[3][32]) {
    float k = 1.f, mean = mean_of_row<T, WARP>(p, row, k, tid, threads, part[0]);
    if (!in_range(mean)) {
        k = mean < 1.f ? kUp : kDown;
        mean = mean_of_row<T, WARP>(p, row, k, tid, threads, part[1]);
    }
    const float r = rsqrtf(mean);
    uint8_t *codes = p.codes + row * p.code_stride, *scales = p.scales + row * p.scale_stride;
    for (int c0 = 0; c0 < p.chunks; c0 += threads) {
        const int c = c0 + tid;
        float h[8], w[8];
        load_h<T>(h, p, row, c * 8);
        if (p.sum) store8(h, static_cast<T *>(p.sum) + row * p.sum_stride, c * 8, p.cols, p.wide_sum);
        load8(w, static_cast<const T *>(p.weight), c * 8, p.cols, p.wide_weight);
#pragma unroll
        for (int i = 0; i < 8; ++i) h[i] = h[i] * k * r * w[i];
        quant::quantize8<KIND>(h, codes, scales, c, c < p.chunks, g);
    }
    const int blocks = quant::scale_bytes<KIND>(p.chunks);
    if (tid < ((blocks + 15) & ~15) - blocks) scales[blocks + tid] = 0;
    if constexpr (!WARP) __syncthreads();      // part[0] is read
}

// The same as a function of its own: inlined, it cost two-chunk kernels spilled
// registers (91 us for the NVFP4 rows above).
template <typename T, int KIND, bool WARP>
__device__ __noinline__ void whole_row_apart(const NormParams &p, int64_t row, int tid, int threads, float g, float (&part)[3][32]) {
    whole_row<T, KIND, WARP>(p, row, tid, threads, g, part);
}

// One row at a time per block of blockDim.x threads (WARP: per warp), rows a
// grid apart.
//   CHUNKS > 0  a row stays in registers, that many chunks a thread; 0: it is
//               read twice.
//   AHEAD       the next row is loaded before this one's sum is formed, and
//               16-bit weights stay in registers (16-byte loads, whole chunks)
template <typename T, int KIND, int CHUNKS, bool WARP, bool AHEAD>
__global__ void __launch_bounds__(WARP ? 256 : AHEAD ? max_ahead<T>() : kNormMaxThreads)
rms_norm_kernel(const __grid_constant__ NormParams p) {
    __shared__ float part[3][32];      // two rows' in turn: one's are read while the next one's are written; a row done again
    __shared__ uint32_t again;         // a row is marked
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int tid = WARP ? lane : threadIdx.x, threads = WARP ? 32 : blockDim.x;
    const int per_block = WARP ? blockDim.x >> 5 : 1;
    const int64_t step = (int64_t)gridDim.x * per_block;
    const float g = KIND == CSF_ROWS_NVFP4 && p.tensor_scale ? *p.tensor_scale : 1.f;
    int64_t row = (int64_t)blockIdx.x * per_block + (WARP ? warp : 0);
    if constexpr (CHUNKS == 0) {
        for (; row < p.rows; row += step) whole_row<T, KIND, WARP>(p, row, tid, threads, g, part);
    } else {
        constexpr bool kMark = AHEAD && !WARP && (CHUNKS == 2 || sizeof(T) == 2);
        const T *weight = static_cast<const T *>(p.weight);
        const int blocks = quant::scale_bytes<KIND>(p.chunks);
        constexpr bool kHoldWeight = AHEAD && sizeof(T) == 2;      // 32-bit ones would not fit the registers
        Raw<T> xr[CHUNKS], rr[CHUNKS], wr[CHUNKS];
        auto load_ahead = [&](int64_t row) {
#pragma unroll
            for (int j = 0; j < CHUNKS; ++j) {
                const int c = (tid + j * threads) * 8;
                if (c >= p.cols) continue;
                load_raw(xr[j], static_cast<const T *>(p.x) + row * p.x_stride + c);
                if (p.residual) load_raw(rr[j], static_cast<const T *>(p.residual) + row * p.residual_stride + c);
            }
        };
        if constexpr (AHEAD) {
#pragma unroll
            for (int j = 0; j < CHUNKS; ++j) {
#pragma unroll
                for (int i = 0; i < (int)(sizeof(T) / 2); ++i) xr[j].q[i] = rr[j].q[i] = wr[j].q[i] = make_uint4(0, 0, 0, 0);
                const int c = (tid + j * threads) * 8;
                if (kHoldWeight && c < p.cols) load_raw(wr[j], weight + c);
            }
            if (row < p.rows) load_ahead(row);
        }
        if (kMark && threadIdx.x == 0) again = 0;      // that thread sets it, too
        for (int set = 0; row < p.rows; row += step, set ^= 1) {
            float h[CHUNKS][8];
            float sum = 0.f;
            if constexpr (AHEAD) {
#pragma unroll
                for (int j = 0; j < CHUNKS; ++j) {
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        h[j][i] = Elem<T>::to(xr[j].e[i]);
                        if (p.residual) h[j][i] += Elem<T>::to(rr[j].e[i]);
                    }
                }
                if (row + step < p.rows) load_ahead(row + step);
            } else {
#pragma unroll
                for (int j = 0; j < CHUNKS; ++j) load_h<T>(h[j], p, row, (tid + j * threads) * 8);
            }
#pragma unroll
            for (int j = 0; j < CHUNKS; ++j) {
#pragma unroll
                for (int i = 0; i < 8; ++i) sum = fmaf(h[j][i], h[j][i], sum);
            }
            auto store_sum = [&](int j) {
                store8(h[j], static_cast<T *>(p.sum) + row * p.sum_stride, (tid + j * threads) * 8, p.cols, p.wide_sum);
            };
            if (!kMark && p.sum) {
#pragma unroll
                for (int j = 0; j < CHUNKS; ++j) store_sum(j);
            }
            float mean = add_up<WARP>(sum, part[set]) * p.inv_cols + p.eps;
            const bool keep = in_range(mean);
            if (!kMark && !keep) {      // alike in every thread of the row
                const float k = mean < 1.f ? kUp : kDown;
                sum = 0.f;
#pragma unroll
                for (int j = 0; j < CHUNKS; ++j) {
#pragma unroll
                    for (int i = 0; i < 8; ++i) h[j][i] *= k, sum = fmaf(h[j][i], h[j][i], sum);
                }
                mean = add_up<WARP>(sum, part[2]) * p.inv_cols + p.eps * k * k;
            }
            const float r = rsqrtf(mean);
            uint8_t *codes = p.codes + row * p.code_stride, *scales = p.scales + row * p.scale_stride;
#pragma unroll
            for (int j = 0; j < CHUNKS; ++j) {
                const int c = tid + j * threads;
                // only now: a row that is not kept is read again, and the sum may go where it lies
                if (kMark && p.sum && keep) store_sum(j);
                float w[8];
                if constexpr (kHoldWeight) {
#pragma unroll
                    for (int i = 0; i < 8; ++i) w[i] = Elem<T>::to(wr[j].e[i]);
                } else {
                    load8(w, weight, c * 8, p.cols, p.wide_weight);
                }
#pragma unroll
                for (int i = 0; i < 8; ++i) h[j][i] = h[j][i] * r * w[i];
                quant::quantize8<KIND>(h[j], codes, scales, c, c < p.chunks, g);
            }
            if (kMark && !keep && tid == 0) {
                *(KIND == CSF_ROWS_NVFP4 ? scales : codes) = kAgain;
                again = 1;
            }
            if (tid < ((blocks + 15) & ~15) - blocks) scales[blocks + tid] = 0;
        }
        if constexpr (!kMark) return;
        __syncthreads();      // the marks are written
        if (!again) return;
        // opaque copies: nothing of this is to be held in registers before
        int tid1 = tid, threads1 = threads;
        float g1 = g;
        asm volatile("" : "+r"(tid1), "+r"(threads1), "+f"(g1)::"memory");
        for (row = blockIdx.x; row < p.rows; row += step) {
            const uint8_t *mark = KIND == CSF_ROWS_NVFP4 ? p.scales + row * p.scale_stride : p.codes + row * p.code_stride;
            if (*const_cast<const volatile uint8_t *>(mark) != kAgain) continue;
            if constexpr (CHUNKS == 1) whole_row<T, KIND, WARP>(p, row, tid1, threads1, g1, part);
            else whole_row_apart<T, KIND, WARP>(p, row, tid1, threads1, g1, part);
        }
    }
}

template <typename T, int KIND, int CHUNKS, bool WARP>
cudaError_t launch_shape(const NormParams &p, int threads, bool ahead, cudaStream_t s) {
    const int64_t units = WARP ? (p.rows + threads / 32 - 1) / (threads / 32) : p.rows;
    if constexpr (CHUNKS > 0) {
        if (ahead && threads <= max_ahead<T>()) {
            // enough blocks to fill the SMs; each then takes rows in turn
            auto k = rms_norm_kernel<T, KIND, CHUNKS, WARP, true>;
            static std::atomic<int> per_sm[kNormMaxThreads / 32 + 1];      // by warps; alike on every device of this architecture
            int n = per_sm[threads / 32];
            if (n == 0) {
                int got = 0;
                const cudaError_t err = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&got, k, threads, 0);
                if (err != cudaSuccess) return err;
                per_sm[threads / 32] = n = got > 0 ? got : 1;
            }
            const int64_t grid = std::min<int64_t>(units, (int64_t)n * sm_count());
            if (grid < 1) return cudaErrorUnknown;
            k<<<(unsigned)grid, threads, 0, s>>>(p);
            return cudaGetLastError();
        }
    }
    rms_norm_kernel<T, KIND, CHUNKS, WARP, false><<<(unsigned)units, threads, 0, s>>>(p);
    return cudaGetLastError();
}

template <typename T, int KIND>
cudaError_t launch_norm(const NormParams &p, cudaStream_t s) {
    const bool ahead = p.wide_x && p.wide_residual && p.wide_weight && p.cols % 8 == 0;
    if (p.chunks <= 32) return launch_shape<T, KIND, 1, true>(p, 256, ahead, s);
    const int one = (p.chunks + 31) & ~31, two = ((p.chunks + 1) / 2 + 31) & ~31;
    if (one <= 256) return launch_shape<T, KIND, 1, false>(p, one, ahead, s);
    if (two <= kNormMaxThreads) return launch_shape<T, KIND, 2, false>(p, two, ahead, s);
    return launch_shape<T, KIND, 0, false>(p, kNormMaxThreads, false, s);
}

template <typename T>
cudaError_t launch_norm_kind(int kind, const NormParams &p, cudaStream_t s) {
    return kind == CSF_ROWS_NVFP4  ? launch_norm<T, CSF_ROWS_NVFP4>(p, s)
           : kind == CSF_ROWS_FP8 ? launch_norm<T, CSF_ROWS_FP8>(p, s)
                                  : launch_norm<T, CSF_ROWS_MXFP8>(p, s);
}

bool wide(const void *p, int64_t stride, int dtype) {
    return aligned_to(p, 16) && (stride * (int64_t)dtype_bytes(dtype)) % 16 == 0;
}

}  // namespace
}  // namespace csfk

using namespace csfk;

extern "C" csf_status csf_rms_norm(const csf_rms_norm_args *a, void *stream) {
    if (!a || !dtype_known(a->dtype) || !rows_valid(a->out, true)) return CSF_ERR_ARG;
    if (a->out.rows == 0) return CSF_OK;
    const int64_t cols = a->out.cols;
    if (!a->x || !a->weight || a->x_stride < cols) return CSF_ERR_ARG;
    if ((a->residual && a->residual_stride < cols) || (a->sum_out && a->sum_stride < cols)) return CSF_ERR_ARG;
    const uintptr_t e = dtype_bytes(a->dtype);
    if (!aligned_to(a->x, e) || !aligned_to(a->weight, e) || !aligned_to(a->residual, e) || !aligned_to(a->sum_out, e)) return CSF_ERR_ARG;
    if (!aligned_to(a->out.tensor_scale, 4)) return CSF_ERR_ARG;
    if (a->out.rows >= (1ll << 31) || cols > (1 << 24)) return CSF_ERR_UNSUPPORTED;
    NormParams p;
    p.x = a->x;
    p.residual = a->residual;
    p.weight = a->weight;
    p.sum = a->sum_out;
    p.x_stride = a->x_stride;
    p.residual_stride = a->residual_stride;
    p.sum_stride = a->sum_stride;
    p.codes = a->out.codes;
    p.scales = a->out.scales;
    p.code_stride = a->out.code_stride;
    p.scale_stride = a->out.scale_stride;
    p.tensor_scale = a->out.tensor_scale;
    p.rows = a->out.rows;
    p.cols = (int32_t)cols;
    p.chunks = (int32_t)(round_up(cols, 32) / 8);
    p.eps = a->eps;
    p.inv_cols = 1.f / (float)cols;
    p.wide_x = wide(a->x, a->x_stride, a->dtype);
    p.wide_residual = wide(a->residual, a->residual_stride, a->dtype);
    p.wide_sum = wide(a->sum_out, a->sum_stride, a->dtype);
    p.wide_weight = aligned_to(a->weight, 16);
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const cudaError_t err = a->dtype == CSF_BF16  ? launch_norm_kind<__nv_bfloat16>(a->out.kind, p, s)
                            : a->dtype == CSF_F16 ? launch_norm_kind<__half>(a->out.kind, p, s)
                                                  : launch_norm_kind<float>(a->out.kind, p, s);
    if (err == cudaSuccess) return CSF_OK;
    cudaGetLastError();      // not left to the caller's next check
    return CSF_ERR_CUDA;
}
