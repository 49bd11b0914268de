// The gradient of the router's weights for its logits (csf_route_grad).
//
// A token is a warp's or half a warp's: lane j < k has choice j, and each lane
// pieces of 8 neighbouring experts, whose logits (for the softmax over all
// experts) stay in registers.  The row is written once without the choices'
// own parts, and then the choices' places once more: k of them, still in L2.
// 32768 bfloat16 tokens of 384 experts, k = 8: 13.9 us, bound by instructions,
// 220 a token (a warp a token took 322 and 19.8 us; memory alone 7.9).
#include <algorithm>

#include "csf_elem.cuh"
#include "csf_internal.cuh"
#include "csf_layer.h"

namespace csfk {
namespace {

constexpr int kGradThreads = 256;
constexpr int kGradBlocks = 8;       // blocks an SM, which take tokens in turn

struct RouteGradParams {
    const char *logits;
    char *out;
    int64_t logits_stride, out_stride;   // bytes
    const int32_t *ids;
    const float *weights, *dweights;
    int32_t tokens, experts, k;
    int32_t wide_logits, wide_out;
};

__device__ __forceinline__ float at(const char *row, int e, int dtype) {
    if (dtype == CSF_F32) return reinterpret_cast<const float *>(row)[e];
    const uint16_t v = reinterpret_cast<const uint16_t *>(row)[e];
    return dtype == CSF_BF16 ? __uint_as_float((uint32_t)v << 16) : __half2float(__ushort_as_half(v));
}

// Over the lanes of a token.
template <int LANES>
__device__ __forceinline__ float lanes_sum(float v) {
#pragma unroll
    for (int s = LANES / 2; s > 0; s >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, s);
    return v;
}

template <int LANES>
__device__ __forceinline__ float lanes_max(float v) {
#pragma unroll
    for (int s = LANES / 2; s > 0; s >>= 1) v = fmaxf(v, __shfl_xor_sync(0xFFFFFFFFu, v, s));
    return v;
}

// exp of a difference from the row's largest.  For 16-bit results, whose
// rounding is 2^-12 at least, within |x| 2^-23 + 2^-22 of itself (and 0 below
// 2^-126).
template <int DTYPE>
__device__ __forceinline__ float exp_below(float x) {
    if constexpr (DTYPE == CSF_F32) return expf(x);
    float e;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(x * 1.4426950408889634f));
    return e;
}

// LANES of a token, 16 or 32.  CHUNKS: pieces of 8 experts a lane; 0:
// renormalised weights, whose gradient is 0 but for the choices.  WIDE: rows
// in whole 16-byte pieces, read and written.
template <int DTYPE, int LANES, int CHUNKS, bool WIDE>
__global__ void __launch_bounds__(kGradThreads) route_grad_kernel(const __grid_constant__ RouteGradParams p) {
    const int lane = threadIdx.x & (LANES - 1);
    constexpr bool kAll = CHUNKS > 0;
    // A token's choices and logits are under way while the one before is done.
    struct Token {
        int id;
        float w, d;
        elem::Raw r[kAll ? CHUNKS : 1];
    };
    auto load = [&](Token &n, int64_t t) {
        n.id = -1;
        n.w = n.d = 0.f;
        if constexpr (kAll) {
            // past the row's end: -infinity
            constexpr uint32_t kOff = DTYPE == CSF_F32 ? 0xFF800000u : DTYPE == CSF_BF16 ? 0xFF80FF80u : 0xFC00FC00u;
#pragma unroll
            for (int i = 0; i < CHUNKS; ++i) n.r[i].a = n.r[i].b = make_uint4(kOff, kOff, kOff, kOff);
        }
        if (t >= p.tokens) return;
        const char *row = p.logits + t * p.logits_stride;
        if constexpr (kAll) {
#pragma unroll
            for (int i = 0; i < CHUNKS; ++i) {
                if constexpr (WIDE) {
                    const uint4 *from = reinterpret_cast<const uint4 *>(row) + (lane + LANES * i) * (DTYPE == CSF_F32 ? 2 : 1);
                    if ((lane + LANES * i) * 8 < p.experts) {
                        n.r[i].a = __ldg(from);
                        if (DTYPE == CSF_F32) n.r[i].b = __ldg(from + 1);
                    }
                } else {
                    n.r[i] = elem::load(row, (lane + LANES * i) * 8, p.experts, DTYPE, p.wide_logits);
                }
            }
        }
        if (lane < p.k) {
            n.id = __ldg(p.ids + t * p.k + lane);
            n.w = __ldg(p.weights + t * p.k + lane), n.d = __ldg(p.dweights + t * p.k + lane);
        }
    };
    constexpr int kPerBlock = kGradThreads / LANES;
    const int64_t step = (int64_t)gridDim.x * kPerBlock;
    const int nth = threadIdx.x / LANES, first = (threadIdx.x >> 5) * (32 / LANES);      // of the block's, and of the warp's
    Token next;
    load(next, (int64_t)blockIdx.x * kPerBlock + nth);
    for (int64_t t0 = (int64_t)blockIdx.x * kPerBlock; t0 + first < p.tokens; t0 += step) {
        const int64_t t = t0 + nth;
        const bool live = t < p.tokens;
        Token n = next;
        load(next, t + step);
        if (n.id < 0 || n.id >= p.experts) n.id = -1, n.w = 0.f, n.d = 0.f;
        // (again, from a cache: where it lies in the registers is not known when this is compiled)
        const float mine = kAll && n.id >= 0 ? at(p.logits + t * p.logits_stride, n.id, DTYPE) : 0.f;
        char *out = p.out + t * p.out_stride;
        const float dot = lanes_sum<LANES>(n.w * n.d);
        float own = kAll ? n.w * n.d : n.w * (n.d - dot);
        // a choice made twice has both parts
        bool again = false;
        if (p.k <= 8) {
#pragma unroll
            for (int j = 1; j < 8; ++j) again |= __shfl_down_sync(0xFFFFFFFFu, n.id, j, 8) == n.id && (lane & 7) + j < 8;
        } else {
            for (int j = 0; j < p.k; ++j) again |= __shfl_sync(0xFFFFFFFFu, n.id, j, LANES) == n.id && j != lane;
        }
        if (__any_sync(0xFFFFFFFFu, again && n.id >= 0)) {
            float both = 0.f;
            for (int j = 0; j < p.k; ++j) {
                const float other = __shfl_sync(0xFFFFFFFFu, own, j, LANES);
                if (__shfl_sync(0xFFFFFFFFu, n.id, j, LANES) == n.id) both += other;
            }
            own = both;
        }
        if constexpr (kAll) {
            float most = __int_as_float(0xFF800000), sum = 0.f;
            float v[CHUNKS][8];
#pragma unroll
            for (int i = 0; i < CHUNKS; ++i) {
                elem::to_floats(v[i], n.r[i], DTYPE);
#pragma unroll
                for (int q = 0; q < 8; ++q) {
                    if (!WIDE && (lane + LANES * i) * 8 + q >= p.experts) v[i][q] = __int_as_float(0xFF800000);
                    most = fmaxf(most, v[i][q]);
                }
            }
            most = lanes_max<LANES>(most);
            const bool none = most == __int_as_float(0xFF800000);      // every expert is off: their exponentials are 0
            const float zero = none ? 0.f : most;
#pragma unroll
            for (int i = 0; i < CHUNKS; ++i)
#pragma unroll
                for (int q = 0; q < 8; ++q) sum += v[i][q] = exp_below<DTYPE>(v[i][q] - zero);
            sum = lanes_sum<LANES>(sum);
            const float rate = none ? 0.f : -dot / sum;
            own += exp_below<DTYPE>(mine - zero) * rate;
            __syncwarp();      // every lane has read: the row may be written where it lay
#pragma unroll
            for (int i = 0; i < CHUNKS; ++i) {
                const int c = (lane + LANES * i) * 8;
                if (!live || c >= p.experts) break;
#pragma unroll
                for (int q = 0; q < 8; ++q) v[i][q] *= rate;
                elem::store(out, c, p.experts, elem::from_floats(v[i], DTYPE), DTYPE, WIDE || p.wide_out);
            }
        } else {
            const elem::Raw zeros = {make_uint4(0, 0, 0, 0), make_uint4(0, 0, 0, 0)};
            for (int c = lane * 8; live && c < p.experts; c += 8 * LANES) elem::store(out, c, p.experts, zeros, DTYPE, p.wide_out);
        }
        __syncwarp();      // the row is written: the choices' places once more
        if (n.id >= 0) {
            if (DTYPE == CSF_F32) reinterpret_cast<float *>(out)[n.id] = own;
            else if (DTYPE == CSF_BF16) reinterpret_cast<__nv_bfloat16 *>(out)[n.id] = __float2bfloat16_rn(own);
            else reinterpret_cast<__half *>(out)[n.id] = __float2half_rn(own);
        }
    }
}

template <int DTYPE, int LANES, int CHUNKS>
void launch_chunks(const RouteGradParams &p, cudaStream_t s) {
    constexpr int kPerBlock = kGradThreads / LANES;
    const int64_t blocks = ((int64_t)p.tokens + kPerBlock - 1) / kPerBlock;
    const unsigned grid = (unsigned)std::min<int64_t>(blocks, kGradBlocks * (int64_t)std::max(sm_count(), 1));
    if (CHUNKS > 0 && p.wide_logits && p.wide_out && p.experts % 8 == 0)
        route_grad_kernel<DTYPE, LANES, CHUNKS, true><<<grid, kGradThreads, 0, s>>>(p);
    else route_grad_kernel<DTYPE, LANES, CHUNKS, false><<<grid, kGradThreads, 0, s>>>(p);
}

template <int DTYPE>
void launch(const RouteGradParams &p, bool renormalize, cudaStream_t s) {
    if (renormalize) return launch_chunks<DTYPE, 32, 0>(p, s);
    // Two tokens a warp: what a warp does once a token it then does for two.
    // 32768 tokens of 256 / 384 / 512 experts, 16 bits: 10.3 / 14.0 / 16.5 us,
    // a warp a token 13.3 / 17.0 / 17.7; 32 bits, whose four pieces a lane want too
    // many registers: 14.8 / 20.8 / 27.2 and 16.6 / 22.0 / 26.1.  64 tokens of 512:
    // 2.6 (3.6) us, a warp a token 2.3 (2.8).
    if (p.k <= 16 && p.experts <= 384) {
        switch ((p.experts + 127) / 128) {
            case 1: return launch_chunks<DTYPE, 16, 1>(p, s);
            case 2: return launch_chunks<DTYPE, 16, 2>(p, s);
            default: return launch_chunks<DTYPE, 16, 3>(p, s);
        }
    }
    switch ((p.experts + 255) / 256) {
        case 1: return launch_chunks<DTYPE, 32, 1>(p, s);
        case 2: return launch_chunks<DTYPE, 32, 2>(p, s);
        case 3: return launch_chunks<DTYPE, 32, 3>(p, s);
        default: return launch_chunks<DTYPE, 32, 4>(p, s);
    }
}

}  // namespace
}  // namespace csfk

using namespace csfk;

extern "C" csf_status csf_route_grad(const csf_route_grad_args *a, void *stream) {
    if (!a || !dtype_known(a->dtype) || a->tokens < 0 || a->experts < 1 || a->k < 1 || a->k > a->experts) return CSF_ERR_ARG;
    if (a->experts > 1024 || a->k > 32) return CSF_ERR_UNSUPPORTED;
    if (a->tokens == 0) return CSF_OK;
    const uintptr_t e = dtype_bytes(a->dtype);
    if (!a->dlogits || a->dlogits_stride < a->experts || !aligned_to(a->dlogits, e)) return CSF_ERR_ARG;
    if (!a->renormalize && (!a->logits || a->logits_stride < a->experts || !aligned_to(a->logits, e))) return CSF_ERR_ARG;
    if (!a->ids || !a->weights || !a->dweights || !aligned_to(a->ids, 4) || !aligned_to(a->weights, 4) || !aligned_to(a->dweights, 4))
        return CSF_ERR_ARG;
    RouteGradParams p;
    p.logits = static_cast<const char *>(a->logits);
    p.out = static_cast<char *>(a->dlogits);
    p.logits_stride = a->logits_stride * (int64_t)e;
    p.out_stride = a->dlogits_stride * (int64_t)e;
    p.ids = a->ids;
    p.weights = a->weights;
    p.dweights = a->dweights;
    p.tokens = a->tokens;
    p.experts = a->experts;
    p.k = a->k;
    p.wide_logits = wide_rows(a->logits, a->logits_stride, a->dtype);
    p.wide_out = wide_rows(a->dlogits, a->dlogits_stride, a->dtype);
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (a->dtype == CSF_BF16) launch<CSF_BF16>(p, a->renormalize, s);
    else if (a->dtype == CSF_F16) launch<CSF_F16>(p, a->renormalize, s);
    else launch<CSF_F32>(p, a->renormalize, s);
    return cudaGetLastError() == cudaSuccess ? CSF_OK : CSF_ERR_CUDA;
}
