// The gradient of the router's weights for its logits (csf_route_grad).
//
// A token is a warp's: lane j < k has choice j, and each lane up to 4 times 8
// neighbouring experts, whose logits (for the softmax over all experts) stay
// in registers.  The row is written once without the choices' own parts, and
// then the choices' places once more: k of them, still in L2.  Bound by memory.
#include "csf_elem.cuh"
#include "csf_internal.cuh"
#include "csf_layer.h"

namespace csfk {
namespace {

constexpr int kGradThreads = 256;

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

// CHUNKS: 256 experts each; 0: renormalised weights, whose gradient is 0 but
// for the choices.
template <int DTYPE, int CHUNKS>
__global__ void __launch_bounds__(kGradThreads) route_grad_kernel(const __grid_constant__ RouteGradParams p) {
    const int lane = threadIdx.x & 31;
    const int64_t t = (int64_t)blockIdx.x * (kGradThreads / 32) + (threadIdx.x >> 5);
    if (t >= p.tokens) return;
    constexpr bool kAll = CHUNKS > 0;
    const char *row = p.logits + t * p.logits_stride;
    char *out = p.out + t * p.out_stride;
    int id = -1;
    float w = 0.f, d = 0.f;
    if (lane < p.k) {
        id = p.ids[t * p.k + lane];
        if (id < 0 || id >= p.experts) id = -1;
        if (id >= 0) w = p.weights[t * p.k + lane], d = p.dweights[t * p.k + lane];
    }
    float dot = w * d;
#pragma unroll
    for (int s = 16; s > 0; s >>= 1) dot += __shfl_xor_sync(0xFFFFFFFFu, dot, s);
    float own = kAll ? w * d : w * (d - dot);
    // a choice made twice has both parts
    float both = 0.f;
    for (int j = 0; j < p.k; ++j) {
        const float other = __shfl_sync(0xFFFFFFFFu, own, j);
        if (__shfl_sync(0xFFFFFFFFu, id, j) == id) both += other;
    }
    own = both;
    if constexpr (kAll) {
        elem::Raw r[CHUNKS];
#pragma unroll
        for (int i = 0; i < CHUNKS; ++i) r[i] = elem::load(row, (lane + 32 * i) * 8, p.experts, DTYPE, p.wide_logits);
        const float mine = id >= 0 ? at(row, id, DTYPE) : 0.f;
        float most = __int_as_float(0xFF800000), sum = 0.f;
        float v[CHUNKS][8];
#pragma unroll
        for (int i = 0; i < CHUNKS; ++i) {
            elem::to_floats(v[i], r[i], DTYPE);
#pragma unroll
            for (int q = 0; q < 8; ++q) {
                if ((lane + 32 * i) * 8 + q >= p.experts) v[i][q] = __int_as_float(0xFF800000);
                most = fmaxf(most, v[i][q]);
            }
        }
#pragma unroll
        for (int s = 16; s > 0; s >>= 1) most = fmaxf(most, __shfl_xor_sync(0xFFFFFFFFu, most, s));
        const bool none = most == __int_as_float(0xFF800000);      // every expert is off: their exponentials are 0
        const float zero = none ? 0.f : most;
#pragma unroll
        for (int i = 0; i < CHUNKS; ++i)
#pragma unroll
            for (int q = 0; q < 8; ++q) sum += v[i][q] = expf(v[i][q] - zero);
#pragma unroll
        for (int s = 16; s > 0; s >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, s);
        const float rate = none ? 0.f : -dot / sum;
        own += expf(mine - zero) * rate;
        __syncwarp();      // every lane has read: the row may be written where it lay
#pragma unroll
        for (int i = 0; i < CHUNKS; ++i) {
            const int c = (lane + 32 * i) * 8;
            if (c >= p.experts) break;
#pragma unroll
            for (int q = 0; q < 8; ++q) v[i][q] *= rate;
            elem::store(out, c, p.experts, elem::from_floats(v[i], DTYPE), DTYPE, p.wide_out);
        }
    } else {
        const elem::Raw zeros = {make_uint4(0, 0, 0, 0), make_uint4(0, 0, 0, 0)};
        for (int c = lane * 8; c < p.experts; c += 256) elem::store(out, c, p.experts, zeros, DTYPE, p.wide_out);
    }
    __syncwarp();
    if (id >= 0) {
        if (DTYPE == CSF_F32) reinterpret_cast<float *>(out)[id] = own;
        else if (DTYPE == CSF_BF16) reinterpret_cast<__nv_bfloat16 *>(out)[id] = __float2bfloat16_rn(own);
        else reinterpret_cast<__half *>(out)[id] = __float2half_rn(own);
    }
}

template <int DTYPE>
void launch(const RouteGradParams &p, bool renormalize, cudaStream_t s) {
    const unsigned grid = (unsigned)(((int64_t)p.tokens + kGradThreads / 32 - 1) / (kGradThreads / 32));
    const int chunks = renormalize ? 0 : (p.experts + 255) / 256;
    switch (chunks) {
        case 0: route_grad_kernel<DTYPE, 0><<<grid, kGradThreads, 0, s>>>(p); break;
        case 1: route_grad_kernel<DTYPE, 1><<<grid, kGradThreads, 0, s>>>(p); break;
        case 2: route_grad_kernel<DTYPE, 2><<<grid, kGradThreads, 0, s>>>(p); break;
        case 3: route_grad_kernel<DTYPE, 3><<<grid, kGradThreads, 0, s>>>(p); break;
        default: route_grad_kernel<DTYPE, 4><<<grid, kGradThreads, 0, s>>>(p); break;
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
