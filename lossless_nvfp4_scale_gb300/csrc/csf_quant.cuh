// Quantised rows (csf_rows in csf_ops.h): block scales, code conversions and
// element types shared by the operator kernels.  Internal to the library.
#pragma once

#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp4.h>
#include <cuda_fp8.h>

#include "csf_ops.h"

namespace csfk {
namespace quant {

// Smallest power of two s with amax <= 448 s, as its UE8M0 byte: 448 =
// 1.75 * 2^8, so the exponent of amax less 8, and one more when its fraction
// is above .75.  amax_bits: the bits of a non-negative float.
__device__ __forceinline__ uint32_t mx_scale(uint32_t amax_bits) {
    const int x = (int)(amax_bits >> 23);
    if (x == 255) return 255;
    const int b = x - 8 + ((amax_bits & 0x7FFFFFu) > 0x600000u ? 1 : 0);
    return b < 0 ? 0 : (uint32_t)b;
}

// 1 / scale, exact (a NaN scale's codes mean nothing: 1).
__device__ __forceinline__ float mx_inverse(uint32_t byte) {
    return __uint_as_float(byte == 255 ? 127u << 23 : (254u - byte) << 23);
}

// UE4M3 byte of amax / (6 * tensor scale).
__device__ __forceinline__ uint32_t nv_scale(uint32_t amax_bits, float six_tensor_scales) {
    if ((amax_bits >> 23) == 255) return 0x7F;
    return __nv_cvt_float_to_fp8(__fdiv_rn(__uint_as_float(amax_bits), six_tensor_scales), __NV_SATFINITE, __NV_E4M3);
}

// scale * tensor scale, and its inverse to a unit in the last place (0 for a
// zero scale; whole ones are normal numbers up to 2^126).
struct Whole {
    float value, inverse;
};

__device__ __forceinline__ Whole nv_whole(uint32_t byte, float tensor_scale) {
    const float s = __half2float(__half(__nv_cvt_fp8_to_halfraw((__nv_fp8_storage_t)byte, __NV_E4M3)));
    Whole w;
    w.value = s * tensor_scale;
    float inverse;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(inverse) : "f"(w.value));
    w.inverse = s > 0.f ? inverse : 0.f;
    return w;
}

// v / whole: the product with the inverse, corrected by its remainder
// (Markstein's last step of a division, 1990), so that values next to the
// middle of two codes round as the quotient does.
__device__ __forceinline__ float over(float v, const Whole &w) {
    const float q = v * w.inverse;
    return fmaf(fmaf(-q, w.value, v), w.inverse, q);
}

// Two values -> two E4M3 bytes, the first in the low byte.
__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
    return __nv_cvt_float2_to_fp8x2(make_float2(lo, hi), __NV_SATFINITE, __NV_E4M3);
}

// Two values -> two E2M1 codes, the first in the low nibble.
__device__ __forceinline__ uint32_t e2m1x2(float lo, float hi) {
    return __nv_cvt_float2_to_fp4x2(make_float2(lo, hi), __NV_E2M1, cudaRoundNearest);
}

// Quantise columns 8 * chunk .. +7 of a row.  Every lane of a block's 4 (32
// columns, MXFP8) or 2 (16 columns, NVFP4) calls it together, `write` or not.
template <int KIND>
__device__ __forceinline__ void quantize8(const float (&y)[8], uint8_t *codes, uint8_t *scales, int chunk, bool write,
                                          float tensor_scale) {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = max(m, __float_as_uint(y[i]) & 0x7FFFFFFFu);
    m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, 1));
    if constexpr (KIND == CSF_ROWS_MXFP8) m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, 2));
    if (!write) return;
    if constexpr (KIND == CSF_ROWS_MXFP8) {
        const uint32_t s = mx_scale(m);
        const float inv = mx_inverse(s);
        uint2 q;
        q.x = e4m3x2(y[0] * inv, y[1] * inv) | e4m3x2(y[2] * inv, y[3] * inv) << 16;
        q.y = e4m3x2(y[4] * inv, y[5] * inv) | e4m3x2(y[6] * inv, y[7] * inv) << 16;
        *reinterpret_cast<uint2 *>(codes + chunk * 8) = q;
        if ((chunk & 3) == 0) scales[chunk >> 2] = (uint8_t)s;
    } else {
        const uint32_t s = nv_scale(m, 6.f * tensor_scale);
        const Whole w = nv_whole(s, tensor_scale);
        float v[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = y[i];
        if (s == 0x7E) {
            // The largest scale: values may be far past 6 of it, and a quotient
            // that overflows has no remainder to correct it by.  What is past
            // 5 of it is coded 6.
            const float most = 6.5f * w.value;
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = fminf(fmaxf(v[i], -most), most);
        }
        *reinterpret_cast<uint32_t *>(codes + chunk * 4) =
            e2m1x2(over(v[0], w), over(v[1], w)) | e2m1x2(over(v[2], w), over(v[3], w)) << 8 |
            e2m1x2(over(v[4], w), over(v[5], w)) << 16 | e2m1x2(over(v[6], w), over(v[7], w)) << 24;
        if ((chunk & 1) == 0) scales[chunk >> 1] = (uint8_t)s;
    }
}

}  // namespace quant

// SMs of the current device (0: no device).
int sm_count();

inline int64_t round_up(int64_t n, int64_t m) { return (n + m - 1) / m * m; }
inline size_t dtype_bytes(int dtype) { return dtype == CSF_F32 ? 4 : 2; }
inline bool dtype_known(int dtype) { return dtype == CSF_BF16 || dtype == CSF_F16 || dtype == CSF_F32; }
inline bool aligned_to(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

// A csf_rows that a call reads or writes; `rows` of 0 need no buffers.
inline bool rows_valid(const csf_rows &r) {
    if ((r.kind != CSF_ROWS_NVFP4 && r.kind != CSF_ROWS_MXFP8) || r.cols < 1 || r.rows < 0) return false;
    if (r.rows == 0) return true;
    const int64_t cols = round_up(r.cols, 32);
    const int64_t code_bytes = r.kind == CSF_ROWS_NVFP4 ? cols / 2 : cols;
    const int64_t blocks = r.kind == CSF_ROWS_NVFP4 ? cols / 16 : cols / 32;
    return r.codes && r.scales && aligned_to(r.codes, 16) && aligned_to(r.scales, 16) && r.code_stride % 16 == 0 &&
           r.scale_stride % 16 == 0 && r.code_stride >= code_bytes && r.scale_stride >= round_up(blocks, 16);
}

}  // namespace csfk
