// 8 neighbouring elements of a plain row, of a type known at run time, as
// floats.  Internal to the library.
#pragma once

#include <cstring>

#include "csf_quant.cuh"

namespace csfk {
namespace elem {

// 8 elements as stored: 16 bytes of 16-bit types (in a), 32 of float32.
struct Raw {
    uint4 a, b;
};

// A row's elements from column c on; `wide`: 16-byte aligned.  Columns past
// `cols` are 0.
__device__ __forceinline__ Raw load(const void *row, int c, int cols, int dtype, bool wide) {
    Raw r = {make_uint4(0, 0, 0, 0), make_uint4(0, 0, 0, 0)};
    if (dtype == CSF_F32) {
        const float *at = static_cast<const float *>(row) + c;
        if (wide && c + 8 <= cols) {
            r.a = __ldg(reinterpret_cast<const uint4 *>(at));
            r.b = __ldg(reinterpret_cast<const uint4 *>(at) + 1);
        } else {
            uint32_t v[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = c + i < cols ? __float_as_uint(at[i]) : 0u;
            r.a = make_uint4(v[0], v[1], v[2], v[3]);
            r.b = make_uint4(v[4], v[5], v[6], v[7]);
        }
    } else {
        const uint16_t *at = static_cast<const uint16_t *>(row) + c;
        if (wide && c + 8 <= cols) {
            r.a = __ldg(reinterpret_cast<const uint4 *>(at));
        } else {
            uint32_t v[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = c + i < cols ? at[i] : 0u;
            r.a = make_uint4(v[0] | v[1] << 16, v[2] | v[3] << 16, v[4] | v[5] << 16, v[6] | v[7] << 16);
        }
    }
    return r;
}

__device__ __forceinline__ void to_floats(float (&y)[8], const Raw &r, int dtype) {
    const uint32_t u[8] = {r.a.x, r.a.y, r.a.z, r.a.w, r.b.x, r.b.y, r.b.z, r.b.w};
    if (dtype == CSF_BF16) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            y[2 * i] = __uint_as_float(u[i] << 16);
            y[2 * i + 1] = __uint_as_float(u[i] & 0xFFFF0000u);
        }
    } else if (dtype == CSF_F32) {
#pragma unroll
        for (int i = 0; i < 8; ++i) y[i] = __uint_as_float(u[i]);
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            __half2 h;
            memcpy(&h, &u[i], 4);
            const float2 f = __half22float2(h);
            y[2 * i] = f.x;
            y[2 * i + 1] = f.y;
        }
    }
}

// Rounded once, to nearest, ties to even.
__device__ __forceinline__ Raw from_floats(const float (&y)[8], int dtype) {
    Raw r;
    if (dtype == CSF_F32) {
        r.a = make_uint4(__float_as_uint(y[0]), __float_as_uint(y[1]), __float_as_uint(y[2]), __float_as_uint(y[3]));
        r.b = make_uint4(__float_as_uint(y[4]), __float_as_uint(y[5]), __float_as_uint(y[6]), __float_as_uint(y[7]));
        return r;
    }
    uint32_t u[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if (dtype == CSF_BF16) {
            const __nv_bfloat162 h = __floats2bfloat162_rn(y[2 * i], y[2 * i + 1]);
            memcpy(&u[i], &h, 4);
        } else {
            const __half2 h = __floats2half2_rn(y[2 * i], y[2 * i + 1]);
            memcpy(&u[i], &h, 4);
        }
    }
    r.a = make_uint4(u[0], u[1], u[2], u[3]);
    r.b = make_uint4(0, 0, 0, 0);
    return r;
}

__device__ __forceinline__ void store(void *row, int c, int cols, const Raw &r, int dtype, bool wide) {
    if (wide && c + 8 <= cols) {
        uint4 *at = reinterpret_cast<uint4 *>(static_cast<char *>(row) + (size_t)c * (dtype == CSF_F32 ? 4 : 2));
        at[0] = r.a;
        if (dtype == CSF_F32) at[1] = r.b;
        return;
    }
    const uint32_t u[8] = {r.a.x, r.a.y, r.a.z, r.a.w, r.b.x, r.b.y, r.b.z, r.b.w};
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        if (c + i >= cols) break;
        if (dtype == CSF_F32) static_cast<uint32_t *>(row)[c + i] = u[i];
        else static_cast<uint16_t *>(row)[c + i] = (uint16_t)(u[i >> 1] >> (16 * (i & 1)));
    }
}

// The same for kernels that are short of registers: what is not wide is a
// function of its own.
static __device__ __noinline__ Raw load_few(const void *row, int c, int cols, int dtype) { return load(row, c, cols, dtype, false); }
static __device__ __noinline__ void store_few(void *row, int c, int cols, const Raw r, int dtype) { store(row, c, cols, r, dtype, false); }

__device__ __forceinline__ Raw load_apart(const void *row, int c, int cols, int dtype, bool wide) {
    if (!wide || c + 8 > cols) return load_few(row, c, cols, dtype);
    Raw r;
    const uint4 *at = reinterpret_cast<const uint4 *>(static_cast<const char *>(row) + (size_t)c * (dtype == CSF_F32 ? 4 : 2));
    r.a = __ldg(at);
    r.b = dtype == CSF_F32 ? __ldg(at + 1) : make_uint4(0, 0, 0, 0);
    return r;
}

__device__ __forceinline__ void store_apart(void *row, int c, int cols, const Raw &r, int dtype, bool wide) {
    if (!wide || c + 8 > cols) {
        store_few(row, c, cols, r, dtype);
        return;
    }
    uint4 *at = reinterpret_cast<uint4 *>(static_cast<char *>(row) + (size_t)c * (dtype == CSF_F32 ? 4 : 2));
    at[0] = r.a;
    if (dtype == CSF_F32) at[1] = r.b;
}

}  // namespace elem

// Whether rows may be accessed 16 bytes at a time.
inline bool wide_rows(const void *p, int64_t stride, int dtype) {
    return aligned_to(p, 16) && (stride * (int64_t)dtype_bytes(dtype)) % 16 == 0;
}

}  // namespace csfk
