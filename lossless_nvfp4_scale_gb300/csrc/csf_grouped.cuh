// What the grouped products share: the tiles of slots that belong to experts,
// the position in a ring of stages, and the activations.  Internal to the
// library.
#pragma once

#include <cstdint>

#include "csf_ops.h"

namespace csfk {
namespace mm {

// v / (1 + exp(-z)), within 2^-20 of itself: with h = exp(-|z| / 2) the divisor
// is 1 + h^2, and the dividend v or, for a negative z, v h^2, one factor at a
// time so that neither a large v nor a small h^2 is lost.  The exponent's
// product with log2(e) carries its rounding error along (the error of a
// product by fma), and the quotient its remainder (Markstein's last step of a
// division, 1990).  (expf and the division cost the dense product 52 us of
// 130; the approximate forms alone are off by 1e-6 of the value, which shows
// where the result is rounded to 8 bits.)
__device__ __forceinline__ float times_sigmoid(float v, float z) {
    constexpr double kHalfLog2e = 0.72134752044448170;
    constexpr float kScale = (float)kHalfLog2e, kRest = (float)(kHalfLog2e - (double)kScale), kLn2 = 0.6931471805599453f;
    const float m = fminf(fabsf(z), 180.f);           // h of more is 0
    const float t = -m * kScale;
    const float rest = fmaf(-m, kScale, -t) - m * kRest;
    float h;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(h) : "f"(t));
    h = fmaf(h, rest * kLn2, h);
    const float d = fmaf(h, h, 1.f);
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(d));
    const float s = z < 0.f ? h : 1.f;
    const float n = v * s * s;                        // -inf * 0: NaN, as inf / inf
    const float q = n * r;
    return fabsf(n) < __int_as_float(0x7F800000) ? fmaf(fmaf(-q, d, n), r, q) : n;     // an infinity has no remainder
}

// v * sigmoid(z), z = 2 * sqrt(2 / pi) * (v + 0.044715 v^3), is the tanh form of
// GELU.  z's roundings (2^-22 of it at most) add |z| 2^-21 to the 2^-20 above.
__device__ __forceinline__ float smooth(float v, bool gelu) {
    return times_sigmoid(v, gelu ? 1.5957691216057308f * (v + 0.044715f * v * v * v) : v);
}

template <class P>
__device__ __forceinline__ int64_t start_at(const P &p, int e) {
    if (!p.start) return e == 0 ? 0 : p.slots;
    const int64_t v = p.es64 ? static_cast<const long long *>(p.start)[e] : static_cast<const int *>(p.start)[e];
    return v < 0 ? 0 : v > p.slots ? p.slots : v;
}

struct Tile {
    int e, n, rt;     // expert, slots, row tile
    uint32_t slot;    // first slot
};

// The tile with this number.  Row tiles of one slot tile are neighbours, so
// their x rows are shared in L2.  Its expert is the last whose first slot tile
// is not past the tile's, found 32 candidates at a time.
template <class P>
__device__ __forceinline__ Tile find_tile(const P &p, const uint32_t *first, const uint32_t *slot0, uint32_t tile, int lane) {
    const uint32_t rt = (uint32_t)p.row_tiles;
    uint32_t st = rt == 1 ? tile : __umulhi(tile, p.row_tiles_magic);      // tile / row tiles, or one more
    int row_tile = (int)(tile - st * rt);
    if (row_tile < 0) --st, row_tile += (int)rt;
    int lo = 0, len = p.E;
    while (len > 1) {
        const int step = (len + 31) >> 5;
        const int i = lo + lane * step;
        const uint32_t m = __ballot_sync(0xFFFFFFFFu, i < lo + len && first[i] <= st);
        const int at = lo + (31 - __clz(m)) * step;
        len = min(step, lo + len - at);
        lo = at;
    }
    Tile t;
    t.e = lo;
    t.rt = row_tile;
    const uint32_t part = st - first[lo], parts = first[lo + 1] - first[lo];
    const uint32_t s = slot0[lo], cnt = slot0[lo + 1] - s;
    // an expert's slot tiles are alike
    const uint32_t per = parts == 1 ? cnt : ((cnt + parts - 1) / parts + 15u) & ~15u;
    t.slot = s + part * per;
    t.n = (int)min(per, cnt - part * per);
    return t;
}

// first[e]: the number of the first slot tile of expert e (of up to p.nt
// slots), slot0[e] its first slot.  Returns how many there are; `bad`: an
// expert_start out of order or range was seen by this thread.  All THREADS of
// the block; warp_sum holds a word a warp.
template <int THREADS, class P>
__device__ __forceinline__ uint32_t number_tiles(const P &p, uint32_t *first, uint32_t *slot0, uint32_t *warp_sum, bool &bad) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    uint32_t running = 0;
    for (int e0 = 0; e0 < p.E; e0 += THREADS) {
        const int e = e0 + tid;
        uint32_t tiles = 0;
        if (e < p.E) {
            const int64_t a = start_at(p, e), b = start_at(p, e + 1);
            slot0[e] = (uint32_t)a;
            if (b > a) tiles = (uint32_t)((b - a + p.nt - 1) / p.nt);
            if (p.start) {
                const long long raw = p.es64 ? static_cast<const long long *>(p.start)[e + 1] : static_cast<const int *>(p.start)[e + 1];
                const long long raw0 = p.es64 ? static_cast<const long long *>(p.start)[e] : static_cast<const int *>(p.start)[e];
                bad |= raw != b || raw0 != a || b < a;
            }
        }
        uint32_t sum = tiles;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const uint32_t o = __shfl_up_sync(0xFFFFFFFFu, sum, d);
            if (lane >= d) sum += o;
        }
        if (lane == 31) warp_sum[warp] = sum;
        __syncthreads();
        uint32_t before = running;
        for (int w = 0; w < THREADS / 32; ++w) {
            const uint32_t s = warp_sum[w];
            if (w < warp) before += s;
            running += s;
        }
        if (e < p.E) first[e] = before + sum - tiles;
        __syncthreads();
    }
    return running;
}

// Position in the ring of stages, and the parity of its round.
struct Ring {
    uint32_t s = 0, parity = 0;
    __device__ __forceinline__ void next(int stages) {
        if (++s == (uint32_t)stages) s = 0, parity ^= 1u;
    }
};

}  // namespace mm
}  // namespace csfk
