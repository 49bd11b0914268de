// Top-k router (csf_route): expert choice, weights, and slots grouped by
// expert in token order.
//
// Tokens are taken 64 at a time by a block, one token a warp: the row's
// logits sit in registers as order-preserving integers and each of the k
// choices is one warp maximum and one warp minimum over the experts that hold
// it.  A token picks an expert at most once, so a 64-bit mask per expert holds
// a block's choices: its population is the block's count and the bits below a
// token its rank, whatever the order of the updates -- the slots depend on the
// logits alone.  Up to 64 tokens one block does everything; else a scan over
// the blocks' counts and a placing pass follow.
#include "csf_internal.cuh"
#include "csf_quant.cuh"

namespace csfk {
namespace {

constexpr int kRouteTokens = 64;       // tokens per block
constexpr int kRouteThreads = 512;
constexpr int kRouteMaxExperts = 1024;
constexpr int kRouteMaxK = 32;

struct RouteParams {
    const void *logits;
    int64_t stride;
    int32_t T, E, k, renormalize;
    int32_t *ids, *start, *rows, *slots;
    float *weights;
    uint32_t *counts;    // [blocks][E]: counts, then their prefixes over the blocks
    uint32_t *totals;    // [E]
};

// Larger logit, larger key; -inf (an expert switched off) has key 0, NaN the largest.
__device__ __forceinline__ uint32_t key_of(float v) {
    const uint32_t b = __float_as_uint(v + 0.f);      // -0 becomes 0
    if ((b & 0x7FFFFFFFu) > 0x7F800000u) return 0xFFFFFFFFu;
    if (b == 0xFF800000u) return 0;
    return b ^ ((b >> 31) ? 0xFFFFFFFFu : 0x80000000u);
}

__device__ __forceinline__ float value_of(uint32_t key) {
    if (key == 0xFFFFFFFFu) return __uint_as_float(0x7FC00000u);
    if (key == 0) return __uint_as_float(0xFF800000u);
    return __uint_as_float(key ^ ((key >> 31) ? 0x80000000u : 0xFFFFFFFFu));
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, d);
    return v;
}

// Exclusive prefix of cnt[0..E) (shared) into out[0..E], by the whole block.
__device__ __forceinline__ void scan_experts(const uint32_t *cnt, uint32_t *out, int E, uint32_t *warp_sums) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    uint32_t running = 0;
    for (int e0 = 0; e0 < E; e0 += kRouteThreads) {
        const int e = e0 + threadIdx.x;
        const uint32_t c = e < E ? cnt[e] : 0;
        uint32_t sum = c;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const uint32_t o = __shfl_up_sync(0xFFFFFFFFu, sum, d);
            if (lane >= d) sum += o;
        }
        if (lane == 31) warp_sums[warp] = sum;
        __syncthreads();
        uint32_t before = running;
        for (int w = 0; w < kRouteThreads / 32; ++w) {
            const uint32_t s = warp_sums[w];
            if (w < warp) before += s;
            running += s;
        }
        if (e < E) out[e] = before + sum - c;
        __syncthreads();
    }
    if (threadIdx.x == 0) out[E] = running;
    __syncthreads();
}

// VPL: logits per lane (E <= 32 * VPL).  ONE: the only block, which also
// places the slots.
template <typename T, int VPL, bool ONE>
__global__ void __launch_bounds__(kRouteThreads)
route_choose_kernel(const __grid_constant__ RouteParams p) {
    __shared__ uint32_t mask[2][kRouteMaxExperts];
    __shared__ uint32_t start[ONE ? kRouteMaxExperts + 1 : 1];
    __shared__ uint32_t cnt[ONE ? kRouteMaxExperts : 1];
    __shared__ uint32_t sums[kRouteThreads / 32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int t0 = blockIdx.x * kRouteTokens;
    const int nt = min(kRouteTokens, p.T - t0);
    for (int e = threadIdx.x; e < p.E; e += kRouteThreads) mask[0][e] = mask[1][e] = 0;
    __syncthreads();
    for (int i = warp; i < nt; i += kRouteThreads / 32) {
        const int64_t t = t0 + i;
        const T *row = static_cast<const T *>(p.logits) + t * p.stride;
        T raw[VPL];
        uint32_t key[VPL];
#pragma unroll
        for (int j = 0; j < VPL; ++j) {
            const int e = lane + 32 * j;
            raw[j] = e < p.E ? row[e] : T(0.f);
        }
#pragma unroll
        for (int j = 0; j < VPL; ++j) key[j] = lane + 32 * j < p.E ? key_of((float)raw[j]) : 0;
        // The lane's two best, ties to the lower expert.  Eight choices seldom
        // take a lane's third: only then are its logits gone through again.
        uint32_t best, second;
        int best_at, second_at;
        auto look = [&]() {
            best = second = 0;
            best_at = second_at = 0;
#pragma unroll
            for (int j = 0; j < VPL; ++j) {
                if (key[j] > best) second = best, second_at = best_at, best = key[j], best_at = j;
                else if (key[j] > second) second = key[j], second_at = j;
            }
        };
        look();
        const float vmax = value_of(__reduce_max_sync(0xFFFFFFFFu, best));
        float total = 0.f;
        if (!p.renormalize) {
#pragma unroll
            for (int j = 0; j < VPL; ++j)
                if (key[j]) total += expf(value_of(key[j]) - vmax);
            total = warp_sum(total);
        }
        int id = -1;
        uint32_t mine = 0, taken = 0;      // this lane's choice; which of its logits are gone
        int spare = 1;
        for (int c = 0; c < p.k; ++c) {
            const uint32_t top = __reduce_max_sync(0xFFFFFFFFu, best);
            if (top == 0) break;                       // no expert left
            const uint32_t e = __reduce_min_sync(0xFFFFFFFFu, best == top ? (uint32_t)(lane + 32 * best_at) : 0xFFFFFFFFu);
            if (lane == c) id = (int)e, mine = top;
            if ((e & 31) == (uint32_t)lane) {
                taken |= 1u << (e >> 5);
                if (spare) {
                    best = second, best_at = second_at;
                    spare = 0;
                } else {
#pragma unroll
                    for (int j = 0; j < VPL; ++j)
                        if (taken >> j & 1) key[j] = 0;
                    look();
                    spare = 1;
                }
            }
        }
        const float w = id < 0 ? 0.f : expf(value_of(mine) - vmax);
        if (p.renormalize) total = warp_sum(w);
        if (lane < p.k) {
            p.ids[t * p.k + lane] = id;
            p.weights[t * p.k + lane] = id < 0 ? 0.f : w / total;
            if (id >= 0) atomicOr(&mask[i >> 5][id], 1u << (i & 31));
        }
    }
    __syncthreads();
    if constexpr (ONE) {
        for (int e = threadIdx.x; e < p.E; e += kRouteThreads) cnt[e] = __popc(mask[0][e]) + __popc(mask[1][e]);
        __syncthreads();
        scan_experts(cnt, start, p.E, sums);
        for (int e = threadIdx.x; e <= p.E; e += kRouteThreads) p.start[e] = (int32_t)start[e];
        for (int i = (int)start[p.E] + threadIdx.x; i < p.T * p.k; i += kRouteThreads) p.rows[i] = -1;
    } else {
        for (int e = threadIdx.x; e < p.E; e += kRouteThreads)
            p.counts[(int64_t)blockIdx.x * p.E + e] = __popc(mask[0][e]) + __popc(mask[1][e]);
    }
    // the rank of each choice in its expert, within the block
    for (int i = threadIdx.x; i < nt * p.k; i += kRouteThreads) {
        const int64_t at = (int64_t)t0 * p.k + i;
        const int t = i / p.k;
        const int id = p.ids[at];
        int slot = -1;
        if (id >= 0) {
            const uint32_t lo = mask[0][id], hi = mask[1][id];
            const uint32_t below = (1u << (t & 31)) - 1u;
            slot = t < 32 ? __popc(lo & below) : __popc(lo) + __popc(hi & below);
            if constexpr (ONE) {
                slot += (int)start[id];
                p.rows[slot] = t;
            }
        }
        p.slots[at] = slot;
    }
}

// Exclusive prefix of the blocks' counts per expert, 32 experts a block and
// one segment of the blocks a warp.
__global__ void __launch_bounds__(1024)
route_scan_kernel(const __grid_constant__ RouteParams p, int blocks) {
    __shared__ uint32_t part[32][33];
    const int lane = threadIdx.x & 31, seg = threadIdx.x >> 5;
    const int e = blockIdx.x * 32 + lane;
    const int per = (blocks + 31) / 32, b0 = min(blocks, seg * per), b1 = min(blocks, b0 + per);
    uint32_t sum = 0;
    if (e < p.E) {
#pragma unroll 8
        for (int b = b0; b < b1; ++b) sum += p.counts[(int64_t)b * p.E + e];
    }
    part[seg][lane] = sum;
    __syncthreads();
    uint32_t before = 0, total = 0;
#pragma unroll
    for (int s = 0; s < 32; ++s) {
        const uint32_t v = part[s][lane];
        before += s < seg ? v : 0;
        total += v;
    }
    if (e < p.E) {
        if (seg == 0) p.totals[e] = total;
        for (int b = b0; b < b1; ++b) {
            const uint32_t c = p.counts[(int64_t)b * p.E + e];
            p.counts[(int64_t)b * p.E + e] = before;
            before += c;
        }
    }
}

// Ranks within the blocks become slots.
__global__ void __launch_bounds__(kRouteThreads)
route_place_kernel(const __grid_constant__ RouteParams p) {
    __shared__ uint32_t start[kRouteMaxExperts + 1], cnt[kRouteMaxExperts], sums[kRouteThreads / 32];
    for (int e = threadIdx.x; e < p.E; e += kRouteThreads) cnt[e] = p.totals[e];
    __syncthreads();
    scan_experts(cnt, start, p.E, sums);
    if (blockIdx.x == 0)
        for (int e = threadIdx.x; e <= p.E; e += kRouteThreads) p.start[e] = (int32_t)start[e];
    const int t0 = blockIdx.x * kRouteTokens;
    const int nt = min(kRouteTokens, p.T - t0);
    const uint32_t *before = p.counts + (int64_t)blockIdx.x * p.E;
    for (int i = threadIdx.x; i < nt * p.k; i += kRouteThreads) {
        const int64_t at = (int64_t)t0 * p.k + i;
        const int id = p.ids[at];
        if (id < 0) continue;
        const int slot = (int)(start[id] + before[id]) + p.slots[at];
        p.slots[at] = slot;
        p.rows[slot] = t0 + i / p.k;
    }
    const int64_t all = (int64_t)p.T * p.k, threads = (int64_t)gridDim.x * kRouteThreads;
    for (int64_t i = start[p.E] + (int64_t)blockIdx.x * kRouteThreads + threadIdx.x; i < all; i += threads) p.rows[i] = -1;
}

__global__ void route_none_kernel(int32_t *start, int E) {
    for (int e = threadIdx.x; e <= E; e += blockDim.x) start[e] = 0;
}

template <typename T, bool ONE>
void choose_type(const RouteParams &p, int blocks, cudaStream_t s) {
    if (p.E <= 128) route_choose_kernel<T, 4, ONE><<<blocks, kRouteThreads, 0, s>>>(p);
    else if (p.E <= 256) route_choose_kernel<T, 8, ONE><<<blocks, kRouteThreads, 0, s>>>(p);
    else if (p.E <= 512) route_choose_kernel<T, 16, ONE><<<blocks, kRouteThreads, 0, s>>>(p);
    else route_choose_kernel<T, 32, ONE><<<blocks, kRouteThreads, 0, s>>>(p);
}

template <bool ONE>
void choose(const RouteParams &p, int dtype, int blocks, cudaStream_t s) {
    if (dtype == CSF_BF16) choose_type<__nv_bfloat16, ONE>(p, blocks, s);
    else if (dtype == CSF_F16) choose_type<__half, ONE>(p, blocks, s);
    else choose_type<float, ONE>(p, blocks, s);
}

}  // namespace
}  // namespace csfk

using namespace csfk;

extern "C" size_t csf_route_scratch_bytes(int32_t tokens, int32_t experts) {
    if (tokens <= kRouteTokens || experts < 1) return 0;
    const size_t blocks = ((size_t)tokens + kRouteTokens - 1) / kRouteTokens;
    return (size_t)round_up((int64_t)((blocks + 1) * (size_t)experts * 4), 16);
}

extern "C" csf_status csf_route(const csf_route_args *a, void *stream) {
    if (!a || !dtype_known(a->dtype) || a->tokens < 0 || a->experts < 1 || a->k < 1 || a->k > a->experts) return CSF_ERR_ARG;
    if (a->experts > kRouteMaxExperts || a->k > kRouteMaxK) return CSF_ERR_UNSUPPORTED;
    if ((int64_t)a->tokens * a->k >= (1ll << 31)) return CSF_ERR_UNSUPPORTED;
    if (!a->expert_start) return CSF_ERR_ARG;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (a->tokens > 0) {
        if (!a->logits || !a->ids || !a->weights || !a->rows || !a->slots || a->logits_stride < a->experts) return CSF_ERR_ARG;
        if (!aligned_to(a->logits, dtype_bytes(a->dtype))) return CSF_ERR_ARG;
    }
    const size_t need = csf_route_scratch_bytes(a->tokens, a->experts);
    if (need > 0) {
        if (!a->scratch || !aligned_to(a->scratch, 16)) return CSF_ERR_ARG;
        if (a->scratch_bytes < need) return CSF_ERR_SIZE;
    }
    RouteParams p;
    p.logits = a->logits;
    p.stride = a->logits_stride;
    p.T = a->tokens;
    p.E = a->experts;
    p.k = a->k;
    p.renormalize = a->renormalize;
    p.ids = a->ids;
    p.start = a->expert_start;
    p.rows = a->rows;
    p.slots = a->slots;
    p.weights = a->weights;
    const int blocks = (p.T + kRouteTokens - 1) / kRouteTokens;
    p.totals = static_cast<uint32_t *>(a->scratch);
    p.counts = p.totals + p.E;
    if (p.T == 0) {
        route_none_kernel<<<1, 256, 0, s>>>(p.start, p.E);
    } else if (blocks == 1) {
        choose<true>(p, a->dtype, 1, s);
    } else {
        choose<false>(p, a->dtype, blocks, s);
        route_scan_kernel<<<(p.E + 31) / 32, 1024, 0, s>>>(p, blocks);
        route_place_kernel<<<blocks, kRouteThreads, 0, s>>>(p);
    }
    return cudaGetLastError() == cudaSuccess ? CSF_OK : CSF_ERR_CUDA;
}
