// Top-k router (csf_route): expert choice, weights, and slots grouped by
// expert in token order.
//
// Tokens are taken 64 at a time by a block, one token a warp: the row's
// logits sit in registers as order-preserving integers and each of the k
// choices is one or two warp reductions.  A token picks an expert at most
// once, so a 64-bit mask per expert holds a block's choices: its population
// is the block's count and the bits below a token its rank, whatever the
// order of the updates -- the slots depend on the logits alone.
//
// Up to 512 tokens a cluster of blocks does everything and passes its counts
// through shared memory (333 tokens of 129 experts: 12.5 us, 15 as three
// launches); else a scan over the blocks' counts and a placing pass follow.
// Bound by instructions: 32768 tokens of 384 bfloat16 experts, k = 8, take
// 38.8 us, 0.76 TB/s, about 600 warp instructions a token.
#include "csf_internal.cuh"
#include "csf_quant.cuh"
#include "csf_tc.cuh"

namespace csfk {
namespace {

constexpr int kRouteTokens = 64;       // tokens per block
constexpr int kRouteThreads = 512;
constexpr int kRouteCluster = 8;       // blocks of the one-launch form, at most
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

// Order-preserving integers of logits: larger logit, larger rank; -0 as 0; NaN
// above every number; ranks up to `off` are -inf, an expert switched off.
template <typename T> struct Rank;
template <> struct Rank<float> {
    static constexpr uint32_t off = 0;
    static __device__ __forceinline__ uint32_t of(float v) {
        const uint32_t b = __float_as_uint(v + 0.f);
        if ((b & 0x7FFFFFFFu) > 0x7F800000u) return 0xFFFFFFFFu;
        if (b == 0xFF800000u) return 0;
        return b ^ ((b >> 31) ? 0xFFFFFFFFu : 0x80000000u);
    }
    static __device__ __forceinline__ float value(uint32_t r) {
        if (r == 0xFFFFFFFFu) return __uint_as_float(0x7FC00000u);
        return __uint_as_float(r ^ ((r >> 31) ? 0x80000000u : 0xFFFFFFFFu));
    }
};
// 16-bit types: a rank in 16 bits, 0x8000 plus or less the magnitude; INF the
// bits of infinity.
template <uint32_t INF>
struct Rank16 {
    static constexpr uint32_t inf = INF, off = 0x8000u - INF;
    static __device__ __forceinline__ uint32_t bits(uint32_t r) { return r & 0x8000u ? r ^ 0x8000u : (0x8000u - r) | 0x8000u; }
};
template <> struct Rank<__nv_bfloat16> : Rank16<0x7F80u> {
    static __device__ __forceinline__ float value(uint32_t r) { return __uint_as_float(bits(r) << 16); }
};
template <> struct Rank<__half> : Rank16<0x7C00u> {
    static __device__ __forceinline__ float value(uint32_t r) { return __half2float(__ushort_as_half((unsigned short)bits(r))); }
};

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

// A warp's choice among E logits, VPL a lane (E <= 32 * VPL): lane c gets the
// c-th best's expert and rank.  Each lane keeps the two best of its own (eight
// choices of hundreds seldom take a lane's third; only then are its logits
// gone through again).  16-bit ranks carry the expert in their low half, ties
// to the lower one, so that a choice is one warp maximum; 32-bit ones take a
// second reduction for the expert.
template <typename T, int VPL>
struct Choice {
    static constexpr bool kPacked = sizeof(T) == 2;
    uint32_t key[VPL];
    uint32_t best, second;
    int best_at, second_at;

    __device__ __forceinline__ static uint32_t rank(uint32_t k) { return kPacked ? k >> 16 : k; }

    __device__ __forceinline__ void set(const T (&raw)[VPL], int E, int lane) {
        bool nan = false;
#pragma unroll
        for (int j = 0; j < VPL; ++j) {
            const int e = lane + 32 * j;
            if constexpr (kPacked) {
                // a sign and magnitude as two's complement, which ranks -0 as 0
                uint16_t b;
                memcpy(&b, &raw[j], 2);
                const int32_t x = (int32_t)((uint32_t)b << 16), sign = x >> 31;
                const int32_t mag = x & 0x7FFFFFFF;
                nan |= mag > (int32_t)(Rank<T>::inf << 16);
                key[j] = (uint32_t)((mag ^ sign) - sign) + (0x80000000u + 0xFFFFu - (uint32_t)e);
                if (e >= E) key[j] = 0;
            } else {
                key[j] = e < E ? Rank<T>::of(raw[j]) : 0;
            }
        }
        if (kPacked && nan) {
#pragma unroll
            for (int j = 0; j < VPL; ++j) {
                const float v = (float)raw[j];
                if (v != v && lane + 32 * j < E) key[j] = 0xFFFF0000u | (0xFFFFu - (uint32_t)(lane + 32 * j));
            }
        }
    }

    // The two best of the lane: of all (first), then of those below `limit`
    // (packed) or left (not).
    template <bool FIRST>
    __device__ __forceinline__ void look(uint32_t limit) {
        best = second = 0;
        best_at = second_at = 0;
#pragma unroll
        for (int j = 0; j < VPL; ++j) {
            if constexpr (kPacked) {
                const uint32_t k = FIRST || key[j] < limit ? key[j] : 0;
                second = max(second, min(best, k));
                best = max(best, k);
            } else {
                if (key[j] > best) second = best, second_at = best_at, best = key[j], best_at = j;
                else if (key[j] > second) second = key[j], second_at = j;
            }
        }
    }

    __device__ __forceinline__ void choose(int k, int lane, int &id, uint32_t &mine) {
        uint32_t taken = 0;
        bool spare = true;
        id = -1;
        mine = 0;
        for (int c = 0; c < k; ++c) {
            const uint32_t top = __reduce_max_sync(0xFFFFFFFFu, best);
            if (rank(top) <= Rank<T>::off) break;      // no expert left
            uint32_t e;
            if constexpr (kPacked) e = 0xFFFFu - (top & 0xFFFFu);
            else e = __reduce_min_sync(0xFFFFFFFFu, best == top ? (uint32_t)(lane + 32 * best_at) : 0xFFFFFFFFu);
            if (lane == c) id = (int)e, mine = rank(top);
            if ((e & 31) == (uint32_t)lane) {
                if constexpr (!kPacked) taken |= 1u << (e >> 5);
                if (spare) {
                    best = second, best_at = second_at;
                } else {
                    if constexpr (!kPacked) {
#pragma unroll
                        for (int j = 0; j < VPL; ++j)
                            if (taken >> j & 1) key[j] = 0;
                    }
                    look<false>(top);
                }
                spare = !spare;
            }
        }
    }
};

// ONE: the only block, or cluster of blocks, which also places the slots.
template <typename T, int VPL, bool ONE>
__global__ void __launch_bounds__(kRouteThreads)
route_choose_kernel(const __grid_constant__ RouteParams p) {
    __shared__ uint32_t mask[2][kRouteMaxExperts];
    __shared__ uint32_t start[ONE ? kRouteMaxExperts + 1 : 1];
    __shared__ uint32_t cnt[ONE ? kRouteMaxExperts : 1];
    __shared__ uint32_t total_of[ONE ? kRouteMaxExperts : 1];
    __shared__ uint32_t before[ONE ? kRouteMaxExperts : 1];
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
#pragma unroll
        for (int j = 0; j < VPL; ++j) raw[j] = lane + 32 * j < p.E ? row[lane + 32 * j] : T(0.f);
        Choice<T, VPL> choice;
        choice.set(raw, p.E, lane);
        choice.template look<true>(0);
        const uint32_t top = choice.rank(__reduce_max_sync(0xFFFFFFFFu, choice.best));
        const bool any = top > Rank<T>::off;
        const float vmax = Rank<T>::value(top);
        float total = 0.f;
        if (!p.renormalize && any) {
#pragma unroll
            for (int j = 0; j < VPL; ++j)
                if (choice.rank(choice.key[j]) > Rank<T>::off) total += expf((float)raw[j] - vmax);
            total = warp_sum(total);
        }
        int id;
        uint32_t mine;
        choice.choose(p.k, lane, id, mine);
        const float w = id < 0 ? 0.f : expf(Rank<T>::value(mine) - vmax);
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
        if (gridDim.x > 1) tc::cluster_sync();
        else __syncthreads();
        for (int e = threadIdx.x; e < p.E; e += kRouteThreads) {
            uint32_t all = 0, earlier = 0;
            for (uint32_t r = 0; r < gridDim.x; ++r) {
                const uint32_t c = r == blockIdx.x ? cnt[e] : tc::load_cluster(tc::in_block(tc::smem_u32(&cnt[e]), r));
                all += c;
                earlier += r < blockIdx.x ? c : 0;
            }
            total_of[e] = all;
            before[e] = earlier;
        }
        if (gridDim.x > 1) tc::cluster_sync();      // the counts of a block that leaves are read
        else __syncthreads();
        scan_experts(total_of, start, p.E, sums);
        const int first = (int)blockIdx.x * kRouteThreads + threadIdx.x, threads = (int)gridDim.x * kRouteThreads;
        for (int e = first; e <= p.E; e += threads) p.start[e] = (int32_t)start[e];
        for (int i = (int)start[p.E] + first; i < p.T * p.k; i += threads) p.rows[i] = -1;
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
                slot += (int)(start[id] + before[id]);
                p.rows[slot] = t0 + t;
            }
        }
        p.slots[at] = slot;
    }
}

// Exclusive prefix of the blocks' counts per expert: 8 experts a block (32
// bytes of a row of counts), 128 segments of the blocks.
__global__ void __launch_bounds__(1024)
route_scan_kernel(const __grid_constant__ RouteParams p, int blocks) {
    __shared__ uint32_t part[32][8];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int e = blockIdx.x * 8 + (lane & 7), seg = warp * 4 + (lane >> 3);
    const int per = (blocks + 127) / 128, b0 = min(blocks, seg * per), b1 = e < p.E ? min(blocks, b0 + per) : b0;
    uint32_t sum = 0;
#pragma unroll 8
    for (int b = b0; b < b1; ++b) sum += p.counts[(int64_t)b * p.E + e];
    uint32_t upto = sum;
#pragma unroll
    for (int d = 8; d < 32; d <<= 1) {
        const uint32_t o = __shfl_up_sync(0xFFFFFFFFu, upto, d);
        if (lane >= d) upto += o;
    }
    if (lane >= 24) part[warp][lane & 7] = upto;
    __syncthreads();
    uint32_t before = upto - sum;
    for (int w = 0; w < warp; ++w) before += part[w][lane & 7];
    if (seg == 127 && e < p.E) p.totals[e] = before + sum;
#pragma unroll 4
    for (int b = b0; b < b1; ++b) {
        uint32_t *at = p.counts + (int64_t)b * p.E + e;
        const uint32_t c = *at;
        *at = before;
        before += c;
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

template <bool ONE>
using ChooseKernel = void (*)(RouteParams);

template <typename T, bool ONE>
ChooseKernel<ONE> choose_kernel(int E) {
    if (E <= 128) return route_choose_kernel<T, 4, ONE>;
    if (E <= 256) return route_choose_kernel<T, 8, ONE>;
    if (E <= 384) return route_choose_kernel<T, 12, ONE>;
    if (E <= 512) return route_choose_kernel<T, 16, ONE>;
    return route_choose_kernel<T, 32, ONE>;
}

template <bool ONE>
ChooseKernel<ONE> choose_kernel(int dtype, int E) {
    if (dtype == CSF_BF16) return choose_kernel<__nv_bfloat16, ONE>(E);
    if (dtype == CSF_F16) return choose_kernel<__half, ONE>(E);
    return choose_kernel<float, ONE>(E);
}

}  // namespace
}  // namespace csfk

using namespace csfk;

extern "C" size_t csf_route_scratch_bytes(int32_t tokens, int32_t experts) {
    if (tokens <= kRouteTokens * kRouteCluster || experts < 1) return 0;
    const size_t blocks = ((size_t)tokens + kRouteTokens - 1) / kRouteTokens;
    return (size_t)round_up((int64_t)((blocks + 1) * (size_t)experts * 4), 16);
}

extern "C" csf_status csf_route(const csf_route_args *a, void *stream) {
    if (!a || !dtype_known(a->dtype) || a->tokens < 0 || a->experts < 1 || a->k < 1 || a->k > a->experts) return CSF_ERR_ARG;
    if (a->experts > kRouteMaxExperts || a->k > kRouteMaxK) return CSF_ERR_UNSUPPORTED;
    if ((int64_t)a->tokens * a->k >= (1ll << 31)) return CSF_ERR_UNSUPPORTED;
    if (!a->expert_start || !aligned_to(a->expert_start, 4)) return CSF_ERR_ARG;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (a->tokens > 0) {
        if (!a->logits || !a->ids || !a->weights || !a->rows || !a->slots || a->logits_stride < a->experts) return CSF_ERR_ARG;
        if (!aligned_to(a->logits, dtype_bytes(a->dtype))) return CSF_ERR_ARG;
        if (!aligned_to(a->ids, 4) || !aligned_to(a->weights, 4) || !aligned_to(a->rows, 4) || !aligned_to(a->slots, 4)) return CSF_ERR_ARG;
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
    const int blocks = (int)(((int64_t)p.T + kRouteTokens - 1) / kRouteTokens);
    p.totals = static_cast<uint32_t *>(a->scratch);
    p.counts = p.totals + p.E;
    if (p.T == 0) {
        route_none_kernel<<<1, 256, 0, s>>>(p.start, p.E);
    } else if (blocks <= kRouteCluster) {
        unsigned cluster = 1;
        while (cluster < (unsigned)blocks) cluster *= 2;
        cudaLaunchConfig_t config = {};
        config.gridDim = dim3(cluster);
        config.blockDim = dim3(kRouteThreads);
        config.stream = s;
        cudaLaunchAttribute attr;
        attr.id = cudaLaunchAttributeClusterDimension;
        attr.val.clusterDim.x = cluster;
        attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
        config.attrs = &attr;
        config.numAttrs = cluster > 1 ? 1 : 0;
        if (cudaLaunchKernelEx(&config, choose_kernel<true>(a->dtype, p.E), p) != cudaSuccess) {
            cudaGetLastError();
            return CSF_ERR_CUDA;
        }
    } else {
        choose_kernel<false>(a->dtype, p.E)<<<blocks, kRouteThreads, 0, s>>>(p);
        route_scan_kernel<<<(p.E + 7) / 8, 1024, 0, s>>>(p, blocks);
        route_place_kernel<<<blocks, kRouteThreads, 0, s>>>(p);
    }
    return cudaGetLastError() == cudaSuccess ? CSF_OK : CSF_ERR_CUDA;
}
