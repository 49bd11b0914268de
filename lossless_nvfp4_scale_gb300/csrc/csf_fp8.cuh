// Products of FP8 rows with E4M3 weights that have a scale per 128 x 128
// block (csf_fp8_matmul): the kernel.
//
// The slots are the M side, 128 to a block of threads, and the weights' output
// columns the N side.  The 5th-generation tensor cores sum 128 products
// exactly scaled alike at a time, into tensor memory; eight warps then take
// each such partial sum out, multiply it with its row's scale times the weight
// block's and add it up in registers, in 32 bits: lane and register are row
// and column, so the factor is one number a thread and block, and two columns
// go through a multiply-add at once.  Meanwhile the next partial sums form in
// other columns of tensor memory.
//
// Where slots are many, two neighbouring blocks pair up: 256 slots by 256
// columns, each block holding its 128 slots and 128 of the columns, which
// halves what shared memory has to take in per product.  A gated product's
// tile has 128 gate and the 128 up columns of the same numbers, so that both
// lie in one thread.  Where tiles are few, a cluster of 2 to 8 blocks shares
// one: each sums its part of the depth, hands the rows' sums round, and
// finishes its share of the rows.
//
//   warp 0      weights, and x rows where slots are rows (TMA, 128-byte swizzle)
//   warp 1      matrix instructions (the first block's of a pair)
//   warps 2, 3  x rows through the index: 16-byte asynchronous copies,
//               swizzled as TMA would
//   warps 4-11  partial sums, then the epilogue: the sums go back to tensor
//               memory, whose columns a rolled loop can take one by one
#pragma once

#include <cuda.h>

#include "csf_elem.cuh"
#include "csf_grouped.cuh"
#include "csf_internal.cuh"
#include "csf_layer.h"
#include "csf_tc.cuh"

namespace csfk {
namespace f8 {

using mm::Ring;
using mm::Tile;

constexpr int kThreads = 384;
constexpr int kSumWarps = 8, kFirstSumWarp = 4;
constexpr int kMaxStages = 8;
constexpr int kSmemLimit = 227 * 1024;
constexpr int kMaxExperts = 8192;
constexpr int kMaxSplit = 8;
constexpr int kSplitSlots = 64;          // slots of a tile that a cluster shares
constexpr uint32_t kTileBytes = 128 * 128;
constexpr uint32_t kTmemCols = 512;
constexpr int kTurnStride = 36;          // floats between rows of a warp's 32 x 32 piece
constexpr uint32_t kTurnBytes = kSumWarps * 32 * kTurnStride * 4;
// Registers of the warps that copy and of those that sum, where a thread holds
// 128 sums: together what the block was launched with, 384 x 168.
constexpr int kCopyRegs = 72, kSumRegs = 216, kLaunchRegs = 168;
static_assert(128 * kCopyRegs + 256 * kSumRegs == kThreads * kLaunchRegs, "registers of a block");

struct Params {
    const uint8_t *x_codes, *x_scales;
    int64_t x_code_stride, x_scale_stride;
    const int32_t *rows;
    const void *start;
    const float *w_scales;
    int64_t ws_expert;           // floats between experts' scales
    int32_t ws_f, ws_b;          // floats between output blocks, and between summed blocks
    const void *bias;
    const float *row_scale;
    const void *residual;
    int64_t residual_stride;     // elements
    char *out;
    int64_t out_stride;          // bytes
    uint8_t *out_scales;
    int64_t out_scale_stride;
    uint32_t *err;
    int64_t slots;
    int32_t x_rows, es64, E;
    int32_t depth, blocks;       // summed length, and in blocks of 128
    int32_t O, F;                // weight outputs per expert (a bias row), output columns
    int32_t f_blocks;            // blocks of 128 of O
    int32_t row_tiles;           // tiles of O per slot tile
    uint32_t row_tiles_magic;    // 2^32 / row_tiles, rounded up
    int32_t tile_step, second;   // columns of O from a tile to the next, from its first 128 to its second
    int32_t nt;                  // most slots per tile
    int32_t stages;
    uint32_t stage_bytes;
    int32_t act, gated, transposed;
    int32_t bias_dtype, residual_dtype, out_dtype;
    int32_t bias_wide, residual_wide, out_wide;
    int32_t split;               // blocks of a cluster that share a tile's depth
};

struct Shared {
    uint64_t full[kMaxStages], empty[kMaxStages], acc_full[4], acc_empty[4];
    uint32_t tmem, abort, warp_sum[kThreads / 32];
    float amax[2][2][2][128];    // by tile, half, weight block and row
};

__device__ __forceinline__ float activate(float v, int act) {
    if (act == CSF_ACT_SILU || act == CSF_ACT_GELU_TANH) return mm::smooth(v, act == CSF_ACT_GELU_TANH);
    return act == CSF_ACT_RELU && v < 0.f ? 0.f : v;
}

// One slot's columns f .. f+7 of y = act(p): row weight, residual, and out.
// The 16 lanes of a block of 128 columns call it together; `live` ones write.
template <bool QUANT>
__device__ __forceinline__ void finish8(const Params &p, float (&y)[8], int64_t slot, int f, bool live) {
    if (p.row_scale) {
        const float s = live ? __ldg(p.row_scale + slot) : 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) y[i] *= s;
    }
    if (p.residual && live) {
        float r[8];
        const char *row = static_cast<const char *>(p.residual) + slot * p.residual_stride * (p.residual_dtype == CSF_F32 ? 4 : 2);
        elem::to_floats(r, elem::load(row, f, p.F, p.residual_dtype, p.residual_wide), p.residual_dtype);
#pragma unroll
        for (int i = 0; i < 8; ++i) y[i] += r[i];
    }
    char *out = p.out + slot * p.out_stride;
    if constexpr (QUANT) {
#pragma unroll
        for (int i = 0; i < 8; ++i) y[i] = live && f + i < p.F ? y[i] : 0.f;
        const int chunks = ((p.F + 31) & ~31) >> 3, chunk = f >> 3;
        uint8_t *scales = p.out_scales + slot * p.out_scale_stride;
        quant::quantize8<CSF_ROWS_FP8>(y, reinterpret_cast<uint8_t *>(out), scales, chunk, live && chunk < chunks, 1.f);
        if (live && chunk + 1 == chunks) {     // the row's last columns: clear the scale row's padding
            const int n = quant::scale_bytes<CSF_ROWS_FP8>(chunks);
            for (int i = n; i < ((n + 15) & ~15); i += 4) *reinterpret_cast<float *>(scales + i) = 0.f;
        }
    } else {
        if (live && f < p.F) elem::store(out, f, p.F, elem::from_floats(y, p.out_dtype), p.out_dtype, p.out_wide);
    }
}

// 8 columns of an expert's bias from c on, added to y.
__device__ __forceinline__ void add_bias8(const Params &p, float *y, int e, int c) {
    float b[8];
    const char *row = static_cast<const char *>(p.bias) + (int64_t)e * p.O * (p.bias_dtype == CSF_F32 ? 4 : 2);
    elem::to_floats(b, elem::load(row, c, p.O, p.bias_dtype, p.bias_wide), p.bias_dtype);
#pragma unroll
    for (int i = 0; i < 8; ++i) y[i] += b[i];
}

// CTAS: blocks of a pair.  AT: 128-column weight blocks per tile.  ROWS: slot
// s reads row rows[s] of x, else row s.  SPLIT: clusters share a tile's depth.
// QUANT: FP8 rows come out.
template <int CTAS, int AT, bool ROWS, bool SPLIT, bool QUANT>
__global__ void __launch_bounds__(kThreads, 1)
fp8_matmul_kernel(const __grid_constant__ CUtensorMap wmap, const __grid_constant__ CUtensorMap xmap, const __grid_constant__ Params p) {
    static_assert(CTAS == 1 || (AT == 2 && !SPLIT), "a pair has 256 columns and all of the depth");
    extern __shared__ __align__(1024) uint8_t dyn[];
    __shared__ Shared sh;
    constexpr int kSets = (int)kTmemCols / (128 * AT);      // partial sums under way
    constexpr int kWeights = CTAS == 2 ? 1 : AT;            // weight blocks of this block of threads
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const uint32_t ring0 = (tc::smem_u32(dyn) + 1023u) & ~1023u;
    uint8_t *after_ring = dyn + (ring0 - tc::smem_u32(dyn)) + (size_t)p.stages * p.stage_bytes;
    // the epilogue's pieces, or the sums handed round: [from][row][column]
    float *region = reinterpret_cast<float *>(after_ring);
    uint32_t *first = reinterpret_cast<uint32_t *>(after_ring + (SPLIT ? kSplitSlots * AT * 512u : kTurnBytes));
    uint32_t *slot0 = first + p.E + 1;
    const uint32_t rank = CTAS == 2 || SPLIT ? tc::cluster_rank() : 0, split = SPLIT ? (uint32_t)p.split : 1;
    const int pair_rank = CTAS == 2 ? (int)rank : 0;
    const uint32_t full0 = tc::smem_u32(sh.full), empty0 = tc::smem_u32(sh.empty);
    const uint32_t accf0 = tc::smem_u32(sh.acc_full), acce0 = tc::smem_u32(sh.acc_empty);

    if (tid == 0) {
        for (int i = 0; i < p.stages; ++i) {
            tc::bar_init(full0 + 8 * i, ROWS ? 1 + 2 * CTAS : 1);      // the weights; the copying warps
            tc::bar_init(empty0 + 8 * i, 1);
        }
        for (int i = 0; i < kSets; ++i) {
            tc::bar_init(accf0 + 8 * i, 1);
            tc::bar_init(acce0 + 8 * i, kSumWarps * CTAS);
        }
        sh.abort = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 1) tc::tmem_alloc_n<CTAS>(tc::smem_u32(&sh.tmem), kTmemCols);
    bool bad = false;
    const uint32_t running = mm::number_tiles<kThreads>(p, first, slot0, sh.warp_sum, bad);
    if (tid == 0) first[p.E] = running, slot0[p.E] = (uint32_t)mm::start_at(p, p.E);
    tc::fence_before();
    bad = __syncthreads_or(bad);
    tc::fence_after();
    if (bad && p.err && blockIdx.x == 0 && tid == 0) atomicOr(p.err, CSF_DEV_ERR_CORRUPT);
    // An expert_start out of order or range makes no tiles.
    uint32_t total = bad ? 0 : first[p.E] * (uint32_t)p.row_tiles;
    constexpr bool kCluster = CTAS == 2 || SPLIT;
    const uint32_t per = CTAS == 2 ? 2 : split;
    const uint32_t unit = kCluster ? blockIdx.x / per : blockIdx.x, units = kCluster ? gridDim.x / per : gridDim.x;
    if constexpr (SPLIT) total = min(total, units);         // one tile a cluster
    const uint32_t tmem = sh.tmem;
    volatile uint32_t *abort = &sh.abort;
    const int k0 = SPLIT ? (int)(rank * (uint32_t)p.blocks / split) : 0;
    const int k1 = SPLIT ? (int)((rank + 1) * (uint32_t)p.blocks / split) : p.blocks;
    if constexpr (kCluster) tc::cluster_sync();             // the other blocks' barriers are set up

    // This block's slots of a tile.
    auto rows_of = [&](const Tile &t, int r) { return CTAS == 1 ? t.n : max(0, min(128, t.n - 128 * r)); };
    auto stopped = [&]() { return __any_sync(0xFFFFFFFFu, *abort != 0); };

    if (warp < kFirstSumWarp) {
        if constexpr (AT == 2) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kCopyRegs));
        if (warp == 0) {
            // ---- weights, and x rows in order ----
            const bool one = tc::elect_one();
            Ring ring;
            for (uint32_t tile = unit; tile < total && !stopped(); tile += units) {
                const Tile t = mm::find_tile(p, first, slot0, tile, lane);
                if (one) {
                    uint32_t bytes = CTAS * kWeights * kTileBytes;
                    const int n = rows_of(t, pair_rank);
                    if (!ROWS)
                        for (int r = 0; r < CTAS; ++r) bytes += (uint32_t)((rows_of(t, r) + 31) >> 5) * 4096u;
                    const int col = t.rt * p.tile_step + pair_rank * p.second, row = (int)t.slot + 128 * pair_rank;
                    for (int k = k0; k < k1; ++k, ring.next(p.stages)) {
                        if (!tc::bar_wait(empty0 + 8 * ring.s, ring.parity ^ 1u, abort)) break;
                        const uint32_t base = ring0 + ring.s * p.stage_bytes;
                        uint32_t bar = full0 + 8 * ring.s;
                        if (CTAS == 1 || rank == 0) tc::bar_expect(bar, bytes);
                        if (CTAS == 2) bar = tc::in_block(bar, 0);
#pragma unroll
                        for (int b = 0; b < kWeights; ++b) {
                            const int c = col + b * p.second;
                            tc::tma_load_3d_n<CTAS>(base + (1 + b) * kTileBytes, &wmap, p.transposed ? c : k * 128, p.transposed ? k * 128 : c, t.e, bar);
                        }
                        if (!ROWS)
                            for (int c = 0; c < n; c += 32) tc::tma_load_2d_n<CTAS>(base + c * 128u, &xmap, k * 128, row + c, bar);
                    }
                }
                __syncwarp();
            }
        } else if (warp == 1) {
            // ---- matrix instructions ----
            if (rank == 0 || CTAS == 1) {
                if (tc::elect_one()) {
                    // D in 32 bits, E4M3 operands, B's order, N / 8, M / 16
                    const uint32_t idesc = (1u << 4) | (p.transposed ? 1u << 16 : 0) | ((uint32_t)(AT * 128 / 8) << 17) | ((uint32_t)(CTAS * 128 / 16) << 24);
                    const uint32_t b_step = p.transposed ? 4096 >> 4 : 32 >> 4;
                    Ring ring, sets;
                    bool ok = true;
                    for (uint32_t tile = unit; ok && tile < total; tile += units) {
                        for (int k = k0; k < k1; ++k, ring.next(p.stages), sets.next(kSets)) {
                            ok = tc::bar_wait<CTAS == 2>(acce0 + 8 * sets.s, sets.parity ^ 1u, abort) &&
                                 tc::bar_wait<CTAS == 2>(full0 + 8 * ring.s, ring.parity, abort);
                            if (!ok) break;
                            tc::fence_after();
                            const uint32_t base = ring0 + ring.s * p.stage_bytes, d = tmem + sets.s * (AT * 128);
                            const uint64_t ad = tc::desc_sw128(base);
                            const uint64_t bd = p.transposed ? tc::desc_across(base + kTileBytes) : tc::desc_sw128(base + kTileBytes);
#pragma unroll
                            for (uint32_t i = 0; i < 4; ++i) tc::mma_f8<CTAS>(d, ad + 2 * i, bd + b_step * i, idesc, i != 0);
                            tc::commit_n<CTAS>(empty0 + 8 * ring.s);
                            tc::commit_n<CTAS>(accf0 + 8 * sets.s);
                        }
                    }
                }
                __syncwarp();
            }
        } else if constexpr (ROWS) {
            // ---- x rows through the index ----
            const int g = warp - 2, piece = lane & 7, sub = lane >> 3;      // 8 lanes a row, 4 rows a copy, every other 4 rows
            const uint32_t row0 = (uint32_t)(4 * g + sub);
            // row r's 16-byte piece q lies at piece q ^ (r % 8) of its 128 bytes
            const uint32_t dst0 = row0 * 128u + (((uint32_t)piece ^ (row0 & 7)) << 4);
            const int lag = p.stages >= 3 ? 2 : 1;       // copies of that many stages are under way
            int pending = 0;
            Ring ring, done;
            auto signal = [&]() {
                tc::fence_async_proxy();
                __syncwarp();
                if (lane == 0) {
                    if (CTAS == 1) tc::bar_arrive(full0 + 8 * done.s);
                    else tc::bar_arrive_cluster(tc::in_block(full0 + 8 * done.s, 0));
                }
                done.next(p.stages);
                --pending;
            };
            bool ok = true;
            for (uint32_t tile = unit; ok && tile < total; tile += units) {
                const Tile t = mm::find_tile(p, first, slot0, tile, lane);
                const int n = rows_of(t, pair_rank), copies = (n + 7) >> 3;
                int32_t r[16];
#pragma unroll
                for (int j = 0; j < 16; ++j) {
                    r[j] = 0;
                    if (j < copies) {
                        const int32_t v = __ldg(p.rows + (int64_t)t.slot + 128 * pair_rank + min(8 * j + (int)row0, n - 1));
                        r[j] = v < 0 || v >= p.x_rows ? 0 : v;
                    }
                }
                for (int k = k0; k < k1; ++k, ring.next(p.stages)) {
                    ok = __all_sync(0xFFFFFFFFu, tc::bar_wait(empty0 + 8 * ring.s, ring.parity ^ 1u, abort));
                    if (!ok) break;
                    const uint32_t dst = ring0 + ring.s * p.stage_bytes + dst0;
                    const int at = k * 128 + 16 * piece;
                    const bool live = at < p.depth;
                    const uint8_t *src = p.x_codes + (live ? at : 0);
#pragma unroll
                    for (int j = 0; j < 16; ++j)
                        if (j < copies) tc::cp_async16(dst + j * 1024u, src + r[j] * p.x_code_stride, live);
                    tc::cp_async_group();
                    if (++pending > lag) {
                        if (lag == 2) tc::cp_async_wait<2>();
                        else tc::cp_async_wait<1>();
                        signal();
                    }
                }
            }
            tc::cp_async_wait<0>();
            while (pending > 0) signal();
        }
    } else {
        // ---- partial sums and the epilogue ----
        if constexpr (AT == 2) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSumRegs));
        const int w = warp & 3, half = (warp - kFirstSumWarp) >> 2;        // lanes 32 w .., columns 64 half .. of each weight block
        float *buf = region + (warp - kFirstSumWarp) * 32 * kTurnStride;
        const uint32_t mine = tmem + ((uint32_t)(32 * w) << 16) + 64 * half;
        const int part = lane & 3, sub = lane >> 2;                         // after the turn: 8 columns of a row
        // What a tile's first sums need, fetched before the last tile's epilogue.
        struct Head {
            Tile t;
            const float4 *xs;
            const float *ws[AT];
            float4 x0, x1;               // the row's scales of 4 blocks, and of the next 4
            float w0[AT], w1[AT];        // a lane's block of 32, and of the next 32
        };
        bool bad_row = false;
        auto open = [&](Head &h, uint32_t tile) {
            h.t.n = 0;
            if (tile >= total) return;
            h.t = mm::find_tile(p, first, slot0, tile, lane);
            const int r = 128 * pair_rank + 32 * w + lane;
            const int64_t slot = (int64_t)h.t.slot + min(r, h.t.n - 1);
            int64_t row = slot;
            if constexpr (ROWS) {
                row = __ldg(p.rows + slot);
                const bool out = row < 0 || row >= p.x_rows;
                bad_row |= out;
                if (out) row = 0;
            }
            h.xs = reinterpret_cast<const float4 *>(p.x_scales + row * p.x_scale_stride);
            const int last = (p.blocks - 1) >> 2;
            h.x0 = __ldg(h.xs + (k0 >> 2));
            h.x1 = __ldg(h.xs + min((k0 >> 2) + 1, last));
#pragma unroll
            for (int a = 0; a < AT; ++a) {
                const int f = min((h.t.rt * p.tile_step + a * p.second) >> 7, p.f_blocks - 1);
                h.ws[a] = p.w_scales + h.t.e * p.ws_expert + (int64_t)f * p.ws_f;
                h.w0[a] = __ldg(h.ws[a] + (int64_t)min(k0 + lane, p.blocks - 1) * p.ws_b);
                h.w1[a] = k1 - k0 > 32 ? __ldg(h.ws[a] + (int64_t)min(k0 + 32 + lane, p.blocks - 1) * p.ws_b) : 0.f;
            }
        };
        Ring sets;
        Head h;
        open(h, unit);
        bool ok = true;
        for (uint32_t tile = unit, nth = 0; tile < total; tile += units, ++nth) {
            const Tile t = h.t;
            const int n = rows_of(t, pair_rank) - 32 * w;       // this warp's rows, if any
            uint64_t sum[AT][32];
#pragma unroll
            for (int a = 0; a < AT; ++a)
#pragma unroll
                for (int i = 0; i < 32; ++i) sum[a][i] = 0;
            const int groups = (p.blocks + 3) >> 2;
            for (int k = k0; k < k1; ++k) {
                ok = __all_sync(0xFFFFFFFFu, tc::bar_wait(accf0 + 8 * sets.s, sets.parity, abort));
                if (!ok) break;
                tc::fence_after();
                if (n > 0) {
                    const int q = k & 3, i = (k - k0) & 31;
                    const float xs = q < 2 ? (q == 0 ? h.x0.x : h.x0.y) : (q == 2 ? h.x0.z : h.x0.w);
                    uint64_t factor[AT];
#pragma unroll
                    for (int a = 0; a < AT; ++a) {
                        const uint32_t f = __float_as_uint(xs * __shfl_sync(0xFFFFFFFFu, h.w0[a], i));
                        factor[a] = tc::pack2(f, f);
                    }
                    if (q == 3) {
                        h.x0 = h.x1;
                        if ((k >> 2) + 2 < groups) h.x1 = __ldg(h.xs + (k >> 2) + 2);
                    }
                    if (i == 31) {
#pragma unroll
                        for (int a = 0; a < AT; ++a) {
                            h.w0[a] = h.w1[a];
                            h.w1[a] = __ldg(h.ws[a] + (int64_t)min(k + 33 + lane, p.blocks - 1) * p.ws_b);
                        }
                    }
                    const uint32_t d = mine + sets.s * (AT * 128);
                    uint32_t v[2][32];
                    tc::tmem_load(d, v[0]);
#pragma unroll
                    for (int c = 0; c < 2 * AT; ++c) {
                        tc::wait_ld(v[c & 1]);
                        if (c + 1 < 2 * AT) tc::tmem_load(d + ((c + 1) >> 1) * 128 + ((c + 1) & 1) * 32, v[(c + 1) & 1]);
#pragma unroll
                        for (int j = 0; j < 16; ++j) tc::fma2(sum[c >> 1][(c & 1) * 16 + j], tc::pack2(v[c & 1][2 * j], v[c & 1][2 * j + 1]), factor[c >> 1]);
                    }
                }
                if (k + 1 < k1 || SPLIT) {
                    tc::fence_before();
                    __syncwarp();
                    if (lane == 0) {
                        if (CTAS == 1) tc::bar_arrive(acce0 + 8 * sets.s);
                        else tc::bar_arrive_cluster(tc::in_block(acce0 + 8 * sets.s, 0));
                    }
                    sets.next(kSets);
                }
            }
            if (!ok) break;
            if constexpr (SPLIT) {
                // a row's sums to the block that finishes it
                const uint32_t share = ((uint32_t)t.n + split - 1) / split, r = (uint32_t)(32 * w + lane);
                if (lane < n) {
                    const uint32_t to = r / share;
                    const uint32_t at = tc::in_block(tc::smem_u32(region + ((rank * share + (r - to * share)) * AT) * 128 + 64 * half), to);
#pragma unroll
                    for (int a = 0; a < AT; ++a)
#pragma unroll
                        for (int j = 0; j < 32; j += 2) {
                            uint32_t v[4];
                            tc::unpack2(sum[a][j], v[0], v[1]);
                            tc::unpack2(sum[a][j + 1], v[2], v[3]);
                            tc::store_cluster4(at + a * 512u + j * 8u, v[0], v[1], v[2], v[3]);
                        }
                }
                break;
            }
            // The sums, back to where the last partial ones were.
            const uint32_t d = mine + sets.s * (AT * 128);
            if (n > 0) {
#pragma unroll
                for (int a = 0; a < AT; ++a)
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        uint32_t v[16];
#pragma unroll
                        for (int j = 0; j < 8; ++j) tc::unpack2(sum[a][c * 8 + j], v[2 * j], v[2 * j + 1]);
                        tc::tmem_store(d + a * 128 + c * 16, v);
                    }
                tc::wait_st();
            }
            open(h, tile + units);
            if (n > 0) {
                const int64_t slot = (int64_t)t.slot + 128 * pair_rank + 32 * w;
                const int outs = p.gated ? 1 : AT, f_tile = t.rt * p.tile_step + 64 * half;
                // 16 columns of y from f on, this lane's row: d's columns are c on
                auto values = [&](float (&y)[16], int c, int f) {
                    uint32_t v[16];
                    tc::tmem_load(d + c, v);
                    if (AT == 2 && p.gated) {
                        uint32_t u[16];
                        tc::tmem_load(d + 128 + c, u);
                        tc::wait_ld(v);
                        tc::wait_ld(u);
                        float up[16];
#pragma unroll
                        for (int i = 0; i < 16; ++i) y[i] = __uint_as_float(v[i]), up[i] = __uint_as_float(u[i]);
                        if (p.bias) {
                            add_bias8(p, y, t.e, f);
                            add_bias8(p, y + 8, t.e, f + 8);
                            add_bias8(p, up, t.e, p.F + f);
                            add_bias8(p, up + 8, t.e, p.F + f + 8);
                        }
#pragma unroll
                        for (int i = 0; i < 16; ++i) y[i] = activate(y[i], p.act) * up[i];
                    } else {
                        tc::wait_ld(v);
#pragma unroll
                        for (int i = 0; i < 16; ++i) y[i] = __uint_as_float(v[i]);
                        if (p.bias) {
                            add_bias8(p, y, t.e, f);
                            add_bias8(p, y + 8, t.e, f + 8);
                        }
                        if (p.act != CSF_ACT_NONE) {
#pragma unroll
                            for (int i = 0; i < 16; ++i) y[i] = activate(y[i], p.act);
                        }
                    }
                };
                if constexpr (!QUANT) {
#pragma unroll 1
                    for (int piece = 0; piece < 2 * outs; ++piece) {
                        const int c = (piece >> 1) * 128 + (piece & 1) * 32, f = f_tile + c;
                        if (f >= p.F) continue;
#pragma unroll 1
                        for (int q = 0; q < 32; q += 16) {
                            float y[16];
                            values(y, c + q, f + q);
#pragma unroll
                            for (int i = 0; i < 16; i += 4)
                                *reinterpret_cast<float4 *>(buf + lane * kTurnStride + q + i) = make_float4(y[i], y[i + 1], y[i + 2], y[i + 3]);
                        }
                        __syncwarp();
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const int r = 8 * i + sub;
                            const float4 *from = reinterpret_cast<const float4 *>(buf + r * kTurnStride + 8 * part);
                            const float4 lo = from[0], hi = from[1];
                            float y[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
                            finish8<false>(p, y, slot + r, f + 8 * part, r < n);
                        }
                        __syncwarp();
                    }
                } else {
                    // The largest magnitude of a block of 128 columns comes from
                    // both warps of these rows.
                    const int padded = (p.F + 31) & ~31;
                    const bool live = lane < n;
                    const float rs = p.row_scale && live ? __ldg(p.row_scale + slot + lane) : 1.f;
                    const char *res = p.residual ? static_cast<const char *>(p.residual) + (slot + (live ? lane : 0)) * p.residual_stride * (p.residual_dtype == CSF_F32 ? 4 : 2) : nullptr;
                    float (&amax)[2][2][128] = sh.amax[nth & 1];
                    for (int a = 0; a < outs; ++a) {
                        uint32_t m = 0;
#pragma unroll 1
                        for (int q = 0; q < 64; q += 16) {
                            const int c = a * 128 + q, f = f_tile + c;
                            if (f >= padded) break;
                            float y[16];
                            values(y, c, f);
                            uint32_t v[16];
                            if (p.row_scale) {
#pragma unroll
                                for (int i = 0; i < 16; ++i) y[i] *= rs;
                            }
                            if (res) {
                                float b[8];
#pragma unroll
                                for (int g = 0; g < 16; g += 8) {
                                    elem::to_floats(b, elem::load(res, f + g, p.F, p.residual_dtype, p.residual_wide), p.residual_dtype);
#pragma unroll
                                    for (int i = 0; i < 8; ++i) y[g + i] += b[i];
                                }
                            }
#pragma unroll
                            for (int i = 0; i < 16; ++i) {
                                v[i] = f + i < p.F ? __float_as_uint(y[i]) : 0;
                                m = max(m, v[i] & 0x7FFFFFFFu);
                            }
                            tc::tmem_store(d + c, v);
                        }
                        amax[half][a][32 * w + lane] = __uint_as_float(m);
                    }
                    tc::wait_st();
                    tc::named_sync(1 + w, 64);
                    for (int a = 0; a < outs; ++a) {
                        const int f = f_tile + a * 128;
                        if (f >= padded) break;
                        const uint32_t m = max(__float_as_uint(amax[0][a][32 * w + lane]), __float_as_uint(amax[1][a][32 * w + lane]));
                        const float scale = quant::fp8_scale(m), up = quant::fp8_up(scale);
                        const quant::Whole whole = quant::fp8_whole(scale * up);
#pragma unroll 1
                        for (int q = 0; q < 64; q += 16) {
                            if (f + q >= padded) break;
                            uint32_t v[16];
                            tc::tmem_load(d + a * 128 + q, v);
                            tc::wait_ld(v);
                            uint32_t o[4];
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                float y[4];
#pragma unroll
                                for (int j = 0; j < 4; ++j) y[j] = quant::over(__uint_as_float(v[4 * i + j]) * up, whole);
                                o[i] = quant::e4m3x2(y[0], y[1]) | quant::e4m3x2(y[2], y[3]) << 16;
                            }
                            *reinterpret_cast<uint4 *>(buf + lane * 20 + (q >> 2)) = make_uint4(o[0], o[1], o[2], o[3]);
                        }
                        __syncwarp();
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const int r = 8 * i + sub;
                            if (r < n && f + 16 * part < padded)
                                *reinterpret_cast<uint4 *>(p.out + (slot + r) * p.out_stride + f + 16 * part) =
                                    *reinterpret_cast<const uint4 *>(buf + r * 20 + 4 * part);
                        }
                        __syncwarp();
                        if (half == 0 && live) {
                            float *scales = reinterpret_cast<float *>(p.out_scales + (slot + lane) * p.out_scale_stride);
                            const int b = f >> 7, n_blocks = (p.F + 127) >> 7;
                            scales[b] = scale;
                            if (b + 1 == n_blocks)       // clear the scale row's padding
                                for (int i = n_blocks; i & 3; ++i) scales[i] = 0.f;
                        }
                    }
                }
            }
            tc::fence_before();
            __syncwarp();
            if (lane == 0) {
                if (CTAS == 1) tc::bar_arrive(acce0 + 8 * sets.s);
                else tc::bar_arrive_cluster(tc::in_block(acce0 + 8 * sets.s, 0));
            }
            sets.next(kSets);
        }
        if (bad_row && p.err) atomicOr(p.err, CSF_DEV_ERR_CORRUPT);
    }

    tc::fence_before();      // the last tensor-memory reads, before they are freed
    __syncthreads();
    tc::fence_after();
    if (sh.abort) {
        // A wait that gave up: let copies and products in flight land before
        // the block's memory goes.
        if (tid == 0 && p.err) atomicOr(p.err, CSF_DEV_ERR_TIMEOUT);
        const uint64_t t0 = tc::timer_ns();
        while (tc::timer_ns() - t0 < 5000000ull) __nanosleep(1000);
        __syncthreads();
    }
    if constexpr (kCluster) tc::cluster_sync();      // the sums have come; nothing is under way to a block that leaves
    if constexpr (SPLIT) {
        if (unit < total && !sh.abort) {
            const Tile t = mm::find_tile(p, first, slot0, unit, lane);
            const int share = (t.n + (int)split - 1) / (int)split, rows = min(share, t.n - (int)rank * share);
            const int f = t.rt * p.tile_step + 8 * (lane & 15);
            for (int r0 = 2 * warp; r0 < rows; r0 += 2 * (kThreads / 32)) {
                const int r = r0 + (lane >> 4);
                const bool live = r < rows;
                float y[AT][8] = {};
                for (uint32_t from = 0; from < split; ++from) {
#pragma unroll
                    for (int a = 0; a < AT; ++a) {
                        const float4 *at = reinterpret_cast<const float4 *>(region + ((from * share + (live ? r : r0)) * AT + a) * 128 + 8 * (lane & 15));
                        const float4 lo = at[0], hi = at[1];
                        const float v[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
#pragma unroll
                        for (int i = 0; i < 8; ++i) y[a][i] += v[i];
                    }
                }
                if (p.bias) {
                    add_bias8(p, y[0], t.e, f);
                    if (AT == 2) add_bias8(p, y[AT - 1], t.e, p.F + f);
                }
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    y[0][i] = activate(y[0][i], p.act);
                    if (AT == 2) y[0][i] *= y[AT - 1][i];       // gated
                }
                finish8<QUANT>(p, y[0], (int64_t)t.slot + (int64_t)rank * share + r, f, live);
            }
        }
    }
    if (warp == 1) tc::tmem_free_n<CTAS>(tmem, kTmemCols);
}

using Kernel = void (*)(CUtensorMap, CUtensorMap, Params);

// A pair, one block of 128 or 256 columns, or those with the depth shared.
enum Shape { kPair = 0, kOne = 1, kTwo = 2, kOneShared = 3, kTwoShared = 4 };

template <bool ROWS, bool QUANT>
Kernel pick(int shape) {
    switch (shape) {
        case kPair: return fp8_matmul_kernel<2, 2, ROWS, false, QUANT>;
        case kOne: return fp8_matmul_kernel<1, 1, ROWS, false, QUANT>;
        case kTwo: return fp8_matmul_kernel<1, 2, ROWS, false, QUANT>;
        case kOneShared: return fp8_matmul_kernel<1, 1, ROWS, true, QUANT>;
        default: return fp8_matmul_kernel<1, 2, ROWS, true, QUANT>;
    }
}

// The kernel of a shape, one translation unit each for x rows in order and
// through an index.
Kernel rows_in_order(int shape, bool quant);
Kernel rows_by_index(int shape, bool quant);

}  // namespace f8
}  // namespace csfk
