// Products of FP8 rows with E4M3 weights that have a scale per 128 x 128
// block (csf_fp8_matmul): the kernel.
//
// The slots are the M side, 128 to a block of threads, and the weights' output
// columns the N side.  The 5th-generation tensor cores form the partial sum of
// a block of 128 of the depth, whose products are all scaled alike, in tensor
// memory; eight warps then take it out, multiply it with its row's scale times
// the weight block's and add it up in registers, in 32 bits.  Lane and
// register are row and column, so the factor is one number a thread.  Tensor
// memory holds four partial sums of 128 columns: two steps of the depth are
// under way while one is taken out.
//
// A tile is 128 slots by 128 or 256 columns.  A gated product's tile has 128
// gate columns and the 128 up columns of the same numbers.  Where tiles are
// few, a cluster of 2 to 8 blocks shares one: each sums its part of the depth,
// hands the rows' sums round, and finishes its share of the rows.
//
// (Tiles of 256 by 256 on two neighbouring blocks, whose instructions one block
// issues, halve what shared memory has to take in per product, which is not
// the bound.  With factors and arrivals that pass between the blocks in order,
// they took 193 us for the first line below and 215 for the second.)
//
// What bounds it: taking the partial sums out.  A step of 256 columns takes
// the matrix instructions 0.26 us (0.32 with their copies), the eight warps
// 0.34 alone, both together 0.44: a load of 64 columns from tensor memory is
// 160 to 190 cycles under way, twice a step, and 128 sums leave registers for
// no more in flight.  Measured (2070 MHz):
//   8191 slots, 5120 x 5120, bfloat16 out           193 us, 2.23 PFLOP/s
//     with a residual and row weights               215 us
//   32768 slots on 128 experts, gated 4096 x 2048   403 us to bfloat16, 440 to
//     FP8: 2.5 tiles of 128 slots an expert of 256, the SiLU
//   4000 slots on 64 experts, 1600 x 2048 across    51 us, 4.6 TB/s
//   64 slots on 8 of 128 experts, gated 1024 x 1600 14.8 us: latency
//   one slot of 2048 x 5120, of 4096 x 5120 gated   9.7, 14.6 us: latency
// What that took: waits whose ready path has no taken branch (180 -> 57
// cycles); issue code that the whole warp runs, with one lane's predicate on
// the instructions; partial sums a weight block each; packed multiply-adds; the
// factors by warps of their own, for the registers.
//
//   warp 0      weights, and x rows where slots are rows (TMA, 128-byte swizzle)
//   warp 1      matrix instructions
//   warps 2, 3  the factors, a step's 128 rows at a time, into shared memory
//   warps 4-7   x rows through an index, where there is one: 16-byte
//               asynchronous copies, swizzled as TMA would
//   the last 8  partial sums, then the epilogue: the sums go back to tensor
//               memory, whose columns a rolled loop can take one by one
#pragma once

#include <cuda.h>

#include "csf_elem.cuh"
#include "csf_fp8_plan.h"
#include "csf_grouped.cuh"
#include "csf_internal.cuh"
#include "csf_layer.h"
#include "csf_tc.cuh"

namespace csfk {
namespace f8 {

using mm::Ring;
using mm::Tile;

constexpr int kFactorWarps = 2, kFirstFactorWarp = 2;      // 64 rows each
constexpr int kXWarps = 4, kFirstXWarp = 4;                // 32 rows each, where an index is followed
__host__ __device__ constexpr int threads_of(bool rows) { return rows ? 512 : 384; }
constexpr uint32_t kTmemCols = 512;
// Registers of the warps that copy and of those that sum, where a thread holds
// 128 sums and takes out 64 or 32 partial ones: together what the block was
// launched with.
__host__ __device__ constexpr int launch_regs(bool rows) { return rows ? 128 : 168; }
template <bool ROWS> constexpr int kCopyRegs = ROWS ? 48 : 56;
template <bool ROWS> constexpr int kSumRegs = ROWS ? 208 : 224;
static_assert(256 * kCopyRegs<true> + 256 * kSumRegs<true> == 512 * launch_regs(true), "registers of a block");
static_assert(128 * kCopyRegs<false> + 256 * kSumRegs<false> == 384 * launch_regs(false), "registers of a block");

struct Params {
    const uint8_t *x_codes, *x_scales;
    int64_t x_code_stride, x_scale_stride;
    const int32_t *rows;
    const void *start;
    const float *w_scales;
    int32_t ws_expert, ws_f, ws_b;   // floats between experts' scales, output blocks, summed blocks
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

__device__ __forceinline__ float activate(float v, int act) {
    if (act == CSF_ACT_SILU || act == CSF_ACT_GELU_TANH) return mm::smooth(v, act == CSF_ACT_GELU_TANH);
    return act == CSF_ACT_RELU && v < 0.f ? 0.f : v;
}

__device__ __forceinline__ void activate32(float (&y)[32], int act) {
    if (act == CSF_ACT_NONE) return;
    if (act == CSF_ACT_RELU) {
#pragma unroll
        for (int i = 0; i < 32; ++i) y[i] = y[i] < 0.f ? 0.f : y[i];
    } else if (act == CSF_ACT_SILU) {
#pragma unroll
        for (int i = 0; i < 32; ++i) y[i] = mm::smooth(y[i], false);
    } else {
#pragma unroll
        for (int i = 0; i < 32; ++i) y[i] = mm::smooth(y[i], true);
    }
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
        elem::to_floats(r, elem::load_apart(row, f, p.F, p.residual_dtype, p.residual_wide), p.residual_dtype);
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
        if (live && f < p.F) elem::store_apart(out, f, p.F, elem::from_floats(y, p.out_dtype), p.out_dtype, p.out_wide);
    }
}

// 8 columns of an expert's bias from c on, added to y.
__device__ __forceinline__ void add_bias8(const Params &p, float *y, int e, int c) {
    float b[8];
    const char *row = static_cast<const char *>(p.bias) + (int64_t)e * p.O * (p.bias_dtype == CSF_F32 ? 4 : 2);
    elem::to_floats(b, elem::load_apart(row, c, p.O, p.bias_dtype, p.bias_wide), p.bias_dtype);
#pragma unroll
    for (int i = 0; i < 8; ++i) y[i] += b[i];
}

// What comes out: 16-bit rows, any plain rows, FP8 rows, 16-bit rows with a
// 16-bit residual (both in whole 16-byte pieces).  Kernels of their own, since
// what one holds in registers another would spill.
enum Mode { kHalves = 0, kPlain = 1, kQuant = 2, kHalvesSum = 3 };

// AT: 128-column weight blocks per tile.  ROWS: slot s reads row rows[s] of x,
// else row s.  SPLIT: clusters share a tile's depth.  MODE: what comes out.
template <int AT, bool ROWS, bool SPLIT, int MODE>
__global__ void __launch_bounds__(threads_of(ROWS), 1)
fp8_matmul_kernel(const __grid_constant__ CUtensorMap wmap, const __grid_constant__ CUtensorMap xmap, const __grid_constant__ Params p) {
    extern __shared__ __align__(1024) uint8_t dyn[];
    __shared__ Shared sh;
    __shared__ float factors[kFactorSteps][AT][128];        // a row's scale times the weight block's
    constexpr int kThreads = threads_of(ROWS), kFirstSumWarp = ROWS ? 8 : 4;
    constexpr int kSets = (int)kTmemCols / 128;             // partial sums of 128 columns under way
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const uint32_t ring0 = (tc::smem_u32(dyn) + 1023u) & ~1023u;
    uint8_t *after_ring = dyn + (ring0 - tc::smem_u32(dyn)) + (size_t)p.stages * p.stage_bytes;
    // the epilogue's pieces, or the sums handed round: [from][row][column]
    float *region = reinterpret_cast<float *>(after_ring);
    uint32_t *first = reinterpret_cast<uint32_t *>(after_ring + (SPLIT ? kSplitSlots * AT * 512u : kTurnBytes));
    uint32_t *slot0 = first + p.E + 1;
    const uint32_t rank = SPLIT ? tc::cluster_rank() : 0, split = SPLIT ? (uint32_t)p.split : 1;
    const uint32_t full0 = tc::smem_u32(sh.full), empty0 = tc::smem_u32(sh.empty);
    const uint32_t accf0 = tc::smem_u32(sh.acc_full), acce0 = tc::smem_u32(sh.acc_empty);

    if (tid == 0) {
        for (int i = 0; i < p.stages; ++i) {
            // the weights, the factors, the copying lanes
            tc::bar_init(full0 + 8 * i, 1 + kFactorWarps + (ROWS ? 32 * kXWarps : 0));
            tc::bar_init(empty0 + 8 * i, 1);
        }
        for (int i = 0; i < kSets; ++i) {
            tc::bar_init(accf0 + 8 * i, 1);
            tc::bar_init(acce0 + 8 * i, kSumWarps / AT);
        }
        sh.abort = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 1) tc::tmem_alloc(tc::smem_u32(&sh.tmem), kTmemCols);
    bool bad = false;
    const uint32_t running = mm::number_tiles<kThreads>(p, first, slot0, sh.warp_sum, bad);
    if (tid == 0) first[p.E] = running, slot0[p.E] = (uint32_t)mm::start_at(p, p.E);
    tc::fence_before();
    bad = __syncthreads_or(bad);
    tc::fence_after();
    if (bad && p.err && blockIdx.x == 0 && tid == 0) atomicOr(p.err, CSF_DEV_ERR_CORRUPT);
    // An expert_start out of order or range makes no tiles.
    uint32_t total = bad ? 0 : first[p.E] * (uint32_t)p.row_tiles;
    const uint32_t unit = SPLIT ? blockIdx.x / split : blockIdx.x, units = SPLIT ? gridDim.x / split : gridDim.x;
    if constexpr (SPLIT) total = min(total, units);         // one tile a cluster
    const uint32_t tmem = sh.tmem;
    volatile uint32_t *abort = &sh.abort;
    const int k0 = SPLIT ? (int)(rank * (uint32_t)p.blocks / split) : 0;
    const int k1 = SPLIT ? (int)((rank + 1) * (uint32_t)p.blocks / split) : p.blocks;
    if constexpr (SPLIT) tc::cluster_sync();                // the other blocks have begun

    if (warp < kFirstSumWarp) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kCopyRegs<ROWS>));
        if (warp == 0) {
            // ---- weights, and x rows in order ----
            const uint32_t one = tc::elect_one();
            Ring ring;
            bool ok = true;
#pragma unroll 1
            for (uint32_t tile = unit; ok && tile < total; tile += units) {
                const Tile t = mm::find_tile(p, first, slot0, tile, lane);
                const uint32_t bytes = AT * kTileBytes + (ROWS ? 0 : (uint32_t)((t.n + 31) >> 5) * 4096u);
                const int col = t.rt * p.tile_step, row = (int)t.slot;
#pragma unroll 1
                for (int k = k0; k < k1; ++k, ring.next(p.stages)) {
                    ok = __all_sync(0xFFFFFFFFu, tc::bar_wait_ready(empty0 + 8 * ring.s, ring.parity ^ 1u, abort));
                    if (!ok) break;
                    const uint32_t base = ring0 + ring.s * p.stage_bytes, bar = full0 + 8 * ring.s;
                    tc::bar_expect_if(one, bar, bytes);
#pragma unroll
                    for (int a = 0; a < AT; ++a) {
                        const int c = col + a * p.second;
                        tc::tma_load_3d_if(one, base + kTileBytes + a * kTileBytes, &wmap, p.transposed ? c : k * 128, p.transposed ? k * 128 : c, t.e, bar);
                    }
                    if (!ROWS) {
#pragma unroll
                        for (int c = 0; c < 128; c += 32)
                            if (c < t.n) tc::tma_load_2d_if(one, base + c * 128u, &xmap, k * 128, row + c, bar);
                    }
                }
            }
        } else if (warp == 1) {
            // ---- matrix instructions ----
            const uint32_t one = tc::elect_one();
            // D in 32 bits, E4M3 operands, B's order, N / 8, M / 16
            const uint32_t idesc = (1u << 4) | (p.transposed ? 1u << 16 : 0) | ((128u / 8) << 17) | ((128u / 16) << 24);
            const uint32_t b_step = (p.transposed ? 4096 : 32) >> 4;
            const uint64_t a0 = tc::desc_sw128(ring0);
            const uint64_t b0 = p.transposed ? tc::desc_across(ring0 + kTileBytes) : tc::desc_sw128(ring0 + kTileBytes);
            const uint32_t a_hi = (uint32_t)(a0 >> 32), b_hi = (uint32_t)(b0 >> 32), stage = p.stage_bytes >> 4;
            Ring ring;
            uint32_t count = 0;      // steps of the depth so far: AT sets each
            bool ok = true;
#pragma unroll 1
            for (uint32_t tile = unit; ok && tile < total; tile += units) {
#pragma unroll 1
                for (int k = k0; k < k1; ++k, ++count, ring.next(p.stages)) {
                    const uint32_t set = AT == 2 ? (count & 1) * 2 : count & 3, parity = ~(count >> (AT == 2 ? 1 : 2)) & 1;
                    const uint32_t acce = acce0 + 8 * set, accf = accf0 + 8 * set, full = full0 + 8 * ring.s;
                    bool here = tc::bar_try(full, ring.parity);
                    here &= tc::bar_try(acce, parity);
                    if (!__all_sync(0xFFFFFFFFu, here)) {
                        ok = __all_sync(0xFFFFFFFFu, tc::bar_wait_on(full, ring.parity, abort) && tc::bar_wait_on(acce, parity, abort));
                        if (!ok) break;
                    }
                    tc::fence_after();
                    if (ROWS) tc::fence_async_proxy();       // x came by ordinary copies
                    const uint32_t at = ring.s * stage, a_lo = (uint32_t)a0 + at, b_lo = (uint32_t)b0 + at, d = tmem + set * 128;
                    tc::mma_f8_128(one, d, a_lo, a_hi, b_lo, b_hi, b_step, idesc, accf);
                    if constexpr (AT == 2) {
                        if (!__all_sync(0xFFFFFFFFu, tc::bar_try(acce + 8, parity))) {
                            ok = __all_sync(0xFFFFFFFFu, tc::bar_wait_on(acce + 8, parity, abort));
                            if (!ok) break;
                        }
                        tc::fence_after();
                        tc::mma_f8_128(one, d + 128, a_lo, a_hi, b_lo + (kTileBytes >> 4), b_hi, b_step, idesc, accf + 8);
                    }
                    tc::commit_if(one, empty0 + 8 * ring.s);
                }
            }
        } else if (warp < kFirstXWarp) {
            // ---- factors ----
            // Two rows a lane; a row's scales of 4 blocks and of the next 4, and of each weight block a lane's block
            // of 32 and of the next 32.
            const int r0 = 64 * (warp - kFirstFactorWarp) + lane, groups = (p.blocks + 3) >> 2;
            uint32_t count = 0;
            bool ok = true, bad_row = false;
            Ring ring;
#pragma unroll 1
            for (uint32_t tile = unit; ok && tile < total; tile += units) {
                const Tile t = mm::find_tile(p, first, slot0, tile, lane);
                const float4 *xs[2];
                float4 x0[2], x1[2];
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const int64_t slot = (int64_t)t.slot + min(r0 + 32 * j, t.n - 1);
                    int64_t row = slot;
                    if constexpr (ROWS) {
                        row = __ldg(p.rows + slot);
                        const bool out = row < 0 || row >= p.x_rows;
                        bad_row |= out;
                        if (out) row = 0;
                    }
                    xs[j] = reinterpret_cast<const float4 *>(p.x_scales + row * p.x_scale_stride);
                    x0[j] = __ldg(xs[j] + (k0 >> 2));
                    x1[j] = __ldg(xs[j] + min((k0 >> 2) + 1, groups - 1));
                }
                const float *ws[AT];
                float w0[AT], w1[AT];
#pragma unroll
                for (int a = 0; a < AT; ++a) {
                    const int f = min((t.rt * p.tile_step + a * p.second) >> 7, p.f_blocks - 1);
                    ws[a] = p.w_scales + t.e * p.ws_expert + (int64_t)f * p.ws_f;
                    w0[a] = __ldg(ws[a] + (int64_t)min(k0 + lane, p.blocks - 1) * p.ws_b);
                    w1[a] = __ldg(ws[a] + (int64_t)min(k0 + 32 + lane, p.blocks - 1) * p.ws_b);
                }
#pragma unroll 1
                for (int k = k0; k < k1; ++k, ++count, ring.next(p.stages)) {
                    const int q = k & 3, i = (k - k0) & 31;
                    float *at = &factors[count % kFactorSteps][0][r0];
                    ok = __all_sync(0xFFFFFFFFu, tc::bar_wait_ready(empty0 + 8 * ring.s, ring.parity ^ 1u, abort));
                    if (!ok) break;
#pragma unroll
                    for (int a = 0; a < AT; ++a) {
                        const float w = __shfl_sync(0xFFFFFFFFu, w0[a], i);
#pragma unroll
                        for (int j = 0; j < 2; ++j)
                            at[a * 128 + 32 * j] = w * (q < 2 ? (q == 0 ? x0[j].x : x0[j].y) : (q == 2 ? x0[j].z : x0[j].w));
                    }
                    __syncwarp();
                    tc::bar_arrive_if(full0 + 8 * ring.s, lane == 0);
                    if (q == 3) {
#pragma unroll
                        for (int j = 0; j < 2; ++j) {
                            x0[j] = x1[j];
                            x1[j] = __ldg(xs[j] + min((k >> 2) + 2, groups - 1));
                        }
                    }
                    if (i == 31) {
#pragma unroll
                        for (int a = 0; a < AT; ++a) {
                            w0[a] = w1[a];
                            w1[a] = __ldg(ws[a] + (int64_t)min(k + 33 + lane, p.blocks - 1) * p.ws_b);
                        }
                    }
                }
            }
            if (bad_row && p.err) atomicOr(p.err, CSF_DEV_ERR_CORRUPT);
        } else if constexpr (ROWS) {
            // ---- x rows through the index ----
            const int g = warp - kFirstXWarp, piece = lane & 7, sub = lane >> 3;      // 8 lanes a row, 4 rows a copy, every fourth 4 rows
            const uint32_t row0 = (uint32_t)(4 * g + sub);
            // row r's 16-byte piece q lies at piece q ^ (r % 8) of its 128 bytes
            const uint32_t dst0 = row0 * 128u + (((uint32_t)piece ^ (row0 & 7)) << 4);
            Ring ring;
            bool ok = true;
#pragma unroll 1
            for (uint32_t tile = unit; ok && tile < total; tile += units) {
                const Tile t = mm::find_tile(p, first, slot0, tile, lane);
                const int n = t.n, copies = (n + 15) >> 4;
                const uint8_t *src[8];
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    src[j] = p.x_codes;
                    if (j < copies) {
                        const int32_t v = __ldg(p.rows + (int64_t)t.slot + min(16 * j + (int)row0, n - 1));
                        src[j] += (v < 0 || v >= p.x_rows ? 0 : v) * p.x_code_stride;
                    }
                    src[j] += k0 * 128 + 16 * piece;
                }
                int at = k0 * 128 + 16 * piece;
#pragma unroll 1
                for (int k = k0; k < k1; ++k, at += 128, ring.next(p.stages)) {
                    ok = __all_sync(0xFFFFFFFFu, tc::bar_wait_ready(empty0 + 8 * ring.s, ring.parity ^ 1u, abort));
                    if (!ok) break;
                    const uint32_t dst = ring0 + ring.s * p.stage_bytes + dst0;
                    const bool live = at < p.depth;
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        if (j < copies) tc::cp_async16(dst + j * 2048u, src[j], live);
                        src[j] += 128;
                    }
                    tc::cp_async_arrive(full0 + 8 * ring.s);
                }
            }
        }
    } else {
        // ---- partial sums and the epilogue ----
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSumRegs<ROWS>));
        // Two weight blocks: warps 4-7 sum the first one's columns and warps 8-11
        // the second one's; one: 64 columns each.  Warps w and w + 4 have the
        // same 32 rows.
        const int w = warp & 3, half = (warp - kFirstSumWarp) >> 2;
        constexpr int kCols = AT * 64;                                      // this warp's columns
        // columns taken out of tensor memory at a time: as many as the registers
        // hold beside the sums (128 experts of 256 slots, gated, through an index:
        // 402 us with 32, 434 with 64; dense 8191 x 5120 x 5120: 200 and 194)
        constexpr int kTaken = ROWS ? 32 : 64;
        const int col0 = kCols * half;
        float *buf = region + (warp - kFirstSumWarp) * 32 * 32;
        const uint32_t lanes = tmem + ((uint32_t)(32 * w) << 16);
        auto release = [&](uint32_t set) {
            tc::fence_before();
            __syncwarp();
            tc::bar_arrive_if(acce0 + 8 * set, lane == 0);
        };
        auto meet = [&]() { tc::named_sync(1 + w, 64); };      // warps w and w + 4
        uint32_t count = 0;              // partial sums so far
        // where the partial sum with that number is: its set, and the parity of its round
        auto set_of = [&](uint32_t i) { return AT == 2 ? (i & 1) * 2 + half : i & 3; };
        bool ok = true;
        uint32_t tile = unit;
#pragma unroll 1
        for (uint32_t nth = 0; tile < total; tile += units, ++nth) {
            const Tile t = mm::find_tile(p, first, slot0, tile, lane);
            const int n = t.n - 32 * w;         // this warp's rows, if any
            if (MODE != kHalves && !SPLIT && (MODE == kHalvesSum || p.residual) && lane < n) {
                // what the epilogue will add to this lane's row, into L2
                const int bytes = p.residual_dtype == CSF_F32 ? 4 : 2, f = t.rt * p.tile_step + (p.gated ? 64 * half : col0);
                const char *at = static_cast<const char *>(p.residual) + (((int64_t)t.slot + 32 * w + lane) * p.residual_stride + f) * bytes;
                const int end = min(p.gated ? 64 : kCols, p.F - f) * bytes;
                for (int b = 0; b < end; b += 32) tc::prefetch_l2(at + b);
            }
            uint64_t sum[kCols / 2];     // two columns each
#pragma unroll
            for (int i = 0; i < kCols / 2; ++i) sum[i] = 0;
            bool there = false;          // the next partial sums: asked for while these come out of tensor memory
#pragma unroll 1
            for (int k = k0; k < k1; ++k, ++count) {
                const uint32_t set = set_of(count), next = set_of(count + 1);
                constexpr int kRound = AT == 2 ? 1 : 2;
                if (!__any_sync(0xFFFFFFFFu, there)) {
                    ok = __all_sync(0xFFFFFFFFu, tc::bar_wait_here(accf0 + 8 * set, (count >> kRound) & 1, abort));
                    if (!ok) break;
                }
                tc::fence_after();
                const bool last = k + 1 == k1, keep = last && !SPLIT;        // the whole sums go back there
                there = false;
                if (n > 0) {
                    const uint32_t at = lanes + set * 128 + (AT == 2 ? 0 : col0);
                    uint64_t factor = 0;
#pragma unroll
                    for (int c = 0; c < kCols; c += kTaken) {
                        uint32_t v[kTaken / 16][16];
#pragma unroll
                        for (int i = 0; i < kTaken / 16; ++i) tc::tmem_load(at + c + 16 * i, v[i]);
                        if (c == 0) factor = tc::twice(factors[count % kFactorSteps][AT == 2 ? half : 0][32 * w + lane]);
                        if (c + kTaken >= kCols) there = tc::bar_try_if(accf0 + 8 * next, ((count + 1) >> kRound) & 1, lane == 0 && !last);
                        tc::wait_ld();
                        if (c + kTaken >= kCols && !keep) release(set);
#pragma unroll
                        for (int j = 0; j < kTaken / 2; ++j)
                            if (c / 2 + j < kCols / 2) tc::fma2_after(sum[c / 2 + j], v[j >> 3][2 * (j & 7)], v[j >> 3][2 * (j & 7) + 1], factor);
                    }
                } else if (!keep) {
                    release(set);
                }
            }
            if (!ok) break;
            if constexpr (SPLIT) {
                // a row's sums to the block that finishes it
                const uint32_t share = ((uint32_t)t.n + split - 1) / split, r = (uint32_t)(32 * w + lane);
                if (lane < n) {
                    const uint32_t to = r / share;
                    const uint32_t at = tc::in_block(tc::smem_u32(region + (rank * share + (r - to * share)) * (AT * 128) + col0), to);
#pragma unroll
                    for (int j = 0; j < kCols; j += 4) {
                        float v[4];
                        tc::halves(sum[j / 2], v[0], v[1]);
                        tc::halves(sum[j / 2 + 1], v[2], v[3]);
                        tc::store_cluster4(at + j * 4u, v[0], v[1], v[2], v[3]);
                    }
                }
                break;
            }
            // The sums, back to where the last partial ones were.
            const uint32_t set = set_of(count - 1), own = lanes + set * 128 + (AT == 2 ? 0 : col0);
            if (n > 0) {
#pragma unroll
                for (int c = 0; c < kCols / 16; ++c) {
                    uint32_t v[16];
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        float lo, hi;
                        tc::halves(sum[c * 8 + j], lo, hi);
                        v[2 * j] = __float_as_uint(lo), v[2 * j + 1] = __float_as_uint(hi);
                    }
                    tc::tmem_store(own + c * 16, v);
                }
                tc::wait_st();
            }
            if (n > 0) {
                const int64_t slot = (int64_t)t.slot + 32 * w;
                const bool gated = AT == 2 && p.gated;
                // this warp's columns of the output, and where their sums are (a gated product's: 64 of both blocks)
                const int f0 = t.rt * p.tile_step + (gated ? 64 * half : col0), cols = gated ? 64 : kCols;
                const uint32_t gate = gated ? lanes + (set & 2) * 128 + 64 * half : own, up = gate + 128;
                if (gated) {
                    tc::fence_before();
                    meet();
                    tc::fence_after();
                }
                const bool live = lane < n;
                const float rs = p.row_scale && live ? __ldg(p.row_scale + slot + lane) : 1.f;
                // 32 columns of this lane's row from column c of f0 on: act(p) and the row's weight
                auto values = [&](float (&y)[32], int c) {
                    uint32_t v[32];
                    tc::tmem_load(gate + c, v);
                    if (gated) {
                        uint32_t u[32];
                        tc::tmem_load(up + c, u);
                        tc::wait_ld(v);
                        tc::wait_ld(u);
                        float b[32];
#pragma unroll
                        for (int i = 0; i < 32; ++i) y[i] = __uint_as_float(v[i]), b[i] = __uint_as_float(u[i]);
                        if (p.bias) {
#pragma unroll
                            for (int i = 0; i < 32; i += 8) add_bias8(p, y + i, t.e, f0 + c + i);
#pragma unroll
                            for (int i = 0; i < 32; i += 8) add_bias8(p, b + i, t.e, p.F + f0 + c + i);
                        }
                        activate32(y, p.act);
#pragma unroll
                        for (int i = 0; i < 32; ++i) y[i] *= b[i];
                    } else {
                        tc::wait_ld(v);
#pragma unroll
                        for (int i = 0; i < 32; ++i) y[i] = __uint_as_float(v[i]);
                        if (p.bias) {
#pragma unroll
                            for (int i = 0; i < 32; i += 8) add_bias8(p, y + i, t.e, f0 + c + i);
                        }
                        activate32(y, p.act);
                    }
                    if (p.row_scale) {
#pragma unroll
                        for (int i = 0; i < 32; ++i) y[i] *= rs;
                    }
                };
                // A warp's piece lies as 32 rows of 128 bytes, row r's 16-byte
                // part q at q ^ (r % 8): written a row a lane and read 4 or 8
                // rows at a time, both without bank conflicts.
                auto piece_at = [&](int r, int q) { return buf + r * 32 + ((q ^ (r & 7)) << 2); };
                if constexpr (MODE == kHalves || MODE == kHalvesSum) {
                    // 64 columns at a time, rounded before the turn.  A residual
                    // comes the other way through the same piece, the next 64
                    // columns' under way meanwhile.
                    constexpr bool kSum = MODE == kHalvesSum;
                    const int q8 = lane & 7, r8 = lane >> 3;
                    uint4 next[8] = {};           // (defined on every path: else it is held through the products, too)
                    auto fetch = [&](int c0) {
                        const uint4 *at = reinterpret_cast<const uint4 *>(static_cast<const char *>(p.residual) + ((slot + r8) * p.residual_stride + f0 + c0) * 2) + q8;
#pragma unroll
                        for (int i = 0; i < 8; ++i)
                            if (4 * i + r8 < n && f0 + c0 + 8 * q8 < p.F) next[i] = __ldg(at + i * (p.residual_stride >> 1));
                    };
                    if (kSum) fetch(0);
#pragma unroll 1
                    for (int c0 = 0; c0 < cols && f0 + c0 < p.F; c0 += 64) {
                        if (kSum) {
#pragma unroll
                            for (int i = 0; i < 8; ++i) *reinterpret_cast<uint4 *>(piece_at(4 * i + r8, q8)) = next[i];
                            __syncwarp();
                            if (c0 + 64 < cols) fetch(c0 + 64);
                        }
#pragma unroll 1
                        for (int q = 0; q < 8; q += 4) {
                            float y[32];
                            values(y, c0 + 8 * q);
                            if (kSum) {
#pragma unroll
                                for (int i = 0; i < 4; ++i) {
                                    elem::Raw raw;
                                    raw.a = *reinterpret_cast<const uint4 *>(piece_at(lane, q + i));
                                    raw.b = raw.a;
                                    float b[8];
                                    elem::to_floats(b, raw, p.residual_dtype);
#pragma unroll
                                    for (int j = 0; j < 8; ++j) y[8 * i + j] += b[j];
                                }
                            }
                            uint32_t o[16];
#pragma unroll
                            for (int i = 0; i < 16; ++i) {
                                if (p.out_dtype == CSF_BF16) {
                                    const __nv_bfloat162 b = __floats2bfloat162_rn(y[2 * i], y[2 * i + 1]);
                                    memcpy(&o[i], &b, 4);
                                } else {
                                    const __half2 b = __floats2half2_rn(y[2 * i], y[2 * i + 1]);
                                    memcpy(&o[i], &b, 4);
                                }
                            }
#pragma unroll
                            for (int i = 0; i < 4; ++i) *reinterpret_cast<uint4 *>(piece_at(lane, q + i)) = make_uint4(o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3]);
                        }
                        __syncwarp();
                        const int q = lane & 7, f = f0 + c0 + 8 * q;
                        char *out = p.out + (slot + (lane >> 3)) * p.out_stride;
                        if (p.out_wide && f + 8 <= p.F) {
#pragma unroll
                            for (int i = 0; i < 8; ++i) {
                                const int r = 4 * i + (lane >> 3);
                                if (r < n) *reinterpret_cast<uint4 *>(out + 4 * i * p.out_stride + 2 * f) = *reinterpret_cast<const uint4 *>(piece_at(r, q));
                            }
                        } else {
                            for (int r = lane >> 3; r < min(n, 32); r += 4) {
                                elem::Raw o;
                                o.a = *reinterpret_cast<const uint4 *>(piece_at(r, q));
                                o.b = o.a;
                                elem::store_few(p.out + (slot + r) * p.out_stride, f, p.F, o, p.out_dtype);
                            }
                        }
                        __syncwarp();
                    }
                } else if constexpr (MODE == kPlain) {
                    // 32 columns as floats; a residual's piece is fetched while the sums of the last are turned
                    const int part = lane & 3, sub = lane >> 2;
                    const int res_bytes = p.residual_dtype == CSF_F32 ? 4 : 2;
                    const char *res = static_cast<const char *>(p.residual) + (slot + sub) * p.residual_stride * res_bytes;
                    elem::Raw next[4] = {};       // (defined on every path: else it is held through the products, too)
                    auto fetch = [&](int c0) {
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            if (8 * i + sub < n) next[i] = elem::load_apart(res + 8 * i * p.residual_stride * res_bytes, f0 + c0 + 8 * part, p.F, p.residual_dtype, p.residual_wide);
                    };
                    if (p.residual) fetch(0);
#pragma unroll 1
                    for (int c0 = 0; c0 < cols && f0 + c0 < p.F; c0 += 32) {
                        elem::Raw now[4];
#pragma unroll
                        for (int i = 0; i < 4; ++i) now[i] = next[i];
                        if (p.residual && c0 + 32 < cols) fetch(c0 + 32);
                        {
                            float y[32];
                            values(y, c0);
#pragma unroll
                            for (int i = 0; i < 8; ++i)
                                *reinterpret_cast<float4 *>(piece_at(lane, i)) = make_float4(y[4 * i], y[4 * i + 1], y[4 * i + 2], y[4 * i + 3]);
                        }
                        __syncwarp();
                        const int f = f0 + c0 + 8 * part;
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const int r = 8 * i + sub;
                            const float4 lo = *reinterpret_cast<const float4 *>(piece_at(r, 2 * part)), hi = *reinterpret_cast<const float4 *>(piece_at(r, 2 * part + 1));
                            float y[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
                            if (r >= n || f >= p.F) continue;
                            if (p.residual) {
                                float b[8];
                                elem::to_floats(b, now[i], p.residual_dtype);
#pragma unroll
                                for (int j = 0; j < 8; ++j) y[j] += b[j];
                            }
                            elem::store_apart(p.out + (slot + r) * p.out_stride, f, p.F, elem::from_floats(y, p.out_dtype), p.out_dtype, p.out_wide);
                        }
                        __syncwarp();
                    }
                } else {
                    const int padded = (p.F + 31) & ~31;
                    const char *res = p.residual ? static_cast<const char *>(p.residual) + (slot + (live ? lane : 0)) * p.residual_stride * (p.residual_dtype == CSF_F32 ? 4 : 2) : nullptr;
                    uint32_t m = 0;
#pragma unroll 1
                    for (int c = 0; c < cols && f0 + c < padded; c += 32) {
                        float y[32];
                        values(y, c);
                        if (res) {
                            float b[8];
#pragma unroll
                            for (int g = 0; g < 32; g += 8) {
                                elem::to_floats(b, elem::load_apart(res, f0 + c + g, p.F, p.residual_dtype, p.residual_wide), p.residual_dtype);
#pragma unroll
                                for (int i = 0; i < 8; ++i) y[g + i] += b[i];
                            }
                        }
#pragma unroll
                        for (int h = 0; h < 32; h += 16) {
                            uint32_t v[16];
#pragma unroll
                            for (int i = 0; i < 16; ++i) {
                                v[i] = f0 + c + h + i < p.F ? __float_as_uint(y[h + i]) : 0;
                                m = max(m, v[i] & 0x7FFFFFFFu);
                            }
                            tc::tmem_store(gate + c + h, v);
                        }
                    }
                    tc::wait_st();
                    if (cols == 64) {
                        // the largest magnitude of a block of 128 columns comes from both warps of these rows
                        float (&amax)[2][128] = sh.amax[nth & 1];
                        amax[half][32 * w + lane] = __uint_as_float(m);
                        meet();
                        m = max(m, __float_as_uint(amax[half ^ 1][32 * w + lane]));
                    }
                    const float scale = quant::fp8_scale(m), scale_up = scale < quant::kLeastWhole ? quant::kWholeUp : 1.f;
                    const quant::Whole whole = quant::fp8_whole(scale * scale_up);
                    const int part = lane & 3, sub = lane >> 2;
#pragma unroll 1
                    for (int c0 = 0; c0 < cols && f0 + c0 < padded; c0 += 64) {
#pragma unroll 1
                        for (int q = 0; q < 4 && f0 + c0 + 16 * q < padded; q += 2) {
                            uint32_t v[32];
                            tc::tmem_load(gate + c0 + 16 * q, v);
                            tc::wait_ld(v);
                            uint32_t o[8];
#pragma unroll
                            for (int i = 0; i < 8; ++i) {
                                float y[4];
#pragma unroll
                                for (int j = 0; j < 4; ++j) y[j] = quant::over(__uint_as_float(v[4 * i + j]) * scale_up, whole);
                                o[i] = quant::e4m3x2(y[0], y[1]) | quant::e4m3x2(y[2], y[3]) << 16;
                            }
                            *reinterpret_cast<uint4 *>(piece_at(lane, q)) = make_uint4(o[0], o[1], o[2], o[3]);
                            *reinterpret_cast<uint4 *>(piece_at(lane, q + 1)) = make_uint4(o[4], o[5], o[6], o[7]);
                        }
                        __syncwarp();
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const int r = 8 * i + sub, f = f0 + c0 + 16 * part;
                            if (r < n && f < padded) *reinterpret_cast<uint4 *>(p.out + (slot + r) * p.out_stride + f) = *reinterpret_cast<const uint4 *>(piece_at(r, part));
                        }
                        __syncwarp();
                    }
                    if ((f0 & 127) == 0 && f0 < padded && live) {
                        float *scales = reinterpret_cast<float *>(p.out_scales + (slot + lane) * p.out_scale_stride);
                        const int b = f0 >> 7, n_blocks = (p.F + 127) >> 7;
                        scales[b] = scale;
                        if (b + 1 == n_blocks)       // clear the scale row's padding
                            for (int i = n_blocks; i & 3; ++i) scales[i] = 0.f;
                    }
                }
                if (gated) meet();      // the other warp has read this one's block, too
            }
            release(set);
        }
        if (!SPLIT && !ok && ((AT == 2 && p.gated) || (MODE == kQuant && AT == 1))) {
            // A wait gave up.  The other warp of these rows may not have: it is
            // met as often as the tiles that are left have it do.
            const int meetings = AT == 1 ? 1 : MODE == kQuant ? 3 : 2;
            for (; tile < total; tile += units)
                if (mm::find_tile(p, first, slot0, tile, lane).n > 32 * w)
                    for (int i = 0; i < meetings; ++i) meet();
        }
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
    if constexpr (SPLIT) tc::cluster_sync();         // the sums have come; nothing is under way to a block that leaves
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
                finish8<MODE == kQuant>(p, y[0], (int64_t)t.slot + (int64_t)rank * share + r, f, live);
            }
        }
    }
    if (warp == 1) tc::tmem_free(tmem, kTmemCols);
}

using Kernel = void (*)(CUtensorMap, CUtensorMap, Params);

template <bool ROWS, int MODE>
Kernel pick(int shape) {
    // where the depth is shared, what comes out is asked at run time
    constexpr int kAny = MODE == kQuant ? kQuant : kPlain;
    switch (shape) {
        case kOne: return fp8_matmul_kernel<1, ROWS, false, MODE>;
        case kTwo: return fp8_matmul_kernel<2, ROWS, false, MODE>;
        case kOneShared: return fp8_matmul_kernel<1, ROWS, true, kAny>;
        default: return fp8_matmul_kernel<2, ROWS, true, kAny>;
    }
}

template <bool ROWS>
Kernel pick_kernel(int shape, int mode) {
    switch (mode) {
        case kHalves: return pick<ROWS, kHalves>(shape);
        case kHalvesSum: return pick<ROWS, kHalvesSum>(shape);
        case kPlain: return pick<ROWS, kPlain>(shape);
        default: return pick<ROWS, kQuant>(shape);
    }
}

// The kernel of a shape, one translation unit each for x rows in order and
// through an index.
Kernel rows_in_order(int shape, int mode);
Kernel rows_by_index(int shape, int mode);

}  // namespace f8
}  // namespace csfk
