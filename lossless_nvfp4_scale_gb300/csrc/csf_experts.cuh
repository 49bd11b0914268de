// Block-scaled products of quantised rows with the experts' FP4 weights
// (csf_expert_matmul): the kernel.
//
// Per expert the weight rows are the M side (128 a tile), its slots the N
// side: experts have few slots each, and N can be any multiple of 16.  The
// 5th-generation tensor cores multiply codes and block scales as stored
// (E2M1 x E2M1 with UE4M3 scales per 16, or E2M1 x E4M3 with UE8M0 scales per
// 32) and accumulate in 32 bits, so nothing is dequantised on the way.  The
// weight scales are read in the 128 x 4 tile layout that csf_decode writes:
// a tile copies straight to tensor memory.
//
// One persistent block per SM walks tiles (expert, slot tile, row tile):
//   warp 0   weights (TMA, 128-byte swizzle) and their scale tiles
//   warps 2, 3, 12, 13  x rows: through TMA, 32 rows a request, where slots are
//            rows; gathered through the index by 16-byte asynchronous copies,
//            swizzled as TMA would, where they are not (TMA's gather of four
//            rows took 64 cycles a request)
//   warp 14  the scale bytes of those rows, through registers into the tile
//            layout (with the copying warps that TMA leaves free)
//   warp 15  which tile comes next and which x rows it takes, a few tiles ahead
//   warp 1   scale copies to tensor memory and the matrix instructions
//   warps 4-11  epilogue
// Their inner loops run alone on a scheduler, a few cycles an instruction, so
// pointers advance and the ring's position is counted rather than computed.
// A ring of shared-memory stages of 128 code bytes per row joins them; two
// accumulator sets let the epilogue of a tile overlap the next tile's
// products.  A gated product holds two accumulators: row tile t of the gate
// half and of the up half, from the same x rows.
//
// Where few slots make few tiles, a cluster of 2 to 8 blocks shares a tile:
// each sums its part of K, the others send their sums to the first block's
// shared memory, which adds them in order and runs the epilogue.
//
// The epilogue reads an accumulator a weight row a lane, 8 or 16 slots at a
// time, applies what belongs to the row (alpha, bias, activation), and turns
// the piece around in shared memory, so that a lane then holds 8 columns of
// one slot: residual and output move 16 bytes a lane, and the lanes of a
// scale block are neighbours.
//
// What bounds it, measured with two input sets in turn (copy 6.78 TB/s,
// bfloat16 products 1.94 PFLOP/s):
//   512 experts of 64 slots, 1024 x 1600 NVFP4, gated   88 us, 5.86 TB/s: memory
//   384 experts of 5, 2048 x 5120 MXFP4, gated         351 us, 6.12 TB/s: memory
//   512 of 64, 2048 x 800 NVFP4, bias and residual     150 us, 5.05 TB/s: the
//     epilogue (108 us without a residual) and short K: a tile is 4 stages
//   8191 slots of one 2048 x 5120 MXFP4                 79 us, 2.2 PFLOP/s:
//     shared-memory bandwidth (operands in, operands to the tensor cores)
//   64 slots on 8 of 512, gated                        8.2 us: latency
//   one slot of 2048 x 5120 MXFP4                      9.4 us: latency
#pragma once

#include <type_traits>

#include <cuda.h>

#include "csf_grouped.cuh"
#include "csf_internal.cuh"
#include "csf_quant.cuh"
#include "csf_tc.cuh"

namespace csfk {
namespace mm {

constexpr int kMmThreads = 512;
constexpr int kEpiWarps = 8;
constexpr int kXWarps = 4;
constexpr int kXBox = 32;             // x rows per TMA request
constexpr int kTurnStride = 36;      // floats between slots of a warp's 16 x 32 piece: reads and writes without bank conflicts
constexpr int kMmMaxExperts = 8192;
constexpr uint32_t kTmemCols = 512;
constexpr int kSmemLimit = 227 * 1024;
constexpr int kMaxStages = 12;

struct MmParams {
    const uint8_t *x_codes, *x_scales;
    int64_t x_code_stride, x_scale_stride;
    const uint8_t *w_scales;
    int64_t w_scale_expert;      // bytes between experts' scale stacks
    const int32_t *rows;
    const void *start;
    const float *alpha;
    const void *bias;
    const float *row_scale;
    const void *residual;
    int64_t residual_stride;
    void *out;
    int64_t out_stride;          // elements, or code bytes of a quantised output
    uint8_t *out_scales;
    int64_t out_scale_stride;
    const float *out_tensor_scale;
    uint32_t *err;
    int64_t slots;
    int32_t x_rows;
    int32_t es64;
    int32_t E, N, K, F;          // F: output columns (N, or N / 2 gated)
    int32_t ncb;                 // scale tiles per 128-row block of a weight stack
    int32_t row_tiles;           // row tiles per expert
    uint32_t row_tiles_magic;    // 2^32 / row_tiles, rounded up
    int32_t second;              // weight rows from a tile's first 128 rows to its second
    int32_t nt;                  // most slots per tile (a multiple of 16)
    int32_t stages;
    uint32_t stage_bytes;
    int32_t act, bias_dtype, residual_dtype;
    int32_t split;               // blocks of a cluster that share a tile's K
    int32_t b_rows;              // x rows of a stage
    int32_t out_wide, residual_wide;   // 16-byte accesses allowed
};

enum Out { kOutBf16 = 0, kOutF16 = 1, kOutF32 = 2, kOutNv = 3, kOutMx = 4 };

__device__ __forceinline__ uint32_t load_raw(const void *base, int64_t at, int dtype) {
    return dtype == CSF_F32 ? static_cast<const uint32_t *>(base)[at] : static_cast<const uint16_t *>(base)[at];
}

__device__ __forceinline__ float raw_as_float(uint32_t v, int dtype) {
    if (dtype == CSF_F32) return __uint_as_float(v);
    if (dtype == CSF_BF16) return __uint_as_float(v << 16);
    return __half2float(__ushort_as_half((unsigned short)v));
}

// 8 values of a row of type `dtype`, as stored.
struct Raw8 {
    uint4 a, b;
};

// The first `cols` of 8 values, one at a time: ragged or unaligned rows.
static __device__ __noinline__ Raw8 load_few(const char *p, int dtype, int cols) {
    uint32_t v[8];
    for (int i = 0; i < 8; ++i) v[i] = i < cols ? load_raw(p, i, dtype) : 0;
    Raw8 r;
    r.a = dtype == CSF_F32 ? make_uint4(v[0], v[1], v[2], v[3])
                           : make_uint4(v[0] | v[1] << 16, v[2] | v[3] << 16, v[4] | v[5] << 16, v[6] | v[7] << 16);
    r.b = make_uint4(v[4], v[5], v[6], v[7]);
    return r;
}

__device__ __forceinline__ Raw8 load_raw8(const char *p, int dtype, int cols, bool wide) {
    Raw8 r = {make_uint4(0, 0, 0, 0), make_uint4(0, 0, 0, 0)};
    if (wide && cols >= 8) {
        r.a = reinterpret_cast<const uint4 *>(p)[0];
        if (dtype == CSF_F32) r.b = reinterpret_cast<const uint4 *>(p)[1];
    } else if (cols > 0) {
        r = load_few(p, dtype, cols);
    }
    return r;
}

__device__ __forceinline__ void add_raw8(float (&y)[8], const Raw8 &r, int dtype) {
    const uint32_t u[8] = {r.a.x, r.a.y, r.a.z, r.a.w, r.b.x, r.b.y, r.b.z, r.b.w};
    if (dtype == CSF_BF16) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            y[2 * i] += __uint_as_float(u[i] << 16);
            y[2 * i + 1] += __uint_as_float(u[i] & 0xFFFF0000u);
        }
    } else if (dtype == CSF_F32) {
#pragma unroll
        for (int i = 0; i < 8; ++i) y[i] += __uint_as_float(u[i]);
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            __half2 h;
            memcpy(&h, &u[i], 4);
            const float2 f = __half22float2(h);
            y[2 * i] += f.x;
            y[2 * i + 1] += f.y;
        }
    }
}

// The first `cols` of 8 elements of 2 bytes (in u) or 4 (y), one at a time.
template <bool F32>
static __device__ __noinline__ void store_few(char *o, uint4 u, float4 lo, float4 hi, int cols) {
    const uint32_t h[4] = {u.x, u.y, u.z, u.w};
    const float y[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
    for (int i = 0; i < 8; ++i) {
        if (i >= cols) break;
        if (F32) reinterpret_cast<float *>(o)[i] = y[i];
        else reinterpret_cast<uint16_t *>(o)[i] = (uint16_t)(h[i >> 1] >> (16 * (i & 1)));
    }
}

// Columns f .. f+7 of one slot's output, at o (and the slot's scales at
// srow).  Every lane calls it (a scale block is 2 or 4 lanes wide); `live`
// lanes write.
template <int OUT>
__device__ __forceinline__ void emit8(const MmParams &p, float (&y)[8], int f, char *o, uint8_t *srow, bool live,
                                      float tensor_scale) {
    const int cols = p.F - f;
    if constexpr (OUT == kOutNv || OUT == kOutMx) {
        constexpr int kKind = OUT == kOutNv ? CSF_ROWS_NVFP4 : CSF_ROWS_MXFP8;
        const int fp = (p.F + 31) & ~31;
        if (cols < 8) {
#pragma unroll
            for (int i = 0; i < 8; ++i) y[i] = i < cols ? y[i] : 0.f;
        }
        quant::quantize8<kKind>(y, reinterpret_cast<uint8_t *>(o), srow, f >> 3, live && f < fp, tensor_scale);
        if (live && f + 8 == fp) {     // the row's last columns: clear the scale row's padding
            const int blocks = OUT == kOutNv ? fp >> 4 : fp >> 5;
            for (int i = blocks; i < ((blocks + 15) & ~15); ++i) srow[i] = 0;
        }
    } else if constexpr (OUT == kOutF32) {
        if (!live || cols <= 0) return;
        const float4 lo = make_float4(y[0], y[1], y[2], y[3]), hi = make_float4(y[4], y[5], y[6], y[7]);
        if (p.out_wide && cols >= 8) {
            reinterpret_cast<float4 *>(o)[0] = lo;
            reinterpret_cast<float4 *>(o)[1] = hi;
        } else {
            store_few<true>(o, make_uint4(0, 0, 0, 0), lo, hi, cols);
        }
    } else {
        if (!live || cols <= 0) return;
        uint32_t u[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if constexpr (OUT == kOutBf16) {
                const __nv_bfloat162 h = __floats2bfloat162_rn(y[2 * i], y[2 * i + 1]);
                memcpy(&u[i], &h, 4);
            } else {
                const __half2 h = __floats2half2_rn(y[2 * i], y[2 * i + 1]);
                memcpy(&u[i], &h, 4);
            }
        }
        const uint4 q = make_uint4(u[0], u[1], u[2], u[3]);
        if (p.out_wide && cols >= 8) *reinterpret_cast<uint4 *>(o) = q;
        else store_few<false>(o, q, make_float4(0, 0, 0, 0), make_float4(0, 0, 0, 0), cols);
    }
}

constexpr int kMaxTileSlots = 224;
__host__ __device__ constexpr int tile_slots(int shape) {
    return shape == 1 ? kMaxTileSlots : shape == 0 || shape == 3 ? 128 : 96;
}
constexpr int kSplitSlots = 16;      // slots of a tile that a cluster shares
constexpr int kMaxSplit = 8;
constexpr int kTileRing = 4;         // tiles that the roles may be apart

struct Shared {
    uint64_t full[kMaxStages], empty[kMaxStages], acc_full[2], acc_empty[2], tile_full[kTileRing], tile_empty[kTileRing], sums_full;
    Tile tile[kTileRing];                        // n = 0: no more
    int32_t x_row[kTileRing][kMaxTileSlots];
    uint32_t tmem, abort, warp_sum[kMmThreads / 32];
};

// What a tile spans: 128 weight rows and up to 128 or 224 slots, or 128 gate
// rows, their 128 up rows and up to 96 slots.  (Tensor memory holds two sets
// of accumulators and the scales.)  The shared ones are the narrow and the
// gated tile with K spread over a cluster.
enum Shape { kNarrow = 0, kWide = 1, kGated = 2, kNarrowShared = 3, kGatedShared = 4 };

// KIND: csf_rows_kind of x.  ROWS: slot s reads row rows[s] of x, else row s.
// RES: there is a residual or a row weight.  (Each is a kernel of its own
// because the roles' loops share an instruction cache: what is not run should
// not lie between them.)
template <int KIND, bool ROWS, int SHAPE, bool RES, int OUT>
__global__ void __launch_bounds__(kMmThreads, 1)
expert_matmul_kernel(const __grid_constant__ CUtensorMap wmap, const __grid_constant__ CUtensorMap xmap,
                     const __grid_constant__ MmParams p) {
    extern __shared__ __align__(1024) uint8_t dyn[];
    __shared__ Shared sh;
    __shared__ __align__(16) float turn[kEpiWarps][16 * kTurnStride];
    constexpr bool GATED = SHAPE == kGated || SHAPE == kGatedShared, SHARED = SHAPE >= kNarrowShared;
    constexpr int AT = GATED ? 2 : 1;                     // 128-row weight tiles per tile
    constexpr bool kNv = KIND == CSF_ROWS_NVFP4;
    constexpr int kScaleWarps = ROWS || RES ? 1 : kXWarps;   // warps that bring the x scales
    // warps that take tiles: weights, products, x, x scales, epilogue
    constexpr int kTileUsers = 2 + (ROWS ? kXWarps : 1) + kScaleWarps + kEpiWarps;
    constexpr int kStepK = kNv ? 256 : 128;               // elements per stage: 128 bytes of codes a row
    constexpr int kTilesPerStage = kNv ? 4 : 1;           // 128 x 4 scale tiles per stage and 128 rows
    constexpr uint32_t kABytes = 128 * 128;
    constexpr uint32_t kACopied = kNv ? kABytes : kABytes / 2;   // E2M1 codes unpack on the way: counted as stored
    constexpr int kAccCols = tile_slots(SHAPE);           // accumulator columns
    constexpr int kGroups = RES && !GATED ? 2 : 1;        // 8-slot groups an epilogue warp takes a round
    constexpr int kRowBlocks = (kAccCols + 127) / 128;    // 128-row blocks of x scales
    constexpr uint32_t kSfCols = 4 * kTilesPerStage;      // tensor-memory columns of one operand's scales
    constexpr uint32_t kSfBase = 2 * AT * kAccCols;
    constexpr uint32_t kSfA = kSfBase + kRowBlocks * kSfCols;
    static_assert(kSfA + AT * kSfCols <= kTmemCols, "tensor memory");

    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const uint32_t ring0 = (tc::smem_u32(dyn) + 1023u) & ~1023u;
    uint32_t *first = reinterpret_cast<uint32_t *>(dyn + (ring0 - tc::smem_u32(dyn)) + (size_t)p.stages * p.stage_bytes);

    uint32_t *slot0 = first + p.E + 1;          // an expert's first slot
    // the other blocks' sums of a shared tile: [block][weight tile][slot][row]
    float *sums = reinterpret_cast<float *>(first + ((2 * p.E + 2 + 3) & ~3));
    const uint32_t rank = SHARED ? tc::cluster_rank() : 0, split = SHARED ? (uint32_t)p.split : 1;

    const uint32_t b_off = AT * kABytes, sfa_off = b_off + (uint32_t)p.b_rows * 128u,
                   sfb_off = sfa_off + AT * kTilesPerStage * 512u;
    const uint32_t full0 = tc::smem_u32(sh.full), empty0 = tc::smem_u32(sh.empty);
    const uint32_t accf0 = tc::smem_u32(sh.acc_full), acce0 = tc::smem_u32(sh.acc_empty);
    const uint32_t tilef0 = tc::smem_u32(sh.tile_full), tilee0 = tc::smem_u32(sh.tile_empty);

    if (tid == 0) {
        for (int i = 0; i < p.stages; ++i) {
            tc::bar_init(full0 + 8 * i, ROWS ? 2 + 32 * kXWarps : 2 + kScaleWarps);    // weights; x and x scales (by warps and their lanes)
            tc::bar_init(empty0 + 8 * i, 1);
        }
        for (int i = 0; i < 2; ++i) {
            tc::bar_init(accf0 + 8 * i, 1);
            tc::bar_init(acce0 + 8 * i, 32 * kEpiWarps);
        }
        for (int i = 0; i < kTileRing; ++i) {
            tc::bar_init(tilef0 + 8 * i, 1);
            tc::bar_init(tilee0 + 8 * i, kTileUsers);
        }
        tc::bar_init(tc::smem_u32(&sh.sums_full), SHARED ? (split - 1) * 32u * kEpiWarps : 1);
        sh.abort = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 1) tc::tmem_alloc(tc::smem_u32(&sh.tmem), kTmemCols);

    bool bad = false;
    const uint32_t running = number_tiles<kMmThreads>(p, first, slot0, sh.warp_sum, bad);
    if (tid == 0) first[p.E] = running, slot0[p.E] = (uint32_t)start_at(p, p.E);
    tc::fence_before();
    bad = __syncthreads_or(bad);
    tc::fence_after();
    if (bad && p.err && blockIdx.x == 0 && tid == 0) atomicOr(p.err, CSF_DEV_ERR_CORRUPT);
    // An expert_start out of order or range makes no tiles: its experts could
    // overlap, and their tiles be more than 32 bits count.
    uint32_t total = bad ? 0 : first[p.E] * (uint32_t)p.row_tiles;
    if constexpr (SHARED) total = min(total, gridDim.x / split);      // one tile a cluster
    const uint32_t tmem = sh.tmem;
    volatile uint32_t *abort = &sh.abort;
    // this block's part of K, in whole 16-byte units of x scales
    constexpr int kStagesPer16 = 4 / kTilesPerStage;
    const int all_units = (p.ncb + 3) / 4, all_steps = (p.K + kStepK - 1) / kStepK;
    const int unit0 = (int)(rank * (uint32_t)all_units / split), unit1 = (int)((rank + 1) * (uint32_t)all_units / split);
    const int k0 = unit0 * kStagesPer16, ksteps = min(all_steps, unit1 * kStagesPer16) - k0;
    const int left0 = p.ncb - k0 * kTilesPerStage;      // scale tiles from there on
    const uint32_t tile0 = blockIdx.x / split, tile_step = gridDim.x / split;
    if constexpr (SHARED) tc::cluster_sync();           // the barriers of the first block are set up

    // Roles that take tiles: wait for the next one's description; done with
    // it, one lane of each says so.
    auto take = [&](const Ring &r, Tile &t) {
        if (!tc::bar_wait(tilef0 + 8 * r.s, r.parity, abort)) return false;
        t = sh.tile[r.s];
        return t.n > 0;
    };
    auto done_with = [&](Ring &r) {
        tc::bar_arrive(tilee0 + 8 * r.s);
        r.next(kTileRing);
    };

    // What the epilogue will add to a tile, into L2: 32 bytes a lane.  (Asked
    // for by the scale warp as it opens a tile: the product above with bias
    // and residual takes 150 us; 164 where the epilogue asks a tile ahead, 189
    // where a warp of its own asks as early as it can, 200 unasked.)
    auto prefetch_residual = [&](const Tile &t) {
        const int bytes = p.residual_dtype == CSF_F32 ? 4 : 2;
        const int sectors = 128 * bytes / 32, per = 32 / sectors, sec = lane % sectors;
        const int f = t.rt * 128 + sec * (32 / bytes);
        const char *at = static_cast<const char *>(p.residual) + ((t.slot + (int64_t)(lane / sectors)) * p.residual_stride + f) * bytes;
        for (int r = lane / sectors; r < t.n; r += per, at += per * p.residual_stride * bytes)
            if (f < p.F) tc::prefetch_l2(at);
    };

    // Scales of the x rows, by one warp or by several (32 rows in turn each).
    // 16 bytes of a row are four scale tiles: one stage (NVFP4) or four
    // (MXFP8).  A unit is 32 bytes of each row where registers and stages
    // allow, else 16.  The next one, of the next tile where this one ends, is
    // under way before this one waits for its stages (gate/up experts of 64
    // slots: 88 us, 99 with the load after the wait).
    auto x_scale_role = [&](auto warps, const int which) {
        constexpr int kWarps = decltype(warps)::value, kRows = ((kAccCols + 31) / 32 + kWarps - 1) / kWarps;
        constexpr int kParts = kNv && kRows <= 4 ? 2 : 1;
        const int units = unit1 - unit0;              // of 16 bytes
        uint4 next[kRows][kParts];
        int next_n = -1, next_stages = 0;             // its slots (-1: nothing yet, 0: no more tiles) and stages
        Ring ring, tr;
        Tile t;
        const uint4 *src[kRows];
        int u = units;
        bool more = true;
        auto open = [&]() {
            if (!__all_sync(0xFFFFFFFFu, take(tr, t))) return false;
#pragma unroll
            for (int j = 0; j < kRows; ++j) {
                const int c = 32 * (j * kWarps + which) + lane;
                src[j] = reinterpret_cast<const uint4 *>(p.x_scales + (c < t.n ? sh.x_row[tr.s][c] * p.x_scale_stride : 0)) + unit0;
            }
            __syncwarp();
            if (lane == 0) tc::bar_arrive(tilee0 + 8 * tr.s);
            tr.next(kTileRing);
            if (RES && p.residual) prefetch_residual(t);
            return true;
        };
        while (next_n != 0) {
            const int n = next_n, stages = next_stages;
            uint4 now[kRows][kParts];
#pragma unroll
            for (int j = 0; j < kRows; ++j)
#pragma unroll
                for (int h = 0; h < kParts; ++h) now[j][h] = next[j][h];
            if (more && u >= units) more = open(), u = 0;
            next_n = more ? t.n : 0;
            if (more) {
                next_stages = min(kParts * kStagesPer16, ksteps - u * kStagesPer16);
#pragma unroll
                for (int j = 0; j < kRows; ++j)
#pragma unroll
                    for (int h = 0; h < kParts; ++h)
                        if (32 * (j * kWarps + which) < t.n && u + h < units) next[j][h] = __ldg(src[j] + u + h);
                u += kParts;
            }
            bool ok = true;
#pragma unroll
            for (int q = 0; q < kParts * kStagesPer16; ++q) {
                if (n < 0 || q >= stages) break;
                ok = __all_sync(0xFFFFFFFFu, tc::bar_wait(empty0 + 8 * ring.s, ring.parity ^ 1u, abort));
                if (!ok) break;
                const uint32_t dst = ring0 + ring.s * p.stage_bytes + sfb_off + lane * 16u;
#pragma unroll
                for (int j = 0; j < kRows; ++j) {
                    const int block = j * kWarps + which;      // of 32 rows
                    if (32 * block < n) {
                        const uint4 v = now[j][q / kStagesPer16];
                        const uint32_t to = dst + (block >> 2) * (kTilesPerStage * 512u) + (block & 3) * 4u;
                        if constexpr (kNv) {
                            tc::store_shared(to, v.x);
                            tc::store_shared(to + 512u, v.y);
                            tc::store_shared(to + 1024u, v.z);
                            tc::store_shared(to + 1536u, v.w);
                        } else {
                            tc::store_shared(to, q % 4 == 0 ? v.x : q % 4 == 1 ? v.y : q % 4 == 2 ? v.z : v.w);
                        }
                    }
                }
                __syncwarp();
                if (lane == 0) tc::bar_arrive(full0 + 8 * ring.s);
                ring.next(p.stages);
            }
            if (!ok) break;
        }
    };

    if (warp == 15) {
        // ---- tiles and their x rows ----
        Ring tr;
        bool bad_row = false;
        for (uint32_t tile = tile0;; tile += tile_step) {
            Tile t = {};
            if (tile < total) t = find_tile(p, first, slot0, tile, lane);
            if (!__all_sync(0xFFFFFFFFu, tc::bar_wait(tilee0 + 8 * tr.s, tr.parity ^ 1u, abort))) break;
            // columns past the tile's slots repeat its last row
            for (int c = lane; c < ((t.n + 15) & ~15); c += 32) {
                const int64_t s = (int64_t)t.slot + min(c, t.n - 1);
                const int64_t v = ROWS ? (int64_t)p.rows[s] : s;
                const int32_t r = v < 0 || v >= p.x_rows ? 0 : (int32_t)v;
                bad_row |= r != v;
                sh.x_row[tr.s][c] = r;
            }
            if (lane == 0) sh.tile[tr.s] = t;
            __syncwarp();
            if (lane == 0) tc::bar_arrive(tilef0 + 8 * tr.s);
            tr.next(kTileRing);
            if (tile >= total) break;
        }
        if (bad_row && p.err) atomicOr(p.err, CSF_DEV_ERR_CORRUPT);
    } else if (warp == 0) {
        // ---- weights and their scales ----
        if (tc::elect_one()) {
            Ring ring, tr;
            Tile t;
            bool ok = true;
            while (ok && take(tr, t)) {
                done_with(tr);
                const int row = t.rt * 128;
                const uint8_t *sf = p.w_scales + (int64_t)t.e * p.w_scale_expert + ((int64_t)t.rt * p.ncb + k0 * kTilesPerStage) * 512;
                int left = left0;
                for (int k = 0; k < ksteps; ++k, left -= kTilesPerStage, sf += kTilesPerStage * 512, ring.next(p.stages)) {
                    ok = tc::bar_wait(empty0 + 8 * ring.s, ring.parity ^ 1u, abort);
                    if (!ok) break;
                    const uint32_t base = ring0 + ring.s * p.stage_bytes, bar = full0 + 8 * ring.s;
                    const uint32_t bytes = (uint32_t)min(kTilesPerStage, left) * 512u;
                    tc::bar_expect(bar, (uint32_t)AT * (kACopied + bytes));
#pragma unroll
                    for (int a = 0; a < AT; ++a) {
                        tc::tma_load_3d(base + a * kABytes, &wmap, (k0 + k) * (kNv ? 128 : kStepK), row + a * p.second, t.e, bar);
                        tc::bulk_load(base + sfa_off + a * kTilesPerStage * 512u, sf + (int64_t)a * (p.second >> 7) * p.ncb * 512, bytes, bar);
                    }
                }
            }
        }
        __syncwarp();
    } else if (warp == 2 || warp == 3 || warp == 12 || warp == 13) {
        // ---- x rows ----
        if constexpr (!ROWS) {
            if (warp == 2 && tc::elect_one()) {
                Ring ring, tr;
                Tile t;
                bool ok = true;
                while (ok && take(tr, t)) {
                    done_with(tr);
                    for (int k = 0; k < ksteps; ++k, ring.next(p.stages)) {
                        ok = tc::bar_wait(empty0 + 8 * ring.s, ring.parity ^ 1u, abort);
                        if (!ok) break;
                        const uint32_t base = ring0 + ring.s * p.stage_bytes + b_off, bar = full0 + 8 * ring.s;
                        tc::bar_expect(bar, (uint32_t)((t.n + kXBox - 1) / kXBox) * (kXBox * 128u));
                        for (int c = 0; c < t.n; c += kXBox) tc::tma_load_2d(base + c * 128u, &xmap, (k0 + k) * 128, (int)t.slot + c, bar);
                    }
                }
            }
            __syncwarp();
            // The other copying warps share the scales: one alone was late for
            // short stages (512 experts of 64 slots, 2048 x 800: 108 us, 116
            // alone).  Not with a residual: there the epilogue is the bound,
            // and warps that share its schedulers slow it (164 us, 173).
            if constexpr (kScaleWarps > 1) {
                if (warp != 2) x_scale_role(std::integral_constant<int, kScaleWarps>{}, warp == 3 ? 0 : warp - 11);
            }
        } else {
        const int xw = warp < 4 ? warp - 2 : warp - 10;
        const int piece = lane & 7, sub = lane >> 3;      // 8 lanes a row, 4 rows a copy; every fourth group of 4 rows
        const int code_bytes = kNv ? p.K / 2 : p.K;
        const uint32_t r8 = (uint32_t)(4 * (xw & 1) + sub);   // row mod 8
        // row r's 16-byte piece q lies at piece q ^ (r % 8) of its 128 bytes
        const uint32_t b_dst = b_off + (uint32_t)(4 * xw + sub) * 128u + (((uint32_t)piece ^ r8) << 4);
        constexpr int kCopies = kAccCols / 16;
        const int at0 = k0 * 128 + 16 * piece;
        Ring ring, tr;
        Tile t;
        bool ok = true;
        while (ok && __all_sync(0xFFFFFFFFu, take(tr, t))) {
            const uint8_t *src[kCopies];
#pragma unroll
            for (int j = 0; j < kCopies; ++j)
                src[j] = p.x_codes + (16 * j < t.n ? sh.x_row[tr.s][16 * j + 4 * xw + sub] * p.x_code_stride : 0) + at0;
            __syncwarp();
            if (lane == 0) tc::bar_arrive(tilee0 + 8 * tr.s);
            tr.next(kTileRing);
            const int copies = (t.n + 15) >> 4;
            int at = at0;
            for (int k = 0; k < ksteps; ++k, at += 128, ring.next(p.stages)) {
                ok = __all_sync(0xFFFFFFFFu, tc::bar_wait(empty0 + 8 * ring.s, ring.parity ^ 1u, abort));
                if (!ok) break;
                const uint32_t dst = ring0 + ring.s * p.stage_bytes + b_dst;
                const bool live = at < code_bytes;
#pragma unroll
                for (int j = 0; j < kCopies; ++j) {
                    if (j < copies) tc::cp_async16(dst + j * 2048u, src[j], live);
                    src[j] += 128;
                }
                tc::cp_async_arrive(full0 + 8 * ring.s);
            }
        }
        }
    } else if (warp == 14) {
        x_scale_role(std::integral_constant<int, kScaleWarps>{}, kScaleWarps - 1);
    } else if (warp == 1) {
        // ---- matrix instructions ----
        if (tc::elect_one()) {
            // Instruction descriptor: operand types, scale type, N / 8, M / 128.
            const uint32_t idesc0 = kNv ? (1u << 7) | (1u << 10) | (1u << 27) : (5u << 7) | (0u << 10) | (1u << 23) | (1u << 27);
            Ring ring, tr;
            Tile t;
            uint32_t nth = 0;
            bool ok = true;
            const uint32_t sfb = tmem + kSfBase, sfa = tmem + kSfA;
            while (ok && take(tr, t)) {
                done_with(tr);
                const uint32_t set = nth & 1u, aph = (nth >> 1) & 1u;
                ++nth;
                const uint32_t idesc = idesc0 | ((uint32_t)((t.n + 15) >> 4) << 18);
                const bool wide = t.n > 128;
                ok = tc::bar_wait(acce0 + 8 * set, aph ^ 1u, abort);
                tc::fence_after();
                const uint32_t d0 = tmem + set * (AT * kAccCols);
                int left = left0;
                for (int k = 0; ok && k < ksteps; ++k, left -= kTilesPerStage, ring.next(p.stages)) {
                    ok = tc::bar_wait(full0 + 8 * ring.s, ring.parity, abort);
                    if (!ok) break;
                    tc::fence_async_proxy();     // x and its scales came by ordinary stores and copies
                    const uint32_t base = ring0 + ring.s * p.stage_bytes;
                    const uint64_t sb = tc::desc_plain(base + sfb_off), sa = tc::desc_plain(base + sfa_off);
                    const uint64_t bd = tc::desc_sw128(base + b_off), ad = tc::desc_sw128(base);
                    auto issue = [&](int tiles) {
#pragma unroll
                        for (int i = 0; i < kTilesPerStage; ++i) {
                            if (i < tiles) {
                                // tensor-memory columns of an operand's scales: a k tile's 128-row blocks side by side
                                tc::copy_scales(sfb + 4 * kRowBlocks * i, sb + i * 32);
                                if (kRowBlocks > 1 && wide) tc::copy_scales(sfb + 4 * kRowBlocks * i + 4, sb + (kTilesPerStage + i) * 32);
#pragma unroll
                                for (int a = 0; a < AT; ++a)
                                    tc::copy_scales(sfa + a * kSfCols + 4 * i, sa + (a * kTilesPerStage + i) * 32);
                            }
                        }
#pragma unroll
                        for (int a = 0; a < AT; ++a) {
                            const uint32_t d = d0 + a * kAccCols;
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                if constexpr (kNv) {
                                    if (i < tiles)
                                        tc::mma_nvfp4(d, ad + a * (kABytes >> 4) + 2 * i, bd + 2 * i, idesc, sfa + a * kSfCols + 4 * i,
                                                      sfb + 4 * kRowBlocks * i, (k | i) != 0);
                                } else {
                                    tc::mma_mxf8(d, ad + a * (kABytes >> 4) + 2 * i, bd + 2 * i,
                                                 idesc | ((uint32_t)i << 29) | ((uint32_t)i << 4), sfa + a * kSfCols, sfb, (k | i) != 0);
                                }
                            }
                        }
                    };
                    if (left >= kTilesPerStage) issue(kTilesPerStage);
                    else issue(left);
                    tc::commit(empty0 + 8 * ring.s);
                    if (k + 1 == ksteps) tc::commit(accf0 + 8 * set);
                }
            }
        }
        __syncwarp();
    } else {
        // ---- epilogue ----
        // Warps w and w + 4 read the same 32 weight rows and take every other
        // 8 G slots.  One rolled loop: longer code ran out of the instruction
        // cache.
        constexpr int G = kGroups;
        const int w = (warp - 4) & 3, half = (warp - 4) >> 2;
        const int part = lane & 3, sub = lane >> 2;           // after the turn: 8 columns of a slot
        float *buf = turn[warp - 4];
        float tensor_scale = 1.f;
        if constexpr (OUT == kOutNv) {
            if (p.out_tensor_scale) tensor_scale = *p.out_tensor_scale;
        }
        constexpr int kOutBytes = OUT == kOutF32 ? 4 : OUT == kOutBf16 || OUT == kOutF16 ? 2 : 1;
        const int res_bytes = p.residual_dtype == CSF_F32 ? 4 : 2;
        const int64_t out_8 = 8 * p.out_stride * kOutBytes, res_8 = 8 * p.residual_stride * res_bytes, srow_8 = 8 * p.out_scale_stride;
        // What a tile needs before its first round, fetched a tile ahead.
        struct Head {
            Tile t;
            Raw8 res[G];
            float alpha, rs[G];
            uint32_t bias[AT];      // as stored
        };
        Ring tr;
        if (SHARED && rank > 0) {
            // Not the tile's first block: its sums go there.  (Each cluster
            // has one tile at most.)
            Tile t;
            if (__all_sync(0xFFFFFFFFu, take(tr, t)) && __all_sync(0xFFFFFFFFu, tc::bar_wait(accf0, 0, abort))) {
                tc::fence_after();
                const uint32_t d = tmem + ((uint32_t)(32 * w) << 16) + 8 * half;
#pragma unroll
                for (int a = 0; a < AT; ++a) {
                    float acc[8];
                    tc::tmem_load(d + a * kAccCols, acc);
                    tc::wait_ld();
                    float *at = sums + (((rank - 1) * AT + a) * kSplitSlots + 8 * half) * 128 + 32 * w + lane;
                    const uint32_t to = tc::in_block(tc::smem_u32(at), 0);
#pragma unroll
                    for (int j = 0; j < 8; ++j) tc::store_cluster(to + j * 512u, acc[j]);
                }
                tc::bar_arrive_cluster(tc::in_block(tc::smem_u32(&sh.sums_full), 0));
            }
        }
        auto open = [&](Head &h) {
            if ((SHARED && rank > 0) || !__all_sync(0xFFFFFFFFu, take(tr, h.t))) {
                h.t.n = 0;
                return;
            }
            __syncwarp();
            if (lane == 0) tc::bar_arrive(tilee0 + 8 * tr.s);
            tr.next(kTileRing);
            const int row = h.t.rt * 128 + 32 * w, f = row + 8 * part;
#pragma unroll
            for (int i = 0; i < G; ++i) {
                const int c = 8 * G * half + 8 * i + sub;
                if (RES && p.residual && c < h.t.n)
                    h.res[i] = load_raw8(static_cast<const char *>(p.residual) + (((int64_t)h.t.slot + c) * p.residual_stride + f) * res_bytes,
                                         p.residual_dtype, p.F - f, p.residual_wide);
                if (RES && p.row_scale && c < h.t.n) h.rs[i] = p.row_scale[(int64_t)h.t.slot + c];
            }
            if (p.alpha) h.alpha = p.alpha[h.t.e];
#pragma unroll
            for (int a = 0; a < AT; ++a) {
                const int r = row + lane + a * p.second;
                if (p.bias && r < p.N) h.bias[a] = load_raw(p.bias, (int64_t)h.t.e * p.N + r, p.bias_dtype);
            }
        };
        uint32_t nth = 0;
        Head next = {};
        next.alpha = 1.f;
#pragma unroll
        for (int i = 0; i < G; ++i) next.rs[i] = 1.f;
        open(next);
        for (; next.t.n > 0; ++nth) {
            const Tile t = next.t;
            const uint32_t set = nth & 1u, aph = (nth >> 1) & 1u;
            const int f = t.rt * 128 + 32 * w + 8 * part;
            const int64_t slot = (int64_t)t.slot + 8 * G * half + sub;     // the first of this lane's slots
            const char *res_at = static_cast<const char *>(p.residual) + (slot * p.residual_stride + f) * res_bytes;
            const float *scale_at = p.row_scale + slot;
            char *out_at = static_cast<char *>(p.out) + slot * p.out_stride * kOutBytes + (OUT == kOutNv || OUT == kOutMx ? 0 : (int64_t)f * kOutBytes);
            uint8_t *srow = p.out_scales + slot * p.out_scale_stride;
            int c = 8 * G * half;
            Raw8 res[G];
            float rs[G];
#pragma unroll
            for (int i = 0; i < G; ++i) res[i] = next.res[i], rs[i] = next.rs[i];
            const float alpha = next.alpha;
            float bias[AT];
#pragma unroll
            for (int a = 0; a < AT; ++a) bias[a] = raw_as_float(next.bias[a], p.bias_dtype);
            open(next);
            const bool ok = tc::bar_wait(accf0 + 8 * set, aph, abort);
            if (!__all_sync(0xFFFFFFFFu, ok)) break;
            tc::fence_after();
            uint32_t d = tmem + set * (AT * kAccCols) + ((uint32_t)(32 * w) << 16) + c;
            if (c >= t.n) tc::bar_arrive(acce0 + 8 * set);     // no slots of this tile are this warp's
#pragma unroll 1
            for (; c < t.n; c += 16 * G, d += 16 * G) {
                float acc[AT][8 * G];
#pragma unroll
                for (int a = 0; a < AT; ++a) tc::tmem_load(d + a * kAccCols, acc[a]);
                tc::wait_ld();
                if constexpr (SHARED) {
                    if (!__all_sync(0xFFFFFFFFu, tc::bar_wait<true>(tc::smem_u32(&sh.sums_full), 0, abort))) break;
                    for (uint32_t r = 0; r + 1 < split; ++r) {
#pragma unroll
                        for (int a = 0; a < AT; ++a)
#pragma unroll
                            for (int j = 0; j < 8 * G; ++j)
                                acc[a][j] += sums[((r * AT + a) * kSplitSlots + c + j) * 128 + 32 * w + lane];
                    }
                }
                if (c + 16 * G >= t.n) {
                    tc::fence_before();
                    tc::bar_arrive(acce0 + 8 * set);
                }
                __syncwarp();      // the last round's reads
                auto turn_in = [&](auto act) {
#pragma unroll
                    for (int j = 0; j < 8 * G; ++j) {
                        float y = act(fmaf(acc[0][j], alpha, bias[0]));
                        if constexpr (GATED) y *= fmaf(acc[AT - 1][j], alpha, bias[AT - 1]);
                        buf[j * kTurnStride + lane] = y;
                    }
                };
                if (p.act == CSF_ACT_SILU || p.act == CSF_ACT_GELU_TANH) {
                    const bool gelu = p.act == CSF_ACT_GELU_TANH;
                    turn_in([&](float v) { return smooth(v, gelu); });
                } else {
                    const float least = p.act == CSF_ACT_RELU ? 0.f : __int_as_float(0xFF800000);
                    turn_in([&](float v) { return v < least ? least : v; });
                }
                __syncwarp();
#pragma unroll
                for (int i = 0; i < G; ++i) {
                    const float4 *from = reinterpret_cast<const float4 *>(buf + (8 * i + sub) * kTurnStride + 8 * part);
                    const float4 lo = from[0], hi = from[1];
                    float y[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
                    const int j = c + 8 * i + sub;
                    const bool more = j + 16 * G < t.n;
                    if (RES && p.row_scale) {
#pragma unroll
                        for (int q = 0; q < 8; ++q) y[q] *= rs[i];
                        if (more) rs[i] = scale_at[8 * i + 16 * G];
                    }
                    if (RES && p.residual) {
                        add_raw8(y, res[i], p.residual_dtype);
                        if (more) res[i] = load_raw8(res_at + (i + 2 * G) * res_8, p.residual_dtype, p.F - f, p.residual_wide);
                    }
                    emit8<OUT>(p, y, f, out_at + i * out_8, srow + i * srow_8, j < t.n, tensor_scale);
                }
                scale_at += 16 * G;
                res_at += 2 * G * res_8;
                out_at += 2 * G * out_8;
                srow += 2 * G * srow_8;
            }
        }
    }

    // A wait that gave up: let copies and products in flight land before the
    // block's memory goes.
    tc::fence_before();      // the last tensor-memory reads, before they are freed
    __syncthreads();
    tc::fence_after();
    if (sh.abort) {
        if (tid == 0 && p.err) atomicOr(p.err, CSF_DEV_ERR_TIMEOUT);
        const uint64_t t0 = tc::timer_ns();
        while (tc::timer_ns() - t0 < 5000000ull) __nanosleep(1000);
        __syncthreads();
    }
    if constexpr (SHARED) tc::cluster_sync();      // nothing is under way to a block that leaves
    if (warp == 1) tc::tmem_free(tmem, kTmemCols);
}

using Kernel = void (*)(CUtensorMap, CUtensorMap, MmParams);

template <int KIND, bool ROWS, int OUT>
Kernel pick(int shape, bool res) {
    switch (shape) {
        case kNarrow: return res ? expert_matmul_kernel<KIND, ROWS, kNarrow, true, OUT> : expert_matmul_kernel<KIND, ROWS, kNarrow, false, OUT>;
        case kWide: return res ? expert_matmul_kernel<KIND, ROWS, kWide, true, OUT> : expert_matmul_kernel<KIND, ROWS, kWide, false, OUT>;
        case kGated: return res ? expert_matmul_kernel<KIND, ROWS, kGated, true, OUT> : expert_matmul_kernel<KIND, ROWS, kGated, false, OUT>;
        // for these the residual is asked for at run time: their epilogues are short
        case kNarrowShared: return expert_matmul_kernel<KIND, ROWS, kNarrowShared, true, OUT>;
        default: return expert_matmul_kernel<KIND, ROWS, kGatedShared, true, OUT>;
    }
}

template <int KIND, bool ROWS>
Kernel pick_kernel(int out, int shape, bool res) {
    switch (out) {
        case kOutBf16: return pick<KIND, ROWS, kOutBf16>(shape, res);
        case kOutF16: return pick<KIND, ROWS, kOutF16>(shape, res);
        case kOutF32: return pick<KIND, ROWS, kOutF32>(shape, res);
        case kOutNv: return pick<KIND, ROWS, kOutNv>(shape, res);
        default: return pick<KIND, ROWS, kOutMx>(shape, res);
    }
}

// The kernel for a kind of x, an output, a shape and a residual's presence
// (one translation unit a kind and an indexing of x).
Kernel nvfp4_kernel(int out, int shape, bool res);
Kernel nvfp4_rows_kernel(int out, int shape, bool res);
Kernel mxfp8_kernel(int out, int shape, bool res);
Kernel mxfp8_rows_kernel(int out, int shape, bool res);

}  // namespace mm
}  // namespace csfk
