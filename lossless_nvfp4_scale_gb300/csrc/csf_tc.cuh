// PTX wrappers for the tensor-core kernels: mbarriers with bounded waits, TMA
// loads, tensor memory and block-scaled tcgen05 instructions.  Internal to
// the library.
#pragma once

#include <cstdint>

namespace csfk {
namespace tc {

__device__ __forceinline__ uint32_t smem_u32(const void *p) { return (uint32_t)__cvta_generic_to_shared(p); }

__device__ __forceinline__ uint64_t timer_ns() {
    uint64_t t;
    asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t));
    return t;
}

// One thread of the warp, known to the compiler as one: what it issues needs
// no loop over lanes.
__device__ __forceinline__ bool elect_one() {
    uint32_t is;
    asm volatile(
        "{\n .reg .pred p;\n elect.sync _|p, 0xFFFFFFFF;\n selp.u32 %0, 1, 0, p;\n}"
        : "=r"(is));
    return is != 0;
}

// ---- mbarriers ----------------------------------------------------------------------------------------------------

__device__ __forceinline__ void bar_init(uint32_t bar, uint32_t count) {
    asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(count) : "memory");
}

__device__ __forceinline__ void bar_arrive(uint32_t bar) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}

__device__ __forceinline__ void bar_expect(uint32_t bar, uint32_t bytes) {
    asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes) : "memory");
}

__device__ __forceinline__ bool bar_try(uint32_t bar, uint32_t parity) {
    uint32_t done;
    asm volatile(
        "{\n .reg .pred p;\n"
        " mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n"
        " selp.u32 %0, 1, 0, p;\n}"
        : "=r"(done)
        : "r"(bar), "r"(parity)
        : "memory");
    return done != 0;
}

// The same for a barrier that other blocks of the cluster arrive on: what they
// wrote before is visible after.
__device__ __forceinline__ bool bar_try_cluster(uint32_t bar, uint32_t parity) {
    uint32_t done;
    asm volatile(
        "{\n .reg .pred p;\n"
        " mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n"
        " selp.u32 %0, 1, 0, p;\n}"
        : "=r"(done)
        : "r"(bar), "r"(parity)
        : "memory");
    return done != 0;
}

constexpr uint64_t kWaitLimitNs = 2000000000ull;   // a wait that lasts this long gives up

// Whether a wait that began at t0 (0: now) goes on: its start, or 0 to give up,
// after the limit or because another thread of the block did (*abort).  Apart
// from the waits: inlined in each it made the products' kernel a tenth
// longer, which its instruction fetches feel.
static __device__ __noinline__ uint64_t keep_waiting(uint64_t t0, volatile uint32_t *abort) {
    if (*abort) return 0;
    const uint64_t t = timer_ns();
    if (t0 == 0) return t;
    if (t - t0 <= kWaitLimitNs) return t0;
    *abort = 1;
    return 0;
}

// Wait for a phase, or give up.  A false return means the caller stops.
template <bool CLUSTER = false>
__device__ __forceinline__ bool bar_wait(uint32_t bar, uint32_t parity, volatile uint32_t *abort) {
    uint64_t t0 = 0;
    do {
#pragma unroll 1
        for (int i = 0; i < 64; ++i)
            if (CLUSTER ? bar_try_cluster(bar, parity) : bar_try(bar, parity)) return true;
        t0 = keep_waiting(t0, abort);
    } while (t0 != 0);
    return false;
}

// The same with nothing but the barrier's answer in the way of a phase that
// is there already: the loop above took 180 cycles then, in a warp alone on
// its scheduler, and this takes 57.
static __device__ __noinline__ bool bar_wait_on(uint32_t bar, uint32_t parity, volatile uint32_t *abort) {
    return bar_wait(bar, parity, abort);
}

__device__ __forceinline__ bool bar_wait_ready(uint32_t bar, uint32_t parity, volatile uint32_t *abort) {
    if (__builtin_expect(bar_try(bar, parity), 1)) return true;
    return bar_wait_on(bar, parity, abort);
}

// The same without a call, for warps whose registers are full of sums: they
// would be saved around it.
__device__ __forceinline__ bool bar_wait_here(uint32_t bar, uint32_t parity, volatile uint32_t *abort) {
    if (__builtin_expect(bar_try(bar, parity), 1)) return true;
    uint64_t t0 = 0;
#pragma unroll 1
    for (uint32_t i = 0; !bar_try(bar, parity); ++i) {
        if ((i & 63) != 63) continue;
        if (*abort) return false;
        const uint64_t t = timer_ns();
        if (t0 == 0) t0 = t;
        if (t - t0 > kWaitLimitNs) {
            *abort = 1;
            return false;
        }
    }
    return true;
}

// ---- clusters -----------------------------------------------------------------------------------------------------

__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}

// Every thread of every block of the cluster.
__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// A shared-memory address of this block, in the block of that rank.
__device__ __forceinline__ uint32_t in_block(uint32_t addr, uint32_t rank) {
    uint32_t r;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
    return r;
}

__device__ __forceinline__ void store_cluster(uint32_t dst, float v) {
    asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(dst), "f"(v) : "memory");
}

__device__ __forceinline__ uint32_t load_cluster(uint32_t src) {
    uint32_t v;
    asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(src) : "memory");
    return v;
}

__device__ __forceinline__ void bar_arrive_cluster(uint32_t bar) {
    asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}

// One lane's arrival, without a branch that the warp would have to come
// together after.
__device__ __forceinline__ void bar_arrive_if(uint32_t bar, bool is) {
    asm volatile("{\n .reg .pred p;\n setp.ne.u32 p, %1, 0;\n @p mbarrier.arrive.shared::cta.b64 _, [%0];\n}" ::"r"(bar), "r"((uint32_t)is)
                 : "memory");
}

// ---- copies -------------------------------------------------------------------------------------------------------

__device__ __forceinline__ void bulk_load(uint32_t dst, const void *src, uint32_t bytes, uint32_t bar) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
                 "l"(src), "r"(bytes), "r"(bar)
                 : "memory");
}

__device__ __forceinline__ void tma_load_3d(uint32_t dst, const void *map, int x, int y, int z, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], "
        "[%5];" ::"r"(dst),
        "l"(map), "r"(x), "r"(y), "r"(z), "r"(bar)
        : "memory");
}

__device__ __forceinline__ void tma_load_2d(uint32_t dst, const void *map, int x, int y, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
        "l"(map), "r"(x), "r"(y), "r"(bar)
        : "memory");
}

__device__ __forceinline__ void prefetch_l2(const void *p) { asm volatile("prefetch.global.L2 [%0];" ::"l"(p)); }

__device__ __forceinline__ void store_shared(uint32_t dst, uint32_t v) {
    asm volatile("st.shared.u32 [%0], %1;" ::"r"(dst), "r"(v) : "memory");
}

// 16 bytes, past L1; zeros where `live` is false.
__device__ __forceinline__ void cp_async16(uint32_t dst, const void *src, bool live) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(live ? 16 : 0) : "memory");
}

// One arrival on bar (already counted in it) once this thread's copies so far have landed.
__device__ __forceinline__ void cp_async_arrive(uint32_t bar) {
    asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(bar) : "memory");
}

__device__ __forceinline__ void fence_async_proxy() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

// ---- tensor memory and tcgen05 ------------------------------------------------------------------------------------

__device__ __forceinline__ void tmem_alloc(uint32_t result, uint32_t cols) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(result), "r"(cols) : "memory");
}

__device__ __forceinline__ void tmem_free(uint32_t addr, uint32_t cols) {
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(addr), "r"(cols));
}

__device__ __forceinline__ void fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }

// One arrival on bar once every tcgen05 operation this thread issued so far is done.
__device__ __forceinline__ void commit(uint32_t bar) {
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
}

// Shared-memory matrix descriptors: start address, byte offset between 8-row
// groups, descriptor version 1, and the swizzle (2: 128 bytes).
__device__ __forceinline__ uint64_t desc_sw128(uint32_t addr) {
    return (uint64_t)((addr & 0x3FFFFu) >> 4) | (1ull << 16) | ((uint64_t)(1024 >> 4) << 32) | (1ull << 46) | (2ull << 61);
}

__device__ __forceinline__ uint64_t desc_plain(uint32_t addr) {
    return (uint64_t)((addr & 0x3FFFFu) >> 4) | (1ull << 16) | ((uint64_t)(128 >> 4) << 32) | (1ull << 46);
}

// One 512-byte scale tile (CSF_LAYOUT_BLOCKED order) to four tensor-memory
// columns: lane r % 32 of column r / 32 gets row r's four scales, in all four
// lane quarters.
__device__ __forceinline__ void copy_scales(uint32_t taddr, uint64_t desc) {
    asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(desc) : "memory");
}

// D[128 x N] (+)= A * B^T with E2M1 operands, UE4M3 scales per 16, K = 64.
__device__ __forceinline__ void mma_nvfp4(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t sfa, uint32_t sfb,
                                          uint32_t accumulate) {
    asm volatile(
        "{\n .reg .pred p;\n setp.ne.u32 p, %6, 0;\n"
        " tcgen05.mma.cta_group::1.kind::mxf4nvf4.block_scale.scale_vec::4X [%0], %1, %2, %3, [%4], [%5], p;\n}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate)
        : "memory");
}

// The same with 8-bit containers (E2M1 A, E4M3 B), UE8M0 scales per 32, K = 32.
__device__ __forceinline__ void mma_mxf8(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t sfa, uint32_t sfb,
                                         uint32_t accumulate) {
    asm volatile(
        "{\n .reg .pred p;\n setp.ne.u32 p, %6, 0;\n"
        " tcgen05.mma.cta_group::1.kind::mxf8f6f4.block_scale.scale_vec::1X [%0], %1, %2, %3, [%4], [%5], p;\n}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate)
        : "memory");
}

// ---- 8-bit products -----------------------------------------------------------------------------------------------

// What follows is issued by the lane whose `one` is set, in code that the whole
// warp runs: addresses and descriptors then stay in uniform registers, where
// the instructions want them.  (In a branch of one lane's own each operand had
// to be moved there: 160 cycles a step of the loop alone, before any wait.)

__device__ __forceinline__ void tma_load_3d_if(uint32_t one, uint32_t dst, const void *map, int x, int y, int z, uint32_t bar) {
    asm volatile(
        "{\n .reg .pred p;\n setp.ne.u32 p, %6, 0;\n"
        " @p cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];\n}" ::"r"(dst),
        "l"(map), "r"(x), "r"(y), "r"(z), "r"(bar), "r"(one)
        : "memory");
}

__device__ __forceinline__ void tma_load_2d_if(uint32_t one, uint32_t dst, const void *map, int x, int y, uint32_t bar) {
    asm volatile(
        "{\n .reg .pred p;\n setp.ne.u32 p, %5, 0;\n"
        " @p cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];\n}" ::"r"(dst),
        "l"(map), "r"(x), "r"(y), "r"(bar), "r"(one)
        : "memory");
}

__device__ __forceinline__ void bar_expect_if(uint32_t one, uint32_t bar, uint32_t bytes) {
    asm volatile(
        "{\n .reg .pred p;\n setp.ne.u32 p, %2, 0;\n @p mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;\n}" ::"r"(bar),
        "r"(bytes), "r"(one)
        : "memory");
}

// One arrival on bar once every tcgen05 operation this thread issued so far is
// done.
__device__ __forceinline__ void commit_if(uint32_t one, uint32_t bar) {
    asm volatile(
        "{\n .reg .pred p;\n setp.ne.u32 p, %1, 0;\n"
        " @p tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n}" ::"r"(bar),
        "r"(one)
        : "memory");
}

// D[128 x N] = A * B^T with E4M3 operands, K = 128 in four steps, and an
// arrival on bar when they are done.  Descriptors come as their halves, of
// which the low ones advance; all in one piece, since each instruction that the
// loop around it takes waits for its turn among the summing warps'.
__device__ __forceinline__ void mma_f8_128(uint32_t one, uint32_t d, uint32_t a_lo, uint32_t a_hi, uint32_t b_lo, uint32_t b_hi,
                                           uint32_t b_step, uint32_t idesc, uint32_t bar) {
    asm volatile(
            "{\n .reg .pred p, t, f;\n .reg .b32 x;\n .reg .b64 ad, bd;\n setp.ne.u32 p, %8, 0;\n setp.eq.u32 t, %8, %8;\n setp.ne.u32 f, %8, %8;\n"
            " add.u32 x, %1, 0;\n mov.b64 ad, {x, %2};\n mad.lo.u32 x, %5, 0, %3;\n mov.b64 bd, {x, %4};\n"
            " @p tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], ad, bd, %6, f;\n"
            " add.u32 x, %1, 2;\n mov.b64 ad, {x, %2};\n mad.lo.u32 x, %5, 1, %3;\n mov.b64 bd, {x, %4};\n"
            " @p tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], ad, bd, %6, t;\n"
            " add.u32 x, %1, 4;\n mov.b64 ad, {x, %2};\n mad.lo.u32 x, %5, 2, %3;\n mov.b64 bd, {x, %4};\n"
            " @p tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], ad, bd, %6, t;\n"
            " add.u32 x, %1, 6;\n mov.b64 ad, {x, %2};\n mad.lo.u32 x, %5, 3, %3;\n mov.b64 bd, {x, %4};\n"
            " @p tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], ad, bd, %6, t;\n"
            " @p tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%7];\n"
            "}" ::"r"(d),
            "r"(a_lo), "r"(a_hi), "r"(b_lo), "r"(b_hi), "r"(b_step), "r"(idesc), "r"(bar), "r"(one)
            : "memory");
}

// Descriptor of 128 elements of 8 bits a row and rows along the summed index
// (128-byte swizzle): groups of 8 rows 1024 bytes apart, the next 128
// elements 16 KB.
__device__ __forceinline__ uint64_t desc_across(uint32_t addr) {
    return (uint64_t)((addr & 0x3FFFFu) >> 4) | ((uint64_t)(16384 >> 4) << 16) | ((uint64_t)(1024 >> 4) << 32) | (1ull << 46) |
           (2ull << 61);
}

// Columns of this warp's lanes, as they are; wait_ld on them makes what uses
// them come after.
__device__ __forceinline__ void tmem_load(uint32_t taddr, uint32_t (&r)[32]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {"
        "%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, %17, %18, %19, %20, %21, "
        "%22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
          "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]),
          "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]),
          "=r"(r[30]), "=r"(r[31])
        : "r"(taddr));
}

__device__ __forceinline__ void wait_ld(uint32_t (&r)[32]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                   "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]),
                   "+r"(r[14]), "+r"(r[15]), "+r"(r[16]), "+r"(r[17]), "+r"(r[18]), "+r"(r[19]),
                   "+r"(r[20]), "+r"(r[21]), "+r"(r[22]), "+r"(r[23]), "+r"(r[24]), "+r"(r[25]),
                   "+r"(r[26]), "+r"(r[27]), "+r"(r[28]), "+r"(r[29]), "+r"(r[30]), "+r"(r[31])
                 :
                 : "memory");
}

__device__ __forceinline__ void tmem_load(uint32_t taddr, uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, "
        "[%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr));
}

__device__ __forceinline__ void wait_ld(uint32_t (&r)[16]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]), "+r"(r[8]),
                   "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15])
                 :
                 : "memory");
}

__device__ __forceinline__ void tmem_store(uint32_t taddr, const uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
        "%15};" ::"r"(r[0]),
        "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]),
        "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(taddr)
        : "memory");
}

__device__ __forceinline__ void wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// Two sums' d += a * b, each rounded once.  (Volatile: what comes out of tensor
// memory is used after the wait for it, in the order written here.)
__device__ __forceinline__ void fma2_after(uint64_t &d, uint32_t a_lo, uint32_t a_hi, uint64_t b) {
    asm volatile("{\n .reg .b64 a;\n mov.b64 a, {%1, %2};\n fma.rn.f32x2 %0, a, %3, %0;\n}" : "+l"(d) : "r"(a_lo), "r"(a_hi), "l"(b));
}

__device__ __forceinline__ uint64_t twice(float v) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %1};" : "=l"(r) : "f"(v));
    return r;
}

__device__ __forceinline__ void halves(uint64_t v, float &lo, float &hi) { asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v)); }

// Whether a phase is there, asked by one lane alone: the barriers answer the
// lanes one after the other.
__device__ __forceinline__ bool bar_try_if(uint32_t bar, uint32_t parity, bool is) {
    uint32_t done;
    asm volatile(
        "{\n .reg .pred p, q;\n setp.ne.u32 q, %3, 0;\n setp.ne.u32 p, %3, %3;\n"
        " @q mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n"
        " selp.u32 %0, 1, 0, p;\n}"
        : "=r"(done)
        : "r"(bar), "r"(parity), "r"((uint32_t)is)
        : "memory");
    return done != 0;
}

// A named barrier of `threads` threads.
__device__ __forceinline__ void named_sync(uint32_t id, uint32_t threads) {
    asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
}

__device__ __forceinline__ void store_cluster4(uint32_t dst, float a, float b, float c, float d) {
    asm volatile("st.shared::cluster.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(dst), "f"(a), "f"(b), "f"(c), "f"(d) : "memory");
}

// 8 columns of this warp's 32 lanes.
__device__ __forceinline__ void tmem_load(uint32_t taddr, float (&v)[8]) {
    uint32_t r[8];
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
                 : "r"(taddr));
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(r[i]);
}

// 16 columns.
__device__ __forceinline__ void tmem_load(uint32_t taddr, float (&v)[16]) {
    uint32_t r[16];
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, "
        "[%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr));
#pragma unroll
    for (int i = 0; i < 16; ++i) v[i] = __uint_as_float(r[i]);
}

}  // namespace tc
}  // namespace csfk
