// Host side of csf_expert_matmul: argument checks, tensor maps, the choice of
// a kernel and its launch.
#include <algorithm>
#include <atomic>
#include <cstring>
#include <mutex>
#include <set>

#include "csf_experts.cuh"
#include "csf_host.cuh"

namespace csfk {
namespace mm {
namespace {

csf_status check(const csf_expert_matmul_args *a) {
    if (!a) return CSF_ERR_ARG;
    if (!rows_valid(a->x) || a->experts < 1 || a->n < 1 || a->slots < 0) return CSF_ERR_ARG;
    if (a->act < CSF_ACT_NONE || a->act > CSF_ACT_GELU_TANH) return CSF_ERR_ARG;
    if (a->experts > kMmMaxExperts || a->slots >= (1ll << 31) || a->x.rows >= (1ll << 31)) return CSF_ERR_UNSUPPORTED;
    if (a->n > INT32_MAX - 255 || a->x.cols > INT32_MAX - 511) return CSF_ERR_UNSUPPORTED;      // whole tiles of them count in 32 bits
    if (a->x.cols % (a->x.kind == CSF_ROWS_NVFP4 ? 32 : 128) || (a->gated && a->n % 256)) return CSF_ERR_UNSUPPORTED;
    if (!a->expert_start && a->experts != 1) return CSF_ERR_ARG;
    if (!a->rows && a->slots > a->x.rows) return CSF_ERR_ARG;
    if (a->slots == 0) return CSF_OK;
    if (a->x.rows == 0) return CSF_ERR_ARG;
    if (!a->w || !a->w_scales || !aligned_to(a->w, 32) || !aligned_to(a->w_scales, 16)) return CSF_ERR_ARG;
    const int32_t F = a->gated ? a->n / 2 : a->n;
    if (!aligned_to(a->rows, 4) || !aligned_to(a->expert_start, a->expert_start_is_int64 ? 8 : 4)) return CSF_ERR_ARG;
    if (!aligned_to(a->alpha, 4) || !aligned_to(a->row_scale, 4) || !aligned_to(a->error_word, 4)) return CSF_ERR_ARG;
    if (a->bias && (!dtype_known(a->bias_dtype) || !aligned_to(a->bias, dtype_bytes(a->bias_dtype)))) return CSF_ERR_ARG;
    if (a->residual && (!dtype_known(a->residual_dtype) || a->residual_stride < F ||
                        !aligned_to(a->residual, dtype_bytes(a->residual_dtype))))
        return CSF_ERR_ARG;
    if (a->out) {
        if (!dtype_known(a->out_dtype) || a->out_stride < F || !aligned_to(a->out, dtype_bytes(a->out_dtype))) return CSF_ERR_ARG;
    } else if (!rows_valid(a->out_rows) || a->out_rows.cols != F || a->out_rows.rows != a->slots ||
               !aligned_to(a->out_rows.tensor_scale, 4)) {
        return CSF_ERR_ARG;
    }
    return CSF_OK;
}

}  // namespace
}  // namespace mm

EncodeFn encode_fn() {
    static EncodeFn fn = [] {
        void *f = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12080, cudaEnableDefault, &q) != cudaSuccess ||
            q != cudaDriverEntryPointSuccess) {
            cudaGetLastError();
            f = nullptr;
        }
        return reinterpret_cast<EncodeFn>(f);
    }();
    return fn;
}

// (The standard library may throw; the C entry must not.)
bool allow_smem(const void *kernel, int limit, int least_regs) noexcept {
    static std::mutex mu;
    static std::set<std::pair<const void *, int>> done;
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) {
        cudaGetLastError();
        return false;
    }
    try {
        std::lock_guard<std::mutex> lock(mu);
        if (done.count({kernel, dev})) return true;
        cudaFuncAttributes attr;
        if (cudaFuncGetAttributes(&attr, kernel) != cudaSuccess || attr.numRegs < least_regs ||
            cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 limit - (int)round_up(attr.sharedSizeBytes, 1024)) != cudaSuccess) {
            cudaGetLastError();
            return false;
        }
        done.insert({kernel, dev});
    } catch (...) {
        return false;
    }
    return true;
}

int sm_count() {
    static std::atomic<int> counts[64];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) {
        cudaGetLastError();
        return 0;
    }
    if (counts[dev] == 0) {
        int n = 0;
        if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) {
            cudaGetLastError();
            return 0;
        }
        counts[dev] = n;
    }
    return counts[dev];
}

}  // namespace csfk

using namespace csfk;
using namespace csfk::mm;

extern "C" csf_status csf_expert_matmul(const csf_expert_matmul_args *a, void *stream) {
    csf_status st = check(a);
    if (st != CSF_OK || a->slots == 0) return st;
    const bool nv = a->x.kind == CSF_ROWS_NVFP4;
    const int32_t K = a->x.cols, N = a->n, E = a->experts;
    const int at = a->gated ? 2 : 1;

    MmParams p;
    std::memset(&p, 0, sizeof(p));
    p.x_codes = a->x.codes;
    p.x_code_stride = a->x.code_stride;
    p.x_scales = a->x.scales;
    p.x_scale_stride = a->x.scale_stride;
    const int32_t C = K / (nv ? 16 : 32);
    p.ncb = (C + 3) / 4;
    p.w_scales = a->w_scales;
    p.w_scale_expert = round_up(N, 128) * 4 * p.ncb;
    p.rows = a->rows;
    p.start = a->expert_start;
    p.es64 = a->expert_start_is_int64;
    p.alpha = a->alpha;
    p.bias = a->bias;
    p.bias_dtype = a->bias_dtype;
    p.row_scale = a->row_scale;
    p.residual = a->residual;
    p.residual_stride = a->residual_stride;
    p.residual_dtype = a->residual_dtype;
    p.residual_wide = a->residual && aligned_to(a->residual, 16) &&
                      (a->residual_stride * (int64_t)dtype_bytes(a->residual_dtype)) % 16 == 0;
    p.err = a->error_word;
    p.slots = a->slots;
    p.x_rows = (int32_t)a->x.rows;
    p.E = E;
    p.N = N;
    p.K = K;
    p.F = a->gated ? N / 2 : N;
    p.act = a->act;
    int out;
    if (a->out) {
        out = a->out_dtype;
        p.out_wide = aligned_to(a->out, 16) && (a->out_stride * (int64_t)dtype_bytes(out)) % 16 == 0;
        p.out = a->out;
        p.out_stride = a->out_stride;
    } else {
        out = a->out_rows.kind == CSF_ROWS_NVFP4 ? kOutNv : kOutMx;
        p.out = a->out_rows.codes;
        p.out_stride = a->out_rows.code_stride;
        p.out_scales = a->out_rows.scales;
        p.out_scale_stride = a->out_rows.scale_stride;
        p.out_tensor_scale = a->out_rows.tensor_scale;
    }
    p.second = a->gated ? N / 2 : 128;
    p.row_tiles = a->gated ? N / 256 : (N + 127) / 128;
    p.row_tiles_magic = (uint32_t)((1ull << 32) / (uint32_t)p.row_tiles + 1);
    // Wide tiles where the experts' slots fill more than a narrow one on
    // average: a dense 8191-slot product takes 79 us in wide tiles and 94 in
    // narrow ones, 512 experts of 64 slots (2048 x 800 NVFP4) 138 and 119.
    const int64_t mean = a->slots / std::min<int64_t>(E, a->slots);
    int shape = a->gated ? kGated : mean > tile_slots(kNarrow) ? kWide : kNarrow;
    p.nt = (int)std::min<int64_t>(tile_slots(shape), round_up(a->slots, kXBox));
    const int64_t busy = std::min<int64_t>(E, a->slots);      // experts with slots, at most
    int64_t most_tiles = (int64_t)p.row_tiles * (busy + a->slots / p.nt);
    const int sms = sm_count();
    // Few tiles of a long K: clusters share them.  That costs 1.3 us and a
    // stage takes 0.2, so K has 16 stages at least and a part 5; and clusters
    // of half the SMs' blocks are placed at once, of more in turns.  One slot
    // of a 5120-deep MXFP4 product, 1 / 2 / 4 / 8 blocks a tile: 14.1 / 11.0 /
    // 9.2 / 15.9 us with 2048 rows (8: 128 blocks), 14.2 / 11.0 / 9.1 / 8.5
    // with 256; of a 1280-deep one 7.3 / 7.9.
    const int64_t small_tiles = (int64_t)p.row_tiles * (busy + a->slots / kSplitSlots);
    const int units = (p.ncb + 3) / 4, steps = nv ? units : p.ncb;
    const uint32_t sf = nv ? 2048u : 512u;
    const int held = (int)round_up(sizeof(Shared) + sizeof(float) * kEpiWarps * 16 * kTurnStride, 1024);
    // Shared memory of a launch whose clusters have `split` blocks: what is
    // not stages, a stage, and how many stages that leaves.
    int fixed = 0;
    auto fit = [&](int split) {
        const int slots = split > 1 ? kSplitSlots : p.nt;
        p.b_rows = std::max(slots, kXBox);
        p.stage_bytes = (uint32_t)round_up(at * 16384 + p.b_rows * 128 + (at + (slots + 127) / 128) * sf, 1024);
        fixed = 1024 + 8 * (E + 1) + 32 + (split - 1) * at * kSplitSlots * 128 * 4;
        p.stages = std::min<int>(kMaxStages, (kSmemLimit - held - fixed) / (int)p.stage_bytes);
    };
    p.split = 1;
    while (p.split < kMaxSplit && steps >= 16 && small_tiles * p.split * 2 <= sms / 2 && steps >= 5 * p.split * 2 && units >= p.split * 2)
        p.split *= 2;
    // many experts' prefixes leave less for the exchanged sums
    for (fit(p.split); p.split > 1 && p.stages < 3; fit(p.split)) p.split /= 2;
    if (p.split > 1) {
        shape = a->gated ? kGatedShared : kNarrowShared;
        p.nt = kSplitSlots;
        most_tiles = small_tiles;
    }
    if (p.stages < 2) return CSF_ERR_UNSUPPORTED;
    // never two blocks on an SM: each holds the whole tensor memory
    const int smem = std::max(fixed + p.stages * (int)p.stage_bytes, 120 * 1024);

    if (most_tiles >= (1ll << 31)) return CSF_ERR_UNSUPPORTED;
    EncodeFn encode = encode_fn();
    if (sms < 1 || !encode) return CSF_ERR_CUDA;

    CUtensorMap wmap, xmap;
    {
        const cuuint64_t dims[3] = {(cuuint64_t)(nv ? K / 2 : K), (cuuint64_t)N, (cuuint64_t)E};
        const cuuint64_t strides[2] = {(cuuint64_t)K / 2, (cuuint64_t)K / 2 * (cuuint64_t)N};
        const cuuint32_t box[3] = {128, 128, 1}, ones[3] = {1, 1, 1};
        if (encode(&wmap, nv ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_16U4_ALIGN16B, 3,
                   const_cast<uint8_t *>(a->w), dims, strides, box, ones, CU_TENSOR_MAP_INTERLEAVE_NONE,
                   CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
            return CSF_ERR_CUDA;
    }
    if (!a->rows) {
        const cuuint64_t dims[2] = {(cuuint64_t)(nv ? K / 2 : K), (cuuint64_t)a->x.rows};
        const cuuint64_t strides[1] = {(cuuint64_t)a->x.code_stride};
        const cuuint32_t box[2] = {128, kXBox}, ones[2] = {1, 1};
        if (encode(&xmap, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, a->x.codes, dims, strides, box, ones, CU_TENSOR_MAP_INTERLEAVE_NONE,
                   CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
            return CSF_ERR_CUDA;
    } else {
        xmap = wmap;      // not read
    }
    const bool res = a->residual || a->row_scale;
    Kernel k = a->rows ? (nv ? nvfp4_rows_kernel(out, shape, res) : mxfp8_rows_kernel(out, shape, res))
                       : (nv ? nvfp4_kernel(out, shape, res) : mxfp8_kernel(out, shape, res));
    if (!allow_smem(reinterpret_cast<const void *>(k), kSmemLimit)) return CSF_ERR_CUDA;
    cudaLaunchConfig_t config = {};
    config.gridDim = dim3((unsigned)(p.split > 1 ? most_tiles * p.split : std::min<int64_t>(sms, most_tiles)));
    config.blockDim = dim3(kMmThreads);
    config.dynamicSmemBytes = (size_t)smem;
    config.stream = static_cast<cudaStream_t>(stream);
    cudaLaunchAttribute cluster;
    if (p.split > 1) {
        cluster.id = cudaLaunchAttributeClusterDimension;
        cluster.val.clusterDim.x = (unsigned)p.split;
        cluster.val.clusterDim.y = cluster.val.clusterDim.z = 1;
        config.attrs = &cluster;
        config.numAttrs = 1;
    }
    if (cudaLaunchKernelEx(&config, k, wmap, xmap, p) != cudaSuccess) {
        cudaGetLastError();
        return CSF_ERR_CUDA;
    }
    return CSF_OK;
}
