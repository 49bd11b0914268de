// Host side of csf_fp8_matmul: argument checks, tensor maps, the choice of a
// kernel and its launch.
#include <algorithm>
#include <cstring>

#include "csf_fp8.cuh"
#include "csf_host.cuh"

namespace csfk {
namespace f8 {
namespace {

csf_status check(const csf_fp8_matmul_args *a) {
    if (!a) return CSF_ERR_ARG;
    if (a->x.kind != CSF_ROWS_FP8 || !rows_valid(a->x, true) || a->experts < 1 || a->n < 1 || a->k < 1 || a->slots < 0) return CSF_ERR_ARG;
    if (a->x.cols != (a->transposed ? a->n : a->k)) return CSF_ERR_ARG;
    if (a->act < CSF_ACT_NONE || a->act > CSF_ACT_GELU_TANH) return CSF_ERR_ARG;
    if (a->experts > kMaxExperts || a->slots >= (1ll << 31) || a->x.rows >= (1ll << 31)) return CSF_ERR_UNSUPPORTED;
    if (a->n > INT32_MAX - 511 || a->k > INT32_MAX - 511) return CSF_ERR_UNSUPPORTED;      // whole tiles of them count in 32 bits
    if (a->k % 16 || (a->transposed && (a->n % 16 || a->gated)) || (a->gated && a->n % 256)) return CSF_ERR_UNSUPPORTED;
    if (!a->expert_start && a->experts != 1) return CSF_ERR_ARG;
    if (!a->rows && a->slots > a->x.rows) return CSF_ERR_ARG;
    if (a->slots == 0) return CSF_OK;
    if (a->x.rows == 0) return CSF_ERR_ARG;
    if (!a->w || !a->w_scales || !aligned_to(a->w, 16) || !aligned_to(a->w_scales, 4)) return CSF_ERR_ARG;
    const int32_t O = a->transposed ? a->k : a->n, F = a->gated ? O / 2 : O;
    if (!aligned_to(a->rows, 4) || !aligned_to(a->expert_start, a->expert_start_is_int64 ? 8 : 4)) return CSF_ERR_ARG;
    if (!aligned_to(a->row_scale, 4) || !aligned_to(a->error_word, 4)) return CSF_ERR_ARG;
    if (a->bias && (!dtype_known(a->bias_dtype) || !aligned_to(a->bias, dtype_bytes(a->bias_dtype)))) return CSF_ERR_ARG;
    if (a->residual && (!dtype_known(a->residual_dtype) || a->residual_stride < F || !aligned_to(a->residual, dtype_bytes(a->residual_dtype))))
        return CSF_ERR_ARG;
    if (a->out) {
        if (!dtype_known(a->out_dtype) || a->out_stride < F || !aligned_to(a->out, dtype_bytes(a->out_dtype))) return CSF_ERR_ARG;
    } else if (a->out_rows.kind != CSF_ROWS_FP8 || !rows_valid(a->out_rows, true) || a->out_rows.cols != F || a->out_rows.rows != a->slots) {
        return CSF_ERR_ARG;
    }
    return CSF_OK;
}

}  // namespace
}  // namespace f8
}  // namespace csfk

using namespace csfk;
using namespace csfk::f8;

extern "C" csf_status csf_fp8_matmul(const csf_fp8_matmul_args *a, void *stream) {
    csf_status st = check(a);
    if (st != CSF_OK || a->slots == 0) return st;
    const int32_t N = a->n, K = a->k, E = a->experts;

    Params p;
    std::memset(&p, 0, sizeof(p));
    p.x_codes = a->x.codes;
    p.x_code_stride = a->x.code_stride;
    p.x_scales = a->x.scales;
    p.x_scale_stride = a->x.scale_stride;
    p.rows = a->rows;
    p.start = a->expert_start;
    p.es64 = a->expert_start_is_int64;
    const int32_t nb = (N + 127) / 128, kb = (K + 127) / 128;
    p.w_scales = a->w_scales;
    if ((int64_t)nb * kb * E > INT32_MAX) return CSF_ERR_UNSUPPORTED;      // scales count in 32 bits
    p.ws_expert = nb * kb;
    p.ws_f = a->transposed ? 1 : kb;
    p.ws_b = a->transposed ? kb : 1;
    p.bias = a->bias;
    p.bias_dtype = a->bias_dtype;
    p.row_scale = a->row_scale;
    p.residual = a->residual;
    p.residual_stride = a->residual_stride;
    p.residual_dtype = a->residual_dtype;
    p.residual_wide = a->residual && wide_rows(a->residual, a->residual_stride, a->residual_dtype);
    p.err = a->error_word;
    p.slots = a->slots;
    p.x_rows = (int32_t)a->x.rows;
    p.E = E;
    p.depth = a->transposed ? N : K;
    p.blocks = a->transposed ? nb : kb;
    p.O = a->transposed ? K : N;
    p.F = a->gated ? p.O / 2 : p.O;
    p.f_blocks = a->transposed ? kb : nb;
    p.bias_wide = a->bias && wide_rows(a->bias, p.O, a->bias_dtype);
    p.act = a->act;
    p.gated = a->gated;
    p.transposed = a->transposed;
    if (a->out) {
        p.out = static_cast<char *>(a->out);
        p.out_dtype = a->out_dtype;
        p.out_stride = a->out_stride * (int64_t)dtype_bytes(a->out_dtype);
        p.out_wide = wide_rows(a->out, a->out_stride, a->out_dtype);
    } else {
        p.out = reinterpret_cast<char *>(a->out_rows.codes);
        p.out_stride = a->out_rows.code_stride;
        p.out_scales = a->out_rows.scales;
        p.out_scale_stride = a->out_rows.scale_stride;
    }

    const int sms = sm_count();
    const Plan plan = plan_of({sms, a->slots, E, p.F, p.blocks, a->gated != 0});
    if (plan.stages < 2 || plan.most_tiles >= (1ll << 31)) return CSF_ERR_UNSUPPORTED;
    if (sms < 1) return CSF_ERR_CUDA;
    p.tile_step = plan.tile_step;
    p.second = a->gated ? N / 2 : 128;
    p.row_tiles = plan.row_tiles;
    p.row_tiles_magic = (uint32_t)((1ull << 32) / (uint32_t)p.row_tiles + 1);
    p.nt = plan.nt;
    p.stage_bytes = plan.stage_bytes;
    p.stages = plan.stages;
    p.split = plan.split;

    CUtensorMap wmap, xmap;
    {
        const cuuint64_t dims[3] = {(cuuint64_t)K, (cuuint64_t)N, (cuuint64_t)E};
        const cuuint64_t strides[2] = {(cuuint64_t)K, (cuuint64_t)K * (cuuint64_t)N};
        const cuuint32_t box[3] = {128, 128, 1};
        if (!byte_map(&wmap, a->w, 3, dims, strides, box)) return CSF_ERR_CUDA;
    }
    if (!a->rows) {
        const cuuint64_t dims[2] = {(cuuint64_t)p.depth, (cuuint64_t)a->x.rows};
        const cuuint64_t strides[1] = {(cuuint64_t)a->x.code_stride};
        const cuuint32_t box[2] = {128, 32};
        if (!byte_map(&xmap, a->x.codes, 2, dims, strides, box)) return CSF_ERR_CUDA;
    } else {
        xmap = wmap;      // not read
    }
    const bool sums = a->residual && a->residual_dtype != CSF_F32 && p.residual_wide && p.out_wide && p.F % 8 == 0;
    const int mode = !a->out ? kQuant : a->out_dtype == CSF_F32 ? kPlain : !a->residual ? kHalves : sums ? kHalvesSum : kPlain;
    Kernel k = a->rows ? rows_by_index(plan.shape, mode) : rows_in_order(plan.shape, mode);
    // the register split waits for what the block was launched with (given out in eights)
    if (!allow_smem(reinterpret_cast<const void *>(k), kSmemLimit, launch_regs(a->rows) - 7)) return CSF_ERR_CUDA;
    const unsigned per = (unsigned)p.split;      // blocks of a cluster
    cudaLaunchConfig_t config = {};
    config.gridDim = dim3((unsigned)(per > 1 ? plan.most_tiles * per : std::min<int64_t>(sms, plan.most_tiles)));
    config.blockDim = dim3((unsigned)threads_of(a->rows));
    config.dynamicSmemBytes = (size_t)plan.smem;
    config.stream = static_cast<cudaStream_t>(stream);
    cudaLaunchAttribute cluster;
    if (per > 1) {
        cluster.id = cudaLaunchAttributeClusterDimension;
        cluster.val.clusterDim.x = per;
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
