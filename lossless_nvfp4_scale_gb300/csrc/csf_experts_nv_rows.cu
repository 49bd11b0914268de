// The expert products' kernels for NVFP4 rows, taken through an index.
#include "csf_experts.cuh"

namespace csfk {
namespace mm {

Kernel nvfp4_rows_kernel(int out, int shape, bool res) { return pick_kernel<CSF_ROWS_NVFP4, true>(out, shape, res); }

}  // namespace mm
}  // namespace csfk
