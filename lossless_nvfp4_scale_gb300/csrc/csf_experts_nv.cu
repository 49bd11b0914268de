// The expert products' kernels for NVFP4 rows, one a slot.
#include "csf_experts.cuh"

namespace csfk {
namespace mm {

Kernel nvfp4_kernel(int out, int shape, bool res) { return pick_kernel<CSF_ROWS_NVFP4, false>(out, shape, res); }

}  // namespace mm
}  // namespace csfk
