// The expert products' kernels for MXFP8 rows, one a slot.
#include "csf_experts.cuh"

namespace csfk {
namespace mm {

Kernel mxfp8_kernel(int out, int shape, bool res) { return pick_kernel<CSF_ROWS_MXFP8, false>(out, shape, res); }

}  // namespace mm
}  // namespace csfk
