// The expert products' kernels for MXFP8 rows, taken through an index.
#include "csf_experts.cuh"

namespace csfk {
namespace mm {

Kernel mxfp8_rows_kernel(int out, int shape, bool res) { return pick_kernel<CSF_ROWS_MXFP8, true>(out, shape, res); }

}  // namespace mm
}  // namespace csfk
