// The 8-bit products' kernels for x rows in the slots' order.
#include "csf_fp8.cuh"

namespace csfk {
namespace f8 {

Kernel rows_in_order(int shape, bool quant) { return quant ? pick<false, true>(shape) : pick<false, false>(shape); }

}  // namespace f8
}  // namespace csfk
