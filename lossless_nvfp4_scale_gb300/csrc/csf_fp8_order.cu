// The 8-bit products' kernels for x rows in the slots' order.
#include "csf_fp8.cuh"

namespace csfk {
namespace f8 {

Kernel rows_in_order(int shape, int mode) { return pick_kernel<false>(shape, mode); }

}  // namespace f8
}  // namespace csfk
