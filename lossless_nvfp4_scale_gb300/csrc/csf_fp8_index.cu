// The 8-bit products' kernels for x rows taken through an index.
#include "csf_fp8.cuh"

namespace csfk {
namespace f8 {

Kernel rows_by_index(int shape, bool quant) { return quant ? pick<true, true>(shape) : pick<true, false>(shape); }

}  // namespace f8
}  // namespace csfk
