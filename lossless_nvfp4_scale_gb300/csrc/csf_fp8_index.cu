// The 8-bit products' kernels for x rows taken through an index.
#include "csf_fp8.cuh"

namespace csfk {
namespace f8 {

Kernel rows_by_index(int shape, int mode) { return pick_kernel<true>(shape, mode); }

}  // namespace f8
}  // namespace csfk
