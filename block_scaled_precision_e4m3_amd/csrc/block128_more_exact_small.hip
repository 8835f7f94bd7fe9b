// Block-128 product, float32 C, smaller tiles, with what follows the product or in groups: instantiations.
#include "block128_launch.hpp"

namespace mxg {
namespace b128 {

hipError_t launch_more_exact64x128(Form form, const MoreParams& p, int fa, int fb, int, int64_t grid, hipStream_t s) {
  return launch_more_exact<Exact64x128>(form, p, fa, fb, grid, s);
}

hipError_t launch_more_exact64(Form form, const MoreParams& p, int fa, int fb, int, int64_t grid, hipStream_t s) {
  return launch_more_exact<Exact64>(form, p, fa, fb, grid, s);
}

}  // namespace b128
}  // namespace mxg
