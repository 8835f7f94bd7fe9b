// Block-128 product, 16-bit C, 64 x 64 tiles, with what follows the product or rows in groups: instantiations.
#include "block128_launch.hpp"

namespace mxg {
namespace b128 {

hipError_t launch_more64(Form form, const MoreParams& p, int fa, int fb, int ct, int64_t grid, hipStream_t s) {
  return launch_more<Tile64>(form, p, fa, fb, ct, grid, s);
}

}  // namespace b128
}  // namespace mxg
