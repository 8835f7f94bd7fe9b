// Block-128 product, 16-bit C, 128 x 256 tiles: instantiations.
#include "block128_launch.hpp"

namespace mxg {
namespace b128 {

hipError_t launch_tile128x256(const GemmParams& p, int fa, int fb, int ct, int64_t grid, hipStream_t s) {
  return launch_tile<Tile128x256>(p, fa, fb, ct, grid, s);
}

}  // namespace b128
}  // namespace mxg
