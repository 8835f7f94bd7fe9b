// Block-128 product, float32 C: instantiations.
#include "block128_launch.hpp"

namespace mxg {
namespace b128 {

hipError_t launch_exact256(const GemmParams& p, int fa, int fb, int64_t grid, hipStream_t s) {
  return launch_exact<TileShape<256, 128, 4, 2, 2>>(p, fa, fb, grid, s);
}
hipError_t launch_exact128(const GemmParams& p, int fa, int fb, int64_t grid, hipStream_t s) {
  return launch_exact<TileShape<128, 128, 2, 2, 2>>(p, fa, fb, grid, s);
}

}  // namespace b128
}  // namespace mxg
