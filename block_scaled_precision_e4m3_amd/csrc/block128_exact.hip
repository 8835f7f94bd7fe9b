// Block-128 product, float32 C: instantiations.
#include "block128_launch.hpp"

namespace mxg {
namespace b128 {

hipError_t launch_exact128x256(const GemmParams& p, int fa, int fb, int64_t grid, hipStream_t s) {
  return launch_exact<Exact128x256>(p, fa, fb, grid, s);
}

hipError_t launch_exact128(const GemmParams& p, int fa, int fb, int64_t grid, hipStream_t s) {
  return launch_exact<Exact128>(p, fa, fb, grid, s);
}

hipError_t launch_exact64x128(const GemmParams& p, int fa, int fb, int64_t grid, hipStream_t s) {
  return launch_exact<Exact64x128>(p, fa, fb, grid, s);
}

hipError_t launch_exact64(const GemmParams& p, int fa, int fb, int64_t grid, hipStream_t s) {
  return launch_exact<Exact64>(p, fa, fb, grid, s);
}

}  // namespace b128
}  // namespace mxg
