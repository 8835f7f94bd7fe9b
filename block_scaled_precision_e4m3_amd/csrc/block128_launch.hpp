// Launches of the block-128 product's kernels, one translation unit per group.
#pragma once

#include <hip/hip_runtime.h>

#include "block128_gemm.hpp"

namespace mxg {
namespace b128 {

// The tile shapes.  16-bit C: the eight waves of a 256 x 256 or 128 x 256 tile hold most registers and move the
// operands themselves; the smaller tiles, whose steps are short, leave that to four more waves.  float32 C: the
// accumulators and the block's sums together allow 64 x 64 outputs per wave.
using Tile256 = TileShape<256, 256, 2, 4, 2, 1>;
using Tile128x256 = TileShape<128, 256, 2, 4, 3, 1>;
using Tile128 = TileShape<128, 128, 2, 2, 3, 1, 4, false>;
using Tile64x128 = TileShape<64, 128, 2, 2, 3, 2, 4>;
using Tile64 = TileShape<64, 64, 2, 2, 3, 2, 4>;
using Exact128x256 = TileShape<128, 256, 2, 4, 2, 1>;
using Exact128 = TileShape<128, 128, 2, 2, 2, 2, 4>;
using Exact64x128 = TileShape<64, 128, 2, 2, 3, 2, 4>;
using Exact64 = TileShape<64, 64, 2, 2, 3, 2, 4>;

hipError_t launch_tile256(const GemmParams& p, int fa, int fb, int ct, int64_t grid, hipStream_t s);
hipError_t launch_tile128x256(const GemmParams& p, int fa, int fb, int ct, int64_t grid, hipStream_t s);
hipError_t launch_tile128(const GemmParams& p, int fa, int fb, int ct, int64_t grid, hipStream_t s);
hipError_t launch_tile64x128(const GemmParams& p, int fa, int fb, int ct, int64_t grid, hipStream_t s);
hipError_t launch_tile64(const GemmParams& p, int fa, int fb, int ct, int64_t grid, hipStream_t s);
hipError_t launch_exact128x256(const GemmParams& p, int fa, int fb, int64_t grid, hipStream_t s);
hipError_t launch_exact128(const GemmParams& p, int fa, int fb, int64_t grid, hipStream_t s);
hipError_t launch_exact64x128(const GemmParams& p, int fa, int fb, int64_t grid, hipStream_t s);
hipError_t launch_exact64(const GemmParams& p, int fa, int fb, int64_t grid, hipStream_t s);
// up to 32 rows; p.tilesN counts groups of `cols` (16 or 32) columns
hipError_t launch_rows(const GemmParams& p, int fa, int fb, int ct, int cols, unsigned grid, hipStream_t s);

// f<FA, FB>(...) for the formats of A and B.
template <class F>
hipError_t by_format(int fa, int fb, F f) {
  using std::integral_constant;
  if (fa == 0) return fb == 0 ? f(integral_constant<int, 0>{}, integral_constant<int, 0>{}) : f(integral_constant<int, 0>{}, integral_constant<int, 1>{});
  return fb == 0 ? f(integral_constant<int, 1>{}, integral_constant<int, 0>{}) : f(integral_constant<int, 1>{}, integral_constant<int, 1>{});
}

template <class T>
hipError_t launch_tile(const GemmParams& p, int fa, int fb, int ct, int64_t grid, hipStream_t s) {
  const dim3 g((unsigned)grid), b(64 * T::kAllWaves);
  return by_format(fa, fb, [&](auto a, auto c) {
    constexpr int FA = decltype(a)::value, FB = decltype(c)::value;
    if (ct == 1) {
      if (p.b_rows) hipLaunchKernelGGL((block128_tile_kernel<T, FA, FB, 1, true>), g, b, 0, s, p);
      else hipLaunchKernelGGL((block128_tile_kernel<T, FA, FB, 1, false>), g, b, 0, s, p);
    } else {
      if (p.b_rows) hipLaunchKernelGGL((block128_tile_kernel<T, FA, FB, 2, true>), g, b, 0, s, p);
      else hipLaunchKernelGGL((block128_tile_kernel<T, FA, FB, 2, false>), g, b, 0, s, p);
    }
    return hipGetLastError();
  });
}

template <class T>
hipError_t launch_exact(const GemmParams& p, int fa, int fb, int64_t grid, hipStream_t s) {
  const dim3 g((unsigned)grid), b(64 * T::kAllWaves);
  return by_format(fa, fb, [&](auto a, auto c) {
    constexpr int FA = decltype(a)::value, FB = decltype(c)::value;
    if (p.b_rows) hipLaunchKernelGGL((block128_exact_kernel<T, FA, FB, true>), g, b, 0, s, p);
    else hipLaunchKernelGGL((block128_exact_kernel<T, FA, FB, false>), g, b, 0, s, p);
    return hipGetLastError();
  });
}

}  // namespace b128
}  // namespace mxg
