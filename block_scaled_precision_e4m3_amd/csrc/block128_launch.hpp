// Launches of the block-128 product's kernels, one translation unit per group.
#pragma once

#include <hip/hip_runtime.h>

#include "block128_gemm.hpp"

namespace mxg {
namespace b128 {

// 16-bit C (ct MXG_DT_BF16 or MXG_DT_F16) in tiles of 256 x 256, 128 x 128 or 64 x 64.
hipError_t launch_tile256(const GemmParams& p, int fa, int fb, int ct, int64_t grid, hipStream_t s);
hipError_t launch_tile128(const GemmParams& p, int fa, int fb, int ct, int64_t grid, hipStream_t s);
hipError_t launch_tile64(const GemmParams& p, int fa, int fb, int ct, int64_t grid, hipStream_t s);
// float32 C in tiles of 256 x 128 or 128 x 128.
hipError_t launch_exact256(const GemmParams& p, int fa, int fb, int64_t grid, hipStream_t s);
hipError_t launch_exact128(const GemmParams& p, int fa, int fb, int64_t grid, hipStream_t s);
// up to 64 rows; p.tilesN counts groups of 16 * nt columns, mt rows of 16
hipError_t launch_rows(const GemmParams& p, int fa, int fb, int ct, int mt, int nt, int64_t grid, hipStream_t s);

// f<FA, FB>(...) for the formats of A and B.
template <class F>
hipError_t by_format(int fa, int fb, F f) {
  using std::integral_constant;
  if (fa == 0) return fb == 0 ? f(integral_constant<int, 0>{}, integral_constant<int, 0>{}) : f(integral_constant<int, 0>{}, integral_constant<int, 1>{});
  return fb == 0 ? f(integral_constant<int, 1>{}, integral_constant<int, 0>{}) : f(integral_constant<int, 1>{}, integral_constant<int, 1>{});
}

template <class T>
hipError_t launch_tile(const GemmParams& p, int fa, int fb, int ct, int64_t grid, hipStream_t s) {
  const dim3 g((unsigned)grid), b(64 * T::kWaves);
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
  const dim3 g((unsigned)grid), b(64 * T::kWaves);
  return by_format(fa, fb, [&](auto a, auto c) {
    constexpr int FA = decltype(a)::value, FB = decltype(c)::value;
    if (p.b_rows) hipLaunchKernelGGL((block128_exact_kernel<T, FA, FB, true>), g, b, 0, s, p);
    else hipLaunchKernelGGL((block128_exact_kernel<T, FA, FB, false>), g, b, 0, s, p);
    return hipGetLastError();
  });
}

}  // namespace b128
}  // namespace mxg
