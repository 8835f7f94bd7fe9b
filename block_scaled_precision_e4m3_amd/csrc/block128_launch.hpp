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

// A tile size's kernels of one form: 16-bit C by its type, or float32 C.
using TileLaunch = hipError_t (*)(const GemmParams& p, int fa, int fb, int ct, int64_t grid, hipStream_t s);
using MoreLaunch = hipError_t (*)(Form form, const MoreParams& p, int fa, int fb, int ct, int64_t grid, hipStream_t s);
hipError_t launch_tile256(const GemmParams& p, int fa, int fb, int ct, int64_t grid, hipStream_t s);
hipError_t launch_tile128x256(const GemmParams& p, int fa, int fb, int ct, int64_t grid, hipStream_t s);
hipError_t launch_tile128(const GemmParams& p, int fa, int fb, int ct, int64_t grid, hipStream_t s);
hipError_t launch_tile64x128(const GemmParams& p, int fa, int fb, int ct, int64_t grid, hipStream_t s);
hipError_t launch_tile64(const GemmParams& p, int fa, int fb, int ct, int64_t grid, hipStream_t s);
hipError_t launch_exact128x256(const GemmParams& p, int fa, int fb, int ct, int64_t grid, hipStream_t s);
hipError_t launch_exact128(const GemmParams& p, int fa, int fb, int ct, int64_t grid, hipStream_t s);
hipError_t launch_exact64x128(const GemmParams& p, int fa, int fb, int ct, int64_t grid, hipStream_t s);
hipError_t launch_exact64(const GemmParams& p, int fa, int fb, int ct, int64_t grid, hipStream_t s);
// kEnds and kRowGroups; the exact ones also kDeepGroups
hipError_t launch_more256(Form form, const MoreParams& p, int fa, int fb, int ct, int64_t grid, hipStream_t s);
hipError_t launch_more128x256(Form form, const MoreParams& p, int fa, int fb, int ct, int64_t grid, hipStream_t s);
hipError_t launch_more128(Form form, const MoreParams& p, int fa, int fb, int ct, int64_t grid, hipStream_t s);
hipError_t launch_more64x128(Form form, const MoreParams& p, int fa, int fb, int ct, int64_t grid, hipStream_t s);
hipError_t launch_more64(Form form, const MoreParams& p, int fa, int fb, int ct, int64_t grid, hipStream_t s);
hipError_t launch_more_exact128x256(Form form, const MoreParams& p, int fa, int fb, int ct, int64_t grid, hipStream_t s);
hipError_t launch_more_exact128(Form form, const MoreParams& p, int fa, int fb, int ct, int64_t grid, hipStream_t s);
hipError_t launch_more_exact64x128(Form form, const MoreParams& p, int fa, int fb, int ct, int64_t grid, hipStream_t s);
hipError_t launch_more_exact64(Form form, const MoreParams& p, int fa, int fb, int ct, int64_t grid, hipStream_t s);
// up to 32 rows; p.tilesN counts groups of `cols` (16 or 32) columns
hipError_t launch_rows(const GemmParams& p, int fa, int fb, int ct, int cols, unsigned grid, hipStream_t s);
// kEnds: as above; kRowGroups: `rows` (16 or 32) of a group to a workgroup
hipError_t launch_rows_more(Form form, const MoreParams& p, int fa, int fb, int ct, int rows, int cols, unsigned grid, hipStream_t s);

// f<FA, FB>(...) for the formats of A and B.
template <class F>
hipError_t by_format(int fa, int fb, F f) {
  using std::integral_constant;
  if (fa == 0) return fb == 0 ? f(integral_constant<int, 0>{}, integral_constant<int, 0>{}) : f(integral_constant<int, 0>{}, integral_constant<int, 1>{});
  return fb == 0 ? f(integral_constant<int, 1>{}, integral_constant<int, 0>{}) : f(integral_constant<int, 1>{}, integral_constant<int, 1>{});
}

// BROWS: scales in rows of blocks are among the kernels (and a call may ask for them).
template <class T, Form FORM, bool BROWS, class P>
hipError_t launch_tile(const P& p, int fa, int fb, int ct, int64_t grid, hipStream_t s) {
  const dim3 g((unsigned)grid), b(64 * T::kAllWaves);
  return by_format(fa, fb, [&](auto a, auto c) {
    constexpr int FA = decltype(a)::value, FB = decltype(c)::value;
    if constexpr (BROWS) {
      if (p.b_rows) {
        if (ct == 1) hipLaunchKernelGGL((block128_tile_kernel<T, FA, FB, 1, true, FORM>), g, b, 0, s, p);
        else hipLaunchKernelGGL((block128_tile_kernel<T, FA, FB, 2, true, FORM>), g, b, 0, s, p);
        return hipGetLastError();
      }
    }
    if (ct == 1) hipLaunchKernelGGL((block128_tile_kernel<T, FA, FB, 1, false, FORM>), g, b, 0, s, p);
    else hipLaunchKernelGGL((block128_tile_kernel<T, FA, FB, 2, false, FORM>), g, b, 0, s, p);
    return hipGetLastError();
  });
}

template <class T, Form FORM, class P>
hipError_t launch_exact(const P& p, int fa, int fb, int64_t grid, hipStream_t s) {
  const dim3 g((unsigned)grid), b(64 * T::kAllWaves);
  return by_format(fa, fb, [&](auto a, auto c) {
    constexpr int FA = decltype(a)::value, FB = decltype(c)::value;
    if constexpr (FORM == kPlain || FORM == kDeepGroups) {
      if (p.b_rows) {
        hipLaunchKernelGGL((block128_exact_kernel<T, FA, FB, true, FORM>), g, b, 0, s, p);
        return hipGetLastError();
      }
    }
    if constexpr (FORM != kDeepGroups) hipLaunchKernelGGL((block128_exact_kernel<T, FA, FB, false, FORM>), g, b, 0, s, p);
    return hipGetLastError();
  });
}

template <class T>
hipError_t launch_more(Form form, const MoreParams& p, int fa, int fb, int ct, int64_t grid, hipStream_t s) {
  return form == kEnds ? launch_tile<T, kEnds, false>(p, fa, fb, ct, grid, s) : launch_tile<T, kRowGroups, false>(p, fa, fb, ct, grid, s);
}
template <class T>
hipError_t launch_more_exact(Form form, const MoreParams& p, int fa, int fb, int64_t grid, hipStream_t s) {
  return form == kEnds        ? launch_exact<T, kEnds>(p, fa, fb, grid, s)
         : form == kRowGroups ? launch_exact<T, kRowGroups>(p, fa, fb, grid, s)
                              : launch_exact<T, kDeepGroups>(p, fa, fb, grid, s);
}

}  // namespace b128
}  // namespace mxg
