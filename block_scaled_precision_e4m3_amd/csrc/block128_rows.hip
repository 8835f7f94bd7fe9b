// Block-128 product, few rows of A: instantiations.
#include "block128_launch.hpp"

namespace mxg {
namespace b128 {

namespace {

template <int FA, int FB, int CT, bool BROWS>
void launch(const GemmParams& p, int cols, unsigned grid, hipStream_t s) {
  const dim3 g(grid), b(64 * kRowWaves);
  if (p.M <= 16) {
    if (cols == 16) hipLaunchKernelGGL((block128_rows_kernel<FA, FB, CT, BROWS, 16, 1, kPlain>), g, b, 0, s, p);
    else hipLaunchKernelGGL((block128_rows_kernel<FA, FB, CT, BROWS, 32, 1, kPlain>), g, b, 0, s, p);
  } else {
    if (cols == 16) hipLaunchKernelGGL((block128_rows_kernel<FA, FB, CT, BROWS, 16, 2, kPlain>), g, b, 0, s, p);
    else hipLaunchKernelGGL((block128_rows_kernel<FA, FB, CT, BROWS, 32, 2, kPlain>), g, b, 0, s, p);
  }
}

}  // namespace

hipError_t launch_rows(const GemmParams& p, int fa, int fb, int ct, int cols, unsigned grid, hipStream_t s) {
  return by_format(fa, fb, [&](auto a, auto c) {
    constexpr int FA = decltype(a)::value, FB = decltype(c)::value;
    if (ct == 0) {
      if (p.b_rows) launch<FA, FB, 0, true>(p, cols, grid, s);
      else launch<FA, FB, 0, false>(p, cols, grid, s);
    } else if (ct == 1) {
      if (p.b_rows) launch<FA, FB, 1, true>(p, cols, grid, s);
      else launch<FA, FB, 1, false>(p, cols, grid, s);
    } else {
      if (p.b_rows) launch<FA, FB, 2, true>(p, cols, grid, s);
      else launch<FA, FB, 2, false>(p, cols, grid, s);
    }
    return hipGetLastError();
  });
}

}  // namespace b128
}  // namespace mxg
