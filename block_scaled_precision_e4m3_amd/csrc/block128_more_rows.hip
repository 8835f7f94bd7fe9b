// Block-128 product, few rows of A, with what follows the product or rows in groups: instantiations.
#include "block128_launch.hpp"

namespace mxg {
namespace b128 {

namespace {

template <int FA, int FB, int CT, Form FORM>
void launch(const MoreParams& p, int rows, int cols, unsigned grid, hipStream_t s) {
  const dim3 g(grid), b(64 * kRowWaves);
  if (rows == 16) {
    if (cols == 16) hipLaunchKernelGGL((block128_rows_kernel<FA, FB, CT, false, 16, 1, FORM>), g, b, 0, s, p);
    else hipLaunchKernelGGL((block128_rows_kernel<FA, FB, CT, false, 32, 1, FORM>), g, b, 0, s, p);
  } else {
    if (cols == 16) hipLaunchKernelGGL((block128_rows_kernel<FA, FB, CT, false, 16, 2, FORM>), g, b, 0, s, p);
    else hipLaunchKernelGGL((block128_rows_kernel<FA, FB, CT, false, 32, 2, FORM>), g, b, 0, s, p);
  }
}

}  // namespace

hipError_t launch_rows_more(Form form, const MoreParams& p, int fa, int fb, int ct, int rows, int cols, unsigned grid, hipStream_t s) {
  return by_format(fa, fb, [&](auto a, auto c) {
    constexpr int FA = decltype(a)::value, FB = decltype(c)::value;
    if (form == kEnds) {
      if (ct == 0) launch<FA, FB, 0, kEnds>(p, rows, cols, grid, s);
      else if (ct == 1) launch<FA, FB, 1, kEnds>(p, rows, cols, grid, s);
      else launch<FA, FB, 2, kEnds>(p, rows, cols, grid, s);
    } else {
      if (ct == 0) launch<FA, FB, 0, kRowGroups>(p, rows, cols, grid, s);
      else if (ct == 1) launch<FA, FB, 1, kRowGroups>(p, rows, cols, grid, s);
      else launch<FA, FB, 2, kRowGroups>(p, rows, cols, grid, s);
    }
    return hipGetLastError();
  });
}

}  // namespace b128
}  // namespace mxg
