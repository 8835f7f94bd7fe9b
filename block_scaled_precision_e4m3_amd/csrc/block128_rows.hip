// Block-128 product, few rows of A: instantiations.
#include "block128_launch.hpp"

namespace mxg {
namespace b128 {

namespace {

template <int FA, int FB, int CT, bool BROWS>
void launch(const GemmParams& p, int mt, int nt, int64_t grid, hipStream_t s) {
  const dim3 g((unsigned)grid), b(64 * kRowWaves);
  if (mt == 1 && nt == 1) hipLaunchKernelGGL((block128_rows_kernel<FA, FB, CT, BROWS, 1, 1, 4>), g, b, 0, s, p);
  else if (mt == 1) hipLaunchKernelGGL((block128_rows_kernel<FA, FB, CT, BROWS, 1, 2, 2>), g, b, 0, s, p);
  else if (mt == 2 && nt == 1) hipLaunchKernelGGL((block128_rows_kernel<FA, FB, CT, BROWS, 2, 1, 2>), g, b, 0, s, p);
  else if (mt == 2) hipLaunchKernelGGL((block128_rows_kernel<FA, FB, CT, BROWS, 2, 2, 2>), g, b, 0, s, p);
  else if (nt == 1) hipLaunchKernelGGL((block128_rows_kernel<FA, FB, CT, BROWS, 4, 1, 2>), g, b, 0, s, p);
  else hipLaunchKernelGGL((block128_rows_kernel<FA, FB, CT, BROWS, 4, 2, 2>), g, b, 0, s, p);
}

}  // namespace

hipError_t launch_rows(const GemmParams& p, int fa, int fb, int ct, int mt, int nt, int64_t grid, hipStream_t s) {
  return by_format(fa, fb, [&](auto a, auto c) {
    constexpr int FA = decltype(a)::value, FB = decltype(c)::value;
    if (ct == 0) {
      if (p.b_rows) launch<FA, FB, 0, true>(p, mt, nt, grid, s);
      else launch<FA, FB, 0, false>(p, mt, nt, grid, s);
    } else if (ct == 1) {
      if (p.b_rows) launch<FA, FB, 1, true>(p, mt, nt, grid, s);
      else launch<FA, FB, 1, false>(p, mt, nt, grid, s);
    } else {
      if (p.b_rows) launch<FA, FB, 2, true>(p, mt, nt, grid, s);
      else launch<FA, FB, 2, false>(p, mt, nt, grid, s);
    }
    return hipGetLastError();
  });
}

}  // namespace b128
}  // namespace mxg
