// C-ABI entry point of the gradients through bias, activation and gate (include/mxgemm.h).
#include <hip/hip_runtime.h>

#include <algorithm>
#include <initializer_list>

#include "../../include/mxgemm.h"
#include "activation.hpp"
#include "host_checks.hpp"
#include "overlap.hpp"

namespace {

using namespace mxg::host;
using mxg::activation::Params;

// How a call's rows and columns are shared out: a rule on the sizes alone, which the workspace depends on.
struct Shares {
  int lanes, strips;
  int64_t parts, rows;
};
constexpr int64_t kFewRows = 256;
// Past these columns 64 lanes to a row make a single part as well, in fewer workgroups: a launch's work items have to stay
// below 2^32, which strips of 64 columns would not from 2^29 on.
constexpr int64_t kFewColumns = 1 << 19;
Shares shares(int64_t M, int64_t N) {
  Shares s;
  // Few rows: 8 lanes to a row, which still are whole lines, so that a workgroup takes 128 rows at a time and one part
  // does (40 x 2048 float32: 4.3 us on the GPU; with 64 lanes in three parts and a second kernel 8.3 us).
  const bool few = M <= kFewRows && N <= kFewColumns;
  s.lanes = 1;
  while (s.lanes < (few ? 8 : 64) && 8 * s.lanes < N) s.lanes *= 2;
  s.strips = (int)cdiv(N, 8 * s.lanes);
  const int64_t step = mxg::activation::kThreads / s.lanes * mxg::activation::kAhead;  // rows a workgroup takes at a time
  if (few) {
    s.rows = kFewRows;
    s.parts = 1;
    return s;
  }
  const int64_t wanted = std::max<int64_t>(1, std::min<int64_t>(mxg::activation::kMaxParts, 1024 / s.strips));
  s.rows = cdiv(cdiv(M, wanted), step) * step;
  s.parts = cdiv(M, s.rows);
  return s;
}

template <int DT>
void launch(const Params& p, unsigned grid, hipStream_t s) {
  const dim3 g(grid), b(mxg::activation::kThreads);
  if (p.gate) hipLaunchKernelGGL((mxg::activation::activation_backward_kernel<DT, true>), g, b, 0, s, p);
  else hipLaunchKernelGGL((mxg::activation::activation_backward_kernel<DT, false>), g, b, 0, s, p);
}

bool sizes_ok(int64_t M, int64_t N) {
  return M >= 0 && N >= 0 && M <= 0x7FFFFF00LL && N <= 0x7FFFFF00LL && (M == 0 || N <= (1LL << 58) / M);
}

}  // namespace

extern "C" {

size_t mxgemm_activation_backward_workspace_bytes(int64_t M, int64_t N) {
  if (!sizes_ok(M, N) || M == 0 || N == 0) return 0;
  const Shares s = shares(M, N);
  return s.parts > 1 ? (size_t)(s.parts * N * 4) : 0;
}

int mxgemm_activation_backward(const void* DY, const void* Z, const void* GATE, void* DZ, void* DGATE, float* DBIAS,
                               const int64_t* strides, int64_t M, int64_t N, int activation, int dtype, unsigned flags,
                               void* workspace, size_t workspace_bytes, void* stream) {
  const bool trusted = take_trust(&flags);
  if (!sizes_ok(M, N)) return MXG_ERR_SHAPE;
  if (activation < MXG_ACT_NONE || activation > MXG_ACT_GELU_TANH || dtype < MXG_DT_F32 || dtype > MXG_DT_F16) return MXG_ERR_FMT;
  if (flags) return MXG_ERR_FLAGS;
  if (!strides) return MXG_ERR_NULL;
  const void* all[5] = {DY, Z, GATE, DZ, DGATE};
  for (int i = 0; i < 5; ++i)
    if (all[i] && (strides[i] < N || strides[i] > (1LL << 40) || (M > 0 && strides[i] > (1LL << 59) / M))) return MXG_ERR_SHAPE;
  if (N == 0) return MXG_OK;
  if ((GATE != nullptr) != (DGATE != nullptr) || (M > 0 && (!DY || !Z || !DZ))) return MXG_ERR_NULL;
  const size_t need = DBIAS ? mxgemm_activation_backward_workspace_bytes(M, N) : 0;
  if (need > 0 && !workspace) return MXG_ERR_NULL;
  if (need > workspace_bytes) return MXG_ERR_SHAPE;
  for (const void* t : all)
    if (!aligned_to(t, mxg::elem_bytes(dtype))) return MXG_ERR_ALIGN;
  if (!aligned_to(DBIAS, 4) || (need > 0 && !aligned16(workspace))) return MXG_ERR_ALIGN;
  int dev = 0, cus = 0;
  const int st = device_check(&dev, &cus);
  if (st != MXG_OK) return st;
  if (!trusted) {
    for (const void* t : {DY, Z, GATE, (const void*)DZ, (const void*)DGATE, (const void*)DBIAS})
      if (t && !on_device(t, dev)) return MXG_ERR_DEVICE;
    if (need > 0 && !on_device(workspace, dev)) return MXG_ERR_DEVICE;
  }
  // Workgroups would read what others have written, or write the same places.  dz and dgate may be one of what is read, the
  // same rows of it: a lane has read what it writes.
  RowsAt of[5];
  for (int i = 0; i < 5; ++i) of[i] = rows_at(all[i], M, N, strides[i], mxg::elem_bytes(dtype));
  const RowsAt sums = flat(DBIAS, 4 * N), scratch = flat(workspace, (int64_t)need);
  for (int i = 0; i < 5; ++i) {
    if (overlap(of[i], sums) || overlap(of[i], scratch)) return MXG_ERR_SHAPE;
    for (int j = 3; i < 3 && j < 5; ++j)
      if (overlap(of[i], of[j]) && !same(of[i], of[j])) return MXG_ERR_SHAPE;
  }
  if (overlap(of[3], of[4]) || overlap(sums, scratch)) return MXG_ERR_SHAPE;
  hipStream_t s = (hipStream_t)stream;
  if (M == 0) {
    if (DBIAS) hipLaunchKernelGGL(mxg::activation::bias_zero_kernel, dim3((unsigned)cdiv(N, 256)), dim3(256), 0, s, DBIAS, (int)N);
    return hipGetLastError() == hipSuccess ? MXG_OK : MXG_ERR_LAUNCH;
  }
  const Shares sh = shares(M, N);
  Params p{};
  p.dy = DY;
  p.z = Z;
  p.gate = GATE;
  p.dz = DZ;
  p.dgate = DGATE;
  p.sums = !DBIAS ? nullptr : need > 0 ? static_cast<float*>(workspace) : DBIAS;
  p.ld_dy = strides[0];
  p.ld_z = strides[1];
  p.ld_gate = strides[2];
  p.ld_dz = strides[3];
  p.ld_dgate = strides[4];
  p.M = M;
  p.rows = sh.rows;
  p.N = (int)N;
  p.act = activation;
  p.lanes = sh.lanes;
  p.strips = sh.strips;
  const unsigned grid = (unsigned)(sh.strips * sh.parts);
  if (dtype == MXG_DT_F32) launch<0>(p, grid, s);
  else if (dtype == MXG_DT_BF16) launch<1>(p, grid, s);
  else launch<2>(p, grid, s);
  if (need > 0)
    hipLaunchKernelGGL(mxg::activation::bias_sum_kernel, dim3((unsigned)cdiv(N, 64)), dim3(1024), 0, s,
                       static_cast<const float*>(workspace), (int)sh.parts, DBIAS, (int)N);
  return hipGetLastError() == hipSuccess ? MXG_OK : MXG_ERR_LAUNCH;
}

}  // extern "C"
