// C-ABI entry points of the block-128 quantiser and product (include/mxgemm.h).
#include <hip/hip_runtime.h>

#include <algorithm>
#include <initializer_list>

#include "../../include/mxgemm.h"
#include "block128_launch.hpp"
#include "block128_quantize.hpp"
#include "host_checks.hpp"

namespace {

using namespace mxg::host;

using mxg::b128::GemmParams;
using mxg::b128::QuantParams;

int64_t up16(int64_t v) { return (v + 15) / 16 * 16; }

// --- quantiser --------------------------------------------------------------------

int check_quantize(int64_t ldx, int64_t M, int64_t K, int64_t L, int dt, int fmt, unsigned flags) {
  if (M < 0 || K < 0 || L < 0 || ldx < K) return MXG_ERR_SHAPE;
  if (dt < MXG_DT_F32 || dt > MXG_DT_F16 || (fmt != MXG_FMT_E4M3 && fmt != MXG_FMT_E5M2)) return MXG_ERR_FMT;
  if (flags & ~(unsigned)(MXG_QUANT_SQUARE | MXG_QUANT_POW2)) return MXG_ERR_FLAGS;
  // sizes are 32-bit in the kernels, offsets 64-bit
  const int64_t top = 0x7FFFFF00LL;
  if (M > top || K > top || L > top || ldx > (1LL << 40)) return MXG_ERR_SHAPE;
  if (M && L && ldx && (ldx > (1LL << 58) / M || M * ldx > (1LL << 58) / L)) return MXG_ERR_SHAPE;
  if (M && L && K && M * K > (1LL << 58) / L) return MXG_ERR_SHAPE;
  if (M && K && L && cdiv(M, 16) * cdiv(K, 128) > 0x7FFFFFFFLL / L) return MXG_ERR_SHAPE;
  return MXG_OK;
}

template <int DT, int FMT, int RT>
void launch_quantize(const QuantParams& p, bool rows, bool cols, bool square, unsigned grid, hipStream_t s) {
  using namespace mxg::b128;
  const dim3 g(grid), b(kQThreads);
  if constexpr (RT == 8) {
    if (square && rows && cols) hipLaunchKernelGGL((block128_quantize_kernel<DT, FMT, RT, true, true, true>), g, b, 0, s, p);
    else if (square && rows) hipLaunchKernelGGL((block128_quantize_kernel<DT, FMT, RT, true, false, true>), g, b, 0, s, p);
    else if (square) hipLaunchKernelGGL((block128_quantize_kernel<DT, FMT, RT, false, true, true>), g, b, 0, s, p);
    else if (rows && cols) hipLaunchKernelGGL((block128_quantize_kernel<DT, FMT, RT, true, true, false>), g, b, 0, s, p);
    else if (cols) hipLaunchKernelGGL((block128_quantize_kernel<DT, FMT, RT, false, true, false>), g, b, 0, s, p);
    else hipLaunchKernelGGL((block128_quantize_kernel<DT, FMT, RT, true, false, false>), g, b, 0, s, p);
  } else {
    hipLaunchKernelGGL((block128_quantize_kernel<DT, FMT, RT, true, false, false>), g, b, 0, s, p);
  }
}

template <int DT>
void launch_quantize(const QuantParams& p, int fmt, bool few, bool rows, bool cols, bool square, unsigned grid,
                     hipStream_t s) {
  if (fmt == MXG_FMT_E4M3) {
    if (few) launch_quantize<DT, 0, 1>(p, rows, cols, square, grid, s);
    else launch_quantize<DT, 0, 8>(p, rows, cols, square, grid, s);
  } else {
    if (few) launch_quantize<DT, 1, 1>(p, rows, cols, square, grid, s);
    else launch_quantize<DT, 1, 8>(p, rows, cols, square, grid, s);
  }
}

// --- product ----------------------------------------------------------------------

int check_gemm(int64_t ldc, int64_t M, int64_t N, int64_t K, int64_t L, int fa, int fb, int ct, unsigned flags) {
  if (M < 0 || N < 0 || K < 0 || L < 0 || ldc < N) return MXG_ERR_SHAPE;
  for (int f : {fa, fb})
    if (f != MXG_FMT_E4M3 && f != MXG_FMT_E5M2) return MXG_ERR_FMT;
  if (ct < MXG_DT_F32 || ct > MXG_DT_F16) return MXG_ERR_FMT;
  if (flags & ~(unsigned)(MXG_B128_B_ROWS | MXG_B128_ACCUMULATE)) return MXG_ERR_FLAGS;
  if ((flags & MXG_B128_ACCUMULATE) && ct != MXG_DT_F32) return MXG_ERR_FLAGS;
  const int64_t top = 0x7FFFFF00LL;
  // a tile's 256 rows of A, B or C are addressed with 32-bit byte offsets
  if (M > top || N > top || L > top || K > (1LL << 23) - 16 || ldc > (1LL << 21)) return MXG_ERR_SHAPE;
  if (L * cdiv(M, 32) > 0x7FFFFFFFLL / std::max<int64_t>(1, cdiv(N, 32))) return MXG_ERR_SHAPE;
  // K steps of all tiles are counted in 32 bits
  if (L * cdiv(M, 32) * cdiv(N, 32) > 0x7FFFFFFFLL / (cdiv(K, 128) + 1) * 16) return MXG_ERR_SHAPE;
  if (K % 16 != 0) return MXG_ERR_ALIGN;
  return MXG_OK;
}

// Which kernel, tile and division of K.  rows: a kernel for few rows of A.
//
// Tiles: the time in microseconds of a tile size is taken as
//   rounds of work items over the compute units x (blocks of K x block x (1 - idle x gain) + end)
// where idle is the share of compute units without work (the larger tiles, which
// power bounds, gain by it; the smaller ones wait for memory), and, where K is
// divided, the second kernel that adds the parts up.  block and end were measured on MI355X, one
// size forced at a time.  16-bit C, the best and its neighbours:
//   128x7168x2048     64 x 64 7.1     64 x 128 8.4   128 x 128 11.1
//   512x4096x7168     64 x 128 21.7   64 x 64 27.7   128 x 128 28.6
//   1024x4096x7168    128 x 128 36.5  64 x 128 40.9  128 x 256 54.1
//   2048x4096x4096    128 x 256 38.6  128 x 128 46.6 256 x 256 48.5
//   4096x4096x4096    256 x 256 63.3  128 x 256 74.9 128 x 128 81.5
// float32 C:
//   128x7168x2048     64 x 64 10.1    64 x 128 12.4  128 x 128 17.0
//   512x4096x7168     64 x 128 36.4   64 x 64 44.1   128 x 128 47.5
//   4000x7168x2048    128 x 128 115.4 128 x 256 121.3 64 x 128 139.9
//   2048x4096x4096    128 x 256 61.6  128 x 128 64.1 64 x 128 77.1
// K is divided only where tiles leave compute units idle: 64x1024x7168 in 4
// parts 10.3 us, in one 14.8; 128x2048x7168 12.7 and 14.3; 256x1024x4096 10.5
// and 9.9, with a float32 C 12.7 and 15.4.
struct Choice {
  int rows;                // columns per workgroup of the rows kernel, 0: tiles
  int bm, bn, kb, splits;  // tile; blocks of K per step; parts of K
};

constexpr int kUnits = 256;  // compute units: the choice, and with it the workspace, must not need a device

Choice choose(int64_t M, int64_t N, int64_t K, int64_t L, bool exact) {
  // a rows workgroup reads A once for its columns, so more columns are better as long as they leave enough
  // workgroups (7168 columns: 32 at a time 4.9 us, 16 5.1 us; 4096: 7.3 and 5.8 us; K = 2048 and 4096)
  // Up to 32 rows too, unless there are more workgroups than compute units (32x24576x1536: 11.7 us, tiles 9.7) or, for
  // a 16-bit C, K is long (32x7168x2048: 6.9 us, tiles 7.0; 32x6144x4096: 10.8 and 10.1; float32 C: 7.3 and 9.8, 11.3
  // and 14.0).  Where the two cross moves with rows and columns: 32 rows at K = 2560 from 6144 columns on and past 4096
  // below that (32x4096x4096: 8.9 us, tiles 10.0), 24 rows at 3328, 17 rows past 6144 (17x7168x4096: 9.4 and 10.0);
  // 2048 is on the safe side of all of them.  With 64 rows tiles are as fast or faster (64x7168x2048: 9.2 us, tiles 7.2; float32 C: 9.5 and 9.6).
  if (M <= 16 || (M <= 32 && L * cdiv(N, 32) <= kUnits && (exact || K <= 2048))) return {L * cdiv(N, 32) >= kUnits * 3 / 4 ? 32 : 16, 16, 0, 1, 1};
  struct Size {
    int bm, bn, kb;
    bool divides;  // its kernel can take part of K
    double block, end, gain;
  };
  static constexpr Size kSizes[2][5] = {{{64, 64, 2, true, 0.215, 0.5, 0.0},
                                         {64, 128, 2, true, 0.335, 0.7, 0.0},
                                         {128, 128, 1, false, 0.64, 1.0, 0.3},
                                         {128, 256, 1, false, 1.08, 2.0, 0.3},
                                         {256, 256, 1, false, 1.8, 3.0, 0.3}},
                                        {{64, 64, 2, true, 0.355, 0.8, 0.0},
                                         {64, 128, 2, true, 0.585, 1.0, 0.0},
                                         {128, 128, 2, true, 0.97, 1.3, 0.3},
                                         {128, 256, 1, false, 1.85, 2.0, 0.3}}};
  const int64_t blocks = cdiv(K, 128);
  Choice best{};
  double best_time = 0;
  for (const Size& t : kSizes[exact]) {
    if (t.bm == 0) break;
    const int64_t tiles = L * cdiv(M, t.bm) * cdiv(N, t.bn), steps = cdiv(blocks, t.kb);
    for (int splits : {1, 2, 3, 4, 6, 8, 12, 16}) {
      if (splits > 1 && (!t.divides || splits > steps || tiles * (splits - 1) >= kUnits)) break;
      const int64_t per = cdiv(steps, splits), parts = cdiv(steps, per);
      const double idle = 1.0 - std::min<double>(tiles * parts, kUnits) / kUnits;
      double time = (double)cdiv(tiles * parts, kUnits) * (per * t.kb * t.block * (1.0 - idle * t.gain) + t.end);
      // written and read at 3 TB/s, one part after the other
      if (parts > 1) time += 4.0 + 0.12 * parts + parts * L * M * N * 8 / 3e6;
      if (best.bm == 0 || time < best_time) {
        best = {0, t.bm, t.bn, t.kb, (int)parts};
        best_time = time;
      }
    }
  }
  return best;
}

// float32 columns of a row of the parts' sums
int64_t sums_ld(int64_t N) { return (N + 3) / 4 * 4; }

}  // namespace

extern "C" {

int mxgemm_block128_quantize(const void* X, int64_t ldx, void* Q, float* S, void* QT, float* ST, int64_t M, int64_t K,
                             int64_t L, int x_dtype, int fmt, unsigned flags, void* stream) {
  const bool trusted = take_trust(&flags);
  int st = check_quantize(ldx, M, K, L, x_dtype, fmt, flags);
  if (st != MXG_OK) return st;
  if (M == 0 || K == 0 || L == 0) return MXG_OK;
  const bool rows = Q != nullptr, cols = QT != nullptr, square = (flags & MXG_QUANT_SQUARE) != 0;
  if (!X || (!rows && !cols) || rows != (S != nullptr) || cols != (ST != nullptr)) return MXG_ERR_NULL;
  const size_t e = mxg::elem_bytes(x_dtype);
  if (!aligned_to(X, e) || !aligned16(Q) || !aligned16(QT) || !aligned_to(S, 4) || !aligned_to(ST, 4))
    return MXG_ERR_ALIGN;
  int dev = 0, cus = 0;
  st = device_check(&dev, &cus);
  if (st != MXG_OK) return st;
  if (!trusted && (!on_device(X, dev) || (rows && (!on_device(Q, dev) || !on_device(S, dev))) ||
      (cols && (!on_device(QT, dev) || !on_device(ST, dev)))))
    return MXG_ERR_DEVICE;
  QuantParams p{};
  p.X = X;
  p.Q = static_cast<uint8_t*>(Q);
  p.S = S;
  p.QT = static_cast<uint8_t*>(QT);
  p.ST = ST;
  p.ldx = ldx;
  p.M = (int)M;
  p.K = (int)K;
  p.L = (int)L;
  p.K16 = (int)up16(K);
  p.M16 = (int)up16(M);
  p.Mb = (int)cdiv(M, 128);
  p.Kb = (int)cdiv(K, 128);
  p.pow2 = (flags & MXG_QUANT_POW2) != 0;
  // rows alone, and too few of them for 128-row tiles to fill the chip: 16 rows to a workgroup
  const bool few = rows && !cols && !square && L * p.Mb * p.Kb < 4LL * cus;
  p.tiles_m = few ? (int)cdiv(M, 16) : p.Mb;
  const int64_t grid = L * p.tiles_m * p.Kb;
  hipStream_t s = (hipStream_t)stream;
  launch_runs(grid, [&](int64_t first, unsigned count) {
    p.first = (int)first;
    if (x_dtype == MXG_DT_F32) launch_quantize<0>(p, fmt, few, rows, cols, square, count, s);
    else if (x_dtype == MXG_DT_BF16) launch_quantize<1>(p, fmt, few, rows, cols, square, count, s);
    else launch_quantize<2>(p, fmt, few, rows, cols, square, count, s);
  });
  return hipGetLastError() == hipSuccess ? MXG_OK : MXG_ERR_LAUNCH;
}

size_t mxgemm_block128_workspace_bytes(int64_t M, int64_t N, int64_t K, int64_t L, int c_dtype) {
  if (check_gemm(N, M, N, K, L, MXG_FMT_E4M3, MXG_FMT_E4M3, c_dtype, 0) != MXG_OK || M == 0 || N == 0 || K == 0 || L == 0)
    return 0;
  const Choice ch = choose(M, N, K, L, c_dtype == MXG_DT_F32);
  return ch.splits > 1 ? (size_t)(ch.splits * L * M * sums_ld(N) * 4) : 0;
}

int mxgemm_block128(const void* A, const float* SA, const void* B, const float* SB, void* C, int64_t ldc, int64_t M,
                    int64_t N, int64_t K, int64_t L, int a_fmt, int b_fmt, int c_dtype, unsigned flags, void* workspace,
                    size_t workspace_bytes, void* stream) {
  const bool trusted = take_trust(&flags);
  int st = check_gemm(ldc, M, N, K, L, a_fmt, b_fmt, c_dtype, flags);
  if (st != MXG_OK) return st;
  if (M == 0 || N == 0 || L == 0) return MXG_OK;
  if (!C || (K > 0 && (!A || !B || !SA || !SB))) return MXG_ERR_NULL;
  const size_t need = mxgemm_block128_workspace_bytes(M, N, K, L, c_dtype);
  if (need > 0 && !workspace) return MXG_ERR_NULL;
  if (need > workspace_bytes) return MXG_ERR_SHAPE;
  if (!aligned16(A) || !aligned16(B) || !aligned_to(SA, 4) || !aligned_to(SB, 4) ||
      !aligned_to(C, mxg::elem_bytes(c_dtype)) || (need > 0 && !aligned16(workspace)))
    return MXG_ERR_ALIGN;
  int dev = 0, cus = 0;
  st = device_check(&dev, &cus);
  if (st != MXG_OK) return st;
  if (!trusted && (!on_device(C, dev) || (K > 0 && (!on_device(A, dev) || !on_device(B, dev) || !on_device(SA, dev) ||
                                       !on_device(SB, dev))) ||
      (need > 0 && !on_device(workspace, dev))))
    return MXG_ERR_DEVICE;
  GemmParams p{};
  p.A = static_cast<const uint8_t*>(A);
  p.B = static_cast<const uint8_t*>(B);
  p.SA = SA;
  p.SB = SB;
  p.C = C;
  p.ldc = ldc;
  p.M = (int)M;
  p.N = (int)N;
  p.K = (int)K;
  p.L = (int)L;
  p.Kb = (int)cdiv(K, 128);
  p.Nb = (int)cdiv(N, 128);
  p.b_rows = (flags & MXG_B128_B_ROWS) != 0;
  p.accumulate = (flags & MXG_B128_ACCUMULATE) != 0;
  hipStream_t s = (hipStream_t)stream;
  if (K == 0) {
    if (p.accumulate) return MXG_OK;
    const dim3 g((unsigned)std::min<int64_t>(cdiv(L * M * N, 256), 16LL * cus)), b(256);
    if (c_dtype == MXG_DT_F32) hipLaunchKernelGGL((mxg::b128::block128_zero_kernel<0>), g, b, 0, s, p);
    else if (c_dtype == MXG_DT_BF16) hipLaunchKernelGGL((mxg::b128::block128_zero_kernel<1>), g, b, 0, s, p);
    else hipLaunchKernelGGL((mxg::b128::block128_zero_kernel<2>), g, b, 0, s, p);
    return hipGetLastError() == hipSuccess ? MXG_OK : MXG_ERR_LAUNCH;
  }
  const bool exact = c_dtype == MXG_DT_F32;
  const int per16 = exact ? 4 : 8;
  p.c_vec = aligned16(C) && ldc % per16 == 0 && N % per16 == 0;
  const Choice ch = choose(M, N, K, L, exact);
  if (ch.rows) {
    p.tilesN = (int)cdiv(N, ch.rows);
    hipError_t e = hipSuccess;
    launch_runs(L * p.tilesN, [&](int64_t first, unsigned count) {
      p.first = (int)first;
      if (e == hipSuccess) e = mxg::b128::launch_rows(p, a_fmt, b_fmt, c_dtype, ch.rows, count, s);
    });
    return e == hipSuccess ? MXG_OK : MXG_ERR_LAUNCH;
  }
  p.tilesM = (int)cdiv(M, ch.bm);
  p.tilesN = (int)cdiv(N, ch.bn);
  p.num_tiles = (int)(L * p.tilesM * p.tilesN);
  p.steps = (int)cdiv(p.Kb, ch.kb);
  p.per = (int)cdiv(p.steps, ch.splits);
  p.splits = ch.splits;
  const int64_t grid = std::min<int64_t>((int64_t)p.num_tiles * p.splits, cus);
  p.xcd_remap = grid % 8 == 0;
  GemmParams last = p;  // what adds the parts up
  if (p.splits > 1) {
    p.sums = last.sums = static_cast<float*>(workspace);
    p.ldw = last.ldw = (int)sums_ld(N);
    if (exact) {
      // a part's sums are a float32 C of their own
      p.C = workspace;
      p.ldc = p.ldw;
      p.c_vec = N % 4 == 0;
      p.accumulate = false;
    }
  }
  hipError_t e;
  if (exact) {
    const auto f = ch.bn == 256   ? mxg::b128::launch_exact128x256
                   : ch.bm == 128 ? mxg::b128::launch_exact128
                   : ch.bn == 128 ? mxg::b128::launch_exact64x128
                                  : mxg::b128::launch_exact64;
    e = f(p, a_fmt, b_fmt, grid, s);
  } else {
    const auto f = ch.bm == 256   ? mxg::b128::launch_tile256
                   : ch.bn == 256 ? mxg::b128::launch_tile128x256
                   : ch.bm == 128 ? mxg::b128::launch_tile128
                   : ch.bn == 128 ? mxg::b128::launch_tile64x128
                                  : mxg::b128::launch_tile64;
    e = f(p, a_fmt, b_fmt, c_dtype, grid, s);
  }
  if (e == hipSuccess && p.splits > 1) {
    const dim3 g((unsigned)std::min<int64_t>(cdiv(L * M * (last.ldw / 4), 256), 8LL * cus)), b(256);
    if (exact) hipLaunchKernelGGL((mxg::b128::block128_sum_kernel<0>), g, b, 0, s, last, p.splits);
    else if (c_dtype == MXG_DT_BF16) hipLaunchKernelGGL((mxg::b128::block128_sum_kernel<1>), g, b, 0, s, last, p.splits);
    else hipLaunchKernelGGL((mxg::b128::block128_sum_kernel<2>), g, b, 0, s, last, p.splits);
    e = hipGetLastError();
  }
  return e == hipSuccess ? MXG_OK : MXG_ERR_LAUNCH;
}

}  // extern "C"
