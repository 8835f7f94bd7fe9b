// C-ABI entry points of the block-128 quantiser and product (include/mxgemm.h).
#include <hip/hip_runtime.h>

#include <algorithm>
#include <initializer_list>

#include "../../include/mxgemm.h"
#include "block128_choose.hpp"
#include "block128_ends.hpp"
#include "block128_launch.hpp"
#include "block128_quantize.hpp"
#include "host_checks.hpp"

namespace {

using namespace mxg::host;

using mxg::b128::GemmParams;
using mxg::b128::MoreParams;
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

// C from the sums of `splits` parts, or of none.
template <int CT>
void add_up(const MoreParams& p, bool ends, int splits, unsigned grid, hipStream_t s) {
  if (ends) hipLaunchKernelGGL((mxg::b128::block128_sum_kernel<CT, mxg::b128::kEnds>), dim3(grid), dim3(256), 0, s, p, splits);
  else hipLaunchKernelGGL((mxg::b128::block128_sum_kernel<CT, mxg::b128::kPlain>), dim3(grid), dim3(256), 0, s, static_cast<const GemmParams&>(p), splits);
}
hipError_t add_up(const MoreParams& p, bool ends, int splits, int c_dtype, int cus, hipStream_t s) {
  const unsigned grid = (unsigned)std::min<int64_t>(cdiv((int64_t)p.L * p.M * (p.ldw / 4), 256), 8LL * cus);
  if (c_dtype == MXG_DT_F32) add_up<0>(p, ends, splits, grid, s);
  else if (c_dtype == MXG_DT_BF16) add_up<1>(p, ends, splits, grid, s);
  else add_up<2>(p, ends, splits, grid, s);
  return hipGetLastError();
}

// C = A B^T, and with ends what follows it.
int product(const void* A, const float* SA, const void* B, const float* SB, void* C, int64_t ldc, int64_t M, int64_t N,
            int64_t K, int64_t L, int a_fmt, int b_fmt, int c_dtype, const mxgemm_ends_t* ends, unsigned flags,
            void* workspace, size_t workspace_bytes, void* stream) {
  const bool trusted = take_trust(&flags);
  int st = check_gemm(ldc, M, N, K, L, a_fmt, b_fmt, c_dtype, flags);
  if (st != MXG_OK) return st;
  if (ends && (st = mxg::b128::check_ends(*ends, N, c_dtype)) != MXG_OK) return st;
  if (M == 0 || N == 0 || L == 0) return MXG_OK;
  if (!C || (K > 0 && (!A || !B || !SA || !SB))) return MXG_ERR_NULL;
  const size_t need = mxgemm_block128_workspace_bytes(M, N, K, L, c_dtype);
  if (need > 0 && !workspace) return MXG_ERR_NULL;
  if (need > workspace_bytes) return MXG_ERR_SHAPE;
  if (!aligned16(A) || !aligned16(B) || !aligned_to(SA, 4) || !aligned_to(SB, 4) ||
      !aligned_to(C, mxg::elem_bytes(c_dtype)) || (need > 0 && !aligned16(workspace)))
    return MXG_ERR_ALIGN;
  if (ends && !mxg::b128::ends_aligned(*ends, c_dtype)) return MXG_ERR_ALIGN;
  int dev = 0, cus = 0;
  st = device_check(&dev, &cus);
  if (st != MXG_OK) return st;
  if (!trusted && (!on_device(C, dev) || (K > 0 && (!on_device(A, dev) || !on_device(B, dev) || !on_device(SA, dev) ||
                                       !on_device(SB, dev))) ||
      (need > 0 && !on_device(workspace, dev))))
    return MXG_ERR_DEVICE;
  if (ends && !trusted && !mxg::b128::ends_on_device(*ends, dev)) return MXG_ERR_DEVICE;
  if (ends) {
    const int64_t kb = cdiv(K, 128);
    if (mxg::b128::outputs_overlap(rows_at(C, M, N, ldc, mxg::elem_bytes(c_dtype)), ends, c_dtype,
                                   {flat(A, M * K), flat(SA, 4 * kb * M), flat(B, N * K), flat(SB, 4 * kb * cdiv(N, 128)),
                                    flat(workspace, (int64_t)need)}))
      return MXG_ERR_SHAPE;
  }
  MoreParams p{};
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
  if (ends) p.ends = mxg::b128::kernel_ends(*ends);
  hipStream_t s = (hipStream_t)stream;
  if (K == 0 && ends) {
    p.ldw = (int)mxg::b128::sums_ld(N);
    return add_up(p, true, 0, c_dtype, cus, s) == hipSuccess ? MXG_OK : MXG_ERR_LAUNCH;
  }
  if (K == 0) {
    if (p.accumulate) return MXG_OK;
    const dim3 g((unsigned)std::min<int64_t>(cdiv(L * M * N, 256), 16LL * cus)), b(256);
    if (c_dtype == MXG_DT_F32) hipLaunchKernelGGL((mxg::b128::block128_zero_kernel<0>), g, b, 0, s, static_cast<const GemmParams&>(p));
    else if (c_dtype == MXG_DT_BF16) hipLaunchKernelGGL((mxg::b128::block128_zero_kernel<1>), g, b, 0, s, static_cast<const GemmParams&>(p));
    else hipLaunchKernelGGL((mxg::b128::block128_zero_kernel<2>), g, b, 0, s, static_cast<const GemmParams&>(p));
    return hipGetLastError() == hipSuccess ? MXG_OK : MXG_ERR_LAUNCH;
  }
  const bool exact = c_dtype == MXG_DT_F32;
  const int per16 = exact ? 4 : 8;
  p.c_vec = aligned16(C) && ldc % per16 == 0 && N % per16 == 0 && (!ends || mxg::b128::ends_whole(*ends, per16));
  const mxg::b128::Choice ch = mxg::b128::choose(M, N, K, L, exact);
  if (ch.rows) {
    p.tilesN = (int)cdiv(N, ch.rows);
    hipError_t e = hipSuccess;
    launch_runs(L * p.tilesN, [&](int64_t first, unsigned count) {
      p.first = (int)first;
      if (e != hipSuccess) return;
      if (ends) e = mxg::b128::launch_rows_more(mxg::b128::kEnds, p, a_fmt, b_fmt, c_dtype, M <= 16 ? 16 : 32, ch.rows, count, s);
      else e = mxg::b128::launch_rows(p, a_fmt, b_fmt, c_dtype, ch.rows, count, s);
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
  MoreParams last = p;  // what adds the parts up
  if (p.splits > 1) {
    p.sums = last.sums = static_cast<float*>(workspace);
    p.ldw = last.ldw = (int)mxg::b128::sums_ld(N);
    if (exact) {
      // a part's sums are a float32 C of their own
      p.C = workspace;
      p.ldc = p.ldw;
      p.c_vec = N % 4 == 0;
      p.accumulate = false;
    }
  }
  hipError_t e = ends && p.splits == 1 ? mxg::b128::more_launch(ch, exact)(mxg::b128::kEnds, p, a_fmt, b_fmt, c_dtype, grid, s)
                                       : mxg::b128::tile_launch(ch, exact)(p, a_fmt, b_fmt, c_dtype, grid, s);
  if (e == hipSuccess && p.splits > 1) e = add_up(last, ends != nullptr, p.splits, c_dtype, cus, s);
  return e == hipSuccess ? MXG_OK : MXG_ERR_LAUNCH;
}

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
  const mxg::b128::Choice ch = mxg::b128::choose(M, N, K, L, c_dtype == MXG_DT_F32);
  return ch.splits > 1 ? (size_t)(ch.splits * L * M * mxg::b128::sums_ld(N) * 4) : 0;
}

int mxgemm_block128(const void* A, const float* SA, const void* B, const float* SB, void* C, int64_t ldc, int64_t M,
                    int64_t N, int64_t K, int64_t L, int a_fmt, int b_fmt, int c_dtype, unsigned flags, void* workspace,
                    size_t workspace_bytes, void* stream) {
  return product(A, SA, B, SB, C, ldc, M, N, K, L, a_fmt, b_fmt, c_dtype, nullptr, flags, workspace, workspace_bytes, stream);
}

int mxgemm_block128_linear(const void* A, const float* SA, const void* B, const float* SB, void* C, int64_t ldc, int64_t M,
                           int64_t N, int64_t K, int a_fmt, int b_fmt, int c_dtype, const mxgemm_ends_t* ends, unsigned flags,
                           void* workspace, size_t workspace_bytes, void* stream) {
  if (!ends) return MXG_ERR_NULL;
  if (flags & ~(unsigned)MXG_TRUSTED_POINTERS) return MXG_ERR_FLAGS;
  return product(A, SA, B, SB, C, ldc, M, N, K, 1, a_fmt, b_fmt, c_dtype, ends, flags, workspace, workspace_bytes, stream);
}

}  // extern "C"
