// C-ABI entry points of the block-128 products and quantiser on rows in groups (include/mxgemm.h).
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
using namespace mxg::b128;

int64_t up16(int64_t v) { return (v + 15) / 16 * 16; }

constexpr int64_t kTop = 0x7FFFFF00LL;

int check_groups(int64_t T, int64_t E) {
  return T < 0 || E < 0 || T > mxg::groups::kMaxRows || E > mxg::groups::kMaxGroups ? MXG_ERR_SHAPE : MXG_OK;
}

// Sizes of the weights' gradient.
int check_deep(int64_t blocks, int64_t E, int64_t M, int64_t N) {
  if (blocks < 0 || M < 0 || N < 0 || check_groups(0, E) != MXG_OK) return MXG_ERR_SHAPE;
  if (M > kTop || N > kTop || blocks > (1 << 16) - 1) return MXG_ERR_SHAPE;
  if (E * cdiv(M, 32) > 0x7FFFFFFFLL / std::max<int64_t>(1, cdiv(N, 32))) return MXG_ERR_SHAPE;
  return MXG_OK;
}

bool offsets_aligned(const void* offsets, unsigned flags) {
  return aligned_to(offsets, (flags & MXG_GROUP_OFFSETS64) ? 8 : 4);
}

int64_t offsets_bytes(int64_t E, unsigned flags) { return (E + 1) * ((flags & MXG_GROUP_OFFSETS64) ? 8 : 4); }

mxg::groups::Groups groups_of(const void* offsets, int64_t T, int64_t E, unsigned flags) {
  return {offsets, (int)E, (int)T, (flags & MXG_GROUP_OFFSETS64) != 0};
}

// C (L, M, N) = 0
hipError_t zero(const GemmParams& p, int c_dtype, int cus, hipStream_t s) {
  const dim3 g((unsigned)std::min<int64_t>(cdiv((int64_t)p.L * p.M * p.N, 256), 16LL * cus)), b(256);
  if (c_dtype == MXG_DT_F32) hipLaunchKernelGGL((block128_zero_kernel<0>), g, b, 0, s, p);
  else if (c_dtype == MXG_DT_BF16) hipLaunchKernelGGL((block128_zero_kernel<1>), g, b, 0, s, p);
  else hipLaunchKernelGGL((block128_zero_kernel<2>), g, b, 0, s, p);
  return hipGetLastError();
}

template <int DT, int FMT>
void launch_quantize(const GroupQuantParams& p, bool rows, unsigned grid, hipStream_t s) {
  const dim3 g(grid), b(kQThreads);
  if (rows) hipLaunchKernelGGL((block128_quantize_kernel<DT, FMT, 8, true, true, false, true>), g, b, 0, s, p);
  else hipLaunchKernelGGL((block128_quantize_kernel<DT, FMT, 8, false, true, false, true>), g, b, 0, s, p);
}
template <int DT>
void launch_quantize(const GroupQuantParams& p, int fmt, bool rows, unsigned grid, hipStream_t s) {
  if (fmt == MXG_FMT_E4M3) launch_quantize<DT, 0>(p, rows, grid, s);
  else launch_quantize<DT, 1>(p, rows, grid, s);
}

}  // namespace

extern "C" {

int64_t mxgemm_group_blocks(int64_t T, int64_t E) { return check_groups(T, E) == MXG_OK ? group_blocks(T, E) : 0; }

int mxgemm_block128_quantize_grouped(const void* X, int64_t ldx, const void* offsets, void* Q, float* S, void* QT, float* ST,
                                     int64_t T, int64_t E, int64_t K, int x_dtype, int fmt, unsigned flags, void* stream) {
  const bool trusted = take_trust(&flags);
  int st = check_groups(T, E);
  if (st != MXG_OK) return st;
  if (K < 0 || ldx < K) return MXG_ERR_SHAPE;
  if (x_dtype < MXG_DT_F32 || x_dtype > MXG_DT_F16 || (fmt != MXG_FMT_E4M3 && fmt != MXG_FMT_E5M2)) return MXG_ERR_FMT;
  if (flags & ~(unsigned)(MXG_QUANT_POW2 | MXG_GROUP_OFFSETS64)) return MXG_ERR_FLAGS;
  if (K > kTop || ldx > (1LL << 40)) return MXG_ERR_SHAPE;
  const int64_t blocks = group_blocks(T, E);
  // the blocks, and those of rows before the first group and behind the last one
  const int64_t tiles = Q ? (T + 127 * (std::min(T, E) + 2)) / 128 : blocks;
  if (K && tiles > 0x7FFFFFFFLL / cdiv(K, 128)) return MXG_ERR_SHAPE;
  if (T == 0 || K == 0) return MXG_OK;
  if (!X || !offsets || (blocks > 0 && (!QT || !ST)) || (Q != nullptr) != (S != nullptr)) return MXG_ERR_NULL;
  if (!aligned_to(X, mxg::elem_bytes(x_dtype)) || !aligned16(Q) || !aligned16(QT) || !aligned_to(S, 4) || !aligned_to(ST, 4) ||
      !offsets_aligned(offsets, flags))
    return MXG_ERR_ALIGN;
  int dev = 0, cus = 0;
  st = device_check(&dev, &cus);
  if (st != MXG_OK) return st;
  if (!trusted)
    for (const void* t : {X, offsets, (const void*)Q, (const void*)S, (const void*)QT, (const void*)ST})
      if (t && !on_device(t, dev)) return MXG_ERR_DEVICE;
  GroupQuantParams p{};
  p.X = X;
  p.Q = static_cast<uint8_t*>(Q);
  p.S = S;
  p.QT = static_cast<uint8_t*>(QT);
  p.ST = ST;
  p.ldx = ldx;
  p.M = (int)T;
  p.K = (int)K;
  p.L = 1;
  p.K16 = (int)up16(K);
  p.M16 = (int)(128 * blocks);
  p.Mb = (int)blocks;
  p.Kb = (int)cdiv(K, 128);
  p.tiles_m = (int)tiles;
  p.pow2 = (flags & MXG_QUANT_POW2) != 0;
  p.groups = groups_of(offsets, T, E, flags);
  hipStream_t s = (hipStream_t)stream;
  launch_runs(tiles * p.Kb, [&](int64_t first, unsigned count) {
    p.first = (int)first;
    if (x_dtype == MXG_DT_F32) launch_quantize<0>(p, fmt, Q != nullptr, count, s);
    else if (x_dtype == MXG_DT_BF16) launch_quantize<1>(p, fmt, Q != nullptr, count, s);
    else launch_quantize<2>(p, fmt, Q != nullptr, count, s);
  });
  return hipGetLastError() == hipSuccess ? MXG_OK : MXG_ERR_LAUNCH;
}

int mxgemm_block128_grouped(const void* A, const float* SA, const void* B, const float* SB, const void* offsets, void* C,
                            int64_t ldc, int64_t T, int64_t E, int64_t N, int64_t K, int a_fmt, int b_fmt, int c_dtype,
                            const mxgemm_ends_t* ends, unsigned flags, void* stream) {
  const bool trusted = take_trust(&flags);
  int st = check_groups(T, E);
  if (st != MXG_OK) return st;
  if (N < 0 || K < 1 || ldc < N) return MXG_ERR_SHAPE;
  for (int f : {a_fmt, b_fmt})
    if (f != MXG_FMT_E4M3 && f != MXG_FMT_E5M2) return MXG_ERR_FMT;
  if (c_dtype < MXG_DT_F32 || c_dtype > MXG_DT_F16) return MXG_ERR_FMT;
  if (flags & ~(unsigned)(MXG_GROUP_OFFSETS64 | MXG_GROUP_ZERO_REST | MXG_GROUP_ZERO_PREACT)) return MXG_ERR_FLAGS;
  if (N > kTop || K > (1LL << 23) - 16 || ldc > (1LL << 21)) return MXG_ERR_SHAPE;
  if ((cdiv(T, 16) + E) > 0x7FFFFFFFLL / std::max<int64_t>(1, cdiv(N, 16))) return MXG_ERR_SHAPE;
  if (ends) {
    if (ends->bias || ends->residual) return MXG_ERR_FLAGS;
    st = check_ends(*ends, N, c_dtype);
    if (st != MXG_OK) return st;
  }
  if (K % 16 != 0) return MXG_ERR_ALIGN;
  if (T == 0 || N == 0) return MXG_OK;
  if (!offsets || !C || (E > 0 && (!A || !SA || !B || !SB))) return MXG_ERR_NULL;
  if (!aligned16(A) || !aligned16(B) || !aligned_to(SA, 4) || !aligned_to(SB, 4) || !aligned_to(C, mxg::elem_bytes(c_dtype)) ||
      !offsets_aligned(offsets, flags) || (ends && !ends_aligned(*ends, c_dtype)))
    return MXG_ERR_ALIGN;
  int dev = 0, cus = 0;
  st = device_check(&dev, &cus);
  if (st != MXG_OK) return st;
  if (!trusted) {
    for (const void* t : {A, (const void*)SA, B, (const void*)SB, offsets, (const void*)C})
      if (t && !on_device(t, dev)) return MXG_ERR_DEVICE;
    if (ends && !ends_on_device(*ends, dev)) return MXG_ERR_DEVICE;
  }
  if (outputs_overlap(rows_at(C, T, N, ldc, mxg::elem_bytes(c_dtype)), ends, c_dtype,
                      {flat(A, T * K), flat(SA, 4 * cdiv(K, 128) * T), flat(B, E * N * K), flat(SB, 4 * E * cdiv(N, 128) * cdiv(K, 128)),
                       flat(offsets, offsets_bytes(E, flags))}))
    return MXG_ERR_SHAPE;
  MoreParams p{};
  p.A = static_cast<const uint8_t*>(A);
  p.B = static_cast<const uint8_t*>(B);
  p.SA = SA;
  p.SB = SB;
  p.C = C;
  p.ldc = ldc;
  p.M = (int)T;
  p.N = (int)N;
  p.K = (int)K;
  p.L = 1;
  p.Kb = (int)cdiv(K, 128);
  p.Nb = (int)cdiv(N, 128);
  p.groups = groups_of(offsets, T, E, flags);
  p.zero_c = (flags & MXG_GROUP_ZERO_REST) != 0;
  p.zero_z = (flags & MXG_GROUP_ZERO_PREACT) != 0;
  if (ends) p.ends = kernel_ends(*ends);
  hipStream_t s = (hipStream_t)stream;
  if (E == 0) {  // every row is of no group
    hipError_t e = p.zero_c ? zero(p, c_dtype, cus, s) : hipSuccess;
    if (e == hipSuccess && p.zero_z && p.ends.Z) {
      p.C = p.ends.Z;
      p.ldc = p.ends.ldz;
      e = zero(p, c_dtype, cus, s);
    }
    return e == hipSuccess ? MXG_OK : MXG_ERR_LAUNCH;
  }
  const bool exact = c_dtype == MXG_DT_F32;
  const int per16 = exact ? 4 : 8;
  p.c_vec = aligned16(C) && ldc % per16 == 0 && N % per16 == 0 && (!ends || ends_whole(*ends, per16));
  const Choice ch = choose_grouped(T, E, N, K, exact);
  const int64_t some = std::min(T, E);  // groups that can have rows
  if (ch.rows) {
    p.tilesN = (int)cdiv(N, ch.rows);
    const int64_t chunks = (T + (ch.bm - 1) * some) / ch.bm;
    p.num_tiles = (int)(chunks * p.tilesN);
    hipError_t e = hipSuccess;
    launch_runs(p.num_tiles, [&](int64_t first, unsigned count) {
      p.first = (int)first;
      if (e == hipSuccess) e = launch_rows_more(kRowGroups, p, a_fmt, b_fmt, c_dtype, ch.bm, ch.rows, count, s);
    });
    return e == hipSuccess ? MXG_OK : MXG_ERR_LAUNCH;
  }
  p.tilesM = (int)((T + (ch.bm - 1) * some) / ch.bm);  // of all groups, at most
  p.tilesN = (int)cdiv(N, ch.bn);
  p.num_tiles = (int)((int64_t)p.tilesM * p.tilesN);
  p.steps = (int)cdiv(p.Kb, ch.kb);
  p.splits = 1;
  const int64_t grid = std::min<int64_t>(p.num_tiles, cus);
  p.xcd_remap = grid % 8 == 0;
  return more_launch(ch, exact)(kRowGroups, p, a_fmt, b_fmt, c_dtype, grid, s) == hipSuccess ? MXG_OK : MXG_ERR_LAUNCH;
}

size_t mxgemm_block128_grouped_weight_gradient_workspace_bytes(int64_t blocks, int64_t E, int64_t M, int64_t N) {
  if (check_deep(blocks, E, M, N) != MXG_OK || blocks == 0 || E == 0 || M == 0 || N == 0) return 0;
  const Choice ch = choose_deep(blocks, E, M, N);
  return ch.splits > 1 ? (size_t)(ch.splits * E * M * sums_ld(N) * 4) : 0;
}

int mxgemm_block128_grouped_weight_gradient(const void* A, const float* SA, const void* B, const float* SB, const void* offsets,
                                            float* C, int64_t ldc, int64_t blocks, int64_t E, int64_t M, int64_t N, int a_fmt,
                                            int b_fmt, unsigned flags, void* workspace, size_t workspace_bytes,
                                            void* stream) {
  const bool trusted = take_trust(&flags);
  int st = check_deep(blocks, E, M, N);
  if (st != MXG_OK) return st;
  if (ldc < N || ldc > (1LL << 21)) return MXG_ERR_SHAPE;
  for (int f : {a_fmt, b_fmt})
    if (f != MXG_FMT_E4M3 && f != MXG_FMT_E5M2) return MXG_ERR_FMT;
  if (flags & ~(unsigned)(MXG_GROUP_OFFSETS64 | MXG_B128_ACCUMULATE)) return MXG_ERR_FLAGS;
  if (E == 0 || M == 0 || N == 0) return MXG_OK;
  if (!C || (blocks > 0 && (!A || !SA || !B || !SB || !offsets))) return MXG_ERR_NULL;
  const size_t need = mxgemm_block128_grouped_weight_gradient_workspace_bytes(blocks, E, M, N);
  if (need > 0 && !workspace) return MXG_ERR_NULL;
  if (need > workspace_bytes) return MXG_ERR_SHAPE;
  if (!aligned16(A) || !aligned16(B) || !aligned_to(SA, 4) || !aligned_to(SB, 4) || !aligned_to(C, 4) ||
      !offsets_aligned(offsets, flags) || (need > 0 && !aligned16(workspace)))
    return MXG_ERR_ALIGN;
  int dev = 0, cus = 0;
  st = device_check(&dev, &cus);
  if (st != MXG_OK) return st;
  if (!trusted)
    for (const void* t : {A, (const void*)SA, B, (const void*)SB, offsets, (const void*)C, need > 0 ? (const void*)workspace : nullptr})
      if (t && !on_device(t, dev)) return MXG_ERR_DEVICE;
  if (outputs_overlap(rows_at(C, E * M, N, ldc, 4), nullptr, MXG_DT_F32,
                      {flat(A, 128 * blocks * M), flat(SA, 4 * blocks * M), flat(B, 128 * blocks * N), flat(SB, 4 * blocks * N),
                       flat(offsets, offsets_bytes(E, flags)), flat(workspace, (int64_t)need)}))
    return MXG_ERR_SHAPE;
  MoreParams p{};
  p.A = static_cast<const uint8_t*>(A);
  p.B = static_cast<const uint8_t*>(B);
  p.SA = SA;
  p.SB = SB;
  p.C = C;
  p.ldc = ldc;
  p.M = (int)M;
  p.N = (int)N;
  p.K = (int)(128 * blocks);
  p.L = (int)E;
  p.Kb = (int)blocks;
  p.b_rows = true;
  p.accumulate = (flags & MXG_B128_ACCUMULATE) != 0;
  hipStream_t s = (hipStream_t)stream;
  if (blocks == 0) return p.accumulate || zero(p, MXG_DT_F32, cus, s) == hipSuccess ? MXG_OK : MXG_ERR_LAUNCH;
  p.groups = groups_of(offsets, 128 * blocks, E, flags);
  p.c_vec = aligned16(C) && ldc % 4 == 0 && N % 4 == 0;
  const Choice ch = choose_deep(blocks, E, M, N);
  p.tilesM = (int)cdiv(M, ch.bm);
  p.tilesN = (int)cdiv(N, ch.bn);
  p.num_tiles = (int)(E * p.tilesM * p.tilesN);
  p.splits = ch.splits;
  const int64_t grid = std::min<int64_t>((int64_t)p.num_tiles * p.splits, cus);
  p.xcd_remap = grid % 8 == 0;
  GemmParams last = p;  // what adds the parts up
  if (p.splits > 1) {
    // a part's sums are a float32 C of their own
    last.sums = static_cast<float*>(workspace);
    last.ldw = (int)sums_ld(N);
    p.C = workspace;
    p.ldc = last.ldw;
    p.c_vec = N % 4 == 0;
    p.accumulate = false;
  }
  hipError_t e = more_launch(ch, true)(kDeepGroups, p, a_fmt, b_fmt, MXG_DT_F32, grid, s);
  if (e == hipSuccess && p.splits > 1) {
    const dim3 g((unsigned)std::min<int64_t>(cdiv(E * M * (last.ldw / 4), 256), 8LL * cus)), b(256);
    hipLaunchKernelGGL((block128_sum_kernel<0, kPlain>), g, b, 0, s, last, p.splits);
    e = hipGetLastError();
  }
  return e == hipSuccess ? MXG_OK : MXG_ERR_LAUNCH;
}

}  // extern "C"
