// C-ABI entry points of the rotary positions and the per-head norm (include/mxgemm.h).
#include <hip/hip_runtime.h>

#include <algorithm>
#include <initializer_list>

#include "../../include/mxgemm.h"
#include "heads.hpp"
#include "host_checks.hpp"

namespace {

using namespace mxg::host;

using mxg::heads::Params;
using mxg::heads::Tensor;

// Sizes, layout and types that every entry shares (no HIP call).
int check(int64_t T, int64_t Hq, int64_t Hk, int64_t D, int64_t rot, int64_t off, int64_t table, bool positions,
          int layout, int dtype, int w_dtype, unsigned flags, unsigned known, const int64_t* strides, int tensors) {
  if (T < 0 || Hq < 0 || Hk < 0 || D < 1 || D > mxg::heads::kMaxD) return MXG_ERR_SHAPE;
  if (rot < 0 || rot % 2 != 0 || off < 0 || rot > D || off > D - rot || table < 0) return MXG_ERR_SHAPE;
  if (layout < MXG_ROPE_HALF || layout > MXG_ROPE_INTERLEAVED_TO_HALF) return MXG_ERR_FMT;
  if (dtype < MXG_DT_F32 || dtype > MXG_DT_F16) return MXG_ERR_FMT;
  if (w_dtype != dtype && w_dtype != MXG_DT_F32) return MXG_ERR_FMT;
  if (flags & ~known) return MXG_ERR_FLAGS;
  if (!fits_i32(T) || Hq > (1 << 20) || Hk > (1 << 20) - Hq || !fits_i32(table)) return MXG_ERR_SHAPE;
  if (!positions && rot > 0 && T > table) return MXG_ERR_SHAPE;
  // a wave takes a head of a token at least
  if (T > 0 && Hq + Hk > (1LL << 36) / T) return MXG_ERR_SHAPE;
  if (!strides) return MXG_ERR_NULL;
  for (int i = 0; i < tensors; ++i) {
    // byte offsets stay below 2^62
    const int64_t ts = strides[2 * i], hs = strides[2 * i + 1];
    if (ts < 0 || hs < 0 || ts > (1LL << 40) || hs > (1LL << 36)) return MXG_ERR_SHAPE;
    if (T > 0 && ts > 0 && T > (1LL << 59) / ts) return MXG_ERR_SHAPE;
  }
  return MXG_OK;
}

// Whether rows of an output surely lie on each other: neighbouring tokens or heads nearer than a row, or the same distance
// for both.
bool overlap(int64_t T, int64_t H, int64_t D, const int64_t* s) {
  return T > 0 && H > 0 && ((T > 1 && s[0] < D) || (H > 1 && s[1] < D) || (T > 1 && H > 1 && s[0] == s[1]));
}

void layouts(Params* p, int layout, bool transpose) {
  const bool in = layout == MXG_ROPE_HALF, out = layout != MXG_ROPE_INTERLEAVED;
  p->halves_in = transpose ? out : in;
  p->halves_out = transpose ? in : out;
  p->sign = transpose ? -1.f : 1.f;
}

template <int MODE>
void launch_rows(const Params& p, int dtype, int64_t grid, hipStream_t s) {
  const dim3 g((unsigned)grid), b(mxg::heads::kThreads);
  if (dtype == MXG_DT_F32) hipLaunchKernelGGL((mxg::heads::rows_kernel<0, MODE>), g, b, 0, s, p);
  else if (dtype == MXG_DT_BF16) hipLaunchKernelGGL((mxg::heads::rows_kernel<1, MODE>), g, b, 0, s, p);
  else hipLaunchKernelGGL((mxg::heads::rows_kernel<2, MODE>), g, b, 0, s, p);
}

// Workgroups of the backward pass, each with a row of its workspace.
int64_t backward_parts(int64_t T) {
  return std::max<int64_t>(2, std::min<int64_t>(cdiv(T, mxg::heads::kWaves), mxg::heads::kMaxParts));
}

// Those of the vector kernel, of which there are no more.
int64_t vector_parts(int64_t T) { return std::min<int64_t>(backward_parts(T), mxg::heads::kBackParts); }

// Whether the head, its rotary part and what lies before it are whole chunks of 8 features, as the vector kernels want
// them, in pairs of chunks.
bool whole_chunks(const Params& p) { return p.D % 16 == 0 && p.rot % 16 == 0 && p.off % 8 == 0; }

template <int DT, int MODE, bool IN, bool OUT>
void launch_heads(Params& p, int64_t grid, hipStream_t s) {
  if constexpr (MODE == mxg::heads::kBackward) {
    hipLaunchKernelGGL((mxg::heads::heads_backward_kernel<DT, IN, OUT>), dim3((unsigned)grid), dim3(64 * mxg::heads::kBackWaves), 0, s, p);
  } else {
    launch_runs(grid, [&](int64_t first, unsigned count) {
      p.first = first * mxg::heads::kWaves;
      hipLaunchKernelGGL((mxg::heads::heads_kernel<DT, MODE, IN, OUT>), dim3(count), dim3(mxg::heads::kThreads), 0, s, p);
    });
  }
}

template <int DT, int MODE>
void launch_heads(Params& p, int64_t grid, hipStream_t s) {
  if (p.halves_in && p.halves_out) launch_heads<DT, MODE, true, true>(p, grid, s);
  else if (p.halves_out) launch_heads<DT, MODE, false, true>(p, grid, s);
  else if (!p.halves_in) launch_heads<DT, MODE, false, false>(p, grid, s);
  else if constexpr (MODE == mxg::heads::kRope) launch_heads<DT, MODE, true, false>(p, grid, s);  // a transposed map only
}

// Launches the pass; returns its workgroups.
template <int MODE>
int launch(Params& p, int dtype, int cus, hipStream_t s) {
  int64_t grid;
  if (whole_chunks(p)) {
    p.lpr = 1;
    while (16 * p.lpr < p.D) p.lpr *= 2;
    p.rpw = 64 / p.lpr;
    for (int k = 0; k < 2; ++k) p.groups[k] = (int)cdiv(p.H[k], p.rpw);
    const int64_t groups = p.groups[0] + p.groups[1];
    // Groups of heads to a wave, which share the token's angles and weights: 2 (rope, 8192 tokens of 128 heads of 192:
    // 1 174 us, 2 146 us, 8 159 us) or 8 (norm, 8192 tokens of 32 + 8 heads of 128: 1 56 us, 2 50 us, 5 and 8 41 us);
    // fewer while that leaves less than 16 waves per compute unit.
    p.gpw = (int)std::max<int64_t>(1, std::min<int64_t>({groups, MODE == mxg::heads::kRope ? 2 : 8, p.T * groups / (16LL * cus)}));
    if (MODE == mxg::heads::kBackward) {
      // workgroups in proportion to the groups of queries and keys, at least one of each that there is
      const int64_t parts = vector_parts(p.T);
      const int64_t q = p.groups[1] == 0 ? parts : std::min(parts - 1, std::max<int64_t>(1, cdiv(parts * p.groups[0], groups)));
      p.parts_q = p.groups[0] == 0 ? 0 : (int)q;
    }
    grid = MODE == mxg::heads::kBackward ? vector_parts(p.T) : cdiv(p.T * cdiv(groups, p.gpw), mxg::heads::kWaves);
    if (dtype == MXG_DT_F32) launch_heads<0, MODE>(p, grid, s);
    else if (dtype == MXG_DT_BF16) launch_heads<1, MODE>(p, grid, s);
    else launch_heads<2, MODE>(p, grid, s);
  } else {
    const int64_t rows = p.T * (p.H[0] + p.H[1]);
    grid = std::min<int64_t>(cdiv(rows, mxg::heads::kWaves), 64LL * cus);
    if (MODE == mxg::heads::kBackward) grid = std::min(grid, backward_parts(p.T));
    launch_rows<MODE>(p, dtype, grid, s);
  }
  return (int)grid;
}

}  // namespace

extern "C" {

int mxgemm_rope(const void* X, void* Y, const float* cos, const float* sin, const void* positions,
                const int64_t* strides, int64_t T, int64_t H, int64_t D, int64_t rot, int64_t rot_offset,
                int64_t table_rows, int layout, int dtype, unsigned flags, void* stream) {
  const bool trusted = take_trust(&flags);
  int st = check(T, H, 0, D, rot, rot_offset, table_rows, positions != nullptr, layout, dtype, dtype, flags,
                 MXG_ROPE_TRANSPOSE | MXG_ROPE_POS64, strides, 2);
  if (st != MXG_OK) return st;
  if (overlap(T, H, D, strides + 2)) return MXG_ERR_SHAPE;
  if (T == 0 || H == 0) return MXG_OK;
  if (!X || !Y || (rot > 0 && (!cos || !sin))) return MXG_ERR_NULL;
  const size_t e = mxg::elem_bytes(dtype), pe = (flags & MXG_ROPE_POS64) ? 8 : 4;
  if (!aligned_to(X, e) || !aligned_to(Y, e) || !aligned_to(cos, 4) || !aligned_to(sin, 4) ||
      !aligned_to(positions, pe))
    return MXG_ERR_ALIGN;
  int dev = 0, cus = 0;
  st = device_check(&dev, &cus);
  if (st != MXG_OK) return st;
  if (!trusted && (!on_device(X, dev) || !on_device(Y, dev) || (rot > 0 && (!on_device(cos, dev) || !on_device(sin, dev))) ||
      (positions && !on_device(positions, dev))))
    return MXG_ERR_DEVICE;
  Params p{};
  p.x[0] = {const_cast<void*>(X), strides[0], strides[1]};
  p.y[0] = {Y, strides[2], strides[3]};
  p.cos = cos;
  p.sin = sin;
  p.pos = positions;
  p.T = T;
  p.H[0] = (int)H;
  p.D = (int)D;
  p.rot = (int)rot;
  p.off = (int)rot_offset;
  p.table = table_rows;
  p.pos64 = (flags & MXG_ROPE_POS64) != 0;
  layouts(&p, layout, (flags & MXG_ROPE_TRANSPOSE) != 0);
  launch<mxg::heads::kRope>(p, dtype, cus, (hipStream_t)stream);
  return hipGetLastError() == hipSuccess ? MXG_OK : MXG_ERR_LAUNCH;
}

int mxgemm_qk_norm_rope(const void* Q, const void* K, void* YQ, void* YK, const void* WQ, const void* WK,
                        const float* cos, const float* sin, const void* positions, const int64_t* strides, int64_t T,
                        int64_t Hq, int64_t Hk, int64_t D, int64_t rot, int64_t rot_offset, int64_t table_rows,
                        float eps, int layout, int dtype, int w_dtype, unsigned flags, void* stream) {
  const bool trusted = take_trust(&flags);
  int st = check(T, Hq, Hk, D, rot, rot_offset, table_rows, positions != nullptr, layout, dtype, w_dtype, flags,
                 MXG_ROPE_POS64, strides, 4);
  if (st != MXG_OK) return st;
  if (overlap(T, Hq, D, strides + 4) || overlap(T, Hk, D, strides + 6)) return MXG_ERR_SHAPE;
  if (T == 0 || Hq + Hk == 0) return MXG_OK;
  if ((Hq > 0 && (!Q || !YQ || !WQ)) || (Hk > 0 && (!K || !YK || !WK)) || (rot > 0 && (!cos || !sin)))
    return MXG_ERR_NULL;
  const size_t e = mxg::elem_bytes(dtype), we = mxg::elem_bytes(w_dtype), pe = (flags & MXG_ROPE_POS64) ? 8 : 4;
  for (const void* q : {Q, K, (const void*)YQ, (const void*)YK})
    if (!aligned_to(q, e)) return MXG_ERR_ALIGN;
  if (!aligned_to(WQ, we) || !aligned_to(WK, we) || !aligned_to(cos, 4) || !aligned_to(sin, 4) ||
      !aligned_to(positions, pe))
    return MXG_ERR_ALIGN;
  int dev = 0, cus = 0;
  st = device_check(&dev, &cus);
  if (st != MXG_OK) return st;
  if (!trusted) {
    if (Hq > 0)
      for (const void* q : {Q, (const void*)YQ, WQ})
        if (!on_device(q, dev)) return MXG_ERR_DEVICE;
    if (Hk > 0)
      for (const void* q : {K, (const void*)YK, WK})
        if (!on_device(q, dev)) return MXG_ERR_DEVICE;
    if ((rot > 0 && (!on_device(cos, dev) || !on_device(sin, dev))) || (positions && !on_device(positions, dev)))
      return MXG_ERR_DEVICE;
  }
  Params p{};
  p.x[0] = {const_cast<void*>(Q), strides[0], strides[1]};
  p.x[1] = {const_cast<void*>(K), strides[2], strides[3]};
  p.y[0] = {YQ, strides[4], strides[5]};
  p.y[1] = {YK, strides[6], strides[7]};
  p.w[0] = WQ;
  p.w[1] = WK;
  p.cos = cos;
  p.sin = sin;
  p.pos = positions;
  p.T = T;
  p.H[0] = (int)Hq;
  p.H[1] = (int)Hk;
  p.D = (int)D;
  p.rot = (int)rot;
  p.off = (int)rot_offset;
  p.table = table_rows;
  p.eps = eps;
  p.inv_d = 1.f / (float)D;
  p.pos64 = (flags & MXG_ROPE_POS64) != 0;
  p.w_f32 = w_dtype == MXG_DT_F32;
  layouts(&p, layout, false);
  launch<mxg::heads::kNorm>(p, dtype, cus, (hipStream_t)stream);
  return hipGetLastError() == hipSuccess ? MXG_OK : MXG_ERR_LAUNCH;
}

size_t mxgemm_qk_norm_rope_backward_workspace_bytes(int64_t T, int64_t D) {
  if (T < 0 || D < 1) return 0;
  return (size_t)(backward_parts(T) * 2 * D * 4);
}

int mxgemm_qk_norm_rope_backward(const void* GQ, const void* GK, const void* Q, const void* K, void* DQ, void* DK,
                                 float* DWQ, float* DWK, const void* WQ, const void* WK, const float* cos,
                                 const float* sin, const void* positions, const int64_t* strides, int64_t T,
                                 int64_t Hq, int64_t Hk, int64_t D, int64_t rot, int64_t rot_offset,
                                 int64_t table_rows, float eps, int layout, int dtype, int w_dtype, unsigned flags,
                                 void* workspace, size_t workspace_bytes, void* stream) {
  const bool trusted = take_trust(&flags);
  int st = check(T, Hq, Hk, D, rot, rot_offset, table_rows, positions != nullptr, layout, dtype, w_dtype, flags,
                 MXG_ROPE_POS64, strides, 6);
  if (st != MXG_OK) return st;
  if (overlap(T, Hq, D, strides + 8) || overlap(T, Hk, D, strides + 10)) return MXG_ERR_SHAPE;
  const bool empty = T == 0 || Hq + Hk == 0;
  if (!DWQ || (Hk > 0 && !DWK) || !workspace) return MXG_ERR_NULL;
  if (!empty && ((Hq > 0 && (!GQ || !Q || !DQ || !WQ)) || (Hk > 0 && (!GK || !K || !DK || !WK)) ||
                 (rot > 0 && (!cos || !sin))))
    return MXG_ERR_NULL;
  if (workspace_bytes < mxgemm_qk_norm_rope_backward_workspace_bytes(T, D)) return MXG_ERR_SHAPE;
  const size_t e = mxg::elem_bytes(dtype), we = mxg::elem_bytes(w_dtype), pe = (flags & MXG_ROPE_POS64) ? 8 : 4;
  for (const void* q : {GQ, GK, Q, K, (const void*)DQ, (const void*)DK})
    if (!aligned_to(q, e)) return MXG_ERR_ALIGN;
  if (!aligned_to(WQ, we) || !aligned_to(WK, we) || !aligned_to(cos, 4) || !aligned_to(sin, 4) ||
      !aligned_to(positions, pe) || !aligned_to(DWQ, 4) || !aligned_to(DWK, 4) || !aligned16(workspace))
    return MXG_ERR_ALIGN;
  int dev = 0, cus = 0;
  st = device_check(&dev, &cus);
  if (st != MXG_OK) return st;
  if (!trusted && (!on_device(DWQ, dev) || (DWK && !on_device(DWK, dev)) || !on_device(workspace, dev)))
    return MXG_ERR_DEVICE;
  if (!empty && !trusted) {
    if (Hq > 0)
      for (const void* q : {GQ, Q, (const void*)DQ, WQ})
        if (!on_device(q, dev)) return MXG_ERR_DEVICE;
    if (Hk > 0)
      for (const void* q : {GK, K, (const void*)DK, WK})
        if (!on_device(q, dev)) return MXG_ERR_DEVICE;
    if ((rot > 0 && (!on_device(cos, dev) || !on_device(sin, dev))) || (positions && !on_device(positions, dev)))
      return MXG_ERR_DEVICE;
  }
  Params p{};
  p.g[0] = {const_cast<void*>(GQ), strides[0], strides[1]};
  p.g[1] = {const_cast<void*>(GK), strides[2], strides[3]};
  p.x[0] = {const_cast<void*>(Q), strides[4], strides[5]};
  p.x[1] = {const_cast<void*>(K), strides[6], strides[7]};
  p.y[0] = {DQ, strides[8], strides[9]};
  p.y[1] = {DK, strides[10], strides[11]};
  p.w[0] = WQ;
  p.w[1] = WK;
  p.parts = static_cast<float*>(workspace);
  p.cos = cos;
  p.sin = sin;
  p.pos = positions;
  p.T = T;
  p.H[0] = (int)Hq;
  p.H[1] = (int)Hk;
  p.D = (int)D;
  p.rot = (int)rot;
  p.off = (int)rot_offset;
  p.table = table_rows;
  p.eps = eps;
  p.inv_d = 1.f / (float)D;
  p.pos64 = (flags & MXG_ROPE_POS64) != 0;
  p.w_f32 = w_dtype == MXG_DT_F32;
  layouts(&p, layout, false);
  int parts = 0;  // none: the sums are zero
  if (!empty) {
    parts = launch<mxg::heads::kBackward>(p, dtype, cus, (hipStream_t)stream);
    if (hipGetLastError() != hipSuccess) return MXG_ERR_LAUNCH;
  }
  // the wave-per-row kernel leaves queries' and keys' sums side by side, the vector kernel in rows of their own
  const bool rows = p.lpr == 0;
  const int64_t row = rows ? 2 * D : D;
  const int parts_q = rows ? parts : p.parts_q, parts_k = rows ? parts : parts - p.parts_q;
  const float* sums_k = rows ? p.parts + D : p.parts + p.parts_q * row;
  hipLaunchKernelGGL(mxg::heads::weight_sum_kernel, dim3((unsigned)cdiv(D, 16), DWK ? 2 : 1), dim3(1024), 0,
                     (hipStream_t)stream, p.parts, parts_q, sums_k, parts_k, row, DWQ, DWK, (int)D);
  return hipGetLastError() == hipSuccess ? MXG_OK : MXG_ERR_LAUNCH;
}

}  // extern "C"
