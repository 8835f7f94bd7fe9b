// Rotary positions and the per-head norm of queries and keys, forward and
// backward, for gfx950.
//
// One head row x (D features) of one token at position p:
//   rope:      y = R_p x
//   norm:      y = R_p (x r w),            r = 1 / sqrt(mean(x^2) + eps)
//   backward:  u = R_p^T g,  n = x r,      dw += u n,
//              dx = r (u w - n mean(u w n))
// R_p turns the pairs (a_i, b_i) of the rotary features [off, off + rot):
//   a' = a cos - b sin,  b' = b cos + a sin,   its transpose has -sin,
// with the pairs at (i, i + rot/2) or (2i, 2i + 1) of that part, separately on
// the way in and on the way out.  Everything is float32 between the load and
// the one rounding at the store.
#pragma once

#include "dtypes.hpp"

namespace mxg {
namespace heads {

constexpr int kWaves = 4;           // waves per workgroup
constexpr int kThreads = 64 * kWaves;
constexpr int kMaxD = 1024;
constexpr int kMaxParts = 1024;     // workgroups of the backward pass (rows of its workspace)

constexpr int kRope = 0, kNorm = 1, kBackward = 2;

// One (T, heads, D) tensor: element strides between tokens and heads.
struct Tensor {
  void* p;
  int64_t ts, hs;
};

struct Params {
  Tensor x[2];        // q and k (rope: x[0] only)
  Tensor y[2];        // outputs; backward: dq, dk
  Tensor g[2];        // backward: gradients of the outputs
  const void* w[2];   // weights
  float* parts;       // backward: (workgroups, 2, D) sums of u n
  const float* cos;
  const float* sin;
  const void* pos;
  int64_t T;
  int H[2];           // query and key heads
  int D, rot, off;
  int64_t table;      // rows of cos and sin
  float eps, inv_d;
  bool pos64, w_f32;
  bool halves_in, halves_out;  // where the pairs of x (and dx, u) and of y (and g) lie
  float sign;         // -1: the transposed rotation (rope only)
  // vector kernel: lanes per row, rows per wave, groups of rows of q and k per token, groups per wave
  int lpr, rpw, groups[2], gpw;
};

// The position of token t as a table row, -1 if it lies outside the table.
__device__ __forceinline__ int64_t table_row(const Params& p, int64_t t) {
  int64_t at = t;
  if (p.pos) at = p.pos64 ? static_cast<const int64_t*>(p.pos)[t] : (int64_t) static_cast<const int*>(p.pos)[t];
  return at >= 0 && at < p.table ? at : -1;
}

template <int DT>
__device__ __forceinline__ float weight(const Params& p, int which, int i) {
  return p.w_f32 ? static_cast<const float*>(p.w[which])[i] : (float)static_cast<const elem_t<DT>*>(p.w[which])[i];
}

// --- any strides, alignment and sizes ------------------------------------------
//
// A wave per row: the row (and the gradient) is staged in LDS as float32, so
// that a lane finds the other half of its pairs wherever they lie and Y may be
// X.  Lane l owns features l, l + 64, ....  Used where the vector kernel's
// 16-byte accesses do not fit.

// Where output feature f of the rotary part comes from: pair j, and which half.
struct Pair {
  int j;
  bool second;
};
__device__ __forceinline__ Pair pair_of(int f, int half, bool halves) {
  return halves ? (f < half ? Pair{f, false} : Pair{f - half, true}) : Pair{f >> 1, (f & 1) != 0};
}
__device__ __forceinline__ int feature_of(int j, bool second, int half, bool halves) {
  return halves ? j + (second ? half : 0) : 2 * j + (second ? 1 : 0);
}

// Feature i of the row in `v` after the rotation that reads pairs in one layout and leaves them in another.
__device__ __forceinline__ float rotated(const Params& p, const float* v, int i, int64_t row, bool in, bool out,
                                         float sign) {
  const int f = i - p.off, half = p.rot >> 1;
  if (f < 0 || f >= p.rot) return v[i];
  const Pair q = pair_of(f, half, out);
  const float c = row < 0 ? __builtin_nanf("") : p.cos[row * half + q.j];
  const float s = row < 0 ? __builtin_nanf("") : sign * p.sin[row * half + q.j];
  const float a = v[p.off + feature_of(q.j, false, half, in)], b = v[p.off + feature_of(q.j, true, half, in)];
  return q.second ? b * c + a * s : a * c - b * s;
}

__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
  for (int s = 1; s < 64; s <<= 1) v += __shfl_xor(v, s);
  return v;
}

template <int DT, int MODE>
__global__ __launch_bounds__(kThreads) void rows_kernel(Params p) {
  using E = elem_t<DT>;
  constexpr int kOwn = kMaxD / 64;
  __shared__ float lds[kWaves][MODE == kBackward ? 2 : 1][kMaxD];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int heads = p.H[0] + p.H[1];
  const int64_t rows = p.T * heads;
  float dw[2][kOwn];
  if constexpr (MODE == kBackward) {
#pragma unroll
    for (int j = 0; j < kOwn; ++j) dw[0][j] = dw[1][j] = 0.f;
  }
  for (int64_t r0 = (int64_t)blockIdx.x * kWaves; r0 < rows; r0 += (int64_t)gridDim.x * kWaves) {
    const int64_t r = r0 + wave;
    const bool live = r < rows;  // the same for every lane of a wave
    const int64_t t = live ? r / heads : 0;
    int h = live ? (int)(r - t * heads) : 0;
    const int which = h < p.H[0] ? 0 : 1;
    h -= which ? p.H[0] : 0;
    float* v = lds[wave][0];
    const int64_t at = live ? table_row(p, t) : 0;
    float ss = 0.f;
    if (live) {
      const E* x = static_cast<const E*>(p.x[which].p) + t * p.x[which].ts + h * p.x[which].hs;
      for (int i = lane; i < p.D; i += 64) {
        const float f = (float)x[i];
        v[i] = f;
        ss += f * f;
      }
      if constexpr (MODE == kBackward) {
        const E* g = static_cast<const E*>(p.g[which].p) + t * p.g[which].ts + h * p.g[which].hs;
        for (int i = lane; i < p.D; i += 64) lds[wave][1][i] = (float)g[i];
      }
    }
    float r_ = 1.f;
    if constexpr (MODE != kRope) {
      r_ = 1.f / sqrtf(wave_sum(ss) * p.inv_d + p.eps);
    }
    __syncthreads();
    if constexpr (MODE == kNorm) {
      if (live)
        for (int i = lane; i < p.D; i += 64) v[i] = v[i] * r_ * weight<DT>(p, which, i);
      __syncthreads();
    }
    E* y = static_cast<E*>(p.y[which].p) + t * p.y[which].ts + h * p.y[which].hs;
    if constexpr (MODE != kBackward) {
      if (live)
        for (int i = lane; i < p.D; i += 64) y[i] = (E)rotated(p, v, i, at, p.halves_in, p.halves_out, p.sign);
    } else {
      float u[kOwn], dot = 0.f;
#pragma unroll
      for (int j = 0; j < kOwn; ++j) {
        const int i = lane + 64 * j;
        u[j] = 0.f;
        if (live && i < p.D) {
          // the transposed rotation reads g where y's pairs lie and leaves them where x's lie
          u[j] = rotated(p, lds[wave][1], i, at, p.halves_out, p.halves_in, -1.f);
          const float n = v[i] * r_;
          if (which) dw[1][j] += u[j] * n; else dw[0][j] += u[j] * n;
          u[j] *= weight<DT>(p, which, i);
          dot += u[j] * n;
        }
      }
      dot = wave_sum(dot) * p.inv_d;
#pragma unroll
      for (int j = 0; j < kOwn; ++j) {
        const int i = lane + 64 * j;
        if (live && i < p.D) y[i] = (E)(r_ * (u[j] - v[i] * r_ * dot));
      }
    }
    __syncthreads();  // the staging is reused by the next row
  }
  if constexpr (MODE == kBackward) {
    // the workgroup's sums, waves added in order
#pragma unroll
    for (int s = 0; s < 2; ++s)
#pragma unroll
      for (int j = 0; j < kOwn; ++j)
        if (lane + 64 * j < p.D) lds[wave][s][lane + 64 * j] = dw[s][j];
    __syncthreads();
    for (int i = threadIdx.x; i < 2 * p.D; i += kThreads) {
      const int s = i >= p.D ? 1 : 0, f = i - s * p.D;
      float sum = 0.f;
      for (int w = 0; w < kWaves; ++w) sum += lds[w][s][f];
      p.parts[((int64_t)blockIdx.x * 2 + s) * p.D + f] = sum;
    }
  }
}

// dW: the sums of `parts` workgroups, 16 columns and 16 groups of rows to a
// workgroup, added in a fixed order.
__global__ __launch_bounds__(256) void weight_sum_kernel(const float* parts, float* dwq, float* dwk, int count, int D) {
  __shared__ float lds[16][17];
  const int c = threadIdx.x & 15, g = threadIdx.x >> 4;
  const int i = blockIdx.x * 16 + c;
  float sum = 0.f;
  if (i < 2 * D)
    for (int w = g; w < count; w += 16) sum += parts[(int64_t)w * 2 * D + i];
  lds[g][c] = sum;
  __syncthreads();
  if (g == 0 && i < 2 * D) {
    float s = 0.f;
    for (int w = 0; w < 16; ++w) s += lds[w][c];
    if (i < D) dwq[i] = s;
    else if (dwk) dwk[i - D] = s;
  }
}

}  // namespace heads
}  // namespace mxg
