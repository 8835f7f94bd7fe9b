// Gradients through y = act(z) gate + residual, z = product + bias, on gfx950:
//   dz = dy gate act'(z),  dgate = dy act(z),  dbias = sum over rows of dz
// in float32, rounded once; the sum is over dz before its rounding, in an order that the sizes alone fix.
//
// Memory is the bound, so every tensor is touched once, in 16-byte chunks: a wave takes 8 columns to a lane of one row
// (of several rows where they are short), a workgroup's waves the rows of one part in turn.  Each lane adds up its
// columns' dz over its rows, the lanes of a column meet in LDS, and a second kernel adds up the parts; a single part
// needs none.
//
// 8192 x 8192 bfloat16, silu with gate and dbias: 137 us, 4.9 TB/s (a copy moves 5.1); without dbias 132.  1000 x 4096 with
// dbias 9.3 us, of which the second kernel is 4; 40 x 2048 float32 with dbias, one part: 4.3 us.
#pragma once

#include "ends.hpp"

namespace mxg {
namespace activation {

constexpr int kWaves = 8;
constexpr int kThreads = 64 * kWaves;
constexpr int kAhead = 2;   // rows of a lane whose loads are under way together
constexpr int kMaxParts = 512;

struct Params {
  const void *dy, *z, *gate;
  void *dz, *dgate;
  float* sums;  // (parts, N), or dbias where there is one part; null: not wanted
  int64_t ld_dy, ld_z, ld_gate, ld_dz, ld_dgate;
  int64_t M, rows;  // rows of a part
  int N, act;
  int lanes;    // lanes to a row: a power of two
  int strips;   // of 8 `lanes` columns
};

template <int DT, bool GATE>
__global__ __launch_bounds__(kThreads) void activation_backward_kernel(Params p) {
  using E = elem_t<DT>;
  __shared__ float lds[kThreads][9];  // a lane's 8 sums; 9 words apart, as the lanes that add them up read across
  const int tid = threadIdx.x, c = tid & (p.lanes - 1), sub = tid / p.lanes, subs = kThreads / p.lanes;
  const int strip = blockIdx.x % p.strips, part = blockIdx.x / p.strips;
  const int n = 8 * (strip * p.lanes + c), valid = p.N - n;
  const int64_t first = part * p.rows + sub, end = min(p.M, (part + 1) * p.rows);
  const E *dy = static_cast<const E*>(p.dy) + n, *z = static_cast<const E*>(p.z) + n, *gate = static_cast<const E*>(p.gate) + n;
  E *dz = static_cast<E*>(p.dz) + n, *dgate = static_cast<E*>(p.dgate) + n;
  v8f sum;
#pragma unroll
  for (int i = 0; i < 8; ++i) sum[i] = 0.f;
  ends::with_slope<DT != 0>(p.act, [&](auto slope) {
    for (int64_t m = first; m < end; m += kAhead * subs) {
      Raw8<DT> a[kAhead], b[kAhead], g[kAhead];
#pragma unroll
      for (int j = 0; j < kAhead; ++j) {
        const int64_t row = m + (int64_t)j * subs;
        const int there = row < end ? valid : 0;
        a[j] = load_chunk<DT>(dy + row * p.ld_dy, there);
        b[j] = load_chunk<DT>(z + row * p.ld_z, there);
        if constexpr (GATE) g[j] = load_chunk<DT>(gate + row * p.ld_gate, there);
      }
#pragma unroll
      for (int j = 0; j < kAhead; ++j) {
        const int64_t row = m + (int64_t)j * subs;
        if (row >= end || valid <= 0) continue;
        const v8f d = widen8<DT>(a[j]), x = widen8<DT>(b[j]);
        v8f w, dg, out;
        if constexpr (GATE) w = widen8<DT>(g[j]);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const ends::Slope s = slope(x[i]);
          if constexpr (GATE) {
            dg[i] = d[i] * s.value;
            out[i] = d[i] * w[i] * s.slope;
          } else {
            out[i] = d[i] * s.slope;
          }
          sum[i] += out[i];
        }
        store_chunk<DT>(dz + row * p.ld_dz, out, valid);
        if constexpr (GATE) store_chunk<DT>(dgate + row * p.ld_dgate, dg, valid);
      }
    }
  });
  if (!p.sums) return;
#pragma unroll
  for (int i = 0; i < 8; ++i) lds[tid][i] = sum[i];
  __syncthreads();
  // column 8 c + i is in the rows c, c + lanes, ... of lds
  for (int j = tid; j < 8 * p.lanes; j += kThreads) {
    const int col = 8 * strip * p.lanes + j;
    if (col >= p.N) break;
    float total = 0.f;
    for (int s = 0; s < subs; ++s) total += lds[s * p.lanes + (j >> 3)][j & 7];
    p.sums[(int64_t)part * p.N + col] = total;
  }
}

// dbias from the parts' sums: 64 columns and 16 shares of the parts to a workgroup.
__global__ __launch_bounds__(1024) void bias_sum_kernel(const float* sums, int parts, float* dbias, int N) {
  __shared__ float lds[16][64];
  const int c = threadIdx.x & 63, g = threadIdx.x >> 6, n = blockIdx.x * 64 + c;
  float sum = 0.f;
  if (n < N) {
#pragma unroll 8
    for (int i = g; i < parts; i += 16) sum += sums[(int64_t)i * N + n];
  }
  lds[g][c] = sum;
  __syncthreads();
  if (g == 0 && n < N) {
    float total = 0.f;
#pragma unroll
    for (int i = 0; i < 16; ++i) total += lds[i][c];
    dbias[n] = total;
  }
}

__global__ __launch_bounds__(256) void bias_zero_kernel(float* dbias, int N) {
  const int n = blockIdx.x * 256 + threadIdx.x;
  if (n < N) dbias[n] = 0.f;
}

}  // namespace activation
}  // namespace mxg
