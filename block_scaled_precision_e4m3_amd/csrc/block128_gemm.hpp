// The product of two block-128 quantised operands on gfx950:
//   C[m,n] = sum_j SA[j,m] SB(j,n) sum_{k in block j} dec(A[m,k]) dec(B[n,k])
#pragma once

#include "dtypes.hpp"

namespace mxg {
namespace b128 {

struct GemmParams {
  const uint8_t* A;
  const uint8_t* B;
  const float* SA;   // (L, Kb, M)
  const float* SB;   // (L, Nb, Kb), or (L, Kb, N) when b_rows
  void* C;
  int64_t ldc;
  int M, N, K, L;
  int Kb, Nb;        // ceil(K / 128), ceil(N / 128)
  int tilesM, tilesN, num_tiles, xcd_remap;
  bool b_rows, accumulate;
};

// One wave per 32 x 32 outputs, operands straight from memory, codes widened to
// bfloat16: right for every size, the form the faster kernels are checked against.
template <int FA, int FB, int CT>
__global__ __launch_bounds__(64) void block128_plain_kernel(GemmParams p) {
  const int lane = threadIdx.x, r = lane & 31, h = lane >> 5;
  const int tiles = ((p.M + 31) / 32) * ((p.N + 31) / 32);
  const int l = blockIdx.x / tiles, rest = blockIdx.x % tiles;
  const int m0 = 32 * (rest % ((p.M + 31) / 32)), n0 = 32 * (rest / ((p.M + 31) / 32));
  const int m = min(m0 + r, p.M - 1), n = min(n0 + r, p.N - 1);
  const uint8_t* a = p.A + ((int64_t)l * p.M + m) * p.K;
  const uint8_t* b = p.B + ((int64_t)l * p.N + n) * p.K;
  v16f acc;
  for (int i = 0; i < 16; ++i) acc[i] = 0.f;
  for (int j = 0; j < p.Kb; ++j) {
    v16f part;
    for (int i = 0; i < 16; ++i) part[i] = 0.f;
    for (int k = 128 * j; k < min(p.K, 128 * j + 128); k += 16) {  // K % 16 == 0
      const uint2 ua = *reinterpret_cast<const uint2*>(a + k + 8 * h), ub = *reinterpret_cast<const uint2*>(b + k + 8 * h);
      part = __builtin_amdgcn_mfma_f32_32x32x16_bf16(cvt8<FB>(ub.x, ub.y, 1.f), cvt8<FA>(ua.x, ua.y, 1.f), part, 0, 0, 0);
    }
    // element e of this lane: n = n0 + 8 (e / 4) + 4 h + e % 4, m = m0 + r
    const float sa = p.SA[((int64_t)l * p.Kb + j) * p.M + m];
    for (int e = 0; e < 16; ++e) {
      const int nn = min(n0 + 8 * (e / 4) + 4 * h + e % 4, p.N - 1);
      const float sb = p.b_rows ? p.SB[((int64_t)l * p.Kb + j) * p.N + nn] : p.SB[((int64_t)l * p.Nb + nn / 128) * p.Kb + j];
      acc[e] += part[e] * (sa * sb);
    }
  }
  if (m0 + r >= p.M) return;
  elem_t<CT>* c = static_cast<elem_t<CT>*>(p.C) + ((int64_t)l * p.M + m0 + r) * p.ldc;
  for (int e = 0; e < 16; ++e) {
    const int nn = n0 + 8 * (e / 4) + 4 * h + e % 4;
    if (nn >= p.N) continue;
    if (CT == 0 && p.accumulate) acc[e] += (float)c[nn];
    c[nn] = (elem_t<CT>)acc[e];
  }
}

}  // namespace b128
}  // namespace mxg
