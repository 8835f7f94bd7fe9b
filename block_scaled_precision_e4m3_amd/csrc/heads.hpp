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
// Workgroups of the backward pass, each with a row of its workspace, at most.  The vector kernel's are of 16 waves, one
// to a compute unit: as many waves as four workgroups of four, and fewer sums to add up at the end (workgroups x waves,
// 4001 tokens, 32 + 8 heads of 128, both kernels: 512 x 4 38.9 us, 1024 x 4 35.6, 512 x 8 35.4, 256 x 16 34.6, 512 x 16
// 41.4).
constexpr int kMaxParts = 512, kBackParts = 256;
constexpr int kBackWaves = 16;

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
  float* parts;       // backward: sums of u n, a row of D (2 D in the wave-per-row kernel) per workgroup
  int parts_q;        // backward, vector kernel: workgroups that work on queries
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
  int64_t first;      // the launch's first work item
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

// --- any sizes -------------------------------------------------------------------
//
// A wave per row: the row (and the gradient) is staged in LDS as float32, so
// that a lane finds the other half of its pairs wherever they lie and Y may be
// X.  Lane l owns features l, l + 64, ....  Used where the vector kernel's
// chunks do not fit.

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

// --- 16-byte accesses ------------------------------------------------------------
//
// A head is D / 8 chunks of 8 features; a lane owns two of them, so that it has
// both members of its 8 pairs and no lane needs another's features: the chunks
// at off + 8p and off + rot/2 + 8p where the pairs lie in halves, 16
// consecutive features from off + 16p where they are interleaved (the first
// members are then the even ones), and any two of the remaining chunks for
// features that are only copied or normed.  D / 16 lanes, rounded up to a power
// of two (lpr), share a head; a wave works on 64 / lpr heads of one token at a
// time, and keeps that token's cos and sin (and the weights) in registers over
// the heads it does.  The bound is memory: every feature is read once and
// written once, cos and sin once per wave and token (rope, 8192 tokens of 128
// heads of 192, 64 of them rotary: 140 us, 5.8 TB/s; norm and rope, 8192 tokens
// of 32 + 8 heads of 128: 38 us, 4.5 TB/s).  Rows and heads may lie at
// any stride: chunks that are not aligned to 16 bytes are accessed all the same
// (1024 tokens of 32 + 8 heads of 128, rows one element apart from aligned ones,
// backward: 130 us in the wave-per-row kernel, 14.5 us here).

// A lane's share of a head, as feature offsets: first and second chunk as read and as written.
struct Lane {
  int in0, in1, out0, out1;
  bool rot;          // its pairs turn
  int pair;          // index of its first pair
};
__device__ __forceinline__ Lane lane_of(const Params& p, int q, bool halves_in, bool halves_out) {
  Lane l;
  const int half = p.rot >> 1;
  l.rot = q < (p.rot >> 4);
  l.pair = 8 * q;
  if (l.rot) {
    l.in0 = p.off + (halves_in ? 8 * q : 16 * q);
    l.in1 = l.in0 + (halves_in ? half : 8);
    l.out0 = p.off + (halves_out ? 8 * q : 16 * q);
    l.out1 = l.out0 + (halves_out ? half : 8);
  } else {
    // the chunks outside the rotary part, two at a time
    const int c = 16 * (q - (p.rot >> 4));
    l.in0 = l.out0 = c < p.off ? c : c + p.rot;
    l.in1 = l.out1 = c + 8 < p.off ? c + 8 : c + 8 + p.rot;
  }
  return l;
}

struct Two {
  v8f a, b;
};
// Two chunks as first and second members of 8 pairs, and back.
template <bool HALVES>
__device__ __forceinline__ Two split(const v8f& x, const v8f& y) {
  if constexpr (HALVES) return {x, y};
  return {__builtin_shufflevector(x, y, 0, 2, 4, 6, 8, 10, 12, 14), __builtin_shufflevector(x, y, 1, 3, 5, 7, 9, 11, 13, 15)};
}
template <bool HALVES>
__device__ __forceinline__ Two join(const Two& t) {
  if constexpr (HALVES) return t;
  return {__builtin_shufflevector(t.a, t.b, 0, 8, 1, 9, 2, 10, 3, 11), __builtin_shufflevector(t.a, t.b, 4, 12, 5, 13, 6, 14, 7, 15)};
}
// The rotation between layouts; a lane whose pairs do not turn has its chunks back in the order they came.
template <bool IN, bool OUT>
__device__ __forceinline__ Two turn(const Two& t, const v8f& c, const v8f& s, bool rot) {
  Two r;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float a = t.a[i] * c[i] - t.b[i] * s[i], b = t.b[i] * c[i] + t.a[i] * s[i];
    r.a[i] = rot ? a : t.a[i];
    r.b[i] = rot ? b : t.b[i];
  }
  if constexpr (IN == OUT) return join<OUT>(r);
  const Two x = join<OUT>(r), y = join<IN>(r);
  Two z;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    z.a[i] = rot ? x.a[i] : y.a[i];
    z.b[i] = rot ? x.b[i] : y.b[i];
  }
  return z;
}

struct Angles {
  v8f c, s;
};
__device__ __forceinline__ Angles angles_of(const Params& p, int64_t t, const Lane& l, float sign) {
  Angles a;
#pragma unroll
  for (int i = 0; i < 8; ++i) a.c[i] = a.s[i] = 0.f;
  if (l.rot) {
    const int64_t row = table_row(p, t);
    if (row >= 0) {
      const int64_t at = row * (p.rot >> 1) + l.pair;
      a.c = widen8<0>(load8<0>(p.cos + at));
      a.s = widen8<0>(load8<0>(p.sin + at)) * sign;
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) a.c[i] = a.s[i] = __builtin_nanf("");
    }
  }
  return a;
}

// Sum over the lanes of a head, the same bits in each: pairs, quads, then the mirrored half and row (whose quads hold
// equal sums) through the lane crossbar of the VALU, wider exchanges through LDS.
template <int CTRL>
__device__ __forceinline__ float add_across(float v) {
  return v + __builtin_bit_cast(float, __builtin_amdgcn_mov_dpp(__builtin_bit_cast(int, v), CTRL, 0xF, 0xF, true));
}
__device__ __forceinline__ float head_sum(float v, int lpr) {
  if (lpr > 1) v = add_across<0xB1>(v);    // quad_perm 1 0 3 2
  if (lpr > 2) v = add_across<0x4E>(v);    // quad_perm 2 3 0 1
  if (lpr > 4) v = add_across<0x141>(v);   // row_half_mirror
  if (lpr > 8) v = add_across<0x140>(v);   // row_mirror
  if (lpr > 16) v += __shfl_xor(v, 16);
  if (lpr > 32) v += __shfl_xor(v, 32);
  return v;
}
template <int DT>
__device__ __forceinline__ v8f weights8(const Params& p, int which, int i) {
  if (p.w_f32) return widen8<0>(load8<0>(static_cast<const float*>(p.w[which]) + i));
  return widen8<DT>(load8<DT>(static_cast<const elem_t<DT>*>(p.w[which]) + i));
}

// IN, OUT: the pairs lie in halves on the way in, and on the way out.
template <int DT, int MODE, bool IN, bool OUT>
__global__ __launch_bounds__(kThreads) void heads_kernel(Params p) {
  using E = elem_t<DT>;
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  const int all = p.groups[0] + p.groups[1], parts = (all + p.gpw - 1) / p.gpw;
  const int64_t item = p.first + (int64_t)blockIdx.x * kWaves + wave;
  const int64_t t = item / parts;
  if (t >= p.T) return;
  const int first = (int)(item - t * parts) * p.gpw, last = min(first + p.gpw, all);
  const int q = lane & (p.lpr - 1), sub = lane / p.lpr;
  const bool mine = 16 * q < p.D;
  const Lane l = lane_of(p, q, IN, OUT);
  struct Group {
    Raw8<DT> x[2];
    E* to;       // where the head goes, null: none
  };
  auto load = [&](Group& v, int g) {
    const int k = g < p.groups[0] ? 0 : 1;
    const int h = (k ? g - p.groups[0] : g) * p.rpw + sub;
    v.to = nullptr;
    if (mine && g < last && h < p.H[k]) {
      v.to = static_cast<E*>(p.y[k].p) + t * p.y[k].ts + h * p.y[k].hs;
      const E* at = static_cast<const E*>(p.x[k].p) + t * p.x[k].ts + h * p.x[k].hs;
      v.x[0] = load8<DT>(at + l.in0);
      v.x[1] = load8<DT>(at + l.in1);
    }
  };
  // the first heads are asked for before the position is waited for; the next ones before these are worked on
  constexpr int U = 2;
  Group next[U];
#pragma unroll
  for (int u = 0; u < U; ++u) load(next[u], first + u);
  const Angles ang = angles_of(p, t, l, p.sign);
  Two w[2];
  if constexpr (MODE == kNorm) {
#pragma unroll
    for (int k = 0; k < 2; ++k)
      if (mine && p.groups[k] > 0) w[k] = split<IN>(weights8<DT>(p, k, l.in0), weights8<DT>(p, k, l.in1));
  }
  for (int g0 = first; g0 < last; g0 += U) {
    Group now[U];
#pragma unroll
    for (int u = 0; u < U; ++u) now[u] = next[u];
    if (g0 + U < last) {
#pragma unroll
      for (int u = 0; u < U; ++u) load(next[u], g0 + U + u);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (g0 + u >= last) break;
      const bool live = now[u].to != nullptr;
      Two v = split<IN>(widen8<DT>(now[u].x[0]), widen8<DT>(now[u].x[1]));
      if constexpr (MODE == kNorm) {
        const int k = g0 + u < p.groups[0] ? 0 : 1;
        float ss = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) ss += v.a[i] * v.a[i] + v.b[i] * v.b[i];
        ss = head_sum(live ? ss : 0.f, p.lpr);
        const float r = rsqrtf(ss * p.inv_d + p.eps);
        v.a = v.a * r * (k ? w[1].a : w[0].a);
        v.b = v.b * r * (k ? w[1].b : w[0].b);
      }
      const Two y = turn<IN, OUT>(v, ang.c, ang.s, l.rot);
      if (live) {
        store8<DT>(now[u].to + l.out0, y.a);
        store8<DT>(now[u].to + l.out1, y.b);
      }
    }
  }
}

// Backward.  A workgroup works on the queries only or on the keys only (the first p.parts_q on queries), so that a
// lane holds one weight and one weight gradient for each of its features, to the end.  A work item is one token and
// one group of its heads.  More waves hide the loads better than more loads per wave; asking for the next item's
// position ahead changes nothing.  4001 tokens of 32 + 8 heads of 128: 30.6 us, 4.05 TB/s, besides 3.3 for the sums;
// the bound is memory, its latency more than its rate, at five items to a wave.
template <int DT, bool IN, bool OUT>
__global__ __launch_bounds__(64 * kBackWaves) void heads_backward_kernel(Params p) {
  using E = elem_t<DT>;
  __shared__ float lds[kBackWaves][kMaxD];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  const int k = (int)blockIdx.x < p.parts_q ? 0 : 1;
  const int wg = k ? (int)blockIdx.x - p.parts_q : (int)blockIdx.x, wgs = k ? (int)gridDim.x - p.parts_q : p.parts_q;
  const Tensor X = p.x[k], G = p.g[k], Y = p.y[k];
  const int H = p.H[k];
  const int q = lane & (p.lpr - 1), sub = lane / p.lpr;
  const bool mine = 16 * q < p.D;
  const Lane l = lane_of(p, q, IN, OUT);
  const int per = p.groups[k];  // items per token
  const int64_t items = p.T * per, step = (int64_t)wgs * kBackWaves;
  Two w, dw;
#pragma unroll
  for (int i = 0; i < 8; ++i) dw.a[i] = dw.b[i] = w.a[i] = w.b[i] = 0.f;
  if (mine) w = split<IN>(weights8<DT>(p, k, l.in0), weights8<DT>(p, k, l.in1));
  for (int64_t it = (int64_t)wg * kBackWaves + wave; it < items; it += step) {
    const int64_t t = it / per;
    const int h = (int)(it - t * per) * p.rpw + sub;
    const bool live = mine && h < H;
    Raw8<DT> x[2], g[2];
    if (live) {
      const E* xa = static_cast<const E*>(X.p) + t * X.ts + h * X.hs;
      const E* ga = static_cast<const E*>(G.p) + t * G.ts + h * G.hs;
      x[0] = load8<DT>(xa + l.in0);
      x[1] = load8<DT>(xa + l.in1);
      g[0] = load8<DT>(ga + l.out0);
      g[1] = load8<DT>(ga + l.out1);
    }
    const Angles ang = angles_of(p, t, l, -1.f);
    const Two v = split<IN>(widen8<DT>(x[0]), widen8<DT>(x[1]));
    // the transposed rotation: from where y's pairs lie to where x's lie, as chunks and then as pairs again
    Two d = turn<OUT, IN>(split<OUT>(widen8<DT>(g[0]), widen8<DT>(g[1])), ang.c, ang.s, l.rot);
    d = split<IN>(d.a, d.b);
    float ss = 0.f, dot = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      ss += v.a[i] * v.a[i] + v.b[i] * v.b[i];
      dot += d.a[i] * w.a[i] * v.a[i] + d.b[i] * w.b[i] * v.b[i];
    }
    ss = head_sum(live ? ss : 0.f, p.lpr);
    dot = head_sum(live ? dot : 0.f, p.lpr);
    const float r = rsqrtf(ss * p.inv_d + p.eps);
    const float m = dot * r * p.inv_d;  // mean(u w n)
    if (live) {
      Two dx;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float na = v.a[i] * r, nb = v.b[i] * r;
        dw.a[i] += d.a[i] * na;
        dw.b[i] += d.b[i] * nb;
        dx.a[i] = r * (d.a[i] * w.a[i] - na * m);
        dx.b[i] = r * (d.b[i] * w.b[i] - nb * m);
      }
      const Two out = join<IN>(dx);
      E* at = static_cast<E*>(Y.p) + t * Y.ts + h * Y.hs;
      store8<DT>(at + l.in0, out.a);
      store8<DT>(at + l.in1, out.b);
    }
  }
  // the workgroup's sums: lanes that own the same features, then waves, in order
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    float a = dw.a[i], b = dw.b[i];
    for (int s = p.lpr; s < 64; s <<= 1) {
      a += __shfl_xor(a, s);
      b += __shfl_xor(b, s);
    }
    if (mine && sub == 0) {
      lds[wave][IN ? l.in0 + i : (i < 4 ? l.in0 + 2 * i : l.in1 + 2 * (i - 4))] = a;
      lds[wave][IN ? l.in1 + i : (i < 4 ? l.in0 + 2 * i + 1 : l.in1 + 2 * (i - 4) + 1)] = b;
    }
  }
  __syncthreads();
  for (int f = threadIdx.x; f < p.D; f += 64 * kBackWaves) {
    float sum = 0.f;
#pragma unroll
    for (int v = 0; v < kBackWaves; ++v) sum += lds[v][f];
    p.parts[(int64_t)blockIdx.x * p.D + f] = sum;
  }
}

// dWQ from the first parts_q workgroups' sums and dWK from the others' (their rows `stride` apart), 16 columns and 64
// groups of rows to a workgroup, added in a fixed order.
__global__ __launch_bounds__(1024) void weight_sum_kernel(const float* q, int count_q, const float* k, int count_k,
                                                          int64_t stride, float* dwq, float* dwk, int D) {
  __shared__ float lds[64][17];
  const int c = threadIdx.x & 15, g = threadIdx.x >> 4;
  const bool keys = blockIdx.y != 0;
  const float* parts = keys ? k : q;
  const int count = keys ? count_k : count_q, i = blockIdx.x * 16 + c;
  float sum = 0.f;
  if (i < D) {
#pragma unroll 8
    for (int w = g; w < count; w += 64) sum += parts[w * stride + i];
  }
  lds[g][c] = sum;
  __syncthreads();
  if (g == 0 && i < D) {
    float s = 0.f;
#pragma unroll
    for (int w = 0; w < 64; ++w) s += lds[w][c];
    (keys ? dwk : dwq)[i] = s;
  }
}

}  // namespace heads
}  // namespace mxg
