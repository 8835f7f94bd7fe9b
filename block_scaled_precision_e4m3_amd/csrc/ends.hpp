// What a product's values z pass through before they are stored:
//   z = product + bias,  y = act(z) gate + residual
// and the activations with their slopes, in float32.
//
//   relu       max(z, 0)                            slope z > 0
//   silu       z s(z), s(u) = 1 / (1 + e^-u)
//   gelu       z P(z), P the normal distribution's
//   gelu_tanh  z s(u), u = 2 sqrt(2/pi) (z + 0.044715 z^3), which is z (1 + tanh(u/2)) / 2 without its cancellation
//
// P's tail, and from it P, is e^(-x^2/2) R(x), x = |z|, with R a polynomial in 1 / (1 + p x) fitted to erfcx(x / sqrt 2) /
// 2 over 0..14 for the least relative error.  FAST is for results that are rounded to 16 bits: hardware exponential and
// reciprocal (about 2^-22, and |u| 2^-24 for the exponential's argument), and R of degree 6, off by 4.7e-6: a fiftieth of
// float16's rounding.  Slopes take R of degree 8 all the same, since their sums, the bias' gradient, are float32 (degree 6:
// 1.4e-6 off over 8192 rows, degree 8: 1.5e-7, in the same time).  The others keep what the exponential's argument loses,
// divide, and take R of degree 8, off by 4e-7 of the tail with the rounding of its own sums.
#pragma once

#include "../../include/mxgemm.h"
#include "dtypes.hpp"

namespace mxg {
namespace ends {

struct Ends {
  const void* bias;      // (N), of C's type or float32
  const void* gate;      // (M, N), rows ldg apart
  const void* residual;  // (M, N), rows ldr apart
  void* Z;               // (M, N), rows ldz apart: z, rounded
  int64_t ldg, ldr, ldz;
  int act;               // MXG_ACT_*
  bool bias_f32;
};

// e^u
template <bool FAST>
__device__ __forceinline__ float exponential(float u) {
  constexpr float log2e = 1.44269502f, rest = 1.925963033e-8f;  // their sum is log2 of e
  if constexpr (FAST) {
    return __builtin_amdgcn_exp2f(log2e * u);
  } else {
    const float hi = log2e * u, lo = __builtin_fmaf(log2e, u, -hi) + rest * u;
    const float e = __builtin_amdgcn_exp2f(hi);
    // an infinite e has no part that could be added, and next to zero none that counts
    return fabsf(hi) < 128.f ? __builtin_fmaf(e, 0.6931471806f * lo, e) : e;
  }
}

// s(u) and what is left of one, from e = e^-u.  The rest is e s: 1 - s would lose a rounding of s, which slopes multiply by z
// and more (gelu_tanh's at z = 5 was off by 2.0e-6, silu's at 8.7 by 7e-7; 2e-7 so).  An infinite e, with s zero, leaves one.
struct Sigmoid {
  float s, rest;
};
template <bool FAST>
__device__ __forceinline__ Sigmoid sigmoid_of(float e) {
  float s;
  if constexpr (FAST) s = __builtin_amdgcn_rcpf(1.f + e);
  else s = 1.f / (1.f + e);
  return {s, fminf(e * s, 1.f)};
}
template <bool FAST>
__device__ __forceinline__ Sigmoid sigmoid(float u) {
  return sigmoid_of<FAST>(exponential<FAST>(-u));
}

// gelu_tanh's s(u), u = a z + b z^3.  What u's rounding loses is a part |u| 2^-22 of the tail: float32 results keep it.
// z^2 stays finite, so that an infinite z keeps its sign.
template <bool FAST>
__device__ __forceinline__ Sigmoid tanh_sigmoid(float z) {
  constexpr float a = 1.5957692f, b = 0.071354814f;
  const float q = fminf(z * z, 1e30f);
  if constexpr (FAST) {
    return sigmoid<true>(z * __builtin_fmaf(q, b, a));
  } else {
    constexpr float a_rest = -4.534068e-8f, b_rest = 2.3988325e-9f;  // of 2 sqrt(2/pi) and 0.044715 times it
    const float t = b * q, t_rest = __builtin_fmaf(b, q, -t) + __builtin_fmaf(b, __builtin_fmaf(z, z, -q), b_rest * q);
    const float p = t + a, back = p - t, p_rest = (t - (p - back)) + (a - back) + t_rest + a_rest;
    const float u = z * p, u_rest = __builtin_fmaf(z, p, -u) + z * p_rest;
    const float e = exponential<false>(-u);
    return sigmoid_of<false>(fabsf(u) < 80.f ? __builtin_fmaf(-e, u_rest, e) : e);
  }
}

// P's lower tail at -|z|, and e^(-z^2/2).
struct Tail {
  float p, e;
};
// R of degree 8.
__device__ __forceinline__ float long_tail(float t) {
  float r = 0.0356745869f;
  r = __builtin_fmaf(r, t, -0.157202214f);
  r = __builtin_fmaf(r, t, 0.206351876f);
  r = __builtin_fmaf(r, t, -0.0536820367f);
  r = __builtin_fmaf(r, t, 0.128560722f);
  r = __builtin_fmaf(r, t, 0.0999137834f);
  r = __builtin_fmaf(r, t, 0.120753907f);
  r = __builtin_fmaf(r, t, 0.119629301f);
  return r * t;
}
template <bool FAST, bool LONG = !FAST>
__device__ __forceinline__ Tail tail(float z) {
  if constexpr (FAST && LONG) {
    const float w = 0.8493218003f * z;
    const float e = __builtin_amdgcn_exp2f(-(w * w));
    return {long_tail(__builtin_amdgcn_rcpf(__builtin_fmaf(fabsf(z), 0.3f, 1.f))) * e, e};
  } else if constexpr (FAST) {
    const float w = 0.8493218003f * z;  // w^2 is z^2/2 in powers of 2
    const float e = __builtin_amdgcn_exp2f(-(w * w));
    const float t = __builtin_amdgcn_rcpf(__builtin_fmaf(fabsf(w), 0.31f / 0.8493218003f, 1.f));
    float r = -0.0739273363f;
    r = __builtin_fmaf(r, t, 0.180445171f);
    r = __builtin_fmaf(r, t, 0.0157504037f);
    r = __builtin_fmaf(r, t, 0.133426788f);
    r = __builtin_fmaf(r, t, 0.120442029f);
    r = __builtin_fmaf(r, t, 0.12386063f);
    return {r * t * e, e};
  } else {
    const float s = -0.5f * z, q = s * z;
    float e = exponential<false>(q);
    if (q > -150.f) e = __builtin_fmaf(e, __builtin_fmaf(s, z, -q), e);  // what q's rounding loses
    const float t = 1.f / __builtin_fmaf(fabsf(z), 0.3f, 1.f);
    return {long_tail(t) * e, e};
  }
}
// z P(z) = max(z, 0) - |z| P(-|z|), |z| held finite, as the tail of an infinity is zero.  A NaN is one in the tail.
__device__ __forceinline__ float gelu_of(float z, const Tail& t) {
  return __builtin_fmaf(-fminf(fabsf(z), 3e38f), t.p, fmaxf(z, 0.f));
}

// f(g) with g(z) the activation of that kind: the choice stands outside of what loops over values.
template <bool FAST, class F>
__device__ __forceinline__ void with_activation(int act, F f) {
  if (act == MXG_ACT_RELU) f([](float z) { return z < 0.f ? 0.f : z; });
  else if (act == MXG_ACT_SILU) f([](float z) { return z * sigmoid<FAST>(z).s; });
  else if (act == MXG_ACT_GELU) f([](float z) { return gelu_of(z, tail<FAST>(z)); });
  else if (act == MXG_ACT_GELU_TANH) f([](float z) { return z * tanh_sigmoid<FAST>(z).s; });
}

struct Slope {
  float value, slope;
};
// f(g) with g(z) the activation and its slope.
template <bool FAST, class F>
__device__ __forceinline__ void with_slope(int act, F f) {
  if (act == MXG_ACT_RELU) {
    f([](float z) { return Slope{z < 0.f ? 0.f : z, z > 0.f ? 1.f : 0.f}; });
  } else if (act == MXG_ACT_SILU) {
    f([](float z) {
      const Sigmoid s = sigmoid<FAST>(z);
      const float y = z * s.s;
      return Slope{y, __builtin_fmaf(y, s.rest, s.s)};
    });
  } else if (act == MXG_ACT_GELU) {
    f([](float z) {
      const Tail t = tail<FAST, true>(z);
      return Slope{gelu_of(z, t), __builtin_fmaf(0.3989422804f * z, t.e, z > 0.f ? 1.f - t.p : t.p)};
    });
  } else if (act == MXG_ACT_GELU_TANH) {
    f([](float z) {
      const Sigmoid s = tanh_sigmoid<FAST>(z);
      const float y = z * s.s;
      const float du = __builtin_fmaf(fminf(z * z, 1e30f), 3.f * 0.044715f * 1.5957691216f, 1.5957691216f);
      return Slope{y, __builtin_fmaf(y * s.rest, du, s.s)};
    });
  } else {
    f([](float z) { return Slope{z, 1.f}; });
  }
}

template <int CT>
__device__ __forceinline__ float bias_at(const void* bias, bool f32, int n) {
  return f32 ? static_cast<const float*>(bias)[n] : (float)static_cast<const elem_t<CT>*>(bias)[n];
}

// The value to store for the product's value z at (m, n); stores what is kept of z.
template <int CT>
__device__ __forceinline__ float finish(const Ends& e, float z, int64_t m, int n) {
  using E = elem_t<CT>;
  if (e.bias) z += bias_at<CT>(e.bias, e.bias_f32, n);
  if (e.Z) static_cast<E*>(e.Z)[m * e.ldz + n] = (E)z;
  with_activation<CT != 0>(e.act, [&](auto act) { z = act(z); });
  if (e.gate) z *= (float)static_cast<const E*>(e.gate)[m * e.ldg + n];
  if (e.residual) z += (float)static_cast<const E*>(e.residual)[m * e.ldr + n];
  return z;
}

}  // namespace ends
}  // namespace mxg
