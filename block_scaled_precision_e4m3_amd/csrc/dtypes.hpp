// Plain (unquantised) element types by their MXG_DT_* number: loads and stores
// of runs of 8 elements as float32, and of single elements.
#pragma once

#include "mxgemm_common.hpp"

namespace mxg {

template <int DT>
struct Elem;
template <>
struct Elem<0> { using type = float; };
template <>
struct Elem<1> { using type = __bf16; };
template <>
struct Elem<2> { using type = _Float16; };
template <int DT>
using elem_t = typename Elem<DT>::type;

typedef _Float16 v8h __attribute__((ext_vector_type(8)));
typedef float v8f __attribute__((ext_vector_type(8)));

// 8 consecutive elements, raw and as float32.  They may lie at any address an element may have: gfx950 takes 16-byte
// accesses at any alignment, and aligned ones as fast.
template <int DT>
struct Raw8 {
  v4u w[DT == 0 ? 2 : 1];
};
template <int DT>
struct __attribute__((packed, aligned(DT == 0 ? 4 : 2))) Raw8At {
  Raw8<DT> v;
};
template <int DT>
__device__ __forceinline__ Raw8<DT> load8(const elem_t<DT>* p) {
  return reinterpret_cast<const Raw8At<DT>*>(p)->v;
}
template <int DT>
__device__ __forceinline__ v8f widen8(const Raw8<DT>& r) {
  v8f f;
  if constexpr (DT == 0) {
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = __uint_as_float(r.w[i >> 2][i & 3]);
  } else if constexpr (DT == 1) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[2 * i] = __uint_as_float(r.w[0][i] << 16);
      f[2 * i + 1] = __uint_as_float(r.w[0][i] & 0xFFFF0000u);
    }
  } else {
    f = __builtin_convertvector(__builtin_bit_cast(v8h, r.w[0]), v8f);
  }
  return f;
}
// Rounded to nearest even (float16 overflows to infinity).
template <int DT>
__device__ __forceinline__ void store8(elem_t<DT>* p, const v8f& f) {
  Raw8<DT> r;
  if constexpr (DT == 0) {
#pragma unroll
    for (int i = 0; i < 8; ++i) r.w[i >> 2][i & 3] = __float_as_uint(f[i]);
  } else if constexpr (DT == 1) {
    r.w[0] = __builtin_bit_cast(v4u, __builtin_convertvector(f, v8bf));
  } else {
    r.w[0] = __builtin_bit_cast(v4u, __builtin_convertvector(f, v8h));
  }
  reinterpret_cast<Raw8At<DT>*>(p)->v = r;
}

// 8 elements at p, those at or past `valid` as zero.
template <int DT>
__device__ __forceinline__ Raw8<DT> load_chunk(const elem_t<DT>* p, int valid) {
  if (valid >= 8) return load8<DT>(p);
  Raw8<DT> r;
#pragma unroll
  for (int i = 0; i < (DT == 0 ? 2 : 1); ++i) r.w[i] = (v4u){0, 0, 0, 0};
  if (valid > 0) {  // the end of a row
#pragma unroll
    for (int i = 0; i < 7; ++i) {
      if constexpr (DT == 0) {
        r.w[i >> 2][i & 3] = i < valid ? __float_as_uint(p[i]) : 0u;
      } else {
        const unsigned h = i < valid ? (unsigned)__builtin_bit_cast(unsigned short, p[i]) : 0u;
        r.w[0][i >> 1] |= h << (16 * (i & 1));
      }
    }
  }
  return r;
}

// The first `valid` (1..8) of 8 elements, rounded as above.
template <int DT>
__device__ __forceinline__ void store_chunk(elem_t<DT>* p, const v8f& f, int valid) {
  if (valid >= 8) return store8<DT>(p, f);
#pragma unroll
  for (int i = 0; i < 7; ++i)
    if (i < valid) p[i] = (elem_t<DT>)f[i];
}

// The number of bytes of one element on the host.
inline int elem_bytes(int dt) { return dt == 0 ? 4 : 2; }

}  // namespace mxg
