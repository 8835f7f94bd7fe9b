// Quantisation to 8-bit codes with one float32 scale per block of 128, on
// gfx950: rows (blocks of 1 x 128 along K), columns (blocks of 128 x 1, stored
// transposed) or both from one read of X, or 128 x 128 blocks.
//
//   a = max |x| over the block, at least 448 * 2^-100;  scale = a / FMAX,
//   code = rne(x FMAX / a);  power-of-two scales: 2^e, e the smallest integer
//   with FMAX * 2^e >= a.
//
// x FMAX / a is taken as x hi + x lo with hi + lo = FMAX / a to about 2^-47, or
// 2^-30.8 where a is so large that lo is subnormal: one multiply and one
// multiply-add per element, after which a ratio that lies on a boundary between
// two codes, as those of 16-bit values often do, stays on it.  With hi alone 0.3%
// of the codes of bfloat16 activations came out on the other side.  Quotients of
// 16-bit values are either on a boundary or 2^-16 of themselves away; one of
// float32 values can be so near that float32 rounds it onto the boundary, about
// one in 2^20, and settle() then looks at what was rounded off.  No clamp is
// needed: the quotient never exceeds FMAX.
//
// A workgroup takes a tile of 16 RT rows x 128 columns: thread (g, c) holds
// rows RT g .. RT g + RT - 1 of columns 8c .. 8c + 7 in registers, RT chunks of
// 8 elements as loaded.  Row maxima finish across the 16 lanes of a row; column
// maxima across the 16 threads of a chunk, in LDS.  Magnitudes are compared as
// the integers of their bits without the sign, which orders NaN above infinity
// above the finite, so a block that holds either gets a scale that is neither
// lost nor finite.  The transposed codes are converted along the thread's 8
// rows, gathered in LDS as (column, row) bytes and stored as whole 128-byte
// rows.
//
// The bound is memory: 8192 x 7168 bfloat16, rows and columns, 51 us (4.65
// TB/s), 7168 x 2048 float32 squares with their transpose 14.9 us; 8 x 7168 rows
// take 2.3 us, of which 1.95 are an empty launch.
#pragma once

#include "dtypes.hpp"
#include "mx_quantize.hpp"

namespace mxg {
namespace b128 {

constexpr int kQThreads = 256;

struct QuantParams {
  const void* X;
  uint8_t* Q;
  float* S;
  uint8_t* QT;
  float* ST;
  int64_t ldx;
  int M, K, L;
  int K16, M16;      // row lengths of Q and QT
  int Mb, Kb;        // ceil(M / 128), ceil(K / 128)
  int tiles_m;       // row tiles per batch
  int first;         // the launch's first tile
  bool pow2;
};

constexpr unsigned kTinyBits = 0x11E00000u;  // 448 * 2^-100 = 1.75 * 2^-92

struct Scale {
  float scale, hi, lo;  // lo: what hi leaves out of FMAX / a
};
// The value of another lane of the 16 that share a row, so that four maxima in turn cover them: the pair's other, the
// quad's other pair, then the mirrored half and row.
__device__ __forceinline__ unsigned across16(unsigned v, int step) {
  if (step == 0) return (unsigned)__builtin_amdgcn_mov_dpp((int)v, 0xB1, 0xF, 0xF, true);
  if (step == 1) return (unsigned)__builtin_amdgcn_mov_dpp((int)v, 0x4E, 0xF, 0xF, true);
  if (step == 2) return (unsigned)__builtin_amdgcn_mov_dpp((int)v, 0x141, 0xF, 0xF, true);
  return (unsigned)__builtin_amdgcn_mov_dpp((int)v, 0x140, 0xF, 0xF, true);
}

// Scale and multiplier of a block from the bits of its largest magnitude (float32).
template <int FMT>
__device__ __forceinline__ Scale block_scale(unsigned bits, bool pow2) {
  constexpr float kMax = FMT == 0 ? 448.f : 57344.f;
  const float a = __uint_as_float(bits > kTinyBits ? bits : kTinyBits);
  if (pow2 && bits < 0x7F800000u) {
    const int e = quant::block_exponent<FMT>(a);
    return {__uint_as_float((unsigned)(127 + e) << 23), __uint_as_float((unsigned)(127 - e) << 23), 0.f};
  }
  const float near = kMax / a;  // correctly rounded; an infinity or NaN makes every code NaN
  const float rest = __builtin_fmaf(-near, a, kMax) / a;
  // hi is the quotient rounded down, so that lo is not negative: x hi + x lo then keeps the sign of a zero
  const float hi = rest < 0.f ? __int_as_float(__float_as_int(near) - 1) : near;
  return {a / kMax, hi, rest + (near - hi)};
}

__device__ __forceinline__ float scaled(float x, const Scale& s) { return __builtin_fmaf(x, s.hi, x * s.lo); }

// A quotient r that float32 has rounded onto a boundary between codes, moved to the side it came from by one unit in
// its last place.  One that is not on the boundary is more than 2^-29 r away from it (x FMAX and boundary times a are
// integers of 27 and 29 bits, times powers of two).  What is known of it is within 2^-30.8 r: lo is off by 2^-150 at
// most, half the smallest subnormal, next to hi of at least 448 / 2^128 (a below 2^103: within 2^-46 r).  So the
// distance is found above 2^-29.5 r, or below 2^-30.8 r, and 2^-30 r tells them apart.
__device__ __forceinline__ float settle(float r, float x, const Scale& s) {
  const float off = __builtin_fmaf(x, s.hi, -r) + x * s.lo;
  const int away = (__float_as_int(off) ^ __float_as_int(r)) < 0 ? -1 : 1;
  const bool move = (__float_as_uint(r) & 0x7FFFFu) == 0 && fabsf(off) > fabsf(r) * 0x1p-30f;
  return __int_as_float(__float_as_int(r) + (move ? away : 0));
}

// The four columns of a 4 x 4 square of bytes from its four rows.
__device__ __forceinline__ void turn4(unsigned a, unsigned b, unsigned c, unsigned d, unsigned* w) {
  const unsigned ab0 = __builtin_amdgcn_perm(b, a, 0x05010400u), ab1 = __builtin_amdgcn_perm(b, a, 0x07030602u);
  const unsigned cd0 = __builtin_amdgcn_perm(d, c, 0x05010400u), cd1 = __builtin_amdgcn_perm(d, c, 0x07030602u);
  w[0] = __builtin_amdgcn_perm(cd0, ab0, 0x05040100u);
  w[1] = __builtin_amdgcn_perm(cd0, ab0, 0x07060302u);
  w[2] = __builtin_amdgcn_perm(cd1, ab1, 0x05040100u);
  w[3] = __builtin_amdgcn_perm(cd1, ab1, 0x07060302u);
}

// Codes of four elements of a block.
template <int DT, int FMT>
__device__ __forceinline__ unsigned codes_of(float x0, float x1, float x2, float x3, const Scale& s) {
  float r0 = scaled(x0, s), r1 = scaled(x1, s), r2 = scaled(x2, s), r3 = scaled(x3, s);
  if constexpr (DT == 0) {
    // boundaries have at most 5 significant bits, so the last 19 of the 23 stored ones are zero
    const unsigned a = min(__float_as_uint(r0) << 13, __float_as_uint(r1) << 13);
    const unsigned b = min(__float_as_uint(r2) << 13, __float_as_uint(r3) << 13);
    if (min(a, b) == 0) {
      r0 = settle(r0, x0, s);
      r1 = settle(r1, x1, s);
      r2 = settle(r2, x2, s);
      r3 = settle(r3, x3, s);
    }
  }
  return quant::codes4<FMT>(r0, r1, r2, r3);
}

// Bits of the magnitudes of 8 elements, as loaded: two 16-bit ones to a dword.
template <int DT>
struct Mag8 {
  unsigned w[DT == 0 ? 8 : 4];
};
template <int DT>
__device__ __forceinline__ Mag8<DT> magnitudes(const Raw8<DT>& r) {
  Mag8<DT> m;
  if constexpr (DT == 0) {
#pragma unroll
    for (int i = 0; i < 8; ++i) m.w[i] = r.w[i >> 2][i & 3] & 0x7FFFFFFFu;
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) m.w[i] = r.w[0][i] & 0x7FFF7FFFu;
  }
  return m;
}
typedef unsigned short v2us __attribute__((ext_vector_type(2)));
template <int DT>
__device__ __forceinline__ unsigned mag_max(unsigned a, unsigned b) {
  if constexpr (DT == 0) return max(a, b);
  else return __builtin_bit_cast(unsigned, __builtin_elementwise_max(__builtin_bit_cast(v2us, a), __builtin_bit_cast(v2us, b)));
}
// float32 bits of the larger half of a dword of two 16-bit magnitudes (or of a float32 magnitude).
template <int DT>
__device__ __forceinline__ unsigned half_bits(unsigned h) {
  if constexpr (DT == 1) return h << 16;
  else return __float_as_uint((float)__builtin_bit_cast(_Float16, (unsigned short)h));
}
template <int DT>
__device__ __forceinline__ unsigned mag_bits(unsigned m) {
  if constexpr (DT == 0) return m;
  else return half_bits<DT>(max(m & 0xFFFFu, m >> 16));
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

template <int DT, int FMT, int RT, bool ROWS, bool COLS, bool SQUARE>
__global__ __launch_bounds__(kQThreads) void block128_quantize_kernel(QuantParams p) {
  static_assert(RT == 8 || (!COLS && !SQUARE), "columns and squares need the 128 rows of a block");
  constexpr int kRows = 16 * RT, kPitch = 132;  // LDS bytes between columns of the transposed codes
  __shared__ __attribute__((aligned(16))) uint8_t tile[COLS ? 128 * kPitch : 16];
  __shared__ unsigned colmax[COLS && !SQUARE ? 4 : 1][COLS && !SQUARE ? 128 : 4];
  __shared__ float rowscale[ROWS && !SQUARE ? kRows : 1];

  const int tid = threadIdx.x, c = tid & 15, g = tid >> 4, wave = tid >> 6;
  int b = p.first + (int)blockIdx.x;
  const int kb = b % p.Kb;
  b /= p.Kb;
  const int tm = b % p.tiles_m, l = b / p.tiles_m;
  const int m0 = tm * kRows, k0 = kb * 128, k = k0 + 8 * c;
  const elem_t<DT>* x = static_cast<const elem_t<DT>*>(p.X) + ((int64_t)l * p.M + m0) * p.ldx + k;

  Raw8<DT> v[RT];
#pragma unroll
  for (int i = 0; i < RT; ++i) {
    const int m = RT * g + i;
    v[i] = load_chunk<DT>(x + (int64_t)m * p.ldx, m0 + m < p.M ? p.K - k : 0);
  }

  // largest magnitudes: of the thread's rows, and of its columns
  constexpr int kW = DT == 0 ? 8 : 4;
  unsigned rmax[RT];
  Mag8<DT> cmax;
#pragma unroll
  for (int i = 0; i < RT; ++i) {
    const Mag8<DT> m = magnitudes<DT>(v[i]);
    unsigned r = m.w[0];
#pragma unroll
    for (int j = 1; j < kW; ++j) r = mag_max<DT>(r, m.w[j]);
    rmax[i] = mag_bits<DT>(r);
    if constexpr (COLS && !SQUARE) {
#pragma unroll
      for (int j = 0; j < kW; ++j) cmax.w[j] = i == 0 ? m.w[j] : mag_max<DT>(cmax.w[j], m.w[j]);
    }
  }

  Scale row[RT], col[8];
  if constexpr (SQUARE) {
    unsigned t = rmax[0];
#pragma unroll
    for (int i = 1; i < RT; ++i) t = max(t, rmax[i]);
#pragma unroll
    for (int s = 0; s < 4; ++s) t = max(t, across16(t, s));
    t = max(t, (unsigned)__shfl_xor((int)t, 16));
    t = max(t, (unsigned)__shfl_xor((int)t, 32));
    if ((tid & 63) == 0) colmax[0][wave] = t;
    __syncthreads();
    t = max(max(colmax[0][0], colmax[0][1]), max(colmax[0][2], colmax[0][3]));
    const Scale s = block_scale<FMT>(t, p.pow2);
#pragma unroll
    for (int i = 0; i < RT; ++i) row[i] = s;
    if (tid == 0) {
      if constexpr (ROWS) p.S[((int64_t)l * p.Mb + tm) * p.Kb + kb] = s.scale;
      if constexpr (COLS) p.ST[((int64_t)l * p.Kb + kb) * p.Mb + tm] = s.scale;
    }
  } else {
    if constexpr (ROWS) {
#pragma unroll
      for (int i = 0; i < RT; ++i) {
        unsigned t = rmax[i];
#pragma unroll
        for (int s = 0; s < 4; ++s) t = max(t, across16(t, s));
        row[i] = block_scale<FMT>(t, p.pow2);
        if (c == 0) rowscale[RT * g + i] = row[i].scale;
      }
    }
    if constexpr (COLS) {
      // across the wave's four rows of threads, then across the waves
#pragma unroll
      for (int j = 0; j < kW; ++j) {
        unsigned t = cmax.w[j];
        t = mag_max<DT>(t, (unsigned)__shfl_xor((int)t, 16));
        t = mag_max<DT>(t, (unsigned)__shfl_xor((int)t, 32));
        if ((tid & 48) == 0) {
          if constexpr (DT == 0) {
            colmax[wave][8 * c + j] = t;
          } else {
            colmax[wave][8 * c + 2 * j] = half_bits<DT>(t & 0xFFFFu);
            colmax[wave][8 * c + 2 * j + 1] = half_bits<DT>(t >> 16);
          }
        }
      }
    }
    __syncthreads();
    if constexpr (COLS) {
      // each column's scale once, left in place of its maximum: thread j < 128 makes column j's
      if (tid < 128) {
        const unsigned t = max(max(colmax[0][tid], colmax[1][tid]), max(colmax[2][tid], colmax[3][tid]));
        const Scale s = block_scale<FMT>(t, p.pow2);
        if (k0 + tid < p.K) p.ST[((int64_t)l * p.Mb + tm) * p.K + k0 + tid] = s.scale;
        colmax[0][tid] = __float_as_uint(s.hi);
        colmax[1][tid] = __float_as_uint(s.lo);
      }
      __syncthreads();
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        col[j].hi = __uint_as_float(colmax[0][8 * c + j]);
        col[j].lo = __uint_as_float(colmax[1][8 * c + j]);
      }
    }
    if constexpr (ROWS) {
      if (tid < kRows && m0 + tid < p.M) p.S[((int64_t)l * p.Kb + kb) * p.M + m0 + tid] = rowscale[tid];
    }
  }

  uint2 u[RT];  // codes of the rows
  if constexpr (ROWS || SQUARE) {
#pragma unroll
    for (int i = 0; i < RT; ++i) {
      const v8f f = widen8<DT>(v[i]);
      const Scale& s = row[SQUARE ? 0 : i];
      u[i] = make_uint2(codes_of<DT, FMT>(f[0], f[1], f[2], f[3], s), codes_of<DT, FMT>(f[4], f[5], f[6], f[7], s));
    }
  }
  if constexpr (ROWS) {
    uint8_t* q = p.Q + ((int64_t)l * p.M + m0) * p.K16 + k;
#pragma unroll
    for (int i = 0; i < RT; ++i) {
      const int m = RT * g + i;
      if (m0 + m < p.M && k < p.K16) *reinterpret_cast<uint2*>(q + (int64_t)m * p.K16) = u[i];
    }
  }
  if constexpr (COLS) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      unsigned w[8];  // column j's codes of rows 4h .. 4h + 3
      if constexpr (SQUARE) {
        // the same codes, turned in registers
        turn4(u[4 * h].x, u[4 * h + 1].x, u[4 * h + 2].x, u[4 * h + 3].x, w);
        turn4(u[4 * h].y, u[4 * h + 1].y, u[4 * h + 2].y, u[4 * h + 3].y, w + 4);
      } else {
        const v8f f0 = widen8<DT>(v[4 * h]), f1 = widen8<DT>(v[4 * h + 1]), f2 = widen8<DT>(v[4 * h + 2]),
                  f3 = widen8<DT>(v[4 * h + 3]);
#pragma unroll
        for (int j = 0; j < 8; ++j) w[j] = codes_of<DT, FMT>(f0[j], f1[j], f2[j], f3[j], col[j]);
      }
#pragma unroll
      for (int j = 0; j < 8; ++j)
        *reinterpret_cast<unsigned*>(tile + (8 * c + j) * kPitch + 8 * g + 4 * h) = w[j];
    }
    __syncthreads();
    uint8_t* q = p.QT + ((int64_t)l * p.K + k0) * p.M16 + m0;
    const int at = 16 * (tid & 7);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int r = (tid >> 3) + 32 * i;
      const unsigned* t = reinterpret_cast<const unsigned*>(tile + r * kPitch + at);
      const v4u u = {t[0], t[1], t[2], t[3]};
      if (k0 + r < p.K && m0 + at < p.M16) *reinterpret_cast<v4u*>(q + (int64_t)r * p.M16 + at) = u;
    }
  }
}

}  // namespace b128
}  // namespace mxg
