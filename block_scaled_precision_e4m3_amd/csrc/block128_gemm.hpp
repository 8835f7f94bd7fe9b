// The product of two block-128 quantised operands on gfx950:
//   C[m,n] = sum_j SA[j,m] SB(j,n) sum_{k in block j} dec(A[m,k]) dec(B[n,k])
//
// Two tile kernels share the movement of operands (Stream): a 16-bit C is made
// on the 8-bit matrix cores, a float32 C from codes widened to bfloat16, whose
// products and sums are exact to float32.  Either way the sum over one block of
// 128 starts from zero and goes into float32 accumulators with one multiply-add
// by the product of its two scales, which are float32 and cannot ride on the
// matrix cores' power-of-two scales.  Few rows of A go through a third kernel
// that reads B straight from memory.
#pragma once

#include <type_traits>

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
  int steps, splits, per;  // steps of a tile's whole K; parts it is cut into, of `per` steps each (the last may be shorter)
  float* sums;       // splits > 1: (splits, L, M, ldw) float32 partial sums in place of C
  int ldw;
  int first;         // kernel for few rows: the launch's first group of columns
  bool b_rows, accumulate;
  bool c_vec;        // base, ldc and N in multiples of 16 bytes: every store of C is a whole one
};

// 16 bytes where an element of C may lie: gfx950 takes 16-byte accesses at any alignment.
typedef v4u v4u_at2 __attribute__((aligned(2)));
typedef v4u v4u_at4 __attribute__((aligned(4)));

constexpr unsigned kOob = 0x80000000u;  // an offset past every resource: reads as zero, is not stored

// A tile of BM x BN outputs by WM x WN waves, operands in a ring of NST stages of KB blocks of K each, moved by the
// same waves (NP = 0) or by NP more that do nothing else.  PARTS: the kernel can take part of K.
template <int BM, int BN, int WM, int WN, int NST, int KB, int NP = 0, bool PARTS = (NP > 0)>
struct TileShape {
  static constexpr int kBM = BM, kBN = BN, kWaves = WM * WN, kWn = WN, kStages = NST, kKB = KB;
  static constexpr bool kParts = PARTS;
  static constexpr int kProducers = NP, kDmaWaves = NP ? NP : kWaves, kAllWaves = kWaves + NP;
  static constexpr int kTM = BM / WM, kTN = BN / WN;     // a wave's outputs
  static constexpr int kOffB = BM * 128, kOffSA = kOffB + BN * 128, kOffSB = kOffSA + BM * 4;
  static constexpr int kBlock = kOffSB + BN * 4;         // LDS bytes of one block of K
  static constexpr int kStage = KB * kBlock;
  static constexpr int kDa = BM / 8 / kDmaWaves, kDb = BN / 8 / kDmaWaves;  // operand DMA instructions per wave and step
  static constexpr int kPerBlock = kDa + kDb + 1;                     // and the scales', for one block
  static constexpr int kIssued = KB * kPerBlock;
  static_assert(kDmaWaves % 4 == 0 && (BM / 8) % kDmaWaves == 0 && (BN / 8) % kDmaWaves == 0, "DMA shares");
  static_assert(BM % 64 == 0 && BN % 64 == 0 && BM / 64 + BN / 64 <= kDmaWaves, "one scale DMA per wave");
  static_assert(kTN % 32 == 0 && 128 % kTN == 0, "one 128-column block per wave");
  static constexpr int kLds = NST * kStage + 256;        // and where waves without scales to fetch write zeros
  static_assert(kLds <= 160 * 1024, "LDS");
};

// As dma16_at, 4 bytes per lane to m0 + 4 * lane.
#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"
__device__ __forceinline__ void dma4_at(__amdgpu_buffer_rsrc_t rs, unsigned voff, unsigned lds_addr) {
  const unsigned m0 = __builtin_amdgcn_readfirstlane(lds_addr);
  asm volatile("s_mov_b32 m0, %2\n\ts_nop 3\n\tbuffer_load_dword %0, %1, 0 offen lds" ::"v"(voff), "s"(rs), "s"(m0)
               : "memory", "m0");
}
#pragma clang diagnostic pop

struct TileAt {
  int l, m0, n0;
};
struct Part {
  int at, count;  // first step and number of steps
};
template <class T>
__device__ __forceinline__ Part part_of(const GemmParams& p, int item) {
  if (!T::kParts || p.splits == 1) return {0, p.steps};
  const int at = __builtin_amdgcn_readfirstlane(item / p.num_tiles * p.per);
  return {at, min(p.per, p.steps - at)};
}
// Tile t: batches, then groups of kGroupM tile rows walked column by column.  A work item is a tile and a part of
// its K; items of one part follow each other.
template <class T>
__device__ __forceinline__ TileAt tile_at(const GemmParams& p, int t) {
  constexpr int bm = T::kBM, bn = T::kBN;
  if (T::kParts && p.splits > 1) t %= p.num_tiles;
  const int per = p.tilesM * p.tilesN, l = t / per, r = t - l * per;
  const int group = kGroupM * p.tilesN, g = r / group, first = g * kGroupM;
  const int rows = min(p.tilesM - first, kGroupM), rg = r - g * group;
  return {__builtin_amdgcn_readfirstlane(l), __builtin_amdgcn_readfirstlane((first + rg % rows) * bm),
          __builtin_amdgcn_readfirstlane(rg / rows * bn)};
}

// The workgroup's stream of K steps, tile after tile.  A step is one scale
// block: 128 bytes of every row of A and B and the scales beside them, by
// global->LDS DMA.  Wave w fills the 8-row groups w, w + waves, ... of each
// operand, lane l the 16-byte slot l % 8 of row l / 8; slot s of row R holds
// chunk s ^ f(R) with f an operand's swizzle SwA or SwB.  A 16-byte LDS read is
// served in four passes of 16 lanes, lanes {0-3, 12-15, 20-27} and
// {4-11, 16-19, 28-31} and the same of the upper half (found by timing access
// patterns); the swizzles let each pass cover all 64 banks.  Rows past the
// matrix fall past the resource and chunks past K get an offset that does:
// both read as zero.
template <class T, bool BROWS, int (*SwA)(int), int (*SwB)(int)>
struct Stream {
  const GemmParams& p;
  const int wave, G, items;
  int item, left = 0;       // of the next step to fetch: its work item and the steps that are left of it
  unsigned k;               // and its first K
  unsigned lds0, chunk_a, chunk_b, row_k, next_k;
  __amdgpu_buffer_rsrc_t ra, rb;
  const char* sc_at;        // the block's scales: the first waves fetch A's, 64 rows each, the next ones B's
  unsigned sc_bytes, sc_voff;
  int64_t sc_inc;           // bytes from one block's scales to the next one's: past 32 bits for 2^30 rows
  unsigned base, va[T::kKB], vb[T::kKB];  // of the step being fetched

  __device__ __forceinline__ Stream(const GemmParams& p_, const uint8_t* lds, int lane, int wave_, int first)
      : p(p_), wave(wave_), G((int)gridDim.x), items(T::kParts ? p_.num_tiles * p_.splits : p_.num_tiles), item(first) {
    lds0 = lds_addr(lds);
    const int row = 8 * wave + (lane >> 3);
    chunk_a = (unsigned)((lane & 7) ^ SwA(row)) * 16;
    chunk_b = (unsigned)((lane & 7) ^ SwB(row)) * 16;
    row_k = (unsigned)row * (unsigned)p.K;
    next_k = 8u * T::kDmaWaves * (unsigned)p.K;
    const unsigned mine = (unsigned)(wave < T::kBM / 64 ? wave : wave - T::kBM / 64) * 64 + lane;
    sc_voff = 4 * mine;
    if (!BROWS && wave >= T::kBM / 64)  // one scale per 128 columns: lane j takes block j of the tile
      sc_voff = mine < (unsigned)((T::kBN + 127) / 128) ? 4u * mine * (unsigned)p.Kb : kOob;
    sc_inc = 4 * (wave < T::kBM / 64 ? (int64_t)p.M : BROWS ? (int64_t)p.N : 1);
    open();
  }
  __device__ __forceinline__ void open() {
    TileAt f{0, 0, 0};
    unsigned mv = 0, nv = 0;
    int at = 0;
    left = 0x7FFFFFFF;
    if (item < items) {
      f = tile_at<T>(p, item);
      mv = (unsigned)min(p.M - f.m0, T::kBM);
      nv = (unsigned)min(p.N - f.n0, T::kBN);
      const Part part = part_of<T>(p, item);
      at = T::kKB * part.at;
      left = part.count;
    }
    k = 128u * (unsigned)at;
    ra = make_rsrc(p.A + ((int64_t)f.l * p.M + f.m0) * p.K, mv * (unsigned)p.K);
    rb = make_rsrc(p.B + ((int64_t)f.l * p.N + f.n0) * p.K, nv * (unsigned)p.K);
    if (wave < T::kBM / 64) {
      sc_at = (const char*)(p.SA + ((int64_t)f.l * p.Kb + at) * p.M + f.m0);
      sc_bytes = 4 * mv;
    } else if constexpr (BROWS) {
      sc_at = (const char*)(p.SB + ((int64_t)f.l * p.Kb + at) * p.N + f.n0);
      sc_bytes = 4 * nv;
    } else {
      const int nb = min(p.Nb - f.n0 / 128, (T::kBN + 127) / 128);
      sc_at = (const char*)(p.SB + ((int64_t)f.l * p.Nb + f.n0 / 128) * p.Kb + at);
      sc_bytes = nv ? 4u * (unsigned)((nb - 1) * p.Kb + 1) : 0u;
    }
    if (wave >= T::kBM / 64 + T::kBN / 64) sc_bytes = 0;
  }
  __device__ __forceinline__ void begin(int stage) {
    base = lds0 + (unsigned)(stage * T::kStage) + 1024 * (unsigned)wave;
#pragma unroll
    for (int b = 0; b < T::kKB; ++b) {
      va[b] = k + 128 * b + chunk_a < (unsigned)p.K ? row_k + k + 128 * b + chunk_a : kOob;
      vb[b] = k + 128 * b + chunk_b < (unsigned)p.K ? row_k + k + 128 * b + chunk_b : kOob;
    }
  }
  // One of the step's kIssued DMA instructions (every wave issues as many, some on an empty resource, so that
  // waits can count them).
  __device__ __forceinline__ void one(int i) {
    const int b = i / T::kPerBlock, q = i % T::kPerBlock;
    const unsigned to = base + b * T::kBlock;
    if (q < T::kDa) dma16_at(ra, va[b] + q * next_k, to + 1024 * T::kDmaWaves * q);
    else if (q < T::kDa + T::kDb) dma16_at(rb, vb[b] + (q - T::kDa) * next_k, to + T::kOffB + 1024 * T::kDmaWaves * (q - T::kDa));
    else {
      const bool any = wave < T::kBM / 64 + T::kBN / 64;
      const bool in = T::kKB == 1 || k + 128 * b < (unsigned)p.K;  // a step's last blocks may lie past K
      dma4_at(make_rsrc(sc_at + (in ? b : 0) * sc_inc, in ? sc_bytes : 0u), sc_voff,
              any ? to + T::kOffSA - 768 * (unsigned)wave : lds0 + T::kStages * T::kStage);
    }
  }
  __device__ __forceinline__ void end() {
    sc_at += T::kKB * sc_inc;
    k += 128 * T::kKB;
    if (--left == 0) {
      item += G;
      open();
    }
  }
  __device__ __forceinline__ void all(int stage) {
    begin(stage);
#pragma unroll
    for (int q = 0; q < T::kIssued; ++q) one(q);
    end();
  }
};

// Waits until the DMA of this step is in LDS.  It was issued kStages - 1 steps ago; behind it in the queue of
// vector-memory instructions, which retires in order, are the DMA of the steps since and, in a tile's first
// steps, the kStores store instructions of the tile before (fixed in number where c_vec; else everything is
// waited for): those may still be on their way.
template <class T, int kStores>
__device__ __forceinline__ void wait_step(bool stores_fixed, bool stores_behind) {
  constexpr int kAhead = (T::kStages - 2) * T::kIssued;
  static_assert(kAhead + kStores <= 63, "vmcnt");
  if (!stores_behind) wait_vm<kAhead>();
  else if (stores_fixed) wait_vm<kAhead + kStores>();
  else wait_vm<0>();
}

// A wave that only moves operands: it meets the computing waves at their barrier of every step, when its DMA of that
// step has landed, and then refills the stage they have left.  A wave whose DMA instruction finds the queue full
// issues nothing until it drains, which these waves can afford.
template <class T, class S>
__device__ __forceinline__ void produce(const GemmParams& p, S& in, int item, int items) {
  for (int s = 0; s < T::kStages - 1; ++s) in.all(s);
  int stage = 0;
  for (; item < items; item += (int)gridDim.x)
    for (int n = part_of<T>(p, item).count; n > 0; --n) {
      wait_vm<(T::kStages - 2) * T::kIssued>();
      barrier();
      in.all(stage == 0 ? T::kStages - 1 : stage - 1);
      stage = stage + 1 == T::kStages ? 0 : stage + 1;
    }
  wait_vm<0>();  // no DMA may land after the workgroup's LDS is handed on
}

__device__ __forceinline__ int first_tile_of(const GemmParams& p) {
  const int G = (int)gridDim.x, b = (int)blockIdx.x;
  return p.xcd_remap ? (b & 7) * (G >> 3) + (b >> 3) : b;
}

// --- 16-bit C: the 8-bit matrix cores ---------------------------------------------
//
// v_mfma_f32_16x16x128_f8f6f4 contracts a whole block in one instruction of 32
// cycles, under which the four multiply-adds per lane of an earlier one run.
// VALU instructions reach only ordinary registers, so the accumulators live
// there and a wave holds 128 x 64 of them, eight waves a 256 x 256 tile.
// 8192 x 24576 x 1536 takes 290 to 300 us (2.1 PFLOP/s), of which the C stores
// are 43, 8192^3 460 (2.4), with the matrix cores busy 56% and 63% of the cycles at
// a clock of 1.7 to 2 GHz and no LDS bank conflicts.
//
// B is the MFMA's first operand: lane (r = lane % 16, g = lane / 16) owns output
// row r of a 16-row block and the MFMA's columns 4g .. 4g + 3.  Which tile
// column each of its 16 is, is free: MFMA nt takes columns
// 32 (nt / 2) + 8 (r / 4) + 4 (nt % 2) + r % 4, so a lane's results of two MFMAs
// are 8 consecutive columns; at the end rows r and r ^ 1 exchange halves, and a
// store instruction writes whole 128-byte rows.  A lane's 32 bytes of K are
// chunks g and g + 4 of the row, in A and B alike.
__device__ __forceinline__ int swizzle_a16(int row) { return (row >> 1) & 7; }
__device__ __forceinline__ int swizzle_b16(int row) { return ((row >> 1) & 1) | ((row >> 2) & 6); }

template <class T, int FA, int FB, int CT, bool BROWS>
__global__ __launch_bounds__(64 * T::kAllWaves, (T::kAllWaves + 3) / 4) void block128_tile_kernel(GemmParams p) {
  static_assert(CT != 0, "16-bit C");
  constexpr int kMt = T::kTM / 16, kNt = T::kTN / 16, kPairs = kNt / 2;
  constexpr int kStores = kMt * kPairs;                     // C store instructions per lane and tile
  constexpr int kRows = T::kKB * kMt;                        // rows of MFMAs in a step
  constexpr int kPerRow = (T::kIssued + kRows - 2) / (kRows - 1);  // DMA instructions between two of them
  __shared__ __attribute__((aligned(1024))) uint8_t lds[T::kLds];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  const int wm = wave / T::kWn, wn = wave % T::kWn;
  const int r = lane & 15, g = lane >> 4;
  const int G = (int)gridDim.x;
  int item = first_tile_of(p);
  const int items = T::kParts ? p.num_tiles * p.splits : p.num_tiles;
  Stream<T, BROWS, swizzle_a16, swizzle_b16> in(p, lds, lane, T::kProducers ? wave - T::kWaves : wave, item);
  if constexpr (T::kProducers > 0) {
    if (wave >= T::kWaves) {
      produce<T>(p, in, item, items);
      return;
    }
  }

  const int a_row = T::kTM * wm + r, b_row = T::kTN * wn + 8 * (r >> 2) + (r & 3);
  const unsigned a_off = (unsigned)(a_row * 128 + 16 * (g ^ swizzle_a16(a_row)));
  const unsigned b_off = (unsigned)(T::kOffB + b_row * 128 + 16 * (g ^ swizzle_b16(b_row)));
  auto frag = [&](const uint8_t* lo_at, const uint8_t* hi_at, int imm) {
    const v4u lo = *reinterpret_cast<const v4u*>(lo_at + imm);
    const v4u hi = *reinterpret_cast<const v4u*>(hi_at + imm);
    return (v8i){(int)lo[0], (int)lo[1], (int)lo[2], (int)lo[3], (int)hi[0], (int)hi[1], (int)hi[2], (int)hi[3]};
  };

  if constexpr (T::kProducers == 0)
    for (int s = 0; s < T::kStages - 1; ++s) in.all(s);
  int step = 0, stage = 0, count = item < items ? part_of<T>(p, item).count : 0;
  bool stored = false;
  const v4f zero = {0.f, 0.f, 0.f, 0.f};
  v4f acc[kMt][kNt];
  while (item < items) {
    if constexpr (T::kProducers == 0) wait_step<T, kStores>(p.c_vec, stored && step < T::kStages - 1);
    barrier();
    const uint8_t* st = lds + stage * T::kStage;
    const uint8_t *a_lo = st + a_off, *a_hi = st + (a_off ^ 64), *b_lo = st + b_off, *b_hi = st + (b_off ^ 64);
    const float* ssa = reinterpret_cast<const float*>(st + T::kOffSA) + a_row;
    const float* ssb = reinterpret_cast<const float*>(st + T::kOffSB) + (BROWS ? T::kTN * wn + 8 * g : T::kTN * wn / 128);
    // row t of MFMAs is row t % kMt of block t / kMt; A's fragments are read two rows ahead of their use
    auto a_frag = [&](int t) { return frag(a_lo, a_hi, t / kMt * T::kBlock + 2048 * (t % kMt)); };
    v8i b[T::kKB][kNt], a[3];
    a[0] = a_frag(0);
#pragma unroll
    for (int nt = 0; nt < kNt; ++nt) b[0][nt] = frag(b_lo, b_hi, 128 * (32 * (nt >> 1) + 4 * (nt & 1)));
    a[1] = a_frag(1);
    float sa[T::kKB][kMt];
    v4f sb[T::kKB][BROWS ? kNt : 1];
#pragma unroll
    for (int kb = 0; kb < T::kKB; ++kb) {
      if (kb > 0) {
#pragma unroll
        for (int nt = 0; nt < kNt; ++nt) b[kb][nt] = frag(b_lo, b_hi, kb * T::kBlock + 128 * (32 * (nt >> 1) + 4 * (nt & 1)));
      }
#pragma unroll
      for (int mt = 0; mt < kMt; ++mt) sa[kb][mt] = ssa[kb * (T::kBlock / 4) + 16 * mt];
      if constexpr (BROWS) {
#pragma unroll
        for (int nt = 0; nt < kNt; ++nt)
          sb[kb][nt] = *reinterpret_cast<const v4f*>(ssb + kb * (T::kBlock / 4) + 32 * (nt >> 1) + 4 * (nt & 1));
      } else {
        sb[kb][0][0] = ssb[kb * (T::kBlock / 4)];
      }
    }
    if (step == 0) {
#pragma unroll
      for (int mt = 0; mt < kMt; ++mt)
#pragma unroll
        for (int nt = 0; nt < kNt; ++nt) acc[mt][nt] = zero;
    }
    v4f part[kNt];
    auto fold = [&](int t, int nt) {
      const int kb = t / kMt, mt = t % kMt;
      const v4f pt = part[nt];
      const float s0 = BROWS ? sa[kb][mt] : sa[kb][mt] * sb[kb][0][0];
#pragma unroll
      for (int e = 0; e < 4; ++e) acc[mt][nt][e] = __builtin_fmaf(pt[e], BROWS ? s0 * sb[kb][nt][e] : s0, acc[mt][nt][e]);
      // keeps the multiply-adds here: moved past the step's branches, all parts would have to be kept
      asm volatile("" : "+v"(acc[mt][nt]));
    };
    // Each MFMA's result goes into the accumulators right before the MFMA of the next row that overwrites it, one
    // between two MFMAs: a wave that issues a row's MFMAs and then all its multiply-adds leaves the matrix core idle
    // under most of them (8192 x 24576 x 1536: 319 -> 295 us, 1024 x 4096 x 7168: 41.3 -> 36.5 us).
    // The stage the step before used takes the DMA that is furthest ahead, issued between the rows of MFMAs.
    if constexpr (T::kProducers == 0) in.begin(stage == 0 ? T::kStages - 1 : stage - 1);
#pragma unroll
    for (int t = 0; t < kRows; ++t) {
#pragma unroll
      for (int nt = 0; nt < kNt; ++nt) {
        if (t > 0) fold(t - 1, nt);
        part[nt] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(b[t / kMt][nt], a[t % 3], zero, FB, FA, 0, 0, 0, 0);
        if (T::kProducers > 0 && nt == 0 && t + 2 < kRows) a[(t + 2) % 3] = a_frag(t + 2);
        __builtin_amdgcn_sched_barrier(0);
      }
      if (T::kProducers == 0) {
        if (t + 2 < kRows) a[(t + 2) % 3] = a_frag(t + 2);
#pragma unroll
        for (int q = 0; q < T::kIssued; ++q)
          if (q / kPerRow == t) in.one(q);
        __builtin_amdgcn_sched_barrier(0);
      }
    }
#pragma unroll
    for (int nt = 0; nt < kNt; ++nt) fold(kRows - 1, nt);
    if constexpr (T::kProducers == 0) in.end();
    stage = stage + 1 == T::kStages ? 0 : stage + 1;

    if (++step == count) {
      step = 0;
      stored = true;
      const TileAt at = tile_at<T>(p, item);
      const int rows = min(p.M - at.m0, T::kBM);
      if (T::kParts && p.splits > 1) {
        // a part's sums, four columns at a time (ldw is a multiple of 4)
        float* w = p.sums + (((int64_t)(item / p.num_tiles) * p.L + at.l) * p.M + at.m0) * p.ldw + at.n0;
#pragma unroll
        for (int mt = 0; mt < kMt; ++mt)
#pragma unroll
          for (int nt = 0; nt < kNt; ++nt) {
            const int m = a_row + 16 * mt, n = T::kTN * wn + 32 * (nt >> 1) + 8 * g + 4 * (nt & 1);
            if (m < rows && at.n0 + n < p.ldw) *reinterpret_cast<v4f*>(w + (int64_t)m * p.ldw + n) = acc[mt][nt];
          }
        item += G;
        count = item < items ? part_of<T>(p, item).count : 0;
        continue;
      }
      item += G;
      count = item < items ? part_of<T>(p, item).count : 0;
      using E = elem_t<CT>;
      E* c = static_cast<E*>(p.C) + ((int64_t)at.l * p.M + at.m0) * p.ldc + at.n0;
      const bool odd = (r & 1) != 0;
      // stores 8 columns to a call; non-temporal: C is not read here, and keeping it would push A and B out of the
      // caches (8192 x 24576 x 1536: 341 -> 318 us)
      auto put = [&](auto store) {
#pragma unroll
        for (int mt = 0; mt < kMt; ++mt) {
          v4u u[kPairs];
#pragma unroll
          for (int h = 0; h < kPairs; ++h) {
            const v8f v = __builtin_shufflevector(acc[mt][2 * h], acc[mt][2 * h + 1], 0, 1, 2, 3, 4, 5, 6, 7);
            if constexpr (CT == 1) u[h] = __builtin_bit_cast(v4u, __builtin_convertvector(v, v8bf));
            else u[h] = __builtin_bit_cast(v4u, __builtin_convertvector(v, v8h));
          }
          const int m = a_row + 16 * mt, n = T::kTN * wn + 8 * g;
          if constexpr (kPairs % 2 == 0) {
#pragma unroll
            for (int h = 0; h < kPairs; h += 2) {
              // even lanes take columns 0..31 of their row and the next, odd lanes 32..63 of theirs and the one before
              v4u got, mine;
#pragma unroll
              for (int w = 0; w < 4; ++w) {
                got[w] = (unsigned)__builtin_amdgcn_mov_dpp((int)(odd ? u[h][w] : u[h + 1][w]), 0xB1, 0xF, 0xF, true);
                mine[w] = odd ? u[h + 1][w] : u[h][w];
              }
              const int nn = n + 32 * h + (odd ? 32 : 0);
              v4u first, second;
#pragma unroll
              for (int w = 0; w < 4; ++w) {
                first[w] = odd ? got[w] : mine[w];
                second[w] = odd ? mine[w] : got[w];
              }
              store(first, m & ~1, nn);
              store(second, m | 1, nn);
            }
          } else {
#pragma unroll
            for (int h = 0; h < kPairs; ++h) store(u[h], m, n + 32 * h);
          }
        }
      };
      if (p.c_vec) {
        // N and ldc are multiples of 8 here: a lane's 8 columns lie inside or outside N together
        int ldc = (int)p.ldc;
        // with 16 scales more to a lane, the stores' offsets are made here, not kept in registers through the K loop
        if constexpr (BROWS) asm volatile("" : "+s"(ldc));
        const __amdgpu_buffer_rsrc_t rc = make_rsrc(c, 2u * (unsigned)((int64_t)(rows - 1) * ldc + min(p.N - at.n0, T::kBN)));
        put([&](const v4u& u, int m, int n) {
          const unsigned off = m < rows && at.n0 + n < p.N ? 2u * (unsigned)(m * ldc + n) : kOob;
          __builtin_amdgcn_raw_buffer_store_b128(u, rc, (int)off, 0, 2);
        });
      } else {
        // 16-byte stores at any alignment but for the last columns of a row (8192 x 8191 x 1024: 184 us element by
        // element)
        int64_t ldc = p.ldc;
        asm volatile("" : "+s"(ldc));  // as above
        put([&](const v4u& u, int m, int n) {
          const int left = p.N - at.n0 - n;
          E* to = c + m * ldc + n;
          if (m < rows && left >= 8) {
            __builtin_nontemporal_store(u, reinterpret_cast<v4u_at2*>(to));
          } else if (m < rows) {
#pragma unroll
            for (int e = 0; e < 7; ++e)
              if (e < left) to[e] = __builtin_bit_cast(E, (unsigned short)(u[e >> 1] >> (16 * (e & 1))));
          }
        });
      }
    }
  }
  wait_vm<0>();  // no DMA may land after the workgroup's LDS is handed on
}

// --- float32 C: codes widened to bfloat16 -----------------------------------------
//
// v_mfma_f32_32x32x16_bf16 takes products of bfloat16 exactly and adds them in
// float32; every 8-bit code is a bfloat16 number.  A wave holds 64 x 64 outputs
// in 2 x 2 blocks of 32 x 32, whose 8 MFMAs per scale block chain from zero;
// codes are widened under the MFMAs of the slice before.  8192^3 takes 910 to
// 950 us (1.2 PFLOP/s); without widening and multiply-adds it would be 800, what
// a bfloat16 product takes: their cost is power.
//
// B is the first operand: lane (r = lane % 32, h = lane / 32) owns output row r
// and the MFMA's rows 8 q + 4 h + i, q, i < 4, which are tile columns
// 16 h + 4 q + i: 16 consecutive floats.  At the end four neighbouring rows
// exchange quads, and a store instruction writes whole 128-byte rows.
__device__ __forceinline__ int swizzle_a32(int row) { return (row >> 1) & 7; }
__device__ __forceinline__ int swizzle_b32(int row) { return ((row >> 1) & 1) | ((row >> 3) & 2) | (row & 4); }

template <class T, int FA, int FB, bool BROWS>
__global__ __launch_bounds__(64 * T::kAllWaves, (T::kAllWaves + 3) / 4) void block128_exact_kernel(GemmParams p) {
  constexpr int kMt = T::kTM / 32, kNt = T::kTN / 32;  // a wave's MFMA blocks
  constexpr int kStores = 4 * kMt * kNt;               // C store instructions per lane and tile
  __shared__ __attribute__((aligned(1024))) uint8_t lds[T::kLds];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  const int wm = wave / T::kWn, wn = wave % T::kWn;
  const int r = lane & 31, h = lane >> 5;
  const int G = (int)gridDim.x;
  int item = first_tile_of(p);
  const int items = T::kParts ? p.num_tiles * p.splits : p.num_tiles;
  Stream<T, BROWS, swizzle_a32, swizzle_b32> in(p, lds, lane, T::kProducers ? wave - T::kWaves : wave, item);
  if constexpr (T::kProducers > 0) {
    if (wave >= T::kWaves) {
      produce<T>(p, in, item, items);
      return;
    }
  } else {
    for (int s = 0; s < T::kStages - 1; ++s) in.all(s);
  }

  const int a_row = T::kTM * wm + r, b_row = T::kTN * wn + 16 * ((r >> 2) & 1) + 4 * (r >> 3) + (r & 3);
  // a lane's chunk c of K (c = 0..3) is 2c + h of the row: at 32 c ^ its offset
  const unsigned a_off = (unsigned)(a_row * 128 + 16 * (h ^ swizzle_a32(a_row)));
  const unsigned b_off = (unsigned)(T::kOffB + b_row * 128 + 16 * (h ^ swizzle_b32(b_row)));

  int step = 0, stage = 0, count = item < items ? part_of<T>(p, item).count : 0;
  bool stored = false;
  v16f acc[kMt][kNt];
  while (item < items) {
    if constexpr (T::kProducers == 0) {
      wait_step<T, kStores>(p.c_vec && !p.accumulate, stored && step < T::kStages - 1);
    }
    barrier();
    if constexpr (T::kProducers == 0) in.begin(stage == 0 ? T::kStages - 1 : stage - 1);
    const uint8_t* st = lds + stage * T::kStage;
    if (step == 0) {
#pragma unroll
      for (int t = 0; t < kMt * kNt; ++t)
#pragma unroll
        for (int e = 0; e < 16; ++e) acc[t / kNt][t % kNt][e] = 0.f;
    }
#pragma unroll
    for (int kb = 0; kb < T::kKB; ++kb) {
      const uint8_t* sk = st + kb * T::kBlock;
      v4u ra[2][kMt], rb[2][kNt];  // raw chunks: this one's and the next one's
      auto read = [&](int c) {
#pragma unroll
        for (int t = 0; t < kMt; ++t) ra[c & 1][t] = *reinterpret_cast<const v4u*>(sk + (a_off ^ (32 * c)) + 4096 * t);
#pragma unroll
        for (int t = 0; t < kNt; ++t) rb[c & 1][t] = *reinterpret_cast<const v4u*>(sk + (b_off ^ (32 * c)) + 4096 * t);
      };
      v16f part[kMt][kNt];
      read(0);
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        if (c < 3) read(c + 1);
#pragma unroll
        for (int s = 0; s < 2; ++s) {
          v8bf a[kMt], b[kNt];
#pragma unroll
          for (int t = 0; t < kMt; ++t) a[t] = cvt8<FA>(ra[c & 1][t][2 * s], ra[c & 1][t][2 * s + 1], 1.f);
#pragma unroll
          for (int t = 0; t < kNt; ++t) b[t] = cvt8<FB>(rb[c & 1][t][2 * s], rb[c & 1][t][2 * s + 1], 1.f);
#pragma unroll
          for (int t = 0; t < kMt * kNt; ++t) {
            v16f from = part[t / kNt][t % kNt];
            if (c == 0 && s == 0) {
#pragma unroll
              for (int e = 0; e < 16; ++e) from[e] = 0.f;
            }
            part[t / kNt][t % kNt] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(b[t % kNt], a[t / kNt], from, 0, 0, 0);
          }
        }
        if constexpr (T::kProducers == 0) {
#pragma unroll
          for (int q = 0; q < T::kPerBlock; ++q)
            if (q / ((T::kPerBlock + 2) / 3) == c) in.one(kb * T::kPerBlock + q);
        }
      }
      const float* ssa = reinterpret_cast<const float*>(sk + T::kOffSA) + a_row;
      const float* ssb = reinterpret_cast<const float*>(sk + T::kOffSB) + (BROWS ? T::kTN * wn + 16 * h : T::kTN * wn / 128);
#pragma unroll
      for (int n = 0; n < kNt; ++n) {
        v4f sb[4];
#pragma unroll
        for (int q = 0; q < (BROWS ? 4 : 1); ++q) {
          if constexpr (BROWS) sb[q] = *reinterpret_cast<const v4f*>(ssb + 32 * n + 4 * q);
          else sb[0][0] = ssb[0];
        }
#pragma unroll
        for (int m = 0; m < kMt; ++m) {
          const float sa = ssa[32 * m];
#pragma unroll
          for (int e = 0; e < 16; ++e)
            acc[m][n][e] = __builtin_fmaf(part[m][n][e], sa * (BROWS ? sb[e >> 2][e & 3] : sb[0][0]), acc[m][n][e]);
        }
      }
    }
    if constexpr (T::kProducers == 0) in.end();
    stage = stage + 1 == T::kStages ? 0 : stage + 1;

    if (++step == count) {
      step = 0;
      stored = true;
      const TileAt at = tile_at<T>(p, item);
      // a part's sums go to the workspace, which the host has described as C: (splits, L, M, ldc)
      const int l = at.l + (T::kParts && p.splits > 1 ? item / p.num_tiles * p.L : 0);
      item += G;
      count = item < items ? part_of<T>(p, item).count : 0;
      const int rows = min(p.M - at.m0, T::kBM);
      float* c = static_cast<float*>(p.C) + ((int64_t)l * p.M + at.m0) * p.ldc + at.n0;
      // finish(v, m, n): quad q of v is columns n .. n + 3 of row m + q
      auto quads = [&](auto finish) {
#pragma unroll
        for (int m = 0; m < kMt; ++m)
#pragma unroll
          for (int n = 0; n < kNt; ++n) {
            // quad q of row r (r % 4 = j) goes to lane j' = q of the four, as its quad of row j: a 4 x 4
            // transposition in two exchanges, with lane ^ 1 and lane ^ 2
            float v[4][4];
#pragma unroll
            for (int e = 0; e < 16; ++e) v[e >> 2][e & 3] = acc[m][n][e];
#pragma unroll
            for (int s = 1; s < 4; s <<= 1) {
              const bool up = (r & s) != 0;
#pragma unroll
              for (int q = 0; q < 4; ++q) {
                if (q & s) continue;
#pragma unroll
                for (int w = 0; w < 4; ++w) {
                  const float x = v[q][w], y = v[q | s][w];
                  const int give = __builtin_bit_cast(int, up ? x : y);
                  const float got = __builtin_bit_cast(float, s == 1 ? __builtin_amdgcn_mov_dpp(give, 0xB1, 0xF, 0xF, true)
                                                                     : __builtin_amdgcn_mov_dpp(give, 0x4E, 0xF, 0xF, true));
                  v[q][w] = up ? got : x;
                  v[q | s][w] = up ? y : got;
                }
              }
            }
            finish(v, (a_row & ~3) + 32 * m, T::kTN * wn + 32 * n + 16 * h + 4 * (r & 3));
          }
      };
      if (p.c_vec) {
        // N and ldc are multiples of 4 here
        const __amdgpu_buffer_rsrc_t rc = make_rsrc(c, 4u * (unsigned)((int64_t)(rows - 1) * p.ldc + min(p.N - at.n0, T::kBN)));
        quads([&](float(&v)[4][4], int m, int n) {
          unsigned off[4];
#pragma unroll
          for (int q = 0; q < 4; ++q) off[q] = m + q < rows && at.n0 + n < p.N ? 4u * (unsigned)((m + q) * (int)p.ldc + n) : kOob;
          if (p.accumulate) {
            v4u old[4];
#pragma unroll
            for (int q = 0; q < 4; ++q) old[q] = __builtin_amdgcn_raw_buffer_load_b128(rc, (int)off[q], 0, 0);
#pragma unroll
            for (int q = 0; q < 4; ++q)
#pragma unroll
              for (int w = 0; w < 4; ++w) v[q][w] += __uint_as_float(old[q][w]);
          }
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const v4u out = {__float_as_uint(v[q][0]), __float_as_uint(v[q][1]), __float_as_uint(v[q][2]), __float_as_uint(v[q][3])};
            __builtin_amdgcn_raw_buffer_store_b128(out, rc, (int)off[q], 0, 2);
          }
        });
      } else {
        // 16-byte accesses at any alignment but for the last columns of a row (8192 x 8191 x 1024: 396 us element by
        // element)
        quads([&](float(&v)[4][4], int m, int n) {
          const int left = p.N - at.n0 - n;
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            float* to = c + (int64_t)(m + q) * p.ldc + n;
            if (m + q < rows && left >= 4) {
              if (p.accumulate) {
                const v4u old = *reinterpret_cast<const v4u_at4*>(to);
#pragma unroll
                for (int w = 0; w < 4; ++w) v[q][w] += __uint_as_float(old[w]);
              }
              const v4u out = {__float_as_uint(v[q][0]), __float_as_uint(v[q][1]), __float_as_uint(v[q][2]), __float_as_uint(v[q][3])};
              __builtin_nontemporal_store(out, reinterpret_cast<v4u_at4*>(to));
            } else if (m + q < rows) {
#pragma unroll
              for (int w = 0; w < 3; ++w)
                if (w < left) to[w] = (p.accumulate ? to[w] : 0.f) + v[q][w];
            }
          }
        });
      }
    }
  }
  if constexpr (T::kProducers == 0) wait_vm<0>();
}

// --- few rows of A -----------------------------------------------------------------
//
// Up to 16 MT rows.  B is read once, straight from memory into the MFMA's
// registers: a workgroup takes COLS columns, its W waves every W-th block of K,
// and the waves' sums meet in LDS in a fixed order.  B's bytes bound it, so a
// wave asks for its next block before it uses this one (1 x 7168 x 2048: 4.9 us,
// 3 TB/s; 4 x 7168 x 7168: 11.0 us, 4.7 TB/s).  More waves or more blocks ahead
// change nothing: a compute unit reads 26 to 35 B/ns.  Rows and columns past
// the matrix repeat the last one and are not stored.  Lane (r, g) owns row r and
// columns 4g .. 4g + 3 of 16; a 16-bit C takes the 8-bit matrix cores, a float32
// C the widened codes, as in the tile kernels.
constexpr int kRowWaves = 8;

template <int FA, int FB, int CT, bool BROWS, int COLS, int MT>
__global__ __launch_bounds__(64 * kRowWaves) void block128_rows_kernel(GemmParams p) {
  constexpr int W = kRowWaves;
  constexpr int NT = COLS / 16;
  __shared__ float lds[W][16 * MT][16 * NT + 4];
  const int lane = threadIdx.x & 63, r = lane & 15, g = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  const int item = p.first + (int)blockIdx.x, l = item / p.tilesN, n0 = item % p.tilesN * COLS;
  const uint8_t* a[MT];
  const float* sa[MT];
#pragma unroll
  for (int s = 0; s < MT; ++s) {
    const int m = min(16 * s + r, p.M - 1);
    a[s] = p.A + ((int64_t)l * p.M + m) * p.K + 16 * g;
    sa[s] = p.SA + (int64_t)l * p.Kb * p.M + m;
  }
  const uint8_t* b[NT];
  const float* sb[NT];
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    b[t] = p.B + ((int64_t)l * p.N + min(n0 + 16 * t + r, p.N - 1)) * p.K + 16 * g;
    sb[t] = BROWS ? p.SB + (int64_t)l * p.Kb * p.N : p.SB + ((int64_t)l * p.Nb + min(n0 + 16 * t, p.N - 1) / 128) * p.Kb;
  }
  struct Block {
    v4u a[MT][2], b[NT][2];
    float sa[MT];
    v4f sb[NT];
  };
  auto load = [&](Block& k, int j) {
    // chunks g and g + 4 of the block; those past K repeat the row's last and are zeroed before use
    const int64_t lo = (int64_t)min(128 * j, p.K - 16 - 16 * g), hi = (int64_t)min(128 * j + 64, p.K - 16 - 16 * g);
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      k.b[t][0] = *reinterpret_cast<const v4u*>(b[t] + lo);
      k.b[t][1] = *reinterpret_cast<const v4u*>(b[t] + hi);
    }
#pragma unroll
    for (int s = 0; s < MT; ++s) {
      k.a[s][0] = *reinterpret_cast<const v4u*>(a[s] + lo);
      k.a[s][1] = *reinterpret_cast<const v4u*>(a[s] + hi);
      k.sa[s] = sa[s][(int64_t)j * p.M];
    }
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      if constexpr (BROWS) {
#pragma unroll
        for (int e = 0; e < 4; ++e) k.sb[t][e] = sb[t][(int64_t)j * p.N + min(n0 + 16 * t + 4 * g + e, p.N - 1)];
      } else {
        k.sb[t][0] = sb[t][j];
      }
    }
  };
  const v4f zero = {0.f, 0.f, 0.f, 0.f};
  v4f acc[MT][NT];
#pragma unroll
  for (int s = 0; s < MT; ++s)
#pragma unroll
    for (int t = 0; t < NT; ++t) acc[s][t] = zero;
  auto multiply = [&](Block& k, int j) {
    if (128 * j + 128 > p.K) {
      const v4u none = {0, 0, 0, 0};
      const bool lo_in = 128 * j + 16 * g < p.K, hi_in = 128 * j + 64 + 16 * g < p.K;
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        k.b[t][0] = lo_in ? k.b[t][0] : none;
        k.b[t][1] = hi_in ? k.b[t][1] : none;
      }
#pragma unroll
      for (int s = 0; s < MT; ++s) {
        k.a[s][0] = lo_in ? k.a[s][0] : none;
        k.a[s][1] = hi_in ? k.a[s][1] : none;
      }
    }
#pragma unroll
    for (int i = 0; i < MT * NT; ++i) {
      const int s = i / NT, t = i % NT;
      v4f part = zero;
      if constexpr (CT != 0) {
        struct Bytes32 { v4u lo, hi; };
        part = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(__builtin_bit_cast(v8i, (Bytes32{k.b[t][0], k.b[t][1]})),
                                                                __builtin_bit_cast(v8i, (Bytes32{k.a[s][0], k.a[s][1]})), zero,
                                                                FB, FA, 0, 0, 0, 0);
      } else {
#pragma unroll
        for (int q = 0; q < 4; ++q)
          part = __builtin_amdgcn_mfma_f32_16x16x32_bf16(cvt8<FB>(k.b[t][q >> 1][2 * (q & 1)], k.b[t][q >> 1][2 * (q & 1) + 1], 1.f),
                                                         cvt8<FA>(k.a[s][q >> 1][2 * (q & 1)], k.a[s][q >> 1][2 * (q & 1) + 1], 1.f),
                                                         part, 0, 0, 0);
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) acc[s][t][e] = __builtin_fmaf(part[e], k.sa[s] * k.sb[t][BROWS ? e : 0], acc[s][t][e]);
    }
  };
  if (wave < p.Kb) {
    Block k0, k1;
    load(k0, wave);
    for (int j = wave;;) {
      const bool more = j + W < p.Kb;
      if (more) load(k1, j + W);
      multiply(k0, j);
      if (!more) break;
      j += W;
      const bool again = j + W < p.Kb;
      if (again) load(k0, j + W);
      multiply(k1, j);
      if (!again) break;
      j += W;
    }
  }
#pragma unroll
  for (int s = 0; s < MT; ++s)
#pragma unroll
    for (int t = 0; t < NT; ++t) *reinterpret_cast<v4f*>(&lds[wave][16 * s + r][16 * t + 4 * g]) = acc[s][t];
  __syncthreads();
  elem_t<CT>* c = static_cast<elem_t<CT>*>(p.C) + (int64_t)l * p.M * p.ldc + n0;
  for (int i = threadIdx.x; i < p.M * COLS; i += 64 * W) {
    const int row = i / COLS, n = i % COLS;
    float sum = 0.f;
#pragma unroll
    for (int w = 0; w < W; ++w) sum += lds[w][row][n];
    if (n0 + n < p.N) {
      elem_t<CT>* to = c + (int64_t)row * p.ldc + n;
      if (CT == 0 && p.accumulate) sum += (float)*to;
      *to = (elem_t<CT>)sum;
    }
  }
}

// C from the parts' sums, four columns to a thread, parts added in order.
template <int CT>
__global__ __launch_bounds__(256) void block128_sum_kernel(GemmParams p, int splits) {
  const int quads = p.ldw / 4;
  const int64_t rows = (int64_t)p.L * p.M, all = rows * quads, stride = (int64_t)gridDim.x * 256;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < all; i += stride) {
    const int64_t row = i / quads;
    const int n = 4 * (int)(i - row * quads);
    const float* w = p.sums + row * p.ldw + n;
    v4f sum = *reinterpret_cast<const v4f*>(w);
    for (int s = 1; s < splits; ++s) sum += *reinterpret_cast<const v4f*>(w + s * rows * p.ldw);
    elem_t<CT>* c = static_cast<elem_t<CT>*>(p.C) + row * p.ldc + n;
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (n + e < p.N) c[e] = (elem_t<CT>)(CT == 0 && p.accumulate ? (float)c[e] + sum[e] : sum[e]);
  }
}

// C = 0: an empty sum.
template <int CT>
__global__ __launch_bounds__(256) void block128_zero_kernel(GemmParams p) {
  const int64_t all = (int64_t)p.L * p.M * p.N, stride = (int64_t)gridDim.x * 256;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < all; i += stride)
    static_cast<elem_t<CT>*>(p.C)[i / p.N * p.ldc + i % p.N] = (elem_t<CT>)0.f;
}

}  // namespace b128
}  // namespace mxg
