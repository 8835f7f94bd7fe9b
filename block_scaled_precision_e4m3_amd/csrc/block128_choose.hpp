// Which kernel a block-128 product takes: a rule on sizes and types alone, so that the workspace it needs is known
// without a device.
#pragma once

#include <stdint.h>

#include <algorithm>
#include <cmath>

#include "host_checks.hpp"

namespace mxg {
namespace b128 {

using host::cdiv;

// Which kernel, tile and division of K.  rows: a kernel for few rows of A.
//
// Tiles: the time in microseconds of a tile size is taken as
//   rounds of work items over the compute units x (blocks of K x block x (1 - idle x gain) + end)
// where idle is the share of compute units without work (the larger tiles, which
// power bounds, gain by it; the smaller ones wait for memory), and, where K is
// divided, the second kernel that adds the parts up.  block and end were measured on MI355X, one
// size forced at a time.  16-bit C, the best and its neighbours:
//   128x7168x2048     64 x 64 7.1     64 x 128 8.4   128 x 128 11.1
//   512x4096x7168     64 x 128 21.7   64 x 64 27.7   128 x 128 28.6
//   1024x4096x7168    128 x 128 36.5  64 x 128 40.9  128 x 256 54.1
//   2048x4096x4096    128 x 256 38.6  128 x 128 46.6 256 x 256 48.5
//   4096x4096x4096    256 x 256 63.3  128 x 256 74.9 128 x 128 81.5
// float32 C:
//   128x7168x2048     64 x 64 10.1    64 x 128 12.4  128 x 128 17.0
//   512x4096x7168     64 x 128 36.4   64 x 64 44.1   128 x 128 47.5
//   4000x7168x2048    128 x 128 115.4 128 x 256 121.3 64 x 128 139.9
//   2048x4096x4096    128 x 256 61.6  128 x 128 64.1 64 x 128 77.1
// K is divided only where tiles leave compute units idle: 64x1024x7168 in 4
// parts 10.3 us, in one 14.8; 128x2048x7168 12.7 and 14.3; 256x1024x4096 10.5
// and 9.9, with a float32 C 12.7 and 15.4.
struct Choice {
  int rows;                // columns per workgroup of the rows kernel, 0: tiles
  int bm, bn, kb, splits;  // tile; blocks of K per step; parts of K
};

constexpr int kUnits = 256;  // compute units: the choice, and with it the workspace, must not need a device

struct Size {
  int bm, bn, kb;
  bool divides;  // its kernel can take part of K
  double block, end, gain;
};
constexpr Size kSizes[2][5] = {{{64, 64, 2, true, 0.215, 0.5, 0.0},
                                       {64, 128, 2, true, 0.335, 0.7, 0.0},
                                       {128, 128, 1, false, 0.64, 1.0, 0.3},
                                       {128, 256, 1, false, 1.08, 2.0, 0.3},
                                       {256, 256, 1, false, 1.8, 3.0, 0.3}},
                                      {{64, 64, 2, true, 0.355, 0.8, 0.0},
                                       {64, 128, 2, true, 0.585, 1.0, 0.0},
                                       {128, 128, 2, true, 0.97, 1.3, 0.3},
                                       {128, 256, 1, false, 1.85, 2.0, 0.3}}};

inline Choice choose(int64_t M, int64_t N, int64_t K, int64_t L, bool exact) {
  // a rows workgroup reads A once for its columns, so more columns are better as long as they leave enough
  // workgroups (7168 columns: 32 at a time 4.9 us, 16 5.1 us; 4096: 7.3 and 5.8 us; K = 2048 and 4096)
  // Up to 32 rows too, unless there are more workgroups than compute units (32x24576x1536: 11.7 us, tiles 9.7) or, for
  // a 16-bit C, K is long (32x7168x2048: 6.9 us, tiles 7.0; 32x6144x4096: 10.8 and 10.1; float32 C: 7.3 and 9.8, 11.3
  // and 14.0).  Where the two cross moves with rows and columns: 32 rows at K = 2560 from 6144 columns on and past 4096
  // below that (32x4096x4096: 8.9 us, tiles 10.0), 24 rows at 3328, 17 rows past 6144 (17x7168x4096: 9.4 and 10.0);
  // 2048 is on the safe side of all of them.  With 64 rows tiles are as fast or faster (64x7168x2048: 9.2 us, tiles 7.2; float32 C: 9.5 and 9.6).
  if (M <= 16 || (M <= 32 && L * cdiv(N, 32) <= kUnits && (exact || K <= 2048))) return {L * cdiv(N, 32) >= kUnits * 3 / 4 ? 32 : 16, 16, 0, 1, 1};
  const int64_t blocks = cdiv(K, 128);
  Choice best{};
  double best_time = 0;
  for (const Size& t : kSizes[exact]) {
    if (t.bm == 0) break;
    const int64_t tiles = L * cdiv(M, t.bm) * cdiv(N, t.bn), steps = cdiv(blocks, t.kb);
    for (int splits : {1, 2, 3, 4, 6, 8, 12, 16}) {
      if (splits > 1 && (!t.divides || splits > steps || tiles * (splits - 1) >= kUnits)) break;
      const int64_t per = cdiv(steps, splits), parts = cdiv(steps, per);
      const double idle = 1.0 - std::min<double>(tiles * parts, kUnits) / kUnits;
      double time = (double)cdiv(tiles * parts, kUnits) * (per * t.kb * t.block * (1.0 - idle * t.gain) + t.end);
      // written and read at 3 TB/s, one part after the other
      if (parts > 1) time += 4.0 + 0.12 * parts + parts * L * M * N * 8 / 3e6;
      if (best.bm == 0 || time < best_time) {
        best = {0, t.bm, t.bn, t.kb, (int)parts};
        best_time = time;
      }
    }
  }
  return best;
}

// float32 columns of a row of the parts' sums
inline int64_t sums_ld(int64_t N) { return (N + 3) / 4 * 4; }

// The best tile for `tiles(t)` tiles, as a rule not a whole number, of `blocks` blocks of K, which may be cut into parts
// where values > 0 of them are then added up (as in choose).  A last round with few tiles costs less than a whole one
// where many came before: the units have drifted apart by then, and groups differ in length.  Tiles of
// 64 rows, which read B most often, lose against the larger ones the longer the chip is full (up to 15% from 1 to 8 rounds).
template <class F>
inline Choice choose_tile(int64_t blocks, bool exact, double values, F tiles) {
  Choice best{};
  double best_time = 0;
  for (const Size& t : kSizes[exact]) {
    if (t.bm == 0) break;
    const double all = tiles(t);
    const int64_t steps = cdiv(blocks, t.kb);
    for (int splits : {1, 2, 3, 4, 6, 8, 12, 16}) {
      if (splits > 1 && (values == 0 || !t.divides || splits > steps || all * (splits - 1) >= kUnits)) break;
      const int64_t per = cdiv(steps, splits), parts = cdiv(steps, per);
      const double full = all * parts / kUnits, whole = std::ceil(full), idle = 1.0 - std::min(1.0, full);
      const double slow = exact || t.bm > 64 ? 1.0 : 1.0 + 0.15 * std::min(1.0, std::max(0.0, (full - 1.0) / 7));
      double time = slow * (whole - 0.5 * (whole - full) * std::min(1.0, full / 4)) * (per * t.kb * t.block * (1.0 - idle * t.gain) + t.end);
      if (parts > 1) time += 4.0 + 0.12 * parts + parts * values * 8 / 3e6;
      if (best.bm == 0 || time < best_time) {
        best = {0, t.bm, t.bn, t.kb, (int)parts};
        best_time = time;
      }
    }
  }
  return best;
}

// Rows in E groups, whose sizes the host does not know: taken as T / E and spread around it, so that a group has a tile at
// least and half a tile more than its rows where they are more.  Forced one at a time over 128 cases of 4 to 128
// groups of 24 to 2000 rows, 512 x 2048 to 2048 x 7168, sizes e^(0.5 normal), the tiles chosen cost 2.3% more than the best.
//
// The kernel for few rows, 16 or 32 of a group and 16 or 32 columns to a workgroup, divides K between its waves, which is
// the faster where there are no more workgroups than compute units (of 16 rows and for a float32 C: twice as many)
//   1 x 2048 x 4096, 3 rows     16 x 16 6.0 us   16 x 32 7.7   tiles 10.6   float32 6.3, 15.7
//   2 x 2048 x 4096, 12 each    32 x 16 8.0 us   16 x 32 9.3   tiles 10.6           8.3, 15.9
//   8 x 1024 x 4096, 3 each     16 x 32 8.4 us   16 x 16 9.2   tiles 10.6           8.6, 15.8
//   16 x 1024 x 1024, 12 each   32 x 32 7.2 us   16 x 32 8.2   tiles  6.7           10.0, 8.1
// and, since its workgroups ask for B at once, with a row or two to a group, whatever their number
//   32 x 2048 x 7168     1 row 51.2 us (tiles 54.5), 4 rows 78.3 (79.6), 8 rows 88.4 (82.1)
//   128 x 512 x 2048     1 row 17.2 us (19.4), 4 rows 26.4 (23.9)
inline Choice choose_grouped(int64_t T, int64_t E, int64_t N, int64_t K, bool exact) {
  const int64_t groups = std::max<int64_t>(1, std::min(T, E));
  // pieces of `of` rows that the groups make
  const auto pieces = [&](int of) {
    const double rows = (double)T / groups / of;
    return groups * std::max(1.0, rows + 0.5);
  };
  if (T <= 32 * groups) {
    const int rows = T <= 8 * groups ? 16 : 32;
    const double units = exact && rows == 16 ? 2 * kUnits : kUnits;
    if (pieces(rows) * cdiv(N, 16) <= kUnits) return {16, rows, 0, 1, 1};
    if (pieces(rows) * cdiv(N, 32) <= units || T <= 2 * groups) return {32, rows, 0, 1, 1};
  }
  return choose_tile(cdiv(K, 128), exact, 0, [&](const Size& t) { return pieces(t.bm) * cdiv(N, t.bn); });
}

// Groups along K: E products (M, N) over their shares of all blocks; a group with few of them leaves parts empty.
inline Choice choose_deep(int64_t all, int64_t E, int64_t M, int64_t N) {
  return choose_tile(cdiv(all, E), true, (double)E * M * N, [&](const Size& t) { return (double)(E * cdiv(M, t.bm) * cdiv(N, t.bn)); });
}

// Blocks of 128 rows that E groups of T rows in all take at most, each starting with a block of its own.
inline int64_t group_blocks(int64_t T, int64_t E) { return E == 0 ? 0 : (T + 127 * std::min(T, E)) / 128; }

}  // namespace b128
}  // namespace mxg
