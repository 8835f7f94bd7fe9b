// Rows in order of the group (expert) they belong to: group e holds rows
// offsets[e] .. offsets[e + 1] - 1, offsets in device memory, so that a call
// needs no answer from the GPU.  A kernel looks for the group its work falls to:
// one wave reads 64 offsets at a time and adds up the groups' units (rows in
// tiles or blocks) across its lanes.
//
// Offsets are taken as they are found but held within 0 .. T, so those that
// decrease or lie outside give a wrong result and never an access out of bounds.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace mxg {
namespace groups {

constexpr int kMaxGroups = 1024;       // a tile kernel keeps a table of them in LDS
constexpr int64_t kMaxRows = 1 << 24;  // the units of 1024 groups are counted in 32 bits, whatever the offsets

struct Groups {
  const void* offsets;
  int E, T;
  bool off64;
};

// Offset i (at most E), within 0 .. T.
__device__ __forceinline__ int offset(const Groups& g, int i) {
  const int at = min(i, g.E);
  if (g.off64) {
    const int64_t v = static_cast<const int64_t*>(g.offsets)[at];
    return (int)(v < 0 ? 0 : v > g.T ? g.T : v);
  }
  return min(max(static_cast<const int*>(g.offsets)[at], 0), g.T);
}

// Inclusive sum over the lanes of a wave, all of them active: within rows of 16 by shifts, then from row to row.
__device__ __forceinline__ int wave_sum(int v) {
  v += __builtin_amdgcn_update_dpp(0, v, 0x111, 0xF, 0xF, false);
  v += __builtin_amdgcn_update_dpp(0, v, 0x112, 0xF, 0xF, false);
  v += __builtin_amdgcn_update_dpp(0, v, 0x114, 0xF, 0xF, false);
  v += __builtin_amdgcn_update_dpp(0, v, 0x118, 0xF, 0xF, false);
  v += __builtin_amdgcn_update_dpp(0, v, 0x142, 0xA, 0xF, false);  // lane 15 of rows 0 and 2 to the next row
  v += __builtin_amdgcn_update_dpp(0, v, 0x143, 0xC, 0xF, false);  // lane 31 to the upper half
  return v;
}

// Offsets i + 64 j + lane, j <= 4: asked for together, since one waits for memory as long as all of them.
struct Ahead {
  int at[5];
  __device__ __forceinline__ Ahead(const Groups& g, int i, int lane) {
#pragma unroll
    for (int j = 0; j < 5; ++j) at[j] = offset(g, i + 64 * j + lane);
  }
};

// Groups i .. i + 63, one to a lane: its first row, its units of `per` rows, and the units up to its end where `before`
// lie in the groups before i.  Its offset is `start` in the lane; `next` starts with the offset behind the last lane's.
struct Span {
  int start, rows, units, end;
};
__device__ __forceinline__ Span span(const Groups& g, int i, int lane, int per, int before, int start, int next) {
  Span s;
  s.start = start;
  const int behind = __builtin_amdgcn_readfirstlane(next);
  const int stop = __builtin_amdgcn_update_dpp(behind, start, 0x130, 0xF, 0xF, false);  // lane + 1's
  s.rows = i + lane < g.E ? max(stop - start, 0) : 0;
  s.units = (s.rows + per - 1) / per;
  s.end = before + wave_sum(s.units);
  return s;
}

// The unit `want` of all groups' units: its group, the group's rows, the first of them, and which of the group's units it
// is.  group < 0: there are no more than `total`, which is known then.  Every lane of the wave takes part and gets the
// answer.
struct Unit {
  int group, start, rows, at, total;
};
__device__ __forceinline__ Unit find(const Groups& g, int want, int lane, int per) {
  Unit u = {-1, 0, 0, 0, 0};
  for (int i = 0; i < g.E; i += 256) {
    const Ahead a(g, i, lane);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if (i + 64 * j >= g.E) break;
      const Span s = span(g, i + 64 * j, lane, per, u.total, a.at[j], a.at[j + 1]);
      const uint64_t past = __ballot(s.end > want);
      if (past) {
        const int from = __builtin_ctzll(past);
        u.group = i + 64 * j + from;
        u.start = __builtin_amdgcn_readlane(s.start, from);
        u.rows = __builtin_amdgcn_readlane(s.rows, from);
        u.at = want - (__builtin_amdgcn_readlane(s.end, from) - __builtin_amdgcn_readlane(s.units, from));
        return u;
      }
      u.total = __builtin_amdgcn_readlane(s.end, 63);
    }
  }
  return u;
}

// Every group's first row and the units up to it, in LDS; entry E closes both.
struct Table {
  int start[kMaxGroups + 1], units[kMaxGroups + 1];
};
// Filled by one wave.  No count exceeds `most`, what the groups can have at most.
__device__ __forceinline__ void fill(Table* t, const Groups& g, int lane, int per, int most) {
  int before = 0;
  for (int i = 0; i < g.E; i += 256) {
    const Ahead a(g, i, lane);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int first = i + 64 * j;
      if (first >= g.E) break;
      const Span s = span(g, first, lane, per, before, a.at[j], a.at[j + 1]);
      if (first + lane < g.E) {
        t->start[first + lane] = s.start;
        t->units[first + lane + 1] = min(s.end, most);
      }
      before = __builtin_amdgcn_readlane(s.end, 63);
    }
  }
  if (lane == 0) {
    t->start[g.E] = offset(g, g.E);
    t->units[0] = 0;
  }
}
// The group of unit `want`, which there is; the search starts at group `from`, which is not past it.
__device__ __forceinline__ int lookup(const Table* t, int E, int want, int from, int lane) {
  for (int i = from;; i += 64) {
    const int at = min(i + lane, E - 1);
    const uint64_t past = __ballot(i + lane >= E || t->units[at + 1] > want);
    if (past) return min(i + __builtin_ctzll(past), E - 1);
  }
}

}  // namespace groups
}  // namespace mxg
