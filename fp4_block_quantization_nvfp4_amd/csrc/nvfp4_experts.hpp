// Row ranges of experts, found on the device from the cumulative row counts
// `ends` (int32 [E]).  Rows [ends[e - 1], ends[e]) belong to expert e; rows
// at or past the last end belong to none and form the extra range E.  Counts
// are clamped to [0, rows] and taken as their running maximum, so whatever
// `ends` holds, the ranges are disjoint, cover all rows and stay inside.
#pragma once

#include "nvfp4_mx8.hpp"
#include "nvfp4_plan.hpp"

namespace nvfp4 {

struct RowRange {
  int e;       // expert, or E for rows of none
  int row0;    // first row
  int rows;    // rows in the range
  int before;  // tiles of the ranges before it
};

// One wave walks the ranges 64 at a time.  `tile` rows make a tile; a range
// has ceil(rows / tile) of them.  There are at most 2^29 rows (K >= 16), so a
// tile more does not pass 31 bits.
struct RangeScan {
  const int* ends;
  int E, T, tile, lane;
  int base, prev, tiles;         // ranges done, running end, tiles done
  int begin, count, first, own;  // this lane's range of the current 64

  NV_DEV RangeScan(const int* ends_, int E_, int T_, int tile_)
      : ends(ends_), E(E_), T(T_), tile(tile_), lane(threadIdx.x & 63), base(0), prev(0), tiles(0) {}

  // Loads the next 64 ranges; false when none are left.
  NV_DEV bool next() {
    if (base > E) return false;
    const int e = base + lane;
    int v = T;
    if (e < E) {
      v = ends[e];
      v = v < 0 ? 0 : (v > T ? T : v);
    }
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
      const int p = __shfl_up(v, o, 64);
      if (lane >= o) v = p > v ? p : v;
    }
    v = v > prev ? v : prev;
    const int p = __shfl_up(v, 1, 64);
    begin = lane ? p : prev;
    count = v - begin;
    own = (count + tile - 1) / tile;
    int s = own;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
      const int q = __shfl_up(s, o, 64);
      if (lane >= o) s += q;
    }
    first = tiles + s - own;
    prev = __shfl(v, 63, 64);
    tiles += __shfl(s, 63, 64);
    base += 64;
    return true;
  }
};

NV_DEV int uniform(int v) { return __builtin_amdgcn_readfirstlane(v); }

// The range in s's current 64 that holds `unit`, where each tile stands for
// `per` consecutive units; rows = -1 when none does.
NV_DEV RowRange range_of(const RangeScan& s, int64_t per, int64_t unit) {
  RowRange r = {0, 0, -1, 0};
  const uint64_t vote = __ballot(unit >= (int64_t)s.first * per && unit < (int64_t)(s.first + s.own) * per);
  if (vote) {
    const int l = __builtin_ctzll(vote);
    r.e = uniform(s.base - 64 + l);
    r.row0 = uniform(__shfl(s.begin, l, 64));
    r.rows = uniform(__shfl(s.count, l, 64));
    r.before = uniform(__shfl(s.first, l, 64));
  }
  return r;
}

// A workgroup's unit of work among `units`; false for a surplus workgroup.
// Each XCD (workgroups go to the eight in turn) takes a contiguous run.  With
// SPLIT the units past the last whole round of kGroupedSlots are shared by two
// or four workgroups each, as long as each of these has a CU of its own: part
// is then the number of parts times 256 plus the workgroup's own, else 0.
template <bool SPLIT>
NV_DEV bool unit_of_block(int64_t units, uint32_t block, int64_t& unit, int& part) {
  const int64_t over = SPLIT ? units % kGroupedSlots : 0;
  const int split = over * 8 <= kGroupedSlots ? 4 : over * 4 <= kGroupedSlots ? 2 : 1;
  const int64_t whole = units - (split > 1 ? over : 0), share = (whole + 7) / 8, slot = block >> 3;
  part = 0;
  unit = (block & 7) * share + slot;
  if (slot < share) return unit < whole;
  if (!SPLIT || split == 1) return false;
  const int64_t parts = over * split, more = (parts + 7) / 8, p = (block & 7) * more + slot - share;
  unit = whole + p / split;
  part = split * 256 + (int)(p % split);
  return slot - share < more && p < parts;
}

// The unit of a workgroup, `per` units a tile of a range, and the range that
// holds it, rows = -1 for a surplus workgroup.  Up to 63 experts take one
// scan, more of them two.
template <bool SPLIT>
NV_DEV RowRange find_unit(const int* ends, int E, int T, int tile, int64_t per, uint32_t block, int64_t& unit, int& part) {
  RangeScan s(ends, E, T, tile);
  s.next();
  const bool one = s.base > E;
  while (!one && s.next()) {
  }
  RowRange r = {0, 0, -1, 0};
  if (!unit_of_block<SPLIT>(uniform(s.tiles) * per, block, unit, part)) return r;
  if (one) return range_of(s, per, unit);
  RangeScan again(ends, E, T, tile);
  while (r.rows < 0 && again.next()) r = range_of(again, per, unit);
  return r;
}

// Rows of expert e alone (e < E): the running maximum of the ends before it.
NV_DEV RowRange expert_range(const int* ends, int T, int e) {
  const int lane = threadIdx.x & 63;
  int lo = 0;
  for (int b = lane; b < e; b += 64) {
    const int v = ends[b];
    lo = v > lo ? v : lo;
  }
#pragma unroll
  for (int o = 32; o >= 1; o >>= 1) {
    const int p = __shfl_xor(lo, o, 64);
    lo = p > lo ? p : lo;
  }
  lo = lo > T ? T : lo;
  int hi = ends[e];
  hi = hi > T ? T : hi;
  hi = hi > lo ? hi : lo;
  return {e, uniform(lo), uniform(hi - lo), 0};
}

}  // namespace nvfp4
