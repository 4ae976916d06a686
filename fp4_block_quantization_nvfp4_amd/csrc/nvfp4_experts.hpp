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

NV_DEV int uniform(int v) { return __builtin_amdgcn_readfirstlane(v); }

// Running maximum and running sum over a wave's lanes, of numbers >= 0: within
// rows of 16 lanes, then the last lane of a row to the next, then that of the
// lower half to the upper.  Data moves between registers: with shuffles through
// shared memory, and a second scan to see that no tile is left, the matvec of 64
// rows, 32 experts 4096 x 2048 took 39.4 us, not 33.7, and of 256 rows, 8 experts
// 1024 x 1024 7.3, not 6.0.
#define NV_SCAN_STEPS(OP)                                                                        \
  OP(0x111, 0xF) OP(0x112, 0xF) OP(0x114, 0xF) OP(0x118, 0xF) OP(0x142, 0xA) OP(0x143, 0xC)
NV_DEV int running_max(int v) {
#define NV_STEP(CTRL, ROWS)                                                  \
  {                                                                          \
    const int o = __builtin_amdgcn_update_dpp(0, v, CTRL, ROWS, 0xF, false); \
    v = o > v ? o : v;                                                       \
  }
  NV_SCAN_STEPS(NV_STEP)
#undef NV_STEP
  return v;
}
NV_DEV int running_sum(int v) {
#define NV_STEP(CTRL, ROWS) v += __builtin_amdgcn_update_dpp(0, v, CTRL, ROWS, 0xF, false);
  NV_SCAN_STEPS(NV_STEP)
#undef NV_STEP
  return v;
}
#undef NV_SCAN_STEPS

// One wave walks the ranges 64 at a time.  `tile` rows make a tile; a range
// has ceil(rows / tile) of them.  There are at most 2^29 rows (K >= 16), so a
// tile more does not pass 31 bits.
struct RangeScan {
  const int* ends;
  int E, T, tile, lane;
  int base, prev, tiles;         // ranges done, running end, tiles done
  int ahead;                     // the lane's end of the next 64
  int begin, count, first, own;  // this lane's range of the current 64

  NV_DEV RangeScan(const int* ends_, int E_, int T_, int tile_)
      : ends(ends_), E(E_), T(T_), tile(tile_), lane(threadIdx.x & 63), base(0), prev(0), tiles(0), ahead(T_) {
    if (lane < E) ahead = ends[lane];
  }

  // Takes the next 64 ranges; false when none are left.
  NV_DEV bool next() {
    if (base > E) return false;
    int v = ahead < 0 ? 0 : ahead > T ? T : ahead;
    ahead = base + 64 + lane < E ? ends[base + 64 + lane] : T;
    v = running_max(v);
    v = v > prev ? v : prev;
    begin = __builtin_amdgcn_update_dpp(prev, v, 0x138, 0xF, 0xF, false);  // the lane before's; lane 0: prev
    count = v - begin;
    own = (int)((uint32_t)(count + tile - 1) / (uint32_t)tile);
    const int s = running_sum(own);
    first = tiles + s - own;
    prev = __builtin_amdgcn_readlane(v, 63);
    tiles += __builtin_amdgcn_readlane(s, 63);
    base += 64;
    return true;
  }
};

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

// The range that holds tile `unit` of all ranges' tiles, rows = -1 when there are
// fewer; tiles: how many there are.
NV_DEV RowRange range_of_tile(const int* ends, int E, int T, int tile, int unit, int& tiles) {
  RangeScan s(ends, E, T, tile);
  RowRange r = {0, 0, -1, 0};
  while (s.next())
    if (r.rows < 0) r = range_of(s, 1, unit);
  tiles = uniform(s.tiles);
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
