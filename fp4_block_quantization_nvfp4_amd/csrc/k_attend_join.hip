// Joins what the attention kernels leave of units whose keys several waves or
// workgroups had: partial results are sums o of weights times values, the sum l of the
// weights, and the maximum m that the weights are relative to; together
//
//   m = max m_i,  l = sum l_i exp2(m_i - m),  o = sum o_i exp2(m_i - m),
//
// taken in the order of the keys' parts, so a result does not depend on which wave was
// first.  One launch for both kernels (one each: 16 sequences of up to 64 queries and 1500
// keys 35.2 -> 34.5 us).  Bound by the latency of its loads, several in flight a lane: 4 us
// for one sequence of 1000 keys, 8 for 7 sequences of up to 301 queries.
#include "nvfp4_attend.hpp"

namespace nvfp4 {

struct JoinPlan {
  int units, parts, rows;  // of the tiled kernel
};

// Workgroup (g, y) of the split kernel's part: a wave joins rows y, y + 4, .. of the unit
// that begins in its piece, a wave of workgroup g, and goes on in the next ones; of a unit
// that workgroups share, all four waves of its first do.  D / 4 lanes take four sums each, groups of them every so many'th
// part, four parts in flight at a time.
NV_DEV void join_split(const AttendArgs& a, int wg, int y, int pieces) {
  constexpr int FLY = 4;
  __shared__ nv_f4 sums[4][64];
  __shared__ float stat[2][4];
  const int D = a.c.dim, Hk = a.c.heads, G = a.q.heads / Hk, lane = threadIdx.x & 63, wv = uniform(threadIdx.x >> 6);
  const JoinHeader* all = headers(a, D, pieces) + 4 * wg;
  const bool shared = all[0].shared != 0;
  const JoinHeader j = all[shared ? 0 : wv];
  if (j.parts == 0) return;
  const int i = 4 * wg + (shared ? 0 : wv);
  const Sequence q{0, j.q0, j.n, 0, 0, 0};
  const float vdec = a.c.va ? a.c.va[j.unit % Hk] / 2688.0f : 1.0f;
  const int lanes = D <= 32 ? 8 : D <= 64 ? 16 : D <= 128 ? 32 : 64, groups = 64 / lanes * (shared ? 4 : 1);
  const int g = lane / lanes * (shared ? 4 : 1) + (shared ? wv : 0), d = lane % lanes * 4;
  const bool in = d < D;
  // few parts of many rows: the groups take rows of their own
  const bool apart = !shared && j.parts <= 2 * FLY && unit_row(q, G, Hk, j.unit, 4).token >= 0;
  const int first = apart ? 0 : g, step = apart ? 1 : groups;
  for (int r0 = y; r0 < 16; r0 += apart ? 4 * groups : 4) {
    if (unit_row(q, G, Hk, j.unit, r0).token < 0) break;
    const int r = apart ? r0 + 4 * g : r0;
    const UnitRow row = unit_row(q, G, Hk, j.unit, r);
    const bool mine = in && r < 16 && row.token >= 0;
    float m = -INFINITY, l = 0.0f;
    nv_f4 o = (nv_f4){0, 0, 0, 0};
    for (int v0 = 0; v0 < j.parts; v0 += FLY * step) {
      float pm[FLY], pl[FLY];
      nv_f4 x[FLY];
#pragma unroll
      for (int k = 0; k < FLY; ++k) {
        const int v = v0 + k * step + first;
        const int p = v < j.head ? i + v : v < j.head + j.middle ? 4 * (i / 4 + 1 + v - j.head) : 4 * j.w1 + v - j.head - j.middle;
        pm[k] = -INFINITY;
        pl[k] = 0.0f;
        x[k] = (nv_f4){0, 0, 0, 0};
        if (v < j.parts && mine) {
          const float* part = a.part + (2 * (int64_t)p + (p == i ? 1 : 0)) * part_size(D);
          pm[k] = part[16 * D + r];
          pl[k] = part[16 * D + 16 + r];
          x[k] = *reinterpret_cast<const nv_f4*>(part + r * D + d);
        }
      }
      float mn = m;
#pragma unroll
      for (int k = 0; k < FLY; ++k) mn = fmaxf(mn, pm[k]);
      const float base = mn == -INFINITY ? 0.0f : mn, f = exp2_fast(m - base);
      l *= f;
#pragma unroll
      for (int e = 0; e < 4; ++e) o[e] *= f;
#pragma unroll
      for (int k = 0; k < FLY; ++k) {
        const float w = exp2_fast(pm[k] - base);
        l = __builtin_fmaf(pl[k], w, l);
#pragma unroll
        for (int e = 0; e < 4; ++e) o[e] = __builtin_fmaf(x[k][e], w, o[e]);
      }
      m = mn;
    }
    // the groups' sums, in pairs, then the waves'
    for (int off = lanes; !apart && off < 64; off <<= 1) {
      const float om = __shfl_xor(m, off, 64), ol = __shfl_xor(l, off, 64), mn = fmaxf(m, om), base = mn == -INFINITY ? 0.0f : mn;
      const float f = exp2_fast(m - base), w = exp2_fast(om - base);
      l = l * f + ol * w;
#pragma unroll
      for (int e = 0; e < 4; ++e) o[e] = o[e] * f + __shfl_xor(o[e], off, 64) * w;
      m = mn;
    }
    if (shared) {
      __syncthreads();
      sums[wv][lane] = o;
      if (lane == 0) {
        stat[0][wv] = m;
        stat[1][wv] = l;
      }
      __syncthreads();
      m = fmaxf(fmaxf(stat[0][0], stat[0][1]), fmaxf(stat[0][2], stat[0][3]));
      l = 0.0f;
      o = (nv_f4){0, 0, 0, 0};
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        const float f = exp2_fast(stat[0][w] - (m == -INFINITY ? 0.0f : m));
        l = __builtin_fmaf(stat[1][w], f, l);
#pragma unroll
        for (int e = 0; e < 4; ++e) o[e] = __builtin_fmaf(sums[w][lane][e], f, o[e]);
      }
    }
    if (mine && (apart || lane < lanes) && (!shared || wv == 0)) write_row(a, (int64_t)row.token * a.q.heads + row.head, d, o, m, l, vdec);
  }
}

// Workgroup (unit, y) of the tiled kernel's part: rows 16 y .. 16 y + 15, D / 4 lanes take four sums each.
NV_DEV void join_tiles(const AttendArgs& a, int unit, int y, const JoinPlan& p) {
  const TileHeader t = tile_headers(a)[unit];
  if (t.parts == 0) return;
  const int D = a.c.dim, Hk = a.c.heads, G = a.q.heads / Hk;
  const float vdec = a.c.va ? a.c.va[t.h] / 2688.0f : 1.0f;
  for (int e = threadIdx.x; e < 4 * D; e += 256) {
    const int r = 16 * y + e / (D / 4), d = e % (D / 4) * 4;
    const int row = t.m0 + r, i = row / G, head = t.h * G + row - i * G;
    if (i >= t.n) break;
    float m = -INFINITY, l = 0.0f;
    nv_f4 o = (nv_f4){0, 0, 0, 0};
    constexpr int FLY = 4;
    for (int p0 = 0; p0 < t.parts; p0 += FLY) {
      float pm[FLY], pl[FLY];
      nv_f4 x[FLY];
#pragma unroll
      for (int k = 0; k < FLY; ++k) {
        const float* part = tile_part(a, p.units, p.parts, p.rows, unit, p0 + k < t.parts ? p0 + k : t.parts - 1);
        pm[k] = part[p.rows * D + r];
        pl[k] = part[p.rows * (D + 1) + r];
        x[k] = *reinterpret_cast<const nv_f4*>(part + r * D + d);
      }
#pragma unroll
      for (int k = 0; k < FLY; ++k) {
        if (p0 + k >= t.parts) break;
        const float mn = fmaxf(m, pm[k]), base = mn == -INFINITY ? 0.0f : mn, f = exp2_fast(m - base), w = exp2_fast(pm[k] - base);
        l = __builtin_fmaf(pl[k], w, l * f);
#pragma unroll
        for (int j = 0; j < 4; ++j) o[j] = __builtin_fmaf(x[k][j], w, o[j] * f);
        m = mn;
      }
    }
    write_row(a, (int64_t)(t.q0 + i) * a.q.heads + head, d, o, m, l, vdec);
  }
}

// `wgs` workgroups of the split kernel, four joining each; then the tiled kernel's units.
__global__ __launch_bounds__(256) void k_attend_join(const AttendArgs a, int wgs, const JoinPlan p) {
  const int x = (int)blockIdx.x - 4 * wgs;
  if (x < 0) join_split(a, blockIdx.x % wgs, blockIdx.x / wgs, 4 * wgs);
  else join_tiles(a, x % p.units, x / p.units, p);
}

void launch_attend_split(const AttendArgs& a, hipStream_t st);
void launch_attend_tiles(const AttendArgs& a, const TilesPlan& p, hipStream_t st);

int launch_attend(AttendArgs a, int which, void* workspace, void* stream) {
  hipStream_t st = (hipStream_t)stream;
  const int64_t keys = (int64_t)a.width << a.c.shift;
  const int Hq = a.q.heads, Hk = a.c.heads, D = a.c.dim;
  const size_t bytes = attend_split_bytes(a.T, a.B, Hq, Hk, D, keys);
  a.part = bytes ? (float*)workspace : nullptr;  // a caller's may be there and empty
  a.tiles = (float*)((uint8_t*)workspace + bytes);
  launch_attend_split(a, st);
  JoinPlan joined{1, 1, 0};
  if (which & 2) {
    const TilesPlan p = tiles_plan(a.T, a.B, Hq, Hk, D, keys);
    launch_attend_tiles(a, p, st);
    joined = {(int)p.units, p.parts, 32 * p.waves};
  }
  const LayerLaunch j = plan_attend_join(a.T, a.B, Hq, Hk, D, keys, which);
  if (j.grid) k_attend_join<<<(uint32_t)j.grid, j.block, 0, st>>>(a, (int)attend_pieces(a.T, a.B, Hq, Hk, D, keys), joined);
  return (int)hipGetLastError();
}

}  // namespace nvfp4
