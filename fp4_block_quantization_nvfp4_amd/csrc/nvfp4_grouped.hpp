// Products of many rows with 4-bit weights, grouped by expert: for the rows
// t of expert e, out[t, n] = S_n sum_k x[t, k] v[n, k] s[n, k / 16] (see
// k_matvec.hip; without `ends` all rows belong to expert 0).
//
// A workgroup of four waves makes a tile of BM rows by 256 n's and walks k in
// steps of 128.  The rows of x are staged as bf16 in shared memory (two
// buffers, half a step's loads in flight at a time); each wave decodes the
// weights of its own 64 n's straight from global memory into fragments, so no
// weight is decoded twice in a workgroup and the weights cost no shared
// memory.  Codes are fetched into the registers that the step has just
// consumed, and the next fragments are decoded and read while the matrix cores
// work on the present ones.  The weight is the first operand of the matrix
// product: a lane then holds four consecutive n's of one row.
//
// The row ranges are known on the device only, so the grid is an upper bound
// and surplus workgroups leave at once.  Tiles are numbered per expert in
// blocks of 8 row tiles, and each XCD takes a contiguous run of them: what
// runs at one time on an XCD shares rows of x and weights in its L2.
#pragma once

#include "nvfp4_experts.hpp"
#include "nvfp4_launch.hpp"
#include "nvfp4_plan.hpp"
#include "nvfp4_weight.hpp"

namespace nvfp4 {

// The tile of expert e's rows row0 .. row0 + rows - 1 (rows <= BM) and n's from
// 128 NI n_tile on; e >= E (rows of no expert) gives zeros.  lds: two buffers
// of BM x 128, and 4 NI KB a wave for the way out.
template <bool MX8, int BLK, int BM, int NI>
NV_DEV void grouped_tile(const MatmulArgs& a, uint16_t* lds, int e, int64_t row0, int rows, int n_tile) {
  constexpr int MI = BM / 32;
  const int tid = threadIdx.x, wave = uniform(tid >> 6), lane = tid & 63, l32 = lane & 31, half = lane >> 5;
  const bool none = a.ends && e >= a.E;
  const int n0 = n_tile * (128 * NI) + wave * (32 * NI);

  nv_f16 acc[NI][MI];
#pragma unroll
  for (int i = 0; i < NI; ++i)
#pragma unroll
    for (int m = 0; m < MI; ++m)
#pragma unroll
      for (int r = 0; r < 16; ++r) acc[i][m][r] = 0.0f;

  const int nk = none ? 0 : (a.K + 127) / 128;
  if (nk) {
    const WeightStream<BLK, NI> w(a, e, n0, l32, half);
    const RowsView<MX8> x(a, row0, rows);
    typedef RowsHalf<MX8, BM> Half;
    constexpr int PR = Half::PR, PIECES = Half::PIECES;
    const int xr = tid / PR, xp = tid % PR;
    Half st;
    auto fetch = [&](int k0, int h) { st.load(x, tid, k0, h); };
    // row r of a buffer: 16 chunks of 16 bytes, chunk c at c ^ (r % 16)
    auto put = [&](uint16_t* buf, int r, int c, nv_u4 v) {
      *reinterpret_cast<nv_u4*>(buf + r * 128 + ((c ^ (r & 15)) * 8)) = v;
    };
    auto stage = [&](int i, uint16_t* buf, int h) {
      if (Half::HALF < 256 && tid >= Half::HALF) return;
      const int r = h * (BM / 2) + i * (256 / PR) + xr;
      if (MX8) {
        const float sc = e8m0_scale(st.s[i]);
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const nv_u2 u = mx8_to_bf16(st.c[i][2 * j], sc), v = mx8_to_bf16(st.c[i][2 * j + 1], sc);
          put(buf, r, 2 * xp + j, (nv_u4){u.x, u.y, v.x, v.y});
        }
      } else {
        put(buf, r, xp, st.c[i]);
      }
    };
    nv_u4 wc[NI][2];
    uint32_t ws[NI], wsn[4];  // scales of this step; of the next as fetched
    nv_u2 wf[2][NI][2];
    nv_bf8 xf[MI];
    auto fetch_codes = [&](int k0, int q) {
#pragma unroll
      for (int i = 0; i < NI; ++i) wc[i][q] = w.codes(i, k0, q);
    };
    // quarter d of the weight fragments of k's 8 s .. 8 s + 7 of each half
    auto decode = [&](int s, int d) {
      wf[s & 1][d >> 1][d & 1] = fp4_half_to_bf16(wc[d >> 1][s >> 2][s & 3], e4m3_byte(ws[d >> 1], s >> 1), d & 1);
    };
    auto load_x = [&](const uint16_t* buf, int s, int m) {
      xf[m] = *reinterpret_cast<const nv_bf8*>(buf + (m * 32 + l32) * 128 + (((8 * half + s) ^ (l32 & 15)) * 8));
    };
    auto fragment = [&](int s, int i) {
      const nv_u2 u = wf[s & 1][i][0], v = wf[s & 1][i][1];
      return __builtin_bit_cast(nv_bf8, (nv_u4){u.x, u.y, v.x, v.y});
    };
    fetch_codes(0, 0);
    fetch_codes(0, 1);
    w.fetch_scales(0, wsn);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      fetch(0, h);
#pragma unroll
      for (int i = 0; i < PIECES; ++i) stage(i, lds, h);
    }
    fetch(128, 0);
    w.scales(0, wsn, ws);
    w.fetch_scales(128, wsn);
    __syncthreads();
#pragma unroll
    for (int m = 0; m < MI; ++m) load_x(lds, 0, m);
#pragma unroll
    for (int d = 0; d < 2 * NI; ++d) decode(0, d);
    // Eight parts of 16 k's a step.  While the matrix cores work on part s,
    // part s + 1 is read and decoded, a piece after each pair of products; the
    // next step's rows are written in parts 2 and 6 and its codes fetched once
    // this one's are decoded.
    for (int kt = 0; kt < nk; ++kt) {
      const uint16_t* buf = lds + (kt & 1) * (BM * 128);
      uint16_t* next = lds + (~kt & 1) * (BM * 128);
      const int k1 = kt * 128 + 128;
#pragma unroll
      for (int s = 0; s < 8; ++s) {
        if (s == 3) fetch_codes(k1, 0);
        if (s == 7) {
          fetch_codes(k1, 1);
          w.scales(k1, wsn, ws);
          w.fetch_scales(k1 + 128, wsn);
        }
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int m = 0; m < MI; ++m) {
#pragma unroll
          for (int i = 0; i < NI; ++i) acc[i][m] = mfma32(fragment(s, i), xf[m], acc[i][m]);
          load_x(s < 7 ? buf : next, (s + 1) & 7, m);
#pragma unroll
          for (int d = m * 2 * NI / MI; d < (m + 1) * 2 * NI / MI; ++d) decode((s + 1) & 7, d);
#pragma unroll
          for (int i = 0; i < PIECES; ++i) {
            if (i % MI != m) continue;
            if (s == 2) stage(i, next, 0);
            if (s == 6) stage(i, next, 1);
          }
          if (m == MI - 1 && s == 2) fetch(k1, 1);
          if (m == MI - 1 && s == 7) fetch(k1 + 128, 0);
          __builtin_amdgcn_sched_barrier(0);
        }
        if (s == 6) __syncthreads();  // the next step's rows are written, this one's are all read
      }
    }
  }
  __syncthreads();  // the rows' buffers are free
  if (n0 >= a.N) return;
  // A lane holds, of each 32x32 tile, row l32 of x and n = 8 q + 4 half + 0..3.
  // 32 rows at a time go through the wave's part of shared memory (16-byte
  // chunk c of row t at c ^ t) and leave as whole rows of 32 NI n's.
  constexpr int ROW = 8 * NI;  // chunks of a row
  nv_f4* out = reinterpret_cast<nv_f4*>(lds) + wave * (32 * ROW);
  const int n = n0 + lane % ROW * 4;
  float sc[4];
#pragma unroll
  for (int r = 0; r < 4; ++r) sc[r] = none || n + r >= a.N ? 0.0f : second_scale(a, e, n + r);
#pragma unroll
  for (int m = 0; m < MI; ++m) {
#pragma unroll
    for (int i = 0; i < NI; ++i)
#pragma unroll
      for (int q = 0; q < 4; ++q)
        out[l32 * ROW + ((i * 8 + q * 2 + half) ^ (l32 % ROW))] =
            nv_f4{acc[i][m][q * 4], acc[i][m][q * 4 + 1], acc[i][m][q * 4 + 2], acc[i][m][q * 4 + 3]};
    const int left = rows - m * 32 < 32 ? rows - m * 32 : 32;
#pragma unroll 4
    for (int t = lane / ROW; t < left; t += 64 / ROW) {
      const nv_f4 v = out[t * ROW + ((lane % ROW) ^ (t % ROW))];
      store_out4(a, v[0] * sc[0], v[1] * sc[1], v[2] * sc[2], v[3] * sc[3], row0 + m * 32 + t, n);
    }
  }
}

// BM: rows of a unit of work.  Units past the last whole round of the chip
// (kGroupedSlots workgroups) are split among more workgroups where each still
// gets a CU of its own: by four up to an eighth of a round, by two up to a
// quarter.  A tile with few rows takes the path made for as many.
template <bool MX8, int BLK, int BM, int NI>
__global__ __launch_bounds__(256, 2) void k_grouped(MatmulArgs a) {
  __shared__ uint16_t lds[2 * (BM < 64 ? 64 : BM) * 128];
  const int ntiles = (a.N + 128 * NI - 1) / (128 * NI);
  int64_t unit;
  int part;
  RowRange rr = {0, 0, a.T, 0};
  if (a.ends) rr = find_unit<BM == 128>(a.ends, a.E, a.T, BM, ntiles, blockIdx.x, unit, part);
  else if (!unit_of_block<BM == 128>((int64_t)((a.T + BM - 1) / BM) * ntiles, blockIdx.x, unit, part)) return;
  if (rr.rows < 0) return;
  // units of a range are numbered in blocks of eight row tiles
  const int mt = (rr.rows + BM - 1) / BM;
  const int local = (int)(unit - (int64_t)rr.before * ntiles), block = local / (8 * ntiles);
  const int in = local - block * 8 * ntiles, bm = mt - block * 8 < 8 ? mt - block * 8 : 8;
  const int n_tile = in / bm, m_tile = block * 8 + in % bm;
  const int split = part >> 8, of = split ? BM / split : BM;  // rows of a workgroup
  const int first = m_tile * BM + (part & 255) * of;
  const int rows = rr.rows - first < of ? rr.rows - first : of;
  if (rows <= 0) return;
  const int64_t row0 = (int64_t)rr.row0 + first;
  if (BM == 128 && rows > 64) grouped_tile<MX8, BLK, BM, NI>(a, lds, rr.e, row0, rows, n_tile);
  else if (BM >= 64 && rows > 32) grouped_tile<MX8, BLK, BM < 64 ? BM : 64, NI>(a, lds, rr.e, row0, rows, n_tile);
  else grouped_tile<MX8, BLK, 32, NI>(a, lds, rr.e, row0, rows, n_tile);
}

template <bool MX8, int BLK, int NI>
static void grouped_rows_go(const MatmulArgs& a, const GroupedPlan& p, hipStream_t st) {
  const uint32_t grid = (uint32_t)p.grid;
  if (p.rows == 128) k_grouped<MX8, BLK, 128, NI><<<grid, 256, 0, st>>>(a);
  else if (p.rows == 64) k_grouped<MX8, BLK, 64, NI><<<grid, 256, 0, st>>>(a);
  else k_grouped<MX8, BLK, 32, NI><<<grid, 256, 0, st>>>(a);
}

template <bool MX8, int BLK>
static void grouped_go(const MatmulArgs& a, hipStream_t st) {
  const GroupedPlan p = plan_grouped(a.T, a.ends ? a.E : 0, a.N);
  if (p.width == 256) grouped_rows_go<MX8, BLK, 2>(a, p, st);
  else grouped_rows_go<MX8, BLK, 1>(a, p, st);
}

template <bool MX8>
static int grouped_launch(const MatmulArgs& a, void* stream) {
  hipStream_t st = (hipStream_t)stream;
  a.blocks == 0 ? grouped_go<MX8, 0>(a, st) : a.blocks == 1 ? grouped_go<MX8, 1>(a, st) : grouped_go<MX8, 2>(a, st);
  return (int)hipGetLastError();
}

}  // namespace nvfp4
