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
#include "nvfp4_experts.hpp"
#include "nvfp4_launch.hpp"
#include "nvfp4_plan.hpp"
#include "nvfp4_weight.hpp"

namespace nvfp4 {

template <bool MX8, int BLK, int BM, bool WORDS>
__global__ __launch_bounds__(256, 2) void k_grouped(MatmulArgs a) {
  constexpr int MI = BM / 32;
  __shared__ uint16_t lds[2][(BM < 64 ? 64 : BM) * 128];  // at least 8 KB a wave for the way out
  const int tid = threadIdx.x, wave = uniform(tid >> 6), lane = tid & 63, l32 = lane & 31, half = lane >> 5;
  const int ntiles = (a.N + 255) / 256;

  // this workgroup's tile
  int e = 0, row0, rows, n_tile;
  {
    RowRange rr = {0, 0, a.T, 0};
    int64_t unit;
    if (a.ends) rr = find_unit(a.ends, a.E, a.T, BM, ntiles, blockIdx.x, unit);
    else {
      const int64_t units = (int64_t)((a.T + BM - 1) / BM) * ntiles, share = (units + 7) / 8, slot = blockIdx.x >> 3;
      unit = (blockIdx.x & 7) * share + slot;
      if (slot >= share || unit >= units) return;
    }
    if (rr.rows < 0) return;
    const int mt = (rr.rows + BM - 1) / BM;
    const int local = (int)(unit - (int64_t)rr.before * ntiles), block = local / (8 * ntiles);
    const int in = local - block * 8 * ntiles, bm = mt - block * 8 < 8 ? mt - block * 8 : 8;
    n_tile = in / bm;
    const int m_tile = block * 8 + in % bm;
    e = rr.e;
    row0 = rr.row0 + m_tile * BM;
    rows = rr.rows - m_tile * BM < BM ? rr.rows - m_tile * BM : BM;
  }
  const bool none = a.ends && e >= a.E;
  const int n0 = n_tile * 256 + wave * 64;

  nv_f16 acc[2][MI];
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int m = 0; m < MI; ++m)
#pragma unroll
      for (int r = 0; r < 16; ++r) acc[i][m][r] = 0.0f;

  const int nk = none ? 0 : (a.K + 127) / 128;
  if (nk) {
    const WeightStream<BLK, WORDS> w(a, e, n0, l32, half);
    const RowsView<MX8> x(a, row0, rows);
    // staging of half a step's rows: 16-byte pieces, piece p of a row
    constexpr int PR = MX8 ? 8 : 16, HALF = BM / 2 * PR, PIECES = HALF > 256 ? HALF / 256 : 1;
    nv_u4 st[PIECES];
    uint32_t sts[PIECES];
    auto fetch = [&](int i, int k0, int h) {
      const int id = tid + i * 256, r = h * (BM / 2) + id / PR, p = id % PR;
      if (HALF < 256 && id >= HALF) return;
      if (MX8) {
        const int k = k0 + p * 16;
        st[i] = buf16(x.x, k < a.K ? (uint32_t)(r * a.K + k) : kOutside);
        sts[i] = buf1(x.s, k < a.K ? (uint32_t)(r * x.ns + k / kMxGroup) : kOutside);
      } else {
        const int k = k0 + p * 8;
        st[i] = buf16(x.x, k < a.K ? (uint32_t)(r * a.K + k) * 2u : kOutside);
      }
    };
    // row r of a buffer: 16 chunks of 16 bytes, chunk c at c ^ (r % 16)
    auto put = [&](uint16_t* buf, int r, int c, nv_u4 v) {
      *reinterpret_cast<nv_u4*>(buf + r * 128 + ((c ^ (r & 15)) * 8)) = v;
    };
    auto stage = [&](int i, uint16_t* buf, int h) {
      const int id = tid + i * 256, r = h * (BM / 2) + id / PR, p = id % PR;
      if (HALF < 256 && id >= HALF) return;
      if (MX8) {
        const float sc = e8m0_value(sts[i]);
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const nv_u2 u = mx8_to_bf16(st[i][2 * j], sc), v = mx8_to_bf16(st[i][2 * j + 1], sc);
          put(buf, r, 2 * p + j, (nv_u4){u.x, u.y, v.x, v.y});
        }
      } else {
        put(buf, r, p, st[i]);
      }
    };
    nv_u4 wc[2][2];
    uint32_t ws[2][2];  // scales of this step and the next
    nv_u2 wf[2][2][2];
    nv_bf8 xf[MI];
    auto fetch_codes = [&](int k0, int q) {
#pragma unroll
      for (int i = 0; i < 2; ++i) wc[i][q] = w.codes(i, k0, q);
    };
    // quarter d of the weight fragments of k's 8 s .. 8 s + 7 of each half
    auto decode = [&](int s, const uint32_t v[2], int d) {
      wf[s & 1][d >> 1][d & 1] = fp4_half_to_bf16(wc[d >> 1][s >> 2][s & 3], e4m3_byte(v[d >> 1], s >> 1), d & 1);
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
    w.scales(0, ws[0]);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
#pragma unroll
      for (int i = 0; i < PIECES; ++i) fetch(i, 0, h);
#pragma unroll
      for (int i = 0; i < PIECES; ++i) stage(i, lds[0], h);
    }
#pragma unroll
    for (int i = 0; i < PIECES; ++i) fetch(i, 128, 0);
    w.scales(128, ws[1]);
    __syncthreads();
#pragma unroll
    for (int m = 0; m < MI; ++m) load_x(lds[0], 0, m);
#pragma unroll
    for (int d = 0; d < 4; ++d) decode(0, ws[0], d);
    // Eight parts of 16 k's a step.  While the matrix cores work on part s,
    // part s + 1 is read and decoded, a piece after each pair of products; the
    // next step's rows are written in parts 2 and 6 and its codes fetched once
    // this one's are decoded.  Past the last step every load is outside and
    // gives zeros.
    for (int kt = 0; kt < nk; ++kt) {
      const uint16_t* buf = lds[kt & 1];
      uint16_t* next = lds[(kt + 1) & 1];
      const int k1 = kt * 128 + 128;
#pragma unroll
      for (int s = 0; s < 8; ++s) {
        if (s == 3) fetch_codes(k1, 0);
        if (s == 7) {
          fetch_codes(k1, 1);
          ws[0][0] = ws[1][0];
          ws[0][1] = ws[1][1];
          w.scales(k1 + 128, ws[1]);
        }
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int m = 0; m < MI; ++m) {
#pragma unroll
          for (int i = 0; i < 2; ++i) acc[i][m] = mfma32(fragment(s, i), xf[m], acc[i][m]);
          load_x(s < 7 ? buf : next, (s + 1) & 7, m);
#pragma unroll
          for (int d = m * 4 / MI; d < (m + 1) * 4 / MI; ++d) decode((s + 1) & 7, ws[0], d);
#pragma unroll
          for (int i = 0; i < PIECES; ++i) {
            if (i % MI != m) continue;
            if (s == 2) {
              stage(i, next, 0);
              fetch(i, k1, 1);
            }
            if (s == 6) stage(i, next, 1);
            if (s == 7) fetch(i, k1 + 128, 0);
          }
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
  // chunk c of row t at c ^ (t % 16)) and leave as whole rows of 64 n's.
  nv_f4* out = reinterpret_cast<nv_f4*>(&lds[0][0]) + wave * 512;
  const int n = n0 + (lane & 15) * 4;
  float sc[4];
#pragma unroll
  for (int r = 0; r < 4; ++r) sc[r] = none || n + r >= a.N ? 0.0f : second_scale(a, e, n + r);
#pragma unroll
  for (int m = 0; m < MI; ++m) {
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int q = 0; q < 4; ++q)
        out[l32 * 16 + ((i * 8 + q * 2 + half) ^ (l32 & 15))] =
            nv_f4{acc[i][m][q * 4], acc[i][m][q * 4 + 1], acc[i][m][q * 4 + 2], acc[i][m][q * 4 + 3]};
    const int left = rows - m * 32 < 32 ? rows - m * 32 : 32;
#pragma unroll 1
    for (int t = lane >> 4; t < left; t += 4) {
      const nv_f4 v = out[t * 16 + ((lane & 15) ^ (t & 15))];
      store_out4(a, v[0] * sc[0], v[1] * sc[1], v[2] * sc[2], v[3] * sc[3], row0 + m * 32 + t, n);
    }
  }
}

template <bool MX8, int BLK, bool WORDS>
static void grouped_go(const MatmulArgs& a, int bm, hipStream_t st) {
  const uint32_t grid = (uint32_t)grouped_grid(a.T, a.ends ? a.E : 0, a.N, bm);
  if (bm == 128) k_grouped<MX8, BLK, 128, WORDS><<<grid, 256, 0, st>>>(a);
  else if (bm == 64) k_grouped<MX8, BLK, 64, WORDS><<<grid, 256, 0, st>>>(a);
  else k_grouped<MX8, BLK, 32, WORDS><<<grid, 256, 0, st>>>(a);
}

template <bool MX8, int BLK>
static void grouped_words(const MatmulArgs& a, int bm, hipStream_t st) {
  if (a.K % 32 == 0 && a.K >= 64) grouped_go<MX8, BLK, true>(a, bm, st);
  else grouped_go<MX8, BLK, false>(a, bm, st);
}

int launch_grouped(const MatmulArgs& a, void* stream) {
  hipStream_t st = (hipStream_t)stream;
  const int bm = grouped_rows(a.T, a.ends ? a.E : 1);
#define NV_GR(MX8) \
  (a.blocks == 0 ? grouped_words<MX8, 0>(a, bm, st) : a.blocks == 1 ? grouped_words<MX8, 1>(a, bm, st) : grouped_words<MX8, 2>(a, bm, st))
  if (a.xs) NV_GR(true);
  else NV_GR(false);
#undef NV_GR
  return (int)hipGetLastError();
}

}  // namespace nvfp4
