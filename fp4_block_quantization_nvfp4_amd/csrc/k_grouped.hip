// Products of many rows with 4-bit weights, grouped by expert: for the rows
// t of expert e, out[t, n] = S_n sum_k x[t, k] v[n, k] s[n, k / 16] (see
// k_matvec.hip; without `ends` all rows belong to expert 0).
//
// A workgroup of four waves makes a tile of BM rows by 256 n's and walks k in
// steps of 128.  The rows of x are staged as bf16 in shared memory (two
// buffers, the loads of the next step in flight during the products of this
// one); each wave decodes the weights of its own 64 n's straight from global
// memory into fragments, so no weight is decoded twice in a workgroup and
// the weights cost no shared memory.  The weight is the first operand of the
// matrix product: a lane then holds four consecutive n's of one row.
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

template <bool MX8, int BLK, int BM>
__global__ __launch_bounds__(256, 2) void k_grouped(MatmulArgs a) {
  constexpr int MI = BM / 16;
  __shared__ uint16_t lds[2][BM * 128];
  const int tid = threadIdx.x, wave = uniform(tid >> 6), lane = tid & 63, l16 = lane & 15, grp = lane >> 4;
  const int ntiles = (a.N + 255) / 256;

  // this workgroup's tile
  int e = 0, row0, rows, n_tile;
  {
    const int total = a.ends ? count_tiles(a.ends, a.E, a.T, BM) : (a.T + BM - 1) / BM;
    const int64_t units = (int64_t)total * ntiles, per = (units + 7) / 8;
    const int64_t slot = blockIdx.x >> 3, unit = (blockIdx.x & 7) * per + slot;
    if (slot >= per || unit >= units) return;
    RowRange rr = {0, 0, a.T, 0};
    if (a.ends) rr = find_range(a.ends, a.E, a.T, BM, ntiles, unit);
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

  nv_f4 acc[4][MI];
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int m = 0; m < MI; ++m) acc[i][m] = nv_f4{0.0f, 0.0f, 0.0f, 0.0f};

  const int nk = none ? 0 : (a.K + 127) / 128;
  if (nk) {
    const WeightView<BLK> w(a, e, n0 < a.N ? n0 : 0, 64);
    const RowsView<MX8> x(a, row0, rows);
    // staging: 16-byte pieces of the step's x, piece p of a row
    constexpr int PR = MX8 ? 8 : 16, PIECES = BM * PR / 256 > 0 ? BM * PR / 256 : 1;
    constexpr bool ALL = BM * PR >= 256;
    nv_u4 st[PIECES];
    uint32_t sts[PIECES];
    auto fetch = [&](int k0) {
#pragma unroll
      for (int i = 0; i < PIECES; ++i) {
        const int id = tid + i * 256, r = id / PR, p = id % PR;
        if (!ALL && r >= BM) continue;
        if (MX8) {
          const int k = k0 + p * 16;
          st[i] = buf16(x.x, k < a.K ? (uint32_t)(r * a.K + k) : kOutside);
          sts[i] = buf1(x.s, k < a.K ? (uint32_t)(r * x.ns + k / kMxGroup) : kOutside);
        } else {
          const int k = k0 + p * 8;
          st[i] = buf16(x.x, k < a.K ? (uint32_t)(r * a.K + k) * 2u : kOutside);
        }
      }
    };
    // row r of a buffer: 16 chunks of 16 bytes, chunk c at c ^ (r % 16)
    auto put = [&](uint16_t* buf, int r, int c, nv_u4 v) {
      *reinterpret_cast<nv_u4*>(buf + r * 128 + ((c ^ (r & 15)) * 8)) = v;
    };
    auto stage = [&](uint16_t* buf) {
#pragma unroll
      for (int i = 0; i < PIECES; ++i) {
        const int id = tid + i * 256, r = id / PR, p = id % PR;
        if (!ALL && r >= BM) continue;
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
      }
    };
    nv_u4 wc[4];
    uint32_t ws[4][2];
    auto fetch_w = [&](int k0) {
      const int k = k0 + grp * 32;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        wc[i] = w.codes(i * 16 + l16, k);
        ws[i][0] = w.scale(i * 16 + l16, k);
        ws[i][1] = w.scale(i * 16 + l16, k + 16);
      }
    };
    fetch(0);
    fetch_w(0);
    stage(lds[0]);
    __syncthreads();
    for (int kt = 0; kt < nk; ++kt) {
      const uint16_t* buf = lds[kt & 1];
      nv_u4 c[4];
      float s[4][2];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        c[i] = wc[i];
        s[i][0] = __builtin_amdgcn_cvt_f32_fp8((int)ws[i][0], 0);
        s[i][1] = __builtin_amdgcn_cvt_f32_fp8((int)ws[i][1], 0);
      }
      const bool more = kt + 1 < nk;
      if (more) {
        fetch(kt * 128 + 128);
        fetch_w(kt * 128 + 128);
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        nv_bf8 wf[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) wf[i] = fp4_to_bf16(c[i][j], s[i][j >> 1]);
#pragma unroll
        for (int m = 0; m < MI; ++m) {
          const nv_bf8 xf = *reinterpret_cast<const nv_bf8*>(buf + (m * 16 + l16) * 128 + (((4 * grp + j) ^ l16) * 8));
#pragma unroll
          for (int i = 0; i < 4; ++i) acc[i][m] = mfma16(wf[i], xf, acc[i][m]);
        }
      }
      if (more) stage(lds[(kt + 1) & 1]);
      __syncthreads();
    }
  }
  if (n0 >= a.N) return;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int n = n0 + i * 16 + grp * 4;
    float sc[4];
#pragma unroll
    for (int r = 0; r < 4; ++r) sc[r] = none || n + r >= a.N ? 0.0f : second_scale(a, e, n + r);
#pragma unroll
    for (int m = 0; m < MI; ++m) {
      const int t = m * 16 + l16;
      if (t >= rows) continue;
      const nv_f4 v = none ? nv_f4{0.0f, 0.0f, 0.0f, 0.0f} : acc[i][m];
      store_out4(a, v[0] * sc[0], v[1] * sc[1], v[2] * sc[2], v[3] * sc[3], row0 + t, n);
    }
  }
}

template <bool MX8, int BLK>
static void grouped_go(const MatmulArgs& a, int bm, hipStream_t st) {
  const uint32_t grid = (uint32_t)grouped_grid(a.T, a.ends ? a.E : 0, a.N, bm);
  if (bm == 128) k_grouped<MX8, BLK, 128><<<grid, 256, 0, st>>>(a);
  else if (bm == 64) k_grouped<MX8, BLK, 64><<<grid, 256, 0, st>>>(a);
  else k_grouped<MX8, BLK, 32><<<grid, 256, 0, st>>>(a);
}

int launch_grouped(const MatmulArgs& a, void* stream) {
  hipStream_t st = (hipStream_t)stream;
  const int bm = grouped_rows(a.T, a.ends ? a.E : 1);
#define NV_GR(MX8) \
  (a.blocks == 0 ? grouped_go<MX8, 0>(a, bm, st) : a.blocks == 1 ? grouped_go<MX8, 1>(a, bm, st) : grouped_go<MX8, 2>(a, bm, st))
  if (a.xs) NV_GR(true);
  else NV_GR(false);
#undef NV_GR
  return (int)hipGetLastError();
}

}  // namespace nvfp4
