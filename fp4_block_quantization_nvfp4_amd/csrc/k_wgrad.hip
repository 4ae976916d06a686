// Weight gradient of products grouped by expert: dw[e, n, k] = sum over the
// rows t of expert e of dy[t, n] x[t, k], dy bf16, x bf16 or mx8.
//
// The sum runs over rows, the slow axis of both operands.  A workgroup of
// four waves makes 256 n's (or 128, below) by 128 k's and walks the rows 64 at
// a time.  Each wave has 64 n's (32) of its own and takes dy straight into
// registers: four (two) n's of eight rows a lane, turned into as many fragments
// by byte permutes.  x is shared and goes through shared memory (two buffers):
// a lane takes a word (two bf16 or four e4m3) of eight rows and writes, for
// each column, the eight rows as
// one 16-byte chunk.  Loads of the next step fill the registers that this one
// has just consumed.  x is the first operand: a lane then holds four
// consecutive k's of one n.  Each XCD takes an eighth of every expert's tiles,
// since experts differ in rows.  An expert without rows gets zeros.
#include "nvfp4_experts.hpp"
#include "nvfp4_launch.hpp"
#include "nvfp4_plan.hpp"

namespace nvfp4 {

constexpr int kWgT = 64;

// Chunk address (in 16-bit elements) of rows 8 o .. 8 o + 7 of column c.
NV_DEV int wg_at(int c, int o) { return c * kWgT + ((o ^ ((c >> 1) & 7)) * 8); }

// Words of eight rows, two bf16 each -> the two columns' chunks.
NV_DEV void transpose2(const uint32_t v[8], nv_u4& c0, nv_u4& c1) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    c0[i] = __builtin_amdgcn_perm(v[2 * i + 1], v[2 * i], 0x05040100u);
    c1[i] = __builtin_amdgcn_perm(v[2 * i + 1], v[2 * i], 0x07060302u);
  }
}

// SPLIT: blocks of a.block rows of an expert are units of their own.  An expert
// of one block is written as without; the sums of more go to a.part, by the
// number of the block, and k_wgrad_join adds them.
// NM: n's of a lane.  Two instead of four (tiles of 128 n's) where experts have
// few rows or tiles are few: workgroups need half the registers, twice as many
// run at a time (8 experts 2048 x 2048, 16 rows each: 18.9 -> 15.3 us; 1777 rows,
// 5 experts 1040 x 528: 21.1 -> 19.1).
template <bool MX8, bool SPLIT, int NM>
__global__ __launch_bounds__(256, NM == 4 ? 2 : MX8 ? 3 : 4) void k_wgrad(WgradArgs a) {
  __shared__ uint16_t lx[2][kWgK * kWgT];
  const int tid = threadIdx.x, wave = uniform(tid >> 6), lane = tid & 63, l16 = lane & 15, grp = lane >> 4;
  const int nk = (a.K + kWgK - 1) / kWgK, nn = (a.N + 64 * NM - 1) / (64 * NM);
  int e, in, part = -1;
  RowRange rr;
  if (SPLIT) {
    int64_t unit;
    int whole;
    rr = find_unit<false>(a.ends, a.E, a.T, a.block, nk * nn, blockIdx.x, unit, whole);
    if (rr.rows <= 0 || rr.e >= a.E) return;
    e = rr.e;
    const int local = (int)(unit - (int64_t)rr.before * (nk * nn)), block = local / (nk * nn);
    in = local - block * (nk * nn);
    if (rr.rows > a.block) {
      part = rr.before + block;
      rr.row0 += block * a.block;
      rr.rows = rr.rows - block * a.block < a.block ? rr.rows - block * a.block : a.block;
    }
  } else {
    const int share = (nk * nn + 7) / 8, slot = blockIdx.x >> 3;  // share: tiles of one expert on one XCD
    e = slot / share;
    in = (blockIdx.x & 7) * share + slot % share;
    if (in >= nk * nn) return;
    rr = expert_range(a.ends, a.T, e);
  }
  const int n0 = (in / nk) * (64 * NM), k0 = (in % nk) * kWgK;
  const int ns = (a.K + kMxGroup - 1) / kMxGroup;

  nv_f4 acc[8][NM];  // 128 k's by this wave's 16 NM n's
#pragma unroll
  for (int i = 0; i < 8; ++i)
#pragma unroll
    for (int m = 0; m < NM; ++m) acc[i][m] = nv_f4{0.0f, 0.0f, 0.0f, 0.0f};

  // dy: rows 32 j + 8 grp + t of the step, n's nl .. nl + NM - 1
  const int nl = n0 + wave * (16 * NM) + NM * l16;
  const uint32_t yat = nl < a.N ? (uint32_t)(8 * grp) * (uint32_t)a.N * 2u + (uint32_t)nl * 2u : kOutside;
  uint32_t vy[2][NM / 2][8];
  auto fetch_y = [&](int t0, int j) {
    const int left = rr.rows - t0, rows = left < 0 ? 0 : left < kWgT ? left : kWgT;
    const nv_buf by = make_buf((const char*)a.dy + (int64_t)(rr.row0 + t0) * 2 * a.N, (uint32_t)rows * 2u * (uint32_t)a.N);
#pragma unroll
    for (int t = 0; t < 8; ++t) {
      const uint32_t at = yat + (uint32_t)(32 * j + t) * (uint32_t)a.N * 2u;
      if (NM == 4) {
        const nv_u2 v = buf8(by, at);
        vy[j][0][t] = v.x;
        vy[j][NM / 2 - 1][t] = v.y;
      } else {
        vy[j][0][t] = buf4(by, at);
      }
    }
  };
  // x: words of eight consecutive rows
  constexpr int XI = MX8 ? 1 : 2, XW = MX8 ? 32 : 64, XE = MX8 ? 4 : 2;  // words a row, elements a word
  uint32_t vx[XI][8], vs[8];
  const uint32_t xp = MX8 ? (uint32_t)a.K : 2u * (uint32_t)a.K;
  auto fetch_x = [&](int t0) {
    const int left = rr.rows - t0, rows = left < 0 ? 0 : left < kWgT ? left : kWgT;
    const nv_buf bx = make_buf((const char*)a.x + (int64_t)(rr.row0 + t0) * xp, (uint32_t)rows * xp);
#pragma unroll
    for (int i = 0; i < XI; ++i) {
      const int id = tid + i * 256, c = k0 + (id % XW) * XE, o = id / XW;
      const uint32_t at = c < a.K ? (uint32_t)(8 * o) * xp + (uint32_t)(id % XW) * 4u + (uint32_t)(k0 * (MX8 ? 1 : 2)) : kOutside;
#pragma unroll
      for (int t = 0; t < 8; ++t) vx[i][t] = buf4(bx, at + (uint32_t)t * xp);
    }
    if (MX8) {
      const nv_buf bs = make_buf(a.xs + (int64_t)(rr.row0 + t0) * ns, (uint32_t)(rows * ns));
      const int c = k0 + (tid % 32) * 4, o = tid / 32;
      const uint32_t at = c < a.K ? (uint32_t)(8 * o) * (uint32_t)ns + (uint32_t)(c / kMxGroup) : kOutside;
#pragma unroll
      for (int t = 0; t < 8; ++t) vs[t] = buf1(bs, at + (uint32_t)(t * ns));
    }
  };
  auto put2 = [&](uint16_t* buf, int c, int o, const uint32_t v[8]) {
    nv_u4 c0, c1;
    transpose2(v, c0, c1);
    *reinterpret_cast<nv_u4*>(buf + wg_at(c, o)) = c0;
    *reinterpret_cast<nv_u4*>(buf + wg_at(c + 1, o)) = c1;
  };
  auto stage_x = [&](uint16_t* buf) {
    if (MX8) {
      uint32_t lo[8], hi[8];
#pragma unroll
      for (int t = 0; t < 8; ++t) {
        const nv_u2 p = mx8_to_bf16(vx[0][t], e8m0_scale(vs[t]));
        lo[t] = p.x;
        hi[t] = p.y;
      }
      put2(buf, (tid % 32) * 4, tid / 32, lo);
      put2(buf, (tid % 32) * 4 + 2, tid / 32, hi);
    } else {
#pragma unroll
      for (int i = 0; i < XI; ++i) {
        const int id = tid + i * 256;
        put2(buf, (id % 64) * 2, id / 64, vx[i]);
      }
    }
  };
  const int steps = (rr.rows + kWgT - 1) / kWgT;
  if (steps) {
    fetch_x(0);
    fetch_y(0, 0);
    fetch_y(0, 1);
    stage_x(lx[0]);
    __syncthreads();
  }
  for (int s = 0; s < steps; ++s) {
    const uint16_t* buf = lx[s & 1];
    const int t1 = (s + 1) * kWgT;  // past the last row every load is outside and gives zeros
    fetch_x(t1);
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      nv_bf8 yf[NM];
#pragma unroll
      for (int p = 0; p < NM / 2; ++p) {
        nv_u4 c0, c1;
        transpose2(vy[j][p], c0, c1);
        yf[2 * p] = __builtin_bit_cast(nv_bf8, c0);
        yf[2 * p + 1] = __builtin_bit_cast(nv_bf8, c1);
      }
      fetch_y(t1, j);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const nv_bf8 xf = *reinterpret_cast<const nv_bf8*>(buf + wg_at(i * 16 + l16, 4 * j + grp));
#pragma unroll
        for (int m = 0; m < NM; ++m) acc[i][m] = mfma16(xf, yf[m], acc[i][m]);
      }
    }
    stage_x(lx[(s + 1) & 1]);
    __syncthreads();
  }
  // A lane holds, of each fragment pair (i, m), k = 16 i + 4 grp + 0..3 of n =
  // NM l16 + m.  16 n's at a time go through the wave's part of shared memory
  // (16-byte chunk c of row l16 at c ^ l16) and leave as rows of 128 k's.
  nv_f4* out = reinterpret_cast<nv_f4*>(&lx[0][0]) + wave * 512;
  const int k = k0 + (lane & 31) * 4;
#pragma unroll
  for (int m = 0; m < NM; ++m) {
#pragma unroll
    for (int i = 0; i < 8; ++i) out[l16 * 32 + ((4 * i + grp) ^ l16)] = acc[i][m];
#pragma unroll 8
    for (int r = lane >> 5; r < 16; r += 2) {
      const int n = n0 + wave * (16 * NM) + NM * r + m;
      const nv_f4 v = out[r * 32 + ((lane & 31) ^ r)];
      if (n >= a.N || k >= a.K) continue;
      const int64_t at = ((int64_t)(part < 0 ? e : part) * a.N + n) * a.K + k;
      if (SPLIT && part >= 0) *reinterpret_cast<nv_f4*>(a.part + at) = v;
      else if (a.out_bf16) stream_out(reinterpret_cast<nv_u2*>((uint16_t*)a.dw + at), (nv_u2){pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3])});
      else stream_out(reinterpret_cast<nv_f4*>((float*)a.dw + at), v);
    }
  }
}

// Adds the blocks of each expert that has several, in their order, and clears
// the gradient of those without rows.  Grid y walks the experts.
__global__ __launch_bounds__(256) void k_wgrad_join(WgradArgs a) {
  const int e = blockIdx.y;
  RangeScan s(a.ends, a.E, a.T, a.block);
  while (s.next() && s.base <= e) {
  }
  const int l = e & 63;  // the scan holds e's 64
  const int rows = uniform(__shfl(s.count, l, 64)), blocks = uniform(__shfl(s.own, l, 64));
  const int64_t first = uniform(__shfl(s.first, l, 64)), size = (int64_t)a.N * a.K;
  if (rows > 0 && blocks == 1) return;
  for (int64_t i = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 4; i < size; i += (int64_t)gridDim.x * 1024) {
    nv_f4 v = {0.0f, 0.0f, 0.0f, 0.0f};
    const float* p = a.part + first * size + i;
#pragma unroll 4
    for (int b = 0; b < blocks; ++b) {
      const nv_f4 w = *reinterpret_cast<const nv_f4*>(p + b * size);
#pragma unroll
      for (int r = 0; r < 4; ++r) v[r] += w[r];
    }
    const int64_t at = e * size + i;
    if (a.out_bf16) *reinterpret_cast<nv_u2*>((uint16_t*)a.dw + at) = (nv_u2){pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3])};
    else *reinterpret_cast<nv_f4*>((float*)a.dw + at) = v;
  }
}

template <bool MX8>
static void wgrad_go(const WgradArgs& a, hipStream_t st) {
  const LayerLaunch p = plan_wgrad(a.T, a.E, a.N, a.K, a.block);
  const uint32_t grid = (uint32_t)p.grid;
  if (a.block) {
    k_wgrad<MX8, true, 4><<<grid, p.block, 0, st>>>(a);
    const LayerLaunch j = plan_wgrad_join(a.E, a.N, a.K);
    k_wgrad_join<<<dim3((uint32_t)j.grid, (uint32_t)j.y), j.block, 0, st>>>(a);
  } else if (wgrad_narrow(a.T, a.E, ceil_div(a.N, kWgN) * ceil_div(a.K, kWgK))) {
    k_wgrad<MX8, false, 2><<<grid, p.block, 0, st>>>(a);
  } else {
    k_wgrad<MX8, false, 4><<<grid, p.block, 0, st>>>(a);
  }
}

int launch_wgrad(const WgradArgs& a, void* stream) {
  if (a.xs) wgrad_go<true>(a, (hipStream_t)stream);
  else wgrad_go<false>(a, (hipStream_t)stream);
  return (int)hipGetLastError();
}

}  // namespace nvfp4
