// Weight gradient of products grouped by expert: dw[e, n, k] = sum over the
// rows t of expert e of dy[t, n] x[t, k], dy bf16, x bf16 or mx8.
//
// The sum runs over rows, the slow axis of both operands, so both tiles are
// transposed on their way into shared memory: a lane takes a word (two bf16
// or four e4m3) of eight consecutive rows and writes, for each column, the
// eight rows as one 16-byte chunk.  A workgroup of four waves makes 256 n's by
// 128 k's and walks the rows 64 at a time, the next rows' loads in flight
// during the products.  x is the first operand: a lane then holds four
// consecutive k's of one n.  An expert without rows gets zeros.
#include "nvfp4_experts.hpp"
#include "nvfp4_launch.hpp"
#include "nvfp4_plan.hpp"

namespace nvfp4 {

constexpr int kWgN = 256, kWgK = 128, kWgT = 64;

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

template <bool MX8>
__global__ __launch_bounds__(256, 2) void k_wgrad(WgradArgs a) {
  __shared__ uint16_t ldy[kWgN * kWgT];
  __shared__ uint16_t lx[kWgK * kWgT];
  const int tid = threadIdx.x, wave = uniform(tid >> 6), lane = tid & 63, l16 = lane & 15, grp = lane >> 4;
  const int nk = (a.K + kWgK - 1) / kWgK, nn = (a.N + kWgN - 1) / kWgN;
  const int64_t units = (int64_t)a.E * nk * nn, per = (units + 7) / 8;
  const int64_t slot = blockIdx.x >> 3, unit = (blockIdx.x & 7) * per + slot;
  if (slot >= per || unit >= units) return;
  const int e = (int)(unit / ((int64_t)nk * nn)), in = (int)(unit - (int64_t)e * nk * nn);
  const int n0 = (in / nk) * kWgN, k0 = (in % nk) * kWgK;
  const RowRange rr = expert_range(a.ends, a.T, e);
  const int ns = (a.K + kMxGroup - 1) / kMxGroup;

  nv_f4 acc[8][4];  // 128 k's by this wave's 64 n's
#pragma unroll
  for (int i = 0; i < 8; ++i)
#pragma unroll
    for (int m = 0; m < 4; ++m) acc[i][m] = nv_f4{0.0f, 0.0f, 0.0f, 0.0f};

  constexpr int XI = MX8 ? 1 : 2;
  uint32_t vy[4][8], vx[XI][8], vs[8];
  const int64_t xp = MX8 ? a.K : 2 * (int64_t)a.K;
  auto fetch = [&](int t0) {
    const int rows = rr.rows - t0 < kWgT ? rr.rows - t0 : kWgT;
    const nv_buf by = make_buf((const char*)a.dy + (int64_t)(rr.row0 + t0) * 2 * a.N, (uint32_t)rows * 2u * (uint32_t)a.N);
    const nv_buf bx = make_buf((const char*)a.x + (int64_t)(rr.row0 + t0) * xp, (uint32_t)(rows * xp));
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int id = tid + i * 256, c = n0 + (id % 128) * 2, o = id / 128;
#pragma unroll
      for (int t = 0; t < 8; ++t) vy[i][t] = buf4(by, c < a.N ? ((uint32_t)(8 * o + t) * (uint32_t)a.N + c) * 2u : kOutside);
    }
    if (MX8) {
      const nv_buf bs = make_buf(a.xs + (int64_t)(rr.row0 + t0) * ns, (uint32_t)(rows * ns));
      const int c = k0 + (tid % 32) * 4, o = tid / 32;
#pragma unroll
      for (int t = 0; t < 8; ++t) {
        vx[0][t] = buf4(bx, c < a.K ? (uint32_t)(8 * o + t) * (uint32_t)a.K + c : kOutside);
        vs[t] = buf1(bs, c < a.K ? (uint32_t)(8 * o + t) * (uint32_t)ns + c / kMxGroup : kOutside);
      }
    } else {
#pragma unroll
      for (int i = 0; i < XI; ++i) {
        const int id = tid + i * 256, c = k0 + (id % 64) * 2, o = id / 64;
#pragma unroll
        for (int t = 0; t < 8; ++t) vx[i][t] = buf4(bx, c < a.K ? ((uint32_t)(8 * o + t) * (uint32_t)a.K + c) * 2u : kOutside);
      }
    }
  };
  auto put2 = [&](uint16_t* buf, int c, int o, const uint32_t v[8]) {
    nv_u4 c0, c1;
    transpose2(v, c0, c1);
    *reinterpret_cast<nv_u4*>(buf + wg_at(c, o)) = c0;
    *reinterpret_cast<nv_u4*>(buf + wg_at(c + 1, o)) = c1;
  };
  auto stage = [&]() {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int id = tid + i * 256;
      put2(ldy, (id % 128) * 2, id / 128, vy[i]);
    }
    if (MX8) {
      uint32_t lo[8], hi[8];
#pragma unroll
      for (int t = 0; t < 8; ++t) {
        const nv_u2 p = mx8_to_bf16(vx[0][t], e8m0_value(vs[t]));
        lo[t] = p.x;
        hi[t] = p.y;
      }
      put2(lx, (tid % 32) * 4, tid / 32, lo);
      put2(lx, (tid % 32) * 4 + 2, tid / 32, hi);
    } else {
#pragma unroll
      for (int i = 0; i < XI; ++i) {
        const int id = tid + i * 256;
        put2(lx, (id % 64) * 2, id / 64, vx[i]);
      }
    }
  };
  const int steps = (rr.rows + kWgT - 1) / kWgT;
  if (steps) fetch(0);
  for (int s = 0; s < steps; ++s) {
    stage();
    __syncthreads();
    if (s + 1 < steps) fetch((s + 1) * kWgT);
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      nv_bf8 yf[4];
#pragma unroll
      for (int m = 0; m < 4; ++m) yf[m] = *reinterpret_cast<const nv_bf8*>(ldy + wg_at(wave * 64 + m * 16 + l16, 4 * j + grp));
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const nv_bf8 xf = *reinterpret_cast<const nv_bf8*>(lx + wg_at(i * 16 + l16, 4 * j + grp));
#pragma unroll
        for (int m = 0; m < 4; ++m) acc[i][m] = mfma16(xf, yf[m], acc[i][m]);
      }
    }
    __syncthreads();
  }
#pragma unroll
  for (int m = 0; m < 4; ++m) {
    const int n = n0 + wave * 64 + m * 16 + l16;
    if (n >= a.N) continue;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int k = k0 + i * 16 + grp * 4;
      if (k >= a.K) continue;
      const int64_t at = ((int64_t)e * a.N + n) * a.K + k;
      const nv_f4 v = acc[i][m];
      if (a.out_bf16) *reinterpret_cast<nv_u2*>((uint16_t*)a.dw + at) = (nv_u2){pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3])};
      else *reinterpret_cast<nv_f4*>((float*)a.dw + at) = v;
    }
  }
}

int launch_wgrad(const WgradArgs& a, void* stream) {
  const int64_t units = a.E * ceil_div(a.N, kWgN) * ceil_div(a.K, kWgK);
  const dim3 grid((uint32_t)xcd_grid(units));
  if (a.xs) k_wgrad<true><<<grid, 256, 0, (hipStream_t)stream>>>(a);
  else k_wgrad<false><<<grid, 256, 0, (hipStream_t)stream>>>(a);
  return (int)hipGetLastError();
}

}  // namespace nvfp4
