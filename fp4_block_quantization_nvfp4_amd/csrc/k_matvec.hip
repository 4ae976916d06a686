// Products of a few rows with 4-bit weights: out[t, n] = S_n sum_k x[t, k]
// v[n, k] s[n, k / 16], x bf16 or mx8, v the e2m1 value, s the block scale,
// S_n the second-level scale.  Bound by reading the weights once.
//
// A workgroup takes 16 R rows of the weight; its waves take every W-th piece
// of 128 k's, each lane one 16-byte load of codes (32 k's) a row, decoded in
// registers and multiplied on the matrix cores by up to 16 rows of x.  The
// waves' sums join in shared memory, in a fixed order.  With experts, grid y
// walks the experts and the rows of one are taken 16 at a time; the row of
// the grid past the last expert clears the rows that belong to none.
#include "nvfp4_experts.hpp"
#include "nvfp4_launch.hpp"
#include "nvfp4_plan.hpp"
#include "nvfp4_weight.hpp"

namespace nvfp4 {

template <bool MX8, int BLK, int R, bool GROUPED>
__global__ __launch_bounds__(kMatvecThreads) void k_matvec(MatmulArgs a) {
  constexpr int W = kMatvecThreads / 64;
  __shared__ float lds[W * R * 256];
  const int wave = uniform(threadIdx.x >> 6), lane = threadIdx.x & 63, l16 = lane & 15, grp = lane >> 4;
  const int n0 = (int)blockIdx.x * (16 * R);
  RowRange rr = {0, 0, a.T, 0};
  if (GROUPED) {
    if ((int)blockIdx.y < a.E) rr = expert_range(a.ends, a.T, blockIdx.y);
    else rr = expert_range(a.ends, a.T, a.E - 1), rr.row0 += rr.rows, rr.rows = a.T - rr.row0, rr.e = a.E;
  }
  if (rr.rows <= 0) return;
  const bool none = rr.e >= a.E;
  const WeightView<BLK> w(a, none ? 0 : rr.e, n0, 16 * R);
  const int nk = none ? 0 : (a.K + 127) / 128;
  for (int t0 = 0; t0 < rr.rows; t0 += 16) {
    const int row0 = rr.row0 + t0, rows = rr.rows - t0 < 16 ? rr.rows - t0 : 16;
    const RowsView<MX8> x(a, row0, rows);
    nv_f4 acc[R];
#pragma unroll
    for (int r = 0; r < R; ++r) acc[r] = nv_f4{0.0f, 0.0f, 0.0f, 0.0f};
    for (int kt = wave; kt < nk; kt += W) {
      const int k = kt * 128 + grp * 32;
      nv_bf8 xf[4];
      x.load32(l16, k, xf);
#pragma unroll
      for (int r = 0; r < R; ++r) {
        nv_bf8 wf[4];
        w.load32(r * 16 + l16, k, wf);
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[r] = mfma16(wf[j], xf[j], acc[r]);
      }
    }
    if (t0) __syncthreads();
#pragma unroll
    for (int r = 0; r < R; ++r) *reinterpret_cast<nv_f4*>(&lds[(wave * R + r) * 256 + lane * 4]) = acc[r];
    __syncthreads();
    for (int i = threadIdx.x; i < R * 256; i += kMatvecThreads) {
      float s = 0.0f;
#pragma unroll
      for (int v = 0; v < W; ++v) s += lds[v * R * 256 + i];
      // lane l of the tile holds rows 4 (l / 16) + i % 4 of the weight for row l % 16 of x
      const int r = i >> 8, l = (i >> 2) & 63;
      const int n = n0 + r * 16 + (l >> 4) * 4 + (i & 3), t = l & 15;
      if (n < a.N && t < rows) store_out(a, none ? 0.0f : s * second_scale(a, rr.e, n), row0 + t, n);
    }
  }
}

template <bool MX8, int BLK, int R>
static void matvec_go(const MatmulArgs& a, hipStream_t st) {
  const dim3 grid((uint32_t)ceil_div(a.N, 16 * R), a.ends ? (uint32_t)a.E + 1 : 1);
  if (a.ends) k_matvec<MX8, BLK, R, true><<<grid, kMatvecThreads, 0, st>>>(a);
  else k_matvec<MX8, BLK, R, false><<<grid, kMatvecThreads, 0, st>>>(a);
}

template <bool MX8>
static void matvec_blk(const MatmulArgs& a, int r, hipStream_t st) {
#define NV_MV(B) \
  (r == 4 ? matvec_go<MX8, B, 4>(a, st) : r == 2 ? matvec_go<MX8, B, 2>(a, st) : matvec_go<MX8, B, 1>(a, st))
  if (a.blocks == 0) NV_MV(0);
  else if (a.blocks == 1) NV_MV(1);
  else NV_MV(2);
#undef NV_MV
}

int launch_matvec(const MatmulArgs& a, void* stream) {
  const int r = matvec_frags(a.N, a.ends ? a.E : 1);
  if (a.xs) matvec_blk<true>(a, r, (hipStream_t)stream);
  else matvec_blk<false>(a, r, (hipStream_t)stream);
  return (int)hipGetLastError();
}

}  // namespace nvfp4
