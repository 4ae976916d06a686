// Products of a few rows with 4-bit weights: out[t, n] = S_n sum_k x[t, k]
// v[n, k] s[n, k / 16], x bf16 or mx8, v the e2m1 value, s the block scale,
// S_n the second-level scale.  Bound by reading the weights once.
//
// A workgroup takes 16 R rows of the weight; its waves take every W-th piece
// of 256 k's and multiply it on the matrix cores by up to 16 rows of x.  Both
// are read as whole lines (eight rows of 128 bytes of codes an instruction)
// and turned into fragments in shared memory: read by fragments, 16 rows of 64
// bytes, the same loop moves 2.3 TB/s instead of 4.8 (65536 x 7168, 16 rows).
// The next piece is in flight while one is decoded and multiplied.  The waves'
// sums join in shared memory, in a fixed order.  With experts, grid y walks
// the experts and the rows of one are taken 16 at a time; the row of the grid
// past the last expert clears the rows that belong to none.
#include "nvfp4_experts.hpp"
#include "nvfp4_launch.hpp"
#include "nvfp4_plan.hpp"
#include "nvfp4_weight.hpp"

namespace nvfp4 {

// This wave's share of the products of 16 R rows of the weight with up to XR
// rows of x; own: its shared memory.
template <bool MX8, int BLK, bool WORDS, int R, int XR>
NV_DEV void matvec_sums(const RowsView<MX8>& x, const WeightView<BLK>& w, int nk, nv_u4* own, nv_f4 acc[R]) {
  constexpr int W = kMatvecThreads / 64;
  const int lane = threadIdx.x & 63;
  RowsPiece<MX8, XR> xp;
  WeightPiece<BLK, WORDS> wp[R], wn[R];
  auto load = [&](int kt) {
#pragma unroll
    for (int r = 0; r < R; ++r) wn[r].load(w, r, lane, kt * 256);
    xp.load(x, lane, kt * 256);
  };
  const int first = uniform(threadIdx.x >> 6);
  load(first);
  for (int k = first; k < nk; k += W) {
#pragma unroll
    for (int r = 0; r < R; ++r) {
      wp[r] = wn[r];
      wp[r].turn(own + r * 128, lane);
    }
    const RowsPiece<MX8, XR> now = xp;
    now.put(own, lane);
    __builtin_amdgcn_sched_barrier(0);
    load(k + W);
    __builtin_amdgcn_sched_barrier(0);  // in flight during all of the products
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      nv_bf8 xf[4];
      now.fragments(own, lane, q, xf);
#pragma unroll
      for (int d = 0; d < 4; ++d)
#pragma unroll
        for (int r = 0; r < R; ++r) acc[r] = mfma16(wp[r].fragment(q, d), xf[d], acc[r]);
    }
  }
}

template <bool MX8, int BLK, bool WORDS, int R, bool GROUPED>
__global__ __launch_bounds__(kMatvecThreads, 3) void k_matvec(MatmulArgs a) {
  constexpr int W = kMatvecThreads / 64, SPAN = MX8 && R < 4 ? 256 : 512;  // SPAN: 16-byte chunks of a wave's own memory
  static_assert(SPAN >= R * 128, "the codes fit where x goes, and so do the sums");
  __shared__ nv_u4 lds[W * SPAN];
  const int wave = uniform(threadIdx.x >> 6), lane = threadIdx.x & 63;
  const int n0 = (int)blockIdx.x * (16 * R);
  RowRange rr = {0, 0, a.T, 0};
  if (GROUPED) {
    if ((int)blockIdx.y < a.E) rr = expert_range(a.ends, a.T, blockIdx.y);
    else rr = expert_range(a.ends, a.T, a.E - 1), rr.row0 += rr.rows, rr.rows = a.T - rr.row0, rr.e = a.E;
  }
  if (rr.rows <= 0) return;
  const bool none = rr.e >= a.E;
  const WeightView<BLK> w(a, none ? 0 : rr.e, n0, 16 * R);
  const int nk = none ? 0 : (a.K + 255) / 256;
  nv_u4* own = lds + wave * SPAN;
  for (int t0 = 0; t0 < rr.rows; t0 += 16) {
    const int row0 = rr.row0 + t0, rows = rr.rows - t0 < 16 ? rr.rows - t0 : 16;
    const RowsView<MX8> x(a, row0, rows);
    nv_f4 acc[R];
#pragma unroll
    for (int r = 0; r < R; ++r) acc[r] = nv_f4{0.0f, 0.0f, 0.0f, 0.0f};
    if (rows <= 4) matvec_sums<MX8, BLK, WORDS, R, 4>(x, w, nk, own, acc);
    else matvec_sums<MX8, BLK, WORDS, R, 16>(x, w, nk, own, acc);
    float* sums = reinterpret_cast<float*>(lds);  // of wave v: at v * SPAN * 4
#pragma unroll
    for (int r = 0; r < R; ++r) reinterpret_cast<nv_f4*>(own)[r * 64 + lane] = acc[r];
    __syncthreads();
    for (int i = threadIdx.x; i < R * 256; i += kMatvecThreads) {
      // lane l of the tile holds rows 4 (l / 16) + i % 4 of the weight for row l % 16 of x
      const int r = i >> 8, l = (i >> 2) & 63;
      const int n = n0 + r * 16 + (l >> 4) * 4 + (i & 3), t = l & 15;
      if (n >= a.N || t >= rows) continue;
      float s = 0.0f;
#pragma unroll
      for (int v = 0; v < W; ++v) s += sums[v * SPAN * 4 + i];
      store_out(a, none ? 0.0f : s * second_scale(a, rr.e, n), row0 + t, n);
    }
    if (t0 + 16 < rr.rows) __syncthreads();  // the sums are read before the next rows go where they lie
  }
}

template <bool MX8, int BLK, bool WORDS, int R>
static void matvec_go(const MatmulArgs& a, hipStream_t st) {
  const dim3 grid((uint32_t)ceil_div(a.N, 16 * R), a.ends ? (uint32_t)a.E + 1 : 1);
  if (a.ends) k_matvec<MX8, BLK, WORDS, R, true><<<grid, kMatvecThreads, 0, st>>>(a);
  else k_matvec<MX8, BLK, WORDS, R, false><<<grid, kMatvecThreads, 0, st>>>(a);
}

template <bool MX8>
static void matvec_blk(const MatmulArgs& a, int r, hipStream_t st) {
  const bool words = a.K % 64 == 0;
#define NV_MV(B, P) \
  (r == 4 ? matvec_go<MX8, B, P, 4>(a, st) : r == 2 ? matvec_go<MX8, B, P, 2>(a, st) : matvec_go<MX8, B, P, 1>(a, st))
  if (a.blocks == 0) words ? NV_MV(0, true) : NV_MV(0, false);
  else if (a.blocks == 1) words ? NV_MV(1, true) : NV_MV(1, false);
  else NV_MV(2, false);
#undef NV_MV
}

int launch_matvec(const MatmulArgs& a, void* stream) {
  const int r = matvec_frags(a.T, a.N, a.ends ? a.E : 1, a.xs != nullptr);
  if (a.xs) matvec_blk<true>(a, r, (hipStream_t)stream);
  else matvec_blk<false>(a, r, (hipStream_t)stream);
  return (int)hipGetLastError();
}

}  // namespace nvfp4
