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
// sums join in shared memory, in a fixed order.
//
// With experts, the rows of each, and those of none (cleared), make tiles of 16
// (or 32), and the workgroups along grid y take all experts' tiles in turn.  T <=
// 16 E rows are at most 2 E + 1 tiles (T <= 96 E in 32s: 4 E + 1), so E + 1
// workgroups have two (four) each, however uneven the experts are.  Where a
// workgroup had all rows of one expert, 2048 rows of one of 128 experts 4096 x 2048
// took 637 us, now 139 (even: 194, 197); 512 of one of 32 150, now 34 (even 40, 39).
#include "nvfp4_experts.hpp"
#include "nvfp4_launch.hpp"
#include "nvfp4_plan.hpp"
#include "nvfp4_weight.hpp"

namespace nvfp4 {

// This wave's share of the products of 16 R rows of the weight with up to XR
// rows of x; own: its shared memory.
template <bool MX8, int BLK, bool WORDS, int R, int XR, int G>
NV_DEV void matvec_sums(const RowsView<MX8>& x, const WeightView<BLK>& w, int nk, nv_u4* own, int first, int lane,
                        nv_f4 acc[R][G]) {
  constexpr int W = kMatvecThreads / 64;
  RowsPiece<MX8, XR> xp;
  WeightPiece<BLK, WORDS> wp[R], wn[R];
  auto load = [&](int kt) {
#pragma unroll
    for (int r = 0; r < R; ++r) wn[r].load(w, r, lane, kt * 256);
    xp.load(x, lane, kt * 256);
  };
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
      if (RowsPiece<MX8, XR>::G == 1) {
        nv_bf8 xf[4];
        now.fragments(own, lane, 0, q, xf);
#pragma unroll
        for (int d = 0; d < 4; ++d)
#pragma unroll
          for (int r = 0; r < R; ++r) acc[r][0] = mfma16(wp[r].fragment(q, d), xf[d], acc[r][0]);
      } else {
        nv_bf8 wf[R][4];
#pragma unroll
        for (int r = 0; r < R; ++r)
#pragma unroll
          for (int d = 0; d < 4; ++d) wf[r][d] = wp[r].fragment(q, d);
#pragma unroll
        for (int g = 0; g < RowsPiece<MX8, XR>::G; ++g) {
          nv_bf8 xf[4];
          now.fragments(own, lane, g, q, xf);
#pragma unroll
          for (int d = 0; d < 4; ++d)
#pragma unroll
            for (int r = 0; r < R; ++r) acc[r][g] = mfma16(wf[r][d], xf[d], acc[r][g]);
        }
      }
    }
  }
}

// Clears `bytes` bytes.
__global__ __launch_bounds__(256) void k_zero(uint8_t* __restrict__ out, int64_t bytes) {
  const nv_u4 z = {0, 0, 0, 0};
  for (int64_t i = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 16; i < bytes; i += (int64_t)gridDim.x * 4096) {
    if (i + 16 <= bytes) *reinterpret_cast<nv_u4*>(out + i) = z;
    else
      for (int64_t j = i; j < bytes; ++j) out[j] = 0;
  }
}

// XM: rows of x that are taken at a time, 16 or 32.
template <bool MX8, int BLK, bool WORDS, int R, int XM, bool GROUPED>
__global__ __launch_bounds__(kMatvecThreads, XM == 16 ? 3 : 2) void k_matvec(MatmulArgs a) {
  constexpr int W = kMatvecThreads / 64, G = XM / 16;
  constexpr int ROWS = XM * (MX8 ? 16 : 32), SPAN = ROWS > R * 128 ? ROWS : R * 128;  // SPAN: 16-byte chunks of a wave's own memory
  static_assert(SPAN >= R * G * 64, "the sums fit where codes and rows go");
  __shared__ nv_u4 lds[W * SPAN];
  const int wave = uniform(threadIdx.x >> 6);
  const int n0 = (int)blockIdx.x * (16 * R);
  nv_u4* own = lds + wave * SPAN;
  int tiles = GROUPED ? a.T : (a.T + XM - 1) / XM;  // with experts their tiles, once known
  const int mine = GROUPED ? (int)blockIdx.y : 0;
  for (int unit = mine; unit < tiles; unit += GROUPED ? a.E + 1 : 1) {
    RowRange rr = {0, 0, a.T, 0};
    if (GROUPED) rr = range_of_tile(a.ends, a.E, a.T, XM, unit, tiles);
    const int t0 = (unit - rr.before) * XM, left = rr.rows - t0;
    if (left <= 0) return;
    if (unit != mine) __syncthreads();  // the sums are read before the next rows go where they lie
    int lane = threadIdx.x & 63;
    asm("" : "+v"(lane));  // else what follows from it stays in registers from tile to tile
    const bool none = GROUPED && rr.e >= a.E;
    const WeightView<BLK> w(a, none ? 0 : rr.e, n0, 16 * R);
    const int nk = none ? 0 : (a.K + 255) / 256;
    const int row0 = rr.row0 + t0, rows = left < XM ? left : XM;
    const RowsView<MX8> x(a, row0, rows);
    nv_f4 acc[R][G];
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
      for (int g = 0; g < G; ++g) acc[r][g] = nv_f4{0.0f, 0.0f, 0.0f, 0.0f};
    if (XM == 32 && rows > 16) matvec_sums<MX8, BLK, WORDS, R, XM, G>(x, w, nk, own, wave, lane, acc);
    else if (XM == 32 || rows > 4) matvec_sums<MX8, BLK, WORDS, R, 16, G>(x, w, nk, own, wave, lane, acc);
    else matvec_sums<MX8, BLK, WORDS, R, 4, G>(x, w, nk, own, wave, lane, acc);
    float* sums = reinterpret_cast<float*>(lds);  // of wave v: at v * SPAN * 4
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
      for (int g = 0; g < G; ++g) reinterpret_cast<nv_f4*>(own)[(r * G + g) * 64 + lane] = acc[r][g];
    __syncthreads();
    for (int i = threadIdx.x; i < R * G * 256; i += kMatvecThreads) {
      // lane l of a tile holds rows 4 (l / 16) + i % 4 of the weight for row l % 16 of x
      const int r = (i >> 8) / G, g = (i >> 8) % G, l = (i >> 2) & 63;
      const int n = n0 + r * 16 + (l >> 4) * 4 + (i & 3), t = g * 16 + (l & 15);
      if (n >= a.N || t >= rows) continue;
      float s = 0.0f;
#pragma unroll
      for (int v = 0; v < W; ++v) s += sums[v * SPAN * 4 + i];
      store_out(a, none ? 0.0f : s * second_scale(a, rr.e, n), row0 + t, n);
    }
    // Up to 16 rows alone are one tile.  Said to the compiler it saves 6% (1 x 4096 x
    // 4096: 4.8 -> 4.5 us), but two fragments spill (16 x 65536 x 7168: 57 -> 90).
    if (!GROUPED && XM == 16 && R != 2) return;
  }
}

template <bool MX8, int BLK, bool WORDS, int R, int XM>
static void matvec_go(const MatmulArgs& a, hipStream_t st) {
  const LayerLaunch p = plan_matvec(a.T, a.ends ? a.E : 0, a.N, MX8);
  const dim3 grid((uint32_t)p.grid, (uint32_t)p.y);
  if (a.ends) k_matvec<MX8, BLK, WORDS, R, XM, true><<<grid, p.block, 0, st>>>(a);
  else k_matvec<MX8, BLK, WORDS, R, XM, false><<<grid, p.block, 0, st>>>(a);
}

template <bool MX8, int BLK, bool WORDS>
static void matvec_size(const MatmulArgs& a, int r, bool more, hipStream_t st) {
  if (more) r == 2 ? matvec_go<MX8, BLK, WORDS, 2, 32>(a, st) : matvec_go<MX8, BLK, WORDS, 1, 32>(a, st);
  else if (r == 4) matvec_go<MX8, BLK, WORDS, 4, 16>(a, st);
  else r == 2 ? matvec_go<MX8, BLK, WORDS, 2, 16>(a, st) : matvec_go<MX8, BLK, WORDS, 1, 16>(a, st);
}

template <bool MX8>
static void matvec_blk(const MatmulArgs& a, int r, bool more, hipStream_t st) {
  const bool words = a.K % 64 == 0;
  if (a.blocks == 0) words ? matvec_size<MX8, 0, true>(a, r, more, st) : matvec_size<MX8, 0, false>(a, r, more, st);
  else if (a.blocks == 1) words ? matvec_size<MX8, 1, true>(a, r, more, st) : matvec_size<MX8, 1, false>(a, r, more, st);
  else matvec_size<MX8, 2, false>(a, r, more, st);
}

int launch_zero(void* out, int64_t bytes, void* stream) {
  const LayerLaunch p = plan_zero(bytes);
  k_zero<<<(uint32_t)p.grid, p.block, 0, (hipStream_t)stream>>>((uint8_t*)out, bytes);
  return (int)hipGetLastError();
}

int launch_matvec(const MatmulArgs& a, void* stream) {
  const int64_t E = a.ends ? a.E : 1;
  const int r = matvec_frags(a.T, a.N, E, a.xs != nullptr);
  const bool more = a.T > 16 * E;
  if (a.xs) matvec_blk<true>(a, r, more, (hipStream_t)stream);
  else matvec_blk<false>(a, r, more, (hipStream_t)stream);
  return (int)hipGetLastError();
}

}  // namespace nvfp4
