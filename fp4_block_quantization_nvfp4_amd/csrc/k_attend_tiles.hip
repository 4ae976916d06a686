// Attention of many queries a sequence over an NVFP4 cache: prompts, pieces of
// prompts, a decoder's tokens over an encoder's states.  Formula and numbers as
// in k_attend_split.hip.
//
// Bound by the matrix cores and the vector instructions beside them.  A unit is
// 128 rows (queries, and heads that share keys) of one sequence and shared head,
// 32 to a wave.  Its keys pass in tiles of 64, decoded once for the workgroup
// into shared memory while the tile before is used; scores are formed transposed
// (keys times queries), so a lane holds one query's scores, and its weights are
// an operand of the second product as they lie.
#include "nvfp4_attend.hpp"

namespace nvfp4 {

struct TileCount {
  int G, Hk, most, rows;
  NV_DEV int operator()(bool real, int n, int) const {
    return !real || (int64_t)n * G <= most ? 0 : (int)(((int64_t)n * G + rows - 1) / rows) * Hk;
  }
};

#ifndef TILES_W
#define TILES_W 4
#define TILES_RB 1
#define TILES_OCC 2
#endif
constexpr int kKeys = 64;  // keys of a tile

// A lane's part of a tile as loaded: RUN elements of key tid / 4, and the same of the value.
template <int DP>
struct RawTile {
  static constexpr int NS = DP / 32;
  uint32_t k[NS], v[NS];
  uint32_t ks[DP == 256 ? 2 : 1], vs[DP == 256 ? 2 : 1];
  // page: that of the lane's key, or -1; in: the key is one of the sequence's
  NV_DEV void load(const AttendArgs& a, int page, int h, int key, bool in, int g4) {
    const int D = a.c.dim;
#pragma unroll
    for (int i = 0; i < NS; ++i) k[i] = v[i] = 0;
#pragma unroll
    for (int i = 0; i < (DP == 256 ? 2 : 1); ++i) ks[i] = vs[i] = 0;
    if (!in) return;
    if (page < 0) {  // no such page: scores are NaN
#pragma unroll
      for (int i = 0; i < (DP == 256 ? 2 : 1); ++i) ks[i] = kNanScales;
      return;
    }
    const int64_t row = (((int64_t)page * a.c.heads + h) << a.c.shift) + (key & ((1 << a.c.shift) - 1));
    const uint8_t *kc = a.c.k + row * (D / 2), *vc = a.c.v + row * (D / 2), *kb = a.c.ks + row * (D / 16), *vb = a.c.vs + row * (D / 16);
    if constexpr (DP == 64) {
      if (16 * g4 < D) {
        const nv_u2 x = *reinterpret_cast<const nv_u2*>(kc + 8 * g4), y = *reinterpret_cast<const nv_u2*>(vc + 8 * g4);
        k[0] = x.x, k[1] = x.y, v[0] = y.x, v[1] = y.y;
        ks[0] = kb[g4], vs[0] = vb[g4];
      }
    } else {
#pragma unroll
      for (int i = 0; i < NS / 4; ++i) {
        const int d = 8 * NS * g4 + 32 * i;
        if (d < D) {
          const nv_u4 x = *reinterpret_cast<const nv_u4*>(kc + d / 2), y = *reinterpret_cast<const nv_u4*>(vc + d / 2);
#pragma unroll
          for (int j = 0; j < 4; ++j) k[4 * i + j] = x[j], v[4 * i + j] = y[j];
          ks[i] = *reinterpret_cast<const uint16_t*>(kb + d / 16), vs[i] = *reinterpret_cast<const uint16_t*>(vb + d / 16);
        }
      }
    }
  }
  // Decoded to shared memory: eight elements c of a key at c ^ key.
  NV_DEV void store(uint8_t* K, uint8_t* V, int key, int g4) const {
#pragma unroll
    for (int i = 0; i < NS; ++i) {
      const int c = NS * g4 + i, at = key * DP * 2 + ((c ^ (key & 7)) << 4);
      const nv_h2 p = scale_pair(ks[i / 4], false), q = scale_pair(vs[i / 4], false);
      *reinterpret_cast<nv_h8*>(K + at) = fp4_to_f16(k[i], both((i & 2) ? p.y : p.x));
      *reinterpret_cast<nv_h8*>(V + at) = fp4_to_f16(v[i], both((i & 2) ? q.y : q.x));
    }
  }
};

// W waves, each with RB blocks of 32 rows.
template <int DP, int W, int RB>
__global__ __launch_bounds__(64 * W, TILES_OCC) void k_attend_tiles(const AttendArgs a) {
  constexpr int NQ = DP / 16, NT = DP / 32;  // steps of 16 along d; tiles of 32 of it
  constexpr int TILE = kKeys * DP * 2;       // bytes of a tile's keys, or values
  constexpr int ROWS = 32 * RB * W;
  __shared__ __align__(16) uint8_t lds[4 * TILE];
  const int lane = threadIdx.x & 63, wv = uniform(threadIdx.x >> 6), col = lane & 31, half = lane >> 5;
  const int D = a.c.dim, Hk = a.c.heads, G = a.q.heads / Hk;
  const TileCount count{G, Hk, a.most, ROWS};
  SequenceScan<TileCount> scan(a, count);
  Sequence s{};
  if (!scan.find(blockIdx.x, s)) return;
  // the last rows first: with a causal mask they have the most keys
  const int u = (int)blockIdx.x - s.first, h = u % Hk, units = (int)(((int64_t)s.n * G + ROWS - 1) / ROWS);
  const int m0 = (units - 1 - u / Hk) * ROWS;
  const float kdec = a.c.ka ? a.c.ka[h] / 2688.0f : 1.0f, vdec = a.c.va ? a.c.va[h] / 2688.0f : 1.0f;
  nv_h8 Q[RB][NQ];
  float by[RB], m[RB], l[RB];
  int limit[RB];
  nv_f16 O[RB][NT];
#pragma unroll
  for (int b = 0; b < RB; ++b) {
    const int row = m0 + 32 * (RB * wv + b) + col, i = row / G, head = h * G + row - i * G;
    nv_u4 raw[NQ];
    uint32_t big = 0;
#pragma unroll
    for (int k = 0; k < NQ; ++k) {
      const int d = 16 * k + 8 * half;
      raw[k] = (nv_u4){0, 0, 0, 0};
      if (i < s.n && d < D) raw[k] = *reinterpret_cast<const nv_u4*>((const uint16_t*)a.q.at + (int64_t)(s.q0 + i) * a.q.token + head * a.q.head + d);
      big = amax_bits(raw[k], big);
    }
    const uint32_t o = (uint32_t)__shfl_xor((int)big, 32, 64);
    const float factor = query_factor(o > big ? o : big);
#pragma unroll
    for (int k = 0; k < NQ; ++k) Q[b][k] = query_to_f16(raw[k], factor);
    by[b] = score_scale(a.scale * kLog2e / factor * kdec);
    limit[b] = i < s.n ? seen_by(a, s, i) : 0;
    m[b] = -INFINITY;
    l[b] = 0.0f;
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int r = 0; r < 16; ++r) O[b][t][r] = 0.0f;
  }
  // keys that the unit's rows see, and those that all of them do
  const int m1 = m0 + ROWS - 1, last = m1 / G < s.n ? m1 / G : s.n - 1;
  const int most = seen_by(a, s, last), least = seen_by(a, s, m0 / G);
  const int tiles = (most + kKeys - 1) / kKeys;
  const bool loads = threadIdx.x < 256;
  const int tk = (threadIdx.x & 255) >> 2, g4 = threadIdx.x & 3;
  RawTile<DP> next;
  int page = tk < s.L ? page_of(a, s, tk) : 0;
  if (tiles > 0 && loads) {
    next.load(a, page, h, tk, tk < s.L, g4);
    page = kKeys + tk < s.L ? page_of(a, s, kKeys + tk) : 0;
    next.store(lds, lds + TILE, tk, g4);
  }
  __syncthreads();
  for (int j = 0; j < tiles; ++j) {
    const uint8_t* K = lds + (j & 1) * 2 * TILE;
    const uint8_t* V = K + TILE;
    const int key0 = j * kKeys, nk = key0 + kKeys + tk;
    if (j + 1 < tiles && loads) {
      next.load(a, page, h, nk, nk < s.L, g4);
      page = nk + kKeys < s.L ? page_of(a, s, nk + kKeys) : 0;
    }
    nv_f16 S[RB][2];
#pragma unroll
    for (int t = 0; t < 2; ++t) {
#pragma unroll
      for (int b = 0; b < RB; ++b)
#pragma unroll
        for (int r = 0; r < 16; ++r) S[b][t][r] = 0.0f;
#pragma unroll
      for (int k = 0; k < NQ; ++k) {
        const int key = 32 * t + col, c = 2 * k + half;
        const nv_h8 A = *reinterpret_cast<const nv_h8*>(K + key * DP * 2 + ((c ^ (key & 7)) << 4));
#pragma unroll
        for (int b = 0; b < RB; ++b) S[b][t] = __builtin_amdgcn_mfma_f32_32x32x16_f16(A, Q[b][k], S[b][t], 0, 0, 0);
      }
    }
    if (key0 + kKeys > least) {
#pragma unroll
      for (int b = 0; b < RB; ++b)
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
          for (int r = 0; r < 16; ++r)
            if (key0 + 32 * t + 8 * (r / 4) + 4 * half + r % 4 >= limit[b]) S[b][t][r] = -INFINITY;
    }
    nv_h8 P[RB][2][2];
#pragma unroll
    for (int b = 0; b < RB; ++b) {
      float top = -INFINITY;
#pragma unroll
      for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int r = 0; r < 16; ++r) top = fmaxf(top, S[b][t][r]);
      top = half_max(top) * by[b];
      if (__builtin_amdgcn_ballot_w64(top > m[b] + kSlack)) {
        const float mn = fmaxf(m[b], top), alpha = exp2_fast(m[b] - (mn == -INFINITY ? 0.0f : mn));
        m[b] = mn;
        l[b] *= alpha;
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
          for (int r = 0; r < 16; ++r) O[b][t][r] *= alpha;
      }
      const float up = kWeightBits - (m[b] == -INFINITY ? 0.0f : m[b]);
#pragma unroll
      for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int q = 0; q < 2; ++q) {  // sixteen keys: 4 half + 0..3, and 8 more
          nv_u4 w;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float x = exp2_fast(__builtin_fmaf(S[b][t][8 * q + 2 * i], by[b], up));
            const float y = exp2_fast(__builtin_fmaf(S[b][t][8 * q + 2 * i + 1], by[b], up));
            l[b] += x + y;
            w[i] = pack_f16(x, y);
          }
          P[b][t][q] = __builtin_bit_cast(nv_h8, w);
        }
    }
#pragma unroll
    for (int t = 0; t < 2; ++t)
#pragma unroll
      for (int q = 0; q < 2; ++q)
#pragma unroll
        for (int i = 0; i < NT; ++i) {
          nv_h4 part[2];
#pragma unroll
          for (int g = 0; g < 2; ++g) {
            const int c16 = lane & 15, key = 32 * t + 16 * q + 8 * g + 4 * half + (c16 >> 2);
            const int c = 4 * i + 2 * ((lane >> 4) & 1) + ((c16 & 3) >> 1);
            part[g] = read_turned(V + key * DP * 2 + ((c ^ (key & 7)) << 4) + 8 * (c16 & 1));
          }
          const nv_h8 A = __builtin_shufflevector(part[0], part[1], 0, 1, 2, 3, 4, 5, 6, 7);
#pragma unroll
          for (int b = 0; b < RB; ++b) O[b][i] = __builtin_amdgcn_mfma_f32_32x32x16_f16(A, P[b][t][q], O[b][i], 0, 0, 0);
        }
    if (j + 1 < tiles && loads) {
      uint8_t* to = lds + ((j + 1) & 1) * 2 * TILE;
      next.store(to, to + TILE, tk, g4);
    }
    __syncthreads();
  }
#pragma unroll
  for (int b = 0; b < RB; ++b) {
    const float sum = l[b] + __shfl_xor(l[b], 32, 64);
    const int row = m0 + 32 * (RB * wv + b) + col, i = row / G, head = h * G + row - i * G;
    if (i >= s.n) continue;
    const float inv = sum == 0.0f ? 0.0f : vdec / sum;
    const int64_t out = (int64_t)(s.q0 + i) * a.q.heads + head;
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int d = 32 * t + 8 * r + 4 * half;
        if (d >= D) continue;
        nv_u2 w;
        w.x = pack_bf16(O[b][t][4 * r] * inv, O[b][t][4 * r + 1] * inv);
        w.y = pack_bf16(O[b][t][4 * r + 2] * inv, O[b][t][4 * r + 3] * inv);
        *reinterpret_cast<nv_u2*>(a.out + out * D + d) = w;
      }
    if (half == 0) a.lse[out] = sum == 0.0f ? -INFINITY : log_sum(m[b], sum);
  }
}

template <int DP>
static int tiles_go(const AttendArgs& a, hipStream_t st) {
  const LayerLaunch p = plan_attend_tiles(a.T, a.B, a.q.heads, a.c.heads);
  k_attend_tiles<DP, TILES_W, TILES_RB><<<(uint32_t)p.grid, 64 * TILES_W, 0, st>>>(a);
  return (int)hipGetLastError();
}

int launch_attend_tiles(const AttendArgs& a, hipStream_t st) {
  if (a.c.dim <= 64) return tiles_go<64>(a, st);
  if (a.c.dim <= 128) return tiles_go<128>(a, st);
  return tiles_go<256>(a, st);
}

}  // namespace nvfp4
