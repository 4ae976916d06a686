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
  int G, Hk, most;
  NV_DEV int operator()(bool real, int n, int) const {
    return !real || (int64_t)n * G <= most ? 0 : (int)(((int64_t)n * G + kAttendRows - 1) / kAttendRows) * Hk;
  }
};

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

template <int DP>
__global__ __launch_bounds__(256) void k_attend_tiles(const AttendArgs a) {
  constexpr int NQ = DP / 16, NT = DP / 32;  // steps of 16 along d; tiles of 32 of it
  constexpr int TILE = kKeys * DP * 2;       // bytes of a tile's keys, or values
  __shared__ __align__(16) uint8_t lds[4 * TILE];
  const int lane = threadIdx.x & 63, wv = uniform(threadIdx.x >> 6), col = lane & 31, half = lane >> 5;
  const int D = a.c.dim, Hk = a.c.heads, G = a.q.heads / Hk;
  const TileCount count{G, Hk, a.most};
  SequenceScan<TileCount> scan(a, count);
  Sequence s{};
  if (!scan.find(blockIdx.x, s)) return;
  // the last rows first: with a causal mask they have the most keys
  const int u = (int)blockIdx.x - s.first, h = u % Hk, units = (int)(((int64_t)s.n * G + kAttendRows - 1) / kAttendRows);
  const int m0 = (units - 1 - u / Hk) * kAttendRows;
  const int row = m0 + 32 * wv + col, mine = row / G;
  const bool real = mine < s.n;
  const int head = h * G + row - mine * G;
  nv_u4 raw[NQ];
  uint32_t big = 0;
#pragma unroll
  for (int i = 0; i < NQ; ++i) {
    const int d = 16 * i + 8 * half;
    raw[i] = (nv_u4){0, 0, 0, 0};
    if (real && d < D) raw[i] = *reinterpret_cast<const nv_u4*>((const uint16_t*)a.q.at + (int64_t)(s.q0 + mine) * a.q.token + head * a.q.head + d);
    big = amax_bits(raw[i], big);
  }
  {
    const uint32_t o = (uint32_t)__shfl_xor((int)big, 32, 64);
    big = o > big ? o : big;
  }
  const float factor = query_factor(big);
  nv_h8 Q[NQ];
#pragma unroll
  for (int i = 0; i < NQ; ++i) Q[i] = query_to_f16(raw[i], factor);
  const float kdec = a.c.ka ? a.c.ka[h] / 2688.0f : 1.0f, vdec = a.c.va ? a.c.va[h] / 2688.0f : 1.0f;
  const float by = a.scale * kLog2e / factor * kdec;
  const int limit = real ? seen_by(a, s, mine) : 0;
  // keys that the unit's rows see, and those that all of them do
  const int m1 = m0 + kAttendRows - 1, last = m1 / G < s.n ? m1 / G : s.n - 1;
  const int most = seen_by(a, s, last), least = seen_by(a, s, m0 / G);
  nv_f16 O[NT];
#pragma unroll
  for (int i = 0; i < NT; ++i)
#pragma unroll
    for (int r = 0; r < 16; ++r) O[i][r] = 0.0f;
  float m = -INFINITY, l = 0.0f;
  const int tiles = (most + kKeys - 1) / kKeys, tk = threadIdx.x >> 2, g4 = threadIdx.x & 3;
  RawTile<DP> next;
  int page = tk < s.L ? page_of(a, s, tk) : 0;
  if (tiles > 0) {
    next.load(a, page, h, tk, tk < s.L, g4);
    page = kKeys + tk < s.L ? page_of(a, s, kKeys + tk) : 0;
    next.store(lds, lds + TILE, tk, g4);
  }
  __syncthreads();
  for (int j = 0; j < tiles; ++j) {
    const uint8_t* K = lds + (j & 1) * 2 * TILE;
    const uint8_t* V = K + TILE;
    const int key0 = j * kKeys, nk = key0 + kKeys + tk;
    if (j + 1 < tiles) {
      next.load(a, page, h, nk, nk < s.L, g4);
      page = nk + kKeys < s.L ? page_of(a, s, nk + kKeys) : 0;
    }
    nv_f16 S[2];
#pragma unroll
    for (int t = 0; t < 2; ++t) {
#pragma unroll
      for (int r = 0; r < 16; ++r) S[t][r] = 0.0f;
#pragma unroll
      for (int i = 0; i < NQ; ++i) {
        const int key = 32 * t + col, c = 2 * i + half;
        const nv_h8 A = *reinterpret_cast<const nv_h8*>(K + key * DP * 2 + ((c ^ (key & 7)) << 4));
        S[t] = __builtin_amdgcn_mfma_f32_32x32x16_f16(A, Q[i], S[t], 0, 0, 0);
      }
    }
    float top = -INFINITY;
    const bool edge = key0 + kKeys > least;
#pragma unroll
    for (int t = 0; t < 2; ++t)
#pragma unroll
      for (int r = 0; r < 16; ++r) {
        float x = S[t][r] * by;
        if (edge) {
          const int key = key0 + 32 * t + 8 * (r / 4) + 4 * half + r % 4;
          x = key < limit ? x : -INFINITY;
        }
        S[t][r] = x;
        top = fmaxf(top, x);
      }
    top = other_half_max(top);
    const float mn = fmaxf(m, top), base = mn == -INFINITY ? 0.0f : mn;
    const float alpha = exp2_fast(m - base);
    m = mn;
    l *= alpha;
#pragma unroll
    for (int i = 0; i < NT; ++i)
#pragma unroll
      for (int r = 0; r < 16; ++r) O[i][r] *= alpha;
#pragma unroll
    for (int t = 0; t < 2; ++t)
#pragma unroll
      for (int q = 0; q < 2; ++q) {  // sixteen keys: 4 half + 0..3, and 8 more
        nv_u4 w;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float x = exp2_fast(S[t][8 * q + 2 * i] - base + kWeightBits), y = exp2_fast(S[t][8 * q + 2 * i + 1] - base + kWeightBits);
          l += x + y;
          w[i] = pack_f16(x, y);
        }
        const nv_h8 P = __builtin_bit_cast(nv_h8, w);
#pragma unroll
        for (int i = 0; i < NT; ++i) {
          nv_h4 part[2];
#pragma unroll
          for (int g = 0; g < 2; ++g) {
            const int c16 = lane & 15, key = 32 * t + 16 * q + 8 * g + 4 * half + (c16 >> 2);
            const int c = 4 * i + 2 * ((lane >> 4) & 1) + ((c16 & 3) >> 1);
            typedef __attribute__((address_space(3))) short lds_s;
            typedef short s4 __attribute__((ext_vector_type(4)));
            typedef __attribute__((address_space(3))) s4 lds_s4;
            const uint32_t off = (uint32_t)(uintptr_t)(lds_s*)(V + key * DP * 2 + ((c ^ (key & 7)) << 4) + 8 * (c16 & 1));
            part[g] = __builtin_bit_cast(nv_h4, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s4*)(uintptr_t)off));
          }
          O[i] = __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_shufflevector(part[0], part[1], 0, 1, 2, 3, 4, 5, 6, 7), P, O[i], 0, 0, 0);
        }
      }
    if (j + 1 < tiles) {
      uint8_t* to = lds + ((j + 1) & 1) * 2 * TILE;
      next.store(to, to + TILE, tk, g4);
    }
    __syncthreads();
  }
  l += __shfl_xor(l, 32, 64);
  if (!real) return;
  const float inv = l == 0.0f ? 0.0f : vdec / l;
  const int64_t out = (int64_t)(s.q0 + mine) * a.q.heads + head;
#pragma unroll
  for (int i = 0; i < NT; ++i)
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int d = 32 * i + 8 * r + 4 * half;
      if (d >= D) continue;
      nv_u2 w;
      w.x = pack_bf16(O[i][4 * r] * inv, O[i][4 * r + 1] * inv);
      w.y = pack_bf16(O[i][4 * r + 2] * inv, O[i][4 * r + 3] * inv);
      *reinterpret_cast<nv_u2*>(a.out + out * D + d) = w;
    }
  if (half == 0) a.lse[out] = l == 0.0f ? -INFINITY : (float)(kLn2 * ((double)m - kWeightBits + (double)__builtin_amdgcn_logf(l)));
}

template <int DP>
static int tiles_go(const AttendArgs& a, hipStream_t st) {
  const LayerLaunch p = plan_attend_tiles(a.T, a.B, a.q.heads, a.c.heads);
  k_attend_tiles<DP><<<(uint32_t)p.grid, p.block, 0, st>>>(a);
  return (int)hipGetLastError();
}

int launch_attend_tiles(const AttendArgs& a, hipStream_t st) {
  if (a.c.dim <= 64) return tiles_go<64>(a, st);
  if (a.c.dim <= 128) return tiles_go<128>(a, st);
  return tiles_go<256>(a, st);
}

}  // namespace nvfp4
