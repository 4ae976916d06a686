// Attention of many queries a sequence over an NVFP4 cache: prompts, pieces of
// prompts, a decoder's tokens over an encoder's states.  Formula and numbers as
// in k_attend_split.hip.
//
// Bound by what a wave does between the matrix instructions, which are at work 44% of
// the time (two prompts of 3201 and 8192 tokens, 32 heads on 8 of 128: 657 to 669 us, 945 to 965
// TFLOP/s of the 1300 that a large bf16 product reaches), and by shared memory, which they read for a
// third of it.  A unit is
// 32 rows a wave (queries, and heads that share keys) of one sequence and shared
// head.  Its keys pass in tiles of 64, decoded once for the workgroup into shared
// memory while the tile before is used, and read from memory two tiles ahead;
// scores are formed transposed (keys times queries), so a lane holds one query's
// scores, and its weights are an operand of the second product as they lie.
//
// Where units are few, the keys of each are shared by `parts` workgroups, which
// leave their sums in the workspace, and a second launch joins them in order.
#include "nvfp4_attend.hpp"

namespace nvfp4 {

struct TileCount {
  int G, Hk, most, rows;
  NV_DEV int operator()(bool real, int n, int) const {
    return !real || (int64_t)n * G <= most ? 0 : (int)(((int64_t)n * G + rows - 1) / rows) * Hk;
  }
};

constexpr int kKeys = 64;  // keys of a tile

// A lane's part of a tile of keys, or of values, as loaded: DP / 4 elements of one slot.
template <int DP>
struct RawTile {
  static constexpr int NS = DP / 32, PIECES = DP == 256 ? 2 : 1;
  uint32_t w[NS], s[PIECES];
  // page: that of the slot, or -1 (scores are NaN); in: the key is one of the sequence's
  NV_DEV void load(const CacheView& c, bool keys, int page, int h, int key, bool in, int g4) {
    const int D = c.dim;
#pragma unroll
    for (int i = 0; i < NS; ++i) w[i] = 0;
#pragma unroll
    for (int i = 0; i < PIECES; ++i) s[i] = in && page < 0 && keys ? kNanScales : 0;
    if (!in || page < 0) return;
    const int64_t row = (((int64_t)page * c.heads + h) << c.shift) + (key & ((1 << c.shift) - 1));
    const uint8_t *codes = (keys ? c.k : c.v) + row * (D / 2), *scales = (keys ? c.ks : c.vs) + row * (D / 16);
    if constexpr (DP == 64) {
      if (16 * g4 < D) {
        const nv_u2 x = *reinterpret_cast<const nv_u2*>(codes + 8 * g4);
        w[0] = x.x, w[1] = x.y;
        s[0] = scales[g4];
      }
    } else {
#pragma unroll
      for (int i = 0; i < PIECES; ++i) {
        const int d = 8 * NS * g4 + 32 * i;
        if (d < D) {
          const nv_u4 x = *reinterpret_cast<const nv_u4*>(codes + d / 2);
#pragma unroll
          for (int j = 0; j < 4; ++j) w[4 * i + j] = x[j];
          s[i] = *reinterpret_cast<const uint16_t*>(scales + d / 16);
        }
      }
    }
  }
  // Decoded to shared memory, chunk by chunk.
  NV_DEV void store(uint8_t* to, int key, int g4) const {
#pragma unroll
    for (int i = 0; i < NS; ++i) {
      const nv_h2 p = scale_pair(s[i / 4], false);
      *reinterpret_cast<nv_h8*>(to + key * DP * 2 + (((NS * g4 + i) ^ chunk_at(key)) << 4)) = fp4_to_f16(w[i], both((i & 2) ? p.y : p.x));
    }
  }
};

// W waves of 32 rows.  parts: workgroups that share a unit's keys at most.
template <int DP, int W>
__global__ __launch_bounds__(64 * W, DP == 256 ? 1 : 2) void k_attend_tiles(const AttendArgs a, int units, int parts) {
  constexpr int NQ = DP / 16, NT = DP / 32;  // steps of 16 along d; tiles of 32 of it
  constexpr int TILE = kKeys * DP * 2;       // bytes of a tile's keys, or values
  constexpr int ROWS = 32 * W;
  __shared__ __align__(16) uint8_t lds[4 * TILE];
  const int lane = threadIdx.x & 63, wv = uniform(threadIdx.x >> 6), col = lane & 31, half = lane >> 5;
  const int D = a.c.dim, Hk = a.c.heads, G = a.q.heads / Hk;
  const int split = blockIdx.x / units, unit = blockIdx.x - split * units;
  const TileCount count{G, Hk, a.most, ROWS};
  SequenceScan<TileCount> scan(a, count);
  Sequence s{};
  // pieces are as long for all units, so that the longest sequence has `parts` of them
  int per = 1 << 30;
  if (parts > 1) {
    scan.total();
    const int longest = (scan.longest + kKeys - 1) / kKeys, even = (longest + parts - 1) / parts;
    per = even > kAttendLeast ? even : kAttendLeast;
    scan.restart();
  }
  if (!scan.find(unit, s)) {
    if (parts > 1 && split == 0 && threadIdx.x == 0) tile_headers(a)[unit].parts = 0;
    return;
  }
  // the last rows first: with a causal mask they have the most keys
  const int u = unit - s.first, h = u % Hk, blocks = (int)(((int64_t)s.n * G + ROWS - 1) / ROWS);
  const int m0 = (blocks - 1 - u / Hk) * ROWS;
  // keys that the unit's rows see, and those that all of them do
  const int m1 = m0 + ROWS - 1, last = m1 / G < s.n ? m1 / G : s.n - 1;
  const int most = uniform(seen_by(a, s, last)), least = uniform(seen_by(a, s, m0 / G));
  const int all = (most + kKeys - 1) / kKeys;
  const int first = split * per, tiles = all - first > per ? first + per : all;
  const bool whole = all <= per;
  if (parts > 1 && split == 0 && threadIdx.x == 0) tile_headers(a)[unit] = {whole ? 0 : (all + per - 1) / per, m0, h, s.q0, s.n, {0, 0, 0}};
  if (split != 0 && first >= all) return;

  const int tk = (threadIdx.x & 255) >> 2, g4 = threadIdx.x & 3;
  // Of eight waves four load and decode: the others run ahead, and a SIMD's two are out of
  // step, one at its products while the other is not (eight, one side each: 660 -> 710 us,
  // two prompts of 8192).
  const bool loads = W == 4 || wv < 4;
  auto page_at = [&](int j) {
    const int key = j * kKeys + tk;
    return key < s.L ? page_of(a, s, key) : 0;
  };
  RawTile<DP> raw[2][2];
  auto load = [&](RawTile<DP>* r, int j, int page) {
    const int key = j * kKeys + tk;
    r[0].load(a.c, true, page, h, key, key < s.L, g4);
    r[1].load(a.c, false, page, h, key, key < s.L, g4);
  };
  auto store = [&](RawTile<DP>* r, int buf) {
    uint8_t* to = lds + buf * 2 * TILE;
#pragma unroll
    for (int i = 0; i < RawTile<DP>::PIECES; ++i) nan_to_key(r[0].s[i], r[1].s[i]);
    r[0].store(to, tk, g4);
    r[1].store(to + TILE, tk, g4);
  };
  int page = 0;
  if (first < tiles && loads) {
    load(raw[0], first, page_at(first));
    load(raw[1], first + 1, page_at(first + 1));
    page = page_at(first + 2);
  }

  const float kdec = a.c.ka ? a.c.ka[h] / 2688.0f : 1.0f, vdec = a.c.va ? a.c.va[h] / 2688.0f : 1.0f;
  const int row = m0 + 32 * wv + col, i = row / G, head = h * G + row - i * G;
  nv_h8 Q[NQ];
  float by;
  {
    nv_u4 x[NQ];
    uint32_t big = 0;
#pragma unroll
    for (int k = 0; k < NQ; ++k) {
      const int d = 16 * k + 8 * half;
      x[k] = (nv_u4){0, 0, 0, 0};
      if (i < s.n && d < D) x[k] = *reinterpret_cast<const nv_u4*>((const uint16_t*)a.q.at + (int64_t)(s.q0 + i) * a.q.token + head * a.q.head + d);
      big = amax_bits(x[k], big);
    }
    const uint32_t o = (uint32_t)__shfl_xor((int)big, 32, 64);
    const float factor = query_factor(o > big ? o : big), full = a.scale * kLog2e / factor * kdec;
    by = score_scale(full);
#pragma unroll
    for (int k = 0; k < NQ; ++k) Q[k] = query_to_f16(x[k], query_scale(factor, full));
  }
  const int limit = i < s.n ? seen_by(a, s, i) : 0;
  nv_f16 O[NT];
#pragma unroll
  for (int t = 0; t < NT; ++t)
#pragma unroll
    for (int r = 0; r < 16; ++r) O[t][r] = 0.0f;
  float m = -INFINITY, l = 0.0f;
  bool far = false;  // a row's scores are large
  if (first < tiles && loads) store(raw[0], 0);
  __syncthreads();

  // tile j from buffer buf; tile j + 2 into r, from where tile j was stored; then tile j + 1 from n
  auto tile = [&](int j, int buf, RawTile<DP>* r, RawTile<DP>* n) {
    const uint8_t* K = lds + buf * 2 * TILE;
    const uint8_t* V = K + TILE;
    const int key0 = j * kKeys;
    if (j + 2 < tiles && loads) {
      load(r, j + 2, page);
      page = page_at(j + 3);
    }
    // The two halves of the tile in turn: a product waits for the one before it only
    // every second time (two prompts of 8192: 660 us one half after the other, 652 so; heads of
    // 256: 501 and 478).
    nv_f16 S[2];
#pragma unroll
    for (int t = 0; t < 2; ++t)
#pragma unroll
      for (int e = 0; e < 16; ++e) S[t][e] = 0.0f;
#pragma unroll
    for (int k = 0; k < NQ; ++k)
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        const int key = 32 * t + col, c = 2 * k + half;
        const nv_h8 A = *reinterpret_cast<const nv_h8*>(K + key * DP * 2 + ((c ^ chunk_at(key)) << 4));
        S[t] = __builtin_amdgcn_mfma_f32_32x32x16_f16(A, Q[k], S[t], 0, 0, 0);
      }
    if (key0 + kKeys > least) {
      const int hidden = limit - key0 - 4 * half;
#pragma unroll
      for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int e = 0; e < 16; ++e)
          if (32 * t + 8 * (e / 4) + e % 4 >= hidden) S[t][e] = -INFINITY;
    }
    float top = -INFINITY;
#pragma unroll
    for (int t = 0; t < 2; ++t)
#pragma unroll
      for (int e = 0; e < 16; ++e) top = fmaxf(top, S[t][e]);
    top = half_max(top) * by;
    if (__builtin_amdgcn_ballot_w64(top - m > kSlack)) {
      const float mn = fmaxf(m, top), alpha = exp2_fast(m - (mn == -INFINITY ? 0.0f : mn));
      m = mn;
      l *= alpha;
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int e = 0; e < 16; ++e) O[t][e] *= alpha;
      far = __builtin_amdgcn_ballot_w64(far_up(m)) != 0;
    }
    float f = by, up = kWeightBits - (m == -INFINITY ? 0.0f : m);
    if (far) {
      const FarScores less(m, f, up);
#pragma unroll
      for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int e = 0; e < 16; ++e) S[t][e] = less(S[t][e]);
    }
#pragma unroll
    for (int t = 0; t < 2; ++t)
#pragma unroll
      for (int q = 0; q < 2; ++q) {  // sixteen keys: 4 half + 0..3, and 8 more
        nv_u4 w;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float x = exp2_fast(__builtin_fmaf(S[t][8 * q + 2 * e], f, up));
          const float y = exp2_fast(__builtin_fmaf(S[t][8 * q + 2 * e + 1], f, up));
          l += x + y;
          w[e] = pack_f16(x, y);
        }
        const nv_h8 P = __builtin_bit_cast(nv_h8, w);
#pragma unroll
        for (int k = 0; k < NT; ++k) {
          nv_h4 part[2];
#pragma unroll
          for (int g = 0; g < 2; ++g) {
            const int c16 = lane & 15, key = 32 * t + 16 * q + 8 * g + 4 * half + (c16 >> 2);
            const int c = 4 * k + 2 * ((lane >> 4) & 1) + ((c16 & 3) >> 1);
            part[g] = read_turned(V + key * DP * 2 + ((c ^ chunk_at(key)) << 4) + 8 * (c16 & 1));
          }
          O[k] = __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_shufflevector(part[0], part[1], 0, 1, 2, 3, 4, 5, 6, 7), P, O[k], 0, 0, 0);
        }
      }
    if (j + 1 < tiles && loads) store(n, buf ^ 1);
    __syncthreads();
  };
  for (int j = first; j < tiles; j += 2) {
    tile(j, 0, raw[0], raw[1]);
    if (j + 1 < tiles) tile(j + 1, 1, raw[1], raw[0]);
  }
  l += __shfl_xor(l, 32, 64);
  m = left_max(m, l, limit);
  if (i >= s.n) return;
  if (!whole) {
    float* part = tile_part(a, units, parts, ROWS, unit, split);
    const int r0 = 32 * wv + col;
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int d = 32 * t + 8 * r + 4 * half;
        if (d < D) *reinterpret_cast<nv_f4*>(part + r0 * D + d) = (nv_f4){O[t][4 * r], O[t][4 * r + 1], O[t][4 * r + 2], O[t][4 * r + 3]};
      }
    if (half == 0) {
      part[ROWS * D + r0] = m;
      part[ROWS * (D + 1) + r0] = l;
    }
    return;
  }
  const int64_t out = (int64_t)(s.q0 + i) * a.q.heads + head;
#pragma unroll
  for (int t = 0; t < NT; ++t)
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int d = 32 * t + 8 * r + 4 * half;
      if (d < D) write_row(a, out, d, (nv_f4){O[t][4 * r], O[t][4 * r + 1], O[t][4 * r + 2], O[t][4 * r + 3]}, m, l, vdec);
    }
}

void launch_attend_tiles(const AttendArgs& a, const TilesPlan& p, hipStream_t st) {
  const uint32_t grid = (uint32_t)(p.units * p.parts);
  const int units = (int)p.units;
  if (a.c.dim > 128) k_attend_tiles<256, 4><<<grid, 256, 0, st>>>(a, units, p.parts);
  else if (a.c.dim > 64 && p.waves == 8) k_attend_tiles<128, 8><<<grid, 512, 0, st>>>(a, units, p.parts);
  else if (a.c.dim > 64) k_attend_tiles<128, 4><<<grid, 256, 0, st>>>(a, units, p.parts);
  else k_attend_tiles<64, 4><<<grid, 256, 0, st>>>(a, units, p.parts);
}

}  // namespace nvfp4
