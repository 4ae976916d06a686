// Attention of few queries a sequence over an NVFP4 cache: decoding.
//
//   s_j = scale q . k_j for the keys j that the query sees, p = softmax(s),
//   out = sum_j p_j v_j, lse = log sum_j exp(s_j); without keys 0 and -inf
//
// Bound by reading the cache, 9/16 byte an element.  The queries of a sequence
// and of the heads that share keys form rows, sixteen to a unit; a unit's keys
// are tiles of 128.  All tiles of all units are one line, cut into as many even
// pieces as there are workgroups, whatever the sequences' lengths: a long one is
// shared by many, short ones are taken several by one.  A unit that lies in
// several pieces leaves its parts (sums, maxima) in the workspace, and a second
// launch joins them in order.
//
// Of a tile a wave takes 32 keys: keys times queries (transposed, a lane has one
// query's scores), the running maximum and sum of the softmax, weights back into
// the matrix cores as they lie, with values read across from shared memory
// (turned by the load).  The four waves keep sums of their own and join at the
// piece's end.
#include "nvfp4_attend.hpp"

namespace nvfp4 {

struct SplitCount {
  int G, Hk, most, tile;
  // units of a sequence times their tiles of keys; a unit without keys counts as one
  NV_DEV int units(int n) const { return (int)(((int64_t)n * G + 15) / 16) * Hk; }
  NV_DEV int tiles(int L) const { return L > 0 ? (L + tile - 1) / tile : 1; }
  NV_DEV int operator()(bool real, int n, int L) const { return real && (int64_t)n * G > most ? 0 : units(n) * tiles(L); }
};

// Piece i of `total` tiles among `pieces`.
NV_DEV int piece_start(int total, int pieces, int i) { return (int)((int64_t)total * i / pieces); }

// A partial result: sixteen rows of D sums, then their maxima, then their sums of weights.
NV_DEV int64_t part_size(int D) { return 16 * (int64_t)D + 32; }

// Sixteen rows of unit `unit` of sequence s: row r is query r / G, head r % G of the unit's shared head.
struct UnitRow {
  int token, head;  // token -1: no such row
};
NV_DEV UnitRow unit_row(const Sequence& s, int G, int Hk, int unit, int r) {
  const int h = unit % Hk, m = unit / Hk * 16 + r, i = m / G;
  return {i < s.n ? s.q0 + i : -1, h * G + m - i * G};
}

NV_DEV void write_row(const AttendArgs& a, const UnitRow& u, int d, nv_f4 o, float m, float l, float vdec) {
  if (u.token < 0 || d >= a.c.dim) return;
  const float inv = l == 0.0f ? 0.0f : vdec / l;
  const int64_t row = (int64_t)u.token * a.q.heads + u.head;
  nv_u2 w;
  w.x = pack_bf16(o[0] * inv, o[1] * inv);
  w.y = pack_bf16(o[2] * inv, o[3] * inv);
  *reinterpret_cast<nv_u2*>(a.out + row * a.c.dim + d) = w;
  if (d == 0) a.lse[row] = l == 0.0f ? -INFINITY : (float)(kLn2 * ((double)m - kWeightBits + (double)__builtin_amdgcn_logf(l)));
}

template <int DP>
struct SplitShape {
  static constexpr int NS = DP / 32, NT = DP / 16;        // steps of 32 along d; tiles of 16 of it
  static constexpr int RUN = DP / 4;                      // elements of a key that a lane loads
  static constexpr int ROW = DP + 4;                      // floats of a row of sums in shared memory
  static constexpr int WAVE = 16 * ROW * 4 > 32 * DP * 2 ? 16 * ROW * 4 : 32 * DP * 2;
};

// Raw keys or values of 16 slots: a lane has RUN elements of key lane % 16.
template <int DP>
struct RawKeys {
  static constexpr int NS = DP / 32;
  uint32_t w[NS];
  uint32_t s[DP == 256 ? 2 : 1];
  NV_DEV void load(const uint8_t* codes, const uint8_t* scales, const AttendArgs& a, int page, int h, int at, int rows, int lane) {
    const int D = a.c.dim, grp = lane >> 4;
    const int64_t row0 = ((int64_t)page * a.c.heads + h) << a.c.shift;
    const nv_buf cb = make_buf(codes + row0 * (D / 2), (uint32_t)rows * (uint32_t)(D / 2));
    const nv_buf sb = make_buf(scales + row0 * (D / 16), (uint32_t)rows * (uint32_t)(D / 16));
    const uint32_t r = (uint32_t)(at + (lane & 15));
    const uint32_t co = r * (uint32_t)(D / 2), so = r * (uint32_t)(D / 16);
    if constexpr (DP == 64) {
      const bool in = 16 * grp < D;
      const nv_u2 v = buf8(cb, in ? co + 8 * grp : kOutside);
      w[0] = v.x;
      w[1] = v.y;
      s[0] = buf1(sb, in ? so + grp : kOutside);
    } else {
#pragma unroll
      for (int i = 0; i < NS / 4; ++i) {
        const int d = 8 * NS * grp + 32 * i;
        const bool in = d < D;
        const nv_u4 v = buf16(cb, in ? co + d / 2 : kOutside);
#pragma unroll
        for (int j = 0; j < 4; ++j) w[4 * i + j] = v[j];
        s[i] = (uint32_t)(uint16_t)__builtin_amdgcn_raw_buffer_load_b16(sb.at, (int)(in ? so + d / 16 : kOutside), 0, 0);
      }
    }
  }
  // Elements 8 i .. 8 i + 7 of the run.
  NV_DEV nv_h8 values(int i) const {
    const nv_h2 p = scale_pair(s[i / 4], false);
    return fp4_to_f16(w[i], both((i & 2) ? p.y : p.x));
  }
};

template <int DP>
__global__ __launch_bounds__(256) void k_attend_split(const AttendArgs a) {
  using S = SplitShape<DP>;
  constexpr int NS = S::NS, NT = S::NT;
  __shared__ __align__(16) uint8_t lds[4][S::WAVE];
  __shared__ float stat[2][4][16];
  const int lane = threadIdx.x & 63, wv = uniform(threadIdx.x >> 6), col = lane & 15, grp = lane >> 4;
  const int D = a.c.dim, Hk = a.c.heads, G = a.q.heads / Hk;
  const SplitCount count{G, Hk, a.most, 128};
  SequenceScan<SplitCount> scan(a, count);
  const int total = scan.total();
  int tile = piece_start(total, gridDim.x, blockIdx.x);
  const int stop = piece_start(total, gridDim.x, blockIdx.x + 1);
  if (tile >= stop) return;
  scan.restart();
  Sequence q{};
  while (tile < stop) {
    if (!scan.find(tile, q)) break;
    const int kt = count.tiles(q.L), u = (tile - q.first) / kt, j0 = tile - q.first - u * kt;
    const int j1 = j0 + (stop - tile) < kt ? j0 + (stop - tile) : kt;
    const int h = u % Hk;
    const UnitRow mine = unit_row(q, G, Hk, u, col);
    // a lane's query: RUN elements of row `col`
    nv_u4 raw[NS];
    uint32_t big = 0;
#pragma unroll
    for (int i = 0; i < NS; ++i) {
      const int d = S::RUN * grp + 8 * i;
      raw[i] = (nv_u4){0, 0, 0, 0};
      if (mine.token >= 0 && d < D)
        raw[i] = *reinterpret_cast<const nv_u4*>((const uint16_t*)a.q.at + mine.token * a.q.token + mine.head * a.q.head + d);
      big = amax_bits(raw[i], big);
    }
    {
      const uint32_t o = (uint32_t)__shfl_xor((int)big, 16, 64);
      big = o > big ? o : big;
      const uint32_t p = (uint32_t)__shfl_xor((int)big, 32, 64);
      big = p > big ? p : big;
    }
    const float factor = query_factor(big);
    nv_h8 Q[NS];
#pragma unroll
    for (int i = 0; i < NS; ++i) Q[i] = query_to_f16(raw[i], factor);
    const float kdec = a.c.ka ? a.c.ka[h] / 2688.0f : 1.0f, vdec = a.c.va ? a.c.va[h] / 2688.0f : 1.0f;
    const float by = a.scale * kLog2e / factor * kdec;
    const int limit = mine.token < 0 ? 0 : seen_by(a, q, mine.token - q.q0);
    nv_f4 O[NT];
#pragma unroll
    for (int i = 0; i < NT; ++i) O[i] = (nv_f4){0, 0, 0, 0};
    float m = -INFINITY, l = 0.0f;
    uint8_t* vs = lds[wv];
    for (int j = j0; j < j1; ++j) {
      const int key0 = j * 128 + wv * 32;
      if (key0 >= q.L) break;
      RawKeys<DP> K[2], V[2];
#pragma unroll
      for (int g = 0; g < 2; ++g) {
        const int k = key0 + 16 * g, left = q.L - k;
        const int p = left > 0 ? page_of(a, q, k) : 0;
        const int at = k & ((1 << a.c.shift) - 1), rows = p < 0 || left <= 0 ? 0 : at + (left < 16 ? left : 16);
        K[g].load(a.c.k, a.c.ks, a, p < 0 ? 0 : p, h, at, rows, lane);
        V[g].load(a.c.v, a.c.vs, a, p < 0 ? 0 : p, h, at, rows, lane);
        if (p < 0) {
#pragma unroll
          for (int i = 0; i < (DP == 256 ? 2 : 1); ++i) K[g].s[i] = kNanScales;
        }
      }
      nv_f4 Sc[2];
#pragma unroll
      for (int g = 0; g < 2; ++g) {
        Sc[g] = (nv_f4){0, 0, 0, 0};
#pragma unroll
        for (int i = 0; i < NS; ++i) Sc[g] = __builtin_amdgcn_mfma_f32_16x16x32_f16(K[g].values(i), Q[i], Sc[g], 0, 0, 0);
      }
      float top = -INFINITY;
#pragma unroll
      for (int g = 0; g < 2; ++g)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const int key = key0 + 16 * g + 4 * grp + r;
          const float s = key < limit ? Sc[g][r] * by : -INFINITY;
          Sc[g][r] = s;
          top = fmaxf(top, s);
        }
      top = fmaxf(top, __shfl_xor(top, 16, 64));
      top = fmaxf(top, __shfl_xor(top, 32, 64));
      const float mn = fmaxf(m, top), base = mn == -INFINITY ? 0.0f : mn;
      const float alpha = exp2_fast(m - base);
      m = mn;
      l *= alpha;
      float w[8];
#pragma unroll
      for (int g = 0; g < 2; ++g)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          w[4 * g + r] = exp2_fast(Sc[g][r] - base + kWeightBits);
          l += w[4 * g + r];
        }
      nv_u4 pw;
#pragma unroll
      for (int i = 0; i < 4; ++i) pw[i] = pack_f16(w[2 * i], w[2 * i + 1]);
      const nv_h8 P = __builtin_bit_cast(nv_h8, pw);
      // values to shared memory, key by key; eight elements c of a key at c ^ key
#pragma unroll
      for (int g = 0; g < 2; ++g)
#pragma unroll
        for (int i = 0; i < NS; ++i) {
          const int key = 16 * g + col, c = NS * grp + i;
          *reinterpret_cast<nv_h8*>(vs + key * DP * 2 + ((c ^ (key & 7)) << 4)) = V[g].values(i);
        }
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
      __builtin_amdgcn_wave_barrier();
#pragma unroll
      for (int i = 0; i < NT; ++i) {
        nv_h4 part[2];
#pragma unroll
        for (int g = 0; g < 2; ++g) {
          // lane 4 x + y of a group of sixteen names a quarter of key 4 grp + x, and gets element (its number) of all four
          const int key = 16 * g + 4 * grp + (col >> 2), c = 2 * i + ((col & 3) >> 1);
          typedef __attribute__((address_space(3))) short lds_s;
          typedef short s4 __attribute__((ext_vector_type(4)));
          typedef __attribute__((address_space(3))) s4 lds_s4;
          const uint32_t off = (uint32_t)(uintptr_t)(lds_s*)(vs + key * DP * 2 + ((c ^ (key & 7)) << 4) + 8 * (col & 1));
          part[g] = __builtin_bit_cast(nv_h4, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s4*)(uintptr_t)off));
        }
        const nv_h8 A = __builtin_shufflevector(part[0], part[1], 0, 1, 2, 3, 4, 5, 6, 7);
        nv_f4 o = O[i];
#pragma unroll
        for (int r = 0; r < 4; ++r) o[r] *= alpha;
        O[i] = __builtin_amdgcn_mfma_f32_16x16x32_f16(A, P, o, 0, 0, 0);
      }
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
      __builtin_amdgcn_wave_barrier();
    }
    l += __shfl_xor(l, 16, 64);
    l += __shfl_xor(l, 32, 64);
    // the four waves' sums are joined
    float* mysum = reinterpret_cast<float*>(lds[wv]);
#pragma unroll
    for (int i = 0; i < NT; ++i) *reinterpret_cast<nv_f4*>(mysum + col * S::ROW + 16 * i + 4 * grp) = O[i];
    if (grp == 0) {
      stat[0][wv][col] = m;
      stat[1][wv][col] = l;
    }
    __syncthreads();
    const bool whole = j0 == 0 && j1 == kt;
    float* part = a.part + (2 * (int64_t)blockIdx.x + (j0 == 0 ? 1 : 0)) * part_size(D);
    for (int e = threadIdx.x; e < 16 * (DP / 4); e += 256) {
      const int r = e / (DP / 4), d = e % (DP / 4) * 4;
      float mm = -INFINITY, ll = 0.0f;
#pragma unroll
      for (int w = 0; w < 4; ++w) mm = fmaxf(mm, stat[0][w][r]);
      nv_f4 o = (nv_f4){0, 0, 0, 0};
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        const float f = exp2_fast(stat[0][w][r] - (mm == -INFINITY ? 0.0f : mm));
        ll = __builtin_fmaf(stat[1][w][r], f, ll);
        const nv_f4 x = *reinterpret_cast<const nv_f4*>(reinterpret_cast<const float*>(lds[w]) + r * S::ROW + d);
#pragma unroll
        for (int i = 0; i < 4; ++i) o[i] = __builtin_fmaf(x[i], f, o[i]);
      }
      if (whole) {
        write_row(a, unit_row(q, G, Hk, u, r), d, o, mm, ll, vdec);
      } else if (d < D) {
        *reinterpret_cast<nv_f4*>(part + r * D + d) = o;
        if (d == 0) {
          part[16 * D + r] = mm;
          part[16 * D + 16 + r] = ll;
        }
      }
    }
    __syncthreads();
    tile += j1 - j0;
  }
}

// Workgroup (i, y) joins rows 4 y .. 4 y + 3 of the unit that starts in piece i
// and goes on in the next ones.
__global__ __launch_bounds__(256) void k_attend_join(const AttendArgs a, int pieces) {
  const int D = a.c.dim, Hk = a.c.heads, G = a.q.heads / Hk, i = blockIdx.x;
  const SplitCount count{G, Hk, a.most, 128};
  SequenceScan<SplitCount> scan(a, count);
  const int total = scan.total(), start = piece_start(total, pieces, i), stop = piece_start(total, pieces, i + 1);
  if (start >= stop) return;
  scan.restart();
  Sequence q{};
  if (!scan.find(stop - 1, q)) return;
  const int kt = count.tiles(q.L), u = (stop - 1 - q.first) / kt, begin = q.first + u * kt, end = begin + kt;
  if (begin < start || end <= stop) return;
  const float vdec = a.c.va ? a.c.va[u % Hk] / 2688.0f : 1.0f;
  for (int e = threadIdx.x; e < D; e += 256) {
    const int r = 4 * blockIdx.y + e / (D / 4), d = e % (D / 4) * 4;
    const UnitRow row = unit_row(q, G, Hk, u, r);
    if (row.token < 0) continue;
    float m = -INFINITY, l = 0.0f;
    nv_f4 o = (nv_f4){0, 0, 0, 0};
    for (int p = i; p < pieces && (p == i || piece_start(total, pieces, p) < end); ++p) {
      if (p != i && piece_start(total, pieces, p) >= piece_start(total, pieces, p + 1)) continue;
      const float* part = a.part + (2 * (int64_t)p + (p == i ? 1 : 0)) * part_size(D);
      const float pm = part[16 * D + r], mn = fmaxf(m, pm), base = mn == -INFINITY ? 0.0f : mn;
      const float f = exp2_fast(m - base), g = exp2_fast(pm - base);
      l = __builtin_fmaf(part[16 * D + 16 + r], g, l * f);
      const nv_f4 x = *reinterpret_cast<const nv_f4*>(part + r * D + d);
#pragma unroll
      for (int k = 0; k < 4; ++k) o[k] = __builtin_fmaf(x[k], g, o[k] * f);
      m = mn;
    }
    write_row(a, row, d, o, m, l, vdec);
  }
}

int launch_attend_tiles(const AttendArgs& a, hipStream_t st);

int launch_attend(const AttendArgs& a, int which, void* stream) {
  hipStream_t st = (hipStream_t)stream;
  if (which & 1) {
    const LayerLaunch p = plan_attend_split(a.T, a.B, a.q.heads, a.c.heads, (int64_t)a.width << a.c.shift);
    if (a.c.dim <= 64) k_attend_split<64><<<(uint32_t)p.grid, p.block, 0, st>>>(a);
    else if (a.c.dim <= 128) k_attend_split<128><<<(uint32_t)p.grid, p.block, 0, st>>>(a);
    else k_attend_split<256><<<(uint32_t)p.grid, p.block, 0, st>>>(a);
    const LayerLaunch j = plan_attend_join(a.T, a.B, a.q.heads, a.c.heads, (int64_t)a.width << a.c.shift);
    if (j.grid) k_attend_join<<<dim3((uint32_t)j.grid, (uint32_t)j.y), j.block, 0, st>>>(a, (int)p.grid);
  }
  if (which & 2) return launch_attend_tiles(a, st);
  return (int)hipGetLastError();
}

}  // namespace nvfp4
