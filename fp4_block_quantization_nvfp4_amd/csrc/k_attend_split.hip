// Attention of few queries a sequence over an NVFP4 cache: decoding.
//
//   s_j = scale q . k_j for the keys j that the query sees, p = softmax(s),
//   out = sum_j p_j v_j, lse = log sum_j exp(s_j); without keys 0 and -inf
//
// Bound by reading the cache, 9/16 byte an element.  The queries of a sequence
// and of the heads that share keys form rows, sixteen to a unit; a unit's keys
// are tiles of 64.  All tiles of all units are one line, cut into even pieces, one
// a wave, whatever the sequences' lengths: a long one is shared by many waves,
// short ones are taken several by one.  A unit that lies in several pieces leaves
// its parts (sums, maxima) in the workspace, and a second launch joins them in
// order.
//
// A wave takes 32 keys at a time: keys times queries (transposed, a lane has one
// query's scores), the running maximum and sum of the softmax, weights back into
// the matrix cores as they lie, with values read across from the wave's own shared
// memory (turned by the load).  Waves wait for each other only at the end, where all
// four of a workgroup lie in one unit: their sums meet in shared memory.
//
// 64 sequences of up to 8192 keys, 32 heads on 8 of 128: 80 us and 7 for the join, 4.3
// TB/s of the 5.1 that a large copy reaches; two of up to 131072 keys 47 and 8.  What is
// left is the start (scan of the sequences, page numbers, first keys: 4 us, one after the
// other) and the two launches; the vector pipes are busy half of the time, decoding
// and softmax.  Two or four blocks of sixteen rows a unit, decoded for once, were slower:
// 24 queries a sequence 81 -> 93 us, 16 sequences of up to 64 queries 35 -> 43, the chain
// from scores to weights being longer than what it saves.
#include "nvfp4_attend.hpp"

namespace nvfp4 {

struct SplitCount {
  int G, Hk, most;
  // units of a sequence times their tiles of keys; a unit without keys counts as one
  NV_DEV int units(int n) const { return (int)(((int64_t)n * G + 15) / 16) * Hk; }
  NV_DEV int tiles(int L) const { return L > 0 ? (L + kAttendTile - 1) / kAttendTile : 1; }
  NV_DEV int operator()(bool real, int n, int L) const { return real && (int64_t)n * G > most ? 0 : units(n) * tiles(L); }
};

NV_DEV int min_of(int64_t a, int b) { return a < b ? (int)a : b; }

// The pieces: the waves take as many tiles each (attend_piece_tiles).
struct Pieces {
  int total, per;
  NV_DEV Pieces(const SplitCount& count, int total_, int longest, int pieces)
      : total(total_), per(attend_piece_tiles(total_, count.tiles(longest), pieces)) {}
  NV_DEV int start(int piece) const { return min_of((int64_t)per * piece, total); }
  // Whether the four pieces of workgroup w lie in the unit of tiles begin .. end - 1.
  NV_DEV bool shared(int w, int begin, int end) const { return start(4 * w) >= begin && start(4 * w + 4) <= end; }
  // Of a unit up to tile `end` whose first part is this piece of workgroup w0, which has
  // up to `most` parts of it.
  NV_DEV JoinHeader header(int w0, int piece, int most, int end, int unit, const Sequence& q, bool one) const {
    const int last = (end - 1) / per, w1 = last / 4;  // the piece that has the unit's last tile
    const int head = most < last - piece + 1 ? most : last - piece + 1, middle = w1 == w0 ? 0 : w1 - w0 - 1;
    const int tail = w1 == w0 ? 0 : start(4 * w1 + 4) <= end ? 1 : last - 4 * w1 + 1;
    return {head + middle + tail, head, middle, w1, unit, q.q0, q.n, one ? 1 : 0};
  }
};

template <int DP>
struct SplitShape {
  static constexpr int NS = DP / 32, NT = DP / 16;        // steps of 32 along d; tiles of 16 of it
  static constexpr int RUN = DP / 4;                      // elements of a key that a lane loads
  static constexpr int ROW = DP + 4;                      // floats of a row of sums in shared memory
  static constexpr int WAVE = 16 * ROW * 4;               // holds 32 keys' values too
  static_assert(32 * DP * 2 <= WAVE, "values, or sums");
};

// Where a head's keys and values of one page lie, and a lane's offsets into a
// group of 16 slots of it: a lane has DP / 4 elements of key lane % 16.
template <int DP>
struct PageView {
  static constexpr int PIECES = DP == 256 ? 2 : 1;
  const uint8_t *k, *ks, *v, *vs;  // of the head, page 0
  int64_t page;                    // bytes of a page's codes
  uint32_t row, co[PIECES], so[PIECES];
  NV_DEV PageView(const CacheView& c, int h, int lane) : page(((int64_t)c.heads << c.shift) * (c.dim / 2)), row((uint32_t)(c.dim / 2)) {
    const int64_t at = ((int64_t)h << c.shift) * (c.dim / 2);
    k = c.k + at, v = c.v + at, ks = c.ks + at / 8, vs = c.vs + at / 8;
#pragma unroll
    for (int i = 0; i < PIECES; ++i) {
      const uint32_t d = (uint32_t)(lane >> 4) * (DP / 4) + 32 * i;
      co[i] = d < (uint32_t)c.dim ? (uint32_t)(lane & 15) * row + d / 2 : kOutside;
      so[i] = d < (uint32_t)c.dim ? (uint32_t)(lane & 15) * (row / 8) + d / 16 : kOutside;
    }
  }
};

// Raw keys or values of 16 slots.
template <int DP>
struct RawKeys {
  static constexpr int NS = DP / 32, PIECES = PageView<DP>::PIECES;
  uint32_t w[NS], s[PIECES];
  // codes, scales: of the page, up to the last slot that may be read; at: the first
  // slot's offset into the codes, not past their end (a scalar)
  NV_DEV void load(const PageView<DP>& p, nv_buf codes, nv_buf scales, uint32_t at) {
#pragma unroll
    for (int i = 0; i < PIECES; ++i) {
      if constexpr (DP == 64) {
        const nv_u2 x = __builtin_amdgcn_raw_buffer_load_b64(codes.at, (int)p.co[i], (int)at, 0);
        w[0] = x.x;
        w[1] = x.y;
        s[i] = (uint32_t)(uint8_t)__builtin_amdgcn_raw_buffer_load_b8(scales.at, (int)p.so[i], (int)(at >> 3), 0);
      } else {
        const nv_u4 x = __builtin_amdgcn_raw_buffer_load_b128(codes.at, (int)p.co[i], (int)at, 0);
#pragma unroll
        for (int j = 0; j < 4; ++j) w[4 * i + j] = x[j];
        s[i] = (uint32_t)(uint16_t)__builtin_amdgcn_raw_buffer_load_b16(scales.at, (int)p.so[i], (int)(at >> 3), 0);
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
__global__ __launch_bounds__(256, DP == 256 ? 1 : 2) void k_attend_split(const AttendArgs a) {
  using S = SplitShape<DP>;
  constexpr int NS = S::NS, NT = S::NT;
  __shared__ __align__(16) uint8_t lds[4][S::WAVE];  // values of 32 keys, or sums
  __shared__ float stat[2][4][16];
  const int lane = threadIdx.x & 63, wv = uniform(threadIdx.x >> 6), col = lane & 15, grp = lane >> 4;
  const int D = a.c.dim, Hk = a.c.heads, G = a.q.heads / Hk;
  const SplitCount count{G, Hk, a.most};
  SequenceScan<SplitCount> scan(a, count);
  const int total = scan.total();
  const Pieces cut(count, total, scan.longest, 4 * gridDim.x);
  const int piece = 4 * blockIdx.x + wv, first = cut.start(4 * blockIdx.x);
  int tile = cut.start(piece);
  const int stop = cut.start(piece + 1);
  JoinHeader* join = a.part ? headers(a, D, 4 * gridDim.x) + piece : nullptr;
  if (join && lane == 0) *join = JoinHeader{};
  bool shared = false;
  Sequence q{};
  if (first < total) {
    scan.restart();
    if (scan.find(first, q)) {
      const int kt = count.tiles(q.L), begin = first - (first - q.first) % kt;
      shared = cut.shared(blockIdx.x, begin, begin + kt);
    }
  }
  while (tile < stop || shared) {
    if (tile < stop && !scan.find(tile, q)) break;
    const int at = tile < stop ? tile : first;  // a wave without a tile joins in all the same
    const int kt = count.tiles(q.L), u = (at - q.first) / kt, j0 = at - q.first - u * kt;
    const int j1 = tile < stop ? (j0 + (stop - tile) < kt ? j0 + (stop - tile) : kt) : j0;
    const int h = u % Hk;
    const UnitRow mine = unit_row(q, G, Hk, u, col);
    const int keys = uniform(j1 * kAttendTile < q.L ? j1 * kAttendTile : q.L);  // end of the piece
    PageWindow pages(a, q, j0 * kAttendTile < keys ? j0 * kAttendTile : 0);
    // a lane's query: RUN elements of row `col`
    nv_u4 raw[NS];
#pragma unroll
    for (int i = 0; i < NS; ++i) {
      const int d = S::RUN * grp + 8 * i;
      raw[i] = (nv_u4){0, 0, 0, 0};
      if (mine.token >= 0 && d < D)
        raw[i] = *reinterpret_cast<const nv_u4*>((const uint16_t*)a.q.at + mine.token * a.q.token + mine.head * a.q.head + d);
    }
    const PageView<DP> view(a.c, h, lane);
    // without branches, so that what is in flight is not waited for; outside the piece nothing is read
    auto load = [&](RawKeys<DP>(&K)[2], RawKeys<DP>(&V)[2], int key0) {
#pragma unroll
      for (int g = 0; g < 2; ++g) {
        const int k = key0 + 16 * g, left = keys - k;
        const int p = left > 0 ? pages(k) : -1;
        const int at = k & ((1 << a.c.shift) - 1), rows = p < 0 ? 0 : at + (left < 16 ? left : 16);
        const int64_t off = p < 0 ? 0 : p * view.page;
        const uint32_t bytes = (uint32_t)rows * view.row, first = (uint32_t)at * view.row;
        const uint32_t base = (uint32_t)uniform((int)(first < bytes ? first : bytes));
        K[g].load(view, make_buf(view.k + off, bytes), make_buf(view.ks + off / 8, bytes / 8), base);
        V[g].load(view, make_buf(view.v + off, bytes), make_buf(view.vs + off / 8, bytes / 8), base);
        if (left > 0 && p < 0) {
#pragma unroll
          for (int i = 0; i < RawKeys<DP>::PIECES; ++i) K[g].s[i] = kNanScales;
        }
      }
    };
    RawKeys<DP> K0[2], V0[2], K1[2], V1[2];
    int key0 = uniform(j0 * kAttendTile);
    load(K0, V0, key0);
    uint32_t big = 0;
#pragma unroll
    for (int i = 0; i < NS; ++i) big = amax_bits(raw[i], big);
    {
      const uint32_t o = (uint32_t)__shfl_xor((int)big, 16, 64);
      big = o > big ? o : big;
      const uint32_t p = (uint32_t)__shfl_xor((int)big, 32, 64);
      big = p > big ? p : big;
    }
    const float kdec = a.c.ka ? a.c.ka[h] / 2688.0f : 1.0f, vdec = a.c.va ? a.c.va[h] / 2688.0f : 1.0f;
    const float factor = query_factor(big), full = a.scale * kLog2e / factor * kdec, by = score_scale(full);
    nv_h8 Q[NS];
#pragma unroll
    for (int i = 0; i < NS; ++i) Q[i] = query_to_f16(raw[i], query_scale(factor, full));
    const int limit = mine.token < 0 ? 0 : seen_by(a, q, mine.token - q.q0);
    const int least = uniform(seen_by(a, q, u / Hk * 16 / G));  // what all rows of the unit see
    nv_f4 O[NT];
#pragma unroll
    for (int i = 0; i < NT; ++i) O[i] = (nv_f4){0, 0, 0, 0};
    float m = -INFINITY, l = 0.0f;
    bool far = false;  // a row's scores are large
    uint8_t* vs = lds[wv];
    auto step = [&](RawKeys<DP>(&K)[2], RawKeys<DP>(&V)[2], int key0, auto masked) {
#pragma unroll
      for (int g = 0; g < 2; ++g)
#pragma unroll
        for (int i = 0; i < RawKeys<DP>::PIECES; ++i) nan_to_key(K[g].s[i], V[g].s[i]);
      nv_f4 Sc[2];
#pragma unroll
      for (int g = 0; g < 2; ++g) {
        Sc[g] = (nv_f4){0, 0, 0, 0};
#pragma unroll
        for (int i = 0; i < NS; ++i) Sc[g] = __builtin_amdgcn_mfma_f32_16x16x32_f16(K[g].values(i), Q[i], Sc[g], 0, 0, 0);
      }
      // values to shared memory, key by key; chunk by chunk
#pragma unroll
      for (int g = 0; g < 2; ++g)
#pragma unroll
        for (int i = 0; i < NS; ++i) {
          const int key = 16 * g + col, c = NS * grp + i;
          *reinterpret_cast<nv_h8*>(vs + key * DP * 2 + ((c ^ chunk_at(key)) << 4)) = V[g].values(i);
        }
      if constexpr (masked.value) {
        const int hidden = limit - key0 - 4 * grp;
#pragma unroll
        for (int g = 0; g < 2; ++g)
#pragma unroll
          for (int r = 0; r < 4; ++r)
            if (16 * g + r >= hidden) Sc[g][r] = -INFINITY;
      }
      const float top = quarter_max(fmaxf(fmaxf(fmaxf(Sc[0][0], Sc[0][1]), fmaxf(Sc[0][2], Sc[0][3])),
                                          fmaxf(fmaxf(Sc[1][0], Sc[1][1]), fmaxf(Sc[1][2], Sc[1][3])))) * by;
      if (__builtin_amdgcn_ballot_w64(top - m > kSlack)) {
        const float mn = fmaxf(m, top), alpha = exp2_fast(m - (mn == -INFINITY ? 0.0f : mn));
        m = mn;
        l *= alpha;
#pragma unroll
        for (int i = 0; i < NT; ++i)
#pragma unroll
          for (int r = 0; r < 4; ++r) O[i][r] *= alpha;
        far = __builtin_amdgcn_ballot_w64(far_up(m)) != 0;
      }
      float f = by, up = kWeightBits - (m == -INFINITY ? 0.0f : m);
      if (far) {
        const FarScores less(m, f, up);
#pragma unroll
        for (int g = 0; g < 2; ++g)
#pragma unroll
          for (int r = 0; r < 4; ++r) Sc[g][r] = less(Sc[g][r]);
      }
      float w[8];
#pragma unroll
      for (int g = 0; g < 2; ++g)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          w[4 * g + r] = exp2_fast(__builtin_fmaf(Sc[g][r], f, up));
          l += w[4 * g + r];
        }
      nv_u4 pw;
#pragma unroll
      for (int i = 0; i < 4; ++i) pw[i] = pack_f16(w[2 * i], w[2 * i + 1]);
      const nv_h8 P = __builtin_bit_cast(nv_h8, pw);
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
      __builtin_amdgcn_wave_barrier();
#pragma unroll
      for (int i = 0; i < NT; ++i) {
        nv_h4 part[2];
#pragma unroll
        for (int g = 0; g < 2; ++g) {
          const int key = 16 * g + 4 * grp + (col >> 2), c = 2 * i + ((col & 3) >> 1);
          part[g] = read_turned(vs + key * DP * 2 + ((c ^ chunk_at(key)) << 4) + 8 * (col & 1));
        }
        const nv_h8 A = __builtin_shufflevector(part[0], part[1], 0, 1, 2, 3, 4, 5, 6, 7);
        O[i] = __builtin_amdgcn_mfma_f32_16x16x32_f16(A, P, O[i], 0, 0, 0);
      }
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
      __builtin_amdgcn_wave_barrier();
    };
    // the next 32 keys are on their way while these are used
    for (; key0 + 64 <= least && key0 + 64 <= keys; key0 += 64) {
      load(K1, V1, key0 + 32);
      step(K0, V0, key0, Masked<false>{});
      load(K0, V0, key0 + 64);
      step(K1, V1, key0 + 32, Masked<false>{});
    }
    for (; key0 < keys; key0 += 64) {
      load(K1, V1, key0 + 32);
      step(K0, V0, key0, Masked<true>{});
      load(K0, V0, key0 + 64);
      if (key0 + 32 < keys) step(K1, V1, key0 + 32, Masked<true>{});
    }
    l = quarter_sum(l);
    m = left_max(m, l, limit);
    if (shared) {
      float* mysum = reinterpret_cast<float*>(lds[wv]);
#pragma unroll
      for (int i = 0; i < NT; ++i) *reinterpret_cast<nv_f4*>(mysum + col * S::ROW + 16 * i + 4 * grp) = O[i];
      if (grp == 0) {
        stat[0][wv][col] = m;
        stat[1][wv][col] = l;
      }
      __syncthreads();
      const int begin = first - (first - q.first) % kt;
      const bool whole = first == begin && cut.start(4 * blockIdx.x + 4) == begin + kt;
      if (threadIdx.x == 0 && first == begin && !whole) *join = cut.header(blockIdx.x, 4 * blockIdx.x, 1, begin + kt, u, q, true);
      float* part = a.part + (8 * (int64_t)blockIdx.x + (first == begin ? 1 : 0)) * part_size(D);
      for (int e = threadIdx.x; e < 16 * (DP / 4); e += 256) {
        const int r = e / (DP / 4), d = e % (DP / 4) * 4;
        const UnitRow row = unit_row(q, G, Hk, u, r);
        if (row.token < 0 || d >= D) continue;
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
          write_row(a, (int64_t)row.token * a.q.heads + row.head, d, o, mm, ll, vdec);
        } else {
          *reinterpret_cast<nv_f4*>(part + r * D + d) = o;
          if (d == 0) {
            part[16 * D + r] = mm;
            part[16 * D + 16 + r] = ll;
          }
        }
      }
      break;
    }
    if (j0 == 0 && j1 < kt && lane == 0) *join = cut.header(blockIdx.x, piece, 4 - wv, tile + kt, u, q, false);
    if (mine.token >= 0) {
      const bool whole = j0 == 0 && j1 == kt;
      float* part = a.part + (2 * (int64_t)piece + (j0 == 0 ? 1 : 0)) * part_size(D);
#pragma unroll
      for (int i = 0; i < NT; ++i) {
        const int d = 16 * i + 4 * grp;
        if (d >= D) continue;
        if (whole) write_row(a, (int64_t)mine.token * a.q.heads + mine.head, d, O[i], m, l, vdec);
        else *reinterpret_cast<nv_f4*>(part + col * D + d) = O[i];
      }
      if (!whole && grp == 0) {
        part[16 * D + col] = m;
        part[16 * D + 16 + col] = l;
      }
    }
    tile += j1 - j0;
  }
}

void launch_attend_split(const AttendArgs& a, hipStream_t st) {
  const LayerLaunch p = plan_attend_split(a.T, a.B, a.q.heads, a.c.heads, a.c.dim, (int64_t)a.width << a.c.shift);
  if (a.c.dim <= 64) k_attend_split<64><<<(uint32_t)p.grid, p.block, 0, st>>>(a);
  else if (a.c.dim <= 128) k_attend_split<128><<<(uint32_t)p.grid, p.block, 0, st>>>(a);
  else k_attend_split<256><<<(uint32_t)p.grid, p.block, 0, st>>>(a);
}

}  // namespace nvfp4
