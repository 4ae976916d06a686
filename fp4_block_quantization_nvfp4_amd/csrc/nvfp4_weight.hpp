// Operands of the matrix products: rows of x (bf16 or mx8) and 4-bit weights.
#pragma once

#include "nvfp4_launch.hpp"
#include "nvfp4_mx8.hpp"

namespace nvfp4 {

// Rows row0 .. row0 + rows - 1 of x; rows outside read as zeros.
template <bool MX8>
struct RowsView {
  nv_buf x, s;
  int K, ns;
  NV_DEV RowsView(const MatmulArgs& a, int64_t row0, int rows) : K(a.K), ns((a.K + kMxGroup - 1) / kMxGroup) {
    const int64_t pitch = MX8 ? a.K : 2 * (int64_t)a.K;
    x = make_buf((const char*)a.x + row0 * pitch, (uint32_t)(rows * pitch));
    s = make_buf(MX8 ? a.xs + row0 * ns : nullptr, MX8 ? (uint32_t)(rows * ns) : 0u);
  }
};

// A wave's piece of 256 k's of XR rows of x.  It is loaded as whole lines of
// memory, passes through the wave's own shared memory, and is read as
// fragments: (g, q, d) holds for lane (l16, grp) the k's 64 grp + 32 q + 8 d ..
// + 7 of row 16 g + l16.  k's at or past K read as zeros.  Pieces are loaded
// without branches, also past the last one: what is in flight can then be
// counted.  XR is 4 where there are few rows: the products of the others are
// not used.
template <bool MX8, int XR>
struct RowsPiece {
  static constexpr int kLanes = MX8 ? 16 : 32, kLoads = XR * kLanes / 64, G = XR > 16 ? XR / 16 : 1;  // kLanes: lanes to a row
  nv_u4 c[kLoads];
  uint32_t s[G][2];
  NV_DEV void load(const RowsView<MX8>& v, int lane, int k0) {
    const int l16 = lane & 15, grp = lane >> 4, at = lane % kLanes;
    const bool in = k0 + at * (MX8 ? 16 : 8) < v.K;
    const uint32_t pitch = (uint32_t)v.K * (MX8 ? 1u : 2u), off = in ? (uint32_t)(lane / kLanes) * pitch + 16u * at : kOutside;
#pragma unroll
    for (int i = 0; i < kLoads; ++i) c[i] = buf16(v.x, off, (uint32_t)(i * (64 / kLanes)) * pitch + (uint32_t)k0 * (MX8 ? 1u : 2u));
    if (MX8) {
      const int left = v.ns - k0 / kMxGroup - 2 * grp;
#pragma unroll
      for (int q = 0; q < 2; ++q)
#pragma unroll
        for (int g = 0; g < G; ++g)
          s[g][q] = buf1(v.s, q < left ? (uint32_t)(l16 * v.ns + 2 * grp + q) : kOutside,
                         (uint32_t)k0 / kMxGroup + (uint32_t)(16 * g * v.ns));
    }
  }
  // Chunk c of a row lies at c ^ row: neither this nor the reads meet in a bank.
  NV_DEV void put(nv_u4* lds, int lane) const {
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      const int row = i * (64 / kLanes) + lane / kLanes;
      lds[row * kLanes + ((lane % kLanes) ^ (row % kLanes))] = c[i];
    }
  }
  // Fragments (g, q, 0..3).
  NV_DEV void fragments(const nv_u4* lds, int lane, int g, int q, nv_bf8 f[4]) const {
    const int row = 16 * g + (lane & 15), grp = lane >> 4;
    if (!MX8) {
#pragma unroll
      for (int d = 0; d < 4; ++d) f[d] = __builtin_bit_cast(nv_bf8, lds[row * kLanes + ((8 * grp + 4 * q + d) ^ (row % kLanes))]);
      return;
    }
    const float sc = e8m0_scale(s[g][q]);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const nv_u4 w = lds[row * kLanes + ((4 * grp + 2 * q + h) ^ (row % kLanes))];
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const nv_u2 a = mx8_to_bf16(w[2 * j], sc), b = mx8_to_bf16(w[2 * j + 1], sc);
        f[2 * h + j] = __builtin_bit_cast(nv_bf8, (nv_u4){a.x, a.y, b.x, b.y});
      }
    }
  }
};

// Half a step's rows of k_grouped as its 256 lanes load them: 128 k's of BM / 2
// rows in 16-byte pieces, PR a row; lane tid takes piece tid % PR of rows
// tid / PR + 256 / PR * i.  k's at or past K read as zeros.
template <bool MX8, int BM>
struct RowsHalf {
  static constexpr int PR = MX8 ? 8 : 16, HALF = BM / 2 * PR, PIECES = HALF > 256 ? HALF / 256 : 1;
  nv_u4 c[PIECES];
  uint32_t s[PIECES];
  NV_DEV void load(const RowsView<MX8>& v, int tid, int k0, int h) {
    if (HALF < 256 && tid >= HALF) return;
    const int xr = tid / PR, xp = tid % PR;
    const uint32_t pitch = MX8 ? (uint32_t)v.K : 2u * (uint32_t)v.K;
    const uint32_t xat = (uint32_t)xr * pitch + (uint32_t)xp * 16u, sat = (uint32_t)(xr * v.ns + xp / 2);
    const bool in = k0 + 128 <= v.K || k0 + xp * (MX8 ? 16 : 8) < v.K;
#pragma unroll
    for (int i = 0; i < PIECES; ++i) {
      const uint32_t r = (uint32_t)(h * (BM / 2) + i * (256 / PR));
      c[i] = buf16(v.x, in ? xat : kOutside, (uint32_t)k0 * (MX8 ? 1u : 2u) + r * pitch);
      if (MX8) s[i] = buf1(v.s, in ? sat : kOutside, (uint32_t)k0 / kMxGroup + r * (uint32_t)v.ns);
    }
  }
};

// Rows n0 .. n0 + rows - 1 of expert e's weight [N, K]; BLK 0: a scale for
// 1x16 elements [N, K / 16]; 1: for 16x16 tiles [N / 16, K / 16]; 2: the same
// tiles stored as those of the transposed weight, [K / 16, N / 16].
template <int BLK>
struct WeightView {
  nv_buf w, s;
  int K, kb, nb;  // kb blocks along k, nb tiles along n
  NV_DEV WeightView(const MatmulArgs& a, int e, int n0, int most) : K(a.K), kb(a.K / 16), nb(a.N / 16) {
    const int rows = a.N - n0 < most ? a.N - n0 : most, t0 = n0 / 16;
    const int64_t NK = (int64_t)a.N * a.K;
    w = make_buf(a.w + e * (NK / 2) + (int64_t)n0 * (a.K / 2), (uint32_t)rows * (uint32_t)(a.K / 2));
    if (BLK == 0) s = make_buf(a.ws + e * (NK / 16) + (int64_t)n0 * kb, (uint32_t)rows * (uint32_t)kb);
    else if (BLK == 1)
      s = make_buf(a.ws + e * (NK / 256) + (int64_t)t0 * kb, (uint32_t)(rows / 16) * (uint32_t)kb);
    else s = make_buf(a.ws + e * (NK / 256) + t0, (uint32_t)kb * (uint32_t)nb - (uint32_t)t0);
  }
};

// The same piece of rows 16 i .. 16 i + 15 of a weight, through 2 KB.  k's at
// or past K have code 0 or scale 0.  WORDS: the four scales of a lane are a
// word (K % 64 == 0; tiles of the transposed weight always take four bytes).
template <int BLK, bool WORDS>
struct WeightPiece {
  static constexpr bool kWord = BLK != 2 && WORDS;
  nv_u4 c[2];
  uint32_t s[kWord ? 1 : 4];
  NV_DEV void load(const WeightView<BLK>& v, int i, int lane, int k0) {
    const int l16 = lane & 15, grp = lane >> 4, l8 = lane & 7;
    const uint32_t pitch = (uint32_t)v.K / 2u;
    const uint32_t off = k0 + 32 * l8 < v.K ? (uint32_t)(lane / 8) * pitch + 16u * l8 : kOutside;
#pragma unroll
    for (int h = 0; h < 2; ++h) c[h] = buf16(v.w, off, (uint32_t)(16 * i + 8 * h) * pitch + (uint32_t)k0 / 2u);
    const int left = v.kb - k0 / 16 - 4 * grp;  // blocks from the lane's first on
    const uint32_t step = BLK == 2 ? (uint32_t)v.nb : 1u;
    const uint32_t at = (BLK == 0 ? (uint32_t)l16 * (uint32_t)v.kb : 0u) + 4u * grp * step;
    const uint32_t base = (BLK == 2 ? (uint32_t)i : (uint32_t)(BLK == 0 ? 16 * i : i) * (uint32_t)v.kb) + (uint32_t)(k0 / 16) * step;
    if (kWord) s[0] = buf4(v.s, left > 0 ? at : kOutside, base);
    else
#pragma unroll
      for (int j = 0; j < 4; ++j) s[kWord ? 0 : j] = buf1(v.s, j < left ? at + j * step : kOutside, base);
  }
  // Turns the codes as loaded into the lane's 64: word d of c[q] is fragment (q, d).
  NV_DEV void turn(nv_u4* lds, int lane) {
    const int l16 = lane & 15, grp = lane >> 4;
#pragma unroll
    for (int h = 0; h < 2; ++h) lds[(8 * h + lane / 8) * 8 + ((lane & 7) ^ (lane / 8))] = c[h];
#pragma unroll
    for (int q = 0; q < 2; ++q) c[q] = lds[l16 * 8 + ((2 * grp + q) ^ (l16 & 7))];
  }
  NV_DEV nv_bf8 fragment(int q, int d) const {
    const int b = 2 * q + (d >> 1);
    return fp4_to_bf16(c[q][d], kWord ? e4m3_byte(s[0], b) : e4m3_byte(s[kWord ? 0 : b], 0));
  }
};

// A wave's walk along k in steps of 128 over 32 NI rows of a weight: lane
// (l32, half) takes, of rows 32 i + l32, the 64 codes from k0 + 64 half on as
// two 16-byte words and their four scales as one.  Steps that lie within K
// take their offset along k from a scalar; the last, partial one is checked
// lane by lane.  Past N and K the scales read as 0 (the codes there are
// whatever the next row holds).
template <int BLK, int NI>
struct WeightStream {
  nv_buf w, s;
  int K, kb, nb, at;         // at: 64 half
  uint32_t end;              // bytes of codes
  uint32_t row[NI], srow[NI];  // byte offsets of the lane's rows; BLK 2: srow[i] is the lane's byte of a word of four tiles
  NV_DEV WeightStream(const MatmulArgs& a, int e, int n0, int l32, int half)
      : K(a.K), kb(a.K / 16), nb(a.N / 16), at(64 * half) {
    const int rows = n0 < a.N ? (a.N - n0 < 32 * NI ? a.N - n0 : 32 * NI) : 0, t0 = rows ? n0 / 16 : 0, base = rows ? n0 : 0;
    const int c0 = t0 < nb - 4 ? t0 : nb > 4 ? nb - 4 : 0;  // BLK 2: first of the four tiles that a word holds
    const int64_t NK = (int64_t)a.N * a.K;
    end = (uint32_t)rows * (uint32_t)(a.K / 2);
    w = make_buf(a.w + e * (NK / 2) + (int64_t)base * (a.K / 2), end);
    if (BLK == 0) s = make_buf(a.ws + e * (NK / 16) + (int64_t)base * kb, (uint32_t)rows * (uint32_t)kb);
    else if (BLK == 1) s = make_buf(a.ws + e * (NK / 256) + (int64_t)t0 * kb, (uint32_t)(rows / 16) * (uint32_t)kb);
    else s = make_buf(a.ws + e * (NK / 256) + c0, rows ? (uint32_t)kb * (uint32_t)nb - (uint32_t)c0 : 0u);
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      const int r = i * 32 + l32;
      row[i] = r < rows ? (uint32_t)r * (uint32_t)(K / 2) + (uint32_t)at / 2 : kOutside;
      if (BLK == 2) srow[i] = (uint32_t)(r / 16 + t0 - c0) & 3u;
      else srow[i] = r < rows ? (uint32_t)(BLK == 0 ? r : r / 16) * (uint32_t)kb : kOutside;
    }
  }
  // Codes of the lane's k's 32 q .. 32 q + 31 of row i; nothing is read for a step past K.
  NV_DEV nv_u4 codes(int i, int k0, int q) const { return buf16(w, row[i] + 16u * q, k0 < K ? (uint32_t)k0 / 2 : end); }
  // Scales of 1x16 blocks are taken for two steps at a time, 16 bytes of a row a
  // lane: a line of memory holds a row's scales for 16 steps, and would be
  // fetched anew for each (8192 rows x 4096 x 4096 bf16: 1088 -> 1120 TFLOP/s).
  static constexpr bool kPairs = BLK == 0 && NI == 2;
  NV_DEV bool paired(int k0) const { return kPairs && (k0 & ~255) + 256 <= K; }
  // Loads what the scales of the step at k0 are made from; of a pair, the first
  // step's call loads both.
  NV_DEV void fetch_scales(int k0, uint32_t v[4]) const {
    const int b = (k0 + at) / 16;
    if (paired(k0)) {
      if (k0 & 128) return;
      const nv_u4 w = buf16(s, (uint32_t)(threadIdx.x & 63) * (uint32_t)kb, (uint32_t)k0 / 16);
#pragma unroll
      for (int j = 0; j < 4; ++j) v[j] = w[j];
    } else if (BLK == 2) {
      if (nb >= 4) {
#pragma unroll
        for (int j = 0; j < 4; ++j)
          v[j] = buf4(s, b + j < kb ? (uint32_t)(at / 16) * (uint32_t)nb : kOutside, (uint32_t)(k0 / 16 + j) * (uint32_t)nb);
      } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          v[j] = 0;
#pragma unroll
          for (int t = 0; t < 3; ++t) v[j] |= buf1(s, t < nb && b + j < kb ? (uint32_t)(b + j) * (uint32_t)nb + t : kOutside) << (8 * t);
        }
      }
    } else if (k0 + 128 <= K) {
#pragma unroll
      for (int i = 0; i < NI; ++i) v[i] = buf4(s, srow[i] + (uint32_t)at / 16, (uint32_t)k0 / 16);
    } else if (kb >= 4) {
      // the last word of a row starts at its fourth last byte: shifted down, it has zeros past the row
      const int c = b < kb - 4 ? b : kb - 4, d = b - c;
#pragma unroll
      for (int i = 0; i < NI; ++i) v[i] = buf4(s, b < kb ? srow[i] + (uint32_t)c : kOutside) >> (8 * (d & 3));
    } else {
#pragma unroll
      for (int i = 0; i < NI; ++i) {
        v[i] = 0;
#pragma unroll
        for (int j = 0; j < 3; ++j) v[i] |= buf1(s, b + j < kb ? srow[i] + (uint32_t)(b + j) : kOutside) << (8 * j);
      }
    }
  }
  // The lane's four scales of its rows, one in a byte.
  NV_DEV void scales(int k0, const uint32_t v[4], uint32_t ws[NI]) const {
    if (paired(k0)) {
      // lane l has row l: the halves of the first 64 k's and of the second trade places
      const int h = k0 & 128 ? 2 : 0;
      const nv_u2 r = __builtin_bit_cast(nv_u2, __builtin_amdgcn_permlane32_swap(h ? v[2] : v[0], h ? v[3] : v[1], false, false));
      ws[0] = r.x;
      ws[NI - 1] = r.y;
      return;
    }
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      if (BLK != 2) {
        ws[i] = v[i];
        continue;
      }
      const uint32_t pick = srow[i] | (4u + srow[i]) << 8;  // that byte of two words; 0x0c gives zero
      ws[i] = __builtin_amdgcn_perm(v[1], v[0], 0x0c0c0000u | pick) | __builtin_amdgcn_perm(v[3], v[2], pick << 16 | 0x0c0cu);
    }
  }
};

// Second-level scale of row n of expert e's weight.
NV_DEV float second_scale(const MatmulArgs& a, int e, int n) {
  if (a.mode == 0) return 1.0f;
  return a.amax[a.mode == 1 ? (int64_t)e : (int64_t)e * a.N + n] / a.D;
}

NV_DEV void store_out(const MatmulArgs& a, float v, int64_t t, int n) {
  const int64_t i = t * a.N + n;
  if (a.out_bf16) ((uint16_t*)a.out)[i] = (uint16_t)pack_bf16(v, v);
  else ((float*)a.out)[i] = v;
}

// Four consecutive n's (n % 4 == 0) of one row; those at or past N are left.
NV_DEV void store_out4(const MatmulArgs& a, float v0, float v1, float v2, float v3, int64_t t, int n) {
  const int64_t i = t * a.N + n;
  if (n + 4 <= a.N && a.N % 4 == 0) {
    if (a.out_bf16) *reinterpret_cast<nv_u2*>((uint16_t*)a.out + i) = (nv_u2){pack_bf16(v0, v1), pack_bf16(v2, v3)};
    else *reinterpret_cast<nv_f4*>((float*)a.out + i) = (nv_f4){v0, v1, v2, v3};
    return;
  }
  if (n < a.N) store_out(a, v0, t, n);
  if (n + 1 < a.N) store_out(a, v1, t, n + 1);
  if (n + 2 < a.N) store_out(a, v2, t, n + 2);
  if (n + 3 < a.N) store_out(a, v3, t, n + 3);
}

}  // namespace nvfp4
