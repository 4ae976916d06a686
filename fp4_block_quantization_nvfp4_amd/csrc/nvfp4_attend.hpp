// What the attention kernels share: sequences and their units of work, found on
// the device from `ends` and `lens`; 4-bit keys and values as fp16 operands.
//
// A code has 2 significant bits and a block scale 4; the product has at most 6
// and lies in 2^-10 .. 2688, so fp16 holds every stored key and value exactly:
// the matrix cores multiply what the cache holds.  A query's row (bf16, 8 bits) is
// taken times the power of two that brings its largest element to 2^13 and is
// exact too, but for elements below 2^-24 of that one, which lose bits that the
// sums in fp32 do not have.  The second-level scales are applied to the sums.
// Weights exp(s - max) are rounded to fp16 times 2^11, the maximum being one that
// may lie up to 2^4 below the row's, so that sums are rescaled seldom: they keep 11
// bits down to 2^-25 (a bf16 result has 8), and below are off by 2^-36 of the
// largest at most.  Their sum is taken before that rounding, which adds 0.3 to 0.7% to the
// result's error: 1.64e-3 of its size for one sequence, 1.63e-3 of which is bf16's own rounding.
// Weights in two fp16, the second holding what the first leaves, add nothing, but their products
// cost two prompts of 8192 tokens 657 -> 876 us, decoding 87.5 -> 91.5, two long sequences
// 54.5 -> 58.6, an encoder's states 34.8 -> 36.2.
#pragma once

#include <float.h>

#include "nvfp4_cache.hpp"
#include "nvfp4_experts.hpp"
#include "nvfp4_plan.hpp"

namespace nvfp4 {

typedef _Float16 nv_h2 __attribute__((ext_vector_type(2)));
typedef _Float16 nv_h4 __attribute__((ext_vector_type(4)));
typedef _Float16 nv_h8 __attribute__((ext_vector_type(8)));

constexpr float kLog2e = 1.44269504088896340736f, kWeightBits = 11.0f, kSlack = 4.0f;
constexpr double kLn2 = 0.693147180559945309417;

NV_DEV float exp2_fast(float x) { return __builtin_amdgcn_exp2f(x); }

// Eight codes times their block's scale (in both halves) -> fp16, exact.
NV_DEV nv_h8 fp4_to_f16(uint32_t w, nv_h2 s) {
  const nv_h2 a = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, 1.0f, 0) * s, b = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, 1.0f, 1) * s;
  const nv_h2 c = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, 1.0f, 2) * s, d = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, 1.0f, 3) * s;
  return (nv_h8){a.x, a.y, b.x, b.y, c.x, c.y, d.x, d.y};
}
// Two scale bytes of a word.
NV_DEV nv_h2 scale_pair(uint32_t w, bool high) {
  return high ? __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w, 1.0f, true) : __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w, 1.0f, false);
}
NV_DEV nv_h2 both(_Float16 v) { return (nv_h2){v, v}; }

// A query's power of two from its largest magnitude's bits: 2^13 for the largest element.
NV_DEV float query_factor(uint32_t m) {
  const int e = (int)(m >> 23);
  const int f = 267 - e;
  return bits2f((uint32_t)(m == 0 ? 127 : f > 254 ? 254 : f) << 23);
}

// Eight bf16 times a power of two -> fp16.
NV_DEV nv_h8 query_to_f16(nv_u4 w, float f) {
  nv_h8 r;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    r[2 * i] = (_Float16)(bits2f(w[i] << 16) * f);
    r[2 * i + 1] = (_Float16)(bits2f(w[i] & 0xFFFF0000u) * f);
  }
  return r;
}
NV_DEV uint32_t amax_bits(nv_u4 w, uint32_t m) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t a = w[i] << 16 & 0x7FFFFFFFu, b = w[i] & 0x7FFF0000u;
    m = a > m ? a : m;
    m = b > m ? b : m;
  }
  return m;
}

NV_DEV uint32_t pack_f16(float a, float b) {
  nv_f2 v;
  v.x = a;
  v.y = b;
  return __builtin_bit_cast(uint32_t, __builtin_convertvector(v, nv_h2));
}

// Maximum (sum) over the lanes that are 32, or 16 and 32 apart, register to
// register: a swap of two copies gives each lane its own and the other's.
NV_DEV nv_f2 halves(float v) {
  const nv_u32x2 r = __builtin_bit_cast(nv_u32x2, __builtin_amdgcn_permlane32_swap(f2bits(v), f2bits(v), false, false));
  return (nv_f2){bits2f(r.x), bits2f(r.y)};
}
NV_DEV nv_f2 quarters(float v) {
  const nv_u32x2 r = __builtin_bit_cast(nv_u32x2, __builtin_amdgcn_permlane16_swap(f2bits(v), f2bits(v), false, false));
  return (nv_f2){bits2f(r.x), bits2f(r.y)};
}
NV_DEV float half_max(float v) {
  const nv_f2 r = halves(v);
  return fmaxf(r.x, r.y);
}
NV_DEV float quarter_max(float v) {
  const nv_f2 r = quarters(v);
  return half_max(fmaxf(r.x, r.y));
}
NV_DEV float quarter_sum(float v) {
  const nv_f2 r = quarters(v);
  const nv_f2 h = halves(r.x + r.y);
  return h.x + h.y;
}

// Whether a step's scores are masked, known when compiled (a branch in the loop became
// selections in every step).
template <bool B>
struct Masked {
  static constexpr bool value = B;
};

// What a score is taken times; never zero or NaN, so that hidden scores stay -infinity.  Where it
// would be NaN (the second-level scale is) the query is taken times that instead of its
// power of two: NaN are then the scores of the keys that are seen, and no others.
NV_DEV float score_scale(float v) { return v >= 0x1p-120f ? v : 0x1p-120f; }
NV_DEV float query_scale(float factor, float by) { return by == by ? factor : by; }

// A weight is 2^(score * by - m + 11), one multiply-add whose product is not rounded, while m
// is.  From 2^23 on the two part by half and more, and far up by more than fp16 holds.  Rows with
// such a maximum take rounded scores, and the difference from m by itself, which is exact near m:
// scores become fl(score * by) - m for them, and stay for the other rows of the wave.
NV_DEV bool far_up(float m) { return __builtin_fabsf(m) >= 0x1p23f && __builtin_fabsf(m) < INFINITY; }
struct FarScores {
  float mul, sub;
  NV_DEV FarScores(float m, float& by, float& up) : mul(1.0f), sub(0.0f) {
    if (!far_up(m)) return;
    mul = by, sub = m;
    by = 1.0f, up = kWeightBits;
  }
  NV_DEV float operator()(float score) const { return score * mul - sub; }
};

// log of the sum of exp from the running maximum and the sum of weights.
NV_DEV float log_sum(float m, float l) { return (float)(kLn2 * ((double)m - kWeightBits + (double)__builtin_amdgcn_logf(l))); }

// Decoded keys and values in shared memory: chunk c (eight elements) of key j lies
// at c ^ chunk_at(j): neither eight keys' same chunk (rows as an operand) nor two
// chunks of four keys in a row (columns, turned) meet in a bank.
NV_DEV int chunk_at(int key) { return (key & 3) << 1 | ((key >> 2) & 1); }

// Of each sixteen lanes, lane 4 x + y names a quarter (four fp16) of row x; lane i
// gets element i of the four rows.
NV_DEV nv_h4 read_turned(const uint8_t* p) {
  typedef __attribute__((address_space(3))) const uint8_t lds_byte;
  typedef short s4 __attribute__((ext_vector_type(4)));
  typedef __attribute__((address_space(3))) s4 lds_s4;
  return __builtin_bit_cast(nv_h4, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s4*)(uintptr_t)(uint32_t)(uintptr_t)(lds_byte*)p));
}

// ------------------------------------------------------------- sequences

// Sequence b has the queries [q0, q0 + n) and L keys.  `ends` are clamped to
// [0, T] and taken as their running maximum, so the ranges are disjoint whatever
// they hold; the queries past the last end form sequence B, without keys.  L
// is clamped to what the table's rows name; more than that is `over`, and the
// sequence's results are NaN.
struct Sequence {
  int b, q0, n, L, first, over;  // first: units of the sequences before it
};

// One wave walks the sequences, kScan at a time, four of them a lane; Count gives a
// sequence's units.  (64 at a time, one a lane: 256 sequences of up to 500 keys took
// five rounds of loads and sums before the first key was read.)
constexpr int kScan = 256;
template <typename Count>
struct SequenceScan {
  static constexpr int PER = kScan / 64;
  const AttendArgs& a;
  const Count& count;
  int lane, base, prev, before;  // sequences done, running end, units done
  int end[PER], len[PER], first[PER], begin, stop;  // this lane's: ends, lengths, units before each, first query, units up to the last
  int next, last, longest;       // units and queries up to the current ones' end; the largest length so far

  NV_DEV SequenceScan(const AttendArgs& a_, const Count& c_) : a(a_), count(c_), lane(threadIdx.x & 63), base(0), prev(0), before(0), longest(0) { load(); }
  NV_DEV void restart() {
    if (base == 0) return;
    base = prev = before = 0;
    load();
  }
  NV_DEV int keys(int raw) const {
    const int64_t most = (int64_t)a.width << a.c.shift;
    return raw < 0 ? 0 : (int64_t)raw > most ? (int)most : raw;
  }
  NV_DEV void load() {
    const int b0 = base + PER * lane;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      end[i] = a.T;
      len[i] = 0;
      if (b0 + i < a.B) {
        end[i] = a.ends ? a.ends[b0 + i] : b0 + i + 1;
        len[i] = a.lens[b0 + i];
      }
    }
    int top = prev;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      end[i] = end[i] < 0 ? 0 : end[i] > a.T ? a.T : end[i];
      top = end[i] = end[i] > top ? end[i] : top;
    }
    top = running_max(top);
    begin = __builtin_amdgcn_update_dpp(prev, top, 0x138, 0xF, 0xF, false);  // the lane before's; lane 0: prev
    int at = begin, sum = 0;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      end[i] = end[i] > begin ? end[i] : begin;
      const int n = b0 + i <= a.B ? end[i] - at : 0, L = keys(len[i]);
      longest = L > longest ? L : longest;
      first[i] = sum;
      sum += n > 0 ? count(b0 + i < a.B, n, L) : 0;
      at = end[i];
    }
    stop = before + running_sum(sum);
#pragma unroll
    for (int i = 0; i < PER; ++i) first[i] += stop - sum;
    next = __builtin_amdgcn_readlane(stop, 63);
    last = __builtin_amdgcn_readlane(top, 63);
  }
  // On; false where there are none.
  NV_DEV bool advance() {
    if (base + kScan > a.B) return false;
    base += kScan;
    prev = last;
    before = next;
    load();
    return true;
  }
  NV_DEV int total() {
    while (advance()) {}
    longest = __builtin_amdgcn_readlane(running_max(longest), 63);
    return next;
  }
  // The sequence that has unit x, at or past the current ones; false: no sequence has.
  NV_DEV bool find(int x, Sequence& s) {
    while (x >= next)
      if (!advance()) return false;
    const int from = (int)__builtin_ctzll(__builtin_amdgcn_ballot_w64(x >= first[0] && x < stop));
    // a sequence without units starts where the next one does: the last that starts up to x has it
    int i = 0, q0 = __builtin_amdgcn_readlane(begin, from), e = __builtin_amdgcn_readlane(end[0], from), raw = __builtin_amdgcn_readlane(len[0], from);
    s.first = __builtin_amdgcn_readlane(first[0], from);
#pragma unroll
    for (int k = 1; k < PER; ++k) {
      const int f = __builtin_amdgcn_readlane(first[k], from), ek = __builtin_amdgcn_readlane(end[k], from), rk = __builtin_amdgcn_readlane(len[k], from);
      if (f <= x) {
        q0 = __builtin_amdgcn_readlane(end[k - 1], from);
        s.first = f, e = ek, raw = rk, i = k;
      }
    }
    s.b = base + PER * from + i;
    s.q0 = q0;
    s.n = e - q0;
    s.L = keys(raw);
    s.over = raw > s.L ? 1 : 0;
    return true;
  }
};

// Keys that query i of the sequence sees.  Of one that is `over` all do all that the row
// names (sixteen at least, and all NaN): counted back from the clamped L the first queries would see none, and get 0.
NV_DEV int seen_by(const AttendArgs& a, const Sequence& s, int i) {
  const int m = s.L - s.n + i + 1;
  return !a.causal || s.over ? s.L : m < 0 ? 0 : m;
}

// Page that holds key j of a sequence (j < L), or -1 where the table names none.
// Keys of such a page have NaN for their scales, and so have the scores.
NV_DEV int page_of(const AttendArgs& a, const Sequence& s, int j) {
  const int p = a.table[(int64_t)s.b * a.width + (j >> a.c.shift)];
  return p >= 0 && p < a.c.pages && !s.over ? p : -1;
}
constexpr uint32_t kNanScales = 0x7F7F;
// Scales of a key's and of its value's blocks, up to two bytes each: a NaN of the value's goes
// to the key's, so that a query that does not see the key (weight 0) has none of it.
NV_DEV void nan_to_key(uint32_t& k, uint32_t& v) {
  const bool nan = (((v & 0x7F7Fu) + 0x0101u) & 0x8080u) != 0;
  k = nan ? kNanScales : k;
  v = nan ? 0 : v;
}

// A sequence's pages for a wave that walks along the keys: 64 entries of its row of
// the table in a register, the next 64 on their way, so that no load waits for a
// page number.
struct PageWindow {
  const int* row;
  int width, pages, shift, base, now, ahead;
  // (A sequence without keys, as that of the queries past the last end, may have no row.)
  NV_DEV PageWindow(const AttendArgs& a, const Sequence& s, int key)
      : row(a.table + (int64_t)s.b * a.width), width(s.L > 0 ? a.width : 0), pages(s.over ? 0 : a.c.pages), shift(a.c.shift) {
    base = key >> shift;
    now = fetch(base);
    ahead = fetch(base + 64);
  }
  NV_DEV int fetch(int at) const {
    const int i = at + (int)(threadIdx.x & 63);
    return i < width ? row[i] : -1;
  }
  // Page of key (at or past the last one asked for, below L), or -1.
  NV_DEV int operator()(int key) {
    const int i = key >> shift;
    while (i >= base + 64) {
      base += 64;
      now = ahead;
      ahead = fetch(base + 64);
    }
    const int p = __builtin_amdgcn_readlane(now, i - base);
    return p >= 0 && p < pages ? p : -1;
  }
};

// ------------------------------------------------------------- what is joined

// What the join needs of a unit whose first part is this piece's; parts 0: no unit.
// The parts: `head` pieces from here on, then one of each of `middle` workgroups,
// then the others from the first piece of workgroup w1 on.  (The join scanned the
// sequences itself before: 10 to 27 us.)
struct JoinHeader {
  int parts, head, middle, w1, unit, q0, n, shared;
};

// A partial result: sixteen rows of D sums, then their maxima, then their sums of weights.
NV_DEV int64_t part_size(int D) { return 16 * (int64_t)D + 32; }
// The workspace: two partial results for each piece (of a unit that began before it,
// and of one that it begins), then the headers.
NV_DEV JoinHeader* headers(const AttendArgs& a, int D, int pieces) { return reinterpret_cast<JoinHeader*>(a.part + 2 * (int64_t)pieces * part_size(D)); }

// Sixteen rows of unit `unit` of sequence s: row r is query r / G, head r % G of the unit's shared head.
struct UnitRow {
  int token, head;  // token -1: no such row
};
NV_DEV UnitRow unit_row(const Sequence& s, int G, int Hk, int unit, int r) {
  const int h = unit % Hk, m = unit / Hk * 16 + r, i = m / G;
  return {i < s.n ? s.q0 + i : -1, h * G + m - i * G};
}

// What the join needs of a unit; parts 0: nothing to join.
struct TileHeader {
  int parts, m0, h, q0, n, pad[3];
};
// The workspace: headers, then `parts` partial results for each unit, of rows x D
// sums, their maxima and their sums of weights.
NV_DEV TileHeader* tile_headers(const AttendArgs& a) { return reinterpret_cast<TileHeader*>(a.tiles); }
NV_DEV float* tile_part(const AttendArgs& a, int units, int parts, int rows, int unit, int i) {
  return a.tiles + 8 * (int64_t)units + ((int64_t)unit * parts + i) * rows * (a.c.dim + 2);
}

// The maximum that a row leaves.  Without weights it stays -infinity where the row sees no
// key, and is the lowest finite number where it does: those scores are all -infinity, or lie
// in other parts, next to which this one counts nothing.
NV_DEV float left_max(float m, float l, int seen) { return l == 0.0f && seen > 0 ? -FLT_MAX : m; }

// Four elements of row `row` of the outputs, from its sums o, maximum and sum of weights.  No
// weights: 0 and -infinity for a row without keys, NaN where all its scores are -infinity.
NV_DEV void write_row(const AttendArgs& a, int64_t row, int d, nv_f4 o, float m, float l, float vdec) {
  const float inv = l != 0.0f ? vdec / l : m == -INFINITY ? 0.0f : __builtin_nanf("");
  nv_u2 w;
  w.x = pack_bf16(o[0] * inv, o[1] * inv);
  w.y = pack_bf16(o[2] * inv, o[3] * inv);
  *reinterpret_cast<nv_u2*>(a.out + row * a.c.dim + d) = w;
  if (d == 0) a.lse[row] = l != 0.0f ? log_sum(m, l) : m == -INFINITY ? m : inv;
}

}  // namespace nvfp4
