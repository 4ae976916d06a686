// What the attention kernels share: sequences and their units of work, found on
// the device from `ends` and `lens`; 4-bit keys and values as fp16 operands.
//
// A code has 2 significant bits and a block scale 4; the product has at most 6
// and lies in 2^-10 .. 2688, so fp16 holds every stored key and value exactly:
// the matrix cores multiply what the cache holds.  A query's row (bf16, 8 bits) is
// taken times the power of two that brings its largest element to 2^13 and is
// exact too, but for elements below 2^-24 of that one, which lose bits that the
// sums in fp32 do not have.  The second-level scales are applied to the sums.
// Weights exp(s - max) are rounded to fp16 times 2^14, so that they keep 11 bits
// down to 2^-28 (a bf16 result has 8); their sum is taken before that rounding.
#pragma once

#include "nvfp4_cache.hpp"
#include "nvfp4_plan.hpp"

namespace nvfp4 {

typedef _Float16 nv_h2 __attribute__((ext_vector_type(2)));
typedef _Float16 nv_h4 __attribute__((ext_vector_type(4)));
typedef _Float16 nv_h8 __attribute__((ext_vector_type(8)));

constexpr float kLog2e = 1.44269504088896340736f, kWeightBits = 14.0f;
constexpr double kLn2 = 0.693147180559945309417;

NV_DEV int uniform(int v) { return __builtin_amdgcn_readfirstlane(v); }
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

NV_DEV float other_half_max(float v) { return fmaxf(v, __shfl_xor(v, 32, 64)); }

// ------------------------------------------------------------- sequences

// Sequence b has the queries [q0, q0 + n) and L keys.  `ends` are clamped to
// [0, T] and taken as their running maximum, so the ranges are disjoint whatever
// they hold; the queries past the last end form sequence B, without keys.  L
// is clamped to what the table's rows name; more than that is `over`, and the
// sequence's results are NaN.
struct Sequence {
  int b, q0, n, L, first, over;  // first: units of the sequences before it
};

// One wave walks the sequences 64 at a time; Count gives a sequence's units.
template <typename Count>
struct SequenceScan {
  const AttendArgs& a;
  const Count& count;
  int lane, base, prev, before;       // sequences done, running end, units done
  int q0, n, L, over, first, own;     // this lane's sequence of the current 64

  NV_DEV SequenceScan(const AttendArgs& a_, const Count& c_) : a(a_), count(c_), lane(threadIdx.x & 63) { restart(); }
  NV_DEV void restart() {
    base = prev = before = 0;
    load();
  }
  NV_DEV void load() {
    const int b = base + lane;
    int end = a.T, len = 0;
    if (b < a.B) {
      end = a.ends ? a.ends[b] : b + 1;
      end = end < 0 ? 0 : end > a.T ? a.T : end;
      len = a.lens[b];
    }
    end = end > prev ? end : prev;
#pragma unroll
    for (int off = 1; off < 64; off <<= 1) {
      const int o = __shfl_up(end, off, 64);
      end = lane >= off && o > end ? o : end;
    }
    const int up = __shfl_up(end, 1, 64);
    q0 = lane ? up : prev;
    n = b <= a.B ? end - q0 : 0;
    const int64_t most = (int64_t)a.width << a.c.shift;
    over = (int64_t)len > most ? 1 : 0;
    L = len < 0 ? 0 : over ? (int)most : len;
    own = n > 0 ? count(b < a.B, n, L) : 0;
    int sum = own;
#pragma unroll
    for (int off = 1; off < 64; off <<= 1) {
      const int o = __shfl_up(sum, off, 64);
      sum += lane >= off ? o : 0;
    }
    first = before + sum - own;
    next = before + __shfl(sum, 63, 64);
    last = __shfl(end, 63, 64);
  }
  int next, last;
  // To the next 64; false where there are none.
  NV_DEV bool advance() {
    if (base + 64 > a.B) return false;
    base += 64;
    prev = last;
    before = next;
    load();
    return true;
  }
  NV_DEV int total() {
    while (advance()) {}
    return next;
  }
  // The sequence that has unit x, at or past the current 64; false: no sequence has.
  NV_DEV bool find(int x, Sequence& s) {
    while (x >= next)
      if (!advance()) return false;
    const uint64_t hit = __builtin_amdgcn_ballot_w64(x >= first && x < first + own);
    const int from = (int)__builtin_ctzll(hit);
    s.b = base + from;
    s.q0 = __builtin_amdgcn_readlane(q0, from);
    s.n = __builtin_amdgcn_readlane(n, from);
    s.L = __builtin_amdgcn_readlane(L, from);
    s.over = __builtin_amdgcn_readlane(over, from);
    s.first = __builtin_amdgcn_readlane(first, from);
    return true;
  }
};

// Keys that query i of the sequence sees.
NV_DEV int seen_by(const AttendArgs& a, const Sequence& s, int i) {
  const int m = s.L - s.n + i + 1;
  return !a.causal ? s.L : m < 0 ? 0 : m;
}

// Page that holds key j of a sequence (j < L), or -1 where the table names none.
// Keys of such a page have NaN for their scales, and so have the scores.
NV_DEV int page_of(const AttendArgs& a, const Sequence& s, int j) {
  const int p = a.table[(int64_t)s.b * a.width + (j >> a.c.shift)];
  return p >= 0 && p < a.c.pages && !s.over ? p : -1;
}
constexpr uint32_t kNanScales = 0x7F7F;

NV_DEV uint16_t bf16_bits(float v) { return (uint16_t)(pack_bf16(v, 0.0f) & 0xFFFFu); }

}  // namespace nvfp4
