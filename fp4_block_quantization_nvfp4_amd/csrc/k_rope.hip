// Norms of queries and keys for each head with the rotation of their positions
// in the same pass, straight to the outputs or, keys and values, quantized into
// the cache; and the gradient.
//
//   rstd = (mean_d x_d^2 + eps)^(-1/2),  y = x rstd w  (y = x without weights)
//   angle_i = position f_i,  c = m cos angle,  s = m sin angle
//   (a, b) -> (a c - b s, b c + a s) for the pairs (y_i, y_{i + R/2}), or
//   (y_2i, y_2i+1) where they are interleaved; elements from R on stay
//   gradient: dy = the rotation back of dz, n = x rstd, d = dy w,
//   dx = rstd (d - n mean(d n)), dw = sum over tokens and heads of dy n
//
// All are bound by memory: every row is read once and written once.  A lane
// holds sixteen elements of a row as two runs of eight, placed so that both
// halves of a pair are its own: no data crosses lanes but the row's sum.  A wave
// has one token, whose angles are worked out once, a lane each, for all heads.
//
// Angles are products in 64 bits, reduced by pi / 2 in two parts, and sine and
// cosine are sums of their series in 64 bits: at position 10^6 a 32-bit angle is
// off by 0.03 radians.  The forward pass stays in 64 bits up to the result: what is
// quantized next shows the last bits in every code near a
// border.  (Vector instructions of 64 bits run at the rate of 32.)
#include "nvfp4_cache.hpp"
#include "nvfp4_plan.hpp"

namespace nvfp4 {

struct SinCos {
  double s, c;
};

// A constant in a scalar, made where it is used: kept in vector registers over the
// loop, those of the series cost 40 of them.
NV_DEV double scalar(double v) {
  asm volatile("" : "+s"(v));
  return v;
}

NV_DEV SinCos sincos64(double a) {
  const double n = __builtin_rint(a * scalar(0x1.45f306dc9c883p-1));  // 2 / pi
  double r = __builtin_fma(-n, scalar(0x1.921fb54442d18p+0), a);       // pi / 2, the first 53 bits: the product's own bits are kept
  r = __builtin_fma(-n, scalar(0x1.1a62633145c07p-54), r);              // and the next 53
  const double q = r * r;
  // Taylor's series on |r| <= pi / 4: the first term left out is below 1e-19 (sine, r^19 / 19!), 3e-18 (cosine, r^18 / 18!)
  double s = scalar(1.0 / 355687428096000.0);
  s = __builtin_fma(s, q, scalar(-1.0 / 1307674368000.0));
  s = __builtin_fma(s, q, scalar(1.0 / 6227020800.0));
  s = __builtin_fma(s, q, scalar(-1.0 / 39916800.0));
  s = __builtin_fma(s, q, scalar(1.0 / 362880.0));
  s = __builtin_fma(s, q, scalar(-1.0 / 5040.0));
  s = __builtin_fma(s, q, scalar(1.0 / 120.0));
  s = __builtin_fma(s, q, scalar(-1.0 / 6.0));
  s = __builtin_fma(s * q, r, r);
  double c = scalar(1.0 / 20922789888000.0);
  c = __builtin_fma(c, q, scalar(-1.0 / 87178291200.0));
  c = __builtin_fma(c, q, scalar(1.0 / 479001600.0));
  c = __builtin_fma(c, q, scalar(-1.0 / 3628800.0));
  c = __builtin_fma(c, q, scalar(1.0 / 40320.0));
  c = __builtin_fma(c, q, scalar(-1.0 / 720.0));
  c = __builtin_fma(c, q, scalar(1.0 / 24.0));
  c = __builtin_fma(c, q, scalar(-0.5));
  c = __builtin_fma(c, q, 1.0);
  const int quarter = (int)(n - 4.0 * __builtin_floor(n * 0.25));  // 0..3
  const double x = quarter & 1 ? c : s, y = quarter & 1 ? s : c;
  return {quarter & 2 ? -x : x, ((quarter + 1) & 2) ? -y : y};
}

// (mean x^2 + eps)^(-1/2) from the sum of squares: the instruction's 2^-22 or so
// and two steps of Newton's method; zero and infinity as they come.
NV_DEV double inverse_root(double var) {
  const double a = __builtin_amdgcn_rsq(var);
  const double o = a * (0.5 * __builtin_fma(-var * a, a, 1.0));
  if (o != o) return a;
  const double b = a + o;
  return b + b * (0.5 * __builtin_fma(-var * b, b, 1.0));
}

template <int LN, typename V>
NV_DEV V row_sum(V v) {
#pragma unroll
  for (int off = LN / 2; off >= 1; off >>= 1) v += __shfl_xor(v, off, 64);
  return v;
}

NV_DEV void load8(const float* p, float x[8]) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const nv_f4 w = reinterpret_cast<const nv_f4*>(p)[i];
#pragma unroll
    for (int j = 0; j < 4; ++j) x[4 * i + j] = w[j];
  }
}
NV_DEV void store8(uint16_t* p, const float x[8]) {
  nv_u4 w;
#pragma unroll
  for (int i = 0; i < 4; ++i) w[i] = pack_bf16(x[2 * i], x[2 * i + 1]);
  *reinterpret_cast<nv_u4*>(p) = w;
}
NV_DEV void store8(float* p, const float x[8]) {
#pragma unroll
  for (int i = 0; i < 2; ++i) reinterpret_cast<nv_f4*>(p)[i] = (nv_f4){x[4 * i], x[4 * i + 1], x[4 * i + 2], x[4 * i + 3]};
}

// Two runs of eight elements of a row as loaded, on their way while others are used.
template <typename T>
struct RawRuns {
  static constexpr int N = sizeof(T) / 2;  // 16-byte words of a run
  nv_u4 w[2 * N];
  NV_DEV void load(bool has, const T* row, int e0, int e1) {
#pragma unroll
    for (int i = 0; i < 2 * N; ++i) w[i] = (nv_u4){0, 0, 0, 0};
    if (has) {
#pragma unroll
      for (int i = 0; i < N; ++i) {
        w[i] = reinterpret_cast<const nv_u4*>(row + e0)[i];
        w[N + i] = reinterpret_cast<const nv_u4*>(row + e1)[i];
      }
    }
  }
  NV_DEV void values(float x[16]) const {
#pragma unroll
    for (int i = 0; i < 2 * N; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if (N == 1) {
          x[8 * i + 2 * j] = bits2f(w[i][j] << 16);
          x[8 * i + 2 * j + 1] = bits2f(w[i][j] & 0xFFFF0000u);
        } else {
          x[4 * i + j] = bits2f(w[i][j]);
        }
      }
  }
};

// The value that T holds for 64-bit v: rounded to fp32, and from there to bf16 as
// torch converts them.  (A value within 2^-24 of the middle between two bf16 may
// take the other one.)
template <typename T>
NV_DEV float rounded(double v) {
  if (sizeof(T) == 4) return (float)v;
  return bits2f(pack_bf16((float)v, 0.0f) << 16);
}

// Where a lane's two runs of eight elements lie in a row, and whether they turn.
template <bool INTER>
struct Runs {
  int e0, e1;
  bool in, turn;
  NV_DEV Runs(int p, int D, int R) {
    in = 16 * p < D;
    turn = 16 * p < R;
    const bool half = !INTER && turn;
    e0 = half ? 8 * p : 16 * p;
    e1 = half ? 8 * p + R / 2 : 16 * p + 8;
  }
};

// Pairs of the two runs: (a_j, b_j), or neighbours within each run.
template <bool INTER, typename V>
NV_DEV void rotate(V y[16], const V c[8], const V s[8], bool back) {
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const int i = INTER ? 2 * j : j, k = INTER ? 2 * j + 1 : 8 + j;
    const V sj = back ? -s[j] : s[j], a = y[i], b = y[k];
    if constexpr (sizeof(V) == 8) {
      y[i] = __builtin_fma(a, c[j], -(b * sj));
      y[k] = __builtin_fma(b, c[j], a * sj);
    } else {
      y[i] = __builtin_fmaf(a, c[j], -(b * sj));
      y[k] = __builtin_fmaf(b, c[j], a * sj);
    }
  }
}

// A token's sines and cosines, a lane each, through the wave's own shared memory
// to the lanes that turn pairs 8 p .. 8 p + 7.
template <int LN, typename V>
NV_DEV void angles(const RopeArgs& a, int t, int lane, bool turn, SinCos* lds, V c[8], V s[8]) {
  const double at = (double)a.positions[t];
  for (int i = lane; i < a.R / 2; i += 64) lds[i] = sincos64(at * a.freqs[i]);
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
  const int p = lane % LN;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const SinCos v = turn ? lds[8 * p + j] : SinCos{0.0, 1.0};
    c[j] = turn ? (V)(v.c * a.mult) : (V)1;
    s[j] = turn ? (V)(v.s * a.mult) : (V)0;
  }
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
}

// A lane group's row of a token: of which kind, of which head, where its runs lie.
struct Row {
  bool is_q, is_v, has;
  int h, e0, e1;
};

// The next row is on its way while one is used, within a token.  Measured, us, without and with
// it: 16384 tokens of 8 heads of 128 to the cache 29 and 25, 8192 of 40 heads with norm and
// rotation 60 and 50; the grid of what runs at a time (rope_groups) takes these to 23 and 49.
// Over the end of a token too, as the gradient has it, costs 170 registers: 27 and 59.
// 16-bit rows that go to the outputs have registers for four waves on a SIMD: 8192 tokens of 40
// heads of 128 36.5 -> 34.3.  32-bit rows spill with so few: 20 heads of 64 21 -> 26.
template <typename T, int LN, bool INTER, bool CACHE>
__global__ __launch_bounds__(256, sizeof(T) == 2 && !CACHE ? 4 : 2) void k_norm_rope(const RopeArgs a, int chunks, int per) {
  constexpr int RW = 64 / LN;
  __shared__ SinCos lds[4][8 * LN];
  const int lane = threadIdx.x & 63, p = lane % LN;
  const int Hq = a.q.heads, Hk = a.k.heads, rows = Hq + Hk + (CACHE ? Hk : 0);
  const Runs<INTER> at(p, a.D, a.R);
  for (int64_t u = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6); u < (int64_t)a.T * chunks; u += (int64_t)gridDim.x * 4) {
    const int64_t t = u / chunks;
    const int first = (int)(u - t * chunks) * per * RW;
    const int slot = CACHE ? a.slots[t] : 0;
    const bool kept = !CACHE || slot_ok(a.c, slot);
    const int stop = first + per * RW < rows ? first + per * RW : rows;
    auto row_of = [&](int r0) {
      Row o;
      const int row = r0 + lane / LN;
      o.is_q = row < Hq, o.is_v = CACHE && row >= Hq + Hk, o.has = row < stop && at.in && (o.is_q || kept);
      o.h = o.is_q ? row : o.is_v ? row - Hq - Hk : row - Hq;
      o.e0 = o.is_v ? 16 * p : at.e0, o.e1 = o.is_v ? 16 * p + 8 : at.e1;
      return o;
    };
    auto fetch = [&](const Row& o, RawRuns<T>& raw) {
      const HeadsView& view = o.is_q ? a.q : o.is_v ? a.v : a.k;
      raw.load(o.has, (const T*)view.at + t * view.token + o.h * view.head, o.e0, o.e1);
    };
    RawRuns<T> next;
    fetch(row_of(first), next);
    double c[8], s[8];
    if (a.R) angles<LN>(a, (int)t, lane, at.turn, lds[threadIdx.x >> 6], c, s);
    for (int r0 = first; r0 < stop; r0 += RW) {
      const Row row = row_of(r0);
      const bool is_q = row.is_q, is_v = row.is_v, has = row.has;
      const int h = row.h, e0 = row.e0, e1 = row.e1, heads = is_q ? Hq : Hk;
      float x[16];
      next.values(x);
      if (r0 + RW < stop) fetch(row_of(r0 + RW), next);
      const float* w = is_q ? a.qw : a.kw;
      float o[16];
      if (w != nullptr || a.R) {  // otherwise the rows are taken as they are
        double y[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) y[i] = (double)x[i];
        if (a.qw || a.kw) {
          double sum = 0.0;
#pragma unroll
          for (int i = 0; i < 16; ++i) sum = __builtin_fma(y[i], y[i], sum);
          const double rstd = inverse_root(row_sum<LN>(sum) / a.D + a.eps);
          if (w && has && !is_v) {
            float f[16];
            load8(w + e0, f);
            load8(w + e1, f + 8);
#pragma unroll
            for (int i = 0; i < 16; ++i) y[i] = y[i] * rstd * (double)f[i];
          }
        }
        if (a.R && at.turn) rotate<INTER>(y, c, s, false);
#pragma unroll
        for (int i = 0; i < 16; ++i) o[i] = is_v ? x[i] : rounded<T>(y[i]);
      } else {
#pragma unroll
        for (int i = 0; i < 16; ++i) o[i] = x[i];
      }
      if (has && (is_q || !CACHE)) {
        T* dst = (T*)(is_q ? a.q_out : a.k_out) + (t * heads + h) * a.D;
        store8(dst + e0, o);
        store8(dst + e1, o + 8);
      }
      if (!CACHE || __builtin_amdgcn_ballot_w64(has && !is_q) == 0) continue;
      if (!INTER && a.R && __builtin_amdgcn_ballot_w64(has && !is_q && !is_v)) {
        // keys in the layout of halves: back to sixteen elements in a row for a lane
        const int base = lane - p, turned = a.R / 16;
        float n[16];
#pragma unroll
        for (int g = 0; g < 2; ++g) {
          const int run = 2 * p + g;
          const bool second = run < 2 * turned ? run >= turned : g == 1;
          const int from = base + (run < turned ? run : run < 2 * turned ? run - turned : p);
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const float lo = __shfl(o[j], from, 64), hi = __shfl(o[8 + j], from, 64);
            n[8 * g + j] = second ? hi : lo;
          }
        }
#pragma unroll
        for (int i = 0; i < 16; ++i) o[i] = is_v ? o[i] : n[i];
      }
      if (has && !is_q) {
        const float* amax = is_v ? a.c.va : a.c.ka;
        uint32_t byte;
        const nv_u2 code = encode16(o, amax != nullptr, amax ? amax[h] : 1.0f, byte);
        const int64_t to = cache_row(a.c, slot, h);
        *reinterpret_cast<nv_u2*>((is_v ? a.c.v : a.c.k) + to * (a.D / 2) + 8 * p) = code;
        (is_v ? a.c.vs : a.c.ks)[to * (a.D / 16) + p] = (uint8_t)byte;
      }
    }
  }
}

// A wave has tokens in turn and keeps its sums of dw in registers over all of them; a
// workgroup's four meet in shared memory, and a second kernel adds the workgroups' in order.
// 8192 tokens, 40 heads of 128, bf16: called by itself over and over, 51 to 54 us with the second
// kernel's 4.7, 252 MB at 4.7 to 4.9 TB/s, a part of them still in the last cache; behind the forward
// pass 57 + 5.  Bound by memory; three waves on a SIMD (two, 32-bit rows), each with its next rows on
// their way, also over the end of a token, are all of the grid.
template <typename T, int LN, bool INTER>
__global__ __launch_bounds__(256, sizeof(T) == 2 ? 3 : 2) void k_norm_rope_bwd(const RopeArgs a, const HeadsView dq, const HeadsView dk, float* __restrict__ partial) {
  constexpr int RW = 64 / LN;
  __shared__ SinCos lds[4][8 * LN];
  __shared__ float sums[4][16 * LN];
  const int lane = threadIdx.x & 63, p = lane % LN, wv = threadIdx.x >> 6;
  const Runs<INTER> at(p, a.D, a.R);
  float dw[2][16];
#pragma unroll
  for (int i = 0; i < 32; ++i) dw[i / 16][i % 16] = 0.0f;
  // the next rows are on their way while these are used, across kinds and tokens
  RawRuns<T> gn, yn;
  auto fetch = [&](bool keys, int64_t t, int h0) {
    const HeadsView &dz = keys ? dk : dq, &view = keys ? a.k : a.q;
    const int h = h0 + lane / LN;
    const bool has = h < view.heads && at.in;
    gn.load(has, (const T*)dz.at + t * dz.token + h * dz.head, at.e0, at.e1);
    yn.load(has && (keys ? a.kw : a.qw), (const T*)view.at + t * view.token + h * view.head, at.e0, at.e1);
  };
  const int64_t t0 = (int64_t)blockIdx.x * 4 + wv, step = (int64_t)gridDim.x * 4;
  if (t0 < a.T) fetch(a.q.heads == 0, t0, 0);
  for (int64_t t = t0; t < a.T; t += step) {
    float c[8], s[8];
    if (a.R) angles<LN>(a, (int)t, lane, at.turn, lds[wv], c, s);
#pragma unroll
    for (int kind = 0; kind < 2; ++kind) {
      const HeadsView& view = kind ? a.k : a.q;
      const float* w = kind ? a.kw : a.qw;
      T* dst = (T*)(kind ? a.k_out : a.q_out);
      for (int h0 = 0; h0 < view.heads; h0 += RW) {
        const int h = h0 + lane / LN;
        const bool has = h < view.heads && at.in;
        float d[16], x[16];
        gn.values(d);
        yn.values(x);
        const bool more = h0 + RW < view.heads, keys = more ? kind : kind == 0 && a.k.heads || a.q.heads == 0;
        const int64_t then = more || (kind == 0 && a.k.heads) ? t : t + step;
        if (then < a.T) fetch(keys, then, more ? h0 + RW : 0);
        if (a.R && at.turn) rotate<INTER>(d, c, s, true);
        if (w) {
          float f[16];
#pragma unroll
          for (int i = 0; i < 16; ++i) f[i] = 0.0f;
          if (has) {
            load8(w + at.e0, f);
            load8(w + at.e1, f + 8);
          }
          // sums in 64 bits: squares of 32-bit rows may leave the range of fp32
          double sq = 0.0, dx = 0.0;
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            sq = __builtin_fma((double)x[i], (double)x[i], sq);
            dx = __builtin_fma((double)(d[i] * f[i]), (double)x[i], dx);
          }
          const double root = inverse_root(row_sum<LN>(sq) / a.D + a.eps);
          const float rstd = (float)root, mean = (float)(row_sum<LN>(dx) * root / a.D);
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            const float n = x[i] * rstd;
            if (has) dw[kind][i] = __builtin_fmaf(d[i], n, dw[kind][i]);
            d[i] = rstd * __builtin_fmaf(-n, mean, d[i] * f[i]);
          }
        }
        if (has) {
          T* to = dst + (t * view.heads + h) * a.D;
          store8(to + at.e0, d);
          store8(to + at.e1, d + 8);
        }
      }
    }
  }
  if (!partial) return;
#pragma unroll
  for (int kind = 0; kind < 2; ++kind) {
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      float v = dw[kind][i];
#pragma unroll
      for (int off = LN; off < 64; off <<= 1) v += __shfl_xor(v, off, 64);
      const int e = (i < 8 ? at.e0 : at.e1 - 8) + i;
      if (lane < LN && at.in) sums[wv][e] = v;
    }
    __syncthreads();
    for (int e = threadIdx.x; e < a.D; e += 256)
      partial[((int64_t)blockIdx.x * 2 + kind) * a.D + e] = (sums[0][e] + sums[1][e]) + (sums[2][e] + sums[3][e]);
    __syncthreads();
  }
}

// Sixteen elements a lane; grid y: keys, values.  16384 tokens of 8 heads of 128: 16 us,
// 86 MB at 5.3 TB/s.  (Stores past the caches: 30 us.)
template <typename T>
__global__ __launch_bounds__(256) void k_read_cache(const CacheView c, const int* __restrict__ slots, int64_t n, T* __restrict__ k, T* __restrict__ v) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= n) return;
  const int per = c.dim / 16, p = (int)(i % per);
  const int64_t row = i / per, t = row / c.heads;
  const int h = (int)(row - t * c.heads), slot = slots[t];
  const bool keys = blockIdx.y == 0;
  float x[16];
#pragma unroll
  for (int j = 0; j < 16; ++j) x[j] = 0.0f;
  if (slot_ok(c, slot)) {
    const int64_t at = cache_row(c, slot, h) * per + p;
    const nv_u2 w = reinterpret_cast<const nv_u2*>(keys ? c.k : c.v)[at];
    const float s = hw_e4m3_value<0>((keys ? c.ks : c.vs)[at]);
    const float* amax = keys ? c.ka : c.va;
    const float dec = amax ? amax[h] / 2688.0f : 1.0f;
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const nv_f2 v0 = hw_fp4_values<0>(w[j]), v1 = hw_fp4_values<1>(w[j]), v2 = hw_fp4_values<2>(w[j]), v3 = hw_fp4_values<3>(w[j]);
      const float f[8] = {v0.x, v0.y, v1.x, v1.y, v2.x, v2.y, v3.x, v3.y};
#pragma unroll
      for (int e = 0; e < 8; ++e) x[8 * j + e] = (f[e] * s) * dec;
    }
  }
  T* to = (keys ? k : v) + i * 16;
  store8(to, x);
  store8(to + 8, x + 8);
}

template <typename T, int LN, bool INTER>
static void rope_go(const RopeArgs& a, hipStream_t st) {
  const int rows = a.q.heads + a.k.heads + (a.slots ? a.k.heads : 0);
  const LayerLaunch p = plan_rope(a.T, rows, a.D, a.in_bf16, a.slots != nullptr);
  const int64_t chunks = rope_chunks(a.T, rows, a.D), per = ceil_div(rope_passes(rows, a.D), chunks);
  if (a.slots) k_norm_rope<T, LN, INTER, true><<<(uint32_t)p.grid, p.block, 0, st>>>(a, (int)chunks, (int)per);
  else k_norm_rope<T, LN, INTER, false><<<(uint32_t)p.grid, p.block, 0, st>>>(a, (int)chunks, (int)per);
}

#define NV_ROPE(CALL)                                       \
  {                                                         \
    switch (rope_lanes(a.D)) {                              \
      case 4: CALL(4); break;                               \
      case 8: CALL(8); break;                               \
      case 16: CALL(16); break;                             \
      default: CALL(32);                                    \
    }                                                       \
  }

int launch_norm_rope(const RopeArgs& a, void* stream) {
  hipStream_t st = (hipStream_t)stream;
#define NV_GO(LN)                                                                                  \
  if (a.in_bf16) a.interleaved ? rope_go<uint16_t, LN, true>(a, st) : rope_go<uint16_t, LN, false>(a, st); \
  else a.interleaved ? rope_go<float, LN, true>(a, st) : rope_go<float, LN, false>(a, st)
  NV_ROPE(NV_GO)
#undef NV_GO
  return (int)hipGetLastError();
}

size_t rope_bwd_workspace_bytes(int64_t T, int64_t D) { return (size_t)(rope_bwd_groups(T, true) * 2 * D * 4); }

template <typename T, int LN, bool INTER>
static void rope_bwd_go(const RopeArgs& a, const HeadsView& dq, const HeadsView& dk, float* partial, hipStream_t st) {
  const LayerLaunch p = plan_rope_bwd(a.T, a.in_bf16);
  k_norm_rope_bwd<T, LN, INTER><<<(uint32_t)p.grid, p.block, 0, st>>>(a, dq, dk, partial);
}

int launch_norm_rope_bwd(const RopeArgs& a, const HeadsView& dq, const HeadsView& dk, float* dw, void* ws, void* stream) {
  hipStream_t st = (hipStream_t)stream;
  float* partial = dw ? (float*)ws : nullptr;
  if (a.T > 0) {
#define NV_GO(LN)                                                                                                            \
  if (a.in_bf16) a.interleaved ? rope_bwd_go<uint16_t, LN, true>(a, dq, dk, partial, st) : rope_bwd_go<uint16_t, LN, false>(a, dq, dk, partial, st); \
  else a.interleaved ? rope_bwd_go<float, LN, true>(a, dq, dk, partial, st) : rope_bwd_go<float, LN, false>(a, dq, dk, partial, st)
    NV_ROPE(NV_GO)
#undef NV_GO
  }
  if (dw) return launch_sum_rows(partial, (int)rope_bwd_groups(a.T, a.in_bf16), 2 * (int64_t)a.D, dw, stream);
  return (int)hipGetLastError();
}

int launch_read_cache(const CacheView& c, const int* slots, int64_t T, void* k, void* v, int out_bf16, void* stream) {
  const LayerLaunch p = plan_read_cache(T, c.heads, c.dim);
  const dim3 grid((uint32_t)p.grid, (uint32_t)p.y);
  const int64_t n = T * c.heads * (c.dim / 16);
  if (out_bf16) k_read_cache<uint16_t><<<grid, p.block, 0, (hipStream_t)stream>>>(c, slots, n, (uint16_t*)k, (uint16_t*)v);
  else k_read_cache<float><<<grid, p.block, 0, (hipStream_t)stream>>>(c, slots, n, (float*)k, (float*)v);
  return (int)hipGetLastError();
}

}  // namespace nvfp4
