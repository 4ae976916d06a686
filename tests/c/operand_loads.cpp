// The operand loads of the matrix products (nvfp4_weight.hpp, nvfp4_buffer.hpp)
// on the CPU: the same source with the range check of a raw buffer load in the
// builtins' place.  The check is the documented one: a word at a lane's offset
// `off` is outside, and reads as zero, where off >= num_records - scalar offset,
// in unsigned 32-bit arithmetic.  Every word that passes has to lie inside the
// buffer, and every buffer inside the array that a caller gives.  Each lane of
// each wave is run over the walks that the kernels make.
#include <stdint.h>
#include <stdio.h>
#include <stdlib.h>
#include <string.h>

#include <string>
#include <vector>

struct Rsrc {
  const char* p;
  uint32_t num;
};
struct Array {
  const char* p;
  size_t n;
};
static std::vector<Array> arrays;  // what a caller gives
static std::string where;
static long faults, loads;

static void fault(const char* what) {
  if (faults++ < 20) printf("%s: %s\n", where.c_str(), what);
}
static Rsrc make_rsrc(void* p, short, int num, int) {
  bool in = num == 0;
  for (const Array& a : arrays) in |= (const char*)p >= a.p && (const char*)p + (uint32_t)num <= a.p + a.n;
  if (!in) fault("a buffer that no array holds");
  return {(const char*)p, (uint32_t)num};
}
// `size` bytes at off of a load whose scalar offset is base
static uint32_t word(Rsrc r, uint32_t off, uint32_t base, uint32_t size) {
  ++loads;
  if (off >= r.num - base) return 0;
  const uint64_t at = (uint64_t)off + base;
  if (at + size > r.num) {
    fault("a load past the end of its buffer");
    return 0;
  }
  uint32_t v = 0;
  memcpy(&v, r.p + at, size);
  return v;
}

typedef unsigned int U4 __attribute__((ext_vector_type(4)));
typedef unsigned int U2 __attribute__((ext_vector_type(2)));
static U4 load4(Rsrc r, int off, int base, int) {
  U4 v;
  for (int i = 0; i < 4; ++i) v[i] = word(r, (uint32_t)off + 4u * i, (uint32_t)base, 4);
  return v;
}
static U2 load2(Rsrc r, int off, int base, int) {
  return U2{word(r, (uint32_t)off, (uint32_t)base, 4), word(r, (uint32_t)off + 4u, (uint32_t)base, 4)};
}

#define NV_DEV inline
#define __amdgpu_buffer_rsrc_t Rsrc
#define __builtin_amdgcn_readfirstlane(v) (v)
#define __builtin_amdgcn_make_buffer_rsrc make_rsrc
#define __builtin_amdgcn_raw_buffer_load_b128 load4
#define __builtin_amdgcn_raw_buffer_load_b64 load2
#define __builtin_amdgcn_raw_buffer_load_b32(r, off, base, aux) word(r, (uint32_t)(off), (uint32_t)(base), 4)
#define __builtin_amdgcn_raw_buffer_load_b8(r, off, base, aux) word(r, (uint32_t)(off), (uint32_t)(base), 1)
// Not run here.
#define __builtin_amdgcn_permlane32_swap(a, b, c, d) (U2{(a), (b)})
#define __builtin_amdgcn_perm(a, b, c) ((a) ^ (b) ^ (c))
static struct {
  unsigned x;
} threadIdx;

#include "nvfp4_weight.hpp"

using namespace nvfp4;

static bool zero(U4 v) { return !(v[0] | v[1] | v[2] | v[3]); }

// The walks of matvec_sums (k_matvec.hip): pieces of 256 k's, one in flight past the last.
template <bool MX8, int BLK, bool WORDS, int XR>
static void matvec(const MatmulArgs& a, int e, int row0, int rows, int n0, int R) {
  const WeightView<BLK> w(a, e, n0, 16 * R);
  const RowsView<MX8> x(a, row0, rows);
  const int nk = (a.K + 255) / 256;
  for (int k = 0; k < nk + 4; ++k)
    for (int lane = 0; lane < 64; ++lane) {
      RowsPiece<MX8, XR> xp;
      xp.load(x, lane, k * 256);
      if (k >= nk)
        for (int i = 0; i < xp.kLoads; ++i)
          if (!zero(xp.c[i])) fault("rows past K are not zero");
      for (int r = 0; r < R; ++r) {
        WeightPiece<BLK, WORDS> wp;
        wp.load(w, r, lane, k * 256);
        if (k >= nk && (wp.s[0] || !zero(wp.c[0]) || !zero(wp.c[1]))) fault("weights past K are not zero");
      }
    }
}

// The walk of grouped_tile (nvfp4_grouped.hpp): steps of 128 k's.
template <bool MX8, int BLK, int BM, int NI>
static void grouped(const MatmulArgs& a, int e, int row0, int rows, int n_tile) {
  const int nk = (a.K + 127) / 128;
  const RowsView<MX8> x(a, row0, rows);
  for (unsigned tid = 0; tid < 256; ++tid) {
    threadIdx.x = tid;
    const int wave = tid >> 6, lane = tid & 63;
    const WeightStream<BLK, NI> w(a, e, n_tile * (128 * NI) + wave * (32 * NI), lane & 31, lane >> 5);
    RowsHalf<MX8, BM> st;
    for (int kt = 0; kt < nk + 2; ++kt) {
      const int k0 = kt * 128;
      for (int h = 0; h < 2; ++h) {
        st.load(x, tid, k0, h);
        if (tid < (unsigned)st.HALF && kt >= nk)
          for (int i = 0; i < st.PIECES; ++i)
            if (!zero(st.c[i])) fault("rows past K are not zero");
      }
      uint32_t v[4];
      w.fetch_scales(k0, v);
      if (kt > nk) continue;
      for (int i = 0; i < NI; ++i)
        for (int q = 0; q < 2; ++q)
          if (!zero(w.codes(i, k0, q)) && kt == nk) fault("codes are read for a step past K");
    }
  }
}

template <bool MX8, int BLK>
static void both(const MatmulArgs& a, int e, int row0, int rows) {
  for (int R : {1, 2, 4})
    for (int n0 = 0; n0 < a.N; n0 += 16 * R) {
      if (a.K % 64 == 0 && BLK != 2) {
        if (rows <= 4) matvec<MX8, BLK, true, 4>(a, e, row0, rows, n0, R);
        if (rows <= 16) matvec<MX8, BLK, true, 16>(a, e, row0, rows, n0, R);
        if (rows <= 32) matvec<MX8, BLK, true, 32>(a, e, row0, rows, n0, R);
      } else {
        if (rows <= 4) matvec<MX8, BLK, false, 4>(a, e, row0, rows, n0, R);
        if (rows <= 16) matvec<MX8, BLK, false, 16>(a, e, row0, rows, n0, R);
        if (rows <= 32) matvec<MX8, BLK, false, 32>(a, e, row0, rows, n0, R);
      }
    }
  for (int t = 0; t * 128 < a.N; ++t) {
    if (rows <= 32) grouped<MX8, BLK, 32, 1>(a, e, row0, rows, t);
    if (rows <= 64) grouped<MX8, BLK, 64, 1>(a, e, row0, rows, t);
    grouped<MX8, BLK, 128, 1>(a, e, row0, rows, t);
  }
  for (int t = 0; t * 256 < a.N; ++t) {
    if (rows <= 32) grouped<MX8, BLK, 32, 2>(a, e, row0, rows, t);
    if (rows <= 64) grouped<MX8, BLK, 64, 2>(a, e, row0, rows, t);
    grouped<MX8, BLK, 128, 2>(a, e, row0, rows, t);
  }
}

int main() {
  const int E = 2;
  for (int K : {16, 48, 64, 128, 144, 256, 272, 400, 528})
    for (int N : {1, 16, 31, 48, 100, 272})
      for (int rows : {1, 3, 4, 5, 16, 17, 33, 64, 100, 128}) {
        if (N == 272 && rows != 1 && rows != 17 && rows != 100) continue;
        const int T = rows + 3, ns = (K + 31) / 32;
        std::vector<char> x(2 * T * K, 0x55), xs(T * ns, 0x55), w(E * N * K / 2, 0x55), ws(E * N * (K / 16), 0x55);
        for (int mx8 = 0; mx8 < 2; ++mx8)
          for (int blk = 0; blk < (N % 16 ? 1 : 3); ++blk) {
            const size_t scales = blk ? (size_t)E * (N / 16) * (K / 16) : ws.size();
            arrays = {{x.data(), (size_t)T * K * (mx8 ? 1 : 2)}, {xs.data(), xs.size()}, {w.data(), w.size()}, {ws.data(), scales}};
            MatmulArgs a = {x.data(), (const uint8_t*)xs.data(), (const uint8_t*)w.data(), (const uint8_t*)ws.data(), nullptr, nullptr, nullptr, T, E, N, K, blk, 0, 0.0f, 1};
            char name[120];
            snprintf(name, sizeof name, "rows %d N %d K %d, %s, blocks %d", rows, N, K, mx8 ? "mx8" : "bf16", blk);
            where = name;
            const int e = E - 1, row0 = T - rows;  // the last ones: nothing lies behind them
            if (mx8) blk == 0 ? both<true, 0>(a, e, row0, rows) : blk == 1 ? both<true, 1>(a, e, row0, rows) : both<true, 2>(a, e, row0, rows);
            else blk == 0 ? both<false, 0>(a, e, row0, rows) : blk == 1 ? both<false, 1>(a, e, row0, rows) : both<false, 2>(a, e, row0, rows);
          }
      }
  printf("%ld words, %ld faults\n", loads, faults);
  return faults != 0;
}
