// Root-mean-square norm of x + residual with 8-bit output, and its gradient.
//
//   h = x + r,  rstd = (mean_j h_j^2 + eps)^(-1/2),  y_j = h_j rstd w_j
//   forward writes y as mx8 (codes, scales), h in x's type and rstd
//   n = h rstd,  d = dy w,  dh = rstd (d - n mean_j(d_j n_j)) + dhidden,
//   dw_j = sum over rows of dy_j n_j
//
// Both directions are bound by memory: every tensor is read once and written
// once, the row stays in registers between its sum and its output.  A lane
// holds 16 elements (half an mx8 group, so a group's maximum is one
// cross-lane step) of one row, two such chunks for rows over 16384.
#include "nvfp4_launch.hpp"
#include "nvfp4_mx8.hpp"
#include "nvfp4_plan.hpp"

namespace nvfp4 {

NV_DEV double value_of(uint16_t v) { return (double)bits2f((uint32_t)v << 16); }
NV_DEV double value_of(float v) { return (double)v; }

template <typename T, int C, bool RES>
__global__ __launch_bounds__(1024) void k_add_rms_norm(const T* __restrict__ x, const T* __restrict__ res,
                                                       const float* __restrict__ weight, int64_t rows, int H,
                                                       float eps, uint8_t* __restrict__ codes,
                                                       uint8_t* __restrict__ scales, T* __restrict__ hidden,
                                                       float* __restrict__ rstd_out) {
  // A code next to a border shows the last bits of y.  The sum over the row's
  // lanes and the root are in 64 bits.  Of 32-bit rows all else is too, from both
  // addends (8.9 -> 9.9 us at 1021 x 2064, no code off where 32 bits had 1 in 2
  // million).  Of 16-bit ones 64 bits would cost 67 -> 88 us (8192 x 7168): y takes
  // 32 bits, and 64 where that lies within four units of its last place from a
  // border, one element in 60 thousand, read again so that no registers wait for it
  // (all of it kept: 74 us; so: 65.8 -> 66.9, 4096 x 18432 109 -> 114).  Of 59 million
  // codes 7 are off, by the lanes' 32-bit sums of squares; of y in 32 bits with its
  // rounding errors carried along 30 were, a plain fp32 norm has 39.
  constexpr bool WIDE = sizeof(T) == 4;
  __shared__ double lds[16];
  const int nt = blockDim.x, ns = (H + kMxGroup - 1) / kMxGroup;
  const double inv_h = 1.0 / H;
  for (int64_t row = blockIdx.x; row < rows; row += gridDim.x) {
    const int64_t at = row * H;
    float h[C][16], r[C][16];
    double total = 0.0;
    float sum = 0.0f;
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const int j = (c * nt + threadIdx.x) * 16;
#pragma unroll
      for (int i = 0; i < 16; ++i) h[c][i] = r[c][i] = 0.0f;
      if (j < H) {
        load16(x + at + j, h[c]);
        if (RES) load16(res + at + j, r[c]);
      }
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        if (WIDE) {
          const double v = (double)h[c][i] + (double)r[c][i];
          total = __builtin_fma(v, v, total);
        } else {
          if (RES) h[c][i] += r[c][i];
          sum = __builtin_fmaf(h[c][i], h[c][i], sum);
        }
      }
    }
    double var = __builtin_fma(block_sum(WIDE ? total : (double)sum, lds), inv_h, (double)eps);
    // Rows of 16 bits whose squares left the range of fp32 (all lanes agree) are
    // taken times a power of two from here on.  (64 bits for them took 114
    // registers, not 70, from all rows: 66 -> 74 us at 8192 x 7168.)
    float by = 1.0f;
    if (!WIDE && !(var > 0x1p-100 && var < INFINITY)) {
      by = var <= 0x1p-100 ? 0x1p80f : 0x1p-80f;
      sum = 0.0f;
#pragma unroll
      for (int c = 0; c < C; ++c)
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const float v = h[c][i] * by;
          sum = __builtin_fmaf(v, v, sum);
        }
      var = __builtin_fma(block_sum((double)sum, lds), inv_h, (double)eps * by * by);
    }
    const double near = __builtin_amdgcn_rsq(var);  // to 2^-22 or so, then one step of Newton's method
    const double off = near * (0.5 * __builtin_fma(-var * near, near, 1.0));
    const double root = off == off ? near + off : near;
    const float rstd = (float)root;
    if (threadIdx.x == 0) rstd_out[row] = WIDE ? rstd : (float)(root * by);
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const int j = (c * nt + threadIdx.x) * 16;
      const bool in = j < H;
      float w[16], y[16];
      if (in) {
        if (RES) {
          float sum16[16];
#pragma unroll
          for (int i = 0; i < 16; ++i) sum16[i] = WIDE ? h[c][i] + r[c][i] : h[c][i];
          store16(hidden + at + j, sum16);
        }
        load16(weight + j, w);
      } else {
#pragma unroll
        for (int i = 0; i < 16; ++i) w[i] = 0.0f;
      }
      if (!WIDE) {
#pragma unroll
        for (int i = 0; i < 16; ++i) h[c][i] *= by;
      }
      if (WIDE && RES) {  // added again: sums kept in 64 bits would take twice the registers
#pragma unroll
        for (int i = 0; i < 16; ++i) asm("" : "+v"(h[c][i]), "+v"(r[c][i]));
      }
      uint32_t border = ~0u;
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        if (WIDE) {
          const double v = RES ? (double)h[c][i] + (double)r[c][i] : (double)h[c][i];
          y[i] = round_odd(v * root * (double)w[i]);
        } else {
          y[i] = h[c][i] * rstd * w[i];
          const uint32_t d = border_distance<4>(y[i]);
          border = d < border ? d : border;
        }
      }
      if (!WIDE && in && border <= 8) {
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          if (border_distance<4>(y[i]) > 8 || y[i] == 0.0f) continue;
          const int64_t k = at + j + i;
          const double v = RES ? value_of(x[k]) + value_of(res[k]) : value_of(x[k]);
          y[i] = round_odd(v * (root * by) * (double)weight[j + i]);
        }
      }
      if (!in) {  // a missing half group counts as zeros, also where rstd is not finite
#pragma unroll
        for (int i = 0; i < 16; ++i) y[i] = 0.0f;
      }
      nv_u4 q;
      const uint32_t byte = mx8_encode16(y, q);
      if (in) {
        stream_out(reinterpret_cast<nv_u4*>(codes + at + j), q);
        if (j % kMxGroup == 0) scales[row * ns + j / kMxGroup] = (uint8_t)byte;
      }
    }
  }
}

// 16 elements of a row as loaded.  again() makes the compiler take them from
// there a second time instead of keeping what values() gave.
template <typename T>
struct Raw {
  nv_u4 q[sizeof(T)];
  NV_DEV void load(const T* p) {
#pragma unroll
    for (int i = 0; i < (int)sizeof(T); ++i) q[i] = reinterpret_cast<const nv_u4*>(p)[i];
  }
  NV_DEV void again() {
#pragma unroll
    for (int i = 0; i < (int)sizeof(T); ++i) asm("" : "+v"(q[i]));
  }
  NV_DEV void values(float v[16]) const {
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      if constexpr (sizeof(T) == 4) v[i] = bits2f(q[i >> 2][i & 3]);
      else v[i] = bits2f(i & 1 ? q[i >> 3][(i >> 1) & 3] & 0xFFFF0000u : q[i >> 3][(i >> 1) & 3] << 16);
    }
  }
};

// A workgroup takes every gridDim-th row, keeps its share of dw in registers
// and leaves one partial row of dw.  Of rows up to 16384 the weight stays in
// registers too (2048 x 16384 fp32: 145 -> 126 us), and bf16 rows have some left
// for the next row's dy and hidden, which are then in flight during this row's
// sum (8192 x 7168 with the sum of the partial rows: 118 -> 96 us).  Rows over
// 16384 keep dy and hidden as loaded and dw in shared memory, and read the
// weight again and dhidden only after the sum: with all of it in registers 37 to
// 71 of them spilled (4096 x 18432 bf16: 313 -> 181 us, 2048 x 18432 fp32: 283 ->
// 238).
template <typename T, int C, bool DH>
__global__ __launch_bounds__(1024) void k_add_rms_norm_bwd(const T* __restrict__ dy, const T* __restrict__ hidden,
                                                           const T* __restrict__ dhidden,
                                                           const float* __restrict__ weight,
                                                           const float* __restrict__ rstd_in, int64_t rows, int H,
                                                           T* __restrict__ dx, float* __restrict__ partial) {
  constexpr bool AHEAD = C == 1 && sizeof(T) == 2;
  __shared__ float lds[16];
  const int nt = blockDim.x, j0 = threadIdx.x * 16;
  const float inv_h = 1.0f / (float)H;
  __shared__ float acc[C > 1 ? kNormMaxH : 1];  // dw of long rows; a lane's own places, so no barriers
  float dw1[16], w1[16];
#pragma unroll
  for (int i = 0; i < 16; ++i) dw1[i] = 0.0f;
  if (C > 1) {
    for (int i = 0; i < 16 * C; ++i) acc[i * nt + threadIdx.x] = 0.0f;
  }
  Raw<T> rd[C], rn[C];
  auto ahead = [&](int64_t row) {
    if (j0 >= H) return;
    rd[0].load(dy + row * H + j0);
    rn[0].load(hidden + row * H + j0);
  };
  if (C == 1 && j0 < H) load16(weight + j0, w1);
  if (AHEAD) ahead(blockIdx.x);
  for (int64_t row = blockIdx.x; row < rows; row += gridDim.x) {
    const int64_t at = row * H;
    const float rstd = rstd_in[row];
    const float* wp = weight;
    if (C > 1) asm volatile("" : "+s"(wp));  // else the weights stay in registers from row to row
    float d1[16], n1[16];  // of one chunk, from pass to pass
    Raw<T> rh1;
    float dot = 0.0f;
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const int j = (c * nt + threadIdx.x) * 16;
      if (j < H) {
        float d2[16], n2[16], w2[16];
        float(&d)[16] = C > 1 ? d2 : d1, (&n)[16] = C > 1 ? n2 : n1, (&w)[16] = C > 1 ? w2 : w1;
        if (!AHEAD) {
          rd[c].load(dy + at + j);
          rn[c].load(hidden + at + j);
        }
        if (DH && C == 1) rh1.load(dhidden + at + j);
        if (C > 1) load16(wp + j, w);
        rd[c].values(d);
        rn[c].values(n);
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          n[i] *= rstd;
          float& dw = C > 1 ? acc[(c * 16 + i) * nt + threadIdx.x] : dw1[i];
          dw = __builtin_fmaf(d[i], n[i], dw);
          d[i] *= w[i];
          dot = __builtin_fmaf(d[i], n[i], dot);
        }
      }
      if (C > 1) asm volatile("" ::: "memory");
    }
    if (AHEAD && row + gridDim.x < rows) ahead(row + gridDim.x);
    const float mean = block_sum(dot, lds) * inv_h;
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const int j = (c * nt + threadIdx.x) * 16;
      if (j < H) {
        float d2[16], n2[16], w[16], dh[16];
        float(&d)[16] = C > 1 ? d2 : d1, (&n)[16] = C > 1 ? n2 : n1;
        Raw<T> rh2, &rh = C > 1 ? rh2 : rh1;
        if (C > 1) {
          rd[c].again();
          rn[c].again();
          rd[c].values(d);
          rn[c].values(n);
          load16(wp + j, w);
          if (DH) rh.load(dhidden + at + j);
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            n[i] *= rstd;
            d[i] *= w[i];
          }
        }
        if (DH) rh.values(dh);
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const float v = rstd * (d[i] - n[i] * mean);
          d[i] = DH ? v + dh[i] : v;
        }
        store16(dx + at + j, d);
      }
      if (C > 1) asm volatile("" ::: "memory");
    }
  }
#pragma unroll
  for (int c = 0; c < C; ++c) {
    const int j = (c * nt + threadIdx.x) * 16;
    if (j < H) {
      if (C > 1) {
#pragma unroll
        for (int i = 0; i < 16; ++i) dw1[i] = acc[(c * 16 + i) * nt + threadIdx.x];
      }
      store16(partial + (int64_t)blockIdx.x * H + j, dw1);
    }
  }
}

// dw = sum of the partial rows in a fixed order: four lanes cover 16 columns,
// the 64 lane groups of the workgroup take every 64th row, and their sums are
// joined in pairs: one after the other their roundings made up most of dw's error
// (1021 x 2064 fp32: 1.6e-7 -> 0.9e-7 of its size, a sum over rows in plain fp32
// 1.1e-7; both directions 22.9 -> 22.7 us).
__global__ __launch_bounds__(256) void k_sum_rows(const float* __restrict__ partial, int n, int H,
                                                  float* __restrict__ out) {
  __shared__ float lds[64][16];
  const int col = blockIdx.x * 16 + (threadIdx.x & 3) * 4, grp = threadIdx.x >> 2;
  nv_f4 s = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll 8
  for (int r = grp; r < n; r += 64) {
    const nv_f4 v = *reinterpret_cast<const nv_f4*>(partial + (int64_t)r * H + col);
#pragma unroll
    for (int i = 0; i < 4; ++i) s[i] += v[i];
  }
  *reinterpret_cast<nv_f4*>(&lds[grp][(threadIdx.x & 3) * 4]) = s;
  __syncthreads();
  if (threadIdx.x < 16) {
    float t[64];
#pragma unroll
    for (int g = 0; g < 64; ++g) t[g] = lds[g][threadIdx.x];
#pragma unroll
    for (int n = 32; n >= 1; n >>= 1)
#pragma unroll
      for (int g = 0; g < n; ++g) t[g] += t[g + n];
    out[blockIdx.x * 16 + threadIdx.x] = t[0];
  }
}

template <typename T>
static void norm_fwd(const T* x, const T* res, const float* w, int64_t rows, int H, float eps, uint8_t* codes,
                     uint8_t* scales, T* hidden, float* rstd, hipStream_t st) {
  const LayerLaunch p = plan_norm(rows, H);
#define NV_NORM(C, RES) k_add_rms_norm<T, C, RES><<<(uint32_t)p.grid, p.block, 0, st>>>(x, res, w, rows, H, eps, codes, scales, hidden, rstd)
  if (H <= 16 * 1024) {
    if (res) NV_NORM(1, true);
    else NV_NORM(1, false);
  } else {
    if (res) NV_NORM(2, true);
    else NV_NORM(2, false);
  }
#undef NV_NORM
}

int launch_add_rms_norm(const void* x, const void* res, int in_bf16, const float* w, int64_t rows, int64_t H,
                        float eps, uint8_t* codes, uint8_t* scales, void* hidden, float* rstd, void* stream) {
  hipStream_t st = (hipStream_t)stream;
  if (in_bf16)
    norm_fwd<uint16_t>((const uint16_t*)x, (const uint16_t*)res, w, rows, (int)H, eps, codes, scales,
                       (uint16_t*)hidden, rstd, st);
  else
    norm_fwd<float>((const float*)x, (const float*)res, w, rows, (int)H, eps, codes, scales, (float*)hidden, rstd, st);
  return (int)hipGetLastError();
}

size_t norm_bwd_workspace_bytes(int64_t rows, int64_t H) { return (size_t)norm_bwd_groups(rows, H) * H * 4; }

template <typename T>
static void norm_bwd(const T* dy, const T* hidden, const T* dh, const float* w, const float* rstd, int64_t rows,
                     int H, T* dx, float* partial, hipStream_t st) {
  const LayerLaunch p = plan_norm_bwd(rows, H);
#define NV_NORM(C, DH) k_add_rms_norm_bwd<T, C, DH><<<(uint32_t)p.grid, p.block, 0, st>>>(dy, hidden, dh, w, rstd, rows, H, dx, partial)
  if (H <= 16 * 1024) {
    if (dh) NV_NORM(1, true);
    else NV_NORM(1, false);
  } else {
    if (dh) NV_NORM(2, true);
    else NV_NORM(2, false);
  }
#undef NV_NORM
}

int launch_add_rms_norm_bwd(const void* dy, const void* hidden, const void* dh, int in_bf16, const float* w,
                            const float* rstd, int64_t rows, int64_t H, void* dx, float* dw, void* ws,
                            void* stream) {
  hipStream_t st = (hipStream_t)stream;
  const int grid = (int)norm_bwd_groups(rows, H);
  float* partial = (float*)ws;
  if (grid > 0) {
    if (in_bf16)
      norm_bwd<uint16_t>((const uint16_t*)dy, (const uint16_t*)hidden, (const uint16_t*)dh, w, rstd, rows, (int)H,
                         (uint16_t*)dx, partial, st);
    else
      norm_bwd<float>((const float*)dy, (const float*)hidden, (const float*)dh, w, rstd, rows, (int)H, (float*)dx,
                      partial, st);
  }
  return launch_sum_rows(partial, grid, H, dw, stream);
}

int launch_sum_rows(const float* partial, int n, int64_t H, float* out, void* stream) {
  const LayerLaunch p = plan_sum_rows(H);
  k_sum_rows<<<(uint32_t)p.grid, p.block, 0, (hipStream_t)stream>>>(partial, n, (int)H, out);
  return (int)hipGetLastError();
}

}  // namespace nvfp4
