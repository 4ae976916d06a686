// Gated activation with 8-bit checkpoints, and its gradient from them.
//
//   y = g sigma(g) u for rows [g | u] of gate_up, written as mx8; with `kept`
//   the same read also writes g and u as mx8, the checkpoint.
//   backward: dg = dy u sigma(g) (1 + g (1 - sigma(g))),  du = dy g sigma(g),
//   with g and u the checkpoint's values.
//
// Bound by memory.  A lane takes 16 elements of g and of u (half an mx8
// group), so every load and code store is 16 bytes wide.
#include "nvfp4_launch.hpp"
#include "nvfp4_mx8.hpp"
#include "nvfp4_plan.hpp"

namespace nvfp4 {

// sigma(g) from t = e^-|g| = 2^(-|g| log2 e), which never overflows: 1 / (1 +
// t) for g >= 0, t / (1 + t) below.  The rounding error of |g| log2 e, up to
// |g| 2^-24 in the exponent, is carried along as a first-order factor.  2^x
// loses subnormal results, so far exponents are raised by 64 (exact there)
// and the result is scaled back.  A NaN gives 0 or 1: callers multiply by g.
NV_DEV float sigmoid(float g) {
  const float L = 1.44269502f, Llo = 1.92596299e-8f, ln2 = 0.693147182f;
  const float a = fminf(__builtin_fabsf(g), 1e4f);
  const float p = -a * L;
  const float err = __builtin_fmaf(-a, L, -p) - a * Llo;
  const bool far = p < -100.0f;
  float t = __builtin_amdgcn_exp2f(far ? p + 64.0f : p);
  t = __builtin_fmaf(t, err * ln2, t) * (far ? 0x1p-64f : 1.0f);
  const float r = __builtin_amdgcn_rcpf(1.0f + t);
  return g < 0.0f ? t * r : r;
}

// The same in 64 bits, to 2^-40 or so.
NV_DEV double sigmoid64(double g) {
  const double t = exp(-fmin(__builtin_fabs(g), 1e4)), d = 1.0 + t;
  double r = __builtin_amdgcn_rcp(d);
  r = __builtin_fma(r, __builtin_fma(-d, r, 1.0), r);
  return g < 0.0 ? t * r : r;
}

template <typename T, bool KEEP>
__global__ __launch_bounds__(256) void k_swiglu(const T* __restrict__ gate_up, uint32_t rows, uint32_t F,
                                                uint32_t lanes_row, uint8_t* __restrict__ codes,
                                                uint8_t* __restrict__ scales, uint8_t* __restrict__ kept,
                                                uint8_t* __restrict__ kept_scales) {
  const uint32_t id = blockIdx.x * 256u + threadIdx.x;
  const uint32_t row = id / lanes_row, j = (id - row * lanes_row) * 16u;
  const bool in = row < rows && j < F;
  const uint32_t ns = lanes_row / 2;
  float g[16], u[16], y[16];
  const int64_t at = (int64_t)row * (2 * (int64_t)F) + j;
  if (in) {
    load16(gate_up + at, g);
    load16(gate_up + at + F, u);
  } else {
#pragma unroll
    for (int i = 0; i < 16; ++i) g[i] = u[i] = 0.0f;
  }
  // A code next to a border shows the last bits of y.  32-bit input takes 64
  // bits for it (1000 x 2048: 6.8 us either way, no code off where 32 bits had 1
  // in 2.5 million); 16-bit input has gates and ups of 8 bits and was not seen to
  // need it.
  constexpr bool WIDE = sizeof(T) == 4;
#pragma unroll
  for (int i = 0; i < 16; ++i)
    y[i] = WIDE ? round_odd((double)g[i] * sigmoid64(g[i]) * (double)u[i]) : g[i] * sigmoid(g[i]) * u[i];
  nv_u4 qy, qg, qu;
  const uint32_t by = mx8_encode16(y, qy);
  uint32_t bg = 0, bu = 0;
  if (KEEP) {
    bg = mx8_encode16(g, qg);
    bu = mx8_encode16(u, qu);
  }
  if (!in) return;
  stream_out(reinterpret_cast<nv_u4*>(codes + (int64_t)row * F + j), qy);
  if (KEEP) {
    stream_out(reinterpret_cast<nv_u4*>(kept + at), qg);
    stream_out(reinterpret_cast<nv_u4*>(kept + at + F), qu);
  }
  if (j % kMxGroup == 0) {
    scales[(int64_t)row * ns + j / kMxGroup] = (uint8_t)by;
    if (KEEP) {
      kept_scales[(int64_t)row * 2 * ns + j / kMxGroup] = (uint8_t)bg;
      kept_scales[(int64_t)row * 2 * ns + ns + j / kMxGroup] = (uint8_t)bu;
    }
  }
}

template <typename T>
__global__ __launch_bounds__(256) void k_swiglu_bwd(const T* __restrict__ dout, uint32_t rows, uint32_t F,
                                                    uint32_t lanes_row, const uint8_t* __restrict__ kept,
                                                    const uint8_t* __restrict__ kept_scales,
                                                    T* __restrict__ dgate_up) {
  const uint32_t id = blockIdx.x * 256u + threadIdx.x;
  const uint32_t row = id / lanes_row, j = (id - row * lanes_row) * 16u;
  if (row >= rows || j >= F) return;
  const uint32_t ns = lanes_row / 2;
  const int64_t at = (int64_t)row * (2 * (int64_t)F) + j;
  float g[16], u[16], d[16];
  const float sg = e8m0_value(kept_scales[(int64_t)row * 2 * ns + j / kMxGroup]);
  const float su = e8m0_value(kept_scales[(int64_t)row * 2 * ns + ns + j / kMxGroup]);
  mx8_values16(*reinterpret_cast<const nv_u4*>(kept + at), sg, g);
  mx8_values16(*reinterpret_cast<const nv_u4*>(kept + at + F), su, u);
  load16(dout + (int64_t)row * F + j, d);
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    const float s = sigmoid(g[i]);
    const float dg = d[i] * u[i] * s * (1.0f + g[i] * (1.0f - s));
    u[i] = d[i] * g[i] * s;
    g[i] = dg;
  }
  store16(dgate_up + at, g);
  store16(dgate_up + at + F, u);
}

int launch_swiglu(const void* gate_up, int in_bf16, int64_t rows, int64_t F, uint8_t* codes, uint8_t* scales,
                  uint8_t* kept, uint8_t* kept_scales, void* stream) {
  hipStream_t st = (hipStream_t)stream;
  const uint32_t lanes = (uint32_t)swiglu_lanes(F);
  const LayerLaunch p = plan_swiglu(rows, F);
  const dim3 grid((uint32_t)p.grid);
#define NV_SW(T, KEEP) k_swiglu<T, KEEP><<<grid, p.block, 0, st>>>((const T*)gate_up, (uint32_t)rows, (uint32_t)F, lanes, codes, scales, kept, kept_scales)
  if (in_bf16) {
    if (kept) NV_SW(uint16_t, true);
    else NV_SW(uint16_t, false);
  } else {
    if (kept) NV_SW(float, true);
    else NV_SW(float, false);
  }
#undef NV_SW
  return (int)hipGetLastError();
}

int launch_swiglu_bwd(const void* dout, int in_bf16, int64_t rows, int64_t F, const uint8_t* kept,
                      const uint8_t* kept_scales, void* dgate_up, void* stream) {
  hipStream_t st = (hipStream_t)stream;
  const uint32_t lanes = (uint32_t)swiglu_lanes(F);
  const LayerLaunch p = plan_swiglu(rows, F);
  const dim3 grid((uint32_t)p.grid);
  if (in_bf16)
    k_swiglu_bwd<uint16_t><<<grid, p.block, 0, st>>>((const uint16_t*)dout, (uint32_t)rows, (uint32_t)F, lanes, kept,
                                                 kept_scales, (uint16_t*)dgate_up);
  else
    k_swiglu_bwd<float><<<grid, p.block, 0, st>>>((const float*)dout, (uint32_t)rows, (uint32_t)F, lanes, kept,
                                              kept_scales, (float*)dgate_up);
  return (int)hipGetLastError();
}

}  // namespace nvfp4
