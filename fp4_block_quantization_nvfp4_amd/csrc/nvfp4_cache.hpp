// Device helpers of the operators on an NVFP4 cache.
#pragma once

#include "nvfp4_launch.hpp"
#include "nvfp4_mx8.hpp"

namespace nvfp4 {

// Row of slot `slot` (in range) and head h, in rows of dim elements.
NV_DEV int64_t cache_row(const CacheView& c, int slot, int h) {
  const int page = slot >> c.shift, at = slot & ((1 << c.shift) - 1);
  return (((int64_t)page * c.heads + h) << c.shift) + at;
}
NV_DEV bool slot_ok(const CacheView& c, int slot) { return slot >= 0 && (slot >> c.shift) < c.pages; }

// One block of sixteen elements to codes and scale byte, step by step as
// nvfp4_quantize: round to nearest, with the amax of a second-level scale
// (bound 448) or without (has false).
NV_DEV nv_u2 encode16(const float x[16], bool has, float amax, uint32_t& byte) {
  float S_dec = 1.0f, mul = 0.0f;
  if (has) {
    float S_enc;
    global_scales(amax, 2688.0f, S_enc, S_dec);
    mul = S_enc * (1.0f / 6.0f);
  }
  uint32_t ab = 0;
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    const uint32_t m = f2bits(x[i]) & 0x7FFFFFFFu;
    ab = m > ab ? m : ab;
  }
  const bool special = ab >= 0x7F800000u;
  float a = bits2f(ab);
  if (special) {
    a = 0.0f;
#pragma unroll
    for (int i = 0; i < 16; ++i) a = fmaxf(a, abs_nan0(x[i]));
  }
  const float sigma = fminf(has ? a * mul : div_guarded(a, 6.0f, 1.0f / 6.0f), kE4m3Max);  // NaN -> 448
  byte = hw_e4m3_pair(sigma, 0.0f) & 0xFFu;
  const float rho = encode_reciprocal(e4m3_decode(byte), S_dec);
  nv_u2 w;
  if (!special) {
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      uint32_t c = any_u32();
      c = hw_fp4_pair<0>(c, x[8 * j] * rho, x[8 * j + 1] * rho);
      c = hw_fp4_pair<1>(c, x[8 * j + 2] * rho, x[8 * j + 3] * rho);
      c = hw_fp4_pair<2>(c, x[8 * j + 4] * rho, x[8 * j + 5] * rho);
      c = hw_fp4_pair<3>(c, x[8 * j + 6] * rho, x[8 * j + 7] * rho);
      w[j] = c;
    }
  } else {
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      uint32_t c = 0;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float v = fabsf(x[8 * j + i]) * rho;
        float q;
        const uint32_t mag = e2m1_rtn(v, q);
        const uint32_t neg = v != v ? 0u : f2bits(x[8 * j + i]) >> 31;
        c |= (mag | neg << 3) << (4 * i);
      }
      w[j] = c;
    }
  }
  return w;
}

}  // namespace nvfp4
