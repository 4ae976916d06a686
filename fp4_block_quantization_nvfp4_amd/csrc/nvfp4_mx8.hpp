// Device helpers of the layer operators: 8-bit rows ("mx8"), 4-bit weight
// decode, wave sums.
//
// mx8: e4m3 codes with one e8m0 scale for each 32 consecutive elements of a
// row (the last group of a row may be shorter).  The scale is the smallest
// 2^s, s >= -117, with max |finite value| <= 448 * 2^s; what is not finite is
// coded as NaN.  s >= -117 keeps every value code * 2^s (smallest 2^-9 *
// 2^-117) a normal bf16, so mx8 rows enter the matrix cores exactly, but for one
// at the top: finite values above 248 * 2^120 are rounded to 256 * 2^120 = 2^128,
// which reads back as infinity.
#pragma once

#include "nvfp4_device.hpp"
#include "nvfp4_buffer.hpp"

namespace nvfp4 {

typedef __bf16 nv_bf2 __attribute__((ext_vector_type(2)));
typedef __bf16 nv_bf8 __attribute__((ext_vector_type(8)));
typedef float nv_f4 __attribute__((ext_vector_type(4)));
typedef float nv_f16 __attribute__((ext_vector_type(16)));

constexpr int kMxGroup = 32;  // elements under one e8m0 scale

// ------------------------------------------------------- storage formats

// fp32 pair -> two bf16 in one word, round to nearest even (one conversion
// instruction; a NaN stays a NaN).
NV_DEV uint32_t pack_bf16(float a, float b) {
  nv_f2 v;
  v.x = a;
  v.y = b;
  return __builtin_bit_cast(uint32_t, __builtin_convertvector(v, nv_bf2));
}

// A store of a result that is not read again here: it passes by the L2, which
// keeps the operands (weight gradient of 16 experts 4096 x 2048 in fp32, 537 MB
// written: 358 -> 318 us; norm 8192 x 7168 bf16: 80 -> 67 us).
template <typename V>
NV_DEV void stream_out(V* p, V v) {
  __builtin_nontemporal_store(v, p);
}

NV_DEV void store16(uint16_t* p, const float x[16]) {
  nv_u4 a, b;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    a[i] = pack_bf16(x[2 * i], x[2 * i + 1]);
    b[i] = pack_bf16(x[8 + 2 * i], x[9 + 2 * i]);
  }
  nv_u4* q = reinterpret_cast<nv_u4*>(p);
  stream_out(q, a);
  stream_out(q + 1, b);
}

// ------------------------------------------------------------------ mx8

// Biased e8m0 byte of a group whose largest finite magnitude has the bits m:
// m = 1.f * 2^(E - 127) needs 2^(E - 135) while 1.f <= 1.75, else 2^(E - 134).
NV_DEV uint32_t mx8_scale_byte(uint32_t m) {
  const int e = (int)(m >> 23) - 8 + ((m & 0x7FFFFFu) > 0x600000u ? 1 : 0);
  return (uint32_t)(e > 10 ? e : 10);
}

// An e8m0 byte as the scale of a conversion instruction, which takes the
// exponent field alone: byte 0 stands for 2^-127 there, and 255 gives NaN.
NV_DEV float e8m0_scale(uint32_t byte) { return bits2f(byte << 23); }

// Value of an e8m0 byte, to multiply by: 2^-127 is subnormal, 255 is NaN.  (The
// encoder gives 10..247.)
NV_DEV float e8m0_value(uint32_t byte) {
  return bits2f(byte == 0 ? 0x00400000u : byte == 255 ? 0x7FC00000u : byte << 23);
}

// Magnitude bits of 16 values, the largest finite one; what is not finite
// counts as 0.
NV_DEV uint32_t finite_amax_bits(const float v[16]) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    const uint32_t b = f2bits(v[i]) & 0x7FFFFFFFu;
    m = b > m ? b : m;
  }
  if (m >= 0x7F800000u) {  // rare: leave out infinities and NaN
    m = 0;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const uint32_t b = f2bits(v[i]) & 0x7FFFFFFFu;
      m = (b < 0x7F800000u && b > m) ? b : m;
    }
  }
  return m;
}

// The value of the neighbouring lane (lane ^ 1).
NV_DEV uint32_t lane_xor1(uint32_t v) {
  return (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0xB1, 0xF, 0xF, true);
}

// One half of an mx8 group held by this lane, the other half by lane ^ 1
// (both lanes must be active; a missing half passes zeros).  Returns the
// scale byte; codes gets 16 e4m3 codes.
NV_DEV uint32_t mx8_encode16(const float v[16], nv_u4& codes) {
  uint32_t m = finite_amax_bits(v);
  const uint32_t o = lane_xor1(m);
  m = m > o ? m : o;
  const uint32_t byte = mx8_scale_byte(m);
  const float inv = bits2f((254u - byte) << 23);  // 2^-s, s = byte - 127 in -117..120
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    float q[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float x = v[4 * j + i] * inv;  // |x| <= 448 where finite: the conversion never saturates
      q[i] = (f2bits(x) & 0x7FFFFFFFu) >= 0x7F800000u ? bits2f(0x7FC00000u) : x;
    }
    int w = __builtin_amdgcn_cvt_pk_fp8_f32(q[0], q[1], (int)any_u32(), false);
    w = __builtin_amdgcn_cvt_pk_fp8_f32(q[2], q[3], w, true);
    codes[j] = (uint32_t)w;
  }
  return byte;
}

// Four e4m3 codes times a power of two (e8m0_scale) -> four bf16, exact where
// the result is a normal number; from 2^128 on infinite.
NV_DEV nv_u2 mx8_to_bf16(uint32_t w, float scale) {
  nv_u2 r;
  r.x = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, scale, false));
  r.y = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, scale, true));
  return r;
}

// 16 codes (one 16-byte load) times a power of two -> 16 fp32 values.
NV_DEV void mx8_values16(nv_u4 c, float scale, float v[16]) {
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const nv_f2 a = __builtin_amdgcn_cvt_pk_f32_fp8((int)c[j], false);
    const nv_f2 b = __builtin_amdgcn_cvt_pk_f32_fp8((int)c[j], true);
    v[4 * j] = a.x * scale;
    v[4 * j + 1] = a.y * scale;
    v[4 * j + 2] = b.x * scale;
    v[4 * j + 3] = b.y * scale;
  }
}

// -------------------------------------------------------- 4-bit weights

// Eight e2m1 codes times their block's e4m3 scale s -> eight bf16.  A code
// has 2 significant bits and a scale 4, so the product has at most 6 and
// bf16 holds it exactly: the matrix cores multiply the stored weight, not a
// rounding of it.  The second-level scale is applied to the sums.
NV_DEV nv_bf8 fp4_to_bf16(uint32_t w, float s) {
  const nv_f2 a = hw_fp4_values<0>(w), b = hw_fp4_values<1>(w), c = hw_fp4_values<2>(w), d = hw_fp4_values<3>(w);
  nv_u4 r;
  r[0] = pack_bf16(a.x * s, a.y * s);
  r[1] = pack_bf16(b.x * s, b.y * s);
  r[2] = pack_bf16(c.x * s, c.y * s);
  r[3] = pack_bf16(d.x * s, d.y * s);
  return __builtin_bit_cast(nv_bf8, r);
}

// The low (h = 0) or high four of eight codes alone.
NV_DEV nv_u2 fp4_half_to_bf16(uint32_t w, float s, int h) {
  const nv_f2 a = h ? hw_fp4_values<2>(w) : hw_fp4_values<0>(w), b = h ? hw_fp4_values<3>(w) : hw_fp4_values<1>(w);
  return (nv_u2){pack_bf16(a.x * s, a.y * s), pack_bf16(b.x * s, b.y * s)};
}

// Value of byte b (0..3) of a word of e4m3 scales.
NV_DEV float e4m3_byte(uint32_t w, int b) {
  return b == 0 ? __builtin_amdgcn_cvt_f32_fp8((int)w, 0) : b == 1 ? __builtin_amdgcn_cvt_f32_fp8((int)w, 1)
       : b == 2 ? __builtin_amdgcn_cvt_f32_fp8((int)w, 2) : __builtin_amdgcn_cvt_f32_fp8((int)w, 3);
}

// D += A B for a 16x32 and a 32x16 bf16 tile.  Lane l holds A[l % 16] and
// B[..][l % 16] at the eight k's of its lane group l / 16, and D[4 (l / 16) +
// r][l % 16], r = 0..3.  Which k's a lane group holds is free as long as A
// and B agree.
NV_DEV nv_f4 mfma16(nv_bf8 a, nv_bf8 b, nv_f4 c) { return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0); }

// The same for a 32x16 and a 16x32 tile: lane l holds A[l % 32] and B[..][l %
// 32] at the eight k's of its half l / 32, and D[8 (r / 4) + 4 (l / 32) + r %
// 4][l % 32], r = 0..15.  Twice the work an instruction: a loop that also
// decodes weights needs the issue slots.
NV_DEV nv_f16 mfma32(nv_bf8 a, nv_bf8 b, nv_f16 c) { return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0); }

// ------------------------------------------------------------ reductions

template <typename V>
NV_DEV V wave_sum(V v) {
#pragma unroll
  for (int off = 32; off >= 1; off >>= 1) v += __shfl_xor(v, off, 64);
  return v;
}

// Sum over the workgroup; every lane gets it.  `lds` holds one number a wave
// and is free again after the next barrier.
template <typename V>
NV_DEV V block_sum(V v, V* lds) {
  v = wave_sum(v);
  const int wave = threadIdx.x >> 6, nw = blockDim.x >> 6;
  if (nw == 1) return v;
  __syncthreads();
  if ((threadIdx.x & 63) == 0) lds[wave] = v;
  __syncthreads();
  V r = 0;
  for (int i = 0; i < nw; ++i) r += lds[i];
  return r;
}

// fp32 with the last bit set where 64-bit v lies between two fp32 numbers: a
// second rounding to 8 bits then takes the side of a border that v is on.  (No
// border is near where r is zero or subnormal.)
NV_DEV float round_odd(double v) {
  const float r = (float)v;
  const double d = v - (double)r;
  const uint32_t b = f2bits(r), back = (d < 0.0) != (r < 0.0f) ? 1u : 0u;
  const float a = __builtin_fabsf(r);
  return d != 0.0 && a >= 0x1p-126f && a < INFINITY ? bits2f((b - back) | 1u) : r;
}

// Distance in units of the last place, plus N and modulo 2^19, from an fp32 number
// with 19 trailing zeros: up to 2 N where one lies within N units.  Those are the
// numbers with four bits after the point, and the borders between e4m3 codes under
// any scale, and between scales, are among them.
template <int N>
NV_DEV uint32_t border_distance(float v) {
  return (f2bits(v) + (uint32_t)N) & 0x7FFFFu;
}

}  // namespace nvfp4
