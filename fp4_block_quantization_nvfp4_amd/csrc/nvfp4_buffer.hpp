// Range-checked loads of the layer operators.  tests/c/operand_loads.cpp compiles
// this header and nvfp4_weight.hpp for the CPU, with the loads' documented
// range check in the builtins' place.
#pragma once

namespace nvfp4 {

typedef unsigned int nv_u4 __attribute__((ext_vector_type(4)));
typedef unsigned int nv_u2 __attribute__((ext_vector_type(2)));

// A buffer of `bytes` bytes: loads outside it return zeros.  p and bytes are
// the same in all lanes; saying so keeps the compiler from a loop around each
// load where it cannot see it.
struct nv_buf {
  __amdgpu_buffer_rsrc_t at;
  uint32_t bytes;
};
NV_DEV nv_buf make_buf(const void* p, uint32_t bytes) {
  const uint64_t at = reinterpret_cast<uint64_t>(p);
  const uint32_t lo = (uint32_t)__builtin_amdgcn_readfirstlane((int)(uint32_t)at);
  const uint32_t hi = (uint32_t)__builtin_amdgcn_readfirstlane((int)(uint32_t)(at >> 32));
  const uint32_t n = (uint32_t)__builtin_amdgcn_readfirstlane((int)bytes);
  return {__builtin_amdgcn_make_buffer_rsrc(reinterpret_cast<void*>((uint64_t)hi << 32 | lo), 0, (int)n, 0x00027000), n};
}
constexpr uint32_t kOutside = 0x80000000u;  // an offset past every buffer (all are below 2^31 bytes)
// off is a lane's own offset, base one that all lanes share (kept in a scalar,
// so a walk along a row costs no vector instruction).  A word at off is outside
// where off >= bytes - base, the difference in 32 bits: a base past the end
// would make it a large number and let every lane through.  Such a base counts
// as the end, where all lanes are outside (one scalar instruction).
NV_DEV int buf_base(nv_buf b, uint32_t base) { return (int)(base < b.bytes ? base : b.bytes); }
NV_DEV nv_u4 buf16(nv_buf b, uint32_t off, uint32_t base = 0) { return __builtin_amdgcn_raw_buffer_load_b128(b.at, (int)off, buf_base(b, base), 0); }
NV_DEV nv_u2 buf8(nv_buf b, uint32_t off, uint32_t base = 0) { return __builtin_amdgcn_raw_buffer_load_b64(b.at, (int)off, buf_base(b, base), 0); }
NV_DEV uint32_t buf4(nv_buf b, uint32_t off, uint32_t base = 0) { return __builtin_amdgcn_raw_buffer_load_b32(b.at, (int)off, buf_base(b, base), 0); }
NV_DEV uint32_t buf1(nv_buf b, uint32_t off, uint32_t base = 0) { return __builtin_amdgcn_raw_buffer_load_b8(b.at, (int)off, buf_base(b, base), 0); }

}  // namespace nvfp4
