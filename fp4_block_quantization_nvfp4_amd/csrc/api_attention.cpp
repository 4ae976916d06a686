// C ABI of attention on an NVFP4 cache: host-side argument validation, then
// dispatch to the kernel launchers.  As in api.cpp, every error branch returns
// before anything is queued and nothing here touches device memory.
#include <limits.h>
#include <math.h>
#include <stdint.h>

#include <initializer_list>

#include "../../include/nvfp4.h"
#include "nvfp4_launch.hpp"
#include "nvfp4_plan.hpp"

namespace {

constexpr int64_t kMaxElems = int64_t(1) << 33;
constexpr int64_t kMaxHeads = 65536, kMaxStride = int64_t(1) << 40, kMaxB = int64_t(1) << 20;
constexpr int64_t kMaxKeys = int64_t(1) << 30;   // a tile more stays in 31 bits
constexpr int64_t kMaxUnits = int64_t(1) << 22;  // sequences times heads: the tiled kernel's grid

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }
bool dtype_ok(int d) { return d == NVFP4_F32 || d == NVFP4_BF16; }
bool fits(int64_t a, int64_t b) { return a == 0 || b <= kMaxElems / a; }
nvfp4_status hip_status(int e) { return e == 0 ? NVFP4_OK : NVFP4_E_HIP; }

nvfp4_status check_tokens(int64_t T, int64_t D, int64_t most) {
  if (T < 0 || D < 16 || D % 16 != 0) return NVFP4_E_SHAPE;
  if (T >= int64_t(1) << 31 || D > most) return NVFP4_E_RANGE;
  return NVFP4_OK;
}

// Sizes of rows; their pointer is checked by check_at.
nvfp4_status check_heads(const nvfp4_heads* h, int64_t T, int64_t D) {
  if (!h) return NVFP4_E_NULL;
  if (h->heads < 0) return NVFP4_E_SHAPE;
  if (h->heads > kMaxHeads || !fits(h->heads * D, T)) return NVFP4_E_RANGE;
  if (h->token < -kMaxStride || h->token > kMaxStride || h->head < -kMaxStride || h->head > kMaxStride) return NVFP4_E_RANGE;
  return NVFP4_OK;
}
nvfp4_status check_at(const nvfp4_heads* h, int64_t T, int dt) {
  if (T == 0 || h->heads == 0) return NVFP4_OK;
  if (!h->at) return NVFP4_E_NULL;
  const int64_t unit = dt == NVFP4_BF16 ? 8 : 4;
  if (!aligned(h->at, 16) || h->token % unit != 0 || h->head % unit != 0) return NVFP4_E_ALIGN;
  return NVFP4_OK;
}

nvfp4_status check_rope(const nvfp4_rope* r, int64_t T, int64_t D) {
  if (!r) return NVFP4_E_NULL;
  if (r->rotated < 0 || r->rotated > D || r->rotated % 16 != 0) return NVFP4_E_SHAPE;
  if (!(r->eps >= 0.0) || !isfinite(r->multiplier)) return NVFP4_E_ARG;
  if (T != 0 && r->rotated != 0 && (!r->positions || !r->freqs)) return NVFP4_E_NULL;
  if (!aligned(r->positions, 4) || !aligned(r->freqs, 8) || !aligned(r->q_weight, 16) || !aligned(r->k_weight, 16))
    return NVFP4_E_ALIGN;
  return NVFP4_OK;
}

nvfp4_status check_cache(const nvfp4_cache* c) {
  if (!c) return NVFP4_E_NULL;
  if (c->pages < 0 || c->heads < 1 || c->dim < 16 || c->dim % 16 != 0) return NVFP4_E_SHAPE;
  if (c->page_size < 16 || c->page_size > 65536 || (c->page_size & (c->page_size - 1)) != 0) return NVFP4_E_SHAPE;
  if (c->heads > kMaxHeads || c->dim > nvfp4::kRopeMaxD) return NVFP4_E_RANGE;
  if (c->pages > ((int64_t(1) << 31) - 1) / c->page_size) return NVFP4_E_RANGE;
  if (c->pages != 0 && (!c->k || !c->k_scales || !c->v || !c->v_scales)) return NVFP4_E_NULL;
  if (!aligned(c->k, 16) || !aligned(c->v, 16) || !aligned(c->k_scales, 2) || !aligned(c->v_scales, 2) ||
      !aligned(c->k_amax, 4) || !aligned(c->v_amax, 4))
    return NVFP4_E_ALIGN;
  return NVFP4_OK;
}

nvfp4::HeadsView view(const nvfp4_heads* h) { return {h->at, h->token, h->head, (int)h->heads}; }
nvfp4::CacheView view(const nvfp4_cache* c) {
  int shift = 0;
  while ((int64_t(1) << shift) < c->page_size) ++shift;
  return {c->k, c->k_scales, c->v, c->v_scales, c->k_amax, c->v_amax, (int)c->pages, (int)c->heads, (int)c->dim, shift};
}

nvfp4::RopeArgs rope_args(const nvfp4_heads* q, const nvfp4_heads* k, int dt, int64_t T, int64_t D, const nvfp4_rope* r) {
  nvfp4::RopeArgs a = {};
  a.q = view(q);
  a.k = view(k);
  a.T = (int)T;
  a.D = (int)D;
  a.in_bf16 = dt == NVFP4_BF16;
  if (r) {
    a.R = (int)r->rotated;
    a.interleaved = r->interleaved != 0;
    a.positions = r->positions;
    a.freqs = r->freqs;
    a.mult = r->multiplier;
    a.eps = r->eps;
    a.qw = r->q_weight;
    a.kw = r->k_weight;
  }
  return a;
}

// Keys and values of the cache's heads, and the slots.
nvfp4_status check_write(const nvfp4_heads* k, const nvfp4_heads* v, int dt, int64_t T, const nvfp4_cache* c,
                         const int32_t* slots) {
  if (nvfp4_status st = check_cache(c)) return st;
  if (nvfp4_status st = check_tokens(T, c->dim, nvfp4::kRopeMaxD)) return st;
  if (nvfp4_status st = check_heads(k, T, c->dim)) return st;
  if (nvfp4_status st = check_heads(v, T, c->dim)) return st;
  if (!dtype_ok(dt)) return NVFP4_E_DTYPE;
  if (k->heads != c->heads || v->heads != c->heads) return NVFP4_E_SHAPE;
  if (nvfp4_status st = check_at(k, T, dt)) return st;
  if (nvfp4_status st = check_at(v, T, dt)) return st;
  if (T != 0 && !slots) return NVFP4_E_NULL;
  if (!aligned(slots, 4)) return NVFP4_E_ALIGN;
  return NVFP4_OK;
}

// Sizes of cache_attention.
nvfp4_status check_attention(int64_t T, int64_t Hq, const nvfp4_cache* c, int64_t B, int64_t width) {
  if (nvfp4_status st = check_cache(c)) return st;
  if (c->dim % 32 != 0 || T < 0 || Hq < 0 || Hq % c->heads != 0 || B < 0 || width < 1) return NVFP4_E_SHAPE;
  if (c->dim > 256 || T >= int64_t(1) << 31 || Hq > kMaxHeads || !fits(Hq * c->dim, T) || B > kMaxB) return NVFP4_E_RANGE;
  if (width > kMaxKeys / c->page_size || B * c->heads > kMaxUnits) return NVFP4_E_RANGE;
  if (Hq == 0) return NVFP4_OK;
  if (nvfp4::attend_split_tiles(T, B, Hq, c->heads, width * c->page_size) >= int64_t(1) << 31) return NVFP4_E_RANGE;
  return NVFP4_OK;
}

}  // namespace

extern "C" {

nvfp4_status nvfp4_norm_rope(const nvfp4_heads* q, const nvfp4_heads* k, nvfp4_dtype dt, int64_t T, int64_t D,
                             const nvfp4_rope* rope, void* q_out, void* k_out, void* stream) {
  if (nvfp4_status st = check_tokens(T, D, nvfp4::kRopeMaxD)) return st;
  if (nvfp4_status st = check_heads(q, T, D)) return st;
  if (nvfp4_status st = check_heads(k, T, D)) return st;
  if (!dtype_ok(dt)) return NVFP4_E_DTYPE;
  if (nvfp4_status st = check_rope(rope, T, D)) return st;
  if (T == 0 || q->heads + k->heads == 0) return NVFP4_OK;
  if (nvfp4_status st = check_at(q, T, dt)) return st;
  if (nvfp4_status st = check_at(k, T, dt)) return st;
  if ((q->heads && !q_out) || (k->heads && !k_out)) return NVFP4_E_NULL;
  if (!aligned(q_out, 16) || !aligned(k_out, 16)) return NVFP4_E_ALIGN;
  nvfp4::RopeArgs a = rope_args(q, k, dt, T, D, rope);
  a.q_out = q_out;
  a.k_out = k_out;
  return hip_status(nvfp4::launch_norm_rope(a, stream));
}

size_t nvfp4_norm_rope_backward_workspace_bytes(int64_t T, int64_t D) {
  if (check_tokens(T, D, nvfp4::kRopeMaxD) != NVFP4_OK) return 0;
  return nvfp4::rope_bwd_workspace_bytes(T, D);
}

nvfp4_status nvfp4_norm_rope_backward(const nvfp4_heads* dq_out, const nvfp4_heads* dk_out, const nvfp4_heads* q,
                                      const nvfp4_heads* k, nvfp4_dtype dt, int64_t T, int64_t D,
                                      const nvfp4_rope* rope, void* dq, void* dk, float* dweights, void* workspace,
                                      size_t workspace_bytes, void* stream) {
  if (nvfp4_status st = check_tokens(T, D, nvfp4::kRopeMaxD)) return st;
  for (const nvfp4_heads* h : {dq_out, dk_out, q, k})
    if (nvfp4_status st = check_heads(h, T, D)) return st;
  if (q->heads != dq_out->heads || k->heads != dk_out->heads) return NVFP4_E_SHAPE;
  if (!dtype_ok(dt)) return NVFP4_E_DTYPE;
  if (nvfp4_status st = check_rope(rope, T, D)) return st;
  const bool weights = rope->q_weight || rope->k_weight;
  for (const nvfp4_heads* h : {dq_out, dk_out})
    if (nvfp4_status st = check_at(h, T, dt)) return st;
  if (rope->q_weight)
    if (nvfp4_status st = check_at(q, T, dt)) return st;
  if (rope->k_weight)
    if (nvfp4_status st = check_at(k, T, dt)) return st;
  if (T != 0 && ((q->heads && !dq) || (k->heads && !dk))) return NVFP4_E_NULL;
  if (weights && !dweights) return NVFP4_E_NULL;
  if (weights && T != 0 && !workspace) return NVFP4_E_NULL;
  if (weights && workspace_bytes < nvfp4::rope_bwd_workspace_bytes(T, D)) return NVFP4_E_ARG;
  if (!aligned(dq, 16) || !aligned(dk, 16) || !aligned(dweights, 16) || !aligned(workspace, 16)) return NVFP4_E_ALIGN;
  if (!weights && (T == 0 || q->heads + k->heads == 0)) return NVFP4_OK;
  nvfp4::RopeArgs a = rope_args(q, k, dt, T, D, rope);
  a.q_out = dq;
  a.k_out = dk;
  return hip_status(nvfp4::launch_norm_rope_bwd(a, view(dq_out), view(dk_out), weights ? dweights : nullptr, workspace, stream));
}

nvfp4_status nvfp4_norm_rope_write(const nvfp4_heads* q, const nvfp4_heads* k, const nvfp4_heads* v, nvfp4_dtype dt,
                                   int64_t T, const nvfp4_rope* rope, const nvfp4_cache* cache, const int32_t* slots,
                                   void* q_out, void* stream) {
  if (nvfp4_status st = check_write(k, v, dt, T, cache, slots)) return st;
  if (nvfp4_status st = check_heads(q, T, cache->dim)) return st;
  if (nvfp4_status st = check_rope(rope, T, cache->dim)) return st;
  if (T == 0) return NVFP4_OK;
  if (nvfp4_status st = check_at(q, T, dt)) return st;
  if (q->heads && !q_out) return NVFP4_E_NULL;
  if (!aligned(q_out, 16)) return NVFP4_E_ALIGN;
  nvfp4::RopeArgs a = rope_args(q, k, dt, T, cache->dim, rope);
  a.v = view(v);
  a.q_out = q_out;
  a.c = view(cache);
  a.slots = slots;
  return hip_status(nvfp4::launch_norm_rope(a, stream));
}

nvfp4_status nvfp4_write_cache(const nvfp4_heads* k, const nvfp4_heads* v, nvfp4_dtype dt, int64_t T,
                               const nvfp4_cache* cache, const int32_t* slots, void* stream) {
  if (nvfp4_status st = check_write(k, v, dt, T, cache, slots)) return st;
  if (T == 0) return NVFP4_OK;
  const nvfp4_heads none = {nullptr, 0, 0, 0};
  nvfp4::RopeArgs a = rope_args(&none, k, dt, T, cache->dim, nullptr);
  a.v = view(v);
  a.c = view(cache);
  a.slots = slots;
  return hip_status(nvfp4::launch_norm_rope(a, stream));
}

nvfp4_status nvfp4_read_cache(const nvfp4_cache* cache, const int32_t* slots, int64_t T, void* k, void* v,
                              nvfp4_dtype out_dt, void* stream) {
  if (nvfp4_status st = check_cache(cache)) return st;
  if (nvfp4_status st = check_tokens(T, cache->dim, nvfp4::kRopeMaxD)) return st;
  if (!fits(cache->heads * cache->dim, T)) return NVFP4_E_RANGE;
  if (!dtype_ok(out_dt)) return NVFP4_E_DTYPE;
  if (T == 0) return NVFP4_OK;
  if (!slots || !k || !v) return NVFP4_E_NULL;
  if (!aligned(slots, 4) || !aligned(k, 16) || !aligned(v, 16)) return NVFP4_E_ALIGN;
  return hip_status(nvfp4::launch_read_cache(view(cache), slots, T, k, v, out_dt == NVFP4_BF16, stream));
}

size_t nvfp4_cache_attention_workspace_bytes(int64_t T, int64_t q_heads, const nvfp4_cache* cache, int64_t B,
                                             int64_t width) {
  if (check_attention(T, q_heads, cache, B, width) != NVFP4_OK || T == 0 || q_heads == 0) return 0;
  return nvfp4::attend_workspace_bytes(T, B, q_heads, cache->heads, cache->dim, width * cache->page_size, true);
}

nvfp4_status nvfp4_cache_attention(const nvfp4_heads* q, int64_t T, const nvfp4_cache* cache, const int32_t* table,
                                   int64_t B, int64_t width, const int32_t* lens, const int32_t* ends, float scale,
                                   int causal, void* out, float* lse, void* workspace, size_t workspace_bytes,
                                   void* stream) {
  if (!q) return NVFP4_E_NULL;
  if (nvfp4_status st = check_attention(T, q->heads, cache, B, width)) return st;
  if (nvfp4_status st = check_heads(q, T, cache->dim)) return st;
  if (!ends && T != B && B != 0) return NVFP4_E_SHAPE;
  if (!(scale > 0.0f) || !isfinite(scale)) return NVFP4_E_ARG;
  if (T == 0 || q->heads == 0) return NVFP4_OK;
  if (nvfp4_status st = check_at(q, T, NVFP4_BF16)) return st;
  if (!out || !lse || (B != 0 && (!table || !lens))) return NVFP4_E_NULL;
  const size_t need = nvfp4::attend_workspace_bytes(T, B, q->heads, cache->heads, cache->dim, width * cache->page_size, ends != nullptr);
  if (need && !workspace) return NVFP4_E_NULL;
  if (workspace_bytes < need) return NVFP4_E_ARG;
  if (!aligned(table, 4) || !aligned(lens, 4) || !aligned(ends, 4) || !aligned(out, 16) || !aligned(lse, 4) ||
      !aligned(workspace, 16))
    return NVFP4_E_ALIGN;
  const int which = nvfp4::attend_kernels(T, q->heads, cache->heads, ends != nullptr);
  const nvfp4::AttendArgs a = {view(q), view(cache), table, lens, ends, (uint16_t*)out, lse, nullptr, nullptr, scale,
                               (int)T, (int)B, (int)width, causal != 0, which == 3 ? nvfp4::kAttendFew : INT_MAX};
  return hip_status(nvfp4::launch_attend(a, which, workspace, stream));
}

nvfp4_status nvfp4_selftest_attention_plan(int entry, int64_t T, int64_t Hq, int64_t Hk, int64_t D, int64_t B,
                                           int64_t keys, int64_t* plan) {
  const bool bf16 = entry < 16;  // 16 and up: of 32-bit rows
  if (entry < 0 || (bf16 ? entry > 6 : entry > 19)) return NVFP4_E_ARG;
  entry &= 15;
  if (!plan) return NVFP4_E_NULL;
  if (nvfp4_status st = check_tokens(T, D, entry < 5 ? nvfp4::kRopeMaxD : 256)) return st;
  if (Hq < 0 || Hk < 1 || B < 0 || keys < 16 || (entry >= 5 && (Hq % Hk != 0 || Hq == 0 || D % 32 != 0))) return NVFP4_E_SHAPE;
  if (Hq > kMaxHeads || Hk > kMaxHeads || !fits(Hq * D, T) || !fits(Hk * D, T) || B > kMaxB || keys > kMaxKeys || B * Hk > kMaxUnits) return NVFP4_E_RANGE;
  nvfp4::LayerLaunch p[4] = {};
  if (T != 0) {
    if (entry == 0) p[0] = nvfp4::plan_rope(T, Hq + Hk, D, bf16, false);
    if (entry == 1) p[0] = nvfp4::plan_rope_bwd(T, bf16), p[1] = nvfp4::plan_rope_sum(D);
    if (entry == 2) p[0] = nvfp4::plan_rope(T, Hq + 2 * Hk, D, bf16, true);
    if (entry == 3) p[0] = nvfp4::plan_rope(T, 2 * Hk, D, bf16, true);
    if (entry == 4) p[0] = nvfp4::plan_read_cache(T, Hk, D);
    if (entry >= 5) {
      if (nvfp4::attend_split_tiles(T, B, Hq, Hk, keys) >= int64_t(1) << 31) return NVFP4_E_RANGE;
      p[0] = nvfp4::plan_attend_split(T, B, Hq, Hk, D, keys);
      const int which = nvfp4::attend_kernels(T, Hq, Hk, entry == 5);
      if (which & 2) p[1] = nvfp4::plan_attend_tiles(T, B, Hq, Hk, D, keys);
      p[2] = nvfp4::plan_attend_join(T, B, Hq, Hk, D, keys, which);
    }
  }
  for (int i = 0; i < 4; ++i) {
    plan[4 * i] = p[i].kernel;
    plan[4 * i + 1] = p[i].grid;
    plan[4 * i + 2] = p[i].y;
    plan[4 * i + 3] = p[i].block;
  }
  return NVFP4_OK;
}

}  // extern "C"
