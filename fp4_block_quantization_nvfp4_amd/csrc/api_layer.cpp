// C ABI of the layer operators: host-side argument validation, then dispatch
// to the kernel launchers.  As in api.cpp, every error branch returns before
// anything is queued and nothing here touches device memory.
#include <stdint.h>

#include "../../include/nvfp4.h"
#include "nvfp4_launch.hpp"
#include "nvfp4_plan.hpp"

namespace {

constexpr int64_t kMaxElems = int64_t(1) << 33;

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }
bool dtype_ok(int d) { return d == NVFP4_F32 || d == NVFP4_BF16; }
bool fits(int64_t a, int64_t b) { return a == 0 || b <= kMaxElems / a; }

nvfp4_status check_rows(int64_t T, int64_t K) {
  if (T < 0 || K < 0 || K % 16 != 0) return NVFP4_E_SHAPE;
  if (T >= int64_t(1) << 31 || !fits(T, K)) return NVFP4_E_RANGE;
  return NVFP4_OK;
}

nvfp4_status check_products(int64_t T, int64_t E, int64_t N, int64_t K) {
  if (N < 0 || E < 1) return NVFP4_E_SHAPE;
  if (nvfp4_status st = check_rows(T, K)) return st;
  if (N > nvfp4::kMatmulMaxK || K > nvfp4::kMatmulMaxK || E > nvfp4::kMatmulMaxE) return NVFP4_E_RANGE;
  if (!fits(T, N) || !fits(E, N * K)) return NVFP4_E_RANGE;
  return NVFP4_OK;
}

nvfp4_status hip_status(int e) { return e == 0 ? NVFP4_OK : NVFP4_E_HIP; }

// What matvec and grouped_matmul share.
nvfp4_status check_weight(int64_t T, int64_t N, int64_t K, const void* x, const uint8_t* x_scales,
                          const uint8_t* packed, const uint8_t* scales, int blocks, const float* amax, int mode,
                          float bound, void* out, int out_dt) {
  if (blocks != NVFP4_BLOCK_1X16 && blocks != NVFP4_BLOCK_16X16 && blocks != NVFP4_BLOCK_16X16_T) return NVFP4_E_ARG;
  if (blocks != NVFP4_BLOCK_1X16 && N % 16 != 0) return NVFP4_E_SHAPE;
  if (!dtype_ok(out_dt)) return NVFP4_E_DTYPE;
  if (mode != NVFP4_SCALE_NONE && mode != NVFP4_SCALE_TENSOR && mode != NVFP4_SCALE_ROW) return NVFP4_E_ARG;
  if (blocks != NVFP4_BLOCK_1X16 && mode == NVFP4_SCALE_ROW) return NVFP4_E_ARG;
  if (mode != NVFP4_SCALE_NONE && !(bound == 256.0f || bound == 448.0f)) return NVFP4_E_ARG;
  if (T == 0 || N == 0) return NVFP4_OK;
  if (!out || (mode != NVFP4_SCALE_NONE && !amax)) return NVFP4_E_NULL;
  if (K != 0 && (!x || !packed || !scales)) return NVFP4_E_NULL;
  if (!aligned(x, 16) || !aligned(packed, 8) || !aligned(amax, 4) || !aligned(out, 16)) return NVFP4_E_ALIGN;
  (void)x_scales;
  return NVFP4_OK;
}

}  // namespace

extern "C" {

nvfp4_status nvfp4_add_rms_norm(const void* x, const void* residual, nvfp4_dtype dt, const float* weight,
                                int64_t T, int64_t H, float eps, uint8_t* codes, uint8_t* scales,
                                void* hidden, float* rstd, void* stream) {
  if (nvfp4_status st = check_rows(T, H)) return st;
  if (H > nvfp4::kNormMaxH) return NVFP4_E_RANGE;
  if (!dtype_ok(dt)) return NVFP4_E_DTYPE;
  if (!(eps >= 0.0f)) return NVFP4_E_ARG;
  if ((residual == nullptr) != (hidden == nullptr)) return NVFP4_E_NULL;
  if (T == 0 || H == 0) return NVFP4_OK;
  if (!x || !weight || !codes || !scales || !rstd) return NVFP4_E_NULL;
  if (!aligned(x, 16) || !aligned(residual, 16) || !aligned(hidden, 16) || !aligned(weight, 16) ||
      !aligned(codes, 16) || !aligned(rstd, 4))
    return NVFP4_E_ALIGN;
  return hip_status(nvfp4::launch_add_rms_norm(x, residual, dt == NVFP4_BF16, weight, T, H, eps, codes, scales,
                                               hidden, rstd, stream));
}

size_t nvfp4_add_rms_norm_backward_workspace_bytes(int64_t T, int64_t H) {
  if (T < 0 || H < 0 || H > nvfp4::kNormMaxH) return 0;
  return nvfp4::norm_bwd_workspace_bytes(T, H);
}

nvfp4_status nvfp4_add_rms_norm_backward(const void* dy, const void* hidden, const void* dhidden, nvfp4_dtype dt,
                                         const float* weight, const float* rstd, int64_t T, int64_t H, void* dx,
                                         float* dweight, void* workspace, size_t workspace_bytes, void* stream) {
  if (nvfp4_status st = check_rows(T, H)) return st;
  if (H > nvfp4::kNormMaxH) return NVFP4_E_RANGE;
  if (!dtype_ok(dt)) return NVFP4_E_DTYPE;
  if (H == 0) return NVFP4_OK;
  if (!dweight) return NVFP4_E_NULL;
  if (T != 0 && (!dy || !hidden || !weight || !rstd || !dx || !workspace)) return NVFP4_E_NULL;
  if (workspace_bytes < nvfp4::norm_bwd_workspace_bytes(T, H)) return NVFP4_E_ARG;
  if (!aligned(dy, 16) || !aligned(hidden, 16) || !aligned(dhidden, 16) || !aligned(weight, 16) ||
      !aligned(rstd, 4) || !aligned(dx, 16) || !aligned(dweight, 16) || !aligned(workspace, 16))
    return NVFP4_E_ALIGN;
  return hip_status(nvfp4::launch_add_rms_norm_bwd(dy, hidden, dhidden, dt == NVFP4_BF16, weight, rstd, T, H, dx,
                                                   dweight, workspace, stream));
}

nvfp4_status nvfp4_swiglu(const void* gate_up, nvfp4_dtype dt, int64_t T, int64_t F, uint8_t* codes,
                          uint8_t* scales, uint8_t* kept, uint8_t* kept_scales, void* stream) {
  if (nvfp4_status st = check_rows(T, F)) return st;
  if (!fits(T, 2 * F)) return NVFP4_E_RANGE;
  if (!dtype_ok(dt)) return NVFP4_E_DTYPE;
  if ((kept == nullptr) != (kept_scales == nullptr)) return NVFP4_E_NULL;
  if (T == 0 || F == 0) return NVFP4_OK;
  if (!gate_up || !codes || !scales) return NVFP4_E_NULL;
  if (!aligned(gate_up, 16) || !aligned(codes, 16) || !aligned(kept, 16)) return NVFP4_E_ALIGN;
  return hip_status(
      nvfp4::launch_swiglu(gate_up, dt == NVFP4_BF16, T, F, codes, scales, kept, kept_scales, stream));
}

nvfp4_status nvfp4_swiglu_backward(const void* dout, nvfp4_dtype dt, int64_t T, int64_t F, const uint8_t* kept,
                                   const uint8_t* kept_scales, void* dgate_up, void* stream) {
  if (nvfp4_status st = check_rows(T, F)) return st;
  if (!fits(T, 2 * F)) return NVFP4_E_RANGE;
  if (!dtype_ok(dt)) return NVFP4_E_DTYPE;
  if (T == 0 || F == 0) return NVFP4_OK;
  if (!dout || !kept || !kept_scales || !dgate_up) return NVFP4_E_NULL;
  if (!aligned(dout, 16) || !aligned(kept, 16) || !aligned(dgate_up, 16)) return NVFP4_E_ALIGN;
  return hip_status(
      nvfp4::launch_swiglu_bwd(dout, dt == NVFP4_BF16, T, F, kept, kept_scales, dgate_up, stream));
}

static nvfp4_status products(const void* x, const uint8_t* x_scales, int64_t T, int64_t E, int64_t N, int64_t K,
                             const int32_t* ends, const uint8_t* packed, const uint8_t* scales, int blocks,
                             const float* amax, int mode, float bound, void* out, int out_dt, void* stream) {
  const nvfp4::MatmulArgs a = {x, x_scales, packed, scales, amax, ends, out, (int)T, (int)E, (int)N, (int)K,
                               blocks, mode, 6.0f * bound, out_dt == NVFP4_BF16};
  if (K == 0) return hip_status(nvfp4::launch_zero(out, T * N * (out_dt == NVFP4_BF16 ? 2 : 4), stream));
  if (nvfp4::use_matvec(T, E, N)) return hip_status(nvfp4::launch_matvec(a, stream));
  return hip_status(x_scales ? nvfp4::launch_grouped_mx8(a, stream) : nvfp4::launch_grouped_bf16(a, stream));
}

nvfp4_status nvfp4_matvec(const void* x, const uint8_t* x_scales, int64_t T, int64_t N, int64_t K,
                          const uint8_t* packed, const uint8_t* scales, nvfp4_block blocks,
                          const float* global_amax, nvfp4_scale_mode scale_mode, float bound, void* out,
                          nvfp4_dtype out_dt, void* stream) {
  if (nvfp4_status st = check_products(T, 1, N, K)) return st;
  if (nvfp4_status st = check_weight(T, N, K, x, x_scales, packed, scales, blocks, global_amax, scale_mode, bound,
                                     out, out_dt))
    return st;
  if (T == 0 || N == 0) return NVFP4_OK;
  return products(x, x_scales, T, 1, N, K, nullptr, packed, scales, blocks, global_amax, scale_mode, bound, out,
                  out_dt, stream);
}

nvfp4_status nvfp4_grouped_matmul(const void* x, const uint8_t* x_scales, int64_t T, int64_t E, int64_t N,
                                  int64_t K, const int32_t* ends, const uint8_t* packed, const uint8_t* scales,
                                  nvfp4_block blocks, const float* global_amax, nvfp4_scale_mode scale_mode,
                                  float bound, void* out, nvfp4_dtype out_dt, void* stream) {
  if (nvfp4_status st = check_products(T, E, N, K)) return st;
  if (nvfp4_status st = check_weight(T, N, K, x, x_scales, packed, scales, blocks, global_amax, scale_mode, bound,
                                     out, out_dt))
    return st;
  if (T == 0 || N == 0) return NVFP4_OK;
  if (!ends) return NVFP4_E_NULL;
  if (!aligned(ends, 4)) return NVFP4_E_ALIGN;
  return products(x, x_scales, T, E, N, K, ends, packed, scales, blocks, global_amax, scale_mode, bound, out,
                  out_dt, stream);
}

static nvfp4_status wgrad(const void* dy, const void* x, const uint8_t* x_scales, int64_t T, int64_t E, int64_t N,
                          int64_t K, const int32_t* ends, void* dw, int out_dt, int64_t block, void* workspace,
                          size_t workspace_bytes, void* stream) {
  if (nvfp4_status st = check_products(T, E, N, K)) return st;
  if (N % 16 != 0) return NVFP4_E_SHAPE;
  if (!dtype_ok(out_dt)) return NVFP4_E_DTYPE;
  if (N == 0 || K == 0) return NVFP4_OK;
  if (!ends || !dw || (T != 0 && (!dy || !x))) return NVFP4_E_NULL;
  if (block && !workspace) return NVFP4_E_NULL;
  if (block && workspace_bytes < nvfp4_grouped_wgrad_workspace_bytes(T, E, N, K)) return NVFP4_E_ARG;
  if (!aligned(dy, 16) || !aligned(x, 16) || !aligned(ends, 4) || !aligned(dw, 16) || !aligned(workspace, 16)) return NVFP4_E_ALIGN;
  const nvfp4::WgradArgs a = {dy, x, x_scales, ends, dw, (int)T, (int)E, (int)N, (int)K, out_dt == NVFP4_BF16,
                              (int)block, (float*)workspace};
  return hip_status(nvfp4::launch_wgrad(a, stream));
}

nvfp4_status nvfp4_grouped_wgrad(const void* dy, const void* x, const uint8_t* x_scales, int64_t T, int64_t E,
                                 int64_t N, int64_t K, const int32_t* ends, void* dw, nvfp4_dtype out_dt,
                                 void* stream) {
  return wgrad(dy, x, x_scales, T, E, N, K, ends, dw, out_dt, 0, nullptr, 0, stream);
}

size_t nvfp4_grouped_wgrad_workspace_bytes(int64_t T, int64_t E, int64_t N, int64_t K) {
  if (check_products(T, E, N, K) != NVFP4_OK) return 0;
  const int64_t b = nvfp4::wgrad_block(T, E, N, K);
  return b ? (size_t)((T / b + E + 1) * N * K * 4) : 0;
}

nvfp4_status nvfp4_grouped_wgrad_split(const void* dy, const void* x, const uint8_t* x_scales, int64_t T, int64_t E,
                                       int64_t N, int64_t K, const int32_t* ends, void* dw, nvfp4_dtype out_dt,
                                       void* workspace, size_t workspace_bytes, void* stream) {
  const int64_t b = check_products(T, E, N, K) == NVFP4_OK ? nvfp4::wgrad_block(T, E, N, K) : 0;
  return wgrad(dy, x, x_scales, T, E, N, K, ends, dw, out_dt, b, workspace, workspace_bytes, stream);
}

nvfp4_status nvfp4_selftest_layer_plan(int entry, int64_t T, int64_t E, int64_t N, int64_t K, int mx8,
                                       int64_t* plan) {
  if (entry < 0 || entry > 6) return NVFP4_E_ARG;
  if (entry < 3) {
    if (nvfp4_status st = check_rows(T, K)) return st;
    if (entry == 2 ? !fits(T, 2 * K) : K > nvfp4::kNormMaxH) return NVFP4_E_RANGE;
  } else {
    if (entry == 3) E = 1;
    if (nvfp4_status st = check_products(T, E, N, K)) return st;
    if (entry > 4 && N % 16 != 0) return NVFP4_E_SHAPE;
  }
  if (!plan) return NVFP4_E_NULL;
  nvfp4::LayerLaunch p[2] = {};
  int64_t rows = 0;
  if (entry == 0) p[0] = nvfp4::plan_norm(T, K);
  if (entry == 1) p[0] = nvfp4::plan_norm_bwd(T, K), p[1] = nvfp4::plan_sum_rows(K);
  if (entry == 2) p[0] = nvfp4::plan_swiglu(T, K);
  if ((entry == 3 || entry == 4) && K == 0) {
    p[0] = nvfp4::plan_zero(T * N * 4);
  } else if (entry == 3 || entry == 4) {
    if (nvfp4::use_matvec(T, E, N)) {
      p[0] = nvfp4::plan_matvec(T, entry == 4 ? E : 0, N, mx8 != 0);
      rows = T > 16 * E ? 32 : 16;
    } else {
      const nvfp4::GroupedPlan g = nvfp4::plan_grouped(T, entry == 4 ? E : 0, N);
      p[0] = {nvfp4::PLAN_GROUPED, g.grid, 1, 256};
      rows = g.rows;
    }
  }
  if (entry >= 5) {
    rows = entry == 6 ? nvfp4::wgrad_block(T, E, N, K) : 0;
    p[0] = nvfp4::plan_wgrad(T, E, N, K, rows);
    if (rows) p[1] = nvfp4::plan_wgrad_join(E, N, K);
  }
  for (int i = 0; i < 2; ++i) {
    plan[5 * i] = p[i].kernel;
    plan[5 * i + 1] = p[i].grid;
    plan[5 * i + 2] = p[i].y;
    plan[5 * i + 3] = p[i].block;
    plan[5 * i + 4] = i ? 0 : rows;
  }
  return NVFP4_OK;
}

}  // extern "C"
