// Host-side launchers of the NVFP4 kernels.  Arguments are already validated
// by the C ABI layer (api.cpp); each launcher returns a hipError_t as int.
#pragma once

#include <stddef.h>
#include <stdint.h>

namespace nvfp4 {

// dtype codes match nvfp4_dtype: 0 fp32, 1 bf16.  out_kind: 0 none, 1 bf16, 2 fp32.
int launch_quant1x16(const void* x, int in_bf16, int64_t M, int64_t K, float* residual,
                     const float* global_amax, int sr, uint32_t seed, uint32_t step,
                     uint8_t* packed, uint8_t* scales, void* out, int out_kind, void* stream);

// scale_mode: 0 none, 1 tensor, 2 row.  out_bf16: 1 bf16, 0 fp32.
int launch_dequant(const uint8_t* packed, const uint8_t* scales, int64_t M, int64_t K,
                   int tile16, const float* global_amax, int scale_mode, float bound,
                   void* out, int out_bf16, void* stream);

// mode: 1 tensor, 2 row.  amax_is_input: row amax read (1) or computed in-pass (0).
int launch_4over6(const void* x, int in_bf16, int64_t M, int64_t K, float* amax, int mode,
                  int amax_is_input, int mse, float bound, uint8_t* packed, uint8_t* scales,
                  void* stream);

int launch_quant2d(const void* x, int in_bf16, int64_t M, int64_t K, const float* global_amax,
                   int sr, uint32_t seed, uint32_t step, int round_up, uint8_t* packed_row,
                   uint8_t* packed_col, uint8_t* tile_scales, void* stream);

int launch_rowcol(const void* x, int in_bf16, int64_t M, int64_t K, const float* global_amax,
                  int four_over_six, int mse, float bound, uint8_t* packed_row,
                  uint8_t* scales_row, uint8_t* packed_col, uint8_t* scales_col, void* stream);

int launch_4over6_2d(const void* x, int in_bf16, int64_t M, int64_t K, const float* global_amax,
                     int mse, float bound, uint8_t* packed_row, uint8_t* packed_col,
                     uint8_t* tile_scales, void* stream);

size_t amax_workspace_bytes(int64_t M, int64_t K);
// mode: 1 tensor (two passes through workspace), 2 row.
int launch_amax(const void* x, int in_bf16, int64_t M, int64_t K, const float* residual,
                int mode, float* amax_out, void* workspace, void* stream);

// Allocation-free per-tensor / per-row amax: partials in the library's own
// device scratch array (k_amax.hip).
int64_t amax_noalloc_max_partials();
int launch_amax_noalloc(const void* x, int in_bf16, int64_t M, int64_t K, const float* residual,
                        int mode, float* amax_out, void* stream);

// ---- layer operators

// rows x H; res, hidden NULL together; codes / scales mx8.
int launch_add_rms_norm(const void* x, const void* res, int in_bf16, const float* w, int64_t rows, int64_t H,
                        float eps, uint8_t* codes, uint8_t* scales, void* hidden, float* rstd, void* stream);
size_t norm_bwd_workspace_bytes(int64_t rows, int64_t H);
int launch_add_rms_norm_bwd(const void* dy, const void* hidden, const void* dh, int in_bf16, const float* w,
                            const float* rstd, int64_t rows, int64_t H, void* dx, float* dw, void* ws,
                            void* stream);

// rows x 2F -> rows x F; kept / kept_scales NULL together.
int launch_swiglu(const void* gate_up, int in_bf16, int64_t rows, int64_t F, uint8_t* codes, uint8_t* scales,
                  uint8_t* kept, uint8_t* kept_scales, void* stream);
int launch_swiglu_bwd(const void* dout, int in_bf16, int64_t rows, int64_t F, const uint8_t* kept,
                      const uint8_t* kept_scales, void* dgate_up, void* stream);

// Product of rows with 4-bit weights (k_matvec.hip, nvfp4_grouped.hpp).
struct MatmulArgs {
  const void* x;       // [T, K] bf16, or e4m3 codes when xs is set
  const uint8_t* xs;   // NULL, or [T, ceil(K / 32)] e8m0
  const uint8_t* w;    // [E, N, K / 2]
  const uint8_t* ws;   // block scales
  const float* amax;   // NULL, [E] or [E * N]
  const int* ends;     // NULL (one expert, all rows), or [E]
  void* out;           // [T, N]
  int T, E, N, K;
  int blocks;          // 0 1x16, 1 16x16 tiles, 2 tiles of the transposed weight
  int mode;            // second level: 0 none, 1 one per expert, 2 one per row
  float D;             // 6 * bound
  int out_bf16;
};
int launch_matvec(const MatmulArgs& a, void* stream);
int launch_zero(void* out, int64_t bytes, void* stream);  // products with K == 0
int launch_grouped_mx8(const MatmulArgs& a, void* stream);
int launch_grouped_bf16(const MatmulArgs& a, void* stream);

// dw[e] = dy^T x over the rows of each expert (k_wgrad.hip).
struct WgradArgs {
  const void* dy;      // [T, N] bf16
  const void* x;       // [T, K] bf16 or e4m3 codes
  const uint8_t* xs;
  const int* ends;
  void* dw;            // [E, N, K]
  int T, E, N, K;
  int out_bf16;
  int block;           // rows of a block (wgrad_block), 0: whole experts
  float* part;         // sums of blocks, at most T / block + E + 1 of [N][K]
};
int launch_wgrad(const WgradArgs& a, void* stream);

// Test support: exhaustive conversion scans (k_selftest.hip).
int launch_selftest_scan(int kind, uint32_t param, uint64_t first, uint64_t count, int chunk_log2,
                         uint32_t* records, void* stream);

}  // namespace nvfp4
