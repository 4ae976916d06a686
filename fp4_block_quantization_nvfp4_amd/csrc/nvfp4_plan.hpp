// Launch geometry of every kernel, computed on the host from the shape only.
// The launchers take their grids from these functions, and the test-support
// entry points nvfp4_selftest_launch_plan and nvfp4_selftest_layer_plan return
// the same numbers, so a CPU test can check that every launch stays inside the
// dispatch limits (grid x workgroup size below 2^32 work-items along each axis)
// for every accepted shape.
#pragma once

#include <stdint.h>

namespace nvfp4 {

// Workgroup shapes (lanes; strips of 16 rows per workgroup for the 16x16 and
// row + column kernels).
constexpr int kThreads = 256;           // k_quant1x16, k_dequant: 4 lanes per 16-element block
constexpr int kRowThreads = 128;        // k_4over6_rows: one two-wave workgroup per row
constexpr int kRowMaxBlocks = kRowThreads * 8;  // longest row (in 16-element blocks) it takes
constexpr int64_t kRowChunk = int64_t(1) << 24;  // rows per k_4over6_rows launch
constexpr int k46MaxThreads = 1024;     // k_4over6 (generic): one workgroup per row
constexpr int64_t k46MaxGrid = int64_t(1) << 20;
constexpr int k2dThreads = 512;         // k_quant2d: columns covered by a workgroup
constexpr int kStrips = 16;
constexpr int kRowColThreads = 256, kRowColFosThreads = 128, kRowColStrips = 16, kRowColFosStrips = 16;
constexpr int k46TileThreads = 512, k46TileStrips = 16;
constexpr int kAmaxThreads = 256;
constexpr int kAmaxMaxGroups = 2048;
constexpr int64_t kAmaxRowGrid = 65536;

enum PlanKernel {
  PLAN_QUANT1X16 = 0,
  PLAN_DEQUANT = 1,
  PLAN_4OVER6_ROWS = 2,
  PLAN_4OVER6_GENERIC = 3,
  PLAN_QUANT2D = 4,
  PLAN_ROWCOL = 5,
  PLAN_4OVER6_2D = 6,
  PLAN_AMAX_PARTIAL = 7,
  PLAN_AMAX_ROWS = 8,
};

struct LaunchPlan {
  int kernel;        // PlanKernel
  int64_t launches;  // launches of that kernel (row chunks)
  int64_t grid;      // workgroups of the largest launch
  int block;         // lanes per workgroup
};

inline int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// XCD-aware padded grid of the row + column and 16x16 kernels (a multiple
// of the 8 XCDs; padding workgroups exit at once).
inline int64_t xcd_grid(int64_t n) { return 8 * ceil_div(n, 8); }

inline LaunchPlan plan_quant1x16(int64_t M, int64_t K) {
  return {PLAN_QUANT1X16, 1, ceil_div(M * K / 4, kThreads), kThreads};
}

inline LaunchPlan plan_dequant(int64_t M, int64_t K) {
  return {PLAN_DEQUANT, 1, ceil_div(M * K / 4, kThreads), kThreads};
}

// bf16 rows of up to kRowMaxBlocks blocks take the row kernel, one workgroup
// per row and at most kRowChunk rows per launch; everything else the generic
// grid-stride kernel.
inline bool use_rows_kernel(int in_bf16, int64_t K) { return in_bf16 && K / 16 <= kRowMaxBlocks; }

inline LaunchPlan plan_4over6(int in_bf16, int64_t M, int64_t K) {
  if (use_rows_kernel(in_bf16, K))
    return {PLAN_4OVER6_ROWS, ceil_div(M, kRowChunk), M < kRowChunk ? M : kRowChunk, kRowThreads};
  int threads = (int)ceil_div(K / 16, 64) * 64;
  if (threads > k46MaxThreads) threads = k46MaxThreads;
  if (threads < 64) threads = 64;
  return {PLAN_4OVER6_GENERIC, 1, M < k46MaxGrid ? M : k46MaxGrid, threads};
}

inline int64_t quant2d_colgroups(int64_t K) { return ceil_div(K, k2dThreads); }
inline LaunchPlan plan_quant2d(int64_t M, int64_t K) {
  return {PLAN_QUANT2D, 1, quant2d_colgroups(K) * ceil_div(M / 16, kStrips), k2dThreads};
}

inline int rowcol_threads(int four_over_six) { return four_over_six ? kRowColFosThreads : kRowColThreads; }
inline int rowcol_strips(int four_over_six) { return four_over_six ? kRowColFosStrips : kRowColStrips; }
inline LaunchPlan plan_rowcol(int64_t M, int64_t K, int four_over_six) {
  const int nt = rowcol_threads(four_over_six);
  return {PLAN_ROWCOL, 1, xcd_grid(ceil_div(K, nt) * ceil_div(M / 16, rowcol_strips(four_over_six))), nt};
}

// Strips per workgroup of the 16x16 four-over-six kernel.  With columnwise
// output every workgroup takes k46TileStrips (each column's codes leave as
// one 128-byte segment).  Rowwise only, a shorter walk is taken when the
// grid would otherwise not give two workgroups per slot of the chip: the
// largest of 16, 8 and 4 strips with at least 1024 workgroups, else 4.
inline int tile_strips_4over6_2d(int64_t M, int64_t K, int columnwise) {
  if (columnwise) return k46TileStrips;
  const int64_t ncolg = ceil_div(K, k46TileThreads), nstrips = M / 16;
  for (int str = k46TileStrips; str > 4; str /= 2)
    if (ncolg * ceil_div(nstrips, str) >= 1024) return str;
  return 4;
}

inline LaunchPlan plan_4over6_2d(int64_t M, int64_t K, int columnwise) {
  const int str = tile_strips_4over6_2d(M, K, columnwise);
  return {PLAN_4OVER6_2D, 1, xcd_grid(ceil_div(K, k46TileThreads) * ceil_div(M / 16, str)), k46TileThreads};
}

inline int64_t amax_partial_groups(int64_t M, int64_t K) {
  int64_t g = ceil_div(M * K / 16, kAmaxThreads * 8);
  if (g < 1) g = 1;
  if (g > kAmaxMaxGroups) g = kAmaxMaxGroups;
  return g;
}
inline LaunchPlan plan_amax(int64_t M, int64_t K, int per_row) {
  if (per_row) return {PLAN_AMAX_ROWS, 1, M < kAmaxRowGrid ? M : kAmaxRowGrid, kAmaxThreads};
  return {PLAN_AMAX_PARTIAL, 1, amax_partial_groups(M, K), kAmaxThreads};
}

// ---- layer operators

enum LayerKernel {
  PLAN_NORM = 0,
  PLAN_NORM_BWD = 1,
  PLAN_SUM_ROWS = 2,
  PLAN_SWIGLU = 3,  // both directions
  PLAN_MATVEC = 4,
  PLAN_GROUPED = 5,
  PLAN_WGRAD = 6,
  PLAN_WGRAD_JOIN = 7,
  PLAN_ZERO = 8,
};

struct LayerLaunch {
  int kernel;       // LayerKernel
  int64_t grid, y;  // workgroups along x and y
  int block;        // lanes per workgroup
};

// Norm: one workgroup a row, 16 elements a lane (32 for rows over 16384), at
// most kNormMaxGrid workgroups (further rows in a loop).
constexpr int64_t kNormMaxH = 32768;
constexpr int64_t kNormMaxGrid = int64_t(1) << 20;
inline int norm_threads(int64_t H) {
  const int64_t per = H <= 16 * 1024 ? 16 : 32;
  return (int)ceil_div(ceil_div(H, per), 64) * 64;
}
inline LayerLaunch plan_norm(int64_t rows, int64_t H) {
  return {PLAN_NORM, rows < kNormMaxGrid ? rows : kNormMaxGrid, 1, norm_threads(H)};
}
// Norm's gradient: workgroups, each with one partial row of dw.  About sixteen
// waves on each of 256 CUs, and two rows a workgroup where there are few: a
// partial row costs as much to write and read as a row.  Of rows over 16384, whose
// dw takes 128 KB of shared memory, one workgroup of 9 to 16 waves runs on a CU at a
// time and the second of the two follows it.
inline int64_t norm_bwd_groups(int64_t rows, int64_t H) {
  const int64_t waves = norm_threads(H) / 64, cu = waves < 1 ? 8 : 16 / waves < 2 ? 2 : 16 / waves > 8 ? 8 : 16 / waves;
  int64_t g = rows / 2 < 256 ? 256 : rows / 2;
  if (g > 256 * cu) g = 256 * cu;
  return rows < g ? rows : g;
}
inline LayerLaunch plan_norm_bwd(int64_t rows, int64_t H) {
  return {PLAN_NORM_BWD, norm_bwd_groups(rows, H), 1, norm_threads(H)};
}
inline LayerLaunch plan_sum_rows(int64_t H) { return {PLAN_SUM_ROWS, H / 16, 1, 256}; }

// Gated activation, both directions: 16 elements a lane, rows padded to whole
// mx8 groups of 32.
inline int64_t swiglu_lanes(int64_t F) { return ceil_div(F, 32) * 2; }
inline LayerLaunch plan_swiglu(int64_t rows, int64_t F) {
  return {PLAN_SWIGLU, ceil_div(rows * swiglu_lanes(F), 256), 1, 256};
}

// Matrix products.
constexpr int kMatvecThreads = 256;
constexpr int64_t kMatmulMaxK = int64_t(1) << 20;  // a tile's rows stay below 2^31 bytes
constexpr int64_t kMatmulMaxE = 65534;             // grid y of k_matvec
// Fragments of 16 n's per workgroup of k_matvec: more of them read x less often,
// fewer spread a small weight over more CUs.  Four of them beside 16 rows of
// bf16 in flight do not fit the registers (65536 x 7168, 16 rows: 83 us, where
// two took 63, 54 now), so they take 8-bit rows or up to four rows an expert, and not where 32
// rows are taken at a time.
inline int matvec_frags(int64_t T, int64_t N, int64_t E, bool mx8) {
  const int64_t tiles = ceil_div(N, 16) * E;
  return tiles >= 4096 && (mx8 ? T <= 16 * E : T <= 4 * E) ? 4 : tiles >= 1024 ? 2 : 1;
}
// E = 0: one expert has all rows.  With experts, the E + 1 workgroups along grid y
// take all ranges' tiles in turn (the rows of none are a range too).
inline LayerLaunch plan_matvec(int64_t T, int64_t E, int64_t N, bool mx8) {
  return {PLAN_MATVEC, ceil_div(N, 16 * matvec_frags(T, N, E > 0 ? E : 1, mx8)), E > 0 ? E + 1 : 1, kMatvecThreads};
}
// Which kernel.  k_matvec decodes the weights anew for every 32 rows (16 up to 16
// an expert) but spreads them over many more workgroups; k_grouped decodes them
// once for up to 128 rows.  Up to 16 rows an expert the weights bound, and it is
// k_matvec; past that while its work, tiles of 32 rows times fragments of 16 n's,
// stays near what the chip runs at a time (512 workgroups of two fragments).  How
// many tiles T rows make goes by the experts' rows: T / 32 + E / 2 is taken, what
// rows that differ from expert to expert come to.  Measured, us, k_matvec
// (k_grouped), such rows: 8 experts 2048 x 2048, 160 rows 13.1 (15.3), 256 rows 16.3
// (15.3); 16 of 1024 x 2048, 320 rows 13.0 (15.2); 6 of 1024 x 1024, 192 rows 8.5
// (9.6), 384 rows 11.2 (11.4); 4 of 1040 x 4096, 256 rows 20 (30); 32 of 512 x 512,
// 1024 rows 10.9 (7.1).  Even rows come to fewer tiles: 8 of 2048 x 2048, 256 rows
// 10.0 (15.3).  One expert: 4096 x 4096, 96 rows 17 (31); 16384 x 4096, 32 rows 16
// (34).  Of up to 16 rows an expert small weights are the exception: 128 of 512 x
// 512, 1024 rows 15.4 (9.4); 32 of 4096 x 2048, 256 rows 41 (43).
inline bool use_matvec(int64_t T, int64_t E, int64_t N) {
  if (T <= 16 * E) return true;
  return T <= 96 * E && (E > 1 ? (T + 16 * E) * ceil_div(N, 16) <= 32 * 1152 : N * T <= 600000);
}
// Products without a k (K == 0), which may have more rows than tiles fit a
// launch: zeros, 16 bytes a lane and turn.
inline LayerLaunch plan_zero(int64_t bytes) {
  const int64_t g = ceil_div(bytes, 16 * 256);
  return {PLAN_ZERO, g < 8192 ? g : 8192, 1, 256};
}
// Workgroups of k_grouped that run at a time: two on each of 256 CUs.
constexpr int kGroupedSlots = 512;
// Tile of k_grouped, rows by n's: rows by what an expert has, and half the n's
// where wide tiles would leave CUs without one (each decodes half as many
// weights then; 8 experts 2048 x 2048, 64 rows each: 27.4 -> 19.4 us).  The
// grid is an upper bound: each of E experts and the rows of none (E = 0: all
// rows in one range) adds less than one tile to T / rows, and units of 128 rows
// that are split in four (up to an eighth of the slots) or two (up to a
// quarter) add at most three eighths of the slots.
struct GroupedPlan {
  int rows, width;
  int64_t grid;
};
inline GroupedPlan plan_grouped(int64_t T, int64_t E, int64_t N) {
  const int64_t per = T / (E > 0 ? E : 1);
  const int rows = per >= 128 ? 128 : per >= 64 ? 64 : 32;
  const int width = (ceil_div(T, rows) + E / 2) * ceil_div(N, 256) <= kGroupedSlots / 2 ? 128 : 256;
  const int64_t m = ceil_div(T, rows) + E;
  return {rows, width, xcd_grid((m < T ? m : T) * ceil_div(N, width)) + (rows == 128 ? kGroupedSlots * 3 / 8 : 0)};
}

// Weight gradient: tiles of kWgN n's by kWgK k's.
constexpr int kWgN = 256, kWgK = 128;
// Tiles of half the n's: up to 128 rows an expert, where writing the gradient
// bounds, and while the chip is not full.
inline bool wgrad_narrow(int64_t T, int64_t E, int64_t tiles) { return T <= 128 * E || tiles * E <= kGroupedSlots / 2; }
// Rows of a block where long experts are split, 0 where they are not.  A
// workgroup takes about 1.1 us for 64 rows while the chip is not full, a block's
// sums some 0.05 us a tile to write and read; block rows b cost 1.1 b / 64 +
// 0.05 tiles T / b us in all, least at b = sqrt(2.9 tiles T).  Split where
// that and one launch more (8 us) take less than 4/5 of the longest expert
// (taken as twice the mean), while the sums stay below 256 MB.  One expert 1024 x 512,
// 16384 rows: 299 us whole, 47 split.
inline int64_t wgrad_block(int64_t T, int64_t E, int64_t N, int64_t K) {
  const int64_t tiles = ceil_div(N, kWgN) * ceil_div(K, kWgK);
  if (T < 1024 || tiles == 0 || tiles * E >= kGroupedSlots) return 0;
  int64_t b = 256;
  while (b * b < 3 * tiles * T) b += 64;
  while ((T / b + E) * N * K * 4 > (int64_t(1) << 28)) b *= 2;
  const double whole = 1.1 * (double)(E > 1 ? 2 * T / E : T) / 64, split = 1.1 * (double)b / 64 + 0.05 * (double)(tiles * T) / (double)b + 8;
  return split < 0.8 * whole && b < T ? b : 0;
}

inline LayerLaunch plan_wgrad(int64_t T, int64_t E, int64_t N, int64_t K, int64_t block) {
  const int64_t tiles = ceil_div(N, kWgN) * ceil_div(K, kWgK);
  if (block) return {PLAN_WGRAD, xcd_grid((T / block + E + 1) * tiles), 1, 256};
  const int64_t wn = wgrad_narrow(T, E, tiles) ? kWgN / 2 : kWgN;
  return {PLAN_WGRAD, E * xcd_grid(ceil_div(N, wn) * ceil_div(K, kWgK)), 1, 256};
}
inline LayerLaunch plan_wgrad_join(int64_t E, int64_t N, int64_t K) {
  const int64_t g = ceil_div(N * K, 1024);
  return {PLAN_WGRAD_JOIN, g < 4096 ? g : 4096, E, 256};
}

// ---- attention on an NVFP4 cache

enum AttentionKernel {
  PLAN_ROPE = 0,
  PLAN_ROPE_BWD = 1,
  PLAN_ROPE_SUM = 2,
  PLAN_READ_CACHE = 3,
  PLAN_ATTEND_SPLIT = 4,
  PLAN_ATTEND_TILES = 5,
  PLAN_ATTEND_JOIN = 6,
};

// Norm and rotation: LN lanes to a row, sixteen elements each, 64 / LN rows a
// wave and pass; `rows` rows of each token.  A wave has one token; few tokens
// share theirs among several waves.
constexpr int64_t kRopeMaxD = 512;
inline int rope_lanes(int64_t D) {
  int n = 4;
  while (16 * n < D) n *= 2;
  return n;
}
inline int64_t rope_passes(int64_t rows, int64_t D) { return ceil_div(rows, 64 / rope_lanes(D)); }
inline int64_t rope_chunks(int64_t T, int64_t rows, int64_t D) {
  const int64_t p = rope_passes(rows, D), c = T > 0 ? ceil_div(4096, T) : 1;
  return c < 1 ? 1 : c < p ? c : p;
}
// Workgroups: what runs at a time by registers, three waves on a SIMD, of 32-bit rows to the cache
// two; rows of 16 bits to the outputs, four and little work each, all at once.  Measured, us, all at
// once (so): 16384 tokens of 8 heads to the cache 24.4 (22.1), 8192 of 40 heads with norm and rotation
// 49.0 (47.0), of 20 in fp32 39.9 (37.8), fp32 to the outputs 20.8 (19.5); bf16 34.5 (1024 groups 35.2).
inline int64_t rope_groups(bool bf16, bool cache) { return cache ? (bf16 ? 768 : 512) : bf16 ? kNormMaxGrid : 768; }
inline LayerLaunch plan_rope(int64_t T, int64_t rows, int64_t D, bool bf16, bool cache) {
  const int64_t g = ceil_div(T * rope_chunks(T, rows, D), 4), most = rope_groups(bf16, cache);
  return {PLAN_ROPE, g < most ? g : most, 1, 256};  // further tokens in a loop
}
// The gradient's workgroups: what runs at a time, three waves on a SIMD of 16-bit rows, two of
// 32-bit ones, so that none waits for a place (8192 tokens, 40 heads of 128 in bf16: 1024 groups
// 59.5 us, 768 50.8; 20 heads of 64 in fp32: 1024 40, 768 40.4, 512 34.5).
constexpr int64_t kRopeBwdGroups = 768;
inline int64_t rope_bwd_groups(int64_t T, bool bf16) {
  const int64_t g = ceil_div(T, 4), most = bf16 ? kRopeBwdGroups : kRopeBwdGroups * 2 / 3;
  return g < most ? g : most;
}
inline LayerLaunch plan_rope_bwd(int64_t T, bool bf16) { return {PLAN_ROPE_BWD, rope_bwd_groups(T, bf16), 1, 256}; }
inline LayerLaunch plan_rope_sum(int64_t D) { return {PLAN_ROPE_SUM, 2 * D / 16, 1, 256}; }
inline LayerLaunch plan_read_cache(int64_t T, int64_t heads, int64_t D) {
  return {PLAN_READ_CACHE, ceil_div(T * heads * (D / 16), 256), 2, 256};
}

// Attention.  Rows: queries times the heads that share keys.  The split kernel takes sequences of up
// to kAttendFew rows, which would not fill a unit of the tiled one, and all where no sequence can
// have more.  Measured, us, split (tiled), 32 heads, 8 of keys, D = 128: 32 sequences of 48 rows and up to
// 4096 keys 60 (90), of 96 rows 85 (98), 8 of 128 rows and up to 2048 keys 38 (32).
constexpr int kAttendFew = 128;
// Workgroups of the split kernel at most: what runs at a time.  Of heads up to 128 the registers of
// two waves on a SIMD (three: 64 sequences of up to 8192 keys 88 -> 105 us, codes spilled), of
// larger ones of one (32 of head size 256: two 67 us, one 61).
constexpr int64_t kAttendPieces = 512;
constexpr int kAttendTile = 64;  // keys of a tile of its work

inline int attend_kernels(int64_t T, int64_t Hq, int64_t Hk, bool ends) { return ends && T * (Hq / Hk) > kAttendFew ? 3 : 1; }
// Tiles of the split kernel at most: with units of sixteen rows, of keys that the table's rows name.
inline int64_t attend_split_tiles(int64_t T, int64_t B, int64_t Hq, int64_t Hk, int64_t keys) {
  const int64_t G = Hq / Hk, few = ceil_div(G > kAttendFew ? G : kAttendFew, 16);
  const int64_t units = B * few * Hk;
  return units * (keys > 0 ? ceil_div(keys, kAttendTile) : 1) + ceil_div(T * G, 16) * Hk;
}
inline int64_t attend_pieces(int64_t T, int64_t B, int64_t Hq, int64_t Hk, int64_t D, int64_t keys) {
  const int64_t n = ceil_div(attend_split_tiles(T, B, Hq, Hk, keys), 4), most = D > 128 ? kAttendPieces / 2 : kAttendPieces;
  return n < most ? n : most;
}
// Tiles of a piece, one of `pieces`: of `total` tiles as many each, and so many that a unit of
// `longest` tiles lies in at most kMostParts pieces (the join takes them one after the other).
// Unsigned: total may come near 2^31, and total + pieces pass it.
constexpr int kMostParts = 512;
constexpr int attend_piece_tiles(uint32_t total, uint32_t longest, uint32_t pieces) {
  const uint32_t even = (total + pieces - 1) / pieces, most = (longest + kMostParts - 1) / kMostParts;
  return (int)(even > most ? even : most);
}
inline LayerLaunch plan_attend_split(int64_t T, int64_t B, int64_t Hq, int64_t Hk, int64_t D, int64_t keys) {
  return {PLAN_ATTEND_SPLIT, attend_pieces(T, B, Hq, Hk, D, keys), 1, 256};
}
// What its pieces leave: none where no unit has two tiles.
inline size_t attend_split_bytes(int64_t T, int64_t B, int64_t Hq, int64_t Hk, int64_t D, int64_t keys) {
  return keys <= kAttendTile ? 0 : (size_t)(4 * attend_pieces(T, B, Hq, Hk, D, keys) * (2 * (16 * D + 32) * 4 + 32));
}
// Tiled kernel.  Units of 32 rows a wave at most: each sequence adds less than one to T * G / rows.
// Eight waves share the decoding of a tile among twice the rows of four, where there are
// enough units and heads over 64 (two prompts of 8192, 32 heads of 128: 705 -> 655 us; 4 of 4096, 16 heads
// of 64: 120 -> 139).
// parts: workgroups that share a unit's keys, in pieces of kAttendLeast tiles of 64 or more, where
// units alone would not make 1024 workgroups: twice what runs at a time with four waves (two on a
// CU, three of heads up to 64, one of heads over 128), four times with eight (one on a CU).  512 queries behind 32768
// keys: 870 us whole, 350 in parts; pieces of four tiles instead of eight, which a piece's start and
// sums cost more than: 43 -> 50 us, 7 sequences of up to 301 queries and 1999 keys.
constexpr int kAttendLeast = 8;
struct TilesPlan {
  int waves, parts;
  int64_t units;
};
inline TilesPlan tiles_plan(int64_t T, int64_t B, int64_t Hq, int64_t Hk, int64_t D, int64_t keys) {
  const int64_t rows = T * (Hq / Hk);
  const int waves = D > 64 && D <= 128 && ceil_div(rows, 256) * Hk >= 256 ? 8 : 4;
  const int64_t units = (ceil_div(rows, 32 * waves) + B) * Hk;
  int64_t parts = 1024 / units, most = ceil_div(keys, 64 * kAttendLeast);
  if (parts > most) parts = most;
  return {waves, (int)(parts < 1 ? 1 : parts > 16 ? 16 : parts), units};
}
inline LayerLaunch plan_attend_tiles(int64_t T, int64_t B, int64_t Hq, int64_t Hk, int64_t D, int64_t keys) {
  const TilesPlan p = tiles_plan(T, B, Hq, Hk, D, keys);
  return {PLAN_ATTEND_TILES, p.units * p.parts, 1, 64 * p.waves};
}
// Joins both kernels' parts: four workgroups to one of the split kernel, one to sixteen rows
// of a shared unit of the tiled one.
inline LayerLaunch plan_attend_join(int64_t T, int64_t B, int64_t Hq, int64_t Hk, int64_t D, int64_t keys, int which) {
  if (keys <= kAttendTile) return {0, 0, 0, 0};  // no unit has two tiles
  const TilesPlan p = tiles_plan(T, B, Hq, Hk, D, keys);
  return {PLAN_ATTEND_JOIN, 4 * attend_pieces(T, B, Hq, Hk, D, keys) + (which & 2 && p.parts > 1 ? p.units * 2 * p.waves : 0), 1, 256};
}
// The split kernel's workspace, then the tiled one's: one launch joins both.
inline size_t attend_workspace_bytes(int64_t T, int64_t B, int64_t Hq, int64_t Hk, int64_t D, int64_t keys, bool ends) {
  size_t n = attend_split_bytes(T, B, Hq, Hk, D, keys);
  if (attend_kernels(T, Hq, Hk, ends) & 2) {
    const TilesPlan p = tiles_plan(T, B, Hq, Hk, D, keys);
    if (p.parts > 1) n += (size_t)(p.units * (32 + (int64_t)p.parts * 32 * p.waves * (D + 2) * 4));
  }
  return n;
}

}  // namespace nvfp4
