// mx_rules.h -- what the sizes of a microscaled product decide, on the host:
// its limits, its workspace, the parts its contraction goes in, and the kernel
// and tile it runs on.  Integer arithmetic only, so that it can be checked
// without a GPU.  Times are in us on one MI355X.
#pragma once
#include <stdint.h>

namespace {

constexpr uint64_t kMxMaxRows = 1ull << 31;
constexpr uint64_t kMxMaxCols = 1ull << 21;
constexpr uint32_t kMxMaxGroups = 4096u;
constexpr uint64_t kMxWsHead = 512u;  // of the workspace: control block, then the one status word
constexpr uint32_t kMxCus = 256u;
constexpr uint32_t kMxDxParts = 8u;
constexpr uint32_t kMxThreads = 256u;                            // of a workgroup (k_mx_few: 512)
constexpr uint64_t kMxMostGroups = 0xFFFFFFFFu / kMxThreads;     // of a launch: below 2^32 threads
constexpr uint32_t kMxUnits = 2u;                                // units of 8 values that a thread encodes or decodes

enum MxOp { kMxMatmul = 0, kMxDx = 1, kMxWgrad = 2, kMxMatmul8 = 3 };

// k_mx_few in its two forms (128 weight rows a workgroup; 16, the contraction
// split), then the tiles of k_mx_gemm and k_mx_gemm8 by rows and columns.
enum MxKernel {
  kMxFew128 = 0,
  kMxFew16 = 1,
  kMx32x128 = 2,
  kMx64x128 = 3,
  kMx128x128 = 4,
  kMx128x256 = 5,
  kMx32x256 = 6,
  kMx64x256 = 7,
  kMx256x128 = 8
};

struct MxSizes {
  uint64_t tokens, n, k;
  uint32_t groups;
  bool offsets;  // a table of offsets is given
};

constexpr uint64_t mx_cdiv(uint64_t a, uint64_t b) { return (a + b - 1u) / b; }

// Token tiles of bm rows that the groups can need between them.
inline uint64_t mx_token_tiles(uint64_t tokens, uint64_t groups, uint32_t bm) {
  return tokens / bm + (groups < tokens ? groups : tokens);
}
inline uint64_t mx_token_tiles(const MxSizes& s, uint32_t bm) {
  return s.offsets ? mx_token_tiles(s.tokens, s.groups, bm) : mx_cdiv(s.tokens, bm);
}

// Workgroups of an encode (cols: the padded ones) or a decode.
inline uint64_t mx_unit_groups(uint64_t rows, uint64_t cols) {
  return mx_cdiv(rows * mx_cdiv(cols, 8u), kMxThreads * kMxUnits);
}
// Workgroups of a product in tiles of bm x bn (dx's parts are the grid's second
// dimension).  k_mx_few's stay far below the limit: cdiv(n, 16) <= 2^13.
inline uint64_t mx_tile_groups(int op, uint32_t bm, uint32_t bn, const MxSizes& s, uint32_t parts) {
  if (op == kMxWgrad) {
    const uint64_t tiles = mx_cdiv(s.n, bm) * mx_cdiv(s.k, bn);
    return (s.groups > 1u ? mx_cdiv(tiles, 8u) * 8u : tiles) * s.groups * parts;  // groups: an eighth of them an XCD
  }
  return mx_token_tiles(s, bm) * mx_cdiv(op == kMxDx ? s.k : s.n, bn);
}

// wgrad: where the tiles would leave CUs idle, each group's tokens go in up to
// eight parts, at least 512 rows each on average, whose FP32 sums k_mx_join
// adds in order (n = k = 2,048, FP32: 8,192 rows 95 against 174 us in one
// part, 2,048 rows 43 against 52; 1,024 rows in parts of 256: 36 against 30 in
// one).
inline uint32_t mx_wgrad_parts(uint64_t tokens, uint64_t n, uint64_t k, uint64_t groups) {
  const uint64_t tiles = mx_cdiv(n, 256u) * mx_cdiv(k, 128u) * groups;
  uint64_t parts = 2u * kMxCus / tiles;
  if (parts > tokens / groups / 512u) parts = tokens / groups / 512u;
  return parts < 1u ? 1u : parts > 8u ? 8u : uint32_t(parts);
}
// dx: where even its smallest tiles leave CUs without a workgroup, n goes in up
// to eight parts of at least 256, joined likewise (n = k = 2,048: 40 rows 14.5
// against 23.0 us in one part, 256 rows 16.2 against 23.3).
inline uint32_t mx_dx_parts(uint64_t tokens, uint64_t n, uint64_t k, uint64_t groups) {
  const uint64_t tiles = mx_token_tiles(tokens, groups, 64u) * mx_cdiv(k, 128u);
  uint64_t parts = tiles ? kMxCus / tiles : 1u;
  if (parts > n / 256u) parts = n / 256u;
  return parts < 1u ? 1u : parts > kMxDxParts ? kMxDxParts : uint32_t(parts);
}

// Workspace bytes; 0 when a size is out of range.
inline uint64_t mx_ws_size(uint64_t tokens, uint64_t n, uint64_t k, uint64_t groups) {
  if (tokens > kMxMaxRows - 1u || !n || !k || n > kMxMaxCols || k > kMxMaxCols || !groups || groups > kMxMaxGroups ||
      groups * n > kMxMaxRows)
    return 0u;
  // Sized for every smaller number of tokens too, some of which dx takes in
  // more parts: as parts * tiles <= kMxCus and tokens < 64 tiles / columns'
  // tiles, the parts' rows stay below 64 kMxCus / columns' tiles.
  const uint64_t wgrad = mx_wgrad_parts(tokens, n, k, groups), cols = mx_cdiv(k, 128u);
  const uint64_t sums = wgrad > 1u ? wgrad * groups * n * k : 0u;
  uint64_t rows = n >= 512u && cols <= kMxCus / 2u ? 64u * kMxCus / cols : 0u;
  if (rows > kMxDxParts * tokens) rows = kMxDxParts * tokens;
  return kMxWsHead + (sums > rows * k ? sums : rows * k) * 4u;
}

// What the rules below go by: tiles of 128 x 256 that the output would make,
// and the rows a group has on average, those without rows counted (which have
// some is known on the GPU alone; calls to a few of many groups get the tiles
// of sparser ones).
inline uint64_t mx_tiles(const MxSizes& s, uint64_t cols) { return mx_cdiv(s.tokens, 128u) * mx_cdiv(cols, 256u); }
inline uint64_t mx_rows_each(const MxSizes& s) { return s.tokens / s.groups; }

// The kernel of y = x W^T with FP32 sums.
//
// k_mx_few: its time grows with the outputs, the tiles' does not until they
// fill the chip, so it is for products of at most kMxFewOutputs (k = 2,048: 16
// rows, n = 8,192: 9.0 against 11.9 us, 24 rows: 14.1 against 12.0; 64 g, n =
// 1,024, 128 rows: 16.9 against 17.5, 512 rows: 33 against 22).  128 weight
// rows a workgroup once that gives every other CU one (one token: n = 8,192:
// 9.0 against 8.2 us, 16,384: 8.8 against 11.0), else 16.
// And its workgroups take a group's rows 16 at a time, one pass after the
// other, while the tiles take them at once, so it is for few rows a group, on
// average; the larger groups of uneven ones (the more groups, the larger) then
// need two passes, or three of the shorter ones of the split form (n = 256, k =
// 2,048 and 8,192):
//   one group, split: 32 rows: 9.1, 24 against 11.8, 40; 48: 12.5, 35 against 11.8, 40; 64: 16.2, 45 against 11.8,
//     40; 2,000 rows of n = 64: 470, 1,434 against 12.3, 41.  x in mx8, k = 2,048: 64: 14.7 against 16.8; 128: 27, 17.
//   groups, split: 96 rows in 4: 12.4, 32 against 12.7, 40; 128 in 4: 14.6, 43 against 12.7, 40; 256 in 16: 12.2, 33
//     against 12.8, 41; 384 in 16: 14.8, 42 against 12.9, 41.  mx8: 512 in 16: 16.1 against 17.8; 1,024 in 16: 25, 18.
//   groups, 128 rows a workgroup: 256 rows in 64: 10.8, 35 against 13.0, 41; 384 in 64: 15.5, 52 against 13.1, 46;
//     n = 1,024: 96 in 16: 11.4, 37 against 13.4, 41; 128 in 16: 17.7, 60 against 13.4, 41.  mx8: 512 in 64: 16.1, 17.4.
//
// The tile shapes.  Small outputs want many small tiles, so that every CU has
// work; large ones want large tiles, which read less; and a group's last tile
// is half empty, so tiles stay below the rows a group has.  Both sides of each
// rule (rows of one group with n = k = 2,048; "8 g", "64 g": rows of so many
// groups together with n = 1,024, k = 2,048):
//   32 or 64 rows: 1,024: 18.0, 18.7; 2,048: 34, 25; 2,000 in 64 g: 25, 27.5; 5,000 in 64 g: 47, 40.
//   64 or 128 rows: 3,000: 32, 34; 4,096: 46, 37; 6,000 in 64 g: 43, 46; 8,192 in 64 g: 55, 48.
//   128 rows, 128 or 256 columns: 4,001: 37, 41; 8,192: 72, 69; 32,768: 265, 252; in 64 g: 154, 150.
//     x in mx8: 8,192 with n = 4,096, k = 8,192: 455, 430; 32,768: 227, 230; in 64 g: 138, 142; 16,384 in 8 g, n = 2,048: 126, 138.
constexpr uint64_t kMxFewOutputs = 1u << 17;  // most outputs (all tokens' n) that k_mx_few is taken for

inline MxKernel mx_matmul_kernel(const MxSizes& s, bool mx8) {
  const uint64_t tiles = mx_tiles(s, s.n), rows = mx_rows_each(s);
  if (s.tokens * s.n <= kMxFewOutputs) {
    const uint64_t live = s.groups < s.tokens ? s.groups : s.tokens;
    const MxKernel form = mx_cdiv(s.n, 128u) * live >= kMxCus / 2u ? kMxFew128 : kMxFew16;
    uint32_t most = mx8 ? 64u : 48u;
    if (s.groups > 1u && form == kMxFew16) most = mx8 ? 32u : s.groups <= 8u ? 24u : 16u;
    if (s.groups > 1u && form == kMxFew128) most = mx8 ? 8u : s.groups <= 32u ? 6u : 5u;
    if (rows <= most) return form;
  }
  if (rows > 64u && tiles >= 2u * kMxCus && !(mx8 && s.groups > 1u)) return kMx128x256;
  if (rows > 64u && tiles > 3u * kMxCus / 4u) return kMx128x128;
  if (!mx8 && (rows <= 48u || tiles <= kMxCus / 4u)) return kMx32x128;
  return kMx64x128;
}

// The tile of k_mx_gemm8: 32 or 64 rows: 2,048: 21, 16; 2,000 in 64 g: 17, 23;
// 6,000 in 64 g: 32, 30; 64 or 128 rows: 3,000: 24, 24; 8,192: 56, 44; 6,000 in
// 64 g: 30, 34.
inline MxKernel mx_scaled_kernel(const MxSizes& s) {
  const uint64_t tiles = mx_tiles(s, s.n), rows = mx_rows_each(s);
  if (rows > 64u && tiles > 3u * kMxCus / 4u) return kMx128x256;
  if (rows > 48u && tiles > kMxCus / 4u) return kMx64x128;
  return kMx32x128;
}

// The tile of dx = dy W, likewise:
//   64 x 128 or 64 x 256: 512: 23, 29; 2,048: 34, 33; 64 in 64 g: 27, 22; 4,000 in 64 g: 40, 32.
//   32 or 64 rows of 256: 999 in 66 g with n = 1,408: 27, 31; 500 in 64 g: 18, 22; 3,000: 30, 31; 4,000: 36, 33.
//   64 or 128 rows: 4,096: 40, 41; 8,192: 70, 62; 32,768: 260, 245; 16,384 in 4 g: 80, 85; 8,192 in 8 g, n = 512: 29, 33;
//     32,768 in 64 g: 167, 170; with n = 2,048: 8,192 in 2 g: 84, 93; 32,768 in 4 g: 272, 264.
inline MxKernel mx_dx_kernel(const MxSizes& s) {
  if (mx_rows_each(s) >= 1024u && mx_tiles(s, s.k) >= (s.groups > 1u ? 8u : 2u) * kMxCus) return kMx128x256;
  if (mx_token_tiles(s, 64u) * mx_cdiv(s.k, 128u) <= 2u * kMxCus) return kMx64x128;
  return mx_rows_each(s) <= 48u ? kMx32x256 : kMx64x256;
}

}  // namespace
