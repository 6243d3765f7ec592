// mx.hip -- microscaled matrices: BF16 matrices held in 8 bits (mx8, e4m3) or
// 4 bits (mx4, e2m1) per value with one power-of-two scale byte per 32 values
// of a row, and the products a linear layer makes of them, gfx950.
//
// A block v_0 .. v_31 is kept as a scale s = 2^max(-126, ceil(log2(max|v| /
// M))), M = 448 (e4m3) or 6 (e2m1), and q_i = v_i / s rounded to the nearest
// value of the element type, ties to even.  No |v_i / s| exceeds M, so nothing
// saturates and every value is off by at most half a step of its grid.  s q_i
// has at most four significant bits, so it is exact in BF16 (the BF16 products
// below multiply exactly what the block stands for and round nowhere before
// the FP32 sum).
//
// Every kernel reads the grouped form: rows offsets[g] .. offsets[g+1] - 1 of
// the token matrices belong to group g, whose weights are rows g n ..
// (g+1) n - 1 of W.  A pair that decreases or leaves 0 .. tokens holds no
// rows; workgroup 0 of every product reports it.
#include "ciera.h"

namespace {

typedef int v4i __attribute__((ext_vector_type(4)));
typedef int v8i __attribute__((ext_vector_type(8)));
typedef float v4f __attribute__((ext_vector_type(4)));
typedef float v16f __attribute__((ext_vector_type(16)));
typedef short v2s __attribute__((ext_vector_type(2)));
typedef short v4s __attribute__((ext_vector_type(4)));
typedef __bf16 v2bf __attribute__((ext_vector_type(2)));
typedef __bf16 v8bf __attribute__((ext_vector_type(8)));
// 16 bytes at any 2-byte address: global memory takes unaligned wide loads.
typedef uint32_t u32x4a2 __attribute__((ext_vector_type(4), aligned(2)));
typedef uint32_t u32x4v __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2v __attribute__((ext_vector_type(2)));

constexpr uint32_t kMxBlock = 32u;
constexpr uint32_t kMxThreads = 256u;
constexpr uint64_t kMxMaxRows = 1ull << 31;
constexpr uint64_t kMxMaxCols = 1ull << 21;
constexpr uint64_t kMxMaxLd = 1ull << 22;
constexpr uint32_t kMxMaxGroups = 4096u;
constexpr uint64_t kMxWsHead = 512u;  // control block, then the one status word

__host__ __device__ constexpr uint64_t mx_pitch(uint64_t cols) { return (cols + 127u) & ~uint64_t(127); }
// Bytes of the value section; the scales start there.
__host__ __device__ constexpr uint64_t mx_scales_at(uint64_t rows, uint64_t cols, uint32_t bits) {
  return (rows * mx_pitch(cols) * bits / 8u + 127u) & ~uint64_t(127);
}
__host__ __device__ constexpr uint64_t mx_size(uint64_t rows, uint64_t cols, uint32_t bits) {
  return mx_scales_at(rows, cols, bits) + rows * (mx_pitch(cols) / kMxBlock);
}

__device__ __forceinline__ float mx_scale(uint32_t byte) { return __uint_as_float(byte << 23); }

__device__ __forceinline__ v2bf mx_bf2(uint32_t w) { return __builtin_bit_cast(v2bf, w); }

// Two BF16 values of byte `sel` (mx4) or half `sel` (mx8) of q, times the
// scale.  A scale byte of 255 gives NaN for every code.
template <int kBits, int kSel>
__device__ __forceinline__ uint32_t mx_pair(uint32_t q, float scale) {
  v2bf v;
  if constexpr (kBits == 8) v = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(q, scale, kSel != 0);
  else v = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(q, scale, kSel);
  return __builtin_bit_cast(uint32_t, v);
}

// Eight values: 8 bytes of mx8 or 4 bytes of mx4 as BF16.
__device__ __forceinline__ u32x4v mx_unit8(uint32_t lo, uint32_t hi, float s) {
  return u32x4v{mx_pair<8, 0>(lo, s), mx_pair<8, 1>(lo, s), mx_pair<8, 0>(hi, s), mx_pair<8, 1>(hi, s)};
}
__device__ __forceinline__ u32x4v mx_unit4(uint32_t q, float s) {
  return u32x4v{mx_pair<4, 0>(q, s), mx_pair<4, 1>(q, s), mx_pair<4, 2>(q, s), mx_pair<4, 3>(q, s)};
}

// Eight BF16 values from `src` of which the first `have` exist, zeros behind.
__device__ __forceinline__ u32x4v mx_part8(const uint16_t* src, uint32_t have) {
  u32x4v w = {0u, 0u, 0u, 0u};
#pragma unroll
  for (uint32_t i = 0; i < 8u; i++)
    if (i < have) w[i >> 1] |= uint32_t(src[i]) << (16u * (i & 1u));
  return w;
}

// ---------------------------------------------------------------------------
// Encode and decode.  A unit is 8 values of a row (16 bytes of BF16); four
// neighbouring lanes hold a block and find its largest magnitude with two
// lane exchanges.  Bound by memory: 2 bytes read and 1.03 (mx8) or 0.53 (mx4)
// written per value, or the reverse.  A thread takes kMxUnits units a
// workgroup's width apart and issues all their loads before it uses one.
// ---------------------------------------------------------------------------
constexpr uint32_t kMxUnits = 4u;

struct MxUnitAt {
  uint64_t row;
  uint32_t col;
};
// Unit `u` of this thread: row and first column (upr units per row).
__device__ __forceinline__ MxUnitAt mx_unit_at(uint64_t first_row, uint32_t first_unit, uint32_t u, uint32_t upr) {
  const uint32_t at = first_unit + u * kMxThreads + threadIdx.x;
  const uint32_t dr = at / upr;
  return {first_row + dr, (at - dr * upr) * 8u};
}

template <int kBits>
__global__ __launch_bounds__(kMxThreads) void k_mx_encode(const uint16_t* __restrict__ x, uint64_t rows, uint32_t cols,
                                                          uint64_t ld, uint8_t* __restrict__ q,
                                                          uint8_t* __restrict__ scales, uint32_t pad_bytes) {
  const uint32_t upr = uint32_t(mx_pitch(cols) / 8u);
  const uint64_t first = uint64_t(blockIdx.x) * (kMxThreads * kMxUnits);
  const uint64_t first_row = first / upr;
  const uint32_t first_unit = uint32_t(first - first_row * upr);
  u32x4v v[kMxUnits];
  MxUnitAt at[kMxUnits];
#pragma unroll
  for (uint32_t u = 0; u < kMxUnits; u++) {
    at[u] = mx_unit_at(first_row, first_unit, u, upr);
    // a unit with no whole 8 values here reads the matrix's first 8 (or
    // nothing when there are not that many) and is mended below
    const bool whole = at[u].row < rows && at[u].col + 8u <= cols;
    const uint16_t* src = x + (whole ? at[u].row * ld + at[u].col : 0u);
    v[u] = cols >= 8u ? u32x4v(*reinterpret_cast<const u32x4a2*>(src)) : u32x4v{0u, 0u, 0u, 0u};
  }
#pragma unroll
  for (uint32_t u = 0; u < kMxUnits; u++) {
    if (at[u].col + 8u > cols) {  // the row's end: what is left of it, then zeros
      const uint32_t have = at[u].row < rows && at[u].col < cols ? cols - at[u].col : 0u;
      v[u] = mx_part8(x + (have ? at[u].row * ld + at[u].col : 0u), have);
    }
    uint32_t m = 0u;
#pragma unroll
    for (int i = 0; i < 4; i++) {
      const uint32_t a = v[u][i] & 0x7FFF7FFFu;
      m = max(m, max(a & 0xFFFFu, a >> 16));
    }
    m = max(m, uint32_t(__shfl_xor(int(m), 1)));
    m = max(m, uint32_t(__shfl_xor(int(m), 2)));
    // 448 = 1.75 2^8, 6 = 1.5 2^2: one binade more when the significand of
    // the largest value is above that
    constexpr int kTopExp = kBits == 8 ? 8 : 2;
    constexpr uint32_t kTopMan = kBits == 8 ? 96u : 64u;
    const int e = int(m >> 7) - kTopExp + int((m & 127u) > kTopMan);
    const bool bad = m >= 0x7F80u;  // an infinity or a NaN in the block
    const uint32_t sb = bad ? 255u : uint32_t(e < 1 ? 1 : e);
    const float s = mx_scale(bad ? 127u : sb);
    if (bad) v[u] = u32x4v{0u, 0u, 0u, 0u};
    if (at[u].row < rows) {
      const uint64_t dst = at[u].row * uint64_t(upr) * kBits + uint64_t(at[u].col) * kBits / 8u;
      if constexpr (kBits == 8) {
        u32x2v out;
#pragma unroll
        for (int h = 0; h < 2; h++) {
          v2s r = {0, 0};
          r = __builtin_amdgcn_cvt_scalef32_pk_fp8_bf16(r, mx_bf2(v[u][2 * h]), s, false);
          r = __builtin_amdgcn_cvt_scalef32_pk_fp8_bf16(r, mx_bf2(v[u][2 * h + 1]), s, true);
          out[h] = __builtin_bit_cast(uint32_t, r);
        }
        *reinterpret_cast<u32x2v*>(q + dst) = out;
      } else {
        uint32_t r = 0u;
        r = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(r, mx_bf2(v[u][0]), s, 0);
        r = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(r, mx_bf2(v[u][1]), s, 1);
        r = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(r, mx_bf2(v[u][2]), s, 2);
        r = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(r, mx_bf2(v[u][3]), s, 3);
        *reinterpret_cast<uint32_t*>(q + dst) = r;
      }
      if ((threadIdx.x & 3u) == 0u) scales[at[u].row * (upr / 4u) + at[u].col / kMxBlock] = uint8_t(sb);
    }
  }
  // zeros between the values and the scales
  if (blockIdx.x == 0u && threadIdx.x < pad_bytes) scales[int64_t(threadIdx.x) - int64_t(pad_bytes)] = 0u;
}

template <int kBits>
__global__ __launch_bounds__(kMxThreads) void k_mx_decode(const uint8_t* __restrict__ q,
                                                          const uint8_t* __restrict__ scales, uint64_t rows,
                                                          uint32_t cols, uint16_t* __restrict__ y, uint64_t ld) {
  const uint32_t upr = (cols + 7u) / 8u;  // only the columns that exist
  const uint32_t kp = uint32_t(mx_pitch(cols));
  const uint64_t first = uint64_t(blockIdx.x) * (kMxThreads * kMxUnits);
  const uint64_t first_row = first / upr;
  const uint32_t first_unit = uint32_t(first - first_row * upr);
  uint32_t lo[kMxUnits], hi[kMxUnits], sb[kMxUnits];
  MxUnitAt at[kMxUnits];
#pragma unroll
  for (uint32_t u = 0; u < kMxUnits; u++) {
    at[u] = mx_unit_at(first_row, first_unit, u, upr);
    const uint64_t row = at[u].row < rows ? at[u].row : 0u;
    const uint8_t* src = q + row * (uint64_t(kp) * kBits / 8u) + at[u].col * kBits / 8u;
    if constexpr (kBits == 8) {
      const u32x2v w = *reinterpret_cast<const u32x2v*>(src);
      lo[u] = w[0];
      hi[u] = w[1];
    } else {
      lo[u] = *reinterpret_cast<const uint32_t*>(src);
      hi[u] = 0u;
    }
    sb[u] = scales[row * (kp / kMxBlock) + at[u].col / kMxBlock];
  }
#pragma unroll
  for (uint32_t u = 0; u < kMxUnits; u++) {
    const u32x4v v = kBits == 8 ? mx_unit8(lo[u], hi[u], mx_scale(sb[u])) : mx_unit4(lo[u], mx_scale(sb[u]));
    if (at[u].row >= rows) continue;
    uint16_t* dst = y + at[u].row * ld + at[u].col;
    if (at[u].col + 8u <= cols) {
      *reinterpret_cast<u32x4a2*>(dst) = v;
    } else {
#pragma unroll
      for (uint32_t i = 0; i < 7u; i++)
        if (at[u].col + i < cols) dst[i] = uint16_t(v[i >> 1] >> (16u * (i & 1u)));
    }
  }
}

// ---------------------------------------------------------------------------
// Products.
// ---------------------------------------------------------------------------
struct MxArgs {
  const uint16_t* a;      // BF16 operand: x (matmul) or dy (dx, wgrad)
  uint64_t lda;           // values from one of its rows to the next
  const uint8_t* xq;      // mx8 operand: values and scales
  const uint8_t* xs;
  const uint8_t* wq;      // mx4 weights: values and scales
  const uint8_t* ws;
  void* out;              // BF16 or FP32
  uint64_t ldo;
  const int64_t* offsets; // groups + 1 row numbers, or null: one group of all rows
  Ctrl* ctrl;
  uint32_t* status;
  uint32_t tokens, n, k, kp, groups;
  uint32_t out_f32, accumulate;
};

// Rows of group g, none when its pair of offsets is not in order or leaves
// the token matrix.
__device__ __forceinline__ bool mx_rows(const MxArgs& p, uint32_t g, uint32_t& r0, uint32_t& r1) {
  if (!p.offsets) {
    r0 = 0u;
    r1 = p.tokens;
    return true;
  }
  const int64_t a = p.offsets[g], b = p.offsets[g + 1u];
  const bool ok = a >= 0 && a <= b && b <= int64_t(p.tokens);
  r0 = ok ? uint32_t(a) : 0u;
  r1 = ok ? uint32_t(b) : 0u;
  return ok;
}

// Workgroup 0 of a product: the status word that ciera_read_error reads.
__device__ __forceinline__ void mx_report(const MxArgs& p) {
  if (threadIdx.x >= 64u) return;
  bool ok = true;
  for (uint32_t g = threadIdx.x; g < p.groups; g += 64u) {
    uint32_t r0, r1;
    ok = mx_rows(p, g, r0, r1) && ok;
  }
  const bool all = __all(ok);
  if (threadIdx.x == 0u) {
    p.ctrl->n_err_slots = 1u;
    *p.status = all ? uint32_t(CIERA_OK) : uint32_t(CIERA_ERR_ARG);
  }
}

// The group and rows of token tile `tile` of `1 << lbm` rows, tiles numbered
// group by group.  Every wave finds it for itself: 64 groups a step, their
// tile counts summed by a lane scan.
__device__ __forceinline__ bool mx_find_tile(const MxArgs& p, uint32_t tile, uint32_t lbm, uint32_t& g, uint32_t& row0,
                                             uint32_t& row1) {
  if (!p.offsets) {
    g = 0u;
    row0 = tile << lbm;
    row1 = p.tokens;
    return row0 < row1;
  }
  const uint32_t lane = threadIdx.x & 63u;
  uint32_t before = 0u;
  for (uint32_t c = 0; c < p.groups; c += 64u) {
    uint32_t r0 = 0u, r1 = 0u;
    if (c + lane < p.groups) mx_rows(p, c + lane, r0, r1);
    const uint32_t mine = (r1 - r0 + (1u << lbm) - 1u) >> lbm;
    uint32_t sum = mine;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const uint32_t up = uint32_t(__shfl_up(int(sum), d));
      if (lane >= uint32_t(d)) sum += up;
    }
    const uint64_t past = __ballot(before + sum > tile);
    if (past) {
      const int l = __ffsll((unsigned long long)past) - 1;
      const uint32_t skip = tile - (before + uint32_t(__shfl(int(sum - mine), l)));
      g = uint32_t(__builtin_amdgcn_readfirstlane(int(c) + l));
      row0 = uint32_t(__builtin_amdgcn_readfirstlane(__shfl(int(r0), l) + int(skip << lbm)));
      row1 = uint32_t(__builtin_amdgcn_readfirstlane(__shfl(int(r1), l)));
      return true;
    }
    before += uint32_t(__shfl(int(sum), 63));
  }
  return false;
}

__device__ __forceinline__ uint16_t mx_bf16(float f) { return __builtin_bit_cast(uint16_t, __bf16(f)); }
__device__ __forceinline__ float mx_f32(uint16_t b) { return __uint_as_float(uint32_t(b) << 16); }

__device__ __forceinline__ void mx_store(const MxArgs& p, uint64_t at, float v) {
  if (p.out_f32) {
    float* o = static_cast<float*>(p.out) + at;
    *o = p.accumulate ? *o + v : v;
  } else {
    uint16_t* o = static_cast<uint16_t*>(p.out) + at;
    *o = mx_bf16(p.accumulate ? mx_f32(*o) + v : v);
  }
}

enum MxOp { kMxMatmul = 0, kMxDx = 1, kMxWgrad = 2, kMxMatmul8 = 3 };

constexpr uint32_t kMxBN = 128u;  // output columns of a tile
constexpr uint32_t kMxBC = 64u;   // contraction values staged per step (BF16 products)

// Byte offsets in the staged tiles.  "Rows": row r of 64 contraction values,
// 128 bytes, its 16-byte chunks exclusive-ored with r / 2, so that the 32
// rows a fragment read touches fall on all banks.  "Cols": contraction row c
// of `cols` values, its 64-byte pieces exclusive-ored with c, so that the
// four rows a transposing read gathers fall on different banks.
__device__ __forceinline__ uint32_t mx_rows_at(uint32_t r, uint32_t chunk) {
  return r * 128u + ((chunk ^ ((r >> 1) & 7u)) << 4);
}
__device__ __forceinline__ uint32_t mx_cols_at(uint32_t c, uint32_t byte, uint32_t cols) {
  return c * cols * 2u + (byte ^ ((c & 3u) << 6));
}

__device__ __forceinline__ v8bf mx_read_rows(const uint8_t* tile, uint32_t r, uint32_t chunk) {
  return *reinterpret_cast<const v8bf*>(tile + mx_rows_at(r, chunk));
}
// Eight contraction values c0 .. c0 + 7 of one column per lane: two reads
// that each transpose 4 rows x 16 columns within 16 lanes.
__device__ __forceinline__ v8bf mx_read_cols(const uint8_t* tile, uint32_t c0, uint32_t col0, uint32_t cols) {
  typedef __attribute__((address_space(3))) v4s lds_v4s;
  const uint32_t l = threadIdx.x & 15u;
  const uint32_t byte = (col0 + (l & 3u) * 4u) * 2u;
  const uint32_t c = c0 + (l >> 2);
  const v4s lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4s*)(tile + mx_cols_at(c, byte, cols)));
  const v4s hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4s*)(tile + mx_cols_at(c + 4u, byte, cols)));
  const v4s both[2] = {lo, hi};
  return __builtin_bit_cast(v8bf, both);
}

// The products on BF16 matrix instructions: tiles of kBM x 128 outputs, four
// waves, 64 contraction values per step.  The mx operand becomes BF16 on its
// way into LDS; a wave keeps its 32 x 32 sums in registers.
//   matmul  M tokens, N weight rows, contraction k:  both operands run along
//           the contraction in memory; x in BF16 or mx8
//   dx      M tokens, N k, contraction n:  W's rows are contraction rows, read
//           back transposed
//   wgrad   M n, N k, contraction tokens of the group:  both transposed
template <int kOp, uint32_t kBM>
__global__ __launch_bounds__(kMxThreads, 2) void k_mx_gemm(MxArgs p) {
  __shared__ __attribute__((aligned(16))) uint8_t s_a[kBM * 128u];
  __shared__ __attribute__((aligned(16))) uint8_t s_b[kMxBN * 128u];
  constexpr bool kRowsB = kOp == kMxMatmul || kOp == kMxMatmul8;  // B runs along the contraction
  constexpr uint32_t kAChunks = kBM * (kOp == kMxMatmul8 ? 4u : 8u) / kMxThreads;  // 16-byte loads of A per thread
  constexpr uint32_t kBChunks = kOp == kMxWgrad ? 2u : 1u;
  constexpr uint32_t kFM = kBM / 64u;  // 32-row fragments of a wave
  constexpr uint32_t kFN = 2u;
  const uint32_t tid = threadIdx.x, lane = tid & 63u, wave = tid >> 6;
  if (blockIdx.x == 0u) mx_report(p);

  // where the tile is: its group, its output rows m0 .. m1 - 1 and columns
  uint32_t g, m0, m1, n0, c1;
  const uint32_t cols = kRowsB ? p.n : p.k;
  const uint32_t ntiles = (cols + kMxBN - 1u) / kMxBN;
  uint32_t r0 = 0u;  // first contraction row (wgrad)
  if constexpr (kOp == kMxWgrad) {
    const uint32_t mtiles = (p.n + kBM - 1u) / kBM;
    g = blockIdx.x / (mtiles * ntiles);
    const uint32_t t = blockIdx.x - g * (mtiles * ntiles);
    m0 = (t / ntiles) * kBM;
    n0 = (t % ntiles) * kMxBN;
    m1 = p.n;
    uint32_t r1;
    mx_rows(p, g, r0, r1);
    c1 = r1 - r0;
  } else {
    const uint32_t t = blockIdx.x / ntiles;
    n0 = (blockIdx.x - t * ntiles) * kMxBN;
    constexpr uint32_t kLog = kBM == 256u ? 8u : 6u;
    if (!mx_find_tile(p, t, kLog, g, m0, m1)) return;
    c1 = kRowsB ? p.k : p.n;
  }
  const uint32_t steps = (c1 + kMxBC - 1u) / kMxBC;

  // A: byte offsets of this thread's chunks from the tile's first row
  const uint8_t* a_base;
  const uint8_t* as_base = nullptr;  // the scales of an mx8 A
  uint32_t a_off[kAChunks];
  if constexpr (kOp == kMxWgrad) {
    a_base = reinterpret_cast<const uint8_t*>(p.a + uint64_t(r0) * p.lda + m0);
  } else if constexpr (kOp == kMxMatmul8) {
    a_base = p.xq + uint64_t(m0) * p.kp;
    as_base = p.xs + uint64_t(m0) * (p.kp / 32u);
#pragma unroll
    for (uint32_t i = 0; i < kAChunks; i++)
      a_off[i] = min(i * 64u + (tid >> 2), m1 - 1u - m0) * p.kp + (tid & 3u) * 16u;
  } else {
    a_base = reinterpret_cast<const uint8_t*>(p.a + uint64_t(m0) * p.lda);
#pragma unroll
    for (uint32_t i = 0; i < kAChunks; i++) {
      const uint32_t r = min(i * 32u + (tid >> 3), m1 - 1u - m0);
      a_off[i] = r * uint32_t(p.lda) * 2u + (tid & 7u) * 16u;
    }
  }
  u32x4v va[kAChunks];
  uint32_t sa[kAChunks];
  v4i vb[kBChunks];
  uint32_t sb[kBChunks];

  const auto load_a = [&](uint32_t step) {
    const uint32_t c0 = step * kMxBC;
    if constexpr (kOp == kMxWgrad) {
      // contraction row c0 + i * 8 + tid / 32 (kBM = 256), 8 columns
      constexpr uint32_t kPerRow = kBM / 8u;
      const uint32_t col = (tid % kPerRow) * 8u;
      const uint8_t* base = a_base + uint64_t(c0) * p.lda * 2u;
      const bool edge = m0 + kBM > p.n;
#pragma unroll
      for (uint32_t i = 0; i < kAChunks; i++) {
        const uint32_t r = (i * kMxThreads + tid) / kPerRow;
        const uint32_t rc = min(r, c1 - 1u - c0);
        const uint8_t* src = base + rc * uint32_t(p.lda) * 2u;
        if (!edge) {
          va[i] = *reinterpret_cast<const u32x4a2*>(src + col * 2u);
        } else {  // columns past n are not read
          const uint32_t have = m0 + col < p.n ? p.n - m0 - col : 0u;
          va[i] = mx_part8(reinterpret_cast<const uint16_t*>(src) + (have ? col : 0u), have);
        }
        if (c0 + kMxBC > c1 && r != rc) va[i] = u32x4v{0u, 0u, 0u, 0u};
      }
    } else if constexpr (kOp == kMxMatmul8) {
#pragma unroll
      for (uint32_t i = 0; i < kAChunks; i++) {
        va[i] = *reinterpret_cast<const u32x4v*>(a_base + a_off[i] + c0);
        sa[i] = as_base[(a_off[i] + c0) / 32u];
      }
    } else {
      const uint8_t* base = a_base + c0 * 2u;
      if (c0 + kMxBC <= c1) {
#pragma unroll
        for (uint32_t i = 0; i < kAChunks; i++) va[i] = *reinterpret_cast<const u32x4a2*>(base + a_off[i]);
      } else {  // the contraction ends in this step: zeros behind it
        const uint32_t c = c0 + (tid & 7u) * 8u;
#pragma unroll
        for (uint32_t i = 0; i < kAChunks; i++) {
          va[i] = mx_part8(reinterpret_cast<const uint16_t*>(base + a_off[i]), c < c1 ? c1 - c : 0u);
        }
      }
    }
  };
  const auto load_b = [&](uint32_t step) {
    const uint32_t c0 = step * kMxBC;
    if constexpr (kRowsB) {  // weight row n0 + tid / 2, one block of 32
      const uint64_t row = uint64_t(g) * p.n + min(n0 + (tid >> 1), p.n - 1u);
      const uint32_t at = c0 + (tid & 1u) * 32u;
      vb[0] = *reinterpret_cast<const v4i*>(p.wq + row * (p.kp / 2u) + at / 2u);
      sb[0] = p.ws[row * (p.kp / 32u) + at / 32u];
    } else if constexpr (kOp == kMxDx) {  // contraction row c0 + tid / 4, one block of 32
      const uint32_t c = c0 + (tid >> 2);
      const uint64_t row = uint64_t(g) * p.n + min(c, c1 - 1u);
      const uint32_t at = n0 + (tid & 3u) * 32u;
      vb[0] = *reinterpret_cast<const v4i*>(p.wq + row * (p.kp / 2u) + at / 2u);
      sb[0] = p.ws[row * (p.kp / 32u) + at / 32u];
      if (c >= c1) {
        vb[0] = v4i{0, 0, 0, 0};
        sb[0] = 127u;
      }
    } else {  // contraction row c0 + i * 32 + tid / 8, 16 values of a block
#pragma unroll
      for (uint32_t i = 0; i < kBChunks; i++) {
        const uint32_t c = c0 + i * 32u + (tid >> 3);
        const uint64_t row = uint64_t(r0) + min(c, c1 - 1u);
        const uint32_t at = n0 + (tid & 7u) * 16u;
        vb[i] = *reinterpret_cast<const v4i*>(p.xq + row * p.kp + at);
        sb[i] = p.xs[row * (p.kp / 32u) + at / 32u];
        if (c >= c1) {
          vb[i] = v4i{0, 0, 0, 0};
          sb[i] = 127u;
        }
      }
    }
  };
  const auto stage = [&]() {
#pragma unroll
    for (uint32_t i = 0; i < kAChunks; i++) {
      if constexpr (kOp == kMxMatmul8) {
        const float s = mx_scale(sa[i]);
#pragma unroll
        for (uint32_t h = 0; h < 2u; h++)
          *reinterpret_cast<u32x4v*>(s_a + mx_rows_at(i * 64u + (tid >> 2), (tid & 3u) * 2u + h)) =
              mx_unit8(va[i][2u * h], va[i][2u * h + 1u], s);
        continue;
      }
      uint32_t at;
      if constexpr (kOp == kMxWgrad) {
        constexpr uint32_t kPerRow = kBM / 8u;
        at = mx_cols_at((i * kMxThreads + tid) / kPerRow, (tid % kPerRow) * 16u, kBM);
      } else {
        at = mx_rows_at(i * 32u + (tid >> 3), tid & 7u);
      }
      *reinterpret_cast<u32x4v*>(s_a + at) = va[i];
    }
#pragma unroll
    for (uint32_t i = 0; i < kBChunks; i++) {
      const float s = mx_scale(sb[i]);
      if constexpr (kOp == kMxWgrad) {
#pragma unroll
        for (uint32_t h = 0; h < 2u; h++)
          *reinterpret_cast<u32x4v*>(s_b + mx_cols_at(i * 32u + (tid >> 3), (tid & 7u) * 32u + h * 16u, kMxBN)) =
              mx_unit8(uint32_t(vb[i][2u * h]), uint32_t(vb[i][2u * h + 1u]), s);
      } else {
#pragma unroll
        for (uint32_t h = 0; h < 4u; h++) {
          const uint32_t at = kRowsB ? mx_rows_at(tid >> 1, (tid & 1u) * 4u + h)
                                               : mx_cols_at(tid >> 2, (tid & 3u) * 64u + h * 16u, kMxBN);
          *reinterpret_cast<u32x4v*>(s_b + at) = mx_unit4(uint32_t(vb[i][h]), s);
        }
      }
    }
  };

  const uint32_t wm = (wave >> 1) * (kBM / 2u), wn = (wave & 1u) * 64u;
  v16f acc[kFM][kFN];
#pragma unroll
  for (uint32_t i = 0; i < kFM; i++)
#pragma unroll
    for (uint32_t j = 0; j < kFN; j++)
#pragma unroll
      for (int r = 0; r < 16; r++) acc[i][j][r] = 0.0f;

  if (steps) {
    load_a(0u);
    load_b(0u);
  }
  for (uint32_t step = 0; step < steps; step++) {
    if (step) __syncthreads();
    stage();
    __syncthreads();
    if (step + 1u < steps) {
      load_a(step + 1u);
      load_b(step + 1u);
    }
#pragma unroll
    for (uint32_t s = 0; s < kMxBC / 16u; s++) {
      v8bf fa[kFM], fb[kFN];
#pragma unroll
      for (uint32_t i = 0; i < kFM; i++) {
        if constexpr (kOp == kMxWgrad)
          fa[i] = mx_read_cols(s_a, s * 16u + (lane >> 5) * 8u, wm + i * 32u + ((lane >> 4) & 1u) * 16u, kBM);
        else
          fa[i] = mx_read_rows(s_a, wm + i * 32u + (lane & 31u), s * 2u + (lane >> 5));
      }
#pragma unroll
      for (uint32_t j = 0; j < kFN; j++) {
        if constexpr (kRowsB)
          fb[j] = mx_read_rows(s_b, wn + j * 32u + (lane & 31u), s * 2u + (lane >> 5));
        else
          fb[j] = mx_read_cols(s_b, s * 16u + (lane >> 5) * 8u, wn + j * 32u + ((lane >> 4) & 1u) * 16u, kMxBN);
      }
#pragma unroll
      for (uint32_t i = 0; i < kFM; i++)
#pragma unroll
        for (uint32_t j = 0; j < kFN; j++)
          acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(fa[i], fb[j], acc[i][j], 0, 0, 0);
    }
  }

  // a fragment's register r holds row 8 (r / 4) + 4 (lane / 32) + r % 4 of
  // column lane % 32
#pragma unroll
  for (uint32_t i = 0; i < kFM; i++)
#pragma unroll
    for (uint32_t j = 0; j < kFN; j++) {
      const uint32_t col = n0 + wn + j * 32u + (lane & 31u);
#pragma unroll
      for (uint32_t r = 0; r < 16u; r++) {
        const uint32_t row = m0 + wm + i * 32u + 8u * (r / 4u) + 4u * (lane >> 5) + (r & 3u);
        if (row < m1 && col < cols) {
          if constexpr (kOp == kMxWgrad) mx_store(p, (uint64_t(g) * p.n + row) * p.k + col, acc[i][j][r]);
          else mx_store(p, uint64_t(row) * p.ldo + col, acc[i][j][r]);
        }
      }
    }
}

// matmul of an mx8 operand with a BF16 result: the scaled matrix instructions
// take e4m3 and e2m1 values with their scale bytes as they are, at twice the
// BF16 instructions' rate.  They add blocks, and earlier sums, in FP32, but
// within a block of 32 they line the products up with the largest and cut what
// lies below 2^(E - 13), 2^E being that product's binade (measured, one small
// product beside a large one).  So a block's sum is off by at most 2^-8 of its
// largest product.  On activations with a few loud channels the result moved
// by 1/7 of a BF16 rounding at the most; where the caller asks for FP32 it
// would show, and k_mx_gemm computes that.  128 contraction values (four
// blocks) per step; the padded pitch leaves no partial step.
template <uint32_t kBM>
__global__ __launch_bounds__(kMxThreads, 2) void k_mx_gemm8(MxArgs p) {
  __shared__ __attribute__((aligned(16))) uint8_t s_a[kBM * 128u];
  __shared__ __attribute__((aligned(16))) uint8_t s_b[kMxBN * 64u];
  __shared__ uint32_t s_sa[kBM], s_sb[kMxBN];  // a row's four scale bytes
  constexpr uint32_t kAChunks = kBM * 8u / kMxThreads;
  constexpr uint32_t kFM = kBM / 64u;
  constexpr uint32_t kFN = 2u;
  const uint32_t tid = threadIdx.x, lane = tid & 63u, wave = tid >> 6;
  if (blockIdx.x == 0u) mx_report(p);
  const uint32_t ntiles = (p.n + kMxBN - 1u) / kMxBN;
  const uint32_t t = blockIdx.x / ntiles;
  const uint32_t n0 = (blockIdx.x - t * ntiles) * kMxBN;
  uint32_t g, m0, m1;
  constexpr uint32_t kLog = kBM == 256u ? 8u : 6u;
  if (!mx_find_tile(p, t, kLog, g, m0, m1)) return;

  const uint8_t* a_base = p.xq + uint64_t(m0) * p.kp;
  const uint8_t* as_base = p.xs + uint64_t(m0) * (p.kp / 32u);
  const uint8_t* b_base = p.wq + (uint64_t(g) * p.n + n0) * (p.kp / 2u);
  const uint8_t* bs_base = p.ws + (uint64_t(g) * p.n + n0) * (p.kp / 32u);
  uint32_t a_off[kAChunks], b_off[2];
#pragma unroll
  for (uint32_t i = 0; i < kAChunks; i++)
    a_off[i] = min(i * 32u + (tid >> 3), m1 - 1u - m0) * p.kp + (tid & 7u) * 16u;
#pragma unroll
  for (uint32_t i = 0; i < 2u; i++)
    b_off[i] = min(i * 64u + (tid >> 2), p.n - 1u - n0) * (p.kp / 2u) + (tid & 3u) * 16u;
  const uint32_t as_off = min(tid, m1 - 1u - m0) * (p.kp / 32u);
  const uint32_t bs_off = min(tid & (kMxBN - 1u), p.n - 1u - n0) * (p.kp / 32u);
  u32x4v va[kAChunks], vb[2];
  uint32_t vsa, vsb;
  const auto load = [&](uint32_t step) {
#pragma unroll
    for (uint32_t i = 0; i < kAChunks; i++)
      va[i] = *reinterpret_cast<const u32x4v*>(a_base + a_off[i] + step * 128u);
#pragma unroll
    for (uint32_t i = 0; i < 2u; i++) vb[i] = *reinterpret_cast<const u32x4v*>(b_base + b_off[i] + step * 64u);
    vsa = *reinterpret_cast<const uint32_t*>(as_base + as_off + step * 4u);
    vsb = *reinterpret_cast<const uint32_t*>(bs_base + bs_off + step * 4u);
  };
  // 64-byte rows of B: chunks exclusive-ored with row / 4
  const auto b_at = [](uint32_t r, uint32_t chunk) { return r * 64u + ((chunk ^ ((r >> 2) & 3u)) << 4); };

  const uint32_t wm = (wave >> 1) * (kBM / 2u), wn = (wave & 1u) * 64u;
  v16f acc[kFM][kFN];
#pragma unroll
  for (uint32_t i = 0; i < kFM; i++)
#pragma unroll
    for (uint32_t j = 0; j < kFN; j++)
#pragma unroll
      for (int r = 0; r < 16; r++) acc[i][j][r] = 0.0f;

  const uint32_t steps = p.kp / 128u, half = lane >> 5;
  load(0u);
  for (uint32_t step = 0; step < steps; step++) {
    if (step) __syncthreads();
#pragma unroll
    for (uint32_t i = 0; i < kAChunks; i++)
      *reinterpret_cast<u32x4v*>(s_a + mx_rows_at(i * 32u + (tid >> 3), tid & 7u)) = va[i];
#pragma unroll
    for (uint32_t i = 0; i < 2u; i++)
      *reinterpret_cast<u32x4v*>(s_b + b_at(i * 64u + (tid >> 2), tid & 3u)) = vb[i];
    if (tid < kBM) s_sa[tid] = vsa;
    if (tid < kMxBN) s_sb[tid] = vsb;
    __syncthreads();
    if (step + 1u < steps) load(step + 1u);
    // Lane half h holds block 2 s + h of B's row, and of A's row the 16
    // values at 16 h and at 32 + 16 h of the 64; its scale byte is block
    // 2 s + h's.  The byte the instruction picks is the same for all lanes,
    // so the word is shifted by h first.
    uint32_t sa[kFM], sb[kFN];
#pragma unroll
    for (uint32_t i = 0; i < kFM; i++) sa[i] = s_sa[wm + i * 32u + (lane & 31u)] >> (8u * half);
#pragma unroll
    for (uint32_t j = 0; j < kFN; j++) sb[j] = s_sb[wn + j * 32u + (lane & 31u)] >> (8u * half);
#pragma unroll
    for (uint32_t s = 0; s < 2u; s++) {
      v8i fa[kFM], fb[kFN];
#pragma unroll
      for (uint32_t i = 0; i < kFM; i++) {
        const uint32_t r = wm + i * 32u + (lane & 31u);
        const v4i lo = *reinterpret_cast<const v4i*>(s_a + mx_rows_at(r, s * 4u + half));
        const v4i hi = *reinterpret_cast<const v4i*>(s_a + mx_rows_at(r, s * 4u + 2u + half));
        fa[i] = v8i{lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
      }
#pragma unroll
      for (uint32_t j = 0; j < kFN; j++) {
        const v4i q = *reinterpret_cast<const v4i*>(s_b + b_at(wn + j * 32u + (lane & 31u), s * 2u + half));
        fb[j] = v8i{q[0], q[1], q[2], q[3], 0, 0, 0, 0};
      }
#pragma unroll
      for (uint32_t i = 0; i < kFM; i++)
#pragma unroll
        for (uint32_t j = 0; j < kFN; j++) {
          if (s == 0u)
            acc[i][j] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(fa[i], fb[j], acc[i][j], 0, 4, 0, int(sa[i]), 0,
                                                                        int(sb[j]));
          else
            acc[i][j] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(fa[i], fb[j], acc[i][j], 0, 4, 2, int(sa[i]), 2,
                                                                        int(sb[j]));
        }
    }
  }
#pragma unroll
  for (uint32_t i = 0; i < kFM; i++)
#pragma unroll
    for (uint32_t j = 0; j < kFN; j++) {
      const uint32_t col = n0 + wn + j * 32u + (lane & 31u);
#pragma unroll
      for (uint32_t r = 0; r < 16u; r++) {
        const uint32_t row = m0 + wm + i * 32u + 8u * (r / 4u) + 4u * half + (r & 3u);
        if (row < m1 && col < p.n) mx_store(p, uint64_t(row) * p.ldo + col, acc[i][j][r]);
      }
    }
}

// matmul for few tokens a group: bound by reading the weights once.  A
// workgroup takes 16 weight rows of a group and all the group's tokens, 16 a
// pass; its waves take turns over the steps of 128 contraction values and
// their sums are added in wave order at the end.  A lane reads 16 bytes, one
// block of a weight row, straight into registers.
constexpr uint32_t kMxFewWaves = 8u;
template <bool kMx8>
__global__ __launch_bounds__(kMxFewWaves * 64u) void k_mx_few(MxArgs p) {
  __shared__ float s_sum[kMxFewWaves][16][16];
  const uint32_t tid = threadIdx.x, lane = tid & 63u, wave = tid >> 6;
  if (blockIdx.x == 0u && blockIdx.y == 0u) mx_report(p);
  const uint32_t g = blockIdx.y, n0 = blockIdx.x * 16u;
  uint32_t r0, r1;
  mx_rows(p, g, r0, r1);
  const uint32_t l16 = lane & 15u, kb = lane >> 4;
  const uint64_t wrow = uint64_t(g) * p.n + min(n0 + l16, p.n - 1u);
  const uint8_t* wq = p.wq + wrow * (p.kp / 2u) + kb * 16u;
  const uint8_t* ws = p.ws + wrow * (p.kp / 32u) + kb;
  const uint32_t steps = p.kp / 128u;
  for (uint32_t t0 = r0; t0 < r1; t0 += 16u) {
    const uint64_t row = min(t0 + l16, r1 - 1u);
    v4f acc = {0.0f, 0.0f, 0.0f, 0.0f};
    for (uint32_t step = wave; step < steps; step += kMxFewWaves) {
      const v4i q = *reinterpret_cast<const v4i*>(wq + step * 64u);
      const uint32_t sb = ws[step * 4u];
      u32x4v xv[4];
      if constexpr (kMx8) {
        const uint8_t* xq = p.xq + row * p.kp + step * 128u + kb * 32u;
        const u32x4v lo = *reinterpret_cast<const u32x4v*>(xq);
        const u32x4v hi = *reinterpret_cast<const u32x4v*>(xq + 16u);
        const float sx = mx_scale(p.xs[row * (p.kp / 32u) + step * 4u + kb]);
        xv[0] = mx_unit8(lo[0], lo[1], sx);
        xv[1] = mx_unit8(lo[2], lo[3], sx);
        xv[2] = mx_unit8(hi[0], hi[1], sx);
        xv[3] = mx_unit8(hi[2], hi[3], sx);
      } else {
        const uint32_t c = step * 128u + kb * 32u;
        const uint16_t* x = p.a + row * p.lda + c;
        if (step * 128u + 128u <= p.k) {
#pragma unroll
          for (int j = 0; j < 4; j++) xv[j] = *reinterpret_cast<const u32x4a2*>(x + 8 * j);
        } else {  // zeros behind the contraction's end
#pragma unroll
          for (int j = 0; j < 4; j++) {
            const uint32_t at = c + 8u * uint32_t(j);
            xv[j] = mx_part8(x + 8 * j, at < p.k ? p.k - at : 0u);
          }
        }
      }
      const float s = mx_scale(sb);
#pragma unroll
      for (int j = 0; j < 4; j++)
        acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(v8bf, xv[j]),
                                                      __builtin_bit_cast(v8bf, mx_unit4(uint32_t(q[j]), s)), acc, 0, 0,
                                                      0);
    }
#pragma unroll
    for (int r = 0; r < 4; r++) s_sum[wave][kb * 4u + r][l16] = acc[r];
    __syncthreads();
    if (tid < 256u) {
      const uint32_t tr = tid >> 4, col = n0 + (tid & 15u);
      float v = 0.0f;
#pragma unroll
      for (uint32_t w = 0; w < kMxFewWaves; w++) v += s_sum[w][tr][tid & 15u];
      if (t0 + tr < r1 && col < p.n) mx_store(p, uint64_t(t0 + tr) * p.ldo + col, v);
    }
    __syncthreads();
  }
}

__global__ void k_mx_status(MxArgs p) { mx_report(p); }

ciera_status mx_matrix(const void* d_m, uint64_t rows, uint64_t cols, uint64_t ld, uint32_t align) {
  if (rows > kMxMaxRows || cols > kMxMaxCols || ld < cols || ld > kMxMaxLd) return CIERA_ERR_ARG;
  if (rows && cols && (!d_m || (reinterpret_cast<uintptr_t>(d_m) & (align - 1u)) != 0u)) return CIERA_ERR_ARG;
  return CIERA_OK;
}

ciera_status mx_encoded(const void* d_q, uint64_t q_bytes, uint64_t rows, uint64_t cols, uint32_t bits,
                        ciera_status small) {
  if (rows > kMxMaxRows || cols > kMxMaxCols) return CIERA_ERR_ARG;
  const uint64_t need = mx_size(rows, cols, bits);
  if (need && (!d_q || !aligned16(d_q))) return CIERA_ERR_ARG;
  return q_bytes < need ? small : CIERA_OK;
}

template <int kBits>
ciera_status mx_encode_impl(const void* d_x, uint64_t rows, uint64_t cols, uint64_t ld, void* d_q, uint64_t q_bytes,
                            hipStream_t stream) {
  ciera_status st = mx_matrix(d_x, rows, cols, ld, 2u);
  if (st == CIERA_OK) st = mx_encoded(d_q, q_bytes, rows, cols, kBits, CIERA_ERR_CAPACITY);
  if (st != CIERA_OK || !rows || !cols) return st;
  const uint64_t at = mx_scales_at(rows, cols, kBits);
  const uint64_t units = rows * (mx_pitch(cols) / 8u);
  const uint64_t grid = cdiv(units, kMxThreads * kMxUnits);
  if (grid > 0x7FFFFFFFu) return CIERA_ERR_ARG;
  uint8_t* q = static_cast<uint8_t*>(d_q);
  (void)hipGetLastError();
  launch(k_mx_encode<kBits>, dim3(uint32_t(grid)), dim3(kMxThreads), stream, static_cast<const uint16_t*>(d_x), rows,
         uint32_t(cols), ld, q, q + at, uint32_t(at - rows * mx_pitch(cols) * kBits / 8u));
  return launch_status();
}

template <int kBits>
ciera_status mx_decode_impl(const void* d_q, uint64_t q_bytes, uint64_t rows, uint64_t cols, void* d_y, uint64_t ld,
                            hipStream_t stream) {
  ciera_status st = mx_matrix(d_y, rows, cols, ld, 2u);
  if (st == CIERA_OK) st = mx_encoded(d_q, q_bytes, rows, cols, kBits, CIERA_ERR_FORMAT);
  if (st != CIERA_OK || !rows || !cols) return st;
  const uint64_t grid = cdiv(rows * cdiv(cols, 8u), kMxThreads * kMxUnits);
  if (grid > 0x7FFFFFFFu) return CIERA_ERR_ARG;
  const uint8_t* q = static_cast<const uint8_t*>(d_q);
  (void)hipGetLastError();
  launch(k_mx_decode<kBits>, dim3(uint32_t(grid)), dim3(kMxThreads), stream, q, q + mx_scales_at(rows, cols, kBits),
         rows, uint32_t(cols), static_cast<uint16_t*>(d_y), ld);
  return launch_status();
}

uint64_t mx_ws_size(uint64_t tokens, uint64_t n, uint64_t k, uint64_t groups) {
  if (tokens > kMxMaxRows - 1u || !n || !k || n > kMxMaxCols || k > kMxMaxCols || !groups || groups > kMxMaxGroups ||
      groups * n > kMxMaxRows)
    return 0u;
  return kMxWsHead;
}

// The checks every product makes, and the arguments they share.
ciera_status mx_product(MxArgs& p, const void* d_w, uint64_t w_bytes, void* d_out, uint64_t ldo, uint64_t out_cols,
                        uint32_t out_f32, uint64_t tokens, uint64_t n, uint64_t k, uint32_t groups,
                        const int64_t* d_offsets, void* d_ws, uint64_t ws_bytes) {
  const uint64_t need = mx_ws_size(tokens, n, k, groups);
  if (!need || out_f32 > 1u) return CIERA_ERR_ARG;
  if (!d_ws || !aligned16(d_ws)) return CIERA_ERR_ARG;
  if (groups > 1u && !d_offsets) return CIERA_ERR_ARG;
  if ((reinterpret_cast<uintptr_t>(d_offsets) & 7u) != 0u) return CIERA_ERR_ARG;
  if (out_cols) {
    const ciera_status st = mx_matrix(d_out, tokens, out_cols, ldo, out_f32 ? 4u : 2u);
    if (st != CIERA_OK) return st;
  }
  if (d_w || w_bytes != ~0ull) {
    const ciera_status st = mx_encoded(d_w, w_bytes, groups * n, k, 4u, CIERA_ERR_FORMAT);
    if (st != CIERA_OK) return st;
  }
  if (ws_bytes < need) return CIERA_ERR_WORKSPACE;
  p.wq = static_cast<const uint8_t*>(d_w);
  p.ws = p.wq + mx_scales_at(groups * n, k, 4u);
  p.out = d_out;
  p.ldo = ldo;
  p.offsets = d_offsets;
  p.ctrl = static_cast<Ctrl*>(d_ws);
  p.status = reinterpret_cast<uint32_t*>(static_cast<uint8_t*>(d_ws) + sizeof(Ctrl));
  p.tokens = uint32_t(tokens);
  p.n = uint32_t(n);
  p.k = uint32_t(k);
  p.kp = uint32_t(mx_pitch(k));
  p.groups = groups;
  p.out_f32 = out_f32;
  return CIERA_OK;
}

// Token tiles of bm rows that the groups can need between them.
uint64_t mx_token_tiles(const MxArgs& p, uint32_t bm) {
  if (!p.offsets) return cdiv(p.tokens, bm);
  return p.tokens / bm + (p.groups < p.tokens ? p.groups : p.tokens);
}

// Few rows a group: the weights' read dominates (k_mx_few).  Otherwise tiles
// of 256 rows, or of 64 where a group's rows would leave most of 256 empty.
uint32_t mx_rows_per_tile(const MxArgs& p) { return p.tokens / p.groups > 96u ? 256u : 64u; }

template <int kOp>
ciera_status mx_gemm(const MxArgs& p, hipStream_t stream) {
  const uint32_t bm = kOp == kMxWgrad ? 256u : mx_rows_per_tile(p);
  const uint64_t ntiles = cdiv(kOp == kMxMatmul || kOp == kMxMatmul8 ? p.n : p.k, kMxBN);
  const uint64_t mtiles = kOp == kMxWgrad ? cdiv(p.n, bm) * p.groups : mx_token_tiles(p, bm);
  const uint64_t grid = ntiles * mtiles;
  if (grid > 0x7FFFFFFFu) return CIERA_ERR_ARG;
  if (bm == 256u) launch(k_mx_gemm<kOp, 256u>, dim3(uint32_t(grid)), dim3(kMxThreads), stream, p);
  else if constexpr (kOp != kMxWgrad) launch(k_mx_gemm<kOp, 64u>, dim3(uint32_t(grid)), dim3(kMxThreads), stream, p);
  return launch_status();
}

template <bool kMx8>
ciera_status mx_matmul_impl(MxArgs& p, hipStream_t stream) {
  (void)hipGetLastError();
  if (p.tokens == 0u) {
    launch(k_mx_status, dim3(1), dim3(64), stream, p);
    return launch_status();
  }
  if (p.tokens <= 32u * uint64_t(p.groups)) {
    launch(k_mx_few<kMx8>, dim3(uint32_t(cdiv(p.n, 16u)), p.groups), dim3(kMxFewWaves * 64u), stream, p);
    return launch_status();
  }
  if constexpr (kMx8) {
    if (p.out_f32) return mx_gemm<kMxMatmul8>(p, stream);
    const uint32_t bm = mx_rows_per_tile(p);
    const uint64_t grid = cdiv(p.n, kMxBN) * mx_token_tiles(p, bm);
    if (grid > 0x7FFFFFFFu) return CIERA_ERR_ARG;
    if (bm == 256u) launch(k_mx_gemm8<256u>, dim3(uint32_t(grid)), dim3(kMxThreads), stream, p);
    else launch(k_mx_gemm8<64u>, dim3(uint32_t(grid)), dim3(kMxThreads), stream, p);
    return launch_status();
  } else {
    return mx_gemm<kMxMatmul>(p, stream);
  }
}

}  // namespace

extern "C" {

uint64_t mx8_encoded_size(uint64_t rows, uint64_t cols) {
  return rows > kMxMaxRows || cols > kMxMaxCols ? 0u : mx_size(rows, cols, 8u);
}
uint64_t mx4_encoded_size(uint64_t rows, uint64_t cols) {
  return rows > kMxMaxRows || cols > kMxMaxCols ? 0u : mx_size(rows, cols, 4u);
}
uint64_t mx_workspace_size(uint64_t tokens, uint64_t n, uint64_t k, uint32_t groups) {
  return mx_ws_size(tokens, n, k, groups);
}

ciera_status mx8_encode(const void* d_x, uint64_t rows, uint64_t cols, uint64_t ld, void* d_q, uint64_t q_bytes,
                        hipStream_t stream) {
  return mx_encode_impl<8>(d_x, rows, cols, ld, d_q, q_bytes, stream);
}
ciera_status mx4_encode(const void* d_x, uint64_t rows, uint64_t cols, uint64_t ld, void* d_q, uint64_t q_bytes,
                        hipStream_t stream) {
  return mx_encode_impl<4>(d_x, rows, cols, ld, d_q, q_bytes, stream);
}
ciera_status mx8_decode(const void* d_q, uint64_t q_bytes, uint64_t rows, uint64_t cols, void* d_y, uint64_t ld,
                        hipStream_t stream) {
  return mx_decode_impl<8>(d_q, q_bytes, rows, cols, d_y, ld, stream);
}
ciera_status mx4_decode(const void* d_q, uint64_t q_bytes, uint64_t rows, uint64_t cols, void* d_y, uint64_t ld,
                        hipStream_t stream) {
  return mx_decode_impl<4>(d_q, q_bytes, rows, cols, d_y, ld, stream);
}

ciera_status mx4_matmul(const void* d_x, uint64_t ldx, const void* d_w, uint64_t w_bytes, void* d_y, uint64_t ldy,
                        uint32_t y_f32, uint64_t tokens, uint64_t n, uint64_t k, uint32_t groups,
                        const int64_t* d_offsets, void* d_ws, uint64_t ws_bytes, hipStream_t stream) {
  MxArgs p{};
  ciera_status st = mx_product(p, d_w, w_bytes, d_y, ldy, n, y_f32, tokens, n, k, groups, d_offsets, d_ws, ws_bytes);
  if (st == CIERA_OK) st = mx_matrix(d_x, tokens, k, ldx, 2u);
  if (st != CIERA_OK) return st;
  p.a = static_cast<const uint16_t*>(d_x);
  p.lda = ldx;
  return mx_matmul_impl<false>(p, stream);
}

ciera_status mx4_matmul_mx8(const void* d_xq, uint64_t xq_bytes, const void* d_w, uint64_t w_bytes, void* d_y,
                            uint64_t ldy, uint32_t y_f32, uint64_t tokens, uint64_t n, uint64_t k, uint32_t groups,
                            const int64_t* d_offsets, void* d_ws, uint64_t ws_bytes, hipStream_t stream) {
  MxArgs p{};
  ciera_status st = mx_product(p, d_w, w_bytes, d_y, ldy, n, y_f32, tokens, n, k, groups, d_offsets, d_ws, ws_bytes);
  if (st == CIERA_OK) st = mx_encoded(d_xq, xq_bytes, tokens, k, 8u, CIERA_ERR_FORMAT);
  if (st != CIERA_OK) return st;
  p.xq = static_cast<const uint8_t*>(d_xq);
  p.xs = p.xq + mx_scales_at(tokens, k, 8u);
  return mx_matmul_impl<true>(p, stream);
}

ciera_status mx4_matmul_dx(const void* d_dy, uint64_t lddy, const void* d_w, uint64_t w_bytes, void* d_dx,
                           uint64_t lddx, uint32_t dx_f32, uint64_t tokens, uint64_t n, uint64_t k, uint32_t groups,
                           const int64_t* d_offsets, void* d_ws, uint64_t ws_bytes, hipStream_t stream) {
  MxArgs p{};
  ciera_status st = mx_product(p, d_w, w_bytes, d_dx, lddx, k, dx_f32, tokens, n, k, groups, d_offsets, d_ws, ws_bytes);
  if (st == CIERA_OK) st = mx_matrix(d_dy, tokens, n, lddy, 2u);
  if (st != CIERA_OK) return st;
  p.a = static_cast<const uint16_t*>(d_dy);
  p.lda = lddy;
  (void)hipGetLastError();
  if (p.tokens == 0u) {
    launch(k_mx_status, dim3(1), dim3(64), stream, p);
    return launch_status();
  }
  return mx_gemm<kMxDx>(p, stream);
}

ciera_status mx8_wgrad(const void* d_dy, uint64_t lddy, const void* d_xq, uint64_t xq_bytes, void* d_dw,
                       uint32_t dw_f32, uint32_t accumulate, uint64_t tokens, uint64_t n, uint64_t k, uint32_t groups,
                       const int64_t* d_offsets, void* d_ws, uint64_t ws_bytes, hipStream_t stream) {
  MxArgs p{};
  ciera_status st =
      mx_product(p, nullptr, ~0ull, d_dw, 0u, 0u, dw_f32, tokens, n, k, groups, d_offsets, d_ws, ws_bytes);
  if (st == CIERA_OK) st = mx_matrix(d_dy, tokens, n, lddy, 2u);
  if (st == CIERA_OK) st = mx_encoded(d_xq, xq_bytes, tokens, k, 8u, CIERA_ERR_FORMAT);
  if (st == CIERA_OK && (accumulate > 1u || !d_dw || (reinterpret_cast<uintptr_t>(d_dw) & (dw_f32 ? 3u : 1u)) != 0u))
    st = CIERA_ERR_ARG;
  if (st != CIERA_OK) return st;
  p.a = static_cast<const uint16_t*>(d_dy);
  p.lda = lddy;
  p.xq = static_cast<const uint8_t*>(d_xq);
  p.xs = p.xq + mx_scales_at(tokens, k, 8u);
  p.accumulate = accumulate;
  (void)hipGetLastError();
  return mx_gemm<kMxWgrad>(p, stream);
}

}  // extern "C"
