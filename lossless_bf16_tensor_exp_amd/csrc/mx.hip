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
#include "mx_rules.h"

namespace {

typedef int v2i __attribute__((ext_vector_type(2)));
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
constexpr uint64_t kMxMaxLd = 1ull << 22;

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
// workgroup's width apart and issues all their loads before it uses one (one,
// two, four and eight units: 72, 70, 75 and 78 us for the mx8 encode of 65,536
// x 2,048).  The BF16 side streams past the last-level cache, which so keeps
// the encoded side for its reader: encode and decode together 125 us instead
// of 145 (mx8) and 106 instead of 130 (mx4), 6.5 and 6.4 TB/s; of 16,384 x
// 2,048 in mx8 36 us, 5.6 TB/s.
// ---------------------------------------------------------------------------
struct MxUnitAt {
  uint64_t row;
  uint32_t col;
};
// Unit `u` of this thread: row and first column (upr units per row).
__device__ __forceinline__ MxUnitAt mx_unit_at(uint64_t first_row, uint32_t first_unit, uint32_t u, uint32_t upr) {
  const uint32_t at = first_unit + u * kMxThreads + threadIdx.x;
  // first_unit is below upr: where a row is as long as a workgroup's units, at
  // most one row is passed
  const uint32_t dr = upr >= kMxThreads * kMxUnits ? uint32_t(at >= upr) : at / upr;
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
    v[u] = cols >= 8u ? u32x4v(__builtin_nontemporal_load(reinterpret_cast<const u32x4a2*>(src))) : u32x4v{0u, 0u, 0u, 0u};
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
    m = max(m, uint32_t(__builtin_amdgcn_mov_dpp(int(m), 0xB1, 0xF, 0xF, true)));  // lane ^ 1
    m = max(m, uint32_t(__builtin_amdgcn_mov_dpp(int(m), 0x4E, 0xF, 0xF, true)));  // lane ^ 2
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
      __builtin_nontemporal_store(v, reinterpret_cast<u32x4a2*>(dst));
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
  uint32_t parts;  // dx, wgrad: the contraction in this many parts, each with an output of its own
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

// Where this workgroup's tile is among the real ones.  Token tiles of 1 << lbm
// rows are numbered group by group; every wave counts them for itself, 64
// groups a step by a lane scan.  `ntiles` column tiles belong to each.  The
// grid is as large as any offsets can need; the workgroups past the real tiles
// end.  Workgroups go to the eight XCDs in turn, so tiles are dealt out in
// eight runs: an XCD's L2 then holds the weights of its own few groups and the
// rows they share.
struct MxTile {
  uint32_t g, row0, row1, col;
};
__device__ __forceinline__ uint32_t mx_xcd_run(uint32_t block, uint32_t total) {
  const uint32_t xcd = block & 7u, per = total >> 3, rem = total & 7u;
  return xcd * per + min(xcd, rem) + (block >> 3);
}
__device__ __forceinline__ uint32_t mx_scan(uint32_t v) {
  const uint32_t lane = threadIdx.x & 63u;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const uint32_t up = uint32_t(__shfl_up(int(v), d));
    if (lane >= uint32_t(d)) v += up;
  }
  return v;
}
__device__ __forceinline__ uint32_t mx_first(uint32_t v) { return uint32_t(__builtin_amdgcn_readfirstlane(int(v))); }
__device__ __forceinline__ bool mx_find_tile(const MxArgs& p, uint32_t lbm, uint32_t ntiles, MxTile& t) {
  const uint32_t lane = threadIdx.x & 63u, up = (1u << lbm) - 1u;
  if (!p.offsets) {
    const uint32_t at = mx_xcd_run(blockIdx.x, gridDim.x);
    t.g = 0u;
    t.row0 = (at / ntiles) << lbm;
    t.row1 = p.tokens;
    t.col = at % ntiles;
    return true;
  }
  uint32_t r0 = 0u, r1 = 0u, sum = 0u, total = 0u;
  for (uint32_t c = 0; c < p.groups; c += 64u) {
    r0 = r1 = 0u;
    if (c + lane < p.groups) mx_rows(p, c + lane, r0, r1);
    sum = mx_scan((r1 - r0 + up) >> lbm);
    total += uint32_t(__builtin_amdgcn_readlane(int(sum), 63));
  }
  if (blockIdx.x >= total * ntiles) return false;
  const uint32_t at = mx_xcd_run(blockIdx.x, total * ntiles);
  const uint32_t tile = at / ntiles;
  t.col = at - tile * ntiles;
  uint32_t before = 0u;
  for (uint32_t c = 0; c < p.groups; c += 64u) {
    if (p.groups > 64u) {
      r0 = r1 = 0u;
      if (c + lane < p.groups) mx_rows(p, c + lane, r0, r1);
      sum = mx_scan((r1 - r0 + up) >> lbm);
    }
    const uint64_t past = __ballot(before + sum > tile);
    if (past) {
      const int l = __ffsll((unsigned long long)past) - 1;
      const uint32_t a = uint32_t(__builtin_amdgcn_readlane(int(r0), l));
      const uint32_t b = uint32_t(__builtin_amdgcn_readlane(int(r1), l));
      const uint32_t end = before + uint32_t(__builtin_amdgcn_readlane(int(sum), l));
      t.g = c + uint32_t(l);
      t.row0 = a + ((tile - (end - ((b - a + up) >> lbm))) << lbm);
      t.row1 = b;
      return true;
    }
    before += uint32_t(__builtin_amdgcn_readlane(int(sum), 63));
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

// Stores of 4 FP32 or 4 / 8 BF16 values at any address of the type.
typedef float v4fa4 __attribute__((ext_vector_type(4), aligned(4)));
typedef uint32_t u32x2a2 __attribute__((ext_vector_type(2), aligned(2)));

__device__ __forceinline__ uint32_t mx_bf16x2(float lo, float hi) {
  return uint32_t(mx_bf16(lo)) | uint32_t(mx_bf16(hi)) << 16;
}

__device__ __forceinline__ void mx_store4(const MxArgs& p, uint64_t at, v4f x) {
  if (p.out_f32) {
    v4fa4* o = reinterpret_cast<v4fa4*>(static_cast<float*>(p.out) + at);
    if (p.accumulate) x += v4f(*o);
    *o = x;
  } else {
    u32x2a2* o = reinterpret_cast<u32x2a2*>(static_cast<uint16_t*>(p.out) + at);
    if (p.accumulate) {
      const u32x2v w = *o;
      x[0] += mx_f32(uint16_t(w[0]));
      x[1] += mx_f32(uint16_t(w[0] >> 16));
      x[2] += mx_f32(uint16_t(w[1]));
      x[3] += mx_f32(uint16_t(w[1] >> 16));
    }
    *o = u32x2v{mx_bf16x2(x[0], x[1]), mx_bf16x2(x[2], x[3])};
  }
}

// One 32 x 32 fragment of sums to the output.  The matrix instructions take
// the output's columns as their rows, so a lane holds one output row, lane %
// 32, and its register r column 8 (r / 4) + 4 (lane / 32) + r % 4: four
// neighbours at a time.  In BF16 the lane halves first exchange every other
// four, which leaves each with eight neighbours, 16 bytes.
__device__ __forceinline__ void mx_store_frag(const MxArgs& p, bool row_ok, uint64_t row_at, uint32_t col0,
                                              uint32_t cols, const v16f& v) {
  const uint32_t half = (threadIdx.x >> 5) & 1u;
  const bool whole = col0 + 32u <= cols;
  if (whole && !p.out_f32 && !p.accumulate) {
    uint16_t* o = static_cast<uint16_t*>(p.out) + row_at + col0 + 8u * half;
#pragma unroll
    for (int q = 0; q < 4; q += 2) {
      u32x4v w;
#pragma unroll
      for (int i = 0; i < 2; i++) {
        const auto x = __builtin_amdgcn_permlane32_swap(mx_bf16x2(v[4 * q + 2 * i], v[4 * q + 2 * i + 1]),
                                                        mx_bf16x2(v[4 * q + 4 + 2 * i], v[4 * q + 5 + 2 * i]), false, false);
        w[i] = x[0];
        w[2 + i] = x[1];
      }
      if (row_ok) *reinterpret_cast<u32x4a2*>(o + 8 * q) = w;
    }
    return;
  }
  if (!row_ok) return;
#pragma unroll
  for (int q = 0; q < 4; q++) {
    const uint32_t col = col0 + 8u * uint32_t(q) + 4u * half;
    if (col + 4u <= cols) {
      mx_store4(p, row_at + col, v4f{v[4 * q], v[4 * q + 1], v[4 * q + 2], v[4 * q + 3]});
    } else {
#pragma unroll
      for (uint32_t i = 0; i < 3u; i++)
        if (col + i < cols) mx_store(p, row_at + col + i, v[4 * q + int(i)]);
    }
  }
}

// The sums of two fragments whose columns alternate, col0 + 2 c and col0 + 2 c
// + 1: a lane's four neighbours of both are eight columns in a row.
__device__ __forceinline__ void mx_store_pair(const MxArgs& p, uint64_t row_at, uint32_t col0, uint32_t cols,
                                              const v16f& even, const v16f& odd) {
#pragma unroll
  for (int q = 0; q < 16; q += 4) {
    const uint32_t col = col0 + 4u * uint32_t(q) + 8u * ((threadIdx.x >> 5) & 1u);
    const v4f lo{even[q], odd[q], even[q + 1], odd[q + 1]}, hi{even[q + 2], odd[q + 2], even[q + 3], odd[q + 3]};
    const uint64_t at = row_at + col;
    if (col + 8u <= cols) {
      if (p.out_f32 || p.accumulate) {
        mx_store4(p, at, lo);
        mx_store4(p, at + 4u, hi);
      } else {
        *reinterpret_cast<u32x4a2*>(static_cast<uint16_t*>(p.out) + at) =
            u32x4v{mx_bf16x2(lo[0], lo[1]), mx_bf16x2(lo[2], lo[3]), mx_bf16x2(hi[0], hi[1]), mx_bf16x2(hi[2], hi[3])};
      }
    } else {
#pragma unroll
      for (uint32_t i = 0; i < 7u; i++)
        if (col + i < cols) mx_store(p, at + i, i < 4u ? lo[i] : hi[i - 4u]);
    }
  }
}

// Eight contraction rows of two neighbouring columns as BF16.  q holds both
// columns' values of row t in byte t (mx4) or 16-bit half t (mx8), w the rows'
// scale bytes, each in a word that `turn` rotates to bring it to bit 23.  The
// conversion takes its scale from the exponent bits alone and converts a row's
// two values together; neighbouring rows are then paired column by column.
template <int kBits>
__device__ __forceinline__ void mx_pairs(const uint32_t (&q)[kBits / 2], u32x4v w0, u32x4v w1, uint32_t turn,
                                         v8bf& even, v8bf& odd) {
  u32x4v e, o;
#pragma unroll
  for (int t = 0; t < 8; t += 2) {
    uint32_t v[2];
#pragma unroll
    for (int i = 0; i < 2; i++) {
      const uint32_t w = t < 4 ? w0[t + i] : w1[t + i - 4];
      const float s = __uint_as_float(__builtin_amdgcn_alignbit(w, w, turn));
      v2bf b;
      if constexpr (kBits == 8) {
        b = i ? __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(q[t / 2], s, true)
              : __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(q[t / 2], s, false);
      } else {
        b = t % 4 ? (i ? __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(q[t / 4], s, 3)
                       : __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(q[t / 4], s, 2))
                  : (i ? __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(q[t / 4], s, 1)
                       : __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(q[t / 4], s, 0));
      }
      v[i] = __builtin_bit_cast(uint32_t, b);
    }
    e[t / 2] = __builtin_amdgcn_perm(v[1], v[0], 0x05040100u);
    o[t / 2] = __builtin_amdgcn_perm(v[1], v[0], 0x07060302u);
  }
  even = __builtin_bit_cast(v8bf, e);
  odd = __builtin_bit_cast(v8bf, o);
}

// Loads from global memory straight into LDS: lane i's 16 (or 4) bytes at
// base + off land at lds + 16 i (4 i).  No register holds them, so they stay
// in flight over whole steps; mx_fence counts them.  m0 is named as written, so
// that no use of it by the compiler is torn apart; the warning that it is a
// reserved register says that it may not be kept, which is meant.
#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"
__device__ __forceinline__ void mx_dma16(uint32_t off, const void* base, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, %1"
               :: "v"(off), "s"(base), "s"(lds) : "memory", "m0");
}
__device__ __forceinline__ void mx_dma4(uint32_t off, const void* base, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\tglobal_load_lds_dword %0, %1"
               :: "v"(off), "s"(base), "s"(lds) : "memory", "m0");
}
#pragma clang diagnostic pop
// All but this wave's last kLeft loads have landed, its LDS reads and writes
// are done, and so are every other wave's.
template <int kLeft>
__device__ __forceinline__ void mx_fence() {
  asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" :: "n"(kLeft) : "memory");
}
__device__ __forceinline__ uint32_t mx_lds(const void* at) {
  return uint32_t(uintptr_t((__attribute__((address_space(3))) const void*)at));
}

// Staged tiles.  A row of R bytes is kept as 16-byte chunks; chunk c of row r
// sits at c ^ mx_turn<R>(r), so that lanes which read (or write) one chunk of
// 16 consecutive rows touch all 64 banks once.  The loads above apply it by
// choosing which chunk a lane fetches.  Two kinds of reads go without: W's rows
// of 32 bytes in the matmuls, whose chunks of 16 rows lie in half the banks
// (turned by r / 8: no change in time), and the scales, 16 bytes a row, whose
// words of 32 rows lie in 16 banks.  They are all of the conflicts that the
// counters show there (a third to a half of the LDS's busy cycles, which are 22
// to 34 % of the time; none with both kinds of reads made free of them).
template <uint32_t kRow>
__device__ __forceinline__ uint32_t mx_turn(uint32_t r) {
  static_assert(kRow == 64u || kRow == 128u, "4 or 8 chunks");
  return (r / (256u / kRow)) & (kRow / 16u - 1u);
}
template <uint32_t kRow>
__device__ __forceinline__ uint32_t mx_at(uint32_t r, uint32_t chunk) {
  return r * kRow + ((chunk ^ mx_turn<kRow>(r)) << 4);
}
// A tile to be read transposed: contraction row c of kRow bytes.  The 64-byte
// piece is exclusive-ored with c, so the four rows a transposing read gathers
// differ in bank, and the chunk within it with c / 4, for the writers.
__device__ __forceinline__ uint32_t mx_turn_cols(uint32_t c) { return ((c & 3u) << 2) ^ ((c >> 2) & 3u); }

// The mx operand of dx and wgrad, read transposed two columns at a time: what
// 32 lanes gather, 8 rows x 32 bytes (dx) or 4 rows x 64 bytes (wgrad), covers
// the 64 banks once.
template <int kBits, uint32_t kRow>
__device__ __forceinline__ uint32_t mx_turn_pairs(uint32_t r) {
  static_assert(kRow == 128u || (kRow == 64u && kBits == 4), "tiles of 128 or 256 columns, mx8 of 128");
  if (kBits == 8) return (r >> 1 & 1u) << 2;
  return kRow == 128u ? (r >> 1 & 3u) << 1 : (r >> 2 & 1u) << 1;
}

// Eight contraction values c0 .. c0 + 7 (c0 a multiple of 8) of one column per
// lane: two reads that each transpose 4 rows x 16 columns within 16 lanes.
// at0, at1: this lane's addresses for c0 = 0 and its two reads.
__device__ __forceinline__ v8bf mx_read_cols(const uint8_t* at0, const uint8_t* at1) {
  typedef __attribute__((address_space(3))) v4s lds_v4s;
  const v4s lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4s*)at0);
  const v4s hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4s*)at1);
  const v4s both[2] = {lo, hi};
  return __builtin_bit_cast(v8bf, both);
}

// The products on BF16 matrix instructions: tiles of kBM x kBN outputs, kWM x
// kWN waves, kBC contraction values a step, a ring of kStages steps in LDS
// filled by loads that need no registers, one barrier a step.  A wave keeps
// its 32 x 32 sums in registers.
//   matmul  M tokens, N weight rows, contraction k: both operands run along
//           the contraction.  W stays in 4 bits in LDS: a lane reads a whole
//           block of 32 of its row (16 bytes) and makes BF16 of it next to the
//           matrix instructions, a quarter of the LDS traffic of a BF16 tile.
//           Lane half h so holds values 32 h .. 32 h + 31 of the step, eight
//           per instruction; x is read in the same order.  x in mx8 likewise.
//   dx      M tokens, N k, contraction n: W's rows are contraction rows, so it
//           is read transposed, in 4 bits; its scales differ from row to row,
//           and a lane converts two neighbouring columns of a row together
//           (mx_pairs: 1.5 instructions a value).  dy is read like x.
//   wgrad   M n, N k, contraction the group's tokens: the same for x in 8
//           bits, and dy is read transposed too.
// A BF16 copy of the tile in LDS, made a step ahead, was slower (dx of 4,000
// rows in 64 groups: 52 against 32 us): 16-byte LDS writes reach 65 B a clock.
// What bounds them: the matrix instructions' 1.83 PFLOP/s at the clock that
// their power leaves, then what a tile cannot hide (dx of 32,768 rows in one
// group, n = k = 2,048: 258 us, 1.07 PFLOP/s; without its loads 25, conversions
// 28, stores 20 us less).  Measured at n = 1,024, k = 2,048, 64 groups of 512
// rows on average: dx 156 us, wgrad 205 us (268 MB of results; 128 x 128, 128 x
// 256 and 256 x 256 tiles within 5 %); matmul of 4,001 x 2,048 x 2,048: 35 us.
template <int kOp, uint32_t kBM, uint32_t kBN, uint32_t kBC, uint32_t kWM, uint32_t kWN, uint32_t kStages, uint32_t kPerCu>
__global__ __launch_bounds__(kWM * kWN * 64u, kWM* kWN / 4u * kPerCu) void k_mx_gemm(MxArgs p) {
  constexpr bool kRowsB = kOp == kMxMatmul || kOp == kMxMatmul8;  // B runs along the contraction
  constexpr uint32_t kW = kWM * kWN;
  constexpr uint32_t kABytes = kBM * kBC * (kOp == kMxMatmul8 ? 1u : 2u);       // of a step's A
  constexpr uint32_t kARow = kOp == kMxWgrad ? kBM * 2u : kABytes / kBM;
  constexpr uint32_t kAPer = kARow / 16u;
  constexpr uint32_t kBBits = kOp == kMxWgrad ? 8u : 4u;
  constexpr uint32_t kRawBytes = kBN * kBC * kBBits / 8u;                       // of a step's mx operand B
  constexpr uint32_t kRawRow = kRawBytes / (kRowsB ? kBN : kBC);
  constexpr uint32_t kRawPer = kRawRow / 16u;
  constexpr uint32_t kScaleWords = kRowsB ? 0u : (kBC * (kBN / 128u) + 63u) / 64u * 64u;  // four scale bytes each, whole waves
  constexpr uint32_t kStage = kABytes + kRawBytes + 4u * kScaleWords;
  // matmul: 16 scale bytes of every row at a time, eight steps' worth, twice
  constexpr uint32_t kScaleRows = kRowsB ? kBN + (kOp == kMxMatmul8 ? kBM : 0u) : 0u;
  constexpr uint32_t kFM = kBM / kWM / 32u, kFN = kBN / kWN / 32u;              // 32 x 32 sums of a wave
  constexpr uint32_t kSub = kBC / 16u;                                          // matrix instructions along a step
  constexpr uint32_t kALoads = kABytes / 1024u, kRawLoads = kRawBytes / 1024u;  // of all waves; fewer than waves: some repeat
  constexpr uint32_t kDmaA = kALoads < kW ? 1u : kALoads / kW;                  // per wave and step
  constexpr uint32_t kDmaRaw = kRawLoads < kW ? 1u : kRawLoads / kW;
  constexpr uint32_t kDma = kDmaA + kDmaRaw;
  static_assert(kALoads * 1024u == kABytes && (kALoads < kW ? kW % kALoads == 0u : kALoads % kW == 0u), "whole loads");
  static_assert(kRawLoads * 1024u == kRawBytes && (kRawLoads < kW ? kW % kRawLoads == 0u : kRawLoads % kW == 0u), "whole loads");
  static_assert(kScaleWords <= 64u * kW && kScaleRows % 64u == 0u, "whole waves");
  static_assert(!kRowsB || kBC == 64u, "a lane half takes a block of 32");
  static_assert(kRowsB || (kBN / kWN % 64u == 0u && (kBN / kWN <= 128u)), "pairs of columns, one scale word a row");
  __shared__ __attribute__((aligned(256))) uint8_t lds[kStages * kStage + 32u * kScaleRows];
  const uint32_t tid = threadIdx.x, lane = tid & 63u, half = lane >> 5;
  const uint32_t wave = mx_first(tid >> 6);
  if (blockIdx.x == 0u) mx_report(p);

  // where the tile is: its group, its output rows m0 .. m1 - 1 and columns
  uint32_t g, m0, m1, n0, c1;
  const uint32_t cols = kRowsB ? p.n : p.k;
  const uint32_t ntiles = (cols + kBN - 1u) / kBN;
  uint32_t r0 = 0u, part = 0u;  // first contraction row, and which part of them (wgrad; dx: of n)
  if constexpr (kOp == kMxWgrad) {
    const uint32_t mtiles = (p.n + kBM - 1u) / kBM;
    const uint32_t all = mtiles * ntiles;  // of a group's part
    uint32_t gp, t;
    if (p.groups > 1u) {
      // a tile takes as long as its group has rows, so each XCD takes an
      // eighth of every group's tiles, the odd ones in turn (64 groups of 512
      // rows on average: 204 us, whole groups an XCD 219)
      const uint32_t per = (all + 7u) / 8u, at = blockIdx.x >> 3;
      gp = at / per;
      t = ((blockIdx.x + gp) & 7u) * per + at % per;
      if (t >= all) return;
    } else {
      const uint32_t at = mx_xcd_run(blockIdx.x, gridDim.x);
      gp = at / all;
      t = at - gp * all;
    }
    part = gp / p.groups;
    g = gp - part * p.groups;
    m0 = t / ntiles * kBM;
    n0 = (t % ntiles) * kBN;
    m1 = p.n;
    uint32_t a, b;
    mx_rows(p, g, a, b);
    const uint32_t each = (b - a + p.parts - 1u) / p.parts;
    const uint32_t from = min(part * each, b - a);
    r0 = mx_first(a + from);
    c1 = mx_first(min(each, b - a - from));
  } else {
    MxTile t;
    if (!mx_find_tile(p, kBM == 128u ? 7u : kBM == 64u ? 6u : 5u, ntiles, t)) return;
    g = t.g;
    m0 = t.row0;
    m1 = t.row1;
    n0 = t.col * kBN;
    c1 = kRowsB ? p.k : p.n;
    if constexpr (kOp == kMxDx) {
      part = blockIdx.y;
      const uint32_t each = (c1 + p.parts * kBC - 1u) / (p.parts * kBC) * kBC;
      r0 = min(part * each, c1);
      c1 = min(each, c1 - r0);
    }
  }
  const uint32_t steps = (c1 + kBC - 1u) / kBC;
  const uint32_t lds0 = mx_lds(lds);

  // A's loads.  Lanes fetch 16-byte chunks at these offsets from the tile's
  // first row (wgrad: from the step's first); rows and columns past the
  // operand's end are fetched from its last (their sums are not stored).
  // Where rows are not 16-byte aligned, and where the contraction ends inside
  // a step, fill_a goes through registers instead.
  const bool wide = kOp == kMxMatmul8 || ((reinterpret_cast<uintptr_t>(p.a) & 15u) == 0u && (p.lda & 7u) == 0u &&
                                          (kOp != kMxWgrad || (p.n & 7u) == 0u));
  const uint8_t* a_next;  // of the step to be loaded next
  uint64_t a_stride = kARow;
  uint32_t a_off[kDmaA];
  if constexpr (kOp == kMxWgrad) {
    a_next = reinterpret_cast<const uint8_t*>(p.a + uint64_t(r0) * p.lda + m0);
    a_stride = p.lda * (2u * kBC);
#pragma unroll
    for (uint32_t i = 0; i < kDmaA; i++) {
      const uint32_t pos = (i * kW + wave) % kALoads * 64u + lane, c = pos / kAPer;
      const uint32_t col = ((pos % kAPer) ^ mx_turn_cols(c)) * 8u;
      a_off[i] = c * uint32_t(p.lda) * 2u + (min(m0 + col, p.n - 8u) - m0) * 2u;
    }
  } else {
    const uint64_t pitch = kOp == kMxMatmul8 ? p.kp : p.lda * 2u;
    a_next = (kOp == kMxMatmul8 ? p.xq : reinterpret_cast<const uint8_t*>(p.a + r0)) + uint64_t(m0) * pitch;
#pragma unroll
    for (uint32_t i = 0; i < kDmaA; i++) {
      const uint32_t pos = (i * kW + wave) % kALoads * 64u + lane, r = pos / kAPer;
      a_off[i] = min(r, m1 - 1u - m0) * uint32_t(pitch) + ((pos % kAPer) ^ mx_turn<kARow>(r)) * 16u;
    }
  }
  const auto fill_a = [&](uint32_t step, uint8_t* to) {
    const uint32_t c0 = step * kBC;
#pragma unroll 1
    for (uint32_t i = 0; i < kDmaA; i++) {
      const uint32_t pos = (i * kW + wave) % kALoads * 64u + lane, r = pos / kAPer;
      uint32_t have;
      uint64_t at;
      if constexpr (kOp == kMxWgrad) {
        const uint32_t col = m0 + ((pos % kAPer) ^ mx_turn_cols(r)) * 8u;
        have = c0 + r < c1 && col < p.n ? p.n - col : 0u;
        at = (uint64_t(r0) + c0 + r) * p.lda + col;
      } else {
        const uint32_t c = c0 + ((pos % kAPer) ^ mx_turn<kARow>(r)) * 8u;
        have = c < c1 ? c1 - c : 0u;
        at = (uint64_t(m0) + min(r, m1 - 1u - m0)) * p.lda + r0 + c;
      }
      const uint16_t* src = p.a + (have ? at : 0u);
      *reinterpret_cast<u32x4v*>(to + pos * 16u) =
          have >= 8u ? u32x4v(*reinterpret_cast<const u32x4a2*>(src)) : mx_part8(src, have);
    }
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");  // the count of loads in flight starts anew
  };
  const auto load_a = [&](uint32_t step, uint32_t slot) {
    const uint32_t at = slot * kStage;
    if (kOp != kMxMatmul8 && (!wide || (step + 1u) * kBC > c1)) {
      fill_a(step, lds + at);
    } else {
#pragma unroll
      for (uint32_t i = 0; i < kDmaA; i++) mx_dma16(a_off[i], a_next, lds0 + at + (i * kW + wave) % kALoads * 1024u);
    }
    a_next += a_stride;
  };

  // the mx operand's loads
  const uint8_t* b_next;
  const uint8_t* bs_next;
  uint32_t b_off[kDmaRaw], b_row[kDmaRaw], bs_off = 0u, bs_row = 0u;
  const uint32_t b_pitch = p.kp * kBBits / 8u, s_pitch = p.kp / 32u;
  {
    const uint64_t row = kOp == kMxWgrad ? uint64_t(r0) : uint64_t(g) * p.n + (kRowsB ? n0 : r0);
    b_next = (kOp == kMxWgrad ? p.xq : p.wq) + row * b_pitch;
    bs_next = (kOp == kMxWgrad ? p.xs : p.ws) + row * s_pitch;
#pragma unroll
    for (uint32_t i = 0; i < kDmaRaw; i++) {
      const uint32_t pos = (i * kW + wave) % kRawLoads * 64u + lane, r = pos / kRawPer;
      b_row[i] = r;
      if constexpr (kRowsB) b_off[i] = min(r, p.n - 1u - n0) * b_pitch + (pos % kRawPer) * 16u;
      else
        b_off[i] = min(n0 * kBBits / 8u + ((pos % kRawPer) ^ mx_turn_pairs<int(kBBits), kRawRow>(r)) * 16u, b_pitch - 16u);
    }
    if constexpr (!kRowsB) {
      bs_row = tid % kBC;  // word by word, a step's rows behind each other
      bs_off = min(n0 / 32u + tid / kBC * 4u, s_pitch - 4u);
    }
  }
  // matmul: bytes from the scales of a row of W (r < kBN) or x to the end of
  // all; a row's 16 may reach past that and are then the section's last 16,
  // `late` bytes early.
  const auto scales_left = [&](uint32_t r) {
    const uint64_t rows = r < kBN ? uint64_t(p.groups - g) * p.n - n0 - min(r, p.n - 1u - n0)
                                  : uint64_t(p.tokens) - m0 - min(r - kBN, m1 - 1u - m0);
    return int(min(rows * s_pitch, uint64_t(1u << 30)));
  };
  const auto late = [](int left, uint32_t chunk) { return uint32_t(max(int(chunk * 16u + 16u) - left, 0)); };
  constexpr uint32_t kScaleLoads = kRowsB ? (kScaleRows + 64u * kW - 1u) / (64u * kW) : 1u;
  uint32_t sc_off[kScaleLoads];
  int sc_left[kScaleLoads];
  const uint8_t* const as_first = kOp == kMxMatmul8 ? p.xs + uint64_t(m0) * s_pitch - 16 : nullptr;
  const uint8_t* const bs_first = bs_next - 16;  // the offsets are 16 up, so that early ones stay positive
  if constexpr (kRowsB) {
#pragma unroll
    for (uint32_t i = 0; i < kScaleLoads; i++) {
      const uint32_t r = i * 64u * kW + tid;
      sc_off[i] = 16u + (r < kBN ? min(r, p.n - 1u - n0) : min(r - kBN, m1 - 1u - m0)) * s_pitch;
      sc_left[i] = scales_left(r);
    }
  }
  const auto scales_at = [](uint32_t chunk) { return kStages * kStage + 16u * kScaleRows * (chunk & 1u); };
  const auto load_scales = [&](uint32_t chunk) {
#pragma unroll
    for (uint32_t i = 0; i < kScaleLoads; i++) {
      const uint32_t first = i * 64u * kW + wave * 64u;
      if (first < kScaleRows)
        mx_dma16(sc_off[i] + chunk * 16u - late(sc_left[i], chunk), first < kBN ? bs_first : as_first,
                 lds0 + scales_at(chunk) + first * 16u);
    }
  };
  const auto load_b = [&](uint32_t step, uint32_t slot) {
    const uint32_t at = lds0 + slot * kStage + kABytes;
    if constexpr (kRowsB) {
#pragma unroll
      for (uint32_t i = 0; i < kDmaRaw; i++) mx_dma16(b_off[i], b_next, at + (i * kW + wave) % kRawLoads * 1024u);
      b_next += kRawRow;
    } else {
      // rows behind the contraction's end are fetched from its last
      const uint32_t last = min(c1 - 1u - step * kBC, kBC - 1u);
#pragma unroll
      for (uint32_t i = 0; i < kDmaRaw; i++)
        mx_dma16(min(b_row[i], last) * b_pitch + b_off[i], b_next, at + (i * kW + wave) % kRawLoads * 1024u);
      if (wave * 64u < kScaleWords)
        mx_dma4(min(bs_row, last) * s_pitch + bs_off, bs_next, at + kRawBytes + wave * 256u);
      b_next += uint64_t(kBC) * b_pitch;
      bs_next += uint64_t(kBC) * s_pitch;
    }
  };

  // A wave's row fragments lie kWM apart, so that where the group's rows end
  // inside the tile every wave has as few left (matmul, dx).
  typedef __attribute__((address_space(3))) v2i lds_v2i;
  typedef __attribute__((address_space(3))) v4s lds_v4s;
  const uint32_t wm = (wave / kWN) * 32u, wn = (wave % kWN) * (kBN / kWN);
  constexpr uint32_t kMStep = kWM * 32u;
  v16f acc[kFM][kFN];
#pragma unroll
  for (uint32_t i = 0; i < kFM; i++)
#pragma unroll
    for (uint32_t j = 0; j < kFN; j++)
#pragma unroll
      for (int r = 0; r < 16; r++) acc[i][j][r] = 0.0f;

  // Batch b of loads: both operands of step b.  kStages - 1 batches are in
  // flight while a step computes.
  const auto next_slot = [](uint32_t s) { return s + 1u == kStages ? 0u : s + 1u; };
  const auto batch = [&](uint32_t b, uint32_t slot) {
    if constexpr (kRowsB)
      if (b % 8u == 0u) load_scales(b / 8u);
    load_a(b, slot);
    load_b(b, slot);
  };
  // All but the last kBatches batches have landed.  Every wave counts its own
  // loads: those that fetch scale words have one more in each batch (in a
  // matmul's every eighth, where waiting for it too costs nothing).
  const auto fence = [&](auto batches) {
    constexpr int kBatches = decltype(batches)::value;
    if (!kRowsB && wave * 64u < kScaleWords) mx_fence<kBatches * int(kDma + 1u)>();
    else mx_fence<kBatches * int(kDma)>();
  };
#pragma unroll
  for (uint32_t b = 0; b + 1u < kStages; b++)
    if (b < steps) batch(b, b);
  int left_b[kFN], left_a[kFM];
  if constexpr (kRowsB) {
#pragma unroll
    for (uint32_t j = 0; j < kFN; j++) left_b[j] = scales_left(wn + j * 32u + (lane & 31u));
#pragma unroll
    for (uint32_t i = 0; i < kFM; i++) left_a[i] = kOp == kMxMatmul8 ? scales_left(kBN + wm + i * kMStep + (lane & 31u)) : 0;
  }
  uint32_t slot = 0u, load_slot = kStages - 1u;
  for (uint32_t step = 0; step < steps; step++) {
    if (step + kStages - 1u <= steps) fence(std::integral_constant<int, int(kStages) - 2>());
    else mx_fence<0>();
    if (step + kStages - 1u < steps) batch(step + kStages - 1u, load_slot);
    load_slot = slot;
    const uint8_t* sa = lds + slot * kStage;
    if constexpr (kRowsB) {
      const uint8_t* sb = sa + kABytes;
      // this step's scale byte of a row lies at ss + 16 row, or later
      const uint32_t chunk = step / 8u;
      const uint8_t* ss = lds + scales_at(chunk) + (step % 8u) * 2u + half;
      v4i rb[kFN];
      float bs[kFN];
#pragma unroll
      for (uint32_t j = 0; j < kFN; j++) {
        const uint32_t r = wn + j * 32u + (lane & 31u);
        rb[j] = *reinterpret_cast<const v4i*>(sb + r * 32u + half * 16u);
        bs[j] = mx_scale(ss[r * 16u + late(left_b[j], chunk)]);
      }
      u32x4v ra[kFM][2];
      float as[kFM];
      if constexpr (kOp == kMxMatmul8) {
#pragma unroll
        for (uint32_t i = 0; i < kFM; i++) {
          const uint32_t r = wm + i * kMStep + (lane & 31u);
          ra[i][0] = *reinterpret_cast<const u32x4v*>(sa + mx_at<64u>(r, half * 2u));
          ra[i][1] = *reinterpret_cast<const u32x4v*>(sa + mx_at<64u>(r, half * 2u + 1u));
          as[i] = mx_scale(ss[(kBN + r) * 16u + late(left_a[i], chunk)]);
        }
      }
#pragma unroll
      for (uint32_t s = 0; s < 4u; s++) {
        v8bf fa[kFM], fb[kFN];
#pragma unroll
        for (uint32_t i = 0; i < kFM; i++) {
          if constexpr (kOp == kMxMatmul8)
            fa[i] = __builtin_bit_cast(v8bf, mx_unit8(ra[i][s / 2u][(s % 2u) * 2u], ra[i][s / 2u][(s % 2u) * 2u + 1u], as[i]));
          else
            fa[i] = *reinterpret_cast<const v8bf*>(sa + mx_at<128u>(wm + i * kMStep + (lane & 31u), half * 4u + s));
        }
#pragma unroll
        for (uint32_t j = 0; j < kFN; j++) fb[j] = __builtin_bit_cast(v8bf, mx_unit4(uint32_t(rb[j][s]), bs[j]));
#pragma unroll
        for (uint32_t i = 0; i < kFM; i++)
#pragma unroll
          for (uint32_t j = 0; j < kFN; j++)
            acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(fb[j], fa[i], acc[i][j], 0, 0, 0);
      }
    } else {
      uint8_t* sb = lds + slot * kStage + kABytes;
      if ((step + 1u) * kBC > c1) {  // the last step: zeros behind the contraction's end
        const uint32_t have = c1 - step * kBC;
        for (uint32_t i = have * kRawPer + tid; i < kBC * kRawPer; i += 64u * kW)
          *reinterpret_cast<u32x4v*>(sb + i * 16u) = u32x4v{0u, 0u, 0u, 0u};
        for (uint32_t i = tid; i < kScaleWords; i += 64u * kW)
          if (i % kBC >= have) *reinterpret_cast<uint32_t*>(sb + kRawBytes + i * 4u) = 0x7F7F7F7Fu;
        mx_fence<0>();
      }
#pragma unroll
      for (uint32_t s = 0; s < kSub; s++) {
        const uint32_t c = s * 16u + half * 8u;  // this lane half's eight contraction rows
        const uint8_t* ss = sb + kRawBytes + (wn / 128u * kBC + c) * 4u;
        const u32x4v w0 = *reinterpret_cast<const u32x4v*>(ss), w1 = *reinterpret_cast<const u32x4v*>(ss + 16);
        v8bf fa[kFM], fb[kFN];
        const uint32_t ct = c + ((lane >> 2) & 3u);  // this lane's row where four are gathered
#pragma unroll
        for (uint32_t i = 0; i < kFM; i++) {
          if constexpr (kOp == kMxWgrad) {
            const uint32_t byte = (wm + i * kMStep) * 2u + ((lane >> 4) & 1u) * 32u + (lane & 3u) * 8u;
            fa[i] = mx_read_cols(sa + ct * kARow + (byte ^ (mx_turn_cols(ct) << 4)),
                                 sa + (ct + 4u) * kARow + (byte ^ (mx_turn_cols(ct + 4u) << 4)));
          } else {
            fa[i] = *reinterpret_cast<const v8bf*>(sa + mx_at<kARow>(wm + i * kMStep + (lane & 31u), s * 2u + half));
          }
        }
#pragma unroll
        for (uint32_t j = 0; j < kFN; j += 2u) {
          const uint32_t block = wn / 32u + j + ((lane >> 4) & 1u);  // of this lane's columns
          uint32_t q[kBBits / 2u];
          if constexpr (kOp == kMxWgrad) {
            const uint32_t byte = block * 32u + (lane & 3u) * 8u;
            const uint8_t* at = sb + ct * kRawRow + (byte ^ (mx_turn_pairs<8, kRawRow>(ct) << 4));
            const v4s lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4s*)at);
            const v4s hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4s*)(at + 4u * kRawRow));
            const u32x2v l = __builtin_bit_cast(u32x2v, lo), h = __builtin_bit_cast(u32x2v, hi);
            q[0] = l[0];
            q[1] = l[1];
            q[2] = h[0];
            q[3] = h[1];
          } else {
            const uint32_t r = c + ((lane >> 1) & 7u);
            const v2i v = __builtin_amdgcn_ds_read_tr8_b64_v2i32(
                (lds_v2i*)(sb + r * kRawRow + ((block ^ mx_turn_pairs<4, kRawRow>(r)) << 4) + (lane & 1u) * 8u));
            q[0] = uint32_t(v[0]);
            q[1] = uint32_t(v[1]);
          }
          mx_pairs<int(kBBits)>(q, w0, w1, (block & 3u) * 8u + 9u, fb[j], fb[j + 1u]);
        }
#pragma unroll
        for (uint32_t i = 0; i < kFM; i++)
#pragma unroll
          for (uint32_t j = 0; j < kFN; j++)
            acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(fb[j], fa[i], acc[i][j], 0, 0, 0);
      }
    }
    slot = next_slot(slot);
  }

#pragma unroll
  for (uint32_t i = 0; i < kFM; i++) {
    const uint32_t row = m0 + wm + i * kMStep + (lane & 31u);
    const uint64_t at = kOp == kMxWgrad ? ((uint64_t(part) * p.groups + g) * p.n + row) * p.k
                                         : (uint64_t(part) * p.tokens + row) * p.ldo;
    if constexpr (kRowsB) {
#pragma unroll
      for (uint32_t j = 0; j < kFN; j++) mx_store_frag(p, row < m1, at, n0 + wn + j * 32u, cols, acc[i][j]);
    } else if (row < m1) {
#pragma unroll
      for (uint32_t j = 0; j < kFN; j += 2u) mx_store_pair(p, at, n0 + wn + j * 32u, cols, acc[i][j], acc[i][j + 1u]);
    }
  }
}

// matmul of an mx8 operand with a BF16 result, where the caller asks for it
// (CIERA_MX_SCALED): the scaled matrix instructions take e4m3 and e2m1 values
// with their scale bytes as they are, at twice the BF16 instructions' rate.
// They add blocks, and earlier sums, in FP32, but within a block of 32 they
// line the products up with the largest and cut what lies below 2^(E - 13),
// 2^E being that product's binade.  So a block's sum is off by at most 2^-8 of
// its largest product, which is more than an FP32 sum may lose: it is the
// caller's choice, and k_mx_gemm and k_mx_few compute what is not asked for
// here.  On activations with a few loud channels the result moved by 1/7 of a
// BF16 rounding at the most.  128 contraction values (four blocks) a step, the
// ring and the tile as in k_mx_gemm; the padded pitch leaves no partial step.
// 8,192 rows in 64 groups, n = 1,024, k = 2,048: 35 us (k_mx_gemm 51); 32,768
// rows: 84 us (141), 1.64 PFLOP/s, bound by what its loads keep in flight, 43
// KB a CU.  A row's four scale bytes of a step are read as one word (byte by
// byte: 87 us).
template <uint32_t kBM, uint32_t kBN, uint32_t kWM, uint32_t kWN, uint32_t kStages, uint32_t kPerCu>
__global__ __launch_bounds__(kWM * kWN * 64u, kWM* kWN / 4u * kPerCu) void k_mx_gemm8(MxArgs p) {
  constexpr uint32_t kW = kWM * kWN;
  constexpr uint32_t kABytes = kBM * 128u, kRawBytes = kBN * 64u;
  constexpr uint32_t kStage = kABytes + kRawBytes;
  // 16 scale bytes of every row (W's, then x's) at a time, four steps' worth, twice
  constexpr uint32_t kScaleRows = (kBN + kBM + 63u) / 64u * 64u;
  constexpr uint32_t kFM = kBM / kWM / 32u, kFN = kBN / kWN / 32u;
  constexpr uint32_t kDmaA = kABytes / (1024u * kW), kDmaB = kRawBytes / (1024u * kW);
  constexpr uint32_t kDma = kDmaA + kDmaB;
  static_assert(kDmaA * 1024u * kW == kABytes && kDmaB * 1024u * kW == kRawBytes, "whole loads for every wave");
  static_assert(kBN % 64u == 0u, "whole waves");
  __shared__ __attribute__((aligned(256))) uint8_t lds[kStages * kStage + 32u * kScaleRows];
  const uint32_t tid = threadIdx.x, lane = tid & 63u, half = lane >> 5;
  const uint32_t wave = uint32_t(__builtin_amdgcn_readfirstlane(int(tid >> 6)));
  if (blockIdx.x == 0u) mx_report(p);
  MxTile t;
  if (!mx_find_tile(p, kBM == 128u ? 7u : kBM == 64u ? 6u : 5u, (p.n + kBN - 1u) / kBN, t)) return;
  const uint32_t m0 = t.row0, m1 = t.row1, n0 = t.col * kBN;
  const uint32_t lds0 = mx_lds(lds);

  const uint8_t* a_base = p.xq + uint64_t(m0) * p.kp;
  const uint8_t* as_base = p.xs + uint64_t(m0) * (p.kp / 32u);
  const uint8_t* b_base = p.wq + (uint64_t(t.g) * p.n + n0) * (p.kp / 2u);
  const uint8_t* bs_base = p.ws + (uint64_t(t.g) * p.n + n0) * (p.kp / 32u);
  uint32_t a_off[kDmaA], b_off[kDmaB];
#pragma unroll
  for (uint32_t i = 0; i < kDmaA; i++) {
    const uint32_t pos = (i * kW + wave) * 64u + lane, r = pos >> 3;
    a_off[i] = min(r, m1 - 1u - m0) * p.kp + ((pos & 7u) ^ mx_turn<128u>(r)) * 16u;
  }
#pragma unroll
  for (uint32_t i = 0; i < kDmaB; i++) {
    const uint32_t pos = (i * kW + wave) * 64u + lane, r = pos >> 2;
    b_off[i] = min(r, p.n - 1u - n0) * (p.kp / 2u) + ((pos & 3u) ^ mx_turn<64u>(r)) * 16u;
  }
  // scales: as in k_mx_gemm
  const uint32_t s_pitch = p.kp / 32u;
  const auto scales_left = [&](uint32_t r) {
    const uint64_t rows = r < kBN ? uint64_t(p.groups - t.g) * p.n - n0 - min(r, p.n - 1u - n0)
                                  : uint64_t(p.tokens) - m0 - min(r - kBN, m1 - 1u - m0);
    return int(min(rows * s_pitch, uint64_t(1u << 30)));
  };
  const auto late = [](int left, uint32_t chunk) { return uint32_t(max(int(chunk * 16u + 16u) - left, 0)); };
  constexpr uint32_t kScaleLoads = (kScaleRows + 64u * kW - 1u) / (64u * kW);
  uint32_t sc_off[kScaleLoads];
  int sc_left[kScaleLoads];
#pragma unroll
  for (uint32_t i = 0; i < kScaleLoads; i++) {
    const uint32_t r = i * 64u * kW + tid;
    sc_off[i] = 16u + (r < kBN ? min(r, p.n - 1u - n0) : min(r - kBN, m1 - 1u - m0)) * s_pitch;
    sc_left[i] = scales_left(r);
  }
  const auto scales_at = [](uint32_t chunk) { return kStages * kStage + 16u * kScaleRows * (chunk & 1u); };
  const auto batch = [&](uint32_t step, uint32_t slot) {
    const uint32_t at = lds0 + slot * kStage;
    if (step % 4u == 0u) {
      const uint32_t chunk = step / 4u;
#pragma unroll
      for (uint32_t i = 0; i < kScaleLoads; i++) {
        const uint32_t first = i * 64u * kW + wave * 64u;
        if (first < kScaleRows)
          mx_dma16(sc_off[i] + chunk * 16u - late(sc_left[i], chunk), (first < kBN ? bs_base : as_base) - 16,
                   lds0 + scales_at(chunk) + first * 16u);
      }
    }
#pragma unroll
    for (uint32_t i = 0; i < kDmaA; i++) mx_dma16(a_off[i], a_base + step * 128u, at + (i * kW + wave) * 1024u);
#pragma unroll
    for (uint32_t i = 0; i < kDmaB; i++) mx_dma16(b_off[i], b_base + step * 64u, at + kABytes + (i * kW + wave) * 1024u);
  };

  const uint32_t wm = (wave / kWN) * 32u, wn = (wave % kWN) * (kBN / kWN);
  constexpr uint32_t kMStep = kWM * 32u;
  v16f acc[kFM][kFN];
#pragma unroll
  for (uint32_t i = 0; i < kFM; i++)
#pragma unroll
    for (uint32_t j = 0; j < kFN; j++)
#pragma unroll
      for (int r = 0; r < 16; r++) acc[i][j][r] = 0.0f;

  const uint32_t steps = p.kp / 128u;
#pragma unroll
  for (uint32_t b = 0; b + 1u < kStages; b++)
    if (b < steps) batch(b, b);
  int left_a[kFM], left_b[kFN];
#pragma unroll
  for (uint32_t i = 0; i < kFM; i++) left_a[i] = scales_left(kBN + wm + i * kMStep + (lane & 31u));
#pragma unroll
  for (uint32_t j = 0; j < kFN; j++) left_b[j] = scales_left(wn + j * 32u + (lane & 31u));
  uint32_t slot = 0u, load_slot = kStages - 1u;
  for (uint32_t step = 0; step < steps; step++) {
    if (step + kStages - 1u <= steps) mx_fence<int((kStages - 2u) * kDma)>();
    else mx_fence<0>();
    if (step + kStages - 1u < steps) batch(step + kStages - 1u, load_slot);
    load_slot = slot;
    const uint8_t* s_a = lds + slot * kStage;
    const uint8_t* s_b = s_a + kABytes;
    const uint32_t chunk = step / 4u;
    const uint8_t* s_s = lds + scales_at(chunk) + (step % 4u) * 4u;
    // Lane half h holds block 2 s + h of B's row, and of A's row the 16
    // values at 16 h and at 32 + 16 h of the 64; its scale byte is block
    // 2 s + h's.  A step's four bytes of a row are one word; turned by the
    // half, the instruction picks byte 0 or 2 of it.
    uint32_t sa[kFM], sb[kFN];
#pragma unroll
    for (uint32_t i = 0; i < kFM; i++) {
      const uint8_t* at = s_s + (kBN + wm + i * kMStep + (lane & 31u)) * 16u + late(left_a[i], chunk);
      sa[i] = *reinterpret_cast<const uint32_t*>(at) >> (8u * half);
    }
#pragma unroll
    for (uint32_t j = 0; j < kFN; j++) {
      const uint8_t* at = s_s + (wn + j * 32u + (lane & 31u)) * 16u + late(left_b[j], chunk);
      sb[j] = *reinterpret_cast<const uint32_t*>(at) >> (8u * half);
    }
#pragma unroll
    for (uint32_t s = 0; s < 2u; s++) {
      v8i fa[kFM], fb[kFN];
#pragma unroll
      for (uint32_t i = 0; i < kFM; i++) {
        const uint32_t r = wm + i * kMStep + (lane & 31u);
        const v4i lo = *reinterpret_cast<const v4i*>(s_a + mx_at<128u>(r, s * 4u + half));
        const v4i hi = *reinterpret_cast<const v4i*>(s_a + mx_at<128u>(r, s * 4u + 2u + half));
        fa[i] = v8i{lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
      }
#pragma unroll
      for (uint32_t j = 0; j < kFN; j++) {
        const v4i q = *reinterpret_cast<const v4i*>(s_b + mx_at<64u>(wn + j * 32u + (lane & 31u), s * 2u + half));
        fb[j] = v8i{q[0], q[1], q[2], q[3], 0, 0, 0, 0};
      }
#pragma unroll
      for (uint32_t i = 0; i < kFM; i++)
#pragma unroll
        for (uint32_t j = 0; j < kFN; j++) {
          if (s == 0u)
            acc[i][j] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(fb[j], fa[i], acc[i][j], 4, 0, 0, int(sb[j]), 0,
                                                                        int(sa[i]));
          else
            acc[i][j] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(fb[j], fa[i], acc[i][j], 4, 0, 2, int(sb[j]), 2,
                                                                        int(sa[i]));
        }
    }
    slot = slot + 1u == kStages ? 0u : slot + 1u;
  }
#pragma unroll
  for (uint32_t i = 0; i < kFM; i++) {
    const uint32_t row = m0 + wm + i * kMStep + (lane & 31u);
#pragma unroll
    for (uint32_t j = 0; j < kFN; j++)
      mx_store_frag(p, row < m1, uint64_t(row) * p.ldo, n0 + wn + j * 32u, p.n, acc[i][j]);
  }
}

// matmul for few tokens a group: bound by reading the weights once.  A wave
// takes 16 weight rows and 16 of the group's tokens; a lane reads 16 bytes of
// a weight row, one block, straight into registers and makes BF16 of it there,
// 128 contraction values a step, eight steps of loads ahead.
//   kSplit 1: the eight waves of a workgroup take 128 weight rows and share
//             the tokens' values through LDS.
//   kSplit 8: eight waves take the same 16 rows and every eighth step, their
//             sums are added in wave order; for calls with too few rows to
//             fill the chip otherwise.
// 64 rows on 42 of 64 groups of 1,024 x 2,048: 13.3 us for 47 MB, 3.5 TB/s;
// one row, n = k = 2,048: 6.9 us, a launch.
constexpr uint32_t kMxFewThreads = 512u;

// Eight values of x, c a multiple of 8: as loaded (mx8: the values, then the
// scale byte), and as BF16.  Behind the contraction's end: zeros.
template <bool kMx8>
__device__ __forceinline__ u32x4v mx_few_load(const MxArgs& p, uint64_t row, uint32_t c) {
  if constexpr (kMx8) {
    const u32x2v q = *reinterpret_cast<const u32x2v*>(p.xq + row * p.kp + c);
    return u32x4v{q[0], q[1], p.xs[row * (p.kp / 32u) + c / 32u], 0u};
  } else {
    return *reinterpret_cast<const u32x4a2*>(p.a + row * p.lda + (c + 8u <= p.k ? c : 0u));
  }
}
template <bool kMx8>
__device__ __forceinline__ u32x4v mx_few_value(const MxArgs& p, u32x4v v, uint64_t row, uint32_t c) {
  if constexpr (kMx8) return mx_unit8(v[0], v[1], mx_scale(v[2]));
  if (c + 8u > p.k) return mx_part8(p.a + row * p.lda + (c < p.k ? c : 0u), c < p.k ? p.k - c : 0u);
  return v;
}

template <bool kMx8, uint32_t kSplit>
__global__ __launch_bounds__(kMxFewThreads, 4) void k_mx_few(MxArgs p) {
  constexpr uint32_t kWaves = kMxFewThreads / 64u;
  constexpr uint32_t kAhead = kSplit == 1u ? 8u : 4u;
  constexpr uint32_t kPitch = kAhead * 128u + 8u;  // a row's start moves on by 16 bytes of banks
  constexpr uint32_t kPer = kAhead * 16u;          // units of 8 values of a row
  constexpr uint32_t kFirst = 2u;                  // units a thread fetches before the weights
  __shared__ __attribute__((aligned(16))) uint16_t s_x[kSplit == 1u ? 16u * kPitch : 8u];
  __shared__ float s_sum[kSplit == 1u ? 1u : kWaves][16][16];
  const uint32_t tid = threadIdx.x, lane = tid & 63u, wave = tid >> 6;
  if (blockIdx.x == 0u && blockIdx.y == 0u) mx_report(p);
  const uint32_t g = blockIdx.y;
  uint32_t r0, r1;
  mx_rows(p, g, r0, r1);
  if (r0 == r1) return;
  const uint32_t n0 = kSplit == 1u ? (blockIdx.x * kWaves + wave) * 16u : blockIdx.x * 16u;
  const uint32_t l16 = lane & 15u, kb = lane >> 4;
  const uint64_t wrow = uint64_t(g) * p.n + min(n0 + l16, p.n - 1u);
  const uint8_t* wq = p.wq + wrow * (p.kp / 2u) + kb * 16u;
  const uint8_t* ws = p.ws + wrow * (p.kp / 32u);
  const uint32_t steps = p.kp / 128u;
  const bool some = p.k >= 8u;  // a whole unit of x exists
  for (uint32_t t0 = r0; t0 < r1; t0 += 16u) {
    const uint32_t have = min(16u, r1 - t0);
    const uint32_t row = min(l16, have - 1u);
    v4f acc[2] = {};
    constexpr uint32_t kBy = kSplit == 1u ? 1u : kWaves;
    for (uint32_t at = kSplit == 1u ? 0u : wave; at < steps; at += kBy * kAhead) {
      const bool whole = at + (kAhead - 1u) * kBy < steps;
      const uint32_t units = have * kPer;
      u32x4v first[kFirst];
      if constexpr (kSplit == 1u) {
#pragma unroll
        for (uint32_t i = 0; i < kFirst; i++) {
          const uint32_t u = min(i * kMxFewThreads + tid, units - 1u);
          const uint32_t c = min(at * 128u + u % kPer * 8u, p.kp - 8u);
          if (kMx8 || some) first[i] = mx_few_load<kMx8>(p, t0 + u / kPer, c);
        }
      }
      v4i q[kAhead];
      uint32_t sb[kAhead];
#pragma unroll
      for (uint32_t i = 0; i < kAhead; i++)
        q[i] = *reinterpret_cast<const v4i*>(wq + min(at + i * kBy, steps - 1u) * 64u);
      if (kSplit == 1u && whole) {  // a word of scale bytes a step, four at a time
#pragma unroll
        for (uint32_t i = 0; i < kAhead; i += 4u) {
          typedef uint32_t u32x4a4 __attribute__((ext_vector_type(4), aligned(4)));
          const u32x4v w = *reinterpret_cast<const u32x4a4*>(ws + (at + i) * 4u);
#pragma unroll
          for (uint32_t j = 0; j < 4u; j++) sb[i + j] = w[j];
        }
      } else {
#pragma unroll
        for (uint32_t i = 0; i < kAhead; i++)
          sb[i] = *reinterpret_cast<const uint32_t*>(ws + min(at + i * kBy, steps - 1u) * 4u);
      }
      if constexpr (kSplit == 1u) {
        if (at) __syncthreads();
#pragma unroll
        for (uint32_t i = 0; i < kFirst; i++) {
          const uint32_t u = i * kMxFewThreads + tid, c = at * 128u + u % kPer * 8u;
          if (u < units && c < p.kp)
            *reinterpret_cast<u32x4v*>(s_x + u / kPer * kPitch + u % kPer * 8u) =
                mx_few_value<kMx8>(p, first[i], t0 + u / kPer, c);
        }
        for (uint32_t u = kFirst * kMxFewThreads + tid; u < units; u += kMxFewThreads) {
          const uint32_t r = u / kPer, c = at * 128u + u % kPer * 8u;
          if (c < p.kp) {
            u32x4v v = {0u, 0u, 0u, 0u};
            if (kMx8 || some) v = mx_few_load<kMx8>(p, t0 + r, c);
            *reinterpret_cast<u32x4v*>(s_x + r * kPitch + u % kPer * 8u) = mx_few_value<kMx8>(p, v, t0 + r, c);
          }
        }
        __syncthreads();
      }
      const auto take = [&](uint32_t i) {
        const float s = mx_scale((sb[i] >> (8u * kb)) & 255u);
#pragma unroll
        for (uint32_t j = 0; j < 4u; j++) {
          u32x4v x;
          if constexpr (kSplit == 1u) {
            x = *reinterpret_cast<const u32x4v*>(s_x + row * kPitch + i * 128u + kb * 32u + j * 8u);
          } else {
            const uint32_t c = (at + i * kBy) * 128u + kb * 32u + j * 8u;
            x = u32x4v{0u, 0u, 0u, 0u};
            if (kMx8 || some) x = mx_few_load<kMx8>(p, t0 + row, c);
            x = mx_few_value<kMx8>(p, x, t0 + row, c);
          }
          acc[j & 1u] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
              __builtin_bit_cast(v8bf, x), __builtin_bit_cast(v8bf, mx_unit4(uint32_t(q[i][j]), s)), acc[j & 1u], 0, 0, 0);
        }
      };
      if (whole) {
#pragma unroll
        for (uint32_t i = 0; i < kAhead; i++) take(i);
      } else {
#pragma unroll
        for (uint32_t i = 0; i < kAhead; i++)
          if (at + i * kBy < steps) take(i);
      }
    }
    const v4f sum = acc[0] + acc[1];
    if constexpr (kSplit == 1u) {
#pragma unroll
      for (uint32_t r = 0; r < 4u; r++)
        if (kb * 4u + r < have && n0 + l16 < p.n) mx_store(p, uint64_t(t0 + kb * 4u + r) * p.ldo + n0 + l16, sum[r]);
    } else {
#pragma unroll
      for (uint32_t r = 0; r < 4u; r++) s_sum[wave][kb * 4u + r][l16] = sum[r];
      __syncthreads();
      if (tid < 256u) {
        const uint32_t tr = tid >> 4, col = n0 + (tid & 15u);
        float v = 0.0f;
#pragma unroll
        for (uint32_t w = 0; w < kWaves; w++) v += s_sum[w][tr][tid & 15u];
        if (tr < have && col < p.n) mx_store(p, uint64_t(t0 + tr) * p.ldo + col, v);
      }
    }
    __syncthreads();
  }
}

__global__ void k_mx_status(MxArgs p) { mx_report(p); }

// wgrad's parts added in order; four values a thread.
__global__ __launch_bounds__(kMxThreads) void k_mx_join(MxArgs p, const float* __restrict__ sums, uint64_t count) {
  const uint64_t at = (uint64_t(blockIdx.x) * kMxThreads + threadIdx.x) * 4u;
  if (at + 4u <= count && count % 4u == 0u) {
    v4f v = *reinterpret_cast<const v4f*>(sums + at);
    for (uint32_t i = 1; i < p.parts; i++) v += *reinterpret_cast<const v4f*>(sums + i * count + at);
    mx_store4(p, at, v);
  } else {
    for (uint64_t j = at; j < at + 4u && j < count; j++) {
      float v = sums[j];
      for (uint32_t i = 1; i < p.parts; i++) v += sums[i * count + j];
      mx_store(p, j, v);
    }
  }
}

// dx's, for one row of a group; other rows are left as they are.
__global__ __launch_bounds__(kMxThreads) void k_mx_join_rows(MxArgs p, const float* __restrict__ sums) {
  const uint32_t row = blockIdx.x;
  bool live = !p.offsets;
  for (uint32_t g = threadIdx.x & 63u; g < p.groups && !live; g += 64u) {
    uint32_t r0, r1;
    mx_rows(p, g, r0, r1);
    live = row >= r0 && row < r1;
  }
  if (!__any(live)) return;
  const uint64_t count = uint64_t(p.tokens) * p.k, from = uint64_t(row) * p.k, to = uint64_t(row) * p.ldo;
  for (uint32_t c = threadIdx.x * 4u; c < p.k; c += kMxThreads * 4u) {
    if (c + 4u <= p.k) {
      v4f v = *reinterpret_cast<const v4fa4*>(sums + from + c);
      for (uint32_t i = 1; i < p.parts; i++) v += v4f(*reinterpret_cast<const v4fa4*>(sums + i * count + from + c));
      mx_store4(p, to + c, v);
    } else {
      for (uint32_t j = c; j < p.k; j++) {
        float v = sums[from + j];
        for (uint32_t i = 1; i < p.parts; i++) v += sums[i * count + from + j];
        mx_store(p, to + j, v);
      }
    }
  }
}

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
  const uint64_t grid = mx_unit_groups(rows, mx_pitch(cols));
  if (grid > kMxMostGroups) return CIERA_ERR_ARG;
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
  const uint64_t grid = mx_unit_groups(rows, cols);
  if (grid > kMxMostGroups) return CIERA_ERR_ARG;
  const uint8_t* q = static_cast<const uint8_t*>(d_q);
  (void)hipGetLastError();
  launch(k_mx_decode<kBits>, dim3(uint32_t(grid)), dim3(kMxThreads), stream, q, q + mx_scales_at(rows, cols, kBits),
         rows, uint32_t(cols), static_cast<uint16_t*>(d_y), ld);
  return launch_status();
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
  p.parts = 1u;
  p.out_f32 = out_f32;
  return CIERA_OK;
}

MxSizes mx_sizes(const MxArgs& p) { return {p.tokens, p.n, p.k, p.groups, p.offsets != nullptr}; }

template <int kOp, uint32_t kBM, uint32_t kBN, uint32_t kBC, uint32_t kWM, uint32_t kWN, uint32_t kStages, uint32_t kPerCu>
ciera_status mx_gemm_as(const MxArgs& p, hipStream_t stream) {
  static_assert(kWM * kWN * 64u == kMxThreads, "what kMxMostGroups counts with");
  const uint64_t grid = mx_tile_groups(kOp, kBM, kBN, mx_sizes(p), p.parts);
  if (grid > kMxMostGroups) return CIERA_ERR_ARG;
  launch(k_mx_gemm<kOp, kBM, kBN, kBC, kWM, kWN, kStages, kPerCu>, dim3(uint32_t(grid), kOp == kMxDx ? p.parts : 1u), dim3(kWM * kWN * 64u), stream, p);
  return launch_status();
}
template <uint32_t kBM, uint32_t kBN, uint32_t kWM, uint32_t kWN, uint32_t kStages, uint32_t kPerCu>
ciera_status mx_gemm8_as(const MxArgs& p, hipStream_t stream) {
  static_assert(kWM * kWN * 64u == kMxThreads, "what kMxMostGroups counts with");
  const uint64_t grid = mx_tile_groups(kMxMatmul8, kBM, kBN, mx_sizes(p), 1u);
  if (grid > kMxMostGroups) return CIERA_ERR_ARG;
  launch(k_mx_gemm8<kBM, kBN, kWM, kWN, kStages, kPerCu>, dim3(uint32_t(grid)), dim3(kWM * kWN * 64u), stream, p);
  return launch_status();
}

template <int kOp>
ciera_status mx_gemm(const MxArgs& p, MxKernel kernel, hipStream_t stream) {
  if constexpr (kOp == kMxDx) {
    switch (kernel) {
      case kMx128x256: return mx_gemm_as<kOp, 128u, 256u, 64u, 1u, 4u, 3u, 2u>(p, stream);
      case kMx64x128: return mx_gemm_as<kOp, 64u, 128u, 64u, 2u, 2u, 3u, 2u>(p, stream);
      case kMx32x256: return mx_gemm_as<kOp, 32u, 256u, 64u, 1u, 4u, 2u, 4u>(p, stream);
      default: return mx_gemm_as<kOp, 64u, 256u, 64u, 1u, 4u, 2u, 3u>(p, stream);
    }
  } else {
    if constexpr (kOp == kMxMatmul)
      if (kernel == kMx32x128) return mx_gemm_as<kOp, 32u, 128u, 64u, 1u, 4u, 3u, 2u>(p, stream);
    switch (kernel) {
      case kMx128x256: return mx_gemm_as<kOp, 128u, 256u, 64u, 2u, 2u, 3u, 2u>(p, stream);
      case kMx128x128: return mx_gemm_as<kOp, 128u, 128u, 64u, 2u, 2u, 2u, 3u>(p, stream);
      default: return mx_gemm_as<kOp, 64u, 128u, 64u, 1u, 4u, 3u, 2u>(p, stream);
    }
  }
}
ciera_status mx_gemm8(const MxArgs& p, hipStream_t stream) {
  switch (mx_scaled_kernel(mx_sizes(p))) {
    case kMx128x256: return mx_gemm8_as<128u, 256u, 2u, 2u, 2u, 2u>(p, stream);
    case kMx64x128: return mx_gemm8_as<64u, 128u, 1u, 4u, 2u, 4u>(p, stream);
    default: return mx_gemm8_as<32u, 128u, 1u, 4u, 3u, 2u>(p, stream);
  }
}

template <bool kMx8>
ciera_status mx_matmul_impl(MxArgs& p, hipStream_t stream, bool scaled = false) {
  (void)hipGetLastError();
  if (p.tokens == 0u) {
    launch(k_mx_status, dim3(1), dim3(64), stream, p);
    return launch_status();
  }
  if (kMx8 && scaled) return mx_gemm8(p, stream);
  const MxKernel kernel = mx_matmul_kernel(mx_sizes(p), kMx8);
  if (kernel == kMxFew128 || kernel == kMxFew16) {
    if (kernel == kMxFew128)
      launch(k_mx_few<kMx8, 1u>, dim3(uint32_t(cdiv(p.n, 128u)), p.groups), dim3(kMxFewThreads), stream, p);
    else
      launch(k_mx_few<kMx8, 8u>, dim3(uint32_t(cdiv(p.n, 16u)), p.groups), dim3(kMxFewThreads), stream, p);
    return launch_status();
  }
  return mx_gemm<kMx8 ? kMxMatmul8 : kMxMatmul>(p, kernel, stream);
}

ciera_status mx_dx_impl(MxArgs p, hipStream_t stream) {
  (void)hipGetLastError();
  if (p.tokens == 0u) {
    launch(k_mx_status, dim3(1), dim3(64), stream, p);
    return launch_status();
  }
  p.parts = mx_dx_parts(p.tokens, p.n, p.k, p.groups);
  const MxKernel kernel = mx_dx_kernel(mx_sizes(p));
  if (p.parts == 1u) return mx_gemm<kMxDx>(p, kernel, stream);
  MxArgs sums = p;
  sums.out = reinterpret_cast<uint8_t*>(p.ctrl) + kMxWsHead;
  sums.ldo = p.k;
  sums.out_f32 = 1u;
  const ciera_status st = mx_gemm<kMxDx>(sums, kernel, stream);
  if (st != CIERA_OK) return st;
  launch(k_mx_join_rows, dim3(p.tokens), dim3(kMxThreads), stream, p, static_cast<const float*>(sums.out));
  return launch_status();
}
ciera_status mx_wgrad_impl(MxArgs p, hipStream_t stream) {
  (void)hipGetLastError();
  p.parts = mx_wgrad_parts(p.tokens, p.n, p.k, p.groups);
  if (p.parts == 1u) return mx_gemm_as<kMxWgrad, 256u, 128u, 32u, 2u, 2u, 3u, 2u>(p, stream);
  MxArgs sums = p;
  sums.out = reinterpret_cast<uint8_t*>(p.ctrl) + kMxWsHead;
  sums.out_f32 = 1u;
  sums.accumulate = 0u;
  const ciera_status st = mx_gemm_as<kMxWgrad, 256u, 128u, 32u, 2u, 2u, 3u, 2u>(sums, stream);
  if (st != CIERA_OK) return st;
  const uint64_t count = uint64_t(p.groups) * p.n * p.k;
  launch(k_mx_join, dim3(uint32_t(cdiv(count, kMxThreads * 4u))), dim3(kMxThreads), stream, p,
         static_cast<const float*>(sums.out), count);
  return launch_status();
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
  const bool scaled = y_f32 == CIERA_MX_SCALED;  // BF16 by the scaled matrix instructions
  ciera_status st = mx_product(p, d_w, w_bytes, d_y, ldy, n, scaled ? 0u : y_f32, tokens, n, k, groups, d_offsets, d_ws,
                               ws_bytes);
  if (st == CIERA_OK) st = mx_encoded(d_xq, xq_bytes, tokens, k, 8u, CIERA_ERR_FORMAT);
  if (st != CIERA_OK) return st;
  p.xq = static_cast<const uint8_t*>(d_xq);
  p.xs = p.xq + mx_scales_at(tokens, k, 8u);
  return mx_matmul_impl<true>(p, stream, scaled);
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
  return mx_dx_impl(p, stream);
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
  return mx_wgrad_impl(p, stream);
}

}  // extern "C"
