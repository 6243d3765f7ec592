// low_rank.hip -- low-rank adapters of many requests beside a projection that
// they share, gfx950:
//
//   y_t = base_t + s_a B_a (A_a x_t),   a the adapter of row t
//
// A_a is rank x k, B_a n x rank.  Rows come sorted by adapter, as the experts'
// do: rows offsets[a] .. offsets[a+1] - 1 of the order are adapter a's, those
// before the first and behind the last have none and take base alone.
//
// One launch: a workgroup of eight waves takes 16 rows of one adapter and a slab
// of the columns.  It makes the rows' inner values v = s_a A_a x (16 x rank, the
// contraction spread over its waves, FP32 sums joined in LDS), and from them
// its columns.  v then goes through the BF16 matrix instructions as three BF16
// parts that hold its 24 significant bits, so that nothing is rounded between
// the two products.
//
// What bounds it (us by the launches' own events): for few rows the launch and
// one pass through dependent loads (64 rows of 24 adapters, rank 16, k = n =
// 2,048: 5.8 us, of which 2.5 launch); for few rows of a large rank and a long
// contraction A x, which every slab of columns makes again (16 rows, k = n =
// 8,192, rank 64: 19 on 2.8 for the bytes); for many rows memory in two phases,
// x and then base and y, that overlap only between workgroups (16,384 rows at
// rank 16, 201 MB: 45 us, 4.5 TB/s), and from rank 64 on the way of A and B from
// L2 through LDS, 512 KB for each tile of 16 rows (4,001 rows at rank 64, 53 MB:
// 16.4 us; 16,384: 73; at rank 128 124).  Base or v's loads further ahead gained
// nothing.
#include "ciera.h"

namespace {

constexpr uint32_t kLowRankMax = 128u;
constexpr uint32_t kLowRankRows = 16u;
constexpr uint32_t kLowRankThreads = 512u;
constexpr uint32_t kLowRankSlab = kLowRankThreads;  // columns that the waves take at once

struct LowRankArgs {
  const uint16_t* x;
  uint64_t ldx;
  const uint16_t* a;
  const uint16_t* b;
  const float* scales;
  const int64_t* offsets;
  const int32_t* order;
  const void* base;
  uint64_t ldb;
  void* y;
  uint64_t ldy;
  Ctrl* ctrl;
  uint32_t* status;
  uint32_t tokens, n, k, rank, adapters;
  uint32_t base_f32, y_f32;
  uint32_t slabs, slab;  // column slabs a row tile, and columns of one
};

// Rows of list `g`: an adapter's; behind the adapters, those after the last
// one's and those before the first one's.
__device__ __forceinline__ bool low_rank_rows(const LowRankArgs& p, uint32_t g, uint32_t& r0, uint32_t& r1) {
  const int64_t most = int64_t(p.tokens);
  if (g < p.adapters) {
    const int64_t a = p.offsets[g], b = p.offsets[g + 1u];
    const bool ok = a >= 0 && a <= b && b <= most;
    r0 = ok ? uint32_t(a) : 0u;
    r1 = ok ? uint32_t(b) : 0u;
    return ok;
  }
  r0 = r1 = 0u;
  if (g > p.adapters + 1u) return true;
  const int64_t at = p.offsets[g == p.adapters ? p.adapters : 0u];
  const uint32_t to = uint32_t(at < 0 ? 0 : at > most ? most : at);
  if (g == p.adapters) {
    r0 = to;
    r1 = p.tokens;
  } else {
    r1 = to;
  }
  return true;
}

// This workgroup's row tile, as for the products: every wave counts the lists'
// tiles, 64 lists a step.
__device__ __forceinline__ bool low_rank_tile(const LowRankArgs& p, uint32_t& g, uint32_t& row0, uint32_t& row1, uint32_t& slab) {
  const uint32_t lane = threadIdx.x & 63u, lists = p.adapters + 2u;
  uint32_t r0 = 0u, r1 = 0u, own = 0u, sum = 0u, total = 0u;
  const auto count = [&](uint32_t c) {
    low_rank_rows(p, c + lane, r0, r1);
    own = (r1 - r0 + kLowRankRows - 1u) / kLowRankRows;
    sum = wave_incl_scan(own);
  };
  for (uint32_t c = 0; c < lists; c += 64u) {
    count(c);
    total += uint32_t(__builtin_amdgcn_readlane(int(sum), 63));
  }
  if (blockIdx.x >= total * p.slabs) return false;
  const uint32_t at = mx_xcd_run(blockIdx.x, total * p.slabs), tile = at / p.slabs;
  slab = at - tile * p.slabs;
  uint32_t before = 0u;
  for (uint32_t c = 0; c < lists; c += 64u) {
    if (lists > 64u) count(c);
    const uint64_t past = __ballot(before + sum > tile);
    if (past) {
      const int l = __ffsll((unsigned long long)past) - 1;
      const uint32_t end = before + uint32_t(__builtin_amdgcn_readlane(int(sum), l));
      g = c + uint32_t(l);
      row0 = uint32_t(__builtin_amdgcn_readlane(int(r0), l)) +
             (tile - (end - uint32_t(__builtin_amdgcn_readlane(int(own), l)))) * kLowRankRows;
      row1 = uint32_t(__builtin_amdgcn_readlane(int(r1), l));
      return true;
    }
    before += uint32_t(__builtin_amdgcn_readlane(int(sum), 63));
  }
  return false;
}

__device__ __forceinline__ void low_rank_report(const LowRankArgs& p) {
  if (threadIdx.x >= 64u) return;
  bool ok = true;
  for (uint32_t g = threadIdx.x; g < p.adapters; g += 64u) {
    uint32_t r0, r1;
    ok = low_rank_rows(p, g, r0, r1) && ok;
  }
  const bool all = __all(ok);
  if (threadIdx.x == 0u) {
    p.ctrl->n_err_slots = 1u;
    *p.status = all ? uint32_t(CIERA_OK) : uint32_t(CIERA_ERR_ARG);
  }
}

// v as three BF16 numbers whose sum it is: its leading 8 significant bits, the
// next 8 and the last.  Cut, not rounded, so that none passes BF16's range;
// an infinity or a NaN is the first alone.  The first is zero only for a v of
// less than 2^-126.
__device__ __forceinline__ void low_rank_split(float v, uint16_t (&part)[3]) {
  const uint32_t b = __float_as_uint(v);
  if ((b & 0x7F800000u) == 0x7F800000u) {
    part[0] = mx_bf16(v);
    part[1] = part[2] = 0u;
    return;
  }
  part[0] = uint16_t(b >> 16);
  const float r = v - __uint_as_float(b & 0xFFFF0000u);
  part[1] = uint16_t(__float_as_uint(r) >> 16);
  part[2] = mx_bf16(r - __uint_as_float(__float_as_uint(r) & 0xFFFF0000u));
}

// LDS of a wave alone: what its lanes wrote before is what they read after.
__device__ __forceinline__ void wave_lds() { asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory"); }

// Where wave `wave` of kW begins in from .. to - 1, each with a stretch of whole
// 64s of its own, and where it ends.
template <uint32_t kW>
__device__ __forceinline__ void low_rank_share(uint32_t wave, uint32_t from, uint32_t to, uint32_t& c, uint32_t& end) {
  const uint32_t each = ((to - from + kW * 64u - 1u) / (kW * 64u)) * 64u;
  c = min(from + wave * each, to);
  end = min(c + each, to);
}

// The row of x or y of the tile's row `at`; false where it has none.
__device__ __forceinline__ bool low_rank_row(const LowRankArgs& p, uint32_t row0, uint32_t row1, uint32_t at, uint32_t& row) {
  const uint32_t slot = min(row0 + at, row1 - 1u);
  row = p.order ? uint32_t(p.order[slot]) : slot;
  const bool live = row0 + at < row1 && row < p.tokens;
  if (row >= p.tokens) row = 0u;
  return live;
}

// v = A x: a wave's part of the contraction, for 16 rows.  The rows come from
// memory as they lie, neighbouring lanes on neighbouring bytes, 64 values of each
// a step (32: more conflicts of banks; 16,384 rows, k = n = 2,048, rank 64: 83 us
// instead of 72), and go
// through LDS into the order of the matrix instructions, whose neighbouring
// lanes hold neighbouring rows (loaded in that order each lane's 16 bytes are a
// request of their own: 16,384 rows at rank 16: 60 us instead of 48).
template <uint32_t kF>
struct LowRankInner {
  static constexpr uint32_t kR = kF * 16u;
  static constexpr uint32_t kStep = 64u;        // values of k at a time
  static constexpr uint32_t kRow = kStep * 2u;  // bytes of a row of them
  static constexpr uint32_t kChunks = kRow / 16u, kPer = 64u / kChunks;  // lanes on a row, rows a load
  static constexpr uint32_t kX = kLowRankRows / kPer, kA = kR / kPer;    // loads
  static constexpr uint32_t kLds = (kLowRankRows + kR) * kRow;
  const uint16_t* x[kX];
  const uint16_t* a[kA];
  u32x4v wx[kX], wa[kA];
  __device__ __forceinline__ void rows(const LowRankArgs& p, uint32_t g, uint32_t row0, uint32_t row1) {
    const uint32_t r = (threadIdx.x & 63u) / kChunks;
#pragma unroll
    for (uint32_t i = 0; i < kA; i++) a[i] = p.a + (uint64_t(g) * p.rank + min(i * kPer + r, p.rank - 1u)) * p.k;
#pragma unroll
    for (uint32_t i = 0; i < kX; i++) {
      uint32_t row;
      low_rank_row(p, row0, row1, i * kPer + r, row);
      x[i] = p.x + uint64_t(row) * p.ldx;
    }
  }
  __device__ __forceinline__ void load(uint32_t c, uint32_t k) {
    const uint32_t at = c + (threadIdx.x % kChunks) * 8u;
#pragma unroll
    for (uint32_t i = 0; i < kX; i++) wx[i] = row_load8(x[i], at, k);
#pragma unroll
    for (uint32_t i = 0; i < kA; i++) wa[i] = row_load8(a[i], at, k);
    loads_first();
  }
  __device__ __forceinline__ void run(uint8_t* lds, uint32_t c, uint32_t end, uint32_t k, v4f (&acc)[kF]) {
    const uint32_t lane = threadIdx.x & 63u, i16 = lane & 15u, quarter = lane >> 4;
    const uint32_t r = lane / kChunks, chunk = lane % kChunks;
#pragma unroll
    for (uint32_t f = 0; f < kF; f++) acc[f] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
    if (c < end) load(c, k);
    for (; c < end; c += kStep) {
      if (c + kStep > k) {
#pragma unroll
        for (uint32_t i = 0; i < kX; i++) row_mend8(wx[i], c + chunk * 8u, k);
#pragma unroll
        for (uint32_t i = 0; i < kA; i++) row_mend8(wa[i], c + chunk * 8u, k);
      }
#pragma unroll
      for (uint32_t i = 0; i < kX; i++) *reinterpret_cast<u32x4v*>(lds + mx_at<kRow>(i * kPer + r, chunk)) = wx[i];
#pragma unroll
      for (uint32_t i = 0; i < kA; i++)
        *reinterpret_cast<u32x4v*>(lds + mx_at<kRow>(kLowRankRows + i * kPer + r, chunk)) = wa[i];
      if (c + kStep < end) load(c + kStep, k);
      wave_lds();
#pragma unroll
      for (uint32_t h = 0; h < kStep / 32u; h++) {
        const v8bf bx = *reinterpret_cast<const v8bf*>(lds + mx_at<kRow>(i16, h * 4u + quarter));
#pragma unroll
        for (uint32_t f = 0; f < kF; f++)
          acc[f] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
              *reinterpret_cast<const v8bf*>(lds + mx_at<kRow>((f + 1u) * 16u + i16, h * 4u + quarter)), bx, acc[f], 0, 0, 0);
      }
      wave_lds();
    }
  }
};

// y = base + B v, 64 columns a step: B's rows through LDS likewise, 64 ranks at a
// time (32: 16,384 rows at rank 64 88 us instead of 83).  Row 4 j + f of the 64 is column j of matrix fragment f, so that a lane
// ends with four neighbouring columns of four rows, and 16 lanes with 64.  16
// ranks fill half a matrix instruction: the other half takes v's next part.
template <uint32_t kF, bool kF32>
struct LowRankOuter {
  static constexpr uint32_t kR = kF * 16u;
  static constexpr uint32_t kRow = kF == 1u ? 32u : kF == 2u ? 64u : 128u;  // bytes of a row's piece
  static constexpr uint32_t kP = kR * 2u / kRow;             // pieces of ranks
  static constexpr uint32_t kHalves = kRow == 128u ? 2u : 1u;  // matrix instructions a piece and part of v
  static constexpr uint32_t kV = kP * kHalves, kSteps = kF == 1u ? 2u : kV * 3u;
  static constexpr uint32_t kChunks = kRow / 16u, kPer = 64u / kChunks, kLoads = 64u / kPer;
  static constexpr uint32_t kFrag = 17u * kRow;            // bytes from one fragment to the next
  static constexpr uint32_t kLds = 4u * kFrag;
  const uint16_t* b;
  uint32_t row[4];
  bool live[4];
  u32x4v w[kLoads];
  u32x4v base[4];  // BF16: the first half
  static __device__ __forceinline__ uint32_t at(uint32_t f, uint32_t j, uint32_t chunk) {
    const uint32_t turn = kRow == 128u ? j & 7u : kRow == 64u ? j >> 2 : j >> 3;
    return f * kFrag + j * kRow + ((chunk ^ turn) * 16u);
  }
  __device__ __forceinline__ void rows(const LowRankArgs& p, uint32_t g, uint32_t row0, uint32_t row1) {
    b = p.b + uint64_t(g) * p.n * p.rank;
#pragma unroll
    for (uint32_t r = 0; r < 4u; r++) {
      uint32_t of;
      live[r] = low_rank_row(p, row0, row1, ((threadIdx.x >> 4) & 3u) * 4u + r, of);
      row[r] = of;
    }
  }
  __device__ __forceinline__ void load_b(const LowRankArgs& p, uint32_t c, uint32_t piece) {
    const uint32_t lane = threadIdx.x & 63u;
#pragma unroll
    for (uint32_t i = 0; i < kLoads; i++)
      w[i] = row_load8(b + uint64_t(min(c + i * kPer + lane / kChunks, p.n - 1u)) * p.rank,
                       piece * (kRow / 2u) + lane % kChunks * 8u, p.rank);
  }
  // Where row r begins (a stride is less than 2^32).  With 17 to 64 ranks made at each use: kept from step to step, the
  // four rows' places in base and in y take 16 registers, and onto an FP32 base at rank 64 some of them memory (16,384
  // rows 98 us instead of 92; at rank 32 55 instead of 53; at rank 16 45 instead of 47, at 128 123 instead of 125).
  __device__ __forceinline__ uint64_t offset(uint32_t r, uint64_t ld) const {
    uint32_t of = row[r];
    if constexpr (kF == 2u || kF == 4u) asm volatile("" : "+v"(of));
    return uint64_t(of) * uint32_t(ld);
  }
  // this lane's four columns of its four rows: whole where none passes the end
  __device__ __forceinline__ void load_base(const LowRankArgs& p, uint32_t c) {
    const uint32_t col = c + (threadIdx.x & 15u) * 4u;
    if (!p.base) return;
#pragma unroll
    for (uint32_t r = 0; r < 4u; r++) {
      const uint64_t from = offset(r, p.ldb) + col;
      if constexpr (kF32) {
        const float* f = static_cast<const float*>(p.base) + from;
        if (col + 4u <= p.n) {
          base[r] = __builtin_bit_cast(u32x4v, v4f(*reinterpret_cast<const v4fa4*>(f)));
        } else {
#pragma unroll
          for (uint32_t i = 0; i < 4u; i++) base[r][i] = col + i < p.n ? __float_as_uint(f[i]) : 0u;
        }
      } else {
        const uint16_t* f = static_cast<const uint16_t*>(p.base) + from;
        if (col + 4u <= p.n) {
          const u32x2v v = *reinterpret_cast<const u32x2a2*>(f);
          base[r][0] = v[0];
          base[r][1] = v[1];
        } else {
          base[r][0] = (col < p.n ? uint32_t(f[0]) : 0u) | (col + 1u < p.n ? uint32_t(f[1]) << 16 : 0u);
          base[r][1] = col + 2u < p.n ? uint32_t(f[2]) : 0u;
        }
      }
    }
  }
  __device__ __forceinline__ float value(const LowRankArgs& p, uint32_t r, uint32_t i) const {
    if (!p.base) return 0.0f;
    if constexpr (kF32) return __uint_as_float(base[r][i]);
    else return i & 1u ? bf_hi(base[r][i >> 1]) : bf_lo(base[r][i >> 1]);
  }
  // past the last-level cache (16,384 rows at rank 16: 45 us instead of 48; rows of no adapter 24
  // instead of 35)
  __device__ __forceinline__ void store(const LowRankArgs& p, uint32_t c, const v4f (&sum)[4]) {
    const uint32_t col = c + (threadIdx.x & 15u) * 4u;
#pragma unroll
    for (uint32_t r = 0; r < 4u; r++) {
      float v[4];
#pragma unroll
      for (uint32_t f = 0; f < 4u; f++) v[f] = value(p, r, f) + sum[f][r];
      if (!live[r]) continue;
      const uint64_t to = offset(r, p.ldy) + col;
      if (p.y_f32) {
        float* o = static_cast<float*>(p.y) + to;
        if (col + 4u <= p.n) {
          __builtin_nontemporal_store(v4f{v[0], v[1], v[2], v[3]}, reinterpret_cast<v4fa4*>(o));
        } else {
#pragma unroll
          for (uint32_t i = 0; i < 3u; i++)
            if (col + i < p.n) o[i] = v[i];
        }
      } else {
        uint16_t* o = static_cast<uint16_t*>(p.y) + to;
        if (col + 4u <= p.n) {
          __builtin_nontemporal_store(u32x2v{mx_bf16x2(v[0], v[1]), mx_bf16x2(v[2], v[3])}, reinterpret_cast<u32x2a2*>(o));
        } else {
#pragma unroll
          for (uint32_t i = 0; i < 3u; i++)
            if (col + i < p.n) o[i] = mx_bf16(v[i]);
        }
      }
    }
  }
  // The sums of columns c .. c + 63 once more, where there is a NaN: an infinity of B times a part of v that is zero is
  // one, also where v is not zero.  The parts behind v's first see zeros for what is not finite in B, which times the
  // first part is what it is times v.  The other sums keep their bits: equal terms in equal order.  (Looking for a NaN:
  // 16,384 rows at rank 128 124.3 us instead of 123.1, up to rank 64 nothing that shows.)
  __device__ __forceinline__ void again(const LowRankArgs& p, const uint8_t* lds, const v8bf (&v)[kSteps], uint32_t c, v4f (&sum)[4]) const {
    const uint32_t i16 = threadIdx.x & 15u, quarter = (threadIdx.x >> 4) & 3u;
#pragma unroll
    for (uint32_t f = 0; f < 4u; f++) {
      sum[f] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (uint32_t step = 0; step < kV; step++) {
        u32x4v w;
        if constexpr (kP == 1u)  // the piece is still there
          w = *reinterpret_cast<const u32x4v*>(lds + at(f, i16, kF == 1u ? quarter & 1u : step * 4u + quarter));
        else
          w = row_get8<false>(b + uint64_t(min(c + i16 * 4u + f, p.n - 1u)) * p.rank, (step * 4u + quarter) * 8u, p.rank);
        const v8bf all = __builtin_bit_cast(v8bf, w);
#pragma unroll
        for (int i = 0; i < 4; i++) {
          if ((w[i] & 0x7F80u) == 0x7F80u) w[i] &= 0xFFFF0000u;
          if ((w[i] & 0x7F800000u) == 0x7F800000u) w[i] &= 0xFFFFu;
        }
        const v8bf fine = __builtin_bit_cast(v8bf, w);
        if constexpr (kF == 1u) {
          sum[f] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(v[1], fine, sum[f], 0, 0, 0);
          sum[f] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(v[0], quarter < 2u ? all : fine, sum[f], 0, 0, 0);
        } else {
#pragma unroll
          for (uint32_t part = 3u; part > 0u; part--)
            sum[f] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(v[(part - 1u) * kV + step], part > 1u ? fine : all, sum[f], 0, 0, 0);
        }
        loads_first();
      }
    }
  }
  // columns c .. n1 - 1, B and base of the first 64 being loaded
  __device__ __forceinline__ void columns(const LowRankArgs& p, uint8_t* lds, const v8bf (&v)[kSteps], uint32_t c, uint32_t n1) {
    const uint32_t lane = threadIdx.x & 63u, i16 = lane & 15u, quarter = lane >> 4;
    for (; c < n1; c += 64u) {
      v4f sum[4];
#pragma unroll
      for (uint32_t f = 0; f < 4u; f++) sum[f] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (uint32_t piece = 0; piece < kP; piece++) {
        if (p.rank != kR) {
#pragma unroll
          for (uint32_t i = 0; i < kLoads; i++) row_mend8(w[i], piece * (kRow / 2u) + lane % kChunks * 8u, p.rank);
        }
#pragma unroll
        for (uint32_t i = 0; i < kLoads; i++) {
          const uint32_t n = i * kPer + lane / kChunks;
          *reinterpret_cast<u32x4v*>(lds + at(n & 3u, n >> 2, lane % kChunks)) = w[i];
        }
        if (piece + 1u < kP) load_b(p, c, piece + 1u);
        else if (c + 64u < n1) load_b(p, c + 64u, 0u);
        loads_first();
        wave_lds();
#pragma unroll
        for (uint32_t h = 0; h < kHalves; h++) {
#pragma unroll
          for (uint32_t f = 0; f < 4u; f++) {
            const v8bf fb = *reinterpret_cast<const v8bf*>(lds + at(f, i16, kF == 1u ? quarter & 1u : h * 4u + quarter));
            if constexpr (kF == 1u) {
              sum[f] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(v[1], fb, sum[f], 0, 0, 0);
              sum[f] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(v[0], fb, sum[f], 0, 0, 0);
            } else {
#pragma unroll
              for (uint32_t part = 3u; part > 0u; part--)  // the smallest part first
                sum[f] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(v[(part - 1u) * kV + piece * kHalves + h], fb, sum[f], 0, 0, 0);
            }
          }
        }
        wave_lds();
      }
      loads_first();
      const v4f t = (sum[0] + sum[1]) + (sum[2] + sum[3]);  // NaN if one of them is (or by overflow, which costs time alone)
      if (__any(__builtin_isnan((t[0] + t[1]) + (t[2] + t[3])))) again(p, lds, v, c, sum);
      store(p, c, sum);
      if (c + 64u < n1) load_base(p, c + 64u);
    }
  }
};

// Rows of no adapter: base alone.  Two rows a wave, its lanes side by side, the
// loads of four units of 8 values together.
template <bool kF32>
__device__ __forceinline__ void low_rank_bare(const LowRankArgs& p, uint32_t row0, uint32_t row1, uint32_t c, uint32_t n1) {
  static_assert(kLowRankThreads / 64u * 2u == kLowRankRows, "two rows a wave");
  const uint32_t lane = threadIdx.x & 63u;
  for (uint32_t r = 0; r < 2u; r++) {
    uint32_t row;
    if (!low_rank_row(p, row0, row1, mx_first(threadIdx.x >> 6) * 2u + r, row)) continue;
    for (uint32_t at = c + lane * 8u; at < n1; at += 4u * 512u) {
      Row8<kF32> v[4];
      if (p.base) {
#pragma unroll
        for (uint32_t i = 0; i < 4u; i++) v[i].load(p.base, uint64_t(row) * p.ldb, at + i * 512u, p.n);
        loads_first();
      }
#pragma unroll
      for (uint32_t i = 0; i < 4u; i++) {
        const uint32_t col = at + i * 512u;
        if (col >= n1) break;
        if (p.base) v[i].mend(col, p.n);
        float e[8];
#pragma unroll
        for (int k = 0; k < 8; k++) e[k] = p.base ? v[i].value(k) : 0.0f;
        const uint64_t to = uint64_t(row) * p.ldy;
        if (!p.y_f32) {
          row_store8<true>(static_cast<uint16_t*>(p.y) + to, col, p.n,
                           u32x4v{mx_bf16x2(e[0], e[1]), mx_bf16x2(e[2], e[3]), mx_bf16x2(e[4], e[5]), mx_bf16x2(e[6], e[7])});
        } else if (col + 8u <= p.n) {
          float* o = static_cast<float*>(p.y) + to + col;
          __builtin_nontemporal_store(v4f{e[0], e[1], e[2], e[3]}, reinterpret_cast<v4fa4*>(o));
          __builtin_nontemporal_store(v4f{e[4], e[5], e[6], e[7]}, reinterpret_cast<v4fa4*>(o + 4));
        } else {
#pragma unroll
          for (uint32_t k = 0; k < 7u; k++)
            if (col + k < p.n) static_cast<float*>(p.y)[to + col + k] = e[k];
        }
      }
    }
  }
}

// kF: fragments of 16 ranks (1, 2, 4 or 8).  Registers and LDS for two workgroups
// a CU; at 128 ranks the LDS holds one.
template <uint32_t kF, bool kF32>
__global__ __launch_bounds__(kLowRankThreads, kF <= 4u ? 4 : 2) void k_low_rank(LowRankArgs p) {
  typedef LowRankInner<kF> Inner;
  typedef LowRankOuter<kF, kF32> Outer;
  constexpr uint32_t kW = kLowRankThreads / 64u;
  constexpr uint32_t kR = kF * 16u;    // ranks, zeros behind the real ones
  constexpr uint32_t kLine = kR + 8u;  // of a row's parts in LDS, 16 bytes more for the banks
  constexpr uint32_t kSum = kR + 4u;   // of a row's sums, likewise
  constexpr uint32_t kMine = Inner::kLds > Outer::kLds ? Inner::kLds : Outer::kLds;
  constexpr uint32_t kSums = kW * kLowRankRows * kSum * 4u, kParts = 3u * kLowRankRows * kLine * 2u;
  // sums and parts lie where the waves' tiles do before and after
  __shared__ __attribute__((aligned(256))) uint8_t lds[kW * kMine > kSums + kParts ? kW * kMine : kSums + kParts];
  const uint32_t tid = threadIdx.x, lane = tid & 63u, i16 = lane & 15u, quarter = lane >> 4;
  const uint32_t wave = mx_first(tid >> 6);
  if (blockIdx.x == 0u) low_rank_report(p);
  uint32_t g, row0, row1, slab;
  if (!low_rank_tile(p, g, row0, row1, slab)) return;
  if (g >= p.adapters) {  // no adapter
    if (p.base != p.y) low_rank_bare<kF32>(p, row0, row1, slab * p.slab, min(p.n, (slab + 1u) * p.slab));
    return;
  }
  uint32_t c, n1;
  low_rank_share<kW>(wave, slab * p.slab, min(p.n, (slab + 1u) * p.slab), c, n1);
  Outer o;
  Inner in;
  in.rows(p, g, row0, row1);
  v4f acc[kF];
  uint32_t k0, k1;
  low_rank_share<kW>(wave, 0u, p.k, k0, k1);
  in.run(lds + wave * kMine, k0, k1, p.k, acc);
  o.rows(p, g, row0, row1);
  if (c < n1) {  // meanwhile
    o.load_b(p, c, 0u);
    o.load_base(p, c);
    loads_first();
  }
  __syncthreads();
  float* sums = reinterpret_cast<float*>(lds);
  typedef uint16_t Part[kLowRankRows][kLine];
  Part* parts = reinterpret_cast<Part*>(lds + kSums);
#pragma unroll
  for (uint32_t f = 0; f < kF; f++)
    *reinterpret_cast<v4f*>(sums + (wave * kLowRankRows + i16) * kSum + f * 16u + quarter * 4u) = acc[f];
  __syncthreads();
  const float s = p.scales ? p.scales[g] : 1.0f;
  for (uint32_t i = tid; i < kR * kLowRankRows; i += kLowRankThreads) {
    const uint32_t t = i / kR, r = i % kR;
    float sum = sums[t * kSum + r];
#pragma unroll
    for (uint32_t w = 1; w < kW; w++) sum += sums[(w * kLowRankRows + t) * kSum + r];
    uint16_t part[3];
    low_rank_split(r < p.rank ? s * sum : 0.0f, part);
#pragma unroll
    for (int j = 0; j < 3; j++) parts[j][t][r] = part[j];
  }
  __syncthreads();
  v8bf v[Outer::kSteps];
#pragma unroll
  for (uint32_t i = 0; i < Outer::kSteps; i++) {
    if constexpr (kF == 1u) {
      const uint32_t part = i * 2u + (quarter >> 1);
      v[i] = part < 3u ? *reinterpret_cast<const v8bf*>(&parts[part][i16][(quarter & 1u) * 8u])
                       : __builtin_bit_cast(v8bf, u32x4v{0u, 0u, 0u, 0u});
    } else {
      v[i] = *reinterpret_cast<const v8bf*>(&parts[i / Outer::kV][i16][i % Outer::kV * 32u + quarter * 8u]);
    }
  }
  __syncthreads();
  o.columns(p, lds + wave * kMine, v, c, n1);
}

// Column slabs of a row tile.  Every slab makes the tile's inner values again,
// so there are only as many as give each of the 256 CUs a workgroup, and no
// more: one workgroup too many takes the time of two.  Each list of rows ends in
// half a tile, about.  us with 1 slab, with as many as make up to 128, 256 and
// 512 workgroups (n, k, rank, tokens in adapters):
//   2,048 x 2,048, 16, 64 in 24      8.7   7.0   6.0   6.0
//   1,999 x 2,051, 24, 777 in 9     15.4  12.7  10.2  10.1
//   8,192 x 2,048, 16, 300 in 8     24.3  10.4   8.2   8.4
//   4,096 x 4,096, 32, 1,000 in 8   18.8  18.9  12.9  16.1
//   8,192 x 2,048, 64, 500 in 8     34.9  18.6  13.6  17.4
//   4,096 x 4,096, 64, 1,000 in 8   25.0  25.2  17.5  23.4
//   4,096 x 4,096, 128, 1,000 in 8  37.6  38.0  27.2  45.2
//   8,192 x 8,192, 128, 300 in 8    68.0  40.3  35.7  61.2
// How many adapters have rows is known on the device alone, so all of them count:
// 1,000 rows of 8 adapters, 4,096 x 4,096 at rank 64, take 17.9 us with 8 adapters
// held, 19.7 with 128 and 35.0 with 1,000.
// (Inner and outer product in launches of their own, the inner values in memory
// between them, took 4 to 10 us more than the best of these, but for the last:
// 29.)
uint32_t low_rank_slabs(uint64_t tokens, uint64_t lists, uint64_t n) {
  const uint64_t tiles = tokens / kLowRankRows + ((lists < tokens ? lists : tokens) + 1u) / 2u;
  const uint64_t most = cdiv(n, kLowRankSlab), fit = tiles ? 256u / tiles : 1u, want = fit ? fit : 1u;
  const uint64_t slab = cdiv(cdiv(n, want < most ? want : most), kLowRankSlab) * kLowRankSlab;
  return uint32_t(cdiv(n, slab));
}

}  // namespace

extern "C" {

uint64_t low_rank_workspace_size(uint64_t tokens, uint64_t n, uint64_t k, uint64_t rank, uint32_t adapters) {
  if (tokens > kMxMaxRows || n == 0u || n > kMxMaxCols || k == 0u || k > kMxMaxCols || rank == 0u || rank > kLowRankMax ||
      adapters == 0u || adapters > kMxMaxGroups)
    return 0u;
  return kMxWsHead;
}

ciera_status low_rank_add(const void* d_x, uint64_t ldx, const void* d_a, const void* d_b, const float* d_scales,
                          const int64_t* d_offsets, const int32_t* d_order, const void* d_base, uint64_t ldb,
                          uint32_t base_f32, void* d_y, uint64_t ldy, uint32_t y_f32, uint64_t tokens, uint64_t n,
                          uint64_t k, uint64_t rank, uint32_t adapters, void* d_ws, uint64_t ws_bytes,
                          hipStream_t stream) {
  const uint64_t need = low_rank_workspace_size(tokens, n, k, rank, adapters);
  if (!need || base_f32 > 1u || y_f32 > 1u || !d_ws || !aligned16(d_ws)) return CIERA_ERR_ARG;
  ciera_status st = mx_matrix(d_x, tokens, k, ldx, 2u);
  if (st == CIERA_OK) st = mx_matrix(d_y, tokens, n, ldy, y_f32 ? 4u : 2u);
  if (st == CIERA_OK && d_base) st = mx_matrix(d_base, tokens, n, ldb, base_f32 ? 4u : 2u);
  if (st == CIERA_OK) st = norm_vector(d_a, 2u);
  if (st == CIERA_OK) st = norm_vector(d_b, 2u);
  if (st == CIERA_OK) st = norm_vector(d_offsets, 8u);
  if (st == CIERA_OK && d_scales) st = norm_vector(d_scales, 4u);
  if (st == CIERA_OK && d_order) st = norm_vector(d_order, 4u);
  if (st == CIERA_OK && d_base == d_y && d_base && (base_f32 != y_f32 || ldb != ldy)) st = CIERA_ERR_ARG;
  if (st != CIERA_OK) return st;
  if (ws_bytes < need) return CIERA_ERR_WORKSPACE;
  LowRankArgs p{};
  p.x = static_cast<const uint16_t*>(d_x);
  p.ldx = ldx;
  p.a = static_cast<const uint16_t*>(d_a);
  p.b = static_cast<const uint16_t*>(d_b);
  p.scales = d_scales;
  p.offsets = d_offsets;
  p.order = d_order;
  p.base = d_base;
  p.ldb = ldb;
  p.y = d_y;
  p.ldy = ldy;
  p.ctrl = static_cast<Ctrl*>(d_ws);
  p.status = reinterpret_cast<uint32_t*>(static_cast<uint8_t*>(d_ws) + sizeof(Ctrl));
  p.tokens = uint32_t(tokens);
  p.n = uint32_t(n);
  p.k = uint32_t(k);
  p.rank = uint32_t(rank);
  p.adapters = adapters;
  p.base_f32 = base_f32;
  p.y_f32 = y_f32;
  // every list of rows may end in a part of a tile
  const uint64_t lists = adapters + 2ull;
  const uint64_t tiles = tokens / kLowRankRows + (lists < tokens ? lists : tokens);
  p.slabs = low_rank_slabs(tokens, lists, n);
  p.slab = uint32_t(cdiv(cdiv(n, p.slabs), kLowRankSlab) * kLowRankSlab);
  const uint64_t grid = tiles ? tiles * p.slabs : 1u;
  if (grid > 0xFFFFFFFFull / kLowRankThreads) return CIERA_ERR_ARG;
  const auto go = [&](auto frags) {
    constexpr uint32_t kF = decltype(frags)::value;
    const dim3 g(static_cast<uint32_t>(grid)), block(kLowRankThreads);
    (void)hipGetLastError();
    if (base_f32) launch(k_low_rank<kF, true>, g, block, stream, p);
    else launch(k_low_rank<kF, false>, g, block, stream, p);
    return launch_status();
  };
  if (rank <= 16u) return go(std::integral_constant<uint32_t, 1u>());
  if (rank <= 32u) return go(std::integral_constant<uint32_t, 2u>());
  if (rank <= 64u) return go(std::integral_constant<uint32_t, 4u>());
  return go(std::integral_constant<uint32_t, 8u>());
}

}  // extern "C"
