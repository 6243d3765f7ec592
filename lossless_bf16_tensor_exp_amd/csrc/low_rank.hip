// low_rank.hip -- low-rank adapters of many requests beside a projection that
// they share, gfx950:
//
//   y_t = base_t + s_a B_a (A_a x_t),   a the adapter of row t
//
// A_a is rank x k, B_a n x rank.  Rows come sorted by adapter, as the experts'
// do: rows offsets[a] .. offsets[a+1] - 1 of the order are adapter a's, those
// before the first and behind the last have none and take base alone.
//
// One launch: a workgroup takes 16 rows of one adapter and a slab of the
// columns.  It makes the rows' inner values v = s_a A_a x (16 x rank, the
// contraction spread over its waves, FP32 sums joined in LDS), and from them
// its columns.  v then goes through the BF16 matrix instructions as three BF16
// parts that hold its 24 significant bits, so that nothing is rounded between
// the two products.
#include "ciera.h"

namespace {

constexpr uint32_t kLowRankMax = 128u;
constexpr uint32_t kLowRankRows = 16u;

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
  uint32_t r0 = 0u, r1 = 0u, sum = 0u, total = 0u;
  for (uint32_t c = 0; c < lists; c += 64u) {
    low_rank_rows(p, c + lane, r0, r1);
    total += uint32_t(__builtin_amdgcn_readlane(int(mx_scan((r1 - r0 + kLowRankRows - 1u) / kLowRankRows)), 63));
  }
  if (blockIdx.x >= total * p.slabs) return false;
  const uint32_t at = mx_xcd_run(blockIdx.x, total * p.slabs), tile = at / p.slabs;
  slab = at - tile * p.slabs;
  uint32_t before = 0u;
  for (uint32_t c = 0; c < lists; c += 64u) {
    low_rank_rows(p, c + lane, r0, r1);
    const uint32_t own = (r1 - r0 + kLowRankRows - 1u) / kLowRankRows;
    sum = mx_scan(own);
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

// Sixteen neighbouring columns of a row: base, or zeros without one.
__device__ __forceinline__ void low_rank_base(const LowRankArgs& p, uint64_t row, uint32_t col, float (&v)[16]) {
  if (!p.base || col >= p.n) {
#pragma unroll
    for (int i = 0; i < 16; i++) v[i] = 0.0f;
    return;
  }
#pragma unroll
  for (uint32_t h = 0; h < 2u; h++) {
    float e[8];
    if (p.base_f32) row_values8<true>(p.base, row * p.ldb, col + 8u * h, p.n, e);
    else row_values8<false>(p.base, row * p.ldb, col + 8u * h, p.n, e);
#pragma unroll
    for (uint32_t i = 0; i < 8u; i++) v[8u * h + i] = e[i];
  }
}
__device__ __forceinline__ void low_rank_store(const LowRankArgs& p, uint64_t row, uint32_t col, const float (&v)[16]) {
#pragma unroll
  for (uint32_t h = 0; h < 2u; h++) {
    const uint32_t c = col + 8u * h;
    const float* e = v + 8u * h;
    if (p.y_f32) {
      float* o = static_cast<float*>(p.y) + row * p.ldy + c;
      if (c + 8u <= p.n) {
        *reinterpret_cast<v4fa4*>(o) = v4f{e[0], e[1], e[2], e[3]};
        *reinterpret_cast<v4fa4*>(o + 4) = v4f{e[4], e[5], e[6], e[7]};
      } else {
#pragma unroll
        for (uint32_t i = 0; i < 7u; i++)
          if (c + i < p.n) o[i] = e[i];
      }
    } else {
      row_store8(static_cast<uint16_t*>(p.y) + row * p.ldy, c, p.n,
                 u32x4v{mx_bf16x2(e[0], e[1]), mx_bf16x2(e[2], e[3]), mx_bf16x2(e[4], e[5]), mx_bf16x2(e[6], e[7])});
    }
  }
}

// v as three BF16 numbers whose sum it is: its leading 8 significant bits, the
// next 8 and the last.  Cut, not rounded, so that none passes BF16's range;
// an infinity or a NaN is the first alone.
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

// kF: fragments of 16 ranks (1, 2, 4 or 8).
template <uint32_t kF>
__global__ __launch_bounds__(256) void k_low_rank(LowRankArgs p) {
  constexpr uint32_t kR = kF * 16u;              // ranks, zeros behind the real ones
  constexpr uint32_t kLine = (kF == 1u ? 16u : kR) + 8u;  // of a row's parts in LDS, 16 bytes more for the banks
  __shared__ float sums[4][kR][kLowRankRows];
  __shared__ __attribute__((aligned(16))) uint16_t parts[3][kLowRankRows][kLine];
  const uint32_t tid = threadIdx.x, lane = tid & 63u, i16 = lane & 15u, quarter = lane >> 4;
  const uint32_t wave = mx_first(tid >> 6);
  if (blockIdx.x == 0u) low_rank_report(p);
  uint32_t g, row0, row1, slab;
  if (!low_rank_tile(p, g, row0, row1, slab)) return;
  const uint32_t n0 = slab * p.slab, n1 = min(p.n, n0 + p.slab);
  const uint32_t slot = min(row0 + i16, row1 - 1u);
  const uint32_t named = p.order ? uint32_t(p.order[slot]) : slot;
  const bool live = row0 + i16 < row1 && named < p.tokens;
  const uint64_t row = named < p.tokens ? named : 0u;
  float v[16];
  if (g >= p.adapters) {  // no adapter
    if (p.base == p.y) return;
    for (uint32_t c = n0 + wave * 64u; c < n1; c += 256u) {
      low_rank_base(p, row, c + quarter * 16u, v);
      if (live) low_rank_store(p, row, c + quarter * 16u, v);
    }
    return;
  }

  // v = A x: lanes hold 16 neighbouring values of k, of a rank and of a row,
  // for two matrix instructions (the contraction's order is the same for both
  // operands); the waves take turns of 64
  const uint16_t* a = p.a + uint64_t(g) * p.rank * p.k;
  const uint16_t* x = p.x + row * p.ldx;
  v4f acc[kF];
#pragma unroll
  for (uint32_t f = 0; f < kF; f++) acc[f] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll 2
  for (uint32_t c = wave * 64u; c < p.k; c += 256u) {
    const uint32_t at = c + quarter * 16u;
    const v8bf x0 = __builtin_bit_cast(v8bf, row_load8(x, at, p.k)), x1 = __builtin_bit_cast(v8bf, row_load8(x, at + 8u, p.k));
#pragma unroll
    for (uint32_t f = 0; f < kF; f++) {
      const uint16_t* ar = a + uint64_t(min(f * 16u + i16, p.rank - 1u)) * p.k;
      acc[f] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(v8bf, row_load8(ar, at, p.k)), x0, acc[f], 0, 0, 0);
      acc[f] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(v8bf, row_load8(ar, at + 8u, p.k)), x1, acc[f], 0, 0, 0);
    }
  }
#pragma unroll
  for (uint32_t f = 0; f < kF; f++)
#pragma unroll
    for (uint32_t r = 0; r < 4u; r++) sums[wave][f * 16u + quarter * 4u + r][i16] = acc[f][r];
  __syncthreads();
  const float s = p.scales ? p.scales[g] : 1.0f;
#pragma unroll
  for (uint32_t i = 0; i < kF; i++) {
    const uint32_t r = i * 16u + (tid >> 4);
    const float sum = s * (sums[0][r][i16] + sums[1][r][i16] + sums[2][r][i16] + sums[3][r][i16]);
    uint16_t part[3];
    low_rank_split(r < p.rank ? sum : 0.0f, part);
#pragma unroll
    for (int j = 0; j < 3; j++) parts[j][i16][r] = part[j];
  }
  __syncthreads();

  // y = base + B v.  Row i of fragment f is column 16 (i / 4) + 4 f + i % 4 of
  // the wave's 64, so that a lane's sums of four fragments are 16 neighbours.
  // 16 ranks fill half an instruction: the other half takes the next part.
  constexpr uint32_t kSteps = kF == 1u ? 2u : kF / 2u * 3u;
  v8bf bv[kSteps];
#pragma unroll
  for (uint32_t i = 0; i < kSteps; i++) {
    if constexpr (kF == 1u) {
      const uint32_t part = i * 2u + (quarter >> 1);
      bv[i] = part < 3u ? *reinterpret_cast<const v8bf*>(&parts[part][i16][(quarter & 1u) * 8u])
                        : __builtin_bit_cast(v8bf, u32x4v{0u, 0u, 0u, 0u});
    } else {
      bv[i] = *reinterpret_cast<const v8bf*>(&parts[i / (kF / 2u)][i16][i % (kF / 2u) * 32u + quarter * 8u]);
    }
  }
  const uint16_t* b = p.b + uint64_t(g) * p.n * p.rank;
  for (uint32_t c = n0 + wave * 64u; c < n1; c += 256u) {
    const uint32_t col = c + quarter * 16u;
    low_rank_base(p, row, col, v);
#pragma unroll
    for (uint32_t f = 0; f < 4u; f++) {
      const uint16_t* br = b + uint64_t(min(c + (i16 >> 2) * 16u + f * 4u + (i16 & 3u), p.n - 1u)) * p.rank;
      v4f sum = {0.0f, 0.0f, 0.0f, 0.0f};
      if constexpr (kF == 1u) {
        const v8bf w = __builtin_bit_cast(v8bf, row_load8(br, (quarter & 1u) * 8u, p.rank));
        sum = __builtin_amdgcn_mfma_f32_16x16x32_bf16(w, bv[1], sum, 0, 0, 0);
        sum = __builtin_amdgcn_mfma_f32_16x16x32_bf16(w, bv[0], sum, 0, 0, 0);
      } else {
        v8bf w[kF / 2u];
#pragma unroll
        for (uint32_t i = 0; i < kF / 2u; i++) w[i] = __builtin_bit_cast(v8bf, row_load8(br, i * 32u + quarter * 8u, p.rank));
#pragma unroll
        for (uint32_t i = kSteps; i > 0u; i--)
          sum = __builtin_amdgcn_mfma_f32_16x16x32_bf16(w[(i - 1u) % (kF / 2u)], bv[i - 1u], sum, 0, 0, 0);
      }
#pragma unroll
      for (uint32_t r = 0; r < 4u; r++) v[f * 4u + r] += sum[r];
    }
    if (live) low_rank_store(p, row, col, v);
  }
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
  p.slab = 512u;
  p.slabs = uint32_t(cdiv(n, p.slab));
  const uint64_t grid = tiles ? tiles * p.slabs : 1u;
  if (grid > kMxMostGroups) return CIERA_ERR_ARG;
  (void)hipGetLastError();
  const dim3 g(static_cast<uint32_t>(grid)), block(256);
  if (rank <= 16u) launch(k_low_rank<1u>, g, block, stream, p);
  else if (rank <= 32u) launch(k_low_rank<2u>, g, block, stream, p);
  else if (rank <= 64u) launch(k_low_rank<4u>, g, block, stream, p);
  else launch(k_low_rank<8u>, g, block, stream, p);
  return launch_status();
}

}  // extern "C"
