// experts.hip -- rows of tokens brought to their experts and back, gfx950.
//
// ids[t][j] is the expert of token t's j-th choice, an entry; -1 for none.
//   sort      offsets[e] = entries of experts below e; place[i] = offsets[e_i]
//             + entries of e_i before i (-1 without expert); order[place[i]] =
//             i, and behind the last expert's the entries without one, in order
//   dispatch  out[place[t][j]] = x[t], in BF16 or mx8
//   combine   out[t] = residual[t] + sum_j w[t][j] rows[place[t][j]]
//   backward  drows[place[t][j]] = w[t][j] dout[t];
//             dw[t][j] = <dout[t], rows[place[t][j]]>
// Entries without a row add nothing and are not read; rows of no entry are not
// written.  Sums are FP32 and in the order of the choices (dw: an order that
// depends on the sizes only); every output is rounded once.
#include "ciera.h"

namespace {

constexpr uint32_t kMaxChoices = 64u;
constexpr uint64_t kMaxEntries = (1ull << 31) - 1u;
constexpr uint32_t kSortWords = 16u * 1024u + 64u;  // of LDS: a count for each wave and bin
constexpr uint32_t kSortBlocks = 256u;

// A sort goes in blocks of 2,048 entries, up to kSortBlocks of them and fewer for
// many experts: every block reads the counts of all of them.  us with a block
// for each 1,024, 2,048 and 4,096 entries, of 64 experts: 32,768 entries 8.2, 8.4,
// 11.5; 262,144 13.9, 11.2, 11.0.  Few entries go in one block, and one launch:
// 4,096 of them 6.6 instead of 8.3.
uint32_t sort_blocks(uint64_t entries, uint32_t experts) {
  uint64_t b = entries < 6144u ? 1u : cdiv(entries, 2048u);
  const uint64_t most = 65536u / (experts + 1u);
  if (b > most) b = most;
  if (b > kSortBlocks) b = kSortBlocks;
  return b < 1u ? 1u : uint32_t(b);
}
constexpr uint32_t sort_waves(uint32_t experts) { return experts < 1024u ? 16u : 4u; }

struct SortArgs {
  const void* ids;
  int64_t* offsets;
  int32_t* place;
  int32_t* order;
  uint32_t* counts;  // blocks x (experts + 1), then a word a block: whether it met a bad id
  Ctrl* ctrl;
  uint32_t* status;
  uint32_t entries, experts, blocks, per;  // per: entries a block
};

// Bins of this lane's entries in the kSortSteps steps of 64 from `at` on: their
// experts, `experts` for none, and experts + 1 behind the stretch's end.  A
// number that is no expert's and not -1 goes with none and is reported.  The
// steps' loads go out together.
constexpr uint32_t kSortSteps = 4u;
template <bool kWide>
__device__ __forceinline__ void sort_bins(const SortArgs& p, uint32_t at, uint32_t to, uint32_t (&bin)[kSortSteps], bool& bad) {
  typedef typename std::conditional<kWide, int64_t, int32_t>::type Id;
  Id e[kSortSteps];
#pragma unroll
  for (uint32_t k = 0; k < kSortSteps; k++) e[k] = static_cast<const Id*>(p.ids)[min(at + k * 64u + (threadIdx.x & 63u), to - 1u)];
  loads_first();
#pragma unroll
  for (uint32_t k = 0; k < kSortSteps; k++) {
    const bool in = e[k] >= 0 && e[k] < Id(p.experts), there = at + k * 64u + (threadIdx.x & 63u) < to;
    bad = bad || (!in && e[k] != -1);
    bin[k] = !there ? p.experts + 1u : in ? uint32_t(e[k]) : p.experts;
  }
}

// Entries of each bin among this wave's, into its row of counts.
template <bool kWide>
__device__ __forceinline__ bool sort_count(const SortArgs& p, uint32_t from, uint32_t to, uint32_t* count) {
  bool bad = false;
  for (uint32_t at = from; at < to; at += 64u * kSortSteps) {
    uint32_t bin[kSortSteps];
    sort_bins<kWide>(p, at, to, bin, bad);
#pragma unroll
    for (uint32_t k = 0; k < kSortSteps; k++)
      if (bin[k] <= p.experts) atomicAdd(count + bin[k], 1u);
  }
  return bad;
}

// This wave's entries: its share of the block's, in order.
__device__ __forceinline__ void sort_share(const SortArgs& p, uint32_t& from, uint32_t& to) {
  const uint32_t waves = blockDim.x >> 6, wave = threadIdx.x >> 6;
  const uint32_t lo = min(blockIdx.x * p.per, p.entries), hi = min(lo + p.per, p.entries);
  const uint32_t each = ((hi - lo + waves - 1u) / waves + 63u) & ~63u;  // whole steps
  from = min(lo + wave * each, hi);
  to = min(from + each, hi);
}

template <bool kWide>
__global__ __launch_bounds__(1024) void k_sort_count(SortArgs p) {
  __shared__ uint32_t count[4097];
  __shared__ uint32_t any;
  const uint32_t bins = p.experts + 1u;
  for (uint32_t b = threadIdx.x; b < bins; b += blockDim.x) count[b] = 0u;
  if (threadIdx.x == 0u) any = 0u;
  __syncthreads();
  uint32_t from, to;
  sort_share(p, from, to);
  if (sort_count<kWide>(p, from, to, count)) any = 1u;
  __syncthreads();
  for (uint32_t b = threadIdx.x; b < bins; b += blockDim.x) p.counts[uint64_t(blockIdx.x) * bins + b] = count[b];
  if (threadIdx.x == 0u) p.counts[uint64_t(p.blocks) * bins + blockIdx.x] = any;
}

// Bound by launches and by dependent steps: 32,768 entries of 64 experts 4.7 us
// for the counts and 5.4 here (medians of a profiler's trace), of which 2.5 are
// each one's launch.
// Each wave takes a stretch of the entries and counts it; the counts become
// the places where the wave's entries of each bin begin; then the wave goes
// through its stretch again, 64 entries a step.  Lanes of one bin find each
// other with a ballot for each bit of the bin's number; the first of them
// draws their places.
template <bool kWide>
__global__ __launch_bounds__(1024) void k_expert_sort(SortArgs p) {
  __shared__ uint32_t count[kSortWords];
  __shared__ uint32_t sums[16];
  __shared__ uint32_t any;
  const uint32_t tid = threadIdx.x, threads = blockDim.x, lane = tid & 63u, wave = tid >> 6, waves = threads >> 6;
  const uint32_t bins = p.experts + 1u;
  for (uint32_t i = tid; i < waves * bins; i += threads) count[i] = 0u;
  if (tid == 0u) any = 0u;
  __syncthreads();
  uint32_t from, to;
  sort_share(p, from, to);
  uint32_t* mine = count + wave * bins;
  const bool bad = sort_count<kWide>(p, from, to, mine);
  if (p.blocks == 1u && bad) any = 1u;
  if (p.blocks > 1u && blockIdx.x == 0u)
    for (uint32_t b = tid; b < p.blocks; b += threads)
      if (p.counts[uint64_t(p.blocks) * bins + b]) any = 1u;
  __syncthreads();
  uint32_t before = 0u;  // entries of the bins so far
  for (uint32_t c = 0; c < bins; c += threads) {
    const uint32_t b = c + tid;
    uint32_t all = 0u, earlier = 0u;
    if (b < bins) {
      if (p.blocks == 1u) {
        for (uint32_t w = 0; w < waves; w++) all += count[w * bins + b];
      } else {
#pragma unroll 16
        for (uint32_t k = 0; k < p.blocks; k++) {
          const uint32_t n = p.counts[uint64_t(k) * bins + b];
          all += n;
          if (k < blockIdx.x) earlier += n;
        }
      }
    }
    const uint32_t sum = wave_incl_scan(all);
    if (lane == 63u) sums[wave] = sum;
    __syncthreads();
    uint32_t at = before + sum - all, total = 0u;
    for (uint32_t w = 0; w < waves; w++) {
      if (w < wave) at += sums[w];
      total += sums[w];
    }
    before += total;
    if (b < bins) {
      if (blockIdx.x == 0u) p.offsets[b] = int64_t(at);  // the bin of none begins where the last expert's end
      at += earlier;
      for (uint32_t w = 0; w < waves; w++) {
        const uint32_t n = count[w * bins + b];
        count[w * bins + b] = at;
        at += n;
      }
    }
    __syncthreads();
  }
  const uint32_t bits = 32u - uint32_t(__clz(int(bins)));
  for (uint32_t i0 = from; i0 < to; i0 += 64u * kSortSteps) {
    uint32_t bin[kSortSteps];
    bool ignored = false;
    sort_bins<kWide>(p, i0, to, bin, ignored);
#pragma unroll
    for (uint32_t k = 0; k < kSortSteps; k++) {
      if (i0 + k * 64u >= to) break;
      const uint32_t b = bin[k], i = i0 + k * 64u + lane;
      uint64_t same = ~0ull;
      for (uint32_t j = 0; j < bits; j++) {
        const uint64_t set = __ballot((b >> j) & 1u);
        same &= ((b >> j) & 1u) ? set : ~set;
      }
      const uint32_t rank = uint32_t(__popcll(same & ((1ull << lane) - 1u)));
      uint32_t first = 0u;
      if (rank == 0u && b < bins) first = atomicAdd(mine + b, uint32_t(__popcll(same)));
      first = uint32_t(__shfl(int(first), __ffsll((unsigned long long)same) - 1));
      if (b < bins) {
        const uint32_t at = first + rank;
        p.place[i] = b < p.experts ? int32_t(at) : -1;
        if (p.order) p.order[at] = int32_t(i);
      }
    }
  }
  if (blockIdx.x == 0u && tid == 0u) {
    p.ctrl->n_err_slots = 1u;
    *p.status = any ? uint32_t(CIERA_ERR_ARG) : uint32_t(CIERA_OK);
  }
}

// ---------------------------------------------------------------------------
// The rows.  A token takes 1 << lt threads, each a unit of 8 values; a workgroup
// of 256 holds 256 >> lt tokens.  Rows longer than a workgroup go on in the
// grid's second dimension (backward, which sums over a row: in a loop).
// ---------------------------------------------------------------------------
struct RowArgs {
  const uint16_t* x;  // dispatch: the tokens; backward: dout
  uint64_t ldx;
  const void* rows;   // combine, backward: the experts' rows, BF16 or FP32
  uint64_t ldrows;
  const int32_t* place;
  const float* weights;
  const uint16_t* residual;
  uint64_t ldr;
  void* out;          // dispatch: rows; combine: tokens; backward: drows
  uint64_t ldo;
  uint8_t* q;         // dispatch: rows in mx8
  uint8_t* qs;
  float* dweights;
  uint32_t out_f32, tokens, choices, cols, slots, lt;
};

// The token of this thread and its place in the token's row.  With a wave or
// more a token its number is the same in all lanes, and is kept so.
template <bool kWave>
__device__ __forceinline__ uint32_t row_token(const RowArgs& p, uint32_t& t) {
  t = threadIdx.x & ((1u << p.lt) - 1u);
  const uint32_t sub = threadIdx.x >> p.lt;
  return blockIdx.x * (256u >> p.lt) + (kWave ? mx_first(sub) : sub);
}

// A token's row is read, and made mx8, once and written for every choice.  Bound
// by memory: 4,096 x 8 choices of 2,048 in mx8, 86 MB: 15.7 us, 5.5 TB/s; in
// BF16, 151 MB: 29.6 us (26 past the last-level cache, but then the product that
// follows has to fetch them: mx8's reader took 34 us instead of 29).
template <bool kWave>
__global__ __launch_bounds__(256) void k_dispatch(RowArgs p) {
  uint32_t t;
  const uint32_t token = row_token<kWave>(p, t);
  if (token >= p.tokens) return;
  const uint16_t* x = p.x + uint64_t(token) * p.ldx;
  const int32_t* place = p.place + uint64_t(token) * p.choices;
  const uint32_t kp = uint32_t(mx_pitch(p.cols));
  const uint32_t col = (blockIdx.y << p.lt | t) * 8u;
  if (col < (p.q ? kp : p.cols)) {
    const u32x4v v = row_get8<!kWave>(x, col, p.cols);
    u32x2v codes = {0u, 0u};
    uint32_t sb = 0u;
    if (p.q) {
      u32x4v e = v;
      sb = mx_block_scale<8>(e);
      codes = mx8_codes(e, mx_scale(sb == 255u ? 127u : sb));
    }
    for (uint32_t j = 0; j < p.choices; j++) {
      const uint32_t at = uint32_t(place[j]);
      if (at >= p.slots) continue;
      if (p.out) row_store8(static_cast<uint16_t*>(p.out) + uint64_t(at) * p.ldo, col, p.cols, v);
      if (p.q) {
        *reinterpret_cast<u32x2v*>(p.q + uint64_t(at) * kp + col) = codes;
        if ((t & 3u) == 0u) p.qs[uint64_t(at) * (kp / 32u) + col / 32u] = uint8_t(sb);
      }
    }
  }
}

// Eight values of a BF16 or FP32 row, zeros behind its end: all loads first, as
// row_load8 and row_mend8.
template <bool kF32, bool kTiny = true>
struct Row8 {
  u32x4v lo, hi;  // BF16: lo alone
  template <bool kStream = false>
  __device__ __forceinline__ void load(const void* rows, uint64_t at, uint32_t col, uint32_t cols) {
    if constexpr (kF32) {
      const float* r = static_cast<const float*>(rows) + at;
      if (kTiny && cols < 8u) {
        lo = hi = u32x4v{0u, 0u, 0u, 0u};
#pragma unroll
        for (uint32_t i = 0; i < 4u; i++) {
          if (col + i < cols) lo[i] = __float_as_uint(r[col + i]);
          if (col + 4u + i < cols) hi[i] = __float_as_uint(r[col + 4u + i]);
        }
      } else {
        const float* f = r + min(col, cols - 8u);
        const v4fa4 *a = reinterpret_cast<const v4fa4*>(f), *b = reinterpret_cast<const v4fa4*>(f + 4);
        lo = __builtin_bit_cast(u32x4v, kStream ? v4f(__builtin_nontemporal_load(a)) : v4f(*a));
        hi = __builtin_bit_cast(u32x4v, kStream ? v4f(__builtin_nontemporal_load(b)) : v4f(*b));
      }
    } else {
      lo = row_load8<kStream, kTiny>(static_cast<const uint16_t*>(rows) + at, col, cols);
    }
  }
  __device__ __forceinline__ void mend(uint32_t col, uint32_t cols) {
    if constexpr (kF32) {
      if (col + 8u <= cols || (kTiny && cols < 8u)) return;
      const uint32_t by = col - (cols - 8u);
      const u32x4v none = {0u, 0u, 0u, 0u};
      if (by & 4u) lo = hi, hi = none;
      if (by & 2u) lo = u32x4v{lo[2], lo[3], hi[0], hi[1]}, hi = u32x4v{hi[2], hi[3], 0u, 0u};
      if (by & 1u) lo = u32x4v{lo[1], lo[2], lo[3], hi[0]}, hi = u32x4v{hi[1], hi[2], hi[3], 0u};
      if (by >= 8u) lo = hi = none;
    } else {
      row_mend8<kTiny>(lo, col, cols);
    }
  }
  __device__ __forceinline__ float value(int i) const {
    if constexpr (kF32) return __uint_as_float(i < 4 ? lo[i] : hi[i - 4]);
    else return i & 1 ? bf_hi(lo[i / 2]) : bf_lo(lo[i / 2]);
  }
};

constexpr uint32_t kRowsAtOnce = 4u;  // of a token's, all their loads in flight (8: the same for combine, 6 % more backward)

// Bound by memory: 4,096 x 8 rows of 2,048 onto the residual, 168 MB: 30 us, 5.6
// TB/s; the rows, read once, go past the last-level cache (36 us through it).  A
// workgroup a token: with a wave a token and four units a lane 43 us.

template <bool kWave, bool kF32>
__global__ __launch_bounds__(256) void k_combine(RowArgs p) {
  uint32_t t;
  const uint32_t token = row_token<kWave>(p, t);
  if (token >= p.tokens) return;
  const int32_t* place = p.place + uint64_t(token) * p.choices;
  const float* weights = p.weights ? p.weights + uint64_t(token) * p.choices : nullptr;
  const uint32_t col = (blockIdx.y << p.lt | t) * 8u;
  if (col < p.cols) {
    float sum[8];
    Row8<false, !kWave> r;
    if (p.residual) r.load(p.residual, uint64_t(token) * p.ldr, col, p.cols);
    for (uint32_t j0 = 0; j0 < p.choices; j0 += kRowsAtOnce) {
      Row8<kF32, !kWave> v[kRowsAtOnce];
      float w[kRowsAtOnce];
      bool has[kRowsAtOnce];
#pragma unroll
      for (uint32_t i = 0; i < kRowsAtOnce; i++) {
        const uint32_t at = j0 + i < p.choices ? uint32_t(place[j0 + i]) : ~0u;
        has[i] = at < p.slots;
        w[i] = has[i] && weights ? weights[j0 + i] : 1.0f;
        if (has[i]) v[i].template load<kWave>(p.rows, uint64_t(at) * p.ldrows, col, p.cols);
      }
      loads_first();
      if (j0 == 0u) {
        if (p.residual) r.mend(col, p.cols);
#pragma unroll
        for (int c = 0; c < 8; c++) sum[c] = p.residual ? r.value(c) : 0.0f;
      }
#pragma unroll
      for (uint32_t i = 0; i < kRowsAtOnce; i++)
        if (has[i]) {
          v[i].mend(col, p.cols);
#pragma unroll
          for (int c = 0; c < 8; c++) sum[c] = fmaf(w[i], v[i].value(c), sum[c]);
        }
    }
    const uint64_t to = uint64_t(token) * p.ldo;
    if (p.out_f32) {
      float* o = static_cast<float*>(p.out) + to + col;
      if (col + 8u <= p.cols) {
        *reinterpret_cast<v4fa4*>(o) = v4f{sum[0], sum[1], sum[2], sum[3]};
        *reinterpret_cast<v4fa4*>(o + 4) = v4f{sum[4], sum[5], sum[6], sum[7]};
      } else {
#pragma unroll
        for (uint32_t i = 0; i < 7u; i++)
          if (col + i < p.cols) o[i] = sum[i];
      }
    } else {
      row_store8(static_cast<uint16_t*>(p.out) + to, col, p.cols,
                 u32x4v{mx_bf16x2(sum[0], sum[1]), mx_bf16x2(sum[2], sum[3]), mx_bf16x2(sum[4], sum[5]), mx_bf16x2(sum[6], sum[7])});
    }
  }
}

// dout is read again for each kRowsAtOnce of the choices (from L2).  Bound by
// memory: 4,096 x 8 rows of 2,048, 286 MB: 55 us, 5.2 TB/s; rows and their
// gradients go past the last-level cache (62 us through it).  With fewer choices
// than kRowsAtOnce fewer loads are in flight behind each barrier: 16,384 x 2 rows
// 62 us on 54 for the bytes, 32,768 x 1 96 on 64.
template <bool kWave, bool kF32>
__global__ __launch_bounds__(256) void k_combine_back(RowArgs p) {
  __shared__ float part[2][4][kRowsAtOnce];
  uint32_t t;
  const uint32_t token = row_token<kWave>(p, t);
  const bool live = token < p.tokens;
  const int32_t* place = p.place + uint64_t(live ? token : 0u) * p.choices;
  const float* weights = p.weights ? p.weights + uint64_t(live ? token : 0u) * p.choices : nullptr;
  const uint16_t* x = p.x + uint64_t(live ? token : 0u) * p.ldx;
  const uint32_t span = min(1u << p.lt, 64u);
  for (uint32_t j0 = 0, turn = 0; j0 < p.choices; j0 += kRowsAtOnce, turn ^= 1u) {
    uint32_t at[kRowsAtOnce];
    float w[kRowsAtOnce], dot[kRowsAtOnce];
#pragma unroll
    for (uint32_t i = 0; i < kRowsAtOnce; i++) {
      at[i] = live && j0 + i < p.choices ? uint32_t(place[j0 + i]) : ~0u;
      w[i] = at[i] < p.slots && weights ? weights[j0 + i] : 1.0f;
      dot[i] = 0.0f;
    }
    for (uint32_t col = t * 8u; live && col < p.cols; col += 8u << p.lt) {
      Row8<false, !kWave> d;
      Row8<kF32, !kWave> v[kRowsAtOnce];
      d.load(x, 0u, col, p.cols);
      if (p.dweights) {
#pragma unroll
        for (uint32_t i = 0; i < kRowsAtOnce; i++)
          if (at[i] < p.slots) v[i].template load<kWave>(p.rows, uint64_t(at[i]) * p.ldrows, col, p.cols);
      }
      loads_first();
      d.mend(col, p.cols);
      if (p.out) {
#pragma unroll
        for (uint32_t i = 0; i < kRowsAtOnce; i++)
          if (at[i] < p.slots) {
            u32x4v o;
#pragma unroll
            for (int c = 0; c < 4; c++) o[c] = mx_bf16x2(w[i] * d.value(2 * c), w[i] * d.value(2 * c + 1));
            row_store8<kWave>(static_cast<uint16_t*>(p.out) + uint64_t(at[i]) * p.ldo, col, p.cols, o);
          }
      }
      if (p.dweights) {
#pragma unroll
        for (uint32_t i = 0; i < kRowsAtOnce; i++)
          if (at[i] < p.slots) {
            v[i].mend(col, p.cols);
#pragma unroll
            for (int c = 0; c < 8; c++) dot[i] = fmaf(d.value(c), v[i].value(c), dot[i]);
          }
      }
    }
    if (!p.dweights) continue;
    for (uint32_t s = span >> 1; s > 0u; s >>= 1)
#pragma unroll
      for (uint32_t i = 0; i < kRowsAtOnce; i++) dot[i] += __shfl_xor(dot[i], int(s));
    if (p.lt > 6u) {
      if ((threadIdx.x & 63u) == 0u)
#pragma unroll
        for (uint32_t i = 0; i < kRowsAtOnce; i++) part[turn][threadIdx.x >> 6][i] = dot[i];
      __syncthreads();
      const uint32_t waves = 1u << (p.lt - 6u), w0 = threadIdx.x >> 6 & ~(waves - 1u);
#pragma unroll
      for (uint32_t i = 0; i < kRowsAtOnce; i++) {
        dot[i] = 0.0f;
        for (uint32_t k = 0; k < waves; k++) dot[i] += part[turn][w0 + k][i];
      }
    }
    if (live && t == 0u)
#pragma unroll
      for (uint32_t i = 0; i < kRowsAtOnce; i++)
        if (j0 + i < p.choices) p.dweights[uint64_t(token) * p.choices + j0 + i] = at[i] < p.slots ? dot[i] : 0.0f;
  }
}

// log2 of the threads a token takes: a unit each, at least a block of mx8 and
// at most a workgroup.
uint32_t row_threads(uint64_t cols) {
  uint32_t lt = 2u;
  while (lt < 8u && (8ull << lt) < cols) lt++;
  return lt;
}

ciera_status row_common(RowArgs& p, const int32_t* d_place, uint64_t tokens, uint64_t choices, uint64_t cols, uint64_t slots) {
  if (choices == 0u || choices > kMaxChoices || tokens > kMxMaxRows || tokens * choices > kMaxEntries || slots > kMxMaxRows ||
      cols > kMxMaxCols)
    return CIERA_ERR_ARG;
  if (tokens && (!d_place || (reinterpret_cast<uintptr_t>(d_place) & 3u) != 0u)) return CIERA_ERR_ARG;
  p.place = d_place;
  p.tokens = uint32_t(tokens);
  p.choices = uint32_t(choices);
  p.cols = uint32_t(cols);
  p.slots = uint32_t(slots);
  p.lt = row_threads(cols);
  return cdiv(tokens, 256u >> p.lt) * cdiv(mx_pitch(cols), 8u << p.lt) > kMxMostGroups ? CIERA_ERR_ARG : CIERA_OK;
}
dim3 row_grid(const RowArgs& p, uint64_t cols) { return dim3(uint32_t(cdiv(p.tokens, 256u >> p.lt)), uint32_t(cdiv(cols, 8u << p.lt))); }

}  // namespace

extern "C" {

uint64_t expert_workspace_size(uint64_t tokens, uint64_t choices, uint32_t experts) {
  if (choices == 0u || choices > kMaxChoices || tokens > kMxMaxRows || tokens * choices > kMaxEntries || experts == 0u ||
      experts > kMxMaxGroups)
    return 0u;
  // any smaller number of tokens takes no more blocks
  return align256(kMxWsHead + 4ull * sort_blocks(tokens * choices, experts) * (experts + 2u));
}

ciera_status expert_sort(const void* d_ids, uint32_t ids_i64, uint64_t tokens, uint64_t choices, uint32_t experts,
                         int64_t* d_offsets, int32_t* d_place, int32_t* d_order, void* d_ws, uint64_t ws_bytes,
                         hipStream_t stream) {
  const uint64_t need = expert_workspace_size(tokens, choices, experts);
  if (!need || ids_i64 > 1u) return CIERA_ERR_ARG;
  ciera_status st = norm_vector(d_offsets, 8u);
  if (st == CIERA_OK && tokens) st = norm_vector(d_ids, ids_i64 ? 8u : 4u);
  if (st == CIERA_OK && tokens) st = norm_vector(d_place, 4u);
  if (st == CIERA_OK && d_order) st = norm_vector(d_order, 4u);
  if (st != CIERA_OK || !d_ws || !aligned16(d_ws)) return CIERA_ERR_ARG;
  if (ws_bytes < need) return CIERA_ERR_WORKSPACE;
  SortArgs p{};
  p.ids = d_ids;
  p.offsets = d_offsets;
  p.place = d_place;
  p.order = d_order;
  p.ctrl = static_cast<Ctrl*>(d_ws);
  p.status = reinterpret_cast<uint32_t*>(static_cast<uint8_t*>(d_ws) + sizeof(Ctrl));
  p.counts = reinterpret_cast<uint32_t*>(static_cast<uint8_t*>(d_ws) + kMxWsHead);
  p.entries = uint32_t(tokens * choices);
  p.experts = experts;
  p.blocks = sort_blocks(p.entries, experts);
  p.per = uint32_t(cdiv(p.entries, p.blocks));
  const dim3 block(64u * sort_waves(experts));
  (void)hipGetLastError();
  if (p.blocks > 1u) {
    if (ids_i64) launch(k_sort_count<true>, dim3(p.blocks), block, stream, p);
    else launch(k_sort_count<false>, dim3(p.blocks), block, stream, p);
  }
  if (ids_i64) launch(k_expert_sort<true>, dim3(p.blocks), block, stream, p);
  else launch(k_expert_sort<false>, dim3(p.blocks), block, stream, p);
  return launch_status();
}

ciera_status expert_dispatch(const void* d_x, uint64_t ldx, const int32_t* d_place, uint64_t tokens, uint64_t choices,
                             uint64_t cols, uint64_t rows, void* d_out, uint64_t ldo, void* d_outq, uint64_t outq_bytes,
                             hipStream_t stream) {
  RowArgs p{};
  if (!d_out && !d_outq && rows) return CIERA_ERR_ARG;
  ciera_status st = row_common(p, d_place, tokens, choices, cols, rows);
  if (st == CIERA_OK) st = mx_matrix(d_x, tokens, cols, ldx, 2u);
  if (st == CIERA_OK && d_out) st = mx_matrix(d_out, rows, cols, ldo, 2u);
  if (st == CIERA_OK && d_outq) st = mx_encoded(d_outq, outq_bytes, rows, cols, 8u, CIERA_ERR_CAPACITY);
  if (st != CIERA_OK || !tokens || !cols || !rows) return st;
  p.x = static_cast<const uint16_t*>(d_x);
  p.ldx = ldx;
  p.out = d_out;
  p.ldo = ldo;
  p.q = static_cast<uint8_t*>(d_outq);
  p.qs = p.q ? p.q + mx_scales_at(rows, cols, 8u) : nullptr;
  (void)hipGetLastError();
  const dim3 grid = row_grid(p, p.q ? mx_pitch(cols) : cols);
  if (p.lt >= 6u) launch(k_dispatch<true>, grid, dim3(256), stream, p);
  else launch(k_dispatch<false>, grid, dim3(256), stream, p);
  return launch_status();
}

ciera_status expert_combine(const void* d_rows, uint64_t ldrows, uint32_t rows_f32, uint64_t rows, const int32_t* d_place,
                            const float* d_weights, const void* d_residual, uint64_t ldr, void* d_out, uint64_t ldo,
                            uint32_t out_f32, uint64_t tokens, uint64_t choices, uint64_t cols, hipStream_t stream) {
  RowArgs p{};
  if (rows_f32 > 1u || out_f32 > 1u) return CIERA_ERR_ARG;
  ciera_status st = row_common(p, d_place, tokens, choices, cols, rows);
  if (st == CIERA_OK) st = mx_matrix(d_rows, rows, cols, ldrows, rows_f32 ? 4u : 2u);
  if (st == CIERA_OK) st = mx_matrix(d_out, tokens, cols, ldo, out_f32 ? 4u : 2u);
  if (st == CIERA_OK && d_residual) st = mx_matrix(d_residual, tokens, cols, ldr, 2u);
  if (st == CIERA_OK && d_weights) st = norm_vector(d_weights, 4u);
  if (st != CIERA_OK || !tokens || !cols) return st;
  p.rows = d_rows;
  p.ldrows = ldrows;
  p.weights = d_weights;
  p.residual = static_cast<const uint16_t*>(d_residual);
  p.ldr = ldr;
  p.out = d_out;
  p.ldo = ldo;
  p.out_f32 = out_f32;
  (void)hipGetLastError();
  if (p.lt >= 6u) {
    if (rows_f32) launch(k_combine<true, true>, row_grid(p, cols), dim3(256), stream, p);
    else launch(k_combine<true, false>, row_grid(p, cols), dim3(256), stream, p);
  } else {
    if (rows_f32) launch(k_combine<false, true>, row_grid(p, cols), dim3(256), stream, p);
    else launch(k_combine<false, false>, row_grid(p, cols), dim3(256), stream, p);
  }
  return launch_status();
}

ciera_status expert_combine_backward(const void* d_dout, uint64_t lddout, const void* d_rows, uint64_t ldrows,
                                     uint32_t rows_f32, uint64_t rows, const int32_t* d_place, const float* d_weights,
                                     void* d_drows, uint64_t lddrows, float* d_dweights, uint64_t tokens,
                                     uint64_t choices, uint64_t cols, hipStream_t stream) {
  RowArgs p{};
  if (rows_f32 > 1u || (!d_drows && !d_dweights && tokens && rows)) return CIERA_ERR_ARG;
  ciera_status st = row_common(p, d_place, tokens, choices, cols, rows);
  if (st == CIERA_OK) st = mx_matrix(d_dout, tokens, cols, lddout, 2u);
  if (st == CIERA_OK && d_dweights) st = mx_matrix(d_rows, rows, cols, ldrows, rows_f32 ? 4u : 2u);
  if (st == CIERA_OK && d_dweights) st = norm_vector(d_dweights, 4u);
  if (st == CIERA_OK && d_drows) st = mx_matrix(d_drows, rows, cols, lddrows, 2u);
  if (st == CIERA_OK && d_weights) st = norm_vector(d_weights, 4u);
  if (st != CIERA_OK || !tokens) return st;
  p.x = static_cast<const uint16_t*>(d_dout);
  p.ldx = lddout;
  p.rows = d_rows;
  p.ldrows = ldrows;
  p.weights = d_weights;
  p.out = d_drows;
  p.ldo = lddrows;
  p.dweights = d_dweights;
  (void)hipGetLastError();
  if (p.lt >= 6u) {
    if (rows_f32) launch(k_combine_back<true, true>, row_grid(p, 1u), dim3(256), stream, p);
    else launch(k_combine_back<true, false>, row_grid(p, 1u), dim3(256), stream, p);
  } else {
    if (rows_f32) launch(k_combine_back<false, true>, row_grid(p, 1u), dim3(256), stream, p);
    else launch(k_combine_back<false, false>, row_grid(p, 1u), dim3(256), stream, p);
  }
  return launch_status();
}

}  // extern "C"
