// norm.hip -- root-mean-square norm of the rows of a BF16 matrix, with the
// residual's addition before it and its result in BF16, mx8 or both; and its
// gradients; gfx950.
//
//   h = bf16(x + residual)         (x itself without a residual)
//   s = 1 / sqrt(mean(h^2) + eps)  FP32
//   y = bf16(h s w)                yq: the mx8 form of y, mx8_encode's bytes
//
//   u = h s,  g = dy w
//   dx = s (g - u mean(g u)) + dh
//   dw = sum over the rows of dy u
//
// The statistics are those of the rounded h, which is what the backward pass
// reads.  Products and sums are FP32; h, y and dx are rounded to BF16 once.
#include "ciera.h"

namespace {

constexpr uint32_t kNormMaxCols = 32768u;  // 1,024 threads of four units of 8 values

// Workgroups of the backward pass, each with a sum of dw of its own.  us, with
// the join of the sums, with 256, 512, 768 and 1,024 of them (with dh, dw FP32):
//   262,144 x 64      48   34   31   33
//   65,536 x 512      62   50   52   52
//   32,768 x 1,000    67   50   52   56
//   16,384 x 2,048    67   52   59   53
//   8,192 x 4,096     65   53   61   56
//   4,096 x 8,192     59   58   65   67
//   1,677 x 20,000    85   94  108  125
//   1,024 x 32,768    86  113  139  160
constexpr uint32_t kNormParts = 512u;

template <uint32_t k>
using Num = std::integral_constant<uint32_t, k>;

struct NormArgs {
  const uint16_t* x;
  uint64_t ldx;
  const uint16_t* residual;
  uint64_t ldr;
  const uint16_t* w;
  uint16_t* h;
  uint64_t ldh;
  uint16_t* y;
  uint64_t ldy;
  uint8_t* yq;
  uint8_t* ys;
  float* rstd;
  float eps;
  float each, each_rest;  // 1 / cols in two parts
  uint32_t rows, cols;
};

// 1 / sqrt(sum / cols + eps), off by little more than its last rounding: what
// the first value leaves of 1 - mean s^2 corrects it.  (A division, a square
// root and a division, each rounded: s off by 4.5e-8 of itself in the mean
// instead of 3.8e-8, most of it the sum's, and 160 of 268 million values in mx8
// beside the exact norm's instead of 139, at the same time.)  A sum past FP32's
// range gives 0, a NaN itself.
__device__ __forceinline__ float norm_root(const NormArgs& p, float sum) {
  if (sum == INFINITY) return 0.0f;
  const float mean = fmaf(sum, p.each, fmaf(sum, p.each_rest, p.eps)), s = rsqrtf(mean);
  const float t = mean * s, rest = fmaf(mean, s, -t);
  return s > 0.0f ? fmaf(0.5f * s, fmaf(-rest, s, fmaf(-t, s, 1.0f)), s) : s;
}

__device__ __forceinline__ float bf_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf_hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

// Eight values of a row from column `col`, zeros behind its end, in two steps,
// so that a thread's loads all go out before it waits for one: row_load8 reads
// the unit, or for a unit that passes the end the row's last eight values, and
// row_mend8 moves those to where they belong.
// kStream: past the last-level cache.  kTiny: rows of less than 8 are possible.
template <bool kStream = false, bool kTiny = true>
__device__ __forceinline__ u32x4v row_load8(const uint16_t* row, uint32_t col, uint32_t cols) {
  if (kTiny && cols < 8u) return mx_part8(row, col == 0u ? cols : 0u);
  const u32x4a2* at = reinterpret_cast<const u32x4a2*>(row + min(col, cols - 8u));
  if constexpr (kStream) return u32x4v(__builtin_nontemporal_load(at));
  else return u32x4v(*at);
}
// kWhole: the rows are multiples of 8 long, and a unit is theirs or is not.  No
// branches: threads with and without a unit to mend share waves.
template <bool kTiny = true, bool kWhole = false>
__device__ __forceinline__ void row_mend8(u32x4v& v, uint32_t col, uint32_t cols) {
  const u32x4v none = {0u, 0u, 0u, 0u};
  if constexpr (kWhole) {
    v = col < cols ? v : none;
  } else {
    if (kTiny && cols < 8u) return;
    const uint32_t by = col + 8u > cols ? col + 8u - cols : 0u;  // values to move down
    v = by & 4u ? u32x4v{v[2], v[3], 0u, 0u} : v;
    v = by & 2u ? u32x4v{v[1], v[2], v[3], 0u} : v;
    v = by & 1u ? u32x4v{__builtin_amdgcn_alignbit(v[1], v[0], 16), __builtin_amdgcn_alignbit(v[2], v[1], 16),
                         __builtin_amdgcn_alignbit(v[3], v[2], 16), v[3] >> 16}
                : v;
    v = by >= 8u ? none : v;
  }
}
template <bool kTiny = true, bool kWhole = false>
__device__ __forceinline__ u32x4v row_get8(const uint16_t* row, uint32_t col, uint32_t cols) {
  u32x4v v = row_load8<false, kTiny>(row, col, cols);
  row_mend8<kTiny, kWhole>(v, col, cols);
  return v;
}
template <bool kStream = false, bool kWhole = false>
__device__ __forceinline__ void row_store8(uint16_t* row, uint32_t col, uint32_t cols, u32x4v v) {
  if (kWhole ? col < cols : col + 8u <= cols) {
    if constexpr (kStream) __builtin_nontemporal_store(v, reinterpret_cast<u32x4a2*>(row + col));
    else *reinterpret_cast<u32x4a2*>(row + col) = v;
  } else if constexpr (!kWhole) {
#pragma unroll
    for (uint32_t i = 0; i < 7u; i++)
      if (col + i < cols) row[col + i] = uint16_t(v[i >> 1] >> (16u * (i & 1u)));
  }
}
// Loads before this are issued before it: the compiler else sinks them to their
// uses, one after the other.
__device__ __forceinline__ void loads_first() { __builtin_amdgcn_sched_barrier(0); }

// What v holds is not known from here on, so that it is unpacked again where it
// is used again, and not kept unpacked in twice the registers.
__device__ __forceinline__ void keep_packed(u32x4v& v) {
#pragma unroll
  for (int i = 0; i < 4; i++) asm volatile("" : "+v"(v[i]));
}

// Sums over the kT threads of a row, of kN rows at once.  With more than one
// wave a row, `part` has a line for each wave of the workgroup and is free again
// when the next barrier is passed, which every thread of it has to reach.
template <uint32_t kT, uint32_t kN>
__device__ __forceinline__ void row_sums(float (&v)[kN], float (*part)[kN]) {
#pragma unroll
  for (int d = int(kT < 64u ? kT : 64u) / 2; d > 0; d >>= 1)
#pragma unroll
    for (uint32_t n = 0; n < kN; n++) v[n] += __shfl_xor(v[n], d);
  if constexpr (kT > 64u) {
    if ((threadIdx.x & 63u) == 0u)
#pragma unroll
      for (uint32_t n = 0; n < kN; n++) part[threadIdx.x >> 6][n] = v[n];
    __syncthreads();
#pragma unroll
    for (uint32_t n = 0; n < kN; n++) {
      v[n] = 0.0f;
#pragma unroll
      for (uint32_t i = 0; i < kT / 64u; i++) v[n] += part[threadIdx.x / kT * (kT / 64u) + i][n];
    }
  }
}

// A row takes kT threads, each kU units of 8 values, which stay in registers
// between the sum and the result: memory is read and written once, and bounds
// it.  16,384 x 2,048 with a residual, h, y and yq, 302 MB: 50 us, 6.0 TB/s.  All
// but the weight and yq goes past the last-level cache, which keeps yq for its
// reader (55 us through it).  As many threads as a row has units: 65,536 rows of
// 64 with a wave each 79 us, with 16 threads 10; 30,000 of 1,021 with 256 threads
// 69 us, with 128 48.
template <uint32_t kT, uint32_t kU, bool kWhole>
__global__ __launch_bounds__(kT < 256u ? 256u : kT) void k_rms_norm(NormArgs p) {
  constexpr uint32_t kB = kT < 256u ? 256u : kT;
  constexpr bool kTiny = kT < 64u && !kWhole;  // the rule's shape for few columns
  __shared__ float part[kT <= 64u ? 1u : kB / 64u][1];
  const uint32_t t = threadIdx.x % kT;
  const uint32_t at = blockIdx.x * (kB / kT) + threadIdx.x / kT;
  const uint32_t row = min(at, p.rows - 1u);  // rows behind the last: for the barrier alone
  const bool live = at < p.rows;
  if (kT <= 64u && !live) return;
  const uint16_t* x = p.x + uint64_t(row) * p.ldx;
  const uint16_t* r = p.residual ? p.residual + uint64_t(row) * p.ldr : nullptr;
  u32x4v v[kU], a[kU], w[kU];
#pragma unroll
  for (uint32_t u = 0; u < kU; u++) v[u] = row_load8<true, kTiny>(x, (u * kT + t) * 8u, p.cols);
  if (r) {
#pragma unroll
    for (uint32_t u = 0; u < kU; u++) a[u] = row_load8<true, kTiny>(r, (u * kT + t) * 8u, p.cols);
  }
#pragma unroll
  for (uint32_t u = 0; u < kU; u++) w[u] = row_load8<false, kTiny>(p.w, (u * kT + t) * 8u, p.cols);
  loads_first();
#pragma unroll
  for (uint32_t u = 0; u < kU; u++) {
    row_mend8<kTiny, kWhole>(v[u], (u * kT + t) * 8u, p.cols);
    row_mend8<kTiny, kWhole>(w[u], (u * kT + t) * 8u, p.cols);
  }
  if (r) {
#pragma unroll
    for (uint32_t u = 0; u < kU; u++) {
      row_mend8<kTiny, kWhole>(a[u], (u * kT + t) * 8u, p.cols);
#pragma unroll
      for (int i = 0; i < 4; i++) v[u][i] = mx_bf16x2(bf_lo(v[u][i]) + bf_lo(a[u][i]), bf_hi(v[u][i]) + bf_hi(a[u][i]));
    }
    if (p.h && live) {
#pragma unroll
      for (uint32_t u = 0; u < kU; u++) row_store8<true, kWhole>(p.h + uint64_t(row) * p.ldh, (u * kT + t) * 8u, p.cols, v[u]);
    }
  }
  float sum[1] = {0.0f};
#pragma unroll
  for (uint32_t u = 0; u < kU; u++)
#pragma unroll
    for (int i = 0; i < 4; i++)
      sum[0] = fmaf(bf_lo(v[u][i]), bf_lo(v[u][i]), fmaf(bf_hi(v[u][i]), bf_hi(v[u][i]), sum[0]));
  row_sums<kT, 1u>(sum, part);
  if (!live) return;
  const float s = norm_root(p, sum[0]);
  if (p.rstd && t == 0u) p.rstd[row] = s;
  const uint32_t kp = uint32_t(mx_pitch(p.cols));
#pragma unroll
  for (uint32_t u = 0; u < kU; u++) {
    const uint32_t col = (u * kT + t) * 8u;
    u32x4v y;
#pragma unroll
    for (int i = 0; i < 4; i++) y[i] = mx_bf16x2(bf_lo(v[u][i]) * s * bf_lo(w[u][i]), bf_hi(v[u][i]) * s * bf_hi(w[u][i]));
    // behind the row's end: zeros, also where s is NaN
    if constexpr (kWhole) {
      if (col >= p.cols) y = u32x4v{0u, 0u, 0u, 0u};
    } else {
#pragma unroll
      for (uint32_t i = 0; i < 8u; i++) y[i >> 1] &= col + i >= p.cols ? ((i & 1u) ? 0xFFFFu : 0u) : ~0u;
    }
    if (p.y) row_store8<true, kWhole>(p.y + uint64_t(row) * p.ldy, col, p.cols, y);
    if (p.yq && col < kp) {
      const uint32_t sb = mx_block_scale<8>(y);
      *reinterpret_cast<u32x2v*>(p.yq + uint64_t(row) * kp + col) = mx8_codes(y, mx_scale(sb == 255u ? 127u : sb));
      if ((t & 3u) == 0u) p.ys[uint64_t(row) * (kp / 32u) + col / 32u] = uint8_t(sb);
    }
  }
}

struct NormBackArgs {
  const uint16_t* dy;
  uint64_t lddy;
  const uint16_t* h;
  uint64_t ldh;
  const uint16_t* w;
  const float* rstd;
  const uint16_t* dh;
  uint64_t lddh;
  uint16_t* dx;
  uint64_t lddx;
  float* sums;  // of dw: a row of cols for each workgroup
  Ctrl* ctrl;
  uint32_t* status;
  void* dw;
  uint32_t dw_f32, accumulate, rows, cols, parts;
};

// A workgroup takes every parts-th stretch of kB / kT * kN rows, a thread's
// loads of kN rows at once (with one barrier for their sums), and keeps its sums
// of dw in registers to the end.  Bound by memory: 16,384 x 2,048 with dh, 268
// MB: 48 us, 5.6 TB/s (53 through the last-level cache), and 4 for the join of
// the sums.  Registers leave two waves a SIMD (up to 1,024 columns three), two
// workgroups a CU, each with 48 KB in flight.  Two rows of 4,096 with 256
// threads: 8,000 of them 53 us; four with 512 threads 64.  Past 8,192 columns a
// row is read twice by one workgroup of 16 waves a CU: 1,024 x 32,768 100 us
// (and 12) on 43 for the bytes; of odd length 129, with some registers in memory
// (18 of a thread's).
template <uint32_t kT, uint32_t kU, uint32_t kN, bool kWhole>
__global__ __launch_bounds__(kT < 256u ? 256u : kT) void k_rms_norm_back(NormBackArgs p) {
  constexpr uint32_t kB = kT < 256u ? 256u : kT, kSubs = kB / kT;
  constexpr bool kTiny = kT < 64u && !kWhole;
  constexpr bool kAgain = kU > 2u;  // rows that long are read again (from L2) for dx and dw: registers
  __shared__ float part[2][kT <= 64u ? 1u : kB / 64u][kN];
  __shared__ float fold[kSubs > 1u ? kB * 8u : 1u];
  const uint32_t t = threadIdx.x % kT, sub = threadIdx.x / kT;
  const u32x4v none = {0u, 0u, 0u, 0u};
  float dw[kU][8];
#pragma unroll
  for (uint32_t u = 0; u < kU; u++)
#pragma unroll
    for (int i = 0; i < 8; i++) dw[u][i] = 0.0f;
  const auto weight = [&](uint32_t u) { return row_get8<kTiny, kWhole>(p.w, (u * kT + t) * 8u, p.cols); };
  u32x4v w[kAgain ? 1 : kU];
  if constexpr (!kAgain) {
#pragma unroll
    for (uint32_t u = 0; u < kU; u++) w[u] = weight(u);
  }
  uint32_t turn = 0u;
  for (uint32_t first = blockIdx.x * (kSubs * kN); first < p.rows; first += p.parts * (kSubs * kN), turn ^= 1u) {
    // rows behind the last are read as the last, and count nothing
    const auto row_of = [&](uint32_t n) { return uint64_t(min(first + n * kSubs + sub, p.rows - 1u)); };
    const auto live = [&](uint32_t n) { return first + n * kSubs + sub < p.rows; };
    u32x4v h[kN][kAgain ? 1 : kU], d[kN][kAgain ? 1 : kU], e[kN][kAgain ? 1 : kU];
    float s[kN], dot[kN];
    const auto load = [&](uint32_t n, uint32_t u, uint32_t to, bool dh) {
      const uint32_t col = (u * kT + t) * 8u;
      h[n][to] = row_load8<!kAgain, kTiny>(p.h + row_of(n) * p.ldh, col, p.cols);
      d[n][to] = row_load8<!kAgain, kTiny>(p.dy + row_of(n) * p.lddy, col, p.cols);
      if (dh && p.dh) e[n][to] = row_load8<true, kTiny>(p.dh + row_of(n) * p.lddh, col, p.cols);
    };
    const auto mend = [&](uint32_t n, uint32_t u, uint32_t to, bool dh) {
      const uint32_t col = (u * kT + t) * 8u;
      row_mend8<kTiny, kWhole>(h[n][to], col, p.cols);
      row_mend8<kTiny, kWhole>(d[n][to], col, p.cols);
      if (dh && p.dh) row_mend8<kTiny, kWhole>(e[n][to], col, p.cols);
      h[n][to] = live(n) ? h[n][to] : none;
      d[n][to] = live(n) ? d[n][to] : none;
    };
    // dot += sum of dy w h s, and dw += dy h s
    const auto sums = [&](uint32_t n, uint32_t u, uint32_t at, u32x4v wu, bool dots, bool dws) {
#pragma unroll
      for (int i = 0; i < 4; i++) {
        const float u0 = bf_lo(h[n][at][i]) * s[n], u1 = bf_hi(h[n][at][i]) * s[n];
        const float d0 = bf_lo(d[n][at][i]), d1 = bf_hi(d[n][at][i]);
        if (dots) dot[n] = fmaf(d0 * bf_lo(wu[i]), u0, fmaf(d1 * bf_hi(wu[i]), u1, dot[n]));
        if (dws) {
          dw[u][2 * i] = fmaf(d0, u0, dw[u][2 * i]);
          dw[u][2 * i + 1] = fmaf(d1, u1, dw[u][2 * i + 1]);
        }
      }
      loads_first();
    };
    const auto out = [&](uint32_t n, uint32_t u, uint32_t at, u32x4v wu, float m) {
      u32x4v o;
#pragma unroll
      for (int i = 0; i < 4; i++) {
        const float g0 = bf_lo(d[n][at][i]) * bf_lo(wu[i]), g1 = bf_hi(d[n][at][i]) * bf_hi(wu[i]);
        const float e0 = p.dh ? bf_lo(e[n][at][i]) : 0.0f, e1 = p.dh ? bf_hi(e[n][at][i]) : 0.0f;
        o[i] = mx_bf16x2(fmaf(s[n], g0 - bf_lo(h[n][at][i]) * s[n] * m, e0), fmaf(s[n], g1 - bf_hi(h[n][at][i]) * s[n] * m, e1));
      }
      if (live(n)) row_store8<true, kWhole>(p.dx + row_of(n) * p.lddx, (u * kT + t) * 8u, p.cols, o);
      loads_first();
    };
#pragma unroll
    for (uint32_t n = 0; n < kN; n++) {
      s[n] = live(n) ? p.rstd[row_of(n)] : 0.0f;
      dot[n] = 0.0f;
    }
    if constexpr (kAgain) {
      static_assert(kN == 1u, "one row");
      if (p.dx) {
#pragma unroll
        for (uint32_t u = 0; u < kU; u++) {
          load(0u, u, 0u, false);
          mend(0u, u, 0u, false);
          sums(0u, u, 0u, weight(u), true, false);
        }
        row_sums<kT, kN>(dot, part[turn]);
      }
      const float m = dot[0] / float(p.cols);
#pragma unroll
      for (uint32_t u = 0; u < kU; u++) {
        const u32x4v wu = weight(u);
        load(0u, u, 0u, true);
        mend(0u, u, 0u, true);
        sums(0u, u, 0u, wu, false, true);
        if (p.dx) out(0u, u, 0u, wu, m);
      }
    } else {
#pragma unroll
      for (uint32_t n = 0; n < kN; n++)
#pragma unroll
        for (uint32_t u = 0; u < kU; u++) load(n, u, u, true);
      loads_first();
#pragma unroll
      for (uint32_t n = 0; n < kN; n++)
#pragma unroll
        for (uint32_t u = 0; u < kU; u++) {
          mend(n, u, u, true);
          sums(n, u, u, w[u], true, true);
          keep_packed(h[n][u]);
          keep_packed(d[n][u]);
        }
      if (!p.dx) continue;
      row_sums<kT, kN>(dot, part[turn]);
#pragma unroll
      for (uint32_t n = 0; n < kN; n++) {
        const float m = dot[n] / float(p.cols);
#pragma unroll
        for (uint32_t u = 0; u < kU; u++) out(n, u, u, w[u], m);
      }
    }
  }
  if (!p.dw) return;
  float* to = p.sums + uint64_t(blockIdx.x) * p.cols;
#pragma unroll
  for (uint32_t u = 0; u < kU; u++) {
    if constexpr (kSubs > 1u) {
      __syncthreads();
#pragma unroll
      for (int i = 0; i < 8; i++) fold[(sub * 8u + i) * kT + t] = dw[u][i];
      __syncthreads();
      for (uint32_t i = threadIdx.x; i < kT * 8u; i += kB) {
        float v = 0.0f;
#pragma unroll
        for (uint32_t r = 0; r < kSubs; r++) v += fold[(r * 8u + i % 8u) * kT + i / 8u];
        const uint32_t col = u * kT * 8u + i;
        if (col < p.cols) to[col] = v;
      }
    } else {
      const uint32_t col = (u * kT + t) * 8u;
#pragma unroll
      for (uint32_t i = 0; i < 8u; i++)
        if (col + i < p.cols) to[col + i] = dw[u][i];
    }
  }
}

// dw: the workgroups' sums added in order, 32 columns a workgroup, every 32nd
// of the rows of sums to each of its 32 rows of threads, so that a thread waits
// for memory once or twice.  Bound by its launch (4 us).
__global__ __launch_bounds__(1024) void k_rms_norm_join(NormBackArgs p) {
  __shared__ float part[32][32];
  const uint32_t c = threadIdx.x & 31u, r = threadIdx.x >> 5;
  const uint32_t col = blockIdx.x * 32u + c;
  float v = 0.0f;
  if (col < p.cols) {
#pragma unroll 16
    for (uint32_t i = r; i < p.parts; i += 32u) v += p.sums[uint64_t(i) * p.cols + col];
  }
  if (blockIdx.x == 0u && threadIdx.x == 0u) {  // what ciera_read_error reads: nothing can be wrong here
    p.ctrl->n_err_slots = 1u;
    *p.status = uint32_t(CIERA_OK);
  }
  part[r][c] = v;
  __syncthreads();
  if (r || col >= p.cols) return;
#pragma unroll
  for (uint32_t i = 1; i < 32u; i++) v += part[i][c];
  if (p.dw_f32) {
    float* o = static_cast<float*>(p.dw) + col;
    *o = p.accumulate ? *o + v : v;
  } else {
    uint16_t* o = static_cast<uint16_t*>(p.dw) + col;
    *o = mx_bf16(p.accumulate ? mx_f32(*o) + v : v);
  }
}

// Rows a workgroup of the backward pass takes at once, and how many workgroups.
uint32_t norm_back_rows(uint32_t cols) {
  return cols <= 32u ? 256u : cols <= 128u ? 64u : cols <= 512u ? 16u : cols <= 1024u ? 8u : cols <= 2048u ? 4u : cols <= 4096u ? 2u : 1u;
}
uint32_t norm_back_parts(uint64_t rows, uint32_t cols) {
  const uint64_t groups = cdiv(rows, norm_back_rows(cols));
  return uint32_t(groups < kNormParts ? groups : kNormParts);
}

ciera_status norm_vector(const void* d, uint32_t align) {
  return !d || (reinterpret_cast<uintptr_t>(d) & (align - 1u)) != 0u ? CIERA_ERR_ARG : CIERA_OK;
}

}  // namespace

extern "C" {

ciera_status rms_norm(const void* d_x, uint64_t ldx, const void* d_residual, uint64_t ldr, const void* d_w, float eps,
                      void* d_h, uint64_t ldh, void* d_y, uint64_t ldy, void* d_yq, uint64_t yq_bytes, float* d_rstd,
                      uint64_t rows, uint64_t cols, hipStream_t stream) {
  if (cols == 0u || cols > kNormMaxCols || !(eps > 0.0f) || eps > 3.0e38f || (rows && !d_y && !d_yq) || (d_h && !d_residual))
    return CIERA_ERR_ARG;
  ciera_status st = mx_matrix(d_x, rows, cols, ldx, 2u);
  if (st == CIERA_OK && d_residual) st = mx_matrix(d_residual, rows, cols, ldr, 2u);
  if (st == CIERA_OK && d_h) st = mx_matrix(d_h, rows, cols, ldh, 2u);
  if (st == CIERA_OK && d_y) st = mx_matrix(d_y, rows, cols, ldy, 2u);
  if (st == CIERA_OK) st = norm_vector(d_w, 2u);
  if (st == CIERA_OK && d_rstd) st = norm_vector(d_rstd, 4u);
  if (st == CIERA_OK && d_yq) st = mx_encoded(d_yq, yq_bytes, rows, cols, 8u, CIERA_ERR_CAPACITY);
  if (st != CIERA_OK || rows == 0u) return st;
  NormArgs p{};
  p.x = static_cast<const uint16_t*>(d_x);
  p.ldx = ldx;
  p.residual = static_cast<const uint16_t*>(d_residual);
  p.ldr = ldr;
  p.w = static_cast<const uint16_t*>(d_w);
  p.h = static_cast<uint16_t*>(d_h);
  p.ldh = ldh;
  p.y = static_cast<uint16_t*>(d_y);
  p.ldy = ldy;
  p.yq = static_cast<uint8_t*>(d_yq);
  p.ys = p.yq ? p.yq + mx_scales_at(rows, cols, 8u) : nullptr;
  p.rstd = d_rstd;
  p.eps = eps;
  p.each = float(1.0 / double(cols));
  p.each_rest = float(1.0 / double(cols) - double(p.each));
  p.rows = uint32_t(rows);
  p.cols = uint32_t(cols);
  const auto go = [&](auto threads, auto units) {
    constexpr uint32_t kT = decltype(threads)::value, kU = decltype(units)::value, kB = kT < 256u ? 256u : kT;
    const uint64_t grid = cdiv(rows, kB / kT);
    if (grid > 0xFFFFFFFFull / kB) return CIERA_ERR_ARG;
    (void)hipGetLastError();
    if (cols % 8u == 0u) launch(k_rms_norm<kT, kU, true>, dim3(uint32_t(grid)), dim3(kB), stream, p);
    else launch(k_rms_norm<kT, kU, false>, dim3(uint32_t(grid)), dim3(kB), stream, p);
    return launch_status();
  };
  if (cols <= 32u && !d_yq) return go(Num<4u>(), Num<1u>());  // a row of mx8 is 16 units long
  if (cols <= 128u) return go(Num<16u>(), Num<1u>());
  if (cols <= 512u) return go(Num<64u>(), Num<1u>());
  if (cols <= 1024u) return go(Num<128u>(), Num<1u>());
  if (cols <= 2048u) return go(Num<256u>(), Num<1u>());
  if (cols <= 4096u) return go(Num<256u>(), Num<2u>());
  if (cols <= 8192u) return go(Num<256u>(), Num<4u>());
  return go(Num<1024u>(), Num<4u>());
}

uint64_t rms_norm_workspace_size(uint64_t rows, uint64_t cols) {
  if (rows > kMxMaxRows || cols == 0u || cols > kNormMaxCols) return 0u;
  const uint64_t parts = norm_back_parts(rows, uint32_t(cols));
  return align256(kMxWsHead + (parts ? parts : 1u) * cols * 4u);
}

ciera_status rms_norm_backward(const void* d_dy, uint64_t lddy, const void* d_h, uint64_t ldh, const void* d_w,
                               const float* d_rstd, const void* d_dh, uint64_t lddh, void* d_dx, uint64_t lddx,
                               void* d_dw, uint32_t dw_f32, uint32_t accumulate, uint64_t rows, uint64_t cols,
                               void* d_ws, uint64_t ws_bytes, hipStream_t stream) {
  if (cols == 0u || cols > kNormMaxCols || dw_f32 > 1u || accumulate > 1u || (rows && !d_dx && !d_dw) || (d_dh && !d_dx))
    return CIERA_ERR_ARG;
  ciera_status st = mx_matrix(d_dy, rows, cols, lddy, 2u);
  if (st == CIERA_OK) st = mx_matrix(d_h, rows, cols, ldh, 2u);
  if (st == CIERA_OK && d_dh) st = mx_matrix(d_dh, rows, cols, lddh, 2u);
  if (st == CIERA_OK && d_dx) st = mx_matrix(d_dx, rows, cols, lddx, 2u);
  if (st == CIERA_OK) st = norm_vector(d_w, 2u);
  if (st == CIERA_OK && rows) st = norm_vector(d_rstd, 4u);
  if (st == CIERA_OK && d_dw) {
    st = norm_vector(d_dw, dw_f32 ? 4u : 2u);
    if (st == CIERA_OK && (!d_ws || !aligned16(d_ws))) st = CIERA_ERR_ARG;
    if (st == CIERA_OK && ws_bytes < rms_norm_workspace_size(rows, cols)) st = CIERA_ERR_WORKSPACE;
  }
  if (st != CIERA_OK) return st;
  if (!rows && !d_dw) return CIERA_OK;
  NormBackArgs p{};
  p.dy = static_cast<const uint16_t*>(d_dy);
  p.lddy = lddy;
  p.h = static_cast<const uint16_t*>(d_h);
  p.ldh = ldh;
  p.w = static_cast<const uint16_t*>(d_w);
  p.rstd = d_rstd;
  p.dh = static_cast<const uint16_t*>(d_dh);
  p.lddh = lddh;
  p.dx = static_cast<uint16_t*>(d_dx);
  p.lddx = lddx;
  if (d_dw) {
    p.ctrl = static_cast<Ctrl*>(d_ws);
    p.status = reinterpret_cast<uint32_t*>(static_cast<uint8_t*>(d_ws) + sizeof(Ctrl));
    p.sums = reinterpret_cast<float*>(static_cast<uint8_t*>(d_ws) + kMxWsHead);
  }
  p.dw = d_dw;
  p.dw_f32 = dw_f32;
  p.accumulate = accumulate;
  p.rows = uint32_t(rows);
  p.cols = uint32_t(cols);
  p.parts = norm_back_parts(rows, uint32_t(cols));
  (void)hipGetLastError();
  if (rows) {
    const auto go = [&](auto threads, auto units, auto rows_at_once) {
      constexpr uint32_t kT = decltype(threads)::value, kU = decltype(units)::value, kN = decltype(rows_at_once)::value;
      const dim3 grid(p.parts), block(kT < 256u ? 256u : kT);
      if (cols % 8u == 0u) launch(k_rms_norm_back<kT, kU, kN, true>, grid, block, stream, p);
      else launch(k_rms_norm_back<kT, kU, kN, false>, grid, block, stream, p);
    };
    if (cols <= 32u) go(Num<4u>(), Num<1u>(), Num<4u>());
    else if (cols <= 128u) go(Num<16u>(), Num<1u>(), Num<4u>());
    else if (cols <= 512u) go(Num<64u>(), Num<1u>(), Num<4u>());
    else if (cols <= 1024u) go(Num<128u>(), Num<1u>(), Num<4u>());
    else if (cols <= 2048u) go(Num<256u>(), Num<1u>(), Num<4u>());
    else if (cols <= 4096u) go(Num<256u>(), Num<2u>(), Num<2u>());
    else if (cols <= 8192u) go(Num<512u>(), Num<2u>(), Num<1u>());
    else go(Num<1024u>(), Num<4u>(), Num<1u>());
    st = launch_status();
    if (st != CIERA_OK) return st;
  }
  if (d_dw) launch(k_rms_norm_join, dim3(uint32_t(cdiv(cols, 32u))), dim3(1024), stream, p);
  return launch_status();
}

}  // extern "C"
