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
constexpr uint32_t kNormParts = 512u;      // workgroups of the backward pass, each with a sum of dw of its own

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
  uint32_t rows, cols;
};

__device__ __forceinline__ float bf_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf_hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

// Eight values of a row from column `col`, zeros behind its end.
__device__ __forceinline__ u32x4v row_load8(const uint16_t* row, uint32_t col, uint32_t cols) {
  if (col + 8u <= cols) return u32x4v(*reinterpret_cast<const u32x4a2*>(row + col));
  return mx_part8(row + (col < cols ? col : 0u), col < cols ? cols - col : 0u);
}
__device__ __forceinline__ void row_store8(uint16_t* row, uint32_t col, uint32_t cols, u32x4v v) {
  if (col + 8u <= cols) {
    *reinterpret_cast<u32x4a2*>(row + col) = v;
  } else {
#pragma unroll
    for (uint32_t i = 0; i < 7u; i++)
      if (col + i < cols) row[col + i] = uint16_t(v[i >> 1] >> (16u * (i & 1u)));
  }
}

__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
  for (int d = 32; d > 0; d >>= 1) v += __shfl_xor(v, d);
  return v;
}

// The sum over the kT threads of a row.  With more than one wave a row the
// workgroup is the row: `part` holds a word a wave and is free again when the
// next barrier is passed.
template <uint32_t kT>
__device__ __forceinline__ float row_sum(float v, float* part) {
  v = wave_sum(v);
  if constexpr (kT > 64u) {
    if ((threadIdx.x & 63u) == 0u) part[threadIdx.x >> 6] = v;
    __syncthreads();
    v = 0.0f;
#pragma unroll
    for (uint32_t i = 0; i < kT / 64u; i++) v += part[i];
  }
  return v;
}

// A row takes kT threads, each kU units of 8 values, which stay in registers
// between the sum and the result.
template <uint32_t kT, uint32_t kU>
__global__ __launch_bounds__(kT < 256u ? 256u : kT) void k_rms_norm(NormArgs p) {
  constexpr uint32_t kB = kT < 256u ? 256u : kT;
  __shared__ float part[kT / 64u];
  const uint32_t t = threadIdx.x % kT;
  const uint32_t row = blockIdx.x * (kB / kT) + threadIdx.x / kT;
  if (row >= p.rows) return;
  const uint16_t* x = p.x + uint64_t(row) * p.ldx;
  const uint16_t* r = p.residual ? p.residual + uint64_t(row) * p.ldr : nullptr;
  u32x4v v[kU], a[kU];
#pragma unroll
  for (uint32_t u = 0; u < kU; u++) v[u] = row_load8(x, (u * kT + t) * 8u, p.cols);
  if (r) {
#pragma unroll
    for (uint32_t u = 0; u < kU; u++) a[u] = row_load8(r, (u * kT + t) * 8u, p.cols);
#pragma unroll
    for (uint32_t u = 0; u < kU; u++)
#pragma unroll
      for (int i = 0; i < 4; i++) v[u][i] = mx_bf16x2(bf_lo(v[u][i]) + bf_lo(a[u][i]), bf_hi(v[u][i]) + bf_hi(a[u][i]));
    if (p.h) {
#pragma unroll
      for (uint32_t u = 0; u < kU; u++) row_store8(p.h + uint64_t(row) * p.ldh, (u * kT + t) * 8u, p.cols, v[u]);
    }
  }
  float sum = 0.0f;
#pragma unroll
  for (uint32_t u = 0; u < kU; u++)
#pragma unroll
    for (int i = 0; i < 4; i++) sum = fmaf(bf_lo(v[u][i]), bf_lo(v[u][i]), fmaf(bf_hi(v[u][i]), bf_hi(v[u][i]), sum));
  sum = row_sum<kT>(sum, part);
  const float s = 1.0f / sqrtf(sum / float(p.cols) + p.eps);
  if (p.rstd && t == 0u) p.rstd[row] = s;
  const uint32_t kp = uint32_t(mx_pitch(p.cols));
#pragma unroll
  for (uint32_t u = 0; u < kU; u++) {
    const uint32_t col = (u * kT + t) * 8u;
    const u32x4v w = row_load8(p.w, col, p.cols);
    u32x4v y;
#pragma unroll
    for (int i = 0; i < 4; i++) y[i] = mx_bf16x2(bf_lo(v[u][i]) * s * bf_lo(w[i]), bf_hi(v[u][i]) * s * bf_hi(w[i]));
    if (col >= p.cols) y = u32x4v{0u, 0u, 0u, 0u};  // 0 s is NaN where s is
    else if (col + 8u > p.cols)
#pragma unroll
      for (uint32_t i = 1; i < 8u; i++)
        if (col + i >= p.cols) y[i >> 1] &= (i & 1u) ? 0xFFFFu : 0u;
    if (p.y) row_store8(p.y + uint64_t(row) * p.ldy, col, p.cols, y);
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
  void* dw;
  uint32_t dw_f32, accumulate, rows, cols, parts;
};

// A workgroup of kB threads takes every parts-th group of kB / kT rows and
// keeps the weights and its sums of dw in registers.
template <uint32_t kT, uint32_t kU, uint32_t kB>
__global__ __launch_bounds__(kB) void k_rms_norm_back(NormBackArgs p) {
  constexpr uint32_t kRows = kB / kT;
  __shared__ float part[2][kT / 64u];
  __shared__ float fold[kRows > 1u ? kRows * kT * 8u : 1u];
  const uint32_t t = threadIdx.x % kT, sub = threadIdx.x / kT;
  float dw[kU][8];
  u32x4v w[kU];
#pragma unroll
  for (uint32_t u = 0; u < kU; u++) {
    w[u] = row_load8(p.w, (u * kT + t) * 8u, p.cols);
#pragma unroll
    for (int i = 0; i < 8; i++) dw[u][i] = 0.0f;
  }
  uint32_t turn = 0u;
  for (uint32_t row = blockIdx.x * kRows + sub; row - sub < p.rows; row += p.parts * kRows, turn ^= 1u) {
    if (kRows > 1u && row >= p.rows) break;
    u32x4v h[kU], d[kU];
#pragma unroll
    for (uint32_t u = 0; u < kU; u++) h[u] = row_load8(p.h + uint64_t(row) * p.ldh, (u * kT + t) * 8u, p.cols);
#pragma unroll
    for (uint32_t u = 0; u < kU; u++) d[u] = row_load8(p.dy + uint64_t(row) * p.lddy, (u * kT + t) * 8u, p.cols);
    const float s = p.rstd[row];
    float dot = 0.0f;
#pragma unroll
    for (uint32_t u = 0; u < kU; u++)
#pragma unroll
      for (int i = 0; i < 4; i++) {
        const float u0 = bf_lo(h[u][i]) * s, u1 = bf_hi(h[u][i]) * s;
        const float d0 = bf_lo(d[u][i]), d1 = bf_hi(d[u][i]);
        dot = fmaf(d0 * bf_lo(w[u][i]), u0, fmaf(d1 * bf_hi(w[u][i]), u1, dot));
        dw[u][2 * i] = fmaf(d0, u0, dw[u][2 * i]);
        dw[u][2 * i + 1] = fmaf(d1, u1, dw[u][2 * i + 1]);
      }
    if (!p.dx) continue;
    const float m = row_sum<kT>(dot, part[turn]) / float(p.cols);
#pragma unroll
    for (uint32_t u = 0; u < kU; u++) {
      const uint32_t col = (u * kT + t) * 8u;
      u32x4v e = {0u, 0u, 0u, 0u}, o;
      if (p.dh) e = row_load8(p.dh + uint64_t(row) * p.lddh, col, p.cols);
#pragma unroll
      for (int i = 0; i < 4; i++) {
        const float g0 = bf_lo(d[u][i]) * bf_lo(w[u][i]), g1 = bf_hi(d[u][i]) * bf_hi(w[u][i]);
        o[i] = mx_bf16x2(fmaf(s, g0 - bf_lo(h[u][i]) * s * m, bf_lo(e[i])), fmaf(s, g1 - bf_hi(h[u][i]) * s * m, bf_hi(e[i])));
      }
      row_store8(p.dx + uint64_t(row) * p.lddx, col, p.cols, o);
    }
  }
  if (!p.dw) return;
  float* to = p.sums + uint64_t(blockIdx.x) * p.cols;
#pragma unroll
  for (uint32_t u = 0; u < kU; u++) {
    if constexpr (kRows > 1u) {
      __syncthreads();
#pragma unroll
      for (int i = 0; i < 8; i++) fold[(sub * 8u + i) * kT + t] = dw[u][i];
      __syncthreads();
      for (uint32_t i = threadIdx.x; i < kT * 8u; i += kB) {
        float v = 0.0f;
#pragma unroll
        for (uint32_t r = 0; r < kRows; r++) v += fold[(r * 8u + i % 8u) * kT + i / 8u];
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

// dw: the workgroups' sums added in order, 64 columns a workgroup, every
// sixteenth of the rows of sums a wave.
__global__ __launch_bounds__(1024) void k_rms_norm_join(NormBackArgs p) {
  __shared__ float part[16][64];
  const uint32_t lane = threadIdx.x & 63u, wave = threadIdx.x >> 6;
  const uint32_t col = blockIdx.x * 64u + lane;
  float v = 0.0f;
  if (col < p.cols) {
#pragma unroll 8
    for (uint32_t i = wave; i < p.parts; i += 16u) v += p.sums[uint64_t(i) * p.cols + col];
  }
  part[wave][lane] = v;
  __syncthreads();
  if (wave || col >= p.cols) return;
#pragma unroll
  for (uint32_t i = 1; i < 16u; i++) v += part[i][lane];
  if (p.dw_f32) {
    float* o = static_cast<float*>(p.dw) + col;
    *o = p.accumulate ? *o + v : v;
  } else {
    uint16_t* o = static_cast<uint16_t*>(p.dw) + col;
    *o = mx_bf16(p.accumulate ? mx_f32(*o) + v : v);
  }
}

// Rows a workgroup of the backward pass takes at once, and how many workgroups.
uint32_t norm_back_rows(uint32_t cols) { return cols <= 2048u ? 8u : 1u; }
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
  p.rows = uint32_t(rows);
  p.cols = uint32_t(cols);
  const uint64_t grid = cols <= 2048u ? cdiv(rows, 4u) : rows;
  if (grid > (cols <= 8192u ? kMxMostGroups : 0xFFFFFFFFull / 1024u)) return CIERA_ERR_ARG;
  (void)hipGetLastError();
  if (cols <= 2048u) launch(k_rms_norm<64u, 4u>, dim3(uint32_t(grid)), dim3(256), stream, p);
  else if (cols <= 8192u) launch(k_rms_norm<256u, 4u>, dim3(uint32_t(grid)), dim3(256), stream, p);
  else launch(k_rms_norm<1024u, 4u>, dim3(uint32_t(grid)), dim3(1024), stream, p);
  return launch_status();
}

uint64_t rms_norm_workspace_size(uint64_t rows, uint64_t cols) {
  if (rows > kMxMaxRows || cols == 0u || cols > kNormMaxCols) return 0u;
  const uint64_t parts = norm_back_parts(rows, uint32_t(cols));
  return align256((parts ? parts : 1u) * cols * 4u);
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
  p.sums = static_cast<float*>(d_ws);
  p.dw = d_dw;
  p.dw_f32 = dw_f32;
  p.accumulate = accumulate;
  p.rows = uint32_t(rows);
  p.cols = uint32_t(cols);
  p.parts = norm_back_parts(rows, uint32_t(cols));
  (void)hipGetLastError();
  if (rows) {
    if (cols <= 2048u) launch(k_rms_norm_back<64u, 4u, 512u>, dim3(p.parts), dim3(512), stream, p);
    else if (cols <= 8192u) launch(k_rms_norm_back<256u, 4u, 256u>, dim3(p.parts), dim3(256), stream, p);
    else launch(k_rms_norm_back<1024u, 4u, 1024u>, dim3(p.parts), dim3(1024), stream, p);
    st = launch_status();
    if (st != CIERA_OK) return st;
  }
  if (d_dw) launch(k_rms_norm_join, dim3(uint32_t(cdiv(cols, 64u))), dim3(1024), stream, p);
  return launch_status();
}

}  // extern "C"
