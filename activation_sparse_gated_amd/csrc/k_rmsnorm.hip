// RMS norm with the residual's addition, and its gradients, on gfx950.
//
//   r = x + residual, rstd = 1 / sqrt(mean(r^2) + eps), y = r rstd w;
//   h = r rstd, v = w dy: dx = rstd (v - h mean(v h)) + dr, dw = sum_t dy h.
//
// Both are bound by HBM: a row is read once and stays in registers between
// the sum over it and what is written from it. TPR threads share a row, each
// holding NC chunks of 8 elements (16-byte loads of bf16); the sum is a
// butterfly in the wave, and one LDS exchange where a row spans waves. With
// 8-bit output the 16 lanes of a DPP row hold exactly one block of 128
// columns, so a block's maximum is four lane moves and no LDS. Measured (bf16,
// residual, 8-bit output): 4096 x 4096 22.1 us, 5.3 TB/s (from fp32 39.3 us); 1 x
// 4096 2.4 us, all latency. Backward with the residual's gradient, 4095 x 2048:
// 13.4-14.0 us (5.0 TB/s) and 3-4 us for the sum of the workgroups' rows of dw:
// two a CU, so that a row is in flight per wave while they hold 4 MB of partial
// sums.
#include "lin_util.cuh"

namespace ffn {

// Sum over the TPR threads of a row: every one of them gets the same value.
template <int TPR>
__device__ __forceinline__ float row_sum(float v, float* s_red) {
  v = wave_sum(v);
  if constexpr (TPR > 64) {
    const int wave = threadIdx.x >> 6;
    if ((threadIdx.x & 63) == 0) s_red[wave] = v;
    __syncthreads();
    v = 0.f;
#pragma unroll
    for (int i = 0; i < TPR / 64; ++i) v += s_red[i];
  }
  return v;
}

template <typename T, int TPR, int NC>
__global__ __launch_bounds__(TPR < 256 ? 256 : TPR) void k_rmsnorm_fwd(const NormDesc n) {
  constexpr int RPB = TPR < 256 ? 256 / TPR : 1;
  __shared__ float s_red[TPR / 64];
  const int t = threadIdx.x % TPR;
  const int row = (blockIdx.y * gridDim.x + blockIdx.x) * RPB + threadIdx.x / TPR;
  if (row >= n.m) return;                        // TPR > 64: one row a workgroup, all of it returns
  const size_t base = (size_t)row * n.d;
  Row8<T> xv[NC], rv[NC], wv[NC];
#pragma unroll
  for (int i = 0; i < NC; ++i) {
    const int c = (t + i * TPR) * 8;
    xv[i].zero();
    rv[i].zero();
    wv[i].zero();
    if (c < n.d) {
      xv[i].load(n.x, base + c);
      if (n.res) rv[i].load(n.res, base + c);
      wv[i].load(n.w, c);
    }
  }
  float f[NC][8];
  float ss = 0.f;
#pragma unroll
  for (int i = 0; i < NC; ++i) {
    xv[i].get(f[i]);
    if (n.res) {
      float g[8];
      rv[i].get(g);
#pragma unroll
      for (int j = 0; j < 8; ++j) f[i][j] += g[j];
      Row8<T>::round(f[i]);                      // the norm is of the rows as stored, which the backward pass reads
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) ss = fmaf(f[i][j], f[i][j], ss);
    const int c = (t + i * TPR) * 8;
    if (n.r_out && c < n.d) Row8<T>::store(n.r_out, base + c, f[i]);
  }
  ss = row_sum<TPR>(ss, s_red);
  const float rstd = rsqrtf(ss / (float)n.d + n.eps);
#pragma unroll
  for (int i = 0; i < NC; ++i) {
    const int c = (t + i * TPR) * 8;
    float w[8];
    wv[i].get(w);
#pragma unroll
    for (int j = 0; j < 8; ++j) f[i][j] = f[i][j] * rstd * w[j];
    if (n.y && c < n.d) Row8<T>::store(n.y, base + c, f[i]);
    if (n.q) {
      const float s = fp8_scale(row16_max(max8(f[i], 0u)));
      if (c < n.d) {
        *reinterpret_cast<uint2*>(n.q + base + c) = fp8_pack8(f[i], 1.0f / s);
        if ((threadIdx.x & 15) == 0) n.scale[(size_t)(c / kFp8Block) * n.m + row] = s;
      }
    }
  }
}

// dx of the rows, and the sum of dy h over this workgroup's rows (every
// gridDim.x-th group of them, in order) as one row of partial sums.
template <typename T, int TPR, int NC>
__global__ __launch_bounds__(TPR < 256 ? 256 : TPR) void k_rmsnorm_bwd(const NormDesc n) {
  constexpr int RPB = TPR < 256 ? 256 / TPR : 1;
  __shared__ float s_red[2][TPR / 64];
  __shared__ float s_dw[RPB > 1 ? RPB - 1 : 1][RPB > 1 ? NC * TPR * 8 : 1];
  const int t = threadIdx.x % TPR, u = threadIdx.x / TPR;
  float w[NC][8], dw[NC][8];
#pragma unroll
  for (int i = 0; i < NC; ++i) {
    const int c = (t + i * TPR) * 8;
    Row8<T> wv;
    wv.zero();
    if (c < n.d) wv.load(n.w, c);
    wv.get(w[i]);
#pragma unroll
    for (int j = 0; j < 8; ++j) dw[i][j] = 0.f;
  }
  for (int row = blockIdx.x * RPB + u; row < n.m; row += gridDim.x * RPB) {
    const size_t base = (size_t)row * n.d;
    Row8<T> xv[NC], gv[NC], av[NC];
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      const int c = (t + i * TPR) * 8;
      xv[i].zero();
      gv[i].zero();
      av[i].zero();
      if (c < n.d) {
        xv[i].load(n.x, base + c);
        gv[i].load(n.dy, base + c);
        if (n.res) av[i].load(n.res, base + c);
      }
    }
    float ss = 0.f, sv = 0.f;
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      float f[8], g[8];
      xv[i].get(f);
      gv[i].get(g);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        ss = fmaf(f[j], f[j], ss);
        sv = fmaf(f[j] * w[i][j], g[j], sv);
      }
    }
    if constexpr (TPR > 64) __syncthreads();     // the last row's sums have been read
    ss = row_sum<TPR>(ss, s_red[0]);
    sv = row_sum<TPR>(sv, s_red[1]);
    const float rstd = rsqrtf(ss / (float)n.d + n.eps);
    const float mean = sv * rstd / (float)n.d;
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      const int c = (t + i * TPR) * 8;
      float f[8], g[8], a[8];
      xv[i].get(f);
      gv[i].get(g);
      av[i].get(a);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float h = f[j] * rstd;
        dw[i][j] = fmaf(g[j], h, dw[i][j]);
        a[j] = fmaf(rstd, fmaf(w[i][j], g[j], -h * mean), a[j]);
      }
      if (n.dx && c < n.d) Row8<T>::store(n.dx, base + c, a);
    }
  }
  if (!n.dw) return;
  if constexpr (RPB > 1) {
    if (u > 0) {
#pragma unroll
      for (int i = 0; i < NC; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j) s_dw[u - 1][(i * 8 + j) * TPR + t] = dw[i][j];
    }
    __syncthreads();
    if (u > 0) return;
    for (int v = 0; v < RPB - 1; ++v)
#pragma unroll
      for (int i = 0; i < NC; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j) dw[i][j] += s_dw[v][(i * 8 + j) * TPR + t];
  }
#pragma unroll
  for (int i = 0; i < NC; ++i) {
    const int c = (t + i * TPR) * 8;
    if (c < n.d) Row8<float>::store(n.part, (size_t)blockIdx.x * n.d + c, dw[i]);
  }
}

// dw[c] = the partial rows' sum: 32 columns a workgroup, each column's parts
// in 32 interleaved slices that are then added in order.
constexpr int kDwCols = 32, kDwSlices = 32;
__global__ __launch_bounds__(kDwCols* kDwSlices) void k_rmsnorm_dw(const NormDesc n) {
  __shared__ float s[kDwSlices][kDwCols + 1];
  const int c = threadIdx.x % kDwCols, z = threadIdx.x / kDwCols;
  const int col = blockIdx.x * kDwCols + c;
  float v = 0.f;
  if (col < n.d) {
#pragma unroll 8
    for (int p = z; p < n.parts; p += kDwSlices) v += n.part[(size_t)p * n.d + col];
  }
  s[z][c] = v;
  __syncthreads();
  if (z != 0 || col >= n.d) return;
  v = n.accumulate ? n.dw[col] : 0.f;
  for (int i = 0; i < kDwSlices; ++i) v += s[i][c];
  n.dw[col] = v;
}

// Workgroups of the backward pass, each with one partial row of dw: two a CU.
int rmsnorm_bwd_parts(int m, int d) {
  const int rpb = d <= 2048 ? 4 : 1;
  const int groups = (m + rpb - 1) / rpb;
  return groups < 512 ? groups : 512;
}

template <typename T, int TPR, int NC>
static hipError_t go_fwd(const NormDesc& n, hipStream_t s) {
  constexpr int RPB = TPR < 256 ? 256 / TPR : 1;
  // a grid holds fewer than 2^32 threads a dimension
  const int groups = (n.m + RPB - 1) / RPB, y = (groups + (1 << 21) - 1) >> 21;
  ffn_launch((k_rmsnorm_fwd<T, TPR, NC>), dim3((groups + y - 1) / y, y), dim3(TPR < 256 ? 256 : TPR), 0, s, n);
  return hipGetLastError();
}
template <typename T>
static hipError_t fwd(const NormDesc& n, hipStream_t s) {
  // chunks of 8 elements a row: as few threads as hold them in four chunks each
  const int c = n.d / 8;
  if (c <= 64) return go_fwd<T, 64, 1>(n, s);
  if (c <= 128) return go_fwd<T, 64, 2>(n, s);
  if (c <= 256) return go_fwd<T, 256, 1>(n, s);
  if (c <= 512) return go_fwd<T, 256, 2>(n, s);
  if (c <= 1024) return go_fwd<T, 256, 4>(n, s);
  return go_fwd<T, 1024, 2>(n, s);
}
hipError_t launch_rmsnorm_fwd(const NormDesc& n, hipStream_t s) {
  return n.dtype == DT_BF16 ? fwd<uint16_t>(n, s) : fwd<float>(n, s);
}

template <typename T, int TPR, int NC>
static hipError_t go_bwd(const NormDesc& n, hipStream_t s) {
  ffn_launch((k_rmsnorm_bwd<T, TPR, NC>), dim3(n.parts), dim3(TPR < 256 ? 256 : TPR), 0, s, n);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || !n.dw) return e;
  ffn_launch(k_rmsnorm_dw, dim3((n.d + kDwCols - 1) / kDwCols), dim3(kDwCols * kDwSlices), 0, s, n);
  return hipGetLastError();
}
template <typename T>
static hipError_t bwd(const NormDesc& n, hipStream_t s) {
  const int c = n.d / 8;
  if (c <= 64) return go_bwd<T, 64, 1>(n, s);
  if (c <= 128) return go_bwd<T, 64, 2>(n, s);
  if (c <= 256) return go_bwd<T, 64, 4>(n, s);
  if (c <= 512) return go_bwd<T, 256, 2>(n, s);
  if (c <= 1024) return go_bwd<T, 256, 4>(n, s);
  return go_bwd<T, 1024, 2>(n, s);
}
hipError_t launch_rmsnorm_bwd(const NormDesc& n, hipStream_t s) {
  return n.dtype == DT_BF16 ? bwd<uint16_t>(n, s) : bwd<float>(n, s);
}

}  // namespace ffn
