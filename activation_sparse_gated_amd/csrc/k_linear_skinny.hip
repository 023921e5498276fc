// The products of k_linear.hip for few rows (a decode batch, the few tokens of
// an expert), where the weights are read once and everything else is small:
// bound by HBM, so the kernel is made to have many weight loads in flight.
//
// A workgroup of NW waves owns 16 CB columns and the 16 MB rows of one row
// tile; the waves take the 128-byte blocks of the contraction in turn. A wave
// loads its operands straight from memory into registers in the matrix
// instructions' layout (operand lane l: row l % 16, chunks of 16 bytes l / 16
// and l / 16 + 4 of the block), U blocks ahead; nothing is shared, so there is
// no barrier before the waves' sums are added in LDS, in wave order. The rows'
// blocks come from L2, 16 MB rows for 16 CB columns: with more rows a wave
// takes two column tiles, which halves that traffic. Where the columns give
// too few workgroups for the chip, the contraction is also cut into ks slices
// of whole blocks (blockIdx.y), each writing an fp32 slab that k_linear_sum
// adds in slice order. An 8-bit 4096 x 14336 product of one token takes 13.0 us
// (4.5 TB/s of weights), 16 rows over 8 experts of the same size in bf16
// 125-145 us (5.8-6.7 TB/s of those that have rows). Each workgroup finds its
// tile by walking the experts, with a row tile for each in the grid: 8 rows over 8
// experts of 2048 x 1024 take 8 us, over 16 15, over 64 175, over 256 2.76 ms.
#include "lin_util.cuh"

namespace ffn {

template <int KIND, bool EXACT, bool AROW, int MB, int CB, int NW, int U>
__global__ __launch_bounds__(NW * 64) void k_linear_skinny(const LinDesc d, int ctiles) {
  constexpr bool FP8 = KIND == LIN_FP8;
  constexpr int ESZ = FP8 ? 1 : 2, BK = 128 / ESZ, CE = 16 / ESZ;
  __shared__ f32x4_t s_acc[NW][MB * CB][64];
  const int lane = threadIdx.x & 63, l16 = lane & 15, q4 = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int c0 = blockIdx.x % ctiles * (16 * CB), z = blockIdx.y;
  int g, hi, r0;
  if (!lin_tile<16 * MB>(d, blockIdx.x / ctiles, g, r0, hi)) return;
  const int nb = (d.K + BK - 1) / BK;
  const int b0 = (int)((long long)nb * z / d.ks), b1 = (int)((long long)nb * (z + 1) / d.ks);

  const char* A = reinterpret_cast<const char*>(d.A) + (size_t)g * d.a_group * ESZ;
  const char* ap[CB];
  const char* bp[MB];
  const float *sap = nullptr, *sbp[MB];
  const int kblocks = nb;                        // 8-bit: the blocks of a row
#pragma unroll
  for (int c = 0; c < CB; ++c) ap[c] = A + (size_t)min(c0 + c * 16 + l16, d.cols - 1) * d.K * ESZ + q4 * 16;
#pragma unroll
  for (int m = 0; m < MB; ++m) {
    const int row = min(r0 + m * 16 + l16, hi - 1);   // rows past the end repeat the last: their results are not stored
    bp[m] = reinterpret_cast<const char*>(d.B) + (size_t)row * d.K * ESZ + q4 * 16;
    sbp[m] = FP8 ? d.sb + row : nullptr;
  }
  // 16 CB columns lie in one block of 128 rows of A
  if (FP8 && !AROW) sap = d.sa + ((size_t)g * ((d.cols + kFp8Block - 1) / kFp8Block) + c0 / kFp8Block) * kblocks;

  struct Block {
    uint4 a[CB][2], b[MB][2];
    float sa, sb[MB], sr[AROW ? CB : 1][AROW ? 4 : 1];
  };
  Block ring[U];
  auto load = [&](Block& x, int b) {
    const size_t o = (size_t)b * 128;
    const int left = d.K - b * BK;               // contraction elements from here on
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      if (left >= BK) {
#pragma unroll
        for (int c = 0; c < CB; ++c) x.a[c][h] = ldg16(ap[c] + o + h * 64);
#pragma unroll
        for (int m = 0; m < MB; ++m) x.b[m][h] = ldg16(bp[m] + o + h * 64);
      } else {                                   // zeros behind the last element
        const bool in = (q4 + 4 * h) * CE < left;
#pragma unroll
        for (int c = 0; c < CB; ++c) x.a[c][h] = in ? ldg16(ap[c] + o + h * 64) : uint4{0, 0, 0, 0};
#pragma unroll
        for (int m = 0; m < MB; ++m) x.b[m][h] = in ? ldg16(bp[m] + o + h * 64) : uint4{0, 0, 0, 0};
      }
    }
    if constexpr (FP8) {
#pragma unroll
      for (int m = 0; m < MB; ++m) x.sb[m] = sbp[m][(size_t)b * d.rows];
      if constexpr (AROW) {
#pragma unroll
        for (int c = 0; c < CB; ++c)
#pragma unroll
          for (int v = 0; v < 4; ++v) x.sr[c][v] = d.sa[(size_t)b * d.cols + min(c0 + c * 16 + 4 * q4 + v, d.cols - 1)];
      } else {
        x.sa = sap[b];
      }
    }
  };
  f32x4_t acc[MB][CB];
#pragma unroll
  for (int m = 0; m < MB; ++m)
#pragma unroll
    for (int c = 0; c < CB; ++c) acc[m][c] = f32x4_t{0.f, 0.f, 0.f, 0.f};
  auto use = [&](const Block& x) {
#pragma unroll
    for (int m = 0; m < MB; ++m)
#pragma unroll
      for (int c = 0; c < CB; ++c) {
        if constexpr (!FP8) {
#pragma unroll
          for (int h = 0; h < 2; ++h)
            acc[m][c] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(as_bf16x8(x.a[c][h]), as_bf16x8(x.b[m][h]), acc[m][c], 0, 0, 0);
        } else {
          f32x4_t p{0.f, 0.f, 0.f, 0.f};
          if constexpr (EXACT) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              p = __builtin_amdgcn_mfma_f32_16x16x32_bf16(fp8_to_bf16(x.a[c][h].x, x.a[c][h].y), fp8_to_bf16(x.b[m][h].x, x.b[m][h].y), p, 0, 0, 0);
              p = __builtin_amdgcn_mfma_f32_16x16x32_bf16(fp8_to_bf16(x.a[c][h].z, x.a[c][h].w), fp8_to_bf16(x.b[m][h].z, x.b[m][h].w), p, 0, 0, 0);
            }
          } else {
            p = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(as_i32x8(x.a[c][0], x.a[c][1]), as_i32x8(x.b[m][0], x.b[m][1]), p, 0, 0, 0, 0, 0, 0);
          }
#pragma unroll
          for (int v = 0; v < 4; ++v) acc[m][c][v] = fmaf(p[v], (AROW ? x.sr[AROW ? c : 0][AROW ? v : 0] : x.sa) * x.sb[m], acc[m][c][v]);
        }
      }
  };
  int b = b0 + wave;
#pragma unroll
  for (int u = 0; u < U; ++u)
    if (b + u * NW < b1) load(ring[u], b + u * NW);
  for (; b < b1; b += U * NW) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int at = b + u * NW;
      if (at < b1) {
        use(ring[u]);
        if (at + U * NW < b1) load(ring[u], at + U * NW);
      }
    }
  }
#pragma unroll
  for (int m = 0; m < MB; ++m)
#pragma unroll
    for (int c = 0; c < CB; ++c) s_acc[wave][m * CB + c][lane] = acc[m][c];
  __syncthreads();
  for (int t = wave; t < MB * CB; t += NW) {
    f32x4_t a = s_acc[0][t][lane];
#pragma unroll
    for (int w = 1; w < NW; ++w) a += s_acc[w][t][lane];
    const int row = r0 + t / CB * 16 + l16, col = c0 + t % CB * 16 + 4 * q4;
    if (row < hi && col < d.cols) lin_store(d, z, row, col, a);
  }
}

// out = the sum of the ks slabs in slice order, rows of some expert only.
__global__ __launch_bounds__(256) void k_linear_sum(const LinDesc d) {
  const int groups4 = (d.cols + 3) / 4;
  const long long at = (long long)blockIdx.x * 256 + threadIdx.x;
  const int row = (int)(at / groups4), col = (int)(at - (long long)row * groups4) * 4;
  if (row >= d.rows) return;
  // the experts' rows follow each other: all between the first start and the last end
  int end = expert_start(d.offsets, 0, d.rows);
  if (row < end) return;
  for (int g = 1; g <= d.groups; ++g) end = max(end, expert_start(d.offsets, g, d.rows));
  if (row >= end) return;
  const bool vec = (d.cols & 3) == 0;
  f32x4_t a{0.f, 0.f, 0.f, 0.f};
  for (int z = 0; z < d.ks; ++z) {
    const float* p = d.part + ((size_t)z * d.rows + row) * d.cols + col;
    if (vec) {
      a += *reinterpret_cast<const f32x4_t*>(p);
    } else {
#pragma unroll
      for (int v = 0; v < 4; ++v) a[v] += col + v < d.cols ? p[v] : 0.f;
    }
  }
  LinDesc o = d;
  o.ks = 1;
  lin_store(o, 0, row, col, a);
}

template <int KIND, bool EXACT, bool AROW, int MB, int CB, int NW, int U>
static hipError_t go_skinny(const LinDesc& d, hipStream_t s) {
  const int ct = (d.cols + 16 * CB - 1) / (16 * CB);
  const long long rt = d.rows / (16 * MB) + d.groups;
  ffn_launch((k_linear_skinny<KIND, EXACT, AROW, MB, CB, NW, U>), dim3((unsigned)(ct * rt), d.ks), dim3(NW * 64), 0, s, d, ct);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || d.ks == 1) return e;
  return launch_linear_sum(d, s);
}
hipError_t launch_linear_sum(const LinDesc& d, hipStream_t s) {
  const long long items = (long long)d.rows * ((d.cols + 3) / 4);
  ffn_launch(k_linear_sum, dim3((unsigned)((items + 255) / 256)), dim3(256), 0, s, d);
  return hipGetLastError();
}

template <int KIND, bool EXACT, bool AROW>
static hipError_t pick_skinny(const LinDesc& d, const LinPlan& p, hipStream_t s) {
  // exact sums and scales of single rows take registers: one column tile a wave, fewer blocks ahead
  constexpr bool BIG = EXACT || AROW;
  if (p.mb == 1) {
    if (p.nw == 16) return go_skinny<KIND, EXACT, AROW, 1, 1, 16, AROW ? 2 : 4>(d, s);
    return go_skinny<KIND, EXACT, AROW, 1, 1, 8, 4>(d, s);
  }
  return go_skinny<KIND, EXACT, AROW, 2, BIG ? 1 : 2, 8, 2>(d, s);
}
hipError_t launch_linear_skinny(const LinDesc& d, const LinPlan& p, hipStream_t s) {
  if (d.kind == LIN_FWD) return pick_skinny<LIN_FWD, false, false>(d, p, s);
  if (d.kind != LIN_FP8) return hipErrorInvalidValue;
  if (d.a_rows == 1) return d.out_f32 ? pick_skinny<LIN_FP8, true, true>(d, p, s) : pick_skinny<LIN_FP8, false, true>(d, p, s);
  return d.out_f32 ? pick_skinny<LIN_FP8, true, false>(d, p, s) : pick_skinny<LIN_FP8, false, false>(d, p, s);
}

}  // namespace ffn
