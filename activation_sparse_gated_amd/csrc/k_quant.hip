// 8-bit blocks with a scale each, and their transpose, on gfx950.
//
// A workgroup of 256 threads takes a 128 x 128 tile of x: 16 lanes hold a row
// of it (eight elements a lane), so a row's maximum is four lane moves. The
// values are read once; the transposed blocks come from the same tile through
// LDS, where a thread reads half a column (neighbouring lanes neighbouring
// columns: no bank conflicts) and writes 64 bytes of a transposed row. Bound by
// HBM: x once in, one or two bytes a value out. Measured, both outputs, bf16:
// 4091 x 8192 in rows 31.6 us, 14336 x 4096 in 128 x 128 blocks 54.4 us (4.3
// TB/s; with x in the memory-side cache 39 us).
#include <type_traits>

#include "lin_util.cuh"

namespace ffn {

constexpr int kQT = 128;                         // tile edge
// The tile in LDS, written 16 bytes at a time: its start and every row of it lie on 16-byte boundaries.
template <typename T>
struct alignas(16) QTile {
  static constexpr int LD = kQT + 16 / sizeof(T);  // one 16-byte chunk of padding a row
  static_assert(LD * sizeof(T) % 16 == 0, "rows of whole chunks");
  T x[kQT * LD];
};
struct QNoTile {
  static constexpr int LD = 0;
};

__device__ __forceinline__ float q_elem(const uint16_t* p) { return bf2f(*p); }
__device__ __forceinline__ float q_elem(const float* p) { return *p; }

template <typename T, int ROWS, bool TRANS>
__global__ __launch_bounds__(256) void k_fp8_quant(const QuantDesc d, int tiles_k, int tiles_m) {
  using Tile = std::conditional_t<TRANS, QTile<T>, QNoTile>;
  constexpr int LD = Tile::LD;
  static_assert(!TRANS || alignof(Tile) % 16 == 0, "16-byte LDS stores");
  __shared__ Tile s_x;
  __shared__ uint32_t s_max[4];
  __shared__ float s_scale[kQT];
  __shared__ uint32_t s_col[2][kQT];
  const int tid = threadIdx.x, c = tid & 15, r0 = tid >> 4;
  const int tk = blockIdx.x % tiles_k, rest = blockIdx.x / tiles_k;
  const int tm = rest % tiles_m, g = rest / tiles_m;
  const int k0 = tk * kQT, m0 = tm * kQT, col = k0 + c * 8;
  const size_t base = (size_t)g * d.m * d.k;
  Row8<T> v[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int row = m0 + r0 + 16 * i;
    v[i].zero();
    if (row < d.m && col < d.k) v[i].load(d.x, base + (size_t)row * d.k + col);
  }
  uint32_t mx[8], all = 0u;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    float f[8];
    v[i].get(f);
    mx[i] = row16_max(max8(f, 0u));
    all = max(all, mx[i]);
  }
  float sall = 0.f;
  if constexpr (ROWS > 1) {
    all = max(all, (uint32_t)wave_xchg_i<16>((int)all));
    all = max(all, (uint32_t)wave_xchg_i<32>((int)all));
    if ((tid & 63) == 0) s_max[tid >> 6] = all;
    __syncthreads();
    sall = fp8_scale(max(max(s_max[0], s_max[1]), max(s_max[2], s_max[3])));
    if (tid == 0) d.scale[((size_t)g * tiles_m + tm) * tiles_k + tk] = sall;
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int lr = r0 + 16 * i, row = m0 + lr;
    float f[8];
    v[i].get(f);
    const float s = ROWS > 1 ? sall : fp8_scale(mx[i]);
    if (ROWS == 1 && c == 0) s_scale[lr] = s;
    if (row < d.m && col < d.k) *reinterpret_cast<uint2*>(d.q + base + (size_t)row * d.k + col) = fp8_pack8(f, 1.0f / s);
    if constexpr (TRANS) Row8<T>::store(s_x.x, lr * LD + c * 8, f);
  }
  if (ROWS == 1 || TRANS) __syncthreads();
  if (ROWS == 1 && tid < kQT && m0 + tid < d.m) d.scale[((size_t)g * tiles_k + tk) * d.m + m0 + tid] = s_scale[tid];
  if constexpr (TRANS) {
    // column lc, rows 64 half .. + 63 of the tile
    const int lc = tid & (kQT - 1), half = tid >> 7;
    const T* p = s_x.x + half * 64 * LD + lc;
    float s = sall;
    if constexpr (ROWS == 1) {
      uint32_t m = 0u;
#pragma unroll 16
      for (int i = 0; i < 64; ++i) m = max(m, abs_bits(q_elem(p + i * LD)));
      s_col[half][lc] = m;
      __syncthreads();
      s = fp8_scale(max(s_col[0][lc], s_col[1][lc]));
      if (half == 0 && k0 + lc < d.k) d.scale_t[((size_t)g * tiles_m + tm) * d.k + k0 + lc] = s;
    } else if (tid == 0) {
      d.scale_t[((size_t)g * tiles_k + tk) * tiles_m + tm] = sall;
    }
    if (k0 + lc < d.k) {
      const float inv = 1.0f / s;
      uint8_t* out = d.qt + ((size_t)g * d.k + k0 + lc) * d.mt + m0 + half * 64;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if (m0 + half * 64 + j * 16 < d.mt) {
          uint2 h[2];
#pragma unroll
          for (int w = 0; w < 2; ++w) {
            float f[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) f[i] = q_elem(p + (j * 16 + w * 8 + i) * LD);
            h[w] = fp8_pack8(f, inv);
          }
          *reinterpret_cast<uint4*>(out + j * 16) = uint4{h[0].x, h[0].y, h[1].x, h[1].y};
        }
      }
    }
  }
}

template <typename T, int ROWS>
static hipError_t go_quant(const QuantDesc& d, hipStream_t s) {
  const int tk = (d.k + kQT - 1) / kQT, tm = (d.m + kQT - 1) / kQT;
  const dim3 grid((unsigned)((size_t)tk * tm * d.groups));
  if (d.qt) ffn_launch((k_fp8_quant<T, ROWS, true>), grid, dim3(256), 0, s, d, tk, tm);
  else ffn_launch((k_fp8_quant<T, ROWS, false>), grid, dim3(256), 0, s, d, tk, tm);
  return hipGetLastError();
}
hipError_t launch_fp8_quant(const QuantDesc& d, hipStream_t s) {
  if (d.dtype == DT_BF16) return d.block_rows == 1 ? go_quant<uint16_t, 1>(d, s) : go_quant<uint16_t, 128>(d, s);
  return d.block_rows == 1 ? go_quant<float, 1>(d, s) : go_quant<float, 128>(d, s);
}

}  // namespace ffn
