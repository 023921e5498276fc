// Device helpers of the operators around the FFN: typed 8-element rows, bf16
// and e4m3 rounding, the scale of an 8-bit block, the rows of an expert.
#pragma once
#include "common.cuh"
#include "linear.cuh"

namespace ffn {

// Two fp32 values as bf16 bits, rounded to nearest even (NaN stays NaN).
__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
  typedef __bf16 bf2 __attribute__((ext_vector_type(2)));
  typedef float f2 __attribute__((ext_vector_type(2)));
  return __builtin_bit_cast(uint32_t, __builtin_convertvector((f2{a, b}), bf2));
}
__device__ __forceinline__ float round_bf16(float a) { return __uint_as_float(pack_bf16(a, 0.f) << 16); }

// Eight consecutive elements of a bf16 or fp32 row.
template <typename T>
struct Row8;
template <>
struct Row8<uint16_t> {
  uint4 v;
  __device__ __forceinline__ void load(const void* p, size_t i) { v = ldg16(reinterpret_cast<const uint16_t*>(p) + i); }
  __device__ __forceinline__ void zero() { v = uint4{0, 0, 0, 0}; }
  __device__ __forceinline__ void get(float (&f)[8]) const { unpack8(v, f); }
  __device__ __forceinline__ static void round(float (&f)[8]) {
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = round_bf16(f[i]);
  }
  __device__ __forceinline__ static void store(void* p, size_t i, const float (&f)[8]) {
    *reinterpret_cast<uint4*>(reinterpret_cast<uint16_t*>(p) + i) =
        uint4{pack_bf16(f[0], f[1]), pack_bf16(f[2], f[3]), pack_bf16(f[4], f[5]), pack_bf16(f[6], f[7])};
  }
};
template <>
struct Row8<float> {
  float4 a, b;
  __device__ __forceinline__ void load(const void* p, size_t i) {
    const float4* q = reinterpret_cast<const float4*>(reinterpret_cast<const float*>(p) + i);
    a = q[0];
    b = q[1];
  }
  __device__ __forceinline__ void zero() { a = b = float4{0.f, 0.f, 0.f, 0.f}; }
  __device__ __forceinline__ void get(float (&f)[8]) const {
    f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
    f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
  }
  __device__ __forceinline__ static void round(float (&)[8]) {}
  __device__ __forceinline__ static void store(void* p, size_t i, const float (&f)[8]) {
    float4* q = reinterpret_cast<float4*>(reinterpret_cast<float*>(p) + i);
    q[0] = float4{f[0], f[1], f[2], f[3]};
    q[1] = float4{f[4], f[5], f[6], f[7]};
  }
};

// |v| as ordered bits: a NaN is the largest, so that a maximum keeps it.
__device__ __forceinline__ uint32_t abs_bits(float v) { return __float_as_uint(v) & 0x7FFFFFFFu; }
__device__ __forceinline__ uint32_t max8(const float (&f)[8], uint32_t m) {
#pragma unroll
  for (int i = 0; i < 8; ++i) m = max(m, abs_bits(f[i]));
  return m;
}
// Maximum over each 16-lane row of the wave.
__device__ __forceinline__ uint32_t row16_max(uint32_t m) {
  m = max(m, (uint32_t)wave_xchg_i<1>((int)m));
  m = max(m, (uint32_t)wave_xchg_i<2>((int)m));
  m = max(m, (uint32_t)wave_xchg_i<4>((int)m));
  m = max(m, (uint32_t)wave_xchg_i<8>((int)m));
  return m;
}
// Scale of a block whose largest magnitude has these bits: max|x| / 448 as one
// fp32 product, at least 2^-100 (a block of zeros, or of values so small that
// the reciprocal of its scale would overflow). NaN and infinity pass through.
__device__ __forceinline__ float fp8_scale(uint32_t amax_bits) {
  const float s = __uint_as_float(amax_bits) * (1.0f / 448.0f);
  return s < 0x1p-100f ? 0x1p-100f : s;
}
// Eight values times inv as e4m3 (round to nearest even; |v * inv| <= 448 (1 + 2^-22)
// rounds to at most 448).
__device__ __forceinline__ uint2 fp8_pack8(const float (&f)[8], float inv) {
  int lo = __builtin_amdgcn_cvt_pk_fp8_f32(f[0] * inv, f[1] * inv, 0, false);
  lo = __builtin_amdgcn_cvt_pk_fp8_f32(f[2] * inv, f[3] * inv, lo, true);
  int hi = __builtin_amdgcn_cvt_pk_fp8_f32(f[4] * inv, f[5] * inv, 0, false);
  hi = __builtin_amdgcn_cvt_pk_fp8_f32(f[6] * inv, f[7] * inv, hi, true);
  return uint2{(uint32_t)lo, (uint32_t)hi};
}

// Where the rows of expert g start (g = groups: where the last one's end),
// whatever the offsets hold: inside 0..m here, and by the callers never before
// an earlier one, so that every row belongs to one expert at most.
__device__ __forceinline__ int expert_start(const int32_t* offsets, int g, int m) {
  return offsets ? min(max(offsets[g], 0), m) : g ? m : 0;
}
// Tile `tile` of RT rows: expert g, first output row r0, end of its rows.
// Tiles count expert by expert; false past the last one.
template <int RT>
__device__ __forceinline__ bool lin_tile(const LinDesc& d, int tile, int& g, int& r0, int& rend) {
  int lo = expert_start(d.offsets, 0, d.rows);
  for (g = 0; g < d.groups; ++g) {
    rend = max(lo, expert_start(d.offsets, g + 1, d.rows));
    const int t = (rend - lo + RT - 1) / RT;
    if (tile < t) {
      r0 = lo + tile * RT;
      return true;
    }
    tile -= t;
    lo = rend;
  }
  return false;
}

// Four neighbouring outputs (row, col ..) in one store of 16 (bf16: 8) bytes:
// to the slab of slice z, or to the output. d.cols is a multiple of 4.
__device__ __forceinline__ void lin_store4(const LinDesc& d, int z, int row, int col, f32x4_t a) {
  const size_t at = (size_t)row * d.cols + col;
  if (d.ks > 1) *reinterpret_cast<f32x4_t*>(d.part + (size_t)z * d.rows * d.cols + at) = a;
  else if (d.out_f32) *reinterpret_cast<f32x4_t*>(reinterpret_cast<float*>(d.out) + at) = a;
  else *reinterpret_cast<uint2*>(reinterpret_cast<uint16_t*>(d.out) + at) = uint2{pack_bf16(a[0], a[1]), pack_bf16(a[2], a[3])};
}
// The same, added to what the output holds if the product accumulates; columns
// past the end are left out.
__device__ __forceinline__ void lin_store(const LinDesc& d, int z, int row, int col, f32x4_t a) {
  const bool add = d.ks == 1 && d.accumulate;
  const size_t at = (size_t)row * d.cols + col;
  float* f = (d.ks > 1 ? d.part + (size_t)z * d.rows * d.cols : reinterpret_cast<float*>(d.out)) + at;
  if ((d.cols & 3) == 0) {
    if (add) a += *reinterpret_cast<const f32x4_t*>(f);
    lin_store4(d, z, row, col, a);
    return;
  }
#pragma unroll
  for (int v = 0; v < 4; ++v) {
    if (col + v >= d.cols) break;
    if (d.ks > 1 || d.out_f32) f[v] = add ? f[v] + a[v] : a[v];
    else reinterpret_cast<uint16_t*>(d.out)[at + v] = (uint16_t)pack_bf16(a[v], 0.f);
  }
}

// ---------------------------------------------------------------- matrix operands
typedef int i32x8_t __attribute__((ext_vector_type(8)));
__device__ __forceinline__ i32x8_t as_i32x8(const uint4 a, const uint4 b) {
  return i32x8_t{(int)a.x, (int)a.y, (int)a.z, (int)a.w, (int)b.x, (int)b.y, (int)b.z, (int)b.w};
}
// Eight e4m3 values as bf16 (exact).
__device__ __forceinline__ bf16x8_t fp8_to_bf16(uint32_t lo, uint32_t hi) {
  typedef __bf16 bf2 __attribute__((ext_vector_type(2)));
  const bf2 a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 1.0f, false), b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 1.0f, true);
  const bf2 c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 1.0f, false), d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 1.0f, true);
  return bf16x8_t{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
}

}  // namespace ffn
