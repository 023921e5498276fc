// Low-rank adapters of many requests beside a shared projection, on gfx950.
//
//   h = x A_g^T,  y = base + s_g h B_g^T;
//   dh = dy B_g,  dx = base + s_g dh A_g,  dA_g = s_g dh^T x,  dB_g = s_g dy^T h.
//
// Rows come by adapter; a tile is up to RT of one adapter's rows. The operands
// go from memory straight to registers in the order that the matrix
// instructions want: v_mfma_f32_16x16x32_bf16 takes from lane l eight
// consecutive elements of the contraction, group l / 16, of row l % 16, and
// leaves in it elements 4 (l / 16) + v of the first operand's rows, row l % 16 of
// the second's.
//
// h and dh stay in fp32 between the kernels and enter the second product as
// hi + lo, two bf16 numbers (2^-16 of the value is lost, a 256th of what the bf16
// output's rounding takes), for fp32 outputs as three (2^-24); with ranks up to 16
// the first two share one instruction, hi in the contraction's first half and
// lo in its second.
#include "adapter.cuh"
#include "lin_util.cuh"

namespace ffn {

constexpr int kDownWaves = 8;

// ---------------------------------------------------------------- tiles
// The first place of group g, never before an earlier one's: lanes hold P = ceil(groups / 64) groups each, one after the
// other; `before` is the largest start of the lanes before.
struct Groups {
  int per, before, lane;
};
__device__ __forceinline__ Groups groups_of(const AdapterDesc& d) {
  Groups s;
  s.lane = lane_id();
  s.per = (d.groups + 63) >> 6;
  int mine = 0;
  for (int i = 0; i < s.per; ++i) {
    const int g = s.lane * s.per + i;
    if (g < d.groups) mine = max(mine, expert_start(d.offsets, g, d.m));
  }
  int v = mine;
#pragma unroll
  for (int o = 1; o < 64; o *= 2) {
    const int w = __shfl_up(v, o, 64);
    if (s.lane >= o) v = max(v, w);
  }
  const int w = __shfl_up(v, 1, 64);
  s.before = s.lane ? w : 0;
  return s;
}
// Calls f(g, first place, end) for this lane's groups in order.
template <typename F>
__device__ __forceinline__ void each_group(const AdapterDesc& d, const Groups& s, F f) {
  int lo = s.before;
  const int g0 = s.lane * s.per;
  if (g0 < d.groups) lo = max(lo, expert_start(d.offsets, g0, d.m));
  for (int i = 0; i < s.per; ++i) {
    const int g = g0 + i;
    if (g >= d.groups) break;
    const int hi = max(lo, expert_start(d.offsets, g + 1, d.m));
    f(g, lo, hi);
    lo = hi;
  }
}
// Tile `tile`: {adapter, first place, end, index of the adapter's first tile}. Tiles of rows without an adapter (-1) stand
// behind the others'. adapter -2: there is no such tile.
template <int RT>
__device__ __forceinline__ int4 adapter_tile(const AdapterDesc& d, int tile) {
  const Groups s = groups_of(d);
  int mine = 0, last = 0;
  each_group(d, s, [&](int, int lo, int hi) {
    mine += (hi - lo + RT - 1) / RT;
    last = hi;
  });
  const int incl = wave_incl_scan(mine);
  const uint64_t at = ballot64(incl > tile);
  if (at) {
    const int from = __ffsll((unsigned long long)at) - 1;
    int4 t = {0, 0, 0, 0};
    int first = incl - mine;
    each_group(d, s, [&](int g, int lo, int hi) {
      const int n = (hi - lo + RT - 1) / RT;
      if (tile >= first && tile < first + n) {
        const int r0 = lo + (tile - first) * RT;
        t = int4{g, r0, min(hi, r0 + RT), first};
      }
      first += n;
    });
    return int4{wave_read(t.x, from), wave_read(t.y, from), wave_read(t.z, from), wave_read(t.w, from)};
  }
  // rows of no adapter: before the first group, and behind the last
  const int total = wave_read(incl, 63);
  int end = last;
#pragma unroll
  for (int o = 1; o < 64; o *= 2) end = max(end, __shfl_xor(end, o, 64));
  const int lead = expert_start(d.offsets, 0, d.m), n0 = (lead + RT - 1) / RT;
  tile -= total;
  if (tile < n0) return int4{-1, tile * RT, min(lead, (tile + 1) * RT), 0};
  const int r0 = max(end, lead) + (tile - n0) * RT;
  if (r0 < d.m) return int4{-1, r0, min(d.m, r0 + RT), 0};
  return int4{-2, 0, 0, 0};
}
// The row at a place, -1 where there is none.
__device__ __forceinline__ int row_at(const AdapterDesc& d, int place) {
  const int row = d.rows ? d.rows[place] : place;
  return row < 0 || row >= d.m ? -1 : row;
}

__device__ __forceinline__ uint4 ldg16_if(bool in, const uint16_t* p) { return in ? ldg16(p) : uint4{0, 0, 0, 0}; }

// ---------------------------------------------------------------- first product
// h[place][j] = sum over i of u[row][i] A[j][i] for one tile and one slice of the contraction, whose steps the waves take
// in turn; their sums are added in order. ALONG: the weights' rows run along the contraction (A), otherwise across it (B).
template <int RT, int RB, bool ALONG>
__device__ __forceinline__ void down_tile(const AdapterDesc& d, const int4 tile, int z, const uint16_t* u, const uint16_t* w,
                                          int K, float* out, float* s_part) {
  constexpr int MB = RT / 16;
  const int lane = lane_id(), wave = threadIdx.x >> 6, l16 = lane & 15, q = lane >> 4;
  const uint16_t* up[MB];
#pragma unroll
  for (int i = 0; i < MB; ++i) {
    const int row = row_at(d, min(tile.y + i * 16 + l16, tile.z - 1));
    up[i] = u + (size_t)max(row, 0) * K;
  }
  const uint16_t* wg = w + (size_t)tile.x * d.r * K;
  f32x4_t acc[RB][MB];
#pragma unroll
  for (int b = 0; b < RB; ++b)
#pragma unroll
    for (int i = 0; i < MB; ++i) acc[b][i] = f32x4_t{0.f, 0.f, 0.f, 0.f};
  // steps of 64 elements
  const int steps = (K + 63) / 64, s0 = (int)((long long)steps * z / d.p.ks), s1 = (int)((long long)steps * (z + 1) / d.p.ks);
  auto step = [&](int at, bool whole) {
    uint4 uv[MB][2], wv[RB][2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int c = at * 64 + h * 32 + q * 8;
      const bool in = whole || c < K;
#pragma unroll
      for (int i = 0; i < MB; ++i) uv[i][h] = ldg16_if(in, up[i] + c);
#pragma unroll
      for (int b = 0; b < RB; ++b) {
        const int j = b * 16 + l16;
        if constexpr (ALONG) {
          wv[b][h] = ldg16_if(in, wg + (size_t)min(j, d.r - 1) * K + c);
        } else {
          uint32_t v[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) v[e] = in ? wg[(size_t)(c + e) * d.r + min(j, d.r - 1)] : 0u;
          wv[b][h] = uint4{v[0] | v[1] << 16, v[2] | v[3] << 16, v[4] | v[5] << 16, v[6] | v[7] << 16};
        }
      }
    }
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int b = 0; b < RB; ++b)
#pragma unroll
        for (int i = 0; i < MB; ++i)
          acc[b][i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(as_bf16x8(wv[b][h]), as_bf16x8(uv[i][h]), acc[b][i], 0, 0, 0);
  };
  const int whole = min(s1, K / 64);
  int at = s0 + wave;
#pragma unroll 2
  for (; at < whole; at += kDownWaves) step(at, true);
  if (at < s1) step(at, false);
  // the waves' sums, a block of 16 ranks at a time
#pragma unroll
  for (int b = 0; b < RB; ++b) {
    if (b) __syncthreads();
#pragma unroll
    for (int i = 0; i < MB; ++i)
      *reinterpret_cast<f32x4_t*>(s_part + ((wave * RT + i * 16 + l16) * 16 + q * 4)) = acc[b][i];
    __syncthreads();
    for (int e = threadIdx.x; e < RT * 16; e += kDownWaves * 64) {
      float v = 0.f;
#pragma unroll
      for (int w8 = 0; w8 < kDownWaves; ++w8) v += s_part[w8 * RT * 16 + e];
      const int row = e >> 4, j = b * 16 + (e & 15);
      const bool live = tile.y + row < tile.z && row_at(d, tile.y + row) >= 0;
      if (j < d.r) out[(size_t)row * d.r + j] = live ? v : 0.f;
    }
  }
}

template <int RT, int RB>
__global__ __launch_bounds__(kDownWaves * 64) void k_adapter_down(const AdapterDesc d, int with_h, int with_dh) {
  __shared__ __attribute__((aligned(16))) float s_part[kDownWaves * RT * 16];
  const int t = blockIdx.x, z = blockIdx.y;
  const int4 tile = adapter_tile<RT>(d, t);
  const bool back = blockIdx.z != 0 || !with_h;
  if (z == 0 && blockIdx.z == 0 && threadIdx.x == 0) d.tab[t] = tile;
  if (tile.x < 0) return;
  const size_t at = ((size_t)z * d.p.tiles + t) * RT * d.r;
  if (!back) down_tile<RT, RB, true>(d, tile, z, d.x, d.a, d.k, d.h + at, s_part);
  else down_tile<RT, RB, false>(d, tile, z, d.dy, d.b, d.n, d.dh + at, s_part);
}

template <int RT>
static hipError_t down(const AdapterDesc& d, hipStream_t s) {
  const int with_h = d.h != nullptr, with_dh = d.dh != nullptr;
  const dim3 grid(d.p.tiles, d.p.ks, with_h + with_dh), block(kDownWaves * 64);
  if (d.r <= 16) ffn_launch((k_adapter_down<RT, 1>), grid, block, 0, s, d, with_h, with_dh);
  else if (d.r <= 32) ffn_launch((k_adapter_down<RT, 2>), grid, block, 0, s, d, with_h, with_dh);
  else if (d.r <= 64) ffn_launch((k_adapter_down<RT, 4>), grid, block, 0, s, d, with_h, with_dh);
  else if (d.r <= 128) ffn_launch((k_adapter_down<RT, 8>), grid, block, 0, s, d, with_h, with_dh);
  else ffn_launch((k_adapter_down<RT, 16>), grid, block, 0, s, d, with_h, with_dh);
  return hipGetLastError();
}
hipError_t launch_adapter_down(const AdapterDesc& d, hipStream_t s) { return d.p.rt == 16 ? down<16>(d, s) : down<32>(d, s); }

// ---------------------------------------------------------------- second product
// 8 x 8 values of bf16, row e in in[e], as their columns.
__device__ __forceinline__ void transpose8(const uint4 (&in)[8], uint4 (&out)[8]) {
  uint32_t r[8][4];
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    r[e][0] = in[e].x;
    r[e][1] = in[e].y;
    r[e][2] = in[e].z;
    r[e][3] = in[e].w;
  }
#pragma unroll
  for (int c = 0; c < 8; ++c) {
    const uint32_t sel = c & 1 ? 0x07060302u : 0x05040100u;
    out[c] = uint4{__builtin_amdgcn_perm(r[1][c >> 1], r[0][c >> 1], sel), __builtin_amdgcn_perm(r[3][c >> 1], r[2][c >> 1], sel),
                   __builtin_amdgcn_perm(r[5][c >> 1], r[4][c >> 1], sel), __builtin_amdgcn_perm(r[7][c >> 1], r[6][c >> 1], sel)};
  }
}
__device__ __forceinline__ uint4 pack8(const float (&f)[8]) {
  return uint4{pack_bf16(f[0], f[1]), pack_bf16(f[2], f[3]), pack_bf16(f[4], f[5]), pack_bf16(f[6], f[7])};
}
// f - bf16(f); nothing behind an infinity
__device__ __forceinline__ void remainder8(float (&f)[8], const uint4 hi) {
  float g[8];
  unpack8(hi, g);
#pragma unroll
  for (int e = 0; e < 8; ++e) f[e] = fabsf(g[e]) == __builtin_huge_valf() ? 0.f : f[e] - g[e];
}

// out = base + s h W^T for a tile: wave w has 128 columns, column 8 (q + 4 v) + i of them in value v of accumulator i, so
// that a lane reads and writes eight neighbours. F: groups of 32 ranks (0: up to 16, hi and lo in one group).
// ALONG: W = B, rows of r elements a column; otherwise W = A^T, rows of the output's columns.
template <typename T, int RT, int F, bool ALONG>
__global__ __launch_bounds__(256) void k_adapter_up(const AdapterDesc d) {
  constexpr int NF = F == 0 ? 1 : F;
  const int lane = lane_id(), wave = threadIdx.x >> 6, l16 = lane & 15, q = lane >> 4;
  const int cols = ALONG ? d.n : d.k;
  const int c0 = (blockIdx.y * 4 + wave) * 128;
  if (c0 >= cols) return;
  const int4 tile = d.tab[blockIdx.x];
  if (tile.x == -2) return;
  if (tile.x == -1) {                            // no adapter: the base alone
    if (d.base == d.out) return;
    for (int e = lane; e < (tile.z - tile.y) * 16; e += 64) {
      const int row = row_at(d, tile.y + e / 16), c = c0 + e % 16 * 8;
      if (row < 0 || c >= cols) continue;
      Row8<T> v;
      float f[8];
      v.zero();
      if (d.base) v.load(d.base, (size_t)row * cols + c);
      v.get(f);
      Row8<T>::store(d.out, (size_t)row * cols + c, f);
    }
    return;
  }
  const float* hsrc = (ALONG ? d.h : d.dh) + (size_t)blockIdx.x * RT * d.r;
  const size_t slab = (size_t)d.p.tiles * RT * d.r;
  const float scale = d.scales ? d.scales[tile.x] : 1.f;
  const uint16_t* w = ALONG ? d.b + (size_t)tile.x * d.n * d.r : d.a + (size_t)tile.x * d.r * d.k;
  const int jq = F == 0 ? (q & 1) * 8 : q * 8;   // this lane's first rank in a group
  const int cb = c0 + 8 * ((l16 >> 2) + 4 * (l16 & 3));
#pragma unroll
  for (int i = 0; i < RT / 16; ++i) {
    const int place = tile.y + i * 16 + l16;
    if (tile.y + i * 16 >= tile.z) break;
    const int row = place < tile.z ? row_at(d, place) : -1;
    f32x4_t acc[8];
#pragma unroll
    for (int v = 0; v < 4; ++v) {
      const int c = c0 + 8 * (q + 4 * v);
      Row8<T> b;
      float f[8];
      b.zero();
      if (d.base && row >= 0 && c < cols) b.load(d.base, (size_t)row * cols + c);
      b.get(f);
#pragma unroll
      for (int e = 0; e < 8; ++e) acc[e][v] = f[e];
    }
#pragma unroll
    for (int g = 0; g < NF; ++g) {
      const int j = g * 32 + jq;
      float f[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
      if (j < d.r) {
        for (int z = 0; z < d.p.ks; ++z) {
          const f32x4_t* p = reinterpret_cast<const f32x4_t*>(hsrc + z * slab + (size_t)(i * 16 + l16) * d.r + j);
          const f32x4_t a = p[0], b = p[1];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            f[e] += a[e];
            f[4 + e] += b[e];
          }
        }
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) f[e] *= scale;
      uint4 hi = pack8(f);
      remainder8(f, hi);
      const uint4 lo = pack8(f);
      uint4 rest = {0, 0, 0, 0};
      if constexpr (sizeof(T) == 4) {
        remainder8(f, lo);
        if (F != 0 || q < 2) rest = pack8(f);
      }
      if constexpr (F == 0) hi = q < 2 ? hi : lo;
      uint4 wv[8];
      if constexpr (ALONG) {
#pragma unroll
        for (int e = 0; e < 8; ++e) wv[e] = ldg16_if(j < d.r, w + (size_t)min(cb + e, cols - 1) * d.r + j);
      } else {
        uint4 in[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) in[e] = ldg16_if(j < d.r && cb < cols, w + (size_t)(j + e) * cols + cb);
        transpose8(in, wv);
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) acc[e] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(as_bf16x8(wv[e]), as_bf16x8(hi), acc[e], 0, 0, 0);
      if constexpr (F != 0) {
#pragma unroll
        for (int e = 0; e < 8; ++e) acc[e] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(as_bf16x8(wv[e]), as_bf16x8(lo), acc[e], 0, 0, 0);
      }
      if constexpr (sizeof(T) == 4) {
#pragma unroll
        for (int e = 0; e < 8; ++e) acc[e] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(as_bf16x8(wv[e]), as_bf16x8(rest), acc[e], 0, 0, 0);
      }
    }
    if (row < 0) continue;
#pragma unroll
    for (int v = 0; v < 4; ++v) {
      const int c = c0 + 8 * (q + 4 * v);
      if (c >= cols) continue;
      float f[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) f[e] = acc[e][v];
      Row8<T>::store(d.out, (size_t)row * cols + c, f);
    }
  }
}

template <typename T, int RT, bool ALONG>
static hipError_t up(const AdapterDesc& d, hipStream_t s) {
  const int cols = ALONG ? d.n : d.k;
  const dim3 grid(d.p.tiles, (cols + 511) / 512), block(256);
  if (d.r <= 16) ffn_launch((k_adapter_up<T, RT, 0, ALONG>), grid, block, 0, s, d);
  else if (d.r <= 32) ffn_launch((k_adapter_up<T, RT, 1, ALONG>), grid, block, 0, s, d);
  else if (d.r <= 64) ffn_launch((k_adapter_up<T, RT, 2, ALONG>), grid, block, 0, s, d);
  else if (d.r <= 128) ffn_launch((k_adapter_up<T, RT, 4, ALONG>), grid, block, 0, s, d);
  else ffn_launch((k_adapter_up<T, RT, 8, ALONG>), grid, block, 0, s, d);
  return hipGetLastError();
}
hipError_t launch_adapter_up(const AdapterDesc& d, bool back, hipStream_t s) {
  if (back) return d.p.rt == 16 ? up<uint16_t, 16, false>(d, s) : up<uint16_t, 32, false>(d, s);
  if (d.out_f32) return d.p.rt == 16 ? up<float, 16, true>(d, s) : up<float, 32, true>(d, s);
  return d.p.rt == 16 ? up<uint16_t, 16, true>(d, s) : up<uint16_t, 32, true>(d, s);
}

// ---------------------------------------------------------------- gradients of the adapters
// dA[j][c] = s sum over the adapter's rows t of dh[t][j] x[t][c], and dB[c][j] = s sum of h[t][j] dy[t][c]: a workgroup
// has 128 columns c of one adapter and up to 16 RB ranks; its waves take 32 rows in turn, whose 8 x 8 pieces are turned
// in registers, and their sums are added in order. h enters as three bf16 numbers.
constexpr int kDwWaves = 8;
template <int RT, int RB, bool OF_A>
__device__ __forceinline__ void dw_tile(const AdapterDesc& d, int g, int c0, int j0, float* s_part) {
  const int lane = lane_id(), wave = threadIdx.x >> 6, l16 = lane & 15, q = lane >> 4;
  const int cols = OF_A ? d.k : d.n;
  const uint16_t* u = OF_A ? d.x : d.dy;
  // the adapter's places and its first tile
  const Groups s = groups_of(d);
  int mine = 0, start = 0, stop = 0, tiles = 0;
  each_group(d, s, [&](int at, int lo, int hi) {
    if (at == g) {
      start = lo;
      stop = hi;
      tiles = mine;
    }
    mine += (hi - lo + RT - 1) / RT;
  });
  const int owner = g / s.per;
  const int before = wave_read(wave_incl_scan(mine) - mine, owner) + wave_read(tiles, owner);
  const int lo = wave_read(start, owner), hi = wave_read(stop, owner);
  const float* h = (OF_A ? d.dh : d.h) + (size_t)before * RT * d.r;
  f32x4_t acc[8][RB];
#pragma unroll
  for (int i = 0; i < 8; ++i)
#pragma unroll
    for (int b = 0; b < RB; ++b) acc[i][b] = f32x4_t{0.f, 0.f, 0.f, 0.f};
  const int cb = c0 + 8 * ((l16 >> 2) + 4 * (l16 & 3));
  for (int r0 = wave * 32; r0 < hi - lo; r0 += kDwWaves * 32) {
    uint4 in[8], uv[8];
    int live = 0;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const int t = r0 + q * 8 + e;
      const int row = t < hi - lo ? row_at(d, lo + t) : -1;
      if (row >= 0) live |= 1 << e;
      in[e] = ldg16_if(row >= 0 && cb < cols, u + (size_t)max(row, 0) * cols + cb);
    }
    transpose8(in, uv);
#pragma unroll
    for (int b = 0; b < RB; ++b) {
      const int j = j0 + b * 16 + l16;
      float f[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) f[e] = j < d.r && (live >> e & 1) ? h[(size_t)(r0 + q * 8 + e) * d.r + j] : 0.f;
#pragma unroll
      for (int part = 0; part < 3; ++part) {
        const uint4 hv = pack8(f);
        remainder8(f, hv);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          if constexpr (OF_A) acc[i][b] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(as_bf16x8(uv[i]), as_bf16x8(hv), acc[i][b], 0, 0, 0);
          else acc[i][b] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(as_bf16x8(hv), as_bf16x8(uv[i]), acc[i][b], 0, 0, 0);
        }
      }
    }
  }
  // the waves' sums, 16 ranks of the 128 columns at a time: s_part[wave][value][lane] in fours
  const float scale = d.scales ? d.scales[g] : 1.f;
#pragma unroll
  for (int b = 0; b < RB; ++b) {
    if (b) __syncthreads();
#pragma unroll
    for (int i = 0; i < 8; ++i) *reinterpret_cast<f32x4_t*>(s_part + ((wave * 8 + i) * 64 + lane) * 4) = acc[i][b];
    __syncthreads();
    // thread (wave, lane) finishes accumulator `wave` of lane `lane`
    f32x4_t v = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int w = 0; w < kDwWaves; ++w) v += *reinterpret_cast<const f32x4_t*>(s_part + ((w * 8 + wave) * 64 + lane) * 4);
    const int i = wave;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      int j, c;
      if constexpr (OF_A) {
        j = j0 + b * 16 + l16;
        c = c0 + 8 * (q + 4 * e) + i;
      } else {
        j = j0 + b * 16 + 4 * q + e;
        c = cb + i;
      }
      if (j >= d.r || c >= cols) continue;
      float* out = OF_A ? d.da + ((size_t)g * d.r + j) * cols + c : d.db + ((size_t)g * cols + c) * d.r + j;
      const float o = scale * v[e];
      *out = d.accumulate ? *out + o : o;
    }
  }
}

template <int RT, int RB>
__global__ __launch_bounds__(kDwWaves * 64) void k_adapter_dw(const AdapterDesc d, int cols_a) {
  __shared__ __attribute__((aligned(16))) float s_part[kDwWaves * 8 * 64 * 4];
  const int j0 = blockIdx.z * (16 * RB);
  if ((int)blockIdx.x < cols_a) dw_tile<RT, RB, true>(d, blockIdx.y, blockIdx.x * 128, j0, s_part);
  else dw_tile<RT, RB, false>(d, blockIdx.y, (blockIdx.x - cols_a) * 128, j0, s_part);
}

template <int RT>
static hipError_t dw(const AdapterDesc& d, hipStream_t s) {
  const int ca = d.da ? (d.k + 127) / 128 : 0, cb = d.db ? (d.n + 127) / 128 : 0;
  const dim3 block(kDwWaves * 64);
  if (d.r <= 16) ffn_launch((k_adapter_dw<RT, 1>), dim3(ca + cb, d.groups, 1), block, 0, s, d, ca);
  else if (d.r <= 32) ffn_launch((k_adapter_dw<RT, 2>), dim3(ca + cb, d.groups, 1), block, 0, s, d, ca);
  else ffn_launch((k_adapter_dw<RT, 4>), dim3(ca + cb, d.groups, (d.r + 63) / 64), block, 0, s, d, ca);
  return hipGetLastError();
}
hipError_t launch_adapter_dw(const AdapterDesc& d, hipStream_t s) { return d.p.rt == 16 ? dw<16>(d, s) : dw<32>(d, s); }

// ---------------------------------------------------------------- plan
AdapterPlan adapter_plan(int m, int n, int k, int r, int groups, bool backward) {
  AdapterPlan p;
  p.rt = m >= 1024 ? 32 : 16;
  // every adapter's last tile may be short, and so may the two runs of rows without one
  const long long tiles = (long long)m / p.rt + groups + 2;
  p.tiles = (int)(tiles < m ? tiles : m);
  // slices: enough workgroups for the chip, while a wave still has a whole step
  int ks = 1;
  if (!backward) {
    const int live = (m + p.rt - 1) / p.rt;
    while (ks < 8 && live * ks < 256 && k / (ks * 2) >= 64 * kDownWaves) ks *= 2;
  }
  p.ks = ks;
  return p;
}

}  // namespace ffn
