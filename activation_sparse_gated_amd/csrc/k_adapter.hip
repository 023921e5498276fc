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
//
// Bound by HBM: 2 r operations for each element of x, y, A and B. Many rows:
// 8192 x 4096 x 14336, rank 64, 29.8 us for the first product and 100.7 for the
// second (525 MB, 5.2 TB/s). Few rows: by the latency of the chain of loads and
// by the launches, one row 8.7 us in one launch, 48 rows of 32 adapters 5.9 and
// 7.1 in two.
#include <type_traits>

#include "adapter.cuh"
#include "lin_util.cuh"

namespace ffn {

constexpr int kDownWaves = 8;

// ---------------------------------------------------------------- tiles
// Running maximum over the wave's lanes (of values from 0 up), in DPP moves.
__device__ __forceinline__ int wave_incl_max(int v) {
  v = max(v, __builtin_amdgcn_update_dpp(0, v, 0x111, 0xF, 0xF, false));
  v = max(v, __builtin_amdgcn_update_dpp(0, v, 0x112, 0xF, 0xF, false));
  v = max(v, __builtin_amdgcn_update_dpp(0, v, 0x114, 0xF, 0xF, false));
  v = max(v, __builtin_amdgcn_update_dpp(0, v, 0x118, 0xF, 0xF, false));
  v = max(v, __builtin_amdgcn_update_dpp(0, v, 0x142, 0xA, 0xF, false));
  v = max(v, __builtin_amdgcn_update_dpp(0, v, 0x143, 0xC, 0xF, false));
  return v;
}
// Lanes hold `per` = ceil(groups / 64) groups each, one after the other. A group never starts before an earlier one:
// `before` is the largest start of the lanes before, `first` and `second` the starts of this lane's first group and of
// the one behind it as the offsets give them.
struct Groups {
  int per, g0, before, first, second;
};
__device__ __forceinline__ Groups groups_of(const AdapterDesc& d) {
  Groups s;
  s.per = (d.groups + 63) >> 6;
  s.g0 = lane_id() * s.per;
  s.first = expert_start(d.offsets, min(s.g0, d.groups), d.m);
  s.second = expert_start(d.offsets, min(s.g0 + 1, d.groups), d.m);
  int mine = s.first;
  for (int i = 1; i < s.per; ++i) mine = max(mine, expert_start(d.offsets, min(s.g0 + i, d.groups), d.m));
  const int v = wave_incl_max(mine), w = __shfl_up(v, 1, 64);
  s.before = lane_id() ? w : 0;
  return s;
}
// Calls f(g, first place, end) for this lane's groups in order.
template <typename F>
__device__ __forceinline__ void each_group(const AdapterDesc& d, const Groups& s, F f) {
  int lo = max(s.before, s.first);
  for (int i = 0; i < s.per; ++i) {
    const int g = s.g0 + i;
    if (g >= d.groups) break;
    const int hi = max(lo, i == 0 ? s.second : expert_start(d.offsets, g + 1, d.m));
    f(g, lo, hi);
    lo = hi;
  }
}
// The tile of workgroup `block` of `blocks` (a multiple of 8, no fewer than there are tiles): {adapter, first place, end,
// number}. Workgroups go to the 8 XCDs in turn; each XCD takes a run of neighbouring tiles, so that an adapter's weights
// are read into few of their L2s. Tiles of rows without an adapter (-1) stand behind the others'. adapter -2: no rows.
template <int RT>
__device__ __forceinline__ int4 adapter_tile(const AdapterDesc& d, int block, int blocks) {
  const Groups s = groups_of(d);
  int mine = 0, last = 0;
  each_group(d, s, [&](int, int lo, int hi) {
    mine += (hi - lo + RT - 1) / RT;
    last = hi;
  });
  const int incl = wave_incl_scan(mine), total = wave_read(incl, 63);
  const int per = (total + 7) >> 3, xcd = block & 7, at = block >> 3;
  int tile = xcd * per + at;
  if (at >= per) tile = total + (at - per) * 8 + xcd;            // the workgroups that no tile with an adapter is left for
  else if (tile >= total) tile += blocks - 8 * per;
  if (tile < total) {
    const int from = __ffsll((unsigned long long)ballot64(incl > tile)) - 1;
    int4 t = {0, 0, 0, 0};
    int first = incl - mine;
    each_group(d, s, [&](int g, int lo, int hi) {
      const int n = (hi - lo + RT - 1) / RT;
      if (tile >= first && tile < first + n) {
        const int r0 = lo + (tile - first) * RT;
        t = int4{g, r0, min(hi, r0 + RT), 0};
      }
      first += n;
    });
    return int4{wave_read(t.x, from), wave_read(t.y, from), wave_read(t.z, from), tile};
  }
  // rows of no adapter: before the first group, and behind the last
  const int end = wave_read(wave_incl_max(last), 63);
  const int lead = wave_read(s.first, 0), n0 = (lead + RT - 1) / RT, n = tile - total;
  if (n < n0) return int4{-1, n * RT, min(lead, (n + 1) * RT), tile};
  const int r0 = max(end, lead) + (n - n0) * RT;
  if (r0 < d.m) return int4{-1, r0, min(d.m, r0 + RT), tile};
  return int4{-2, 0, 0, tile};
}
// The row at a place, -1 where there is none.
__device__ __forceinline__ int row_at(const AdapterDesc& d, int place) {
  const int row = d.rows ? d.rows[place] : place;
  return row < 0 || row >= d.m ? -1 : row;
}
// v, or zeros. (Loads are made unconditionally, from a place that is there: a branch around each would end their overlap.)
__device__ __forceinline__ uint4 keep_if(bool in, const uint4 v) { return uint4{in ? v.x : 0u, in ? v.y : 0u, in ? v.z : 0u, in ? v.w : 0u}; }
__device__ const uint4 adapter_zero[2] = {{0, 0, 0, 0}, {0, 0, 0, 0}};
// f less the bf16 number that it became; nothing behind an infinity
__device__ __forceinline__ float rest_of(float f, uint32_t bf16) {
  const float g = bf2f(bf16);
  return fabsf(g) == __builtin_huge_valf() ? 0.f : f - g;
}

// ---------------------------------------------------------------- first product
// h[place][j] = sum over i of u[row][i] W[j][i] for one tile, one slice of the contraction and up to 16 RB ranks from j0
// on. The waves take the slice's steps of 64 elements in turn, each with the loads of its next one under way; their sums
// are added in order. (48 rows of 32 adapters, 4096 wide, rank 16, 8 slices: 5.9 us. With three to six steps' loads under
// way instead of one: no faster, 14.9 instead of 14.3 us in k_adapter_few.) ALONG: the weights' rows run along the
// contraction (A). Otherwise across it (B, rows of r elements): a step's 64 rows go through the wave's own part of LDS,
// which the transposing read turns: in each 16 lanes, lane 4 v + u points at row 8 q + 4 h + v, elements 4 u .. + 3, and
// lane j receives element j % 4 of lane 4 v + j / 4.
constexpr int kDownRanks = 64, kDown64Ranks = 128;               // of a workgroup, with tiles of 16 and of 64 rows
template <int RT, int RB>
struct DownLds {
  static constexpr int PART = kDownWaves * RT * 16 * 4;          // bytes of the waves' sums of 16 ranks
  static constexpr int W = 64 * 16 * RB * 2 + 32;                // of a wave's step of B; the last row's read runs on a little
  static constexpr int BYTES = PART > kDownWaves * W ? PART : kDownWaves * W;
};
// emit(row, j, sum) is called once for every row of the tile and rank.
template <int RT, int RB, bool ALONG, typename Emit>
__device__ __forceinline__ void down_tile(const AdapterDesc& d, const int4 tile, int z, int j0, char* lds, Emit emit) {
  constexpr int MB = RT / 16;
  const int lane = lane_id(), wave = threadIdx.x >> 6, l16 = lane & 15, q = lane >> 4;
  const uint16_t* u = ALONG ? d.x : d.dy;
  const int K = ALONG ? d.k : d.n;
  const uint16_t* up[MB];
#pragma unroll
  for (int i = 0; i < MB; ++i) up[i] = u + (size_t)max(row_at(d, min(tile.y + i * 16 + l16, tile.z - 1)), 0) * K;
  const uint16_t* wg = (ALONG ? d.a : d.b) + (size_t)tile.x * d.r * K + (ALONG ? (size_t)j0 * K : (size_t)j0);
  const int rw = min(d.r - j0, 16 * RB);         // ranks here
  const int lw = d.r <= kDownRanks ? d.r : kDownRanks;           // row of B in LDS
  char* mine = lds + wave * DownLds<RT, RB>::W;
  f32x4_t acc[RB][MB];
#pragma unroll
  for (int b = 0; b < RB; ++b)
#pragma unroll
    for (int i = 0; i < MB; ++i) acc[b][i] = f32x4_t{0.f, 0.f, 0.f, 0.f};
  const int ks = ALONG ? d.p.ks : d.p.kd;         // slices
  const int steps = (K + 63) / 64, s0 = (int)((long long)steps * z / ks), s1 = (int)((long long)steps * (z + 1) / ks);
  uint4 uv[2][MB][2], wv[2][RB * 2];
  int brow[RB * 2], bcol[RB * 2];                // this lane's chunks of eight elements of a step of B
  if constexpr (!ALONG) {
#pragma unroll
    for (int n = 0; n < RB * 2; ++n) {
      const int c = n * 64 + lane;
      brow[n] = d.r <= kDownRanks ? c * 8 / lw : c >> 3;
      bcol[n] = d.r <= kDownRanks ? c * 8 - brow[n] * lw : (c & 7) * 8;
    }
  }
  auto load = [&](auto slot, int at) {
    constexpr int D = decltype(slot)::value;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int c = min(at * 64 + h * 32 + q * 8, K - 8);
#pragma unroll
      for (int i = 0; i < MB; ++i) uv[D][i][h] = ldg16(up[i] + c);
      if constexpr (ALONG) {
#pragma unroll
        for (int b = 0; b < RB; ++b) wv[D][b * 2 + h] = ldg16(wg + (size_t)min(b * 16 + l16, rw - 1) * K + c);
      }
    }
    if constexpr (!ALONG) {
#pragma unroll
      for (int n = 0; n < RB * 2; ++n)
        wv[D][n] = ldg16(wg + (size_t)min(at * 64 + brow[n], K - 1) * d.r + min(bcol[n], rw - 8));
    }
  };
  auto use = [&](auto slot, int at) {
    constexpr int D = decltype(slot)::value;
    if (at * 64 + 64 > K) {                      // the last step: nothing behind the contraction's end
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const bool in = at * 64 + h * 32 + q * 8 < K;
#pragma unroll
        for (int i = 0; i < MB; ++i) uv[D][i][h] = keep_if(in, uv[D][i][h]);
        if constexpr (ALONG) {
#pragma unroll
          for (int b = 0; b < RB; ++b) wv[D][b * 2 + h] = keep_if(in, wv[D][b * 2 + h]);
        }
      }
      if constexpr (!ALONG) {
#pragma unroll
        for (int n = 0; n < RB * 2; ++n) wv[D][n] = keep_if(at * 64 + brow[n] < K, wv[D][n]);
      }
    }
    if constexpr (!ALONG) {
#pragma unroll
      for (int n = 0; n < RB * 2; ++n)
        if (brow[n] < 64) *reinterpret_cast<uint4*>(mine + (brow[n] * lw + bcol[n]) * 2) = wv[D][n];
    }
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int b = 0; b < RB; ++b) {
        bf16x8_t w;
        if constexpr (ALONG) {
          w = as_bf16x8(wv[D][b * 2 + h]);
        } else {
          typedef short s16x4 __attribute__((ext_vector_type(4)));
          typedef short s16x8 __attribute__((ext_vector_type(8)));
          const char* p = mine + ((h * 32 + 8 * q + (l16 >> 2)) * lw + b * 16 + 4 * (l16 & 3)) * 2;
          const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) s16x4*)p);
          const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) s16x4*)(p + 4 * lw * 2));
          w = __builtin_bit_cast(bf16x8_t, s16x8{lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]});
        }
#pragma unroll
        for (int i = 0; i < MB; ++i) acc[b][i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(w, as_bf16x8(uv[D][i][h]), acc[b][i], 0, 0, 0);
      }
  };
  using Zero = std::integral_constant<int, 0>;
  using One = std::integral_constant<int, 1>;
  int at = s0 + wave;
  if (at < s1) load(Zero{}, at);
  while (at < s1) {
    const bool more = at + kDownWaves < s1;
    if (more) load(One{}, at + kDownWaves);
    __builtin_amdgcn_sched_barrier(0);           // the loads go out before this step's products, not among them
    use(Zero{}, at);
    __builtin_amdgcn_sched_barrier(0);
    at += kDownWaves;
    if (!more) break;
    if (at + kDownWaves < s1) load(Zero{}, at + kDownWaves);
    __builtin_amdgcn_sched_barrier(0);
    use(One{}, at);
    __builtin_amdgcn_sched_barrier(0);
    at += kDownWaves;
  }
  // the waves' sums, a block of 16 ranks at a time
  float* s_part = reinterpret_cast<float*>(lds);
#pragma unroll
  for (int b = 0; b < RB; ++b) {
    __syncthreads();
#pragma unroll
    for (int i = 0; i < MB; ++i)
      *reinterpret_cast<f32x4_t*>(s_part + ((wave * RT + i * 16 + l16) * 16 + q * 4)) = acc[b][i];
    __syncthreads();
    for (int e = threadIdx.x; e < RT * 16; e += kDownWaves * 64) {
      float v = 0.f;
#pragma unroll
      for (int w = 0; w < kDownWaves; ++w) v += s_part[w * RT * 16 + e];
      const int row = e >> 4, j = j0 + b * 16 + (e & 15);
      if (tile.y + row >= tile.z || row_at(d, tile.y + row) < 0) v = 0.f;
      if (j < d.r) emit(row, j, v);
    }
  }
}

template <int RT, int RB>
__global__ __launch_bounds__(kDownWaves * 64) void k_adapter_down(const AdapterDesc d, int with_h, int chunks) {
  __shared__ __attribute__((aligned(16))) char lds[DownLds<RT, RB>::BYTES];
  const int z = blockIdx.y;
  const int4 tile = adapter_tile<RT>(d, blockIdx.x, gridDim.x);
  const int t = tile.w;
  if (t >= d.p.tiles) return;
  const bool back = (int)blockIdx.z >= chunks || !with_h;
  const int j0 = (blockIdx.z % chunks) * kDownRanks;
  if (z == 0 && blockIdx.z == 0 && threadIdx.x == 0) d.tab[t] = tile;
  if (tile.x < 0 || z >= (back ? d.p.kd : d.p.ks)) return;
  // backward and whole: what k_adapter_sum would make of it
  uint16_t* rows = back ? d.dhp : d.hp;
  uint16_t* turned = back ? d.dht : d.ht;
  const bool whole = (rows || turned) && (back ? d.p.kd : d.p.ks) == 1;
  const float scale = whole && d.scales ? d.scales[tile.x] : 1.f;
  const size_t at = (size_t)t * 3 * RT * d.r;
  float* out = (back ? d.dh : d.h) + ((size_t)z * d.p.tiles + t) * RT * d.r;
  auto emit = [&](int row, int j, float v) {
    if (!whole) {
      out[(size_t)row * d.r + j] = v;
      return;
    }
    v *= scale;
#pragma unroll
    for (int n = 0; n < 3; ++n) {
      const uint32_t part = pack_bf16(v, 0.f) & 0xFFFFu;
      if (rows && n < 2) rows[at + ((size_t)n * RT + row) * d.r + j] = (uint16_t)part;
      if (turned) turned[at + ((size_t)n * d.r + j) * RT + row] = (uint16_t)part;
      v = rest_of(v, part);
    }
  };
  if (!back) down_tile<RT, RB, true>(d, tile, z, j0, lds, emit);
  else down_tile<RT, RB, false>(d, tile, z, j0, lds, emit);
}

// The same for tiles of 64 rows: both operands' steps go straight from memory to LDS, 256 bytes of a row by neighbouring
// lanes, STAGES - 1 steps ahead of the products (a lane of the version above takes 16 bytes of a row of its own, and the
// weights come in anew for every 16 or 32 rows: 8192 x 4096, 64 ranks, 55 us). Wave (i, h) has rows 16 i .. and half h of
// each step, for all ranks. 8192 x 4096, 64 ranks: 29.8 us, of which the products take nothing (without them 29.1) and the
// weights 5.5; a plain read of the same 67 MB takes 15 to 16. Steps of 64 elements in 3 to 8 stages and two or four slices:
// 28.3 to 32.1, and 5.2 to 5.5 for the slices' sum. Tiles start at different steps, or all of them would read the same few
// channels of memory at a time. Rows of 256 bytes in LDS, chunk c at c ^ (row & 15): reads of rows meet no bank twice.
constexpr int kStep = 128, kStepBytes = 2 * kStep; // elements and bytes of a row in a step
__device__ __forceinline__ void to_lds16(const void* p, const char* l) {
  const uint32_t at = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) const char*)l;
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, off" ::"s"(at), "v"(p) : "m0");
}
// At most N loads to LDS are under way in this wave and its LDS reads are done, then every wave's.
template <int N>
__device__ __forceinline__ void lds_sync() {
  asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" ::"n"(N) : "memory");
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}
template <int RB>
struct Down64 {
  static constexpr int X = 64 * kStepBytes, W = 16 * RB * kStepBytes, STAGE = X + W;
  static constexpr int STAGES = RB == 8 ? 3 : 4;
  static constexpr int XL = X / 1024 / kDownWaves;                             // loads of a step of each wave
  static constexpr int WL = (W / 1024 + kDownWaves - 1) / kDownWaves;          // loads of the weights, of the waves that have any
  static constexpr int BYTES = STAGES * STAGE;
  static_assert(BYTES >= 4 * RB * 64 * 16 && BYTES <= 160 * 1024, "the second halves' sums, LDS of a CU");
};
template <int RB, bool ALONG>
__device__ __forceinline__ void down64_tile(const AdapterDesc& d, const int4 tile, int t, int z, int j0, char* lds) {
  using L = Down64<RB>;
  constexpr int RT = 64, S = L::STAGES;
  const int lane = lane_id(), l16 = lane & 15, q = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), wi = wave & 3, wh = wave >> 2;
  const uint16_t* u = ALONG ? d.x : d.dy;
  const int K = ALONG ? d.k : d.n;
  const int rw = min(d.r - j0, 16 * RB);         // ranks here
  const int lw = d.r <= kDown64Ranks ? d.r : kDown64Ranks;           // row of B in LDS
  const int ks = ALONG ? d.p.ks : d.p.kd;         // slices
  const int steps = (K + kStep - 1) / kStep, s0 = (int)((long long)steps * z / ks), n = (int)((long long)steps * (z + 1) / ks) - s0;
  // where this lane's loads come from: four rows of the tile for each, chunk (lane % 16) ^ row of them
  const uint16_t* xp[L::XL];
  int xk[L::XL];
#pragma unroll
  for (int i = 0; i < L::XL; ++i) {
    const int row = (i * kDownWaves + wave) * 4 + (lane >> 4);
    xk[i] = ((lane & 15) ^ (row & 15)) * 8;
    xp[i] = u + (size_t)max(row_at(d, min(tile.y + row, tile.z - 1)), 0) * K + xk[i];
  }
  const uint16_t* wp[L::WL];
  int wk[L::WL];                                 // contraction element of a step that the chunk starts at
#pragma unroll
  for (int i = 0; i < L::WL; ++i) {
    const int c = (i * kDownWaves + wave) * 64 + lane;
    if constexpr (ALONG) {
      const int row = c >> 4;
      wk[i] = ((c & 15) ^ (row & 15)) * 8;
      wp[i] = d.a + ((size_t)tile.x * d.r + j0 + min(row, rw - 1)) * K + wk[i];
    } else {
      const int row = d.r <= kDown64Ranks ? c * 8 / lw : c >> 4, col = d.r <= kDown64Ranks ? c * 8 - row * lw : (c & 15) * 8;
      wk[i] = min(row, kStep - 1);               // chunks past the step's rows: not read
      wp[i] = d.b + ((size_t)tile.x * K + wk[i]) * d.r + j0 + min(col, rw - 8);
    }
  }
  const bool has_w = L::W / 1024 >= kDownWaves || wave < L::W / 1024;
  const size_t wstep = ALONG ? kStep : (size_t)kStep * d.r;
  const int turn = n > 0 ? (int)((unsigned)(t * 5) % (unsigned)n) : 0;
  auto load = [&](int s) {
    int at = s + turn;
    at = s0 + (at >= n ? at - n : at);
    char* stage = lds + s % S * L::STAGE;
    const bool part = (at + 1) * kStep > K;
    const void* p;
#pragma unroll
    for (int i = 0; i < L::XL; ++i) {
      p = xp[i] + (size_t)at * kStep;
      if (part && at * kStep + xk[i] >= K) p = adapter_zero;
      to_lds16(p, stage + (i * kDownWaves + wave) * 1024);
    }
    if (has_w) {
#pragma unroll
      for (int i = 0; i < L::WL; ++i) {
        p = wp[i] + (size_t)at * wstep;
        if (part && at * kStep + wk[i] >= K) p = adapter_zero;
        to_lds16(p, stage + L::X + (i * kDownWaves + wave) * 1024);
      }
    }
  };
  f32x4_t acc[RB];
#pragma unroll
  for (int b = 0; b < RB; ++b) acc[b] = f32x4_t{0.f, 0.f, 0.f, 0.f};
  for (int s = 0; s < S - 1 && s < n; ++s) load(s);
  for (int s = 0; s < n; ++s) {
    // step s is there; the S - 2 behind it may still be under way
    if (s + S - 1 > n) lds_sync<0>();
    else if (has_w) lds_sync<(S - 2) * (L::XL + L::WL)>();
    else lds_sync<(S - 2) * L::XL>();
    if (s + S - 1 < n) load(s + S - 1);
    const char* stage = lds + s % S * L::STAGE;
#pragma unroll
    for (int k = 0; k < kStep / 64; ++k) {       // 32 elements of the wave's half
      const int h = wh * (kStep / 64) + k, chunk = ((h * 4 + q) ^ l16) << 4;
      const bf16x8_t xv = as_bf16x8(*reinterpret_cast<const uint4*>(stage + (wi * 16 + l16) * kStepBytes + chunk));
#pragma unroll
      for (int b = 0; b < RB; ++b) {
        bf16x8_t w;
        if constexpr (ALONG) {
          w = as_bf16x8(*reinterpret_cast<const uint4*>(stage + L::X + (b * 16 + l16) * kStepBytes + chunk));
        } else {
          typedef short s16x4 __attribute__((ext_vector_type(4)));
          typedef short s16x8 __attribute__((ext_vector_type(8)));
          const char* p = stage + L::X + ((h * 32 + 8 * q + (l16 >> 2)) * lw + min(b * 16 + 4 * (l16 & 3), lw - 4)) * 2;
          const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) s16x4*)p);
          const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) s16x4*)(p + 4 * lw * 2));
          w = __builtin_bit_cast(bf16x8_t, s16x8{lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]});
        }
        acc[b] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(w, xv, acc[b], 0, 0, 0);
      }
    }
  }
  lds_sync<0>();
  // the two halves' sums: lane l has ranks 16 b + 4 q .. of row 16 i + l16
  f32x4_t* s_half = reinterpret_cast<f32x4_t*>(lds) + wi * RB * 64 + lane;
  if (wh) {
#pragma unroll
    for (int b = 0; b < RB; ++b) s_half[b * 64] = acc[b];
  }
  __syncthreads();
  if (wh) return;
  const int row = wi * 16 + l16;
  const bool live = tile.y + row < tile.z && row_at(d, min(tile.y + row, tile.z - 1)) >= 0;
  if (ks > 1) {                                  // a slice of the sum
    float* out = (ALONG ? d.h : d.dh) + (((size_t)z * d.p.tiles + t) * RT + row) * d.r;
#pragma unroll
    for (int b = 0; b < RB; ++b) {
      const int j = j0 + b * 16 + q * 4;
      f32x4_t v = acc[b] + s_half[b * 64];
      if (!live) v = f32x4_t{0.f, 0.f, 0.f, 0.f};
      if (j < d.r) *reinterpret_cast<f32x4_t*>(out + j) = v;
    }
    return;
  }
  // the whole of it: what k_adapter_sum makes of slices
  const float scale = d.scales ? d.scales[tile.x] : 1.f;
  uint16_t* rows = (ALONG ? d.hp : d.dhp);
  uint16_t* turned = ALONG ? d.ht : d.dht;
  const size_t at = (size_t)t * 3 * RT * d.r;
#pragma unroll
  for (int b = 0; b < RB; ++b) {
    const int j = j0 + b * 16 + q * 4;
    const f32x4_t v = acc[b] + s_half[b * 64];
    float f[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) f[k] = live ? v[k] * scale : 0.f;
    if (j >= d.r) continue;
#pragma unroll
    for (int n = 0; n < 3; ++n) {
      const uint32_t p[2] = {pack_bf16(f[0], f[1]), pack_bf16(f[2], f[3])};
      if (rows && (n < 2 || d.out_f32)) *reinterpret_cast<uint2*>(rows + at + ((size_t)n * RT + row) * d.r + j) = uint2{p[0], p[1]};
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const uint32_t one = k & 1 ? p[k >> 1] >> 16 : p[k >> 1] & 0xFFFFu;
        if (turned) turned[at + ((size_t)n * d.r + j + k) * RT + row] = (uint16_t)one;
        const float g = bf2f(one);
        f[k] = fabsf(g) == __builtin_huge_valf() ? 0.f : f[k] - g;
      }
    }
  }
}

template <int RB>
__global__ __launch_bounds__(kDownWaves * 64) void k_adapter_down64(const AdapterDesc d, int with_h, int chunks) {
  __shared__ __attribute__((aligned(16))) char lds[Down64<RB>::BYTES];
  const int z = blockIdx.y;
  const int4 tile = adapter_tile<64>(d, blockIdx.x, gridDim.x);
  const int t = tile.w;
  if (t >= d.p.tiles) return;
  const bool back = (int)blockIdx.z >= chunks || !with_h;
  const int j0 = (blockIdx.z % chunks) * kDown64Ranks;
  if (z == 0 && blockIdx.z == 0 && threadIdx.x == 0) d.tab[t] = tile;
  if (tile.x < 0 || z >= (back ? d.p.kd : d.p.ks)) return;
  if (!back) down64_tile<RB, true>(d, tile, t, z, j0, lds);
  else down64_tile<RB, false>(d, tile, t, z, j0, lds);
}

// Behind it (4.7 us for 4095 rows, rank 16, most of it latency), for each of h and dh: the slices' sums times
// the adapter's scale, as two bf16 numbers (three for fp32 outputs) in rows of ranks for the second product, and as three
// with the tile's rows along for the adapters' gradients. Four rows of four ranks a thread.
template <int KS>
__device__ __forceinline__ void sum_rows(const AdapterDesc& d, const float* h, size_t slab, float (&f)[4][4], float scale) {
  f32x4_t v[4][KS];
#pragma unroll
  for (int z = 0; z < KS; ++z)
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i][z] = *reinterpret_cast<const f32x4_t*>(h + z * slab + (size_t)i * d.r);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
#pragma unroll
    for (int z = 1; z < KS; ++z) v[i][0] += v[i][z];
#pragma unroll
    for (int e = 0; e < 4; ++e) f[i][e] = v[i][0][e] * scale;
  }
}
template <int RT>
__global__ __launch_bounds__(64) void k_adapter_sum(const AdapterDesc d, int with_h) {
  const int t = blockIdx.x, which = !with_h || blockIdx.z, r4 = d.r >> 2;
  const int e = blockIdx.y * 64 + threadIdx.x, r0 = e / r4 * 4, j = (e - e / r4 * r4) * 4;
  const int g = d.tab[t].x;
  if (g < 0 || r0 >= RT || (which ? d.p.kd : d.p.ks) == 1) return;
  const size_t at = (size_t)t * RT * d.r;
  const float* h = (which ? d.dh : d.h) + at + (size_t)r0 * d.r + j;
  uint16_t* rows = which ? d.dhp : d.hp;
  uint16_t* turned = which ? d.dht : d.ht;
  const size_t slab = (size_t)d.p.tiles * RT * d.r;
  const float scale = d.scales ? d.scales[g] : 1.f;
  float f[4][4];
  switch (which ? d.p.kd : d.p.ks) {
    case 2: sum_rows<2>(d, h, slab, f, scale); break;
    case 4: sum_rows<4>(d, h, slab, f, scale); break;
    default: sum_rows<8>(d, h, slab, f, scale);
  }
#pragma unroll
  for (int n = 0; n < 3; ++n) {
    uint32_t p[4][2];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      p[i][0] = pack_bf16(f[i][0], f[i][1]);
      p[i][1] = pack_bf16(f[i][2], f[i][3]);
      if (rows && (n < 2 || d.out_f32)) *reinterpret_cast<uint2*>(rows + 3 * at + ((size_t)n * RT + r0 + i) * d.r + j) = uint2{p[i][0], p[i][1]};
    }
    if (turned) {
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const uint32_t sel = k & 1 ? 0x07060302u : 0x05040100u;
        *reinterpret_cast<uint2*>(turned + 3 * at + ((size_t)n * d.r + j + k) * RT + r0) =
            uint2{__builtin_amdgcn_perm(p[1][k >> 1], p[0][k >> 1], sel), __builtin_amdgcn_perm(p[3][k >> 1], p[2][k >> 1], sel)};
      }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float v = __uint_as_float(k & 1 ? p[i][k >> 1] & 0xFFFF0000u : p[i][k >> 1] << 16);
        f[i][k] = fabsf(v) == __builtin_huge_valf() ? 0.f : f[i][k] - v;
      }
  }
}

// First products: h (of x, if d.h) and dh (of dy, if d.dh), what is made of them, and the table of tiles.
static hipError_t launch_adapter_down(const AdapterDesc& d, hipStream_t s) {
  const int with_h = d.h != nullptr, with_dh = d.dh != nullptr, ranks = d.p.rt == 16 ? kDownRanks : kDown64Ranks;
  const int chunks = (d.r + ranks - 1) / ranks, ks = d.p.ks > d.p.kd ? d.p.ks : d.p.kd;
  const dim3 grid((d.p.tiles + 7) / 8 * 8, ks, (with_h + with_dh) * chunks), block(kDownWaves * 64);
  if (d.p.rt == 16) {
    if (d.r <= 16) ffn_launch((k_adapter_down<16, 1>), grid, block, 0, s, d, with_h, chunks);
    else if (d.r <= 32) ffn_launch((k_adapter_down<16, 2>), grid, block, 0, s, d, with_h, chunks);
    else ffn_launch((k_adapter_down<16, 4>), grid, block, 0, s, d, with_h, chunks);
  } else {
    if (d.r <= 16) ffn_launch((k_adapter_down64<1>), grid, block, 0, s, d, with_h, chunks);
    else if (d.r <= 32) ffn_launch((k_adapter_down64<2>), grid, block, 0, s, d, with_h, chunks);
    else if (d.r <= 64) ffn_launch((k_adapter_down64<4>), grid, block, 0, s, d, with_h, chunks);
    else ffn_launch((k_adapter_down64<8>), grid, block, 0, s, d, with_h, chunks);
  }
  const hipError_t e = hipGetLastError();
  // forward with tiles of 16 rows, the second product adds the slices as it reads them: a launch less
  if (e != hipSuccess || (d.p.rt == 16 && !with_dh && !d.ht)) return e;
  // and otherwise a product that is not sliced is finished by its own kernel
  if ((!with_h || d.p.ks == 1) && (!with_dh || d.p.kd == 1)) return e;
  if (d.p.rt == 16) ffn_launch(k_adapter_sum<16>, dim3(d.p.tiles, (d.r + 63) / 64, with_h + with_dh), dim3(64), 0, s, d, with_h);
  else ffn_launch(k_adapter_sum<64>, dim3(d.p.tiles, (d.r * 4 + 63) / 64, with_h + with_dh), dim3(64), 0, s, d, with_h);
  return hipGetLastError();
}

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

// out = base + s h W^T for a tile: a wave has 128 columns, accumulator e of lane l column 8 (l % 16) + e of row 4 (l / 16)
// + v in its value v, so that a lane reads and writes eight neighbours and 16 lanes 256 bytes of a row. (With the lanes'
// rows and columns exchanged, 16 bytes a row from each of 16 lanes, 8192 x 4096 x 14336, rank 64, took 160 us; so 100.7:
// 235 MB of the base, as many of the output and 55 of s h and the weights, 5.2 TB/s. Stores past the caches: no gain.)
// ALONG: W = B, rows of r elements a column; otherwise W = A^T, rows of the output's columns. F: groups of 32 ranks (0: up
// to 16, hi and lo in one group). s h stands in LDS in bf16 numbers, which the workgroup's WAVES waves share, in rows of an
// odd number of 16-byte chunks, so that the lanes' rows lie in different banks.
__device__ __forceinline__ int h_pitch(int r) { return ((r >> 3) | 1) * 16; }
template <typename T, int RT, int F, bool ALONG, int WAVES = 4>
struct Up {
  static constexpr int NF = F == 0 ? 1 : F;
  static constexpr int PARTS = sizeof(T) == 4 ? 3 : 2;
  static constexpr int PIECES = F == 0 ? 2 : 4;  // 16-byte chunks of a column's ranks in a group
  static constexpr bool STAY = NF <= 2;          // weights of up to 64 ranks stay in registers for all of the tile's rows
  static constexpr int MB = RT == 64 && !STAY ? 2 : 1;           // 16 rows each, for a group's weights
  static constexpr int AHEAD = RT == 16 && NF > 1 ? (NF < 3 ? NF : 3) : 1;     // groups whose loads are under way
  static constexpr int W = ALONG ? 128 * PIECES * 16 + 256 : 0;  // LDS of a wave's weights
  static constexpr int H = PARTS * RT * ((F == 0 ? 2 : NF * 4) + 1) * 16;      // LDS of s h
  static constexpr int BYTES = WAVES * W + H;
};
// The columns of the workgroup's waves, 128 each, of a tile. fill() brings s h to LDS, while the first loads are under way.
template <typename T, int RT, int F, bool ALONG, int WAVES, typename Fill>
__device__ __forceinline__ void up_tile(const AdapterDesc& d, int block, const int4 tile, char* s_mem, Fill fill) {
  using U = Up<T, RT, F, ALONG, WAVES>;
  constexpr int NF = U::NF, PARTS = U::PARTS, PIECES = U::PIECES, MB = U::MB, AHEAD = U::AHEAD;
  const int lane = lane_id(), wave = threadIdx.x >> 6, l16 = lane & 15, q = lane >> 4;
  const int cols = ALONG ? d.n : d.k;
  const int c0 = (block * WAVES + wave) * 128;
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
  const uint16_t* w = ALONG ? d.b + (size_t)tile.x * d.n * d.r : d.a + (size_t)tile.x * d.r * d.k;
  const int jq = F == 0 ? (q & 1) * 8 : q * 8;   // this lane's first rank in a group
  const int wc = c0 + 8 * l16;                   // this lane's eight columns
  // lane l has the row of place l of the tile
  const int mine = row_at(d, min(tile.y + min(lane, RT - 1), tile.z - 1)), rows = tile.z - tile.y;

  // ---------------------------------------------------------------- weights
  // B's come through the wave's own part of LDS: neighbouring lanes load neighbouring chunks of a column's ranks, and 16
  // bytes of padding every eight columns keep the operands' reads, eight columns apart, out of each other's banks.
  uint4 wv[U::STAY ? NF : 1][8], raw[AHEAD][ALONG ? 2 * PIECES : 8];
  char* lds = s_mem + U::H + wave * U::W;
  auto chunk = [&](int n, int& col, int& piece) {
    const int c = n * 64 + lane;
    col = c / PIECES;
    piece = c % PIECES;
  };
  auto ask = [&](int g) {
    uint4(&to)[ALONG ? 2 * PIECES : 8] = raw[g % AHEAD];
    int first = g * 32;
    if constexpr (NF > 2) asm volatile("" : "+v"(first));        // addresses are made here, not all of them up front and spilt
    if constexpr (ALONG) {
#pragma unroll
      for (int n = 0; n < 2 * PIECES; ++n) {
        int col, piece;
        chunk(n, col, piece);
        to[n] = ldg16(w + (size_t)min(c0 + col, cols - 1) * d.r + min(first + piece * 8, d.r - 8));
      }
    } else {
      const int jc = min(first + jq, d.r - 8);
#pragma unroll
      for (int e = 0; e < 8; ++e) to[e] = ldg16(w + (size_t)(jc + e) * cols + min(wc, cols - 8));
    }
  };
  auto weights = [&](int g) {
    uint4(&o)[8] = wv[U::STAY ? g : 0];
    uint4(&got)[ALONG ? 2 * PIECES : 8] = raw[g % AHEAD];
    if constexpr (ALONG) {
#pragma unroll
      for (int n = 0; n < 2 * PIECES; ++n) {
        int col, piece;
        chunk(n, col, piece);
        *reinterpret_cast<uint4*>(lds + (col * PIECES + piece + (col >> 3)) * 16) = got[n];
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) o[e] = *reinterpret_cast<const uint4*>(lds + ((8 * l16 + e) * PIECES + (jq >> 3) + l16) * 16);
#pragma unroll
      for (int e = 0; e < 8; ++e) o[e] = keep_if(g * 32 + jq < d.r, o[e]);
    } else {
      uint4 in[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) in[e] = keep_if(g * 32 + jq < d.r, got[e]);
      transpose8(in, o);
    }
  };
  // ---------------------------------------------------------------- s h
  auto part_of = [&](int i0, int g, int n) {     // F = 0: hi for q < 2 and lo for the others in part 0; then the third
    const int which = F == 0 && n == 0 ? q >> 1 : n;
    const uint4 v = *reinterpret_cast<const uint4*>(s_mem + (which * RT + min(i0 + l16, RT - 1)) * h_pitch(d.r) + min(g * 32 + jq, d.r - 8) * 2);
    return as_bf16x8(keep_if(g * 32 + jq < d.r && (F != 0 || n == 0 || q < 2), v));
  };
  // ---------------------------------------------------------------- base
  // without one, every row is the same eight zeros
  const void* from = d.base ? d.base : adapter_zero;
  const size_t pitch = d.base ? cols : 0;
  const int at = d.base ? min(wc, cols - 8) : 0;
  int row[MB][4];
  Row8<T> base[MB][4];
  auto fetch = [&](int i0) {
#pragma unroll
    for (int i = 0; i < MB; ++i)
#pragma unroll
      for (int v = 0; v < 4; ++v) {
        row[i][v] = __shfl(mine, min(i0 + i * 16 + 4 * q + v, rows - 1), 64);
        base[i][v].load(from, (size_t)max(row[i][v], 0) * pitch + at);
      }
  };

#pragma unroll
  for (int g = 0; g < AHEAD; ++g) ask(g);
  fetch(0);
  __builtin_amdgcn_sched_barrier(0);
  fill();
  if (c0 >= cols) return;
  if constexpr (U::STAY) {
    weights(0);
    if constexpr (NF > 1) {
      if constexpr (AHEAD == 1) ask(1);
      weights(1);
    }
  }
#pragma unroll 1
  for (int i0 = 0; i0 < rows; i0 += 16 * MB) {
    f32x4_t acc[MB][8];                          // the sums start from the base
    int to[MB][4];
#pragma unroll
    for (int i = 0; i < MB; ++i)
#pragma unroll
      for (int v = 0; v < 4; ++v) {
        float f[8];
        base[i][v].get(f);
#pragma unroll
        for (int e = 0; e < 8; ++e) acc[i][e][v] = f[e];
        to[i][v] = i0 + i * 16 + 4 * q + v < rows ? row[i][v] : -1;
      }
    // the next rows' (past the last: the last row's again), ahead of this one's stores, which a wait for loads behind
    // them would be a wait for
    if (RT > 16) fetch(i0 + 16 * MB);
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int g = 0; g < NF; ++g) {
      if constexpr (!U::STAY) {
        weights(g);
        if (g + AHEAD < NF || RT > 16) ask((g + AHEAD) % NF);
      }
      const uint4(&o)[8] = wv[U::STAY ? g : 0];
#pragma unroll
      for (int i = 0; i < MB; ++i)
#pragma unroll
        for (int n = 0; n < PARTS; ++n) {
          if (F == 0 && n == 1) continue;
          const bf16x8_t h = part_of(i0 + i * 16, g, n);
#pragma unroll
          for (int e = 0; e < 8; ++e) acc[i][e] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(h, as_bf16x8(o[e]), acc[i][e], 0, 0, 0);
        }
    }
    if (wc >= cols) continue;
#pragma unroll
    for (int i = 0; i < MB; ++i)
#pragma unroll
      for (int v = 0; v < 4; ++v) {
        if (to[i][v] < 0) continue;
        float f[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) f[e] = acc[i][e][v];
        Row8<T>::store(d.out, (size_t)to[i][v] * cols + wc, f);
      }
  }
}

// s h from memory, [PARTS][RT][r] in bf16 numbers.
template <int ROWS, int THREADS>
__device__ __forceinline__ void fill_made(const uint16_t* from, int r, char* s_mem) {
  const int r8 = r >> 3, pitch = h_pitch(r);
  for (int c = threadIdx.x; c < ROWS * r8; c += THREADS) {
    const int line = c / r8;
    *reinterpret_cast<uint4*>(s_mem + line * pitch + (c - line * r8) * 16) = ldg16(from + (size_t)c * 8);
  }
  __syncthreads();
}
// s h of a tile of 16 rows from the slices' sums.
template <int PARTS>
__device__ __forceinline__ void fill_slices(const AdapterDesc& d, int t, int g, char* s_mem) {
  const int r4 = d.r >> 2, pitch = h_pitch(d.r);
  const float scale = d.scales ? d.scales[g] : 1.f;
  const size_t slab = (size_t)d.p.tiles * 16 * d.r;
  for (int e = threadIdx.x; e < 16 * r4; e += 256) {
    const int row = e / r4, j = (e - row * r4) * 4;
    const float* p = d.h + ((size_t)t * 16 + row) * d.r + j;
    f32x4_t v = *reinterpret_cast<const f32x4_t*>(p);
#pragma unroll 4
    for (int z = 1; z < d.p.ks; ++z) v += *reinterpret_cast<const f32x4_t*>(p + z * slab);
    float f[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) f[i] = v[i] * scale;
#pragma unroll
    for (int n = 0; n < PARTS; ++n) {
      const uint32_t part[2] = {pack_bf16(f[0], f[1]), pack_bf16(f[2], f[3])};
      *reinterpret_cast<uint2*>(s_mem + (n * 16 + row) * pitch + j * 2) = uint2{part[0], part[1]};
#pragma unroll
      for (int i = 0; i < 4; ++i) f[i] = rest_of(f[i], i & 1 ? part[i >> 1] >> 16 : part[i >> 1] & 0xFFFFu);
    }
  }
  __syncthreads();
}

template <typename T, int RT, int F>
__global__ __launch_bounds__(256, F == 0 ? (RT == 16 ? 4 : 3) : F == 1 ? 3 : 2) void k_adapter_up(const AdapterDesc d) {
  using U = Up<T, RT, F, true>;
  __shared__ __attribute__((aligned(16))) char s_mem[U::BYTES];
  const int t = blockIdx.y + blockIdx.z * gridDim.y;
  if (t >= d.p.tiles) return;
  const int4 tile = d.tab[t];
  up_tile<T, RT, F, true, 4>(d, blockIdx.x, tile, s_mem, [&] {
    if constexpr (RT == 16) fill_slices<U::PARTS>(d, t, tile.x, s_mem);
    else fill_made<U::PARTS * RT, 256>(d.hp + (size_t)t * 3 * RT * d.r, d.r, s_mem);
  });
}

// Both products of a tile of 16 rows in one launch, for few rows and ranks up to 32, where a launch costs as much as the
// work: each of d.p.few workgroups makes all of s h for its tile, and takes every d.p.few-th block of 1024 columns, the
// first one's weights and base on their way meanwhile. 4096 x 14336, rank 16, one row: 8.7 us a call instead of 12.7 in two
// launches (in a captured graph 9.1 and 8.2); 16 rows of 16 adapters 9.2 and 12.3 (9.7 either way).
template <typename T, int F>
__global__ __launch_bounds__(kDownWaves * 64, 2) void k_adapter_few(const AdapterDesc d) {
  using U = Up<T, 16, F, true, kDownWaves>;
  constexpr int RB = F == 0 ? 1 : 2, PART = DownLds<16, RB>::PART;
  static_assert(F <= 1, "ranks of one pass");
  __shared__ __attribute__((aligned(16))) char s_mem[U::H + (kDownWaves * U::W > PART ? kDownWaves * U::W : PART)];
  const int4 tile = adapter_tile<16>(d, blockIdx.x, gridDim.x);
  if (tile.x == -2) return;
  auto up = [&](int block, auto fill) { up_tile<T, 16, F, true, kDownWaves>(d, block, tile, s_mem, fill); };
  auto down = [&] {
    const float scale = d.scales ? d.scales[tile.x] : 1.f;
    const int pitch = h_pitch(d.r);
    down_tile<16, RB, true>(d, tile, 0, 0, s_mem + U::H, [&](int row, int j, float v) {
      v *= scale;
#pragma unroll
      for (int n = 0; n < U::PARTS; ++n) {
        const uint32_t part = pack_bf16(v, 0.f) & 0xFFFFu;
        *reinterpret_cast<uint16_t*>(s_mem + (n * 16 + row) * pitch + j * 2) = (uint16_t)part;
        v = rest_of(v, part);
      }
    });
    __syncthreads();
  };
  const int n = (d.n + kDownWaves * 128 - 1) / (kDownWaves * 128), first = blockIdx.y, step = gridDim.y;
  up(first, down);
  for (int block = first + step; block < n; block += step) up(block, [] {});
}

template <typename T>
static hipError_t few(const AdapterDesc& d, hipStream_t s) {
  const dim3 grid((d.p.tiles + 7) / 8 * 8, d.p.few), block(kDownWaves * 64);
  if (d.r <= 16) ffn_launch((k_adapter_few<T, 0>), grid, block, 0, s, d);
  else ffn_launch((k_adapter_few<T, 1>), grid, block, 0, s, d);
  return hipGetLastError();
}
template <typename T, int RT>
static hipError_t up(const AdapterDesc& d, hipStream_t s) {
  // a grid's second dimension holds 65535 workgroups: tiles go on in the third
  const int ty = d.p.tiles < 32768 ? d.p.tiles : 32768;
  const dim3 grid((d.n + 511) / 512, ty, (d.p.tiles + ty - 1) / ty), block(256);
  if (d.r <= 16) ffn_launch((k_adapter_up<T, RT, 0>), grid, block, 0, s, d);
  else if (d.r <= 32) ffn_launch((k_adapter_up<T, RT, 1>), grid, block, 0, s, d);
  else if (d.r <= 64) ffn_launch((k_adapter_up<T, RT, 2>), grid, block, 0, s, d);
  else if (d.r <= 128) ffn_launch((k_adapter_up<T, RT, 4>), grid, block, 0, s, d);
  else ffn_launch((k_adapter_up<T, RT, 8>), grid, block, 0, s, d);
  return hipGetLastError();
}
hipError_t launch_adapter_forward(const AdapterDesc& d, hipStream_t s) {
  if (d.p.few) return d.out_f32 ? few<float>(d, s) : few<uint16_t>(d, s);
  const hipError_t e = launch_adapter_down(d, s);
  if (e != hipSuccess) return e;
  if (d.out_f32) return d.p.rt == 16 ? up<float, 16>(d, s) : up<float, 64>(d, s);
  return d.p.rt == 16 ? up<uint16_t, 16>(d, s) : up<uint16_t, 64>(d, s);
}

// ---------------------------------------------------------------- gradients of the adapters
// dA[j][c] = sum over the adapter's rows t of s dh[t][j] x[t][c], and dB[c][j] = sum of s h[t][j] dy[t][c]. A wave has 128
// columns c of one adapter and up to 16 RB ranks, and takes 32 rows at a time: whose 8 x 8 pieces are turned in registers,
// the next ones under way; s h enters as three bf16 numbers. A workgroup's four waves are `split` waves for each of its 4 /
// split column blocks, which take the steps of 32 rows in turn and whose sums are added in order (waves of different
// columns share the reads of s h, 1.5 times as many bytes as x with 64 ranks). Where that leaves the chip empty, the rows
// are cut into slices besides, whose sums k_adapter_dw_sum adds. One adapter, 4096 rows, 1024 x 1024, rank 16: with 1, 2, 4
// waves a block 133, 76, 47 us the whole pass; with 4 and 1, 2, 4, 8, 16 slices 46.8, 34.0, 27.5, 25.5, 26.8.
constexpr int kDwWaves = 4;
template <int RT, int RB, bool OF_A>
__device__ __forceinline__ void dw_tile(const AdapterDesc& d, int g, int block, int j0, int slice, float* s_part) {
  const int lane = lane_id(), wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), l16 = lane & 15, q = lane >> 4;
  const int split = d.p.split, colw = kDwWaves / split, cw = wave % colw, rw = wave / colw;
  const int cols = OF_A ? d.k : d.n, c0 = (block * colw + cw) * 128;
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
  const int lo = wave_read(start, owner), rows = wave_read(stop, owner) - lo;
  const bool whole = d.p.slices == 1;
  if (rows == 0 && whole && d.accumulate) return;
  const uint16_t* h = (OF_A ? d.dht : d.ht) + (size_t)before * 3 * d.r * RT;
  f32x4_t acc[8][RB];
#pragma unroll
  for (int i = 0; i < 8; ++i)
#pragma unroll
    for (int b = 0; b < RB; ++b) acc[i][b] = f32x4_t{0.f, 0.f, 0.f, 0.f};
  const int cb = min(c0 + 8 * l16, cols - 8);
  int at[8];
  uint4 in[8];
  // the rows of step r0 (clamped: what lies behind the last is cleared before it is used)
  auto load = [&](int r0) {
#pragma unroll
    for (int e = 0; e < 8; ++e) at[e] = row_at(d, lo + min(r0 + q * 8 + e, rows - 1));
#pragma unroll
    for (int e = 0; e < 8; ++e) in[e] = ldg16(u + (size_t)max(at[e], 0) * cols + cb);
  };
  const int steps = (rows + 31) / 32, last = (int)((long long)steps * (slice + 1) / d.p.slices) * 32;
  int r0 = ((int)((long long)steps * slice / d.p.slices) + rw) * 32;
  if (r0 < last && c0 < cols) {
    load(r0);
    for (; r0 < last; r0 += split * 32) {
      // places and rows past the adapter's: zeros
      uint4 uv[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) in[e] = keep_if(at[e] >= 0 && r0 + q * 8 + e < rows, in[e]);
      transpose8(in, uv);
      const int first = r0 + q * 8, tile = min(first, rows - 1) / RT;
      const uint16_t* hp = h + ((size_t)tile * 3 * d.r) * RT + (first & (RT - 1));
      const bool has = first < rows;             // a tile of 16 rows may be the last
      uint4 hv[RB > 1 ? 2 : 1][3];               // of two blocks of 16 ranks at a time
      auto ranks = [&](int b) {
#pragma unroll
        for (int part = 0; part < 3; ++part) hv[b & 1][part] = ldg16(hp + ((size_t)part * d.r + min(j0 + b * 16 + l16, d.r - 1)) * RT);
      };
      ranks(0);
      if constexpr (RB > 1) ranks(1);
      if constexpr (RB <= 2) load(min(r0 + split * 32, rows - 1));
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int b = 0; b < RB; ++b) {
#pragma unroll
        for (int part = 0; part < 3; ++part) {
          const bf16x8_t hb = as_bf16x8(keep_if(has, hv[b & 1][part]));
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            if constexpr (OF_A) acc[i][b] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(as_bf16x8(uv[i]), hb, acc[i][b], 0, 0, 0);
            else acc[i][b] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(hb, as_bf16x8(uv[i]), acc[i][b], 0, 0, 0);
          }
        }
        if (b + 2 < RB) {
          __builtin_amdgcn_sched_barrier(0);
          ranks(b + 2);
          if (b + 3 == RB) load(min(r0 + split * 32, rows - 1));
          __builtin_amdgcn_sched_barrier(0);
        }
      }
    }
  }
  // the waves' sums, 16 ranks of the 128 columns at a time: part(wave, accumulator, lane) in fours
  float* to = OF_A ? d.da : d.db;
  if (!whole) to = d.part + (size_t)slice * d.p.part + (OF_A || !d.da ? 0 : (size_t)d.groups * d.r * d.k);
  const bool add = whole && d.accumulate;
  auto part = [&](int w, int i, int l) { return s_part + (((w * colw + cw) * 8 + i) * 64 + l) * 4; };
#pragma unroll
  for (int b = 0; b < RB; ++b) {
    if (b) __syncthreads();
#pragma unroll
    for (int i = 0; i < 8; ++i) *reinterpret_cast<f32x4_t*>(part(rw, i, lane)) = acc[i][b];
    __syncthreads();
    if constexpr (OF_A) {
      // eight neighbouring columns of a rank a thread: those of blk = 4 q + v are value v of lane q * 16 + j's accumulators
      for (int n = rw * 64 + lane; n < 256; n += split * 64) {
        const int blk = n & 15, j = j0 + b * 16 + (n >> 4), l = (blk >> 2) * 16 + (n >> 4), c = c0 + 8 * blk;
        float f[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] = part(0, i, l)[blk & 3];
        for (int w = 1; w < split; ++w)
#pragma unroll
          for (int i = 0; i < 8; ++i) f[i] += part(w, i, l)[blk & 3];
        if (j >= d.r || c >= cols) continue;
        float* out = to + ((size_t)g * d.r + j) * cols + c;
        if (add) {
#pragma unroll
          for (int i = 0; i < 8; ++i) f[i] += out[i];
        }
        Row8<float>::store(out, 0, f);
      }
    } else {
      // four neighbouring ranks of a column a thread: lane q * 16 + p of accumulator i has column 8 p + i
      for (int n = rw * 64 + lane; n < 512; n += split * 64) {
        const int lq = n & 3, col = n >> 2, p = col >> 3;
        const int j = j0 + b * 16 + 4 * lq, c = c0 + col;
        f32x4_t f = *reinterpret_cast<const f32x4_t*>(part(0, col & 7, lq * 16 + p));
        for (int w = 1; w < split; ++w) f += *reinterpret_cast<const f32x4_t*>(part(w, col & 7, lq * 16 + p));
        if (j >= d.r || c >= cols) continue;
        f32x4_t* out = reinterpret_cast<f32x4_t*>(to + ((size_t)g * cols + c) * d.r + j);
        if (add) f += *out;
        *out = f;
      }
    }
  }
}

// Blocks of 16 ranks that a workgroup of the gradients takes.
constexpr int back_ranks(int r) { return r <= 16 ? 1 : r <= 32 ? 2 : 4; }
// The second half of the backward pass, whose two parts read nothing of each other: workgroups of the adapters' gradients
// (the longer ones), then those of dx. One launch lets the one's memory traffic fill the other's gaps: 4095 x 2048 x 8192,
// rank 16, 26.4 us for 132 MB from memory (5.0 TB/s); the whole pass 53 us instead of 59. Both read their operand for the
// second time, of which dy, for dB, is the larger: that needs h, not dh, so it could be summed where dy is read first.
template <int RT, int F>
__global__ __launch_bounds__(kDwWaves * 64, F == 0 ? 3 : 2) void k_adapter_back(const AdapterDesc d, const BackGrid grid) {
  constexpr int RB = back_ranks(F == 0 ? 16 : 32 * F), PART = kDwWaves * 8 * 64 * 16;
  using U = Up<uint16_t, RT, F, false>;
  static_assert(kDwWaves * 64 == 256, "one size of workgroup");
  __shared__ __attribute__((aligned(16))) char s_mem[PART > U::BYTES ? PART : U::BYTES];
  const long long n = (long long)blockIdx.y * gridDim.x + blockIdx.x;
  const int what = adapter_back_part(grid, n);
  if (what == BACK_NOTHING) return;
  if (what == BACK_GRADIENTS) {
    const int block = (int)(n % (grid.a + grid.b)), rest = (int)(n / (grid.a + grid.b));
    const int g = rest % grid.groups, z = rest / grid.groups;
    const int slice = z % d.p.slices, j0 = z / d.p.slices * (16 * RB);
    float* s_part = reinterpret_cast<float*>(s_mem);
    if (block < grid.a) dw_tile<RT, RB, true>(d, g, block, j0, slice, s_part);
    else dw_tile<RT, RB, false>(d, g, block - grid.a, j0, slice, s_part);
    return;
  }
  const long long at = n - grid.dw;
  const int t = (int)(at / grid.x);
  up_tile<uint16_t, RT, F, false, 4>(d, (int)(at - (long long)t * grid.x), d.tab[t], s_mem, [&] {
    fill_made<U::PARTS * RT, 256>(d.dhp + (size_t)t * 3 * RT * d.r, d.r, s_mem);
  });
}
// The slices' sums, to da (na values) and db (nb behind them), four values a thread.
__global__ __launch_bounds__(256) void k_adapter_dw_sum(const AdapterDesc d, size_t na, size_t nb) {
  for (size_t i = ((size_t)blockIdx.x * 256 + threadIdx.x) * 4; i < na + nb; i += (size_t)gridDim.x * 1024) {
    f32x4_t v = *reinterpret_cast<const f32x4_t*>(d.part + i);
    for (int z = 1; z < d.p.slices; ++z) v += *reinterpret_cast<const f32x4_t*>(d.part + z * d.p.part + i);
    f32x4_t* out = reinterpret_cast<f32x4_t*>(i < na ? d.da + i : d.db + (i - na));
    if (d.accumulate) v += *out;
    *out = v;
  }
}

BackGrid adapter_back_grid(const AdapterPlan& p, int n, int k, int r, int groups, bool dx, bool da, bool db) {
  const int w = 128 * kDwWaves / p.split, ranks = 16 * back_ranks(r);          // columns and ranks of a workgroup of da and db
  BackGrid b;
  b.a = da ? (k + w - 1) / w : 0;
  b.b = db ? (n + w - 1) / w : 0;
  b.groups = groups;
  b.z = (r + ranks - 1) / ranks * p.slices;
  b.x = dx ? (k + 511) / 512 : 0;
  b.dw = (long long)(b.a + b.b) * groups * b.z;
  b.all = b.dw + (long long)b.x * p.tiles;
  // a grid holds fewer than 2^32 threads a dimension
  b.gy = (unsigned)((b.all + (1 << 23) - 1) >> 23);
  b.gx = (unsigned)((b.all + b.gy - 1) / b.gy);
  return b;
}
template <int RT, int F>
static void back_launch(const AdapterDesc& d, hipStream_t s) {
  const BackGrid b = adapter_back_grid(d.p, d.n, d.k, d.r, d.groups, d.out, d.da, d.db);
  ffn_launch((k_adapter_back<RT, F>), dim3(b.gx, b.gy), dim3(kDwWaves * 64), 0, s, d, b);
}
template <int RT>
static void back(const AdapterDesc& d, hipStream_t s) {
  if (d.r <= 16) back_launch<RT, 0>(d, s);
  else if (d.r <= 32) back_launch<RT, 1>(d, s);
  else if (d.r <= 64) back_launch<RT, 2>(d, s);
  else if (d.r <= 128) back_launch<RT, 4>(d, s);
  else back_launch<RT, 8>(d, s);
}
hipError_t launch_adapter_backward(const AdapterDesc& d, hipStream_t s) {
  hipError_t e = launch_adapter_down(d, s);
  if (e != hipSuccess) return e;
  if (d.p.rt == 16) back<16>(d, s);
  else back<64>(d, s);
  e = hipGetLastError();
  if (e != hipSuccess || d.p.slices == 1 || (!d.da && !d.db)) return e;
  const size_t na = d.da ? (size_t)d.groups * d.r * d.k : 0, nb = d.db ? (size_t)d.groups * d.r * d.n : 0;
  const size_t blocks = (na + nb + 1023) / 1024;
  ffn_launch(k_adapter_dw_sum, dim3((unsigned)(blocks < 4096 ? blocks : 4096)), dim3(256), 0, s, d, na, nb);
  return hipGetLastError();
}

// ---------------------------------------------------------------- plan
AdapterPlan adapter_plan(int m, int n, int k, int r, int groups, bool backward) {
  AdapterPlan p;
  // Tiles of 64 rows where adapters have rows to share their weights' reads, and where there is work enough for more
  // launches. Forward, rank 64, 4096 x 4096, 8 adapters, tiles of 16 and of 64: 1024 rows 20.7 and 21.1 us, 2048 28.4 and
  // 24.4, 4096 50.8 and 40.4; rank 16: 4096 rows 29.0 and 33.0; 1024 x 1024, rank 64: 4096 rows 19.5 and 20.6, 8192 of 256
  // adapters 44.8 and 36.0; 16 rows an adapter: 29.9 and 36.0. Backward, rank 64, 32 rows an adapter: 256 rows, 4096 x 4096,
  // 30.5 and 25.8; 512, 1024 x 1024, 21.8 and 23.2.
  const bool long_way = backward ? (long long)m * (n + k) >= 1 << 21 : m >= 8192 || (long long)m * r * k >= 1LL << 29;
  p.rt = long_way && m / 32 >= groups ? 64 : 16;
  // every adapter's last tile may be short, and so may the two runs of rows without one
  const long long tiles = (long long)m / p.rt + groups + 2;
  p.tiles = (int)(tiles < m ? tiles : m);
  // Slices of the first products, where there are too few tiles for the chip. Tiles of 16 rows: 48 rows of 32 adapters,
  // 4096 x 14336, rank 16, in 1, 2, 4, 8 slices 15.0, 13.0, 12.5, 12.7 us; 16 of 16, 4096 x 4096, rank 64: 24.8, 18.1,
  // 15.1, 14.7. Tiles of 64, forward, 4096 x 4096, rank 64: 2048 rows 31.9, 26.9, 24.2, 24.8; 4096 rows 47.7, 41.3, 39.0,
  // 43.1; 8192 rows of uneven adapters, 4096 x 14336, whole 127, in two 134. Backward (of dy B), 4095 x 2048 x 8192, rank
  // 16: 58.1, 51.2, 50.0, 50.3.
  const int live = p.rt == 64 ? (m + 63) / 64 : m / 16 + groups < m ? m / 16 + groups : m;
  const int wanted = p.rt == 64 && (backward || live >= 128) ? 128 : 256;
  auto slices = [&](int width) {
    const int steps = width / (p.rt == 64 ? kStep : 64), least = p.rt == 64 ? 4 : kDownWaves;
    int ks = 1;
    // (backward, slices of both products besides that are about as long as each other)
    while (ks < 8 && steps / (ks * 2) >= least && (live * ks < wanted || (backward && p.rt == 64 && steps / ks > 32))) ks *= 2;
    return ks;
  };
  // Backward with tiles of 16 rows, whole where that is short or tiles are many, which saves the sum's launch: 2048 x 2048, 31
  // rows, rank 16, 12.4 us in slices, 12.2 whole (with the host's time 16.1, 13.5), rank 64 19.7, 24.1; 300 rows of 100
  // adapters 27.0, 20.7 and 65.6, 52.8.
  const bool whole = backward && p.rt == 16 && (live >= 96 || (long long)(n > k ? n : k) * (r < 64 ? r : 64) < 65536);
  p.ks = whole ? 1 : slices(k);
  p.kd = backward && !whole ? slices(n) : 1;
  // Both products in one launch, with about a workgroup a CU, if there are columns for as many; where that costs less than
  // a launch: a workgroup reads its tile's operands of the first product (160 KB at most: 16 rows of 16 adapters, rank 32,
  // 4096 x 14336, 14.7 us a call instead of 12.3), and a tile's workgroups all read the same (30 MB at most together). Rank
  // 16, one launch and two, us a call: 24 rows of 24 adapters 11.4 and 12.2, 32 of 32 11.6 and 12.2, 48 of 24 12.1 and 12.2,
  // 48 of 30 (29 MB) 12.3 and 12.3, 48 of 32 (31 MB) 12.3 and 12.2, 64 of 64 (fewer workgroups a tile) 15.0 and 16.1: from
  // there on neither is ahead. Without the host's time, in a captured graph: 12.1 and 11.4, 12.4 and 12.2, 12.8 and 11.5,
  // 13.0 and 12.6, 12.9 and 12.2, 15.8 and 16.9.
  p.few = 0;
  if (!backward && p.rt == 16 && r <= 32) {
    const int blocks = (n + kDownWaves * 128 - 1) / (kDownWaves * 128);
    const int most = live < 256 ? 256 / live : 1, turns = (blocks + most - 1) / most;
    const int few = (blocks + turns - 1) / turns, rows = m / groups < 16 ? (m + groups - 1) / groups : 16;
    const long long read = 2LL * (r + rows) * k;
    if (read <= 160 << 10 && read * live * (few - 1) <= 30000000) {
      p.few = few;
      p.ks = 1;
    }
  }
  // Waves of the adapters' gradients: two for each SIMD, if there are steps of 32 rows for as many. Planned by the average
  // adapter; where one has nearly all rows, its waves walk them one after the other: 8192 rows of 8 adapters, 4096 x 14336,
  // rank 16, the whole pass even 146 us, all but 7 in one 257, and 169 with that one adapter alone; 4096 rows of 100
  // adapters, 1024 x 1024, 28.6, 80.5 and 26.8.
  const int steps = (m / groups + 31) / 32;
  const long long waves = ((long long)(n + 127) / 128 + (k + 127) / 128) * groups * ((r + 63) / 64);
  p.split = 1;
  while (p.split < kDwWaves && waves * p.split < 2048 && p.split * 2 <= steps) p.split *= 2;
  p.slices = 1;
  while (p.split == kDwWaves && p.slices < 16 && waves * p.split * p.slices < 1024 && p.slices * p.split * 4 <= steps) p.slices *= 2;
  p.part = (size_t)groups * r * ((size_t)n + k);
  return p;
}

}  // namespace ffn
