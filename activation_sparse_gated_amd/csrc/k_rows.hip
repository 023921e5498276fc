// Rows to their experts and back on gfx950: the order by expert, the gather,
// the weighted combination and its gradients.
//
// The order is a counting sort that keeps entries of a group in their own
// order, without atomics: waves take runs of consecutive entries, a wave ranks
// its 64 entries of a turn by ballots over the bits of their group, and counts
// of the earlier turns, waves and blocks come in front. Up to 8192 entries are
// one launch's work, of one workgroup or, with fewer than 64 groups, of one for
// every 1024 entries; more are counted by blocks of 4096 first.
//
// The rest is bound by HBM: every row is read and written once, 16 bytes (fp32:
// 32) a lane, a token's rows by the same lanes, so that x (gather) and dout
// (gradient) are read once for all of a token's slots. 4096 rows of 4096 to two
// slots each in 8 bits 14.3 us, 4.8 TB/s; the sum of 8 slots each 56.5 us, 5.35
// TB/s; its gradients, 4095 x 2048, two slots, 14.1 us, 6.0 TB/s, part of it from
// the memory-side cache. The order of 8192 entries of 8 groups takes 6.0 us, of
// 16 entries 2.3: a chain of loads, ballots and LDS accesses.
#include "experts.cuh"
#include "lin_util.cuh"

namespace ffn {

// ---------------------------------------------------------------- order by group
constexpr int kOneBlock = 8192;                  // entries ordered in one launch (256 groups, 8192: 11.1 us, in blocks 11.3; 16384: 19.4, 11.7)
constexpr int kBlock = 4096;                     // entries of a block, where there are more

// The place of each of this lane's entries (entry i * 64 + lane of the wave's run) among those of its group in the run,
// and the run's counts in cnt[0 .. groups] (this wave's own, cleared). key: the group, `groups` for none, -1 past the end.
template <int TURNS, int BITS>
__device__ __forceinline__ void rank_run(const int (&key)[TURNS], int (&rank)[TURNS], uint16_t* cnt) {
#pragma unroll
  for (int i = 0; i < TURNS; ++i) {
    const bool in = key[i] >= 0;
    uint64_t same = ballot64(in);                // lanes of this lane's group
    if (same == 0) break;
#pragma unroll
    for (int b = 0; b < BITS; ++b) {
      const int mine = (int)((uint32_t)key[i] << (31 - b)) >> 31;
      const uint64_t set = ballot64(mine != 0);
      same &= ~(set ^ ((uint64_t)(uint32_t)mine << 32 | (uint32_t)mine));
    }
    const int before = __builtin_amdgcn_mbcnt_hi((uint32_t)(same >> 32), __builtin_amdgcn_mbcnt_lo((uint32_t)same, 0u));
    const int had = cnt[max(key[i], 0)];
    rank[i] = had + before;
    // every lane has read its count before the group's first lane adds to it (a wave's LDS accesses are in order)
    __builtin_amdgcn_wave_barrier();
    if (in && before == 0) cnt[key[i]] = (uint16_t)(had + __popcll(same));
    __builtin_amdgcn_wave_barrier();
  }
}

// COUNT: only the block's counts, to hist[block]. Otherwise the places, with the counts of the other blocks from hist if
// there are any.
template <int NT, int TURNS, int BITS, bool COUNT>
__global__ __launch_bounds__(NT) void k_group_rows(const GroupDesc d, int blocks) {
  constexpr int W = NT / 64, KPT = (kRowsMaxGroups + NT - 1) / NT;
  __shared__ uint16_t s_cnt[W][kRowsMaxGroups + 2];
  __shared__ int s_base[kRowsMaxGroups + 1];
  __shared__ int s_scan[W];
  const int tid = threadIdx.x, wave = tid >> 6, lane = tid & 63;
  const int G = d.groups;
  const int begin = blockIdx.x * (NT * TURNS), run = begin + wave * (64 * TURNS);
  int key[TURNS], rank[TURNS];
#pragma unroll
  for (int i = 0; i < TURNS; ++i) {
    key[i] = d.ids[min(run + i * 64 + lane, d.n - 1)];
    rank[i] = 0;
  }
  for (int c = lane; c <= G; c += 64) s_cnt[wave][c] = 0;
#pragma unroll
  for (int i = 0; i < TURNS; ++i) key[i] = run + i * 64 + lane >= d.n ? -1 : key[i] >= 0 && key[i] < G ? key[i] : G;
  __builtin_amdgcn_wave_barrier();
  rank_run<TURNS, BITS>(key, rank, s_cnt[wave]);
  __syncthreads();
  if constexpr (COUNT) {
    for (int c = tid; c <= G; c += NT) {
      int v = 0;
#pragma unroll
      for (int w = 0; w < W; ++w) v += s_cnt[w][c];
      d.hist[(size_t)blockIdx.x * (G + 1) + c] = (uint32_t)v;
    }
    return;
  }
  // s_cnt becomes the counts of the waves before; `all` and `earlier`: of every block, and of the blocks before this one
  int all[KPT + 1], earlier[KPT + 1];
  auto count = [&](int c, int& total, int& before) {
    int v = 0, n[W];
#pragma unroll
    for (int w = 0; w < W; ++w) n[w] = s_cnt[w][c];
#pragma unroll
    for (int w = 0; w < W; ++w) {
      s_cnt[w][c] = (uint16_t)v;
      v += n[w];
    }
    total = v;
    before = 0;
    if (blocks > 1) {
      total = 0;
#pragma unroll 4
      for (int b = 0; b < blocks; ++b) {
        const int n = (int)d.hist[(size_t)b * (G + 1) + c];
        before += b < (int)blockIdx.x ? n : 0;
        total += n;
      }
    }
  };
  int mine = 0;
#pragma unroll
  for (int i = 0; i < KPT; ++i) {
    const int c = tid * KPT + i;
    all[i] = earlier[i] = 0;
    if (c < G) count(c, all[i], earlier[i]);
    mine += all[i];
  }
  if (tid == 0) count(G, all[KPT], earlier[KPT]);
  int total;
  int start = block_excl_scan<NT>(mine, s_scan, &total);
#pragma unroll
  for (int i = 0; i < KPT; ++i) {
    const int c = tid * KPT + i;
    if (c < G) {
      s_base[c] = start + earlier[i];
      if (blockIdx.x == 0) d.offsets[c] = start;
      start += all[i];
    }
  }
  if (tid == 0) {
    s_base[G] = total + earlier[KPT];
    if (blockIdx.x == 0) d.offsets[G] = total;
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < TURNS; ++i) {
    if (key[i] < 0) continue;
    const int at = run + i * 64 + lane, place = s_base[key[i]] + s_cnt[wave][key[i]] + rank[i];
    if (d.rows) d.rows[place] = at;
    if (d.slots) d.slots[at] = key[i] == G ? -1 : place;
  }
}

// The same for fewer than 64 groups in one launch of several workgroups: each has 1024 entries to place and counts all the
// others', up to 1024 CHUNKS, besides. A wave's lane g counts group g, from the same ballots. 4096 and 8192 entries of 8
// groups 4.2 and 5.6 us, in one workgroup 5.3 and 7.9; 16384: 8.9, as in blocks.
template <int CHUNKS, int BITS>
__global__ __launch_bounds__(1024) void k_group_few(const GroupDesc d) {
  constexpr int W = 16;
  static_assert(CHUNKS * 64 < 1 << 11, "a wave's counts in bits");
  // a wave's entries of a group: in the blocks before this one (from bit 0), in it (11), everywhere (20)
  __shared__ uint32_t s_count[W][64];
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63, G = d.groups, own = blockIdx.x;
  int key[CHUNKS], rank = 0, mine = 0;
  uint32_t count = 0;
#pragma unroll
  for (int c = 0; c < CHUNKS; ++c) key[c] = d.ids[min(c * 1024 + (int)threadIdx.x, d.n - 1)];
#pragma unroll
  for (int c = 0; c < CHUNKS; ++c) {
    const bool in = c * 1024 + (int)threadIdx.x < d.n;
    const int k = key[c] >= 0 && key[c] < G ? key[c] : G;
    uint64_t of_lane = ballot64(in), of_key = of_lane;           // entries of group `lane`, and of this entry's group
    auto both = [](int v, int b) {               // bit b of v in every bit
      const uint32_t m = (uint32_t)((int)((uint32_t)v << (31 - b)) >> 31);
      return (uint64_t)m << 32 | m;
    };
#pragma unroll
    for (int b = 0; b < BITS; ++b) {
      const uint64_t set = ballot64((k >> b & 1) != 0);
      of_lane &= ~(set ^ both(lane, b));
      if (c == own) of_key &= ~(set ^ both(k, b));
    }
    const uint32_t n = lane >> BITS ? 0u : (uint32_t)__popcll(of_lane);
    count += (n << 20) + (c < own ? n : c == own ? n << 11 : 0u);
    if (c == own) {
      rank = __builtin_amdgcn_mbcnt_hi((uint32_t)(of_key >> 32), __builtin_amdgcn_mbcnt_lo((uint32_t)of_key, 0u));
      mine = k;
    }
  }
  s_count[wave][lane] = count;
  __syncthreads();
  // every wave sums for itself: lane g the start of group g, and where this wave's entries of it go
  int all = 0, earlier = 0;
#pragma unroll
  for (int w = 0; w < W; ++w) {
    const uint32_t v = s_count[w][lane];
    all += (int)(v >> 20);
    earlier += (int)((v & 2047u) + (w < wave ? v >> 11 & 511u : 0u));
  }
  const int start = wave_incl_scan(all) - all;
  if (own == 0 && wave == 0 && lane <= G) d.offsets[lane] = start;
  const int place = __shfl(start + earlier, mine, 64) + rank, at = own * 1024 + threadIdx.x;
  if (at >= d.n) return;
  if (d.rows) d.rows[place] = at;
  if (d.slots) d.slots[at] = mine == G ? -1 : place;
}

// Every block adds up the counts of all of them, which takes less than a launch between up to some hundred thousand entries
// and grows with their square: 8, 256, 1024 groups of 2^16 entries 10.5, 13.7, 15.7 us, 2^18 17.5, 21.6, 24.5, 2^20 46, 57,
// 63, 2^22 238, 333, 383, 2^24 (4096 blocks) 3.1, 4.8, 9.8 ms.
int group_rows_blocks(int n) { return n <= kOneBlock ? 1 : (n + kBlock - 1) / kBlock; }

template <int BITS>
static hipError_t group_rows(const GroupDesc& d, hipStream_t s) {
  const int blocks = group_rows_blocks(d.n);
  if (blocks > 1) {
    ffn_launch((k_group_rows<1024, 4, BITS, true>), dim3(blocks), dim3(1024), 0, s, d, blocks);
    ffn_launch((k_group_rows<1024, 4, BITS, false>), dim3(blocks), dim3(1024), 0, s, d, blocks);
  } else if (d.n <= 256) {
    ffn_launch((k_group_rows<256, 1, BITS, false>), dim3(1), dim3(256), 0, s, d, 1);
  } else if constexpr (BITS <= 6) {
    const dim3 grid((d.n + 1023) / 1024);
    if (d.n <= 2048) ffn_launch((k_group_few<2, BITS>), grid, dim3(1024), 0, s, d);
    else if (d.n <= 4096) ffn_launch((k_group_few<4, BITS>), grid, dim3(1024), 0, s, d);
    else ffn_launch((k_group_few<8, BITS>), grid, dim3(1024), 0, s, d);
  } else if (d.n <= 4096) {
    ffn_launch((k_group_rows<1024, 4, BITS, false>), dim3(1), dim3(1024), 0, s, d, 1);
  } else {
    ffn_launch((k_group_rows<1024, 8, BITS, false>), dim3(1), dim3(1024), 0, s, d, 1);
  }
  return hipGetLastError();
}
hipError_t launch_group_rows(const GroupDesc& d, hipStream_t s) {
  // bits of a group's number, `groups` (none) among them (8192 entries of 8 groups in one workgroup: 7.1 us; by 11 bits 10.8)
  if (d.groups < 16) return group_rows<4>(d, s);
  if (d.groups < 64) return group_rows<6>(d, s);
  if (d.groups < 512) return group_rows<9>(d, s);
  return group_rows<11>(d, s);
}

// ---------------------------------------------------------------- gather
// TPR threads a row, 8 elements each at a time.
template <typename T, int TPR, bool FP8>
__global__ __launch_bounds__(256) void k_gather(const RowsDesc d) {
  constexpr int RPB = 256 / TPR;
  const int u = threadIdx.x % TPR;
  const long long row = ((long long)blockIdx.y * gridDim.x + blockIdx.x) * RPB + threadIdx.x / TPR;
  const bool here = row < d.m;
  const size_t t = here ? (size_t)row : (size_t)d.m - 1;
  const int n = d.m * d.top_k;
  const int32_t* slots = d.slots + t * d.top_k;
  for (int c0 = 0; c0 < d.d; c0 += TPR * 8) {    // all of a row's lanes stay: they share blocks of 128 columns
    const int c = c0 + u * 8;
    const bool in = here && c < d.d;
    Row8<T> v;
    v.zero();
    if (in) v.load(d.x, t * d.d + c);
    float f[8];
    v.get(f);
    float scale = 0.f;
    uint2 q = {0, 0};
    if constexpr (FP8) {
      scale = fp8_scale(row16_max(max8(f, 0u)));
      q = fp8_pack8(f, 1.0f / scale);
    }
    if (!in) continue;
    for (int s = 0; s < d.top_k; ++s) {
      const int to = slots[s];
      if (to < 0 || to >= n) continue;
      if (d.y) Row8<T>::store(d.y, (size_t)to * d.d + c, f);
      if constexpr (FP8) {
        *reinterpret_cast<uint2*>(d.q + (size_t)to * d.d + c) = q;
        if ((threadIdx.x & 15) == 0) d.scale[(size_t)(c / kFp8Block) * n + to] = scale;
      }
    }
  }
}

template <typename T, int TPR>
static hipError_t go_gather(const RowsDesc& d, hipStream_t s) {
  const dim3 grid = grid2(((long long)d.m + 256 / TPR - 1) / (256 / TPR));
  if (d.q) ffn_launch((k_gather<T, TPR, true>), grid, dim3(256), 0, s, d);
  else ffn_launch((k_gather<T, TPR, false>), grid, dim3(256), 0, s, d);
  return hipGetLastError();
}
// 4096 rows with 16, 64 and 256 threads each, us: gather of 128 columns 2.8, 3.1, 4.1, of 512 5.3, 4.1, 4.8, of 1024 9.4,
// 6.5, 6.3; combination's gradients of 128 columns 3.0, 3.5, 5.2, of 512 6.3, 5.8, 6.9, of 1024 9.4, 8.6, 9.3.
template <typename T>
static hipError_t gather(const RowsDesc& d, hipStream_t s) {
  if (d.d <= 128) return go_gather<T, 16>(d, s);
  if (d.d <= 512) return go_gather<T, 64>(d, s);
  return go_gather<T, 256>(d, s);
}
hipError_t launch_gather(const RowsDesc& d, hipStream_t s) {
  return d.dtype == DT_BF16 ? gather<uint16_t>(d, s) : gather<float>(d, s);
}

// ---------------------------------------------------------------- combination
// K slots a token at most: their rows' loads go out together.
template <typename T, int TPR, int K>
__global__ __launch_bounds__(256) void k_combine_fwd(const RowsDesc d) {
  constexpr int RPB = 256 / TPR;
  const int u = threadIdx.x % TPR;
  const long long t = ((long long)blockIdx.y * gridDim.x + blockIdx.x) * RPB + threadIdx.x / TPR;
  if (t >= d.m) return;
  const int n = d.m * d.top_k;
  int from[K];
  float w[K];
#pragma unroll
  for (int s = 0; s < K; ++s) {
    from[s] = s < d.top_k ? d.slots[t * d.top_k + s] : -1;
    if (from[s] >= n) from[s] = -1;
    w[s] = s >= d.top_k ? 0.f : d.weights ? d.weights[t * d.top_k + s] : 1.f;
  }
  for (int c = u * 8; c < d.d; c += TPR * 8) {
    Row8<T> v[K], r;
    r.zero();
    if (d.residual) r.load(d.residual, (size_t)t * d.d + c);
#pragma unroll
    for (int s = 0; s < K; ++s)
      if (from[s] >= 0) v[s].load(d.x, (size_t)from[s] * d.d + c);
    float acc[8];
    r.get(acc);
#pragma unroll
    for (int s = 0; s < K; ++s) {
      if (from[s] < 0) continue;
      float f[8];
      v[s].get(f);
#pragma unroll
      for (int j = 0; j < 8; ++j) acc[j] = fmaf(w[s], f[j], acc[j]);
    }
    Row8<T>::store(d.y, (size_t)t * d.d + c, acc);
  }
}

template <typename T, int TPR, int K>
__global__ __launch_bounds__(256) void k_combine_bwd(const RowsDesc d) {
  constexpr int RPB = 256 / TPR;
  __shared__ float s_dot[4][K];
  const int u = threadIdx.x % TPR;
  const long long row = ((long long)blockIdx.y * gridDim.x + blockIdx.x) * RPB + threadIdx.x / TPR;
  const bool here = row < d.m;
  const size_t t = here ? (size_t)row : (size_t)d.m - 1;
  const int n = d.m * d.top_k;
  int at[K];
  float w[K], dot[K];
#pragma unroll
  for (int s = 0; s < K; ++s) {
    at[s] = here && s < d.top_k ? d.slots[t * d.top_k + s] : -1;
    if (at[s] >= n) at[s] = -1;
    w[s] = s >= d.top_k ? 0.f : d.weights ? d.weights[t * d.top_k + s] : 1.f;
    dot[s] = 0.f;
  }
  for (int c = u * 8; c < d.d; c += TPR * 8) {
    Row8<T> g, v[K];
    g.load(d.dout, t * d.d + c);
    if (d.dweights) {
#pragma unroll
      for (int s = 0; s < K; ++s)
        if (at[s] >= 0) v[s].load(d.x, (size_t)at[s] * d.d + c);
    }
    float f[8];
    g.get(f);
#pragma unroll
    for (int s = 0; s < K; ++s) {
      if (at[s] < 0) continue;
      if (d.dweights) {
        float y[8];
        v[s].get(y);
#pragma unroll
        for (int j = 0; j < 8; ++j) dot[s] = fmaf(f[j], y[j], dot[s]);
      }
      if (d.y) {
        float o[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) o[j] = w[s] * f[j];
        Row8<T>::store(d.y, (size_t)at[s] * d.d + c, o);
      }
    }
  }
  if (!d.dweights) return;
#pragma unroll
  for (int s = 0; s < K; ++s) {
    float v = dot[s];
    if constexpr (TPR >= 64) {
      v = wave_sum(v);
      if constexpr (TPR > 64) {
        if ((threadIdx.x & 63) == 0) s_dot[threadIdx.x >> 6][s] = v;
      }
    } else {
      v += wave_xchg<8>(v);
      v += wave_xchg<4>(v);
      v += wave_xchg<2>(v);
      v += wave_xchg<1>(v);
    }
    dot[s] = v;
  }
  if constexpr (TPR > 64) {
    __syncthreads();
#pragma unroll
    for (int s = 0; s < K; ++s) dot[s] = ((s_dot[0][s] + s_dot[1][s]) + s_dot[2][s]) + s_dot[3][s];
  }
  if (here && u == 0) {
#pragma unroll
    for (int s = 0; s < K; ++s)
      if (s < d.top_k) d.dweights[t * d.top_k + s] = at[s] >= 0 ? dot[s] : 0.f;
  }
}

template <typename T, int TPR, int K>
static hipError_t go_combine(const RowsDesc& d, bool fwd, hipStream_t s) {
  const dim3 grid = grid2(((long long)d.m + 256 / TPR - 1) / (256 / TPR));
  if (fwd) ffn_launch((k_combine_fwd<T, TPR, K>), grid, dim3(256), 0, s, d);
  else ffn_launch((k_combine_bwd<T, TPR, K>), grid, dim3(256), 0, s, d);
  return hipGetLastError();
}
template <typename T, int TPR>
static hipError_t by_slots(const RowsDesc& d, bool fwd, hipStream_t s) {
  if (d.top_k <= 1) return go_combine<T, TPR, 1>(d, fwd, s);
  if (d.top_k <= 2) return go_combine<T, TPR, 2>(d, fwd, s);
  if (d.top_k <= 4) return go_combine<T, TPR, 4>(d, fwd, s);
  if (d.top_k <= 8) return go_combine<T, TPR, 8>(d, fwd, s);
  return go_combine<T, TPR, 16>(d, fwd, s);
}
// As gather.
template <typename T>
static hipError_t combine(const RowsDesc& d, bool fwd, hipStream_t s) {
  if (d.d <= 128) return by_slots<T, 16>(d, fwd, s);
  if (d.d <= 512) return by_slots<T, 64>(d, fwd, s);
  return by_slots<T, 256>(d, fwd, s);
}
hipError_t launch_combine_fwd(const RowsDesc& d, hipStream_t s) {
  return d.dtype == DT_BF16 ? combine<uint16_t>(d, true, s) : combine<float>(d, true, s);
}
hipError_t launch_combine_bwd(const RowsDesc& d, hipStream_t s) {
  return d.dtype == DT_BF16 ? combine<uint16_t>(d, false, s) : combine<float>(d, false, s);
}

}  // namespace ffn
