// Products of 8-bit blocks and products grouped by expert on gfx950.
//
// out[r][c] = sum_j B[r][j] A[c][j]: a workgroup of eight waves owns an RT x CT
// tile of the output (RT rows, CT columns) and walks the contraction in steps
// of 128 bytes of a row: one 8-bit block, or 64 bf16 elements. Both operands'
// slices of the next step travel from memory straight into the other of two LDS
// stages (16-byte loads to LDS, no registers) while the matrix cores work on
// this one; one barrier a step. Products run on 16 x 16 MFMA tiles (operand
// lane l: row l % 16, contraction elements in group l / 16; accumulator lane l:
// columns 4 (l / 16) + v of the output, row l % 16, so a lane stores four
// neighbours). Workgroups stay and walk over the tiles, the next tile's loads
// going out before this one is stored.
//
// What bounds it. A 256 x 256 step needs 2048 cycles of the matrix cores, 64 KB
// into LDS and 192 KB out of it (770 cycles); whole rounds of such tiles run at
// 1.37-1.40 PFLOP/s in bf16 (4096 x 8192 x 4096: 197-203 us) and 2.1-2.2 in 8
// bits (4096 x 4096 x 8192: 120-124 us), where the chip is held by its power:
// the bf16 product of zeros takes 190 us where normal numbers took 215-260 on
// an earlier version of the loop. Beyond that it is shape: half-empty last
// rounds (4096 x 4096 x 14336 8-bit, 3.5 rounds: 235 us, 2.05 PFLOP/s) and last
// tiles of the experts (8192 rows over 8 experts, 4096 x 14336: 840-880 us, 1.1
// PFLOP/s). Exact 8-bit sums take 128 x 256 tiles, whose registers also hold
// the converted operand (14336 x 4096 over 4096: 446-464 us, 1.04-1.08 PFLOP/s).
// dW is bound by the seams between short tiles and its stores there (8 x 8192 x
// 2048 over 4095 rows: 187-196 us for 137 GFLOP and 537 MB; 165 without the
// stores, its whole steps alone 105). Adding to old sums takes 330 us.
//
// LDS layouts, both without bank conflicts. An operand whose rows run along the
// contraction keeps 128-byte rows, chunk c of 16 bytes at c ^ (row % 8): the 16
// rows of a 16-byte operand read fall into different banks. An operand read
// across its rows (W in dx, both in dW: the contraction is the slower index)
// keeps the rows as they lie in memory, 64 of them a step, and is transposed on
// the way to the registers by ds_read_b64_tr_b16; chunk c lies at c ^ f(row), f
// spreading the 16 rows one such read touches. Loads to LDS write 16 bytes a lane in lane order, so the
// permutation is applied to the address that is read.
//
// How 8-bit products are summed. The e4m3 matrix instructions hold each sum of
// 8 products (8 consecutive k of a row) to 13 bits below its largest product
// and add such sums in fp32 (measured: 2^16 + 2^3 is exact, 2^16 + 2^2 is
// 2^16, and sums of different eights are exact to 24 bits). That is at most
// 7 * 2^-13 of each eight's largest product; of the norm of a product of 4096
// normal values 2e-5, with one channel in a hundred 20 times as large 6e-5, far
// below a bf16 output's rounding. Where products cancel it is not: 0.5% of
// those outputs lose more than half a bf16 step, with the large channels 1.2%.
// So bf16 outputs are made this way, for twice the rate, as the header says, and an
// fp32 output (a weight's gradient) is made on the bf16 instructions, at half
// their rate: every e4m3 value is a bf16 value, products of two are exact in
// fp32, and so are their sums to fp32 roundings. A block's sum starts at zero, is scaled in fp32 and
// added to the accumulator.
#include <algorithm>
#include <type_traits>

#include "lin_util.cuh"

namespace ffn {

typedef short s16x4_t __attribute__((ext_vector_type(4)));

constexpr int LIN_THREADS = 512;
constexpr int kCUs = 256;                        // MI355X
constexpr int LIN_BYTES = 128;                   // contraction bytes of a step

// 16 (or 4) bytes a lane from base + off to LDS: the wave's lanes in order from
// address `l` on. In assembly, because the compiler takes a load to LDS for a
// possible writer of whatever LDS is read next and waits for it there, which
// would end the overlap; lin_sync() is the wait. Such a load has no register
// to write, and the compiler's own waits for other loads only become stricter.
__device__ __forceinline__ uint32_t lds_address(const char* l) {
  return (uint32_t)(uintptr_t)(__attribute__((address_space(3))) const char*)l;
}
__device__ __forceinline__ void lds_load16(const char* base, uint32_t off, uint32_t l) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, %2" ::"s"(l), "v"(off), "s"(base) : "m0");
}
__device__ __forceinline__ void lds_load16(const char* p, uint32_t l) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, off" ::"s"(l), "v"(p) : "m0");
}
__device__ __forceinline__ void lds_load4(const char* base, uint32_t off, uint32_t l) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dword %1, %2" ::"s"(l), "v"(off), "s"(base) : "m0");
}
// Every load to LDS and every LDS read of this wave is done, then every wave's.
__device__ __forceinline__ void lin_sync() {
  asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" ::: "memory");
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

__device__ const uint4 lin_zero = {0, 0, 0, 0};  // what lies behind the contraction's end

// One operand's slice of a step in LDS: R rows of the output's side.
// ALONG: rows of 128 bytes along the contraction; otherwise 64 contraction
// rows of R bf16 elements.
template <int R, bool ALONG>
struct LinTile {
  static constexpr int BYTES = R * LIN_BYTES;
  static constexpr int LOADS = BYTES / (LIN_THREADS * 16);     // 16-byte loads of a thread
  static_assert(LOADS >= 1, "tile too small");
  static constexpr int CPR = ALONG ? 8 : R / 8;                // chunks of an LDS row
  __host__ __device__ __forceinline__ static constexpr int swz(int row) { return (ALONG ? row : ((row & 3) << 1) | (row & 8)) & (CPR < 16 ? CPR - 1 : 15); }
  // load q = i * 512 + thread: LDS chunk q, that is row q / CPR, place q % CPR
  __device__ __forceinline__ static int row_of(int q) { return q / CPR; }
  __device__ __forceinline__ static int chunk_of(int q) { return (q % CPR) ^ swz(q / CPR); }
};

// Where a thread's loads of one operand come from: `base` (uniform, moving on
// by `step` bytes a step) + min(first + i * stride, last). All loads of a
// thread lie at the same place of their LDS rows (512 threads are whole groups
// of rows with the same permutation), so two registers describe them.
template <int R, bool ALONG, int ESZ>
struct LinSrc {
  using T = LinTile<R, ALONG>;
  static constexpr int ROWS = LIN_THREADS / T::CPR;            // LDS rows of one load of the workgroup
  static_assert(T::LOADS == 1 || T::swz(ROWS) == 0, "loads at one place of their rows");
  const char* base;
  size_t step;
  uint32_t first, last, stride;
  // rows r0.. of at most rend rows of p, contraction from k0 on, ld elements apart.
  // Rows past the end repeat the last one: their results are not stored.
  __device__ __forceinline__ void init(const char* p, int ld, int r0, int rend, int k0, int tid) {
    const uint32_t pitch = (uint32_t)ld * ESZ;
    if constexpr (ALONG) {
      base = p + ((size_t)r0 * ld + k0) * ESZ;
      step = LIN_BYTES;
      first = T::row_of(tid) * pitch + T::chunk_of(tid) * 16;
      last = (uint32_t)min(rend - 1 - r0, R - 1) * pitch + T::chunk_of(tid) * 16;   // of the tile: 32 bits hold that, not the operand
    } else {
      base = p + ((size_t)k0 * ld + r0) * ESZ;
      step = (size_t)64 * pitch;
      first = T::row_of(tid) * pitch + min(T::chunk_of(tid) * 8, rend - 8 - r0) * ESZ;
      last = 0xFFFFFFFFu;
    }
    stride = ROWS * pitch;
  }
  // load i of the step that `base` points at; `at`: the wave's place in the operand's LDS tile
  __device__ __forceinline__ void load(int i, uint32_t at) const {
    uint32_t o = first + i * stride;
    asm volatile("" : "+v"(o));                  // made here, not kept (as a 64-bit pair) over the loop
    lds_load16(base, ALONG ? min(o, last) : o, at + i * LIN_THREADS * 16);
  }
  // load i of the last, partial step: `left` contraction elements, zeros behind them
  __device__ __forceinline__ void load_part(int i, uint32_t at, int left, int tid) const {
    const int q = i * LIN_THREADS + tid;
    const bool in = ALONG ? T::chunk_of(q) * (16 / ESZ) < left : T::row_of(q) < left;
    const uint32_t o = first + i * stride;
    lds_load16(in ? base + (ALONG ? min(o, last) : o) : reinterpret_cast<const char*>(&lin_zero), at + i * LIN_THREADS * 16);
  }
};

template <int KIND, int RT, int CT, bool EXACT, bool AROW>
__global__ __launch_bounds__(LIN_THREADS, RT * CT > 128 * 128 ? 2 : 4) void k_linear(const LinDesc d) {
  constexpr bool FP8 = KIND == LIN_FP8;
  constexpr bool AALONG = KIND == LIN_FP8 || KIND == LIN_FWD, BALONG = KIND != LIN_DW;
  constexpr int ESZ = FP8 ? 1 : 2, BK = LIN_BYTES / ESZ;
  constexpr int WR = RT >= 128 ? 2 : 1, WC = 8 / WR;           // waves along rows and columns
  constexpr int BT = RT / WR / 16, AT = CT / WC / 16;          // 16 x 16 tiles of a wave
  using TA = LinTile<CT, AALONG>;
  using TB = LinTile<RT, BALONG>;
  constexpr int SCALES = FP8 ? (RT + CT) * 4 : 0;
  constexpr int STAGE = TA::BYTES + TB::BYTES + SCALES;
  __shared__ __attribute__((aligned(16))) char smem[2][STAGE];
  __shared__ int s_start[kLinMaxGroups + 1], s_first[kLinMaxGroups];   // first row (or end) and first row tile of an expert
  __shared__ int s_scan[LIN_THREADS / 64];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wc = wave % WC, wr = wave / WC;

  // ---------------------------------------------------------------- the tiles of this workgroup
  int rtiles;
  {
    // starts: never before an earlier one, by a running maximum over the waves' lanes and then the waves
    int v = tid <= d.groups ? expert_start(d.offsets, tid, KIND == LIN_DW ? d.K : d.rows) : 0;
#pragma unroll
    for (int o = 1; o < 64; o *= 2) {
      const int w = __shfl_up(v, o, 64);
      if (lane >= o) v = max(v, w);
    }
    if (lane == 63) s_scan[wave] = v;
    __syncthreads();
    for (int w = 0; w < wave; ++w) v = max(v, s_scan[w]);
    if (tid <= kLinMaxGroups) s_start[tid] = v;
    __syncthreads();
    const int rows = tid < d.groups ? s_start[tid + 1] - s_start[tid] : 0;
    const int mine = tid >= d.groups ? 0 : ((KIND == LIN_DW ? d.rows : rows) + RT - 1) / RT;
    const int first = block_excl_scan<LIN_THREADS>(mine, s_scan, &rtiles);
    rtiles = __builtin_amdgcn_readfirstlane(rtiles);
    if (tid < kLinMaxGroups) s_first[tid] = tid < d.groups ? first : 0x7FFFFFFF;
    __syncthreads();
  }
  const int ctiles = (d.cols + CT - 1) / CT, tiles = ctiles * rtiles;
  // Workgroups go to the 8 XCDs in turn; each XCD takes a contiguous run of tiles, its workgroups one after the other.
  // Tiles come in patches of 8 row tiles by 4 column tiles, about what an XCD works on at a time, so that a step's
  // slices are read by 8 or 4 of its workgroups and come from its L2 but once; patches run down all rows before the
  // next 4 columns, so that the weights are read about once in all. Slices of the contraction come last.
  const int total = tiles * d.ks, per = (total + 7) / 8, stride = gridDim.x >> 3;
  const int run0 = (blockIdx.x & 7) * per, end = min(run0 + per, total), begin = run0 + (blockIdx.x >> 3);
  struct Tile {
    int g, r0, rend, c0, z, klo, full, left, steps;
  };
  auto tile_at = [&](int at) {
    constexpr int PR = 8, PC = 4;
    Tile x;
    x.z = d.ks == 1 ? 0 : at / tiles;
    const int lin = at - x.z * tiles;
    const int strip = lin / (PC * rtiles), ins = lin - strip * PC * rtiles;
    const int sw = min(PC, ctiles - strip * PC);
    const int patch = sw == PC ? ins / (PR * PC) : ins / (PR * sw), inp = ins - patch * PR * sw;
    const int ph = min(PR, rtiles - patch * PR), down = ph == PR ? inp / PR : inp / ph;
    const int rt = patch * PR + inp - down * ph;
    x.c0 = (strip * PC + down) * CT;
    int n = 0;                                   // the last expert that starts at or before row tile rt
#pragma unroll
    for (int i = 0; i < kLinMaxGroups / 64; ++i) n += __popcll(ballot64(s_first[i * 64 + lane] <= rt));
    x.g = n - 1;
    const int lo = __builtin_amdgcn_readfirstlane(s_start[x.g]), hi = __builtin_amdgcn_readfirstlane(s_start[x.g + 1]);
    const int in = rt - __builtin_amdgcn_readfirstlane(s_first[x.g]);
    x.r0 = (KIND == LIN_DW ? 0 : lo) + in * RT;
    x.rend = KIND == LIN_DW ? d.rows : hi;
    x.klo = KIND == LIN_DW ? lo : 0;
    const int k = KIND == LIN_DW ? hi - lo : d.K, all = k / BK;
    // a slice: whole steps, the last one with what is left
    const int s0 = (int)((long long)all * x.z / d.ks);
    x.full = (int)((long long)all * (x.z + 1) / d.ks) - s0;
    x.klo += s0 * BK;
    x.left = x.z + 1 == d.ks ? k - all * BK : 0;
    x.steps = x.full + (x.left > 0);
    return x;
  };

  // ---------------------------------------------------------------- loads
  // The cursor: the step whose loads go out, up to two steps ahead of the products and so, at the end of a tile, in
  // the next one: its first slices arrive while this tile is finished and stored.
  LinSrc<CT, AALONG, ESZ> sa;
  LinSrc<RT, BALONG, ESZ> sb;
  int cat = begin - stride, cstep = 0, cfull = 0, cleft = 0, ckb = 0;
  Tile ctile;                                    // the cursor's tile
  bool more = true;
  // 8-bit blocks: the step's scales travel with it, one float a row of B (threads 0 .. RT - 1) and a column of the
  // tile (the next CT threads; with blocks of 128 rows of A, columns of a block all get its scale)
  static_assert(RT + CT <= LIN_THREADS, "one scale a thread");
  const int kblocks = (d.K + kFp8Block - 1) / kFp8Block;
  const char *scb = nullptr, *sca = nullptr;
  const size_t sca_step = AROW ? (size_t)d.cols * 4 : 4;
  uint32_t scoff = 0;
  auto advance = [&] {
    sa.base += sa.step;
    sb.base += sb.step;
    if (++cstep < cfull + (cleft > 0)) return;
    Tile x;
    do {
      cat += stride;
      more = cat < end;
      if (!more) return;
      x = tile_at(cat);
    } while (x.steps == 0);
    ctile = x;
    cstep = 0;
    cfull = x.full;
    cleft = x.left;
    const char* A = reinterpret_cast<const char*>(d.A) + (KIND == LIN_DW ? 0 : (size_t)x.g * d.a_group * ESZ);
    sa.init(A, AALONG ? d.K : d.cols, x.c0, d.cols, x.klo, tid);
    sb.init(reinterpret_cast<const char*>(d.B), BALONG ? d.K : d.rows, x.r0, x.rend, x.klo, tid);
    if constexpr (FP8) {
      ckb = x.klo / BK;
      scb = reinterpret_cast<const char*>(d.sb + x.r0);
      const int c = min(tid - RT, d.cols - 1 - x.c0);
      if constexpr (AROW) {
        sca = reinterpret_cast<const char*>(d.sa + x.c0);
        scoff = (uint32_t)c * 4;
      } else {
        sca = reinterpret_cast<const char*>(d.sa + ((size_t)x.g * ((d.cols + kFp8Block - 1) / kFp8Block) + x.c0 / kFp8Block) * kblocks);
        scoff = (uint32_t)(c / kFp8Block * kblocks) * 4;
      }
      if (tid < RT) scoff = (uint32_t)min(tid, x.rend - 1 - x.r0) * 4;
    }
  };

  // The steps. A step is KK * BT turns of AT matrix instructions (of AT * 4 for an exact sum); the operand of turn
  // t + AHEAD is read during turn t, A's next slice in the last turn that uses this one, so that the reads of a step
  // are all behind it AHEAD turns before its end. There the workgroup meets: the next step has arrived, nobody reads
  // this step's stage any more, and the loads of the step after the next go into it. They go out a few a turn over
  // half a step: the address unit takes 16 cycles for each, and a wave that finds its queue full stands still, matrix
  // instructions and all.
  constexpr int KK = FP8 ? 1 : 2, TURNS = KK * BT, AHEAD = FP8 ? 1 : 3, RING = AHEAD + 1;
  static_assert(TURNS % RING == 0 && TURNS > AHEAD && TURNS % 4 == 0, "turns of a step");
  constexpr int LOADS = TA::LOADS + TB::LOADS, PER = (LOADS + TURNS / 2 - 1) / (TURNS / 2), LTURNS = (LOADS + PER - 1) / PER;
  auto load = [&](char* st, int turn, bool known) {   // turn: turns since the meeting; known: a whole step
    const uint32_t at = lds_address(st) + wave * 1024;
    const bool whole = known || cstep < cfull;
#pragma unroll
    for (int i = turn * PER; i < (turn + 1) * PER && i < LOADS; ++i) {
      if (i < TA::LOADS) {
        if (whole) sa.load(i, at);
        else sa.load_part(i, at, cleft, tid);
      } else {
        if (whole) sb.load(i - TA::LOADS, at + TA::BYTES);
        else sb.load_part(i - TA::LOADS, at + TA::BYTES, cleft, tid);
      }
    }
    if (FP8 && turn == 0) {
      const uint32_t sat = lds_address(st) + TA::BYTES + TB::BYTES + wave * 256;
      const size_t kb = ckb + cstep;
      if (wave * 64 < RT) lds_load4(scb + kb * d.rows * 4, scoff, sat);
      else if (wave * 64 < RT + CT) lds_load4(sca + kb * sca_step, scoff, sat);
    }
  };

  // ---------------------------------------------------------------- operands and sums
  const int l16 = lane & 15, q4 = lane >> 4;
  // operand reads of a 16-row tile. Along the contraction: chunks q4 and q4 + 4 of a row (bf16: one for each half step;
  // 8-bit: both, in the same order for both operands); the tile's rows are l16 modulo 16, so the places are those of
  // row l16, 64 bytes apart. (8-bit chunks 2 q4 and 2 q4 + 1 would meet in banks: half the reads' cycles.)
  const int fo = l16 * LIN_BYTES + ((q4 ^ (l16 & 7)) << 4);
  // Across it (bf16), through the transposing read: in each 16 lanes, lane 4 v + u points at row 8 q4 + 4 h + v,
  // elements 4 u .. + 3, and lane j receives element j % 4 of lane 4 v + j / 4 as its value v.
  using Frag = std::conditional_t<FP8, i32x8_t, bf16x8_t>;
  auto along = [&](const char* t, int tile, int kk) -> Frag {
    const char* p = t + tile * (16 * LIN_BYTES);
    if constexpr (FP8) {
      const uint4 a = *reinterpret_cast<const uint4*>(p + fo), b = *reinterpret_cast<const uint4*>(p + (fo ^ 64));
      return as_i32x8(a, b);
    } else {
      return as_bf16x8(*reinterpret_cast<const uint4*>(p + (fo ^ (kk * 64))));
    }
  };
  auto across = [&](auto rl, const char* t, int tile, int kk) -> bf16x8_t {
    constexpr int RL = decltype(rl)::value;
    s16x4_t h[2];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int kr = kk * 32 + 8 * q4 + 4 * e + (l16 >> 2), c = tile * 16 + 4 * (l16 & 3);
      const int at = kr * RL * 2 + (((c >> 3) ^ LinTile<RL, false>::swz(kr)) << 4) + (c & 7) * 2;
      h[e] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) s16x4_t*)(t + at));
    }
    typedef short s16x8 __attribute__((ext_vector_type(8)));
    return __builtin_bit_cast(bf16x8_t, s16x8{h[0][0], h[0][1], h[0][2], h[0][3], h[1][0], h[1][1], h[1][2], h[1][3]});
  };
  auto read_a = [&](const char* st, int i, int kk) -> Frag {
    if constexpr (AALONG) return along(st, wc * AT + i, kk);
    else return across(std::integral_constant<int, CT>{}, st, wc * AT + i, kk);
  };
  auto read_b = [&](const char* st, int j, int kk) -> Frag {
    if constexpr (BALONG) return along(st + TA::BYTES, wr * BT + j, kk);
    else return across(std::integral_constant<int, RT>{}, st + TA::BYTES, wr * BT + j, kk);
  };
  // the block's sum of matrix instruction n (turn n / AT, column tile n % AT) joins the accumulator, three instructions
  // later: its result takes that long (an exact sum's four are one behind)
  constexpr int LATER = EXACT ? 1 : AT == 1 ? 2 : 3;
  // a turn's scale is replaced three turns later, before that turn's joins
  static_assert(TURNS * AT > LATER && (LATER + AT - 1) / AT <= 2, "instructions of a step");
  Frag af[AT], bf[RING];
  bf16x8_t ax[EXACT ? AT : 1][4];
  f32x4_t acc[AT][BT], fa[AROW ? AT : 1], z[LATER + 1];
  float fs[4], s1 = 0.f;
  auto scale_of = [&](const char* st) { return reinterpret_cast<const float*>(st + TA::BYTES + TB::BYTES); };
  auto fetch_b = [&](const char* st, int t) {
    bf[t % RING] = read_b(st, t % BT, t / BT);
    if constexpr (FP8) fs[t % 4] = scale_of(st)[(wr * BT + t % BT) * 16 + l16];
  };
  auto fetch_scales = [&](const char* st) {
    if constexpr (AROW) {
#pragma unroll
      for (int i = 0; i < AT; ++i) fa[i] = *reinterpret_cast<const f32x4_t*>(scale_of(st) + RT + (wc * AT + i) * 16 + 4 * q4);
    } else if constexpr (FP8) {
      s1 = scale_of(st)[RT + wc * AT * 16];
    }
  };
  auto join = [&](int n) {
    const float s = AROW ? fs[n / AT % 4] : s1 * fs[n / AT % 4];
    f32x4_t& o = acc[n % AT][n / AT % BT];
#pragma unroll
    for (int v = 0; v < 4; ++v) o[v] = fmaf(z[n % (LATER + 1)][v], AROW ? fa[AROW ? n % AT : 0][v] * s : s, o[v]);
    asm volatile("" : "+v"(o));                  // here, not where the compiler would gather them, with every z kept till then
  };

  // ---------------------------------------------------------------- the walk
  cstep = -1;
  sa.step = sb.step = 0;
  sa.base = sb.base = nullptr;
  advance();
  if (more) {
#pragma unroll
    for (int t = 0; t < LTURNS; ++t) load(smem[0], t, false);
    lin_sync();
    advance();
    if (more) {
#pragma unroll
      for (int t = 0; t < AHEAD && t < LTURNS; ++t) load(smem[1], t, false);
    }
#pragma unroll
    for (int i = 0; i < AT; ++i) af[i] = read_a(smem[0], i, 0);
#pragma unroll
    for (int t = 0; t < AHEAD; ++t) fetch_b(smem[0], t);
    fetch_scales(smem[0]);
  }
  int par = 0;
  // One step. INSIDE: the cursor's step is not the tile's last and the next is whole, so that nothing is to be decided;
  // a branch in every turn costs a sixth of the time.
  auto step = [&](auto inside) {
    constexpr bool INSIDE = decltype(inside)::value;
    char* st = smem[par];
    char* nx = smem[par ^ 1];
    if constexpr (EXACT) {
#pragma unroll
      for (int i = 0; i < AT; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) ax[i][e] = fp8_to_bf16(af[i][2 * e], af[i][2 * e + 1]);
    }
#pragma unroll
    for (int t = 0; t < TURNS; ++t) {
      const int j = t % BT;
      if (t < TURNS - AHEAD) {
        if (t + AHEAD < LTURNS && (INSIDE || more)) load(nx, t + AHEAD, INSIDE);
      } else {
        if (t == TURNS - AHEAD && (INSIDE || more)) {
          lin_sync();
          if constexpr (INSIDE) {
            sa.base += sa.step;
            sb.base += sb.step;
            ++cstep;
          } else {
            advance();
          }
        }
        if (t - (TURNS - AHEAD) < LTURNS && (INSIDE || more)) load(st, t - (TURNS - AHEAD), INSIDE);
      }
      // past the last step of all this reads a stage that nobody writes, for nothing
      if (t + AHEAD < TURNS) fetch_b(st, t + AHEAD);
      else fetch_b(nx, t + AHEAD - TURNS);
      bf16x8_t bx[4];
      if constexpr (EXACT) {
#pragma unroll
        for (int e = 0; e < 4; ++e) bx[e] = fp8_to_bf16(bf[t % RING][2 * e], bf[t % RING][2 * e + 1]);
      }
#pragma unroll
      for (int i = 0; i < AT; ++i) {
        if constexpr (FP8) {
          const int n = t * AT + i;
          f32x4_t p{0.f, 0.f, 0.f, 0.f};
          if constexpr (EXACT) {
#pragma unroll
            for (int e = 0; e < 4; ++e) p = __builtin_amdgcn_mfma_f32_16x16x32_bf16(ax[i][e], bx[e], p, 0, 0, 0);
          } else {
            p = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(af[i], bf[t % RING], p, 0, 0, 0, 0, 0, 0);
          }
          z[n % (LATER + 1)] = p;
          if (n >= LATER) join(n - LATER);
        } else {
          acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(af[i], bf[t % RING], acc[i][j], 0, 0, 0);
        }
        if (FP8 || j == BT - 1) __builtin_amdgcn_sched_barrier(0);
        if (j == BT - 1) af[i] = t + 1 < TURNS ? read_a(st, i, t / BT + 1) : read_a(nx, i, 0);
      }
      if (FP8 && t == TURNS - 1) {
#pragma unroll
        for (int n = TURNS * AT - LATER; n < TURNS * AT; ++n) join(n);
        fetch_scales(nx);
      }
      __builtin_amdgcn_sched_barrier(0);
    }
    par ^= 1;
  };
  for (int at = begin; at < end; at += stride) {
    const Tile x = cat == at ? ctile : tile_at(at);
#pragma unroll
    for (int i = 0; i < AT; ++i)
#pragma unroll
      for (int j = 0; j < BT; ++j) acc[i][j] = f32x4_t{0.f, 0.f, 0.f, 0.f};
    for (int s = 0; s < x.steps;) {
      // steps until the cursor's tile has one whole step left beyond the one under way
      const int fast = more ? min(cfull - 1 - cstep, x.steps - s) : 0;
      for (int i = 0; i < fast; ++i) step(std::true_type{});
      s += max(fast, 0);
      if (s < x.steps) {
        step(std::false_type{});
        ++s;
      }
    }
    if (KIND == LIN_DW && x.steps == 0 && d.accumulate) continue;
    const int orow = KIND == LIN_DW ? x.g * d.rows : 0;
    if (x.r0 + RT <= x.rend && x.c0 + CT <= d.cols && (d.cols & 3) == 0 && !(d.accumulate && d.ks == 1)) {
      const int row0 = orow + x.r0 + wr * BT * 16, col0 = x.c0 + wc * AT * 16 + 4 * q4;
      constexpr bool LINES = AT % 2 == 0 && !(EXACT && RT * CT <= 128 * 128);   // registers: 52 spilled there, 1% slower
      if (LINES && (KIND == LIN_DW || EXACT || d.ks > 1 || d.out_f32)) {
        // fp32 in whole lines of 128 bytes, past the caches: of two neighbouring 16 x 16 tiles, lanes 8 .. 15 of a DPP row
        // swap their rows with lanes 0 .. 7 of the other tile, so that a store has 8 rows of 32 columns. (Both gradients
        // of 4095 rows, 8 x 8192 x 2048: through the caches 462 us, past them 423, with whole lines 398; the 8-bit
        // weight gradient 475 -> 464. bf16 outputs are parts of lines, which L2 has to join: 234 -> 270.)
        float* out = d.ks > 1 ? d.part + (size_t)x.z * d.rows * d.cols : reinterpret_cast<float*>(d.out);
        out += (size_t)(row0 + (l16 & 7)) * d.cols + col0 + (l16 >> 3) * 16;
#pragma unroll
        for (int j = 0; j < BT; ++j) {
          f32x4_t* o = reinterpret_cast<f32x4_t*>(out + (size_t)(j * 16) * d.cols);
          f32x4_t* o8 = reinterpret_cast<f32x4_t*>(out + (size_t)(j * 16 + 8) * d.cols);
#pragma unroll
          for (int i = 0; i + 1 < AT; i += 2) {
            f32x4_t a = acc[i][j], b = acc[i + 1][j];
#pragma unroll
            for (int v = 0; v < 4; ++v) {
              const int av = __float_as_int(a[v]), bv = __float_as_int(b[v]);
              a[v] = __int_as_float(__builtin_amdgcn_update_dpp(av, bv, 0x128, 0xf, 0xc, false));   // row_ror:8
              b[v] = __int_as_float(__builtin_amdgcn_update_dpp(bv, av, 0x128, 0xf, 0x3, false));
            }
            __builtin_nontemporal_store(a, o + 4 * i);
            __builtin_nontemporal_store(b, o8 + 4 * i);
          }
        }
        continue;
      }
#pragma unroll
      for (int j = 0; j < BT; ++j)
#pragma unroll
        for (int i = 0; i < AT; ++i) lin_store4(d, x.z, row0 + j * 16 + l16, col0 + 16 * i, acc[i][j]);
      continue;
    }
#pragma unroll
    for (int j = 0; j < BT; ++j) {
      const int row = x.r0 + (wr * BT + j) * 16 + l16;
      if (row >= x.rend) continue;
#pragma unroll
      for (int i = 0; i < AT; ++i) {
        const int col = x.c0 + (wc * AT + i) * 16 + 4 * q4;
        if (col < d.cols) lin_store(d, x.z, orow + row, col, acc[i][j]);
      }
    }
  }
}

template <int KIND, int RT, int CT, bool EXACT, bool AROW>
static hipError_t go_linear(const LinDesc& d, hipStream_t s) {
  // as many workgroups as run at once (what their LDS allows), or as there are tiles at most: whole ones, and one
  // ragged one for each expert
  constexpr int OCC = RT * CT >= 128 * 256 ? 1 : RT * CT >= 128 * 128 ? 2 : 3;
  const long long ct = (d.cols + CT - 1) / CT;
  const long long rt = KIND == LIN_DW ? (long long)(d.rows + RT - 1) / RT * d.groups : d.rows / RT + d.groups;
  const long long wgs = std::min<long long>(ct * rt * d.ks, kCUs * OCC);
  if (ct * rt * d.ks > 0x3FFFFFFF) return hipErrorInvalidValue;
  ffn_launch((k_linear<KIND, RT, CT, EXACT, AROW>), dim3((unsigned)(wgs + 7) / 8 * 8), dim3(LIN_THREADS), 0, s, d);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || d.ks == 1) return e;
  return launch_linear_sum(d, s);
}
template <int KIND, bool EXACT = false, bool AROW = false>
static hipError_t pick_linear(const LinDesc& d, const LinPlan& p, hipStream_t s) {
  if (p.rt == 64) return go_linear<KIND, 64, 128, EXACT, AROW>(d, s);
  if (p.rt == 128 && p.ct == 128) return go_linear<KIND, 128, 128, EXACT, AROW>(d, s);
  if constexpr (EXACT) return go_linear<KIND, 128, 256, EXACT, AROW>(d, s);
  else return p.rt == 128 ? go_linear<KIND, 128, 256, EXACT, AROW>(d, s) : go_linear<KIND, 256, 256, EXACT, AROW>(d, s);
}
hipError_t launch_linear_tiled(const LinDesc& d, const LinPlan& p, hipStream_t s) {
  switch (d.kind) {
    case LIN_FP8:
      if (d.a_rows == 1) return d.out_f32 ? pick_linear<LIN_FP8, true, true>(d, p, s) : pick_linear<LIN_FP8, false, true>(d, p, s);
      return d.out_f32 ? pick_linear<LIN_FP8, true>(d, p, s) : pick_linear<LIN_FP8>(d, p, s);
    case LIN_FWD: return pick_linear<LIN_FWD>(d, p, s);
    case LIN_DX: return pick_linear<LIN_DX>(d, p, s);
    case LIN_DW: return pick_linear<LIN_DW>(d, p, s);
  }
  return hipErrorInvalidValue;
}

// Which kernel, tile and slices, by the time that each would take, in
// microseconds, round by round of the tiles that run at once. A step of a
// round takes what the CU's tiles need for it (measured over whole rounds of
// large products: 8-bit / exact 8-bit / bf16), or its latency where a CU has
// one small tile, or, with more weights than the memory-side cache keeps, what
// HBM takes to bring the round's; to that come what a tile costs besides and
// the slabs of a sliced product, written and read, with their kernel. How the
// rows are spread over the experts only the device knows: half a tile of each
// is taken to be empty, at least. Small products end up in small tiles and
// slices (200 x 4096 x 14336 8-bit: 256-row tiles 155 us, 128 x 128 in 4 slices
// 31), weight streams in small tiles (500 rows over 5 experts of 14336 x 4096:
// 256 x 256 224 us, 64 x 128 166), large ones in large tiles (4096 x 4096 x
// 8192: 256 x 256 120 us, 128 x 128 160).
LinPlan lin_plan(int kind, int exact, int rows, int cols, int K, int groups) {
  struct Option {
    int rt, ct, occ;
    float step[3], tile;
  };
  static const Option options[] = {{256, 256, 1, {1.66f, 1e9f, 1.50f}, 7.f},
                                   {128, 256, 1, {1.01f, 1.92f, 0.94f}, 5.f},
                                   {128, 128, 2, {0.57f, 1.06f, 0.47f}, 2.5f},
                                   {64, 128, 3, {0.42f, 0.69f, 0.32f}, 1.7f}};
  constexpr float kHbm = 4.5e6f, kSlabRate = 4e6f, kSlabLaunch = 5.f;   // bytes per us, us
  constexpr double kCached = 128e6;
  LinPlan p{};
  p.ks = 1;
  const int per = kind == LIN_DW ? rows : (rows + groups - 1) / groups, bytes = kind == LIN_FP8 ? 1 : 2;
  // Few rows: k_linear_skinny up to 16, and up to 32 while the weights are few enough for latency to count (24 rows of
  // five experts: 21 MB 13.5 us, 64 x 128 tiles 14.2; 587 MB 167 us, tiles 127). Experts of more than 10 rows on the
  // average have some of more than 16: 32-row tiles then, or for large 8-bit weights k_linear (128 rows over 8 experts:
  // 268 MB bf16 16-row tiles 90 us, 32-row 68, k_linear 69; 470 MB 8-bit 162, 143, 112).
  const double weights = (double)groups * cols * K * bytes;
  const bool few = weights <= 48e6, uneven = groups > 1 && per > 10;
  // A grid holds fewer than 2^32 threads.
  const bool fits = ((long long)(cols + 15) / 16) * (rows / 16 + groups) < 1 << 22;
  if ((kind == LIN_FP8 || kind == LIN_FWD) && fits && (per <= 16 ? few || !uneven || kind == LIN_FWD : per <= 32 && few)) {
    p.skinny = 1;
    p.mb = per <= 16 && !uneven ? 1 : 2;
    const int cw = p.mb == 1 || exact ? 16 : 32, nb = (K * bytes + 127) / 128;
    const int rt = (per + 16 * p.mb - 1) / (16 * p.mb) * groups;
    const long long wgs = (long long)(cols + cw - 1) / cw * rt;
    p.nw = p.mb == 1 && wgs < 512 && nb >= 32 ? 16 : 8;
    // slices, where the workgroups leave CUs empty: at least two turns of the waves each
    while (wgs * p.ks < 256 && p.ks < 16 && nb / (p.ks * 2) >= 2 * p.nw) p.ks *= 2;
    return p;
  }
  // in 64 bits: the contraction of dW is the rows, up to 2^31
  const int steps = (int)(((long long)(kind == LIN_DW ? (K + groups - 1) / groups : K) * bytes + LIN_BYTES - 1) / LIN_BYTES);
  double best = 1e30;                            // us: a float would lose the tiles' own costs beside 2^24 steps
  for (const Option& o : options) {
    long long rt = (long long)((per + o.rt - 1) / o.rt) * groups;
    if (kind != LIN_DW && groups > 1) rt = std::max<long long>(rt, (rows + o.rt - 1) / o.rt + groups / 2);
    const long long tiles = rt * ((cols + o.ct - 1) / o.ct);
    for (const int ks : {1, 2, 3, 4, 6, 8, 12, 16}) {
      if (ks > 1 && (kind == LIN_DW || steps / ks < 4)) break;
      const long long n = tiles * ks, slots = (long long)kCUs * o.occ, rounds = (n + slots - 1) / slots;
      const long long at_once = std::min(n, slots), each = rounds > 1 ? o.occ : (n + kCUs - 1) / kCUs;   // of a CU
      const bool cold = kind != LIN_DW && weights > kCached;
      float step = std::max(o.step[kind == LIN_FP8 ? exact : 2] * each, cold ? 0.95f : 0.6f);
      if (cold) step = std::max(step, (float)(weights / ((double)tiles * steps)) * at_once / kHbm);
      double t = rounds * ((double)step * ((steps + ks - 1) / ks) + o.tile * each);
      if (ks > 1) t += kSlabLaunch + 2. * 4. * ks * rows * cols / kSlabRate;
      if (t < best) {
        best = t;
        p.rt = o.rt;
        p.ct = o.ct;
        p.ks = ks;
      }
    }
  }
  return p;
}
size_t lin_workspace(const LinPlan& p, int rows, int cols) { return p.ks > 1 ? (size_t)p.ks * rows * cols * 4 : 0; }

hipError_t launch_linear(LinDesc d, float* workspace, size_t workspace_bytes, hipStream_t s) {
  LinPlan p = lin_plan(d.kind, d.kind == LIN_FP8 && d.out_f32, d.rows, d.cols, d.K, d.groups);
  if (p.ks > 1 && (!workspace || workspace_bytes < lin_workspace(p, d.rows, d.cols))) p.ks = 1;   // whole sums then
  d.ks = p.ks;
  d.part = workspace;
  return p.skinny ? launch_linear_skinny(d, p, s) : launch_linear_tiled(d, p, s);
}

}  // namespace ffn
