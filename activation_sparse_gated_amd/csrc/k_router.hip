// The router on gfx950: scores of a token's experts, the choice of the best,
// their weights, and the gradient.
//
// LPT lanes hold a token's logits, EPL each, so a wave has 64 / LPT tokens and
// everything between the load and the result stays in registers: sums and
// maxima over a token are lane moves. The top k are k turns of a maximum, the
// first of those who have it leaving.
//
// Bound by the length of that chain of dependent steps, not by its bytes: 8 of
// 256 experts with a bias and groups, fp32, take 5.3 us for one token and 10.6
// for 8192 (0.85 TB/s; the card copies at 5.2), 16.3 and 26.0 for 16384 and 32768
// in a captured graph. The gradient, 4095 tokens of 64 experts: 3.6 us.
// All scores besides cost as much again as the choice (8192 x 256: 18.0 us): a
// lane writes its 16 experts one by one, 64 places of a wave at a time.
// Values that are equal take the long way below: 8192 x 256 logits of bf16 with a
// bias 9.8 us, with one of zeros 17.5, and all of them equal 22.2.
#include "experts.cuh"
#include "lin_util.cuh"

namespace ffn {

constexpr float kInf = __builtin_huge_valf();

template <int O>
__device__ __forceinline__ double xchg(double v) {
  const uint64_t b = __builtin_bit_cast(uint64_t, v);
  const uint32_t lo = (uint32_t)wave_xchg_i<O>((int)(uint32_t)b), hi = (uint32_t)wave_xchg_i<O>((int)(b >> 32));
  return __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}
template <int O>
__device__ __forceinline__ float xchg(float v) { return wave_xchg<O>(v); }

// Sum and maximum over the LPT lanes of a token; all of them get it.
template <int LPT, typename V>
__device__ __forceinline__ V token_sum(V v) {
  if constexpr (LPT > 32) v += xchg<32>(v);
  if constexpr (LPT > 16) v += xchg<16>(v);
  if constexpr (LPT > 8) v += xchg<8>(v);
  v += xchg<4>(v);
  v += xchg<2>(v);
  v += xchg<1>(v);
  return v;
}
template <int LPT>
__device__ __forceinline__ float token_max(float v) {
  if constexpr (LPT > 32) v = fmaxf(v, xchg<32>(v));
  if constexpr (LPT > 16) v = fmaxf(v, xchg<16>(v));
  if constexpr (LPT > 8) v = fmaxf(v, xchg<8>(v));
  v = fmaxf(v, xchg<4>(v));
  v = fmaxf(v, xchg<2>(v));
  v = fmaxf(v, xchg<1>(v));
  return v;
}
template <typename T>
__device__ __forceinline__ float logit_at(const void* p, size_t i) {
  if constexpr (sizeof(T) == 2) return bf2f(reinterpret_cast<const uint16_t*>(p)[i]);
  else return reinterpret_cast<const float*>(p)[i];
}

// log(1 / (1 + exp(-l))), which does not underflow.
__device__ __forceinline__ float log_sigmoid(float l) { return fminf(l, 0.f) - log1pf(expf(-fabsf(l))); }

// A token's chosen experts' weights without the scale, lane s (of LPT) holding slot s: `live` says whether it has an
// expert, l is its logit; mx and inv are the largest logit and 1 / (sum of exponentials) of the whole token.
template <int LPT>
__device__ __forceinline__ float chosen_weight(const RouterDesc& d, bool live, float l, float mx, float inv) {
  if (!d.renormalize) return !live ? 0.f : d.sigmoid ? 1.0f / (1.0f + expf(-l)) : expf(l - mx) * inv;
  if (!d.sigmoid && mx == kInf) return __builtin_nanf("");
  // s / (sum of s): from the logarithms, so that scores too small for fp32 keep their ratio
  const float t = !live ? -kInf : d.sigmoid ? log_sigmoid(l) : l;
  const float top = token_max<LPT>(t);
  const float e = live ? expf(t - top) : 0.f;
  const float sum = token_sum<LPT>(e);
  return live ? e / sum : 0.f;
}

// ---------------------------------------------------------------- the choice
// Expert sub * EPL + j stands in register j of the token's lane sub, so that a group of experts is a run of lanes (or of
// a lane's registers).
template <typename Key>
__device__ __forceinline__ Key maximum(Key a, Key b) { return a > b ? a : b; }
__device__ __forceinline__ float maximum(float a, float b) { return fmaxf(a, b); }

template <int LPT, typename Key>
__device__ __forceinline__ Key token_top(Key v) {
  if constexpr (LPT > 32) v = maximum(v, xchg<32>(v));
  if constexpr (LPT > 16) v = maximum(v, xchg<16>(v));
  if constexpr (LPT > 8) v = maximum(v, xchg<8>(v));
  v = maximum(v, xchg<4>(v));
  v = maximum(v, xchg<2>(v));
  v = maximum(v, xchg<1>(v));
  return v;
}
template <int LPT>
__device__ __forceinline__ int token_min(int v) {
  if constexpr (LPT > 32) v = min(v, wave_xchg_i<32>(v));
  if constexpr (LPT > 16) v = min(v, wave_xchg_i<16>(v));
  if constexpr (LPT > 8) v = min(v, wave_xchg_i<8>(v));
  v = min(v, wave_xchg_i<4>(v));
  v = min(v, wave_xchg_i<2>(v));
  v = min(v, wave_xchg_i<1>(v));
  return v;
}
// The two largest of (a, b) and of the partner lanes' at distance O.
template <int O, typename Key>
__device__ __forceinline__ void merge2(Key& a, Key& b) {
  const Key oa = xchg<O>(a), ob = xchg<O>(b);
  b = maximum(oa < a ? oa : a, maximum(b, ob));
  a = maximum(a, oa);
}
template <int N>
__device__ __forceinline__ float turned(float v) { return __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), 0x120 + N, 0xF, 0xF, false)); }
template <int N>
__device__ __forceinline__ double turned(double v) {
  const uint64_t b = __builtin_bit_cast(uint64_t, v);
  const uint32_t lo = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)(uint32_t)b, 0x120 + N, 0xF, 0xF, false);
  const uint32_t hi = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)(b >> 32), 0x120 + N, 0xF, 0xF, false);
  return __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}
__device__ __forceinline__ float read_lane(float v, int l) { return __int_as_float(wave_read(__float_as_int(v), l)); }
__device__ __forceinline__ double read_lane(double v, int l) {
  const uint64_t b = __builtin_bit_cast(uint64_t, v);
  return __builtin_bit_cast(double, (uint64_t)(uint32_t)wave_read((int)(b >> 32), l) << 32 | (uint32_t)wave_read((int)(uint32_t)b, l));
}
// Lanes of 16 whose value beats this lane's: a larger one, or an equal one of a lower group.
template <int N, typename Key>
__device__ __forceinline__ int beaten(Key v, int group, int sub, int shift) {
  if constexpr (N == 16) {
    return 0;
  } else {
    const Key o = turned<N>(v);                  // of lane (sub - N) % 16
    const int g = ((sub - N) & 15) >> shift;
    return (o > v || (o == v && g < group) ? 1 : 0) + beaten<N + 1>(v, group, sub, shift);
  }
}

// A group's value, by the two largest of its experts (-inf: none). Two biases near the lowest number sum to less than it: that
// is held at it, since -inf marks a group without experts (equal fp32 values are settled in fp64, where no sum gets there).
__device__ __forceinline__ float group_value(const RouterDesc& d, float a, float b) {
  return d.group_best == 2 && b != -kInf ? fmaxf(a + b, -__FLT_MAX__) : a;
}
__device__ __forceinline__ double group_value(const RouterDesc& d, double a, double b) {
  return d.group_best == 2 && b != -(double)kInf ? a + b : a;
}

// The lanes of a group, if every group is a run of 2^n whole lanes; 0 otherwise.
template <int LPT, int EPL>
__device__ __forceinline__ int group_lanes(const RouterDesc& d) {
  const int size = d.experts / d.groups, lanes = LPT >= 16 && size % EPL == 0 ? size / EPL : 0;
  return (lanes & (lanes - 1)) == 0 ? lanes : 0;
}
// Whether a lane's group stays, from the lane's two largest values. `gap` gets the distance between the last group that
// stays and the first that does not.
template <int LPT, typename Key>
__device__ __forceinline__ bool run_stays(const RouterDesc& d, Key a, Key b, int lanes, int sub, Key& gap) {
  const Key none = -(Key)kInf;
  const int shift = __builtin_ctz(lanes), group = sub >> shift;
  if (lanes > 1) merge2<1>(a, b);
  if (lanes > 2) merge2<2>(a, b);
  if (lanes > 4) merge2<4>(a, b);
  if constexpr (LPT == 64) {
    if (lanes > 8) merge2<8>(a, b);
    if (lanes > 16) merge2<16>(a, b);
  }
  const Key v = group_value(d, a, b);
  int rank = 0;                                  // groups that beat this one
  if constexpr (LPT == 64) {
    for (int g = 0; g < d.groups; ++g) {
      const Key o = read_lane(v, g << shift);
      rank += o > v || (o == v && g < group) ? 1 : 0;
    }
  } else {
    rank = beaten<1>(v, group, sub, shift) >> shift;
  }
  const bool stays = rank < d.top_groups && v != none;
  gap = token_top<LPT>(stays ? -v : none);       // minus the least that stays
  const Key out = token_top<LPT>(stays ? none : v);
  gap = out == none ? (Key)kInf : -gap - out;
  return stays;
}

// Which of this lane's experts (a bit each) are in the groups that stay, by their values (-inf: not to be chosen).
template <int LPT, int EPL, typename Key>
__device__ __forceinline__ uint32_t keep_groups(const RouterDesc& d, const Key (&key)[EPL], int sub, Key* lds, Key& gap) {
  const Key none = -(Key)kInf;
  const int size = d.experts / d.groups, lanes = group_lanes<LPT, EPL>(d);
  Key a = none, b = none;
  if (lanes > 0) {
#pragma unroll
    for (int j = 0; j < EPL; ++j) {
      b = maximum(b, key[j] < a ? key[j] : a);
      a = maximum(a, key[j]);
    }
    return run_stays<LPT, Key>(d, a, b, lanes, sub, gap) ? 0xFFFFu : 0u;
  }
  // through LDS: a lane reads its groups' members one after the other
#pragma unroll
  for (int j = 0; j < EPL; ++j) lds[sub * EPL + j] = key[j];
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
  constexpr int GPL = 32 / LPT > 0 ? 32 / LPT : 1;               // groups of a lane
  Key value[GPL];
#pragma unroll
  for (int i = 0; i < GPL; ++i) {
    const int g = i * LPT + sub;
    a = b = none;
    if (g < d.groups) {
      for (int n = 0; n < size; ++n) {
        const Key v = lds[g * size + n];
        b = maximum(b, v < a ? v : a);
        a = maximum(a, v);
      }
    }
    value[i] = group_value(d, a, b);
  }
  __builtin_amdgcn_wave_barrier();
  uint32_t keep = 0;
  Key last = (Key)kInf;
  gap = (Key)kInf;
  for (int n = 0; n <= d.top_groups; ++n) {
    Key v = value[0];
#pragma unroll
    for (int i = 1; i < GPL; ++i) v = maximum(v, value[i]);
    const Key top = token_top<LPT>(v);
    if (n == d.top_groups) {
      if (top != none) gap = last - top;
      break;
    }
    last = top;
    int g = 32;
#pragma unroll
    for (int i = GPL - 1; i >= 0; --i) g = value[i] == top && top != none ? i * LPT + sub : g;
    g = token_min<LPT>(g);
    if (g < 32) keep |= 1u << g;
#pragma unroll
    for (int i = 0; i < GPL; ++i)
      if (i * LPT + sub == g) value[i] = none;
  }
  const uint32_t rsize = (65536 + size - 1) / size;             // e / size for e, size <= 256
  uint32_t in = 0;
#pragma unroll
  for (int j = 0; j < EPL; ++j) {
    const uint32_t g = (uint32_t)(sub * EPL + j) * rsize >> 16;
    in |= g < 32 && (keep >> g & 1u) ? 1u << j : 0u;
  }
  return in;
}

// The expert of slot `sub` (-1: none) by its keys (-inf: not to be chosen; changed), in top_k turns: any keys, exactly.
template <int LPT, int EPL, typename Key>
__device__ __forceinline__ int pick(const RouterDesc& d, Key (&key)[EPL], int sub) {
  const Key none = -(Key)kInf;
  int id = -1;
  for (int s = 0; s < d.top_k; ++s) {
    Key v = key[0];
#pragma unroll
    for (int j = 1; j < EPL; ++j) v = maximum(v, key[j]);
    const Key top = token_top<LPT>(v);
    int e = LPT * EPL;
#pragma unroll
    for (int j = EPL - 1; j >= 0; --j) e = key[j] == top ? sub * EPL + j : e;
    e = token_min<LPT>(e);
    if (sub == s && top != none) id = e;
#pragma unroll
    for (int j = 0; j < EPL; ++j) key[j] = sub * EPL + j == e ? none : key[j];
  }
  return id;
}

// fp32 as integers of the same order, and back. (-0 as 0, which it is equal to: their bits are not.)
__device__ __forceinline__ int ordered(float v) {
  const int b = __float_as_int(v + 0.f);
  return b ^ (b >> 31 & 0x7FFFFFFF);
}
__device__ __forceinline__ float unordered(int o) { return __int_as_float(o ^ (o >> 31 & 0x7FFFFFFF)); }

// Sorts a lane's keys, the largest first: comparators of an odd-even merge sort.
template <int EPL>
__device__ __forceinline__ void sort_lane(int (&k)[EPL]) {
#pragma unroll
  for (int p = 1; p < EPL; p *= 2)
#pragma unroll
    for (int q = p; q >= 1; q /= 2)
#pragma unroll
      for (int i = q % p; i + q < EPL; i += 2 * q)
#pragma unroll
        for (int j = 0; j < q; ++j) {
          const int x = i + j, y = i + j + q;
          if (y < EPL && x / (2 * p) == y / (2 * p)) {
            const int hi = max(k[x], k[y]), lo = min(k[x], k[y]);
            k[x] = hi;
            k[y] = lo;
          }
        }
}
// The head leaves, if `own`. (In bits: a choice between two of the list's elements becomes one by a variable index.)
template <int EPL>
__device__ __forceinline__ void leave(int (&k)[EPL], bool own) {
  const int m = own ? -1 : 0;
#pragma unroll
  for (int j = 0; j + 1 < EPL; ++j) k[j] = (k[j + 1] & m) | (k[j] & ~m);
  k[EPL - 1] = ((int)0x80000000 & m) | (k[EPL - 1] & ~m);
}
template <int LPT>
__device__ __forceinline__ int token_max_i(int v) {
  if constexpr (LPT > 32) v = max(v, wave_xchg_i<32>(v));
  if constexpr (LPT > 16) v = max(v, wave_xchg_i<16>(v));
  if constexpr (LPT > 8) v = max(v, wave_xchg_i<8>(v));
  v = max(v, wave_xchg_i<4>(v));
  v = max(v, wave_xchg_i<2>(v));
  v = max(v, wave_xchg_i<1>(v));
  return v;
}

// SCORED: scores decide (a bias, or groups by sums of two); otherwise the logits do, and without a bias they always order
// the experts. The way through: values in fp32, the groups' ranks, then every lane sorts its experts, as integers whose
// lowest bits (all 16 below a bf16 logit) hold the expert's place in the lane, and top_k + 2 times the largest head leaves
// its list. Where two values lie closer than those bits and the scores' errors allow to tell, the wave orders its
// candidates again by their exact values, each in a lane of its own; where that does not settle it (groups, many equal
// values), it goes the long way: every score in fp64, one turn over all of them a slot. (The long way alone: 19.9 us for
// 8192 tokens of 256 experts, 13.2 for one; so: 10.6 and 5.3.)
template <typename T, int LPT, int EPL, bool SCORED>
__global__ __launch_bounds__(256) void k_router_fwd(const RouterDesc d) {
  constexpr int TPW = 64 / LPT;
  constexpr bool EXACT16 = sizeof(T) == 2 && !SCORED;            // the integers hold value and expert whole
  __shared__ double s_key[4 * TPW * LPT * EPL];
  __shared__ __attribute__((aligned(16))) float s_logit[4 * TPW * LPT * EPL];    // for the chosen ones: sooner there than from memory
  const int lane = lane_id(), sub = lane % LPT, wave = threadIdx.x >> 6, slot = lane / LPT;
  const long long token = ((long long)blockIdx.y * gridDim.x + blockIdx.x) * (4 * TPW) + wave * TPW + slot;
  const bool here = token < d.m;
  const size_t t = here ? (size_t)token : (size_t)d.m - 1;      // the last token again: lanes stay together
  double* lds = s_key + (wave * TPW + slot) * LPT * EPL;
  float* logits = s_logit + (wave * TPW + slot) * LPT * EPL;
  float l[EPL];
  float mx = -kInf;
  const size_t row = t * d.experts + sub * EPL;
  if (EPL * sizeof(T) % 16 == 0 && d.experts == LPT * EPL) {
    if constexpr (EPL >= 8) {
#pragma unroll
      for (int j = 0; j < EPL; j += 8) {
        Row8<T> v;
        float f[8];
        v.load(d.logits, row + j);
        v.get(f);
#pragma unroll
        for (int i = 0; i < 8; ++i) l[j + i] = f[i];
      }
    } else if constexpr (EPL == 4 && sizeof(T) == 4) {
      const float4 v = *reinterpret_cast<const float4*>(reinterpret_cast<const float*>(d.logits) + row);
      l[0] = v.x;
      l[1] = v.y;
      l[2] = v.z;
      l[3] = v.w;
    }
  } else {
#pragma unroll
    for (int j = 0; j < EPL; ++j) l[j] = sub * EPL + j < d.experts ? logit_at<T>(d.logits, row + j) : -kInf;
  }
  float bias[EPL];
  if constexpr (SCORED) {
    if (EPL % 4 == 0 && d.bias && d.experts == LPT * EPL) {
#pragma unroll
      for (int j = 0; j < EPL; j += 4) {
        const float4 v = *reinterpret_cast<const float4*>(d.bias + sub * EPL + j);
        bias[j] = v.x;
        bias[(j + 1) % EPL] = v.y;
        bias[(j + 2) % EPL] = v.z;
        bias[(j + 3) % EPL] = v.w;
      }
    } else {
#pragma unroll
      for (int j = 0; j < EPL; ++j) bias[j] = d.bias && sub * EPL + j < d.experts ? d.bias[sub * EPL + j] : 0.f;
    }
  }
#pragma unroll
  for (int j = 0; j < EPL; ++j) logits[sub * EPL + j] = l[j];
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
#pragma unroll
  for (int j = 0; j < EPL; ++j) mx = fmaxf(mx, l[j] != l[j] ? kInf : l[j]);    // a NaN as +inf: either makes every score of a softmax NaN
  mx = token_max<LPT>(mx);
  float inv = 0.f;
  const float shift = mx == -kInf ? 0.f : mx;
  if (!d.sigmoid && (SCORED || d.scores || !d.renormalize)) {
    float sum = 0.f;
#pragma unroll
    for (int j = 0; j < EPL; ++j) sum += expf(l[j] - shift);
    sum = token_sum<LPT>(sum);
    inv = sum == 0.f ? 0.f : 1.0f / sum;
  }
  if (d.scores && here) {
#pragma unroll
    for (int j = 0; j < EPL; ++j)
      if (sub * EPL + j < d.experts) d.scores[row + j] = d.sigmoid ? 1.0f / (1.0f + expf(-l[j])) : expf(l[j] - shift) * inv;
  }

  // values, and the groups that stay
  float v[EPL], off = 0.f, gap = kInf;
  bool sure = true;
  if constexpr (SCORED) {
    float most = 0.f;
#pragma unroll
    for (int j = 0; j < EPL; ++j) {
      const float x = __builtin_amdgcn_exp2f((d.sigmoid ? -l[j] : l[j] - shift) * 1.44269504f);
      const float p = (d.sigmoid ? __builtin_amdgcn_rcpf(1.0f + x) : x * inv) + bias[j];
      v[j] = l[j] == -kInf ? -kInf : p != p ? kInf : p;
      most = fmaxf(most, l[j] == -kInf ? 0.f : fabsf(p));
    }
    most = token_max<LPT>(most);
    // A sigmoid is off by at most 2^-22 (a third of a 2^-24 by the exponential's argument, half of one by itself, one by
    // the sum, two by the reciprocal), a softmax by 2^-18 of the largest score, which is inv (a sum of 256 besides); the
    // bias' sum by 2^-24 of what comes out.
    off = (d.sigmoid ? 0x1p-22f : 0x1p-18f * inv) + 0x1p-24f * most;
    if (d.top_groups < d.groups) {
      uint32_t in = keep_groups<LPT, EPL, float>(d, v, sub, reinterpret_cast<float*>(lds), gap);
      sure = gap > 4.0f * off + 0x1p-22f * most; // two sums of two values each, rounded
      const int lanes = group_lanes<LPT, EPL>(d);
      if (lanes > 0 && (d.sigmoid || !d.bias) && ballot64(!sure)) {
        // the groups again, by the exact values of each lane's two largest, if its third is surely below them
        float a = -kInf, b = -kInf, c = -kInf, la = -kInf, lb = -kInf, ba = 0.f, bb = 0.f;
#pragma unroll
        for (int j = 0; j < EPL; ++j) {
          const bool over = v[j] > a, next = v[j] > b;
          c = fmaxf(c, next ? b : v[j]);
          b = over ? a : next ? v[j] : b;
          lb = over ? la : next ? l[j] : lb;
          bb = over ? ba : next ? bias[j] : bb;
          a = over ? v[j] : a;
          la = over ? l[j] : la;
          ba = over ? bias[j] : ba;
        }
        auto exact = [&](float li, float bi) {
          const double x = exp((d.sigmoid ? -(double)li : (double)li - (double)shift));
          const double e = (d.sigmoid ? 1.0 / (1.0 + x) : x) + (double)bi;
          return li == -kInf ? -(double)kInf : e != e ? (double)kInf : e;
        };
        const int known = c == -kInf || b - c > 2.0f * off + 0x1p-23f * most;
        double far;
        const double ea = exact(la, ba), eb = exact(lb, bb);     // in their own order, which may be the other one
        in = run_stays<LPT, double>(d, maximum(ea, eb), ea < eb ? ea : eb, lanes, sub, far) ? 0xFFFFu : 0u;
        sure = token_min<LPT>(known) != 0;
      }
#pragma unroll
      for (int j = 0; j < EPL; ++j) v[j] = in >> j & 1u ? v[j] : -kInf;
    }
    if (!d.bias) {
      off = 0.f;
#pragma unroll
      for (int j = 0; j < EPL; ++j) v[j] = v[j] == -kInf ? -kInf : l[j] != l[j] ? kInf : l[j];
    }
  } else {
#pragma unroll
    for (int j = 0; j < EPL; ++j) v[j] = l[j] != l[j] ? kInf : l[j];
    if (d.top_groups < d.groups) {
      const uint32_t in = keep_groups<LPT, EPL, float>(d, v, sub, reinterpret_cast<float*>(lds), gap);
#pragma unroll
      for (int j = 0; j < EPL; ++j) v[j] = in >> j & 1u ? v[j] : -kInf;
    }
  }

  // the heads of the lanes' sorted lists, largest first
  constexpr int MASK = EXACT16 ? 0xFFFF : EPL - 1;
  constexpr float PLACE = EXACT16 || EPL == 1 ? 0.f : 2.0f * EPL * 0x1p-23f;   // what the lowest bits took from two values
  const int bottom = ordered(-kInf) & ~MASK;     // and below: not to be chosen
  int k[EPL];
#pragma unroll
  for (int j = 0; j < EPL; ++j) {
    const int place = EXACT16 ? LPT * EPL - 1 - (sub * EPL + j) : EPL - 1 - j;
    k[j] = v[j] == -kInf ? (int)0x80000000 : ((ordered(v[j]) & ~MASK) | place);
  }
  sort_lane<EPL>(k);
  int id = -1;
  if constexpr (EXACT16) {
    for (int s = 0; s < d.top_k; ++s) {
      const int top = token_max_i<LPT>(k[0]);
      if (sub == s && top > bottom) id = LPT * EPL - 1 - (top & MASK);
      leave<EPL>(k, k[0] == top);
    }
  } else {
    // whether a value is surely above the next one (an infinity or a NaN never is)
    auto above = [&](float a, float b) { return a - b > 2.0f * off + PLACE * fmaxf(fabsf(a), fabsf(b)); };
    const int turns = min(d.top_k + 2, LPT);
    float last = kInf, kth = -kInf;
    bool close = false;
    for (int s = 0; s < turns; ++s) {
      const int top = token_max_i<LPT>(k[0]);
      const bool any = top > bottom;
      const uint64_t who = ballot64(k[0] == top);
      const int first = LPT == 64 ? __ffsll((unsigned long long)who) - 1
                                  : __ffs((int)((uint32_t)(who >> (slot * LPT)) & (uint32_t)((1ull << (LPT & 63)) - 1))) - 1;
      if (sub == s && any) id = first * EPL + EPL - 1 - (top & MASK);
      const float now = unordered(top & ~MASK);
      close |= any && s > 0 && s <= d.top_k && !above(last, now);
      last = now;
      if (s == d.top_k - 1) kth = any ? now : -kInf;
      leave<EPL>(k, sub == first);
    }
    // the candidates hold the chosen ones if the last slot's value is surely above all that is left
    const int rest = token_max_i<LPT>(k[0]);
    sure &= rest <= bottom || above(kth, unordered(rest & ~MASK));
    if (ballot64(close)) {
      // the exact values, a candidate a lane, and how many come before each
      double x = -(double)kInf;
      if (id >= 0) {
        const float li = logits[id];
        x = li;
        if constexpr (SCORED) {
          if (d.bias && d.sigmoid) x = 1.0 / (1.0 + exp(-(double)li)) + (double)d.bias[id];
          else if (d.bias) x = exp((double)li - (double)shift);
        }
      }
      if constexpr (SCORED) {
        if (d.bias && !d.sigmoid) {
          double sum = 0.0;
#pragma unroll
          for (int j = 0; j < EPL; ++j) sum += exp((double)l[j] - (double)shift);
          sum = token_sum<LPT>(sum);
          if (id >= 0) x = x * (1.0 / sum) + (double)d.bias[id];
        }
      }
      if (x != x) x = kInf;
      int rank = 0;
      for (int c = 0; c < turns; ++c) {
        const double xc = __shfl(x, lane - sub + c, 64);
        const int ic = __shfl(id, lane - sub + c, 64);
        rank += ic >= 0 && (xc > x || (xc == x && ic < id)) ? 1 : 0;
      }
      int* order = reinterpret_cast<int*>(lds);
      if (id >= 0) order[rank] = id;
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
      __builtin_amdgcn_wave_barrier();
      if (id >= 0) id = order[sub];
    }
    if (ballot64(!sure)) {
      if constexpr (SCORED) {
        double k64[EPL], far, rinv = 1.0;
        if (d.sigmoid) {
#pragma unroll
          for (int j = 0; j < EPL; ++j) k64[j] = 1.0 / (1.0 + exp(-(double)l[j]));
        } else {
          double sum = 0.0;
#pragma unroll
          for (int j = 0; j < EPL; ++j) {
            k64[j] = exp((double)l[j] - (double)shift);
            sum += k64[j];
          }
          rinv = 1.0 / token_sum<LPT>(sum);
        }
        uint32_t in = 0xFFFFu;
#pragma unroll
        for (int j = 0; j < EPL; ++j) {
          const double w = k64[j] * rinv + (double)bias[j];
          k64[j] = l[j] == -kInf ? -(double)kInf : w != w ? (double)kInf : w;
        }
        if (d.top_groups < d.groups) in = keep_groups<LPT, EPL, double>(d, k64, sub, lds, far);
#pragma unroll
        for (int j = 0; j < EPL; ++j) {
          if (!d.bias) k64[j] = l[j] != l[j] ? (double)kInf : (double)l[j];
          k64[j] = in >> j & 1u ? k64[j] : -(double)kInf;
        }
        id = pick<LPT, EPL, double>(d, k64, sub);
      } else {
        id = pick<LPT, EPL, float>(d, v, sub);
      }
    }
  }
  const bool live = id >= 0 && sub < d.top_k;   // candidates beyond the slots fall away
  const float w = chosen_weight<LPT>(d, live, live ? logits[id] : 0.f, shift, inv);
  if (here && sub < d.top_k) {
    d.ids[t * d.top_k + sub] = id;
    d.weights[t * d.top_k + sub] = live ? w * d.scale : 0.f;
  }
}

// With p the scores, c the scale, g = dweights, w the weights over c:
//   chosen ones, renormalised:  dl_e = c w_e (g_e - <g, w>)         (softmax)
//                                    = c w_e (1 - p_e) (g_e - <g, w>)  (sigmoid)
//   otherwise and dscores: G = dscores + c g at the chosen;
//                          dl = p (G - <G, p>)                      (softmax)
//                             = G p (1 - p)                         (sigmoid)
template <typename T, int LPT, int EPL>
__global__ __launch_bounds__(256) void k_router_bwd(const RouterDesc d) {
  constexpr int TPW = 64 / LPT;
  const int lane = lane_id(), sub = lane % LPT, wave = threadIdx.x >> 6, slot = lane / LPT;
  const long long token = ((long long)blockIdx.y * gridDim.x + blockIdx.x) * (4 * TPW) + wave * TPW + slot;
  const bool here = token < d.m;
  const size_t t = here ? (size_t)token : (size_t)d.m - 1;
  float l[EPL], G[EPL];
  float mx = -kInf;
#pragma unroll
  for (int j = 0; j < EPL; ++j) {
    const int e = j * LPT + sub;
    const bool in = e < d.experts;
    l[j] = in ? logit_at<T>(d.logits, t * d.experts + e) : -kInf;
    G[j] = in && d.dscores ? d.dscores[t * d.experts + e] : 0.f;
    mx = fmaxf(mx, l[j] != l[j] ? kInf : l[j]);    // a NaN as +inf: either makes every score of a softmax NaN
  }
  int id = -1;
  float g = 0.f, lc = 0.f;
  if (sub < d.top_k) {
    id = d.ids_in[t * d.top_k + sub];
    g = d.dweights[t * d.top_k + sub];
  }
  const bool live = id >= 0 && id < d.experts;
  if (live) lc = logit_at<T>(d.logits, t * d.experts + id);
  mx = token_max<LPT>(mx);
  const float shift = mx == -kInf ? 0.f : mx;
  float p[EPL];
  if (d.sigmoid) {
#pragma unroll
    for (int j = 0; j < EPL; ++j) p[j] = 1.0f / (1.0f + expf(-l[j]));
  } else {
    float sum = 0.f;
#pragma unroll
    for (int j = 0; j < EPL; ++j) {
      p[j] = expf(l[j] - shift);
      sum += p[j];
    }
    sum = token_sum<LPT>(sum);
    const float inv = sum == 0.f ? 0.f : 1.0f / sum;
#pragma unroll
    for (int j = 0; j < EPL; ++j) p[j] *= inv;
  }
  // the chosen slots' part: of the scores (renormalised: of the logits)
  float part;
  if (d.renormalize) {
    const float w = chosen_weight<LPT>(d, live, lc, shift, 0.f);
    const float mean = token_sum<LPT>(live ? g * w : 0.f);
    part = live ? d.scale * w * (g - mean) : 0.f;
    if (d.sigmoid) part *= 1.0f / (1.0f + expf(lc));            // 1 - p
  } else {
    part = live ? d.scale * g : 0.f;
  }
  float add[EPL];
#pragma unroll
  for (int j = 0; j < EPL; ++j) add[j] = 0.f;
  for (int s = 0; s < d.top_k; ++s) {
    const int e = __shfl(live ? id : -1, lane - sub + s, 64);
    const float v = __shfl(part, lane - sub + s, 64);
#pragma unroll
    for (int j = 0; j < EPL; ++j)
      if (j * LPT + sub == e) add[j] += v;
  }
  if (!d.renormalize) {
#pragma unroll
    for (int j = 0; j < EPL; ++j) G[j] += add[j];
  }
  float mean = 0.f;
  if (!d.sigmoid) {
#pragma unroll
    for (int j = 0; j < EPL; ++j) mean = fmaf(G[j], p[j], mean);
    mean = token_sum<LPT>(mean);
  }
#pragma unroll
  for (int j = 0; j < EPL; ++j) {
    const int e = j * LPT + sub;
    float v = d.sigmoid ? G[j] * p[j] * (1.0f / (1.0f + expf(l[j]))) : p[j] * (G[j] - mean);
    if (d.renormalize) v += add[j];
    if (here && e < d.experts) {
      if constexpr (sizeof(T) == 2) reinterpret_cast<uint16_t*>(d.dlogits)[t * d.experts + e] = (uint16_t)pack_bf16(v, 0.f);
      else reinterpret_cast<float*>(d.dlogits)[t * d.experts + e] = v;
    }
  }
}

template <typename T, int LPT, int EPL>
static hipError_t go(const RouterDesc& d, bool fwd, hipStream_t s) {
  constexpr int TPB = 4 * 64 / LPT;
  const dim3 grid = grid2(((long long)d.m + TPB - 1) / TPB);
  if constexpr (LPT < 64) {
    if (!fwd) {
      ffn_launch((k_router_bwd<T, LPT, EPL>), grid, dim3(256), 0, s, d);
      return hipGetLastError();
    }
  }
  if (d.bias || (d.group_best == 2 && d.top_groups < d.groups)) ffn_launch((k_router_fwd<T, LPT, EPL, true>), grid, dim3(256), 0, s, d);
  else ffn_launch((k_router_fwd<T, LPT, EPL, false>), grid, dim3(256), 0, s, d);
  return hipGetLastError();
}
// Up to this many tokens a wave takes one token of more than 128 experts, four registers a lane: the shorter way through;
// with more of them four tokens, which leaves fewer waves to a SIMD. One token, 512, 1024, 4096 of 256 experts: 5.9, 6.1, 6.9,
// 9.9 us one a wave, 6.3, 7.6, 7.9, 8.0 four a wave; of 128 experts 5.7, 5.9, 6.3, 9.4 and 5.4, 6.1, 6.5, 6.9.
constexpr int kWideTokens = 1024;
// Otherwise a token has 16 lanes (8 for as few experts), and its experts so many registers of each.
template <typename T>
static hipError_t by_experts(const RouterDesc& d, bool fwd, hipStream_t s) {
  if (d.experts <= 8) return go<T, 8, 1>(d, fwd, s);
  if (d.experts <= 16) return go<T, 16, 1>(d, fwd, s);
  if (d.experts <= 32) return go<T, 16, 2>(d, fwd, s);
  if (d.experts <= 64) return go<T, 16, 4>(d, fwd, s);
  if (d.experts <= 128) return go<T, 16, 8>(d, fwd, s);
  if (d.m <= kWideTokens && fwd) return go<T, 64, 4>(d, fwd, s);
  return go<T, 16, 16>(d, fwd, s);
}
hipError_t launch_router_fwd(const RouterDesc& d, hipStream_t s) {
  return d.dtype == DT_BF16 ? by_experts<uint16_t>(d, true, s) : by_experts<float>(d, true, s);
}
hipError_t launch_router_bwd(const RouterDesc& d, hipStream_t s) {
  return d.dtype == DT_BF16 ? by_experts<uint16_t>(d, false, s) : by_experts<float>(d, false, s);
}

}  // namespace ffn
