// The router on gfx950: scores of a token's experts, the choice of the best,
// their weights, and the gradient.
//
// LPT lanes hold a token's logits (expert j * LPT + lane in register j), so a
// wave has 64 / LPT tokens and everything between the load and the result stays
// in registers: sums and maxima over a token are lane moves. The top k are k
// turns of a maximum over (value, lower index first), the winner leaving.
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
// The largest value and its index, the lower one of equals.
template <int O, typename V>
__device__ __forceinline__ void best_with(V& v, int& e) {
  const V ov = xchg<O>(v);
  const int oe = wave_xchg_i<O>(e);
  const bool take = ov > v || (ov == v && oe < e);
  v = take ? ov : v;
  e = take ? oe : e;
}
template <int LPT, typename V>
__device__ __forceinline__ void token_best(V& v, int& e) {
  if constexpr (LPT > 32) best_with<32>(v, e);
  if constexpr (LPT > 16) best_with<16>(v, e);
  if constexpr (LPT > 8) best_with<8>(v, e);
  best_with<4>(v, e);
  best_with<2>(v, e);
  best_with<1>(v, e);
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

// Key: fp32 where the logits themselves decide, fp64 where scores do.
template <typename T, int LPT, int EPL, typename Key>
__global__ __launch_bounds__(256) void k_router_fwd(const RouterDesc d) {
  constexpr int TPW = 64 / LPT;
  constexpr int GPL = (32 + LPT - 1) / LPT;      // groups of a lane
  __shared__ Key s_key[4][TPW][LPT * EPL];
  const int lane = lane_id(), sub = lane % LPT, wave = threadIdx.x >> 6, slot = lane / LPT;
  const long long token = ((long long)blockIdx.y * gridDim.x + blockIdx.x) * (4 * TPW) + wave * TPW + slot;
  const bool here = token < d.m;
  const size_t t = here ? (size_t)token : (size_t)d.m - 1;      // the last token again: lanes stay together
  float l[EPL];
  float mx = -kInf;
#pragma unroll
  for (int j = 0; j < EPL; ++j) {
    const int e = j * LPT + sub;
    l[j] = e < d.experts ? logit_at<T>(d.logits, t * d.experts + e) : -kInf;
    mx = fmaxf(mx, l[j] != l[j] ? kInf : l[j]);    // a NaN as +inf: either makes every score of a softmax NaN
  }
  mx = token_max<LPT>(mx);
  float inv = 0.f;
  const float shift = mx == -kInf ? 0.f : mx;
  if (!d.sigmoid && (d.scores || !d.renormalize)) {
    float sum = 0.f;
#pragma unroll
    for (int j = 0; j < EPL; ++j) sum += expf(l[j] - shift);
    sum = token_sum<LPT>(sum);
    inv = sum == 0.f ? 0.f : 1.0f / sum;
  }
  if (d.scores && here) {
#pragma unroll
    for (int j = 0; j < EPL; ++j) {
      const int e = j * LPT + sub;
      if (e < d.experts) d.scores[t * d.experts + e] = d.sigmoid ? 1.0f / (1.0f + expf(-l[j])) : expf(l[j] - shift) * inv;
    }
  }
  Key key[EPL];
  if constexpr (sizeof(Key) == 4) {
#pragma unroll
    for (int j = 0; j < EPL; ++j) key[j] = l[j] != l[j] ? kInf : l[j];
  } else {
    double rinv = 1.0;
    if (d.sigmoid) {
#pragma unroll
      for (int j = 0; j < EPL; ++j) key[j] = 1.0 / (1.0 + exp(-(double)l[j]));
    } else {
      double sum = 0.0;
#pragma unroll
      for (int j = 0; j < EPL; ++j) {
        key[j] = exp((double)l[j] - (double)shift);
        sum += key[j];
      }
      sum = token_sum<LPT>(sum);
      rinv = 1.0 / sum;
    }
#pragma unroll
    for (int j = 0; j < EPL; ++j) {
      const int e = j * LPT + sub;
      const double v = key[j] * rinv + (d.bias && e < d.experts ? (double)d.bias[e] : 0.0);
      key[j] = l[j] == -kInf ? -(double)kInf : v != v ? (double)kInf : v;
    }
  }
  if (d.top_groups < d.groups) {
    const int size = d.experts / d.groups;
    Key* mine = s_key[wave][slot];
#pragma unroll
    for (int j = 0; j < EPL; ++j) mine[j * LPT + sub] = key[j];
    __syncthreads();
    Key gv[GPL];
#pragma unroll
    for (int i = 0; i < GPL; ++i) {
      const int g = i * LPT + sub;
      Key a = -(Key)kInf, b = -(Key)kInf;
      if (g < d.groups) {
        int at = g % size;                       // lanes start apart: their groups lie in the same banks
        for (int n = 0; n < size; ++n) {
          const Key v = mine[g * size + at];
          b = v > a ? a : v > b ? v : b;
          a = v > a ? v : a;
          at = at + 1 == size ? 0 : at + 1;
        }
      }
      gv[i] = d.group_best == 2 && b != -(Key)kInf ? a + b : a;
    }
    uint32_t keep = 0;
    for (int n = 0; n < d.top_groups; ++n) {
      Key v = -(Key)kInf;
      int g = 0x7FFFFFFF;
#pragma unroll
      for (int i = 0; i < GPL; ++i) {
        if (gv[i] > v) {
          v = gv[i];
          g = i * LPT + sub;
        }
      }
      token_best<LPT>(v, g);
      if (g < 32) keep |= 1u << g;
#pragma unroll
      for (int i = 0; i < GPL; ++i)
        if (i * LPT + sub == g) gv[i] = -(Key)kInf;
    }
    const uint32_t rsize = (65536 + size - 1) / size;           // e / size for e, size <= 256
#pragma unroll
    for (int j = 0; j < EPL; ++j) {
      const int g = (int)((uint32_t)(j * LPT + sub) * rsize >> 16);
      if (g > 31 || !(keep >> g & 1u)) key[j] = -(Key)kInf;
    }
  }
  int id = -1;
  for (int s = 0; s < d.top_k; ++s) {
    Key v = -(Key)kInf;
    int e = 0x7FFFFFFF;
#pragma unroll
    for (int j = 0; j < EPL; ++j) {
      if (key[j] > v) {
        v = key[j];
        e = j * LPT + sub;
      }
    }
    token_best<LPT>(v, e);
    if (sub == s) id = e == 0x7FFFFFFF ? -1 : e;
#pragma unroll
    for (int j = 0; j < EPL; ++j)
      if (j * LPT + sub == e) key[j] = -(Key)kInf;
  }
  const bool live = id >= 0;
  const float w = chosen_weight<LPT>(d, live, live ? logit_at<T>(d.logits, t * d.experts + id) : 0.f, shift, inv);
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
  if (!fwd) ffn_launch((k_router_bwd<T, LPT, EPL>), grid, dim3(256), 0, s, d);
  else if (d.bias || (d.group_best == 2 && d.top_groups < d.groups)) ffn_launch((k_router_fwd<T, LPT, EPL, double>), grid, dim3(256), 0, s, d);
  else ffn_launch((k_router_fwd<T, LPT, EPL, float>), grid, dim3(256), 0, s, d);
  return hipGetLastError();
}
template <typename T>
static hipError_t by_experts(const RouterDesc& d, bool fwd, hipStream_t s) {
  if (d.experts <= 8) return go<T, 8, 1>(d, fwd, s);
  if (d.experts <= 16) return go<T, 16, 1>(d, fwd, s);
  if (d.experts <= 32) return go<T, 16, 2>(d, fwd, s);
  if (d.experts <= 64) return go<T, 16, 4>(d, fwd, s);
  if (d.experts <= 128) return go<T, 16, 8>(d, fwd, s);
  return go<T, 16, 16>(d, fwd, s);
}
hipError_t launch_router_fwd(const RouterDesc& d, hipStream_t s) {
  return d.dtype == DT_BF16 ? by_experts<uint16_t>(d, true, s) : by_experts<float>(d, true, s);
}
hipError_t launch_router_bwd(const RouterDesc& d, hipStream_t s) {
  return d.dtype == DT_BF16 ? by_experts<uint16_t>(d, false, s) : by_experts<float>(d, false, s);
}

}  // namespace ffn
