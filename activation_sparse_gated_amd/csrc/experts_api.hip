// C ABI of routing to experts (include/ffn_experts.h): argument checks and
// launches. The calls keep no state.
#include <hip/hip_runtime.h>

#include <cmath>

#include "../../include/ffn_experts.h"
#include "experts.cuh"

using namespace ffn;

static_assert(kRowsMaxGroups == FFN_ROWS_MAX_GROUPS, "one limit");

namespace {

bool al16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool need(const void* p) { return p && al16(p); }
bool opt(const void* p) { return al16(p); }
bool flag_ok(int32_t f) { return f == 0 || f == 1; }
bool dtype_ok(int32_t t) { return t == FFN_F32 || t == FFN_BF16; }
ffn_status done(hipError_t e) { return e == hipSuccess ? FFN_OK : FFN_E_HIP; }
hipStream_t st(void* stream) { return reinterpret_cast<hipStream_t>(stream); }

constexpr long long kMaxRows = 0x7FFF0000;
constexpr int kMaxWidth = 1 << 22;
constexpr int kMaxEntries = 1 << 24;

bool route_ok(int32_t dtype, int32_t m, int32_t experts, int32_t top_k, int32_t score, int32_t renormalize, float scale) {
  return dtype_ok(dtype) && m >= 0 && experts >= 1 && experts <= FFN_ROUTE_MAX_EXPERTS && top_k >= 1 &&
         top_k <= FFN_ROUTE_MAX_TOP_K && top_k <= experts && (long long)m * top_k <= kMaxRows &&
         (score == FFN_ROUTE_SOFTMAX || score == FFN_ROUTE_SIGMOID) && flag_ok(renormalize) && std::isfinite(scale);
}
bool rows_ok(int32_t dtype, int32_t m, int32_t d, int32_t top_k) {
  return dtype_ok(dtype) && m >= 0 && top_k >= 1 && top_k <= FFN_ROUTE_MAX_TOP_K && (long long)m * top_k <= kMaxRows &&
         d >= 8 && d % 8 == 0 && d <= kMaxWidth;
}
RowsDesc rows_desc(int32_t dtype, int32_t m, int32_t d, const int32_t* slots, int32_t top_k) {
  RowsDesc r{};
  r.dtype = dtype;
  r.m = m;
  r.d = d;
  r.slots = slots;
  r.top_k = top_k;
  return r;
}

}  // namespace

extern "C" {

int32_t ffn_experts_abi_version(void) { return FFN_EXPERTS_ABI_VERSION; }

ffn_status ffn_route_forward(const void* logits, int32_t dtype, int32_t m, int32_t experts, int32_t top_k, int32_t score,
                             const float* bias, int32_t groups, int32_t top_groups, int32_t group_best,
                             int32_t renormalize, float scale, float* weights, int32_t* ids, float* scores, void* stream) {
  if (!route_ok(dtype, m, experts, top_k, score, renormalize, scale)) return FFN_E_INVALID;
  if (groups < 1 || groups > FFN_ROUTE_MAX_GROUPS || experts % groups != 0 || top_groups < 1 || top_groups > groups ||
      (group_best != 1 && group_best != 2))
    return FFN_E_INVALID;
  if (m == 0) return FFN_OK;
  if (!need(logits) || !opt(bias) || !need(weights) || !need(ids) || !opt(scores)) return FFN_E_INVALID;
  RouterDesc d{};
  d.logits = logits;
  d.dtype = dtype;
  d.m = m;
  d.experts = experts;
  d.top_k = top_k;
  d.sigmoid = score == FFN_ROUTE_SIGMOID;
  d.groups = groups;
  d.top_groups = top_groups;
  d.group_best = group_best;
  d.renormalize = renormalize;
  d.scale = scale;
  d.bias = bias;
  d.weights = weights;
  d.ids = ids;
  d.scores = scores;
  return done(launch_router_fwd(d, st(stream)));
}

ffn_status ffn_route_backward(const void* logits, int32_t dtype, int32_t m, int32_t experts, int32_t top_k, int32_t score,
                              int32_t renormalize, float scale, const int32_t* ids, const float* dweights,
                              const float* dscores, void* dlogits, void* stream) {
  if (!route_ok(dtype, m, experts, top_k, score, renormalize, scale)) return FFN_E_INVALID;
  if (m == 0) return FFN_OK;
  if (!need(logits) || !need(ids) || !need(dweights) || !opt(dscores) || !need(dlogits)) return FFN_E_INVALID;
  RouterDesc d{};
  d.logits = logits;
  d.dtype = dtype;
  d.m = m;
  d.experts = experts;
  d.top_k = top_k;
  d.sigmoid = score == FFN_ROUTE_SIGMOID;
  d.renormalize = renormalize;
  d.scale = scale;
  d.ids_in = ids;
  d.dweights = dweights;
  d.dscores = dscores;
  d.dlogits = dlogits;
  return done(launch_router_bwd(d, st(stream)));
}

size_t ffn_group_rows_workspace_bytes(int32_t n, int32_t groups) {
  if (n < 0 || n > kMaxEntries || groups < 1 || groups > FFN_ROWS_MAX_GROUPS) return 0;
  const int blocks = group_rows_blocks(n);
  return blocks > 1 ? (size_t)blocks * (groups + 1) * 4 : 0;
}

ffn_status ffn_group_rows(const int32_t* ids, int32_t n, int32_t groups, int32_t* offsets, int32_t* rows, int32_t* slots,
                          void* workspace, size_t workspace_bytes, void* stream) {
  if (n < 0 || groups < 1 || groups > FFN_ROWS_MAX_GROUPS || !need(offsets)) return FFN_E_INVALID;
  if (n > kMaxEntries) return FFN_E_UNSUPPORTED;
  if (n == 0) return done(launch_fill_u32(reinterpret_cast<uint32_t*>(offsets), 0u, groups + 1, st(stream)));
  if (!need(ids) || !opt(rows) || !opt(slots) || !opt(workspace)) return FFN_E_INVALID;
  const size_t bytes = ffn_group_rows_workspace_bytes(n, groups);
  if (bytes && !workspace) return FFN_E_INVALID;
  if (workspace_bytes < bytes) return FFN_E_WORKSPACE;
  GroupDesc d{};
  d.ids = ids;
  d.n = n;
  d.groups = groups;
  d.offsets = offsets;
  d.rows = rows;
  d.slots = slots;
  d.hist = static_cast<uint32_t*>(workspace);
  return done(launch_group_rows(d, st(stream)));
}

ffn_status ffn_gather_forward(const void* x, int32_t dtype, int32_t m, int32_t d, const int32_t* slots, int32_t top_k,
                              void* y, uint8_t* q, float* scale, void* stream) {
  if (!rows_ok(dtype, m, d, top_k)) return FFN_E_INVALID;
  if (m == 0) return FFN_OK;
  if (!need(x) || !need(slots) || !opt(y) || !opt(q) || !opt(scale) || (!y && !q) || (q != nullptr) != (scale != nullptr))
    return FFN_E_INVALID;
  RowsDesc r = rows_desc(dtype, m, d, slots, top_k);
  r.x = x;
  r.y = y;
  r.q = q;
  r.scale = scale;
  return done(launch_gather(r, st(stream)));
}

ffn_status ffn_combine_forward(const void* y, int32_t dtype, int32_t m, int32_t d, const int32_t* slots, int32_t top_k,
                               const float* weights, const void* residual, void* out, void* stream) {
  if (!rows_ok(dtype, m, d, top_k)) return FFN_E_INVALID;
  if (m == 0) return FFN_OK;
  if (!need(y) || !need(slots) || !opt(weights) || !opt(residual) || !need(out)) return FFN_E_INVALID;
  RowsDesc r = rows_desc(dtype, m, d, slots, top_k);
  r.x = y;
  r.weights = weights;
  r.residual = residual;
  r.y = out;
  return done(launch_combine_fwd(r, st(stream)));
}

ffn_status ffn_combine_backward(const void* y, int32_t dtype, int32_t m, int32_t d, const int32_t* slots, int32_t top_k,
                                const float* weights, const void* dout, void* dy, float* dweights, void* stream) {
  if (!rows_ok(dtype, m, d, top_k)) return FFN_E_INVALID;
  if (m == 0) return FFN_OK;
  if (!opt(y) || !need(slots) || !opt(weights) || !need(dout) || !opt(dy) || !opt(dweights) || (!dy && !dweights) ||
      (dweights && !y))
    return FFN_E_INVALID;
  RowsDesc r = rows_desc(dtype, m, d, slots, top_k);
  r.x = y;
  r.weights = weights;
  r.dout = dout;
  r.y = dy;
  r.dweights = dweights;
  return done(launch_combine_bwd(r, st(stream)));
}

}  // extern "C"
