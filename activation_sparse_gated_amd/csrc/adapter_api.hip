// C ABI of the low-rank adapters (include/ffn_adapter.h): argument checks and
// launches. The calls keep no state.
#include <hip/hip_runtime.h>

#include "../../include/ffn_adapter.h"
#include "adapter.cuh"

using namespace ffn;

static_assert(kAdapterMaxGroups == FFN_ADAPTER_MAX_GROUPS && kAdapterMaxRank == FFN_ADAPTER_MAX_RANK, "one limit");

namespace {

bool al16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool need(const void* p) { return p && al16(p); }
bool opt(const void* p) { return al16(p); }
bool flag_ok(int32_t f) { return f == 0 || f == 1; }
bool dtype_ok(int32_t t) { return t == FFN_F32 || t == FFN_BF16; }
ffn_status done(hipError_t e) { return e == hipSuccess ? FFN_OK : FFN_E_HIP; }
hipStream_t st(void* stream) { return reinterpret_cast<hipStream_t>(stream); }

constexpr int kMaxRows = 1 << 26;    // tiles of 16 or more rows and their workgroups stay within a grid's 2^32 threads
constexpr int kMaxWidth = 1 << 22;

bool shape_ok(int32_t m, int32_t n, int32_t k, int32_t r, int32_t groups) {
  return m >= 0 && m <= kMaxRows && n >= 8 && n % 8 == 0 && n <= kMaxWidth && k >= 8 && k % 8 == 0 && k <= kMaxWidth &&
         r >= 8 && r % 8 == 0 && r <= FFN_ADAPTER_MAX_RANK && groups >= 1 && groups <= FFN_ADAPTER_MAX_GROUPS;
}
size_t up256(size_t b) { return (b + 255) / 256 * 256; }
size_t tab_bytes(const AdapterPlan& p) { return up256((size_t)p.tiles * 16); }
size_t h_bytes(const AdapterPlan& p, int32_t r) { return up256((size_t)p.ks * p.tiles * p.rt * r * 4); }
size_t dh_bytes(const AdapterPlan& p, int32_t r) { return up256((size_t)p.kd * p.tiles * p.rt * r * 4); }
size_t parts_bytes(const AdapterPlan& p, int32_t r) { return up256((size_t)p.tiles * p.rt * r * 6); }
size_t forward_bytes(const AdapterPlan& p, int32_t r) {
  return p.few ? 0 : tab_bytes(p) + h_bytes(p, r) + (p.rt == 64 ? parts_bytes(p, r) : 0);
}
size_t backward_bytes(const AdapterPlan& p, int32_t r) {
  return tab_bytes(p) + h_bytes(p, r) + dh_bytes(p, r) + 3 * parts_bytes(p, r) + (p.slices > 1 ? p.slices * p.part * 4 : 0);
}

}  // namespace

extern "C" {

int32_t ffn_adapter_abi_version(void) { return FFN_ADAPTER_ABI_VERSION; }

size_t ffn_adapter_forward_workspace_bytes(int32_t m, int32_t n, int32_t k, int32_t r, int32_t groups) {
  if (!shape_ok(m, n, k, r, groups) || m == 0) return 0;
  const AdapterPlan p = adapter_plan(m, n, k, r, groups, false);
  return forward_bytes(p, r);
}

ffn_status ffn_adapter_forward(const void* x, const void* a, const void* b, const float* scales, const int32_t* offsets,
                               const int32_t* rows, int32_t groups, int32_t m, int32_t n, int32_t k, int32_t r,
                               const void* base, void* y, int32_t y_dtype, void* workspace, size_t workspace_bytes,
                               void* stream) {
  if (!shape_ok(m, n, k, r, groups) || !dtype_ok(y_dtype)) return FFN_E_INVALID;
  if (m == 0) return FFN_OK;
  if (!need(x) || !need(a) || !need(b) || !opt(scales) || !need(offsets) || !opt(rows) || !opt(base) || !need(y) ||
      !opt(workspace))
    return FFN_E_INVALID;
  AdapterDesc d{};
  d.p = adapter_plan(m, n, k, r, groups, false);
  if (forward_bytes(d.p, r) && !workspace) return FFN_E_INVALID;
  if (workspace_bytes < forward_bytes(d.p, r)) return FFN_E_WORKSPACE;
  d.x = static_cast<const uint16_t*>(x);
  d.a = static_cast<const uint16_t*>(a);
  d.b = static_cast<const uint16_t*>(b);
  d.scales = scales;
  d.offsets = offsets;
  d.rows = rows;
  d.groups = groups;
  d.m = m;
  d.n = n;
  d.k = k;
  d.r = r;
  d.base = base;
  d.out = y;
  d.out_f32 = y_dtype == FFN_F32;
  if (!d.p.few) {
    d.tab = static_cast<int4*>(workspace);
    d.h = reinterpret_cast<float*>(static_cast<char*>(workspace) + tab_bytes(d.p));
    if (d.p.rt == 64) d.hp = reinterpret_cast<uint16_t*>(reinterpret_cast<char*>(d.h) + h_bytes(d.p, r));
  }
  return done(launch_adapter_forward(d, st(stream)));
}

size_t ffn_adapter_backward_workspace_bytes(int32_t m, int32_t n, int32_t k, int32_t r, int32_t groups) {
  if (!shape_ok(m, n, k, r, groups) || m == 0) return 0;
  const AdapterPlan p = adapter_plan(m, n, k, r, groups, true);
  return backward_bytes(p, r);
}

ffn_status ffn_adapter_backward(const void* x, const void* a, const void* b, const float* scales, const void* dy,
                                const int32_t* offsets, const int32_t* rows, int32_t groups, int32_t m, int32_t n,
                                int32_t k, int32_t r, const void* base, void* dx, float* da, float* db,
                                int32_t accumulate, void* workspace, size_t workspace_bytes, void* stream) {
  if (!shape_ok(m, n, k, r, groups) || !flag_ok(accumulate) || !opt(da) || !opt(db)) return FFN_E_INVALID;
  if (m == 0) {
    if (accumulate) return FFN_OK;
    hipError_t e = hipSuccess;
    if (da) e = launch_fill_u32(reinterpret_cast<uint32_t*>(da), 0u, (size_t)groups * r * k, st(stream));
    if (db && e == hipSuccess) e = launch_fill_u32(reinterpret_cast<uint32_t*>(db), 0u, (size_t)groups * n * r, st(stream));
    return done(e);
  }
  if (!need(dy) || !need(offsets) || !opt(x) || !opt(a) || !opt(b) || !opt(scales) || !opt(rows) || !opt(base) ||
      !opt(dx) || !need(workspace))
    return FFN_E_INVALID;
  const bool with_dh = dx || da, with_h = db != nullptr;
  if ((!with_dh && !with_h) || (base && !dx) || ((da || db) && !x) || ((dx || db) && !a) || (with_dh && !b)) return FFN_E_INVALID;
  AdapterDesc d{};
  d.p = adapter_plan(m, n, k, r, groups, true);
  if (workspace_bytes < backward_bytes(d.p, r)) return FFN_E_WORKSPACE;
  d.x = static_cast<const uint16_t*>(x);
  d.dy = static_cast<const uint16_t*>(dy);
  d.a = static_cast<const uint16_t*>(a);
  d.b = static_cast<const uint16_t*>(b);
  d.scales = scales;
  d.offsets = offsets;
  d.rows = rows;
  d.groups = groups;
  d.m = m;
  d.n = n;
  d.k = k;
  d.r = r;
  d.base = base;
  d.out = dx;
  d.da = da;
  d.db = db;
  d.accumulate = accumulate;
  d.tab = static_cast<int4*>(workspace);
  char* at = static_cast<char*>(workspace) + tab_bytes(d.p);
  if (with_h) d.h = reinterpret_cast<float*>(at);
  at += h_bytes(d.p, r);
  if (with_dh) d.dh = reinterpret_cast<float*>(at);
  at += dh_bytes(d.p, r);
  if (db) d.ht = reinterpret_cast<uint16_t*>(at);
  if (da) d.dht = reinterpret_cast<uint16_t*>(at + parts_bytes(d.p, r));
  if (dx) d.dhp = reinterpret_cast<uint16_t*>(at + 2 * parts_bytes(d.p, r));
  if (d.p.slices > 1) d.part = reinterpret_cast<float*>(at + 3 * parts_bytes(d.p, r));
  return done(launch_adapter_backward(d, st(stream)));
}

}  // extern "C"
