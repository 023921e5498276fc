// C ABI of the operators around the FFN (include/ffn_linear.h): argument
// checks and launches. The calls keep no state.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>

#include "../../include/ffn_linear.h"
#include "linear.cuh"

using namespace ffn;

namespace {

bool al16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
// A pointer that has to be there, and one that may be null.
bool need(const void* p) { return p && al16(p); }
bool opt(const void* p) { return al16(p); }
bool dtype_ok(int32_t t) { return t == FFN_F32 || t == FFN_BF16; }
bool flag_ok(int32_t f) { return f == 0 || f == 1; }
ffn_status done(hipError_t e) { return e == hipSuccess ? FFN_OK : FFN_E_HIP; }
hipStream_t st(void* stream) { return reinterpret_cast<hipStream_t>(stream); }

constexpr int kMaxRowTiles = 1 << 30;
constexpr int kMaxWidth = 1 << 22;   // 256 rows of it stay within 32-bit byte offsets
constexpr int kMaxRows = 0x7FFF0000; // a row's number and a few tiles more stay within 32 bits

bool norm_shape_ok(int32_t dtype, int32_t m, int32_t d, float eps) {
  return dtype_ok(dtype) && m >= 0 && m <= kMaxRows && d >= 8 && d % 8 == 0 && d <= 16384 && std::isfinite(eps) && eps >= 0.f;
}
// Tiles of the largest grid any kernel makes for this product, in workgroups.
bool product_shape_ok(int32_t m, int32_t n, int32_t k, int32_t groups) {
  if (m < 0 || m > kMaxRows || n < 1 || k < 1 || groups < 1 || groups > FFN_LINEAR_MAX_GROUPS) return false;
  if (n > kMaxWidth || k > kMaxWidth) return false;
  const long long rt = m / 16 + groups, ct = n / 16 + 1, kt = k / 16 + 1;
  return rt * ct < kMaxRowTiles && ct * kt * groups < kMaxRowTiles && rt * kt < kMaxRowTiles;
}

}  // namespace

extern "C" {

int32_t ffn_linear_abi_version(void) { return FFN_LINEAR_ABI_VERSION; }

ffn_status ffn_rmsnorm_forward(const void* x, const void* residual, const void* w, int32_t dtype, int32_t m,
                               int32_t d, float eps, void* r_out, void* y, uint8_t* q, float* scale, void* stream) {
  if (!norm_shape_ok(dtype, m, d, eps)) return FFN_E_INVALID;
  if (m == 0) return FFN_OK;
  if (!need(x) || !need(w) || !opt(residual) || !opt(r_out) || !opt(y) || !opt(q) || !opt(scale)) return FFN_E_INVALID;
  if ((!y && !q) || (q != nullptr) != (scale != nullptr) || (residual && !r_out)) return FFN_E_INVALID;
  NormDesc n{};
  n.x = x;
  n.res = residual;
  n.w = w;
  n.dtype = dtype;
  n.m = m;
  n.d = d;
  n.eps = eps;
  n.r_out = r_out;
  n.y = y;
  n.q = q;
  n.scale = scale;
  return done(launch_rmsnorm_fwd(n, st(stream)));
}

size_t ffn_rmsnorm_backward_workspace_bytes(int32_t m, int32_t d) {
  if (!norm_shape_ok(FFN_F32, m, d, 0.f)) return 0;
  return (size_t)rmsnorm_bwd_parts(m, d) * d * 4 + 16;
}

ffn_status ffn_rmsnorm_backward(const void* r, const void* w, const void* dy, const void* dr, int32_t dtype, int32_t m,
                                int32_t d, float eps, void* dx, float* dw, int32_t accumulate, void* workspace,
                                size_t workspace_bytes, void* stream) {
  if (!norm_shape_ok(dtype, m, d, eps) || !flag_ok(accumulate) || !opt(dw)) return FFN_E_INVALID;
  if (m == 0) {
    if (!dw || accumulate) return FFN_OK;
    return done(launch_fill_u32(reinterpret_cast<uint32_t*>(dw), 0u, d, st(stream)));
  }
  if (!need(r) || !need(w) || !need(dy) || !opt(dr) || !opt(dx) || (!dx && !dw)) return FFN_E_INVALID;
  if (dw) {
    if (!need(workspace)) return FFN_E_INVALID;
    if (workspace_bytes < ffn_rmsnorm_backward_workspace_bytes(m, d)) return FFN_E_WORKSPACE;
  }
  NormDesc n{};
  n.x = r;
  n.res = dx ? dr : nullptr;                     // dr reaches dx alone: not read without it
  n.w = w;
  n.dy = dy;
  n.dtype = dtype;
  n.m = m;
  n.d = d;
  n.eps = eps;
  n.dx = dx;
  n.dw = dw;
  n.part = static_cast<float*>(workspace);
  n.parts = rmsnorm_bwd_parts(m, d);
  n.accumulate = accumulate;
  return done(launch_rmsnorm_bwd(n, st(stream)));
}

ffn_status ffn_fp8_quantize(const void* x, int32_t dtype, int32_t groups, int32_t m, int32_t k, int32_t block_rows,
                            uint8_t* q, float* scale, uint8_t* qt, float* scale_t, void* stream) {
  if (!dtype_ok(dtype) || groups < 1 || m < 0 || k < 16 || k % 16 != 0 || (block_rows != 1 && block_rows != 128))
    return FFN_E_INVALID;
  if (m > kMaxRows || k > kMaxRows) return FFN_E_UNSUPPORTED;
  // a grid holds fewer than 2^32 threads: 256 for each tile
  const long long tiles = (long long)((k + 127) / 128) * ((m + 127) / 128);
  if (tiles >= 1 << 24 || tiles * groups >= 1 << 24) return FFN_E_UNSUPPORTED;
  if (m == 0) return FFN_OK;
  if (!need(x) || !need(q) || !need(scale) || !opt(qt) || !opt(scale_t) || (qt != nullptr) != (scale_t != nullptr))
    return FFN_E_INVALID;
  QuantDesc d{};
  d.x = x;
  d.dtype = dtype;
  d.groups = groups;
  d.m = m;
  d.k = k;
  d.block_rows = block_rows;
  d.q = q;
  d.scale = scale;
  d.qt = qt;
  d.scale_t = scale_t;
  d.mt = (m + 15) / 16 * 16;
  return done(launch_fp8_quant(d, st(stream)));
}

size_t ffn_fp8_linear_workspace_bytes(int32_t m, int32_t n, int32_t k, int32_t groups) {
  if (!product_shape_ok(m, n, k, groups) || m == 0) return 0;
  return std::max(lin_workspace(lin_plan(LIN_FP8, 0, m, n, k, groups), m, n),
                  lin_workspace(lin_plan(LIN_FP8, 1, m, n, k, groups), m, n));
}

ffn_status ffn_fp8_linear(const uint8_t* x, const float* x_scale, const uint8_t* w, const float* w_scale,
                          int32_t w_block_rows, int32_t m, int32_t n, int32_t k, const int32_t* offsets, int32_t groups,
                          void* y, int32_t y_dtype, int32_t accumulate, void* workspace, size_t workspace_bytes,
                          void* stream) {
  if (!product_shape_ok(m, n, k, groups) || k % 16 != 0 || !dtype_ok(y_dtype) || !flag_ok(accumulate) ||
      (w_block_rows != 1 && w_block_rows != 128))
    return FFN_E_INVALID;
  if (!offsets && groups != 1) return FFN_E_INVALID;
  if ((offsets && w_block_rows != 128) || (accumulate && y_dtype != FFN_F32)) return FFN_E_UNSUPPORTED;
  if (m == 0) return FFN_OK;
  if (!need(x) || !need(x_scale) || !need(w) || !need(w_scale) || !opt(offsets) || !need(y) || !opt(workspace))
    return FFN_E_INVALID;
  LinDesc d{};
  d.kind = LIN_FP8;
  d.A = w;
  d.B = x;
  d.rows = m;
  d.cols = n;
  d.K = k;
  d.a_group = (long long)n * k;
  d.offsets = offsets;
  d.groups = groups;
  d.out = y;
  d.out_f32 = y_dtype == FFN_F32;
  d.accumulate = accumulate;
  d.sa = w_scale;
  d.sb = x_scale;
  d.a_rows = w_block_rows;
  return done(launch_linear(d, static_cast<float*>(workspace), workspace_bytes, st(stream)));
}

size_t ffn_grouped_forward_workspace_bytes(int32_t m, int32_t n, int32_t k, int32_t groups) {
  return product_shape_ok(m, n, k, groups) && m > 0 ? lin_workspace(lin_plan(LIN_FWD, 0, m, n, k, groups), m, n) : 0;
}

ffn_status ffn_grouped_forward(const void* x, const void* w, const int32_t* offsets, int32_t groups, int32_t m, int32_t n,
                               int32_t k, void* y, int32_t y_dtype, void* workspace, size_t workspace_bytes, void* stream) {
  if (!product_shape_ok(m, n, k, groups) || n % 8 != 0 || k % 8 != 0 || !dtype_ok(y_dtype)) return FFN_E_INVALID;
  if (m == 0) return FFN_OK;
  if (!need(x) || !need(w) || !need(offsets) || !need(y) || !opt(workspace)) return FFN_E_INVALID;
  LinDesc d{};
  d.kind = LIN_FWD;
  d.A = w;
  d.B = x;
  d.rows = m;
  d.cols = n;
  d.K = k;
  d.a_group = (long long)n * k;
  d.offsets = offsets;
  d.groups = groups;
  d.out = y;
  d.out_f32 = y_dtype == FFN_F32;
  return done(launch_linear(d, static_cast<float*>(workspace), workspace_bytes, st(stream)));
}

size_t ffn_grouped_backward_workspace_bytes(int32_t m, int32_t n, int32_t k, int32_t groups) {
  return product_shape_ok(m, n, k, groups) && m > 0 ? lin_workspace(lin_plan(LIN_DX, 0, m, k, n, groups), m, k) : 0;
}

ffn_status ffn_grouped_backward(const void* x, const void* w, const void* dy, const int32_t* offsets, int32_t groups,
                                int32_t m, int32_t n, int32_t k, void* dx, float* dw, int32_t accumulate, void* workspace,
                                size_t workspace_bytes, void* stream) {
  if (!product_shape_ok(m, n, k, groups) || n % 8 != 0 || k % 8 != 0 || !flag_ok(accumulate) || !opt(dw)) return FFN_E_INVALID;
  if (m == 0) {
    if (!dw || accumulate) return FFN_OK;
    return done(launch_fill_u32(reinterpret_cast<uint32_t*>(dw), 0u, (size_t)groups * n * k, st(stream)));
  }
  if (!need(dy) || !need(offsets) || !opt(x) || !opt(w) || !opt(dx) || !opt(workspace) || (!dx && !dw) || (dx && !w) ||
      (dw && !x))
    return FFN_E_INVALID;
  LinDesc d{};
  d.offsets = offsets;
  d.groups = groups;
  if (dx) {
    d.kind = LIN_DX;
    d.A = w;
    d.B = dy;
    d.rows = m;
    d.cols = k;
    d.K = n;
    d.a_group = (long long)n * k;
    d.out = dx;
    const hipError_t e = launch_linear(d, static_cast<float*>(workspace), workspace_bytes, st(stream));
    if (e != hipSuccess) return FFN_E_HIP;
  }
  if (dw) {
    d.kind = LIN_DW;
    d.A = x;
    d.B = dy;
    d.rows = n;
    d.cols = k;
    d.K = m;
    d.a_group = 0;
    d.out = dw;
    d.out_f32 = 1;
    d.accumulate = accumulate;
    return done(launch_linear(d, static_cast<float*>(workspace), workspace_bytes, st(stream)));
  }
  return FFN_OK;
}

}  // extern "C"
