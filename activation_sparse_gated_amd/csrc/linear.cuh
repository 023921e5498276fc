// Internal interface of the operators around the FFN (include/ffn_linear.h):
// descriptors and launches shared by the C ABI layer (linear_api.hip) and the
// kernels (k_rmsnorm.hip, k_quant.hip, k_linear.hip).
#pragma once
#include "kernels.cuh"

namespace ffn {

constexpr int kFp8Block = 128;                 // columns (and rows) of an 8-bit block
constexpr int kLinMaxGroups = 256;             // experts of one call

struct NormDesc {
  const void *x, *res, *w;       // forward: x, residual or null; backward: r, dr or null
  const void* dy;                // backward only
  int dtype, m, d;
  float eps;
  void *r_out, *y;               // forward
  uint8_t* q;
  float* scale;
  void* dx;                      // backward
  float* dw;
  float* part;                   // [parts x d] partial rows of dw
  int parts, accumulate;
};
int rmsnorm_bwd_parts(int m, int d);
hipError_t launch_rmsnorm_fwd(const NormDesc& n, hipStream_t s);
hipError_t launch_rmsnorm_bwd(const NormDesc& n, hipStream_t s);

struct QuantDesc {
  const void* x;
  int dtype, groups, m, k, block_rows;
  uint8_t *q, *qt;
  float *scale, *scale_t;
  int mt;                        // row length of qt
};
hipError_t launch_fp8_quant(const QuantDesc& q, hipStream_t s);

// out[r][c] = sum_j B[r][j] A[c][j]: A gives the output's columns, B its rows.
enum LinKind : int {
  LIN_FP8 = 0,      // y = x w^T of 8-bit blocks: A = w, B = x
  LIN_FWD = 1,      // y = x W_g^T, bf16: A = W_g, B = x
  LIN_DX = 2,       // dx = dy W_g: A = W_g read along its rows, B = dy
  LIN_DW = 3        // dW_g = dy^T x over the rows of g: A = x, B = dy, both along their rows
};
struct LinDesc {
  int kind;
  const void *A, *B;
  int rows, cols, K;             // output rows (all experts' together; LIN_DW: of one expert), columns, contraction length (LIN_DW: rows of x)
  long long a_group;             // elements of A per expert (LIN_FP8, LIN_FWD, LIN_DX)
  const int32_t* offsets;        // null: one expert that has every row
  int groups;
  void* out;
  int out_f32, accumulate;
  const float *sa, *sb;          // LIN_FP8: scales of A and B
  int a_rows;                    // LIN_FP8: rows of a block of A, 1 or 128
  int ks;                        // slices of the contraction; > 1: fp32 slabs part[ks][rows][cols]
  float* part;
};
// How a product is run (lin_plan, a rule on sizes alone).
struct LinPlan {
  int skinny;                    // k_linear_skinny, else k_linear
  int mb, nw;                    // skinny: 16-row blocks of a row tile, waves
  int rt, ct;                    // k_linear: rows and columns of a tile
  int ks;                        // slices of the contraction
};
LinPlan lin_plan(int kind, int exact, int rows, int cols, int K, int groups);
size_t lin_workspace(const LinPlan& p, int rows, int cols);
hipError_t launch_linear(LinDesc d, float* workspace, size_t workspace_bytes, hipStream_t s);
hipError_t launch_linear_tiled(const LinDesc& d, const LinPlan& p, hipStream_t s);
hipError_t launch_linear_skinny(const LinDesc& d, const LinPlan& p, hipStream_t s);
hipError_t launch_linear_sum(const LinDesc& d, hipStream_t s);

}  // namespace ffn
