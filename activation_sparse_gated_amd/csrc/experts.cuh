// Internal interface of routing to experts (include/ffn_experts.h): descriptors
// and launches shared by the C ABI layer (experts_api.hip) and the kernels
// (k_router.hip, k_rows.hip).
#pragma once
#include "kernels.cuh"

namespace ffn {

constexpr int kRowsMaxGroups = 1024;

struct RouterDesc {
  const void* logits;
  int dtype, m, experts, top_k;
  int sigmoid, groups, top_groups, group_best, renormalize;
  float scale;
  const float* bias;             // forward
  float *weights, *scores;
  int32_t* ids;
  const int32_t* ids_in;         // backward
  const float *dweights, *dscores;
  void* dlogits;
};
hipError_t launch_router_fwd(const RouterDesc& d, hipStream_t s);
hipError_t launch_router_bwd(const RouterDesc& d, hipStream_t s);

struct GroupDesc {
  const int32_t* ids;
  int n, groups;
  int32_t *offsets, *rows, *slots;
  uint32_t* hist;                // [blocks][groups + 1] entries of each block, if there is more than one
};
int group_rows_blocks(int n);    // 1: no workspace
hipError_t launch_group_rows(const GroupDesc& d, hipStream_t s);

struct RowsDesc {
  int dtype, m, d, top_k;
  const int32_t* slots;
  const void* x;                 // gather: tokens; combine: the experts' rows
  const float* weights;
  const void *residual, *dout;
  void* y;                       // gather: rows; combine: tokens; combine's gradient: rows
  uint8_t* q;
  float *scale, *dweights;
};
hipError_t launch_gather(const RowsDesc& d, hipStream_t s);
hipError_t launch_combine_fwd(const RowsDesc& d, hipStream_t s);
hipError_t launch_combine_bwd(const RowsDesc& d, hipStream_t s);

// A grid of `groups` workgroups of up to 1024 threads: it holds fewer than 2^32 threads a dimension.
inline dim3 grid2(long long groups) {
  const long long y = (groups + (1 << 21) - 1) >> 21;
  return dim3((unsigned)((groups + y - 1) / y), (unsigned)y);
}

}  // namespace ffn
