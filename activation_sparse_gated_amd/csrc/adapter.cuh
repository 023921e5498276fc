// Internal interface of the low-rank adapters (include/ffn_adapter.h):
// descriptors and launches shared by the C ABI layer (adapter_api.hip) and the
// kernels (k_adapter.hip).
#pragma once
#include "kernels.cuh"

namespace ffn {

constexpr int kAdapterMaxGroups = 1024;
constexpr int kAdapterMaxRank = 256;

// How a call is run (adapter_plan, a rule on sizes alone).
struct AdapterPlan {
  int rt;                        // rows of a tile: 16 or 64
  int ks, kd;                    // slices of the contraction of x A^T and of dy B
  int tiles;                     // tiles at most, those of rows without an adapter among them
  int few;                       // forward: 0, or both products in one launch, by so many workgroups a tile
  int split, slices;             // of an adapter's rows for its gradients: waves that share a column block, and slices besides
  size_t part;                   // values of a slice's gradients
};

struct AdapterDesc {
  const uint16_t *x, *dy, *a, *b;
  const float* scales;
  const int32_t *offsets, *rows;
  int groups, m, n, k, r;
  const void* base;
  void* out;                     // y or dx
  int out_f32;
  float *da, *db;
  int accumulate;
  AdapterPlan p;
  // workspace (none with p.few)
  int4* tab;                     // [tiles]: adapter (-1: none, -2: no tile), first place, end
  float *h, *dh;                 // [ks or kd][tiles][rt][r]: x A^T and dy B
  uint16_t *hp, *dhp;            // null, or [tiles][3][rt][r]: s h (forward, tiles of 64 rows) and s dh in bf16 numbers
  uint16_t *ht, *dht;            // null, or [tiles][3][r][rt]: the same with the rows along
  float* part;                   // [slices][part]: partial gradients, if slices > 1
};

AdapterPlan adapter_plan(int m, int n, int k, int r, int groups, bool backward);

// The workgroups of the second half of the backward pass: those of the adapters' gradients, then those of dx. The grid may
// hold some more, which have nothing to do.
struct BackGrid {
  int a, b;                      // column blocks of da and db
  int groups, z;                 // z: rank blocks times slices
  int x;                         // column blocks of dx (0: not asked for)
  unsigned gx, gy;               // the grid
  long long dw, all;             // (a + b) groups z workgroups of da and db; with those of dx
};
BackGrid adapter_back_grid(const AdapterPlan& p, int n, int k, int r, int groups, bool dx, bool da, bool db);
enum BackPart : int { BACK_GRADIENTS = 0, BACK_DX = 1, BACK_NOTHING = 2 };
__host__ __device__ __attribute__((used)) inline int adapter_back_part(const BackGrid& g, long long workgroup) {
  return workgroup < g.dw ? BACK_GRADIENTS : workgroup < g.all ? BACK_DX : BACK_NOTHING;
}
// out = base + scale (x A^T) B^T
hipError_t launch_adapter_forward(const AdapterDesc& d, hipStream_t s);
// out = base + scale dh A, and the gradients da and db; those that are not null. d.dh is needed for out and da, d.h for db
hipError_t launch_adapter_backward(const AdapterDesc& d, hipStream_t s);

}  // namespace ffn
