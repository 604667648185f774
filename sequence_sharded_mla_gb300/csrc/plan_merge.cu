// Work planning and split merging for the partial kernel.
//
// mla_plan_kernel      counts the 64-token tiles of every work unit
//                      (request, shard, 64-row query group), charges every
//                      unit with tiles unit_cost extra positions for its fixed
//                      costs, forms the exclusive prefix of these work
//                      positions and splits them evenly over the persistent
//                      CTAs (a CTA with many short units gets fewer tiles).
// mla_merge_kernel     writes every unit the partial kernel did not write
//                      itself: units with no tokens (o = 0, lse = -inf) and
//                      units split across CTAs, whose pieces it merges by
//                      their LSEs -- the same reweighting that merges shards
//                      ("Decode Context Parallelism", section 4.1).
#include <math_constants.h>

#include "common.cuh"
#include "host_util.h"
#include "ptx.cuh"
#include "unit_merge.cuh"

namespace mla {

__global__ void __launch_bounds__(1024) mla_plan_kernel(ProblemDesc pd, WsHeader* hdr, int* prefix,
                                                        int grid, int min_tiles,
                                                        int unit_cost) {
  griddep_launch_dependents();   // the partial kernel may start launching
  __shared__ unsigned bad_qlen;
  if (threadIdx.x == 0) bad_qlen = 0;
  __syncthreads();
  if (pd.q_lens != nullptr)
    for (int b = threadIdx.x; b < pd.B; b += 1024)
      if (pd.q_lens[b] < 1 || pd.q_lens[b] > pd.q_len) atomicOr(&bad_qlen, kErrQLens);
  __syncthreads();
  plan_units(pd.B * pd.n_out * pd.G, [&](int u) { return make_unit(pd, u).tiles; }, hdr, prefix,
             grid, min_tiles, unit_cost, bad_qlen);
}

__global__ void __launch_bounds__(256, 4) mla_merge_kernel(
    ProblemDesc pd, const WsHeader* hdr, const int* prefix, const float* ws_o,
    const float* ws_lse, float* out_partial, float* lse_partial) {
  extern __shared__ __align__(16) float4 merge_stage[];   // [8 warps][kMergeBatch][32]
  griddep_wait();                // the partial kernel's pieces and outputs
  griddep_launch_dependents();
  merge_unit_rows<1, kMergeBatch>(pd, hdr, prefix, ws_o, ws_lse, out_partial, lse_partial,
                                  blockIdx.x, blockIdx.y, merge_stage);
}

cudaError_t launch_plan(const ProblemDesc& pd, WsHeader* hdr, int* prefix, int grid,
                        int min_tiles, int unit_cost, cudaStream_t stream) {
  mla_plan_kernel<<<1, 1024, 0, stream>>>(pd, hdr, prefix, grid, min_tiles, unit_cost);
  return cudaGetLastError();
}

cudaError_t launch_merge(const ProblemDesc& pd, const WsHeader* hdr, const int* prefix,
                         const float* ws_o, const float* ws_lse, float* out_partial,
                         float* lse_partial, int num_units, cudaStream_t stream) {
  const cudaError_t e =
      host::ensure_dynamic_smem(reinterpret_cast<const void*>(&mla_merge_kernel), kMergeSmem);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(num_units, kRows / kMergeRowsPerBlock);
  cfg.blockDim = dim3(256);
  cfg.dynamicSmemBytes = kMergeSmem;
  cfg.stream = stream;
  cudaLaunchAttribute attr = pdl_attribute();
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, mla_merge_kernel, pd, hdr, prefix, ws_o, ws_lse, out_partial,
                            lse_partial);
}

}  // namespace mla
