// Merge of the pieces of a split work unit of the per-request kernels, one
// block of 256 threads per two query rows.
#pragma once

#include <math_constants.h>

#include "common.cuh"
#include "merge.cuh"

namespace mla {

// The pieces of a split unit: CTA c0 + k's piece of the unit, in the
// workspace slot it wrote (a CTA writes its first piece to slot 0 and its
// last to slot 1; the unit's first CTA had an earlier piece iff its range
// starts before the unit's positions).
struct UnitPieces {
  const float* ws_o;
  const float* ws_lse;
  struct Ctx {
    int c0, count, r, first_in_slot1;
  };
  __device__ void piece(const Ctx& c, int k, const float*& src, float& lse) const {
    const size_t cc = (size_t)(c.c0 + k);
    const size_t slot = (k == 0 && c.first_in_slot1) ? 2 * cc + 1 : 2 * cc;
    src = ws_o + (slot * kRows + c.r) * kDv;
    lse = ws_lse[slot * kRows + c.r];
  }
};

// Block (u, y) handles query rows 2y and 2y + 1 of unit u with four warps
// per row, each merging 128 of the 512 latent dims over the unit's pieces
// (kMergeBatch pieces in flight per warp).
constexpr int kMergeRowsPerBlock = 2;
constexpr int kMergeBatch = 12;
constexpr int kMergeSmem = 8 * kMergeBatch * 32 * (int)sizeof(float4);

// Rows of unit u, block y of 2 * kVec rows, if the partial kernel left them: 0 and
// -inf, or the merge of their pieces, 4 / kVec warps per row and kB pieces in
// flight.  `stage`: 8 * kB * kVec * 512 bytes of shared memory.
template <int kVec, int kB>
__device__ __forceinline__ void merge_unit_rows(const ProblemDesc& pd, const WsHeader* hdr,
                                                const int* prefix, const float* ws_o,
                                                const float* ws_lse, float* out_partial,
                                                float* lse_partial, int u, int y, float4* stage) {
  const Unit x = make_unit(pd, u);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  constexpr int kWarps = 4 / kVec;               // per row
  const int r = y * (8 / kWarps) + warp / kWarps, part = warp % kWarps;
  if (r >= x.rows_out) return;
  const int ps = prefix[u], ue = prefix[u + 1];
  const int us = unit_tile_start(prefix, u, hdr->unit_cost);
  const size_t orow = out_row(pd, x, r);
  float4* dst = reinterpret_cast<float4*>(out_partial + orow * kDv) + 32 * kVec * part;
  const int per = hdr->per_cta;
  const bool split = us < ue && us / per != (ue - 1) / per;
  // rows with no token to see: the shard holds none of the request's
  // positions, or the row is padding of a request with fewer query tokens
  // (a whole unit's padding rows are written by the partial kernel)
  if (us == ue || (split && r >= x.rows)) {
#pragma unroll
    for (int v = 0; v < kVec; ++v) dst[lane + 32 * v] = make_float4(0.f, 0.f, 0.f, 0.f);
    if (part == 0 && lane == 0) lse_partial[orow] = -CUDART_INF_F;
    return;
  }
  const int c0 = us / per, c1 = (ue - 1) / per;
  if (c0 == c1) return;  // written directly by the partial kernel
  const UnitPieces src{ws_o, ws_lse};
  const UnitPieces::Ctx ctx{c0, c1 - c0 + 1, r, c0 * per < ps ? 1 : 0};
  float4 acc[kVec];
  float M, wsum;
  merge_pieces_staged<kVec, kB>(src, ctx, lane, 32 * kVec * part, stage + warp * (kB * kVec * 32), acc,
                                M, wsum);
  const float inv = wsum != 0.f ? 1.0f / wsum : 0.f;   // or NaN
#pragma unroll
  for (int v = 0; v < kVec; ++v)
    dst[lane + 32 * v] =
        make_float4(acc[v].x * inv, acc[v].y * inv, acc[v].z * inv, acc[v].w * inv);
  if (part == 0 && lane == 0) lse_partial[orow] = wsum != 0.f ? M + __logf(wsum) : -CUDART_INF_F;
}

}  // namespace mla
