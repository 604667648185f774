// bf16 query rows as two-term e4m3 sums for the e4m3 tensor cores: row r under
// a power-of-two scale s_r that puts max|q| in [128, 256) is hi + lo with hi =
// e4m3(q s_r), lo = e4m3(q s_r - hi).  Exact for components within 2^10 of the
// row's largest, within 2^-10 of s_r's unit below that.
#pragma once

#include <cstdint>

#include "common.cuh"
#include "ptx.cuh"

namespace mla {

// One warp: row `q` of 576 bf16 to terms[2][576] and 1 / s_r; NaN in its place
// if a value is infinite or NaN.  A row that is not live gets zeros.
__device__ __forceinline__ void split_query_row(const uint16_t* q, bool live, uint8_t* terms,
                                                float* inv_scale, int lane) {
  constexpr int kUnits = kDqk / 8;   // 16-byte units of a row: 72, three rounds of a warp
  uint4 v[3];
  uint32_t mx = 0;
#pragma unroll
  for (int k = 0; k < 3; ++k) {
    const int u = lane + 32 * k;
    v[k] = make_uint4(0, 0, 0, 0);
    if (live && u < kUnits) v[k] = reinterpret_cast<const uint4*>(q)[u];
    const uint32_t w[4] = {v[k].x, v[k].y, v[k].z, v[k].w};
#pragma unroll
    for (int e = 0; e < 4; ++e) mx = max(mx, max(w[e] & 0x7FFFu, (w[e] >> 16) & 0x7FFFu));
  }
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) mx = max(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, off));
  // s_r = 2^(134 - e), clamped so that it and 1 / s_r are normal floats
  const uint32_t e = min(max(mx >> 7, 8u), 254u);
  const float sc = __uint_as_float((261u - e) << 23);
  if (lane == 0)
    *inv_scale = (mx >> 7) == 255u ? __uint_as_float(0x7FC00000u) : __uint_as_float((e - 7u) << 23);
#pragma unroll
  for (int k = 0; k < 3; ++k) {
    const int u = lane + 32 * k;
    if (u < kUnits) {
      const uint32_t w[4] = {v[k].x, v[k].y, v[k].z, v[k].w};
      uint32_t sp[4];
#pragma unroll
      for (int i = 0; i < 4; ++i)
        sp[i] = split_e4m3x2(__uint_as_float(w[i] << 16) * sc,
                             __uint_as_float(w[i] & 0xFFFF0000u) * sc);
      reinterpret_cast<uint2*>(terms)[u] =
          make_uint2((sp[0] & 0xFFFFu) | (sp[1] << 16), (sp[2] & 0xFFFFu) | (sp[3] << 16));
      reinterpret_cast<uint2*>(terms + kDqk)[u] =
          make_uint2((sp[0] >> 16) | (sp[1] & 0xFFFF0000u), (sp[2] >> 16) | (sp[3] & 0xFFFF0000u));
    }
  }
}

}  // namespace mla
