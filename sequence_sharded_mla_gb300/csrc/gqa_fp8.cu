// Grouped-query attention over an e4m3 cache with a scale for each block of
// tokens and KV head.  For a query row and the tokens it sees in a shard:
//
//   s_t = scale q . K_t sk(t),  lse = ln sum exp(s_t),
//   o = sum exp(s_t - lse) V_t sv(t)
//
// with K_t, V_t the codes' values and sk, sv the scales of t's block.
//
// One block per output row: each warp walks every fourth token of the shard
// with a running maximum and sum, and the four are joined at the end.
#include <cuda_bf16.h>
#include <math_constants.h>

#include <algorithm>
#include <cmath>

#include "common.cuh"
#include "host_util.h"
#include "mla_dcp.h"
#include "ptx.cuh"

namespace mla {
namespace gqa8 {

constexpr int kD = 128;
constexpr int kThreads = 128;

struct Desc {
  int B, q_len, H, Hkv, G;
  int num_shards, shard_first, n_out, layout, local, causal;
  int num_pages, max_pages, lg_block;
  float scale_log2;
  const uint16_t* q;
  const uint8_t *k, *v;
  const float *ks, *vs;
  const int32_t *block_table, *seq_lens, *q_lens;
  unsigned* err;
};

__global__ void __launch_bounds__(kThreads) gqa_fp8_row_kernel(Desc d, float* out, float* lse) {
  __shared__ float so[4][kD], sm[4], sl[4];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int u = blockIdx.x;
  const size_t row = u;
  const int h = u % d.H;
  u /= d.H;
  const int i = u % d.q_len;
  u /= d.q_len;
  const int b = u % d.B, s = d.shard_first + u / d.B;
  const int kh = h / d.G, L = max(d.seq_lens[b], 0);
  int n = d.q_len;
  if (d.q_lens != nullptr) {
    n = d.q_lens[b];
    if ((n < 1 || n > d.q_len) && threadIdx.x == 0) atomicOr(d.err, kErrQLens);
    n = min(max(n, 0), d.q_len);
  }
  const int seen = i >= n ? 0 : (d.causal ? min(L, max(0, L - n + i + 1)) : L);
  // tokens t0 + k * step, k < cnt, of the shard are seen; slot k (+ off) of the cache holds token k
  int t0, step, cnt;
  if (d.layout == kInterleaved) {
    t0 = s;
    step = d.num_shards;
    cnt = seen > s ? (seen - 1 - s) / step + 1 : 0;
  } else {
    const int c = ceil_div(L, d.num_shards);
    t0 = s * c;
    step = 1;
    cnt = max(0, min(min(t0 + c, L), seen) - t0);
  }
  float qv[4];
  bool bad = false;
  {
    const size_t qr = ((size_t)b * d.q_len + i) * d.H + h;
    const uint2 w = reinterpret_cast<const uint2*>(d.q + qr * kD)[lane];
    qv[0] = __uint_as_float(w.x << 16);
    qv[1] = __uint_as_float(w.x & 0xFFFF0000u);
    qv[2] = __uint_as_float(w.y << 16);
    qv[3] = __uint_as_float(w.y & 0xFFFF0000u);
    for (int e = 0; e < 4; ++e) bad |= !(fabsf(qv[e]) < INFINITY);
  }
  if (bad && i < n) atomicOr(d.err, kErrQRange);
  float m = -CUDART_INF_F, l = 0.f, o[4] = {0.f, 0.f, 0.f, 0.f};
  for (int k = warp; k < cnt; k += 4) {
    const int slot = d.local ? k : t0 + k * step;
    const int idx = slot / kPage, r = slot % kPage;
    int page = idx < d.max_pages ? __ldg(d.block_table + (size_t)b * d.max_pages + idx) : -1;
    float a = 0.f, sv = 0.f, vv[4] = {0.f, 0.f, 0.f, 0.f};
    if (page < 0 || page >= d.num_pages) {
      if (lane == 0) atomicOr(d.err, kErrBadPage);
    } else {
      const size_t e = (((size_t)page * kPage + r) * d.Hkv + kh) * kD;
      const size_t si = ((size_t)page * (kPage >> d.lg_block) + (r >> d.lg_block)) * d.Hkv + kh;
      const uint32_t kw = __ldg(reinterpret_cast<const uint32_t*>(d.k + e) + lane);
      const uint32_t vw = __ldg(reinterpret_cast<const uint32_t*>(d.v + e) + lane);
      float kv[4];
      e4m3x2_to_f32x2(kw, kv[0], kv[1]);
      e4m3x2_to_f32x2(kw >> 16, kv[2], kv[3]);
      e4m3x2_to_f32x2(vw, vv[0], vv[1]);
      e4m3x2_to_f32x2(vw >> 16, vv[2], vv[3]);
      a = qv[0] * kv[0] + qv[1] * kv[1] + qv[2] * kv[2] + qv[3] * kv[3];
#pragma unroll
      for (int off = 16; off > 0; off >>= 1) a += __shfl_xor_sync(0xffffffffu, a, off);
      a *= d.scale_log2 * __ldg(d.ks + si);
      sv = __ldg(d.vs + si);
    }
    const float mn = a > m ? a : (a != a ? a : m);
    const float al = m == -CUDART_INF_F ? 0.f : exp2f(m - mn);
    const float p = exp2f(a - mn);
    m = mn;
    l = l * al + p;
#pragma unroll
    for (int e = 0; e < 4; ++e) o[e] = o[e] * al + p * (vv[e] * sv);
  }
  reinterpret_cast<float4*>(so[warp])[lane] = make_float4(o[0], o[1], o[2], o[3]);
  if (lane == 0) {
    sm[warp] = m;
    sl[warp] = l;
  }
  __syncthreads();
  float M = -CUDART_INF_F;
  for (int w = 0; w < 4; ++w) M = sl[w] != 0.f ? (sm[w] > M || sm[w] != sm[w] ? sm[w] : M) : M;
  float tot = 0.f, acc = 0.f;
  for (int w = 0; w < 4; ++w) {
    if (sl[w] == 0.f) continue;
    const float f = exp2f(sm[w] - M);
    tot += f * sl[w];
    acc += f * so[w][threadIdx.x];
  }
  out[row * kD + threadIdx.x] = tot == 0.f ? 0.f : acc / tot;
  if (threadIdx.x == 0)
    lse[row] = tot == 0.f ? -CUDART_INF_F : (M + log2f(tot)) * 0.69314718055994530942f;
}

bool shape_ok(const gqa_shape* s) {
  if (s == nullptr || s->batch < 1 || s->q_len < 1 || s->num_heads < 1 || s->num_kv_heads < 1)
    return false;
  if (s->causal != 0 && s->causal != 1) return false;
  if (!std::isfinite(s->softmax_scale) || s->softmax_scale <= 0.f) return false;
  return (long long)s->batch * s->q_len * s->num_heads < (1LL << 24);
}

bool shape_supported(const gqa_shape* s) {
  return s->head_dim == kD && s->num_heads % s->num_kv_heads == 0 &&
         s->num_heads / s->num_kv_heads <= kRows;
}

bool shards_ok(int num_shards, int shard_id) {
  return num_shards >= 1 && num_shards <= kMaxShards &&
         (shard_id == MLA_ALL_SHARDS || (shard_id >= 0 && shard_id < num_shards));
}

}  // namespace gqa8
}  // namespace mla

using namespace mla;

extern "C" {

size_t gqa_fp8_workspace_size(const gqa_shape* shape, int num_shards, int shard_id) {
  if (!gqa8::shape_ok(shape) || !gqa8::shape_supported(shape) ||
      !gqa8::shards_ok(num_shards, shard_id))
    return 0;
  return sizeof(WsHeader);
}

mla_status gqa_decode_partial_fp8(const void* q, const gqa_block_pages* cache,
                                  const int32_t* block_table, int max_pages_per_req,
                                  const int32_t* seq_lens, const int32_t* q_lens,
                                  const gqa_shape* shape, int shard_id, int num_shards,
                                  mla_layout layout, float* out_partial, float* lse_partial,
                                  void* workspace, size_t workspace_bytes, void* stream) {
  using host::aligned16;
  using host::aligned4;
  if (!q || !cache || !block_table || !seq_lens || !out_partial || !lse_partial)
    return MLA_ERR_INVALID;
  if (!gqa8::shape_ok(shape) || !gqa8::shards_ok(num_shards, shard_id)) return MLA_ERR_INVALID;
  if (layout < MLA_LAYOUT_INTERLEAVED || layout > MLA_LAYOUT_CONTIGUOUS_LOCAL)
    return MLA_ERR_INVALID;
  const bool local = layout >= MLA_LAYOUT_INTERLEAVED_LOCAL;
  if (local && shard_id == MLA_ALL_SHARDS) return MLA_ERR_INVALID;
  if (!cache->k || !cache->v || !cache->k_scale || !cache->v_scale || cache->num_pages < 1 ||
      max_pages_per_req < 1)
    return MLA_ERR_INVALID;
  if (cache->dtype != MLA_KV_FP8_E4M3 || cache->num_kv_heads != shape->num_kv_heads)
    return MLA_ERR_INVALID;
  if (cache->block < 1 || cache->block > kPage || (cache->block & (cache->block - 1)))
    return MLA_ERR_INVALID;
  if (cache->page_size != kPage || !gqa8::shape_supported(shape)) return MLA_ERR_UNSUPPORTED;
  if (layout == MLA_LAYOUT_INTERLEAVED && kPage % num_shards != 0) return MLA_ERR_UNSUPPORTED;
  // cache rows are addressed with 31-bit coordinates
  if (((long long)cache->num_pages + 1) * kPage * cache->num_kv_heads >= (1LL << 31))
    return MLA_ERR_UNSUPPORTED;
  if (!aligned16(q) || !aligned16(cache->k) || !aligned16(cache->v) || !aligned16(out_partial) ||
      !aligned16(lse_partial) || !aligned4(cache->k_scale) || !aligned4(cache->v_scale) ||
      !aligned4(block_table) || !aligned4(seq_lens) || !aligned4(q_lens))
    return MLA_ERR_INVALID;
  if (workspace == nullptr || !aligned16(workspace)) return MLA_ERR_WORKSPACE;
  if (workspace_bytes < gqa_fp8_workspace_size(shape, num_shards, shard_id))
    return MLA_ERR_WORKSPACE;

  gqa8::Desc d;
  d.B = shape->batch;
  d.q_len = shape->q_len;
  d.H = shape->num_heads;
  d.Hkv = shape->num_kv_heads;
  d.G = d.H / d.Hkv;
  d.num_shards = num_shards;
  d.shard_first = shard_id == MLA_ALL_SHARDS ? 0 : shard_id;
  d.n_out = shard_id == MLA_ALL_SHARDS ? num_shards : 1;
  d.layout = (layout & 1) ? kContiguous : kInterleaved;
  d.local = local;
  d.causal = shape->causal;
  d.num_pages = cache->num_pages;
  d.max_pages = max_pages_per_req;
  d.lg_block = 0;
  while ((1 << d.lg_block) < cache->block) ++d.lg_block;
  d.scale_log2 = shape->softmax_scale * 1.4426950408889634f;
  d.q = static_cast<const uint16_t*>(q);
  d.k = static_cast<const uint8_t*>(cache->k);
  d.v = static_cast<const uint8_t*>(cache->v);
  d.ks = cache->k_scale;
  d.vs = cache->v_scale;
  d.block_table = block_table;
  d.seq_lens = seq_lens;
  d.q_lens = q_lens;
  d.err = &static_cast<WsHeader*>(workspace)->err;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (cudaMemsetAsync(workspace, 0, sizeof(WsHeader), st) != cudaSuccess) return MLA_ERR_CUDA;
  gqa8::gqa_fp8_row_kernel<<<d.n_out * d.B * d.q_len * d.H, gqa8::kThreads, 0, st>>>(
      d, out_partial, lse_partial);
  return cudaGetLastError() == cudaSuccess ? MLA_OK : MLA_ERR_CUDA;
}

}  // extern "C"
