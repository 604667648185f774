// Rotary positions on query heads, and the append of a step's new tokens to
// the paged caches: k rotated, quantised and written to its page in one pass,
// the step's query rotated by further blocks of the same launch.
//
// The new rows are read once and written once; nothing else of the cache
// moves, except the earlier codes of an e4m3 block whose scale has to grow.
// The work is bound by memory for prompt chunks and by the launch for single
// tokens.
#include <cuda_bf16.h>

#include <algorithm>
#include <cmath>

#include "common.cuh"
#include "host_util.h"
#include "mla_dcp.h"
#include "ptx.cuh"
#include "rope.cuh"

namespace mla {
namespace append {

constexpr int kGD = 128;          // GQA head width
constexpr int kThreads = 128;     // cache and query blocks
constexpr int kMaxPairs = 512;    // rotated pairs of the widest head
constexpr float kMinScale = 8.67361737988403547e-19f;   // 2^-60

struct Tokens {
  int B, q_len;
  const int32_t* seq_lens;
  const int32_t* q_lens;
  const int32_t* positions;
};

// Query heads to rotate (heads == 0: none).
struct Rows {
  const uint16_t* x;
  uint16_t* y;
  long long xs, ys;    // elements between tokens
  int heads, D;
  Div split;           // blocks a token's heads are spread over
  Div items;           // a head's work items (see turn_heads)
};

struct Cache {
  uint8_t* k;          // GQA: K and V; MLA: the latent rows in k
  uint8_t* v;
  float* ks;
  float* vs;
  int fp8, block, num_pages, Hkv;
  const int32_t* bt;
  int max_pages;
  int shard;
  Div num_shards;
  unsigned* err;
};

__device__ __forceinline__ int new_count(const Tokens& t, int b, unsigned* err) {
  if (t.q_lens == nullptr) return t.q_len;
  const int n = t.q_lens[b];
  if (err != nullptr && (n < 1 || n > t.q_len)) atomicOr(err, kErrQLens);
  return min(max(n, 0), t.q_len);
}

__device__ __forceinline__ int rope_pos(const Tokens& t, int b, int i, int stand) {
  return t.positions != nullptr ? t.positions[(size_t)b * t.q_len + i] : stand;
}

// Page of slot index `p` of request b, or -1 (reported) if there is none.
__device__ __forceinline__ int page_of(const Cache& c, int b, int p) {
  const int idx = p / kPage;
  const int page = idx < c.max_pages ? __ldg(c.bt + (size_t)b * c.max_pages + idx) : -1;
  if (page >= 0 && page < c.num_pages) return page;
  atomicOr(c.err, kErrBadPage);
  return -1;
}

__device__ __forceinline__ float bf_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf_hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }
__device__ __forceinline__ uint32_t bf_pack(float a, float b) {
  __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<uint32_t*>(&h);
}

__device__ __forceinline__ float finite_abs(float x) {
  const float a = fabsf(x);
  return a < INFINITY ? a : 0.0f;   // NaN and infinities do not set a scale
}

// Smallest power of two s >= 2^-60 with a <= 448 s (a finite, >= 0):
// a = m 2^e with m in [1, 2) and 448 = 1.75 2^8, so s = 2^(e - 8), one more if
// m > 1.75.
__device__ __forceinline__ float pow2_scale(float a) {
  const uint32_t bits = __float_as_uint(a);
  const int e = (int)(bits >> 23) - 8 + ((bits & 0x7FFFFFu) > 0x600000u ? 1 : 0);
  return e < 127 - 60 ? kMinScale : __uint_as_float((uint32_t)e << 23);
}

// e4m3 code of x / s: the nearest code; infinities become NaN.
__device__ __forceinline__ uint32_t codes2(float a, float b) {
  const float fa = fabsf(a) < INFINITY ? a : __int_as_float(0x7fffffff);
  const float fb = fabsf(b) < INFINITY ? b : __int_as_float(0x7fffffff);
  return f32x2_to_e4m3x2(fa, fb);
}

// The (cos, sin) of every rotated pair of one position, by the whole block.
__device__ __forceinline__ void fill_cs(const RopeArgs& r, int pos, float2* cs, int tid, int n) {
  for (int i = tid; i < r.rot / 2; i += n) cs[i] = turn_cs(turn_rate(__ldg(r.inv_freq + i)), pos, r.factor);
}

__device__ __forceinline__ uint4 turn_interleaved(uint4 w, const float2* cs) {
  uint32_t* p = &w.x;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    float a = bf_lo(p[e]), b = bf_hi(p[e]);
    turn_pair(a, b, cs[e]);
    p[e] = bf_pack(a, b);
  }
  return w;
}

__device__ __forceinline__ void turn_half(uint4& wa, uint4& wb, const float2* cs) {
  uint32_t *pa = &wa.x, *pb = &wb.x;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    float a0 = bf_lo(pa[e]), b0 = bf_lo(pb[e]), a1 = bf_hi(pa[e]), b1 = bf_hi(pb[e]);
    turn_pair(a0, b0, cs[2 * e]);
    turn_pair(a1, b1, cs[2 * e + 1]);
    pa[e] = bf_pack(a0, a1);
    pb[e] = bf_pack(b0, b1);
  }
}

// Work items of a head: a rotation of 8 (interleaved) or 16 dims (half), or,
// unless in place, a copy of 8.
__host__ __device__ inline int head_items(int D, int rot, int interleaved, bool inplace) {
  return (interleaved ? rot / 8 : rot / 16) + (inplace ? 0 : (D - rot) / 8);
}

// Heads [h0, h1) of one token, D wide, src -> dst, by n threads; in place if
// src == dst (only the rotated dims move).  rot == 0 copies.  A thread has
// two items' loads in flight.
__device__ __forceinline__ void turn_heads(const uint16_t* src, uint16_t* dst, int D, int h0,
                                           int h1, const RopeArgs& r, const Div& items,
                                           const float2* cs, int tid, int n) {
  const int f8 = r.first >> 3, r8 = r.rot >> 3;
  const int turns = r.interleaved ? r8 : r8 >> 1;
  const uint4* s = reinterpret_cast<const uint4*>(src + (size_t)h0 * D);
  uint4* d = reinterpret_cast<uint4*>(dst + (size_t)h0 * D);
  const int total = (h1 - h0) * items, d8 = D >> 3;
  for (int x0 = tid; x0 < total; x0 += 2 * n) {
    uint4 a[2], b[2];
    int at[2], it[2];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const int x = x0 + k * n;
      if (x >= total) break;
      const int h = x / items, i = x - h * items, c = i - turns;
      it[k] = i;
      at[k] = h * d8 + (i < turns ? f8 + i : c < f8 ? c : c + r8);
      a[k] = s[at[k]];
      if (!r.interleaved && i < turns) b[k] = s[at[k] + turns];
    }
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      if (x0 + k * n >= total) break;
      if (it[k] < turns) {
        if (r.interleaved) {
          a[k] = turn_interleaved(a[k], cs + 4 * it[k]);
        } else {
          turn_half(a[k], b[k], cs + 8 * it[k]);
          d[at[k] + turns] = b[k];
        }
      }
      d[at[k]] = a[k];
    }
  }
}

// Block `blk` of the query rotation: token blk / split, a share of its heads.
__device__ __forceinline__ void query_block(const Rows& q, const Tokens& t, const RopeArgs& r,
                                            int blk, float2* cs) {
  const int tok = blk / q.split, part = blk % q.split;
  const int b = tok / t.q_len, i = tok - b * t.q_len;
  const int n = new_count(t, b, nullptr);
  if (i >= n) return;
  const int stand = t.seq_lens != nullptr ? t.seq_lens[b] - n + i : 0;
  fill_cs(r, rope_pos(t, b, i, stand), cs, threadIdx.x, blockDim.x);
  __syncthreads();
  const int per = (q.heads - 1) / q.split + 1;
  turn_heads(q.x + tok * q.xs, q.y + tok * q.ys, q.D, part * per, min(q.heads, (part + 1) * per), r,
             q.items, cs, threadIdx.x, blockDim.x);
}

// Bound by DRAM for prompt chunks: 8191 tokens x 64 heads x 128 (268 MB) 44.7
// us, 6.0 TB/s; four items a thread in place of two take the registers of half
// the blocks (50 us).  144 tokens x 64 heads x 576 (21 MB): 4.3 us.
__global__ void __launch_bounds__(kThreads, 10) rope_kernel(Rows q, Tokens t, RopeArgs r) {
  __shared__ float2 cs[kMaxPairs];
  griddep_wait();
  griddep_launch_dependents();
  query_block(q, t, r, blockIdx.x, cs);
}

// ----------------------------------------------------------- latent rows
// One block per new token: the 576 values in shared memory as fp32, rotated
// there, then rounded (bf16) or scaled by the row's power of two (e4m3).  Bound
// by the launch and the chain of loads: 2053 tokens 3.6 us in one wave of 16
// blocks an SM (4.9 us at 12); 64 tokens with 64 query heads 3.5 us.
__global__ void __launch_bounds__(kThreads, 16) latent_append_kernel(const uint16_t* x, long long xs,
                                                                 Cache c, Tokens t, RopeArgs r,
                                                                 Rows q, int cache_blocks) {
  __shared__ float2 cs[kDqk / 2];
  __shared__ float row[kDqk];
  __shared__ float red[kThreads / 32];
  griddep_wait();
  griddep_launch_dependents();
  if ((int)blockIdx.x >= cache_blocks) {
    query_block(q, t, r, blockIdx.x - cache_blocks, cs);
    return;
  }
  const int tid = threadIdx.x, tok = blockIdx.x;
  const int b = tok / t.q_len, i = tok - b * t.q_len;
  const int n = new_count(t, b, c.err);
  if (i >= n) return;
  const int p = t.seq_lens[b] - n + i;
  if (p < 0) {
    if (tid == 0) atomicOr(c.err, kErrQLens);
    return;
  }
  if (p % c.num_shards != c.shard) return;
  const int lp = p / c.num_shards, page = page_of(c, b, lp);
  if (page < 0) return;
  const size_t dst = (size_t)page * kPage + lp % kPage;
  const uint32_t* src = reinterpret_cast<const uint32_t*>(x + tok * xs);
  for (int e = tid; e < kDqk / 2; e += kThreads) {
    const uint32_t w = __ldg(src + e);
    row[2 * e] = bf_lo(w);
    row[2 * e + 1] = bf_hi(w);
  }
  fill_cs(r, rope_pos(t, b, i, p), cs, tid, kThreads);
  __syncthreads();
  for (int e = tid; e < r.rot / 2; e += kThreads) {
    const int ia = r.first + (r.interleaved ? 2 * e : e);
    const int ib = r.interleaved ? ia + 1 : ia + r.rot / 2;
    turn_pair(row[ia], row[ib], cs[e]);
  }
  __syncthreads();
  if (!c.fp8) {
    uint32_t* d = reinterpret_cast<uint32_t*>(c.k) + dst * (kDqk / 2);
    for (int e = tid; e < kDqk / 2; e += kThreads) d[e] = bf_pack(row[2 * e], row[2 * e + 1]);
    return;
  }
  float a = 0.0f;
  for (int e = tid; e < kDqk; e += kThreads) a = fmaxf(a, finite_abs(row[e]));
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, off));
  if ((tid & 31) == 0) red[tid >> 5] = a;
  __syncthreads();
  a = fmaxf(fmaxf(red[0], red[1]), fmaxf(red[2], red[3]));
  const float s = pow2_scale(a), inv = 1.0f / s;   // both exact
  uint16_t* d = reinterpret_cast<uint16_t*>(c.k) + dst * (kDqk / 2);
  for (int e = tid; e < kDqk / 2; e += kThreads)
    d[e] = (uint16_t)codes2(row[2 * e] * inv, row[2 * e + 1] * inv);
  if (tid == 0) c.ks[dst] = s;
}

// --------------------------------------------------------------- K/V, bf16
// One block per new token: K heads rotated into their page, V heads copied.
// 16 x up to 9 tokens, 8 KV heads, 64 query heads: 3.2 us, the launch's.
__global__ void __launch_bounds__(kThreads, 10) gqa_append_kernel(const uint16_t* k, long long ks,
                                                              const uint16_t* v, long long vs,
                                                              Cache c, Tokens t, RopeArgs r,
                                                              Rows q, int cache_blocks,
                                                              Div items) {
  __shared__ float2 cs[kGD / 2];
  griddep_wait();
  griddep_launch_dependents();
  if ((int)blockIdx.x >= cache_blocks) {
    query_block(q, t, r, blockIdx.x - cache_blocks, cs);
    return;
  }
  const int tok = blockIdx.x, b = tok / t.q_len, i = tok - b * t.q_len;
  const int n = new_count(t, b, c.err);
  if (i >= n) return;
  const int p = t.seq_lens[b] - n + i;
  if (p < 0) {
    if (threadIdx.x == 0) atomicOr(c.err, kErrQLens);
    return;
  }
  if (p % c.num_shards != c.shard) return;
  const int lp = p / c.num_shards, page = page_of(c, b, lp);
  if (page < 0) return;
  const size_t dst = ((size_t)page * kPage + lp % kPage) * c.Hkv * kGD;
  fill_cs(r, rope_pos(t, b, i, p), cs, threadIdx.x, kThreads);
  __syncthreads();
  turn_heads(k + tok * ks, reinterpret_cast<uint16_t*>(c.k) + dst, kGD, 0, c.Hkv, r, items,
             cs, threadIdx.x, kThreads);
  const uint4* s = reinterpret_cast<const uint4*>(v + tok * vs);
  uint4* d = reinterpret_cast<uint4*>(reinterpret_cast<uint16_t*>(c.v) + dst);
  for (int e = threadIdx.x; e < c.Hkv * (kGD / 8); e += kThreads) d[e] = s[e];
}

// --------------------------------------------------------------- K/V, e4m3
// A block takes one block of token slots of a request that the new tokens
// touch, K or V, and as many KV heads as its four warps hold: a warp has 16
// tokens of a head (8 dims a lane, two tokens a load) in registers, from the
// one read to the codes, so a head takes block / 16 warps.  The block's warps
// share one table of its tokens' sines and cosines: computed for every head
// again (one head a block), they cost more than the memory does (4091 tokens x
// 8 heads, 23.5 us against 12.7, and 10.7 with fewer operations a value).
constexpr int kF8Warps = 4;

__global__ void __launch_bounds__(32 * kF8Warps, 4)
    gqa_append_fp8_kernel(const uint16_t* k, long long ks, const uint16_t* v, long long vs, Cache c,
                          Tokens t, RopeArgs r, Rows q, int cache_blocks, Div nblk, Div hgroups,
                          Div wph) {
  // per token: (cos, sin) of two pairs, those of the 16 (or 8) lanes that turn
  // them side by side
  __shared__ float4 cs[kPage][kGD / 4];
  __shared__ float red[kF8Warps];
  griddep_wait();
  griddep_launch_dependents();
  if ((int)blockIdx.x >= cache_blocks) {
    query_block(q, t, r, blockIdx.x - cache_blocks, reinterpret_cast<float2*>(cs));
    return;
  }
  int u = blockIdx.x;
  const bool is_v = u & 1;
  u >>= 1;
  const int hg = u % hgroups;
  u = u / hgroups;
  const int j = u % nblk, b = u / nblk;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int n = new_count(t, b, c.err);
  const int L = t.seq_lens[b], N = c.num_shards, lg_block = 31 - __clz(c.block);
  if (L < n && threadIdx.x == 0) atomicOr(c.err, kErrQLens);
  // local slots [p0, p1) of this shard are new: positions max(L - n, 0) .. L - 1
  const int first_new = max(L - n, 0);
  const int p0 = first_new > c.shard ? (first_new - c.shard - 1) / c.num_shards + 1 : 0;
  const int p1 = L > c.shard ? (L - 1 - c.shard) / c.num_shards + 1 : 0;
  // counted from the first touched block's start: slots go up to 2^31 - 2
  const int start = p0 & ~(c.block - 1), off = j * c.block;
  const int nt = min(p1 - start, off + c.block) - max(p0 - start, off);
  if (nt <= 0) return;
  const int slot0 = start + off, lo = max(p0, slot0);
  const int page = page_of(c, b, slot0);
  if (page < 0) return;
  const int row0 = slot0 % kPage;
  const int W = wph, wh = warp % wph;            // warps of a head, and this one among them
  const int kh = hg * (kF8Warps / W) + warp / wph;
  const bool live = kh < c.Hkv;
  const int half = lane >> 4, l16 = lane & 15;
  auto token = [&](int p) { return p * N + c.shard - (L - n); };   // its place in the new ones

  // the warp's tokens: lo + 2 (i W + wh) + half for i < 8
  uint4 w[8];
  const uint16_t* x = (is_v ? v : k) + (size_t)kh * kGD + 8 * l16;
  const long long xs = is_v ? vs : ks;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int tt = 2 * (i * W + wh) + half;
    w[i] = make_uint4(0, 0, 0, 0);
    if (live && tt < nt)
      w[i] = __ldg(reinterpret_cast<const uint4*>(x + ((size_t)b * t.q_len + token(lo + tt)) * xs));
  }
  const bool had = lo > slot0;
  float* sp = (is_v ? c.vs : c.ks) + (((size_t)page * kPage + row0) >> lg_block) * c.Hkv + kh;
  const float old = had && live ? *sp : 0.0f;

  const bool turn = !is_v && r.rot > 0;
  // lanes that turn a pair's side: 8 dims each, all pairs' (interleaved) or
  // the lower sides' first (half)
  const int r8 = r.rot >> 3, nl = r.interleaved ? r8 : r8 >> 1;
  if (turn) {
    const int lg = r.interleaved ? 2 : 3;        // log2 of a lane's pairs
    for (int p = lane; p < r.rot / 2; p += 32) {
      const unsigned long long rate = turn_rate(__ldg(r.inv_freq + p));
      const int at = ((p & ((1 << lg) - 1)) >> 1) * nl + (p >> lg);
      for (int tt = warp; tt < nt; tt += kF8Warps) {
        const int i = token(lo + tt);
        reinterpret_cast<float2*>(&cs[tt][at])[p & 1] =
            turn_cs(rate, rope_pos(t, b, i, L - n + i), r.factor);
      }
    }
    __syncthreads();
  }
  const int li = l16 - (r.first >> 3);           // the lane's place in the rotated dims
  const bool turns = turn && li >= 0 && li < r8;
  const bool upper = !r.interleaved && li >= nl;
  const int lc = upper ? li - nl : li;
  const int partner = turns && !r.interleaved ? (upper ? lane - nl : lane + nl) : lane;
  float f[8][8];
  float amax = 0.0f;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int tt = 2 * (i * W + wh) + half;
    const uint32_t* p = &w[i].x;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      f[i][2 * e] = bf_lo(p[e]);
      f[i][2 * e + 1] = bf_hi(p[e]);
    }
    if (2 * (i * W + wh) < nt && turn) {
      if (r.interleaved) {
        if (turns) {
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const float4 z = cs[tt][e * nl + lc];
            turn_pair(f[i][4 * e], f[i][4 * e + 1], make_float2(z.x, z.y));
            turn_pair(f[i][4 * e + 2], f[i][4 * e + 3], make_float2(z.z, z.w));
          }
        }
      } else {
        uint32_t o[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) o[e] = __shfl_sync(0xffffffffu, p[e], partner);
        if (turns) {
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float4 z = cs[tt][e * nl + lc];
            float o0 = bf_lo(o[e]), o1 = bf_hi(o[e]);
            float &a0 = f[i][2 * e], &a1 = f[i][2 * e + 1];
            if (upper) {
              turn_pair(o0, a0, make_float2(z.x, z.y));
              turn_pair(o1, a1, make_float2(z.z, z.w));
            } else {
              turn_pair(a0, o0, make_float2(z.x, z.y));
              turn_pair(a1, o1, make_float2(z.z, z.w));
            }
          }
        }
      }
    }
    if (tt < nt) {
#pragma unroll
      for (int e = 0; e < 8; ++e) amax = fmaxf(amax, fabsf(f[i][e]));   // skips NaN
    }
  }
  // an infinity sets no scale, and its code is NaN
  if (__any_sync(0xffffffffu, amax == INFINITY)) {
    amax = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        if (fabsf(f[i][e]) == INFINITY) f[i][e] = __int_as_float(0x7fffffff);
        if (2 * (i * W + wh) + half < nt) amax = fmaxf(amax, fabsf(f[i][e]));
      }
  }
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, off));
  if (lane == 0) red[warp] = amax;
  __syncthreads();                               // every warp has read the old scale too
  if (!live) return;
  amax = 0.0f;
  for (int e = 0; e < W; ++e) amax = fmaxf(amax, red[warp - wh + e]);
  const float need = pow2_scale(amax);
  const bool grow = had && fabsf(old) < need;
  const float s = had && !grow ? old : need;
  uint8_t* base = (is_v ? c.v : c.k) + (((size_t)page * kPage + row0) * c.Hkv + kh) * kGD + 8 * l16;
  const size_t rs = (size_t)c.Hkv * kGD;
  if (grow) {
    const float g = old / s;                     // s is a power of two: exact
    for (int p = 2 * wh + half; p < lo - slot0; p += 2 * W) {
      uint2* d = reinterpret_cast<uint2*>(base + p * rs);
      uint32_t z[2] = {d->x, d->y};
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float y[4];
        e4m3x2_to_f32x2(z[e], y[0], y[1]);
        e4m3x2_to_f32x2(z[e] >> 16, y[2], y[3]);
        z[e] = codes2(y[0] * g, y[1] * g) | (codes2(y[2] * g, y[3] * g) << 16);
      }
      *d = make_uint2(z[0], z[1]);
    }
  }
  // a power of two, as this kernel writes them, has an exact inverse
  const uint32_t sb = __float_as_uint(s);
  const bool exact = (sb & 0x807FFFFFu) == 0 && sb >= (1u << 23) && sb <= (253u << 23);
  const float inv = exact ? __uint_as_float((254u << 23) - sb) : 1.0f;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int tt = 2 * (i * W + wh) + half;
    if (tt >= nt) break;
    if (exact) {
#pragma unroll
      for (int e = 0; e < 8; ++e) f[i][e] *= inv;
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) f[i][e] /= s;
    }
    *reinterpret_cast<uint2*>(base + (lo - slot0 + tt) * rs) =
        make_uint2(f32x2_to_e4m3x2(f[i][0], f[i][1]) | (f32x2_to_e4m3x2(f[i][2], f[i][3]) << 16),
                   f32x2_to_e4m3x2(f[i][4], f[i][5]) | (f32x2_to_e4m3x2(f[i][6], f[i][7]) << 16));
  }
  if (wh == 0 && lane == 0) *sp = s;
}

// ------------------------------------------------------------------ host side
bool tokens_ok(const mla_tokens* t, bool need_lens) {
  using host::aligned4;
  if (t == nullptr || t->batch < 1 || t->q_len < 1) return false;
  if (t->seq_lens == nullptr && (need_lens || t->positions == nullptr)) return false;
  if (!aligned4(t->seq_lens) || !aligned4(t->q_lens) || !aligned4(t->positions)) return false;
  return (long long)t->batch * t->q_len < (1LL << 24);
}

bool rope_ok(const mla_rope* r, int D) {
  if (r->inv_freq == nullptr || (reinterpret_cast<uintptr_t>(r->inv_freq) & 7u)) return false;
  if (r->interleaved != 0 && r->interleaved != 1) return false;
  if (!std::isfinite(r->attention_factor)) return false;
  return r->rot_dim >= 2 && r->rot_dim <= D && r->first_dim >= 0 && r->first_dim <= D - r->rot_dim;
}

bool rope_supported(const mla_rope* r) { return r->rot_dim % 16 == 0 && r->first_dim % 8 == 0; }

Tokens make_tokens(const mla_tokens* t) {
  return Tokens{t->batch, t->q_len, t->seq_lens, t->q_lens, t->positions};
}

RopeArgs make_rope(const mla_rope* r) {
  if (r == nullptr) return RopeArgs{nullptr, 0, 0, 0, 1.0f};
  return RopeArgs{r->inv_freq, r->rot_dim, r->first_dim, r->interleaved, r->attention_factor};
}

bool rows_ok(const void* x, long long xs, long long width) {
  return x != nullptr && host::aligned16(x) && xs >= width && xs % 8 == 0 && xs < (1LL << 32);
}

// Query rows to rotate in an append call: checked, `out` filled.
mla_status make_rows(const void* q, long long qs, void* y, long long ys, int heads, int D,
                     const mla_tokens* t, const mla_rope* r, Rows& out) {
  if (heads < 1 || heads > (1 << 16)) return MLA_ERR_INVALID;
  const long long width = (long long)heads * D;
  if (!rows_ok(q, qs, width) || !rows_ok(y, ys, width)) return MLA_ERR_INVALID;
  if (q == y && qs != ys) return MLA_ERR_INVALID;
  // about 8 KB of a token's heads to a block
  out = Rows{static_cast<const uint16_t*>(q), static_cast<uint16_t*>(y), qs, ys, heads, D,
             make_div(std::min(heads, std::max(1, heads * D / 4096))),
             make_div(head_items(D, r->rot_dim, r->interleaved, q == y))};
  if ((long long)t->batch * t->q_len * out.split >= (1LL << 30)) return MLA_ERR_INVALID;
  return MLA_OK;
}

// The checks that both cache appends share; fills everything but the cache.
mla_status append_args(const int32_t* block_table, int max_pages, const mla_tokens* tokens,
                       const mla_rope* rope, int D, const void* q, long long qs, void* q_out,
                       long long qos, int heads, int shard, int num_shards, void* workspace,
                       size_t workspace_bytes, int num_pages, int page_size, Rows& rows) {
  if (!tokens_ok(tokens, true) || block_table == nullptr || !host::aligned4(block_table) ||
      max_pages < 1 || num_pages < 1)
    return MLA_ERR_INVALID;
  if (num_shards < 1 || num_shards > kMaxShards || shard < 0 || shard >= num_shards)
    return MLA_ERR_INVALID;
  if (rope != nullptr && !rope_ok(rope, D)) return MLA_ERR_INVALID;
  if (rope != nullptr && !rope_supported(rope)) return MLA_ERR_UNSUPPORTED;
  if (page_size != kPage) return MLA_ERR_UNSUPPORTED;
  rows = Rows{nullptr, nullptr, 0, 0, 0, D, make_div(1), make_div(1)};
  if (q != nullptr) {
    if (rope == nullptr) return MLA_ERR_INVALID;
    const mla_status st = make_rows(q, qs, q_out, qos, heads, D, tokens, rope, rows);
    if (st != MLA_OK) return st;
  }
  if (workspace == nullptr || !host::aligned16(workspace) || workspace_bytes < sizeof(WsHeader))
    return MLA_ERR_WORKSPACE;
  return MLA_OK;
}

// Launches that may begin while the kernel before them ends (their
// griddep_wait() waits for its results).
template <class... P, class... A>
mla_status launch(void (*kernel)(P...), unsigned blocks, unsigned threads, void* stream, A... args) {
  cudaLaunchAttribute attr = pdl_attribute();
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(blocks);
  cfg.blockDim = dim3(threads);
  cfg.stream = static_cast<cudaStream_t>(stream);
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, static_cast<P>(args)...) == cudaSuccess ? MLA_OK
                                                                                  : MLA_ERR_CUDA;
}

}  // namespace append
}  // namespace mla

using namespace mla;

extern "C" {

mla_status mla_rope_apply(const void* x, long long x_stride, void* out, long long out_stride,
                          const mla_tokens* tokens, int num_heads, int head_dim,
                          const mla_rope* rope, void* stream) {
  if (!append::tokens_ok(tokens, false) || rope == nullptr) return MLA_ERR_INVALID;
  if (head_dim < 1 || !append::rope_ok(rope, head_dim)) return MLA_ERR_INVALID;
  if (head_dim % 8 != 0 || head_dim > 2 * append::kMaxPairs || !append::rope_supported(rope))
    return MLA_ERR_UNSUPPORTED;
  append::Rows q;
  const mla_status st =
      append::make_rows(x, x_stride, out, out_stride, num_heads, head_dim, tokens, rope, q);
  if (st != MLA_OK) return st;
  return append::launch(append::rope_kernel, tokens->batch * tokens->q_len * q.split,
                        append::kThreads, stream, q, append::make_tokens(tokens),
                        append::make_rope(rope));
}

mla_status mla_cache_append(const void* latent, long long latent_stride, const mla_kv_pages* kv,
                            const int32_t* block_table, int max_pages_per_req,
                            const mla_tokens* tokens, const mla_rope* rope, const void* q,
                            long long q_stride, void* q_out, long long q_out_stride,
                            int num_heads, int shard_id, int num_shards, void* workspace,
                            size_t workspace_bytes, void* stream) {
  if (kv == nullptr || kv->data == nullptr || !host::aligned16(kv->data)) return MLA_ERR_INVALID;
  if (!append::rows_ok(latent, latent_stride, kDqk)) return MLA_ERR_INVALID;
  if (kv->dtype != MLA_KV_BF16 && kv->dtype != MLA_KV_FP8_E4M3) return MLA_ERR_INVALID;
  if ((kv->dtype == MLA_KV_FP8_E4M3) != (kv->scale != nullptr) || !host::aligned4(kv->scale))
    return MLA_ERR_INVALID;
  append::Rows rows;
  const mla_status st = append::append_args(block_table, max_pages_per_req, tokens, rope, kDqk, q,
                                            q_stride, q_out, q_out_stride, num_heads, shard_id,
                                            num_shards, workspace, workspace_bytes, kv->num_pages,
                                            kv->page_size, rows);
  if (st != MLA_OK) return st;
  const append::Cache c{static_cast<uint8_t*>(const_cast<void*>(kv->data)), nullptr,
                        const_cast<float*>(kv->scale), nullptr, kv->dtype == MLA_KV_FP8_E4M3, 1,
                        kv->num_pages, 1, block_table, max_pages_per_req, shard_id, make_div(num_shards),
                        &static_cast<WsHeader*>(workspace)->err};
  const int n = tokens->batch * tokens->q_len;
  return append::launch(append::latent_append_kernel, n + (rows.heads ? n * rows.split : 0),
                        append::kThreads, stream, static_cast<const uint16_t*>(latent),
                        latent_stride, c, append::make_tokens(tokens), append::make_rope(rope),
                        rows, n);
}

mla_status gqa_cache_append(const void* k, long long k_stride, const void* v, long long v_stride,
                            const gqa_block_pages* cache, const int32_t* block_table,
                            int max_pages_per_req, const mla_tokens* tokens, const mla_rope* rope,
                            const void* q, long long q_stride, void* q_out,
                            long long q_out_stride, int num_heads, int shard_id, int num_shards,
                            void* workspace, size_t workspace_bytes, void* stream) {
  using append::kGD;
  if (cache == nullptr || cache->k == nullptr || cache->v == nullptr ||
      !host::aligned16(cache->k) || !host::aligned16(cache->v))
    return MLA_ERR_INVALID;
  if (cache->num_kv_heads < 1 || cache->num_kv_heads > (1 << 16)) return MLA_ERR_INVALID;
  const long long width = (long long)cache->num_kv_heads * kGD;
  if (!append::rows_ok(k, k_stride, width) || !append::rows_ok(v, v_stride, width))
    return MLA_ERR_INVALID;
  if (cache->dtype != MLA_KV_BF16 && cache->dtype != MLA_KV_FP8_E4M3) return MLA_ERR_INVALID;
  const bool fp8 = cache->dtype == MLA_KV_FP8_E4M3;
  if (fp8 != (cache->k_scale != nullptr) || fp8 != (cache->v_scale != nullptr) ||
      !host::aligned4(cache->k_scale) || !host::aligned4(cache->v_scale))
    return MLA_ERR_INVALID;
  if (fp8 && (cache->block < 1 || cache->block > kPage || (cache->block & (cache->block - 1))))
    return MLA_ERR_INVALID;
  append::Rows rows;
  const mla_status st = append::append_args(block_table, max_pages_per_req, tokens, rope, kGD, q,
                                            q_stride, q_out, q_out_stride, num_heads, shard_id,
                                            num_shards, workspace, workspace_bytes,
                                            cache->num_pages, cache->page_size, rows);
  if (st != MLA_OK) return st;
  const append::Cache c{static_cast<uint8_t*>(cache->k), static_cast<uint8_t*>(cache->v),
                        cache->k_scale, cache->v_scale, fp8, fp8 ? cache->block : kPage,
                        cache->num_pages, cache->num_kv_heads, block_table, max_pages_per_req,
                        shard_id, make_div(num_shards), &static_cast<WsHeader*>(workspace)->err};
  const int n = tokens->batch * tokens->q_len;
  const int qb = rows.heads ? n * rows.split : 0;
  const uint16_t *kp = static_cast<const uint16_t*>(k), *vp = static_cast<const uint16_t*>(v);
  const RopeArgs r = append::make_rope(rope);
  if (!fp8)
    return append::launch(append::gqa_append_kernel, n + qb, append::kThreads, stream, kp, k_stride,
                          vp, v_stride, c, append::make_tokens(tokens), r, rows, n,
                          make_div(append::head_items(kGD, r.rot, r.interleaved, false)));
  // blocks that ceil(q_len / N) consecutive local slots can touch
  const int local = ceil_div(tokens->q_len, num_shards);
  const int nblk = (local + cache->block - 2) / cache->block + 1;
  const int wph = std::max(1, cache->block / 16);
  const int hgroups = ceil_div(cache->num_kv_heads, append::kF8Warps / wph);
  const long long blocks = 2LL * tokens->batch * nblk * hgroups;
  if (blocks + qb >= (1LL << 31)) return MLA_ERR_INVALID;
  return append::launch(append::gqa_append_fp8_kernel, (unsigned)(blocks + qb),
                        32 * append::kF8Warps, stream, kp, k_stride, vp, v_stride, c,
                        append::make_tokens(tokens), r, rows, (int)blocks, make_div(nblk),
                        make_div(hgroups), make_div(wph));
}

}  // extern "C"
