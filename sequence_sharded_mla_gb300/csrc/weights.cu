// The attention weight that a step gives to every cached token:
//
//   w_t = sum over the step's rows (i, h) that see t of exp(s_t - lse[i, h]),
//   s_t = softmax_scale * q[i, h] . K_t,
//
// with the step's own log-sum-exps (of the combine), added to what earlier
// steps gave.  What an eviction by accumulated weight selects by.
//
// Work is a list of (request, tile of 128 tokens), split over one persistent
// CTA per SM.  S^T = K Q^T on the tensor cores, M = 128 tokens, N = a group of
// 64 or 128 query rows, K = 576: a TMEM lane is a token and its columns are
// the rows, so the sum over rows stays inside a thread (fixed order, nothing
// to exchange) and every thread ends with one token's weight.
//
//   warp 0      K producer, two pages a tile, by TMA: boxes of three 64-dim chunks
//               a page; e4m3, whole pages (in 192-byte pieces of the
//               576-byte rows a million tokens took 119 instead of 105 us)
//   warp 1      MMA issue
//   warps 2..5  one token a thread: exp2 of every column, summed
//   warp 6      Q producer: a group's nine chunks.  A request of one group of
//               64 rows keeps them for all its tiles; with more rows they pass
//               through the ring once per tile and group (out of L2) while the
//               tile's keys stay
//
// e4m3 caches: the codes as they are, the query as two-term e4m3 sums
// (qterms.cuh), hi and lo terms as neighbouring MMA rows; the thread adds their
// two columns and multiplies by the token's scale.
//
// What bounds it: with one query token, memory bandwidth (1152 or 580 bytes a
// token); with hundreds of rows, the tensor cores and the operands' way to them.
#include <math_constants.h>

#include <algorithm>
#include <cmath>
#include <cstdint>

#include "common.cuh"
#include "host_util.h"
#include "mla_dcp.h"
#include "ptx.cuh"
#include "qterms.cuh"

namespace mla {
namespace weights {

constexpr int kThreads = 224;
constexpr int kTokens = 128;               // tokens per tile: MMA M
constexpr int kMaxDepth = 3;
constexpr uint32_t kBarSum = 1;            // named barrier of the summing warps
constexpr int kSumThreads = 128;
constexpr uint32_t kTmemCols = 512;        // two accumulators of up to 256 columns
constexpr int kPrepThreads = 1024;
constexpr int kUnitCost = 1;
constexpr float kLog2e = 1.4426950408889634f;

struct Params {
  int B, q_len, H, R, causal;
  int max_pages, num_pages;
  int width;                               // tokens per row of the weights
  float scale_log2;
  const int32_t* block_table;
  const int32_t* seq_lens;
  const int32_t* q_lens;                   // or null
  const float* lse;                        // [B, q_len, H]
  const float* kv_scale;                   // e4m3: [num_pages * 64]
  const uint16_t* q;                       // [B * R, 576]
  uint8_t* terms;                          // e4m3: [B * R, 2, 576]
  float* inv_scale;                        // e4m3: [B * R]
  const float* before;                     // earlier weights, or null
  long long before_stride;
  float* out;
  long long out_stride;
  WsHeader* hdr;
  int* prefix;                             // [B + 1]
  unsigned long long timeout_ns;
  int withhold_query;                      // testing aid: the query is never loaded
};

__device__ __forceinline__ int context(const Params& p, int b) {
  const long long room = min((long long)p.width, (long long)p.max_pages * kPage);
  return (int)max(0LL, min((long long)p.seq_lens[b], room));
}
__device__ __forceinline__ int new_tokens(const Params& p, int b) {
  return p.q_lens != nullptr ? min(max(p.q_lens[b], 1), p.q_len) : p.q_len;
}

// Block 0: the work list.  The others (e4m3): a query row per warp.
template <int kRowsN>
__global__ void __launch_bounds__(kPrepThreads) weights_prep_kernel(Params p, int grid) {
  griddep_launch_dependents();
  if (blockIdx.x > 0) {
    const int row = ((int)blockIdx.x - 1) * (kPrepThreads / 32) + (threadIdx.x >> 5);
    if (row >= p.B * p.R) return;
    const int b = row / p.R;
    griddep_wait();
    split_query_row(p.q + (size_t)row * kDqk, row - b * p.R < new_tokens(p, b) * p.H,
                    p.terms + (size_t)row * 2 * kDqk, p.inv_scale + row, threadIdx.x & 31);
    return;
  }
  __shared__ unsigned bad;
  if (threadIdx.x == 0) bad = 0;
  __syncthreads();
  griddep_wait();
  for (int b = threadIdx.x; b < p.B; b += kPrepThreads) {
    const bool ql = p.q_lens != nullptr && p.q_lens[b] != new_tokens(p, b);
    if (ql || context(p, b) != p.seq_lens[b]) atomicOr(&bad, kErrQLens);
  }
  __syncthreads();
  // a request's positions: its tiles times its groups of rows
  plan_units(
      p.B,
      [&](int b) {
        return ceil_div(context(p, b), kTokens) * ceil_div(new_tokens(p, b) * p.H, kRowsN);
      },
      p.hdr, p.prefix, grid, 1, kUnitCost, bad);
}

struct Misc {
  uint64_t kf[kMaxDepth], ke[kMaxDepth];   // K ring
  uint64_t qf[kChunks], qe[kChunks];       // Q ring
  uint64_t df[2], de[2];                   // accumulators
  uint64_t drain;
  uint32_t tmem_base;
  int abort;
  alignas(16) float row_lse[2][128];       // log2 units, by parity of (tile, group)
  alignas(16) float row_f[2][128];         // e4m3: 1 / s_r, in log2 units of the logit
};

// kRowsN: query rows per group.  An MMA has kRowsN columns (bf16), or twice as
// many (e4m3: both terms of a row).
template <bool kFp8, int kRowsN>
struct Cfg {
  static constexpr int kN = kFp8 ? 2 * kRowsN : kRowsN;
  static constexpr int kLine = kFp8 ? 64 : 128;            // bytes of a chunk's row
  // a slot of K: [16 groups of 8 tokens][kCg chunks][8 tokens][64 dims]
  static constexpr int kCg = kFp8 ? kChunks : 3;
  static constexpr int kKGroup = kCg * 8 * kLine;
  static constexpr int kKBytes = kTokens / 8 * kKGroup;    // 72 or 48 KB
  static constexpr int kQBytes = kN * kLine;               // Q chunk: 8 or 16 KB
  // with more than 64 rows the query's chunks stream (one tile of e4m3 keys and
  // nine chunks of the query in flight took 2 us more of a 9-token step's 54)
  static constexpr int kKDepth = kFp8 ? 2 : 3;
  static constexpr int kQDepth = kRowsN == 64 ? 9 : 4;
  static constexpr int kSmemQ = kKDepth * kKBytes;
  static constexpr int kSmemMisc = kSmemQ + kQDepth * kQBytes;
  static constexpr int kSmem = kSmemMisc + (int)sizeof(Misc) + 1024;
  static_assert(kSmem <= 232448, "shared memory");
};

// The pieces of one CTA: request, tiles [t0, t1), groups of rows.
struct Walk {
  PieceIter it;
  __device__ void init(const Params& p) {
    const int W = p.hdr->total_cost, per = p.hdr->per_cta;
    const int lo = (int)min((long long)W, (long long)blockIdx.x * per);
    it.init(p.prefix, p.B, lo, (int)min((long long)W, (long long)lo + per), p.hdr->unit_cost);
  }
  template <int kRowsN>
  __device__ bool next(const Params& p, int& b, int& L, int& rows, int& groups, int& t0, int& t1) {
    bool whole;
    int slot, a, z;
    while (it.next(b, a, z, whole, slot)) {
      L = context(p, b);
      rows = new_tokens(p, b) * p.H;
      groups = ceil_div(rows, kRowsN);
      // the tiles whose first position is this CTA's
      t0 = ceil_div(a, groups);
      t1 = ceil_div(z, groups);
      if (t0 < t1) return true;
    }
    return false;
  }
};

template <bool kFp8, int kRowsN>
__global__ void __launch_bounds__(kThreads, 1)
    weights_kernel(const __grid_constant__ CUtensorMap tm_k,
                   const __grid_constant__ CUtensorMap tm_q, Params p) {
  using C = Cfg<kFp8, kRowsN>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  Misc* misc = reinterpret_cast<Misc*>(smem + C::kSmemMisc);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  volatile int* abort_flag = &misc->abort;
  const uint64_t tmo = p.timeout_ns;
  auto fail = [&]() {
    atomicOr(&p.hdr->err, kErrTimeout);
    *(volatile int*)&misc->abort = 1;
  };
  // one thread's wait: a warp whose 32 lanes poll takes a few times as long
  auto wait = [&](uint64_t* bar, uint32_t parity) {
    return mbar_wait(smem_u32(bar), parity, tmo, abort_flag);
  };

  if (threadIdx.x == 0) {
    for (int i = 0; i < kMaxDepth; ++i) {
      mbar_init(smem_u32(&misc->kf[i]), 1);
      mbar_init(smem_u32(&misc->ke[i]), 1);
    }
    for (int i = 0; i < kChunks; ++i) {
      mbar_init(smem_u32(&misc->qf[i]), 1);
      mbar_init(smem_u32(&misc->qe[i]), 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_u32(&misc->df[i]), 1);
      mbar_init(smem_u32(&misc->de[i]), 4);
    }
    mbar_init(smem_u32(&misc->drain), 1);
    misc->abort = 0;
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(&misc->tmem_base), kTmemCols);
    tmem_relinquish();
  }
  if (warp == 0 && lane == 0) {
    tma_prefetch_desc(&tm_k);
    tma_prefetch_desc(&tm_q);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = misc->tmem_base;
  const uint32_t sK = smem_u32(smem), sQ = smem_u32(smem + C::kSmemQ);
  griddep_wait();                // the work list, the query's terms
  griddep_launch_dependents();

  Walk walk;
  walk.init(p);
  int b, L, rows, groups, t0, t1;
  bool ok = true;
  int armed = 0;                 // loads issued into this warp's ring so far
  // a request's only group of 64 rows stays for all the piece's tiles
  constexpr bool stay = kRowsN == 64;

  if (warp == 0) {
    // ---------------------------------------------------------- K producer
    // (one thread; so are the other producer and the issuer)
    if (lane == 0) {
      while (ok && walk.next<kRowsN>(p, b, L, rows, groups, t0, t1)) {
        const int npages = ceil_div(L, kPage);
        const int32_t* bt = p.block_table + (size_t)b * p.max_pages;
        // the table's entries are read a tile ahead
        int e[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) e[h] = 2 * t0 + h < npages ? __ldg(bt + 2 * t0 + h) : -1;
        for (int t = t0; ok && t < t1; ++t) {
          // a page past the context or out of range lies behind the pool, and its
          // rows are zeros
          int group[2];
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const bool valid = e[h] >= 0 && e[h] < p.num_pages;
            if (2 * t + h < npages && !valid) atomicOr(&p.hdr->err, kErrBadPage);
            group[h] = (valid ? e[h] : p.num_pages) * (kPage / 8);
            const int i = 2 * t + 2 + h;
            e[h] = i < npages ? __ldg(bt + i) : -1;
          }
#pragma unroll
          for (int c = 0; c < kChunks / C::kCg; ++c, ++armed) {
            const int s = armed % C::kKDepth, use = armed / C::kKDepth;
            if (use > 0) ok = wait(&misc->ke[s], (use - 1) & 1);
            if (!ok) break;
            const uint32_t bar = smem_u32(&misc->kf[s]);
            mbar_arrive_expect_tx(bar, C::kKBytes);
#pragma unroll
            for (int h = 0; h < 2; ++h)
              tma_load_4d(sK + s * C::kKBytes + h * (C::kKBytes / 2), &tm_k, bar, 0, 0,
                          C::kCg * c, group[h]);
          }
        }
      }
      if (!ok) fail();
    }
  } else if (warp == 6) {
    // ---------------------------------------------------------- Q producer
    if (lane == 0 && !p.withhold_query) {
      while (ok && walk.next<kRowsN>(p, b, L, rows, groups, t0, t1)) {
        for (int t = t0; ok && t < (stay ? t0 + 1 : t1); ++t)
          for (int g = 0; ok && g < groups; ++g)
            for (int c = 0; c < kChunks; ++c, ++armed) {
              const int s = armed % C::kQDepth, use = armed / C::kQDepth;
              if (use > 0) ok = wait(&misc->qe[s], (use - 1) & 1);
              if (!ok) break;
              mbar_arrive_expect_tx(smem_u32(&misc->qf[s]), C::kQBytes);
              tma_load_2d(sQ + s * C::kQBytes, &tm_q, smem_u32(&misc->qf[s]), 64 * c,
                          (b * p.R + g * kRowsN) * (kFp8 ? 2 : 1));
            }
      }
      if (!ok) fail();
    }
  } else if (warp == 1) {
    // ----------------------------------------------------------- MMA issue
    if (lane == 0) {
      constexpr uint32_t kQGroup = 8 * C::kLine;           // eight rows
      constexpr int kSteps = kFp8 ? 2 : 4;                 // 32-byte steps of a chunk
      const uint64_t dk0 = kFp8 ? sw64_desc(sK, 16, C::kKGroup) : sw128_desc(sK, 16, C::kKGroup);
      const uint64_t dq0 = kFp8 ? sw64_desc(sQ, 16, kQGroup) : sw128_desc(sQ, 16, kQGroup);
      int nk = 0, nq = 0, nd = 0;                          // loads and sums so far
      while (ok && walk.next<kRowsN>(p, b, L, rows, groups, t0, t1)) {
        for (int t = t0; ok && t < t1; ++t) {
          for (int g = 0; ok && g < groups; ++g, ++nd) {
            const int buf = nd & 1;
            if (nd >= 2) ok = wait(&misc->de[buf], ((nd >> 1) - 1) & 1);
            const uint32_t d = tmem + 256 * buf;
            // columns of the group's rows: the last of five groups of a 576-row
            // step has half
            const int cols = min(kRowsN, rows - g * kRowsN) * (kFp8 ? 2 : 1);
            const uint32_t id = kFp8 ? idesc_e4m3_f32(kTokens, cols, false, false)
                                     : idesc_bf16_f32(kTokens, cols, false, false);
#pragma unroll 1
            for (int cg = 0; ok && cg < kChunks / C::kCg; ++cg) {
              const int ks = (nk + cg) % C::kKDepth;
              if (g == 0) ok = wait(&misc->kf[ks], ((nk + cg) / C::kKDepth) & 1);
              const uint64_t dk = dk0 + ((ks * C::kKBytes) >> 4);
#pragma unroll
              for (int c = 0; c < C::kCg; ++c) {
                const int i = nq + cg * C::kCg + c, qs = i % C::kQDepth;
                if (ok && (!stay || t == t0)) ok = wait(&misc->qf[qs], (i / C::kQDepth) & 1);
                if (!ok) break;
                tc_fence_after();
                const uint64_t dq = dq0 + ((qs * C::kQBytes) >> 4);
#pragma unroll
                for (int k = 0; k < kSteps; ++k) {
                  const uint64_t a = dk + ((c * 8 * C::kLine + 32 * k) >> 4), q = dq + ((32 * k) >> 4);
                  const uint32_t acc = (cg > 0 || c > 0 || k > 0) ? 1u : 0u;
                  if (kFp8) mma_e4m3_ss(d, a, q, id, acc);
                  else mma_bf16_ss(d, a, q, id, acc);
                }
                if (!stay || t == t1 - 1) mma_commit(smem_u32(&misc->qe[qs]));
              }
              if (ok && g == groups - 1) mma_commit(smem_u32(&misc->ke[ks]));
            }
            if (ok) mma_commit(smem_u32(&misc->df[buf]));
            if (!stay) nq += kChunks;
          }
          nk += kChunks / C::kCg;
        }
        if (stay) nq += kChunks;
      }
      if (!ok) fail();
    }
  } else {
    // ---------------------------------------------------------- summing
    const int quad = warp & 3, tid = 32 * quad + lane;     // the thread's token of a tile
    const uint32_t lane_off = (uint32_t)(32 * quad) << 16;
    int nd = 0, last_b = -1, have = 0;
    while (ok && walk.next<kRowsN>(p, b, L, rows, groups, t0, t1)) {
      const int before_step = L - new_tokens(p, b);         // tokens of earlier steps
      // the thread's row of a group
      float next_l = 0.0f, next_f = 0.0f;
      auto fetch = [&](int g) {
        if (g * kRowsN + tid >= min(rows, (g + 1) * kRowsN)) return;
        const size_t r = (size_t)b * p.R + g * kRowsN + tid;
        next_l = p.lse[r];
        if (kFp8) next_f = p.inv_scale[r];
      };
      if (groups > 1 || b != last_b) fetch(0);
      for (int t = t0; ok && t < t1; ++t) {
        const int tok = t * kTokens + tid;
        // the token's scale and earlier weight: on their way while the MMAs run
        float sigma = 1.0f, sum = 0.0f;
        if (tok < L) {
          if (kFp8) {
            const int page = __ldg(p.block_table + (size_t)b * p.max_pages + tok / kPage);
            if (page >= 0 && page < p.num_pages)
              sigma = __ldg(p.kv_scale + (size_t)page * kPage + tok % kPage);
          }
          if (p.before != nullptr && tok < before_step)
            sum = p.before[(size_t)b * p.before_stride + tok];
        }
        // rows from first_row on see the token
        const bool masked = p.causal && t * kTokens + kTokens - 1 > before_step;
        const int first_row = masked ? max(0, (tok - before_step) * p.H) : 0;
        float w = 0.0f;
        for (int g = 0; ok && g < groups; ++g, ++nd) {
          const int n = min(kRowsN, rows - g * kRowsN);     // a multiple of 16
          // the rows' log-sum-exps (a row that saw nothing gives nothing) and
          // query scales, unless the last group's are this group's; the next
          // group's are on their way meanwhile
          if (groups > 1 || b != last_b) {
            have ^= 1;           // the other buffer: a warp may still read this one
            if (tid < n) {
              misc->row_lse[have][tid] = next_l == -CUDART_INF_F ? CUDART_INF_F : next_l * kLog2e;
              if (kFp8) {
                if (next_f != next_f) atomicOr(&p.hdr->err, kErrQRange);
                misc->row_f[have][tid] = next_f * p.scale_log2;
              }
            }
            last_b = b;
            if (groups > 1) fetch(g + 1 < groups ? g + 1 : 0);
            named_bar_sync(kBarSum, kSumThreads);
          }
          const int buf = nd & 1;
          ok = __all_sync(0xffffffffu, wait(&misc->df[buf], (nd >> 1) & 1));
          if (named_bar_or(kBarSum, kSumThreads, !ok)) {
            ok = false;
            break;
          }
          tc_fence_after();
          float part[4] = {0.f, 0.f, 0.f, 0.f};
          const float* lse = misc->row_lse[have];
          const float* rf = misc->row_f[have];
          for (int r0 = 0; r0 < n; r0 += 16) {
            float s[16];
            if (kFp8) {
              uint32_t v[32];
              tmem_ld32(tmem + lane_off + 256 * buf + 2 * r0, v);
              tmem_wait_ld();
#pragma unroll
              for (int i = 0; i < 16; ++i)
                s[i] = (__uint_as_float(v[2 * i]) + __uint_as_float(v[2 * i + 1])) * sigma;
            } else {
              uint32_t v[16];
              tmem_ld16(tmem + lane_off + 256 * buf + r0, v);
              tmem_wait_ld();
#pragma unroll
              for (int i = 0; i < 16; ++i) s[i] = __uint_as_float(v[i]);
            }
#pragma unroll
            for (int i4 = 0; i4 < 4; ++i4) {
              const float4 l4 = *reinterpret_cast<const float4*>(lse + r0 + 4 * i4);
              float4 f4 = make_float4(p.scale_log2, p.scale_log2, p.scale_log2, p.scale_log2);
              if (kFp8) f4 = *reinterpret_cast<const float4*>(rf + r0 + 4 * i4);
              const float l[4] = {l4.x, l4.y, l4.z, l4.w}, f[4] = {f4.x, f4.y, f4.z, f4.w};
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                const float e = ex2_approx(fmaf(s[4 * i4 + i], f[i], -l[i]));
                part[i] += (!masked || g * kRowsN + r0 + 4 * i4 + i >= first_row) ? e : 0.0f;
              }
            }
          }
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(smem_u32(&misc->de[buf]));
          w += (part[0] + part[1]) + (part[2] + part[3]);
        }
        if (ok && tok < L) p.out[(size_t)b * p.out_stride + tok] = sum + w;
      }
    }
    if (!ok && tid == 0) fail();
  }

  // ---------------------------------------------------------------- teardown
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (*abort_flag) {
    // after a failure, the MMAs and copies in flight land before TMEM is freed
    int never = 0;
    if (warp == 1 && lane == 0) {
      mma_commit(smem_u32(&misc->drain));
      mbar_wait(smem_u32(&misc->drain), 0, kDrainNs, &never);
    }
    if ((warp == 0 || warp == 6) && lane == 0) {
      const int depth = warp == 0 ? C::kKDepth : C::kQDepth;
      for (int i = max(0, armed - depth); i < armed; ++i)
        mbar_wait(smem_u32(warp == 0 ? &misc->kf[i % depth] : &misc->qf[i % depth]),
                  (i / depth) & 1, kDrainNs, &never);
    }
    tc_fence_before();
    __syncthreads();
  }
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
}

struct Layout {
  size_t prefix, terms, inv_scale, total;
};

Layout layout(const mla_shape* s, bool fp8) {
  auto up = [](size_t v) { return (v + 255) & ~static_cast<size_t>(255); };
  const size_t rows = (size_t)s->batch * s->q_len * s->num_heads;
  Layout l;
  l.prefix = up(sizeof(WsHeader));
  l.terms = l.prefix + up(sizeof(int) * ((size_t)s->batch + 1));
  l.inv_scale = l.terms + (fp8 ? up(rows * 2 * kDqk) : 0);
  l.total = l.inv_scale + (fp8 ? up(rows * sizeof(float)) : 0);
  return l;
}

bool shape_ok(const mla_shape* s) {
  return s != nullptr && s->batch >= 1 && s->q_len >= 1 && s->num_heads >= 1 &&
         (s->causal == 0 || s->causal == 1) && std::isfinite(s->softmax_scale) &&
         s->softmax_scale > 0.f && (long long)s->batch * s->q_len * s->num_heads < (1LL << 30);
}

bool encode(CUtensorMap* m, bool fp8, const void* base, int rank, const cuuint64_t* dims,
            const cuuint64_t* strides, const cuuint32_t* box) {
  const cuuint32_t es[4] = {1, 1, 1, 1};
  return host::encode_fn()(m, fp8 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16,
                           rank, const_cast<void*>(base), dims, strides, box, es,
                           CU_TENSOR_MAP_INTERLEAVE_NONE,
                           fp8 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B,
                           fp8 ? CU_TENSOR_MAP_L2_PROMOTION_NONE : CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
                           CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <bool kFp8, int kRowsN>
mla_status run(const Params& p, const void* kv, int grid, cudaStream_t st) {
  using C = Cfg<kFp8, kRowsN>;
  CUtensorMap tm_k, tm_q;
  const void* q = kFp8 ? static_cast<const void*>(p.terms) : p.q;
  const uint64_t rows = (uint64_t)p.B * p.R * (kFp8 ? 2 : 1);
  const cuuint64_t e = kFp8 ? 1 : 2;
  // cache: (64 dims, row of 8, chunk, 8-row group); query: (dim, row)
  const cuuint64_t kd[4] = {64, 8, (cuuint64_t)kChunks, (cuuint64_t)p.num_pages * (kPage / 8)};
  const cuuint64_t ks[3] = {kDqk * e, 64 * e, 8 * kDqk * e};
  const cuuint32_t kb[4] = {64, 8, (cuuint32_t)C::kCg, (cuuint32_t)(kPage / 8)};
  const cuuint64_t qd[2] = {(cuuint64_t)kDqk, rows}, qs[1] = {kDqk * e};
  const cuuint32_t qb[2] = {64, (cuuint32_t)C::kN};
  if (!encode(&tm_k, kFp8, kv, 4, kd, ks, kb) || !encode(&tm_q, kFp8, q, 2, qd, qs, qb))
    return MLA_ERR_CUDA;
  cudaLaunchAttribute attr = pdl_attribute();
  cudaLaunchConfig_t cfg = {};
  cfg.stream = st;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  cfg.gridDim = dim3(1 + (kFp8 ? ceil_div(p.B * p.R, kPrepThreads / 32) : 0));
  cfg.blockDim = dim3(kPrepThreads);
  if (cudaLaunchKernelEx(&cfg, weights_prep_kernel<kRowsN>, p, grid) != cudaSuccess)
    return MLA_ERR_CUDA;
  if (host::ensure_dynamic_smem(reinterpret_cast<const void*>(&weights_kernel<kFp8, kRowsN>),
                                C::kSmem) != cudaSuccess)
    return MLA_ERR_CUDA;
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = C::kSmem;
  return cudaLaunchKernelEx(&cfg, weights_kernel<kFp8, kRowsN>, tm_k, tm_q, p) == cudaSuccess
             ? MLA_OK
             : MLA_ERR_CUDA;
}

}  // namespace weights
}  // namespace mla

using namespace mla;

extern "C" {

size_t mla_attention_weights_workspace_size(const mla_shape* shape, mla_kv_dtype dtype) {
  if (!weights::shape_ok(shape)) return 0;
  if (dtype != MLA_KV_BF16 && dtype != MLA_KV_FP8_E4M3) return 0;
  return weights::layout(shape, dtype == MLA_KV_FP8_E4M3).total;
}

mla_status mla_attention_weights(const void* q, const mla_kv_pages* kv, const int32_t* block_table,
                                 int max_pages_per_req, const int32_t* seq_lens,
                                 const mla_shape* shape, const float* lse, const float* before,
                                 long long before_stride, float* out, long long out_stride,
                                 int width, void* workspace, size_t workspace_bytes, void* stream) {
  using host::aligned16;
  using host::aligned4;
  if (!q || !kv || !block_table || !seq_lens || !lse || !out || !weights::shape_ok(shape))
    return MLA_ERR_INVALID;
  if (kv->data == nullptr || kv->num_pages < 1 || max_pages_per_req < 1) return MLA_ERR_INVALID;
  if (kv->dtype != MLA_KV_BF16 && kv->dtype != MLA_KV_FP8_E4M3) return MLA_ERR_INVALID;
  const bool fp8 = kv->dtype == MLA_KV_FP8_E4M3;
  if (fp8 != (kv->scale != nullptr) || !aligned4(kv->scale)) return MLA_ERR_INVALID;
  if (!aligned16(q) || !aligned16(kv->data) || !aligned4(block_table) || !aligned4(seq_lens) ||
      !aligned4(shape->q_lens) || !aligned4(lse) || !aligned4(before) || !aligned4(out))
    return MLA_ERR_INVALID;
  if (width < 1 || out_stride < width || (before != nullptr && before_stride < width))
    return MLA_ERR_INVALID;
  if (kv->page_size != kPage || shape->num_heads % 16 != 0) return MLA_ERR_UNSUPPORTED;
  // rows of both query terms, cache rows and work positions are 32-bit numbers
  const int R = shape->q_len * shape->num_heads;
  const int n = R <= 64 ? 64 : 128;
  const long long tiles = (std::min((long long)width, (long long)max_pages_per_req * kPage) - 1) /
                              weights::kTokens + 1;
  if (kv->num_pages > (1 << 24) || width > (1 << 30) || (long long)shape->batch * R >= (1LL << 29) ||
      shape->batch * (tiles * ceil_div(R, n) + weights::kUnitCost) >= (1LL << 31))
    return MLA_ERR_UNSUPPORTED;
  // earlier weights are read where they are written, or apart
  if (before != nullptr && (before != out || before_stride != out_stride)) {
    const uintptr_t a = reinterpret_cast<uintptr_t>(before), z = reinterpret_cast<uintptr_t>(out);
    const size_t na = sizeof(float) * ((shape->batch - 1) * (size_t)before_stride + width);
    const size_t nz = sizeof(float) * ((shape->batch - 1) * (size_t)out_stride + width);
    if (a < z + nz && z < a + na) return MLA_ERR_INVALID;
  }
  const weights::Layout l = weights::layout(shape, fp8);
  if (workspace == nullptr || !aligned16(workspace) || workspace_bytes < l.total)
    return MLA_ERR_WORKSPACE;
  const int grid = host::device_sm_count();
  if (grid <= 0 || host::encode_fn() == nullptr) return MLA_ERR_CUDA;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  weights::Params p;
  p.B = shape->batch;
  p.q_len = shape->q_len;
  p.H = shape->num_heads;
  p.R = R;
  p.causal = shape->causal;
  p.max_pages = max_pages_per_req;
  p.num_pages = kv->num_pages;
  p.width = width;
  p.scale_log2 = shape->softmax_scale * weights::kLog2e;
  p.block_table = block_table;
  p.seq_lens = seq_lens;
  p.q_lens = shape->q_lens;
  p.lse = lse;
  p.kv_scale = kv->scale;
  p.q = static_cast<const uint16_t*>(q);
  p.terms = ws + l.terms;
  p.inv_scale = reinterpret_cast<float*>(ws + l.inv_scale);
  p.before = before;
  p.before_stride = before_stride;
  p.out = out;
  p.out_stride = out_stride;
  p.hdr = reinterpret_cast<WsHeader*>(ws);
  p.prefix = reinterpret_cast<int*>(ws + l.prefix);
  p.timeout_ns = host::wait_budget_ns(2000000000ull);
  p.withhold_query = host::g_withhold_query.load();
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (fp8)
    return n == 64 ? weights::run<true, 64>(p, kv->data, grid, st)
                   : weights::run<true, 128>(p, kv->data, grid, st);
  return n == 64 ? weights::run<false, 64>(p, kv->data, grid, st)
                 : weights::run<false, 128>(p, kv->data, grid, st);
}

}  // extern "C"
