// Attention of a batch over long prefixes that its requests share: the shared
// pages are attended once for all the rows of a group of requests, in tiles of
// 128 rows, instead of once per request.
//
//   o = sum_t exp(s_t - lse) c_t,  lse = ln sum_t exp(s_t),  s_t = scale q . K_t
//
// over the group's shared pages, for every query row of its requests.  What
// lies behind them (the requests' own tokens) the per-request kernel attends;
// the two partials meet in the LSE combine, as two shards do.
//
// A group of many rows is bounded by the tensor cores, not by memory: 128 rows
// do 242 operations for every byte of a bf16 row.  An accumulator of 128 rows x
// 512 dims would fill a CTA's tensor memory, so two CTAs (a cluster of two, one
// per SM) hold it between them, 64 rows each, and their tensor cores work
// together (cta_group::2, M = 128): each CTA gives the MMAs its 64 rows of A
// and half of B.
//
//   S = Q K^T   N = 128 tokens: CTA r gives page 2j + r (all 576 dims)
//   O += P V    K = 128 tokens, N = 256 dims, twice: CTA r gives the dims
//               256 r .. 256 r + 255 of both pages
//
// Both descriptors mean the same offset in both CTAs, which fixes the tile's
// place in shared memory: the nine 64-dim chunks of the CTA's own page, A =
// chunks 0-3, B = chunks 4-7, C = chunk 8 (rope).  P V reads page 2j at A and
// page 2j + 1 at B.  CTA 0 keeps its A (its dims of its page) and, once S is
// done, loads its dims of page 2j + 1 over B; CTA 1 keeps B and loads over A.
// So a tile costs a CTA 13 chunks of loads and 9 of space.
//
//   warp 0      K producer: the query, and the tiles ahead
//   warps 1, 2  S issue (leader only): half of every chunk's products each, into an
//               accumulator each -- one thread issues an MMA every 44 cycles or
//               so, and one of M = 128, N = 128 takes 33
//   warp 12     P V issue (leader only)
//   warp 3      V producer; e4m3: the tile's token scales, split into mantissa
//               and exponent
//   warps 4..11 softmax: a thread has one row and 32 tokens; the four threads of
//               a row exchange their maxima; O is rescaled only when a tile's is
//               2^8 above the reference (e4m3: or far below); the epilogue
//
// e4m3 caches: the MMAs take the codes as they are, the query and the
// probabilities as two-term e4m3 sums, as in the per-request kernel; three
// stages.  bf16: two stages, probabilities in the stage's rope chunk (tokens
// 0-63) and one chunk of their own (64-127).
//
// Work is (group, 128 rows, tile of 128 tokens), split evenly over the pairs;
// pieces of a unit that was split are joined by their LSEs.
#include <cuda_bf16.h>
#include <math_constants.h>

#include <algorithm>
#include <cstddef>

#include "common.cuh"
#include "host_util.h"
#include "merge.cuh"
#include "pair.cuh"
#include "prefix.h"
#include "ptx.cuh"
#include "qterms.cuh"
#include "unit_merge.cuh"

namespace mla {
namespace prefix {

namespace {

constexpr int kSoftmaxWarps = 8;             // warps 4 .. 11
constexpr int kThreads = 32 * (4 + kSoftmaxWarps + 1);
constexpr int kHalf = 64;                    // rows, and tokens of a tile, per CTA
constexpr int kPrepThreads = 1024;
// Work positions charged to a unit for its fixed costs (query load, pipeline
// refill, the epilogue's 256 KB of output).
constexpr int kUnitCost = 3;
constexpr int kMinTiles = 2;
constexpr uint32_t kBarRows = 2;             // named barriers 2, 3: the warps of the same rows
constexpr float kRescale = 8.0f;             // log2 units
constexpr float kRefSet = 5.0f;              // e4m3: what a new reference leaves a tile at
constexpr uint32_t kTmemCols = 512, kColS = 0, kColO = 256;
constexpr int kQBytes = kTileBytes;          // 73728, either type

// ------------------------------------------------------------------ planning
__device__ __forceinline__ int queries(const Params& p, int b) {
  return p.q_lens != nullptr ? min(max(p.q_lens[b], 0), p.q_len) : p.q_len;
}

// A context longer than its table is cut at the table's end, for what is shared as
// for the own tokens.
__device__ __forceinline__ int context(const Params& p, int b) {
  return (int)min((long long)p.seq_lens[b], (long long)p.max_pages * kPage);
}

// Whether the groups are consecutive ranges that cover the batch (whole block).
__device__ __forceinline__ bool groups_ok(const Params& p) {
  bool ok = true;
  for (int g = threadIdx.x; g <= p.groups; g += blockDim.x) {
    const int s = p.group_starts[g];
    if (g == 0) ok &= s == 0;
    if (g == p.groups) ok &= s == p.B;
    else ok &= s >= 0 && s <= p.group_starts[g + 1];
  }
  return __syncthreads_and(ok) != 0;
}

// Requests of group g; one group of everything if the groups are no ranges.
__device__ __forceinline__ void group_range(const Params& p, bool ok, int g, int& b0, int& b1) {
  b0 = ok ? p.group_starts[g] : 0;
  b1 = ok ? p.group_starts[g + 1] : g == 0 ? p.B : 0;
  b1 = max(b0, b1);
}

// What a group would share.
struct Group {
  int pages;                     // whole pages that every query row of it sees
  int runs;                      // its query rows, in runs of 16, padding rows apart
  int units;                     // 64-row units of the per-request kernel
};

// (whole warp)
__device__ __forceinline__ Group measure(const Params& p, bool ok, int g, int b0, int b1) {
  Group x{ok ? min(p.prefix_lens[g] / kPage, p.max_pages) : 0, 0, 0};
  for (int b = b0 + (int)(threadIdx.x & 31); b < b1; b += 32) {
    const int L = context(p, b), n = queries(p, b), seen = p.causal ? L - n + 1 : L;
    x.pages = min(x.pages, seen / kPage);
    x.runs += n * p.H / 16;
    x.units += ceil_div(n * p.H, kRows);
  }
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) {
    x.pages = min(x.pages, __shfl_xor_sync(0xFFFFFFFFu, x.pages, off));
    x.runs += __shfl_xor_sync(0xFFFFFFFFu, x.runs, off);
    x.units += __shfl_xor_sync(0xFFFFFFFFu, x.units, off);
  }
  x.pages = max(x.pages, 0);
  return x;
}

// Nanoseconds that a group's sharing saves: the per-request kernel takes 10 ns
// for every unit and page (a 64 x 64 tile, over all SMs), this one 25 ns for
// every 128 rows and two pages.  A launch with shared pages costs 12 us more.
// (Measured with the combine, bf16, 64 heads, one token, 500 own tokens:
//   4 requests behind 16384 tokens 54 us shared, 47 not; behind 65536 86 and 85;
//   8 behind 4096 47 and 38, 16384 56 and 54, 65536 107 and 134;
//   32 behind 4096 69 and 63, 16384 108 and 126, 65536 263 and 368;
//   e4m3 32 behind 65536 229 and 367.)
__device__ __forceinline__ long long gain_of(const Group& x) {
  return 10LL * x.units * x.pages - 25LL * ((x.runs + 7) / 8) * ((x.pages + 1) / 2);
}

// f(group, its requests, what it would share) for every group, a warp each; true
// if the batch is to share at all (whole block).  A group that gains nothing is
// handed on without pages.
template <class F>
__device__ __forceinline__ bool survey(const Params& p, bool ok, F&& f) {
  __shared__ unsigned long long gain;
  if (threadIdx.x == 0) gain = 0;
  __syncthreads();
  for (int g = threadIdx.x >> 5; g < p.groups; g += kPrepThreads / 32) {
    int b0, b1;
    group_range(p, ok, g, b0, b1);
    Group x = measure(p, ok, g, b0, b1);
    const long long n = gain_of(x);
    if (n <= 0 && !p.always) x.pages = 0;
    else if (n > 0 && (threadIdx.x & 31) == 0) atomicAdd(&gain, (unsigned long long)n);
    f(g, b0, b1, x);
  }
  __syncthreads();
  return p.always || gain > (unsigned long long)kMinGain;
}

// Block 0: units and their split.  Block 1: the own tokens' lengths, and the
// per-request kernel's plan.  Blocks 2 .. B + 1: a request's own pages.  The
// others (e4m3): a query row per warp.
__global__ void __launch_bounds__(kPrepThreads) prefix_prep_kernel(Params p, OwnPlan own, int pairs) {
  griddep_wait();
  griddep_launch_dependents();
  if (blockIdx.x > (unsigned)p.B + 1) {
    const int row = ((int)blockIdx.x - 2 - p.B) * (kPrepThreads / 32) + (threadIdx.x >> 5);
    if (row >= p.B * p.R) return;
    const int b = row / p.R;
    split_query_row(p.q + (size_t)row * kDqk, row - b * p.R < queries(p, b) * p.H,
                    p.terms + (size_t)row * 2 * kDqk, p.inv_scale + row, threadIdx.x & 31);
    return;
  }
  const bool ok = groups_ok(p);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (blockIdx.x > 1) {
    const int b = (int)blockIdx.x - 2;
    __shared__ int pages;
    const bool share = survey(p, ok, [&](int, int b0, int b1, const Group& x) {
      if (lane == 0 && b0 <= b && b < b1) pages = x.pages;
    });
    const int n = share ? pages : 0, live = ceil_div(max(context(p, b), 0), kPage) - n;
    const int32_t* from = p.block_table + (size_t)b * p.max_pages + n;
    int32_t* to = p.own_table + (size_t)b * p.max_pages;
    for (int i = tid; i < live; i += kPrepThreads) to[i] = from[i];
    return;
  }
  int2* const info = p.group_info + (size_t)blockIdx.x * p.groups;
  if (blockIdx.x == 1) {
    bool good = true;
    for (int b = tid; b < p.B; b += kPrepThreads)
      good &= p.q_lens == nullptr || (p.q_lens[b] >= 1 && p.q_lens[b] <= p.q_len);
    const bool share = survey(p, ok, [&](int g, int, int, const Group& x) {
      if (lane == 0) info[g].x = x.pages;
    });
    for (int g = warp; g < p.groups; g += kPrepThreads / 32) {
      int b0, b1;
      group_range(p, ok, g, b0, b1);
      const int n = share ? info[g].x : 0;
      for (int b = b0 + lane; b < b1; b += 32) p.own_lens[b] = context(p, b) - n * kPage;
    }
    good = __syncthreads_and(good) != 0;
    plan_units(own.pd.B * own.pd.n_out * own.pd.G,
               [&](int u) { return make_unit(own.pd, u).tiles; }, own.hdr, own.positions, own.grid,
               own.min_tiles, own.unit_cost, good ? 0u : kErrQLens);
    return;
  }
  bool fits = true;
  for (int b = tid; b < p.B; b += kPrepThreads)
    fits &= p.seq_lens[b] <= (long long)p.max_pages * kPage;
  const unsigned bad = (ok ? 0u : kErrQLens) | (__syncthreads_and(fits) ? 0u : kErrBadPage);
  const bool share = survey(p, ok, [&](int g, int, int, const Group& x) {
    if (lane == 0) info[g] = make_int2(x.pages, (x.runs + 7) / 8);
  });
  // first units of the groups that share: a scan over the groups
  __shared__ int sums[32];
  const int per = ceil_div(p.groups, kPrepThreads), g0 = min(p.groups, tid * per);
  const int g1 = min(p.groups, g0 + per);
  auto units_of = [&](int g) { return share && info[g].x > 0 ? info[g].y : 0; };
  int sum = 0;
  for (int g = g0; g < g1; ++g) sum += units_of(g);
  int run = sum;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const int v = __shfl_up_sync(0xFFFFFFFFu, run, off);
    if (lane >= off) run += v;
  }
  if (lane == 31) sums[warp] = run;
  __syncthreads();
  int total = 0;
  run -= sum;
  for (int v = 0; v < kPrepThreads / 32; ++v) {
    if (v < warp) run += sums[v];
    total += sums[v];
  }
  for (int g = g0; g < g1; ++g) {
    const int n = units_of(g);
    info[g].y = n > 0 ? run : -1;
    run += n;
  }
  for (int v = total + tid; v < p.max_units; v += kPrepThreads) p.units[v] = make_int4(0, 0, 0, 0);
  __syncthreads();
  // a warp per group: its requests' first runs, its units
  for (int g = warp; g < p.groups; g += kPrepThreads / 32) {
    int b0, b1;
    group_range(p, ok, g, b0, b1);
    const int first = info[g].y, pages = info[g].x;
    int runs = 0;
    for (int c = b0; c < b1; c += 32) {
      const int b = c + lane, n = b < b1 ? queries(p, b) * p.H / 16 : 0;
      int at = n;
#pragma unroll
      for (int off = 1; off < 32; off <<= 1) {
        const int v = __shfl_up_sync(0xFFFFFFFFu, at, off);
        if (lane >= off) at += v;
      }
      if (b < b1) p.members[b] = make_int2(runs + at - n, first);
      runs += __shfl_sync(0xFFFFFFFFu, at, 31);
    }
    if (first >= 0)
      for (int u = lane; 8 * u < runs; u += 32)
        p.units[first + u] = make_int4(min(8, runs - 8 * u), 0, b0, pages);
  }
  __syncthreads();
  // a warp per request: where its rows are
  const int mine = p.R / 16;
  for (int b = warp; b < p.B; b += kPrepThreads / 32) {
    const int2 m = p.members[b];
    const int live = m.y >= 0 ? queries(p, b) * p.H / 16 : 0;
    for (int k = lane; k < mine; k += 32) {
      const int at = k < live ? m.y * 8 + m.x + k : -1;
      p.where[(size_t)b * mine + k] = at;
      if (at >= 0) p.runs[at] = b * p.R + 16 * k;
    }
  }
  plan_units(p.max_units, [&](int v) { return (p.units[v].w + 1) / 2; }, p.work, p.positions,
             pairs, kMinTiles, kUnitCost, bad);
}

// ------------------------------------------------------------------ attention
enum Part { kA = 0, kB = 1, kC = 2, kV = 3 };   // of a tile's loads

template <bool kFp8>
struct Cfg {
  static constexpr int kStages = kFp8 ? 3 : 2;
  static constexpr int kLine = kFp8 ? 64 : 128;          // bytes of a chunk's row
  static constexpr int kSlot = kHalf * kLine;            // a page's chunk
  static constexpr int kTile = kChunks * kSlot;
  static constexpr int kGroup = 8 * kLine;               // eight rows of a chunk
  static constexpr int kQGroup = kChunks * kGroup;       // eight query rows: [chunk][8][64]
  static constexpr int kSmemKV = kQBytes;
  static constexpr int kSmemP = kSmemKV + kStages * kTile;
  // bf16: the second half's probabilities; e4m3: two buffers of both terms
  static constexpr int kSmemMisc = kSmemP + (kFp8 ? 2 * 4 * kSlot : kSlot);
};

template <bool kFp8>
struct Misc {
  static constexpr int kStages = Cfg<kFp8>::kStages;
  uint64_t full[kStages][4];     // leader: loads of both CTAs landed
  uint64_t a_free[kStages];      // P V has read A
  uint64_t pv_done[kStages];     // P V has read everything
  uint64_t s_full[2];            // both S issuers; e4m3: the tile's scales
  uint64_t k_read[kStages];      // S is done: V goes over half of K
  uint64_t s_empty[2], p_full[2], o_free;   // leader: the softmax warps of both
  uint64_t q_full, q_empty;
  uint64_t drain;
  uint64_t sc_full[kFp8 ? kStages : 1];
  uint32_t tmem_base;
  int abort;
  uint32_t armed[kStages][4];    // loads announced on full, for a teardown
  uint32_t armed_q;
  float xmax[2][4][kHalf];       // by tile parity and quarter of the tokens
  // token scales (copied in 16-byte units, read as float4) and their exponents
  alignas(16) float sigma[kFp8 ? kStages : 1][kFp8 ? 128 : 4];
  alignas(16) float lge[kFp8 ? kStages : 1][kFp8 ? 128 : 4];
};
static_assert(offsetof(Misc<true>, sigma) % 16 == 0 && offsetof(Misc<true>, lge) % 16 == 0,
              "16-byte units");
static_assert(Cfg<true>::kSmemMisc % 1024 == 0 && Cfg<false>::kSmemMisc % 1024 == 0,
              "swizzle atoms and 16-byte units");

template <bool kFp8>
constexpr int smem_bytes() {
  return Cfg<kFp8>::kSmemMisc + (int)sizeof(Misc<kFp8>);
}
static_assert(smem_bytes<false>() <= 232448 && smem_bytes<true>() <= 232448, "shared memory");

// One role's walk over the pair's tiles.
struct Walk {
  PieceIter it;
  const int4* units;
  int4 u;                        // the unit: runs, -, table row, pages
  int unit;
  int j, t1;                     // the tile, the piece's end
  int g;                         // tiles before this one
  bool whole, first;             // the piece is the whole unit; its first tile
  int slot;
  __device__ void init(const Params& p, int lo, int hi, int lane) {   // whole warp
    it.init_warp(p.positions, p.work->num_units, lo, hi, p.work->unit_cost, lane);
    units = p.units;
    j = t1 = 0;
    g = -1;
  }
  __device__ bool next() {
    first = ++j >= t1;
    if (first) {
      if (!it.next(unit, j, t1, whole, slot)) return false;
      u = units[unit];
    }
    ++g;
    return true;
  }
};

// The two pages of a walk's tiles, read a tile ahead by one thread.
struct Pages {
  const int32_t* row;
  int count, ahead[2];
  __device__ int entry(int i) const { return i < count ? __ldg(row + i) : -1; }
  // The tile's pages; one behind the prefix or out of range gives num_pages,
  // which lies behind the pool, where loads give zeros.
  __device__ void next(const Params& p, const Walk& w, int (&page)[2]) {
    if (w.first) {
      row = p.block_table + (size_t)w.u.z * p.max_pages;
      count = w.u.w;
      ahead[0] = entry(2 * w.j);
      ahead[1] = entry(2 * w.j + 1);
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int e = ahead[h];
      page[h] = e >= 0 && e < p.num_pages ? e : p.num_pages;
      ahead[h] = entry(2 * w.j + 2 + h);
    }
  }
};

__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
  __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<uint32_t*>(&h);
}

template <bool kFp8>
__global__ void __launch_bounds__(kThreads, 1)
    prefix_kernel(const __grid_constant__ CUtensorMap tm_q,
                  const __grid_constant__ CUtensorMap tm_kv4,
                  const __grid_constant__ CUtensorMap tm_kv1, Params p) {
  using C = Cfg<kFp8>;
  constexpr int kStages = C::kStages;
  extern __shared__ __align__(1024) uint8_t smem[];   // whole swizzle atoms
  Misc<kFp8>* misc = reinterpret_cast<Misc<kFp8>*>(smem + C::kSmemMisc);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_rank();
  const bool leader = rank == 0;
  volatile int* abort_flag = &misc->abort;
  const uint64_t tmo = p.timeout_ns;
  const uint32_t peer_abort = map_rank(smem_u32(&misc->abort), rank ^ 1);
  auto fail = [&]() {            // one thread: both CTAs leave their loops
    atomicOr(p.err, kErrTimeout);
    *(volatile int*)&misc->abort = 1;
    st_cluster(peer_abort, 1);
  };
  // one thread's wait, and a warp's
  auto wait1 = [&](uint64_t* bar, uint32_t parity) {
    return mbar_try_wait_hint(smem_u32(bar), parity, 200000u) ||
           mbar_wait_long(smem_u32(bar), parity, tmo, abort_flag);
  };
  auto wait = [&](uint64_t* bar, uint32_t parity) {
    return __all_sync(0xffffffffu, wait1(bar, parity)) != 0;
  };
  auto at_leader = [&](uint64_t* bar) { return map_rank(smem_u32(bar), 0); };

  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      for (int k = 0; k < 4; ++k) {
        mbar_init(smem_u32(&misc->full[s][k]), 2);
        misc->armed[s][k] = 0;
      }
      mbar_init(smem_u32(&misc->a_free[s]), 1);
      mbar_init(smem_u32(&misc->k_read[s]), 2);
      mbar_init(smem_u32(&misc->pv_done[s]), 1);
      if (kFp8) {
        mbar_init(smem_u32(&misc->sc_full[s]), 1);
      }
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_u32(&misc->s_full[i]), kFp8 ? 3 : 2);
      mbar_init(smem_u32(&misc->s_empty[i]), 2 * kSoftmaxWarps);
      mbar_init(smem_u32(&misc->p_full[i]), 2 * kSoftmaxWarps);
    }
    mbar_init(smem_u32(&misc->o_free), 2 * kSoftmaxWarps);
    mbar_init(smem_u32(&misc->q_full), 2);
    mbar_init(smem_u32(&misc->q_empty), 2);
    mbar_init(smem_u32(&misc->drain), 3);
    misc->armed_q = 0;
    misc->abort = 0;
    fence_mbar_init();
  }
  if (warp == 1) tmem_alloc_pair(smem_u32(&misc->tmem_base), kTmemCols);
  if (warp == 0 && lane == 0) {
    tma_prefetch_desc(&tm_q);
    tma_prefetch_desc(&tm_kv4);
    tma_prefetch_desc(&tm_kv1);
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync_all();            // the peer's barriers and tensor memory are there
  tc_fence_after();
  griddep_wait();                // the work list, the query's terms
  griddep_launch_dependents();
  // (a pair without work falls through to the teardown; so would every pair if
  // the declared alignment of shared memory did not hold)
  const bool aligned = (smem_u32(smem) & 1023u) == 0;
  if (!aligned && threadIdx.x == 0) atomicOr(p.err, kErrTimeout);
  const int W = aligned ? p.work->total_cost : 0, per = p.work->per_cta;
  const int pair = (int)blockIdx.x >> 1;
  const int lo = (int)min((long long)W, (long long)pair * per);
  const int hi = (int)min((long long)W, (long long)lo + per);
  const uint32_t tmem = misc->tmem_base;
  const uint32_t sQ = smem_u32(smem), sKV = smem_u32(smem + C::kSmemKV);
  const uint32_t sP = smem_u32(smem + C::kSmemP);

  // Announces `bytes` of a part of a stage on the leader's barrier.
  auto arm = [&](int s, int part, uint32_t bytes) {
    misc->armed[s][part]++;
    mbar_arrive_expect_tx_pair(at_leader(&misc->full[s][part]), bytes);
  };
  // descriptors of the buffers' starts; an offset adds its sixteenth
  auto desc = [&](uint32_t at, uint32_t lbo) {
    return kFp8 ? sw64_desc(at, lbo, C::kGroup) : sw128_desc(at, lbo, C::kGroup);
  };

  Walk w;
  w.init(p, lo, hi, lane);
  bool ok = true;

  if (warp == 0) {
    // ---------------------------------------------------------- K producer
    // (one thread; so are the other producer and the issuers)
    if (lane == 0) {
      Pages pages;
      int pieces = 0;
      while (ok && w.next()) {
        const int s = w.g % kStages, use = w.g / kStages;
        const uint32_t st = sKV + s * C::kTile;
        int page[2];
        pages.next(p, w, page);
        const int mine = leader ? page[0] : page[1], row = mine * kPage;
        if (mine == p.num_pages && 2 * w.j + (int)rank < w.u.w) atomicOr(p.err, kErrBadPage);
        if (use > 0) ok = wait1(&misc->a_free[s], (use - 1) & 1);
        if (!ok) break;
        arm(s, kA, 4 * C::kSlot);
        tma_load_3d_pair(st, &tm_kv4, at_leader(&misc->full[s][kA]), 0, row, 0);
        if (use > 0) ok = wait1(&misc->pv_done[s], (use - 1) & 1);
        if (!ok) break;
        arm(s, kB, 4 * C::kSlot);
        tma_load_3d_pair(st + 4 * C::kSlot, &tm_kv4, at_leader(&misc->full[s][kB]), 0, row, 4);
        arm(s, kC, C::kSlot);
        tma_load_3d_pair(st + 8 * C::kSlot, &tm_kv1, at_leader(&misc->full[s][kC]), 0, row, 8);
        if (kFp8) {
          // both pages' token scales; 1 where there is no page (its codes are 0)
          const uint32_t bar = smem_u32(&misc->sc_full[s]);
          uint32_t bytes = 0;
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            if (page[h] < p.num_pages) bytes += kPage * 4;
            else
              for (int a = 0; a < kPage; ++a) misc->sigma[s][64 * h + a] = 1.0f;
          }
          mbar_arrive_expect_tx(bar, bytes);
#pragma unroll
          for (int h = 0; h < 2; ++h)
            if (page[h] < p.num_pages)
              bulk_load(smem_u32(&misc->sigma[s][64 * h]), p.kv_scale + (size_t)page[h] * kPage,
                        kPage * 4, bar);
        }
        if (w.first) {
          // the piece's query, once S of the piece before is done
          if (pieces > 0) ok = wait1(&misc->q_empty, (pieces - 1) & 1);
          if (!ok) break;
          if (p.withhold_query && pieces == 0) continue;
          misc->armed_q++;
          mbar_arrive_expect_tx_pair(at_leader(&misc->q_full), kQBytes);
          // four runs of 16 rows; a run behind the group's last lies behind the
          // query, where loads give zeros
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const int run = 4 * (int)rank + k;
            const int g8 = (run < w.u.x ? p.runs[8 * w.unit + run] : p.B * p.R) / 8;
            const uint32_t to = sQ + 2 * k * C::kQGroup, bar = at_leader(&misc->q_full);
            if (kFp8) {
              tma_load_5d_pair(to, &tm_q, bar, 0, 0, 0, g8, 0);
              tma_load_5d_pair(to + kQBytes / 2, &tm_q, bar, 0, 0, 0, g8, 1);
            } else {
              tma_load_4d_pair(to, &tm_q, bar, 0, 0, 0, g8);
            }
          }
          ++pieces;
        }
      }
      if (!ok) fail();
    }
  } else if (warp == 3) {
    // ---------------------------------------------------------- V producer
    // The CTA's dims of the other CTA's page, over what S has read; e4m3: before
    // that the tile's token scales, by the whole warp.
    Pages pages;
    while (ok && w.next()) {
      const int s = w.g % kStages;
      if (kFp8) {
        // token scales sigma = mant 2^E with mant in [0.5, 1): sigma sanitised
        // in place, E apart
        ok = wait(&misc->sc_full[s], (w.g / kStages) & 1);
        if (!ok) break;
#pragma unroll
        for (int h = 0; h < 4; ++h) {
          const int a = lane + 32 * h;
          float sg = misc->sigma[s][a];
          uint32_t eb = (__float_as_uint(sg) >> 23) & 0xFFu;
          if (eb < 27u) {
            // zero, subnormal or below 2^-100: as 2^-60
            sg = copysignf(8.6736174e-19f, sg);
            eb = (__float_as_uint(sg) >> 23) & 0xFFu;
          }
          misc->sigma[s][a] = sg;
          // inf, NaN or >= 2^126: exponent 0, and the value itself propagates
          misc->lge[s][a] = eb >= 253u ? 0.0f : (float)((int)eb - 126);
        }
        __syncwarp();
        // (S of the tile before is done, so the phase of two tiles before has
        // ended: this arrival counts for this tile)
        if (lane == 0) mbar_arrive(smem_u32(&misc->s_full[w.g & 1]));
      }
      if (lane == 0) {
        int page[2];
        pages.next(p, w, page);
        const int other = leader ? page[1] : page[0], row = other * kPage;
        if (other == p.num_pages && 2 * w.j + (int)(rank ^ 1) < w.u.w)
          atomicOr(p.err, kErrBadPage);
        ok = wait1(&misc->k_read[s], (w.g / kStages) & 1);
        if (ok) {
          arm(s, kV, 4 * C::kSlot);
          tma_load_3d_pair(sKV + s * C::kTile + (leader ? 4 : 0) * C::kSlot, &tm_kv4,
                           at_leader(&misc->full[s][kV]), 0, row, leader ? 0 : 4);
        }
      }
      ok = __shfl_sync(0xffffffffu, ok, 0) != 0;
    }
    if (!ok && lane == 0) fail();
  } else if ((warp == 1 || warp == 2) && leader) {
    // ------------------------------------------------------------ S issue
    constexpr uint32_t id = kFp8 ? idesc_e4m3_f32(128, 128, false, false)
                                 : idesc_bf16_f32(128, 128, false, false);
    if (lane == 0) {
      // bf16: issuer i takes the 16-dim steps 2 i, 2 i + 1 of every chunk; e4m3:
      // the query's term i
      const int i = warp - 1;
      const uint64_t dq = kFp8 ? sw64_desc(sQ + i * (kQBytes / 2), 16, C::kQGroup)
                               : sw128_desc(sQ + i * 64, 16, C::kQGroup);
      int pieces = 0;
      Walk n = w;                // the next tile: is this one its piece's last?
      n.next();
      while (ok && w.next()) {
        const int s = w.g % kStages, sb = w.g & 1;
        if (w.first) {
          ok = wait1(&misc->q_full, pieces & 1);
          ++pieces;
        }
        if (ok && w.g >= 2) ok = wait1(&misc->s_empty[sb], ((w.g >> 1) - 1) & 1);
        const bool last = !n.next() || n.first;
        const uint32_t d = tmem + kColS + 128 * sb + 64 * i;
        const uint64_t dk = desc(sKV + s * C::kTile + (kFp8 ? 0 : 64 * i), 16);
#pragma unroll
        for (int c = 0; c < kChunks; ++c) {
          if ((c & 3) == 0) {    // a part's first chunk
            ok = ok && wait1(&misc->full[s][c >> 2], (w.g / kStages) & 1);
            if (!ok) break;
            tc_fence_after();
          }
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            const uint32_t acc = (c > 0 || k > 0) ? 1u : 0u;
            const uint32_t oq = (c * C::kGroup + 32 * k) >> 4, o = (c * C::kSlot + 32 * k) >> 4;
            if (kFp8) mma_e4m3_pair(d, dq + oq, dk + o, id, acc);
            else mma_bf16_pair(d, dq + oq, dk + o, id, acc);
          }
        }
        if (!ok) break;
        mma_commit_pair(smem_u32(&misc->s_full[sb]));
        mma_commit_pair(smem_u32(&misc->k_read[s]));
        if (last) mma_commit_pair(smem_u32(&misc->q_empty));
      }
      if (!ok) fail();
    }
  } else if (warp == 12 && leader) {
    // ------------------------------------------------------------ P V issue
    constexpr uint32_t id = kFp8 ? idesc_e4m3_f32(128, 256, false, true)
                                 : idesc_bf16_f32(128, 256, false, true);
    if (lane == 0) {
      int pieces = 0;
      while (ok && w.next()) {
        const int s = w.g % kStages;
        ok = wait1(&misc->full[s][kV], (w.g / kStages) & 1);
        if (w.first) {
          if (ok && pieces > 0) ok = wait1(&misc->o_free, (pieces - 1) & 1);
          ++pieces;
        }
        if (ok) ok = wait1(&misc->p_full[w.g & 1], (w.g >> 1) & 1);
        if (!ok) break;
        tc_fence_after();
        const uint64_t dv = desc(sKV + s * C::kTile, C::kSlot);
        const uint64_t dp0 = kFp8 ? desc(sP + (w.g & 1) * 4 * C::kSlot, 16)
                                  : desc(sKV + s * C::kTile + 8 * C::kSlot, 16);
        const uint64_t dp1 = kFp8 ? dp0 + (C::kSlot >> 4) : desc(sP, 16);
        // (rolled: unrolled, the e4m3 kernel waits for instructions, 171 instead
        // of 161 us over nine prefixes)
#pragma unroll 1
        for (int half = 0; half < 2; ++half) {             // tokens 64 half ..
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            // bf16: 16 tokens; e4m3: 32 tokens k / 2, term k % 2
            const uint32_t oa = kFp8 ? (k & 1) * 2 * C::kSlot + 32 * (k >> 1) : 32 * k;
            const uint32_t ov = 4 * half * C::kSlot + 2048 * (kFp8 ? k >> 1 : k);
            const uint64_t a = (half == 0 ? dp0 : dp1) + (oa >> 4);
#pragma unroll
            for (int nb = 0; nb < 2; ++nb) {               // 128 dims of each CTA
              const uint32_t d = tmem + kColO + 128 * nb;
              const uint64_t b = dv + ((ov + 2 * nb * C::kSlot) >> 4);
              const uint32_t acc = (w.first && half == 0 && k == 0) ? 0u : 1u;
              if (kFp8) mma_e4m3_pair(d, a, b, id, acc);
              else mma_bf16_pair(d, a, b, id, acc);
            }
          }
          mma_commit_pair(smem_u32(half == 0 ? &misc->a_free[s] : &misc->pv_done[s]));
        }
      }
      if (!ok) fail();
    }
  } else if (warp >= 4 && warp < 12) {
    // ------------------------------------------------------------ softmax
    const int quad = warp & 3, half = quad >> 1;           // TMEM lanes 32 quad ..
    const int grp = (warp - 4) >> 2;                       // tokens 64 half + 32 grp ..
    const int r = 32 * (quad & 1) + lane;                  // the thread's row of the CTA
    const int part = 2 * half + grp;
    const uint32_t bar = kBarRows + (quad & 1);            // the four warps of these rows
    const uint32_t lanes = (uint32_t)(32 * quad) << 16;
    while (w.next()) {
      // one piece; `w` is at its first tile
      const int tr = (int)rank * kHalf + r;                // row of the tile
      const bool live = (tr >> 4) < w.u.x;
      const int gr = live ? p.runs[8 * w.unit + (tr >> 4)] + (tr & 15) : 0;   // of the query
      float qs = p.scale_log2;
      if (kFp8) {
        const float f = live ? p.inv_scale[gr] : 1.0f;
        if (f != f) atomicOr(p.err, kErrQRange);
        qs *= f;
      }
      const f32x2 qs2 = pack2(qs, qs);                     // logits in log2 units
      float m_run = -CUDART_INF_F, m_top = -CUDART_INF_F;  // the reference, the largest logit
      float l_run = 0.0f;                                  // this thread's tokens
      while (true) {
        const int s = w.g % kStages, sb = w.g & 1;
        ok = ok && wait(&misc->s_full[sb], (w.g >> 1) & 1);
        f32x2 a[16];             // bf16: S; e4m3: S sigma
        float mx = -CUDART_INF_F;
        // the last tile of an odd number of pages has no second page
        const bool there = 2 * w.j + half < w.u.w;
        if (ok) {
          tc_fence_after();
          // both issuers' accumulators (the second in two parts, for registers)
          uint32_t v[32];
          const uint32_t s0 = tmem + lanes + kColS + 128 * sb + 32 * grp;
          tmem_ld32(s0, v);
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            uint32_t u[16];
            tmem_ld16(s0 + 64 + 16 * h, u);
            tmem_wait_ld();
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const int k = 16 * h + 2 * i;
              a[8 * h + i] = add2(pack2(__uint_as_float(v[k]), __uint_as_float(v[k + 1])),
                                  pack2(__uint_as_float(u[2 * i]), __uint_as_float(u[2 * i + 1])));
            }
          }
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive_pair(at_leader(&misc->s_empty[sb]));
          float m4[4] = {mx, mx, mx, mx};
#pragma unroll
          for (int i = 0; i < 16; i += 2) {
            f32x2 b0 = a[i], b1 = a[i + 1];
            if (kFp8) {
              // b_t = S sigma qs + E_t
              const int t = 32 * part + 2 * i;
              const ulonglong2 sg = *reinterpret_cast<const ulonglong2*>(&misc->sigma[s][t]);
              const ulonglong2 eg = *reinterpret_cast<const ulonglong2*>(&misc->lge[s][t]);
              a[i] = mul2(a[i], sg.x);
              a[i + 1] = mul2(a[i + 1], sg.y);
              b0 = fma2(a[i], qs2, eg.x);
              b1 = fma2(a[i + 1], qs2, eg.y);
            }
            const float2 y0 = unpack2(b0), y1 = unpack2(b1);
            m4[i & 2] = max3(m4[i & 2], y0.x, y0.y);
            m4[(i & 2) + 1] = max3(m4[(i & 2) + 1], y1.x, y1.y);
          }
          mx = max3(fmaxf(m4[0], m4[1]), m4[2], m4[3]);
          if (!kFp8) mx *= p.scale_log2;
          if (!there) mx = -CUDART_INF_F;
          misc->xmax[sb][part][r] = mx;
        }
        if (named_bar_or(bar, 128, !ok)) {
          ok = false;
          break;
        }
        const float m_tile = fmaxf(fmaxf(mx, misc->xmax[sb][part ^ 1][r]),
                                   fmaxf(misc->xmax[sb][part ^ 2][r], misc->xmax[sb][part ^ 3][r]));
        float alpha = 1.0f;
        bool rescale = false;
        if (kFp8) {
          rescale = move_reference(m_tile, kRefSet, m_run, m_top, alpha);
        } else if (m_tile > m_run + kRescale) {
          alpha = m_run == -CUDART_INF_F ? 0.0f : ex2_approx(m_run - m_tile);
          m_run = m_tile;
          rescale = true;
        }
        l_run *= alpha;
        rescale = rescale && live && !w.first;
        // (a page that is not there has keys of 0: finite logits, and weights of 0)
        const float m_use = !there ? CUDART_INF_F : m_run == -CUDART_INF_F ? 0.0f : m_run;
        // P V of the tile before: O is rescaled behind it, and it has read the
        // probabilities that are written over
        const int gp = w.g - 1, ga = kFp8 ? w.g - 2 : w.g - 1;
        auto pv_of = [&](int g) {
          return wait(&misc->pv_done[g % kStages], (g / kStages) & 1);
        };
        if (__any_sync(0xffffffffu, rescale)) {
          ok = pv_of(gp);
          tc_fence_after();
          if (ok) {
#pragma unroll 1
            for (int c = 128 * grp; c < 128 * grp + 128; c += 32) {
              uint32_t v[32];
              tmem_ld32(tmem + lanes + kColO + c, v);
              tmem_wait_ld();
#pragma unroll
              for (int i = 0; i < 32; ++i) v[i] = __float_as_uint(__uint_as_float(v[i]) * alpha);
              tmem_st32(tmem + lanes + kColO + c, v);
            }
            tmem_wait_st();
          }
        }
        const f32x2 m2 = pack2(-m_use, -m_use);
        f32x2 ls[2] = {0, 0};
        if (kFp8) {
          // two-term sums of P' = u sigma: hi to 4 significant bits in integers
          // (converting a code back takes three conversions a pair, at an eighth
          // of the rate; a product and two differences are fused into hi = P'),
          // lo what is left.  Off by 2^-8 of P' at most from 2^-2 up, by 2^-9
          // below, where codes are multiples of that (move_reference).
          ulonglong2 sg;
          uint32_t hi4[8], lo4[8];
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            const float2 x = unpack2(fma2(a[i], qs2, m2));
            const f32x2 u = pack2(ex2_approx(x.x), ex2_approx(x.y));
            ls[i & 1] = add2(ls[i & 1], u);
            if (i % 2 == 0)
              sg = *reinterpret_cast<const ulonglong2*>(&misc->sigma[s][32 * part + 2 * i]);
            const f32x2 pv = mul2(u, i % 2 == 0 ? sg.x : sg.y);
            const float2 y = unpack2(pv);
            const float2 h =
                make_float2(__uint_as_float((__float_as_uint(y.x) + 0x80000u) & 0xFFF00000u),
                            __uint_as_float((__float_as_uint(y.y) + 0x80000u) & 0xFFF00000u));
            const float2 l = unpack2(sub2(pv, pack2(h.x, h.y)));
            const uint32_t ch = f32x2_to_e4m3x2(h.x, h.y), cl = f32x2_to_e4m3x2(l.x, l.y);
            if (i % 2 == 0) {
              hi4[i / 2] = ch;
              lo4[i / 2] = cl;
            } else {
              hi4[i / 2] |= ch << 16;
              lo4[i / 2] |= cl << 16;
            }
          }
          if (ok && ga >= 0) ok = pv_of(ga);
          if (ok) {
            // 64-byte rows, 16-byte units under a 64-byte swizzle
            uint8_t* row = smem + C::kSmemP + (w.g & 1) * 4 * C::kSlot + half * C::kSlot + r * 64;
            const int sw = (r >> 1) & 3;
#pragma unroll
            for (int c = 0; c < 2; ++c) {
              const int at = ((2 * grp + c) ^ sw) << 4;
              *reinterpret_cast<uint4*>(row + at) =
                  make_uint4(hi4[4 * c], hi4[4 * c + 1], hi4[4 * c + 2], hi4[4 * c + 3]);
              *reinterpret_cast<uint4*>(row + 2 * C::kSlot + at) =
                  make_uint4(lo4[4 * c], lo4[4 * c + 1], lo4[4 * c + 2], lo4[4 * c + 3]);
            }
          }
        } else {
          uint32_t pk[16];
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            // bf16: P is rounded to 8 bits, relative 2^-8, as in the
            // per-request kernel; its sum is taken before the rounding
            const float2 x = unpack2(fma2(a[i], qs2, m2));
            const float2 u = make_float2(ex2_approx(x.x), ex2_approx(x.y));
            pk[i] = pack_bf16(u.x, u.y);
            ls[i & 1] = add2(ls[i & 1], pack2(u.x, u.y));
          }
          // tokens 0-63 go into the stage's rope chunk, which S has read;
          // tokens 64-127 into the one chunk that every tile uses
          if (ok && half == 1 && ga >= 0) ok = pv_of(ga);
          if (ok) {
            uint8_t* row = smem + (half == 0 ? C::kSmemKV + s * C::kTile + 8 * C::kSlot : C::kSmemP) +
                           r * 128;
#pragma unroll
            for (int c = 0; c < 4; ++c)
              *reinterpret_cast<uint4*>(row + (((4 * grp + c) ^ (r & 7)) << 4)) =
                  make_uint4(pk[4 * c], pk[4 * c + 1], pk[4 * c + 2], pk[4 * c + 3]);
          }
        }
        const float2 lt = unpack2(add2(ls[0], ls[1]));
        l_run += lt.x + lt.y;
        fence_proxy_async_smem();
        tc_fence_before();
        __syncwarp();
        // a failed wait is seen by all four warps at the next reduction
        if (ok && lane == 0) mbar_arrive_pair(at_leader(&misc->p_full[sb]));
        if (w.j + 1 >= w.t1) break;
        w.next();
      }
      // ---------------------------------------------------------- epilogue
      ok = ok && wait(&misc->pv_done[w.g % kStages], (w.g / kStages) & 1);
      // (the other buffer of xmax: this tile's may still be read)
      misc->xmax[(w.g & 1) ^ 1][part][r] = l_run;
      if (named_bar_or(bar, 128, !ok)) {
        ok = false;
        break;
      }
      tc_fence_after();
      // the four sums in one order for all of the row's threads
      const float* ls = &misc->xmax[(w.g & 1) ^ 1][0][r];
      const float l = (ls[0] + ls[kHalf]) + (ls[2 * kHalf] + ls[3 * kHalf]);
      const size_t at = w.whole ? (size_t)gr : ((size_t)2 * pair + w.slot) * kPairRows + tr;
      float* const orow = (w.whole ? p.out : p.ws_o) + at * kDv + 128 * part;
      const bool wide = (reinterpret_cast<uintptr_t>(orow) & 31u) == 0;
      const float inv = l != 0.0f ? 1.0f / l : 0.0f;       // or NaN
      if (live && part == 0)
        (w.whole ? p.lse : p.ws_lse)[at] =
            l != 0.0f ? (m_run + __log2f(l)) * 0.69314718055994530942f : -CUDART_INF_F;
      auto put = [&](int c, const uint32_t (&v)[32]) {
        if (!live) return;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          float x[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) x[e] = __uint_as_float(v[8 * i + e]) * inv;
          float* const to = orow + c + 8 * i;
          if (wide) {
            // a sector a lane: the lanes' rows are 2 KB apart
            st_global_8(to, x);
          } else {
            reinterpret_cast<float4*>(to)[0] = make_float4(x[0], x[1], x[2], x[3]);
            reinterpret_cast<float4*>(to)[1] = make_float4(x[4], x[5], x[6], x[7]);
          }
        }
      };
      {
        uint32_t va[32], vb[32];
        const uint32_t o = tmem + lanes + kColO + 128 * grp;
        tmem_ld32(o, va);
#pragma unroll
        for (int c = 0; c < 128; c += 64) {
          tmem_wait_ld();
          tmem_ld32(o + c + 32, vb);
          put(c, va);
          tmem_wait_ld();
          if (c + 64 < 128) tmem_ld32(o + c + 64, va);
          put(c + 32, vb);
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_pair(at_leader(&misc->o_free));
      // xmax is written again by the next piece's first tile
      named_bar_sync(bar, 128);
    }
    if (!ok && lane == 0) fail();
  }

  // ---------------------------------------------------------------- teardown
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  cluster_sync_all();            // nothing is issued any more, by either CTA
  const bool failed = *abort_flag != 0 || ld_cluster(peer_abort) != 0;
  if (failed) {
    // after a failure, the MMAs and copies in flight land before tensor and
    // shared memory are given back
    int never = 0;
    if (leader && (warp == 1 || warp == 2 || warp == 12) && lane == 0) {
      asm volatile(
          "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(
              smem_u32(&misc->drain))
          : "memory");
      mbar_wait(smem_u32(&misc->drain), 0, kDrainNs, &never);
    }
    if (leader && warp == 0 && lane == 0) {
      // a load that one CTA announced and the other never did: the missing
      // arrival is made up, then the phase ends with the announced bytes
      bool good = true;
      auto settle = [&](uint64_t* bar, uint32_t mine_n, uint32_t theirs) {
        if (mine_n != theirs) mbar_arrive(smem_u32(bar));
        const uint32_t n = max(mine_n, theirs);
        if (n > 0 && good) good = mbar_wait(smem_u32(bar), (n - 1) & 1, kDrainNs, &never);
      };
      for (int s = 0; s < kStages; ++s)
        for (int k = 0; k < 4; ++k)
          settle(&misc->full[s][k], misc->armed[s][k],
                 ld_cluster(map_rank(smem_u32(&misc->armed[s][k]), 1)));
      settle(&misc->q_full, misc->armed_q, ld_cluster(map_rank(smem_u32(&misc->armed_q), 1)));
    }
    if (kFp8 && warp == 0 && lane == 0) {
      // the scales of a stage are announced behind its chunk C
      for (int s = 0; s < kStages; ++s) {
        const uint32_t n = misc->armed[s][kC];
        if (n > 0) mbar_wait(smem_u32(&misc->sc_full[s]), (n - 1) & 1, kDrainNs, &never);
      }
    }
    tc_fence_before();
    __syncthreads();
  }
  cluster_sync_all();            // the peer reads this CTA no more
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc_pair(tmem, kTmemCols);
  }
}

// ------------------------------------------------------------ joining pieces
struct PairPieces {
  const float* ws_o;
  const float* ws_lse;
  struct Ctx {
    int c0, count, r, first_in_slot1;
  };
  __device__ void piece(const Ctx& c, int k, const float*& src, float& lse) const {
    const size_t cc = (size_t)(c.c0 + k);
    const size_t slot = (k == 0 && c.first_in_slot1) ? 2 * cc + 1 : 2 * cc;
    src = ws_o + (slot * kPairRows + c.r) * kDv;
    lse = ws_lse[slot * kPairRows + c.r];
  }
};

// Few rows, which may have dozens of pieces: four warps a row (kVec 1), twelve
// pieces in flight; from kManyRows rows, a warp a row (kVec 4) and three, for
// fewer waves of blocks (joining a ragged verify step of 5120 rows 21.5 -> 12.4 us).
constexpr int kManyRows = 1024;
template <int kVec>
struct Join {
  static constexpr int kRowsB = 2 * kVec, kBatch = kVec == 1 ? kMergeBatch : 3;
  static constexpr int kSmem = 8 * kBatch * kVec * 32 * (int)sizeof(float4);
};

// Slice 0, 2 kVec rows a block: 0 and -inf for rows in no unit, else the LSE join
// of their pieces unless a pair computed the unit whole.  The blocks behind them:
// the own tokens' units.
template <int kVec>
__global__ void __launch_bounds__(256, 4) prefix_join_kernel(Params p, OwnPieces own) {
  using J = Join<kVec>;
  extern __shared__ __align__(16) float4 join_stage[];
  griddep_wait();
  griddep_launch_dependents();
  constexpr int kOwnBlocks = kRows / J::kRowsB;
  const int i = (int)blockIdx.x - p.B * p.R / J::kRowsB;
  if (i >= 0) {
    merge_unit_rows<kVec, J::kBatch>(own.pd, own.hdr, own.positions, own.ws_o, own.ws_lse, own.out,
                                     own.lse, i / kOwnBlocks, i % kOwnBlocks, join_stage);
    return;
  }
  if (blockIdx.x == 0 && threadIdx.x == 0 && p.work->err != 0) atomicOr(p.err, p.work->err);
  constexpr int kWarps = 4 / kVec;               // per row
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, part = warp % kWarps;
  const int gr = (int)blockIdx.x * J::kRowsB + warp / kWarps;
  const int w = p.where[gr >> 4], u = w >> 3, r = (w & 7) * 16 + (gr & 15);
  int ps = 0, ue = 0, us = 0, per = 1;
  if (w >= 0) {
    ps = p.positions[u];
    ue = p.positions[u + 1];
    us = unit_tile_start(p.positions, u, p.work->unit_cost);
    per = p.work->per_cta;
    if (us / per == (ue - 1) / per) return;    // written by the pair that computed it
  }
  float4* dst = reinterpret_cast<float4*>(p.out + (size_t)gr * kDv) + 32 * kVec * part;
  if (w < 0) {
#pragma unroll
    for (int v = 0; v < kVec; ++v) dst[lane + 32 * v] = make_float4(0.f, 0.f, 0.f, 0.f);
    if (part == 0 && lane == 0) p.lse[gr] = -CUDART_INF_F;
    return;
  }
  const int c0 = us / per, c1 = (ue - 1) / per;
  const PairPieces src{p.ws_o, p.ws_lse};
  const PairPieces::Ctx ctx{c0, c1 - c0 + 1, r, c0 * per < ps ? 1 : 0};
  float4 acc[kVec];
  float M, wsum;
  merge_pieces_staged<kVec, J::kBatch>(src, ctx, lane, 32 * kVec * part,
                                       join_stage + warp * (J::kBatch * kVec * 32), acc, M, wsum);
  const float inv = wsum != 0.f ? 1.0f / wsum : 0.f;   // or NaN
#pragma unroll
  for (int v = 0; v < kVec; ++v)
    dst[lane + 32 * v] =
        make_float4(acc[v].x * inv, acc[v].y * inv, acc[v].z * inv, acc[v].w * inv);
  if (part == 0 && lane == 0) p.lse[gr] = wsum != 0.f ? M + __logf(wsum) : -CUDART_INF_F;
}

// ------------------------------------------------------------------ launches
bool encode(CUtensorMap* m, bool fp8, int rank, const void* base, const cuuint64_t* dims,
            const cuuint64_t* strides, const cuuint32_t* box) {
  const cuuint32_t es[5] = {1, 1, 1, 1, 1};
  return host::encode_fn()(m, fp8 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16,
                           rank, const_cast<void*>(base), dims, strides, box, es,
                           CU_TENSOR_MAP_INTERLEAVE_NONE,
                           fp8 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B,
                           fp8 ? CU_TENSOR_MAP_L2_PROMOTION_NONE : CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
                           CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <bool kFp8>
cudaError_t attend(const Params& p, const void* kv, int pairs, cudaStream_t stream) {
  if (host::encode_fn() == nullptr) return cudaErrorInitializationError;
  const cuuint64_t e = kFp8 ? 1 : 2;
  CUtensorMap tm_q, tm_kv4, tm_kv1;
  bool ok;
  // query: (64 dims, row of 8, chunk, 8-row group), e4m3 of each term: a run of 16
  // rows as [group][chunk][8 rows][64 dims]
  const cuuint64_t qd[5] = {64, 8, (cuuint64_t)kChunks, (cuuint64_t)p.B * p.R / 8, 2};
  const cuuint64_t qs[4] = {2 * kDqk, 64 * e, 8 * 2 * kDqk, kDqk};
  const cuuint32_t qb[5] = {64, 8, (cuuint32_t)kChunks, 2, 1};
  ok = encode(&tm_q, kFp8, kFp8 ? 5 : 4, kFp8 ? static_cast<const void*>(p.terms) : p.q, qd, qs, qb);
  // (64 dims, cache row, chunk): a page's chunks as [chunk][row][64 dims]
  const cuuint64_t d[3] = {64, (cuuint64_t)p.num_pages * kPage, (cuuint64_t)kChunks};
  const cuuint64_t s[2] = {kDqk * e, 64 * e};
  const cuuint32_t b4[3] = {64, (cuuint32_t)kPage, 4}, b1[3] = {64, (cuuint32_t)kPage, 1};
  ok = ok && encode(&tm_kv4, kFp8, 3, kv, d, s, b4) && encode(&tm_kv1, kFp8, 3, kv, d, s, b1);
  if (!ok) return cudaErrorInvalidValue;
  const cudaError_t err = host::ensure_dynamic_smem(
      reinterpret_cast<const void*>(&prefix_kernel<kFp8>), smem_bytes<kFp8>());
  if (err != cudaSuccess) return err;
  cudaLaunchAttribute attr[2];
  attr[0] = pdl_attribute();
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = 2;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(2 * pairs);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem_bytes<kFp8>();
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, prefix_kernel<kFp8>, tm_q, tm_kv4, tm_kv1, p);
}

}  // namespace

int max_pairs() {
  // CTA pairs that the device runs at once (its GPCs may leave SMs without a
  // partner): one wave of them, asked once per context
  static host::PerContext<int> known;
  int n = 0;
  const void* kernel = reinterpret_cast<const void*>(&prefix_kernel<false>);
  if (!known.get(kernel, n, [&](int& v) {
        if (host::ensure_dynamic_smem(kernel, smem_bytes<false>()) != cudaSuccess) return false;
        cudaLaunchAttribute attr;
        attr.id = cudaLaunchAttributeClusterDimension;
        attr.val.clusterDim.x = 2;
        attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3(2);
        cfg.blockDim = dim3(kThreads);
        cfg.dynamicSmemBytes = smem_bytes<false>();
        cfg.attrs = &attr;
        cfg.numAttrs = 1;
        return cudaOccupancyMaxActiveClusters(&v, kernel, &cfg) == cudaSuccess && v > 0;
      }))
    return 0;
  return std::min(n, 256);
}

cudaError_t launch_prep(const Params& p, bool fp8, int pairs, const OwnPlan& own,
                        cudaStream_t stream) {
  cudaLaunchAttribute attr = pdl_attribute();
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(2 + p.B + (fp8 ? ceil_div(p.B * p.R, kPrepThreads / 32) : 0));
  cfg.blockDim = dim3(kPrepThreads);
  cfg.stream = stream;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, prefix_prep_kernel, p, own, pairs);
}

cudaError_t launch_attend(const Params& p, const void* kv, bool fp8, int pairs, cudaStream_t stream) {
  return fp8 ? attend<true>(p, kv, pairs, stream) : attend<false>(p, kv, pairs, stream);
}

template <int kVec>
static cudaError_t join(const Params& p, const OwnPieces& own, cudaStream_t stream) {
  using J = Join<kVec>;
  const cudaError_t e = host::ensure_dynamic_smem(
      reinterpret_cast<const void*>(&prefix_join_kernel<kVec>), J::kSmem);
  if (e != cudaSuccess) return e;
  cudaLaunchAttribute attr = pdl_attribute();
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(p.B * p.R / J::kRowsB + own.num_units * (kRows / J::kRowsB));
  cfg.blockDim = dim3(256);
  cfg.dynamicSmemBytes = J::kSmem;
  cfg.stream = stream;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, prefix_join_kernel<kVec>, p, own);
}

cudaError_t launch_join(const Params& p, const OwnPieces& own, cudaStream_t stream) {
  return p.B * p.R >= kManyRows ? join<4>(p, own, stream) : join<1>(p, own, stream);
}

}  // namespace prefix
}  // namespace mla
