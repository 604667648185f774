// Grouped-query attention over an e4m3 cache with a scale for each block of
// tokens and KV head.  For a query row and the tokens it sees in a shard:
//
//   s_t = scale q . K_t sk(t),  lse = ln sum exp(s_t),
//   o = sum exp(s_t - lse) V_t sv(t)
//
// with K_t, V_t the codes' values and sk, sv the scales of t's block.
//
// Work unit: (request, shard, KV head, group of up to R query rows), R = 16,
// 32 or 48 rows (of the KV head's q_len * G, position by position).
// Persistent CTAs walk a stream-K list of 128-token tiles.
// The kernel is bound by the cache's bytes as long as it feeds the tensor
// cores from what TMA brings in, so nothing of the cache is expanded: both
// MMAs take K and V as e4m3 codes from shared memory, as their 128-row A
// operand, and a tile is read from there once for all query rows:
//
//   S^T [128 tokens, R]  = K Q^T     (A: K, K-major; B: Q, two e4m3 terms)
//   O^T [128 dims, 3R]  += V^T P^T   (A: V, MN-major; B: P, three e5m2 terms)
//
//   Q: a power-of-two scale per row puts max|q| in [128, 256), then q = hi +
//      lo in e4m3: exact for values within 2^-10 of the row's largest, off by
//      2^-18 of it below.  The two terms are two MMA chains into one S.
//   P: thread t holds token t of the tile for every row.  The weight carries
//      its block's V scale: with b_t = s_t log2(e) + log2|sv|, P_t = 2^(b_t -
//      m), and the normaliser sums P_t / |sv| = 2^(s_t log2(e) - m), so one
//      running reference m serves rows whose scales lie far apart.  m puts the
//      largest weight at 2^12 and moves (rescaling O) once one passes 2^15.
//      P goes to fp16, off by 2^-11 of its value, and from there without loss
//      to three e5m2 terms, down to 2^-17: a token 2^-29 below the row's
//      largest weight (2^-27 below that of the first tile, whose references
//      are likely to grow) still counts.  (Two e4m3 terms end 2^-18 below it,
//      and a million such tokens are not nothing.)  The terms are three blocks
//      of the MMA's columns, so V is read once for all three; the epilogue
//      adds their sums.
//
// Tile g belongs to softmax group g & 1, each with its own S buffer, weights,
// reference and O^T accumulator, joined by their references at the end of a
// piece.  The groups never wait for one another inside a piece.
//
// CTAs work in teams of up to 8, a member per KV head: the members walk the
// same tiles of neighbouring heads at the same time, so that the heads' 128-byte
// runs of a token, which lie side by side, are read together.  (Each CTA on its
// own, heads are read at unrelated times: 128 against 114 us for 32 requests x
// 20000 tokens x 4 heads, 200 against 170 us for 8 x 65536 tokens x 8 heads.)
//
// Warps: 0 and 3 producers (block table, TMA boxes of K or V, cp.async of the
// tokens' scales); 1 loads and splits each piece's query rows but the first's,
// a piece ahead of the softmax, and issues K Q^T; 2 issues V^T P^T; 4..7 and
// 8..11 the softmax groups (TMEM lane quadrant = warp % 4), which write the
// outputs.
//
// Measured, with the join and the shards' combine: 32 requests x 20000 tokens x
// 4 heads, 16 rows a unit, 112 us (5.8 TB/s; the partial kernel 6.0, of 6.5
// that it reaches where nothing is ragged); one request of 1M tokens x 8 heads
// in 8 shards 363 us (5.9 TB/s, the producers' cp.async); a ragged verify of up
// to 9 tokens over 16 x 6600 tokens x 8 heads, 32 rows a unit, 83 us (the
// softmax groups: 2900 cycles a tile each); 1024 tokens 11.5 us.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <math_constants.h>

#include <algorithm>
#include <climits>
#include <cmath>
#include <type_traits>

#include "common.cuh"
#include "host_util.h"
#include "mla_dcp.h"
#include "ptx.cuh"

namespace mla {
namespace gqa8 {

constexpr int kD = 128;                    // head width
constexpr int kTok = 128;                  // tokens of a tile
constexpr int kStageBytes = kTok * kD;     // 16384: K or V of a tile
constexpr int kMaxStages = 6, kSBufs = 4;
constexpr int kThreads = 384;
constexpr int kGroupThreads = 128;
constexpr uint32_t kBarAll = 1, kBarGroup = 2;   // group g: kBarGroup + g
constexpr int kMinTilesPerCta = 2;
constexpr int kMaxR = 48;                  // query rows of the largest work unit
constexpr int kMaxOwnPlan = 768;           // units that every CTA plans for itself
constexpr int kOwnPerThread = (kMaxOwnPlan + kThreads - 1) / kThreads;
constexpr unsigned long long kTimeoutNs = 2000000000ull;
constexpr float kTop = 12.0f;              // log2 of the largest weight at a new reference
constexpr float kTopFirst = 10.0f;         // and at a piece's first (verify of 48 rows a unit: 8 of
                                           // 8 tiles moved a reference at 12, 2 of 8 at 10)
constexpr float kMost = 15.0f;             // log2 of the largest weight that fits fp16
constexpr float kNoRef = -1.0e38f;         // reference of a row that has seen nothing
constexpr float kMinScale = 8.67361737988403547e-19f;   // 2^-60
constexpr float kMaxScale = 1.32922799578491587e36f;    // 2^120

struct Desc {
  int B, q_len, H;
  int Hkv, lg_team;    // KV heads; log2 of the CTAs of a team
  Div Hg;              // teams' worth of KV heads: Hkv >> lg_team
  Div G;
  int rg;              // query rows per group
  int unit_cost;       // tiles that a unit's start and end are worth
  Div Gq;              // row groups per (request, KV head)
  Div num_shards;
  int shard_first;
  Div n_out;
  int layout, local, causal;
  int num_pages, max_pages, lg_block;
  int room;            // tokens of a context that its block-table row has pages for
  int lg_run;          // log2 of the consecutive slots of a tile that share a scale
  int nv;              // page boxes per 64 slots: shards of a whole-request interleaved cache, else 1
  float scale_log2;
  const uint16_t* q;
  const uint8_t *k, *v;
  const float *ks, *vs;
  const int32_t *block_table, *seq_lens, *q_lens;
};

struct Params {
  Desc d;
  float* out;          // [n_out, B, q_len, H, 128]
  float* lse;          // [n_out, B, q_len, H]
  WsHeader* hdr;
  int* prefix;
  float* ws_o;         // [grid * 2, 64, 128]
  float* ws_lse;       // [grid * 2, 64]
  int4* rec;           // [grid] what each CTA leaves for the merge kernel (make_record)
  int units;
  int own_plan;        // 1: every CTA plans for itself
  unsigned long long timeout_ns;
  int withhold_query;
};

struct Rows {
  int b, so, kh;
  int r0;              // first row: row r0 + r is position (r0 + r) / G, head (r0 + r) % G
  int rows;            // rows of the group in the output
};

struct Unit : Rows {
  int s, L, qn;
  int live;            // rows that attend
  int tiles, tstart, tend, p0, npages;
};

// Unit u (batch, shard, heads of a team, row group) of a team's member.
__device__ __forceinline__ Rows make_rows(const Desc& d, int u, int member) {
  Rows x;
  int t = u / d.Gq;
  x.r0 = (u - t * d.Gq) * d.rg;
  const int v = t / d.Hg;
  x.kh = ((t - v * d.Hg) << d.lg_team) + member;
  x.b = v / d.n_out;
  x.so = v - x.b * d.n_out;
  x.rows = min(d.rg, d.q_len * d.G - x.r0);
  return x;
}

__device__ __forceinline__ Unit make_unit(const Desc& d, int u, int member) {
  Unit x;
  static_cast<Rows&>(x) = make_rows(d, u, member);
  x.s = d.shard_first + x.so;
  x.L = max(d.seq_lens[x.b], 0);
  x.qn = d.q_lens ? min(max(d.q_lens[x.b], 0), d.q_len) : d.q_len;
  x.live = min(max(x.qn * d.G - x.r0, 0), x.rows);
  const int room = min(x.L, d.room);           // a longer context is cut there and reported
  x.tstart = x.p0 = 0;
  x.tend = room;
  const int L = x.live > 0 ? room : 0;
  int n;                                       // the shard's tokens
  if (d.layout == kInterleaved) {
    n = L > x.s ? (L - 1 - x.s) / d.num_shards + 1 : 0;
    x.tiles = ceil_div(n, kTok);
  } else {
    const int c = L / d.num_shards + (L % d.num_shards != 0);
    x.tstart = min(x.s * c, L);
    x.tend = min(x.tstart + c, L);
    n = x.tend - x.tstart;
    if (d.local || n == 0) {
      x.tiles = ceil_div(n, kTok);
    } else {
      x.p0 = x.tstart / kPage;
      x.tiles = ceil_div((x.tend - 1) / kPage - x.p0 + 1, kTok / kPage);
    }
  }
  x.npages = ceil_div(d.local ? n : L, kPage);
  return x;
}

// Slot a of tile j holds position base + (128 j + a) step, if that is in
// [tstart, tend).
struct Slots {
  int base, step;
};

__device__ __forceinline__ Slots make_slots(const Desc& d, const Unit& x) {
  if (d.layout == kInterleaved) return Slots{x.s, d.num_shards};
  return Slots{d.local ? x.tstart : x.p0 * kPage, 1};
}

__device__ __forceinline__ size_t out_row(const Desc& d, const Rows& x, int r) {
  const int i = (x.r0 + r) / d.G, h = x.kh * d.G + (x.r0 + r) - i * d.G;
  return (((size_t)x.so * d.B + x.b) * d.q_len + i) * d.H + h;
}

// A piece's query, by row.
struct Query {
  alignas(16) float qs[kMaxR];   // 1 / the row's query scale
  int lim[kMaxR];                // last position the row sees
  alignas(16) int orow[kMaxR];   // its output row
};

struct Misc {
  uint64_t k_full[kMaxStages], k_empty[kMaxStages], v_full[kMaxStages], v_empty[kMaxStages];
  uint64_t s_full[kSBufs], s_empty[kSBufs], p_full[2], pv_done[2];
  uint64_t q_full[2], q_empty[2], drain;
  uint32_t tmem_base;
  int abort;
  unsigned err;
  int wsum[kThreads / 32];      // planning: the warps' sums
  Query query[2];               // of this piece and the next
  alignas(16) float m[2][kMaxR];      // per group: the rows' references, negated
  // per group, by row: the factor of what has been summed so far when the
  // references move, and of the group's accumulator at the end of a piece
  alignas(16) float f[2][kMaxR];
  // per group, warp and row: the largest logits when the references move, and
  // the sums at the end of a piece
  float part[2][4][kMaxR];
  int moved[2][kMaxR / 16];     // per group: a reference of these 16 rows moved
  // this piece, the next; per dim: the first partly seen token whose V is NaN
  int nan_from[2][kD];
  float ksc[kMaxStages][kTok], vsc[kMaxStages][kTok];   // by run of slots with one scale
  int4 rec;
  int prefix[kMaxOwnPlan + 1];
};

// A CTA whose first tile is not its unit's first: (unit, 2 c0 + slot of c0's
// piece, pieces, error bits), c0 being the team of the unit's first piece; team
// c0 + k holds piece k, in slot 0.  Other CTAs: unit -1.
__device__ __forceinline__ int4 make_record(const int* prefix, int u, int lo, int hi, int per,
                                            int unit_cost) {
  int4 r = make_int4(-1, 0, 0, 0);
  if (lo >= hi) return r;
  const int us = unit_tile_start(prefix, u, unit_cost), ue = prefix[u + 1];
  if (lo <= us || lo >= ue) return r;
  const int c0 = us / per;
  r.x = u;
  r.y = 2 * c0 + (c0 * per < prefix[u] ? 1 : 0);
  r.z = (ue - 1) / per - c0 + 1;
  return r;
}

// Stages: what fits beside the weights and the queries.  A tile's V is held
// until its P V; where fewer than six of both fit, K is let go after the
// logits, has fewer of them, and the scales come with V (9-token verify over 8
// heads 136 -> 123 us; the same at R = 16: 132 -> 137 us, as the logits then
// wait for V).  Two S buffers per group, so that a tile's logits are there
// when the group comes back from the one before.
template <int R>
struct Smem {
  static constexpr bool kEarlyK = R > 16;
  static constexpr int kKStages = kEarlyK ? 4 : 6;
  static constexpr int kVStages = R == 48 ? 5 : 6;
  static_assert(kEarlyK || kKStages == kVStages, "one ring");
  // The query's two terms side by side as 2R columns of one MMA chain, added
  // by the softmax, or (no columns left) as two chains into the same R.  Half
  // the MMAs to issue, about 100 cycles each, against an addition per logit:
  // 32 requests x 20000 tokens x 4 heads, R = 16: 137.6 against 139.5 us.
  static constexpr bool kSplit = R <= 32;
  static constexpr uint32_t kSCols = kSplit ? 2 * R : R;
  static constexpr uint32_t kColO = kSBufs * kSCols;        // O^T after the S buffers
  static constexpr uint32_t kTmemCols = R == 16 ? 256 : 512;
  static_assert(kColO + 6 * R <= kTmemCols, "TMEM columns");
  static constexpr int kQBuf = 2 * R * kD;
  static constexpr int kQ = 0;                              // two buffers
  // term `term` of row r within a buffer
  static __device__ __forceinline__ int q_row(int r, int term) {
    return (kSplit ? 2 * (r & ~15) + 16 * term + (r & 15) : term * R + r) * kD;
  }
  // P: blocks of 16 weights (rows of one term), unswizzled
  static constexpr int kP = 2 * kQBuf;                      // [2 groups][3][R / 16][128 tokens][16]
  static constexpr int kPBlock = 16 * kTok;
  static constexpr int kPGroup = 3 * R * kTok;
  static constexpr int kK = (kP + 2 * kPGroup + 1023) & ~1023;
  static constexpr int kV = kK + kKStages * kStageBytes;
  static constexpr int kMisc = kV + kVStages * kStageBytes;
  static constexpr int kBytes = kMisc + (int)sizeof(Misc) + 1024;   // + alignment slack
  static_assert(kBytes <= 232448, "shared memory budget");
};

__global__ void __launch_bounds__(1024) gqa_fp8_plan_kernel(Desc d, WsHeader* hdr, int* prefix,
                                                            int4* rec, int teams) {
  griddep_launch_dependents();
  __shared__ unsigned bad;
  if (threadIdx.x == 0) bad = 0;
  __syncthreads();
  if (d.q_lens != nullptr)
    for (int b = threadIdx.x; b < d.B; b += 1024)
      if (d.q_lens[b] < 1 || d.q_lens[b] > d.q_len) atomicOr(&bad, kErrQLens);
  __syncthreads();
  plan_units(d.B * d.n_out * d.Hg * d.Gq, [&](int u) { return make_unit(d, u, 0).tiles; }, hdr,
             prefix, teams, kMinTilesPerCta, d.unit_cost, 0u);
  if (threadIdx.x == 0) *rec = make_int4(-1, 0, 0, (int)bad);
}

// Largest of the lanes' values that are not NaN.
__device__ __forceinline__ float warp_max(float x) {
  float y;
  asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(y) : "f"(x));
  return y;
}

// Sums of 16 values over the warp: lane k, and lane 16 + k, gets that of v[k].
__device__ __forceinline__ float warp_sums(float (&v)[16], int lane) {
#pragma unroll
  for (int s = 8; s > 0; s >>= 1) {
    const bool upper = lane & s;
#pragma unroll
    for (int k = 0; k < s; ++k)
      v[k] = (upper ? v[k + s] : v[k]) +
             __shfl_xor_sync(0xffffffffu, upper ? v[k] : v[k + s], s);
  }
  return v[0] + __shfl_xor_sync(0xffffffffu, v[0], 16);
}

__device__ __forceinline__ float lg2_approx(float x) {
  float y;
  asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ float rcp_approx(float x) {   // within 1 ulp
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ float2 as_f2(uint32_t a, uint32_t b) {
  return make_float2(__uint_as_float(a), __uint_as_float(b));
}
// Two fp32 operations in one instruction.
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 d;
  asm("{\n\t.reg .b64 a, b, c, d;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\t"
      "mov.b64 c, {%6, %7};\n\tfma.rn.f32x2 d, a, b, c;\n\tmov.b64 {%0, %1}, d;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return d;
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  float2 d;
  asm("{\n\t.reg .b64 a, b, d;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\t"
      "mul.rn.f32x2 d, a, b;\n\tmov.b64 {%0, %1}, d;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  float2 d;
  asm("{\n\t.reg .b64 a, b, d;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\t"
      "add.rn.f32x2 d, a, b;\n\tmov.b64 {%0, %1}, d;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}

// Weights of two rows as three e5m2 terms, which are the top bytes of fp16
// values: of the weight in fp16, of what that leaves, and of what is left then,
// each rounded to nearest (half a last place added to the bits).  The first
// term leaves at most 2^-3 of the value's power of two, the second 2^-7; that
// is a multiple of fp16's last place, 2^-10, of three bits: the third is exact,
// down to e5m2's least value 2^-16.  Returns the first two terms in the top
// bytes of t0, t1 and the third as a byte pair.  (A NaN's first two terms come
// out as zeros, its third as NaN.)
__device__ __forceinline__ void split_e5m2(float a, float b, uint32_t& t0, uint32_t& t1,
                                           uint32_t& t2) {
  constexpr uint32_t kHalf = 0x00800080u, kTopBytes = 0xFF00FF00u;
  __half2 x = __floats2half2_rn(a, b);
  t0 = *reinterpret_cast<uint32_t*>(&x) + kHalf;
  uint32_t h = t0 & kTopBytes;
  __half2 y = __hsub2(x, *reinterpret_cast<__half2*>(&h));
  t1 = *reinterpret_cast<uint32_t*>(&y) + kHalf;
  h = t1 & kTopBytes;
  y = __hsub2(y, *reinterpret_cast<__half2*>(&h));
  unsigned short c;
  asm("cvt.rn.satfinite.e5m2x2.f16x2 %0, %1;" : "=h"(c) : "r"(*reinterpret_cast<uint32_t*>(&y)));
  t2 = c;
}

template <int R>
__global__ void __launch_bounds__(kThreads, 1)
    gqa_fp8_partial_kernel(const __grid_constant__ CUtensorMap tm_k,
                           const __grid_constant__ CUtensorMap tm_v, Params p) {
  using S = Smem<R>;
  constexpr int kKStages = S::kKStages, kVStages = S::kVStages;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  Misc* misc = reinterpret_cast<Misc*>(smem + S::kMisc);
  const Desc& d = p.d;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t sQ = smem_u32(smem + S::kQ), sP = smem_u32(smem + S::kP);
  const uint32_t sK = smem_u32(smem + S::kK), sV = smem_u32(smem + S::kV);
  auto bar = [&](const uint64_t* b) { return smem_u32(b); };
  volatile int* abort_flag = &misc->abort;
  const uint64_t tmo = p.timeout_ns;
  auto fail = [&]() {
    atomicOr(&misc->err, kErrTimeout);
    *abort_flag = 1;
  };
  // Waits as a warp; a wait that runs out ends the kernel for every role.
  auto wait = [&](const uint64_t* b, int parity) {
    const bool ok = __all_sync(0xffffffffu, mbar_wait(bar(b), parity, tmo, abort_flag));
    if (!ok && lane == 0) fail();
    return ok;
  };

  if (threadIdx.x == 0) {
    for (int st = 0; st < kMaxStages; ++st) {
      // expect_tx, and one cp.async arrival per lane
      mbar_init(bar(&misc->k_full[st]), 1 + 32);
      mbar_init(bar(&misc->v_full[st]), 1 + 32);
      mbar_init(bar(&misc->k_empty[st]), 1);
      mbar_init(bar(&misc->v_empty[st]), 1);
    }
    for (int k = 0; k < kSBufs; ++k) {
      mbar_init(bar(&misc->s_full[k]), 1);
      mbar_init(bar(&misc->s_empty[k]), 4);
    }
    for (int g = 0; g < 2; ++g) {
      mbar_init(bar(&misc->p_full[g]), 4);
      mbar_init(bar(&misc->pv_done[g]), 1);
    }
    for (int k = 0; k < 2; ++k) {
      mbar_init(bar(&misc->q_full[k]), 8);
      mbar_init(bar(&misc->q_empty[k]), 8);
    }
    mbar_init(bar(&misc->drain), 2);
    misc->abort = 0;
    misc->err = 0;
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(&misc->tmem_base), S::kTmemCols);
    tmem_relinquish();
  }
  if (warp == 0 && lane == 0) {
    tma_prefetch_desc(&tm_k);
    tma_prefetch_desc(&tm_v);
  }
  if (threadIdx.x < 2 * kMaxR) misc->m[threadIdx.x / kMaxR][threadIdx.x % kMaxR] = -kNoRef;
  if (threadIdx.x < 2 * kD) misc->nan_from[threadIdx.x / kD][threadIdx.x % kD] = INT_MAX;
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = misc->tmem_base;
  griddep_wait();                // everything before reads and writes nothing global
  griddep_launch_dependents();

  // The plan: the exclusive prefix of the units' work positions, and every
  // CTA's share of them.  A few units are planned by every CTA for itself in
  // shared memory, which costs less than another launch and its results'
  // way through global memory.
  const int member = blockIdx.x & ((1 << d.lg_team) - 1), team = blockIdx.x >> d.lg_team;
  const int teams = gridDim.x >> d.lg_team;
  const int* prefix = p.prefix;
  int W, per;
  if (p.own_plan) {
    const int upt = ceil_div(p.units, kThreads), u0 = threadIdx.x * upt;
    int cost[kOwnPerThread], sum = 0;
#pragma unroll
    for (int k = 0; k < kOwnPerThread; ++k) {
      cost[k] = 0;
      if (k < upt && u0 + k < p.units) {
        const int t = make_unit(d, u0 + k, 0).tiles;
        cost[k] = t > 0 ? t + d.unit_cost : 0;
      }
      sum += cost[k];
    }
    int run = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, run, o);
      if (lane >= o) run += v;
    }
    if (lane == 31) misc->wsum[warp] = run;
    if (blockIdx.x == 0 && d.q_lens != nullptr)
      for (int b = threadIdx.x; b < d.B; b += kThreads)
        if (d.q_lens[b] < 1 || d.q_lens[b] > d.q_len) atomicOr(&misc->err, kErrQLens);
    __syncthreads();
    int base = run - sum;
    W = 0;
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) {
      if (w < warp) base += misc->wsum[w];
      W += misc->wsum[w];
    }
#pragma unroll
    for (int k = 0; k < kOwnPerThread; ++k) {
      if (k < upt && u0 + k < p.units) misc->prefix[u0 + k] = base;
      base += cost[k];
    }
    per = max(kMinTilesPerCta, ceil_div(W, teams));
    if (threadIdx.x == 0) misc->prefix[p.units] = W;
    prefix = misc->prefix;
    __syncthreads();
  } else {
    W = p.hdr->total_cost;
    per = p.hdr->per_cta;
  }
  const int lo = team * per, hi = min(lo + per, W);   // no piece if lo >= W

  PieceIter it;
  it.init_warp(prefix, p.units, lo, hi, d.unit_cost, lane);
  int armed[kMaxStages];                         // the round a producer last filled a stage in
  for (int st = 0; st < kMaxStages; ++st) armed[st] = -1;
  int unit, t0, t1, slot;
  bool whole, ok = true;

  // Rows [ra, rb) of a piece's query, by a warp: they come in by cp.async, half
  // a row to each of the places of its two terms, and are split in place, a few
  // at a time.  The loops stay rolled: code that runs once a piece costs its
  // own fetch (unrolled over 48 rows, 38000 cycles).
  auto fetch_query = [&](const Rows& x, int buf, int ra, int rb) {
    const int L = max(d.seq_lens[x.b], 0);
    const int qn = d.q_lens ? min(max(d.q_lens[x.b], 0), d.q_len) : d.q_len;
    const int live = min(qn * d.G - x.r0, x.rows);
    Query& query = misc->query[buf];
    const int first_src = (x.b * d.q_len) * d.H + x.kh * d.G + x.r0;
    const int step = d.H - d.G;                  // between a position's heads and the next's
#pragma unroll 2
    for (int r0 = ra; r0 < rb; r0 += 2) {
      const int r = r0 + (lane >> 4), c = lane & 15;
      const int i = (x.r0 + r) / d.G, src = first_src + r + i * step;
      const bool there = r < live;
      cp_async_16_zfill(sQ + buf * S::kQBuf + S::q_row(r, c >> 3) + 16 * (c & 7),
                        d.q + (there ? (size_t)src * kD + 8 * c : 0), there ? 16 : 0);
      if (c == 0) {
        query.orow[r] = x.so * (d.B * d.q_len * d.H) + src;
        query.lim[r] = d.causal && there ? L - qn + i : INT_MAX - 1;
      }
    }
    cp_async_commit();
  };
  auto split_query = [&](int buf, int r0, auto rows) {   // rows r0 .. r0 + n - 1
    constexpr int n = decltype(rows)::value;
    cp_async_wait_all();
    __syncwarp();
    uint8_t* const sq = smem + S::kQ + buf * S::kQBuf;
    uint2 w[n];
    uint32_t mx[n];
#pragma unroll
    for (int k = 0; k < n; ++k)
      w[k] = *reinterpret_cast<const uint2*>(sq + S::q_row(r0 + k, lane >> 4) + 8 * (lane & 15));
#pragma unroll
    for (int k = 0; k < n; ++k)
      mx[k] = __reduce_max_sync(0xffffffffu,
                                max(max(w[k].x & 0x7FFFu, (w[k].x >> 16) & 0x7FFFu),
                                    max(w[k].y & 0x7FFFu, (w[k].y >> 16) & 0x7FFFu)));
    uint32_t mine = 0;
#pragma unroll
    for (int k = 0; k < n; ++k) {
      // s_r = 2^(134 - e) puts max|q| (exponent e) in [128, 256); clamped so
      // that it and its inverse are normal
      const float sc = __uint_as_float((261u - min(max(mx[k] >> 7, 8u), 254u)) << 23);
      const uint32_t s0 = split_e4m3x2(__uint_as_float(w[k].x << 16) * sc,
                                       __uint_as_float(w[k].x & 0xFFFF0000u) * sc);
      const uint32_t s1 = split_e4m3x2(__uint_as_float(w[k].y << 16) * sc,
                                       __uint_as_float(w[k].y & 0xFFFF0000u) * sc);
      uint8_t* dst = sq + (((lane >> 2) ^ ((r0 + k) & 7)) << 4) + (lane & 3) * 4;
      *reinterpret_cast<uint32_t*>(dst + S::q_row(r0 + k, 0)) = __byte_perm(s0, s1, 0x5410);
      *reinterpret_cast<uint32_t*>(dst + S::q_row(r0 + k, 1)) = __byte_perm(s0, s1, 0x7632);
      if (lane == k) mine = mx[k] >> 7;
    }
    if (lane < n) {
      if (mine == 255u) atomicOr(&misc->err, kErrQRange);
      misc->query[buf].qs[r0 + lane] = __uint_as_float((min(max(mine, 8u), 254u) - 7u) << 23);
    }
    fence_proxy_async_smem();
    __syncwarp();
  };

  if (warp == 0 || warp == 3) {
    // ------------------------------------------------------------ producers
    // warp 0 loads K, warp 3 V: a box costs the warp that issues it 100 cycles
    // and more (1 GB over 8 shards, 2 x 16 boxes a tile: one warp 320 us, two
    // 222 us)
    const bool is_v = warp == 3;
    if (is_v && lane == 0) misc->rec = make_record(prefix, it.u, lo, hi, per, d.unit_cost);
    const int nb = 2 * d.nv;                     // page boxes per tile
    const int rp = kPage / d.nv;                 // slots per box
    const int lg_rp = 31 - __clz(rp);
    const CUtensorMap* tm = is_v ? &tm_v : &tm_k;
    const uint64_t* full_bars = is_v ? misc->v_full : misc->k_full;
    const uint64_t* empty_bars = is_v ? misc->v_empty : misc->k_empty;
    const int stages = is_v ? kVStages : kKStages;
    const uint32_t dst0 = is_v ? sV : sK;
    const int lg_sub = 6 - d.lg_block;           // log2 of the scales per page and head
    // 8 shards: 8 rows, 1 KB, of a page.  32 such boxes take longer than the
    // tile's share of HBM; cp.async takes 8 lanes a row instead (one request of
    // 1M tokens x 8 heads: 422 us by boxes, 355 us by rows).
    const bool by_row = d.nv == 8;
    const unsigned page_bytes = kPage * d.Hkv * kD;
    const uint8_t* row_src = (is_v ? d.v : d.k) + 16 * (lane & 7);
    const uint32_t row_dst0 = (lane >> 3) * 128 + (((lane & 7) ^ (lane >> 3)) << 4);
    const uint32_t row_dst1 = row_dst0 + 4 * 128 - 2 * (row_dst0 & 64) + 64;   // row + 4, chunk ^ 4
    const int runs = kTok >> d.lg_run;
    int st = 0, round = 0;
    while (ok && it.next(unit, t0, t1, whole, slot)) {
      const Unit x = make_unit(d, unit, member);
      if (x.L > d.room) atomicOr(&misc->err, kErrBadPage);
      const int32_t* bt = d.block_table + (size_t)x.b * d.max_pages;
      const int res = d.nv > 1 ? x.s : 0;
      auto entry = [&](int j) {                  // page of this lane's box of tile j, or -1
        const int idx = x.p0 + j * nb + lane;
        return (lane < nb && idx < x.npages && idx < d.max_pages) ? __ldg(bt + idx) : -1;
      };
      int next = entry(t0);
      for (int j = t0; j < t1; ++j) {
        int page = next;
        if (j + 1 < t1) next = entry(j + 1);
        const bool there = page >= 0 && page < d.num_pages;
        if (!there) {
          if (lane < nb && x.p0 + j * nb + lane < x.npages) atomicOr(&misc->err, kErrBadPage);
          page = d.num_pages;                    // out of the map: TMA fills zeros
        }
        if (round >= 1 && !(ok = wait(&empty_bars[st], (round - 1) & 1))) break;
        const uint32_t full = bar(&full_bars[st]);
        const uint32_t dst = dst0 + st * kStageBytes;
        if (by_row) {
          if (lane == 0) mbar_arrive(full);
          const uint8_t* src = row_src + (size_t)((res + 8 * (lane >> 3)) * d.Hkv + x.kh) * kD;
          const int step = 32 * d.Hkv * kD;
#pragma unroll
          for (int b0 = 0; b0 < 16; b0 += 8) {
            int pg[8];
#pragma unroll
            for (int b = 0; b < 8; ++b) pg[b] = __shfl_sync(0xffffffffu, page, b0 + b);
#pragma unroll
            for (int b = 0; b < 8; ++b) {
              const uint8_t* from = src + (size_t)(unsigned)pg[b] * page_bytes;
              const uint32_t bytes = pg[b] < d.num_pages ? 16 : 0;
              cp_async_16_zfill(dst + (b0 + b) * 1024 + row_dst0, from, bytes);
              cp_async_16_zfill(dst + (b0 + b) * 1024 + row_dst1, from + step, bytes);
            }
          }
        } else {
          if (lane == 0) {
            mbar_arrive_expect_tx(full, kStageBytes);
            armed[st] = round;
          }
          __syncwarp();
          if (lane < nb)
            tma_load_3d(dst + lane * (rp * kD), tm, full, 0, 0, (page * kPage + res) * d.Hkv + x.kh);
        }
        for (int h = 0; is_v == S::kEarlyK && h < runs; h += 32) {
          const int e = h + lane, a = min(e << d.lg_run, kTok - 1);
          const int pg = __shfl_sync(0xffffffffu, page, a >> lg_rp);
          const int row = res + (a & (rp - 1)) * d.nv;
          const bool ok_pg = pg < d.num_pages;
          // below 2^31, as the cache's rows are
          const int si = ok_pg ? ((pg << lg_sub) + (row >> d.lg_block)) * d.Hkv + x.kh : 0;
          if (e < runs) {
            cp_async_4_zfill(smem_u32(&misc->ksc[st][e]), d.ks + si, ok_pg);
            cp_async_4_zfill(smem_u32(&misc->vsc[st][e]), d.vs + si, ok_pg);
          }
        }
        cp_async_mbar_arrive_noinc(full);
        __syncwarp();
        if (++st == stages) {
          st = 0;
          ++round;
        }
      }
    }
    for (int u = team; is_v && u < p.units; u += teams) {
      if (prefix[u + 1] > prefix[u]) continue;
      const Rows x = make_rows(d, u, member);    // no token in the shard: o = 0, lse = -inf
      for (int r = 0; r < x.rows; ++r) {
        const size_t row = out_row(d, x, r);
        reinterpret_cast<float4*>(p.out + row * kD)[lane] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (lane == 0) p.lse[row] = -CUDART_INF_F;
      }
    }
  } else if (warp == 1) {
    // ------------------------------------------------- the query, K Q^T
    const uint32_t id = idesc_e4m3_f32(kTok, S::kSCols, false, false);
    const uint64_t dk = sw128_desc(sK, 16, 1024);
    int g = 0, pc = 0, st = 0, phase = 0;
    while (ok && it.next(unit, t0, t1, whole, slot)) {
      const int buf = pc & 1;
      if (pc == 0) {
        if (!(ok = wait(&misc->q_full[0], 0))) break;
      } else {
        if (pc >= 2 && !(ok = wait(&misc->q_empty[buf], ((pc >> 1) - 1) & 1))) break;
        fetch_query(make_rows(d, unit, member), buf, 0, R);
#pragma unroll 1
        for (int r0 = 0; r0 < R; r0 += 8) split_query(buf, r0, std::integral_constant<int, 8>());
        if (lane < 8) mbar_arrive(bar(&misc->q_full[buf]));
      }
      const uint64_t dq = sw128_desc(sQ + buf * S::kQBuf, 16, 1024);
      for (int j = t0; j < t1; ++j, ++g) {
        const int sb = g % kSBufs, sr = g / kSBufs;
        if (!(ok = wait(&misc->k_full[st], phase))) break;
        if (d.nv == 8) fence_proxy_async_smem();   // K came by cp.async
        if (sr >= 1 && !(ok = wait(&misc->s_empty[sb], (sr - 1) & 1))) break;
        tc_fence_after();
        if (lane == 0) {
          const uint32_t off = (uint32_t)(st * kStageBytes) >> 4;
#pragma unroll
          for (int k = 0; k < (S::kSplit ? 4 : 8); ++k)   // 32 dims each
            mma_e4m3_ss(tmem + S::kSCols * sb, dk + off + ((32 * (k & 3)) >> 4),
                        dq + (((k >> 2) * R * kD + 32 * (k & 3)) >> 4), id, k != 0);
          mma_commit(bar(&misc->s_full[sb]));
          if (S::kEarlyK) mma_commit(bar(&misc->k_empty[st]));
        }
        __syncwarp();
        if (++st == kKStages) {
          st = 0;
          phase ^= 1;
        }
      }
      ++pc;
    }
  } else if (warp == 2) {
    // ------------------------------------------------------------ V^T P^T
    const uint32_t id = idesc_e4m3_e5m2_f32(kD, 3 * R, true, true);
    const uint64_t dv = sw128_desc(sV, 16, 1024);
    int g = 0, st = 0, phase = 0;
    while (ok && it.next(unit, t0, t1, whole, slot)) {
      for (int j = t0; j < t1; ++j, ++g) {
        const int grp = g & 1, gr = g >> 1;
        if (!(ok = wait(&misc->v_full[st], phase))) break;
        if (!(ok = wait(&misc->p_full[grp], gr & 1))) break;
        if (d.nv == 8) fence_proxy_async_smem();
        tc_fence_after();
        if (lane == 0) {
          // MN-major without swizzling: 8-token groups 128 bytes apart
          const uint64_t dp = sw0_desc(sP + grp * S::kPGroup, 128, S::kPBlock);
          const uint32_t off = (uint32_t)(st * kStageBytes) >> 4;
#pragma unroll
          for (int k = 0; k < 4; ++k)   // 32 tokens each
            mma_e4m3_ss(tmem + S::kColO + 3 * R * grp, dv + off + ((k * 4 * 1024) >> 4),
                        dp + ((k * 32 * 16) >> 4), id, (j >= t0 + 2 || k != 0) ? 1u : 0u);
          mma_commit(bar(&misc->v_empty[st]));
          if (!S::kEarlyK) mma_commit(bar(&misc->k_empty[st]));
          mma_commit(bar(&misc->pv_done[grp]));
        }
        __syncwarp();
        if (++st == kVStages) {
          st = 0;
          phase ^= 1;
        }
      }
    }
  } else {
    // ------------------------------------------------------------ softmax
    const int grp = (warp - 4) >> 2, quad = warp & 3;
    const int gtid = (threadIdx.x - 128) & 127;    // 0..127 in the group: its token of a tile
    const int tid = threadIdx.x - 128;             // 0..255
    const uint32_t lane_off = (uint32_t)(32 * quad) << 16;
    const uint32_t tS = tmem + lane_off, tO = tmem + lane_off + S::kColO;
    float* ref = misc->m[grp];
    // A thread's own wait; the lanes' answers are joined before they matter.
    auto poll = [&](const uint64_t* b, int parity) {
      const bool k = mbar_wait(bar(b), parity, tmo, abort_flag);
      if (!k) fail();
      return k;
    };
    int g = 0, pc = 0;                             // tiles and pieces so far
    int st = grp, phase = 0, gr = 0;               // the group's next tile: stage, its phase, number
    while (ok && it.next(unit, t0, t1, whole, slot)) {
      const Unit x = make_unit(d, unit, member);
      const Slots slots = make_slots(d, x);
      // tiles whose first position is in [tstart, last_full] hold a token that
      // every row sees in every slot
      const int last_all = d.causal ? x.L - x.qn + x.r0 / d.G : INT_MAX;   // that every row sees
      const int last_full = min(x.tend - 1, last_all) - (kTok - 1) * slots.step;
      const Query& query = misc->query[pc & 1];
      int* nan_from = misc->nan_from[pc & 1];
      if (pc == 0) {
        const int first_row = 2 * (warp - 4);
        for (int r0 = first_row; r0 < R; r0 += 16) fetch_query(x, 0, r0, r0 + 2);
#pragma unroll 1
        for (int r0 = first_row; r0 < R; r0 += 16)
          split_query(0, r0, std::integral_constant<int, 2>());
        if (lane == 0 && !p.withhold_query) mbar_arrive(bar(&misc->q_full[0]));
      }
      // the end of the previous piece, or the kernel's start, has set the references
      ok = __all_sync(0xffffffffu, poll(&misc->q_full[pc & 1], (pc >> 1) & 1));

      float2 l[R / 2];
#pragma unroll
      for (int r = 0; r < R / 2; ++r) l[r] = make_float2(0.0f, 0.0f);
      bool first = true;                           // the group's first tile of the piece
      for (int j = t0 + ((g ^ grp) & 1); j < t1; j += 2) {
        // -------------------------------------------------------- logits
        const int sb = kSBufs == 4 ? 2 * (gr & 1) + grp : grp;
        const int s_phase = (kSBufs == 4 ? gr >> 1 : gr) & 1;
        const int tok0 = slots.base + j * kTok * slots.step, t = tok0 + gtid * slots.step;
        const bool full = tok0 >= x.tstart && tok0 <= last_full;
        const bool valid = full || (t >= x.tstart && t < x.tend);
        bool ok_s = ok && poll(S::kEarlyK ? &misc->v_full[st] : &misc->k_full[st], phase);
        float c = 0.0f, lv = 0.0f, inv = 0.0f, fv = 1.0f;
        if (ok_s && valid) {
          c = misc->ksc[st][gtid >> d.lg_run] * d.scale_log2;
          const float sv = misc->vsc[st][gtid >> d.lg_run];
          // |sv| below 2^-60 counts as 2^-60 in the reference and as itself in
          // the product; a scale that is not finite goes to the product alone;
          // one above 2^120, whose inverse may be no normal number, is reported
          float ve = sv;
          if (!(sv >= kMinScale && sv <= kMaxScale)) {
            ve = fabsf(sv) < INFINITY ? fmaxf(fabsf(sv), kMinScale) : 1.0f;
            fv = sv / ve;
            if (ve > kMaxScale) atomicOr(&misc->err, kErrQRange);
          }
          lv = lg2_approx(ve);
          inv = rcp_approx(ve);
        }
        const bool scaled = __any_sync(0xffffffffu, fv != 1.0f);
        ok_s = __all_sync(0xffffffffu, ok_s && poll(&misc->s_full[sb], s_phase));
        // 16 rows' logits of this token in log2 units, with the V scale: into
        // b (two rows each), less the references (or, less = 0, without)
        auto logits = [&](int r0, const uint32_t (&sr)[S::kSplit ? 32 : 16], float2* b, float less) {
          const float4* q4 = reinterpret_cast<const float4*>(query.qs + r0);
          const float4* m4 = reinterpret_cast<const float4*>(ref + r0);
          const float2 c2 = make_float2(c, c), lv2 = make_float2(lv, lv);
          const float2 less2 = make_float2(less, less);
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const float4 q = q4[k], m = m4[k];
            float2 v0 = as_f2(sr[4 * k], sr[4 * k + 1]), v1 = as_f2(sr[4 * k + 2], sr[4 * k + 3]);
            if constexpr (S::kSplit) {
              v0 = add2(v0, as_f2(sr[16 + 4 * k], sr[17 + 4 * k]));
              v1 = add2(v1, as_f2(sr[18 + 4 * k], sr[19 + 4 * k]));
            }
            b[2 * k] = fma2(mul2(v0, make_float2(q.x, q.y)), c2, fma2(make_float2(m.x, m.y), less2, lv2));
            b[2 * k + 1] =
                fma2(mul2(v1, make_float2(q.z, q.w)), c2, fma2(make_float2(m.z, m.w), less2, lv2));
          }
          if (!full) {
#pragma unroll
            for (int k = 0; k < 8; ++k) {
              if (!valid || t > query.lim[r0 + 2 * k]) b[k].x = -CUDART_INF_F;
              if (!valid || t > query.lim[r0 + 2 * k + 1]) b[k].y = -CUDART_INF_F;
            }
          }
        };
        // 16 rows' columns of the tile's S
        auto load_s = [&](int r0, uint32_t (&sr)[S::kSplit ? 32 : 16]) {
          const uint32_t a = tS + S::kSCols * sb + (S::kSplit ? 2 * r0 : r0);
          if constexpr (S::kSplit) tmem_ld32(a, sr);
          else tmem_ld16(a, sr);
        };
        float2 b[R / 2];
        auto all_logits = [&](float less) {
          uint32_t sr[2][S::kSplit ? 32 : 16];
          load_s(0, sr[0]);
#pragma unroll
          for (int r0 = 0; r0 < R; r0 += 16) {
            tmem_wait_ld();
            if (r0 + 16 < R) load_s(r0 + 16, sr[((r0 >> 4) + 1) & 1]);
            logits(r0, sr[(r0 >> 4) & 1], b + r0 / 2, less);
          }
        };
        if (ok_s) tc_fence_after();
        bool move = first;                         // a piece's first tile has no references yet
        if (!first) {
          float mx = -CUDART_INF_F;
          if (ok_s) {
            all_logits(1.0f);
#pragma unroll
            for (int k = 0; k < R / 2; ++k) mx = fmaxf(mx, fmaxf(b[k].x, b[k].y));
          }
          move = named_bar_or(kBarGroup + grp, kGroupThreads, mx > kMost || !ok_s);
        }
        // A weight would pass 2^kMost: the logits without references, for new
        // ones, which are then taken off them.
        if (move) {
          if (ok_s) all_logits(0.0f);
          // ---------------------------------------------- new references
          if (ok_s) {
#pragma unroll
            for (int r0 = 0; r0 < R; r0 += 32) {
              float mine = 0.0f;
#pragma unroll
              for (int k = 0; k < 32 && r0 + k < R; ++k) {
                const float2 v = b[(r0 + k) >> 1];
                const float mx = warp_max((k & 1) ? v.y : v.x);
                if (lane == k) mine = mx;
              }
              if (r0 + lane < R) misc->part[grp][quad][r0 + lane] = mine;
            }
          }
          if (named_bar_or(kBarGroup + grp, kGroupThreads, !ok_s)) {
            ok = false;
            break;
          }
          bool up = false;
          if (gtid < R) {
            float top = misc->part[grp][0][gtid];  // NaN loses to any number
            for (int k = 1; k < 4; ++k) top = fmaxf(top, misc->part[grp][k][gtid]);
            const float old = -ref[gtid];
            up = top > old + kMost;
            const float now = top - (first ? kTopFirst : kTop);
            misc->f[grp][gtid] = up ? ex2_approx(old - now) : 1.0f;
            if (up) ref[gtid] = -now;
          }
          const uint32_t ups = __ballot_sync(0xffffffffu, up);
          if (gtid < R && (lane & 15) == 0) misc->moved[grp][gtid >> 4] = (ups >> lane) & 0xFFFFu;
          const bool ok_pv = first || poll(&misc->pv_done[grp], (gr - 1) & 1);
          if (named_bar_or(kBarGroup + grp, kGroupThreads, !ok_pv)) {
            ok = false;
            break;
          }
          if (!first) {
            tc_fence_after();
#pragma unroll
            for (int r = 0; r < R / 2; ++r)
              l[r] = mul2(l[r], make_float2(misc->f[grp][2 * r], misc->f[grp][2 * r + 1]));
#pragma unroll 1
            for (int r0 = 0; r0 < R; r0 += 16) {
              if (!misc->moved[grp][r0 >> 4]) continue;
              const float4* f4 = reinterpret_cast<const float4*>(misc->f[grp] + r0);
#pragma unroll 1
              for (int term = 0; term < 3; ++term) {
                uint32_t v[16];
                tmem_ld16(tO + 3 * R * grp + R * term + r0, v);
                tmem_wait_ld();
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                  const float4 f = f4[k];
                  v[4 * k] = __float_as_uint(__uint_as_float(v[4 * k]) * f.x);
                  v[4 * k + 1] = __float_as_uint(__uint_as_float(v[4 * k + 1]) * f.y);
                  v[4 * k + 2] = __float_as_uint(__uint_as_float(v[4 * k + 2]) * f.z);
                  v[4 * k + 3] = __float_as_uint(__uint_as_float(v[4 * k + 3]) * f.w);
                }
                tmem_st16(tO + 3 * R * grp + R * term + r0, v);
              }
            }
            tmem_wait_st();
          }
#pragma unroll
          for (int k = 0; k < R / 4; ++k) {
            const float4 m = reinterpret_cast<const float4*>(ref)[k];
            b[2 * k] = add2(b[2 * k], make_float2(m.x, m.y));
            b[2 * k + 1] = add2(b[2 * k + 1], make_float2(m.z, m.w));
          }
        }
        // ------------------------------------------------------- weights
        tc_fence_before();                         // the logits are in registers
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(&misc->s_empty[sb]));
        // the group's last P V has read the weights' buffer
        if (!first && !__all_sync(0xffffffffu, poll(&misc->pv_done[grp], (gr - 1) & 1))) {
          ok = false;
          continue;                                // the next reduction ends the piece
        }
        // before the next wait that may give up in some warps only: they all
        // have to meet the others in the same reductions of the next tile
        first = false;
        uint8_t* prow = smem + S::kP + grp * S::kPGroup + gtid * 16;
        const float2 inv2 = make_float2(inv, inv);
#pragma unroll
        for (int r0 = 0; r0 < R; r0 += 16) {
          uint32_t w0[4], w1[4], w2[4];
#pragma unroll
          for (int q4 = 0; q4 < 4; ++q4) {
            const int i = (r0 >> 1) + 2 * q4;
            float2 pa = make_float2(ex2_approx(b[i].x), ex2_approx(b[i].y));
            float2 pb = make_float2(ex2_approx(b[i + 1].x), ex2_approx(b[i + 1].y));
            l[i] = fma2(pa, inv2, l[i]);
            l[i + 1] = fma2(pb, inv2, l[i + 1]);
            if (scaled) {                          // a weight of 0 stays 0 under any scale
              pa.x = pa.x != 0.0f ? pa.x * fv : 0.0f;
              pa.y = pa.y != 0.0f ? pa.y * fv : 0.0f;
              pb.x = pb.x != 0.0f ? pb.x * fv : 0.0f;
              pb.y = pb.y != 0.0f ? pb.y * fv : 0.0f;
            }
            uint32_t a0, a1, a2, b0, b1, b2;
            split_e5m2(pa.x, pa.y, a0, a1, a2);
            split_e5m2(pb.x, pb.y, b0, b1, b2);
            w0[q4] = __byte_perm(a0, b0, 0x7531);
            w1[q4] = __byte_perm(a1, b1, 0x7531);
            w2[q4] = a2 | (b2 << 16);
          }
          uint8_t* pb = prow + (r0 >> 4) * S::kPBlock;
          *reinterpret_cast<uint4*>(pb) = make_uint4(w0[0], w0[1], w0[2], w0[3]);
          *reinterpret_cast<uint4*>(pb + R * kTok) = make_uint4(w1[0], w1[1], w1[2], w1[3]);
          *reinterpret_cast<uint4*>(pb + 2 * R * kTok) = make_uint4(w2[0], w2[1], w2[2], w2[3]);
        }
        if (!full) {
          if (!S::kEarlyK && !__all_sync(0xffffffffu, poll(&misc->v_full[st], phase))) {
            ok = false;
            continue;
          }
          // V rows of slots without a token become zeros; a NaN code of a token
          // that not every row sees is taken out too and comes back in the
          // epilogue for the rows that see it (rows see a prefix)
          const int u = gtid & 7;
          uint8_t* vt = smem + S::kV + st * kStageBytes;
#pragma unroll 1
          for (int a = gtid >> 3; a < kTok; a += 16) {
            const int ta = tok0 + a * slots.step;
            uint4* v = reinterpret_cast<uint4*>(vt + a * kD + ((u ^ (a & 7)) << 4));
            if (ta < x.tstart || ta >= x.tend) {
              *v = make_uint4(0, 0, 0, 0);
            } else if (ta > last_all) {
              const uint4 w = *v;
              uint32_t ww[4] = {w.x, w.y, w.z, w.w};
              uint32_t any = 0;
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                // 1 in each byte that is a NaN, whose low seven bits are all ones
                const uint32_t nan = (((ww[k] & 0x7F7F7F7Fu) + 0x01010101u) >> 7) & 0x01010101u;
                any |= nan;
                ww[k] &= ~(nan * 0xFFu);
                for (uint32_t left = nan; left != 0; left &= left - 1)
                  atomicMin(&nan_from[16 * u + 4 * k + ((__ffs(left) - 1) >> 3)], ta);
              }
              if (any) *v = make_uint4(ww[0], ww[1], ww[2], ww[3]);
            }
          }
        }
        fence_proxy_async_smem();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(&misc->p_full[grp]));
        st += 2;
        if (st >= kVStages) {
          st -= kVStages;
          phase ^= 1;
        }
        ++gr;
      }
      g += t1 - t0;
      // ------------------------------------------------------------ epilogue
      // sums over the group's threads, then over its warps, in a fixed order
#pragma unroll
      for (int r0 = 0; r0 < R; r0 += 16) {
        float v[16];
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          v[2 * k] = l[r0 / 2 + k].x;
          v[2 * k + 1] = l[r0 / 2 + k].y;
        }
        const float sum = warp_sums(v, lane);
        if (lane < 16) misc->part[grp][quad][r0 + lane] = sum;
      }
      // the groups' shares of the tiles so far, and of this piece
      const int n0 = (g + 1) >> 1, n1 = g >> 1;
      const int has0 = t1 - t0 > 1 || (g & 1), has1 = t1 - t0 > 1 || !(g & 1);
      bool ok_e = ok;
      if (ok_e && has0) ok_e = poll(&misc->pv_done[0], (n0 - 1) & 1);
      if (ok_e && has1) ok_e = poll(&misc->pv_done[1], (n1 - 1) & 1);
      if (named_bar_or(kBarAll, 2 * kGroupThreads, !ok_e)) {
        ok = false;
        break;
      }
      tc_fence_after();
      const size_t sl = 2 * (size_t)blockIdx.x + slot;
      if (gtid < R) {                              // group 0: factors; group 1: lse
        const int r = gtid;
        float lg[2], M = kNoRef;
        for (int k = 0; k < 2; ++k) {
          lg[k] = (misc->part[k][0][r] + misc->part[k][1][r]) +
                  (misc->part[k][2][r] + misc->part[k][3][r]);
          M = fmaxf(M, -misc->m[k][r]);
        }
        const float w0 = ex2_approx(-misc->m[0][r] - M), w1 = ex2_approx(-misc->m[1][r] - M);
        const float tot = w0 * lg[0] + w1 * lg[1];
        const bool none = tot == 0.0f || r >= x.live;   // not NaN
        if (grp == 0) {
          const float it_ = none ? 0.0f : 1.0f / tot;
          misc->f[0][r] = w0 * it_;
          misc->f[1][r] = w1 * it_;
        } else if (r < x.rows) {
          // the reference and the sum's exponent nearly cancel where V's scales are
          // far from 1 (M = -70, tot = 2^73 under a scale of 0): exact first
          const uint32_t bits = __float_as_uint(tot);
          const bool normal = bits >= (1u << 23) && bits < (255u << 23);
          const int e = normal ? (int)(bits >> 23) - 127 : 0;
          const float one = normal ? __uint_as_float((bits & 0x7FFFFFu) | (127u << 23)) : tot;
          const float v = none ? -CUDART_INF_F
                               : ((M + (float)e) + log2f(one)) * 0.69314718055994530942f;
          if (whole) p.lse[query.orow[r]] = v;
          else p.ws_lse[sl * kRows + r] = v;
        }
      }
      named_bar_sync(kBarAll, 2 * kGroupThreads);
      // thread (quad, lane) holds dim 32 quad + lane of every row; the groups
      // take turns over 16 rows
      const int dim = 32 * quad + lane;
      const int nf = nan_from[dim];
#pragma unroll 1
      for (int r0 = 16 * grp; r0 < x.rows; r0 += 32) {
        float o[16];
#pragma unroll
        for (int k = 0; k < 16; ++k) o[k] = 0.0f;
#pragma unroll 1
        for (int gg = 0; gg < 2; ++gg) {
          if (!(gg ? has1 : has0)) continue;       // its accumulator holds nothing of this piece
          uint32_t v[3][16];
#pragma unroll
          for (int term = 0; term < 3; ++term) tmem_ld16(tO + 3 * R * gg + R * term + r0, v[term]);
          tmem_wait_ld();
          const float4* f4 = reinterpret_cast<const float4*>(misc->f[gg] + r0);
#pragma unroll
          for (int k = 0; k < 16; ++k) {
            const float4 f = f4[k >> 2];
            const float a = (__uint_as_float(v[0][k]) + __uint_as_float(v[1][k])) +
                            __uint_as_float(v[2][k]);
            o[k] = fmaf(a, (k & 3) == 0 ? f.x : (k & 3) == 1 ? f.y : (k & 3) == 2 ? f.z : f.w, o[k]);
          }
        }
        if (nf != INT_MAX || r0 + 16 > x.live) {
#pragma unroll
          for (int k = 0; k < 16; ++k) {
            if (query.lim[r0 + k] >= nf) o[k] = CUDART_NAN_F;
            if (r0 + k >= x.live) o[k] = 0.0f;
          }
        }
        const int n = x.rows - r0;
        if (whole) {
          const int4* o4 = reinterpret_cast<const int4*>(query.orow + r0);
          float* dst = p.out + dim;
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const int4 at = o4[k];
            if (4 * k < n) dst[(size_t)at.x * kD] = o[4 * k];
            if (4 * k + 1 < n) dst[(size_t)at.y * kD] = o[4 * k + 1];
            if (4 * k + 2 < n) dst[(size_t)at.z * kD] = o[4 * k + 2];
            if (4 * k + 3 < n) dst[(size_t)at.w * kD] = o[4 * k + 3];
          }
        } else {
          float* dst = p.ws_o + (sl * kRows + r0) * kD + dim;
#pragma unroll
          for (int k = 0; k < 16; ++k)
            if (k < n) dst[k * kD] = o[k];
        }
      }
      // for the next piece
      if (gtid < R) ref[gtid] = -kNoRef;
      if (tid < kD) misc->nan_from[(pc + 1) & 1][tid] = INT_MAX;
      tc_fence_before();
      named_bar_sync(kBarAll, 2 * kGroupThreads);  // accumulators and exchange are free again
      if (lane == 0) mbar_arrive(bar(&misc->q_empty[pc & 1]));
      ++pc;
    }
  }

  // ---------------------------------------------------------------- teardown
  if (warp == 0 || warp == 3) {
    cp_async_commit();
    cp_async_wait_all();
  }
  tc_fence_before();
  __syncthreads();
  if (*abort_flag) {
    // after a failure, let this CTA's own MMAs and copies complete first
    int never = 0;
    if (lane == 0 && (warp == 1 || warp == 2)) {
      mma_commit(bar(&misc->drain));
      mbar_wait(bar(&misc->drain), 0, kDrainNs, &never);
    }
    if ((warp == 0 || warp == 3) && lane == 0)
      for (int st = 0; st < kMaxStages; ++st)
        if (armed[st] >= 0)
          mbar_wait(bar(warp == 0 ? &misc->k_full[st] : &misc->v_full[st]), armed[st] & 1,
                    kDrainNs, &never);
    tc_fence_before();
    __syncthreads();
  }
  if (threadIdx.x == 0)
    p.rec[blockIdx.x] = make_int4(misc->rec.x, misc->rec.y, misc->rec.z, (int)misc->err);
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, S::kTmemCols);
  }
}

// Joins the pieces of units that teams share, by LSE.  A unit of np pieces has
// np - 1 CTAs that begin inside it; block c stands for CTA c, and those of a
// unit take its rows in turn, so that one long request over all CTAs is joined
// by as many blocks as it has rows.  A block's warps split its rows and, where
// there are fewer rows than warps, a row's pieces; sums go in a fixed order.
// (One block per unit took 180 of 361 us for one request of 4M tokens over
// one KV head, 152 pieces.)  Block 0 joins the error bits.
constexpr int kMergeWarps = 16;

__global__ void __launch_bounds__(32 * kMergeWarps)
    gqa_fp8_merge_kernel(Desc d, WsHeader* hdr, const int4* rec, int records, const float* ws_o,
                         const float* ws_lse, float* out, float* lse) {
  __shared__ float4 part[kMergeWarps][32];
  __shared__ float psum[kMergeWarps];
  const int c = blockIdx.x;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  griddep_wait();
  griddep_launch_dependents();
  if (c == 0) {
    if (warp != 0) return;
    unsigned e = 0;
    for (int k = lane; k < records; k += 32) e |= (unsigned)rec[k].w;
    e = __reduce_or_sync(0xffffffffu, e);
    if (lane == 0) hdr->err = e;
    return;
  }
  const int4 rc = rec[c];
  if (rc.x < 0) return;
  const int member = c & ((1 << d.lg_team) - 1);
  const int c0 = rc.y >> 1, np = rc.z, turn = (c >> d.lg_team) - c0 - 1;
  const Rows x = make_rows(d, rc.x, member);
  const int mine = turn < x.rows ? (x.rows - 1 - turn) / (np - 1) + 1 : 0;
  int wpr = 1;                                   // warps per row
  while (2 * wpr * mine <= kMergeWarps && 2 * wpr <= np) wpr *= 2;
  const int sub = warp % wpr;
  for (int i0 = 0; i0 < mine; i0 += kMergeWarps / wpr) {
    const int i = i0 + warp / wpr;
    const int r = turn + min(i, mine - 1) * (np - 1);
    auto slot_row = [&](int k) -> size_t {       // row r of piece k
      const int cta = ((c0 + k) << d.lg_team) + member;
      return (size_t)(2 * cta + (k == 0 ? rc.y & 1 : 0)) * kRows + r;
    };
    constexpr int kBatch = 4;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    float M = -CUDART_INF_F, wsum = 0.f;
    for (int k0 = sub; k0 < np; k0 += kBatch * wpr) {
      float e[kBatch];
      float4 o[kBatch];
#pragma unroll
      for (int k = 0; k < kBatch; ++k) {
        const int at = k0 + k * wpr;
        e[k] = -CUDART_INF_F;
        if (at < np) {
          const size_t s = slot_row(at);
          e[k] = ws_lse[s];
          o[k] = reinterpret_cast<const float4*>(ws_o + s * kD)[lane];
        }
      }
      if (k0 == sub) {
        for (int k = lane; k < np; k += 32) M = fmaxf(M, ws_lse[slot_row(k)]);
#pragma unroll
        for (int off = 16; off > 0; off >>= 1)
          M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, off));
      }
#pragma unroll
      for (int k = 0; k < kBatch; ++k) {
        if (e[k] == -CUDART_INF_F) continue;     // a NaN goes on
        const float w = __expf(e[k] - M);
        wsum += w;
        acc.x = fmaf(w, o[k].x, acc.x);
        acc.y = fmaf(w, o[k].y, acc.y);
        acc.z = fmaf(w, o[k].z, acc.z);
        acc.w = fmaf(w, o[k].w, acc.w);
      }
    }
    if (wpr > 1) {
      part[warp][lane] = acc;
      if (lane == 0) psum[warp] = wsum;
      __syncthreads();
      if (sub == 0) {
        for (int k = 1; k < wpr; ++k) {
          const float4 a = part[warp + k][lane];
          acc.x += a.x;
          acc.y += a.y;
          acc.z += a.z;
          acc.w += a.w;
          wsum += psum[warp + k];
        }
      }
    }
    if (sub == 0 && i < mine) {
      const size_t row = out_row(d, x, r);
      const bool none = wsum == 0.f;
      const float inv = none ? 0.f : 1.0f / wsum;
      reinterpret_cast<float4*>(out + row * kD)[lane] =
          make_float4(acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv);
      if (lane == 0) lse[row] = none ? -CUDART_INF_F : M + logf(wsum);
    }
  }
}

// ------------------------------------------------------------------ host side
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

// Query rows per work unit: all of a KV head's q_len * G rows of a request up
// to 48, in the smallest tile that holds them; more rows go to groups of 32.
// 16 requests x 6400 tokens x 4 heads, us with groups of up to 48 and 32 rows:
// 36 rows 46 and 50, 48 rows 46 and 50, 64 rows 65 and 52, 72 rows 70 and 69,
// 96 rows 69 and 69, 126 rows 93 and 88; a ragged verify of up to 72 rows 90
// and 82.  Full groups and a rest, not groups of even size, as a padded batch's
// requests often need no rest (that verify in three groups of 24 rows: 110
// when full ones took 93).
//
// Work shared out by tiles: a unit's start and end are worth 4 tiles at 16 rows,
// 6 above (us at 4 and 6: seven requests of up to 5000 tokens, one row a head,
// 14.3 and 14.6; 32 requests x 20000 tokens x 4 heads, 16 rows, 112.4 and
// 113.5; 16 requests x 6400 tokens x 4 heads of 48, 72 and 96 rows, 46 and 44.5,
// 71 and 68, 71 and 68).
struct Split {
  int R, rg, Gq, unit_cost;
  int lg_team, units;   // units a team
};

Split split_for(const gqa_shape* s, int num_shards, int shard_id, int grid) {
  const int n = s->q_len * (s->num_heads / s->num_kv_heads);
  Split x;
  x.Gq = n <= 48 ? 1 : ceil_div(n, 32);
  x.rg = x.Gq == 1 ? n : 32;
  x.R = ceil_div(x.rg, 16) * 16;
  x.unit_cost = x.R == 16 ? 4 : 6;
  x.lg_team = 0;
  while (x.lg_team < 3 && ((s->num_kv_heads | grid) & (1 << x.lg_team)) == 0) ++x.lg_team;
  x.units = s->batch * (shard_id == MLA_ALL_SHARDS ? num_shards : 1) *
            (s->num_kv_heads >> x.lg_team) * x.Gq;
  return x;
}

struct WsLayout {
  size_t rec, prefix, ws_o, ws_lse, total;
};

WsLayout ws_layout(int num_units, int grid) {
  auto up = [](size_t v) { return (v + 255) & ~static_cast<size_t>(255); };
  WsLayout w;
  w.rec = up(sizeof(WsHeader));
  w.prefix = w.rec + up(sizeof(int4) * (size_t)(grid + 1));       // + the plan kernel's
  w.ws_o = w.prefix + up(sizeof(int) * (size_t)(num_units + 1));
  w.ws_lse = w.ws_o + up(sizeof(float) * (size_t)grid * 2 * kRows * kD);
  w.total = w.ws_lse + up(sizeof(float) * (size_t)grid * 2 * kRows);
  return w;
}

int grid_size() { return std::min(host::device_sm_count(), 512); }

template <int R>
cudaError_t launch_partial(const CUtensorMap& tm_k, const CUtensorMap& tm_v, const Params& p,
                           int grid, cudaStream_t st) {
  const cudaError_t e = host::ensure_dynamic_smem(
      reinterpret_cast<const void*>(&gqa_fp8_partial_kernel<R>), Smem<R>::kBytes);
  if (e != cudaSuccess) return e;
  cudaLaunchAttribute attr = pdl_attribute();
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = Smem<R>::kBytes;
  cfg.stream = st;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, gqa_fp8_partial_kernel<R>, tm_k, tm_v, p);
}

}  // namespace gqa8
}  // namespace mla

using namespace mla;

extern "C" {

size_t gqa_fp8_workspace_size(const gqa_shape* shape, int num_shards, int shard_id) {
  if (!gqa8::shape_ok(shape) || !gqa8::shape_supported(shape) ||
      !gqa8::shards_ok(num_shards, shard_id))
    return 0;
  const int grid = gqa8::grid_size();
  if (grid <= 0) return 0;
  return gqa8::ws_layout(gqa8::split_for(shape, num_shards, shard_id, grid).units, grid).total;
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
  const int grid = gqa8::grid_size();
  if (grid <= 0) return MLA_ERR_CUDA;
  const gqa8::Split sp = gqa8::split_for(shape, num_shards, shard_id, grid);
  const gqa8::WsLayout wl = gqa8::ws_layout(sp.units, grid);
  if (workspace_bytes < wl.total) return MLA_ERR_WORKSPACE;
  host::EncodeTiledFn encode = host::encode_fn();
  if (encode == nullptr) return MLA_ERR_CUDA;

  // work positions are 31-bit numbers
  const long long slots = (long long)max_pages_per_req * kPage;
  const long long room = std::min((local ? num_shards : 1) * slots, (long long)INT_MAX);
  const long long tiles = (local ? slots : slots / num_shards) / gqa8::kTok + 3;
  if (sp.units * (tiles + sp.unit_cost) >= (1LL << 31)) return MLA_ERR_UNSUPPORTED;

  gqa8::Desc d;
  d.B = shape->batch;
  d.q_len = shape->q_len;
  d.H = shape->num_heads;
  d.Hkv = shape->num_kv_heads;
  d.lg_team = sp.lg_team;
  d.Hg = make_div(shape->num_kv_heads >> sp.lg_team);
  d.G = make_div(shape->num_heads / shape->num_kv_heads);
  d.rg = sp.rg;
  d.unit_cost = sp.unit_cost;
  d.Gq = make_div(sp.Gq);
  d.num_shards = make_div(num_shards);
  d.shard_first = shard_id == MLA_ALL_SHARDS ? 0 : shard_id;
  d.n_out = make_div(shard_id == MLA_ALL_SHARDS ? num_shards : 1);
  d.layout = (layout & 1) ? kContiguous : kInterleaved;
  d.local = local;
  d.causal = shape->causal;
  d.num_pages = cache->num_pages;
  d.max_pages = max_pages_per_req;
  d.room = (int)room;
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
  d.nv = layout == MLA_LAYOUT_INTERLEAVED ? num_shards : 1;
  d.lg_run = d.lg_block;   // less the stride of a shard's rows within a page
  for (int n = d.nv; n > 1 && d.lg_run > 0; n >>= 1) --d.lg_run;

  // K and V [pages * 64, Hkv, 128 codes] read as (128 codes, row of one shard
  // in a page, cache row x KV head): a box from row (page * 64 + residue) *
  // Hkv + kh lands one page's 64 / nv slots of the shard, 128 bytes each
  CUtensorMap tm_k, tm_v;
  for (int which = 0; which < 2; ++which) {
    const cuuint64_t row = (cuuint64_t)gqa8::kD * d.Hkv;
    cuuint64_t dims[3] = {gqa8::kD, (cuuint64_t)(kPage / d.nv),
                          (cuuint64_t)cache->num_pages * kPage * d.Hkv};
    cuuint64_t strides[2] = {row * d.nv, gqa8::kD};
    cuuint32_t box[3] = {gqa8::kD, (cuuint32_t)(kPage / d.nv), 1};
    cuuint32_t es[3] = {1, 1, 1};
    if (encode(which ? &tm_v : &tm_k, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, which ? cache->v : cache->k,
               dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
               CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
      return MLA_ERR_CUDA;
  }

  uint8_t* ws = static_cast<uint8_t*>(workspace);
  gqa8::Params p;
  p.d = d;
  p.out = out_partial;
  p.lse = lse_partial;
  p.hdr = reinterpret_cast<WsHeader*>(ws);
  p.prefix = reinterpret_cast<int*>(ws + wl.prefix);
  p.ws_o = reinterpret_cast<float*>(ws + wl.ws_o);
  p.ws_lse = reinterpret_cast<float*>(ws + wl.ws_lse);
  p.rec = reinterpret_cast<int4*>(ws + wl.rec);
  p.units = sp.units;
  p.own_plan = sp.units <= gqa8::kMaxOwnPlan;
  p.timeout_ns = host::wait_budget_ns(gqa8::kTimeoutNs);
  p.withhold_query = host::g_withhold_query.load();

  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (!p.own_plan) {
    gqa8::gqa_fp8_plan_kernel<<<1, 1024, 0, st>>>(d, p.hdr, p.prefix, p.rec + grid,
                                                grid >> sp.lg_team);
    if (cudaGetLastError() != cudaSuccess) return MLA_ERR_CUDA;
  }
  void* ev0 = host::g_ev_before.load();
  void* ev1 = host::g_ev_after.load();
  if (ev0 != nullptr && cudaEventRecord(static_cast<cudaEvent_t>(ev0), st) != cudaSuccess)
    return MLA_ERR_CUDA;
  const cudaError_t e = sp.R == 16   ? gqa8::launch_partial<16>(tm_k, tm_v, p, grid, st)
                        : sp.R == 32 ? gqa8::launch_partial<32>(tm_k, tm_v, p, grid, st)
                                     : gqa8::launch_partial<48>(tm_k, tm_v, p, grid, st);
  if (e != cudaSuccess) return MLA_ERR_CUDA;
  if (ev1 != nullptr && cudaEventRecord(static_cast<cudaEvent_t>(ev1), st) != cudaSuccess)
    return MLA_ERR_CUDA;
  cudaLaunchAttribute attr = pdl_attribute();
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(32 * gqa8::kMergeWarps);
  cfg.stream = st;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, gqa8::gqa_fp8_merge_kernel, d, p.hdr,
                            (const int4*)p.rec, p.own_plan ? grid : grid + 1,
                            (const float*)p.ws_o, (const float*)p.ws_lse, out_partial, lse_partial) == cudaSuccess
             ? MLA_OK
             : MLA_ERR_CUDA;
}

}  // extern "C"
