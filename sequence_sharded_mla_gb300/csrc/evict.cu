// Eviction from the paged latent cache by accumulated attention weight: which
// tokens of a context stay, and the move of their rows to new pages.
//
// A context of L tokens with a budget of K keeps its `first` leading tokens,
// its `recent` newest ones and, of the candidates between, the k = K - first -
// recent with the largest weights, the lowest index first among equals.
//
// evict_select_kernel  one cluster of CTAs per request.  A weight becomes a
//     32-bit key whose unsigned order is the weights' order; three passes of
//     11, 11 and 10 bits histogram the keys that match the digits chosen so
//     far and descend into the bin that holds the k-th largest, which leaves
//     its key T and how many of the candidates equal to T are kept.  Then
//     every warp counts the keys above and equal to T in its slice, and with
//     the counts before it writes its kept positions in order.  Counts are
//     integers: the order of the shared-memory atomics cannot change them.
// evict_copy_kernel    one block per new page: 64 rows of the source pages to
//     one page, 16 bytes a thread and load, with their scales and weights.
//
// What bounds them: the copy, memory bandwidth (2 x 1152 or 2 x 580 bytes a
// kept token); the selection of a short context, its chain of cluster
// barriers; of a long one, the instructions of three passes over the weights.
#include <cooperative_groups.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "common.cuh"
#include "host_util.h"
#include "mla_dcp.h"
#include "ptx.cuh"

namespace cg = cooperative_groups;

namespace mla {
namespace evict {

constexpr int kBins = 2048;
constexpr int kCopyThreads = 256;
constexpr int kHold = 16;             // weights per thread in registers
constexpr int kList = 96;             // undecided weights per warp that are listed

struct Select {
  const int32_t* seq_lens;
  const float* weights;
  long long stride;                   // floats between requests' weights
  int width;                          // weights per request
  const int32_t* keep;
  const int32_t* keep_first;          // or null
  int recent;
  int max_pages;
  int32_t* new_lens;
  int32_t* kept;
  int max_keep;
  unsigned* err;
};

struct Copy {
  uint8_t* data;
  float* scale;                       // e4m3 only
  int num_pages;
  const int32_t* seq_lens;
  const int32_t* block_table;
  int max_pages;
  const int32_t* new_block_table;
  int new_max_pages;
  const float* weights;
  long long stride;
  float* weights_out;                 // or null
  const int32_t* new_lens;
  const int32_t* kept;
  int max_keep;
  Div pages;                          // blocks per request
  unsigned* err;
};

// Unsigned key in the order of the weights: -inf first, both zeros alike, NaN
// above everything (a sum with 0 makes -0 the other zero, and any NaN the one of
// all ones behind a sign of 0).
__device__ __forceinline__ uint32_t key_of(float w) {
  const uint32_t u = __float_as_uint(__fadd_rn(w, 0.0f));
  return u ^ ((uint32_t)((int)u >> 31) | 0x80000000u);
}

template <int kWarps>
struct Shared {
  uint32_t hist[kBins];               // this CTA's digits
  uint32_t total[3][kBins];           // rank 0: the cluster's, by pass
  uint32_t warp_sum[kWarps];
  uint32_t gt[kWarps], eq[kWarps];    // per warp's slice: keys above, equal to T
  uint32_t total_gt, total_eq;        // the CTA's
  uint32_t bin[3], above[3];          // the descent's choices
  uint32_t list[kWarps][kList];       // keys with the first chosen digit, in order
};

// C: CTAs per request (a cluster of them).  (One CTA per SM: without that bound
// the 512 threads get 40 registers, spill and take 12.1 instead of 10.7 us.)
template <int C, int kThreads>
__global__ void __launch_bounds__(kThreads, 1) evict_select_kernel(Select p) {
  constexpr int kWarps = kThreads / 32, kOwn = kBins / kThreads;   // bins per thread
  __shared__ Shared<kWarps> sm;
  cg::cluster_group cluster = cg::this_cluster();
  auto sync = [&]() {
    if (C == 1) __syncthreads();
    else cluster.sync();
  };
  const int rank = (int)(blockIdx.x % C), b = (int)(blockIdx.x / C);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  griddep_wait();
  griddep_launch_dependents();
  const int given = p.seq_lens[b], budget = p.keep[b];
  const int L = (int)max(0LL, min((long long)given, min((long long)p.width,
                                                        (long long)p.max_pages * kPage)));
  const int K = max(0, min(budget, p.max_keep));
  if (rank == 0 && tid == 0 && (L != given || K != budget)) atomicOr(p.err, kErrQLens);
  const int n_new = min(L, K);
  const int first = p.keep_first != nullptr ? max(0, min(p.keep_first[b], n_new)) : 0;
  const int recent = min(p.recent, n_new - first);
  int32_t* out = p.kept + (size_t)b * p.max_keep;
  if (rank == 0 && tid == 0) p.new_lens[b] = n_new;
  const int gid = rank * kThreads + tid, step = C * kThreads;
  const bool cut = n_new < L;
  const int head = cut ? first : n_new;
  for (int j = gid; j < head; j += step) out[j] = j;
  for (int j = n_new + gid; j < p.max_keep; j += step) out[j] = -1;
  if (cut)
    for (int i = gid; i < recent; i += step) out[n_new - recent + i] = L - recent + i;
  const int k = n_new - first - recent;       // candidates to keep
  if (!cut || k == 0) return;                 // uniform over the cluster

  const float* w = p.weights + (size_t)b * p.stride + first;
  const int n = L - recent - first;           // candidates, more than k
  // each warp has a slice [wa, wz) of whole groups of 32; its keys stay in
  // registers if there are at most kHold a thread, else every pass reads them
  const int per_warp = ((n + C * kWarps - 1) / (C * kWarps) + 31) & ~31;
  const int wa = (int)min((long long)n, (long long)(rank * kWarps + warp) * per_warp);
  const int wz = min(n, wa + per_warp);
  const bool held = per_warp <= 32 * kHold;
  uint32_t key[kHold];
  auto load = [&](int i0) {
    float v[kHold];
#pragma unroll
    for (int u = 0; u < kHold; ++u) {
      const int i = i0 + 32 * u + lane;
      v[u] = i < wz ? __ldg(w + i) : 0.0f;
    }
#pragma unroll
    for (int u = 0; u < kHold; ++u) key[u] = key_of(v[u]);
  };
  // f(key, candidate) in every lane for 32 candidates at a time, in order
  auto each = [&](auto&& f) {
    for (int i0 = wa; i0 < wz; i0 += 32 * kHold) {
      if (!held) load(i0);
#pragma unroll
      for (int u = 0; u < kHold; ++u)
        if (i0 + 32 * u < wz) f(key[u], i0 + 32 * u + lane);
    }
  };
  if (held) load(wa);

  uint32_t sure = 0, listed = 0;              // above the first digit; sharing it
  const uint32_t below = (1u << lane) - 1;
  // f(key, whether there is one) for the weights that share the first digit,
  // from the list or, if they are too many for it, from all of the slice
  auto undecided = [&](auto&& f) {
    if (listed <= kList) {
      for (uint32_t i0 = 0; i0 < listed; i0 += 32)
        f(i0 + lane < listed ? sm.list[warp][i0 + lane] : 0u, i0 + lane < listed);
    } else {
      each([&](uint32_t x, int i) { f(x, i < wz && (x >> 21) == sm.bin[0]); });
    }
  };

  for (int i = tid; i < 3 * kBins; i += kThreads) (&sm.total[0][0])[i] = 0;
  uint32_t match = 0, left = (uint32_t)k;     // digits so far; still to take below them
  int upper = 32;
#pragma unroll 1
  for (int pass = 0; pass < 3; ++pass) {
    const int bits = pass < 2 ? 11 : 10;
    const int shift = upper - bits;
    const uint32_t mask = (1u << bits) - 1;
    // one CTA counts straight into the totals
    uint32_t* hist = C == 1 ? sm.total[pass] : sm.hist;
    if (C > 1)
      for (int i = tid; i < kBins; i += kThreads) hist[i] = 0;
    if (C > 1 && pass == 0) cluster.sync();   // rank 0's totals are zero
    else __syncthreads();
    // Equal digits, such as those of many weights of zero, meet in one addition of
    // the shared-memory atomics.  (Counting zeros by ballot took 104 instead of
    // 100 us for a million tokens, grouping all equal digits 2.5 times as long.)
    auto count = [&](uint32_t x, bool in) {
      if (in) atomicAdd(&hist[(x >> shift) & mask], 1u);
    };
    if (pass == 0) {
      each([&](uint32_t x, int i) { count(x, i < wz); });
    } else if (pass == 1) {
      // the weights above the first digit are kept; those that share it are
      // listed, so that later passes read only them (two of five reads less)
      each([&](uint32_t x, int i) {
        const bool in = i < wz && (x >> upper) == match;
        sure += __popc(__ballot_sync(0xFFFFFFFFu, i < wz && (x >> upper) > match));
        const uint32_t m = __ballot_sync(0xFFFFFFFFu, in);
        if (m == 0) return;
        const uint32_t at = listed + __popc(m & below);
        if (in && at < kList) sm.list[warp][at] = x;
        listed += __popc(m);
        count(x, in);
      });
      __syncwarp();
    } else {
      undecided([&](uint32_t x, bool in) { count(x, in && (x >> upper) == match); });
    }
    __syncthreads();
    if (C > 1) {
      // the few digits that occur go to rank 0 (every CTA reading all of the
      // others' bins took 15 us a pass)
      uint32_t* total = cluster.map_shared_rank(sm.total[pass], 0);
      for (int i = tid; i < kBins; i += kThreads)
        if (hist[i] != 0) atomicAdd(total + i, hist[i]);
      cluster.sync();
    }
    if (rank == 0) {
      uint32_t c[kOwn], own = 0;
#pragma unroll
      for (int j = 0; j < kOwn; ++j) own += c[j] = sm.total[pass][kOwn * tid + j];
      // keys in bins above this thread's: a suffix sum over the threads
      uint32_t suf = own;
#pragma unroll
      for (int off = 1; off < 32; off <<= 1) {
        const uint32_t o = __shfl_down_sync(0xFFFFFFFFu, suf, off);
        if (lane + off < 32) suf += o;
      }
      if (lane == 0) sm.warp_sum[warp] = suf;
      __syncthreads();
      uint32_t above = suf - own;
      for (int v = warp + 1; v < kWarps; ++v) above += sm.warp_sum[v];
#pragma unroll
      for (int j = kOwn - 1; j >= 0; --j) {
        if (above < left && left <= above + c[j])   // one bin of one thread
          for (int r = 0; r < C; ++r) {
            *(C == 1 ? &sm.bin[pass] : cluster.map_shared_rank(&sm.bin[pass], r)) = kOwn * tid + j;
            *(C == 1 ? &sm.above[pass] : cluster.map_shared_rank(&sm.above[pass], r)) = above;
          }
        above += c[j];
      }
    }
    sync();
    match = (match << bits) | sm.bin[pass];
    left -= sm.above[pass];
    upper = shift;
  }
  const uint32_t T = match;      // the k-th largest key; `left` of its equals stay

  // each warp's slice, in order
  uint32_t gt = sure, eq = 0;
  undecided([&](uint32_t x, bool in) {
    gt += __popc(__ballot_sync(0xFFFFFFFFu, in && x > T));
    eq += __popc(__ballot_sync(0xFFFFFFFFu, in && x == T));
  });
  if (lane == 0) {
    sm.gt[warp] = gt;
    sm.eq[warp] = eq;
  }
  __syncthreads();
  uint32_t gt0 = 0, eq0 = 0;     // before this warp's slice
  for (int v = 0; v < warp; ++v) {
    gt0 += sm.gt[v];
    eq0 += sm.eq[v];
  }
  if (tid == kThreads - 1) {     // the last warp's: the CTA's totals
    sm.total_gt = gt0 + gt;
    sm.total_eq = eq0 + eq;
  }
  if (C > 1) cluster.sync();
  for (int r = 0; r < rank; ++r) {
    gt0 += *cluster.map_shared_rank(&sm.total_gt, r);
    eq0 += *cluster.map_shared_rank(&sm.total_eq, r);
  }
  // (at: where the slice's next weight goes, of those above T and the equal ones
  // that stay)
  uint32_t at = (uint32_t)first + gt0 + min(eq0, left);
  each([&](uint32_t x, int i) {
    bool stays = i < wz && x > T;
    const uint32_t me = __ballot_sync(0xFFFFFFFFu, i < wz && x == T);
    if (me != 0) {
      stays |= i < wz && x == T && eq0 + __popc(me & below) < left;
      eq0 += __popc(me);
    }
    const uint32_t m = __ballot_sync(0xFFFFFFFFu, stays);
    if (stays) out[at + __popc(m & below)] = first + i;
    at += __popc(m);
  });
  if (C > 1) cluster.sync();     // peers have read this CTA's totals
}

// Block: one new page of one request.  kVec 16-byte pieces per row.
template <int kVec>
__global__ void __launch_bounds__(kCopyThreads) evict_copy_kernel(Copy p) {
  __shared__ long long src[kPage];    // first row's byte / 16 .. of each row, -1: not moved
  __shared__ int bad;
  const int b = (int)blockIdx.x / p.pages, pg = (int)blockIdx.x - b * p.pages.d;
  const int tid = threadIdx.x;
  if (tid == 0) bad = 0;
  griddep_wait();
  griddep_launch_dependents();
  const int n = p.new_lens[b], j0 = pg * kPage;
  if (j0 >= n) return;
  const int rows = min(kPage, n - j0);
  const int page = p.new_block_table[(size_t)b * p.new_max_pages + pg];
  const bool page_ok = page >= 0 && page < p.num_pages;
  if (!page_ok) {
    if (tid == 0) atomicOr(p.err, kErrBadPage);
  }
  __syncthreads();
  const int32_t* bt = p.block_table + (size_t)b * p.max_pages;
  float w = 0.f, sc = 0.f;
  bool move = false;
  if (tid < kPage) {
    long long at = -1;
    if (tid < rows) {
      const int j = j0 + tid;
      const int t = p.kept[(size_t)b * p.max_keep + j];
      const int sp = bt[t / kPage];
      const bool ok = sp >= 0 && sp < p.num_pages;
      if (!ok) atomicOr(p.err, kErrBadPage);
      if (p.weights_out != nullptr) w = p.weights[(size_t)b * p.stride + t];
      // a row that stays where it is; any other into the request's own page of
      // that index would overwrite rows that other blocks still read
      const bool stays = page == sp && t == j;
      if (!stays && page_ok && pg < p.max_pages && j0 < p.seq_lens[b] && bt[pg] == page) bad = 1;
      if (ok && page_ok && !stays) {
        at = (long long)sp * kPage + t % kPage;
        move = true;
        if (p.scale != nullptr) sc = p.scale[at];
      }
      if (p.weights_out != nullptr) p.weights_out[(size_t)b * p.max_keep + j] = w;
    }
    src[tid] = at;
  }
  __syncthreads();
  if (bad) {
    if (tid == 0) atomicOr(p.err, kErrQLens);
    return;
  }
  if (p.scale != nullptr && move) p.scale[(size_t)page * kPage + tid] = sc;
  if (!page_ok) return;
  const uint4* from = reinterpret_cast<const uint4*>(p.data);
  uint4* to = reinterpret_cast<uint4*>(p.data) + (size_t)page * kPage * kVec;
  constexpr int kItems = kPage * kVec / kCopyThreads;   // 18 (bf16), 9 (e4m3)
  constexpr int kBatch = 9;
  static_assert(kItems % kBatch == 0, "whole batches");
#pragma unroll 1
  for (int i0 = 0; i0 < kItems; i0 += kBatch) {
    uint4 v[kBatch];
    bool live[kBatch];
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      const int e = (i0 + i) * kCopyThreads + tid, r = e / kVec, c = e - r * kVec;
      const long long s = src[r];
      live[i] = s >= 0;
      if (live[i]) v[i] = from[s * kVec + c];
    }
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      const int e = (i0 + i) * kCopyThreads + tid;
      if (live[i]) to[e] = v[i];
    }
  }
}

// Bytes of an array, or null.
struct Span {
  const void* p;
  size_t n;
};
inline bool overlap(const Span& a, const Span& b) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a.p), y = reinterpret_cast<uintptr_t>(b.p);
  return a.p != nullptr && b.p != nullptr && x < y + b.n && y < x + a.n;
}

// CTAs per request, by the width of the weights.  A whole eviction to a quarter
// (e4m3) with one CTA of 512 threads, and clusters of 4, 8 and 16 of 1024:
//   4 x 777       9.0,  14.5,  14.5,  16.6 us
//   16 x 8000    13.8,  18.1,  28.6,  44.1
//   16 x 40000   64.3,  50.7,  61.8,  78.4
//   4 x 131000    154,  54.4,  47.1,  47.5
//   1 x 1048576  1004,   225,   145,  97.6 (107 if all weights are equal)
template <int C, int kThreads>
cudaError_t select(const Select& s, int batch, cudaStream_t stream) {
  const void* kernel = reinterpret_cast<const void*>(&evict_select_kernel<C, kThreads>);
  if (C > 8) {
    // beyond the portable cluster size: allowed once per context
    static host::PerContext<int> done;
    int ok = 0;
    if (!done.get(kernel, ok, [&](int& v) {
          v = 1;
          return cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) ==
                 cudaSuccess;
        }))
      return cudaErrorInitializationError;
  }
  cudaLaunchAttribute attr[2];
  attr[0] = pdl_attribute();
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = C;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = C > 1 ? 2 : 1;
  cfg.gridDim = dim3((unsigned)(batch * C));
  cfg.blockDim = dim3(kThreads);
  return cudaLaunchKernelEx(&cfg, evict_select_kernel<C, kThreads>, s);
}

}  // namespace evict
}  // namespace mla

using namespace mla;

extern "C" mla_status mla_cache_evict(const mla_kv_pages* kv, const int32_t* block_table,
                                      int max_pages_per_req, const int32_t* seq_lens, int batch,
                                      const float* weights, long long weights_stride,
                                      int weights_width, const int32_t* keep,
                                      const int32_t* keep_first, int recent,
                                      const int32_t* new_block_table, int new_max_pages,
                                      int32_t* new_seq_lens, int32_t* kept, int max_keep,
                                      float* weights_out, void* workspace, size_t workspace_bytes,
                                      void* stream) {
  using host::aligned4;
  if (kv == nullptr || kv->data == nullptr || !host::aligned16(kv->data) || kv->num_pages < 1)
    return MLA_ERR_INVALID;
  if (kv->dtype != MLA_KV_BF16 && kv->dtype != MLA_KV_FP8_E4M3) return MLA_ERR_INVALID;
  const bool fp8 = kv->dtype == MLA_KV_FP8_E4M3;
  if (fp8 != (kv->scale != nullptr) || !aligned4(kv->scale)) return MLA_ERR_INVALID;
  if (!block_table || !seq_lens || !weights || !keep || !new_block_table || !new_seq_lens || !kept)
    return MLA_ERR_INVALID;
  if (!aligned4(block_table) || !aligned4(seq_lens) || !aligned4(weights) || !aligned4(keep) ||
      !aligned4(keep_first) || !aligned4(new_block_table) || !aligned4(new_seq_lens) ||
      !aligned4(kept) || !aligned4(weights_out))
    return MLA_ERR_INVALID;
  if (batch < 1 || max_pages_per_req < 1 || new_max_pages < 1 || recent < 0 || max_keep < 1 ||
      weights_width < 1 || weights_stride < weights_width)
    return MLA_ERR_INVALID;
  const int pages = (max_keep - 1) / kPage + 1;
  if (new_max_pages < pages) return MLA_ERR_INVALID;
  if (kv->page_size != kPage) return MLA_ERR_UNSUPPORTED;
  if (workspace == nullptr || !host::aligned16(workspace) || workspace_bytes < sizeof(WsHeader))
    return MLA_ERR_WORKSPACE;
  // candidates and kept positions are indexed in 32 bits, with a cluster's rounding
  // behind them
  if (weights_width > (1 << 30) || max_keep > (1 << 30)) return MLA_ERR_UNSUPPORTED;
  // inputs are read by every CTA while another writes, and the copy takes the
  // lengths and positions of the selection for indexes
  const size_t row = sizeof(int32_t) * (size_t)batch;   // of 4-byte values, one a request
  const evict::Span in[] = {
      {seq_lens, row},
      {keep, row},
      {keep_first, row},
      {weights, sizeof(float) * ((batch - 1) * (size_t)weights_stride + weights_width)},
      {block_table, row * max_pages_per_req},
      {new_block_table, row * new_max_pages}};
  const evict::Span out[] = {
      {new_seq_lens, row}, {kept, row * max_keep}, {weights_out, row * max_keep}};
  for (int i = 0; i < 3; ++i) {
    for (const evict::Span& x : in)
      if (evict::overlap(out[i], x)) return MLA_ERR_INVALID;
    for (int j = 0; j < i; ++j)
      if (evict::overlap(out[i], out[j])) return MLA_ERR_INVALID;
  }
  if ((long long)batch * pages >= (1LL << 31) || (long long)batch * 16 >= (1LL << 31))
    return MLA_ERR_INVALID;
  unsigned* err = &static_cast<WsHeader*>(workspace)->err;
  const evict::Select s{seq_lens,   weights,           weights_stride, weights_width, keep,
                        keep_first, recent,            max_pages_per_req, new_seq_lens, kept,
                        max_keep,   err};
  const evict::Copy c{static_cast<uint8_t*>(const_cast<void*>(kv->data)),
                      const_cast<float*>(kv->scale),
                      kv->num_pages,
                      seq_lens,
                      block_table,
                      max_pages_per_req,
                      new_block_table,
                      new_max_pages,
                      weights,
                      weights_stride,
                      weights_out,
                      new_seq_lens,
                      kept,
                      max_keep,
                      make_div(pages),
                      err};
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const cudaError_t se = weights_width <= 8192     ? evict::select<1, 512>(s, batch, st)
                         : weights_width <= 65536  ? evict::select<4, 1024>(s, batch, st)
                         : weights_width <= 262144 ? evict::select<8, 1024>(s, batch, st)
                                                   : evict::select<16, 1024>(s, batch, st);
  if (se != cudaSuccess) return MLA_ERR_CUDA;
  cudaLaunchAttribute attr = pdl_attribute();
  cudaLaunchConfig_t cfg = {};
  cfg.stream = st;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  cfg.gridDim = dim3((unsigned)(batch * pages));
  cfg.blockDim = dim3(evict::kCopyThreads);
  const cudaError_t e =
      fp8 ? cudaLaunchKernelEx(&cfg, evict::evict_copy_kernel<kDqk / 16>, c)
          : cudaLaunchKernelEx(&cfg, evict::evict_copy_kernel<2 * kDqk / 16>, c);
  return e == cudaSuccess ? MLA_OK : MLA_ERR_CUDA;
}
