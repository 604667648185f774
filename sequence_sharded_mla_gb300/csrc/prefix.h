// What the C entry of the shared-prefix attention hands its kernels.
#pragma once

#include "common.cuh"

namespace mla {
namespace prefix {

constexpr int kPairRows = 128;   // query rows of a CTA pair (64 per CTA)
constexpr long long kMinGain = 12000;   // ns that sharing has to save

struct Params {
  int B, q_len, H, R;            // R = q_len * H rows per request
  int causal, num_pages, max_pages, groups;
  int max_units;
  float scale_log2;
  const int32_t* block_table;
  const int32_t* seq_lens;
  const int32_t* q_lens;         // or null
  const int32_t* group_starts;   // [groups + 1]
  const int32_t* prefix_lens;    // [groups]
  const uint16_t* q;             // [B * R, 576]
  const float* kv_scale;         // e4m3: [num_pages * 64]
  uint8_t* terms;                // e4m3: the query's two terms [B * R, 2, 576]
  float* inv_scale;              // e4m3: [B * R]
  int32_t* own_lens;             // [B] tokens behind the shared pages
  int32_t* own_table;            // [B, max_pages] their pages
  int2* group_info;              // [2, groups] shared pages and first unit, a block's each
  int2* members;                 // [B] a request's first run in its group, the group's first unit
  int4* units;                   // [max_units] runs, -, table row, shared pages
  int32_t* runs;                 // [max_units, 8] first row of every 16 rows of a unit
  int32_t* where;                // [B * R / 16] unit * 8 + run of every 16 rows, -1: in none
  int* positions;                // [max_units + 1] work positions before each unit
  WsHeader* work;                // the work list's header
  unsigned* err;                 // the call's error word
  float* ws_o;                   // [pairs * 2, 128, 512] pieces of split units
  float* ws_lse;                 // [pairs * 2, 128]
  float* out;                    // [B * R, 512]: slice 0 of the outputs
  float* lse;                    // [B * R]
  unsigned long long timeout_ns;
  int withhold_query;            // testing aid: a pair's first query is never loaded
  int always;                    // testing aid: share whatever can be shared
};

// The per-request kernel's work over the own tokens: its plan, and what it
// leaves in pieces.
struct OwnPlan {
  ProblemDesc pd;
  WsHeader* hdr;
  int* positions;
  int grid, min_tiles, unit_cost;
};
struct OwnPieces {
  ProblemDesc pd;
  const WsHeader* hdr;
  const int* positions;
  const float* ws_o;
  const float* ws_lse;
  float* out;
  float* lse;
  int num_units;
};

int max_pairs();                 // CTA pairs that can run at once; 0 on an error
cudaError_t launch_prep(const Params& p, bool fp8, int pairs, const OwnPlan& own, cudaStream_t stream);
cudaError_t launch_attend(const Params& p, const void* kv, bool fp8, int pairs, cudaStream_t stream);
cudaError_t launch_join(const Params& p, const OwnPieces& own, cudaStream_t stream);

}  // namespace prefix
}  // namespace mla
