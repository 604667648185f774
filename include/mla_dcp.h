/*
 * mla_dcp.h -- C ABI of the sequence-sharded MLA decode library (sm_103a).
 *
 * The operation is the data-parallel core of Decode Context Parallelism
 * ("Decode Context Parallelism", sections 4 and 4.1): the latent KV cache of
 * a multi-head latent attention (MLA) model is split along the sequence;
 * every shard attends the full query over only its slice and emits a partial
 * output plus a log-sum-exp (LSE); a combine step reweights the partials by
 * their LSEs, optionally fused with the per-head value up-projection
 * ("Kimi K3 in vLLM: Specialized CuTe DSL Decode on NVIDIA GB300",
 * section 1).  On one GPU the N shards are logical partitions of the cache.
 *
 * Conventions for every entry point:
 *   - Pointers named "device" must be device memory of the current CUDA
 *     device, 16-byte aligned (4-byte for the int32 arrays block_table,
 *     seq_lens and q_lens, so that views of a larger batch can be passed).
 *     The caller owns every buffer; the library
 *     keeps no pointer after a call returns and allocates no device memory
 *     at run time (its one static buffer, the scratch of
 *     mla_decode_partial_noalloc, exists from library load to process exit).
 *   - Calls are asynchronous on `stream` (a cudaStream_t passed as void*;
 *     NULL is the legacy default stream).  Argument errors are detected on
 *     the host and returned before anything is launched.
 *   - No C++ exception crosses this boundary.
 *   - Results are deterministic: the same inputs give bitwise-identical
 *     outputs (fixed reduction order, no atomics on data).
 *
 * Layouts (row-major, bf16 = IEEE bfloat16 bit patterns in uint16):
 *   q            bf16  [B, q_len, H, 576]  absorbed queries: 512 latent + 64 rope
 *   kv data      bf16  [num_pages, 64, 576]  latent rows [c_kv(512) | k_rope(64)]
 *                e4m3  [num_pages, 64, 576]  (fp8 caches, OCP e4m3 codes)
 *   kv scale     fp32  [num_pages, 64]     fp8 only: value = e4m3(code) * scale
 *   block_table  int32 [B, max_pages_per_req]  page of token t of request b is
 *                                          block_table[b][t / 64], row t % 64
 *   seq_lens     int32 [B]                 context length L_b (>= 1), device
 *   out_partial  fp32  [n_out, B, q_len, H, 512]  normalised partial outputs
 *   lse_partial  fp32  [n_out, B, q_len, H]       natural-log LSE, -inf if empty
 *   w_uv         bf16  [H, 512, 128]       per-head value up-projection
 *   out          bf16  [B, q_len, H, 512]  (or [B, q_len, H, 128] with w_uv)
 *   lse_out      fp32  [B, q_len, H]
 */
#ifndef MLA_DCP_H_
#define MLA_DCP_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum mla_status {
  MLA_OK = 0,
  MLA_ERR_INVALID = -1,       /* bad argument; nothing was launched */
  MLA_ERR_UNSUPPORTED = -2,   /* well-formed but outside what this build supports */
  MLA_ERR_CUDA = -3,          /* a CUDA runtime or driver call failed */
  MLA_ERR_TIMEOUT = -4,       /* a device-side wait gave up (from mla_get_device_error) */
  MLA_ERR_DEVICE_BOUNDS = -5, /* a block-table entry was outside [0, num_pages) */
  MLA_ERR_WORKSPACE = -6,     /* workspace missing or smaller than mla_workspace_size() */
  MLA_ERR_RANGE = -7          /* fp8 cache: an inf or NaN query value in a row that attends,
                                 or a finite V scale of a block above 2^120 */
} mla_status;

/* Which token positions of a request belong to shard s of N
 * ("Decode Context Parallelism", section 4):
 *   INTERLEAVED  t mod N == s                  (any N <= 8)
 *   CONTIGUOUS   s*c <= t < min((s+1)*c, L),   c = ceil(L / N)
 * The section's worked example (a 200K-token request on 4 GPUs holding
 * 0-50K, 50K-100K, 100K-150K, 150K-200K) is the CONTIGUOUS layout.
 * With these two the cache and block table describe whole requests (every
 * position t at page block_table[b][t / 64], row t % 64).
 *
 * The *_LOCAL layouts are the same shards, stored the way each GPU of a
 * multi-GPU deployment holds its slice (section 4: each GPU stores only its
 * chunk): the cache and block table hold only shard `shard_id`'s positions,
 * in order, compactly -- local position p of request b is page
 * block_table[b][p / 64], row p % 64, and is global position p*N + s
 * (INTERLEAVED_LOCAL, any N <= 8) or s*c + p (CONTIGUOUS_LOCAL).  seq_lens
 * stay the global lengths L_b: they fix the shard's token count and the
 * causal mask.  shard_id must name one shard. */
typedef enum mla_layout {
  MLA_LAYOUT_INTERLEAVED = 0,
  MLA_LAYOUT_CONTIGUOUS = 1,
  MLA_LAYOUT_INTERLEAVED_LOCAL = 2,
  MLA_LAYOUT_CONTIGUOUS_LOCAL = 3
} mla_layout;

typedef enum mla_kv_dtype { MLA_KV_BF16 = 0, MLA_KV_FP8_E4M3 = 1 } mla_kv_dtype;

/* Decode-step shape.  num_heads must be a multiple of 16.  With an fp8
 * cache the tensor cores take each query row as a two-term e4m3 sum under a
 * power-of-two row scale (exact for components within 2^10 of the row's
 * largest; any finite bf16 value is accepted); an inf or NaN component of a
 * row that attends is reported as MLA_ERR_RANGE by mla_get_device_error.
 * Probabilities times token scales are two-term e4m3 sums as well, under a
 * reference that follows the logits tile by tile: off by 2^-8 of themselves
 * near the largest of their tile (64 tokens; 128 behind a shared prefix), and lost
 * only where they are 2^-7 of that or less at worst, 2^-12 mostly.
 * With causal != 0
 * (a speculative verify step of q_len = 1 + drafts tokens whose KV is the
 * last q_len entries of the cache), query i sees tokens t <= L - q_len + i. */
typedef struct mla_shape {
  int batch;            /* B >= 1 */
  int q_len;            /* query tokens per request >= 1 (the padded count, see q_lens) */
  int num_heads;        /* H: multiple of 16 */
  int causal;           /* 0 or 1 */
  float softmax_scale;  /* logits = softmax_scale * q . k  (1/sqrt(192) for the workloads here) */
  /* Optional (NULL = every request has q_len query tokens), device int32
   * [B]: request b has q_lens[b] in [1, q_len] query tokens -- a batch of
   * verify steps with different draft counts padded to q_len.  Rows
   * i >= q_lens[b] are padding: their partials are o = 0, lse = -inf and
   * their combined output is 0.  With causal, query i of request b sees
   * t <= L_b - q_lens[b] + i.  A value outside [1, q_len] is clamped and
   * reported as MLA_ERR_INVALID by mla_get_device_error.  Ignored by
   * mla_shard_combine and mla_workspace_size. */
  const int32_t* q_lens;
} mla_shape;

/* The paged latent cache (device memory, not modified). */
typedef struct mla_kv_pages {
  const void* data;     /* [num_pages, page_size, 576] bf16 or e4m3 */
  const float* scale;   /* fp8 only: [num_pages, page_size]; must be NULL for bf16 */
  mla_kv_dtype dtype;
  int num_pages;        /* >= 1 */
  int page_size;        /* must be 64 */
} mla_kv_pages;

/* shard_id value that computes every shard 0..N-1 in one call (n_out = N). */
#define MLA_ALL_SHARDS (-1)

/*
 * Bytes of device workspace mla_decode_partial needs for this shape on the
 * current device (work list, split-piece partials and an error word).
 * Returns 0 for invalid arguments.
 */
size_t mla_workspace_size(const mla_shape* shape, int num_shards, int shard_id);

/*
 * Per-shard partial attention ("Decode Context Parallelism", section 4.1,
 * the "Compute" step; section 5.3: each rank attends over its latent slice).
 * For every request b, query row (i, h) and computed shard s, over the tokens
 * T_s of request b that shard s owns (see mla_layout) and the query may see:
 *     s_t = softmax_scale * q[b,i,h,:] . K_t            (K_t = cache row, 576 wide)
 *     lse_partial = ln sum_{t in T_s} exp(s_t)           (-inf if T_s is empty)
 *     out_partial = sum_{t in T_s} exp(s_t - lse) * K_t[0:512]   (0 if empty)
 * A NaN in a cache row makes the query rows that see it NaN; with causal, one
 * among the step's own tokens reaches the outputs of the rows before it too
 * (0 x NaN).
 * shard_id = MLA_ALL_SHARDS computes all N shards (out_partial holds N
 * slices, shard-major); shard_id in [0, N) computes that shard only
 * (n_out = 1), which is the per-GPU call of a multi-GPU deployment.
 *
 * Arguments: q, block_table, seq_lens, out_partial, lse_partial, workspace:
 * device pointers, layouts above.  max_pages_per_req: row stride of
 * block_table; it must cover the pages of every request (ceil(L_b / 64), or
 * ceil(n_s / 64) for a local layout holding n_s of the request's positions;
 * only those entries are read).  num_shards: 1..8.  workspace_bytes must be at
 * least mla_workspace_size(shape, num_shards, shard_id).
 *
 * Errors: MLA_ERR_INVALID / MLA_ERR_UNSUPPORTED / MLA_ERR_WORKSPACE before
 * any launch; MLA_ERR_CUDA if a launch fails.  Device-side problems (a
 * block-table entry out of range, which then reads as zeros; a wait that
 * timed out) are recorded in the workspace and read with
 * mla_get_device_error.
 */
mla_status mla_decode_partial(const void* q, const mla_kv_pages* kv, const int32_t* block_table,
                              int max_pages_per_req, const int32_t* seq_lens,
                              const mla_shape* shape, int shard_id, int num_shards,
                              mla_layout layout, float* out_partial, float* lse_partial,
                              void* workspace, size_t workspace_bytes, void* stream);

/*
 * The per-rank call of a multi-GPU DCP step with the exchanges' own layouts
 * ("Decode Context Parallelism", section 4.1: AllGather Q -> Compute -> a
 * combine of the partials; "Kimi K3 Performance Optimizations in vLLM",
 * section "Decode context parallelism": the partial outputs and LSEs travel
 * by an all-to-all).  Computes what mla_decode_partial computes for shard
 * `rank` of `num_ranks` (shard_id = rank, num_shards = num_ranks) with no copy
 * around it:
 *   q_gathered: bf16 [num_ranks, batch_total, q_len, H/num_ranks, 576], the
 *     all-gather of every rank's query heads as it lands (rank k's block
 *     holds heads k*H/num_ranks ..); this call computes requests
 *     batch_first .. batch_first + shape->batch - 1 of it.
 *   block_table, seq_lens (and shape->q_lens): those requests' rows.
 *   out_send: fp32 [num_ranks, shape->batch, q_len, H/num_ranks, 512];
 *   lse_send: fp32 [num_ranks, shape->batch, q_len, H/num_ranks]: slice k
 *     holds this shard's partial of heads k*H/num_ranks .., i.e. the send
 *     buffers of an all-to-all after which rank k holds every shard's
 *     partial of its own heads, shard-major, as mla_shard_combine takes
 *     them.
 * layout: MLA_LAYOUT_INTERLEAVED_LOCAL or MLA_LAYOUT_CONTIGUOUS_LOCAL (the
 * rank's own slice of the cache; else MLA_ERR_INVALID).  H must be a multiple
 * of num_ranks with H/num_ranks a multiple of 8 that divides 64 or is a
 * multiple of 64 (else MLA_ERR_UNSUPPORTED).  Other
 * arguments, the workspace (mla_workspace_size(shape, num_ranks, rank)) and
 * errors as for mla_decode_partial.
 */
mla_status mla_decode_partial_dcp(const void* q_gathered, int batch_total, int batch_first,
                                  const mla_kv_pages* kv, const int32_t* block_table,
                                  int max_pages_per_req, const int32_t* seq_lens,
                                  const mla_shape* shape, int rank, int num_ranks,
                                  mla_layout layout, float* out_send, float* lse_send,
                                  void* workspace, size_t workspace_bytes, void* stream);

/*
 * mla_decode_partial without a workspace argument, for callers that cannot
 * allocate device memory (for example code running while a serving engine's
 * pool already owns the whole GPU, allocator or out-of-memory callbacks, or
 * loops where an allocation is not allowed).  The pages this library follows
 * have no counterpart of this call; it exists only for such callers.
 *
 * The work list and split partial results live in a fixed scratch buffer
 * that the library keeps in device memory: about 40 MiB on every GPU that
 * loads the library, held until the process exits.  Shapes whose workspace
 * (mla_workspace_size) would exceed it, i.e. more than 8192 work units
 * (batch x computed shards x ceil(q_len * num_heads / 64)) or a GPU with
 * more than 160 SMs, return MLA_ERR_UNSUPPORTED before any launch.
 * Arguments, layouts, results and host-side errors are those of
 * mla_decode_partial.
 *
 * The first call in a CUDA context (normally: on a device) looks up the
 * scratch's device address (cudaGetSymbolAddress) and keeps it for that
 * context; make that first call before any stream capture.  All calls on a
 * device share the one scratch buffer, so calls whose kernels overlap on the
 * GPU (different streams, or different host threads) race: order them on
 * one stream.  Nothing needs clearing between calls; each call rebuilds what
 * it reads.  Device-side errors (a bad block-table page, a wait that timed
 * out) are kept in the scratch's error word: read them with
 * mla_get_device_error_noalloc.
 */
mla_status mla_decode_partial_noalloc(const void* q, const mla_kv_pages* kv,
                                      const int32_t* block_table, int max_pages_per_req,
                                      const int32_t* seq_lens, const mla_shape* shape,
                                      int shard_id, int num_shards, mla_layout layout,
                                      float* out_partial, float* lse_partial, void* stream);

/*
 * The device error word of mla_decode_partial_noalloc's scratch on the
 * current device: synchronises `stream`, reads and clears it, with the
 * results of mla_get_device_error.  Like the entry point it serves, this has
 * no counterpart on the pages; it lets callers that cannot allocate see a
 * bad block-table page or a timed-out wait.  It reads the state left by the
 * last mla_decode_partial_noalloc on the device, whatever its stream.
 */
mla_status mla_get_device_error_noalloc(void* stream);

/*
 * LSE combine of N shard partials ("Decode Context Parallelism", section 4.1:
 * partial outputs reweighted by their LSE and summed into the true output):
 *     M = max_s lse_s,  w_s = exp(lse_s - M),  lse_out = M + ln sum_s w_s
 *     o = sum_s w_s out_s / sum_s w_s                  (fp32)
 *     out = bf16(o)                                    if w_uv == NULL
 *     out = bf16(o . w_uv[h])  ([B,q_len,H,128])       otherwise (the fused
 *           v-projection of "Kimi K3 in vLLM ...", section 1)
 * partials / lses: as written by mla_decode_partial with MLA_ALL_SHARDS (or
 * the N per-shard slices stacked shard-major).  lse_out may be NULL.
 * A row whose shards are all empty gives out = 0 and lse_out = -inf.
 */
mla_status mla_shard_combine(const float* partials, const float* lses, int num_shards,
                             const mla_shape* shape, const void* w_uv, void* out, float* lse_out,
                             void* stream);

/*
 * One whole decode step on one GPU: every shard's partial attention
 * (mla_decode_partial with MLA_ALL_SHARDS) and their LSE combine
 * (mla_shard_combine, optionally fused with W_UV) in one call, with the shard
 * partials kept in the workspace instead of caller buffers.  The N shards are
 * logical partitions of the cache ("Decode Context Parallelism", section 4.1:
 * Compute, then the LSE reweighting of the partials into the true output).
 * A shard's unit that the work split divides between several CTAs leaves one
 * partial per CTA; these pieces are merged together with the other shards'
 * partials in the combine itself (the LSE merge is associative), so no merged
 * per-shard partial is written.  With w_uv and B * q_len >= 64 query rows per
 * head, the combine writes the output o in bf16 into the workspace and the
 * W_UV projection runs as one tensor-core GEMM per head (o rounded to bf16
 * before the product, as when projecting the unfused bf16 output); with
 * fewer rows the combine projects on the fly.
 *
 * Arguments as for mla_decode_partial and mla_shard_combine; layout must be
 * MLA_LAYOUT_INTERLEAVED or MLA_LAYOUT_CONTIGUOUS.  out: bf16
 * [B, q_len, H, 512], or [B, q_len, H, 128] with w_uv; lse_out: fp32
 * [B, q_len, H] or NULL.  workspace_bytes must be at least
 * mla_decode_step_workspace_size(shape, num_shards).  Device-side errors are
 * read with mla_get_device_error(workspace, stream).
 */
size_t mla_decode_step_workspace_size(const mla_shape* shape, int num_shards);
mla_status mla_decode_step(const void* q, const mla_kv_pages* kv, const int32_t* block_table,
                           int max_pages_per_req, const int32_t* seq_lens, const mla_shape* shape,
                           int num_shards, mla_layout layout, const void* w_uv, void* out,
                           float* lse_out, void* workspace, size_t workspace_bytes,
                           void* stream);

/*
 * Synchronises `stream`, reads and clears the device error word kept in
 * `workspace` by the last mla_decode_partial on it.  Returns MLA_OK,
 * MLA_ERR_TIMEOUT, MLA_ERR_DEVICE_BOUNDS, MLA_ERR_RANGE or MLA_ERR_INVALID (a
 * q_lens entry out of range), in that order of precedence when several
 * occurred, or MLA_ERR_CUDA.
 */
mla_status mla_get_device_error(void* workspace, void* stream);

/*
 * Testing and diagnostic aid (not part of the method): sets the time limit,
 * in nanoseconds, of every device-side wait of the partial-attention kernels
 * launched from now on (process-wide, any thread).  A wait that runs out
 * makes its kernel stop early, with MLA_ERR_TIMEOUT in the error word and
 * its outputs undefined; the kernel still lets its own copies and tensor-core
 * operations finish and releases its tensor memory, so later calls work
 * normally.  0 restores the default of 2 s.  Always MLA_OK.
 */
mla_status mla_set_wait_budget_ns(unsigned long long ns);

/*
 * Testing aid (not part of the method): while `on` is non-zero, the
 * partial-attention kernels of mla_decode_partial (and those of
 * mla_prefix_partial and mla_attention_weights) launched from now on never
 * load the query rows of each CTA's first piece of work (process-wide).  The
 * waits for those rows cannot succeed, so each CTA stops once its wait
 * budget (mla_set_wait_budget_ns) runs out, and mla_get_device_error then
 * reads MLA_ERR_TIMEOUT; outputs are undefined.  This exercises the
 * time-out path without any fault.  0 turns it off.  Always MLA_OK.
 */
mla_status mla_set_withhold_query(int on);

/*
 * Profiling aid (not part of the method): while set, every later
 * mla_decode_partial call (both entry points, any thread) records
 * `before_partial` and `after_partial` -- two cudaEvent_t handles passed as
 * void*, owned by the caller -- on its stream immediately before and after
 * the launch of its partial-attention kernel, so that kernel's device time
 * can be read without the planning and merge kernels around it.  Pass two
 * NULLs to stop.  Exactly one NULL is MLA_ERR_INVALID.  The caller keeps the
 * events alive while they are set; the setting is process-wide.
 */
mla_status mla_set_profile_events(void* before_partial, void* after_partial);

/*
 * Grouped-query attention (GQA) with the same sequence sharding ("Decode
 * Context Parallelism", section 5.4, the GQA backend): the cache stores
 * num_kv_heads KV heads of width head_dim in separate K and V caches, and
 * query head h attends with KV head h / (num_heads / num_kv_heads) (each KV
 * head broadcast over its group of consecutive query heads).
 *
 *   q            bf16  [B, q_len, H, D]
 *   k, v         bf16  [num_pages, 64, Hkv, D]   (token t of request b at
 *                                                 page block_table[b][t / 64],
 *                                                 row t % 64)
 *   out_partial  fp32  [n_out, B, q_len, H, D]
 *   lse_partial  fp32  [n_out, B, q_len, H]
 *   out          bf16  [B, q_len, H, D]
 *
 * This build supports head_dim = 128 and groups H / Hkv that are powers of
 * two up to 64; layouts INTERLEAVED and CONTIGUOUS.  Everything else matches
 * the MLA calls: logits scaled by softmax_scale (1/sqrt(D) for the workloads
 * here), causal verify steps, shard_id / MLA_ALL_SHARDS, workspace, error
 * reporting through mla_get_device_error, asynchronous on `stream`.
 */
typedef struct gqa_shape {
  int batch;            /* B >= 1 */
  int q_len;            /* query tokens per request >= 1 */
  int num_heads;        /* H */
  int num_kv_heads;     /* Hkv, divides H */
  int head_dim;         /* D: 128 */
  int causal;           /* 0 or 1 */
  float softmax_scale;
} gqa_shape;

typedef struct gqa_kv_pages {
  const void* k;        /* bf16 [num_pages, page_size, Hkv, D] */
  const void* v;        /* bf16 [num_pages, page_size, Hkv, D] */
  int num_pages;        /* >= 1 */
  int page_size;        /* must be 64 */
} gqa_kv_pages;

/* Workspace bytes gqa_decode_partial needs (0 for invalid or unsupported shapes). */
size_t gqa_workspace_size(const gqa_shape* shape, int num_shards, int shard_id);

/* Per-shard partial GQA attention: for every request b, query row (i, h) and
 * computed shard s, over the shard's visible tokens T_s:
 *   s_t = softmax_scale * q[b,i,h,:] . K_t[kh,:],  kh = h / (H / Hkv)
 *   lse_partial = ln sum exp(s_t)  (-inf if empty);
 *   out_partial = sum exp(s_t - lse) V_t[kh,:]  (0 if empty).
 * A NaN key makes the rows that see it NaN, a NaN value one dim; with causal, a
 * NaN value among the step's own tokens reaches the rows before it too (0 x NaN;
 * not so in gqa_decode_partial_fp8).  There is no q_lens here and no *_LOCAL layout:
 * of what gqa_cache_append writes to bf16 caches this call attends to whole
 * requests with q_len new tokens each. */
mla_status gqa_decode_partial(const void* q, const gqa_kv_pages* kv, const int32_t* block_table,
                              int max_pages_per_req, const int32_t* seq_lens,
                              const gqa_shape* shape, int shard_id, int num_shards,
                              mla_layout layout, float* out_partial, float* lse_partial,
                              void* workspace, size_t workspace_bytes, void* stream);

/* LSE combine of N GQA shard partials (head_dim wide) into bf16 out
 * [B, q_len, H, D] and lse_out (may be NULL).  A shard with lse -inf counts for
 * nothing; one with lse NaN makes the row NaN. */
mla_status gqa_shard_combine(const float* partials, const float* lses, int num_shards,
                             const gqa_shape* shape, void* out, float* lse_out, void* stream);

/*
 * Rotary positions.  Pair i < rot_dim / 2 of a head turns by position *
 * inv_freq[i] radians:
 *     y_a = f (x_a cos - x_b sin),  y_b = f (x_a sin + x_b cos),
 *     f = attention_factor,
 * with (a, b) = first_dim + (2i, 2i + 1) if interleaved, else first_dim +
 * (i, i + rot_dim / 2).  Dims outside [first_dim, first_dim + rot_dim) pass
 * through.  Computed in fp32 and rounded once; the angle is reduced modulo a
 * turn in 64-bit integers, so far positions lose no accuracy.  Scalings for
 * long contexts enter through inv_freq and attention_factor.
 */
typedef struct mla_rope {
  const double* inv_freq;  /* device, [rot_dim / 2], radians per token, finite; 8-byte aligned */
  int rot_dim;             /* multiple of 16, >= 16, at most the head's width */
  int first_dim;           /* multiple of 8; first_dim + rot_dim <= the head's width */
  int interleaved;         /* 0 or 1 */
  float attention_factor;  /* finite */
} mla_rope;

/* The new tokens of a step: request b appends its last n_b = q_lens[b] (or
 * q_len) tokens to a context that then has seq_lens[b] tokens, i.e. token i
 * stands at position seq_lens[b] - n_b + i -- the same seq_lens and q_lens the
 * attention calls of the step take.  Rows i >= n_b are padding: nothing is
 * read from or written for them. */
typedef struct mla_tokens {
  int batch;                    /* B >= 1 */
  int q_len;                    /* >= 1 (the padded count, see q_lens) */
  const int32_t* seq_lens;      /* device [B] */
  const int32_t* q_lens;        /* device [B] in [1, q_len], or NULL (all q_len); clamped */
  const int32_t* positions;     /* device [B, q_len]: rotary positions (any int32), or NULL
                                   (where the token stands); cache slots do not change */
} mla_tokens;

/*
 * Rotates query heads: x bf16, token (b, i)'s heads [num_heads, head_dim]
 * contiguous at x + (b * q_len + i) * x_stride elements; out likewise with
 * out_stride.  out == x with equal strides rotates in place (and moves only
 * the rotated dims); otherwise the two must not overlap.  head_dim a multiple
 * of 8, at most 1024; strides multiples of 8, at least num_heads * head_dim.
 * tokens->seq_lens may be NULL if positions is given.  Padding rows of out
 * are left as they were.
 */
mla_status mla_rope_apply(const void* x, long long x_stride, void* out, long long out_stride,
                          const mla_tokens* tokens, int num_heads, int head_dim,
                          const mla_rope* rope, void* stream);

/*
 * Appends a step's latent rows to the paged latent cache, and rotates the
 * step's queries in the same launch.
 *   latent  bf16, row (b, i) of 576 values at latent + (b * q_len + i) *
 *           latent_stride; rotated by `rope` (in a latent row the rope dims
 *           are 512..575: first_dim 512), or stored as it is if rope is NULL
 *   kv      the cache; its data (and scale) are written.  bf16: values rounded
 *           once.  e4m3: each row gets as its scale the smallest power of two
 *           s >= 2^-60 with max|x| <= 448 s over its finite values, and the
 *           codes of x / s; an infinite or NaN value is stored as NaN.
 *   q, q_out bf16 [.., num_heads, 576] rows as in mla_rope_apply (rope must be
 *           given then), or q NULL
 * Whole-request caches: num_shards 1, shard_id 0.  num_shards N > 1: the cache
 * is shard shard_id's MLA_LAYOUT_INTERLEAVED_LOCAL slice; tokens of other
 * shards are skipped.  (CONTIGUOUS_LOCAL slices move as a context grows and
 * are not appended to.)  Only the new tokens' rows change.  The pages they
 * fall on must belong to one request each.
 *
 * workspace: 256 bytes of device memory, zeroed once before its first use:
 * MLA_ERR_DEVICE_BOUNDS (a page outside [0, num_pages): its rows are not
 * written) and MLA_ERR_INVALID (a q_lens entry outside [1, q_len], or more new
 * tokens than seq_lens) stay there until mla_get_device_error reads them.
 */
mla_status mla_cache_append(const void* latent, long long latent_stride, const mla_kv_pages* kv,
                            const int32_t* block_table, int max_pages_per_req,
                            const mla_tokens* tokens, const mla_rope* rope, const void* q,
                            long long q_stride, void* q_out, long long q_out_stride,
                            int num_heads, int shard_id, int num_shards, void* workspace,
                            size_t workspace_bytes, void* stream);

/*
 * A GQA cache held in e4m3 with a scale for each block of tokens and KV head
 * (or, for gqa_cache_append, in bf16 with null scales):
 *   k, v              e4m3 (or bf16) [num_pages, 64, Hkv, 128]
 *   k_scale, v_scale  fp32 [num_pages, 64 / block, Hkv]: value of row r, head h
 *                     = code * scale[page][r / block][h]
 * Scales written by gqa_cache_append are powers of two between 2^-60 and
 * 2^120.  The attention takes any finite K scale, and V scales as
 * gqa_decode_partial_fp8 says.
 */
typedef struct gqa_block_pages {
  void* k;
  void* v;
  float* k_scale;
  float* v_scale;
  mla_kv_dtype dtype;
  int block;            /* tokens per scale: 1, 2, 4, .. 64 (ignored for bf16) */
  int num_pages;        /* >= 1 */
  int page_size;        /* must be 64 */
  int num_kv_heads;
} gqa_block_pages;

/*
 * Appends a step's K and V heads to the paged GQA cache, and rotates the
 * step's queries in the same launch.  k, v: bf16, token (b, i)'s heads
 * [Hkv, 128] at k + (b * q_len + i) * k_stride; k is rotated by `rope` (NULL:
 * stored as it is), v never.  Sharding, q, workspace and errors as for
 * mla_cache_append.
 *
 * e4m3: for each block of `block` token slots, KV head and cache, with a the
 * largest finite |x| of the new tokens in it and s_new the smallest power of
 * two >= 2^-60 with a <= 448 s_new: a block without earlier tokens (slots
 * before the request's first new token) takes s = s_new; otherwise s = the
 * block's scale s_old if |s_old| >= s_new (or s_old is NaN), else s = s_new
 * and the earlier tokens' codes are rounded again, to code * s_old / s.  With
 * power-of-two scales that is exact except for codes that become subnormal.
 * New codes are x / s.  Slots behind the context are left as they were.
 */
mla_status gqa_cache_append(const void* k, long long k_stride, const void* v, long long v_stride,
                            const gqa_block_pages* cache, const int32_t* block_table,
                            int max_pages_per_req, const mla_tokens* tokens, const mla_rope* rope,
                            const void* q, long long q_stride, void* q_out,
                            long long q_out_stride, int num_heads, int shard_id, int num_shards,
                            void* workspace, size_t workspace_bytes, void* stream);

/* Workspace bytes gqa_decode_partial_fp8 needs (0 for invalid or unsupported shapes). */
size_t gqa_fp8_workspace_size(const gqa_shape* shape, int num_shards, int shard_id);

/*
 * gqa_decode_partial over an e4m3 cache with block scales (cache->dtype
 * MLA_KV_FP8_E4M3).  Differences from gqa_decode_partial: any group H / Hkv up
 * to 64; all four layouts (the *_LOCAL ones with one shard_id); q_lens
 * (device [B] or NULL) as in mla_shape: rows i >= q_lens[b] give o = 0, lse =
 * -inf, and with causal query i sees t <= L_b - q_lens[b] + i.  With
 * INTERLEAVED num_shards must divide 64.  An inf or NaN query value of a row
 * that attends is reported as MLA_ERR_RANGE; a block-table entry out of range
 * reads as zeros, and a context longer than its block-table row is cut at the
 * row's end, both reported as MLA_ERR_DEVICE_BOUNDS.  Shapes whose work could
 * pass 2^31 tiles (units times pages per row) are MLA_ERR_UNSUPPORTED.
 *
 * Made for decode and verify steps.  A prompt chunk's many queries are answered
 * rightly, but K and V are read and multiplied once for every 32 rows of a KV
 * head, those behind the rows' last visible token too.
 *
 * Accuracy.  A query value is held to 2^-18 of its row's largest or better.  A
 * token's weight p_t carries its V scale sv_t, and one reference serves a row:
 * p_t sv_t is off by up to 2^-11 of itself and 2^-27 max_u (p_u |sv_u|), the
 * row's largest.  So where one seen block's V scale is S times another's, the
 * other's weights have log2 S fewer of these 27 bits, whatever the wide block's
 * codes are: at S = 2^16 a token with the same p is still held to 2^-10, at
 * S = 2^28 it is gone.  (Scales follow the largest value of their block, so a
 * wide one goes with large outputs, but a dim that has zeros there has them
 * too.)  The lse does not depend on this while the row's V scales lie within
 * 2^100 of one another; one below 2^-60 in magnitude counts as 2^-60 in this,
 * and weighs its block with that much less precision (0 is exact).  A finite V
 * scale above 2^120 of a token in the context is reported as MLA_ERR_RANGE.
 *
 * The workspace may hold anything before a call, and serves one call at a
 * time; mla_get_device_error reads the last call's errors from it.
 */
mla_status gqa_decode_partial_fp8(const void* q, const gqa_block_pages* cache,
                                  const int32_t* block_table, int max_pages_per_req,
                                  const int32_t* seq_lens, const int32_t* q_lens,
                                  const gqa_shape* shape, int shard_id, int num_shards,
                                  mla_layout layout, float* out_partial, float* lse_partial,
                                  void* workspace, size_t workspace_bytes, void* stream);

/* Workspace bytes mla_prefix_partial needs on the current device (0 for invalid
 * shapes). */
size_t mla_prefix_workspace_size(const mla_shape* shape, int num_groups, int max_pages_per_req,
                                 mla_kv_dtype dtype);

/*
 * Partial attention of a batch whose requests share prefixes, each prefix read
 * and multiplied once for all the query rows that share it.  Group g is the
 * consecutive requests [group_starts[g], group_starts[g + 1]); the first
 * prefix_lens[g] tokens of their contexts are the same, and their block-table
 * rows name the same pages for them.  Two partials, as of two shards:
 *   out_partial fp32 [2, B, q_len, H, 512], lse_partial fp32 [2, B, q_len, H]
 * which mla_shard_combine (num_shards 2, with or without w_uv) turns into the
 * attention of every request over its whole context.  Slice 0 is over shared
 * pages, slice 1 over the rest.  What falls into which is the library's choice,
 * made on the device from the lengths: whole pages of a prefix that every row of
 * the group sees are shared where that takes less time than attending them per
 * request (mla_set_prefix_sharing); prefix_lens below a page, 0 or negative share
 * nothing.  The alternative is mla_decode_step, which takes whole contexts and
 * is a launch or two shorter: it is the faster call for few requests, short
 * prefixes and verify steps behind some thousand shared tokens (two requests
 * behind 1024 tokens 35 us, 36 here; 16 of 5 tokens behind three prefixes of
 * 2000 to 16000 120, 122 here; 32 behind 114k 651, 444 here).
 *
 *   block_table, seq_lens, shape (q_lens, causal)  as in mla_decode_partial:
 *                 whole contexts, the prefix among them
 *   group_starts  device int32 [num_groups + 1]: from 0 to B, ascending (empty
 *                 groups allowed); num_groups 1 .. B
 *   prefix_lens   device int32 [num_groups]
 * Whole-request caches; a DCP rank passes its slice's own lengths, with causal
 * 0 (one query token), and the combine takes two partials from each rank.
 *
 * workspace: mla_prefix_workspace_size bytes, which may hold anything and serve
 * one call at a time.  mla_get_device_error reads the last call's errors: as
 * for mla_decode_partial, and MLA_ERR_INVALID for group_starts that are not
 * such ranges (no prefix is shared then, the result is right all the same),
 * MLA_ERR_DEVICE_BOUNDS for a context longer than its block-table row (cut at
 * the row's end).
 */
mla_status mla_prefix_partial(const void* q, const mla_kv_pages* kv, const int32_t* block_table,
                              int max_pages_per_req, const int32_t* seq_lens,
                              const mla_shape* shape, const int32_t* group_starts,
                              const int32_t* prefix_lens, int num_groups, float* out_partial,
                              float* lse_partial, void* workspace, size_t workspace_bytes,
                              void* stream);

/*
 * Testing aid (not part of the method): while `always` is non-zero,
 * mla_prefix_partial calls made from now on share all the pages that can be
 * shared, also where attending them per request is faster (process-wide).  0
 * turns it off.  Always MLA_OK.
 */
mla_status mla_set_prefix_sharing(int always);

/* Workspace bytes mla_attention_weights needs (0 for invalid shapes). */
size_t mla_attention_weights_workspace_size(const mla_shape* shape, mla_kv_dtype dtype);

/*
 * The attention weight that a step gives to every cached token, summed over
 * its query rows and added to what earlier steps gave -- what mla_cache_evict
 * selects by.  For request b with n_b = q_lens[b] (or q_len) query tokens:
 *   w[t] = sum over i < n_b, h, with t visible to i, of
 *          exp(softmax_scale * q[b,i,h,:] . K_t - lse[b,i,h])
 *   out[b,t] = w[t] + (before[b,t] if before != NULL and t < L_b - n_b, else 0)
 * for t < L_b: the last n_b tokens, which the step appended, start from 0.
 * Entries from L_b on are left as they were.  Visibility is that of the
 * attention calls (causal: t <= L_b - n_b + i; else every t < L_b).
 *
 *   lse     fp32 [B, q_len, H]: the whole contexts' log-sum-exps, the lse_out of
 *           mla_shard_combine or mla_decode_step for the same step; a row at
 *           -inf gives nothing
 *   before  fp32 [B, width], before_stride floats between requests, or NULL
 *   out     fp32 [B, width], out_stride floats between requests; before itself
 *           (with its stride), or apart from it
 * Whole-request caches of either type, not a rank's slice (whose last n_b
 * tokens are not the step's new ones), every num_heads that is a multiple of
 * 16; width at least every L_b, at most 2^30.  Sums are fp32 in a fixed order.
 * A NaN in a cache row makes that token's weight NaN, a NaN lse every weight
 * of its request.  With an e4m3 cache the query is held as in
 * mla_decode_partial, and an inf or NaN query value of a row i < n_b is
 * reported as MLA_ERR_RANGE.
 *
 * workspace: mla_attention_weights_workspace_size bytes, which may hold
 * anything and serve one call at a time; mla_get_device_error reads the last
 * call's errors: MLA_ERR_DEVICE_BOUNDS (a page out of range, its rows count as
 * zeros), MLA_ERR_INVALID (a seq_lens entry below 0, above width or beyond the
 * block table's row, or a q_lens entry outside [1, q_len], clamped),
 * MLA_ERR_RANGE, MLA_ERR_TIMEOUT.
 */
mla_status mla_attention_weights(const void* q, const mla_kv_pages* kv, const int32_t* block_table,
                                 int max_pages_per_req, const int32_t* seq_lens,
                                 const mla_shape* shape, const float* lse, const float* before,
                                 long long before_stride, float* out, long long out_stride,
                                 int width, void* workspace, size_t workspace_bytes, void* stream);

/*
 * Eviction from a paged latent cache by accumulated attention weight.  Request
 * b keeps n_b = min(seq_lens[b], keep[b]) of its tokens:
 *   - the first f_b = min(keep_first[b], n_b) (keep_first NULL: none): attention
 *     sinks, or a prefix that it shares with other requests;
 *   - the newest r_b = min(recent, n_b - f_b);
 *   - of the others the n_b - f_b - r_b with the largest weights; equal ones
 *     from the lowest position on.  NaN counts as larger than everything, the
 *     two zeros as equal.
 * They move in order: token kept[b][j] becomes row j of the new context, whose
 * pages are new_block_table[b].  Rotary positions are in the rows and do not
 * change; later appends give theirs in mla_tokens.positions.
 *
 *   kv               the cache, with its scales (both written; the new pages
 *                    are pages of the same pool)
 *   weights          fp32 [B, weights_width], weights_stride floats between
 *                    requests (weights_width at most 2^30, at least seq_lens)
 *   keep             int32 [B], 0 .. max_keep; keep_first int32 [B] or NULL
 *   new_block_table  int32 [B, new_max_pages], new_max_pages >= ceil(max_keep / 64);
 *                    entries behind a request's new pages are not read
 *   new_seq_lens     int32 [B]: n_b
 *   kept             int32 [B, max_keep]: positions in the old context, ascending;
 *                    -1 from n_b on (max_keep at most 2^30)
 *   weights_out      fp32 [B, max_keep] or NULL: the kept tokens' weights; entries
 *                    from n_b on are left as they were
 * The three outputs share memory with each other and with the other arrays
 * nowhere (MLA_ERR_INVALID).
 * The new pages are pages that no context uses, each in one place of
 * new_block_table, but for leading ones: where new_block_table[b][i] is
 * block_table[b][i] and the rows of page i all keep their place (a kept
 * prefix), the page is left as it is and may be shared.  The same page with
 * rows that would move is reported as MLA_ERR_INVALID and not written.  Rows
 * behind a new context's end are left as they were, and so are the old pages.
 * Where a new context ends inside such a page, the request's next append writes
 * behind its last row there: a shared page that can be the last one needs a page
 * of its own in new_block_table, into which its rows are then copied.
 *
 * The selection runs on 1 to 16 SMs a request, chosen by weights_width: rows
 * much wider than the contexts cost time (16 contexts of 8000 tokens 14 us in
 * rows of 8192, 44 in rows above 262144); pass the part that contexts reach.
 *
 * workspace: 256 bytes of device memory, zeroed once before its first use:
 * MLA_ERR_DEVICE_BOUNDS (a page outside [0, num_pages): its rows are not moved)
 * and MLA_ERR_INVALID (a seq_lens entry below 0, above weights_width or beyond
 * the block table's row, a keep entry outside [0, max_keep], all clamped; a
 * page that would be overwritten) stay there until mla_get_device_error reads
 * them.
 */
mla_status mla_cache_evict(const mla_kv_pages* kv, const int32_t* block_table,
                           int max_pages_per_req, const int32_t* seq_lens, int batch,
                           const float* weights, long long weights_stride, int weights_width,
                           const int32_t* keep, const int32_t* keep_first, int recent,
                           const int32_t* new_block_table, int new_max_pages,
                           int32_t* new_seq_lens, int32_t* kept, int max_keep, float* weights_out,
                           void* workspace, size_t workspace_bytes, void* stream);

/* Static description of a status code. */
const char* mla_status_string(mla_status status);

/* Library version: major * 10000 + minor * 100 + patch.  0.2.0 added
 * mla_shape.q_lens, the *_LOCAL layouts and MLA_ERR_RANGE. */
int mla_version(void);

#ifdef __cplusplus
}
#endif

#endif /* MLA_DCP_H_ */
