// Internal interfaces of the serving operators (paged key/value cache, paged
// attention, draft verification): launch arguments shared by serve_api.cpp and
// the kernels.  Not installed; not part of the ABI.
#pragma once

#include <stddef.h>
#include <stdint.h>

#include <hip/hip_runtime_api.h>

#include "../../include/spear_serve.h"
#include "internal.h"

namespace spear {

struct KvShape {
  int32_t dtype, num_pages, heads, dim, page_log2;
};

struct KvAppendArgs {
  KvShape kv;
  int32_t tokens;
  const void *k, *v;
  int64_t k_ts, k_hs, v_ts, v_hs;   // strides in elements
  const int64_t* slots;
  void *k_cache, *v_cache;
  float *k_scale, *v_scale;
};
hipError_t launch_kv_append(const KvAppendArgs& a, void* stream);

// Entry of a sequence's block table row for output row `row` of a sequence whose
// first row is `first`: within the table whatever the offsets hold, -1 for a row
// before the first (offsets that do not rise give such rows).
constexpr int64_t table_entry(int64_t row, int64_t first, int page_log2, int64_t table_stride) {
  if (row < first) return -1;
  const int64_t entry = (row - first) >> page_log2;
  return entry < table_stride ? entry : table_stride - 1;
}

struct KvGatherArgs {
  KvShape kv;
  int32_t batch, rows;
  const int32_t* table;
  int64_t table_stride;
  const int32_t* cu;
  const void *k_cache, *v_cache;
  const float *k_scale, *v_scale;
  void *k_out, *v_out;
};
hipError_t launch_kv_gather(const KvGatherArgs& a, void* stream);

// Whether an attention kernel's 32-bit counts hold for any offsets at all: with
// ones that do not rise, each of the sequences can have all rows.  `extra` steps
// count for each row tile beside those of its keys; `most` is the count's bound.
constexpr bool counts_hold(int64_t batch, int64_t rows, int64_t tile_rows, int64_t max_kv, int64_t step_keys,
                           int64_t extra, int64_t heads, int64_t most) {
  const double tiles = (double)((rows + tile_rows - 1) / tile_rows), steps = (double)((max_kv + step_keys - 1) / step_keys);
  return (double)batch * tiles * (steps + (double)extra) * (double)heads <= (double)most;
}

// Launch shape of an attention call.
struct AttnPlan {
  bool tiles;         // sequences of many rows go to the kernel of 128-row tiles ..
  bool both;          // .. and those of at most few_rows to the other one
  int row_tiles;      // 16-row operands a workgroup of the latter holds (1 or 2)
  int few_rows;       // 16 * row_tiles
  int grid, tile_grid;   // workgroups of the latter and of the former
  int cus;
  bool fits;          // the work of rising offsets can be counted in 32 bits
  bool check_few, check_tiles;   // that of any others need not: the kernel looks whether they rise
  size_t part, part_bytes;            // partial results in the workspace
  size_t tile_part, tile_part_bytes;
  size_t bytes;       // workspace
};
AttnPlan attn_plan(const spear_attention_desc_t& d, int cus);

struct AttnArgs {
  KvShape kv;
  int32_t batch, total_q, q_heads, group, max_kv;
  float scale;
  const void* q;
  int64_t q_ts, q_hs;
  const int32_t *cu_q, *kv_lens, *table;
  int64_t table_stride;
  const void *k_cache, *v_cache;
  const float *k_scale, *v_scale;
  void* out;
  void* workspace;      // its header's first counters are zero before and after
};
hipError_t launch_attention(const AttnArgs& a, const AttnPlan& p, void* stream);

// Workgroups that share one sequence's vocabulary in a verification call.
int verify_splits(const spear_verify_desc_t& d, int cus);
struct VerifyArgs {
  int32_t batch, drafts, vocab, splits;
  const float *target, *draft;
  int64_t target_bs, target_rs, draft_bs, draft_rs;
  const int32_t* drafted;
  const float *u, *noise;
  const int32_t* num_drafts;
  int32_t *accepted, *tokens;
  uint32_t* counters;   // [batch], zero before and after
  uint64_t* part;       // [batch][splits]
};
hipError_t launch_verify(const VerifyArgs& a, void* stream);

}  // namespace spear
