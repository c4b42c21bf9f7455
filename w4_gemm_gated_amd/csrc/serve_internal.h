// Internal interfaces of the serving operators (paged key/value cache, paged
// attention, draft verification, and what a step does around them): launch
// arguments shared by serve_api.cpp, step_api.cpp and the kernels.  Not
// installed; not part of the ABI.
#pragma once

#include <stddef.h>
#include <stdint.h>

#include <hip/hip_runtime_api.h>

#include <atomic>

#include "../../include/spear_serve.h"
#include "internal.h"

namespace spear {

inline bool aligned(const void* p, uintptr_t a) { return ((uintptr_t)p % a) == 0; }
inline spear_status_t hip_status(hipError_t e) { return e == hipSuccess ? SPEAR_OK : SPEAR_ERR_HIP; }

// CUs to plan for: the caller's number, or the current device's (looked up once).
inline spear_status_t cus_of(int32_t asked, int* out) {
  constexpr int kMaxDevices = 64;
  static std::atomic<int> cache[kMaxDevices];
  if (asked < 0) return SPEAR_ERR_INVALID_ARGUMENT;
  if (asked > 0) {
    *out = asked < 4096 ? asked : 4096;
    return SPEAR_OK;
  }
  int dev = 0, cus = 0;
  if (hipGetDevice(&dev) != hipSuccess) return SPEAR_ERR_HIP;
  const bool kept = dev >= 0 && dev < kMaxDevices;
  if (kept && (cus = cache[dev].load(std::memory_order_relaxed)) > 0) {
    *out = cus;
    return SPEAR_OK;
  }
  if (hipDeviceGetAttribute(&cus, hipDeviceAttributeMultiprocessorCount, dev) != hipSuccess || cus <= 0)
    return SPEAR_ERR_HIP;
  if (kept) cache[dev].store(cus, std::memory_order_relaxed);
  *out = cus;
  return SPEAR_OK;
}

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

// A step's plan: workgroups of `threads` threads, each for that many rows.
struct KvPlanArgs {
  int32_t batch, rows, max_pages, page_log2, free_slots, threads;
  const int32_t *lens, *ask, *held;
  int32_t* table;
  int64_t table_stride;
  int32_t* free_pages;
  const int32_t* free_count;
  int32_t *cu_q, *kv_lens;
  int64_t* slots;
  int32_t *positions, *sequence, *held_out, *free_out;
  bool in_place;        // a state output is its input: the last workgroup writes them all
  uint32_t* counter;    // zero before and after
};
int kv_plan_threads(int batch);
hipError_t launch_kv_plan(const KvPlanArgs& a, void* stream);

// Adapters of many requests.
constexpr int kMaxAdapters = 4096;   // counted in LDS by the plan
constexpr int kAdapterTile = 64;     // rows of one adapter that a workgroup takes
constexpr int kAdapterRanks = 64;    // most ranks of the first product that one takes at once
constexpr int kAdapterColumns = 256; // columns of the output that one takes at once
struct AdapterPlanArgs {
  int32_t batch, adapters, rows, most_tiles;
  const int32_t *cu, *adapter;
  int32_t* plan;
};
hipError_t launch_adapter_plan(const AdapterPlanArgs& a, void* stream);
int64_t adapter_most_tiles(int64_t rows, int64_t batch, int64_t adapters);
size_t adapter_plan_size(int64_t rows, int64_t batch, int64_t adapters);

// A tile: rows [first, first + rows) of the plan's list belong to `adapter`.  Within the
// list and the adapters whatever the plan holds (one that was made for other sizes, or not
// yet).
struct AdapterTile {
  int32_t adapter, first, rows;
};
constexpr AdapterTile adapter_tile(int32_t adapter, int32_t first, int32_t rows, int32_t adapters, int32_t all_rows) {
  first = first < 0 ? 0 : first < all_rows ? first : all_rows - 1;
  const int32_t most = all_rows - first < kAdapterTile ? all_rows - first : kAdapterTile;
  return {adapter < 0 ? 0 : adapter < adapters ? adapter : adapters - 1, first, rows < 1 ? 1 : rows < most ? rows : most};
}

// Launch shape and workspace (offsets in bytes) of an adapter call.
struct AdapterShape {
  int tiles, rank_pad, slices, slice_k, groups, chunk_columns;     // groups: of ranks
  bool fused;           // both products in one launch
  size_t H, factor, part, bytes;
};
AdapterShape adapter_shape(const spear_adapter_desc_t& d, int cus);
struct AdapterArgs {
  int32_t rows, adapters, K, N, rank, rank_pad, most_tiles, slices, slice_k, groups, chunks, chunk_columns;
  bool fused;
  const void *X, *A, *B;
  const float* scale;      // [adapters], or null: 1
  const int32_t* plan;
  void* Y;
  int64_t x_stride, y_stride;
  bool y_vectors;          // Y's rows are 16-byte aligned
  uint32_t* counters;      // [tiles], zero before and after
  char* part;              // fp32 [tiles][slices][64][rank]
  void* H;                 // fp16 [tiles][64][2][rank_pad]
  float* factor;           // [tiles][64]
};
hipError_t launch_adapter(const AdapterArgs& a, void* stream);

// The draw of next tokens.
constexpr int kSampleLeast = 4096;      // tokens of the vocabulary that a workgroup takes, two or four times as many for bins
constexpr int kSampleShares = 512;      // most workgroups of a row's bins
constexpr int kSampleList = 4094;       // tokens of the bins that are cut, gathered for the row's end
constexpr int kSampleInfoBytes = 256;
struct ShareInfo {
  unsigned long long best;              // the largest (logit, token)
  unsigned long long number;            // a double: the place of its first bin
  unsigned long long mass;              // a double: of all its tokens
  unsigned long long used;              // tokens and bins written
};
struct PartInfo {
  unsigned long long best;              // the largest (score, token)
  double mass;                          // of what is kept
};
struct SampleShape {
  int share_tokens, shares;             // tokens of a workgroup of the bins, their workgroups of a row
  int parts, group;                     // workgroups of a row after that, rows of a launch
  size_t info, share, part, list, hist, list_noise, bytes;
};
SampleShape sample_shape(const spear_sample_desc_t& d);
struct SampleArgs {
  int32_t batch, vocab, share_tokens, shares, parts, num_rows;
  int32_t first;                        // the group's first draw: row `first` + b where no rows are given
  bool f16, only_first;                 // only_first: every row keeps its first token alone
  const void* logits;
  int64_t stride;
  const int32_t* rows;
  const float* noise;
  const float *temperature, *top_p, *min_p;
  const int32_t* top_k;
  float one_temperature, one_top_p, one_min_p;
  int32_t one_top_k;
  int32_t* tokens;
  float* probs;
  void* info;
  ShareInfo* share;                     // [batch][shares], as hist where there are several
  PartInfo* part;                       // [batch][parts], as list and list_noise where there are several
  unsigned long long *list, *hist;      // [batch][kSampleList], [batch][shares][bins]
  float* list_noise;                    // [batch][kSampleList]
};
hipError_t launch_sample(const SampleArgs& a, void* stream);

}  // namespace spear
