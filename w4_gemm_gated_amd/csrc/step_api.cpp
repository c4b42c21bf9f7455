// C ABI entry points of what a serving step does around the layers and the cache
// (declared in include/spear_serve.h): argument checks and launches.  Nothing here
// allocates device memory or synchronizes; every check runs before anything is
// enqueued.
#include <hip/hip_runtime_api.h>

#include "serve_internal.h"

using namespace spear;

namespace {

spear_status_t check_kv_plan(const spear_kv_plan_desc_t& d) {
  if (d.batch < 0 || d.rows < 0 || d.max_pages < 1 || d.page_size < 1 || d.free_slots < 0) return SPEAR_ERR_INVALID_SHAPE;
  if (d.page_size < 16 || d.page_size > 1024 || (d.page_size & (d.page_size - 1)) != 0) return SPEAR_ERR_UNSUPPORTED;
  // 32-bit positions and rows
  const int64_t most = (int64_t)1 << 30;
  if (d.batch > (1 << 20) || d.rows > most || (int64_t)d.max_pages * d.page_size > most) return SPEAR_ERR_UNSUPPORTED;
  return SPEAR_OK;
}

// (a call of one workgroup needs no counter)
size_t kv_plan_bytes(const spear_kv_plan_desc_t& d) { return d.rows > kv_plan_threads(d.batch) ? kSyncHeaderBytes : 0; }

spear_status_t check_workspace(const void* workspace, size_t have, size_t need) {
  if (need > 0 && !workspace) return SPEAR_ERR_NULL_POINTER;
  if (have < need) return SPEAR_ERR_WORKSPACE_TOO_SMALL;
  return workspace && !aligned(workspace, 16) ? SPEAR_ERR_MISALIGNED : SPEAR_OK;
}

spear_status_t check_batch(int32_t batch, int32_t adapters, int32_t rows) {
  if (batch < 0 || rows < 0 || adapters < 1) return SPEAR_ERR_INVALID_SHAPE;
  if (adapters > kMaxAdapters || batch > (1 << 20) || rows > (1 << 24)) return SPEAR_ERR_UNSUPPORTED;
  return SPEAR_OK;
}

spear_status_t check_adapter(const spear_adapter_desc_t& d) {
  const spear_status_t st = check_batch(d.batch, d.adapters, d.rows);
  if (st != SPEAR_OK) return st;
  if (d.K < 8 || d.K % 8 != 0 || d.N < 1 || d.rank < 8 || d.rank % 8 != 0) return SPEAR_ERR_INVALID_SHAPE;
  if (d.rank > SPEAR_MAX_RANK || d.K > (1 << 24) || d.N > (1 << 24)) return SPEAR_ERR_UNSUPPORTED;
  if (d.device_cus < 0) return SPEAR_ERR_INVALID_ARGUMENT;
  // (a launch holds fewer than 2^32 threads: 256 for every tile and 256 columns)
  if (adapter_most_tiles(d.rows, d.batch, d.adapters) * ceil_div(d.N, kAdapterColumns) >= (1 << 24))
    return SPEAR_ERR_UNSUPPORTED;
  return SPEAR_OK;
}

static_assert((1 << 22) / (4 * kSampleLeast) <= kSampleShares, "room for every share");
spear_status_t check_sample(const spear_sample_desc_t& d) {
  if (d.batch < 0 || d.vocab < 1 || d.num_rows < 0) return SPEAR_ERR_INVALID_SHAPE;
  if (d.dtype != SPEAR_LOGITS_FP16 && d.dtype != SPEAR_LOGITS_FP32) return SPEAR_ERR_INVALID_ARGUMENT;
  if (d.batch > (1 << 20) || d.vocab > (1 << 22)) return SPEAR_ERR_UNSUPPORTED;
  return SPEAR_OK;
}

}  // namespace

extern "C" {

spear_status_t spear_kv_plan_workspace_bytes(const spear_kv_plan_desc_t* desc, size_t* bytes) {
  if (!desc || !bytes) return SPEAR_ERR_NULL_POINTER;
  const spear_status_t st = check_kv_plan(*desc);
  if (st == SPEAR_OK) *bytes = kv_plan_bytes(*desc);
  return st;
}

spear_status_t spear_kv_plan(const spear_kv_plan_desc_t* desc, const int32_t* lens, const int32_t* new_tokens,
                             const int32_t* held, int32_t* block_table, int64_t table_stride, int32_t* free_pages,
                             const int32_t* free_count, int32_t* cu_q, int32_t* kv_lens, int64_t* slots,
                             int32_t* positions, int32_t* sequence, int32_t* held_out, int32_t* free_out,
                             void* workspace, size_t workspace_bytes, void* stream) {
  if (!desc) return SPEAR_ERR_NULL_POINTER;
  spear_status_t st = check_kv_plan(*desc);
  if (st != SPEAR_OK) return st;
  if (table_stride < desc->max_pages || table_stride > (int64_t)1 << 31) return SPEAR_ERR_INVALID_SHAPE;
  const bool some = desc->batch > 0, rows = desc->rows > 0;   // (buffers of no entries may be NULL)
  if ((some && (!lens || !new_tokens || !held || !block_table || !kv_lens || !held_out)) ||
      (rows && (!slots || !positions || !sequence)) || (desc->free_slots > 0 && !free_pages) || !free_count || !cu_q ||
      !free_out)
    return SPEAR_ERR_NULL_POINTER;
  if (!aligned(lens, 4) || !aligned(new_tokens, 4) || !aligned(held, 4) || !aligned(block_table, 4) ||
      !aligned(free_pages, 4) || !aligned(free_count, 4) || !aligned(cu_q, 4) || !aligned(kv_lens, 4) ||
      !aligned(slots, 8) || !aligned(positions, 4) || !aligned(sequence, 4) || !aligned(held_out, 4) ||
      !aligned(free_out, 4))
    return SPEAR_ERR_MISALIGNED;
  st = check_workspace(workspace, workspace_bytes, kv_plan_bytes(*desc));
  if (st != SPEAR_OK) return st;
  KvPlanArgs a;
  a.batch = desc->batch; a.rows = desc->rows; a.max_pages = desc->max_pages; a.free_slots = desc->free_slots;
  a.page_log2 = 0;
  while ((1 << a.page_log2) < desc->page_size) ++a.page_log2;
  a.threads = kv_plan_threads(desc->batch);
  a.lens = lens; a.ask = new_tokens; a.held = held;
  a.table = block_table; a.table_stride = table_stride; a.free_pages = free_pages; a.free_count = free_count;
  a.cu_q = cu_q; a.kv_lens = kv_lens; a.slots = slots; a.positions = positions; a.sequence = sequence;
  a.held_out = held_out; a.free_out = free_out;
  a.in_place = kv_lens == lens || held_out == held || free_out == free_count;
  a.counter = (uint32_t*)workspace;   // the header's first counter
  return hip_status(launch_kv_plan(a, stream));
}

spear_status_t spear_adapter_plan_bytes(int32_t batch, int32_t adapters, int32_t rows, size_t* bytes) {
  if (!bytes) return SPEAR_ERR_NULL_POINTER;
  const spear_status_t st = check_batch(batch, adapters, rows);
  if (st == SPEAR_OK) *bytes = adapter_plan_size(rows, batch, adapters);
  return st;
}

spear_status_t spear_adapter_plan(int32_t batch, int32_t adapters, int32_t rows, const int32_t* cu_q,
                                  const int32_t* adapter, int32_t* plan, size_t plan_bytes, void* stream) {
  const spear_status_t st = check_batch(batch, adapters, rows);
  if (st != SPEAR_OK) return st;
  if (!plan || (batch > 0 && (!cu_q || !adapter))) return SPEAR_ERR_NULL_POINTER;
  if (plan_bytes < adapter_plan_size(rows, batch, adapters)) return SPEAR_ERR_WORKSPACE_TOO_SMALL;
  if (!aligned(cu_q, 4) || !aligned(adapter, 4) || !aligned(plan, 16)) return SPEAR_ERR_MISALIGNED;
  AdapterPlanArgs a;
  a.batch = batch; a.adapters = adapters; a.rows = rows;
  a.most_tiles = (int32_t)adapter_most_tiles(rows, batch, adapters);
  a.cu = cu_q; a.adapter = adapter; a.plan = plan;
  return hip_status(launch_adapter_plan(a, stream));
}

spear_status_t spear_adapter_workspace_bytes(const spear_adapter_desc_t* desc, size_t* bytes) {
  if (!desc || !bytes) return SPEAR_ERR_NULL_POINTER;
  spear_status_t st = check_adapter(*desc);
  if (st != SPEAR_OK) return st;
  int cus = 0;
  st = cus_of(desc->device_cus, &cus);
  if (st == SPEAR_OK) *bytes = desc->rows == 0 || desc->batch == 0 ? 0 : adapter_shape(*desc, cus).bytes;
  return st;
}

spear_status_t spear_adapter_add(const spear_adapter_desc_t* desc, const void* X, int64_t x_stride, const void* A,
                                 const void* B, const float* scale, const int32_t* plan, size_t plan_bytes, void* Y,
                                 int64_t y_stride, void* workspace, size_t workspace_bytes, void* stream) {
  if (!desc) return SPEAR_ERR_NULL_POINTER;
  spear_status_t st = check_adapter(*desc);
  if (st != SPEAR_OK) return st;
  const int64_t most = (int64_t)1 << 31;
  if (x_stride < 0 || x_stride % 8 != 0 || x_stride > most || y_stride < desc->N || y_stride > most)
    return SPEAR_ERR_INVALID_SHAPE;
  if (desc->rows == 0 || desc->batch == 0) return SPEAR_OK;
  if (!X || !A || !B || !plan || !Y) return SPEAR_ERR_NULL_POINTER;
  if (!aligned(X, 16) || !aligned(A, 16) || !aligned(B, 16) || !aligned(scale, 4) || !aligned(plan, 16) || !aligned(Y, 2))
    return SPEAR_ERR_MISALIGNED;
  if (plan_bytes < adapter_plan_size(desc->rows, desc->batch, desc->adapters)) return SPEAR_ERR_WORKSPACE_TOO_SMALL;
  int cus = 0;
  st = cus_of(desc->device_cus, &cus);
  if (st != SPEAR_OK) return st;
  const AdapterShape s = adapter_shape(*desc, cus);
  st = check_workspace(workspace, workspace_bytes, s.bytes);
  if (st != SPEAR_OK) return st;
  AdapterArgs a;
  a.rows = desc->rows; a.adapters = desc->adapters; a.K = desc->K; a.N = desc->N; a.rank = desc->rank;
  a.rank_pad = s.rank_pad; a.most_tiles = s.tiles; a.slices = s.slices; a.slice_k = s.slice_k;
  a.groups = s.groups; a.fused = s.fused; a.chunk_columns = s.chunk_columns;
  a.chunks = (int32_t)ceil_div(desc->N, s.chunk_columns);
  a.X = X; a.A = A; a.B = B; a.scale = scale; a.plan = plan; a.Y = Y;
  a.x_stride = x_stride; a.y_stride = y_stride;
  a.y_vectors = aligned(Y, 16) && y_stride % 8 == 0;
  char* ws = (char*)workspace;
  a.counters = (uint32_t*)ws;   // the header's first counters
  a.part = ws + s.part; a.H = ws + s.H; a.factor = (float*)(ws + s.factor);
  return hip_status(launch_adapter(a, stream));
}

spear_status_t spear_sample_workspace_bytes(const spear_sample_desc_t* desc, size_t* bytes) {
  if (!desc || !bytes) return SPEAR_ERR_NULL_POINTER;
  const spear_status_t st = check_sample(*desc);
  if (st == SPEAR_OK) *bytes = desc->batch == 0 ? 0 : sample_shape(*desc).bytes;
  return st;
}

spear_status_t spear_sample(const spear_sample_desc_t* desc, const void* logits, int64_t row_stride,
                            const int32_t* rows, const float* noise, const float* temperature,
                            const int32_t* top_k, const float* top_p, const float* min_p, int32_t* tokens,
                            float* probs, void* workspace, size_t workspace_bytes, void* stream) {
  if (!desc) return SPEAR_ERR_NULL_POINTER;
  spear_status_t st = check_sample(*desc);
  if (st != SPEAR_OK) return st;
  if (row_stride < 0 || row_stride > (int64_t)1 << 31 || (!rows && desc->batch > desc->num_rows))
    return SPEAR_ERR_INVALID_SHAPE;
  if (desc->batch == 0 || (!tokens && !probs)) return SPEAR_OK;
  const bool one = (!temperature && !(desc->temperature > 0.0f)) || (!top_k && desc->top_k == 1) ||
                   (!top_p && desc->top_p <= 0.0f);
  if ((desc->num_rows > 0 && !logits) || (tokens && !noise && !one)) return SPEAR_ERR_NULL_POINTER;
  const bool f16 = desc->dtype == SPEAR_LOGITS_FP16;
  if (!aligned(logits, f16 ? 2 : 4) || !aligned(rows, 4) || !aligned(noise, 4) || !aligned(temperature, 4) ||
      !aligned(top_k, 4) || !aligned(top_p, 4) || !aligned(min_p, 4) || !aligned(tokens, 4) || !aligned(probs, 4))
    return SPEAR_ERR_MISALIGNED;
  const SampleShape s = sample_shape(*desc);
  st = check_workspace(workspace, workspace_bytes, s.bytes);
  if (st != SPEAR_OK) return st;
  char* ws = (char*)workspace;
  SampleArgs a;
  a.vocab = desc->vocab; a.share_tokens = s.share_tokens; a.shares = s.shares; a.parts = s.parts;
  a.num_rows = desc->num_rows;
  a.f16 = f16; a.only_first = one;
  a.logits = logits; a.stride = row_stride;
  a.one_temperature = desc->temperature; a.one_top_k = desc->top_k; a.one_top_p = desc->top_p; a.one_min_p = desc->min_p;
  a.info = ws + s.info; a.share = (ShareInfo*)(ws + s.share); a.part = (PartInfo*)(ws + s.part);
  a.list = (unsigned long long*)(ws + s.list); a.hist = (unsigned long long*)(ws + s.hist);
  a.list_noise = (float*)(ws + s.list_noise);
  for (int32_t at = 0; at < desc->batch; at += s.group) {
    a.batch = desc->batch - at < s.group ? desc->batch - at : s.group;
    a.first = at;
    a.rows = rows ? rows + at : nullptr;
    a.noise = noise ? noise + (int64_t)at * desc->vocab : nullptr;
    a.temperature = temperature ? temperature + at : nullptr;
    a.top_k = top_k ? top_k + at : nullptr;
    a.top_p = top_p ? top_p + at : nullptr;
    a.min_p = min_p ? min_p + at : nullptr;
    a.tokens = tokens ? tokens + at : nullptr;
    a.probs = probs ? probs + (int64_t)at * desc->vocab : nullptr;
    st = hip_status(launch_sample(a, stream));
    if (st != SPEAR_OK) return st;
  }
  return SPEAR_OK;
}

}  // extern "C"
