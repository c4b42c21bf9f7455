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

}  // extern "C"
