// C ABI entry points of the serving operators (declared in
// include/spear_serve.h): argument checks and launches.  Nothing here allocates
// device memory or synchronizes; every check runs before anything is enqueued.
#include <hip/hip_runtime_api.h>

#include <cmath>

#include "serve_internal.h"

using namespace spear;

namespace {

// Sizes whose products the kernels index with are bounded here: a head's rows
// of the cache and the tensors' elements stay below 2^62.
spear_status_t check_kv(const spear_kv_desc_t& d, KvShape* s) {
  if (d.num_pages < 1 || d.kv_heads < 1 || d.head_dim < 1 || d.page_size < 1) return SPEAR_ERR_INVALID_SHAPE;
  if (d.dtype != SPEAR_KV_FP16 && d.dtype != SPEAR_KV_INT8) return SPEAR_ERR_INVALID_ARGUMENT;
  if (d.head_dim != 64 && d.head_dim != 128) return SPEAR_ERR_UNSUPPORTED;
  if (d.page_size < 16 || d.page_size > 1024 || (d.page_size & (d.page_size - 1)) != 0) return SPEAR_ERR_UNSUPPORTED;
  if (d.kv_heads > 1024) return SPEAR_ERR_UNSUPPORTED;
  s->dtype = d.dtype;
  s->num_pages = d.num_pages;
  s->heads = d.kv_heads;
  s->dim = d.head_dim;
  s->page_log2 = 0;
  while ((1 << s->page_log2) < d.page_size) ++s->page_log2;
  return SPEAR_OK;
}

// Cache pointers: codes and values 16-byte, scales 16-byte (whole vectors of
// them are read).
spear_status_t check_cache(const KvShape& s, const void* k, const void* v, const float* ks, const float* vs) {
  const bool i8 = s.dtype == SPEAR_KV_INT8;
  if (!k || !v || (i8 && (!ks || !vs))) return SPEAR_ERR_NULL_POINTER;
  if (!aligned(k, 16) || !aligned(v, 16) || (i8 && (!aligned(ks, 16) || !aligned(vs, 16)))) return SPEAR_ERR_MISALIGNED;
  return SPEAR_OK;
}

bool row_strides(int64_t token, int64_t head) {
  const int64_t most = (int64_t)1 << 31;
  return token >= 0 && head >= 0 && token % 8 == 0 && head % 8 == 0 && token <= most && head <= most;
}

spear_status_t check_attention(const spear_attention_desc_t& d, KvShape* s) {
  spear_status_t st = check_kv(d.kv, s);
  if (st != SPEAR_OK) return st;
  if (d.batch < 0 || d.total_q < 0 || d.max_q < 1 || d.max_pages < 1 || d.q_heads < 1 || d.q_heads % d.kv.kv_heads != 0)
    return SPEAR_ERR_INVALID_SHAPE;
  if (!(std::fabs(d.scale) <= 1e30f) || d.device_cus < 0) return SPEAR_ERR_INVALID_ARGUMENT;
  // 32-bit counts of rows and keys inside the kernels
  const int64_t most = (int64_t)1 << 30;
  if ((int64_t)d.total_q * d.q_heads > most || (int64_t)d.max_pages * d.kv.page_size > most ||
      (int64_t)d.batch > (1 << 20))
    return SPEAR_ERR_UNSUPPORTED;
  return SPEAR_OK;
}

spear_status_t plan_attention(const spear_attention_desc_t& d, AttnPlan* p) {
  int cus = 0;
  const spear_status_t st = cus_of(d.device_cus, &cus);
  if (st != SPEAR_OK) return st;
  spear_attention_desc_t e = d;
  if (e.max_q > e.total_q) e.max_q = e.total_q;
  *p = attn_plan(e, cus);
  return p->fits ? SPEAR_OK : SPEAR_ERR_UNSUPPORTED;
}

spear_status_t check_verify(const spear_verify_desc_t& d) {
  if (d.batch < 0 || d.max_drafts < 0 || d.vocab < 1) return SPEAR_ERR_INVALID_SHAPE;
  if (d.device_cus < 0) return SPEAR_ERR_INVALID_ARGUMENT;
  // (a launch holds fewer than 2^32 threads; a sequence takes a workgroup of 256 at least)
  if (d.vocab > (1 << 30) || d.max_drafts > (1 << 20) || d.batch >= (1 << 24)) return SPEAR_ERR_UNSUPPORTED;
  return SPEAR_OK;
}

size_t verify_bytes(const spear_verify_desc_t& d, int splits) {
  return splits > 1 ? kSyncHeaderBytes + (size_t)d.batch * splits * sizeof(uint64_t) : 0;
}

}  // namespace

extern "C" {

spear_status_t spear_kv_append(const spear_kv_desc_t* kv, int32_t tokens, const void* k, int64_t k_token_stride,
                               int64_t k_head_stride, const void* v, int64_t v_token_stride,
                               int64_t v_head_stride, const int64_t* slots, void* k_cache, void* v_cache,
                               float* k_scale, float* v_scale, void* stream) {
  if (!kv) return SPEAR_ERR_NULL_POINTER;
  KvAppendArgs a;
  spear_status_t st = check_kv(*kv, &a.kv);
  if (st != SPEAR_OK) return st;
  if (tokens < 0 || !row_strides(k_token_stride, k_head_stride) || !row_strides(v_token_stride, v_head_stride))
    return SPEAR_ERR_INVALID_SHAPE;
  if (tokens == 0) return SPEAR_OK;
  // (a launch holds fewer than 2^32 threads; a workgroup of 256 takes 16 rows at least)
  if ((int64_t)tokens * a.kv.heads > (int64_t)1 << 27) return SPEAR_ERR_UNSUPPORTED;
  if (!k || !v || !slots) return SPEAR_ERR_NULL_POINTER;
  st = check_cache(a.kv, k_cache, v_cache, k_scale, v_scale);
  if (st != SPEAR_OK) return st;
  if (!aligned(k, 16) || !aligned(v, 16) || !aligned(slots, 8)) return SPEAR_ERR_MISALIGNED;
  a.tokens = tokens;
  a.k = k; a.v = v;
  a.k_ts = k_token_stride; a.k_hs = k_head_stride; a.v_ts = v_token_stride; a.v_hs = v_head_stride;
  a.slots = slots;
  a.k_cache = k_cache; a.v_cache = v_cache; a.k_scale = k_scale; a.v_scale = v_scale;
  return hip_status(launch_kv_append(a, stream));
}

spear_status_t spear_kv_gather(const spear_kv_desc_t* kv, int32_t batch, int32_t rows, const int32_t* block_table,
                               int64_t table_stride, const int32_t* cu_kv, const void* k_cache, const void* v_cache,
                               const float* k_scale, const float* v_scale, void* k_out, void* v_out, void* stream) {
  if (!kv) return SPEAR_ERR_NULL_POINTER;
  KvGatherArgs a;
  spear_status_t st = check_kv(*kv, &a.kv);
  if (st != SPEAR_OK) return st;
  if (batch < 0 || rows < 0 || (batch > 0 && table_stride < 1)) return SPEAR_ERR_INVALID_SHAPE;
  if (rows == 0) return SPEAR_OK;
  if ((int64_t)rows * a.kv.heads > (int64_t)1 << 28) return SPEAR_ERR_UNSUPPORTED;   // as above, 32 rows each
  if ((batch > 0 && !block_table) || !cu_kv || !k_out || !v_out) return SPEAR_ERR_NULL_POINTER;   // no table of none
  st = check_cache(a.kv, k_cache, v_cache, k_scale, v_scale);
  if (st != SPEAR_OK) return st;
  if (!aligned(block_table, 4) || !aligned(cu_kv, 4) || !aligned(k_out, 16) || !aligned(v_out, 16))
    return SPEAR_ERR_MISALIGNED;
  a.batch = batch; a.rows = rows;
  a.table = block_table; a.table_stride = table_stride; a.cu = cu_kv;
  a.k_cache = k_cache; a.v_cache = v_cache; a.k_scale = k_scale; a.v_scale = v_scale;
  a.k_out = k_out; a.v_out = v_out;
  return hip_status(launch_kv_gather(a, stream));
}

spear_status_t spear_attention_workspace_bytes(const spear_attention_desc_t* desc, size_t* bytes) {
  if (!desc || !bytes) return SPEAR_ERR_NULL_POINTER;
  KvShape s;
  spear_status_t st = check_attention(*desc, &s);
  if (st != SPEAR_OK) return st;
  *bytes = 0;
  if (desc->total_q == 0 || desc->batch == 0) return SPEAR_OK;
  AttnPlan p;
  st = plan_attention(*desc, &p);
  if (st == SPEAR_OK) *bytes = p.bytes;
  return st;
}

spear_status_t spear_paged_attention(const spear_attention_desc_t* desc, const void* q, int64_t q_token_stride,
                                     int64_t q_head_stride, const int32_t* cu_q, const int32_t* kv_lens,
                                     const int32_t* block_table, int64_t table_stride, const void* k_cache,
                                     const void* v_cache, const float* k_scale, const float* v_scale, void* out,
                                     void* workspace, size_t workspace_bytes, void* stream) {
  if (!desc) return SPEAR_ERR_NULL_POINTER;
  AttnArgs a;
  spear_status_t st = check_attention(*desc, &a.kv);
  if (st != SPEAR_OK) return st;
  if (!row_strides(q_token_stride, q_head_stride) || table_stride < desc->max_pages) return SPEAR_ERR_INVALID_SHAPE;
  if (desc->total_q == 0 || desc->batch == 0) return SPEAR_OK;
  if (!q || !cu_q || !kv_lens || !block_table || !out) return SPEAR_ERR_NULL_POINTER;
  st = check_cache(a.kv, k_cache, v_cache, k_scale, v_scale);
  if (st != SPEAR_OK) return st;
  if (!aligned(q, 16) || !aligned(out, 16) || !aligned(cu_q, 4) || !aligned(kv_lens, 4) || !aligned(block_table, 4))
    return SPEAR_ERR_MISALIGNED;
  AttnPlan p;
  st = plan_attention(*desc, &p);
  if (st != SPEAR_OK) return st;
  if (!workspace) return SPEAR_ERR_NULL_POINTER;
  if (workspace_bytes < p.bytes) return SPEAR_ERR_WORKSPACE_TOO_SMALL;
  if (!aligned(workspace, 16)) return SPEAR_ERR_MISALIGNED;
  a.batch = desc->batch; a.total_q = desc->total_q; a.q_heads = desc->q_heads;
  a.group = desc->q_heads / desc->kv.kv_heads;
  a.max_kv = desc->max_pages * desc->kv.page_size;
  a.scale = desc->scale;
  a.q = q; a.q_ts = q_token_stride; a.q_hs = q_head_stride;
  a.cu_q = cu_q; a.kv_lens = kv_lens; a.table = block_table; a.table_stride = table_stride;
  a.k_cache = k_cache; a.v_cache = v_cache; a.k_scale = k_scale; a.v_scale = v_scale;
  a.out = out;
  a.workspace = workspace;
  return hip_status(launch_attention(a, p, stream));
}

spear_status_t spear_verify_workspace_bytes(const spear_verify_desc_t* desc, size_t* bytes) {
  if (!desc || !bytes) return SPEAR_ERR_NULL_POINTER;
  spear_status_t st = check_verify(*desc);
  if (st != SPEAR_OK) return st;
  int cus = 0;
  st = cus_of(desc->device_cus, &cus);
  if (st == SPEAR_OK) *bytes = verify_bytes(*desc, verify_splits(*desc, cus));
  return st;
}

spear_status_t spear_verify_draft(const spear_verify_desc_t* desc, const float* target, int64_t target_batch_stride,
                                  int64_t target_row_stride, const float* draft, int64_t draft_batch_stride,
                                  int64_t draft_row_stride, const int32_t* drafted, const float* u,
                                  const float* noise, const int32_t* num_drafts, int32_t* accepted,
                                  int32_t* tokens, void* workspace, size_t workspace_bytes, void* stream) {
  if (!desc) return SPEAR_ERR_NULL_POINTER;
  spear_status_t st = check_verify(*desc);
  if (st != SPEAR_OK) return st;
  if (target_batch_stride < 0 || target_row_stride < 0 || draft_batch_stride < 0 || draft_row_stride < 0)
    return SPEAR_ERR_INVALID_SHAPE;
  if (desc->batch == 0) return SPEAR_OK;
  if (!target || !noise || !accepted || !tokens) return SPEAR_ERR_NULL_POINTER;
  if (desc->max_drafts > 0 && (!drafted || !u)) return SPEAR_ERR_NULL_POINTER;
  if (!aligned(target, 4) || !aligned(draft, 4) || !aligned(drafted, 4) || !aligned(u, 4) || !aligned(noise, 4) ||
      !aligned(num_drafts, 4) || !aligned(accepted, 4) || !aligned(tokens, 4))
    return SPEAR_ERR_MISALIGNED;
  int cus = 0;
  st = cus_of(desc->device_cus, &cus);
  if (st != SPEAR_OK) return st;
  VerifyArgs a;
  a.splits = verify_splits(*desc, cus);
  const size_t bytes = verify_bytes(*desc, a.splits);
  if (bytes > 0 && !workspace) return SPEAR_ERR_NULL_POINTER;
  if (workspace_bytes < bytes) return SPEAR_ERR_WORKSPACE_TOO_SMALL;
  if (workspace && !aligned(workspace, 16)) return SPEAR_ERR_MISALIGNED;
  a.batch = desc->batch; a.drafts = desc->max_drafts; a.vocab = desc->vocab;
  a.target = target; a.target_bs = target_batch_stride; a.target_rs = target_row_stride;
  a.draft = draft; a.draft_bs = draft_batch_stride; a.draft_rs = draft_row_stride;
  a.drafted = drafted; a.u = u; a.noise = noise; a.num_drafts = num_drafts;
  a.accepted = accepted; a.tokens = tokens;
  a.counters = (uint32_t*)workspace;   // the first counters of the header
  a.part = bytes > 0 ? (uint64_t*)((char*)workspace + kSyncHeaderBytes) : nullptr;
  return hip_status(launch_verify(a, stream));
}

}  // extern "C"
