// Drives the serving operators' host code (argument checks, planning) under
// AddressSanitizer and UndefinedBehaviorSanitizer, on the CPU: descriptors from
// small to extreme, and calls that the checks must end before a launch.
#include <climits>
#include <cstdint>
#include <cstdio>
#include <cstdlib>
#include <initializer_list>

#include "spear_serve.h"

static int failures = 0;
#define CHECK(c)                                                   \
  do {                                                             \
    if (!(c)) {                                                    \
      std::printf("line %d: %s\n", __LINE__, #c);                  \
      ++failures;                                                  \
    }                                                              \
  } while (0)

int main() {
  const int32_t odd[] = {INT_MIN, -1, 0, 1, 2, 3, 7, 16, 64, 65, 128, 1000, 1024, 4097, 1 << 20, 1 << 30, INT_MAX};
  alignas(64) static char mem[1 << 12];
  int planned = 0;
  for (int32_t batch : odd)
    for (int32_t total : odd)
      for (int32_t max_q : odd)
        for (int32_t pages : odd)
          for (int32_t heads : {1, 8, 1024})
            for (int32_t group : {1, 5, 64})
              for (int32_t cus : {1, 256, INT_MAX}) {
                spear_attention_desc_t d = {{SPEAR_KV_INT8, 4, heads, 128, 1024}, batch, total, max_q, pages,
                                            heads * group, 0.1f, cus};
                size_t n = 12345;
                const spear_status_t st = spear_attention_workspace_bytes(&d, &n);
                if (st == SPEAR_OK) {
                  ++planned;
                  CHECK(batch == 0 || total == 0 ? n == 0 : n > (1u << 20) && n < ((size_t)1 << 32));
                }
                // A call never gets past the checks: no workspace.
                const spear_status_t call = spear_paged_attention(
                    &d, mem, 128 * heads * group, 128, (int32_t*)mem, (int32_t*)mem, (int32_t*)mem, INT_MAX, mem, mem,
                    (float*)mem, (float*)mem, mem, mem, 0, nullptr);
                CHECK(st == SPEAR_OK && n > 0 ? call == SPEAR_ERR_WORKSPACE_TOO_SMALL : call == st);
              }
  CHECK(planned > 0);
  for (int32_t batch : odd)
    for (int32_t drafts : odd)
      for (int32_t vocab : odd)
        for (int32_t cus : {1, 256, INT_MAX}) {
          spear_verify_desc_t d = {batch, drafts, vocab, cus};
          size_t n = 12345;
          const spear_status_t st = spear_verify_workspace_bytes(&d, &n);
          if (st == SPEAR_OK && batch > 0 && n > 0)
            CHECK(spear_verify_draft(&d, (float*)mem, 1, 1, (float*)mem, 1, 1, (int32_t*)mem, (float*)mem, (float*)mem,
                                     nullptr, (int32_t*)mem, (int32_t*)mem, mem, n - 1, nullptr) ==
                  SPEAR_ERR_WORKSPACE_TOO_SMALL);
        }
  for (int32_t dtype : odd)
    for (int32_t pages : odd)
      for (int32_t heads : odd)
        for (int32_t dim : odd)
          for (int32_t page : odd) {
            spear_kv_desc_t d = {dtype, pages, heads, dim, page};
            // Null tensors: refused, or the shape is.
            CHECK(spear_kv_append(&d, 1, nullptr, INT64_MAX, 8, nullptr, 8, 8, nullptr, nullptr, nullptr, nullptr,
                                  nullptr, nullptr) != SPEAR_OK);
            CHECK(spear_kv_append(&d, 1, nullptr, 8, 8, nullptr, 8, 8, nullptr, nullptr, nullptr, nullptr, nullptr,
                                  nullptr) != SPEAR_OK);
            CHECK(spear_kv_gather(&d, 1, 1, nullptr, 1, nullptr, nullptr, nullptr, nullptr, nullptr, nullptr, nullptr,
                                  nullptr) != SPEAR_OK);
          }
  if (failures) return 1;
  std::printf("all checks passed (%d plans)\n", planned);
  return 0;
}
