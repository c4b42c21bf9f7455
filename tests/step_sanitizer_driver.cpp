// Drives the host code of a serving step's other operators (argument checks, launch shapes)
// under AddressSanitizer and UndefinedBehaviorSanitizer, on the CPU: descriptors from
// small to extreme, and calls that the checks must end before a launch.
#include <climits>
#include <cmath>
#include <cstdint>
#include <cstdio>
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
  const int32_t odd[] = {INT_MIN, -8, -1, 0, 1, 7, 8, 16, 63, 64, 65, 256, 257, 1000, 1024, 4096, 4097, 1 << 20, (1 << 22) + 1,
                         1 << 24, 1 << 26, 1 << 30, INT_MAX};
  alignas(64) static char mem[1 << 12];
  int32_t* const words = (int32_t*)mem;
  float* const values = (float*)mem;
  int planned = 0;
  for (int32_t batch : odd)
    for (int32_t rows : odd)
      for (int32_t pages : odd)
        for (int32_t page : odd)
          for (int32_t slots : {-1, 0, INT_MAX}) {
            spear_kv_plan_desc_t d = {batch, rows, pages, page, slots};
            size_t n = 12345;
            const spear_status_t st = spear_kv_plan_workspace_bytes(&d, &n);
            planned += st == SPEAR_OK;
            // A call never gets past the checks: no workspace, or a pointer that is not aligned.
            const spear_status_t call = spear_kv_plan(&d, words, words, words, words, (int64_t)1 << 31, words, words, words,
                                                      words, (int64_t*)mem, words, words, words, (int32_t*)(mem + 1), mem, 0,
                                                      nullptr);
            CHECK(st == SPEAR_OK ? call == SPEAR_ERR_MISALIGNED : call == st);
            for (int64_t stride : {INT64_MIN, (int64_t)-1, INT64_MAX}) {
              const spear_status_t s = spear_kv_plan(&d, words, words, words, words, stride, words, words, words, words,
                                                     (int64_t*)mem, words, words, words, words, mem, 0, nullptr);
              CHECK(st == SPEAR_OK ? s == SPEAR_ERR_INVALID_SHAPE : s == st);
            }
          }
  for (int32_t batch : odd)
    for (int32_t adapters : odd)
      for (int32_t rows : odd) {
        size_t plan = 12345;
        const spear_status_t st = spear_adapter_plan_bytes(batch, adapters, rows, &plan);
        CHECK(st != SPEAR_OK || (plan >= 16 && plan < ((size_t)1 << 28)));
        if (st == SPEAR_OK)
          CHECK(spear_adapter_plan(batch, adapters, rows, words, words, words, plan - 1, nullptr) ==
                SPEAR_ERR_WORKSPACE_TOO_SMALL);
        for (int32_t K : odd)
          for (int32_t N : {0, 1, 4096, 1 << 24, INT_MAX})
            for (int32_t rank : {-8, 0, 8, 24, 64, 256, 264, INT_MAX})
              for (int32_t cus : {1, 256, INT_MAX}) {
                spear_adapter_desc_t d = {batch, adapters, rows, K, N, rank, cus};
                size_t n = 12345;
                const spear_status_t s = spear_adapter_workspace_bytes(&d, &n);
                CHECK(st == SPEAR_OK || s == st);
                if (s != SPEAR_OK) continue;
                ++planned;
                CHECK(batch == 0 || rows == 0 ? n == 0 : n > (1u << 20) && n < ((size_t)1 << 36));
                if (n > 0)
                  CHECK(spear_adapter_add(&d, mem, (int64_t)1 << 31, mem, mem, values, words, plan, mem, (int64_t)1 << 31, mem,
                                          n - 1, nullptr) == SPEAR_ERR_WORKSPACE_TOO_SMALL);
                for (int64_t stride : {INT64_MIN, (int64_t)-8, (int64_t)4, INT64_MAX})
                  CHECK(spear_adapter_add(&d, mem, stride, mem, mem, values, words, plan, mem, N, mem, 0, nullptr) ==
                        SPEAR_ERR_INVALID_SHAPE);
                CHECK(spear_adapter_add(&d, mem, 8, mem, mem, values, words, plan, mem, INT64_MIN, mem, 0, nullptr) ==
                      SPEAR_ERR_INVALID_SHAPE);
              }
      }
  for (int32_t batch : odd)
    for (int32_t vocab : odd)
      for (int32_t rows : odd)
        for (int32_t dtype : {-1, 0, 1, 2})
          for (float setting : {-INFINITY, -1.0f, 0.0f, 1.0f, INFINITY, NAN}) {
            spear_sample_desc_t d = {batch, vocab, rows, dtype, setting, (int32_t)1 << 30, setting, setting};
            size_t n = 12345;
            const spear_status_t st = spear_sample_workspace_bytes(&d, &n);
            if (st != SPEAR_OK) continue;
            ++planned;
            CHECK(batch == 0 ? n == 0 : n > (1u << 20) && n < ((size_t)1 << 32));
            if (n > 0)
              CHECK(spear_sample(&d, mem, (int64_t)1 << 31, words, values, values, nullptr, values, nullptr, words, values, mem,
                                 n - 1, nullptr) == SPEAR_ERR_WORKSPACE_TOO_SMALL);
            for (int64_t stride : {INT64_MIN, (int64_t)-1, INT64_MAX})
              CHECK(spear_sample(&d, mem, stride, words, values, values, words, values, values, words, values, mem, 0, nullptr) ==
                    SPEAR_ERR_INVALID_SHAPE);
          }
  if (failures) return 1;
  std::printf("all checks passed (%d plans)\n", planned);
  return 0;
}
