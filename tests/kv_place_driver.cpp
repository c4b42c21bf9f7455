// Places that the cache's read-back computes from its offsets, over offsets that
// keep the contract and offsets that break it (falling, negative, huge), on the CPU.
#include <climits>
#include <cstdio>

#include "serve_internal.h"

static int failures = 0;
#define CHECK(c)                                  \
  do {                                            \
    if (!(c)) {                                   \
      std::printf("line %d: %s\n", __LINE__, #c); \
      ++failures;                                 \
    }                                             \
  } while (0)

int main() {
  const int32_t firsts[] = {INT_MIN, INT_MIN + 1, -100000, -17, -1, 0, 1, 5, 16, 100, 1 << 20, INT_MAX - 1, INT_MAX};
  const int64_t rows[] = {0, 1, 4, 5, 15, 16, 17, 1000, 1 << 28};
  const int64_t strides[] = {1, 2, 7, 1 << 20, INT_MAX, (int64_t)1 << 40};
  for (int log2 = 4; log2 <= 10; ++log2)
    for (int64_t stride : strides)
      for (int64_t row : rows)
        for (int32_t first : firsts) {
          const int64_t e = spear::table_entry(row, first, log2, stride);
          if (row < first) {
            CHECK(e == -1);
          } else {
            const int64_t want = (row - (int64_t)first) / (1 << log2);
            CHECK(e >= 0 && e < stride);
            CHECK(e == (want < stride ? want : stride - 1));
          }
        }
  if (failures) return 1;
  std::printf("all checks passed\n");
  return 0;
}
