// Tiles that the adapters' products read from a plan, over plans of theirs and over words that
// are no plan's (negative, huge, of other sizes), on the CPU.
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
  const int32_t words[] = {INT_MIN, INT_MIN + 1, -65, -1, 0, 1, 2, 15, 16, 17, 63, 64, 65, 99, 100, 101, 1 << 24, INT_MAX - 1, INT_MAX};
  const int32_t sizes[] = {1, 2, 63, 64, 65, 100, 4096, 1 << 24};
  for (int32_t adapters : {1, 5, 64, 4096})
    for (int32_t all : sizes)
      for (int32_t adapter : words)
        for (int32_t first : words)
          for (int32_t rows : words) {
            const spear::AdapterTile t = spear::adapter_tile(adapter, first, rows, adapters, all);
            CHECK(t.adapter >= 0 && t.adapter < adapters);
            CHECK(t.rows >= 1 && t.rows <= spear::kAdapterTile);
            CHECK(t.first >= 0 && t.first + t.rows <= all);
            // (a plan's own tiles stay as they are)
            if (adapter >= 0 && adapter < adapters && first >= 0 && rows >= 1 && rows <= spear::kAdapterTile && first < all &&
                rows <= all - first)
              CHECK(t.adapter == adapter && t.first == first && t.rows == rows);
          }
  if (failures) return 1;
  std::printf("all checks passed\n");
  return 0;
}
