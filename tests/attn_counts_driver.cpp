// Whether attention's 32-bit counts hold for any offsets, against a 64-bit count of
// the worst ones (each second sequence has all rows), on the CPU.
#include <climits>
#include <cstdio>

#include "serve_internal.h"

int main() {
  int failures = 0, held = 0, passed = 0;
  const int64_t batches[] = {1, 2, 41, 96, 1000, 4096, 65536, 1 << 20};
  const int64_t totals[] = {1, 7, 96, 2048, 16384, 262144, 1 << 24};
  const int64_t keys[] = {16, 128, 8192, 131072, 1 << 24};
  for (int64_t batch : batches)
    for (int64_t rows : totals)
      for (int64_t max_kv : keys)
        for (int64_t heads : {1, 8, 1024}) {
          // few rows: tiles of 16, steps of 128 keys and two more; tiles of 128 rows, 64 keys
          const struct { int64_t r, k, extra, h, most; } kinds[] = {{16, 128, 2, heads, INT32_MAX}, {128, 64, 0, 1, INT32_MAX / 2}};
          for (const auto& c : kinds) {
            __int128 count = 0;
            for (int64_t b = 0; b < batch; b += 2)
              count += (__int128)((rows + c.r - 1) / c.r) * ((max_kv + c.k - 1) / c.k + c.extra) * c.h;
            const bool hold = spear::counts_hold(batch, rows, c.r, max_kv, c.k, c.extra, c.h, c.most);
            if (hold && count > c.most) ++failures;         // would wrap unseen
            if (!hold && count * 2 <= c.most) ++failures;   // looked at for nothing
            ++(hold ? held : passed);
          }
        }
  if (spear::counts_hold(96, 96 * 4, 16, 8192, 128, 2, 8, INT32_MAX) == false) ++failures;   // an ordinary decode step
  if (failures || !held || !passed) return std::printf("%d failures\n", failures), 1;
  std::printf("all checks passed\n");
  return 0;
}
