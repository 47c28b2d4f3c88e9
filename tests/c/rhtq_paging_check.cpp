// Host check of the paged cache's index arithmetic (randomized_hadamard_rotation_amd/csrc/rhtq_paging.h): whatever a table and the
// lengths hold, no page outside [0, pages) comes out, and the tiles a query looks at cover exactly the visible positions.
#include <stdio.h>
#include <stdlib.h>

#include <vector>

#include "rhtq_paging.h"

#define REQUIRE(c)                                              \
  do {                                                          \
    if (!(c)) {                                                 \
      printf("line %d: %s\n", __LINE__, #c);                    \
      exit(1);                                                  \
    }                                                           \
  } while (0)

int main() {
  const int32_t row[6] = {3, -1, 7, 1 << 30, INT32_MIN, 0};
  REQUIRE(rhtq::page_at(row, 6, 8, 0) == 3 && rhtq::page_at(row, 6, 8, 2) == 7 && rhtq::page_at(row, 6, 8, 5) == 0);
  REQUIRE(rhtq::page_at(row, 6, 7, 2) == -1 && rhtq::page_at(row, 6, 0, 5) == -1);
  for (int64_t i : {(int64_t)-1, (int64_t)1, (int64_t)3, (int64_t)4, (int64_t)6, (int64_t)1 << 40})
    REQUIRE(rhtq::page_at(row, 6, 8, i) == -1);
  REQUIRE(rhtq::clamp_length(-5, 4, 16) == 0 && rhtq::clamp_length(65, 4, 16) == 64 && rhtq::clamp_length(9, 0, 16) == 0);
  REQUIRE(rhtq::row_position(0, 1, 1) == 0 && rhtq::row_position(2, 5, 2) == -1 && rhtq::row_position(4, 5, 100) == 99);
  REQUIRE(rhtq::row_position(0, INT32_MAX, INT32_MIN) < 0);
  for (int len = -1; len <= 150; ++len)
    for (int window = 0; window <= 150; window += (window < 40 ? 1 : 13))
      for (int sinks = 0; sinks <= 70; sinks += (sinks < 20 ? 1 : 9)) {
        const rhtq::Visible v = rhtq::visible_of(len, 9, 16, window, sinks);
        const int n = len < 0 ? 0 : (len > 144 ? 144 : len);
        std::vector<int> seen(160, 0);
        REQUIRE(v.tiles >= 0);
        int last = -1;
        for (int i = 0; i < v.tiles; ++i) {
          const int t = rhtq::tile_at(v, i);
          REQUIRE(t > last && t >= 0 && t < 9);
          last = t;
          for (int k = 0; k < 16; ++k)
            if (rhtq::is_visible(v, 16 * t + k)) seen[16 * t + k]++;
        }
        for (int p = 0; p < 160; ++p)
          REQUIRE(seen[p] == (p < n && (window == 0 || p >= n - window || p < sinks)));
        for (int splits = 1; splits < 9; ++splits) {
          const int per = rhtq::tiles_per_split(v.tiles, splits, 4);
          REQUIRE(per % 4 == 0 && (int64_t)per * splits >= v.tiles);
        }
      }
  printf("ok\n");
  return 0;
}
