// Host check of the index logic that the paged kernels share with it (csrc/paged.h): prints "ok".
#include "../softmax_attention_chunk_gb300/csrc/paged.h"

#include <stdio.h>
#include <vector>

using namespace pathattn;

#define REQUIRE(x) do { if (!(x)) { printf("failed at line %d: %s\n", __LINE__, #x); return 1; } } while (0)

int main() {
  // every row that some new token sees lies in a live tile, tiles rise and stay below t0
  for (int t0 = 0; t0 <= 300; t0 += (t0 < 70 ? 1 : 13))
    for (int window : {0, 1, 2, 16, 63, 64, 65, 200, 1000})
      for (int sinks : {0, 1, 4, 64, 70, 500})
        for (int rows : {16, 64}) {
          const LiveTiles l = live_tiles(t0, window, sinks, rows);
          std::vector<bool> in(t0 / rows + 2, false);
          int last = -1;
          for (int i = 0; i < l.count; ++i) {
            const int t = live_tile(l, i);
            REQUIRE(t > last && t * rows < t0);
            last = t;
            in[t] = true;
          }
          for (int j = 0; j < t0; ++j)
            if (sees(window, sinks, t0, j)) REQUIRE(in[j / rows]);
          // and no tile without a visible row is listed between the two runs
          if (l.skip > 0)
            for (int t = l.nh; t < l.nh + l.skip; ++t)
              for (int j = t * rows; j < (t + 1) * rows && j < t0; ++j) REQUIRE(!sees(window, sinks, t0, j));
        }
  // spans: counts, codes
  const int starts[] = {0, 3, 3, 2, 9, 20, 2147483647};
  REQUIRE(slot_span_of(0, starts, 5, 10, 4, 2, 16).n == 3);
  REQUIRE(slot_span_of(1, starts, 5, 10, 4, 2, 16).n == 0 && slot_span_of(1, starts, 5, 10, 4, 2, 16).code == 0);
  REQUIRE(slot_span_of(1, starts, -1, 10, 4, 2, 16).code == 0);
  REQUIRE(slot_span_of(2, starts, 5, 10, 4, 2, 16).code == PATH_PAGED_BAD_START);   // falls
  REQUIRE(slot_span_of(3, starts, 5, 10, 4, 2, 16).code == PATH_PAGED_BAD_START);   // more than max_new
  REQUIRE(slot_span_of(3, starts, 5, 10, 7, 2, 16).n == 7);
  REQUIRE(slot_span_of(4, starts, 5, 10, 99, 2, 16).code == PATH_PAGED_BAD_START);  // past total
  REQUIRE(slot_span_of(5, starts, 5, 2147483647, 2147483647, 2, 16).code == PATH_PAGED_CAPACITY);
  REQUIRE(slot_span_of(0, starts, -1, 10, 4, 2, 16).code == PATH_PAGED_BAD_SLOT);
  REQUIRE(slot_span_of(0, starts, 29, 10, 4, 2, 16).n == 3);
  REQUIRE(slot_span_of(0, starts, 30, 10, 4, 2, 16).code == PATH_PAGED_CAPACITY);
  REQUIRE(slot_span_of(0, starts, 2147483647, 10, 4, 2, 16).code == PATH_PAGED_CAPACITY);
  REQUIRE(slot_span_of(3, nullptr, -1, 4, 1, 2, 16).n == 0 && slot_span_of(3, nullptr, -1, 4, 1, 2, 16).code == 0);
  REQUIRE(slot_span_of(3, nullptr, 0, 4, 1, 2, 16).q0 == 3);
  // rows of pages: offsets past 32 bits of elements, pages that are none
  path_paged_cache_t c{};
  c.heads = 32;
  c.page_size = 256;
  c.table_width = 3;
  const int table[] = {200000, -1, 7, 250000, 2147483647, 0};
  REQUIRE(pool_row(c, table, 250000, 0, 31, 255) == ((long long)200000 * 32 + 31) * 256 + 255);
  REQUIRE(pool_row(c, table, 250000, 0, 0, 256) == -1);
  REQUIRE(pool_row(c, table, 250000, 0, 2, 513) == ((long long)7 * 32 + 2) * 256 + 1);
  REQUIRE(pool_row(c, table, 250000, 1, 0, 0) == -1);
  REQUIRE(pool_row(c, table, 250000, 1, 0, 300) == -1);
  REQUIRE(pool_row(c, table, 250000, 1, 0, 700) == 188);
  printf("ok\n");
  return 0;
}
