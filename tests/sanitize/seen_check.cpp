// The tokens that the cut into parts takes a tile's rows to see are no fewer than those between the first and the last one that any of
// them sees, and no more than there are; windows and first tokens of any size.  Prints the number of tiles and ends with 0.
#include <algorithm>
#include <cstdio>
#include <initializer_list>

#include "qv_runs_internal.h"

int main() {
  long checked = 0;
  for (int64_t capacity : {64, 1024, 3008})
    for (int64_t run : {1, 40, 128, 300, 1000})
      for (int64_t share : {1, 3, 128, 200})
        for (int64_t window : {0, 1, 70, 500, 5000})
          for (int64_t sinks : {0, 5, 90, 2000})
            for (bool causal : {true, false}) {
              if (run > capacity) continue;
              const int64_t seen = qv::tokens_of_tile(capacity, run, window, sinks, causal);
              for (int64_t row = 0; row < run * share; row += qv::kRowsPerTile) {
                const int64_t last = std::min(row + qv::kRowsPerTile, run * share) - 1, before = capacity - run;
                const int64_t high = causal ? before + last / share + 1 : capacity;
                const int64_t low = window ? std::max<int64_t>(0, before + row / share - window + 1) : 0;
                const int64_t all = high - low + std::min(sinks, low);
                if (all > seen || seen > capacity) {
                  std::printf("capacity %ld run %ld share %ld window %ld sinks %ld causal %d row %ld: sees %ld, taken as %ld\n",
                              (long)capacity, (long)run, (long)share, (long)window, (long)sinks, (int)causal, (long)row, (long)all,
                              (long)seen);
                  return 1;
                }
                ++checked;
              }
            }
  const int64_t far = (int64_t{1} << 31) - 128;
  for (int64_t window : {int64_t{0}, int64_t{7}, far - 1, far, INT64_MAX})  // no sum overflows
    for (int64_t sinks : {int64_t{0}, int64_t{3}, far, int64_t{1} << 31, INT64_MAX})
      for (int64_t capacity : {int64_t{0}, int64_t{64}, far})
        for (bool causal : {true, false}) {
          const int64_t seen = qv::tokens_of_tile(capacity, far, window, sinks, causal);
          if (seen < 0 || seen > capacity) return 1;
          ++checked;
        }
  std::printf("%ld\n", checked);
  return checked > 1000 ? 0 : 1;
}
