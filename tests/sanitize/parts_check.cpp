// The cut of a batch's tokens into parts never needs more of them than the workspace and the grid have, whatever the
// lengths are: random batches and the largest ones.  Prints the number of batches and ends with 0.
#include <cstdio>
#include <random>
#include <vector>

#include "qv_decode_internal.h"

template <typename U>
static int64_t parts_of(const std::vector<int64_t>& tiles, int64_t few, int64_t many) {
  uint64_t total = 0;
  for (int64_t n : tiles) total += (uint64_t)n;
  const int64_t per = qv::tiles_of_part((U)total, (U)few, (U)many);
  if (per <= 0) return INT64_MAX;
  int64_t parts = 0;
  for (int64_t n : tiles) parts += n > per ? (n + per - 1) / per : 1;
  return parts;
}

int main() {
  std::mt19937_64 rng(1);
  auto pick = [&](int64_t lo, int64_t hi) { return lo + (int64_t)(rng() % (uint64_t)(hi - lo + 1)); };
  int checked = 0;
  for (int i = 0; i < 200000; ++i) {
    const int64_t heads = i % 5 == 0 ? pick(1, 65536) : pick(1, 64), share = pick(1, 3) == 1 ? pick(1, 40) : 1;
    if (heads * share > 65536) continue;
    const int64_t B = i % 7 == 0 ? pick(1, 2000) : pick(1, 70);
    const int64_t capacity = 16 * (i % 3 == 0 ? pick(0, (1 << 27) - 1) : pick(0, 4000));
    const auto p = qv::paged_attention_parts(B, heads * share, heads, capacity);
    std::vector<int64_t> tiles(B);
    for (auto& n : tiles) n = i % 2 ? capacity / 16 : pick(0, capacity / 16);
    const int64_t few = pick(1, p.many);
    const bool fits = capacity / 16 * B < (int64_t{1} << 31) - qv::kManyBlocks;
    const int64_t wide = parts_of<uint64_t>(tiles, few, p.many);
    if (wide > p.most || (fits && parts_of<uint32_t>(tiles, few, p.many) != wide)) {
      std::printf("B %lld heads %lld share %lld capacity %lld few %lld: %lld parts, room for %lld\n", (long long)B,
                  (long long)heads, (long long)share, (long long)capacity, (long long)few, (long long)wide, (long long)p.most);
      return 1;
    }
    ++checked;
  }
  std::printf("%d\n", checked);
  return checked > 100000 ? 0 : 1;
}
