// Host-side checks of the paged cache's and the windowed attention's index
// arithmetic: the library's own __host__ __device__ helpers, compiled by nvcc
// and run on the CPU (no GPU is touched).  Run by tests/test_kv_index_checks.py.
//   * the pages of a call's entries: running sums beyond 2^31 serve nobody
//     twice and leave the search for a page's entry in order;
//   * the parts of a tile's keys: they follow one another from the first key
//     tile to the last, each as long as the others but for one tile, up to 2^30
//     keys in tiles of 32 and as many parts as there are CTAs at once;
//   * the rounds of a token's keys, up to 2^31 - 1 of them.
#include <cstdio>
#include <vector>

#include "../block_denoising_gb300/csrc/window_attention.cuh"

using namespace dinfer;

static long long g_fail = 0;
#define CHECK(cond, ...)                   \
  do {                                     \
    if (!(cond)) {                         \
      if (g_fail < 20) {                   \
        std::printf("FAIL %s: ", #cond);   \
        std::printf(__VA_ARGS__);          \
        std::printf("\n");                 \
      }                                    \
      ++g_fail;                            \
    }                                      \
  } while (0)

// needs in order, `found` free pages: an entry is served while the sum so far stays within them
static void pages_of_a_call(const std::vector<int>& needs, int found) {
  __int128 sum = 0;
  int last = 0;
  for (size_t i = 0; i < needs.size(); ++i) {
    CHECK(kv_reaches((long long)sum, needs[i], found) == (sum + needs[i] <= found), "entry %zu of %d pages", i, needs[i]);
    const int place = kv_place((long long)sum);
    CHECK(place >= last, "place %d of entry %zu behind %d", place, i, last);  // what the search of an entry relies on
    CHECK(sum > found ? place > found : place == (int)sum, "place %d of entry %zu", place, i);
    last = place;
    sum += needs[i];
  }
}

static void parts_of_keys() {
  for (int w : {1, 2, 3, 7, 271, 4096, 7375000, 7400000, (1 << 25) - 1, 1 << 25})
    for (int parts = 1; parts <= 304 && parts <= w; ++parts)
      for (int part = 0; part < parts; ++part) {
        const int a = wa_part_begin(w, part, parts), b = wa_part_begin(w, part + 1, parts);
        CHECK(a == (long long)part * w / parts, "part %d of %d of %d tiles: %d", part, parts, w, a);
        CHECK(b - a == w / parts || b - a == w / parts + 1, "part %d of %d of %d tiles: %d", part, parts, w, b - a);
        CHECK((part > 0 || a == 0) && (part + 1 < parts || b == w), "ends of %d tiles in %d parts", w, parts);
        CHECK((long long)b * kWfKeys <= 1 << 30, "key %d beyond 2^30", b);
      }
}

static void rounds_of_keys() {
  for (int round : {64, 128, 256})
    for (int seen : {1, 63, 64, 65, 128, 256, 257, 1 << 20, (1 << 30) + 1, 0x7fffffff - 256, 0x7fffffff - 254, 0x7fffffff - 1, 0x7fffffff})
      CHECK(ka_rounds(seen, round) == ((long long)seen + round - 1) / round, "%d keys in rounds of %d", seen, round);
}

int main() {
  const int big = 0x7fffffff;
  for (int found : {0, 1, 7, 1000, 1 << 30, big - 1}) {
    for (int need : {1, 5, 1 << 21, 1 << 30, big}) {
      pages_of_a_call(std::vector<int>(1024, need), found);
      std::vector<int> mixed;
      for (int i = 0; i < 1024; ++i) mixed.push_back(i % 3 == 0 ? need : i % 3 == 1 ? 0 : i);
      pages_of_a_call(mixed, found);
    }
    // sums that come back to a small number modulo 2^32
    pages_of_a_call({1 << 30, 1 << 30, 1 << 30, 1 << 30, 3, 2}, found);
  }
  parts_of_keys();
  rounds_of_keys();
  std::printf("kv index checks: %lld failures\n", g_fail);
  return g_fail ? 1 : 0;
}
