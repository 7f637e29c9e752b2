// Drives zero_piece_table over random layouts with tables of exactly the size
// it asks for, and with short ones; built with the sanitizers.
#include <cstdio>
#include <cstdlib>
#include <vector>

#include "zero_shard.h"

static uint64_t state = 12345;
static uint64_t rnd(uint64_t n) {
  state = state * 6364136223846793005ull + 1442695040888963407ull;
  return (state >> 33) % n;
}

#define CHECK(x)                                         \
  do {                                                   \
    if (!(x)) {                                          \
      std::printf("line %d: %s\n", __LINE__, #x);        \
      return 1;                                          \
    }                                                    \
  } while (0)

int main() {
  for (int it = 0; it < 4000; ++it) {
    const uint32_t n = 1 + (uint32_t)rnd(30), ranks = 1 + (uint32_t)rnd(6);
    const uint32_t aligns[] = {1, 8, 64, 128};
    const uint64_t most[] = {4, 100, 9000};
    std::vector<uint64_t> numel(n), off(n), b(ranks), e(ranks);
    for (auto& x : numel) x = 1 + rnd(most[rnd(3)]);
    uint64_t total = 0;
    CHECK(zero_shard_layout(numel.data(), n, ranks, aligns[rnd(4)], off.data(), &total, b.data(), e.data()) == ZERO_OK);
    const uint32_t r = (uint32_t)rnd(ranks);
    uint64_t pieces = 0, masks = 0, p2 = 0, m2 = 0;
    CHECK(zero_piece_table(numel.data(), off.data(), n, b[r], e[r], nullptr, 0, nullptr, 0, &pieces, &masks) == ZERO_OK);
    std::vector<zero_piece> out(pieces);
    std::vector<uint8_t> bytes(masks * (ZERO_PIECE / 8));
    CHECK(zero_piece_table(numel.data(), off.data(), n, b[r], e[r], out.data(), pieces, bytes.data(), masks, &p2, &m2) ==
          ZERO_OK);
    CHECK(p2 == pieces && m2 == masks);
    uint64_t real = 0, want = 0;
    for (const auto& p : out) {
      if (p.mask == ZERO_PIECE_WHOLE) {
        real += p.len;
      } else {
        CHECK(p.mask < masks);
        for (uint32_t i = 0; i < ZERO_PIECE / 8; ++i)
          real += (uint64_t)__builtin_popcount(bytes[(uint64_t)p.mask * (ZERO_PIECE / 8) + i]);
      }
    }
    for (uint32_t k = 0; k < n; ++k) {
      const uint64_t lo = off[k] > b[r] ? off[k] : b[r], hi = off[k] + numel[k] < e[r] ? off[k] + numel[k] : e[r];
      if (lo < hi) want += hi - lo;
    }
    CHECK(real == want);
    if (pieces > 1) {
      std::vector<zero_piece> less(pieces / 2);
      std::vector<uint8_t> fewer(masks / 2 * (ZERO_PIECE / 8));
      CHECK(zero_piece_table(numel.data(), off.data(), n, b[r], e[r], less.data(), less.size(), fewer.data(), masks / 2,
                             &p2, &m2) == ZERO_ERANGE);
      CHECK(p2 == pieces && m2 == masks);
    }
  }
  std::printf("clean\n");
  return 0;
}
