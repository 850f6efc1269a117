// Host check of kv_layout.h: every index function against a plain count, over
// small sizes exhaustively. Prints "ok" or the first thing that is wrong.
#include <cstdio>
#include <cstring>
#include <vector>

#include "kv_layout.h"

using namespace ringsim;

#define CHECK(x)                                              \
  do {                                                        \
    if (!(x)) {                                               \
      std::printf("line %d: %s\n", __LINE__, #x);             \
      return 1;                                               \
    }                                                         \
  } while (0)

static float value(uint32_t bits) {
  float f;
  std::memcpy(&f, &bits, 4);
  return f;
}
static uint32_t bits_of(float f) {
  uint32_t u;
  std::memcpy(&u, &f, 4);
  return u;
}

int main() {
  // Exponents: the least e >= -126 with max <= 7 * 2^e, at most 125.
  for (uint32_t i = 0; i < 0x7f800000u; i += 9973) {
    for (int near = -1; near <= 1; ++near) {
      const uint32_t top = near == 0 ? i : (i & 0x7f800000u) + 0x600000u + (uint32_t)near;  // beside 1.75 * 2^x
      if (top >= 0x7f800000u) continue;
      const int byte = kv_exponent_byte(top);
      CHECK(byte >= 1 && byte <= 252);
      const double max = value(top), unit = value((uint32_t)byte << 23);
      if (byte < 252) CHECK(max <= 7 * unit);
      if (byte > 1) CHECK(max > 3.5 * unit);
    }
  }
  CHECK(kv_exponent_byte(bits_of(7.0f)) == 127 && kv_exponent_byte(bits_of(7.0f) + 1) == 128);
  CHECK(kv_exponent_byte(0) == 1 && kv_exponent_byte(0x7f800000u) == 255 && kv_exponent_byte(0x7fc00000u) == 255);

  // Slots.
  for (int shift = 4; shift <= 10; ++shift) {
    for (int64_t pages = 1; pages < 5; ++pages) {
      int32_t page;
      int token;
      for (int64_t s = 0; s < pages << shift; ++s)
        CHECK(kv_slot(s, pages, shift, &page, &token) && page == s / (1 << shift) && token == s % (1 << shift));
      for (int64_t s : {(int64_t)-1, pages << shift, (int64_t)1 << 40, INT64_MAX, INT64_MIN})
        CHECK(!kv_slot(s, pages, shift, &page, &token));
    }
  }

  // Places of tiles: always inside the row, the tile's own where it has one.
  for (int shift = 4; shift <= 6; ++shift) {
    for (int64_t max_pages = 1; max_pages <= 8; ++max_pages) {
      for (int64_t end = 0; end <= 9 << shift; end += 5) {
        for (int64_t tile = -2; tile < 10 << (shift - 4); ++tile) {
          int64_t place = -1;
          const bool got = kv_place_of_tile(tile, end, shift, max_pages, &place);
          const int64_t own = tile * 16 >> shift;
          CHECK(place >= 0 && place < max_pages);
          CHECK(got == (tile >= 0 && tile * 16 < end && own < max_pages));
          if (got) CHECK(place == own);
        }
      }
    }
  }
  CHECK(kv_is_page(0, 1) && !kv_is_page(1, 1) && !kv_is_page(-1, 1) && !kv_is_page(INT32_MIN, 7) && !kv_is_page(INT32_MAX, 7));

  // Tiles of rows: each tile of each sequence has one number below the bound, and leads back to its sequence.
  uint32_t seed = 1;
  const auto next = [&](uint32_t n) { return (int64_t)((seed = seed * 1664525u + 1013904223u) >> 8) % n; };
  for (int turn = 0; turn < 3000; ++turn) {
    const int64_t seqs = 1 + next(9), group = 1 + next(9), rows = 16 << next(4);
    std::vector<int32_t> starts = {(int32_t)next(3)};
    for (int64_t b = 0; b < seqs; ++b) starts.push_back(starts.back() + (next(3) ? (int32_t)next(40) : 0));
    const int64_t tokens = starts.back() + next(4), bound = tokens * group / rows + seqs;
    std::vector<int> taken(bound, 0);
    for (int64_t b = 0; b < seqs; ++b) {
      const int64_t n = (starts[b + 1] - starts[b]) * group;
      for (int64_t t = 0; t * rows < n; ++t) {
        const int64_t number = kv_first_tile(starts[b], b, group, rows) + t;
        CHECK(number >= 0 && number < bound && !taken[number]++);
        CHECK(kv_seq_of_tile(starts.data(), seqs, tokens, group, rows, number) == b);
      }
    }
    // Starts that decrease or lead outside still give a sequence of the call.
    for (auto& s : starts) s = (int32_t)next(200) - 100;
    for (int64_t t = 0; t < bound; ++t) {
      const int64_t b = kv_seq_of_tile(starts.data(), seqs, tokens, group, rows, t);
      CHECK(b >= 0 && b < seqs);
    }
  }

  // Spans.
  for (int64_t end = 0; end < 12; ++end)
    for (int64_t p = -4; p < 14; ++p)
      for (int causal = 0; causal < 2; ++causal)
        for (int64_t window = 0; window < 6; ++window) {
          int64_t lo, hi;
          kv_span(p, end, causal, window, &lo, &hi);
          for (int64_t j = -2; j < 14; ++j) {
            const bool sees = j >= 0 && j < end && (!causal || j <= p) && (!window || j > p - window);
            CHECK((j >= lo && j <= hi) == sees);
          }
        }
  // Units: as many as cover a span, from the pass that holds its first position.
  for (int64_t lo = 0; lo < 300; lo += 7)
    for (int64_t hi = lo - 3; hi < lo + 700; ++hi) {
      const int64_t n = kv_units(lo, hi), first = lo - lo % 32;
      if (hi < lo) {
        CHECK(n == 1);
      } else {
        CHECK(first + n * 128 > hi && first + (n - 1) * 128 <= hi);
        CHECK(n <= kv_units(31, 30 + hi - lo + 1));  // the host's bound
      }
    }

  // Shares: they follow one another, hold all units and differ by one at most.
  const auto shares = [](uint32_t units, uint32_t groups) {
    CHECK(kv_share_begin(units, 0, groups) == 0 && kv_share_begin(units, groups, groups) == units);
    for (uint32_t w = 0; w < groups; ++w) {
      const uint32_t n = kv_share_begin(units, w + 1, groups) - kv_share_begin(units, w, groups);
      CHECK(n >= units / groups && n <= units / groups + 1);
    }
    return 0;
  };
  for (uint32_t units = 1; units < 200; units += 3)
    for (uint32_t groups = 1; groups <= 64; ++groups) CHECK(shares(units, groups) == 0);
  CHECK(shares(0x7fffffffu, 512) == 0 && shares(0x7ffffe00u, 511) == 0 && shares(0x7fffffffu, 65535) == 0);
  std::printf("ok\n");
  return 0;
}
