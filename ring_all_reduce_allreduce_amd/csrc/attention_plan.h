// attention_plan.h -- how an attention call is cut into workgroups. Plain
// functions of whole numbers, tested on the host.
#pragma once

#include <stdint.h>

#include <algorithm>

#include "../../include/ringsim_attention.h"
#include "kv_layout.h"

namespace ringsim {

// How a call is cut: rows of a tile, tiles, and workgroups that share them.
struct AttentionPlan {
  int wide;               // 1: many rows, a wave its own rows; 0: waves share rows
  int fine;               // of wide ones: 16-bit queries are split finely
  int tile_rows;
  int64_t tiles;
  int groups;             // 0: a workgroup a tile and key head
};

// Most tiles whose work is shared: their units are counted in LDS.
constexpr int kSharedTiles = 512;

// Tiles of 16 rows of a wave with rows of its own: two where a wave's registers
// hold them, else one (types whose products take several parts, long heads).
// Three prompts of 2048 tokens of 32 heads of 128: 163 us, with one 212.
constexpr int wide_tiles(int dtype, int dim, bool fine) {
  return dtype == RINGSIM_BFLOAT16 && dim <= 128 && !fine ? 2 : 1;
}

inline int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

constexpr int kNarrowRows = 16;

// Workgroups that share a call's work: as many as the card runs at once, two a
// CU. (64 sequences of 16384 with random pages of 64 positions take 212 us; with
// half as many 244, with twice as many 220. 512 tokens of 32 heads at the end of
// 32768: 324, 434 and 362.)
constexpr int kGroups = 512;

// A tile that many rows share, over `units` of 128 positions: a workgroup alone
// on its CU takes 3.2 us a unit; shares take 1 / 128 us a unit of all
// items, but 28 us and items / 14 to write the parts of tiles and to join them
// (bf16, heads of 128). 512 tokens of 32 heads at the end of 32768 positions:
// 319 us shared, 804 a workgroup a tile; two sequences of 256 at the end of 8192:
// 113 and 207; of 512 at the end of 4096: 118 and 111; three prompts of 2048: 254
// and 160.
inline bool wide_shares(int64_t items, int64_t units) { return (410 - items) * units > 3584 + 9 * items; }

// Few tiles of many rows, in contexts long enough to matter and too short for
// shares: waves that share 16 rows each are more workgroups. 8 sequences of 32
// tokens of 32 heads: 22 us against 16 over 512 positions, 35 against 21 over
// 1024, 61 against 29 over 2048, 50 against 45 over 4096 (33 units: left out,
// though the two meet behind it) and 68 against 76 over 8192; one of 128 tokens
// over 1024 34 against 18; 8 of 64 over 1024 36 both.
inline bool too_few(int64_t items, int64_t units) { return items < 128 && units > 4 && units <= 32; }

// Rows of 16 bits that see few positions, where lse is wanted: the coarse split's
// errors of the scores do not average out in it (1.2e-6 of it over 27 positions,
// 7e-7 over 128, single rows up to 3e-4 off; the fine split 4e-8 and 4e-6). bf16
// tiles are then half as long: two prompts of 2048 tokens of 32 heads of 128 with a
// window of 128 take 49 us for 37, 50 of 100 tokens 54 for 52.
inline bool fine_split(int dtype, int64_t positions, bool lse) {
  return lse && dtype != RINGSIM_FLOAT32 && positions <= kKvUnit;
}

// With few rows of a key head all waves of a workgroup take the same 16, which
// reads each tile of keys once for these alone; with many each wave has its own
// and values are converted once for all. 64 sequences of 2048 positions: 56 us
// against 64 with 32 rows, 150 against 84 with 96. (With 64 rows 105 against
// 81, but the weights in two parts.)
// `window`: 0 where positions are not bounded by it from both sides.
inline AttentionPlan plan_attention(int64_t tokens, int64_t seqs, bool ragged, int heads, int kv_heads, int dim,
                                    int dtype, int64_t cap, int64_t window, bool lse) {
  const int64_t group = heads / kv_heads, rows = tokens * group / seqs;  // of a sequence's key head, on average
  AttentionPlan p;
  p.fine = fine_split(dtype, window > 0 ? std::min(window, cap) : cap, lse);
  int64_t units, items;
  const auto cut = [&](bool wide) {
    p.wide = wide;
    p.tile_rows = wide ? 64 * wide_tiles(dtype, dim, p.fine) : kNarrowRows;
    p.tiles = ragged ? tokens * group / p.tile_rows + seqs : seqs * ceil_div(tokens / seqs * group, p.tile_rows);
    // Positions that a tile may see: all, or a window for each of its tokens.
    // The first unit may begin before the first of them.
    int64_t span = cap;
    if (window > 0 && window < cap) span = std::min(span, window + ceil_div(p.tile_rows, group) + 1);
    units = kv_units(kKvStep - 1, kKvStep - 2 + std::max<int64_t>(span, 1));
    items = p.tiles * kv_heads;
  };
  cut(rows > 64);
  if (p.wide && too_few(items, units)) cut(false);
  // Units are counted in 32 bits.
  const bool shares = (!p.wide || wide_shares(items, units)) && p.tiles <= kSharedTiles && units > 1 &&
                      items <= INT32_MAX / units;
  p.groups = shares ? (int)std::min<int64_t>(kGroups, ceil_div(items * units, 8) * 8) : 0;
  return p;
}

}  // namespace ringsim
