// kv_layout.h -- where the paged cache keeps a token, how a block's exponent
// is chosen, and which rows of queries a workgroup takes. Plain functions of
// whole numbers, used by the kernels and tested on the host.
#pragma once

#include <stdint.h>

#if defined(__HIPCC__)
#define KV_FN __host__ __device__ __forceinline__
#else
#define KV_FN inline
#endif

namespace ringsim {

constexpr int kKvBlock = 32;         // columns that share an exponent
constexpr int kKvNan = 255;          // exponent byte of 32 NaN
constexpr int kKvMinByte = 1;        // 2^-126, the smallest normal fp32
constexpr int kKvMaxByte = 252;      // 2^125: 6 times it is still finite
constexpr int kKvTile = 16;          // tokens of a matrix instruction's operand
constexpr int kKvStep = 32;          // tokens of one pass of the attention's loop

// Exponent byte of a block whose largest magnitude has the bits `top`: with
// 2^x <= max < 2^(x+1), the least e with max <= 7 * 2^e is x - 2 if the
// mantissa is at most 1.75 (7 = 1.75 * 4), else x - 1; the addition carries
// into the exponent exactly above 1.75.
KV_FN int kv_exponent_byte(uint32_t top) {
  if (top >= 0x7f800000u) return kKvNan;
  const int b = (int)((top + 0x1fffffu) >> 23) - 2;
  return b < kKvMinByte ? kKvMinByte : b > kKvMaxByte ? kKvMaxByte : b;
}

// Whether a slot lies in the cache; its page and token there.
KV_FN bool kv_slot(int64_t slot, int64_t pages, int page_shift, int32_t* page, int* token) {
  if (slot < 0 || (slot >> page_shift) >= pages) return false;
  *page = (int32_t)(slot >> page_shift);
  *token = (int)(slot & ((1 << page_shift) - 1));
  return true;
}

// Place of a sequence's tile of kKvTile tokens in its row of the table, kept
// inside the row, which holds at least one; false where the tile has none: past
// the sequence or past the row.
KV_FN bool kv_place_of_tile(int64_t tile, int64_t end, int page_shift, int64_t max_pages, int64_t* place) {
  const int64_t at = tile * kKvTile >> page_shift;
  *place = at < 0 ? 0 : at < max_pages ? at : max_pages - 1;
  return tile >= 0 && tile * kKvTile < end && at < max_pages;
}
// Whether a number of the table is a page.
KV_FN bool kv_is_page(int32_t id, int64_t pages) { return id >= 0 && id < pages; }

// Rows of queries. Sequence b has (starts[b+1] - starts[b]) * group rows of a
// key head, which are cut into tiles of `rows`; its tiles are numbered from
// kv_first_tile(starts[b], ...). ceil(n / rows) <= floor((a + n) / rows) -
// floor(a / rows) + 1, so that no two sequences share a number, and all
// numbers lie below tokens * group / rows + seqs.
KV_FN int64_t kv_first_tile(int64_t start, int64_t b, int64_t group, int64_t rows) { return start * group / rows + b; }

KV_FN int64_t kv_clamp(int64_t v, int64_t lo, int64_t hi) { return v < lo ? lo : v > hi ? hi : v; }

// The sequence whose tiles hold number `tile`: the last b with first(b) <= tile.
KV_FN int64_t kv_seq_of_tile(const int32_t* starts, int64_t seqs, int64_t tokens, int64_t group, int64_t rows,
                             int64_t tile) {
  int64_t lo = 0, hi = seqs - 1;
  while (lo < hi) {
    const int64_t mid = (lo + hi + 1) >> 1;
    if (kv_first_tile(kv_clamp(starts[mid], 0, tokens), mid, group, rows) <= tile)
      lo = mid;
    else
      hi = mid - 1;
  }
  return lo;
}

// Positions [*lo, *hi] that the token at position p sees, of `end` positions. A
// window may be any number: it is only subtracted where the result is one of p's.
KV_FN void kv_span(int64_t p, int64_t end, int causal, int64_t window, int64_t* lo, int64_t* hi) {
  *hi = causal && p < end - 1 ? p : end - 1;
  *lo = window > 0 && p >= window ? p - window + 1 : 0;
}

// Shares of the work. A tile of rows that sees positions lo to hi has units of
// kKvUnit positions, at least one (rows that see nothing are written too). All
// units of all tiles and key heads stand in one line, key heads outermost,
// which is cut into equal shares, one for each workgroup.
constexpr int kKvUnit = 128;
KV_FN int64_t kv_units(int64_t lo, int64_t hi) {
  return hi < lo ? 1 : (hi - lo / kKvStep * kKvStep) / kKvUnit + 1;
}
// Shares of units / groups each, some with one more, spread over the groups; up to 2^16 groups.
KV_FN uint32_t kv_share_begin(uint32_t units, uint32_t group, uint32_t groups) {
  const uint32_t each = units / groups, more = units - each * groups;
  return group * each + group * more / groups;
}

}  // namespace ringsim
