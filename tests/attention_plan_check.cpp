// Host check of attention_plan.h: which kernel the calls of the GPU tests and of
// the design's table take, so that a change of the rules cannot take a kernel
// out of the tests unseen; and that wanting lse changes no workspace. Prints
// "ok" or the first thing that is wrong.
#include <cstdio>

#include "attention_plan.h"

using namespace ringsim;

#define CHECK(x)                                              \
  do {                                                        \
    if (!(x)) {                                               \
      std::printf("line %d: %s\n", __LINE__, #x);             \
      return 1;                                               \
    }                                                         \
  } while (0)

enum { F32 = RINGSIM_FLOAT32, BF16 = RINGSIM_BFLOAT16, F16 = RINGSIM_FLOAT16 };

// n: waves share 16 rows; w: rows of their own; f: those with the fine split in 16 bits; s behind it: shared contexts.
static const char* kernel(const AttentionPlan& p, int dtype) {
  const bool fine = p.wide && p.fine && dtype != F32;
  return !p.wide ? (p.groups ? "ns" : "n") : fine ? (p.groups ? "fs" : "f") : p.groups ? "ws" : "w";
}

struct Call {
  int64_t tokens, seqs;
  bool ragged;
  int heads, kv_heads, dim, dtype;
  int64_t cap, window;
  const char *plain, *lse;  // the kernel without and with lse
};

int main() {
  const Call calls[] = {
      // single and some tokens: shared where a context is longer than a unit, up to 512 tiles
      {1, 1, false, 32, 8, 128, BF16, 4096, 0, "ns", "ns"},
      {64, 64, false, 32, 8, 128, BF16, 16384, 0, "ns", "ns"},
      {64, 64, false, 32, 8, 128, BF16, 64, 0, "n", "n"},
      {600, 600, false, 32, 8, 128, F16, 16384, 0, "n", "n"},
      {23 * 5, 23, true, 7, 7, 64, F16, 2999, 1500, "ns", "ns"},
      // prompts, and the last tokens of long documents
      {3 * 2048, 3, true, 32, 8, 128, BF16, 6000, 0, "w", "w"},
      {512, 1, false, 32, 8, 128, BF16, 32768, 0, "ws", "ws"},
      {2 * 2048, 2, false, 32, 8, 128, F32, 2048, 0, "w", "w"},
      // few tiles over contexts of middling length: tiles of 16 rows
      {128, 1, false, 8, 8, 128, BF16, 1024, 0, "ns", "ns"},
      {100, 1, true, 1, 1, 64, BF16, 6000, 3000, "ns", "ns"},
      // windows: 128 positions are few, 129 are not
      {6 * 1774, 6, true, 16, 16, 128, BF16, 1774, 27, "w", "f"},
      {6 * 1774, 6, true, 16, 16, 128, F16, 1774, 128, "w", "f"},
      {6 * 1774, 6, true, 16, 16, 128, BF16, 1774, 129, "w", "w"},
      {6 * 1774, 6, true, 16, 16, 128, F32, 1774, 27, "w", "w"},
      {100, 1, true, 2, 2, 192, F16, 1 << 20, 33, "w", "f"},
      // short contexts
      {50 * 100, 50, false, 32, 8, 128, BF16, 128, 0, "w", "f"},
      {50 * 100, 50, false, 32, 8, 128, BF16, 129, 0, "w", "w"},
      {50 * 100, 50, false, 32, 8, 128, BF16, 128, 500, "w", "f"},
      // test_gpu_attention_wide.py (with both ways a window bounds no span), test_gpu_attention_unseen.py
      {127, 2, true, 2, 1, 128, BF16, 336, 27, "w", "f"},
      {127, 2, true, 2, 1, 64, F16, 336, 300, "w", "w"},
      {91, 3, true, 4, 1, 96, F16, 384, 128, "w", "f"},
      {91, 3, true, 4, 1, 256, BF16, 384, 200, "w", "w"},
      {57, 2, true, 5, 1, 64, BF16, 208, 0, "w", "w"},
      {230, 2, true, 4, 2, 128, F16, 272, 150, "w", "w"},
      {100, 1, false, 1, 1, 64, BF16, RINGSIM_ATTENTION_MAX_LENGTH, 250, "w", "w"},
      {100, 1, false, 1, 1, 64, F16, RINGSIM_ATTENTION_MAX_LENGTH, 100, "w", "f"},
      {250, 2, true, 2, 1, 64, BF16, 336, 140, "w", "w"},
      {141, 2, true, 2, 1, 192, F16, 4512, 0, "ws", "ws"},
  };
  for (const Call& c : calls) {
    for (const bool lse : {false, true}) {
      const AttentionPlan p =
          plan_attention(c.tokens, c.seqs, c.ragged, c.heads, c.kv_heads, c.dim, c.dtype, c.cap, c.window, lse);
      const char *got = kernel(p, c.dtype), *want = lse ? c.lse : c.plain;
      if (got[0] != want[0] || got[1] != want[1]) {
        std::printf("call %d, lse %d: %s, not %s\n", (int)(&c - calls), (int)lse, got, want);
        return 1;
      }
      CHECK(p.tile_rows == (!p.wide ? 16 : 64 * wide_tiles(c.dtype, c.dim, p.fine)));
    }
  }

  // Over all sizes: the same rows fit, and the workspace, which the caller may have asked for without lse, stays the same.
  uint32_t seed = 7;
  const auto next = [&](uint32_t n) { return (int64_t)((seed = seed * 1664525u + 1013904223u) >> 8) % n; };
  for (int turn = 0; turn < 200000; ++turn) {
    const int64_t seqs = 1 + next(next(2) ? 8 : 700), each = 1 + next(next(2) ? 8 : 2500), cap = 1 + next(1 << next(20));
    const int64_t window = next(2) ? 0 : 1 + next(1 << next(20));
    const int kv_heads = 1 + (int)next(8), group = 1 + (int)next(16), dims[] = {64, 96, 128, 192, 256};
    const int dim = dims[next(5)], types[] = {F32, BF16, F16}, dtype = types[next(3)];
    const bool ragged = next(2);
    const AttentionPlan a =
        plan_attention(seqs * each, seqs, ragged, kv_heads * group, kv_heads, dim, dtype, cap, window, false);
    const AttentionPlan b =
        plan_attention(seqs * each, seqs, ragged, kv_heads * group, kv_heads, dim, dtype, cap, window, true);
    CHECK(a.groups == b.groups && a.wide == b.wide);
    if (a.groups) CHECK(a.tile_rows == b.tile_rows && a.tiles == b.tiles && a.tiles <= kSharedTiles);
    for (const AttentionPlan& p : {a, b}) {
      CHECK(p.tiles * p.tile_rows >= seqs * each * group && p.groups % 8 == 0 && p.groups <= kGroups);
      CHECK(p.wide == (each * group > 64) || !p.wide);
    }
  }
  std::printf("ok\n");
  return 0;
}
