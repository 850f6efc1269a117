// attention_internal.h -- kernel arguments and launch rules of the
// attention-step operators.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "attention_plan.h"
#include "ops_internal.h"

namespace ringsim {

// Whole-number division by a value known at launch: n / d for n below 2^31 is
// (n * mul) >> (32 + shift), with mul rounded up from 2^(32 + shift) / d and
// 2^shift the least power of two that is not below d.
struct FastDiv {
  uint32_t d, mul, shift;
};
inline FastDiv fast_div(uint32_t d) {
  uint32_t shift = 0;
  while ((1ull << shift) < d) ++shift;
  return FastDiv{d, (uint32_t)((((1ull << shift) - d) << 32) / d + 1), shift};
}
__host__ __device__ __forceinline__ uint32_t divide(uint32_t n, const FastDiv& f) {
  const uint32_t t = (uint32_t)(((uint64_t)n * f.mul) >> 32);
  return (uint32_t)(((uint64_t)t + n) >> f.shift);
}

// Whole numbers of either width in device memory, [outer, inner].
struct Index {
  const void* p;
  int64_t s0, s1;
  int wide;  // 64 bits
};

// [outer, inner, heads, dim]
struct HeadRows {
  const void* p;
  int64_t s0, s1, s2;
};
struct HeadRowsOut {
  void* p;
  int64_t s0, s1, s2;
};

struct RotaryArgs {
  HeadRows x;
  HeadRowsOut out;
  Index positions;
  const double* frequencies;
  uint32_t tokens, inner, heads;
  int dim, pairs;
  int packs;        // items of a head
  int turned;       // of them, those that hold pairs; the others copy
  int block_tokens; // of a workgroup
  int block_heads;
  uint32_t blocks;  // of tokens
  FastDiv by_packs, by_heads, by_pairs;
  int interleaved;
  float sign, scale;
};
hipError_t launch_rotary(RotaryArgs a, int dtype, hipStream_t s);

struct KvCacheArgs {
  uint8_t* data[2];    // keys, values
  uint8_t* scales[2];
  int64_t page, head;  // strides in bytes
  int64_t scale_page, scale_head;
  int32_t pages;
  int heads, dim, page_shift;
};

struct KvAppendArgs {
  KvCacheArgs cache;
  HeadRows x[2];       // keys, values
  Index slots, positions;
  const double* frequencies;
  uint32_t tokens, inner;
  int pairs, interleaved;
  float scale;
  int block_tokens, block_heads;
  uint32_t blocks;     // of tokens
  FastDiv by_packs, by_tokens, by_pairs;
};
hipError_t launch_kv_append(KvAppendArgs a, int dtype, hipStream_t s);

struct KvReadArgs {
  KvCacheArgs cache;
  HeadRowsOut out[2];  // p null: not wanted
  Index slots;
  uint32_t tokens, inner;
  FastDiv by_packs, by_heads;
};
hipError_t launch_kv_read(KvReadArgs a, int dtype, hipStream_t s);

struct AttentionArgs {
  KvCacheArgs cache;
  HeadRows q;          // {sequence, token, head}
  HeadRowsOut out;
  float* lse;
  const int32_t* pages;
  const int32_t* lengths;
  const int32_t* starts;  // null: `each` tokens a sequence
  // Shared work (groups > 0): workgroups take equal shares of all units, and
  // leave what they hold of a tile that others hold parts of in a slot of theirs.
  float* part_out;        // [2 * groups, tile_rows, dim]
  float* part_ml;         // [2 * groups, tile_rows, 4]: reference exponent, sum, sum of unrounded weights
  int32_t* part_of;       // [tiles * key heads, 2]: first and last workgroup of a tile
  int64_t page_stride;
  int64_t max_pages;
  int64_t window;
  int cap;                // positions that a sequence can have
  int tokens, seqs;
  int each;               // tokens of a sequence without starts, and
  int seq_tiles;          // tiles of its rows
  int groups;             // workgroups that share the work; 0: a workgroup a tile and key head
  int group;              // query heads of a key head
  int heads;              // of queries
  int tiles;              // of rows, over all sequences
  int tile_rows;
  int causal;
  float scale_log2;       // scale * log2(e) * 2^kQueryExponent
};

// Queries go into the first product divided by this power of two, which the
// scale takes back: the largest queries have products with a cache's usual
// values that fp32 would not hold.
constexpr int kQueryExponent = 8;

// Most positions of a sequence: with the passes that waves and their loads are
// ahead of each other, they are counted in 32 bits.
constexpr int kMaxPositions = RINGSIM_ATTENTION_MAX_LENGTH;
// Where a workgroup leaves its part of a tile: the one that it begins but does
// not end last in its share, one that it only goes on with first.
__host__ __device__ __forceinline__ int part_slot(int group, bool begins) { return 2 * group + (begins ? 1 : 0); }

hipError_t launch_attention(const AttentionArgs& a, const AttentionPlan& plan, int dtype, hipStream_t s);
// One unit for each head size, so that they compile side by side.
hipError_t launch_attention_64(const AttentionArgs&, const AttentionPlan&, int, hipStream_t);
hipError_t launch_attention_96(const AttentionArgs&, const AttentionPlan&, int, hipStream_t);
hipError_t launch_attention_128(const AttentionArgs&, const AttentionPlan&, int, hipStream_t);
hipError_t launch_attention_192(const AttentionArgs&, const AttentionPlan&, int, hipStream_t);
hipError_t launch_attention_256(const AttentionArgs&, const AttentionPlan&, int, hipStream_t);
hipError_t launch_attention_join(const AttentionArgs& a, int dtype, hipStream_t s);

}  // namespace ringsim
