// attention_rows.h -- which rows and positions a tile of queries has, and
// where its results go: what the attention kernel and its join share.
#pragma once

#include "attention_device.h"

namespace ringsim {

// A tile's rows: sequence, its first token in q and that one's position, its
// rows, the first of them here, and its positions.
struct RowTile {
  int seq, token, first, rows, row, length;
};

// False: no rows. `starts`: a.starts or a copy of it.
__device__ __forceinline__ bool row_tile(const AttentionArgs& a, const int32_t* starts, int tile, RowTile& t) {
  int count;
  if (a.starts) {
    t.seq = (int)kv_seq_of_tile(starts, a.seqs, a.tokens, a.group, a.tile_rows, tile);
    t.token = (int)kv_clamp(starts[t.seq], 0, a.tokens);
    count = (int)kv_clamp(starts[t.seq + 1], 0, a.tokens) - t.token;
    tile -= (int)kv_first_tile(t.token, t.seq, a.group, a.tile_rows);
  } else {
    t.seq = tile / a.seq_tiles;
    t.token = t.seq * a.each;
    count = a.each;
    tile -= t.seq * a.seq_tiles;
  }
  t.row = tile * a.tile_rows;
  t.rows = count * a.group;
  if (tile < 0 || t.row >= t.rows) return false;
  const int n = max(a.lengths[t.seq], 0);
  t.length = min(n, a.cap);
  t.first = n - count;
  return true;
}

// The same tile, told to be the same for all lanes of a wave.
__device__ __forceinline__ RowTile same_tile(const RowTile& t) {
  return RowTile{__builtin_amdgcn_readfirstlane(t.seq),   __builtin_amdgcn_readfirstlane(t.token),
                 __builtin_amdgcn_readfirstlane(t.first), __builtin_amdgcn_readfirstlane(t.rows),
                 __builtin_amdgcn_readfirstlane(t.row),   __builtin_amdgcn_readfirstlane(t.length)};
}

// The tile that lane `i` holds.
__device__ __forceinline__ RowTile tile_of_lane(const RowTile& t, int i) {
  return RowTile{__builtin_amdgcn_readlane(t.seq, i),  __builtin_amdgcn_readlane(t.token, i),
                 __builtin_amdgcn_readlane(t.first, i), __builtin_amdgcn_readlane(t.rows, i),
                 __builtin_amdgcn_readlane(t.row, i),  __builtin_amdgcn_readlane(t.length, i)};
}

// Positions [lo, hi] that the token at position p sees.
__device__ __forceinline__ void span(const AttentionArgs& a, int p, int length, int* lo, int* hi) {
  int64_t l, h;
  kv_span(p, length, a.causal, a.window, &l, &h);
  *lo = (int)l;
  *hi = (int)h;
}

// Positions that any row of the tile sees; of none [0, -1], so that sums with
// the first of them stay below kMaxPositions.
__device__ __forceinline__ void tile_span(const AttentionArgs& a, const RowTile& t, int* lo, int* hi) {
  const int last = min(t.row + a.tile_rows, t.rows) - 1;
  int x;
  span(a, t.first + t.row / a.group, t.length, lo, &x);
  span(a, t.first + last / a.group, t.length, &x, hi);
  if (*hi < *lo) {
    *lo = 0;
    *hi = -1;
  }
}

__device__ __forceinline__ int64_t lse_index(const AttentionArgs& a, const RowTile& t, int token, int head) {
  return (int64_t)(t.token + token) * a.heads + head;
}
template <int DT>
__device__ __forceinline__ typename OpElem<DT>::T* out_row(const AttentionArgs& a, const RowTile& t, int token,
                                                           int head) {
  const int64_t at = a.starts ? (t.token + token) * a.out.s1 : t.seq * a.out.s0 + token * a.out.s1;
  return static_cast<typename OpElem<DT>::T*>(a.out.p) + at + head * a.out.s2;
}
template <int DT>
__device__ __forceinline__ const typename OpElem<DT>::T* query_row(const AttentionArgs& a, const RowTile& t, int token,
                                                                   int head) {
  const int64_t at = a.starts ? (t.token + token) * a.q.s1 : t.seq * a.q.s0 + token * a.q.s1;
  return static_cast<const typename OpElem<DT>::T*>(a.q.p) + at + head * a.q.s2;
}

// Of a sum of weights over 2^ref.
__device__ __forceinline__ float lse_of(float ref, float sum) {
  return sum == 0.0f ? -__builtin_inff() : (ref + __builtin_amdgcn_logf(sum)) * 0.69314718055994531f;
}

}  // namespace ringsim
