// attention.hip -- the attention kernel's launch, and the kernel that joins the
// parts of contexts that were split.
#include <algorithm>

#include "attention_rows.h"

namespace ringsim {

// A NaN counts as no maximum; it comes into the result through its sums.
struct MaxF32 {
  static __device__ __forceinline__ float of(float a, float b) { return fmaxf(a, b); }
};

static_assert(kGroups == 2 * kComputeUnits, "workgroups that share a call's work");

hipError_t launch_attention(const AttentionArgs& a, const AttentionPlan& plan, int dtype, hipStream_t s) {
  hipError_t e = hipErrorInvalidValue;
  switch (a.cache.dim) {
    case 64: e = launch_attention_64(a, plan, dtype, s); break;
    case 96: e = launch_attention_96(a, plan, dtype, s); break;
    case 128: e = launch_attention_128(a, plan, dtype, s); break;
    case 192: e = launch_attention_192(a, plan, dtype, s); break;
    case 256: e = launch_attention_256(a, plan, dtype, s); break;
    default: break;
  }
  if (e != hipSuccess || a.groups == 0) return e;
  return launch_attention_join(a, dtype, s);
}

// out = sum_s 2^(m_s - M) O_s / sum_s 2^(m_s - M) l_s over the parts s of a
// row's tile, M the largest m_s; tiles that one workgroup took whole are
// done. A wave takes a row: its lanes first hold the parts' m and l (64 of them
// at a time), then 4 columns each, so that no load waits for another one but
// the outputs for the weights. Heads of 128 columns and fewer leave half of
// the lanes for a second part: even ones go to the first half, odd ones to the
// second.
constexpr int kJoinRows = 4;   // of a workgroup at a time
constexpr int kJoinAhead = 8;  // outputs whose loads are under way

template <int DT, int HALVES>
__device__ __forceinline__ void join_row(const AttentionArgs& a, const RowTile& tile, int key_head, int in_tile,
                                         int first, int parts) {
  const int lane = threadIdx.x & 63, row = tile.row + in_tile;
  const int token = row / a.group, head = key_head * a.group + row - token * a.group;
  const int half = HALVES == 2 ? lane >> 5 : 0, col = (HALVES == 2 ? lane & 31 : lane) * 4;
  const float inf = __builtin_inff();
  const auto row_of = [&](int s) { return (int64_t)part_slot(first + s, s == 0) * a.tile_rows + in_tile; };
  const auto ml_of = [&](int s) {  // of no part: nothing
    const f32x4 v = *reinterpret_cast<const f32x4*>(a.part_ml + 4 * row_of(min(s, parts - 1)));
    return s < parts ? v : f32x4{-inf, 0.0f, 0.0f, 0.0f};
  };
  float best = -inf;
  for (int s = lane; s < parts; s += 64) best = fmaxf(best, ml_of(s)[0]);
  best = lanes_reduce<64, MaxF32>(best);
  float sum = 0.0f, exact = 0.0f, f[4] = {0.0f, 0.0f, 0.0f, 0.0f};
  const bool there = col < a.cache.dim;
  const float* out = a.part_out + (there ? col : 0);
  for (int base = 0; base < parts; base += 64) {
    const f32x4 ml = ml_of(base + lane);
    // A part without a position has written no output.
    const float w = ml[1] == 0.0f ? 0.0f : ml[0] == best ? 1.0f : __builtin_amdgcn_exp2f(ml[0] - best);
    sum += w * ml[1];
    exact += w * ml[2];
    const uint64_t used = __ballot(ml[1] != 0.0f);
    const int n = min(64, parts - base);
    for (int s0 = 0; s0 < n; s0 += kJoinAhead * HALVES) {
      f32x4 o[kJoinAhead];
#pragma unroll
      for (int k = 0; k < kJoinAhead; ++k) {
        const int s = s0 + HALVES * k + half;
        o[k] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
        if (s < n && (used >> (s & 63) & 1))
          o[k] = *reinterpret_cast<const f32x4*>(out + row_of(base + s) * a.cache.dim);
      }
#pragma unroll
      for (int k = 0; k < kJoinAhead; ++k) {
        const int s = s0 + HALVES * k + half;
        const float by = __shfl(w, s & 63);
#pragma unroll
        for (int i = 0; i < 4; ++i) f[i] += s < n ? o[k][i] * by : 0.0f;
      }
    }
  }
  sum = lanes_reduce<64, AddF32>(sum);
  exact = lanes_reduce<64, AddF32>(exact);
  if constexpr (HALVES == 2) {
#pragma unroll
    for (int i = 0; i < 4; ++i) f[i] += __shfl_xor(f[i], 32);
  }
  if (a.lse && lane == 0) a.lse[lse_index(a, tile, token, head)] = lse_of(best, exact);
  if (!there || half) return;
  const float by = sum == 0.0f ? 0.0f : 1.0f / sum;
#pragma unroll
  for (int i = 0; i < 4; ++i) f[i] *= by;
  Packed<DT, 4> y;
  y.set(f);
  y.store(out_row<DT>(a, tile, token, head) + col);
}

template <int DT, int HALVES>
__global__ __launch_bounds__(64 * kJoinRows) void attention_join_kernel(const AttentionArgs a) {
  const int item = blockIdx.x, tile_index = item / a.cache.heads, key_head = item - tile_index * a.cache.heads;
  RowTile tile;
  if (!row_tile(a, a.starts, tile_index, tile)) return;
  const int first = a.part_of[2 * item], parts = a.part_of[2 * item + 1] - first + 1;
  if (parts == 1) return;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int rows = min(a.tile_rows, tile.rows - tile.row);
  for (int row = blockIdx.y * kJoinRows + wave; row < rows; row += gridDim.y * kJoinRows)
    join_row<DT, HALVES>(a, tile, key_head, row, first, parts);
}

template <int DT>
static hipError_t launch_join(const AttentionArgs& a, hipStream_t s) {
  // Rows of a tile over some workgroups, as far as that fills the card.
  const int items = a.tiles * a.cache.heads;
  const int rows = a.starts ? a.tile_rows : std::min(a.tile_rows, a.each * a.group);
  const int blocks = std::min((rows + kJoinRows - 1) / kJoinRows, std::max(1, 16 * kComputeUnits / items));
  const dim3 grid((unsigned)items, (unsigned)blocks);
  const dim3 block(64 * kJoinRows);
  if (a.cache.dim <= 128)
    hipLaunchKernelGGL((attention_join_kernel<DT, 2>), grid, block, 0, s, a);
  else
    hipLaunchKernelGGL((attention_join_kernel<DT, 1>), grid, block, 0, s, a);
  return hipGetLastError();
}

hipError_t launch_attention_join(const AttentionArgs& a, int dtype, hipStream_t s) {
  switch (dtype) {
    case RINGSIM_FLOAT32: return launch_join<RINGSIM_FLOAT32>(a, s);
    case RINGSIM_BFLOAT16: return launch_join<RINGSIM_BFLOAT16>(a, s);
    case RINGSIM_FLOAT16: return launch_join<RINGSIM_FLOAT16>(a, s);
    default: return hipErrorInvalidValue;
  }
}

}  // namespace ringsim
