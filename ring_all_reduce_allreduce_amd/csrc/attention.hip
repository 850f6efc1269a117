// attention.hip -- how an attention call is cut into workgroups, and the
// kernel that joins the parts of contexts that were split.
#include <algorithm>

#include "attention_device.h"

#ifndef RINGSIM_TARGET
#define RINGSIM_TARGET 2048
#define RINGSIM_LEAST 256
#endif

namespace ringsim {

// A NaN counts as no maximum; it comes into the result through its sums.
struct MaxF32 {
  static __device__ __forceinline__ float of(float a, float b) { return fmaxf(a, b); }
};

namespace {

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// Rows of a workgroup whose waves have their own rows, by type: two tiles of
// 16 a wave for bf16, one for the types whose products take several parts.
int wide_rows(int dtype) { return dtype == RINGSIM_BFLOAT16 ? 128 : 64; }
constexpr int kNarrowRows = 16;

}  // namespace

AttentionPlan plan_attention(int64_t tokens, int64_t seqs, bool ragged, int heads, int kv_heads, int dim, int dtype,
                             int64_t cap, int64_t window) {
  AttentionPlan p;
  const int64_t group = heads / kv_heads, rows = tokens * group / seqs;  // of a sequence's key head, on average
  p.wide = rows > 64;
  p.tile_rows = p.wide ? wide_rows(dtype) : kNarrowRows;
  p.tiles = ragged ? tokens * group / p.tile_rows + seqs : seqs * ceil_div(tokens / seqs * group, p.tile_rows);
  // Positions that a workgroup may see: all, or a window for each of its tokens.
  int64_t span = cap;
  if (window > 0) span = std::min(span, window + ceil_div(p.tile_rows, group) + 1);
  span += kKvStep;  // the first pass may begin before the first position
  const int64_t groups = p.tiles * kv_heads, target = p.wide ? 512 : RINGSIM_TARGET, least = p.wide ? 1024 : RINGSIM_LEAST;
  const int64_t splits = std::max<int64_t>(1, std::min(ceil_div(target, std::max<int64_t>(groups, 1)), span / least));
  p.chunk = ceil_div(ceil_div(span, splits), kKvStep) * kKvStep;
  p.splits = (int)ceil_div(span, p.chunk);
  return p;
}

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
  if (e != hipSuccess || a.splits == 1) return e;
  return launch_attention_join(a, dtype, s);
}

// out = sum_s 2^(m_s - M) O_s / sum_s 2^(m_s - M) l_s with M the largest m_s. A
// wave takes a row: its lanes first hold the splits' m and l (64 of them at a
// time), then 4 columns each, so that no load waits for another one but the
// outputs for the weights. Heads of 128 columns and fewer leave half of the lanes for
// a second split: even splits go to the first half, odd ones to the second.
constexpr int kJoinRows = 4;     // of a workgroup
constexpr int kJoinAhead = 8;    // outputs whose loads are under way

template <int DT, int HALVES>
__global__ __launch_bounds__(64 * kJoinRows) void attention_join_kernel(const AttentionArgs a) {
  const int64_t all = (int64_t)a.tokens * a.heads;
  const int64_t at = (int64_t)blockIdx.x * kJoinRows + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  if (at >= all) return;
  const int token = (int)(at / a.heads), head = (int)(at - (int64_t)token * a.heads), lane = threadIdx.x & 63;
  const int half = HALVES == 2 ? lane >> 5 : 0, col = (HALVES == 2 ? lane & 31 : lane) * 4;
  int seq = 0;
  if (a.starts) {
    if (token < a.starts[0] || token >= a.starts[a.seqs]) return;  // of no sequence
  } else {
    seq = token / a.each;
  }
  const float inf = __builtin_inff();
  const auto ml_of = [&](int s) {  // of no split: nothing
    const f32x2 v = *reinterpret_cast<const f32x2*>(a.part_ml + 2 * (min(s, a.splits - 1) * all + at));
    return s < a.splits ? v : f32x2{-inf, 0.0f};
  };
  float best = -inf;
  for (int s = lane; s < a.splits; s += 64) best = fmaxf(best, ml_of(s).x);
  best = lanes_reduce<64, MaxF32>(best);
  float sum = 0.0f, f[4] = {0.0f, 0.0f, 0.0f, 0.0f};
  const bool there = col < a.cache.dim;
  const float* part = a.part_out + at * a.cache.dim + (there ? col : 0);
  for (int base = 0; base < a.splits; base += 64) {
    const f32x2 ml = ml_of(base + lane);
    // A split without a position has written no output.
    float w = ml.y == 0.0f ? 0.0f : ml.x == best ? 1.0f : __builtin_amdgcn_exp2f(ml.x - best);
    sum += w * ml.y;
    const uint64_t used = __ballot(ml.y != 0.0f);
    const int n = min(64, a.splits - base);
    for (int s0 = 0; s0 < n; s0 += kJoinAhead * HALVES) {
      f32x4 o[kJoinAhead];
#pragma unroll
      for (int k = 0; k < kJoinAhead; ++k) {
        const int s = s0 + HALVES * k + half;
        const bool on = s < n && (used >> (s & 63) & 1);
        o[k] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
        if (on) o[k] = *reinterpret_cast<const f32x4*>(part + (int64_t)(base + s) * all * a.cache.dim);
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
  if constexpr (HALVES == 2) {
#pragma unroll
    for (int i = 0; i < 4; ++i) f[i] += __shfl_xor(f[i], 32);
  }
  constexpr float kLn2 = 0.69314718055994531f;
  if (a.lse && lane == 0) a.lse[at] = sum == 0.0f ? -inf : (best + __builtin_amdgcn_logf(sum)) * kLn2;
  if (!there || half) return;
  const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
#pragma unroll
  for (int i = 0; i < 4; ++i) f[i] *= inv;
  const int64_t to = a.starts ? token * a.out.s1 : seq * a.out.s0 + (token - seq * a.each) * a.out.s1;
  Packed<DT, 4> y;
  y.set(f);
  y.store(static_cast<typename OpElem<DT>::T*>(a.out.p) + to + head * a.out.s2 + col);
}

template <int DT>
static hipError_t launch_join(const AttentionArgs& a, hipStream_t s) {
  const int64_t rows = (int64_t)a.tokens * a.heads;
  const dim3 grid((unsigned)ceil_div(rows, kJoinRows)), block(64 * kJoinRows);
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
