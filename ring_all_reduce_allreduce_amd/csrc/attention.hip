// attention.hip -- how an attention call is cut into workgroups, and the
// kernel that joins the parts of contexts that were split.
#include <algorithm>

#include "attention_device.h"

namespace ringsim {

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
  const int64_t groups = p.tiles * kv_heads, target = p.wide ? 512 : 2048, least = p.wide ? 1024 : 256;
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

// out = sum_s 2^(m_s - M) O_s / sum_s 2^(m_s - M) l_s with M the largest m_s,
// splits in order. LANES lanes a row, 4 columns each.
template <int DT, int LANES>
__global__ __launch_bounds__(256) void attention_join_kernel(const AttentionArgs a) {
  const int64_t all = (int64_t)a.tokens * a.heads;
  const int64_t at = (int64_t)blockIdx.x * (256 / LANES) + threadIdx.x / LANES;
  if (at >= all) return;
  const int64_t token = at / a.heads;
  const int head = (int)(at - token * a.heads), col = (int)(threadIdx.x % LANES) * 4;
  int64_t seq = 0;
  if (a.starts) {
    if (token < a.starts[0] || token >= a.starts[a.seqs]) return;  // of no sequence
  } else {
    seq = token / a.each;
  }
  float best = -__builtin_inff();
  for (int s = 0; s < a.splits; ++s) best = fmaxf(best, a.part_ml[2 * (s * all + at)]);
  float sum = 0.0f, f[4] = {0.0f, 0.0f, 0.0f, 0.0f};
  for (int s = 0; s < a.splits; ++s) {
    const float ref = a.part_ml[2 * (s * all + at)], l = a.part_ml[2 * (s * all + at) + 1];
    if (l == 0.0f) continue;  // no position there, nothing written
    const float by = ref == best ? 1.0f : __builtin_amdgcn_exp2f(ref - best);
    sum += l * by;
    if (col < a.cache.dim) {
      const f32x4 o = *reinterpret_cast<const f32x4*>(a.part_out + (s * all + at) * a.cache.dim + col);
#pragma unroll
      for (int i = 0; i < 4; ++i) f[i] += o[i] * by;
    }
  }
  constexpr float kLn2 = 0.69314718055994531f;
  if (a.lse && col == 0) a.lse[at] = sum == 0.0f ? -__builtin_inff() : (best + __builtin_amdgcn_logf(sum)) * kLn2;
  if (col >= a.cache.dim) return;
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
  if (a.cache.dim <= 128)
    hipLaunchKernelGGL((attention_join_kernel<DT, 32>), dim3((unsigned)ceil_div(rows, 8)), dim3(256), 0, s, a);
  else
    hipLaunchKernelGGL((attention_join_kernel<DT, 64>), dim3((unsigned)ceil_div(rows, 4)), dim3(256), 0, s, a);
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
