// rotary.hip -- rotary positions of queries and keys, and their gradient.
//
// Pair i of a head at position p is turned by p * frequency[i]:
//     a' = scale * (a cos - b sin),  b' = scale * (b cos + a sin)
// and back for the gradient, since the transposed rotation is the one by the
// opposite angle. What bounds it is memory, an element in and an element out
// against 3 operations. A workgroup takes some tokens with all or some of
// their heads: its threads first form the cosines and sines of those tokens
// once, in LDS, then walk over heads and packs. Without a table in memory
// there is nothing more to read than positions and frequencies, and no
// longest position.
#include <algorithm>

#include "attention_device.h"

namespace ringsim {

constexpr int kRotaryThreads = 256;
constexpr int kRotaryTable = 1024;  // most pairs of a workgroup's tokens: 8 KiB, or one token's
// Items of a thread: two where an item is one pack, else one, so two packs. More
// of them leave fewer workgroups to be under way: 8192 tokens of 40 heads of
// 128 take 27.6 us with one item (halves), 28.5 with two and 30.0 with four;
// 20000 tokens of 9 heads of 100 fp32 (neighbours) 31.6, 29.6 and 36.9.
template <bool NEXT>
constexpr int kRotaryAhead = NEXT ? 2 : 1;

// An item is a pack of N columns: one of each half, or N / 2 neighbouring
// pairs, or columns that are copied (one by one where there are less than N).
// A pack that would pass the end of its part starts N before it: the columns
// that it shares with the pack before get the same values from both. Packs need
// the alignment of an element only.
template <int DT, int N, bool NEXT>
__global__ __launch_bounds__(kRotaryThreads) void rotary_kernel(const RotaryArgs a) {
  extern __shared__ float2 turn[];  // {cos, sin} * scale of [token, pair]
  using T = typename OpElem<DT>::T;
  const uint32_t head0 = blockIdx.y * a.block_heads;
  const int span = NEXT ? 2 * a.pairs : a.pairs, rest = a.dim - 2 * a.pairs;
  struct Item {
    const T* x;
    uint32_t t, head;
    int kind, c;  // 0 nothing, 1 turned, 2 copied, 3 one column copied; first column
    Packed<DT, N> u, v;
  } item[kRotaryAhead<NEXT>];
  for (uint32_t block = blockIdx.x; block < a.blocks; block += gridDim.x) {
    const uint32_t token0 = block * a.block_tokens;
    const uint32_t tokens = min((uint32_t)a.block_tokens, a.tokens - token0);
    const uint32_t items = tokens * a.block_heads * a.packs;
    for (uint32_t base = 0; base < items; base += kRotaryThreads * kRotaryAhead<NEXT>) {
      // All loads, the first ones before the angles are formed.
#pragma unroll
      for (int k = 0; k < kRotaryAhead<NEXT>; ++k) {
        const uint32_t n = base + k * kRotaryThreads + threadIdx.x;
        const uint32_t row = divide(n, a.by_packs);
        const int p = (int)(n - row * a.packs);
        Item& e = item[k];
        e.t = divide(row, a.by_heads);
        e.head = head0 + row - e.t * a.block_heads;
        e.kind = 0;
        if (n >= items || e.head >= a.heads) continue;
        e.x = head_ptr<DT>(a.x, token_at(token0 + e.t, a.inner), e.head);
        if (p < a.turned) {
          e.kind = 1;
          e.c = min(p * N, span - N);
          e.u.load(e.x + e.c);
          if constexpr (!NEXT) e.v.load(e.x + a.pairs + e.c);
        } else if (rest >= N) {
          e.kind = 2;
          e.c = 2 * a.pairs + min((p - a.turned) * N, rest - N);
          e.u.load(e.x + e.c);
        } else {
          e.kind = 3;
          e.c = 2 * a.pairs + p - a.turned;
          e.u.w[0] = e.x[e.c];
        }
      }
      if (base == 0) {
        if (block != blockIdx.x) __syncthreads();  // the last block's angles have been read
        for (uint32_t k = threadIdx.x; k < tokens * a.pairs; k += kRotaryThreads) {
          const uint32_t t = divide(k, a.by_pairs), i = k - t * a.pairs;
          const TokenAt at = token_at(token0 + t, a.inner);
          float s, c;
          // Rounded to fp32 here, as the rotation is: 2^-25 half turns at most, 9e-8 of a
          // radian beside the cosine's and the sine's own roundings of 3e-8.
          sincospif((float)half_turns(read_index(a.positions, at.o, at.i), a.frequencies[i]), &s, &c);
          turn[k] = float2{c * a.scale, s * a.sign * a.scale};
        }
        __syncthreads();
      }
#pragma unroll
      for (int k = 0; k < kRotaryAhead<NEXT>; ++k) {
        Item& e = item[k];
        if (e.kind == 0) continue;
        T* y = head_ptr<DT>(a.out, token_at(token0 + e.t, a.inner), e.head) + e.c;
        if (e.kind == 3) {
          *y = (T)e.u.w[0];
        } else if (e.kind == 2) {
          e.u.store(y);
        } else if constexpr (NEXT) {
          const float2* cs = turn + e.t * a.pairs + e.c / 2;
          float f[N];
#pragma unroll
          for (int i = 0; i < N / 2; ++i) {
            const float p = e.u.get(2 * i), q = e.u.get(2 * i + 1), c = cs[i].x, s = cs[i].y;
            f[2 * i] = __builtin_fmaf(p, c, -(q * s));
            f[2 * i + 1] = __builtin_fmaf(q, c, p * s);
          }
          e.u.set(f);
          e.u.store(y);
        } else {
          const float2* cs = turn + e.t * a.pairs + e.c;
          float f[N], g[N];
#pragma unroll
          for (int i = 0; i < N; ++i) {
            const float p = e.u.get(i), q = e.v.get(i), c = cs[i].x, s = cs[i].y;
            f[i] = __builtin_fmaf(p, c, -(q * s));
            g[i] = __builtin_fmaf(q, c, p * s);
          }
          e.u.set(f);
          e.v.set(g);
          e.u.store(y);
          e.v.store(y + a.pairs);
        }
      }
    }
  }
}

template <int DT, int N, bool NEXT>
static hipError_t launch_packed(RotaryArgs a, hipStream_t s) {
  const auto packs_of = [](int columns) { return (columns + N - 1) / N; };
  const int rest = a.x.p == a.out.p ? 0 : a.dim - 2 * a.pairs;  // in place, what is not turned stays
  a.turned = packs_of(NEXT ? 2 * a.pairs : a.pairs);
  a.packs = a.turned + (rest >= N ? packs_of(rest) : rest);
  if (a.packs == 0) return hipSuccess;
  // A thread's loads all at once, and the angles shared by as many heads as
  // there are; heads are cut where tokens are few (256 tokens of 40 heads of 128:
  // 3.9 us, else 4.2), or a token's are many.
  constexpr int kItems = kRotaryThreads * kRotaryAhead<NEXT>;
  const int64_t row = (int64_t)a.heads * a.packs;
  a.block_heads = (int)a.heads;
  a.block_tokens = (int)std::max<int64_t>(1, std::min<int64_t>(kItems / std::max<int64_t>(row, 1), a.tokens));
  if (a.pairs > 0) a.block_tokens = std::max(1, std::min(a.block_tokens, kRotaryTable / a.pairs));
  int64_t groups = ((int64_t)a.tokens + a.block_tokens - 1) / a.block_tokens;
  if (groups < 2 * kComputeUnits) {
    const int64_t even = (int64_t)a.tokens / (2 * kComputeUnits);
    a.block_tokens = (int)std::max<int64_t>(1, std::min<int64_t>(a.block_tokens, even));
    groups = ((int64_t)a.tokens + a.block_tokens - 1) / a.block_tokens;
  }
  if (groups < 2 * kComputeUnits || row > 8 * kItems) {
    const int least = std::max(1, (groups < 2 * kComputeUnits ? kRotaryThreads : kItems) / a.packs);
    a.block_heads = std::min<int>((int)a.heads, least);
  }
  a.by_packs = fast_div((uint32_t)a.packs);
  a.by_heads = fast_div((uint32_t)a.block_heads);
  a.by_pairs = fast_div((uint32_t)std::max(a.pairs, 1));
  a.blocks = (uint32_t)groups;
  const dim3 grid((unsigned)std::min<int64_t>(groups, 1 << 20),
                  (unsigned)((a.heads + a.block_heads - 1) / a.block_heads));
  const size_t lds = sizeof(float2) * (size_t)a.block_tokens * (size_t)a.pairs;
  hipLaunchKernelGGL((rotary_kernel<DT, N, NEXT>), grid, dim3(kRotaryThreads), lds, s, a);
  return hipGetLastError();
}

template <int DT, int N>
static hipError_t launch_layout(const RotaryArgs& a, hipStream_t s) {
  if constexpr (N > 1) {
    if (a.interleaved) return launch_packed<DT, N, true>(a, s);
  }
  return launch_packed<DT, N, false>(a, s);
}

// The longest packs that the turned part has; in place they must divide it, as
// a column that two packs share would be turned twice.
template <int DT>
static hipError_t launch_type(const RotaryArgs& a, hipStream_t s) {
  const int span = a.interleaved ? 2 * a.pairs : a.pairs;
  const auto fits = [&](int n) { return a.pairs == 0 || (span >= n && (a.x.p != a.out.p || span % n == 0)); };
  if constexpr (OpElem<DT>::kPack == 8) {
    if (fits(8)) return launch_layout<DT, 8>(a, s);
  }
  if (fits(4)) return launch_layout<DT, 4>(a, s);
  if (fits(2)) return launch_layout<DT, 2>(a, s);
  return launch_layout<DT, 1>(a, s);
}

hipError_t launch_rotary(RotaryArgs a, int dtype, hipStream_t s) {
  switch (dtype) {
    case RINGSIM_FLOAT32: return launch_type<RINGSIM_FLOAT32>(a, s);
    case RINGSIM_BFLOAT16: return launch_type<RINGSIM_BFLOAT16>(a, s);
    case RINGSIM_FLOAT16: return launch_type<RINGSIM_FLOAT16>(a, s);
    default: return hipErrorInvalidValue;
  }
}

}  // namespace ringsim
