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
constexpr int kRotaryAhead = 4;     // items of a thread whose loads are under way together

// N columns an item: a 16-byte pack of each half (or of neighbouring pairs),
// or one pair (one column that is copied).
template <int DT, int N, bool NEXT>
__global__ __launch_bounds__(kRotaryThreads) void rotary_kernel(const RotaryArgs a) {
  extern __shared__ float2 turn[];  // {cos, sin} * scale of [token, pair]
  using T = typename OpElem<DT>::T;
  const uint32_t head0 = blockIdx.y * a.block_heads;
  for (uint32_t block = blockIdx.x; block < a.blocks; block += gridDim.x) {
    const uint32_t token0 = block * a.block_tokens;
    const uint32_t tokens = min((uint32_t)a.block_tokens, a.tokens - token0);
    if (block != blockIdx.x) __syncthreads();  // the last block's angles have been read
    for (uint32_t k = threadIdx.x; k < tokens * a.pairs; k += kRotaryThreads) {
      const uint32_t t = divide(k, a.by_pairs), i = k - t * a.pairs;
      const TokenAt at = token_at(token0 + t, a.inner);
      float s, c;
      sincospif((float)half_turns(read_index(a.positions, at.o, at.i), a.frequencies[i]), &s, &c);
      turn[k] = float2{c * a.scale, s * a.sign * a.scale};
    }
    __syncthreads();

    constexpr int kSpan = NEXT && N == 1 ? 2 : N;  // columns of a load; a pair of neighbours is two
    struct Item {
      TokenAt at;
      uint32_t t, head;
      int p;
      bool on;
      Packed<DT, kSpan> u, v;
    } item[kRotaryAhead];
    const uint32_t items = tokens * a.block_heads * a.packs;
    for (uint32_t base = threadIdx.x; base < items; base += kRotaryThreads * kRotaryAhead) {
#pragma unroll
      for (int k = 0; k < kRotaryAhead; ++k) {
        const uint32_t n = base + k * kRotaryThreads;
        const uint32_t row = divide(n, a.by_packs), t = divide(row, a.by_heads);
        Item& e = item[k];
        e.t = t;
        e.p = (int)(n - row * a.packs);
        e.head = head0 + row - t * a.block_heads;
        e.on = n < items && e.head < a.heads;
        if (!e.on) continue;
        e.at = token_at(token0 + t, a.inner);
        const T* x = head_ptr<DT>(a.x, e.at, e.head);
        if (e.p >= a.turned) {
          const T* rest = x + 2 * a.pairs + (e.p - a.turned) * N;
          if constexpr (kSpan == N)
            e.u.load(rest);
          else
            e.u.w[0] = rest[0];
        } else if constexpr (NEXT) {
          e.u.load(x + e.p * kSpan);
        } else {
          e.u.load(x + e.p * N);
          e.v.load(x + a.pairs + e.p * N);
        }
      }
#pragma unroll
      for (int k = 0; k < kRotaryAhead; ++k) {
        Item& e = item[k];
        if (!e.on) continue;
        T* y = head_ptr<DT>(a.out, e.at, e.head);
        if (e.p >= a.turned) {
          T* rest = y + 2 * a.pairs + (e.p - a.turned) * N;
          if constexpr (kSpan == N)
            e.u.store(rest);
          else
            rest[0] = (T)e.u.w[0];
          continue;
        }
        const float2* cs = turn + e.t * a.pairs + e.p * (NEXT ? kSpan / 2 : N);
        if constexpr (NEXT) {
          float f[kSpan];
#pragma unroll
          for (int i = 0; i < kSpan / 2; ++i) {
            const float p = e.u.get(2 * i), q = e.u.get(2 * i + 1), c = cs[i].x, s = cs[i].y;
            f[2 * i] = __builtin_fmaf(p, c, -(q * s));
            f[2 * i + 1] = __builtin_fmaf(q, c, p * s);
          }
          e.u.set(f);
          e.u.store(y + e.p * kSpan);
        } else {
          float f[N], g[N];
#pragma unroll
          for (int i = 0; i < N; ++i) {
            const float p = e.u.get(i), q = e.v.get(i), c = cs[i].x, s = cs[i].y;
            f[i] = __builtin_fmaf(p, c, -(q * s));
            g[i] = __builtin_fmaf(q, c, p * s);
          }
          e.u.set(f);
          e.v.set(g);
          e.u.store(y + e.p * N);
          e.v.store(y + a.pairs + e.p * N);
        }
      }
    }
  }
}

template <int DT, int N>
static hipError_t launch_packed(RotaryArgs a, hipStream_t s) {
  const bool in_place = a.x.p == a.out.p;
  a.turned = a.interleaved ? (N == 1 ? a.pairs : 2 * a.pairs / N) : a.pairs / N;
  a.packs = a.turned + (in_place ? 0 : (a.dim - 2 * a.pairs) / N);
  if (a.packs == 0) return hipSuccess;  // nothing is turned, in place
  // About a thousand items a workgroup, so that a thread has some loads under
  // way and the angles are shared; heads are cut where tokens are few.
  const int items = 1024;
  const int64_t row = (int64_t)a.heads * a.packs;
  a.block_heads = (int)a.heads;
  a.block_tokens = (int)std::max<int64_t>(1, std::min<int64_t>(items / std::max<int64_t>(row, 1), a.tokens));
  if (a.pairs > 0) a.block_tokens = std::max(1, std::min(a.block_tokens, kRotaryTable / a.pairs));
  const int64_t groups = ((int64_t)a.tokens + a.block_tokens - 1) / a.block_tokens;
  if (groups < 2 * kComputeUnits || row > 8 * items) {
    const int least = std::max(1, (groups < 2 * kComputeUnits ? kRotaryThreads : items) / a.packs);
    a.block_heads = std::min<int>((int)a.heads, least);
  }
  a.by_packs = fast_div((uint32_t)a.packs);
  a.by_heads = fast_div((uint32_t)a.block_heads);
  a.by_pairs = fast_div((uint32_t)std::max(a.pairs, 1));
  a.blocks = (uint32_t)groups;
  const dim3 grid((unsigned)std::min<int64_t>(groups, 1 << 20), (unsigned)((a.heads + a.block_heads - 1) / a.block_heads));
  const size_t lds = sizeof(float2) * (size_t)a.block_tokens * (size_t)a.pairs;
  if (a.interleaved)
    hipLaunchKernelGGL((rotary_kernel<DT, N, true>), grid, dim3(kRotaryThreads), lds, s, a);
  else
    hipLaunchKernelGGL((rotary_kernel<DT, N, false>), grid, dim3(kRotaryThreads), lds, s, a);
  return hipGetLastError();
}

template <int DT>
static hipError_t launch_type(const RotaryArgs& a, hipStream_t s) {
  constexpr int kPack = OpElem<DT>::kPack;
  const bool whole = (a.interleaved ? 2 * a.pairs : a.pairs) % kPack == 0 && (a.dim - 2 * a.pairs) % kPack == 0;
  return whole ? launch_packed<DT, kPack>(a, s) : launch_packed<DT, 1>(a, s);
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
