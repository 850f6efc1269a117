// kv_cache.hip -- tokens into the paged 4-bit cache, and back.
//
// Append: keys are turned by their positions, then of every 32 columns w of
// keys and values e = the least exponent with max|w| <= 7 * 2^e, and 4 bits
// hold the nearest to w / 2^e. What bounds it is memory: 2 or 4 bytes a column
// in, 17/32 out. A lane holds 16 columns of a key and the same of its value,
// all asked for before the workgroup forms the angles of its tokens, once for
// all heads, in LDS. Columns lie side by side, two lanes to a block; where the
// halves of a head are turned against each other, 8 lie in either half, so
// that a lane has both of each pair, and four lanes make a block. The block's
// maximum takes one or two lane permutations, and the conversion instruction
// divides by the power of two and rounds. Keys are turned in fp64: a last bit
// may decide between two codes.
#include <algorithm>

#include "attention_device.h"

namespace ringsim {

constexpr int kKvThreads = 256;
constexpr int kKvColumns = 16;     // of a lane
constexpr int kKvTable = 512;      // most pairs of a workgroup's tokens: 8 KiB, or one token's

// How keys are turned, and so which columns a lane has: kRotHalves if pairs
// are a multiple of 32 and what is left over one of 64, kRotAny for halves of
// other sizes, whose partners a lane reads one by one.
enum KvRotation : int { kRotNone = 0, kRotNext = 1, kRotHalves = 2, kRotAny = 3 };

// First columns of a lane's two packs of 8.
struct Columns {
  int c[2];
};
template <int ROT>
__device__ __forceinline__ Columns columns_of(int i, int pairs, int dim) {
  if constexpr (ROT != kRotHalves) return Columns{{16 * i, 16 * i + 8}};
  const int r = i - pairs / 8;
  return r < 0 ? Columns{{8 * i, 8 * i + pairs}} : Columns{{2 * pairs + 8 * r, pairs + dim / 2 + 8 * r}};
}

template <int DT>
struct Half {
  Packed<DT, 8> u[2];
  __device__ __forceinline__ void load(const typename OpElem<DT>::T* x, const Columns& at) {
    u[0].load(x + at.c[0]);
    u[1].load(x + at.c[1]);
  }
  __device__ __forceinline__ void get(float (&w)[16]) const {
#pragma unroll
    for (int j = 0; j < 16; ++j) w[j] = u[j / 8].get(j % 8);
  }
};

template <int DT, int ROT>
__device__ __forceinline__ void turn_columns(float (&w)[16], const typename OpElem<DT>::T* x, const Columns& at,
                                             int pairs, const double2* turn) {
  const int c = at.c[0];
  if constexpr (ROT == kRotNext) {
#pragma unroll
    for (int j = 0; j < 16; j += 2) {
      if (c + j < 2 * pairs) {
        const double2 t = turn[(c + j) / 2];
        const double p = w[j], q = w[j + 1];
        w[j] = (float)__builtin_fma(p, t.x, -(q * t.y));
        w[j + 1] = (float)__builtin_fma(q, t.x, p * t.y);
      }
    }
  } else if constexpr (ROT == kRotHalves) {
    if (c < pairs) {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const double2 t = turn[c + j];
        const double p = w[j], q = w[8 + j];
        w[j] = (float)__builtin_fma(p, t.x, -(q * t.y));
        w[8 + j] = (float)__builtin_fma(q, t.x, p * t.y);
      }
    }
  } else if constexpr (ROT == kRotAny) {
#pragma unroll
    for (int j = 0; j < 16; ++j) {
      if (c + j < 2 * pairs) {
        const bool first = c + j < pairs;
        const int i = first ? c + j : c + j - pairs;
        const double2 t = turn[i];
        const double other = (double)elem_to_f32<DT>(x[first ? i + pairs : i]) * t.y;
        w[j] = (float)__builtin_fma((double)w[j], t.x, first ? -other : other);
      }
    }
  }
}

// 8 columns as codes; `unit` their block's power of two.
__device__ __forceinline__ uint32_t to_codes(const float* w, float unit) {
  uint32_t codes = 0;
  codes = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(codes, w[0], w[1], unit, 0);
  codes = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(codes, w[2], w[3], unit, 1);
  codes = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(codes, w[4], w[5], unit, 2);
  return __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(codes, w[6], w[7], unit, 3);
}

// Magnitudes order like their bits, infinity above every finite one and NaN above infinity.
__device__ __forceinline__ uint32_t top_of(const float* w) {
  uint32_t top = 0;
#pragma unroll
  for (int j = 0; j < 8; ++j) top = MaxBits::of(top, __float_as_uint(w[j]) & 0x7fffffffu);
  return top;
}

// A lane's columns into their slot of keys or values.
template <int ROT>
__device__ __forceinline__ void store_columns(const KvCacheArgs& c, int which, int32_t page, int off, uint32_t head,
                                              const Columns& at, const float (&w)[16]) {
  uint8_t* data = c.data[which] + (int64_t)page * c.page + (int64_t)head * c.head + (int64_t)off * (c.dim / 2);
  uint8_t* scale = c.scales[which] + (int64_t)page * c.scale_page + (int64_t)head * c.scale_head + off;
  const auto put_scale = [&](int column, int byte) {
    if (column % kKvBlock == 0) scale[(column / kKvBlock) << c.page_shift] = (uint8_t)byte;
  };
  if constexpr (ROT == kRotHalves) {
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const int byte = kv_exponent_byte(lanes_reduce<4, MaxBits>(top_of(w + 8 * k)));
      const uint32_t codes = to_codes(w + 8 * k, __uint_as_float((uint32_t)byte << 23));
      *reinterpret_cast<uint32_t*>(data + at.c[k] / 2) = byte == kKvNan ? 0 : codes;
      put_scale(at.c[k], byte);
    }
  } else {
    uint32_t top = MaxBits::of(top_of(w), top_of(w + 8));
    top = MaxBits::of(top, dpp<0xB1>(top));  // of the neighbour lane
    const int byte = kv_exponent_byte(top);
    const float unit = __uint_as_float((uint32_t)byte << 23);
    const uint32_t lo = to_codes(w, unit), hi = to_codes(w + 8, unit);
    *reinterpret_cast<u32x2*>(data + at.c[0] / 2) = byte == kKvNan ? u32x2{0, 0} : u32x2{lo, hi};
    put_scale(at.c[0], byte);
  }
}

template <int DT, int ROT>
__global__ __launch_bounds__(kKvThreads) void kv_append_kernel(const KvAppendArgs a) {
  extern __shared__ double2 angles[];  // {cos, sin} * scale of [token, pair]
  const uint32_t head0 = blockIdx.y * a.block_heads;
  const int packs = a.cache.dim / kKvColumns;  // a multiple of 2 (of 4 with halves), so a block's lanes stay together
  const uint32_t items = (uint32_t)a.block_tokens * a.block_heads * packs;
  for (uint32_t block = blockIdx.x; block < a.blocks; block += gridDim.x) {
    const uint32_t token0 = block * a.block_tokens;
    const uint32_t tokens = min((uint32_t)a.block_tokens, a.tokens - token0);
    for (uint32_t base = 0; base < items; base += kKvThreads) {
      const uint32_t n = base + threadIdx.x;
      const uint32_t row = divide(n, a.by_packs), h = divide(row, a.by_tokens), t = row - h * a.block_tokens;
      const uint32_t head = head0 + h;
      const bool on = n < items && t < tokens && head < (uint32_t)a.cache.heads;
      const Columns at = columns_of<ROT>((int)(n - row * packs), a.pairs, a.cache.dim);
      const TokenAt token = token_at(token0 + (on ? t : 0), a.inner);
      Half<DT> k, v;
      int64_t slot = -1;
      const typename OpElem<DT>::T* key = head_ptr<DT>(a.x[0], token, on ? head : 0);
      if (on) {
        slot = read_index(a.slots, token.o, token.i);
        k.load(key, at);
        v.load(head_ptr<DT>(a.x[1], token, head), at);
      }
      if constexpr (ROT != kRotNone) {
        if (base == 0) {
          if (block != blockIdx.x) __syncthreads();  // the last block's angles have been read
          for (uint32_t i = threadIdx.x; i < tokens * a.pairs; i += kKvThreads) {
            const uint32_t of = divide(i, a.by_pairs), pair = i - of * a.pairs;
            const TokenAt there = token_at(token0 + of, a.inner);
            double s, c;
            sincospi(half_turns(read_index(a.positions, there.o, there.i), a.frequencies[pair]), &s, &c);
            angles[i] = double2{c * a.scale, s * a.scale};
          }
          __syncthreads();
        }
      }
      int32_t page;
      int off;
      if (!on || !kv_slot(slot, a.cache.pages, a.cache.page_shift, &page, &off)) continue;
      float w[16];
      k.get(w);
      turn_columns<DT, ROT>(w, key, at, a.pairs, angles + t * a.pairs);
      store_columns<ROT>(a.cache, 0, page, off, head, at, w);
      v.get(w);
      store_columns<ROT>(a.cache, 1, page, off, head, at, w);
    }
  }
}

template <int DT, int ROT>
static hipError_t launch_rotation(const KvAppendArgs& a, dim3 grid, hipStream_t s) {
  const size_t lds = ROT == kRotNone ? 0 : sizeof(double2) * (size_t)a.block_tokens * (size_t)a.pairs;
  hipLaunchKernelGGL((kv_append_kernel<DT, ROT>), grid, dim3(kKvThreads), lds, s, a);
  return hipGetLastError();
}

template <int DT>
static hipError_t launch_append(KvAppendArgs a, hipStream_t s) {
  const int packs = a.cache.dim / kKvColumns;
  const int64_t row = (int64_t)a.cache.heads * packs;
  // A workgroup's lanes take an item each where a token has no more of them;
  // its heads are cut where tokens are few, or many heads would make it long:
  // 200 tokens of 64 heads of 128 4.8 us, with whole tokens 5.5; 4000 of 128 heads
  // whole 49 us, with cut heads, which form the angles several times, 56.
  a.block_heads = a.cache.heads;
  a.block_tokens = (int)std::max<int64_t>(1, std::min<int64_t>(kKvThreads / row, a.tokens));
  if (a.pairs > 0) a.block_tokens = std::max(1, std::min(a.block_tokens, kKvTable / a.pairs));
  const int64_t groups = ((int64_t)a.tokens + a.block_tokens - 1) / a.block_tokens;
  if (row > (groups < kComputeUnits ? 1 : 8) * kKvThreads)
    a.block_heads = std::min(a.cache.heads, std::max(1, kKvThreads / packs));
  a.blocks = (uint32_t)groups;
  a.by_packs = fast_div((uint32_t)packs);
  a.by_tokens = fast_div((uint32_t)a.block_tokens);
  a.by_pairs = fast_div((uint32_t)std::max(a.pairs, 1));
  const dim3 grid((unsigned)std::min<int64_t>(groups, 1 << 20),
                  (unsigned)((a.cache.heads + a.block_heads - 1) / a.block_heads));
  if (a.pairs == 0) return launch_rotation<DT, kRotNone>(a, grid, s);
  if (a.interleaved) return launch_rotation<DT, kRotNext>(a, grid, s);
  return a.pairs % 32 == 0 && (a.cache.dim - 2 * a.pairs) % 64 == 0 ? launch_rotation<DT, kRotHalves>(a, grid, s)
                                                                    : launch_rotation<DT, kRotAny>(a, grid, s);
}

hipError_t launch_kv_append(KvAppendArgs a, int dtype, hipStream_t s) {
  switch (dtype) {
    case RINGSIM_FLOAT32: return launch_append<RINGSIM_FLOAT32>(a, s);
    case RINGSIM_BFLOAT16: return launch_append<RINGSIM_BFLOAT16>(a, s);
    case RINGSIM_FLOAT16: return launch_append<RINGSIM_FLOAT16>(a, s);
    default: return hipErrorInvalidValue;
  }
}

// Reading back: a lane takes 8 columns of one token, 4 bytes and an exponent
// in, a pack out, so that a wave's stores leave no gaps (16 columns a lane: 14.2
// us for 8192 tokens of 8 heads of 128, now 9.6). blockIdx.y: keys or values.
constexpr int kReadColumns = 8;

template <int DT>
__global__ __launch_bounds__(kKvThreads) void kv_read_kernel(const KvReadArgs a) {
  const int which = blockIdx.y;
  if (!a.out[which].p) return;
  const uint64_t packs = a.cache.dim / kReadColumns, items = (uint64_t)a.tokens * a.cache.heads * packs;
  for (uint64_t n = (uint64_t)blockIdx.x * kKvThreads + threadIdx.x; n < items; n += (uint64_t)gridDim.x * kKvThreads) {
    uint32_t token, head;
    int c;
    if (items <= 0x7fffffffu) {
      const uint32_t row = divide((uint32_t)n, a.by_packs);
      token = divide(row, a.by_heads);
      head = row - token * a.cache.heads;
      c = (int)((uint32_t)n - row * (uint32_t)packs) * kReadColumns;
    } else {
      const uint64_t row = n / packs;
      token = (uint32_t)(row / a.cache.heads);
      head = (uint32_t)(row - (uint64_t)token * a.cache.heads);
      c = (int)(n - row * packs) * kReadColumns;
    }
    const TokenAt at = token_at(token, a.inner);
    int32_t page;
    int off;
    uint32_t codes = 0, byte = kKvMinByte;
    if (kv_slot(read_index(a.slots, at.o, at.i), a.cache.pages, a.cache.page_shift, &page, &off)) {
      const uint8_t* data = a.cache.data[which] + (int64_t)page * a.cache.page + (int64_t)head * a.cache.head;
      codes = *reinterpret_cast<const uint32_t*>(data + ((int64_t)off * a.cache.dim + c) / 2);
      const uint8_t* scale =
          a.cache.scales[which] + (int64_t)page * a.cache.scale_page + (int64_t)head * a.cache.scale_head;
      byte = scale[((c / kKvBlock) << a.cache.page_shift) + off];
    }
    const float unit = __uint_as_float(byte << 23);  // 255: the conversion gives NaN
    const uint32_t v[4] = {__builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, unit, 0)),
                           __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, unit, 1)),
                           __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, unit, 2)),
                           __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, unit, 3))};
    Packed<DT, 8> y;
    if constexpr (DT == RINGSIM_BFLOAT16) {
#pragma unroll
      for (int j = 0; j < 4; ++j) y.w[j] = v[j];
    } else {
      float f[8];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        f[2 * j] = bf16_lo(v[j]);
        f[2 * j + 1] = bf16_hi(v[j]);
      }
      y.set(f);
    }
    y.store(head_ptr<DT>(a.out[which], at, head) + c);
  }
}

template <int DT>
static hipError_t launch_read(KvReadArgs a, hipStream_t s) {
  const int packs = a.cache.dim / kReadColumns;
  a.by_packs = fast_div((uint32_t)packs);
  a.by_heads = fast_div((uint32_t)a.cache.heads);
  const int64_t groups = ((int64_t)a.tokens * a.cache.heads * packs + kKvThreads - 1) / kKvThreads;
  const dim3 grid((unsigned)std::min<int64_t>(groups, 1 << 20), 2);
  hipLaunchKernelGGL((kv_read_kernel<DT>), grid, dim3(kKvThreads), 0, s, a);
  return hipGetLastError();
}

hipError_t launch_kv_read(KvReadArgs a, int dtype, hipStream_t s) {
  switch (dtype) {
    case RINGSIM_FLOAT32: return launch_read<RINGSIM_FLOAT32>(a, s);
    case RINGSIM_BFLOAT16: return launch_read<RINGSIM_BFLOAT16>(a, s);
    case RINGSIM_FLOAT16: return launch_read<RINGSIM_FLOAT16>(a, s);
    default: return hipErrorInvalidValue;
  }
}

}  // namespace ringsim
