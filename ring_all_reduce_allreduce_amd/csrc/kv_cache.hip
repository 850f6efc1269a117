// kv_cache.hip -- tokens into the paged 4-bit cache, and back.
//
// Append: keys are turned by their positions, then of every 32 columns w of
// keys and values e = the least exponent with max|w| <= 7 * 2^e, and 4 bits
// hold the nearest to w / 2^e. A lane holds 8 columns, whose codes are one
// 32-bit store; four neighbouring lanes hold a block and find its maximum
// with two lane permutations; the conversion instruction divides by the
// power of two and rounds. What bounds it is memory: 2 or 4 bytes a column in,
// 17/32 out. Keys are turned in fp64: a last bit may decide between two
// codes, and the angles, which all heads of a token share, are formed once in
// LDS, so that what is left is four operations a column.
#include <algorithm>

#include "attention_device.h"

namespace ringsim {

constexpr int kKvThreads = 256;
constexpr int kKvColumns = 8;      // of a lane
constexpr int kKvTable = 512;      // most pairs of a workgroup's tokens: 8 KiB, or one token's

// Columns c .. c + 7 of a key after its rotation. `ROT`: 1 neighbouring
// columns, 2 halves of whole packs, 3 halves of any size.
enum KvRotation : int { kRotNone = 0, kRotNext = 1, kRotHalves = 2, kRotAny = 3 };

template <int DT, int ROT>
__device__ __forceinline__ void turned_columns(const typename OpElem<DT>::T* x, int c, int pairs, const double2* turn,
                                               float (&w)[kKvColumns]) {
  Packed<DT, kKvColumns> u;
  u.load(x + c);
#pragma unroll
  for (int j = 0; j < kKvColumns; ++j) w[j] = u.get(j);
  if constexpr (ROT == kRotNext) {
#pragma unroll
    for (int j = 0; j < kKvColumns; j += 2) {
      if (c + j < 2 * pairs) {
        const double2 t = turn[(c + j) / 2];
        const double p = w[j], q = w[j + 1];
        w[j] = (float)__builtin_fma(p, t.x, -(q * t.y));
        w[j + 1] = (float)__builtin_fma(q, t.x, p * t.y);
      }
    }
  } else if constexpr (ROT == kRotHalves) {
    if (c < 2 * pairs) {
      const bool first = c < pairs;
      const int i = first ? c : c - pairs;
      Packed<DT, kKvColumns> v;
      v.load(x + (first ? c + pairs : i));
#pragma unroll
      for (int j = 0; j < kKvColumns; ++j) {
        const double2 t = turn[i + j];
        const double other = (double)v.get(j) * t.y;
        w[j] = (float)__builtin_fma((double)w[j], t.x, first ? -other : other);
      }
    }
  } else if constexpr (ROT == kRotAny) {
#pragma unroll
    for (int j = 0; j < kKvColumns; ++j) {
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

template <int DT, int ROT>
__device__ __forceinline__ void append_rows(const KvAppendArgs& a, int which, uint32_t token0, uint32_t tokens,
                                            uint32_t head0, const double2* turn) {
  const int packs = a.cache.dim / kKvColumns;  // a multiple of 8, so four lanes of a block stay together
  const uint32_t items = (uint32_t)a.block_tokens * a.block_heads * packs;
  for (uint32_t n = threadIdx.x; n < items; n += kKvThreads) {
    const uint32_t row = divide(n, a.by_packs), h = divide(row, a.by_tokens), t = row - h * a.block_tokens;
    const uint32_t head = head0 + h;
    const int c = (int)(n - row * packs) * kKvColumns;
    if (t >= tokens || head >= (uint32_t)a.cache.heads) continue;
    const TokenAt at = token_at(token0 + t, a.inner);
    int32_t page;
    int off;
    if (!kv_slot(read_index(a.slots, at.o, at.i), a.cache.pages, a.cache.page_shift, &page, &off)) continue;
    float w[kKvColumns];
    turned_columns<DT, ROT>(head_ptr<DT>(a.x[which], at, head), c, a.pairs, turn + t * a.pairs, w);
    // Magnitudes order like their bits, infinity above every finite one and
    // NaN above infinity.
    uint32_t top = 0;
#pragma unroll
    for (int j = 0; j < kKvColumns; ++j) top = MaxBits::of(top, __float_as_uint(w[j]) & 0x7fffffffu);
    top = lanes_reduce<4, MaxBits>(top);
    const int byte = kv_exponent_byte(top);
    uint32_t codes = 0;
    if (byte != kKvNan) {
      const float unit = __uint_as_float((uint32_t)byte << 23);
      codes = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(codes, w[0], w[1], unit, 0);
      codes = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(codes, w[2], w[3], unit, 1);
      codes = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(codes, w[4], w[5], unit, 2);
      codes = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(codes, w[6], w[7], unit, 3);
    }
    uint8_t* data = a.cache.data[which] + (int64_t)page * a.cache.page + (int64_t)head * a.cache.head;
    *reinterpret_cast<uint32_t*>(data + ((int64_t)off * a.cache.dim + c) / 2) = codes;
    if (c % kKvBlock == 0) {
      uint8_t* scale = a.cache.scales[which] + (int64_t)page * a.cache.scale_page + (int64_t)head * a.cache.scale_head;
      scale[((c / kKvBlock) << a.cache.page_shift) + off] = (uint8_t)byte;
    }
  }
}

// blockIdx.z: keys or values. No branch on ROT inside: values take kRotNone.
template <int DT, int ROT>
__global__ __launch_bounds__(kKvThreads) void kv_append_kernel(const KvAppendArgs a) {
  extern __shared__ double2 angles[];  // {cos, sin} * scale of [token, pair]
  const uint32_t head0 = blockIdx.y * a.block_heads;
  for (uint32_t block = blockIdx.x; block < a.blocks; block += gridDim.x) {
    const uint32_t token0 = block * a.block_tokens;
    const uint32_t tokens = min((uint32_t)a.block_tokens, a.tokens - token0);
    if (ROT == kRotNone || blockIdx.z == 1) {
      append_rows<DT, kRotNone>(a, (int)blockIdx.z, token0, tokens, head0, angles);
      continue;
    }
    if constexpr (ROT != kRotNone) {
      if (block != blockIdx.x) __syncthreads();
      for (uint32_t k = threadIdx.x; k < tokens * a.pairs; k += kKvThreads) {
        const uint32_t t = divide(k, a.by_pairs), i = k - t * a.pairs;
        const TokenAt at = token_at(token0 + t, a.inner);
        double s, c;
        sincospi(half_turns(read_index(a.positions, at.o, at.i), a.frequencies[i]), &s, &c);
        angles[k] = double2{c * a.scale, s * a.scale};
      }
      __syncthreads();
      append_rows<DT, ROT>(a, 0, token0, tokens, head0, angles);
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
  a.block_heads = a.cache.heads;
  a.block_tokens = (int)std::max<int64_t>(1, std::min<int64_t>(2 * kKvThreads / row, a.tokens));
  if (a.pairs > 0) a.block_tokens = std::max(1, std::min(a.block_tokens, kKvTable / a.pairs));
  const int64_t groups = ((int64_t)a.tokens + a.block_tokens - 1) / a.block_tokens;
  if (groups < kComputeUnits || row > 8 * kKvThreads)
    a.block_heads = std::min(a.cache.heads, std::max(1, kKvThreads / packs));
  a.blocks = (uint32_t)groups;
  a.by_packs = fast_div((uint32_t)packs);
  a.by_tokens = fast_div((uint32_t)a.block_tokens);
  a.by_pairs = fast_div((uint32_t)std::max(a.pairs, 1));
  const dim3 grid((unsigned)std::min<int64_t>(groups, 1 << 20),
                  (unsigned)((a.cache.heads + a.block_heads - 1) / a.block_heads), 2);
  if (a.pairs == 0) return launch_rotation<DT, kRotNone>(a, grid, s);
  if (a.interleaved) return launch_rotation<DT, kRotNext>(a, grid, s);
  return a.pairs % kKvColumns == 0 ? launch_rotation<DT, kRotHalves>(a, grid, s)
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
// in, a pack out. blockIdx.y: keys or values.
template <int DT>
__global__ __launch_bounds__(kKvThreads) void kv_read_kernel(const KvReadArgs a) {
  const int which = blockIdx.y;
  if (!a.out[which].p) return;
  const uint64_t packs = a.cache.dim / kKvColumns, items = (uint64_t)a.tokens * a.cache.heads * packs;
  for (uint64_t n = (uint64_t)blockIdx.x * kKvThreads + threadIdx.x; n < items; n += (uint64_t)gridDim.x * kKvThreads) {
    uint32_t token, head;
    int c;
    if (items <= 0x7fffffffu) {
      const uint32_t row = divide((uint32_t)n, a.by_packs);
      token = divide(row, a.by_heads);
      head = row - token * a.cache.heads;
      c = (int)((uint32_t)n - row * (uint32_t)packs) * kKvColumns;
    } else {
      const uint64_t row = n / packs;
      token = (uint32_t)(row / a.cache.heads);
      head = (uint32_t)(row - (uint64_t)token * a.cache.heads);
      c = (int)(n - row * packs) * kKvColumns;
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
    const bf16x2 v[4] = {__builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, unit, 0),
                         __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, unit, 1),
                         __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, unit, 2),
                         __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, unit, 3)};
    Packed<DT, kKvColumns> y;
    if constexpr (DT == RINGSIM_BFLOAT16) {
#pragma unroll
      for (int j = 0; j < 4; ++j) y.w[j] = __builtin_bit_cast(uint32_t, v[j]);
    } else {
      float f[kKvColumns];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        f[2 * j] = bf16_lo(__builtin_bit_cast(uint32_t, v[j]));
        f[2 * j + 1] = bf16_hi(__builtin_bit_cast(uint32_t, v[j]));
      }
      y.set(f);
    }
    y.store(head_ptr<DT>(a.out[which], at, head) + c);
  }
}

template <int DT>
static hipError_t launch_read(KvReadArgs a, hipStream_t s) {
  const int packs = a.cache.dim / kKvColumns;
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
