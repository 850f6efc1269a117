// ops_device.h -- device building blocks of the step operators: 16-byte packs
// of elements in registers, rounding to the element types, and sums over
// lanes and waves.
#pragma once

#include "ops_internal.h"
#include "ringsim_device.h"

namespace ringsim {

// The same vectors at an address that is only aligned to an element: gfx950
// reads and writes them with one 128-bit access all the same.
typedef u32x4 u32x4_e2 __attribute__((aligned(2)));
typedef u32x2 u32x2_e2 __attribute__((aligned(2)));
typedef uint32_t u32_e2 __attribute__((aligned(2)));
typedef u32x2 u32x2_e1 __attribute__((aligned(1)));
typedef uint32_t u32_e1 __attribute__((aligned(1)));

// A lane holds 16 bytes side by side, whatever the type, so that a wave's
// access covers 1024 bytes without gaps. (With 32 bytes a lane for fp32, each
// non-temporal store left half-written lines: 236 us against 173 for the
// gradients of 16384 rows of 4096.)
template <int DT>
struct OpElem {
  using T = uint16_t;
  static constexpr int kPack = 8;
};
template <>
struct OpElem<RINGSIM_FLOAT32> {
  using T = uint32_t;
  static constexpr int kPack = 4;
};

template <int DT>
__device__ __forceinline__ float elem_to_f32(typename OpElem<DT>::T e) {
  if constexpr (DT == RINGSIM_FLOAT32) {
    return __uint_as_float(e);
  } else if constexpr (DT == RINGSIM_BFLOAT16) {
    return __uint_as_float((uint32_t)e << 16);
  } else {
    return (float)__builtin_bit_cast(_Float16, e);
  }
}

template <int DT>
__device__ __forceinline__ typename OpElem<DT>::T f32_to_elem(float f) {
  if constexpr (DT == RINGSIM_FLOAT32) {
    return __float_as_uint(f);
  } else if constexpr (DT == RINGSIM_BFLOAT16) {
    return (uint16_t)to_bf16(f);
  } else {
    return __builtin_bit_cast(uint16_t, (_Float16)f);
  }
}

// A vector in device memory: said so, the load needs no test for LDS addresses
// where the compiler cannot tell where a pointer comes from.
typedef __attribute__((address_space(1))) u32x4_e2 GlobalVec;

// How a kernel reads its rows: through the caches, past them (data that the
// Infinity Cache will not hold until it is needed again), or element by
// element, for rows shorter than a vector.
enum LoadKind : int { kLoadCached = 0, kLoadStream = 1, kLoadShort = 2 };

// 16 bytes at byte `at` of a sequence of `bytes`, whose length need not be a
// multiple of 16. No branch around the load: a vector that would pass the end
// is read from where the last whole one starts, so every lane reads inside
// the sequence and all loads of a thread are under way before the first one
// is used; fix16 then moves the elements to their places and puts zeros
// behind them. (Reading the rest element by element, the compiler made
// dependent loads of it and waited after each.) `bytes` is at least 16 unless
// the kind is kLoadShort; `at` may start at or past the end.
template <int LK>
__device__ __forceinline__ u32x4 load16(const void* p, int at, int bytes) {
  const char* c = static_cast<const char*>(p);
  if constexpr (LK == kLoadShort) {
    uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (at + 2 * i < bytes) w[i / 2] |= (uint32_t)*reinterpret_cast<const uint16_t*>(c + at + 2 * i) << (16 * (i % 2));
    return u32x4{w[0], w[1], w[2], w[3]};
  } else {
    const int start = at < bytes - 16 ? at : bytes - 16;
    const GlobalVec* q = (const GlobalVec*)(c + start);
    return LK == kLoadStream ? __builtin_nontemporal_load(q) : *q;
  }
}

template <int LK>
__device__ __forceinline__ u32x4 fix16(u32x4 v, int at, int bytes) {
  const int over = at - (bytes - 16);  // bytes to move down by
  if (LK == kLoadShort || over <= 0) return v;
  if (over >= 16) return u32x4{0, 0, 0, 0};
  if (over & 8) v = u32x4{v[2], v[3], 0, 0};
  if (over & 4) v = u32x4{v[1], v[2], v[3], 0};
  if (over & 2) v = u32x4{v[0] >> 16 | v[1] << 16, v[1] >> 16 | v[2] << 16, v[2] >> 16 | v[3] << 16, v[3] >> 16};
  return v;
}

// Writes what lies below `bytes` of 16 bytes at byte `at`. Results go out
// non-temporally (NT): written lines that stay out of the L2s leave them to
// the reads. A 64 MiB copy over three buffer sets takes 20.2 us so and 24.5
// us with plain stores; a kernel that reads the result next takes as much
// longer as was saved at 32-128 MiB, and less at 512 MiB (272 us for the
// pair against 294).
template <bool NT>
__device__ __forceinline__ void store16(void* p, u32x4 v, int at, int bytes) {
  char* c = static_cast<char*>(p) + at;
  const int left = bytes - at;
  if (left >= 16) {
    if constexpr (NT)
      __builtin_nontemporal_store(v, reinterpret_cast<u32x4_e2*>(c));
    else
      *reinterpret_cast<u32x4_e2*>(c) = v;
  } else if (left > 0) {
    // 8, 4 and 2 bytes as the rest's length has them.
    if (left & 8) {
      *reinterpret_cast<u32x2_e2*>(c) = u32x2{v[0], v[1]};
      v[0] = v[2];
      v[1] = v[3];
      c += 8;
    }
    if (left & 4) {
      *reinterpret_cast<u32_e2*>(c) = v[0];
      v[0] = v[1];
      c += 4;
    }
    if (left & 2) *reinterpret_cast<uint16_t*>(c) = (uint16_t)v[0];
  }
}

template <int DT>
__device__ __forceinline__ int byte_of(int element) {
  return element * (int)sizeof(typename OpElem<DT>::T);
}

// The pack at element c of a row of `cols`; fix_pack before its elements count.
template <int DT, int LK>
__device__ __forceinline__ u32x4 load_pack(const void* row, int c, int cols) {
  return load16<LK>(row, byte_of<DT>(c), byte_of<DT>(cols));
}
template <int DT, int LK>
__device__ __forceinline__ u32x4 fix_pack(u32x4 v, int c, int cols) {
  return fix16<LK>(v, byte_of<DT>(c), byte_of<DT>(cols));
}

template <int DT>
__device__ __forceinline__ void unpack(u32x4 v, float* f) {
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    if constexpr (DT == RINGSIM_FLOAT32) {
      f[j] = __uint_as_float(v[j]);
    } else if constexpr (DT == RINGSIM_BFLOAT16) {
      f[2 * j] = bf16_lo(v[j]);
      f[2 * j + 1] = bf16_hi(v[j]);
    } else {
      f[2 * j] = elem_to_f32<DT>((uint16_t)(v[j] & 0xffffu));
      f[2 * j + 1] = elem_to_f32<DT>((uint16_t)(v[j] >> 16));
    }
  }
}

// Rounds a pack of floats to the type, to nearest even.
template <int DT>
__device__ __forceinline__ u32x4 to_pack(const float* f) {
  u32x4 v;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    if constexpr (DT == RINGSIM_FLOAT32) {
      v[j] = __float_as_uint(f[j]);
    } else if constexpr (DT == RINGSIM_BFLOAT16) {
      v[j] = to_bf16x2(f[2 * j], f[2 * j + 1]);
    } else {
      v[j] = (uint32_t)f32_to_elem<DT>(f[2 * j]) | (uint32_t)f32_to_elem<DT>(f[2 * j + 1]) << 16;
    }
  }
  return v;
}

template <int DT>
__device__ __forceinline__ void store_pack(void* row, u32x4 v, int c, int cols) {
  store16<true>(row, v, byte_of<DT>(c), byte_of<DT>(cols));
}

// ---------------------------------------------------------------------------
// Reductions over neighbouring lanes
// ---------------------------------------------------------------------------

struct AddF32 {
  static __device__ __forceinline__ float of(float a, float b) { return a + b; }
};
// Largest magnitude, given as the bits of |v|: they order like the values,
// infinity above every finite one and NaN above infinity, so a NaN wins.
struct MaxBits {
  static __device__ __forceinline__ uint32_t of(uint32_t a, uint32_t b) { return a > b ? a : b; }
};

template <int CTRL, typename V>
__device__ __forceinline__ V dpp(V v) {
  return __builtin_bit_cast(
      V, __builtin_amdgcn_mov_dpp(__builtin_bit_cast(int, v), CTRL, 0xf, 0xf, true));
}

// Joins each row of 16 lanes, whose lanes are equal, with its neighbour.
template <typename OP, typename V>
__device__ __forceinline__ V swap16_reduce(V v) {
  const uint32_t u = __builtin_bit_cast(uint32_t, v);
  const auto s = __builtin_amdgcn_permlane16_swap(u, u, false, false);
  return OP::of(__builtin_bit_cast(V, (uint32_t)s[0]), __builtin_bit_cast(V, (uint32_t)s[1]));
}

// The reduction of `LANES` neighbouring lanes (a power of two, 4 to 64),
// known to each of them. Steps 1, 2, 4, 8 stay inside a row of 16 lanes and
// are lane permutations of the vector unit (quad permutes, half-row and row
// mirrors: the steps before have made the mirrored lanes equal); 16 and 32
// swap rows and halves. Each lane combines the same pairs, so all of them
// hold the same bits.
template <int LANES, typename OP, typename V>
__device__ __forceinline__ V lanes_reduce(V v) {
  static_assert(LANES >= 4 && LANES <= 64 && (LANES & (LANES - 1)) == 0, "lanes");
  v = OP::of(v, dpp<0xB1>(v));                          // quad_perm [1,0,3,2]
  v = OP::of(v, dpp<0x4E>(v));                          // quad_perm [2,3,0,1]
  if constexpr (LANES >= 8) v = OP::of(v, dpp<0x141>(v));   // row_half_mirror
  if constexpr (LANES >= 16) v = OP::of(v, dpp<0x140>(v));  // row_mirror
  if constexpr (LANES >= 32) v = swap16_reduce<OP>(v);
  if constexpr (LANES >= 64) {
    const uint32_t u = __builtin_bit_cast(uint32_t, v);
    const auto s = __builtin_amdgcn_permlane32_swap(u, u, false, false);
    v = OP::of(__builtin_bit_cast(V, (uint32_t)s[0]), __builtin_bit_cast(V, (uint32_t)s[1]));
  }
  return v;
}

// ---------------------------------------------------------------------------
// Rows
// ---------------------------------------------------------------------------

// Lanes that hold a row: TPR of them up to a wave, several rows a workgroup;
// above, one row a workgroup of whole waves, TPR the most it may have.
template <int TPR>
__device__ __forceinline__ int row_lanes() {
  return TPR <= 64 ? TPR : (int)blockDim.x;
}
template <int TPR>
constexpr int kRowsPerBlock = TPR <= 64 ? 256 / TPR : 1;
template <int TPR>
constexpr int kMaxBlock = TPR <= 64 ? 256 : TPR;

// Where the waves of a row leave what they reduced. Two buffers in turn, so
// one barrier a reduction is enough: a wave that writes a buffer again has
// passed the barrier of the other one, which every wave reached after it had
// read this one. Slots of waves that the workgroup does not have stay 0.
template <int TPR, typename V>
struct RowBuffers {
  static constexpr int kWaves = TPR > 64 ? TPR / 64 : 1;
  V slot[2][kWaves];

  // Before the first reduction; its barrier orders these writes too.
  __device__ __forceinline__ void clear() {
    if constexpr (TPR > 64) {
      const int i = threadIdx.x;
      if (i < kWaves && i >= (int)(blockDim.x >> 6)) slot[0][i] = slot[1][i] = V{};
    }
  }
};

// Sum (or largest) over the lanes that hold a row, known to each of them.
// Rows of one wave or less need no barrier.
template <int TPR, typename OP, typename V>
__device__ __forceinline__ V row_reduce(V v, RowBuffers<TPR, V>& buf, int& turn) {
  v = lanes_reduce<(TPR < 64 ? TPR : 64), OP>(v);
  if constexpr (TPR > 64) {
    if ((threadIdx.x & 63) == 0) buf.slot[turn][threadIdx.x >> 6] = v;
    __syncthreads();
    v = buf.slot[turn][0];
#pragma unroll
    for (int i = 1; i < TPR / 64; ++i) v = OP::of(v, buf.slot[turn][i]);
    turn ^= 1;
  }
  return v;
}

// Two sums with one barrier.
template <int TPR>
__device__ __forceinline__ void row_reduce2(float& a, float& b, RowBuffers<TPR, f32x2>& buf, int& turn) {
  constexpr int kLanes = TPR < 64 ? TPR : 64;
  a = lanes_reduce<kLanes, AddF32>(a);
  b = lanes_reduce<kLanes, AddF32>(b);
  if constexpr (TPR > 64) {
    if ((threadIdx.x & 63) == 0) buf.slot[turn][threadIdx.x >> 6] = f32x2{a, b};
    __syncthreads();
    a = b = 0.0f;
#pragma unroll
    for (int i = 0; i < TPR / 64; ++i) {
      const f32x2 v = buf.slot[turn][i];
      a += v.x;
      b += v.y;
    }
    turn ^= 1;
  }
}

template <int DT>
__device__ __forceinline__ const typename OpElem<DT>::T* row_ptr(const RowsIn& t, uint32_t o, uint32_t i) {
  return static_cast<const typename OpElem<DT>::T*>(t.p) + ((int64_t)o * t.s0 + (int64_t)i * t.s1);
}
template <typename T>
__device__ __forceinline__ T* row_ptr(const RowsOut& t, uint32_t o, uint32_t i) {
  return static_cast<T*>(t.p) + ((int64_t)o * t.s0 + (int64_t)i * t.s1);
}

// The weights of a pack as they lie in memory: in the rows' type, or in fp32
// (twice the bytes of a pack of a 16-bit type).
struct WeightPack {
  u32x4 v[2];
};

template <int DT, int LK>
__device__ __forceinline__ WeightPack load_weight(const void* w, int kind, int c, int cols) {
  constexpr int kSize = (int)sizeof(typename OpElem<DT>::T);
  constexpr int kKind = LK == kLoadShort ? kLoadShort : kLoadCached;
  WeightPack r;
  r.v[0] = r.v[1] = u32x4{0, 0, 0, 0};
  if (kind != kWeightNone) {
    const int size = kind == kWeightF32 ? 4 : kSize;
    r.v[0] = load16<kKind>(w, c * size, cols * size);
    if (kSize == 2 && size == 4) r.v[1] = load16<kKind>(w, c * 4 + 16, cols * 4);
  }
  return r;
}

// The weights as fp32, zeros beyond the row (ones without a weight).
template <int DT, int LK>
__device__ __forceinline__ void unpack_weight(const WeightPack& r, int kind, int c, int cols, float* f) {
  if (kind == kWeightNone) {
#pragma unroll
    for (int i = 0; i < OpElem<DT>::kPack; ++i) f[i] = 1.0f;
  } else if (DT == RINGSIM_FLOAT32 || kind == kWeightF32) {
#pragma unroll
    for (int i = 0; i < OpElem<DT>::kPack / 4; ++i)
      unpack<RINGSIM_FLOAT32>(fix_pack<RINGSIM_FLOAT32, LK>(r.v[i], c + 4 * i, cols), f + 4 * i);
  } else {
    unpack<DT>(fix_pack<DT, LK>(r.v[0], c, cols), f);
  }
}

}  // namespace ringsim
