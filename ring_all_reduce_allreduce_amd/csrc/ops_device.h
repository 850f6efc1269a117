// ops_device.h -- device building blocks of the step operators: packs of
// eight elements in registers, rounding to the element types, and sums over
// lanes and waves.
#pragma once

#include "ops_internal.h"
#include "ringsim_device.h"

namespace ringsim {

typedef float f32x4 __attribute__((ext_vector_type(4)));
// The same vectors at an address that is only aligned to an element: gfx950
// reads and writes them with one 128-bit access all the same.
typedef u32x4 u32x4_e2 __attribute__((aligned(2)));
typedef u32x4 u32x4_e4 __attribute__((aligned(4)));
typedef u32x2 u32x2_e1 __attribute__((aligned(1)));

constexpr int kPack = 8;  // elements a lane holds side by side: 16 bytes of a 16-bit type, 32 of fp32

template <int DT>
struct OpElem {
  using T = uint16_t;
  using V = u32x4_e2;
  static constexpr int kVecs = 1;  // 16-byte vectors of a pack
};
template <>
struct OpElem<RINGSIM_FLOAT32> {
  using T = uint32_t;
  using V = u32x4_e4;
  static constexpr int kVecs = 2;
};

// Eight consecutive elements as they lie in memory.
template <int DT>
struct Pack {
  u32x4 v[OpElem<DT>::kVecs];
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

// Elements [0, n) of a pack at p; the others become 0. n >= kPack reads whole
// vectors, n <= 0 nothing.
template <int DT>
__device__ __forceinline__ Pack<DT> load_pack(const typename OpElem<DT>::T* p, int n) {
  using E = OpElem<DT>;
  Pack<DT> r;
  if (n >= kPack) {
#pragma unroll
    for (int i = 0; i < E::kVecs; ++i) r.v[i] = reinterpret_cast<const typename E::V*>(p)[i];
  } else {
    uint32_t w[4 * E::kVecs];
#pragma unroll
    for (int i = 0; i < 4 * E::kVecs; ++i) w[i] = 0;
#pragma unroll
    for (int i = 0; i < kPack - 1; ++i) {
      if (i < n) {
        if constexpr (E::kVecs == 2) {
          w[i] = p[i];
        } else {
          w[i / 2] |= (uint32_t)p[i] << (16 * (i % 2));
        }
      }
    }
#pragma unroll
    for (int i = 0; i < E::kVecs; ++i) r.v[i] = u32x4{w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]};
  }
  return r;
}

template <int DT>
__device__ __forceinline__ void unpack(const Pack<DT>& r, float* f) {
#pragma unroll
  for (int i = 0; i < OpElem<DT>::kVecs; ++i) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint32_t w = r.v[i][j];
      if constexpr (DT == RINGSIM_FLOAT32) {
        f[4 * i + j] = __uint_as_float(w);
      } else if constexpr (DT == RINGSIM_BFLOAT16) {
        f[2 * j] = bf16_lo(w);
        f[2 * j + 1] = bf16_hi(w);
      } else {
        f[2 * j] = elem_to_f32<DT>((uint16_t)(w & 0xffffu));
        f[2 * j + 1] = elem_to_f32<DT>((uint16_t)(w >> 16));
      }
    }
  }
}

// Rounds eight floats to the type, to nearest even.
template <int DT>
__device__ __forceinline__ Pack<DT> to_pack(const float* f) {
  Pack<DT> r;
#pragma unroll
  for (int i = 0; i < OpElem<DT>::kVecs; ++i) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if constexpr (DT == RINGSIM_FLOAT32) {
        r.v[i][j] = __float_as_uint(f[4 * i + j]);
      } else if constexpr (DT == RINGSIM_BFLOAT16) {
        r.v[i][j] = to_bf16x2(f[2 * j], f[2 * j + 1]);
      } else {
        r.v[i][j] = (uint32_t)f32_to_elem<DT>(f[2 * j]) | ((uint32_t)f32_to_elem<DT>(f[2 * j + 1]) << 16);
      }
    }
  }
  return r;
}

// Writes elements [0, n) of a pack to p.
template <int DT>
__device__ __forceinline__ void store_pack(typename OpElem<DT>::T* p, const Pack<DT>& r, int n) {
  using E = OpElem<DT>;
  if (n >= kPack) {
#pragma unroll
    for (int i = 0; i < E::kVecs; ++i) reinterpret_cast<typename E::V*>(p)[i] = r.v[i];
  } else {
#pragma unroll
    for (int i = 0; i < kPack - 1; ++i) {
      if (i < n) {
        if constexpr (E::kVecs == 2) {
          p[i] = r.v[i / 4][i % 4];
        } else {
          p[i] = (uint16_t)(r.v[0][i / 2] >> (16 * (i % 2)));
        }
      }
    }
  }
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
  if constexpr (LANES >= 32) {
    const uint32_t u = __builtin_bit_cast(uint32_t, v);
    const auto s = __builtin_amdgcn_permlane16_swap(u, u, false, false);
    v = OP::of(__builtin_bit_cast(V, (uint32_t)s[0]), __builtin_bit_cast(V, (uint32_t)s[1]));
  }
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

// Sum (or largest) over the TPR lanes that hold a row. Rows of one wave or
// less need no barrier. Longer ones join their waves' results through LDS:
// two buffers in turn, so one barrier a reduction is enough (a wave that
// writes a buffer again has passed the barrier of the other one, which every
// wave reached after it had read this one).
template <int TPR, typename OP, typename V>
__device__ __forceinline__ V row_reduce(V v, V (*buf)[16], int& turn) {
  v = lanes_reduce<(TPR < 64 ? TPR : 64), OP>(v);
  if constexpr (TPR > 64) {
    constexpr int kWaves = TPR / 64;
    if ((threadIdx.x & 63) == 0) buf[turn][threadIdx.x >> 6] = v;
    __syncthreads();
    v = buf[turn][0];
#pragma unroll
    for (int i = 1; i < kWaves; ++i) v = OP::of(v, buf[turn][i]);
    turn ^= 1;
  }
  return v;
}

template <int DT>
__device__ __forceinline__ const typename OpElem<DT>::T* row_ptr(const RowsIn& t, uint32_t o, uint32_t i) {
  return static_cast<const typename OpElem<DT>::T*>(t.p) + ((int64_t)o * t.s0 + (int64_t)i * t.s1);
}
template <typename T>
__device__ __forceinline__ T* row_ptr(const RowsOut& t, uint32_t o, uint32_t i) {
  return static_cast<T*>(t.p) + ((int64_t)o * t.s0 + (int64_t)i * t.s1);
}

// Eight weights as fp32.
template <int DT>
__device__ __forceinline__ void load_weight(const void* w, int kind, int c, int n, float* f) {
  if (kind == kWeightNone) {
#pragma unroll
    for (int i = 0; i < kPack; ++i) f[i] = 1.0f;
  } else if (DT == RINGSIM_FLOAT32 || kind == kWeightF32) {
    unpack<RINGSIM_FLOAT32>(load_pack<RINGSIM_FLOAT32>(static_cast<const uint32_t*>(w) + c, n), f);
  } else {
    unpack<DT>(load_pack<DT>(static_cast<const typename OpElem<DT>::T*>(w) + c, n), f);
  }
}

}  // namespace ringsim
