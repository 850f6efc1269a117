// attention_device.h -- device building blocks of the attention-step
// operators.
#pragma once

#include "attention_internal.h"
#include "ops_device.h"

namespace ringsim {

typedef float f32x4 __attribute__((ext_vector_type(4)));

__device__ __forceinline__ int64_t read_index(const Index& x, uint32_t o, uint32_t i) {
  const int64_t at = (int64_t)o * x.s0 + (int64_t)i * x.s1;
  return x.wide ? static_cast<const int64_t*>(x.p)[at] : static_cast<const int32_t*>(x.p)[at];
}

// A token's place in its [outer, inner] array.
struct TokenAt {
  uint32_t o, i;
};
__device__ __forceinline__ TokenAt token_at(uint32_t n, uint32_t inner) {
  if (inner == 1) return TokenAt{n, 0};
  const uint32_t o = n / inner;
  return TokenAt{o, n - o * inner};
}

template <int DT>
__device__ __forceinline__ const typename OpElem<DT>::T* head_ptr(const HeadRows& r, TokenAt t, uint32_t head) {
  return static_cast<const typename OpElem<DT>::T*>(r.p) + ((int64_t)t.o * r.s0 + (int64_t)t.i * r.s1 +
                                                            (int64_t)head * r.s2);
}
template <int DT>
__device__ __forceinline__ typename OpElem<DT>::T* head_ptr(const HeadRowsOut& r, TokenAt t, uint32_t head) {
  return static_cast<typename OpElem<DT>::T*>(r.p) + ((int64_t)t.o * r.s0 + (int64_t)t.i * r.s1 +
                                                      (int64_t)head * r.s2);
}

// Half turns of the angle position * frequency, in [-1, 1]: the whole turns
// are taken off in 64 bits, where a million radians still have 33 bits behind
// the point. fp32 would leave 4.
__device__ __forceinline__ double half_turns(int64_t position, double frequency) {
  const double t = (double)position * frequency * 0.15915494309189535;  // 1 / (2 pi)
  return 2.0 * (t - __builtin_rint(t));
}

// N elements side by side in registers, N a power of two; vectors need the
// alignment of an element only.
template <int DT, int N>
struct Packed {
  static constexpr int kBytes = N * (int)sizeof(typename OpElem<DT>::T);
  uint32_t w[kBytes < 4 ? 1 : kBytes / 4];

  __device__ __forceinline__ void load(const void* p) {
    if constexpr (kBytes == 2) {
      w[0] = *static_cast<const uint16_t*>(p);
    } else if constexpr (kBytes == 4) {
      w[0] = *static_cast<const u32_e2*>(p);
    } else {
      static_assert(kBytes == 8 || kBytes % 16 == 0, "pack");
      if constexpr (kBytes == 8) {
        const u32x2 v = *static_cast<const u32x2_e2*>(p);
        w[0] = v[0];
        w[1] = v[1];
      } else {
#pragma unroll
        for (int k = 0; k < kBytes / 16; ++k) {
          const u32x4 v = static_cast<const u32x4_e2*>(p)[k];
#pragma unroll
          for (int i = 0; i < 4; ++i) w[4 * k + i] = v[i];
        }
      }
    }
  }
  // KEEP: what is read again soon, or written by lanes that lie apart, whose
  // bytes the L2 then puts together.
  template <bool KEEP = false>
  __device__ __forceinline__ void store(void* p) const {
    if constexpr (kBytes == 2) {
      *static_cast<uint16_t*>(p) = (uint16_t)w[0];
    } else if constexpr (kBytes == 4) {
      *static_cast<u32_e2*>(p) = w[0];
    } else if constexpr (kBytes == 8) {
      *static_cast<u32x2_e2*>(p) = u32x2{w[0], w[1]};
    } else {
#pragma unroll
      for (int k = 0; k < kBytes / 16; ++k) {
        const u32x4 v = {w[4 * k], w[4 * k + 1], w[4 * k + 2], w[4 * k + 3]};
        if constexpr (KEEP)
          static_cast<u32x4_e2*>(p)[k] = v;
        else
          __builtin_nontemporal_store(v, static_cast<u32x4_e2*>(p) + k);
      }
    }
  }
  __device__ __forceinline__ float get(int i) const {
    if constexpr (DT == RINGSIM_FLOAT32)
      return __uint_as_float(w[i]);
    else if constexpr (DT == RINGSIM_BFLOAT16)
      return i % 2 ? bf16_hi(w[i / 2]) : bf16_lo(w[i / 2]);
    else
      return elem_to_f32<DT>((uint16_t)(w[i / 2] >> (16 * (i % 2))));
  }
  // Rounds to the type, to nearest even.
  __device__ __forceinline__ void set(const float (&f)[N]) {
    if constexpr (N == 1) {
      w[0] = f32_to_elem<DT>(f[0]);
    } else if constexpr (DT == RINGSIM_FLOAT32) {
#pragma unroll
      for (int i = 0; i < N; ++i) w[i] = __float_as_uint(f[i]);
    } else {
#pragma unroll
      for (int i = 0; i < N / 2; ++i) {
        if constexpr (DT == RINGSIM_BFLOAT16)
          w[i] = to_bf16x2(f[2 * i], f[2 * i + 1]);
        else
          w[i] = (uint32_t)f32_to_elem<DT>(f[2 * i]) | (uint32_t)f32_to_elem<DT>(f[2 * i + 1]) << 16;
      }
    }
  }
};

}  // namespace ringsim
