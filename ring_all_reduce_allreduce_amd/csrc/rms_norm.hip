// rms_norm.hip -- root-mean-square norm of rows, forward.
//
// For every row:  h = x (+ residual),  y = h / sqrt(mean(h^2) + eps) * w,
// y in the input's type or in 8 bits with scales. The row is read once: its
// lanes keep h in registers as fp32 between the sum of squares and the
// product. What bounds it is memory: 4 x 2 bytes an element in bf16 with a
// residual (x, residual, h, y) against about 6 operations.
//
// One row (or the rows of one workgroup's lanes) a workgroup, no loop: all
// loads of a row, the weights among them, are under way at once, and the
// hardware starts the next workgroup while this one waits at its barrier.
// Workgroups that walked rows with the weights kept in registers took 94
// against 78 us for 8192 rows of 8192 into 8 bits, 13.5 against 10.2 us for
// 1021 rows of 5119, and one more memory latency for a single row.
#include <algorithm>

#include "ops_device.h"

namespace ringsim {

template <int DT, int TPR, int NP, bool Q, int LK>
__global__ void __launch_bounds__(kMaxBlock<TPR>) rms_norm_kernel(RmsNormArgs a) {
  constexpr int kRows = kRowsPerBlock<TPR>;
  constexpr int kPack = OpElem<DT>::kPack;
  using T = typename OpElem<DT>::T;
  __shared__ RowBuffers<TPR, float> sums;
  __shared__ RowBuffers<TPR, uint32_t> tops;
  sums.clear();
  if constexpr (Q) tops.clear();
  int turn = 0, qturn = 0;
  const int lanes = row_lanes<TPR>(), t = TPR <= 64 ? threadIdx.x % TPR : threadIdx.x;
  const auto column = [&](int k) { return (k * lanes + t) * kPack; };  // first of pack k
  const uint32_t row = (blockIdx.y * gridDim.x + blockIdx.x) * kRows + (TPR <= 64 ? threadIdx.x / TPR : 0);
  if (row >= a.rows) return;  // the same for all lanes of a row
  const uint32_t o = a.inner == 1 ? row : row / a.inner, in = a.inner == 1 ? 0 : row - o * a.inner;
  float h[NP][kPack];
  u32x4 x[NP], res[NP];
  WeightPack w[NP];
  const T* px = row_ptr<DT>(a.x, o, in);
#pragma unroll
  for (int k = 0; k < NP; ++k) x[k] = load_pack<DT, LK>(px, column(k), a.cols);
  if (a.residual.p) {
    const T* pr = row_ptr<DT>(a.residual, o, in);
#pragma unroll
    for (int k = 0; k < NP; ++k) res[k] = load_pack<DT, LK>(pr, column(k), a.cols);
  }
#pragma unroll
  for (int k = 0; k < NP; ++k) w[k] = load_weight<DT, LK>(a.weight, a.weight_kind, column(k), a.cols);
#pragma unroll
  for (int k = 0; k < NP; ++k) unpack<DT>(fix_pack<DT, LK>(x[k], column(k), a.cols), h[k]);
  if (a.residual.p) {
    T* ph = row_ptr<T>(a.residual_out, o, in);
#pragma unroll
    for (int k = 0; k < NP; ++k) {
      const int c = column(k);
      float f[kPack];
      unpack<DT>(fix_pack<DT, LK>(res[k], c, a.cols), f);
#pragma unroll
      for (int i = 0; i < kPack; ++i) h[k][i] += f[i];
      store_pack<DT>(ph, to_pack<DT>(h[k]), c, a.cols);
    }
  }
  float ss = 0.0f;
#pragma unroll
  for (int k = 0; k < NP; ++k) {
#pragma unroll
    for (int i = 0; i < kPack; ++i) ss = __builtin_fmaf(h[k][i], h[k][i], ss);
  }
  ss = row_reduce<TPR, AddF32>(ss, sums, turn);
  const float r = rsqrtf(__builtin_fmaf(ss, a.inv_cols, a.eps));
#pragma unroll
  for (int k = 0; k < NP; ++k) {
    float fw[kPack];
    unpack_weight<DT, LK>(w[k], a.weight_kind, column(k), a.cols, fw);
#pragma unroll
    for (int i = 0; i < kPack; ++i) h[k][i] = h[k][i] * r * fw[i];
  }
  if constexpr (!Q) {
    T* py = row_ptr<T>(a.out, o, in);
#pragma unroll
    for (int k = 0; k < NP; ++k) store_pack<DT>(py, to_pack<DT>(h[k]), column(k), a.cols);
  } else {
    // Largest |y| of the row, or of the lanes that hold a group: groups start
    // at multiples of their width, lanes beyond the row hold 0.
    uint32_t top[NP];
#pragma unroll
    for (int k = 0; k < NP; ++k) {
      const int c = column(k);
      top[k] = 0;
#pragma unroll
      for (int i = 0; i < kPack; ++i)
        if (c + i < a.cols) top[k] = MaxBits::of(top[k], __float_as_uint(h[k][i]) & 0x7fffffffu);
    }
    if (a.group == 0) {
#pragma unroll
      for (int k = 1; k < NP; ++k) top[0] = MaxBits::of(top[0], top[k]);
      top[0] = row_reduce<TPR, MaxBits>(top[0], tops, qturn);
#pragma unroll
      for (int k = 1; k < NP; ++k) top[k] = top[0];
    } else {
      const int wide = a.group / kPack;  // lanes of a group: 4 to 32 (a row of 16 is shorter than a group of 32)
#pragma unroll
      for (int k = 0; k < NP; ++k) {
        top[k] = lanes_reduce<4, MaxBits>(top[k]);
        if (wide >= 8) top[k] = MaxBits::of(top[k], dpp<0x141>(top[k]));
        if (wide >= 16) top[k] = MaxBits::of(top[k], dpp<0x140>(top[k]));
        if constexpr (TPR >= 32 && DT == RINGSIM_FLOAT32) {
          if (wide >= 32) top[k] = swap16_reduce<MaxBits>(top[k]);
        }
      }
    }
    uint8_t* py = row_ptr<uint8_t>(a.out, o, in);
    float* ps = a.scales + (int64_t)row * a.groups;
#pragma unroll
    for (int k = 0; k < NP; ++k) {
      const int c = column(k);
      // Not fmaxf, which would drop a NaN.
      float scale = __uint_as_float(top[k]) / 448.0f;
      scale = scale < 0x1p-126f ? 0x1p-126f : scale;
      if (a.group == 0) {
        if (k == 0 && t == 0) ps[0] = scale;
      } else if (c < a.cols && c % a.group == 0) {
        ps[c / a.group] = scale;
      }
      // |y| * inv is at most 448 (1 + 2^-22), which rounds to 448, the
      // largest e4m3 value: nothing to clamp.
      const float inv = 1.0f / scale;
      uint32_t b[kPack / 4];
#pragma unroll
      for (int j = 0; j < kPack / 4; ++j) {
        int v = 0;
        v = __builtin_amdgcn_cvt_pk_fp8_f32(h[k][4 * j] * inv, h[k][4 * j + 1] * inv, v, false);
        v = __builtin_amdgcn_cvt_pk_fp8_f32(h[k][4 * j + 2] * inv, h[k][4 * j + 3] * inv, v, true);
        b[j] = (uint32_t)v;
      }
      if (c + kPack <= a.cols) {
        if constexpr (kPack == 8)
          *reinterpret_cast<u32x2_e1*>(py + c) = u32x2{b[0], b[1]};
        else
          *reinterpret_cast<u32_e1*>(py + c) = b[0];
      } else {
#pragma unroll
        for (int i = 0; i < kPack - 1; ++i)
          if (c + i < a.cols) py[c + i] = (uint8_t)(b[i / 4] >> (8 * (i % 4)));
      }
    }
  }
}

template <int DT, int TPR, int NP, int LK>
static hipError_t launch_kind(const RmsNormArgs& a, int lanes, hipStream_t s) {
  constexpr int kRows = kRowsPerBlock<TPR>;
  const int64_t need = ((int64_t)a.rows + kRows - 1) / kRows;
  // A dimension of a grid holds below 2^32 threads.
  const unsigned gx = (unsigned)std::min<int64_t>(need, 1 << 20);
  const dim3 grid(gx, (unsigned)((need + gx - 1) / gx)), block(lanes * kRows);
  if (a.scales)
    hipLaunchKernelGGL((rms_norm_kernel<DT, TPR, NP, true, LK>), grid, block, 0, s, a);
  else
    hipLaunchKernelGGL((rms_norm_kernel<DT, TPR, NP, false, LK>), grid, block, 0, s, a);
  return hipGetLastError();
}

template <int DT, int TPR, int NP>
static hipError_t launch_shape(const RmsNormArgs& a, int lanes, hipStream_t s) {
  const int64_t bytes = (int64_t)a.rows * a.cols * (int64_t)sizeof(typename OpElem<DT>::T) * (a.residual.p ? 4 : 2);
  return bytes > kStreamBytes ? launch_kind<DT, TPR, NP, kLoadStream>(a, lanes, s)
                              : launch_kind<DT, TPR, NP, kLoadCached>(a, lanes, s);
}

// Lanes by the packs of a row: a part of a wave, a wave, or as many whole
// waves as `np` packs a lane leave. TODO
template <int DT>
static hipError_t launch_type(const RmsNormArgs& a, hipStream_t s) {
  constexpr int kPack = OpElem<DT>::kPack;
  if (a.cols < kPack) return launch_kind<DT, 16, 1, kLoadShort>(a, 16, s);
  const int packs = (a.cols + kPack - 1) / kPack;
  const auto lanes = [&](int np) { return (packs + 64 * np - 1) / (64 * np) * 64; };
  if (packs <= 16) return launch_shape<DT, 16, 1>(a, 16, s);
  if (packs <= 32) return launch_shape<DT, 32, 1>(a, 32, s);
  if (packs <= 64) return launch_shape<DT, 64, 1>(a, 64, s);
  if (packs <= 128) return launch_shape<DT, 64, 2>(a, 64, s);
  if (packs <= 256) return launch_shape<DT, 256, 1>(a, lanes(1), s);
  if (packs <= 1024) return launch_shape<DT, 512, 2>(a, lanes(2), s);
  if (packs <= 2048) return launch_shape<DT, 1024, 2>(a, lanes(2), s);
  if (packs <= 4096) return launch_shape<DT, 1024, 4>(a, lanes(4), s);
  if constexpr (DT == RINGSIM_FLOAT32) return launch_shape<DT, 1024, 8>(a, lanes(8), s);
  return hipErrorInvalidValue;
}

hipError_t launch_rms_norm(const RmsNormArgs& a, int dtype, hipStream_t s) {
  switch (dtype) {
    case RINGSIM_FLOAT32: return launch_type<RINGSIM_FLOAT32>(a, s);
    case RINGSIM_BFLOAT16: return launch_type<RINGSIM_BFLOAT16>(a, s);
    case RINGSIM_FLOAT16: return launch_type<RINGSIM_FLOAT16>(a, s);
    default: return hipErrorInvalidValue;
  }
}

}  // namespace ringsim
