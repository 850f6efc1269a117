// rms_norm.hip -- root-mean-square norm of rows, forward.
//
// For every row:  h = x (+ residual),  y = h / sqrt(mean(h^2) + eps) * w,
// y in the input's type or in 8 bits with scales. The row is read once: its
// lanes keep h in registers as fp32 between the sum of squares and the
// product. What bounds it is memory: 4 x 2 bytes an element in bf16 with a
// residual (x, residual, h, y) against about 6 operations. 4096 rows of 4096
// take 20.3 us, 6.6 TB/s, as fast as a copy of that size; one row 2.5 us.
//
// One row (or the rows of one workgroup's lanes) a workgroup, no loop: all
// loads of a row, the weights among them, are under way at once, and the
// hardware starts the next workgroup while this one waits at its barrier.
// Workgroups that walked rows with the weights kept in registers took 94
// against 78 us for 8192 rows of 8192 into 8 bits, 13.5 against 10.2 us for
// 1021 rows of 5119 (on four waves each; on the five they have now 8.4), and
// one more memory latency for a single row.
#include <algorithm>

#include "ops_device.h"

namespace ringsim {

// A row's part of a lane as it lies in memory.
template <int NP>
struct NormRow {
  u32x4 x[NP], res[NP];
};

// From four packs a lane on, which 1024 lanes with their 128 registers hold,
// the weights are read where they are used, two packs' at a time: 2048 rows of
// 32768 fp32 with a residual take 185 us so and 247 with all of them loaded
// before the sum, of bf16 94 and 98.
template <int NP>
constexpr bool kReadLate = NP >= 4;

template <int TPR>
struct NormShared {
  RowBuffers<TPR, float> sums;
  RowBuffers<TPR, uint32_t> tops;
};

template <int DT, int TPR, int NP, int LK>
__device__ __forceinline__ NormRow<NP> load_row(const RmsNormArgs& a, uint32_t row, int t) {
  constexpr int kPack = OpElem<DT>::kPack;
  const int lanes = row_lanes<TPR>();
  const uint32_t o = a.inner == 1 ? row : row / a.inner, in = a.inner == 1 ? 0 : row - o * a.inner;
  NormRow<NP> r;
  const auto* px = row_ptr<DT>(a.x, o, in);
#pragma unroll
  for (int k = 0; k < NP; ++k) r.x[k] = load_pack<DT, LK>(px, (k * lanes + t) * kPack, a.cols);
  if (a.residual.p) {
    const auto* pr = row_ptr<DT>(a.residual, o, in);
#pragma unroll
    for (int k = 0; k < NP; ++k) r.res[k] = load_pack<DT, LK>(pr, (k * lanes + t) * kPack, a.cols);
  }
  return r;
}

template <int DT, int TPR, int NP, bool Q, int LK>
__device__ __forceinline__ void take_row(const RmsNormArgs& a, const NormRow<NP>& in_row, WeightPack (&w)[NP],
                                         uint32_t row, int t, NormShared<TPR>& lds) {
  constexpr int kPack = OpElem<DT>::kPack;
  using T = typename OpElem<DT>::T;
  int turn = 0, qturn = 0;  // one reduction of each a row and workgroup above a wave
  const int lanes = row_lanes<TPR>();
  const auto column = [&](int k) { return (k * lanes + t) * kPack; };  // first of pack k
  const uint32_t o = a.inner == 1 ? row : row / a.inner, in = a.inner == 1 ? 0 : row - o * a.inner;
  float h[NP][kPack];
#pragma unroll
  for (int k = 0; k < NP; ++k) unpack<DT>(fix_pack<DT, LK>(in_row.x[k], column(k), a.cols), h[k]);
  if (a.residual.p) {
    T* ph = row_ptr<T>(a.residual_out, o, in);
#pragma unroll
    for (int k = 0; k < NP; ++k) {
      const int c = column(k);
      float f[kPack];
      unpack<DT>(fix_pack<DT, LK>(in_row.res[k], c, a.cols), f);
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
  ss = row_reduce<TPR, AddF32>(ss, lds.sums, turn);
  const float r = rsqrtf(__builtin_fmaf(ss, a.inv_cols, a.eps));
#pragma unroll
  for (int k = 0; k < NP; ++k) {
    float fw[kPack];
    if constexpr (kReadLate<NP>) {
      if (k % 2 == 0) asm volatile("" : "+v"(t) : "v"(r));  // not before r is known
      w[k] = load_weight<DT, LK>(a.weight, a.weight_kind, column(k), a.cols);
    }
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
      top[0] = row_reduce<TPR, MaxBits>(top[0], lds.tops, qturn);
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
      // One division a scale, one product an element, whose two roundings of
      // 2^-24 decide only which side a value next to a tie falls on (8 of 16
      // million). |y| * inv is at most 448 (1 + 2^-22), which rounds to 448,
      // the largest e4m3 value: nothing to clamp.
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

// NR rows for each of the workgroup's groups of lanes, their loads all at once.
template <int DT, int TPR, int NP, bool Q, int LK, int NR>
__global__ void __launch_bounds__(kMaxBlock<TPR>) rms_norm_kernel(RmsNormArgs a) {
  static_assert(NR == 1 || TPR <= 64, "several rows only where no barrier is needed");
  constexpr int kRows = kRowsPerBlock<TPR>;
  constexpr int kPack = OpElem<DT>::kPack;
  __shared__ NormShared<TPR> lds;
  lds.sums.clear();
  if constexpr (Q) lds.tops.clear();
  const int lanes = row_lanes<TPR>(), t = TPR <= 64 ? threadIdx.x % TPR : threadIdx.x;
  const uint32_t first = (blockIdx.y * gridDim.x + blockIdx.x) * (kRows * NR) + (TPR <= 64 ? threadIdx.x / TPR : 0);
  if (first >= a.rows) return;  // the same for all lanes of a row
  NormRow<NP> r[NR];
  WeightPack w[NP];
#pragma unroll
  for (int j = 0; j < NR; ++j) {
    const uint32_t row = first + j * kRows;
    r[j] = load_row<DT, TPR, NP, LK>(a, row < a.rows ? row : first, t);
  }
#pragma unroll
  for (int k = 0; k < NP; ++k) {
    if constexpr (!kReadLate<NP>) w[k] = load_weight<DT, LK>(a.weight, a.weight_kind, (k * lanes + t) * kPack, a.cols);
  }
#pragma unroll
  for (int j = 0; j < NR; ++j) {
    const uint32_t row = first + j * kRows;
    if (row < a.rows) take_row<DT, TPR, NP, Q, LK>(a, r[j], w, row, t, lds);
  }
}

template <int DT, int TPR, int NP, int LK, int NR>
static hipError_t launch_rows(const RmsNormArgs& a, int lanes, hipStream_t s) {
  constexpr int kRows = kRowsPerBlock<TPR>;
  const int64_t need = ((int64_t)a.rows + kRows * NR - 1) / (kRows * NR);
  // A dimension of a grid holds below 2^32 threads.
  const unsigned gx = (unsigned)std::min<int64_t>(need, 1 << 20);
  const dim3 grid(gx, (unsigned)((need + gx - 1) / gx)), block(lanes * kRows);
  if (a.scales)
    hipLaunchKernelGGL((rms_norm_kernel<DT, TPR, NP, true, LK, NR>), grid, block, 0, s, a);
  else
    hipLaunchKernelGGL((rms_norm_kernel<DT, TPR, NP, false, LK, NR>), grid, block, 0, s, a);
  return hipGetLastError();
}

// Rows of a wave's lanes or fewer are a few hundred bytes: two of them a group
// of lanes halve the workgroups, whose start is what such calls wait for, once
// there are four workgroups a compute unit all the same. 65536 rows of 128
// bf16: 7.0 us, one row 7.7, four 7.2; 10^6 rows of 64: 57.6, 67.5, 52.0; but
// with a residual four rows of 128 lose what two keep (into 8 bits 14.0 us,
// two 13.3, one 12.3).
constexpr int kShortRows = 2;

template <int DT, int TPR, int NP, int LK>
static hipError_t launch_kind(const RmsNormArgs& a, int lanes, hipStream_t s) {
  if constexpr (TPR <= 64 && NP == 1) {
    if (a.rows >= (uint32_t)(kComputeUnits * 4 * kShortRows * kRowsPerBlock<TPR>))
      return launch_rows<DT, TPR, NP, LK, kShortRows>(a, lanes, s);
  }
  return launch_rows<DT, TPR, NP, LK, 1>(a, lanes, s);
}

template <int DT, int TPR, int NP>
static hipError_t launch_shape(const RmsNormArgs& a, int lanes, hipStream_t s) {
  const int64_t bytes = (int64_t)a.rows * a.cols * (int64_t)sizeof(typename OpElem<DT>::T) * (a.residual.p ? 4 : 2);
  return bytes > kStreamBytes ? launch_kind<DT, TPR, NP, kLoadStream>(a, lanes, s)
                              : launch_kind<DT, TPR, NP, kLoadCached>(a, lanes, s);
}

// Lanes by the packs of a row: a part of a wave, a wave, or as many whole
// waves as `np` packs a lane leave. Few packs a lane keep short rows spread
// out; more of them, up to what 1024 lanes need, keep the waves that meet at
// the barrier few. 1021 rows of 5119 fp16 (640 packs) take 8.4 us on five
// waves and 9.8 on four of four packs, half of the last one empty; 4096 rows
// of 12288 bf16 into 8 bits (1536 packs) 59 us on 12 waves of two packs and
// 71 on six of four, whose registers leave fewer workgroups on a compute unit.
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
