// rms_norm_backward.hip -- gradients of the root-mean-square norm.
//
// With r = 1 / sqrt(mean(h^2) + eps) and g = grad_out * w, for every row
//   grad_in = grad_residual + r g - h r^3 mean(g h)
// and over all rows  grad_weight = sum of grad_out h r.
// One pass reads each row once: both sums over the row (h^2 and g h) are taken
// together, r is recomputed from h rather than stored by the forward call
// (the row is here anyway), and every lane adds its columns' part of
// grad_weight into registers over all rows its workgroup walks. Workgroups
// leave these sums in a workspace, and a second small kernel adds them in a
// fixed order: no atomics, the same bits every time.
#include <algorithm>

#include "ops_device.h"

namespace ringsim {

template <int DT, int TPR, int NP, int LK>
__global__ void __launch_bounds__(TPR < 256 ? 256 : TPR) rms_norm_backward_kernel(RmsNormBackwardArgs a) {
  constexpr int kBlock = TPR < 256 ? 256 : TPR;
  constexpr int kRows = kBlock / TPR;
  using T = typename OpElem<DT>::T;
  __shared__ float sums_hh[2][16];
  __shared__ float sums_gh[2][16];
  __shared__ float dws[kRows > 1 ? kRows : 1][kRows > 1 ? TPR * NP * kPack : 1];
  const int t = threadIdx.x % TPR;
  int turn_hh = 0, turn_gh = 0;
  WeightPack w[NP];
  float dw[NP][kPack];
#pragma unroll
  for (int k = 0; k < NP; ++k) {
    w[k] = load_weight<DT, LK>(a.weight, a.weight_kind, (k * TPR + t) * kPack, a.cols);
#pragma unroll
    for (int i = 0; i < kPack; ++i) dw[k][i] = 0.0f;
  }
  for (uint32_t row = blockIdx.x * kRows + threadIdx.x / TPR; row < a.rows; row += gridDim.x * kRows) {
    const uint32_t o = a.inner == 1 ? row : row / a.inner, in = a.inner == 1 ? 0 : row - o * a.inner;
    Pack<DT> dy[NP], h[NP], res[NP];
    const T* pdy = row_ptr<DT>(a.grad_out, o, in);
    const T* ph = row_ptr<DT>(a.h, o, in);
#pragma unroll
    for (int k = 0; k < NP; ++k) {
      const int c = (k * TPR + t) * kPack;
      dy[k] = load_pack<DT, LK>(pdy, c, a.cols);
      h[k] = load_pack<DT, LK>(ph, c, a.cols);
    }
    if (a.grad_residual.p) {
      const T* pr = row_ptr<DT>(a.grad_residual, o, in);
#pragma unroll
      for (int k = 0; k < NP; ++k) res[k] = load_pack<DT, LK>(pr, (k * TPR + t) * kPack, a.cols);
    }
    float g[NP][kPack], hh = 0.0f, gh = 0.0f;
#pragma unroll
    for (int k = 0; k < NP; ++k) {
      const int c = (k * TPR + t) * kPack;
      float fh[kPack], fw[kPack];
      fix_pack<DT, LK>(h[k], c, a.cols);
      fix_pack<DT, LK>(dy[k], c, a.cols);
      unpack<DT>(h[k], fh);
      unpack<DT>(dy[k], g[k]);
      unpack_weight<DT, LK>(w[k], a.weight_kind, c, a.cols, fw);
#pragma unroll
      for (int i = 0; i < kPack; ++i) {
        g[k][i] *= fw[i];
        hh = __builtin_fmaf(fh[i], fh[i], hh);
        gh = __builtin_fmaf(g[k][i], fh[i], gh);
      }
    }
    hh = row_reduce<TPR, AddF32>(hh, sums_hh, turn_hh);
    gh = row_reduce<TPR, AddF32>(gh, sums_gh, turn_gh);
    const float r = rsqrtf(__builtin_fmaf(hh, a.inv_cols, a.eps));
    const float m = r * r * r * (gh * a.inv_cols);
    T* pout = row_ptr<T>(a.grad_in, o, in);
#pragma unroll
    for (int k = 0; k < NP; ++k) {
      const int c = (k * TPR + t) * kPack;
      float fh[kPack], fdy[kPack];
      unpack<DT>(h[k], fh);
      unpack<DT>(dy[k], fdy);
#pragma unroll
      for (int i = 0; i < kPack; ++i) {
        g[k][i] = g[k][i] * r - fh[i] * m;
        dw[k][i] = __builtin_fmaf(fdy[i], fh[i] * r, dw[k][i]);
      }
      if (a.grad_residual.p) {
        float fr[kPack];
        fix_pack<DT, LK>(res[k], c, a.cols);
        unpack<DT>(res[k], fr);
#pragma unroll
        for (int i = 0; i < kPack; ++i) g[k][i] += fr[i];
      }
      store_pack<DT>(pout, to_pack<DT>(g[k]), c, a.cols);
    }
  }
  if (!a.partial) return;
  float* part = a.partial + (int64_t)blockIdx.x * a.cols;
  if constexpr (kRows == 1) {
#pragma unroll
    for (int k = 0; k < NP; ++k) {
      const int c = (k * TPR + t) * kPack;
      store_pack<RINGSIM_FLOAT32>(part, to_pack<RINGSIM_FLOAT32>(dw[k]), c, a.cols);
    }
  } else {
    float* mine = dws[threadIdx.x / TPR];
#pragma unroll
    for (int k = 0; k < NP; ++k) {
#pragma unroll
      for (int i = 0; i < kPack; ++i) mine[(k * TPR + t) * kPack + i] = dw[k][i];
    }
    __syncthreads();
    for (int c = threadIdx.x; c < a.cols; c += kBlock) {
      float sum = dws[0][c];
#pragma unroll
      for (int i = 1; i < kRows; ++i) sum += dws[i][c];
      part[c] = sum;
    }
  }
}

// grad_weight[c] = sum over `parts` rows of partial. A workgroup takes 16
// columns: 16 lanes side by side read a 64-byte line of a row, 64 such groups
// share the rows out, and their sums are added through LDS in a fixed order.
constexpr int kSumCols = 16;
constexpr int kSumSlices = 64;
__global__ void __launch_bounds__(kSumCols * kSumSlices)
    rms_norm_weight_sum_kernel(const float* partial, int parts, int cols, void* out, int dtype) {
  __shared__ float s[kSumSlices][kSumCols + 1];
  const int t = threadIdx.x % kSumCols, slice = threadIdx.x / kSumCols;
  const int c = blockIdx.x * kSumCols + t;
  float sum = 0.0f;
  if (c < cols) {
#pragma unroll 4
    for (int p = slice; p < parts; p += kSumSlices) sum += partial[(int64_t)p * cols + c];
  }
  s[slice][t] = sum;
  __syncthreads();
#pragma unroll
  for (int half = kSumSlices / 2; half > 0; half /= 2) {
    if (slice < half) s[slice][t] += s[slice + half][t];
    __syncthreads();
  }
  if (slice != 0 || c >= cols) return;
  sum = s[0][t];
  if (dtype == RINGSIM_FLOAT32)
    static_cast<float*>(out)[c] = sum;
  else if (dtype == RINGSIM_BFLOAT16)
    static_cast<uint16_t*>(out)[c] = f32_to_elem<RINGSIM_BFLOAT16>(sum);
  else
    static_cast<uint16_t*>(out)[c] = f32_to_elem<RINGSIM_FLOAT16>(sum);
}

RowShape norm_backward_shape(int64_t rows, int64_t cols) {
  const int64_t packs = (cols + kPack - 1) / kPack;
  if (packs <= 16) return {16, 1};
  if (packs <= 64) return {64, 1};
  if (packs <= 128) return {64, 2};
  if (packs <= 256) return {256, 1};
  if (packs <= 512) return {256, 2};
  if (packs <= 1024) return {512, 2};
  if (packs <= 2048) return {1024, 2};
  return {1024, 4};
}

int norm_backward_workgroups(int64_t rows, int64_t cols) {
  const RowShape sh = norm_backward_shape(rows, cols);
  const int block = sh.lanes < 256 ? 256 : sh.lanes;
  const int64_t at_once = block / sh.lanes;
  // As many workgroups as fill the waves of two workgroups of 256 a compute unit.
  const int64_t most = (int64_t)kComputeUnits * 512 / block;
  return (int)std::max<int64_t>(1, std::min(most, (rows + at_once - 1) / at_once));
}

template <int DT, int TPR, int NP, int LK>
static hipError_t launch_kind(const RmsNormBackwardArgs& a, hipStream_t s) {
  hipLaunchKernelGGL((rms_norm_backward_kernel<DT, TPR, NP, LK>), dim3(norm_backward_workgroups(a.rows, a.cols)),
                     dim3(TPR < 256 ? 256 : TPR), 0, s, a);
  return hipGetLastError();
}

template <int DT, int TPR, int NP>
static hipError_t launch_shape(const RmsNormBackwardArgs& a, hipStream_t s) {
  const int64_t bytes =
      (int64_t)a.rows * a.cols * (int64_t)sizeof(typename OpElem<DT>::T) * (a.grad_residual.p ? 4 : 3);
  return bytes > kStreamBytes ? launch_kind<DT, TPR, NP, kLoadStream>(a, s)
                              : launch_kind<DT, TPR, NP, kLoadCached>(a, s);
}

template <int DT>
static hipError_t launch_type(const RmsNormBackwardArgs& a, hipStream_t s) {
  if (a.cols < kPack) return launch_kind<DT, 16, 1, kLoadShort>(a, s);
  const RowShape sh = norm_backward_shape(a.rows, a.cols);
  switch (sh.lanes * 16 + sh.packs) {
    case 16 * 16 + 1: return launch_shape<DT, 16, 1>(a, s);
    case 64 * 16 + 1: return launch_shape<DT, 64, 1>(a, s);
    case 64 * 16 + 2: return launch_shape<DT, 64, 2>(a, s);
    case 256 * 16 + 1: return launch_shape<DT, 256, 1>(a, s);
    case 256 * 16 + 2: return launch_shape<DT, 256, 2>(a, s);
    case 512 * 16 + 2: return launch_shape<DT, 512, 2>(a, s);
    case 1024 * 16 + 2: return launch_shape<DT, 1024, 2>(a, s);
    case 1024 * 16 + 4: return launch_shape<DT, 1024, 4>(a, s);
    default: return hipErrorInvalidValue;
  }
}

hipError_t launch_rms_norm_backward(const RmsNormBackwardArgs& a, int dtype, hipStream_t s) {
  switch (dtype) {
    case RINGSIM_FLOAT32: return launch_type<RINGSIM_FLOAT32>(a, s);
    case RINGSIM_BFLOAT16: return launch_type<RINGSIM_BFLOAT16>(a, s);
    case RINGSIM_FLOAT16: return launch_type<RINGSIM_FLOAT16>(a, s);
    default: return hipErrorInvalidValue;
  }
}

hipError_t launch_rms_norm_weight_sum(const float* partial, int parts, int cols, void* grad_weight, int dtype,
                                      hipStream_t s) {
  hipLaunchKernelGGL(rms_norm_weight_sum_kernel, dim3((cols + kSumCols - 1) / kSumCols), dim3(kSumCols * kSumSlices),
                     0, s, partial, parts, cols, grad_weight, dtype);
  return hipGetLastError();
}

}  // namespace ringsim
