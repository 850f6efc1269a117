// grad_norm.hip -- the 2-norm of many gradients together, and the clipping by
// it.
//
//   norm = |scale| sqrt(sum g^2),  out = g * scale * min(1, max_norm / (norm + eps))
// A launch walks all tensors of its table: each is cut into tiles of 16 KiB,
// and the workgroups walk the tiles of all tensors with one stride. Squares
// are summed in fp64: the product of two fp32 values is exact there and
// cannot leave its range, and the vector unit's fp64 rate is several times
// what the memory delivers. Workgroups leave one sum each; whoever needs the
// norm adds these in a fixed order, so no atomics and the same bits every
// time. Both kernels are bound by memory.
#include <algorithm>

#include "ops_device.h"

namespace ringsim {

constexpr int kWaves = kThreads / 64;

struct GradTile {
  int tensor;
  int64_t first;  // element of the tensor the tile starts at
  int n;          // its elements
};

__device__ __forceinline__ int tile_elems(int dtype) {
  return dtype == RINGSIM_FLOAT32 ? kGradTileBytes / 4 : kGradTileBytes / 2;
}

// The tensor that holds tile t: the last one whose first tile is <= t and
// that has any.
__device__ __forceinline__ GradTile find_tile(const GradTable& tab, uint32_t t) {
  int lo = 0, hi = tab.ntensors;
  while (hi - lo > 1) {
    const int mid = (lo + hi) / 2;
    if (tab.tile0[mid] <= t)
      lo = mid;
    else
      hi = mid;
  }
  const int elems = tile_elems(tab.dtype[lo]);
  const uint32_t k = t - tab.tile0[lo];
  return GradTile{lo, (int64_t)k * elems, t + 1 == tab.tile0[lo + 1] ? (int)tab.last[lo] : elems};
}

template <int DT>
__device__ __forceinline__ double tile_squares(const void* base, int64_t first, int n) {
  using T = typename OpElem<DT>::T;
  const T* p = static_cast<const T*>(base) + first;
  constexpr int kPacks = kGradTileBytes / (int)sizeof(T) / (kThreads * kPack);
  Pack<DT> v[kPacks];
#pragma unroll
  for (int k = 0; k < kPacks; ++k) {
    const int c = (k * kThreads + (int)threadIdx.x) * kPack;
    v[k] = load_pack<DT>(p + c, n - c);
  }
  double s = 0.0;
#pragma unroll
  for (int k = 0; k < kPacks; ++k) {
    float f[kPack];
    unpack<DT>(v[k], f);
#pragma unroll
    for (int i = 0; i < kPack; ++i) s = __builtin_fma((double)f[i], (double)f[i], s);
  }
  return s;
}

// Sum over the workgroup, known to every thread; the order is fixed.
__device__ __forceinline__ double block_sum(double v, double* lds) {
#pragma unroll
  for (int m = 1; m < 64; m *= 2) v += __shfl_xor(v, m, 64);
  if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = v;
  __syncthreads();
  v = lds[0];
#pragma unroll
  for (int i = 1; i < kWaves; ++i) v += lds[i];
  return v;
}

__global__ void __launch_bounds__(kThreads) grad_squares_kernel(GradTable tab, double* partial) {
  __shared__ double lds[kWaves];
  const uint32_t tiles = tab.tile0[tab.ntensors];
  double s = 0.0;
  for (uint32_t t = blockIdx.x; t < tiles; t += gridDim.x) {
    const GradTile g = find_tile(tab, t);
    switch (tab.dtype[g.tensor]) {
      case RINGSIM_FLOAT32: s += tile_squares<RINGSIM_FLOAT32>(tab.in[g.tensor], g.first, g.n); break;
      case RINGSIM_BFLOAT16: s += tile_squares<RINGSIM_BFLOAT16>(tab.in[g.tensor], g.first, g.n); break;
      default: s += tile_squares<RINGSIM_FLOAT16>(tab.in[g.tensor], g.first, g.n); break;
    }
  }
  s = block_sum(s, lds);
  if (threadIdx.x == 0) partial[blockIdx.x] = s;
}

// The norm from the workgroups' sums, in fp32, known to every thread.
__device__ __forceinline__ float join_norm(const double* partial, int parts, float scale, double* lds) {
  double s = 0.0;
  for (int i = threadIdx.x; i < parts; i += kThreads) s += partial[i];
  s = block_sum(s, lds);
  return (float)(__builtin_fabs((double)scale) * __builtin_sqrt(s));
}

__global__ void __launch_bounds__(kThreads) grad_norm_join_kernel(const double* partial, int parts, float scale,
                                                                  float* norm) {
  __shared__ double lds[kWaves];
  const float v = join_norm(partial, parts, scale, lds);
  if (threadIdx.x == 0) *norm = v;
}

template <int DT>
__device__ __forceinline__ void tile_scale(const void* in, void* out, int64_t first, int n, float f) {
  using T = typename OpElem<DT>::T;
  const T* p = static_cast<const T*>(in) + first;
  T* q = static_cast<T*>(out) + first;
  constexpr int kPacks = kGradTileBytes / (int)sizeof(T) / (kThreads * kPack);
  Pack<DT> v[kPacks];
#pragma unroll
  for (int k = 0; k < kPacks; ++k) {
    const int c = (k * kThreads + (int)threadIdx.x) * kPack;
    v[k] = load_pack<DT>(p + c, n - c);
  }
#pragma unroll
  for (int k = 0; k < kPacks; ++k) {
    const int c = (k * kThreads + (int)threadIdx.x) * kPack;
    float e[kPack];
    unpack<DT>(v[k], e);
#pragma unroll
    for (int i = 0; i < kPack; ++i) e[i] *= f;
    store_pack<DT>(q + c, to_pack<DT>(e), n - c);
  }
}

// Walks the tiles from the last to the first: what the norm's pass read last
// is still in the Infinity Cache.
__global__ void __launch_bounds__(kThreads) grad_scale_kernel(GradTable tab, GradFactor fac, int in_place) {
  __shared__ double lds[kWaves];
  float norm;
  if (fac.partial) {
    norm = join_norm(fac.partial, fac.parts, fac.scale, lds);
    if (fac.norm && blockIdx.x == 0 && threadIdx.x == 0) *fac.norm = norm;
  } else {
    norm = *fac.norm;
  }
  // One rounding, of the whole factor. A NaN norm fails the comparison the
  // other way and stays.
  double c = (double)fac.max_norm / ((double)norm + (double)fac.eps);
  c = c > 1.0 ? 1.0 : c;
  const float f = (float)(c * (double)fac.scale);
  if (in_place && f == 1.0f) return;
  const uint32_t tiles = tab.tile0[tab.ntensors];
  for (uint32_t t = blockIdx.x; t < tiles; t += gridDim.x) {
    const GradTile g = find_tile(tab, tiles - 1 - t);
    switch (tab.dtype[g.tensor]) {
      case RINGSIM_FLOAT32: tile_scale<RINGSIM_FLOAT32>(tab.in[g.tensor], tab.out[g.tensor], g.first, g.n, f); break;
      case RINGSIM_BFLOAT16: tile_scale<RINGSIM_BFLOAT16>(tab.in[g.tensor], tab.out[g.tensor], g.first, g.n, f); break;
      default: tile_scale<RINGSIM_FLOAT16>(tab.in[g.tensor], tab.out[g.tensor], g.first, g.n, f); break;
    }
  }
}

hipError_t launch_grad_squares(const GradTable& t, double* partial, int workgroups, hipStream_t s) {
  hipLaunchKernelGGL(grad_squares_kernel, dim3(workgroups), dim3(kThreads), 0, s, t, partial);
  return hipGetLastError();
}

hipError_t launch_grad_norm_join(const double* partial, int parts, float scale, float* norm, hipStream_t s) {
  hipLaunchKernelGGL(grad_norm_join_kernel, dim3(1), dim3(kThreads), 0, s, partial, parts, scale, norm);
  return hipGetLastError();
}

hipError_t launch_grad_scale(const GradTable& t, const GradFactor& f, int in_place, int workgroups, hipStream_t s) {
  hipLaunchKernelGGL(grad_scale_kernel, dim3(workgroups), dim3(kThreads), 0, s, t, f, in_place);
  return hipGetLastError();
}

}  // namespace ringsim
