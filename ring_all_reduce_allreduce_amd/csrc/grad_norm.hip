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
  int type;
  int bytes;      // of the tile
  bool small;     // the whole tensor is shorter than a vector
  int64_t first;  // byte of the tensor the tile starts at
};

// Finds a tile's tensor: lanes hold the first tiles of all tensors, one vote
// counts those at or below the tile. Two dependent loads at most, where a
// binary search over the table makes one for every doubling of it.
template <typename TABLE>
struct TileFinder {
  static constexpr int kPerLane = (TABLE::kTensors + 63) / 64;
  uint32_t first[kPerLane];

  __device__ __forceinline__ explicit TileFinder(const TABLE& tab) {
#pragma unroll
    for (int i = 0; i < kPerLane; ++i) {
      const int j = (int)(threadIdx.x & 63) + 64 * i;
      first[i] = j < tab.ntensors ? tab.tile0[j] : ~0u;
    }
  }

  __device__ __forceinline__ GradTile find(const TABLE& tab, uint32_t t) const {
    int k = -1;
#pragma unroll
    for (int i = 0; i < kPerLane; ++i) k += __builtin_popcountll(__builtin_amdgcn_ballot_w64(first[i] <= t));
    const uint32_t meta = tab.meta[k / 2] >> (16 * (k % 2)) & 0xffffu;
    const int type = (int)(meta >> kGradLastBits);
    const uint32_t from = tab.tile0[k], to = tab.tile0[k + 1];
    const int last = (int)(meta & ((1u << kGradLastBits) - 1)) * (type == kGradF32 ? 4 : 2);
    return GradTile{k, type, t + 1 == to ? last : kGradTileBytes, to - from == 1 && last < 16,
                    (int64_t)(t - from) * kGradTileBytes};
  }
};

// A tile in registers: four 16-byte vectors a thread, whatever the type.
constexpr int kTileVecs = kGradTileBytes / 16 / kThreads;
struct TileData {
  u32x4 v[kTileVecs];
};

__device__ __forceinline__ int vec_at(int i) { return (i * kThreads + (int)threadIdx.x) * 16; }

template <int LK>
__device__ __forceinline__ TileData load_tile(const char* tile, int bytes) {
  TileData d;
#pragma unroll
  for (int i = 0; i < kTileVecs; ++i) d.v[i] = load16<LK>(tile, vec_at(i), bytes);
  return d;
}

__device__ __forceinline__ void fix_tile(TileData& d, int bytes) {
#pragma unroll
  for (int i = 0; i < kTileVecs; ++i) d.v[i] = fix16<kLoadCached>(d.v[i], vec_at(i), bytes);
}

template <int DT>
__device__ __forceinline__ void vec_to_f32(u32x4 v, float* f) {
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

template <int DT>
__device__ __forceinline__ double tile_squares(const TileData& d) {
  double s = 0.0;
#pragma unroll
  for (int i = 0; i < kTileVecs; ++i) {
    float f[OpElem<DT>::kPerVec];
    vec_to_f32<DT>(d.v[i], f);
#pragma unroll
    for (int j = 0; j < OpElem<DT>::kPerVec; ++j) s = __builtin_fma((double)f[j], (double)f[j], s);
  }
  return s;
}

__device__ __forceinline__ double squares_of(const TileData& d, int type) {
  switch (type) {
    case kGradF32: return tile_squares<RINGSIM_FLOAT32>(d);
    case kGradBF16: return tile_squares<RINGSIM_BFLOAT16>(d);
    default: return tile_squares<RINGSIM_FLOAT16>(d);
  }
}

// Element i of a tensor of any type.
__device__ __forceinline__ float grad_elem(const void* p, int type, int i) {
  if (type == kGradF32) return static_cast<const float*>(p)[i];
  const uint16_t e = static_cast<const uint16_t*>(p)[i];
  return type == kGradBF16 ? elem_to_f32<RINGSIM_BFLOAT16>(e) : elem_to_f32<RINGSIM_FLOAT16>(e);
}

// The squares of tiles t, t + step, ... below `end`; t is left at the first
// one at or past it. One tile ahead: the next one's loads are under way
// while this one's squares are added (40 buckets of 25 MiB: 160 us, without
// 166). The two tiles take turns in two sets of registers, since moving a
// loaded vector waits for it, and the loads stand under no condition, since a
// wait that some path reaches without them waits for everything: where there
// is no next tile, and for a tensor shorter than a vector, the lanes read 16
// bytes of `spare` for nothing. Such a tensor's elements are read when its
// turn comes.
template <int LK>
__device__ __forceinline__ double walk_squares(const GradSquareTable& tab, const TileFinder<GradSquareTable>& finder,
                                               uint32_t& t, uint32_t end, uint32_t step, const void* spare) {
  if (t >= end) return 0.0;
  const auto load = [&](const GradTile& g, bool wanted) {
    const bool real = wanted && !g.small;
    const char* p = static_cast<const char*>(real ? tab.in[g.tensor] : spare) + (real ? g.first : 0);
    return load_tile<LK>(p, real ? g.bytes : 16);
  };
  const auto squares = [&](TileData& d, const GradTile& g) {
    if (g.small) {
      const int i = threadIdx.x, n = g.bytes / (g.type == kGradF32 ? 4 : 2);
      const double e = i < n ? (double)grad_elem(tab.in[g.tensor], g.type, i) : 0.0;
      return e * e;
    }
    if (g.bytes != kGradTileBytes) fix_tile(d, g.bytes);
    return squares_of(d, g.type);
  };
  double s = 0.0;
  GradTile ga = finder.find(tab, t), gb;
  TileData da = load(ga, true), db;
  for (;;) {
    t += step;
    gb = finder.find(tab, t < end ? t : end - 1);
    db = load(gb, t < end);
    s += squares(da, ga);
    if (t >= end) return s;
    t += step;
    ga = finder.find(tab, t < end ? t : end - 1);
    da = load(ga, t < end);
    s += squares(db, gb);
    if (t >= end) return s;
  }
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

__global__ void __launch_bounds__(kThreads)
    grad_squares_kernel(GradSquareTable tab, uint32_t keep, double* partial) {
  __shared__ double lds[kWaves];
  const uint32_t tiles = tab.tile0[tab.ntensors];
  const TileFinder<GradSquareTable> finder(tab);
  uint32_t t = blockIdx.x;
  double s = walk_squares<kLoadStream>(tab, finder, t, tiles - keep, gridDim.x, partial);
  s += walk_squares<kLoadCached>(tab, finder, t, tiles, gridDim.x, partial);
  s = block_sum(s, lds);
  if (threadIdx.x == 0) partial[blockIdx.x] = s;
}

// The norm from the workgroups' sums, in fp32, known to every thread.
__device__ __forceinline__ float join_norm(const double* partial, int parts, float scale, double* lds) {
  // Eight loads at a time before the first addition: one memory latency for
  // the sums of a launch, not one for each of a thread's additions.
  constexpr int kAhead = 8;
  double s = 0.0;
  for (int base = threadIdx.x; base < parts; base += kAhead * kThreads) {
    double v[kAhead];
#pragma unroll
    for (int i = 0; i < kAhead; ++i) v[i] = base + i * kThreads < parts ? partial[base + i * kThreads] : 0.0;
#pragma unroll
    for (int i = 0; i < kAhead; ++i) s += v[i];
  }
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
__device__ __forceinline__ void tile_scale(const TileData& d, int bytes, char* out, float factor) {
#pragma unroll
  for (int i = 0; i < kTileVecs; ++i) {
    float f[OpElem<DT>::kPerVec];
    vec_to_f32<DT>(d.v[i], f);
#pragma unroll
    for (int j = 0; j < OpElem<DT>::kPerVec; ++j) f[j] *= factor;
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
    store16(out, v, vec_at(i), bytes);
  }
}

// Walks the tiles from the last to the first: what the norm's pass read last
// is still in the Infinity Cache.
__global__ void __launch_bounds__(kThreads) grad_scale_kernel(GradScaleTable tab, GradFactor fac, int in_place) {
  __shared__ double lds[kWaves];
  const TileFinder<GradScaleTable> finder(tab);
  float norm;
  if (fac.partial) {
    norm = join_norm(fac.partial, fac.parts, fac.scale, lds);
    if (fac.norm && blockIdx.x == 0 && threadIdx.x == 0) *fac.norm = norm;
  } else {
    norm = *fac.norm;
  }
  // One rounding, of the whole factor. A NaN norm fails the comparison and
  // stays.
  double c = (double)fac.max_norm / ((double)norm + (double)fac.eps);
  c = c > 1.0 ? 1.0 : c;
  const float f = (float)(c * (double)fac.scale);
  if (in_place && f == 1.0f) return;
  const uint32_t tiles = tab.tile0[tab.ntensors];
  for (uint32_t t = blockIdx.x; t < tiles; t += gridDim.x) {
    const GradTile g = finder.find(tab, tiles - 1 - t);
    const void* in = tab.in[g.tensor];
    void* out = tab.out[g.tensor];
    if (g.small) {
      const int i = threadIdx.x;
      if (i >= g.bytes / (g.type == kGradF32 ? 4 : 2)) continue;
      const float e = grad_elem(in, g.type, i) * f;
      if (g.type == kGradF32)
        static_cast<float*>(out)[i] = e;
      else
        static_cast<uint16_t*>(out)[i] =
            g.type == kGradBF16 ? f32_to_elem<RINGSIM_BFLOAT16>(e) : f32_to_elem<RINGSIM_FLOAT16>(e);
      continue;
    }
    TileData d = load_tile<kLoadStream>(static_cast<const char*>(in) + g.first, g.bytes);
    if (g.bytes != kGradTileBytes) fix_tile(d, g.bytes);
    char* to = static_cast<char*>(out) + g.first;
    switch (g.type) {
      case kGradF32: tile_scale<RINGSIM_FLOAT32>(d, g.bytes, to, f); break;
      case kGradBF16: tile_scale<RINGSIM_BFLOAT16>(d, g.bytes, to, f); break;
      default: tile_scale<RINGSIM_FLOAT16>(d, g.bytes, to, f); break;
    }
  }
}

hipError_t launch_grad_squares(const GradSquareTable& t, uint32_t keep, double* partial, int workgroups,
                               hipStream_t s) {
  hipLaunchKernelGGL(grad_squares_kernel, dim3(workgroups), dim3(kThreads), 0, s, t, keep, partial);
  return hipGetLastError();
}

hipError_t launch_grad_norm_join(const double* partial, int parts, float scale, float* norm, hipStream_t s) {
  hipLaunchKernelGGL(grad_norm_join_kernel, dim3(1), dim3(kThreads), 0, s, partial, parts, scale, norm);
  return hipGetLastError();
}

hipError_t launch_grad_scale(const GradScaleTable& t, const GradFactor& f, int in_place, int workgroups,
                             hipStream_t s) {
  hipLaunchKernelGGL(grad_scale_kernel, dim3(workgroups), dim3(kThreads), 0, s, t, f, in_place);
  return hipGetLastError();
}

}  // namespace ringsim
