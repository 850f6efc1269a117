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

// A tile in registers: four 16-byte vectors a thread of 256, whatever the type.
constexpr int kTileVecs = kGradTileBytes / 16 / kThreads;
struct TileData {
  u32x4 v[kTileVecs];
};

constexpr int kWaves = kThreads / 64;
__device__ __forceinline__ int tile_thread() { return (int)(threadIdx.x % kThreads); }
__device__ __forceinline__ int vec_at(int i) { return (i * kThreads + tile_thread()) * 16; }

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
__device__ __forceinline__ double tile_squares(const TileData& d) {
  double s = 0.0;
#pragma unroll
  for (int i = 0; i < kTileVecs; ++i) {
    float f[OpElem<DT>::kPack];
    unpack<DT>(d.v[i], f);
#pragma unroll
    for (int j = 0; j < OpElem<DT>::kPack; ++j) s = __builtin_fma((double)f[j], (double)f[j], s);
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

// The squares of a tensor shorter than a vector, one element a thread.
__device__ __forceinline__ double small_squares(const void* in, const GradTile& g) {
  const int i = tile_thread(), n = g.bytes / (g.type == kGradF32 ? 4 : 2);
  const double e = i < n ? (double)grad_elem(in, g.type, i) : 0.0;
  return e * e;
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
    if (g.small) return small_squares(tab.in[g.tensor], g);
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

// Sum over a workgroup of `WAVES` waves, known to every thread; the order is
// fixed.
template <int WAVES>
__device__ __forceinline__ double block_sum(double v, double* lds) {
#pragma unroll
  for (int m = 1; m < 64; m *= 2) v += __shfl_xor(v, m, 64);
  if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = v;
  __syncthreads();
  v = lds[0];
#pragma unroll
  for (int i = 1; i < WAVES; ++i) v += lds[i];
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
  s = block_sum<kWaves>(s, lds);
  if (threadIdx.x == 0) partial[blockIdx.x] = s;
}

__device__ __forceinline__ float norm_of(double squares, float scale) {
  return (float)(__builtin_fabs((double)scale) * __builtin_sqrt(squares));
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
  s = block_sum<kWaves>(s, lds);
  return norm_of(s, scale);
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
    float f[OpElem<DT>::kPack];
    unpack<DT>(d.v[i], f);
#pragma unroll
    for (int j = 0; j < OpElem<DT>::kPack; ++j) f[j] *= factor;
    store16<true>(out, to_pack<DT>(f), vec_at(i), bytes);
  }
}

// Writes a tile in registers, scaled.
__device__ __forceinline__ void scale_tile(const TileData& d, const GradTile& g, const void* in, void* out, float f) {
  if (g.small) {
    const int i = tile_thread();
    if (i >= g.bytes / (g.type == kGradF32 ? 4 : 2)) return;
    const float e = grad_elem(in, g.type, i) * f;
    if (g.type == kGradF32)
      static_cast<float*>(out)[i] = e;
    else
      static_cast<uint16_t*>(out)[i] =
          g.type == kGradBF16 ? f32_to_elem<RINGSIM_BFLOAT16>(e) : f32_to_elem<RINGSIM_FLOAT16>(e);
    return;
  }
  char* to = static_cast<char*>(out) + g.first;
  switch (g.type) {
    case kGradF32: tile_scale<RINGSIM_FLOAT32>(d, g.bytes, to, f); break;
    case kGradBF16: tile_scale<RINGSIM_BFLOAT16>(d, g.bytes, to, f); break;
    default: tile_scale<RINGSIM_FLOAT16>(d, g.bytes, to, f); break;
  }
}

// What the gradients are multiplied with: one rounding, of the whole factor.
// A NaN norm fails the comparison and stays.
__device__ __forceinline__ float factor_of(float norm, const GradFactor& fac) {
  double c = (double)fac.max_norm / ((double)norm + (double)fac.eps);
  c = c > 1.0 ? 1.0 : c;
  return (float)(c * (double)fac.scale);
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
  const float f = factor_of(norm, fac);
  if (in_place && f == 1.0f) return;
  const uint32_t tiles = tab.tile0[tab.ntensors];
  for (uint32_t t = blockIdx.x; t < tiles; t += gridDim.x) {
    const GradTile g = finder.find(tab, tiles - 1 - t);
    const void* in = tab.in[g.tensor];
    TileData d;
    if (!g.small) {
      d = load_tile<kLoadStream>(static_cast<const char*>(in) + g.first, g.bytes);
      if (g.bytes != kGradTileBytes) fix_tile(d, g.bytes);
    }
    scale_tile(d, g, in, tab.out[g.tensor], f);
  }
}

// Norm and scaling of a list of at most kGradSmallTiles tiles by one
// workgroup: every tile is read once and stays in registers until it is
// scaled, and there is one launch instead of two. A call takes 4.4 us for one
// tensor of 4 KiB and 5.0 (norm) or 6.8 (clip) for 192 KiB, the 12 tiles that
// are the limit; two launches take 8.8 and 9.7. In a graph, where a launch
// costs less, 12 tiles are even (4.5 and 6.6 against 4.8 and 6.1), 16 lose.
__global__ void __launch_bounds__(kGradSmallThreads)
    grad_small_kernel(GradSmallTable tab, GradFactor fac, int clip, int in_place) {
  constexpr int kGroups = kGradSmallThreads / kThreads, kRounds = kGradSmallTiles / kGroups;
  __shared__ double lds[kGradSmallThreads / 64];
  const uint32_t tiles = tab.tile0[tab.ntensors];
  const TileFinder<GradSmallTable> finder(tab);
  const uint32_t group = __builtin_amdgcn_readfirstlane(threadIdx.x / kThreads);
  TileData d[kRounds];
  GradTile g[kRounds];
#pragma unroll
  for (int k = 0; k < kRounds; ++k) {
    const uint32_t t = group + k * kGroups;
    if (t >= tiles) continue;
    g[k] = finder.find(tab, t);
    if (!g[k].small) d[k] = load_tile<kLoadCached>(static_cast<const char*>(tab.in[g[k].tensor]) + g[k].first, g[k].bytes);
  }
  double s = 0.0;
#pragma unroll
  for (int k = 0; k < kRounds; ++k) {
    if (group + k * kGroups >= tiles) continue;
    if (g[k].small) {
      s += small_squares(tab.in[g[k].tensor], g[k]);
      continue;
    }
    if (g[k].bytes != kGradTileBytes) fix_tile(d[k], g[k].bytes);
    s += squares_of(d[k], g[k].type);
  }
  s = block_sum<kGradSmallThreads / 64>(s, lds);
  const float norm = norm_of(s, fac.scale);
  if (threadIdx.x == 0) *fac.norm = norm;
  if (!clip) return;
  const float f = factor_of(norm, fac);
  if (in_place && f == 1.0f) return;
#pragma unroll
  for (int k = 0; k < kRounds; ++k) {
    if (group + k * kGroups >= tiles) continue;
    scale_tile(d[k], g[k], tab.in[g[k].tensor], tab.out[g[k].tensor], f);
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

hipError_t launch_grad_small(const GradSmallTable& t, const GradFactor& f, int clip, int in_place, hipStream_t s) {
  hipLaunchKernelGGL(grad_small_kernel, dim3(1), dim3(kGradSmallThreads), 0, s, t, f, clip, in_place);
  return hipGetLastError();
}

hipError_t launch_grad_scale(const GradScaleTable& t, const GradFactor& f, int in_place, int workgroups,
                             hipStream_t s) {
  hipLaunchKernelGGL(grad_scale_kernel, dim3(workgroups), dim3(kThreads), 0, s, t, f, in_place);
  return hipGetLastError();
}

}  // namespace ringsim
