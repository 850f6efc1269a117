// grad_norm.hip -- the 2-norm of many gradients together, and the clipping by
// it.
//
//   norm = |scale| sqrt(sum g^2),  out = g * scale * min(1, max_norm / (norm + eps))
// A launch takes all tensors of its table: each is cut into tiles of 16 KiB,
// which the workgroups share out, walking them with one stride where each
// leaves a sum (40 buckets of 25 MiB bf16: 6.3-6.6 TB/s), one tile a workgroup
// where it only writes (6.3 TB/s). Squares are summed in fp64: the product of
// two fp32 values is exact there and cannot leave its range, and the vector
// unit's fp64 rate is several times what the memory delivers. Workgroups leave
// one sum each; whoever needs the norm adds these in a fixed order, so no
// atomics and the same bits every time. Both kernels are bound by memory.
#include <type_traits>

#include "ops_device.h"

namespace ringsim {

struct GradTile {
  const void* in;
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
      first[i] = j < TABLE::kTensors ? tab.tile0[j] : ~0u;
    }
  }

  __device__ __forceinline__ GradTile find(const TABLE& tab, uint32_t t) const {
    int k = -1;
#pragma unroll
    for (int i = 0; i < kPerLane; ++i) k += __builtin_popcountll(__builtin_amdgcn_ballot_w64(first[i] <= t));
    uint64_t in = tab.in[k];
    uint32_t from = tab.tile0[k], to = tab.tile0[k + 1];
    asm volatile("" : "+s"(in), "+s"(from), "+s"(to));  // all three on their way before one is waited for
    const uint32_t meta = (uint32_t)(in >> kGradAddressBits);
    const int type = (int)(meta >> kGradLastBits);
    const int last = (int)(meta & ((1u << kGradLastBits) - 1)) * (type == kGradF32 ? 4 : 2);
    return GradTile{reinterpret_cast<const void*>(in & ((1ull << kGradAddressBits) - 1)), k, type,
                    t + 1 == to ? last : kGradTileBytes, to - from == 1 && last < 16, (int64_t)(t - from) * kGradTileBytes};
  }
};

// A tile in registers: V 16-byte vectors for each of THREADS threads, whatever
// the type.
template <int THREADS, int V>
struct TileData {
  u32x4 v[V];
  static __device__ __forceinline__ int thread() { return (int)(threadIdx.x % THREADS); }
  static __device__ __forceinline__ int at(int i) { return (i * THREADS + thread()) * 16; }

  template <int LK>
  __device__ __forceinline__ void load(const char* tile, int bytes) {
#pragma unroll
    for (int i = 0; i < V; ++i) v[i] = load16<LK>(tile, at(i), bytes);
  }
  // Waits for the loads of a tile that is not used, so that no path leaves
  // them pending (its registers' next loads would wait for all others).
  __device__ __forceinline__ void settle() {
#pragma unroll
    for (int i = 0; i < V; ++i) asm volatile("" ::"v"(v[i]));
  }
  __device__ __forceinline__ void fix(int bytes) {
    if (bytes == THREADS * V * 16) return;
#pragma unroll
    for (int i = 0; i < V; ++i) v[i] = fix16<kLoadCached>(v[i], at(i), bytes);
  }
};
using BigTile = TileData<kThreads, kGradTileBytes / 16 / kThreads>;
using SmallTile = TileData<64, kGradShortTileBytes / 16 / 64>;

constexpr int kWaves = kThreads / 64;

template <int DT, int THREADS, int V>
__device__ __forceinline__ double tile_squares(const TileData<THREADS, V>& d) {
  double s = 0.0;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    float f[OpElem<DT>::kPack];
    unpack<DT>(d.v[i], f);
#pragma unroll
    for (int j = 0; j < OpElem<DT>::kPack; ++j) s = __builtin_fma((double)f[j], (double)f[j], s);
  }
  return s;
}

template <typename TILE>
__device__ __forceinline__ double squares_of(const TILE& d, int type) {
  switch (type) {
    case kGradF32: return tile_squares<RINGSIM_FLOAT32>(d);
    case kGradBF16: return tile_squares<RINGSIM_BFLOAT16>(d);
    default: return tile_squares<RINGSIM_FLOAT16>(d);
  }
}

typedef __attribute__((address_space(1))) uint16_t GlobalHalf;

// Element i of a tensor shorter than a vector (thread i has it): its two
// halves as they lie in memory (the same half twice for a 16-bit type), and
// its value, 0 beyond the tensor.
struct Halves {
  uint32_t lo, hi;
};
__device__ __forceinline__ Halves small_load(const void* in, int size, int n, int i) {
  const GlobalHalf* p = (const GlobalHalf*)(static_cast<const char*>(in) + (i < n ? i : n - 1) * size);
  return Halves{p[0], p[size / 2 - 1]};
}
__device__ __forceinline__ float small_value(Halves h, int type, int n, int i) {
  const float e = type == kGradF32    ? __uint_as_float(h.lo | h.hi << 16)
                  : type == kGradBF16 ? elem_to_f32<RINGSIM_BFLOAT16>((uint16_t)h.lo)
                                      : elem_to_f32<RINGSIM_FLOAT16>((uint16_t)h.lo);
  return i < n ? e : 0.0f;
}
__device__ __forceinline__ float small_elem(const GradTile& g, int i) {
  const int size = g.type == kGradF32 ? 4 : 2, n = g.bytes / size;
  return small_value(small_load(g.in, size, n, i), g.type, n, i);
}

// 16 bytes that can be read: where a thread's load is not wanted, but stands
// under no condition since a wait that some path reaches without it would
// wait for everything, it reads these.
__device__ const u32x4 g_spare = {0, 0, 0, 0};
__device__ __forceinline__ const char* spare_bytes() { return reinterpret_cast<const char*>(&g_spare); }

// The squares of tiles t, t + step, ... below `end`; t is left at the first
// one at or past it. One tile ahead: the next one's loads are under way
// while this one's squares are added (40 buckets of 25 MiB: 160 us, without
// 166). The two tiles take turns in two sets of registers, since moving a
// loaded vector waits for it. A tensor shorter than a vector is read when its
// turn comes.
template <int LK>
__device__ __forceinline__ double walk_squares(const GradTable& tab, const TileFinder<GradTable>& finder,
                                               uint32_t& t, uint32_t end, uint32_t step) {
  if (t >= end) return 0.0;
  const auto load = [&](const GradTile& g, bool wanted) {
    const bool real = wanted && !g.small;
    const char* p = real ? static_cast<const char*>(g.in) + g.first : spare_bytes();
    BigTile d;
    d.load<LK>(p, real ? g.bytes : 16);
    return d;
  };
  const auto squares = [&](BigTile& d, const GradTile& g) {
    if (g.small) {
      d.settle();
      const double e = (double)small_elem(g, BigTile::thread());
      return e * e;
    }
    d.fix(g.bytes);
    return squares_of(d, g.type);
  };
  double s = 0.0;
  GradTile ga = finder.find(tab, t), gb;
  BigTile da = load(ga, true), db;
  for (;;) {
    t += step;
    gb = finder.find(tab, t < end ? t : end - 1);
    db = load(gb, t < end);
    s += squares(da, ga);
    if (t >= end) {
      db.settle();
      return s;
    }
    t += step;
    ga = finder.find(tab, t < end ? t : end - 1);
    da = load(ga, t < end);
    s += squares(db, gb);
    if (t >= end) {
      da.settle();
      return s;
    }
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
    grad_squares_kernel(GradTable tab, uint32_t keep, double* partial) {
  __shared__ double lds[kWaves];
  const uint32_t tiles = tab.tiles;
  const TileFinder<GradTable> finder(tab);
  uint32_t t = blockIdx.x;
  double s = walk_squares<kLoadStream>(tab, finder, t, tiles - keep, gridDim.x);
  s += walk_squares<kLoadCached>(tab, finder, t, tiles, gridDim.x);
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

template <int DT, int THREADS, int V>
__device__ __forceinline__ void scale_vecs(const TileData<THREADS, V>& d, int bytes, char* out, float factor) {
#pragma unroll
  for (int i = 0; i < V; ++i) {
    float f[OpElem<DT>::kPack];
    unpack<DT>(d.v[i], f);
#pragma unroll
    for (int j = 0; j < OpElem<DT>::kPack; ++j) f[j] *= factor;
    store16<true>(out, to_pack<DT>(f), d.at(i), bytes);
  }
}

// Writes a tile in registers, scaled; `e` is the thread's element of a tensor
// shorter than a vector.
template <typename TILE>
__device__ __forceinline__ void scale_tile(const TILE& d, const GradTile& g, float e, void* out, float f) {
  char* to = static_cast<char*>(out) + g.first;
  if (g.small) {
    const int i = TILE::thread();
    if (i >= g.bytes / (g.type == kGradF32 ? 4 : 2)) return;
    if (g.type == kGradF32)
      reinterpret_cast<float*>(to)[i] = e * f;
    else
      reinterpret_cast<uint16_t*>(to)[i] =
          g.type == kGradBF16 ? f32_to_elem<RINGSIM_BFLOAT16>(e * f) : f32_to_elem<RINGSIM_FLOAT16>(e * f);
    return;
  }
  switch (g.type) {
    case kGradF32: scale_vecs<RINGSIM_FLOAT32>(d, g.bytes, to, f); break;
    case kGradBF16: scale_vecs<RINGSIM_BFLOAT16>(d, g.bytes, to, f); break;
    default: scale_vecs<RINGSIM_FLOAT16>(d, g.bytes, to, f); break;
  }
}

// What the gradients are multiplied with: one rounding, of the whole factor.
// A NaN norm fails the comparison and stays.
__device__ __forceinline__ float factor_of(float norm, const GradFactor& fac) {
  double c = (double)fac.max_norm / ((double)norm + (double)fac.eps);
  c = c > 1.0 ? 1.0 : c;
  return (float)(c * (double)fac.scale);
}

// Takes the tiles from the last to the first: what the norm's pass read last
// is still in the Infinity Cache.
template <typename TABLE>
__global__ void __launch_bounds__(kThreads) grad_scale_kernel(TABLE tab, GradFactor fac) {
  constexpr bool kInPlace = std::is_same_v<TABLE, GradTable>;
  __shared__ double lds[kWaves];
  const TileFinder<TABLE> finder(tab);
  float norm;
  if (fac.partial) {
    norm = join_norm(fac.partial, fac.parts, fac.scale, lds);
    if (blockIdx.x == 0 && threadIdx.x == 0) *fac.norm = norm;
  } else {
    norm = *fac.norm;
  }
  const float f = factor_of(norm, fac);
  if (kInPlace && f == 1.0f) return;
  const uint32_t tiles = tab.tiles;
  for (uint32_t t = blockIdx.x; t < tiles; t += gridDim.x) {
    const GradTile g = finder.find(tab, tiles - 1 - t);
    BigTile d;
    float e = 0.0f;
    if (g.small) {
      e = small_elem(g, BigTile::thread());
    } else {
      d.load<kLoadStream>(static_cast<const char*>(g.in) + g.first, g.bytes);
      d.fix(g.bytes);
    }
    if constexpr (kInPlace)
      scale_tile(d, g, e, const_cast<void*>(g.in), f);
    else
      scale_tile(d, g, e, tab.out[g.tensor], f);
  }
}

// A value of lane k, the same for the whole wave afterwards.
template <typename P>
__device__ __forceinline__ P* lane_ptr(P* p, int k) {
  const uint64_t v = reinterpret_cast<uint64_t>(p);
  const uint32_t lo = __builtin_amdgcn_readlane((uint32_t)v, k), hi = __builtin_amdgcn_readlane((uint32_t)(v >> 32), k);
  return reinterpret_cast<P*>((uint64_t)hi << 32 | lo);
}

// Norm and scaling of a short list by one workgroup: every tile is read once
// and stays in registers until it is scaled, and there is one launch instead
// of two. A call takes 4.3 us for the norm and 4.6 for the clipping of one
// tensor of 4 KiB, 4.9 and 5.3 for 34 tensors of 600 bytes, 5.4 and 8.6 for
// one of 192 KiB, the most it holds; two launches take 8.8 and 9.7. In a
// graph, where a launch costs less, 192 KiB take 5.0 and 8.3 against 4.8 and
// 6.1, 64 KiB 3.1 and 4.4.
// Lane k of a wave reads the table for the wave's round k, and all loads of
// tiles are under way before the first is used: what a call waits for is the
// table, the tiles and the barrier.
template <int ROUNDS>
__global__ void __launch_bounds__(kGradShortWaves * 64)
    grad_short_kernel(GradShortTable tab, GradFactor fac, int clip, int in_place) {
  __shared__ double lds[kGradShortWaves];
  const int lane = SmallTile::thread();
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
  const auto wanted = [&](int k) { return wave + k * kGradShortWaves < tab.tiles; };
  const void* in = spare_bytes();
  void* out = nullptr;
  uint32_t meta = kGradBF16 << 12 | 16;
  if (lane < ROUNDS && wanted(lane)) {
    in = tab.in[wave + lane * kGradShortWaves];
    out = tab.out[wave + lane * kGradShortWaves];
    meta = tab.meta[wave + lane * kGradShortWaves];
  }
  GradTile g[ROUNDS];
  SmallTile d[ROUNDS];
  float e[ROUNDS];
  bool small = false;
#pragma unroll
  for (int k = 0; k < ROUNDS; ++k) {
    const uint32_t m = __builtin_amdgcn_readlane(meta, k);
    g[k] = GradTile{lane_ptr(in, k), k, (int)(m >> 12), (int)(m & 2047), (m >> 11 & 1) != 0, 0};
    d[k].template load<kLoadCached>(g[k].small ? spare_bytes() : static_cast<const char*>(g[k].in),
                                    g[k].small ? 16 : g[k].bytes);
    small = small || g[k].small;
    e[k] = 0.0f;
  }
  if (small) {
    Halves h[ROUNDS];
#pragma unroll
    for (int k = 0; k < ROUNDS; ++k) {
      const int size = g[k].type == kGradF32 ? 4 : 2;
      h[k] = small_load(g[k].small ? g[k].in : spare_bytes(), size, g[k].small ? g[k].bytes / size : 1, lane);
    }
#pragma unroll
    for (int k = 0; k < ROUNDS; ++k) asm volatile("" : "+v"(h[k].lo), "+v"(h[k].hi));
#pragma unroll
    for (int k = 0; k < ROUNDS; ++k)
      e[k] = small_value(h[k], g[k].type, g[k].bytes / (g[k].type == kGradF32 ? 4 : 2), lane);
  }
  double s = 0.0;
#pragma unroll
  for (int k = 0; k < ROUNDS; ++k) {
    if (!wanted(k)) continue;
    if (g[k].small) {
      s += (double)e[k] * (double)e[k];
    } else {
      d[k].fix(g[k].bytes);
      s += squares_of(d[k], g[k].type);
    }
  }
  s = block_sum<kGradShortWaves>(s, lds);
  const float norm = norm_of(s, fac.scale);
  if (threadIdx.x == 0) *fac.norm = norm;
  if (!clip) return;
  const float f = factor_of(norm, fac);
  if (in_place && f == 1.0f) return;
#pragma unroll
  for (int k = 0; k < ROUNDS; ++k)
    if (wanted(k)) scale_tile(d[k], g[k], e[k], lane_ptr(out, k), f);
}

hipError_t launch_grad_squares(const GradTable& t, uint32_t keep, double* partial, int workgroups,
                               hipStream_t s) {
  hipLaunchKernelGGL(grad_squares_kernel, dim3(workgroups), dim3(kThreads), 0, s, t, keep, partial);
  return hipGetLastError();
}

hipError_t launch_grad_norm_join(const double* partial, int parts, float scale, float* norm, hipStream_t s) {
  hipLaunchKernelGGL(grad_norm_join_kernel, dim3(1), dim3(kThreads), 0, s, partial, parts, scale, norm);
  return hipGetLastError();
}

hipError_t launch_grad_short(const GradShortTable& t, const GradFactor& f, int clip, int in_place, hipStream_t s) {
  const dim3 grid(1), block(kGradShortWaves * 64);
  if (t.tiles <= kGradShortWaves)
    hipLaunchKernelGGL(grad_short_kernel<1>, grid, block, 0, s, t, f, clip, in_place);
  else if (t.tiles <= 4 * kGradShortWaves)
    hipLaunchKernelGGL(grad_short_kernel<4>, grid, block, 0, s, t, f, clip, in_place);
  else
    hipLaunchKernelGGL(grad_short_kernel<kGradShortRounds>, grid, block, 0, s, t, f, clip, in_place);
  return hipGetLastError();
}

template <typename TABLE>
static hipError_t launch_scale(const TABLE& t, const GradFactor& f, int workgroups, hipStream_t s) {
  hipLaunchKernelGGL(grad_scale_kernel<TABLE>, dim3(workgroups), dim3(kThreads), 0, s, t, f);
  return hipGetLastError();
}
hipError_t launch_grad_scale(const GradScaleTable& t, const GradFactor& f, int workgroups, hipStream_t s) {
  return launch_scale(t, f, workgroups, s);
}
hipError_t launch_grad_scale(const GradTable& t, const GradFactor& f, int workgroups, hipStream_t s) {
  return launch_scale(t, f, workgroups, s);
}

}  // namespace ringsim
