// ops_internal.h -- kernel arguments and launch rules of the step operators.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/ringsim_ops.h"

namespace ringsim {

constexpr int kComputeUnits = 256;  // of one MI355X

inline int op_dtype_size(int dtype) {
  switch (dtype) {
    case RINGSIM_FLOAT32: return 4;
    case RINGSIM_BFLOAT16: return 2;
    case RINGSIM_FLOAT16: return 2;
    case RINGSIM_FLOAT8_E4M3: return 1;
    default: return 0;
  }
}

// A call that moves more than the 256 MiB of the Infinity Cache reads its
// inputs non-temporally: nothing of them will be found there again. Norm of
// 16384 x 8192 fp32 355 us so, 385 through the caches; backward of 16384 x
// 4096 bf16 96 and 102; norm of 4096 x 4096 bf16 (128 MiB) 24.0 and 20.5, of
// 4096 x 6144 35.3 and 34.4.
constexpr int64_t kStreamBytes = 256ll << 20;

// A [outer, inner, cols] tensor: row r is at p + (r / inner) * s0 + (r % inner) * s1 elements.
struct RowsIn {
  const void* p;
  int64_t s0, s1;
};
struct RowsOut {
  void* p;
  int64_t s0, s1;
};

enum WeightKind : int { kWeightNone = 0, kWeightSame = 1, kWeightF32 = 2 };

struct RmsNormArgs {
  RowsIn x, residual;        // residual.p null: none
  const void* weight;
  RowsOut out, residual_out;
  float* scales;             // null: out has the input's type
  uint32_t rows, inner;
  int cols, groups, group;   // group 0: one scale a row
  int weight_kind;
  float eps, inv_cols;
};

struct RmsNormBackwardArgs {
  RowsIn grad_out, h, grad_residual;  // grad_residual.p null: none
  const void* weight;
  RowsOut grad_in;
  float* partial;            // [workgroups, cols] sums of grad_out * h * r; null: not wanted
  void* grad_weight;         // what a launch of one workgroup writes instead; null: not wanted
  int weight_dtype;
  uint32_t rows, inner;
  int cols;
  int weight_kind;
  float eps, inv_cols;
};

// Workgroups, and so rows of partial sums, of the backward pass.
int norm_backward_workgroups(int64_t rows, int64_t cols, int dtype);

hipError_t launch_rms_norm(const RmsNormArgs& a, int dtype, hipStream_t s);
hipError_t launch_rms_norm_backward(const RmsNormBackwardArgs& a, int dtype, hipStream_t s);
// grad_weight[c] = sum over `parts` rows of partial, in a fixed order.
hipError_t launch_rms_norm_weight_sum(const float* partial, int parts, int cols, void* grad_weight, int dtype,
                                      hipStream_t s);

// A launch's tensors and the tiles they are cut into: tensor i holds tiles
// [tile0[i], tile0[i + 1]) of kGradTileBytes each, its last one shorter.
// Tables travel as kernel arguments (below 4 KiB), which a graph's capture
// keeps by itself.
constexpr int kGradTileBytes = 16384;
constexpr int kGradWorkgroups = 1024;  // most of a launch that leaves a sum each
// Scaling takes a workgroup a tile: the hardware starts the next one while
// this one's stores drain. 40 buckets of 25 MiB take 332 us so, with 1024
// workgroups that walk the tiles 365, although each joins the 1024 sums of one
// launch of squares for itself (a list of several launches has as many times
// the sums to join in the first launch that scales).
constexpr uint32_t kGradScaleWorkgroups = 1u << 22;
constexpr int kGradTensors = 330;     // of a launch that reads, or writes in place
constexpr int kGradOutTensors = 196;  // of one that writes elsewhere

// Type and last tile of a tensor in 16 bits.
enum GradType : int { kGradF32 = 0, kGradBF16 = 1, kGradF16 = 2 };
constexpr int grad_type(int dtype) {
  return dtype == RINGSIM_FLOAT32 ? kGradF32 : dtype == RINGSIM_BFLOAT16 ? kGradBF16 : kGradF16;
}
constexpr int kGradLastBits = 14;  // elements of a tensor's last tile: up to 8192

// An address has 48 bits (the host refuses others); the 16 above them hold
// GradType << kGradLastBits | elements of the last tile.
constexpr int kGradAddressBits = 48;

template <int N>
struct GradInTable {
  static constexpr int kTensors = N;
  uint64_t in[N];
  uint32_t tile0[N + 1];  // tile0[tensors] == tiles, ~0 above
  uint32_t tiles;
};
template <int N>
struct GradOutTable : GradInTable<N> {
  void* out[N];
};
using GradTable = GradInTable<kGradTensors>;
using GradScaleTable = GradOutTable<kGradOutTensors>;
static_assert(sizeof(GradTable) <= 4000 && sizeof(GradScaleTable) <= 4000, "kernel arguments");

// A short list is one workgroup's, which keeps it in registers: tiles of 1
// KiB, one for each wave and round. Its table says for every tile where it
// lies, so there is nothing to look up.
constexpr int kGradShortTileBytes = 1024;
constexpr int kGradShortWaves = 16;
constexpr int kGradShortRounds = 12;
constexpr int kGradShortTiles = kGradShortWaves * kGradShortRounds;
struct GradShortTable {
  const void* in[kGradShortTiles];
  void* out[kGradShortTiles];
  // GradType << 12 | tensor shorter than a vector << 11 | bytes of the tile. 32
  // bits though 14 would do: a scalar load drops the two lowest bits of its
  // base and of its offset each, and an index that a 16-bit array shares with
  // the pointers is split by the compiler into parts that have them.
  uint32_t meta[kGradShortTiles];
  int tiles;
};
static_assert(sizeof(GradShortTable) <= 4000, "kernel arguments");

// The last `keep` tiles are read so that they stay in the Infinity Cache.
hipError_t launch_grad_squares(const GradTable& t, uint32_t keep, double* partial, int workgroups, hipStream_t s);
hipError_t launch_grad_norm_join(const double* partial, int parts, float scale, float* norm, hipStream_t s);
struct GradFactor {
  const double* partial;  // join these into the norm, or
  int parts;
  float* norm;            // partial null: read the norm here; else workgroup 0 writes it here
  float scale, max_norm, eps;
};
// Norm and, if `clip`, scaling of a short list in one launch; f.partial is not read.
hipError_t launch_grad_short(const GradShortTable& t, const GradFactor& f, int clip, int in_place, hipStream_t s);
hipError_t launch_grad_scale(const GradScaleTable& t, const GradFactor& f, int workgroups, hipStream_t s);
// The same in place.
hipError_t launch_grad_scale(const GradTable& t, const GradFactor& f, int workgroups, hipStream_t s);

}  // namespace ringsim
