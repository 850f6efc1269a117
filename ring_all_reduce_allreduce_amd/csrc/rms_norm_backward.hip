// rms_norm_backward.hip -- gradients of the root-mean-square norm.
//
// With r = 1 / sqrt(mean(h^2) + eps), n = h r and g = grad_out * w, for every row
//   grad_in = grad_residual + r (g - n mean(g n))
// and over all rows  grad_weight = sum of grad_out n.
// mean(g n) is taken as r mean(g h), so that both sums need the row but once.
// r itself is never raised to a power: r^3 leaves fp32's range for rows above
// 1e13 and below 1e-13, where every factor of this form is as large as g or n.
// One pass reads each row once: both sums over the row (h^2 and g h) are taken
// together, r is recomputed from h rather than stored by the forward call
// (the row is here anyway), and every lane adds its columns' part of
// grad_weight over all rows its workgroup walks, in registers or, for the
// widest rows, in LDS. Workgroups leave these sums in a workspace, and a second
// small kernel adds them in a fixed order: no atomics, the same bits every
// time. Bound by memory: 16384 rows of 4096 take 92 us in bf16 (5.8 TB/s) and
// 168 us in fp32, the sum another 4.8 us.
#include <algorithm>

#include "ops_device.h"

namespace ringsim {

// A row's part of a lane as it lies in memory.
template <int NP>
struct BackwardRow {
  u32x4 dy[NP], h[NP], res[NP];
};

typedef float f32x4 __attribute__((ext_vector_type(4)));

// A workgroup of 1024 lanes has a compute unit for itself, with 128 registers
// a lane: too few for a row, the next row and 16 or 32 sums of the weight's
// gradient. Such wide rows keep the sums in LDS, which nothing else needs, and
// load the next row a pack at a time, each into the registers of the pack just
// written. 2048 rows of 32768 bf16 with a residual's gradient take 123 us so
// and 215 with sums in registers that spill, of 16384 51 us on 1024 lanes and
// 61 on 512 lanes that have the registers but load a row after another.
template <int TPR>
constexpr bool kWide = TPR == 1024;

// With 32 elements a lane the weights and the residual's gradient do not fit
// beside dy and h either: they are read where they are used.
template <int DT, int TPR, int NP>
constexpr bool kReadLate = kWide<TPR> && NP * OpElem<DT>::kPack > 16;

// Makes a wide row's offsets unknown from here on, and those of its later
// packs unknown until `after` is: the compiler would compute and load what
// eight packs need at once, and spill it. Two packs at a time hide the loads
// (one at a time takes up to 4% longer).
template <int TPR>
__device__ __forceinline__ void offsets_after(int k, int& t, float& after) {
  if (kWide<TPR> && k % 2 == 0) asm volatile("" : "+v"(t), "+v"(after));
}

// Where a row is read from. No condition stands around a load, since a wait
// that some path reaches without it would wait for everything: where the row
// is not wanted, or there is no residual's gradient, the lanes read the first
// bytes of a row of h for nothing.
template <int DT>
struct RowSource {
  const typename OpElem<DT>::T *dy, *h, *res;
  int n, n_res;
};

template <int DT>
__device__ __forceinline__ RowSource<DT> row_source(const RmsNormBackwardArgs& a, uint32_t row, bool wanted) {
  const uint32_t o = a.inner == 1 ? row : row / a.inner, in = a.inner == 1 ? 0 : row - o * a.inner;
  const int least = a.cols < OpElem<DT>::kPack ? a.cols : OpElem<DT>::kPack;
  const bool res = wanted && a.grad_residual.p;
  RowSource<DT> s;
  s.h = row_ptr<DT>(a.h, o, in);
  s.dy = wanted ? row_ptr<DT>(a.grad_out, o, in) : s.h;
  s.res = res ? row_ptr<DT>(a.grad_residual, o, in) : s.h;
  s.n = wanted ? a.cols : least;
  s.n_res = res ? a.cols : least;
  return s;
}

template <int DT, int TPR, int NP, int LK>
__device__ __forceinline__ void load_part(BackwardRow<NP>& r, const RowSource<DT>& s, int k, int c) {
  r.dy[k] = load_pack<DT, LK>(s.dy, c, s.n);
  r.h[k] = load_pack<DT, LK>(s.h, c, s.n);
  if constexpr (!kReadLate<DT, TPR, NP>) r.res[k] = load_pack<DT, LK>(s.res, c, s.n_res);
}

template <int DT, int TPR, int NP, int LK>
__device__ __forceinline__ BackwardRow<NP> load_row(const RmsNormBackwardArgs& a, uint32_t row, bool wanted, int t) {
  const RowSource<DT> s = row_source<DT>(a, row, wanted);
  BackwardRow<NP> r;
#pragma unroll
  for (int k = 0; k < NP; ++k) load_part<DT, TPR, NP, LK>(r, s, k, (k * row_lanes<TPR>() + t) * OpElem<DT>::kPack);
  return r;
}

// A lane's sums for its columns of the weight's gradient: in registers, or
// for wide rows in LDS, where lanes side by side have vectors side by side and
// only the lane itself reads and writes them.
template <int TPR, int NP, int P>
struct WeightSums {
  float f[NP][P];
  __device__ __forceinline__ void get(int k, int, float* d) const {
#pragma unroll
    for (int i = 0; i < P; ++i) d[i] = f[k][i];
  }
  __device__ __forceinline__ void put(int k, int, const float* d) {
#pragma unroll
    for (int i = 0; i < P; ++i) f[k][i] = d[i];
  }
};
template <int NP, int P>
struct WeightSums<1024, NP, P> {
  f32x4* lds;  // [NP * P / 4][1024]
  __device__ __forceinline__ void get(int k, int t, float* d) const {
#pragma unroll
    for (int j = 0; j < P / 4; ++j) {
      const f32x4 v = lds[(k * (P / 4) + j) * 1024 + t];
#pragma unroll
      for (int i = 0; i < 4; ++i) d[4 * j + i] = v[i];
    }
  }
  __device__ __forceinline__ void put(int k, int t, const float* d) {
#pragma unroll
    for (int j = 0; j < P / 4; ++j)
      lds[(k * (P / 4) + j) * 1024 + t] = f32x4{d[4 * j], d[4 * j + 1], d[4 * j + 2], d[4 * j + 3]};
  }
};

// One row in registers: its gradient is written, its part of the weight's
// gradient added to dw, and a wide row's registers filled from `next`.
// Everything stays as it lies in memory until it is used, also over the
// barrier: unpacking again costs an operation an element and saves the
// registers.
template <int DT, int TPR, int NP, int LK>
__device__ __forceinline__ void take_row(const RmsNormBackwardArgs& a, BackwardRow<NP>& r, uint32_t row, int t,
                                         WeightPack (&w)[NP], WeightSums<TPR, NP, OpElem<DT>::kPack>& dw,
                                         RowBuffers<TPR, f32x2>& lds, int& turn, const RowSource<DT>& next) {
  constexpr int kPack = OpElem<DT>::kPack;
  constexpr bool kLate = kReadLate<DT, TPR, NP>;
  // Eight packs have no registers for branches around late loads either (2048
  // rows of 20480 fp32 with a residual's gradient: 144 us, 168 with branches;
  // of fewer packs, the loads for nothing cost more): without a weight, or a
  // residual's gradient, they read h.
  constexpr bool kPlain = kLate && NP == 8;
  const int lanes = row_lanes<TPR>();
  const RowSource<DT> here = row_source<DT>(a, row, true);
  const void* weight = kPlain && a.weight_kind == kWeightNone ? (const void*)here.h : a.weight;
  const int kind = kPlain ? (int)kWeightF32 : a.weight_kind;
  static_assert(!kPlain || DT == RINGSIM_FLOAT32, "eight packs");
  float hh = 0.0f, gh = 0.0f;
#pragma unroll
  for (int k = 0; k < NP; ++k) {
    offsets_after<TPR>(k, t, gh);
    const int c = (k * lanes + t) * kPack;
    float fh[kPack], fdy[kPack], fw[kPack];
    r.h[k] = fix_pack<DT, LK>(r.h[k], c, a.cols);
    r.dy[k] = fix_pack<DT, LK>(r.dy[k], c, a.cols);
    unpack<DT>(r.h[k], fh);
    unpack<DT>(r.dy[k], fdy);
    if constexpr (kLate)
      w[k] = load_weight<DT, LK>(weight, kind, c, a.cols);
    else
      asm volatile("" : "+v"(w[k].v[0]), "+v"(w[k].v[1]));
    unpack_weight<DT, LK>(w[k], a.weight_kind, c, a.cols, fw);
#pragma unroll
    for (int i = 0; i < kPack; ++i) {
      hh = __builtin_fmaf(fh[i], fh[i], hh);
      gh = __builtin_fmaf(fdy[i] * fw[i], fh[i], gh);
    }
  }
  row_reduce2<TPR>(hh, gh, lds, turn);
  const float rr = rsqrtf(__builtin_fmaf(hh, a.inv_cols, a.eps));
  const float m = rr * (gh * a.inv_cols);
  const uint32_t o = a.inner == 1 ? row : row / a.inner, in = a.inner == 1 ? 0 : row - o * a.inner;
  auto* pout = row_ptr<typename OpElem<DT>::T>(a.grad_in, o, in);
  float last = m;  // of the pack before
#pragma unroll
  for (int k = 0; k < NP; ++k) {
    offsets_after<TPR>(k, t, last);
    const int c = (k * lanes + t) * kPack;
    float fh[kPack], fdy[kPack], fw[kPack], g[kPack], d[kPack];
    asm volatile("" : "+v"(r.h[k]), "+v"(r.dy[k]));
    unpack<DT>(r.h[k], fh);
    unpack<DT>(r.dy[k], fdy);
    dw.get(k, t, d);
    if constexpr (kLate) {
      if (kPlain || a.grad_residual.p) r.res[k] = load_pack<DT, LK>(here.res, c, here.n_res);
      w[k] = load_weight<DT, LK>(weight, kind, c, a.cols);
    } else {
      asm volatile("" : "+v"(w[k].v[0]), "+v"(w[k].v[1]));
    }
    unpack_weight<DT, LK>(w[k], a.weight_kind, c, a.cols, fw);
#pragma unroll
    for (int i = 0; i < kPack; ++i) {
      const float n = fh[i] * rr;
      g[i] = __builtin_fmaf(-n, m, fdy[i] * fw[i]) * rr;
      d[i] = __builtin_fmaf(fdy[i], n, d[i]);
    }
    dw.put(k, t, d);
    last = g[0] + g[kPack - 1];
    if (a.grad_residual.p) {
      float fr[kPack];
      unpack<DT>(fix_pack<DT, LK>(r.res[k], c, a.cols), fr);
#pragma unroll
      for (int i = 0; i < kPack; ++i) g[i] += fr[i];
    }
    store_pack<DT>(pout, to_pack<DT>(g), c, a.cols);
    if constexpr (kWide<TPR>) load_part<DT, TPR, NP, LK>(r, next, k, c);
  }
}

// A lane's fp32 sums of a pack's columns, left for the kernel that adds them.
template <int P>
__device__ __forceinline__ void store_sums(float* row, const float* f, int c, int cols) {
#pragma unroll
  for (int i = 0; i < P / 4; ++i)
    store16<false>(row, to_pack<RINGSIM_FLOAT32>(f + 4 * i), 4 * (c + 4 * i), 4 * cols);
}

template <int DT, int TPR, int NP, int LK>
__global__ void __launch_bounds__(kMaxBlock<TPR>) rms_norm_backward_kernel(RmsNormBackwardArgs a) {
  constexpr int kRows = kRowsPerBlock<TPR>;
  constexpr int kPack = OpElem<DT>::kPack;
  using T = typename OpElem<DT>::T;
  __shared__ RowBuffers<TPR, f32x2> lds;
  __shared__ float dws[kRows > 1 ? kRows : 1][kRows > 1 ? TPR * NP * kPack : 1];
  lds.clear();
  const int lanes = row_lanes<TPR>(), t = TPR <= 64 ? threadIdx.x % TPR : threadIdx.x;
  int turn = 0;
  WeightPack w[NP];
  WeightSums<TPR, NP, kPack> dw;
  if constexpr (kWide<TPR>) {
    __shared__ f32x4 sums[NP * (kPack / 4) * 1024];
    dw.lds = sums;
  }
#pragma unroll
  for (int k = 0; k < NP; ++k) {
    if constexpr (!kReadLate<DT, TPR, NP>)
      w[k] = load_weight<DT, LK>(a.weight, a.weight_kind, (k * lanes + t) * kPack, a.cols);
    const float zeros[kPack] = {};
    dw.put(k, t, zeros);
  }
  uint32_t row = blockIdx.x * kRows + (TPR <= 64 ? threadIdx.x / TPR : 0);
  const uint32_t step = gridDim.x * kRows;
  if constexpr (kWide<TPR>) {
    if (row < a.rows) {
      BackwardRow<NP> r = load_row<DT, TPR, NP, LK>(a, row, true, t);
      do {
        const uint32_t next = row + step;
        take_row<DT, TPR, NP, LK>(a, r, row, t, w, dw, lds, turn,
                                  row_source<DT>(a, next < a.rows ? next : row, next < a.rows));
        row = next;
      } while (row < a.rows);
    }
  } else if (row < a.rows) {
    // Two sets of registers in turn, since moving a loaded vector waits for it.
    BackwardRow<NP> ra = load_row<DT, TPR, NP, LK>(a, row, true, t), rb;
    for (;;) {
      uint32_t next = row + step;  // below 2^31 + 2^14
      rb = load_row<DT, TPR, NP, LK>(a, next < a.rows ? next : row, next < a.rows, t);
      take_row<DT, TPR, NP, LK>(a, ra, row, t, w, dw, lds, turn, {});
      row = next;
      if (row >= a.rows) break;
      next = row + step;
      ra = load_row<DT, TPR, NP, LK>(a, next < a.rows ? next : row, next < a.rows, t);
      take_row<DT, TPR, NP, LK>(a, rb, row, t, w, dw, lds, turn, {});
      row = next;
      if (row >= a.rows) break;
    }
  }
  if (!a.partial && !a.grad_weight) return;
  float* part = a.partial ? a.partial + (int64_t)blockIdx.x * a.cols : nullptr;
  if constexpr (kRows == 1) {
#pragma unroll
    for (int k = 0; k < NP; ++k) {
      const int c = (k * lanes + t) * kPack;
      float d[kPack];
      dw.get(k, t, d);
      if (part || a.weight_dtype == RINGSIM_FLOAT32)
        store_sums<kPack>(part ? part : static_cast<float*>(a.grad_weight), d, c, a.cols);
      else
        store_pack<DT>(a.grad_weight, to_pack<DT>(d), c, a.cols);
    }
  } else {
    float* mine = dws[threadIdx.x / TPR];
#pragma unroll
    for (int k = 0; k < NP; ++k) {
      dw.get(k, t, mine + (k * lanes + t) * kPack);
    }
    __syncthreads();
    for (int c = threadIdx.x; c < a.cols; c += kMaxBlock<TPR>) {
      float sum = dws[0][c];
#pragma unroll
      for (int i = 1; i < kRows; ++i) sum += dws[i][c];
      if (part)
        part[c] = sum;
      else if (a.weight_dtype == RINGSIM_FLOAT32)
        static_cast<float*>(a.grad_weight)[c] = sum;
      else
        static_cast<T*>(a.grad_weight)[c] = f32_to_elem<DT>(sum);
    }
  }
}

// grad_weight[c] = sum over `parts` rows of partial. A workgroup takes 16
// columns: 16 lanes side by side read a 64-byte line of a row, 64 such groups
// share the rows out, and their sums are added through LDS in a fixed order.
// 512 rows of 4096 take 4.3 us and 512 of 1111 2.7: mostly the start of a
// launch and one trip to sums that other dies wrote (128-byte segments with
// sums inside the waves first: 4.2 and 3.1).
constexpr int kSumCols = 16;
template <int kSumSlices>
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

// How a row is laid over lanes: a part of a wave, a wave, or as many whole
// waves as `packs` packs of 16 bytes a lane leave. `most`: the kernel's TPR.
struct RowShape {
  int lanes, packs, most;
};

// Turns of two rows a compute unit, above which rows count as many.
constexpr int kManyTurns = 4;

static RowShape backward_shape(int64_t rows, int64_t cols, int dtype) {
  const int per = 16 / op_dtype_size(dtype), packs = (int)((cols + per - 1) / per);
  const auto lanes = [&](int np) { return (packs + 64 * np - 1) / (64 * np) * 64; };
  if (packs <= 16) return {16, 1, 16};
  if (packs <= 32) return {32, 1, 32};
  if (packs <= 64) return {64, 1, 64};
  if (packs <= 128) return {64, 2, 64};
  if (packs <= 256) return {lanes(1), 1, 256};
  // 3 or 4 waves with 3 packs a lane instead of 5 or 6 with 2, so that a
  // compute unit holds two rows and its four SIMDs the same work: 8192 rows of
  // 5120 bf16 take 52 us, 60 with 2 packs. Few rows end sooner on more lanes
  // (1536 of them 18.5 us, 19.8 with 3 packs), and fp32, with less to compute a
  // byte, is as fast or faster on them (8192 rows of 2560: 44.2 and 44.2 us, of
  // 2816 49.3 and 51.2).
  if (packs > 512 && packs <= 768 && dtype != RINGSIM_FLOAT32 && rows > kManyTurns * kComputeUnits * 2)
    return {lanes(3), 3, 256};
  if (packs <= 1024) return {lanes(2), 2, 512};
  // 4 packs a lane are 16 elements of fp32, so that 512 lanes have room for two
  // rows (4096 rows of 8192: 74 us, 77 as wide rows), and 32 of the others.
  if (packs <= 2048) return dtype == RINGSIM_FLOAT32 ? RowShape{lanes(4), 4, 512} : RowShape{lanes(2), 2, 1024};
  if (packs <= 4096) return {lanes(4), 4, 1024};
  return {lanes(8), 8, 1024};
}

// So few rows that one workgroup's turns take no longer than a second launch:
// it writes the weight's gradient itself. A turn takes 0.6 us (1024 columns
// fp32) to 1.5 us (4096 bf16), a second launch 3.4 us of a call and 1.5 us in
// a graph: three rows of 4096 bf16 take 6.8 us a call and 6.4 in a graph, with
// workgroups of their own 8.9 and 5.8; four would take 8.2 and 7.8.
constexpr int kOneWorkgroupTurns = 3;
// Waves a compute unit is given. Each workgroup leaves a row of partial sums,
// so more of them cost more there than they hide: 16384 rows of 4096 bf16 take
// 96 us with 8 waves and 104 with 12.
constexpr int kBackwardWaves = 8;

int norm_backward_workgroups(int64_t rows, int64_t cols, int dtype) {
  const RowShape sh = backward_shape(rows, cols, dtype);
  const int64_t at_once = sh.lanes <= 64 ? 256 / sh.lanes : 1;
  if (rows <= kOneWorkgroupTurns * at_once) return 1;
  const int waves = sh.lanes <= 64 ? 4 : sh.lanes / 64;
  const int64_t most = (int64_t)kComputeUnits * std::max(1, kBackwardWaves / waves);
  const int64_t units = (rows + at_once - 1) / at_once;
  // Rows above a wave that most workgroups would take one of and some two: as
  // many as take two each, which leaves fewer sums (777 rows of 4096 bf16 14.0
  // against 15.4 us, 600 of them 12.7 against 14.9; from three turns on, and
  // for short rows, the workgroups that start early win by as much: 1984 rows
  // of 4224 22.1 against 21.7, 12186 of 80 7.3 against 6.6 in a graph).
  if (at_once == 1 && units > most && units < 2 * most) return (int)((units + 1) / 2);
  return (int)std::min(most, units);
}

template <int DT, int TPR, int NP, int LK>
static hipError_t launch_kind(const RmsNormBackwardArgs& a, int lanes, hipStream_t s) {
  hipLaunchKernelGGL((rms_norm_backward_kernel<DT, TPR, NP, LK>), dim3(norm_backward_workgroups(a.rows, a.cols, DT)),
                     dim3(lanes * kRowsPerBlock<TPR>), 0, s, a);
  return hipGetLastError();
}

template <int DT, int TPR, int NP>
static hipError_t launch_shape(const RmsNormBackwardArgs& a, int lanes, hipStream_t s) {
  const int64_t bytes =
      (int64_t)a.rows * a.cols * (int64_t)sizeof(typename OpElem<DT>::T) * (a.grad_residual.p ? 4 : 3);
  return bytes > kStreamBytes ? launch_kind<DT, TPR, NP, kLoadStream>(a, lanes, s)
                              : launch_kind<DT, TPR, NP, kLoadCached>(a, lanes, s);
}

template <int DT>
static hipError_t launch_type(const RmsNormBackwardArgs& a, hipStream_t s) {
  if (a.cols < OpElem<DT>::kPack) return launch_kind<DT, 16, 1, kLoadShort>(a, 16, s);
  const RowShape sh = backward_shape(a.rows, a.cols, DT);
  switch (sh.most * 16 + sh.packs) {
    case 16 * 16 + 1: return launch_shape<DT, 16, 1>(a, sh.lanes, s);
    case 32 * 16 + 1: return launch_shape<DT, 32, 1>(a, sh.lanes, s);
    case 64 * 16 + 1: return launch_shape<DT, 64, 1>(a, sh.lanes, s);
    case 64 * 16 + 2: return launch_shape<DT, 64, 2>(a, sh.lanes, s);
    case 256 * 16 + 1: return launch_shape<DT, 256, 1>(a, sh.lanes, s);
    case 512 * 16 + 2: return launch_shape<DT, 512, 2>(a, sh.lanes, s);
    case 1024 * 16 + 4: return launch_shape<DT, 1024, 4>(a, sh.lanes, s);
  }
  if constexpr (DT == RINGSIM_FLOAT32)
    return sh.packs == 4 ? launch_shape<DT, 512, 4>(a, sh.lanes, s) : launch_shape<DT, 1024, 8>(a, sh.lanes, s);
  else
    return sh.packs == 3 ? launch_shape<DT, 256, 3>(a, sh.lanes, s) : launch_shape<DT, 1024, 2>(a, sh.lanes, s);
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
  const dim3 grid((cols + kSumCols - 1) / kSumCols);
  if (parts > 64)
    hipLaunchKernelGGL(rms_norm_weight_sum_kernel<64>, grid, dim3(kSumCols * 64), 0, s, partial, parts, cols, grad_weight,
                       dtype);
  else
    hipLaunchKernelGGL(rms_norm_weight_sum_kernel<16>, grid, dim3(kSumCols * 16), 0, s, partial, parts, cols, grad_weight,
                       dtype);
  return hipGetLastError();
}

}  // namespace ringsim
