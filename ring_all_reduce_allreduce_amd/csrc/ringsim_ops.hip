// ringsim_ops.hip -- host side of the step operators: argument checks and
// launches. Exports the C ABI of include/ringsim_ops.h.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstring>
#include <type_traits>

#include "ops_internal.h"
#include "ringsim_host.h"

using namespace ringsim;

namespace {

constexpr int64_t kMaxElements = INT64_MAX / 16;

bool valid_input_type(int dtype) {
  return dtype == RINGSIM_FLOAT32 || dtype == RINGSIM_BFLOAT16 || dtype == RINGSIM_FLOAT16;
}

bool aligned(const void* p, int bytes) { return reinterpret_cast<uintptr_t>(p) % (uintptr_t)bytes == 0; }

// Rows of an output must not overlap: every row starts at least cols past
// the other ones, whichever of the two strides is the larger.
bool rows_apart(const int64_t stride[2], int64_t outer, int64_t inner, int64_t cols) {
  int64_t so = stride[0] < 0 ? -stride[0] : stride[0], si = stride[1] < 0 ? -stride[1] : stride[1];
  if (inner == 1) return outer == 1 || so >= cols;
  if (outer == 1) return si >= cols;
  if (si < cols || so < cols) return false;
  return so >= si ? (so - cols) / si >= inner - 1 : (si - cols) / so >= outer - 1;
}

// Strides whose products with the row numbers stay far from overflow.
bool strides_fit(const int64_t stride[2], int64_t outer, int64_t inner) {
  for (int i = 0; i < 2; ++i) {
    const int64_t n = i == 0 ? outer : inner, most = kMaxElements / 4 / std::max<int64_t>(n, 1);
    if (n > 1 && (stride[i] > most || stride[i] < -most)) return false;
  }
  return true;
}

// One tensor of a row operator; NULL is checked by the caller.
bool valid_rows(const void* p, const int64_t stride[2], int64_t outer, int64_t inner, int64_t cols, int dtype,
                bool output) {
  return p && aligned(p, op_dtype_size(dtype)) && strides_fit(stride, outer, inner) &&
         (!output || rows_apart(stride, outer, inner, cols));
}

// Shape and types that the norm and its gradients share. *rows is outer * inner.
bool valid_norm_shape(int64_t outer, int64_t inner, int64_t cols, int dtype, int weight_dtype, float eps,
                      int64_t* rows) {
  if (!valid_input_type(dtype) || (weight_dtype != dtype && weight_dtype != RINGSIM_FLOAT32)) return false;
  if (outer < 0 || inner < 0 || cols < 1 || cols > RINGSIM_NORM_MAX_COLS) return false;
  if (!(eps >= 0.0f) || !std::isfinite(eps)) return false;
  if (outer > 0 && inner > INT32_MAX / outer) return false;  // rows are counted in 32 bits
  *rows = outer * inner;
  return true;
}

RowsIn rows_in(const void* p, const int64_t stride[2]) { return RowsIn{p, stride[0], stride[1]}; }
RowsOut rows_out(void* p, const int64_t stride[2]) { return RowsOut{p, stride[0], stride[1]}; }

int weight_kind(const void* w, int dtype, int weight_dtype) {
  if (!w) return kWeightNone;
  return weight_dtype == dtype ? kWeightSame : kWeightF32;
}

ringsim_result_t result_of(hipError_t e) {
  return e == hipSuccess ? RINGSIM_SUCCESS : RINGSIM_UNHANDLED_DEVICE_ERROR;
}

// ---------------------------------------------------------------------------
// Lists of gradients
// ---------------------------------------------------------------------------

int64_t tiles_of(int64_t count, int dtype, int tile_bytes = kGradTileBytes) {
  const int64_t elems = tile_bytes / op_dtype_size(dtype);
  return (count + elems - 1) / elems;
}

// All tensors together stay below 2^31 tiles (32 TiB), so that a launch's
// tiles are counted in 32 bits wherever the list is cut.
bool valid_grads(int n, const void* const* grads, void* const* outs, const int64_t* counts, const int* dtypes) {
  if (n < 0 || (n > 0 && (!grads || !counts || !dtypes))) return false;
  int64_t tiles = 0;
  for (int i = 0; i < n; ++i) {
    if (!valid_input_type(dtypes[i]) || counts[i] < 0 || counts[i] > kMaxElements) return false;
    if (counts[i] == 0) continue;
    const int e = op_dtype_size(dtypes[i]);
    tiles += tiles_of(counts[i], dtypes[i]);
    if (tiles > INT32_MAX) return false;
    if (!grads[i] || !aligned(grads[i], e) || reinterpret_cast<uintptr_t>(grads[i]) >> kGradAddressBits) return false;
    if (outs && (!outs[i] || !aligned(outs[i], e))) return false;
  }
  return true;
}

// Fills a table with the next tensors of the list that hold elements,
// beginning with *next; advances *next. No tiles: the rest was empty.
template <typename TABLE>
void fill_table(TABLE& t, int n, const void* const* grads, void* const* outs, const int64_t* counts,
                const int* dtypes, int* next) {
  int tensors = 0;
  t.tiles = 0;
  t.tile0[0] = 0;
  for (; *next < n && tensors < TABLE::kTensors; ++*next) {
    const int i = *next;
    if (counts[i] == 0) continue;
    const int64_t k = tiles_of(counts[i], dtypes[i]);
    const int64_t last = counts[i] - (k - 1) * (kGradTileBytes / op_dtype_size(dtypes[i]));
    const uint64_t meta = (uint64_t)grad_type(dtypes[i]) << kGradLastBits | (uint64_t)last;
    t.in[tensors] = (uint64_t)reinterpret_cast<uintptr_t>(grads[i]) | meta << kGradAddressBits;
    if constexpr (std::is_same_v<TABLE, GradScaleTable>) t.out[tensors] = outs[i];
    t.tiles += (uint32_t)k;
    t.tile0[++tensors] = t.tiles;
  }
  for (int j = tensors + 1; j <= TABLE::kTensors; ++j) t.tile0[j] = ~0u;
}

int grad_workgroups(uint32_t tiles) { return (int)std::min<uint32_t>(tiles, kGradWorkgroups); }
int grad_scale_workgroups(uint32_t tiles) { return (int)std::min<uint32_t>(tiles, kGradScaleWorkgroups); }

// Sums of squares of every launch's workgroups into the workspace. `left`:
// tiles still to come. `keep` bytes at the end are read so that they stay in
// the Infinity Cache.
ringsim_result_t enqueue_squares(int n, const void* const* grads, const int64_t* counts, const int* dtypes,
                                 int64_t left, int64_t keep, double* partial, int* parts, hipStream_t s) {
  *parts = 0;
  keep /= kGradTileBytes;
  for (int next = 0; next < n;) {
    GradTable t;
    fill_table(t, n, grads, nullptr, counts, dtypes, &next);
    if (t.tiles == 0) break;
    left -= t.tiles;
    const int g = grad_workgroups(t.tiles);
    const uint32_t here = (uint32_t)std::min<int64_t>(t.tiles, std::max<int64_t>(0, keep - left));
    if (launch_grad_squares(t, here, partial + *parts, g, s) != hipSuccess) return RINGSIM_UNHANDLED_DEVICE_ERROR;
    *parts += g;
  }
  return RINGSIM_SUCCESS;
}

template <typename TABLE>
ringsim_result_t enqueue_scale(int n, const void* const* grads, void* const* outs, const int64_t* counts,
                               const int* dtypes, GradFactor f, hipStream_t s) {
  for (int next = 0; next < n;) {
    TABLE t;
    fill_table(t, n, grads, outs, counts, dtypes, &next);
    if (t.tiles == 0) break;
    if (launch_grad_scale(t, f, grad_scale_workgroups(t.tiles), s) != hipSuccess) return RINGSIM_UNHANDLED_DEVICE_ERROR;
    f.partial = nullptr;  // the first launch has written the norm
  }
  return RINGSIM_SUCCESS;
}

ringsim_result_t enqueue_scale(int n, const void* const* grads, void* const* outs, const int64_t* counts,
                               const int* dtypes, const GradFactor& f, hipStream_t s) {
  return outs ? enqueue_scale<GradScaleTable>(n, grads, outs, counts, dtypes, f, s)
              : enqueue_scale<GradTable>(n, grads, outs, counts, dtypes, f, s);
}

// Tiles of the whole list.
int64_t total_tiles(int n, const int64_t* counts, const int* dtypes) {
  int64_t tiles = 0;
  for (int i = 0; i < n; ++i) tiles += tiles_of(counts[i], dtypes[i]);
  return tiles;
}

// Whether one workgroup takes the list: as many tiles as its registers.
bool is_short(int n, const int64_t* counts, const int* dtypes) {
  int64_t tiles = 0;
  for (int i = 0; i < n && tiles <= kGradShortTiles; ++i) tiles += tiles_of(counts[i], dtypes[i], kGradShortTileBytes);
  return tiles <= kGradShortTiles;
}

size_t norm_workspace(int n) {
  return sizeof(double) * kGradWorkgroups * (size_t)((n + kGradTensors - 1) / kGradTensors);
}

bool valid_workspace(const void* ws, size_t bytes, int n) {
  return ws && aligned(ws, 16) && bytes >= norm_workspace(n);
}

// Norm, and scaling if `clip`, of a list that one workgroup takes.
ringsim_result_t enqueue_short(int n, const void* const* grads, void* const* outs, const int64_t* counts,
                               const int* dtypes, const GradFactor& f, bool clip, hipStream_t s) {
  GradShortTable t;
  t.tiles = 0;
  for (int i = 0; i < n; ++i) {
    const int64_t bytes = counts[i] * op_dtype_size(dtypes[i]);
    for (int64_t at = 0; at < bytes; at += kGradShortTileBytes, ++t.tiles) {
      t.in[t.tiles] = static_cast<const char*>(grads[i]) + at;
      t.out[t.tiles] = static_cast<char*>(outs ? outs[i] : const_cast<void*>(grads[i])) + at;
      t.meta[t.tiles] = (uint32_t)grad_type(dtypes[i]) << 12 | (uint32_t)(bytes < 16) << 11 |
                        (uint32_t)std::min<int64_t>(kGradShortTileBytes, bytes - at);
    }
  }
  return result_of(launch_grad_short(t, f, clip, outs == nullptr, s));
}

// What a pass over the gradients may leave for the next one in the Infinity
// Cache of 256 MiB. (Clipping 40 buckets of 25 MiB: 485 us, with nothing read
// to stay 491, with everything 492.)
constexpr int64_t kGradKeepBytes = 192ll << 20;

bool valid_factor(float scale, float max_norm, float eps) {
  return std::isfinite(scale) && std::isfinite(max_norm) && max_norm >= 0.0f && std::isfinite(eps) && eps >= 0.0f;
}

}  // namespace

extern "C" {

ringsim_result_t ringsim_rms_norm(const ringsim_rms_norm_t* a, ringsim_stream_t stream) {
  const RoctxRange range("ringsim_rms_norm");
  int64_t rows = 0;
  if (!a || !valid_norm_shape(a->outer, a->inner, a->cols, a->dtype, a->weight_dtype, a->eps, &rows))
    return RINGSIM_INVALID_ARGUMENT;
  const bool quant = a->out_dtype == RINGSIM_FLOAT8_E4M3;
  if (!quant && a->out_dtype != a->dtype) return RINGSIM_INVALID_ARGUMENT;
  if (quant ? a->group != 0 && a->group != 32 && a->group != 64 && a->group != 128 : a->group != 0 || a->scales)
    return RINGSIM_INVALID_ARGUMENT;
  if (!a->residual != !a->residual_out) return RINGSIM_INVALID_ARGUMENT;
  if (rows == 0) return RINGSIM_SUCCESS;
  const auto ok = [&](const void* p, const int64_t stride[2], int dtype, bool output) {
    return valid_rows(p, stride, a->outer, a->inner, a->cols, dtype, output);
  };
  if (!ok(a->x, a->x_stride, a->dtype, false) || !ok(a->out, a->out_stride, a->out_dtype, true))
    return RINGSIM_INVALID_ARGUMENT;
  if (a->residual && (!ok(a->residual, a->residual_stride, a->dtype, false) ||
                      !ok(a->residual_out, a->residual_out_stride, a->dtype, true)))
    return RINGSIM_INVALID_ARGUMENT;
  if (a->weight && !aligned(a->weight, op_dtype_size(a->weight_dtype))) return RINGSIM_INVALID_ARGUMENT;
  if (quant && (!a->scales || !aligned(a->scales, 4))) return RINGSIM_INVALID_ARGUMENT;
  RmsNormArgs k;
  std::memset(&k, 0, sizeof(k));
  k.x = rows_in(a->x, a->x_stride);
  k.out = rows_out(a->out, a->out_stride);
  if (a->residual) {
    k.residual = rows_in(a->residual, a->residual_stride);
    k.residual_out = rows_out(a->residual_out, a->residual_out_stride);
  }
  k.weight = a->weight;
  k.scales = quant ? a->scales : nullptr;
  k.rows = (uint32_t)rows;
  k.inner = (uint32_t)a->inner;
  k.cols = (int)a->cols;
  k.group = a->group;
  k.groups = a->group ? (int)((a->cols + a->group - 1) / a->group) : 1;
  k.weight_kind = weight_kind(a->weight, a->dtype, a->weight_dtype);
  k.eps = a->eps;
  k.inv_cols = 1.0f / (float)a->cols;
  return result_of(launch_rms_norm(k, a->dtype, static_cast<hipStream_t>(stream)));
}

ringsim_result_t ringsim_rms_norm_backward_workspace(int64_t rows, int64_t cols, int dtype, size_t* bytes) {
  if (!bytes || !valid_input_type(dtype) || rows < 0 || rows > INT32_MAX || cols < 1 || cols > RINGSIM_NORM_MAX_COLS)
    return RINGSIM_INVALID_ARGUMENT;
  const int g = norm_backward_workgroups(rows, cols, dtype);
  *bytes = g == 1 ? 0 : sizeof(float) * (size_t)g * (size_t)cols;
  return RINGSIM_SUCCESS;
}

ringsim_result_t ringsim_rms_norm_backward(const ringsim_rms_norm_backward_t* a, ringsim_stream_t stream) {
  const RoctxRange range("ringsim_rms_norm_backward");
  int64_t rows = 0;
  if (!a || !valid_norm_shape(a->outer, a->inner, a->cols, a->dtype, a->weight_dtype, a->eps, &rows))
    return RINGSIM_INVALID_ARGUMENT;
  const auto ok = [&](const void* p, const int64_t stride[2], bool output) {
    return valid_rows(p, stride, a->outer, a->inner, a->cols, a->dtype, output);
  };
  if (rows > 0 && (!ok(a->grad_out, a->grad_out_stride, false) || !ok(a->h, a->h_stride, false) ||
                   !ok(a->grad_in, a->grad_in_stride, true) ||
                   (a->grad_residual && !ok(a->grad_residual, a->grad_residual_stride, false))))
    return RINGSIM_INVALID_ARGUMENT;
  if (a->weight && !aligned(a->weight, op_dtype_size(a->weight_dtype))) return RINGSIM_INVALID_ARGUMENT;
  if (a->grad_weight) {
    size_t need = 0;
    ringsim_rms_norm_backward_workspace(rows, a->cols, a->dtype, &need);
    if (!aligned(a->grad_weight, op_dtype_size(a->weight_dtype))) return RINGSIM_INVALID_ARGUMENT;
    if (need > 0 && (!a->workspace || !aligned(a->workspace, 16) || a->workspace_bytes < need))
      return RINGSIM_INVALID_ARGUMENT;
  }
  hipStream_t s = static_cast<hipStream_t>(stream);
  const int g = rows > 0 ? norm_backward_workgroups(rows, a->cols, a->dtype) : 0;
  float* const partial = a->grad_weight && g > 1 ? static_cast<float*>(a->workspace) : nullptr;
  if (rows > 0) {
    RmsNormBackwardArgs k;
    std::memset(&k, 0, sizeof(k));
    k.grad_out = rows_in(a->grad_out, a->grad_out_stride);
    k.h = rows_in(a->h, a->h_stride);
    if (a->grad_residual) k.grad_residual = rows_in(a->grad_residual, a->grad_residual_stride);
    k.grad_in = rows_out(a->grad_in, a->grad_in_stride);
    k.weight = a->weight;
    k.partial = partial;
    k.grad_weight = g == 1 ? a->grad_weight : nullptr;
    k.weight_dtype = a->weight_dtype;
    k.rows = (uint32_t)rows;
    k.inner = (uint32_t)a->inner;
    k.cols = (int)a->cols;
    k.weight_kind = weight_kind(a->weight, a->dtype, a->weight_dtype);
    k.eps = a->eps;
    k.inv_cols = 1.0f / (float)a->cols;
    if (launch_rms_norm_backward(k, a->dtype, s) != hipSuccess) return RINGSIM_UNHANDLED_DEVICE_ERROR;
  }
  if (!a->grad_weight || g == 1) return RINGSIM_SUCCESS;
  // Without rows the sum runs over no parts and writes zeros.
  return result_of(launch_rms_norm_weight_sum(partial, g, (int)a->cols, a->grad_weight, a->weight_dtype, s));
}

ringsim_result_t ringsim_grad_norm_workspace(int ntensors, const int64_t* counts, const int* dtypes, size_t* bytes) {
  if (!bytes || ntensors < 0 || (ntensors > 0 && (!counts || !dtypes))) return RINGSIM_INVALID_ARGUMENT;
  for (int i = 0; i < ntensors; ++i)
    if (!valid_input_type(dtypes[i]) || counts[i] < 0 || counts[i] > kMaxElements) return RINGSIM_INVALID_ARGUMENT;
  *bytes = is_short(ntensors, counts, dtypes) ? 0 : norm_workspace(ntensors);
  return RINGSIM_SUCCESS;
}

ringsim_result_t ringsim_grad_norm(int ntensors, const void* const* grads, const int64_t* counts, const int* dtypes,
                                   float scale, float* norm, void* workspace, size_t workspace_bytes,
                                   ringsim_stream_t stream) {
  const RoctxRange range("ringsim_grad_norm");
  if (!valid_grads(ntensors, grads, nullptr, counts, dtypes) || !std::isfinite(scale) || !norm || !aligned(norm, 4))
    return RINGSIM_INVALID_ARGUMENT;
  hipStream_t s = static_cast<hipStream_t>(stream);
  if (is_short(ntensors, counts, dtypes))
    return enqueue_short(ntensors, grads, nullptr, counts, dtypes, GradFactor{nullptr, 0, norm, scale, 0.0f, 0.0f},
                         false, s);
  if (!valid_workspace(workspace, workspace_bytes, ntensors)) return RINGSIM_INVALID_ARGUMENT;
  double* const partial = static_cast<double*>(workspace);
  int parts = 0;
  const ringsim_result_t res =
      enqueue_squares(ntensors, grads, counts, dtypes, total_tiles(ntensors, counts, dtypes), kGradKeepBytes, partial,
                      &parts, s);
  if (res != RINGSIM_SUCCESS) return res;
  return result_of(launch_grad_norm_join(partial, parts, scale, norm, s));
}

ringsim_result_t ringsim_scale_grads(int ntensors, const void* const* grads, void* const* outs, const int64_t* counts,
                                     const int* dtypes, float scale, const float* norm, float max_norm, float eps,
                                     ringsim_stream_t stream) {
  const RoctxRange range("ringsim_scale_grads");
  if (!valid_grads(ntensors, grads, outs, counts, dtypes) || !valid_factor(scale, max_norm, eps) || !norm ||
      !aligned(norm, 4))
    return RINGSIM_INVALID_ARGUMENT;
  const GradFactor f{nullptr, 0, const_cast<float*>(norm), scale, max_norm, eps};
  return enqueue_scale(ntensors, grads, outs, counts, dtypes, f, static_cast<hipStream_t>(stream));
}

ringsim_result_t ringsim_clip_grads(int ntensors, const void* const* grads, void* const* outs, const int64_t* counts,
                                    const int* dtypes, float scale, float max_norm, float eps, float* norm,
                                    void* workspace, size_t workspace_bytes, ringsim_stream_t stream) {
  const RoctxRange range("ringsim_clip_grads");
  if (!valid_grads(ntensors, grads, outs, counts, dtypes) || !valid_factor(scale, max_norm, eps) || !norm ||
      !aligned(norm, 4))
    return RINGSIM_INVALID_ARGUMENT;
  hipStream_t s = static_cast<hipStream_t>(stream);
  if (is_short(ntensors, counts, dtypes))
    return enqueue_short(ntensors, grads, outs, counts, dtypes, GradFactor{nullptr, 0, norm, scale, max_norm, eps}, true,
                         s);
  if (!valid_workspace(workspace, workspace_bytes, ntensors)) return RINGSIM_INVALID_ARGUMENT;
  double* const partial = static_cast<double*>(workspace);
  int parts = 0;
  const ringsim_result_t res =
      enqueue_squares(ntensors, grads, counts, dtypes, total_tiles(ntensors, counts, dtypes), kGradKeepBytes, partial,
                      &parts, s);
  if (res != RINGSIM_SUCCESS) return res;
  const GradFactor f{partial, parts, norm, scale, max_norm, eps};
  return enqueue_scale(ntensors, grads, outs, counts, dtypes, f, s);
}

}  // extern "C"
