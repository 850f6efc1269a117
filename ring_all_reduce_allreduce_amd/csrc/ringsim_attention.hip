// ringsim_attention.hip -- host side of the attention-step operators: argument
// checks and launches. Exports the C ABI of include/ringsim_attention.h.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstring>

#include "attention_internal.h"
#include "ringsim_host.h"

using namespace ringsim;

namespace {

constexpr int64_t kMaxOffset = INT64_MAX / 64;  // elements between two of a tensor
constexpr int64_t kMaxHeads = 65535;            // a dimension of a grid
constexpr int64_t kMaxBlocks = (1 << 24) - 1;   // workgroups of 256 lanes: below 2^32 lanes

bool value_type(int t) { return t == RINGSIM_FLOAT32 || t == RINGSIM_BFLOAT16 || t == RINGSIM_FLOAT16; }
bool index_type(int t) { return t == RINGSIM_INT32 || t == RINGSIM_INT64; }

bool aligned(const void* p, int bytes) { return reinterpret_cast<uintptr_t>(p) % (uintptr_t)bytes == 0; }

int64_t magnitude(int64_t v) { return v < 0 ? -v : v; }

// Strides whose products with the sizes stay far from overflow.
bool strides_fit(const int64_t* stride, const int64_t* size, int dims) {
  for (int i = 0; i < dims; ++i) {
    if (size[i] <= 1) continue;
    const int64_t most = kMaxOffset / 4 / size[i];
    if (stride[i] > most || stride[i] < -most) return false;
  }
  return true;
}

// Whether rows of `cols` elements that lie `stride` apart in each dimension
// overlap nowhere: taken from the smallest stride up, each has to clear what
// those before it span. (Arrangements that interleave without meeting are
// refused too.)
bool rows_apart(const int64_t* stride, const int64_t* size, int dims, int64_t cols) {
  int order[4];
  int n = 0;
  for (int i = 0; i < dims; ++i)
    if (size[i] > 1) order[n++] = i;
  std::sort(order, order + n, [&](int a, int b) { return magnitude(stride[a]) < magnitude(stride[b]); });
  int64_t span = cols;
  for (int i = 0; i < n; ++i) {
    const int64_t st = magnitude(stride[order[i]]);
    if (st < span) return false;
    span += st * (size[order[i]] - 1);
  }
  return true;
}

// One tensor of heads; pointers may be anything where there are no rows.
bool valid_heads(const void* p, const int64_t stride[3], int64_t outer, int64_t inner, int64_t heads, int64_t dim,
                 int dtype, bool output) {
  const int64_t size[3] = {outer, inner, heads};
  return p && aligned(p, op_dtype_size(dtype)) && strides_fit(stride, size, 3) &&
         (!output || rows_apart(stride, size, 3, dim));
}

bool valid_index(const void* p, const int64_t stride[2], int64_t outer, int64_t inner, int type) {
  const int64_t size[2] = {outer, inner};
  return p && index_type(type) && aligned(p, type == RINGSIM_INT64 ? 8 : 4) && strides_fit(stride, size, 2);
}

// Tokens are counted in 32 bits.
bool token_count(int64_t outer, int64_t inner, int64_t* tokens) {
  if (outer < 0 || inner < 0 || (outer > 0 && inner > INT32_MAX / outer)) return false;
  *tokens = outer * inner;
  return true;
}

Index index_of(const void* p, const int64_t stride[2], int type) {
  return Index{p, stride[0], stride[1], type == RINGSIM_INT64};
}

int shift_of(int64_t page) {
  int s = 0;
  while ((int64_t)1 << s < page) ++s;
  return s;
}

// Sizes of a cache but its number of pages.
bool valid_page(const ringsim_kv_cache_t& c) {
  if (c.dim != 64 && c.dim != 96 && c.dim != 128 && c.dim != 192 && c.dim != 256) return false;
  if (c.page_size < kKvTile || c.page_size > RINGSIM_KV_MAX_PAGE || (c.page_size & (c.page_size - 1))) return false;
  return c.heads >= 1 && c.heads <= kMaxHeads;
}

// `written`: no two pages or heads may overlap.
bool valid_cache(const ringsim_kv_cache_t& c, bool written) {
  if (!valid_page(c) || c.pages < 1 || c.pages > INT32_MAX) return false;
  for (const void* p : {c.keys, c.values, c.key_scales, c.value_scales})
    if (!p || !aligned(p, 16)) return false;
  const int64_t size[2] = {c.pages, c.heads};
  for (const int64_t* st : {c.stride, c.scale_stride})
    for (int i = 0; i < 2; ++i)
      if (size[i] > 1 && st[i] % 16) return false;
  if (!strides_fit(c.stride, size, 2) || !strides_fit(c.scale_stride, size, 2)) return false;
  return !written || (rows_apart(c.stride, size, 2, c.page_size * c.dim / 2) &&
                      rows_apart(c.scale_stride, size, 2, c.page_size * c.dim / kKvBlock));
}

KvCacheArgs cache_args(const ringsim_kv_cache_t& c) {
  KvCacheArgs k;
  k.data[0] = c.keys;
  k.data[1] = c.values;
  k.scales[0] = c.key_scales;
  k.scales[1] = c.value_scales;
  // A stride that no index multiplies may be anything.
  k.page = c.pages > 1 ? c.stride[0] : 0;
  k.head = c.heads > 1 ? c.stride[1] : 0;
  k.scale_page = c.pages > 1 ? c.scale_stride[0] : 0;
  k.scale_head = c.heads > 1 ? c.scale_stride[1] : 0;
  k.pages = (int32_t)c.pages;
  k.heads = (int)c.heads;
  k.dim = (int)c.dim;
  k.page_shift = shift_of(c.page_size);
  return k;
}

ringsim_result_t result_of(hipError_t e) {
  return e == hipSuccess ? RINGSIM_SUCCESS : RINGSIM_UNHANDLED_DEVICE_ERROR;
}

bool valid_frequencies(const double* f, int64_t pairs) { return pairs == 0 || (f && aligned(f, 8)); }

// Sizes and types of an attention call, and how it is cut.
bool plan_of(const ringsim_paged_attention_t& a, AttentionPlan* plan, int64_t* cap) {
  const ringsim_kv_cache_t& c = a.cache;
  if (!value_type(a.dtype) || !valid_page(c)) return false;
  if (a.tokens < 0 || a.seqs < 0 || a.heads < 1 || a.heads > kMaxHeads || a.heads % c.heads) return false;
  if (a.tokens > INT32_MAX / a.heads || a.seqs > INT32_MAX || a.max_pages < 0 || a.max_pages > INT32_MAX) return false;
  if (a.max_length < 0 || a.window < 0) return false;
  if (a.seqs == 0 || a.tokens == 0) return true;
  if (!a.starts && a.tokens % a.seqs) return false;
  *cap = std::min<int64_t>(a.max_pages * c.page_size, kMaxPositions);
  if (a.max_length > 0) *cap = std::min(*cap, a.max_length);
  *plan = plan_attention(a.tokens, a.seqs, a.starts != nullptr, (int)a.heads, (int)c.heads, (int)c.dim, a.dtype, *cap,
                         a.causal ? a.window : 0, a.lse != nullptr);
  return plan->tiles * c.heads <= kMaxBlocks;
}

float scale_log2(float scale) { return (float)std::ldexp((double)scale * 1.4426950408889634, kQueryExponent); }

// What the parts of tiles take: outputs, {reference, sums}, and who holds them.
struct PartSizes {
  size_t out, ml, of;
  size_t bytes() const { return out + ml + of; }
};
PartSizes part_sizes(const ringsim_paged_attention_t& a, const AttentionPlan& plan) {
  const size_t rows = 2 * (size_t)plan.groups * (size_t)plan.tile_rows;
  if (plan.groups == 0) return PartSizes{0, 0, 0};
  return PartSizes{sizeof(float) * rows * (size_t)a.cache.dim, sizeof(float) * rows * 4,
                   sizeof(int32_t) * 2 * (size_t)(plan.tiles * a.cache.heads)};
}

}  // namespace

extern "C" {

ringsim_result_t ringsim_rotary(const ringsim_rotary_t* a, ringsim_stream_t stream) {
  const RoctxRange range("ringsim_rotary");
  int64_t tokens = 0;
  if (!a || !value_type(a->dtype) || !index_type(a->position_dtype) || !std::isfinite(a->scale) ||
      !token_count(a->outer, a->inner, &tokens))
    return RINGSIM_INVALID_ARGUMENT;
  if (a->heads < 0 || a->heads > kMaxHeads || a->dim < 1 || a->dim > RINGSIM_ROTARY_MAX_DIM || a->pairs < 0 ||
      a->pairs > a->dim / 2)
    return RINGSIM_INVALID_ARGUMENT;
  if (tokens == 0 || a->heads == 0) return RINGSIM_SUCCESS;
  const int64_t size[3] = {a->outer, a->inner, a->heads};
  if (!valid_heads(a->x, a->x_stride, a->outer, a->inner, a->heads, a->dim, a->dtype, false) ||
      !valid_heads(a->out, a->out_stride, a->outer, a->inner, a->heads, a->dim, a->dtype, true) ||
      !valid_index(a->positions, a->position_stride, a->outer, a->inner, a->position_dtype) ||
      !valid_frequencies(a->frequencies, a->pairs))
    return RINGSIM_INVALID_ARGUMENT;
  if (a->x == a->out)  // in place, so in the same places
    for (int i = 0; i < 3; ++i)
      if (size[i] > 1 && a->x_stride[i] != a->out_stride[i]) return RINGSIM_INVALID_ARGUMENT;
  RotaryArgs k;
  std::memset(&k, 0, sizeof(k));
  k.x = HeadRows{a->x, a->x_stride[0], a->x_stride[1], a->x_stride[2]};
  k.out = HeadRowsOut{a->out, a->out_stride[0], a->out_stride[1], a->out_stride[2]};
  k.positions = index_of(a->positions, a->position_stride, a->position_dtype);
  k.frequencies = a->frequencies;
  k.tokens = (uint32_t)tokens;
  k.inner = (uint32_t)a->inner;
  k.heads = (uint32_t)a->heads;
  k.dim = (int)a->dim;
  k.pairs = (int)a->pairs;
  k.interleaved = a->interleaved != 0;
  k.sign = a->inverse ? -1.0f : 1.0f;
  k.scale = a->scale;
  return result_of(launch_rotary(k, a->dtype, static_cast<hipStream_t>(stream)));
}

ringsim_result_t ringsim_kv_append(const ringsim_kv_append_t* a, ringsim_stream_t stream) {
  const RoctxRange range("ringsim_kv_append");
  int64_t tokens = 0;
  if (!a || !value_type(a->dtype) || !std::isfinite(a->scale) || !valid_cache(a->cache, true) ||
      !token_count(a->outer, a->inner, &tokens) || a->pairs < 0 || a->pairs > a->cache.dim / 2)
    return RINGSIM_INVALID_ARGUMENT;
  if (!index_type(a->slot_dtype) || (a->pairs > 0 && !index_type(a->position_dtype))) return RINGSIM_INVALID_ARGUMENT;
  if (tokens == 0) return RINGSIM_SUCCESS;
  const ringsim_kv_cache_t& c = a->cache;
  if (!valid_heads(a->k, a->k_stride, a->outer, a->inner, c.heads, c.dim, a->dtype, false) ||
      !valid_heads(a->v, a->v_stride, a->outer, a->inner, c.heads, c.dim, a->dtype, false) ||
      !valid_index(a->slots, a->slot_stride, a->outer, a->inner, a->slot_dtype) ||
      (a->pairs > 0 && !valid_index(a->positions, a->position_stride, a->outer, a->inner, a->position_dtype)) ||
      !valid_frequencies(a->frequencies, a->pairs))
    return RINGSIM_INVALID_ARGUMENT;
  KvAppendArgs k;
  std::memset(&k, 0, sizeof(k));
  k.cache = cache_args(c);
  k.x[0] = HeadRows{a->k, a->k_stride[0], a->k_stride[1], a->k_stride[2]};
  k.x[1] = HeadRows{a->v, a->v_stride[0], a->v_stride[1], a->v_stride[2]};
  k.slots = index_of(a->slots, a->slot_stride, a->slot_dtype);
  k.positions = index_of(a->positions, a->position_stride, a->position_dtype);
  k.frequencies = a->frequencies;
  k.tokens = (uint32_t)tokens;
  k.inner = (uint32_t)a->inner;
  k.pairs = (int)a->pairs;
  k.interleaved = a->interleaved != 0;
  k.scale = a->scale;
  return result_of(launch_kv_append(k, a->dtype, static_cast<hipStream_t>(stream)));
}

ringsim_result_t ringsim_kv_read(const ringsim_kv_read_t* a, ringsim_stream_t stream) {
  const RoctxRange range("ringsim_kv_read");
  int64_t tokens = 0;
  if (!a || !value_type(a->dtype) || !index_type(a->slot_dtype) || !valid_cache(a->cache, false) ||
      !token_count(a->outer, a->inner, &tokens))
    return RINGSIM_INVALID_ARGUMENT;
  if (tokens == 0 || (!a->k && !a->v)) return RINGSIM_SUCCESS;
  const ringsim_kv_cache_t& c = a->cache;
  if ((a->k && !valid_heads(a->k, a->k_stride, a->outer, a->inner, c.heads, c.dim, a->dtype, true)) ||
      (a->v && !valid_heads(a->v, a->v_stride, a->outer, a->inner, c.heads, c.dim, a->dtype, true)) ||
      !valid_index(a->slots, a->slot_stride, a->outer, a->inner, a->slot_dtype))
    return RINGSIM_INVALID_ARGUMENT;
  KvReadArgs k;
  std::memset(&k, 0, sizeof(k));
  k.cache = cache_args(c);
  k.out[0] = HeadRowsOut{a->k, a->k_stride[0], a->k_stride[1], a->k_stride[2]};
  k.out[1] = HeadRowsOut{a->v, a->v_stride[0], a->v_stride[1], a->v_stride[2]};
  k.slots = index_of(a->slots, a->slot_stride, a->slot_dtype);
  k.tokens = (uint32_t)tokens;
  k.inner = (uint32_t)a->inner;
  return result_of(launch_kv_read(k, a->dtype, static_cast<hipStream_t>(stream)));
}

ringsim_result_t ringsim_paged_attention_workspace(const ringsim_paged_attention_t* a, size_t* bytes) {
  AttentionPlan plan;
  int64_t cap = 0;
  plan.groups = 0;
  if (!a || !bytes || !plan_of(*a, &plan, &cap)) return RINGSIM_INVALID_ARGUMENT;
  *bytes = part_sizes(*a, plan).bytes();
  return RINGSIM_SUCCESS;
}

ringsim_result_t ringsim_paged_attention(const ringsim_paged_attention_t* a, ringsim_stream_t stream) {
  const RoctxRange range("ringsim_paged_attention");
  AttentionPlan plan;
  int64_t cap = 0;
  if (!a || !valid_cache(a->cache, false) || !plan_of(*a, &plan, &cap) || !(a->scale > 0.0f) ||
      !std::isfinite(scale_log2(a->scale)))
    return RINGSIM_INVALID_ARGUMENT;
  if (a->seqs == 0 || a->tokens == 0) return RINGSIM_SUCCESS;
  const ringsim_kv_cache_t& c = a->cache;
  const int64_t seqs = a->starts ? 1 : a->seqs, each = a->tokens / seqs;
  const int64_t q_stride[3] = {a->q_seq_stride, a->q_stride[0], a->q_stride[1]};
  const int64_t out_stride[3] = {a->out_seq_stride, a->out_stride[0], a->out_stride[1]};
  if (!valid_heads(a->q, q_stride, seqs, each, a->heads, c.dim, a->dtype, false) ||
      !valid_heads(a->out, out_stride, seqs, each, a->heads, c.dim, a->dtype, true))
    return RINGSIM_INVALID_ARGUMENT;
  if (!a->lengths || !aligned(a->lengths, 4) || (a->starts && !aligned(a->starts, 4)) ||
      (a->lse && !aligned(a->lse, 4)))
    return RINGSIM_INVALID_ARGUMENT;
  const int64_t table[1] = {a->seqs}, table_stride[1] = {a->page_stride};
  if (a->max_pages > 0 && (!a->pages || !aligned(a->pages, 4) || !strides_fit(table_stride, table, 1)))
    return RINGSIM_INVALID_ARGUMENT;
  const PartSizes parts = part_sizes(*a, plan);
  if (parts.bytes() > 0 && (!a->workspace || !aligned(a->workspace, 16) || a->workspace_bytes < parts.bytes()))
    return RINGSIM_INVALID_ARGUMENT;
  AttentionArgs k;
  std::memset(&k, 0, sizeof(k));
  k.cache = cache_args(c);
  k.q = HeadRows{a->q, q_stride[0], q_stride[1], q_stride[2]};
  k.out = HeadRowsOut{a->out, out_stride[0], out_stride[1], out_stride[2]};
  k.lse = a->lse;
  k.pages = a->pages;
  k.lengths = a->lengths;
  k.starts = a->starts;
  if (parts.bytes() > 0) {
    char* const at = static_cast<char*>(a->workspace);
    k.part_out = reinterpret_cast<float*>(at);
    k.part_ml = reinterpret_cast<float*>(at + parts.out);
    k.part_of = reinterpret_cast<int32_t*>(at + parts.out + parts.ml);
  }
  k.page_stride = a->page_stride;
  k.cap = (int)cap;
  k.max_pages = a->max_pages;
  k.tokens = (int)a->tokens;
  k.seqs = (int)a->seqs;
  k.window = a->window;
  k.each = (int)(a->tokens / a->seqs);
  k.seq_tiles = (int)(plan.tiles / a->seqs);  // read without starts
  k.groups = plan.groups;
  k.group = (int)(a->heads / c.heads);
  k.heads = (int)a->heads;
  k.tiles = (int)plan.tiles;
  k.tile_rows = plan.tile_rows;
  k.causal = a->causal != 0;
  k.scale_log2 = scale_log2(a->scale);
  return result_of(launch_attention(k, plan, a->dtype, static_cast<hipStream_t>(stream)));
}

}  // extern "C"
