// attention_binding.cpp -- the attention-step operators in the Python
// extension: checks torch tensors, allocates results and workspaces on the
// current stream, and calls the C ABI of include/ringsim_attention.h.
// attention.py holds the functions users call; arguments arrive here by
// position.
#include "binding.h"

#include "../../include/ringsim_attention.h"

using namespace ringsim_binding;

namespace {

int index_code(at::ScalarType t) {
  return t == at::kInt ? RINGSIM_INT32 : t == at::kLong ? RINGSIM_INT64 : -1;
}

// A [tokens, heads, dim] or [outer, inner, heads, dim] shape.
struct HeadShape {
  int64_t outer, inner, heads, dim;
};
HeadShape head_shape(at::IntArrayRef s, const char* name) {
  if (s.size() != 3 && s.size() != 4)
    throw WrongValue(std::string(name) + " must have three or four dimensions, not " + std::to_string(s.size()));
  if (s.size() == 3) return HeadShape{s[0], 1, s[1], s[2]};
  return HeadShape{s[0], s[1], s[2], s[3]};
}

void check_shape(const at::Tensor& t, const char* name, at::IntArrayRef shape) {
  if (t.sizes() != shape)
    throw WrongValue(std::string(name) + " must have shape " + shape_text(shape) + ", not " + shape_text(t.sizes()));
}
void check_type(const at::Tensor& t, const char* name, at::ScalarType type) {
  if (t.scalar_type() != type)
    throw WrongType(std::string(name) + " must have dtype " + c10::toString(type) + ", not " +
                    c10::toString(t.scalar_type()));
}
int value_code(const at::Tensor& t, const char* name) {
  const int code = type_code(t.scalar_type());
  if (code < 0) throw WrongType(std::string("unsupported dtype ") + c10::toString(t.scalar_type()) + " of " + name);
  return code;
}

// {outer, inner, head} strides of a tensor of heads; the shape has been checked.
void head_strides(const at::Tensor& t, const char* name, int64_t stride[3]) {
  check_strided(t, name);
  const auto st = t.strides();
  if (t.sizes().back() > 1 && st.back() != 1)
    throw WrongValue(std::string("the last dimension of ") + name + " must be contiguous");
  const bool four = t.dim() == 4;
  stride[0] = st[0];
  stride[1] = four ? st[1] : 0;
  stride[2] = st[four ? 2 : 1];
}

int check_index(const at::Tensor& t, const char* name) {
  const int code = index_code(t.scalar_type());
  if (code < 0)
    throw WrongType(std::string(name) + " must have dtype Int or Long, not " + c10::toString(t.scalar_type()));
  return code;
}

// Whole numbers, one a token: of the tokens' shape, or, for positions, of the
// inner dimension alone where all of the outer one share them.
int index_strides(const at::Tensor& t, const char* name, at::IntArrayRef tokens, bool shared, int64_t stride[2]) {
  check_strided(t, name);
  const int code = check_index(t, name);
  if (shared && tokens.size() == 2 && t.dim() == 1) {
    check_shape(t, name, tokens.slice(1));
    stride[0] = 0;
    stride[1] = t.stride(0);
  } else {
    check_shape(t, name, tokens);
    stride[0] = t.stride(0);
    stride[1] = t.dim() == 2 ? t.stride(1) : 0;
  }
  return code;
}

int64_t frequency_pairs(const at::Tensor& f, int64_t dim) {
  check_strided(f, "frequencies");
  if (f.dim() != 1) throw WrongValue("frequencies must have one dimension");
  if (2 * f.size(0) > dim)
    throw WrongValue(std::to_string(f.size(0)) + " frequencies turn more than " + std::to_string(dim) + " columns");
  if (!f.is_contiguous()) throw WrongValue("frequencies must be contiguous");
  return f.size(0);
}

int truth(PyObject* o) {
  const int v = PyObject_IsTrue(o);
  if (v < 0) throw PythonError{};
  return v;
}

template <typename T>
T* typed(const at::Tensor& t) {
  return static_cast<T*>(data(t));
}

// rotary(x, positions, frequencies, interleaved, inverse, scale, out)
PyObject* rotary(PyObject*, PyObject* const* args, Py_ssize_t nargs) {
  return guarded([&] {
    want_args(nargs, 7);
    const int inverse = truth(args[4]);
    const at::Tensor &x = required(args[0], inverse ? "grad_out" : "x"), &pos = required(args[1], "positions"),
                     &freq = required(args[2], "frequencies");
    const at::Tensor* out = tensor(args[6], inverse ? "grad_in" : "out");
    const int device = current_device();
    ringsim_rotary_t a{};
    a.interleaved = truth(args[3]);
    a.inverse = inverse;
    a.scale = (float)number(args[5]);
    const char *x_name = inverse ? "grad_out" : "x", *out_name = inverse ? "grad_in" : "out";
    a.dtype = value_code(x, x_name);
    if (out) check_type(*out, out_name, x.scalar_type());
    check_index(pos, "positions");
    check_type(freq, "frequencies", at::kDouble);
    const HeadShape s = head_shape(x.sizes(), x_name);
    const auto tokens = x.sizes().slice(0, x.dim() - 2);
    if (out) {
      check_shape(*out, out_name, x.sizes());
      head_strides(*out, out_name, a.out_stride);
      check_device(*out, device, out_name);
    }
    a.position_dtype = index_strides(pos, "positions", tokens, true, a.position_stride);
    a.pairs = frequency_pairs(freq, s.dim);
    head_strides(x, x_name, a.x_stride);
    check_device(x, device, x_name);
    check_device(pos, device, "positions");
    check_device(freq, device, "frequencies");
    a.outer = s.outer;
    a.inner = s.inner;
    a.heads = s.heads;
    a.dim = s.dim;
    at::Tensor made;
    {
      const Unlocked unlocked;
      if (!out) {
        made = empty(x.sizes(), x.scalar_type(), device);
        head_strides(made, out_name, a.out_stride);
        out = &made;
      }
      a.x = data(x);
      a.out = data(*out);
      a.positions = data(pos);
      a.frequencies = typed<const double>(freq);
      check(ringsim_rotary(&a, current_stream(device)), "ringsim_rotary");
    }
    written(args[6]);
    return result(args[6], made);
  });
}

// A cache's four tensors, which have to agree.
struct Cache {
  const at::Tensor* t[4];
  ringsim_kv_cache_t c{};

  static constexpr const char* names[4] = {"cache.keys", "cache.values", "cache.key_scales", "cache.value_scales"};

  explicit Cache(PyObject* o) {
    if (!PyTuple_Check(o) || PyTuple_GET_SIZE(o) != 4) throw WrongType("cache must be a KvCache");
    for (int i = 0; i < 4; ++i) {
      t[i] = &required(PyTuple_GET_ITEM(o, i), names[i]);
      check_type(*t[i], names[i], at::kByte);
    }
  }

  // Shapes and places, after the types of all of a call's arguments.
  void take(int device) {
    for (int i = 0; i < 4; ++i) {
      if (t[i]->dim() != 4) throw WrongValue(std::string(names[i]) + " must have four dimensions");
      check_strided(*t[i], names[i]);
    }
    const auto s = t[0]->sizes();
    c.pages = s[0];
    c.heads = s[1];
    c.page_size = s[2];
    c.dim = 2 * s[3];
    if (c.dim != 64 && c.dim != 96 && c.dim != 128 && c.dim != 192 && c.dim != 256)
      throw WrongValue("a cache's heads have 64, 96, 128, 192 or 256 columns, not " + std::to_string(c.dim));
    if (c.page_size < 16 || c.page_size > RINGSIM_KV_MAX_PAGE || (c.page_size & (c.page_size - 1)))
      throw WrongValue("a cache's pages hold a power of two of tokens from 16 to " +
                       std::to_string(RINGSIM_KV_MAX_PAGE) + ", not " + std::to_string(c.page_size));
    check_shape(*t[1], names[1], s);
    const int64_t scales[4] = {c.pages, c.heads, c.dim / 32, c.page_size};
    for (int i = 2; i < 4; ++i) check_shape(*t[i], names[i], scales);
    for (int i = 0; i < 4; ++i) {
      const auto st = t[i]->strides();
      if (st[3] != 1 || st[2] != t[i]->size(3))
        throw WrongValue(std::string("the last two dimensions of ") + names[i] + " must be contiguous");
      for (int d = 0; d < 2; ++d)
        if (t[i]->size(d) > 1 && st[d] != t[i & 2]->stride(d))
          throw WrongValue(i < 2 ? "cache.keys and cache.values must have the same strides"
                                 : "cache.key_scales and cache.value_scales must have the same strides");
      check_device(*t[i], device, names[i]);
    }
    for (int d = 0; d < 2; ++d) {
      c.stride[d] = t[0]->stride(d);
      c.scale_stride[d] = t[2]->stride(d);
    }
    c.keys = typed<uint8_t>(*t[0]);
    c.values = typed<uint8_t>(*t[1]);
    c.key_scales = typed<uint8_t>(*t[2]);
    c.value_scales = typed<uint8_t>(*t[3]);
  }
};

// kv_append(cache, k, v, slots, positions, frequencies, interleaved, scale)
PyObject* kv_append(PyObject*, PyObject* const* args, Py_ssize_t nargs) {
  return guarded([&] {
    want_args(nargs, 8);
    const int device = current_device();
    Cache cache(args[0]);
    const at::Tensor &k = required(args[1], "k"), &v = required(args[2], "v"), &slots = required(args[3], "slots");
    const at::Tensor *pos = tensor(args[4], "positions"), *freq = tensor(args[5], "frequencies");
    ringsim_kv_append_t a{};
    a.interleaved = truth(args[6]);
    a.scale = (float)number(args[7]);
    a.dtype = value_code(k, "k");
    check_type(v, "v", k.scalar_type());
    check_index(slots, "slots");
    if (pos) check_index(*pos, "positions");
    if (freq) check_type(*freq, "frequencies", at::kDouble);
    cache.take(device);
    a.cache = cache.c;
    const HeadShape s = head_shape(k.sizes(), "k");
    if (s.heads != cache.c.heads || s.dim != cache.c.dim)
      throw WrongValue("k has heads of another number or size than the cache");
    check_shape(v, "v", k.sizes());
    const auto tokens = k.sizes().slice(0, k.dim() - 2);
    a.slot_dtype = index_strides(slots, "slots", tokens, false, a.slot_stride);
    if (freq) a.pairs = frequency_pairs(*freq, s.dim);
    if (a.pairs > 0) {
      if (!pos) throw WrongValue("frequencies need positions");
      a.position_dtype = index_strides(*pos, "positions", tokens, true, a.position_stride);
      check_device(*pos, device, "positions");
      check_device(*freq, device, "frequencies");
    }
    head_strides(k, "k", a.k_stride);
    head_strides(v, "v", a.v_stride);
    check_device(k, device, "k");
    check_device(v, device, "v");
    check_device(slots, device, "slots");
    a.outer = s.outer;
    a.inner = s.inner;
    {
      const Unlocked unlocked;
      a.k = data(k);
      a.v = data(v);
      a.slots = data(slots);
      a.positions = a.pairs > 0 ? data(*pos) : nullptr;
      a.frequencies = a.pairs > 0 ? typed<const double>(*freq) : nullptr;
      check(ringsim_kv_append(&a, current_stream(device)), "ringsim_kv_append");
    }
    for (int i = 0; i < 4; ++i) written(PyTuple_GET_ITEM(args[0], i));
    return none();
  });
}

// kv_read(cache, slots, dtype of the code, keys, values)
PyObject* kv_read(PyObject*, PyObject* const* args, Py_ssize_t nargs) {
  return guarded([&] {
    want_args(nargs, 5);
    const int device = current_device();
    Cache cache(args[0]);
    const at::Tensor& slots = required(args[1], "slots");
    ringsim_kv_read_t a{};
    a.dtype = (int)whole(args[2]);
    const at::ScalarType type = a.dtype == RINGSIM_FLOAT32 ? at::kFloat : a.dtype == RINGSIM_BFLOAT16 ? at::kBFloat16
                                                                                                     : at::kHalf;
    check_index(slots, "slots");
    const at::Tensor* given[2] = {tensor(args[3], "keys"), tensor(args[4], "values")};
    static const char* const names[2] = {"keys", "values"};
    for (int i = 0; i < 2; ++i)
      if (given[i]) check_type(*given[i], names[i], type);
    cache.take(device);
    a.cache = cache.c;
    if (slots.dim() != 1 && slots.dim() != 2) throw WrongValue("slots must have one or two dimensions");
    a.slot_dtype = index_strides(slots, "slots", slots.sizes(), false, a.slot_stride);
    check_device(slots, device, "slots");
    c10::SmallVector<int64_t, 4> shape(slots.sizes().begin(), slots.sizes().end());
    shape.push_back(cache.c.heads);
    shape.push_back(cache.c.dim);
    for (int i = 0; i < 2; ++i) {
      if (!given[i]) continue;
      check_shape(*given[i], names[i], shape);
      head_strides(*given[i], names[i], i ? a.v_stride : a.k_stride);
      check_device(*given[i], device, names[i]);
    }
    a.outer = slots.size(0);
    a.inner = slots.dim() == 2 ? slots.size(1) : 1;
    at::Tensor made[2];
    {
      const Unlocked unlocked;
      for (int i = 0; i < 2; ++i) {
        if (!given[i]) {
          made[i] = empty(shape, type, device);
          head_strides(made[i], names[i], i ? a.v_stride : a.k_stride);
          given[i] = &made[i];
        }
      }
      a.k = data(*given[0]);
      a.v = data(*given[1]);
      a.slots = data(slots);
      check(ringsim_kv_read(&a, current_stream(device)), "ringsim_kv_read");
    }
    written(args[3]);
    written(args[4]);
    return pack({result(args[3], made[0]), result(args[4], made[1])});
  });
}

// paged_attention(q, cache, pages, lengths, starts, causal, window, scale, max_length, out, lse, need_lse)
PyObject* paged_attention(PyObject*, PyObject* const* args, Py_ssize_t nargs) {
  return guarded([&] {
    want_args(nargs, 12);
    const int device = current_device();
    const at::Tensor& q = required(args[0], "q");
    Cache cache(args[1]);
    const at::Tensor &pages = required(args[2], "pages"), &lengths = required(args[3], "lengths");
    const at::Tensor *starts = tensor(args[4], "starts"), *out = tensor(args[9], "out"), *lse = tensor(args[10], "lse");
    ringsim_paged_attention_t a{};
    a.causal = truth(args[5]);
    a.window = whole(args[6]);
    a.max_length = args[8] == Py_None ? 0 : whole(args[8]);
    const int need_lse = truth(args[11]);
    const double scale = args[7] == Py_None ? 0.0 : number(args[7]);
    a.dtype = value_code(q, "q");
    check_type(pages, "pages", at::kInt);
    check_type(lengths, "lengths", at::kInt);
    if (starts) check_type(*starts, "starts", at::kInt);
    if (out) check_type(*out, "out", q.scalar_type());
    if (lse) check_type(*lse, "lse", at::kFloat);
    if (a.window < 0) throw WrongValue("window must not be negative");
    if (args[8] != Py_None && a.max_length < 1) throw WrongValue("max_length must be above 0");
    cache.take(device);
    a.cache = cache.c;
    const HeadShape s = head_shape(q.sizes(), "q");
    a.scale = args[7] == Py_None ? (float)(1.0 / std::sqrt((double)s.dim)) : (float)scale;
    if (s.dim != cache.c.dim) throw WrongValue("q has heads of another size than the cache");
    if (s.heads < 1 || s.heads % cache.c.heads)
      throw WrongValue("q must have a multiple of the cache's " + std::to_string(cache.c.heads) + " heads, not " +
                       std::to_string(s.heads));
    check_strided(pages, "pages");
    if (pages.dim() != 2) throw WrongValue("pages must have two dimensions");
    a.seqs = pages.size(0);
    a.max_pages = pages.size(1);
    if (a.max_pages > 1 && pages.stride(1) != 1) throw WrongValue("the last dimension of pages must be contiguous");
    a.page_stride = pages.stride(0);
    check_shape(lengths, "lengths", {a.seqs});
    if (!lengths.is_contiguous()) throw WrongValue("lengths must be contiguous");
    if (starts) {
      if (q.dim() != 3) throw WrongValue("q must have three dimensions with starts");
      check_shape(*starts, "starts", {a.seqs + 1});
      if (!starts->is_contiguous()) throw WrongValue("starts must be contiguous");
      check_device(*starts, device, "starts");
    } else if (s.outer != a.seqs) {
      throw WrongValue("without starts q must have the " + std::to_string(a.seqs) + " sequences of pages, not " +
                       std::to_string(s.outer));
    }
    check_device(pages, device, "pages");
    check_device(lengths, device, "lengths");
    const auto strides = [&](const at::Tensor& t, const char* name, int64_t* seq, int64_t stride[2]) {
      int64_t st[3];
      head_strides(t, name, st);
      check_device(t, device, name);
      *seq = st[0];
      stride[0] = starts ? st[0] : st[1];
      stride[1] = st[2];
    };
    strides(q, "q", &a.q_seq_stride, a.q_stride);
    if (out) {
      check_shape(*out, "out", q.sizes());
      strides(*out, "out", &a.out_seq_stride, a.out_stride);
    }
    const auto lse_shape = q.sizes().slice(0, q.dim() - 1);
    if (lse) {
      check_shape(*lse, "lse", lse_shape);
      if (!lse->is_contiguous()) throw WrongValue("lse must be contiguous");
      check_device(*lse, device, "lse");
    }
    a.tokens = s.outer * s.inner;
    a.heads = s.heads;
    at::Tensor made_out, made_lse, workspace;
    {
      const Unlocked unlocked;
      if (!out) {
        made_out = empty(q.sizes(), q.scalar_type(), device);
        strides(made_out, "out", &a.out_seq_stride, a.out_stride);
        out = &made_out;
      }
      if (!lse && need_lse) {
        made_lse = empty(lse_shape, at::kFloat, device);
        lse = &made_lse;
      }
      a.q = data(q);
      a.out = data(*out);
      a.lse = lse ? typed<float>(*lse) : nullptr;
      a.pages = typed<const int32_t>(pages);
      a.lengths = typed<const int32_t>(lengths);
      a.starts = starts ? typed<const int32_t>(*starts) : nullptr;
      check(ringsim_paged_attention_workspace(&a, &a.workspace_bytes), "ringsim_paged_attention_workspace");
      if (a.workspace_bytes) {
        workspace = empty({(int64_t)a.workspace_bytes}, at::kByte, device);
        a.workspace = data(workspace);
      }
      check(ringsim_paged_attention(&a, current_stream(device)), "ringsim_paged_attention");
    }
    written(args[9]);
    written(args[10]);
    return pack({result(args[9], made_out), result(args[10], made_lse)});
  });
}

}  // namespace

PyMethodDef g_attention_methods[] = {
    {"rotary", fast(rotary), METH_FASTCALL, nullptr},
    {"kv_append", fast(kv_append), METH_FASTCALL, nullptr},
    {"kv_read", fast(kv_read), METH_FASTCALL, nullptr},
    {"paged_attention", fast(paged_attention), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr},
};
