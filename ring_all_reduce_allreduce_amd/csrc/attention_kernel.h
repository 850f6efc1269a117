// attention_kernel.h -- softmax attention over the paged 4-bit cache.
//
// A workgroup takes one key head of one sequence and some rows of queries: a
// row is a token with one of the query heads that share the key head. Per
// pass of 32 positions a wave forms
//     S^T = K Q^T       (16 positions x 16 rows a matrix instruction),
//     P   = exp2(S * scale * log2(e) - m),
//     O^T += V^T P^T,   l += 1^T P^T.
// With S transposed, a lane's results S^T are the four positions 4 g + i (g
// its group of 16 lanes) of one row, and two tiles of 16 positions are just
// the eight positions that the lane has to bring into the second product: the
// weights never change lanes. V's operand then has the same eight positions
// of one column, so a lane reads a few columns of each of its positions,
// dequantises pairs of columns, and swaps halves between positions.
//
// Keys and values go from memory to registers and never through LDS. The
// conversion instruction turns two codes and an exponent into two bf16, which
// hold every value of the cache.
#pragma once

#include "attention_device.h"

namespace ringsim {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

typedef uint32_t u32x4a __attribute__((ext_vector_type(4)));

constexpr int kAttentionWaves = 4;
constexpr int kAttentionThreads = 64 * kAttentionWaves;

// How far (as a power of two) weights may grow before a row's reference
// exponent follows its maximum. Sums and products in fp32 lose nothing by it,
// and most passes need no maximum over lanes and no rescaling.
constexpr float kSlack = 8.0f;

// A head's columns in the second product: parts of n blocks of 32 columns, n
// a power of two. Lane c of a group of 16 holds the 2 n columns from 2 n c on,
// n bytes a position.
template <int D>
struct HeadParts {
  static constexpr int kBlocks = D / 32;
  static constexpr int kParts = (kBlocks & (kBlocks - 1)) ? 2 : 1;
  static constexpr int n(int p) {
    int top = 1;
    while (2 * top <= kBlocks) top *= 2;
    return p == 0 ? top : kBlocks - top;
  }
  static constexpr int base(int p) { return p == 0 ? 0 : 32 * n(0); }
  static constexpr int regs(int p) { return n(p) > 4 ? 2 : 1; }
  static constexpr int reg0(int p) { return p == 0 ? 0 : regs(0); }
  static constexpr int kRegs = regs(0) + (kParts == 2 ? regs(1) : 0);
};

// 32 positions of the cache as they lie in memory.
template <int D>
struct KvRaw {
  using H = HeadParts<D>;
  // A lane holds D / 4 columns of a key: one exponent where that is a whole
  // part of a block, else two.
  static constexpr int kKeyScales = 32 % (D / 4) == 0 ? 1 : 2;
  uint32_t k[2][D / 32];
  uint32_t ks[2][kKeyScales];
  uint32_t v[8][H::kRegs];
  uint32_t vs[2][H::kParts];
};

template <int N>
__device__ __forceinline__ void load_bytes(uint32_t* w, const uint8_t* p) {
  if constexpr (N == 1) {
    w[0] = *p;
  } else if constexpr (N == 2) {
    w[0] = *reinterpret_cast<const uint16_t*>(p);
  } else if constexpr (N == 4) {
    w[0] = *reinterpret_cast<const uint32_t*>(p);
  } else if constexpr (N == 8) {
    const u32x2 x = *reinterpret_cast<const u32x2*>(p);
    w[0] = x[0];
    w[1] = x[1];
  } else if constexpr (N == 12) {
    typedef uint32_t u32x3 __attribute__((ext_vector_type(3)));
    typedef u32x3 u32x3_e4 __attribute__((aligned(4)));
    const u32x3_e4 x = *reinterpret_cast<const u32x3_e4*>(p);
    w[0] = x[0];
    w[1] = x[1];
    w[2] = x[2];
  } else if constexpr (N == 24) {
    load_bytes<8>(w, p);
    load_bytes<8>(w + 2, p + 8);
    load_bytes<8>(w + 4, p + 16);
  } else {
    static_assert(N % 16 == 0, "bytes");
#pragma unroll
    for (int i = 0; i < N / 16; ++i) {
      const u32x4a x = *reinterpret_cast<const u32x4a*>(p + 16 * i);
#pragma unroll
      for (int j = 0; j < 4; ++j) w[4 * i + j] = x[j];
    }
  }
}

// Exponent byte I of a word where the conversion reads it, in the exponent's
// place of an fp32; it takes no notice of the other bits.
template <int I>
__device__ __forceinline__ float unit_of(uint32_t w) {
  return __uint_as_float(I == 3 ? w >> 1 : w << (23 - 8 * I));
}

template <int SEL>
__device__ __forceinline__ uint32_t two_columns(uint32_t codes, float unit) {
  return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, unit, SEL));
}
__device__ __forceinline__ uint32_t two_columns(uint32_t codes, float unit, int sel) {
  switch (sel) {
    case 0: return two_columns<0>(codes, unit);
    case 1: return two_columns<1>(codes, unit);
    case 2: return two_columns<2>(codes, unit);
    default: return two_columns<3>(codes, unit);
  }
}

__device__ __forceinline__ f32x4 mfma(const u32x4a& x, const u32x4a& y, f32x4 acc) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, x), __builtin_bit_cast(bf16x8, y), acc, 0,
                                                 0, 0);
}

// The largest over the four groups of 16 lanes, known to each.
__device__ __forceinline__ float groups_max(float v) {
  uint32_t u = __float_as_uint(v);
  const auto s = __builtin_amdgcn_permlane16_swap(u, u, false, false);
  v = fmaxf(__uint_as_float(s[0]), __uint_as_float(s[1]));
  u = __float_as_uint(v);
  const auto t = __builtin_amdgcn_permlane32_swap(u, u, false, false);
  return fmaxf(__uint_as_float(t[0]), __uint_as_float(t[1]));
}

// bf16 parts that queries of a type are split into: their 8, 11 or 24 bits.
template <int DT>
constexpr int kQueryTerms = DT == RINGSIM_FLOAT32 ? 3 : DT == RINGSIM_FLOAT16 ? 2 : 1;

// Splits x into bf16 parts whose sum it is, by cutting off (rounding could
// carry a large x to infinity). Only the first part of an infinity is one.
template <int TERMS>
__device__ __forceinline__ void split_exact(float x, uint32_t (&part)[TERMS]) {
  if (!(x == x)) x = __uint_as_float(0x7fc00000u);
  const bool finite = fabsf(x) < __uint_as_float(0x7f800000u);
#pragma unroll
  for (int t = 0; t < TERMS; ++t) {
    const uint32_t hi = __float_as_uint(x) & 0xffff0000u;
    part[t] = hi >> 16;
    x = finite ? x - __uint_as_float(hi) : 0.0f;
  }
}

// What a wave has to do, the same for all of its lanes.
struct WaveJob {
  const uint8_t* k;        // of the key head: keys, values and their scales of page 0
  const uint8_t* v;
  const uint8_t* ks;
  const uint8_t* vs;
  const int32_t* pages;    // of the sequence
  int64_t begin, end;      // positions, begin a multiple of kKvStep; `end` past the last one wanted
  int64_t stride;          // from one pass of this wave to the next
  int64_t full_lo, full_hi;// positions that every row of the wave sees
  int64_t length;          // positions of the sequence
};

template <int DT, int D, int NQ, int PT>
struct AttentionWave {
  using H = HeadParts<D>;
  static constexpr int kSteps = D / 32;  // matrix instructions over a head's columns
  static constexpr int kQT = kQueryTerms<DT>;

  u32x4a q[NQ][kQT][kSteps];
  f32x4 o[NQ][D / 16];
  f32x4 l[NQ];
  float m[NQ];             // reference exponent, minus infinity until a position is seen
  int64_t lo[NQ], hi[NQ];  // positions that this lane's row sees
  int32_t ids;             // lane i: page of the wave's tile i of the next 64, -1: none

  __device__ __forceinline__ void clear() {
    const f32x4 zero = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int r = 0; r < NQ; ++r) {
      m[r] = -__builtin_inff();
      l[r] = zero;
#pragma unroll
      for (int d = 0; d < D / 16; ++d) o[r][d] = zero;
    }
  }

  // Columns g * D / 4 + 8 s + i of the row are element i of step s.
  __device__ __forceinline__ void load_queries(int r, const typename OpElem<DT>::T* row) {
    const int g = (threadIdx.x & 63) >> 4;
#pragma unroll
    for (int s = 0; s < kSteps; ++s) {
      Packed<DT, 8> x;
      x.load(row + g * (D / 4) + 8 * s);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        uint32_t a[kQT], b[kQT];
        split_exact<kQT>(x.get(2 * j) * kQueryUnit, a);
        split_exact<kQT>(x.get(2 * j + 1) * kQueryUnit, b);
#pragma unroll
        for (int t = 0; t < kQT; ++t) q[r][t][s][j] = a[t] | b[t] << 16;
      }
    }
  }

  // Pages of the 64 tiles of the next 32 passes, from position `at` on.
  __device__ __forceinline__ void load_pages(const AttentionArgs& a, const WaveJob& job, int64_t at) {
    const int lane = threadIdx.x & 63;
    const int64_t tile = (at + (lane >> 1) * job.stride) / kKvTile + (lane & 1);
    ids = kv_page_of_tile(job.pages, tile, job.length, a.cache.page_shift, a.max_pages, a.cache.pages);
  }

  // `n`: the pass's number modulo 32. A tile without a page is read from page 0 and not seen.
  __device__ __forceinline__ void load(const AttentionArgs& a, const WaveJob& job, int64_t at, int n, KvRaw<D>& raw) {
    const int lane = threadIdx.x & 63, c = lane & 15, g = lane >> 4;
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      const int32_t id = __builtin_amdgcn_readlane(ids, 2 * n + t);
      const int64_t page = id < 0 ? 0 : id;
      const int off = (int)((at + kKvTile * t) & ((1 << a.cache.page_shift) - 1));
      const int64_t data = page * a.cache.page + (int64_t)off * (D / 2);
      const int64_t scale = page * a.cache.scale_page + off;
      load_bytes<D / 8>(raw.k[t], job.k + data + c * (D / 2) + g * (D / 8));
      const int block = g * (D / 4) / 32;
#pragma unroll
      for (int i = 0; i < KvRaw<D>::kKeyScales; ++i)
        raw.ks[t][i] = job.ks[scale + ((block + i < D / 32 ? block + i : block) << a.cache.page_shift) + c];
#pragma unroll
      for (int p = 0; p < H::kParts; ++p) {
        const int n_p = H::n(p);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint8_t* from = job.v + data + (4 * g + i) * (D / 2) + H::base(p) / 2 + c * n_p;
          uint32_t* to = raw.v[4 * t + i] + H::reg0(p);
          if (n_p == 1) load_bytes<1>(to, from);
          if (n_p == 2) load_bytes<2>(to, from);
          if (n_p == 4) load_bytes<4>(to, from);
          if (n_p == 8) load_bytes<8>(to, from);
        }
        const int b = H::base(p) / 32 + c * n_p / 16;
        raw.vs[t][p] = *reinterpret_cast<const uint32_t*>(job.vs + scale + (b << a.cache.page_shift) + 4 * g);
      }
    }
  }

  // One pass over the 32 positions from `at` on. SLOW: a position's NaN values
  // reach the rows that see it and no others, which 0 * NaN would not do.
  template <bool SLOW>
  __device__ __forceinline__ void pass(const AttentionArgs& a, const WaveJob& job, int64_t at, int n,
                                       const KvRaw<D>& raw) {
    const int lane = threadIdx.x & 63, g = lane >> 4;
    const f32x4 zero = {0.0f, 0.0f, 0.0f, 0.0f};
    f32x4 s[NQ][2];
#pragma unroll
    for (int t = 0; t < 2; ++t) {
#pragma unroll
      for (int r = 0; r < NQ; ++r) s[r][t] = zero;
#pragma unroll
      for (int k = 0; k < kSteps; ++k) {
        float unit;
        if constexpr (KvRaw<D>::kKeyScales == 1) {
          unit = unit_of<0>(raw.ks[t][0]);
        } else {
          const bool next = (g * (D / 4) + 8 * k) / 32 != g * (D / 4) / 32;
          unit = next ? unit_of<0>(raw.ks[t][1]) : unit_of<0>(raw.ks[t][0]);
        }
        const uint32_t w = raw.k[t][k];
        const u32x4a key = {two_columns<0>(w, unit), two_columns<1>(w, unit), two_columns<2>(w, unit),
                            two_columns<3>(w, unit)};
#pragma unroll
        for (int r = 0; r < NQ; ++r) {
#pragma unroll
          for (int e = kQT - 1; e >= 0; --e) s[r][t] = mfma(key, q[r][e][k], s[r][t]);
        }
      }
    }
    const bool there0 = __builtin_amdgcn_readlane(ids, 2 * n) >= 0, there1 = __builtin_amdgcn_readlane(ids, 2 * n + 1) >= 0;
    uint32_t seen[NQ];  // SLOW: a bit a position
    if (SLOW || !there0 || !there1 || at < job.full_lo || at + kKvStep - 1 > job.full_hi) {
#pragma unroll
      for (int r = 0; r < NQ; ++r) {
        seen[r] = 0;
#pragma unroll
        for (int t = 0; t < 2; ++t) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int64_t j = at + kKvTile * t + 4 * g + i;
            const bool on = j >= lo[r] && j <= hi[r] && (t ? there1 : there0);
            s[r][t][i] = on ? s[r][t][i] : -__builtin_inff();
            seen[r] |= (uint32_t)on << (4 * t + i);
          }
        }
      }
    }
    u32x4a p[NQ][PT];
#pragma unroll
    for (int r = 0; r < NQ; ++r) {
      float top = fmaxf(fmaxf(fmaxf(s[r][0][0], s[r][0][1]), fmaxf(s[r][0][2], s[r][0][3])),
                        fmaxf(fmaxf(s[r][1][0], s[r][1][1]), fmaxf(s[r][1][2], s[r][1][3])));
      top *= a.scale_log2;
      if (__any(top > m[r] + kSlack)) {
        const float next = fmaxf(m[r], groups_max(top));
        // exp2(-inf) = 0 on a row's first positions; a row without any keeps its zeros.
        const float by = next == m[r] ? 1.0f : __builtin_amdgcn_exp2f(m[r] - next);
        m[r] = next;
        l[r] *= by;
#pragma unroll
        for (int d = 0; d < D / 16; ++d) o[r][d] *= by;
      }
      const float ref = m[r] == -__builtin_inff() ? 0.0f : m[r];
      float w[8];
#pragma unroll
      for (int i = 0; i < 8; ++i)
        w[i] = __builtin_amdgcn_exp2f(__builtin_fmaf(s[r][i / 4][i % 4], a.scale_log2, -ref));
#pragma unroll
      for (int e = 0; e < PT; ++e) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const uint32_t x = to_bf16x2(w[2 * j], w[2 * j + 1]);
          p[r][e][j] = x;
          if (e + 1 < PT) {
            w[2 * j] -= bf16_lo(x);
            w[2 * j + 1] -= bf16_hi(x);
          }
        }
        // The sums are those of the rounded weights, so a row that one
        // position rules gets that position's values.
        const u32x4a ones = {0x3f803f80u, 0x3f803f80u, 0x3f803f80u, 0x3f803f80u};
        l[r] = mfma(ones, p[r][e], l[r]);
      }
    }
#pragma unroll
    for (int part = 0; part < H::kParts; ++part) {
      float unit[8];
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        unit[4 * t] = unit_of<0>(raw.vs[t][part]);
        unit[4 * t + 1] = unit_of<1>(raw.vs[t][part]);
        unit[4 * t + 2] = unit_of<2>(raw.vs[t][part]);
        unit[4 * t + 3] = unit_of<3>(raw.vs[t][part]);
      }
#pragma unroll
      for (int b = 0; b < H::n(part); ++b) {  // two columns a byte
        uint32_t w[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) w[i] = two_columns(raw.v[i][H::reg0(part) + b / 4], unit[i], b % 4);
        uint32_t nan[8];
        if constexpr (SLOW) {
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const bool bad = (raw.vs[i / 4][part] >> (8 * (i % 4)) & 0xff) == kKvNan;
            w[i] = bad ? 0 : w[i];
            nan[i] = bad ? 0x3f803f80u : 0;
          }
        }
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          const uint32_t pick = half ? 0x07060302u : 0x05040100u;
          u32x4a v;
#pragma unroll
          for (int j = 0; j < 4; ++j) v[j] = __builtin_amdgcn_perm(w[2 * j + 1], w[2 * j], pick);
          const int d = H::base(part) / 16 + 2 * b + half;
#pragma unroll
          for (int r = 0; r < NQ; ++r) {
#pragma unroll
            for (int e = PT - 1; e >= 0; --e) o[r][d] = mfma(v, p[r][e], o[r][d]);
            if constexpr (SLOW) {
              u32x4a x, y;
#pragma unroll
              for (int j = 0; j < 4; ++j) {
                x[j] = __builtin_amdgcn_perm(nan[2 * j + 1], nan[2 * j], pick);
                y[j] = (seen[r] >> (2 * j) & 1 ? 0x3f80u : 0u) | (seen[r] >> (2 * j + 1) & 1 ? 0x3f800000u : 0u);
              }
              const f32x4 hits = mfma(x, y, zero);
#pragma unroll
              for (int i = 0; i < 4; ++i) o[r][d][i] = hits[i] > 0.0f ? __builtin_nanf("") : o[r][d][i];
            }
          }
        }
      }
    }
  }

  template <bool SLOW>
  __device__ __forceinline__ void run(const AttentionArgs& a, const WaveJob& job) {
    clear();
    if (job.begin >= job.end) return;
    KvRaw<D> raw[2];
    load_pages(a, job, job.begin);
    load(a, job, job.begin, 0, raw[0]);
    int n = 0;
    for (int64_t at = job.begin; at < job.end; at += job.stride) {
      const int64_t next = at + job.stride;
      const int32_t here = ids;
      const int n_next = (n + 1) & 31;
      if (next < job.end) {
        if (n_next == 0) load_pages(a, job, next);
        load(a, job, next, n_next, raw[1]);
      }
      const int32_t ahead = ids;
      ids = here;
      pass<SLOW>(a, job, at, n, raw[0]);
      ids = ahead;
      raw[0] = raw[1];
      n = n_next;
    }
  }

  // Whether a NaN of the cache (or of a query) has come into any row.
  __device__ __forceinline__ bool has_nan() const {
    bool bad = false;
#pragma unroll
    for (int r = 0; r < NQ; ++r) {
#pragma unroll
      for (int d = 0; d < D / 16; ++d) {
#pragma unroll
        for (int i = 0; i < 4; ++i) bad |= !(o[r][d][i] == o[r][d][i]);
      }
    }
    return __any(bad);
  }
};

// A workgroup's rows: sequence, first row, rows, tokens and positions.
struct RowTile {
  int64_t seq, row, rows, token, length, first;  // first: position of the sequence's first token in q
};

__device__ __forceinline__ bool row_tile(const AttentionArgs& a, int64_t tile, RowTile& t) {
  int64_t count;
  if (a.starts) {
    t.seq = kv_seq_of_tile(a.starts, a.seqs, a.tokens, a.group, a.tile_rows, tile);
    t.token = kv_clamp(a.starts[t.seq], 0, a.tokens);
    count = kv_clamp(a.starts[t.seq + 1], 0, a.tokens) - t.token;
    tile -= kv_first_tile(t.token, t.seq, a.group, a.tile_rows);
  } else {
    const int64_t per = (a.each * a.group + a.tile_rows - 1) / a.tile_rows;
    t.seq = tile / per;
    t.token = t.seq * a.each;
    count = a.each;
    tile -= t.seq * per;
  }
  t.row = tile * a.tile_rows;
  t.rows = count * a.group;
  if (tile < 0 || t.row >= t.rows) return false;
  const int64_t n = a.lengths[t.seq];
  t.length = kv_clamp(n, 0, a.cap);
  t.first = (n < 0 ? 0 : n) - count;
  return true;
}

template <int DT, int D, int NQ, int WT, int PT>
__global__ __launch_bounds__(kAttentionThreads) void attention_kernel(const AttentionArgs a) {
  using W = AttentionWave<DT, D, NQ, PT>;
  using T = typename OpElem<DT>::T;
  using H = HeadParts<D>;
  const int key_head = (int)(blockIdx.x % a.cache.heads);
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63, c = lane & 15, g = lane >> 4;
  RowTile tile;
  if (!row_tile(a, blockIdx.x / a.cache.heads, tile)) return;

  // Positions that any row of the workgroup sees, and this split's part of them.
  const int64_t last = min(tile.row + a.tile_rows, tile.rows) - 1;
  int64_t lo, hi, x;
  kv_span(tile.first + tile.row / a.group, tile.length, a.causal, a.window, &lo, &x);
  kv_span(tile.first + last / a.group, tile.length, a.causal, a.window, &x, &hi);
  const int64_t begin = lo / kKvStep * kKvStep + blockIdx.y * a.chunk;
  const int64_t end = min(begin + a.chunk, hi + 1);

  const int64_t row0 = tile.row + (WT == 1 ? wave * NQ * 16 : 0);  // of this wave
  W w;
  WaveJob job;
  {
    const int64_t head = (int64_t)key_head * a.cache.head, scale_head = (int64_t)key_head * a.cache.scale_head;
    job.k = a.cache.data[0] + head;
    job.v = a.cache.data[1] + head;
    job.ks = a.cache.scales[0] + scale_head;
    job.vs = a.cache.scales[1] + scale_head;
    job.pages = a.pages + tile.seq * a.page_stride;
    job.length = tile.length;
    job.stride = WT * kKvStep;
    const int64_t row1 = min(row0 + NQ * 16, tile.rows) - 1;
    int64_t wave_lo, wave_hi;
    kv_span(tile.first + row0 / a.group, tile.length, a.causal, a.window, &wave_lo, &job.full_hi);
    kv_span(tile.first + row1 / a.group, tile.length, a.causal, a.window, &job.full_lo, &wave_hi);
    job.begin = begin + (WT == 1 ? 0 : wave * kKvStep);
    job.end = min(end, wave_hi + 1);
    if (WT == 1) job.begin = max(job.begin, wave_lo / kKvStep * kKvStep);
    if (row0 >= tile.rows) job.end = job.begin;
  }
  // A row beyond the last one repeats it, and is not stored.
  int64_t token[NQ];
  int head[NQ];
#pragma unroll
  for (int r = 0; r < NQ; ++r) {
    const int64_t row = min(row0 + 16 * r + c, tile.rows - 1);
    token[r] = row / a.group;
    head[r] = key_head * a.group + (int)(row - token[r] * a.group);
    kv_span(tile.first + token[r], tile.length, a.causal, a.window, &w.lo[r], &w.hi[r]);
  }
  const auto q_row = [&](int r) {
    const int64_t at = a.starts ? (tile.token + token[r]) * a.q.s1 : tile.seq * a.q.s0 + token[r] * a.q.s1;
    return static_cast<const T*>(a.q.p) + at + head[r] * a.q.s2;
  };
#pragma unroll
  for (int r = 0; r < NQ; ++r) w.load_queries(r, q_row(r));
  w.template run<false>(a, job);
  if (w.has_nan()) w.template run<true>(a, job);

  // A row's place among all rows, for lse and for the parts of a split.
  const auto index_of = [&](int64_t t, int h) { return (tile.token + t) * a.heads + h; };
  const auto out_row = [&](int64_t t, int h) {
    const int64_t at = a.starts ? (tile.token + t) * a.out.s1 : tile.seq * a.out.s0 + t * a.out.s1;
    return static_cast<T*>(a.out.p) + at + h * a.out.s2;
  };
  const int64_t all = a.tokens * a.heads;
  constexpr float kLn2 = 0.69314718055994531f;
  const auto lse_of = [&](float ref, float sum) {
    return ref == -__builtin_inff() && sum == 0.0f ? ref : (ref + __builtin_amdgcn_logf(sum)) * kLn2;
  };

  if constexpr (WT == 1) {
#pragma unroll
    for (int r = 0; r < NQ; ++r) {
      if (row0 + 16 * r + c >= tile.rows) continue;
      const float sum = w.l[r][0];
      const int64_t at = index_of(token[r], head[r]);
      const float ref = w.m[r] == -__builtin_inff() && sum != 0.0f ? 0.0f : w.m[r];
      if (a.splits > 1) {
        if (g == 0) {
          float* ml = a.part_ml + 2 * (blockIdx.y * all + at);
          ml[0] = ref;
          ml[1] = sum;
        }
        if (sum == 0.0f) continue;
      } else if (a.lse && g == 0) {
        a.lse[at] = lse_of(ref, sum);
      }
      const float by = a.splits > 1 ? 1.0f : sum == 0.0f ? 0.0f : 1.0f / sum;
#pragma unroll
      for (int part = 0; part < H::kParts; ++part) {
        const int n = H::n(part), d0 = H::base(part) / 16;
        const int col = H::base(part) + 8 * n * g;
#pragma unroll
        for (int k = 0; k < n; ++k) {  // 8 columns each
          float f[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const int at_col = 8 * k + e, i = at_col / (2 * n), j = at_col % (2 * n);
            f[e] = w.o[r][d0 + j][i] * by;
          }
          if (a.splits > 1) {
            Packed<RINGSIM_FLOAT32, 8> y;
            y.set(f);
            y.store(a.part_out + (blockIdx.y * all + at) * D + col + 8 * k);
          } else {
            Packed<DT, 8> y;
            y.set(f);
            y.store(out_row(token[r], head[r]) + col + 8 * k);
          }
        }
      }
    }
  } else {
    // The waves' parts of the positions, joined in LDS in a fixed order.
    static_assert(NQ == 1, "waves that share rows have one tile of them");
    constexpr int kRow = D + 4;  // rows start 4 banks apart
    __shared__ float refs[WT][16], sums[WT][16];
    __shared__ float outs[WT][16][kRow];
    const float own = w.m[0] == -__builtin_inff() && w.l[0][0] != 0.0f ? 0.0f : w.m[0];  // NaN sums without a maximum
    if (g == 0) {
      refs[wave][c] = own;
      sums[wave][c] = w.l[0][0];
    }
    __syncthreads();
    float top = refs[0][c];
#pragma unroll
    for (int i = 1; i < WT; ++i) top = fmaxf(top, refs[i][c]);
    const float by = own == -__builtin_inff() ? 0.0f : own == top ? 1.0f : __builtin_amdgcn_exp2f(own - top);
#pragma unroll
    for (int part = 0; part < H::kParts; ++part) {
      const int n = H::n(part), d0 = H::base(part) / 16;
#pragma unroll
      for (int k = 0; k < 2 * n; ++k) {  // 4 columns each
        f32x4 f;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int at_col = 4 * k + e, i = at_col / (2 * n), j = at_col % (2 * n);
          f[e] = w.o[0][d0 + j][i] * by;
        }
        *reinterpret_cast<f32x4*>(&outs[wave][c][H::base(part) + 8 * n * g + 4 * k]) = f;
      }
    }
    __syncthreads();
    const int rows = (int)min((int64_t)16, tile.rows - tile.row);
    for (int k = threadIdx.x; k < rows * (D / 8); k += kAttentionThreads) {
      const int row = k / (D / 8), col = (k - row * (D / 8)) * 8;
      float best = refs[0][row], sum = 0.0f;
#pragma unroll
      for (int i = 1; i < WT; ++i) best = fmaxf(best, refs[i][row]);
#pragma unroll
      for (int i = 0; i < WT; ++i) {
        const float ref = refs[i][row];
        if (ref != -__builtin_inff()) sum += sums[i][row] * (ref == best ? 1.0f : __builtin_amdgcn_exp2f(ref - best));
      }
      float f[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        f[e] = outs[0][row][col + e];
#pragma unroll
        for (int i = 1; i < WT; ++i) f[e] += outs[i][row][col + e];
      }
      const int64_t t = (tile.row + row) / a.group;
      const int h = key_head * a.group + (int)(tile.row + row - t * a.group);
      const int64_t at = index_of(t, h);
      if (a.splits > 1) {
        if (col == 0) {
          float* ml = a.part_ml + 2 * (blockIdx.y * all + at);
          ml[0] = best;
          ml[1] = sum;
        }
        if (sum == 0.0f) continue;
        Packed<RINGSIM_FLOAT32, 8> y;
        y.set(f);
        y.store(a.part_out + (blockIdx.y * all + at) * D + col);
      } else {
        if (a.lse && col == 0) a.lse[at] = lse_of(best, sum);
        const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
#pragma unroll
        for (int e = 0; e < 8; ++e) f[e] *= inv;
        Packed<DT, 8> y;
        y.set(f);
        y.store(out_row(t, h) + col);
      }
    }
  }
}

template <int DT, int D, int NQ, int WT, int PT>
hipError_t launch_shape(const AttentionArgs& a, hipStream_t s) {
  const dim3 grid((unsigned)(a.tiles * a.cache.heads), (unsigned)a.splits);
  hipLaunchKernelGGL((attention_kernel<DT, D, NQ, WT, PT>), grid, dim3(kAttentionThreads), 0, s, a);
  return hipGetLastError();
}

// bf16 outputs: with few rows memory bounds, and weights in two parts cost
// nothing; with many the matrix units do.
template <int D>
hipError_t launch_head(const AttentionArgs& a, const AttentionPlan& plan, int dtype, hipStream_t s) {
  constexpr int kWide = 2;
  switch (dtype) {
    case RINGSIM_FLOAT32:
      return plan.wide ? launch_shape<RINGSIM_FLOAT32, D, 1, 1, 3>(a, s) : launch_shape<RINGSIM_FLOAT32, D, 1, 4, 3>(a, s);
    case RINGSIM_BFLOAT16:
      return plan.wide ? launch_shape<RINGSIM_BFLOAT16, D, kWide, 1, 1>(a, s)
                       : launch_shape<RINGSIM_BFLOAT16, D, 1, 4, 2>(a, s);
    case RINGSIM_FLOAT16:
      return plan.wide ? launch_shape<RINGSIM_FLOAT16, D, 1, 1, 2>(a, s) : launch_shape<RINGSIM_FLOAT16, D, 1, 4, 2>(a, s);
    default: return hipErrorInvalidValue;
  }
}

}  // namespace ringsim
