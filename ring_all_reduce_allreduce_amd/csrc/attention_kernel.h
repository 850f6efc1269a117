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
// weights never change lanes.
//
// Keys go into the matrix unit as they lie in memory, 4-bit codes with an
// exponent for every 32 columns, which is what its scaled instruction takes: a
// lane's operand is one block. The other operand may be in 8 bits, so queries
// are split once into parts of 8 bits with exponents of their own. Values are
// needed by columns: a lane reads a few columns of each of its eight positions,
// the conversion instruction turns two codes and an exponent into two bf16
// (which hold every value of the cache), and halves are swapped between
// positions. With few rows nothing passes through LDS.
//
// What bounds it: with few rows memory, 17/32 bytes a column of keys and of
// values. 64 sequences of up to 16384 positions of 8 heads of 128, 636 MB of
// cache, take 130 us (4.9 TB/s); their loads alone take 117 us, their arithmetic
// alone 87. With many rows staging and the vector unit beside the matrix one: 3
// prompts of 2048 tokens of 32 heads behind up to 4000 positions take 283 us (844
// TFLOP/s), about a third of it less where nothing has to be loaded, converted and
// put into LDS (201 us of then 299) and 42 us less without a softmax;
// of the 1500 clocks of a pass of 32 positions the matrix unit works in 544 and the
// vector unit, with exponentials and conversions, in 630 to 730, and with two
// waves a SIMD the two overlap in part only.
#pragma once

#include <type_traits>

#include "attention_rows.h"

namespace ringsim {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

typedef int i32x8 __attribute__((ext_vector_type(8)));

constexpr int kAttentionWaves = 4;
constexpr int kAttentionThreads = 64 * kAttentionWaves;

// How far (as a power of two) weights may grow before a row's reference
// exponent follows its maximum. Sums and products in fp32 lose nothing by it,
// and most passes need no maximum over lanes and no rescaling. (Three prompts of
// 2048 tokens of 32 heads of 128: 163 us, without slack 179.)
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

// A head's columns in the first product: a matrix instruction takes 128 of
// them. Of 4-bit operands group g of 16 lanes holds block g, columns 32 g to 32
// g + 31; of 8-bit ones columns 16 g + j and 64 + 16 g + j, j below 16; a lane's
// exponent is that of block g of either. Heads of 64 bring two parts of the
// queries into one instruction; where a head ends, the last block is repeated
// against zeros.
template <int D, int TERMS>
struct HeadBlocks {
  static constexpr int kBlocks = D / 32;
  static constexpr int kSets = (kBlocks + 3) / 4;  // of four blocks
  static constexpr bool kPaired = kBlocks == 2;
  static constexpr int kTurns = kPaired ? (TERMS + 1) / 2 : TERMS;  // instructions a set
  static constexpr int kHalves = kPaired ? 1 : 2;  // of 16 columns that a lane holds of a set
  static __device__ __forceinline__ int block(int set, int g) {
    return kPaired ? g & 1 : min(4 * set + g, kBlocks - 1);
  }
  static __device__ __forceinline__ int column(int set, int half, int g) { return 128 * set + 64 * half + 16 * g; }
};

// 32 positions of the cache as they lie in memory.
template <int D>
struct KvRaw {
  using H = HeadParts<D>;
  static constexpr int kSets = (D / 32 + 3) / 4;
  u32x4 k[2][kSets];
  uint32_t ks[2][kSets];
  uint32_t v[8][H::kRegs];
  uint32_t vs[2][H::kParts];
  bool there[2];           // whether the tiles have a page
};

// A place in device memory that is the same for all lanes, in scalar
// registers: a load adds a lane's own 32 bits to it by itself. Without the
// barriers the compiler would add the lane's part first, or widen it, once for
// all passes, and then spend an addition and two registers on every load.
typedef const __attribute__((address_space(1))) uint8_t* GlobalBytes;
__device__ __forceinline__ GlobalBytes uniform(const uint8_t* p) {
  asm("" : "+s"(p));
  return (GlobalBytes)p;
}

template <int N>
__device__ __forceinline__ void load_bytes(uint32_t* w, GlobalBytes p, uint32_t at) {
  typedef const __attribute__((address_space(1))) uint16_t* P16;
  typedef const __attribute__((address_space(1))) uint32_t* P32;
  typedef const __attribute__((address_space(1))) u32x2* P64;
  typedef const __attribute__((address_space(1))) u32x4* P128;
  asm("" : "+v"(at));
  if constexpr (N == 1) {
    w[0] = p[at];
  } else if constexpr (N == 2) {
    w[0] = *(P16)(p + at);
  } else if constexpr (N == 4) {
    w[0] = *(P32)(p + at);
  } else if constexpr (N == 8) {
    const u32x2 x = *(P64)(p + at);
    w[0] = x[0];
    w[1] = x[1];
  } else {
    static_assert(N == 16, "bytes");
    const u32x4 x = *(P128)(p + at);
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = x[i];
  }
}

// One or two bytes at each of two places into the halves of a register.
template <int N>
__device__ __forceinline__ void load_two(uint32_t* w, GlobalBytes p, GlobalBytes q, uint32_t at) {
  typedef const __attribute__((address_space(1))) uint16_t* P16;
  typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));
  static_assert(N == 1 || N == 2, "bytes");
  asm("" : "+v"(at));
  u16x2 x;
  x[0] = N == 1 ? (uint16_t)p[at] : *(P16)(p + at);
  x[1] = N == 1 ? (uint16_t)q[at] : *(P16)(q + at);
  *w = __builtin_bit_cast(uint32_t, x);
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

// A value's exponents of four positions.
__device__ __forceinline__ void value_units(uint32_t w, float* unit) {
  unit[0] = unit_of<0>(w);
  unit[1] = unit_of<1>(w);
  unit[2] = unit_of<2>(w);
  unit[3] = unit_of<3>(w);
}

// Of eight positions' pairs of columns the first or the second column.
__device__ __forceinline__ u32x4 one_column(const uint32_t (&w)[8], int half) {
  u32x4 v;
#pragma unroll
  for (int j = 0; j < 4; ++j) v[j] = __builtin_amdgcn_perm(w[2 * j + 1], w[2 * j], half ? 0x07060302u : 0x05040100u);
  return v;
}

// The largest of three, NaN if one is: one instruction, which fmaxf, having to
// look at the kinds of NaN, is not.
__device__ __forceinline__ float larger(float x, float y, float z) {
  return __builtin_elementwise_maximum(__builtin_elementwise_maximum(x, y), z);
}

__device__ __forceinline__ f32x4 mfma(const u32x4& x, const u32x4& y, f32x4 acc) {
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

// Codes of 4 bits with exponents `ks` times 8-bit ones with exponents `qs`.
__device__ __forceinline__ f32x4 mfma_scaled(const u32x4& k, uint32_t ks, const i32x8& q, uint32_t qs, f32x4 acc) {
  // 4-bit operands are the first half.
  const i32x8 x = __builtin_bit_cast(i32x8, __builtin_shufflevector(k, k, 0, 1, 2, 3, -1, -1, -1, -1));
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(x, q, acc, 4, 0, 0, (int)ks, 0, (int)qs);
}

// Parts that queries of a type are split into. With a row's largest magnitude
// in [128, 256) a part keeps 4 bits, and each remainder is at most 8, so the
// next part takes it times 32: 2 parts hold the 8 bits of bf16, 3 the 11 of
// fp16, and what is left after 5 is a rounding of fp32. Columns that are small
// beside their row's largest keep their place to 2^-22, 2^-27 and 2^-37 of it
// (half the smallest step of the last part).
//
// The matrix unit, however, adds products of neighbouring columns in 14 bits of
// the largest of them (measured: beside 1, 2^-13 counts and 2^-14 does not). So in
// the FINE split a column below kTermLeast waits for the next part, but in the
// last two, and bf16 and fp16 have one part more, so that those that waited still
// have all of their bits: products of what is above, whose last bit is 2^-2 or
// more, times codes, whose last bit is 1/2, reach down from 256 * 6 to 2^-3 and
// lose nothing; the last two parts lose 2^-13 of what is 32 times smaller for
// each part before. Scores of 192 columns in fp32 are 8e-8 of their size off, 5e-6
// without. With few rows memory bounds, and the part costs nothing; with many
// bf16 and fp16 stay with the coarse split, whose errors are below those of
// weights and outputs in 16 bits, but where lse, which is fp32, is wanted over
// few positions.
constexpr int query_terms(int dtype, bool fine) {
  return dtype == RINGSIM_FLOAT32 ? 5 : (dtype == RINGSIM_FLOAT16 ? 3 : 2) + (fine ? 1 : 0);
}
constexpr int kTermBits = 5;
constexpr float kTermStep = 1 << kTermBits;
constexpr int kTermTop = 7;  // exponent of a row's largest magnitude in its first part
constexpr float kTermLeast = 2.0f;

// The rows of a wave: queries, sums, and the mathematics of a pass of 32
// positions. DT, D: type of queries and columns of a head. NQ: tiles of 16
// rows. PT: bf16 parts of a weight. EXACT: sums of the weights before their
// rounding too, which lse takes where there are one or two parts: rounded, they
// would be off by 2^-8 or 2^-17, and not by fp32's last bits. FINE: how queries
// are split.
template <int DT, int D, int NQ, int PT, bool EXACT, bool FINE>
struct RowSums {
  static constexpr int kTerms = query_terms(DT, FINE);
  using H = HeadParts<D>;
  using B = HeadBlocks<D, kTerms>;

  i32x8 q[NQ][B::kSets][B::kTurns];
  uint32_t qs[NQ][B::kSets][B::kTurns];
  f32x4 o[NQ][D / 16];
  f32x4 l[NQ];
  float exact[NQ];         // EXACT: the lane's own part
  float m[NQ];             // reference exponent, minus infinity until a position is seen
  int lo[NQ], hi[NQ];      // positions that this lane's row sees

  __device__ __forceinline__ void clear() {
    const f32x4 zero = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int r = 0; r < NQ; ++r) {
      m[r] = -__builtin_inff();
      exact[r] = 0.0f;
      l[r] = zero;
#pragma unroll
      for (int d = 0; d < D / 16; ++d) o[r][d] = zero;
    }
  }

  // A lane's columns of its row in parts of 8 bits. A NaN or an infinity makes
  // the row NaN.
  __device__ __forceinline__ void load_queries(int r, const typename OpElem<DT>::T* row) {
    const int g = (threadIdx.x & 63) >> 4;
    float x[B::kSets][B::kHalves][16];
    uint32_t top = 0;
#pragma unroll
    for (int set = 0; set < B::kSets; ++set) {
#pragma unroll
      for (int half = 0; half < B::kHalves; ++half) {
        const int col = B::column(set, half, g);
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          Packed<DT, 8> p;
          p.load(row + (col < D ? col : 0) + 8 * k);
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const float v = col < D ? p.get(i) : 0.0f;
            x[set][half][8 * k + i] = v;
            top = MaxBits::of(top, __float_as_uint(v) & 0x7fffffffu);
          }
        }
      }
    }
    const auto s = __builtin_amdgcn_permlane16_swap(top, top, false, false);
    top = MaxBits::of(s[0], s[1]);
    const auto u = __builtin_amdgcn_permlane32_swap(top, top, false, false);
    top = MaxBits::of(u[0], u[1]);  // of the row
    const bool finite = top < 0x7f800000u;
    // Exponent of the first part; the last one's has to stay above 2^-127.
    int e = (int)(top >> 23) - 127 - kTermTop;
    e = max(e, kQueryExponent + kTermBits * kTerms - 126);
    // -93 to 120, so that 2^-e is a normal number.
    const float up = __builtin_ldexpf(1.0f, -e);
#pragma unroll
    for (int set = 0; set < B::kSets; ++set) {
#pragma unroll
      for (int term = 0; term < kTerms; ++term) {
        const int turn = B::kPaired ? term / 2 : term;
#pragma unroll
        for (int half = 0; half < B::kHalves; ++half) {
          float* v = x[set][half];
#pragma unroll
          for (int w = 0; w < 4; ++w) {
            if (term == 0) {
#pragma unroll
              for (int i = 0; i < 4; ++i) v[4 * w + i] *= up;
            }
            const auto now = [&](int i) {
              return FINE && term + 2 < kTerms && __builtin_fabsf(v[4 * w + i]) < kTermLeast ? 0.0f : v[4 * w + i];
            };
            int c = 0;
            c = __builtin_amdgcn_cvt_pk_fp8_f32(now(0), now(1), c, false);
            c = __builtin_amdgcn_cvt_pk_fp8_f32(now(2), now(3), c, true);
            v[4 * w] = (v[4 * w] - __builtin_amdgcn_cvt_f32_fp8(c, 0)) * kTermStep;
            v[4 * w + 1] = (v[4 * w + 1] - __builtin_amdgcn_cvt_f32_fp8(c, 1)) * kTermStep;
            v[4 * w + 2] = (v[4 * w + 2] - __builtin_amdgcn_cvt_f32_fp8(c, 2)) * kTermStep;
            v[4 * w + 3] = (v[4 * w + 3] - __builtin_amdgcn_cvt_f32_fp8(c, 3)) * kTermStep;
            q[r][set][turn][4 * (B::kPaired ? term & 1 : half) + w] = finite ? c : 0x7f7f7f7f;  // NaN
          }
        }
        const uint32_t scale = (uint32_t)(e - kTermBits * term - kQueryExponent + 127);
        qs[r][set][turn] = B::kPaired && term % 2 == 1 && g < 2 ? qs[r][set][turn] : scale;
      }
      if (B::kPaired && kTerms % 2 == 1) {
#pragma unroll
        for (int w = 4; w < 8; ++w) q[r][set][B::kTurns - 1][w] = 0;
      }
    }
  }

  // Products with the keys of two tiles; key(t, set, k, ks) gives a lane's block.
  template <typename KEY>
  __device__ __forceinline__ void scores(f32x4 (&s)[NQ][2], const KEY& key) const {
#pragma unroll
    for (int t = 0; t < 2; ++t) {
#pragma unroll
      for (int r = 0; r < NQ; ++r) s[r][t] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int set = 0; set < B::kSets; ++set) {
        u32x4 k;
        uint32_t ks;
        key(t, set, k, ks);
#pragma unroll
        for (int turn = B::kTurns - 1; turn >= 0; --turn) {
#pragma unroll
          for (int r = 0; r < NQ; ++r) s[r][t] = mfma_scaled(k, ks, q[r][set][turn], qs[r][set][turn], s[r][t]);
        }
      }
    }
  }

  // Takes out what a row does not see. seen: a bit a position.
  __device__ __forceinline__ void mask(f32x4 (&s)[NQ][2], int at, bool there0, bool there1,
                                       uint32_t (&seen)[NQ]) const {
    const int g = (threadIdx.x & 63) >> 4;
#pragma unroll
    for (int r = 0; r < NQ; ++r) {
      seen[r] = 0;
#pragma unroll
      for (int t = 0; t < 2; ++t) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int j = at + kKvTile * t + 4 * g + i;
          const bool on = j >= lo[r] && j <= hi[r] && (t ? there1 : there0);
          s[r][t][i] = on ? s[r][t][i] : -__builtin_inff();
          seen[r] |= (uint32_t)on << (4 * t + i);
        }
      }
    }
  }

  // Lets the rows' references follow their maxima where one has grown past the
  // slack. One branch for all tiles.
  __device__ __forceinline__ void follow(const AttentionArgs& a, const f32x4 (&s)[NQ][2]) {
    float top[NQ];
    bool above = false;
#pragma unroll
    for (int r = 0; r < NQ; ++r) {
      // A NaN stays one, so the row keeps its reference.
      top[r] = a.scale_log2 * larger(larger(larger(s[r][0][0], s[r][0][1], s[r][0][2]), s[r][0][3], s[r][1][0]),
                                     s[r][1][1], larger(s[r][1][2], s[r][1][3], s[r][1][3]));
      above |= top[r] > m[r] + kSlack;
    }
    if (!__any(above)) return;
#pragma unroll
    for (int r = 0; r < NQ; ++r) {
      const float next = fmaxf(m[r], groups_max(top[r]));
      // exp2(-inf) = 0 on a row's first positions; a row without any keeps its zeros.
      const float by = next == m[r] ? 1.0f : __builtin_amdgcn_exp2f(m[r] - next);
      m[r] = next;
      exact[r] *= by;
      l[r] *= by;
#pragma unroll
      for (int d = 0; d < D / 16; ++d) o[r][d] *= by;
    }
  }

  // Weights of the lane's eight positions in PT parts, and their sums.
  __device__ __forceinline__ void weights(const AttentionArgs& a, const f32x4 (&s)[NQ][2], u32x4 (&p)[NQ][PT]) {
#pragma unroll
    for (int r = 0; r < NQ; ++r) {
      const float ref = m[r] == -__builtin_inff() ? 0.0f : m[r];
      float w[8];
#pragma unroll
      for (int i = 0; i < 8; ++i)
        w[i] = __builtin_amdgcn_exp2f(__builtin_fmaf(s[r][i / 4][i % 4], a.scale_log2, -ref));
      if (EXACT) exact[r] += ((w[0] + w[1]) + (w[2] + w[3])) + ((w[4] + w[5]) + (w[6] + w[7]));
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
        const u32x4 ones = {0x3f803f80u, 0x3f803f80u, 0x3f803f80u, 0x3f803f80u};
        l[r] = mfma(ones, p[r][e], l[r]);
      }
    }
  }

  // Adds 16 columns of the values, positions as the lane's weights have them.
  __device__ __forceinline__ void add_values(int d, const u32x4& v, const u32x4 (&p)[NQ][PT]) {
#pragma unroll
    for (int r = 0; r < NQ; ++r) {
#pragma unroll
      for (int e = PT - 1; e >= 0; --e) o[r][d] = mfma(v, p[r][e], o[r][d]);
    }
  }

  // A row's sum of weights as lse takes it.
  __device__ __forceinline__ float exact_sum(int r) const {
    if constexpr (!EXACT) return l[r][0];
    float v = exact[r] + __shfl_xor(exact[r], 16);
    return v + __shfl_xor(v, 32);
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

// What a wave has to do, the same for all of its lanes.
struct WaveJob {
  const uint8_t* k;        // of the key head: keys, values and their scales of page 0
  const uint8_t* v;
  const uint8_t* ks;
  const uint8_t* vs;
  const int32_t* pages;    // of the sequence
  int begin, end;          // positions, begin a multiple of kKvStep; `end` past the last one wanted
  int stride;              // from one pass of this wave to the next
  int full_lo, full_hi;    // positions that every row of the wave sees
  int length;              // positions of the sequence
};

// Where the 64 tiles of the next passes lie in memory, one a lane: the products
// with the strides are done once for all of them in the vector unit, and a
// pass reads its tiles' places out of the lanes. (In scalar registers they took
// up to half of a pass's instructions.) The page numbers are asked for some
// passes before they are needed.
struct TileWindow {
  uint64_t there;          // the tiles that have a page, a bit each
  uint32_t data[2], scale[2];
  int32_t asked;

  __device__ __forceinline__ void ask(const AttentionArgs& a, const WaveJob& job, int64_t tile) {
    int64_t place;
    kv_place_of_tile(tile, job.length, a.cache.page_shift, a.max_pages, &place);
    asked = job.pages[place];
  }
  // `tile` as it was asked for. Tiles without a page are read from page 0.
  __device__ __forceinline__ void take(const AttentionArgs& a, const WaveJob& job, int64_t tile) {
    int64_t place;
    const bool on = kv_place_of_tile(tile, job.length, a.cache.page_shift, a.max_pages, &place) &&
                    kv_is_page(asked, a.cache.pages);
    there = __ballot(on);
    const int64_t page = on ? asked : 0;
    const int off = (int)(tile * kKvTile) & ((1 << a.cache.page_shift) - 1);
    const uint64_t d = (uint64_t)(page * a.cache.page + (int64_t)off * (a.cache.dim / 2));
    const uint64_t s = (uint64_t)(page * a.cache.scale_page + off);
    data[0] = (uint32_t)d;
    data[1] = (uint32_t)(d >> 32);
    scale[0] = (uint32_t)s;
    scale[1] = (uint32_t)(s >> 32);
  }
  static __device__ __forceinline__ int64_t of(const uint32_t (&x)[2], int i) {
    return (int64_t)((uint64_t)(uint32_t)__builtin_amdgcn_readlane(x[1], i) << 32 |
                     (uint32_t)__builtin_amdgcn_readlane(x[0], i));
  }
  __device__ __forceinline__ int64_t data_of(int i) const { return of(data, i); }
  __device__ __forceinline__ int64_t scale_of(int i) const { return of(scale, i); }
};

// A wave on its own: keys and values go from memory to its registers. AHEAD:
// passes whose loads are under way. ONE: all rows of the wave belong to one
// token, so a position is seen by all of them or none, and what the cache holds
// where none sees is taken as ones. Else what is not finite in a position has to
// reach the rows that see it and no others, for which there is the slow way.
template <int DT, int D, int NQ, int PT, int AHEAD, bool ONE>
struct AttentionWave : RowSums<DT, D, NQ, PT, (PT < 3), true> {
  using R = RowSums<DT, D, NQ, PT, (PT < 3), true>;
  using typename R::B;
  using typename R::H;
  using R::o;

  TileWindow window;       // of the next 32 passes

  // A lane's tile of pass `pass` and the 31 behind it.
  __device__ __forceinline__ int64_t tile_of(const WaveJob& job, int pass) const {
    const int lane = threadIdx.x & 63;
    return ((int64_t)job.begin + (int64_t)(pass + (lane >> 1)) * job.stride) / kKvTile + (lane & 1);
  }

  // Pass `n` of the window's 32.
  __device__ __forceinline__ void load(const AttentionArgs& a, const WaveJob& job, int n, KvRaw<D>& raw) {
    const int lane = threadIdx.x & 63, c = lane & 15, g = lane >> 4;
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      // Addresses: a place that is the same for all lanes, and a lane's own 32 bits.
      const int64_t data = window.data_of(2 * n + t), scale = window.scale_of(2 * n + t);
      raw.there[t] = window.there >> (2 * n + t) & 1;
      const GlobalBytes pk = uniform(job.k + data), pv = uniform(job.v + data);
      const GlobalBytes pks = uniform(job.ks + scale), pvs = uniform(job.vs + scale);
#pragma unroll
      for (int set = 0; set < KvRaw<D>::kSets; ++set) {
        const uint32_t block = B::block(set, g);
        uint32_t k[4];
        load_bytes<16>(k, pk, (uint32_t)c * (D / 2) + block * 16);
        raw.k[t][set] = u32x4{k[0], k[1], k[2], k[3]};
        load_bytes<1>(&raw.ks[t][set], pks, (block << a.cache.page_shift) + (uint32_t)c);
      }
#pragma unroll
      for (int p = 0; p < H::kParts; ++p) {
        constexpr int kRow = D / 2;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint32_t from = (uint32_t)(4 * g * kRow + H::base(p) / 2 + c * H::n(p));
          uint32_t* to = raw.v[4 * t + i] + H::reg0(p);
          if (H::n(p) == 1) load_bytes<1>(to, pv + i * kRow, from);
          if (H::n(p) == 2) load_bytes<2>(to, pv + i * kRow, from);
          if (H::n(p) == 4) load_bytes<4>(to, pv + i * kRow, from);
          if (H::n(p) == 8) load_bytes<8>(to, pv + i * kRow, from);
        }
        const uint32_t b = H::base(p) / 32 + c * H::n(p) / 16;
        load_bytes<4>(&raw.vs[t][p], pvs, (b << a.cache.page_shift) + (uint32_t)(4 * g));
      }
    }
  }

  // One pass over the 32 positions from `at` on. SLOW: a position's values that
  // are not finite make NaN of the rows that see it and no others, which a weight
  // of 0 times them would not do.
  template <bool SLOW>
  __device__ __forceinline__ void pass(const AttentionArgs& a, const WaveJob& job, int at, const KvRaw<D>& raw) {
    const f32x4 zero = {0.0f, 0.0f, 0.0f, 0.0f};
    f32x4 s[NQ][2];
    R::scores(s, [&](int t, int set, u32x4& k, uint32_t& ks) {
      k = raw.k[t][set];
      ks = raw.ks[t][set];
    });
    uint32_t seen[NQ];
    bool masked = SLOW;
    if (SLOW || !raw.there[0] || !raw.there[1] || at < job.full_lo || at + kKvStep - 1 > job.full_hi) {
      masked = true;
      R::mask(s, at, raw.there[0], raw.there[1], seen);
    }
    u32x4 p[NQ][PT];
    R::follow(a, s);
    R::weights(a, s, p);
#pragma unroll
    for (int part = 0; part < H::kParts; ++part) {
      float unit[8];
#pragma unroll
      for (int t = 0; t < 2; ++t) value_units(raw.vs[t][part], unit + 4 * t);
      if constexpr (ONE) {
        // The lane's positions are those of its weights, and all rows see the same.
        if (masked) {
#pragma unroll
          for (int i = 0; i < 8; ++i) unit[i] = seen[0] >> i & 1 ? unit[i] : 1.0f;
        }
      }
#pragma unroll
      for (int b = 0; b < H::n(part); ++b) {  // two columns a byte
        uint32_t w[8], nan[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) w[i] = two_columns(raw.v[i][H::reg0(part) + b / 4], unit[i], b % 4);
        if constexpr (SLOW) {
          // NaN blocks, and infinities, which exponents of 253 and 254 make of the larger codes.
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const uint32_t bad = ((w[i] & 0x7f80u) == 0x7f80u ? 0xffffu : 0) |
                                 ((w[i] & 0x7f800000u) == 0x7f800000u ? 0xffff0000u : 0);
            w[i] &= ~bad;
            nan[i] = bad & 0x3f803f80u;
          }
        }
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          const int d = H::base(part) / 16 + 2 * b + half;
          R::add_values(d, one_column(w, half), p);
          if constexpr (SLOW) {
            const u32x4 x = one_column(nan, half);
#pragma unroll
            for (int r = 0; r < NQ; ++r) {
              u32x4 y;
#pragma unroll
              for (int j = 0; j < 4; ++j)
                y[j] = (seen[r] >> (2 * j) & 1 ? 0x3f80u : 0u) | (seen[r] >> (2 * j + 1) & 1 ? 0x3f800000u : 0u);
              const f32x4 hits = mfma(x, y, zero);
#pragma unroll
              for (int i = 0; i < 4; ++i) o[r][d][i] = hits[i] > 0.0f ? __builtin_nanf("") : o[r][d][i];
            }
          }
        }
      }
    }
  }

  // `prepare` is called with the first loads under way.
  template <bool SLOW, typename PREPARE>
  __device__ __forceinline__ void run(const AttentionArgs& a, const WaveJob& job, const PREPARE& prepare) {
    R::clear();
    if (job.begin >= job.end) return;
    // Buffers in turn, loaded AHEAD passes before they are worked on. No load
    // stands under a condition: behind one, the compiler would wait for all that
    // are under way and not for the oldest buffer's alone. So after the last
    // pass's loads they are repeated, out of the cache.
    KvRaw<D> raw[AHEAD + 1];
    const int passes = (job.end - 1 - job.begin) / job.stride + 1;
    int next = 0;  // pass to be loaded
    window.ask(a, job, tile_of(job, 0));
    const auto load_next = [&](KvRaw<D>& to) {
      if ((next & 31) == 0) window.take(a, job, tile_of(job, next));
      load(a, job, next & 31, to);
      if ((next & 31) == 16) window.ask(a, job, tile_of(job, (next | 31) + 1));
      if (next < passes - 1) ++next;
    };
#pragma unroll
    for (int i = 0; i < AHEAD; ++i) load_next(raw[i]);
    prepare();
    for (int at = job.begin;;) {
#pragma unroll
      for (int i = 0; i <= AHEAD; ++i) {
        load_next(raw[(i + AHEAD) % (AHEAD + 1)]);
        pass<SLOW>(a, job, at, raw[i]);
        at += job.stride;
        if (at >= job.end) return;
      }
    }
  }
};

// The waves of a workgroup together, each with rows of its own. Per stage of 64
// positions each wave brings a quarter of the keys and values: keys as they
// lie in memory, values already as operands of the second product, so that the
// conversion is done once for all rows of the workgroup. Two buffers, one
// barrier a stage, the loads of two stages under way.
constexpr int kStage = 64;
constexpr int kStageTiles = kStage / kKvTile;

template <int D>
struct WideBuffers {
  static constexpr int kSets = (D / 32 + 3) / 4, kBuffers = 2;
  u32x4 k[kBuffers][kStageTiles][kSets][64];
  u32x4 v[kBuffers][2][D / 16][64];
  uint32_t ks[kBuffers][kStageTiles][kSets][64];
};

template <int DT, int D, int NQ, int PT, bool EXACT, bool FINE>
struct WideWave : RowSums<DT, D, NQ, PT, EXACT, FINE> {
  using R = RowSums<DT, D, NQ, PT, EXACT, FINE>;
  using typename R::B;
  using typename R::H;
  static constexpr int kSets = B::kSets;

  TileWindow window;       // of the next 16 stages

  // What a wave brings: the keys of tile `wave`, and of the values of 32
  // positions (wave / 2 of two) one half of the bytes, wave % 2: half of each
  // lane's, or where a head has two parts, one part.
  static constexpr int bytes(int half) { return H::kParts == 1 ? H::n(0) / 2 : H::n(half); }
  static constexpr int kWords = bytes(0) == 4 || bytes(1) == 4 ? 8 : 4;
  struct Raw {
    u32x4 k[kSets];
    uint32_t ks[kSets];
    uint32_t v[kWords];    // of 8 positions: a register each, or two in one
    uint32_t vs[2];
  };

  // Values of tile t of the two; `half` is HALF, or where a lane has half of its bytes a number of the wave.
  template <int HALF>
  __device__ __forceinline__ void load_values(const AttentionArgs& a, const uint8_t* v, const uint8_t* vs, int half,
                                              Raw& raw, int t) {
    constexpr int kPart = H::kParts == 1 ? 0 : HALF, kRow = D / 2, kBytes = bytes(HALF);
    const int lane = threadIdx.x & 63, c = lane & 15, g = lane >> 4;
    const uint32_t from =
        (uint32_t)(4 * g * kRow + H::base(kPart) / 2 + c * H::n(kPart) + (H::kParts == 1 ? half * kBytes : 0));
    const GlobalBytes pv = uniform(v), pvs = uniform(vs);
    if constexpr (kBytes == 4) {
#pragma unroll
      for (int i = 0; i < 4; ++i) load_bytes<4>(&raw.v[4 * t + i], pv + i * kRow, from);
    } else {
#pragma unroll
      for (int i = 0; i < 2; ++i) load_two<kBytes>(&raw.v[2 * t + i], pv + 2 * i * kRow, pv + (2 * i + 1) * kRow, from);
    }
    const uint32_t b = H::base(kPart) / 32 + c * H::n(kPart) / 16;
    load_bytes<4>(&raw.vs[t], pvs, (b << a.cache.page_shift) + (uint32_t)(4 * g));
  }

  // The stage whose first tile is number `first` of the window. Returns which of
  // its tiles have a page, a bit each.
  __device__ __forceinline__ uint32_t load_stage(const AttentionArgs& a, const WaveJob& job, int wave, int first,
                                                 Raw& raw) {
    const int lane = threadIdx.x & 63, c = lane & 15, g = lane >> 4;
    const GlobalBytes pk = uniform(job.k + window.data_of(first + wave));
    const GlobalBytes pks = uniform(job.ks + window.scale_of(first + wave));
#pragma unroll
    for (int set = 0; set < kSets; ++set) {
      const uint32_t block = B::block(set, g);
      uint32_t k[4];
      load_bytes<16>(k, pk, (uint32_t)c * (D / 2) + block * 16);
      raw.k[set] = u32x4{k[0], k[1], k[2], k[3]};
      load_bytes<1>(&raw.ks[set], pks, (block << a.cache.page_shift) + (uint32_t)c);
    }
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      const uint8_t* v = job.v + window.data_of(first + (wave & 2) + t);
      const uint8_t* vs = job.vs + window.scale_of(first + (wave & 2) + t);
      if (H::kParts == 2 && (wave & 1))
        load_values<1>(a, v, vs, 1, raw, t);
      else
        load_values<0>(a, v, vs, wave & 1, raw, t);
    }
    return (uint32_t)(window.there >> first) & ((1 << kStageTiles) - 1);
  }

  template <int HALF>
  __device__ __forceinline__ void put_values(const Raw& raw, int half, u32x4 (&v)[D / 16][64]) {
    constexpr int kPart = H::kParts == 1 ? 0 : HALF, kBytes = bytes(HALF);
    const int first = H::base(kPart) / 16 + (H::kParts == 1 ? 2 * kBytes * half : 0);
    const int lane = threadIdx.x & 63;
    float unit[8];
    value_units(raw.vs[0], unit);
    value_units(raw.vs[1], unit + 4);
#pragma unroll
    for (int b = 0; b < kBytes; ++b) {
      uint32_t w[8];
#pragma unroll
      for (int i = 0; i < 8; ++i)
        w[i] = kBytes == 4 ? two_columns(raw.v[i], unit[i], b) : two_columns(raw.v[i / 2], unit[i], 2 * (i % 2) + b);
#pragma unroll
      for (int i = 0; i < 2; ++i) v[first + 2 * b + i][lane] = one_column(w, i);
    }
  }

  __device__ __forceinline__ void put(WideBuffers<D>& lds, int buffer, int wave, const Raw& raw) {
    const int lane = threadIdx.x & 63;
#pragma unroll
    for (int set = 0; set < kSets; ++set) {
      lds.k[buffer][wave][set][lane] = raw.k[set];
      lds.ks[buffer][wave][set][lane] = raw.ks[set];
    }
    if (H::kParts == 2 && (wave & 1))
      put_values<1>(raw, 1, lds.v[buffer][wave >> 1]);
    else
      put_values<0>(raw, wave & 1, lds.v[buffer][wave >> 1]);
  }

  // One pass over the 32 positions from `at` on, half `sub` of a stage; there: which of its two tiles have a page.
  __device__ __forceinline__ void pass(const AttentionArgs& a, const WaveJob& job, int at, const WideBuffers<D>& lds,
                                       int buffer, int sub, uint32_t there) {
    const int lane = threadIdx.x & 63;
    // Operands are asked for together: left to itself the compiler reads
    // each one where it is used, and waits for it. The second half of the
    // values follows while the first one is multiplied.
    constexpr int kHalf = D / 32;
    u32x4 k[2][kSets], v[kHalf];
    uint32_t ks[2][kSets];
#pragma unroll
    for (int t = 0; t < 2; ++t) {
#pragma unroll
      for (int set = 0; set < kSets; ++set) {
        k[t][set] = lds.k[buffer][2 * sub + t][set][lane];
        ks[t][set] = lds.ks[buffer][2 * sub + t][set][lane];
      }
    }
#pragma unroll
    for (int d = 0; d < kHalf; ++d) v[d] = lds.v[buffer][sub][d][lane];
    __builtin_amdgcn_sched_barrier(0);
    f32x4 s[NQ][2];
    R::scores(s, [&](int t, int set, u32x4& x, uint32_t& xs) {
      x = k[t][set];
      xs = ks[t][set];
    });
    if (there != 3 || at < job.full_lo || at + kKvStep - 1 > job.full_hi) {
      uint32_t seen[NQ];
      R::mask(s, at, there & 1, there & 2, seen);
    }
    R::follow(a, s);
    u32x4 p[NQ][PT];
    R::weights(a, s, p);
    u32x4 more[kHalf];
#pragma unroll
    for (int d = 0; d < kHalf; ++d) more[d] = lds.v[buffer][sub][kHalf + d][lane];
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int d = 0; d < kHalf; ++d) R::add_values(d, v[d], p);
#pragma unroll
    for (int d = 0; d < kHalf; ++d) R::add_values(kHalf + d, more[d], p);
  }

  // job.begin to job.end: the workgroup's positions; [own_begin, own_end) of them this wave's rows see.
  __device__ __forceinline__ void run(const AttentionArgs& a, const WaveJob& job, int wave, int own_begin, int own_end,
                                      WideBuffers<D>& lds) {
    R::clear();
    if (job.begin >= job.end) return;
    const int stages = (job.end - job.begin + kStage - 1) / kStage;
    constexpr int kWindow = 64 / kStageTiles;  // stages whose pages `ids` holds
    Raw raw[2];
    const auto tile_of = [&](int i) {
      return ((int64_t)job.begin + (int64_t)i * kStage) / kKvTile + (threadIdx.x & 63);
    };
    // Behind a condition loads would be waited for at its end, not where they
    // are used; so the last stage's are repeated, and put where none reads.
    const auto load = [&](int stage, Raw& to) {
      const int i = min(stage, stages - 1);
      if (i % kWindow == 0) window.take(a, job, tile_of(i));
      const uint32_t there = load_stage(a, job, wave, i % kWindow * kStageTiles, to);
      if (i % kWindow == kWindow / 2) window.ask(a, job, tile_of(i + kWindow / 2));
      return there;
    };
    window.ask(a, job, tile_of(0));
    uint32_t there = load(0, raw[0]), there_next = load(1, raw[1]);
    __syncthreads();  // the buffers have been read
    put(lds, 0, wave, raw[0]);
    __syncthreads();
    for (int i = 0;;) {
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const uint32_t later = load(i + 2, raw[u]);
#pragma unroll
        for (int sub = 0; sub < 2; ++sub) {
          const int at = job.begin + i * kStage + sub * kKvStep;
          if (at < own_end && at + kKvStep > own_begin) pass(a, job, at, lds, u, sub, there >> (2 * sub) & 3);
        }
        put(lds, u ^ 1, wave, raw[u ^ 1]);
        __syncthreads();
        there = there_next;
        there_next = later;
        if (++i == stages) return;
      }
    }
  }
};

// What one kernel is made for. WIDE: waves have rows of their own, NQ tiles of
// 16 each; else they share one tile and take turns with the positions. EXACT and
// FINE: of wide ones, as in RowSums.
template <int DT_, int D_, int NQ_, int PT_, bool WIDE_, bool ONE_, bool EXACT_ = false, bool FINE_ = true>
struct AttentionShape {
  static constexpr int DT = DT_, D = D_, NQ = NQ_, PT = PT_;
  static constexpr bool WIDE = WIDE_, ONE = ONE_, EXACT = EXACT_, FINE = FINE_;
};

// Where waves that share rows join their parts.
template <int D>
struct JoinBuffers {
  static constexpr int kRow = D + 4;  // rows start 4 banks apart
  float refs[kAttentionWaves][16], sums[kAttentionWaves][16];
  float exact[kAttentionWaves][16];  // sums of unrounded weights
  float outs[kAttentionWaves][16][kRow];
};

// A row's result, or with a slot its part.
template <class S>
__device__ __forceinline__ void store_sums(const AttentionArgs& a, const RowTile& tile, int slot, int in_tile,
                                           int token, int head, float ref, float sum, float exact) {
  if (slot >= 0)
    *reinterpret_cast<f32x4*>(a.part_ml + 4 * ((int64_t)slot * a.tile_rows + in_tile)) = f32x4{ref, sum, exact, 0.0f};
  else if (a.lse)
    a.lse[lse_index(a, tile, token, head)] = lse_of(ref, exact);
}
template <class S>
__device__ __forceinline__ void store_columns(const AttentionArgs& a, const RowTile& tile, int slot, int in_tile,
                                              int token, int head, int col, float sum, float (&f)[8]) {
  if (slot >= 0) {
    if (sum == 0.0f) return;  // no position, nothing to join
    Packed<RINGSIM_FLOAT32, 8> y;
    y.set(f);
    y.store<true>(a.part_out + ((int64_t)slot * a.tile_rows + in_tile) * S::D + col);
  } else {
    const float by = sum == 0.0f ? 0.0f : 1.0f / sum;
#pragma unroll
    for (int e = 0; e < 8; ++e) f[e] *= by;
    Packed<S::DT, 8> y;
    y.set(f);
    y.template store<true>(out_row<S::DT>(a, tile, token, head) + col);
  }
}

__device__ __forceinline__ WaveJob wave_job(const AttentionArgs& a, const RowTile& tile, int key_head) {
  const int64_t head = key_head * a.cache.head, scale_head = key_head * a.cache.scale_head;
  WaveJob job;
  job.k = a.cache.data[0] + head;
  job.v = a.cache.data[1] + head;
  job.ks = a.cache.scales[0] + scale_head;
  job.vs = a.cache.scales[1] + scale_head;
  job.pages = a.pages + tile.seq * a.page_stride;
  job.length = tile.length;
  return job;
}

// The rows row0 to row0 + rows of a tile that a wave has: what all of them see
// into job, and [*lo, *hi] what any of them sees.
__device__ __forceinline__ void wave_span(const AttentionArgs& a, const RowTile& tile, int row0, int rows, WaveJob& job,
                                          int* lo, int* hi) {
  const int row1 = min(row0 + rows, tile.rows) - 1;
  span(a, tile.first + row0 / a.group, tile.length, lo, &job.full_hi);
  span(a, tile.first + row1 / a.group, tile.length, &job.full_lo, hi);
}

// A lane's row of each tile of 16 from row0 on. One beyond the tile's last row
// repeats it, and is not stored.
template <int NQ>
struct LaneRows {
  int token[NQ], head[NQ];
};
template <int DT, int D, int NQ, int PT, bool EXACT, bool FINE>
__device__ __forceinline__ LaneRows<NQ> take_rows(const AttentionArgs& a, const RowTile& tile, int key_head, int row0,
                                                  RowSums<DT, D, NQ, PT, EXACT, FINE>& w) {
  const int c = threadIdx.x & 15;
  LaneRows<NQ> at;
#pragma unroll
  for (int r = 0; r < NQ; ++r) {
    const int row = min(row0 + 16 * r + c, tile.rows - 1);
    at.token[r] = row / a.group;
    at.head[r] = key_head * a.group + row - at.token[r] * a.group;
    span(a, tile.first + at.token[r], tile.length, &w.lo[r], &w.hi[r]);
  }
#pragma unroll
  for (int r = 0; r < NQ; ++r) w.load_queries(r, query_row<DT>(a, tile, at.token[r], at.head[r]));
  return at;
}

// The tile of 16 rows from row0 on out of a wave's sums.
template <class S, int NQ, bool EXACT, bool FINE>
__device__ __forceinline__ void store_rows(const AttentionArgs& a, const RowTile& tile, int slot, int row0,
                                           const RowSums<S::DT, S::D, NQ, S::PT, EXACT, FINE>& w,
                                           const LaneRows<NQ>& at, int r) {
  using H = HeadParts<S::D>;
  const int lane = threadIdx.x & 63, c = lane & 15, g = lane >> 4;
  const int in_tile = row0 - tile.row + c;
  const float exact = w.exact_sum(r);
  if (row0 + c >= tile.rows) return;
  const float sum = w.l[r][0];
  const float ref = w.m[r] == -__builtin_inff() && sum != 0.0f ? 0.0f : w.m[r];  // NaN sums without a maximum
  if (g == 0) store_sums<S>(a, tile, slot, in_tile, at.token[r], at.head[r], ref, sum, exact);
#pragma unroll
  for (int part = 0; part < H::kParts; ++part) {
    const int n = H::n(part), d0 = H::base(part) / 16;
#pragma unroll
    for (int k = 0; k < n; ++k) {  // 8 columns each
      float f[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const int at_col = 8 * k + e, i = at_col / (2 * n), j = at_col % (2 * n);
        f[e] = w.o[r][d0 + j][i];
      }
      store_columns<S>(a, tile, slot, in_tile, at.token[r], at.head[r], H::base(part) + 8 * n * g + 8 * k, sum, f);
    }
  }
}

// Rows of a tile with one key head over the positions [begin, end), begin a
// multiple of kKvStep; the result goes out, or into a slot if it is a part.
template <class S>
__device__ __forceinline__ void attend(const AttentionArgs& a, const RowTile& tile, int key_head, int begin, int end,
                                       int slot, WideBuffers<S::D>& lds) {
  constexpr int D = S::D, NQ = S::NQ;
  // What is the same for all lanes of a wave, and told to be, stays in scalar
  // registers: the loop's places and counts among it.
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int row0 = tile.row + wave * NQ * 16;
  WaveJob job = wave_job(a, tile, key_head);
  job.begin = begin;
  job.end = end;
  job.stride = kKvStep;
  bool bad;
  {
    WideWave<S::DT, D, NQ, S::PT, S::EXACT, S::FINE> w;
    int lo, hi;
    wave_span(a, tile, row0, NQ * 16, job, &lo, &hi);
    if (row0 >= tile.rows) hi = lo - 1;
    const auto at = take_rows(a, tile, key_head, row0, w);
    w.run(a, job, wave, max(begin, lo), min(end, hi + 1), lds);
    bad = w.has_nan();
    if (!bad) {
#pragma unroll
      for (int r = 0; r < NQ; ++r) store_rows<S>(a, tile, slot, row0 + 16 * r, w, at, r);
    }
  }
  if (bad) {
    for (int r = 0; r < NQ; ++r) {
      const int first = row0 + 16 * r;
      if (first >= tile.rows) break;
      AttentionWave<S::DT, D, 1, S::PT, 1, false> w;
      int lo, hi;
      wave_span(a, tile, first, 16, job, &lo, &hi);
      job.begin = max(begin, lo / kKvStep * kKvStep);
      job.end = min(end, hi + 1);
      const auto at = take_rows(a, tile, key_head, first, w);
      w.template run<true>(a, job, [] {});
      store_rows<S>(a, tile, slot, first, w, at, 0);
    }
  }
}

template <class S>
__device__ __forceinline__ void attend(const AttentionArgs& a, const RowTile& tile, int key_head, int begin, int end,
                                       int slot, JoinBuffers<S::D>& lds) {
  constexpr int D = S::D;
  using H = HeadParts<D>;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int lane = threadIdx.x & 63, c = lane & 15, g = lane >> 4;
  AttentionWave<S::DT, D, 1, S::PT, 1, S::ONE> w;
  WaveJob job = wave_job(a, tile, key_head);
  int lo, hi;
  wave_span(a, tile, tile.row, 16, job, &lo, &hi);
  job.stride = kAttentionWaves * kKvStep;
  job.begin = begin + wave * kKvStep;
  job.end = min(end, hi + 1);
  w.template run<false>(a, job, [&] { take_rows(a, tile, key_head, tile.row, w); });
  if constexpr (!S::ONE) {
    if (w.has_nan()) w.template run<true>(a, job, [] {});
  }
  // The waves' parts of the positions, joined in a fixed order.
  const float own = w.m[0] == -__builtin_inff() && w.l[0][0] != 0.0f ? 0.0f : w.m[0];  // NaN sums without a maximum
  const float unrounded = w.exact_sum(0);
  if (g == 0) {
    lds.refs[wave][c] = own;
    lds.sums[wave][c] = w.l[0][0];
    lds.exact[wave][c] = unrounded;
  }
  __syncthreads();
  float top = lds.refs[0][c];
#pragma unroll
  for (int i = 1; i < kAttentionWaves; ++i) top = fmaxf(top, lds.refs[i][c]);
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
      *reinterpret_cast<f32x4*>(&lds.outs[wave][c][H::base(part) + 8 * n * g + 4 * k]) = f;
    }
  }
  __syncthreads();
  const int rows = min(16, tile.rows - tile.row);
  for (int k = threadIdx.x; k < rows * (D / 8); k += kAttentionThreads) {
    const int row = k / (D / 8), col = (k - row * (D / 8)) * 8;
    float best = lds.refs[0][row], sum = 0.0f, exact = 0.0f;
#pragma unroll
    for (int i = 1; i < kAttentionWaves; ++i) best = fmaxf(best, lds.refs[i][row]);
#pragma unroll
    for (int i = 0; i < kAttentionWaves; ++i) {
      const float ref = lds.refs[i][row];
      if (ref == -__builtin_inff()) continue;
      const float scale = ref == best ? 1.0f : __builtin_amdgcn_exp2f(ref - best);
      sum += lds.sums[i][row] * scale;
      exact += lds.exact[i][row] * scale;
    }
    float f[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      f[e] = lds.outs[0][row][col + e];
#pragma unroll
      for (int i = 1; i < kAttentionWaves; ++i) f[e] += lds.outs[i][row][col + e];
    }
    const int t = (tile.row + row) / a.group, h = key_head * a.group + tile.row + row - t * a.group;
    if (col == 0) store_sums<S>(a, tile, slot, row, t, h, best, sum, exact);
    store_columns<S>(a, tile, slot, row, t, h, col, sum, f);
  }
  __syncthreads();  // before the buffers are written again
}

// Units of all tiles, counted by each workgroup for itself.
struct SharedUnits {
  int32_t starts[kSharedTiles + 1];  // a copy, with starts
  int32_t units[kSharedTiles];
};

// Either a workgroup a tile and key head, or an equal share of all units a
// workgroup: it walks over the tiles that its share touches.
template <class S>
__global__ __launch_bounds__(kAttentionThreads, S::WIDE && S::D <= 192 ? 2 : 1) void attention_kernel(
    const AttentionArgs a) {
  __shared__ std::conditional_t<S::WIDE, WideBuffers<S::D>, JoinBuffers<S::D>> lds;
  RowTile tile;
  if (a.groups == 0) {
    // The last tiles first: in causal order they see most.
    const int from_last = blockIdx.x / a.cache.heads, index = a.tiles - 1 - from_last;
    if (!row_tile(a, a.starts, index, tile)) return;
    tile = same_tile(tile);
    int lo, hi;
    tile_span(a, tile, &lo, &hi);
    attend<S>(a, tile, blockIdx.x - from_last * a.cache.heads, lo / kKvStep * kKvStep, hi + 1, -1, lds);
    return;
  }
  __shared__ SharedUnits all;
  if (a.starts) {
    for (int i = threadIdx.x; i <= a.seqs; i += kAttentionThreads) all.starts[i] = a.starts[i];
    __syncthreads();
  }
  // Units of each tile: with up to 64 tiles one a lane, in each wave for itself;
  // otherwise they are counted in LDS, and a lane adds kRun of them.
  constexpr int kRun = kSharedTiles / 64;
  const int lane = threadIdx.x & 63;
  const bool few = !S::WIDE && a.tiles <= 64;  // with many rows the registers are needed
  const auto units_of = [&](int i, RowTile& t) {
    if (i >= a.tiles || !row_tile(a, all.starts, i, t)) return 0;
    int lo, hi;
    tile_span(a, t, &lo, &hi);
    return (int)kv_units(lo, hi);
  };
  RowTile mine = {0, 0, 0, 0, 0, 0};
  int own = 0;
  if (few) {
    own = units_of(lane, mine);
  } else {
    for (int i = threadIdx.x; i < kSharedTiles; i += kAttentionThreads) all.units[i] = units_of(i, mine);
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kRun; ++i) own += all.units[lane * kRun + i];
  }
  int upto = own;
#pragma unroll
  for (int d = 1; d < 64; d *= 2) {
    const int x = __shfl_up(upto, d);
    upto += lane >= d ? x : 0;
  }
  const int64_t per_head = __builtin_amdgcn_readlane(upto, 63);
  if (per_head == 0) return;
  const uint32_t units = (uint32_t)per_head * (uint32_t)a.cache.heads;
  // No share is empty, so that the parts of a tile are those of consecutive
  // workgroups. Neighbouring shares, which read the same keys where tiles of one
  // sequence follow one another, go to workgroups of one XCD: those take turns.
  const int groups = (int)min((uint32_t)a.groups, units), per_xcd = (groups + 7) / 8;
  const int group = (blockIdx.x & 7) * per_xcd + (blockIdx.x >> 3);
  if ((int)(blockIdx.x >> 3) >= per_xcd || group >= groups) return;
  int64_t at = __builtin_amdgcn_readfirstlane((int)kv_share_begin(units, group, groups));
  const int64_t end = __builtin_amdgcn_readfirstlane((int)kv_share_begin(units, group + 1, groups));
  int key_head = __builtin_amdgcn_readfirstlane((uint32_t)at / (uint32_t)per_head);
  const int in_head = (int)(at - key_head * per_head);
  const int run = __builtin_ctzll(__ballot(upto > in_head));  // the lane whose tiles hold the first unit
  int index = few ? run : run * kRun;
  int before = __builtin_amdgcn_readlane(upto - own, run);  // units of the key head before tile `index`
  while (at < end) {
    int n;
    for (;;) {
      n = few ? __builtin_amdgcn_readlane(own, index) : __builtin_amdgcn_readfirstlane(all.units[index]);
      if (at - key_head * per_head < before + n) break;
      before += n;
      if (++index == a.tiles) {
        index = before = 0;
        ++key_head;
      }
    }
    const int64_t first = key_head * per_head + before;  // the tile's units are [first, first + n)
    const int skip = (int)(at - first), take = (int)min((int64_t)n - skip, end - at);
    if (few) {
      tile = tile_of_lane(mine, index);
    } else {
      row_tile(a, all.starts, index, tile);
    }
    tile = same_tile(tile);
    int lo, hi;
    tile_span(a, tile, &lo, &hi);
    if (threadIdx.x == 0) {  // the first and the last workgroup with a part of the tile say so
      int32_t* of = a.part_of + 2 * ((int64_t)index * a.cache.heads + key_head);
      if (skip == 0) of[0] = group;
      if (skip + take == n) of[1] = group;
    }
    const int begin = lo / kKvStep * kKvStep + skip * kKvUnit;
    const int slot = take == n ? -1 : part_slot(group, skip == 0);
    const auto uniform = [](int x) { return __builtin_amdgcn_readfirstlane(x); };
    attend<S>(a, tile, uniform(key_head), uniform(begin), uniform(min(begin + take * kKvUnit, hi + 1)), uniform(slot),
              lds);
    at += take;
  }
}

template <class S>
hipError_t launch_shape(const AttentionArgs& a, hipStream_t s) {
  const unsigned grid = a.groups ? (unsigned)a.groups : (unsigned)a.tiles * (unsigned)a.cache.heads;
  hipLaunchKernelGGL((attention_kernel<S>), dim3(grid), dim3(kAttentionThreads), 0, s, a);
  return hipGetLastError();
}

// bf16 outputs: with few rows memory bounds, and weights in two parts cost
// nothing; with many they would take 222 us for 163 (three prompts of 2048 tokens
// of 32 heads of 128).
template <int DT, int D>
hipError_t launch_type(const AttentionArgs& a, const AttentionPlan& plan, hipStream_t s) {
  constexpr int kParts = DT == RINGSIM_FLOAT32 ? 3 : 2;
  if (plan.wide) {
    constexpr int kWideParts = DT == RINGSIM_BFLOAT16 ? 1 : kParts, kTiles = wide_tiles(DT, D, false);
    if constexpr (DT == RINGSIM_FLOAT32) {
      return launch_shape<AttentionShape<DT, D, kTiles, kWideParts, true, false>>(a, s);
    } else {
      if (plan.fine)
        return launch_shape<AttentionShape<DT, D, wide_tiles(DT, D, true), kWideParts, true, false, true>>(a, s);
      return a.lse ? launch_shape<AttentionShape<DT, D, kTiles, kWideParts, true, false, true, false>>(a, s)
                   : launch_shape<AttentionShape<DT, D, kTiles, kWideParts, true, false, false, false>>(a, s);
    }
  }
  return !a.starts && a.each == 1 ? launch_shape<AttentionShape<DT, D, 1, kParts, false, true>>(a, s)
                                  : launch_shape<AttentionShape<DT, D, 1, kParts, false, false>>(a, s);
}

template <int D>
hipError_t launch_head(const AttentionArgs& a, const AttentionPlan& plan, int dtype, hipStream_t s) {
  switch (dtype) {
    case RINGSIM_FLOAT32: return launch_type<RINGSIM_FLOAT32, D>(a, plan, s);
    case RINGSIM_BFLOAT16: return launch_type<RINGSIM_BFLOAT16, D>(a, plan, s);
    case RINGSIM_FLOAT16: return launch_type<RINGSIM_FLOAT16, D>(a, plan, s);
    default: return hipErrorInvalidValue;
  }
}

}  // namespace ringsim
