// kv_attention.hip -- attention over the paged 4-bit cache of kv_cache.hip.
//
//   e[i,t] = scale q_i . k_t,   y_i = sum_t exp(e[i,t]) v_t / sum_t exp(e[i,t])
//
// over the tokens t that query i sees.  Keys and values are s (n - z), one scale s
// and zero z per token and group g of 64 channels, so the codes enter the matrix
// products as they are and everything else stays with the (query, token) pairs:
//
//   q . k_t        = sum_g s_g (sum_d q_d n_d - z_g sum_d q_d)
//   sum_t p_t v_t  = sum_t (p_t s_g) n_d - sum_t (p_t s_g) z_g
//
// (where the result is fp16 or fp32 the second is summed as (p_t s_g) (n_d - z_g), which
// costs a subtraction a pair of codes and keeps what the difference cancels).
// A nibble n at the low end of a 16-bit half is a subnormal fp16 number, which the
// matrix unit takes without loss; the powers of two go into the factors and the end.
// But the unit aligns the terms of a sum by the exponents that their operands have,
// which for every subnormal number is that of 2^-14.  Shifted to n 2^-18 (FINE: four
// masks and four shifts for eight codes) a sum keeps fp32's 2^-20 of its largest q
// (or p s).  As n 2^-24 and n 2^-20, where the nibbles lie (four masks and one shift),
// it keeps 2^-14: scores of about 30, and lse, would be off by 3e-4 instead of 2e-6, so
// the keys are shifted; for the values that is a sixteenth of what rounding p s
// leaves, and they are shifted where the result is not bf16.
// Queries are held in fp16 under a power of two per row
// (what that loses is below 2^-34 of the row's largest channel), their sums
// against 1 and not against a code of 1.  p s is the only value that is rounded: to
// fp16 (11 bits, three more than a bf16 result has), or, where the result is fp16 or fp32,
// to the sum of two: in 11 bits it would add as much to an fp16 result as its own rounding
// does (up to 1.8 times the error of fp32 sums; the second term takes 2 x 1024 rows over
// 6000 tokens, 32 heads of 128, from 330 to 455 us).  Its range is
// kept by the row's offset o, a whole number: p = 2^(e log2(e) - o) with o such
// that p s stays below 2^15; o moves, and the sums with it by an exact power of
// two, only when a tile would exceed that (seven doublings above the tile that set
// it), so the running maximum of the softmax costs one comparison a tile.  All groups
// share it, and fp16 ends at 2^-24: p s is not held finer than 2^-32 of the row's largest,
// which a group of values that small beside another feels.  Whole numbers
// are exact up to 2^24, and e log2(e) - o is then one fused operation.  A row whose scores go
// beyond 2^22 (kFar) has a base b besides, its largest score as fp32 rounds it: the
// difference to it is 0 for that token and all that tie with it, and p = 2^((e log2(e) - b)
// - o).  b and o of such rows lie in LDS, and the loop holds the offset of a row that has
// seen nothing for them, which every tile exceeds: they cost the others nothing (as a branch
// around them in the loop they took 3 % of a prompt's time).
//
// Three forms, by the query rows that share a head of the cache in one sequence:
//
// - Up to 8 rows (a token or two of a few heads each), 4 with heads of 256: the 4 x 4
//   products.  A lane is a token of its group's channels in the first and two channels in
//   the second, so no lane's work is lost on rows that do not exist, which in 16 x 16
//   tiles is three quarters at four rows.  The first product leaves tokens 4 c .. 4 c + 3
//   of row j in lane 4 c + j, which is the second's operand.  The call is bound by
//   the read of the cache.
// - Up to 63 rows: 16 x 16 products, transposed (tokens x queries, channels x
//   queries), so that here too a lane needs for the second product the tokens that
//   the first one gave it.
// - More (prompts): the same, two row tiles to a wave, and each wave has rows of its own.
//
// In none of them p leaves the registers, and the loop has no barrier and no LDS but a
// base's.
// In the first two the waves of a workgroup deal out its tokens, and
// workgroups split long sequences (k_kv_join adds their parts).
#include "hsq_internal.h"

#include <algorithm>
#include <utility>

namespace hsq {

namespace {

typedef _Float16 v8h __attribute__((ext_vector_type(8)));

constexpr float kNoOffset = -0x1.fffffep127f;   // of a row that has seen nothing: no score lies below
constexpr float kTop = 8.0f;             // p s of the tile that sets the offset stays below 2^kTop
constexpr float kMaxPs = 32768.0f;       // what moves the offset
constexpr float kMaxP = 1099511627776.0f;   // 2^40: the same for tokens of scale 0
constexpr float kHidden = -__builtin_inff();   // the score of a token that is not seen
constexpr float kFar = 4194304.0f;             // 2^22: scores from which a row has a base of its own
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kTiny = 5.9604644775390625e-8f;   // 2^-24: of a code in the lowest bits

__device__ __forceinline__ v4f mfma16(v4u a, v4u b, v4f c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(v8h, a), __builtin_bit_cast(v8h, b), c, 0, 0, 0);
}

// 16 products of 4 x 4; with BLOCK >= 0 each half of the wave takes block BLOCK of
// its own eight blocks of a for all of them.
template <int BLOCK>
__device__ __forceinline__ v4f mfma4(v2u a, v2u b, v4f c) {
  return __builtin_amdgcn_mfma_f32_4x4x4f16(__builtin_bit_cast(v4h, a), __builtin_bit_cast(v4h, b), c, BLOCK >= 0 ? 3 : 0,
                                            BLOCK >= 0 ? BLOCK : 0, 0);
}

// Eight codes as subnormal numbers: the low nibbles of a dword's bytes 0, 2 and 1, 3
// and the high ones.  FINE: all n 2^-18, otherwise n 2^-24 and n 2^-20, which saves
// three shifts a dword.
constexpr uint32_t kLow = 0x000F000Fu, kHigh = 0x00F000F0u, kTopBits = 0x03C003C0u, kOnes = 0x3C003C00u;
template <bool FINE>
struct Unit {
  static constexpr float low = FINE ? 262144.0f : 16777216.0f, high = FINE ? 262144.0f : 1048576.0f;   // one code is 1 / low
};
template <bool FINE>
__device__ __forceinline__ v2u low_codes(uint32_t w) {
  return FINE ? (v2u){w << 6 & kTopBits, w >> 2 & kTopBits} : (v2u){w & kLow, w >> 8 & kLow};
}
template <bool FINE>
__device__ __forceinline__ v2u high_codes(uint32_t w) {
  return FINE ? (v2u){w << 2 & kTopBits, w >> 6 & kTopBits} : (v2u){w & kHigh, w >> 8 & kHigh};
}

__device__ __forceinline__ uint32_t pack_h(float a, float b) {
  v2h h = {(_Float16)a, (_Float16)b};
  return __builtin_bit_cast(uint32_t, h);
}
// n - z, two at a time, under the same power of two (exact, subnormal)
__device__ __forceinline__ uint32_t minus_h(uint32_t a, uint32_t b) {
  return __builtin_bit_cast(uint32_t, __builtin_bit_cast(v2h, a) - __builtin_bit_cast(v2h, b));
}
__device__ __forceinline__ float half_of(v4u w, int i) { return f16_to_f32((uint16_t)(w[i >> 1] >> (16 * (i & 1)))); }
__device__ __forceinline__ float half_of(v2u w, int i) { return f16_to_f32((uint16_t)(w[i >> 1] >> (16 * (i & 1)))); }
// The zeros of four tokens in a dword (bytes 0, 2, 1, 3), masked at once.
__device__ __forceinline__ uint32_t zeros_of(uint32_t w) {
  w &= 0x0F0F0F0Fu;
  asm("" : "+v"(w));      // else every byte is masked by itself
  return w;
}
__device__ __forceinline__ float zero_of(uint32_t w, int r) {
  return (float)(w >> (8 * (((r & 1) << 1) | (r >> 1))) & 0xFFu);
}

// The lane's number, formed where it is used: no register holds it through the loop.
__device__ __forceinline__ int lane_here() {
  uint32_t all = ~0u;
  asm volatile("" : "+s"(all));
  return (int)__builtin_amdgcn_mbcnt_hi(all, __builtin_amdgcn_mbcnt_lo(all, 0u));
}

// Reductions over lanes that differ in the bits of FROM .. TO.
template <int FROM, int TO>
__device__ __forceinline__ float max_over(float v) {
#pragma unroll
  for (int m = FROM; m <= TO; m <<= 1) v = fmaxf(v, __shfl_xor(v, m));
  return v;
}
template <int FROM, int TO>
__device__ __forceinline__ float sum_over(float v) {
#pragma unroll
  for (int m = FROM; m <= TO; m <<= 1) v += __shfl_xor(v, m);
  return v;
}

__device__ __forceinline__ void unpack8(v4u w, int dtype, float *f) {
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    f[2 * e] = dtype == kBf16 ? bf16_to_f32(w[e] & 0xFFFFu) : f16_to_f32((uint16_t)w[e]);
    f[2 * e + 1] = dtype == kBf16 ? __uint_as_float(w[e] & 0xFFFF0000u) : f16_to_f32((uint16_t)(w[e] >> 16));
  }
}
typedef unsigned short v2us __attribute__((ext_vector_type(2)));
// The larger magnitudes of two pairs, by their bits: infinities and NaN on top.
__device__ __forceinline__ uint32_t larger(uint32_t a, uint32_t b) {
  return __builtin_bit_cast(uint32_t, __builtin_elementwise_max(__builtin_bit_cast(v2us, a), __builtin_bit_cast(v2us, b & 0x7FFF7FFFu)));
}
__device__ __forceinline__ uint32_t larger8(uint32_t top, v4u w) {
#pragma unroll
  for (int e = 0; e < 4; ++e) top = larger(top, w[e]);
  return top;
}
__device__ __forceinline__ float magnitude(uint32_t top, int dtype) {
  const uint32_t h = max(top & 0xFFFFu, top >> 16);
  return dtype == kBf16 ? bf16_to_f32(h) : f16_to_f32((uint16_t)h);
}
// Eight channels of a query as fp16 by `by`.
__device__ __forceinline__ v4u scaled8(v4u w, int dtype, float by) {
  float f[8];
  unpack8(w, dtype, f);
  return (v4u){pack_h(f[0] * by, f[1] * by), pack_h(f[2] * by, f[3] * by), pack_h(f[4] * by, f[5] * by),
               pack_h(f[6] * by, f[7] * by)};
}
// The power of two that takes a row's largest channel to [2^13, 2^14), and the
// factor from the products' sums to scores in powers of two.  The factor stays a normal
// number: as 0 it would make NaN of a hidden token's -infinity, as an infinity of a sum
// of 0.  Below 2^-126 it leaves every weight 1 as it was (sums are below 2^40); beyond
// fp32 any two sums that differ are more than 2^60 apart, and only lse is cut.
__device__ __forceinline__ float row_power(float top, float scale2, float &to_score) {
  const int ex = min(max((int)(__float_as_uint(top) >> 23) - 13, 1), 240);
  to_score = __uint_as_float((uint32_t)ex << 23) * (Unit<true>::low * scale2);
  to_score = fminf(fmaxf(to_score, 0x1p-126f), 0x1.fffffep127f);
  return __uint_as_float((uint32_t)(254 - ex) << 23);
}

// Tokens [lo, hi) that token i of a sequence sees.
struct Seen { int lo, hi; };
__device__ __forceinline__ Seen seen_by(const KvAttnArgs &a, int i, int p0, int len) {
  const int pos = p0 + i;                 // may be negative: sees nothing
  Seen s{0, len};
  if (a.causal) {
    s.hi = min(max(pos + 1, 0), len);
    if (a.window > 0 && a.window <= pos) s.lo = pos - a.window + 1;
  }
  return s;
}

// Tiles [first, last) that rows [r0, r1) of a sequence see.
__device__ __forceinline__ void tiles_of_rows(const KvAttnArgs &a, int r0, int r1, int p0, int len, int &first,
                                              int &last) {
  const Seen s0 = seen_by(a, r0 / a.gr, p0, len), s1 = seen_by(a, (r1 - 1) / a.gr, p0, len);
  first = s0.lo / kKvTile;
  last = (s1.hi + kKvTile - 1) / kKvTile;
}

// Tiles of one part of [first, last).
constexpr int kMinTiles = 32;             // a part is 1024 tokens at least
constexpr int kMaxParts = 64;
__device__ __forceinline__ int tiles_of_part(int first, int last, int splits) {
  return max((last - first + splits - 1) / splits, kMinTiles);
}

template <int DT>
__device__ __forceinline__ void store4(void *Y, size_t at, v4f y) {
  if constexpr (DT == kF32) {
    *reinterpret_cast<v4f *>(static_cast<float *>(Y) + at) = y;
  } else {
    uint32_t u[4];
#pragma unroll
    for (int r = 0; r < 4; ++r)
      u[r] = DT == kBf16 ? __builtin_bit_cast(uint16_t, (__bf16)y[r]) : f32_to_f16(y[r]);
    *reinterpret_cast<v2u *>(static_cast<uint16_t *>(Y) + at) = (v2u){u[0] | u[1] << 16, u[2] | u[3] << 16};
  }
}

__device__ __forceinline__ void store_y(const KvAttnArgs &a, size_t at, v4f y) {
  if (a.y_dtype == kF32) store4<kF32>(a.Y, at, y);
  else if (a.y_dtype == kBf16) store4<kBf16>(a.Y, at, y);
  else store4<kF16>(a.Y, at, y);
}

__device__ __forceinline__ float lse_of(float o, float l) {
  return l == 0.0f ? -__builtin_inff() : (__builtin_amdgcn_logf(l) + o) * kLn2;
}
__device__ __forceinline__ float inverse(float l) { return l == 0.0f ? 0.0f : 1.0f / l; }


// ------------------------------------------------------------------ 16 x 16
// One side of a tile: codes, scales, zeros.
template <int D>
struct Side {
  static constexpr int G = D / kKvGroup;
  v4u code[G], s[G];
  v2u z[G];
};

template <int D, bool V>
__device__ __forceinline__ void load_side(const uint8_t *p, int lane, Side<D> &t) {
  constexpr int G = D / kKvGroup;
  const int q = lane >> 4;
#pragma unroll
  for (int x = 0; x < G; ++x) t.code[x] = *reinterpret_cast<const v4u *>(p + (V ? 16 * D : 0) + x * 1024 + lane * 16);
#pragma unroll
  for (int x = 0; x < G; ++x) {
    t.s[x] = *reinterpret_cast<const v4u *>(p + 32 * D + (V ? 64 * G : 0) + x * 64 + q * 16);
    t.z[x] = *reinterpret_cast<const v2u *>(p + 32 * D + 128 * G + (V ? 32 * G : 0) + (q * G + x) * 8);
  }
}

// Sums of a wave: MT row tiles, lane's query is column lane % 16 of each.
template <int D, int MT>
struct Sums {
  static constexpr int G = D / kKvGroup;
  v4f acc[MT][D / 16];     // channels 16 nt + 4 (lane / 16) + r, under the codes' Unit (nt even low, odd high)
  v4f zero[MT][G];         // the sums of (p s) z, under Unit's low: all four alike; 0 with two terms
  float o[MT], l[MT];      // l: this lane's tokens only
};

// The scores of 32 tokens: e[m][4 a + r] of token 16 a + 4 q + r.
template <int D, int MT>
__device__ __forceinline__ void scores(const Side<D> &t, const v4u (&Q)[MT][D / 32], const float (&qs)[MT][D / 64],
                                       float (&e)[MT][8]) {
  constexpr int G = D / kKvGroup;
#pragma unroll
  for (int a = 0; a < 2; ++a) {
#pragma unroll
    for (int g = 0; g < G; ++g) {
      v4u k[2];
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        const int i = a * (D / 32) + 2 * g + x;
        const v2u low = low_codes<true>(t.code[i >> 2][i & 3]), high = high_codes<true>(t.code[i >> 2][i & 3]);
        k[x] = (v4u){low[0], low[1], high[0], high[1]};
      }
      const uint32_t zw = zeros_of(t.z[g][a]);
#pragma unroll
      for (int m = 0; m < MT; ++m) {
        v4f d = mfma16(k[0], Q[m][2 * g], (v4f){0.0f, 0.0f, 0.0f, 0.0f});
        d = mfma16(k[1], Q[m][2 * g + 1], d);
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const float u = __builtin_fmaf(-zero_of(zw, r), qs[m][g], d[r]);
          e[m][4 * a + r] = __builtin_fmaf(u, half_of(t.s[g], 4 * a + r), g ? e[m][4 * a + r] : 0.0f);
        }
      }
    }
    __builtin_amdgcn_sched_barrier(0);   // half of the operands at a time
  }
}

// The base of a row that had `had` (0: none) and whose tile's largest score is `high`.
__device__ __forceinline__ float base_with(float2 had, float high) {
  const float b = had.x != 0.0f ? fmaxf(had.x, high) : high;
  return b == 0.0f ? 0x1p-126f : b;      // 0 is none, and scores do not tell the two apart
}
// The offset beside base b, where the tile's largest p s is at `near` from it: it moves down
// only with the base.
__device__ __forceinline__ float rebase(float near, float b, float2 had) {
  const float o = __builtin_ceilf(near) - kTop;
  return had.x == b ? fmaxf(o, had.y) : o;
}

// Their weights: l, and p s as the second product's operand (w, and w2 what its
// rounding leaves).  vs: the values' scales; c2: from e to powers of two; masked:
// some e is hidden; base: the wave's rows' b and o, b = 0 where a row has none.
template <int D, int MT, bool SPLIT>
__device__ __forceinline__ void weigh(const float (&e)[MT][8], v4u (&vs)[D / 64], const float (&c2)[MT], bool masked,
                                      float2 *base, Sums<D, MT> &s, v4u (&w)[MT][D / 64], v4u (&w2)[MT][D / 64]) {
  constexpr int G = D / kKvGroup;
  float p[MT][8], top[MT], topp[MT];
  bool any_base = false;                  // of this tile: such a row exceeds the range in every one
  auto form = [&](auto again) __attribute__((always_inline)) {
    // the scales stay packed: converted for both uses at once they would hold 8 G registers
#pragma unroll
    for (int g = 0; g < G; ++g) asm volatile("" : "+v"(vs[g]));
    bool moved = false;
#pragma unroll
    for (int m = 0; m < MT; ++m) {
      topp[m] = 0.0f;
#pragma unroll
      for (int i = 0; i < 8; ++i) p[m][i] = __builtin_fmaf(e[m][i], c2[m], -s.o[m]);
      if (decltype(again)::value && any_base) {
        const float2 b = base[16 * m + (lane_here() & 15)];
#pragma unroll
        for (int i = 0; i < 8; ++i) p[m][i] = b.x != 0.0f ? (e[m][i] * c2[m] - b.x) - b.y : p[m][i];
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        p[m][i] = __builtin_amdgcn_exp2f(p[m][i]);
        topp[m] = fmaxf(topp[m], p[m][i]);
      }
      top[m] = 0.0f;
#pragma unroll
      for (int g = 0; g < G; ++g) {
        float ps[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) ps[i] = __builtin_fmaf(p[m][i], half_of(vs[g], i), 0.0f);
        if (masked) {      // a hidden token's scale may be anything, NaN among it
#pragma unroll
          for (int i = 0; i < 8; ++i) ps[i] = e[m][i] == kHidden ? 0.0f : ps[i];
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) top[m] = fmaxf(top[m], ps[i]);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint32_t hi = pack_h(ps[2 * i], ps[2 * i + 1]);   // (a bit_cast of w[m][g][i] reads w[m][g][0])
          w[m][g][i] = hi;
          if (SPLIT) {
            const v2h h = __builtin_bit_cast(v2h, hi);
            w2[m][g][i] = pack_h(ps[2 * i] - (float)h[0], ps[2 * i + 1] - (float)h[1]);
          }
        }
      }
      moved |= top[m] > kMaxPs || topp[m] > kMaxP;
    }
    return __any(moved) != 0;
  };
  if (__builtin_expect(form(std::false_type{}), 0)) {
    // rare: the rows that exceed the range take the offset of this tile's largest
    // p s; one value at a time, since the registers used here are the kernel's
#pragma unroll
    for (int m = 0; m < MT; ++m) {
      const float mine = top[m] > kMaxPs || topp[m] > kMaxP ? 1.0f : 0.0f;
      const bool move = max_over<16, 32>(mine) > 0.0f;
      float2 &own = base[16 * m + (lane_here() & 15)];
      const float2 had = own;
      float most = kHidden;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
#pragma unroll
        for (int g = 0; g < G; ++g) {
          asm volatile("" : "+v"(vs[g]));
          most = fmaxf(most, __builtin_fmaf(e[m][i], c2[m], __builtin_amdgcn_logf(fmaxf(half_of(vs[g], i), kTiny))));
        }
        __builtin_amdgcn_sched_barrier(0);
      }
      most = max_over<16, 32>(most);
      float o = move ? __builtin_ceilf(most) - kTop : s.o[m], al = move ? __builtin_amdgcn_exp2f(s.o[m] - o) : 1.0f;
      const bool based = move && (had.x != 0.0f || fabsf(most) >= kFar);
      if (__any(based)) {
        any_base = true;
        float high = kHidden;
#pragma unroll
        for (int i = 0; i < 8; ++i) high = fmaxf(high, e[m][i] * c2[m]);
        high = max_over<16, 32>(high);
        const float b = base_with(had, high);
        float near = kHidden;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
#pragma unroll
          for (int g = 0; g < G; ++g) {
            asm volatile("" : "+v"(vs[g]));
            near = fmaxf(near, (e[m][i] * c2[m] - b) + __builtin_amdgcn_logf(fmaxf(half_of(vs[g], i), kTiny)));
          }
          __builtin_amdgcn_sched_barrier(0);
        }
        near = rebase(max_over<16, 32>(near), b, had);
        if (based) {
          al = __builtin_amdgcn_exp2f((had.x - b) + ((had.x != 0.0f ? had.y : s.o[m]) - near));
          o = kNoOffset;
          own = make_float2(b, near);
        }
      }
      s.o[m] = o;
      s.l[m] *= al;
#pragma unroll
      for (int n = 0; n < D / 16; ++n) s.acc[m][n] *= al;
#pragma unroll
      for (int g = 0; g < G; ++g) s.zero[m][g] *= al;
    }
    form(std::true_type{});
  }
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int i = 0; i < 8; ++i) s.l[m] += p[m][i];
}

// The second product.
template <int D, int MT, bool SPLIT>
__device__ __forceinline__ void values(const Side<D> &t, const v4u (&w)[MT][D / 64], const v4u (&w2)[MT][D / 64],
                                       Sums<D, MT> &s) {
#pragma unroll
  for (int g = 0; g < D / kKvGroup; ++g) {
    const uint32_t z0 = t.z[g][0], z1 = t.z[g][1];
    const v2u l0 = low_codes<SPLIT>(z0), l1 = low_codes<SPLIT>(z1);
    const v4u zz = {l0[0], l0[1], l1[0], l1[1]};
    if (!SPLIT) {
#pragma unroll
      for (int m = 0; m < MT; ++m) s.zero[m][g] = mfma16(zz, w[m][g], s.zero[m][g]);
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {         // channels 32 p ..: 32 tokens in two dwords
      const int pr = 2 * g + h;
      const uint32_t v0 = t.code[pr >> 1][2 * (pr & 1)], v1 = t.code[pr >> 1][2 * (pr & 1) + 1];
      const v2u low0 = low_codes<SPLIT>(v0), low1 = low_codes<SPLIT>(v1), high0 = high_codes<SPLIT>(v0), high1 = high_codes<SPLIT>(v1);
      v4u b0 = {low0[0], low0[1], low1[0], low1[1]}, b1 = {high0[0], high0[1], high1[0], high1[1]};
      if (SPLIT) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          b0[i] = minus_h(b0[i], zz[i]);
          b1[i] = minus_h(b1[i], zz[i]);
        }
      }
#pragma unroll
      for (int m = 0; m < MT; ++m) {
        s.acc[m][2 * pr] = mfma16(b0, w[m][g], s.acc[m][2 * pr]);
        s.acc[m][2 * pr + 1] = mfma16(b1, w[m][g], s.acc[m][2 * pr + 1]);
        if (SPLIT) {
          s.acc[m][2 * pr] = mfma16(b0, w2[m][g], s.acc[m][2 * pr]);
          s.acc[m][2 * pr + 1] = mfma16(b1, w2[m][g], s.acc[m][2 * pr + 1]);
        }
      }
    }
  }
}

// Where a workgroup of rows [r0, ..) of a sequence stands.
struct Place {
  int b, h, block, part, start, rows, len, p0;
};
__device__ __forceinline__ Place place_of(const KvAttnArgs &a, int splits, int block, int block_rows) {
  Place c;
  c.h = blockIdx.y;
  c.part = splits == 1 ? 0 : blockIdx.z % splits;
  c.b = splits == 1 ? blockIdx.z : blockIdx.z / splits;
  c.block = block;
  c.rows = 0;
  if (a.c.searched) {
    c.b = kv_block(a.c, block, a.gr, block_rows, 1, c.block);
    if (c.b < 0) {
      c.block = 0;                        // no rows: every wave returns
      return c;
    }
  }
  int n;
  kv_rows(a.c, c.b, c.start, n);
  c.rows = min(n, a.c.max_tokens) * a.gr;      // positions count all rows, the others are left alone
  c.len = kv_len(a.c, c.b);
  c.p0 = max(a.c.lens[c.b], 0) - n;
  return c;
}

// The sums of a workgroup's waves, in LDS as [wave][row][D + 4] and (offset,
// weight) [wave][row], joined and stored: the result, or a part of it.
template <int D, int ROWS, int W>
__device__ __forceinline__ void join_waves(const KvAttnArgs &a, const Place &c, int r0, const float *lds, const float2 *ol) {
  constexpr int kLd = D + 4;
  for (int i = threadIdx.x; i < ROWS * (D / 4); i += 64 * W) {
    const int row = i / (D / 4), d = i % (D / 4) * 4, rr = r0 + row;
    if (rr >= c.rows) continue;
    float o = kNoOffset, l = 0.0f;
#pragma unroll
    for (int w = 0; w < W; ++w) {
      const float v = ol[w * ROWS + row].x;
      o = v != v || v > o ? v : o;
    }
    v4f y = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int w = 0; w < W; ++w) {
      const float2 u = ol[w * ROWS + row];
      const float f = __builtin_amdgcn_exp2f(u.x - o);
      l = __builtin_fmaf(u.y, f, l);
      const v4f v = *reinterpret_cast<const v4f *>(lds + (w * ROWS + row) * kLd + d);
#pragma unroll
      for (int r = 0; r < 4; ++r) y[r] = __builtin_fmaf(v[r], f, y[r]);
    }
    const int ti = rr / a.gr;
    const size_t yr = (size_t)(c.start + ti) * a.Hq + c.h * a.gr + (rr - ti * a.gr);
    if (a.splits == 1) {
      store_y(a, yr * D + d, y * inverse(l));
      if (a.lse && d == 0) a.lse[yr] = lse_of(o, l);
    } else {
      *reinterpret_cast<v4f *>(a.part + (yr * a.splits + c.part) * D + d) = y;
      if (d == 0) a.part_ol[yr * a.splits + c.part] = make_float2(o, l);
    }
  }
}

template <int D, int MT, int W, bool SPLIT, bool ROWS>
__global__ __launch_bounds__(64 * W, D == 64 ? (MT == 2 ? 3 : 4) : MT == 2 || D == 256 ? 2 : 3) void k_kv_attention(KvAttnArgs a) {
  constexpr int G = D / kKvGroup, kRows = 16 * MT * (ROWS ? W : 1), kLd = D + 4;
  extern __shared__ float lds[];
  __shared__ float2 base_of[W][16 * MT];
  const int lane = threadIdx.x & 63, q = lane >> 4, col = lane & 15;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  float2 *base = base_of[wave];
  if (lane < 16 * MT) base[lane] = make_float2(0.0f, 0.0f);
  // the last rows see the most: first
  const Place c = place_of(a, ROWS ? 1 : a.splits, (int)(gridDim.x - 1 - blockIdx.x), kRows);
  const int r0 = c.block * kRows + (ROWS ? wave * 16 * MT : 0);
  if (r0 >= c.rows) return;
  const int r1 = min(r0 + 16 * MT, c.rows);
  int first, last;
  tiles_of_rows(a, r0, r1, c.p0, c.len, first, last);
  if (!ROWS) {
    const int per = tiles_of_part(first, last, a.splits);
    first += c.part * per;
    if (c.part > 0 && first >= last) return;
    last = min(last, first + per);
  }
  // this lane's queries
  v4u Q[MT][D / 32];
  float qs[MT][G], c2[MT];
  int lo[MT], hi[MT];
  size_t at[MT];                                // row of Y (heads counted)
  bool live[MT];
#pragma unroll
  for (int m = 0; m < MT; ++m) {
    const int row = r0 + 16 * m + col;
    live[m] = row < c.rows;
    const int i = min(row, c.rows - 1) / a.gr, head = c.h * a.gr + (live[m] ? row - i * a.gr : 0);
    const Seen s = seen_by(a, i, c.p0, c.len);
    lo[m] = s.lo;
    hi[m] = s.hi;
    at[m] = (size_t)(c.start + i) * a.Hq + head;
    const uint16_t *src = a.Q + (size_t)(c.start + i) * a.q_stride + (size_t)head * D + 8 * q;
    uint32_t top = 0;
#pragma unroll
    for (int x = 0; x < D / 32; ++x) {
      Q[m][x] = live[m] ? *reinterpret_cast<const v4u *>(src + 32 * x) : (v4u){0u, 0u, 0u, 0u};
      top = larger8(top, Q[m][x]);
    }
    const float by = row_power(max_over<16, 32>(magnitude(top, a.dtype)), a.scale2, c2[m]);
#pragma unroll
    for (int x = 0; x < D / 32; ++x) Q[m][x] = scaled8(Q[m][x], a.dtype, by);
    const v4u ones = {kOnes, kOnes, kOnes, kOnes};
#pragma unroll
    for (int g = 0; g < G; ++g) {
      v4f d = mfma16(ones, Q[m][2 * g], (v4f){0.0f, 0.0f, 0.0f, 0.0f});
      d = mfma16(ones, Q[m][2 * g + 1], d);
      qs[m][g] = d[0] * (1.0f / Unit<true>::low);
    }
  }
  // tokens that every row of the wave sees
  const int full_lo = seen_by(a, (r1 - 1) / a.gr, c.p0, c.len).lo, full_hi = seen_by(a, r0 / a.gr, c.p0, c.len).hi;
  Sums<D, MT> s;
#pragma unroll
  for (int m = 0; m < MT; ++m) {
    s.o[m] = kNoOffset;
    s.l[m] = 0.0f;
#pragma unroll
    for (int x = 0; x < D / 16; ++x) s.acc[m][x] = (v4f){0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int g = 0; g < G; ++g) s.zero[m][g] = (v4f){0.0f, 0.0f, 0.0f, 0.0f};
  }
  // A side's registers are loaded again as soon as they have been used: the next
  // keys travel while this tile's weights and values are worked on, the next
  // values while its scores are.  A tile on no page reads page 0 and is hidden.
  constexpr int kStep = ROWS ? 1 : W;
  int tile = first + (ROWS ? 0 : wave);
  if (tile < last) {
    Side<D> tk, tv;
    const uint8_t *p = kv_tile_at(a.c, c.b, c.h, tile);
    bool there = p != nullptr;
    if (!there) p = a.c.cache;
    load_side<D, false>(p, lane, tk);
    load_side<D, true>(p, lane, tv);
    for (;;) {
      const int next = tile + kStep;
      const uint8_t *pn = kv_tile_at(a.c, c.b, c.h, min(next, last - 1));
      const bool there_n = pn != nullptr;
      if (!there_n) pn = a.c.cache;
      float e[MT][8];
      scores<D, MT>(tk, Q, qs, e);
      __builtin_amdgcn_sched_barrier(0);
      load_side<D, false>(pn, lane, tk);
      __builtin_amdgcn_sched_barrier(0);
      const int t0 = tile * kKvTile;
      const bool masked = t0 < full_lo || t0 + kKvTile > full_hi || !there;
      if (masked) {
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const int tok = t0 + 16 * (i >> 2) + 4 * q + (i & 3);
            if (tok < lo[m] || tok >= hi[m] || !there) e[m][i] = kHidden;
          }
      }
      v4u w[MT][G], w2[MT][G];
      weigh<D, MT, SPLIT>(e, tv.s, c2, masked, base, s, w, w2);
      values<D, MT, SPLIT>(tv, w, w2, s);
      if (next >= last) break;
      __builtin_amdgcn_sched_barrier(0);
      load_side<D, true>(pn, lane, tv);
      __builtin_amdgcn_sched_barrier(0);
      tile = next;
      there = there_n;
    }
  }
#pragma unroll
  for (int m = 0; m < MT; ++m) {
    s.l[m] = sum_over<16, 32>(s.l[m]);
#pragma unroll
    for (int x = 0; x < D / 16; ++x) {
      const float up = x & 1 ? Unit<SPLIT>::high : Unit<SPLIT>::low;
      s.acc[m][x] = s.acc[m][x] * up - s.zero[m][x / 4] * Unit<SPLIT>::low;
    }
    const float2 b = base[16 * m + col];
    if (__any(b.x != 0.0f)) {             // such rows leave with b as their offset: it would swallow o
      const float back = b.x != 0.0f ? __builtin_amdgcn_exp2f(b.y) : 1.0f;
      s.l[m] *= back;
      s.o[m] = b.x != 0.0f ? b.x : s.o[m];
#pragma unroll
      for (int x = 0; x < D / 16; ++x) s.acc[m][x] *= back;
    }
  }
  if (ROWS) {
#pragma unroll
    for (int m = 0; m < MT; ++m) {
      if (!live[m]) continue;
      const float inv = inverse(s.l[m]);
#pragma unroll
      for (int x = 0; x < D / 16; ++x) store_y(a, at[m] * D + 16 * x + 4 * q, s.acc[m][x] * inv);
      if (a.lse && q == 0) a.lse[at[m]] = lse_of(s.o[m], s.l[m]);
    }
    return;
  }
  float2 *ol = reinterpret_cast<float2 *>(lds + W * 16 * MT * kLd);
#pragma unroll
  for (int m = 0; m < MT; ++m) {
    const int row = wave * 16 * MT + 16 * m + col;
#pragma unroll
    for (int x = 0; x < D / 16; ++x) *reinterpret_cast<v4f *>(lds + row * kLd + 16 * x + 4 * q) = s.acc[m][x];
    if (q == 0) ol[row] = make_float2(s.o[m], s.l[m]);
  }
  __syncthreads();
  join_waves<D, 16 * MT, W>(a, c, r0, lds, ol);
}

// ------------------------------------------------------------------ 4 x 4
// A lane's half u = lane / 32 has groups 2 j + u (j < kSets), or, where there is one
// group, the second of two tiles.  As a token t = lane % 32 (= 4 c + r): its
// group's channels, two dwords of each lane slot t % 16 + 16 q; the scales and zeros
// of the four tokens 4 c ...  As channels: 32 p + lane % 16 and 16 more, p = 2 g +
// (lane / 16) % 2, the tokens 16 a + 4 q .. as dword 2 p + a of slot lane % 16 + 16 q.
template <int D>
struct Side4 {
  static constexpr int kSets = D <= 128 ? 1 : D / 128;
  v2u code[kSets][4], s[kSets];
  uint32_t z[kSets];
};

// A lane's offsets within a tile: codes of K and V, scales, zeros of K (those of V
// lie a constant further).
struct Lane4 { uint32_t k, v, s, z; };
template <int D>
__device__ __forceinline__ Lane4 lane4(int lane, int j) {
  constexpr int G = D / kKvGroup;
  const uint32_t g = G == 1 ? 0 : 2 * j + (lane >> 5), c = (lane >> 2) & 7;
  const uint32_t xk = ((lane >> 4) & 1) * (D / 32) + 2 * g, xv = 2 * (2 * g + ((lane >> 4) & 1)), slot = (lane & 15) * 16;
  return {(xk >> 2) * 1024 + (xk & 3) * 4 + slot, 16 * D + (xv >> 2) * 1024 + (xv & 3) * 4 + slot,
          32 * D + g * 64 + (c & 3) * 16 + (c >> 2) * 8, 32 * D + 128 * G + ((c & 3) * G + g) * 8 + (c >> 2) * 4};
}

template <int D, bool V>
__device__ __forceinline__ void load_side4(const uint8_t *p, const Lane4 (&o)[Side4<D>::kSets], Side4<D> &t) {
  constexpr int G = D / kKvGroup;
#pragma unroll
  for (int j = 0; j < Side4<D>::kSets; ++j) {
#pragma unroll
    for (int q = 0; q < 4; ++q) t.code[j][q] = *reinterpret_cast<const v2u *>(p + (V ? o[j].v : o[j].k) + q * 256);
    t.s[j] = *reinterpret_cast<const v2u *>(p + o[j].s + (V ? 64 * G : 0));
    t.z[j] = *reinterpret_cast<const uint32_t *>(p + o[j].z + (V ? 32 * G : 0));
  }
}

// The zeros of all 32 tokens, as a lane of channels meets them: [q][a].
template <int D>
__device__ __forceinline__ void load_zeros4(const uint8_t *p, int lane, v2u (&z)[Side4<D>::kSets][4]) {
  constexpr int G = D / kKvGroup;
#pragma unroll
  for (int j = 0; j < Side4<D>::kSets; ++j) {
    const uint32_t at = 32 * D + 160 * G + (G == 1 ? 0 : 2 * j + (lane >> 5)) * 8;
#pragma unroll
    for (int q = 0; q < 4; ++q) z[j][q] = *reinterpret_cast<const v2u *>(p + at + q * G * 8);
  }
}

// Sums of a wave: R sets of four rows; lane's row of each is lane % 4 in o, l, zero
// (and there its tokens only), the four of acc are rows.
template <int D, int R>
struct Sums4 {
  static constexpr int kSets = Side4<D>::kSets;
  v4f low[R][kSets], high[R][kSets];   // channels 32 p + lane % 16, and 16 more, under the codes' Unit
  float zero[R][kSets], o[R], l[R];
};

template <int I>
__device__ __forceinline__ float quad(float v) {   // of lane I of the four
  return dpp_f32<I * 0x55>(v);
}

template <int D, int R, bool SPLIT, int... C>
__device__ __forceinline__ void values4(const Side4<D> &t, const v2u (&w)[R][Side4<D>::kSets],
                                        const v2u (&w2)[R][Side4<D>::kSets],
                                        const v2u (&z)[Side4<D>::kSets][4], Sums4<D, R> &s,
                                        std::integer_sequence<int, C...>) {
  auto chunk = [&](auto ic) __attribute__((always_inline)) {
    constexpr int c = decltype(ic)::value;     // tokens 4 c ..: a = c / 4, q = c % 4
#pragma unroll
    for (int j = 0; j < Side4<D>::kSets; ++j) {
      v2u lo = low_codes<SPLIT>(t.code[j][c & 3][c >> 2]), hi = high_codes<SPLIT>(t.code[j][c & 3][c >> 2]);
      if (SPLIT) {
        const v2u x = low_codes<SPLIT>(z[j][c & 3][c >> 2]);
        lo = (v2u){minus_h(lo[0], x[0]), minus_h(lo[1], x[1])};
        hi = (v2u){minus_h(hi[0], x[0]), minus_h(hi[1], x[1])};
      }
#pragma unroll
      for (int r = 0; r < R; ++r) {
        s.low[r][j] = mfma4<c>(w[r][j], lo, s.low[r][j]);
        s.high[r][j] = mfma4<c>(w[r][j], hi, s.high[r][j]);
        if (SPLIT) {
          s.low[r][j] = mfma4<c>(w2[r][j], lo, s.low[r][j]);
          s.high[r][j] = mfma4<c>(w2[r][j], hi, s.high[r][j]);
        }
      }
    }
  };
  (chunk(std::integral_constant<int, C>{}), ...);
}

template <int D, int R, int W, bool SPLIT>
__global__ __launch_bounds__(64 * W, R == 1 && D < 256 ? 4 : 2) void k_kv_attention4(KvAttnArgs a) {
  constexpr int G = D / kKvGroup, kSets = Side4<D>::kSets, kTiles = G == 1 ? 2 : 1, kRows = 4 * R, kLd = D + 4;
  __shared__ float lds[W * kRows * kLd];
  __shared__ float2 ol[W * kRows];
  __shared__ float2 base_of[W][kRows];
  const int lane = threadIdx.x & 63, half = lane >> 5, c4 = (lane >> 2) & 7, j4 = lane & 3;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  float2 *base = base_of[wave];         // as in weigh
  if (lane < kRows) base[lane] = make_float2(0.0f, 0.0f);
  const Place c = place_of(a, a.splits, blockIdx.x, kRows);
  const int r0 = c.block * kRows;
  if (r0 >= c.rows) return;
  const int r1 = min(r0 + kRows, c.rows);
  int first, last;
  tiles_of_rows(a, r0, r1, c.p0, c.len, first, last);
  const int per = tiles_of_part(first, last, a.splits);
  first += c.part * per;
  if (c.part > 0 && first >= last) return;
  last = min(last, first + per);

  // the first tiles' pages, keys and values are on their way before the queries are
  int tile = first + wave * kTiles;
  const uint8_t *p = a.c.cache;
  bool there = false;
  Side4<D> tk, tv;
  auto locate = [&](int t, const uint8_t *&at, bool &is) __attribute__((always_inline)) {
    const uint8_t *x = t < last ? kv_tile_at(a.c, c.b, c.h, t) : nullptr;
    if (kTiles == 2) {
      const uint8_t *y = t + 1 < last ? kv_tile_at(a.c, c.b, c.h, t + 1) : nullptr;
      x = half ? y : x;
    }
    is = x != nullptr;
    at = is ? x : a.c.cache;
  };
  locate(tile, p, there);
  Lane4 at4[kSets];
#pragma unroll
  for (int j = 0; j < kSets; ++j) at4[j] = lane4<D>(lane, j);
  load_side4<D, false>(p, at4, tk);
  load_side4<D, true>(p, at4, tv);
  v2u zeros[kSets][4];
  if (SPLIT) load_zeros4<D>(p, lane, zeros);

  // Q: dims 64 g + 32 i + 8 q .. of row j4, eight at a time
  v4u Q[R][kSets][8];
  float qs[R][kSets], c2[R];
  int lo[R], hi[R];
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const int row = r0 + 4 * r + j4, i = min(row, c.rows - 1) / a.gr;
    const bool live = row < c.rows;
    const int head = c.h * a.gr + (live ? row - i * a.gr : 0);
    const Seen s = seen_by(a, i, c.p0, c.len);
    lo[r] = s.lo;
    hi[r] = s.hi;
    const uint16_t *src = a.Q + (size_t)(c.start + i) * a.q_stride + (size_t)head * D;
    uint32_t most = 0;
#pragma unroll
    for (int j = 0; j < kSets; ++j)
#pragma unroll
      for (int n = 0; n < 8; ++n) {
        const int g = G == 1 ? 0 : 2 * j + half;
        Q[r][j][n] = live ? *reinterpret_cast<const v4u *>(src + 64 * g + 32 * (n & 1) + 8 * (n >> 1)) : (v4u){0u, 0u, 0u, 0u};
        most = larger8(most, Q[r][j][n]);
      }
    float top = magnitude(most, a.dtype);
    if (G > 1) top = max_over<32, 32>(top);
    const float by = row_power(top, a.scale2, c2[r]);
#pragma unroll
    for (int j = 0; j < kSets; ++j) {
      v4f d = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int n = 0; n < 8; ++n) {
        Q[r][j][n] = scaled8(Q[r][j][n], a.dtype, by);
        d = mfma4<-1>((v2u){kOnes, kOnes}, (v2u){Q[r][j][n][0], Q[r][j][n][1]}, d);
        d = mfma4<-1>((v2u){kOnes, kOnes}, (v2u){Q[r][j][n][2], Q[r][j][n][3]}, d);
      }
      qs[r][j] = d[0] * (1.0f / Unit<true>::low);
    }
  }
  const int full_lo = seen_by(a, (r1 - 1) / a.gr, c.p0, c.len).lo, full_hi = seen_by(a, r0 / a.gr, c.p0, c.len).hi;
  Sums4<D, R> s;
#pragma unroll
  for (int r = 0; r < R; ++r) {
    s.o[r] = kNoOffset;
    s.l[r] = 0.0f;
#pragma unroll
    for (int j = 0; j < kSets; ++j) {
      s.low[r][j] = s.high[r][j] = (v4f){0.0f, 0.0f, 0.0f, 0.0f};
      s.zero[r][j] = 0.0f;
    }
  }

  for (; tile < last;) {
    const int next = tile + W * kTiles;
    const uint8_t *pn;
    bool there_n;
    locate(min(next, last - 1), pn, there_n);
    // scores of tokens 4 c4 + i, this half's groups, then all
    float e[R][4];
#pragma unroll
    for (int j = 0; j < kSets; ++j) {
      v4f d[R][2];
#pragma unroll
      for (int r = 0; r < R; ++r) d[r][0] = d[r][1] = (v4f){0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int n = 0; n < 8; ++n) {
        const v2u lo2 = low_codes<true>(tk.code[j][n >> 1][n & 1]), hi2 = high_codes<true>(tk.code[j][n >> 1][n & 1]);
#pragma unroll
        for (int r = 0; r < R; ++r) {
          d[r][0] = mfma4<-1>(lo2, (v2u){Q[r][j][n][0], Q[r][j][n][1]}, d[r][0]);
          d[r][1] = mfma4<-1>(hi2, (v2u){Q[r][j][n][2], Q[r][j][n][3]}, d[r][1]);
        }
      }
      const uint32_t zw = zeros_of(tk.z[j]);
#pragma unroll
      for (int r = 0; r < R; ++r)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float u = __builtin_fmaf(-zero_of(zw, i), qs[r][j], d[r][0][i] + d[r][1][i]);
          e[r][i] = __builtin_fmaf(u, half_of(tk.s[j], i), j ? e[r][i] : 0.0f);
        }
    }
    __builtin_amdgcn_sched_barrier(0);
    load_side4<D, false>(pn, at4, tk);
    __builtin_amdgcn_sched_barrier(0);
    if (G > 1) {
#pragma unroll
      for (int r = 0; r < R; ++r)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint32_t x = __float_as_uint(e[r][i]);
          const auto y = __builtin_amdgcn_permlane32_swap(x, x, false, false);
          e[r][i] = __uint_as_float(y[0]) + __uint_as_float(y[1]);
        }
    }
    const int t0 = tile * kKvTile;
    const bool masked = t0 < full_lo || t0 + kTiles * kKvTile > full_hi || !__all(there);
    if (masked) {
      const int tok0 = t0 + (kTiles == 2 ? 32 * half : 0) + 4 * c4;
#pragma unroll
      for (int r = 0; r < R; ++r)
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (tok0 + i < lo[r] || tok0 + i >= hi[r] || !there) e[r][i] = kHidden;
    }
    // weights
    v2u w[R][kSets], w2[R][kSets];
    float pw[R][4], ps[R][kSets][4], top[R], topp[R];
    bool any_base = false;
    auto form = [&](auto again) __attribute__((always_inline)) {
      bool moved = false;
#pragma unroll
      for (int r = 0; r < R; ++r) {
        top[r] = topp[r] = 0.0f;
#pragma unroll
        for (int i = 0; i < 4; ++i) pw[r][i] = __builtin_fmaf(e[r][i], c2[r], -s.o[r]);
        if (decltype(again)::value && any_base) {
          const float2 b = base[4 * r + (lane_here() & 3)];
#pragma unroll
          for (int i = 0; i < 4; ++i) pw[r][i] = b.x != 0.0f ? (e[r][i] * c2[r] - b.x) - b.y : pw[r][i];
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          pw[r][i] = __builtin_amdgcn_exp2f(pw[r][i]);
          topp[r] = fmaxf(topp[r], pw[r][i]);
        }
#pragma unroll
        for (int j = 0; j < kSets; ++j)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            ps[r][j][i] = __builtin_fmaf(pw[r][i], half_of(tv.s[j], i), 0.0f);
            // a hidden token's scale may be anything, NaN among it
            if (masked) ps[r][j][i] = e[r][i] == kHidden ? 0.0f : ps[r][j][i];
            top[r] = fmaxf(top[r], ps[r][j][i]);
          }
        moved |= top[r] > kMaxPs || topp[r] > kMaxP;
      }
      return __any(moved) != 0;
    };
    if (__builtin_expect(form(std::false_type{}), 0)) {
#pragma unroll
      for (int r = 0; r < R; ++r) {
        const float mine = top[r] > kMaxPs || topp[r] > kMaxP ? 1.0f : 0.0f;
        const bool move = max_over<4, 32>(mine) > 0.0f;
        float2 &own = base[4 * r + (lane_here() & 3)];
        const float2 had = own;
        float most = kHidden;
#pragma unroll
        for (int j = 0; j < kSets; ++j)
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (!masked || e[r][i] != kHidden)
              most = fmaxf(most, __builtin_fmaf(e[r][i], c2[r], __builtin_amdgcn_logf(fmaxf(half_of(tv.s[j], i), kTiny))));
        most = max_over<4, 32>(most);
        float o = move ? __builtin_ceilf(most) - kTop : s.o[r], al = move ? __builtin_amdgcn_exp2f(s.o[r] - o) : 1.0f;
        const bool based = move && (had.x != 0.0f || fabsf(most) >= kFar);
        if (__any(based)) {
          any_base = true;
          float high = kHidden;
#pragma unroll
          for (int i = 0; i < 4; ++i) high = fmaxf(high, e[r][i] * c2[r]);
          high = max_over<4, 32>(high);
          const float b = base_with(had, high);
          float near = kHidden;
#pragma unroll
          for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < kSets; ++j)
              if (!masked || e[r][i] != kHidden)
                near = fmaxf(near, (e[r][i] * c2[r] - b) + __builtin_amdgcn_logf(fmaxf(half_of(tv.s[j], i), kTiny)));
          near = rebase(max_over<4, 32>(near), b, had);
          if (based) {
            al = __builtin_amdgcn_exp2f((had.x - b) + ((had.x != 0.0f ? had.y : s.o[r]) - near));
            o = kNoOffset;
            own = make_float2(b, near);
          }
        }
        s.o[r] = o;
        s.l[r] *= al;
        const v4f rows = {quad<0>(al), quad<1>(al), quad<2>(al), quad<3>(al)};
#pragma unroll
        for (int j = 0; j < kSets; ++j) {
          s.zero[r][j] *= al;
          s.low[r][j] *= rows;
          s.high[r][j] *= rows;
        }
      }
      form(std::true_type{});
    }
#pragma unroll
    for (int r = 0; r < R; ++r) {
#pragma unroll
      for (int i = 0; i < 4; ++i) s.l[r] += pw[r][i];
#pragma unroll
      for (int j = 0; j < kSets; ++j) {
        const uint32_t zw = SPLIT ? 0 : zeros_of(tv.z[j]);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const uint32_t x = pack_h(ps[r][j][2 * i], ps[r][j][2 * i + 1]);
          w[r][j][i] = x;
          const v2h h = __builtin_bit_cast(v2h, x);
          if (SPLIT) w2[r][j][i] = pack_h(ps[r][j][2 * i] - (float)h[0], ps[r][j][2 * i + 1] - (float)h[1]);
          // the zeros' share of what the product will hold: of the rounded weights
#pragma unroll
          for (int y = 0; y < 2; ++y)
            if (!SPLIT) s.zero[r][j] = __builtin_fmaf((float)h[y], zero_of(zw, 2 * i + y), s.zero[r][j]);
        }
      }
    }
    values4<D, R, SPLIT>(tv, w, w2, zeros, s, std::make_integer_sequence<int, 8>{});
    __builtin_amdgcn_sched_barrier(0);
    load_side4<D, true>(pn, at4, tv);
    if (SPLIT) load_zeros4<D>(pn, lane, zeros);
    __builtin_amdgcn_sched_barrier(0);
    tile = next;
    there = there_n;
  }
  // rows of channels, less the zeros' share; the sums over tokens of o, l are a row's
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const float l = G == 1 ? sum_over<4, 32>(s.l[r]) : sum_over<4, 16>(s.l[r]);
    const float2 b = base[4 * r + j4];
    const float back = b.x != 0.0f ? __builtin_amdgcn_exp2f(b.y) : 1.0f;
    if (lane < 4) ol[wave * kRows + 4 * r + lane] = make_float2(b.x != 0.0f ? b.x : s.o[r], l * back);
    const v4f backs = {quad<0>(back), quad<1>(back), quad<2>(back), quad<3>(back)};
#pragma unroll
    for (int j = 0; j < kSets; ++j) {
      const float z = sum_over<4, 16>(s.zero[r][j]);
      const v4f zr = {quad<0>(z), quad<1>(z), quad<2>(z), quad<3>(z)};
      v4f y0 = (s.low[r][j] * Unit<SPLIT>::low - zr) * backs, y1 = (s.high[r][j] * Unit<SPLIT>::high - zr) * backs;
      if (G == 1) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          y0[i] = sum_over<32, 32>(y0[i]);
          y1[i] = sum_over<32, 32>(y1[i]);
        }
      }
      const int g = G == 1 ? 0 : 2 * j + half, ch = 32 * (2 * g + ((lane >> 4) & 1)) + (lane & 15);
      if (G > 1 || half == 0) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          lds[(wave * kRows + 4 * r + i) * kLd + ch] = y0[i];
          lds[(wave * kRows + 4 * r + i) * kLd + ch + 16] = y1[i];
        }
      }
    }
  }
  __syncthreads();
  join_waves<D, kRows, W>(a, c, r0, lds, ol);
}

// The parts of a row: groups of D / 4 lanes take every kGroups-th part, and their
// sums meet in order.
template <int D>
__global__ __launch_bounds__(256) void k_kv_join(KvAttnArgs a, int block_rows) {
  constexpr int kLanes = D / 4, kGroups = 256 / kLanes;
  __shared__ float l_of[kGroups];
  __shared__ v4f y_of[kGroups][kLanes];
  const int tid = threadIdx.x, lane = tid % kLanes, grp = tid / kLanes, r = blockIdx.x, h = blockIdx.y, b = blockIdx.z;
  int start, n;
  kv_rows(a.c, b, start, n);
  const int rows = min(n, a.c.max_tokens) * a.gr, r0 = r / block_rows * block_rows;
  if (r >= rows) return;
  const int len = kv_len(a.c, b), p0 = max(a.c.lens[b], 0) - n;
  int first, last;
  tiles_of_rows(a, r0, min(r0 + block_rows, rows), p0, len, first, last);
  const int per = tiles_of_part(first, last, a.splits), parts = max(1, (last - first + per - 1) / per);
  const int ti = r / a.gr;
  const size_t yr = (size_t)(start + ti) * a.Hq + h * a.gr + (r - ti * a.gr);
  const float2 *ol = a.part_ol + yr * a.splits;
  const float *part = a.part + yr * a.splits * D + lane * 4;
  // splits <= kMaxParts: this group's parts, all on their way at once
  constexpr int kMine = kMaxParts / kGroups;
  v4f v[kMine];
  float2 u[kMine];
#pragma unroll
  for (int i = 0; i < kMine; ++i) {
    const int w = grp + i * kGroups;
    if (w >= parts) continue;
    u[i] = ol[w];
    v[i] = *reinterpret_cast<const v4f *>(part + (size_t)w * D);
  }
  float o = kNoOffset, l = 0.0f;
  for (int w = 0; w < parts; w += 64) {       // the largest offset, NaN above all
    const float x = ol[min(w + (tid & 63), parts - 1)].x;
    o = x != x || x > o ? x : o;
  }
#pragma unroll
  for (int m = 32; m >= 1; m >>= 1) {
    const float x = __shfl_xor(o, m);
    o = x != x || x > o ? x : o;
  }
  v4f y = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
  for (int i = 0; i < kMine; ++i) {
    if (grp + i * kGroups >= parts) continue;
    const float f = __builtin_amdgcn_exp2f(u[i].x - o);
    l = __builtin_fmaf(u[i].y, f, l);
#pragma unroll
    for (int e = 0; e < 4; ++e) y[e] = __builtin_fmaf(v[i][e], f, y[e]);
  }
  y_of[grp][lane] = y;
  if (lane == 0) l_of[grp] = l;
  __syncthreads();
  if (grp != 0) return;
#pragma unroll
  for (int g = 1; g < kGroups; ++g) {
    y += y_of[g][lane];
    l += l_of[g];
  }
  store_y(a, yr * D + lane * 4, y * inverse(l));
  if (a.lse && lane == 0) a.lse[yr] = lse_of(o, l);
}

template <typename Kernel>
hipError_t go(Kernel kernel, dim3 grid, int threads, size_t lds, const KvAttnArgs &a, hipStream_t s) {
  if (lds > 64 * 1024) {
    const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void *>(kernel),
                                             hipFuncAttributeMaxDynamicSharedMemorySize, (int)lds);
    if (e != hipSuccess) return e;
  }
  hipLaunchKernelGGL(kernel, grid, dim3((unsigned)threads), lds, s, a);
  return hipGetLastError();
}

constexpr int kWaves = 4;

template <int D, int MT, bool ROWS>
hipError_t launch16(const KvAttnArgs &a, dim3 grid, hipStream_t s) {
  const size_t lds = ROWS ? 0 : (size_t)kWaves * 16 * MT * ((D + 4) * sizeof(float) + sizeof(float2));
  return a.y_dtype != kBf16 ? go(k_kv_attention<D, MT, kWaves, true, ROWS>, grid, 64 * kWaves, lds, a, s)
                           : go(k_kv_attention<D, MT, kWaves, false, ROWS>, grid, 64 * kWaves, lds, a, s);
}

template <int D, int R, int W>
hipError_t launch4(const KvAttnArgs &a, dim3 grid, hipStream_t s) {
  return a.y_dtype != kBf16 ? go(k_kv_attention4<D, R, W, true>, grid, 64 * W, 0, a, s)
                           : go(k_kv_attention4<D, R, W, false>, grid, 64 * W, 0, a, s);
}

template <int D>
hipError_t launch_d(const KvAttnArgs &a, const KvAttnPlan &p, hipStream_t s) {
  const KvBlocks blocks = plan_kv_attention_blocks(a.c, a.gr, p);
  const dim3 grid = blocks.searched ? dim3((unsigned)blocks.total, (unsigned)a.c.H)
                                    : dim3((unsigned)blocks.each, (unsigned)a.c.H, (unsigned)(a.c.B * p.splits));
  hipError_t e;
  constexpr int kMt = D == 256 ? 1 : 2;      // two row tiles of 256 channels would not fit the registers
  if (p.by_rows) return launch16<D, kMt, true>(a, grid, s);
  if (p.rows == 4) e = p.waves == 8 ? launch4<D, 1, 8>(a, grid, s) : launch4<D, 1, 4>(a, grid, s);
  else if (p.rows == 16) e = launch16<D, 1, false>(a, grid, s);
  else if constexpr (D == 256) e = hipErrorInvalidValue;      // the plan has no others for these heads
  else e = p.rows == 8 ? launch4<D, 2, kWaves>(a, grid, s) : launch16<D, kMt, false>(a, grid, s);
  if (e == hipSuccess && p.splits > 1) {
    hipLaunchKernelGGL((k_kv_join<D>), dim3((unsigned)(a.c.max_tokens * a.gr), (unsigned)a.c.H, (unsigned)a.c.B), dim3(256),
                       0, s, a, p.rows);
    e = hipGetLastError();
  }
  return e;
}

}  // namespace

KvAttnPlan plan_kv_attention(int T, int Hq, int H, int D, int B, int max_tokens, int64_t capacity) {
  KvAttnPlan p;
  const long long rows = (long long)max_tokens * (Hq / H);
  p.by_rows = rows >= 64;
  if (p.by_rows) {
    p.rows = kWaves * (D == 256 ? 16 : 32);
    return p;
  }
  p.rows = rows <= 4 ? 4 : rows <= 8 && D < 256 ? 8 : rows <= 16 || D == 256 ? 16 : 32;
  const long long wgs = (rows + p.rows - 1) / p.rows * H * B;
  const long long most = std::max<long long>(1, (capacity + kMinTiles * kKvTile - 1) / (kMinTiles * kKvTile));
  p.splits = (int)std::min<long long>({std::max<long long>(1, 512 / wgs), most, kMaxParts});
  if (p.rows == 4 && wgs * p.splits <= 256) p.waves = 8;
  if (p.splits > 1) {
    const size_t parts = (size_t)T * Hq * p.splits;
    p.part_off = align_up(parts * sizeof(float2), 256);
    p.total = p.part_off + parts * D * sizeof(float);
  }
  return p;
}

KvBlocks plan_kv_attention_blocks(const KvCache &c, int gr, const KvAttnPlan &p) {
  const long long each = ((long long)c.max_tokens * gr + p.rows - 1) / p.rows;
  return p.by_rows ? kv_blocks(c, each, gr, p.rows, 1) : KvBlocks{0, each, each * c.B};
}

hipError_t launch_kv_attention(KvAttnArgs a, const KvAttnPlan &p, hipStream_t s) {
  a.c.searched = plan_kv_attention_blocks(a.c, a.gr, p).searched;
  switch (a.c.D) {
    case 64: return launch_d<64>(a, p, s);
    case 128: return launch_d<128>(a, p, s);
    case 256: return launch_d<256>(a, p, s);
    default: return hipErrorInvalidValue;
  }
}

}  // namespace hsq
