// kv_attention.hip -- attention over the paged 4-bit cache of kv_cache.hip.
//
//   e[i,t] = scale q_i . k_t,   y_i = sum_t exp(e[i,t]) v_t / sum_t exp(e[i,t])
//
// over the tokens t that query i sees.  Keys and values are s (n - z) with one
// scale s and zero z per token and group g of 64 channels, so the codes enter the
// matrix products as small integers (exact in 16 bits) and the scales stay with
// the (query, token) pairs in fp32:
//
//   q . k_t        = sum_g s_g (sum_d q_d (16 + n_d) - (16 + z_g) sum_d q_d)
//   sum_t p_t v_t  = sum_t (p_t s_g) (n_d - z_g)
//
// 16 + n is a nibble under a constant exponent, two operations a pair; the second
// product runs in fp16, where one packed subtraction a pair makes it n - z.  p s is
// the only value that is rounded: to fp16 (11 bits), or, where the result is fp32,
// to the sum of two.  Its range is kept by the row's offset o, a whole number:
// p = 2^(e log2(e) - o) with o such that p s stays below 2^15; o moves, and the
// sums with it by an exact power of two, only when a tile would exceed that (seven
// doublings above the tile that set it), so the running maximum of the softmax
// costs one comparison a tile.
//
// Both products are formed transposed (tokens x queries, channels x queries): a
// lane then holds tokens 16 a + 4 q + r of its query in the first product's result
// and needs the same ones for the second's operand, so p never leaves the
// registers, and the loop has no LDS and no barrier.
#include "hsq_internal.h"

#include <algorithm>

namespace hsq {

namespace {

typedef __bf16 v8bf __attribute__((ext_vector_type(8)));
typedef _Float16 v8h __attribute__((ext_vector_type(8)));

constexpr float kNoOffset = -1e30f;      // of a row that has seen nothing
constexpr float kTop = 8.0f;             // p s of the tile that sets the offset stays below 2^kTop
constexpr float kMaxPs = 32768.0f;       // what moves the offset
constexpr float kMaxP = 1099511627776.0f;   // 2^40: the same for tokens of scale 0
constexpr float kLn2 = 0.6931471805599453f;

template <int DT>
__device__ __forceinline__ v4f mfma16(v4u a, v4u b, v4f c) {
  if constexpr (DT == kBf16)
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(v8bf, a), __builtin_bit_cast(v8bf, b), c, 0, 0, 0);
  else
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(v8h, a), __builtin_bit_cast(v8h, b), c, 0, 0, 0);
}

// The eight codes of a dword as 16 + n: the low nibbles of bytes 0, 2 | 1, 3, then the high ones.
template <int DT>
__device__ __forceinline__ v4u expand(uint32_t w) {
  if constexpr (DT == kBf16) {
    constexpr uint32_t m = 0x00780078u, k = 0x41804180u;
    return (v4u){(w << 3 & m) | k, (w >> 5 & m) | k, (w >> 1 & m) | k, (w >> 9 & m) | k};
  } else {
    constexpr uint32_t m = 0x03C003C0u, k = 0x4C004C00u;
    return (v4u){(w << 6 & m) | k, (w >> 2 & m) | k, (w << 2 & m) | k, (w >> 6 & m) | k};
  }
}

__device__ __forceinline__ uint32_t pack_h(float a, float b) {
  v2h h = {(_Float16)a, (_Float16)b};
  return __builtin_bit_cast(uint32_t, h);
}

// (16 + n) - (16 + z), two at a time
__device__ __forceinline__ uint32_t minus_h(uint32_t a, uint32_t b) {
  return __builtin_bit_cast(uint32_t, __builtin_bit_cast(v2h, a) - __builtin_bit_cast(v2h, b));
}

__device__ __forceinline__ float over_q(float v, bool sum) {   // lanes of one column: 16 and 32 apart
  const float a = __shfl_xor(v, 16);
  v = sum ? v + a : fmaxf(v, a);
  const float b = __shfl_xor(v, 32);
  return sum ? v + b : fmaxf(v, b);
}

template <int D>
struct TileRegs {
  static constexpr int G = D / kKvGroup;
  v4u k[G], v[G], ks[G], vs[G];
  v2u kz[G], vz[G];
};

template <int D>
__device__ __forceinline__ void load_tile(const uint8_t *p, int lane, TileRegs<D> &t) {
  constexpr int G = D / kKvGroup;
  const int q = lane >> 4;
#pragma unroll
  for (int x = 0; x < G; ++x) {
    t.k[x] = *reinterpret_cast<const v4u *>(p + x * 1024 + lane * 16);
    t.v[x] = *reinterpret_cast<const v4u *>(p + 16 * D + x * 1024 + lane * 16);
    t.ks[x] = *reinterpret_cast<const v4u *>(p + 32 * D + x * 64 + q * 16);
    t.vs[x] = *reinterpret_cast<const v4u *>(p + 32 * D + 64 * G + x * 64 + q * 16);
    t.kz[x] = *reinterpret_cast<const v2u *>(p + 32 * D + 128 * G + (q * G + x) * 8);
    t.vz[x] = *reinterpret_cast<const v2u *>(p + 32 * D + 160 * G + (q * G + x) * 8);
  }
}

__device__ __forceinline__ float half_of(v4u w, int i) { return f16_to_f32((uint16_t)(w[i >> 1] >> (16 * (i & 1)))); }

// Sums of a wave: MT row tiles, lane's query is column lane % 16 of each.
template <int D, int MT>
struct Sums {
  static constexpr int G = D / kKvGroup;
  v4f acc[MT][D / 16];     // channels 16 nt + 4 (lane / 16) + r
  float o[MT], l[MT];      // l: this lane's tokens only
};

// One tile of 32 tokens.  MASK: token t0 + i is seen by row tile m's query where
// lo[m] <= t0 + i < hi[m].
template <int D, int MT, int DT, bool SPLIT, bool MASK>
__device__ __forceinline__ void step(const TileRegs<D> &t, const v4u (&Q)[MT][D / 32], const float (&qs)[MT][D / 64],
                                     float c2, int t0, const int *lo, const int *hi, Sums<D, MT> &s) {
  constexpr int G = D / kKvGroup;
  const int q = (threadIdx.x & 63) >> 4;
  float e[MT][8];
#pragma unroll
  for (int a = 0; a < 2; ++a) {
#pragma unroll
    for (int g = 0; g < G; ++g) {
      const int x = a * (D / 32) + 2 * g;
      const v4u k0 = expand<DT>(t.k[x >> 2][x & 3]), k1 = expand<DT>(t.k[(x + 1) >> 2][(x + 1) & 3]);
#pragma unroll
      for (int m = 0; m < MT; ++m) {
        v4f d = mfma16<DT>(k0, Q[m][2 * g], (v4f){0.0f, 0.0f, 0.0f, 0.0f});
        d = mfma16<DT>(k1, Q[m][2 * g + 1], d);
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const float z = (float)(t.kz[g][a] >> (8 * (((r & 1) << 1) | (r >> 1))) & 0xFFu);
          const float u = __builtin_fmaf(-z, qs[m][g], d[r]);
          const float k = half_of(t.ks[g], 4 * a + r);
          e[m][4 * a + r] = g ? __builtin_fmaf(u, k, e[m][4 * a + r]) : u * k;
        }
      }
    }
  }
  if (MASK) {
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int tok = t0 + 16 * (i >> 2) + 4 * q + (i & 3);
        if (tok < lo[m] || tok >= hi[m]) e[m][i] = -__builtin_inff();
      }
  }
  float p[MT][8], ps[MT][G][8];
  bool moved = false;
  auto weigh = [&](int m) __attribute__((always_inline)) {
    float top = 0.0f, topp = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      p[m][i] = __builtin_amdgcn_exp2f(__builtin_fmaf(e[m][i], c2, -s.o[m]));
      topp = fmaxf(topp, p[m][i]);
#pragma unroll
      for (int g = 0; g < G; ++g) {
        float w = p[m][i] * half_of(t.vs[g], i);
        // a hidden token's scale may be anything, NaN among it
        if (MASK) w = e[m][i] == -__builtin_inff() ? 0.0f : w;
        ps[m][g][i] = w;
        top = fmaxf(top, w);
      }
    }
    return top > kMaxPs || topp > kMaxP;
  };
#pragma unroll
  for (int m = 0; m < MT; ++m) moved |= weigh(m);
  if (__builtin_expect(__any(moved), 0)) {
#pragma unroll
    for (int m = 0; m < MT; ++m) {
      float top = -__builtin_inff();
      bool mine = false;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float b = e[m][i] * c2;
        mine |= p[m][i] > kMaxP;
#pragma unroll
        for (int g = 0; g < G; ++g) {
          mine |= ps[m][g][i] > kMaxPs;
          const float v = half_of(t.vs[g], i);
          top = fmaxf(top, b + __builtin_amdgcn_logf(fmaxf(v, 5.9604644775390625e-8f)));
        }
      }
      top = over_q(top, false);
      if (over_q(mine ? 1.0f : 0.0f, false) > 0.0f) {
        const float o = __builtin_ceilf(top) - kTop;
        const float al = __builtin_amdgcn_exp2f(s.o[m] - o);
        s.o[m] = o;
        s.l[m] *= al;
#pragma unroll
        for (int n = 0; n < D / 16; ++n) s.acc[m][n] *= al;
      }
      weigh(m);
    }
  }
  v4u w[MT][G], w2[MT][G];
#pragma unroll
  for (int m = 0; m < MT; ++m) {
#pragma unroll
    for (int i = 0; i < 8; ++i) s.l[m] += p[m][i];
#pragma unroll
    for (int g = 0; g < G; ++g)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t hi = pack_h(ps[m][g][2 * i], ps[m][g][2 * i + 1]);   // (a bit_cast of w[m][g][i] reads w[m][g][0])
        w[m][g][i] = hi;
        if (SPLIT) {
          const v2h h = __builtin_bit_cast(v2h, hi);
          w2[m][g][i] = pack_h(ps[m][g][2 * i] - (float)h[0], ps[m][g][2 * i + 1] - (float)h[1]);
        }
      }
  }
#pragma unroll
  for (int g = 0; g < G; ++g) {
    v4u zz;
#pragma unroll
    for (int a = 0; a < 2; ++a) {
      const v4u z = expand<kF16>(t.vz[g][a]);
      zz[2 * a] = z[0];
      zz[2 * a + 1] = z[1];
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {         // channels 32 p ..: 32 tokens in two dwords
      const int pr = 2 * g + h;
      const v4u v0 = expand<kF16>(t.v[pr >> 1][2 * (pr & 1)]), v1 = expand<kF16>(t.v[pr >> 1][2 * (pr & 1) + 1]);
      const v4u b0 = {minus_h(v0[0], zz[0]), minus_h(v0[1], zz[1]), minus_h(v1[0], zz[2]), minus_h(v1[1], zz[3])};
      const v4u b1 = {minus_h(v0[2], zz[0]), minus_h(v0[3], zz[1]), minus_h(v1[2], zz[2]), minus_h(v1[3], zz[3])};
#pragma unroll
      for (int m = 0; m < MT; ++m) {
        s.acc[m][2 * pr] = mfma16<kF16>(b0, w[m][g], s.acc[m][2 * pr]);
        s.acc[m][2 * pr + 1] = mfma16<kF16>(b1, w[m][g], s.acc[m][2 * pr + 1]);
        if (SPLIT) {
          s.acc[m][2 * pr] = mfma16<kF16>(b0, w2[m][g], s.acc[m][2 * pr]);
          s.acc[m][2 * pr + 1] = mfma16<kF16>(b1, w2[m][g], s.acc[m][2 * pr + 1]);
        }
      }
    }
  }
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
constexpr int kMinTiles = 16;             // a part is 512 tokens at least
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

template <int D, int MT, int W, int DT, bool SPLIT, bool ROWS>
__global__ __launch_bounds__(64 * W) void k_kv_attention(KvAttnArgs a, int blocks) {
  constexpr int G = D / kKvGroup, kRows = 16 * MT * (ROWS ? W : 1), kLd = D + 4;
  extern __shared__ float lds[];
  const int lane = threadIdx.x & 63, q = lane >> 4, col = lane & 15;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  int id = blockIdx.x;
  const int blk = blocks - 1 - id % blocks;     // the last rows see the most: first
  id /= blocks;
  const int h = id % a.c.H;
  id /= a.c.H;
  const int part = ROWS ? 0 : id % a.splits, b = ROWS ? id : id / a.splits;
  int start, n;
  kv_rows(a.c, b, start, n);
  const int rows = n * a.gr, r0 = blk * kRows + (ROWS ? wave * 16 * MT : 0);
  if (r0 >= rows) return;
  const int len = kv_len(a.c, b), p0 = max(a.c.lens[b], 0) - n;
  int first, last;
  tiles_of_rows(a, r0, min(r0 + 16 * MT, rows), p0, len, first, last);
  if (!ROWS) {
    const int per = tiles_of_part(first, last, a.splits);
    first += part * per;
    if (part > 0 && first >= last) return;
    last = min(last, first + per);
  }

  // this lane's queries
  v4u Q[MT][D / 32];
  float qs[MT][G];
  int lo[MT], hi[MT];
  int full_lo = 0, full_hi = 1 << 30;           // tokens that every row of the wave sees
  size_t at[MT];                                // row of Y (heads counted), or none
  bool live[MT];
#pragma unroll
  for (int m = 0; m < MT; ++m) {
    const int row = r0 + 16 * m + col;
    live[m] = row < rows;
    const int i = min(row, rows - 1) / a.gr, head = h * a.gr + (live[m] ? row - i * a.gr : 0);
    const Seen s = seen_by(a, i, p0, len);
    lo[m] = s.lo;
    hi[m] = s.hi;
    at[m] = (size_t)(start + i) * a.Hq + head;
    const uint16_t *src = a.Q + (size_t)(start + i) * a.q_stride + (size_t)head * D + 8 * q;
#pragma unroll
    for (int x = 0; x < D / 32; ++x)
      Q[m][x] = live[m] ? *reinterpret_cast<const v4u *>(src + 32 * x) : (v4u){0u, 0u, 0u, 0u};
    constexpr uint32_t one = DT == kBf16 ? 0x3F803F80u : 0x3C003C00u;
    const v4u ones = {one, one, one, one};
#pragma unroll
    for (int g = 0; g < G; ++g) {
      v4f d = mfma16<DT>(ones, Q[m][2 * g], (v4f){0.0f, 0.0f, 0.0f, 0.0f});
      d = mfma16<DT>(ones, Q[m][2 * g + 1], d);
      qs[m][g] = d[0];
    }
  }
  {
    const Seen s0 = seen_by(a, r0 / a.gr, p0, len), s1 = seen_by(a, (min(r0 + 16 * MT, rows) - 1) / a.gr, p0, len);
    full_lo = s1.lo;
    full_hi = s0.hi;
  }
  Sums<D, MT> s;
#pragma unroll
  for (int m = 0; m < MT; ++m) {
    s.o[m] = kNoOffset;
    s.l[m] = 0.0f;
#pragma unroll
    for (int x = 0; x < D / 16; ++x) s.acc[m][x] = (v4f){0.0f, 0.0f, 0.0f, 0.0f};
  }
  for (int tile = first + (ROWS ? 0 : wave); tile < last; tile += ROWS ? 1 : W) {
    const uint8_t *p = kv_tile_at(a.c, b, h, tile);
    if (!p) continue;                           // on no page: not there
    TileRegs<D> t;
    load_tile<D>(p, lane, t);
    const int t0 = tile * kKvTile;
    if (t0 >= full_lo && t0 + kKvTile <= full_hi)
      step<D, MT, DT, SPLIT, false>(t, Q, qs, a.scale2, t0, lo, hi, s);
    else
      step<D, MT, DT, SPLIT, true>(t, Q, qs, a.scale2, t0, lo, hi, s);
  }
#pragma unroll
  for (int m = 0; m < MT; ++m) s.l[m] = over_q(s.l[m], true);
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
  // the waves' sums meet in LDS: [wave][row][D + 4], then (offset, weight) [wave][row]
  float2 *ol = reinterpret_cast<float2 *>(lds + W * 16 * MT * kLd);
#pragma unroll
  for (int m = 0; m < MT; ++m) {
    const int row = wave * 16 * MT + 16 * m + col;
#pragma unroll
    for (int x = 0; x < D / 16; ++x) *reinterpret_cast<v4f *>(lds + row * kLd + 16 * x + 4 * q) = s.acc[m][x];
    if (q == 0) ol[row] = make_float2(s.o[m], s.l[m]);
  }
  __syncthreads();
  for (int i = threadIdx.x; i < 16 * MT * (D / 4); i += 64 * W) {
    const int row = i / (D / 4), d = i % (D / 4) * 4, rr = r0 + row;
    if (rr >= rows) continue;
    float o = kNoOffset, l = 0.0f;
#pragma unroll
    for (int w = 0; w < W; ++w) {
      const float v = ol[w * 16 * MT + row].x;
      o = v != v || v > o ? v : o;
    }
    v4f y = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int w = 0; w < W; ++w) {
      const float2 u = ol[w * 16 * MT + row];
      const float f = __builtin_amdgcn_exp2f(u.x - o);
      l = __builtin_fmaf(u.y, f, l);
      const v4f v = *reinterpret_cast<const v4f *>(lds + (w * 16 * MT + row) * kLd + d);
#pragma unroll
      for (int r = 0; r < 4; ++r) y[r] = __builtin_fmaf(v[r], f, y[r]);
    }
    const int ti = rr / a.gr;
    const size_t yr = (size_t)(start + ti) * a.Hq + h * a.gr + (rr - ti * a.gr);
    if (a.splits == 1) {
      store_y(a, yr * D + d, y * inverse(l));
      if (a.lse && d == 0) a.lse[yr] = lse_of(o, l);
    } else {
      *reinterpret_cast<v4f *>(a.part + (yr * a.splits + part) * D + d) = y;
      if (d == 0) a.part_ol[yr * a.splits + part] = make_float2(o, l);
    }
  }
}

// The parts of a row, in order: a wave a row, D / 4 lanes of it at work.
template <int D>
__global__ __launch_bounds__(256) void k_kv_join(KvAttnArgs a, int blocks, int block_rows) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  int id = blockIdx.x;
  const int blk = id % blocks;
  id /= blocks;
  const int h = id % a.c.H, b = id / a.c.H;
  int start, n;
  kv_rows(a.c, b, start, n);
  const int rows = n * a.gr, r0 = blk * block_rows;
  if (r0 >= rows) return;
  const int len = kv_len(a.c, b), p0 = max(a.c.lens[b], 0) - n;
  int first, last;
  tiles_of_rows(a, r0, min(r0 + block_rows, rows), p0, len, first, last);
  const int per = tiles_of_part(first, last, a.splits), parts = max(1, (last - first + per - 1) / per);
  for (int r = wave; r < block_rows && r0 + r < rows; r += 4) {
    const int ti = (r0 + r) / a.gr;
    const size_t yr = (size_t)(start + ti) * a.Hq + h * a.gr + (r0 + r - ti * a.gr);
    const float2 *ol = a.part_ol + yr * a.splits;
    float o = kNoOffset, l = 0.0f;
    for (int w = 0; w < parts; ++w) {
      const float v = ol[w].x;
      o = v != v || v > o ? v : o;
    }
    if (lane * 4 >= D) continue;
    v4f y = {0.0f, 0.0f, 0.0f, 0.0f};
    for (int w = 0; w < parts; ++w) {
      const float f = __builtin_amdgcn_exp2f(ol[w].x - o);
      l = __builtin_fmaf(ol[w].y, f, l);
      const v4f v = *reinterpret_cast<const v4f *>(a.part + (yr * a.splits + w) * D + lane * 4);
#pragma unroll
      for (int e = 0; e < 4; ++e) y[e] = __builtin_fmaf(v[e], f, y[e]);
    }
    store_y(a, yr * D + lane * 4, y * inverse(l));
    if (a.lse && lane == 0) a.lse[yr] = lse_of(o, l);
  }
}

template <int D, int MT, int W, bool ROWS>
hipError_t launch_cfg(const KvAttnArgs &a, hipStream_t s) {
  constexpr int kRows = 16 * MT * (ROWS ? W : 1);
  const int blocks = ceil_div(a.c.max_tokens * a.gr, kRows);
  const unsigned grid = (unsigned)blocks * a.c.H * a.c.B * (ROWS ? 1 : a.splits);
  const size_t lds = ROWS ? 0 : (size_t)W * 16 * MT * ((D + 4) * sizeof(float) + sizeof(float2));
  auto go = [&](auto kernel) {
    if (lds > 64 * 1024) {
      const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void *>(kernel),
                                               hipFuncAttributeMaxDynamicSharedMemorySize, (int)lds);
      if (e != hipSuccess) return e;
    }
    hipLaunchKernelGGL(kernel, dim3(grid), dim3(64 * W), lds, s, a, blocks);
    return hipGetLastError();
  };
  hipError_t e;
  if (a.dtype == kBf16)
    e = a.y_dtype == kF32 ? go(k_kv_attention<D, MT, W, kBf16, true, ROWS>)
                          : go(k_kv_attention<D, MT, W, kBf16, false, ROWS>);
  else
    e = a.y_dtype == kF32 ? go(k_kv_attention<D, MT, W, kF16, true, ROWS>)
                          : go(k_kv_attention<D, MT, W, kF16, false, ROWS>);
  if (e == hipSuccess && !ROWS && a.splits > 1) {
    hipLaunchKernelGGL((k_kv_join<D>), dim3((unsigned)blocks * a.c.H * a.c.B), dim3(256), 0, s, a, blocks, kRows);
    e = hipGetLastError();
  }
  return e;
}

template <int D>
hipError_t launch_d(const KvAttnArgs &a, const KvAttnPlan &p, hipStream_t s) {
  if (p.by_rows) return D == 256 ? launch_cfg<D, 1, 4, true>(a, s) : launch_cfg<D, D == 256 ? 1 : 2, 4, true>(a, s);
  return launch_cfg<D, 1, D == 256 ? 4 : 8, false>(a, s);
}

}  // namespace

KvAttnPlan plan_kv_attention(int T, int Hq, int H, int D, int B, int max_tokens, int64_t capacity) {
  KvAttnPlan p;
  const long long rows = (long long)max_tokens * (Hq / H);
  p.by_rows = rows >= 64;
  p.mt = p.by_rows && D < 256 ? 2 : 1;
  p.waves = p.by_rows || D == 256 ? 4 : 8;
  if (!p.by_rows) {
    const long long wgs = ((rows + 15) / 16) * H * B;
    const long long most = std::max<long long>(1, (capacity + kMinTiles * kKvTile - 1) / (kMinTiles * kKvTile));
    p.splits = (int)std::min<long long>({std::max<long long>(1, 512 / wgs), most, 64});
    if (p.splits > 1) {
      const size_t parts = (size_t)T * Hq * p.splits;
      p.part_off = align_up(parts * sizeof(float2), 256);
      p.total = p.part_off + parts * D * sizeof(float);
    }
  }
  return p;
}

hipError_t launch_kv_attention(const KvAttnArgs &a, const KvAttnPlan &p, hipStream_t s) {
  switch (a.c.D) {
    case 64: return launch_d<64>(a, p, s);
    case 128: return launch_d<128>(a, p, s);
    case 256: return launch_d<256>(a, p, s);
    default: return hipErrorInvalidValue;
  }
}

}  // namespace hsq
