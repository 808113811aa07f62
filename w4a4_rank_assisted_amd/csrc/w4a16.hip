// w4a16.hip -- the layer with its activations left in 16 bits, for few tokens
// (M <= 64): the packed 4-bit residual against X itself.
//
//   xh = X / lambda,  U = xh L1
//   Y  = sum_g sw[g,n] sum_{k in g} xh[m,k] qw[k,n] + U L2 + bias + residual
//
// Bound by the read of the weights (K N / 2 bytes for 2 M K N operations), as the
// weight-streaming contraction of the W4A4 layer, whose mapping this is: a
// workgroup owns some tiles of 16 columns, its waves deal out the 128-channel
// pairs of blocks, and their partial tiles meet in LDS.  At these sizes a launch is as
// long as the read (25 MB: 5 us), so up to four rows take one launch (k_w4a16_small),
// more rows one that prepares xh and U, one that contracts and, where N has too few
// columns for 256 compute units, one that joins the parts of K.
//
// Measured (bf16, group 64, of a graph of calls), K x N:
//   M = 1   4096 x 12288: 7.3 us (3.7 TB/s), 4096 x 4096: 4.4, 12288 x 4096: 8.3,
//           4096 x 65536: 30.5 (4.7 TB/s); 3 x 4096 x 4096 with lambda and rank 16: 13.0
//   M = 16  12288 x 4096: 11.8, with lambda, rank 4 and fp32 Y 21.8 (5 preparing, 12
//           contracting, 4 joining); M = 64  4096 x 12288: 25.4
//
// The codes become matrix operands without a conversion.  Against X itself a nibble
// under a constant exponent is 24 + code, in bf16 and in fp16 alike (a shift and an
// and-xor a pair).  With smoothing xh is formed once, as fp16 numbers
// under a power of two per row and scale group: one of 11 bits where Y is bf16, two
// (22 bits) where it is finer, so that what is rounded is far below the rounding of
// Y.  Against those a nibble in the lowest bits of a half is the subnormal number (8 +
// code) 2^-24, in the next four (8 + code) 2^-20, which the matrix unit takes exactly (one
// mask a pair); xh is stored in the order of the nibbles, its half that meets the
// higher ones by 1/16.  The unit aligns a sum's terms by their operands' exponents,
// which for a subnormal number is that of 2^-14, so that a sum keeps 2^-14 of its
// largest xh: less than the 2^-12 that rounding xh costs.  Against two terms the
// codes are shifted to (8 + code) 2^-18, which keeps 2^-20, for three shifts a dword
// (12288 x 4096, 16 rows: 21.8 us either way).  The 24 or 8 times the sum of xh that
// is too much in every column is the accumulator's first value, the product of the
// same xh with a constant, one for all column tiles.  U's products and sums are fp32: up
// to four rows of xh as its terms hold it (the same xh as in the other sum: 11 bits for a bf16
// Y), above of xh before it is rounded.
#include "hsq_internal.h"

#include <algorithm>
#include <type_traits>

namespace hsq {

namespace {

typedef __bf16 v8bf __attribute__((ext_vector_type(8)));
typedef _Float16 v8h __attribute__((ext_vector_type(8)));

constexpr int kStreamLoad = 2;    // the weights are read once: non-temporal
constexpr int kPrepThreads = 256;
constexpr int kCUs = 256;
constexpr size_t kSmallLds = 128 * 1024;
constexpr int kPrepChannels = 2048;   // of a workgroup, at most

template <int DT>
__device__ __forceinline__ v4f mfma16(v4u a, v4u b, v4f c) {
  if constexpr (DT == kBf16)
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(v8bf, a), __builtin_bit_cast(v8bf, b), c, 0, 0, 0);
  else
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(v8h, a), __builtin_bit_cast(v8h, b), c, 0, 0, 0);
}

// What X is: bf16 or fp16 as given, or xh under powers of two.
constexpr int kScaled = 3;
// One over the code of the low nibbles (the codes with one or two terms of xh).
constexpr float code_scale(int terms) { return terms == 2 ? 262144.0f : 16777216.0f; }

// A dword of the packed residual, channels p = 0 .. 7, as 24 + code in the order
// 0 2 1 3 4 6 5 7 (high nibbles of bytes 0, 2 | 1, 3, then the low ones), or as 8 +
// code in the order 4 6 5 7 | 0 2 1 3, under 2^-24 and 2^-20, or 2^-18 against two
// terms of xh (NX).
template <int DT, int NX>
__device__ __forceinline__ v4u expand(uint32_t w) {
  if constexpr (DT == kScaled && NX == 2) {
    constexpr uint32_t m = 0x03C003C0u;
    const uint32_t u = w ^ 0x88888888u;
    return (v4u){u << 6 & m, u >> 2 & m, u << 2 & m, u >> 6 & m};
  } else if constexpr (DT == kScaled) {
    constexpr uint32_t l = 0x000F000Fu, h = 0x00F000F0u;
    const uint32_t u = w ^ 0x88888888u, v = u >> 8;
    return (v4u){u & l, v & l, u & h, v & h};
  } else if constexpr (DT == kBf16) {
    constexpr uint32_t m = 0x00780078u, k = 0x41C041C0u;
    return (v4u){(w >> 1 & m) ^ k, (w >> 9 & m) ^ k, (w << 3 & m) ^ k, (w >> 5 & m) ^ k};
  } else {
    constexpr uint32_t m = 0x03C003C0u, k = 0x4E004E00u;
    return (v4u){(w << 2 & m) ^ k, (w >> 6 & m) ^ k, (w << 6 & m) ^ k, (w >> 2 & m) ^ k};
  }
}
// The constant that takes the 24 or 8 off.
template <int DT, int NX>
__device__ __forceinline__ v4u minus_one() {
  if constexpr (DT == kScaled && NX == 2) return (v4u){0x82008200u, 0x82008200u, 0x82008200u, 0x82008200u};
  if constexpr (DT == kScaled) return (v4u){0x80088008u, 0x80088008u, 0x80808080u, 0x80808080u};
  constexpr uint32_t m = DT == kBf16 ? 0xC1C0C1C0u : 0xCE00CE00u;
  return (v4u){m, m, m, m};
}

// Eight consecutive channels in the order of expand.
template <int DT>
__device__ __forceinline__ v4u in_order(v4u x) {
  if constexpr (DT == kScaled) return x;
  return (v4u){__builtin_amdgcn_perm(x[1], x[0], 0x05040100u), __builtin_amdgcn_perm(x[1], x[0], 0x07060302u),
               __builtin_amdgcn_perm(x[3], x[2], 0x05040100u), __builtin_amdgcn_perm(x[3], x[2], 0x07060302u)};
}

__device__ __forceinline__ float half_or_bf(uint16_t v, int dtype) {
  return dtype == kBf16 ? bf16_to_f32(v) : f16_to_f32(v);
}

// Eight channels of xh under a power of two of their group's (gl lanes in a row): the
// terms in the order of expand, and what a product of them with the codes is
// multiplied by.  2^e has the largest |xh| / 2^e in [2^13, 2^14); from the bits of the
// exponent alone: a zero, tiny or infinite group keeps a scale that is finite.
__device__ __forceinline__ void scale_run(v4u x, v4u lam, int dtype, int gl, int terms, v4u &hi, v4u &lo, float &sc) {
  float v[8], top = 0.0f;
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const uint32_t w = x[e >> 1], u = lam[e >> 1];
    v[e] = half_or_bf((uint16_t)(e & 1 ? w >> 16 : w), dtype) * (1.0f / f16_to_f32((uint16_t)(e & 1 ? u >> 16 : u)));
    top = fmaxf(top, fabsf(v[e]));
  }
  for (int o = 1; o < gl; o <<= 1) top = fmaxf(top, __shfl_xor(top, o));
  const int ex = min(max((int)(__float_as_uint(top) >> 23) - 13, 1), 229);
  const float inv = __uint_as_float((uint32_t)(254 - ex) << 23);
  sc = __uint_as_float((uint32_t)ex << 23) * code_scale(terms);
  const float high = terms == 2 ? 1.0f : 0.0625f;      // of what meets the high nibbles
  constexpr int order[8] = {4, 6, 5, 7, 0, 2, 1, 3};
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    uint32_t h[2], l[2];
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      const float y = v[order[2 * e + c]] * inv * (e < 2 ? 1.0f : high);
      const _Float16 t = (_Float16)y;
      h[c] = __builtin_bit_cast(uint16_t, t);
      l[c] = fabsf(y) <= 65504.0f ? f32_to_f16(y - (float)t) : 0u;   // not finite: in hi alone
    }
    hi[e] = h[0] | h[1] << 16;
    lo[e] = l[0] | l[1] << 16;
  }
}

// Smoothing and U: a workgroup has `slice` channels of up to kPrepRows rows, and a
// projection's L1 of them.  R: the rank, 0 one without a form of its own; then a thread
// has a column and some channels, otherwise eight values in order, which is eight
// columns of a channel or four of two.  Bound by latency: 16 x 12288 with rank 4 takes
// 4.9 us (L1 one value a load and its sums through LDS alone: 6.2), of which a launch
// that does nothing takes 2.5.
constexpr int kPrepRows = 4, kPrepLoads = 16;

template <int R>
__global__ __launch_bounds__(kPrepThreads) void k_w4a16_prep(W4a16Args a) {
  constexpr int W = kPrepThreads / 64, RV = R > 8 ? R / 8 : 1, PER = R == 4 ? 2 : 1;
  extern __shared__ float xh[];                // [rows][slice], then partial sums
  float *red = xh + kPrepRows * a.slice;       // R: [W][32 RV], otherwise [rows][threads]
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, proj = blockIdx.z;
  const int k0 = blockIdx.x * a.slice, nk = min(a.slice, a.K - k0), M16 = (a.M + 15) / 16 * 16;
  const int m0 = blockIdx.y * kPrepRows, rows = min(kPrepRows, a.M - m0);
  const uint16_t *l1 = a.r ? a.L1 + ((size_t)proj * a.K + k0) * a.r : nullptr;
  // what the sums need first goes out ahead of X
  const int items = nk * (R ? R : 1) / 8;
  v4u w0[4];
  if constexpr (R > 0) {
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (tid + e * kPrepThreads < items) w0[e] = *reinterpret_cast<const v4u *>(l1 + (size_t)(tid + e * kPrepThreads) * 8);
  }
  // runs of eight channels; the lanes of a group are neighbours
  const int runs = nk / 8, gl = 8 * a.bpg;
  for (int i = tid; i < rows * runs; i += kPrepThreads) {
    const int m = i / runs, k = i % runs * 8;
    const size_t at = (size_t)(m0 + m) * a.K + k0 + k;
    const v4u x = *reinterpret_cast<const v4u *>(a.X + at);
    v4u lam = {0u, 0u, 0u, 0u};
    if (a.lam) lam = *reinterpret_cast<const v4u *>(a.lam + k0 + k);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float v = half_or_bf((uint16_t)(x[e >> 1] >> (16 * (e & 1))), a.dtype);
      xh[m * a.slice + k + e] = a.lam ? v * (1.0f / f16_to_f32((uint16_t)(lam[e >> 1] >> (16 * (e & 1))))) : v;
    }
    if (!a.lam || a.small || proj > 0) continue;     // U alone
    v4u hi, lo;
    float sc;
    scale_run(x, lam, a.dtype, gl, a.terms, hi, lo, sc);
    *reinterpret_cast<v4u *>(a.hi + at) = hi;
    if (a.terms == 2) *reinterpret_cast<v4u *>(a.lo + at) = lo;
    if (i % gl == 0) a.es[(size_t)((k0 + k) / (64 * a.bpg)) * M16 + m0 + m] = sc;
  }
  if (a.r == 0) return;
  __syncthreads();
  float *uw = a.uw + ((size_t)blockIdx.x * a.batch + proj) * a.r * M16 + m0;
  if constexpr (R > 0) {
    float u[32];                               // [row][column]
#pragma unroll
    for (int e = 0; e < 32; ++e) u[e] = 0.0f;
    auto add = [&](int i, v4u w) __attribute__((always_inline)) {
      const int k = PER == 2 ? 2 * i : i / RV;
#pragma unroll
      for (int m = 0; m < kPrepRows; ++m) {
        if (m >= rows) continue;
        const float x0 = xh[m * a.slice + k], x1 = PER == 2 ? xh[m * a.slice + k + 1] : x0;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const uint32_t t = w[e >> 1];
          u[8 * m + e] = __builtin_fmaf(e < 4 ? x0 : x1, half_or_bf((uint16_t)(e & 1 ? t >> 16 : t), a.dtype), u[8 * m + e]);
        }
      }
    };
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (tid + e * kPrepThreads < items) add(tid + e * kPrepThreads, w0[e]);
#pragma unroll 1
    for (int i = tid + 4 * kPrepThreads; i < items; i += kPrepThreads)
      add(i, *reinterpret_cast<const v4u *>(l1 + (size_t)i * 8));
    // lanes RV apart have the same columns: each step leaves a lane half of the values
    int n = 32, o = 32, first = 0;
#pragma unroll
    for (int step = 0; step < 5; ++step) {
      if (o < RV) break;
      n /= 2;
      const bool up = lane & o;
#pragma unroll
      for (int e = 0; e < n; ++e) u[e] = (up ? u[n + e] : u[e]) + __shfl_xor(up ? u[e] : u[n + e], o);
      first += up ? n : 0;
      o /= 2;
    }
    if constexpr (RV == 1) u[0] += __shfl_xor(u[0], 1);
#pragma unroll
    for (int e = 0; e < n; ++e)
      if (RV > 1 || (lane & 1) == 0) red[wave * 32 * RV + (first + e) * RV + (lane & (RV - 1))] = u[e];
    __syncthreads();
    for (int p = tid; p < rows * R; p += kPrepThreads) {
      const int m = p / R, j = p % R;
      float v = 0.0f;
#pragma unroll
      for (int e = 0; e < W; ++e) {
        const float *at = red + e * 32 * RV;
        v += PER == 2 ? at[8 * m + j] + at[8 * m + j + 4] : at[(8 * m + j % 8) * RV + j / 8];
      }
      uw[(size_t)j * M16 + m] = v;
    }
  } else {
    // a thread a column and every per-th channel, so that neighbours read neighbours;
    // then eight lanes a sum
    const int per = kPrepThreads / a.r, col = tid % a.r, sub = tid / a.r;
    if (sub < per) {
      float u[kPrepRows] = {0.0f, 0.0f, 0.0f, 0.0f};
      for (int k = sub; k < nk; k += per * kPrepLoads) {
        uint16_t w[kPrepLoads];
#pragma unroll
        for (int e = 0; e < kPrepLoads; ++e) w[e] = k + e * per < nk ? l1[(k + e * per) * a.r + col] : (uint16_t)0;
#pragma unroll
        for (int e = 0; e < kPrepLoads; ++e) {
          if (k + e * per >= nk) continue;
          const float f = half_or_bf(w[e], a.dtype);
#pragma unroll
          for (int m = 0; m < kPrepRows; ++m)
            if (m < rows) u[m] = __builtin_fmaf(xh[m * a.slice + k + e * per], f, u[m]);
        }
      }
#pragma unroll
      for (int m = 0; m < kPrepRows; ++m) red[m * kPrepThreads + tid] = u[m];
    }
    __syncthreads();
    for (int p = tid >> 3; p < rows * a.r; p += kPrepThreads / 8) {
      const int m = p / a.r, c = p % a.r;
      float v = 0.0f;
      for (int n = tid & 7; n < per; n += 8) v += red[m * kPrepThreads + n * a.r + c];
      v += __shfl_xor(v, 1);
      v += __shfl_xor(v, 2);
      v += __shfl_xor(v, 4);
      if ((tid & 7) == 0) uw[(size_t)c * M16 + m] = v;
    }
  }
}

// U of projection `proj` into LDS as [j][ld]: eight lanes add the slices of one value,
// four of theirs on their way at once.
__device__ __forceinline__ void sum_u(const W4a16Args &a, int proj, int m0, int rows, float *eu, int ld, int tid, int nthr) {
  const int cols = a.batch * a.r, M16 = (a.M + 15) / 16 * 16;
  for (int p = tid >> 3; p < a.r * rows; p += nthr >> 3) {
    const int j = p / rows, row = p % rows;
    const float *src = a.uw + ((size_t)proj * a.r + j) * M16 + m0 + row;
    float u = 0.0f;
    for (int sl = tid & 7; sl < a.u_slices; sl += 32) {
      float v[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) v[e] = sl + 8 * e < a.u_slices ? src[(size_t)(sl + 8 * e) * cols * M16] : 0.0f;
      u += (v[0] + v[1]) + (v[2] + v[3]);
    }
    u += __shfl_xor(u, 1);
    u += __shfl_xor(u, 2);
    u += __shfl_xor(u, 4);
    if ((tid & 7) == 0) eu[j * ld + row] = u;
  }
}

__device__ __forceinline__ float residual_at(const W4a16Args &a, size_t off) {
  return a.y_dtype == kF32 ? static_cast<const float *>(a.res)[off] : half_or_bf(static_cast<const uint16_t *>(a.res)[off], a.y_dtype);
}
__device__ __forceinline__ void store_at(const W4a16Args &a, size_t off, float y) {
  if (a.y_dtype == kF32) static_cast<float *>(a.Y)[off] = y;
  else
    static_cast<uint16_t *>(a.Y)[off] = a.y_dtype == kBf16 ? __builtin_bit_cast(uint16_t, (__bf16)y) : f32_to_f16(y);
}

// More than four rows.  X comes from the L2 cache once per workgroup, and that is what
// bounds this kernel (rows x K halves, per term, for every group of columns): four
// tiles a workgroup and, up to two tiles of rows, one pair of blocks a wave.  16 x 12288
// x 4096 with two terms took 27 us a call with four tiles and four parts of K, 35 with one
// tile and no parts; eight tiles do not fit the registers.  64 rows as two blocks of 32
// took 53 us where one block of 64 with one tile took 126 (lambda, fp32 Y).
constexpr int kColumnTiles = 4;

// Waves of a workgroup, at most.
constexpr int most_waves(int mt, int nx) { return mt > 1 ? 8 : nx > 1 ? 12 : 16; }

// NX: terms of xh (lo in the second).  The blocks of
// a.splits workgroups in z add to one output (k_w4a16_join).
template <int DT, int MT, int BPG, int NX>
__global__ __launch_bounds__(64 * most_waves(MT, NX)) void k_w4a16(W4a16Args a, int W) {
  constexpr int CT = kColumnTiles;
  constexpr int NS = BPG == 1 ? 2 : 1;             // scale groups of a pair of blocks
  constexpr bool XS = DT == kScaled;
  extern __shared__ float red[];                   // partial tiles [W][CT][MT][4][64], U [r][16 MT], L2 [r][16 CT], bias
  float *eu = red + W * CT * MT * 4 * 64;
  float *el2 = eu + a.r * MT * 16;
  float *eb = el2 + a.r * 16 * CT;
  const int tid = threadIdx.x, lane = tid & 63, colq = lane & 15, q = lane >> 4, nthr = blockDim.x;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int NT = (a.N + 15) / 16, nt0 = blockIdx.x * CT, proj = blockIdx.y % a.batch;
  const int m0 = blockIdx.y / a.batch * 16 * MT, rows = min(16 * MT, a.M - m0);
  const int G64 = a.K / kGroup, GP = (G64 + 1) / 2, SG = BPG == 1 ? G64 : G64 / 2, M16 = (a.M + 15) / 16 * 16;
  // pairs of this split
  const int per = (GP + a.splits - 1) / a.splits, g0 = blockIdx.z * per, g1 = min(g0 + per, GP);
  const __amdgpu_buffer_rsrc_t rs_w = buffer_rsrc(a.w + (size_t)proj * a.w_stride, (uint32_t)NT * GP * 1024);
  const __amdgpu_buffer_rsrc_t rs_s = buffer_rsrc(a.sw + (size_t)proj * SG * a.N, (uint32_t)SG * a.N * 2);
  uint32_t offw[CT], offs[CT];
#pragma unroll
  for (int c = 0; c < CT; ++c) {
    const int nt = min(nt0 + c, NT - 1);           // past the last tile: read, not stored
    offw[c] = ((uint32_t)nt * GP * 64 + lane) * 16;
    offs[c] = (uint32_t)min(nt * 16 + colq, a.N - 1) * 2;
  }
  const uint16_t *xsrc = XS ? a.hi : a.X;
  const __amdgpu_buffer_rsrc_t rs_x = buffer_rsrc(xsrc, (uint32_t)a.M * a.K * 2);
  const __amdgpu_buffer_rsrc_t rs_l = buffer_rsrc(NX == 2 ? a.lo : xsrc, (uint32_t)a.M * a.K * 2);
  uint32_t offx[MT];
#pragma unroll
  for (int i = 0; i < MT; ++i) offx[i] = ((uint32_t)(m0 + min(16 * i + colq, rows - 1)) * a.K + 16 * q) * 2;

  float acc[CT][MT][4];
#pragma unroll
  for (int c = 0; c < CT; ++c)
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
      for (int r = 0; r < 4; ++r) acc[c][i][r] = 0.0f;

  // the pair on its way
  v4u wv[CT], xv[NX][MT][4];
  _Float16 sv[CT][NS];
  v4f ev[NS][MT];
  auto load = [&](int gp) __attribute__((always_inline)) {
#pragma unroll
    for (int c = 0; c < CT; ++c) wv[c] = __builtin_amdgcn_raw_buffer_load_b128(rs_w, offw[c], gp * 1024, kStreamLoad);
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) {              // block j / 2, channels 8 (j % 2) ..
        const int blk = min(2 * gp + j / 2, G64 - 1);   // a pad block: the one before, times 0 below
        const uint32_t so = (uint32_t)blk * 128 + (j & 1) * 16;
        xv[0][i][j] = __builtin_amdgcn_raw_buffer_load_b128(rs_x, offx[i], so, 0);
        if constexpr (NX == 2) xv[1][i][j] = __builtin_amdgcn_raw_buffer_load_b128(rs_l, offx[i], so, 0);
      }
#pragma unroll
    for (int h = 0; h < NS; ++h) {
      const int sg = min(NS * gp + h, SG - 1);
#pragma unroll
      for (int c = 0; c < CT; ++c)
        sv[c][h] = __builtin_bit_cast(_Float16, __builtin_amdgcn_raw_buffer_load_b16(rs_s, offs[c], sg * a.N * 2, 0));
      if constexpr (XS) {
#pragma unroll
        for (int i = 0; i < MT; ++i) ev[h][i] = *reinterpret_cast<const v4f *>(a.es + (size_t)sg * M16 + min(m0 + 16 * i, M16 - 16) + 4 * q);
      }
    }
    __builtin_amdgcn_sched_barrier(0);
  };
  auto multiply = [&](int gp) __attribute__((always_inline)) {
    // a pad block (K an odd number of blocks) has X = 0
    if (NS == 2 && 2 * gp + 1 >= G64) {
#pragma unroll
      for (int t = 0; t < NX; ++t)
#pragma unroll
        for (int i = 0; i < MT; ++i) xv[t][i][2] = xv[t][i][3] = (v4u){0u, 0u, 0u, 0u};
    }
    const v4u neg = minus_one<DT, NX>();
    v4f base[NS][MT];
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int t = 0; t < NX; ++t) {
          xv[t][i][j] = in_order<DT>(xv[t][i][j]);
          const int h = NS == 2 ? j / 2 : 0;
          const bool start = t == 0 && (NS == 2 ? (j & 1) == 0 : j == 0);
          base[h][i] = mfma16<DT>(xv[t][i][j], neg, start ? (v4f){0.0f, 0.0f, 0.0f, 0.0f} : base[h][i]);
        }
#pragma unroll
    for (int c = 0; c < CT; ++c) {
      v4u b[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) b[j] = expand<DT, NX>(wv[c][j]);
#pragma unroll
      for (int h = 0; h < NS; ++h) {
        const float s = (float)sv[c][h];
#pragma unroll
        for (int i = 0; i < MT; ++i) {
          v4f d = base[h][i];
#pragma unroll
          for (int j = (NS == 2 ? 2 * h : 0); j < (NS == 2 ? 2 * h + 2 : 4); ++j)
#pragma unroll
            for (int t = 0; t < NX; ++t) d = mfma16<DT>(xv[t][i][j], b[j], d);
#pragma unroll
          for (int r = 0; r < 4; ++r)
            acc[c][i][r] = __builtin_fmaf(XS ? d[r] * ev[h][i][r] : d[r], s, acc[c][i][r]);
        }
      }
      __builtin_amdgcn_sched_barrier(0);
    }
  };

  const int first = wave < W ? g0 + wave : g1;
  if (first < g1) load(first);
  // what the epilogue adds, while the first weights travel
  const size_t base_off = (size_t)proj * a.M * a.N;
  auto out_of = [&](int o, int &m, int &n) __attribute__((always_inline)) {
    const int e = o >> 6, l = o & 63, c = e / (MT * 4), i = (e >> 2) % MT, r = e & 3;
    n = (nt0 + c) * 16 + (l & 15);
    m = i * 16 + 4 * (l >> 4) + r;
    const bool in = n < a.N && m < rows;
    m += m0;
    return in;
  };
  constexpr int E = CT * MT * 4;
  float res0 = 0.0f;
  if (a.splits == 1) {
    int m, n;
    if (a.res && tid < E * 64 && out_of(tid, m, n)) res0 = residual_at(a, base_off + (size_t)m * a.N + n);
    if (tid < 16 * CT) eb[tid] = a.bias ? half_or_bf(a.bias[(size_t)proj * a.N + min(nt0 * 16 + tid, a.N - 1)], a.dtype) : 0.0f;
    for (int p = tid; p < a.r * 16 * CT; p += nthr)
      el2[p] = half_or_bf(a.L2[((size_t)proj * a.r + p / (16 * CT)) * a.N + min(nt0 * 16 + p % (16 * CT), a.N - 1)], a.dtype);
    sum_u(a, proj, m0, rows, eu, MT * 16, tid, nthr);
  }
  for (int gp = first; gp < g1; gp += W) {
    multiply(gp);
    if (gp + W < g1) load(gp + W);
  }

  if (wave < W)
#pragma unroll
    for (int c = 0; c < CT; ++c)
#pragma unroll
      for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int r = 0; r < 4; ++r) red[(wave * E + (c * MT + i) * 4 + r) * 64 + lane] = acc[c][i][r];
  __syncthreads();
  for (int o = tid; o < E * 64; o += nthr) {
    int m, n;
    if (!out_of(o, m, n)) continue;
    float y = 0.0f;
    for (int w = 0; w < W; ++w) y += red[w * E * 64 + o];
    const size_t off = base_off + (size_t)m * a.N + n;
    if (a.splits > 1) {
      a.part[(size_t)blockIdx.z * a.batch * a.M * a.N + off] = y;
      continue;
    }
    const int cn = n - nt0 * 16;
    for (int k = 0; k < a.r; ++k) y = __builtin_fmaf(eu[k * MT * 16 + m - m0], el2[k * 16 * CT + cn], y);
    y += eb[cn];
    if (a.res) y += o == tid ? res0 : residual_at(a, off);
    store_at(a, off, y);
  }
}

// The splits of one row in order, U L2, bias and residual: 256 columns of it.
__global__ __launch_bounds__(256) void k_w4a16_join(W4a16Args a) {
  __shared__ float u[kMaxRank];
  const int tid = threadIdx.x, n = blockIdx.x * 256 + tid, m = blockIdx.y, proj = blockIdx.z;
  const bool live = n < a.N;
  const size_t off = ((size_t)proj * a.M + m) * a.N + (live ? n : 0), step = (size_t)a.batch * a.M * a.N;
  float p[kW4a16Splits];
#pragma unroll
  for (int s = 0; s < kW4a16Splits; ++s) p[s] = s < a.splits ? a.part[s * step + off] : 0.0f;
  const float res = a.res ? residual_at(a, off) : 0.0f;
  const float bias = a.bias ? half_or_bf(a.bias[(size_t)proj * a.N + (live ? n : 0)], a.dtype) : 0.0f;
  sum_u(a, proj, m, 1, u, 1, tid, 256);
  __syncthreads();
  if (!live) return;
  float y = 0.0f;
#pragma unroll
  for (int s = 0; s < kW4a16Splits; ++s) y += p[s];
  for (int k = 0; k < a.r; ++k) y = __builtin_fmaf(u[k], half_or_bf(a.L2[((size_t)proj * a.r + k) * a.N + n], a.dtype), y);
  store_at(a, off, y + bias + res);
}

// ------------------------------------------------------------------ up to 4 rows
// One launch: every workgroup forms xh of all its rows in LDS (K / 8 runs of eight
// channels), as the matrix operands take it, so that its waves load nothing but
// weights, four pairs on their way at once, each loaded again as soon as it is used.
// U from L1 (K r numbers, from the L2 cache) is formed here too while the first weights
// travel, as long as that is little (plan_w4a16); a launch of its own costs five
// microseconds.
constexpr int kSmallRows = 4, kSmallPairs = 4;

// Of eight values a lane, summed over the lanes that agree in the bits below
// `step`: the value of index lane / 8, in every lane.
__device__ __forceinline__ float scatter8(const float *u, int lane, int step) {
  float a[4], b[2], c;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const bool up = lane & 32;
    a[i] = (up ? u[4 + i] : u[i]) + __shfl_xor(up ? u[i] : u[4 + i], 32);
  }
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const bool up = lane & 16;
    b[i] = (up ? a[2 + i] : a[i]) + __shfl_xor(up ? a[i] : a[2 + i], 16);
  }
  const bool up = lane & 8;
  c = (up ? b[1] : b[0]) + __shfl_xor(up ? b[0] : b[1], 8);
  for (int o = 4; o >= step; o >>= 1) c += __shfl_xor(c, o);
  return c;
}

struct SmallLds {                          // offsets in floats
  int ldx, terms, es, red, u, eu, el2, eb, total;
};
inline __host__ __device__ SmallLds small_lds(int M, int K, int r, bool own_u, int nx, int ct, int bpg, int threads) {
  SmallLds l;
  l.ldx = (K + 127) / 128 * 128 + 16;      // halves of a row: whole pairs, and rows on other banks
  l.terms = 0;
  l.es = nx * M * l.ldx / 2;
  l.red = l.es + (K / (64 * bpg) + 1) * 4;
  l.u = l.red + threads / 64 * ct * 64;   // [waves][ct][4][16]
  l.eu = l.u + (own_u ? kSmallRows * threads : 0);
  l.el2 = l.eu + r * kSmallRows;
  l.eb = l.el2 + r * 16 * ct;
  l.total = l.eb + 16 * ct;
  return l;
}

// How the rank branch's U comes: there is none, formed here, from the launch before.
enum { kNoRank, kOwnU, kGivenU };

template <int DT, int CT, int BPG, int NX, int RANK, int T>
__global__ __launch_bounds__(T) void k_w4a16_small(W4a16Args a) {
  constexpr int NS = BPG == 1 ? 2 : 1, W = T / 64, P = kSmallPairs;
  constexpr bool XS = DT == kScaled;
  extern __shared__ __attribute__((aligned(16))) float lds[];
  const SmallLds L = small_lds(a.M, a.K, a.r, RANK == kOwnU, NX, CT, BPG, T);
  uint16_t *xt = reinterpret_cast<uint16_t *>(lds);
  float *es = lds + L.es, *red = lds + L.red, *us = lds + L.u, *eu = lds + L.eu, *el2 = lds + L.el2, *eb = lds + L.eb;
  const int tid = threadIdx.x, lane = tid & 63, colq = lane & 15, q = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int NT = (a.N + 15) / 16, nt0 = blockIdx.x * CT, proj = blockIdx.y;
  const int G64 = a.K / kGroup, GP = (G64 + 1) / 2, SG = BPG == 1 ? G64 : G64 / 2;
  const __amdgpu_buffer_rsrc_t rs_w = buffer_rsrc(a.w + (size_t)proj * a.w_stride, (uint32_t)NT * GP * 1024);
  const __amdgpu_buffer_rsrc_t rs_s = buffer_rsrc(a.sw + (size_t)proj * SG * a.N, (uint32_t)SG * a.N * 2);
  uint32_t offw[CT], offs[CT];
#pragma unroll
  for (int c = 0; c < CT; ++c) {
    const int nt = min(nt0 + c, NT - 1);           // past the last tile: read, not stored
    offw[c] = ((uint32_t)nt * GP * 64 + lane) * 16;
    offs[c] = (uint32_t)min(nt * 16 + colq, a.N - 1) * 2;
  }
  v4u wv[P][CT];
  _Float16 sv[P][CT][NS];
  auto load = [&](auto slot, int gp) __attribute__((always_inline)) {
    constexpr int p = decltype(slot)::value;
    gp = min(gp, GP - 1);
#pragma unroll
    for (int c = 0; c < CT; ++c) wv[p][c] = __builtin_amdgcn_raw_buffer_load_b128(rs_w, offw[c], gp * 1024, kStreamLoad);
#pragma unroll
    for (int h = 0; h < NS; ++h)
#pragma unroll
      for (int c = 0; c < CT; ++c)
        sv[p][c][h] = __builtin_bit_cast(
            _Float16, __builtin_amdgcn_raw_buffer_load_b16(rs_s, offs[c], min(NS * gp + h, SG - 1) * a.N * 2, 0));
    __builtin_amdgcn_sched_barrier(0);
  };
  auto each = [&](auto f) __attribute__((always_inline)) {
    f(std::integral_constant<int, 0>{});
    f(std::integral_constant<int, 1>{});
    f(std::integral_constant<int, 2>{});
    f(std::integral_constant<int, 3>{});
  };
  static_assert(P == 4, "four slots");
  // Loads are counted in order: what is needed before the weights goes out ahead of
  // them.  L1 as vectors of eight: eight columns of a channel, or four of two.
  const uint16_t *l1 = a.r > 0 ? a.L1 + (size_t)proj * a.K * a.r : nullptr;
  const bool vec = a.r == 4 || a.r == 8 || a.r == 16 || a.r == 32;
  const int rvs = a.r == 32 ? 2 : a.r == 16, rv = 1 << rvs, nv = a.r == 4 ? 4 : 8, items = (a.K / 8) << rvs, vstep = T;
  const int runs = GP * 16, gl = 8 * BPG;
  v4u x0, lam0 = {0u, 0u, 0u, 0u};
  auto load_x = [&](int i) __attribute__((always_inline)) {
    const int m = i / runs, k = i % runs * 8;
    const bool real = k < a.K;
    x0 = real ? *reinterpret_cast<const v4u *>(a.X + (size_t)m * a.K + k) : (v4u){0u, 0u, 0u, 0u};
    if constexpr (XS)
      lam0 = real ? *reinterpret_cast<const v4u *>(a.lam + k) : (v4u){0x3C003C00u, 0x3C003C00u, 0x3C003C00u, 0x3C003C00u};
  };
  if (tid < a.M * runs) load_x(tid);
  constexpr int A = CT == 4 ? 1 : 2;        // items of L1 ahead
  v4u w1[A][8];
  auto load_l1 = [&](int i, v4u (&w1)[8]) __attribute__((always_inline)) {
    const uint16_t *at = l1 + (size_t)(i >> rvs) * 8 * a.r + (i & (rv - 1)) * 8;
#pragma unroll
    for (int n = 0; n < 8; ++n)
      if (n < nv) w1[n] = *reinterpret_cast<const v4u *>(at + n * (nv == 4 ? 8 : a.r));
  };
  if (RANK == kOwnU && vec) {
    if (tid < items) load_l1(tid, w1[0]);
    if (A == 2 && tid + vstep < items) load_l1(tid + vstep, w1[A - 1]);
  }
  // what the epilogue adds
  float res0 = 0.0f;
  const int on = nt0 * 16 + (tid >> 6) * 16 + (tid & 15), om = (tid >> 4) & 3;     // output of this thread
  const bool out = tid < CT * 64 && on < a.N && om < a.M;
  const size_t off = ((size_t)proj * a.M + om) * a.N + on;
  if (out && a.res) res0 = residual_at(a, off);
  const uint16_t bias0 = tid < 16 * CT && a.bias ? a.bias[(size_t)proj * a.N + min(nt0 * 16 + tid, a.N - 1)] : (uint16_t)0;
  const int l2s = a.r * 16 * CT;
  auto l2_at = [&](int p) { return a.L2[((size_t)proj * a.r + p / (16 * CT)) * a.N + min(nt0 * 16 + p % (16 * CT), a.N - 1)]; };
  const uint16_t l20 = RANK && tid < l2s ? l2_at(tid) : (uint16_t)0;
  each([&](auto slot) { load(slot, wave + decltype(slot)::value * W); });

  // xh in LDS, a pad block of zeros behind an odd number of blocks
  for (int i = tid; i < a.M * runs; i += T) {
    if (i != tid) load_x(i);
    const int m = i / runs, k = i % runs * 8;
    v4u hi, lo = {0u, 0u, 0u, 0u};
    if constexpr (XS) {
      float sc;
      scale_run(x0, lam0, a.dtype, gl, NX, hi, lo, sc);
      if (i % gl == 0 && k < a.K) es[k / (64 * BPG) * 4 + m] = sc;
    } else {
      hi = in_order<DT>(x0);
    }
    *reinterpret_cast<v4u *>(xt + m * L.ldx + k) = hi;
    if constexpr (NX == 2) *reinterpret_cast<v4u *>(xt + (a.M + m) * L.ldx + k) = lo;
  }
  if (tid < 16 * CT) eb[tid] = half_or_bf(bias0, a.dtype);
  if (RANK) {
    if (tid < l2s) el2[tid] = half_or_bf(l20, a.dtype);
    for (int p = tid + T; p < l2s; p += T) el2[p] = half_or_bf(l2_at(p), a.dtype);
  }
  // LDS alone: the weights stay on their way
  asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
  if constexpr (RANK == kGivenU) sum_u(a, proj, 0, a.M, eu, kSmallRows, tid, T);
  // U: a run of eight channels and eight columns a lane (or one column), its sums
  // over the lanes' runs into LDS
  if constexpr (RANK == kOwnU) {
#pragma unroll 1
    for (int m = 0; m < a.M; ++m) {
      float u[8] = {0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f};
      auto channels = [&](int run, float *x) __attribute__((always_inline)) {
        const float f = XS ? es[run / (8 * BPG) * 4 + m] * (1.0f / code_scale(NX)) : 1.0f;
        const v4u hi = *reinterpret_cast<const v4u *>(xt + m * L.ldx + 8 * run);
        v4u lo = {0u, 0u, 0u, 0u};
        if constexpr (NX == 2) lo = *reinterpret_cast<const v4u *>(xt + (a.M + m) * L.ldx + 8 * run);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          constexpr int place[8] = {0, 2, 1, 3, 4, 6, 5, 7};     // of channel e in in_order's order
          const int at = XS ? place[e] ^ 4 : place[e];
          const uint32_t h = hi[at >> 1] >> (16 * (at & 1)), l = lo[at >> 1] >> (16 * (at & 1));
          x[e] = DT == kBf16 ? bf16_to_f32(h & 0xFFFFu) : f16_to_f32((uint16_t)h);
          if constexpr (NX == 2) x[e] += f16_to_f32((uint16_t)l);
          if constexpr (XS) x[e] *= NX == 1 && e < 4 ? f * 16.0f : f;
        }
      };
      if (vec) {
        // four columns of two channels, or eight of one, in either type
        auto add = [&](auto type, const v4u (&w1)[8], const float *x) __attribute__((always_inline)) {
          constexpr int kType = decltype(type)::value;
          auto value = [&](uint32_t t, int e) __attribute__((always_inline)) {
            if constexpr (kType == kBf16) return __uint_as_float(e & 1 ? t & 0xFFFF0000u : t << 16);
            else return f16_to_f32((uint16_t)(e & 1 ? t >> 16 : t));
          };
          if (nv == 4) {
#pragma unroll
            for (int n = 0; n < 4; ++n)
#pragma unroll
              for (int e = 0; e < 8; ++e) u[e] = __builtin_fmaf(x[2 * n + (e >> 2)], value(w1[n][e >> 1], e), u[e]);
          } else {
#pragma unroll
            for (int n = 0; n < 8; ++n)
#pragma unroll
              for (int e = 0; e < 8; ++e) u[e] = __builtin_fmaf(x[n], value(w1[n][e >> 1], e), u[e]);
          }
        };
        auto item = [&](int i, v4u (&w)[8]) __attribute__((always_inline)) {
          float x[8];
          // a row's own expansion: kept for all rows, it would be 64 registers an item
#pragma unroll
          for (int n = 0; n < 8; ++n) asm volatile("" : "+v"(w[n]));
          channels(i >> rvs, x);
          if (a.dtype == kBf16) add(std::integral_constant<int, kBf16>{}, w, x);
          else add(std::integral_constant<int, kF16>{}, w, x);
          __builtin_amdgcn_sched_barrier(0);
        };
        if (tid < items) item(tid, w1[0]);
        if (A == 2 && tid + vstep < items) item(tid + vstep, w1[A - 1]);
        for (int i = tid + A * vstep; i < items; i += vstep) {
          v4u w[8];
          load_l1(i, w);
          item(i, w);
        }
        const float v = scatter8(u, lane, rv);
        if ((lane & 7) < rv) us[(m * W + wave) * 8 * rv + 8 * (lane & (rv - 1)) + (lane >> 3)] = v;
      } else {
        const int step = T / a.r, j = tid % a.r;
        if (tid < step * a.r)
          for (int run = tid / a.r; run < a.K / 8; run += step) {
            uint16_t w[8];
#pragma unroll
            for (int n = 0; n < 8; ++n) w[n] = l1[(size_t)(8 * run + n) * a.r + j];
            float x[8];
            channels(run, x);
#pragma unroll
            for (int n = 0; n < 8; ++n) u[0] = __builtin_fmaf(x[n], half_or_bf(w[n], a.dtype), u[0]);
          }
        us[m * T + tid] = u[0];
      }
    }
  }

  float acc[CT][4];
#pragma unroll
  for (int c = 0; c < CT; ++c)
#pragma unroll
    for (int r = 0; r < 4; ++r) acc[c][r] = 0.0f;
  const uint16_t *xrow = xt + min(colq, a.M - 1) * L.ldx + 16 * q;
  const v4u neg = minus_one<DT, NX>();
  for (int g = wave; g < GP; g += P * W) {
    each([&](auto slot) __attribute__((always_inline)) {
      constexpr int p = decltype(slot)::value;
      const int gp = g + p * W;
      if (gp >= GP) return;
      v4u x[NX][4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint16_t *at = xrow + gp * 128 + (j >> 1) * 64 + (j & 1) * 8;
        x[0][j] = *reinterpret_cast<const v4u *>(at);
        if constexpr (NX == 2) x[1][j] = *reinterpret_cast<const v4u *>(at + a.M * L.ldx);
      }
      v4f base[NS], ev[NS];
#pragma unroll
      for (int h = 0; h < NS; ++h) {
        if constexpr (XS) ev[h] = *reinterpret_cast<const v4f *>(es + min(NS * gp + h, SG - 1) * 4);
        base[h] = (v4f){0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int j = (NS == 2 ? 2 * h : 0); j < (NS == 2 ? 2 * h + 2 : 4); ++j)
#pragma unroll
          for (int t = 0; t < NX; ++t) base[h] = mfma16<DT>(x[t][j], neg, base[h]);
      }
#pragma unroll
      for (int c = 0; c < CT; ++c) {
        v4u b[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) b[j] = expand<DT, NX>(wv[p][c][j]);
#pragma unroll
        for (int h = 0; h < NS; ++h) {
          const float s = (float)sv[p][c][h];
          v4f d = base[h];
#pragma unroll
          for (int j = (NS == 2 ? 2 * h : 0); j < (NS == 2 ? 2 * h + 2 : 4); ++j)
#pragma unroll
            for (int t = 0; t < NX; ++t) d = mfma16<DT>(x[t][j], b[j], d);
#pragma unroll
          for (int r = 0; r < 4; ++r) acc[c][r] = __builtin_fmaf(XS ? d[r] * ev[h][r] : d[r], s, acc[c][r]);
        }
      }
      if (gp + P * W < GP) load(slot, gp + P * W);      // its place is free
    });
  }
  // rows 0 .. 3 are the lanes of q = 0
  if (q == 0) {
#pragma unroll
    for (int c = 0; c < CT; ++c)
#pragma unroll
      for (int r = 0; r < 4; ++r) red[((wave * CT + c) * 4 + r) * 16 + colq] = acc[c][r];
  }
  __syncthreads();
  if (RANK == kOwnU) {
    if (vec) {
      if (tid < a.r * a.M) {
        const int m = tid / a.r, j = tid % a.r;
        float v = 0.0f;
#pragma unroll
        for (int w = 0; w < W; ++w) {
          const float *at = us + (m * W + w) * 8 * rv + j;
          v += a.r == 4 ? at[0] + at[4] : at[0];
        }
        eu[j * kSmallRows + m] = v;
      }
    } else {
      const int step = T / a.r;
      for (int p = tid >> 3; p < a.r * a.M; p += T / 8) {   // eight lanes a value
        const int m = p / a.r, j = p % a.r;
        float v = 0.0f;
        for (int n = tid & 7; n < step; n += 8) v += us[m * T + n * a.r + j];
        v += __shfl_xor(v, 1);
        v += __shfl_xor(v, 2);
        v += __shfl_xor(v, 4);
        if ((tid & 7) == 0) eu[j * kSmallRows + m] = v;
      }
    }
    __syncthreads();
  }
  if (!out) return;
  float y = 0.0f;
#pragma unroll
  for (int w = 0; w < W; ++w) y += red[((w * CT + (tid >> 6)) * 4 + om) * 16 + (tid & 15)];
  const int cn = (tid >> 6) * 16 + (tid & 15);
  if (RANK)
#pragma unroll 4
    for (int k = 0; k < a.r; ++k) y = __builtin_fmaf(eu[k * kSmallRows + om], el2[k * 16 * CT + cn], y);
  store_at(a, off, y + eb[cn] + res0);
}

template <int DT, int CT, int BPG, int NX, int RANK, int T>
hipError_t launch_small(const W4a16Args &a, hipStream_t s) {
  const size_t lds = (size_t)small_lds(a.M, a.K, a.r, RANK == kOwnU, NX, CT, BPG, T).total * sizeof(float);
  auto kernel = k_w4a16_small<DT, CT, BPG, NX, RANK, T>;
  if (lds > 64 * 1024) {
    const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void *>(kernel),
                                             hipFuncAttributeMaxDynamicSharedMemorySize, (int)lds);
    if (e != hipSuccess) return e;
  }
  hipLaunchKernelGGL(kernel, dim3((unsigned)ceil_div(ceil_div(a.N, kTile), CT), (unsigned)a.batch), dim3(T), lds, s, a);
  return hipGetLastError();
}

template <int DT, int BPG, int NX>
hipError_t launch_small_ct(const W4a16Args &a, hipStream_t s) {
  if (a.own_u) {
    switch (a.ct) {
      case 1: return launch_small<DT, 1, BPG, NX, kOwnU, 512>(a, s);
      case 2: return launch_small<DT, 2, BPG, NX, kOwnU, 512>(a, s);
      case 3: return launch_small<DT, 3, BPG, NX, kOwnU, 512>(a, s);
      default: return launch_small<DT, 4, BPG, NX, kOwnU, 512>(a, s);
    }
  }
  // 1 x 12288 x 4096: 8.3 us with 16 waves, 10.5 with eight; 1 x 4096 x 4096: 5.2, 4.4
  if (a.K > 8192) return a.r > 0 ? launch_small<DT, 1, BPG, NX, kGivenU, 1024>(a, s) : launch_small<DT, 1, BPG, NX, kNoRank, 1024>(a, s);
  return a.r > 0 ? launch_small<DT, 1, BPG, NX, kGivenU, 512>(a, s) : launch_small<DT, 1, BPG, NX, kNoRank, 512>(a, s);
}

template <int DT, int MT, int BPG, int NX>
hipError_t launch_cfg(const W4a16Args &a, hipStream_t s) {
  constexpr int CT = kColumnTiles;
  const int NT = ceil_div(a.N, kTile), GP = ceil_div(ceil_div(a.K / kGroup, 2), a.splits);
  const int W = ceil_div(GP, ceil_div(GP, most_waves(MT, NX)));
  const size_t lds = ((size_t)W * CT * MT * 4 * 64 + (size_t)a.r * 16 * (MT + CT) + 16 * CT) * sizeof(float);
  auto kernel = k_w4a16<DT, MT, BPG, NX>;
  if (lds > 64 * 1024) {
    const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void *>(kernel),
                                             hipFuncAttributeMaxDynamicSharedMemorySize, (int)lds);
    if (e != hipSuccess) return e;
  }
  hipLaunchKernelGGL(kernel, dim3((unsigned)ceil_div(NT, CT), (unsigned)(a.batch * ceil_div(a.M, 16 * MT)), (unsigned)a.splits),
                     dim3(64 * most_waves(MT, NX)), lds, s, a, W);
  return hipGetLastError();
}

template <int DT, int BPG, int NX>
hipError_t launch_rows(const W4a16Args &a, hipStream_t s) {
  return a.M <= kTile ? launch_cfg<DT, 1, BPG, NX>(a, s) : launch_cfg<DT, 2, BPG, NX>(a, s);
}

template <int BPG>
hipError_t launch_bpg(const W4a16Args &a, hipStream_t s) {
  if (a.small) {
    if (a.lam) return a.terms == 2 ? launch_small_ct<kScaled, BPG, 2>(a, s) : launch_small_ct<kScaled, BPG, 1>(a, s);
    return a.dtype == kBf16 ? launch_small_ct<kBf16, BPG, 1>(a, s) : launch_small_ct<kF16, BPG, 1>(a, s);
  }
  if (a.lam) return a.terms == 2 ? launch_rows<kScaled, BPG, 2>(a, s) : launch_rows<kScaled, BPG, 1>(a, s);
  return a.dtype == kBf16 ? launch_rows<kBf16, BPG, 1>(a, s) : launch_rows<kF16, BPG, 1>(a, s);
}

}  // namespace

W4a16Plan plan_w4a16(int M, int K, int N, int r, int batch, int group, bool smooth, int y_dtype) {
  W4a16Plan p;
  p.terms = smooth && y_dtype != kBf16 ? 2 : 1;
  const int groups = K / group, m16 = ceil_div(M, kTile) * kTile;
  // 32 slices of whole groups, more where one would not fit the LDS
  p.slice = std::min(ceil_div(groups, 32), kPrepChannels / group) * group;
  p.u_slices = ceil_div(K, p.slice);
  const int tiles = ceil_div(N, kTile);
  // Every workgroup of the small form prepares all rows, which many workgroups repeat: 4
  // rows with lambda and rank 16 at 4096 x 4096 take 13.3 us that way and 14.2 the
  // other, 4096 x 65536 89 and 47.  (LDS: that of its widest kernel.)
  p.small = M <= kSmallRows && (M == 1 || (long long)M * tiles * batch <= 2048) &&
            small_lds(M, K, r, true, p.terms, 4, group / kGroup, 1024).total * sizeof(float) <= kSmallLds;
  if (p.small) {
    // U in every workgroup reads K r numbers each: it pays while M K r is small and the
    // workgroups, with up to four tiles each, are all at work at once.  4096 x 4096, M = 1:
    // 6.7 us for rank 4, 9.0 for 16, against 10.5 with a launch before it; M = 4 with rank
    // 16 16.0 against 13.3.  One tile each otherwise (4096 x 12288 without a rank branch:
    // 7.3 us, two 8.5, four 9.7).
    if ((long long)M * K * r <= 65536)
      for (int ct = 4; r > 0 && ct >= 1 && ceil_div(tiles, ct) * batch <= kCUs; --ct) {
        p.own_u = true;
        p.ct = ct;
      }
    p.total = r > 0 && !p.own_u ? align_up((size_t)p.u_slices * batch * r * m16 * sizeof(float), 256) : 0;
    return p;
  }
  // Parts of K until there is a workgroup per compute unit.  They cost a launch, so none
  // has fewer than eight pairs (16 x 1024 x 4096 takes 4.9 us whole and 6.3 in two, 8 x
  // 4096 x 1024 8.2 and in four 6.4), or about four where that launch then has the rank
  // branch (37 x 1088 x 1000, rank 5: 16.9 whole, 14.1 in three, and 12.5 since L1 is
  // read in order; 16 x 512 x 1024, rank 8: 8.7 whole, 10.0 in two).
  const int wgs = ceil_div(tiles, kColumnTiles) * batch * (M <= kTile ? 1 : ceil_div(M, 2 * kTile));
  p.splits = std::max(1, std::min({kW4a16Splits, kCUs / wgs, r > 0 ? ceil_div(K, 8 * kGroup) : K / (16 * kGroup)}));
  size_t off = 0;
  if (smooth) {
    p.hi_off = off;
    off = align_up(off + (size_t)M * K * 2, 256);
    p.lo_off = off;
    if (p.terms == 2) off = align_up(off + (size_t)M * K * 2, 256);
    p.es_off = off;
    off = align_up(off + (size_t)m16 * groups * sizeof(float), 256);
  }
  p.uw_off = off;
  off = align_up(off + (size_t)p.u_slices * batch * r * m16 * sizeof(float), 256);
  p.part_off = off;
  if (p.splits > 1) off = align_up(off + (size_t)p.splits * batch * M * N * sizeof(float), 256);
  p.total = off;
  return p;
}

hipError_t launch_w4a16(const W4a16Args &a, hipStream_t s) {
  hipError_t e = hipSuccess;
  if (a.small ? a.r > 0 && !a.own_u : a.lam || a.r > 0) {
    const size_t lds = (size_t)kPrepRows * (a.slice + kPrepThreads) * sizeof(float);
    auto kernel = a.r == 4 ? k_w4a16_prep<4> : a.r == 8 ? k_w4a16_prep<8> : a.r == 16 ? k_w4a16_prep<16> : a.r == 32 ? k_w4a16_prep<32> : k_w4a16_prep<0>;
    hipLaunchKernelGGL(kernel, dim3((unsigned)ceil_div(a.K, a.slice), (unsigned)ceil_div(a.M, kPrepRows), (unsigned)(a.r ? a.batch : 1)),
                       dim3(kPrepThreads), lds, s, a);
    e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  e = a.bpg == 2 ? launch_bpg<2>(a, s) : launch_bpg<1>(a, s);
  if (e == hipSuccess && a.splits > 1) {
    hipLaunchKernelGGL(k_w4a16_join, dim3((unsigned)ceil_div(a.N, 256), (unsigned)a.M, (unsigned)a.batch), dim3(256), 0, s, a);
    e = hipGetLastError();
  }
  return e;
}

}  // namespace hsq
