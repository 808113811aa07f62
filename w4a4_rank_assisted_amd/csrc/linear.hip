// linear.hip -- the 16-bit linear layer with bias, activation and residual in
// its epilogue, and its backward products.
//
//   Z = X W + b,  Y = act(Z) + R
//   dZ = dY act'(Z),  dX = dZ W^T,  dW = X^T dZ,  db = sum over rows of dZ
//
// All three products are one kernel, k_lin_gemm: out(i, j) = sum_r A(i, r)
// B(r, j) on the 16x16x32 MFMA, where each operand is stored either with r
// contiguous (X in X W, both operands of dZ W^T) or with r as its rows (W in
// X W, both operands of X^T dZ).  Both kinds travel to LDS unchanged by
// direct-to-LDS loads; the second kind is transposed on the way into the
// registers by the transposing LDS read.  Few rows (M <= 64) of the forward
// product stream the weights instead (k_lin_skinny).
#include "hsq_internal.h"

#include <algorithm>

namespace hsq {

namespace {

typedef __bf16 v8bf __attribute__((ext_vector_type(8)));
typedef _Float16 v8h __attribute__((ext_vector_type(8)));
typedef short v4s __attribute__((ext_vector_type(4)));
struct __attribute__((packed, aligned(2))) U16 { uint32_t d[4]; };   // 16 bytes at any element
struct __attribute__((packed, aligned(4))) F32x4 { float f[4]; };

template <int DT>
__device__ __forceinline__ v4f mfma(v4u a, v4u b, v4f c) {
  if constexpr (DT == kBf16)
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(v8bf, a), __builtin_bit_cast(v8bf, b), c, 0, 0, 0);
  else
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(v8h, a), __builtin_bit_cast(v8h, b), c, 0, 0, 0);
}

template <int DT>
__device__ __forceinline__ float half_to_f32(uint32_t h) {
  return DT == kBf16 ? bf16_to_f32(h) : f16_to_f32((uint16_t)h);
}
template <int DT>
__device__ __forceinline__ uint32_t f32_to_half(float f) {
  if constexpr (DT == kBf16) return __builtin_bit_cast(uint16_t, (__bf16)f);
  return f32_to_f16(f);
}

// ---------------------------------------------------------------- activations
// Sigmoid from one exponential: p = 1 / (1 + e), e = exp(-x); its complement
// is 1 - p = e p.  The hardware exp2 and reciprocal are good to about one
// unit in the last place; the argument's rounding adds |x| 2^-24.
__device__ __forceinline__ float exp_neg(float x) { return __builtin_amdgcn_exp2f(x * -1.44269504f); }
__device__ __forceinline__ float sigmoid(float x) { return __builtin_amdgcn_rcpf(1.0f + exp_neg(x)); }

// z, its magnitude at most lim (NaN stays NaN).  The derivatives are 0 or 1 to
// within 2^-80 beyond the limits below, where the products of their terms would
// leave fp32.
__device__ __forceinline__ float limited(float z, float lim) { return fabsf(z) > lim ? copysignf(lim, z) : z; }

constexpr float kG0 = 1.5957691216f;     // 2 sqrt(2 / pi)
constexpr float kG1 = 0.0713548162726f;  // 2 sqrt(2 / pi) 0.044715

__device__ __forceinline__ float act_fwd(float z, int act) {
  if (act == kActGeluTanh)               // 0.5 (1 + tanh u) = sigmoid(2 u)
    return z * sigmoid(z * fmaf(kG1, z * z, kG0));
  if (act == kActGelu) return 0.5f * z * (1.0f + erff(z * 0.70710678f));
  if (act == kActSilu) return z * sigmoid(z);
  return z;
}
__device__ __forceinline__ float act_grad(float z, int act) {
  if (act == kActGeluTanh) {             // 2 u(-10) = 87, so e stays finite
    z = limited(z, 10.0f);
    const float z2 = z * z, e = exp_neg(z * fmaf(kG1, z2, kG0)), p = __builtin_amdgcn_rcpf(1.0f + e);
    return fmaf(z * fmaf(3.0f * kG1, z2, kG0), e * p * p, p);
  }
  if (act == kActGelu)
    return fmaf(z * 0.39894228f, __builtin_amdgcn_exp2f(z * z * -0.72134752f), 0.5f * (1.0f + erff(z * 0.70710678f)));
  if (act == kActSilu) {
    z = limited(z, 64.0f);
    const float e = exp_neg(z), p = __builtin_amdgcn_rcpf(1.0f + e);
    return fmaf(z, e * p * p, p);
  }
  return 1.0f;
}

// ---------------------------------------------------------------- epilogue
// NV consecutive values (8 or 16) of output row i from column j on: bias,
// Z, activation, residual, store.  Rows of any length: 16-byte accesses at
// any element where the run lies inside the row, single elements at its end.
template <int DT, int NV>
__device__ __forceinline__ void finish(const LinGemm &a, int i, int j, const float *bias, float *v) {
  const size_t o = (size_t)i * a.J + j;
  const int n = a.J - j;
  if (n <= 0) return;
  if (a.bias) {
#pragma unroll
    for (int e = 0; e < NV; ++e) v[e] += bias[e];
  }
  auto store_half = [&](uint16_t *p) __attribute__((always_inline)) {
    if (n >= NV) {
#pragma unroll
      for (int c = 0; c < NV / 8; ++c) {
        U16 t;
#pragma unroll
        for (int e = 0; e < 4; ++e)
          t.d[e] = f32_to_half<DT>(v[8 * c + 2 * e]) | (f32_to_half<DT>(v[8 * c + 2 * e + 1]) << 16);
        *reinterpret_cast<U16 *>(p + o + 8 * c) = t;
      }
    } else {
#pragma unroll
      for (int e = 0; e < NV; ++e)
        if (e < n) p[o + e] = (uint16_t)f32_to_half<DT>(v[e]);
    }
  };
  if (a.Z) store_half(a.Z);
  if (a.act == kActGeluTanh) {
#pragma unroll
    for (int e = 0; e < NV; ++e) v[e] = act_fwd(v[e], kActGeluTanh);
  } else if (a.act == kActGelu) {
#pragma unroll
    for (int e = 0; e < NV; ++e) v[e] = act_fwd(v[e], kActGelu);
  } else if (a.act == kActSilu) {
#pragma unroll
    for (int e = 0; e < NV; ++e) v[e] = act_fwd(v[e], kActSilu);
  }
  if (a.out_f32) {
    const float *r = static_cast<const float *>(a.res);
    float *y = static_cast<float *>(a.out);
    if (n >= NV) {
#pragma unroll
      for (int c = 0; c < NV / 4; ++c) {
        F32x4 t;
        if (r) {
          t = *reinterpret_cast<const F32x4 *>(r + o + 4 * c);
#pragma unroll
          for (int e = 0; e < 4; ++e) v[4 * c + e] += t.f[e];
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) t.f[e] = v[4 * c + e];
        *reinterpret_cast<F32x4 *>(y + o + 4 * c) = t;
      }
    } else {
#pragma unroll
      for (int e = 0; e < NV; ++e)
        if (e < n) y[o + e] = r ? v[e] + r[o + e] : v[e];
    }
    return;
  }
  if (a.res) {
    const uint16_t *r = static_cast<const uint16_t *>(a.res);
    if (n >= NV) {
#pragma unroll
      for (int c = 0; c < NV / 8; ++c) {
        const U16 t = *reinterpret_cast<const U16 *>(r + o + 8 * c);
#pragma unroll
        for (int e = 0; e < 8; ++e) v[8 * c + e] += half_to_f32<DT>((t.d[e / 2] >> (16 * (e & 1))) & 0xFFFFu);
      }
    } else {
#pragma unroll
      for (int e = 0; e < NV; ++e)
        if (e < n) v[e] += half_to_f32<DT>(r[o + e]);
    }
  }
  store_half(static_cast<uint16_t *>(a.out));
}

template <int DT, int NV>
__device__ __forceinline__ void load_bias(const LinGemm &a, int j, float *b) {
#pragma unroll
  for (int e = 0; e < NV; ++e) b[e] = a.bias && j + e < a.J ? half_to_f32<DT>(a.bias[j + e]) : 0.0f;
}

int part_ld(int J) { return ceil_div(J, 16) * 16; }   // row stride of the fp32 partial sums

// ---------------------------------------------------------------- tiled product
// Workgroup tile TI x TJ, WI x WJ waves of (16 NI) x (16 NJ) each, BK of the
// reduction per stage, NS stage buffers in LDS.
template <int TI_, int TJ_, int WI_, int WJ_, int BK_, int NS_, int MINW_>
struct Cfg {
  static constexpr int TI = TI_, TJ = TJ_, WI = WI_, WJ = WJ_, BK = BK_, NS = NS_, MINW = MINW_;
  static constexpr int NW = WI * WJ, NT = 64 * NW, NI = TI / WI / 16, NJ = TJ / WJ / 16;
  static constexpr int kA = TI * BK * 2, kB = TJ * BK * 2;          // stage bytes
  static constexpr int PA = kA / 1024 / NW, PB = kB / 1024 / NW;    // 1 KB loads per wave and stage
  static_assert(NJ == 4, "a lane holds 16 consecutive columns");
  static_assert(PA * NW * 1024 == kA && PB * NW * 1024 == kB, "whole loads per wave");
};

// Position of a 16-byte chunk in a staged row.
//
// r-contiguous operand: rows of BK elements (4 or 8 chunks), read 16 rows
// at a time, one chunk each.  The rows of one read are consecutive (A) or
// four runs of four, 16 rows apart (B, see the output layout below); the XOR
// moves them to 16 different chunk positions of 256 bytes.
template <int BK, bool ISB>
__device__ __forceinline__ int swz_cont(int row) {
  if constexpr (BK == 32) return ISB ? (row >> 4) & 3 : (row >> 2) & 3;
  return ISB ? ((row >> 1) & 1) | (((row >> 4) & 3) << 1) : (row >> 1) & 7;
}
// r-strided operand: rows of TI or TJ elements.  A transposing read of 16
// lanes touches four rows (r = 8 g + jt) at two adjacent chunks (A) or at
// four chunks two apart (B).
template <bool ISB>
__device__ __forceinline__ int swz_strided(int r) {
  if constexpr (ISB) return (r & 1) | (((r >> 1) & 1) << 3);
  return 2 * ((r & 3) | (((r >> 3) & 1) << 2));
}

// Operand staging of one workgroup: this wave's P direct-to-LDS loads of a
// stage.  Rows past the matrix and r past R read zero (an offset beyond the
// buffer); the chunks past the last column of an r-strided operand only reach
// output columns that are not stored.
template <int T, int BK, int P, bool STRIDED, bool ISB>
struct Stager {
  v4u rs;
  uint32_t voff[P];
  int ld, R, n, x0, wave, lane;
  static constexpr uint32_t kBad = 0x80000000u;   // operands are below 2^31 bytes
  static constexpr int CPR = STRIDED ? T / 8 : BK / 8;   // chunks of a staged row
  static constexpr int RPL = 64 / CPR > 0 ? 64 / CPR : 1;   // staged rows per 1 KB load
  static_assert(CPR <= 64, "a load covers whole staged rows");

  __device__ __forceinline__ void init(const uint16_t *p, int n_, int x0_, int R_, int ld_, int w, int l) {
    ld = ld_; R = R_; n = n_; x0 = x0_; wave = w; lane = l;
    rs = raw_rsrc(p, (uint32_t)((size_t)(STRIDED ? R : n) * ld * 2));
#pragma unroll
    for (int u = 0; u < P; ++u) voff[u] = offset(u, 0, false);
  }
  // byte offset of this lane's chunk of load u, stage start r0 (0: the start is
  // in the scalar offset); `tail` tests r against R
  __device__ __forceinline__ uint32_t offset(int u, int r0, bool tail) const {
    const int row = (wave * P + u) * RPL + lane / CPR, pos = lane % CPR;
    if constexpr (STRIDED) {
      const int col = x0 + 8 * (pos ^ swz_strided<ISB>(row));
      if (col >= n || (tail && r0 + row >= R)) return kBad;
      return ((uint32_t)row * (uint32_t)ld + (uint32_t)col) * 2u;
    } else {
      const int k = 8 * (pos ^ swz_cont<BK, ISB>(row));
      if (x0 + row >= n || (tail && r0 + k >= R)) return kBad;
      return ((uint32_t)(x0 + row) * (uint32_t)ld + (uint32_t)k) * 2u;
    }
  }
  __device__ __forceinline__ void issue(int r0, uint32_t lds) const {
    const uint32_t soff = (uint32_t)r0 * (STRIDED ? (uint32_t)ld * 2u : 2u);
    const uint32_t dst = lds + (uint32_t)(wave * P) * 1024u;
    if (r0 + BK <= R) {
#pragma unroll
      for (int u = 0; u < P; ++u) block_to_lds(rs, dst + u * 1024, voff[u], soff);
    } else {
#pragma unroll
      for (int u = 0; u < P; ++u) block_to_lds(rs, dst + u * 1024, offset(u, r0, true), soff);
    }
  }
};

template <int N>
__device__ __forceinline__ void stage_wait() {   // all but this wave's N newest loads, its LDS reads, the workgroup
  asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(N) : "memory");
}

template <class C, int DT, bool ASTR, bool BSTR, bool PART>
__global__ __launch_bounds__(C::NT, C::MINW) void k_lin_gemm(LinGemm a) {
  struct alignas(16) Stage { char a[C::kA]; char b[C::kB]; };
  __shared__ Stage sm[C::NS];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wi = wave / C::WJ, wj = wave % C::WJ;
  const int nbi = (a.I + C::TI - 1) / C::TI, nbj = (a.J + C::TJ - 1) / C::TJ;
  int bi, bj;
  xcd_tile_of(blockIdx.x, nbj, nbi, 4, bi, bj);
  const int i0 = bi * C::TI, j0 = bj * C::TJ;
  const int nst = (a.R + C::BK - 1) / C::BK, z = PART ? (int)blockIdx.y : 0;
  const int s0 = PART ? (int)((long long)z * nst / a.splits) : 0;
  const int s1 = PART ? (int)((long long)(z + 1) * nst / a.splits) : nst;

  Stager<C::TI, C::BK, C::PA, ASTR, false> la;
  Stager<C::TJ, C::BK, C::PB, BSTR, true> lb;
  la.init(a.A, a.I, i0, a.R, a.lda, wave, lane);
  lb.init(a.B, a.J, j0, a.R, a.ldb, wave, lane);

  // Operand reads.  MFMA operand lane l holds row l % 16 and r = 8 (l / 16) ..
  // + 7 of the 32.  The product is formed transposed: the MFMA's row operand
  // is B, its column operand A, so lane l of a result holds output row l %
  // 16 and, in its four registers, MFMA rows 4 g .. 4 g + 3 (g = l / 16).
  // MFMA row rr of column tile jj is output column 16 (rr / 4) + 4 jj + rr %
  // 4 of the wave's 64, so a lane's four tiles are 16 consecutive columns.
  const int g = lane >> 4, rr = lane & 15, jt = rr >> 2, q = rr & 3;
  uint32_t oa[ASTR ? C::NI : 2], ob[2];
  if constexpr (ASTR) {
    // lane 4 jt + q of a transposing read addresses r = 8 g + jt (then + 4)
    // and columns 4 q .. 4 q + 3; lane i gets column i of the 16
#pragma unroll
    for (int i = 0; i < C::NI; ++i) {
      const int ch = (wi * 16 * C::NI + 16 * i) / 8 + (q >> 1);
      oa[i] = (uint32_t)((8 * g + jt) * C::TI * 2 + (ch ^ swz_strided<false>(8 * g + jt)) * 16 + (q & 1) * 8);
    }
  } else {
    const int row = wi * 16 * C::NI + rr;
#pragma unroll
    for (int h = 0; h < 2; ++h) oa[h] = (uint32_t)(row * C::BK * 2 + (((4 * h + g) & (C::BK / 8 - 1)) ^ swz_cont<C::BK, false>(row)) * 16);
  }
  if constexpr (BSTR) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int ch = wj * 8 + 2 * q + h;
      ob[h] = (uint32_t)((8 * g + jt) * C::TJ * 2 + (ch ^ swz_strided<true>(8 * g + jt)) * 16);
    }
  } else {
    const int row = wj * 64 + 16 * (rr >> 2) + (rr & 3);
#pragma unroll
    for (int h = 0; h < 2; ++h) ob[h] = (uint32_t)(row * C::BK * 2 + (((4 * h + g) & (C::BK / 8 - 1)) ^ swz_cont<C::BK, true>(row)) * 16);
  }
  auto tr = [&](const char *p) __attribute__((always_inline)) -> v2u {
    return __builtin_bit_cast(v2u, __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) v4s *)p));
  };
  auto read_a = [&](const char *p, int i, int kk) __attribute__((always_inline)) -> v4u {
    if constexpr (ASTR) {
      const char *b = p + oa[i] + kk * 32 * C::TI * 2;
      const v2u lo = tr(b), hi = tr(b + 4 * C::TI * 2);
      return (v4u){lo[0], lo[1], hi[0], hi[1]};
    } else {
      return *reinterpret_cast<const v4u *>(p + oa[kk] + i * 16 * C::BK * 2);
    }
  };
  auto read_b = [&](const char *p, int jj, int kk) __attribute__((always_inline)) -> v4u {
    if constexpr (BSTR) {
      const char *b = p + ob[jj >> 1] + (jj & 1) * 8 + kk * 32 * C::TJ * 2;
      const v2u lo = tr(b), hi = tr(b + 4 * C::TJ * 2);
      return (v4u){lo[0], lo[1], hi[0], hi[1]};
    } else {
      return *reinterpret_cast<const v4u *>(p + ob[kk] + jj * 4 * C::BK * 2);
    }
  };

  v4f acc[C::NI][C::NJ];
#pragma unroll
  for (int i = 0; i < C::NI; ++i)
#pragma unroll
    for (int j = 0; j < C::NJ; ++j) acc[i][j] = (v4f){0.0f, 0.0f, 0.0f, 0.0f};

  auto issue = [&](int s, int buf) __attribute__((always_inline)) {
    la.issue(s * C::BK, lds_addr(sm[buf].a));
    lb.issue(s * C::BK, lds_addr(sm[buf].b));
  };
  // NS - 1 stages ahead.  At stage s's barrier every wave has its loads of
  // stage s and its reads of stage s - 1 behind it, so the loads issued after
  // it may overwrite the buffer of stage s - 1 = s + NS - 1 (mod NS).
#pragma unroll
  for (int p = 0; p < C::NS - 1; ++p)
    if (s0 + p < s1) issue(s0 + p, p);
  int buf = 0;
  for (int s = s0; s < s1; ++s) {
    if (s + C::NS - 2 < s1) stage_wait<(C::NS - 2) * (C::PA + C::PB)>();
    else stage_wait<0>();
    if (s + C::NS - 1 < s1) issue(s + C::NS - 1, buf == 0 ? C::NS - 1 : buf - 1);
    const char *pa = sm[buf].a, *pb = sm[buf].b;
#pragma unroll
    for (int kk = 0; kk < C::BK / 32; ++kk) {
      v4u fa[C::NI], fb[C::NJ];
#pragma unroll
      for (int j = 0; j < C::NJ; ++j) fb[j] = read_b(pb, j, kk);
#pragma unroll
      for (int i = 0; i < C::NI; ++i) fa[i] = read_a(pa, i, kk);
#pragma unroll
      for (int i = 0; i < C::NI; ++i)
#pragma unroll
        for (int j = 0; j < C::NJ; ++j) acc[i][j] = mfma<DT>(fb[j], fa[i], acc[i][j]);
    }
    buf = buf + 1 == C::NS ? 0 : buf + 1;
  }

  const int j = j0 + wj * 64 + 16 * g;
  if constexpr (PART) {
    const int ld = (a.J + 15) / 16 * 16;
    if (j < a.J) {
      float *dst = a.part + (size_t)z * a.I * ld + j;
#pragma unroll
      for (int i = 0; i < C::NI; ++i) {
        const int row = i0 + wi * 16 * C::NI + 16 * i + rr;
        if (row < a.I)
#pragma unroll
          for (int jj = 0; jj < C::NJ; ++jj) *reinterpret_cast<v4f *>(dst + (size_t)row * ld + 4 * jj) = acc[i][jj];
      }
    }
  } else {
    float bias[16];
    load_bias<DT, 16>(a, j, bias);
#pragma unroll
    for (int i = 0; i < C::NI; ++i) {
      const int row = i0 + wi * 16 * C::NI + 16 * i + rr;
      float v[16];
#pragma unroll
      for (int e = 0; e < 16; ++e) v[e] = acc[i][e >> 2][e & 3];
      if (row < a.I) finish<DT, 16>(a, row, j, bias, v);
    }
  }
}

// Sums the splits' partial sums in split order and finishes eight columns per thread.
template <int DT>
__global__ __launch_bounds__(256) void k_lin_reduce(LinGemm a) {
  const int ld = (a.J + 15) / 16 * 16, cols = (a.J + 7) / 8;
  const long long t = (long long)blockIdx.x * 256 + threadIdx.x;
  if (t >= (long long)a.I * cols) return;
  const int i = (int)(t / cols), j = (int)(t % cols) * 8;
  const float *p = a.part + (size_t)i * ld + j;
  float v[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) v[e] = 0.0f;
  for (int z = 0; z < a.splits; ++z, p += (size_t)a.I * ld) {
    const v4f lo = *reinterpret_cast<const v4f *>(p), hi = *reinterpret_cast<const v4f *>(p + 4);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      v[e] += lo[e];
      v[4 + e] += hi[e];
    }
  }
  float bias[8];
  load_bias<DT, 8>(a, j, bias);
  finish<DT, 8>(a, i, j, bias, v);
}

// ---------------------------------------------------------------- few rows
// Y of up to 16 MT rows, bound by the one read of W.  A workgroup owns 128
// columns and a share of K; its four waves split that share in runs of 32.
// Lane l loads, for its 8 rows k = 8 (l / 16) .. + 7 of a run, the 8
// columns 8 (l % 16) .. + 7 (16 bytes each, a row's 128 columns are 256
// consecutive bytes), transposes the 8 x 8 block in registers (32 byte
// permutes), and has the MFMA operands of 8 column tiles: tile j holds
// columns 8 c + j.  W never passes through LDS.  The result lane holds row
// l % 16 and 32 consecutive columns.
constexpr int kSkCols = 128, kSkWaves = 4;

template <int DT, int MT, bool PART>
__global__ __launch_bounds__(64 * kSkWaves) void k_lin_skinny(LinGemm a) {
  __shared__ float red[kSkWaves][16][kSkCols + 4];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int g = lane >> 4, c = lane & 15;
  const int j0 = blockIdx.x * kSkCols, jc = j0 + 8 * c;
  const int runs = (a.R + 31) / 32, shares = PART ? a.splits : 1, z = PART ? (int)blockIdx.y : 0;
  // runs [r0, r1) of this share, dealt to the waves in turn
  const int r0 = (int)((long long)z * runs / shares), r1 = (int)((long long)(z + 1) * runs / shares);
  v4f acc[MT][8];
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int j = 0; j < 8; ++j) acc[m][j] = (v4f){0.0f, 0.0f, 0.0f, 0.0f};

  const bool whole = jc + 8 <= a.J;
  auto load = [&](int run, U16 (&w)[8]) __attribute__((always_inline)) {
    const int k = 32 * run + 8 * g;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      w[e] = U16{{0u, 0u, 0u, 0u}};
      const uint16_t *p = a.B + (size_t)(k + e) * a.ldb + jc;
      if (k + e < a.R) {
        if (whole) {
          w[e] = *reinterpret_cast<const U16 *>(p);
        } else {
#pragma unroll
          for (int h = 0; h < 8; ++h)
            if (jc + h < a.J) w[e].d[h / 2] |= (uint32_t)p[h] << (16 * (h & 1));
        }
      }
    }
  };
  auto step = [&](int run, const U16 (&w)[8]) __attribute__((always_inline)) {
    const int k = 32 * run + 8 * g;
    v4u x[MT];
#pragma unroll
    for (int m = 0; m < MT; ++m) {
      x[m] = (v4u){0u, 0u, 0u, 0u};
      const int row = 16 * m + c;
      if (row < a.I) {
        const uint16_t *p = a.A + (size_t)row * a.lda + k;
        if (k + 8 <= a.R) {
          const U16 t = *reinterpret_cast<const U16 *>(p);
          x[m] = (v4u){t.d[0], t.d[1], t.d[2], t.d[3]};
        } else {
#pragma unroll
          for (int h = 0; h < 8; ++h)
            if (k + h < a.R) x[m][h / 2] |= (uint32_t)p[h] << (16 * (h & 1));
        }
      }
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      v4u b;   // column 8 c + j, k .. k + 7
#pragma unroll
      for (int e = 0; e < 4; ++e)
        b[e] = __builtin_amdgcn_perm(w[2 * e + 1].d[j / 2], w[2 * e].d[j / 2], (j & 1) ? 0x07060302u : 0x05040100u);
#pragma unroll
      for (int m = 0; m < MT; ++m) acc[m][j] = mfma<DT>(b, x[m], acc[m][j]);
    }
  };
  U16 w0[8], w1[8];
  int run = r0 + wave;
  if (run < r1) load(run, w0);
  while (run < r1) {
    if (run + kSkWaves < r1) load(run + kSkWaves, w1);
    step(run, w0);
    run += kSkWaves;
    if (run >= r1) break;
    if (run + kSkWaves < r1) load(run + kSkWaves, w0);
    step(run, w1);
    run += kSkWaves;
  }

  // waves summed in order, 16 rows at a time: thread t finishes row t / 16, columns 8 (t % 16) .. + 7
  const int tr = threadIdx.x >> 4, tc = 8 * (threadIdx.x & 15);
  const int ld = (a.J + 15) / 16 * 16;
  float bias[8];
  if constexpr (!PART) load_bias<DT, 8>(a, j0 + tc, bias);
#pragma unroll
  for (int m = 0; m < MT; ++m) {
    if (m > 0) __syncthreads();
    if (16 * m + c < a.I)
#pragma unroll
      for (int qq = 0; qq < 4; ++qq)
#pragma unroll
        for (int h = 0; h < 2; ++h)
          *reinterpret_cast<v4f *>(&red[wave][c][32 * g + 8 * qq + 4 * h]) =
              (v4f){acc[m][4 * h][qq], acc[m][4 * h + 1][qq], acc[m][4 * h + 2][qq], acc[m][4 * h + 3][qq]};
    __syncthreads();
    const int row = 16 * m + tr;
    if (row < a.I && j0 + tc < a.J) {
      float v[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        v[e] = red[0][tr][tc + e];
#pragma unroll
        for (int w = 1; w < kSkWaves; ++w) v[e] += red[w][tr][tc + e];
      }
      if constexpr (PART) {
        float *dst = a.part + ((size_t)z * a.I + row) * ld + j0 + tc;
        *reinterpret_cast<v4f *>(dst) = (v4f){v[0], v[1], v[2], v[3]};
        *reinterpret_cast<v4f *>(dst + 4) = (v4f){v[4], v[5], v[6], v[7]};
      } else {
        finish<DT, 8>(a, row, j0 + tc, bias, v);
      }
    }
  }
}

// ---------------------------------------------------------------- staging passes
__global__ __launch_bounds__(256) void k_pad_rows(const uint16_t *src, int rows, int cols, uint16_t *dst, int ld) {
  const long long t = (long long)blockIdx.x * 256 + threadIdx.x;
  const int cpr = ld / 8;
  if (t >= (long long)rows * cpr) return;
  const int r = (int)(t / cpr), c = (int)(t % cpr) * 8;
  const uint16_t *p = src + (size_t)r * cols + c;
  U16 v = U16{{0u, 0u, 0u, 0u}};
  if (c + 8 <= cols) {
    v = *reinterpret_cast<const U16 *>(p);
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (c + e < cols) v.d[e / 2] |= (uint32_t)p[e] << (16 * (e & 1));
  }
  *reinterpret_cast<v4u *>(dst + (size_t)r * ld + c) = (v4u){v.d[0], v.d[1], v.d[2], v.d[3]};
}

// dZ = dY act'(Z), rounded to the operand type of the two products, and the
// column sums of the unrounded dZ over a slice of the rows.  256 columns per
// workgroup: thread t takes columns 8 (t % 32) .. + 7 of rows t / 32, t / 32 +
// 8, ... of its slice.
constexpr int kDzCols = 256, kDzRows = 8;

template <int DT>
__global__ __launch_bounds__(256) void k_lin_dz(LinDz a) {
  __shared__ float red[kDzRows][kDzCols];
  const int cx = threadIdx.x & 31, ry = threadIdx.x >> 5;
  const int j = blockIdx.x * kDzCols + 8 * cx, n = a.N - j;
  const int m0 = (int)((long long)blockIdx.y * a.M / a.slices), m1 = (int)((long long)(blockIdx.y + 1) * a.M / a.slices);
  float s[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) s[e] = 0.0f;
  auto half8 = [&](const uint16_t *p, float *v) __attribute__((always_inline)) {
    if (n >= 8) {
      const U16 t = *reinterpret_cast<const U16 *>(p);
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] = half_to_f32<DT>((t.d[e / 2] >> (16 * (e & 1))) & 0xFFFFu);
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] = e < n ? half_to_f32<DT>(p[e]) : 0.0f;
    }
  };
  if (n > 0)
    for (int m = m0 + ry; m < m1; m += kDzRows) {
      const size_t o = (size_t)m * a.N + j;
      float d[8], z[8];
      if (a.dy_f32) {
        const float *p = static_cast<const float *>(a.dY) + o;
#pragma unroll
        for (int e = 0; e < 8; ++e) d[e] = e < n ? p[e] : 0.0f;
      } else {
        half8(static_cast<const uint16_t *>(a.dY) + o, d);
      }
      if (a.act != kActIdentity) {
        half8(a.Z + o, z);
        if (a.act == kActGeluTanh) {
#pragma unroll
          for (int e = 0; e < 8; ++e) d[e] *= act_grad(z[e], kActGeluTanh);
        } else if (a.act == kActGelu) {
#pragma unroll
          for (int e = 0; e < 8; ++e) d[e] *= act_grad(z[e], kActGelu);
        } else {
#pragma unroll
          for (int e = 0; e < 8; ++e) d[e] *= act_grad(z[e], kActSilu);
        }
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) s[e] += d[e];
      if (a.dZ) {
        v4u t;
#pragma unroll
        for (int e = 0; e < 4; ++e) t[e] = f32_to_half<DT>(d[2 * e]) | (f32_to_half<DT>(d[2 * e + 1]) << 16);
        *reinterpret_cast<v4u *>(a.dZ + (size_t)m * a.np + j) = t;
      }
    }
  if (!a.db) return;
#pragma unroll
  for (int e = 0; e < 8; ++e) red[ry][8 * cx + e] = s[e];
  __syncthreads();
  const int col = blockIdx.x * kDzCols + threadIdx.x;
  if (col >= a.N) return;
  float v = 0.0f;
#pragma unroll
  for (int r = 0; r < kDzRows; ++r) v += red[r][threadIdx.x];
  a.part[(size_t)blockIdx.y * a.N + col] = v;
}

// ---------------------------------------------------------------- planning
using Big = Cfg<256, 128, 2, 2, 32, 3, 2>;     // 72 KB of LDS: two workgroups per CU
using Small = Cfg<128, 128, 2, 2, 32, 3, 2>;   // few tiles

bool big_tiles(int I, int J) {
  return (long long)ceil_div(I, Big::TI) * ceil_div(J, Big::TJ) >= 256;
}

int gemm_splits(int I, int J, int R) {
  const long long tiles = big_tiles(I, J) ? (long long)ceil_div(I, Big::TI) * ceil_div(J, Big::TJ)
                                          : (long long)ceil_div(I, Small::TI) * ceil_div(J, Small::TJ);
  if (tiles >= 256) return 1;
  return (int)std::max(1LL, std::min({512 / tiles, (long long)R / 512, 16LL}));
}

int skinny_splits(int J, int K) {
  return std::max(1, std::min({512 / ceil_div(J, kSkCols), K / 256, 16}));
}

size_t part_bytes(int I, int J, int splits) {
  return splits > 1 ? (size_t)splits * I * part_ld(J) * sizeof(float) : 0;
}

template <class C, int DT, bool AS, bool BS>
hipError_t run_tiles(const LinGemm &a, hipStream_t s) {
  const unsigned tiles = (unsigned)(ceil_div(a.I, C::TI) * ceil_div(a.J, C::TJ));
  if (a.splits > 1)
    hipLaunchKernelGGL((k_lin_gemm<C, DT, AS, BS, true>), dim3(tiles, (unsigned)a.splits), dim3(C::NT), 0, s, a);
  else
    hipLaunchKernelGGL((k_lin_gemm<C, DT, AS, BS, false>), dim3(tiles), dim3(C::NT), 0, s, a);
  return hipGetLastError();
}

template <int DT, bool AS, bool BS>
hipError_t pick_tiles(const LinGemm &a, hipStream_t s) {
  return big_tiles(a.I, a.J) ? run_tiles<Big, DT, AS, BS>(a, s) : run_tiles<Small, DT, AS, BS>(a, s);
}

template <int DT, int MT>
hipError_t run_skinny(const LinGemm &a, hipStream_t s) {
  const unsigned strips = (unsigned)ceil_div(a.J, kSkCols);
  if (a.splits > 1)
    hipLaunchKernelGGL((k_lin_skinny<DT, MT, true>), dim3(strips, (unsigned)a.splits), dim3(64 * kSkWaves), 0, s, a);
  else
    hipLaunchKernelGGL((k_lin_skinny<DT, MT, false>), dim3(strips), dim3(64 * kSkWaves), 0, s, a);
  return hipGetLastError();
}

template <int DT>
hipError_t run_linear(const LinGemm &a, bool skinny, hipStream_t s) {
  hipError_t e;
  if (skinny) {
    const int mt = ceil_div(a.I, 16);
    e = mt == 1 ? run_skinny<DT, 1>(a, s) : mt == 2 ? run_skinny<DT, 2>(a, s)
        : mt == 3 ? run_skinny<DT, 3>(a, s) : run_skinny<DT, 4>(a, s);
  } else if (a.b_rows) {
    e = a.a_rows ? pick_tiles<DT, true, true>(a, s) : pick_tiles<DT, false, true>(a, s);
  } else {
    e = pick_tiles<DT, false, false>(a, s);
  }
  if (e != hipSuccess || a.splits <= 1) return e;
  const long long items = (long long)a.I * ceil_div(a.J, 8);
  hipLaunchKernelGGL(k_lin_reduce<DT>, dim3((unsigned)((items + 255) / 256)), dim3(256), 0, s, a);
  return hipGetLastError();
}

}  // namespace

LinPlan plan_linear(int M, int K, int N) {
  LinPlan p;
  p.kp = ceil_div(K, 8) * 8;
  p.np = ceil_div(N, 8) * 8;
  p.skinny = M <= kLinSkinnyMaxM;
  p.splits = p.skinny ? skinny_splits(N, K) : gemm_splits(M, N, K);
  p.pad_x = !p.skinny && p.kp != K;
  p.pad_w = !p.skinny && p.np != N;
  size_t off = 0;
  p.x_off = off;
  if (p.pad_x) off = align_up(off + (size_t)M * p.kp * 2, 256);
  p.w_off = off;
  if (p.pad_w) off = align_up(off + (size_t)K * p.np * 2, 256);
  p.part_off = off;
  off = align_up(off + part_bytes(M, N, p.splits), 256);
  p.total = off;
  return p;
}

LinPlan plan_linear_backward(int M, int K, int N) {
  LinPlan p;
  p.kp = ceil_div(K, 8) * 8;
  p.np = ceil_div(N, 8) * 8;
  p.pad_x = p.kp != K;
  p.pad_w = p.np != N;
  p.splits_dx = gemm_splits(M, K, N);
  p.splits_dw = gemm_splits(K, N, M);
  // row slices of the dZ pass: about 1024 workgroups, at least 32 rows each
  p.slices = std::max(1, std::min(1024 / ceil_div(p.np, kDzCols), ceil_div(M, 32)));
  size_t off = 0;
  p.x_off = off;
  if (p.pad_x) off = align_up(off + (size_t)M * p.kp * 2, 256);
  p.w_off = off;
  if (p.pad_w) off = align_up(off + (size_t)K * p.np * 2, 256);
  p.dz_off = off;
  off = align_up(off + (size_t)M * p.np * 2, 256);
  p.db_off = off;
  off = align_up(off + (size_t)p.slices * N * sizeof(float), 256);
  p.part_off = off;
  off = align_up(off + std::max(part_bytes(M, K, p.splits_dx), part_bytes(K, N, p.splits_dw)), 256);
  p.total = off;
  return p;
}

hipError_t launch_linear(const LinGemm &a, bool skinny, hipStream_t s) {
  return a.dtype == kBf16 ? run_linear<kBf16>(a, skinny, s) : run_linear<kF16>(a, skinny, s);
}

hipError_t launch_pad_rows(const uint16_t *src, int rows, int cols, uint16_t *dst, int ld, hipStream_t s) {
  const long long items = (long long)rows * (ld / 8);
  hipLaunchKernelGGL(k_pad_rows, dim3((unsigned)((items + 255) / 256)), dim3(256), 0, s, src, rows, cols, dst, ld);
  return hipGetLastError();
}

hipError_t launch_linear_dz(const LinDz &a, hipStream_t s) {
  const dim3 grid((unsigned)ceil_div(a.np, kDzCols), (unsigned)a.slices);
  if (a.dtype == kBf16) hipLaunchKernelGGL(k_lin_dz<kBf16>, grid, dim3(256), 0, s, a);
  else hipLaunchKernelGGL(k_lin_dz<kF16>, grid, dim3(256), 0, s, a);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || !a.db) return e;
  return launch_sum_parts(a.part, (size_t)a.N, a.slices, 1, a.N, a.db, a.dtype, s);
}

}  // namespace hsq
