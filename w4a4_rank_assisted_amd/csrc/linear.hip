// linear.hip -- the 16-bit linear layer with bias, activation and residual in
// its epilogue, and its backward products.
//
//   Z = X W + b,  Y = act(Z) + R
//   dZ = dY act'(Z),  dX = dZ W^T,  dW = X^T dZ,  db = sum over rows of dZ
//
// All three products are one device function, lin_tile: out(i, j) = sum_r
// A(i, r) B(r, j) on the 16x16x32 MFMA, where each operand is stored either
// with r contiguous (X in X W, both operands of dZ W^T) or with r as its rows
// (W in X W, both operands of X^T dZ).  Both kinds travel to LDS unchanged by
// direct-to-LDS loads; the second kind is transposed on the way into the
// registers by the transposing LDS read.  Few rows (M <= 48) of the forward
// product stream the weights instead (k_lin_skinny).
//
// What bounds them (MI355X; torch's copy of 2 GiB runs at 4.92 TB/s, its bf16
// product of 8192^3 at 1230 TFLOP/s; other boxes gave 5.1 and 1330):
//   - many tokens: power and the feeding of the matrix cores.  2048 x 4096 x 12288
//     with silu takes 175-191 us (1080-1180 TFLOP/s); 4096 x 8192 x 8192, two
//     whole rounds of tiles, runs at 1.93 GHz with the matrix cores busy for 63 %
//     of the cycles and waits in 28 % of the waves' (without loads and LDS reads:
//     2.10 GHz, 82 % busy); on zeros it runs a quarter faster, and deeper
//     buffers, fewer barriers or staging through registers change nothing.  The
//     two gradients of 2048 x 12288 x 4096 take 350-375 us.
//   - one to 48 tokens forward: the read of W.  1 x 4096 x 12288: 21.3 us, 4.7
//     TB/s; 16 x 12288 x 4096 with residual: 23.3 us, 4.35 TB/s, the second
//     launch 4 us of it.
//   - 49 to some 200 tokens, and the gradients of few rows: tiles of 128 rows for
//     few of them.  64 x 4096 x 12288: 46 us, gradients of 6 x 8768 x 9471: 192,
//     two and three times what their bytes take.
//   - small ones: their launches.  333 x 1001 x 777 in two: 15-15.5 us in bf16
//     without an epilogue, 16.8 in fp16 with GELU, residual and fp32 Y.
#include "hsq_internal.h"

#include <algorithm>

namespace hsq {

namespace {

typedef __bf16 v8bf __attribute__((ext_vector_type(8)));
typedef _Float16 v8h __attribute__((ext_vector_type(8)));
typedef short v4s __attribute__((ext_vector_type(4)));
// 16 bytes at any element: global memory takes them as they come
typedef uint32_t U16 __attribute__((ext_vector_type(4), aligned(2)));
typedef float F32x4 __attribute__((ext_vector_type(4), aligned(4)));

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
  if (act == kActGelu) {                 // an infinite Z has slope 0 or 1 too
    z = limited(z, 16.0f);
    return fmaf(z * 0.39894228f, __builtin_amdgcn_exp2f(z * z * -0.72134752f), 0.5f * (1.0f + erff(z * 0.70710678f)));
  }
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
          t[e] = f32_to_half<DT>(v[8 * c + 2 * e]) | (f32_to_half<DT>(v[8 * c + 2 * e + 1]) << 16);
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
          for (int e = 0; e < 4; ++e) v[4 * c + e] += t[e];
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) t[e] = v[4 * c + e];
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
        for (int e = 0; e < 8; ++e) v[8 * c + e] += half_to_f32<DT>((t[e / 2] >> (16 * (e & 1))) & 0xFFFFu);
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
// Workgroup tile TI x TJ, WI x WJ waves of (16 NI) x 64 each, 32 of the
// reduction per stage, NS stage buffers in LDS.
constexpr int BK = 32;

template <int TI_, int TJ_, int WI_, int WJ_, int NS_>
struct Cfg {
  static constexpr int TI = TI_, TJ = TJ_, WI = WI_, WJ = WJ_, NS = NS_;
  static constexpr int NW = WI * WJ, NI = TI / WI / 16, NJ = TJ / WJ / 16;
  static constexpr int kA = TI * BK * 2, kB = TJ * BK * 2;          // stage bytes
  static constexpr int PA = kA / 1024 / NW, PB = kB / 1024 / NW;    // 1 KB loads per wave and stage
  static_assert(NW == 8 && NJ == 4, "eight waves; a lane holds 16 consecutive columns");
  static_assert(PA * NW * 1024 == kA && PB * NW * 1024 == kB, "whole loads per wave");
};

using Big = Cfg<256, 256, 2, 4, 4>;
using Half = Cfg<256, 128, 4, 2, 5>;
using Quarter = Cfg<128, 128, 4, 2, 8>;
constexpr int kLinLds = 131072;   // four, five and eight stages of these: one workgroup per CU

// Position of a 16-byte chunk in a staged row.
//
// r-contiguous operand: rows of BK elements (4 chunks), 16 rows read at a
// time, one chunk each.  The LDS serves a 16-byte read in four turns of 16
// lanes, which are not the lanes of one chunk column: lanes 0-3, 12-15 and
// 20-27 share a turn, 4-11, 16-19 and 28-31 the next.  With quad t of
// four rows at chunk c ^ f(t), f = 0, 2, 3, 1, each turn reaches 16 different
// chunk positions of 256 bytes.  The rows of one read are consecutive (A) or
// four runs of four, 16 rows apart (B, see the output layout below).
template <bool ISB>
__device__ __forceinline__ int swz_cont(int row) {
  const int t = (ISB ? row >> 4 : row >> 2) & 3;
  return ((t & 1) << 1) ^ (3 * (t >> 1));
}
// r-strided operand: rows of TI or TJ elements.  A transposing read of 32
// lanes touches eight rows (r = 8 g + jt) at two adjacent chunks (A), or at
// four chunks two apart of which every other lane takes the other half (B).
template <bool ISB>
__device__ __forceinline__ int swz_strided(int r) {
  if constexpr (ISB) return (r & 3) | (r & 8);
  return 2 * ((r & 3) | (((r >> 3) & 1) << 2));
}

// Operand staging of one workgroup: this wave's P direct-to-LDS loads of a
// stage.  Rows past the matrix and r past R read zero (an offset beyond the
// buffer), so stages past the end may be issued like any other; the chunks
// past the last column of an r-strided operand only reach output columns
// that are not stored.
template <int T, int P, bool STRIDED, bool ISB>
struct Stager {
  v4u rs;
  uint32_t voff[P];
  int ld, R, wave, lane;
  static constexpr uint32_t kBad = 0x80000000u;   // operands are below 2^31 bytes
  static constexpr int CPR = STRIDED ? T / 8 : BK / 8;   // chunks of a staged row
  static constexpr int RPL = 64 / CPR;                    // staged rows per 1 KB load
  static_assert(CPR <= 64, "a load covers whole staged rows");

  __device__ __forceinline__ void init(const uint16_t *p, int n, int x0, int R_, int ld_, int w, int l) {
    ld = ld_; R = R_; wave = w; lane = l;
    rs = raw_rsrc(p, (uint32_t)((size_t)(STRIDED ? R : n) * ld * 2));
#pragma unroll
    for (int u = 0; u < P; ++u) {
      const int row = (wave * P + u) * RPL + lane / CPR;
      if constexpr (STRIDED) {
        const int col = x0 + 8 * (lane % CPR ^ swz_strided<ISB>(row));
        voff[u] = col < n ? ((uint32_t)row * (uint32_t)ld + (uint32_t)col) * 2u : kBad;
      } else {
        voff[u] = x0 + row < n ? ((uint32_t)(x0 + row) * (uint32_t)ld + (uint32_t)chunk_r(u)) * 2u : kBad;
      }
    }
  }
  // first r (within the stage) of this lane's chunk of load u
  __device__ __forceinline__ int chunk_r(int u) const {
    const int row = (wave * P + u) * RPL + lane / CPR;
    return STRIDED ? row : 8 * (lane % CPR ^ swz_cont<ISB>(row));
  }
  // load u of the stage whose first r is r0, into the operand's buffer at lds
  __device__ __forceinline__ void issue(int u, int r0, uint32_t lds) const {
    // the scalar offset stays inside the buffer, behind the last stage too: the
    // bounds test compares the lane's offset with the buffer's size less it
    const uint32_t soff = r0 < R ? (uint32_t)r0 * (STRIDED ? (uint32_t)ld * 2u : 2u) : 0u;
    block_to_lds(rs, lds + (uint32_t)(wave * P + u) * 1024u, chunk_r(u) < R - r0 ? voff[u] : kBad, soff);
  }
};

// Eight elements from i on of an array of `end` >= 8; those past the end are
// anything.
__device__ __forceinline__ v4u load_within(const uint16_t *p, long long i, long long end) {
  const long long at = i < end - 8 ? i : end - 8;
  const int d = (int)(i - at), s = d >> 1;
  const v4u t = *reinterpret_cast<const U16 *>(p + at);
  v4u u;   // t shifted down by s dwords, then by the odd element
#pragma unroll
  for (int h = 0; h < 4; ++h) {
    u[h] = t[h];
#pragma unroll
    for (int k = 1; h + k < 4; ++k) u[h] = s == k ? t[h + k] : u[h];
  }
#pragma unroll
  for (int h = 0; h < 4; ++h) u[h] = __builtin_amdgcn_alignbit(h < 3 ? u[h + 1] : 0u, u[h], (uint32_t)(d & 1) * 16u);
  return u;
}

// The same staging through registers, for rows of any length: this thread's one
// 16-byte chunk of a stage, loaded at any element, zero past R.  Chunks of
// rows or columns past the matrix hold anything that lies inside it.
template <int T, bool STRIDED, bool ISB>
struct RaggedStager {
  const uint16_t *p;
  long long base, end;
  int ld, R, x0, off;
  static constexpr int CPR = STRIDED ? T / 8 : BK / 8;
  static_assert(T * BK / 8 == 512, "one chunk per thread");

  __device__ __forceinline__ void init(const uint16_t *p_, int n, int x0_, int R_, int ld_, int w, int l) {
    p = p_; ld = ld_; R = R_; x0 = x0_;
    end = (long long)(STRIDED ? R : n) * ld;
    const int row = w * (64 / CPR) + l / CPR;
    if constexpr (STRIDED) {
      off = row;
      base = (long long)row * ld + x0 + 8 * (l % CPR ^ swz_strided<ISB>(row));
    } else {
      off = 8 * (l % CPR ^ swz_cont<ISB>(row));
      base = (long long)min(x0 + row, n - 1) * ld + off;
    }
  }
  __device__ __forceinline__ v4u load(int r0) const {
    const long long i = base + (STRIDED ? (long long)r0 * ld : r0);
    const bool inside = r0 + BK <= R && (!STRIDED || (long long)(r0 + BK - 1) * ld + x0 + T <= end);
    if (inside) return *reinterpret_cast<const U16 *>(p + i);
    const int n = R - r0 - off;            // elements (rows) left from here
    v4u t = load_within(p, n > 0 ? i : 0, end);
#pragma unroll
    for (int h = 0; h < 4; ++h) {
      if constexpr (STRIDED) t[h] = n > 0 ? t[h] : 0u;
      else t[h] = n >= 2 * h + 2 ? t[h] : n == 2 * h + 1 ? t[h] & 0xFFFFu : 0u;
    }
    return t;
  }
};

template <int N>
__device__ __forceinline__ void stage_wait() {   // all but this wave's N newest loads, its LDS reads, the workgroup
  asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(N) : "memory");
}

// One tile of a job: rows i0 .. + TI, columns j0 .. + TJ, split z of the
// reduction (PART: the sum goes to the split's partial matrix).  RAGGED: rows
// of any length, staged through registers.
template <class C, int DT, bool ASTR, bool BSTR, bool PART, bool RAGGED = false>
__device__ __forceinline__ void lin_tile(const LinGemm &a, char *lds, int i0, int j0, int z) {
  struct alignas(16) Stage { char a[C::kA]; char b[C::kB]; };
  static_assert(sizeof(Stage) * C::NS <= kLinLds, "stage buffers");
  Stage *sm = reinterpret_cast<Stage *>(lds);
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wi = wave / C::WJ, wj = wave % C::WJ;
  const int nst = (a.R + BK - 1) / BK;
  const int s0 = PART ? __builtin_amdgcn_readfirstlane((int)((long long)z * nst / a.splits)) : 0;
  const int s1 = PART ? __builtin_amdgcn_readfirstlane((int)((long long)(z + 1) * nst / a.splits)) : nst;

  // Operand reads.  MFMA operand lane l holds row l % 16 and r = 8 (l / 16) ..
  // + 7 of the 32.  The product is formed transposed: the MFMA's row operand
  // is B, its column operand A, so lane l of a result holds output row l %
  // 16 and, in its four registers, MFMA rows 4 g .. 4 g + 3 (g = l / 16).
  // MFMA row rr of column tile jj is output column 16 (rr / 4) + 4 jj + rr %
  // 4 of the wave's 64, so a lane's four tiles are 16 consecutive columns.
  // An r-strided B has tiles jj and jj ^ 1 changed over in odd runs rr / 4,
  // which spreads its reads over the banks; odd g undo it at the end.
  const int g = lane >> 4, rr = lane & 15, jt = rr >> 2, q = rr & 3;
  uint32_t oa[ASTR ? C::NI : 1], ob[BSTR ? C::NJ : 1];
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
    oa[0] = (uint32_t)(row * BK * 2 + (g ^ swz_cont<false>(row)) * 16);
  }
  if constexpr (BSTR) {
#pragma unroll
    for (int jj = 0; jj < C::NJ; ++jj) {
      const int ch = wj * 8 + 2 * q + (jj >> 1);
      ob[jj] = (uint32_t)((8 * g + jt) * C::TJ * 2 + (ch ^ swz_strided<true>(8 * g + jt)) * 16 + ((jj ^ q) & 1) * 8);
    }
  } else {
    const int row = wj * 64 + 16 * (rr >> 2) + (rr & 3);
    ob[0] = (uint32_t)(row * BK * 2 + (g ^ swz_cont<true>(row)) * 16);
  }
  auto tr = [&](const char *p) __attribute__((always_inline)) -> v2u {
    return __builtin_bit_cast(v2u, __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) v4s *)p));
  };
  struct Frags { v4u a[C::NI], b[C::NJ]; };
  auto read_b = [&](int buf, int jj, Frags &f) __attribute__((always_inline)) {
    if constexpr (BSTR) {
      const char *p = sm[buf].b + ob[jj];
      const v2u lo = tr(p), hi = tr(p + 4 * C::TJ * 2);
      f.b[jj] = (v4u){lo[0], lo[1], hi[0], hi[1]};
    } else {
      f.b[jj] = *reinterpret_cast<const v4u *>(sm[buf].b + ob[0] + jj * 4 * BK * 2);
    }
  };
  auto read_a = [&](int buf, int i, Frags &f) __attribute__((always_inline)) {
    if constexpr (ASTR) {
      const char *p = sm[buf].a + oa[i];
      const v2u lo = tr(p), hi = tr(p + 4 * C::TI * 2);
      f.a[i] = (v4u){lo[0], lo[1], hi[0], hi[1]};
    } else {
      f.a[i] = *reinterpret_cast<const v4u *>(sm[buf].a + oa[0] + i * 16 * BK * 2);
    }
  };

  v4f acc[C::NI][C::NJ];
#pragma unroll
  for (int i = 0; i < C::NI; ++i)
#pragma unroll
    for (int j = 0; j < C::NJ; ++j) acc[i][j] = (v4f){0.0f, 0.0f, 0.0f, 0.0f};
  if constexpr (RAGGED) {
    // Four stages on their way in registers, two in LDS: a wave writes stage s
    // + 1 while others may still read stage s, and reaches the barrier of stage
    // s + 1 only behind its reads of stage s.
    RaggedStager<C::TI, ASTR, false> la;
    RaggedStager<C::TJ, BSTR, true> lb;
    la.init(a.A, a.I, i0, a.R, a.lda, wave, lane);
    lb.init(a.B, a.J, j0, a.R, a.ldb, wave, lane);
    v4u ra[4], rb[4];
    auto fetch = [&](int d, int s) __attribute__((always_inline)) {
      if (s < s1) {
        ra[d] = la.load(s * BK);
        rb[d] = lb.load(s * BK);
      }
    };
#pragma unroll
    for (int d = 0; d < 4; ++d) fetch(d, s0 + d);
    for (int s = s0; s < s1; s += 4)
#pragma unroll
      for (int d = 0; d < 4; ++d)
        if (s + d < s1) {
          *reinterpret_cast<v4u *>(sm[d & 1].a + wave * 1024 + lane * 16) = ra[d];
          *reinterpret_cast<v4u *>(sm[d & 1].b + wave * 1024 + lane * 16) = rb[d];
          fetch(d, s + d + 4);
          asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
          Frags f;
#pragma unroll
          for (int j = 0; j < C::NJ; ++j) read_b(d & 1, j, f);
#pragma unroll
          for (int i = 0; i < C::NI; ++i) read_a(d & 1, i, f);
#pragma unroll
          for (int i = 0; i < C::NI; ++i)
#pragma unroll
            for (int j = 0; j < C::NJ; ++j) acc[i][j] = mfma<DT>(f.b[j], f.a[i], acc[i][j]);
        }
  } else {
    Stager<C::TI, C::PA, ASTR, false> la;
    Stager<C::TJ, C::PB, BSTR, true> lb;
    la.init(a.A, a.I, i0, a.R, a.lda, wave, lane);
    lb.init(a.B, a.J, j0, a.R, a.ldb, wave, lane);
    constexpr int P = C::PA + C::PB;       // this wave's loads of a stage
    auto issue = [&](int u, int s, int buf) __attribute__((always_inline)) {
      if (u < C::PA) la.issue(u, s * BK, lds_addr(sm[buf].a));
      else lb.issue(u - C::PA, s * BK, lds_addr(sm[buf].b));
    };

    // The operands of stage s are in registers when stage s is multiplied: they
    // are read from LDS between the MFMAs of stage s - 1, and their buffer takes
    // the loads of stage s + NS.  One barrier per stage: behind it every wave
    // has its operands of stage s (its buffer is free) and its loads of stage s +
    // 1 (they may be read).  A stage's work is dealt into P parts of one load, a
    // share of the next operands' reads and a share of the MFMAs, so that
    // neither the loads of eight waves nor their reads meet in one burst.
    // Stages past s1 are loaded and read, not multiplied.
#pragma unroll
    for (int p = 0; p < C::NS; ++p)
#pragma unroll
      for (int u = 0; u < P; ++u) issue(u, s0 + p, p);
    int buf = 0;               // of the stage in registers
    auto step = [&](int s, const Frags &cur, Frags &nxt) __attribute__((always_inline)) {
      stage_wait<(C::NS - 2) * P>();
      const int next = buf + 1 == C::NS ? 0 : buf + 1;
#pragma unroll
      for (int u = 0; u < P; ++u) {
        issue(u, s + C::NS, buf);
#pragma unroll
        for (int x = u * (C::NJ + C::NI) / P; x < (u + 1) * (C::NJ + C::NI) / P; ++x) {
          if (x < C::NJ) read_b(next, x, nxt);
          else read_a(next, x - C::NJ, nxt);
        }
#pragma unroll
        for (int i = u * C::NI / P; i < (u + 1) * C::NI / P; ++i)
#pragma unroll
          for (int j = 0; j < C::NJ; ++j) acc[i][j] = mfma<DT>(cur.b[j], cur.a[i], acc[i][j]);
        __builtin_amdgcn_sched_barrier(0);
      }
      buf = next;
    };
    Frags f0, f1;
    stage_wait<(C::NS - 1) * P>();
#pragma unroll
    for (int j = 0; j < C::NJ; ++j) read_b(0, j, f0);
#pragma unroll
    for (int i = 0; i < C::NI; ++i) read_a(0, i, f0);
    int s = s0;
    for (; s + 1 < s1; s += 2) {
      step(s, f0, f1);
      step(s + 1, f1, f0);
    }
    if (s < s1) {
#pragma unroll
      for (int i = 0; i < C::NI; ++i)
#pragma unroll
        for (int j = 0; j < C::NJ; ++j) acc[i][j] = mfma<DT>(f0.b[j], f0.a[i], acc[i][j]);
    }
    // no load may land in LDS that the next workgroup owns
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
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
          for (int jj = 0; jj < C::NJ; ++jj)
            *reinterpret_cast<v4f *>(dst + (size_t)row * ld + 4 * (BSTR ? jj ^ (g & 1) : jj)) = acc[i][jj];
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
      for (int e = 0; e < 16; ++e) {
        v[e] = acc[i][e >> 2][e & 3];
        if (BSTR && (g & 1)) v[e] = acc[i][(e >> 2) ^ 1][e & 3];
      }
      if (row < a.I) finish<DT, 16>(a, row, j, bias, v);
    }
  }
}

// The tile of unit u among `count` units, t = first + u / cut in the walking
// order, and its part u % cut.  Workgroup ids go round the XCDs, each with its
// own L2: XCD x gets a contiguous range of the order, which walks the matrix
// in bands of four tile rows, so the tiles it runs at once share rows of A and
// columns of B.
__device__ __forceinline__ void lin_unit(const LinGemm &a, int u, int first, int count, int cut, int &bi, int &bj,
                                         int &part) {
  const int per = count / 8, rem = count % 8, x = u % 8;
  const int v = x * per + min(x, rem) + u / 8, t = first + v / cut;
  part = v % cut;
  constexpr int kBand = 4;
  const int span = kBand * a.nbj, band = t / span, top = band * kBand, rows = min(a.nbi - top, kBand), w = t % span;
  bi = top + w % rows;
  bj = w / rows;
}

// The units of one job: `full` whole 256 x 256 tiles, then the remaining tiles
// as two 256 x 128 or four 128 x 128 parts (`cut`), or all tiles in four for
// each split of the reduction.
template <int DT, bool AS, bool BS>
__device__ __forceinline__ void lin_full(const LinGemm &a, char *lds, int u) {
  int bi, bj, part;
  lin_unit(a, u, 0, a.full, 1, bi, bj, part);
  lin_tile<Big, DT, AS, BS, false>(a, lds, bi * 256, bj * 256, 0);
}
template <int DT, bool AS, bool BS>
__device__ __forceinline__ void lin_part(const LinGemm &a, char *lds, int u) {
  int bi, bj, part;
  const int count = (a.nbi * a.nbj - a.full) * a.cut, z = u / count;
  lin_unit(a, u % count, a.full, count, a.cut, bi, bj, part);
  const int i0 = bi * 256 + (a.cut == 4 ? part >> 1 : 0) * 128, j0 = bj * 256 + (part & 1) * 128;
  if (i0 >= a.I || j0 >= a.J) return;
  if (a.ragged) {
    if (a.splits > 1) lin_tile<Quarter, DT, AS, BS, true, true>(a, lds, i0, j0, z);
    else lin_tile<Quarter, DT, AS, BS, false, true>(a, lds, i0, j0, 0);
  } else if (a.splits > 1) lin_tile<Quarter, DT, AS, BS, true>(a, lds, i0, j0, z);
  else if (a.cut == 4) lin_tile<Quarter, DT, AS, BS, false>(a, lds, i0, j0, 0);
  else lin_tile<Half, DT, AS, BS, false>(a, lds, i0, j0, 0);
}

// Forward: one job.  Backward: dX and dW in one launch, so that the last
// tiles of the one run beside those of the other; whole tiles first.
template <int DT>
__global__ __launch_bounds__(512, 2) void k_lin_fwd(LinGemm a) {
  __shared__ __attribute__((aligned(16))) char lds[kLinLds];
  const int u = blockIdx.x;
  if (u < a.full) lin_full<DT, false, true>(a, lds, u);
  else lin_part<DT, false, true>(a, lds, u - a.parts0);
}
// The last workgroups sum the bias gradient's partial rows (of the launch
// before): 32 columns each, 16 shares of the rows, added in order.
constexpr int kDbCols = 32, kDbShares = 16;
template <int DT>
__device__ __forceinline__ void lin_db(const SumArgs &a, char *lds, int block) {
  float *sh = reinterpret_cast<float *>(lds);
  const int cx = threadIdx.x % kDbCols, y = threadIdx.x / kDbCols, c = block * kDbCols + cx;
  float s[4] = {0.0f, 0.0f, 0.0f, 0.0f};
  if (c < a.C) {
    const float *src = a.src + c;
    int p = y;
    for (; p + 3 * kDbShares < a.parts; p += 4 * kDbShares) {
      float v[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) v[k] = src[(size_t)(p + k * kDbShares) * a.ld];
#pragma unroll
      for (int k = 0; k < 4; ++k) s[k] += v[k];
    }
    for (; p < a.parts; p += kDbShares) s[0] += src[(size_t)p * a.ld];
  }
  sh[y * (kDbCols + 1) + cx] = (s[0] + s[1]) + (s[2] + s[3]);
  __syncthreads();
  if (y != 0 || c >= a.C) return;
  float v = 0.0f;
#pragma unroll
  for (int k = 0; k < kDbShares; ++k) v += sh[k * (kDbCols + 1) + cx];
  static_cast<uint16_t *>(a.dst)[c] = (uint16_t)f32_to_half<DT>(v);
}

template <int DT>
__global__ __launch_bounds__(512, 2) void k_lin_bwd(LinGemm x, LinGemm w, SumArgs db, int db0) {
  __shared__ __attribute__((aligned(16))) char lds[kLinLds];
  const int u = blockIdx.x;
  auto in = [&](int first, int count) { return u >= first && u < first + count; };
  if (in(x.full0, x.full)) lin_full<DT, false, false>(x, lds, u - x.full0);
  else if (in(w.full0, w.full)) lin_full<DT, true, true>(w, lds, u - w.full0);
  else if (in(x.parts0, x.parts)) lin_part<DT, false, false>(x, lds, u - x.parts0);
  else if (in(w.parts0, w.parts)) lin_part<DT, true, true>(w, lds, u - w.parts0);
  else lin_db<DT>(db, lds, u - db0);
}

// Sums the splits' partial sums in split order and finishes eight columns per thread.
// Grid y: the job.
template <int DT>
__global__ __launch_bounds__(256) void k_lin_reduce(LinGemm first, LinGemm second) {
  const LinGemm &a = blockIdx.y == 0 ? first : second;
  const int ld = (a.J + 15) / 16 * 16, cols = (a.J + 7) / 8;
  const long long t = (long long)blockIdx.x * 256 + threadIdx.x;
  if (t >= (long long)a.I * cols) return;
  const int i = (int)(t / cols), j = (int)(t % cols) * 8;
  const float *p = a.part + (size_t)i * ld + j;
  float v[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) v[e] = 0.0f;
  const size_t next = (size_t)a.I * ld;
  for (int z = 0; z < a.splits; z += 4, p += 4 * next) {   // four splits in flight
    v4f lo[4], hi[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float *pk = p + (z + k < a.splits ? k : 0) * next;
      lo[k] = *reinterpret_cast<const v4f *>(pk);
      hi[k] = *reinterpret_cast<const v4f *>(pk + 4);
    }
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (z + k < a.splits) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          v[e] += lo[k][e];
          v[4 + e] += hi[k][e];
        }
      }
  }
  float bias[8];
  load_bias<DT, 8>(a, j, bias);
  finish<DT, 8>(a, i, j, bias, v);
}

// ---------------------------------------------------------------- few rows
// Y of up to 48 rows (16 MT), bound by the one read of W.  A workgroup owns 128
// columns and a share of K; its four waves split that share in runs of 32.
// Lane l loads, for its 8 rows k = 8 (l / 16) .. + 7 of a run, the 8
// columns 8 (l % 16) .. + 7 (16 bytes each, a row's 128 columns are 256
// consecutive bytes), transposes the 8 x 8 block in registers (32 byte
// permutes), and has the MFMA operands of 8 column tiles: tile j holds
// columns 8 c + j.  W never passes through LDS.  The result lane holds row
// l % 16 and 32 consecutive columns.
constexpr int kSkCols = 128, kSkWaves = 4;

template <int DT, int MT, bool PART>
__global__ __launch_bounds__(64 * kSkWaves, 5 - MT) void k_lin_skinny(LinGemm a) {
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

  // Columns past J only reach outputs that are not stored, so a run may read
  // on into the next row wherever that stays inside W; at the end of W the
  // loads are moved back and shifted, and the rows past K are zeros.
  const long long w_end = (long long)a.R * a.ldb, x_end = (long long)a.I * a.lda;
  auto load = [&](int run, v4u (&w)[8]) __attribute__((always_inline)) {
    const int k = 32 * run + 8 * g;
    if ((long long)(32 * run + 31) * a.ldb + j0 + kSkCols <= w_end) {
      const uint16_t *p = a.B + (size_t)k * a.ldb + jc;
#pragma unroll
      for (int e = 0; e < 8; ++e) w[e] = *reinterpret_cast<const U16 *>(p + (size_t)e * a.ldb);
      return;
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const v4u t = load_within(a.B, (long long)min(k + e, a.R - 1) * a.ldb + jc, w_end);
#pragma unroll
      for (int h = 0; h < 4; ++h) w[e][h] = k + e < a.R ? t[h] : 0u;
    }
  };
  auto step = [&](int run, const v4u (&w)[8]) __attribute__((always_inline)) {
    const int k = 32 * run + 8 * g;
    v4u x[MT];
#pragma unroll
    for (int m = 0; m < MT; ++m) {
      const int row = 16 * m + c;
      if (32 * run + 32 <= a.R) {
        x[m] = (v4u){0u, 0u, 0u, 0u};
        if (row < a.I) x[m] = *reinterpret_cast<const U16 *>(a.A + (size_t)row * a.lda + k);
      } else {
        const v4u t = load_within(a.A, (long long)min(row, a.I - 1) * a.lda + min(k, a.R - 1), x_end);
        const int n = row < a.I ? a.R - k : 0;      // elements of this row
#pragma unroll
        for (int h = 0; h < 4; ++h) x[m][h] = n >= 2 * h + 2 ? t[h] : n == 2 * h + 1 ? t[h] & 0xFFFFu : 0u;
      }
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      v4u b;   // column 8 c + j, k .. k + 7
#pragma unroll
      for (int e = 0; e < 4; ++e)
        b[e] = __builtin_amdgcn_perm(w[2 * e + 1][j / 2], w[2 * e][j / 2], (j & 1) ? 0x07060302u : 0x05040100u);
#pragma unroll
      for (int m = 0; m < MT; ++m) acc[m][j] = mfma<DT>(b, x[m], acc[m][j]);
    }
  };
  // One run of 8 KB in flight per wave.  Two spilled within the 128 registers
  // that leave room for four workgroups a CU (MT = 1); skinny_splits launches
  // fewer: 256 workgroups for 16 x 12288 x 4096, four waves and 32 KB a CU, 480
  // for 1 x 4096 x 12288.
  for (int run = r0 + wave; run < r1; run += kSkWaves) {
    v4u w[8];
    load(run, w);
    step(run, w);
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
// Rows of a length that is no multiple of 8 elements, copied to a multiple
// with zeros behind them (the direct-to-LDS loads are 16 bytes, aligned).
__device__ __forceinline__ void pad_rows(const uint16_t *src, int rows, int cols, uint16_t *dst, int ld, int block) {
  const long long t = (long long)block * 256 + threadIdx.x;
  const int cpr = ld / 8;
  if (t >= (long long)rows * cpr) return;
  const int r = (int)(t / cpr), c = (int)(t % cpr) * 8;
  const uint16_t *p = src + (size_t)r * cols + c;
  v4u v = {0u, 0u, 0u, 0u};
  if (c + 8 <= cols) {
    v = *reinterpret_cast<const U16 *>(p);
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (c + e < cols) v[e / 2] |= (uint32_t)p[e] << (16 * (e & 1));
  }
  *reinterpret_cast<v4u *>(dst + (size_t)r * ld + c) = v;
}

// dZ = dY act'(Z), rounded to the operand type of the two products, and the
// column sums of the unrounded dZ over a slice of the rows.  The rounding is
// what the 16-bit matrix cores take; it puts dX and dW 1.4 times as far from the
// exact gradient as their own rounding does (2.3e-3 against 1.7e-3 in bf16,
// 4096 x 1152 x 4608), and a second operand for its rest would double the
// products' time.  256 columns per
// workgroup: thread t takes columns 8 (t % 32) .. + 7 of rows t / 32, t / 32 +
// 8, ... of its slice.
constexpr int kDzCols = 256, kDzRows = 8;

template <int DT>
__device__ __forceinline__ void lin_dz(const LinDz &a, int bx, int by) {
  __shared__ float red[kDzRows][kDzCols];
  const int cx = threadIdx.x & 31, ry = threadIdx.x >> 5;
  const int j = bx * kDzCols + 8 * cx, n = a.N - j;
  const int m0 = (int)((long long)by * a.M / a.slices), m1 = (int)((long long)(by + 1) * a.M / a.slices);
  float s[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) s[e] = 0.0f;
  auto half8 = [&](const uint16_t *p, float *v) __attribute__((always_inline)) {
    if (n >= 8) {
      const U16 t = *reinterpret_cast<const U16 *>(p);
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] = half_to_f32<DT>((t[e / 2] >> (16 * (e & 1))) & 0xFFFFu);
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] = e < n ? half_to_f32<DT>(p[e]) : 0.0f;
    }
  };
  auto load = [&](int m, float *d, float *z) __attribute__((always_inline)) {
    const size_t o = (size_t)m * a.N + j;
    if (a.dy_f32) {
      const float *p = static_cast<const float *>(a.dY) + o;
      if (n >= 8) {
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          const F32x4 t = *reinterpret_cast<const F32x4 *>(p + 4 * c);
#pragma unroll
          for (int e = 0; e < 4; ++e) d[4 * c + e] = t[e];
        }
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) d[e] = e < n ? p[e] : 0.0f;
      }
    } else {
      half8(static_cast<const uint16_t *>(a.dY) + o, d);
    }
    if (a.act != kActIdentity) half8(a.Z + o, z);
  };
  auto work = [&](int m, float *d, const float *z) __attribute__((always_inline)) {
    if (a.act == kActGeluTanh) {
#pragma unroll
      for (int e = 0; e < 8; ++e) d[e] *= act_grad(z[e], kActGeluTanh);
    } else if (a.act == kActGelu) {
#pragma unroll
      for (int e = 0; e < 8; ++e) d[e] *= act_grad(z[e], kActGelu);
    } else if (a.act == kActSilu) {
#pragma unroll
      for (int e = 0; e < 8; ++e) d[e] *= act_grad(z[e], kActSilu);
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) s[e] += d[e];
    if (a.dZ) {
      v4u t;
#pragma unroll
      for (int e = 0; e < 4; ++e) t[e] = f32_to_half<DT>(d[2 * e]) | (f32_to_half<DT>(d[2 * e + 1]) << 16);
      *reinterpret_cast<v4u *>(a.dZ + (size_t)m * a.np + j) = t;
    }
  };
  if (n > 0) {
    int m = m0 + ry;
    for (; m + kDzRows < m1; m += 2 * kDzRows) {   // two rows in flight
      float d0[8], z0[8], d1[8], z1[8];
      load(m, d0, z0);
      load(m + kDzRows, d1, z1);
      work(m, d0, z0);
      work(m + kDzRows, d1, z1);
    }
    if (m < m1) {
      float d[8], z[8];
      load(m, d, z);
      work(m, d, z);
    }
  }
  if (!a.part) return;
#pragma unroll
  for (int e = 0; e < 8; ++e) red[ry][8 * cx + e] = s[e];
  __syncthreads();
  const int col = bx * kDzCols + threadIdx.x;
  if (col >= a.N) return;
  float v = 0.0f;
#pragma unroll
  for (int r = 0; r < kDzRows; ++r) v += red[r][threadIdx.x];
  a.part[(size_t)by * a.N + col] = v;
}

// Everything the products read that is not there yet, in one launch: padded X,
// padded W, dZ with its column sums.  Bound by HBM: dZ of 4096 x 4608 with
// the GELU's derivative, 113 MB, takes 30 us (3.8 TB/s).
template <int DT>
__global__ __launch_bounds__(256) void k_lin_prep(LinPrep p) {
  int b = blockIdx.x;
  if (b < p.x_blocks) return pad_rows(p.X, p.x_rows, p.x_cols, p.Xp, p.x_ld, b);
  b -= p.x_blocks;
  if (b < p.w_blocks) return pad_rows(p.W, p.w_rows, p.w_cols, p.Wp, p.w_ld, b);
  b -= p.w_blocks;
  const int cols = (p.dz.np + kDzCols - 1) / kDzCols;
  lin_dz<DT>(p.dz, b % cols, b / cols);
}


// ---------------------------------------------------------------- planning
constexpr int kCus = 256;

int quarters(int I, int J) { return ceil_div(I, 128) * ceil_div(J, 128); }

// Splits of the reduction, each of at least 256, for fewer 128 x 128 tiles
// than CUs: the cheapest by what was measured.  A stage of 32 takes 0.3 us, a
// streamed operand arrives at 3 TB/s, the second launch takes 3 us, and the
// partial sums go out and back at 2.5 TB/s.  64 x 12288 x 4096 (32 tiles): 4
// splits 39 us, 8 44, 2 64, none 112; 64 x 4096 x 12288 (96): none 44, 2 49; 1000 x
// 1024 x 1024 (64): none 13.6, 2 19.8; 256 x 8192 x 256 (4): 16 16.7, none 65.
int gemm_splits(int I, int J, int R) {
  const int most = std::min({kCus / quarters(I, J), R / 256, 16});
  const float stream = 2.0f / 3e6f * ((float)I + J) * R;
  int best = 1;
  float least = 0.0f;
  for (int s = 1; s <= most; ++s) {
    const float us = std::max(0.3f / 32 * R / s, stream) + (s > 1 ? 3.0f + 3.2e-6f * s * I * J : 0.0f);
    if (s == 1 || us < least) least = us, best = s;
  }
  return best;
}

// Whether a product with rows that are no multiple of 8 reads them as they are
// (128 x 128 tiles staged through registers, 0.45 us a stage instead of 0.3) or
// from padded copies of `elems` elements (3.5 us and their way out and back at
// 4.5 TB/s).  As they are / padded, us (no epilogue): 202 x 1502 x 359 13.7 / 16.9,
// 333 x 1001 x 777 14.8 / 17.9, 900 x 2500 x 1201 26 / 31, 1000 x 4001 x 2001 (128
// tiles, two splits) 42 / 46, gradients of 6 x 8768 x 9471 192 / 224; the other
// way, gradients of 1500 x 1023 x 1401 36 / 31 and many tiles, 4000 x 999 x 3999,
// 81 / 54.
bool reads_ragged(int I, int J, int R, long long elems) {
  return quarters(I, J) <= kCus / 2 && 0.15f / 32 * R / gemm_splits(I, J, R) <= 3.5f + 4.0f / 4.5e6f * elems;
}

// Units of a job whose tiles are all cut in 1, 2 or 4 (empty parts left out),
// and the time of one relative to a stage of a whole tile.
int units_of(const LinGemm &a, int cut) {
  return cut == 1 ? a.nbi * a.nbj : cut == 2 ? a.nbi * ceil_div(a.J, 128) : quarters(a.I, a.J);
}
float unit_time(const LinGemm &a, int cut) { return (cut == 1 ? 1.0f : cut == 2 ? 0.6f : 0.4f) * a.R; }

// Sets the units of the jobs of one launch: which tiles are cut.  Either the
// last of the second job are, those left over from whole rounds of one tile
// per CU, or all tiles of a job.  Estimated: one round takes its longest unit
// (shorter where CUs idle: the chip is power-limited), more rounds the work
// over the CUs and half of a last unit.  Measured, us: 1.5 rounds whole 192,
// last cut in halves 176, in quarters 193; 1.125 rounds 76, 62, 56; 0.66 rounds
// whole 76, all in halves 90, in quarters 88; 18 tiles of 144 stages beside 162 of
// 14 whole 116.
// The job with the longer reduction runs first; jobs with a split reduction
// or ragged rows are all quarters and start before the others.
void plan_units(LinGemm &a, LinGemm &b) {
  LinGemm *order[2] = {&a, &b};
  if (b.R > a.R) std::swap(order[0], order[1]);
  auto apart = [](const LinGemm *j) { return j->splits > 1 || j->ragged; };
  int base = 0, t[2] = {0, 0};
  for (int i = 0; i < 2; ++i) {
    LinGemm *j = order[i];
    j->nbi = ceil_div(j->I, 256);
    j->nbj = ceil_div(j->J, 256);
    j->full = j->parts = j->full0 = j->parts0 = 0;
    j->cut = 1;
    if (apart(j)) {
      j->cut = 4;
      j->parts = 4 * j->nbi * j->nbj * std::max(1, j->splits);
      j->parts0 = base;
      base += j->parts;
    } else {
      t[i] = j->nbi * j->nbj;
    }
  }
  if (t[0] + t[1] > 0) {
    LinGemm *last = t[1] > 0 ? order[1] : order[0];
    const int tl = t[1] > 0 ? t[1] : t[0];
    const double whole = ((double)t[0] * order[0]->R + (double)t[1] * order[1]->R) / last->R;
    const int rem = std::min(tl, (int)whole % kCus);
    auto estimate = [&](double units, double work, double longest, double end) {
      return units <= kCus ? longest * (0.5 + 0.5 * units / kCus) : std::max(longest, work / kCus + 0.5 * end);
    };
    const double others = t[0] + t[1] - tl, first = t[1] > 0 && t[0] > 0 ? order[0]->R : 0.0;
    double least = 0.0;
    int tail = 1, cuts[2] = {1, 1};
    for (int c : {1, 2, 4}) {           // the last job's last tiles
      const double u = unit_time(*last, c), work = others * first + (double)(tl - rem) * last->R + (double)rem * c * u;
      const double e = estimate(others + tl - rem + (double)rem * c, work, std::max(first, tl > rem ? (double)last->R : u), u);
      if (c == 1 || e < least) least = e, tail = c;
    }
    bool all = false;
    for (int c0 : {1, 2, 4})            // all tiles of either job
      for (int c1 : {1, 2, 4}) {
        if ((t[0] == 0 && c0 > 1) || (t[1] == 0 && c1 > 1)) continue;
        double units = 0.0, work = 0.0, longest = 0.0, end = 0.0;
        const int c[2] = {c0, c1};
        for (int i = 0; i < 2; ++i)
          if (t[i] > 0) {
            end = unit_time(*order[i], c[i]);
            longest = std::max(longest, end);
            units += units_of(*order[i], c[i]);
            work += units_of(*order[i], c[i]) * end;
          }
        const double e = estimate(units, work, longest, end);
        if (e < least) least = e, all = true, cuts[0] = c0, cuts[1] = c1;
      }
    for (int i = 0; i < 2; ++i)
      if (t[i] > 0) {
        LinGemm *j = order[i];
        const int cut = all ? cuts[i] : j == last ? tail : 1, n = cut == 1 ? 0 : all ? t[i] : rem;
        j->cut = cut;
        j->full = t[i] - n;
        j->parts = n * cut;
      }
  }
  for (LinGemm *j : order) {
    j->full0 = base;
    base += j->full;
  }
  for (LinGemm *j : order)
    if (!apart(j)) {
      j->parts0 = base;
      base += j->parts;
    }
}

// Splits of K of the weight-streaming kernel: the fewest whose workgroups
// fill nine tenths of whole rounds of one a CU, at least 256 of K each.
// 1 x 4096 x 12288 (96 strips): 5 splits 22.1 us, 4 and 8 22.4, 3 25.8; 16 x
// 12288 x 4096 (32 strips): 8 splits 23.6 us, 16 24.9, 12 26.8.
int skinny_splits(int J, int K) {
  const int strips = ceil_div(J, kSkCols), most = std::max(1, std::min(K / 256, 16));
  for (int s = 1; s < most; ++s)
    if (10 * strips * s >= 9 * kCus * ceil_div(strips * s, kCus)) return s;
  return most;
}

size_t part_bytes(int I, int J, int splits) {
  return splits > 1 ? (size_t)splits * I * part_ld(J) * sizeof(float) : 0;
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
hipError_t run_reduce(const LinGemm &a, const LinGemm &b, hipStream_t s) {
  long long items = a.splits > 1 ? (long long)a.I * ceil_div(a.J, 8) : 0;
  const bool two = b.splits > 1;
  if (two) items = std::max(items, (long long)b.I * ceil_div(b.J, 8));
  if (items == 0) return hipSuccess;
  const LinGemm &first = a.splits > 1 ? a : b;
  hipLaunchKernelGGL(k_lin_reduce<DT>, dim3((unsigned)((items + 255) / 256), a.splits > 1 && two ? 2u : 1u), dim3(256), 0,
                     s, first, b);
  return hipGetLastError();
}

template <int DT>
hipError_t run_forward(LinGemm a, bool skinny, hipStream_t s) {
  hipError_t e;
  if (skinny) {
    const int mt = ceil_div(a.I, 16);
    e = mt == 1 ? run_skinny<DT, 1>(a, s) : mt == 2 ? run_skinny<DT, 2>(a, s) : run_skinny<DT, 3>(a, s);
  } else {
    LinGemm none{};
    plan_units(a, none);
    hipLaunchKernelGGL(k_lin_fwd<DT>, dim3((unsigned)(a.full + a.parts)), dim3(512), 0, s, a);
    e = hipGetLastError();
  }
  return e != hipSuccess ? e : run_reduce<DT>(a, LinGemm{}, s);
}

template <int DT>
hipError_t run_backward(const LinGemm &x, const LinGemm &w, const SumArgs &db, hipStream_t s) {
  LinGemm job[2] = {x, w};
  const bool has_x = x.out != nullptr, has_w = w.out != nullptr;
  plan_units(job[0], job[1]);
  const int units = job[0].full + job[0].parts + job[1].full + job[1].parts;
  hipLaunchKernelGGL(k_lin_bwd<DT>, dim3((unsigned)(units + (db.dst ? ceil_div(db.C, kDbCols) : 0))), dim3(512), 0, s,
                     job[0], job[1], db, units);
  const hipError_t e = hipGetLastError();
  return e != hipSuccess ? e : run_reduce<DT>(has_x ? job[0] : LinGemm{}, has_w ? job[1] : LinGemm{}, s);
}

}  // namespace

LinPlan plan_linear(int M, int K, int N) {
  LinPlan p;
  p.kp = ceil_div(K, 8) * 8;
  p.np = ceil_div(N, 8) * 8;
  // (its loads at the end of X and W are moved back inside them: 8 elements at least)
  p.skinny = M <= kLinSkinnyMaxM && (long long)M * K >= 8 && (long long)K * N >= 8;
  p.splits = p.skinny ? skinny_splits(N, K) : gemm_splits(M, N, K);
  const bool odd = p.kp != K || p.np != N, whole = (long long)M * K >= 8 && (long long)K * N >= 8;
  const long long copied = (p.kp != K ? (long long)M * K : 0) + (p.np != N ? (long long)K * N : 0);
  p.ragged_x = p.ragged_w = !p.skinny && odd && whole && reads_ragged(M, N, K, copied);
  p.pad_x = !p.skinny && !p.ragged_x && p.kp != K;
  p.pad_w = !p.skinny && !p.ragged_x && p.np != N;
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
  // dZ always has whole rows; W is read for dX, X for dW
  p.ragged_w = p.np != N && (long long)K * N >= 8 && reads_ragged(M, K, N, (long long)K * N);
  p.ragged_x = p.kp != K && (long long)M * K >= 8 && reads_ragged(K, N, M, (long long)M * K);
  p.pad_x = p.kp != K && !p.ragged_x;
  p.pad_w = p.np != N && !p.ragged_w;
  p.splits_dx = gemm_splits(M, K, N);
  p.splits_dw = gemm_splits(K, N, M);
  // row slices of the dZ pass: about 1024 workgroups, at least one row per
  // thread
  p.slices = std::max(1, std::min(1024 / ceil_div(p.np, kDzCols), ceil_div(M, kDzRows)));
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
  off = align_up(off + part_bytes(M, K, p.splits_dx), 256);
  p.part_w_off = off;
  off = align_up(off + part_bytes(K, N, p.splits_dw), 256);
  p.total = off;
  return p;
}

extern "C" void hsq_internal_linear_units(int M, int K, int N, int backward, int *out) {
  LinGemm job[2] = {};
  bool skinny = false;
  if (backward) {
    const LinPlan p = plan_linear_backward(M, K, N);
    job[0].I = M; job[0].J = K; job[0].R = N; job[0].splits = p.splits_dx; job[0].ragged = p.ragged_w;
    job[1].I = K; job[1].J = N; job[1].R = M; job[1].splits = p.splits_dw; job[1].ragged = p.ragged_x;
  } else {
    const LinPlan p = plan_linear(M, K, N);
    skinny = p.skinny;
    job[0].I = M; job[0].J = N; job[0].R = K; job[0].splits = p.splits; job[0].ragged = p.ragged_x;
  }
  if (!skinny) plan_units(job[0], job[1]);
  for (const LinGemm &j : job) {
    const int v[6] = {skinny, j.splits, j.ragged, j.full, j.cut, j.parts};
    out = std::copy(v, v + 6, out);
  }
}

hipError_t launch_linear(const LinGemm &a, bool skinny, hipStream_t s) {
  return a.dtype == kBf16 ? run_forward<kBf16>(a, skinny, s) : run_forward<kF16>(a, skinny, s);
}

hipError_t launch_linear_backward(const LinGemm &x, const LinGemm &w, const SumArgs &db, int dtype, hipStream_t s) {
  return dtype == kBf16 ? run_backward<kBf16>(x, w, db, s) : run_backward<kF16>(x, w, db, s);
}

hipError_t launch_linear_prep(LinPrep p, int dtype, hipStream_t s) {
  auto blocks = [](const uint16_t *src, int rows, int ld) {
    return src ? (int)(((long long)rows * (ld / 8) + 255) / 256) : 0;
  };
  p.x_blocks = blocks(p.X, p.x_rows, p.x_ld);
  p.w_blocks = blocks(p.W, p.w_rows, p.w_ld);
  const bool dz = p.dz.dY != nullptr;
  const int n = p.x_blocks + p.w_blocks + (dz ? ceil_div(p.dz.np, kDzCols) * p.dz.slices : 0);
  if (n == 0) return hipSuccess;
  if (dtype == kBf16) hipLaunchKernelGGL(k_lin_prep<kBf16>, dim3((unsigned)n), dim3(256), 0, s, p);
  else hipLaunchKernelGGL(k_lin_prep<kF16>, dim3((unsigned)n), dim3(256), 0, s, p);
  return hipGetLastError();
}

}  // namespace hsq
