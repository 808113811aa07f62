// w4a16.hip -- the layer with its activations left in 16 bits, for few tokens
// (M <= 64): the packed 4-bit residual against X itself.
//
//   xh = X / lambda,  U = xh L1
//   Y  = sum_g sw[g,n] sum_{k in g} xh[m,k] qw[k,n] + U L2 + bias + residual
//
// Bound by the read of the weights (K N / 2 bytes for 2 M K N operations), as the
// weight-streaming contraction of the W4A4 layer, whose mapping this is: a
// workgroup owns CT tiles of 16 columns, its waves deal out the 128-channel
// pairs of blocks, and their partial tiles meet in LDS.
//
// The codes become matrix operands by one shift and one and-xor a pair: a nibble
// under a constant exponent is 24 + code in bf16 and in fp16 alike.  The 24 sum
// xh that this adds to every column is taken off by the accumulator's first value,
// the product of the same xh with a constant -24, one for all column tiles.
//
// With smoothing a first launch forms xh once, as fp16 numbers under a power of
// two per row and scale group: one of 11 bits where Y is bf16, two (22 bits) where
// it is finer, so that what is rounded is far below the rounding of Y.  That
// launch also forms U in fp32.
#include "hsq_internal.h"

#include <algorithm>

namespace hsq {

namespace {

typedef __bf16 v8bf __attribute__((ext_vector_type(8)));
typedef _Float16 v8h __attribute__((ext_vector_type(8)));

constexpr int kStreamLoad = 2;    // the weights are read once: non-temporal
constexpr int kPrepThreads = 256;
constexpr int kPrepFloats = 12288;   // values of xh that its workgroup holds

template <int DT>
__device__ __forceinline__ v4f mfma16(v4u a, v4u b, v4f c) {
  if constexpr (DT == kBf16)
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(v8bf, a), __builtin_bit_cast(v8bf, b), c, 0, 0, 0);
  else
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(v8h, a), __builtin_bit_cast(v8h, b), c, 0, 0, 0);
}

// A dword of the packed residual, channels p = 0 .. 7, as 24 + code in the order
// 0 2 1 3 4 6 5 7 (high nibbles of bytes 0, 2 | 1, 3, then the low ones).
template <int DT>
__device__ __forceinline__ v4u expand(uint32_t w) {
  if constexpr (DT == kBf16) {
    constexpr uint32_t m = 0x00780078u, k = 0x41C041C0u;
    return (v4u){(w >> 1 & m) ^ k, (w >> 9 & m) ^ k, (w << 3 & m) ^ k, (w >> 5 & m) ^ k};
  } else {
    constexpr uint32_t m = 0x03C003C0u, k = 0x4E004E00u;
    return (v4u){(w << 2 & m) ^ k, (w >> 6 & m) ^ k, (w << 6 & m) ^ k, (w >> 2 & m) ^ k};
  }
}
template <int DT>
constexpr uint32_t kMinus24 = DT == kBf16 ? 0xC1C0C1C0u : 0xCE00CE00u;

// Eight consecutive channels in the order of expand.
__device__ __forceinline__ v4u in_order(v4u x) {
  return (v4u){__builtin_amdgcn_perm(x[1], x[0], 0x05040100u), __builtin_amdgcn_perm(x[1], x[0], 0x07060302u),
               __builtin_amdgcn_perm(x[3], x[2], 0x05040100u), __builtin_amdgcn_perm(x[3], x[2], 0x07060302u)};
}

__device__ __forceinline__ float half_or_bf(uint16_t v, int dtype) {
  return dtype == kBf16 ? bf16_to_f32(v) : f16_to_f32(v);
}

// Smoothing and U.  A workgroup has `slice` channels of all M rows.
__global__ __launch_bounds__(kPrepThreads) void k_w4a16_prep(W4a16Args a) {
  extern __shared__ float lds[];               // xh [M][slice], then partial U [threads]
  const int tid = threadIdx.x, k0 = blockIdx.x * a.slice, nk = min(a.slice, a.K - k0), M16 = (a.M + 15) / 16 * 16;
  float *xh = lds, *red = lds + a.M * a.slice;
  for (int i = tid; i < a.M * nk; i += kPrepThreads) {
    const int m = i / nk, k = i % nk;
    float v = half_or_bf(a.X[(size_t)m * a.K + k0 + k], a.dtype);
    if (a.lam) v *= 1.0f / f16_to_f32(a.lam[k0 + k]);
    xh[m * a.slice + k] = v;
  }
  __syncthreads();
  if (a.lam) {
    const int gw = 64 * a.bpg, ng = nk / gw, lane = tid & 63, wave = tid >> 6;
    for (int i = wave; i < a.M * ng; i += kPrepThreads / 64) {
      const int m = i / ng, g = i % ng;
      float v[2] = {xh[m * a.slice + g * gw + lane], 0.0f};
      if (a.bpg == 2) v[1] = xh[m * a.slice + g * gw + 64 + lane];
      float top = fmaxf(fabsf(v[0]), fabsf(v[1]));
#pragma unroll
      for (int o = 32; o >= 1; o >>= 1) top = fmaxf(top, __shfl_xor(top, o));
      // 2^e with the largest |xh| / 2^e in [2^13, 2^14); bits of the exponent
      // alone; a zero, tiny or infinite group keeps a scale that is finite
      const int ex = min(max((int)(__float_as_uint(top) >> 23) - 13, 1), 240);
      const float sc = __uint_as_float((uint32_t)ex << 23), inv = __uint_as_float((uint32_t)(254 - ex) << 23);
      for (int h = 0; h < a.bpg; ++h) {
        const size_t at = (size_t)m * a.K + k0 + g * gw + 64 * h + lane;
        const float y = v[h] * inv;
        const _Float16 hi = (_Float16)y;
        a.hi[at] = __builtin_bit_cast(uint16_t, hi);
        // not finite: in hi alone
        if (a.terms == 2) a.lo[at] = fabsf(y) <= 65504.0f ? f32_to_f16(y - (float)hi) : (uint16_t)0;
      }
      if (lane == 0) a.es[(size_t)(k0 / gw + g) * M16 + m] = sc;
    }
  }
  // U: threads deal out (row, rank column), and what is left of them the channels
  const int cols = a.batch * a.r;
  if (cols == 0) return;
  const int items = cols * a.M, per = max(1, kPrepThreads / items);
  for (int i0 = 0; i0 < items; i0 += kPrepThreads / per) {
    const int it = i0 + tid / per, sub = tid % per;
    float u = 0.0f;
    if (it < items && tid / per < kPrepThreads / per) {
      const int m = it / cols, c = it % cols;
      const uint16_t *l1 = a.L1 + ((size_t)(c / a.r) * a.K + k0) * a.r + c % a.r;
      for (int k = sub; k < nk; k += per)
        u = __builtin_fmaf(xh[m * a.slice + k], half_or_bf(l1[(size_t)k * a.r], a.dtype), u);
    }
    red[tid] = u;
    __syncthreads();
    if (sub == 0 && it < items && tid / per < kPrepThreads / per) {
      for (int p = 1; p < per; ++p) u += red[tid + p];
      a.uw[((size_t)blockIdx.x * cols + it % cols) * M16 + it / cols] = u;
    }
    __syncthreads();
  }
}

// XS: xh under powers of two (es); NX: its terms (lo in the second)
template <int DT, int MT, int CT, int P, int BPG, bool XS, int NX>
__global__ __launch_bounds__(MT == 1 ? 1024 : 512) void k_w4a16(W4a16Args a, int W) {
  constexpr int NS = BPG == 1 ? 2 : 1;             // scale groups of a pair of blocks
  extern __shared__ float red[];                   // partial tiles [W][CT][MT][4][64], U [r][16 MT], L2 [r][16 CT]
  float *eu = red + W * CT * MT * 4 * 64;
  float *el2 = eu + a.r * MT * 16;
  const int tid = threadIdx.x, lane = tid & 63, colq = lane & 15, q = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int NT = (a.N + 15) / 16, nt0 = blockIdx.x * CT, proj = blockIdx.y;
  const int G64 = a.K / kGroup, GP = (G64 + 1) / 2, SG = BPG == 1 ? G64 : G64 / 2, M16 = (a.M + 15) / 16 * 16;
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
  for (int i = 0; i < MT; ++i) offx[i] = ((uint32_t)min(16 * i + colq, a.M - 1) * a.K + 16 * q) * 2;

  float acc[CT][MT][4];
#pragma unroll
  for (int c = 0; c < CT; ++c)
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
      for (int r = 0; r < 4; ++r) acc[c][i][r] = 0.0f;

  for (int c0 = wave * P; c0 < GP; c0 += W * P) {
    v4u wv[P][CT], xv[P][NX][MT][4];
    _Float16 sv[P][CT][NS];
    v4f ev[P][NS][MT];
#pragma unroll
    for (int p = 0; p < P; ++p) {
      const int gp = min(c0 + p, GP - 1);
#pragma unroll
      for (int c = 0; c < CT; ++c) wv[p][c] = __builtin_amdgcn_raw_buffer_load_b128(rs_w, offw[c], gp * 1024, kStreamLoad);
#pragma unroll
      for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) {              // block j / 2, channels 8 (j % 2) ..
          const int blk = min(2 * gp + j / 2, G64 - 1);   // a pad block: the one before, times 0 below
          const uint32_t so = (uint32_t)blk * 128 + (j & 1) * 16;
          xv[p][0][i][j] = __builtin_amdgcn_raw_buffer_load_b128(rs_x, offx[i], so, 0);
          if constexpr (NX == 2) xv[p][1][i][j] = __builtin_amdgcn_raw_buffer_load_b128(rs_l, offx[i], so, 0);
        }
#pragma unroll
      for (int h = 0; h < NS; ++h) {
        const int sg = min(NS * gp + h, SG - 1);
#pragma unroll
        for (int c = 0; c < CT; ++c)
          sv[p][c][h] = __builtin_bit_cast(_Float16, __builtin_amdgcn_raw_buffer_load_b16(rs_s, offs[c], sg * a.N * 2, 0));
        if constexpr (XS) {
#pragma unroll
          for (int i = 0; i < MT; ++i) ev[p][h][i] = *reinterpret_cast<const v4f *>(a.es + (size_t)sg * M16 + 16 * i + 4 * q);
        }
      }
    }
#pragma unroll
    for (int p = 0; p < P; ++p) {
      const int gp = c0 + p;
      if (gp >= GP) break;
      // a pad block (K an odd number of blocks) has X = 0
      if (NS == 2 && 2 * gp + 1 >= G64) {
#pragma unroll
        for (int t = 0; t < NX; ++t)
#pragma unroll
          for (int i = 0; i < MT; ++i) xv[p][t][i][2] = xv[p][t][i][3] = (v4u){0u, 0u, 0u, 0u};
      }
      constexpr uint32_t m24 = kMinus24<DT>;
      const v4u neg = {m24, m24, m24, m24};
      v4f base[NS][MT];
#pragma unroll
      for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
          for (int t = 0; t < NX; ++t) {
            xv[p][t][i][j] = in_order(xv[p][t][i][j]);
            const int h = NS == 2 ? j / 2 : 0;
            const bool start = t == 0 && (NS == 2 ? (j & 1) == 0 : j == 0);
            base[h][i] = mfma16<DT>(xv[p][t][i][j], neg, start ? (v4f){0.0f, 0.0f, 0.0f, 0.0f} : base[h][i]);
          }
#pragma unroll
      for (int c = 0; c < CT; ++c) {
        v4u b[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) b[j] = expand<DT>(wv[p][c][j]);
#pragma unroll
        for (int h = 0; h < NS; ++h) {
          const float s = (float)sv[p][c][h];
#pragma unroll
          for (int i = 0; i < MT; ++i) {
            v4f d = base[h][i];
#pragma unroll
            for (int j = (NS == 2 ? 2 * h : 0); j < (NS == 2 ? 2 * h + 2 : 4); ++j)
#pragma unroll
              for (int t = 0; t < NX; ++t) d = mfma16<DT>(xv[p][t][i][j], b[j], d);
#pragma unroll
            for (int r = 0; r < 4; ++r)
              acc[c][i][r] = __builtin_fmaf(XS ? d[r] * ev[p][h][i][r] : d[r], s, acc[c][i][r]);
          }
        }
      }
    }
  }

  // U (its slices in order) and L2 into LDS beside the partial tiles
  const int nthr = W * 64, cols = a.batch * a.r;
  for (int p = tid; p < a.r * MT * 16; p += nthr) {
    const int j = p / (MT * 16), row = p % (MT * 16);
    float u = 0.0f;
    if (row < a.M)
      for (int sl = 0; sl < a.u_slices; ++sl) u += a.uw[((size_t)sl * cols + proj * a.r + j) * M16 + row];
    eu[p] = u;
  }
  for (int p = tid; p < a.r * 16 * CT; p += nthr)
    el2[p] = half_or_bf(a.L2[((size_t)proj * a.r + p / (16 * CT)) * a.N + min(nt0 * 16 + p % (16 * CT), a.N - 1)], a.dtype);
  constexpr int E = CT * MT * 4;
#pragma unroll
  for (int c = 0; c < CT; ++c)
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
      for (int r = 0; r < 4; ++r) red[(wave * E + (c * MT + i) * 4 + r) * 64 + lane] = acc[c][i][r];
  __syncthreads();
  for (int o = tid; o < E * 64; o += nthr) {
    const int e = o >> 6, l = o & 63, c = e / (MT * 4), i = (e >> 2) % MT, r = e & 3;
    const int n = (nt0 + c) * 16 + (l & 15), m = i * 16 + 4 * (l >> 4) + r;
    if (n >= a.N || m >= a.M) continue;
    float y = 0.0f;
    for (int w = 0; w < W; ++w) y += red[w * E * 64 + o];
    for (int k = 0; k < a.r; ++k) y = __builtin_fmaf(eu[k * MT * 16 + m], el2[k * 16 * CT + c * 16 + (l & 15)], y);
    if (a.bias) y += half_or_bf(a.bias[(size_t)proj * a.N + n], a.dtype);
    const size_t off = ((size_t)proj * a.M + m) * a.N + n;
    if (a.y_dtype == kF32) {
      if (a.res) y += static_cast<const float *>(a.res)[off];
      static_cast<float *>(a.Y)[off] = y;
    } else {
      if (a.res) y += half_or_bf(static_cast<const uint16_t *>(a.res)[off], a.y_dtype);
      static_cast<uint16_t *>(a.Y)[off] =
          a.y_dtype == kBf16 ? __builtin_bit_cast(uint16_t, (__bf16)y) : f32_to_f16(y);
    }
  }
}

template <int DT, int MT, int CT, int P, int BPG, bool XS, int NX>
hipError_t launch_cfg(const W4a16Args &a, hipStream_t s) {
  const int NT = ceil_div(a.N, kTile), GP = ceil_div(a.K / kGroup, 2);
  const int runs = ceil_div(GP, P), most = MT == 1 ? 16 : 8;
  const int W = ceil_div(runs, ceil_div(runs, most));
  const size_t lds = ((size_t)W * CT * MT * 4 * 64 + (size_t)a.r * 16 * (MT + CT)) * sizeof(float);
  auto kernel = k_w4a16<DT, MT, CT, P, BPG, XS, NX>;
  if (lds > 64 * 1024) {
    const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void *>(kernel),
                                             hipFuncAttributeMaxDynamicSharedMemorySize, (int)lds);
    if (e != hipSuccess) return e;
  }
  hipLaunchKernelGGL(kernel, dim3((unsigned)ceil_div(NT, CT), (unsigned)a.batch), dim3((unsigned)(64 * W)), lds, s, a, W);
  return hipGetLastError();
}

template <int DT, int BPG, bool XS, int NX>
hipError_t launch_rows(const W4a16Args &a, hipStream_t s) {
  const long long tiles = (long long)ceil_div(a.N, kTile) * a.batch;
  switch (ceil_div(a.M, kTile)) {
    case 1:
      if (tiles >= 512) return launch_cfg<DT, 1, NX == 2 && BPG == 1 ? 2 : 3, 2, BPG, XS, NX>(a, s);
      return launch_cfg<DT, 1, 1, 2, BPG, XS, NX>(a, s);
    case 2: return launch_cfg<DT, 2, 2, 1, BPG, XS, NX>(a, s);
    case 3: return launch_cfg<DT, 3, 2, 1, BPG, XS, NX>(a, s);
    case 4: return launch_cfg<DT, 4, NX == 2 ? 1 : 2, 1, BPG, XS, NX>(a, s);
    default: return hipErrorInvalidValue;
  }
}

template <int BPG>
hipError_t launch_bpg(const W4a16Args &a, hipStream_t s) {
  if (a.lam) return a.terms == 2 ? launch_rows<kF16, BPG, true, 2>(a, s) : launch_rows<kF16, BPG, true, 1>(a, s);
  return a.dtype == kBf16 ? launch_rows<kBf16, BPG, false, 1>(a, s) : launch_rows<kF16, BPG, false, 1>(a, s);
}

}  // namespace

W4a16Plan plan_w4a16(int M, int K, int r, int batch, int group, bool smooth, int y_dtype) {
  W4a16Plan p;
  if (!smooth && r == 0) return p;
  p.terms = smooth && y_dtype != kBf16 ? 2 : 1;
  const int groups = K / group;
  // 32 slices of whole groups, more where M rows of one would not fit the LDS
  p.slice = std::min(ceil_div(groups, 32), std::max(1, kPrepFloats / (M * group))) * group;
  p.u_slices = ceil_div(K, p.slice);
  const int m16 = ceil_div(M, kTile) * kTile;
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
  p.total = off;
  return p;
}

hipError_t launch_w4a16(const W4a16Args &a, hipStream_t s) {
  if (a.lam || a.r > 0) {
    const size_t lds = ((size_t)a.M * a.slice + kPrepThreads) * sizeof(float);
    if (lds > 64 * 1024) {
      const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void *>(k_w4a16_prep),
                                               hipFuncAttributeMaxDynamicSharedMemorySize, (int)lds);
      if (e != hipSuccess) return e;
    }
    hipLaunchKernelGGL(k_w4a16_prep, dim3((unsigned)ceil_div(a.K, a.slice)), dim3(kPrepThreads), lds, s, a);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return a.bpg == 2 ? launch_bpg<2>(a, s) : launch_bpg<1>(a, s);
}

}  // namespace hsq
