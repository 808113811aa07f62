// layer_norm.hip -- layer normalisation over the last dimension, forward and
// backward, for 16-bit and fp32 rows.
//
//   mean = (1/C) sum_c x,  rstd = (mean of (x - mean)^2 + eps)^(-1/2)
//   y    = (x - mean) rstd w + b
// and, with xh = (x - mean) rstd and g = dy w,
//   dx   = rstd (g - mean_c(g) - xh mean_c(g xh))
//   dw   = sum over the rows of a group of dy xh,  db = sum of dy.
//
// Both passes are bound by HBM: a row is read once into registers (the
// variance is summed from the registers around the finished mean, so a
// large common offset costs no precision) and written once.  A row belongs
// to one wave, four waves or eight, the fewest whose registers hold it.
// Statistics and parameter sums are fp32.
//
// Measured on an MI355X (a large copy: 4.92 TB/s): 8192 x 1152 bf16 with
// parameters per half of the rows, forward 11-12 us (38 MB; one row alone takes
// 3 us), backward 18.6 us a call in a stream of calls (57 MB, 3.1 TB/s; under
// the tracer its two launches take 18.0 and 3.8); 1537 x 2241 fp32 backward 16
// us (35 MB).  The backward pass runs eight waves a CU, too few for the memory:
// its accumulators leave no room for more at these widths.  Rows that do not
// start on 16 bytes: 8192 x 8191 76 us, 8192 x 8192 48.
#include "hsq_internal.h"

#include <algorithm>

namespace hsq {

namespace {

// Eight consecutive elements of a row.  Rows of a length that is no
// multiple of 8 start at any element, so the 16-byte accesses are typed
// with the element's alignment (global memory takes them as they come).
struct __attribute__((packed, aligned(2))) V16 { uint32_t d[4]; };
struct __attribute__((packed, aligned(4))) V32 { float f[8]; };

template <int DT>
__device__ __forceinline__ void put(void *p, size_t i, float v) {
  if constexpr (DT == kF32) static_cast<float *>(p)[i] = v;
  if constexpr (DT == kBf16) static_cast<__bf16 *>(p)[i] = (__bf16)v;
  if constexpr (DT == kF16) static_cast<_Float16 *>(p)[i] = (_Float16)v;
}

// Eight elements as loaded; n of them from i on exist, the others read 0.
template <int DT>
struct Run { uint32_t d[DT == kF32 ? 8 : 4]; };

template <int DT>
__device__ __forceinline__ Run<DT> load_run(const void *p, size_t i, int n) {
  Run<DT> r{};
  if (n >= 8) {
    if constexpr (DT == kF32) {
      const V32 t = *reinterpret_cast<const V32 *>(static_cast<const float *>(p) + i);
#pragma unroll
      for (int e = 0; e < 8; ++e) r.d[e] = __float_as_uint(t.f[e]);
    } else {
      const V16 t = *reinterpret_cast<const V16 *>(static_cast<const uint16_t *>(p) + i);
#pragma unroll
      for (int e = 0; e < 4; ++e) r.d[e] = t.d[e];
    }
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (e < n) {
        if constexpr (DT == kF32) r.d[e] = static_cast<const uint32_t *>(p)[i + e];
        else r.d[e / 2] |= (uint32_t)static_cast<const uint16_t *>(p)[i + e] << (16 * (e & 1));
      }
  }
  return r;
}

template <int DT>
__device__ __forceinline__ float value(const Run<DT> &r, int e) {
  if constexpr (DT == kF32) return __uint_as_float(r.d[e]);
  const uint32_t h = (r.d[e / 2] >> (16 * (e & 1))) & 0xFFFFu;
  return DT == kBf16 ? bf16_to_f32(h) : f16_to_f32((uint16_t)h);
}

template <int DT>
__device__ __forceinline__ void load8(const void *p, size_t i, int n, float v[8]) {
  const Run<DT> r = load_run<DT>(p, i, n);
#pragma unroll
  for (int e = 0; e < 8; ++e) v[e] = value<DT>(r, e);
}

template <int DT>
__device__ __forceinline__ void store8(void *p, size_t i, int n, const float v[8]) {
  if (n >= 8) {
    if constexpr (DT == kF32) {
      V32 t;
#pragma unroll
      for (int e = 0; e < 8; ++e) t.f[e] = v[e];
      *reinterpret_cast<V32 *>(static_cast<float *>(p) + i) = t;
    } else {
      uint16_t h[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) put<DT>(h, e, v[e]);
      V16 t;
#pragma unroll
      for (int e = 0; e < 4; ++e) t.d[e] = (uint32_t)h[2 * e] | ((uint32_t)h[2 * e + 1] << 16);
      *reinterpret_cast<V16 *>(static_cast<uint16_t *>(p) + i) = t;
    }
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (e < n) put<DT>(p, i + e, v[e]);
  }
}

// parameters are fp32 or of the 16-bit type of Y
template <int DT>
__device__ __forceinline__ void load8p(const void *p, bool f32, size_t i, int n, float v[8]) {
  if (f32) load8<kF32>(p, i, n, v);
  else load8<DT>(p, i, n, v);
}

__device__ __forceinline__ float wave_sum(float v) {
  v = row16_sum(v);
  v += __shfl_xor(v, 16);
  return v + __shfl_xor(v, 32);
}

// Sum over the W waves of a row; every lane of the row returns it.  Two
// sums of one row alternate between two LDS slots, so one barrier each.
template <int W>
__device__ __forceinline__ float row_sum(float v, float *slot, int wave) {
  v = wave_sum(v);
  if constexpr (W > 1) {
    if ((threadIdx.x & 63) == 0) slot[wave] = v;
    __syncthreads();
    v = 0.0f;
#pragma unroll
    for (int w = 0; w < W; ++w) v += slot[w];
  }
  return v;
}

constexpr int kRowThreads = 256;   // threads of a workgroup with one or four waves to a row

template <int W>
constexpr int norm_threads() { return W > 4 ? W * 64 : kRowThreads; }

// W waves to a row, NV runs of 8 elements to a lane: C <= 512 W NV.  A launch
// has sixteen waves a CU that go from row to row with the next one on its way:
// 8192 x 8192 bf16 47 us (5.7 TB/s) against 60 with a workgroup per row, 4096 x
// 2240 fp32 16 against 19, 16384 x 1152 18 against 21; 32 waves 52, 17 and 19.
// Above 12288 channels, and for fp32 rows above 8192, a lane needs more than 128
// registers and eight of the waves are resident: the workgroups run in two
// rounds (4096 x 16384 bf16 54 us, 5.0 TB/s; 2048 x 12288 fp32 42 us, 4.8).
template <int TX, int TY, int W, int NV>
__global__ __launch_bounds__(norm_threads<W>()) void k_layer_norm(NormArgs a) {
  constexpr int RPB = norm_threads<W>() / (64 * W);     // rows per workgroup
  __shared__ float red[4][W > 1 ? W : 1];
  const int t = threadIdx.x % (64 * W), wave = t >> 6;
  const bool pf = a.p_dtype == kF32;
  // the next row is loaded while this one is worked on; the parameters stay in
  // registers from row to row of a group
  Run<TX> nx[NV];
  auto fetch = [&](int row) __attribute__((always_inline)) {
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int c = 8 * (t + v * 64 * W);
      nx[v] = load_run<TX>(a.X, (size_t)row * a.C + c, a.C - c);
    }
  };
  float w[NV][8], b[NV][8];
  int group = -1, turn = 0;
  int row = blockIdx.x * RPB + threadIdx.x / (64 * W);
  if (row < a.M) fetch(row);
  for (; row < a.M; row += gridDim.x * RPB, turn ^= 2) {   // (no barrier with W = 1, one row at a time with more)
    if (group != row / a.rows) {
      group = row / a.rows;
      const size_t g = (size_t)group * a.C;
#pragma unroll
      for (int v = 0; v < NV; ++v) {
        const int c = 8 * (t + v * 64 * W);
        if (a.w) load8p<TY>(a.w, pf, g + c, a.C - c, w[v]);
        if (a.b) load8p<TY>(a.b, pf, g + c, a.C - c, b[v]);
      }
    }
    const size_t base = (size_t)row * a.C;
    float x[NV][8];
    float s = 0.0f;
#pragma unroll
    for (int v = 0; v < NV; ++v)
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        x[v][e] = value<TX>(nx[v], e);
        s += x[v][e];
      }
    if (row + (int)gridDim.x * RPB < a.M) fetch(row + gridDim.x * RPB);
    const float mean = row_sum<W>(s, red[turn], wave) / (float)a.C;
    float q = 0.0f;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int c = 8 * (t + v * 64 * W);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float d = c + e < a.C ? x[v][e] - mean : 0.0f;
        q = fmaf(d, d, q);
      }
    }
    const float rstd = 1.0f / sqrtf(row_sum<W>(q, red[turn + 1], wave) / (float)a.C + a.eps);
    if (t == 0) {
      if (a.mean) a.mean[row] = mean;
      if (a.rstd) a.rstd[row] = rstd;
    }
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int c = 8 * (t + v * 64 * W), n = a.C - c;
      if (n <= 0) continue;
      float y[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) y[e] = (x[v][e] - mean) * rstd;
      if (a.w) {
#pragma unroll
        for (int e = 0; e < 8; ++e) y[e] *= w[v][e];
      }
      if (a.b) {
#pragma unroll
        for (int e = 0; e < 8; ++e) y[e] += b[v][e];
      }
      store8<TY>(a.Y, base + c, n, y);
    }
  }
}

// Backward: workgroup p of group gi takes RPB rows at a time of the group (a
// row to one wave, four or eight), keeps its columns' sums of dy xh and dy in
// registers and writes them as one partial row; the partial rows are summed
// by k_sum_parts.  The next row is loaded while this one is
// worked on, where the registers allow it (NV < 4).
constexpr int kBwdWaves = 8;

template <int TX, int TY, int W, int NV>
__global__ __launch_bounds__(64 * kBwdWaves) void k_layer_norm_bwd(NormArgs a) {
  constexpr int RPB = kBwdWaves / W;
  __shared__ float red[4][RPB][W];
  __shared__ float comb[RPB > 1 ? RPB - 1 : 1][RPB > 1 ? 1024 * W : 1];
  const int t = threadIdx.x % (64 * W), wave = t >> 6, sub = threadIdx.x / (64 * W);
  const int gi = blockIdx.y;
  const size_t g = (size_t)gi * a.C;
  const bool pf = a.p_dtype == kF32;
  float w[NV][8], dw[NV][8], db[NV][8];
#pragma unroll
  for (int v = 0; v < NV; ++v) {
    const int c = 8 * (t + v * 64 * W);
    if (a.w) load8p<TY>(a.w, pf, g + c, a.C - c, w[v]);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      if (!a.w) w[v][e] = 1.0f;
      dw[v][e] = db[v][e] = 0.0f;
    }
  }
  constexpr bool kAhead = NV < 4;
  Run<TX> nx[NV];
  Run<TY> ny[NV];
  float nmean = 0.0f, nrstd = 0.0f;
  auto fetch = [&](int r) __attribute__((always_inline)) {   // rows past the group's: zeros
    const bool has = r < a.rows;
    const size_t row = (size_t)gi * a.rows + (has ? r : 0), base = row * a.C;
    nmean = a.mean[row];
    nrstd = a.rstd[row];
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int c = 8 * (t + v * 64 * W), n = has ? a.C - c : 0;
      nx[v] = load_run<TX>(a.X, base + c, n);
      ny[v] = load_run<TY>(a.dY, base + c, n);
    }
  };
  const int stride = gridDim.x * RPB;
  int turn = 0;
  if (kAhead) fetch(blockIdx.x * RPB + sub);
  for (int r0 = blockIdx.x * RPB; r0 < a.rows; r0 += stride, turn ^= 2) {
    const int r = r0 + sub;
    const bool has = r < a.rows;
    if (!kAhead) fetch(r);
    const size_t base = ((size_t)gi * a.rows + r) * a.C;
    const float mean = nmean, rstd = nrstd;
    float xh[NV][8], gr[NV][8];
    float s1 = 0.0f, s2 = 0.0f;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int c = 8 * (t + v * 64 * W);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float h = has && c + e < a.C ? (value<TX>(nx[v], e) - mean) * rstd : 0.0f;
        const float dy = value<TY>(ny[v], e);
        dw[v][e] = fmaf(dy, h, dw[v][e]);
        db[v][e] += dy;
        xh[v][e] = h;
        gr[v][e] = dy * w[v][e];
        s1 += gr[v][e];
        s2 = fmaf(gr[v][e], h, s2);
      }
    }
    if (kAhead && r0 + stride < a.rows) fetch(r + stride);
    if (a.dX) {
      const float c1 = row_sum<W>(s1, red[turn][sub], wave) / (float)a.C;
      const float c2 = row_sum<W>(s2, red[turn + 1][sub], wave) / (float)a.C;
#pragma unroll
      for (int v = 0; v < NV; ++v) {
        const int c = 8 * (t + v * 64 * W);
        if (!has || a.C - c <= 0) continue;
        float d[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) d[e] = rstd * (gr[v][e] - c1 - xh[v][e] * c2);
        store8<TX>(a.dX, base + c, a.C - c, d);
      }
    }
  }
  if (!a.part) return;
  // the rows' shares in order, 512 W columns at a time
  float *out = a.part + ((size_t)gi * a.parts + blockIdx.x) * 2 * a.C;
#pragma unroll
  for (int v = 0; v < NV; ++v) {
    const int c = 8 * (t + v * 64 * W), n = a.C - c;
    if constexpr (RPB > 1) {
      __syncthreads();
      if (sub > 0)
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          comb[sub - 1][e * 64 * W + t] = dw[v][e];
          comb[sub - 1][512 * W + e * 64 * W + t] = db[v][e];
        }
      __syncthreads();
      if (sub == 0)
        for (int k = 0; k < RPB - 1; ++k)
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            dw[v][e] += comb[k][e * 64 * W + t];
            db[v][e] += comb[k][512 * W + e * 64 * W + t];
          }
    }
    if (sub == 0 && n > 0) {
      store8<kF32>(out, c, n, dw[v]);
      store8<kF32>(out, (size_t)a.C + c, n, db[v]);
    }
  }
}

// Sums of partial rows: 32 columns per workgroup, 32 shares of the rows each
// with four rows in flight, the shares summed in order.  Grid z: the
// second half of a partial row (the norm's db beside dw).
constexpr int kSumCols = 32, kSumShares = 32;
__global__ __launch_bounds__(kSumCols * kSumShares) void k_sum_parts(SumArgs a) {
  __shared__ float sh[kSumShares][kSumCols + 1];
  void *dst = blockIdx.z == 0 ? a.dst : a.dst2;
  const int cx = threadIdx.x % kSumCols, y = threadIdx.x / kSumCols;
  const int c = blockIdx.x * kSumCols + cx, g = blockIdx.y;
  const float *src = a.src + (size_t)g * a.parts * a.ld + (blockIdx.z == 0 ? 0 : a.C) + c;
  float s[4] = {0.0f, 0.0f, 0.0f, 0.0f};
  if (c < a.C) {
    int p = y;
    for (; p + 3 * kSumShares < a.parts; p += 4 * kSumShares) {
      float v[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) v[k] = src[(size_t)(p + k * kSumShares) * a.ld];
#pragma unroll
      for (int k = 0; k < 4; ++k) s[k] += v[k];
    }
    for (; p < a.parts; p += kSumShares) s[0] += src[(size_t)p * a.ld];
  }
  sh[y][cx] = (s[0] + s[1]) + (s[2] + s[3]);
  __syncthreads();
  if (y != 0 || c >= a.C) return;
  float v = 0.0f;
#pragma unroll
  for (int k = 0; k < kSumShares; ++k) v += sh[k][cx];
  const size_t o = (size_t)g * a.C + c;
  if (a.dtype == kF32) put<kF32>(dst, o, v);
  else if (a.dtype == kBf16) put<kBf16>(dst, o, v);
  else put<kF16>(dst, o, v);
}

template <int TX, int TY, int W, int NV>
hipError_t run_norm(const NormArgs &a, bool backward, hipStream_t s) {
  // forward: a grid of sixteen waves a CU, each going from row to row
  constexpr int RPB = norm_threads<W>() / (64 * W), kGrid = 256 * 1024 / norm_threads<W>();
  if (backward)
    hipLaunchKernelGGL((k_layer_norm_bwd<TX, TY, W, NV>), dim3((unsigned)a.parts, (unsigned)a.groups),
                       dim3(64 * kBwdWaves), 0, s, a);
  else
    hipLaunchKernelGGL((k_layer_norm<TX, TY, W, NV>), dim3((unsigned)std::min(ceil_div(a.M, RPB), kGrid)),
                       dim3(norm_threads<W>()), 0, s, a);
  return hipGetLastError();
}

template <int TX, int TY>
hipError_t pick_width(const NormArgs &a, bool backward, hipStream_t s) {
  if (a.C <= 512) return run_norm<TX, TY, 1, 1>(a, backward, s);
  if (a.C <= 1024) return run_norm<TX, TY, 1, 2>(a, backward, s);
  if (a.C <= 1536) return run_norm<TX, TY, 1, 3>(a, backward, s);
  if (a.C <= 2048) return run_norm<TX, TY, 4, 1>(a, backward, s);
  if (a.C <= 4096) return run_norm<TX, TY, 4, 2>(a, backward, s);
  if (a.C <= 8192) return run_norm<TX, TY, 8, 2>(a, backward, s);
  if (a.C <= 12288) return run_norm<TX, TY, 8, 3>(a, backward, s);
  return run_norm<TX, TY, 8, 4>(a, backward, s);
}

hipError_t pick_types(const NormArgs &a, bool backward, hipStream_t s) {
  if (a.x_dtype == kBf16) return pick_width<kBf16, kBf16>(a, backward, s);
  if (a.x_dtype == kF16) return pick_width<kF16, kF16>(a, backward, s);
  if (a.y_dtype == kBf16) return pick_width<kF32, kBf16>(a, backward, s);
  if (a.y_dtype == kF16) return pick_width<kF32, kF16>(a, backward, s);
  return pick_width<kF32, kF32>(a, backward, s);
}

}  // namespace

// Workgroups per group of the backward pass: one per CU over all groups (each
// keeps its rows' sums in registers and writes one partial row), fewer where
// a workgroup would not get two turns of rows.
int norm_backward_parts(int M, int C, int groups) {
  const int rows = M / groups, rpb = C <= 1536 ? 8 : C <= 4096 ? 2 : 1;
  return std::max(1, std::min(ceil_div(rows, 2 * rpb), std::max(1, 256 / groups)));
}

hipError_t launch_layer_norm(const NormArgs &a, hipStream_t s) { return pick_types(a, false, s); }
hipError_t launch_layer_norm_backward(const NormArgs &a, hipStream_t s) { return pick_types(a, true, s); }

hipError_t launch_sum_parts(const SumArgs &a, int groups, hipStream_t s) {
  SumArgs b = a;
  const bool both = a.dst && a.dst2;
  if (!a.dst) {
    b.src += a.C;
    b.dst = a.dst2;
  }
  hipLaunchKernelGGL(k_sum_parts, dim3((unsigned)ceil_div(a.C, kSumCols), (unsigned)groups, both ? 2u : 1u),
                     dim3(kSumCols * kSumShares), 0, s, b);
  return hipGetLastError();
}

}  // namespace hsq
