// kv_cache.hip -- keys and values quantised to 4 bits as they are written into
// a paged cache, and read back.
//
// Per token, head and group of 64 channels x (asymmetric, symmetric):
//   lo = min(0, min x), hi = max(0, max x)      s = fp16((hi - lo) / 15)
//   z = clamp(rint(-lo / s), 0, 15)             n = clamp(rint(x / s) + z, 0, 15)
//   s = fp16(max |x| / 7), z = 8                n = clamp(rint(x / s), -8, 7) + 8
// and the value held is s (n - z).  The quotients are those of the real numbers
// s and x, ties to even: x / s is taken as x (1/s) and one correction, which
// returns a quotient exactly where fp32 holds it, and a tie is such a quotient (others
// are 2^-12 away from one, since x and s have 11 bits); 1/s may be off by a few units
// for that.  (hi - lo) / 15 is the same with 1/15 rounded correctly, which makes it
// the rounded quotient; fp32 holds hi - lo unless one of the two is below 2^-12 of the
// other, and its quotient is then more than half a unit of fp32 from any tie of fp16 but
// an exact one, so that rounding it again is harmless.  Where fp32 does not hold it
// (span_scale's branch, which data of one spread never take), the quotient is rounded to
// odd, by the sign of what is left, before it is rounded to fp16.
//
// A workgroup owns one tile of 32 token positions of one head: it quantises
// what of them the call brings (eight lanes a group, 16 bytes a lane), lays the
// tile out in LDS, and stores it whole, or, at the ends of a run, token by token
// (no byte belongs to two tokens, so nothing is read back).  A tile per workgroup is
// also what a token of a long batch needs: its 32 positions hold one row, and the
// call is as long as a launch and one read (5.2 us for 64 sequences of 8 heads).
//
// Measured, bf16, 8 heads of 128: 8192 tokens are written in 13.5 us (3.2 TB/s; 11.0
// symmetric) and read back in 11.4 (3.8), 16384 in 22.1 and 17.4 (4.9).  Writing is
// bound by its arithmetic, 80 instructions for eight channels: with IEEE divisions
// and codes packed by shifts it took 16.7 us, with one load on its way at a time 13.9.
#include "hsq_internal.h"

#include <algorithm>

namespace hsq {

namespace {

constexpr int kThreads = 256;

// The place of token row r = 0 .. 3 among the four bytes of a dword.
__device__ __forceinline__ int byte_of(int r) { return ((r & 1) << 1) | (r >> 1); }

// Offsets within a tile, by token t, group g, and lane c = 0 .. 7 of the group
// (channels 64 g + 8 c ..).
template <int D>
struct Tile {
  static constexpr int G = D / kKvGroup, kBytes = kv_tile_bytes(D);
  static constexpr int kV = 16 * D, kScale = 32 * D, kZero = 32 * D + 128 * G;
  static __device__ __forceinline__ int dword(int x, int lane) { return (x >> 2) * 1024 + lane * 16 + (x & 3) * 4; }
  static __device__ __forceinline__ int k_dword(int t, int g, int c) {
    return dword((t >> 4) * (D / 32) + 2 * g + (c >> 2), (t & 15) + 16 * (c & 3));
  }
  // channel 64 g + 8 c + j
  static __device__ __forceinline__ int v_byte(int t, int g, int c, int j) {
    return kV + dword(2 * (2 * g + (c >> 2)) + (t >> 4), (c & 1) * 8 + j + 16 * ((t >> 2) & 3)) + byte_of(t & 3);
  }
  static __device__ __forceinline__ int scale(int side, int t, int g) {
    return kScale + side * 64 * G + g * 64 + ((t >> 2) & 3) * 16 + (4 * (t >> 4) + (t & 3)) * 2;
  }
  static __device__ __forceinline__ int zero(int side, int t, int g) {
    return kZero + side * 32 * G + (((t >> 2) & 3) * G + g) * 8 + 4 * (t >> 4) + byte_of(t & 3);
  }
};

// Sequence of a workgroup, and which of its tiles it has.  n positions touch n / 32 tiles,
// rounded down, and two more at most.
__device__ __forceinline__ int block_of(const KvCache &c, int tiles, int &at) {
  if (c.searched) return kv_block(c, blockIdx.x, 1, kKvTile, 2, at);
  at = (int)(blockIdx.x % tiles);
  return (int)(blockIdx.x / tiles);
}

// The positions of a workgroup: tile number, and [lo, hi) of the positions that
// the call brings there; false where there are none.
struct Span { int b, tile, lo, hi, row0; };   // row of position p: row0 + p
__device__ __forceinline__ bool span_of(const KvCache &c, int tiles, Span &s) {
  int at, start, n;
  s.b = block_of(c, tiles, at);
  if (s.b < 0) return false;
  kv_rows(c, s.b, start, n);
  const int len = max(c.lens[s.b], 0), p0 = len - n, first = max(p0, 0);
  s.tile = first / kKvTile + at;
  s.lo = (int)max((int64_t)first, min((int64_t)s.tile * kKvTile, (int64_t)len));
  // rows beyond max_tokens are left alone: they may lie in a tile that others begin
  s.hi = (int)min((int64_t)min(kv_len(c, s.b), p0 + min(n, c.max_tokens)), (int64_t)(s.tile + 1) * kKvTile);
  s.row0 = start - p0;
  return s.lo < s.hi;
}

template <int DT>
__device__ __forceinline__ void unpack8(v4u w, float *f) {
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    f[2 * e] = DT == kBf16 ? bf16_to_f32(w[e] & 0xFFFFu) : f16_to_f32((uint16_t)w[e]);
    f[2 * e + 1] = DT == kBf16 ? __uint_as_float(w[e] & 0xFFFF0000u) : f16_to_f32((uint16_t)(w[e] >> 16));
  }
}

// Reductions over eight neighbouring lanes.
template <typename F>
__device__ __forceinline__ float over8(float v, F f) {
  v = f(v, dpp_f32<0xB1>(v));
  v = f(v, dpp_f32<0x4E>(v));
  return f(v, dpp_f32<0x141>(v));   // row_half_mirror
}

__device__ __forceinline__ uint16_t scale16(float v) {
  const uint16_t s = f32_to_f16(v);
  return s == 0x7C00u ? (uint16_t)0x7BFFu : s;
}

// x / s, ties exact (see the top of the file); inv = 1 / s
__device__ __forceinline__ float quotient(float x, float s, float inv) {
  const float r = x * inv;
  return __builtin_fmaf(__builtin_fmaf(-r, s, x), inv, r);
}

// (hi - lo) / 15 as fp16, rounded once, lo <= 0 <= hi
__device__ __forceinline__ uint16_t span_scale(float hi, float lo) {
  // (fp16 ends at 65504: nothing is lost, and no product overflows)
  const float d = fminf(hi - lo, 2097152.0f);
  float q = quotient(d, 15.0f, 1.0f / 15.0f);
  const float lost = fminf(hi, -lo) - (d - fmaxf(hi, -lo));     // of the sum, exactly, where it is not cut
  if (__builtin_expect(__any(lost != 0.0f), 0)) {
    const float left = __builtin_fmaf(-q, 15.0f, d) + lost;     // 15 times what the quotient lacks, its sign exact
    const uint32_t u = __float_as_uint(q);
    if (left != 0.0f && d < 2097152.0f) q = __uint_as_float((left < 0.0f ? u - 1 : u) | 1u);
  }
  return scale16(q);
}

// Eight lanes quantise one group; this lane's eight channels -> the codes less the
// zero, the group's scale and zero.
template <bool ASYM>
__device__ __forceinline__ float quantise(const float *x, uint16_t &s16, float *m) {
  float lo = 0.0f, hi = 0.0f;
  uint32_t ab = 0;                        // largest |x| by its bits: infinities and NaN on top
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    ab = max(ab, __float_as_uint(x[e]) & 0x7FFFFFFFu);
    if (ASYM) lo = fminf(lo, x[e]), hi = fmaxf(hi, x[e]);
  }
  ab = __float_as_uint(over8(__uint_as_float(ab), [](float p, float q) {
    return __uint_as_float(max(__float_as_uint(p), __float_as_uint(q)));
  }));
  if (ASYM) {
    lo = over8(lo, [](float p, float q) { return fminf(p, q); });
    hi = over8(hi, [](float p, float q) { return fmaxf(p, q); });
  }
  if (ab >= 0x7F800000u) {                // not finite: the whole group reads back as NaN
    s16 = 0x7E00u;
#pragma unroll
    for (int e = 0; e < 8; ++e) m[e] = 0.0f;
    return 0.0f;
  }
  s16 = ASYM ? span_scale(hi, lo) : scale16(quotient(fminf(__uint_as_float(ab), 2097152.0f), 7.0f, 1.0f / 7.0f));
  const float s = f16_to_f32(s16), inv = s > 0.0f ? __builtin_amdgcn_rcpf(s) : 0.0f;
  const float z = ASYM ? fminf(__builtin_rintf(quotient(-lo, s, inv)), 15.0f) : 8.0f;
#pragma unroll
  for (int e = 0; e < 8; ++e) m[e] = __builtin_amdgcn_fmed3f(__builtin_rintf(quotient(x[e], s, inv)), -z, 15.0f - z);
  return z;
}

template <int DT, int D, bool ASYM>
__global__ __launch_bounds__(kThreads) void k_kv_write(KvMoveArgs a, int tiles) {
  using L = Tile<D>;
  constexpr int G = L::G;
  __shared__ __attribute__((aligned(16))) uint8_t buf[L::kBytes];
  Span sp;
  if (!span_of(a.c, tiles, sp)) return;
  const int h = blockIdx.y, tid = threadIdx.x;
  uint8_t *dst = const_cast<uint8_t *>(kv_tile_at(a.c, sp.b, h, sp.tile));
  if (!dst) return;
  const int c = tid & 7, p0 = sp.tile * kKvTile;
  static_assert(32 * G * 8 == G * kThreads, "a side is G passes of the workgroup");
  v4u raw[2 * G];                         // all on their way at once
#pragma unroll
  for (int it = 0; it < 2 * G; ++it) {
    const int side = it / G, i = (it % G) * kThreads + tid, g = (i >> 3) % G, p = p0 + (i >> 3) / G;
    const int q = min(max(p, (int)sp.lo), (int)sp.hi - 1);      // no position of the call: not stored
    raw[it] = *reinterpret_cast<const v4u *>(static_cast<const uint16_t *>(side ? a.v : a.k) +
                                             (size_t)(sp.row0 + q) * (side ? a.v_stride : a.k_stride) + h * D + 64 * g + 8 * c);
  }
  __builtin_amdgcn_sched_barrier(0);
#pragma unroll
  for (int it = 0; it < 2 * G; ++it) {
    const int side = it / G, i = (it % G) * kThreads + tid, g = (i >> 3) % G, t = (i >> 3) / G;
    float x[8];
    unpack8<DT>(raw[it], x);
    // small whole numbers: packed as such, which is an instruction a code
    uint16_t s16;
    float m[8];
    const float z = quantise<ASYM>(x, s16, m);
    if (side == 0) {
      // channels 0 1 2 3 | 4 5 6 7 -> bytes 0 2 1 3, low | high nibbles
      float b[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) b[e] = __builtin_fmaf(m[4 + e], 16.0f, m[e]);
      const float lo = __builtin_fmaf(b[2], 256.0f, b[0]), hi = __builtin_fmaf(b[3], 256.0f, b[1]);
      *reinterpret_cast<uint32_t *>(buf + L::k_dword(t, g, c)) =
          (uint32_t)__builtin_fmaf(z, 4369.0f, lo) | (uint32_t)__builtin_fmaf(z, 4369.0f, hi) << 16;
    } else {
      // lanes c and c ^ 2 hold the two halves of the same bytes; each stores four
      uint32_t w[2];                       // four nibbles each
#pragma unroll
      for (int y = 0; y < 2; ++y) {
        const float *n = m + 4 * y;
        const float lo = __builtin_fmaf(n[1], 16.0f, n[0]), hi = __builtin_fmaf(n[3], 16.0f, n[2]);
        w[y] = (uint32_t)__builtin_fmaf(z, 4369.0f, __builtin_fmaf(hi, 256.0f, lo));
      }
      const bool high = c & 2;
      const uint32_t send = high ? w[0] : w[1], keep = high ? w[1] : w[0];
      const uint32_t got = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)send, 0x4E, 0xF, 0xF, false);
      auto spread = [](uint32_t v) {       // nibbles to bytes
        v = (v | v << 8) & 0x00FF00FFu;
        return (v | v << 4) & 0x0F0F0F0Fu;
      };
      const uint32_t v = spread(high ? got : keep) | spread(high ? keep : got) << 4;
#pragma unroll
      for (int e = 0; e < 4; ++e) buf[L::v_byte(t, g, c, (high ? 4 : 0) + e)] = (uint8_t)(v >> (8 * e));
    }
    if (c == 0) {
      *reinterpret_cast<uint16_t *>(buf + L::scale(side, t, g)) = s16;
      buf[L::zero(side, t, g)] = (uint8_t)(16.0f + z);
    }
  }
  __syncthreads();
  if (sp.hi - sp.lo == kKvTile) {
    for (int i = tid; i < L::kBytes / 16; i += kThreads)
      reinterpret_cast<v4u *>(dst)[i] = reinterpret_cast<const v4u *>(buf)[i];
    return;
  }
  // single tokens: D / 8 dwords of K, D / 2 bytes of V, 2 G scales and zeros each
  constexpr int kItems = D / 8 + D / 2 + 4 * G;
  for (int i = tid; i < (sp.hi - sp.lo) * kItems; i += kThreads) {
    const int t = sp.lo - p0 + i / kItems, e = i % kItems;
    if (e < D / 8) {
      const int off = L::k_dword(t, e >> 3, e & 7);
      *reinterpret_cast<uint32_t *>(dst + off) = *reinterpret_cast<const uint32_t *>(buf + off);
    } else if (e < D / 8 + D / 2) {
      const int d = e - D / 8;            // pair d of channels: 32 (d / 16) + d % 16 and 16 more
      const int off = L::v_byte(t, d >> 5, ((d >> 4) & 1) * 4 + ((d >> 3) & 1), d & 7);
      dst[off] = buf[off];
    } else {
      const int f = e - D / 8 - D / 2, side = f & 1, g = (f >> 1) % G;
      if (f >= 2 * G) {
        const int off = L::zero(side, t, g);
        dst[off] = buf[off];
      } else {
        const int off = L::scale(side, t, g);
        *reinterpret_cast<uint16_t *>(dst + off) = *reinterpret_cast<const uint16_t *>(buf + off);
      }
    }
  }
}

template <int DT, int D>
__global__ __launch_bounds__(kThreads) void k_kv_read(KvMoveArgs a, int tiles) {
  using L = Tile<D>;
  constexpr int G = L::G;
  __shared__ __attribute__((aligned(16))) uint8_t buf[L::kBytes];
  int at, start, n;
  const int b = block_of(a.c, tiles, at), h = blockIdx.y, tid = threadIdx.x, c = tid & 7;
  if (b < 0) return;
  kv_rows(a.c, b, start, n);
  // row i of the sequence is position p0 + i; one that holds nothing (negative,
  // past the table, on no page) is a row all the same, and reads zero
  const int p0 = max(a.c.lens[b], 0) - n, len = kv_len(a.c, b), rows = min(n, a.c.max_tokens);
  const int first = p0 >= 0 ? p0 / kKvTile : -((kKvTile - 1 - p0) / kKvTile);
  const int tile = first + at;
  const int64_t base = (int64_t)tile * kKvTile;
  if (base >= (int64_t)p0 + rows) return;
  const uint8_t *src = base >= 0 && base < len ? kv_tile_at(a.c, b, h, tile) : nullptr;
  if (src) {
    for (int i = tid; i < L::kBytes / 16; i += kThreads)
      reinterpret_cast<v4u *>(buf)[i] = reinterpret_cast<const v4u *>(src)[i];
  }
  __syncthreads();
#pragma unroll
  for (int it = 0; it < 2 * G; ++it) {
    const int side = it / G, i = (it % G) * kThreads + tid;
    const int g = (i >> 3) % G, t = (i >> 3) / G;
    const int64_t p = base + t, row = p - p0;
    if (row < 0 || row >= rows) continue;
    float y[8] = {0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f};
    if (src && p < len) {
      const float s = f16_to_f32(*reinterpret_cast<const uint16_t *>(buf + L::scale(side, t, g)));
      const int z = (int)buf[L::zero(side, t, g)] - 16;
      if (side == 0) {
        const uint32_t w = *reinterpret_cast<const uint32_t *>(buf + L::k_dword(t, g, c));
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const int n4 = (int)(w >> (8 * byte_of(j & 3) + 4 * (j >> 2)) & 0xFu);
          y[j] = s * (float)(n4 - z);
        }
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const int n4 = buf[L::v_byte(t, g, c, j)] >> (c & 2 ? 4 : 0) & 0xF;
          y[j] = s * (float)(n4 - z);
        }
      }
    }
    const size_t off = (size_t)(start + row) * (side ? a.v_stride : a.k_stride) + h * D + 64 * g + 8 * c;
    void *out = side ? a.v : a.k;
    if constexpr (DT == kF32) {
      float4 *o = reinterpret_cast<float4 *>(static_cast<float *>(out) + off);
      o[0] = make_float4(y[0], y[1], y[2], y[3]);
      o[1] = make_float4(y[4], y[5], y[6], y[7]);
    } else {
      v4u w;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        uint32_t u[2];
#pragma unroll
        for (int q = 0; q < 2; ++q)
          u[q] = DT == kBf16 ? __builtin_bit_cast(uint16_t, (__bf16)y[2 * e + q]) : f32_to_f16(y[2 * e + q]);
        w[e] = u[0] | u[1] << 16;
      }
      *reinterpret_cast<v4u *>(static_cast<uint16_t *>(out) + off) = w;
    }
  }
}

template <int D>
hipError_t write_d(const KvMoveArgs &a, const KvBlocks &p, hipStream_t s) {
  const int tiles = (int)p.each;
  const dim3 grid((unsigned)p.total, (unsigned)a.c.H);
  if (a.dtype == kBf16) {
    if (a.asym) hipLaunchKernelGGL((k_kv_write<kBf16, D, true>), grid, dim3(kThreads), 0, s, a, tiles);
    else hipLaunchKernelGGL((k_kv_write<kBf16, D, false>), grid, dim3(kThreads), 0, s, a, tiles);
  } else {
    if (a.asym) hipLaunchKernelGGL((k_kv_write<kF16, D, true>), grid, dim3(kThreads), 0, s, a, tiles);
    else hipLaunchKernelGGL((k_kv_write<kF16, D, false>), grid, dim3(kThreads), 0, s, a, tiles);
  }
  return hipGetLastError();
}

template <int D>
hipError_t read_d(const KvMoveArgs &a, const KvBlocks &p, hipStream_t s) {
  const int tiles = (int)p.each;
  const dim3 grid((unsigned)p.total, (unsigned)a.c.H);
  if (a.dtype == kBf16) hipLaunchKernelGGL((k_kv_read<kBf16, D>), grid, dim3(kThreads), 0, s, a, tiles);
  else if (a.dtype == kF16) hipLaunchKernelGGL((k_kv_read<kF16, D>), grid, dim3(kThreads), 0, s, a, tiles);
  else hipLaunchKernelGGL((k_kv_read<kF32, D>), grid, dim3(kThreads), 0, s, a, tiles);
  return hipGetLastError();
}

}  // namespace

// Tiles that max_tokens positions in a row can touch, to each sequence.
KvBlocks plan_kv_move(const KvCache &c) {
  return kv_blocks(c, (c.max_tokens + 2LL * kKvTile - 2) / kKvTile, 1, kKvTile, 2);
}

hipError_t launch_kv_write(KvMoveArgs a, hipStream_t s) {
  const KvBlocks p = plan_kv_move(a.c);
  a.c.searched = p.searched;
  switch (a.c.D) {
    case 64: return write_d<64>(a, p, s);
    case 128: return write_d<128>(a, p, s);
    case 256: return write_d<256>(a, p, s);
    default: return hipErrorInvalidValue;
  }
}

hipError_t launch_kv_read(KvMoveArgs a, hipStream_t s) {
  const KvBlocks p = plan_kv_move(a.c);
  a.c.searched = p.searched;
  switch (a.c.D) {
    case 64: return read_d<64>(a, p, s);
    case 128: return read_d<128>(a, p, s);
    case 256: return read_d<256>(a, p, s);
    default: return hipErrorInvalidValue;
  }
}

}  // namespace hsq
