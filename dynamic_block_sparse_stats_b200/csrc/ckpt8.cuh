// The 8-bit activation checkpoint: a row's channels in blocks of 32, each block
// held as signed 8-bit codes and one power-of-two scale 2^(s - 127).
//   s     the smallest integer >= 1 with max|x| <= 127 * 2^(s - 127)
//   code  x / 2^(s - 127) rounded to nearest, ties to even (|code| <= 127)
// A code times its scale has at most 7 significant bits, so it is exact in
// bf16 and the tensor cores multiply the stored values without a second
// rounding; the rounding of the checkpoint itself is at most half a scale, less
// than 1/127 of the block's largest value unless s = 1 (int8 with a power-of-two
// scale: about a third of the error that an 8-bit float with 3 mantissa bits makes
// on normally distributed values, whose error grows with the value).  A block that
// holds an infinity or NaN gets s = 255 and codes 0, which restore as 0 * inf = NaN.
// Finite values above 127 * 2^121 (the upper 0.4% of the last binade) are held
// as that value: a larger scale could restore them as infinities.
#pragma once

#include "common.cuh"

namespace prism {

constexpr int kCkptBlock = 32;    // channels per scale
constexpr int kCkptRow = 128;     // row lengths of codes are padded to this
constexpr uint32_t kCkptBad = 255;
constexpr uint32_t kCkptTop = 0x7f7e0000u;  // bits of 127 * 2^121

// s from the bits of max|x| (fp32): 127 = 1.984375 * 2^6, so s = e - 6 for a
// significand up to 1.984375 and e - 5 above it (the addition carries into the
// exponent exactly then).
__device__ __forceinline__ uint32_t ckpt8_scale(uint32_t max_bits) {
  if (max_bits >= 0x7f800000u) return kCkptBad;
  const int s = (int)((min(max_bits, kCkptTop) + 0x1ffffu) >> 23) - 6;
  return (uint32_t)(s < 1 ? 1 : s);
}
// 2^(127 - s), the factor before rounding; 0 for a bad block
__device__ __forceinline__ float ckpt8_inverse(uint32_t s) { return __uint_as_float(s == kCkptBad ? 0u : (254u - s) << 23); }

__device__ __forceinline__ float ckpt8_clamp(float x) {
  const float top = __uint_as_float(kCkptTop);
  return fminf(fmaxf(x, -top), top);
}

// four codes in a word: x * inv + 1.5 * 2^23 rounds x * inv (exact: a power of
// two) to an integer, whose two's complement stands in the low bits
__device__ __forceinline__ uint32_t ckpt8_code4(float a, float b, float c, float d, float inv) {
  const float2 lo = ffma2(make_float2(a, b), inv, 12582912.f), hi = ffma2(make_float2(c, d), inv, 12582912.f);
  return __byte_perm(__byte_perm(__float_as_uint(lo.x), __float_as_uint(lo.y), 0x0040),
                     __byte_perm(__float_as_uint(hi.x), __float_as_uint(hi.y), 0x0040), 0x5410);
}

// one block held by one thread: returns s, codes in q
__device__ __forceinline__ uint32_t ckpt8_quantise(const float2 (&v)[16], uint32_t (&q)[8]) {
  // magnitudes as integers: a NaN compares above everything, so it is never lost
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < 16; ++i)
    top = max(top, max(__float_as_uint(v[i].x) & 0x7fffffffu, __float_as_uint(v[i].y) & 0x7fffffffu));
  const uint32_t s = ckpt8_scale(top);
  const float inv = ckpt8_inverse(s);
  if (top <= kCkptTop) {
#pragma unroll
    for (int i = 0; i < 8; ++i) q[i] = ckpt8_code4(v[2 * i].x, v[2 * i].y, v[2 * i + 1].x, v[2 * i + 1].y, inv);
  } else if (s == kCkptBad) {
#pragma unroll
    for (int i = 0; i < 8; ++i) q[i] = 0;
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      q[i] = ckpt8_code4(ckpt8_clamp(v[2 * i].x), ckpt8_clamp(v[2 * i].y), ckpt8_clamp(v[2 * i + 1].x),
                         ckpt8_clamp(v[2 * i + 1].y), inv);
  }
  return s;
}

__device__ __forceinline__ uint32_t hadd2_bf16(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("add.rn.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
__device__ __forceinline__ uint32_t hmul2_bf16(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
// two codes in the bytes `sel` picks (as 16-bit lanes) -> bf16 pair times the
// scale pair.  A code c = low7 - 128 * sign is (128 + low7) - (sign ? 256 : 128):
// both terms are bit patterns of the byte, their sum and its product are exact.
__device__ __forceinline__ uint32_t ckpt8_restore2(uint32_t word, uint32_t sel, uint32_t scale2) {
  const uint32_t b = __byte_perm(word, 0, sel);
  const uint32_t x = (b & 0x007f007fu) | 0x43004300u;
  const uint32_t y = (b & 0x00800080u) | 0xc300c300u;
  return hmul2_bf16(hadd2_bf16(x, y), scale2);
}
__device__ __forceinline__ uint32_t ckpt8_scale2(uint32_t s) { return (s << 7) | (s << 23); }
// 16 codes of one block -> 16 bf16 (lo: the first eight)
__device__ __forceinline__ void ckpt8_restore16(const uint4 &q, uint32_t s, uint4 &lo, uint4 &hi) {
  const uint32_t s2 = ckpt8_scale2(s);
  lo = make_uint4(ckpt8_restore2(q.x, 0x4140, s2), ckpt8_restore2(q.x, 0x4342, s2), ckpt8_restore2(q.y, 0x4140, s2),
                  ckpt8_restore2(q.y, 0x4342, s2));
  hi = make_uint4(ckpt8_restore2(q.z, 0x4140, s2), ckpt8_restore2(q.z, 0x4342, s2), ckpt8_restore2(q.w, 0x4140, s2),
                  ckpt8_restore2(q.w, 0x4342, s2));
}

// Groups 0 .. groups-1, gpr to a row; a half-warp takes every nhalf-th.  Its
// place (row, group of the row) moves by (row_step, col_step), nhalf divided by gpr.
struct Walk {
  long long groups, nhalf, row_step;
  int gpr, col_step;
};
struct Place {
  long long g, row;
  int col;
  __device__ __forceinline__ Place(const Walk &w, long long start) : g(start), row(start / w.gpr) {
    col = (int)(start - row * w.gpr);
  }
  __device__ __forceinline__ void step(const Walk &w) {
    g += w.nhalf;
    row += w.row_step;
    col += w.col_step;
    if (col >= w.gpr) {
      col -= w.gpr;
      ++row;
    }
  }
};

inline Walk make_walk(long long n, long long ld, long long nhalf) {
  Walk w;
  w.gpr = (int)(ld / 128);
  w.groups = n * w.gpr;
  w.nhalf = nhalf;
  w.row_step = nhalf / w.gpr;
  w.col_step = (int)(nhalf % w.gpr);
  return w;
}

// The half-warp `half` of `w.nhalf` restores its groups, UNROLL at a time; vec:
// 16-byte vectors of a row that exist.
template <int UNROLL>
__device__ __forceinline__ void unpack_walk(const uint2 *__restrict__ codes, const uint8_t *__restrict__ scales,
                                            const Walk &w, int vec, uint4 *__restrict__ x, long long ld_vec,
                                            long long half) {
  const int l16 = threadIdx.x & 15;
  Place p(w, half);
  while (p.g < w.groups) {
    uint2 q[UNROLL];
    uint32_t s[UNROLL];
    uint4 *dst[UNROLL];
#pragma unroll
    for (int u = 0; u < UNROLL; ++u) {
      const int c = p.col * 16 + l16;
      dst[u] = nullptr;
      if (p.g < w.groups) {
        q[u] = __ldcs(codes + p.g * 16 + l16);
        s[u] = __ldcs(scales + p.g * 4 + (l16 >> 2));
        if (c < vec) dst[u] = x + p.row * ld_vec + c;
      }
      p.step(w);
    }
#pragma unroll
    for (int u = 0; u < UNROLL; ++u) {
      if (!dst[u]) continue;
      const uint32_t s2 = ckpt8_scale2(s[u]);
      __stcs(dst[u], make_uint4(ckpt8_restore2(q[u].x, 0x4140, s2), ckpt8_restore2(q[u].x, 0x4342, s2),
                                ckpt8_restore2(q[u].y, 0x4140, s2), ckpt8_restore2(q[u].y, 0x4342, s2)));
    }
  }
}

}  // namespace prism
