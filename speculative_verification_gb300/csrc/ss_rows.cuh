// ss_rows.cuh -- rows of the paged cache, 16 lanes of 8 channels each: bf16 to
// 4 or 8 bits and back.
#pragma once
#include <stdint.h>

#include "ss_cache.h"

namespace ssc {
using namespace ss;

constexpr int kRowLanes = 16;           // a row is at most 16 lanes of 8 channels
constexpr uint32_t kNaN2 = 0x7fc07fc0u;  // a bf16 pair of NaNs

__device__ __forceinline__ uint32_t min2(uint32_t a, uint32_t b) {  // bf16 pairs; a NaN stays
  uint32_t r;
  asm("min.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ uint32_t max2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

// Eight channels of a row, quantised: the row's low value and step come from
// the 16 lanes of the row, as the pair (min x, min -x), so that one shuffle and
// one instruction join two lanes.
//
// round((x - m) / s) without a division per channel: with y = x - m and
// q = y * (1 / s), the remainder y - q s is exact in fp32 (q is off by a few
// units at most and s has 8 bits), and q + (y - q s) / s is the quotient to
// within 2^-20 of its last place before the one rounding.  A quotient that is
// no half differs from every half by more than 1.003 times half a unit (y has
// 24 bits, s has 8), so it is not rounded onto one: adding 1.5 * 2^23 then
// leaves the integer, ties to even, in the low bits.
__device__ __forceinline__ uint32_t quantise8(const uint4 x, bool live, uint32_t lanes, uint32_t& pair) {
  uint32_t w[4] = {x.x, x.y, x.z, x.w};
  const uint32_t mn = min2(min2(w[0], w[1]), min2(w[2], w[3]));
  const uint32_t mx = max2(max2(w[0], w[1]), max2(w[2], w[3])) ^ 0x80008000u;
  uint32_t both = min2(__byte_perm(mn, mx, 0x5410), __byte_perm(mn, mx, 0x7632));
  if (!live) both = 0x7f807f80u;
#pragma unroll
  for (int o = kRowLanes / 2; o > 0; o >>= 1) both = min2(both, __shfl_xor_sync(lanes, both, o, kRowLanes));
  float lo = bf16_lo(both);
  const float range = __fsub_rn(-bf16_hi(both), lo);
  if (!(range < __int_as_float(0x7f800000))) {  // a NaN, an infinity or too wide
    pair = kNaN2;
    return 0;
  }
  // the smallest bf16 that is not below range / 15: then 15 steps reach the
  // highest channel (the division as above)
  constexpr float kTiny = 1.0e-28f, kUp = 18446744073709551616.0f;
  float step = range * (1.0f / 15.0f);
  step = __fmaf_rn(__fmaf_rn(-step, 15.0f, range), 1.0f / 15.0f, step);
  if (range < kTiny) step = __fdiv_rn(range, 15.0f);
  step = __uint_as_float((__float_as_uint(step) + 0xffffu) & 0xffff0000u);
  pair = (__float_as_uint(step) >> 16) | __float_as_uint(lo);  // lo is one of the row's bf16
  if (step == 0.0f) return 0;
  if (range < kTiny) {  // keep 1 / step and the remainders in the normal range: all of it times 2^64
#pragma unroll
    for (int i = 0; i < 4; ++i) asm("mul.rn.bf16x2 %0, %0, %1;" : "+r"(w[i]) : "r"(0x5f805f80u));
    lo *= kUp;
    step *= kUp;
  }
  const float inv = __fdividef(1.0f, step);
  const uint64_t low2 = two(-lo, -lo), inv2 = two(inv, inv), step2 = two(-step, -step);
  constexpr uint32_t kRound = 0x4b400000u;  // 1.5 * 2^23
  uint32_t out = 0u - 0x11111111u * kRound;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint64_t y = add_2(two(bf16_lo(w[i]), bf16_hi(w[i])), low2), q = mul_2(y, inv2);
    const uint64_t t = add_2(fma_2(fma_2(q, step2, y), inv2, q), two(__uint_as_float(kRound), __uint_as_float(kRound)));
    out += (static_cast<uint32_t>(t) << (4 * i)) + (static_cast<uint32_t>(t >> 32) << (16 + 4 * i));
  }
  return out;
}

__device__ __forceinline__ uint4 dequantise8(uint32_t w, uint32_t pair) {
  const float s = bf16_lo(pair), m = bf16_hi(pair);
  const uint64_t s2 = two(s, s), m2 = two(m, m), off = two(-8388608.0f, -8388608.0f);
  uint32_t o[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {  // 2^23 + n, minus 2^23: no conversion
    const uint64_t n = add_2(two(__uint_as_float(((w >> (4 * i)) & 15u) | 0x4b000000u),
                                 __uint_as_float(((w >> (16 + 4 * i)) & 15u) | 0x4b000000u)), off);
    const uint64_t v = fma_2(n, s2, m2);
    float a, b;
    split(v, a, b);
    o[i] = bf16_pair(a, b);
  }
  return make_uint4(o[0], o[1], o[2], o[3]);
}

// ----------------------------------------------------------------- 8 bits --
// A block's scale is the smallest power of two 2^e, e >= -100, with 448 2^e no
// less than the block's largest magnitude: e4m3 is a floating-point format, so a
// scale only has to keep the range, and a power of two does it without a
// rounding of its own; rows written again under another scale lose bits only
// where they fall below 2^-6 of it.
struct Scale8 {
  float s, inv;
};
__device__ __forceinline__ Scale8 scale8(float top) {
  // 448 = 1.75 * 2^8: a mantissa above 1.75 carries into the exponent
  const int e = max(static_cast<int>((__float_as_uint(top) + 0x1fffffu) >> 23) - 8, 27);
  return {__int_as_float(e << 23), __int_as_float((254 - e) << 23)};
}

// x where it is finite, else NaN (x - x is 0 or NaN; a zero keeps its sign).
__device__ __forceinline__ float finite_or_nan(float x) { return __fsub_rn(x, __fsub_rn(x, x)); }

// The largest of |x| over the finite ones.
__device__ __forceinline__ float finite_top(const float (&x)[8]) {
  float top = 0.0f;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float m = fabsf(x[i]);
    top = fmaxf(top, m < __int_as_float(0x7f800000) ? m : 0.0f);
  }
  return top;
}

// Eight values over a scale, in channel order (what is not finite: NaN).
__device__ __forceinline__ uint2 encode8(const float (&x)[8], float inv) {
  uint32_t w[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    uint16_t lo, hi;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;"
        : "=h"(lo)
        : "f"(finite_or_nan(x[4 * h + 1]) * inv), "f"(finite_or_nan(x[4 * h]) * inv));
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;"
        : "=h"(hi)
        : "f"(finite_or_nan(x[4 * h + 3]) * inv), "f"(finite_or_nan(x[4 * h + 2]) * inv));
    w[h] = static_cast<uint32_t>(hi) << 16 | lo;
  }
  return make_uint2(w[0], w[1]);
}

__device__ __forceinline__ void decode8(uint2 w, float s, float (&x)[8]) {
  const uint32_t v[2] = {w.x, w.y};
#pragma unroll
  for (int h = 0; h < 4; ++h) {
    uint32_t f;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(f) : "h"(static_cast<uint16_t>(v[h >> 1] >> (16 * (h & 1)))));
    asm("{\n\t.reg .f16 l, u;\n\tmov.b32 {l, u}, %2;\n\tcvt.f32.f16 %0, l;\n\tcvt.f32.f16 %1, u;\n\t}"
        : "=f"(x[2 * h]), "=f"(x[2 * h + 1])
        : "r"(f));
    split(mul_2(two(x[2 * h], x[2 * h + 1]), two(s, s)), x[2 * h], x[2 * h + 1]);
  }
}

// What eight bytes stand for, in bf16, rounded once.  By a power of two the product
// is exact in fp32; by another scale it has up to 28 bits and is rounded to odd (toward
// zero, the last bit set where something is left), so that the rounding to bf16
// knows on which side of a tie it lay.
__device__ __forceinline__ uint4 read8(uint2 w, float s) {
  float f[8];
  if ((__float_as_uint(s) & 0x7fffffu) == 0) {
    decode8(w, s, f);
  } else {
    decode8(w, 1.0f, f);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const uint32_t down = __float_as_uint(__fmul_rd(f[i], s)), up = __float_as_uint(__fmul_ru(f[i], s));
      f[i] = __uint_as_float(min(down, up) | static_cast<uint32_t>(down != up));
    }
  }
  return make_uint4(bf16_pair(f[0], f[1]), bf16_pair(f[2], f[3]), bf16_pair(f[4], f[5]), bf16_pair(f[6], f[7]));
}

// The largest magnitude of eight bf16 values, as bits (0x7f80 and up: one is not
// finite): magnitudes compare as integers, in pairs.
__device__ __forceinline__ uint32_t magnitude(const uint4& x) {
  const uint32_t m = __vmaxu2(__vmaxu2(x.x & 0x7fff7fffu, x.y & 0x7fff7fffu), __vmaxu2(x.z & 0x7fff7fffu, x.w & 0x7fff7fffu));
  return max(m & 0xffffu, m >> 16);
}

__device__ __forceinline__ void floats_of(const uint4& w, float (&x)[8]) {
  const uint32_t v[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = bf16_lo(v[i]);
    x[2 * i + 1] = bf16_hi(v[i]);
  }
}

// Finite bf16 values.
__device__ __forceinline__ uint2 encode8(const uint4& x, float inv) {
  const uint32_t w[4] = {x.x, x.y, x.z, x.w};
  const uint64_t inv2 = two(inv, inv);
  uint32_t o[2] = {0u, 0u};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float a, b;
    split(mul_2(two(bf16_lo(w[i]), bf16_hi(w[i])), inv2), a, b);
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(b), "f"(a));
    o[i >> 1] |= static_cast<uint32_t>(r) << (16 * (i & 1));
  }
  return make_uint2(o[0], o[1]);
}

}  // namespace ssc
