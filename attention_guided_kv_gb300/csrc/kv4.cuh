// The 4-bit cache's number format and addressing (sm_103a).
//
// A row is one token's K or V of one kv head: 128 values in four groups of
// 32.  Each group holds its minimum z (exact in bf16, as the inputs are bf16),
// a scale s = (max - min) / 15 rounded to bf16 (to zero below 2^-100) and 32
// codes n = (x - z) / s, rounded to nearest with ties to even and clamped to
// 0..15; it stands for s * n + z.  Codes are 64 bytes a row (value 2i in the
// low half of byte i), scales and minima 16 bytes ({s, z} per group), so a
// row takes 80 bytes instead of 256.  Groups run along the head dimension and
// not over tokens: a token then carries all it needs, and appending one token
// or evicting any set of tokens never requantises another.
//
// Both roundings are to the exact quotient's nearest, whatever fp32 does in
// between: where an fp32 value sits on a rounding border, the sign of the
// exact remainder (error-free sums, fused multiply-add) decides.
//
// A group with a NaN, an infinity or a magnitude above 2^126 is held as
// {NaN, NaN} with codes 0: what attends to it gets NaN, as from a bf16 cache.
#pragma once

#include "common.cuh"

namespace kvsel {

constexpr int kQ4D = 128;           // head dimension
constexpr int kQ4CodeBytes = 64;    // codes of a row
constexpr int kQ4ScaleBytes = 16;   // {scale, minimum} bf16 x 4 of a row
constexpr uint32_t kQ4NaN2 = 0x7FC07FC0u;

// a + b = sum + err exactly (no overflow)
__device__ __forceinline__ float two_sum(float a, float b, float& err) {
  const float s = __fadd_rn(a, b);
  const float bb = __fsub_rn(s, a);
  err = __fadd_rn(__fsub_rn(a, __fsub_rn(s, bb)), __fsub_rn(b, bb));
  return s;
}

// bf16 bits of (hi_v - lo_v) / 15 rounded to nearest even, 0 below 2^-100.
// The product with 1 / 15 is within 2 units of its last place: only within 4 of
// a border of bf16 can that matter, and there 15 times the border is compared
// with the difference and its rounding error.
__device__ __forceinline__ uint32_t q4_scale_bits(float hi_v, float lo_v) {
  float err;
  const float r = two_sum(hi_v, -lo_v, err);
  const uint32_t u = __float_as_uint(r * (1.0f / 15.0f));
  uint32_t b = (u + 0x7FFFu + ((u >> 16) & 1u)) >> 16;
  if ((u & 0xFFFFu) - 0x7FFCu <= 8u) {
    const uint32_t down = u >> 16;
    const float e = __fadd_rn(__fmaf_rn(-15.0f, __uint_as_float((down << 16) | 0x8000u), r), err);
    b = e > 0.0f || (e == 0.0f && (down & 1u)) ? down + 1u : down;
  }
  return b < (27u << 7) ? 0u : b;       // 2^-100 has exponent field 27
}

// Packed bf16 minimum and maximum (a NaN wins), and the smaller magnitude (of
// either sign).
__device__ __forceinline__ uint32_t bf2_min(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("min.NaN.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
__device__ __forceinline__ uint32_t bf2_max(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
__device__ __forceinline__ uint32_t bf2_min_abs(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("min.xorsign.abs.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
// Two fp32 operations an instruction: (x, y) + c and (x, y) * b + (c, e).
__device__ __forceinline__ void add2(float (&d)[2], float x, float y, float c) {
  asm("{\n\t.reg .b64 a, b;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %4};\n\tadd.rn.f32x2 a, a, b;\n\tmov.b64 {%0, %1}, a;\n\t}"
      : "=f"(d[0]), "=f"(d[1])
      : "f"(x), "f"(y), "f"(c));
}
__device__ __forceinline__ void fma2(float (&d)[2], float x, float y, float b, float c, float e) {
  asm("{\n\t.reg .b64 a, b, c;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %4};\n\tmov.b64 c, {%5, %6};\n\t"
      "fma.rn.f32x2 a, a, b, c;\n\tmov.b64 {%0, %1}, a;\n\t}"
      : "=f"(d[0]), "=f"(d[1])
      : "f"(x), "f"(y), "f"(b), "f"(c), "f"(e));
}
__device__ __forceinline__ uint32_t swap_halves(uint32_t v) { return __funnelshift_l(v, v, 16); }

// The code of x >= z in a group of minimum z and scale s, whatever the
// magnitudes: x - z may need more than 24 bits, so its rounding error decides
// where the quotient looks like a border.
__device__ __forceinline__ float q4_code_any(float x, float z, float s, float inv) {
  float err;
  const float r = two_sum(x, -z, err);
  float n = rintf(r * inv);
  const float d = __fmaf_rn(-n, s, r);
  if (fabsf(d) >= 0.5f * s) {
    const float f = d > 0.0f ? n : n - 1.0f;
    const float e = __fadd_rn(__fsub_rn(r, (f + 0.5f) * s), err);
    const bool up = e > 0.0f || (e == 0.0f && (int(f) & 1));
    n = up ? f + 1.0f : f;
  }
  return n;
}

// One group spread over 32 / NV neighbouring lanes of NV values each (bf16
// pairs in raw): returns this lane's NV codes (4 bits each, value 0 lowest)
// and the group's {s, z} bits.  All lanes of the warp take part.
//
// The usual case (no value below 2^-15 of the largest magnitude) has x - z
// exact in fp32.  r / s is rounded by adding 1.5 * 2^23 to r * inv in one fused
// step, with inv slightly above 1 / s: the result is the right code or one too
// high, a tie always the upper one.  The exact remainder d = r - n s tells: it
// is below -s/2, or equal to it at an odd n, where n is one too high; both in
// one comparison with a threshold that is the next float below -s/2 for even n.
// s is at least (1 - 2^-8) / 15 of the range, so n is at most 15.
template <int NV>
__device__ __forceinline__ uint32_t q4_group(const uint32_t (&raw)[NV / 2], uint32_t& sz) {
  uint32_t lo2 = raw[0], hi2 = raw[0], ab2 = raw[0];
#pragma unroll
  for (int i = 1; i < NV / 2; ++i) {
    lo2 = bf2_min(lo2, raw[i]);
    hi2 = bf2_max(hi2, raw[i]);
    ab2 = bf2_min_abs(ab2, raw[i]);
  }
#pragma unroll
  for (int o = 1; o < 32 / NV; o <<= 1) {
    lo2 = bf2_min(lo2, __shfl_xor_sync(0xffffffffu, lo2, o));
    hi2 = bf2_max(hi2, __shfl_xor_sync(0xffffffffu, hi2, o));
    ab2 = bf2_min_abs(ab2, __shfl_xor_sync(0xffffffffu, ab2, o));
  }
  const float lo = bf16lo_to_f32(bf2_min(lo2, swap_halves(lo2))) + 0.0f;   // -0 -> +0
  const float hi = bf16lo_to_f32(bf2_max(hi2, swap_halves(hi2)));
  const float mag = fmaxf(fabsf(lo), fabsf(hi));
  const float small = fabsf(bf16lo_to_f32(bf2_min_abs(ab2, swap_halves(ab2))));
  if (!(fabsf(lo) <= 0x1p126f && fabsf(hi) <= 0x1p126f)) {   // larger, infinite or NaN
    sz = kQ4NaN2;
    return 0u;
  }
  const uint32_t sb = q4_scale_bits(hi, lo);
  sz = sb | (__float_as_uint(lo) & 0xFFFF0000u);
  if (sb == 0u) return 0u;
  const float s = __uint_as_float(sb << 16);
  const float inv = __fdividef(1.0f, s);
  constexpr float kMagic = 12582912.f;
  float v[NV / 4];   // four codes as one integer below 2^16 in the mantissa of 2^23 + it
#pragma unroll
  for (int q = 0; q < NV / 4; ++q) v[q] = 8388608.f;
  if (small * 32768.f >= mag) {
    const float inv_up = inv * (1.0f + 0x1p-20f);
    const uint32_t thr = __float_as_uint(-0.5f * s);
#pragma unroll
    for (int i = 0; i < NV; i += 2) {
      float r[2], y[2], n[2], d[2];
      add2(r, bf16lo_to_f32(raw[i / 2]), bf16hi_to_f32(raw[i / 2]), -lo);
      fma2(y, r[0], r[1], inv_up, kMagic, kMagic);
      add2(n, y[0], y[1], -kMagic);
      fma2(d, n[0], n[1], -s, r[0], r[1]);
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        if (d[k] <= __uint_as_float(thr | (~__float_as_uint(y[k]) & 1u))) n[k] = __fsub_rn(n[k], 1.0f);
        v[i / 4] = __fmaf_rn(n[k], float(1 << (4 * ((i + k) & 3))), v[i / 4]);
      }
    }
  } else {
#pragma unroll 1
    for (int i = 0; i < NV; ++i) {
      uint32_t w = raw[0];
#pragma unroll
      for (int k = 1; k < NV / 2; ++k) w = i / 2 == k ? raw[k] : w;
      const float n = q4_code_any(i & 1 ? bf16hi_to_f32(w) : bf16lo_to_f32(w), lo, s, inv);
      const float add = n * float(1 << (4 * (i & 3)));
#pragma unroll
      for (int q = 0; q < NV / 4; ++q) v[q] += i / 4 == q ? add : 0.f;
    }
  }
  uint32_t codes = 0;
#pragma unroll
  for (int q = 0; q < NV / 4; ++q) codes |= (__float_as_uint(v[q]) & 0xFFFFu) << (16 * q);
  return codes;
}

}  // namespace kvsel
