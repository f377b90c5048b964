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
__device__ __forceinline__ uint32_t q4_scale_bits(float hi_v, float lo_v) {
  float err;
  const float r = two_sum(hi_v, -lo_v, err);
  const float q = __fdiv_rn(r, 15.0f);
  const float rem = __fadd_rn(__fmaf_rn(-q, 15.0f, r), err);
  uint32_t u = __float_as_uint(q);
  if ((u & 0xFFFFu) == 0x8000u && rem != 0.0f) {
    u = rem > 0.0f ? u + 1u : u - 1u;   // off the border, to the side of the exact quotient
  }
  u = (u + 0x7FFFu + ((u >> 16) & 1u)) >> 16;
  return u < (27u << 7) ? 0u : u;       // 2^-100 has exponent field 27
}

// The code of x >= z in a group of minimum z and scale s > 0 (inv ~ 1 / s), as
// a float.  Adding 1.5 * 2^23 rounds to an integer, ties to even.  No clamp:
// s is at least (1 - 2^-8) / 15 of the range, so the quotient is below 15.1.
__device__ __forceinline__ float q4_code(float x, float z, float s, float half_s, float inv) {
  constexpr float kMagic = 12582912.f;
  const float r = __fsub_rn(x, z);
  float n = __fsub_rn(__fmaf_rn(r, inv, kMagic), kMagic);
  const float d = __fmaf_rn(-n, s, r);
  if (fabsf(d) >= half_s) {             // on or past a border: settle it exactly
    float err;
    const float rr = two_sum(x, -z, err);
    const float f = d > 0.0f ? n : n - 1.0f;
    const float e = __fadd_rn(__fsub_rn(rr, (f + 0.5f) * s), err);
    const bool up = e > 0.0f || (e == 0.0f && (int(f) & 1));
    n = up ? f + 1.0f : f;
  }
  return n;
}

// One group spread over 32 / NV neighbouring lanes of NV values each (bf16
// pairs in raw): returns this lane's NV codes (4 bits each, value 0 lowest)
// and the group's {s, z} bits.  All the group's lanes take part.
template <int NV>
__device__ __forceinline__ uint32_t q4_group(const uint32_t (&raw)[NV / 2], uint32_t& sz) {
  float x[NV];
  uint32_t mag = 0;
#pragma unroll
  for (int i = 0; i < NV / 2; ++i) {
    x[2 * i] = bf16lo_to_f32(raw[i]);
    x[2 * i + 1] = bf16hi_to_f32(raw[i]);
    mag = max(mag, max((raw[i] << 16) & 0x7FFF0000u, raw[i] & 0x7FFF0000u));
  }
  float lo = x[0], hi = x[0];
#pragma unroll
  for (int i = 1; i < NV; ++i) {
    lo = fminf(lo, x[i]);
    hi = fmaxf(hi, x[i]);
  }
#pragma unroll
  for (int o = 1; o < 32 / NV; o <<= 1) {
    lo = fminf(lo, __shfl_xor_sync(0xffffffffu, lo, o));
    hi = fmaxf(hi, __shfl_xor_sync(0xffffffffu, hi, o));
    mag = max(mag, __shfl_xor_sync(0xffffffffu, mag, o));
  }
  if (mag > 0x7E800000u) {              // above 2^126, infinite or NaN
    sz = kQ4NaN2;
    return 0u;
  }
  lo += 0.0f;                           // -0 -> +0
  const uint32_t sb = q4_scale_bits(hi, lo);
  sz = sb | (__float_as_uint(lo) & 0xFFFF0000u);
  if (sb == 0u) return 0u;
  const float s = __uint_as_float(sb << 16);
  const float inv = __fdividef(1.0f, s), half_s = 0.5f * s;
  // four codes at a time as one integer below 2^16 in a float's mantissa
  uint32_t codes = 0;
#pragma unroll
  for (int q = 0; q < NV / 4; ++q) {
    float v = 8388608.f;
#pragma unroll
    for (int i = 0; i < 4; ++i) v = __fmaf_rn(q4_code(x[4 * q + i], lo, s, half_s, inv), float(1 << (4 * i)), v);
    codes |= (__float_as_uint(v) & 0xFFFFu) << (16 * q);
  }
  return codes;
}

}  // namespace kvsel
