// The 8-bit formats of the key/value cache: codes to and from fp32.
#pragma once

#include <cstdint>

#include "qg_common.cuh"

namespace qg {

template <int FMT>
__host__ __device__ constexpr float kv8_qmax() {
  return FMT == QG_KV_I8 ? 127.f : 448.f;
}

// two fp32 rounded to nearest even, as a bf16 pair (lo in the low half)
__device__ __forceinline__ uint32_t f32_to_bf16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// two e4m3 codes (low byte first) -> f16x2, exact
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint16_t c) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(c));
  return r;
}

// four codes of one word -> fp32
template <int FMT>
__device__ __forceinline__ void kv8_decode4(uint32_t w, float& a, float& b, float& c, float& d) {
  if (FMT == QG_KV_I8) {
    a = (float)(int8_t)(w & 0xFFu);
    b = (float)(int8_t)(w >> 8 & 0xFFu);
    c = (float)(int8_t)(w >> 16 & 0xFFu);
    d = (float)(int8_t)(w >> 24);
  } else {
    const uint32_t lo = e4m3x2_to_f16x2((uint16_t)w), hi = e4m3x2_to_f16x2((uint16_t)(w >> 16));
    a = f16_bits_to_f32((uint16_t)lo), b = f16_bits_to_f32((uint16_t)(lo >> 16));
    c = f16_bits_to_f32((uint16_t)hi), d = f16_bits_to_f32((uint16_t)(hi >> 16));
  }
}

// 1.5 * 2^23: added to |v| < 2^22 it leaves v rounded to the nearest integer (ties to even) in the low bits
constexpr float kRoundInt = 12582912.f;

// four fp32 to the nearest codes (ties to even), first in the low byte; int8: |v| < 127.5, e4m3 is clamped to +-448
template <int FMT>
__device__ __forceinline__ uint32_t kv8_encode4(float a, float b, float c, float d) {
  if (FMT == QG_KV_I8) {
    const uint32_t lo = __byte_perm(__float_as_uint(a + kRoundInt), __float_as_uint(b + kRoundInt), 0x0040),
                   hi = __byte_perm(__float_as_uint(c + kRoundInt), __float_as_uint(d + kRoundInt), 0x0040);
    return __byte_perm(lo, hi, 0x5410);
  }
  uint16_t lo, hi;  // saturates at +-448
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(b), "f"(a));
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(d), "f"(c));
  return (uint32_t)lo | (uint32_t)hi << 16;
}

// Codes of eight values over s > 0: the IEEE quotient v / s to the nearest code,
// made without a division (8 instructions and a branch) wherever the code does
// not depend on the quotient's last bits: v times 1 / s is at most 2 ulp off it.
// int8: only where that product lies within 1e-4 of a border between two codes
// are the divisions made; e4m3: only where v times the reciprocals 2^-21 to
// either side of 1 / s gives two different codes (about 1 in 5000 values each).
// A quotient passes +-127 by a few ulp only, as s is the largest value / 127
// rounded, except where s is subnormal: the divided ones are clamped.
template <int FMT>
__device__ __forceinline__ uint2 kv8_quantize8(const float (&v)[8], float s, float inv) {
  bool close = !(s > 1e-30f);
  uint2 codes;
  float q[8];
  if (FMT == QG_KV_I8) {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      q[j] = v[j] * inv;
      close |= !(fabsf(q[j] - ((q[j] + kRoundInt) - kRoundInt)) < 0.4999f);
    }
    codes = make_uint2(kv8_encode4<FMT>(q[0], q[1], q[2], q[3]), kv8_encode4<FMT>(q[4], q[5], q[6], q[7]));
  } else {
    const float lo = inv * (1.f - 0x1p-21f), hi = inv * (1.f + 0x1p-21f);
    codes = make_uint2(kv8_encode4<FMT>(v[0] * lo, v[1] * lo, v[2] * lo, v[3] * lo),
                       kv8_encode4<FMT>(v[4] * lo, v[5] * lo, v[6] * lo, v[7] * lo));
    close |= codes.x != kv8_encode4<FMT>(v[0] * hi, v[1] * hi, v[2] * hi, v[3] * hi) ||
             codes.y != kv8_encode4<FMT>(v[4] * hi, v[5] * hi, v[6] * hi, v[7] * hi);
  }
  if (close) {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      q[j] = __fdiv_rn(v[j], s);
      if (FMT == QG_KV_I8) q[j] = fminf(fmaxf(q[j], -127.f), 127.f);
    }
    codes = make_uint2(kv8_encode4<FMT>(q[0], q[1], q[2], q[3]), kv8_encode4<FMT>(q[4], q[5], q[6], q[7]));
  }
  return codes;
}

}  // namespace qg
