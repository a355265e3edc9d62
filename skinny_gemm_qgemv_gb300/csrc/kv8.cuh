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

// four fp32 to the nearest codes (ties to even, clamped to +-qmax), first in the low byte
template <int FMT>
__device__ __forceinline__ uint32_t kv8_encode4(float a, float b, float c, float d) {
  if (FMT == QG_KV_I8) {
    auto q = [](float v) { return (uint32_t)(int)fminf(fmaxf(rintf(v), -127.f), 127.f) & 0xFFu; };
    return q(a) | q(b) << 8 | q(c) << 16 | q(d) << 24;
  }
  uint16_t lo, hi;  // saturates at +-448
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(b), "f"(a));
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(d), "f"(c));
  return (uint32_t)lo | (uint32_t)hi << 16;
}

}  // namespace qg
