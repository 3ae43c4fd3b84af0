// The 4-bit cache format (include/ekv.h, ekv_cache_q4) and the device helpers
// that read it.
//
// One record per 16 tokens of a (page, KV head), R = 16·d + 128 bytes:
//   [K codes 16 × d/2][V codes 16 × d/2][K (step, zero) 16 × 2 bf16][V the same]
// Code i of a row sits in half i & 1 (low first) of byte i / 2; it stands for
// zero + step·n.  The records of a page's S/16 tiles, of its KV heads, and of
// the physical pages follow one another.  Everything a decode needs of 16
// tokens is one contiguous block (2176 B at d = 128), so one bulk copy brings it.
#pragma once

#include "kernels.cuh"

namespace ekv {

constexpr int kTile = 16;  // tokens per record, and per step of the decode kernels

__host__ __device__ constexpr int q4_record_bytes(int d) { return 16 * d + 128; }

// fp32 → bf16 toward +inf (up) or −inf, from the encodings: dropping the low
// half moves a number toward zero; adding 0xffff to the bits first moves it away.
__device__ __forceinline__ bf16 bf16_away(float x, bool up) {
  uint32_t b = __float_as_uint(x);
  if ((b >> 31 == 0u) == up && (b & 0x7f800000u) != 0x7f800000u) b += 0xffffu;
  return __ushort_as_bfloat16(static_cast<unsigned short>(b >> 16));
}

__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

// The value a code stands for: zero + step·n, rounded once to fp32.
__device__ __forceinline__ float q4_value(uint32_t step_zero, uint32_t n) {
  return fmaf(bf16_lo(step_zero), static_cast<float>(n), bf16_hi(step_zero));
}

}  // namespace ekv
