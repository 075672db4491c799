// Codes of the 8-bit cache.
//
// A tile is the 16 x 128 codes of one (block, kv head, K or V), e4m3 or int8,
// with one exponent byte e: a code c stands for c * 2^(e - 127), 255 for NaN
// (the e8m0 format).  Powers of two make every scaling exact, so a value that is
// written is rounded once, and a scale that grows moves e4m3 codes without rounding
// them again (but for their subnormals; int8 codes are: below one step of the last
// scale in all).  For int8 an exact amax / 127 would gain
// half a bit on average at the first write; a growing scale would then round
// the block's earlier rows again at every new maximum (about three times in a
// block written token by token) instead of only when the maximum doubles.
#pragma once

#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "pa_internal.h"

namespace pa {

constexpr int kRow8 = kHeadDim;               // bytes of a row of codes
constexpr int kTile8 = kBlock * kRow8;        // of a tile: 2 KiB
constexpr int kPair8 = 2 * kTile8;            // K tile, then V tile of a (block, kv head)
constexpr int kNanExponent = 255;
constexpr int kTasks8 = 4;                    // tiles of a block that a CTA of the cache write has, with one claim
constexpr int claim_groups(int n_kv_heads) { return (2 * n_kv_heads + kTasks8 - 1) / kTasks8; }

// Biased exponent of the smallest power of two 2^x >= 2^-126 whose largest code
// (448 or 127) holds a magnitude, given as its bits; 255 if it is not finite.
template <bool kE4M3>
__device__ __forceinline__ int exponent_for(uint32_t amax_bits) {
  if (amax_bits >= 0x7f800000u) return kNanExponent;
  const int e = static_cast<int>(amax_bits >> 23);
  const uint32_t m = amax_bits & 0x7fffffu;
  // 448 = 1.75 * 2^8, 127 = 1.984375 * 2^6
  const int x = kE4M3 ? e - 8 + (m > 0x600000u) : e - 6 + (m > 0x7e0000u);
  return x < 1 ? 1 : x;
}

// 2^(127 - e), exact; 0 for NaN (no code stands for it).
__device__ __forceinline__ float inverse_scale(int e) {
  return e >= 254 ? (e == 254 ? __int_as_float(0x00400000) : 0.f) : __int_as_float((254 - e) << 23);
}
__device__ __forceinline__ float scale_of(int e) {
  return e == 0 ? __int_as_float(0x00400000) : __int_as_float(e == kNanExponent ? 0x7fffffff : e << 23);
}

// Four scaled values as four codes, to nearest even, the first in the low byte.
template <bool kE4M3>
__device__ __forceinline__ uint32_t pack_codes(float a, float b, float c, float d) {
  if (kE4M3) {
    const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
    const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(c, d), __NV_SATFINITE, __NV_E4M3);
    return lo | hi << 16;
  }
  const uint32_t x = __float2int_rn(a) & 0xff, y = __float2int_rn(b) & 0xff;
  const uint32_t z = __float2int_rn(c) & 0xff, w = __float2int_rn(d) & 0xff;
  return x | y << 8 | z << 16 | w << 24;
}

// Two codes (low and high byte of 16 bits) as two halves; exact.
__device__ __forceinline__ uint32_t e4m3x2_to_half2(uint16_t c) {
  const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(c, __NV_E4M3);
  return *reinterpret_cast<const uint32_t*>(&h);
}
// Four codes as two pairs of halves (bytes 0, 1 and 2, 3).  An int8 code
// with its top bit flipped is c + 128; as the low byte of a half of 1024 it
// makes 1024 + 128 + c, and 1152 is taken off again, all exact.
template <bool kE4M3>
__device__ __forceinline__ void unpack_codes(uint32_t w, uint32_t& p0, uint32_t& p1) {
  if (kE4M3) {
    p0 = e4m3x2_to_half2(static_cast<uint16_t>(w));
    p1 = e4m3x2_to_half2(static_cast<uint16_t>(w >> 16));
    return;
  }
  const uint32_t u = w ^ 0x80808080u;
  const uint32_t x = __byte_perm(u, 0x64646464u, 0x4140), y = __byte_perm(u, 0x64646464u, 0x4342);
  const __half2 off = __half2half2(__ushort_as_half(0x6480));  // 1152
  const __half2 a = __hsub2(*reinterpret_cast<const __half2*>(&x), off);
  const __half2 b = __hsub2(*reinterpret_cast<const __half2*>(&y), off);
  p0 = *reinterpret_cast<const uint32_t*>(&a);
  p1 = *reinterpret_cast<const uint32_t*>(&b);
}
template <bool kE4M3>
__device__ __forceinline__ float4 codes_to_float4(uint32_t w) {
  uint32_t p0, p1;
  unpack_codes<kE4M3>(w, p0, p1);
  const float2 a = __half22float2(*reinterpret_cast<const __half2*>(&p0));
  const float2 b = __half22float2(*reinterpret_cast<const __half2*>(&p1));
  return make_float4(a.x, a.y, b.x, b.y);
}
// Four codes of a scale that grows by 2^d: c * 2^-d to nearest even.
template <bool kE4M3>
__device__ __forceinline__ uint32_t shrink_codes(uint32_t w, float ratio) {
  const float4 f = codes_to_float4<kE4M3>(w);
  return pack_codes<kE4M3>(f.x * ratio, f.y * ratio, f.z * ratio, f.w * ratio);
}

}  // namespace pa
