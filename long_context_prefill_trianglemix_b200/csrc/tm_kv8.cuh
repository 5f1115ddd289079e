// Device helpers of the 8-bit cache: codes, their conversion and rounding.
//
// A code c of a block with range r stands for c * r / F, F = 127 (int8) or 448
// (e4m3). Rounding is defined on the real quotient (nearest, ties to even), and
// the kernels reach it without a division per element:
//   - x and r are bf16 (8 significant bits), so F x / r is a ratio of small
//     integers. Against a rounding border (an odd multiple of half a step, at
//     most 8 significant bits for int8 and 5 for e4m3) it is either exactly on
//     it or at least 2^-16 (int8) or 2^-13 (e4m3) away, relative to it, while
//     x * fl(F / r) is within 2^-22. Dropping the product's last bits (snap)
//     therefore puts every tie back on its border and moves nothing across one.
//   - For int8 the only such ties are x = r / 2 (63.5, to the even 64) and those of
//     r = 254 * 2^e, where F / r is exact: rounding F / r upwards settles both, and
//     one FMA with 1.5 * 2^23 multiplies and rounds.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include <cstdint>

#include "tm.h"
#include "tm_sm100.cuh"

namespace trimix {
namespace kv8 {

template <int FMT>
__device__ constexpr float full() { return FMT == TM_KV_INT8 ? 127.f : 448.f; }

// y with its significand rounded to 24 - BITS bits.
template <int BITS>
__device__ __forceinline__ float snap(float y) {
  const uint32_t u = __float_as_uint(y);
  return __uint_as_float((u + (1u << (BITS - 1))) & ~((1u << BITS) - 1u));
}

// The int8 code (in the low byte) nearest to y, |y| < 2^22: adding 1.5 * 2^23
// rounds to an integer, ties to even, and leaves it in the low bits.
__device__ __forceinline__ uint32_t round_low(float y) {
  return __float_as_uint(y + 12582912.f);
}

__device__ __forceinline__ uint32_t pack_bytes(uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  return __byte_perm(__byte_perm(a, b, 0x0040), __byte_perm(c, d, 0x0040), 0x5410);
}

__device__ __forceinline__ uint32_t pack_e4m3(float a, float b, float c, float d) {
  const uint32_t l = __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
  const uint32_t h = __nv_cvt_float2_to_fp8x2(make_float2(c, d), __NV_SATFINITE, __NV_E4M3);
  return l | (h << 16);
}

// Four codes of the quotients y (already within 2^-22 of the real ones).
template <int FMT>
__device__ __forceinline__ uint32_t encode4(float a, float b, float c, float d) {
  if (FMT == TM_KV_INT8)
    return pack_bytes(round_low(snap<4>(a)), round_low(snap<4>(b)), round_low(snap<4>(c)),
                      round_low(snap<4>(d)));
  return pack_e4m3(snap<7>(a), snap<7>(b), snap<7>(c), snap<7>(d));
}

// Four codes as floats.
template <int FMT>
__device__ __forceinline__ void decode4(uint32_t w, float (&f)[4]) {
  if (FMT == TM_KV_INT8) {
#pragma unroll
    for (int e = 0; e < 4; ++e) f[e] = static_cast<float>(static_cast<int8_t>(w >> (8 * e)));
  } else {
    const __half2 l(__nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(w), __NV_E4M3));
    const __half2 h(
        __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(w >> 16), __NV_E4M3));
    f[0] = __low2float(l); f[1] = __high2float(l);
    f[2] = __low2float(h); f[3] = __high2float(h);
  }
}

// F / r for encode8, r of 8 significant bits.
template <int FMT>
__device__ __forceinline__ float code_factor(float r) {
  return FMT == TM_KV_INT8 ? __fdiv_ru(full<FMT>(), r) : __fdiv_rn(full<FMT>(), r);
}

// The codes of 8 bf16 values: x[e] * f to the nearest code, two values an instruction.
// e4m3 snaps the product to 17 bits by Veltkamp's splitting (hi = g + (y - g), g = 129 y).
// TINY: x is scaled by 2^64 first (f is that of the range scaled alike).
template <int FMT, bool TINY>
__device__ __forceinline__ uint2 encode8(const uint4& x, float f) {
  using namespace sm100;
  const uint32_t w[4] = {x.x, x.y, x.z, x.w};
  const F2 ff = pack2(f, f);
  uint32_t c[8];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    F2 v = pack2(w[e] << 16, w[e] & 0xFFFF0000u);
    if (TINY) v = mul2(v, pack2(18446744073709551616.f, 18446744073709551616.f));
    float a, b;
    if (FMT == TM_KV_INT8) {
      unpack2(fma2(v, ff, pack2(12582912.f, 12582912.f)), a, b);
      c[2 * e] = __float_as_uint(a);
      c[2 * e + 1] = __float_as_uint(b);
    } else {
      const F2 y = mul2(v, ff);
      const F2 g = mul2(y, pack2(129.f, 129.f));
      unpack2(add2(g, fma2(g, pack2(-1.f, -1.f), y)), a, b);
      c[e] = __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
    }
  }
  if (FMT == TM_KV_INT8)
    return make_uint2(pack_bytes(c[0], c[1], c[2], c[3]), pack_bytes(c[4], c[5], c[6], c[7]));
  return make_uint2(__byte_perm(c[0], c[1], 0x5410), __byte_perm(c[2], c[3], 0x5410));
}

// Codes of a block of range r0 in the same block at range r >= r0: rne(c r0 / r),
// ratio = r0 / r.
template <int FMT>
__device__ __forceinline__ uint32_t rescale4(uint32_t w, float ratio) {
  float f[4];
  decode4<FMT>(w, f);
  return encode4<FMT>(f[0] * ratio, f[1] * ratio, f[2] * ratio, f[3] * ratio);
}

__device__ __forceinline__ bool finite(float r) {
  return (__float_as_uint(r) & 0x7F800000u) != 0x7F800000u;
}

__device__ __forceinline__ uint32_t warp_max(uint32_t v) { return __reduce_max_sync(0xffffffffu, v); }

}  // namespace kv8
}  // namespace trimix
