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

__device__ __forceinline__ uint32_t pack_bytes(uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  return __byte_perm(__byte_perm(a, b, 0x0040), __byte_perm(c, d, 0x0040), 0x5410);
}

// Both values rounded to 24 - BITS significant bits (Veltkamp's splitting: hi = g + (y - g),
// g = (2^BITS + 1) y).
template <int BITS>
__device__ __forceinline__ sm100::F2 snap2(sm100::F2 y) {
  using namespace sm100;
  const float c = static_cast<float>((1 << BITS) + 1);
  const F2 g = mul2(y, pack2(c, c));
  return add2(g, fma2(g, pack2(-1.f, -1.f), y));
}

// F / r for encode8, r of 8 significant bits.
template <int FMT>
__device__ __forceinline__ float code_factor(float r) {
  return FMT == TM_KV_INT8 ? __fdiv_ru(full<FMT>(), r) : __fdiv_rn(full<FMT>(), r);
}

// The codes of 8 bf16 values: x[e] * f to the nearest code, two values an instruction.
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
      unpack2(snap2<7>(mul2(v, ff)), a, b);
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
  using namespace sm100;
  const F2 rr = pack2(ratio, ratio);
  float a, b, c, d;
  if (FMT == TM_KV_INT8) {
    // 2^23 + code + 128 by its bits, so that one addition gives the code as a float
    const uint32_t u = w ^ 0x80808080u;
    const F2 bias = pack2(-8388736.f, -8388736.f), round = pack2(12582912.f, 12582912.f);
    F2 x = add2(pack2(__byte_perm(u, 0x4B000000u, 0x7440), __byte_perm(u, 0x4B000000u, 0x7441)), bias);
    F2 y = add2(pack2(__byte_perm(u, 0x4B000000u, 0x7442), __byte_perm(u, 0x4B000000u, 0x7443)), bias);
    unpack2(add2(snap2<4>(mul2(x, rr)), round), a, b);
    unpack2(add2(snap2<4>(mul2(y, rr)), round), c, d);
    return pack_bytes(__float_as_uint(a), __float_as_uint(b), __float_as_uint(c), __float_as_uint(d));
  }
  const float2 x = __half22float2(
      __half2(__nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(w), __NV_E4M3)));
  const float2 y = __half22float2(
      __half2(__nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(w >> 16), __NV_E4M3)));
  unpack2(snap2<7>(mul2(pack2(x.x, x.y), rr)), a, b);
  unpack2(snap2<7>(mul2(pack2(y.x, y.y), rr)), c, d);
  return __byte_perm(__nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3),
                     __nv_cvt_float2_to_fp8x2(make_float2(c, d), __NV_SATFINITE, __NV_E4M3), 0x5410);
}

__device__ __forceinline__ bool finite(float r) {
  return (__float_as_uint(r) & 0x7F800000u) != 0x7F800000u;
}

__device__ __forceinline__ uint32_t warp_max(uint32_t v) { return __reduce_max_sync(0xffffffffu, v); }

}  // namespace kv8
}  // namespace trimix
