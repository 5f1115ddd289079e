// Rotary positions: rotate the first `rot` columns of every q and k head by the
// angles pos * inv_freq[i], i < rot / 2, out of place or in place.
//
//   y_a = m (x_a cos t - x_b sin t),  y_b = m (x_b cos t + x_a sin t)
//
// with the pair (a, b) = (i, i + rot/2) (half layout) or (2i, 2i + 1)
// (interleaved) and t = pos * inv_freq[i]. Far positions make t large (10^5 to
// 10^6 radians), where fp32 has no digits left for the fraction of a turn, so
// pos * inv_freq / (2 pi) is formed and reduced to [-1/2, 1/2] turns in fp64 and only
// the remainder goes to fp32. For positions of 32 bits one double is enough (three
// roundings of 2^-53 of 2^28.4 turns, and fp32's: an error below 2^-23 of a turn). A
// call whose `first` lies beyond takes kernels that carry what the products' roundings
// dropped in a second double: the same bound up to 2^52, where one double would be 1/8
// of a turn off. Carried always, it costs 2 x 4173 rows of half-turned heads 17.0 us
// instead of 16.05; behind a branch on the position, 17.3.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "tm.h"
#include "tm_internal.h"
#include "tm_launch.cuh"

namespace trimix {
namespace {

struct RopeParams {
  const uint16_t* q;
  uint16_t* q_out;
  const uint16_t* k;
  uint16_t* k_out;
  long long rows;
  int N, Hq, Hkv, D, rot;
  long long q_stride, q_out_stride, k_stride, k_out_stride;
  int interleaved, heads_per_slice, copy_q, copy_k;
  float sign, mscale;
  const double* inv_freq;
  const int* positions;
  long long first;
};

template <bool FAR>
__device__ __forceinline__ void angle(const RopeParams& p, double pos, int i, float& c, float& s) {
  constexpr double kInv = 0.15915494309189533577, kInvLow = -9.839338337591243e-18;  // 1 / (2 pi)
  const double f = p.inv_freq[i], t = pos * f, turns = t * kInv;
  double rest = turns - rint(turns);
  if (FAR) rest += fma(t, kInv, -turns) + fma(t, kInvLow, fma(pos, f, -t) * kInv);
  const float half_turns = static_cast<float>(2.0 * rest);
  sincospif(half_turns, &s, &c);
  c *= p.mscale;
  s *= p.mscale * p.sign;
}

__device__ __forceinline__ double position(const RopeParams& p, long long row) {
  if (p.positions) return static_cast<double>(p.positions[row]);
  return static_cast<double>(p.first + row % p.N);
}

__device__ __forceinline__ float lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }
__device__ __forceinline__ uint32_t pack(float a, float b) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// Rotates 16 columns of one head held as two 16-byte words: in the half layout
// u holds the 8 first elements of the pairs and v the 8 second ones, interleaved
// u and v hold pairs 0..3 and 4..7.
__device__ __forceinline__ void turn16(uint4& u, uint4& v, const float (&c)[8], const float (&s)[8],
                                       bool interleaved) {
  uint32_t* a = reinterpret_cast<uint32_t*>(&u);
  uint32_t* b = reinterpret_cast<uint32_t*>(&v);
  if (interleaved) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float x = lo(a[e]), y = hi(a[e]), z = lo(b[e]), w = hi(b[e]);
      a[e] = pack(x * c[e] - y * s[e], y * c[e] + x * s[e]);
      b[e] = pack(z * c[e + 4] - w * s[e + 4], w * c[e + 4] + z * s[e + 4]);
    }
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float x0 = lo(a[e]), x1 = hi(a[e]), y0 = lo(b[e]), y1 = hi(b[e]);
      a[e] = pack(x0 * c[2 * e] - y0 * s[2 * e], x1 * c[2 * e + 1] - y1 * s[2 * e + 1]);
      b[e] = pack(y0 * c[2 * e] + x0 * s[2 * e], y1 * c[2 * e + 1] + x1 * s[2 * e + 1]);
    }
  }
}

// One thread per (token, 16 columns, slice of heads): the 8 angles are computed
// once and kept in registers while the thread walks its heads, so their fp64
// work is shared by up to Hq + Hkv heads. D / 16 neighbouring threads cover a
// head's row: 128-byte runs of loads and stores. rot is a multiple of 16. Memory
// bounds it: 131072 tokens of 32 + 8 heads of 128 take 411 us (6.53 TB/s).
template <bool FAR>
__global__ void __launch_bounds__(256) rope_kernel(const RopeParams p) {
  pdl_launch();
  pdl_wait();
  const int per = p.D >> 4;
  const long long gid = static_cast<long long>(blockIdx.x) * 256 + threadIdx.x;
  const long long row = gid / per;
  if (row >= p.rows) return;
  const int c0 = static_cast<int>(gid - row * per);
  const bool turns = c0 * 16 < p.rot;
  float c[8], s[8];
  int ua, ub;  // the thread's two 8-column runs
  if (turns && !p.interleaved) {
    ua = c0 * 8;
    ub = p.rot / 2 + c0 * 8;
  } else {
    ua = c0 * 16;
    ub = ua + 8;
  }
  const int h0 = blockIdx.y * p.heads_per_slice;
  const int h1 = min(h0 + p.heads_per_slice, p.Hq + p.Hkv);
  constexpr int kBatch = 4;  // heads whose loads are in flight together, the first batch's behind the angles
  for (int hb = h0; hb < h1; hb += kBatch) {
    uint4 u[kBatch], v[kBatch];
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      const int h = min(hb + k, h1 - 1);
      const uint16_t* src = h < p.Hq ? p.q + row * p.q_stride + static_cast<long long>(h) * p.D
                                     : p.k + row * p.k_stride + static_cast<long long>(h - p.Hq) * p.D;
      u[k] = *reinterpret_cast<const uint4*>(src + ua);
      v[k] = *reinterpret_cast<const uint4*>(src + ub);
    }
    if (hb == h0 && turns) {
      const double pos = position(p, row);
#pragma unroll
      for (int e = 0; e < 8; ++e) angle<FAR>(p, pos, c0 * 8 + e, c[e], s[e]);
    }
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      const int h = hb + k;
      if (h >= h1) break;
      const bool is_q = h < p.Hq;
      if (!turns && !(is_q ? p.copy_q : p.copy_k)) continue;
      uint16_t* dst = is_q ? p.q_out + row * p.q_out_stride + static_cast<long long>(h) * p.D
                           : p.k_out + row * p.k_out_stride + static_cast<long long>(h - p.Hq) * p.D;
      if (turns) turn16(u[k], v[k], c, s, p.interleaved);
      *reinterpret_cast<uint4*>(dst + ua) = u[k];
      *reinterpret_cast<uint4*>(dst + ub) = v[k];
    }
  }
}

// Threads of a token: its rot / 2 pairs, then single columns in twos up to a multiple
// of 8, then 8 columns each.
__host__ __device__ inline int any_slots(int rot, int D) {
  const int r8 = (rot + 7) / 8 * 8;
  return r8 / 2 + (D - r8) / 8;
}

// Any even rot: one thread per (token, pair or copied columns, slice of heads). The
// 2-byte loads and stores of the turned columns bound it: 2 x 4173 tokens of 28 + 4
// heads of 64 take 22, 27 and 36 us at rot 6, 24 and 40, rope_kernel 14 to 16 at 32.
template <bool FAR>
__global__ void __launch_bounds__(256) rope_any_kernel(const RopeParams p) {
  pdl_launch();
  pdl_wait();
  const int per = any_slots(p.rot, p.D), r8 = (p.rot + 7) / 8 * 8;
  const long long gid = static_cast<long long>(blockIdx.x) * 256 + threadIdx.x;
  const long long row = gid / per;
  if (row >= p.rows) return;
  const int i = static_cast<int>(gid - row * per);
  const bool turns = 2 * i < p.rot, wide = 2 * i >= r8;
  float c = 1.f, s = 0.f;
  if (turns) angle<FAR>(p, position(p, row), i, c, s);
  const int ua = turns && !p.interleaved ? i : wide ? r8 + 8 * (i - r8 / 2) : 2 * i;
  const int ub = turns && !p.interleaved ? i + p.rot / 2 : 2 * i + 1;
  const int h0 = blockIdx.y * p.heads_per_slice;
  const int h1 = min(h0 + p.heads_per_slice, p.Hq + p.Hkv);
#pragma unroll 4
  for (int h = h0; h < h1; ++h) {
    const bool is_q = h < p.Hq;
    if (!turns && !(is_q ? p.copy_q : p.copy_k)) continue;
    const uint16_t* src = is_q ? p.q + row * p.q_stride + static_cast<long long>(h) * p.D
                               : p.k + row * p.k_stride + static_cast<long long>(h - p.Hq) * p.D;
    uint16_t* dst = is_q ? p.q_out + row * p.q_out_stride + static_cast<long long>(h) * p.D
                         : p.k_out + row * p.k_out_stride + static_cast<long long>(h - p.Hq) * p.D;
    if (wide) {
      *reinterpret_cast<uint4*>(dst + ua) = *reinterpret_cast<const uint4*>(src + ua);
      continue;
    }
    const uint32_t xa = src[ua], xb = src[ub];
    uint32_t w = xa | (xb << 16);
    if (turns) w = pack(lo(w) * c - hi(w) * s, hi(w) * c + lo(w) * s);
    dst[ua] = static_cast<uint16_t>(w);
    dst[ub] = static_cast<uint16_t>(w >> 16);
  }
}

}  // namespace

int launch_rope(const RopeArgs& a) {
  int sms = 0;
  if (int rc = device_sms(&sms)) return rc;
  RopeParams p;
  p.q = static_cast<const uint16_t*>(a.q);
  p.q_out = static_cast<uint16_t*>(a.q_out);
  p.k = static_cast<const uint16_t*>(a.k);
  p.k_out = static_cast<uint16_t*>(a.k_out);
  p.rows = a.rows;
  p.N = a.N; p.Hq = a.Hq; p.Hkv = a.Hkv; p.D = a.D; p.rot = a.rot;
  p.q_stride = a.q_stride; p.q_out_stride = a.q_out_stride;
  p.k_stride = a.k_stride; p.k_out_stride = a.k_out_stride;
  p.interleaved = a.layout == TM_ROPE_INTERLEAVED;
  p.copy_q = a.q != a.q_out;
  p.copy_k = a.k != a.k_out;
  p.sign = a.inverse ? -1.f : 1.f;
  p.mscale = a.mscale;
  p.inv_freq = a.inv_freq;
  p.positions = a.positions;
  p.first = a.first;
  const bool wide = a.rot % 16 == 0;
  const int per = wide ? a.D / 16 : any_slots(a.rot, a.D), heads = a.Hq + a.Hkv;
  const long long blocks = (a.rows * per + 255) / 256;
  // Short calls cut the heads into slices until every SM has a few blocks; each
  // slice computes the angles again.
  long long slices = blocks >= 8LL * sms ? 1 : (8LL * sms + blocks - 1) / blocks;
  if (slices > (heads + 3) / 4) slices = (heads + 3) / 4;
  p.heads_per_slice = static_cast<int>((heads + slices - 1) / slices);
  const dim3 grid(static_cast<unsigned>(blocks),
                  static_cast<unsigned>((heads + p.heads_per_slice - 1) / p.heads_per_slice));
  const long long far = 1LL << 31;
  auto kernel = wide ? rope_kernel<false> : rope_any_kernel<false>;
  if (!a.positions && (a.first < -far || a.first + a.N > far))
    kernel = wide ? rope_kernel<true> : rope_any_kernel<true>;
  if (launch_early(kernel, grid, 256, 0, static_cast<cudaStream_t>(a.stream), 1, p))
    return TM_ERR_CUDA;
  return count_launches(1);
}

}  // namespace trimix
