// Writing the paged 8-bit cache: new tokens into it (append), kept tokens into
// other pages of it (compact). Layout: codes [num_pages, Hkv, page, D], one
// range per (page, head) in ranges [num_pages, Hkv]; the rows of a (page, head)
// block are contiguous.
#include <cuda_runtime.h>

#include "tm.h"
#include "tm_internal.h"
#include "tm_kv8.cuh"
#include "tm_launch.cuh"

namespace trimix {
namespace {

using namespace kv8;

constexpr int kCacheThreads = 128;

struct AppendParams {
  Kv8AppendArgs a;
  int row_chunks_log;  // log2 of the 8-element chunks of a row
};

// One CTA per (touched block, head, k or v). The block's range becomes the
// larger of its old range (if it already holds tokens of this sequence) and the
// new tokens' largest |x|; where it grows, the old codes are moved to it.
// The block's new elements stay in registers between the maximum and the
// rounding, so k and v are read once: 2 bytes read and 1 written an element.
template <int FMT, int NC>
__global__ void __launch_bounds__(kCacheThreads) append_kernel(const AppendParams p) {
  pdl_launch();
  pdl_wait();
  const Kv8AppendArgs& a = p.a;
  const int P = a.c.page, D = a.c.D, H = a.c.Hkv, b = blockIdx.z;
  // heads vary fastest: the CTAs that run together read whole rows of k and v
  const int frame = blockIdx.x / (2 * H), hv = blockIdx.x - frame * 2 * H;
  const bool is_v = hv >= H;
  const int h = is_v ? hv - H : hv;
  const long long cap = static_cast<long long>(a.max_pages) * P;
  const long long len = min(max(static_cast<long long>(a.lens[b]), 0LL), cap);
  const int count = a.counts ? min(max(a.counts[b], 0), a.n) : a.n;
  const int blk = static_cast<int>(len / P) + frame;
  if (blk >= a.max_pages) return;
  const long long base = static_cast<long long>(blk) * P;
  const int r_lo = static_cast<int>(max(len - base, 0LL));
  const int r_hi = static_cast<int>(min(len + count - base, static_cast<long long>(P)));
  if (r_hi <= r_lo) return;
  const int page = a.table[static_cast<long long>(b) * a.max_pages + blk];
  if (page < 0 || page >= a.c.num_pages) return;

  const int t = threadIdx.x, cl = p.row_chunks_log, cm = (1 << cl) - 1;
  const long long stride = is_v ? a.v_stride : a.k_stride;
  const uint16_t* src = static_cast<const uint16_t*>(is_v ? a.v : a.k) +
                        static_cast<long long>(b) * a.n_src * stride + h * D;
  const long long tok0 = base - len;  // source token of the block's row 0
  const int* index = a.index ? a.index + (static_cast<long long>(b) * H + h) * a.n : nullptr;
  uint4 x[NC];
  uint32_t mx = 0;
#pragma unroll
  for (int i = 0; i < NC; ++i) {
    const int ch = i * kCacheThreads + t, row = ch >> cl;
    x[i] = make_uint4(0, 0, 0, 0);
    if (row >= r_lo && row < r_hi) {
      long long tok = tok0 + row;
      if (index) tok = index[tok];
      if (tok >= 0 && tok < a.n_src)
        x[i] = __ldg(reinterpret_cast<const uint4*>(src + tok * stride) + (ch & cm));
    }
  }
#pragma unroll
  for (int i = 0; i < NC; ++i) {  // |x| of bf16 orders as its bits do, NaN above infinity
    const uint32_t m01 = __vmaxu2(x[i].x & 0x7FFF7FFFu, x[i].y & 0x7FFF7FFFu);
    const uint32_t m23 = __vmaxu2(x[i].z & 0x7FFF7FFFu, x[i].w & 0x7FFF7FFFu);
    mx = __vmaxu2(mx, __vmaxu2(m01, m23));
  }
  __shared__ uint32_t red[kCacheThreads / 32];
  mx = warp_max(max(mx & 0xFFFFu, mx >> 16));
  if ((t & 31) == 0) red[t >> 5] = mx;
  float* range = (is_v ? a.c.v_range : a.c.k_range) + static_cast<long long>(page) * H + h;
  const float r_old = r_lo > 0 ? *range : 0.f;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kCacheThreads / 32; ++w) mx = max(mx, red[w]);
  const uint32_t r_bits = max(mx << 16, __float_as_uint(r_old));  // NaN and inf propagate
  const float r = __uint_as_float(r_bits);

  uint8_t* codes = static_cast<uint8_t*>(is_v ? a.c.v8 : a.c.k8) +
                   (static_cast<long long>(page) * H + h) * P * D;
  const bool live = finite(r) && r > 0.f;
  // A range below 2^-64 would overflow F / r: both sides are scaled by 2^64.
  const float up = r < 5.421010862427522e-20f ? 18446744073709551616.f : 1.f;
  const float inv = live ? __fdiv_rn(full<FMT>(), r * up) : 0.f;
#pragma unroll
  for (int i = 0; i < NC; ++i) {
    const int ch = i * kCacheThreads + t, row = ch >> cl;
    if (row < r_lo || row >= r_hi) continue;
    const uint32_t w[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
    float f[8];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      f[2 * e] = __uint_as_float(w[e] << 16) * up * inv;
      f[2 * e + 1] = __uint_as_float(w[e] & 0xFFFF0000u) * up * inv;
    }
    uint2 o = make_uint2(encode4<FMT>(f[0], f[1], f[2], f[3]), encode4<FMT>(f[4], f[5], f[6], f[7]));
    if (!live) o = make_uint2(0, 0);
    reinterpret_cast<uint2*>(codes)[ch] = o;
  }
  if (r_lo > 0 && r != r_old) {
    const float ratio = live ? __fdiv_rn(r_old, r) : 0.f;
    for (int ch = t; ch < (r_lo << cl); ch += kCacheThreads) {
      uint2 o = reinterpret_cast<uint2*>(codes)[ch];
      o = live ? make_uint2(rescale4<FMT>(o.x, ratio), rescale4<FMT>(o.y, ratio)) : make_uint2(0, 0);
      reinterpret_cast<uint2*>(codes)[ch] = o;
    }
  }
  if (t == 0) *range = r;
}

// One CTA per (new block, head, k or v): gathers the block's tokens from the old
// pages. The new range is the largest range among their source blocks, so codes
// from a block of that range move unchanged and the others are rounded once to
// its step; no token's values are scanned for a maximum.
template <int FMT>
__global__ void __launch_bounds__(kCacheThreads) compact_kernel(const Kv8CompactArgs a) {
  pdl_launch();
  pdl_wait();
  const int P = a.c.page, D = a.c.D, H = a.c.Hkv, b = blockIdx.z, blk = blockIdx.x, t = threadIdx.x;
  const int h = blockIdx.y >> 1;
  const bool is_v = blockIdx.y & 1;
  const int kept = a.kept ? min(max(a.kept[b], 0), a.keep) : a.keep;
  const int rows = min(kept - blk * P, P);
  if (rows <= 0) return;
  const int to = a.new_table[static_cast<long long>(b) * a.new_max_pages + blk];
  if (to < 0 || to >= a.c.num_pages) return;
  const float* ranges = is_v ? a.c.v_range : a.c.k_range;
  uint8_t* codes = static_cast<uint8_t*>(is_v ? a.c.v8 : a.c.k8);
  __shared__ long long s_src[128];  // first byte of the source row, or -1
  __shared__ float s_range[128];
  __shared__ uint32_t red[kCacheThreads / 32];
  uint32_t mx = 0;
  if (t < rows) {
    const long long at = static_cast<long long>(b) * H + h;
    const int i = a.index[at * a.keep + blk * P + t];
    long long src = -1;
    float r = 0.f;
    const long long len = min(static_cast<long long>(a.lens[b]),
                              static_cast<long long>(a.max_pages) * P);
    if (i >= 0 && i < len) {
      const int page = a.table[static_cast<long long>(b) * a.max_pages + i / P];
      if (page >= 0 && page < a.c.num_pages) {
        src = ((static_cast<long long>(page) * H + h) * P + i % P) * D;
        r = ranges[static_cast<long long>(page) * H + h];
      }
    }
    s_src[t] = src;
    s_range[t] = r;
    mx = __float_as_uint(r);
    if (!is_v && a.new_weights)
      a.new_weights[at * a.new_weights_stride + blk * P + t] =
          src >= 0 && i < a.weights_stride ? a.weights[at * a.weights_stride + i] : 0.f;
  }
  mx = warp_max(mx);
  if ((t & 31) == 0) red[t >> 5] = mx;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kCacheThreads / 32; ++w) mx = max(mx, red[w]);
  const float r = __uint_as_float(mx);
  const bool live = finite(r) && r > 0.f;
  const int cl = D == 128 ? 3 : 2;  // 16-byte chunks of a row, log2
  uint4* dst = reinterpret_cast<uint4*>(codes + (static_cast<long long>(to) * H + h) * P * D);
  for (int ch = t; ch < (rows << cl); ch += kCacheThreads) {
    const int row = ch >> cl;
    const long long src = s_src[row];
    uint4 o = make_uint4(0, 0, 0, 0);
    if (src >= 0 && live) {
      o = *(reinterpret_cast<const uint4*>(codes + src) + (ch & ((1 << cl) - 1)));
      const float r1 = s_range[row];
      if (r1 != r) {
        const float ratio = __fdiv_rn(r1, r);
        o = make_uint4(rescale4<FMT>(o.x, ratio), rescale4<FMT>(o.y, ratio),
                       rescale4<FMT>(o.z, ratio), rescale4<FMT>(o.w, ratio));
      }
    }
    dst[ch] = o;
  }
  if (t == 0) (is_v ? a.c.v_range : a.c.k_range)[static_cast<long long>(to) * H + h] = r;
}

template <int FMT>
int append_fmt(const Kv8AppendArgs& a) {
  AppendParams p;
  p.a = a;
  p.row_chunks_log = a.c.D == 128 ? 4 : 3;
  const long long frames = (a.n + a.c.page - 2LL) / a.c.page + 1;
  const dim3 grid(static_cast<unsigned>(frames * 2 * a.c.Hkv), 1, a.B);
  cudaStream_t st = static_cast<cudaStream_t>(a.stream);
  auto kernel = append_kernel<FMT, 16>;
  switch (a.c.page * a.c.D / (8 * kCacheThreads)) {
    case 1: kernel = append_kernel<FMT, 1>; break;
    case 2: kernel = append_kernel<FMT, 2>; break;
    case 4: kernel = append_kernel<FMT, 4>; break;
    case 8: kernel = append_kernel<FMT, 8>; break;
    default: break;
  }
  if (launch_early(kernel, grid, kCacheThreads, 0, st, 1, p)) return TM_ERR_CUDA;
  return count_launches(1);
}

}  // namespace

int launch_kv8_append(const Kv8AppendArgs& a) {
  int sms = 0;
  if (int rc = device_sms(&sms)) return rc;
  return a.c.format == TM_KV_INT8 ? append_fmt<TM_KV_INT8>(a) : append_fmt<TM_KV_E4M3>(a);
}

int launch_kv8_compact(const Kv8CompactArgs& a) {
  int sms = 0;
  if (int rc = device_sms(&sms)) return rc;
  const dim3 grid((a.keep + a.c.page - 1) / a.c.page, 2 * a.c.Hkv, a.B);
  cudaStream_t st = static_cast<cudaStream_t>(a.stream);
  auto kernel = a.c.format == TM_KV_INT8 ? compact_kernel<TM_KV_INT8> : compact_kernel<TM_KV_E4M3>;
  if (launch_early(kernel, grid, kCacheThreads, 0, st, 1, a)) return TM_ERR_CUDA;
  return count_launches(1);
}

}  // namespace trimix
