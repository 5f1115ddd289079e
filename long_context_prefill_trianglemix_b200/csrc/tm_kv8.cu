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
  long long frames;  // blocks a sequence's new tokens can touch
};

// A block's range becomes the larger of its old range (if it already holds tokens
// of this sequence) and the new tokens' largest |x|; where it grows, the old codes
// are moved to it. BW warps share a block of P = 32 BW NC 8 / D rows, NC chunks of 8
// elements a lane, and a CTA takes several small blocks; the elements stay in
// registers between the maximum and the rounding, so k and v are read once: 2 bytes
// read and 1 written an element. Heads vary fastest over the grid: CTAs that run
// together read whole rows. A block that is new throughout (all but the first and
// last of a prompt) takes the path without bounds: 17 instructions an element with
// them kept this kernel at 0.7 of the memory's rate.
template <int FMT, int D, int BW, int NC>
__global__ void __launch_bounds__(BW > 4 ? BW * 32 : 128) append_kernel(const AppendParams p) {
  constexpr int P = 32 * BW * NC * 8 / D, NT = 32 * BW, RC = D / 8, STEP = NT / RC;
  pdl_launch();
  pdl_wait();
  __shared__ uint32_t red[8];
  const Kv8AppendArgs& a = p.a;
  const int H = a.c.Hkv, b = blockIdx.z;
  const bool is_v = blockIdx.x >= static_cast<unsigned>(H);
  const int h = is_v ? blockIdx.x - H : blockIdx.x;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int sub = warp / BW, t = (warp % BW) * 32 + lane;  // block of the trip, thread of the block
  const int per = (blockDim.x >> 5) / BW;
  const long long cap = static_cast<long long>(a.max_pages) * P;
  const long long len = min(max(static_cast<long long>(a.lens[b]), 0LL), cap);
  const int count = a.counts ? min(max(a.counts[b], 0), a.n) : a.n;
  const long long first = len / P;
  const long long stride = is_v ? a.v_stride : a.k_stride;
  const uint16_t* src = static_cast<const uint16_t*>(is_v ? a.v : a.k) +
                        static_cast<long long>(b) * a.n_src * stride + h * D + (t % RC) * 8;
  const int* index = a.index ? a.index + (static_cast<long long>(b) * H + h) * a.n : nullptr;

  for (long long f0 = static_cast<long long>(blockIdx.y) * per; f0 < p.frames;
       f0 += static_cast<long long>(gridDim.y) * per) {  // the same trips for the whole CTA
    const long long blk = first + f0 + sub;
    const long long base = blk * P;
    // rows [r_lo, r_hi) of the block are new; none if the block is not touched or not there
    const int r_lo = static_cast<int>(max(len - base, 0LL));
    int r_hi = static_cast<int>(min(len + count - base, static_cast<long long>(P)));
    int page = -1;
    if (f0 + sub < p.frames && blk < a.max_pages && r_hi > r_lo)
      page = a.table[static_cast<long long>(b) * a.max_pages + blk];
    if (page < 0 || page >= a.c.num_pages) r_hi = r_lo;
    const bool used = r_hi > r_lo;

    const long long tok0 = base - len;  // source token of the block's row 0
    const bool full = !index && r_lo == 0 && r_hi == P;  // then n <= n_src bounds the tokens
    uint4 x[NC];
    if (full) {
      const uint16_t* at = src + (tok0 + t / RC) * stride;
#pragma unroll
      for (int i = 0; i < NC; ++i) {
        x[i] = __ldg(reinterpret_cast<const uint4*>(at));
        at += STEP * stride;
      }
    } else {
#pragma unroll
      for (int i = 0; i < NC; ++i) {
        const int row = t / RC + i * STEP;
        x[i] = make_uint4(0, 0, 0, 0);
        if (row >= r_lo && row < r_hi) {
          long long tok = tok0 + row;
          if (index) tok = index[tok];
          if (tok >= 0 && tok < a.n_src)
            x[i] = __ldg(reinterpret_cast<const uint4*>(src + tok * stride));
        }
      }
    }
    float* range = (is_v ? a.c.v_range : a.c.k_range) + static_cast<long long>(page) * H + h;
    const float r_old = used && r_lo > 0 ? *range : 0.f;
    __nv_bfloat162 top = __halves2bfloat162(__ushort_as_bfloat16(0), __ushort_as_bfloat16(0));
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      const uint32_t w[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
#pragma unroll
      for (int e = 0; e < 4; ++e)
        top = __hmax2_nan(top, __habs2(*reinterpret_cast<const __nv_bfloat162*>(&w[e])));
    }
    uint32_t mx = *reinterpret_cast<const uint32_t*>(&top);  // bits of |x| order as the values, NaN on top
    mx = warp_max(max(mx & 0xFFFFu, mx >> 16));
    if (BW > 1) {
      if (lane == 0) red[warp] = mx;
      __syncthreads();
#pragma unroll
      for (int w = 0; w < BW; ++w) mx = max(mx, red[sub * BW + w]);
      __syncthreads();  // read before the next trip writes it, and *range before it is replaced
    }
    __syncwarp();
    if (!used) continue;
    const uint32_t r_bits = max(mx << 16, __float_as_uint(r_old));  // NaN and inf propagate
    const float r = __uint_as_float(r_bits);

    uint2* codes = reinterpret_cast<uint2*>(static_cast<uint8_t*>(is_v ? a.c.v8 : a.c.k8) +
                                            (static_cast<long long>(page) * H + h) * (P * D)) + t;
    const bool live = finite(r) && r > 0.f;
    // A range below 2^-64 would overflow F / r: both sides are scaled by 2^64.
    const bool tiny = r < 5.421010862427522e-20f;
    const float inv = live ? code_factor<FMT>(tiny ? r * 18446744073709551616.f : r) : 0.f;
    if (full && live && !tiny) {
#pragma unroll
      for (int i = 0; i < NC; ++i) codes[i * NT] = encode8<FMT, false>(x[i], inv);
    } else {
#pragma unroll
      for (int i = 0; i < NC; ++i) {
        const int row = t / RC + i * STEP;
        if (row < r_lo || row >= r_hi) continue;
        uint2 o = tiny ? encode8<FMT, true>(x[i], inv) : encode8<FMT, false>(x[i], inv);
        codes[i * NT] = live ? o : make_uint2(0, 0);
      }
    }
    if (r_lo > 0 && r != r_old) {
      const float ratio = live ? __fdiv_rn(r_old, r) : 0.f;
      for (int ch = t; ch < r_lo * RC; ch += NT) {
        const uint2 o = codes[ch - t];
        codes[ch - t] =
            live ? make_uint2(rescale4<FMT>(o.x, ratio), rescale4<FMT>(o.y, ratio)) : make_uint2(0, 0);
      }
    }
    if (t == 0) *range = r;
  }
}

template <int FMT, int D, int BW, int NC>
int append_run(AppendParams& p) {
  const Kv8AppendArgs& a = p.a;
  // a short call leaves a block to a CTA of its own, a long one fills CTAs of four warps
  const int threads = p.frames < 8 || BW > 4 ? 32 * BW : 128;
  const long long per = threads / (32 * BW), groups = (p.frames + per - 1) / per;
  const dim3 grid(2 * a.c.Hkv, static_cast<unsigned>(groups < 65535 ? groups : 65535), a.B);
  if (launch_early(append_kernel<FMT, D, BW, NC>, grid, threads, 0, static_cast<cudaStream_t>(a.stream),
                   1, p))
    return TM_ERR_CUDA;
  return count_launches(1);
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
  p.frames = (a.n + a.c.page - 2LL) / a.c.page + 1;
  if (a.c.D == 128) {
    switch (a.c.page) {
      case 16: return append_run<FMT, 128, 1, 8>(p);
      case 32: return append_run<FMT, 128, 2, 8>(p);
      case 64: return append_run<FMT, 128, 4, 8>(p);
      default: return append_run<FMT, 128, 8, 8>(p);
    }
  }
  switch (a.c.page) {
    case 16: return append_run<FMT, 64, 1, 4>(p);
    case 32: return append_run<FMT, 64, 1, 8>(p);
    case 64: return append_run<FMT, 64, 2, 8>(p);
    default: return append_run<FMT, 64, 4, 8>(p);
  }
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
