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
// last of a prompt) takes the path without bounds, which cost a third of the
// instructions: 131072 tokens of 8 heads in 117 us (6.87 TB/s), with them in 139 us.
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
        x[i] = *reinterpret_cast<const uint4*>(at);
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
            x[i] = *reinterpret_cast<const uint4*>(src + tok * stride);
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

// One CTA per (new block, head): gathers the block's tokens of k and v from the old
// pages. The new range is the largest range among their source blocks, so codes
// from a block of that range move unchanged and the others are rounded once to
// its step; no token's values are scanned for a maximum. The chain index, page,
// range, codes bounds a short call, so every lane's loads of k and v go out together.
// 16 sequences that keep up to 2048 tokens of 8 heads: 37 MB read and as much written
// in 13 us behind the selection.
template <int FMT, int D, int P>
__global__ void __launch_bounds__(kCacheThreads) compact_kernel(const Kv8CompactArgs a) {
  constexpr int RC = D / 16;                          // 16-byte chunks of a row
  constexpr int NC = (P * RC + kCacheThreads - 1) / kCacheThreads;
  pdl_launch();
  pdl_wait();
  const int H = a.c.Hkv, b = blockIdx.z, blk = blockIdx.y, h = blockIdx.x, t = threadIdx.x;
  const int kept = a.kept ? min(max(a.kept[b], 0), a.keep) : a.keep;
  const int rows = min(kept - blk * P, P);
  if (rows <= 0) return;
  const int to = a.new_table[static_cast<long long>(b) * a.new_max_pages + blk];
  if (to < 0 || to >= a.c.num_pages) return;
  __shared__ long long s_src[P];  // first byte of the source row, or -1
  __shared__ float s_kr[P], s_vr[P];
  __shared__ uint32_t red[2][kCacheThreads / 32];
  uint32_t mk = 0, mv = 0;
  if (t < rows) {
    const long long at = static_cast<long long>(b) * H + h;
    const int i = a.index[at * a.keep + blk * P + t];
    long long src = -1;
    float kr = 0.f, vr = 0.f, w = 0.f;
    const long long len = min(static_cast<long long>(a.lens[b]),
                              static_cast<long long>(a.max_pages) * P);
    if (i >= 0 && i < len) {
      const int page = a.table[static_cast<long long>(b) * a.max_pages + i / P];
      if (a.new_weights && i < a.weights_stride) w = a.weights[at * a.weights_stride + i];
      if (page >= 0 && page < a.c.num_pages) {
        const long long block = static_cast<long long>(page) * H + h;
        src = (block * P + i % P) * D;
        kr = a.c.k_range[block];
        vr = a.c.v_range[block];
      } else {
        w = 0.f;
      }
    }
    s_src[t] = src;
    s_kr[t] = kr;
    s_vr[t] = vr;
    mk = __float_as_uint(kr);
    mv = __float_as_uint(vr);
    if (a.new_weights) a.new_weights[at * a.new_weights_stride + blk * P + t] = w;
  }
  mk = warp_max(mk);
  mv = warp_max(mv);
  if ((t & 31) == 0) {
    red[0][t >> 5] = mk;
    red[1][t >> 5] = mv;
  }
  __syncthreads();
  const uint4* k8 = static_cast<const uint4*>(a.c.k8);
  const uint4* v8 = static_cast<const uint4*>(a.c.v8);
  uint4 ck[NC], cv[NC];
#pragma unroll
  for (int i = 0; i < NC; ++i) {
    const int ch = i * kCacheThreads + t, row = ch / RC;
    ck[i] = cv[i] = make_uint4(0, 0, 0, 0);
    if (row < rows && s_src[row] >= 0) {
      const long long at = s_src[row] / 16 + ch % RC;
      ck[i] = k8[at];
      cv[i] = v8[at];
    }
  }
#pragma unroll
  for (int w = 0; w < kCacheThreads / 32; ++w) {
    mk = max(mk, red[0][w]);
    mv = max(mv, red[1][w]);
  }
  const float rk = __uint_as_float(mk), rv = __uint_as_float(mv);
  const bool lk = finite(rk) && rk > 0.f, lv = finite(rv) && rv > 0.f;
  const long long block = static_cast<long long>(to) * H + h;
  uint4* dk = static_cast<uint4*>(a.c.k8) + block * (P * RC);
  uint4* dv = static_cast<uint4*>(a.c.v8) + block * (P * RC);
  auto moved = [](uint4 c, float r1, float r, bool live) {
    if (!live) return make_uint4(0, 0, 0, 0);
    if (r1 == r) return c;
    const float ratio = __fdiv_rn(r1, r);
    return make_uint4(rescale4<FMT>(c.x, ratio), rescale4<FMT>(c.y, ratio), rescale4<FMT>(c.z, ratio),
                      rescale4<FMT>(c.w, ratio));
  };
#pragma unroll
  for (int i = 0; i < NC; ++i) {
    const int ch = i * kCacheThreads + t, row = ch / RC;
    if (row >= rows) continue;
    dk[ch] = moved(ck[i], s_kr[row], rk, lk);
    dv[ch] = moved(cv[i], s_vr[row], rv, lv);
  }
  if (t == 0) {
    a.c.k_range[block] = rk;
    a.c.v_range[block] = rv;
  }
}

template <int FMT>
int compact_run(const Kv8CompactArgs& a) {
  auto kernel = compact_kernel<FMT, 128, 128>;
  if (a.c.D == 128)
    kernel = a.c.page == 16   ? compact_kernel<FMT, 128, 16>
             : a.c.page == 32 ? compact_kernel<FMT, 128, 32>
             : a.c.page == 64 ? compact_kernel<FMT, 128, 64>
                              : compact_kernel<FMT, 128, 128>;
  else
    kernel = a.c.page == 16   ? compact_kernel<FMT, 64, 16>
             : a.c.page == 32 ? compact_kernel<FMT, 64, 32>
             : a.c.page == 64 ? compact_kernel<FMT, 64, 64>
                              : compact_kernel<FMT, 64, 128>;
  const dim3 grid(a.c.Hkv, (a.keep + a.c.page - 1) / a.c.page, a.B);
  if (launch_early(kernel, grid, kCacheThreads, 0, static_cast<cudaStream_t>(a.stream), 1, a))
    return TM_ERR_CUDA;
  return count_launches(1);
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
  return a.c.format == TM_KV_INT8 ? compact_run<TM_KV_INT8>(a) : compact_run<TM_KV_E4M3>(a);
}

}  // namespace trimix
