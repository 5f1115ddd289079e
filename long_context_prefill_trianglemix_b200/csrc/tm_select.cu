// Choosing the keys a cache keeps: per (sequence, kv head), the first `sinks`
// and last `recent` of n tokens, and the heaviest of the others up to `keep` in
// all, as ascending indices. Ties go to the lowest index; NaN weighs least.
//
// A radix selection: weights map to 32-bit keys that order as they do, and three
// passes over the row (11, 11 and 10 bits) find the smallest kept key T by
// histograms from the top; then the tokens above T and the first of those equal
// to it are written in order. One thread-block cluster per row shares the
// histograms through distributed shared memory, so a long row uses several SMs
// and the whole selection is one launch.
//
// Latency bounds it (a row of 131072 weights is 0.5 MB): each warp owns a
// contiguous run and keeps its keys in registers, 16 a lane, so that a part of
// up to 16384 weights is read once, its loads all in flight together; ranks
// come from ballots and one scan over the warps; each pass has its own
// histogram, so a pass costs one cluster barrier. 8 rows of 131072 weights: 12.7 us
// (14.9 where all lie in a few bins); 128 rows of 8192: 6.7 to 7.8. Clusters of 16 do
// not all fit at once: 35 us for the 8 rows. Many long rows have a CTA each, whose part
// above 16384 weights is read again by every pass: 128 rows of 32768 take 25 us, of
// 131072 77 us (67 MB, 10 us to read once).
#include <cooperative_groups.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "tm.h"
#include "tm_internal.h"
#include "tm_launch.cuh"

namespace trimix {
namespace {

namespace cg = cooperative_groups;

constexpr int kSelThreads = 1024;
constexpr int kSelMaxCluster = 8;
constexpr int kBins = 2048;
constexpr int kSelMaxKeys = 16;  // keys a lane holds at most

// 1 for NaN, 0x007FFFFF (-inf) to 0xFF800000 (+inf) otherwise; 0 is left for no weight
// and 0xFFFFFFFF for a protected one.
__device__ __forceinline__ uint32_t sort_key(float w) {
  const uint32_t u = __float_as_uint(w + 0.f);  // -0 counts as 0
  const uint32_t k = u ^ (static_cast<uint32_t>(static_cast<int>(u) >> 31) | 0x80000000u);
  return w == w ? k : 1u;
}

// The sum of v over the lanes above this one, and its own included.
__device__ __forceinline__ int sum_from_above(int v, int lane) {
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_down_sync(0xffffffffu, v, o);
    if (lane + o < 32) v += y;
  }
  return v;
}

// KPL: keys a lane holds (of a round; a part of more than 1024 KPL weights takes
// several rounds and reads them again in every pass).
template <int KPL>
__global__ void __launch_bounds__(kSelThreads, 1) select_kernel(const KvSelectArgs a) {
  constexpr int kRun = 32 * KPL;  // weights of a warp in a round
  __shared__ __align__(16) int hist[3][kBins];
  __shared__ int coarse[3][32];       // sums of 64 bins
  __shared__ int s_pick[3][3];        // of a pass: chosen bin, its tokens, kept tokens above it
  __shared__ int s_gt[32], s_eq[32];  // per warp: tokens above T, equal to T
  __shared__ int s_count[2];          // the same of this CTA
  cg::cluster_group cluster = cg::this_cluster();
  const int C = static_cast<int>(cluster.num_blocks()), rank = static_cast<int>(cluster.block_rank());
  const int row = blockIdx.x / C, b = row / a.H, t = threadIdx.x, lane = t & 31, warp = t >> 5;
  for (int i = t; i < 3 * kBins / 4; i += kSelThreads)
    reinterpret_cast<int4*>(&hist[0][0])[i] = make_int4(0, 0, 0, 0);
  if (t < 2) s_count[t] = 0;
  pdl_launch();
  pdl_wait();
  const int n = min(max(a.lens ? a.lens[b] : a.n, 0), a.n);
  int* out = a.index + static_cast<long long>(row) * a.keep;
  const int kept = min(n, a.keep);
  if (rank == 0 && row % a.H == 0 && t == 0 && a.kept) a.kept[b] = kept;
  for (int i = kept + rank * kSelThreads + t; i < a.keep; i += C * kSelThreads) out[i] = -1;
  if (n <= a.keep) {  // uniform over the cluster
    for (int i = rank * kSelThreads + t; i < n; i += C * kSelThreads) out[i] = i;
    return;
  }
  const float* w = a.weights + static_cast<long long>(row) * a.stride;
  const int per = (n + C - 1) / C;
  const int lo = min(rank * per, n), hi = min(lo + per, n);
  const int rounds = (hi - lo + kSelThreads * KPL - 1) / (kSelThreads * KPL);

  // Round r: warp v holds weights base + k 32 + lane, k < KPL, of its run.
  uint32_t key[KPL];
  int base = 0;
  bool any = false;  // the warp's run holds a weight
  auto load = [&](int r) {
    base = lo + r * kSelThreads * KPL + warp * kRun;
    any = base < hi;
    if (!any) return;
    const float* at = w + base + lane;
    if (base + kRun <= hi) {
      float x[KPL];
#pragma unroll
      for (int k = 0; k < KPL; ++k) x[k] = at[32 * k];
#pragma unroll
      for (int k = 0; k < KPL; ++k) key[k] = sort_key(x[k]);
    } else {
#pragma unroll
      for (int k = 0; k < KPL; ++k)
        key[k] = base + 32 * k + lane < hi ? sort_key(at[32 * k]) : 0u;
    }
    if (base < a.sinks || base + kRun > n - a.recent) {
#pragma unroll
      for (int k = 0; k < KPL; ++k) {
        const int i = base + 32 * k + lane;
        if (i < hi && (i < a.sinks || i >= n - a.recent)) key[k] = 0xFFFFFFFFu;
      }
    }
  };
  load(0);
  __syncthreads();

  uint32_t prefix = 0;
  int need = kept;  // tokens still to take among those that match the prefix
#pragma unroll
  for (int pass = 0; pass < 3; ++pass) {
    constexpr int kShift[3] = {21, 10, 0};
    const int shift = kShift[pass];
    const uint32_t bins = pass == 2 ? 1024u : 2048u;
    for (int r = 0; r < rounds; ++r) {
      if (rounds > 1) load(r);
      if (!any) continue;
#pragma unroll
      for (int k = 0; k < KPL; ++k) {
        if (pass == 0)
          atomicAdd(&hist[0][key[k] >> 21], 1);
        else if ((key[k] ^ prefix) >> kShift[pass > 0 ? pass - 1 : 0] == 0)
          atomicAdd(&hist[pass][(key[k] >> shift) & (bins - 1)], 1);
      }
    }
    __syncthreads();
    {
      const int2 h = *reinterpret_cast<const int2*>(&hist[pass][64 * warp + 2 * lane]);
      const int sum = __reduce_add_sync(0xffffffffu, h.x + h.y);
      if (lane == 0) coarse[pass][warp] = sum;
    }
    if (C > 1) cluster.sync(); else __syncthreads();
    // One warp finds the bin: the 64 it lies in by the coarse sums, then itself. It
    // reads 3 KB of the other CTAs' memory in two steps instead of their histograms.
    if (warp == 0) {
      int c = 0;
#pragma unroll
      for (int r = 0; r < kSelMaxCluster; ++r)
        if (r < C) c += *cluster.map_shared_rank(&coarse[pass][lane], r);
      int upto = sum_from_above(c, lane);
      const int top = 31 - __clz(__ballot_sync(0xffffffffu, upto >= need));
      const int above = __shfl_sync(0xffffffffu, upto - c, top);
      int2 f = make_int2(0, 0);
#pragma unroll
      for (int r = 0; r < kSelMaxCluster; ++r) {
        if (r < C) {
          const int2 h = *reinterpret_cast<const int2*>(
              cluster.map_shared_rank(&hist[pass][64 * top + 2 * lane], r));
          f.x += h.x;
          f.y += h.y;
        }
      }
      upto = above + sum_from_above(f.x + f.y, lane);
      const int in = 31 - __clz(__ballot_sync(0xffffffffu, upto >= need));
      if (lane == in) {
        const bool hi_bin = upto - f.x >= need;  // bins above, and the lane's upper one
        s_pick[pass][0] = 64 * top + 2 * lane + hi_bin;
        s_pick[pass][1] = hi_bin ? f.y : f.x;
        s_pick[pass][2] = hi_bin ? upto - f.x - f.y : upto - f.x;
      }
    }
    __syncthreads();
    prefix |= static_cast<uint32_t>(s_pick[pass][0]) << shift;
    need -= s_pick[pass][2];
    // The whole bin is kept (usual once it is down to a token or two): every key from its
    // lowest on. Key 0 is no weight, so a bin that starts there is looked into.
    if (pass < 2 && need == s_pick[pass][1] && prefix != 0) {
      --prefix;
      need = 0;
      break;
    }
  }
  // prefix is T; `need` tokens equal to it are kept, the first ones of the row.
  auto count = [&](int& gt, int& eq) {
    gt = eq = 0;
    if (any) {
#pragma unroll
      for (int k = 0; k < KPL; ++k) {
        gt += key[k] > prefix;
        eq += key[k] == prefix;
      }
      gt = __reduce_add_sync(0xffffffffu, gt);
      eq = __reduce_add_sync(0xffffffffu, eq);
    }
  };
  int gt = 0, eq = 0;
  for (int r = 0; r < rounds; ++r) {
    if (rounds > 1) load(r);
    int g, e;
    count(g, e);
    gt += g;
    eq += e;
  }
  if (lane == 0) {
    s_gt[warp] = gt;
    s_eq[warp] = eq;
    atomicAdd(&s_count[0], gt);
    atomicAdd(&s_count[1], eq);
  }
  if (C > 1) cluster.sync(); else __syncthreads();
  int gt_before = 0, eq_before = 0;
  for (int r = 0; r < rank; ++r) {
    const int* c = cluster.map_shared_rank(s_count, r);
    gt_before += c[0];
    eq_before += c[1];
  }
  for (int r = 0; r < rounds; ++r) {
    if (rounds > 1) {  // the counts of each warp for these weights
      load(r);
      int g, e;
      count(g, e);
      __syncthreads();
      if (lane == 0) {
        s_gt[warp] = g;
        s_eq[warp] = e;
      }
      __syncthreads();
    }
    const int wg = s_gt[lane], we = s_eq[lane];
    if (any) {
      int g0 = gt_before + __reduce_add_sync(0xffffffffu, lane < warp ? wg : 0);
      int e0 = eq_before + __reduce_add_sync(0xffffffffu, lane < warp ? we : 0);
      const uint32_t below = (1u << lane) - 1u;
#pragma unroll
      for (int k = 0; k < KPL; ++k) {
        const uint32_t bg = __ballot_sync(0xffffffffu, key[k] > prefix);
        const uint32_t be = __ballot_sync(0xffffffffu, key[k] == prefix);
        if ((bg | be) == 0) continue;
        const int eq_at = e0 + __popc(be & below);
        if (((bg >> lane) & 1u) || (((be >> lane) & 1u) && eq_at < need))
          out[g0 + __popc(bg & below) + min(eq_at, need)] = base + 32 * k + lane;
        g0 += __popc(bg);
        e0 += __popc(be);
      }
    }
    gt_before += __reduce_add_sync(0xffffffffu, wg);
    eq_before += __reduce_add_sync(0xffffffffu, we);
  }
  if (C > 1) cluster.sync();  // no CTA leaves while another reads its shared memory
}

}  // namespace

int launch_kv_select(const KvSelectArgs& a) {
  int sms = 0;
  if (int rc = device_sms(&sms)) return rc;
  // Clusters grow with the row until about 4096 keys a CTA, while all rows'
  // clusters fit the SMs together.
  int C = 1;
  const long long rows = static_cast<long long>(a.B) * a.H;
  while (C < kSelMaxCluster && a.n > 4096LL * C && rows * C * 2 <= sms) C *= 2;
  const int per = (a.n + C - 1) / C;
  auto kernel = per <= 2 * kSelThreads   ? select_kernel<2>
                : per <= 4 * kSelThreads ? select_kernel<4>
                : per <= 8 * kSelThreads ? select_kernel<8>
                                         : select_kernel<kSelMaxKeys>;
  if (launch_early(kernel, dim3(static_cast<unsigned>(rows * C)), kSelThreads, 0,
                   static_cast<cudaStream_t>(a.stream), C, a))
    return TM_ERR_CUDA;
  return count_launches(1);
}

}  // namespace trimix
