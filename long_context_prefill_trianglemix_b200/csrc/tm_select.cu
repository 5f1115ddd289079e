// Choosing the keys a cache keeps: per (sequence, kv head), the first `sinks`
// and last `recent` of n tokens, and the heaviest of the others up to `keep` in
// all, as ascending indices. Ties go to the lowest index; NaN weighs least.
//
// A radix selection: weights map to 32-bit keys that order as they do, and three
// passes over the row (11, 11 and 10 bits) find the smallest kept key T by
// histograms from the top; a fourth writes the tokens above T and the first of
// those equal to it. One thread-block cluster per row shares the histograms
// through distributed shared memory, so a long row uses several SMs and the
// whole selection is one launch.
#include <cooperative_groups.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "tm.h"
#include "tm_internal.h"

namespace trimix {
namespace {

namespace cg = cooperative_groups;

constexpr int kSelThreads = 1024;
constexpr int kSelMaxCluster = 8;
constexpr int kBins = 2048;

struct SelParams {
  KvSelectArgs a;
  int cached;  // keys of a CTA's part that fit its shared memory
};

__device__ __forceinline__ uint32_t sort_key(float w) {
  if (w != w) return 0u;
  const uint32_t u = __float_as_uint(w + 0.f);  // -0 counts as 0
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

// Exclusive prefix of v over the CTA's threads; *total gets the sum.
__device__ __forceinline__ int block_scan(int v, int* part, int* total) {
  const int t = threadIdx.x, lane = t & 31, w = t >> 5;
  int x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  if (lane == 31) part[w] = x;
  __syncthreads();
  if (w == 0) {
    int s = part[lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, s, o);
      if (lane >= o) s += y;
    }
    part[lane] = s;
  }
  __syncthreads();
  const int before = w ? part[w - 1] : 0;
  *total = part[31];
  __syncthreads();
  return before + x - v;
}

__global__ void __launch_bounds__(kSelThreads, 1) select_kernel(const SelParams p) {
  const KvSelectArgs& a = p.a;
  extern __shared__ uint32_t s_keys[];
  __shared__ int hist[kBins];
  __shared__ int part[32];
  __shared__ int s_pick[2];   // chosen bin, kept tokens above it
  __shared__ int s_count[2];  // this CTA's tokens above T, equal to T
  cg::cluster_group cluster = cg::this_cluster();
  const int C = static_cast<int>(cluster.num_blocks()), rank = static_cast<int>(cluster.block_rank());
  const int row = blockIdx.x / C, b = row / a.H, t = threadIdx.x;
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
  const int cached = min(hi - lo, p.cached);
  auto fresh = [&](int i) {
    return i < a.sinks || i >= n - a.recent ? 0xFFFFFFFFu : sort_key(w[i]);
  };
  auto key_of = [&](int i) { return i - lo < cached ? s_keys[i - lo] : fresh(i); };

  uint32_t prefix = 0, mask = 0;
  int need = kept;  // tokens still to take among those that match the prefix
#pragma unroll 1
  for (int pass = 0; pass < 3; ++pass) {
    const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0;
    const uint32_t bins = pass == 2 ? 1024u : 2048u;
    for (int i = t; i < kBins; i += kSelThreads) hist[i] = 0;
    __syncthreads();
    for (int i = lo + t; i < hi; i += kSelThreads) {
      uint32_t key;
      if (pass == 0) {
        key = fresh(i);
        if (i - lo < cached) s_keys[i - lo] = key;
      } else {
        key = key_of(i);
      }
      if ((key & mask) == prefix) atomicAdd(&hist[(key >> shift) & (bins - 1)], 1);
    }
    cluster.sync();
    // bins from the top: thread t owns the two bins 2047 - 2t, 2046 - 2t
    const int b1 = kBins - 1 - 2 * t, b0 = b1 - 1;
    int c1 = 0, c0 = 0;
    for (int r = 0; r < C; ++r) {
      const int* h = cluster.map_shared_rank(hist, r);
      c1 += h[b1];
      c0 += h[b0];
    }
    int total;
    const int above = block_scan(c1 + c0, part, &total);
    if (above < need && above + c1 >= need) {
      s_pick[0] = b1;
      s_pick[1] = above;
    } else if (above + c1 < need && above + c1 + c0 >= need) {
      s_pick[0] = b0;
      s_pick[1] = above + c1;
    }
    cluster.sync();  // every CTA has read the histograms; s_pick is visible
    prefix |= static_cast<uint32_t>(s_pick[0]) << shift;
    mask |= (bins - 1) << shift;
    need -= s_pick[1];
  }
  // prefix is T; `need` tokens equal to it are kept, the first ones of the row.
  if (t < 2) s_count[t] = 0;
  __syncthreads();
  int gt = 0, eq = 0;
  for (int i = lo + t; i < hi; i += kSelThreads) {
    const uint32_t key = key_of(i);
    gt += key > prefix;
    eq += key == prefix;
  }
  atomicAdd(&s_count[0], gt);
  atomicAdd(&s_count[1], eq);
  cluster.sync();
  int gt_before = 0, eq_before = 0;
  for (int r = 0; r < rank; ++r) {
    const int* c = cluster.map_shared_rank(s_count, r);
    gt_before += c[0];
    eq_before += c[1];
  }
  int pos = gt_before + min(eq_before, need);
  for (int i0 = lo; i0 < hi; i0 += kSelThreads) {
    const int i = i0 + t;
    const uint32_t key = i < hi ? key_of(i) : 0u;
    const bool is_eq = i < hi && key == prefix;
    int n_eq, n_keep;
    const int eq_at = block_scan(is_eq, part, &n_eq);
    const bool take = i < hi && (key > prefix || (is_eq && eq_before + eq_at < need));
    const int at = block_scan(take, part, &n_keep);
    if (take) out[pos + at] = i;
    pos += n_keep;
    eq_before += n_eq;
  }
  cluster.sync();  // no CTA leaves while another reads its shared memory
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
  SelParams p;
  p.a = a;
  p.cached = per < 40960 ? per : 40960;
  const int smem = p.cached * 4;
  if (cudaFuncSetAttribute(select_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, 40960 * 4) !=
      cudaSuccess)
    return TM_ERR_CUDA;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(rows * C));
  cfg.blockDim = dim3(kSelThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = static_cast<cudaStream_t>(a.stream);
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = C;
  attr.val.clusterDim.y = 1;
  attr.val.clusterDim.z = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  if (cudaLaunchKernelEx(&cfg, select_kernel, p) != cudaSuccess) {
    cudaGetLastError();
    return TM_ERR_CUDA;
  }
  return count_launches(1);
}

}  // namespace trimix
