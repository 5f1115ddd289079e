// Attention weight of each key from the last queries of a prompt: for batch b,
// kv head g and key j,
//
//   w_j = sum over the rows i in [len - L, len), i >= j, and the q heads h of
//         the group, of  p_ihj = softmax_j(scale q_ih . k_j)  (causal).
//
// The denominators need a whole row before any weight is known, and the
// probabilities (L N per head) are too many to keep, so the products are formed
// twice: pass 1 for each row's log-sum-exp, pass 2 for the sums. Both are the
// same pipeline, C = A B^T with two stationary 128-row A tiles and a stream of
// 128-row B tiles, and both reduce along their own TMEM lane only:
//   pass 1  A = q rows, B = keys: a thread owns a row, running max and sum;
//   pass 2  A = keys, B = q rows: a thread owns a key and adds 2^(s - lse_row).
// Included by tm_attn.cu inside namespace trimix (status word, bounded waits,
// tensor-core helpers).
//
// CTA (320 threads, one per SM, persistent): warps 0-3 and 4-7 are two reduction
// warpgroups, one per A tile; warp 8 loads by TMA; warp 9 issues the MMAs. Each
// warpgroup has two 128-column S buffers in TMEM, so the tensor core runs ahead
// while it works. A q tile packs floor(128 / G) tokens of all G q heads of the
// group, so short L wastes no rows.
//
// Bound: one exponential per score and pass. At 16 MUFU results a clock and SM a
// 128 x 128 tile takes 1024 clocks, twice its MMA time.

constexpr int kWtThreads = 320;
constexpr int kWtStages = 2;
constexpr int kWtLse = 4;  // slots of a B tile's lse

struct WtItem {
  int b, g;     // batch, kv head
  int a0;       // first A tile (q tile in pass 1, key tile in pass 2) of the pair
  int t0, t1;   // B tiles
  int len, r0;  // tokens of the sequence, its first row
  int split;
};

struct WtParams {
  int B, Hq, Hkv, N, G, L;
  int tpt;           // tokens of a q tile
  int nqt, nkt;      // q tiles, key tiles (of the longest sequence)
  int splits;        // pass 1: parts of the key range
  int items;
  float sl2;
  const int* lens;
  float2* stats;     // pass 1: (m, l) [B Hkv][splits][nqt * 128]
  float* lse;        // [B Hkv][nqt * 128]
  float* weights;
  long long stride;
  int accumulate;
};

template <int D>
struct WtCfg {
  static constexpr int kTile = 128 * D * 2;
  static constexpr int kPanel = 128 * 64 * 2;
  static constexpr int kRing = 4 * kTile;  // two A pairs
  static constexpr int kLse = kRing + kWtStages * kTile;
  static constexpr int kBar = kLse + kWtLse * 512;
  static constexpr int kSmem = kBar + 256 + 1024;
};

struct WtBars {
  uint64_t a_full[2], a_empty[2];
  uint64_t b_full[kWtStages], b_empty[kWtStages];
  uint64_t s_full[4], s_empty[4];  // [warpgroup * 2 + buffer]
  uint64_t l_full[kWtLse];
  uint64_t mma_done;
  uint32_t tmem;
  int abort_flag;
};

__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes,
                                          uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
          dst),
      "l"(reinterpret_cast<uint64_t>(src)), "r"(bytes), "r"(smem_addr(bar))
      : "memory");
}

__device__ __forceinline__ int wt_len(const WtParams& p, int b) {
  return p.lens ? imin(p.N, p.lens[b] < 0 ? 0 : p.lens[b]) : p.N;
}

// Item i of a pass; false if it has no work (padding of a shorter sequence).
template <int PASS>
__device__ __forceinline__ bool wt_item(const WtParams& p, int i, WtItem& it) {
  const int pairs = ((PASS == 1 ? p.nqt : p.nkt) + 1) / 2;
  int x = i;
  it.split = 0;
  if (PASS == 1) {
    it.split = x % p.splits;
    x /= p.splits;
  }
  it.a0 = 2 * (x % pairs);
  x /= pairs;
  it.g = x % p.Hkv;
  it.b = x / p.Hkv;
  it.len = wt_len(p, it.b);
  const int rows = imin(p.L, it.len);
  it.r0 = it.len - rows;
  const int nqt = (rows + p.tpt - 1) / p.tpt;
  if (PASS == 1) {
    if (it.a0 >= nqt) return false;
    // keys up to the pair's last row
    const int last = it.r0 + imin(rows, (it.a0 + 2) * p.tpt);
    const int nk = (last + BN - 1) / BN;
    it.t0 = static_cast<int>(static_cast<long long>(nk) * it.split / p.splits);
    it.t1 = static_cast<int>(static_cast<long long>(nk) * (it.split + 1) / p.splits);
    return true;  // an empty part still writes its (neutral) statistics
  }
  if (it.a0 * BN >= it.len) return false;
  // q tiles with a row at or after the pair's first key
  it.t0 = imax(0, (it.a0 * BN - it.r0) / p.tpt);
  it.t1 = nqt;
  return true;
}

template <int D, int PASS>
__global__ void __launch_bounds__(kWtThreads, 1)
    weights_kernel(const __grid_constant__ CUtensorMap tq, const __grid_constant__ CUtensorMap tk,
                   const __grid_constant__ WtParams p) {
  using C = WtCfg<D>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = align1024(smem_raw);
  WtBars* bars = reinterpret_cast<WtBars*>(smem + C::kBar);
  volatile int* abort_flag = &bars->abort_flag;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  // rows that a q tile's box does not cover stay zero
  for (int i = tid; i < C::kLse / 16; i += kWtThreads)
    reinterpret_cast<uint4*>(smem)[i] = make_uint4(0, 0, 0, 0);
  if (tid == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(&bars->a_full[i], 1);
      mbar_init(&bars->a_empty[i], 1);
    }
    for (int i = 0; i < kWtStages; ++i) {
      mbar_init(&bars->b_full[i], 1);
      mbar_init(&bars->b_empty[i], 1);
    }
    for (int i = 0; i < kWtLse; ++i) mbar_init(&bars->l_full[i], 1);
    mbar_init(&bars->mma_done, 1);
    for (int i = 0; i < 4; ++i) {
      mbar_init(&bars->s_full[i], 1);
      mbar_init(&bars->s_empty[i], 4);
    }
    bars->abort_flag = 0;
    fence_barrier_init();
  }
  fence_proxy_async_smem();
  if (warp == 9) {
    tmem_alloc(&bars->tmem, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = bars->tmem;
  const uint32_t sA = smem_addr(smem), sB = sA + C::kRing;
  const int q_bytes = p.tpt * p.G * D * 2;

  if (warp == 8) {
    if (lane == 0) {
      tma_prefetch_desc(&tq);
      tma_prefetch_desc(&tk);
      uint32_t ac = 0, bc = 0;
      bool ok = true;
      // one q or key tile as D / 64 panels
      auto load_q = [&](uint32_t dst, uint64_t* bar, const WtItem& it, int tile) {
        for (int pn = 0; pn < D / 64; ++pn)
          tma_load_4d(dst + pn * C::kPanel, &tq, bar, pn * 64, it.g * p.G, it.r0 + tile * p.tpt, it.b);
      };
      auto load_k = [&](uint32_t dst, uint64_t* bar, const WtItem& it, int tile) {
        for (int pn = 0; pn < D / 64; ++pn)
          tma_load_4d(dst + pn * C::kPanel, &tk, bar, pn * 64, it.g, tile * BN, it.b);
      };
      for (int i = blockIdx.x; i < p.items && ok; i += gridDim.x) {
        WtItem it;
        if (!wt_item<PASS>(p, i, it) || it.t0 >= it.t1) continue;
        const int ab = ac & 1;
        if (!(ok = wait_bar(&bars->a_empty[ab], ((ac >> 1) & 1) ^ 1, abort_flag, kSiteWeights))) break;
        mbar_arrive_expect_tx(&bars->a_full[ab], 2 * (PASS == 1 ? q_bytes : C::kTile));
        for (int w = 0; w < 2; ++w) {
          if (PASS == 1)
            load_q(sA + (2 * ab + w) * C::kTile, &bars->a_full[ab], it, it.a0 + w);
          else
            load_k(sA + (2 * ab + w) * C::kTile, &bars->a_full[ab], it, it.a0 + w);
        }
        ++ac;
        for (int t = it.t0; t < it.t1; ++t) {
          const int st = bc % kWtStages;
          if (!(ok = wait_bar(&bars->b_empty[st], ((bc / kWtStages) & 1) ^ 1, abort_flag,
                              kSiteWeights)))
            break;
          mbar_arrive_expect_tx(&bars->b_full[st], PASS == 1 ? C::kTile : q_bytes);
          if (PASS == 1) {
            load_k(sB + st * C::kTile, &bars->b_full[st], it, t);
          } else {
            load_q(sB + st * C::kTile, &bars->b_full[st], it, t);
            // Slot reuse needs no barrier of its own: b_empty of tile n - 2 means its MMAs ran,
            // so both warpgroups had released (and so finished reading) tile n - 4.
            const int ls = bc % kWtLse;
            mbar_arrive_expect_tx(&bars->l_full[ls], 512);
            bulk_load(smem_addr(smem + C::kLse + ls * 512),
                      p.lse + (static_cast<size_t>(it.b * p.Hkv + it.g) * p.nqt + t) * 128, 512,
                      &bars->l_full[ls]);
          }
          ++bc;
        }
      }
      // Let the copies in flight land before the memory goes away (they have, unless a wait gave up).
      for (uint32_t i = 0; i < 2; ++i)
        if (ac > i) drain_wait(&bars->a_full[i], ((ac - 1 - i) / 2) & 1);
      for (uint32_t i = 0; i < kWtStages; ++i)
        if (bc > i) drain_wait(&bars->b_full[i], ((bc - 1 - i) / kWtStages) & 1);
      for (uint32_t i = 0; i < kWtLse; ++i)
        if (PASS == 2 && bc > i) drain_wait(&bars->l_full[i], ((bc - 1 - i) / kWtLse) & 1);
    }
  } else if (warp == 9) {
    const bool leader = elect_one();
    uint32_t ac = 0, bc = 0;
    bool ok = true;
    for (int i = blockIdx.x; i < p.items && ok; i += gridDim.x) {
      WtItem it;
      if (!wt_item<PASS>(p, i, it) || it.t0 >= it.t1) continue;
      const int ab = ac & 1;
      ok = __all_sync(0xffffffffu, wait_bar(&bars->a_full[ab], (ac >> 1) & 1, abort_flag, kSiteWeights));
      for (int t = it.t0; t < it.t1 && ok; ++t) {
        const int st = bc % kWtStages, buf = bc & 1;
        const uint32_t sp = ((bc >> 1) & 1) ^ 1;
        ok = __all_sync(0xffffffffu,
                        wait_bar(&bars->b_full[st], (bc / kWtStages) & 1, abort_flag, kSiteWeights));
        for (int w = 0; w < 2 && ok; ++w) {
          ok = __all_sync(0xffffffffu,
                          wait_bar(&bars->s_empty[2 * w + buf], sp, abort_flag, kSiteWeights));
          if (!ok) break;
          tc_fence_after();
          if (leader) {
            issue_qk<D>(tmem + (2 * w + buf) * 128, desc_lo_sw128(sA + (2 * ab + w) * C::kTile, 16),
                        desc_lo_sw128(sB + st * C::kTile, 16));
            mma_commit(&bars->s_full[2 * w + buf]);
          }
          __syncwarp();
        }
        if (!ok) break;
        if (leader) mma_commit(&bars->b_empty[st]);
        __syncwarp();
        ++bc;
      }
      if (!ok) break;
      if (leader) mma_commit(&bars->a_empty[ab]);
      __syncwarp();
      ++ac;
    }
    if (leader) mma_commit(&bars->mma_done);
    __syncwarp();
    drain_wait(&bars->mma_done, 0);
  } else {
    const int wg = warp >> 2, r = tid & 127;
    const uint32_t lane_addr = static_cast<uint32_t>((warp & 3) * 32) << 16;
    uint32_t bc = 0;
    bool ok = true;
    for (int i = blockIdx.x; i < p.items && ok; i += gridDim.x) {
      WtItem it;
      if (!wt_item<PASS>(p, i, it)) continue;
      const int rows = it.len - it.r0;
      const int a = it.a0 + wg;
      // pass 1: this thread's row; pass 2: its key
      const int tok = PASS == 1 ? a * p.tpt + r / p.G : 0;
      const bool live = PASS == 1 ? (r < p.tpt * p.G && tok < rows) : a * BN + r < it.len;
      const int pos = PASS == 1 ? it.r0 + tok : a * BN + r;
      float m = -1.7e38f, sum = 0.f;
      for (int t = it.t0; t < it.t1 && ok; ++t) {
        const int buf = bc & 1, ls = bc % kWtLse;
        bool here = wait_bar(&bars->s_full[2 * wg + buf], (bc >> 1) & 1, abort_flag, kSiteWeights);
        if (PASS == 2)
          here = here && wait_bar(&bars->l_full[ls], (bc / kWtLse) & 1, abort_flag, kSiteWeights);
        ok = __all_sync(0xffffffffu, here);
        if (!ok) break;
        tc_fence_after();
        const uint32_t ts = tmem + lane_addr + (2 * wg + buf) * 128;
        // columns [c_lo, c_hi) count for this thread
        int c_lo = 0, c_hi = 128;
        if (PASS == 1) {
          c_hi = imax(0, imin(128, pos + 1 - t * BN));
        } else {
          c_lo = imax(0, imin(128, (pos - (it.r0 + t * p.tpt)) * p.G));
          c_hi = imin(p.tpt, rows - t * p.tpt) * p.G;
        }
        const bool full = __all_sync(0xffffffffu, !live || (c_lo == 0 && c_hi == 128));
        const float4* z = reinterpret_cast<const float4*>(smem + C::kLse + ls * 512);
#pragma unroll
        for (int c4 = 0; c4 < 4; ++c4) {
          uint32_t s[32];
          tmem_ld32(ts + 32 * c4, s);
          tmem_wait_ld(s);
          if (PASS == 1) {
            if (!full) {
#pragma unroll
              for (int e = 0; e < 32; ++e)
                if (32 * c4 + e >= c_hi) s[e] = 0xFF800000u;
            }
            float mx = __uint_as_float(s[0]);
#pragma unroll
            for (int e = 1; e < 32; ++e) mx = fmaxf(mx, __uint_as_float(s[e]));
            mx *= p.sl2;
            if (mx > m) {
              sum *= ex2(m - mx);
              m = mx;
            }
            float a0 = 0.f, a1 = 0.f, a2 = 0.f, a3 = 0.f;
#pragma unroll
            for (int e = 0; e < 32; e += 4) {
              a0 += ex2(fmaf(__uint_as_float(s[e]), p.sl2, -m));
              a1 += ex2(fmaf(__uint_as_float(s[e + 1]), p.sl2, -m));
              a2 += ex2(fmaf(__uint_as_float(s[e + 2]), p.sl2, -m));
              a3 += ex2(fmaf(__uint_as_float(s[e + 3]), p.sl2, -m));
            }
            sum += (a0 + a1) + (a2 + a3);
          } else {
            float a0 = 0.f, a1 = 0.f, a2 = 0.f, a3 = 0.f;
#pragma unroll
            for (int e = 0; e < 32; e += 4) {
              const float4 y = z[8 * c4 + e / 4];
              float x0 = ex2(fmaf(__uint_as_float(s[e]), p.sl2, -y.x));
              float x1 = ex2(fmaf(__uint_as_float(s[e + 1]), p.sl2, -y.y));
              float x2 = ex2(fmaf(__uint_as_float(s[e + 2]), p.sl2, -y.z));
              float x3 = ex2(fmaf(__uint_as_float(s[e + 3]), p.sl2, -y.w));
              if (!full) {
                const int c = 32 * c4 + e;
                if (c < c_lo || c >= c_hi) x0 = 0.f;
                if (c + 1 < c_lo || c + 1 >= c_hi) x1 = 0.f;
                if (c + 2 < c_lo || c + 2 >= c_hi) x2 = 0.f;
                if (c + 3 < c_lo || c + 3 >= c_hi) x3 = 0.f;
              }
              a0 += x0;
              a1 += x1;
              a2 += x2;
              a3 += x3;
            }
            sum += (a0 + a1) + (a2 + a3);
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars->s_empty[2 * wg + buf]);
        ++bc;
      }
      if (!ok) break;
      const size_t bg = static_cast<size_t>(it.b) * p.Hkv + it.g;
      if (PASS == 1) {
        if (a < p.nqt)
          p.stats[(bg * p.splits + it.split) * p.nqt * 128 + a * 128 + r] =
              live ? make_float2(m, sum) : make_float2(0.f, 0.f);
      } else if (live) {
        float* dst = p.weights + bg * p.stride + pos;
        *dst = p.accumulate ? *dst + sum : sum;
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 9) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// Joins pass 1's parts: lse = m + log2(l) of each row, +inf for a row that is not there.
__global__ void __launch_bounds__(256) weights_lse_kernel(const WtParams p) {
  const long long per = static_cast<long long>(p.nqt) * 128, n = per * p.B * p.Hkv;
  const long long i = blockIdx.x * 256LL + threadIdx.x;
  if (i >= n) return;
  const long long bg = i / per, r = i - bg * per;
  const int rows = imin(p.L, wt_len(p, static_cast<int>(bg / p.Hkv)));
  const int c = static_cast<int>(r & 127);
  float lse = INFINITY;
  if (c < p.tpt * p.G && (r >> 7) * p.tpt + c / p.G < rows) {
    const float2* s = p.stats + bg * p.splits * per + r;
    float m = -1.7e38f, l = 0.f;
    for (int k = 0; k < p.splits; ++k) m = fmaxf(m, s[k * per].x);
    for (int k = 0; k < p.splits; ++k) l += s[k * per].y * ex2(s[k * per].x - m);
    lse = m + log2f(l);
  }
  p.lse[i] = lse;
}
