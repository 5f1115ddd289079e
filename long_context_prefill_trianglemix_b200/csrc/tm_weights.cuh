// Attention weight of each key from the last queries of a prompt: for batch b,
// kv head g and key j,
//
//   w_j = sum over the rows i in [len - L, len), i >= j, and the q heads h of
//         the group, of  p_ihj = softmax_j(scale q_ih . k_j)  (causal).
//
// The denominators need a whole row before any weight is known, and the
// probabilities (L N per head) are too many to keep, so the products are formed
// twice: pass 1 for each row's log-sum-exp, pass 2 for the sums. Both are the
// same pipeline, C = A B^T with up to four stationary 128-row A tiles and a
// stream of 128-row B tiles, and both reduce along their own TMEM lane only:
//   pass 1  A = q rows, B = keys: a thread owns a row, running max and sum;
//   pass 2  A = keys, B = q rows: a thread owns a key and adds 2^(s - lse_row).
// Included by tm_attn.cu inside namespace trimix (status word, bounded waits,
// tensor-core helpers).
//
// CTA (576 threads, one per SM, persistent): warps 0-15 are four reduction
// warpgroups, each with a 128-column S buffer in TMEM; warp 16 loads by TMA; warp
// 17 issues the MMAs. With four A tiles an item each warpgroup has one; with fewer
// the warpgroups of a tile take its B tiles in turn (phases). A warpgroup takes its
// scores to registers in halves, so the next MMA into its buffer runs while it
// reduces the second half and the other warpgroups work. A q tile packs
// floor(128 / G) tokens of all G q heads of the group, so short L wastes no rows.
// Where G does not divide 128 the rest of a q tile is no row: pass 2 then goes through
// every tile with bounds, as through the diagonal and the last tile, because zeros in
// its place would turn an infinite key into NaN.
//
// Bound: one exponential per score and pass. At 16 MUFU results a clock and SM a
// 128 x 128 tile takes 1024 clocks, twice its MMA time, so 2 of 8 exponentials
// run on the FMA pipe (ex2x2_quintic). Four warpgroups rather than two hide the
// dependent-issue latency of the reductions. Measured: 131072 keys, the last 256
// queries, 32 q and 8 kv heads, D = 128: 560 us (2 x 275 GFLOP, 0.98 PFLOP/s; 1.07 G
// exponentials a pass, 231 us of MUFU alone at 1965 MHz), 625 to 670 us under the
// power cap of a long run. 28 q and 4 kv heads (bounds, all exponentials on MUFU in
// pass 2) 672 us where 32 and 4 take 550.

constexpr int kWtTiles = 4;  // A tiles, reduction warpgroups
constexpr int kWtThreads = 128 * kWtTiles + 64;
constexpr int kWtStages = 2;
constexpr int kWtLse = 8;  // slots of a B tile's lse

__device__ __forceinline__ float fmax3_nan(float a, float b, float c) {
  float d;
  asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

// A constant in both halves, opaque to the compiler: it stays in a register pair
// instead of being moved there again for every use.
__device__ __forceinline__ F2 both(float c) {
  F2 r;
  asm volatile("mov.b64 %0, {%1, %1};" : "=l"(r) : "f"(c));
  return r;
}

struct Quintic {
  F2 magic, minus_magic, minus_one, c0, c1, c2, c3, c4, c5;
};
__device__ __forceinline__ Quintic quintic() {
  Quintic k;
  k.magic = both(12582912.0f);  // 1.5 * 2^23
  k.minus_magic = both(-12582912.0f);
  k.minus_one = both(-1.0f);
  k.c0 = both(TM_EXP2_P5_C0); k.c1 = both(TM_EXP2_P5_C1); k.c2 = both(TM_EXP2_P5_C2);
  k.c3 = both(TM_EXP2_P5_C3); k.c4 = both(TM_EXP2_P5_C4); k.c5 = both(TM_EXP2_P5_C5);
  return k;
}

// 2^x of two values on the FMA pipe, good to 2^-22: x = n + f with n = round(x)
// (through 1.5 * 2^23), the fitted quintic for 2^f in packed FMAs, times 2^n built
// in the exponent field. x is clamped at -126 (2^-126 instead of less); NaN stays.
__device__ __forceinline__ F2 ex2x2_quintic(const Quintic& k, F2 x) {
  float xa, xb;
  unpack2(x, xa, xb);
  asm("max.NaN.f32 %0, %0, 0fC2FC0000;" : "+f"(xa));
  asm("max.NaN.f32 %0, %0, 0fC2FC0000;" : "+f"(xb));
  x = pack2(xa, xb);
  const F2 t = add2(x, k.magic);
  const F2 n = add2(t, k.minus_magic);
  const F2 f = fma2(n, k.minus_one, x);
  F2 p = fma2(k.c5, f, k.c4);
  p = fma2(p, f, k.c3);
  p = fma2(p, f, k.c2);
  p = fma2(p, f, k.c1);
  p = fma2(p, f, k.c0);
  float ta, tb;
  unpack2(t, ta, tb);
  return mul2(p, pack2(__float_as_uint(ta) * 8388608u + 0x3F800000u,
                       __float_as_uint(tb) * 8388608u + 0x3F800000u));
}

// Two of every 8 pairs go to the FMA pipe, the others to MUFU. The 131072-key case
// with 0, 1, 2, 3 and 4 of them: 625, 575, 560, 576-595 and 627-654 us.
__device__ __forceinline__ F2 wt_exp_pair(const Quintic& k, int e, F2 x) {
  constexpr uint32_t kMask = 0x22u;
  if ((kMask >> ((e >> 1) & 7)) & 1u) return ex2x2_quintic(k, x);
  float a, b;
  unpack2(x, a, b);
  return pack2(ex2(a), ex2(b));
}

struct WtItem {
  int b, g;     // batch, kv head
  int a0, na;   // first A tile (q tile in pass 1, key tile in pass 2) and how many
  int t0, t1;   // B tiles
  int len, r0;  // tokens of the sequence, its first row
  int split;
};

struct WtParams {
  int B, Hq, Hkv, N, G, L;
  int tpt;           // tokens of a q tile
  int nqt, nkt;      // q tiles, key tiles (of the longest sequence)
  int splits;        // pass 1: parts of the key range
  int items, group;  // A tiles of an item: 1, 2 or 4; 4 / group phases
  int parts;         // splits * phases of pass 1
  float sl2;
  const int* lens;
  float2* stats;     // pass 1: (m, l) [B Hkv][splits * phases of pass 1][nqt * 128]
  float* nlse;       // minus the rows' log-sum-exps [B Hkv][nqt * 128], -inf where there is no row
  float* weights;
  long long stride;
  int accumulate;
};

template <int D>
struct WtCfg {
  static constexpr int kTile = 128 * D * 2;
  static constexpr int kPanel = 128 * 64 * 2;
  static constexpr int kRing = kWtTiles * kTile;
  static constexpr int kLse = kRing + kWtStages * kTile;
  static constexpr int kSum = kLse + kWtLse * 512;  // pass 2: later phases' sums, 3 x 128 floats
  static constexpr int kBar = kSum + 3 * 512;
  static constexpr int kSmem = kBar + 384 + 1024;
};

struct WtBars {
  uint64_t a_full[kWtTiles], a_empty[kWtTiles];
  uint64_t b_full[kWtStages], b_empty[kWtStages];
  uint64_t s_full[kWtTiles], s_empty[kWtTiles];
  uint64_t l_full[kWtLse], l_empty[kWtLse];
  uint64_t x_full[2], x_empty[2];  // [A tile]: the sums above
  uint64_t j_full;                 // the joined statistics
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
  const int groups = ((PASS == 1 ? p.nqt : p.nkt) + p.group - 1) / p.group;
  int x = i;
  it.split = 0;
  if (PASS == 1) {
    it.split = x % p.splits;
    x /= p.splits;
  }
  it.a0 = p.group * (x % groups);
  x /= groups;
  it.g = x % p.Hkv;
  it.b = x / p.Hkv;
  it.len = wt_len(p, it.b);
  const int rows = imin(p.L, it.len);
  it.r0 = it.len - rows;
  const int nqt = (rows + p.tpt - 1) / p.tpt;
  if (PASS == 1) {
    it.na = imin(p.group, nqt - it.a0);
    if (it.na <= 0) return false;
    // keys up to the group's last row
    const int last = it.r0 + imin(rows, (it.a0 + p.group) * p.tpt);
    const int nk = (last + BN - 1) / BN;
    it.t0 = static_cast<int>(static_cast<long long>(nk) * it.split / p.splits);
    it.t1 = static_cast<int>(static_cast<long long>(nk) * (it.split + 1) / p.splits);
    return true;  // an empty part still writes its (neutral) statistics
  }
  it.na = imin(p.group, (it.len + BN - 1) / BN - it.a0);
  if (it.na <= 0) return false;
  // q tiles with a row at or after the group's first key
  it.t0 = imax(0, (it.a0 * BN - it.r0) / p.tpt);
  it.t1 = nqt;
  return true;
}

// Joins parts j, j + step, ... of a row's statistics (`per` apart), F loads at a time.
template <int F>
__device__ __forceinline__ void wt_join(const WtParams& p, const float2* s, long long per, int j,
                                        int step, float& m, float& l) {
  m = -1.7e38f;
  l = 0.f;
  for (int k0 = j; k0 < p.parts; k0 += F * step) {
    float2 v[F];
#pragma unroll
    for (int u = 0; u < F; ++u)
      v[u] = k0 + step * u < p.parts ? s[(k0 + step * u) * per] : make_float2(-1.7e38f, 0.f);
#pragma unroll
    for (int u = 0; u < F; ++u) {
      const float mn = fmax3_nan(m, v[u].x, v[u].x);
      l = l * ex2(m - mn) + v[u].y * ex2(v[u].x - mn);
      m = mn;
    }
  }
}

// Whether row x of the q tiles of a sequence of len tokens is one.
__device__ __forceinline__ bool wt_there(const WtParams& p, int len, int x) {
  const int c = x & 127;
  return c < p.tpt * p.G && (x >> 7) * p.tpt + c / p.G < imin(p.L, len);
}

// JOIN (pass 2): the statistics of a kv head's rows are joined from pass 1's parts by
// the reducing warps, into the memory of the lse slots; at most kWtLse q tiles, and one
// item a CTA. Without it weights_lse_kernel does so in between.
template <int D, int PASS, bool JOIN = false>
__global__ void __launch_bounds__(kWtThreads, 1)
    weights_kernel(const __grid_constant__ CUtensorMap tq, const __grid_constant__ CUtensorMap tk,
                   const __grid_constant__ WtParams p) {
  using C = WtCfg<D>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = align1024(smem_raw);
  WtBars* bars = reinterpret_cast<WtBars*>(smem + C::kBar);
  volatile int* abort_flag = &bars->abort_flag;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  // Rows that a q tile's box does not cover stay zero (the q tiles are the A tiles in
  // pass 1 and the ring in pass 2).
  const int q_rows = p.tpt * p.G, q_tiles = PASS == 1 ? kWtTiles : kWtStages;
  for (int i = tid; i < (128 - q_rows) * 8 * (D / 64) * q_tiles; i += kWtThreads) {
    const int panel = i / ((128 - q_rows) * 8), x = i - panel * (128 - q_rows) * 8;
    reinterpret_cast<uint4*>(smem + (PASS == 1 ? 0 : C::kRing) + panel * C::kPanel + q_rows * 128)[x] =
        make_uint4(0, 0, 0, 0);
  }
  if (tid == 0) {
    for (int i = 0; i < kWtTiles; ++i) {
      mbar_init(&bars->a_full[i], 1);
      mbar_init(&bars->a_empty[i], 1);
      mbar_init(&bars->s_full[i], 1);
      mbar_init(&bars->s_empty[i], 4);
    }
    for (int i = 0; i < kWtStages; ++i) {
      mbar_init(&bars->b_full[i], 1);
      mbar_init(&bars->b_empty[i], 1);
    }
    for (int i = 0; i < kWtLse; ++i) {
      mbar_init(&bars->l_full[i], 1);
      mbar_init(&bars->l_empty[i], 4 * kWtTiles);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&bars->x_full[i], 4 * (kWtTiles / p.group > 1 ? kWtTiles / p.group - 1 : 1));
      mbar_init(&bars->x_empty[i], 4);
    }
    mbar_init(&bars->j_full, 4 * kWtTiles);
    mbar_init(&bars->mma_done, 1);
    bars->abort_flag = 0;
    fence_barrier_init();
  }
  fence_proxy_async_smem();
  if (warp == 4 * kWtTiles + 1) {
    tmem_alloc(&bars->tmem, 128 * kWtTiles);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  pdl_launch();
  pdl_wait();
  const uint32_t tmem = bars->tmem;
  const uint32_t sA = smem_addr(smem), sB = sA + C::kRing;
  const int q_bytes = q_rows * D * 2;

  if (warp == 4 * kWtTiles) {
    if (lane == 0) {
      tma_prefetch_desc(&tq);
      tma_prefetch_desc(&tk);
      uint32_t ac[kWtTiles] = {}, bc = 0;
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
#pragma unroll
        for (int w = 0; w < kWtTiles; ++w) {
          if (w >= it.na || !ok) continue;
          if (!(ok = wait_bar(&bars->a_empty[w], (ac[w] & 1) ^ 1, abort_flag, kSiteWeights))) continue;
          mbar_arrive_expect_tx(&bars->a_full[w], PASS == 1 ? q_bytes : C::kTile);
          if (PASS == 1)
            load_q(sA + w * C::kTile, &bars->a_full[w], it, it.a0 + w);
          else
            load_k(sA + w * C::kTile, &bars->a_full[w], it, it.a0 + w);
          ++ac[w];
        }
        if (!ok) break;
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
            if (JOIN) {
              ++bc;
              continue;
            }
            const int ls = bc % kWtLse;
            if (!(ok = wait_bar(&bars->l_empty[ls], ((bc / kWtLse) & 1) ^ 1, abort_flag,
                                kSiteWeights))) {
              ++bc;
              break;
            }
            mbar_arrive_expect_tx(&bars->l_full[ls], 512);
            bulk_load(smem_addr(smem + C::kLse + ls * 512),
                      p.nlse + (static_cast<size_t>(it.b * p.Hkv + it.g) * p.nqt + t) * 128, 512,
                      &bars->l_full[ls]);
          }
          ++bc;
        }
      }
      // Let the copies in flight land before the memory goes away (they have, unless a wait gave up).
#pragma unroll
      for (int w = 0; w < kWtTiles; ++w)
        if (ac[w] > 0) drain_wait(&bars->a_full[w], (ac[w] - 1) & 1);
      for (uint32_t i = 0; i < kWtStages; ++i)
        if (bc > i) drain_wait(&bars->b_full[i], ((bc - 1 - i) / kWtStages) & 1);
      for (uint32_t i = 0; i < kWtLse; ++i)
        if (PASS == 2 && !JOIN && bc > i) drain_wait(&bars->l_full[i], ((bc - 1 - i) / kWtLse) & 1);
    }
  } else if (warp == 4 * kWtTiles + 1) {
    const bool leader = elect_one();
    uint32_t a_par = 0, s_par = 0, bc = 0;  // phase bits of the A tiles and S buffers
    const int phases = kWtTiles / p.group;
    bool ok = true;
    for (int i = blockIdx.x; i < p.items && ok; i += gridDim.x) {
      WtItem it;
      if (!wt_item<PASS>(p, i, it) || it.t0 >= it.t1) continue;
      for (int t = it.t0; t < it.t1 && ok; ++t) {
        const int w0 = ((t - it.t0) & (phases - 1)) * p.group;  // first warpgroup of the phase
        const int st = bc % kWtStages;
        ok = __all_sync(0xffffffffu,
                        wait_bar(&bars->b_full[st], (bc / kWtStages) & 1, abort_flag, kSiteWeights));
        for (int ai = 0; ai < it.na && ok; ++ai) {
          const int w = w0 + ai;
          bool here = t > it.t0 || wait_bar(&bars->a_full[ai], (a_par >> ai) & 1, abort_flag, kSiteWeights);
          here = here && wait_bar(&bars->s_empty[w], ((s_par >> w) & 1) ^ 1, abort_flag, kSiteWeights);
          if (!(ok = __all_sync(0xffffffffu, here))) break;
          tc_fence_after();
          if (leader) {
            issue_qk<D>(tmem + w * 128, desc_lo_sw128(sA + ai * C::kTile, 16),
                        desc_lo_sw128(sB + st * C::kTile, 16));
            mma_commit(&bars->s_full[w]);
            if (t + 1 == it.t1) mma_commit(&bars->a_empty[ai]);
          }
          __syncwarp();
          s_par ^= 1u << w;
        }
        if (!ok) break;
        if (leader) mma_commit(&bars->b_empty[st]);
        __syncwarp();
        ++bc;
      }
      a_par ^= (1u << it.na) - 1u;
    }
    if (leader) mma_commit(&bars->mma_done);
    __syncwarp();
    drain_wait(&bars->mma_done, 0);
  } else {
    const int wg = warp >> 2, r = tid & 127;
    const uint32_t lane_addr = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const Quintic kq = quintic();
    const F2 sl2 = both(p.sl2);
    uint32_t bc = 0, sc = 0, xc = 0;  // B tiles of the CTA, scores and items of this warpgroup
    const int phases = kWtTiles / p.group, ai = wg & (p.group - 1), phase = wg / p.group;
    bool ok = true;
    // another's B tile: only let its lse slot go
    auto pass_over = [&](uint32_t n) {
      if (JOIN) return true;
      const int ls = n % kWtLse;
      const bool here = __all_sync(
          0xffffffffu, wait_bar(&bars->l_full[ls], (n / kWtLse) & 1, abort_flag, kSiteWeights));
      if (here && lane == 0) mbar_arrive(&bars->l_empty[ls]);
      return here;
    };
    for (int i = blockIdx.x; i < p.items && ok; i += gridDim.x) {
      WtItem it;
      if (!wt_item<PASS>(p, i, it)) continue;
      if (PASS == 2 && JOIN) {
        // The item's (the CTA's only one's) kv head: each of the 16 warps joins some of its rows.
        const long long per = static_cast<long long>(p.nqt) * 128;
        const float2* st = p.stats + (static_cast<long long>(it.b) * p.Hkv + it.g) * p.parts * per;
        float* table = reinterpret_cast<float*>(smem + C::kLse);
        for (int x = tid; x < p.nqt * 128; x += 128 * kWtTiles) {
          float m, l;
          wt_join<8>(p, st + x, per, 0, 1, m, l);
          table[x] = wt_there(p, it.len, x) ? -(m + log2f(l)) : -INFINITY;
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars->j_full);
        ok = __all_sync(0xffffffffu, wait_bar(&bars->j_full, 0, abort_flag, kSiteWeights));
        if (!ok) break;
      }
      if (ai >= it.na) {  // no A tile for this warpgroup
        for (int t = it.t0; PASS == 2 && t < it.t1 && ok; ++t, ++bc) ok = pass_over(bc);
        continue;
      }
      const int rows = it.len - it.r0;
      const int a = it.a0 + ai;
      // pass 1: this thread's row; pass 2: its key
      const int tok = PASS == 1 ? a * p.tpt + r / p.G : 0;
      const bool live = PASS == 1 ? (r < p.tpt * p.G && tok < rows) : a * BN + r < it.len;
      const bool warp_live = __any_sync(0xffffffffu, live);
      const int pos = PASS == 1 ? it.r0 + tok : a * BN + r;
      const uint32_t ts = tmem + lane_addr + wg * 128;
      float m = -1.7e38f, sum = 0.f;
      for (int t = it.t0; t < it.t1; ++t, ++bc) {
        if (((t - it.t0) & (phases - 1)) != phase) {
          if (PASS == 2 && !(ok = pass_over(bc))) break;
          continue;
        }
        const int ls = bc % kWtLse;
        bool here = wait_bar(&bars->s_full[wg], sc & 1, abort_flag, kSiteWeights);
        if (PASS == 2 && !JOIN)
          here = here && wait_bar(&bars->l_full[ls], (bc / kWtLse) & 1, abort_flag, kSiteWeights);
        if (!(ok = __all_sync(0xffffffffu, here))) break;
        ++sc;
        tc_fence_after();
        // columns [c_lo, c_hi) count for this thread
        int c_lo = 0, c_hi = 128;
        if (PASS == 1) {
          c_hi = imax(0, imin(128, pos + 1 - t * BN));
        } else {
          c_lo = imax(0, imin(128, (pos - (it.r0 + t * p.tpt)) * p.G));
          c_hi = imin(p.tpt, rows - t * p.tpt) * p.G;
        }
        const bool full = __all_sync(0xffffffffu, !live || (c_lo == 0 && c_hi == 128));
        const ulonglong2* z =
            reinterpret_cast<const ulonglong2*>(smem + C::kLse + (JOIN ? t : ls) * 512);
#pragma unroll 1
        for (int h = 0; h < 2; ++h) {
          uint32_t s[2][32];
          tmem_ld32(ts + 64 * h, s[0]);
          tmem_ld32(ts + 64 * h + 32, s[1]);
          tmem_wait_ld(s[0]);
          reg_fence(s[1]);
          if (h == 1) {  // the scores are in registers
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&bars->s_empty[wg]);
          }
          if (!warp_live) continue;
          F2 acc0 = 0, acc1 = 0;  // pairs of zeros
          float a0 = 0.f;
          if (PASS == 1) {
            if (!full) {
              const int c_end = c_hi - 64 * h;
#pragma unroll
              for (int c = 0; c < 2; ++c)
#pragma unroll
                for (int e = 0; e < 32; ++e)
                  if (32 * c + e >= c_end) s[c][e] = 0xFF800000u;
            }
            float mx[4];
#pragma unroll
            for (int c = 0; c < 4; ++c) {
              uint32_t* q = &s[c >> 1][16 * (c & 1)];
              mx[c] = __uint_as_float(q[0]);
#pragma unroll
              for (int e = 1; e < 15; e += 2)
                mx[c] = fmax3_nan(mx[c], __uint_as_float(q[e]), __uint_as_float(q[e + 1]));
              mx[c] = fmax3_nan(mx[c], __uint_as_float(q[15]), mx[c]);
            }
            const float mt = fmax3_nan(fmax3_nan(mx[0], mx[1], mx[2]), mx[3], mx[3]) * p.sl2;
            const float mn = fmax3_nan(m, mt, mt);
            sum *= ex2(m - mn);
            m = mn;
            const F2 minus_m = pack2(-m, -m);
#pragma unroll
            for (int c = 0; c < 2; ++c)
#pragma unroll
              for (int e = 0; e < 32; e += 4) {
                const F2 x = fma2(pack2(s[c][e], s[c][e + 1]), sl2, minus_m);
                const F2 y = fma2(pack2(s[c][e + 2], s[c][e + 3]), sl2, minus_m);
                acc0 = add2(acc0, wt_exp_pair(kq, e, x));
                acc1 = add2(acc1, wt_exp_pair(kq, e + 2, y));
              }
          } else if (full) {
#pragma unroll
            for (int c = 0; c < 2; ++c)
#pragma unroll
              for (int e = 0; e < 32; e += 4) {
                const ulonglong2 nl = z[16 * h + 8 * c + e / 4];
                const F2 x = fma2(pack2(s[c][e], s[c][e + 1]), sl2, nl.x);
                const F2 y = fma2(pack2(s[c][e + 2], s[c][e + 3]), sl2, nl.y);
                acc0 = add2(acc0, wt_exp_pair(kq, e, x));
                acc1 = add2(acc1, wt_exp_pair(kq, e + 2, y));
              }
          } else {
            const int lo = c_lo - 64 * h, end = c_hi - 64 * h;
#pragma unroll
            for (int c = 0; c < 2; ++c) {
              if (32 * c >= end) continue;
#pragma unroll
              for (int e = 0; e < 32; ++e) {
                const float y = reinterpret_cast<const float*>(z)[64 * h + 32 * c + e];
                const float x = fmaf(__uint_as_float(s[c][e]), p.sl2, y);
                a0 += ex2(32 * c + e >= lo && 32 * c + e < end ? x : -INFINITY);
              }
            }
          }
          float r0, r1;
          unpack2(add2(acc0, acc1), r0, r1);
          sum += r0 + r1 + a0;
        }
        if (PASS == 2 && !JOIN) {
          __syncwarp();
          if (lane == 0) mbar_arrive(&bars->l_empty[ls]);
        }
      }
      if (!ok) break;
      const size_t bg = static_cast<size_t>(it.b) * p.Hkv + it.g;
      if (PASS == 1) {
        p.stats[(bg * p.parts + it.split * phases + phase) * p.nqt * 128 + a * 128 + r] =
            live ? make_float2(m, sum) : make_float2(0.f, 0.f);
        continue;
      }
      if (phases > 1) {  // the first phase adds the others' sums, in order
        float* xs = reinterpret_cast<float*>(smem + C::kSum);
        if (phase > 0) {
          ok = __all_sync(0xffffffffu,
                          wait_bar(&bars->x_empty[ai], (xc & 1) ^ 1, abort_flag, kSiteWeights));
          if (!ok) break;
          xs[((phase - 1) * p.group + ai) * 128 + r] = sum;
          __syncwarp();
          if (lane == 0) mbar_arrive(&bars->x_full[ai]);
        } else {
          ok = __all_sync(0xffffffffu, wait_bar(&bars->x_full[ai], xc & 1, abort_flag, kSiteWeights));
          if (!ok) break;
          for (int k = 0; k + 1 < phases; ++k) sum += xs[(k * p.group + ai) * 128 + r];
          __syncwarp();
          if (lane == 0) mbar_arrive(&bars->x_empty[ai]);
        }
        ++xc;
      }
      if (live && phase == 0) {
        float* dst = p.weights + bg * p.stride + pos;
        *dst = p.accumulate ? *dst + sum : sum;
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 4 * kWtTiles + 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 128 * kWtTiles);
  }
}

// Joins pass 1's parts: -(m + log2(l)) of each row, -inf for a row that is not there.
// 32 rows a CTA; eight threads a row share its parts and are joined in order.
__global__ void __launch_bounds__(256) weights_lse_kernel(const WtParams p) {
  pdl_launch();
  pdl_wait();
  __shared__ float2 s_part[8][32];
  const long long per = static_cast<long long>(p.nqt) * 128;
  const int x = threadIdx.x & 31, j = threadIdx.x >> 5;
  const long long i = blockIdx.x * 32LL + x, bg = i / per, r = i - bg * per;
  float m, l;
  wt_join<4>(p, p.stats + bg * p.parts * per + r, per, j, 8, m, l);
  s_part[j][x] = make_float2(m, l);
  __syncthreads();
  if (j) return;
  for (int k = 1; k < 8; ++k) {
    const float2 v = s_part[k][x];
    const float mn = fmax3_nan(m, v.x, v.x);
    l = l * ex2(m - mn) + v.y * ex2(v.x - mn);
    m = mn;
  }
  p.nlse[i] = wt_there(p, wt_len(p, static_cast<int>(bg / p.Hkv)), static_cast<int>(r))
                  ? -(m + log2f(l))
                  : -INFINITY;
}
