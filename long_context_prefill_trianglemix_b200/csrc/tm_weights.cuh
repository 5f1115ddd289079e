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
// warpgroups, one per A tile and 128-column S buffer in TMEM; warp 16 loads by
// TMA; warp 17 issues the MMAs. A warpgroup takes its scores to registers in
// halves, so the next MMA into its buffer runs while it reduces the second half
// and the other warpgroups work. A q tile packs floor(128 / G) tokens of all G q
// heads of the group, so short L wastes no rows.
//
// Bound: one exponential per score and pass. At 16 MUFU results a clock and SM a
// 128 x 128 tile takes 1024 clocks, twice its MMA time, so 3 of 8 exponentials
// run on the FMA pipe (ex2x2_quintic). Four warpgroups rather than two hide the
// dependent-issue latency of the reductions.

constexpr int kWtTiles = 4;  // A tiles, reduction warpgroups
constexpr int kWtThreads = 128 * kWtTiles + 64;
constexpr int kWtStages = 2;
constexpr int kWtLse = 8;  // slots of a B tile's lse

__device__ __forceinline__ float fmax3_nan(float a, float b, float c) {
  float d;
  asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

__device__ __forceinline__ void fadd2(float& a0, float& a1, float b0, float b1) {
  asm("{\n\t.reg .b64 a, b;\n\tmov.b64 a, {%0, %1};\n\tmov.b64 b, {%2, %3};\n\t"
      "add.rn.f32x2 a, a, b;\n\tmov.b64 {%0, %1}, a;\n\t}"
      : "+f"(a0), "+f"(a1)
      : "f"(b0), "f"(b1));
}

// 2^x of two values on the FMA pipe, good to 2^-22: x = n + f with n = round(x)
// (through 1.5 * 2^23), the fitted quintic for 2^f in packed FMAs, times 2^n built
// in the exponent field. x is clamped at -126 (2^-126 instead of less); NaN stays.
__device__ __forceinline__ void ex2x2_quintic(float& x0, float& x1) {
  uint32_t ta, tb;
  float p0, p1;
  asm("{\n\t.reg .b64 x, m, t, n, f, p, c;\n\t.reg .f32 u, v;\n\t"
      "max.NaN.f32 u, %4, 0fC2FC0000;\n\t"
      "max.NaN.f32 v, %5, 0fC2FC0000;\n\t"
      "mov.b64 x, {u, v};\n\t"
      "mov.b64 m, {%6, %6};\n\t"
      "add.rn.f32x2 t, x, m;\n\t"
      "sub.rn.f32x2 n, t, m;\n\t"
      "sub.rn.f32x2 f, x, n;\n\t"
      "mov.b64 c, {%7, %7};\n\t"
      "mov.b64 p, {%8, %8};\n\t"
      "fma.rn.f32x2 p, c, f, p;\n\t"
      "mov.b64 c, {%9, %9};\n\t"
      "fma.rn.f32x2 p, p, f, c;\n\t"
      "mov.b64 c, {%10, %10};\n\t"
      "fma.rn.f32x2 p, p, f, c;\n\t"
      "mov.b64 c, {%11, %11};\n\t"
      "fma.rn.f32x2 p, p, f, c;\n\t"
      "mov.b64 c, {%12, %12};\n\t"
      "fma.rn.f32x2 p, p, f, c;\n\t"
      "mov.b64 {%0, %1}, t;\n\t"
      "mov.b64 {%2, %3}, p;\n\t}"
      : "=r"(ta), "=r"(tb), "=f"(p0), "=f"(p1)
      : "f"(x0), "f"(x1), "f"(12582912.0f), "f"(TM_EXP2_P5_C5), "f"(TM_EXP2_P5_C4),
        "f"(TM_EXP2_P5_C3), "f"(TM_EXP2_P5_C2), "f"(TM_EXP2_P5_C1), "f"(TM_EXP2_P5_C0));
  const float sa = __uint_as_float(ta * 8388608u + 0x3F800000u);
  const float sb = __uint_as_float(tb * 8388608u + 0x3F800000u);
  x0 = p0 * sa;
  x1 = p1 * sb;
}

// kWtPoly of every 8 pairs go to the FMA pipe, the others to MUFU.
constexpr int kWtPoly = 3;
__device__ __forceinline__ void wt_exp_pair(int e, float& x0, float& x1) {
  constexpr uint32_t kMask = kWtPoly == 0 ? 0u : kWtPoly == 2 ? 0x22u : kWtPoly == 3 ? 0x4Au : 0xAAu;
  if ((kMask >> ((e >> 1) & 7)) & 1u) {
    ex2x2_quintic(x0, x1);
  } else {
    x0 = ex2(x0);
    x1 = ex2(x1);
  }
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
  int items;
  float sl2;
  const int* lens;
  float2* stats;     // pass 1: (m, l) [B Hkv][splits][nqt * 128]
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
  static constexpr int kBar = kLse + kWtLse * 512;
  static constexpr int kSmem = kBar + 256 + 1024;
};

struct WtBars {
  uint64_t a_full[kWtTiles], a_empty[kWtTiles];
  uint64_t b_full[kWtStages], b_empty[kWtStages];
  uint64_t s_full[kWtTiles], s_empty[kWtTiles];
  uint64_t l_full[kWtLse], l_empty[kWtLse];
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
  const int groups = ((PASS == 1 ? p.nqt : p.nkt) + kWtTiles - 1) / kWtTiles;
  int x = i;
  it.split = 0;
  if (PASS == 1) {
    it.split = x % p.splits;
    x /= p.splits;
  }
  it.a0 = kWtTiles * (x % groups);
  x /= groups;
  it.g = x % p.Hkv;
  it.b = x / p.Hkv;
  it.len = wt_len(p, it.b);
  const int rows = imin(p.L, it.len);
  it.r0 = it.len - rows;
  const int nqt = (rows + p.tpt - 1) / p.tpt;
  if (PASS == 1) {
    it.na = imin(kWtTiles, nqt - it.a0);
    if (it.na <= 0) return false;
    // keys up to the group's last row
    const int last = it.r0 + imin(rows, (it.a0 + kWtTiles) * p.tpt);
    const int nk = (last + BN - 1) / BN;
    it.t0 = static_cast<int>(static_cast<long long>(nk) * it.split / p.splits);
    it.t1 = static_cast<int>(static_cast<long long>(nk) * (it.split + 1) / p.splits);
    return true;  // an empty part still writes its (neutral) statistics
  }
  it.na = imin(kWtTiles, (it.len + BN - 1) / BN - it.a0);
  if (it.na <= 0) return false;
  // q tiles with a row at or after the group's first key
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
  const uint32_t tmem = bars->tmem;
  const uint32_t sA = smem_addr(smem), sB = sA + C::kRing;
  const int q_bytes = p.tpt * p.G * D * 2;

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
        if (PASS == 2 && bc > i) drain_wait(&bars->l_full[i], ((bc - 1 - i) / kWtLse) & 1);
    }
  } else if (warp == 4 * kWtTiles + 1) {
    const bool leader = elect_one();
    uint32_t ac[kWtTiles] = {}, sc[kWtTiles] = {}, bc = 0;
    bool ok = true;
    for (int i = blockIdx.x; i < p.items && ok; i += gridDim.x) {
      WtItem it;
      if (!wt_item<PASS>(p, i, it) || it.t0 >= it.t1) continue;
      for (int t = it.t0; t < it.t1 && ok; ++t) {
        const int st = bc % kWtStages;
        ok = __all_sync(0xffffffffu,
                        wait_bar(&bars->b_full[st], (bc / kWtStages) & 1, abort_flag, kSiteWeights));
#pragma unroll
        for (int w = 0; w < kWtTiles; ++w) {
          if (w >= it.na || !ok) continue;
          bool here = t > it.t0 || wait_bar(&bars->a_full[w], ac[w] & 1, abort_flag, kSiteWeights);
          here = here && wait_bar(&bars->s_empty[w], (sc[w] & 1) ^ 1, abort_flag, kSiteWeights);
          if (!(ok = __all_sync(0xffffffffu, here))) continue;
          tc_fence_after();
          if (leader) {
            issue_qk<D>(tmem + w * 128, desc_lo_sw128(sA + w * C::kTile, 16),
                        desc_lo_sw128(sB + st * C::kTile, 16));
            mma_commit(&bars->s_full[w]);
            if (t + 1 == it.t1) mma_commit(&bars->a_empty[w]);
          }
          __syncwarp();
          ++sc[w];
        }
        if (!ok) break;
        if (leader) mma_commit(&bars->b_empty[st]);
        __syncwarp();
        ++bc;
      }
#pragma unroll
      for (int w = 0; w < kWtTiles; ++w)
        if (w < it.na) ++ac[w];
    }
    if (leader) mma_commit(&bars->mma_done);
    __syncwarp();
    drain_wait(&bars->mma_done, 0);
  } else {
    const int wg = warp >> 2, r = tid & 127;
    const uint32_t lane_addr = static_cast<uint32_t>((warp & 3) * 32) << 16;
    uint32_t bc = 0, sc = 0;  // B tiles of the CTA, scores of this warpgroup
    bool ok = true;
    for (int i = blockIdx.x; i < p.items && ok; i += gridDim.x) {
      WtItem it;
      if (!wt_item<PASS>(p, i, it)) continue;
      if (wg >= it.na) {  // no tile for this warpgroup: it only lets the lse slots go
        for (int t = it.t0; PASS == 2 && t < it.t1 && ok; ++t, ++bc) {
          const int ls = bc % kWtLse;
          ok = __all_sync(0xffffffffu, wait_bar(&bars->l_full[ls], (bc / kWtLse) & 1, abort_flag,
                                                kSiteWeights));
          if (ok && lane == 0) mbar_arrive(&bars->l_empty[ls]);
        }
        continue;
      }
      const int rows = it.len - it.r0;
      const int a = it.a0 + wg;
      // pass 1: this thread's row; pass 2: its key
      const int tok = PASS == 1 ? a * p.tpt + r / p.G : 0;
      const bool live = PASS == 1 ? (r < p.tpt * p.G && tok < rows) : a * BN + r < it.len;
      const bool warp_live = __any_sync(0xffffffffu, live);
      const int pos = PASS == 1 ? it.r0 + tok : a * BN + r;
      const uint32_t ts = tmem + lane_addr + wg * 128;
      float m = -1.7e38f, sum = 0.f;
      for (int t = it.t0; t < it.t1; ++t, ++bc, ++sc) {
        const int ls = bc % kWtLse;
        bool here = wait_bar(&bars->s_full[wg], sc & 1, abort_flag, kSiteWeights);
        if (PASS == 2)
          here = here && wait_bar(&bars->l_full[ls], (bc / kWtLse) & 1, abort_flag, kSiteWeights);
        if (!(ok = __all_sync(0xffffffffu, here))) break;
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
        const float4* z = reinterpret_cast<const float4*>(smem + C::kLse + ls * 512);
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
          float a0 = 0.f, a1 = 0.f, a2 = 0.f, a3 = 0.f;
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
#pragma unroll
            for (int c = 0; c < 2; ++c)
#pragma unroll
              for (int e = 0; e < 32; e += 4) {
                float x[4];
                ffma2(x[0], x[1], __uint_as_float(s[c][e]), __uint_as_float(s[c][e + 1]), p.sl2, p.sl2,
                      -m, -m);
                ffma2(x[2], x[3], __uint_as_float(s[c][e + 2]), __uint_as_float(s[c][e + 3]), p.sl2,
                      p.sl2, -m, -m);
                wt_exp_pair(e, x[0], x[1]);
                wt_exp_pair(e + 2, x[2], x[3]);
                fadd2(a0, a1, x[0], x[1]);
                fadd2(a2, a3, x[2], x[3]);
              }
          } else if (full) {
#pragma unroll
            for (int c = 0; c < 2; ++c)
#pragma unroll
              for (int e = 0; e < 32; e += 4) {
                const float4 y = z[16 * h + 8 * c + e / 4];
                float x[4];
                ffma2(x[0], x[1], __uint_as_float(s[c][e]), __uint_as_float(s[c][e + 1]), p.sl2, p.sl2,
                      y.x, y.y);
                ffma2(x[2], x[3], __uint_as_float(s[c][e + 2]), __uint_as_float(s[c][e + 3]), p.sl2,
                      p.sl2, y.z, y.w);
                wt_exp_pair(e, x[0], x[1]);
                wt_exp_pair(e + 2, x[2], x[3]);
                fadd2(a0, a1, x[0], x[1]);
                fadd2(a2, a3, x[2], x[3]);
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
          sum += (a0 + a1) + (a2 + a3);
        }
        if (PASS == 2) {
          __syncwarp();
          if (lane == 0) mbar_arrive(&bars->l_empty[ls]);
        }
      }
      if (!ok) break;
      const size_t bg = static_cast<size_t>(it.b) * p.Hkv + it.g;
      if (PASS == 1) {
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
  if (warp == 4 * kWtTiles + 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 128 * kWtTiles);
  }
}

// Joins pass 1's parts: -(m + log2(l)) of each row, -inf for a row that is not there.
__global__ void __launch_bounds__(256) weights_lse_kernel(const WtParams p) {
  const long long per = static_cast<long long>(p.nqt) * 128, n = per * p.B * p.Hkv;
  const long long i = blockIdx.x * 256LL + threadIdx.x;
  if (i >= n) return;
  const long long bg = i / per, r = i - bg * per;
  const int rows = imin(p.L, wt_len(p, static_cast<int>(bg / p.Hkv)));
  const int c = static_cast<int>(r & 127);
  float nlse = -INFINITY;
  if (c < p.tpt * p.G && (r >> 7) * p.tpt + c / p.G < rows) {
    const float2* s = p.stats + bg * p.splits * per + r;
    float m = -1.7e38f, l = 0.f;
    for (int k = 0; k < p.splits; ++k) m = fmaxf(m, s[k * per].x);
    for (int k = 0; k < p.splits; ++k) l += s[k * per].y * ex2(s[k * per].x - m);
    nlse = -(m + log2f(l));
  }
  p.nlse[i] = nlse;
}
