// Attention of a few query tokens per sequence over the paged 8-bit cache.
//
//   s_rj = scale q_r . k_j,  o_r = sum_j softmax_j(s_r)_j v_j,  j <= len - nq + i
//
// for the rows r = (query i, q head of the group) of a kv head. Reading the
// codes once (2 D bytes a token and kv head) bounds it; everything else is
// arranged so that the loads never wait for anything:
//
// - A unit is 16 or 32 tokens of one (page, head): rows of D codes, contiguous. All
//   units of all sequences and heads form one line, cut into equal parts for
//   the CTAs and again for their warps, so ragged batches are balanced to a
//   unit. A warp walks its part alone, across items, fed by its own ring of TMA
//   loads (its lanes hold where the next 32 to 64 units lie).
// - The codes are the A operand of m16n8k16 products and the (at most 8 NT) rows
//   the n side, so a group of 4 or 8 q heads wastes no matrix work: S^T = K Q^T
//   (16 tokens x 8 rows), O^T += V^T P^T (16 dims x 8 rows). mma.sync and not tcgen05:
//   at 8 rows the products take a tenth of the tensor pipe, and operands that are
//   converted from 8 bits on their way are in registers, not in shared memory. The
//   order of the contraction index is free, so each thread loads 16 contiguous bytes
//   of its token rows and uses them in place; P^T goes from accumulator to operand
//   layout by an 8x8 transpose (movmatrix).
// - Codes become fp16 exactly (int8 by 1024 + u in the low mantissa bits, e4m3 by
//   the conversion instruction). q becomes fp16 after an exact scaling of the
//   row by a power of two that brings its largest element to [2^14, 2^15):
//   fp16's 11 bits hold bf16's 8, and elements below 2^-31 of the largest are
//   rounded by at most 2^-39 of it. Products and sums are fp32.
// - P is fp16, scaled by 2^11 against the running reference and allowed to grow
//   to 2^14.5, and carries V's range over a power of two, a factor of 2^-3 to 2:
//   weights down to 2^-22 of the largest keep fp16's 11 bits (2^-22 2^11 2^-3 is its
//   least normal number; rounding 2^-11 of each weight, below the bf16 output's 2^-8),
//   less ones are off by 2^-33 of the largest. The reference moves only when a score
//   exceeds it by more than 3.5 (log2), the power of two when a range leaves its
//   window, so the usual unit needs one vote and no rescale; m, l and O are fp32.
//
// Parts of an item (sequence, kv head, row tile) that end in one CTA are merged
// there; an item cut between CTAs leaves unnormalised partials (O, m, l) in the
// workspace and combine_kernel joins them in order, so results are reproducible. O is
// a sum of up to 2^14.5 times the item's keys of V's values: a partial takes 2^-s of
// it with 2^s above that, so that V near its type's largest value does not overflow.
// Included by tm_attn.cu inside namespace trimix (status word, bounded waits, TMA
// helpers, tensor-map encoding).

namespace {

using namespace kv8;

constexpr int kWarps = 8;       // of a CTA
constexpr int kMaxAttnBatch = 4096;
constexpr int kMaxSms = 192;    // workspaces are sized for this many
constexpr float kLift = 11.f;   // log2 of the scale of P against the reference
constexpr float kSlack = 3.5f;  // scores may exceed the reference by this
constexpr float kFar = 0x1p-3f;   // P takes a V range in while it is this much of V's reference
constexpr float kFarthest = 0x1p-70f;  // a range this far below the part's largest is taken as 0: O, at
                                       // most 2^55 for 2^31 keys, must not overflow as it is rescaled
constexpr float kLowest = -1.7e38f;

struct AttnP {
  Kv8AttnArgs a;
  int G, rows, RT, items_per_b, page_log;
  long long cap;      // tokens a sequence can hold
  float* part_o;      // [2 grid][8 NT][D]
  float2* part_ml;    // [2 grid][8 NT]
  float* warp_o;      // [grid][warps][8 NT][D]: a warp's first partial
  int4* close;        // [grid]: the item from an earlier CTA that ends in this one (item, first CTA,
                      // its slot and, above 16 bits, the item's s, last CTA), or -1
  float* lse;         // [items][8 NT] (log2), +inf where a row keeps nothing
  float* scores;      // [items][cap][rs] (log2), or null
  int rs;             // rows kept of a token's scores: those of an item, to a multiple of 4
  int grid;
};

__device__ __forceinline__ int clamp_len(const AttnP& p, int b) {
  return static_cast<int>(min(max(static_cast<long long>(p.a.lens[b]), 0LL), p.cap));
}

// How the line of T units is cut for `grid` CTAs: at least one unit a warp.
__device__ __forceinline__ int parts_of(long long T, int grid, int warps) {
  const long long most = (T + warps - 1) / warps;
  return static_cast<int>(most < grid ? (most < 1 ? 1 : most) : grid);
}

// Where every item is short, at most two warps' shares, none is cut: a boundary that
// falls inside one moves to its start. (Among long items that would unbalance the
// warps: 24 sequences of 327 to 32768 tokens took 57 us so, 51 us cut evenly.)
__device__ __forceinline__ bool whole_items(long long T, int grid, int warps, int longest) {
  return longest * static_cast<long long>(grid) * warps <= 2 * T || longest <= 2;
}

__device__ __forceinline__ int sequence_of(const int* pre, int B, int x) {
  int lo = 0, hi = B;  // the last b with pre[b] <= x
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (pre[mid] <= x) lo = mid; else hi = mid;
  }
  return lo;
}

__device__ __forceinline__ int item_start(const AttnP& p, const int* pre, int x) {
  if (x >= pre[p.a.B]) return x;
  const int b = sequence_of(pre, p.a.B, x);
  return x - (x - pre[b]) % ((pre[b + 1] - pre[b]) / p.items_per_b);
}

__device__ __forceinline__ void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1,
                                         const float (&c)[4]) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%10,%11,%12,%13};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(c[0]), "f"(c[1]), "f"(c[2]),
        "f"(c[3]));
}

__device__ __forceinline__ uint32_t transpose8x8(uint32_t v) {
  uint32_t r;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
  return r;
}

__device__ __forceinline__ uint32_t pack_half(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// Two f16 values of bytes 0, 1 (first) and 2, 3 (second) of a word of codes.
template <int FMT>
__device__ __forceinline__ void widen(uint32_t w, uint32_t& first, uint32_t& second) {
  if (FMT == TM_KV_INT8) {
    const uint32_t u = w ^ 0x80808080u;  // code + 128, 0..255
    const __half2 bias = __half2half2(__ushort_as_half(0x6480));  // 1024 + 128
    const uint32_t x = __byte_perm(u, 0x64646464u, 0x4140), y = __byte_perm(u, 0x64646464u, 0x4342);
    const __half2 hx = __hsub2(*reinterpret_cast<const __half2*>(&x), bias);
    const __half2 hy = __hsub2(*reinterpret_cast<const __half2*>(&y), bias);
    first = *reinterpret_cast<const uint32_t*>(&hx);
    second = *reinterpret_cast<const uint32_t*>(&hy);
  } else {
    asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\t"
        "cvt.rn.f16x2.e4m3x2 %0, l;\n\tcvt.rn.f16x2.e4m3x2 %1, h;\n\t}"
        : "=r"(first), "=r"(second)
        : "r"(w));
  }
}

// UT tiles of 16 tokens make a unit. Two halve what a unit costs besides its codes but
// need registers or shared memory that one row tile of D = 128 has a better use for:
// 16 warps an SM with one tile each took 338 us where 12 with two took 350 (8 sequences
// of 131072 tokens, e4m3). Under a sustained load the power cap brings the clock to
// 1.5 to 1.6 GHz, where the conversions of int8 bound this kernel (340 to 378 us by what
// the box's cap leaves, 6.3 to 5.7 TB/s; e4m3 338 us, 6.4 TB/s) and memory does not; in
// short runs both take 320 us (6.7 TB/s).
// Each warp has a ring of S units (K rows, then V rows, 128-byte swizzled by the TMA
// load): one unit loads while another is computed; more in flight is slower (three deep
// 347 us, two deep 324 in short runs).
template <int D, int NT, int UT>
struct AttnCfg {
  static constexpr int kCtas = NT == 1 ? 2 : 1;  // an SM, 128 and 255 registers a thread
  static constexpr int kThreads = 32 * kWarps;
  static constexpr int kUnit = 16 * UT;
  static constexpr int kHalf = kUnit * D;  // bytes of a unit's K or V
  static constexpr int S = kHalf == 1024 ? 4 : 2;
  static constexpr int kWarpRing = S * 2 * kHalf;
  static constexpr int kMl = kWarps * kWarpRing;  // float2 [2 warps][8 NT]
  static constexpr int kBar = kMl + 2 * kWarps * 8 * NT * 8;
  static constexpr int kItem = kBar + kWarps * S * 8;
  static constexpr int kPre = kItem + 2 * kWarps * 4 + 16;  // int [B + 1]
  static constexpr int kSmem = kPre + 16 + 1024;            // + 4 B, alignment slack
  static_assert(8 * NT * D * 4 <= kWarpRing, "a partial must fit a warp's ring");
};

// Where one lane's unit of the line lies.
struct UnitAt {
  int item, u;
  int row;       // TMA row of the unit, -1 if its page is not there
  float kr, vr;  // its ranges; kr is kMissing if its page is not there
};
constexpr float kMissing = -1.f;  // ranges are >= 0

template <int D, int UT>
__device__ __forceinline__ UnitAt locate(const AttnP& p, const int* pre, int x, int xe) {
  UnitAt at;
  at.item = -1; at.u = 0; at.row = -1;
  at.kr = kMissing;
  at.vr = 0.f;
  if (x >= xe) return at;
  const int lo = sequence_of(pre, p.a.B, x);
  const int U = (pre[lo + 1] - pre[lo]) / p.items_per_b;
  const int it = (x - pre[lo]) / U;
  at.u = x - pre[lo] - it * U;
  at.item = lo * p.items_per_b + it;
  const int tok0 = at.u * 16 * UT;
  const int page = p.a.table[static_cast<long long>(lo) * p.a.max_pages + (tok0 >> p.page_log)];
  if (static_cast<unsigned>(page) < static_cast<unsigned>(p.a.c.num_pages)) {
    const long long block = static_cast<long long>(page) * p.a.c.Hkv + it / p.RT;
    at.row = static_cast<int>(((block << p.page_log) + (tok0 & (p.a.c.page - 1))) / (128 / D));
  }
  return at;
}

template <int D>
__device__ __forceinline__ void load_ranges(const AttnP& p, UnitAt& at) {
  if (at.row < 0) return;
  const long long block = (static_cast<long long>(at.row) * (128 / D)) >> p.page_log;
  at.kr = p.a.c.k_range[block];
  at.vr = p.a.c.v_range[block];
}

// Prefix sums of the sequences' units (times items per sequence) in shared memory;
// returns the units of the longest.
template <int W, int UT>
__device__ __forceinline__ int unit_prefix(const AttnP& p, int* pre) {
  __shared__ int s_warp[W], s_most[W];
  int most = 0;
  const int t = threadIdx.x, lane = t & 31, w = t >> 5;
  int carry = 0;
  for (int b0 = 0; b0 < p.a.B; b0 += 32 * W) {
    const int b = b0 + t;
    const int U = b < p.a.B ? (clamp_len(p, b) + 16 * UT - 1) / (16 * UT) : 0;
    most = max(most, U);
    int x = U * p.items_per_b;
    const int own = x;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x += y;
    }
    if (lane == 31) s_warp[w] = x;
    __syncthreads();
    int before = carry;
    for (int i = 0; i < W; ++i) {
      if (i < w) before += s_warp[i];
      carry += s_warp[i];
    }
    if (b < p.a.B) pre[b] = before + x - own;
    __syncthreads();
  }
  most = __reduce_max_sync(0xffffffffu, most);
  if (lane == 0) s_most[w] = most;
  if (t == 0) pre[p.a.B] = carry;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < W; ++i) most = max(most, s_most[i]);
  return most;
}

// The exponent s above for an item of U units of `unit` tokens (20 to 47), and 2^s.
__device__ __forceinline__ int sum_bits(int U, int unit) {
  return 47 - __clz(static_cast<unsigned>(U) * static_cast<unsigned>(unit));
}
__device__ __forceinline__ float power_of_two(int s) {
  return __uint_as_float(static_cast<uint32_t>(s + 127) << 23);
}

__device__ __forceinline__ void store_bf16(uint16_t* dst, float a, float b) {
  *reinterpret_cast<uint32_t*>(dst) = sm100::pack_bf16x2(a, b);
}

template <int D>
__device__ __forceinline__ uint16_t* out_row(const AttnP& p, int b, int h, int r) {
  const int i = r / p.G;
  return static_cast<uint16_t*>(p.a.o) +
         ((static_cast<long long>(b) * p.a.nq + i) * p.a.Hq + h * p.G + (r - i * p.G)) * D;
}

template <int D, int FMT, int NT, int UT>
__global__ void __launch_bounds__(AttnCfg<D, NT, UT>::kThreads, AttnCfg<D, NT, UT>::kCtas)
    attn_kernel8(const __grid_constant__ CUtensorMap tk, const __grid_constant__ CUtensorMap tv,
                 const __grid_constant__ AttnP p) {
  using C = AttnCfg<D, NT, UT>;
  constexpr int S = C::S, W = kWarps;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = align1024(smem_raw);
  float2* s_ml = reinterpret_cast<float2*>(smem + C::kMl);
  int* s_item = reinterpret_cast<int*>(smem + C::kItem);  // item of the slot's partial, or -1
  volatile int* abort_flag = s_item + 2 * W;
  int* pre = reinterpret_cast<int*>(smem + C::kPre);
  const Kv8AttnArgs& a = p.a;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::kBar) + warp * S;
  pdl_launch();
  if (tid < 2 * W) s_item[tid] = -1;
  if (tid == 0) {
    *abort_flag = 0;
    tma_prefetch_desc(&tk);
    tma_prefetch_desc(&tv);
  }
  if (lane == 0)
    for (int i = 0; i < S; ++i) mbar_init(&bars[i], 1);
  if (lane == 0) fence_barrier_init();
  pdl_wait();
  const int longest = unit_prefix<W, UT>(p, pre);
  const long long T = pre[a.B];
  const int parts = parts_of(T, p.grid, W), cta = blockIdx.x;
  for (int z = cta; z < a.B; z += gridDim.x) {  // sequences without tokens: zeros
    if (pre[z + 1] != pre[z]) continue;
    uint4* o = reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.o) +
                                        static_cast<long long>(z) * a.nq * a.Hq * D);
    for (int i = tid; i < a.nq * a.Hq * (D / 8); i += C::kThreads) o[i] = make_uint4(0, 0, 0, 0);
  }
  if (cta >= parts) {
    if (tid == 0) p.close[cta] = make_int4(-1, 0, 0, 0);
    return;
  }
  // the CTA's part [cs, ce) and this warp's [xs, xe): lanes 0, 1, 2, 3 look up one bound each
  const bool whole = whole_items(T, p.grid, W, longest);
  int cs, ce, xs, xe;
  {
    const int c0 = static_cast<int>(T * cta / parts), c1 = static_cast<int>(T * (cta + 1) / parts);
    const long long w = warp + (lane & 1);
    const int x = (lane & 2) ? c0 + static_cast<int>((c1 - c0) * w / W) : (lane & 1) ? c1 : c0;
    const int at = whole ? item_start(p, pre, x) : x;
    cs = __shfl_sync(0xffffffffu, at, 0);
    ce = __shfl_sync(0xffffffffu, at, 1);
    xs = __shfl_sync(0xffffffffu, at, 2);
    xe = __shfl_sync(0xffffffffu, at, 3);
  }
  const int n_units = xe - xs;
  const float s_unit = a.scale * 1.4426950408889634f / full<FMT>();
  uint8_t* ring = smem + warp * C::kWarpRing;
  const uint32_t ring_addr = smem_addr(ring);

  // Lane i & 31 holds where unit i lies; the next 32 are looked up a batch ahead.
  UnitAt cur = locate<D, UT>(p, pre, xs + lane, xe), nxt = cur;
  const uint64_t policy = evict_first();  // leaves L2 to the scores
  auto issue = [&](int i, int batch) {
    if (i >= n_units || lane != (i & 31)) return;
    const int row = (i >> 5) == batch ? cur.row : nxt.row;
    const int st = i % S;
    uint64_t* bar = &bars[st];
    if (row < 0) {
      mbar_arrive(bar);
      return;
    }
    mbar_arrive_expect_tx(bar, 2 * C::kHalf);
    tma_load_2d(ring_addr + st * 2 * C::kHalf, &tk, bar, 0, row, policy);
    tma_load_2d(ring_addr + st * 2 * C::kHalf + C::kHalf, &tv, bar, 0, row, policy);
  };
  for (int i = 0; i < S - 1; ++i) issue(i, 0);
  load_ranges<D>(p, cur);
  nxt = locate<D, UT>(p, pre, xs + 32 + lane, xe);
  load_ranges<D>(p, nxt);
  if (tid == 0) {
    // does the item that holds the part's first unit begin before it and end in it?
    int4 rec = make_int4(-1, 0, 0, 0);
    if (ce > cs && item_start(p, pre, cs) < cs) {
      const int sb = sequence_of(pre, a.B, cs), U0 = item_start(p, pre, cs);
      const int U = (pre[sb + 1] - pre[sb]) / p.items_per_b;
      if (U0 + U <= ce) {
        // the part that holds unit U0: the last c with floor(c T / parts) <= U0
        const int c0 = static_cast<int>(((U0 + 1LL) * parts - 1) / T);
        rec = make_int4(sb * p.items_per_b + (U0 - pre[sb]) / U, c0,
                        (2 * c0 + (T * c0 / parts < U0)) | sum_bits(U, C::kUnit) << 16, cta);
      }
    }
    p.close[cta] = rec;
  }

  // Byte offsets of this thread's rows in a unit's first tile. K: tokens g and g + 8,
  // 16-byte chunks 2t, 2t + 1 (D = 128) or t; V: tokens 2t, 2t + 1, 2t + 8, 2t + 9, D / 8
  // bytes at g D / 8. All but the 8-byte V loads of D = 64 are free of conflicts.
  uint32_t k_off[2], v_off[4];
  if (D == 128) {
    k_off[0] = g * 128 + (((2 * t) ^ g) << 4);
    k_off[1] = k_off[0] + 1024;
#pragma unroll
    for (int x = 0; x < 4; ++x) {
      const int r = 2 * t + (x & 1);
      v_off[x] = C::kHalf + (r + 8 * (x >> 1)) * 128 + ((g ^ r) << 4);
    }
  } else {
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      const int r = (g >> 1) + 4 * x;
      k_off[x] = r * 128 + ((((g & 1) * 4 + t) ^ r) << 4);
    }
#pragma unroll
    for (int x = 0; x < 4; ++x) {
      const int r = t + 4 * (x >> 1);
      v_off[x] = C::kHalf + r * 128 + ((((x & 1) * 4 + (g >> 1)) ^ r) << 4) + (g & 1) * 8;
    }
  }
  constexpr int kTile = 16 * D;  // bytes from a unit's tile to its next

  int item = 0, b = 0, h = 0, row0 = 0, len = 0, u = 0, u_first = 0, left = 0, U = 0;
  uint32_t qf[NT][D / 16][2];
  // shift = kLift - reference; O = acc * vref / F
  float sc[NT][2], acc[NT][D / 16][4], ref[NT][2], shift[NT][2], l[NT][2];
  float vref = 0.f, iref = 0.f, vtop = 0.f;  // V's reference (a power of two), 1 / it, its largest so far
  int lim[NT][2];
  float* scores = nullptr;
  bool ok = true;

  for (int i = 0; i < n_units; ++i) {
    if ((i & 31) == 0 && i > 0) {
      cur = nxt;
      nxt = locate<D, UT>(p, pre, xs + i + 32 + lane, xe);
      load_ranges<D>(p, nxt);
    }
    if (left == 0) {
      // ---- enter the next item: q as B operands, in fp16 at a power of two per row
      item = __shfl_sync(0xffffffffu, cur.item, i & 31);
      u = u_first = __shfl_sync(0xffffffffu, cur.u, i & 31);
      b = item / p.items_per_b;
      const int it = item - b * p.items_per_b;
      h = it / p.RT;
      row0 = (it - h * p.RT) * 8 * NT;
      len = clamp_len(p, b);
      U = (len + C::kUnit - 1) / C::kUnit;
      left = min(U - u, n_units - i);
      scores = p.scores ? p.scores + static_cast<long long>(item) * p.cap * p.rs : nullptr;
      vref = iref = vtop = 0.f;
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        const int r = row0 + 8 * n + g;
        uint4 w[D / 32];
        uint32_t mx = 0;
        const uint16_t* q = nullptr;
        if (r < p.rows) {
          const int qi = r / p.G;
          q = static_cast<const uint16_t*>(a.q) +
              ((static_cast<long long>(b) * a.nq + qi) * a.Hq + h * p.G + (r - qi * p.G)) * D +
              (D / 4) * t;
        }
#pragma unroll
        for (int j = 0; j < D / 32; ++j) {
          w[j] = q ? *reinterpret_cast<const uint4*>(q + 8 * j) : make_uint4(0, 0, 0, 0);
          mx = __vmaxu2(mx, __vmaxu2(w[j].x & 0x7FFF7FFFu, w[j].y & 0x7FFF7FFFu));
          mx = __vmaxu2(mx, __vmaxu2(w[j].z & 0x7FFF7FFFu, w[j].w & 0x7FFF7FFFu));
        }
        mx = max(mx & 0xFFFFu, mx >> 16);
        mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
        mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
        const int eb = static_cast<int>(mx >> 7);  // biased exponent of the row's largest
        const int up = eb == 0 || eb == 255 ? 0 : min(141 - eb, 127);
        const float f = __uint_as_float(static_cast<uint32_t>(up + 127) << 23);
        const float row_sc = ldexpf(s_unit, -up);
#pragma unroll
        for (int j = 0; j < D / 32; ++j) {
          const uint32_t ww[4] = {w[j].x, w[j].y, w[j].z, w[j].w};
#pragma unroll
          for (int e = 0; e < 4; ++e)
            qf[n][2 * j + (e >> 1)][e & 1] = pack_half(__uint_as_float(ww[e] << 16) * f,
                                                       __uint_as_float(ww[e] & 0xFFFF0000u) * f);
        }
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          sc[n][e] = __shfl_sync(0xffffffffu, row_sc, 4 * (2 * t + e));
          const int rr = row0 + 8 * n + 2 * t + e;
          lim[n][e] = len - a.nq + min(rr, p.rows - 1) / p.G;  // last key of the row
          ref[n][e] = kLowest;
          shift[n][e] = kLift - kLowest;
          l[n][e] = 0.f;
        }
#pragma unroll
        for (int m = 0; m < D / 16; ++m)
#pragma unroll
          for (int e = 0; e < 4; ++e) acc[n][m][e] = 0.f;
      }
    }
    // ---- one unit
    __syncwarp();  // every lane has read unit i - 1, whose stage the next load fills
    issue(i + S - 1, i >> 5);
    const float kr = __shfl_sync(0xffffffffu, cur.kr, i & 31);
    const float vr = __shfl_sync(0xffffffffu, cur.vr, i & 31);
    const bool there = __float_as_uint(kr) != __float_as_uint(kMissing);
    const bool here = wait_bar(&bars[i % S], (i / S) & 1, abort_flag, kSiteKv8);
    const int tok0 = u * C::kUnit;
    const uint8_t* stage = ring + (i % S) * 2 * C::kHalf;
    float x[UT][NT][4];  // scores, then their exponents log2 p
#pragma unroll
    for (int y = 0; y < UT; ++y)
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) x[y][n][e] = 0.f;
    float x2[NT][4];  // one tile a unit: its odd steps, for half the chain of dependent MMAs
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int e = 0; e < 4; ++e) x2[n][e] = 0.f;
#pragma unroll
    for (int j = 0; j < D / 64; ++j) {
#pragma unroll
      for (int y = 0; y < UT; ++y) {
        const uint4 ka = *reinterpret_cast<const uint4*>(stage + y * kTile + (k_off[0] ^ (j << 4)));
        const uint4 kb = *reinterpret_cast<const uint4*>(stage + y * kTile + (k_off[1] ^ (j << 4)));
        const uint32_t k0[4] = {ka.x, ka.y, ka.z, ka.w}, k1[4] = {kb.x, kb.y, kb.z, kb.w};
#pragma unroll
        for (int w = 0; w < 4; ++w) {
          uint32_t a0, a1, a2, a3;
          widen<FMT>(k0[w], a0, a2);
          widen<FMT>(k1[w], a1, a3);
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            float(&d)[4] = UT == 1 && (w & 1) ? x2[n] : x[y][n];
            mma16816(d, a0, a1, a2, a3, qf[n][4 * j + w][0], qf[n][4 * j + w][1], d);
          }
        }
      }
    }
    if (UT == 1)
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) x[0][n][e] += x2[n][e];
    // keys up to len - nq are seen by every row
    const bool edge = tok0 + C::kUnit - 1 > len - a.nq || !there;
    // V's ranges: P carries vr / vref (less than 2 and at least 2^-3, so that fp16 holds it much as
    // it would hold P) and O accumulates in the products; vref moves when a range leaves that
    // window, by powers of two, so that O is rescaled exactly however often ranges alternate.
    // Infinite and NaN ranges stay out of vref: they are for their rows alone.
    if ((vr >= 2.f * vref || (vr < vref * kFar && vr > vtop * kFarthest)) && vr <= 3.4028234e38f) {
      const float to = __uint_as_float(max(__float_as_uint(vr) & 0x7F800000u, 0x00800000u));
      const float f = vref / to;
      vref = to;
      vtop = fmaxf(vtop, to);
      iref = 1.f / to;
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int m = 0; m < D / 16; ++m)
#pragma unroll
          for (int e = 0; e < 4; ++e) acc[n][m][e] *= f;
    }
    const float rho = vr * iref;  // (NaN where no range was finite yet)
    bool over = !here;
    float f[NT][2], pv[NT][2];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      f[n][0] = sc[n][0] * kr;
      f[n][1] = sc[n][1] * kr;
      pv[n][0] = pv[n][1] = rho;
      if (edge) {  // tokens of the unit that each of the thread's rows sees
        const int see0 = there ? lim[n][0] - tok0 + 1 : 0, see1 = there ? lim[n][1] - tok0 + 1 : 0;
        // a row that sees nothing of the unit takes nothing from it, not even a NaN range
        if (see0 <= 0) pv[n][0] = 0.f;
        if (see1 <= 0) pv[n][1] = 0.f;
#pragma unroll
        for (int y = 0; y < UT; ++y) {
          // (a score that is masked stands as -inf whatever its factor is)
          x[y][n][0] = g + 16 * y >= see0 ? -INFINITY : x[y][n][0] * f[n][0];
          x[y][n][1] = g + 16 * y >= see1 ? -INFINITY : x[y][n][1] * f[n][1];
          x[y][n][2] = g + 16 * y + 8 >= see0 ? -INFINITY : x[y][n][2] * f[n][0];
          x[y][n][3] = g + 16 * y + 8 >= see1 ? -INFINITY : x[y][n][3] * f[n][1];
        }
        f[n][0] = f[n][1] = 1.f;
      }
#pragma unroll
      for (int y = 0; y < UT; ++y) {
        if (scores && 8 * n + 2 * t < p.rs) {
          const int tok = tok0 + 16 * y + g;
          float* at = scores + static_cast<long long>(tok) * p.rs + 8 * n + 2 * t;
          if (tok < len)
            *reinterpret_cast<float2*>(at) = make_float2(x[y][n][0] * f[n][0], x[y][n][1] * f[n][1]);
          if (tok + 8 < len)
            *reinterpret_cast<float2*>(at + 8 * p.rs) =
                make_float2(x[y][n][2] * f[n][0], x[y][n][3] * f[n][1]);
        }
        over = over || fmaxf(fmaf(fmaxf(x[y][n][0], x[y][n][2]), f[n][0], shift[n][0]),
                             fmaf(fmaxf(x[y][n][1], x[y][n][3]), f[n][1], shift[n][1])) >
                           kLift + kSlack;
      }
    }
    if (__any_sync(0xffffffffu, over)) {
      if (__any_sync(0xffffffffu, !here)) {
        ok = false;
        break;
      }
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float m = fmaxf(x[0][n][e], x[0][n][e + 2]);
          if (UT == 2) m = fmaxf(m, fmaxf(x[UT - 1][n][e], x[UT - 1][n][e + 2]));
          m *= f[n][e];
          m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 4));
          m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 8));
          m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 16));
          m = fmaxf(m, ref[n][e]);
          const float k = ex2(ref[n][e] - m);
          ref[n][e] = m;
          shift[n][e] = kLift - m;
          l[n][e] *= k;
#pragma unroll
          for (int m2 = 0; m2 < D / 16; ++m2) {
            acc[n][m2][e] *= k;
            acc[n][m2][e + 2] *= k;
          }
        }
    }
    uint32_t pb[UT][NT][2];
#pragma unroll
    for (int y = 0; y < UT; ++y)
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        float pr[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) pr[e] = ex2(fmaf(x[y][n][e], f[n][e & 1], shift[n][e & 1]));
        l[n][0] += pr[0] + pr[2];
        l[n][1] += pr[1] + pr[3];
        pb[y][n][0] = transpose8x8(pack_half(pr[0] * pv[n][0], pr[1] * pv[n][1]));
        pb[y][n][1] = transpose8x8(pack_half(pr[2] * pv[n][0], pr[3] * pv[n][1]));
      }
#pragma unroll
    for (int y = 0; y < UT; ++y) {
      uint32_t v[4][D / 32];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        if (D == 128) {
          const uint4 w = *reinterpret_cast<const uint4*>(stage + y * kTile + v_off[k]);
          v[k][0] = w.x; v[k][1] = w.y; v[k][2 % (D / 32)] = w.z; v[k][3 % (D / 32)] = w.w;
        } else {
          const uint2 w = *reinterpret_cast<const uint2*>(stage + y * kTile + v_off[k]);
          v[k][0] = w.x; v[k][1] = w.y;
        }
      }
      if (edge) {  // bytes behind the last token may hold anything, NaN codes among it
        const int rest = there ? len - tok0 - 16 * y : 0;
#pragma unroll
        for (int k = 0; k < 4; ++k)
          if (2 * t + (k & 1) + 8 * (k >> 1) >= rest)
#pragma unroll
            for (int w = 0; w < D / 32; ++w) v[k][w] = 0;
      }
#pragma unroll
      for (int m = 0; m < D / 16; ++m) {
        const uint32_t x01 = __byte_perm(v[0][m / 2], v[1][m / 2], m & 1 ? 0x7362 : 0x5140);
        const uint32_t x23 = __byte_perm(v[2][m / 2], v[3][m / 2], m & 1 ? 0x7362 : 0x5140);
        uint32_t a0, a1, a2, a3;
        widen<FMT>(x01, a0, a1);
        widen<FMT>(x23, a2, a3);
#pragma unroll
        for (int n = 0; n < NT; ++n)
          mma16816(acc[n][m], a0, a1, a2, a3, pb[y][n][0], pb[y][n][1], acc[n][m]);
      }
    }
    ++u;
    if (--left > 0) continue;

    // ---- leave the item: its output, or this warp's partial of it
    const float vs = vref * (1.f / full<FMT>());
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        l[n][e] += __shfl_xor_sync(0xffffffffu, l[n][e], 4);
        l[n][e] += __shfl_xor_sync(0xffffffffu, l[n][e], 8);
        l[n][e] += __shfl_xor_sync(0xffffffffu, l[n][e], 16);
      }
    if (u_first == 0 && u == U) {
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int rr = row0 + 8 * n + 2 * t + e;
          const bool some = l[n][e] != 0.f;
          if (p.lse && g == 0)  // rows past the last one weigh nothing
            p.lse[static_cast<long long>(item) * (8 * NT) + 8 * n + 2 * t + e] =
                some && rr < p.rows ? ref[n][e] - kLift + log2f(l[n][e]) : INFINITY;
          if (rr >= p.rows) continue;
          const float inv = some ? 1.f / l[n][e] : 0.f;
          uint16_t* dst = out_row<D>(p, b, h, rr) + g * (D / 8);
#pragma unroll
          for (int m = 0; m < D / 16; ++m)
            store_bf16(dst + 2 * m, acc[n][m][e] * inv * vs, acc[n][m][e + 2] * inv * vs);
        }
    } else {
      // slot 0 (more items follow, the ring is in use): global scratch; slot 1 (the
      // warp's last item, all its units consumed): the ring
      const bool last = i + 1 == n_units;
      const int slot = 2 * warp + last;
      float* o = last ? reinterpret_cast<float*>(ring)
                      : p.warp_o + (static_cast<long long>(cta) * W + warp) * 8 * NT * D;
      if (lane == 0) s_item[slot] = item;
      const float down = power_of_two(-sum_bits(U, C::kUnit));
      __syncwarp();  // every lane has read the last unit
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int c = 8 * n + 2 * t + e;
          if (g == 0) s_ml[slot * 8 * NT + c] = make_float2(ref[n][e], l[n][e]);
          float2* dst = reinterpret_cast<float2*>(o + c * D + g * (D / 8));
#pragma unroll
          for (int m = 0; m < D / 16; ++m)
            dst[m] = make_float2(acc[n][m][e] * down * vs, acc[n][m][e + 2] * down * vs);
        }
    }
  }
  if (!ok) {  // gave up on a load: let those in flight land before the memory goes away
    for (int i = 0; i < S; ++i) drain_wait(&bars[i], 0), drain_wait(&bars[i], 1);
  }
  __syncthreads();
  if (*abort_flag) return;

  // Join the warps' partials of each item, in order. A warp takes one column (row of
  // the item) of one item at a time, D / 4 lanes a column; the loads of all its
  // partials go out together.
  constexpr int kSlots = 2 * W, kLanes = D / 4, kCols = 32 / kLanes;
  int it_of[kSlots];
#pragma unroll
  for (int k = 0; k < kSlots / 4; ++k) {
    const int4 v = reinterpret_cast<const int4*>(s_item)[k];
    it_of[4 * k] = v.x; it_of[4 * k + 1] = v.y; it_of[4 * k + 2] = v.z; it_of[4 * k + 3] = v.w;
  }
  uint32_t first = 0;  // slots that begin an item
  {
    int last = -1;
#pragma unroll
    for (int k = 0; k < kSlots; ++k) {
      if (it_of[k] >= 0 && it_of[k] != last) {
        first |= 1u << k;
        last = it_of[k];
      }
    }
  }
  const int tasks = __popc(first) * (8 * NT / kCols), sub = lane / kLanes, d4 = lane % kLanes;
  for (int task = warp; task < tasks; task += W) {
    const int c = (task % (8 * NT / kCols)) * kCols + sub;
    uint32_t f = first;
    for (int k = task / (8 * NT / kCols); k > 0; --k) f &= f - 1;
    const int s0 = __ffs(f) - 1;
    int it_id = 0;
#pragma unroll
    for (int k = 0; k < kSlots; ++k)
      if (k == s0) it_id = it_of[k];
    float2 ml[kSlots];
    float m = kLowest;
#pragma unroll
    for (int k = 0; k < kSlots; ++k) {
      ml[k] = make_float2(kLowest, 0.f);
      if (it_of[k] == it_id) ml[k] = s_ml[k * 8 * NT + c];
    }
#pragma unroll
    for (int k = 0; k < kSlots; ++k) m = fmaxf(m, ml[k].x);
    float ls = 0.f;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int k0 = 0; k0 < kSlots; k0 += 8) {
      float4 v[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        v[k] = make_float4(0.f, 0.f, 0.f, 0.f);
        const int s = k0 + k;
        if (it_of[s] == it_id) {
          const float* src = s & 1 ? reinterpret_cast<const float*>(smem + (s >> 1) * C::kWarpRing)
                                   : p.warp_o + (static_cast<long long>(cta) * W + (s >> 1)) *
                                                    8 * NT * D;
          v[k] = *reinterpret_cast<const float4*>(src + c * D + 4 * d4);
        }
      }
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const float w = ex2(ml[k0 + k].x - m);
        ls += ml[k0 + k].y * w;
        o.x += v[k].x * w; o.y += v[k].y * w; o.z += v[k].z * w; o.w += v[k].w * w;
      }
    }
    const int ib = it_id / p.items_per_b, it = it_id - ib * p.items_per_b;
    const int U = (pre[ib + 1] - pre[ib]) / p.items_per_b;
    const int U0 = pre[ib] + it * U;
    if (cs <= U0 && U0 + U <= ce) {
      const int hh = it / p.RT, rr = (it - hh * p.RT) * 8 * NT + c;
      const bool some = ls != 0.f;
      if (p.lse && d4 == 0)
        p.lse[static_cast<long long>(it_id) * (8 * NT) + c] =
            some && rr < p.rows ? m - kLift + log2f(ls) : INFINITY;
      if (rr < p.rows) {
        const float inv = some ? power_of_two(sum_bits(U, C::kUnit)) / ls : 0.f;
        *reinterpret_cast<uint2*>(out_row<D>(p, ib, hh, rr) + 4 * d4) =
            make_uint2(pack_bf16x2(o.x * inv, o.y * inv), pack_bf16x2(o.z * inv, o.w * inv));
      }
    } else {
      const long long at = static_cast<long long>(2 * cta + (U0 > cs)) * 8 * NT + c;
      reinterpret_cast<float4*>(p.part_o)[at * kLanes + d4] = o;
      if (d4 == 0) p.part_ml[at] = make_float2(m, ls);
    }
  }
}

// One CTA per (CTA of the main kernel, row): joins the partials of the item that was
// cut and ended in that CTA, in their order.
template <int D, int NT>
__global__ void __launch_bounds__(128) combine_kernel(AttnP p) {
  constexpr int V = D / 4, GR = 128 / V;  // float4 lanes of a row, groups of partials
  const int c = blockIdx.y, t = threadIdx.x, lane4 = t % V, grp = t / V;
  pdl_launch();
  pdl_wait();
  const int4 rec = p.close[blockIdx.x];
  if (rec.x < 0) return;
  const int item = rec.x, c0 = rec.y, first = rec.z & 0xFFFF, c1 = rec.w;
  const int ib = item / p.items_per_b, it = item - ib * p.items_per_b;
  const int h = it / p.RT, rt = it - h * p.RT, rr = rt * 8 * NT + c;
  __shared__ float4 s_o[GR][V];
  __shared__ float2 s_ml[GR];
  float m = kLowest, l = 0.f;
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
  constexpr int kAhead = 4;  // partials a thread loads at once
  for (int k0 = c0 + grp; k0 <= c1; k0 += GR * kAhead) {
    float2 ml[kAhead];
    float4 v[kAhead];
#pragma unroll
    for (int x = 0; x < kAhead; ++x) {
      const int k = k0 + x * GR;
      const long long at = static_cast<long long>(k == c0 ? first : 2 * k) * 8 * NT + c;
      ml[x] = make_float2(kLowest, 0.f);
      v[x] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (k <= c1) {
        ml[x] = p.part_ml[at];
        v[x] = reinterpret_cast<const float4*>(p.part_o)[at * V + lane4];
      }
    }
    float mn = m;
#pragma unroll
    for (int x = 0; x < kAhead; ++x) mn = fmaxf(mn, ml[x].x);
    const float f0 = ex2(m - mn);
    m = mn;
    l *= f0;
    o.x *= f0; o.y *= f0; o.z *= f0; o.w *= f0;
#pragma unroll
    for (int x = 0; x < kAhead; ++x) {
      const float f = ex2(ml[x].x - m);
      l += ml[x].y * f;
      o.x += v[x].x * f; o.y += v[x].y * f; o.z += v[x].z * f; o.w += v[x].w * f;
    }
  }
  s_o[grp][lane4] = o;
  if (lane4 == 0) s_ml[grp] = make_float2(m, l);
  __syncthreads();
  if (grp != 0) return;
  m = kLowest;
#pragma unroll
  for (int k = 0; k < GR; ++k) m = fmaxf(m, s_ml[k].x);
  o = make_float4(0.f, 0.f, 0.f, 0.f);
  l = 0.f;
#pragma unroll
  for (int k = 0; k < GR; ++k) {
    const float f = ex2(s_ml[k].x - m);
    const float4 v = s_o[k][lane4];
    l += s_ml[k].y * f;
    o.x += v.x * f; o.y += v.y * f; o.z += v.z * f; o.w += v.w * f;
  }
  const bool some = l != 0.f;
  if (p.lse && lane4 == 0)
    p.lse[static_cast<long long>(item) * (8 * NT) + c] = some && rr < p.rows ? m - kLift + log2f(l) : INFINITY;
  if (rr >= p.rows) return;
  const float inv = some ? power_of_two(rec.z >> 16) / l : 0.f;
  *reinterpret_cast<uint2*>(out_row<D>(p, ib, h, rr) + 4 * lane4) =
      make_uint2(sm100::pack_bf16x2(o.x * inv, o.y * inv), sm100::pack_bf16x2(o.z * inv, o.w * inv));
}

// The weight of each key: sum over the kv head's rows of 2^(s - lse). A CTA takes runs
// of 1024 keys, four a thread with their loads together. The scores are an eighth of the
// codes' bytes and would leave L2 for memory later; they are read here for the last time,
// so their lines are discarded: 24 sequences of up to 32768 tokens, 4 kv heads of 7 rows,
// take 50.6 us with it and 55.5 without.
constexpr int kKeys = 4, kKeyRun = 256 * kKeys;
template <int NT>
__global__ void __launch_bounds__(256) weight_kernel(AttnP p) {
  pdl_launch();
  pdl_wait();
  const int bh = blockIdx.y, b = bh / p.a.c.Hkv, h = bh - b * p.a.c.Hkv;
  const long long len = min(static_cast<long long>(clamp_len(p, b)), p.a.weights_stride);
  const int lane = threadIdx.x & 31;
  for (long long jw = static_cast<long long>(blockIdx.x) * kKeyRun + threadIdx.x - lane; jw < len;
       jw += static_cast<long long>(gridDim.x) * kKeyRun) {
    const long long j0 = jw + lane;
    float w[kKeys] = {};
    for (int rt = 0; rt < p.RT; ++rt) {
      const long long item = static_cast<long long>(b) * p.items_per_b + h * p.RT + rt;
      const float4* z = reinterpret_cast<const float4*>(p.lse + item * (8 * NT));
      const float4* s[kKeys];  // (a key past the end reads the last one's)
#pragma unroll
      for (int u = 0; u < kKeys; ++u)
        s[u] = reinterpret_cast<const float4*>(p.scores + (item * p.cap + min(j0 + 256 * u, len - 1)) * p.rs);
#pragma unroll
      for (int n = 0; n < 2 * NT; ++n) {
        if (4 * n >= p.rs) break;
        const float4 y = z[n];
        float4 x[kKeys];
#pragma unroll
        for (int u = 0; u < kKeys; ++u) x[u] = s[u][n];
#pragma unroll
        for (int u = 0; u < kKeys; ++u)
          w[u] += (ex2(x[u].x - y.x) + ex2(x[u].y - y.y)) + (ex2(x[u].z - y.z) + ex2(x[u].w - y.w));
      }
    }
    // 32 keys of a row tile are rs lines of 128 bytes, aligned (a page is 16 keys or more)
    __syncwarp();
    for (int rt = 0; rt < p.RT; ++rt) {
      const long long item = static_cast<long long>(b) * p.items_per_b + h * p.RT + rt;
#pragma unroll
      for (int u = 0; u < kKeys; ++u) {
        const long long at = (jw + 256 * u) * p.rs + 32 * lane;
        if (lane < p.rs && at < p.cap * p.rs)
          asm volatile("discard.global.L2 [%0], 128;" ::"l"(p.scores + item * p.cap * p.rs + at) : "memory");
      }
    }
#pragma unroll
    for (int u = 0; u < kKeys; ++u) {
      if (j0 + 256 * u >= len) break;
      float* dst = p.a.weights + static_cast<long long>(bh) * p.a.weights_stride + j0 + 256 * u;
      *dst = p.a.accumulate ? *dst + w[u] : w[u];
    }
  }
}

struct AttnLayout {
  int NT, RT, rs;
  long long part_o, part_ml, warp_o, close, lse, scores, total;
};

AttnLayout attn_layout(int B, int nq, int Hq, int Hkv, int D, int max_pages, int page,
                       int with_weights) {
  auto al = [](long long x) { return (x + 255) / 256 * 256; };
  AttnLayout l;
  const int rows = nq * (Hq / Hkv);
  l.NT = rows > 8 ? 2 : 1;
  l.RT = (rows + 8 * l.NT - 1) / (8 * l.NT);
  const long long slots = 2LL * kMaxSms * (l.NT == 1 ? 2 : 1) * 8 * l.NT;
  const long long items = static_cast<long long>(B) * Hkv * l.RT;
  l.part_o = 0;
  l.part_ml = al(slots * D * 4);
  l.warp_o = l.part_ml + al(slots * 8);
  l.close = l.warp_o + al(slots / 2 * kWarps * D * 4);
  l.lse = l.close + al(2LL * kMaxSms * 16);
  l.scores = l.lse + (with_weights ? al(items * 8 * l.NT * 4) : 0);
  l.rs = (std::min(rows, 8 * l.NT) + 3) / 4 * 4;
  l.total = l.scores + (with_weights ? al(items * l.rs * max_pages * page * 4) : 0);
  return l;
}

// The codes of a pool as rows of 128 bytes, one unit a box, 128-byte swizzle.
template <int D, int UT>
int encode_codes(CUtensorMap* m, const void* codes, const Kv8Cache& c) {
  const cuuint64_t dims[2] = {128, static_cast<cuuint64_t>(c.num_pages) * c.Hkv * c.page * D / 128};
  const cuuint64_t strides[1] = {128};
  const cuuint32_t box[2] = {128, 16 * UT * D / 128};
  const cuuint32_t estr[2] = {1, 1};
  return g_encode(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(codes), dims, strides, box,
                  estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                  CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS
             ? TM_OK
             : TM_ERR_CUDA;
}

template <int D, int FMT, int NT, int UT>
int attn_run(AttnP& p, DeviceInfo* di) {
  using C = AttnCfg<D, NT, UT>;
  const Kv8AttnArgs& a = p.a;
  constexpr int kidx = (D == 128) * 8 + (FMT == TM_KV_E4M3) * 4 + (NT == 2) * 2 + (UT == 2);
  if (int rc = set_smem_once(di->kv8_attr_set[kidx], attn_kernel8<D, FMT, NT, UT>,
                             C::kSmem + 4 * kMaxAttnBatch))
    return rc;
  CUtensorMap tk, tv;
  if (encode_codes<D, UT>(&tk, a.c.k8, a.c) || encode_codes<D, UT>(&tv, a.c.v8, a.c))
    return TM_ERR_CUDA;
  cudaStream_t st = static_cast<cudaStream_t>(a.stream);
  // a CTA for every unit a warp could get, at most what is resident at once
  const long long units =
      static_cast<long long>(a.B) * p.items_per_b * ((p.cap + C::kUnit - 1) / C::kUnit);
  p.grid = static_cast<int>(
      std::min<long long>(std::min(di->sms, kMaxSms) * C::kCtas, (units + kWarps - 1) / kWarps));
  if (launch_early(attn_kernel8<D, FMT, NT, UT>, dim3(p.grid), C::kThreads, C::kSmem + a.B * 4, st, 1,
                   tk, tv, p))
    return TM_ERR_CUDA;
  const dim3 grid(p.grid, 8 * NT);
  if (launch_early(combine_kernel<D, NT>, grid, 128, 0, st, 1, p)) return TM_ERR_CUDA;
  if (!p.scores) return counted(2);
  const long long want = (p.cap + kKeyRun - 1) / kKeyRun;
  const dim3 wgrid(static_cast<unsigned>(want < 256 ? want : 256), a.B * a.c.Hkv);
  if (launch_early(weight_kernel<NT>, wgrid, 256, 0, st, 1, p)) return TM_ERR_CUDA;
  return counted(3);
}

template <int D, int FMT>
int attn_nt(AttnP& p, int NT, DeviceInfo* di) {
  constexpr int kOne = D == 64 ? 2 : 1;  // tiles of a unit with one row tile
  if (p.a.c.page >= 32)
    return NT == 1 ? attn_run<D, FMT, 1, kOne>(p, di) : attn_run<D, FMT, 2, 2>(p, di);
  return NT == 1 ? attn_run<D, FMT, 1, 1>(p, di) : attn_run<D, FMT, 2, 1>(p, di);
}

}  // namespace

long long kv8_attn_workspace_bytes(int B, int nq, int Hq, int Hkv, int D, int max_pages, int page,
                                   int with_weights) {
  return attn_layout(B, nq, Hq, Hkv, D, max_pages, page, with_weights).total;
}

int launch_kv8_attn(const Kv8AttnArgs& a) {
  DeviceInfo* di = nullptr;
  if (int rc = device_info(&di)) return rc;
  const AttnLayout l = attn_layout(a.B, a.nq, a.Hq, a.c.Hkv, a.c.D, a.max_pages, a.c.page,
                                   a.weights != nullptr);
  if (a.ws_bytes < l.total) return TM_ERR_INVALID_ARG;
  uint8_t* ws = static_cast<uint8_t*>(a.ws);
  AttnP p;
  p.a = a;
  p.G = a.Hq / a.c.Hkv;
  p.rows = a.nq * p.G;
  p.RT = l.RT;
  p.rs = l.rs;
  p.items_per_b = a.c.Hkv * l.RT;
  p.page_log = a.c.page == 16 ? 4 : a.c.page == 32 ? 5 : a.c.page == 64 ? 6 : 7;
  p.cap = static_cast<long long>(a.max_pages) * a.c.page;
  p.part_o = reinterpret_cast<float*>(ws + l.part_o);
  p.part_ml = reinterpret_cast<float2*>(ws + l.part_ml);
  p.warp_o = reinterpret_cast<float*>(ws + l.warp_o);
  p.close = reinterpret_cast<int4*>(ws + l.close);
  p.lse = a.weights ? reinterpret_cast<float*>(ws + l.lse) : nullptr;
  p.scores = a.weights ? reinterpret_cast<float*>(ws + l.scores) : nullptr;
  if (a.c.D == 128)
    return a.c.format == TM_KV_INT8 ? attn_nt<128, TM_KV_INT8>(p, l.NT, di)
                                    : attn_nt<128, TM_KV_E4M3>(p, l.NT, di);
  return a.c.format == TM_KV_INT8 ? attn_nt<64, TM_KV_INT8>(p, l.NT, di)
                                  : attn_nt<64, TM_KV_E4M3>(p, l.NT, di);
}
