// C ABI of the operators around the attention (declared in include/tm.h):
// rotary positions, the 8-bit cache and its attention, key weights and
// eviction. Argument validation only; the work is in the files beside this one.
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "tm.h"
#include "tm_internal.h"

namespace {

constexpr long long kIntMax = (1LL << 31) - 1;
constexpr int kMaxAttnBatch = 4096;

uintptr_t addr(const void* p) { return reinterpret_cast<uintptr_t>(p); }
bool aligned(const void* p, unsigned n) { return addr(p) % n == 0; }

bool overlaps(const void* a, long long abytes, const void* b, long long bbytes) {
  return addr(a) < addr(b) + static_cast<uintptr_t>(bbytes) &&
         addr(b) < addr(a) + static_cast<uintptr_t>(abytes);
}

// `rows` rows of `width` bytes, `stride` bytes apart.
struct Rows {
  const void* p;
  long long rows, width, stride;
  long long span() const { return (rows - 1) * stride + width; }
};

// Rows of one stride may interleave without sharing a byte (columns of a packed
// buffer); rows of different strides may not.
bool overlaps(const Rows& a, const Rows& b) {
  if (!a.p || !b.p || !overlaps(a.p, a.span(), b.p, b.span())) return false;
  if (a.stride != b.stride) return true;
  const long long s = a.stride;
  long long d = static_cast<long long>((addr(b.p) - addr(a.p)) % static_cast<uintptr_t>(s));
  if (addr(b.p) < addr(a.p)) {
    const long long e = static_cast<long long>((addr(a.p) - addr(b.p)) % static_cast<uintptr_t>(s));
    d = e ? s - e : 0;
  }
  return d < a.width || d + b.width > s;  // d: b's columns within a's rows
}

bool bad_stride(long long stride, long long width) {
  return stride < width || stride % 8 != 0 || stride > (1LL << 40);
}

int validate_cache(const void* k8, const void* v8, const float* k_range, const float* v_range,
                   int num_pages, int page, int format, int Hkv, int D) {
  if (!k8 || !v8 || !k_range || !v_range || num_pages < 1 || Hkv < 1) return TM_ERR_INVALID_ARG;
  if (!aligned(k8, 16) || !aligned(v8, 16) || !aligned(k_range, 4) || !aligned(v_range, 4))
    return TM_ERR_INVALID_ARG;
  if (format != TM_KV_INT8 && format != TM_KV_E4M3) return TM_ERR_INVALID_ARG;
  if (2LL * Hkv > 65535) return TM_ERR_INVALID_ARG;
  if (D != 64 && D != 128) return TM_ERR_UNSUPPORTED;
  if (page != 16 && page != 32 && page != 64 && page != 128) return TM_ERR_UNSUPPORTED;
  if (overlaps(k8, static_cast<long long>(num_pages) * Hkv * page * D, v8,
               static_cast<long long>(num_pages) * Hkv * page * D))
    return TM_ERR_INVALID_ARG;
  return TM_OK;
}

int validate_table(const int* table, int B, int max_pages, int page) {
  if (!table || !aligned(table, 4) || max_pages < 1) return TM_ERR_INVALID_ARG;
  if (static_cast<long long>(max_pages) * page > kIntMax) return TM_ERR_INVALID_ARG;
  if (B < 1 || B > 65535) return TM_ERR_INVALID_ARG;
  return TM_OK;
}

trimix::Kv8Cache cache(void* k8, void* v8, float* k_range, float* v_range, int num_pages, int page,
                       int format, int Hkv, int D) {
  trimix::Kv8Cache c;
  c.k8 = k8; c.v8 = v8;
  c.k_range = k_range; c.v_range = v_range;
  c.num_pages = num_pages; c.page = page; c.format = format; c.Hkv = Hkv; c.D = D;
  return c;
}

int validate_attn_sizes(int B, int nq, int Hq, int Hkv, int D, int max_pages, int page) {
  if (B < 1 || nq < 1 || Hq < 1 || Hkv < 1 || Hq % Hkv != 0 || max_pages < 1)
    return TM_ERR_INVALID_ARG;
  if (D != 64 && D != 128) return TM_ERR_UNSUPPORTED;
  if (page != 16 && page != 32 && page != 64 && page != 128) return TM_ERR_UNSUPPORTED;
  if (B > kMaxAttnBatch) return TM_ERR_UNSUPPORTED;
  const long long cap = static_cast<long long>(max_pages) * page;
  if (cap > kIntMax - 128 || static_cast<long long>(nq) * Hq > kIntMax / 128)
    return TM_ERR_INVALID_ARG;
  // work units (16 tokens of a head and row tile) of the whole call in 32 bits
  const long long rows = static_cast<long long>(nq) * (Hq / Hkv);
  const long long tiles = rows > 8 ? (rows + 15) / 16 : 1;
  const long long per = static_cast<long long>(Hkv) * tiles;
  if (per > kIntMax / B || per * B > kIntMax / (cap / 16 + 1)) return TM_ERR_INVALID_ARG;
  // each (sequence, kv head) is a grid row of the weights' kernel, each item a CTA of the join
  if (static_cast<long long>(B) * Hkv > 65535) return TM_ERR_INVALID_ARG;
  return TM_OK;
}

int validate_weights_sizes(int B, int Hq, int Hkv, int N, int D, int L) {
  if (B < 1 || Hq < 1 || Hkv < 1 || N < 1 || L < 1 || Hq % Hkv != 0) return TM_ERR_INVALID_ARG;
  if (D != 64 && D != 128) return TM_ERR_UNSUPPORTED;
  const int G = Hq / Hkv;
  if (G > 128) return TM_ERR_UNSUPPORTED;
  const long long rows = static_cast<long long>(B) * N;
  if (rows > kIntMax || static_cast<long long>(N) * Hq > kIntMax) return TM_ERR_INVALID_ARG;
  // work items of either pass, and rows of the statistics, in 32 bits
  const long long bg = static_cast<long long>(B) * Hkv, tpt = 128 / G;
  const long long q_tiles = (static_cast<long long>(L < N ? L : N) + tpt - 1) / tpt;
  const long long k_tiles = (static_cast<long long>(N) + 127) / 128;
  if (bg * k_tiles > kIntMax || bg * q_tiles > kIntMax / 128 || bg > kIntMax / 1024)
    return TM_ERR_INVALID_ARG;
  return TM_OK;
}

}  // namespace

extern "C" {

TM_API int tm_rope_fwd(const void* q, void* q_out, const void* k, void* k_out, int B, int N, int Hq,
                       int Hkv, int D, long long q_stride, long long q_out_stride,
                       long long k_stride, long long k_out_stride, int rot, int layout, int inverse,
                       const double* inv_freq, float mscale, const int* positions, long long first,
                       void* stream) {
  if (B < 1 || N < 1 || Hq < 0 || Hkv < 0 || Hq + static_cast<long long>(Hkv) < 1 || D < 1)
    return TM_ERR_INVALID_ARG;
  if (D % 16 != 0 || D > 512) return TM_ERR_UNSUPPORTED;
  if (rot < 2 || rot > D || rot % 2 != 0) return TM_ERR_INVALID_ARG;
  if (layout != TM_ROPE_HALF && layout != TM_ROPE_INTERLEAVED) return TM_ERR_INVALID_ARG;
  if (!inv_freq || !aligned(inv_freq, 8) || !aligned(positions, 4) || !std::isfinite(mscale))
    return TM_ERR_INVALID_ARG;
  if ((Hq > 0) != (q != nullptr) || (Hq > 0) != (q_out != nullptr) ||
      (Hkv > 0) != (k != nullptr) || (Hkv > 0) != (k_out != nullptr))
    return TM_ERR_INVALID_ARG;
  if (!aligned(q, 16) || !aligned(q_out, 16) || !aligned(k, 16) || !aligned(k_out, 16))
    return TM_ERR_INVALID_ARG;
  const long long rows = static_cast<long long>(B) * N;
  if (rows > kIntMax || (static_cast<long long>(Hq) + Hkv) * D > kIntMax) return TM_ERR_INVALID_ARG;
  const long long wq = static_cast<long long>(Hq) * D, wk = static_cast<long long>(Hkv) * D;
  if (Hq > 0 && (bad_stride(q_stride, wq) || bad_stride(q_out_stride, wq))) return TM_ERR_INVALID_ARG;
  if (Hkv > 0 && (bad_stride(k_stride, wk) || bad_stride(k_out_stride, wk)))
    return TM_ERR_INVALID_ARG;
  if (first > (1LL << 52) || first < -(1LL << 52)) return TM_ERR_INVALID_ARG;
  const Rows qi = {q, rows, wq * 2, q_stride * 2}, qo = {q_out, rows, wq * 2, q_out_stride * 2};
  const Rows ki = {k, rows, wk * 2, k_stride * 2}, ko = {k_out, rows, wk * 2, k_out_stride * 2};
  if (q == q_out ? q_stride != q_out_stride : overlaps(qo, qi)) return TM_ERR_INVALID_ARG;
  if (k == k_out ? k_stride != k_out_stride : overlaps(ko, ki)) return TM_ERR_INVALID_ARG;
  if (overlaps(qo, ko) || overlaps(qo, ki) || overlaps(ko, qi)) return TM_ERR_INVALID_ARG;
  trimix::RopeArgs a;
  a.q = q; a.q_out = q_out; a.k = k; a.k_out = k_out;
  a.rows = rows;
  a.N = N; a.Hq = Hq; a.Hkv = Hkv; a.D = D;
  a.q_stride = q_stride; a.q_out_stride = q_out_stride;
  a.k_stride = k_stride; a.k_out_stride = k_out_stride;
  a.rot = rot; a.layout = layout; a.inverse = inverse;
  a.inv_freq = inv_freq;
  a.mscale = mscale;
  a.positions = positions;
  a.first = first;
  a.stream = stream;
  return trimix::launch_rope(a);
}

TM_API int tm_rope_inv_freq(int rot, double base, double factor, double trained_len,
                            double low_turns, double high_turns, double* out) {
  if (!out || rot < 2 || rot % 2 != 0 || !std::isfinite(base) || !(base > 0.0) ||
      !std::isfinite(factor) || !(factor >= 1.0) || !std::isfinite(trained_len) ||
      !(trained_len >= 1.0) || !(low_turns >= 0.0) || !(high_turns >= low_turns))
    return TM_ERR_INVALID_ARG;
  for (int i = 0; i < rot / 2; ++i) {
    const double f = std::pow(base, -2.0 * i / rot);
    if (factor == 1.0) {
      out[i] = f;
      continue;
    }
    const double turns = trained_len * f / 6.283185307179586476925;
    double s;
    if (turns <= low_turns)
      s = 0.0;
    else if (turns >= high_turns)
      s = 1.0;
    else
      s = (turns - low_turns) / (high_turns - low_turns);
    out[i] = f * (s + (1.0 - s) / factor);
  }
  return TM_OK;
}

TM_API int tm_kv8_append(const void* k, const void* v, long long k_stride, long long v_stride,
                         int B, int n_src, int n, int Hkv, int D, const int* counts,
                         const int* index, const int* lens, const int* table, int max_pages,
                         void* k8, void* v8, float* k_range, float* v_range, int num_pages,
                         int page, int format, void* stream) {
  if (!k || !v || !lens || n < 1 || n_src < 1 || (!index && n > n_src)) return TM_ERR_INVALID_ARG;
  if (int rc = validate_cache(k8, v8, k_range, v_range, num_pages, page, format, Hkv, D)) return rc;
  if (int rc = validate_table(table, B, max_pages, page)) return rc;
  if (!aligned(k, 16) || !aligned(v, 16) || !aligned(counts, 4) || !aligned(index, 4) ||
      !aligned(lens, 4))
    return TM_ERR_INVALID_ARG;
  const long long w = static_cast<long long>(Hkv) * D;
  if (bad_stride(k_stride, w) || bad_stride(v_stride, w)) return TM_ERR_INVALID_ARG;
  if (static_cast<long long>(B) * n_src > kIntMax) return TM_ERR_INVALID_ARG;
  const long long pool = static_cast<long long>(num_pages) * w * page;
  const long long kb = ((static_cast<long long>(B) * n_src - 1) * k_stride + w) * 2;
  const long long vb = ((static_cast<long long>(B) * n_src - 1) * v_stride + w) * 2;
  if (overlaps(k8, pool, k, kb) || overlaps(k8, pool, v, vb) || overlaps(v8, pool, k, kb) ||
      overlaps(v8, pool, v, vb))
    return TM_ERR_INVALID_ARG;
  trimix::Kv8AppendArgs a;
  a.c = cache(k8, v8, k_range, v_range, num_pages, page, format, Hkv, D);
  a.k = k; a.v = v;
  a.k_stride = k_stride; a.v_stride = v_stride;
  a.B = B; a.n_src = n_src; a.n = n;
  a.counts = counts; a.index = index; a.lens = lens; a.table = table; a.max_pages = max_pages;
  a.stream = stream;
  return trimix::launch_kv8_append(a);
}

TM_API int tm_kv8_compact(const int* index, int keep, const int* kept, const int* lens, int B,
                          int Hkv, int D, const int* table, int max_pages, const int* new_table,
                          int new_max_pages, void* k8, void* v8, float* k_range, float* v_range,
                          int num_pages, int page, int format, const float* weights,
                          long long weights_stride, float* new_weights,
                          long long new_weights_stride, void* stream) {
  if (!index || !lens || keep < 1) return TM_ERR_INVALID_ARG;
  if (int rc = validate_cache(k8, v8, k_range, v_range, num_pages, page, format, Hkv, D)) return rc;
  if (int rc = validate_table(table, B, max_pages, page)) return rc;
  if (int rc = validate_table(new_table, B, new_max_pages, page)) return rc;
  if (static_cast<long long>(new_max_pages) * page < keep || (keep - 1) / page >= 65535)
    return TM_ERR_INVALID_ARG;
  if ((weights != nullptr) != (new_weights != nullptr)) return TM_ERR_INVALID_ARG;
  if (!aligned(index, 4) || !aligned(kept, 4) || !aligned(lens, 4) || !aligned(weights, 4) ||
      !aligned(new_weights, 4))
    return TM_ERR_INVALID_ARG;
  if (weights) {
    const long long rows = static_cast<long long>(B) * Hkv;
    if (weights_stride < 1 || new_weights_stride < keep || weights_stride > kIntMax ||
        new_weights_stride > kIntMax)
      return TM_ERR_INVALID_ARG;
    if (overlaps(weights, rows * weights_stride * 4, new_weights, rows * new_weights_stride * 4))
      return TM_ERR_INVALID_ARG;
  }
  trimix::Kv8CompactArgs a;
  a.c = cache(k8, v8, k_range, v_range, num_pages, page, format, Hkv, D);
  a.index = index; a.keep = keep; a.kept = kept; a.lens = lens; a.B = B;
  a.table = table; a.max_pages = max_pages;
  a.new_table = new_table; a.new_max_pages = new_max_pages;
  a.weights = weights; a.weights_stride = weights_stride;
  a.new_weights = new_weights; a.new_weights_stride = new_weights_stride;
  a.stream = stream;
  return trimix::launch_kv8_compact(a);
}

TM_API int tm_kv8_attn_workspace_size(int B, int nq, int Hq, int Hkv, int D, int max_pages,
                                      int page, int with_weights, long long* bytes) {
  if (!bytes) return TM_ERR_INVALID_ARG;
  if (int rc = validate_attn_sizes(B, nq, Hq, Hkv, D, max_pages, page)) return rc;
  *bytes = trimix::kv8_attn_workspace_bytes(B, nq, Hq, Hkv, D, max_pages, page, with_weights != 0);
  return TM_OK;
}

TM_API int tm_kv8_attn_fwd(const void* q, void* o, int B, int nq, int Hq, int Hkv, int D,
                           float scale, const void* k8, const void* v8, const float* k_range,
                           const float* v_range, int num_pages, int page, int format,
                           const int* table, int max_pages, const int* lens, float* weights,
                           long long weights_stride, int accumulate, void* workspace,
                           long long workspace_bytes, void* stream) {
  if (!q || !o || !lens || !workspace) return TM_ERR_INVALID_ARG;
  if (int rc = validate_attn_sizes(B, nq, Hq, Hkv, D, max_pages, page)) return rc;
  if (int rc = validate_cache(k8, v8, k_range, v_range, num_pages, page, format, Hkv, D)) return rc;
  if (int rc = validate_table(table, B, max_pages, page)) return rc;
  if (!std::isfinite(scale) || !(scale > 0.f)) return TM_ERR_INVALID_ARG;
  if (!aligned(q, 16) || !aligned(o, 16) || !aligned(lens, 4) || !aligned(weights, 4) ||
      !aligned(workspace, 256))
    return TM_ERR_INVALID_ARG;
  if (weights && (weights_stride < 1 || weights_stride > kIntMax)) return TM_ERR_INVALID_ARG;
  const long long qb = static_cast<long long>(B) * nq * Hq * D * 2;
  const long long pool = static_cast<long long>(num_pages) * Hkv * page * D;
  if (pool / 64 > kIntMax) return TM_ERR_INVALID_ARG;  // rows of the pool in 32 bits
  const long long wb = static_cast<long long>(B) * Hkv * (weights ? weights_stride : 0) * 4;
  if (overlaps(o, qb, q, qb) || overlaps(o, qb, k8, pool) || overlaps(o, qb, v8, pool))
    return TM_ERR_INVALID_ARG;
  if (weights && (overlaps(weights, wb, o, qb) || overlaps(weights, wb, q, qb) ||
                  overlaps(weights, wb, k8, pool) || overlaps(weights, wb, v8, pool)))
    return TM_ERR_INVALID_ARG;
  const long long need =
      trimix::kv8_attn_workspace_bytes(B, nq, Hq, Hkv, D, max_pages, page, weights != nullptr);
  if (workspace_bytes < need) return TM_ERR_INVALID_ARG;
  if (overlaps(workspace, need, q, qb) || overlaps(workspace, need, o, qb) ||
      overlaps(workspace, need, k8, pool) || overlaps(workspace, need, v8, pool) ||
      (weights && overlaps(workspace, need, weights, wb)))
    return TM_ERR_INVALID_ARG;
  trimix::Kv8AttnArgs a;
  a.c = cache(const_cast<void*>(k8), const_cast<void*>(v8), const_cast<float*>(k_range),
              const_cast<float*>(v_range), num_pages, page, format, Hkv, D);
  a.q = q; a.o = o;
  a.B = B; a.nq = nq; a.Hq = Hq;
  a.scale = scale;
  a.table = table; a.max_pages = max_pages; a.lens = lens;
  a.weights = weights; a.weights_stride = weights_stride; a.accumulate = accumulate;
  a.ws = workspace; a.ws_bytes = workspace_bytes;
  a.stream = stream;
  return trimix::launch_kv8_attn(a);
}

TM_API int tm_key_weights_workspace_size(int B, int Hq, int Hkv, int N, int D, int L,
                                         long long* bytes) {
  if (!bytes) return TM_ERR_INVALID_ARG;
  if (int rc = validate_weights_sizes(B, Hq, Hkv, N, D, L)) return rc;
  *bytes = trimix::key_weights_workspace_bytes(B, Hq, Hkv, N, D, L);
  return TM_OK;
}

TM_API int tm_key_weights_fwd(const void* q, const void* k, int B, int Hq, int Hkv, int N, int D,
                              float scale, int L, const int* lens, float* weights,
                              long long weights_stride, int accumulate, void* workspace,
                              long long workspace_bytes, void* stream) {
  if (!q || !k || !weights || !workspace) return TM_ERR_INVALID_ARG;
  if (int rc = validate_weights_sizes(B, Hq, Hkv, N, D, L)) return rc;
  if (!std::isfinite(scale) || !(scale > 0.f)) return TM_ERR_INVALID_ARG;
  if (!aligned(q, 16) || !aligned(k, 16) || !aligned(lens, 4) || !aligned(weights, 4) ||
      !aligned(workspace, 256))
    return TM_ERR_INVALID_ARG;
  if (weights_stride < N || weights_stride > kIntMax) return TM_ERR_INVALID_ARG;
  const long long rows = static_cast<long long>(B) * N;
  const long long qb = rows * Hq * D * 2, kb = rows * Hkv * D * 2;
  const long long wb = static_cast<long long>(B) * Hkv * weights_stride * 4;
  const long long need = trimix::key_weights_workspace_bytes(B, Hq, Hkv, N, D, L);
  if (workspace_bytes < need) return TM_ERR_INVALID_ARG;
  if (overlaps(weights, wb, q, qb) || overlaps(weights, wb, k, kb) ||
      overlaps(workspace, need, q, qb) || overlaps(workspace, need, k, kb) ||
      overlaps(workspace, need, weights, wb))
    return TM_ERR_INVALID_ARG;
  trimix::KeyWeightsArgs a;
  a.q = q; a.k = k;
  a.B = B; a.Hq = Hq; a.Hkv = Hkv; a.N = N; a.D = D;
  a.scale = scale;
  a.L = L < N ? L : N;
  a.lens = lens;
  a.weights = weights; a.stride = weights_stride; a.accumulate = accumulate;
  a.ws = workspace; a.ws_bytes = workspace_bytes;
  a.stream = stream;
  return trimix::launch_key_weights(a);
}

TM_API int tm_kv_select(const float* weights, long long weights_stride, const int* lens, int B,
                        int H, int n, int keep, int sinks, int recent, int* index, int* kept,
                        void* stream) {
  if (!weights || !index || B < 1 || H < 1 || n < 1 || keep < 1 || sinks < 0 || recent < 0)
    return TM_ERR_INVALID_ARG;
  if (static_cast<long long>(sinks) + recent > keep || weights_stride < n ||
      weights_stride > kIntMax)
    return TM_ERR_INVALID_ARG;
  // the kernel's loops over n and keep step by a cluster's threads or keys, in 32 bits
  if (n > kIntMax - 65536 || keep > kIntMax - 65536) return TM_ERR_INVALID_ARG;
  const long long rows = static_cast<long long>(B) * H;
  if (rows > kIntMax / 8 || B > 65535 || 2LL * H > 65535) return TM_ERR_INVALID_ARG;
  if (!aligned(weights, 4) || !aligned(lens, 4) || !aligned(index, 4) || !aligned(kept, 4))
    return TM_ERR_INVALID_ARG;
  if (overlaps(index, rows * keep * 4, weights, rows * weights_stride * 4) ||
      (kept && overlaps(kept, 4LL * B, weights, rows * weights_stride * 4)) ||
      (kept && overlaps(kept, 4LL * B, index, rows * keep * 4)))
    return TM_ERR_INVALID_ARG;
  trimix::KvSelectArgs a;
  a.weights = weights; a.stride = weights_stride; a.lens = lens;
  a.B = B; a.H = H; a.n = n; a.keep = keep; a.sinks = sinks; a.recent = recent;
  a.index = index; a.kept = kept;
  a.stream = stream;
  return trimix::launch_kv_select(a);
}

}  // extern "C"
