// Internal interface between the C ABI (tm_api.cu) and the kernel translation
// unit (tm_attn.cu). Not installed; not part of the public ABI.
#pragma once

#include <cstdint>

#include "tm_tiles.cuh"

namespace trimix {

// Codes the kernels write into the device status word.
enum DeviceStatus : int { kDevOk = 0, kDevTimeout = 1 };

struct LaunchArgs {
  const void* q;
  const void* k;
  const void* v;
  void* o;
  int B, Hq, Hkv, N, D;
  float scale;
  Pattern pat;
  void* ws;           // split workspace (device), or nullptr: no item is split
  long long ws_bytes;
  const int* bs_off;  // block-sparse index (device CSR), or nullptr: pat's tile list
  const int* bs_idx;
  long long bs_nnz;
  const int* hS;      // per-head sinks and windows (host, Hq each), or nullptr
  const int* hW;
  int inject_cta;     // test hook: -1, or the CTA whose first Q is never delivered
  void* stream;
  int qb_lo = 0;      // the q-blocks [qb_lo, qb_hi) of the sequence; qb_hi -1: to the end
  int qb_hi = -1;
};

struct DiscArgs {
  const void* q;
  const void* k;
  int B, Hq, Hkv, N, D, P;
  float scale, alpha;
  void* ws;
  long long ws_bytes;
  int* offsets;
  int* indices;
  float* scores_out;  // optional: the block scores land here instead of the workspace
  void* stream;
};

// Rotary positions (tm_rope.cu). Strides are elements between consecutive tokens.
struct RopeArgs {
  const void* q;
  void* q_out;
  const void* k;
  void* k_out;
  long long rows;  // B * N
  int N, Hq, Hkv, D;
  long long q_stride, q_out_stride, k_stride, k_out_stride;
  int rot, layout, inverse;
  const double* inv_freq;
  float mscale;
  const int* positions;
  long long first;
  void* stream;
};

// The paged 8-bit cache: codes [num_pages, Hkv, page, D], ranges [num_pages, Hkv].
struct Kv8Cache {
  void* k8;
  void* v8;
  float* k_range;
  float* v_range;
  int num_pages, page, format, Hkv, D;
};

struct Kv8AppendArgs {
  Kv8Cache c;
  const void* k;
  const void* v;
  long long k_stride, v_stride;
  int B, n_src, n;
  const int* counts;
  const int* index;
  const int* lens;
  const int* table;
  int max_pages;
  void* stream;
};

struct Kv8CompactArgs {
  Kv8Cache c;
  const int* index;
  int keep;
  const int* kept;
  const int* lens;
  int B;
  const int* table;
  int max_pages;
  const int* new_table;
  int new_max_pages;
  const float* weights;
  long long weights_stride;
  float* new_weights;
  long long new_weights_stride;
  void* stream;
};

struct Kv8AttnArgs {
  Kv8Cache c;
  const void* q;
  void* o;
  int B, nq, Hq;
  float scale;
  const int* table;
  int max_pages;
  const int* lens;
  float* weights;
  long long weights_stride;
  int accumulate;
  void* ws;
  long long ws_bytes;
  void* stream;
};

struct KvSelectArgs {
  const float* weights;
  long long stride;
  const int* lens;
  int B, H, n, keep, sinks, recent;
  int* index;
  int* kept;
  void* stream;
};

struct KeyWeightsArgs {
  const void* q;
  const void* k;
  int B, Hq, Hkv, N, D;
  float scale;
  int L;
  const int* lens;
  float* weights;
  long long stride;
  int accumulate;
  void* ws;
  long long ws_bytes;
  void* stream;
};

// For the other translation units: the current device's SM count (TM_ERR_UNSUPPORTED
// unless it is an sm_100), and the bookkeeping after n launches.
int device_sms(int* sms);
int count_launches(int n);

int launch_rope(const RopeArgs& a);
int launch_kv8_append(const Kv8AppendArgs& a);
int launch_kv8_compact(const Kv8CompactArgs& a);
int launch_kv8_attn(const Kv8AttnArgs& a);
// Workspace of launch_kv8_attn on `sms` SMs.
long long kv8_attn_workspace_bytes(int B, int nq, int Hq, int Hkv, int D, int max_pages, int page,
                                   int with_weights);
int launch_kv_select(const KvSelectArgs& a);
int launch_key_weights(const KeyWeightsArgs& a);
long long key_weights_workspace_bytes(int B, int Hq, int Hkv, int N, int D, int L);

// All return a tm_status value.
int launch_attention(const LaunchArgs& a);
int launch_dump_tiles(const Pattern& p, int* out_dev, long long cap, void* stream);
int launch_mma_probe(const void* q, const void* k, const void* v, float* s_out, float* o_out,
                     int D, void* stream);
int read_and_clear_device_status(void* stream);
// Kernels launched by the library so far in this process.
long long kernel_launches();
int launch_discovery(const DiscArgs& a);
long long discovery_workspace_bytes(int B, int Hq, int Hkv, int N, int D, int P);
int debug_schedule(int B, int Hq, int Hkv, int N, const Pattern& pat, int max_ctas, int split,
                   int qb_lo, int qb_hi, int* out, long long cap, long long* count,
                   const int* hS = nullptr, const int* hW = nullptr);
// Workspace bytes the split schedule needs on num_ctas CTAs (<= 0: the
// current device's SM count); 0 if no item is split.
int workspace_bytes(int B, int Hq, int Hkv, int N, int D, const Pattern& pat, int num_ctas,
                    long long* bytes);

}  // namespace trimix
