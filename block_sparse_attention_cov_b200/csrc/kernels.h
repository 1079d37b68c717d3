// kernels.h -- internal launch interface between the C ABI layer and the CUDA
// kernels (not part of the public ABI).
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

namespace solattn {

struct PooledPtrs {
  float* qbar;
  float* kbar;
  float* vbar;
  float* kmean;
  float* kcov;
  uint16_t* kbar16;  // bf16 copies for the per-token correction
  uint16_t* vbar16;
};

// Element strides of q, k, v and out; the d elements of a token are contiguous.
struct Strides {
  long long b, h, n;
};

struct ForwardArgs {
  const uint16_t* q;
  const uint16_t* k;
  const uint16_t* v;
  uint16_t* out;
  float* lse;          // may be null
  int32_t* density;    // may be null
  PooledPtrs pooled;   // unused when route == false
  float beta;
  int rule;            // 0 threshold, 1 top-k, 2 top-p (solattn_rule)
  int topk;
  float topp;
  int n_forced;        // leading key blocks always kept
  int token_corr;      // 1: per-token correction through pooled-key tiles
  bool route;          // false: dense attention (no routing, no correction)
  int BH, H, N, d;
  Strides st;          // of q, k, v and out
  void* status;        // DeviceStatus in the caller's workspace
};

cudaError_t launch_pool(const uint16_t* q, const uint16_t* k, const uint16_t* v, const PooledPtrs& p, int BH,
                        int H, int N, int d, const Strides& st, int num_sms, cudaStream_t stream);

// Fused forward with per-unit key lists (any kept-set rule, either
// correction): one unit in flight per CTA (forward.cu).
cudaError_t launch_forward(const ForwardArgs& a, int num_sms, cudaStream_t stream);

// Fused forward with two units in flight per CTA (forward_pp.cu): threshold
// rule with the block-level correction (forced blocks allowed), and the dense
// path.
cudaError_t launch_forward_pp(const ForwardArgs& a, int num_sms, cudaStream_t stream);

// Mean and covariance of the pooled keys (the second launch of launch_pool).
cudaError_t launch_key_stats(const float* kbar, float* kmean, float* kcov, int BH, int NB, int d,
                             cudaStream_t stream);

enum { kBF16 = 0, kF16 = 1, kF32 = 2 };  // == solattn_dtype

// Rotary positions (rotary.cu).
struct RotaryTable {
  const unsigned long long* freq;  // turns per unit of position, in 2^-64
  const int32_t* axis;             // position axis of each pair; null: axis 0
  const int32_t* pos;
  long long pos_b, pos_n;          // strides of pos (batch, token)
  int rot, axes, layout;           // layout 0: interleaved pairs, 1: halves
  int inverse;
  float gain;
};
struct RotaryArgs {
  const void* x[2];  // queries, keys (x[1] null: queries only)
  void* y[2];
  Strides xs[2], ys[2];
  int heads[2];
  int dtype, B, N, d;
  RotaryTable t;
};
cudaError_t launch_rotary(const RotaryArgs& a, int num_sms, cudaStream_t stream);

struct RotaryPoolArgs {
  const uint16_t* x[3];  // q, k, v
  uint16_t* y[2];        // rotated q, k
  float* bar[3];         // qbar, kbar, vbar
  uint16_t* bar16[3];    // null, kbar16, vbar16
  Strides st, ys;        // of q, k, v and of the rotated q, k
  int B, H, N, d;
  RotaryTable t;
};
cudaError_t launch_rotary_pool(const RotaryPoolArgs& a, int num_sms, cudaStream_t stream);

// 8-bit cache: writing tokens (cache_append.cu).
struct DeviceStatus;
struct CacheAppendArgs {
  const void* x[2];    // keys, values [B][H][N][d]
  uint8_t* data[2];    // e4m3 pages
  float* scale[2];
  Strides st;          // of x
  long long page_stride, scale_stride, table_stride;
  const int32_t* table;
  const int32_t* lengths;
  const int32_t* counts;  // may be null
  int dtype, pages, columns, B, H, N, d;
  DeviceStatus* status;   // may be null
};
cudaError_t launch_cache_append(const CacheAppendArgs& a, cudaStream_t stream);

// 8-bit cache: attention (cache_step.cu, cache_chunk.cu).
struct CacheAttnArgs {
  const uint16_t* q;
  uint16_t* out;
  float* lse;  // may be null
  const uint8_t* k;
  const uint8_t* v;
  const float* k_scale;
  const float* v_scale;
  const int32_t* table;
  const int32_t* lengths;
  const int32_t* counts;  // may be null: N each
  Strides st, ost;        // of q and of out
  long long page_stride, scale_stride, table_stride;
  float scale_log2;       // softmax scale * log2(e)
  int dtype, pages, columns, B, H, Hk, N, d;
  int group;              // H / Hk
  uint32_t group_mul;     // row / group = (umulhi(group_mul, row) + row) >> group_shift, row < 2^31
  uint32_t group_shift;
  int causal;
  int splits;             // parts of the key axis, joined from part_o / part_ml when > 1
  int longest_first;      // the grid takes the sequences by falling length (B <= 64)
  float* part_o;          // [B][H][N][splits][d]
  float2* part_ml;        // [B][H][N][splits] (reference, sum)
  DeviceStatus* status;
};
// Which kernel a call takes, and how many parts its key axis is split into.
struct CachePlan {
  bool step;
  int splits;
  bool longest_first;
};
CachePlan cache_plan(int B, int H, int Hk, int N, int d, int columns);
cudaError_t launch_cache_step(const CacheAttnArgs& a, cudaStream_t stream);
cudaError_t launch_cache_chunk(const CacheAttnArgs& a, cudaStream_t stream);
cudaError_t launch_cache_join(const CacheAttnArgs& a, cudaStream_t stream);

#ifdef SOLATTN_TEST_HOOKS
// Test builds only: hook variables of each kernel's translation unit.
cudaError_t set_test_hooks_fwd(int skip_cta, unsigned long long wait_budget_ns);
cudaError_t set_route_dump_fwd(uint32_t* mask, float* stats);
cudaError_t set_test_hooks_pp(int skip_cta, unsigned long long wait_budget_ns);
cudaError_t set_test_hooks_step(int skip_cta, unsigned long long wait_budget_ns);
cudaError_t set_test_hooks_chunk(int skip_cta, unsigned long long wait_budget_ns);
cudaError_t set_route_dump_pp(uint32_t* mask, float* stats);
#endif

}  // namespace solattn
