// ops_api.cu -- C ABI of the operators around attention (include/solattn.h):
// rotary positions, rotary positions with the pooled statistics, and the 8-bit
// key/value cache. Argument checks and stream-ordered launches; no allocation.
#include <cuda_runtime.h>
#include <algorithm>
#include <cmath>
#include <cstdint>

#include "../../include/solattn.h"
#include "api_common.h"
#include "kernels.h"
#include "ptx.cuh"

namespace {

using solattn::Strides;

static_assert(static_cast<int>(solattn::kBF16) == SOLATTN_BF16 && static_cast<int>(solattn::kF16) == SOLATTN_F16 &&
                  static_cast<int>(solattn::kF32) == SOLATTN_F32,
              "dtype codes");

// Strides of one tensor: null or all zero = contiguous. Inputs may repeat rows
// (stride 0); an output's heads, batches and tokens must be apart.
int tensor_strides(const solattn_strides_t* in, int B, int H, int N, int d, bool output, Strides* out) {
  if (!in || (in->batch == 0 && in->head == 0 && in->token == 0)) {
    *out = Strides{static_cast<long long>(H) * N * d, static_cast<long long>(N) * d, d};
    return SOLATTN_OK;
  }
  if (in->batch < 0 || in->head < 0 || in->token < 0) return SOLATTN_ERR_ARG;
  if (output && ((N > 1 && in->token < d) || (H > 1 && in->head < d) || (B > 1 && in->batch < d)))
    return SOLATTN_ERR_ARG;
  *out = Strides{in->batch, in->head, in->token};
  return SOLATTN_OK;
}

bool multiple_of_8(const Strides& s) { return ((s.b | s.h | s.n) & 7) == 0; }

int check_rotary(const solattn_rotary_t* r, int N, int d, int inverse, solattn::RotaryTable* t) {
  if (!r || !r->freq || !r->positions) return SOLATTN_ERR_ARG;
  if (r->rot <= 0 || (r->rot & 1) || r->rot > d) return SOLATTN_ERR_ARG;
  if (r->layout != SOLATTN_ROTARY_INTERLEAVED && r->layout != SOLATTN_ROTARY_HALF) return SOLATTN_ERR_ARG;
  if (r->axes < 1 || r->axes > SOLATTN_ROTARY_MAX_AXES || (r->axes > 1 && !r->axis)) return SOLATTN_ERR_ARG;
  if (!std::isfinite(r->gain) || r->position_batch < 0 || r->position_token < 0) return SOLATTN_ERR_ARG;
  if (reinterpret_cast<uintptr_t>(r->freq) & 7u) return SOLATTN_ERR_ALIGN;
  if (!solattn::aligned4(r->axis) || !solattn::aligned4(r->positions)) return SOLATTN_ERR_ALIGN;
  *t = solattn::RotaryTable{};
  t->freq = reinterpret_cast<const unsigned long long*>(r->freq);
  t->axis = r->axes > 1 ? r->axis : nullptr;
  t->pos = r->positions;
  t->pos_b = r->position_batch;
  t->pos_n = r->position_token ? r->position_token : r->axes;
  t->rot = r->rot;
  t->axes = r->axes;
  t->layout = r->layout;
  t->inverse = inverse != 0;
  t->gain = r->gain;
  (void)N;
  return SOLATTN_OK;
}

bool dtype_ok(int dtype, bool fp32) {
  return dtype == SOLATTN_BF16 || dtype == SOLATTN_F16 || (fp32 && dtype == SOLATTN_F32);
}

struct CacheView {
  long long page_stride, scale_stride, table_stride;
};

int check_cache(const solattn_cache_t* c, const int32_t* table, int columns, long long table_stride,
                const int32_t* lengths, const int32_t* counts, CacheView* v) {
  if (!c || !c->k || !c->v || !c->k_scale || !c->v_scale || !table || !lengths) return SOLATTN_ERR_ARG;
  if (c->pages <= 0 || c->heads <= 0 || columns <= 0 || table_stride < 0) return SOLATTN_ERR_ARG;
  if (c->d != 64 && c->d != 128) return SOLATTN_ERR_UNSUPPORTED;
  if (columns > SOLATTN_CACHE_MAX_COLUMNS) return SOLATTN_ERR_UNSUPPORTED;
  const long long page = static_cast<long long>(c->heads) * SOLATTN_BLOCK * c->d;
  if (c->page_stride < 0 || (c->page_stride && c->page_stride < page) || (c->page_stride & 15)) return SOLATTN_ERR_ARG;
  if (c->scale_stride < 0 || (c->scale_stride && c->scale_stride < c->heads)) return SOLATTN_ERR_ARG;
  if (table_stride && table_stride < columns) return SOLATTN_ERR_ARG;
  if (!solattn::aligned16(c->k) || !solattn::aligned16(c->v)) return SOLATTN_ERR_ALIGN;
  if (!solattn::aligned4(c->k_scale) || !solattn::aligned4(c->v_scale) || !solattn::aligned4(table) ||
      !solattn::aligned4(lengths) || !solattn::aligned4(counts))
    return SOLATTN_ERR_ALIGN;
  v->page_stride = c->page_stride ? c->page_stride : page;
  v->scale_stride = c->scale_stride ? c->scale_stride : c->heads;
  v->table_stride = table_stride ? table_stride : columns;
  return SOLATTN_OK;
}

int check_attention_shape(int B, int H, int N, int d, int heads, int columns) {
  if (B <= 0 || H <= 0 || N <= 0 || heads <= 0 || columns <= 0 || H % heads) return SOLATTN_ERR_ARG;
  if (d != 64 && d != 128) return SOLATTN_ERR_UNSUPPORTED;
  if (columns > SOLATTN_CACHE_MAX_COLUMNS || B > 65535) return SOLATTN_ERR_UNSUPPORTED;
  // one grid index per row (joining), one per 16-row tile and key head (steps)
  if (static_cast<long long>(B) * H * N >= (1ll << 31) || H > 16384) return SOLATTN_ERR_UNSUPPORTED;
  return SOLATTN_OK;
}

size_t attention_workspace(int B, int H, int N, int d, int splits) {
  if (splits <= 1) return SOLATTN_WORKSPACE_BYTES;
  const size_t parts = static_cast<size_t>(B) * H * N * splits;
  return SOLATTN_WORKSPACE_BYTES + parts * d * sizeof(float) + parts * sizeof(float2);
}

}  // namespace

extern "C" {

int solattn_rotary_frequencies(int rot, int axes, const int* pairs, double theta, int scaling, double factor,
                               double original, double fast, double slow, uint64_t* freq, int32_t* axis,
                               float* gain) {
  if (!freq || !gain || rot <= 0 || (rot & 1) || axes < 1 || axes > SOLATTN_ROTARY_MAX_AXES) return SOLATTN_ERR_ARG;
  if (axes > 1 && (!pairs || !axis)) return SOLATTN_ERR_ARG;
  if (!(theta > 1.0) || !std::isfinite(theta)) return SOLATTN_ERR_ARG;
  if (scaling < SOLATTN_SCALING_NONE || scaling > SOLATTN_SCALING_YARN) return SOLATTN_ERR_ARG;
  if (scaling != SOLATTN_SCALING_NONE && (!(factor >= 1.0) || !std::isfinite(factor))) return SOLATTN_ERR_ARG;
  if (scaling == SOLATTN_SCALING_YARN && (!(original > 0.0) || !(fast > slow) || !(slow > 0.0) ||
                                          !std::isfinite(original) || !std::isfinite(fast)))
    return SOLATTN_ERR_ARG;
  const int all[1] = {rot / 2};
  const int* count = pairs ? pairs : all;
  int sum = 0;
  for (int a = 0; a < axes; ++a) {
    if (count[a] < 0 || count[a] > rot / 2) return SOLATTN_ERR_ARG;
    if (scaling == SOLATTN_SCALING_NTK && count[a] == 1) return SOLATTN_ERR_ARG;  // its one frequency is theta^0
    sum += count[a];
  }
  if (sum != rot / 2) return SOLATTN_ERR_ARG;
  const double two_pi = 6.283185307179586476925286766559;
  int at = 0;
  for (int a = 0; a < axes; ++a) {
    const double n = count[a];
    const bool ntk = scaling == SOLATTN_SCALING_NTK && count[a] > 1;
    const double base = ntk ? theta * std::pow(factor, 2 * n / (2 * n - 2)) : theta;
    for (int i = 0; i < count[a]; ++i, ++at) {
      double f = std::pow(base, -i / n);
      if (scaling == SOLATTN_SCALING_LINEAR) f /= factor;
      if (scaling == SOLATTN_SCALING_YARN) {
        const double turns = original * f / two_pi;
        double keep = (turns - slow) / (fast - slow);
        keep = keep < 0 ? 0 : (keep > 1 ? 1 : keep);
        f = f / factor * (1 - keep) + f * keep;
      }
      // at most 1 radian per position: below 2^62 of a turn's 2^64
      freq[at] = static_cast<uint64_t>(std::ldexp(f / two_pi, 64) + 0.5);
      if (axis) axis[at] = a;
    }
  }
  *gain = scaling == SOLATTN_SCALING_YARN ? static_cast<float>(0.1 * std::log(factor) + 1.0) : 1.f;
  return SOLATTN_OK;
}

int solattn_rotary(const void* q, const void* k, void* q_out, void* k_out, int dtype, int B, int H, int H_kv, int N,
                   int d, const solattn_strides_t* q_strides, const solattn_strides_t* k_strides,
                   const solattn_strides_t* q_out_strides, const solattn_strides_t* k_out_strides,
                   const solattn_rotary_t* rotary, int inverse, void* stream) {
  if (!q || !q_out || (k && !k_out) || B <= 0 || H <= 0 || N <= 0 || d <= 0 || (k && H_kv <= 0))
    return SOLATTN_ERR_ARG;
  if (!dtype_ok(dtype, true)) return SOLATTN_ERR_UNSUPPORTED;
  if (d > SOLATTN_ROTARY_MAX_DIM || static_cast<long long>(B) * N * d >= (1ll << 31) ||
      static_cast<long long>(H) + (k ? H_kv : 0) > 65535)
    return SOLATTN_ERR_UNSUPPORTED;
  solattn::RotaryArgs a{};
  int rc = check_rotary(rotary, N, d, inverse, &a.t);
  if (rc) return rc;
  const uintptr_t elem = dtype == SOLATTN_F32 ? 3u : 1u;
  const void* ptrs[4] = {q, k, q_out, k ? k_out : nullptr};
  for (const void* p : ptrs)
    if (reinterpret_cast<uintptr_t>(p) & elem) return SOLATTN_ERR_ALIGN;
  if ((rc = tensor_strides(q_strides, B, H, N, d, false, &a.xs[0]))) return rc;
  if ((rc = tensor_strides(q_out_strides, B, H, N, d, true, &a.ys[0]))) return rc;
  if (k) {
    if ((rc = tensor_strides(k_strides, B, H_kv, N, d, false, &a.xs[1]))) return rc;
    if ((rc = tensor_strides(k_out_strides, B, H_kv, N, d, true, &a.ys[1]))) return rc;
  }
  int sms = 0;
  if ((rc = solattn::current_device_sms(&sms))) return rc;
  a.x[0] = q;
  a.x[1] = k;
  a.y[0] = q_out;
  a.y[1] = k ? k_out : nullptr;
  a.heads[0] = H;
  a.heads[1] = k ? H_kv : 0;
  a.dtype = dtype;
  a.B = B;
  a.N = N;
  a.d = d;
  return solattn::launch_rotary(a, sms, static_cast<cudaStream_t>(stream)) == cudaSuccess ? SOLATTN_OK
                                                                                           : SOLATTN_ERR_CUDA;
}

int solattn_rotary_pool(const void* q, const void* k, const void* v, void* q_out, void* k_out, int B, int H, int N,
                        int d, const solattn_strides_t* strides, const solattn_strides_t* out_strides,
                        const solattn_rotary_t* rotary, const solattn_pooled_t* pooled, void* stream) {
  int rc = solattn::check_shape(B, H, N, d);
  if (rc) return rc;
  if ((rc = solattn::check_qkv(q, k, v))) return rc;
  if (!q_out || !k_out) return SOLATTN_ERR_ARG;
  if (!solattn::aligned16(q_out) || !solattn::aligned16(k_out)) return SOLATTN_ERR_ALIGN;
  solattn::RotaryPoolArgs a{};
  if ((rc = check_rotary(rotary, N, d, 0, &a.t))) return rc;
  if (rotary->rot != d) return SOLATTN_ERR_UNSUPPORTED;
  if ((rc = solattn::resolve_strides(strides, B, H, N, d, &a.st))) return rc;
  if ((rc = solattn::resolve_strides(out_strides, B, H, N, d, &a.ys))) return rc;
  if ((rc = solattn::check_pooled(pooled))) return rc;
  if (static_cast<long long>(B) * H > 65535) return SOLATTN_ERR_UNSUPPORTED;  // grid rows of the key statistics
  int sms = 0;
  if ((rc = solattn::current_device_sms(&sms))) return rc;
  a.x[0] = static_cast<const uint16_t*>(q);
  a.x[1] = static_cast<const uint16_t*>(k);
  a.x[2] = static_cast<const uint16_t*>(v);
  a.y[0] = static_cast<uint16_t*>(q_out);
  a.y[1] = static_cast<uint16_t*>(k_out);
  a.bar[0] = pooled->qbar;
  a.bar[1] = pooled->kbar;
  a.bar[2] = pooled->vbar;
  a.bar16[1] = static_cast<uint16_t*>(pooled->kbar16);
  a.bar16[2] = static_cast<uint16_t*>(pooled->vbar16);
  a.B = B;
  a.H = H;
  a.N = N;
  a.d = d;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (solattn::launch_rotary_pool(a, sms, s) != cudaSuccess) return SOLATTN_ERR_CUDA;
  const int nb = (N + SOLATTN_BLOCK - 1) / SOLATTN_BLOCK;
  return solattn::launch_key_stats(pooled->kbar, pooled->kmean, pooled->kcov, B * H, nb, d, s) == cudaSuccess
             ? SOLATTN_OK
             : SOLATTN_ERR_CUDA;
}

int solattn_cache_append(const void* k, const void* v, int dtype, int B, int N, const solattn_strides_t* strides,
                         const solattn_cache_t* cache, const int32_t* table, int columns, long long table_stride,
                         const int32_t* lengths, const int32_t* counts, void* workspace, size_t workspace_bytes,
                         void* stream) {
  if (!k || !v || B <= 0 || N <= 0) return SOLATTN_ERR_ARG;
  if (!dtype_ok(dtype, true)) return SOLATTN_ERR_UNSUPPORTED;
  CacheView cv;
  int rc = check_cache(cache, table, columns, table_stride, lengths, counts, &cv);
  if (rc) return rc;
  if (B > 32767 || cache->heads > 65535) return SOLATTN_ERR_UNSUPPORTED;  // grid limits
  if (!solattn::aligned16(k) || !solattn::aligned16(v)) return SOLATTN_ERR_ALIGN;
  solattn::CacheAppendArgs a{};
  if ((rc = tensor_strides(strides, B, cache->heads, N, cache->d, false, &a.st))) return rc;
  if (!multiple_of_8(a.st)) return SOLATTN_ERR_ARG;
  if (workspace && workspace_bytes < SOLATTN_WORKSPACE_BYTES) return SOLATTN_ERR_WORKSPACE;
  if (!solattn::aligned16(workspace)) return SOLATTN_ERR_ALIGN;
  int sms = 0;
  if ((rc = solattn::current_device_sms(&sms))) return rc;
  a.x[0] = k;
  a.x[1] = v;
  a.data[0] = static_cast<uint8_t*>(cache->k);
  a.data[1] = static_cast<uint8_t*>(cache->v);
  a.scale[0] = cache->k_scale;
  a.scale[1] = cache->v_scale;
  a.page_stride = cv.page_stride;
  a.scale_stride = cv.scale_stride;
  a.table_stride = cv.table_stride;
  a.table = table;
  a.lengths = lengths;
  a.counts = counts;
  a.dtype = dtype;
  a.pages = cache->pages;
  a.columns = columns;
  a.B = B;
  a.H = cache->heads;
  a.N = N;
  a.d = cache->d;
  a.status = static_cast<solattn::DeviceStatus*>(workspace);
  return solattn::launch_cache_append(a, static_cast<cudaStream_t>(stream)) == cudaSuccess ? SOLATTN_OK
                                                                                            : SOLATTN_ERR_CUDA;
}

int solattn_cache_workspace_bytes(int B, int H, int N, int d, int H_kv, int columns, size_t* bytes) {
  if (!bytes) return SOLATTN_ERR_ARG;
  const int rc = check_attention_shape(B, H, N, d, H_kv, columns);
  if (rc) return rc;
  *bytes = attention_workspace(B, H, N, d, solattn::cache_plan(B, H, H_kv, N, d, columns).splits);
  return SOLATTN_OK;
}

int solattn_cache_attention(const void* q, int dtype, int B, int H, int N, int d, const solattn_strides_t* strides,
                            const solattn_cache_t* cache, const int32_t* table, int columns, long long table_stride,
                            const int32_t* lengths, const int32_t* counts, int causal, float scale, void* out,
                            const solattn_strides_t* out_strides, float* lse, void* workspace, size_t workspace_bytes,
                            void* stream) {
  if (!q || !out || !cache) return SOLATTN_ERR_ARG;
  int rc = check_attention_shape(B, H, N, d, cache->heads, columns);
  if (rc) return rc;
  if (!dtype_ok(dtype, false)) return SOLATTN_ERR_UNSUPPORTED;
  if (cache->d != d || !(scale >= 0.f) || !(scale < 0x1p127f)) return SOLATTN_ERR_ARG;  // finite in log2 units too
  CacheView cv;
  if ((rc = check_cache(cache, table, columns, table_stride, lengths, counts, &cv))) return rc;
  if (!solattn::aligned16(q) || !solattn::aligned16(out) || !solattn::aligned4(lse)) return SOLATTN_ERR_ALIGN;
  solattn::CacheAttnArgs a{};
  if ((rc = tensor_strides(strides, B, H, N, d, false, &a.st))) return rc;
  if ((rc = tensor_strides(out_strides, B, H, N, d, true, &a.ost))) return rc;
  if (!multiple_of_8(a.st) || !multiple_of_8(a.ost)) return SOLATTN_ERR_ARG;
  const solattn::CachePlan plan = solattn::cache_plan(B, H, cache->heads, N, d, columns);
  if (!workspace || workspace_bytes < attention_workspace(B, H, N, d, plan.splits)) return SOLATTN_ERR_WORKSPACE;
  if (!solattn::aligned16(workspace)) return SOLATTN_ERR_ALIGN;
  int sms = 0;
  if ((rc = solattn::current_device_sms(&sms))) return rc;
  a.q = static_cast<const uint16_t*>(q);
  a.out = static_cast<uint16_t*>(out);
  a.lse = lse;
  a.k = static_cast<const uint8_t*>(cache->k);
  a.v = static_cast<const uint8_t*>(cache->v);
  a.k_scale = cache->k_scale;
  a.v_scale = cache->v_scale;
  a.table = table;
  a.lengths = lengths;
  a.counts = counts;
  a.page_stride = cv.page_stride;
  a.scale_stride = cv.scale_stride;
  a.table_stride = cv.table_stride;
  a.scale_log2 = (scale == 0.f ? 1.f / std::sqrt(static_cast<float>(d)) : scale) * 1.4426950408889634f;
  a.dtype = dtype;
  a.pages = cache->pages;
  a.columns = columns;
  a.B = B;
  a.H = H;
  a.Hk = cache->heads;
  a.N = N;
  a.d = d;
  a.group = H / cache->heads;
  while ((1ll << a.group_shift) < a.group) ++a.group_shift;
  a.group_mul = static_cast<uint32_t>((1ull << 32) * ((1ull << a.group_shift) - a.group) / a.group + 1);
  a.causal = causal != 0;
  a.splits = plan.splits;
  a.longest_first = plan.longest_first;
  char* ws = static_cast<char*>(workspace) + SOLATTN_WORKSPACE_BYTES;
  a.part_o = reinterpret_cast<float*>(ws);
  a.part_ml = reinterpret_cast<float2*>(a.part_o + static_cast<size_t>(B) * H * N * plan.splits * d);
  a.status = static_cast<solattn::DeviceStatus*>(workspace);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  cudaError_t e = plan.step ? solattn::launch_cache_step(a, s) : solattn::launch_cache_chunk(a, s);
  if (e == cudaSuccess && plan.splits > 1) e = solattn::launch_cache_join(a, s);
  return e == cudaSuccess ? SOLATTN_OK : SOLATTN_ERR_CUDA;
}

}  // extern "C"

#ifdef SOLATTN_TEST_HOOKS
// Test builds only: 1 takes the kernel of few rows for every call that fits its
// grid, 2 the kernel of many rows, 0 what the estimates say.
static int g_hook_cache_kernel = 0;
extern "C" void solattn_test_set_cache_kernel(int which) { g_hook_cache_kernel = which; }
#endif

namespace solattn {

// Estimates in microseconds of the two attention kernels, each at the number of
// parts of the key axis that it does best with; the cheaper one is launched.
// Rows of one key head go in tiles of 16 that read the cache once each, or in
// tiles of 256 on tcgen05: the first starts and finishes sooner and spreads short
// calls over more CTAs, the second reads and converts the cache 16 times less.
// 300 queries x 4 heads, 500 keys: 8.4 and 17.7 us; 2 x 285 queries of 20 heads
// (4 key heads), 900 keys: 39.5 and 32.3 us; 64 key heads of 16384 tokens: 32 rows
// 179 and 278 us, 48 rows 257 and 280, 64 rows 331 and 280. Over 70 calls drawn
// between 49 and 12000 rows and 2 and 8000 keys the estimates took the faster one
// each time, 1.29 times faster than the second alone.
CachePlan cache_plan(int B, int H, int Hk, int N, int d, int columns) {
  constexpr int kSms = 148;
  const long long rows = static_cast<long long>(N) * (H / Hk);
  auto ceil_div = [](long long x, long long y) { return (x + y - 1) / y; };
  CachePlan step{true, 1, false}, chunk{false, 1, false};
  double step_cost = 0, chunk_cost = 0;
  {
    // Three CTAs per SM: a part costs about 5 us to start and finish and 0.75 us
    // per page, all parts together what memory gives (5.9 TB/s, and the start of
    // every wave but the first); among several sequences, which differ in length,
    // some of a part is left at the end. Counts that fill one to eight waves are
    // compared: 8 key heads of 65536 tokens take 33 us in 37 parts, 43 us in 74; 32
    // sequences of 32000 tokens take 388 us whole, 331 us in 5 parts.
    const long long units = static_cast<long long>(B) * Hk * ceil_div(rows, 16);
    const double memory = static_cast<double>(units) * columns * 128 * d / 5.9e6;
    for (int w = 0; w <= 8; ++w) {
      const long long s = w == 0 ? 1 : std::min<long long>(3ll * kSms * w / units, columns);
      if (s < 1) continue;
      const double join = s == 1 ? 0 : 2 + static_cast<double>(B) * H * N * s * d * 8 / 6e6;
      const double part = 5 + 0.75 * ceil_div(columns, s);
      const long long waves = ceil_div(units * s, 3 * kSms);
      const double cost = std::max(waves * part, memory + 5 * (waves - 1)) + join + (B > 1 ? 0.3 * part : 0);
      if (w == 0 || cost < step_cost) {
        step_cost = cost;
        step.splits = static_cast<int>(s);
        step.longest_first = B > 1 && B <= 64 && waves > 1;
      }
    }
  }
  {
    // One CTA per SM: a part of the key axis costs about 9 us to start and finish
    // and 2.5 us per key tile (two pages), parts run in waves of 148, and what is
    // joined is written and read once at about 6 TB/s. The split with the least
    // sum is taken (120 CTAs of 591 key tiles, 8 heads of 3600 queries over 75600
    // keys: 1466 us in one part, 1325 us in 6). With several sequences that fill
    // the GPU by their upper bounds the key axis stays whole: shorter sequences
    // leave fewer CTAs than that (3 of up to 1111 queries: 62 us, 95 us in 2).
    const long long units = static_cast<long long>(B) * Hk * ceil_div(rows, 256), tiles = ceil_div(columns, 2);
    for (int s = 1; s <= 16 && (s == 1 || (s * 2 <= tiles && (B == 1 || units < kSms))); ++s) {
      const double join = s == 1 ? 0 : 3 + static_cast<double>(B) * H * N * s * d * 8 / 6e6;
      const double cost = ceil_div(units * s, kSms) * (9 + 2.5 * ceil_div(tiles, s)) + join;
      if (s == 1 || cost < chunk_cost) {
        chunk_cost = cost;
        chunk.splits = s;
        chunk.longest_first = B > 1 && B <= 64 && units * s > kSms;
      }
    }
  }
  // Calls of several waves over several sequences take the long ones first, so
  // that what is left at the end is short (every CTA ranks the lengths, two per
  // lane, hence 64 sequences at most): 32 sequences of 8000 to 32700 tokens 249 to
  // 209 us, 8 of 1000 to 8000 with 500 queries 232 to 206 us; equal lengths are
  // not slower (334 and 331 us).
  const bool fits = ceil_div(rows, 16) * Hk <= 65535;  // the first kernel's grid
#ifdef SOLATTN_TEST_HOOKS
  if (g_hook_cache_kernel == 1 && fits) return step;
  if (g_hook_cache_kernel == 2) return chunk;
#endif
  return fits && step_cost <= chunk_cost ? step : chunk;
}

}  // namespace solattn
