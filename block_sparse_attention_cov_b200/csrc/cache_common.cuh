// cache_common.cuh -- what the kernels on the 8-bit key/value cache share: the
// cache's address arithmetic and checks, e4m3 conversion, and the softmax
// reference of the two attention kernels (cache_step.cu, cache_chunk.cu).
//
// Cache: pages of 64 tokens, e4m3 [pages][H_kv][64][d], one fp32 scale per page
// and head for keys (ks) and one for values (vs). With t_u the score of a key in
// log2 units and v8 its e4m3 value row, a query's output is
//     sum_u 2^t_u vs_u v8_u / sum_u 2^t_u,
// and the kernels evaluate it with P_u = 2^(t_u + log2 vs_u - M), M a running
// reference of the row:
//     O = sum_u P_u v8_u,   l = sum_u P_u / vs_u,   out = O / l,
//     lse = ln2 (M + log2 l),
// so both scales cost nothing per element: ks rides on the multiply that turns a
// dot product into log2 units, log2 vs on the same instruction's addend, and
// 1 / vs on the page's sum.
//
// P is rounded to fp16 for the value product (11 bits against bf16's 8, and
// e4m3 is exact in fp16); 2^kPBias lifts the range and the lazy reference (raised
// only when a row's maximum passes it by kSlack) keeps P at 2^15 at most, so
// that P down to 2^-29 of the row's largest is held. P is a weight times a value
// scale: were that scale the page's as it is, one page with a large value (2^29
// times its neighbours') would push the others' P out of fp16 even for rows and
// columns in which that page holds nothing. So value scales are taken relative
// to a unit, vs / U, and where a page's differs from U by more than 2^kUnitSlack,
// U becomes that page's scale and O, which is in fp32, is brought to it (rare:
// pages of one head differ by less; the warp that fetches the pages works the
// units out: 1,213 us for 8 heads x 3,600 queries x 75,600 keys, 1,218 without).
// With all scales within 2^kUnitSlack of U, weights down to 2^-17 of the row's
// largest are held whatever the scales are, down to 2^-29 where they are equal.
//
// Queries are scaled by a power of two per row before they are rounded to fp16:
// exact for fp16 inputs, and for bf16 inputs down to 2^-23 of the row's largest
// element.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <climits>
#include <cstdint>

#include "kernels.h"
#include "ptx.cuh"

namespace solattn {
namespace {

constexpr int kPage = 64;
constexpr float kPBias = 5.f;
constexpr float kSlack = 10.f;
constexpr int kUnitSlack = 6;
constexpr float kLog2eC = 1.4426950408889634f;
constexpr float kLn2C = 0.6931471805599453f;
constexpr unsigned int kErrPage = 9;  // == SOLATTN_ERR_PAGE

__device__ __forceinline__ void report_page(DeviceStatus* st, uint32_t unit) {
  if (st && atomicCAS(&st->error, 0u, kErrPage) == 0u) st->unit = unit;
}

// Tokens in the cache and new queries of sequence b, inside what the table and
// the tensors hold; a length or count outside is reported and clamped.
struct Extent {
  int len, cnt;
};
__device__ __forceinline__ Extent extent(const CacheAttnArgs& a, int b, bool report) {
  const int len = a.lengths[b], cnt = a.counts ? a.counts[b] : a.N;
  const long long cap = static_cast<long long>(a.columns) * kPage;
  Extent e;
  e.len = len < 0 ? 0 : (len > cap ? static_cast<int>(cap) : len);
  e.cnt = cnt < 0 ? 0 : (cnt > a.N ? a.N : cnt);
  if (report && (e.len != len || e.cnt != cnt)) report_page(a.status, b);
  return e;
}

// The sequence that is the n-th longest (of equals, the first): a call of several
// waves that takes the long sequences first ends more evenly. B <= 64; every lane
// of a warp calls it and gets the same answer.
__device__ __forceinline__ int nth_longest(const CacheAttnArgs& a, int n, int lane) {
  const int v0 = lane < a.B ? __ldg(a.lengths + lane) : INT_MIN;
  const int v1 = lane + 32 < a.B ? __ldg(a.lengths + lane + 32) : INT_MIN;
  int r0 = 0, r1 = 0;
#pragma unroll 4
  for (int j = 0; j < min(a.B, 32); ++j) {
    const int w = __shfl_sync(0xffffffffu, v0, j);
    r0 += w > v0 || (w == v0 && j < lane);
    r1 += w >= v1;
  }
#pragma unroll 4
  for (int j = 32; j < a.B; ++j) {
    const int w = __shfl_sync(0xffffffffu, v1, j - 32);
    r0 += w > v0;
    r1 += w > v1 || (w == v1 && j < lane + 32);
  }
  const unsigned int m0 = __ballot_sync(0xffffffffu, lane < a.B && r0 == n);
  const unsigned int m1 = __ballot_sync(0xffffffffu, lane + 32 < a.B && r1 == n);
  return m0 ? __ffs(m0) - 1 : 31 + __ffs(m1);
}

// Query token and head within its group of a row (token-major).
__device__ __forceinline__ void row_place(const CacheAttnArgs& a, int r, int* i, int* g) {
  const uint32_t u = static_cast<uint32_t>(r);
  *i = static_cast<int>((__umulhi(a.group_mul, u) + u) >> a.group_shift);
  *g = r - *i * a.group;
}

// Keys seen by query i of a sequence: all of them, or (causal) those up to its
// own place, the queries being the sequence's last cnt tokens.
__device__ __forceinline__ int key_limit(const Extent& e, int causal, int i) {
  if (!causal) return e.len;
  const int l = e.len - e.cnt + i + 1;
  return l < 0 ? 0 : (l > e.len ? e.len : l);
}

// Four e4m3 values to two fp16 pairs (exact).
__device__ __forceinline__ void e4m3x4_f16(uint32_t v, uint32_t& lo, uint32_t& hi) {
  asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, a;\n\tcvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
      : "=r"(lo), "=r"(hi)
      : "r"(v));
}

// Lets the joining kernel of a split call set itself up; it waits for this
// kernel's end before it reads a part.
__device__ __forceinline__ void start_join(const CacheAttnArgs& a) {
  if (a.splits > 1) asm volatile("griddepcontrol.launch_dependents;");
}

// Some byte of w is an e4m3 NaN (0x7f or 0xff).
__device__ __forceinline__ bool has_nan8(uint32_t w) {
  return (((w & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u) != 0;
}
// w with its NaN bytes zeroed.
__device__ __forceinline__ uint32_t drop_nan8(uint32_t w) {
  const uint32_t n = (((w & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u) >> 7;  // 1 in each NaN byte
  return w & ~(n * 0xffu);
}

__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// A 16-bit element pair as floats.
template <typename T>
__device__ __forceinline__ float2 unpack2(uint32_t w);
template <>
__device__ __forceinline__ float2 unpack2<__nv_bfloat16>(uint32_t w) {
  return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}
template <>
__device__ __forceinline__ float2 unpack2<__half>(uint32_t w) {
  return __half22float2(*reinterpret_cast<const __half2*>(&w));
}
template <typename T>
__device__ __forceinline__ uint32_t pack2(float lo, float hi);
template <>
__device__ __forceinline__ uint32_t pack2<__nv_bfloat16>(float lo, float hi) {
  return pack_bf16x2(lo, hi);
}
template <>
__device__ __forceinline__ uint32_t pack2<__half>(float lo, float hi) {
  return pack_f16x2(lo, hi);
}

// Power of two that brings a row with largest magnitude amax to [2^9, 2^10), and
// its inverse. An infinite or NaN row keeps the factor 1 and comes out NaN.
__device__ __forceinline__ void row_factor(float amax, float* mul, float* inv) {
  int e = static_cast<int>((__float_as_uint(amax) >> 23) & 255u) - 127;
  if (amax == 0.f || e > 127) e = 9;
  if (e < -110) e = -110;
  *mul = __int_as_float((127 + 9 - e) << 23);
  *inv = __int_as_float((127 + e - 9) << 23);
}

// Units of the value scales of 32 pages, lane i having page i's scale (0: not
// there): the biased exponent of a power of two, from `unit`, that of the page
// before (0: there was none), which becomes the last page's. Warp-collective.
__device__ __forceinline__ int page_units(float vs, int& unit, int lane) {
  const int x = (__float_as_int(vs) >> 23) & 255;
  const bool known = x != 0 && x < 254;  // neither infinite nor NaN
  const unsigned int m = __ballot_sync(0xffffffffu, known);
  if (unit == 0 && m) unit = __shfl_sync(0xffffffffu, x, __ffs(m) - 1);
  int mine = unit;
  unsigned int far = __ballot_sync(0xffffffffu, known && abs(x - unit) > kUnitSlack);
  while (far) {  // rare
    const int first = __ffs(far) - 1;
    unit = __shfl_sync(0xffffffffu, x, first);
    if (lane >= first) mine = unit;
    far = __ballot_sync(0xffffffffu, known && lane > first && abs(x - unit) > kUnitSlack);
  }
  return mine;
}
// 2^(from - to) of two units: what O is multiplied by when the unit changes.
__device__ __forceinline__ float unit_turn(int from, int to) {
  return __int_as_float((127 + min(max(from - to, -126), 126)) << 23);
}
__device__ __forceinline__ float unit_inverse(int unit) { return __int_as_float((254 - unit) << 23); }

// What a page's scores and weights are multiplied by, from its scales, that of
// the values in their unit; vs = 0 stands for a page that is not there, whose
// tokens then weigh nothing.
struct PageScale {
  float ck;    // ks * scale * log2(e)
  float ev;    // log2(vs)
  float vinv;  // 1 / vs
};
__device__ __forceinline__ PageScale page_scale(const CacheAttnArgs& a, float ks, float vs) {
  PageScale s{0.f, -INFINITY, 0.f};
  if (vs != 0.f) {
    s.ck = ks * a.scale_log2;
    s.ev = __log2f(vs);
    s.vinv = ex2_approx(-s.ev);  // a power of two, as append writes it, comes out exactly
  }
  return s;
}

// Page of block `col` of sequence b, or -1 (reported) when the table's entry is
// outside the cache.
__device__ __forceinline__ int page_of(const CacheAttnArgs& a, int b, int col) {
  const int p = __ldg(a.table + b * a.table_stride + col);
  if (p >= 0 && p < a.pages) return p;
  report_page(a.status, b);
  return -1;
}

// One partial result per row and split: O unnormalised, its reference and sum.
__device__ __forceinline__ long long partial_row(const CacheAttnArgs& a, int b, int head, int i, int split) {
  return ((static_cast<long long>(b) * a.H + head) * a.N + i) * a.splits + split;
}

}  // namespace
}  // namespace solattn
