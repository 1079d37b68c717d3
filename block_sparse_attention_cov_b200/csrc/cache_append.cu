// cache_append.cu -- new tokens' keys and values into the 8-bit cache.
//
// Every page holds 64 tokens of every head in e4m3 with one scale per page and
// head, the smallest power of two that brings the page's largest magnitude to
// 448 or below (2^-32 .. 2^32). A power of two costs an e4m3 value nothing (its
// relative step does not depend on the scale) and makes the division exact; and
// when a later token of an open page is larger, the page's older tokens are
// brought to the new scale by an exact shift, save where a value sinks below
// e4m3's normal range. Values that are not finite are held as NaN and do not
// count towards the scale.
//
// Bound by memory (2 or 4 bytes read and 1 written per element). One CTA per
// page touched, head and tensor: the new rows stay in registers, as they were
// read, between the maximum and the conversion. Their loads go out before the
// page's number is looked up, and the maximum is taken on the bits (magnitudes of
// 16-bit elements in pairs), so that what a thread holds is 16 bytes a row and
// enough CTAs fit an SM to cover the latency.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <cmath>
#include <cstdint>

#include "kernels.h"
#include "ptx.cuh"

namespace solattn {

namespace {

constexpr int kPage = 64;
constexpr unsigned int kErrPage = 9;  // == SOLATTN_ERR_PAGE

// Eight elements of a row as they lie in memory: their largest magnitude's bits,
// and their values.
template <typename T>
struct Raw {  // 16-bit types
  uint4 w;
  __device__ __forceinline__ void load(const T* p) { w = __ldg(reinterpret_cast<const uint4*>(p)); }
  __device__ __forceinline__ void zero() { w = make_uint4(0, 0, 0, 0); }
  __device__ __forceinline__ uint32_t top() const {
    const uint32_t m = __vmaxu2(__vmaxu2(w.x & 0x7fff7fffu, w.y & 0x7fff7fffu),
                                __vmaxu2(w.z & 0x7fff7fffu, w.w & 0x7fff7fffu));
    return max(m & 0xffffu, m >> 16);
  }
  __device__ __forceinline__ void get(float (&f)[8]) const;
  static __device__ __forceinline__ float value(uint32_t bits);  // of a magnitude
};
template <>
__device__ __forceinline__ void Raw<__nv_bfloat16>::get(float (&f)[8]) const {
  const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = __uint_as_float(u[i] << 16);
    f[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
  }
}
template <>
__device__ __forceinline__ float Raw<__nv_bfloat16>::value(uint32_t bits) { return __uint_as_float(bits << 16); }
template <>
__device__ __forceinline__ void Raw<__half>::get(float (&f)[8]) const {
  const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 v = __half22float2(*reinterpret_cast<const __half2*>(&u[i]));
    f[2 * i] = v.x;
    f[2 * i + 1] = v.y;
  }
}
template <>
__device__ __forceinline__ float Raw<__half>::value(uint32_t bits) {
  return __half2float(__ushort_as_half(static_cast<unsigned short>(bits)));
}
template <>
struct Raw<float> {
  uint4 w, x;
  __device__ __forceinline__ void load(const float* p) {
    w = __ldg(reinterpret_cast<const uint4*>(p));
    x = __ldg(reinterpret_cast<const uint4*>(p) + 1);
  }
  __device__ __forceinline__ void zero() { w = x = make_uint4(0, 0, 0, 0); }
  __device__ __forceinline__ uint32_t top() const {
    constexpr uint32_t M = 0x7fffffffu;
    return max(max(max(w.x & M, w.y & M), max(w.z & M, w.w & M)), max(max(x.x & M, x.y & M), max(x.z & M, x.w & M)));
  }
  __device__ __forceinline__ void get(float (&f)[8]) const {
    const uint32_t u[8] = {w.x, w.y, w.z, w.w, x.x, x.y, x.z, x.w};
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = __uint_as_float(u[i]);
  }
  static __device__ __forceinline__ float value(uint32_t bits) { return __uint_as_float(bits); }
};

__device__ __forceinline__ uint32_t to_e4m3x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ uint2 to_e4m3x8(const float (&f)[8]) {
  return make_uint2(to_e4m3x2(f[0], f[1]) | (to_e4m3x2(f[2], f[3]) << 16),
                    to_e4m3x2(f[4], f[5]) | (to_e4m3x2(f[6], f[7]) << 16));
}
__device__ __forceinline__ float2 from_e4m3x2(uint32_t v) {
  uint32_t r;
  asm("{\n\t.reg .b16 h;\n\tcvt.u16.u32 h, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, h;\n\t}" : "=r"(r) : "r"(v));
  return __half22float2(*reinterpret_cast<const __half2*>(&r));
}

// Exponent of the smallest power of two s with amax <= 448 s (448 = 0.875 2^9),
// kept in [-32, 32]. amax is finite.
__device__ __forceinline__ int scale_exponent(float amax) {
  const uint32_t bits = __float_as_uint(amax);
  // amax = (1 + m) 2^x: amax <= 1.75 2^(8 + e) at e = x - 8 when 1 + m <= 1.75
  const int x = static_cast<int>(bits >> 23) - 127;
  const int e = x - 8 + ((bits & 0x7fffffu) > 0x600000u ? 1 : 0);
  return min(32, max(-32, e));
}
__device__ __forceinline__ float pow2i(int e) { return __int_as_float((127 + e) << 23); }

template <typename T, int D>
__global__ void __launch_bounds__(128) cache_append_kernel(const CacheAppendArgs a) {
  constexpr int CH = D / 8, RG = 128 / CH, RPT = kPage / RG;
  __shared__ uint32_t wmax[4];
  const int h = blockIdx.y, b = blockIdx.z >> 1, which = blockIdx.z & 1;
  const int tid = threadIdx.x, c = tid % CH, g = tid / CH;
  const long long cap = static_cast<long long>(a.columns) * kPage;
  int start = __ldg(a.lengths + b), cnt = a.counts ? __ldg(a.counts + b) : a.N;
  bool bad = start < 0 || cnt < 0 || cnt > a.N || static_cast<long long>(start) + cnt > cap;
  if (bad) {  // reported; what fits is written
    cnt = max(0, min(cnt, a.N));
    if (start < 0 || start > cap) cnt = 0, start = 0;
    cnt = static_cast<int>(min(static_cast<long long>(cnt), cap - start));
  }
  const int col = start / kPage + blockIdx.x;
  const int lo = max(start, col * kPage), hi = min(static_cast<long long>(start) + cnt, (col + 1ll) * kPage);
  if (lo >= hi) {
    if (bad && tid == 0 && a.status && atomicCAS(&a.status->error, 0u, kErrPage) == 0u) a.status->unit = b;
    return;
  }
  const int first = lo - col * kPage, last = hi - col * kPage;  // rows of the page that are new
  const T* src = static_cast<const T*>(a.x[which]) + b * a.st.b + h * a.st.h + c * 8;
  int page = __ldg(a.table + b * a.table_stride + col);
  Raw<T> x[RPT];
#pragma unroll
  for (int r = 0; r < RPT; ++r) {
    const int row = g + r * RG;
    if (row >= first && row < last) x[r].load(src + static_cast<long long>(row + col * kPage - start) * a.st.n);
    else x[r].zero();
  }
  if (page < 0 || page >= a.pages) bad = true, page = -1;
  if (bad && tid == 0 && a.status && atomicCAS(&a.status->error, 0u, kErrPage) == 0u) a.status->unit = b;
  if (page < 0) return;
  uint8_t* dst = a.data[which] + page * a.page_stride + static_cast<long long>(h) * kPage * D + c * 8;
  float* sp = a.scale[which] + page * a.scale_stride + h;
  const float old_scale = first > 0 ? *sp : 0.f;
  uint32_t top = 0;
#pragma unroll
  for (int r = 0; r < RPT; ++r) top = max(top, x[r].top());
  top = __reduce_max_sync(0xffffffffu, top);
  if ((tid & 31) == 0) wmax[tid >> 5] = top;
  __syncthreads();  // every thread has read the old scale too
  float mx = Raw<T>::value(max(max(wmax[0], wmax[1]), max(wmax[2], wmax[3])));
  const bool finite = mx < INFINITY;
  if (!finite) {  // rare: the largest finite magnitude, element by element
    mx = 0.f;
#pragma unroll
    for (int r = 0; r < RPT; ++r) {
      float f[8];
      x[r].get(f);
#pragma unroll
      for (int e = 0; e < 8; ++e) mx = fabsf(f[e]) < INFINITY ? fmaxf(mx, fabsf(f[e])) : mx;
    }
    mx = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(mx)));
    __syncthreads();  // the first maxima have been read
    if ((tid & 31) == 0) wmax[tid >> 5] = __float_as_uint(mx);
    __syncthreads();
    mx = __uint_as_float(max(max(wmax[0], wmax[1]), max(wmax[2], wmax[3])));
  }
  const float scale = fmaxf(pow2i(scale_exponent(mx)), old_scale);
  const float inv = 1.f / scale;
  if (tid == 0) *sp = scale;
#pragma unroll
  for (int r = 0; r < RPT; ++r) {
    const int row = g + r * RG;
    if (row >= first && row < last) {
      float f[8];
      x[r].get(f);
#pragma unroll
      for (int e = 0; e < 8; ++e) f[e] = finite || fabsf(f[e]) < INFINITY ? f[e] * inv : NAN;
      *reinterpret_cast<uint2*>(dst + row * D) = to_e4m3x8(f);
    }
  }
  if (first > 0 && scale > old_scale) {  // the older tokens follow the page's new scale
    const float k = old_scale * inv;
    for (int row = g; row < first; row += RG) {
      const uint2 w = *reinterpret_cast<const uint2*>(dst + row * D);
      const float2 v0 = from_e4m3x2(w.x & 0xffffu), v1 = from_e4m3x2(w.x >> 16);
      const float2 v2 = from_e4m3x2(w.y & 0xffffu), v3 = from_e4m3x2(w.y >> 16);
      const float y[8] = {v0.x * k, v0.y * k, v1.x * k, v1.y * k, v2.x * k, v2.y * k, v3.x * k, v3.y * k};
      *reinterpret_cast<uint2*>(dst + row * D) = to_e4m3x8(y);
    }
  }
}

template <typename T>
cudaError_t launch_append_t(const CacheAppendArgs& a, cudaStream_t stream) {
  // a run of N tokens that starts anywhere in a page touches at most this many
  const dim3 grid((a.N + kPage - 2) / kPage + 1, a.H, 2 * a.B);
  if (a.d == 64) cache_append_kernel<T, 64><<<grid, 128, 0, stream>>>(a);
  else cache_append_kernel<T, 128><<<grid, 128, 0, stream>>>(a);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_cache_append(const CacheAppendArgs& a, cudaStream_t stream) {
  if (a.dtype == kF32) return launch_append_t<float>(a, stream);
  if (a.dtype == kF16) return launch_append_t<__half>(a, stream);
  return launch_append_t<__nv_bfloat16>(a, stream);
}

}  // namespace solattn
