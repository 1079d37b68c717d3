// rotary.cu -- rotary positions on queries and keys, alone and fused with the
// pooled statistics of the sparse forward.
//
// Pair p of a token at position m (on the pair's axis) turns by the angle
// m f_p and is scaled by `gain`:
//     y0 = gain (x0 cos - x1 sin),   y1 = gain (x1 cos + x0 sin).
// The transpose (the gradient's direction) turns the other way.
//
// Angles. f_p is stored as the 64-bit fraction F_p of a turn, so m F_p mod 2^64
// IS the angle's fraction of a turn: the reduction modulo 2 pi is the integer
// product's own wrap, exact at every position (in fp32 the product alone is off
// by 0.008 rad at position 262,143). Its top 32 bits go to sincospif.
//
// rotary_kernel is bound by memory: one thread takes one unit of a row (one
// 16-byte chunk of interleaved pairs, or the two chunks that hold eight halves'
// pairs) of one token, forms its angles once and walks over the heads with
// them in registers, four heads' loads in flight, so neither the sines nor the
// tables are paid per head and nothing goes through shared memory.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <cstdint>

#include "kernels.h"

namespace solattn {

namespace {

__device__ __forceinline__ void pair_angle(const RotaryTable& t, const int32_t* pos, int pair, float* c, float* s) {
  const int ax = t.axis ? min(max(__ldg(t.axis + pair), 0), t.axes - 1) : 0;
  const long long m = __ldg(pos + ax);
  unsigned long long turn = static_cast<unsigned long long>(m) * __ldg(t.freq + pair);
  if (t.inverse) turn = 0ull - turn;
  // signed top 32 bits: a fraction in [-1/2, 1/2) of a turn; sincospif takes half turns
  const float half_turns = static_cast<float>(static_cast<int>(turn >> 32)) * 0x1p-31f;
  float sn, cs;
  sincospif(half_turns, &sn, &cs);
  *c = cs * t.gain;
  *s = sn * t.gain;
}

template <typename T>
struct Vec16;  // 16 bytes of T as floats and back
template <>
struct Vec16<float> {
  static constexpr int E = 4;
  static __device__ __forceinline__ void get(const uint4& w, float (&f)[4]) {
    f[0] = __uint_as_float(w.x); f[1] = __uint_as_float(w.y); f[2] = __uint_as_float(w.z); f[3] = __uint_as_float(w.w);
  }
  static __device__ __forceinline__ uint4 put(const float (&f)[4]) {
    return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
  }
};
template <>
struct Vec16<__nv_bfloat16> {
  static constexpr int E = 8;
  static __device__ __forceinline__ void get(const uint4& w, float (&f)[8]) {
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[2 * i] = __uint_as_float(u[i] << 16);
      f[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
    }
  }
  static __device__ __forceinline__ uint4 put(const float (&f)[8]) {
    uint32_t u[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __nv_bfloat162 h = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
      u[i] = *reinterpret_cast<const uint32_t*>(&h);
    }
    return make_uint4(u[0], u[1], u[2], u[3]);
  }
};
template <>
struct Vec16<__half> {
  static constexpr int E = 8;
  static __device__ __forceinline__ void get(const uint4& w, float (&f)[8]) {
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 p = __half22float2(*reinterpret_cast<const __half2*>(&u[i]));
      f[2 * i] = p.x;
      f[2 * i + 1] = p.y;
    }
  }
  static __device__ __forceinline__ uint4 put(const float (&f)[8]) {
    uint32_t u[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __half2 h = __floats2half2_rn(f[2 * i], f[2 * i + 1]);
      u[i] = *reinterpret_cast<const uint32_t*>(&h);
    }
    return make_uint4(u[0], u[1], u[2], u[3]);
  }
};

__device__ __forceinline__ float to_f(float x) { return x; }
__device__ __forceinline__ float to_f(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ float to_f(__half x) { return __half2float(x); }
template <typename T>
__device__ __forceinline__ T from_f(float x);
template <>
__device__ __forceinline__ float from_f<float>(float x) { return x; }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f<__nv_bfloat16>(float x) { return __float2bfloat16_rn(x); }
template <>
__device__ __forceinline__ __half from_f<__half>(float x) { return __float2half_rn(x); }

// Rows of head hh (queries first, then keys) of token (b, n).
template <typename T>
__device__ __forceinline__ const T* row_in(const RotaryArgs& a, int hh, int b, int n) {
  const int w = hh >= a.heads[0];
  const Strides& s = a.xs[w];
  return static_cast<const T*>(a.x[w]) + b * s.b + (hh - w * a.heads[0]) * s.h + n * s.n;
}
template <typename T>
__device__ __forceinline__ T* row_out(const RotaryArgs& a, int hh, int b, int n) {
  const int w = hh >= a.heads[0];
  const Strides& s = a.ys[w];
  return static_cast<T*>(a.y[w]) + b * s.b + (hh - w * a.heads[0]) * s.h + n * s.n;
}

// Units of a row: VEC: 16-byte chunks (LAYOUT 0) or pairs of chunks (LAYOUT 1:
// the rotated part's, then the rest's, the last of which may be a single chunk);
// scalar: the pairs, then single elements.
template <typename T, int LAYOUT, bool VEC>
__host__ __device__ inline int rotary_units(int d, int rot) {
  constexpr int E = VEC ? 16 / static_cast<int>(sizeof(T)) : 1;
  if (!VEC) return rot / 2 + (d - rot);
  return LAYOUT == 0 ? d / E : rot / 2 / E + ((d - rot) / E + 1) / 2;
}

template <typename T, int LAYOUT, bool VEC, bool PART>
__global__ void __launch_bounds__(256) rotary_kernel(const RotaryArgs a, int units, int per_slice) {
  const long long id = static_cast<long long>(blockIdx.x) * blockDim.x + threadIdx.x;
  const long long total = static_cast<long long>(a.B) * a.N * units;
  if (id >= total) return;
  const unsigned int token = static_cast<unsigned int>(id) / static_cast<unsigned int>(units);
  const int u = static_cast<int>(static_cast<unsigned int>(id) - token * units);
  const int b = static_cast<int>(token / static_cast<unsigned int>(a.N));
  const int n = static_cast<int>(token - static_cast<unsigned int>(b) * a.N);
  const int32_t* pos = a.t.pos + b * a.t.pos_b + n * a.t.pos_n;
  const int h0 = blockIdx.y * per_slice, h1 = min(a.heads[0] + a.heads[1], h0 + per_slice);
  const int rot = a.t.rot;
  if constexpr (VEC) {
    using V = Vec16<T>;
    constexpr int E = V::E;
    // PART: a unit behind the rotated part is copied by the same instructions (its
    // words are kept as read), so a warp that holds both kinds does not run twice
    // (5 x 2338 tokens x 24 heads, 64 of 128 turned: 55 -> 37 us).
    const int turned = LAYOUT == 0 ? rot / E : rot / 2 / E;
    const bool turn = !PART || u < turned;
    int e0 = u * E, e1 = rot / 2 + u * E;
    if (PART && LAYOUT == 1 && !turn) {
      e0 = rot + (u - turned) * E;
      e1 = e0 + (units - turned) * E;
    }
    const bool two = LAYOUT == 1 && (!PART || e1 < a.d);
    constexpr int NP = LAYOUT == 0 ? E / 2 : E;  // pairs of this unit
    float c[NP], s[NP];
#pragma unroll
    for (int i = 0; i < NP; ++i) {
      c[i] = s[i] = 0.f;
      if (turn) pair_angle(a.t, pos, u * NP + i, &c[i], &s[i]);
    }
    // heads in flight; the first ones' loads ahead of the sines gain nothing for
    // one head a side (28.7 us either way) and cost 70 us of 482 for forty
    constexpr int UN = LAYOUT == 0 ? 4 : 2;
    for (int h = h0; h < h1; h += UN) {
      uint4 w[UN][2];
#pragma unroll
      for (int x = 0; x < UN; ++x) {
        if (h + x < h1) {
          const T* r = row_in<T>(a, h + x, b, n);
          w[x][0] = *reinterpret_cast<const uint4*>(r + e0);
          w[x][1] = make_uint4(0, 0, 0, 0);
          if (two) w[x][1] = *reinterpret_cast<const uint4*>(r + e1);
        }
      }
#pragma unroll
      for (int x = 0; x < UN; ++x) {
        if (h + x < h1) {
          T* y = row_out<T>(a, h + x, b, n);
          float f[E], g[E];
          V::get(w[x][0], f);
          if constexpr (LAYOUT == 0) {
#pragma unroll
            for (int i = 0; i < NP; ++i) {
              g[2 * i] = f[2 * i] * c[i] - f[2 * i + 1] * s[i];
              g[2 * i + 1] = f[2 * i + 1] * c[i] + f[2 * i] * s[i];
            }
            const uint4 o = V::put(g);
            *reinterpret_cast<uint4*>(y + e0) = turn ? o : w[x][0];
          } else {
            float f1[E], g1[E];
            V::get(w[x][1], f1);
#pragma unroll
            for (int i = 0; i < E; ++i) {
              g[i] = f[i] * c[i] - f1[i] * s[i];
              g1[i] = f1[i] * c[i] + f[i] * s[i];
            }
            const uint4 o = V::put(g), o1 = V::put(g1);
            *reinterpret_cast<uint4*>(y + e0) = turn ? o : w[x][0];
            if (two) *reinterpret_cast<uint4*>(y + e1) = turn ? o1 : w[x][1];
          }
        }
      }
    }
  } else {
    if (u >= rot / 2) {
      const int e = rot + (u - rot / 2);
      for (int h = h0; h < h1; ++h) row_out<T>(a, h, b, n)[e] = row_in<T>(a, h, b, n)[e];
      return;
    }
    float c, s;
    pair_angle(a.t, pos, u, &c, &s);
    const int e0 = LAYOUT == 0 ? 2 * u : u, e1 = LAYOUT == 0 ? 2 * u + 1 : u + rot / 2;
    for (int h = h0; h < h1; ++h) {
      const T* r = row_in<T>(a, h, b, n);
      T* y = row_out<T>(a, h, b, n);
      const float x0 = to_f(r[e0]), x1 = to_f(r[e1]);
      y[e0] = from_f<T>(x0 * c - x1 * s);
      y[e1] = from_f<T>(x1 * c + x0 * s);
    }
  }
}

// 16-byte accesses: every row of every tensor starts on a 16-byte boundary and
// the rotated part splits into whole chunks.
bool rotary_vec_ok(const RotaryArgs& a) {
  const int size = a.dtype == kF32 ? 4 : 2, E = 16 / size;
  auto fits = [&](const void* p, const Strides& s) {
    return (reinterpret_cast<uintptr_t>(p) & 15u) == 0 && s.b % E == 0 && s.h % E == 0 && s.n % E == 0;
  };
  for (int w = 0; w < 2; ++w) {
    if (a.x[w] && (!fits(a.x[w], a.xs[w]) || !fits(a.y[w], a.ys[w]))) return false;
  }
  return a.d % E == 0 && a.t.rot % (a.t.layout == 0 ? E : 2 * E) == 0;
}

template <typename T, int LAYOUT, bool VEC>
cudaError_t launch_rotary_t(const RotaryArgs& a, int num_sms, cudaStream_t stream) {
  const int units = rotary_units<T, LAYOUT, VEC>(a.d, a.t.rot);
  const long long threads = static_cast<long long>(a.B) * a.N * units;
  const int heads = a.heads[0] + a.heads[1];
  // Few tokens: the heads are split over threads too, until two full waves of
  // threads are there (each slice forms its own sines). Many tokens: one thread
  // walks all heads.
  const long long want = (2ll * num_sms * 2048 + threads - 1) / threads;
  int per = static_cast<int>(want >= heads ? 1 : (heads + want - 1) / want);
  if (per < 2 && heads > 1) per = 2;
  const dim3 grid(static_cast<unsigned int>((threads + 255) / 256), (heads + per - 1) / per);
  if (VEC && a.t.rot < a.d)
    rotary_kernel<T, LAYOUT, VEC, VEC><<<grid, 256, 0, stream>>>(a, units, per);
  else
    rotary_kernel<T, LAYOUT, VEC, false><<<grid, 256, 0, stream>>>(a, units, per);
  return cudaGetLastError();
}

template <typename T>
cudaError_t launch_rotary_l(const RotaryArgs& a, int num_sms, cudaStream_t stream) {
  const bool vec = rotary_vec_ok(a);
  if (a.t.layout == 0)
    return vec ? launch_rotary_t<T, 0, true>(a, num_sms, stream) : launch_rotary_t<T, 0, false>(a, num_sms, stream);
  return vec ? launch_rotary_t<T, 1, true>(a, num_sms, stream) : launch_rotary_t<T, 1, false>(a, num_sms, stream);
}

// ---------------------------------------------------------------------------
// Rotary positions and block means in one pass over q, k, v.
//
// One CTA per 64-token block and slice of heads: the block's sines and cosines
// are formed once in shared memory (32 KB at d = 128), then every warp takes
// whole (tensor, head) blocks: it reads the block's rows, writes the rotated
// rows (q, k) and sums the columns, in registers and two or three shuffles, so
// the warps never wait for one another. A lane holds two 16-byte chunks of a
// row, c and c + D/16 (the two halves of eight pairs, or two runs of four
// interleaved pairs). The means are those of the rotated values before their
// rounding to bf16: one rounding fewer than pooling the stored tensors.
// ---------------------------------------------------------------------------
constexpr int kPoolBlock = 64;

template <int D, int LAYOUT>
__global__ void __launch_bounds__(256, 2) rotary_pool_kernel(const RotaryPoolArgs a, int nb, int per_slice) {
  constexpr int U = D / 16;         // lanes per row
  constexpr int RPW = 32 / U;       // rows per warp and step
  constexpr int STEPS = kPoolBlock / RPW;
  constexpr int UNROLL = 4;
  using V = Vec16<__nv_bfloat16>;
  // sines of the pairs that lane-column u needs: [row][4 runs of two pairs][u]
  __shared__ float4 tab[kPoolBlock][4][U];
  const int b = blockIdx.x / nb, j = blockIdx.x % nb;
  const int row0 = j * kPoolBlock, rows = min(kPoolBlock, a.N - row0);
  const int h0 = blockIdx.y * per_slice, h1 = min(a.H, h0 + per_slice);
  for (int i = threadIdx.x; i < rows * 4 * U; i += blockDim.x) {
    const int r = i / (4 * U), run = i / U % 4, u = i % U;
    const int p = LAYOUT == 1 ? 8 * u + 2 * run : (run < 2 ? 4 * u + 2 * run : D / 4 + 4 * u + 2 * (run - 2));
    const int32_t* pos = a.t.pos + b * a.t.pos_b + (row0 + r) * a.t.pos_n;
    float4 v;
    pair_angle(a.t, pos, p, &v.x, &v.y);
    pair_angle(a.t, pos, p + 1, &v.z, &v.w);
    tab[r][run][u] = v;
  }
  __syncthreads();
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int u = lane % U, rl = lane / U;
  const int items = 3 * (h1 - h0);
  for (int it = warp; it < items; it += 8) {
    const int which = it % 3, h = h0 + it / 3;
    const uint16_t* src = a.x[which] + b * a.st.b + h * a.st.h + static_cast<long long>(row0) * a.st.n + u * 8;
    uint16_t* dst = which < 2 ? a.y[which] + b * a.ys.b + h * a.ys.h + static_cast<long long>(row0) * a.ys.n + u * 8
                              : nullptr;
    float s0[8], s1[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) s0[e] = s1[e] = 0.f;
    // four steps are multiplied while the next four are on their way
    uint4 w0[UNROLL], w1[UNROLL], n0[UNROLL], n1[UNROLL];
    auto load = [&](int st) {
#pragma unroll
      for (int x = 0; x < UNROLL; ++x) {
        const int r = (st + x) * RPW + rl;
        n0[x] = n1[x] = make_uint4(0, 0, 0, 0);
        if (r < rows) {
          n0[x] = *reinterpret_cast<const uint4*>(src + r * a.st.n);
          n1[x] = *reinterpret_cast<const uint4*>(src + r * a.st.n + D / 2);
        }
      }
    };
    load(0);
#pragma unroll 1
    for (int st = 0; st < STEPS; st += UNROLL) {
#pragma unroll
      for (int x = 0; x < UNROLL; ++x) w0[x] = n0[x], w1[x] = n1[x];
      if (st + UNROLL < STEPS) load(st + UNROLL);
#pragma unroll
      for (int x = 0; x < UNROLL; ++x) {
        const int r = (st + x) * RPW + rl;
        if (r >= rows) continue;
        float f0[8], f1[8];
        V::get(w0[x], f0);
        V::get(w1[x], f1);
        if (which < 2) {
          float g0[8], g1[8];
#pragma unroll
          for (int run = 0; run < 4; ++run) {
            const float4 t = tab[r][run][u];
            if constexpr (LAYOUT == 1) {
              const int e = 2 * run;
              g0[e] = f0[e] * t.x - f1[e] * t.y;
              g1[e] = f1[e] * t.x + f0[e] * t.y;
              g0[e + 1] = f0[e + 1] * t.z - f1[e + 1] * t.w;
              g1[e + 1] = f1[e + 1] * t.z + f0[e + 1] * t.w;
            } else {
              const int e = 4 * (run & 1);
              const float* f = run < 2 ? f0 : f1;
              float* g = run < 2 ? g0 : g1;
              g[e] = f[e] * t.x - f[e + 1] * t.y;
              g[e + 1] = f[e + 1] * t.x + f[e] * t.y;
              g[e + 2] = f[e + 2] * t.z - f[e + 3] * t.w;
              g[e + 3] = f[e + 3] * t.z + f[e + 2] * t.w;
            }
          }
          *reinterpret_cast<uint4*>(dst + r * a.ys.n) = V::put(g0);
          *reinterpret_cast<uint4*>(dst + r * a.ys.n + D / 2) = V::put(g1);
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            s0[e] += g0[e];
            s1[e] += g1[e];
          }
        } else {
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            s0[e] += f0[e];
            s1[e] += f1[e];
          }
        }
      }
    }
#pragma unroll
    for (int off = U; off < 32; off <<= 1) {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        s0[e] += __shfl_xor_sync(0xffffffffu, s0[e], off);
        s1[e] += __shfl_xor_sync(0xffffffffu, s1[e], off);
      }
    }
    if (lane < U) {
      const float n = static_cast<float>(rows);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        s0[e] = s0[e] / n;
        s1[e] = s1[e] / n;
      }
      const long long o = ((static_cast<long long>(b) * a.H + h) * nb + j) * D + u * 8;
      float4* m = reinterpret_cast<float4*>(a.bar[which] + o);
      m[0] = make_float4(s0[0], s0[1], s0[2], s0[3]);
      m[1] = make_float4(s0[4], s0[5], s0[6], s0[7]);
      float4* m1 = reinterpret_cast<float4*>(a.bar[which] + o + D / 2);
      m1[0] = make_float4(s1[0], s1[1], s1[2], s1[3]);
      m1[1] = make_float4(s1[4], s1[5], s1[6], s1[7]);
      if (a.bar16[which]) {
        *reinterpret_cast<uint4*>(a.bar16[which] + o) = V::put(s0);
        *reinterpret_cast<uint4*>(a.bar16[which] + o + D / 2) = V::put(s1);
      }
    }
  }
}

template <int D, int LAYOUT>
cudaError_t launch_rotary_pool_t(const RotaryPoolArgs& a, int num_sms, cudaStream_t stream) {
  const int nb = (a.N + kPoolBlock - 1) / kPoolBlock;
  const long long blocks = static_cast<long long>(a.B) * nb;
  // heads per CTA: all of them where the blocks alone fill the GPU four times
  // over, fewer (each slice forms its own sines) where they do not
  const long long want = (4ll * num_sms * 4 + blocks - 1) / blocks;
  int per = static_cast<int>(want >= a.H ? 1 : (a.H + want - 1) / want);
  // three items a head for eight warps: eight heads leave no warp over
  if (a.H >= 8) per = (per + 7) / 8 * 8;
  else if (per < 3 && a.H >= 3) per = 3;
  rotary_pool_kernel<D, LAYOUT><<<dim3(static_cast<unsigned int>(blocks), (a.H + per - 1) / per), 256, 0, stream>>>(
      a, nb, per);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_rotary(const RotaryArgs& a, int num_sms, cudaStream_t stream) {
  if (a.dtype == kF32) return launch_rotary_l<float>(a, num_sms, stream);
  if (a.dtype == kF16) return launch_rotary_l<__half>(a, num_sms, stream);
  return launch_rotary_l<__nv_bfloat16>(a, num_sms, stream);
}

cudaError_t launch_rotary_pool(const RotaryPoolArgs& a, int num_sms, cudaStream_t stream) {
  if (a.d == 64)
    return a.t.layout == 0 ? launch_rotary_pool_t<64, 0>(a, num_sms, stream)
                           : launch_rotary_pool_t<64, 1>(a, num_sms, stream);
  return a.t.layout == 0 ? launch_rotary_pool_t<128, 0>(a, num_sms, stream)
                         : launch_rotary_pool_t<128, 1>(a, num_sms, stream);
}

}  // namespace solattn
