// cache_chunk.cu -- attention of many queries (a prompt, a chunk, a video frame)
// over the 8-bit cache, on tcgen05, where that is estimated to be the faster.
//
// One CTA takes 256 query rows of one key head (token-major, the heads of the
// group side by side) as two 128-row tiles, and one part of the keys. Both tiles
// use every key tile that is converted, so the conversion from e4m3 to fp16
// (tcgen05 multiplies operands of one type, and 8-bit queries would lose the
// scores' accuracy) is paid once per 256 rows: 128 threads load a page's bytes,
// convert them and store them in the swizzled operand layout.
//
//   warps 0-3, 4-7  softmax of tile 0 / tile 1: one thread per row; S and P in
//                   TMEM (P in fp16 over the first half of its own S), O scaled
//                   in TMEM only when a row's reference moves
//   warps 8-11      cache pages to fp16 operands, four pages in shared memory
//   warp 12         issues every MMA
//   warp 13         brings the cache's pages into shared memory, two pages ahead
//                   of their conversion (loads into the converters' registers, a
//                   page ahead, were waited for: 2,000 cycles under load)
//   warps 14, 15    only give their registers
//
// Keys go in tiles of two pages, softmax and PV page by page, so that PV of the
// first page runs under the softmax of the second. At d = 64 QK goes by pages too:
// the next scores of a page's columns are there when the softmax comes back to
// them. At d = 128 a QK of 64 columns takes as long as one of 128 (it is bound by
// reading Q from shared memory; 520 cycles against 600), so there it is one QK of
// 128 columns behind the tile's second PV, and the softmax waits for it.
#include <cuda_runtime.h>
#include <cmath>
#include <cstdint>

#include "cache_common.cuh"

namespace solattn {

namespace {

constexpr int kTileRows = 128;
constexpr int kChunkThreads = 512;  // 16 warps, 128 registers per thread at launch
constexpr int kTileKeys = 2 * kPage;
constexpr int kKStages = 2;  // key tiles
constexpr int kVStages = 4;  // pages
constexpr int kRaw = 2;      // pages as they lie in the cache
constexpr int kInfo = 8;     // pages

// Wait sites reported in the status word.
enum : uint32_t {
  kSiteCQ = 40,
  kSiteCRawFull,
  kSiteCRawEmpty,
  kSiteCKFull,
  kSiteCKEmpty,
  kSiteCVFull,
  kSiteCVEmpty,
  kSiteCSFull,
  kSiteCPFull,
  kSiteCPv,
};

template <int D>
struct __align__(1024) ChunkSmem {
  uint8_t q[2][kTileRows * D * 2];        // SW128 K-major panels of 128 rows
  uint8_t k[kKStages][kTileKeys * D * 2]; // the same
  uint8_t v[kVStages][kPage * D * 2];     // SW128 panels of 64 rows
  uint8_t raw[kRaw][2][kPage * D];        // keys and values of a page, e4m3
  float4 info[kInfo];                     // a page's factors (PageScale), and kSlack: NaN where turn is not 1
  float turn[kInfo];                      // what O is multiplied by before the page; NaN: a scale is NaN
  int unit;                               // of the last page, as its exponent
  uint64_t q_full[2], k_full[kKStages], k_empty[kKStages], v_full[kVStages], v_empty[kVStages];
  uint64_t raw_full[kRaw], raw_empty[kRaw];
  uint64_t s_full[2][2], p_full[2][2], pv_done[2][2], mma_done;
  uint32_t tmem_base;
  int abort_flag;
  int nan;
};

// fp16 operands: the format fields of the instruction descriptor are 0.
__host__ __device__ constexpr uint32_t idesc_f16_f32(int M, int N, bool b_mn_major) {
  return (1u << 4) | (static_cast<uint32_t>(b_mn_major) << 16) | (static_cast<uint32_t>(N >> 3) << 17) |
         (static_cast<uint32_t>(M >> 4) << 24);
}

__device__ __forceinline__ uint64_t f2_make(uint32_t lo, uint32_t hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "r"(lo), "r"(hi));
  return r;
}
__device__ __forceinline__ uint64_t f2_both(float x) { return f2_make(__float_as_uint(x), __float_as_uint(x)); }
__device__ __forceinline__ void f2_get(uint64_t v, float& lo, float& hi) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
}
__device__ __forceinline__ uint64_t f2_fma(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}
__device__ __forceinline__ uint64_t f2_add(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("add.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

// The largest of a row's 64 scores of a page.
__device__ __forceinline__ float page_max(const uint32_t (&sv)[64]) {
  float t[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
  for (int i = 0; i < 64; i += 8)
#pragma unroll
    for (int e = 0; e < 4; ++e)
      t[e] = max3(t[e], __uint_as_float(sv[i + 2 * e]), __uint_as_float(sv[i + 2 * e + 1]));
  return fmaxf(max3(t[0], t[1], t[2]), t[3]);
}
// 2^x of a pair on the FMA pipe: x = j + f with an integer j and |f| <= 1/2, a
// polynomial of degree 4 (least squares, reweighted towards the least largest
// relative error: 2.6e-6) for 2^f, times 2^j (0 for j = -127). NaN stays NaN.
__device__ __forceinline__ uint64_t f2_exp2(uint64_t v) {
  float x0, x1;
  f2_get(v, x0, x1);
  asm("max.NaN.f32 %0, %0, %1;" : "+f"(x0) : "f"(-127.f));
  asm("max.NaN.f32 %0, %0, %1;" : "+f"(x1) : "f"(-127.f));
  const uint64_t x = f2_make(__float_as_uint(x0), __float_as_uint(x1));
  const uint64_t t = f2_add(x, f2_both(12582912.f));   // 1.5 2^23: the low bits are j
  const uint64_t f = f2_fma(f2_add(t, f2_both(-12582912.f)), f2_both(-1.f), x);
  uint64_t p = f2_fma(f, f2_both(0.009570101276040077f), f2_both(0.05591786280274391f));
  p = f2_fma(p, f, f2_both(0.240247443318367f));
  p = f2_fma(p, f, f2_both(0.6931217908859253f));
  p = f2_fma(p, f, f2_both(0.9999992847442627f));
  float t0, t1;
  f2_get(t, t0, t1);
  const uint64_t scale = f2_make((__float_as_uint(t0) << 23) + 0x3f800000u, (__float_as_uint(t1) << 23) + 0x3f800000u);
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(p), "l"(scale));
  return r;
}

// P = 2^(s c + add) of the page as 32 fp16 pairs; returns the sum. Every
// kPolyEvery-th pair goes to the FMA pipe.
template <int kPolyEvery>
__device__ __forceinline__ float page_weights(const uint32_t (&sv)[64], float c, float add, uint32_t* pw) {
  const uint64_t c2 = f2_both(c), a2 = f2_both(add);
  uint64_t l0 = 0, l1 = 0;
#pragma unroll
  for (int i = 0; i < 32; ++i) {
    uint64_t x = f2_fma(f2_make(sv[2 * i], sv[2 * i + 1]), c2, a2);
    float x0, x1;
    if (kPolyEvery > 0 && i % (kPolyEvery > 0 ? kPolyEvery : 1) == kPolyEvery - 1) {
      x = f2_exp2(x);
      f2_get(x, x0, x1);
    } else {
      f2_get(x, x0, x1);
      x0 = ex2_approx(x0);
      x1 = ex2_approx(x1);
      x = f2_make(__float_as_uint(x0), __float_as_uint(x1));
    }
    if (i & 1) l1 = f2_add(l1, x);
    else l0 = f2_add(l0, x);
    pw[i] = pack_f16x2(x0, x1);
  }
  float u, v;
  f2_get(f2_add(l0, l1), u, v);
  return u + v;
}
// Log2 units per unit of a row's dot products; never 0, which would turn a
// masked key's -inf into NaN.
__device__ __forceinline__ float row_scale(const PageScale& ps, float rf) { return fmaxf(ps.ck * rf, 1.17549435e-38f); }
// The exponent's addend of a page for a row with reference m.
__device__ __forceinline__ float page_addend(const PageScale& ps, float m) {
  return ps.ev == -INFINITY ? -INFINITY : ps.ev + kPBias - (m == -INFINITY ? 0.f : m);
}

// Rare paths, out of line; warp-collective, a lane with factor 1 keeps its row.
template <int D>
static __device__ __noinline__ void scale_o(uint32_t taddr, float f) {
#pragma unroll 1
  for (int ch = 0; ch < D / 32; ++ch) {
    uint32_t ov[32];
    tmem_ld32_wait(taddr + ch * 32, ov);
#pragma unroll
    for (int x = 0; x < 32; ++x) ov[x] = __float_as_uint(__uint_as_float(ov[x]) * f);
    tmem_st32_wait(taddr + ch * 32, ov);
  }
}

template <int REGION = 0>
__device__ __forceinline__ bool chunk_wait(uint64_t* bar, uint32_t parity, volatile int* abort_flag, DeviceStatus* st,
                                           uint32_t site, uint32_t unit) {
  const bool ok = mbar_wait<REGION>(bar, parity, abort_flag, st, site, unit);
  return __all_sync(0xffffffffu, ok);
}

// Byte offset of 16-byte chunk `ch` (8 fp16) of row `row` in a panel with 128-byte rows, 128-byte swizzle.
__device__ __forceinline__ uint32_t sw128(int row, int ch) { return row * 128 + ((ch ^ (row & 7)) << 4); }

// An untiled asynchronous copy of `bytes` from global to shared memory.
__device__ __forceinline__ void bulk_load(void* dst, const void* src, uint32_t bytes, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(smem_u32(dst)),
      "l"(src), "r"(bytes), "r"(smem_u32(bar))
      : "memory");
}

__device__ __forceinline__ void st_shared_v4(void* p, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" ::"r"(smem_u32(p)), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
}

// 32 rows of queries into the operand layout, scaled to fp16's range by a power
// of two per row: copied as they are (a row's lanes side by side, so that a copy
// touches a few lines and not one per lane; before the sequence's counts are
// read, so rows of the tensor behind them too), then every lane converts one row
// in place, a row that is not there to zeros, and returns its factor. The loops
// are short on purpose: they run once, and what is unrolled is first fetched.
template <int D>
__device__ __forceinline__ void copy_queries(const CacheAttnArgs& a, uint8_t* tile, int b, int hk, int first, int wq,
                                             int lane) {
  const int rows = a.N * a.group;
  constexpr int LPR = D / 8, RPL = 32 / LPR;  // lanes per row, rows per step
  const int ch = lane % LPR;
  uint8_t* to = tile + (ch / 8) * (kTileRows * 128);
  const uint16_t* from = a.q + b * a.st.b + hk * a.group * a.st.h + 8 * ch;
#pragma unroll 4
  for (int i = 0; i < 32 / RPL; ++i) {
    const int lr = wq * 32 + i * RPL + lane / LPR, r = first + lr;
    int qi, g;
    row_place(a, r, &qi, &g);
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(to + sw128(lr, ch % 8))),
                 "l"(r < rows ? from + g * a.st.h + qi * a.st.n : a.q), "r"(r < rows ? 16 : 0)
                 : "memory");
  }
}

// Every copy of the thread has landed.
__device__ __forceinline__ void copies_done() { asm volatile("cp.async.wait_all;" ::: "memory"); }

template <typename Elem, int D>
__device__ __forceinline__ float convert_queries(uint8_t* tile, bool there, int wq, int lane) {
  __syncwarp();
  const int lr = wq * 32 + lane;
  uint8_t* row = tile + lr * 128;
  const uint32_t x = static_cast<uint32_t>(lr & 7) << 4;
  uint32_t top = 0;
#pragma unroll 4
  for (int c = 0; c < D / 8; ++c) {  // largest magnitude's bits, by pairs
    const uint4 w = *reinterpret_cast<const uint4*>(row + (c / 8) * (kTileRows * 128) + ((c % 8 * 16) ^ x));
    constexpr uint32_t M = 0x7fff7fffu;
    top = __vmaxu2(top, __vmaxu2(__vmaxu2(w.x & M, w.y & M), __vmaxu2(w.z & M, w.w & M)));
  }
  float mul, inv;
  row_factor(unpack2<Elem>(max(top & 0xffffu, top >> 16)).x, &mul, &inv);
#pragma unroll 2
  for (int c = 0; c < D / 8; ++c) {
    uint4* p = reinterpret_cast<uint4*>(row + (c / 8) * (kTileRows * 128) + ((c % 8 * 16) ^ x));
    const uint4 w = there ? *p : make_uint4(0, 0, 0, 0);
    const float2 f0 = unpack2<Elem>(w.x), f1 = unpack2<Elem>(w.y), f2 = unpack2<Elem>(w.z), f3 = unpack2<Elem>(w.w);
    *p = make_uint4(pack_f16x2(f0.x * mul, f0.y * mul), pack_f16x2(f1.x * mul, f1.y * mul),
                    pack_f16x2(f2.x * mul, f2.y * mul), pack_f16x2(f3.x * mul, f3.y * mul));
  }
  fence_proxy_async_smem();
  __syncwarp();
  return inv;
}

// A warp's 32 rows of D / 2 columns (half 0 or 1 of the row; columns of 4 bytes
// for parts, 2 for results) from its stage in shared memory to their rows in
// memory: a row's lanes side by side. Row r's 16-byte pieces are rotated by r.
template <int PIECES>
__device__ __forceinline__ void store_rows(const CacheAttnArgs& a, const uint8_t* stage, int b, int hk, int first,
                                           int rows, int half, int split, int lane) {
  constexpr int RPL = 32 / PIECES;
  const int e = lane % PIECES;
#pragma unroll 4
  for (int i = 0; i < 32 / RPL; ++i) {
    const int row = i * RPL + lane / PIECES, r = first + row;
    if (r < rows) {
      const uint4 v = *reinterpret_cast<const uint4*>(stage + (row * PIECES + ((e + row) % PIECES)) * 16);
      int qi, g;
      row_place(a, r, &qi, &g);
      const int h = hk * a.group + g;
      if (a.splits > 1)
        *reinterpret_cast<uint4*>(a.part_o + partial_row(a, b, h, qi, split) * a.d + half * (a.d / 2) + 4 * e) = v;
      else
        *reinterpret_cast<uint4*>(a.out + b * a.ost.b + h * a.ost.h + static_cast<long long>(qi) * a.ost.n +
                                  half * (a.d / 2) + 8 * e) = v;
    }
  }
  __syncwarp();
}

// Out of line: in the kernel its registers cost the softmax loop 3 %.
static __device__ __noinline__ int ranked_sequence(const CacheAttnArgs& a, int n, int lane) {
  return nth_longest(a, n, lane);
}

template <typename Elem, int D>
__global__ void __launch_bounds__(kChunkThreads, 1) cache_chunk_kernel(const CacheAttnArgs a, int tiles) {
  constexpr bool kPageSlots = D == 64;
  // At d = 64 both tiles' exponentials always meet: every eighth pair on the FMA
  // pipe instead took 256 x 8192 x 148 heads from 136 to 127 us (every fourth: 135
  // us). At d = 128 they alternate, and the longer code costs (151 to 159 us).
  constexpr int kPolyEvery = D == 64 ? 8 : 0;
  extern __shared__ uint8_t smem_raw[];
  ChunkSmem<D>& sm =
      *reinterpret_cast<ChunkSmem<D>*>(smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u));
  const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
  // the tiles that see most keys first
  const int split = blockIdx.x % a.splits, mt = tiles - 1 - blockIdx.x / a.splits;
  const int hk = blockIdx.y, b = a.longest_first ? ranked_sequence(a, blockIdx.z, lane) : blockIdx.z;
  DeviceStatus* st = a.status;
  volatile int* abort_flag = &sm.abort_flag;
  start_join(a);
  const int r0 = mt * 2 * kTileRows;
  if (warp < 8) copy_queries<D>(a, sm.q[warp / 4], b, hk, r0 + warp / 4 * kTileRows, warp % 4, lane);
  if (tid == kChunkThreads - 32) {  // a warp with nothing else to do
    for (int i = 0; i < kKStages; ++i) {
      mbar_init(&sm.k_full[i], 8);  // four warps, two pages
      mbar_init(&sm.k_empty[i], 1);
    }
    for (int i = 0; i < kVStages; ++i) {
      mbar_init(&sm.v_full[i], 4);
      mbar_init(&sm.v_empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      for (int e = 0; e < 2; ++e) {
        mbar_init(&sm.s_full[i][e], 2);  // the MMAs' commit, and the issuer itself, which passes on the page scales
        mbar_init(&sm.p_full[i][e], 4);
        mbar_init(&sm.pv_done[i][e], 1);
      }
    }
    for (int i = 0; i < 2; ++i) mbar_init(&sm.q_full[i], 4);
    for (int i = 0; i < kRaw; ++i) {
      mbar_init(&sm.raw_full[i], 2);  // the copies' issue and the scales
      mbar_init(&sm.raw_empty[i], 4);
    }
    mbar_init(&sm.mma_done, 1);
    sm.unit = 127;
    sm.abort_flag = 0;
    sm.nan = 0;
    fence_barrier_init();
  }
  __syncthreads();
  const Extent ex = extent(a, b, split == 0 && hk == 0 && mt == 0 && tid == 0);
  const int rows = ex.cnt * a.group;
  if (r0 >= rows) {  // rows behind the sequence's queries stay as they are
    copies_done();
    return;
  }
  const int nq = rows - r0 > kTileRows ? 2 : 1;  // 128-row tiles with rows in them
  const int last_row = min(rows, r0 + 2 * kTileRows) - 1;
  const int seen = key_limit(ex, a.causal, last_row / a.group);  // keys that some row sees
  const int least = key_limit(ex, a.causal, r0 / a.group);       // keys that every row sees
  const int pages = (seen + kPage - 1) / kPage;
  const int per = (pages + a.splits - 1) / a.splits;
  const int c0 = min(pages, split * per);
  const int P = (min(pages, c0 + per) - c0 + 1) / 2 * 2;  // this part's pages, rounded up to whole key tiles
  const int pend = min(pages, c0 + per) - c0;             // those that are there

  // TMEM columns: S of tile x at 128 x, P of its page e over the first half of that page's scores (128 x + 64 e);
  // O of tile x at 256 + 128 x

  // Registers: 152 for the 256 softmax threads, 104 for the other 256 (65,536 in all).
  if (warp >= 12) {
    regs_dec<104>();
    if (warp == 12) {
      // ======================= MMA issuer =======================
      tmem_alloc(&sm.tmem_base, 512);  // the softmax warps learn of it with the first scores
      tmem_relinquish();
      __syncwarp();
      const uint32_t tmem = *static_cast<volatile uint32_t*>(&sm.tmem_base);
      constexpr uint32_t idesc_qk = idesc_f16_f32(kTileRows, kPageSlots ? kPage : kTileKeys, false);
      constexpr uint32_t idesc_pv = idesc_f16_f32(kTileRows, D, true);
      const uint64_t qd0 = sw128_desc(smem_u32(&sm.q[0][0]), 16, 1024);
      const uint64_t kd0 = sw128_desc(smem_u32(&sm.k[0][0]), 16, 1024);
      const uint64_t vd0 = sw128_desc(smem_u32(&sm.v[0][0]), 8192, 1024);
      // One thread issues everything and waits for what it needs; the others go on
      // to the teardown.
      if (elect_one()) {
        auto wait = [&](uint64_t* bar, uint32_t parity, uint32_t site) {
          return mbar_wait(bar, parity, abort_flag, st, site, blockIdx.x);
        };
        // QK for tile x: of key tile t = n (d = 128), of page n (d = 64)
        auto qk = [&](int n, int x) {
          tc_fence_after();
          const int t = kPageSlots ? n / 2 : n, e = kPageSlots ? n & 1 : 0;
          const uint64_t kd = kd0 + (((t % kKStages) * (kTileKeys * D * 2) + e * (kPage * 128)) >> 4);
          const uint64_t qd = qd0 + (x * (kTileRows * D * 2) >> 4);
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk) {
            const uint32_t off = ((kk / 4) * (kTileRows * 128) + (kk % 4) * 32) >> 4;
            mma_ss(tmem + x * 128 + e * 64, qd + off, kd + off, idesc_qk, kk > 0 ? 1u : 0u);
          }
          mbar_arrive(&sm.s_full[x][e]);
          mma_commit(&sm.s_full[x][e]);
          if (x == nq - 1 && (!kPageSlots || e == 1)) mma_commit(&sm.k_empty[t % kKStages]);
        };
        auto k_there = [&](int t) { return wait(&sm.k_full[t % kKStages], (t / kKStages) & 1, kSiteCKFull); };
        bool ok = P == 0 || k_there(0);
        for (int x = 0; x < nq && ok && P > 0; ++x) {
          ok = wait(&sm.q_full[x], 0, kSiteCQ);
          if (ok) qk(0, x);
          if (ok && kPageSlots) qk(1, x);
        }
        // PV of page p for tile x
        auto pv = [&](int p, int x) {
          if (!wait(&sm.p_full[x][p & 1], (p >> 1) & 1, kSiteCPFull)) return false;
          tc_fence_after();
          const uint64_t vd = vd0 + ((p % kVStages) * (kPage * D * 2) >> 4);
#pragma unroll
          for (int kk = 0; kk < kPage / 16; ++kk)
            mma_ts(tmem + 256 + x * 128, tmem + x * 128 + (p & 1) * 64 + kk * 8, vd + ((kk * 2048) >> 4), idesc_pv,
                   (p > 0 || kk > 0) ? 1u : 0u);
          mma_commit(&sm.pv_done[x][p & 1]);
          if (x == nq - 1) mma_commit(&sm.v_empty[p % kVStages]);
          return true;
        };
        auto v_there = [&](int p) { return wait(&sm.v_full[p % kVStages], (p / kVStages) & 1, kSiteCVFull); };
        // Scores go over the columns that a PV read P from, behind it: one thread's
        // MMAs execute in order.
        if constexpr (kPageSlots) {
          for (int p = 0; p < P && ok; ++p) {
            if ((p & 1) == 0 && p + 2 < P) ok = k_there(p / 2 + 1);
            if (ok) ok = v_there(p);
            for (int x = 0; x < nq && ok; ++x) {
              ok = pv(p, x);
              if (ok && p + 2 < P) qk(p + 2, x);
            }
          }
        } else {
          for (int t = 0; t < P / 2 && ok; ++t) {
            for (int x = 0; x < nq && ok; ++x) {
              for (int e = 0; e < 2 && ok; ++e) {
                if (x == 0) ok = v_there(2 * t + e);
                if (ok) ok = pv(2 * t + e, x);
              }
              if (ok && t + 1 < P / 2) {
                if (x == 0) ok = k_there(t + 1);
                if (ok) qk(t + 1, x);
              }
            }
          }
        }
        mma_commit(&sm.mma_done);  // teardown: issued MMAs complete before TMEM is freed
      }
      __syncwarp();
      mbar_wait_quiet(&sm.mma_done, 0);
      __syncwarp();
    } else if (warp == 13) {
      // ======================= pages on their way =======================
      const int32_t* table = a.table + b * a.table_stride + c0;
      bool ok = true;
      int issued = 0;
      int unit = 0, before = 0;  // of the value scales: the last page's, and the last 32 pages' by lane
      for (int base = 0; base < P && ok; base += 32) {
        // 32 pages' numbers and scales at once; -1 and 0: not there
        int pg = -1;
        float ks = 0.f, vs = 0.f;
        if (base + lane < pend) {
          pg = __ldg(table + base + lane);
          if (pg < 0 || pg >= a.pages) {
            report_page(st, b);
            pg = -1;
          } else {
            ks = __ldg(a.k_scale + pg * a.scale_stride + hk);
            vs = __ldg(a.v_scale + pg * a.scale_stride + hk);
          }
        }
        auto issue = [&](int p, int page) {
#ifdef SOLATTN_TEST_HOOKS
          if (p == 0 && static_cast<int>(blockIdx.x) == g_hook_skip_cta) return;  // this page never arrives
#endif
          if (lane == 0) {
            const int s = p % kRaw;
            if (page >= 0) {
              const long long at = page * a.page_stride + static_cast<long long>(hk) * kPage * D;
              mbar_arrive_expect_tx(&sm.raw_full[s], 2 * kPage * D);
              bulk_load(sm.raw[s][0], a.k + at, kPage * D, &sm.raw_full[s]);
              bulk_load(sm.raw[s][1], a.v + at, kPage * D, &sm.raw_full[s]);
            } else {
              mbar_arrive(&sm.raw_full[s]);
            }
          }
          issued = p + 1;
        };
        // the first pages' copies go out before their scales have come
        const int ahead = base == 0 ? min(kRaw, P) : 0;
        for (int i = 0; i < ahead; ++i) issue(i, __shfl_sync(0xffffffffu, pg, i));
        const int mine = page_units(vs, unit, lane);
        int from = __shfl_sync(0xffffffffu, lane < 31 ? mine : before, (lane + 31) & 31);
        if (base == 0 && lane == 0) from = mine;
        const float turn = unit_turn(from, mine);
        before = mine;
        const PageScale ps = page_scale(a, ks, vs * unit_inverse(mine));
        const bool no_number = isnan(ps.ck) || isnan(ps.ev);
        for (int i = 0; i < min(32, P - base) && ok; ++i) {
          const int p = base + i, s = p % kRaw;
          const int page = __shfl_sync(0xffffffffu, pg, i);
          if (i >= ahead) {
            ok = chunk_wait(&sm.raw_empty[s], ((p / kRaw) & 1) ^ 1, abort_flag, st, kSiteCRawEmpty, blockIdx.x);
            if (!ok) break;
            issue(p, page);
          }
          if (lane == i) {
            // the scales' slot held page p - 8: page p - 2 has been converted, so the QK of page p - 6 is
            // complete, and it was issued behind P of page p - 8 in both tiles
            sm.info[p % kInfo] = no_number ? make_float4(0.f, 0.f, 1.f, NAN)
                                           : make_float4(ps.ck, ps.ev, ps.vinv, turn != 1.f ? NAN : kSlack);
            sm.turn[p % kInfo] = no_number ? NAN : turn;
            sm.unit = mine;
            mbar_arrive(&sm.raw_full[s]);
          }
          __syncwarp();
        }
      }
      // teardown: every copy has landed (none is under way unless a wait gave up)
      if (lane == 0)
        for (int p = max(0, issued - kRaw); p < issued; ++p) mbar_wait_quiet(&sm.raw_full[p % kRaw], (p / kRaw) & 1);
      __syncwarp();
    }
  } else if (warp >= 8) {
    regs_dec<104>();
    // ======================= cache pages to fp16 operands =======================
    const int ct = tid - 256;
    constexpr int LPR = D / 16;           // lanes per row (16 bytes each)
    constexpr int ROWS = 128 / LPR;       // rows per pass of the 128 threads
    constexpr int PASSES = kPage / ROWS;  // 4 (d = 128) or 2
    // chunk of the row and row of the pass: eight neighbouring lanes take four chunks of two rows
    const int c = LPR == 4 ? ct % 4 : ct % 4 + 4 * (ct / 8 % 2);
    const int rr = LPR == 4 ? ct / 4 : ct / 4 % 2 + 2 * (ct / 16);
    // 16 e4m3 of a row become two 16-byte chunks of fp16. A quarter-warp's eight
    // stores cover two rows' chunks of one panel: eight different bank groups.
    const int ch = 2 * (c % 4);
    const uint32_t off0 = sw128(rr, ch), off1 = sw128(rr, ch + 1);  // ROWS is a multiple of the swizzle's 8 rows
    const int at = rr * D + 16 * c;  // of the thread's 16 bytes in a page, and every ROWS rows on
    auto store = [&](const uint4 (&w)[PASSES], uint8_t* dst, int panel_rows) {
      uint8_t* base = dst + (c / 4) * (panel_rows * 128);
#pragma unroll
      for (int i = 0; i < PASSES; ++i) {
        uint32_t f[8];
        e4m3x4_f16(w[i].x, f[0], f[1]);
        e4m3x4_f16(w[i].y, f[2], f[3]);
        e4m3x4_f16(w[i].z, f[4], f[5]);
        e4m3x4_f16(w[i].w, f[6], f[7]);
        st_shared_v4(base + off0 + i * ROWS * 128, f[0], f[1], f[2], f[3]);
        st_shared_v4(base + off1 + i * ROWS * 128, f[4], f[5], f[6], f[7]);
      }
    };
    bool ok = true;
#pragma unroll 1
    for (int p = 0; p < P && ok; ++p) {
      const int kst = p / 2 % kKStages, vst = p % kVStages, rs = p % kRaw;
      if ((p & 1) == 0 && p >= 2 * kKStages)
        ok = chunk_wait(&sm.k_empty[kst], ((p / (2 * kKStages)) & 1) ^ 1, abort_flag, st, kSiteCKEmpty, blockIdx.x);
      if (ok) ok = chunk_wait(&sm.raw_full[rs], (p / kRaw) & 1, abort_flag, st, kSiteCRawFull, blockIdx.x);
      if (!ok) break;
      uint4 w[PASSES];
#pragma unroll
      for (int i = 0; i < PASSES; ++i) w[i] = *reinterpret_cast<const uint4*>(sm.raw[rs][0] + at + i * ROWS * D);
      store(w, sm.k[kst] + (p & 1) * kPage * 128, kTileKeys);
#pragma unroll
      for (int i = 0; i < PASSES; ++i) w[i] = *reinterpret_cast<const uint4*>(sm.raw[rs][1] + at + i * ROWS * D);
      const int rows_in = sm.info[p % kInfo].y == -INFINITY ? 0 : ex.len - (c0 + p) * kPage;
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(&sm.k_full[kst]);
        mbar_arrive(&sm.raw_empty[rs]);
      }
      if (rows_in < kPage) {  // rows behind the sequence may hold anything, NaN too
#pragma unroll
        for (int i = 0; i < PASSES; ++i)
          if (i * ROWS + rr >= rows_in) w[i] = make_uint4(0, 0, 0, 0);
      }
      if (a.causal && (c0 + p + 1) * kPage > least) {  // a NaN value must reach only the rows that see its token
        bool bad = false;
#pragma unroll
        for (int i = 0; i < PASSES; ++i) {
          bad |= has_nan8(w[i].x) | has_nan8(w[i].y) | has_nan8(w[i].z) | has_nan8(w[i].w);
          w[i] = make_uint4(drop_nan8(w[i].x), drop_nan8(w[i].y), drop_nan8(w[i].z), drop_nan8(w[i].w));
        }
        if (bad) sm.nan = 1;
      }
      if (p >= kVStages)
        ok = chunk_wait(&sm.v_empty[vst], ((p / kVStages) & 1) ^ 1, abort_flag, st, kSiteCVEmpty, blockIdx.x);
      store(w, sm.v[vst], kPage);
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&sm.v_full[vst]);
    }
  } else {
    regs_inc<152>();
    copies_done();
    if (warp / 4 < nq) {
      // ======================= softmax =======================
      const int x = warp / 4, wq = warp % 4;
      const int lr = wq * 32 + lane;  // row of the tile == TMEM lane
      const int r = r0 + x * kTileRows + lr;
      const bool there = r < rows;
      int qi, g;
      row_place(a, r, &qi, &g);
      const int h = hk * a.group + g;
      const int lim = there ? key_limit(ex, a.causal, qi) : seen;  // a row that is not there masks nothing by itself
      const uint32_t lane_sel = static_cast<uint32_t>(wq * 32) << 16;
      const float rf = convert_queries<Elem, D>(sm.q[x], there, wq, lane);
      if (lane == 0) mbar_arrive(&sm.q_full[x]);
      uint32_t colS = 0, colO = 0;
      float m = -INFINITY, l = 0.f;
      bool ok = true;
      const int lim_warp = __reduce_min_sync(0xffffffffu, lim);
      for (int p = 0; p < P; ++p) {
        if (kPageSlots || (p & 1) == 0) {
          ok = chunk_wait<1>(&sm.s_full[x][kPageSlots ? p & 1 : 0], (p >> 1) & 1, abort_flag, st, kSiteCSFull, blockIdx.x);
          if (!ok) break;
          tc_fence_after();
          if (p == 0) {
            const uint32_t tmem = *static_cast<volatile uint32_t*>(&sm.tmem_base);
            colS = tmem + x * 128 + lane_sel;
            colO = tmem + 256 + x * 128 + lane_sel;
          }
        }
        const float4 info = sm.info[p % kInfo];
        const PageScale ps{info.x, info.y, info.z};
        const uint32_t col = colS + (p & 1) * 64;
        uint32_t sv[64], pw[32];
        tmem_ld32x2_wait(col, col + 32, sv);
        const int key0 = (c0 + p) * kPage;
        if (key0 + kPage > lim_warp || ps.ev == -INFINITY) {  // -inf: a page that is not there
          const int end = ps.ev == -INFINITY ? key0 : lim;
#pragma unroll
          for (int i = 0; i < 64; ++i)
            if (key0 + i >= end) sv[i] = 0xff800000u;
        }
        const float c = row_scale(ps, rf);
        // P with the reference as it stands, beside the maximum rather than behind
        // it; only a page that passes the reference by kSlack (rare after the first
        // ones) is done again
        // No reference yet: the maximum first, or every row would do the page again.
        // Worth 0.6 us of a short call; at d = 128 the loop's code with it costs long
        // calls 5 % (256 x 8192 x 148 heads: 147 to 155 us).
        if (kPageSlots && p == 0) {
          const float tm = fmaf(page_max(sv), c, ps.ev);
          if (tm > -INFINITY) m = ceilf(tm);
        }
        float sum, slack = info.w;
        while (true) {
          sum = page_weights<kPolyEvery>(sv, c, page_addend(ps, m), pw);
          const float mx = page_max(sv);
          const float tm = fmaxf(fmaf(mx, c, ps.ev), -INFINITY);  // NaN raises nothing
          if (__all_sync(0xffffffffu, tm <= m + slack)) break;
          const float up = tm > m + kSlack ? ceilf(tm) : m;
          const float k = up == m || m == -INFINITY ? 1.f : ex2_approx(m - up);
          // the unit of the value scales that the page turns to; a page without a number for
          // a scale makes the sums of the rows that see it NaN
          const float turn = slack == kSlack ? 1.f : sm.turn[p % kInfo];
          if (p > 0) {  // O follows, once the PV of the page before is complete
            ok = chunk_wait<1>(&sm.pv_done[x][(p - 1) & 1], ((p - 1) >> 1) & 1, abort_flag, st, kSiteCPv, blockIdx.x);
            if (!ok) break;
            tc_fence_after();
            scale_o<D>(colO, isnan(turn) ? k : k * turn);
          }
          l *= isnan(turn) && lim > key0 ? NAN : k;
          m = up;
          slack = kSlack;
        }
        if (!ok) break;
        l = fmaf(sum, ps.vinv, l);
        tmem_st32_wait(col, pw);
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm.p_full[x][p & 1]);
      }
      if (ok && P > 0) {
        ok = chunk_wait<1>(&sm.pv_done[x][(P - 1) & 1], ((P - 1) >> 1) & 1, abort_flag, st, kSiteCPv, blockIdx.x);
        tc_fence_after();
      }
      // Without a page no QK stands between a warp's queries and another warp's
      // stage below, which lies over them.
      if (P == 0) named_bar_sync(1 + x, kTileRows);
      if (ok) {
        // ---- the row's result, or its part. A warp's 32 rows go through its
        // quarter of the Q tile (its last QK is complete, or there was none) 64
        // columns at a time, so that the stores run along rows, a few lines each.
        const bool part = a.splits > 1;
        const int unit = sm.unit;
        const float inv = part ? 1.f : (l != 0.f ? __int_as_float(unit << 23) / l : 0.f);
        const long long pr = partial_row(a, b, h, qi, split);
        uint16_t* dst = a.out + b * a.ost.b + h * a.ost.h + static_cast<long long>(qi) * a.ost.n;
        uint8_t* stage = sm.q[x] + wq * 32 * D * 2;  // 8 KB (D = 128) or 4 KB
        constexpr int COLS = D / 2;                  // columns per pass: 32 rows of COLS floats, or D of 16 bits
#pragma unroll 1
        for (int half = 0; half < 2; ++half) {
          uint32_t o[COLS];
          if (P > 0) {
            if constexpr (D == 128) tmem_ld32x2_wait(colO + half * 64, colO + half * 64 + 32, o);
            else tmem_ld32_wait(colO + half * 32, o);
          } else {
#pragma unroll
            for (int e = 0; e < COLS; ++e) o[e] = 0;
          }
          if (part) {
#pragma unroll
            for (int e = 0; e < COLS / 4; ++e)
              st_shared_v4(stage + (lane * (COLS / 4) + ((e + lane) % (COLS / 4))) * 16, o[4 * e], o[4 * e + 1], o[4 * e + 2],
                           o[4 * e + 3]);
          } else {
#pragma unroll
            for (int e = 0; e < COLS / 8; ++e) {
              uint32_t pk[4];
#pragma unroll
              for (int z = 0; z < 4; ++z)
                pk[z] = pack2<Elem>(__uint_as_float(o[8 * e + 2 * z]) * inv, __uint_as_float(o[8 * e + 2 * z + 1]) * inv);
              st_shared_v4(stage + (lane * (COLS / 8) + ((e + lane) % (COLS / 8))) * 16, pk[0], pk[1], pk[2], pk[3]);
            }
          }
          __syncwarp();
          if (part) store_rows<COLS / 4>(a, stage, b, hk, r - lane, rows, half, split, lane);
          else store_rows<COLS / 8>(a, stage, b, hk, r - lane, rows, half, split, lane);
        }
        if (there) {
          if (part) a.part_ml[pr] = make_float2(m + static_cast<float>(unit - 127), l * unit_inverse(unit));
          else if (a.lse)
            a.lse[(static_cast<long long>(b) * a.H + h) * a.N + qi] =
                l == 0.f ? -INFINITY : (m - kPBias + log2f(l)) * kLn2C;
        }
        if (there && sm.nan) {  // NaN values among the tokens that only some rows see
          for (int u = max(c0 * kPage, least / kPage * kPage); u < min(lim, (c0 + pend) * kPage); ++u) {
            const int page = page_of(a, b, u / kPage);
            if (page < 0) continue;
            const uint8_t* vr = a.v + page * a.page_stride + (static_cast<long long>(hk) * kPage + u % kPage) * D;
            for (int e = 0; e < D; ++e) {
              if ((vr[e] & 0x7f) != 0x7f) continue;
              if (part) a.part_o[pr * D + e] = NAN;
              else dst[e] = static_cast<uint16_t>(pack2<Elem>(NAN, NAN) & 0xffffu);
            }
          }
        }
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 12) {
    tc_fence_after();
    tmem_dealloc(*static_cast<volatile uint32_t*>(&sm.tmem_base), 512);
  }
}

template <typename Elem, int D>
cudaError_t launch_chunk_t(const CacheAttnArgs& a, cudaStream_t stream) {
  const size_t smem = sizeof(ChunkSmem<D>) + 1024;
  static_assert(sizeof(ChunkSmem<D>) + 1024 <= 232448, "shared memory layout too large");
  const cudaError_t e = cudaFuncSetAttribute(cache_chunk_kernel<Elem, D>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             static_cast<int>(smem));
  if (e != cudaSuccess) return e;
  const int tiles = static_cast<int>((static_cast<long long>(a.N) * a.group + 2 * kTileRows - 1) / (2 * kTileRows));
  cache_chunk_kernel<Elem, D><<<dim3(tiles * a.splits, a.Hk, a.B), kChunkThreads, smem, stream>>>(a, tiles);
  return cudaGetLastError();
}

}  // namespace

#ifdef SOLATTN_TEST_HOOKS
cudaError_t set_test_hooks_chunk(int skip_cta, unsigned long long wait_budget_ns) {
  cudaError_t e = cudaMemcpyToSymbol(g_hook_skip_cta, &skip_cta, sizeof(skip_cta));
  if (e == cudaSuccess) e = cudaMemcpyToSymbol(g_wait_budget_ns, &wait_budget_ns, sizeof(wait_budget_ns));
  return e;
}
#endif

cudaError_t launch_cache_chunk(const CacheAttnArgs& a, cudaStream_t stream) {
  if (a.dtype == kF16)
    return a.d == 64 ? launch_chunk_t<__half, 64>(a, stream) : launch_chunk_t<__half, 128>(a, stream);
  return a.d == 64 ? launch_chunk_t<__nv_bfloat16, 64>(a, stream) : launch_chunk_t<__nv_bfloat16, 128>(a, stream);
}

}  // namespace solattn
