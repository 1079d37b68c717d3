// cache_chunk.cu -- attention of many queries (a prompt, a chunk, a video frame)
// over the 8-bit cache, on tcgen05.
//
// One CTA takes 256 query rows of one key head (token-major, the heads of the
// group side by side) as two 128-row tiles, and one part of the keys. Both tiles
// use every key tile that is converted, so the conversion from e4m3 to fp16
// (tcgen05 multiplies operands of one type, and 8-bit queries would lose the
// scores' accuracy) is paid once per 256 rows: 128 threads load a page's bytes,
// convert them and store them in the swizzled operand layout.
//
//   warps 0-3, 4-7  softmax of tile 0 / tile 1: one thread per row, S and P in
//                   TMEM (P in fp16 over the first half of its own S), O scaled
//                   in TMEM only when a row's reference moves
//   warps 8-11      cache pages to fp16 operands: 128 keys a stage, two stages
//   warp 12         issues every MMA: per key tile PV of the tile before, then QK,
//                   tile 0 then tile 1, so one tile's products run while the other
//                   tile's softmax does (warps 13-15 only give their registers)
//
// Bounds per key tile at d = 128 and two tiles: 2,048 cycles of tensor pipe, and
// as many of exponentials (32,768 at 16 a cycle).
#include <cuda_runtime.h>
#include <cmath>
#include <cstdint>

#include "cache_common.cuh"

namespace solattn {

namespace {

constexpr int kTileRows = 128;
constexpr int kTileKeys = 128;
constexpr int kChunkThreads = 512;  // 16 warps, 128 registers per thread at launch
constexpr int kStages = 2;
constexpr int kInfo = 4;

enum : uint32_t {
  kSiteCQ = 40, kSiteCKFull, kSiteCKEmpty, kSiteCVFull, kSiteCVEmpty, kSiteCSFull, kSiteCPFull, kSiteCPv,
  kSiteCInfo,
};

template <int D>
struct __align__(1024) ChunkSmem {
  uint8_t q[2][kTileRows * D * 2];        // SW128 K-major panels of 128 rows
  uint8_t k[kStages][kTileKeys * D * 2];  // the same
  uint8_t v[kStages][kTileKeys * D * 2];  // two 64-token blocks, SW128 panels of 64 rows
  PageScale info[kInfo][2];
  uint64_t q_full, k_full[kStages], k_empty[kStages], v_full[kStages], v_empty[kStages];
  uint64_t s_full[2], p_full[2], pv_done[2], info_full[kInfo], mma_done;
  uint32_t tmem_base;
  int abort_flag;
  int nan;
};

// fp16 operands: the format fields of the instruction descriptor are 0.
__host__ __device__ constexpr uint32_t idesc_f16_f32(int M, int N, bool b_mn_major) {
  return (1u << 4) | (static_cast<uint32_t>(b_mn_major) << 16) | (static_cast<uint32_t>(N >> 3) << 17) |
         (static_cast<uint32_t>(M >> 4) << 24);
}

// 2^k for an integral k <= 0 as an fp16 pair; 0 below fp16's range.
__device__ __forceinline__ uint32_t pow2_f16x2(float k) {
  const __half h = __float2half_rn(k < -30.f ? 0.f : ex2_approx(k));
  const uint32_t u = __half_as_ushort(h);
  return u | (u << 16);
}
__device__ __forceinline__ uint32_t mul_f16x2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}

// Rare paths, out of line; warp-collective, a lane with factor 1 keeps its row.
static __device__ __noinline__ void scale_p_half(uint32_t taddr, float k) {
  const uint32_t f = pow2_f16x2(k);
  uint32_t pw[32];
  tmem_ld32_wait(taddr, pw);
#pragma unroll
  for (int i = 0; i < 32; ++i) pw[i] = mul_f16x2(pw[i], f);
  tmem_st32_wait(taddr, pw);
}
template <int D>
static __device__ __noinline__ void scale_o(uint32_t taddr, float f) {
#pragma unroll 1
  for (int ch = 0; ch < D / 16; ++ch) {
    uint32_t ov[16];
    tmem_ld16_wait(taddr + ch * 16, ov);
#pragma unroll
    for (int x = 0; x < 16; ++x) ov[x] = __float_as_uint(__uint_as_float(ov[x]) * f);
    tmem_st16_wait(taddr + ch * 16, ov);
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

__device__ __forceinline__ void st_shared_v4(void* p, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" ::"r"(smem_u32(p)), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
}

template <typename Elem, int D>
__global__ void __launch_bounds__(kChunkThreads, 1) cache_chunk_kernel(const CacheAttnArgs a, int tiles) {
  extern __shared__ uint8_t smem_raw[];
  ChunkSmem<D>& sm =
      *reinterpret_cast<ChunkSmem<D>*>(smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u));
  const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
  // the tiles that see most keys first
  const int split = blockIdx.x % a.splits, mt = tiles - 1 - blockIdx.x / a.splits;
  const int hk = blockIdx.y, b = blockIdx.z;
  DeviceStatus* st = a.status;
  volatile int* abort_flag = &sm.abort_flag;
  const Extent ex = extent(a, b, split == 0 && hk == 0 && mt == 0 && tid == 0);
  const int rows = ex.cnt * a.group;
  const int r0 = mt * 2 * kTileRows;
  if (r0 >= rows) return;  // rows behind the sequence's queries stay as they are
  const int nq = rows - r0 > kTileRows ? 2 : 1;  // 128-row tiles with rows in them
  const int last_row = min(rows, r0 + 2 * kTileRows) - 1;
  const int seen = key_limit(ex, a.causal, last_row / a.group);  // keys that some row sees
  const int least = key_limit(ex, a.causal, r0 / a.group);       // keys that every row sees
  const int ktiles = (seen + kTileKeys - 1) / kTileKeys;
  const int per = (ktiles + a.splits - 1) / a.splits;
  const int t0 = min(ktiles, split * per), T = min(ktiles, t0 + per) - t0;

  if (tid == 0) {
    mbar_init(&sm.q_full, 4 * nq);
    for (int i = 0; i < kStages; ++i) {
      mbar_init(&sm.k_full[i], 4);
      mbar_init(&sm.v_full[i], 4);
      mbar_init(&sm.k_empty[i], 1);
      mbar_init(&sm.v_empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sm.s_full[i], 1);
      mbar_init(&sm.p_full[i], 4);
      mbar_init(&sm.pv_done[i], 1);
    }
    for (int i = 0; i < kInfo; ++i) mbar_init(&sm.info_full[i], 1);
    mbar_init(&sm.mma_done, 1);
    sm.abort_flag = 0;
    sm.nan = 0;
    fence_barrier_init();
  }
  if (warp == 12) {
    tmem_alloc(&sm.tmem_base, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sm.tmem_base;
  // TMEM columns: S / P of tile 0 at 0, of tile 1 at 128; O of tile 0 at 256, of tile 1 at 384

  // Registers: 152 for the 256 softmax threads, 104 for the other 256 (65,536 in all).
  if (warp >= 12) {
    regs_dec<104>();
    if (warp == 12) {
    // ======================= MMA issuer =======================
    constexpr uint32_t idesc_qk = idesc_f16_f32(kTileRows, kTileKeys, false);
    constexpr uint32_t idesc_pv = idesc_f16_f32(kTileRows, D, true);
    const uint64_t qd0 = sw128_desc(smem_u32(&sm.q[0][0]), 16, 1024);
    const uint64_t kd0 = sw128_desc(smem_u32(&sm.k[0][0]), 16, 1024);
    const uint64_t vd0 = sw128_desc(smem_u32(&sm.v[0][0]), 8192, 1024);
    bool ok = T == 0 || chunk_wait(&sm.q_full, 0, abort_flag, st, kSiteCQ, blockIdx.x);
    for (int t = 0; t <= T && T > 0 && ok; ++t) {
      if (t < T) ok = chunk_wait(&sm.k_full[t % kStages], (t / kStages) & 1, abort_flag, st, kSiteCKFull, blockIdx.x);
      if (t > 0 && ok)
        ok = chunk_wait(&sm.v_full[(t - 1) % kStages], ((t - 1) / kStages) & 1, abort_flag, st, kSiteCVFull,
                        blockIdx.x);
      for (int x = 0; x < nq && ok; ++x) {
        if (t > 0) {  // PV of the tile before
          ok = chunk_wait(&sm.p_full[x], (t - 1) & 1, abort_flag, st, kSiteCPFull, blockIdx.x);
          if (!ok) break;
          tc_fence_after();
          if (elect_one()) {
            const uint32_t vst = (t - 1) % kStages;
            for (int kk = 0; kk < kTileKeys / 16; ++kk) {
              const uint32_t off = vst * (kTileKeys * D * 2) + (kk / 4) * (kPage * D * 2) + (kk % 4) * 2048;
              mma_ts(tmem + 256 + x * 128, tmem + x * 128 + kk * 8, vd0 + (off >> 4), idesc_pv,
                     (t > 1 || kk > 0) ? 1u : 0u);
            }
            mma_commit(&sm.pv_done[x]);
            if (x == nq - 1) mma_commit(&sm.v_empty[vst]);
          }
          __syncwarp();
        }
        if (t < T) {  // QK: after the PV that reads P from the same columns (issued by this thread, in order)
          tc_fence_after();
          if (elect_one()) {
            const uint32_t kst = t % kStages;
            for (int kk = 0; kk < D / 16; ++kk) {
              const uint32_t off = (kk / 4) * (kTileRows * 128) + (kk % 4) * 32;
              mma_ss(tmem + x * 128, qd0 + ((x * (kTileRows * D * 2) + off) >> 4),
                     kd0 + ((kst * (kTileKeys * D * 2) + off) >> 4), idesc_qk, kk > 0 ? 1u : 0u);
            }
            mma_commit(&sm.s_full[x]);
            if (x == nq - 1) mma_commit(&sm.k_empty[kst]);
          }
          __syncwarp();
        }
      }
    }
    if (elect_one()) mma_commit(&sm.mma_done);  // teardown: issued MMAs complete before TMEM is freed
    __syncwarp();
    mbar_wait_quiet(&sm.mma_done, 0);
    __syncwarp();
    }
  } else if (warp >= 8) {
    regs_dec<104>();
    // ======================= cache pages to fp16 operands =======================
    const int ct = tid - 256;
    constexpr int LPR = D / 16;               // lanes per row (16 bytes each)
    constexpr int ROWS = 128 / LPR;           // rows per pass of the 128 threads
    constexpr int PASSES = kTileKeys / ROWS;  // 8 (d = 128) or 4
    const int c = ct % LPR, rr = ct / LPR;
    const long long lane_off = static_cast<long long>(hk) * kPage * D + 16 * c;
    const int32_t* table = a.table + b * a.table_stride;
    const int npages = (ex.len + kPage - 1) / kPage;
    // pages of key tile t (-1: not there)
    auto pages_of = [&](int t, int (&pg)[2]) {
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        const int col = (t0 + t) * 2 + x;
        pg[x] = -1;
        if (t < T && col < npages) {
          pg[x] = __ldg(table + col);
          if (pg[x] < 0 || pg[x] >= a.pages) {
            report_page(st, b);
            pg[x] = -1;
          }
        }
      }
    };
    auto load = [&](uint4 (&w)[PASSES], const uint8_t* src, const int (&pg)[2], int row_end) {
#pragma unroll
      for (int i = 0; i < PASSES; ++i) {
        const int row = i * ROWS + rr;
        const int p = row < kPage ? pg[0] : pg[1];
        w[i] = (p >= 0 && row < row_end)
                   ? __ldg(reinterpret_cast<const uint4*>(src + p * a.page_stride + lane_off + (row % kPage) * D))
                   : make_uint4(0, 0, 0, 0);
      }
    };
    // 16 e4m3 of a row: two 16-byte chunks of fp16; lanes of the second panel
    // store theirs in the other order, so that a quarter-warp's eight stores
    // (one row, or two) fall into different banks
    auto store = [&](const uint4 (&w)[PASSES], uint8_t* dst, int panel_rows, int block_rows) {
#pragma unroll
      for (int i = 0; i < PASSES; ++i) {
        const int row = i * ROWS + rr;
        uint8_t* base = dst + (row / block_rows) * (block_rows * D * 2) + (c / 4) * (panel_rows * 128);
        const int r = row % block_rows;
        const uint32_t u[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
        uint32_t f[8];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          f[2 * e] = e4m3x2_f16x2(u[e] & 0xffffu);
          f[2 * e + 1] = e4m3x2_f16x2(u[e] >> 16);
        }
        const int ch = 2 * (c % 4);
        if (c < 4) {
          st_shared_v4(base + sw128(r, ch), f[0], f[1], f[2], f[3]);
          st_shared_v4(base + sw128(r, ch + 1), f[4], f[5], f[6], f[7]);
        } else {
          st_shared_v4(base + sw128(r, ch + 1), f[4], f[5], f[6], f[7]);
          st_shared_v4(base + sw128(r, ch), f[0], f[1], f[2], f[3]);
        }
      }
    };
    uint4 kw[PASSES], vw[PASSES];
    int pg[2], pn[2];
    pages_of(0, pg);
    if (T > 0) load(kw, a.k, pg, kTileKeys);
    for (int t = 0; t < T; ++t) {
      const int s = t % kStages;
      const uint32_t ph = ((t / kStages) & 1) ^ 1;
      const int key0 = (t0 + t) * kTileKeys;
      load(vw, a.v, pg, ex.len - key0);  // rows behind the sequence as zeros: they may hold NaN
      pages_of(t + 1, pn);
      float ks = 0.f, vs = 0.f;
      if (ct < 2 && pg[ct] >= 0) {
        ks = __ldg(a.k_scale + pg[ct] * a.scale_stride + hk);
        vs = __ldg(a.v_scale + pg[ct] * a.scale_stride + hk);
      }
      if (t >= kStages && !chunk_wait(&sm.k_empty[s], ph, abort_flag, st, kSiteCKEmpty, blockIdx.x)) break;
      if (ct < 2) sm.info[t % kInfo][ct] = page_scale(a, ks, vs);
      store(kw, sm.k[s], kTileKeys, kTileKeys);
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) {
        // the page scales were written by lanes 0 and 1 of the first of these warps
        if (warp == 8) mbar_arrive(&sm.info_full[t % kInfo]);
        mbar_arrive(&sm.k_full[s]);
      }
      if (t + 1 < T) load(kw, a.k, pn, kTileKeys);
      if (a.causal && key0 + kTileKeys > least) {  // a NaN value must reach only the rows that see its token
        bool bad = false;
#pragma unroll
        for (int i = 0; i < PASSES; ++i) {
          bad |= has_nan8(vw[i].x) | has_nan8(vw[i].y) | has_nan8(vw[i].z) | has_nan8(vw[i].w);
          vw[i] = make_uint4(drop_nan8(vw[i].x), drop_nan8(vw[i].y), drop_nan8(vw[i].z), drop_nan8(vw[i].w));
        }
        if (bad) sm.nan = 1;
      }
      if (t >= kStages && !chunk_wait(&sm.v_empty[s], ph, abort_flag, st, kSiteCVEmpty, blockIdx.x)) break;
      store(vw, sm.v[s], kPage, kPage);
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&sm.v_full[s]);
      pg[0] = pn[0];
      pg[1] = pn[1];
    }
  } else {
    regs_inc<152>();
    if (warp / 4 < nq) {
    // ======================= softmax =======================
    const int x = warp / 4, wq = warp % 4;
    const int lr = wq * 32 + lane;  // row of the tile == TMEM lane
    const int r = r0 + x * kTileRows + lr;
    const bool there = r < rows;
    const int qi = r / a.group, h = hk * a.group + r % a.group;
    const int lim = there ? key_limit(ex, a.causal, qi) : 0;
    const uint32_t lane_sel = static_cast<uint32_t>(wq * 32) << 16;
    const uint32_t colS = tmem + x * 128 + lane_sel, colO = tmem + 256 + x * 128 + lane_sel;
    // ---- the row of Q, scaled to fp16's range, into the operand layout
    float rf;
    {
      const uint16_t* src = a.q + b * a.st.b + h * a.st.h + static_cast<long long>(qi) * a.st.n;
      uint4 w[D / 8];
      float amax = 0.f;
#pragma unroll
      for (int i = 0; i < D / 8; ++i) {
        w[i] = there ? __ldg(reinterpret_cast<const uint4*>(src + 8 * i)) : make_uint4(0, 0, 0, 0);
        const uint32_t u[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float2 f = unpack2<Elem>(u[e]);
          amax = fmaxf(amax, fmaxf(fabsf(f.x), fabsf(f.y)));
        }
      }
      float mul;
      row_factor(amax, &mul, &rf);
#pragma unroll
      for (int i = 0; i < D / 8; ++i) {
        const uint32_t u[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
        uint32_t p[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float2 f = unpack2<Elem>(u[e]);
          p[e] = pack_f16x2(f.x * mul, f.y * mul);
        }
        st_shared_v4(&sm.q[x][(i / 8) * (kTileRows * 128) + sw128(lr, i % 8)], p[0], p[1], p[2], p[3]);
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&sm.q_full);
    }
    float m = -INFINITY, l = 0.f;
    bool ok = true;
    for (int t = 0; t < T; ++t) {
      ok = chunk_wait<1>(&sm.info_full[t % kInfo], (t / kInfo) & 1, abort_flag, st, kSiteCInfo, blockIdx.x);
      if (ok) ok = chunk_wait<1>(&sm.s_full[x], t & 1, abort_flag, st, kSiteCSFull, blockIdx.x);
      if (!ok) break;
      tc_fence_after();
      const int key0 = (t0 + t) * kTileKeys;
      float mn = m, lt = 0.f;
#pragma unroll 1
      for (int hh = 0; hh < 2; ++hh) {  // one page at a time
        const PageScale ps = sm.info[t % kInfo][hh];
        uint32_t sv[64];
        tmem_ld32x2_wait(colS + hh * 64, colS + hh * 64 + 32, sv);
        const int valid = lim - (key0 + hh * kPage);
        if (__any_sync(0xffffffffu, valid < kPage)) {
#pragma unroll
          for (int i = 0; i < 64; ++i)
            if (i >= valid) sv[i] = 0xff800000u;
        }
        float mx = -INFINITY;
#pragma unroll
        for (int i = 0; i < 64; i += 2) mx = fmaxf(mx, fmaxf(__uint_as_float(sv[i]), __uint_as_float(sv[i + 1])));
        // never 0, which would turn a masked key's -inf into NaN
        const float c = fmaxf(ps.ck * rf, 1.17549435e-38f);
        const float tm = mx == -INFINITY || ps.vinv == 0.f ? -INFINITY : fmaf(mx, c, ps.ev);
        if (__any_sync(0xffffffffu, tm > mn + kSlack)) {
          const float up = tm > mn + kSlack ? ceilf(tm) : mn;
          if (hh == 1) {  // the first page's P and sum follow
            scale_p_half(colS, mn == up || mn == -INFINITY ? 0.f : mn - up);
            lt = mn == up ? lt : (mn == -INFINITY ? lt : lt * ex2_approx(mn - up));
          }
          mn = up;
        }
        const float add = ps.vinv == 0.f ? -INFINITY : ps.ev + kPBias - (mn == -INFINITY ? 0.f : mn);
        float s0 = 0.f, s1 = 0.f;
        uint32_t pw[32];
#pragma unroll
        for (int i = 0; i < 32; ++i) {
          const float p0 = ex2_approx(fmaf(__uint_as_float(sv[2 * i]), c, add));
          const float p1 = ex2_approx(fmaf(__uint_as_float(sv[2 * i + 1]), c, add));
          s0 += p0;
          s1 += p1;
          pw[i] = pack_f16x2(p0, p1);
        }
        lt = fmaf(s0 + s1, ps.vinv, lt);
        tmem_st32_wait(colS + hh * 32, pw);
      }
      // ---- O and the sum follow the reference (rare after the first tiles)
      const bool moved = mn != m && m != -INFINITY;
      if (__any_sync(0xffffffffu, moved)) {
        // here t > 0: the PV of the tile before has to be complete
        ok = chunk_wait<1>(&sm.pv_done[x], (t - 1) & 1, abort_flag, st, kSiteCPv, blockIdx.x);
        if (!ok) break;
        tc_fence_after();
        scale_o<D>(colO, moved ? ex2_approx(m - mn) : 1.f);
      }
      l = fmaf(l, m == mn || m == -INFINITY ? 1.f : ex2_approx(m - mn), lt);
      m = mn;
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&sm.p_full[x]);
    }
    if (ok && T > 0) {
      ok = chunk_wait<1>(&sm.pv_done[x], (T - 1) & 1, abort_flag, st, kSiteCPv, blockIdx.x);
      tc_fence_after();
    }
    if (ok) {
      // ---- the row's result, or its part
      const bool part = a.splits > 1;
      const float inv = part ? 1.f : (l != 0.f ? 1.f / l : 0.f);
      const long long pr = partial_row(a, b, h, qi, split);
      uint16_t* dst = a.out + b * a.ost.b + h * a.ost.h + static_cast<long long>(qi) * a.ost.n;
#pragma unroll 1
      for (int ch = 0; ch < D / 16; ++ch) {
        uint32_t o[16];
        if (T > 0) {
          tmem_ld16_wait(colO + ch * 16, o);
        } else {
#pragma unroll
          for (int e = 0; e < 16; ++e) o[e] = 0;
        }
        if (there && part) {
          float4* d4 = reinterpret_cast<float4*>(a.part_o + pr * D + ch * 16);
#pragma unroll
          for (int e = 0; e < 4; ++e)
            d4[e] = make_float4(__uint_as_float(o[4 * e]), __uint_as_float(o[4 * e + 1]),
                                __uint_as_float(o[4 * e + 2]), __uint_as_float(o[4 * e + 3]));
        } else if (there) {
          uint32_t pk[8];
#pragma unroll
          for (int e = 0; e < 8; ++e)
            pk[e] = pack2<Elem>(__uint_as_float(o[2 * e]) * inv, __uint_as_float(o[2 * e + 1]) * inv);
          uint4* d4 = reinterpret_cast<uint4*>(dst + ch * 16);
          d4[0] = make_uint4(pk[0], pk[1], pk[2], pk[3]);
          d4[1] = make_uint4(pk[4], pk[5], pk[6], pk[7]);
        }
        __syncwarp();
      }
      if (there) {
        if (part) a.part_ml[pr] = make_float2(m, l);
        else if (a.lse)
          a.lse[(static_cast<long long>(b) * a.H + h) * a.N + qi] =
              l == 0.f ? -INFINITY : (m - kPBias + log2f(l)) * kLn2C;
      }
      if (there && sm.nan) {  // NaN values among the tokens that only some rows see
        for (int u = max(t0 * kTileKeys, least / kTileKeys * kTileKeys); u < min(lim, (t0 + T) * kTileKeys); ++u) {
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
    tmem_dealloc(tmem, 512);
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

cudaError_t launch_cache_chunk(const CacheAttnArgs& a, cudaStream_t stream) {
  if (a.dtype == kF16)
    return a.d == 64 ? launch_chunk_t<__half, 64>(a, stream) : launch_chunk_t<__half, 128>(a, stream);
  return a.d == 64 ? launch_chunk_t<__nv_bfloat16, 64>(a, stream) : launch_chunk_t<__nv_bfloat16, 128>(a, stream);
}

}  // namespace solattn
