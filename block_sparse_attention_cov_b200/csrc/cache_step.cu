// cache_step.cu -- attention of a few queries (a decoding step), or of more over a
// short cache, and the kernel that joins partial results of a split key axis.
//
// cache_step_kernel is bound by reading the cache: 2 d bytes per key and head
// against 4 d flops per query row. One CTA takes up to 16 rows (query heads of
// one key head x new tokens) and one part of the sequence's pages. A producer
// warp keeps four pages of keys and values on their way into shared memory by TMA
// (64 KB per CTA, three CTAs per SM; with one page ahead in registers the kernel
// waited for memory at 4.1 TB/s); four warps take 32 tokens each, half of every
// other page, and keep their own running softmax, joined at the end. Fragments come from
// shared memory with 16-byte loads, which works because the order of the
// contracted index is free as long as both operands agree on it:
//   S = Q K^T: lane (g, t) holds bytes 16t.. of one token's row; word j of them is
//     the fragment of contraction step j, and Q is loaded in the same order;
//   O = P V: the softmax's accumulator layout is the A fragment of P; lane (g, t)
//     holds bytes 16g.. of the four tokens whose weights it has, byte permutes
//     pair the tokens, and byte j is column j of value tile j.
// Column n of a score tile is token n, or n ^ 4 where n is odd: with the 128-byte
// swizzle neither operand's loads meet in a bank.
// The products run on mma.sync (m16n8k16, fp16 operands, fp32 sums): a 16-row
// tile is what these calls have, a tcgen05 tile would be 7/8 empty, and at 16
// rows the tensor pipe is far from the bound.
#include <cuda_runtime.h>
#include <cmath>
#include <cstdint>

#include "cache_common.cuh"
#include "tensor_map.h"

namespace solattn {

namespace {

constexpr int kRows = 16;   // rows per CTA
constexpr int kWarps = 4;

enum : uint32_t { kSiteStepFull = 60, kSiteStepEmpty };

__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t a0, const uint32_t a1, const uint32_t a2,
                                         const uint32_t a3, const uint32_t b0, const uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

template <int D>
struct __align__(1024) StepSmem {
  static constexpr int kStages = 4;
  union {
    struct {
      uint8_t k[kStages][kPage * D];  // 128-byte rows (64 at D = 64), swizzled as wide
      uint8_t v[kStages][kPage * D];
    };
    struct {  // the warps' results, when every page is done
      float o[kWarps][kRows][D + 4];
      float m[kWarps][kRows];
      float l[kWarps][kRows];
    };
  };
  uint4 q[D / 16][32];    // Q fragments of step j, by lane
  float2 scale[kStages];  // of keys, and of values in their unit; 0 values: the page is not there
  float turn[kStages];    // what a warp's O is multiplied by before the page
  int unit[kWarps];       // of each warp's last page
  uint64_t full[kStages], empty[kStages];
  int nan;  // a value that only some rows see is NaN
  int abort_flag;
};

// Offset of 16-byte chunk c of row r: the TMA swizzle of rows of D bytes.
template <int D>
__device__ __forceinline__ uint32_t swizzled(int r, int c) {
  return D == 128 ? r * 128 + ((c ^ (r & 7)) << 4) : r * 64 + ((c ^ ((r >> 1) & 3)) << 4);
}

template <typename T, int D>
__global__ void __launch_bounds__((kWarps + 1) * 32, 3)
    cache_step_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                      const CacheAttnArgs a) {
  using Smem = StepSmem<D>;
  constexpr int ST = Smem::kStages;
  extern __shared__ uint8_t smem_raw[];
  Smem& sm = *reinterpret_cast<Smem*>(smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u));
  const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
  const int g = lane / 4, t = lane % 4;
  const int split = blockIdx.x;
  const int b = a.longest_first ? nth_longest(a, blockIdx.z, lane) : blockIdx.z;
  const int hk = blockIdx.y % a.Hk, tile = blockIdx.y / a.Hk;
  DeviceStatus* st = a.status;
  volatile int* abort_flag = &sm.abort_flag;
  start_join(a);
  if (tid == 0) {
    for (int i = 0; i < ST; ++i) {
      mbar_init(&sm.full[i], 2);  // the copies' issue and the scales
      mbar_init(&sm.empty[i], 2);  // two warps share a page
    }
    for (int i = 0; i < kWarps; ++i) sm.unit[i] = 127;
    sm.nan = 0;
    sm.abort_flag = 0;
    fence_barrier_init();
  }
  __syncthreads();
  const Extent ex = extent(a, b, split == 0 && hk == 0 && tile == 0 && tid == 0);
  const int rows = ex.cnt * a.group;
  const int r0 = tile * kRows;
  if (r0 >= rows) return;  // rows behind the sequence's queries stay as they are

  // the CTA's pages: its split's share of those that its last row sees
  int qi, qg;
  row_place(a, min(rows, r0 + kRows) - 1, &qi, &qg);
  const int seen = key_limit(ex, a.causal, qi);
  const int pages = (seen + kPage - 1) / kPage;
  const int per = (pages + a.splits - 1) / a.splits;
  const int c0 = min(pages, split * per), c1 = min(pages, c0 + per);
  row_place(a, r0, &qi, &qg);
  const int lim_all = key_limit(ex, a.causal, qi);  // row r0 sees least
  const bool zone_rows = a.causal && ex.cnt > 1;

  if (warp == kWarps) {
    // ======================= producer =======================
    const int32_t* table = a.table + b * a.table_stride;
    if (lane == 0) {
      prefetch_tensormap(&tmK);
      prefetch_tensormap(&tmV);
    }
    bool ok = true;
    int issued = 0;
    int unit = 0, before = 0;  // of the value scales: the last page's, and the last 32 pages' by lane
    for (int base = c0; base < c1 && ok; base += 32) {
      // 32 pages' numbers and scales at once
      int pg = -1;
      float ks = 0.f, vs = 0.f;
      if (base + lane < c1) {
        pg = __ldg(table + base + lane);
        if (pg < 0 || pg >= a.pages) {
          report_page(st, b);
          pg = -1;
        } else {
          ks = __ldg(a.k_scale + pg * a.scale_stride + hk);
          vs = __ldg(a.v_scale + pg * a.scale_stride + hk);
        }
      }
      const int count = min(32, c1 - base);
      // the first pages' copies go out before their scales have come
      const int ahead = base == c0 ? min(count, ST) : 0;
      auto issue = [&](int n, int page) {  // by one lane
#ifdef SOLATTN_TEST_HOOKS
        if (n == 0 && static_cast<int>(blockIdx.x) == g_hook_skip_cta) return;  // this page never arrives
#endif
        const int s = n % ST;
        if (page >= 0) {
          mbar_arrive_expect_tx(&sm.full[s], 2 * kPage * D);
          tma_load_4d(sm.k[s], &tmK, &sm.full[s], 0, 0, hk, page);
          tma_load_4d(sm.v[s], &tmV, &sm.full[s], 0, 0, hk, page);
        } else {
          mbar_arrive(&sm.full[s]);
        }
      };
      if (lane < ahead) issue(lane, pg);
      __syncwarp();
      issued = max(issued, ahead);
      const int mine = page_units(vs, unit, lane);
      vs *= unit_inverse(mine);
      // a warp's page before this one is the last but one
      int from = __shfl_sync(0xffffffffu, lane < 30 ? mine : before, (lane + 30) & 31);
      if (base == c0 && lane < 2) from = mine;
      const float turn = unit_turn(from, mine);
      before = mine;
#pragma unroll 1
      for (int i = 0; i < count && ok; ++i) {
        const int n = base + i - c0, s = n % ST;
        if (i >= ahead) {
          if (n >= ST)
            ok = __all_sync(0xffffffffu, mbar_wait(&sm.empty[s], ((n / ST) & 1) ^ 1, abort_flag, st, kSiteStepEmpty,
                                                   blockIdx.x));
          if (!ok) break;
          if (lane == i) issue(n, pg);
          issued = n + 1;
        }
        if (lane == i) {
          sm.scale[s] = make_float2(ks, vs);
          sm.turn[s] = turn;
          sm.unit[2 * (n & 1)] = mine;
          if ((c0 + n) * kPage + 32 < seen) sm.unit[2 * (n & 1) + 1] = mine;  // its warp has rows that see it
          mbar_arrive(&sm.full[s]);
        }
      }
    }
    // every copy has landed before the ring is written over and before the block
    // exits: a warp whose wait gave up has not seen its pages arrive
    if (lane == 0)
      for (int n = max(0, issued - ST); n < issued; ++n) mbar_wait_quiet(&sm.full[n % ST], (n / ST) & 1);
    __syncwarp();
    named_bar_sync(2, (kWarps + 1) * 32);
    __syncthreads();  // with the warps' results
    return;
  }

  // ======================= four warps =======================
  // Q fragments of rows g and g + 8, scaled to fp16's range, in shared memory: in
  // registers they would cost the third block of an SM (all 128 a thread are taken,
  // and at d = 128 one word spills)
  float rf[2];
  int lim[2];
#pragma unroll
  for (int x = 0; x < 2; ++x) {
    const int r = r0 + g + 8 * x;
    row_place(a, r, &qi, &qg);
    const bool there = r < rows;
    lim[x] = there ? key_limit(ex, a.causal, qi) : 0;
    uint4 w[D / 32];
    const uint16_t* src = a.q + b * a.st.b + (hk * a.group + qg) * a.st.h + static_cast<long long>(qi) * a.st.n;
#pragma unroll
    for (int y = 0; y < D / 32; ++y)  // 16 dims at 16t (+ 64) as two chunks of 8
      w[y] = there ? *reinterpret_cast<const uint4*>(src + (y / 2) * 64 + 16 * t + (y % 2) * 8) : make_uint4(0, 0, 0, 0);
    float amax = 0.f;
#pragma unroll
    for (int y = 0; y < D / 32; ++y) {
      const uint32_t u[4] = {w[y].x, w[y].y, w[y].z, w[y].w};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float2 f = unpack2<T>(u[e]);
        amax = fmaxf(amax, fmaxf(fabsf(f.x), fabsf(f.y)));
      }
    }
    amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
    amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
    float mul;
    row_factor(amax, &mul, &rf[x]);
#pragma unroll
    for (int y = 0; y < D / 32; ++y) {
      const uint32_t u[4] = {w[y].x, w[y].y, w[y].z, w[y].w};
#pragma unroll
      for (int e = 0; e < 4; ++e) {  // two dims each; step (4 dims) 2 y + e / 2
        const float2 f = unpack2<T>(u[e]);
        if (warp == 0)
          reinterpret_cast<uint32_t*>(&sm.q[2 * y + e / 2][lane])[(e & 1) * 2 + x] = pack_f16x2(f.x * mul, f.y * mul);
      }
    }
  }
  named_bar_sync(1, kWarps * 32);

  float o[D / 8][4];
#pragma unroll
  for (int j = 0; j < D / 8; ++j)
#pragma unroll
    for (int e = 0; e < 4; ++e) o[j][e] = 0.f;
  float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};

  // A warp takes half of every other page, 32 tokens at a time: two groups of 16,
  // whose products are independent. Token of score column n, and the lane's four
  // tokens of a group:
  const int first = (warp & 1) * 32, kr = (g & 1) ? g ^ 4 : g;
  const int tok[4] = {2 * t, (2 * t + 1) ^ 4, 8 + 2 * t, 8 + ((2 * t + 1) ^ 4)};
  bool ok = true;
  for (int col = c0 + warp / 2; col < c1; col += 2) {
    const int n = col - c0, s = n % ST;
    ok = __all_sync(0xffffffffu, mbar_wait(&sm.full[s], (n / ST) & 1, abort_flag, st, kSiteStepFull, blockIdx.x));
    if (!ok) break;
    const int base = col * kPage + first;
    if (base < seen) {  // warp-uniform
      const float2 kv = sm.scale[s];
      const bool gone = kv.y == 0.f;
      float sc[4][4];
#pragma unroll
      for (int nt = 0; nt < 4; ++nt)
#pragma unroll
        for (int e = 0; e < 4; ++e) sc[nt][e] = 0.f;
#pragma unroll
      for (int y = 0; y < D / 64; ++y) {
        uint4 kw[4];
#pragma unroll
        for (int nt = 0; nt < 4; ++nt)
          kw[nt] = gone ? make_uint4(0, 0, 0, 0)
                        : *reinterpret_cast<const uint4*>(sm.k[s] + swizzled<D>(first + 8 * nt + kr, t + 4 * y));
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const uint4 qf = sm.q[4 * y + j][lane];
#pragma unroll
          for (int nt = 0; nt < 4; ++nt) {
            uint32_t b0, b1;
            e4m3x4_f16(j == 0 ? kw[nt].x : (j == 1 ? kw[nt].y : (j == 2 ? kw[nt].z : kw[nt].w)), b0, b1);
            mma16816(sc[nt], qf.x, qf.y, qf.z, qf.w, b0, b1);
          }
        }
      }
      // scores in log2 units plus log2 of the value scale
      const PageScale ps = page_scale(a, kv.x, kv.y);
      const float c[2] = {ps.ck * rf[0], ps.ck * rf[1]};
#pragma unroll
      for (int nt = 0; nt < 4; ++nt)
#pragma unroll
        for (int e = 0; e < 4; ++e) sc[nt][e] = fmaf(sc[nt][e], c[e >> 1], ps.ev);
      const bool zone = base + 32 > lim_all;
      if (zone) {
#pragma unroll
        for (int nt = 0; nt < 4; ++nt)
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (base + 16 * (nt / 2) + tok[2 * (nt & 1) + (e & 1)] >= lim[e >> 1]) sc[nt][e] = -INFINITY;
      }
      float mx[2];
      bool raise = sm.turn[s] != 1.f;
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        mx[x] = -INFINITY;
#pragma unroll
        for (int nt = 0; nt < 4; ++nt) mx[x] = fmaxf(mx[x], fmaxf(sc[nt][2 * x], sc[nt][2 * x + 1]));
        mx[x] = fmaxf(mx[x], __shfl_xor_sync(0xffffffffu, mx[x], 1));
        mx[x] = fmaxf(mx[x], __shfl_xor_sync(0xffffffffu, mx[x], 2));
        raise |= mx[x] > m[x] + kSlack;
      }
      if (__any_sync(0xffffffffu, raise)) {
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          const float mn = mx[x] > m[x] + kSlack ? ceilf(mx[x]) : m[x];
          const float k = m[x] == mn ? 1.f : ex2_approx(m[x] - mn);  // 0 from -inf
          const float ko = k * sm.turn[s];  // and to the page's unit of value scales
          l[x] *= k;
#pragma unroll
          for (int j = 0; j < D / 8; ++j) {
            o[j][2 * x] *= ko;
            o[j][2 * x + 1] *= ko;
          }
          m[x] = mn;
        }
      }
      float sum[2] = {0.f, 0.f};
      const float sub[2] = {kPBias - (m[0] == -INFINITY ? 0.f : m[0]), kPBias - (m[1] == -INFINITY ? 0.f : m[1])};
#pragma unroll
      for (int nt = 0; nt < 4; ++nt)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          sc[nt][e] = ex2_approx(sc[nt][e] + sub[e >> 1]);
          sum[e >> 1] += sc[nt][e];
        }
      // a row that sees nothing of the page is not touched by its scale, NaN or not
      l[0] = sum[0] == 0.f ? l[0] : fmaf(sum[0], ps.vinv, l[0]);
      l[1] = sum[1] == 0.f ? l[1] : fmaf(sum[1], ps.vinv, l[1]);
#pragma unroll
      for (int grp = 0; grp < 2; ++grp) {
        uint32_t vw[4][D / 32];
#pragma unroll
        for (int y = 0; y < 4; ++y) {
          // rows behind the sequence hold anything, NaN too: zero weights do not
          // silence it in the product
          const int r = first + 16 * grp + tok[y];
          const bool in = !gone && col * kPage + r < ex.len;
          if constexpr (D == 128) {
            const uint4 w = in ? *reinterpret_cast<const uint4*>(sm.v[s] + swizzled<D>(r, g)) : make_uint4(0, 0, 0, 0);
            vw[y][0] = w.x;
            vw[y][1] = w.y;
            vw[y][2] = w.z;
            vw[y][3] = w.w;
          } else {
            const uint2 w = in ? *reinterpret_cast<const uint2*>(sm.v[s] + swizzled<D>(r, g / 2) + 8 * (g & 1))
                               : make_uint2(0, 0);
            vw[y][0] = w.x;
            vw[y][1] = w.y;
          }
        }
        if (zone && zone_rows) {  // a NaN value must reach only the rows that see its token
          bool bad = false;
#pragma unroll
          for (int y = 0; y < 4; ++y)
#pragma unroll
            for (int w = 0; w < D / 32; ++w) {
              bad |= has_nan8(vw[y][w]);
              vw[y][w] = drop_nan8(vw[y][w]);
            }
          if (bad) sm.nan = 1;
        }
        const float(&q0)[4] = sc[2 * grp];
        const float(&q1)[4] = sc[2 * grp + 1];
        const uint32_t p0 = pack_f16x2(q0[0], q0[1]), p1 = pack_f16x2(q0[2], q0[3]);
        const uint32_t p2 = pack_f16x2(q1[0], q1[1]), p3 = pack_f16x2(q1[2], q1[3]);
#pragma unroll
        for (int w = 0; w < D / 32; ++w) {
          // bytes of two tokens side by side: (a0, b0, a1, b1) and (a2, b2, a3, b3)
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            const uint32_t sel = half ? 0x7362 : 0x5140;
            uint32_t x0, x1, y0, y1;
            e4m3x4_f16(__byte_perm(vw[0][w], vw[1][w], sel), x0, x1);
            e4m3x4_f16(__byte_perm(vw[2][w], vw[3][w], sel), y0, y1);
            mma16816(o[4 * w + 2 * half], p0, p1, p2, p3, x0, y0);
            mma16816(o[4 * w + 2 * half + 1], p0, p1, p2, p3, x1, y1);
          }
        }
      }
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(&sm.empty[s]);
  }

  // ---- the four warps' results joined, over the ring (every copy has landed and been read)
  named_bar_sync(2, (kWarps + 1) * 32);
  const int unit = sm.unit[warp];  // references and sums without it
#pragma unroll
  for (int x = 0; x < 2; ++x) {
    l[x] += __shfl_xor_sync(0xffffffffu, l[x], 1);
    l[x] += __shfl_xor_sync(0xffffffffu, l[x], 2);
    const int r = g + 8 * x;
    if (t == 0) {
      sm.m[warp][r] = m[x] + static_cast<float>(unit - 127);
      sm.l[warp][r] = l[x] * unit_inverse(unit);
    }
    // column of value tile j and accumulator e: tile's byte j of the lanes' runs
#pragma unroll
    for (int j = 0; j < D / 8; ++j) {
      sm.o[warp][r][(D / 8) * (2 * t) + j] = o[j][2 * x];
      sm.o[warp][r][(D / 8) * (2 * t + 1) + j] = o[j][2 * x + 1];
    }
  }
  __syncthreads();
  constexpr int CPR = D / 4;  // threads per row, four columns each
  for (int i = tid; i < kRows * CPR; i += kWarps * 32) {
    const int r = i / CPR, cc = (i % CPR) * 4;
    if (r0 + r >= rows) continue;
    float mj = -INFINITY;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) mj = fmaxf(mj, sm.m[w][r]);
    float lj = 0.f;
    float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      const float mw = sm.m[w][r];
      const float k = mw == -INFINITY ? 0.f : ex2_approx(mw - mj);
      const float4 ow = *reinterpret_cast<const float4*>(&sm.o[w][r][cc]);
      // a warp that saw nothing of the row adds nothing, whatever it holds
      if (mw != -INFINITY || sm.l[w][r] != 0.f) {
        lj = fmaf(sm.l[w][r], mw == -INFINITY ? 1.f : k, lj);
        const float ko = mw == -INFINITY ? 1.f : k;
        y.x = fmaf(ow.x, ko, y.x);
        y.y = fmaf(ow.y, ko, y.y);
        y.z = fmaf(ow.z, ko, y.z);
        y.w = fmaf(ow.w, ko, y.w);
      }
    }
    row_place(a, r0 + r, &qi, &qg);
    const int h = hk * a.group + qg;
    if (sm.nan) {  // the row's own tokens of the zone: their NaN values reach its columns
      const int lr = key_limit(ex, a.causal, qi);
      float* yy = &y.x;
      for (int u = max(c0 * kPage, lim_all / 32 * 32); u < min(lr, c1 * kPage); ++u) {
        const int page = page_of(a, b, u / kPage);
        if (page < 0) continue;
        const uint8_t* vr = a.v + page * a.page_stride + (static_cast<long long>(hk) * kPage + u % kPage) * D + cc;
        for (int e = 0; e < 4; ++e)
          if ((vr[e] & 0x7f) == 0x7f) yy[e] = NAN;
      }
    }
    if (a.splits > 1) {
      const long long pr = partial_row(a, b, h, qi, split);
      *reinterpret_cast<float4*>(a.part_o + pr * D + cc) = y;
      if (cc == 0) a.part_ml[pr] = make_float2(mj, lj);
    } else {
      const float inv = lj != 0.f ? 1.f / lj : 0.f;
      uint16_t* dst = a.out + b * a.ost.b + h * a.ost.h + static_cast<long long>(qi) * a.ost.n + cc;
      *reinterpret_cast<uint2*>(dst) = make_uint2(pack2<T>(y.x * inv, y.y * inv), pack2<T>(y.z * inv, y.w * inv));
      if (cc == 0 && a.lse) {
        a.lse[(static_cast<long long>(b) * a.H + h) * a.N + qi] =
            lj == 0.f ? -INFINITY : (mj - kPBias + log2f(lj)) * kLn2C;
      }
    }
  }
}

// Joins the splits of one row: O and l brought to the largest reference. One
// CTA per row, each of its warps taking every so many-th split, eight of their
// results in flight; the order of the sums is fixed.
constexpr int kJoinWarps = 16;

template <typename T, int D>
__global__ void __launch_bounds__(kJoinWarps * 32) cache_join_kernel(const CacheAttnArgs a) {
  __shared__ float so[kJoinWarps][D];
  __shared__ float sl[kJoinWarps];
  const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32, warps = blockDim.x / 32;
  const long long row = blockIdx.x;
  const int qi = static_cast<int>(row % a.N);
  const int h = static_cast<int>(row / a.N % a.H), b = static_cast<int>(row / a.N / a.H);
  const int cnt = a.counts ? __ldg(a.counts + b) : a.N;
  asm volatile("griddepcontrol.wait;" ::: "memory");  // the parts are there
  if (qi >= cnt) return;
  const float2* ml = a.part_ml + row * a.splits;
  float mj = -INFINITY;
  for (int s = lane; s < a.splits; s += 32) mj = fmaxf(mj, ml[s].x);
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) mj = fmaxf(mj, __shfl_xor_sync(0xffffffffu, mj, off));
  constexpr int C = D / 32;
  float y[C], l = 0.f;
#pragma unroll
  for (int e = 0; e < C; ++e) y[e] = 0.f;
#pragma unroll 8
  for (int s = warp; s < a.splits; s += warps) {
    const float2 p = ml[s];
    const float* o = a.part_o + (row * a.splits + s) * D + lane * C;
    float v[C];
    if constexpr (C == 4) *reinterpret_cast<float4*>(v) = *reinterpret_cast<const float4*>(o);
    else *reinterpret_cast<float2*>(v) = *reinterpret_cast<const float2*>(o);
    const bool none = p.x == -INFINITY && p.y == 0.f;  // saw nothing of the row
    const float k = p.x == -INFINITY ? 1.f : ex2_approx(p.x - mj);
    l = none ? l : fmaf(p.y, k, l);
#pragma unroll
    for (int e = 0; e < C; ++e) y[e] = none ? y[e] : fmaf(v[e], k, y[e]);
  }
#pragma unroll
  for (int e = 0; e < C; ++e) so[warp][lane * C + e] = y[e];
  if (lane == 0) sl[warp] = l;
  __syncthreads();
  if (tid < D / 2) {
    const int c = 2 * tid;
    float lj = 0.f, y0 = 0.f, y1 = 0.f;
    for (int w = 0; w < warps; ++w) {
      lj += sl[w];
      y0 += so[w][c];
      y1 += so[w][c + 1];
    }
    const float inv = lj != 0.f ? 1.f / lj : 0.f;
    uint16_t* dst = a.out + b * a.ost.b + h * a.ost.h + static_cast<long long>(qi) * a.ost.n + c;
    *reinterpret_cast<uint32_t*>(dst) = pack2<T>(y0 * inv, y1 * inv);
    if (tid == 0 && a.lse) a.lse[row] = lj == 0.f ? -INFINITY : (mj - kPBias + log2f(lj)) * kLn2C;
  }
}

// Keys or values of a cache as a 4D tensor {d, 64, heads, pages} of bytes; one
// load brings a page of one head.
bool page_map(CUtensorMap* map, const uint8_t* base, const CacheAttnArgs& a) {
  EncodeTiledFn enc = get_encode_fn();
  if (!enc) return false;
  cuuint64_t dims[4] = {static_cast<cuuint64_t>(a.d), kPage, static_cast<cuuint64_t>(a.Hk),
                        static_cast<cuuint64_t>(a.pages)};
  cuuint64_t strides[3] = {static_cast<cuuint64_t>(a.d), static_cast<cuuint64_t>(kPage) * a.d,
                           static_cast<cuuint64_t>(a.page_stride)};
  cuuint32_t box[4] = {static_cast<cuuint32_t>(a.d), kPage, 1, 1};
  cuuint32_t estr[4] = {1, 1, 1, 1};
  return enc(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 4, const_cast<uint8_t*>(base), dims, strides, box, estr,
             CU_TENSOR_MAP_INTERLEAVE_NONE, a.d == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <typename T, int D>
cudaError_t launch_step_t(const CacheAttnArgs& a, cudaStream_t stream) {
  CUtensorMap tmK, tmV;
  if (!page_map(&tmK, a.k, a) || !page_map(&tmV, a.v, a)) return cudaErrorInvalidValue;
  const size_t smem = sizeof(StepSmem<D>) + 1024;
  const cudaError_t e = cudaFuncSetAttribute(cache_step_kernel<T, D>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             static_cast<int>(smem));
  if (e != cudaSuccess) return e;
  const int tiles = (a.N * a.group + kRows - 1) / kRows;
  cache_step_kernel<T, D><<<dim3(a.splits, tiles * a.Hk, a.B), (kWarps + 1) * 32, smem, stream>>>(tmK, tmV, a);
  return cudaGetLastError();
}

template <typename T, int D>
cudaError_t launch_join_t(const CacheAttnArgs& a, cudaStream_t stream) {
  // set up while the parts are still computed (programmatic launch); a warp per
  // four splits, D / 64 warps at least (the last step has D / 2 threads)
  const int warps = a.splits <= 16 ? 4 : (a.splits <= 32 ? 8 : kJoinWarps);
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned int>(static_cast<long long>(a.B) * a.H * a.N));
  cfg.blockDim = dim3(warps * 32);
  cfg.stream = stream;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, cache_join_kernel<T, D>, a);
}

}  // namespace

#ifdef SOLATTN_TEST_HOOKS
cudaError_t set_test_hooks_step(int skip_cta, unsigned long long wait_budget_ns) {
  cudaError_t e = cudaMemcpyToSymbol(g_hook_skip_cta, &skip_cta, sizeof(skip_cta));
  if (e == cudaSuccess) e = cudaMemcpyToSymbol(g_wait_budget_ns, &wait_budget_ns, sizeof(wait_budget_ns));
  return e;
}
#endif

cudaError_t launch_cache_step(const CacheAttnArgs& a, cudaStream_t stream) {
  if (a.dtype == kF16) return a.d == 64 ? launch_step_t<__half, 64>(a, stream) : launch_step_t<__half, 128>(a, stream);
  return a.d == 64 ? launch_step_t<__nv_bfloat16, 64>(a, stream) : launch_step_t<__nv_bfloat16, 128>(a, stream);
}

cudaError_t launch_cache_join(const CacheAttnArgs& a, cudaStream_t stream) {
  if (a.dtype == kF16) return a.d == 64 ? launch_join_t<__half, 64>(a, stream) : launch_join_t<__half, 128>(a, stream);
  return a.d == 64 ? launch_join_t<__nv_bfloat16, 64>(a, stream) : launch_join_t<__nv_bfloat16, 128>(a, stream);
}

}  // namespace solattn
