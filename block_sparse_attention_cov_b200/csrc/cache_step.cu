// cache_step.cu -- attention of a few queries (a decoding step) over the 8-bit
// cache, and the kernel that joins partial results of a split key axis.
//
// cache_step_kernel is bound by reading the cache: 2 d bytes per key and head
// against 4 d flops per query row. One CTA takes up to 16 rows (query heads of
// one key head x new tokens) and one part of the sequence's pages; its four
// warps take 16 of a page's 64 tokens each and keep their own running softmax,
// joined at the end. The next page's keys and values are in flight, in
// registers, while a page is multiplied: fragments are loaded straight from the
// cache with 16-byte loads, which works because the order of the contracted
// index is free as long as both operands agree on it:
//   S = Q K^T: lane (g, t) holds bytes 16t.. of token g's row; word j of them is
//     the fragment of contraction step j, and Q is loaded in the same order;
//   O = P V: the softmax's accumulator layout is the A fragment of P; lane (g, t)
//     holds bytes 16g.. of tokens 2t, 2t+1, 2t+8, 2t+9, byte permutes pair the
//     tokens, and byte j is column j of value tile j: 16 tiles of 8 columns.
// The products run on mma.sync (m16n8k16, fp16 operands, fp32 sums): a 16-row
// tile is what these calls have, a tcgen05 tile would be 7/8 empty, and at 16
// rows the tensor pipe is far from the bound.
#include <cuda_runtime.h>
#include <cmath>
#include <cstdint>

#include "cache_common.cuh"

namespace solattn {

namespace {

constexpr int kRows = 16;   // rows per CTA
constexpr int kWarps = 4;

__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t a0, const uint32_t a1, const uint32_t a2,
                                         const uint32_t a3, const uint32_t b0, const uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint4 ld_cache(const uint8_t* p) {
  uint4 r;
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w)
               : "l"(p));
  return r;
}
__device__ __forceinline__ uint2 ld_cache8(const uint8_t* p) {
  uint2 r;
  asm volatile("ld.global.nc.L1::no_allocate.v2.u32 {%0,%1}, [%2];" : "=r"(r.x), "=r"(r.y) : "l"(p));
  return r;
}

// One warp's 16 tokens of a page, as loaded.
template <int D>
struct Tokens {
  uint32_t k[2][D / 16];  // token 8 nt + g: bytes 16t.. (and 64 + 16t.. at D = 128)
  uint32_t v[4][D / 32];  // tokens 2t, 2t+1, 2t+8, 2t+9: bytes (D/8) g ..
  float ks, vs;           // the page's scales; vs = 0: the page is not there
};

template <int D>
struct StepSmem {
  float o[kWarps][kRows][D + 4];
  float m[kWarps][kRows];
  float l[kWarps][kRows];
  int nan;  // a value of the causal zone is NaN
};

template <typename T, int D>
__global__ void __launch_bounds__(kWarps * 32, 2) cache_step_kernel(const CacheAttnArgs a) {
  __shared__ StepSmem<D> sm;
  const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
  const int g = lane / 4, t = lane % 4;
  const int split = blockIdx.x, b = blockIdx.z;
  const int hk = blockIdx.y % a.Hk, tile = blockIdx.y / a.Hk;
  const Extent ex = extent(a, b, split == 0 && hk == 0 && tile == 0 && tid == 0);
  const int rows = ex.cnt * a.group;
  const int r0 = tile * kRows;
  if (r0 >= rows) return;  // rows behind the sequence's queries stay as they are
  if (tid == 0) sm.nan = 0;
  __syncthreads();

  // the CTA's pages: its split's share of those that its last row sees
  const int last_row = min(rows, r0 + kRows) - 1;
  const int seen = key_limit(ex, a.causal, last_row / a.group);
  const int pages = (seen + kPage - 1) / kPage;
  const int per = (pages + a.splits - 1) / a.splits;
  const int c0 = min(pages, split * per), c1 = min(pages, c0 + per);

  // Q fragments of rows g and g + 8, scaled to fp16's range
  uint32_t qa[D / 16][4];
  float rf[2];
  int lim[2];
#pragma unroll
  for (int x = 0; x < 2; ++x) {
    const int r = r0 + g + 8 * x;
    const int i = r / a.group, h = hk * a.group + r % a.group;
    const bool there = r < rows;
    lim[x] = there ? key_limit(ex, a.causal, i) : 0;
    uint4 w[D / 32];
    const uint16_t* src = a.q + b * a.st.b + h * a.st.h + static_cast<long long>(i) * a.st.n;
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
        qa[2 * y + e / 2][(e & 1) * 2 + x] = pack_f16x2(f.x * mul, f.y * mul);
      }
    }
  }
  const int lim_all = min(__shfl_sync(0xffffffffu, lim[0], 0), ex.len);  // row r0 sees least
  const bool zone_rows = a.causal && ex.cnt > 1;

  float o[D / 8][4];
#pragma unroll
  for (int j = 0; j < D / 8; ++j)
#pragma unroll
    for (int e = 0; e < 4; ++e) o[j][e] = 0.f;
  float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};

  const uint8_t* kb = a.k + static_cast<long long>(hk) * kPage * D + (warp * 16 + g) * D + 16 * t;
  const uint8_t* vb = a.v + static_cast<long long>(hk) * kPage * D + (warp * 16 + 2 * t) * D + (D / 8) * g;
  // Issues a page's loads; nothing here waits for one.
  auto fetch = [&](Tokens<D>& x, int col, int page) {
    const bool there = page >= 0 && page < a.pages;
    if (!there) report_page(a.status, b);
    const long long at = there ? page * a.page_stride : 0;
    x.ks = there ? __ldg(a.k_scale + page * a.scale_stride + hk) : 0.f;
    x.vs = there ? __ldg(a.v_scale + page * a.scale_stride + hk) : 0.f;
#pragma unroll
    for (int nt = 0; nt < 2; ++nt) {
#pragma unroll
      for (int y = 0; y < D / 64; ++y) {
        const uint4 w = there ? ld_cache(kb + at + nt * 8 * D + y * 64) : make_uint4(0, 0, 0, 0);
        x.k[nt][4 * y] = w.x;
        x.k[nt][4 * y + 1] = w.y;
        x.k[nt][4 * y + 2] = w.z;
        x.k[nt][4 * y + 3] = w.w;
      }
    }
    const int pos = col * kPage + warp * 16 + 2 * t;  // of the lane's first token
#pragma unroll
    for (int y = 0; y < 4; ++y) {
      const int off = (y & 1) + (y >> 1) * 8;
      // rows behind the sequence hold anything, NaN too: zero weights do not
      // silence it in the product
      const bool in = there && pos + off < ex.len;
      if constexpr (D == 128) {
        const uint4 w = in ? ld_cache(vb + at + off * D) : make_uint4(0, 0, 0, 0);
        x.v[y][0] = w.x;
        x.v[y][1] = w.y;
        x.v[y][2] = w.z;
        x.v[y][3] = w.w;
      } else {
        const uint2 w = in ? ld_cache8(vb + at + off * D) : make_uint2(0, 0);
        x.v[y][0] = w.x;
        x.v[y][1] = w.y;
      }
    }
  };

  const int32_t* table = a.table + b * a.table_stride;
  Tokens<D> nxt;
  int page = 0;  // of column col + 1, loaded one trip ahead of the page itself
  if (c0 < c1) {
    fetch(nxt, c0, __ldg(table + c0));
    if (c0 + 1 < c1) page = __ldg(table + c0 + 1);
  }
  for (int col = c0; col < c1; ++col) {
    Tokens<D> cur = nxt;
    if (col + 1 < c1) fetch(nxt, col + 1, page);
    if (col + 2 < c1) page = __ldg(table + col + 2);
    const int base = col * kPage + warp * 16;
    if (base >= seen) continue;  // warp-uniform
    float s[2][4];
#pragma unroll
    for (int nt = 0; nt < 2; ++nt) {
#pragma unroll
      for (int e = 0; e < 4; ++e) s[nt][e] = 0.f;
#pragma unroll
      for (int j = 0; j < D / 16; ++j) {
        uint32_t b0, b1;
        e4m3x4_f16(cur.k[nt][j], b0, b1);
        mma16816(s[nt], qa[j][0], qa[j][1], qa[j][2], qa[j][3], b0, b1);
      }
    }
    // scores in log2 units plus log2 of the value scale
    const PageScale ps = page_scale(a, cur.ks, cur.vs);
    const float c[2] = {ps.ck * rf[0], ps.ck * rf[1]};
#pragma unroll
    for (int nt = 0; nt < 2; ++nt)
#pragma unroll
      for (int e = 0; e < 4; ++e) s[nt][e] = fmaf(s[nt][e], c[e >> 1], ps.ev);
    if (base + 16 > lim_all) {
#pragma unroll
      for (int nt = 0; nt < 2; ++nt)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (base + nt * 8 + 2 * t + (e & 1) >= lim[e >> 1]) s[nt][e] = -INFINITY;
      if (zone_rows) {  // a NaN value must reach only the rows that see its token
        bool bad = false;
#pragma unroll
        for (int y = 0; y < 4; ++y)
#pragma unroll
          for (int w = 0; w < D / 32; ++w) {
            bad |= has_nan8(cur.v[y][w]);
            cur.v[y][w] = drop_nan8(cur.v[y][w]);
          }
        if (bad) sm.nan = 1;
      }
    }
    float mx[2];
    bool raise = false;
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      mx[x] = fmaxf(fmaxf(s[0][2 * x], s[0][2 * x + 1]), fmaxf(s[1][2 * x], s[1][2 * x + 1]));
      mx[x] = fmaxf(mx[x], __shfl_xor_sync(0xffffffffu, mx[x], 1));
      mx[x] = fmaxf(mx[x], __shfl_xor_sync(0xffffffffu, mx[x], 2));
      raise |= mx[x] > m[x] + kSlack;
    }
    if (__any_sync(0xffffffffu, raise)) {
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        const float mn = mx[x] > m[x] + kSlack ? ceilf(mx[x]) : m[x];
        const float k = m[x] == mn ? 1.f : ex2_approx(m[x] - mn);  // 0 from -inf
        l[x] *= k;
#pragma unroll
        for (int j = 0; j < D / 8; ++j) {
          o[j][2 * x] *= k;
          o[j][2 * x + 1] *= k;
        }
        m[x] = mn;
      }
    }
    float sum[2] = {0.f, 0.f};
#pragma unroll
    for (int nt = 0; nt < 2; ++nt)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float mr = m[e >> 1] == -INFINITY ? 0.f : m[e >> 1];
        s[nt][e] = ex2_approx(s[nt][e] - mr + kPBias);
        sum[e >> 1] += s[nt][e];
      }
    l[0] = fmaf(sum[0], ps.vinv, l[0]);
    l[1] = fmaf(sum[1], ps.vinv, l[1]);
    const uint32_t p0 = pack_f16x2(s[0][0], s[0][1]), p1 = pack_f16x2(s[0][2], s[0][3]);
    const uint32_t p2 = pack_f16x2(s[1][0], s[1][1]), p3 = pack_f16x2(s[1][2], s[1][3]);
#pragma unroll
    for (int w = 0; w < D / 32; ++w) {
      // bytes of two tokens side by side: (a0, b0, a1, b1) and (a2, b2, a3, b3)
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        const uint32_t sel = half ? 0x7362 : 0x5140;
        uint32_t x0, x1, y0, y1;
        e4m3x4_f16(__byte_perm(cur.v[0][w], cur.v[1][w], sel), x0, x1);
        e4m3x4_f16(__byte_perm(cur.v[2][w], cur.v[3][w], sel), y0, y1);
        mma16816(o[4 * w + 2 * half], p0, p1, p2, p3, x0, y0);
        mma16816(o[4 * w + 2 * half + 1], p0, p1, p2, p3, x1, y1);
      }
    }
  }

  // ---- the four warps' results joined
#pragma unroll
  for (int x = 0; x < 2; ++x) {
    l[x] += __shfl_xor_sync(0xffffffffu, l[x], 1);
    l[x] += __shfl_xor_sync(0xffffffffu, l[x], 2);
    const int r = g + 8 * x;
    if (t == 0) {
      sm.m[warp][r] = m[x];
      sm.l[warp][r] = l[x];
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
    const int qi = (r0 + r) / a.group, h = hk * a.group + (r0 + r) % a.group;
    if (sm.nan) {  // the row's own tokens of the zone: their NaN values reach its columns
      const int lr = key_limit(ex, a.causal, qi);
      float* yy = &y.x;
      for (int u = max(c0 * kPage, lim_all / 16 * 16); u < min(lr, c1 * kPage); ++u) {
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
// CTA per row, its four warps taking every fourth split; the order of the sums
// is fixed.
template <typename T, int D>
__global__ void __launch_bounds__(128) cache_join_kernel(const CacheAttnArgs a) {
  __shared__ float so[4][D];
  __shared__ float sl[4];
  const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
  const long long row = blockIdx.x;
  const int qi = static_cast<int>(row % a.N);
  const int h = static_cast<int>(row / a.N % a.H), b = static_cast<int>(row / a.N / a.H);
  if (qi >= extent(a, b, false).cnt) return;
  const float2* ml = a.part_ml + row * a.splits;
  float mj = -INFINITY;
  for (int s = lane; s < a.splits; s += 32) mj = fmaxf(mj, ml[s].x);
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) mj = fmaxf(mj, __shfl_xor_sync(0xffffffffu, mj, off));
  constexpr int C = D / 32;
  float y[C], l = 0.f;
#pragma unroll
  for (int e = 0; e < C; ++e) y[e] = 0.f;
#pragma unroll 4
  for (int s = warp; s < a.splits; s += 4) {
    const float2 p = ml[s];
    if (p.x == -INFINITY && p.y == 0.f) continue;  // saw nothing of the row
    const float k = p.x == -INFINITY ? 1.f : ex2_approx(p.x - mj);
    l = fmaf(p.y, k, l);
    const float* o = a.part_o + (row * a.splits + s) * D + lane * C;
#pragma unroll
    for (int e = 0; e < C; ++e) y[e] = fmaf(o[e], k, y[e]);
  }
#pragma unroll
  for (int e = 0; e < C; ++e) so[warp][lane * C + e] = y[e];
  if (lane == 0) sl[warp] = l;
  __syncthreads();
  if (tid < D / 2) {
    const float lj = sl[0] + sl[1] + sl[2] + sl[3];
    const float inv = lj != 0.f ? 1.f / lj : 0.f;
    const int c = 2 * tid;
    const float y0 = so[0][c] + so[1][c] + so[2][c] + so[3][c];
    const float y1 = so[0][c + 1] + so[1][c + 1] + so[2][c + 1] + so[3][c + 1];
    uint16_t* dst = a.out + b * a.ost.b + h * a.ost.h + static_cast<long long>(qi) * a.ost.n + c;
    *reinterpret_cast<uint32_t*>(dst) = pack2<T>(y0 * inv, y1 * inv);
    if (tid == 0 && a.lse) a.lse[row] = lj == 0.f ? -INFINITY : (mj - kPBias + log2f(lj)) * kLn2C;
  }
}

template <typename T>
cudaError_t launch_step_t(const CacheAttnArgs& a, cudaStream_t stream) {
  const int tiles = (a.N * a.group + kRows - 1) / kRows;
  const dim3 grid(a.splits, tiles * a.Hk, a.B);
  if (a.d == 64) cache_step_kernel<T, 64><<<grid, kWarps * 32, 0, stream>>>(a);
  else cache_step_kernel<T, 128><<<grid, kWarps * 32, 0, stream>>>(a);
  return cudaGetLastError();
}

template <typename T>
cudaError_t launch_join_t(const CacheAttnArgs& a, cudaStream_t stream) {
  const unsigned int rows = static_cast<unsigned int>(static_cast<long long>(a.B) * a.H * a.N);
  if (a.d == 64) cache_join_kernel<T, 64><<<rows, 128, 0, stream>>>(a);
  else cache_join_kernel<T, 128><<<rows, 128, 0, stream>>>(a);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_cache_step(const CacheAttnArgs& a, cudaStream_t stream) {
  return a.dtype == kF16 ? launch_step_t<__half>(a, stream) : launch_step_t<__nv_bfloat16>(a, stream);
}

cudaError_t launch_cache_join(const CacheAttnArgs& a, cudaStream_t stream) {
  return a.dtype == kF16 ? launch_join_t<__half>(a, stream) : launch_join_t<__nv_bfloat16>(a, stream);
}

}  // namespace solattn
