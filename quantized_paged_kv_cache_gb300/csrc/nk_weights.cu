// nk_weights.cu -- what each page of a cache is worth to the queries
// (nk_page_weights), and the pages worth least given back (nk_evict_pages).
#include <cuda_fp16.h>
#include <math.h>

#include "nk_common.cuh"
#include "nk_host.cuh"
#include "nk_topk.cuh"

namespace nk {

// ---------------------------------------------------------------------------
// nk_page_weights. The attention weight of a page and kv-head is the sum, over
// the T * G query rows, of exp(s_n - lse) over the page's visible keys n, with
// lse the row's log-sum over all of its keys. Only K is read, and only once: the
// first kernel leaves each (row, page) its own log-sum (one number for P keys)
// and each (row, segment) that of the segment; the second joins the segments to
// the rows' lse and adds up exp(page's - lse).
//
// First kernel: the flat list of (sequence, kv-head, page) items is cut into one
// range a CTA (nk_common.cuh), a warp takes a page of the segment at a time, 16
// keys straight from global memory into registers: a thread's 16 bytes of a row
// are, in the product's K order, four steps of four channels. Codes enter
// mma.m16n8k16 as exact fp16, the query rows as fp16 scaled by a power of two
// each (exact for channels within 2^24 of the row's largest), fp32 sums by
// 64-channel group, then the group's scale. Keys are M and query rows N, so a
// decode step pads six rows to eight. Bounded by the K half of the cache, and by
// mma.sync for the T = 16 of a window over a prompt.
// ---------------------------------------------------------------------------
struct WeightParams {
  const uint8_t* pool;
  ChunkLayout lay;
  int num_pages;
  const uint16_t* q;  // bf16 [B][T][Hq][D]
  const int32_t* bt;
  const int32_t* ctx;
  SplitShape sh;
  int G, rows;        // rows: T * G rounded up to whole tiles of eight
  float scale2;       // sm_scale * log2(e)
  int n_ctas;
  float* page_lse;    // [item][rows], base 2, -inf: no key seen
  float* seg_lse;     // [n_ctas + B * Hkv][rows]
  const float* prior; // may be NULL
  const int32_t* seen;  // may be NULL
  float* out;         // [num_pages][Hkv]
  int32_t* status;
};

constexpr int kWgtThreads = 256, kWgtWarps = kWgtThreads / 32;

__device__ __forceinline__ float wgt_ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ uint32_t wgt_prmt(uint32_t a, uint32_t b, uint32_t sel) {
  uint32_t d;
  asm("prmt.b32 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(sel));
  return d;
}
__device__ __forceinline__ uint32_t wgt_f16(uint32_t biased, uint32_t sel) {
  const uint32_t h = wgt_prmt(biased, 0x64646464u, sel);
  const __half2 r = __hsub2(*reinterpret_cast<const __half2*>(&h),
                            __halves2half2(__ushort_as_half(0x6480), __ushort_as_half(0x6480)));
  return *reinterpret_cast<const uint32_t*>(&r);
}
__device__ __forceinline__ void wgt_mma(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// log-sums (m: largest, l: sum of 2^(s - m); l is 0 while m is -inf)
__device__ __forceinline__ void lse_join(float& m, float& l, float m2, float l2) {
  const float mx = fmaxf(m, m2);
  if (mx == -INFINITY) {
    l += l2;  // nothing, or NaN, which stays
    return;
  }
  l = l * wgt_ex2(m - mx) + l2 * wgt_ex2(m2 - mx);
  m = mx;
}
__device__ __forceinline__ float lse_of(float m, float l) { return l == 0.f ? -INFINITY : m + log2f(l); }

// Shared memory: the unit's rows as fp16 [rows][D / 2 + 2 words], their powers
// of two [rows], then a warp's running log-sums: of the page, a lane its own two
// rows of a tile [rows / 8][32] float4, and of the segment [rows] float2.
__host__ __device__ inline int weight_smem(int D, int rows) {
  return rows * (D * 2 + 8) + rows * 4 + kWgtWarps * (rows / 8 * 32 * 16 + rows * 8);
}

template <int D>
__global__ void __launch_bounds__(kWgtThreads) page_lse_kernel(const WeightParams p) {
  constexpr int RS = D * 2 + 8;
  constexpr int NG = D / kGroup;
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ int pre[kMaxBatch + 1], lens[kMaxBatch], warp_tot[kWgtWarps];
  chain_wait();
  chain_release();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, t4 = lane & 3;
  const SplitShape& sh = p.sh;
  const int P = sh.P, Hkv = sh.Hkv, T = sh.T, G = p.G, M = T * G, rows = p.rows, tiles = rows / 8;
  if (blockIdx.x == 0)
    for (int b = tid; b < sh.B; b += kWgtThreads)
      if (pages_of_len(sh, p.ctx[b]) == 0) flag(p.status, NK_DEVFLAG_BAD_CTX);
  block_page_prefix_short(sh, p.ctx, 0, pre, warp_tot, lens);
  const int64_t W = (int64_t)pre[sh.B] * Hkv;
  if (W == 0) return;
  float4* page_st = reinterpret_cast<float4*>(smem) + warp * tiles * 32;
  uint8_t* rest = smem + kWgtWarps * tiles * 32 * 16;
  float2* seg_st = reinterpret_cast<float2*>(rest);  // [warp][rows]
  rest += kWgtWarps * rows * 8;
  float* undo = reinterpret_cast<float*>(rest);      // sm_scale log2(e) / the row's power of two
  uint8_t* qs = rest + rows * 4;
  int64_t x = cta_begin(W, p.n_ctas, blockIdx.x);
  const int64_t x_end = cta_begin(W, p.n_ctas, blockIdx.x + 1);
  Segment seg;
  int64_t item = x;  // of the segment's first page
  while (next_segment(sh, pre, x, x_end, seg)) {
    const int L = lens[seg.b];
    // ---- the unit's rows: a warp each, scaled into [2^14, 2^15)
    for (int r = warp; r < rows; r += kWgtWarps) {
      const int t = r / G, hg = r - t * G;
      const uint16_t* src = p.q + (((int64_t)seg.b * T + t) * (G * Hkv) + seg.h * G + hg) * D;
      constexpr int PER = D / 64;  // words of a lane
      uint32_t w[PER];
      float m = 0.f;
#pragma unroll
      for (int i = 0; i < PER; ++i) {
        w[i] = r < M ? reinterpret_cast<const uint32_t*>(src)[lane + 32 * i] : 0u;
        m = fmaxf(m, fmaxf(fabsf(bf16_lo(w[i])), fabsf(bf16_hi(w[i]))));
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
      int e = 0;
      if (m > 0.f) {
        e = 14 - ((int)((__float_as_uint(m) >> 23) & 0xffu) - 127);
        e = e > 110 ? 110 : (e < -113 ? -113 : e);
      }
      const float up = __uint_as_float((uint32_t)(127 + e) << 23);
#pragma unroll
      for (int i = 0; i < PER; ++i) {
        const __half2 hh = __floats2half2_rn(bf16_lo(w[i]) * up, bf16_hi(w[i]) * up);
        reinterpret_cast<uint32_t*>(qs + r * RS)[lane + 32 * i] = *reinterpret_cast<const uint32_t*>(&hh);
      }
      if (lane == 0) undo[r] = p.scale2 * __uint_as_float((uint32_t)(127 - e) << 23);
    }
    for (int i = lane; i < rows; i += 32) seg_st[warp * rows + i] = make_float2(-INFINITY, 0.f);
    __syncthreads();
    const int pages = seg.page_end - seg.page_begin;
    for (int pg = warp; pg < pages; pg += kWgtWarps) {  // (warp-uniform)
      const int logical = seg.page_begin + pg;
      const int page = p.bt[(int64_t)seg.b * sh.max_pages + logical];
      const bool bad = page < 0 || page >= p.num_pages;
      if (bad && lane == 0) flag(p.status, NK_DEVFLAG_BAD_PAGE);
      const uint8_t* chunk = p.pool + ((int64_t)(bad ? 0 : page) * Hkv + seg.h) * p.lay.chunk;
      const float* scales = reinterpret_cast<const float*>(chunk + p.lay.ks);
      for (int i = 0; i < tiles; ++i) page_st[i * 32 + lane] = make_float4(-INFINITY, 0.f, -INFINITY, 0.f);
      const int live = bad ? 0 : min(P, L - logical * P);
      for (int k0 = 0; k0 < live; k0 += 16) {
        uint4 raw[2][NG];
        float sc[2][NG];
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int c = 0; c < NG; ++c) {
            const int key = k0 + g + 8 * i;  // (a page holds whole 16s)
            raw[i][c] = *reinterpret_cast<const uint4*>(chunk + (int64_t)key * D + 64 * c + 16 * t4);
            sc[i][c] = scales[key * NG + c];
          }
        uint32_t a[NG][4][4];
#pragma unroll
        for (int c = 0; c < NG; ++c)
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const uint4 r0 = raw[0][c], r1 = raw[1][c];
            const uint32_t w0 = (j == 0 ? r0.x : j == 1 ? r0.y : j == 2 ? r0.z : r0.w) ^ 0x80808080u;
            const uint32_t w1 = (j == 0 ? r1.x : j == 1 ? r1.y : j == 2 ? r1.z : r1.w) ^ 0x80808080u;
            a[c][j][0] = wgt_f16(w0, 0x4140);
            a[c][j][1] = wgt_f16(w1, 0x4140);
            a[c][j][2] = wgt_f16(w0, 0x4342);
            a[c][j][3] = wgt_f16(w1, 0x4342);
          }
        const int pos0 = logical * P + k0;
        const bool edge = pos0 + 15 > L - T;  // some row does not see some key
        for (int nt = 0; nt < tiles; ++nt) {
          float acc[NG][4];
#pragma unroll
          for (int c = 0; c < NG; ++c)
#pragma unroll
            for (int k = 0; k < 4; ++k) acc[c][k] = 0.f;
          const uint8_t* qrow = qs + (nt * 8 + g) * RS + 32 * t4;
#pragma unroll
          for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int c = 0; c < NG; ++c) {
              const uint2 b = *reinterpret_cast<const uint2*>(qrow + 128 * c + 8 * j);
              wgt_mma(acc[c], a[c][j][0], a[c][j][1], a[c][j][2], a[c][j][3], b.x, b.y);
            }
          float s[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int c = 0; c < NG; ++c) {
            s[0] = fmaf(sc[0][c], acc[c][0], s[0]);
            s[1] = fmaf(sc[0][c], acc[c][1], s[1]);
            s[2] = fmaf(sc[1][c], acc[c][2], s[2]);
            s[3] = fmaf(sc[1][c], acc[c][3], s[3]);
          }
          const int r0 = nt * 8 + 2 * t4;
          const float2 un = *reinterpret_cast<const float2*>(undo + r0);
          s[0] *= un.x;
          s[1] *= un.y;
          s[2] *= un.x;
          s[3] *= un.y;
          if (edge) {
            const int p0 = L - T + r0 / G, p1 = L - T + (r0 + 1) / G, n0 = pos0 + g, n1 = n0 + 8;
            if (n0 > p0 || n0 >= L) s[0] = -INFINITY;
            if (n0 > p1 || n0 >= L) s[1] = -INFINITY;
            if (n1 > p0 || n1 >= L) s[2] = -INFINITY;
            if (n1 > p1 || n1 >= L) s[3] = -INFINITY;
          }
          float4 st = page_st[nt * 32 + lane];
          const float m0 = fmaxf(st.x, fmaxf(s[0], s[2])), m1 = fmaxf(st.z, fmaxf(s[1], s[3]));
          const float u0 = m0 == -INFINITY ? 0.f : m0, u1 = m1 == -INFINITY ? 0.f : m1;
          st.y = st.y * wgt_ex2(st.x - u0) + (wgt_ex2(s[0] - u0) + wgt_ex2(s[2] - u0));
          st.w = st.w * wgt_ex2(st.z - u1) + (wgt_ex2(s[1] - u1) + wgt_ex2(s[3] - u1));
          st.x = m0;
          st.z = m1;
          page_st[nt * 32 + lane] = st;
        }
      }
      // ---- the page's log-sums: eight lanes hold a row's keys
      float* dst = p.page_lse + (item + pg) * rows;
      for (int nt = 0; nt < tiles; ++nt) {
        float4 st = page_st[nt * 32 + lane];
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) {
          const float mx = __shfl_xor_sync(0xffffffffu, st.x, o), lx = __shfl_xor_sync(0xffffffffu, st.y, o);
          const float mz = __shfl_xor_sync(0xffffffffu, st.z, o), lz = __shfl_xor_sync(0xffffffffu, st.w, o);
          lse_join(st.x, st.y, mx, lx);
          lse_join(st.z, st.w, mz, lz);
        }
        if (g == 0) {
          const int r0 = nt * 8 + 2 * t4;
          *reinterpret_cast<float2*>(dst + r0) = make_float2(lse_of(st.x, st.y), lse_of(st.z, st.w));
          float2* sg = seg_st + warp * rows + r0;
          float2 s0 = sg[0], s1 = sg[1];
          lse_join(s0.x, s0.y, st.x, st.y);
          lse_join(s1.x, s1.y, st.z, st.w);
          sg[0] = s0;
          sg[1] = s1;
        }
      }
    }
    __syncthreads();
    for (int r = tid; r < rows; r += kWgtThreads) {
      float m = -INFINITY, l = 0.f;
      for (int w = 0; w < kWgtWarps; ++w) {
        const float2 s = seg_st[w * rows + r];
        lse_join(m, l, s.x, s.y);
      }
      p.seg_lse[((int64_t)blockIdx.x + seg.u) * rows + r] = lse_of(m, l);
    }
    item += pages;
    __syncthreads();
  }
}

// Second kernel: block (x, unit) takes pages x * 32 .. of the unit; eight lanes
// a page, a lane every eighth row.
constexpr int kWsmThreads = 256;

__global__ void __launch_bounds__(kWsmThreads) page_weight_kernel(const WeightParams p) {
  __shared__ int pre[kMaxBatch + 1], warp_tot[kWsmThreads / 32];
  extern __shared__ float lse[];  // [rows]
  chain_wait();
  chain_release();
  const SplitShape& sh = p.sh;
  block_page_prefix_short(sh, p.ctx, 0, pre, warp_tot);
  const int64_t W = (int64_t)pre[sh.B] * sh.Hkv;
  const int u = blockIdx.y, b = u / sh.Hkv, h = u - b * sh.Hkv;
  const int pages = pre[b + 1] - pre[b], rows = p.rows, M = sh.T * p.G;
  const int per = kWsmThreads / 8;
  if (W == 0 || (int64_t)blockIdx.x * per >= pages) return;
  const int64_t x0 = (int64_t)pre[b] * sh.Hkv + (int64_t)h * pages;
  const int c0 = cta_of_item(W, p.n_ctas, x0), c1 = cta_of_item(W, p.n_ctas, x0 + pages - 1);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  for (int r = warp; r < rows; r += kWsmThreads / 32) {
    float m = -INFINITY, l = 0.f;
    for (int c = c0 + lane; c <= c1; c += 32) {
      // (a CTA owns no item only when there are fewer items than CTAs)
      if (W < p.n_ctas && cta_begin(W, p.n_ctas, c) == cta_begin(W, p.n_ctas, c + 1)) continue;
      const float s = p.seg_lse[((int64_t)c + u) * rows + r];
      if (s != -INFINITY) lse_join(m, l, s, s == s ? 1.f : s);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      const float m2 = __shfl_xor_sync(0xffffffffu, m, o), l2 = __shfl_xor_sync(0xffffffffu, l, o);
      lse_join(m, l, m2, l2);
    }
    if (lane == 0) lse[r] = lse_of(m, l);
  }
  __syncthreads();
  int seen = 0x7fffffff;
  if (p.seen) seen = p.seen[b];
  for (int64_t j = (int64_t)blockIdx.x * per + tid / 8; j < pages; j += (int64_t)gridDim.x * per) {
    const float* src = p.page_lse + (x0 + j) * rows;
    float sum = 0.f;
    for (int r = tid & 7; r < M; r += 8) {
      const float s = src[r], t = lse[r];
      if (s != -INFINITY) sum += wgt_ex2(s - t);
    }
    const uint32_t mask = 0xffu << (lane & 24);
    sum += __shfl_xor_sync(mask, sum, 1);
    sum += __shfl_xor_sync(mask, sum, 2);
    sum += __shfl_xor_sync(mask, sum, 4);
    if ((tid & 7) == 0) {
      const int page = p.bt[(int64_t)b * sh.max_pages + j];
      if (page >= 0 && page < p.num_pages) {
        const int64_t at = (int64_t)page * sh.Hkv + h;
        if (p.prior && j * sh.P < seen) sum += p.prior[at];
        p.out[at] = sum;
      }
    }
  }
}

// ---------------------------------------------------------------------------
// nk_evict_pages. Of each sequence the `keep` pages with the largest weight,
// summed over its kv-heads, stay (the first `sinks` and last `recent` ones in
// any case; of equal ones the lower page), in their order; the others go to the
// list of freed pages, sequence after sequence. The sums are carried as two fp32
// numbers (48 bits, every step exact): 64-bit floating point is slow here, and a
// single one would put pages of nearly equal weight in another order.
//
// A block each sequence: it forms the prefix of the freed counts from the
// lengths itself, as no count depends on a weight; reads its row of the table
// before it writes one. Bounded by latency.
// ---------------------------------------------------------------------------
struct EvictParams {
  const float* w;  // [num_pages][Hkv]
  int num_pages, Hkv, P;
  const int32_t* table;
  int32_t* out;
  int max_pages;
  const int32_t* ctx;
  int B, keep, sinks, recent;
  int32_t* new_ctx;
  int32_t* freed;
  int max_freed;
  int32_t* num_freed;
  int32_t* status;
};

constexpr int kEvThreads = 512;

// Order of a fp32 that is not NaN, as a whole number.
__device__ __forceinline__ uint32_t ordered32(float x) {
  const uint32_t b = __float_as_uint(x);
  return (b >> 31) ? ~b : b | 0x80000000u;
}

// Shared memory: keys [room] and the row of the table [room].
__global__ void __launch_bounds__(kEvThreads) evict_kernel(const EvictParams p) {
  extern __shared__ uint64_t keys[];
  __shared__ TopSmem<kEvThreads> sm;
  chain_wait();
  chain_release();
  const int tid = threadIdx.x, b = blockIdx.x;
  int32_t* ids = reinterpret_cast<int32_t*>(keys + p.max_pages);
  // freed pages of the sequences before this one (and of all)
  const auto held_of = [&](int i) {
    const int L = p.ctx[i];
    if (L < 0 || (int64_t)L > (int64_t)p.max_pages * p.P) return -1;
    return L == 0 ? 0 : (L - 1) / p.P + 1;
  };
  int64_t before = 0, all = 0;
  for (int i = tid; i < p.B; i += kEvThreads) {
    const int held = held_of(i), gone = held > p.keep ? held - p.keep : 0;
    all += gone;
    if (i < b) before += gone;
  }
  int sum_before, sum_all;
  (void)block_exclusive<kEvThreads>((int)before, sm.warp, sum_before);
  (void)block_exclusive<kEvThreads>((int)all, sm.warp, sum_all);
  const int held = held_of(b);
  if (b == 0 && tid == 0) {
    *p.num_freed = sum_all;
    if (sum_all > p.max_freed) flag(p.status, NK_DEVFLAG_NO_PAGES);
  }
  if (held < 0) {
    if (tid == 0) {
      flag(p.status, NK_DEVFLAG_BAD_CTX);
      p.new_ctx[b] = 0;
    }
    return;
  }
  const int64_t row = (int64_t)b * p.max_pages;
  const int L = p.ctx[b];
  if (held <= p.keep) {
    if (tid == 0) p.new_ctx[b] = L;
    if (p.out != p.table)
      for (int i = tid; i < p.max_pages; i += kEvThreads) p.out[row + i] = p.table[row + i];
    return;
  }
  bool bad = false;
  for (int i = tid; i < held; i += kEvThreads) {
    const int page = p.table[row + i];
    float hi = 0.f, lo = 0.f;
    if (page < 0 || page >= p.num_pages) {
      bad = true;
    } else {
      for (int h = 0; h < p.Hkv; ++h) {
        const float v = fminf(fmaxf(p.w[(int64_t)page * p.Hkv + h], -1e36f), 1e36f);  // (NaN: last)
        // hi + v exactly as a sum and its rounding error, the error joined to lo
        const float s = hi + v, z = s - hi;
        const float err = (hi - (s - z)) + (v - z);
        hi = s;
        lo += err;
      }
      const float s = hi + lo;
      lo = lo - (s - hi);
      hi = s;
    }
    ids[i] = page;
    // (+ 0: a negative zero has the order of a positive one)
    keys[i] = ((uint64_t)ordered32(hi + 0.f) << 32) | ordered32(lo + 0.f);
  }
  if (bad) flag(p.status, NK_DEVFLAG_BAD_PAGE);
  __syncthreads();
  const int n = held - p.sinks - p.recent, need = p.keep - p.sinks - p.recent;  // need < n
  const uint64_t* mid = keys + p.sinks;
  const auto key = [&](int i) { return mid[i]; };
  uint64_t kt = ~0ull;
  int it = -1;
  if (need > 0) {
    uint64_t klo, khi;
    block_range<kEvThreads>(key, n, sm, klo, khi);
    block_threshold<kEvThreads>(key, n, need, klo, khi, sm, kt, it);
  }
  const int per = top_run<kEvThreads>(held), a = tid * per, e = a + per < held ? a + per : held;
  const auto stays = [&](int i) {
    if (i < p.sinks || i >= held - p.recent) return true;
    const uint64_t k = keys[i];
    return k > kt || (k == kt && i - p.sinks <= it);
  };
  int mine = 0, total;
  for (int i = a; i < e; ++i) mine += stays(i);
  int at = block_exclusive<kEvThreads>(mine, sm.warp, total);
  for (int i = a; i < e; ++i) {
    const int page = ids[i];
    if (stays(i)) {
      p.out[row + at++] = page;
    } else {
      const int64_t f = (int64_t)sum_before + (i - at);
      if (f < p.max_freed) p.freed[f] = page >= 0 && page < p.num_pages ? page : -1;
    }
  }
  for (int i = p.keep + tid; i < held; i += kEvThreads) p.out[row + i] = -1;
  if (p.out != p.table)
    for (int i = held + tid; i < p.max_pages; i += kEvThreads) p.out[row + i] = p.table[row + i];
  if (tid == 0) p.new_ctx[b] = L - p.P * (held - p.keep);
}

}  // namespace nk

using namespace nk;

namespace {

int weight_rows(int T, int G) { return (T * G + 7) / 8 * 8; }

int weight_ctas(int64_t items) {
  const int sms = device_sms();
  const int64_t n = (int64_t)(sms > 0 ? sms : 148) * 2;
  return (int)(items < n ? (items < 1 ? 1 : items) : n);
}

}  // namespace

extern "C" {

size_t nk_page_weights_workspace_bytes(int32_t B, int32_t T, int32_t num_q_heads, int32_t num_kv_heads,
                                       int32_t page_size, int32_t max_ctx) {
  if (B < 1 || T < 1 || T > NK_MAX_T || num_kv_heads < 1 || num_q_heads < num_kv_heads || page_size < 1 || max_ctx < 1)
    return 0;
  const int64_t items = (int64_t)B * num_kv_heads * (((int64_t)max_ctx + page_size - 1) / page_size);
  const int64_t slots = weight_ctas(items) + (int64_t)B * num_kv_heads;
  return (size_t)(items + slots) * weight_rows(T, num_q_heads / num_kv_heads) * 4;
}

int nk_page_weights(const nk_kv_pool* pool, const void* q_dev, const int32_t* block_table_dev,
                    int32_t max_pages_per_seq, const int32_t* ctx_lens_dev, int32_t B, int32_t T, int32_t num_q_heads,
                    float sm_scale, int32_t max_ctx, const float* prior_dev, const int32_t* seen_dev,
                    void* workspace_dev, size_t workspace_bytes, float* weights_dev, int32_t* status_dev,
                    void* stream) {
  const int err = check_pool(pool);
  if (err != NK_OK) return err;
  if (B < 0 || T < 1 || T > NK_MAX_T || num_q_heads < 1 || num_q_heads % pool->num_kv_heads != 0) return NK_ERR_SHAPE;
  if (B == 0) return NK_OK;
  if (!q_dev || !block_table_dev || !ctx_lens_dev || !weights_dev) return NK_ERR_NULL;
  const int Hkv = pool->num_kv_heads, D = pool->head_dim, P = pool->page_size, G = num_q_heads / Hkv;
  if (max_pages_per_seq < 1 || max_ctx < T || (int64_t)max_ctx > (int64_t)max_pages_per_seq * P) return NK_ERR_SHAPE;
  if (!isfinite(sm_scale) || !aligned_to(q_dev, 16)) return NK_ERR_SHAPE;
  const int rows = weight_rows(T, G), smem = weight_smem(D, rows);
  if (B > kMaxBatch || (int64_t)B * Hkv > 65535 || smem > 200 * 1024) return NK_ERR_UNSUPPORTED;
  const size_t need = nk_page_weights_workspace_bytes(B, T, num_q_heads, Hkv, P, max_ctx);
  if (!workspace_dev || workspace_bytes < need || !aligned_to(workspace_dev, 16)) return NK_ERR_WORKSPACE;
  const int64_t longest = ((int64_t)max_ctx + P - 1) / P, items = (int64_t)B * Hkv * longest;
  WeightParams p = {};
  p.pool = reinterpret_cast<const uint8_t*>(pool->base_dev);
  p.lay = ChunkLayout::make(P, D);
  p.num_pages = pool->num_pages;
  p.q = reinterpret_cast<const uint16_t*>(q_dev);
  p.bt = block_table_dev;
  p.ctx = ctx_lens_dev;
  p.sh = SplitShape{B, Hkv, P, T, max_ctx, max_pages_per_seq};
  p.G = G;
  p.rows = rows;
  p.scale2 = sm_scale * kLog2e;
  p.n_ctas = weight_ctas(items);
  p.page_lse = reinterpret_cast<float*>(workspace_dev);
  p.seg_lse = p.page_lse + items * rows;
  p.prior = prior_dev;
  p.seen = seen_dev;
  p.out = weights_dev;
  p.status = status_dev;
  const cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  const dim3 g((unsigned)p.n_ctas), t(kWgtThreads);
  const void* fn = D == 256   ? reinterpret_cast<const void*>(page_lse_kernel<256>)
                   : D == 128 ? reinterpret_cast<const void*>(page_lse_kernel<128>)
                              : reinterpret_cast<const void*>(page_lse_kernel<64>);
  cudaError_t e = set_smem_limit(fn, smem);
  if (e != cudaSuccess) return NK_ERR_CUDA;
  e = D == 256   ? launch_chained(page_lse_kernel<256>, g, t, (size_t)smem, st, p)
      : D == 128 ? launch_chained(page_lse_kernel<128>, g, t, (size_t)smem, st, p)
                 : launch_chained(page_lse_kernel<64>, g, t, (size_t)smem, st, p);
  if (e != cudaSuccess) return NK_ERR_CUDA;
  const int64_t units = (int64_t)B * Hkv;
  int64_t gx = (longest + kWsmThreads / 8 - 1) / (kWsmThreads / 8), most = 2048 / units;
  if (most < 1) most = 1;
  if (gx > most) gx = most;
  e = launch_chained(page_weight_kernel, dim3((unsigned)gx, (unsigned)units), dim3(kWsmThreads), (size_t)rows * 4, st,
                     p);
  return e == cudaSuccess ? NK_OK : NK_ERR_CUDA;
}

int nk_evict_pages(int32_t page_size, int32_t num_pages, int32_t num_kv_heads, const float* weights_dev,
                   const int32_t* block_table_dev, int32_t* out_table_dev, int32_t max_pages_per_seq,
                   const int32_t* ctx_lens_dev, int32_t B, int32_t keep_pages, int32_t sink_pages,
                   int32_t recent_pages, int32_t* new_ctx_dev, int32_t* freed_dev, int32_t max_freed,
                   int32_t* num_freed_dev, int32_t* status_dev, void* stream) {
  if (page_size < 1 || num_pages < 1 || num_kv_heads < 1 || B < 0 || max_pages_per_seq < 1 || max_freed < 0)
    return NK_ERR_SHAPE;
  if (sink_pages < 0 || recent_pages < 1 || (int64_t)sink_pages + recent_pages > keep_pages) return NK_ERR_SHAPE;
  // a row of the table and its keys stay in shared memory
  if (B > kMaxBatch || max_pages_per_seq > 16384) return NK_ERR_UNSUPPORTED;
  if (B == 0) return NK_OK;
  if (!weights_dev || !block_table_dev || !out_table_dev || !ctx_lens_dev || !new_ctx_dev || !num_freed_dev ||
      (max_freed > 0 && !freed_dev))
    return NK_ERR_NULL;
  if (new_ctx_dev == ctx_lens_dev) return NK_ERR_SHAPE;  // every block reads the lengths while others write theirs
  const EvictParams p{weights_dev, num_pages, num_kv_heads, page_size, block_table_dev, out_table_dev,
                      max_pages_per_seq, ctx_lens_dev, B, keep_pages, sink_pages, recent_pages, new_ctx_dev, freed_dev,
                      max_freed, num_freed_dev, status_dev};
  const int smem = (max_pages_per_seq + 1) / 2 * 2 * 12;
  cudaError_t e = set_smem_limit(reinterpret_cast<const void*>(evict_kernel), smem);
  if (e != cudaSuccess) return NK_ERR_CUDA;
  e = launch_chained(evict_kernel, dim3((unsigned)B), dim3(kEvThreads), (size_t)smem, reinterpret_cast<cudaStream_t>(stream),
                     p);
  return e == cudaSuccess ? NK_OK : NK_ERR_CUDA;
}

}  // extern "C"
