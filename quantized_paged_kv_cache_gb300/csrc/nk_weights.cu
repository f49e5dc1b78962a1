// nk_weights.cu -- what each page of a cache is worth to the queries
// (nk_page_weights), and the pages worth least given back (nk_evict_pages).
#include <cuda_fp16.h>
#include <math.h>

#include "nk_common.cuh"
#include "nk_host.cuh"
#include "nk_ptx.cuh"
#include "nk_topk.cuh"
#include "nk_weights.cuh"

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
// range a CTA (nk_common.cuh), a warp takes a page of the segment at a time, KB
// times 16 keys a step, from a ring of its own in shared memory that bulk
// asynchronous copies fill; no warp waits for another. A thread reads 16
// consecutive channels of a key, in the product's K order four steps of four.
// Codes enter mma.m16n8k16 as exact fp16, the query rows as fp16 scaled by a power
// of two each (exact for channels within 2^24 of the row's largest), fp32 sums by
// 64-channel group, then the group's scale. Keys are M and query rows N, so a
// decode step pads six rows to eight (one tile, whose rows stay in registers); more
// than 48 rows go to the tcgen05 kernel (nk_weights_tc.cu). Bounded by the K half
// of the cache (8 sequences, 274K tokens, 24 heads over 4 of 256: 65 us with the
// second kernel, 4.6 TB/s) and, for several tiles of rows, by instructions (T = 4
// 94 us, T = 8 149). Copies of 16 bytes a lane, which fill the queue of the memory
// instructions, took 79, 116 and 174.
// ---------------------------------------------------------------------------
constexpr int kWgtThreads = 256, kWgtWarps = kWgtThreads / 32;

// A step of a warp in its ring: KB times 16 keys' codes, then their scales.
template <int D, int KB>
struct KeyStep {
  static constexpr int NG = D / kGroup;
  static constexpr int kCodes = KB * 16 * D;
  static constexpr int kBytes = kCodes + KB * 16 * NG * 4;
};

// Shared memory: each warp's running log-sums of the segment [rows] float2, the
// rows' powers of two [rows], the rows as fp16 [rows][D / 2 + 2 words],
// the rings, the
// page prefix and the lengths [2 B + 1].
__host__ __device__ inline int weight_ring_off(int D, int chunk) {
  return (kWgtWarps * chunk * 8 + chunk * 4 + chunk * (D * 2 + 8) + 15) / 16 * 16;
}
// Steps in a warp's ring: three where 227 KB hold them. One tile of rows takes
// steps of 16 keys and two CTAs an SM: their chains of waits cover each other, and
// the kernels before and behind find room beside one that ends.
template <int D, int NT, int KB>
constexpr int weight_stages() {
  return (kWgtWarps * (NT * 64 + 3 * KeyStep<D, KB>::kBytes) + NT * 32 + NT * 8 * (D * 2 + 8) + 16 +
          (2 * kMaxBatch + 32) * 4 + kWgtWarps * 3 * 8 <= 227 * 1024)
             ? 3
             : 2;
}
constexpr int lse_ctas(int NT) { return NT == 1 ? 2 : 1; }  // of an SM

template <int D, int NT, int KB>
__global__ void __launch_bounds__(kWgtThreads, lse_ctas(NT)) page_lse_kernel(const WeightParams p) {
  constexpr int kWarps = kWgtWarps, kThreads = kWgtThreads;
  constexpr int RS = D * 2 + 8;
  constexpr int NG = D / kGroup;
  constexpr int ROWS = NT * 8;
  constexpr int S = weight_stages<D, NT, KB>();
  using Step = KeyStep<D, KB>;
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ int warp_tot[kWarps];
  __shared__ uint64_t bars[kWarps][S];
  if (threadIdx.x < kWarps * S) {
    mbar_init(smem_u32(&bars[0][0] + threadIdx.x), 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  chain_wait();
  chain_release();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, t4 = lane & 3;
  const SplitShape& sh = p.sh;
  const int P = sh.P, Hkv = sh.Hkv, T = sh.T, G = p.G, M = T * G;
  int* pre = reinterpret_cast<int*>(smem + weight_ring_off(D, ROWS) + kWarps * S * Step::kBytes);  // [B + 1]
  int* lens = pre + sh.B + 1;                                                                     // [B]
  if (blockIdx.x == 0)
    for (int b = tid; b < sh.B; b += kThreads)
      if (pages_of_len(sh, p.ctx[b]) == 0) flag(p.status, NK_DEVFLAG_BAD_CTX);
  block_page_prefix_short(sh, p.ctx, 0, pre, warp_tot, lens);
  const int64_t W = (int64_t)pre[sh.B] * Hkv;
  if (W == 0) return;
  float2* seg_st = reinterpret_cast<float2*>(smem) + warp * ROWS;
  float* undo = reinterpret_cast<float*>(smem + kWarps * ROWS * 8);  // sm_scale log2(e) / the row's power of two
  uint8_t* qs = reinterpret_cast<uint8_t*>(undo + ROWS);
  uint8_t* ring = smem + weight_ring_off(D, ROWS) + warp * S * Step::kBytes;
  const uint32_t ring_u32 = smem_u32(ring), bar0 = smem_u32(bars[warp]);
  int64_t x = cta_begin(W, p.n_ctas, blockIdx.x);
  const int64_t x_end = cta_begin(W, p.n_ctas, blockIdx.x + 1);
  Segment seg;
  int64_t item = x;  // of the segment's first page
  int issued = 0, used = 0, sent = 0;  // steps; one past the last that was copied
  bool timed_out = false;
  while (next_segment(sh, pre, x, x_end, seg)) {
    const int L = lens[seg.b], pages = seg.page_end - seg.page_begin;
    const int32_t* row_bt = p.bt + (int64_t)seg.b * sh.max_pages + seg.page_begin;
    const auto live_of = [&](int pg) { return min(P, L - (seg.page_begin + pg) * P); };
    // ---- the copies: page and step of the next one, its page id, the one after's
    int c_pg = warp, c_k = 0;
    uint32_t none = 0;  // steps in flight whose page is none: a bit each, by their number in the CTA
    int id = c_pg < pages ? row_bt[c_pg] : 0, id_next = c_pg + kWarps < pages ? row_bt[c_pg + kWarps] : 0;
    const auto issue = [&]() {  // (warp-uniform)
      if (c_pg >= pages) return;
      const int live = live_of(c_pg), slot = issued % S, keys = min(16 * KB, (live - c_k + 15) / 16 * 16);
      const bool bad = id < 0 || id >= p.num_pages;
      const uint32_t bit = 1u << (issued & 31);
      none = bad ? none | bit : none & ~bit;
      if (lane == 0) {
        const uint32_t dst = ring_u32 + slot * Step::kBytes, bar = bar0 + 8 * slot;
        if (bad) {
          mbar_arrive(bar);
        } else if (!timed_out && !(p.withhold >= 0 && issued >= p.withhold)) {
          const uint8_t* chunk = p.pool + ((int64_t)id * Hkv + seg.h) * p.lay.chunk;
          mbar_arrive_expect_tx(bar, keys * (D + NG * 4));
          bulk_load(dst, chunk + c_k * D, keys * D, bar);
          bulk_load(dst + Step::kCodes, chunk + p.lay.ks + c_k * (NG * 4), keys * (NG * 4), bar);
        }
      }
      if (!timed_out && !(p.withhold >= 0 && issued >= p.withhold)) sent = issued + 1;
      ++issued;
      c_k += 16 * KB;
      if (c_k >= live) {
        c_k = 0;
        c_pg += kWarps;
        id = id_next;
        if (c_pg + kWarps < pages) id_next = row_bt[c_pg + kWarps];
      }
    };
#pragma unroll
    for (int i = 0; i < S - 1; ++i) issue();
    // ---- the unit's rows: a warp each, scaled into [2^14, 2^15)
    for (int r = warp; r < ROWS; r += kWarps) {
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
      const int e = wgt_row_exp(m);
      const float up = wgt_row_factor(m, e);
#pragma unroll
      for (int i = 0; i < PER; ++i) {
        const __half2 hh = __floats2half2_rn(bf16_lo(w[i]) * up, bf16_hi(w[i]) * up);
        reinterpret_cast<uint32_t*>(qs + r * RS)[lane + 32 * i] = *reinterpret_cast<const uint32_t*>(&hh);
      }
      if (lane == 0) undo[r] = p.scale2 * wgt_pow2(-e);
    }
    for (int i = lane; i < ROWS; i += 32) seg_st[i] = make_float2(-INFINITY, 0.f);
    __syncthreads();
    uint2 bq[NT == 1 ? NG : 1][4];  // one tile: the rows as the products take them
    if constexpr (NT == 1) {
#pragma unroll
      for (int c = 0; c < NG; ++c)
#pragma unroll
        for (int j = 0; j < 4; ++j) bq[c][j] = *reinterpret_cast<const uint2*>(qs + g * RS + 32 * t4 + 128 * c + 8 * j);
    }
    for (int pg = warp; pg < pages; pg += kWarps) {  // (warp-uniform)
      const int logical = seg.page_begin + pg, live = live_of(pg);
      float m[NT][2], l[NT][2];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          m[nt][e] = -INFINITY;
          l[nt][e] = 0.f;
        }
      for (int k0 = 0; k0 < live; k0 += 16 * KB) {
        issue();
        const int slot = used % S;
        // (after a wait of the warp has run out it copies nothing more and waits for nothing but, at the end, its copies)
        if (!timed_out && !mbar_wait(bar0 + 8 * slot, (uint32_t)(used / S) & 1u, p.wait_cycles)) {
          flag(p.status, NK_DEVFLAG_TIMEOUT);
          timed_out = true;
        }
        timed_out = __any_sync(0xffffffffu, timed_out);
        const bool bad = (none >> (used & 31)) & 1u;
        ++used;
        if (bad && lane == 0) flag(p.status, NK_DEVFLAG_BAD_PAGE);
        const uint8_t* step = ring + slot * Step::kBytes;
        const int pos0 = logical * P + k0;
        const bool edge = bad || k0 + 16 * KB > live || pos0 + 16 * KB - 1 > L - T;  // some row does not see some key
        float s[NT][KB][4];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int kb = 0; kb < KB; ++kb)
#pragma unroll
            for (int k = 0; k < 4; ++k) s[nt][kb][k] = 0.f;
        float sc[KB][2][NG];  // the scales of keys g and g + 8
#pragma unroll
        for (int kb = 0; kb < KB; ++kb)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const float* f = reinterpret_cast<const float*>(step + Step::kCodes) + (kb * 16 + g + 8 * i) * NG;
            if constexpr (NG == 4) {
              const float4 v = *reinterpret_cast<const float4*>(f);
              sc[kb][i][0] = v.x, sc[kb][i][1] = v.y, sc[kb][i][2] = v.z, sc[kb][i][3] = v.w;
            } else if constexpr (NG == 2) {
              const float2 v = *reinterpret_cast<const float2*>(f);
              sc[kb][i][0] = v.x, sc[kb][i][1] = v.y;
            } else {
              sc[kb][i][0] = *f;
            }
          }
#pragma unroll
        for (int c = 0; c < NG; ++c) {
          uint32_t a[KB][4][4];
#pragma unroll
          for (int kb = 0; kb < KB; ++kb) {
            const uint8_t* src = step + (kb * 16 + g) * D + 64 * c + 16 * t4;
            const uint4 r0 = *reinterpret_cast<const uint4*>(src), r1 = *reinterpret_cast<const uint4*>(src + 8 * D);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const uint32_t w0 = (j == 0 ? r0.x : j == 1 ? r0.y : j == 2 ? r0.z : r0.w) ^ 0x80808080u;
              const uint32_t w1 = (j == 0 ? r1.x : j == 1 ? r1.y : j == 2 ? r1.z : r1.w) ^ 0x80808080u;
              a[kb][j][0] = wgt_f16(w0, 0x4140);
              a[kb][j][1] = wgt_f16(w1, 0x4140);
              a[kb][j][2] = wgt_f16(w0, 0x4342);
              a[kb][j][3] = wgt_f16(w1, 0x4342);
            }
          }
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            float acc[KB][4];
#pragma unroll
            for (int kb = 0; kb < KB; ++kb)
#pragma unroll
              for (int k = 0; k < 4; ++k) acc[kb][k] = 0.f;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              uint2 b;
              if constexpr (NT == 1) b = bq[c][j];
              else b = *reinterpret_cast<const uint2*>(qs + (nt * 8 + g) * RS + 32 * t4 + 128 * c + 8 * j);
#pragma unroll
              for (int kb = 0; kb < KB; ++kb)
                wgt_mma(acc[kb], a[kb][j][0], a[kb][j][1], a[kb][j][2], a[kb][j][3], b.x, b.y);
            }
#pragma unroll
            for (int kb = 0; kb < KB; ++kb) {
              s[nt][kb][0] = fmaf(sc[kb][0][c], acc[kb][0], s[nt][kb][0]);
              s[nt][kb][1] = fmaf(sc[kb][0][c], acc[kb][1], s[nt][kb][1]);
              s[nt][kb][2] = fmaf(sc[kb][1][c], acc[kb][2], s[nt][kb][2]);
              s[nt][kb][3] = fmaf(sc[kb][1][c], acc[kb][3], s[nt][kb][3]);
            }
          }
        }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          const int r0 = nt * 8 + 2 * t4;
          const float2 un = *reinterpret_cast<const float2*>(undo + r0);
#pragma unroll
          for (int kb = 0; kb < KB; ++kb) {
            s[nt][kb][0] *= un.x;
            s[nt][kb][1] *= un.y;
            s[nt][kb][2] *= un.x;
            s[nt][kb][3] *= un.y;
          }
          if (edge) {
            // the last position each row sees; keys past the page's live ones are another page's
            const int end = bad ? -1 : logical * P + live - 1;
            const int p0 = min(L - T + r0 / G, end), p1 = min(L - T + (r0 + 1) / G, end);
#pragma unroll
            for (int kb = 0; kb < KB; ++kb) {
              const int n0 = pos0 + 16 * kb + g, n1 = n0 + 8;
              if (n0 > p0) s[nt][kb][0] = -INFINITY;
              if (n0 > p1) s[nt][kb][1] = -INFINITY;
              if (n1 > p0) s[nt][kb][2] = -INFINITY;
              if (n1 > p1) s[nt][kb][3] = -INFINITY;
            }
          }
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float mx = m[nt][e];
#pragma unroll
            for (int kb = 0; kb < KB; ++kb) mx = fmaxf(mx, fmaxf(s[nt][kb][e], s[nt][kb][e + 2]));
            const float u = mx == -INFINITY ? 0.f : mx;
            float sum = 0.f;
#pragma unroll
            for (int kb = 0; kb < KB; ++kb) sum += wgt_ex2(s[nt][kb][e] - u) + wgt_ex2(s[nt][kb][e + 2] - u);
            l[nt][e] = fmaf(l[nt][e], wgt_ex2(m[nt][e] - u), sum);
            m[nt][e] = mx;
          }
        }
        __syncwarp();  // (the next copies go where this step lay S steps ago)
      }
      // ---- the page's log-sums: eight lanes hold a row's keys
      float* dst = p.page_lse + (item + pg) * ROWS;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
        for (int e = 0; e < 2; ++e)
#pragma unroll
          for (int o = 4; o < 32; o <<= 1) {
            const float m2 = __shfl_xor_sync(0xffffffffu, m[nt][e], o), l2 = __shfl_xor_sync(0xffffffffu, l[nt][e], o);
            lse_join(m[nt][e], l[nt][e], m2, l2);
          }
        if (g == 0) {
          const int r0 = nt * 8 + 2 * t4;
          *reinterpret_cast<float2*>(dst + r0) = make_float2(lse_of(m[nt][0], l[nt][0]), lse_of(m[nt][1], l[nt][1]));
          float2 s0 = seg_st[r0], s1 = seg_st[r0 + 1];
          lse_join(s0.x, s0.y, m[nt][0], l[nt][0]);
          lse_join(s1.x, s1.y, m[nt][1], l[nt][1]);
          seg_st[r0] = s0;
          seg_st[r0 + 1] = s1;
        }
      }
    }
    __syncthreads();
    const float2* all = reinterpret_cast<const float2*>(smem);
    for (int r = tid; r < ROWS; r += kThreads) {
      float m = -INFINITY, l = 0.f;
      for (int w = 0; w < kWarps; ++w) lse_join(m, l, all[w * ROWS + r].x, all[w * ROWS + r].y);
      p.seg_lse[((int64_t)blockIdx.x + seg.u) * ROWS + r] = lse_of(m, l);
    }
    item += pages;
    __syncthreads();
  }
  if (timed_out)
    for (int i = max(0, sent - S); i < sent; ++i) (void)mbar_wait(bar0 + 8 * (i % S), (uint32_t)(i / S) & 1u, p.wait_cycles);
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
  const int tid = threadIdx.x, lane = tid & 31;
  // `sub` lanes a row (a power of two, at most a warp), as many rows at once as fit
  int sub = 32;
  while (sub > 1 && rows * sub > kWsmThreads) sub >>= 1;
  for (int r0 = 0; r0 < rows; r0 += kWsmThreads / sub) {  // (every thread: the shuffles below)
    const int r = min(r0 + tid / sub, rows - 1);
    float m = -INFINITY, l = 0.f;
#pragma unroll 4
    for (int c = c0 + (tid & (sub - 1)); c <= c1; c += sub) {
      // (a CTA owns no item only when there are fewer items than CTAs)
      if (W < p.n_ctas && cta_begin(W, p.n_ctas, c) == cta_begin(W, p.n_ctas, c + 1)) continue;
      for (int k = 0; k < p.takes; ++k) {
        const float s = p.seg_lse[(((int64_t)c + u) * p.takes + k) * rows + r];
        if (s != -INFINITY) lse_join(m, l, s, s == s ? 1.f : s);
      }
    }
    for (int o = sub >> 1; o > 0; o >>= 1) {
      const float m2 = __shfl_xor_sync(0xffffffffu, m, o), l2 = __shfl_xor_sync(0xffffffffu, l, o);
      lse_join(m, l, m2, l2);
    }
    if ((tid & (sub - 1)) == 0) {
      // a row that sees no key (its pages are none) draws nothing: 2^(s - inf) is 0 also where s is -inf
      const float all = lse_of(m, l);
      lse[r] = all == -INFINITY ? INFINITY : all;
    }
  }
  __syncthreads();
  int seen = 0x7fffffff;
  if (p.seen) seen = p.seen[b];
  for (int64_t j = (int64_t)blockIdx.x * per + tid / 8; j < pages; j += (int64_t)gridDim.x * per) {
    const float* src = p.page_lse + (x0 + j) * p.parts * rows;
    float sum = 0.f;
    for (int k = 0; k < p.parts; ++k, src += rows)
#pragma unroll 4
      for (int r = tid & 7; r < M; r += 8) sum += wgt_ex2(src[r] - lse[r]);  // (no key seen: 2^-inf is 0)
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
// list of freed pages, sequence after sequence. A page's weights are summed as whole
// multiples of 2^(e + c - 61), with 2^e the largest power of two in them and 2^c the
// least that Hkv does not pass: the same sum in any order of the heads, which no
// floating-point sum is (64-bit ones are slow here besides), cut to 55 significant
// bits for its key. A sum as two fp32 numbers took 9.5 us where this takes 9.8, and
// let equal sums differ.
//
// A block each sequence: it forms the prefix of the freed counts from the
// lengths itself, as no count depends on a weight; reads its row of the table
// before it writes one. Bounded by latency (8 sequences of up to 2,048 pages 9.8 us,
// 512 of up to 1,250 pages 14.1).
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
constexpr int kEvPages = 16384;  // of a row of the table, at most: 12 bytes of shared memory each

// A weight (the bits of a fp32 that is not NaN) in units of 2^(shift - 188), cut off
// below; `shift` is top + c, with `top` at least the weight's exponent field. Its 24
// bits stand at bit 38 and move right. Infinity is 2^128.
__device__ __forceinline__ uint32_t ev_shr(uint32_t x, uint32_t s) {  // (0 past 31)
  uint32_t y;
  asm("shr.u32 %0, %1, %2;" : "=r"(y) : "r"(x), "r"(s));
  return y;
}
__device__ __forceinline__ int64_t weight_units(uint32_t bits, uint32_t shift) {
  const uint32_t e = (bits >> 23) & 0xffu, s = shift - max(e, 1u);
  const uint32_t m = ((bits << 6) & 0x1fffffc0u) | min(e, 1u) << 29;
  const uint32_t hi = ev_shr(m, s), lo = ev_shr(__funnelshift_rc(0u, m, s), max(s, 32u) - 32u);
  const int64_t x = (int64_t)((uint64_t)hi << 32 | lo);
  return (int32_t)bits < 0 ? -x : x;
}
// Order of a sum of such units (below 2^63) as a whole number: sign, nine bits of
// exponent, 54 bits behind the leading one. 0, below all of them, is a page's with a NaN.
__device__ __forceinline__ uint64_t sum_key(int64_t sum, int top) {
  constexpr uint64_t kSign = 1ull << 63;
  if (sum == 0) return kSign;
  const uint64_t size = (uint64_t)(sum < 0 ? -sum : sum);
  const int n = 63 - __clzll((long long)size);
  const uint64_t k = (uint64_t)(top + n) << 54 | ((size << (63 - n)) << 1) >> 10;
  return sum < 0 ? ~(k | kSign) : k | kSign;
}

// Shared memory: keys [room] and the row of the table [room]. W: weights of a page that
// one load takes. MANY: three blocks an SM with two pages of a thread in flight, in place of
// two with four.
template <int W, bool MANY>
__global__ void __launch_bounds__(kEvThreads, MANY ? 3 : 2) evict_kernel(const EvictParams p) {
  extern __shared__ uint64_t keys[];
  __shared__ TopSmem<kEvThreads> sm;
  __shared__ int before_s[kEvThreads / 32], all_s[kEvThreads / 32];
  chain_wait();
  chain_release();
  const int tid = threadIdx.x, b = blockIdx.x;
  if (p.B == 0) {  // nothing goes
    if (tid == 0) *p.num_freed = 0;
    return;
  }
  int32_t* ids = reinterpret_cast<int32_t*>(keys + p.max_pages);
  // freed pages of the sequences before this one (and of all)
  const auto held_of = [&](int i) {
    const int L = p.ctx[i];
    if (L < 0 || (int64_t)L > (int64_t)p.max_pages * p.P) return -1;
    return L == 0 ? 0 : (L - 1) / p.P + 1;
  };
  // (a warp's sums; whoever needs them adds those up behind a later barrier)
  int before = 0, all = 0;
  for (int i = tid; i < p.B; i += kEvThreads) {
    const int h = held_of(i), gone = h > p.keep ? h - p.keep : 0;
    all += gone;
    if (i < b) before += gone;
  }
  before = __reduce_add_sync(0xffffffffu, before);
  all = __reduce_add_sync(0xffffffffu, all);
  if ((tid & 31) == 0) {
    before_s[tid >> 5] = before;
    all_s[tid >> 5] = all;
  }
  const int held = held_of(b);
  if (b == 0) {  // (block-uniform)
    __syncthreads();
    if (tid == 0) {
      int sum = 0;
      for (int w = 0; w < kEvThreads / 32; ++w) sum += all_s[w];
      *p.num_freed = sum;
      if (sum > p.max_freed) flag(p.status, NK_DEVFLAG_NO_PAGES);
    }
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
  // pages of a thread in flight: their ids, then a head's weights of all of them
  constexpr int U = MANY ? 2 : 4;
  bool bad = false;
  uint64_t klo = ~0ull, khi = 0;
  const int last = held - p.recent;  // one past the last page in question
  const int heads_log2 = 32 - __clz(p.Hkv - 1);  // Hkv weights stay below 2^62 units
  for (int i0 = tid; i0 < held; i0 += kEvThreads * U) {
    int page[U], top[U];
    int64_t sum[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int i = i0 + u * kEvThreads;
      page[u] = i < held ? p.table[row + i] : 0;
      sum[u] = 0;
    }
    // the largest weight without its sign (past infinity: a NaN), then the sum in units
    // below it, W heads at a time (more are read once more, from L1)
    uint32_t v[U][W], most[U] = {};
    const auto fetch = [&](int h0) {
#pragma unroll
      for (int u = 0; u < U; ++u) {
#pragma unroll
        for (int j = 0; j < W; ++j) v[u][j] = 0;
        if (page[u] < 0 || page[u] >= p.num_pages) continue;
        const float* src = p.w + (int64_t)page[u] * p.Hkv + h0;
        if constexpr (W == 4) {
          const uint4 x = *reinterpret_cast<const uint4*>(src);
          v[u][0] = x.x, v[u][1] = x.y, v[u][2] = x.z, v[u][3] = x.w;
        } else if constexpr (W == 2) {
          const uint2 x = *reinterpret_cast<const uint2*>(src);
          v[u][0] = x.x, v[u][1] = x.y;
        } else {
          v[u][0] = __float_as_uint(*src);
        }
      }
    };
    for (int h0 = 0; h0 < p.Hkv; h0 += W) {
      fetch(h0);
#pragma unroll
      for (int u = 0; u < U; ++u)
#pragma unroll
        for (int j = 0; j < W; ++j) most[u] = max(most[u], v[u][j] & 0x7fffffffu);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) top[u] = max((int)(most[u] >> 23), 1);
    for (int h0 = 0; h0 < p.Hkv; h0 += W) {
      if (p.Hkv > W) fetch(h0);
#pragma unroll
      for (int u = 0; u < U; ++u)
#pragma unroll
        for (int j = 0; j < W; ++j) sum[u] += weight_units(v[u][j], (uint32_t)(top[u] + heads_log2));
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int i = i0 + u * kEvThreads;
      if (i >= held) continue;
      bad |= page[u] < 0 || page[u] >= p.num_pages;
      const uint64_t k = most[u] > 0x7f800000u ? 0 : sum_key(sum[u], top[u]);
      ids[i] = page[u];
      keys[i] = k;
      if (i >= p.sinks && i < last) {
        klo = k < klo ? k : klo;
        khi = k > khi ? k : khi;
      }
    }
  }
  if (bad) flag(p.status, NK_DEVFLAG_BAD_PAGE);
  top_range(klo, khi, sm);
  __syncthreads();
  int sum_before = 0;
#pragma unroll
  for (int w = 0; w < kEvThreads / 32; ++w) sum_before += before_s[w];
  const int n = last - p.sinks, need = p.keep - p.sinks - p.recent;  // need < n
  const uint64_t* mid = keys + p.sinks;
  const auto key = [&](int i) { return mid[i]; };
  uint64_t kt = ~0ull;
  int it = -1;
  if (need > 0) {
    range_of(klo, khi, sm);
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

// From how many rows on the tcgen05 kernel takes a call: past one chunk of the
// mma.sync kernel, which would read the keys once more for each. Both kernels, 8
// sequences of 13K to 64K over 4 kv-heads, us on mma.sync / on tcgen05:
//   rows          16           32          48       56
//   head dim  64  62.8/114.2   71.0/115.3   93.1/119.6   -/120.5
//            128  60.0/129.4   86.6/131.4  112.3/138.2   -/139.7
//            256  76.4/175.1  112.1/177.1  151.9/183.9   -/185.6
constexpr int kTcRows = 49;

// Row tiles of the mma.sync kernel's instances: 1, 2, 3, 4, 6; with 16-key pages
// (steps of 16 keys) 1, 3, 6.
int weight_tiles(int tiles, int P) {
  if (P == 16) return tiles <= 1 ? 1 : (tiles <= 3 ? 3 : 6);
  return tiles == 5 ? 6 : tiles;
}

// Rows of a unit: up to 48 in one chunk on mma.sync (six tiles of eight fill a
// thread's registers), chunks of up to 128, alike in size, on tcgen05 (the M of its
// product).
struct WeightRows {
  bool tc;
  int chunks, chunk;  // rows of a chunk, a multiple of eight
  int parts, takes;
  int all() const { return chunks * chunk; }
};
WeightRows weight_rows(int T, int G, int P) {
  const int M = T * G;
  const bool tc = M >= kTcRows;
  if (!tc) return {false, 1, weight_tiles((M + 7) / 8, P) * 8, 1, 1};
  const int n = (M + 127) / 128, tiles = ((M + n - 1) / n + 7) / 8;
  return {true, n, tiles * 8, (P + 31) / 32, 4};
}

// CTAs along the pages: as many as an SM holds, shared by the chunks.
int weight_ctas(int64_t items, const WeightRows& r) {
  const int sms = device_sms();
  int64_t n = (int64_t)(sms > 0 ? sms : 148) * (r.tc ? 1 : lse_ctas(r.chunk / 8)) / r.chunks;
  if (n < 1) n = 1;
  return (int)(items < n ? (items < 1 ? 1 : items) : n);
}

template <int D, int NT, int KB>
cudaError_t launch_lse(const WeightParams& p, cudaStream_t st) {
  const int smem = weight_ring_off(D, NT * 8) + kWgtWarps * weight_stages<D, NT, KB>() * KeyStep<D, KB>::kBytes +
                   (2 * p.sh.B + 1) * 4;
  const cudaError_t e = set_smem_limit(reinterpret_cast<const void*>(page_lse_kernel<D, NT, KB>), smem);
  if (e != cudaSuccess) return e;
  return launch_chained(page_lse_kernel<D, NT, KB>, dim3((unsigned)p.n_ctas), dim3(kWgtThreads), (size_t)smem,
                        st, p);
}

template <int D>
cudaError_t launch_lse_d(const WeightParams& p, cudaStream_t st) {
  if (p.chunk == 8) return launch_lse<D, 1, 1>(p, st);
  if (p.sh.P == 16) switch (p.chunk / 8) {
      case 3: return launch_lse<D, 3, 1>(p, st);
      default: return launch_lse<D, 6, 1>(p, st);
    }
  switch (p.chunk / 8) {
    case 2: return launch_lse<D, 2, 2>(p, st);
    case 3: return launch_lse<D, 3, 2>(p, st);
    case 4: return launch_lse<D, 4, 2>(p, st);
    default: return launch_lse<D, 6, 2>(p, st);
  }
}

// Past two blocks an SM the third is worth more than the loads in flight (512 sequences
// 15.4 -> 14.1 us, on a slower machine 18.9 -> 14.0, where 8 would go from 9.8 to 10.2).
template <int W>
cudaError_t launch_evict(const EvictParams& p, int smem, cudaStream_t st) {
  const int sms = device_sms();
  const auto kernel = p.B > 2 * (sms > 0 ? sms : 148) ? evict_kernel<W, true> : evict_kernel<W, false>;
  const cudaError_t e = set_smem_limit(reinterpret_cast<const void*>(kernel), kEvPages * 12);
  if (e != cudaSuccess) return e;
  return launch_chained(kernel, dim3((unsigned)(p.B > 0 ? p.B : 1)), dim3(kEvThreads), (size_t)smem, st, p);
}

}  // namespace

extern "C" {

size_t nk_page_weights_workspace_bytes(int32_t B, int32_t T, int32_t num_q_heads, int32_t num_kv_heads,
                                       int32_t page_size, int32_t max_ctx) {
  if (B < 1 || T < 1 || T > NK_MAX_T || num_kv_heads < 1 || num_q_heads < num_kv_heads || page_size < 1 || max_ctx < 1)
    return 0;
  const int64_t items = (int64_t)B * num_kv_heads * (((int64_t)max_ctx + page_size - 1) / page_size);
  const WeightRows r = weight_rows(T, num_q_heads / num_kv_heads, page_size);
  const int64_t slots = weight_ctas(items, r) + (int64_t)B * num_kv_heads;
  return (size_t)(items * r.parts + slots * r.takes) * r.all() * 4;
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
  if (B > kMaxBatch || (int64_t)B * Hkv > 65535 || G > 48) return NK_ERR_UNSUPPORTED;
  const WeightRows r = weight_rows(T, G, P);
  const size_t need = nk_page_weights_workspace_bytes(B, T, num_q_heads, Hkv, P, max_ctx);
  if (!workspace_dev || workspace_bytes < need || !aligned_to(workspace_dev, 16)) return NK_ERR_WORKSPACE;
  const int64_t longest = ((int64_t)max_ctx + P - 1) / P, items = (int64_t)B * Hkv * longest;
  if (items * r.parts > 0x7fffffff) return NK_ERR_UNSUPPORTED;  // log-sums are numbered in 32 bits
  WeightParams p = {};
  p.pool = reinterpret_cast<const uint8_t*>(pool->base_dev);
  p.lay = ChunkLayout::make(P, D);
  p.num_pages = pool->num_pages;
  p.D = D;
  p.q = reinterpret_cast<const uint16_t*>(q_dev);
  p.bt = block_table_dev;
  p.ctx = ctx_lens_dev;
  p.sh = SplitShape{B, Hkv, P, T, max_ctx, max_pages_per_seq};
  p.G = G;
  p.rows = r.all();
  p.chunk = r.chunk;
  p.parts = r.parts;
  p.takes = r.takes;
  p.scale2 = sm_scale * kLog2e;
  p.n_ctas = weight_ctas(items, r);
  p.page_lse = reinterpret_cast<float*>(workspace_dev);
  p.seg_lse = p.page_lse + items * r.parts * p.rows;
  p.prior = prior_dev;
  p.seen = seen_dev;
  p.out = weights_dev;
  p.status = status_dev;
  const WaitLimits limits = wait_limits();
  p.wait_cycles = limits.cycles;
  p.withhold = limits.withhold;
  const cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  cudaError_t e = r.tc       ? launch_lse_tc(p, r.chunks, st)
                  : D == 256 ? launch_lse_d<256>(p, st)
                  : D == 128 ? launch_lse_d<128>(p, st)
                             : launch_lse_d<64>(p, st);
  if (e != cudaSuccess) return NK_ERR_CUDA;
  const int64_t units = (int64_t)B * Hkv;
  int64_t gx = (longest + kWsmThreads / 8 - 1) / (kWsmThreads / 8), most = 2048 / units;
  if (most < 1) most = 1;
  if (gx > most) gx = most;
  e = launch_chained(page_weight_kernel, dim3((unsigned)gx, (unsigned)units), dim3(kWsmThreads), (size_t)p.rows * 4, st,
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
  if (B > kMaxBatch || max_pages_per_seq > kEvPages) return NK_ERR_UNSUPPORTED;
  // (a batch of no sequences still tells that no page went)
  if (!num_freed_dev || (B > 0 && (!weights_dev || !block_table_dev || !out_table_dev || !ctx_lens_dev || !new_ctx_dev ||
                                   (max_freed > 0 && !freed_dev))))
    return NK_ERR_NULL;
  if (B > 0 && new_ctx_dev == ctx_lens_dev) return NK_ERR_SHAPE;  // every block reads the lengths while others write theirs
  const EvictParams p{weights_dev, num_pages, num_kv_heads, page_size, block_table_dev, out_table_dev,
                      max_pages_per_seq, ctx_lens_dev, B, keep_pages, sink_pages, recent_pages, new_ctx_dev, freed_dev,
                      max_freed, num_freed_dev, status_dev};
  const int smem = B > 0 ? (max_pages_per_seq + 1) / 2 * 2 * 12 : 16;
  const cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  // four or two weights a load where every page's lie aligned to as many
  const cudaError_t e = num_kv_heads % 4 == 0 && aligned_to(weights_dev, 16)  ? launch_evict<4>(p, smem, st)
                        : num_kv_heads % 2 == 0 && aligned_to(weights_dev, 8) ? launch_evict<2>(p, smem, st)
                                                                              : launch_evict<1>(p, smem, st);
  return e == cudaSuccess ? NK_OK : NK_ERR_CUDA;
}

}  // extern "C"
