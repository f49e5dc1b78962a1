// nk_weights_tc.cu -- the first kernel of nk_page_weights (nk_weights.cu) for
// many query rows: the scores on the 5th-generation tensor cores (tcgen05.mma,
// fp16 operands that hold the codes exactly, fp32 accumulators in tensor memory).
//
// A CTA takes up to 128 query rows of one (sequence, kv-head) after another
// against tiles of 64 keys: the rows are M, the keys N, and each 64-channel group
// has accumulators of its own (64 columns), because its scale is the key's. A row
// is one tensor-memory lane and one thread, which multiplies the groups' columns
// by the key's scales (read as one float4 that all lanes share), adds them, and
// forms the log-sum over the keys of the page: nothing is exchanged between
// threads. A page of more than 64 keys leaves several log-sums, pages of 16 or 32
// keys share a tile.
//
// 18 warps, one CTA per SM:
//   warps 0-7   two warpgroups that take the tiles in turn (each has one of the
//               two sets of accumulators), a thread a row;
//   warps 8-15  codes from the ring to fp16 in the swizzled operand buffer; at a
//               segment's start the unit's rows, scaled into the fp16 range;
//   warp 16     issues the MMAs;
//   warp 17     walks the list, looks up the pages, fills the rings with bulk
//               asynchronous copies (codes for the converters, scales for the
//               rows' threads).
// Every mbarrier wait is bounded; after one has run out nothing more is issued and
// no wait blocks.
#include <math.h>

#include "nk_ptx.cuh"
#include "nk_weights.cuh"

namespace nk {
namespace lse_tc {

constexpr int kKeys = 64;
constexpr int kRowsMost = 128;
constexpr int kSoft = 8, kConv = 8;
constexpr int kMmaWarp = kSoft + kConv, kCopyWarp = kMmaWarp + 1;
constexpr int kThreads = (kCopyWarp + 1) * 32;
constexpr int kRaw = 3, kScales = 4, kRowSets = 4;
constexpr int kCols = 512;

template <int D>
struct Smem {
  static constexpr int NG = D / kGroup;
  static constexpr int off_q = 0;                                   // [NG][128 rows][128 bytes], swizzled
  static constexpr int off_b = off_q + NG * kRowsMost * 128;        // [2][NG][64 keys][128 bytes], swizzled
  static constexpr int off_raw = off_b + 2 * NG * kKeys * 128;      // [kRaw][64][D]
  static constexpr int off_sc = off_raw + kRaw * kKeys * D;         // [kScales][64][NG]
  static constexpr int off_undo = off_sc + kScales * kKeys * NG * 4;  // [kRowSets][128]
  static constexpr int off_pre = off_undo + kRowSets * kRowsMost * 4;
  static constexpr int off_lens = off_pre + (kMaxBatch + 4) * 4;
  static constexpr int off_misc = off_lens + kMaxBatch * 4;         // barriers and the rest
  static constexpr int total = off_misc + 512 + 1024;
};

__host__ __device__ constexpr uint32_t idesc_f16(int M, int N) {
  return (1u << 4) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}
// K-major operand, 128-byte swizzle, atoms of 8 rows of 128 bytes, 1,024 bytes apart
__device__ __forceinline__ uint64_t desc_of(uint32_t addr) {
  return (uint64_t)((addr >> 4) & 0x3fff) | (uint64_t)1 << 16 |
         (uint64_t)((1024 >> 4) | (1u << 14) | (2u << 29)) << 32;
}
__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}\n" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
      : "memory");
}
__device__ __forceinline__ bool elect_one() {
  uint32_t ok;
  asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}\n" : "=r"(ok));
  return ok != 0;
}
__device__ __forceinline__ void mma_commit(uint32_t bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void fence_async() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

__device__ __forceinline__ void tm_ld16(uint32_t taddr, float (&v)[16]) {
  uint32_t r[16];
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr)
      : "memory");
#pragma unroll
  for (int i = 0; i < 16; ++i) v[i] = __uint_as_float(r[i]);
}

// The tiles of a segment: whole pages of up to 64 keys, or parts of longer ones.
struct Tiling {
  int P, parts, share;  // parts of a page; pages of a tile
  __device__ Tiling(int P_, int parts_) : P(P_), parts(parts_), share(P_ < kKeys ? kKeys / P_ : 1) {}
  __device__ int tiles(int pages) const { return parts > 1 ? pages * parts : (pages + share - 1) / share; }
  __device__ int page(int t) const { return parts > 1 ? t / parts : t * share; }
  __device__ int key(int t) const { return parts > 1 ? (t % parts) * kKeys : 0; }  // first key of the tile in its page
};

template <int D>
__global__ void __launch_bounds__(kThreads, 1) lse_tc_kernel(const __grid_constant__ WeightParams p) {
  using SM = Smem<D>;
  constexpr int NG = SM::NG;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  int* pre = reinterpret_cast<int*>(smem + SM::off_pre);
  int* lens = reinterpret_cast<int*>(smem + SM::off_lens);
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + SM::off_misc);
  int* tail = reinterpret_cast<int*>(smem + SM::off_misc + 256);
  int* warp_tot = tail;                                     // [18]
  volatile int* abort_flag = tail + 24;
  uint32_t* tslot = reinterpret_cast<uint32_t*>(tail + 25);
  int* none = tail + 28;                                    // [kScales]: pages of the tile that are none, a bit each
  const uint32_t bar0 = smem_u32(bars);
  // barriers
  const auto raw_full = [&](int i) { return bar0 + 8 * i; };
  const auto raw_empty = [&](int i) { return bar0 + 8 * (kRaw + i); };
  const auto sc_full = [&](int i) { return bar0 + 8 * (2 * kRaw + i); };
  const auto sc_empty = [&](int i) { return bar0 + 8 * (2 * kRaw + kScales + i); };
  constexpr int kB = 2 * kRaw + 2 * kScales;
  const auto b_full = [&](int i) { return bar0 + 8 * (kB + i); };
  const auto b_empty = [&](int i) { return bar0 + 8 * (kB + 2 + i); };
  const auto acc_full = [&](int i) { return bar0 + 8 * (kB + 4 + i); };
  const auto acc_empty = [&](int i) { return bar0 + 8 * (kB + 6 + i); };
  const auto rows_full = [&](int i) { return bar0 + 8 * (kB + 8 + i); };
  static_assert((kB + 8 + kRowSets) * 8 <= 256, "barriers");

  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (warp == 0) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tslot)), "r"(kCols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  if (tid == 32) {
    for (int i = 0; i < kRaw; ++i) {
      mbar_init(raw_full(i), 1);
      mbar_init(raw_empty(i), kConv);
    }
    for (int i = 0; i < kScales; ++i) {
      mbar_init(sc_full(i), 1);
      mbar_init(sc_empty(i), kSoft / 2);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(b_full(i), kConv);
      mbar_init(b_empty(i), 1);
      mbar_init(acc_full(i), 1);
      mbar_init(acc_empty(i), kSoft / 2);
    }
    for (int i = 0; i < kRowSets; ++i) mbar_init(rows_full(i), kConv);
    *abort_flag = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  chain_wait();
  chain_release();
  const SplitShape& sh = p.sh;
  const int P = sh.P, Hkv = sh.Hkv, T = sh.T, G = p.G, M = T * G;
  const int row0 = blockIdx.x * p.chunk;
  if (blockIdx.x == 0 && blockIdx.y == 0)
    for (int b = tid; b < sh.B; b += kThreads)
      if (pages_of_len(sh, p.ctx[b]) == 0) flag(p.status, NK_DEVFLAG_BAD_CTX);
  fence_before();
  block_page_prefix_short(sh, p.ctx, 0, pre, warp_tot, lens);  // (ends with a barrier)
  fence_after();
  const uint32_t tmem = *tslot;
  const int64_t W = (int64_t)pre[sh.B] * Hkv;
  const int cta = blockIdx.y;
  int64_t x = W > 0 ? cta_begin(W, p.n_ctas, cta) : 0;
  const int64_t x_end = W > 0 ? cta_begin(W, p.n_ctas, cta + 1) : 0;
  const Tiling tl(P, p.parts);
  const auto wait = [&](uint32_t bar, uint32_t parity) {  // by whole warps
    if (!*abort_flag && !mbar_wait(bar, parity)) {
      flag(p.status, NK_DEVFLAG_TIMEOUT);
      *abort_flag = 1;
    }
    __syncwarp();
  };
  int n = 0;  // tiles so far
  int segs = 0;
  Segment seg;

  if (warp < kSoft) {
    // ------------------------------------------------------------ rows
    const int wg = warp >> 2, row = (warp & 3) * 32 + lane;
    const bool act = (warp & 3) * 32 < p.chunk;  // (warp-uniform: some of its rows are there)
    const uint32_t acc = tmem + ((uint32_t)((warp & 3) * 32) << 16) + wg * NG * kKeys;
    int64_t item = x;
    while (next_segment(sh, pre, x, x_end, seg)) {
      const int L = lens[seg.b], pages = seg.page_end - seg.page_begin, tiles = tl.tiles(pages);
      wait(rows_full(segs % kRowSets), (uint32_t)(segs / kRowSets) & 1u);
      const float un = reinterpret_cast<const float*>(smem + SM::off_undo)[(segs % kRowSets) * kRowsMost + row];
      ++segs;
      const int pos = L - T + min(row0 + row, M - 1) / G;  // the last one that the row sees
      float ms = -INFINITY, ls = 0.f;
      for (int t = 0; t < tiles; ++t, ++n) {
        if ((n & 1) != wg) continue;
        const int sl = n % kScales, use = n >> 1;
        wait(sc_full(sl), (uint32_t)(n / kScales) & 1u);
        wait(acc_full(wg), (uint32_t)use & 1u);
        fence_after();
        if (act) {
          const int pg0 = tl.page(t), k0 = tl.key(t);
          const uint32_t gone = (uint32_t)none[sl];
          const float* scales = reinterpret_cast<const float*>(smem + SM::off_sc) + sl * kKeys * NG;
          float m = -INFINITY, l = 0.f;
          int pg = pg0, key = k0;  // page (of the segment) and first key of the block
          for (int blk = 0; blk < kKeys / 16; ++blk) {
            if (pg >= pages || pg >= pg0 + tl.share) break;
            const int logical = seg.page_begin + pg, base = logical * P + key;
            const bool live = base < L && !((gone >> (pg - pg0)) & 1u);
            if (live) {
              float v[NG][16];
#pragma unroll
              for (int c = 0; c < NG; ++c) tm_ld16(acc + c * kKeys + blk * 16, v[c]);
              wait_ld();
              float s[16];
#pragma unroll
              for (int i = 0; i < 16; ++i) {
                const float* f = scales + (blk * 16 + i) * NG;
                if constexpr (NG == 4) {
                  const float4 q = *reinterpret_cast<const float4*>(f);
                  s[i] = fmaf(q.w, v[3][i], fmaf(q.z, v[2][i], fmaf(q.y, v[1][i], q.x * v[0][i])));
                } else if constexpr (NG == 2) {
                  const float2 q = *reinterpret_cast<const float2*>(f);
                  s[i] = fmaf(q.y, v[1][i], q.x * v[0][i]);
                } else {
                  s[i] = f[0] * v[0][i];
                }
                s[i] *= un;
              }
              if (base + 15 > L - T) {
#pragma unroll
                for (int i = 0; i < 16; ++i)
                  if (base + i > pos) s[i] = -INFINITY;
              }
              float mx = m;
#pragma unroll
              for (int i = 0; i < 16; i += 2) mx = fmaxf(mx, fmaxf(s[i], s[i + 1]));
              const float u = mx == -INFINITY ? 0.f : mx;
              float s0 = l * wgt_ex2(m - u), s1 = 0.f;
#pragma unroll
              for (int i = 0; i < 16; i += 2) {
                s0 += wgt_ex2(s[i] - u);
                s1 += wgt_ex2(s[i + 1] - u);
              }
              l = s0 + s1;
              m = mx;
            }
            key += 16;
            if (key == P || key == k0 + kKeys) {  // the page's (or the part's) end
              if (row < p.chunk)
                p.page_lse[((item + pg) * p.parts + k0 / kKeys) * p.rows + row0 + row] = lse_of(m, l);
              lse_join(ms, ls, m, l);
              m = -INFINITY;
              l = 0.f;
              if (tl.parts > 1) break;
              key = 0;
              ++pg;
            }
          }
        }
        fence_before();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(acc_empty(wg));
          mbar_arrive(sc_empty(sl));
        }
      }
      if (row < p.chunk) p.seg_lse[(((int64_t)cta + seg.u) * 2 + wg) * p.rows + row0 + row] = lse_of(ms, ls);
      item += pages;
    }
  } else if (warp < kMmaWarp) {
    // ------------------------------------------------------------ codes to fp16
    const int cw = warp - kSoft;
    while (next_segment(sh, pre, x, x_end, seg)) {
      const int pages = seg.page_end - seg.page_begin, tiles = tl.tiles(pages);
      // the unit's rows, once every product over the last unit's is done
      if (n > 0) wait(b_empty((n - 1) & 1), (uint32_t)((n - 1) >> 1) & 1u);
      float* undo = reinterpret_cast<float*>(smem + SM::off_undo) + (segs % kRowSets) * kRowsMost;
      for (int r = cw; r < kRowsMost; r += kConv) {
        const int row = row0 + r, t = row / G, hg = row - t * G;
        const bool there = r < p.chunk && row < M;
        const uint16_t* src = p.q + (((int64_t)seg.b * T + t) * (G * Hkv) + seg.h * G + hg) * D;
        constexpr int PER = D / 64;
        uint32_t w[PER];
        float m = 0.f;
#pragma unroll
        for (int i = 0; i < PER; ++i) {
          w[i] = there ? reinterpret_cast<const uint32_t*>(src)[lane + 32 * i] : 0u;
          m = fmaxf(m, fmaxf(fabsf(bf16_lo(w[i])), fabsf(bf16_hi(w[i]))));
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
        const int e = wgt_row_exp(m);
        const float up = wgt_pow2(e);
#pragma unroll
        for (int i = 0; i < PER; ++i) {  // word lane + 32 i: channels 2 lane + 64 i, + 1, so group i
          const __half2 hh = __floats2half2_rn(bf16_lo(w[i]) * up, bf16_hi(w[i]) * up);
          *reinterpret_cast<uint32_t*>(smem + SM::off_q + i * (kRowsMost * 128) + r * 128 +
                                       (((lane >> 2) ^ (r & 7)) << 4) + (lane & 3) * 4) =
              *reinterpret_cast<const uint32_t*>(&hh);
        }
        if (lane == 0) undo[r] = p.scale2 * wgt_pow2(-e);
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(rows_full(segs % kRowSets));
      ++segs;
      for (int t = 0; t < tiles; ++t, ++n) {
        const int rs = n % kRaw, buf = n & 1;
        wait(raw_full(rs), (uint32_t)(n / kRaw) & 1u);
        if (n >= 2) wait(b_empty(buf), (uint32_t)((n >> 1) - 1) & 1u);
        const uint8_t* raw = smem + SM::off_raw + rs * (kKeys * D);
        uint8_t* dst = smem + SM::off_b + buf * (NG * kKeys * 128);
        constexpr int PCS = D / 16;  // 16-code pieces of a key
#pragma unroll 4
        for (int i = cw * 32 + lane; i < kKeys * PCS; i += kConv * 32) {
          const int key = i / PCS, j = i % PCS;
          const uint4 w = *reinterpret_cast<const uint4*>(raw + i * 16);
          const uint32_t u[4] = {w.x ^ 0x80808080u, w.y ^ 0x80808080u, w.z ^ 0x80808080u, w.w ^ 0x80808080u};
          uint4 c0, c1;  // channels 16 j .. 16 j + 7, + 8 .. 15
          c0.x = wgt_f16(u[0], 0x4140), c0.y = wgt_f16(u[0], 0x4342), c0.z = wgt_f16(u[1], 0x4140), c0.w = wgt_f16(u[1], 0x4342);
          c1.x = wgt_f16(u[2], 0x4140), c1.y = wgt_f16(u[2], 0x4342), c1.z = wgt_f16(u[3], 0x4140), c1.w = wgt_f16(u[3], 0x4342);
          uint8_t* row = dst + (j >> 2) * (kKeys * 128) + key * 128;
          const int ch = 2 * (j & 3), sw = key & 7;
          // eight lanes store at once: those of odd groups their second half first, so
          // that the eight fall on distinct banks
          const bool flip = (j >> 2) & 1;
          *reinterpret_cast<uint4*>(row + (((ch + (flip ? 1 : 0)) ^ sw) << 4)) = flip ? c1 : c0;
          *reinterpret_cast<uint4*>(row + (((ch + (flip ? 0 : 1)) ^ sw) << 4)) = flip ? c0 : c1;
        }
        fence_async();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(b_full(buf));
          mbar_arrive(raw_empty(rs));
        }
      }
    }
  } else if (warp == kMmaWarp) {
    // ------------------------------------------------------------ products
    constexpr uint32_t id = idesc_f16(kRowsMost, kKeys);
    int done[2] = {0, 0};  // commits of each set
    const uint64_t qa = desc_of(smem_u32(smem + SM::off_q)), kb = desc_of(smem_u32(smem + SM::off_b));
    while (next_segment(sh, pre, x, x_end, seg)) {
      const int tiles = tl.tiles(seg.page_end - seg.page_begin);
      for (int t = 0; t < tiles; ++t, ++n) {
        const int buf = n & 1;
        wait(b_full(buf), (uint32_t)(n >> 1) & 1u);
        if (n >= 2) wait(acc_empty(buf), (uint32_t)((n >> 1) - 1) & 1u);
        if (__any_sync(0xffffffffu, *abort_flag != 0)) continue;
        ++done[buf];
        fence_after();
        if (elect_one()) {
#pragma unroll
          for (int c = 0; c < NG; ++c)
#pragma unroll
            for (int k = 0; k < 4; ++k)
              mma_ss(tmem + buf * NG * kKeys + c * kKeys, qa + ((c * kRowsMost * 128 + k * 32) >> 4),
                     kb + ((buf * NG * kKeys * 128 + c * kKeys * 128 + k * 32) >> 4), id, k > 0 ? 1u : 0u);
          mma_commit(b_empty(buf));
          mma_commit(acc_full(buf));
        }
        __syncwarp();
      }
    }
    // after a wait that ran out products may still be under way: they end before tensor memory is given back
    if (*abort_flag)
      for (int i = 0; i < 2; ++i)
        if (done[i] > 0) (void)mbar_wait(b_empty(i), (uint32_t)(done[i] - 1) & 1u);
  } else {
    // ------------------------------------------------------------ copies
    while (next_segment(sh, pre, x, x_end, seg)) {
      const int L = lens[seg.b], pages = seg.page_end - seg.page_begin, tiles = tl.tiles(pages);
      const int32_t* bt = p.bt + (int64_t)seg.b * sh.max_pages + seg.page_begin;
      // page ids of 32 pages of the segment, and the next 32
      int have = 0, ids = lane < pages ? bt[lane] : -1, ids2 = 32 + lane < pages ? bt[32 + lane] : -1;
      for (int t = 0; t < tiles; ++t, ++n) {
        const int pg0 = tl.page(t), k0 = tl.key(t), rs = n % kRaw, sl = n % kScales;
        if (n >= kRaw) wait(raw_empty(rs), (uint32_t)(n / kRaw - 1) & 1u);
        if (n >= kScales) wait(sc_empty(sl), (uint32_t)(n / kScales - 1) & 1u);
        // lane i < share: page pg0 + i
        if (pg0 - have >= 32) {
          have += 32;
          ids = ids2;
          ids2 = have + 32 + lane < pages ? bt[have + 32 + lane] : -1;
        }
        // (32 is a whole number of a tile's pages: 4, 2 or 1)
        const int id = __shfl_sync(0xffffffffu, ids, (pg0 - have + lane) & 31);
        const bool mine = lane < tl.share && pg0 + lane < pages;
        const bool bad = mine && (id < 0 || id >= p.num_pages);
        if (bad) flag(p.status, NK_DEVFLAG_BAD_PAGE);
        const uint32_t gone = __ballot_sync(0xffffffffu, bad);
        const int live = mine && !bad ? min(min(P - k0, kKeys), L - (seg.page_begin + pg0 + lane) * P - k0) : 0;
        const int keys = live > 0 ? (live + 15) / 16 * 16 : 0;
        int all = keys;
#pragma unroll
        for (int o = 1; o < 4; o <<= 1) all += __shfl_xor_sync(0xffffffffu, all, o);
        all = __shfl_sync(0xffffffffu, all, 0);
        const bool go = !__any_sync(0xffffffffu, *abort_flag != 0);
        if (lane == 0) {
          none[sl] = (int)gone;
          if (go && all > 0) {
            mbar_arrive_expect_tx(raw_full(rs), all * D);
            mbar_arrive_expect_tx(sc_full(sl), all * NG * 4);
          } else {
            mbar_arrive(raw_full(rs));
            mbar_arrive(sc_full(sl));
          }
        }
        __syncwarp();
        if (go && keys > 0) {
          const uint8_t* chunk = p.pool + ((int64_t)id * Hkv + seg.h) * p.lay.chunk;
          const int at = lane * P;  // (lane 0 alone where pages have parts)
          bulk_load(smem_u32(smem + SM::off_raw + rs * (kKeys * D) + at * D), chunk + (int64_t)k0 * D, keys * D, raw_full(rs));
          bulk_load(smem_u32(smem + SM::off_sc + (sl * kKeys + at) * NG * 4), chunk + p.lay.ks + k0 * NG * 4, keys * NG * 4,
                    sc_full(sl));
        }
        __syncwarp();
      }
    }
    // after a wait that ran out some copies may still be in flight: they land before the CTA ends
    if (*abort_flag) {
      for (int i = max(0, n - kRaw); i < n; ++i) (void)mbar_wait(raw_full(i % kRaw), (uint32_t)(i / kRaw) & 1u);
      for (int i = max(0, n - kScales); i < n; ++i)
        (void)mbar_wait(sc_full(i % kScales), (uint32_t)(i / kScales) & 1u);
    }
  }
  fence_before();
  __syncthreads();
  fence_after();
  if (warp == 0) {
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kCols) : "memory");
  }
}

template <int D>
static cudaError_t launch(const WeightParams& p, int chunks, cudaStream_t st) {
  const cudaError_t e = set_smem_limit(reinterpret_cast<const void*>(lse_tc_kernel<D>), Smem<D>::total);
  if (e != cudaSuccess) return e;
  return launch_chained(lse_tc_kernel<D>, dim3((unsigned)chunks, (unsigned)p.n_ctas), dim3(kThreads),
                        (size_t)Smem<D>::total, st, p);
}

}  // namespace lse_tc

cudaError_t launch_lse_tc(const WeightParams& p, int chunks, cudaStream_t st) {
  if (p.D == 256) return lse_tc::launch<256>(p, chunks, st);
  if (p.D == 128) return lse_tc::launch<128>(p, chunks, st);
  return lse_tc::launch<64>(p, chunks, st);
}

}  // namespace nk
